// Eviction from a paged cache by accumulated attention weight, and the move of
// cache rows that it (and the acceptance of drafted tokens) needs (sm_103a).
//
// What it computes: of a request's L > budget cached tokens stay the first F, the
// last W and, of those between, the budget - F - W of largest weight (equal
// weights: the earlier token; a NaN weighs less than any number).  The kept
// tokens t_0 < t_1 < ... become tokens 0, 1, ... of the request, K, V and weights
// alike, so that the order of positions, and with it the first/last window of
// the attention calls, keeps its meaning.
//
//  * select_kernel -- one cluster per (request, weight head), each CTA a stretch of
//    the tokens: the threshold weight by radix selection over the order-preserving
//    integer form of the weights, then an ordered pass that lists the kept tokens.
//  * move_kernel -- moves K / V rows and weights.  The sources are increasing and
//    src[j] >= base + j, so a CTA that moves a column slice of the rows in order,
//    each batch read before it is written, never overwrites a row still to be
//    read: a slot in a batch's destination range is either no source or the source
//    of that batch or an earlier one.  So later batches may be read ahead (a ring of
//    cp.async copies), and slices (a head, K or V, and a part of its dimensions) are
//    independent, which gives the parallelism.
#include <cooperative_groups.h>

#include <type_traits>

#include "common.cuh"
#include "evict.h"

namespace attn {
namespace evict {

namespace cg = cooperative_groups;

// ---------------------------------------------------------------------------
// Selection.

constexpr int kSelThreads = 512;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kBins = 2048;
constexpr int kRound = 16384;                     // tokens whose keys a CTA holds at once
constexpr int kMaxCluster = 8;

// Unsigned integers in the order of the weights: NaN lowest (1), -0 equal to +0.
// 0xffffffff is no weight's: it stands for a token that stays in any case.
constexpr uint32_t kStays = 0xffffffffu;
__device__ __forceinline__ uint32_t order_key(float w) {
    const uint32_t u = __float_as_uint(w + 0.f);
    return w != w ? 1u : u ^ ((uint32_t)((int)u >> 31) | 0x80000000u);
}

__device__ __forceinline__ uint32_t warp_scan(uint32_t x, int lane) {  // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t v = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += v;
    }
    return x;
}

// Exclusive prefix sum of x over the CTA, and the CTA's total.  `scratch`: kSelWarps
// words that nobody uses before the next __syncthreads.
__device__ __forceinline__ uint32_t block_scan(uint32_t x, uint32_t* scratch, uint32_t& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t inc = warp_scan(x, lane);
    if (lane == 31) scratch[warp] = inc;
    __syncthreads();
    const uint32_t v = lane < kSelWarps ? scratch[lane] : 0u;
    total = __reduce_add_sync(0xffffffffu, v);
    return inc - x + __reduce_add_sync(0xffffffffu, lane < warp ? v : 0u);
}

// Three digits of the key, 11 + 11 + 10 bits, narrow the `need`-th largest weight
// down; the CTAs of the cluster add their histograms up through distributed shared
// memory.  A CTA takes its stretch of tokens in rounds of 16384, whose keys stay in
// shared memory.  With one round the weights are read once: up to 131072 tokens while a
// cluster of 8 is given to each list (at most 19 lists), down to 16384 where the lists
// fill the GPU by themselves (more than 76).  With more, every digit and the ordered pass
// load all rounds again, one after the other.  For the ordered pass a thread owns a run of
// consecutive tokens (an odd number, so that a warp's reads fall into different banks); a
// scan of the runs' kept counts gives every kept token its rank, and the list leaves
// through shared memory.
// It is bound by the latency of its steps: 256 lists of 8k to 16k tokens take 22 us, one
// of 2k 6.8 us.  (24 us with ballots over 32 tokens at a time, with keys in registers or
// not, and with a list of the candidates after the first digit.)  256 lists of 16384
// tokens take 24 us, of 16385 (two rounds) 41, of 65536 124.
__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs p, int capacity) {
    extern __shared__ uint32_t keys[];  // of a round, `capacity`; then the kept tokens of a round as 16-bit offsets
    __shared__ __align__(16) uint32_t hist[2][kBins];  // read four bins at a time
    __shared__ uint32_t warp_sum[4][kSelWarps];
    __shared__ uint32_t s_prefix, s_rank, s_ties, s_totals[2];
    __shared__ int s_first;
    cg::cluster_group cl = cg::this_cluster();
    const int parts = cl.num_blocks(), part = cl.block_rank();
    auto sync = [&]() {
        if (parts > 1)
            cl.sync();
        else
            __syncthreads();
    };
    const int head = blockIdx.x / parts, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31;
    const size_t at = (size_t)b * p.heads + head;
    const float* w = p.weights + at * p.cap;
    int32_t* kept = p.kept + at * p.budget;

    int L = p.seqlens[b];
    const int cap = (int)min((long long)p.cap, p.token_cap);
    if (L > cap || L < 0) {
        if (tid == 0 && part == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        L = max(0, min(L, cap));
    }
    const int n = min(L, p.budget);
    if (tid == 0 && part == 0 && head == 0) p.new_seqlens[b] = n;
    if (L <= p.budget) {  // the same for the whole cluster
        for (uint32_t t = part * kSelThreads + tid; t < (uint32_t)p.budget; t += parts * kSelThreads)
            kept[t] = t < (uint32_t)L ? (int)t : -1;
        if (tid == 0 && part == 0) p.first_moved[at] = n;
        return;
    }
    const int lo = p.keep_first, hi = L - p.keep_last;  // the tokens that compete
    const int need = p.budget - p.keep_first - p.keep_last;
    const int stretch = (L + parts - 1) / parts;
    const int a0 = min(part * stretch, L), a1 = min(a0 + stretch, L);  // this CTA's tokens
    const int rounds = max(1, (a1 - a0 + kRound - 1) / kRound);

    uint16_t* const offsets = reinterpret_cast<uint16_t*>(keys + capacity);
    int r0 = 0, len = 0;  // of a round: first token, tokens
    auto load = [&](int round) {
        __syncthreads();  // the previous round's keys have been read
        r0 = a0 + round * kRound;
        len = min(kRound, a1 - r0);
        for (int k = tid; k < len; k += kSelThreads)
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(keys + k)), "l"(w + r0 + k)
                         : "memory");
        asm volatile("cp.async.wait_all;" ::: "memory");
#pragma unroll 4
        for (int k = tid; k < len; k += kSelThreads) {
            const int t = r0 + k;
            keys[k] = t < lo || t >= hi ? kStays : order_key(__uint_as_float(keys[k]));
        }
        __syncthreads();
    };
    // The threshold key, how many tokens at it stay, and whether that is all of them.
    // need = 0: the sentinel kStays alone is kept.
    uint32_t prefix = need > 0 ? 0u : kStays, rank = need > 0 ? (uint32_t)need : 0xffffffffu;
    bool all_ties = true;
    if (tid == 0) s_first = n;
    if (tid < 2) s_totals[tid] = 0;
    for (int i = tid; i < kBins; i += kSelThreads) hist[0][i] = 0;
    load(0);
    if (need > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024u : 2048u;
            const uint32_t known = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
            uint32_t* h = hist[pass & 1];
            // in the first pass kStays falls into the last bin, alone
            for (int round = 0; round < rounds; ++round) {
                if (rounds > 1) load(round);
#pragma unroll 4
                for (int i = tid; i < len; i += kSelThreads) {
                    const uint32_t k = keys[i];
                    if ((k & known) == prefix) atomicAdd(&h[(k >> shift) & (bins - 1)], 1u);
                }
            }
            // the next pass's histogram (read by nobody since the pass before)
            for (int i = tid; i < kBins; i += kSelThreads) hist[(pass + 1) & 1][i] = 0;
            sync();
            // Suffix sums from the largest digit: thread i owns digits bins-1-4i and the
            // next three.
            const int d0 = (int)bins - 1 - 4 * tid;
            uint32_t c[4] = {0u, 0u, 0u, 0u};
            if (d0 >= 0) {
                if (parts == 1) {
                    const uint4 x = *reinterpret_cast<const uint4*>(h + d0 - 3);
                    c[0] = x.w, c[1] = x.z, c[2] = x.y, c[3] = x.x;
                } else {
                    uint4 x[kMaxCluster];
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q)
                        x[q] = q < parts ? *reinterpret_cast<const uint4*>(cl.map_shared_rank(h, q) + d0 - 3)
                                         : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                    for (int q = 0; q < kMaxCluster; ++q)
                        c[0] += x[q].w, c[1] += x[q].z, c[2] += x[q].y, c[3] += x[q].x;
                }
            }
            if (pass == 0 && tid == 0) c[0] = 0;
            const uint32_t sum = c[0] + c[1] + c[2] + c[3];
            uint32_t total, before = block_scan(sum, warp_sum[pass & 1], total);
            if (before < rank && rank <= before + sum) {
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    if (before < rank && rank <= before + c[k]) {
                        s_prefix = prefix | ((uint32_t)(d0 - k) << shift);
                        s_rank = rank - before;
                        s_ties = c[k];
                    }
                    before += c[k];
                }
            }
            // everyone has read this histogram before it is cleared again
            sync();
            prefix = s_prefix;
            rank = s_rank;
        }
        all_ties = s_ties == rank;
    }
    // Kept: protected, above the threshold, or one of the first `rank` tokens at it.
    int run0 = 0, run1 = 0;   // this thread's run of the round's tokens
    uint32_t nk = 0, nt = 0;  // of it: kept or at the threshold; at it
    int first = n;            // the first token that is dropped: the first rank that is not its own token
    auto count = [&]() {
        const int per = (len + kSelThreads - 1) / kSelThreads | 1;
        run0 = min(tid * per, len);
        run1 = min(run0 + per, len);
        nk = nt = 0;
#pragma unroll 4
        for (int i = run0; i < run1; ++i) {
            const uint32_t k = keys[i];
            nk += k >= prefix;
            nt += k == prefix;
            if (k < prefix) first = min(first, r0 + i);
        }
    };
    uint32_t out = 0, base_tie = 0;  // before this round: kept tokens, tokens at the threshold
    if (parts > 1) {                 // those of the earlier stretches
        for (int round = 0; round < rounds; ++round) {
            if (rounds > 1) load(round);
            count();
            const uint32_t ws = __reduce_add_sync(0xffffffffu, nk - nt), wt = __reduce_add_sync(0xffffffffu, nt);
            if (lane == 0) {
                atomicAdd(&s_totals[0], ws);
                atomicAdd(&s_totals[1], wt);
            }
        }
        sync();
#pragma unroll
        for (int q = 0; q < kMaxCluster; ++q) {
            if (q >= part) break;
            const uint32_t* tq = cl.map_shared_rank(s_totals, q);
            out += tq[0];
            base_tie += tq[1];
        }
        out += min(base_tie, rank);
    }
    for (int round = 0; round < rounds; ++round) {
        if (rounds > 1) load(round);
        if (rounds > 1 || parts == 1) count();
        __syncthreads();  // offsets and warp_sum have been read
        uint32_t tie = 0, ties = 0, kept_n;
        if (!all_ties) {  // of the run's ties stay those that are among the first `rank`
            tie = base_tie + block_scan(nt, warp_sum[2], ties);
            nk -= nt - min(nt, rank - min(rank, tie));
        }
        uint32_t pos = block_scan(nk, warp_sum[3], kept_n);
#pragma unroll 4
        for (int i = run0; i < run1; ++i) {
            const uint32_t k = keys[i];
            bool keep = k >= prefix;
            if (!all_ties && k == prefix) {
                keep = tie++ < rank;
                if (!keep) first = min(first, r0 + i);
            }
            if (keep) offsets[pos++] = (uint16_t)i;
        }
        __syncthreads();
#pragma unroll 4
        for (uint32_t i = tid; i < kept_n; i += kSelThreads) kept[out + i] = r0 + offsets[i];
        out += kept_n;
        base_tie += ties;
    }
    // first_moved: the least over the cluster (no CTA leaves while its shared memory is in use)
    first = __reduce_min_sync(0xffffffffu, first);
    if (lane == 0 && first < n) atomicMin(parts > 1 ? cl.map_shared_rank(&s_first, 0) : &s_first, first);
    sync();
    if (part == 0 && tid == 0) p.first_moved[at] = s_first;
}

// ---------------------------------------------------------------------------
// Moves.

constexpr int kMoveThreads = 256;
// kBatch rows per thread and batch, kStages batches in flight.
template <int kBatch, int kStages>
constexpr int kMoveSmem = kStages * kBatch * kMoveThreads * (16 + 4);

__device__ __forceinline__ void cp_async_16(void* dst, const void* src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// The kept tokens' weights, in order, and zeros behind them.
__device__ __forceinline__ void move_weights(const float* w, float* wo, const int32_t* src, int n, int cap) {
    constexpr int kB = 8;
    for (int j0 = 0; j0 < n; j0 += kB * kMoveThreads) {
        float x[kB];
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int j = j0 + i * kMoveThreads + (int)threadIdx.x;
            x[i] = j < n ? w[src[j]] : 0.f;
        }
        __syncthreads();  // all of the batch is read before any of it is written
#pragma unroll
        for (int i = 0; i < kB; ++i) {
            const int j = j0 + i * kMoveThreads + (int)threadIdx.x;
            if (j < n) wo[j] = x[i];
        }
    }
    for (uint32_t t = n + threadIdx.x; t < (uint32_t)cap; t += kMoveThreads) wo[t] = 0.f;
}

// It is bound by memory.  32 requests brought from 8k - 16k tokens to 4096 (8 KV heads
// of 128, each keeping tokens of its own: 1.1 GB read and written) take 181 us, a plain
// copy of as many bytes 182 us.  The first form (loads into registers, two barriers a
// batch, pages looked up when they were needed) took 266 us.
// Grid (column slices, heads * {K, V} and then heads for the weights, requests).  A
// slice is `lanes` 16-byte columns of one head group's part of a token row.
template <bool kCheck, int kBatch, int kStages>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveArgs p, int lanes, int head_bytes, int row_bytes,
                                                            int page_shift) {
    extern __shared__ uint4 ring[];  // [stage][batch][thread] rows, then their destination slots
    int* const dest = reinterpret_cast<int*>(ring + kStages * kBatch * kMoveThreads);
    const int b = blockIdx.z, tid = threadIdx.x;
    const bool is_weights = (int)blockIdx.y >= 2 * p.heads;
    const int head = is_weights ? (int)blockIdx.y - 2 * p.heads : (int)blockIdx.y >> 1;
    const size_t at = (size_t)b * p.heads + head;
    const int32_t* src = p.src + at * p.max_rows;
    int n = p.counts[b];
    const int base = p.base ? p.base[b] : 0;
    const int tokens = p.max_pages * p.page_size;  // that the page table holds
    if (n > p.max_rows || n < 0 || base < 0 || n > tokens - base) {
        if (tid == 0 && blockIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        n = base < 0 ? 0 : max(0, min(min(n, p.max_rows), tokens - base));
    }
    if (is_weights) {
        if (blockIdx.x == 0) move_weights(p.weights + at * p.cap, p.weights_out + at * p.cap, src, n, p.cap);
        return;
    }
    char* const cache = reinterpret_cast<char*>((blockIdx.y & 1) ? p.v_cache : p.k_cache);
    const int32_t* table = p.page_table + (size_t)b * p.max_pages;
    const int col = tid % lanes, sub = tid / lanes, step = kMoveThreads / lanes;
    const size_t off = (size_t)head * head_bytes + ((size_t)blockIdx.x * lanes + col) * 16;
    const int j0 = p.first_moved ? p.first_moved[at] : 0;
    const int rows = kBatch * step;  // of a batch
    const int batches = n > j0 ? (n - j0 + rows - 1) / rows : 0;
    // Software pipeline over batches: the sources of batch c + 2 are requested
    // while the pages of batch c + 1 are and the rows of batch c are, so that each
    // of the three dependent loads has an iteration to arrive.
    int t[kBatch], t_prev[kBatch];             // source token, -1: none; the one before it (kCheck)
    int from[kBatch], to[kBatch];          // page ids
    int from_at[kBatch], to_at[kBatch];    // rows in the pages, from_at -1: nothing to move
    auto sources = [&](int c) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int j = j0 + c * rows + i * step + sub;
            const bool in = c < batches && j < n;
            t[i] = in ? src[j] : -1;
            if constexpr (kCheck) t_prev[i] = in && j > 0 ? src[j - 1] : -1;
        }
    };
    auto page_of = [&](int token, int& row) -> int {
        const int pg = page_shift >= 0 ? token >> page_shift : token / p.page_size;
        row = token - pg * p.page_size;
        if (pg < p.max_pages) return table[pg];
        raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        return -2;
    };
    auto pages = [&](int c) {  // of the batch whose sources were requested last
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int token = base + j0 + c * rows + i * step + sub;
            from_at[i] = -1;
            if constexpr (kCheck) {
                const bool in = c < batches && token - base < n;
                if (in && (t[i] < token || t_prev[i] >= t[i])) {
                    raise_status(ATTN_SINK_DEV_ORDER);
                    continue;
                }
            }
            if (t[i] < 0 || t[i] == token) continue;
            from[i] = page_of(t[i], from_at[i]);
            to[i] = page_of(token, to_at[i]);
        }
    };
    auto read = [&](int c) {  // the batch whose pages were requested last
        const int at_stage = c % kStages * kBatch * kMoveThreads + tid;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            int slot = -1;
            if (c < batches && from_at[i] >= 0) {
                const bool ok = (unsigned)from[i] < (unsigned)p.num_pages && (unsigned)to[i] < (unsigned)p.num_pages;
                if (ok) {
                    slot = to[i] * p.page_size + to_at[i];
                    cp_async_16(&ring[at_stage + i * kMoveThreads],
                                cache + ((size_t)from[i] * p.page_size + from_at[i]) * row_bytes + off);
                } else if (from[i] != -2 && to[i] != -2) {
                    raise_status(ATTN_SINK_DEV_PAGE_OOB);
                }
            }
            dest[at_stage + i * kMoveThreads] = slot;
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    sources(0);
    pages(0);
    sources(1);
    for (int c = 0; c < kStages - 1; ++c) {
        read(c);
        pages(c + 1);
        sources(c + 2);
    }
    for (int c = 0; c < batches; ++c) {
        read(c + kStages - 1);
        pages(c + kStages);
        sources(c + kStages + 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
        __syncthreads();  // every thread has this batch's rows
        const int at_stage = c % kStages * kBatch * kMoveThreads + tid;
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int slot = dest[at_stage + i * kMoveThreads];
            if (slot >= 0)
                *reinterpret_cast<uint4*>(cache + (size_t)slot * row_bytes + off) = ring[at_stage + i * kMoveThreads];
        }
    }
}

// ---------------------------------------------------------------------------
// Host side.

constexpr int kPlainSmem = 24 * 1024;  // dynamic, beside the static part, that a launch may have without asking

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    // Several CTAs per (request, head) while the GPU has SMs left and each has 8192
    // tokens or more: adding the histograms up over a cluster costs about as much as
    // 8192 tokens do (2 us a digit).
    const long long cap = a.cap < a.token_cap ? a.cap : a.token_cap;
    int parts = 1;
    while (parts < kMaxCluster && (long long)a.batch * a.heads * parts * 2 <= num_sms() && cap / (2 * parts) >= 8192)
        parts *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.heads * parts), a.batch);
    cfg.blockDim = dim3(kSelThreads);
    cfg.stream = s;
    const long long stretch = (cap + parts - 1) / parts;
    const int capacity = (int)(stretch < kRound ? stretch : kRound);
    cfg.dynamicSmemBytes = (size_t)capacity * 6;  // keys and offsets
    if (cfg.dynamicSmemBytes > kPlainSmem) {
        cudaError_t e = cudaFuncSetAttribute(select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kRound * 6);
        if (e != cudaSuccess) return e;
    }
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, select_kernel, a, capacity);
}

cudaError_t launch_move(const MoveArgs& a, cudaStream_t s) {
    if (a.batch == 0 || a.max_rows == 0) return cudaSuccess;
    const int row_bytes = a.hkv * a.head_dim * 2;
    const int head_bytes = row_bytes / a.heads;
    // Slices: the widest that divides a head group's row, narrower only while there
    // are fewer than two CTAs per SM (1.1 GB moved: 32-byte slices 222 us, 64 189 us, 256
    // 181 us; one request of 100k tokens: 32 88 us, 64 173 us, 256 700 us).
    int lanes = 1;
    while (lanes < 128 && head_bytes % (32 * lanes) == 0) lanes *= 2;
    while (lanes > 2 && (long long)head_bytes / (16 * lanes) * a.heads * 2 * a.batch < 2 * num_sms()) lanes /= 2;
    int page_shift = -1;
    for (int sh = 0; sh < 31; ++sh)
        if ((1 << sh) == a.page_size) page_shift = sh;
    const dim3 grid(head_bytes / (16 * lanes), a.heads * (a.weights ? 3 : 2), a.batch);
    auto launch = [&](auto kernel, int smem) {
        if (smem > kPlainSmem) {
            cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
        }
        kernel<<<grid, kMoveThreads, smem, s>>>(a, lanes, head_bytes, row_bytes, page_shift);
        return cudaGetLastError();
    };
    // Few rows (an accepted draft): one batch.  Few CTAs: larger batches, since a
    // batch costs about a microsecond whatever its size (160 KB of shared memory, one
    // CTA per SM; 80 KB, two).  Otherwise 40 KB, five per SM.
    const long long ctas = (long long)grid.x * grid.y * grid.z;
    auto choose = [&](auto check) {
        constexpr bool kC = decltype(check)::value;
        if (a.max_rows <= 2 * (kMoveThreads / lanes)) return launch(move_kernel<kC, 2, 2>, kMoveSmem<2, 2>);
        if (ctas <= num_sms()) return launch(move_kernel<kC, 8, 4>, kMoveSmem<8, 4>);
        if (ctas <= 2 * num_sms()) return launch(move_kernel<kC, 4, 4>, kMoveSmem<4, 4>);
        return launch(move_kernel<kC, 2, 4>, kMoveSmem<2, 4>);
    };
    return a.first_moved ? choose(std::false_type{}) : choose(std::true_type{});
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace evict
}  // namespace attn
