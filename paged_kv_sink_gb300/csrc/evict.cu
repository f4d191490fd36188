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
//  * select_kernel -- one block per (request, weight head): the threshold weight
//    by radix selection over the order-preserving integer form of the weights,
//    then one ordered pass that lists the kept tokens and moves their weights.
//  * move_kernel -- moves K / V rows.  The sources are increasing and src[j] >=
//    base + j, so a block that moves a column slice of the rows in order, each
//    batch read before it is written, never overwrites a row still to be read:
//    a slot in a batch's destination range is either no source or the source of
//    that batch or an earlier one.  Slices (a head, K or V, and 32 bytes of it or
//    more) are independent, and give the parallelism.
#include "common.cuh"
#include "evict.h"

namespace attn {
namespace evict {

// ---------------------------------------------------------------------------
// Selection.

constexpr int kSelThreads = 1024;
constexpr int kBins = 2048;

// Unsigned integers in the order of the weights: NaN lowest, -0 equal to +0.
__device__ __forceinline__ uint32_t order_key(float w) {
    if (w != w) return 0u;
    const uint32_t u = __float_as_uint(w + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__global__ void __launch_bounds__(kSelThreads) select_kernel(const SelectArgs p) {
    __shared__ uint32_t hist[kBins];
    __shared__ uint32_t warp_sum[32];
    __shared__ uint32_t s_prefix, s_rank;
    __shared__ int s_first;
    const int head = blockIdx.x, b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const size_t at = (size_t)b * p.heads + head;
    const float* w = p.weights + at * p.cap;
    float* wo = p.weights_out + at * p.cap;
    int32_t* kept = p.kept + at * p.budget;

    int L = p.seqlens[b];
    const int cap = (int)min((long long)p.cap, p.token_cap);
    if (L > cap || L < 0) {
        if (tid == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        L = max(0, min(L, cap));
    }
    const int n = min(L, p.budget);
    if (tid == 0) {
        s_first = n;
        if (head == 0) p.new_seqlens[b] = n;
    }
    if (L <= p.budget) {
        for (int t = tid; t < p.budget; t += kSelThreads) kept[t] = t < L ? t : -1;
        for (int t = tid; t < p.cap; t += kSelThreads) {
            if (t >= L) wo[t] = 0.f;
            else if (wo != w) wo[t] = w[t];
        }
        if (tid == 0) p.first_moved[at] = n;
        return;
    }
    // The `need`-th largest of the middle tokens [lo, hi): three digits of the key.
    const int lo = p.keep_first, hi = L - p.keep_last;
    const int need = p.budget - p.keep_first - p.keep_last;
    uint32_t prefix = 0, rank = (uint32_t)need;  // rank-th largest among keys with this prefix
    if (need > 0) {
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
            const uint32_t bins = pass == 2 ? 1024u : 2048u;
            for (int i = tid; i < kBins; i += kSelThreads) hist[i] = 0;
            __syncthreads();
            const uint32_t known = pass == 0 ? 0u : 0xffffffffu << (pass == 1 ? 21 : 10);
            for (int t = lo + tid; t < hi; t += kSelThreads) {
                const uint32_t k = order_key(w[t]);
                if ((k & known) == prefix) atomicAdd(&hist[(k >> shift) & (bins - 1)], 1u);
            }
            __syncthreads();
            // Suffix sums from the largest digit: thread i owns digits bins-1-2i and the next.
            const uint32_t d0 = bins - 1 - 2 * tid, d1 = d0 - 1;
            const bool in = 2 * tid < (int)bins;
            const uint32_t c0 = in ? hist[d0] : 0u, c1 = in ? hist[d1] : 0u;
            uint32_t inc = c0 + c1;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
                if (lane >= o) inc += v;
            }
            if (lane == 31) warp_sum[warp] = inc;
            __syncthreads();
            uint32_t before = inc - c0 - c1;
            for (int i = 0; i < warp; ++i) before += warp_sum[i];
            if (in && before < rank && rank <= before + c0 + c1) {
                const bool first = rank <= before + c0;
                s_prefix = prefix | ((first ? d0 : d1) << shift);
                s_rank = rank - before - (first ? 0u : c0);
            }
            __syncthreads();
            prefix = s_prefix;
            rank = s_rank;
            __syncthreads();
        }
    }
    // Ordered pass.  Kept: protected, above the threshold, or one of the first
    // `rank` tokens at it.
    const uint32_t quota = need > 0 ? rank : 0u;
    uint32_t base_sure = 0, base_tie = 0;
    for (int t0 = 0; t0 < L; t0 += kSelThreads) {
        const int t = t0 + tid;
        bool sure = false, tie = false;
        float wt = 0.f;
        if (t < L) {
            wt = w[t];
            const bool mid = t >= lo && t < hi;
            const uint32_t k = order_key(wt);
            sure = !mid || (need > 0 && k > prefix);
            tie = mid && need > 0 && k == prefix;
        }
        const uint32_t bs = __ballot_sync(0xffffffffu, sure), bt = __ballot_sync(0xffffffffu, tie);
        if (lane == 0) warp_sum[warp] = (uint32_t)__popc(bs) | (uint32_t)__popc(bt) << 16;
        __syncthreads();  // and every weight of this chunk has been read
        const uint32_t mine = warp_sum[lane];
        uint32_t inc = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const uint32_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const uint32_t all = __shfl_sync(0xffffffffu, inc, 31);
        const uint32_t pre = __shfl_sync(0xffffffffu, inc - mine, warp);
        const uint32_t below = (1u << lane) - 1u;
        const uint32_t nsure = base_sure + (pre & 0xffffu) + __popc(bs & below);
        const uint32_t ntie = base_tie + (pre >> 16) + __popc(bt & below);
        if (sure || (tie && ntie < quota)) {
            const int pos = (int)(nsure + min(ntie, quota));
            kept[pos] = t;
            wo[pos] = wt;
            if (pos != t) atomicMin(&s_first, pos);
        }
        base_sure += all & 0xffffu;
        base_tie += all >> 16;
        __syncthreads();  // warp_sum is free again
    }
    for (int t = n + tid; t < p.cap; t += kSelThreads) wo[t] = 0.f;
    if (tid == 0) p.first_moved[at] = s_first;
}

// ---------------------------------------------------------------------------
// Moves.

constexpr int kMoveThreads = 256;
constexpr int kMoveUnroll = 4;

// Grid (column slices, heads * {K, V}, requests).  A slice is `lanes` 16-byte
// columns of one head group's part of a token row.
template <bool kCheck>
__global__ void __launch_bounds__(kMoveThreads) move_kernel(const MoveArgs p, int lanes, int head_bytes, int row_bytes) {
    const int b = blockIdx.z, head = blockIdx.y >> 1;
    char* cache = reinterpret_cast<char*>((blockIdx.y & 1) ? p.v_cache : p.k_cache);
    const size_t at = (size_t)b * p.heads + head;
    const int32_t* src = p.src + at * p.max_rows;
    const int32_t* table = p.page_table + (size_t)b * p.max_pages;
    int n = p.counts[b];
    const int base = p.base ? p.base[b] : 0;
    if (n > p.max_rows || n < 0 || base < 0) {
        if (threadIdx.x == 0 && blockIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        n = base < 0 ? 0 : max(0, min(n, p.max_rows));
    }
    const int col = threadIdx.x % lanes, sub = threadIdx.x / lanes, step = kMoveThreads / lanes;
    const size_t off = (size_t)head * head_bytes + ((size_t)blockIdx.x * lanes + col) * 16;
    auto locate = [&](int t) -> char* {
        if (t / p.page_size >= p.max_pages) {
            raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
            return nullptr;
        }
        const int pg = table[t / p.page_size];
        if (pg < 0 || pg >= p.num_pages) {
            raise_status(ATTN_SINK_DEV_PAGE_OOB);
            return nullptr;
        }
        return cache + ((size_t)pg * p.page_size + t % p.page_size) * row_bytes + off;
    };
    const int j0 = p.first_moved ? p.first_moved[at] : 0;
    for (int jb = j0; jb < n; jb += step * kMoveUnroll) {
        uint4 x[kMoveUnroll];
        char* to[kMoveUnroll];
#pragma unroll
        for (int i = 0; i < kMoveUnroll; ++i) {
            const int j = jb + i * step + sub;
            to[i] = nullptr;
            if (j >= n) continue;
            const int t = src[j];
            if constexpr (kCheck) {
                if (t < base + j || (j > 0 && src[j - 1] >= t)) {
                    raise_status(ATTN_SINK_DEV_ORDER);
                    continue;
                }
            }
            if (t == base + j) continue;
            const char* from = locate(t);
            to[i] = locate(base + j);
            if (!from) to[i] = nullptr;
            if (to[i]) x[i] = *reinterpret_cast<const uint4*>(from);
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kMoveUnroll; ++i)
            if (to[i]) *reinterpret_cast<uint4*>(to[i]) = x[i];
        __syncthreads();  // a later batch reads what this one leaves
    }
}

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    select_kernel<<<dim3(a.heads, a.batch), kSelThreads, 0, s>>>(a);
    return cudaGetLastError();
}

cudaError_t launch_move(const MoveArgs& a, cudaStream_t s) {
    if (a.batch == 0 || a.max_rows == 0) return cudaSuccess;
    const int row_bytes = a.hkv * a.head_dim * 2;
    const int head_bytes = row_bytes / a.heads;
    const int lanes = 4;  // 64-byte slices: every head is a multiple of 128 bytes
    const dim3 grid(head_bytes / (16 * lanes), a.heads * 2, a.batch);
    if (a.first_moved)
        move_kernel<false><<<grid, kMoveThreads, 0, s>>>(a, lanes, head_bytes, row_bytes);
    else
        move_kernel<true><<<grid, kMoveThreads, 0, s>>>(a, lanes, head_bytes, row_bytes);
    return cudaGetLastError();
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace evict
}  // namespace attn
