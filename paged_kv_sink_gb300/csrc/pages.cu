// Bookkeeping of a paged cache's pages on the device: forked page-table rows, pages for
// growing requests, pages given back, pages moved together (sm_103a).
//
// A page is held by as many page-table entries as refs counts.  Everything that is decided
// here is an integer and the same in every run: free pages are given lowest first, to
// requests in their order; counts change by atomic additions, whose order does not show.
//
//  * fork: row b of the new table is row src[b] of the old one.  Entries that a row keeps
//    cost nothing; the others take their old page's count down and their new one's up.
//  * release: the entries of a request that shrinks.
//  * reserve: the entries of requests that grow.  A request that writes into a partly filled
//    page which others hold too gets a copy of it first; of several that all write into one
//    page the last keeps it, where nobody else holds it (as if they came one after the
//    other).  If the free pages do not suffice nothing is changed.
//  * compact: the i-th held page behind the first n = (number of held pages) goes to the
//    i-th free page among them.
// reserve and compact decide in one cluster of CTAs, which scan the counts by slices, tell each
// other their totals through distributed shared memory and meet at the cluster's barrier; the pages
// are then moved by a grid of its own, which reads the list from the device.  The decisions are bound by latency
// (reserve 8 and 12 us for 4 and 512 requests, compact 6 and 13 for pools of 826 and 47k pages), the moves by
// HBM (9.9k pages of 16 KB in K and V, 650 MB read and written: 96 us, the copy's rate).
#include "pages.h"

#include <cooperative_groups.h>
#include <limits.h>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace attn {
namespace pages {

constexpr int kCtas = 8;        // of the deciding cluster
constexpr int kThreads = 1024;  // of its CTAs
constexpr int kRowParts = 4;    // warps that share a row of the table when its entries change
constexpr int kPer = 4;         // counts that a thread reads at once

__device__ __forceinline__ int pages_of(int tokens, int page_size) {
    return tokens / page_size + (tokens % page_size ? 1 : 0);
}

// Whether a row can have `L` tokens; reported if not.
__device__ __forceinline__ bool valid_length(const Table& t, int L) {
    const bool fits = L >= 0 && L <= (long long)t.max_pages * t.page_size;
    if (!fits) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
    return fits;
}

// A length as the row can hold it.
__device__ __forceinline__ int length_of(const Table& t, const int32_t* seqlens, int b) {
    const int L = seqlens[b];
    if (valid_length(t, L)) return L;
    return L < 0 ? 0 : (int)((long long)t.max_pages * t.page_size);
}

__device__ __forceinline__ bool valid_page(const Table& t, int p) { return (unsigned)p < (unsigned)t.num_pages; }

// One reference less.
__device__ __forceinline__ void drop(const Table& t, int p) {
    if (!valid_page(t, p)) {
        raise_status(ATTN_SINK_DEV_PAGE_OOB);
    } else if (atomicSub(t.refs + p, 1) <= 0) {
        atomicAdd(t.refs + p, 1);
        raise_status(ATTN_SINK_DEV_POOL);
    }
}

// ---------------------------------------------------------------------------
// Rows of the table: a warp each.

constexpr int kRowWarps = 4;

__global__ void __launch_bounds__(kRowWarps * 32) fork_kernel(const Table t, const int32_t* seqlens, const int32_t* src,
                                                              int out_batch, int32_t* out_table, int32_t* out_seqlens) {
    const int b = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    const bool had = b < t.batch, has = b < out_batch;
    if (!had && !has) return;
    int from = has ? src[b] : -1;
    if (from < -1 || from >= t.batch) {
        if (lane == 0) raise_status(ATTN_SINK_DEV_POOL);
        from = -1;
    }
    const int held = had ? pages_of(length_of(t, seqlens, b), t.page_size) : 0;
    const int L = from >= 0 ? length_of(t, seqlens, from) : 0, want = pages_of(L, t.page_size);
    const int32_t* const mine = t.table + (size_t)b * t.max_pages;
    const int32_t* const other = t.table + (size_t)max(from, 0) * t.max_pages;
    const int width = has ? t.max_pages : held;
    for (int i = lane; i < width; i += 32) {
        const int was = i < held ? mine[i] : -1, is = i < want ? other[i] : -1;
        if (was != is || (i < held) != (i < want)) {
            if (i < held) drop(t, was);
            if (i < want) {
                if (valid_page(t, is)) atomicAdd(t.refs + is, 1);
                else raise_status(ATTN_SINK_DEV_PAGE_OOB);
            }
        }
        if (has) out_table[(size_t)b * t.max_pages + i] = is;
    }
    if (has && lane == 0) out_seqlens[b] = L;
}

__global__ void __launch_bounds__(kRowWarps * 32) release_kernel(const Table t, const int32_t* seqlens,
                                                                 const int32_t* new_seqlens) {
    const int b = blockIdx.x * kRowWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
    if (b >= t.batch) return;
    // (a row of which a length is no length keeps its pages: nobody knows which of them are in use)
    const int L = seqlens[b], to = new_seqlens[b];
    if (!valid_length(t, L) || !valid_length(t, to)) return;
    if (to > L && lane == 0) raise_status(ATTN_SINK_DEV_POOL);
    const int held = pages_of(L, t.page_size), keep = pages_of(to, t.page_size);
    int32_t* const row = t.table + (size_t)b * t.max_pages;
    for (int i = keep + lane; i < held; i += 32) {
        drop(t, row[i]);
        row[i] = -1;
    }
}

// ---------------------------------------------------------------------------
// Scans inside the cluster.

using u64 = unsigned long long;

// Exclusive sum over the block's threads in order; the block's total in `all`.
__device__ __forceinline__ u64 block_scan(u64 x, u64* warps, u64& all) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    u64 run = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const u64 y = __shfl_up_sync(0xffffffffu, run, o);
        if (lane >= o) run += y;
    }
    if (lane == 31) warps[warp] = run;
    __syncthreads();
    if (warp == 0) {
        u64 w = warps[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        warps[lane] = w;
    }
    __syncthreads();
    const u64 before = warp ? warps[warp - 1] : 0;
    all = warps[31];
    __syncthreads();
    return before + run - x;
}

// Pages of this thread: contiguous, in the order of the cluster's threads, whole int4 of counts.
struct Span {
    int p0, p1;
};

__device__ __forceinline__ Span span_of(int num_pages, int rank) {
    const long long threads = kCtas * kThreads;
    const int len = (int)((num_pages + threads - 1) / threads + kPer - 1) / kPer * kPer;
    const long long at = ((long long)rank * kThreads + threadIdx.x) * len;
    Span s;
    s.p0 = (int)min((long long)num_pages, at);
    s.p1 = (int)min((long long)num_pages, at + len);
    return s;
}

// f(page, whether it is held) for the span's pages, in order.
template <class F>
__device__ __forceinline__ void each_count(const Table& t, Span s, F f) {
    if (reinterpret_cast<uintptr_t>(t.refs) % 16 == 0) {
        int p = s.p0;
        for (; p + kPer <= s.p1; p += kPer) {
            const int4 r = *reinterpret_cast<const int4*>(t.refs + p);
            f(p, r.x > 0);
            f(p + 1, r.y > 0);
            f(p + 2, r.z > 0);
            f(p + 3, r.w > 0);
        }
        for (; p < s.p1; ++p) f(p, t.refs[p] > 0);
    } else {
        for (int p = s.p0; p < s.p1; ++p) f(p, t.refs[p] > 0);
    }
}

// The same as often as wanted: the counts of spans of up to 64 pages (pools of up to 524288)
// are read once.
struct Held {
    Span span;
    u64 mask;
    __device__ __forceinline__ Held(const Table& t, Span s) : span(s), mask(0) {
        if (s.p1 - s.p0 <= 64) each_count(t, s, [&](int p, bool held) { mask |= (u64)held << (p - s.p0); });
    }
    template <class F>
    __device__ __forceinline__ void each(const Table& t, F f) const {
        if (span.p1 - span.p0 <= 64) {
            for (int p = span.p0; p < span.p1; ++p) f(p, mask >> (p - span.p0) & 1);
        } else {
            each_count(t, span, f);
        }
    }
    __device__ __forceinline__ int count(const Table& t) const {
        if (span.p1 - span.p0 <= 64) return __popcll(mask);
        int n = 0;
        each_count(t, span, [&](int, bool held) { n += held; });
        return n;
    }
};

// Totals of the cluster's CTAs, known to all of them after the next cluster barrier.
__device__ __forceinline__ void tell(cg::cluster_group& cluster, u64* totals, u64 mine) {
    if (threadIdx.x < kCtas) *cluster.map_shared_rank(totals + cluster.block_rank(), threadIdx.x) = mine;
}

// Scratch of reserve: per page the requests that are about to write into it and the last
// of them; the free pages in order; what the requests get; the copies; totals.
struct ReserveScratch {
    int4* plan;  // per request: pages held, pages wanted, place in the free pages (top bit: copies), the page that is shared
    int32_t *users, *last, *free, *src, *dst, *head;
    __host__ __device__ ReserveScratch(void* at, const Table& t) {
        int32_t* p = static_cast<int32_t*>(at);
        head = p;  // [0] copies, [1] pages needed
        plan = reinterpret_cast<int4*>(p + 16);
        users = p + 16 + 4 * (size_t)t.batch;
        last = users + t.num_pages;
        free = last + t.num_pages;
        src = free + t.num_pages;
        dst = src + t.batch;
    }
};

struct Growth {
    int from, to;  // pages held, wanted
    int shared;    // the page that the first new token goes into, or -1
};

__device__ __forceinline__ Growth growth_of(const Table& t, const int32_t* seqlens, const int32_t* new_seqlens, int b) {
    const long long cap = (long long)t.max_pages * t.page_size;
    const int L0 = seqlens[b], L1 = new_seqlens[b];
    Growth g = {0, 0, -1};
    if (L0 < 0 || L1 > cap || L1 < L0) return g;  // reported once, below
    g.from = pages_of(L0, t.page_size);
    g.to = pages_of(L1, t.page_size);
    if (L1 > L0 && L0 % t.page_size) {
        const int p = t.table[(size_t)b * t.max_pages + L0 / t.page_size];
        g.shared = valid_page(t, p) ? p : -1;
    }
    return g;
}

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    reserve_kernel(const Table t, const int32_t* seqlens, const int32_t* new_seqlens, int32_t* missing, void* scratch) {
    __shared__ u64 warps[32], totals[kCtas];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // this CTA runs
    const int rank = (int)cluster.block_rank(), tid = threadIdx.x, all_threads = kCtas * kThreads;
    const ReserveScratch s(scratch, t);
    const int b_first = rank * kThreads + tid;
    Growth first = {0, 0, -1};  // of request b_first; those further on are looked up again
    for (int b = b_first; b < t.batch; b += all_threads) {
        const int L0 = seqlens[b], L1 = new_seqlens[b];
        const long long cap = (long long)t.max_pages * t.page_size;
        if (L0 < 0 || L1 > cap) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        else if (L1 < L0) raise_status(ATTN_SINK_DEV_POOL);
        else if (L1 > L0 && L0 % t.page_size && !valid_page(t, t.table[(size_t)b * t.max_pages + L0 / t.page_size]))
            raise_status(ATTN_SINK_DEV_PAGE_OOB);
        const Growth g = growth_of(t, seqlens, new_seqlens, b);
        if (b == b_first) first = g;
        if (g.shared >= 0) {
            s.users[g.shared] = 0;
            s.last[g.shared] = -1;
        }
    }
    const Held held(t, span_of(t.num_pages, rank));
    u64 all;
    const u64 mine = block_scan(held.span.p1 - held.span.p0 - held.count(t), warps, all);  // this thread's first free page in the CTA's order
    cluster.barrier_wait();
    tell(cluster, totals, all);
    cluster.sync();
    for (int b = b_first; b < t.batch; b += all_threads) {
        const Growth g = b == b_first ? first : growth_of(t, seqlens, new_seqlens, b);
        if (g.shared >= 0) {
            atomicAdd(s.users + g.shared, 1);
            atomicMax(s.last + g.shared, b);
        }
    }
    cluster.sync();
    if (rank == 0) {
        // the requests' places: pages in the low bits of a sum (65535 requests of less than
        // 2^31 stay below 2^47), copies in the high ones
        constexpr int kCopyBit = 47;
        constexpr u64 kNeedMask = (1ull << kCopyBit) - 1;
        u64 base = 0;
        for (int b0 = 0; b0 < t.batch; b0 += kThreads) {
            const int b = b0 + tid;
            bool copy = false;
            u64 n = 0;
            Growth g = {0, 0, -1};
            if (b < t.batch) {
                g = b == b_first ? first : growth_of(t, seqlens, new_seqlens, b);
                if (g.shared >= 0) {
                    const int refs = t.refs[g.shared], users = s.users[g.shared], last = s.last[g.shared];
                    if (users > refs) raise_status(ATTN_SINK_DEV_POOL);
                    copy = refs > 1 && users <= refs && !(users == refs && last == b);
                }
                n = (u64)(g.to - g.from + (copy ? 1 : 0)) | (u64)(copy ? 1 : 0) << kCopyBit;
            }
            u64 all;
            const u64 at = base + block_scan(n, warps, all);
            base += all;
            if (b < t.batch) {
                s.plan[b] = make_int4(g.from, g.to, (int)min(at & kNeedMask, 0x7fffffffull) | (copy ? (int)0x80000000 : 0), g.shared);
                const int c = (int)(at >> kCopyBit);
                if (copy) {
                    s.src[c] = g.shared;
                    s.dst[c] = -1 - b;  // the page is not known yet
                }
            }
        }
        if (tid == 0) {
            s.head[0] = (int)(base >> kCopyBit);
            s.head[1] = (int)min(base & kNeedMask, 0x7fffffffull);
        }
    }
    cluster.sync();
    const int need = s.head[1], copies = s.head[0];
    long long before = 0, have = 0;
    for (int c = 0; c < kCtas; ++c) {
        if (c < rank) before += (long long)totals[c];
        have += (long long)totals[c];
    }
    const bool fits = need <= have;
    if (rank == 0 && tid == 0) {
        missing[0] = fits ? 0 : (int)(need - have);
        if (!fits) raise_status(ATTN_SINK_DEV_POOL);
    }
    if (fits) {
        long long r = before + (long long)mine;
        if (r < need)
            held.each(t, [&](int p, bool is_held) {
                if (!is_held) {
                    if (r < need) s.free[r] = p;
                    ++r;
                }
            });
    }
    cluster.sync();
    if (!fits) {
        if (rank == 0 && tid == 0) s.head[0] = 0;  // nothing is copied
        return;
    }
    const int lane = tid & 31;
    for (int b = rank * (kThreads / 32) + (tid >> 5); b < t.batch; b += all_threads / 32) {
        const int4 plan = s.plan[b];
        const int copy = plan.z < 0 ? 1 : 0, from = plan.x - copy;
        const int32_t* const free = s.free + (plan.z & 0x7fffffff) - from;
        int32_t* const row = t.table + (size_t)b * t.max_pages;
        for (int i = from + lane; i < plan.y; i += 32) {
            const int p = free[i];
            row[i] = p;
            t.refs[p] = 1;
        }
        if (copy && lane == 0) atomicSub(t.refs + plan.w, 1);
    }
    for (int c = rank * kThreads + tid; c < copies; c += all_threads) {
        const int b = -1 - s.dst[c];
        s.dst[c] = s.free[s.plan[b].z & 0x7fffffff];
    }
}

// Scratch of compact: which move a held page behind is (-1: it is free), the moves, totals.
struct CompactScratch {
    int32_t *move, *src, *dst, *head;
    __host__ __device__ CompactScratch(void* at, const Table& t) {
        int32_t* p = static_cast<int32_t*>(at);
        head = p;  // [0] moves, [1] held pages
        move = head + 16;
        src = move + t.num_pages;
        dst = src + t.num_pages;
    }
};

__global__ void __cluster_dims__(kCtas, 1, 1) __launch_bounds__(kThreads)
    compact_kernel(const Table t, int32_t* held_out, void* scratch) {
    __shared__ u64 warps[32], totals[2][kCtas];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    cg::cluster_group cluster = cg::this_cluster();
    cluster.barrier_arrive();  // this CTA runs
    const int rank = (int)cluster.block_rank(), tid = threadIdx.x;
    const CompactScratch s(scratch, t);
    const Held held(t, span_of(t.num_pages, rank));
    u64 all;
    block_scan(held.count(t), warps, all);
    cluster.barrier_wait();
    tell(cluster, totals[0], all);
    cluster.sync();
    int n = 0;
    for (int c = 0; c < kCtas; ++c) n += (int)totals[0][c];
    // free ones among the first n (low half), held ones behind (high half), and their ranks
    u64 x = 0;
    held.each(t, [&](int p, bool is_held) { x += p < n ? (is_held ? 0 : 1ull) : is_held ? 1ull << 32 : 0; });
    u64 at = block_scan(x, warps, all);
    tell(cluster, totals[1], all);
    cluster.sync();
    int moves = 0;
    for (int c = 0; c < kCtas; ++c) {
        if (c < rank) at += totals[1][c];
        moves += (int)(totals[1][c] >> 32);
    }
    uint32_t gap = (uint32_t)at, out = (uint32_t)(at >> 32);
    held.each(t, [&](int p, bool is_held) {
        if (p < n) {
            if (!is_held) s.dst[gap++] = p;
        } else if (is_held) {
            s.move[p] = (int)out;
            s.src[out++] = p;
        } else {
            s.move[p] = -1;
        }
    });
    if (rank == 0 && tid == 0) {
        s.head[0] = moves;
        s.head[1] = n;
        held_out[0] = n;
    }
}

// The rows' entries of pages that move: those that a row holds, and all that are pages in a row
// whose length is no length (its pages move as well).
__device__ __forceinline__ void retarget(const Table& t, const int32_t* seqlens, const CompactScratch& s, int n) {
    const int lane = threadIdx.x & 31, warps = gridDim.x * (blockDim.x / 32);
    for (int w = blockIdx.x * (blockDim.x / 32) + (threadIdx.x >> 5); w < t.batch * kRowParts; w += warps) {
        const int b = w / kRowParts, part = w % kRowParts;
        const bool known = valid_length(t, seqlens[b]);
        const int pages = known ? pages_of(seqlens[b], t.page_size) : t.max_pages;
        int32_t* const row = t.table + (size_t)b * t.max_pages;
        for (int i = part * 32 + lane; i < pages; i += 32 * kRowParts) {
            const int p = row[i];
            if (!valid_page(t, p)) {
                if (known) raise_status(ATTN_SINK_DEV_PAGE_OOB);
            } else if (p >= n) {
                const int r = s.move[p];
                if (r >= 0) row[i] = s.dst[r];
                else if (known) raise_status(ATTN_SINK_DEV_POOL);  // held by a row, but not counted
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Page copies: work items of kPiece bytes, (copy, tensor, piece) in that order.

constexpr int kCopyThreads = 256;
constexpr int kAhead = 4;  // 16-byte loads of a thread in flight
constexpr long long kPiece = 16LL * kCopyThreads * kAhead;

template <class V>
__device__ __forceinline__ void copy_piece(const char* from, char* to, long long bytes) {
    const V* const a = reinterpret_cast<const V*>(from);
    V* const b = reinterpret_cast<V*>(to);
    const int n = (int)(bytes / (long long)sizeof(V));
    for (int i = threadIdx.x; i < n; i += kCopyThreads * kAhead) {
        V x[kAhead];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * kCopyThreads < n) x[k] = a[i + k * kCopyThreads];
#pragma unroll
        for (int k = 0; k < kAhead; ++k)
            if (i + k * kCopyThreads < n) b[i + k * kCopyThreads] = x[k];
    }
}

// Copies by all CTAs of the grid.
__device__ __forceinline__ void copy_pages(const Pools& p, const int32_t* src, const int32_t* dst, int n, int num_pages,
                                           bool report) {
    int pieces = 0;  // of one copy
    for (int i = 0; i < p.count; ++i) pieces += p.pieces[i];
    // this CTA's items, gridDim.x apart: copy c, piece k
    long long c = blockIdx.x / pieces;
    int k0 = blockIdx.x % pieces;
    const int dc = gridDim.x / pieces, dk = gridDim.x - dc * pieces;
    for (; c < n; c += dc, k0 += dk) {
        if (k0 >= pieces) {
            k0 -= pieces;
            if (++c >= n) break;
        }
        int k = k0, i = 0;
        for (; k >= p.pieces[i]; ++i) k -= p.pieces[i];
        const int from = src[c], to = dst[c];
        if ((unsigned)from >= (unsigned)num_pages || (unsigned)to >= (unsigned)num_pages) {
            if (report && threadIdx.x == 0 && (from != -1 || to != -1)) raise_status(ATTN_SINK_DEV_PAGE_OOB);
            continue;
        }
        if (from == to) continue;
        const long long at = k * kPiece, len = min(kPiece, p.bytes[i] - at);
        char* const base = static_cast<char*>(p.base[i]);
        const char* const a = base + (long long)from * p.bytes[i] + at;
        char* const b = base + (long long)to * p.bytes[i] + at;
        const unsigned long long odd = (unsigned long long)p.bytes[i] | (unsigned long long)base;
        if (!(odd & 15)) copy_piece<uint4>(a, b, len);
        else if (!(odd & 3)) copy_piece<uint32_t>(a, b, len);
        else copy_piece<uint8_t>(a, b, len);
    }
}

__global__ void __launch_bounds__(kCopyThreads) copy_kernel(const Pools p, const int32_t* src, const int32_t* dst,
                                                            const int32_t* count, int n, int num_pages, bool report) {
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the list is complete (launched behind reserve_kernel)
    copy_pages(p, src, dst, count ? min(n, *count) : n, num_pages, report);
}

// What follows compact_kernel: the counts, the table's entries and the pages.
__global__ void __launch_bounds__(kCopyThreads) move_kernel(const Pools p, const Table t, const int32_t* seqlens, void* scratch) {
    const CompactScratch s(scratch, t);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the decisions are complete
    const int moves = s.head[0];
    for (int r = blockIdx.x * kCopyThreads + threadIdx.x; r < moves; r += gridDim.x * kCopyThreads) {
        const int from = s.src[r], to = s.dst[r];
        t.refs[to] = t.refs[from];
        t.refs[from] = 0;
    }
    retarget(t, seqlens, s, s.head[1]);
    if (p.count) copy_pages(p, s.src, s.dst, moves, t.num_pages, false);
}

// ---------------------------------------------------------------------------
// Host side.

size_t reserve_scratch(const Table& t) { return (16 + 3 * (size_t)t.num_pages + 6 * (size_t)t.batch) * 4; }
size_t compact_scratch(const Table& t) { return (16 + 3 * (size_t)t.num_pages) * 4; }

// Pieces that copies are cut into.
static Pools with_pieces(const Pools& p) {
    Pools q = p;
    for (int i = 0; i < q.count; ++i) q.pieces[i] = (int)((q.bytes[i] + kPiece - 1) / kPiece);
    return q;
}

// CTAs of a grid of copies: 8 of 256 threads an SM, of which 6 are resident at once (38 and 40 registers);
// the others start where the first ones end.  (47k pages brought together: 121.0 us; as many as are
// resident 124.7; 8 resident, in 32 registers with spills, 125.9.)
static int copy_ctas() { return 8 * num_sms(); }

// A grid of copies; `early`: as a programmatic dependent of the deciding kernel before it, whose
// end it waits for itself.
template <class Kernel, class... Args>
static cudaError_t launch_behind(unsigned grid, bool early, cudaStream_t s, Kernel kernel, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kCopyThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = early ? 1 : 0;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
    return e != cudaSuccess ? e : cudaGetLastError();
}

cudaError_t launch_copy(const Pools& p, const int32_t* src, const int32_t* dst, const int32_t* count, int n, int num_pages,
                        bool report, cudaStream_t s) {
    const Pools q = with_pieces(p);
    long long pieces = 0;
    for (int i = 0; i < q.count; ++i) pieces += q.pieces[i];
    if (n <= 0 || pieces == 0) return cudaSuccess;
    if (pieces > INT_MAX / 2) return cudaErrorInvalidConfiguration;
    const long long want = n * pieces, most = copy_ctas();
    return launch_behind((unsigned)(want < most ? want : most), count != nullptr, s, copy_kernel, q, src, dst, count, n,
                         num_pages, report);
}

cudaError_t launch_fork(const Table& t, const int32_t* seqlens, const int32_t* src, int out_batch, int32_t* out_table,
                        int32_t* out_seqlens, cudaStream_t s) {
    const int rows = t.batch > out_batch ? t.batch : out_batch;
    if (rows == 0) return cudaSuccess;
    fork_kernel<<<(rows + kRowWarps - 1) / kRowWarps, kRowWarps * 32, 0, s>>>(t, seqlens, src, out_batch, out_table,
                                                                            out_seqlens);
    return cudaGetLastError();
}

cudaError_t launch_release(const Table& t, const int32_t* seqlens, const int32_t* new_seqlens, cudaStream_t s) {
    if (t.batch == 0) return cudaSuccess;
    release_kernel<<<(t.batch + kRowWarps - 1) / kRowWarps, kRowWarps * 32, 0, s>>>(t, seqlens, new_seqlens);
    return cudaGetLastError();
}

cudaError_t launch_reserve(const Pools& p, const Table& t, const int32_t* seqlens, const int32_t* new_seqlens,
                           int32_t* missing, void* scratch, cudaStream_t s) {
    reserve_kernel<<<kCtas, kThreads, 0, s>>>(t, seqlens, new_seqlens, missing, scratch);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const ReserveScratch r(scratch, t);
    return launch_copy(p, r.src, r.dst, r.head, t.batch, t.num_pages, false, s);
}

cudaError_t launch_compact(const Pools& p, const Table& t, const int32_t* seqlens, int32_t* held, void* scratch,
                           cudaStream_t s) {
    const Pools q = with_pieces(p);
    long long pieces = 0;
    for (int i = 0; i < q.count; ++i) pieces += q.pieces[i];
    if (pieces > INT_MAX / 2) return cudaErrorInvalidConfiguration;
    compact_kernel<<<kCtas, kThreads, 0, s>>>(t, held, scratch);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    const long long want = t.num_pages * (pieces > 0 ? pieces : 1), rows = ((long long)t.batch * kRowParts + 7) / 8;
    long long grid = want > rows ? want : rows;
    if (grid > copy_ctas()) grid = copy_ctas();
    return launch_behind((unsigned)grid, true, s, move_kernel, q, t, seqlens, scratch);
}

ATTN_DEFINE_STATUS_ACCESSOR(status_word)

}  // namespace pages
}  // namespace attn
