// Attention of a tree of drafted tokens over a paged cache, on tcgen05 tensor
// cores (sm_103a).
//
// What it computes: request b has n drafted tokens (nodes), which are the last
// n of its L cached tokens; node i hangs on node parents[i] < i, or on the
// prefix (the first P = L - n tokens) when that is -1.  With depth 0 for nodes on
// the prefix and one more than the parent's otherwise, node i stands at position
// p_i = P + depth_i and sees the prefix tokens and its ancestors and itself, all by
// the first/last-window rule at their positions:
//     O_i = sum_j e^{s_ij - M} v_j / (e^{sink - M} + sum_j e^{s_ij - M}).
//
// All query heads of a KV head share its keys, so the 128 rows of a tensor-core
// tile are (node, head of the group) pairs: 128 / G nodes of the G heads of one KV
// head (one TMA box of Q).  A draft of 16 nodes with G = 8 then fills a tile, and
// K / V are read once for all of it; a tile per query head, as in the paged
// forward, would leave 7/8 of its rows empty and read K / V eight times.
//
// The unit of work is a step: one 128-key tile of one (request, row tile), for one KV
// head.  The grid is one wave of persistent CTAs (two per SM at d 64, one at d 128) in
// gangs of one CTA per KV head.  The gangs share all steps of the batch out evenly,
// each a run of consecutive steps: requests of any lengths balance, and only the first
// and the last row tile of a run can be incomplete.  (A gang reads whole token rows:
// CTAs that were each at another place of the cache read 128 bytes of 1 KB rows at a
// time, 4.1 TB/s against 5.8.)  A run is cut into segments (the steps of one row
// tile); the pipeline goes on across them.  In a CTA
//   warp 0      TMA producer of the K tiles, page segment by page segment
//   warp 1      TMEM allocator, loads Q once per segment and issues S = Q K^T (128 x
//               128, operands in shared memory)
//   warp 2      TMA producer of the V tiles
//   warp 3      issues O += P V (P read from TMEM)
//   warps 4..7  softmax, one row per thread, in the manner of the paged forward:
//               against a running reference that starts at the sink and moves only
//               when a value exceeds it by 2^64.  The sink itself is added once, at
//               the end.
// A segment that has all key tiles of its row tile writes the output; the others leave
// un-normalised fp32 partials (two places per run and KV head), which
// tree_combine_kernel merges.
//
// Rounding: scores, references, sums, O and the partials are fp32.  The weights e^{s - M}
// alone go to the tensor core as bf16, each off by at most 2^-8 of itself (the sum that
// divides them is that of the unrounded ones), because P V takes P in V's type: P as two
// bf16 parts would take twice the tensor work and, at d 64, more tensor memory than two
// CTAs an SM have.  Next to the output's own rounding it takes the error of O, as a
// 2-norm over that of O, from 1.7e-3 to 2.0e-3 - 2.5e-3, as in every attention call of
// this library; LSE does not see it.
//
// Masks: prefix tiles that every row sees whole are not masked at all.  In the
// others each thread builds the 128-bit visibility of its row: ranges for the
// prefix, and its ancestors' bits by walking up the parents, once per tile.
//
// What bounds it, with the times measured:
//   * At d 128 (one row tile a request) the cache's reads.  32 requests of 8 to 32 nodes, 32
//     heads over 8, 1024 + 7168 tokens visible: 187 us, 5.8 TB/s (7 TB/s while the steps
//     run).  (One CTA per (request, row tile, KV head, range of keys), dispatched by the
//     hardware: 222 us.)
//   * At d 64 with several row tiles a request the softmax.  16 requests of 1k to 16k tokens
//     and 16 to 64 nodes, 64 heads over 8: 132 us for 87 steps a CTA of 1.2 us each (two
//     CTAs an SM; 1086 TFLOP/s at 1.175 us: the exponentials' serial chain).  The first S
//     is ready after 6 us, a masked tile with the drafted tokens costs 2 us more than
//     another, the last gang ends 7 us after the median one, the merge takes 4.5 us, and 81
//     % of the tiles' rows hold a node.  HBM is read for 474 MB (301 MB of cache; 781 MB
//     and 138 us while each row tile took its keys from the first on).
//   * One request: latency.  7 nodes over 2000 tokens 13.9 us: first S after 3.7 us, two
//     steps and the epilogue 4.5, the merge 3.
// With plain fp32 arithmetic, a CTA per node and KV head, the first two took 19.7 and 21.8
// ms; without the runs the second 163 us.
// Measured and left out: runs cut into rounds of shorter ones (slower); two gangs a run, on
// neighbouring row tiles, and runs that allow for the masked tiles (each leaves the softmax
// short of registers: all else 2 - 5 % slower); tensor memory allocated before the runs are
// known; drafted tiles' rows cleaned by the warp that issues P V, or a tile later.
#include <cudaTypedefs.h>

#include <type_traits>

#include "common.cuh"
#include "sm103.cuh"
#include "tree.h"

namespace attn {
namespace tree {

using namespace sm103;

constexpr int BM = 128, BN = 128;
constexpr int kStages = 3;  // K and V rings
constexpr int kBadRing = 4;  // segments that the V producer may be ahead, + 1
constexpr int kSegRing = 5;  // segments that the K producer (kStages tiles ahead of S) may be ahead of the softmax, + 1
constexpr int kTileRing = 8;  // tiles that the K producer may be ahead of the softmax, + 1, and more
constexpr int kMinSteps = 2;  // of a run
constexpr int kThreads = 256;
// 128 registers per thread at launch, moved from the control warps to the softmax
// warps: 128 * 48 + 128 * 208 = 256 * 128.  At d 128 they leave 13 words of a thread in
// local memory (written once and read 28 times in the code), at d 64 one.
constexpr int kRegsCtrl = 48, kRegsSoftmax = 208;
constexpr uint32_t kAtom = 128 * 128;  // one 128-byte-swizzled atom column: 128 rows x 64 bf16
constexpr float kRescaleThreshold = 64.0f;      // log2 units
constexpr float kFastSumLimit = 1.8446744e19f;  // 2^64

// TMEM: S at column 0 (128 fp32), O at 128 (D fp32), P behind it (64 columns of
// bf16 pairs).  At d 64 two CTAs share an SM (256 columns and 113 KB each).
template <int D>
struct Cfg {
    static constexpr int kAtoms = D / 64;
    static constexpr uint32_t kTile = kAtom * kAtoms;
    static constexpr uint32_t kTmemCols = D == 64 ? 256 : 512;
    static constexpr uint32_t cS = 0, cO = 128, cP = 128 + D;
    static constexpr bool kTwoPerSm = D == 64;
};

struct Params {
    const float* sink;
    const int32_t* cu_q;
    const int32_t* seqlens_k;
    const int32_t* parents;
    const int32_t* page_table;
    const __nv_bfloat16* v_cache;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;       // (runs, hkv, 2, 128, D) fp32, un-normalised
    float2* part_ml;     // (runs, hkv, 2, 128): (reference in log2 units, sum)
    long long* first;    // (batch + 1): steps before each request; then the steps per run
    int gangs, batch, max_pages, page_shift, seg_shift, num_pages;
    int hq, hkv, group, total_q, max_q;
    int npt;  // nodes per row tile
    int win_first, win_last;
    float scale_log2;
};

// What the kernels derive of a request.
struct Request {
    int q_start, n, L, P;  // first row, nodes, cached tokens, prefix
    int rows, mtiles;      // nodes that get results, row tiles of them
    int ta, tb, ntiles;    // key tiles [0, ta) and [tb, ...), ntiles in all
    __device__ __forceinline__ int tile(int it) const { return it < ta ? it : tb + (it - ta); }
};

__device__ __forceinline__ Request request(const Params& p, int b, bool report) {
    Request r;
    r.q_start = p.cu_q[b];
    r.n = p.cu_q[b + 1] - r.q_start;
    r.L = p.seqlens_k[b];
    const long long cap = (long long)p.max_pages << p.page_shift;
    const bool over = r.n > p.max_q || r.q_start < 0 || (long long)r.q_start + r.n > p.total_q;
    if (over || (r.n > 0 && (r.L > cap || r.L < r.n))) {
        if (report) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        if (r.L > cap) r.L = (int)cap;
    }
    r.rows = r.q_start < 0 ? 0 : max(0, min(min(r.n, p.max_q), p.total_q - r.q_start));
    r.mtiles = (r.rows + p.npt - 1) / p.npt;
    if (r.L < r.n) r.L = 0;  // the nodes are not in the cache: nothing is seen
    r.P = max(0, r.L - r.n);
    const int t_end = (r.L + BN - 1) / BN;
    r.ta = r.tb = t_end;
    if (p.win_last > 0) {
        r.ta = (min(p.win_first, r.L) + BN - 1) / BN;
        const int lo = max(0, r.P + 1 - p.win_last);  // of the shallowest nodes
        r.tb = min(max(r.ta, lo / BN), t_end);
    }
    r.ntiles = r.ta + (t_end - r.tb);
    return r;
}

__device__ __forceinline__ long long steps_of(const Request& r) { return (long long)r.mtiles * r.ntiles; }

// Steps of each gang's run.
__device__ __forceinline__ long long run_steps(long long total, int gangs) {
    return max((long long)kMinSteps, (total + gangs - 1) / gangs);
}

// Prefix tokens [first, end) that nodes on the prefix see as part of the last window
// and the deepest possible node does not (at most kMaxNodes - 1 of them).
__device__ __forceinline__ int some_first(const Params& p, const Request& r) {
    return p.win_last > 0 ? max(max(0, p.win_first), r.P + 1 - p.win_last) : 0;
}
__device__ __forceinline__ int some_end(const Params& p, const Request& r) {
    return p.win_last > 0 ? max(0, min(r.P, r.P + min(r.n, kMaxNodes) - p.win_last)) : 0;
}

// The steps [it0, it0 + ntiles) of one row tile: what a CTA works on at a time.  They take
// its key tiles in turn, from `key0` on and round to the first behind the last.
struct Segment {
    Request rq;
    int b, mt, it0, ntiles;  // request, row tile
    int key0;
    __device__ __forceinline__ int tile(int it) const {
        const int k = key0 + it;
        return rq.tile(k < rq.ntiles ? k : k - rq.ntiles);
    }
    __device__ __forceinline__ bool whole() const { return it0 == 0 && ntiles == rq.ntiles; }
};

// A gang's run of steps, segment by segment.  Warps 0 to 2 walk a cursor of their own,
// kept in shared memory (it is read a few times per tile, and the warps have 48
// registers); warp 0 hands its segments on to warp 3 and the softmax, which find them
// there when its first tile arrives.
struct Cursor : Segment {
    int left;  // steps of the run from this segment on

    __device__ __forceinline__ void start(const Params& p, int b0, int step, int steps, int per_run) {
        b = b0;
        left = steps;
        rq = request(p, b, false);
        mt = step / rq.ntiles;
        it0 = step - mt * rq.ntiles;
        ntiles = min(rq.ntiles - it0, left);
        key0 = it0;
        if (rq.mtiles > 1) turn(it0 > 0 ? (per_run - it0 % per_run) % per_run : 0, per_run);
    }
    // The gangs run side by side, and what one has read another finds in L2 if it comes
    // soon.  So where a request has several row tiles, each begins with the key tile that
    // its first step's place in the run (`at`) stands for, or, if more of its steps
    // are in the next run, such that those begin there with the first key tile.
    __device__ __forceinline__ void turn(int at, int per_run) {
        const int nt = rq.ntiles, first = per_run - at;
        key0 = (it0 + (nt < per_run && 2 * first < nt ? nt - first : at)) % nt;
    }
    // To the next segment; false at the run's end.  A converged warp calls it.
    __device__ __forceinline__ bool next(const Params& p, int run, int per_run) {
        __syncwarp();
        if ((threadIdx.x & 31) == 0) {
            left -= ntiles;
            if (left > 0) {
                it0 = 0;
                if (++mt == rq.mtiles) {
                    mt = 0;
                    do rq = request(p, ++b, false);
                    while (steps_of(rq) == 0);
                }
                ntiles = min(rq.ntiles, left);
                key0 = 0;
                if (rq.mtiles > 1) turn(run - left, per_run);
            }
        }
        __syncwarp();
        return left > 0;
    }
};

template <int D>
struct __align__(1024) Smem {
    uint8_t q[Cfg<D>::kTile];
    uint8_t k[kStages][Cfg<D>::kTile];
    uint8_t v[kStages][Cfg<D>::kTile];
    uint64_t q_full, q_empty;  // one phase per segment
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t s_full, s_free, p_full, o_done;  // one phase per key tile
    uint64_t final_bar, final_pv;
    uint64_t v_fix;  // V tiles that need their rows looked at land here first
    uint32_t tmem_base;
    int abort;
    int start_b, start_step, run;  // the run's first request, step in it, and length
    int per_run;                   // length of all runs but the last
    Cursor cursor[3];              // warps 0 to 2
    int2 tiles[kTileRing];  // per tile: first token, page segments (bits) read through a bad page id
    // Per segment: tokens that some rows see and others do not whose V row holds an
    // infinity or a NaN; nodes, then prefix tokens at the window's start.
    uint32_t v_bad[kBadRing][2 * kMaxNodes / 32];
    union {
        Segment segment[kSegRing];
        long long sums[kThreads / 32];  // while the run is looked for
    };
};

// Waits that ignore the abort flag (they drain work in flight before shared
// memory and TMEM are released); still bounded in time.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    int dummy = 0;
    mbar_wait(bar, parity, &dummy);
}

// The .aligned instructions below -- TMEM loads, stores and their waits, barriers of a
// warpgroup -- are defined for a converged warp only, and nothing but a warp-wide
// synchronisation promises that lanes are together again behind a loop or branch of
// their own.  So a __syncwarp() stands before each that follows one.

// Whether x holds in all 128 threads of the softmax warpgroup (also a barrier of theirs).
__device__ __forceinline__ bool group_all(bool x) {
    __syncwarp();
    uint32_t y;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %1, 0;\n\t"
        "bar.red.and.pred q, 1, 128, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(y)
        : "r"((uint32_t)x)
        : "memory");
    return y != 0;
}

// Bits 15 and 31 of the result: whether the low / high bf16 of some word is an infinity or a NaN.
__device__ __forceinline__ uint32_t nonfinite_in(const uint4& x) {
    auto carry = [](uint32_t w) { return (w & 0x7f807f80u) + 0x00800080u; };
    return (carry(x.x) | carry(x.y) | carry(x.z) | carry(x.w)) & 0x80008000u;
}
__device__ __forceinline__ uint32_t finite_pair(uint32_t w) {  // non-finite halves become 0
    if ((w & 0x7f80u) == 0x7f80u) w &= 0xffff0000u;
    if ((w & 0x7f800000u) == 0x7f800000u) w &= 0xffffu;
    return w;
}

template <int D>
__global__ void __launch_bounds__(kThreads, 2)
    tree_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                const __grid_constant__ CUtensorMap tm_v, const Params p) {
    using C = Cfg<D>;
    constexpr uint32_t kTile = C::kTile;
    constexpr uint32_t cS = C::cS, cO = C::cO, cP = C::cP;
    extern __shared__ uint8_t smem_raw[];
    // Two CTAs of 113 KB fit an SM only without alignment slack: at d 64 the
    // dynamic shared base must be 1024-aligned already (checked); at d 128 it is
    // rounded up inside 1 KB of slack.
    uint8_t* smem_al = C::kTwoPerSm ? smem_raw
                                    : reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                                 ~uintptr_t(1023));
    Smem<D>& S = *reinterpret_cast<Smem<D>*>(smem_al);
    // The combine grid may be scheduled from here on; it waits for this one's end.
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if (smem_u32(smem_al) & 1023u) {
        if (threadIdx.x == 0) raise_status(ATTN_SINK_DEV_LAYOUT);
        return;
    }

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int kvh = blockIdx.x % p.hkv, gang = blockIdx.x / p.hkv;
    if (threadIdx.x == 0) {
        mbar_init(&S.q_full, 1);
        mbar_init(&S.q_empty, 1);
        for (int s = 0; s < kStages; ++s) {
            mbar_init(&S.k_full[s], 1);
            mbar_init(&S.k_empty[s], 1);
            mbar_init(&S.v_full[s], 1);
            mbar_init(&S.v_empty[s], 1);
        }
        mbar_init(&S.s_full, 1);
        mbar_init(&S.s_free, 128);
        mbar_init(&S.p_full, 128);
        mbar_init(&S.o_done, 1);
        mbar_init(&S.final_bar, 1);
        mbar_init(&S.final_pv, 1);
        mbar_init(&S.v_fix, 1);
        S.abort = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < kBadRing * 2 * kMaxNodes / 32) S.v_bad[0][threadIdx.x] = 0;
    // This gang's run: the batch's steps are counted, then the request that holds the
    // run's first step is looked for, 256 requests at a time.
    const int tid = threadIdx.x;
    // Steps of 256 requests: this thread's, up to and including it, of all.
    long long steps = 0, inc = 0, sum_steps = 0;
    auto scan = [&](int i0, bool report) {
        steps = i0 + tid < p.batch ? steps_of(request(p, i0 + tid, report)) : 0;
        inc = steps;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        __syncthreads();  // the previous sums have been read
        if (lane == 31) S.sums[warp] = inc;
        __syncthreads();
        sum_steps = 0;
#pragma unroll
        for (int w = 0; w < kThreads / 32; ++w) {
            if (w < warp) inc += S.sums[w];
            sum_steps += S.sums[w];
        }
    };
    long long total = 0;
    for (int i0 = 0; i0 < p.batch; i0 += kThreads) {
        scan(i0, blockIdx.x == 0);
        total += sum_steps;
    }
    const long long per_run = run_steps(total, p.gangs);
    const long long w0 = gang * per_run;
    if (blockIdx.x != 0 && w0 >= total) return;
    long long before = 0;
    for (int i0 = 0; i0 < p.batch; i0 += kThreads) {
        if (p.batch > kThreads) scan(i0, false);
        const long long at = before + inc - steps;
        if (steps > 0 && at <= w0 && w0 < at + steps) {
            S.start_b = i0 + tid;
            S.start_step = (int)(w0 - at);
        }
        if (blockIdx.x == 0 && i0 + tid < p.batch) p.first[i0 + tid] = at;
        before += sum_steps;
    }
    if (blockIdx.x == 0 && tid == 0) p.first[p.batch] = per_run;
    if (total == 0) return;
    if (tid == 0) S.run = (int)min(per_run, total - w0), S.per_run = (int)per_run;
    __syncthreads();  // the run is known to all, and S.sums has been read
    if (tid < 3) S.cursor[tid].start(p, S.start_b, S.start_step, S.run, S.per_run);
    if (warp == 1) {
        tmem_alloc(&S.tmem_base, C::kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = S.tmem_base;
    volatile int* abort = &S.abort;

    if (warp < 4) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtrl));
        if (warp == 0 || warp == 2) {
            // -------------------------------------------------------- producers
            // Converged warps: lane i resolves the physical slot of the tile's i-th
            // page segment and issues its copies.
            const bool is_k = warp == 0;
            Cursor& c = S.cursor[warp];
            uint64_t* full = is_k ? S.k_full : S.v_full;
            uint64_t* empty = is_k ? S.k_empty : S.v_empty;
            uint8_t* dst0 = is_k ? S.k[0] : S.v[0];
            const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
            const int nseg = BN >> p.seg_shift;
            if (lane == 0) prefetch_tmap(tm);
            // Rows of a V tile that no row of the request may see enter P V as
            // zeros, whatever the memory holds (a weight of 0 times a NaN would not
            // vanish): rows past the last token, in the window's gap, or read through
            // a bad page id.  Of tokens that only some rows see (drafted ones, and the
            // first ones of the last window, which deeper nodes have left behind)
            // infinities and NaNs are zeroed too, and added at the end by the rows that
            // see them.  Such tiles land on v_fix and are released to the tensor core
            // once they are clean.
            int fixes = 0, segs = 0;
            int n = 0;  // tiles so far
            bool ok = true;
            do {
                const int L = c.rq.L, P = c.rq.P;
                const int gap0 = p.win_last > 0 ? p.win_first : 0;
                const int gap1 = p.win_last > 0 ? P + 1 - p.win_last : 0;
                const int some0 = some_first(p, c.rq), some1 = some_end(p, c.rq);
                // this lane's page id of a tile (0 for none), requested a tile ahead
                auto segment_page = [&](int j0) -> int {
                    const int j = j0 + (lane << p.seg_shift);
                    return lane < nseg && j < L ? __ldg(p.page_table + (size_t)c.b * p.max_pages + (j >> p.page_shift))
                                                : 0;
                };
                int next = segment_page(c.tile(0) * BN);
                for (int it = 0; it < c.ntiles; ++it, ++n) {
                    const int st = n % kStages;
                    const int pg = next;
                    if (it + 1 < c.ntiles) next = segment_page(c.tile(it + 1) * BN);
                    if (n >= kStages &&
                        !__all_sync(0xffffffffu, mbar_wait(&empty[st], ((n / kStages) - 1) & 1, abort))) {
                        ok = false;
                        break;
                    }
                    if (is_k && it == 0 && lane == 0) S.segment[segs % kSegRing] = c;  // released with the tile
                    const int j0 = c.tile(it) * BN;
                    const int j = j0 + (lane << p.seg_shift);
                    const bool bad = (unsigned)pg >= (unsigned)p.num_pages;
                    if (bad && is_k) raise_status(ATTN_SINK_DEV_PAGE_OOB);
                    // segments past the last token and bad ones read slot 0
                    const int slot = bad || j >= L ? 0 : (pg << p.page_shift) | (j & ((1 << p.page_shift) - 1));
                    const uint32_t bad_segs = __ballot_sync(0xffffffffu, bad);
                    const bool all = bad_segs != 0 || (j0 < gap1 && j0 + BN > gap0) || (j0 < some1 && j0 + BN > some0);
                    const int from = all ? 0 : max(P - j0, 0);  // the first row to look at
                    const bool fix = !is_k && from < BN;
                    uint64_t* bar = fix ? &S.v_fix : &full[st];
                    if (lane == 0) {
                        if (is_k) S.tiles[n % kTileRing] = make_int2(j0, (int)bad_segs);
                        mbar_expect_tx(bar, kTile);
                    }
                    __syncwarp();
                    if (lane < nseg) {
                        uint8_t* dst = dst0 + st * kTile + ((uint32_t)lane << p.seg_shift) * 128u;
#pragma unroll
                        for (int a = 0; a < C::kAtoms; ++a) tma_load_3d(dst + a * kAtom, tm, bar, 64 * a, kvh, slot);
                    }
                    if (fix) {
                        const uint32_t parity = fixes++ & 1;
                        if (!__all_sync(0xffffffffu, mbar_wait(&S.v_fix, parity, abort))) {
                            ok = false;
                            break;
                        }
                        // Key row r of an atom is the 128 bytes at r * 128 (the swizzle
                        // permutes 16-byte chunks within a row).
                        bool each = true;  // whether to go through the cells one by one
                        if constexpr (!C::kTwoPerSm) {
                            // 32 rows at a time: which are zeroed and which looked at, then 4
                            // rows an instruction; the cells follow if there is something to
                            // mend.  (32 KB in under 2 us; cell by cell 7.3, which held the V
                            // ring up: 32 windowed requests 195 us instead of 187, two row
                            // tiles a request 168 instead of 147.  At d 64 the SM's other CTA
                            // hides it, and this form is 2 - 4 % slower there.)
                            uint4* const cells = reinterpret_cast<uint4*>(dst0 + st * kTile) + lane;
                            uint32_t found = 0;
#pragma unroll 1
                            for (int r0 = from & ~31; r0 < BN; r0 += 32) {
                                const int r = r0 + lane, t = j0 + r;
                                const bool zero =
                                    t >= L || (t >= gap0 && t < gap1) || (bad_segs >> (r >> p.seg_shift) & 1u);
                                const bool look = !zero && (t >= P || (t >= some0 && t < some1));
                                const uint32_t zeros = __ballot_sync(0xffffffffu, zero) >> (lane >> 3);
                                const uint32_t looks = __ballot_sync(0xffffffffu, look) >> (lane >> 3);
#pragma unroll 1
                                for (int a = 0; a < C::kAtoms; ++a) {
                                    uint4* const x = cells + a * (BN * 8) + r0 * 8;
#pragma unroll
                                    for (int g = 0; g < 8; ++g)
                                        if (zeros >> (4 * g) & 1u) x[g * 32] = make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
                                    for (int g = 0; g < 8; ++g)
                                        if (looks >> (4 * g) & 1u) found |= nonfinite_in(x[g * 32]);
                                }
                            }
                            each = __any_sync(0xffffffffu, found != 0);
                        }
                        for (int e = each ? from * 8 + lane : (int)(kTile / 16); e < (int)(kTile / 16); e += 32) {
                            const int r = (e >> 3) & (BN - 1), t = j0 + r;
                            uint4* cell = reinterpret_cast<uint4*>(dst0 + st * kTile) + e;
                            if (t >= L || (t >= gap0 && t < gap1) || (bad_segs >> (r >> p.seg_shift) & 1u)) {
                                *cell = make_uint4(0u, 0u, 0u, 0u);
                            } else if (t >= P || (t >= some0 && t < some1)) {
                                const uint4 x = *cell;
                                if (nonfinite_in(x)) {
                                    *cell = make_uint4(finite_pair(x.x), finite_pair(x.y), finite_pair(x.z),
                                                       finite_pair(x.w));
                                    const int i = t >= P ? t - P : kMaxNodes + t - some0;
                                    if (t < P || i < kMaxNodes)
                                        atomicOr(&S.v_bad[segs % kBadRing][i >> 5], 1u << (i & 31));
                                }
                            }
                        }
                        __threadfence_block();
                        fence_proxy_async_smem();  // the tensor core reads through the async proxy
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&full[st]);
                    }
                }
                ++segs;
            } while (ok && c.next(p, S.run, S.per_run));
            // Drain: every copy issued must have landed before the CTA exits.
            if (lane == 0) {
                if (fixes > 0) drain_wait(&S.v_fix, (fixes - 1) & 1);
                for (int st = 0; st < kStages; ++st) {
                    const int m = n > st ? (n - st + kStages - 1) / kStages : 0;
                    if (m > 0) drain_wait(&full[st], (m - 1) & 1);
                }
            }
            __syncwarp();
        } else {
            // -------------------------------------------------------- MMA issuers
            constexpr uint32_t idS = idesc_bf16_f32(BM, BN, false, false);
            constexpr uint32_t idO = idesc_bf16_f32(BM, D, false, true);
            const uint64_t dq = sdesc_sw128(smem_u32(S.q), 16, 1024);
            const uint64_t dk0 = sdesc_sw128(smem_u32(S.k[0]), 16, 1024);
            const uint64_t dv0 = sdesc_sw128(smem_u32(S.v[0]), kAtom, 1024);
            auto wait_all = [&](uint64_t* bar, uint32_t parity) {
                return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort));
            };
            bool ok = true;
            int n = 0, segs = 0;  // tiles, segments so far
            if (warp == 1) {
                Cursor& c = S.cursor[1];
                // Q is loaded by this warp, as soon as the previous segment's last S has
                // read its predecessor: K is on its way by then.
                if (lane == 0) prefetch_tmap(&tm_q);
                do {
                    if (segs > 0 && !(ok = wait_all(&S.q_empty, (segs - 1) & 1))) break;
                    if (lane == 0) {
                        mbar_expect_tx(&S.q_full, (uint32_t)(p.npt * p.group) * (D * 2));
#pragma unroll
                        for (int a = 0; a < C::kAtoms; ++a)
                            tma_load_3d(S.q + a * kAtom, &tm_q, &S.q_full, 64 * a, kvh * p.group,
                                        c.rq.q_start + c.mt * p.npt);
                    }
                    __syncwarp();
                    if (!(ok = wait_all(&S.q_full, segs & 1))) {
                        if (lane == 0) drain_wait(&S.q_full, segs & 1);  // the copy lands before the CTA exits
                        __syncwarp();
                        break;
                    }
                    for (int it = 0; it < c.ntiles; ++it, ++n) {
                        if (!(ok = wait_all(&S.k_full[n % kStages], (n / kStages) & 1))) break;
                        if (n > 0 && !(ok = wait_all(&S.s_free, (n - 1) & 1))) break;
                        tc_fence_after();
                        const uint64_t dk = dk0 + (n % kStages) * (kTile >> 4);
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t o = (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2;
                            umma_ss_e(tmem + cS, dq + o, dk + o, idS, kk > 0);
                        }
                        umma_commit_e(&S.s_full);
                        umma_commit_e(&S.k_empty[n % kStages]);
                    }
                    if (ok) umma_commit_e(&S.q_empty);
                    ++segs;
                } while (ok && c.next(p, S.run, S.per_run));
                umma_commit_e(&S.final_bar);
                drain_wait(&S.final_bar, 0);
            } else {
                for (int it = 0, ntiles = 0, left = S.run; left > 0; --left, ++n) {
                    if (!(ok = wait_all(&S.v_full[n % kStages], (n / kStages) & 1))) break;
                    if (!(ok = wait_all(&S.p_full, n & 1))) break;
                    tc_fence_after();
                    if (it == ntiles) {  // the first tile of a segment
                        it = 0;
                        ntiles = S.segment[segs++ % kSegRing].ntiles;
                    }
                    const uint64_t dv = dv0 + (n % kStages) * (kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        umma_ts_e(tmem + cO, tmem + cP + kk * 8, dv + 128 * kk, idO, (it > 0 || kk > 0) ? 1u : 0u);
                    umma_commit_e(&S.o_done);
                    umma_commit_e(&S.v_empty[n % kStages]);
                    ++it;
                }
                umma_commit_e(&S.final_pv);
                drain_wait(&S.final_pv, 0);
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
        // ------------------------------------------------------------ softmax
        const int q4 = warp & 3;
        const int r = q4 * 32 + lane;
        const uint32_t lane_base = (uint32_t)(q4 * 32) << 16;
        const uint32_t tS = tmem + lane_base + cS;
        const uint32_t tO = tmem + lane_base + cO;
        const uint32_t tP = tmem + lane_base + cP;
        const int row_node = r / p.group, h = kvh * p.group + r % p.group;
        const float sink = p.sink ? p.sink[h] * ATTN_LOG2E : -INFINITY;
        const float sl2 = p.scale_log2;
        const int nseg = BN >> p.seg_shift;
        int left = S.run, n = 0, segs = 0;  // tiles to come; tiles and segments so far
        while (left > 0) {
            // The four warps go on or give up together (a warp that gave up alone would
            // leave the others waiting at the next group barrier).
            bool ok = mbar_wait(&S.s_full, n & 1, abort);
            if (!group_all(ok)) break;
            const Segment& c = S.segment[segs % kSegRing];  // arrived with its first tile
            const int P = c.rq.P, q_start = c.rq.q_start, ntiles = c.ntiles;
            const int32_t* const pages = p.page_table + (size_t)c.b * p.max_pages;
            const int node = c.mt * p.npt + row_node;
            const bool valid = r < p.npt * p.group && node < c.rq.rows;
            const bool work = __any_sync(0xffffffffu, valid);  // else only the barriers' arrivals
            // parent + 1 of the node a - 1 (0: the prefix)
            auto up = [&](int a) -> int {
                const int pr = __ldg(p.parents + q_start + a - 1);
                if (pr >= -1 && pr < a - 1) return pr + 1;
                raise_status(ATTN_SINK_DEV_TREE);
                return 0;
            };
            const float sg = valid ? sink : -INFINITY;
            float m_ref = sg == INFINITY ? -INFINITY : sg;
            float l = 0.f;
            int pos = P;  // this row's position
            if (p.win_last > 0 && valid)
                for (int a = up(node + 1); a > 0; a = up(a)) ++pos;
            const int pos_max = P + max(c.rq.n, 1) - 1;  // of any node
            for (int it = 0; it < ntiles; ++it, ++n) {
                if (it > 0) {
                    ok = mbar_wait(&S.s_full, n & 1, abort);
                    if (!__all_sync(0xffffffffu, ok)) {
                        ok = false;
                        break;
                    }
                }
                tc_fence_after();
                const int2 here = S.tiles[n % kTileRing];
                const int j0 = here.x;
                const uint32_t bad_segs = (uint32_t)here.y;
                // The previous P V must be complete before P is overwritten or O rescaled.
                auto wait_prev_pv = [&]() -> bool {
                    if (it == 0) return true;
                    const bool done = __all_sync(0xffffffffu, mbar_wait(&S.o_done, (n - 1) & 1, abort));
                    if (done) tc_fence_after();
                    return done;
                };
                if (!work) {
                    tc_fence_before();
                    mbar_arrive(&S.s_free);
                    if (!(ok = wait_prev_pv())) break;
                    mbar_arrive(&S.p_full);
                    continue;
                }
                uint32_t s[4][32];
                __syncwarp();  // a segment's rows have walked to their roots one by one
                tmem_ld32(tS, s[0]);
                tmem_ld32(tS + 32, s[1]);
                tmem_ld_wait();
                tmem_ld32(tS + 64, s[2]);
                tmem_ld32(tS + 96, s[3]);
                bool s_in = false;
                auto finish_s_load = [&]() {
                    if (s_in) return;
                    s_in = true;
                    tmem_ld_wait();
                    tc_fence_before();
                    mbar_arrive(&S.s_free);
                };

                const int jmax = j0 + BN - 1;
                const bool full = jmax < P && !bad_segs &&
                                  (p.win_last <= 0 || jmax < p.win_first || j0 > pos_max - p.win_last);
                uint32_t vis[4] = {0u, 0u, 0u, 0u};
                if (!full) {
                    // Prefix columns [0, c_hi), less the window's gap [f_hi, w_lo).
                    const int c_hi = min(max(P - j0, 0), BN);
                    const int f_hi = p.win_last > 0 ? p.win_first - j0 : BN;
                    const int w_lo = p.win_last > 0 ? pos + 1 - p.win_last - j0 : 0;
                    auto below = [](int c, int w) -> uint32_t {  // bits of word w for columns < c
                        const int k = c - 32 * w;
                        return k <= 0 ? 0u : k >= 32 ? 0xffffffffu : (1u << k) - 1u;
                    };
#pragma unroll
                    for (int w = 0; w < 4; ++w) vis[w] = below(c_hi, w) & (below(f_hi, w) | ~below(w_lo, w));
                    if (jmax >= P && valid) {
                        int at = pos;  // the walked token's position
                        for (int a = node + 1; a > 0; a = up(a), --at) {
                            const int c = P + a - 1 - j0;
                            const bool in = p.win_last <= 0 || at < p.win_first || at > pos - p.win_last;
                            const uint32_t bit = in && c >= 0 && c < BN ? 1u << (c & 31) : 0u;
#pragma unroll
                            for (int w = 0; w < 4; ++w)
                                if ((c >> 5) == w) vis[w] |= bit;
                        }
                    }
                    if (bad_segs) {
                        const uint32_t seg = (p.seg_shift >= 5 ? 0xffffffffu : (1u << (1 << p.seg_shift)) - 1u);
                        for (int i = 0; i < nseg; ++i)
                            if (bad_segs >> i & 1u) {
                                const int c = i << p.seg_shift, len = 1 << p.seg_shift;
#pragma unroll
                                for (int w = 0; w < 4; ++w)
                                    if ((c >> 5) <= w && (c + len - 1) >> 5 >= w) vis[w] &= ~(seg << (c & 31));
                            }
                    }
                    __syncwarp();  // the rows have walked to their roots
                }
                auto mask_half = [&](auto hfc) {
                    constexpr int hf = decltype(hfc)::value;
#pragma unroll
                    for (int c = 2 * hf; c < 2 * hf + 2; ++c)
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            if (!(vis[c] >> i & 1u)) s[c][i] = __float_as_uint(-INFINITY);
                };
                uint32_t w[64];
                auto exps_half = [&](auto hfc, float m_use) -> float {
                    constexpr int hf = decltype(hfc)::value;
                    const uint64_t sc2 = f2_pack(sl2, sl2), nm2 = f2_pack(-m_use, -m_use);
                    uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
                    for (int e = 32 * hf; e < 32 * hf + 32; ++e) {
                        const int i0 = 2 * e;
                        const uint64_t y = f2_fma(f2_pack(__uint_as_float(s[i0 >> 5][i0 & 31]),
                                                          __uint_as_float(s[(i0 + 1) >> 5][(i0 + 1) & 31])),
                                                  sc2, nm2);
                        float y0, y1;
                        f2_unpack(y, y0, y1);
                        const float x0 = fast_exp2(y0), x1 = fast_exp2(y1);
                        acc2[e & 3] = f2_add(acc2[e & 3], f2_pack(x0, x1));
                        w[e] = pack_bf16x2(x0, x1);
                    }
                    float sum = 0.f;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        float lo, hi;
                        f2_unpack(acc2[e], lo, hi);
                        sum += lo + hi;
                    }
                    return sum;
                };
                using H0 = std::integral_constant<int, 0>;
                using H1 = std::integral_constant<int, 1>;
                // Fast path: against the current reference, without the row maximum; every
                // value is <= 2^64 unless a half's sum says otherwise.  Rows without a
                // node have no say.
                bool slow = __any_sync(0xffffffffu, valid && m_ref == -INFINITY);
                bool stored0 = false;
                float rs = 0.f;
                if (!slow) {
                    if (!full) mask_half(H0{});
                    const float rs0 = exps_half(H0{}, m_ref);
                    finish_s_load();
                    const bool ok0 = !__any_sync(0xffffffffu, valid && !(rs0 <= kFastSumLimit));
                    if (!(ok = wait_prev_pv())) break;
                    if (ok0) {
                        tmem_st32(tP, *reinterpret_cast<uint32_t(*)[32]>(&w[0]));
                        stored0 = true;
                    }
                    if (!full) mask_half(H1{});
                    const float rs1 = exps_half(H1{}, m_ref);
                    const bool ok1 = !__any_sync(0xffffffffu, valid && !(rs1 <= kFastSumLimit));
                    if (ok0 && ok1) {
                        rs = rs0 + rs1;
                        tmem_st32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(&w[32]));
                    } else {
                        slow = true;
                    }
                } else {
                    finish_s_load();
                    if (!full) {
                        mask_half(H0{});
                        mask_half(H1{});
                    }
                    if (!(ok = wait_prev_pv())) break;
                }
                if (slow) {
                    float mc[8];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint32_t* x = &s[k >> 1][(k & 1) * 16];
                        float m = max3f(__uint_as_float(x[0]), __uint_as_float(x[1]), __uint_as_float(x[2]));
#pragma unroll
                        for (int i = 3; i < 15; i += 2) m = max3f(m, __uint_as_float(x[i]), __uint_as_float(x[i + 1]));
                        mc[k] = fmaxf(m, __uint_as_float(x[15]));
                    }
                    const float mx = max3f(max3f(mc[0], mc[1], mc[2]), max3f(mc[3], mc[4], mc[5]), fmaxf(mc[6], mc[7]));
                    const float m_new = fmaxf(m_ref, mx * sl2);
                    const bool resc = m_new > m_ref + kRescaleThreshold;
                    const float alpha = resc ? fast_exp2(m_ref - m_new) : 1.f;
                    if (resc) {
                        l *= alpha;
                        m_ref = m_new;
                    }
                    const float m_use = m_ref == -INFINITY ? 0.f : m_ref;
                    rs = exps_half(H0{}, m_use) + exps_half(H1{}, m_use);
                    __syncwarp();
                    if (it > 0 && __any_sync(0xffffffffu, resc)) {
#pragma unroll 1
                        for (int ch = 0; ch < D / 32; ++ch) {
                            uint32_t o[32];
                            tmem_ld32(tO + ch * 32, o);
                            tmem_ld_wait();
#pragma unroll
                            for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                            tmem_st32(tO + ch * 32, o);
                        }
                    }
                    if (stored0) tmem_st_wait();  // the first half's earlier store lands before its rewrite
                    tmem_st32(tP, *reinterpret_cast<uint32_t(*)[32]>(&w[0]));
                    tmem_st32(tP + 32, *reinterpret_cast<uint32_t(*)[32]>(&w[32]));
                }
                l += rs;
                tmem_st_wait();
                tc_fence_before();
                mbar_arrive(&S.p_full);
            }

            // -------------------------------------------------------------- epilogue
            if (ok) ok = mbar_wait(&S.o_done, (n - 1) & 1, abort);
            if (!group_all(ok)) break;
            tc_fence_after();
            const bool direct = c.whole();
            // Direct output: the sink joins the sum, and the row is normalised.
            float f = 1.f, lse_v = 0.f;
            if (direct) {
                const float m = l != 0.f ? m_ref : -INFINITY;
                const float M = fmaxf(m, sg);
                if (M == INFINITY || M == -INFINITY) {
                    f = 0.f;
                    lse_v = M;
                } else {
                    f = l != 0.f ? fast_exp2(m - M) : 0.f;
                    const float Z = l * f + fast_exp2(sg - M);
                    f = l != 0.f ? f / Z : 0.f;
                    lse_v = (M + log2f(Z)) * ATTN_LN2;
                }
            }
            const int row = q_start + node;
            // a run's first segment has the first place, any other the second
            const size_t part = (((size_t)gang * p.hkv + kvh) * 2 + (segs > 0)) * BM + r;
            uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)row * p.hq + h) * D);
            float4* pdst = reinterpret_cast<float4*>(p.part_o + part * D);
            uint32_t* const v_bad = S.v_bad[segs % kBadRing];
            const bool any_bad = __any_sync(0xffffffffu, lane < 2 * kMaxNodes / 32 && v_bad[lane] != 0);
#pragma unroll 1
            for (int ch = 0; ch < D / 32; ++ch) {
                float u[32];
                uint32_t raw[32];
                __syncwarp();  // each row has added its own infinities to the last 32 columns
                tmem_ld32(tO + ch * 32, raw);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = l != 0.f ? __uint_as_float(raw[i]) : 0.f;
                if (valid && any_bad) {
                    // Infinities and NaNs in V of tokens that this row sees.
                    auto add = [&](int t) {
                        const int pg = pages[t >> p.page_shift];
                        const size_t sl = ((size_t)pg << p.page_shift) | (t & ((1 << p.page_shift) - 1));
                        const __nv_bfloat16* v = p.v_cache + (sl * p.hkv + kvh) * D + ch * 32;
#pragma unroll
                        for (int i = 0; i < 32; ++i) {
                            const float x = __bfloat162float(v[i]);
                            if (!(fabsf(x) < INFINITY)) u[i] += x;
                        }
                    };
                    int at = pos;
                    for (int a = node + 1; a > 0; a = up(a), --at)
                        if ((v_bad[(a - 1) >> 5] >> ((a - 1) & 31) & 1u) &&
                            (p.win_last <= 0 || at < p.win_first || at > pos - p.win_last))
                            add(P + a - 1);
                    const int some0 = some_first(p, c.rq);
                    for (int i = max(0, pos + 1 - p.win_last - some0); p.win_last > 0 && i < kMaxNodes; ++i)
                        if (v_bad[(kMaxNodes + i) >> 5] >> (i & 31) & 1u) add(some0 + i);
                }
                if (valid && direct) {
#pragma unroll
                    for (int q = 0; q < 4; ++q) {
                        uint4 wv;
                        wv.x = pack_bf16x2(u[8 * q + 0] * f, u[8 * q + 1] * f);
                        wv.y = pack_bf16x2(u[8 * q + 2] * f, u[8 * q + 3] * f);
                        wv.z = pack_bf16x2(u[8 * q + 4] * f, u[8 * q + 5] * f);
                        wv.w = pack_bf16x2(u[8 * q + 6] * f, u[8 * q + 7] * f);
                        dst[ch * 4 + q] = wv;
                    }
                } else if (valid) {
#pragma unroll
                    for (int q = 0; q < 8; ++q)
                        pdst[ch * 8 + q] = make_float4(u[4 * q], u[4 * q + 1], u[4 * q + 2], u[4 * q + 3]);
                }
            }
            if (valid && direct && p.lse) p.lse[(size_t)h * p.total_q + row] = lse_v;
            if (valid && !direct) p.part_ml[part] = make_float2(l != 0.f ? m_ref : -INFINITY, l);
            __syncwarp();
            if (any_bad) {  // the place is free for a later segment
                asm volatile("bar.sync 1, 128;" ::: "memory");
                if (r < 2 * kMaxNodes / 32) v_bad[r] = 0;
            }
            tc_fence_before();  // O has been read: the next segment's P V may overwrite it
            ++segs;
            left -= ntiles;
        }
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Merges the segments of a row in log-sum-exp form and adds the sink once.  One warp
// per node and kRows query heads of a KV head, whose partial rows are neighbours; lane
// = D / 32 dimensions.  Eight rows a warp keep as many loads in flight; with few rows
// (a wave of warps holds them) a warp has one, and its segments' loads overlap.
// It is bound by latency: one pass loads statistics and partials together, and with few
// rows the place of the partials is worked out while the tree kernel still runs (with
// many, most blocks start when it has ended, and read it).  Two passes, with the place
// read: 7 nodes over 2000 tokens 14.4 us instead of 13.6, 64 nodes over 8000 30.1
// instead of 27.8, 16 requests of 16 nodes 67.9 instead of 65.0.
constexpr int kCombineWarps = 8;

template <int D, int kRows>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const Params p) {
    constexpr int V = D / 32;
    using Vec = typename std::conditional<V == 2, float2, float4>::type;
    const int tid = threadIdx.x, lane = tid & 31, b = blockIdx.y;
    const int blocks = (p.group + kRows - 1) / kRows;  // of a KV head's query heads
    const int idx = blockIdx.x * kCombineWarps + (tid >> 5);
    const int node = idx / (p.hkv * blocks), kvh = idx / blocks % p.hkv, g0 = idx % blocks * kRows;
    const Request rq = request(p, b, false);
    long long before = 0, per_run = 0;  // steps of the requests before this one; of a run
    const bool early = kRows == 1 && p.batch <= kCombineWarps * 32;
    if (early) {
        __shared__ long long sums[kCombineWarps][2];
        long long steps = tid < p.batch ? steps_of(request(p, tid, false)) : 0, earlier = tid < b ? steps : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            steps += __shfl_xor_sync(0xffffffffu, steps, o);
            earlier += __shfl_xor_sync(0xffffffffu, earlier, o);
        }
        if (lane == 0) sums[tid >> 5][0] = steps, sums[tid >> 5][1] = earlier;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < kCombineWarps; ++w) per_run += sums[w][0], before += sums[w][1];
        per_run = run_steps(per_run, p.gangs);
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are complete
    if (!early) before = p.first[b], per_run = p.first[p.batch];
    if (node >= rq.rows) return;
    const int heads = min(kRows, p.group - g0), h0 = kvh * p.group + g0;
    const int mt = node / p.npt, r0 = (node - mt * p.npt) * p.group + g0;
    // The row tile's steps [u0, u1) lie in the runs c0 .. c1.
    const long long u0 = before + (long long)mt * rq.ntiles, u1 = u0 + rq.ntiles;
    const int c0 = (int)(u0 / per_run), c1 = rq.ntiles > 0 ? (int)((u1 - 1) / per_run) : c0 - 1;
    if (c0 == c1) return;  // one run had all of it and wrote the output
    // A run's first segment has the first place, any other the second.
    auto place = [&](int c) { return (((size_t)c * p.hkv + kvh) * 2 + (c == c0 && u0 > c * per_run)) * BM + r0; };
    // Lane k of the first 8 keeps the statistics of row k: the running reference and
    // the sum relative to it, the sink's share included.  An infinite sink takes all.
    const bool has = lane < heads;
    const float sg = has && p.sink ? p.sink[h0 + lane] * ATTN_LOG2E : -INFINITY;
    float M = sg, Z = sg == -INFINITY ? 0.f : 1.f;
    float o[kRows][V] = {};
#pragma unroll(kRows == 1 ? 4 : 2)
    for (int c = c0; c <= c1; ++c) {
        const size_t at = place(c);
        const float2 x = has ? p.part_ml[at + lane] : make_float2(0.f, 0.f);
        Vec u[kRows];
#pragma unroll
        for (int k = 0; k < kRows; ++k)
            if (k < heads) u[k] = reinterpret_cast<const Vec*>(p.part_o + (at + k) * D)[lane];
        float keep = 1.f, w = 0.f;  // factors of what there is and of this segment
        if (x.y != 0.f && sg != INFINITY) {  // else nothing seen in this segment
            const float m = fmaxf(M, x.x);
            keep = Z != 0.f ? fast_exp2(M - m) : 0.f;
            w = fast_exp2(x.x - m);
            Z = Z * keep + x.y * w;
            M = m;
        }
#pragma unroll
        for (int k = 0; k < kRows; ++k) {
            const float fk = __shfl_sync(0xffffffffu, keep, k), fw = __shfl_sync(0xffffffffu, w, k);
            if (k >= heads) continue;
            const float* v = reinterpret_cast<const float*>(&u[k]);
#pragma unroll
            for (int i = 0; i < V; ++i) o[k][i] = o[k][i] * fk + v[i] * fw;
        }
    }
    const float inv = Z != 0.f && sg != INFINITY ? 1.f / Z : 0.f;
    const size_t row = (size_t)rq.q_start + node;
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
        const float f = __shfl_sync(0xffffffffu, inv, k);
        if (k >= heads) continue;
        uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + (row * p.hq + h0 + k) * D + lane * V);
#pragma unroll
        for (int i = 0; i < V; i += 2) dst[i / 2] = f == 0.f ? 0u : pack_bf16x2(o[k][i] * f, o[k][i + 1] * f);
    }
    if (has && p.lse)
        p.lse[(size_t)(h0 + lane) * p.total_q + row] = fabsf(M) == INFINITY ? M : (M + log2f(Z)) * ATTN_LN2;
}

// ---------------------------------------------------------------------------
// Host side.

static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    if (!fn) {
        void* ptr = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault, &q) ==
                cudaSuccess &&
            q == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    }
    return fn;
}

// (rows, heads, D) bf16 as a 3-D map {d, head, row}; one copy is a 128-byte-swizzled
// box of 64 dims, box_heads heads and box_rows rows.
static cudaError_t make_map(CUtensorMap* m, const void* base, int D, int heads, long long rows, int box_heads,
                            int box_rows, std::string* what) {
    auto fn = encode_fn();
    if (!fn) {
        *what = "cuTensorMapEncodeTiled unavailable";
        return cudaErrorNotSupported;
    }
    cuuint64_t dims[3] = {(cuuint64_t)D, (cuuint64_t)heads, (cuuint64_t)rows};
    cuuint64_t strides[2] = {(cuuint64_t)D * 2, (cuuint64_t)D * heads * 2};
    cuuint32_t box[3] = {64u, (cuuint32_t)box_heads, (cuuint32_t)box_rows};
    cuuint32_t estr[3] = {1, 1, 1};
    CUresult r = fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                    CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                    CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    if (r != CUDA_SUCCESS) {
        *what = "cuTensorMapEncodeTiled failed (" + std::to_string((int)r) + ")";
        return cudaErrorInvalidValue;
    }
    return cudaSuccess;
}

Plan make_plan(const Args& a) {
    Plan pl;
    const int slots = num_sms() * (a.head_dim == 64 ? 2 : 1);
    pl.ctas = slots >= a.hkv ? slots / a.hkv * a.hkv : a.hkv;
    pl.part_o_bytes = (size_t)pl.ctas * 2 * BM * a.head_dim * sizeof(float);
    pl.part_ml_bytes = (size_t)pl.ctas * 2 * BM * sizeof(float2);
    pl.first_bytes = ((size_t)a.batch + 1) * sizeof(long long);
    return pl;
}

template <int D>
static cudaError_t launch_d(const Args& a, const Plan& pl, void* scratch, cudaStream_t s, std::string* what) {
    static_assert(sizeof(Smem<64>) <= 113 * 1024, "two CTAs per SM at head dim 64");
    static_assert(sizeof(Smem<128>) + 1024 <= 227 * 1024, "shared memory at head dim 128");
    Params p;
    p.sink = a.sink;
    p.cu_q = a.cu_q;
    p.seqlens_k = a.seqlens_k;
    p.parents = a.parents;
    p.page_table = a.page_table;
    p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.part_o = static_cast<float*>(scratch);
    p.part_ml = reinterpret_cast<float2*>(static_cast<char*>(scratch) + pl.part_o_bytes);
    p.first = reinterpret_cast<long long*>(static_cast<char*>(scratch) + pl.part_o_bytes + pl.part_ml_bytes);
    p.gangs = pl.ctas / a.hkv;
    p.batch = a.batch;
    p.max_pages = a.max_pages;
    p.page_shift = 0;
    while ((1 << p.page_shift) < a.page_size) ++p.page_shift;
    p.seg_shift = p.page_shift < 7 ? p.page_shift : 7;  // segments of min(page_size, 128) rows
    p.num_pages = a.num_pages;
    p.hq = a.hq;
    p.hkv = a.hkv;
    p.group = a.hq / a.hkv;
    p.total_q = a.total_q;
    p.max_q = a.max_seqlen_q;
    p.npt = BM / p.group;
    p.win_first = a.win_first;
    p.win_last = a.win_last;
    p.scale_log2 = a.scale * ATTN_LOG2E;
    CUtensorMap tq, tk, tv;
    cudaError_t e;
    const long long slots = (long long)a.num_pages * a.page_size;
    if ((e = make_map(&tq, a.q, D, a.hq, a.total_q, p.group, p.npt, what)) != cudaSuccess) return e;
    if ((e = make_map(&tk, a.k_cache, D, a.hkv, slots, 1, 1 << p.seg_shift, what)) != cudaSuccess) return e;
    if ((e = make_map(&tv, a.v_cache, D, a.hkv, slots, 1, 1 << p.seg_shift, what)) != cudaSuccess) return e;
    const size_t smem = sizeof(Smem<D>) + (Cfg<D>::kTwoPerSm ? 0 : 1024);
    e = cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
        *what = "smem attribute";
        return e;
    }
    tree_kernel<D><<<pl.ctas, kThreads, smem, s>>>(tq, tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) {
        *what = "launch";
        return e;
    }
    cudaLaunchConfig_t cfg = {};
    const int rows = (long long)a.batch * a.max_seqlen_q * a.hq <= num_sms() * 32 ? 1 : 8;
    const long long warps = (long long)a.max_seqlen_q * a.hkv * ((p.group + rows - 1) / rows);
    cfg.gridDim = dim3((unsigned)((warps + kCombineWarps - 1) / kCombineWarps), a.batch);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = rows == 1 ? cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, 1>, p)
                  : cudaLaunchKernelEx(&cfg, tree_combine_kernel<D, 8>, p);
    if (e != cudaSuccess) *what = "combine launch";
    return e;
}

cudaError_t launch(const Args& a, const Plan& pl, void* scratch, cudaStream_t s, std::string* what) {
    return a.head_dim == 64 ? launch_d<64>(a, pl, scratch, s, what) : launch_d<128>(a, pl, scratch, s, what);
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace tree
}  // namespace attn
