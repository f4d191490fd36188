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
// The keys of a (request, KV head, row tile) are cut into splits of whole
// 128-key tiles, one CTA each:
//   warp 0      TMA producer: Q once, then the K tiles, page segment by segment
//   warp 1      TMEM allocator, issues S = Q K^T (128 x 128, operands in shared memory)
//   warp 2      TMA producer of the V tiles
//   warp 3      issues O += P V (P read from TMEM)
//   warps 4..7  softmax, one row per thread, in the manner of the paged forward:
//               against a running reference that starts at the sink and moves only
//               when a value exceeds it by 2^64.  The sink itself is added once, at
//               the end.
// With more than one split, un-normalised fp32 partials go through scratch to
// tree_combine_kernel; with one, the CTA writes the output itself.
//
// Masks: prefix tiles that every row sees whole are not masked at all.  In the
// others each thread builds the 128-bit visibility of its row: ranges for the
// prefix, and its ancestors' bits by walking up the parents (bytes in shared
// memory), once per tile.
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
constexpr int kThreads = 256;
// 128 registers per thread at launch, moved from the control warps to the softmax
// warps: 128 * 40 + 128 * 216 = 256 * 128.
constexpr int kRegsCtrl = 40, kRegsSoftmax = 216;
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

template <int D>
struct __align__(1024) Smem {
    uint8_t q[Cfg<D>::kTile];
    uint8_t k[kStages][Cfg<D>::kTile];
    uint8_t v[kStages][Cfg<D>::kTile];
    uint64_t q_full;
    uint64_t k_full[kStages], k_empty[kStages];
    uint64_t v_full[kStages], v_empty[kStages];
    uint64_t s_full, s_free, p_full, o_done;  // one phase per key tile
    uint64_t final_bar, final_pv;
    uint64_t v_fix;    // V tiles that need their rows looked at land here first
    uint64_t v_fixed;  // all of them have been
    uint32_t tmem_base;
    int abort;
    uint32_t v_bad[kMaxNodes / 32];  // nodes whose V row holds an infinity or a NaN
    uint8_t parent[kMaxNodes];       // parent + 1
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
    float* part_o;    // (batch, units, splits, 128, D) fp32, un-normalised
    float2* part_ml;  // (batch, units, splits, 128): (reference in log2 units, sum)
    int max_pages, page_shift, seg_shift, num_pages;
    int hq, hkv, group, total_q, max_q;
    int npt, mtiles;   // nodes per row tile, row tiles of the largest request
    int split_tiles, splits;
    int win_first, win_last;
    float scale_log2;
};

// What a CTA (or a combine warp) derives of its request.
struct Request {
    int q_start, n, L, P;  // first row, nodes, cached tokens, prefix
    int rows;              // nodes that get results
    int ta, tb, ntiles;    // key tiles [0, ta) and [tb, ...), ntiles in all
    int per_split, nsplit;
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
    r.per_split = max(p.split_tiles, (r.ntiles + p.splits - 1) / p.splits);
    r.nsplit = (r.ntiles + r.per_split - 1) / r.per_split;
    return r;
}

// Waits that ignore the abort flag (they drain work in flight before shared
// memory and TMEM are released); still bounded in time.
__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
    int dummy = 0;
    mbar_wait(bar, parity, &dummy);
}

__device__ __forceinline__ bool nonfinite_pair(uint32_t w) {
    return (w & 0x7f80u) == 0x7f80u || (w & 0x7f800000u) == 0x7f800000u;
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
    // Row tiles of one (KV head, split) are neighbours in the grid (they share its
    // K / V in L2), then the KV heads (which share the cache's token rows).
    const int mt = blockIdx.x % p.mtiles;
    const int kvh = blockIdx.x / p.mtiles % p.hkv;
    const int split = blockIdx.x / p.mtiles / p.hkv;
    const int b = blockIdx.y;

    const Request rq = request(p, b, threadIdx.x == 0 && blockIdx.x == 0);
    const int node0 = mt * p.npt;
    if (node0 >= rq.rows) return;
    const bool direct = p.splits == 1;
    const int it0 = split * rq.per_split;
    const int ntiles = min(rq.per_split, rq.ntiles - it0);  // of this CTA
    if (ntiles <= 0 && !(direct && split == 0)) return;
    const int L = rq.L, P = rq.P;
    // Tile `it` of this CTA's list.
    auto tile_of = [&](int it) { return it0 + it < rq.ta ? it0 + it : rq.tb + (it0 + it - rq.ta); };
    const bool drafts = ntiles > 0 && (tile_of(ntiles - 1) + 1) * BN > P;  // the list reaches drafted tokens

    if (threadIdx.x == 0) {
        mbar_init(&S.q_full, 1);
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
        mbar_init(&S.v_fixed, 1);
        S.abort = 0;
        fence_mbar_init();
    }
    if (threadIdx.x < kMaxNodes / 32) S.v_bad[threadIdx.x] = 0;
    for (int i = threadIdx.x; i < min(rq.rows, node0 + p.npt); i += kThreads) {
        int pr = p.parents[rq.q_start + i];
        if (pr < -1 || pr >= i) {
            raise_status(ATTN_SINK_DEV_TREE);
            pr = -1;
        }
        S.parent[i] = (uint8_t)(pr + 1);
    }
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
        if ((warp == 0 || warp == 2) && ntiles > 0) {
            // -------------------------------------------------------- producers
            // Converged warps: lane i resolves the physical slot of the tile's i-th
            // page segment and issues its copies.
            const bool is_k = warp == 0;
            uint64_t* full = is_k ? S.k_full : S.v_full;
            uint64_t* empty = is_k ? S.k_empty : S.v_empty;
            uint8_t* dst0 = is_k ? S.k[0] : S.v[0];
            const CUtensorMap* tm = is_k ? &tm_k : &tm_v;
            const int nseg = BN >> p.seg_shift;
            if (lane == 0) {
                prefetch_tmap(tm);
                if (is_k) {
                    mbar_expect_tx(&S.q_full, (uint32_t)(p.npt * p.group) * (D * 2));
#pragma unroll
                    for (int a = 0; a < C::kAtoms; ++a)
                        tma_load_3d(S.q + a * kAtom, &tm_q, &S.q_full, 64 * a, kvh * p.group, rq.q_start + node0);
                }
            }
            // Rows of a V tile that no row of the request may see enter P V as
            // zeros, whatever the memory holds (a weight of 0 times a NaN would not
            // vanish): rows past the last token, in the window's gap, or read through
            // a bad page id.  A drafted token's infinities and NaNs are zeroed too,
            // and added by the rows that see that token at the end.  Such tiles land on
            // v_fix and are released to the tensor core once they are clean.
            const int gap0 = p.win_last > 0 ? p.win_first : 0;
            const int gap1 = p.win_last > 0 ? min(P, P + 1 - p.win_last) : 0;
            int fixes = 0;
            int it = 0;
            for (; it < ntiles; ++it) {
                const int st = it % kStages;
                if (it >= kStages && !__all_sync(0xffffffffu, mbar_wait(&empty[st], ((it / kStages) - 1) & 1, abort)))
                    break;
                const int j0 = tile_of(it) * BN;
                int slot = 0;
                bool bad = false;
                const int j = j0 + (lane << p.seg_shift);
                if (lane < nseg && j < L) {
                    const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + (j >> p.page_shift));
                    bad = (unsigned)pg >= (unsigned)p.num_pages;
                    if (!bad) slot = (pg << p.page_shift) | (j & ((1 << p.page_shift) - 1));
                    if (bad && is_k) raise_status(ATTN_SINK_DEV_PAGE_OOB);
                }
                const uint32_t bad_segs = __ballot_sync(0xffffffffu, bad);
                const bool fix = !is_k && (j0 + BN > P || bad_segs || (j0 < gap1 && j0 + BN > gap0));
                uint64_t* bar = fix ? &S.v_fix : &full[st];
                if (lane == 0) mbar_expect_tx(bar, kTile);
                __syncwarp();
                if (lane < nseg) {
                    uint8_t* dst = dst0 + st * kTile + ((uint32_t)lane << p.seg_shift) * 128u;
#pragma unroll
                    for (int a = 0; a < C::kAtoms; ++a) tma_load_3d(dst + a * kAtom, tm, bar, 64 * a, kvh, slot);
                }
                if (fix) {
                    const uint32_t parity = fixes++ & 1;
                    if (!__all_sync(0xffffffffu, mbar_wait(&S.v_fix, parity, abort))) break;
                    // Key row r of an atom is the 128 bytes at r * 128 (the swizzle
                    // permutes 16-byte chunks within a row).
                    for (int e = lane; e < (int)(kTile / 16); e += 32) {
                        const int r = (e >> 3) & (BN - 1), t = j0 + r;
                        uint4* cell = reinterpret_cast<uint4*>(dst0 + st * kTile) + e;
                        if (t >= L || (t >= gap0 && t < gap1) || (bad_segs >> (r >> p.seg_shift) & 1u)) {
                            *cell = make_uint4(0u, 0u, 0u, 0u);
                        } else if (t >= P) {
                            const uint4 x = *cell;
                            if (nonfinite_pair(x.x) || nonfinite_pair(x.y) || nonfinite_pair(x.z) || nonfinite_pair(x.w)) {
                                *cell = make_uint4(finite_pair(x.x), finite_pair(x.y), finite_pair(x.z), finite_pair(x.w));
                                if (t - P < kMaxNodes) atomicOr(&S.v_bad[(t - P) >> 5], 1u << ((t - P) & 31));
                            }
                        }
                    }
                    fence_proxy_async_smem();  // the tensor core reads through the async proxy
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&full[st]);
                }
            }
            if (lane == 0) {
                if (!is_k) mbar_arrive(&S.v_fixed);
                // Drain: every copy issued must have landed before the CTA exits.
                if (is_k) drain_wait(&S.q_full, 0);
                if (fixes > 0) drain_wait(&S.v_fix, (fixes - 1) & 1);
                for (int st = 0; st < kStages; ++st) {
                    const int n = it > st ? (it - st + kStages - 1) / kStages : 0;
                    if (n > 0) drain_wait(&full[st], (n - 1) & 1);
                }
            }
            __syncwarp();
        } else if ((warp == 1 || warp == 3) && ntiles > 0) {
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
            if (warp == 1) {
                ok = wait_all(&S.q_full, 0);
                for (int it = 0; ok && it < ntiles; ++it) {
                    if (!(ok = wait_all(&S.k_full[it % kStages], (it / kStages) & 1))) break;
                    if (it > 0 && !(ok = wait_all(&S.s_free, (it - 1) & 1))) break;
                    tc_fence_after();
                    const uint64_t dk = dk0 + (it % kStages) * (kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t o = (kk >> 2) * (kAtom >> 4) + (kk & 3) * 2;
                        umma_ss_e(tmem + cS, dq + o, dk + o, idS, kk > 0);
                    }
                    umma_commit_e(&S.s_full);
                    umma_commit_e(&S.k_empty[it % kStages]);
                }
                umma_commit_e(&S.final_bar);
                drain_wait(&S.final_bar, 0);
            } else {
                for (int it = 0; ok && it < ntiles; ++it) {
                    if (!(ok = wait_all(&S.v_full[it % kStages], (it / kStages) & 1))) break;
                    if (!(ok = wait_all(&S.p_full, it & 1))) break;
                    tc_fence_after();
                    const uint64_t dv = dv0 + (it % kStages) * (kTile >> 4);
#pragma unroll
                    for (int kk = 0; kk < BN / 16; ++kk)
                        umma_ts_e(tmem + cO, tmem + cP + kk * 8, dv + 128 * kk, idO, (it > 0 || kk > 0) ? 1u : 0u);
                    umma_commit_e(&S.o_done);
                    umma_commit_e(&S.v_empty[it % kStages]);
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
        const int node = node0 + r / p.group, g = r % p.group;
        const bool valid = r < p.npt * p.group && node < rq.rows;
        const bool work = __any_sync(0xffffffffu, valid);  // else only the barriers' arrivals
        const int h = kvh * p.group + g;
        const float sg = p.sink && valid ? p.sink[h] * ATTN_LOG2E : -INFINITY;
        const float sl2 = p.scale_log2;
        float m_ref = sg == INFINITY ? -INFINITY : sg;
        float l = 0.f;
        int pos = P;  // this row's position
        if (p.win_last > 0 && valid)
            for (int a = S.parent[node]; a > 0; a = S.parent[a - 1]) ++pos;
        const int pos_max = P + max(rq.n, 1) - 1;  // of any node
        const int nseg = BN >> p.seg_shift;
        // Whether this lane's page segment of a tile is read through a bad page id.
        auto segment_bad = [&](int j0) -> bool {
            const int j = j0 + (lane << p.seg_shift);
            if (lane >= nseg || j >= L) return false;
            const int pg = __ldg(p.page_table + (size_t)b * p.max_pages + (j >> p.page_shift));
            return (unsigned)pg >= (unsigned)p.num_pages;
        };
        bool next_bad = ntiles > 0 && segment_bad(tile_of(0) * BN);
        bool ok = true;
        for (int it = 0; it < ntiles; ++it) {
            const int j0 = tile_of(it) * BN;
            const uint32_t bad_segs = __ballot_sync(0xffffffffu, next_bad);
            if (it + 1 < ntiles) next_bad = segment_bad(tile_of(it + 1) * BN);
            ok = mbar_wait(&S.s_full, it & 1, abort);
            if (!__all_sync(0xffffffffu, ok)) {
                ok = false;
                break;
            }
            tc_fence_after();
            // The previous P V must be complete before P is overwritten or O rescaled.
            auto wait_prev_pv = [&]() -> bool {
                if (it == 0) return true;
                const bool done = __all_sync(0xffffffffu, mbar_wait(&S.o_done, (it - 1) & 1, abort));
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
                    for (int a = node + 1; a > 0; a = S.parent[a - 1], --at) {
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
        if (ok && ntiles > 0) ok = mbar_wait(&S.o_done, (ntiles - 1) & 1, abort);
        if (ok && drafts) ok = mbar_wait(&S.v_fixed, 0, abort);
        ok = __all_sync(0xffffffffu, ok);
        const bool have = ok && ntiles > 0;
        if (have) tc_fence_after();
        const bool store = valid && ok;
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
        const int row = rq.q_start + node;
        const size_t unit = ((size_t)b * p.hkv + kvh) * p.mtiles + mt;
        const size_t part = (unit * p.splits + split) * BM + r;
        uint4* dst = reinterpret_cast<uint4*>(p.out + ((size_t)row * p.hq + h) * D);
        float4* pdst = reinterpret_cast<float4*>(p.part_o + part * D);
#pragma unroll 1
        for (int ch = 0; ch < D / 32; ++ch) {
            float u[32];
            if (have) {  // warp-uniform: every lane takes part in the collective load
                uint32_t raw[32];
                tmem_ld32(tO + ch * 32, raw);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = l != 0.f ? __uint_as_float(raw[i]) : 0.f;
            } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) u[i] = 0.f;
            }
            if (store && drafts) {
                // Infinities and NaNs of drafted tokens' V that this row sees.
                int at = pos;
                for (int a = node + 1; a > 0; a = S.parent[a - 1], --at) {
                    const int t = P + a - 1;
                    if (!(S.v_bad[(a - 1) >> 5] >> ((a - 1) & 31) & 1u)) continue;
                    if (p.win_last > 0 && at >= p.win_first && at <= pos - p.win_last) continue;
                    const int pg = p.page_table[(size_t)b * p.max_pages + (t >> p.page_shift)];
                    const size_t sl = ((size_t)pg << p.page_shift) | (t & ((1 << p.page_shift) - 1));
                    const __nv_bfloat16* v = p.v_cache + (sl * p.hkv + kvh) * D + ch * 32;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        const float x = __bfloat162float(v[i]);
                        if (!(fabsf(x) < INFINITY)) u[i] += x;
                    }
                }
            }
            if (store && direct) {
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    uint4 wv;
                    wv.x = pack_bf16x2(u[8 * c + 0] * f, u[8 * c + 1] * f);
                    wv.y = pack_bf16x2(u[8 * c + 2] * f, u[8 * c + 3] * f);
                    wv.z = pack_bf16x2(u[8 * c + 4] * f, u[8 * c + 5] * f);
                    wv.w = pack_bf16x2(u[8 * c + 6] * f, u[8 * c + 7] * f);
                    dst[ch * 4 + c] = wv;
                }
            } else if (store) {
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    pdst[ch * 8 + c] = make_float4(u[4 * c], u[4 * c + 1], u[4 * c + 2], u[4 * c + 3]);
            }
        }
        if (store && direct && p.lse) p.lse[(size_t)h * p.total_q + row] = lse_v;
        if (store && !direct) p.part_ml[part] = make_float2(l != 0.f ? m_ref : -INFINITY, l);
    }

    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, C::kTmemCols);
    }
}

// Merges the splits of a row in log-sum-exp form and adds the sink once.  One warp
// per (node, query head); lane = D / 32 dimensions.
constexpr int kCombineWarps = 8;

template <int D>
__global__ void __launch_bounds__(kCombineWarps * 32) tree_combine_kernel(const Params p) {
    constexpr int V = D / 32;
    const int lane = threadIdx.x & 31, b = blockIdx.y;
    const int idx = blockIdx.x * kCombineWarps + (threadIdx.x >> 5);  // (node, query head)
    const int node = idx / p.hq, h = idx - node * p.hq;
    const Request rq = request(p, b, false);
    asm volatile("griddepcontrol.wait;" ::: "memory");  // the partials are complete
    if (node >= rq.rows) return;
    const int kvh = h / p.group, mt = node / p.npt;
    const int r = (node - mt * p.npt) * p.group + (h - kvh * p.group);
    const size_t unit = ((size_t)b * p.hkv + kvh) * p.mtiles + mt;
    const float sg = p.sink ? p.sink[h] * ATTN_LOG2E : -INFINITY;
    const float2* ml = p.part_ml + unit * p.splits * BM + r;
    const float* po = p.part_o + (unit * p.splits * BM + r) * D + lane * V;
    float M = sg;
    for (int s = 0; s < rq.nsplit; ++s) M = fmaxf(M, ml[(size_t)s * BM].x);
    float o[V] = {}, lse_v = M;
    if (M != INFINITY && M != -INFINITY) {
        float Z = fast_exp2(sg - M);
#pragma unroll 4
        for (int s = 0; s < rq.nsplit; ++s) {
            const float2 x = ml[(size_t)s * BM];
            if (x.y == 0.f) continue;  // nothing seen in this split
            const float f = fast_exp2(x.x - M);
            Z += x.y * f;
#pragma unroll
            for (int v = 0; v < V; ++v) o[v] += po[(size_t)s * BM * D + v] * f;
        }
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] /= Z;
        lse_v = (M + log2f(Z)) * ATTN_LN2;
    }
    uint32_t* dst = reinterpret_cast<uint32_t*>(p.out + ((size_t)(rq.q_start + node) * p.hq + h) * D + lane * V);
#pragma unroll
    for (int v = 0; v < V; v += 2) dst[v / 2] = pack_bf16x2(o[v], o[v + 1]);
    if (p.lse && lane == 0) p.lse[(size_t)h * p.total_q + rq.q_start + node] = lse_v;
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
    const int group = a.hq / a.hkv;
    pl.npt = BM / group;
    pl.mtiles = (a.max_seqlen_q + pl.npt - 1) / pl.npt;
    // Splits: key tiles per CTA so that one wave covers the work if that is at most
    // 8 tiles each, and otherwise about six waves of at least 8 tiles, so that
    // requests of unequal lengths even out.
    const long long slots = 152LL * (a.head_dim == 64 ? 2 : 1);
    const long long units = (long long)a.batch * a.hkv * pl.mtiles;
    long long keys = a.max_seqlen_k > 0 ? a.max_seqlen_k : 1;
    if (a.win_last > 0 && keys > (long long)a.win_first + a.win_last + a.max_seqlen_q)
        keys = (long long)a.win_first + a.win_last + a.max_seqlen_q;
    const long long tiles = (keys + BN - 1) / BN;
    const long long one_wave = (tiles * units + slots - 1) / slots;
    const long long six_waves = (tiles * units + 6 * slots - 1) / (6 * slots);
    long long per = one_wave <= 8 ? one_wave : six_waves < 8 ? 8 : six_waves;
    if (per > tiles) per = tiles;
    pl.split_tiles = (int)per;
    pl.splits = (int)((tiles + per - 1) / per);
    pl.part_o_bytes = pl.splits > 1 ? (size_t)units * pl.splits * BM * a.head_dim * sizeof(float) : 0;
    pl.part_ml_bytes = pl.splits > 1 ? (size_t)units * pl.splits * BM * sizeof(float2) : 0;
    return pl;
}

template <int D>
static cudaError_t launch_d(const Args& a, const Plan& pl, float* part_o, float2* part_ml, cudaStream_t s,
                            std::string* what) {
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
    p.part_o = part_o;
    p.part_ml = part_ml;
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
    p.npt = pl.npt;
    p.mtiles = pl.mtiles;
    p.split_tiles = pl.split_tiles;
    p.splits = pl.splits;
    p.win_first = a.win_first;
    p.win_last = a.win_last;
    p.scale_log2 = a.scale * ATTN_LOG2E;
    CUtensorMap tq, tk, tv;
    cudaError_t e;
    const long long slots = (long long)a.num_pages * a.page_size;
    if ((e = make_map(&tq, a.q, D, a.hq, a.total_q, p.group, pl.npt, what)) != cudaSuccess) return e;
    if ((e = make_map(&tk, a.k_cache, D, a.hkv, slots, 1, 1 << p.seg_shift, what)) != cudaSuccess) return e;
    if ((e = make_map(&tv, a.v_cache, D, a.hkv, slots, 1, 1 << p.seg_shift, what)) != cudaSuccess) return e;
    const size_t smem = sizeof(Smem<D>) + (Cfg<D>::kTwoPerSm ? 0 : 1024);
    e = cudaFuncSetAttribute(tree_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) {
        *what = "smem attribute";
        return e;
    }
    const dim3 grid((unsigned)((long long)pl.splits * a.hkv * pl.mtiles), a.batch);
    tree_kernel<D><<<grid, kThreads, smem, s>>>(tq, tk, tv, p);
    if ((e = cudaGetLastError()) != cudaSuccess) {
        *what = "launch";
        return e;
    }
    if (pl.splits == 1) return cudaSuccess;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)a.max_seqlen_q * a.hq + kCombineWarps - 1) / kCombineWarps), a.batch);
    cfg.blockDim = dim3(kCombineWarps * 32);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, tree_combine_kernel<D>, p);
    if (e != cudaSuccess) *what = "combine launch";
    return e;
}

cudaError_t launch(const Args& a, const Plan& pl, float* part_o, float2* part_ml, cudaStream_t s, std::string* what) {
    return a.head_dim == 64 ? launch_d<64>(a, pl, part_o, part_ml, s, what)
                            : launch_d<128>(a, pl, part_o, part_ml, s, what);
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace tree
}  // namespace attn
