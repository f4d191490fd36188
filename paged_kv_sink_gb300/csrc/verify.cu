// Verification of drafted tokens against the target's probabilities (sm_103a).
//
// A request's nodes are its last sampled token (node 0, which stands) and the drafted
// ones; p_i and q_i are the target's and the draft model's probabilities of the token
// after node i.  From node i, its children are tested in order.  The r-th, with
// token x and its random number u, is taken if
//     u q_i(x) Z_r < max(p_i(x) - S_r q_i(x), 0),    S_0 = 0, Z_0 = 1,
// and refused otherwise:
//     S_{r+1} = S_r + Z_r,   Z_{r+1} = sum_y max(p_i(y) - S_{r+1} q_i(y), 0),
// which is the rule of refused mass, r_{k+1} = max(r_k / Z_k - q, 0) from r_0 = p, written
// so that nothing but two numbers is carried from one sibling to the next.  Without a draft
// model's probabilities (tokens chosen, not drawn) the test is u Z_r < p_i(x) with Z_r =
// 1 - the refused siblings' p_i, whose tokens are then left out.  Where no child is
// taken, the next token is drawn from what is left of p_i: the least x with
//     cum(x) > u' sum.
// Children that are drawn independently from q_i, or are different chosen tokens, leave the
// next tokens distributed as the target's.
//
// Sums are exact: a weight enters them as an integer in units of 2^-44 (two fp32 additions
// of a large constant split it into two integers), so that they depend on no order, every
// CTA finds the same total, and the search of cum(x) cannot miss.  Differences p - S q
// are formed as pairs of fp32, so that a border of cum moves by no more than those units.
// Tests of single tokens are fp64.
//
// One cluster of CTAs per request.  Each CTA walks the tree itself (the nodes' two
// probabilities are gathered up front, by one of them) and the CTAs share the passes over a row, one
// per refused child and one for the drawing, by contiguous slices of the vocabulary; the
// slices' totals are exchanged through distributed shared memory.  CTAs of 256 threads and 64
// registers, so that 64 requests' all run at once.  Bound by latency: a pass over a row of 131072
// takes its warps four loads from HBM in turn.  One request, 8 drafted tokens in a row, 32000 tokens:
// 11.7 us; 64 requests of 131072: 5 drafted in a row 23 us (67 MB of rows, 2.9 TB/s), trees of 8 to 32
// nodes 42, of chosen tokens (bf16, one row each) 18.
#include "verify.h"

#include <cooperative_groups.h>
#include <cuda_fp16.h>

#include <type_traits>

#include "common.cuh"

namespace cg = cooperative_groups;

namespace attn {
namespace verify {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
static_assert(kThreads >= kMaxNodes, "a thread per node");

using u64 = unsigned long long;

template <int T>
struct Elem;
template <>
struct Elem<kF32> {
    using type = float;
    static __device__ __forceinline__ float get(float x) { return x; }
};
template <>
struct Elem<kBF16> {
    using type = __nv_bfloat16;
    static __device__ __forceinline__ float get(__nv_bfloat16 x) { return __bfloat162float(x); }
};
template <>
struct Elem<kF16> {
    using type = __half;
    static __device__ __forceinline__ float get(__half x) { return __half2float(x); }
};

__device__ __forceinline__ float clamp01(float x) { return fminf(fmaxf(x, 0.f), 1.f); }  // NaN: 0

// An fp32 pair hi + lo in [0, 1] as high 2^22 + low units of 2^-44.
struct Fixed {
    uint32_t high;
    int low;
};

__device__ __forceinline__ Fixed to_fixed(float hi, float lo) {
    constexpr float kLow = 7.152557373046875e-07f;  // 1.5 2^-21: its binade's step is 2^-44
    const float t = hi + 2.f;                       // [2, 4): steps of 2^-22
    Fixed f;
    f.high = __float_as_uint(t) - 0x40000000u;
    f.low = __float_as_int((hi - (t - 2.f)) + lo + kLow) - __float_as_int(kLow);
    return f;
}
__device__ __forceinline__ u64 units(u64 high, long long low) { return (high << 22) + (u64)low; }

// What a pass sums: p (K = 0), p - q (K = 1) or p - S q (K = 2), cut at 0.
struct Cover {
    int k;
    float s_hi, s_lo;
};

template <int K>
__device__ __forceinline__ Fixed weight(const Cover& s, float p, float q) {
    p = clamp01(p);
    if constexpr (K == 0) return to_fixed(p, 0.f);
    q = clamp01(q);
    float hi, lo;
    if constexpr (K == 1) {
        hi = p - q;
        lo = -q - (hi - p);  // exact where p >= q
    } else {
        const float m = s.s_hi * q, e = fmaf(s.s_hi, q, -m) + s.s_lo * q;
        const float d = p - m, z = d - p;
        const float rest = ((p - (d - z)) - (m + z)) - e;
        hi = d + rest;
        lo = rest - (hi - d);
    }
    if (!(hi > 0.f)) hi = lo = 0.f;
    return to_fixed(hi, lo);
}

// A warp takes its slice in batches of kBatch elements, as kBatch / 32 / N vectors of N a lane,
// the a-th of them 32 N a elements in.
constexpr int kBatch = 512;
constexpr int kMaxBatches = (1 << 20) / (kMaxCluster * kWarps * kBatch) + 2;  // of a warp

// Elements [v, v + kBatch) of the row from `skew` elements before it; those outside the row
// are 0.
template <int T, int N>
__device__ __forceinline__ void load_batch(const typename Elem<T>::type* row, int skew, int vocab, int v,
                                           float (&x)[kBatch / 32]) {
    using E = typename Elem<T>::type;
    const int lane = threadIdx.x & 31, e0 = v - skew;
    const E* const at = row + (e0 + lane * N);
    if (e0 >= 0 && e0 + kBatch <= vocab) {
        struct alignas(sizeof(E) * N) V {
            E x[N];
        };
        V y[kBatch / 32 / N];
#pragma unroll
        for (int a = 0; a < kBatch / 32 / N; ++a) y[a] = *reinterpret_cast<const V*>(at + a * 32 * N);
#pragma unroll
        for (int a = 0; a < kBatch / 32 / N; ++a)
#pragma unroll
            for (int i = 0; i < N; ++i) x[a * N + i] = Elem<T>::get(y[a].x[i]);
    } else {
#pragma unroll
        for (int a = 0; a < kBatch / 32 / N; ++a)
#pragma unroll
            for (int i = 0; i < N; ++i) {
                const int e = e0 + lane * N + a * 32 * N + i;
                x[a * N + i] = e >= 0 && e < vocab ? Elem<T>::get(at[a * 32 * N + i]) : 0.f;
            }
    }
}

// A drafted token: its parent, its number and its probabilities after the parent; first: taken, if
// no sibling was refused before.
struct Node {
    int parent, token;
    float u, px, qx;
    int first;
};

struct Shared {
    int n, r0;                  // nodes, the request's first row
    Node node[kMaxNodes];
    int path[kMaxNodes];
    int gone[kMaxNodes];        // refused siblings' tokens (without draft probabilities)
    u64 part[kWarps][kMaxBatches];  // the batches' sums of the last pass
    u64 warp[kWarps];               // the warps'
    u64 total[2][kMaxCluster];      // the CTAs'
    // what the walk stands at
    int at, count, refused, ngone, more;
    float s_hi, s_lo;
};

// A warp's elements of a row, counted from the row's last vector border: whole batches.
// wide: p and q lie alike to such a border, so that both are read as vectors.
struct Slice {
    int v0, v1, skew;
    bool wide;
};

template <class E>
__device__ __forceinline__ Slice slice_of(const E* p, const E* q, int vocab, int ctas, int who) {
    constexpr int kVec = 16 / sizeof(E);
    Slice s;
    const int sp = (int)(reinterpret_cast<uintptr_t>(p) / sizeof(E) % kVec);
    s.wide = sp == (int)(reinterpret_cast<uintptr_t>(q) / sizeof(E) % kVec);
    s.skew = s.wide ? sp : 0;
    const int span = vocab + s.skew, warps = ctas * kWarps;
    const int len = ((span + warps - 1) / warps + kBatch - 1) / kBatch * kBatch;
    s.v0 = min(span, who * len);
    s.v1 = min(span, s.v0 + len);
    return s;
}

// Sums of this warp's batches into part[]; returns their sum (lane 0).
template <int T, int N, int K>
__device__ __forceinline__ u64 sum_slice(const typename Elem<T>::type* p, const typename Elem<T>::type* q, const Cover& s,
                                         const Slice& sl, int vocab, u64* part) {
    u64 sum = 0;
    for (int v = sl.v0, j = 0; v < sl.v1; v += kBatch, ++j) {
        float x[kBatch / 32], y[kBatch / 32];
        load_batch<T, N>(p, sl.skew, vocab, v, x);
        if (K) load_batch<T, N>(q, sl.skew, vocab, v, y);
        uint32_t high = 0;  // at most kBatch 2^22 over the warp
        int low = 0;
#pragma unroll
        for (int i = 0; i < kBatch / 32; ++i) {
            const Fixed f = weight<K>(s, x[i], K ? y[i] : 0.f);
            high += f.high;
            low += f.low;
        }
        high = __reduce_add_sync(0xffffffffu, high);
        low = __reduce_add_sync(0xffffffffu, low);
        const u64 one = units(high, low);
        sum += one;
        if ((threadIdx.x & 31) == 0) part[j] = one;
    }
    return sum;
}

// The element of the batch at v at which the running sum first exceeds `left`.
template <int T, int N, int K>
__device__ __forceinline__ int find_in_batch(const typename Elem<T>::type* p, const typename Elem<T>::type* q, const Cover& s,
                                             int skew, int vocab, int v, u64 left, const int* gone, int ngone) {
    const int lane = threadIdx.x & 31;
    float x[kBatch / 32], y[kBatch / 32];
    load_batch<T, N>(p, skew, vocab, v, x);
    if (K) load_batch<T, N>(q, skew, vocab, v, y);
#pragma unroll
    for (int a = 0; a < kBatch / 32 / N; ++a) {
        const int e = v - skew + (a * 32 + lane) * N;
        u64 f[N], mine = 0;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const Fixed z = weight<K>(s, x[a * N + i], K ? y[a * N + i] : 0.f);
            f[i] = units(z.high, z.low);
            for (int j = 0; j < ngone; ++j)
                if (gone[j] == e + i) f[i] = 0;
            mine += f[i];
        }
        u64 run = mine;  // inclusive over lanes
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const u64 z = __shfl_up_sync(0xffffffffu, run, o);
            if (lane >= o) run += z;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, run > left);
        if (past) {
            int found = 0;
            u64 z = run - mine;
            bool open = true;
#pragma unroll
            for (int i = 0; i < N; ++i) {
                z += f[i];
                if (open && z > left) {
                    found = e + i;
                    open = false;
                }
            }
            return __shfl_sync(0xffffffffu, found, __ffs(past) - 1);
        }
        left -= __shfl_sync(0xffffffffu, run, 31);
    }
    return -1;
}

// floor(u x) for u in [0, 1).
__device__ __forceinline__ u64 part_of(float u, u64 x) {
    uint32_t b = __float_as_uint(u);
    if (!(u > 0.f)) return 0;  // NaN too
    if (b >= 0x3f800000u) b = 0x3f7fffffu;
    const int e = b >> 23;
    if (e == 0) return 0;  // below 2^-126
    const u64 m = (u64)((b & 0x7fffffu) | 0x800000u) << 40;  // u = m 2^-64 2^(e - 126)
    const u64 y = __umul64hi(m, x);
    const int down = 126 - e;
    return down < 64 ? y >> down : 0;
}

template <int T>
__global__ void __launch_bounds__(kThreads, 4) verify_kernel(const Args a) {
    using E = typename Elem<T>::type;
    constexpr int kVec = 16 / sizeof(E);
    __shared__ Shared S;
    cg::cluster_group cluster = cg::this_cluster();
    const int ctas = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
    const int b = blockIdx.x / ctas, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    // What the walk goes by is read once, by the first CTA, and handed to the others: all take the
    // same steps and meet at the same barriers, whatever else happens to the inputs meanwhile.
    cluster.barrier_arrive();  // this CTA runs
    if (rank == 0) {
        const int r0 = a.cu[b];
        int n = a.cu[b + 1] - r0;
        if (n > a.max_nodes || r0 < 0 || r0 + (long long)n > a.total) {
            if (tid == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
            n = r0 < 0 ? 0 : min(min(n, a.max_nodes), a.total - r0);
        }
        const E* const target = static_cast<const E*>(a.target) + (long long)r0 * a.target_rs;
        const E* const draft = a.draft ? static_cast<const E*>(a.draft) + (long long)r0 * a.draft_rs : nullptr;
        Node k = {};
        if (tid < n) {  // (kThreads >= kMaxNodes)
            const int i = tid;
            int par = i - 1;
            if (a.parents && i > 0) {
                par = a.parents[r0 + i];
                if (par < 0 || par >= i) {
                    raise_status(ATTN_SINK_DEV_TREE);
                    par = -1;
                }
            }
            const int x = i > 0 ? a.tokens[r0 + i] : 0;
            float px = 0.f, qx = 0.f;
            if (i > 0 && par >= 0) {
                if (x >= 0 && x < a.vocab) {
                    px = clamp01(Elem<T>::get(target[par * a.target_rs + x]));
                    if (draft) qx = clamp01(Elem<T>::get(draft[par * a.draft_rs + x]));
                } else {
                    raise_status(ATTN_SINK_DEV_PROB);
                }
            }
            const float u = a.u[r0 + i];
            k.parent = i > 0 ? par : -1;
            k.token = x;
            k.u = u < 0.f ? 0.f : u;
            k.px = px;
            k.qx = qx;
            k.first = (draft ? (double)k.u * qx : (double)k.u) < px;
        }
        cluster.barrier_wait();  // and so do the others
        for (int c = 0; c < ctas; ++c) {
            Shared* const to = cluster.map_shared_rank(&S, c);
            if (tid < n) to->node[tid] = k;
            if (tid == 0) {
                to->n = n;
                to->r0 = r0;
            }
        }
    } else {
        cluster.barrier_wait();
    }
    cluster.sync();
    const int n = S.n, first_row = S.r0;
    if (n <= 0) {
        if (rank == 0) {
            for (int j = tid; j < a.max_nodes; j += kThreads) a.src[(size_t)b * a.max_nodes + j] = -1;
            if (tid == 0) {
                a.counts[b] = 0;
                a.next[b] = -1;
            }
        }
        return;
    }
    const E* const target = static_cast<const E*>(a.target) + (long long)first_row * a.target_rs;
    const E* const draft = a.draft ? static_cast<const E*>(a.draft) + (long long)first_row * a.draft_rs : nullptr;

    // One pass over the slices: the sum over the cluster of what `w` leaves of a node's row,
    // less the tokens in S.gone; the batches' and warps' sums stay in S.part and S.warp, the CTAs'
    // in S.total.
    int passes = 0;
    auto row_at = [&](const E* base, long long rs, int i) { return base + i * rs; };
    auto each_form = [&](bool wide, const Cover& w, auto f) {  // f(vector length, kind of weight)
        using std::integral_constant;
        if (wide) {
            if (w.k == 0) return f(integral_constant<int, kVec>{}, integral_constant<int, 0>{});
            if (w.k == 1) return f(integral_constant<int, kVec>{}, integral_constant<int, 1>{});
            return f(integral_constant<int, kVec>{}, integral_constant<int, 2>{});
        }
        // (p and q that lie differently: few callers, one form)
        return f(integral_constant<int, 1>{}, integral_constant<int, 2>{});
    };
    auto sum_row = [&](int node, const Cover& w, int ngone) {
        const E* const pr = row_at(target, a.target_rs, node);
        const E* const qr = w.k ? row_at(draft, a.draft_rs, node) : pr;
        const Slice sl = slice_of<E>(pr, qr, a.vocab, ctas, rank * kWarps + warp);
        u64 part = each_form(sl.wide, w, [&](auto n, auto k) {
            return sum_slice<T, decltype(n)::value, decltype(k)::value>(pr, qr, w, sl, a.vocab, S.part[warp]);
        });
        if (ngone) __syncwarp();
        for (int j = 0; j < ngone; ++j) {
            const int v = S.gone[j] + sl.skew;
            if (v >= sl.v0 && v < sl.v1) {
                const Fixed f = to_fixed(clamp01(Elem<T>::get(pr[S.gone[j]])), 0.f);
                part -= units(f.high, f.low);
                if (lane == 0) S.part[warp][(v - sl.v0) / kBatch] -= units(f.high, f.low);
            }
        }
        if (lane == 0) S.warp[warp] = part;
        __syncthreads();
        u64* const totals = S.total[passes++ & 1];
        if (tid < ctas) {
            u64 mine = 0;
            for (int i = 0; i < kWarps; ++i) mine += S.warp[i];
            *cluster.map_shared_rank(totals + rank, tid) = mine;
        }
        cluster.sync();
        u64 sum = 0;
        for (int c = 0; c < ctas; ++c) sum += totals[c];
        return sum;
    };

    // The walk.  Warp 0 has its state; what a pass needs goes through shared memory.
    int node = 0, count = 1, scanned = 1, refused = 0, ngone = 0;
    double cover = 0.0, mass = 1.0;
    u64 sum = 0;
    Cover w = {0, 0.f, 0.f};
    for (;;) {
        if (warp == 0) {
            if (lane == 0 && count == 1) S.path[0] = 0;
            bool more = false;  // a child was refused: what is left of the row has to be summed
            while (scanned < n && !more) {
                const int i = scanned + lane;
                const uint32_t kids = __ballot_sync(0xffffffffu, i < n && S.node[i].parent == node);
                if (!kids) {
                    scanned += 32;
                    continue;
                }
                const int c = scanned + __ffs(kids) - 1;
                scanned = c + 1;
                const double px = S.node[c].px, u = S.node[c].u;
                bool take, again = false;
                if (refused + ngone == 0) {
                    take = S.node[c].first;
                } else if (draft) {
                    const double qx = S.node[c].qx;
                    take = u * qx * mass < fmax(px - cover * qx, 0.0);
                } else {  // a token that a sibling has lost is not there again
                    for (int j = lane; j < ngone; j += 32) again |= S.gone[j] == S.node[c].token;
                    again = __any_sync(0xffffffffu, again);
                    take = !again && u * mass < px;
                }
                if (take) {
                    node = c;
                    if (lane == 0) S.path[count] = c;
                    ++count;
                    refused = ngone = 0;
                    cover = 0.0;
                    mass = 1.0;
                } else if (draft) {
                    ++refused;
                    cover += mass;
                    more = true;
                } else if (!again && S.node[c].token >= 0 && S.node[c].token < a.vocab) {
                    if (lane == 0) S.gone[ngone] = S.node[c].token;
                    ++ngone;
                    mass = fmax(mass - px, 0.0);
                }
                __syncwarp();
            }
            if (lane == 0) {
                S.at = node;
                S.count = count;
                S.refused = refused;
                S.ngone = ngone;
                S.more = more;
                S.s_hi = (float)cover;
                S.s_lo = (float)(cover - (double)(float)cover);
            }
        }
        __syncthreads();
        const bool more = S.more;
        if (!more && S.refused > 0) break;  // the last pass's weights are those to draw from
        w = {S.refused < 2 ? S.refused : 2, S.s_hi, S.s_lo};
        sum = sum_row(S.at, w, S.ngone);
        if (!more) break;
        mass = (double)sum * 0x1p-44;
    }
    int nout = S.ngone;
    if (sum == 0 && (w.k || nout)) {  // nothing is left: the target's own row
        w.k = nout = 0;
        sum = sum_row(S.at, w, 0);
    }

    if (rank == 0) {
        const int from = a.base ? a.base[b] : 0;
        for (int j = tid; j < a.max_nodes; j += kThreads)
            a.src[(size_t)b * a.max_nodes + j] = j < S.count ? from + S.path[j] : -1;
        if (tid == 0) a.counts[b] = S.count;
    }
    if (sum == 0) {
        if (rank == 0 && tid == 0) {
            raise_status(ATTN_SINK_DEV_PROB);
            a.next[b] = -1;
        }
        return;
    }
    // The warp whose slice the drawn place lies in.
    u64 left = part_of(a.u_next[b], sum);
    const u64* const totals = S.total[(passes - 1) & 1];
    for (int c = 0; c < rank; ++c) {
        if (left < totals[c]) return;
        left -= totals[c];
    }
    for (int i = 0; i < warp; ++i) {
        if (left < S.warp[i]) return;
        left -= S.warp[i];
    }
    if (left >= S.warp[warp]) return;
    const E* const pr = row_at(target, a.target_rs, S.at);
    const E* const qr = w.k ? row_at(draft, a.draft_rs, S.at) : pr;
    const Slice sl = slice_of<E>(pr, qr, a.vocab, ctas, rank * kWarps + warp);
    int j = 0;
    for (; left >= S.part[warp][j]; ++j) left -= S.part[warp][j];
    const int x = each_form(sl.wide, w, [&](auto n, auto k) {
        return find_in_batch<T, decltype(n)::value, decltype(k)::value>(pr, qr, w, sl.skew, a.vocab, sl.v0 + j * kBatch, left,
                                                                        S.gone, nout);
    });
    if (lane == 0) a.next[b] = x;
}

cudaError_t launch(const Args& a, cudaStream_t s) {
    if (a.batch == 0) return cudaSuccess;
    const int ctas = a.vocab > 4096 ? kMaxCluster : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)a.batch * ctas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ctas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cudaError_t e = a.dtype == kF32    ? cudaLaunchKernelEx(&cfg, verify_kernel<kF32>, a)
                    : a.dtype == kBF16 ? cudaLaunchKernelEx(&cfg, verify_kernel<kBF16>, a)
                                       : cudaLaunchKernelEx(&cfg, verify_kernel<kF16>, a);
    return e != cudaSuccess ? e : cudaGetLastError();
}

ATTN_DEFINE_STATUS_ACCESSOR(status_word)

}  // namespace verify
}  // namespace attn
