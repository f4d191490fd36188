// Attention over the 8-bit paged cache: one new token a request (decode) or a few
// (drafts in a row), with the sink and the first/last windows (sm_103a).
//
// What it computes, for a query row i with head h of a request:
//     s_t = scale (q_i . kc_t) ks_t,   O = sum_t e^{s_t - M} vs_t vc_t / Z,
//     Z = e^{sink - M} + sum_t e^{s_t - M}
// over the tokens t that the row sees; kc, vc are codes and ks, vs the scales of
// their block of tokens and KV head.
//
// Structure: one CTA per (split of visible tokens, KV head and row tile, request); the
// rows of a tile are (new token, query head of the KV group) pairs, 8 or 16 of them.
//  * Each of the four warps streams 32-token chunks of its own through a ring of
//    shared-memory stages (16-byte cp.async gathers through the page table), so that
//    nothing but the end of the split brings the warps together.
//  * S^T = K q^T and O^T += V^T P^T are small tensor-core products whose A operands
//    are made from the codes in registers: both formats are exact in fp16, and the
//    order of the head dimensions in a product is free, so that a lane takes 16
//    bytes of a token's row as they lie.  q enters as fp16 of a row scaled by a power of
//    two to a largest magnitude in [1, 2): what fp16 loses there is 2^-25 of that.
//  * Scales stay out of the products: ks multiplies the scores; vs is folded into the
//    weights as log2(vs) in the exponent, P = 2^(s log2 e + log2 vs - ref), with the
//    reference kept 7 to 15 below the running maximum of the exponents (it moves, and what came
//    before is rescaled, only where a weight would pass 2^15): P never leaves fp16's range.
//    Its rounding to fp16 is off by at most 2^-11 of a weight (bf16: 2^-8), and among fp16's
//    subnormals, below 2^-21 of the largest, by half their step: at most 2^-32 of the
//    largest.  The denominator sums P / vs, unrounded, in fp32: it loses a token where P falls
//    below 2^-126, which takes V scales 2^100 apart and more, or a share below 2^-33.
//  * The splits are merged in the log-sum-exp sense and the sink is folded in once: by the
//    cluster that they form, through distributed shared memory, where a row has at most 8,
//    by attend_combine_kernel where it has more.
// Bound by HBM: half the bytes of the bf16 cache.  64 requests of 1k to 32k tokens, 64 query
// heads over 8 of 64 (1.2 GB): 207 us, of which the split grid has 200 (6.0 TB/s; the copy's rate is
// 6.8); 32 windows of 8192 tokens, 32 over 8 of 128 (0.54 GB): 97 us.  Warps an SM, 38 KB of
// shared memory a CTA at d 64, tiles of 8 rows: 24 in the e4m3 split grid (80 registers), 20
// in the other seven forms (81 to 96), 12 at d 128: more warps were worth more than more bytes
// in flight (a third stage of the ring: 222 us).
#include "q8.cuh"

#include <cooperative_groups.h>
#include <limits.h>
#include <math.h>

#include <atomic>
#include <type_traits>

namespace cg = cooperative_groups;

namespace attn {
namespace q8 {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTokens = 32;        // tokens of a warp's chunk
constexpr int kGather = 8;         // splits that one cluster holds
// P is at most 2^(kHead + kSlack), and its row's largest at least about 2^kHead.
constexpr float kHead = 7.f, kSlack = 8.f;
constexpr float kNoRef = -1e30f;   // nothing seen yet
constexpr float kMinScale = 5.421010862427522e-20f;  // 2^-64

struct Params {
    Cache c;
    const __nv_bfloat16* q;
    const int32_t* cu_q;
    const int32_t* seqlens;
    const float* sink;
    __nv_bfloat16* out;
    float* lse;
    float* part_o;    // (rows, hq, max_splits, d), un-normalised
    float2* part_ml;  // (rows, hq, max_splits): (reference in log2 units, sum)
    int total_q, hq, group, max_q, max_tokens, win_first, win_last, causal, lse_by_head;
    int page_shift, block_shift, blocks, tiles, split_tokens, max_splits;  // blocks: of a page
    float scale_log2;
};

// One request as the kernels see it.
struct Request {
    int q_start, Lq, L, off;  // off: position of its first row
};

__device__ __forceinline__ Request request_of(const Params& p, int b, bool report) {
    Request r;
    r.q_start = p.cu_q ? p.cu_q[b] : b;
    r.Lq = p.cu_q ? p.cu_q[b + 1] - r.q_start : 1;
    r.L = p.seqlens[b];
    bool bad = r.L > p.max_tokens || r.Lq > p.max_q || r.q_start + (long long)r.Lq > p.total_q || r.q_start < 0;
    r.L = max(0, min(r.L, p.max_tokens));
    // rows past the host's bounds are left alone; the others keep their positions
    r.off = r.L - r.Lq;
    if (r.q_start < 0) r.Lq = 0;
    r.Lq = max(0, min(min(r.Lq, p.max_q), p.total_q - r.q_start));
    if (bad && report) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
    return r;
}

// Tokens that some row of the tile's new tokens [tok0, tok1] sees.
__device__ __forceinline__ Ranges tile_ranges(const Params& p, const Request& r, int tok0, int tok1) {
    Ranges v;
    const int n = p.causal ? max(0, r.off + tok1 + 1) : r.L;
    v.a0 = 0;
    v.b0 = n;
    v.a1 = n;
    v.b1 = n;
    if (p.win_last > 0) {
        v.b0 = min(p.win_first, n);
        v.a1 = (int)max((long long)v.b0, (long long)r.off + tok0 + 1 - p.win_last);
        v.a1 = min(v.a1, n);
    }
    return v;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], const uint32_t (&b)[2]) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b[0]), "r"(b[1]));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ void copy16(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void* src, int bytes) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}

// Byte offset of 16-byte piece `seg` of staged token row t (of a warp's 32).  The pieces
// are permuted so that both readers are free of bank conflicts: 8 rows x 4 pieces (K) and
// 4 rows x 8 lanes (V), with the token order of row_of below.
template <int D>
__device__ __forceinline__ uint32_t stage_off(int t, int seg) {
    if constexpr (D == 64) return t * 64 + ((seg ^ (((t >> 2) & 1) << 1)) << 4);
    return t * 128 + ((seg ^ ((t & 1) << 2) ^ (((t >> 1) & 3) << 1)) << 4);
}

// Staged row (of 8) that row g of a product stands for.
template <int D>
__device__ __forceinline__ int row_of(int g) {
    return D == 64 ? g ^ ((g >> 1) & 1) : g;
}

__device__ __forceinline__ float lg2_approx(float x) {
    float y;
    asm("lg2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_approx(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ float max_g(float x) {  // over lanes with equal lane % 4
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
    x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
    return fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
}
__device__ __forceinline__ float sum_g(float x) {
    x += __shfl_xor_sync(0xffffffffu, x, 4);
    x += __shfl_xor_sync(0xffffffffu, x, 8);
    return x + __shfl_xor_sync(0xffffffffu, x, 16);
}

// The root of the factor 2^x that brings a partial sum to a common reference.  The sums are
// taken against references that kHead and the V scales put below the scores' maximum, so that
// they are large where 2^x may be below fp32's range: it is multiplied in twice.
__device__ __forceinline__ float half_factor(float x) { return fast_exp2(0.5f * x); }

// A row's output from the merged reference, sum and accumulator (an infinite
// reference: nothing seen and no sink, or an infinite sink that takes all the mass).
__device__ __forceinline__ float finish(float M, float Z, float acc, float& lse) {
    if (M == -INFINITY || M == INFINITY) {
        lse = M;
        return 0.f;
    }
    lse = (M + log2f(Z)) * ATTN_LN2;
    return acc / Z;
}

template <int D, int STAGES>
struct Smem {
    static constexpr int kData = 2 * kTokens * D;        // K and V codes of a warp's chunk
    static constexpr int kStage = kData + 3 * kTokens * 4;  // and its tokens' scales and positions
    static constexpr int kBytes = kWarps * (STAGES * kStage + kTokens * 16);
};

// kRows: several new tokens, so that rows see different tokens.  gather: the splits are one
// cluster, which merges them itself.
template <int D, int NT, int STAGES, int F, bool kRows, bool gather>
__global__ void __launch_bounds__(kThreads, NT == 1 ? 0 : D == 64 ? 4 : 3) attend_kernel(const Params p) {
    using SM = Smem<D, STAGES>;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int H = 8 * NT;
    constexpr int kSegs = D / 16;          // 16-byte pieces of a row
    constexpr int kRowsPer = 32 / kSegs;   // rows of a warp's copy instruction
    constexpr int KK = D / 16;             // k steps of S
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

    const Cache& c = p.c;
    const int split = blockIdx.x, b = blockIdx.z;
    const int kvh = blockIdx.y / p.tiles, tile = blockIdx.y % p.tiles;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, cc = lane & 3;

    const Request r = request_of(p, b, tid == 0 && split == 0 && blockIdx.y == 0);
    const int row0 = tile * H, nrows = min(H, r.Lq * p.group - row0);
    if (nrows <= 0) {
        if constexpr (gather) {  // as often as the others of the cluster
            cg::this_cluster().sync();
            cg::this_cluster().sync();
        }
        return;
    }
    const int tok0 = kRows ? row0 / p.group : 0, tok1 = kRows ? (row0 + nrows - 1) / p.group : 0;
    const Ranges vis = tile_ranges(p, r, tok0, tok1);
    const int nvis = visible_count(vis);
    const long long v0l = (long long)split * p.split_tokens;
    if (v0l >= nvis && !gather) return;
    const int v0 = (int)v0l, v1 = (int)min((long long)nvis, v0l + p.split_tokens);
    const int nchunks = (v1 - v0 - warp * kTokens + kWarps * kTokens - 1) / (kWarps * kTokens);  // of this warp

    // Query row, head of tile row j.
    auto row_at = [&](int j, int& tok, int& head) {
        const int x = row0 + j;
        tok = kRows ? x / p.group : 0;
        head = kvh * p.group + (kRows ? x - tok * p.group : x);
    };

    // Tokens up to full_to, and of the last window from full_from on, are seen by every row.
    const int full_to = !p.causal ? INT_MAX : r.off + tok0;
    const int full_from = p.win_last > 0 ? (int)max(0LL, (long long)r.off + tok1 + 1 - p.win_last) : 0;

    uint8_t* const ring = smem + warp * STAGES * SM::kStage;
    const uint32_t ring_at = smem_u32(ring);
    // Copies: lane (row, seg) of an instruction.
    const int my_row = lane / kSegs, my_seg = lane % kSegs;
    const uint8_t* const kb = c.k + (size_t)kvh * D + my_seg * 16;
    const uint8_t* const vb = c.v + (size_t)kvh * D + my_seg * 16;
    const uint32_t row_bytes = (uint32_t)c.hkv * D;
    const int32_t* const pages = c.page_table + (size_t)b * c.max_pages;
    const int n0 = vis.b0, gap = vis.a1 - vis.b0;  // visible token v is token v, behind the first window v + gap
    // Page of this lane's token of a chunk (-1: behind the split's end), one chunk ahead of its
    // copies; and the token's place in the page.
    auto token_at = [&](int chunk) {
        const int v = v0 + (chunk * kWarps + warp) * kTokens + lane;
        return v < v1 ? v + (v >= n0 ? gap : 0) : -1;
    };
    auto page_at = [&](int t) { return t >= 0 ? pages[place_of(t, c.page_size, p.page_shift).page] : -1; };
    auto load = [&](int t, int page, int st) {
        const uint32_t at = ring_at + st * SM::kStage;
        uint32_t slot = 0, sc = kvh;
        bool ok = (unsigned)page < (unsigned)c.num_pages;
        if (ok) {
            const int in = place_of(t, c.page_size, p.page_shift).in_page;
            slot = (uint32_t)page * c.page_size + in;
            sc = p.block_shift >= 0 ? in >> p.block_shift : in / c.block;
        } else if (t >= 0) {
            raise_status(ATTN_SINK_DEV_PAGE_OOB);
            t = -1;
        }
        const size_t so = ok ? ((size_t)page * p.blocks + sc) * c.hkv + kvh : 0;
        const uint32_t meta = at + SM::kData + lane * 4;
        asm volatile("st.shared.s32 [%0], %1;" ::"r"(meta + 2 * kTokens * 4), "r"(t) : "memory");  // -1: takes no weight
        copy4(meta, c.k_scale + so, ok ? 4 : 0);
        copy4(meta + kTokens * 4, c.v_scale + so, ok ? 4 : 0);
        // (the permutation repeats after 8 rows: two instructions at d 128)
        const uint32_t to[2] = {at + stage_off<D>(my_row, my_seg),
                                at + stage_off<D>(my_row + kRowsPer, my_seg) - kRowsPer * D};
        const uint32_t some = __ballot_sync(0xffffffffu, ok);
#pragma unroll
        for (int i = 0; i < kTokens / kRowsPer; ++i) {
            const uint32_t sl = __shfl_sync(0xffffffffu, slot, i * kRowsPer + my_row);
            const int bytes = some == 0xffffffffu || (some >> (i * kRowsPer + my_row) & 1) ? 16 : 0;  // 0: zeros
            const size_t off = (size_t)sl * row_bytes;
            copy16(to[i & 1] + i * kRowsPer * D, kb + off, bytes);
            copy16(to[i & 1] + i * kRowsPer * D + kTokens * D, vb + off, bytes);
        }
    };
    int t_next = token_at(0), page_next = page_at(t_next);
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        const int t = t_next, page = page_next;
        t_next = token_at(s + 1);
        page_next = page_at(t_next);
        if (s < nchunks) load(t, page, s);
        asm volatile("cp.async.commit_group;" ::: "memory");
    }

    // q as the B operand of S^T = K q^T: lane (g, cc) has row g's dims 16 cc .. 16 cc + 15
    // (d 128: and 64 further), k step kk of them 4 kk .. 4 kk + 3.
    uint32_t qf[NT][KK][2];
    float factor[NT][2];  // of this lane's two score columns: softmax scale, q's scale
    int seen_to[NT][2];   // last position that the column's row sees
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        int tok, head;
        row_at(nt * 8 + g, tok, head);
        const bool ok = nt * 8 + g < nrows;
        const uint4* src = reinterpret_cast<const uint4*>(p.q + ((size_t)(r.q_start + (ok ? tok : 0)) * p.hq + (ok ? head : 0)) * D);
        uint32_t w[KK * 2];
#pragma unroll
        for (int i = 0; i < KK / 2; ++i) {  // 8 dims each
            const int at = (i >> 1) * 8 + cc * 2 + (i & 1);
            const uint4 x = ok ? src[at] : make_uint4(0, 0, 0, 0);
            w[4 * i] = x.x;
            w[4 * i + 1] = x.y;
            w[4 * i + 2] = x.z;
            w[4 * i + 3] = x.w;
        }
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < KK * 2; ++i) top = fmaxf(top, fmaxf(fabsf(bf16_lo(w[i])), fabsf(bf16_hi(w[i]))));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
        // exponent of top; rows that are zero or not finite are taken as they are
        int e = (__float_as_int(top) >> 23) - 127;
        if (e == -127 || e == 128) e = 0;
        e = max(-126, min(e, 126));
        const float down = __int_as_float((127 - e) << 23);
#pragma unroll
        for (int i = 0; i < KK * 2; ++i)
            qf[nt][i >> 1][i & 1] = pack_f16x2(bf16_lo(w[i]) * down, bf16_hi(w[i]) * down);
        const float up = p.scale_log2 * __int_as_float((127 + e) << 23);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            factor[nt][i] = __shfl_sync(0xffffffffu, up, (2 * cc + i) * 4);
            if constexpr (kRows) {
                int tk, hd;
                row_at(nt * 8 + 2 * cc + i, tk, hd);
                seen_to[nt][i] = nt * 8 + 2 * cc + i < nrows ? (p.causal ? r.off + tk : r.L - 1) : -1;
            }
        }
    }

    // ref: what the exponents are taken against, kept kHead to kHead + kSlack below the running maximum
    float ref[NT][2], l_run[NT][2], o[KK][NT][4];
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        ref[nt][0] = ref[nt][1] = kNoRef;
        l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < KK; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) o[mt][nt][i] = 0.f;
    }

    // this warp's tokens as the products need them: (ks, log2 vs, 1 / vs, position)
    float4* const ready = reinterpret_cast<float4*>(smem + kWarps * STAGES * SM::kStage) + warp * kTokens;
    for (int chunk = 0, st = 0; chunk < nchunks; ++chunk) {
        asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 2) : "memory");
        __syncwarp();  // the chunk's bytes, copied by all lanes; the stage read last is free
        const uint8_t* const sK = ring + st * SM::kStage;
        const uint8_t* const sV = sK + kTokens * D;
        bool full = true;  // every row sees every token of the chunk
        {
            const float* const meta = reinterpret_cast<const float*>(sK + SM::kData) + lane;
            const float vs = fmaxf(meta[kTokens], kMinScale);
            const int t = __float_as_int(meta[2 * kTokens]);
            ready[lane] = make_float4(meta[0], t >= 0 ? lg2_approx(vs) : -INFINITY, rcp_approx(vs), __int_as_float(t));
            if constexpr (kRows)
                full = __all_sync(0xffffffffu, t <= full_to && (t < p.win_first || t >= full_from));
        }
        {
            const int t = t_next, page = page_next;
            t_next = token_at(chunk + STAGES);
            page_next = page_at(t_next);
            if (chunk + STAGES - 1 < nchunks) load(t, page, st == 0 ? STAGES - 1 : st - 1);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
        __syncwarp();  // `ready` is written
        st = st + 1 == STAGES ? 0 : st + 1;

        float x[2][NT][4];
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) x[tt][nt][i] = 0.f;
            const int ra = tt * 16 + row_of<D>(g);
#pragma unroll
            for (int h = 0; h < D / 64; ++h) {
                const uint4 a = *reinterpret_cast<const uint4*>(sK + stage_off<D>(ra, h * 4 + cc));
                const uint4 d = *reinterpret_cast<const uint4*>(sK + stage_off<D>(ra + 8, h * 4 + cc));
                const uint32_t wa[4] = {a.x, a.y, a.z, a.w}, wd[4] = {d.x, d.y, d.z, d.w};
#pragma unroll
                for (int kk = 0; kk < 4; ++kk) {
                    uint32_t f[4];
                    quad_to_f16<F>(wa[kk], f[0], f[2]);
                    quad_to_f16<F>(wd[kk], f[1], f[3]);
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(x[tt][nt], f, qf[nt][h * 4 + kk]);
                }
            }
        }
        // this lane's tokens: rows ra and ra + 8 of both tiles
        float4 tk[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) tk[i] = ready[(i >> 1) * 16 + (i & 1) * 8 + row_of<D>(g)];
        uint32_t pf[2][NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float y[2][4];
#pragma unroll
            for (int col = 0; col < 2; ++col)
#pragma unroll
                for (int i = 0; i < 4; ++i)  // (tokens without weight have codes of 0 and a log2 vs of -inf)
                    y[col][i] = fmaf(x[i >> 1][nt][(i & 1) * 2 + col], tk[i].x * factor[nt][col], tk[i].y);
            if constexpr (kRows)
                if (!full) {  // (apart: inside the loop above it would be carried as selects)
#pragma unroll
                    for (int col = 0; col < 2; ++col)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int t = __float_as_int(tk[i].w), last = seen_to[nt][col];
                            if (t > last || (p.win_last > 0 && t >= p.win_first && t <= last - p.win_last))
                                y[col][i] = -INFINITY;
                        }
                }
            bool over = false;
#pragma unroll
            for (int col = 0; col < 2; ++col)
                over |= fmaxf(fmaxf(y[col][0], y[col][1]), fmaxf(y[col][2], y[col][3])) > ref[nt][col] + (kHead + kSlack);
            // the reference follows the maximum where a weight would pass 2^(kHead + kSlack)
            if (__any_sync(0xffffffffu, over)) {
#pragma unroll
                for (int col = 0; col < 2; ++col) {
                    const float top = max_g(fmaxf(fmaxf(y[col][0], y[col][1]), fmaxf(y[col][2], y[col][3])));
                    const float r1 = fmaxf(ref[nt][col], top - kHead), al = fast_exp2(ref[nt][col] - r1);
                    ref[nt][col] = r1;
                    l_run[nt][col] *= al;
#pragma unroll
                    for (int mt = 0; mt < KK; ++mt) {
                        o[mt][nt][col] *= al;
                        o[mt][nt][2 + col] *= al;
                    }
                }
            }
            float w[2][4];
#pragma unroll
            for (int col = 0; col < 2; ++col)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    w[col][i] = fast_exp2(y[col][i] - ref[nt][col]);
                    l_run[nt][col] = fmaf(w[col][i], tk[i].z, l_run[nt][col]);
                }
#pragma unroll
            for (int tt = 0; tt < 2; ++tt) {
                pf[tt][nt][0] = transpose8(pack_f16x2(w[0][tt * 2], w[1][tt * 2]));
                pf[tt][nt][1] = transpose8(pack_f16x2(w[0][tt * 2 + 1], w[1][tt * 2 + 1]));
            }
        }
        // O^T (dims x rows) += V^T P^T: lane (g, cc) has dims g D/8 .. of tokens 2cc, 2cc + 1,
        // 2cc + 8, 2cc + 9; product row g of step mt is its dim 2 mt, row g + 8 the next.
#pragma unroll
        for (int tt = 0; tt < 2; ++tt) {
            uint32_t w[4][D / 32];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int t = tt * 16 + (i >> 1) * 8 + row_of<D>(2 * cc + (i & 1));
                if constexpr (D == 64) {
                    const uint2 d = *reinterpret_cast<const uint2*>(sV + stage_off<D>(t, g >> 1) + (g & 1) * 8);
                    w[i][0] = d.x;
                    w[i][1] = d.y;
                } else {
                    const uint4 d = *reinterpret_cast<const uint4*>(sV + stage_off<D>(t, g));
                    w[i][0] = d.x;
                    w[i][1] = d.y;
                    w[i][2] = d.z;
                    w[i][3] = d.w;
                }
            }
#pragma unroll
            for (int j = 0; j < D / 32; ++j) {  // 4 dims each, two steps
                uint32_t f[2][4];
                quad_to_f16<F>(__byte_perm(w[0][j], w[1][j], 0x5140), f[0][0], f[0][1]);
                quad_to_f16<F>(__byte_perm(w[0][j], w[1][j], 0x7362), f[1][0], f[1][1]);
                quad_to_f16<F>(__byte_perm(w[2][j], w[3][j], 0x5140), f[0][2], f[0][3]);
                quad_to_f16<F>(__byte_perm(w[2][j], w[3][j], 0x7362), f[1][2], f[1][3]);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int nt = 0; nt < NT; ++nt) mma_f16(o[2 * j + k][nt], f[k], pf[tt][nt]);
            }
        }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();

    // Merge the four warps through shared memory.
    float* const sm_m = reinterpret_cast<float*>(smem);  // [warp][H]
    float* const sm_l = sm_m + kWarps * H;
    float* const sm_o = sm_l + kWarps * H;               // [warp][H][D]
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int col = 0; col < 2; ++col) {
            const float l = sum_g(l_run[nt][col]);
            const int j = nt * 8 + 2 * cc + col;
            if (g == 0) {
                // (a NaN moves no reference, but its sum is not 0: it is to be seen in the output)
                sm_m[warp * H + j] = ref[nt][col] == kNoRef && l == 0.f ? -INFINITY : ref[nt][col];
                sm_l[warp * H + j] = l;
            }
            float* const dst = sm_o + (warp * H + j) * D + g * (D / 8);
#pragma unroll
            for (int mt = 0; mt < KK; mt += 2)
                *reinterpret_cast<float4*>(dst + 2 * mt) = make_float4(o[mt][nt][col], o[mt][nt][2 + col],
                                                                       o[mt + 1][nt][col], o[mt + 1][nt][2 + col]);
        }
    __syncthreads();
    float* const all_m = sm_o + kWarps * H * D;  // the CTA's: [H], [H], [H][D]
    float* const all_l = all_m + H;
    float* const all_o = all_l + H;
    for (int e = tid; e < nrows * D; e += kThreads) {
        const int j = e / D, dd = e % D;
        float M = -INFINITY;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm_m[w * H + j]);
        const float ref = M == -INFINITY ? 0.f : M;
        float acc = 0.f, l = 0.f;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const float f = half_factor(sm_m[w * H + j] - ref);
            acc += sm_o[(w * H + j) * D + dd] * f * f;
            l += sm_l[w * H + j] * f * f;
        }
        if constexpr (gather) {
            all_o[e] = acc;
            if (dd == 0) {
                all_m[j] = M;
                all_l[j] = l;
            }
        } else {
            int tok, head;
            row_at(j, tok, head);
            const size_t at = ((size_t)(r.q_start + tok) * p.hq + head) * p.max_splits + split;
            p.part_o[at * D + dd] = acc;
            if (dd == 0) p.part_ml[at] = make_float2(M, l);
        }
    }
    if constexpr (gather) {
        cg::cluster_group cluster = cg::this_cluster();
        cluster.sync();
        for (int e = split * kThreads + tid; e < nrows * D; e += p.max_splits * kThreads) {
            const int j = e / D, dd = e % D;
            int tok, head;
            row_at(j, tok, head);
            const size_t row = (size_t)(r.q_start + tok) * p.hq + head;
            const float sg = p.sink ? p.sink[head] * ATTN_LOG2E : -INFINITY;
            float M = sg, m[kGather], l[kGather], x[kGather];
#pragma unroll
            for (int c = 0; c < kGather; ++c) {
                m[c] = -INFINITY;
                if (c < p.max_splits) {
                    m[c] = *cluster.map_shared_rank(all_m + j, c);
                    l[c] = *cluster.map_shared_rank(all_l + j, c);
                    x[c] = *cluster.map_shared_rank(all_o + e, c);
                }
                M = fmaxf(M, m[c]);
            }
            const float ref = M == -INFINITY ? 0.f : M;
            float acc = 0.f, Z = fast_exp2(sg - ref);
#pragma unroll
            for (int c = 0; c < kGather; ++c)
                if (c < p.max_splits) {
                    const float f = half_factor(m[c] - ref);
                    acc += x[c] * f * f;
                    Z += l[c] * f * f;
                }
            float lse;
            p.out[row * D + dd] = __float2bfloat16_rn(finish(M, Z, acc, lse));
            if (p.lse && dd == 0) p.lse[p.lse_by_head ? (size_t)head * p.total_q + r.q_start + tok : row] = lse;
        }
        cluster.sync();  // the others may still read this CTA's sums
    }
}

// A row (query head, new token, request) by W warps of a block, which take its splits in turn, 4 in flight, a
// lane D / 32 dims.
template <int D, int NT, int W>
__global__ void __launch_bounds__(128) attend_combine_kernel(const Params p) {
    constexpr int N = D / 32, kHeads = 4 / W;
    __shared__ float sm[4][D + 2];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, part = warp % W;
    const int head = blockIdx.x * kHeads + warp / W, tok = blockIdx.y, b = blockIdx.z;
    const Request r = request_of(p, b, false);
    if (tok >= r.Lq || (kHeads > 1 && head >= p.hq)) {  // (no grid behind this one starts before attend_kernel has ended)
        asm volatile("griddepcontrol.wait;" ::: "memory");
        return;
    }
    // the splits of the row's tile
    const int x = tok * p.group + head % p.group, row0 = x / (8 * NT) * (8 * NT);
    const int last = min(row0 + 8 * NT, r.Lq * p.group) - 1;
    const int nvis = visible_count(tile_ranges(p, r, row0 / p.group, last / p.group));
    const int nsplit = (int)(((long long)nvis + p.split_tokens - 1) / p.split_tokens);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const size_t row = (size_t)(r.q_start + tok) * p.hq + head, base = row * p.max_splits;
    float M = -INFINITY, Z = 0.f, acc[N] = {};
    for (int s0 = part; s0 < nsplit; s0 += 4 * W) {
        float2 ml[4];
        alignas(16) float o[4][N];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int s = s0 + i * W;
            ml[i] = make_float2(-INFINITY, 0.f);
            if (s < nsplit) {
                ml[i] = p.part_ml[base + s];
                const float* const from = p.part_o + (base + s) * D + lane * N;
                if constexpr (N == 2) *reinterpret_cast<float2*>(o[i]) = *reinterpret_cast<const float2*>(from);
                else *reinterpret_cast<float4*>(o[i]) = *reinterpret_cast<const float4*>(from);
            }
        }
        const float m = fmaxf(M, fmaxf(fmaxf(ml[0].x, ml[1].x), fmaxf(ml[2].x, ml[3].x)));
        const float ref = m == -INFINITY ? 0.f : m, g = half_factor(M - ref);
        M = m;
        Z *= g * g;
#pragma unroll
        for (int k = 0; k < N; ++k) acc[k] *= g * g;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (s0 + i * W < nsplit) {
                const float f = half_factor(ml[i].x - ref);
                Z += ml[i].y * f * f;
#pragma unroll
                for (int k = 0; k < N; ++k) acc[k] += o[i][k] * f * f;
            }
    }
    const float sg = p.sink ? p.sink[head] * ATTN_LOG2E : -INFINITY;
    float lse;
    const size_t lse_at = p.lse_by_head ? (size_t)head * p.total_q + r.q_start + tok : row;
    if constexpr (W == 1) {
        const float m = fmaxf(M, sg), ref = m == -INFINITY ? 0.f : m, f = half_factor(M - ref);
        Z = fast_exp2(sg - ref) + Z * f * f;
#pragma unroll
        for (int k = 0; k < N; k += 2) {
            const float a0 = finish(m, Z, acc[k] * f * f, lse), a1 = finish(m, Z, acc[k + 1] * f * f, lse);
            *reinterpret_cast<uint32_t*>(p.out + row * D + lane * N + k) = pack_bf16x2(a0, a1);
        }
        if (p.lse && lane == 0) p.lse[lse_at] = lse;
    } else {
#pragma unroll
        for (int k = 0; k < N; ++k) sm[warp][lane * N + k] = acc[k];
        if (lane == 0) {
            sm[warp][D] = M;
            sm[warp][D + 1] = Z;
        }
        __syncthreads();
        const int dd = threadIdx.x;
        if (dd >= D) return;
        M = sg;
#pragma unroll
        for (int w = 0; w < W; ++w) M = fmaxf(M, sm[w][D]);
        const float ref = M == -INFINITY ? 0.f : M;
        Z = fast_exp2(sg - ref);
        float a = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) {
            const float f = half_factor(sm[w][D] - ref);
            Z += sm[w][D + 1] * f * f;
            a += sm[w][dd] * f * f;
        }
        p.out[row * D + dd] = __float2bfloat16_rn(finish(M, Z, a, lse));
        if (p.lse && dd == 0) p.lse[lse_at] = lse;
    }
}

// ---------------------------------------------------------------------------
// Host side.

static int max_tokens(const AttendArgs& a) {
    const long long cap = (long long)a.c.max_pages * a.c.page_size;
    return a.max_seqlen < cap ? a.max_seqlen : (int)cap;
}

// One compiled form of attend_kernel.
template <int D_, int NT_, int F_, bool kRows_, bool gather_>
struct Form {
    static constexpr int D = D_, NT = NT_, F = F_;
    static constexpr bool kRows = kRows_, gather = gather_;
    // Two stages and more CTAs rather than three (d 64: 6 of 38 KB instead of 4, 222 -> 212 us on 64
    // requests of 1k to 32k tokens; d 128: 3 instead of 2, 426 -> 406).
    static constexpr int kStages = 2;
    static constexpr int kMerge = (kWarps + (gather ? 1 : 0)) * 8 * NT * (D + 2) * 4;
    static constexpr int kSmem = Smem<D, kStages>::kBytes > kMerge ? Smem<D, kStages>::kBytes : kMerge;
    static auto kernel() { return attend_kernel<D, NT, kStages, F, kRows, gather>; }
};

// f(form) of the form that a call takes.
template <class Fn>
static auto with_form(int head_dim, int nt, int format, bool rows, bool gather, Fn f) {
    auto tail = [&](auto d, auto n, auto fm) {
        constexpr int D = decltype(d)::value, NT = decltype(n)::value, F = decltype(fm)::value;
        if (rows) return gather ? f(Form<D, NT, F, true, true>{}) : f(Form<D, NT, F, true, false>{});
        return gather ? f(Form<D, NT, F, false, true>{}) : f(Form<D, NT, F, false, false>{});
    };
    auto middle = [&](auto d, auto n) {
        return format == kE4M3 ? tail(d, n, std::integral_constant<int, kE4M3>{}) : tail(d, n, std::integral_constant<int, kInt8>{});
    };
    auto head = [&](auto d) {
        return nt == 1 ? middle(d, std::integral_constant<int, 1>{}) : middle(d, std::integral_constant<int, 2>{});
    };
    return head_dim == 64 ? head(std::integral_constant<int, 64>{}) : head(std::integral_constant<int, 128>{});
}

// Shared memory above 48 KB is asked for once per kernel and device.
template <class Kernel>
static cudaError_t allow_smem(Kernel kern, int bytes, std::atomic<uint64_t>& allowed) {
    if (bytes <= 48 << 10) return cudaSuccess;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    const uint64_t bit = dev < 64 ? 1ull << dev : 0;
    if (bit & allowed.load(std::memory_order_relaxed)) return cudaSuccess;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess) allowed.fetch_or(bit, std::memory_order_relaxed);
    return e;
}

template <class Form>
static cudaError_t allow_smem() {
    static std::atomic<uint64_t> allowed{0};  // devices on which the kernel may have its shared memory
    return allow_smem(Form::kernel(), Form::kSmem, allowed);
}

// Clusters of `size` CTAs of a form that `dev`, the current device, holds at once; the driver is asked
// once for each form, size and device.
template <class Form>
static int resident_clusters(int dev, int size) {
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices][kGather + 1];
    int n = dev < kDevices ? known[dev][size].load(std::memory_order_relaxed) : 0;
    if (n > 0) return n;
    cudaError_t e = allow_smem<Form>();
    if (e == cudaSuccess) {
        if (size == 1) {
            e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, Form::kernel(), kThreads, Form::kSmem);
            n *= num_sms();
        } else {
            cudaLaunchConfig_t cfg = {};
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = size;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.gridDim = dim3(size, 32768);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = Form::kSmem;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            e = cudaOccupancyMaxActiveClusters(&n, Form::kernel(), &cfg);
        }
    }
    if (e != cudaSuccess || n < 1) {
        cudaGetLastError();  // (the launch reports what is wrong)
        return 1;
    }
    if (dev < kDevices) known[dev][size].store(n, std::memory_order_relaxed);
    return n;
}

AttendPlan make_plan(const AttendArgs& a) {
    AttendPlan pl;
    const int group = a.hq / a.c.hkv;
    const long long rows = (long long)group * a.max_q;
    const bool several = a.max_q > 1 || !a.causal;
    // What the device holds at once: CTAs of the split grid, clusters that merge.
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) dev = 0;
    auto ctas = [&](int nt) {
        return (long long)with_form(a.c.head_dim, nt, a.c.format, several, false,
                                    [=](auto form) { return resident_clusters<decltype(form)>(dev, 1); });
    };
    auto clusters = [&](int nt, int size) {
        return (long long)with_form(a.c.head_dim, nt, a.c.format, several, true,
                                    [=](auto form) { return resident_clusters<decltype(form)>(dev, size); });
    };
    long long nvis = max_tokens(a);
    if (a.win_last > 0) {  // a tile's rows are at most 16 tokens apart
        const long long w = (long long)a.win_first + a.win_last + (a.max_q > 1 ? 16 : 0);
        nvis = w < nvis ? w : nvis;
    }
    if (nvis < 1) nvis = 1;
    // Rows of a tile: 8 where that leaves all CTAs resident at once (5 new tokens of one request of 2000, 8 heads
    // a KV head: 10.3 us, 16 rows 12.3, 32 14.4), else 16 (drafts of 4 tokens of 16 requests of 1k to 16k:
    // 79 us; 8 rows 110, which read K and V four times; 32 rows, with half the warps, 92; 32 rows by warps that
    // share chunks converted once in shared memory, 100).
    const long long kv = (long long)a.batch * a.c.hkv, least = (nvis + 255) / 256;
    pl.nt = rows <= 8 || (rows <= 4096 && least <= kGather && kv * ((rows + 7) / 8) <= clusters(1, (int)least)) ? 1 : 2;
    pl.tiles = (int)((rows + 8 * pl.nt - 1) / (8 * pl.nt));
    // Splits of 256 to 2048 tokens, in steps of what the CTA's warps take at once: those for which the
    // waves of resident CTAs are shortest, a CTA's start and end counted as kStart tokens
    // (64 requests of 1k to 32k tokens at d 128, 1024 a split: 402 us, 2048: 385; 32 windows of 8192,
    // 4 and 8 splits: 107 us, 5: 99).
    constexpr int kStep = kWarps * kTokens, kStart = 128, kLeast = 256, kMost = 2048;
    const long long units = kv * pl.tiles, slots = ctas(pl.nt);
    long long best = -1;
    for (int sp = kMost; sp >= kLeast; sp -= kStep) {
        const long long n = (nvis + sp - 1) / sp, waves = (units * n + slots - 1) / slots, cost = waves * (sp + kStart);
        if (best < 0 || cost < best) {
            best = cost;
            pl.split_tokens = sp;
            pl.max_splits = (int)n;
        }
    }
    // Few splits that are all resident at once merge as clusters (one launch, no scratch; 5 new tokens
    // of one request of 2000 18.6 -> 14.4 us).  In a batch of several waves the CTAs that end early
    // would wait for their cluster (64 requests of 1k to 16k tokens, 12 heads 162 -> 258 us); clusters that
    // just do not fit cost as much (50 requests of 2000 tokens, d 64: merged 34.0 us, split 28.7).
    pl.gather = pl.max_splits == 1 || (pl.max_splits <= kGather && units <= clusters(pl.nt, pl.max_splits));
    const size_t parts = !pl.gather ? (size_t)a.total_q * a.hq * pl.max_splits : 0;
    pl.part_o_bytes = parts * a.c.head_dim * sizeof(float);
    pl.part_ml_bytes = parts * sizeof(float2);
    return pl;
}

template <class Form>
static cudaError_t run(const Params& p, const AttendArgs& a, const AttendPlan& pl, cudaStream_t s) {
    constexpr int D = Form::D, NT = Form::NT;
    cudaError_t e = allow_smem<Form>();
    if (e != cudaSuccess) return e;
    cudaLaunchAttribute attr[1];
    {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(pl.max_splits, a.c.hkv * pl.tiles, a.batch);
        cfg.blockDim = dim3(kThreads);
        cfg.dynamicSmemBytes = Form::kSmem;
        cfg.stream = s;
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = Form::gather ? pl.max_splits : 1;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        if ((e = cudaLaunchKernelEx(&cfg, Form::kernel(), p)) != cudaSuccess) return e;
    }
    if constexpr (Form::gather) return cudaGetLastError();
    // A row's splits by one warp where the rows alone are 8 warps an SM and have few splits, by four else (8 drafted
    // tokens of 16 requests 133 us, 139 by four; 64 requests of 1k to 32k tokens, 16 splits, 207.9 and 209.2; 12 heads
    // of 64 requests 153.2 and 152.4; beyond the border, 24 splits: decode 285.8 and 285.3, 8 drafted tokens 336 and
    // 341, 32 splits: 392.5 and 392.4; at d 128, where a warp's share of a row is twice as long, 1 to 2 us slower).
    const bool lone = D == 64 && pl.max_splits <= 16 && (long long)a.hq * a.total_q >= 8LL * num_sms();
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(lone ? (a.hq + 3) / 4 : a.hq, a.max_q, a.batch);
    cfg.blockDim = dim3(128);
    cfg.stream = s;
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if constexpr (D == 64)
        if (lone) e = cudaLaunchKernelEx(&cfg, attend_combine_kernel<D, NT, 1>, p);
    if (!lone) e = cudaLaunchKernelEx(&cfg, attend_combine_kernel<D, NT, 4>, p);
    if (e != cudaSuccess) return e;
    return cudaGetLastError();
}

cudaError_t launch_attend(const AttendArgs& a, const AttendPlan& pl, float* part_o, float2* part_ml, cudaStream_t s) {
    if (a.batch == 0 || a.max_q == 0 || a.total_q == 0) return cudaSuccess;
    Params p;
    p.c = a.c;
    p.q = a.q;
    p.cu_q = a.cu_q;
    p.seqlens = a.seqlens;
    p.sink = a.sink;
    p.out = a.out;
    p.lse = a.lse;
    p.part_o = part_o;
    p.part_ml = part_ml;
    p.total_q = a.total_q;
    p.hq = a.hq;
    p.group = a.hq / a.c.hkv;
    p.max_q = a.max_q;
    p.max_tokens = max_tokens(a);
    p.win_first = a.win_first;
    p.win_last = a.win_last;
    p.causal = a.causal;
    p.lse_by_head = a.lse_by_head;
    p.page_shift = shift_of(a.c.page_size);
    p.block_shift = shift_of(a.c.block);
    p.blocks = a.c.page_size / a.c.block;
    p.tiles = pl.tiles;
    p.split_tokens = pl.split_tokens;
    p.max_splits = pl.max_splits;
    p.scale_log2 = a.scale * ATTN_LOG2E;
    return with_form(a.c.head_dim, pl.nt, a.c.format, a.max_q > 1 || !a.causal, pl.gather,
                     [&](auto form) { return run<decltype(form)>(p, a, pl, s); });
}

ATTN_DEFINE_STATUS_ACCESSOR(attend_status_word)

}  // namespace q8
}  // namespace attn
