// The 8-bit cache's other side: new rows into codes and scales, and codes back into
// bf16 pages (sm_103a).
//
// Append.  A block of tokens and a KV head share one scale, a power of two:
//     e = the least exponent >= -64 with max|x| <= qmax 2^e   (qmax 448 or 127)
//     code = round(x 2^-e), to nearest, ties to even.
// A power of two costs e4m3 nothing (a floating-point format has the same digits at
// every scale) and int8 less than one bit, and it lets a block that is filled a few
// tokens at a time keep its digits: when a new row needs a larger scale, the rows
// that the block has are brought to it by a shift, which for e4m3 is exact but in its
// subnormals and for int8 rounds by at most one step of the final scale in all
// (half a step of every scale on the way, each half the next).  The block's scale never
// falls while it has tokens, so that codes do not depend on how many calls filled
// it, but for those roundings.
//
// One warp per (block of tokens, KV head, K or V): the largest magnitude and the codes
// come from one read, its rows kept in registers (as many as a block has, so that a long
// block means more bytes in flight and fewer warps).  Bound by memory for a prompt's chunks: 35k
// rows of 8 heads of 128 into int8 in blocks of 32 take 39 us (5.6 TB/s of rows and codes), of 64
// into e4m3 in blocks of 16 26 us; by latency for single tokens (64 requests: 4.8 us).  Staging
// tiles in shared memory, one CTA for several heads, was slower (46 us; 64 with CTAs that stay): the
// steps around a tile cost more instructions than its conversion.
#include "q8.cuh"

#include <limits.h>

#include <type_traits>

namespace attn {
namespace q8 {

constexpr int kAppendWarps = 4;

// 8 fp32 times `inv` as 8 codes.
template <int F>
__device__ __forceinline__ uint2 encode8(const float (&x)[8], float inv) {
    uint2 r;
    if constexpr (F == kE4M3) {
        uint16_t h[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)  // cvt's first operand is the upper half
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h[i]) : "f"(x[2 * i + 1] * inv), "f"(x[2 * i] * inv));
        r.x = h[0] | (uint32_t)h[1] << 16;
        r.y = h[2] | (uint32_t)h[3] << 16;
    } else {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) u[i] = __float_as_uint(fmaf(x[i], inv, 12582912.f));  // 1.5 2^23: the low byte is round(x inv)
        r.x = __byte_perm(__byte_perm(u[0], u[1], 0x0040), __byte_perm(u[2], u[3], 0x0040), 0x5410);
        r.y = __byte_perm(__byte_perm(u[4], u[5], 0x0040), __byte_perm(u[6], u[7], 0x0040), 0x5410);
    }
    return r;
}

template <int F>
__device__ __forceinline__ void decode8(uint2 w, float (&x)[8]) {
    uint32_t h[4];
    quad_to_f16<F>(w.x, h[0], h[1]);
    quad_to_f16<F>(w.y, h[2], h[3]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 f = f16_to_float2(h[i]);
        x[2 * i] = f.x;
        x[2 * i + 1] = f.y;
    }
}

// Exponent of the scale for a largest magnitude `top` (finite, >= 0).
template <int F>
__device__ __forceinline__ int needed_exp(float top) {
    if (!(top > 0.f)) return kMinExp;
    int k;
    const float f = frexpf(top, &k);  // top = f 2^k, 0.5 <= f < 1
    // 448 = 0.875 2^9, 127 = (127/128) 2^7
    const int e = F == kE4M3 ? k - 9 + (f > 0.875f ? 1 : 0) : k - 7 + (f > 0.9921875f ? 1 : 0);
    return e < kMinExp ? kMinExp : e;
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }  // -126 <= e <= 127

// Request b's new rows as the kernels see them: tokens [from, end), row of token t n0 + t - start.
struct NewRows {
    int n0, start, from, end;
    bool some;
};

__device__ __forceinline__ NewRows new_rows(const AppendArgs& a, int b, bool report) {
    NewRows r;
    r.n0 = a.cu_new ? a.cu_new[b] : b;
    const int n = a.cu_new ? a.cu_new[b + 1] - r.n0 : 1;
    const int L = a.seqlens[b];
    r.start = L - n;
    // as in the bf16 append, rows of negative tokens and behind the page table are left out
    const long long cap = (long long)a.c.max_pages * a.c.page_size;
    if (report && n > 0 && (n > a.max_new || r.start < 0 || L > cap || r.n0 + (long long)n > a.total_new))
        raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
    r.from = max(r.start, 0);
    r.end = L < cap ? L : (int)cap;
    if (r.n0 + (long long)n > a.total_new) r.end = min(r.end, r.start + max(0, a.total_new - r.n0));
    if (n > a.max_new) r.end = min(r.end, r.start + a.max_new);
    r.some = r.n0 >= 0 && n > 0 && r.end > r.from;
    return r;
}

// What a block of one head's K or V has in the cache.
template <int D>
struct Block {
    uint8_t* codes;  // of its first token, at this lane's 8 dims
    size_t step;     // from token to token
    float* scale;
    __device__ __forceinline__ Block(const AppendArgs& a, bool is_v, int page, int in_page, int head, int seg) {
        const Cache& c = a.c;
        codes = (is_v ? c.v : c.k) + (((size_t)page * c.page_size + in_page) * c.hkv + head) * D + seg * 8;
        step = (size_t)c.hkv * D;
        scale = (is_v ? c.v_scale : c.k_scale) +
                ((size_t)page * a.blocks + (a.block_shift >= 0 ? in_page >> a.block_shift : in_page / c.block)) * c.hkv + head;
    }
};

// The block's scale and its reciprocal for new rows of largest magnitude `top`, `have` tokens being
// there with scale `old`; if it grows, their codes (rows r0, r0 + step, ..) are brought to it.
template <int D, int F>
__device__ __forceinline__ float2 settle_scale(const Block<D>& k, uint32_t top, int have, float old, int r0, int step) {
    const int e = needed_exp<F>(__uint_as_float(top << 16));
    float2 s = make_float2(exp2i(e), exp2i(-e));
    if (have > 0) {
        if (old >= s.x) {
            s = make_float2(old, 1.f / old);
        } else {
            const float ratio = old > 0.f ? old / s.x : 0.f;
            for (int r = r0; r < have; r += step) {
                uint2* at = reinterpret_cast<uint2*>(k.codes + r * k.step);
                float x[8];
                decode8<F>(*at, x);
                *at = encode8<F>(x, ratio);
            }
        }
    }
    return s;
}

// Codes of 8 bf16.  odd: there may be infinities (the largest code of their sign) and NaNs (0).
template <int F>
__device__ __forceinline__ uint2 codes_of(const uint4& x, float inv, bool odd) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = bf16_lo(w[i]);
        f[2 * i + 1] = bf16_hi(w[i]);
    }
    if (odd) {
        constexpr float kMax = F == kE4M3 ? 448.f : 127.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = isnan(f[i]) ? 0.f : fminf(fmaxf(f[i] * inv, -kMax), kMax);
        inv = 1.f;
    }
    return encode8<F>(f, inv);
}

// The largest magnitudes of the even and the odd of 8 bf16 and of `top`'s, as integers: they keep
// the values' order, infinities and NaNs are kOdd and above.
constexpr uint32_t kOdd = 0x7f80u;
__device__ __forceinline__ uint32_t max_abs8(uint32_t top, const uint4& x) {
    top = __vimax3_u16x2(top, x.x & 0x7fff7fffu, x.y & 0x7fff7fffu);
    return __vimax3_u16x2(top, x.z & 0x7fff7fffu, x.w & 0x7fff7fffu);
}
// The largest finite magnitude of 8 bf16 and `top`.
__device__ __forceinline__ uint32_t max_finite8(uint32_t top, const uint4& x) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint32_t p = w[i] & 0x7fffu, q = (w[i] >> 16) & 0x7fffu;
        if (p < 0x7f80u) top = max(top, p);
        if (q < 0x7f80u) top = max(top, q);
    }
    return top;
}
__device__ __forceinline__ uint32_t warp_max(uint32_t x) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) x = max(x, __shfl_xor_sync(0xffffffffu, x, o));
    return x;
}

// A warp per (block, head, K or V).  kHeld: 16-byte pieces of the rows that a lane keeps in
// registers (those of longer blocks are read again).
template <int D, int F, int kHeld>
__global__ void __launch_bounds__(kAppendWarps * 32, kHeld == 4 ? 8 : kHeld == 8 ? 6 : 4) append_kernel(const AppendArgs a) {
    constexpr int kLanes = D / 8;          // lanes of a row
    constexpr int kRows = 32 / kLanes;     // rows of a warp's instruction
    const Cache& c = a.c;
    const int b = blockIdx.y, lane = threadIdx.x & 31, sub = lane / kLanes, seg = lane % kLanes;
    const uint32_t task = blockIdx.x * kAppendWarps + (threadIdx.x >> 5);
    const bool is_v = task & 1;
    const uint32_t index = (task >> 1) / (uint32_t)c.hkv;
    const int head = (int)((task >> 1) - index * c.hkv);
    const NewRows n = new_rows(a, b, task == 0 && lane == 0);
    const long long t0l = ((a.block_shift >= 0 ? n.from >> a.block_shift : n.from / c.block) + (long long)index) * c.block;
    if (!n.some || t0l >= n.end) return;
    const int t0 = (int)t0l;
    const Place pl = place_of(t0, c.page_size, a.page_shift);
    const int page = c.page_table[(size_t)b * c.max_pages + pl.page];
    const int lo = max(t0, n.from), rows = min(t0 + c.block, n.end) - lo;
    const long long rs = is_v ? a.v_rs : a.k_rs;
    const __nv_bfloat16* src = (is_v ? a.v_new : a.k_new) + (n.n0 + (long long)(lo - n.start)) * rs + head * D + seg * 8;
    src += sub * rs;  // this lane's rows: sub, sub + kRows, ..
    const long long far = kRows * rs;
    uint4 held[kHeld];
    {
        const __nv_bfloat16* x = src;
#pragma unroll
        for (int i = 0; i < kHeld; ++i, x += far)
            held[i] = i * kRows + sub < rows ? __ldcs(reinterpret_cast<const uint4*>(x)) : make_uint4(0, 0, 0, 0);
    }
    auto row = [&](int r) { return __ldg(reinterpret_cast<const uint4*>(src + (r - sub) * rs)); };
    // (the rows are on their way; where they go)
    if ((unsigned)page >= (unsigned)c.num_pages) {
        if (lane == 0) raise_status(ATTN_SINK_DEV_PAGE_OOB);
        return;
    }
    const Block<D> k(a, is_v, page, pl.in_page, head, seg);
    const float old = lo > t0 ? *k.scale : 0.f;
    uint32_t top2 = 0;
#pragma unroll
    for (int i = 0; i < kHeld; ++i) top2 = max_abs8(top2, held[i]);
    for (int r = kHeld * kRows + sub; r < rows; r += kRows) top2 = max_abs8(top2, row(r));
    uint32_t top = warp_max(max(top2 & 0xffffu, top2 >> 16));
    const bool odd = top >= kOdd;
    if (odd) {
        if (lane == 0) raise_status(ATTN_SINK_DEV_VALUE);
        top = 0;
        for (int r = sub; r < rows; r += kRows) top = max_finite8(top, row(r));
        top = warp_max(top);
    }
    const float2 s = settle_scale<D, F>(k, top, lo - t0, old, sub, kRows);
    uint8_t* to = k.codes + (size_t)(lo - t0 + sub) * k.step;
    const size_t pace = kRows * k.step;
    int r = sub;
    if (!odd) {
#pragma unroll
        for (int i = 0; i < kHeld; ++i, r += kRows, to += pace)
            if (i * kRows + sub < rows) *reinterpret_cast<uint2*>(to) = codes_of<F>(held[i], s.y, false);
    }
    for (; r < rows; r += kRows, to += pace) *reinterpret_cast<uint2*>(to) = codes_of<F>(row(r), s.y, odd);
    __syncwarp();  // every lane has read the old one
    if (lane == 0) *k.scale = s.x;
}

cudaError_t launch_append(const AppendArgs& args, cudaStream_t s) {
    if (args.batch == 0 || args.max_new <= 0) return cudaSuccess;
    AppendArgs a = args;
    a.page_shift = shift_of(a.c.page_size);
    a.block_shift = shift_of(a.c.block);
    a.blocks = a.c.page_size / a.c.block;
    // blocks that max_new tokens can touch, wherever they start
    const long long blocks = ((long long)a.max_new + a.c.block - 2) / a.c.block + 1;
    const long long x = (blocks * a.c.hkv * 2 + kAppendWarps - 1) / kAppendWarps;
    if (x > (1LL << 28)) return cudaErrorInvalidConfiguration;  // (its warps are counted in 32 bits)
    const dim3 grid((unsigned)x, a.batch);
    const int rows = a.max_new < a.c.block ? a.max_new : a.c.block, pieces = (rows + 256 / a.c.head_dim - 1) / (256 / a.c.head_dim);
    auto go = [&](auto d, auto f) {
        constexpr int kD = decltype(d)::value, kF = decltype(f)::value;
        if (pieces <= 4) append_kernel<kD, kF, 4><<<grid, kAppendWarps * 32, 0, s>>>(a);
        else if (pieces <= 8) append_kernel<kD, kF, 8><<<grid, kAppendWarps * 32, 0, s>>>(a);
        else append_kernel<kD, kF, 16><<<grid, kAppendWarps * 32, 0, s>>>(a);
        return cudaGetLastError();
    };
    using std::integral_constant;
    if (a.c.head_dim == 64)
        return a.c.format == kE4M3 ? go(integral_constant<int, 64>{}, integral_constant<int, kE4M3>{})
                                   : go(integral_constant<int, 64>{}, integral_constant<int, kInt8>{});
    return a.c.format == kE4M3 ? go(integral_constant<int, 128>{}, integral_constant<int, kE4M3>{})
                               : go(integral_constant<int, 128>{}, integral_constant<int, kInt8>{});
}

// Codes back into bf16, which holds every c 2^e of either format: the tensor-core
// kernels read the result as a paged cache of its own.  Only the 128-key tiles that the
// windows show are written.  20k tokens of 8 heads of 64: 12 us (61 MB, most of the writes into L2).
constexpr int kExpandThreads = 256;
constexpr int kExpandTokens = 32;  // tokens of a block

template <int F>
__global__ void __launch_bounds__(kExpandThreads) expand_kernel(const ExpandArgs a, int page_shift, int block_shift, int blocks) {
    const Cache& c = a.c;
    const int b = blockIdx.y;
    const int q_start = a.cu_q[b], Lq = max(0, a.cu_q[b + 1] - q_start);
    if (a.parents && blockIdx.x == 0)
        for (int i = threadIdx.x; i < Lq; i += kExpandThreads)
            if ((unsigned)(q_start + i) < (unsigned)a.total_q) a.parents[q_start + i] = i - 1;
    const long long cap = min((long long)c.max_pages * c.page_size, (long long)a.pages * kExpandPage);
    int L = a.seqlens[b];
    if (L > cap) {
        if (blockIdx.x == 0 && threadIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        L = (int)cap;
    }
    if (Lq > a.max_q && blockIdx.x == 0 && threadIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
    if (blockIdx.x == 0 && threadIdx.x == 0) a.lens_out[b] = max(L, 0);
    const int t0 = blockIdx.x * kExpandTokens;
    if (Lq == 0 || t0 >= L) return;
    if (a.win_last > 0) {  // no row sees tokens between the first window and the first row's last one
        const long long lo = max(0LL, (long long)L - Lq + 1 - a.win_last);
        if (t0 >= (a.win_first + 127LL) / 128 * 128 && t0 + kExpandTokens <= lo / 128 * 128) return;
    }
    if (threadIdx.x == 0) a.table_out[(size_t)b * a.pages + t0 / kExpandPage] = b * a.pages + t0 / kExpandPage;
    __shared__ int page_of[kExpandTokens], in_of[kExpandTokens];
    if (threadIdx.x < kExpandTokens) {
        const int t = t0 + threadIdx.x;
        int page = -1, in = 0;
        if (t < L) {
            const Place pl = place_of(t, c.page_size, page_shift);
            page = c.page_table[(size_t)b * c.max_pages + pl.page];
            in = pl.in_page;
            if ((unsigned)page >= (unsigned)c.num_pages) {
                raise_status(ATTN_SINK_DEV_PAGE_OOB);
                page = -2;
            }
        }
        page_of[threadIdx.x] = page;
        in_of[threadIdx.x] = in;
    }
    __syncthreads();
    // 8 codes of K and of V a step, kAhead steps' loads in flight.
    constexpr int kAhead = 4;
    const int vec = c.hkv * c.head_dim / 8, shift = c.head_dim == 64 ? 3 : 4;  // 8-code pieces of a row, log2 of a head's
    const int dr = kExpandThreads / vec, dx = kExpandThreads - dr * vec;
    int r = threadIdx.x / vec, x = threadIdx.x - r * vec;
    const int rows = min(kExpandTokens, L - t0);
    uint4* const ko = reinterpret_cast<uint4*>(a.k_out) + ((size_t)b * a.pages * kExpandPage + t0) * vec;
    uint4* const vo = reinterpret_cast<uint4*>(a.v_out) + ((size_t)b * a.pages * kExpandPage + t0) * vec;
    while (r < rows) {
        uint2 w[kAhead][2];
        float sc[kAhead][2];
        int to[kAhead];
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
            to[i] = r < rows ? r * vec + x : -1;
            w[i][0] = w[i][1] = make_uint2(0, 0);
            sc[i][0] = sc[i][1] = 0.f;
            const int page = r < rows ? page_of[r] : -1;
            if (page >= 0) {  // (a bad page: zeros)
                const size_t at = ((size_t)page * c.page_size + in_of[r]) * vec + x;
                const size_t so = ((size_t)page * blocks + (block_shift >= 0 ? in_of[r] >> block_shift : in_of[r] / c.block)) * c.hkv +
                                  (x >> shift);
                w[i][0] = __ldcs(reinterpret_cast<const uint2*>(c.k) + at);
                w[i][1] = __ldcs(reinterpret_cast<const uint2*>(c.v) + at);
                sc[i][0] = c.k_scale[so];
                sc[i][1] = c.v_scale[so];
            }
            r += dr;
            x += dx;
            if (x >= vec) {
                x -= vec;
                ++r;
            }
        }
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
            if (to[i] >= 0) {
#pragma unroll
                for (int kv = 0; kv < 2; ++kv) {
                    float f[8];
                    decode8<F>(w[i][kv], f);
                    uint4 y;
                    y.x = pack_bf16x2(f[0] * sc[i][kv], f[1] * sc[i][kv]);
                    y.y = pack_bf16x2(f[2] * sc[i][kv], f[3] * sc[i][kv]);
                    y.z = pack_bf16x2(f[4] * sc[i][kv], f[5] * sc[i][kv]);
                    y.w = pack_bf16x2(f[6] * sc[i][kv], f[7] * sc[i][kv]);
                    (kv ? vo : ko)[to[i]] = y;
                }
            }
    }
}

cudaError_t launch_expand(const ExpandArgs& a, cudaStream_t s) {
    if (a.batch == 0 || a.pages == 0) return cudaSuccess;
    dim3 grid((unsigned)a.pages * (kExpandPage / kExpandTokens), a.batch);
    const int sh = shift_of(a.c.page_size);
    if (a.c.format == kE4M3) expand_kernel<kE4M3><<<grid, kExpandThreads, 0, s>>>(a, sh, shift_of(a.c.block), a.c.page_size / a.c.block);
    else expand_kernel<kInt8><<<grid, kExpandThreads, 0, s>>>(a, sh, shift_of(a.c.block), a.c.page_size / a.c.block);
    return cudaGetLastError();
}

ATTN_DEFINE_STATUS_ACCESSOR(append_status_word)

}  // namespace q8
}  // namespace attn
