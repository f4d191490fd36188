// Rotary positions (sm_103a): rotates pairs of a head's first r dimensions by an
// angle proportional to the row's position, optionally writing the rotated
// keys and the values straight into a paged cache.
//
// What it computes: pair i of a head (elements i and i + r/2 of the half layout,
// 2i and 2i + 1 of the interleaved one) becomes
//     u = m (x cos a - y sin a),   w = m (y cos a + x sin a),   a = p f_i,
// p the row's position, f_i the pair's inverse frequency and m a factor on the
// rotated part; dimensions r .. d-1 are copied.  The gradient is the rotation by
// -a with the same factor (`inverse`).
//
// The angle: f_i / 2 pi is kept as a 64-bit fixed-point fraction of a turn, so
// that p f_i modulo one turn is one wrapping 64-bit integer product, exact for
// every int32 position (a fp32 product is 0.06 rad off at position 10^6), and
// the range reduction of sine and cosine is the wrap itself.  The top 32 bits
// (1.5e-9 rad) go to sincospif.
//
// It is bound by memory: every input element is read once and every output
// element written once.  A block takes a few rows: it computes their r/2 sines
// and cosines once into shared memory, for all heads, and then moves units of
// 16 elements (8 pairs) with 16-byte loads and stores.
#include "common.cuh"
#include "rope.h"

namespace attn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;  // rows per block

struct Unit {
    uint32_t a[4], b[4];
};

__device__ __forceinline__ void ld16(uint32_t (&r)[4], const __nv_bfloat16* p) {
    const uint4 v = *reinterpret_cast<const uint4*>(p);
    r[0] = v.x, r[1] = v.y, r[2] = v.z, r[3] = v.w;
}
__device__ __forceinline__ void st16(__nv_bfloat16* p, const uint32_t (&r)[4]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(r[0], r[1], r[2], r[3]);
}

// How a unit's 16 elements lie in its head.
enum Layout { kHalfVec, kInterleaved, kHalfScalar };

// Unit u of a head holds pair slots 8u .. 8u + 7.  Slots below h = r/2 are the
// rotated pairs; slot p >= h stands for the two copied elements 2p and 2p + 1.
//   kHalfVec (h a multiple of 8): the unit is elements 8u and 8u + h, 8 each, or
//     16 copied elements at 16u.
//   kInterleaved: the unit is elements 16u .. 16u + 15.
//   kHalfScalar (any h): pair by pair.
template <Layout kL>
__device__ __forceinline__ void load_unit(Unit& x, const __nv_bfloat16* head, int u, int h) {
    if constexpr (kL == kHalfScalar) {
        const uint16_t* e = reinterpret_cast<const uint16_t*>(head);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = 8 * u + j;
            const uint32_t lo = p < h ? e[p] : e[2 * p], hi = p < h ? e[p + h] : e[2 * p + 1];
            if (j & 1) {
                x.a[j >> 1] |= lo << 16;
                x.b[j >> 1] |= hi << 16;
            } else {
                x.a[j >> 1] = lo;
                x.b[j >> 1] = hi;
            }
        }
    } else {
        const bool split = kL == kHalfVec && 8 * u < h;
        const int o = split ? 8 * u : 16 * u;
        ld16(x.a, head + o);
        ld16(x.b, head + o + (split ? h : 8));
    }
}

template <Layout kL>
__device__ __forceinline__ void store_unit(const Unit& x, __nv_bfloat16* head, int u, int h) {
    if constexpr (kL == kHalfScalar) {
        uint16_t* e = reinterpret_cast<uint16_t*>(head);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = 8 * u + j;
            const int sh = (j & 1) * 16;
            e[p < h ? p : 2 * p] = (uint16_t)(x.a[j >> 1] >> sh);
            e[p < h ? p + h : 2 * p + 1] = (uint16_t)(x.b[j >> 1] >> sh);
        }
    } else {
        const bool split = kL == kHalfVec && 8 * u < h;
        const int o = split ? 8 * u : 16 * u;
        st16(head + o, x.a);
        st16(head + o + (split ? h : 8), x.b);
    }
}

// Rotates the unit's slots below h; the others keep their bits (a copied
// element may be an infinity or a NaN).
template <Layout kL>
__device__ __forceinline__ void rotate_unit(Unit& x, const float2* cs, int u, int h) {
    if constexpr (kL == kInterleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int p = 8 * u + j;
            if (p < h) {
                uint32_t& w = j < 4 ? x.a[j] : x.b[j - 4];
                const float2 c = cs[p];
                const float e = bf16_lo(w), o = bf16_hi(w);
                w = pack_bf16x2(e * c.x - o * c.y, o * c.x + e * c.y);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int p = 8 * u + 2 * j;
            if (p < h) {
                const float2 c0 = cs[p], c1 = cs[p + 1 < h ? p + 1 : p];
                const float e0 = bf16_lo(x.a[j]), e1 = bf16_hi(x.a[j]);
                const float o0 = bf16_lo(x.b[j]), o1 = bf16_hi(x.b[j]);
                const uint32_t a = pack_bf16x2(e0 * c0.x - o0 * c0.y, e1 * c1.x - o1 * c1.y);
                const uint32_t b = pack_bf16x2(o0 * c0.x + e0 * c0.y, o1 * c1.x + e1 * c1.y);
                const uint32_t keep = p + 1 < h ? 0u : 0xffff0000u;  // an odd h: slot h is copied
                x.a[j] = (x.a[j] & keep) | (a & ~keep);
                x.b[j] = (x.b[j] & keep) | (b & ~keep);
            }
        }
    }
}

// Grid (row tiles of the longest request, requests); without caches one
// "request" holds all rows.  heads_mul = ceil(2^32 / heads) (0: one head) turns
// the division of a unit's index by the number of heads into a multiplication.
template <int D, Layout kL, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args p, int tile, uint32_t heads_mul) {
    extern __shared__ float2 cs[];  // (tile, h)
    __shared__ long long slot[kMaxRows];
    constexpr int U = D / 16;
    constexpr int kLogU = U == 4 ? 2 : 3;
    const int h = p.rotary_dim / 2;
    const int b = blockIdx.y;
    int n0 = 0, n = p.rows;
    if constexpr (kAppend) {
        n0 = p.cu_new ? p.cu_new[b] : b;
        n = p.cu_new ? p.cu_new[b + 1] - n0 : 1;
    }
    const int r0 = blockIdx.x * tile;
    if constexpr (kAppend) {
        // rows past the grid or past the tensors' end stay untouched
        const bool over = n > (long long)gridDim.x * tile || n0 < 0 || (long long)n0 + n > p.rows;
        if (over && blockIdx.x == 0 && threadIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        if (n0 < 0) return;
        n = (int)min((long long)n, (long long)p.rows - n0);
    }
    const int m = min(tile, n - r0);
    if (m <= 0) return;

    int L = 0;
    if constexpr (kAppend) {
        L = p.seqlens[b];
        const int n_all = p.cu_new ? p.cu_new[b + 1] - n0 : 1;
        if (threadIdx.x < m) {
            const int t = L - n_all + r0 + (int)threadIdx.x;
            long long sl = -1;
            if (t < 0 || t / p.page_size >= p.max_pages) {
                raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
            } else {
                const int pg = p.page_table[(size_t)b * p.max_pages + t / p.page_size];
                if (pg < 0 || pg >= p.num_pages)
                    raise_status(ATTN_SINK_DEV_PAGE_OOB);
                else
                    sl = (long long)pg * p.page_size + t % p.page_size;
            }
            slot[threadIdx.x] = sl;
        }
        L -= n_all;
    }
    for (int e = threadIdx.x; e < m * h; e += kThreads) {
        const int r = e / h, i = e - r * h;
        const int pos = p.positions ? p.positions[n0 + r0 + r] : L + r0 + r;
        const double f = p.inv_freq[i] * 0.15915494309189535;  // turns per position
        const unsigned long long turn = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
        const int a = (int)(uint32_t)((turn * (unsigned long long)(long long)pos) >> 32);
        float sn, cn;
        sincospif((float)a * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: half turns
        if (p.inverse) sn = -sn;
        cs[e] = make_float2(cn * p.attn_scale, sn * p.attn_scale);
    }
    __syncthreads();

    const int heads = p.hq + (p.k ? p.hkv : 0) + (kAppend ? p.hkv : 0);
    const int total = (m * heads) << kLogU;
    for (int idx = threadIdx.x; idx < total; idx += kThreads) {
        const int u = idx & (U - 1), rh = idx >> kLogU;
        const int r = heads_mul ? (int)__umulhi((uint32_t)rh, heads_mul) : rh, hd = rh - r * heads;
        const long long row = n0 + r0 + r;
        const __nv_bfloat16* src;
        __nv_bfloat16* dst;
        bool turn = true;
        if (hd < p.hq) {
            src = p.q + row * p.q_rs + hd * D;
            dst = p.q_out + row * p.q_out_rs + hd * D;
        } else if (hd < p.hq + p.hkv) {
            const int kh = hd - p.hq;
            src = p.k + row * p.k_rs + kh * D;
            if constexpr (kAppend) {
                if (slot[r] < 0) continue;
                dst = p.k_cache + ((size_t)slot[r] * p.hkv + kh) * D;
            } else {
                dst = p.k_out + row * p.k_out_rs + kh * D;
            }
        } else {
            const int vh = hd - p.hq - p.hkv;
            if (slot[r] < 0) continue;
            src = p.v + row * p.v_rs + vh * D;
            dst = p.v_cache + ((size_t)slot[r] * p.hkv + vh) * D;
            turn = false;
        }
        Unit x;
        load_unit<kL>(x, src, u, h);
        if (turn) rotate_unit<kL>(x, cs + r * h, u, h);
        store_unit<kL>(x, dst, u, h);
    }
}

template <int D, Layout kL>
static cudaError_t launch_d(const Args& a, cudaStream_t s) {
    const bool append = a.page_table != nullptr;
    const int heads = a.hq + (a.k ? a.hkv : 0) + (append ? a.hkv : 0);
    const long long longest = append ? a.max_new : a.rows;
    // Rows per block: one until every SM has several blocks, then up to eight.
    int tile = a.rows / (152 * 8);
    tile = tile < 1 ? 1 : tile > kMaxRows ? kMaxRows : tile;
    const dim3 grid((unsigned)((longest + tile - 1) / tile), append ? a.batch : 1);
    const size_t smem = (size_t)tile * (a.rotary_dim / 2) * sizeof(float2);
    const uint32_t mul = heads == 1 ? 0u : (uint32_t)(((1ull << 32) + heads - 1) / heads);
    if (append)
        rope_kernel<D, kL, true><<<grid, kThreads, smem, s>>>(a, tile, mul);
    else
        rope_kernel<D, kL, false><<<grid, kThreads, smem, s>>>(a, tile, mul);
    return cudaGetLastError();
}

cudaError_t launch(const Args& a, cudaStream_t s) {
    const Layout l = a.interleaved ? kInterleaved : a.rotary_dim % 16 == 0 ? kHalfVec : kHalfScalar;
    if (a.head_dim == 64)
        return l == kInterleaved ? launch_d<64, kInterleaved>(a, s)
               : l == kHalfVec   ? launch_d<64, kHalfVec>(a, s)
                                 : launch_d<64, kHalfScalar>(a, s);
    return l == kInterleaved ? launch_d<128, kInterleaved>(a, s)
           : l == kHalfVec   ? launch_d<128, kHalfVec>(a, s)
                             : launch_d<128, kHalfScalar>(a, s);
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace rope
}  // namespace attn
