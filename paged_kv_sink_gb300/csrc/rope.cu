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
// that p f_i modulo one turn is one wrapping 64-bit integer product that loses
// nothing (a fp32 product is 0.06 rad off at position 10^6), and the range
// reduction of sine and cosine is the wrap itself.  Two roundings are left: f_i / 2 pi is
// formed in fp64, which p multiplies to |p| f_i 2^-52 rad (5e-7 at 2^31 for f_i = 1), and
// the product's top 32 bits become the fp32 argument of sincospif, 24 bits of a half turn or
// 1e-7 rad.  Both lie far below the 2^-8 of the bf16 outputs.
//
// It is bound by memory: every input element is read once and every output
// element written once.  A block takes a few rows: it computes their r/2 sines
// and cosines once into shared memory, for all heads, and moves units of 16
// elements (8 pairs) with 16-byte loads and stores, kBatch units a thread in
// flight.  The first batch is loaded before the angles are computed, so that one
// latency hides the other.  16384 rows of 72 heads of 64 take 48.6 us (6.2 TB/s);
// 35k rows of 48 heads of 128 rotated into a cache 133 us (6.6 TB/s, as fast as a copy;
// with one unit in flight, behind the angles, 218 us).  A decode step's 64 rows take
// 3.7 us, mostly the launch.
#include "common.cuh"
#include "rope.h"

namespace attn {
namespace rope {

constexpr int kThreads = 256;
constexpr int kMaxRows = 8;  // rows per block
constexpr int kBatch = 4;    // units in flight per thread

// How a head is cut into units, each moved by one thread.
//   kHalfVec (half layout, h = r/2 a multiple of 8): 16 elements, the pairs 8u ..
//     8u + 7 (elements 8u and 8u + h, 8 each) or 16 copied elements at 16u.
//   kInterleaved: 16 elements at 16u.
//   kHalfAny (half layout, any h): 8 elements at 8u.  Their partners lie at any
//     alignment in another thread's unit, so a warp, which holds whole heads, passes
//     its units through shared memory.  Pair by pair loads and stores of 2 bytes
//     took 325 us on 16384 rows of 72 heads of 64 (r = 50), this takes 99 us.
enum Layout { kHalfVec, kInterleaved, kHalfAny };

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

// Place of pair p's (cosine, sine) in a row's table: the pairs that the threads of
// a warp read together (the same p % 8) are neighbours.
template <int D>
__device__ __forceinline__ int cs_at(int p) {
    return (p & 7) * (D / 16) + (p >> 3);
}

template <Layout kL>
__device__ __forceinline__ void load_unit(Unit& x, const __nv_bfloat16* head, int u, int h) {
    if constexpr (kL == kHalfAny) {
        ld16(x.a, head + 8 * u);
    } else {
        const bool split = kL == kHalfVec && 8 * u < h;
        const int o = split ? 8 * u : 16 * u;
        ld16(x.a, head + o);
        ld16(x.b, head + o + (split ? h : 8));
    }
}

template <Layout kL>
__device__ __forceinline__ void store_unit(const Unit& x, __nv_bfloat16* head, int u, int h) {
    if constexpr (kL == kHalfAny) {
        st16(head + 8 * u, x.a);
    } else {
        const bool split = kL == kHalfVec && 8 * u < h;
        const int o = split ? 8 * u : 16 * u;
        st16(head + o, x.a);
        st16(head + o + (split ? h : 8), x.b);
    }
}

// Rotates the unit's elements of the first 2h dimensions; the others keep their
// bits (a copied element may be an infinity or a NaN).  `head` is the head's copy in
// shared memory (kHalfAny only).
template <int D, Layout kL>
__device__ __forceinline__ void rotate_unit(Unit& x, const float2* cs, const uint16_t* head, int u, int h) {
    if constexpr (kL == kInterleaved) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            if (8 * u + j < h) {
                uint32_t& w = j < 4 ? x.a[j] : x.b[j - 4];
                const float2 c = cs[j * (D / 16) + u];
                const float e = bf16_lo(w), o = bf16_hi(w);
                w = pack_bf16x2(e * c.x - o * c.y, o * c.x + e * c.y);
            }
        }
    } else if constexpr (kL == kHalfVec) {
        if (8 * u < h) {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 c0 = cs[(2 * j) * (D / 16) + u], c1 = cs[(2 * j + 1) * (D / 16) + u];
                const float e0 = bf16_lo(x.a[j]), e1 = bf16_hi(x.a[j]);
                const float o0 = bf16_lo(x.b[j]), o1 = bf16_hi(x.b[j]);
                x.a[j] = pack_bf16x2(e0 * c0.x - o0 * c0.y, e1 * c1.x - o1 * c1.y);
                x.b[j] = pack_bf16x2(o0 * c0.x + e0 * c0.y, o1 * c1.x + e1 * c1.y);
            }
        }
    } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int e = 8 * u + j;
            if (e < 2 * h) {
                const bool first = e < h;
                const float2 c = cs[cs_at<D>(first ? e : e - h)];
                const float other = __uint_as_float((uint32_t)head[first ? e + h : e - h] << 16);
                uint32_t& w = x.a[j >> 1];
                const float own = (j & 1) ? bf16_hi(w) : bf16_lo(w);
                const float y = first ? own * c.x - other * c.y : own * c.x + other * c.y;
                const uint32_t bits = __bfloat16_as_ushort(__float2bfloat16_rn(y));
                w = (j & 1) ? (w & 0xffffu) | bits << 16 : (w & 0xffff0000u) | bits;
            }
        }
    }
}

// Grid (row tiles of the longest request, requests); without caches one
// "request" holds all rows.  heads_mul = ceil(2^32 / heads) (0: one head) turns
// the division of a unit's index by the number of heads into a multiplication.
template <int D, Layout kL, bool kAppend>
__global__ void __launch_bounds__(kThreads) rope_kernel(const Args p, int tile, uint32_t heads_mul) {
    extern __shared__ float2 cs[];  // (tile, D / 2)
    __shared__ uint4 stage[kL == kHalfAny ? kBatch * kThreads : 1];
    __shared__ long long slot[kMaxRows];
    __shared__ unsigned long long turn[D / 2];
    constexpr int U = kL == kHalfAny ? D / 8 : D / 16;
    constexpr int kLogU = U == 4 ? 2 : U == 8 ? 3 : 4;
    constexpr int kWarpUnits = kBatch * 32;
    const int h = p.rotary_dim / 2;
    const int b = blockIdx.y;
    int n0 = 0, n = p.rows;
    if constexpr (kAppend) {
        n0 = p.cu_new ? p.cu_new[b] : b;
        n = p.cu_new ? p.cu_new[b + 1] - n0 : 1;
    }
    const int r0 = blockIdx.x * tile;
    if constexpr (kAppend) {
        // rows past max_new (the grid covers it rounded up to a tile) or past the tensors' end
        // stay untouched
        const bool over = n > p.max_new || n0 < 0 || (long long)n0 + n > p.rows;
        if (over && blockIdx.x == 0 && threadIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        if (n0 < 0) return;
        n = (int)min((long long)min(n, p.max_new), (long long)p.rows - n0);
    }
    const int m = min(tile, n - r0);
    if (m <= 0) return;

    int t0 = 0;  // logical token of the request's first new row
    if constexpr (kAppend) {
        t0 = p.seqlens[b] - (p.cu_new ? p.cu_new[b + 1] - n0 : 1);
        if (threadIdx.x < m) {
            const int t = t0 + r0 + (int)threadIdx.x;
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
    }
    if (threadIdx.x < h) {
        const double f = p.inv_freq[threadIdx.x] * 0.15915494309189535;  // turns per position
        turn[threadIdx.x] = __double2ull_rz((f - floor(f)) * 18446744073709551616.0);
    }

    const int heads = p.hq + (p.k ? p.hkv : 0) + (kAppend ? p.hkv : 0);
    const int total = (m * heads) << kLogU;
    // Row, head and unit of an index; the source row of that head.
    auto place = [&](int idx, int& r, int& hd) {
        const int rh = idx >> kLogU;
        r = heads_mul ? (int)__umulhi((uint32_t)rh, heads_mul) : rh;
        hd = rh - r * heads;
    };
    auto source = [&](int r, int hd) -> const __nv_bfloat16* {
        const long long row = n0 + r0 + r;
        if (hd < p.hq) return p.q + row * p.q_rs + hd * D;
        hd -= p.hq;
        if (hd < p.hkv) return p.k + row * p.k_rs + hd * D;
        return p.v + row * p.v_rs + (hd - p.hkv) * D;
    };
    for (int base = threadIdx.x; base - (int)threadIdx.x < total; base += kBatch * kThreads) {
        Unit x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int idx = base + i * kThreads;
            if (idx < total) {
                int r, hd;
                place(idx, r, hd);
                load_unit<kL>(x[i], source(r, hd), idx & (U - 1), h);
            }
        }
        if (base == (int)threadIdx.x) {
            __syncthreads();
            for (int e = threadIdx.x; e < m * h; e += kThreads) {
                const int r = e / h, i = e - r * h;
                const int pos = p.positions ? p.positions[n0 + r0 + r] : t0 + r0 + r;
                const int a = (int)(uint32_t)((turn[i] * (unsigned long long)(long long)pos) >> 32);
                float sn, cn;
                sincospif((float)a * 4.656612873077393e-10f, &sn, &cn);  // 2^-31: half turns
                if (p.inverse) sn = -sn;
                cs[r * (D / 2) + cs_at<D>(i)] = make_float2(cn * p.attn_scale, sn * p.attn_scale);
            }
            __syncthreads();
        }
        uint4* const mine = stage + (threadIdx.x >> 5) * kWarpUnits;  // this warp's units
        if constexpr (kL == kHalfAny) {
            __syncwarp();  // the previous batch has been read
#pragma unroll
            for (int i = 0; i < kBatch; ++i)
                mine[i * 32 + (threadIdx.x & 31)] = make_uint4(x[i].a[0], x[i].a[1], x[i].a[2], x[i].a[3]);
            __syncwarp();
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
            const int idx = base + i * kThreads;
            if (idx >= total) continue;
            int r, hd;
            place(idx, r, hd);
            const int u = idx & (U - 1);
            const long long row = n0 + r0 + r;
            __nv_bfloat16* dst;
            if (hd < p.hq) {
                dst = p.q_out + row * p.q_out_rs + hd * D;
            } else if (!kAppend) {
                dst = p.k_out + row * p.k_out_rs + (hd - p.hq) * D;
            } else {
                if (slot[r] < 0) continue;
                const int c = hd - p.hq;
                dst = c < p.hkv ? p.k_cache + ((size_t)slot[r] * p.hkv + c) * D
                                : p.v_cache + ((size_t)slot[r] * p.hkv + c - p.hkv) * D;
            }
            const uint16_t* head = nullptr;
            if constexpr (kL == kHalfAny)
                head = reinterpret_cast<const uint16_t*>(mine + i * 32 + ((threadIdx.x & 31) & ~(U - 1)));
            if (!kAppend || hd < p.hq + p.hkv) rotate_unit<D, kL>(x[i], cs + r * (D / 2), head, u, h);
            store_unit<kL>(x[i], dst, u, h);
        }
    }
}

template <int D, Layout kL>
static cudaError_t launch_d(const Args& a, cudaStream_t s) {
    const bool append = a.page_table != nullptr;
    const int heads = a.hq + (a.k ? a.hkv : 0) + (append ? a.hkv : 0);
    const long long longest = append ? a.max_new : a.rows;
    // Rows per block: one until every SM has several blocks, then up to eight.
    int tile = a.rows / (num_sms() * 8);
    tile = tile < 1 ? 1 : tile > kMaxRows ? kMaxRows : tile;
    const dim3 grid((unsigned)((longest + tile - 1) / tile), append ? a.batch : 1);
    const size_t smem = (size_t)tile * (D / 2) * sizeof(float2);
    const uint32_t mul = heads == 1 ? 0u : (uint32_t)(((1ull << 32) + heads - 1) / heads);
    if (append)
        rope_kernel<D, kL, true><<<grid, kThreads, smem, s>>>(a, tile, mul);
    else
        rope_kernel<D, kL, false><<<grid, kThreads, smem, s>>>(a, tile, mul);
    return cudaGetLastError();
}

cudaError_t launch(const Args& a, cudaStream_t s) {
    const Layout l = a.interleaved ? kInterleaved : a.rotary_dim % 16 == 0 ? kHalfVec : kHalfAny;
    if (a.head_dim == 64)
        return l == kInterleaved ? launch_d<64, kInterleaved>(a, s)
               : l == kHalfVec   ? launch_d<64, kHalfVec>(a, s)
                                 : launch_d<64, kHalfAny>(a, s);
    return l == kInterleaved ? launch_d<128, kInterleaved>(a, s)
           : l == kHalfVec   ? launch_d<128, kHalfVec>(a, s)
                             : launch_d<128, kHalfAny>(a, s);
}

ATTN_DEFINE_STATUS_ACCESSOR(status_word)

}  // namespace rope
}  // namespace attn
