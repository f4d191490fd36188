// Attention of a tree of drafted tokens over a paged cache (sm_103a).
//
// What it computes: request b has n drafted tokens (nodes), which are the last
// n of its L cached tokens; node i hangs on node parents[i] < i, or on the
// prefix (the first P = L - n tokens) when that is -1.  With depth 0 for nodes on
// the prefix and one more than the parent's otherwise, node i stands at position
// p_i = P + depth_i and sees the prefix tokens and its ancestors and itself, all by
// the first/last-window rule at their positions:
//     O_i = sum_j e^{s_ij - M} v_j / (e^{sink - M} + sum_j e^{s_ij - M}).
//
// One block per (node, KV head, request); one warp per query head of the group,
// 32 keys at a time with the running maximum and sum of the softmax.
#include "common.cuh"
#include "tree.h"

namespace attn {
namespace tree {

struct Params {
    const __nv_bfloat16* q;
    const __nv_bfloat16* k_cache;
    const __nv_bfloat16* v_cache;
    const int32_t* page_table;
    const int32_t* cu_q;
    const int32_t* seqlens_k;
    const int32_t* parents;
    const float* sink;
    __nv_bfloat16* out;
    float* lse;
    int max_pages, total_q, hq, hkv, page_size, num_pages, win_first, win_last;
    float scale_log2;
};

template <int D>
__global__ void __launch_bounds__(128) tree_simple_kernel(const Params p) {
    const int i = blockIdx.x, kvh = blockIdx.y, b = blockIdx.z;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    __shared__ int parent[kMaxNodes], depth[kMaxNodes];
    __shared__ uint32_t mask[kMaxNodes / 32];
    __shared__ float qs[4][D];
    const int q_start = p.cu_q[b];
    const int n = p.cu_q[b + 1] - q_start;
    if (i == 0 && kvh == 0 && threadIdx.x == 0 && (n > (int)gridDim.x || q_start + (long long)n > p.total_q))
        raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
    if (i >= n || q_start < 0 || q_start + i >= p.total_q) return;
    int L = p.seqlens_k[b];
    const long long cap = (long long)p.max_pages * p.page_size;
    if (L > cap || L < n) {
        if (threadIdx.x == 0) raise_status(ATTN_SINK_DEV_SEQLEN_OOB);
        L = L < n ? 0 : (int)cap;
    }
    const int P = max(0, L - n);
    for (int j = threadIdx.x; j <= i; j += 128) {
        int pr = p.parents[q_start + j];
        if (pr < -1 || pr >= j) {
            raise_status(ATTN_SINK_DEV_TREE);
            pr = -1;
        }
        parent[j] = pr;
    }
    if (threadIdx.x < kMaxNodes / 32) mask[threadIdx.x] = 0;
    __syncthreads();
    if (threadIdx.x == 0) {
        for (int j = 0; j <= i; ++j) depth[j] = parent[j] < 0 ? 0 : depth[parent[j]] + 1;
        for (int j = i; j >= 0; j = parent[j]) mask[j >> 5] |= 1u << (j & 31);
    }
    __syncthreads();
    const int pos = P + depth[i];
    const int group = p.hq / p.hkv;
    for (int g = warp; g < group; g += 4) {
        const int h = kvh * group + g;
        __syncwarp();
        for (int d = lane; d < D; d += 32)
            qs[warp][d] = __bfloat162float(p.q[((size_t)(q_start + i) * p.hq + h) * D + d]);
        __syncwarp();
        float m = p.sink ? p.sink[h] * ATTN_LOG2E : -INFINITY;
        float l = m == -INFINITY ? 0.f : 1.f;
        float o[D / 32] = {};
        for (int t0 = 0; t0 < L && m != INFINITY; t0 += 32) {  // an infinite sink takes all the mass
            const int t = t0 + lane;
            bool vis = t < L;
            long long slot = 0;
            if (vis) {
                const int j = t - P;
                const int kp = j < 0 ? t : j <= i ? P + depth[j] : pos;
                if (j >= 0) vis = j <= i && (mask[j >> 5] >> (j & 31) & 1);
                if (p.win_last > 0) vis = vis && (kp < p.win_first || kp > pos - p.win_last);
            }
            if (vis) {
                const int pg = p.page_table[(size_t)b * p.max_pages + t / p.page_size];
                if (pg < 0 || pg >= p.num_pages) {
                    raise_status(ATTN_SINK_DEV_PAGE_OOB);
                    vis = false;
                } else {
                    slot = (long long)pg * p.page_size + t % p.page_size;
                }
            }
            float x = -INFINITY;
            if (vis) {
                const uint4* k = reinterpret_cast<const uint4*>(p.k_cache + (slot * p.hkv + kvh) * D);
                float s = 0.f;
                for (int c = 0; c < D / 8; ++c) {
                    const uint4 w = k[c];
                    const float* q8 = &qs[warp][c * 8];
                    s += bf16_lo(w.x) * q8[0] + bf16_hi(w.x) * q8[1] + bf16_lo(w.y) * q8[2] + bf16_hi(w.y) * q8[3] +
                         bf16_lo(w.z) * q8[4] + bf16_hi(w.z) * q8[5] + bf16_lo(w.w) * q8[6] + bf16_hi(w.w) * q8[7];
                }
                x = s * p.scale_log2;
            }
            float mx = x;
#pragma unroll
            for (int s = 16; s; s >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, s));
            if (mx == -INFINITY) continue;
            const float mn = fmaxf(m, mx);
            const float al = fast_exp2(m - mn), e = fast_exp2(x - mn);
            float sum = e;
#pragma unroll
            for (int s = 16; s; s >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, s);
            l = l * al + sum;
            m = mn;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) o[c] *= al;
            for (int k = 0; k < 32; ++k) {
                const float w = __shfl_sync(0xffffffffu, e, k);
                const long long sl = __shfl_sync(0xffffffffu, slot, k);
                if (w == 0.f) continue;
                const __nv_bfloat16* v = p.v_cache + (sl * p.hkv + kvh) * D;
#pragma unroll
                for (int c = 0; c < D / 32; ++c) o[c] += w * __bfloat162float(v[c * 32 + lane]);
            }
        }
        const float inv = l > 0.f && m != INFINITY ? 1.f / l : 0.f;
        __nv_bfloat16* dst = p.out + ((size_t)(q_start + i) * p.hq + h) * D;
#pragma unroll
        for (int c = 0; c < D / 32; ++c) dst[c * 32 + lane] = __float2bfloat16_rn(o[c] * inv);
        if (p.lse && lane == 0)
            p.lse[(size_t)h * p.total_q + q_start + i] = l > 0.f ? (m + log2f(l)) * ATTN_LN2 : -INFINITY;
    }
}

cudaError_t launch(const Args& a, cudaStream_t s, std::string* what) {
    Params p;
    p.q = static_cast<const __nv_bfloat16*>(a.q);
    p.k_cache = static_cast<const __nv_bfloat16*>(a.k_cache);
    p.v_cache = static_cast<const __nv_bfloat16*>(a.v_cache);
    p.page_table = a.page_table;
    p.cu_q = a.cu_q;
    p.seqlens_k = a.seqlens_k;
    p.parents = a.parents;
    p.sink = a.sink;
    p.out = static_cast<__nv_bfloat16*>(a.out);
    p.lse = a.lse;
    p.max_pages = a.max_pages;
    p.total_q = a.total_q;
    p.hq = a.hq;
    p.hkv = a.hkv;
    p.page_size = a.page_size;
    p.num_pages = a.num_pages;
    p.win_first = a.win_first;
    p.win_last = a.win_last;
    p.scale_log2 = a.scale * ATTN_LOG2E;
    const dim3 grid(a.max_seqlen_q, a.hkv, a.batch);
    if (a.head_dim == 64)
        tree_simple_kernel<64><<<grid, 128, 0, s>>>(p);
    else
        tree_simple_kernel<128><<<grid, 128, 0, s>>>(p);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) *what = "launch";
    return e;
}

ATTN_DEFINE_STATUS_ACCESSOR(status_exchange)

}  // namespace tree
}  // namespace attn
