// Device helpers of the 8-bit cache's kernels.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"
#include "q8.h"

namespace attn {
namespace q8 {

// Four codes as two pairs of fp16, in order: both formats are exact in it.
template <int F>
__device__ __forceinline__ void quad_to_f16(uint32_t w, uint32_t& a, uint32_t& b) {
    if constexpr (F == kE4M3) {
        asm("{\n .reg .b16 lo, hi;\n mov.b32 {lo, hi}, %2;\n cvt.rn.f16x2.e4m3x2 %0, lo;\n cvt.rn.f16x2.e4m3x2 %1, hi;\n}"
            : "=r"(a), "=r"(b)
            : "r"(w));
    } else {
        const uint32_t x = w ^ 0x80808080u;  // bytes u = code + 128; 0x6400 + u is 1024 + u
        const uint32_t u = __byte_perm(x, 0x64646464u, 0x4140), v = __byte_perm(x, 0x64646464u, 0x4342);
        const __half2 c = __half2half2(__ushort_as_half(0x6480));
        const __half2 p = __hsub2(*reinterpret_cast<const __half2*>(&u), c);
        const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&v), c);
        a = *reinterpret_cast<const uint32_t*>(&p);
        b = *reinterpret_cast<const uint32_t*>(&q);
    }
}

__device__ __forceinline__ float2 f16_to_float2(uint32_t x) {
    return __half22float2(*reinterpret_cast<const __half2*>(&x));
}

// Page of token t and its place there.
struct Place {
    int page, in_page;
};

__device__ __forceinline__ Place place_of(int t, int page_size, int page_shift) {
    Place p;
    if (page_shift >= 0) {
        p.page = t >> page_shift;
        p.in_page = t & ((1 << page_shift) - 1);
    } else {
        p.page = t / page_size;
        p.in_page = t - p.page * page_size;
    }
    return p;
}

inline int shift_of(int n) {
    for (int s = 0; s < 31; ++s)
        if ((1 << s) == n) return s;
    return -1;
}

}  // namespace q8
}  // namespace attn
