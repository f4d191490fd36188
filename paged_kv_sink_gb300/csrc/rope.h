// Host/device interface of the rotary-position kernel (rope.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {
namespace rope {

// One launch rotates the query heads and the key heads of every row; with
// caches it also writes the rotated keys and the values into their pages.
// Strides are in elements between consecutive rows.
struct Args {
    const __nv_bfloat16* q;
    __nv_bfloat16* q_out;
    const __nv_bfloat16* k;      // NULL: queries only
    __nv_bfloat16* k_out;        // NULL with caches
    const __nv_bfloat16* v;      // with caches only
    long long q_rs, q_out_rs, k_rs, k_out_rs, v_rs;
    const int32_t* positions;    // (rows,), or NULL with caches: the row's logical token
    const double* inv_freq;      // (rotary_dim / 2,) radians per position
    int rows, hq, hkv, head_dim, rotary_dim, interleaved, inverse;
    float attn_scale;
    // Paged append (page_table != NULL): request b's new rows are
    // [cu_new[b], cu_new[b+1]), or row b alone when cu_new is NULL.
    const int32_t* cu_new;
    const int32_t* seqlens;
    const int32_t* page_table;
    __nv_bfloat16* k_cache;
    __nv_bfloat16* v_cache;
    int max_pages, batch, page_size, num_pages, max_new;
};

cudaError_t launch(const Args& a, cudaStream_t s);
cudaError_t status_word(int** word);

}  // namespace rope
}  // namespace attn
