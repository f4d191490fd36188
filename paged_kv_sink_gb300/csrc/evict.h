// Host/device interface of cache eviction and compaction (evict.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {
namespace evict {

// Selection of the tokens that stay: (request, weight head) pairs.
struct SelectArgs {
    const float* weights;  // (batch, heads, cap)
    const int32_t* seqlens;
    int32_t* new_seqlens;  // (batch,)
    int32_t* kept;         // (batch, heads, budget)
    int32_t* first_moved;  // (batch, heads) scratch: the first kept index that is not its own rank
    int batch, heads, cap, budget, keep_first, keep_last;
    long long token_cap;   // tokens that the page table holds
};

// Moves of cache rows inside a request: token src[j] becomes token base + j.
struct MoveArgs {
    __nv_bfloat16* k_cache;
    __nv_bfloat16* v_cache;
    const int32_t* page_table;
    const int32_t* src;          // (batch, heads, max_rows)
    const int32_t* counts;       // (batch,) rows to move, at most max_rows
    const int32_t* base;         // (batch,), or NULL: 0
    const int32_t* first_moved;  // (batch, heads), or NULL: 0
    int max_pages, batch, heads, hkv, head_dim, page_size, num_pages, max_rows;
    // Eviction only: the weights follow the rows, (batch, heads, cap).
    const float* weights;
    float* weights_out;
    int cap;
};

cudaError_t launch_select(const SelectArgs& a, cudaStream_t s);
cudaError_t launch_move(const MoveArgs& a, cudaStream_t s);
int status_exchange(cudaStream_t s, int* host_bits);

}  // namespace evict
}  // namespace attn
