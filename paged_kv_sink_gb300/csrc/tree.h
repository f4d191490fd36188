// Host/device interface of the drafted-tree attention kernels (tree.cu).
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include <string>

namespace attn {
namespace tree {

constexpr int kMaxNodes = 256;  // drafted tokens of one request

struct Args {
    const void* q;
    const void* k_cache;
    const void* v_cache;
    const int32_t* page_table;
    const int32_t* cu_q;
    const int32_t* seqlens_k;
    const int32_t* parents;
    const float* sink;
    void* out;
    float* lse;
    int max_pages, batch, total_q, hq, hkv, head_dim, page_size, num_pages, max_seqlen_q;
    int win_first, win_last;
    float scale;
};

// Grid and scratch sizes.
struct Plan {
    int ctas;  // persistent CTAs, in gangs of hkv
    size_t part_o_bytes, part_ml_bytes, first_bytes;
};

Plan make_plan(const Args& a);
cudaError_t launch(const Args& a, const Plan& pl, void* scratch, cudaStream_t s, std::string* what);
int status_exchange(cudaStream_t s, int* host_bits);

}  // namespace tree
}  // namespace attn
