// Host/device interface of the 8-bit paged cache (q8_append.cu, q8_attend.cu).
//
// Layout: codes (num_pages, page_size, hkv, d), e4m3 or int8; scales
// (num_pages, page_size / block, hkv) fp32, one for `block` tokens of a KV head.
// A code c of a block stands for c * scale.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace attn {
namespace q8 {

enum { kE4M3 = 0, kInt8 = 1 };

// Smallest exponent of a scale that the append writes: blocks below qmax * 2^-64 lose
// digits to it.
constexpr int kMinExp = -64;

struct Cache {
    uint8_t* k;
    uint8_t* v;
    float* k_scale;
    float* v_scale;
    const int32_t* page_table;
    int max_pages, hkv, head_dim, page_size, num_pages, block, format;
};

struct AppendArgs {
    Cache c;
    const __nv_bfloat16* k_new;  // (total_new, hkv, d)
    const __nv_bfloat16* v_new;
    long long k_rs, v_rs;        // row strides, elements
    const int32_t* cu_new;       // (batch+1), or NULL: one row per request
    const int32_t* seqlens;
    int batch, total_new, max_new;
    int page_shift, block_shift, blocks;  // (set by the launch) log2 or -1; blocks of a page
};

// The visible tokens of every request as bf16 pages of a cache of their own, of
// kExpandPage tokens (a key tile of the forward): request b's token t at page
// b * pages + t / kExpandPage.
constexpr int kExpandPage = 128;
struct ExpandArgs {
    Cache c;
    const int32_t* cu_q;
    const int32_t* seqlens;
    int batch, pages, max_q, win_first, win_last;  // max_q: rows of a request at most, else reported
    __nv_bfloat16* k_out;
    __nv_bfloat16* v_out;
    int32_t* table_out;  // (batch, pages)
    int32_t* lens_out;   // (batch,): the lengths, cut at what the table and `pages` hold
    int32_t* parents;    // (total_q,), or NULL: each row's predecessor in its request
    int total_q;
};

struct AttendArgs {
    Cache c;
    const __nv_bfloat16* q;  // (total_q, hq, d)
    const int32_t* cu_q;     // (batch+1), or NULL: row b is request b's
    const int32_t* seqlens;
    const float* sink;
    __nv_bfloat16* out;
    float* lse;              // (total_q, hq), or (hq, total_q) when lse_by_head; may be NULL
    int batch, total_q, hq, max_q, max_seqlen, win_first, win_last, causal, lse_by_head;
    float scale;
};

struct AttendPlan {
    int nt;            // 8-row columns of a CTA's tile
    int tiles;         // row tiles of a KV head
    int split_tokens;  // visible tokens per split
    int max_splits;
    bool gather;       // a row's splits are one cluster, which merges them
    size_t part_o_bytes, part_ml_bytes;  // of all rows
};

cudaError_t launch_append(const AppendArgs& a, cudaStream_t s);
cudaError_t launch_expand(const ExpandArgs& a, cudaStream_t s);
AttendPlan make_plan(const AttendArgs& a);
cudaError_t launch_attend(const AttendArgs& a, const AttendPlan& pl, float* part_o, float2* part_ml, cudaStream_t s);
cudaError_t append_status_word(int** word);
cudaError_t attend_status_word(int** word);

}  // namespace q8
}  // namespace attn
