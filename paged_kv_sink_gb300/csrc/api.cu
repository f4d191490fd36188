// C ABI of the attention-with-sink library: argument validation, scratch
// memory and kernel launches.  Every entry point is asynchronous on the
// caller's stream and returns an ATTN_SINK_* status.
#include <limits.h>
#include <math.h>
#include <stdarg.h>
#include <stdio.h>

#include <mutex>
#include <string>

#include "attn_sink.h"
#include "bwd.h"
#include "common.cuh"
#include "decode.h"
#include "evict.h"
#include "host_io.h"
#include "kv_append.h"
#include "selftest.h"
#include "prefill.h"
#include "rope.h"
#include "tree.h"

namespace {

thread_local std::string t_last_error;

int fail(int code, const char* fmt, ...) {
    char buf[512];
    va_list ap;
    va_start(ap, fmt);
    vsnprintf(buf, sizeof(buf), fmt, ap);
    va_end(ap);
    t_last_error = buf;
    return code;
}

int cuda_fail(cudaError_t e, const char* what) {
    return fail(ATTN_SINK_ERR_CUDA, "%s: %s (%s)", what, cudaGetErrorString(e), cudaGetErrorName(e));
}

// The forward, decode and append grids give the request index a grid dimension
// of at most 65535 blocks, and the forward its 128-row query tiles another.
constexpr int kMaxGridDim = 65535;

int check_grid(const char* who, int batch, int max_seqlen_q) {
    if (batch > kMaxGridDim)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: batch %d above %d requests per call", who, batch, kMaxGridDim);
    if (max_seqlen_q > 0 && (max_seqlen_q + 127) / 128 > kMaxGridDim)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: max_seqlen_q %d above %d query rows per request", who,
                    max_seqlen_q, kMaxGridDim * 128);
    return ATTN_SINK_OK;
}

// One library-owned stream-ordered memory pool per device.  Freed blocks are
// kept (release threshold = max) so that steady-state calls do not go back to
// the driver.
constexpr int kMaxDevices = 64;
std::mutex g_pool_mu;
cudaMemPool_t g_pools[kMaxDevices] = {};

cudaError_t device_pool(cudaMemPool_t* out) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lock(g_pool_mu);
    if (!g_pools[dev]) {
        cudaMemPoolProps props = {};
        props.allocType = cudaMemAllocationTypePinned;
        props.location.type = cudaMemLocationTypeDevice;
        props.location.id = dev;
        cudaMemPool_t pool;
        e = cudaMemPoolCreate(&pool, &props);
        if (e != cudaSuccess) return e;
        uint64_t thr = ~0ull;
        e = cudaMemPoolSetAttribute(pool, cudaMemPoolAttrReleaseThreshold, &thr);
        if (e != cudaSuccess) return e;
        g_pools[dev] = pool;
    }
    *out = g_pools[dev];
    return cudaSuccess;
}

// Stream-ordered scratch block, returned to the pool on the same stream.
struct Scratch {
    void* ptr = nullptr;
    cudaStream_t stream = nullptr;
    cudaError_t alloc(size_t bytes, cudaStream_t s) {
        stream = s;
        if (bytes == 0) return cudaSuccess;
        cudaMemPool_t pool;
        cudaError_t e = device_pool(&pool);
        if (e != cudaSuccess) return e;
        return cudaMallocFromPoolAsync(&ptr, bytes, pool, s);
    }
    ~Scratch() {
        if (ptr) cudaFreeAsync(ptr, stream);
    }
};

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace

namespace attn {
float resolve_scale(float scale, int head_dim) {
    return scale > 0.f ? scale : 1.0f / sqrtf((float)head_dim);
}

// Sets the calling thread's last-error text (used by entry points defined in
// other translation units).
void record_error(const char* msg) { t_last_error = msg; }
}  // namespace attn

extern "C" {

const char* attn_sink_last_error(void) { return t_last_error.c_str(); }

const char* attn_sink_version(void) { return "attn_sink_gb300 0.1 (sm_103a)"; }

}  // extern "C"

namespace attn {

int validate_decode(const char* who, const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                    const int32_t* page_table, int max_pages, const int32_t* seqlens, int batch, int hq,
                    int hkv, int head_dim, int page_size, int num_pages, int win_first, attn_bf16* out) {
    if (batch < 0 || hq <= 0 || hkv <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0)
        return fail(ATTN_SINK_ERR_INVALID, "%s: sizes must be positive (batch may be 0)", who);
    if (win_first < 0) return fail(ATTN_SINK_ERR_INVALID, "%s: win_first must be >= 0", who);
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: head_dim %d not supported (64, 128)", who, head_dim);
    if (hq % hkv) return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: hq %% hkv != 0", who);
    if (batch == 0) return ATTN_SINK_OK;
    if (!q || !k_cache || !v_cache || !page_table || !seqlens || !out)
        return fail(ATTN_SINK_ERR_INVALID, "%s: NULL tensor pointer", who);
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(q) || !aligned16(out))
        return fail(ATTN_SINK_ERR_INVALID, "%s: q, caches and out must be 16-byte aligned", who);
    if ((long long)num_pages * page_size >= (1LL << 31) || (long long)max_pages * page_size >= (1LL << 31))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: cache slots must fit in int32", who);
    return check_grid(who, batch, 0);
}

}  // namespace attn

namespace {

// Scores that a decode with accumulated weights keeps at a time (at least one request's):
// it takes batches that would need more in rounds of requests.  Rounds of long requests
// cost nothing (24 of 64k to 128k tokens, 64 heads: 1.04 ms in one round or four), but the
// lengths are not known here, and rounds of requests that are short for their table wait
// for one another: 256 of up to 2k tokens in a table of 128k take 0.23 ms at once
// (8.6 GB), 0.34 ms in rounds of 2 GiB, 0.72 ms in rounds of 512 MiB.
constexpr size_t kMaxScoreBytes = size_t(2) << 30;

int run_decode(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache, const int32_t* page_table,
               int max_pages, const int32_t* seqlens, int batch, int hq, int hkv, int head_dim, int page_size,
               int num_pages, const float* sink, int win_first, int win_last, float scale, attn_bf16* out,
               float* lse, cudaStream_t s, attn::decode::Weights* w = nullptr, int max_seqlen = -1) {
    if (batch == 0) return ATTN_SINK_OK;
    attn::decode::Args a;
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_table = page_table;
    a.seqlens = seqlens;
    a.sink = sink;
    a.out = out;
    a.lse = lse;
    a.max_pages = max_pages;
    a.batch = batch;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.win_first = win_first;
    a.win_last = win_last;
    a.group = hq / hkv;
    a.scale = attn::resolve_scale(scale, head_dim);
    a.max_seqlen = max_seqlen;
    const attn::decode::Plan pl = attn::decode::make_plan(a);
    // Partials, then (accumulated weights only) scores, of the requests of one round.
    size_t scores = 0;  // bytes, of a request
    int round = batch;
    if (w) {
        w->scores_cap = pl.nvis_max < w->cap ? pl.nvis_max : w->cap;
        scores = (size_t)hkv * pl.hblocks * w->scores_cap * attn::decode::score_heads(a) * sizeof(float);
        const size_t most = scores ? kMaxScoreBytes / scores : (size_t)batch;
        const int rounds = most >= (size_t)batch ? 1 : most ? (int)((batch + most - 1) / most) : batch;
        round = (batch + rounds - 1) / rounds;
    }
    const size_t part_o = pl.part_o_bytes / batch * round, part_ml = pl.part_ml_bytes / batch * round;
    const size_t scores_at = (part_o + part_ml + 255) & ~size_t(255);
    Scratch ws;
    cudaError_t e = ws.alloc(w ? scores_at + scores * round : part_o + part_ml, s);
    if (e != cudaSuccess) return cuda_fail(e, "decode: scratch allocation");
    char* const base = static_cast<char*>(ws.ptr);
    for (int b0 = 0; b0 < batch; b0 += round) {
        attn::decode::Args r = a;
        r.q = q + (size_t)b0 * hq * head_dim;
        r.page_table = page_table + (size_t)b0 * max_pages;
        r.seqlens = seqlens + b0;
        r.out = out + (size_t)b0 * hq * head_dim;
        r.lse = lse ? lse + (size_t)b0 * hq : nullptr;
        r.batch = batch - b0 < round ? batch - b0 : round;
        if (w) {
            w->scores = reinterpret_cast<float*>(base + scores_at);
            if (b0 > 0 && w->weights) w->weights += (size_t)round * w->heads * w->cap;
        }
        e = attn::decode::launch(r, pl, reinterpret_cast<float*>(base), reinterpret_cast<float2*>(base + part_o), s, w);
        if (e != cudaSuccess) return cuda_fail(e, "decode: launch");
    }
    return ATTN_SINK_OK;
}

int run_append(const attn_bf16* k_new, const attn_bf16* v_new, const int32_t* cu_new, const int32_t* seqlens,
               const int32_t* page_table, int max_pages, int batch, int hkv, int head_dim, int page_size,
               int num_pages, int max_new, attn_bf16* k_cache, attn_bf16* v_cache, cudaStream_t s) {
    attn::kvappend::Args a;
    a.k_new = k_new;
    a.v_new = v_new;
    a.cu_new = cu_new;
    a.seqlens = seqlens;
    a.page_table = page_table;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.max_pages = max_pages;
    a.batch = batch;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.max_new = max_new;
    cudaError_t e = attn::kvappend::launch(a, s);
    if (e != cudaSuccess) return cuda_fail(e, "kv_append: launch");
    return ATTN_SINK_OK;
}

}  // namespace

extern "C" {

int attn_sink_decode_paged(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                           const int32_t* page_table, int max_pages, const int32_t* seqlens,
                           int batch, int hq, int hkv, int head_dim, int page_size, int num_pages,
                           const float* sink, int win_first, int win_last, float scale,
                           attn_bf16* out, float* lse, void* stream) {
    t_last_error.clear();
    int rc = attn::validate_decode("decode", q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv, head_dim,
                             page_size, num_pages, win_first, out);
    if (rc != ATTN_SINK_OK || batch == 0) return rc;
    return run_decode(q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv, head_dim, page_size,
                      num_pages, sink, win_first, win_last, scale, out, lse, static_cast<cudaStream_t>(stream));
}

int attn_sink_kv_append(const attn_bf16* k_new, const attn_bf16* v_new, const int32_t* cu_new,
                        const int32_t* seqlens, const int32_t* page_table, int max_pages, int batch, int hkv,
                        int head_dim, int page_size, int num_pages, int max_new, attn_bf16* k_cache,
                        attn_bf16* v_cache, void* stream) {
    t_last_error.clear();
    if (batch < 0 || hkv <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 || max_new < 0)
        return fail(ATTN_SINK_ERR_INVALID, "kv_append: sizes must be positive (batch, max_new may be 0)");
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "kv_append: head_dim %d not supported (64, 128)", head_dim);
    if ((long long)num_pages * page_size >= (1LL << 31) || (long long)max_pages * page_size >= (1LL << 31))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "kv_append: cache slots must fit in int32");
    if (batch == 0 || max_new == 0) return ATTN_SINK_OK;
    if (!k_new || !v_new || !seqlens || !page_table || !k_cache || !v_cache)
        return fail(ATTN_SINK_ERR_INVALID, "kv_append: NULL tensor pointer");
    if (!aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) || !aligned16(v_cache))
        return fail(ATTN_SINK_ERR_INVALID, "kv_append: tensors must be 16-byte aligned");
    if (!cu_new && max_new != 1)
        return fail(ATTN_SINK_ERR_INVALID, "kv_append: without cu_new every request appends one row (max_new 1)");
    if (int rc = check_grid("kv_append", batch, 0)) return rc;
    return run_append(k_new, v_new, cu_new, seqlens, page_table, max_pages, batch, hkv, head_dim, page_size,
                      num_pages, max_new, k_cache, v_cache, static_cast<cudaStream_t>(stream));
}

int attn_sink_decode_paged_append(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new,
                                  attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table,
                                  int max_pages, const int32_t* seqlens, int batch, int hq, int hkv, int head_dim,
                                  int page_size, int num_pages, const float* sink, int win_first, int win_last,
                                  float scale, attn_bf16* out, float* lse, void* stream) {
    t_last_error.clear();
    int rc = attn::validate_decode("decode", q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv, head_dim,
                             page_size, num_pages, win_first, out);
    if (rc != ATTN_SINK_OK || batch == 0) return rc;
    if (!k_new || !v_new) return fail(ATTN_SINK_ERR_INVALID, "decode_append: NULL k_new / v_new");
    if (!aligned16(k_new) || !aligned16(v_new))
        return fail(ATTN_SINK_ERR_INVALID, "decode_append: k_new, v_new must be 16-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    rc = run_append(k_new, v_new, nullptr, seqlens, page_table, max_pages, batch, hkv, head_dim, page_size,
                    num_pages, 1, k_cache, v_cache, s);
    if (rc != ATTN_SINK_OK) return rc;
    return run_decode(q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv, head_dim, page_size,
                      num_pages, sink, win_first, win_last, scale, out, lse, s);
}

int attn_sink_visible_ranges(const int32_t* seqlens, int batch, int win_first, int win_last,
                             int32_t* ranges, void* stream) {
    t_last_error.clear();
    if (batch < 0 || win_first < 0) return fail(ATTN_SINK_ERR_INVALID, "visible_ranges: bad sizes");
    if (batch == 0) return ATTN_SINK_OK;
    if (!seqlens || !ranges) return fail(ATTN_SINK_ERR_INVALID, "visible_ranges: NULL pointer");
    cudaError_t e = attn::decode::launch_visible_ranges(seqlens, batch, win_first, win_last, ranges,
                                                        static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "visible_ranges: launch");
    return ATTN_SINK_OK;
}

int attn_sink_visible_slots(const int32_t* seqlens, const int32_t* page_table, int max_pages,
                            int batch, int page_size, int num_pages, int win_first, int win_last,
                            int32_t* slots, int max_visible, void* stream) {
    t_last_error.clear();
    if (batch < 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 || max_visible < 0 || win_first < 0)
        return fail(ATTN_SINK_ERR_INVALID, "visible_slots: bad sizes");
    if ((long long)num_pages * page_size >= (1LL << 31))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "visible_slots: cache slots must fit in int32");
    if (batch == 0 || max_visible == 0) return ATTN_SINK_OK;
    if (!seqlens || !page_table || !slots) return fail(ATTN_SINK_ERR_INVALID, "visible_slots: NULL pointer");
    cudaError_t e = attn::decode::launch_visible_slots(seqlens, page_table, max_pages, batch, page_size,
                                                       num_pages, win_first, win_last, slots, max_visible,
                                                       static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "visible_slots: launch");
    return ATTN_SINK_OK;
}

static int validate_varlen(const char* who, const void* q, const void* k, const void* v,
                           const int32_t* cu_q, const int32_t* cu_k, int batch, int total_q,
                           int total_k, int hq, int hkv,
                           int head_dim, int max_seqlen_q, int max_seqlen_k, int win_first,
                           int win_last, int causal, bool allow_d128) {
    if (batch < 0 || total_q < 0 || total_k < 0 || hq <= 0 || hkv <= 0 || max_seqlen_q < 0 ||
        max_seqlen_k < 0 || win_first < 0)
        return fail(ATTN_SINK_ERR_INVALID, "%s: sizes must be non-negative (heads positive)", who);
    if (win_last > 0 && !causal)
        return fail(ATTN_SINK_ERR_INVALID, "%s: first/last-window selection needs causal attention", who);
    if (head_dim != 64 && !(allow_d128 && head_dim == 128))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: head_dim %d not supported (%s)", who, head_dim,
                    allow_d128 ? "64, 128" : "64");
    if (hq % hkv) return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: hq %% hkv != 0", who);
    if (batch == 0) return ATTN_SINK_OK;
    if (!q || !k || !v || !cu_q || !cu_k) return fail(ATTN_SINK_ERR_INVALID, "%s: NULL tensor pointer", who);
    if (!aligned16(q) || !aligned16(k) || !aligned16(v))
        return fail(ATTN_SINK_ERR_INVALID, "%s: q, k, v must be 16-byte aligned", who);
    return ATTN_SINK_OK;
}

}  // extern "C"

namespace {

// A row stride (elements) is 0 (contiguous) or covers the row's heads and keeps
// every row 16-byte aligned.
int check_stride(const char* who, const char* name, long long rs, int heads, int head_dim) {
    if (rs == 0) return ATTN_SINK_OK;
    if (rs < (long long)heads * head_dim || rs % 8)
        return fail(ATTN_SINK_ERR_INVALID,
                    "%s: %s row stride %lld must be 0 or >= heads*head_dim and a multiple of 8", who, name, rs);
    return ATTN_SINK_OK;
}

int fwd_impl(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, long long q_rs, long long k_rs,
             long long v_rs, const float* sink, const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch,
             int total_q, int total_k, int hq, int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
             int win_first, int win_last, int causal, float scale, attn_bf16* out, float* lse, void* stream) {
    int rc = validate_varlen("fwd", q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, hq, hkv, head_dim,
                             max_seqlen_q, max_seqlen_k, win_first, win_last, causal, true);
    if (rc != ATTN_SINK_OK || batch == 0 || max_seqlen_q == 0 || total_q == 0) return rc;
    if ((rc = check_grid("fwd", batch, max_seqlen_q)) != ATTN_SINK_OK) return rc;
    if (!out) return fail(ATTN_SINK_ERR_INVALID, "fwd: NULL out");
    if (!aligned16(out)) return fail(ATTN_SINK_ERR_INVALID, "fwd: out must be 16-byte aligned");
    attn::prefill::FwdArgs a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.sink = sink;
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.out = out;
    a.lse = lse;
    a.batch = batch;
    a.total_q = total_q;
    a.total_k = total_k;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.win_first = win_first;
    a.win_last = win_last;
    a.causal = causal ? 1 : 0;
    a.scale = attn::resolve_scale(scale, head_dim);
    a.q_rs = q_rs;
    a.k_rs = k_rs;
    a.v_rs = v_rs;
    std::string err;
    cudaError_t e = attn::prefill::launch_fwd(a, static_cast<cudaStream_t>(stream), &err);
    if (e != cudaSuccess) return fail(ATTN_SINK_ERR_CUDA, "fwd: %s: %s", err.c_str(), cudaGetErrorString(e));
    return ATTN_SINK_OK;
}

}  // namespace

extern "C" {

int attn_sink_fwd(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, const float* sink,
                  const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch, int total_q,
                  int total_k, int hq, int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
                  int win_first, int win_last, int causal, float scale, attn_bf16* out, float* lse,
                  void* stream) {
    t_last_error.clear();
    return fwd_impl(q, k, v, 0, 0, 0, sink, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, hq, hkv, head_dim,
                    max_seqlen_q, max_seqlen_k, win_first, win_last, causal, scale, out, lse, stream);
}

int attn_sink_fwd_strided(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, long long q_row_stride,
                          long long k_row_stride, long long v_row_stride, const float* sink,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch, int total_q,
                          int total_k, int hq, int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
                          int win_first, int win_last, int causal, float scale, attn_bf16* out, float* lse,
                          void* stream) {
    t_last_error.clear();
    int rc;
    if ((rc = check_stride("fwd_strided", "q", q_row_stride, hq, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("fwd_strided", "k", k_row_stride, hkv, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("fwd_strided", "v", v_row_stride, hkv, head_dim)) != ATTN_SINK_OK)
        return rc;
    return fwd_impl(q, k, v, q_row_stride, k_row_stride, v_row_stride, sink, cu_seqlens_q, cu_seqlens_k, batch,
                    total_q, total_k, hq, hkv, head_dim, max_seqlen_q, max_seqlen_k, win_first, win_last, causal,
                    scale, out, lse, stream);
}

int attn_sink_fwd_host(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, const float* sink,
                       const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch, int hq, int hkv,
                       int head_dim, int win_first, int win_last, int causal, float scale, attn_bf16* out,
                       float* lse, void* stream) {
    t_last_error.clear();
    if (batch < 0 || hq <= 0 || hkv <= 0 || win_first < 0)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_host: sizes must be non-negative (heads positive)");
    if (win_last > 0 && !causal)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_host: first/last-window selection needs causal attention");
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_host: head_dim %d not supported (64, 128)", head_dim);
    if (hq % hkv) return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_host: hq %% hkv != 0");
    if (batch == 0) return ATTN_SINK_OK;
    if (!q || !k || !v || !cu_seqlens_q || !cu_seqlens_k || !out)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_host: NULL pointer");
    if (cu_seqlens_q[0] != 0 || cu_seqlens_k[0] != 0)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_host: cu_seqlens must start at 0");
    for (int b = 0; b < batch; ++b)
        if (cu_seqlens_q[b + 1] < cu_seqlens_q[b] || cu_seqlens_k[b + 1] < cu_seqlens_k[b])
            return fail(ATTN_SINK_ERR_INVALID, "fwd_host: cu_seqlens must be non-decreasing");
    attn::hostio::Args a;
    a.q = q;
    a.k = k;
    a.v = v;
    a.sink = sink;
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.out = out;
    a.lse = lse;
    a.batch = batch;
    a.total_q = cu_seqlens_q[batch];
    a.total_k = cu_seqlens_k[batch];
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.win_first = win_first;
    a.win_last = win_last;
    a.causal = causal ? 1 : 0;
    a.scale = attn::resolve_scale(scale, head_dim);
    if (a.total_q == 0) return ATTN_SINK_OK;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch ws;
    cudaError_t e = ws.alloc(attn::hostio::scratch_bytes(a), s);
    if (e != cudaSuccess) return cuda_fail(e, "fwd_host: scratch allocation");
    std::string err;
    e = attn::hostio::run(a, ws.ptr, s, &err);
    if (e != cudaSuccess) return fail(ATTN_SINK_ERR_CUDA, "fwd_host: %s: %s", err.c_str(), cudaGetErrorString(e));
    return ATTN_SINK_OK;
}

int attn_sink_fwd_paged(const attn_bf16* q, const attn_bf16* k_new, const attn_bf16* v_new, attn_bf16* k_cache,
                        attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                        const int32_t* cu_seqlens_q, const int32_t* seqlens_k, int batch, int total_q, int hq,
                        int hkv, int head_dim, int page_size, int num_pages, int max_seqlen_q, int max_seqlen_k,
                        const float* sink, int win_first, int win_last, int causal, float scale,
                        attn_bf16* out, float* lse, void* stream) {
    t_last_error.clear();
    if (batch < 0 || total_q < 0 || hq <= 0 || hkv <= 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0 ||
        max_seqlen_q < 0 || max_seqlen_k < 0 || win_first < 0)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_paged: sizes must be non-negative (heads, pages positive)");
    if (win_last > 0 && !causal)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_paged: first/last-window selection needs causal attention");
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_paged: head_dim %d not supported (64, 128)", head_dim);
    if (hq % hkv) return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_paged: hq %% hkv != 0");
    if (page_size < 8 || (page_size & (page_size - 1)))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_paged: page_size %d not supported (a power of two >= 8)",
                    page_size);
    if ((long long)num_pages * page_size >= (1LL << 31) || (long long)max_pages * page_size >= (1LL << 31))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "fwd_paged: cache slots must fit in int32");
    if ((k_new == nullptr) != (v_new == nullptr))
        return fail(ATTN_SINK_ERR_INVALID, "fwd_paged: k_new and v_new are given together or not at all");
    if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return ATTN_SINK_OK;
    if (!q || !k_cache || !v_cache || !page_table || !cu_seqlens_q || !seqlens_k || !out)
        return fail(ATTN_SINK_ERR_INVALID, "fwd_paged: NULL tensor pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (k_new && (!aligned16(k_new) || !aligned16(v_new))))
        return fail(ATTN_SINK_ERR_INVALID, "fwd_paged: tensors must be 16-byte aligned");
    if (int rc = check_grid("fwd_paged", batch, max_seqlen_q)) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (k_new) {
        int rc = run_append(k_new, v_new, cu_seqlens_q, seqlens_k, page_table, max_pages, batch, hkv, head_dim,
                            page_size, num_pages, max_seqlen_q, k_cache, v_cache, s);
        if (rc != ATTN_SINK_OK) return rc;
    }
    attn::prefill::FwdArgs a = {};
    a.q = q;
    a.k = k_cache;
    a.v = v_cache;
    a.sink = sink;
    a.cu_q = cu_seqlens_q;
    a.cu_k = nullptr;
    a.out = out;
    a.lse = lse;
    a.batch = batch;
    a.total_q = total_q;
    a.total_k = 0;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.win_first = win_first;
    a.win_last = win_last;
    a.causal = causal ? 1 : 0;
    a.scale = attn::resolve_scale(scale, head_dim);
    a.page_table = page_table;
    a.seqlens_k = seqlens_k;
    a.max_pages = max_pages;
    a.page_size = page_size;
    a.num_pages = num_pages;
    std::string err;
    cudaError_t e = attn::prefill::launch_fwd(a, s, &err);
    if (e != cudaSuccess) return fail(ATTN_SINK_ERR_CUDA, "fwd_paged: %s: %s", err.c_str(), cudaGetErrorString(e));
    return ATTN_SINK_OK;
}

}  // extern "C"

namespace {

int bwd_impl(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, const long long* rs, const float* sink,
             const attn_bf16* out, const float* lse, const attn_bf16* dout, const int32_t* cu_seqlens_q,
             const int32_t* cu_seqlens_k, int batch, int total_q, int total_k, int hq, int hkv, int head_dim,
             int max_seqlen_q, int max_seqlen_k, int win_first, int win_last, int causal, float scale,
             attn_bf16* dq, attn_bf16* dk, attn_bf16* dv, float* dsink, void* stream) {
    int rc = validate_varlen("bwd", q, k, v, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, hq, hkv, head_dim,
                             max_seqlen_q, max_seqlen_k, win_first, win_last, causal, true);
    if (rc != ATTN_SINK_OK) return rc;
    if ((sink == nullptr) != (dsink == nullptr))
        return fail(ATTN_SINK_ERR_INVALID, "bwd: dsink must be given exactly when sink is");
    if (batch == 0) return ATTN_SINK_OK;
    if (!out || !lse || !dout || !dq || !dk || !dv)
        return fail(ATTN_SINK_ERR_INVALID, "bwd: NULL tensor pointer");
    if (!aligned16(out) || !aligned16(dout) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
        return fail(ATTN_SINK_ERR_INVALID, "bwd: tensors must be 16-byte aligned");
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    attn::bwd::Args a = {};
    a.q = q;
    a.k = k;
    a.v = v;
    a.sink = sink;
    a.out = out;
    a.lse = lse;
    a.dout = dout;
    a.cu_q = cu_seqlens_q;
    a.cu_k = cu_seqlens_k;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.dsink = dsink;
    a.batch = batch;
    a.total_q = total_q;
    a.total_k = total_k;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.max_seqlen_q = max_seqlen_q;
    a.max_seqlen_k = max_seqlen_k;
    a.win_first = win_first;
    a.win_last = win_last;
    a.causal = causal ? 1 : 0;
    a.scale = attn::resolve_scale(scale, head_dim);
    a.q_rs = rs[0];
    a.k_rs = rs[1];
    a.v_rs = rs[2];
    a.dq_rs = rs[3];
    a.dk_rs = rs[4];
    a.dv_rs = rs[5];
    size_t ws_bytes = attn::bwd::workspace_bytes(a);
    Scratch ws;
    cudaError_t e = ws.alloc(ws_bytes, s);
    if (e != cudaSuccess) return cuda_fail(e, "bwd: scratch allocation");
    std::string err;
    e = attn::bwd::launch(a, ws.ptr, ws_bytes, s, &err);
    if (e != cudaSuccess) return fail(ATTN_SINK_ERR_CUDA, "bwd: %s: %s", err.c_str(), cudaGetErrorString(e));
    return ATTN_SINK_OK;
}

// Checks shared by the rotary entry points.
int check_rope(const char* who, int rows, int hq, int hkv, int min_hkv, long long heads, int head_dim, int rotary_dim,
               float attn_scale) {
    if (rows < 0 || hq <= 0 || hkv < min_hkv)
        return fail(ATTN_SINK_ERR_INVALID, "%s: sizes must be non-negative (heads positive)", who);
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: head_dim %d not supported (64, 128)", who, head_dim);
    if (rotary_dim < 2 || rotary_dim > head_dim || rotary_dim % 2)
        return fail(ATTN_SINK_ERR_INVALID, "%s: rotary_dim %d must be even, from 2 to head_dim", who, rotary_dim);
    if (heads > 16384) return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: %lld heads above 16384", who, heads);
    if (!isfinite(attn_scale)) return fail(ATTN_SINK_ERR_INVALID, "%s: attn_scale must be finite", who);
    return ATTN_SINK_OK;
}

// Sizes of a paged cache.
int check_cache(const char* who, int batch, int max_pages, int page_size, int num_pages) {
    if (batch < 0 || max_pages <= 0 || page_size <= 0 || num_pages <= 0)
        return fail(ATTN_SINK_ERR_INVALID, "%s: sizes must be positive (batch may be 0)", who);
    // A request's tokens stay so far below 2^31 that the end of a tile or batch of them does not wrap.
    if ((long long)num_pages * page_size >= (1LL << 31) || (long long)max_pages * page_size > (1LL << 31) - 65536)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: cache slots must fit in int32, a request's stay 65536 below", who);
    return ATTN_SINK_OK;
}

// Query heads (of every KV head rounded up to 8, or to 16 above 8) whose statistics a
// block of the weights' accumulation keeps in 48 KB of shared memory.
constexpr int kMaxWeightHeads = 6144;

// Heads of the entry points that move cache rows.
int check_moves(const char* who, const char* name, int heads, int hkv, int head_dim) {
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: head_dim %d not supported (64, 128)", who, head_dim);
    if (heads != 1 && heads != hkv) return fail(ATTN_SINK_ERR_INVALID, "%s: %s %d must be 1 or hkv", who, name, heads);
    if (heads > kMaxGridDim / 3)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: %s %d above %d", who, name, heads, kMaxGridDim / 3);
    if ((long long)hkv * head_dim * 2 >= (1LL << 31))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "%s: a token's row must be below 2 GiB", who);
    return ATTN_SINK_OK;
}

const __nv_bfloat16* as_bf16(const attn_bf16* p) { return reinterpret_cast<const __nv_bfloat16*>(p); }
__nv_bfloat16* as_bf16(attn_bf16* p) { return reinterpret_cast<__nv_bfloat16*>(p); }
long long row_stride(long long rs, int heads, int head_dim) { return rs ? rs : (long long)heads * head_dim; }

}  // namespace

extern "C" {

int attn_sink_bwd(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, const float* sink,
                  const attn_bf16* out, const float* lse, const attn_bf16* dout,
                  const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch, int total_q,
                  int total_k, int hq, int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
                  int win_first, int win_last, int causal, float scale, attn_bf16* dq, attn_bf16* dk,
                  attn_bf16* dv, float* dsink, void* stream) {
    t_last_error.clear();
    const long long rs[6] = {0, 0, 0, 0, 0, 0};
    return bwd_impl(q, k, v, rs, sink, out, lse, dout, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, hq,
                    hkv, head_dim, max_seqlen_q, max_seqlen_k, win_first, win_last, causal, scale, dq, dk, dv,
                    dsink, stream);
}

int attn_sink_bwd_strided(const attn_bf16* q, const attn_bf16* k, const attn_bf16* v, long long q_row_stride,
                          long long k_row_stride, long long v_row_stride, const float* sink,
                          const attn_bf16* out, const float* lse, const attn_bf16* dout,
                          const int32_t* cu_seqlens_q, const int32_t* cu_seqlens_k, int batch, int total_q,
                          int total_k, int hq, int hkv, int head_dim, int max_seqlen_q, int max_seqlen_k,
                          int win_first, int win_last, int causal, float scale, attn_bf16* dq, attn_bf16* dk,
                          attn_bf16* dv, long long dq_row_stride, long long dk_row_stride,
                          long long dv_row_stride, float* dsink, void* stream) {
    t_last_error.clear();
    int rc;
    const long long rs[6] = {q_row_stride, k_row_stride, v_row_stride, dq_row_stride, dk_row_stride,
                             dv_row_stride};
    const char* names[6] = {"q", "k", "v", "dq", "dk", "dv"};
    for (int i = 0; i < 6; ++i)
        if ((rc = check_stride("bwd_strided", names[i], rs[i], (i % 3) == 0 ? hq : hkv, head_dim)) != ATTN_SINK_OK) return rc;
    return bwd_impl(q, k, v, rs, sink, out, lse, dout, cu_seqlens_q, cu_seqlens_k, batch, total_q, total_k, hq,
                    hkv, head_dim, max_seqlen_q, max_seqlen_k, win_first, win_last, causal, scale, dq, dk, dv,
                    dsink, stream);
}

int attn_sink_rope(const attn_bf16* q, attn_bf16* q_out, const attn_bf16* k, attn_bf16* k_out,
                   long long q_row_stride, long long q_out_row_stride, long long k_row_stride,
                   long long k_out_row_stride, const int32_t* positions, const double* inv_freq, int rows, int hq,
                   int hkv, int head_dim, int rotary_dim, int interleaved, int inverse, float attn_scale,
                   void* stream) {
    t_last_error.clear();
    if ((k == nullptr) != (k_out == nullptr))
        return fail(ATTN_SINK_ERR_INVALID, "rope: k and k_out are given together or not at all");
    if (!k) hkv = 0;
    int rc = check_rope("rope", rows, hq, hkv, k ? 1 : 0, hq + (long long)hkv, head_dim, rotary_dim, attn_scale);
    if (rc != ATTN_SINK_OK) return rc;
    if ((rc = check_stride("rope", "q", q_row_stride, hq, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope", "q_out", q_out_row_stride, hq, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope", "k", k_row_stride, hkv, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope", "k_out", k_out_row_stride, hkv, head_dim)) != ATTN_SINK_OK)
        return rc;
    if (rows == 0) return ATTN_SINK_OK;
    if (!q || !q_out || !positions || !inv_freq) return fail(ATTN_SINK_ERR_INVALID, "rope: NULL tensor pointer");
    if (!aligned16(q) || !aligned16(q_out) || (k && (!aligned16(k) || !aligned16(k_out))))
        return fail(ATTN_SINK_ERR_INVALID, "rope: q, k and the outputs must be 16-byte aligned");
    attn::rope::Args a = {};
    a.q = as_bf16(q);
    a.q_out = as_bf16(q_out);
    a.k = as_bf16(k);
    a.k_out = as_bf16(k_out);
    a.q_rs = row_stride(q_row_stride, hq, head_dim);
    a.q_out_rs = row_stride(q_out_row_stride, hq, head_dim);
    a.k_rs = row_stride(k_row_stride, hkv, head_dim);
    a.k_out_rs = row_stride(k_out_row_stride, hkv, head_dim);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rows = rows;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.inverse = inverse ? 1 : 0;
    a.attn_scale = attn_scale;
    cudaError_t e = attn::rope::launch(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "rope: launch");
    return ATTN_SINK_OK;
}

int attn_sink_rope_kv_append(const attn_bf16* q, attn_bf16* q_out, const attn_bf16* k_new, const attn_bf16* v_new,
                             long long q_row_stride, long long q_out_row_stride, long long k_row_stride,
                             long long v_row_stride, const int32_t* cu_new, const int32_t* positions,
                             const double* inv_freq, const int32_t* seqlens, const int32_t* page_table,
                             int max_pages, int batch, int total_new, int hq, int hkv, int head_dim, int rotary_dim,
                             int page_size, int num_pages, int max_new, int interleaved, float attn_scale,
                             attn_bf16* k_cache, attn_bf16* v_cache, void* stream) {
    t_last_error.clear();
    int rc = check_rope("rope_kv_append", total_new, hq, hkv, 1, hq + 2LL * hkv, head_dim, rotary_dim, attn_scale);
    if (rc != ATTN_SINK_OK) return rc;
    if ((rc = check_cache("rope_kv_append", batch, max_pages, page_size, num_pages)) != ATTN_SINK_OK) return rc;
    if (max_new < 0) return fail(ATTN_SINK_ERR_INVALID, "rope_kv_append: max_new must be >= 0");
    if ((rc = check_stride("rope_kv_append", "q", q_row_stride, hq, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope_kv_append", "q_out", q_out_row_stride, hq, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope_kv_append", "k_new", k_row_stride, hkv, head_dim)) != ATTN_SINK_OK ||
        (rc = check_stride("rope_kv_append", "v_new", v_row_stride, hkv, head_dim)) != ATTN_SINK_OK)
        return rc;
    if (batch == 0 || max_new == 0 || total_new == 0) return ATTN_SINK_OK;
    if (!q || !q_out || !k_new || !v_new || !inv_freq || !seqlens || !page_table || !k_cache || !v_cache)
        return fail(ATTN_SINK_ERR_INVALID, "rope_kv_append: NULL tensor pointer");
    if (!aligned16(q) || !aligned16(q_out) || !aligned16(k_new) || !aligned16(v_new) || !aligned16(k_cache) ||
        !aligned16(v_cache))
        return fail(ATTN_SINK_ERR_INVALID, "rope_kv_append: tensors must be 16-byte aligned");
    if (!cu_new && (max_new != 1 || total_new < batch))
        return fail(ATTN_SINK_ERR_INVALID,
                    "rope_kv_append: without cu_new every request appends one row (max_new 1, total_new = batch)");
    if ((rc = check_grid("rope_kv_append", batch, 0)) != ATTN_SINK_OK) return rc;
    attn::rope::Args a = {};
    a.q = as_bf16(q);
    a.q_out = as_bf16(q_out);
    a.k = as_bf16(k_new);
    a.v = as_bf16(v_new);
    a.q_rs = row_stride(q_row_stride, hq, head_dim);
    a.q_out_rs = row_stride(q_out_row_stride, hq, head_dim);
    a.k_rs = row_stride(k_row_stride, hkv, head_dim);
    a.v_rs = row_stride(v_row_stride, hkv, head_dim);
    a.positions = positions;
    a.inv_freq = inv_freq;
    a.rows = total_new;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.attn_scale = attn_scale;
    a.cu_new = cu_new;
    a.seqlens = seqlens;
    a.page_table = page_table;
    a.k_cache = as_bf16(k_cache);
    a.v_cache = as_bf16(v_cache);
    a.max_pages = max_pages;
    a.batch = batch;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.max_new = max_new;
    cudaError_t e = attn::rope::launch(a, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "rope_kv_append: launch");
    return ATTN_SINK_OK;
}

int attn_sink_tree_paged(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                         const int32_t* page_table, int max_pages, const int32_t* cu_seqlens_q,
                         const int32_t* seqlens_k, const int32_t* parents, int batch, int total_q, int hq, int hkv,
                         int head_dim, int page_size, int num_pages, int max_seqlen_q, int max_seqlen_k,
                         const float* sink, int win_first, int win_last, float scale, attn_bf16* out, float* lse,
                         void* stream) {
    t_last_error.clear();
    if (total_q < 0 || hq <= 0 || hkv <= 0 || max_seqlen_q < 0 || max_seqlen_k < 0 || win_first < 0)
        return fail(ATTN_SINK_ERR_INVALID, "tree_paged: sizes must be non-negative (heads positive)");
    int rc = check_cache("tree_paged", batch, max_pages, page_size, num_pages);
    if (rc != ATTN_SINK_OK) return rc;
    if (head_dim != 64 && head_dim != 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "tree_paged: head_dim %d not supported (64, 128)", head_dim);
    if (hq % hkv || hq / hkv > 128)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "tree_paged: hq must be a multiple of hkv, at most 128 times it");
    if (page_size < 8 || (page_size & (page_size - 1)))
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "tree_paged: page_size %d not supported (a power of two >= 8)",
                    page_size);
    if (max_seqlen_q > attn::tree::kMaxNodes)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "tree_paged: max_seqlen_q %d above %d nodes per request", max_seqlen_q,
                    attn::tree::kMaxNodes);
    if (batch == 0 || total_q == 0 || max_seqlen_q == 0) return ATTN_SINK_OK;
    if (!q || !k_cache || !v_cache || !page_table || !cu_seqlens_q || !seqlens_k || !parents || !out)
        return fail(ATTN_SINK_ERR_INVALID, "tree_paged: NULL tensor pointer");
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out))
        return fail(ATTN_SINK_ERR_INVALID, "tree_paged: tensors must be 16-byte aligned");
    if ((rc = check_grid("tree_paged", batch, 0)) != ATTN_SINK_OK) return rc;
    attn::tree::Args a = {};
    a.q = q;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.page_table = page_table;
    a.cu_q = cu_seqlens_q;
    a.seqlens_k = seqlens_k;
    a.parents = parents;
    a.sink = sink;
    a.out = out;
    a.lse = lse;
    a.max_pages = max_pages;
    a.batch = batch;
    a.total_q = total_q;
    a.hq = hq;
    a.hkv = hkv;
    a.head_dim = head_dim;
    a.page_size = page_size;
    a.num_pages = num_pages;
    a.max_seqlen_q = max_seqlen_q;
    a.win_first = win_first;
    a.win_last = win_last;
    a.scale = attn::resolve_scale(scale, head_dim);
    const attn::tree::Plan pl = attn::tree::make_plan(a);
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch ws;
    cudaError_t e = ws.alloc(pl.part_o_bytes + pl.part_ml_bytes + pl.first_bytes, s);
    if (e != cudaSuccess) return cuda_fail(e, "tree_paged: scratch allocation");
    std::string err;
    e = attn::tree::launch(a, pl, ws.ptr, s, &err);
    if (e != cudaSuccess)
        return fail(ATTN_SINK_ERR_CUDA, "tree_paged: %s: %s", err.c_str(), cudaGetErrorString(e));
    return ATTN_SINK_OK;
}

int attn_sink_kv_compact(attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                         const int32_t* src, const int32_t* counts, const int32_t* base, int batch, int src_heads,
                         int max_rows, int hkv, int head_dim, int page_size, int num_pages, void* stream) {
    t_last_error.clear();
    if (hkv <= 0 || max_rows < 0)
        return fail(ATTN_SINK_ERR_INVALID, "kv_compact: sizes must be non-negative (heads positive)");
    int rc = check_cache("kv_compact", batch, max_pages, page_size, num_pages);
    if (rc != ATTN_SINK_OK) return rc;
    if ((rc = check_moves("kv_compact", "src_heads", src_heads, hkv, head_dim)) != ATTN_SINK_OK) return rc;
    if (batch == 0 || max_rows == 0) return ATTN_SINK_OK;
    if (!k_cache || !v_cache || !page_table || !src || !counts)
        return fail(ATTN_SINK_ERR_INVALID, "kv_compact: NULL tensor pointer");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(ATTN_SINK_ERR_INVALID, "kv_compact: caches must be 16-byte aligned");
    if (k_cache == v_cache) return fail(ATTN_SINK_ERR_INVALID, "kv_compact: k_cache and v_cache must differ");
    if ((rc = check_grid("kv_compact", batch, 0)) != ATTN_SINK_OK) return rc;
    attn::evict::MoveArgs m = {};
    m.k_cache = as_bf16(k_cache);
    m.v_cache = as_bf16(v_cache);
    m.page_table = page_table;
    m.src = src;
    m.counts = counts;
    m.base = base;
    m.max_pages = max_pages;
    m.batch = batch;
    m.heads = src_heads;
    m.hkv = hkv;
    m.head_dim = head_dim;
    m.page_size = page_size;
    m.num_pages = num_pages;
    m.max_rows = max_rows;
    cudaError_t e = attn::evict::launch_move(m, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "kv_compact: launch");
    return ATTN_SINK_OK;
}

int attn_sink_decode_paged_weights(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                                   const int32_t* page_table, int max_pages, const int32_t* seqlens, int batch,
                                   int hq, int hkv, int head_dim, int page_size, int num_pages, const float* sink,
                                   int win_first, int win_last, float scale, float* weights, int weight_heads,
                                   int weight_cap, attn_bf16* out, float* lse, void* stream) {
    return attn_sink_decode_paged_weights_bounded(q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv,
                                                  head_dim, page_size, num_pages, INT_MAX, sink, win_first, win_last,
                                                  scale, weights, weight_heads, weight_cap, out, lse, stream);
}

int attn_sink_decode_paged_weights_bounded(const attn_bf16* q, const attn_bf16* k_cache, const attn_bf16* v_cache,
                                           const int32_t* page_table, int max_pages, const int32_t* seqlens,
                                           int batch, int hq, int hkv, int head_dim, int page_size, int num_pages,
                                           int max_seqlen, const float* sink, int win_first, int win_last,
                                           float scale, float* weights, int weight_heads, int weight_cap,
                                           attn_bf16* out, float* lse, void* stream) {
    t_last_error.clear();
    int rc = attn::validate_decode("decode_weights", q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq,
                                   hkv, head_dim, page_size, num_pages, win_first, out);
    if (rc != ATTN_SINK_OK) return rc;
    if ((rc = check_cache("decode_weights", batch, max_pages, page_size, num_pages)) != ATTN_SINK_OK) return rc;
    if (weight_heads != 1 && weight_heads != hkv)
        return fail(ATTN_SINK_ERR_INVALID, "decode_weights: weight_heads %d must be 1 or hkv", weight_heads);
    if (weight_cap < 0) return fail(ATTN_SINK_ERR_INVALID, "decode_weights: weight_cap must be >= 0");
    if (max_seqlen < 0) return fail(ATTN_SINK_ERR_INVALID, "decode_weights: max_seqlen must be >= 0");
    if (hq > 4096) return fail(ATTN_SINK_ERR_UNSUPPORTED, "decode_weights: hq %d above 4096", hq);
    const int group = hq / hkv, padded = group <= 8 ? 8 : (group + 15) / 16 * 16;
    if ((long long)(hkv / weight_heads) * padded > kMaxWeightHeads)
        return fail(ATTN_SINK_ERR_UNSUPPORTED, "decode_weights: weight_heads 1 sums at most %d padded query heads",
                    kMaxWeightHeads);
    if (batch == 0) return ATTN_SINK_OK;
    if (!weights && weight_cap > 0) return fail(ATTN_SINK_ERR_INVALID, "decode_weights: NULL weights");
    attn::decode::Weights w = {};
    w.weights = weights;
    w.heads = weight_heads;
    w.cap = weight_cap;
    return run_decode(q, k_cache, v_cache, page_table, max_pages, seqlens, batch, hq, hkv, head_dim, page_size,
                      num_pages, sink, win_first, win_last, scale, out, lse, static_cast<cudaStream_t>(stream), &w,
                      max_seqlen);
}

int attn_sink_evict_paged(attn_bf16* k_cache, attn_bf16* v_cache, const int32_t* page_table, int max_pages,
                          const int32_t* seqlens, const float* weights, int batch, int weight_heads, int weight_cap,
                          int hkv, int head_dim, int page_size, int num_pages, int budget, int keep_first,
                          int keep_last, float* weights_out, int32_t* kept, int32_t* new_seqlens, void* stream) {
    t_last_error.clear();
    if (hkv <= 0 || weight_cap <= 0) return fail(ATTN_SINK_ERR_INVALID, "evict_paged: sizes must be positive");
    int rc = check_cache("evict_paged", batch, max_pages, page_size, num_pages);
    if (rc != ATTN_SINK_OK) return rc;
    if ((rc = check_moves("evict_paged", "weight_heads", weight_heads, hkv, head_dim)) != ATTN_SINK_OK) return rc;
    if (budget < 1 || keep_first < 0 || keep_last < 0 || (long long)keep_first + keep_last > budget)
        return fail(ATTN_SINK_ERR_INVALID,
                    "evict_paged: budget must be positive and hold keep_first + keep_last (both >= 0)");
    if (batch == 0) return ATTN_SINK_OK;
    if (!k_cache || !v_cache || !page_table || !seqlens || !weights || !weights_out || !kept || !new_seqlens)
        return fail(ATTN_SINK_ERR_INVALID, "evict_paged: NULL tensor pointer");
    if (!aligned16(k_cache) || !aligned16(v_cache))
        return fail(ATTN_SINK_ERR_INVALID, "evict_paged: caches must be 16-byte aligned");
    if (k_cache == v_cache) return fail(ATTN_SINK_ERR_INVALID, "evict_paged: k_cache and v_cache must differ");
    if (new_seqlens == seqlens)
        return fail(ATTN_SINK_ERR_INVALID, "evict_paged: new_seqlens must not be seqlens (every head reads it)");
    if ((rc = check_grid("evict_paged", batch, 0)) != ATTN_SINK_OK) return rc;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    Scratch ws;
    cudaError_t e = ws.alloc((size_t)batch * weight_heads * sizeof(int32_t), s);
    if (e != cudaSuccess) return cuda_fail(e, "evict_paged: scratch allocation");
    attn::evict::SelectArgs a = {};
    a.weights = weights;
    a.seqlens = seqlens;
    a.new_seqlens = new_seqlens;
    a.kept = kept;
    a.first_moved = static_cast<int32_t*>(ws.ptr);
    a.batch = batch;
    a.heads = weight_heads;
    a.cap = weight_cap;
    a.budget = budget;
    a.keep_first = keep_first;
    a.keep_last = keep_last;
    a.token_cap = (long long)max_pages * page_size;
    if ((e = attn::evict::launch_select(a, s)) != cudaSuccess) return cuda_fail(e, "evict_paged: select launch");
    attn::evict::MoveArgs m = {};
    m.k_cache = as_bf16(k_cache);
    m.v_cache = as_bf16(v_cache);
    m.page_table = page_table;
    m.src = kept;
    m.counts = new_seqlens;
    m.first_moved = a.first_moved;
    m.max_pages = max_pages;
    m.batch = batch;
    m.heads = weight_heads;
    m.hkv = hkv;
    m.head_dim = head_dim;
    m.page_size = page_size;
    m.num_pages = num_pages;
    m.max_rows = budget;
    m.weights = weights;
    m.weights_out = weights_out;
    m.cap = weight_cap;
    if ((e = attn::evict::launch_move(m, s)) != cudaSuccess) return cuda_fail(e, "evict_paged: move launch");
    return ATTN_SINK_OK;
}

int attn_sink_device_status(void* stream) {
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    int bits = 0;
    int e = attn::decode::status_exchange(s, &bits);
    if (!e) e = attn::prefill::status_exchange(s, &bits);
    if (!e) e = attn::bwd::status_exchange(s, &bits);
    if (!e) e = attn::kvappend::status_exchange(s, &bits);
    if (!e) e = attn::rope::status_exchange(s, &bits);
    if (!e) e = attn::tree::status_exchange(s, &bits);
    if (!e) e = attn::evict::status_exchange(s, &bits);
    if (!e) e = attn::selftest::status_exchange(s, &bits);
    if (e) return cuda_fail(static_cast<cudaError_t>(e), "device_status");
    return bits;
}

int attn_sink_selftest_wait(int complete, void* stream) {
    t_last_error.clear();
    cudaError_t e = attn::selftest::launch_wait(complete, static_cast<cudaStream_t>(stream));
    if (e != cudaSuccess) return cuda_fail(e, "selftest_wait: launch");
    return ATTN_SINK_OK;
}

}  // extern "C"
