// The extern "C" entry points declared in include/pkv.h: argument
// validation, the optional checked mode, and dispatch to the kernels.
//
// Validation order follows the pages' rule for a rejected input: everything
// that can be checked on the host is checked before any work is enqueued, and
// in checked mode the device-resident indices are verified (and the call
// waits for the verdict) before any output byte is written.
#include <math.h>
#include <mutex>

#include "pkv.h"
#include "pkv_internal.h"

// Sticky device status ([0], PKV_DEVERR_* bits) and the verdict word of the
// current checked call ([1]). One copy per device.
static __device__ unsigned int g_pkv_status[2];

namespace pkv {

namespace {

constexpr int kMaxDevices = 64;

struct DeviceInfo {
    unsigned int* status = nullptr;
    int sm_count = 0;
};

DeviceInfo& device_info() {
    static std::mutex mu;
    static DeviceInfo info[kMaxDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    if (dev < 0 || dev >= kMaxDevices) dev = 0;
    std::lock_guard<std::mutex> lock(mu);
    DeviceInfo& d = info[dev];
    if (d.status == nullptr) {
        void* p = nullptr;
        if (cudaGetSymbolAddress(&p, g_pkv_status) == cudaSuccess) d.status = static_cast<unsigned int*>(p);
        int n = 0;
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess) d.sm_count = n;
    }
    return d;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Query heads of an attention call: a positive multiple of the KV heads, at
// most PKV_MAX_Q_HEADS (query-row counts per (sequence, KV head) stay 32-bit).
bool q_heads_ok(int32_t num_q_heads, const pkv_cache_desc* d) {
    return num_q_heads >= 1 && num_q_heads <= PKV_MAX_Q_HEADS && num_q_heads % d->num_kv_heads == 0;
}

// Block-table width of an attention call: the tokens of one sequence
// (max_blocks * 16) and the blocks of one launch's sequences (at most
// kMaxBatchPerLaunch of them, prefix-summed on the device) are 32-bit counts.
bool table_width_ok(int32_t batch, int32_t max_blocks) {
    const int64_t per_launch = batch < kMaxBatchPerLaunch ? batch : kMaxBatchPerLaunch;
    return max_blocks >= 1 && static_cast<int64_t>(max_blocks) * 16 < (int64_t(1) << 31) &&
           per_launch * max_blocks < (int64_t(1) << 31);
}

pkv_status check_desc(const pkv_cache_desc* d) {
    if (d == nullptr) return PKV_ERR_NULL;
    if (d->block_size != 16 || d->num_blocks < 1 || d->num_kv_heads < 1) return PKV_ERR_SHAPE;
    if (d->head_dim != 64 && d->head_dim != 128) return PKV_ERR_SHAPE;
    if (d->dtype != PKV_F32 && d->dtype != PKV_BF16) return PKV_ERR_DTYPE;
    // Rows of one pool (block, head, slot) are addressed with 32-bit coordinates.
    if (d->num_blocks * d->num_kv_heads * 16 >= (int64_t(1) << 31)) return PKV_ERR_SHAPE;
    return PKV_OK;
}

// Runs one validation launch in checked mode and waits for its verdict. The
// verdict word is one per device, so checked calls from different host
// threads take turns (each waits for its verdict before releasing it).
template <typename F>
pkv_status run_checked(F launch, cudaStream_t s) {
    static std::mutex verdict_mu;
    std::lock_guard<std::mutex> lock(verdict_mu);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    unsigned int* verdict = status + 1;
    if (cudaMemsetAsync(verdict, 0, sizeof(unsigned int), s) != cudaSuccess) return PKV_ERR_CUDA;
    if (launch(verdict) != cudaSuccess) return PKV_ERR_CUDA;
    unsigned int host = 0;
    if (cudaMemcpyAsync(&host, verdict, sizeof(unsigned int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return PKV_ERR_CUDA;
    if (host & kVerdictRange) return PKV_ERR_RANGE;
    if (host & kVerdictOverlap) return PKV_ERR_OVERLAP;
    if (host & kVerdictBlocks) return PKV_ERR_OUT_OF_BLOCKS;
    return PKV_OK;
}

pkv_status check_desc_q4(const pkv_cache_desc* d) {
    if (d == nullptr) return PKV_ERR_NULL;
    if (d->block_size != 16 || d->num_blocks < 1 || d->num_kv_heads < 1) return PKV_ERR_SHAPE;
    if (d->head_dim != 64 && d->head_dim != 128) return PKV_ERR_SHAPE;
    if (d->dtype != PKV_INT4) return PKV_ERR_DTYPE;
    // block ids are 32-bit; records are addressed in 64 bits
    if (d->num_blocks >= (int64_t(1) << 31) || d->num_blocks * d->num_kv_heads >= (int64_t(1) << 31)) return PKV_ERR_SHAPE;
    return PKV_OK;
}

// Whether n bytes at p and m bytes at q share one.
bool overlap(const void* p, size_t n, const void* q, size_t m) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    return n > 0 && m > 0 && a < b + m && b < a + n;
}

// The same of `count` rows of n bytes at p, `ps` bytes apart, and of m bytes at q, `qs` apart. (Rows
// of other strides that lie between one another count as sharing.)
bool overlap_rows(int64_t count, const void* p, size_t n, size_t ps, const void* q, size_t m, size_t qs) {
    const size_t all = static_cast<size_t>(count) - 1;
    if (n == 0 || m == 0 || !overlap(p, all * ps + n, q, all * qs + m)) return false;
    if (all == 0 || ps != qs) return true;
    // one stride: where the spans meet, rows share bytes unless those of one begin behind the other's
    const uintptr_t a = reinterpret_cast<uintptr_t>(p), b = reinterpret_cast<uintptr_t>(q);
    const size_t from = b >= a ? (b - a) % ps : (ps - (a - b) % ps) % ps;  // q's first byte in p's rows
    return from < n || ps - from < m;
}

pkv_status check_desc_q8(const pkv_cache_desc* d, bool attention) {
    if (d == nullptr) return PKV_ERR_NULL;
    if (d->block_size != 16 || d->num_blocks < 1 || d->num_kv_heads < 1) return PKV_ERR_SHAPE;
    if (d->head_dim != 128 && (attention || d->head_dim != 64)) return PKV_ERR_SHAPE;
    if (d->dtype != PKV_INT8) return PKV_ERR_DTYPE;
    if (d->num_blocks * d->num_kv_heads * d->head_dim >= (int64_t(1) << 31)) return PKV_ERR_SHAPE;
    return PKV_OK;
}

bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Int8 multi-query calls: which of the two kernels. The one that splits the cache
// (pkv_multiquery.cu) holds 32 rows per (sequence, KV head) of 128; beside the tile
// kernel, which turns the codes into f16 once for all rows, it is ahead where rows are
// few and the caches long. 32 query heads on 8, split : tile in us,
//     sequences x tokens   4 or 8 rows   16 rows      32 rows
//     1 x 1024              36 : 18       46 : 18      60 : 19
//     1 x 4096              37 : 24       49 : 25      56 : 25
//     1 x 32768             44 : 45       63 : 46      80 : 46
//     8 x 4096              33 : 42       48 : 42      64 : 42
//     32 x 4096             58 : 119      95 : 120    159 : 120
//     8 x 32768            102 : 197     170 : 197    304 : 196
//     64 x 8192            178 : 398     308 : 402    582 : 397
// Lengths are the device's: what the tables could hold stands in for them, in (token,
// KV head) pairs.
bool split_kernel_takes(const pkv_cache_desc* d, int32_t batch, int32_t max_blocks, int32_t max_query_len, int G) {
    const int64_t rows = static_cast<int64_t>(max_query_len) * G;
    const int64_t most = rows <= 8 ? 65536 : 524288;  // pairs that tiles take in less time
    return d->head_dim == 128 && rows <= 16 && static_cast<int64_t>(max_blocks) * 16 * d->num_kv_heads > most / batch;
}
static_assert(16 <= kMqMaxRows, "rows of the split kernel");

// Both reading-back calls, after the checks of their descriptors.
pkv_status run_gather(const void* k, const void* v, const float* scales, const int32_t* tables, int32_t max_blocks,
                      const int32_t* lens, const int32_t* token_start, const int32_t* row_start, int32_t batch,
                      int64_t num_rows, void* k_out, void* v_out, int32_t out_dtype, const pkv_cache_desc* desc,
                      uint32_t flags, cudaStream_t s) {
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;
    if (batch < 0 || num_rows < 0 || num_rows >= (int64_t(1) << 31)) return PKV_ERR_SHAPE;
    if (batch == 0 || num_rows == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks)) return PKV_ERR_SHAPE;
    if (!k || !v || !tables || !lens || !row_start || !k_out || !v_out) return PKV_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || !aligned16(k_out) || !aligned16(v_out) || !aligned4(tables) ||
        !aligned4(lens) || !aligned4(token_start) || !aligned4(row_start))
        return PKV_ERR_ALIGN;
    GatherArgs a{};
    a.k = k;
    a.v = v;
    a.scales = scales;
    a.tables = tables;
    a.lens = lens;
    a.token_start = token_start;
    a.row_start = row_start;
    a.k_out = k_out;
    a.v_out = v_out;
    a.status = device_info().status;
    a.num_blocks = desc->num_blocks;
    a.num_rows = num_rows;
    a.max_blocks = max_blocks;
    a.batch = batch;
    a.kv_heads = desc->num_kv_heads;
    if (a.status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        const pkv_status st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(tables, max_blocks, lens, batch, desc->num_blocks, 0, verdict, s);
            return e != cudaSuccess ? e : launch_check_gather(a, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        a.tables = tables + static_cast<int64_t>(b0) * max_blocks;
        a.lens = lens + b0;
        a.token_start = token_start == nullptr ? nullptr : token_start + b0;
        a.row_start = row_start + b0;
        a.batch = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        if (launch_gather(a, *desc, out_dtype, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

}  // namespace

int device_sm_count() {
    const int n = device_info().sm_count;
    return n > 0 ? n : 1;
}

}  // namespace pkv

using namespace pkv;

extern "C" {

const char* pkv_status_string(pkv_status s) {
    switch (s) {
        case PKV_OK: return "PKV_OK";
        case PKV_ERR_NULL: return "PKV_ERR_NULL";
        case PKV_ERR_SHAPE: return "PKV_ERR_SHAPE";
        case PKV_ERR_DTYPE: return "PKV_ERR_DTYPE";
        case PKV_ERR_ALIGN: return "PKV_ERR_ALIGN";
        case PKV_ERR_RANGE: return "PKV_ERR_RANGE";
        case PKV_ERR_OVERLAP: return "PKV_ERR_OVERLAP";
        case PKV_ERR_WORKSPACE: return "PKV_ERR_WORKSPACE";
        case PKV_ERR_TIMEOUT: return "PKV_ERR_TIMEOUT";
        case PKV_ERR_CUDA: return "PKV_ERR_CUDA";
        case PKV_ERR_UNSUPPORTED: return "PKV_ERR_UNSUPPORTED";
        case PKV_ERR_OUT_OF_BLOCKS: return "PKV_ERR_OUT_OF_BLOCKS";
        case PKV_ERR_UNKNOWN_SEQUENCE: return "PKV_ERR_UNKNOWN_SEQUENCE";
        case PKV_ERR_EXISTS: return "PKV_ERR_EXISTS";
        case PKV_ERR_INVARIANT: return "PKV_ERR_INVARIANT";
    }
    return "PKV_ERR_UNKNOWN";
}

int32_t pkv_version(void) { return 100; }

pkv_status pkv_append(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens, void* k_cache,
                      void* v_cache, const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_append");
    pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_SHAPE;
    if (k_cache == nullptr || v_cache == nullptr) return PKV_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    if (num_tokens == 0) return PKV_OK;
    if (k == nullptr || v == nullptr || slot_mapping == nullptr) return PKV_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u)) return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        if (num_tokens > 16384) return PKV_ERR_UNSUPPORTED;
        const int64_t num_slots = desc->num_blocks * 16;
        st = run_checked([&](unsigned int* verdict) { return launch_check_slots(slot_mapping, num_tokens, num_slots, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_append(k, v, slot_mapping, num_tokens, k_cache, v_cache, *desc, status, s) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks(const int64_t* pairs, int64_t num_pairs, void* k_cache, void* v_cache,
                           const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_copy_blocks");
    pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_SHAPE;
    if (k_cache == nullptr || v_cache == nullptr) return PKV_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache)) return PKV_ERR_ALIGN;
    if (num_pairs == 0) return PKV_OK;
    if (pairs == nullptr) return PKV_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pairs) & 7u) return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        if (num_pairs > 16384) return PKV_ERR_UNSUPPORTED;
        st = run_checked([&](unsigned int* verdict) { return launch_check_pairs(pairs, num_pairs, desc->num_blocks, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_copy_blocks(pairs, num_pairs, k_cache, v_cache, *desc, status, s) == cudaSuccess ? PKV_OK
                                                                                                   : PKV_ERR_CUDA;
}

size_t pkv_decode_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                 const pkv_cache_desc* desc, const pkv_decode_opts* opts) {
    if (check_desc(desc) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc))
        return 0;
    DecodePlan plan;
    if (decode_plan(*desc, batch, num_q_heads, max_blocks_per_seq, opts, &plan) != PKV_OK) return 0;
    return decode_workspace_layout(batch, desc->num_kv_heads, plan.num_ctas, num_q_heads / desc->num_kv_heads,
                                   desc->head_dim)
        .total;
}

pkv_status pkv_decode_attention(const void* q, const void* k_cache, const void* v_cache, const int32_t* block_tables,
                                int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
                                int32_t num_q_heads, float scale, void* out, void* workspace,
                                size_t workspace_bytes, const pkv_cache_desc* desc, uint32_t flags,
                                const pkv_decode_opts* opts, void* stream) {
    NvtxRange nvtx_range("pkv_decode_attention");
    pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    if (!isfinite(scale)) return PKV_ERR_SHAPE;
    if (opts != nullptr && opts->num_ctas < 0) return PKV_ERR_SHAPE;
    if ((flags & PKV_FLAG_TEST_STALL) && !(opts != nullptr && opts->kernel == 2)) return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace) return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    DecodePlan plan;
    const int rc = decode_plan(*desc, batch, num_q_heads, max_blocks_per_seq, opts, &plan);
    if (rc != PKV_OK) return static_cast<pkv_status>(rc);
    const int G = num_q_heads / desc->num_kv_heads;
    const WorkspaceLayout wl = decode_workspace_layout(batch, desc->num_kv_heads, plan.num_ctas, G, desc->head_dim);
    if (workspace_bytes < wl.total) return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) {
            return launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch, desc->num_blocks,
                                       1, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    const int elem = desc->dtype == PKV_BF16 ? 2 : 4;
    const int64_t row = static_cast<int64_t>(num_q_heads) * desc->head_dim * elem;
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        const int32_t nb = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        DecodeArgs a{};
        a.q = static_cast<const char*>(q) + b0 * row;
        a.k_cache = k_cache;
        a.v_cache = v_cache;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.out = static_cast<char*>(out) + b0 * row;
        a.partials = reinterpret_cast<float*>(static_cast<char*>(workspace) + wl.partials_offset);
        a.counters = reinterpret_cast<int*>(static_cast<char*>(workspace) + wl.counters_offset);
        a.trace = wl.trace_offset ? static_cast<char*>(workspace) + wl.trace_offset : nullptr;
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = nb;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.dtype = desc->dtype;
        a.num_ctas = plan.num_ctas;
        a.test_stall = (flags & PKV_FLAG_TEST_STALL) ? 1 : 0;
        a.scale = scale;
        if (launch_decode(a, plan, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

size_t pkv_decode_prefixed_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                          int32_t num_groups, int32_t max_group_blocks, const pkv_cache_desc* desc,
                                          const pkv_decode_opts* opts) {
    if (check_desc(desc) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc)) return 0;
    if (num_groups < 0 || num_groups > kMaxBatchPerLaunch || max_group_blocks < 0) return 0;
    DecodePlan plan;
    if (decode_plan(*desc, batch, num_q_heads, max_blocks_per_seq, opts, &plan, true) != PKV_OK) return 0;
    const int G = num_q_heads / desc->num_kv_heads;
    const size_t base = decode_workspace_layout(batch, desc->num_kv_heads, plan.num_ctas, G, desc->head_dim).total;
    if (plan.kernel != 2 || num_groups == 0) return base;
    return prefix_plan(batch, num_groups, num_q_heads, desc->num_kv_heads, desc->head_dim, max_group_blocks, base,
                       opts ? opts->prefix_kernel : 0)
        .total;
}

pkv_status pkv_decode_attention_prefixed(const void* q, const void* k_cache, const void* v_cache,
                                         const int32_t* block_tables, int32_t max_blocks_per_seq,
                                         const int32_t* context_lens, int32_t batch, int32_t num_q_heads,
                                         float scale, const int32_t* prefix_group, const int32_t* group_blocks,
                                         int32_t num_groups, int32_t max_group_blocks, void* out, void* workspace,
                                         size_t workspace_bytes, const pkv_cache_desc* desc, uint32_t flags,
                                         const pkv_decode_opts* opts, void* stream) {
    NvtxRange nvtx_range("pkv_decode_attention_prefixed");
    pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    if (num_groups < 0 || max_group_blocks < 0 || max_group_blocks > max_blocks_per_seq) return PKV_ERR_SHAPE;
    if (num_groups > kMaxBatchPerLaunch) return PKV_ERR_UNSUPPORTED;
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;
    if (num_groups > 0 && batch > 0) {
        if (prefix_group == nullptr || group_blocks == nullptr) return PKV_ERR_NULL;
        if ((reinterpret_cast<uintptr_t>(prefix_group) & 3u) || (reinterpret_cast<uintptr_t>(group_blocks) & 3u))
            return PKV_ERR_ALIGN;
    }
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    DecodePlan plan;
    int rc = decode_plan(*desc, batch, num_q_heads, max_blocks_per_seq, opts, &plan, true);
    if (rc != PKV_OK) return static_cast<pkv_status>(rc);
    // Without groups, or where only the CUDA-core kernel applies, the groups
    // are only a hint: the plain call computes the same result.
    if (num_groups == 0 || plan.kernel != 2 || batch == 0) {
        if (num_groups > 0 && batch > 0 && (flags & PKV_FLAG_CHECKED)) {
            cudaStream_t s = static_cast<cudaStream_t>(stream);
            if (max_blocks_per_seq < 1) return PKV_ERR_SHAPE;
            st = run_checked([&](unsigned int* verdict) {
                return launch_check_groups(block_tables, max_blocks_per_seq, context_lens, prefix_group,
                                           group_blocks, num_groups, max_group_blocks, batch, verdict, s);
            }, s);
            if (st != PKV_OK) return st;
        }
        return pkv_decode_attention(q, k_cache, v_cache, block_tables, max_blocks_per_seq, context_lens, batch,
                                    num_q_heads, scale, out, workspace, workspace_bytes, desc, flags, opts, stream);
    }
    if (!isfinite(scale)) return PKV_ERR_SHAPE;
    if (opts != nullptr && opts->num_ctas < 0) return PKV_ERR_SHAPE;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !out || !workspace) return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    const int G = num_q_heads / desc->num_kv_heads;
    const WorkspaceLayout wl = decode_workspace_layout(batch, desc->num_kv_heads, plan.num_ctas, G, desc->head_dim);
    if (opts != nullptr && (opts->prefix_kernel < 0 || opts->prefix_kernel > 2)) return PKV_ERR_UNSUPPORTED;
    const PrefixPlan pp = prefix_plan(batch, num_groups, num_q_heads, desc->num_kv_heads, desc->head_dim,
                                      max_group_blocks, wl.total, opts ? opts->prefix_kernel : 0);
    if (workspace_bytes < pp.total) return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch,
                                                desc->num_blocks, 1, verdict, s);
            if (e != cudaSuccess) return e;
            return launch_check_groups(block_tables, max_blocks_per_seq, context_lens, prefix_group, group_blocks,
                                       num_groups, max_group_blocks, batch, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    char* ws = static_cast<char*>(workspace);
    const int64_t row = static_cast<int64_t>(num_q_heads) * desc->head_dim * 2;
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        const int32_t nb = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        DecodeArgs a{};
        a.q = static_cast<const char*>(q) + b0 * row;
        a.k_cache = k_cache;
        a.v_cache = v_cache;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.out = static_cast<char*>(out) + b0 * row;
        a.partials = reinterpret_cast<float*>(ws + wl.partials_offset);
        a.counters = reinterpret_cast<int*>(ws + wl.counters_offset);
        a.trace = wl.trace_offset ? ws + wl.trace_offset : nullptr;
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = nb;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.dtype = desc->dtype;
        a.num_ctas = plan.num_ctas;
        a.test_stall = 0;
        a.scale = scale;
        a.prefix_group = prefix_group + b0;
        a.group_blocks = group_blocks;
        a.num_groups = num_groups;
        a.max_group_blocks = max_group_blocks;
        a.fold_o = reinterpret_cast<float*>(ws + pp.fold_o_offset);
        a.fold_lse = reinterpret_cast<float*>(ws + pp.fold_lse_offset);
        if (launch_decode(a, plan, s) != cudaSuccess) return PKV_ERR_CUDA;
        PrefixArgs pa{};
        pa.q = a.q;
        pa.k_cache = k_cache;
        pa.v_cache = v_cache;
        pa.tables = a.tables;
        pa.lens = a.lens;
        pa.prefix_group = a.prefix_group;
        pa.group_blocks = group_blocks;
        pa.fold_o = a.fold_o;
        pa.fold_lse = a.fold_lse;
        pa.out = a.out;
        pa.partials = reinterpret_cast<float*>(ws + pp.partials_offset);
        pa.counters = reinterpret_cast<int*>(ws + pp.counters_offset);
        pa.trace = pp.trace_offset ? ws + pp.trace_offset : nullptr;
        pa.status = status;
        pa.num_blocks = desc->num_blocks;
        pa.max_blocks = max_blocks_per_seq;
        pa.batch = nb;
        pa.num_groups = num_groups;
        pa.max_group_blocks = max_group_blocks;
        pa.q_heads = num_q_heads;
        pa.kv_heads = desc->num_kv_heads;
        pa.head_dim = desc->head_dim;
        pa.group = G;
        pa.tiles = pp.tiles;
        pa.chunks = pp.chunks;
        pa.chunk_blocks = pp.chunk_blocks;
        pa.scale = scale;
        if (launch_prefix(pa, pp.kernel, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

size_t pkv_multiquery_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                     int32_t max_query_len, const pkv_cache_desc* desc,
                                     const pkv_decode_opts* opts) {
    (void)max_blocks_per_seq;
    if (check_desc(desc) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc)) return 0;
    const int G = num_q_heads / desc->num_kv_heads;
    if (desc->dtype != PKV_BF16 || max_query_len < 1 || max_query_len > kMaxQueryLen) return 0;
    if (max_query_len * G > kMqMaxRows) return 256;  // tensor-core prefill path: combines on chip
    size_t co = 0, po = 0;
    return mq_workspace_bytes(batch, desc->num_kv_heads, desc->head_dim, mq_num_ctas(desc->head_dim, batch, opts),
                              &co, &po);
}

pkv_status pkv_multiquery_attention(const void* q, const void* k_cache, const void* v_cache,
                                    const int32_t* block_tables, int32_t max_blocks_per_seq,
                                    const int32_t* context_lens, const int32_t* query_start, int32_t batch,
                                    int32_t num_q_heads, int32_t max_query_len, float scale, void* out,
                                    void* workspace, size_t workspace_bytes, const pkv_cache_desc* desc,
                                    uint32_t flags, const pkv_decode_opts* opts, void* stream) {
    NvtxRange nvtx_range("pkv_multiquery_attention");
    pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    if (!isfinite(scale) || max_query_len < 1) return PKV_ERR_SHAPE;
    if (opts != nullptr && opts->num_ctas < 0) return PKV_ERR_SHAPE;
    const int G = num_q_heads / desc->num_kv_heads;
    if (desc->dtype != PKV_BF16) return PKV_ERR_DTYPE;
    if (max_query_len > kMaxQueryLen) return PKV_ERR_UNSUPPORTED;
    const bool prefill = max_query_len * G > kMqMaxRows;  // many query rows: the tcgen05 kernel
    if (prefill && (flags & PKV_FLAG_TEST_STALL)) return PKV_ERR_UNSUPPORTED;  // the hook is the split kernel's
    if (batch == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !k_cache || !v_cache || !block_tables || !context_lens || !query_start || !out || !workspace)
        return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(out) ||
        (reinterpret_cast<uintptr_t>(block_tables) & 3u) || (reinterpret_cast<uintptr_t>(context_lens) & 3u) ||
        (reinterpret_cast<uintptr_t>(query_start) & 3u) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    const int num_ctas = prefill ? 0 : mq_num_ctas(desc->head_dim, batch, opts);
    size_t co = 0, po = 0;
    const size_t need =
        prefill ? 256 : mq_workspace_bytes(batch, desc->num_kv_heads, desc->head_dim, num_ctas, &co, &po);
    if (workspace_bytes < need) return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch,
                                                desc->num_blocks, 0, verdict, s);
            if (e != cudaSuccess) return e;
            return launch_check_queries(context_lens, query_start, batch, max_query_len, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    if (prefill) {
        for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
            PrefixArgs pa{};
            pa.q = q;
            pa.k_cache = k_cache;
            pa.v_cache = v_cache;
            pa.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
            pa.lens = context_lens + b0;
            pa.qstart = query_start + b0;
            pa.out = out;
            pa.status = status;
            pa.num_blocks = desc->num_blocks;
            pa.max_blocks = max_blocks_per_seq;
            pa.batch = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
            pa.q_heads = num_q_heads;
            pa.kv_heads = desc->num_kv_heads;
            pa.head_dim = desc->head_dim;
            pa.group = G;
            pa.max_query_len = max_query_len;
            pa.scale = scale;
            if (launch_prefill(pa, s) != cudaSuccess) return PKV_ERR_CUDA;
        }
        return PKV_OK;
    }
    char* ws = static_cast<char*>(workspace);
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        const int32_t nb = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        MqArgs a{};
        a.q = q;
        a.k_cache = k_cache;
        a.v_cache = v_cache;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.qstart = query_start + b0;
        a.out = out;
        a.partials = reinterpret_cast<float*>(ws + po);
        a.counters = reinterpret_cast<int*>(ws + co);
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = nb;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.num_ctas = num_ctas;
        a.max_query_len = max_query_len;
        const int row_groups = (max_query_len * G + 7) / 8;
        a.wpu = row_groups <= 1 ? 1 : (row_groups <= 2 ? 2 : 4);
        a.test_stall = (flags & PKV_FLAG_TEST_STALL) ? 1 : 0;
        a.scale = scale;
        if (launch_multiquery(a, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status pkv_append_q8(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens, void* k_codes,
                         void* v_codes, float* scales, const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_append_q8");
    pkv_status st = check_desc_q8(desc, false);
    if (st != PKV_OK) return st;
    if (num_tokens < 0) return PKV_ERR_SHAPE;
    if (!k_codes || !v_codes || !scales) return PKV_ERR_NULL;
    if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(scales)) return PKV_ERR_ALIGN;
    if (num_tokens == 0) return PKV_OK;
    if (k == nullptr || v == nullptr || slot_mapping == nullptr) return PKV_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u)) return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        if (num_tokens > 16384) return PKV_ERR_UNSUPPORTED;
        const int64_t num_slots = desc->num_blocks * 16;
        st = run_checked([&](unsigned int* verdict) { return launch_check_slots(slot_mapping, num_tokens, num_slots, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_append_q8(k, v, slot_mapping, num_tokens, k_codes, v_codes, scales, *desc, status, s) ==
                   cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks_q8(const int64_t* pairs, int64_t num_pairs, void* k_codes, void* v_codes, float* scales,
                              const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_copy_blocks_q8");
    pkv_status st = check_desc_q8(desc, false);
    if (st != PKV_OK) return st;
    if (num_pairs < 0) return PKV_ERR_SHAPE;
    if (!k_codes || !v_codes || !scales) return PKV_ERR_NULL;
    if (!aligned16(k_codes) || !aligned16(v_codes) || !aligned16(scales)) return PKV_ERR_ALIGN;
    if (num_pairs == 0) return PKV_OK;
    if (pairs == nullptr) return PKV_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pairs) & 7u) return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        if (num_pairs > 16384) return PKV_ERR_UNSUPPORTED;
        st = run_checked([&](unsigned int* verdict) { return launch_check_pairs(pairs, num_pairs, desc->num_blocks, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    // the code pools move as whole blocks of num_kv_heads * 16 * head_dim bytes (either layout)
    if (launch_copy_blocks(pairs, num_pairs, k_codes, v_codes, *desc, status, s) != cudaSuccess) return PKV_ERR_CUDA;
    return launch_copy_scales(pairs, num_pairs, scales, *desc, status, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

size_t pkv_decode_q8_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                    int32_t max_query_len, const pkv_cache_desc* desc, const pkv_decode_opts* opts) {
    (void)max_blocks_per_seq;
    if (check_desc_q8(desc, true) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc))
        return 0;
    const int G = num_q_heads / desc->num_kv_heads;
    if (max_query_len < 1 || max_query_len * G > kMqMaxRows) return 0;
    size_t co = 0, po = 0;
    return mq_workspace_bytes(batch, desc->num_kv_heads, desc->head_dim,
                              mq_num_ctas(desc->head_dim, batch, opts, true), &co, &po);
}

// The split kernel over int8 pools (arguments checked). The workspace holds the
// counters of `counted` sequences, then the pieces. wide: scales of any size.
static pkv_status run_split_q8(const void* q, const void* k_codes, const void* v_codes, const float* scales,
                               const int32_t* block_tables, int32_t max_blocks_per_seq, const int32_t* context_lens,
                               const int32_t* query_start, int32_t batch, int32_t num_q_heads, int32_t max_query_len,
                               float scale, void* out, void* workspace, size_t workspace_bytes, int32_t counted,
                               bool wide, const pkv_cache_desc* desc, uint32_t flags, const pkv_decode_opts* opts, void* stream) {
    const int G = num_q_heads / desc->num_kv_heads;
    const int num_ctas = mq_num_ctas(desc->head_dim, batch, opts, true);
    size_t co = 0, po = 0;
    const size_t need = mq_workspace_bytes(counted, desc->num_kv_heads, desc->head_dim, num_ctas, &co, &po);
    if (workspace_bytes < need) return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        const pkv_status st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch,
                                                desc->num_blocks, query_start ? 0 : 1, verdict, s);
            if (e != cudaSuccess || query_start == nullptr) return e;
            return launch_check_queries(context_lens, query_start, batch, max_query_len, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    char* ws = static_cast<char*>(workspace);
    const int64_t row = static_cast<int64_t>(num_q_heads) * desc->head_dim * 2;
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        const int32_t nb = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        MqArgs a{};
        // with query offsets the rows are absolute; without, row i of this launch is sequence b0 + i
        a.q = query_start ? q : static_cast<const char*>(q) + b0 * row;
        a.out = query_start ? out : static_cast<char*>(out) + b0 * row;
        a.qstart = query_start ? query_start + b0 : nullptr;
        a.k_cache = k_codes;
        a.v_cache = v_codes;
        a.scales = scales;
        a.q8 = 1;
        a.wide = wide ? 1 : 0;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.partials = reinterpret_cast<float*>(ws + po);
        a.counters = reinterpret_cast<int*>(ws + co);
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = nb;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.num_ctas = num_ctas;
        a.max_query_len = max_query_len;
        const int row_groups = (max_query_len * G + 7) / 8;
        a.wpu = row_groups <= 1 ? 1 : (row_groups <= 2 ? 2 : 4);
        a.test_stall = (flags & PKV_FLAG_TEST_STALL) ? 1 : 0;
        a.scale = scale;
        if (launch_multiquery(a, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status pkv_decode_attention_q8(const void* q, const void* k_codes, const void* v_codes, const float* scales,
                                   const int32_t* block_tables, int32_t max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* query_start, int32_t batch,
                                   int32_t num_q_heads, int32_t max_query_len, float scale, void* out,
                                   void* workspace, size_t workspace_bytes, const pkv_cache_desc* desc,
                                   uint32_t flags, const pkv_decode_opts* opts, void* stream) {
    NvtxRange nvtx_range("pkv_decode_attention_q8");
    pkv_status st = check_desc_q8(desc, true);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    if (!isfinite(scale) || max_query_len < 1) return PKV_ERR_SHAPE;
    if (opts != nullptr && opts->num_ctas < 0) return PKV_ERR_SHAPE;
    const int G = num_q_heads / desc->num_kv_heads;
    if (max_query_len * G > kMqMaxRows) return PKV_ERR_UNSUPPORTED;
    if (query_start == nullptr && max_query_len != 1) return PKV_ERR_SHAPE;
    if (batch == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !k_codes || !v_codes || !scales || !block_tables || !context_lens || !out || !workspace)
        return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(scales) || !aligned16(out) || (reinterpret_cast<uintptr_t>(block_tables) & 3u) ||
        (reinterpret_cast<uintptr_t>(context_lens) & 3u) || (reinterpret_cast<uintptr_t>(query_start) & 3u) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    return run_split_q8(q, k_codes, v_codes, scales, block_tables, max_blocks_per_seq, context_lens, query_start, batch,
                        num_q_heads, max_query_len, scale, out, workspace, workspace_bytes, batch, false, desc, flags, opts, stream);
}

size_t pkv_multiquery_q8_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                        int32_t max_query_len, const pkv_cache_desc* desc) {
    if (check_desc_q8(desc, false) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc)) return 0;
    if (max_query_len < 1 || max_query_len > kMaxQueryLen) return 0;
    if (batch > 0 && !table_width_ok(batch, max_blocks_per_seq)) return 0;
    // The counters of a launch's most sequences lie first, whatever the batch, so that one
    // workspace serves calls of all sizes on either kernel: none writes another's counters.
    size_t co = 0, po = 0;
    const int ctas = desc->head_dim == 128 ? mq_num_ctas(128, batch, nullptr, true) : 0;
    const size_t split = mq_workspace_bytes(kMaxBatchPerLaunch, desc->num_kv_heads, desc->head_dim, ctas, &co, &po);
    const size_t tiles = po + chunk_q8_workspace_bytes(desc->head_dim);
    return split > tiles ? split : tiles;
}

pkv_status pkv_multiquery_attention_q8(const void* q, const void* k_codes, const void* v_codes, const float* scales,
                                       const int32_t* block_tables, int32_t max_blocks_per_seq,
                                       const int32_t* context_lens, const int32_t* query_start, int32_t batch,
                                       int32_t num_q_heads, int32_t max_query_len, float scale, void* out,
                                       void* workspace, size_t workspace_bytes, const pkv_cache_desc* desc,
                                       uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_multiquery_attention_q8");
    pkv_status st = check_desc_q8(desc, false);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    if (!isfinite(scale) || max_query_len < 1) return PKV_ERR_SHAPE;
    if (max_query_len > kMaxQueryLen) return PKV_ERR_UNSUPPORTED;
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;  // the hook is pkv_decode_attention_q8's
    if (batch == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !k_codes || !v_codes || !scales || !block_tables || !context_lens || !query_start || !out || !workspace)
        return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(k_codes) || !aligned16(v_codes) || !aligned16(scales) || !aligned16(out) ||
        !aligned4(block_tables) || !aligned4(context_lens) || !aligned4(query_start) ||
        (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    const int G = num_q_heads / desc->num_kv_heads;
    if (split_kernel_takes(desc, batch, max_blocks_per_seq, max_query_len, G))
        return run_split_q8(q, k_codes, v_codes, scales, block_tables, max_blocks_per_seq, context_lens, query_start, batch,
                            num_q_heads, max_query_len, scale, out, workspace, workspace_bytes, kMaxBatchPerLaunch, true,
                            desc, flags, nullptr, stream);
    size_t co = 0, po = 0;
    mq_workspace_bytes(kMaxBatchPerLaunch, desc->num_kv_heads, desc->head_dim, 0, &co, &po);
    if (workspace_bytes < po + chunk_q8_workspace_bytes(desc->head_dim)) return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch,
                                                desc->num_blocks, 0, verdict, s);
            if (e != cudaSuccess) return e;
            return launch_check_queries(context_lens, query_start, batch, max_query_len, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        ChunkArgs a{};
        a.q = q;
        a.k_codes = k_codes;
        a.v_codes = v_codes;
        a.scales = scales;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.qstart = query_start + b0;
        a.out = out;
        a.workspace = static_cast<char*>(workspace) + po;
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.max_query_len = max_query_len;
        a.scale = scale;
        a.group_inverse = ((uint64_t(1) << 37) + G - 1) / G;
        if (launch_chunk_q8(a, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status pkv_gather(const void* k_cache, const void* v_cache, const int32_t* block_tables,
                      int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* token_start,
                      const int32_t* row_start, int32_t batch, int64_t num_rows, void* k_out, void* v_out,
                      const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_gather");
    const pkv_status st = check_desc(desc);
    if (st != PKV_OK) return st;
    return run_gather(k_cache, v_cache, nullptr, block_tables, max_blocks_per_seq, context_lens, token_start, row_start,
                      batch, num_rows, k_out, v_out, desc->dtype, desc, flags, static_cast<cudaStream_t>(stream));
}

pkv_status pkv_gather_q8(const void* k_codes, const void* v_codes, const float* scales, const int32_t* block_tables,
                         int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* token_start,
                         const int32_t* row_start, int32_t batch, int64_t num_rows, void* k_out, void* v_out,
                         int32_t out_dtype, const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_gather_q8");
    const pkv_status st = check_desc_q8(desc, false);
    if (st != PKV_OK) return st;
    if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_DTYPE;
    if (num_rows > 0 && batch > 0) {
        if (scales == nullptr) return PKV_ERR_NULL;
        if (!aligned16(scales)) return PKV_ERR_ALIGN;
    }
    return run_gather(k_codes, v_codes, scales, block_tables, max_blocks_per_seq, context_lens, token_start, row_start,
                      batch, num_rows, k_out, v_out, out_dtype, desc, flags, static_cast<cudaStream_t>(stream));
}

pkv_status pkv_verify_drafts(const void* target_probs, int64_t target_stride, int64_t num_target_rows,
                             const void* draft_probs, int64_t draft_stride, int64_t num_draft_rows, int32_t dtype,
                             int32_t vocab, const int32_t* draft_tokens, const float* accept_uniform,
                             const float* sample_uniform, const int32_t* query_start, const int32_t* draft_start,
                             int32_t batch, int32_t max_draft_len, const int32_t* context_lens,
                             int32_t* new_context_lens, int32_t* out_tokens, int32_t* num_accepted, uint32_t flags,
                             void* stream) {
    NvtxRange nvtx_range("pkv_verify_drafts");
    if (dtype != PKV_F32 && dtype != PKV_BF16) return PKV_ERR_DTYPE;
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;
    if (batch < 0 || vocab < 1 || vocab > kMaxVocab || max_draft_len < 0 || max_draft_len > kMaxDraftLen)
        return PKV_ERR_SHAPE;
    if (num_target_rows < 0 || num_target_rows >= (int64_t(1) << 31) || num_draft_rows < 0 ||
        num_draft_rows >= (int64_t(1) << 31))
        return PKV_ERR_SHAPE;
    // a row stride: at least the row, and such that the last row's offset stays far inside 64 bits
    const int64_t most = int64_t(1) << 31;
    if (num_target_rows > 0 && (target_stride < vocab || target_stride >= most)) return PKV_ERR_SHAPE;
    if (draft_probs != nullptr && num_draft_rows > 0 && (draft_stride < vocab || draft_stride >= most))
        return PKV_ERR_SHAPE;
    if (batch == 0) return PKV_OK;
    if (!sample_uniform || !query_start || !draft_start || !out_tokens || !num_accepted) return PKV_ERR_NULL;
    if (num_target_rows > 0 && !target_probs) return PKV_ERR_NULL;
    if (num_draft_rows > 0 && (!draft_tokens || !accept_uniform)) return PKV_ERR_NULL;
    if ((context_lens == nullptr) != (new_context_lens == nullptr)) return PKV_ERR_NULL;
    const uintptr_t elem = dtype == PKV_F32 ? 3u : 1u;
    if ((reinterpret_cast<uintptr_t>(target_probs) & elem) || (reinterpret_cast<uintptr_t>(draft_probs) & elem) ||
        !aligned4(draft_tokens) || !aligned4(accept_uniform) || !aligned4(sample_uniform) || !aligned4(query_start) ||
        !aligned4(draft_start) || !aligned4(context_lens) || !aligned4(new_context_lens) || !aligned4(out_tokens) ||
        !aligned4(num_accepted))
        return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    VerifyArgs a{};
    a.target = target_probs;
    a.draft = draft_probs;
    a.draft_tokens = draft_tokens;
    a.accept = accept_uniform;
    a.sample = sample_uniform;
    a.query_start = query_start;
    a.draft_start = draft_start;
    a.lens = context_lens;
    a.new_lens = new_context_lens;
    a.out_tokens = out_tokens;
    a.num_accepted = num_accepted;
    a.status = device_info().status;
    a.target_stride = target_stride;
    a.draft_stride = draft_stride;
    a.num_target_rows = num_target_rows;
    a.num_draft_rows = num_draft_rows;
    a.vocab = vocab;
    a.batch = batch;
    a.max_draft_len = max_draft_len;
    if (a.status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        const pkv_status st = run_checked([&](unsigned int* verdict) { return launch_check_verify(a, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_verify(a, dtype, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_append_q4(const void* k, const void* v, const int64_t* slot_mapping, int64_t num_tokens, void* cache,
                         const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_append_q4");
    pkv_status st = check_desc_q4(desc);
    if (st != PKV_OK) return st;
    if (num_tokens < 0 || num_tokens >= (int64_t(1) << 31) / (2 * static_cast<int64_t>(desc->num_kv_heads))) return PKV_ERR_SHAPE;  // rows are counted in 32 bits
    if (cache == nullptr) return PKV_ERR_NULL;
    if (!aligned16(cache)) return PKV_ERR_ALIGN;
    if (num_tokens == 0) return PKV_OK;
    if (k == nullptr || v == nullptr || slot_mapping == nullptr) return PKV_ERR_NULL;
    if (!aligned16(k) || !aligned16(v) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u)) return PKV_ERR_ALIGN;
    if ((flags & PKV_FLAG_CHECKED) && num_tokens > 16384) return PKV_ERR_UNSUPPORTED;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RotaryAppendArgs a{};
    a.k = k;
    a.v = v;
    a.k_stride = a.v_stride = static_cast<int64_t>(desc->num_kv_heads) * desc->head_dim;
    a.slots = slot_mapping;
    a.k_cache = cache;
    a.status = device_info().status;
    a.num_tokens = num_tokens;
    a.num_slots = desc->num_blocks * 16;
    a.kv_heads = desc->num_kv_heads;
    if (a.status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) { return launch_check_slots(slot_mapping, num_tokens, a.num_slots, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_append_rotary(a, *desc, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_copy_blocks_q4(const int64_t* pairs, int64_t num_pairs, void* cache, const pkv_cache_desc* desc,
                              uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_copy_blocks_q4");
    pkv_status st = check_desc_q4(desc);
    if (st != PKV_OK) return st;
    if (num_pairs < 0 || num_pairs >= (int64_t(1) << 31)) return PKV_ERR_SHAPE;  // (destinations are distinct blocks)
    if (cache == nullptr) return PKV_ERR_NULL;
    if (!aligned16(cache)) return PKV_ERR_ALIGN;
    if (num_pairs == 0) return PKV_OK;
    if (pairs == nullptr) return PKV_ERR_NULL;
    if (reinterpret_cast<uintptr_t>(pairs) & 7u) return PKV_ERR_ALIGN;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        if (num_pairs > 16384) return PKV_ERR_UNSUPPORTED;
        st = run_checked([&](unsigned int* verdict) { return launch_check_pairs(pairs, num_pairs, desc->num_blocks, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    const int64_t block_vecs = static_cast<int64_t>(desc->num_kv_heads) * (PKV_Q4_RECORD_BYTES(desc->head_dim) / 16);
    return launch_copy_pool(pairs, num_pairs, cache, desc->num_blocks, block_vecs, status, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_gather_q4(const void* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                         const int32_t* context_lens, const int32_t* token_start, const int32_t* row_start, int32_t batch,
                         int64_t num_rows, void* k_out, void* v_out, int32_t out_dtype, const pkv_cache_desc* desc,
                         uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_gather_q4");
    const pkv_status st = check_desc_q4(desc);
    if (st != PKV_OK) return st;
    if (out_dtype != PKV_F32 && out_dtype != PKV_BF16) return PKV_ERR_DTYPE;
    return run_gather(cache, cache, nullptr, block_tables, max_blocks_per_seq, context_lens, token_start, row_start, batch,
                      num_rows, k_out, v_out, out_dtype, desc, flags, static_cast<cudaStream_t>(stream));
}

static size_t q4_counters_bytes(const pkv_cache_desc* desc) {
    return (static_cast<size_t>(kMaxBatchPerLaunch) * desc->num_kv_heads * 4 * sizeof(int) + 255) / 256 * 256;
}

size_t pkv_multiquery_q4_workspace_size(int32_t batch, int32_t num_q_heads, int32_t max_blocks_per_seq,
                                        int32_t max_query_len, const pkv_cache_desc* desc) {
    if (check_desc_q4(desc) != PKV_OK || batch < 0 || !q_heads_ok(num_q_heads, desc)) return 0;
    if (max_query_len < 1 || max_query_len > kMaxQueryLen) return 0;
    if (batch > 0 && !table_width_ok(batch, max_blocks_per_seq)) return 0;
    // the counters of a launch's most sequences lie first, whatever the sizes, so that one workspace
    // serves calls of all sizes on either kernel
    const int64_t rows = static_cast<int64_t>(max_query_len) * (num_q_heads / desc->num_kv_heads);
    const size_t tiles = chunk_q8_workspace_bytes(desc->head_dim);
    const size_t split = q4_partials_bytes(desc->head_dim, q4_plan(desc->head_dim, rows < kMq4Rows ? static_cast<int>(rows) : kMq4Rows));
    return q4_counters_bytes(desc) + (split > tiles ? split : tiles);
}

// 4-bit multi-query calls: up to kMq4Rows query rows per (sequence, KV head) run on the
// kernel that splits the cache (pkv_q4.cu), more in tiles (pkv_chunk_q8.cu), whose 128 rows
// cost the same however many are used. Split / tiles in us, 32 rows of 128 but as noted:
// 32 sequences of 8192 154 / 209 (16 rows 87 / 211; 16 rows of 64 59 / 184), one of 32768 40 /
// 46, of 1024 15.7 / 18.6, 64 of 300 43 / 48, 4 of 300 16.5 / 14.4 (the one size seen that loses).
// The call's largest query count decides for all of its sequences: a chunk of 512 beside 31 that
// decode, all on 8192 tokens, takes 258 us, where the two apart take 72 and 55.
static bool split_takes_q4(int64_t rows) { return rows <= kMq4Rows; }

// Both attention calls over the 4-bit cache, after the checks of their own.
static pkv_status run_attention_q4(const void* q, const void* cache, const int32_t* block_tables, int32_t max_blocks_per_seq,
                                   const int32_t* context_lens, const int32_t* query_start, int32_t batch, int32_t num_q_heads,
                                   int32_t max_query_len, float scale, void* out, void* workspace, size_t workspace_bytes,
                                   const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    if (!isfinite(scale)) return PKV_ERR_SHAPE;
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;
    if (batch == 0) return PKV_OK;
    if (!table_width_ok(batch, max_blocks_per_seq)) return PKV_ERR_SHAPE;
    if (!q || !cache || !block_tables || !context_lens || !out || !workspace) return PKV_ERR_NULL;
    if (!aligned16(q) || !aligned16(cache) || !aligned16(out) || !aligned4(block_tables) || !aligned4(context_lens) ||
        !aligned4(query_start) || (reinterpret_cast<uintptr_t>(workspace) & 255u))
        return PKV_ERR_ALIGN;
    if (workspace_bytes < pkv_multiquery_q4_workspace_size(batch, num_q_heads, max_blocks_per_seq, max_query_len, desc))
        return PKV_ERR_WORKSPACE;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        const pkv_status st = run_checked([&](unsigned int* verdict) {
            cudaError_t e = launch_check_decode(block_tables, max_blocks_per_seq, context_lens, batch, desc->num_blocks,
                                                query_start ? 0 : 1, verdict, s);
            if (e != cudaSuccess || query_start == nullptr) return e;
            return launch_check_queries(context_lens, query_start, batch, max_query_len, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    const int G = num_q_heads / desc->num_kv_heads;
    const int64_t rows = static_cast<int64_t>(max_query_len) * G;
    char* ws = static_cast<char*>(workspace);
    const size_t pieces = q4_counters_bytes(desc);
    const bool tiles = query_start != nullptr && !split_takes_q4(rows);
    const Q4Plan plan = tiles ? Q4Plan{} : q4_plan(desc->head_dim, static_cast<int>(rows));
    const int64_t row = static_cast<int64_t>(num_q_heads) * desc->head_dim * 2;
    for (int32_t b0 = 0; b0 < batch; b0 += kMaxBatchPerLaunch) {
        const int32_t nb = batch - b0 < kMaxBatchPerLaunch ? batch - b0 : kMaxBatchPerLaunch;
        if (tiles) {
            ChunkArgs a{};
            a.q = q;
            a.k_codes = cache;
            a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
            a.lens = context_lens + b0;
            a.qstart = query_start + b0;
            a.out = out;
            a.workspace = ws + pieces;
            a.status = status;
            a.num_blocks = desc->num_blocks;
            a.max_blocks = max_blocks_per_seq;
            a.batch = nb;
            a.q_heads = num_q_heads;
            a.kv_heads = desc->num_kv_heads;
            a.head_dim = desc->head_dim;
            a.group = G;
            a.max_query_len = max_query_len;
            a.scale = scale;
            a.group_inverse = ((uint64_t(1) << 37) + G - 1) / G;
            if (launch_chunk_q4(a, s) != cudaSuccess) return PKV_ERR_CUDA;
            continue;
        }
        Q4Args a{};
        // with query offsets the rows are absolute; without, row i of this launch is sequence b0 + i
        a.q = query_start ? q : static_cast<const char*>(q) + b0 * row;
        a.out = query_start ? out : static_cast<char*>(out) + b0 * row;
        a.qstart = query_start ? query_start + b0 : nullptr;
        a.cache = cache;
        a.tables = block_tables + static_cast<int64_t>(b0) * max_blocks_per_seq;
        a.lens = context_lens + b0;
        a.status = status;
        a.num_blocks = desc->num_blocks;
        a.max_blocks = max_blocks_per_seq;
        a.batch = nb;
        a.q_heads = num_q_heads;
        a.kv_heads = desc->num_kv_heads;
        a.head_dim = desc->head_dim;
        a.group = G;
        a.max_query_len = max_query_len;
        a.scale = scale;
        a.counters = reinterpret_cast<int*>(ws);
        a.partials = reinterpret_cast<float*>(ws + pieces);
        a.num_ctas = plan.num_ctas;
        a.tiles = plan.tiles;
        a.warps_per_unit = plan.warps_per_unit;
        if (launch_mq4(a, plan, s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    return PKV_OK;
}

pkv_status pkv_decode_attention_q4(const void* q, const void* cache, const int32_t* block_tables,
                                   int32_t max_blocks_per_seq, const int32_t* context_lens, int32_t batch,
                                   int32_t num_q_heads, float scale, void* out, void* workspace, size_t workspace_bytes,
                                   const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_decode_attention_q4");
    const pkv_status st = check_desc_q4(desc);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc)) return PKV_ERR_SHAPE;
    if (num_q_heads / desc->num_kv_heads > kMqMaxRows) return PKV_ERR_UNSUPPORTED;
    return run_attention_q4(q, cache, block_tables, max_blocks_per_seq, context_lens, nullptr, batch, num_q_heads, 1, scale, out,
                            workspace, workspace_bytes, desc, flags, stream);
}

pkv_status pkv_multiquery_attention_q4(const void* q, const void* cache, const int32_t* block_tables,
                                       int32_t max_blocks_per_seq, const int32_t* context_lens, const int32_t* query_start,
                                       int32_t batch, int32_t num_q_heads, int32_t max_query_len, float scale, void* out,
                                       void* workspace, size_t workspace_bytes, const pkv_cache_desc* desc, uint32_t flags,
                                       void* stream) {
    NvtxRange nvtx_range("pkv_multiquery_attention_q4");
    const pkv_status st = check_desc_q4(desc);
    if (st != PKV_OK) return st;
    if (batch < 0 || !q_heads_ok(num_q_heads, desc) || max_query_len < 1) return PKV_ERR_SHAPE;
    if (max_query_len > kMaxQueryLen) return PKV_ERR_UNSUPPORTED;
    if (batch > 0 && query_start == nullptr) return PKV_ERR_NULL;
    return run_attention_q4(q, cache, block_tables, max_blocks_per_seq, context_lens, query_start, batch, num_q_heads, max_query_len,
                            scale, out, workspace, workspace_bytes, desc, flags, stream);
}

pkv_status pkv_rotary_frequencies(int32_t rotary_dim, double base, const pkv_rotary_scaling* scaling, double* frequencies) {
    if (frequencies == nullptr) return PKV_ERR_NULL;
    return rotary_frequencies(rotary_dim, base, scaling, frequencies) ? PKV_OK : PKV_ERR_SHAPE;
}

pkv_status pkv_rotary_table(const double* frequencies, int32_t rotary_dim, int64_t first_position, int64_t num_positions,
                            float factor, float* table, void* stream) {
    NvtxRange nvtx_range("pkv_rotary_table");
    const int64_t most = (int64_t(1) << 31) - 1;
    if (rotary_dim < 2 || rotary_dim > 8192 || rotary_dim % 2 || !isfinite(factor)) return PKV_ERR_SHAPE;
    if (first_position < 0 || num_positions < 0 || first_position > most || num_positions > most - first_position) return PKV_ERR_SHAPE;
    if (num_positions == 0) return PKV_OK;
    if (!frequencies || !table) return PKV_ERR_NULL;
    if ((reinterpret_cast<uintptr_t>(frequencies) & 7u) || !aligned16(table)) return PKV_ERR_ALIGN;
    return launch_rotary_table(frequencies, rotary_dim / 2, first_position, num_positions, factor, table,
                               static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_append_rotary(const void* q, int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                             const int32_t* positions, const float* table, int32_t num_positions, int32_t rotary_dim,
                             int32_t interleaved, const int64_t* slot_mapping, int64_t num_tokens, int32_t num_q_heads,
                             void* q_out, int64_t q_out_stride, void* k_cache, void* v_cache, float* scales,
                             const pkv_cache_desc* desc, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_append_rotary");
    if (desc == nullptr) return PKV_ERR_NULL;
    pkv_status st = desc->dtype == PKV_INT4 ? check_desc_q4(desc) : desc->dtype == PKV_INT8 ? check_desc_q8(desc, false) : check_desc(desc);
    if (st != PKV_OK) return st;
    if (num_q_heads < 0 || num_q_heads > PKV_MAX_Q_HEADS || rotary_dim < 2 || rotary_dim > desc->head_dim || rotary_dim % 2 ||
        num_positions < 1 || num_tokens < 0)
        return PKV_ERR_SHAPE;
    // rows are counted in 32 bits
    if (num_tokens >= (int64_t(1) << 31) / (num_q_heads + 2 * static_cast<int64_t>(desc->num_kv_heads))) return PKV_ERR_SHAPE;
    if (!k_cache || (desc->dtype != PKV_INT4 && !v_cache) || (desc->dtype == PKV_INT8 && !scales)) return PKV_ERR_NULL;
    if (!aligned16(k_cache) || !aligned16(v_cache) || !aligned16(scales)) return PKV_ERR_ALIGN;
    if (num_tokens == 0) return PKV_OK;
    if (!k || !v || !positions || !table || !slot_mapping || (num_q_heads > 0 && (!q || !q_out))) return PKV_ERR_NULL;
    const int64_t per_vector = desc->dtype == PKV_F32 ? 4 : 8;  // elements of 16 bytes
    const int64_t q_row = static_cast<int64_t>(num_q_heads) * desc->head_dim, kv_row = static_cast<int64_t>(desc->num_kv_heads) * desc->head_dim;
    const int64_t strides[4] = {num_q_heads > 0 ? q_stride : q_row, num_q_heads > 0 ? q_out_stride : q_row, k_stride, v_stride};
    const int64_t rows[4] = {q_row, q_row, kv_row, kv_row};
    for (int i = 0; i < 4; ++i) {
        if (num_tokens > 1 && (strides[i] < rows[i] || strides[i] >= (int64_t(1) << 31))) return PKV_ERR_SHAPE;
        if (num_tokens > 1 && strides[i] % per_vector) return PKV_ERR_ALIGN;
    }
    if ((num_q_heads > 0 && (!aligned16(q) || !aligned16(q_out))) || !aligned16(k) || !aligned16(v) || !aligned16(table) ||
        !aligned4(positions) || (reinterpret_cast<uintptr_t>(slot_mapping) & 7u))
        return PKV_ERR_ALIGN;
    if ((flags & PKV_FLAG_CHECKED) && num_tokens > 16384) return PKV_ERR_UNSUPPORTED;
    if (num_q_heads > 0) {
        const size_t size = 16 / per_vector, count = static_cast<size_t>(num_tokens);
        const size_t q_bytes = q_row * size, kv_bytes = kv_row * size;
        auto step = [&](int i) { return num_tokens > 1 ? strides[i] * size : rows[i] * size; };
        if ((q_out != q || step(0) != step(1)) && overlap_rows(num_tokens, q_out, q_bytes, step(1), q, q_bytes, step(0))) return PKV_ERR_OVERLAP;
        if (overlap_rows(num_tokens, q_out, q_bytes, step(1), k, kv_bytes, step(2)) || overlap_rows(num_tokens, q_out, q_bytes, step(1), v, kv_bytes, step(3)))
            return PKV_ERR_OVERLAP;
        const size_t records = static_cast<size_t>(desc->num_blocks) * desc->num_kv_heads, codes = 16 * static_cast<size_t>(desc->head_dim);
        const bool q4 = desc->dtype == PKV_INT4;
        const size_t pool = records * (q4 ? PKV_Q4_RECORD_BYTES(desc->head_dim) : desc->dtype == PKV_INT8 ? codes : codes * size);
        const struct {
            const void* p;
            size_t n;
        } others[] = {{positions, 4 * count}, {slot_mapping, 8 * count}, {table, 4 * static_cast<size_t>(num_positions) * rotary_dim},
                      {k_cache, pool}, {v_cache, q4 ? 0 : pool}, {scales, desc->dtype == PKV_INT8 ? records * 128 : 0}};
        for (const auto& x : others)
            if (overlap(q_out, (count - 1) * step(1) + q_bytes, x.p, x.n)) return PKV_ERR_OVERLAP;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    RotaryAppendArgs a{};
    a.q = q;
    a.k = k;
    a.v = v;
    a.positions = positions;
    a.table = table;
    a.slots = slot_mapping;
    a.q_out = q_out;
    a.k_cache = k_cache;
    a.v_cache = v_cache;
    a.scales = scales;
    a.status = device_info().status;
    a.q_stride = strides[0];
    a.q_out_stride = strides[1];
    a.k_stride = k_stride;
    a.v_stride = v_stride;
    a.num_tokens = num_tokens;
    a.num_slots = desc->num_blocks * 16;
    a.num_positions = num_positions;
    a.rotary_dim = rotary_dim;
    a.interleaved = interleaved ? 1 : 0;
    a.q_heads = num_q_heads;
    a.kv_heads = desc->num_kv_heads;
    if (a.status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        st = run_checked([&](unsigned int* verdict) {
            const cudaError_t e = launch_check_slots(slot_mapping, num_tokens, a.num_slots, verdict, s);
            return e != cudaSuccess ? e : launch_check_positions(positions, slot_mapping, num_tokens, num_positions, verdict, s);
        }, s);
        if (st != PKV_OK) return st;
    }
    return launch_append_rotary(a, *desc, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_plan_step(const int32_t* context_lens, const int32_t* new_tokens, const int32_t* held_blocks,
                         const int32_t* free_blocks, int64_t free_capacity, const int32_t* free_count, int32_t* block_tables,
                         int32_t max_blocks_per_seq, int32_t batch, int64_t num_rows, int64_t num_blocks, int64_t* slot_mapping,
                         int32_t* positions, int32_t* query_start, int32_t* new_context_lens, int32_t* new_held_blocks,
                         int32_t* new_free_count, int32_t* result, uint32_t flags, void* stream) {
    NvtxRange nvtx_range("pkv_plan_step");
    const int64_t bound = int64_t(1) << 31;
    if (flags & PKV_FLAG_TEST_STALL) return PKV_ERR_UNSUPPORTED;
    if (batch < 0 || num_rows < 0 || num_rows >= bound || free_capacity < 0 || free_capacity >= bound || num_blocks < 0) return PKV_ERR_SHAPE;
    if (batch > PKV_MAX_PLAN_BATCH) return PKV_ERR_UNSUPPORTED;
    if (max_blocks_per_seq < 1 || static_cast<int64_t>(max_blocks_per_seq) * 16 >= bound) return PKV_ERR_SHAPE;
    if (!free_count || !query_start || !new_free_count || !result) return PKV_ERR_NULL;
    if (batch > 0 && (!context_lens || !new_tokens || !held_blocks || !block_tables || !new_context_lens || !new_held_blocks)) return PKV_ERR_NULL;
    if (free_capacity > 0 && !free_blocks) return PKV_ERR_NULL;
    if (num_rows > 0 && (!slot_mapping || !positions)) return PKV_ERR_NULL;
    const size_t per_seq = 4 * static_cast<size_t>(batch);
    const struct {
        const void* p;
        size_t n;
    } in[] = {{context_lens, per_seq}, {new_tokens, per_seq}, {held_blocks, per_seq}, {free_blocks, 4 * static_cast<size_t>(free_capacity)}, {free_count, 4}},
      out[] = {{block_tables, per_seq * max_blocks_per_seq}, {slot_mapping, 8 * static_cast<size_t>(num_rows)}, {positions, 4 * static_cast<size_t>(num_rows)},
               {query_start, per_seq + 4}, {new_context_lens, per_seq}, {new_held_blocks, per_seq}, {new_free_count, 4}, {result, 8}};
    for (const auto& x : in)
        if (!aligned4(x.p)) return PKV_ERR_ALIGN;
    for (const auto& x : out)
        if (!aligned4(x.p)) return PKV_ERR_ALIGN;
    if (reinterpret_cast<uintptr_t>(slot_mapping) & 7u) return PKV_ERR_ALIGN;
    for (const auto& x : out) {
        for (const auto& y : in)
            if (overlap(x.p, x.n, y.p, y.n)) return PKV_ERR_OVERLAP;
        for (const auto& y : out)
            if (&x != &y && overlap(x.p, x.n, y.p, y.n)) return PKV_ERR_OVERLAP;
    }
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    PlanArgs a{};
    a.lens = context_lens;
    a.new_tokens = new_tokens;
    a.held = held_blocks;
    a.free_blocks = free_blocks;
    a.free_count = free_count;
    a.tables = block_tables;
    a.slots = slot_mapping;
    a.positions = positions;
    a.query_start = query_start;
    a.new_lens = new_context_lens;
    a.new_held = new_held_blocks;
    a.new_free_count = new_free_count;
    a.result = result;
    a.status = device_info().status;
    a.free_capacity = free_capacity;
    a.num_blocks = num_blocks > 0 && num_blocks < bound ? num_blocks : bound;
    a.num_rows = num_rows;
    a.batch = batch;
    a.max_blocks = max_blocks_per_seq;
    if (a.status == nullptr) return PKV_ERR_CUDA;
    if (flags & PKV_FLAG_CHECKED) {
        const pkv_status st = run_checked([&](unsigned int* verdict) { return launch_check_plan(a, verdict, s); }, s);
        if (st != PKV_OK) return st;
    }
    return launch_plan(a, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

pkv_status pkv_device_status(uint32_t* bits_out, int clear, void* stream) {
    unsigned int* status = device_info().status;
    if (status == nullptr) return PKV_ERR_CUDA;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    unsigned int host = 0;
    if (cudaMemcpyAsync(&host, status, sizeof(unsigned int), cudaMemcpyDeviceToHost, s) != cudaSuccess)
        return PKV_ERR_CUDA;
    if (cudaStreamSynchronize(s) != cudaSuccess) return PKV_ERR_CUDA;
    if (clear) {
        if (cudaMemsetAsync(status, 0, sizeof(unsigned int), s) != cudaSuccess) return PKV_ERR_CUDA;
        if (cudaStreamSynchronize(s) != cudaSuccess) return PKV_ERR_CUDA;
    }
    if (bits_out) *bits_out = host;
    return PKV_OK;
}

}  // extern "C"
