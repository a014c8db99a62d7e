// C ABI of the serving operators: prompt attention, block tables, the 8-bit block cache.
// Every entry point returns an rkv_status and never throws; see include/rkv.h.
#include <atomic>
#include <climits>

#include "api_common.h"
#include "launchers.h"

using namespace rkv;
using namespace rkv::api;

namespace {

// SMs of the current device, or RKV_ERR_UNSUPPORTED if it is not an sm_100.  Kept per device
// ordinal: a device's properties do not change within a process.
rkv_status device_sms(int* sms)
{
    constexpr int kDevices = 64;
    static std::atomic<int> known[kDevices];   // 0: not asked, > 0: SMs, < 0: not sm_100
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kDevices)
        return RKV_ERR_CUDA;
    int v = known[dev].load(std::memory_order_relaxed);
    if (v == 0) {
        int major = 0, minor = 0, n = 0;
        if (cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev) != cudaSuccess ||
            cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return RKV_ERR_CUDA;
        v = (major == 10 && minor == 0) ? n : -1;
        known[dev].store(v, std::memory_order_relaxed);
    }
    if (v < 0)
        return RKV_ERR_UNSUPPORTED;
    *sms = v;
    return RKV_OK;
}

// The kernels' workspace is sized for this many SMs or fewer (the B200 has 148).
constexpr int kMaxSms = 160;

bool half_type(int32_t t) { return t == RKV_DTYPE_BF16 || t == RKV_DTYPE_F16; }

// Up to 2^127, so that its product with log2(e) is finite too.
bool scale_ok(float s) { return s == 0.0f || (s > 0.0f && s <= 0x1p127f); }

// Element strides below 2^38, so that byte strides fit a tensor map's 40 bits.
bool stride_ok(int64_t s, int64_t unit) { return s > 0 && s % unit == 0 && s < (int64_t(1) << 38); }

rkv_status check_heads(int32_t head_dim, int32_t n_kv_heads, int32_t n_q_heads, int32_t batch)
{
    if (n_kv_heads <= 0 || n_q_heads <= 0 || n_q_heads % n_kv_heads != 0 || batch <= 0)
        return RKV_ERR_INVALID_ARG;
    if ((head_dim != 64 && head_dim != 128) || n_q_heads / n_kv_heads > 16 || batch > RKV_MAX_BATCH ||
        n_kv_heads > 4096 || n_q_heads > 65535)
        return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

rkv_status check_prefill(const rkv_prefill_config* c)
{
    if (!c)
        return RKV_ERR_INVALID_ARG;
    const rkv_status s = check_heads(c->head_dim, c->n_kv_heads, c->n_q_heads, c->batch);
    if (s != RKV_OK)
        return s;
    if (c->in_dtype == RKV_DTYPE_F32)
        return RKV_ERR_UNSUPPORTED;
    if (!half_type(c->in_dtype) || (c->out_dtype != c->in_dtype && c->out_dtype != RKV_DTYPE_F32) ||
        (c->kv_padded != 0 && c->kv_padded != 1) || !scale_ok(c->scale) || c->q_rows < 0 || c->kv_rows < 0)
        return RKV_ERR_INVALID_ARG;
    // rows are rounded up to query tiles of up to 128 tokens, two at a time, and keys to tiles of 64, in 31 bits
    if (c->q_rows > INT32_MAX - 255 || c->kv_rows > INT32_MAX - 255)
        return RKV_ERR_UNSUPPORTED;
    const int64_t out_unit = c->out_dtype == RKV_DTYPE_F32 ? 4 : 8;
    if (!stride_ok(c->q_row_stride, 8) || !stride_ok(c->q_head_stride, 8) || !stride_ok(c->kv_row_stride, 8) ||
        !stride_ok(c->kv_head_stride, 8) || !stride_ok(c->out_row_stride, out_unit) ||
        !stride_ok(c->out_head_stride, out_unit) || (c->kv_padded && !stride_ok(c->kv_plane_stride, 8)))
        return RKV_ERR_INVALID_ARG;
    return RKV_OK;
}

rkv_status check_blocks(int32_t batch, int32_t max_blocks, int32_t block_size, int32_t n_blocks)
{
    if (batch <= 0 || max_blocks <= 0 || n_blocks <= 0)
        return RKV_ERR_INVALID_ARG;
    if (batch > RKV_MAX_BATCH || (block_size != 16 && block_size != 32 && block_size != 64 && block_size != 128) ||
        static_cast<int64_t>(n_blocks) * block_size > INT32_MAX ||
        static_cast<int64_t>(max_blocks) * block_size > INT32_MAX)
        return RKV_ERR_UNSUPPORTED;
    return RKV_OK;
}

rkv_status check_kv8(const rkv_kv8_cache* c)
{
    if (!c)
        return RKV_ERR_INVALID_ARG;
    rkv_status s = check_heads(c->head_dim, c->n_kv_heads, c->n_q_heads, c->batch);
    if (s == RKV_OK)
        s = check_blocks(c->batch, c->max_blocks, c->block_size, c->n_blocks);
    if (s != RKV_OK)
        return s;
    // the decode rounds lengths up to tiles of 64 tokens in 31 bits
    if (static_cast<int64_t>(c->max_blocks) * c->block_size > INT32_MAX - 63)
        return RKV_ERR_UNSUPPORTED;
    if (c->in_dtype == RKV_DTYPE_F32)
        return RKV_ERR_UNSUPPORTED;
    if (!half_type(c->in_dtype) || (c->out_dtype != c->in_dtype && c->out_dtype != RKV_DTYPE_F32) ||
        (c->code_type != RKV_KV8_INT8 && c->code_type != RKV_KV8_E4M3) || !scale_ok(c->scale))
        return RKV_ERR_INVALID_ARG;
    return RKV_OK;
}

rkv_status check_kv8_buffers(const rkv_kv8_cache* c)
{
    const rkv_status s = check_kv8(c);
    if (s != RKV_OK)
        return s;
    if (!c->codes_K || !c->codes_V || !c->scale_K || !c->scale_V || !c->device_status || !aligned(c->codes_K, 16) ||
        !aligned(c->codes_V, 16) || !aligned(c->scale_K, 4) || !aligned(c->scale_V, 4) ||
        !aligned(c->device_status, 4))
        return RKV_ERR_INVALID_ARG;
    return RKV_OK;
}

bool ints_ok(const void* p) { return p && aligned(p, 4); }

}  // namespace

extern "C" {

rkv_status rkv_prefill_attn(const rkv_prefill_config* cfg, const void* q, const void* K, const void* V,
                            const int32_t* q_off, const int32_t* kv_off, const int32_t* kv_len, void* out, float* lse,
                            int32_t* device_status, void* stream)
{
    const ApiRange range("rkv_prefill_attn");
    rkv_status s = check_prefill(cfg);
    if (s != RKV_OK)
        return s;
    if (cfg->q_rows == 0)
        return RKV_OK;
    if (!q || !out || !aligned(q, 16) || !aligned(out, 16) || !aligned(lse, 4) || !ints_ok(q_off) ||
        !aligned(kv_off, 4) || !aligned(kv_len, 4) || !ints_ok(device_status) ||
        (cfg->kv_rows > 0 && (!K || !V)) || !aligned(K, 16) || !aligned(V, 16))
        return RKV_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != RKV_OK)
        return s;
    return cuda_status(launch_prefill(*cfg, q, K, V, q_off, kv_off, kv_len, out, lse, device_status, sms,
                                      static_cast<cudaStream_t>(stream)));
}

rkv_status rkv_blocks_extend(const rkv_blocks_config* cfg, const int32_t* lengths, const int32_t* new_counts,
                             int32_t* block_table, const int32_t* free_list, const int32_t* n_free, int32_t* new_off,
                             int32_t* slot_map, int64_t max_new, int32_t* lengths_out, int32_t* n_free_out,
                             int32_t* device_status, void* stream)
{
    const ApiRange range("rkv_blocks_extend");
    if (!cfg)
        return RKV_ERR_INVALID_ARG;
    rkv_status s = check_blocks(cfg->batch, cfg->max_blocks, cfg->block_size, cfg->n_blocks);
    if (s != RKV_OK)
        return s;
    if (!ints_ok(lengths) || !ints_ok(new_counts) || !ints_ok(block_table) || !ints_ok(free_list) ||
        !ints_ok(n_free) || !ints_ok(new_off) || !ints_ok(lengths_out) || !ints_ok(n_free_out) ||
        !ints_ok(device_status) || max_new < 0 || max_new > INT32_MAX || (max_new > 0 && !ints_ok(slot_map)))
        return RKV_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != RKV_OK)
        return s;
    return cuda_status(launch_blocks_extend(*cfg, lengths, new_counts, block_table, free_list, n_free, new_off,
                                            slot_map, max_new, lengths_out, n_free_out, device_status,
                                            static_cast<cudaStream_t>(stream)));
}

rkv_status rkv_blocks_release(const rkv_blocks_config* cfg, const int32_t* lengths, const int32_t* ended,
                              const int32_t* block_table, int32_t* free_list, const int32_t* n_free,
                              int32_t* lengths_out, int32_t* n_free_out, int32_t* device_status, void* stream)
{
    const ApiRange range("rkv_blocks_release");
    if (!cfg)
        return RKV_ERR_INVALID_ARG;
    rkv_status s = check_blocks(cfg->batch, cfg->max_blocks, cfg->block_size, cfg->n_blocks);
    if (s != RKV_OK)
        return s;
    if (!ints_ok(lengths) || !ints_ok(ended) || !ints_ok(block_table) || !ints_ok(free_list) || !ints_ok(n_free) ||
        !ints_ok(lengths_out) || !ints_ok(n_free_out) || !ints_ok(device_status))
        return RKV_ERR_INVALID_ARG;
    int sms = 0;
    s = device_sms(&sms);
    if (s != RKV_OK)
        return s;
    return cuda_status(launch_blocks_release(*cfg, lengths, ended, block_table, free_list, n_free, lengths_out,
                                             n_free_out, device_status, static_cast<cudaStream_t>(stream)));
}

rkv_status rkv_kv8_store(const rkv_kv8_cache* cache, const void* K_new, const void* V_new, int64_t row_stride,
                         int64_t head_stride, const int32_t* slot_map, int64_t n_rows, void* stream)
{
    const ApiRange range("rkv_kv8_store");
    rkv_status s = check_kv8_buffers(cache);
    if (s != RKV_OK)
        return s;
    if (n_rows < 0 || !stride_ok(row_stride, 8) || !stride_ok(head_stride, 8))
        return RKV_ERR_INVALID_ARG;
    if (n_rows == 0)
        return RKV_OK;
    if (!K_new || !V_new || !aligned(K_new, 16) || !aligned(V_new, 16) || !ints_ok(slot_map))
        return RKV_ERR_INVALID_ARG;
    if (n_rows > INT32_MAX / cache->n_kv_heads)
        return RKV_ERR_UNSUPPORTED;
    int sms = 0;
    s = device_sms(&sms);
    if (s != RKV_OK)
        return s;
    return cuda_status(launch_kv8_store(*cache, K_new, V_new, row_stride, head_stride, slot_map, n_rows, sms,
                                        static_cast<cudaStream_t>(stream)));
}

rkv_status rkv_kv8_workspace(const rkv_kv8_cache* cache, uint64_t* bytes)
{
    const rkv_status s = check_kv8(cache);
    if (s != RKV_OK)
        return s;
    if (!bytes)
        return RKV_ERR_INVALID_ARG;
    *bytes = align_up(kv8_decode_ws_bytes(*cache, kMaxSms), 256);
    return RKV_OK;
}

rkv_status rkv_kv8_decode_attn(const rkv_kv8_cache* cache, const void* q, const int32_t* block_table,
                               const int32_t* lengths, void* out, void* workspace, uint64_t workspace_bytes,
                               void* stream)
{
    const ApiRange range("rkv_kv8_decode_attn");
    rkv_status s = check_kv8_buffers(cache);
    if (s != RKV_OK)
        return s;
    if (!q || !out || !workspace || !aligned(q, 16) || !aligned(out, 16) || !aligned(workspace, 256) ||
        !ints_ok(block_table) || !ints_ok(lengths))
        return RKV_ERR_INVALID_ARG;
    if (workspace_bytes < align_up(kv8_decode_ws_bytes(*cache, kMaxSms), 256))
        return RKV_ERR_WORKSPACE;
    int sms = 0;
    s = device_sms(&sms);
    if (s != RKV_OK)
        return s;
    return cuda_status(launch_kv8_decode(*cache, q, block_table, lengths, out, workspace,
                                         sms < kMaxSms ? sms : kMaxSms, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
