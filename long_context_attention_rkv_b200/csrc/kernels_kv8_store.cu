// Writer of the 8-bit block cache: rows of K and V into blocks with one scale per (block, head).
//
// For a run of n consecutive rows that one call puts into a block from row `off` of it:
//   a = max |x| of the run,  need = max(fl32(a * fl32(1 / qmax)), 2^-64) (0 if a = 0)
//   off = 0: s' = need.  off > 0: s' = s 2^m, m >= 0 the smallest with s 2^m >= need; the rows before
//   off become round(c 2^-m)
//   new codes = round(fl32(x / s'))
// Growing the scale by powers of two bounds what repeated growth costs: the roundings of an old row are
// at most s'/2 + s'/4 + ... < s', however many tokens the block receives one by one.
//
// Bound by HBM: 2 bytes read and 1 written per element.  One CTA does the K or the V side of the runs
// that start in one window of packed rows, for one head; it holds a run (at most 128 rows) in registers
// between the maximum and the codes, so the rows are read once.  A window is one block's worth of rows
// for prompts (then it holds about one run) and a single row for decode steps (every row is a run of
// its own and all of them go side by side).
#include <cfloat>

#include "kv8_common.cuh"
#include "launchers.h"

namespace rkv {

namespace {

using namespace kv8;

constexpr int kThreads = 256;
constexpr int kMaxBlock = 128;

struct StoreArgs {
    int32_t Hkv, block, n_blocks, window;
    int64_t row_stride, head_stride, n_rows;
    const uint16_t* x[2];
    uint8_t* codes[2];
    float* scale[2];
    const int32_t* slots;
    int32_t* err;
};

template <bool kF16>
__device__ __forceinline__ void widen(const uint4& v, float (&f)[8])
{
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (kF16) {
            const float2 p = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
            f[2 * i] = p.x;
            f[2 * i + 1] = p.y;
        } else {
            f[2 * i] = bf16_bits_to_f32(w[i] & 0xffffu);
            f[2 * i + 1] = bf16_bits_to_f32(w[i] >> 16);
        }
    }
}

// Largest bit pattern of |x| over the CTA (non-negative floats order as their bits).
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red)
{
    v = __reduce_max_sync(0xffffffffu, v);
    __syncthreads();   // the previous round's values have been read
    if ((threadIdx.x & 31) == 0)
        red[threadIdx.x >> 5] = v;
    __syncthreads();
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w)
        m = max(m, red[w]);
    return m;
}

template <int D, bool kE4M3, bool kF16>
__global__ void __launch_bounds__(kThreads) kv8_store_kernel(const StoreArgs a)
{
    constexpr int kCols = D / 8;                                   // 16-byte pieces of an input row
    constexpr int kPieces = kMaxBlock * kCols / kThreads;          // per thread, for a run of 128 rows
    __shared__ int sl[kThreads + 1];                               // slots of the rows from w0 - 1 on
    __shared__ uint32_t starts[kThreads / 32], goes_on[kThreads / 32];
    __shared__ uint32_t red[kThreads / 32];

    const int tid = threadIdx.x, side = blockIdx.y;
    const int h = blockIdx.x % a.Hkv;
    const int64_t w0 = static_cast<int64_t>(blockIdx.x / a.Hkv) * a.window;
    const int mask = a.block - 1;
    const int64_t pool = static_cast<int64_t>(a.n_blocks) * a.block;

    // ---- the runs that start in this window
    bool corrupt = false;
    for (int i = tid; i <= a.window + a.block; i += kThreads) {
        const int64_t r = w0 - 1 + i;
        int v = (r >= 0 && r < a.n_rows) ? a.slots[r] : -1;
        if (v >= pool) {
            corrupt = true;
            v = -1;
        }
        if (i <= kThreads)
            sl[i] = v < 0 ? -2 : v;   // -2: no row follows it as its next slot
    }
    if (corrupt)
        report(a.err, RKV_ERR_CORRUPT);
    __syncthreads();
    const bool near = tid < a.window + a.block;
    const bool on = near && sl[tid + 1] > 0 && sl[tid + 1] == sl[tid] + 1 && (sl[tid + 1] & mask) != 0;
    const bool start = tid < a.window && sl[tid + 1] >= 0 && !on;
    const uint32_t on_word = __ballot_sync(0xffffffffu, on), start_word = __ballot_sync(0xffffffffu, start);
    if ((tid & 31) == 0) {
        goes_on[tid >> 5] = on_word;
        starts[tid >> 5] = start_word;
    }
    __syncthreads();

    const uint16_t* x = a.x[side] + h * a.head_stride;
    for (int word = 0; word * 32 < a.window; ++word) {
        for (uint32_t left = starts[word]; left; left &= left - 1) {
            const int i = word * 32 + __ffs(left) - 1;
            int n = 1;
            while (i + n < kThreads && (goes_on[(i + n) >> 5] >> ((i + n) & 31) & 1u))
                ++n;
            const int slot = sl[i + 1], blk = slot / a.block, off = slot & mask;
            const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + h;
            uint8_t* codes = a.codes[side] + unit * a.block * D;
            float* scale = a.scale[side] + unit;

            // ---- the rows, and the largest |x|
            uint4 v[kPieces];
            uint32_t top = 0;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int p = tid + j * kThreads;
                v[j] = make_uint4(0, 0, 0, 0);
                if (p < n * kCols) {
                    const int64_t row = w0 + i + p / kCols;
                    v[j] = *reinterpret_cast<const uint4*>(x + row * a.row_stride + (p % kCols) * 8);
                }
            }
            float was = off ? *scale : 0.0f;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                if (j * kThreads < n * kCols) {
                    float f[8];
                    widen<kF16>(v[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e)
                        top = max(top, __float_as_uint(f[e]) & 0x7fffffffu);
                }
            }
            top = block_max(top, red);
            if (top >= 0x7f800000u) {
                // an infinity or a NaN: the maximum again over the finite values, NaN becomes 0
                top = 0;
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    float f[8];
                    widen<kF16>(v[j], f);
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const uint32_t b = __float_as_uint(f[e]) & 0x7fffffffu;
                        top = max(top, b < 0x7f800000u ? b : 0u);
                        if (b > 0x7f800000u) {
                            uint32_t* w = e < 2 ? &v[j].x : e < 4 ? &v[j].y : e < 6 ? &v[j].z : &v[j].w;
                            *w &= (e & 1) ? 0x0000ffffu : 0xffff0000u;
                        }
                    }
                }
                top = block_max(top, red);
                if (tid == 0)
                    report(a.err, RKV_ERR_INVALID_ARG);
            }

            // ---- the block's scale
            if (!(was >= 0.0f && was <= FLT_MAX)) {
                was = 0.0f;
                if (tid == 0)
                    report(a.err, RKV_ERR_CORRUPT);
            }
            const float amax = __uint_as_float(top);
            const float need = amax > 0.0f ? fmaxf(__fmul_rn(amax, 1.0f / qmax<kE4M3>()), kMinScale) : 0.0f;
            float s = need;
            int up = 0;
            if (was > 0.0f) {
                if (need > was) {
                    int e_was, e_need;
                    const float m_was = frexpf(was, &e_was), m_need = frexpf(need, &e_need);
                    up = e_need - e_was + (m_need > m_was ? 1 : 0);
                }
                s = ldexpf(was, up);
            }
            if (up > 0) {
                // rows already in the block, at the larger scale
                const float down = ldexpf(1.0f, -up);
                for (int p = tid; p < off * (D / 16); p += kThreads) {
                    uint4 c = reinterpret_cast<const uint4*>(codes)[p];
                    uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        uint32_t o = 0;
#pragma unroll
                        for (int b = 0; b < 4; ++b)
                            o |= encode<kE4M3>(decode<kE4M3>((w[k] >> (8 * b)) & 0xffu) * down) << (8 * b);
                        w[k] = o;
                    }
                    reinterpret_cast<uint4*>(codes)[p] = make_uint4(w[0], w[1], w[2], w[3]);
                }
            }
            if (tid == 0)
                *scale = s;

            // ---- the new codes
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const int p = tid + j * kThreads;
                if (p < n * kCols) {
                    float f[8];
                    widen<kF16>(v[j], f);
                    uint32_t o[2] = {0, 0};
#pragma unroll
                    for (int e = 0; e < 8; ++e) {
                        const float t = s > 0.0f ? __fdiv_rn(f[e], s) : 0.0f;
                        o[e >> 2] |= encode<kE4M3>(t) << (8 * (e & 3));
                    }
                    *reinterpret_cast<uint2*>(codes + (off + p / kCols) * D + (p % kCols) * 8) = make_uint2(o[0], o[1]);
                }
            }
        }
    }
}

template <int D, bool kE4M3>
cudaError_t launch_t(const StoreArgs& a, bool f16, dim3 grid, cudaStream_t st)
{
    if (f16)
        kv8_store_kernel<D, kE4M3, true><<<grid, kThreads, 0, st>>>(a);
    else
        kv8_store_kernel<D, kE4M3, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_kv8_store(const rkv_kv8_cache& c, const void* K_new, const void* V_new, int64_t row_stride,
                             int64_t head_stride, const int32_t* slots, int64_t n_rows, cudaStream_t st)
{
    StoreArgs a;
    a.Hkv = c.n_kv_heads;
    a.block = c.block_size;
    a.n_blocks = c.n_blocks;
    // up to a few rows per request (a decode step): every row a window, so that no CTA does several
    // runs one after the other; otherwise about one run per window
    a.window = n_rows <= 4ll * c.batch ? 1 : c.block_size;
    a.row_stride = row_stride;
    a.head_stride = head_stride;
    a.n_rows = n_rows;
    a.x[0] = static_cast<const uint16_t*>(K_new);
    a.x[1] = static_cast<const uint16_t*>(V_new);
    a.codes[0] = c.codes_K;
    a.codes[1] = c.codes_V;
    a.scale[0] = c.scale_K;
    a.scale[1] = c.scale_V;
    a.slots = slots;
    a.err = c.device_status;
    const int64_t windows = (n_rows + a.window - 1) / a.window;
    const dim3 grid(static_cast<unsigned>(windows * c.n_kv_heads), 2);
    const bool f16 = c.in_dtype == RKV_DTYPE_F16, e4m3 = c.code_type == RKV_KV8_E4M3;
    if (c.head_dim == 128)
        return e4m3 ? launch_t<128, true>(a, f16, grid, st) : launch_t<128, false>(a, f16, grid, st);
    return e4m3 ? launch_t<64, true>(a, f16, grid, st) : launch_t<64, false>(a, f16, grid, st);
}

}  // namespace rkv
