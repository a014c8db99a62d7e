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
// 2 bytes read and 1 written per element; 28616 tokens x 8 heads x 128 take 39.7 us (4.4 TB/s; both code types, values with a
// few large channels), of which the conversion adds 13 to the 27 that moving the bytes takes: the kernel is bound by
// instruction issue (72 to 75 % of its slots).  Either type executes 16.8 instructions per value, 46 % of them on the
// integer pipe (67 to 69 % busy): two conversions, or two fused multiply-adds and the gathering of their low bytes, the
// comparison of the two results, the maximum and the widening.
// One CTA does the K or the V side of the runs
// that start in one window of packed rows, for one head; it holds a run (at most one block of rows) in
// registers between the maximum and the codes, so the rows are read once.  A window is about one run long (window_of
// below): one block's worth of rows for prompts, a single row for decode steps, so that all runs go side by side.  The CTA has block * head_dim / 64 threads, so that each holds
// eight 16-byte pieces of a full block: small CTAs, many of them per SM, keep loads in flight while others
// reduce and convert.
//
// The code is that of the correctly rounded quotient x / s.  x * r with r = fl(1 / s) is within 2^-22 (relative) of
// it, so x * r (1 - 2^-21) and x * r (1 + 2^-21) enclose it; rounding to codes is monotone, so where both give the
// same code that is the quotient's.  The division is done only where they differ.
#include <cfloat>

#include "kv8_common.cuh"
#include "launchers.h"

namespace rkv {

namespace {

using namespace kv8;

constexpr int kMaxBlock = 128;

struct StoreArgs {
    int32_t Hkv, shift, n_blocks, window;
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
template <int kThreads>
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* red)
{
    v = __reduce_max_sync(0xffffffffu, v);
    if constexpr (kThreads == 32) {
        __syncwarp();
        return v;
    }
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

__device__ __forceinline__ uint64_t pair(float x, float y)
{
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
    return r;
}

__device__ __forceinline__ void unpair(uint64_t v, float& x, float& y)
{
    asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(v));
}

__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint32_t e4m3_pair(uint64_t v)
{
    float x, y;
    unpair(v, x, y);
    return __nv_cvt_float2_to_fp8x2(make_float2(x, y), __NV_SATFINITE, __NV_E4M3);
}

// Eight int8 codes by division, kept out of line: 1 piece in 1300 where a few channels are large (2 % of the warps see one).  Of
// plain normal values 1 in 40, most of them in blocks whose largest value is 254 times a power of two (x / s is then half an odd
// number for every odd significand): 28616 tokens x 8 heads x 128 of those take 47.8 us, in e4m3 39.5 us.
__device__ __noinline__ uint2 divide8(float4 a, float4 b, float s)
{
    const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    uint32_t o[2] = {0, 0};
#pragma unroll
    for (int e = 0; e < 8; ++e)
        o[e >> 2] |= encode<false>(__fdiv_rn(x[e], s)) << (8 * (e & 3));
    return make_uint2(o[0], o[1]);
}

// Eight codes of x / s; lo, hi: pairs of the factors that enclose 1 / s.  open: nonzero bytes where they leave the code
// open (int8: all eight if one of them is).
template <bool kE4M3>
__device__ __forceinline__ uint2 quantise8(const float (&x)[8], uint64_t lo, uint64_t hi, uint2& open)
{
    uint32_t o[2];
    if constexpr (kE4M3) {
        uint32_t p[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint64_t a = pair(x[4 * i], x[4 * i + 1]), b = pair(x[4 * i + 2], x[4 * i + 3]);
            o[i] = e4m3_pair(mul2(a, lo)) | (e4m3_pair(mul2(b, lo)) << 16);
            p[i] = e4m3_pair(mul2(a, hi)) | (e4m3_pair(mul2(b, hi)) << 16);
        }
        open = make_uint2(o[0] ^ p[0], o[1] ^ p[1]);
    } else {
        // x * f + 1.5 2^23, rounded once, holds rint(x * f) in its low bits
        const uint64_t magic = pair(12582912.0f, 12582912.0f);
        uint32_t u[8];
        uint64_t differ = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint64_t a = pair(x[2 * i], x[2 * i + 1]);
            const uint64_t l = fma2(a, lo, magic);
            differ |= l ^ fma2(a, hi, magic);
            u[2 * i] = static_cast<uint32_t>(l);
            u[2 * i + 1] = static_cast<uint32_t>(l >> 32);
        }
        open.x = open.y = differ != 0 ? ~0u : 0u;
#pragma unroll
        for (int i = 0; i < 2; ++i)
            o[i] = __byte_perm(__byte_perm(u[4 * i], u[4 * i + 1], 0x0040), __byte_perm(u[4 * i + 2], u[4 * i + 3], 0x0040),
                               0x5410);
    }
    return make_uint2(o[0], o[1]);
}

// e4m3: the codes of the open bytes by division, one by one; v: the values as 16-bit words, the first in the low half of
// v.x.  Quotients of two 8-bit significands times 448 = 7 * 64 lie on a border of 4-bit codes often (one value in a
// few hundred, so most warps see one): dividing whole pieces costs 28616 tokens x 8 heads x 128 4 us more.
template <bool kF16>
__device__ __forceinline__ void settle(const uint4& v, float s, uint2& o, uint2 open)
{
    while (open.x | open.y) {
        const bool up = open.x == 0;
        const int shift = (__ffs(up ? open.y : open.x) - 1) & ~7;
        const uint32_t word = up ? (shift < 16 ? v.z : v.w) : (shift < 16 ? v.x : v.y);
        const uint32_t half = shift & 8 ? word >> 16 : word & 0xffffu;
        float x;
        if constexpr (kF16)
            x = __half2float(__ushort_as_half(static_cast<unsigned short>(half)));
        else
            x = bf16_bits_to_f32(half);
        const uint32_t code = encode<true>(__fdiv_rn(x, s)) << shift, keep = ~(0xffu << shift);
        if (up) {
            o.y = (o.y & keep) | code;
            open.y &= keep;
        } else {
            o.x = (o.x & keep) | code;
            open.x &= keep;
        }
    }
}

// A word of two 16-bit values: the largest finite magnitude, NaN turned into 0.
__device__ __forceinline__ void clean(uint32_t& w, uint32_t& top, uint32_t inf)
{
    const uint32_t lo = w & 0x7fffu, hi = (w >> 16) & 0x7fffu;
    top = max(top, max(lo < inf ? lo : 0u, hi < inf ? hi : 0u));
    w = (lo > inf ? 0u : w & 0xffffu) | (hi > inf ? 0u : w & 0xffff0000u);
}

// Smallest m >= 0 with was * 2^m >= need; 0 < was < need, both normal.
__device__ __forceinline__ int doublings(float was, float need)
{
    const uint32_t w = __float_as_uint(was), n = __float_as_uint(need);
    return static_cast<int>(n >> 23) - static_cast<int>(w >> 23) + ((n & 0x7fffffu) > (w & 0x7fffffu) ? 1 : 0);
}

// 2^e for e in [-126, 127]; 0 below.
__device__ __forceinline__ float pow2(int e) { return e < -126 ? 0.0f : __uint_as_float(static_cast<uint32_t>(e + 127) << 23); }

template <int D, int kThreads, bool kE4M3, bool kF16>
__global__ void __launch_bounds__(kThreads, 1024 / kThreads) kv8_store_kernel(const StoreArgs a)
{
    constexpr int kCols = D / 8;                                   // 16-byte pieces of an input row
    constexpr int kPieces = 8;                                     // per thread, for a full block
    constexpr int kSlots = 2 * kMaxBlock;
    __shared__ int sl[kSlots + 1];                                 // slots of the rows from w0 - 1 on
    __shared__ uint32_t starts[kSlots / 32], goes_on[kSlots / 32];
    __shared__ uint32_t red[kThreads / 32];

    const int tid = threadIdx.x, side = blockIdx.y;
    const int h = blockIdx.x % a.Hkv;
    const int64_t w0 = static_cast<int64_t>(blockIdx.x / a.Hkv) * a.window;
    const int mask = (1 << a.shift) - 1, near = a.window + mask + 1;
    const int64_t pool = static_cast<int64_t>(a.n_blocks) << a.shift;

    const uint16_t* x = (side ? a.x[1] : a.x[0]) + h * a.head_stride;

    // ---- the runs that start in this window
    bool corrupt = false;
    for (int i = tid; i <= near; i += kThreads) {
        const int64_t r = w0 - 1 + i;
        int v = (r >= 0 && r < a.n_rows) ? a.slots[r] : -1;
        if (v >= pool) {
            corrupt = true;
            v = -1;
        }
        sl[i] = v < 0 ? -2 : v;   // -2: no row follows it as its next slot
    }
    if (corrupt)
        report(a.err, RKV_ERR_CORRUPT);
    __syncthreads();
    for (int i = tid; i < ((near + 31) & ~31); i += kThreads) {
        const int v = i < near ? sl[i + 1] : -2;
        const bool on = v > 0 && v == sl[i] + 1 && (v & mask) != 0;
        const uint32_t on_word = __ballot_sync(0xffffffffu, on);
        const uint32_t start_word = __ballot_sync(0xffffffffu, i < a.window && v >= 0 && !on);
        if ((tid & 31) == 0) {
            goes_on[i >> 5] = on_word;
            starts[i >> 5] = start_word;
        }
    }
    __syncthreads();

    for (int word = 0; word * 32 < a.window; ++word) {
        for (uint32_t left = starts[word]; left; left &= left - 1) {
            const int i = word * 32 + __ffs(left) - 1;
            int n = 1;
            for (int k = i + 1; k < near;) {
                const uint32_t stop = ~goes_on[k >> 5] >> (k & 31);
                const int ones = stop ? __ffs(stop) - 1 : 32 - (k & 31);
                n += ones;
                k += ones;
                if (stop)
                    break;
            }
            n = min(n, mask + 1);
            const int slot = sl[i + 1], blk = slot >> a.shift, off = slot & mask;
            const int64_t unit = static_cast<int64_t>(blk) * a.Hkv + h;
            uint8_t* codes = (side ? a.codes[1] : a.codes[0]) + (unit << a.shift) * D;
            float* scale = (side ? a.scale[1] : a.scale[0]) + unit;

            // ---- the rows, and the largest |x|
            uint4 v[kPieces];
            const uint16_t* src = x + (w0 + i + tid / kCols) * a.row_stride + (tid % kCols) * 8;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                v[j] = make_uint4(0, 0, 0, 0);
                if (tid + j * kThreads < n * kCols)
                    v[j] = __ldcs(reinterpret_cast<const uint4*>(src + j * (kThreads / kCols) * a.row_stride));
            }
            float was = off ? *scale : 0.0f;
            uint32_t top = 0;                                      // 16-bit magnitudes order as integers
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                const uint32_t m = __vmaxu2(__vmaxu2(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu),
                                            __vmaxu2(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu));
                top = __vmaxu2(top, m);
            }
            top = block_max<kThreads>(max(top & 0xffffu, top >> 16), red);
            constexpr uint32_t kInf = kF16 ? 0x7c00u : 0x7f80u;
            bool exact = false;
            if (top >= kInf) {
                // an infinity or a NaN: the maximum again over the finite values; NaN becomes 0
                top = 0;
#pragma unroll
                for (int j = 0; j < kPieces; ++j) {
                    clean(v[j].x, top, kInf);
                    clean(v[j].y, top, kInf);
                    clean(v[j].z, top, kInf);
                    clean(v[j].w, top, kInf);
                }
                top = block_max<kThreads>(top, red);
                exact = true;
                if (tid == 0)
                    report(a.err, RKV_ERR_INVALID_ARG);
            }

            // ---- the block's scale
            if (!(was == 0.0f || (was >= FLT_MIN && was <= FLT_MAX))) {
                was = 0.0f;
                if (tid == 0)
                    report(a.err, RKV_ERR_CORRUPT);
            }
            const float amax = kF16 ? __half2float(__ushort_as_half(static_cast<unsigned short>(top)))
                                    : bf16_bits_to_f32(top);
            const float need = amax > 0.0f ? fmaxf(__fmul_rn(amax, 1.0f / qmax<kE4M3>()), kMinScale) : 0.0f;
            const int up = was > 0.0f && need > was ? doublings(was, need) : 0;
            float s = was > 0.0f ? was : need;
            if (up > 0) {
                s = __uint_as_float(__float_as_uint(was) + (static_cast<uint32_t>(up) << 23));
                // rows already in the block, at the larger scale
                const float down = pow2(-up);
                for (int p = tid; p < off * (D / 16); p += kThreads) {
                    const uint4 c = reinterpret_cast<const uint4*>(codes)[p];
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
            const float r = s > 0.0f ? __frcp_rn(s) : 0.0f;
            const float r_lo = __fmul_rn(r, 1.0f - 0x1p-21f), r_hi = __fmul_rn(r, 1.0f + 0x1p-21f);
            const uint64_t lo = pair(r_lo, r_lo), hi = pair(r_hi, r_hi);
            exact |= s < kMinScale;
            uint8_t* dst = codes + (off + tid / kCols) * D + (tid % kCols) * 8;
#pragma unroll
            for (int j = 0; j < kPieces; ++j) {
                if (tid + j * kThreads < n * kCols) {
                    float f[8];
                    widen<kF16>(v[j], f);
                    uint2 open, o = quantise8<kE4M3>(f, lo, hi, open);
                    if (exact)
                        open = make_uint2(~0u, ~0u);
                    if (!(s > 0.0f))
                        o = open = make_uint2(0, 0);
                    if constexpr (kE4M3) {
                        settle<kF16>(v[j], s, o, open);
                    } else {
                        if (open.x)
                            o = divide8(make_float4(f[0], f[1], f[2], f[3]), make_float4(f[4], f[5], f[6], f[7]), s);
                    }
                    *reinterpret_cast<uint2*>(dst + j * (kThreads / kCols) * D) = o;
                }
            }
        }
    }
}

template <int D, int kThreads, bool kE4M3>
cudaError_t launch_n(const StoreArgs& a, bool f16, dim3 grid, cudaStream_t st)
{
    if (f16)
        kv8_store_kernel<D, kThreads, kE4M3, true><<<grid, kThreads, 0, st>>>(a);
    else
        kv8_store_kernel<D, kThreads, kE4M3, false><<<grid, kThreads, 0, st>>>(a);
    return cudaGetLastError();
}

template <int D, bool kE4M3>
cudaError_t launch_t(const StoreArgs& a, bool f16, dim3 grid, cudaStream_t st)
{
    switch ((D << a.shift) / 64) {
    case 256: return launch_n<D, 256, kE4M3>(a, f16, grid, st);
    case 128: return launch_n<D, 128, kE4M3>(a, f16, grid, st);
    case 64: return launch_n<D, 64, kE4M3>(a, f16, grid, st);
    default: return launch_n<D, 32, kE4M3>(a, f16, grid, st);
    }
}

// Rows of a window: the rows of a request where all have equally many (at most a block), as a power of two, so that a
// window has about one run: a CTA does several runs one after the other, and a CTA without a run costs its look at the
// slots.  Fewer rows where that leaves less than four of these small CTAs per SM.  8 heads x 128, blocks of 64, windows
// of 1 / 4 / 16 / 64 rows: 64 requests with 1 token each 4.6 us, in windows of 64 66 us; with 4 to 8 9.8 / 6.3 / 7.0 /
// 16.8 us; with 12 to 24 20.6 / 9.9 / 7.0 / 9.5 us; 4 with 100 to 200 10.8 / 6.0 / 4.4 / 6.7 us; 1 with 28616 411 us in
// windows of 1, 39.4 us in windows of 64.
int window_of(int64_t n_rows, const rkv_kv8_cache& c, int sms)
{
    const int64_t many_ctas = 4ll * sms;
    int w = 1;
    while (2 * w <= c.block_size && 2ll * w * c.batch <= n_rows)
        w *= 2;
    while (w > 1 && 2ll * c.n_kv_heads * ((n_rows + w - 1) / w) < many_ctas)
        w /= 2;
    return w;
}

}  // namespace

cudaError_t launch_kv8_store(const rkv_kv8_cache& c, const void* K_new, const void* V_new, int64_t row_stride,
                             int64_t head_stride, const int32_t* slots, int64_t n_rows, int sms, cudaStream_t st)
{
    StoreArgs a;
    a.Hkv = c.n_kv_heads;
    a.shift = 0;
    while ((1 << a.shift) < c.block_size)
        ++a.shift;
    a.n_blocks = c.n_blocks;
    a.window = window_of(n_rows, c, sms);
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
