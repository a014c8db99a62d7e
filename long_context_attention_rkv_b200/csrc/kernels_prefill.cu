// Causal attention of packed prompts on the 5th-generation tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c q_i.k_j - m_i),  c = scale log2(e),  j <= L - n + i
//
// One pass over the keys in tiles of 128 with the running maximum m_i and sum of each row.  The 128 rows of a
// tile are tokens x query heads of one kv-head: row r = token r / G, head r % G, so the G heads that share K
// and V share every tile of them, and short prompts fill the rows G times better than one head would.
// S = Q K^T and O += P V are tcgen05 products (M 128, N 128, fp32 accumulators in TMEM); P goes back to TMEM in
// the input type as the A operand of the second product.  That rounding (half a step of the input type per
// weight, the sum l taken before it) is no larger than the one of a 16-bit output.
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>

#include "device_common.cuh"
#include "launchers.h"
#include "sm100_ptx.cuh"

namespace rkv {

namespace {

using namespace sm100;

constexpr int kM = 128;                 // rows of a query tile (TMEM lanes)
constexpr int kN = 128;                 // keys of a tile
constexpr int kThreads = 128;
constexpr uint32_t kTmemCols = 256;     // S (P over it): 128, O: 128
constexpr float kNone = -1e30f;         // running maximum before any key
constexpr float kLazy = 8.0f;           // the accumulator is rescaled when the maximum grows by 2^8

// Weights are kept times 2^kBias: binary16 then holds them up to 2^(8 + 7) and down to 2^-32 of the largest
// (a flat row of a million keys stays clear of its smallest step); bf16 has fp32's range.
template <bool kF16>
constexpr float kBias = kF16 ? 7.0f : 0.0f;

struct PrefillArgs {
    int32_t Hq, Hkv, G, batch, ntok, out_dtype, kv_padded;
    float c;
    int64_t q_rows, kv_rows, out_row_stride, out_head_stride;
    const int32_t* q_off;
    const int32_t* kv_off;
    const int32_t* kv_len;
    void* out;
    float* lse;
    int32_t* err;
};

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// D[tmem] (+)= A[tmem] * B[smem]^T, kind::f16.
__device__ __forceinline__ void mma_f16_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc,
                                           uint32_t accumulate)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "setp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
        : "memory");
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t (&r)[32])
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
        "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]),
        "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]),
        "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// 4-D tiled TMA load (no multicast).
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(smem_addr(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// MN-major operand in the 128-byte swizzle: 64-element blocks 16 KB apart, 8-key groups 1 KB apart.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t start)
{
    return static_cast<uint64_t>((start >> 4) & 0x3fff) | (static_cast<uint64_t>(16384 >> 4) << 16) |
           (static_cast<uint64_t>(1024 >> 4) << 32) | (static_cast<uint64_t>(1) << 46) |
           (static_cast<uint64_t>(2) << 61);
}

template <bool kF16>
__host__ __device__ constexpr uint32_t idesc_f32(int M, int N)
{
    return idesc_bf16_f32(M, N) & (kF16 ? ~((1u << 7) | (1u << 10)) : ~0u);
}

// Two values as a pair of the input type, the first in the low half.
template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float x, float y)
{
    if constexpr (kF16) {
        const __half2 h = __floats2half2_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    } else {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
        return *reinterpret_cast<const uint32_t*>(&h);
    }
}

// Rows and keys of a sequence; ok = false if they leave q or K.
struct Seq {
    int q0, n, kv0, L, plane;
    bool ok;
};

__device__ __forceinline__ Seq sequence(const PrefillArgs& a, int b)
{
    Seq s;
    s.q0 = a.q_off[b];
    const int64_t n = static_cast<int64_t>(a.q_off[b + 1]) - s.q0;
    int64_t kv0, L;
    if (a.kv_padded) {
        kv0 = a.kv_off ? a.kv_off[b] : 0;
        L = a.kv_len ? a.kv_len[b] : n;
        s.plane = b;
    } else {
        const int32_t* off = a.kv_off ? a.kv_off : a.q_off;
        kv0 = off[b];
        L = a.kv_len ? a.kv_len[b] : static_cast<int64_t>(off[b + 1]) - kv0;
        s.plane = 0;
    }
    s.ok = s.q0 >= 0 && n >= 0 && s.q0 + n <= a.q_rows && kv0 >= 0 && L >= 0 && kv0 + L <= a.kv_rows;
    s.n = s.ok ? static_cast<int>(n) : 0;
    s.L = s.ok ? static_cast<int>(L) : 0;
    s.kv0 = s.ok ? static_cast<int>(kv0) : 0;
    return s;
}

template <int D>
struct Layout {
    static constexpr uint32_t tile = 128 * D * 2;
    static constexpr uint32_t q = 0, k = tile, v = 2 * tile, bars = 3 * tile;
    static constexpr uint32_t alloc = bars + 256 + 1024;
};

struct Bars {
    uint64_t q_full, k_full, v_full, s_done, o_done, last;
    uint32_t tmem;
    int abort;
};

template <int D, bool kF16>
__global__ void __launch_bounds__(kThreads, 2)
    prefill_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                   const __grid_constant__ CUtensorMap mV, const PrefillArgs a)
{
    using L = Layout<D>;
    constexpr int kHalves = D / 64;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    Bars* bars = reinterpret_cast<Bars*>(sm + L::bars);
    __shared__ int s_seq, s_tile;
    const int tid = threadIdx.x, warp = tid >> 5;

    // ---- the item: sequences in order, their tiles from the last (the longest) to the first
    if (tid == 0) {
        int64_t left = blockIdx.x / a.Hkv;
        int b = 0, tile = -1;
        for (; b < a.batch; ++b) {
            const Seq s = sequence(a, b);
            if (!s.ok && blockIdx.x == 0)
                report(a.err, RKV_ERR_INVALID_ARG);
            const int nt = (s.n + a.ntok - 1) / a.ntok;
            if (tile < 0) {
                if (left < nt) {
                    tile = nt - 1 - static_cast<int>(left);
                    s_seq = b;
                    if (blockIdx.x != 0)
                        break;
                }
                left -= nt;
            }
        }
        s_tile = tile;
        mbar_init(&bars->q_full, 1);
        mbar_init(&bars->k_full, 1);
        mbar_init(&bars->v_full, 1);
        mbar_init(&bars->s_done, 1);
        mbar_init(&bars->o_done, 1);
        mbar_init(&bars->last, 1);
        bars->abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    if (s_tile < 0)
        return;
    if (warp == 0) {
        tmem_alloc(&bars->tmem, kTmemCols);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tm_s = bars->tmem, tm_o = tm_s + 128;
    const uint32_t lane_off = static_cast<uint32_t>(32 * warp) << 16;
    volatile int* abort = &bars->abort;

    const Seq s = sequence(a, s_seq);
    const int kvh = blockIdx.x % a.Hkv, tok0 = s_tile * a.ntok;
    const int last_tok = min(tok0 + a.ntok, s.n) - 1;
    const int64_t last_key = static_cast<int64_t>(s.L) - s.n + last_tok;
    const int n_tiles = last_key >= 0 ? static_cast<int>(last_key / kN) + 1 : 0;
    const int tok = tok0 + tid / a.G;
    const int lim = s.L - s.n + tok;              // last key that this row sees
    const uint32_t q_bytes = static_cast<uint32_t>(a.ntok * a.G * D * 2);
    constexpr uint32_t idescS = idesc_f32<kF16>(kM, kN);
    constexpr uint32_t idescO = idesc_f32<kF16>(kM, D) | (1u << 16);   // B (= V) MN-major

    if (tid == 0 && n_tiles > 0) {
        mbar_arrive_expect_tx(&bars->q_full, q_bytes);
        for (int x = 0; x < kHalves; ++x)
            tma_load_3d(sm + L::q + x * 16384, &mQ, 64 * x, kvh * a.G, s.q0 + tok0, &bars->q_full);
    }
    float m = kNone, l = 0.0f;
    bool ok = true;
    int issued = 0;
    for (int j = 0; j < n_tiles; ++j) {
        const uint32_t ph = j & 1;
        const int k0 = j * kN;
        if (tid == 0) {
            // the previous product has read K, V, S and P
            if (j > 0)
                ok = ok && mbar_wait(&bars->o_done, ph ^ 1, abort);
            if (ok) {
                mbar_arrive_expect_tx(&bars->k_full, L::tile);
                mbar_arrive_expect_tx(&bars->v_full, L::tile);
                for (int x = 0; x < kHalves; ++x)
                    tma_load_4d(sm + L::k + x * 16384, &mK, 64 * x, s.kv0 + k0, kvh, s.plane, &bars->k_full);
                for (int x = 0; x < kHalves; ++x)
                    tma_load_4d(sm + L::v + x * 16384, &mV, 64 * x, s.kv0 + k0, kvh, s.plane, &bars->v_full);
                issued = j + 1;
                if (j == 0)
                    ok = mbar_wait(&bars->q_full, 0, abort);
                ok = ok && mbar_wait(&bars->k_full, ph, abort);
                if (ok) {
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < D / 16; ++kk) {
                        const uint32_t off = (kk / 4) * 16384 + (kk % 4) * 32;
                        mma_f16(tm_s, smem_desc_sw128(smem_addr(sm + L::q) + off),
                                smem_desc_sw128(smem_addr(sm + L::k) + off), idescS, kk > 0 ? 1u : 0u);
                    }
                    mma_commit(&bars->s_done);
                }
            }
            if (!ok)
                *abort = 1;
        }
        ok = ok && mbar_wait(&bars->s_done, ph, abort);
        if (!__syncthreads_and(ok))
            break;
        tc_fence_after();
        float p[128];
#pragma unroll
        for (int x = 0; x < 4; ++x)
            tmem_ld32(tm_s + 32 * x + lane_off, *reinterpret_cast<float(*)[32]>(&p[32 * x]));
        const int cut = lim - k0;                  // columns past it are masked
        float top = kNone;
#pragma unroll
        for (int x = 0; x < 128; ++x) {
            p[x] = x <= cut ? p[x] * a.c : -INFINITY;
            top = fmaxf(top, p[x]);
        }
        // the accumulator keeps its old maximum until the new one is 2^8 larger; a warp rescales together
        float r = 1.0f;
        if (j == 0 || top > m + kLazy) {
            r = ex2(m - top);
            m = fmaxf(m, top);
            l *= r;
        }
        if (j > 0 && __any_sync(0xffffffffu, r != 1.0f)) {
#pragma unroll
            for (int x = 0; x < D / 32; ++x) {
                float o[32];
                uint32_t w[32];
                tmem_ld32(tm_o + 32 * x + lane_off, o);
#pragma unroll
                for (int i = 0; i < 32; ++i)
                    w[i] = __float_as_uint(o[i] * r);
                tmem_st32(tm_o + 32 * x + lane_off, w);
            }
        }
        float sum = 0.0f;
#pragma unroll
        for (int x = 0; x < 128; ++x) {
            p[x] = ex2(p[x] - (m - kBias<kF16>));
            sum += p[x];
        }
        l += sum;
#pragma unroll
        for (int x = 0; x < 2; ++x) {
            uint32_t w[32];
#pragma unroll
            for (int i = 0; i < 32; ++i)
                w[i] = pack2<kF16>(p[64 * x + 2 * i], p[64 * x + 2 * i + 1]);
            tmem_st32(tm_s + 32 * x + lane_off, w);
        }
        tmem_st_wait();
        if (k0 + kN > s.L) {
            // rows of V behind the sequence's keys meet weights of 0: zero them, they may hold NaN
            ok = ok && mbar_wait(&bars->v_full, ph, abort);
            if (ok && tid >= s.L - k0) {
                for (int x = 0; x < kHalves; ++x)
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<uint4*>(sm + L::v + x * 16384 + tid * 128 + i * 16) = make_uint4(0, 0, 0, 0);
            }
            fence_proxy_async_smem();
        }
        tc_fence_before();
        if (!__syncthreads_and(ok))
            break;
        if (tid == 0) {
            ok = mbar_wait(&bars->v_full, ph, abort);
            if (ok) {
                tc_fence_after();
#pragma unroll
                for (int kk = 0; kk < kN / 16; ++kk)
                    mma_f16_ts(tm_o, tm_s + 8 * kk, smem_desc_mn(smem_addr(sm + L::v) + kk * 2048), idescO,
                               (j > 0 || kk > 0) ? 1u : 0u);
                mma_commit(&bars->o_done);
            } else {
                *abort = 1;
            }
        }
    }
    if (n_tiles > 0) {
        ok = ok && mbar_wait(&bars->o_done, (n_tiles - 1) & 1, abort);
        ok = __syncthreads_and(ok);
        tc_fence_after();
    }
    if (ok) {
        const bool store = tid < a.ntok * a.G && tok < s.n;
        const int head = kvh * a.G + tid % a.G;
        const int64_t row = s.q0 + tok;
        const float inv = l > 0.0f ? 1.0f / l : 0.0f;
        if (store && a.lse)
            a.lse[row * a.Hq + head] = l > 0.0f ? (m - kBias<kF16> + log2f(l)) * 0.6931471805599453f : -INFINITY;
        const int64_t e = row * a.out_row_stride + head * a.out_head_stride;
#pragma unroll
        for (int x = 0; x < D / 32; ++x) {
            float o[32];
            if (n_tiles > 0)
                tmem_ld32(tm_o + 32 * x + lane_off, o);
#pragma unroll
            for (int i = 0; i < 32; ++i)
                o[i] = l > 0.0f ? o[i] * inv : 0.0f;
            if (!store)
                continue;
            if (a.out_dtype == RKV_DTYPE_F32) {
                float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + e + 32 * x);
#pragma unroll
                for (int i = 0; i < 8; ++i)
                    dst[i] = make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
            } else {
                uint4* dst = reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + e + 32 * x);
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    dst[i] = make_uint4(pack2<kF16>(o[8 * i], o[8 * i + 1]), pack2<kF16>(o[8 * i + 2], o[8 * i + 3]),
                                        pack2<kF16>(o[8 * i + 4], o[8 * i + 5]), pack2<kF16>(o[8 * i + 6], o[8 * i + 7]));
            }
        }
    } else if (tid == 0) {
        report(a.err, RKV_ERR_TIMEOUT);
        // copies and products in flight end (waited for with the same limit) before the CTA does
        volatile int never = 0;
        mbar_wait(&bars->q_full, 0, &never);
        if (issued > 0) {
            mbar_wait(&bars->k_full, (issued - 1) & 1, &never);
            mbar_wait(&bars->v_full, (issued - 1) & 1, &never);
        }
        mma_commit(&bars->last);
        mbar_wait(&bars->last, 0, &never);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tm_s, kTmemCols);
    }
}

using EncodeFn = PFN_cuTensorMapEncodeTiled_v12000;

EncodeFn map_encoder()
{
    static const EncodeFn fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult qr;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &qr) != cudaSuccess ||
            qr != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<EncodeFn>(f);
    }();
    return fn;
}

// 128-byte-swizzled tiles of 64 channels; dims and strides (bytes) from the second dimension on.
bool make_map(CUtensorMap* m, const void* base, bool f16, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
              const cuuint32_t* box)
{
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return map_encoder()(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank,
                         const_cast<void*>(base), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                         CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                         CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D, bool kF16>
cudaError_t launch_t(const CUtensorMap& mQ, const CUtensorMap& mK, const CUtensorMap& mV, const PrefillArgs& a,
                     int64_t items, cudaStream_t st)
{
    auto kern = prefill_kernel<D, kF16>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::alloc);
    if (e != cudaSuccess)
        return e;
    kern<<<static_cast<unsigned>(items), kThreads, Layout<D>::alloc, st>>>(mQ, mK, mV, a);
    return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prefill(const rkv_prefill_config& c, const void* q, const void* K, const void* V,
                           const int32_t* q_off, const int32_t* kv_off, const int32_t* kv_len, void* out, float* lse,
                           int32_t* err, int sms, cudaStream_t st)
{
    (void)sms;
    if (!map_encoder())
        return cudaErrorNotSupported;
    PrefillArgs a;
    a.Hq = c.n_q_heads;
    a.Hkv = c.n_kv_heads;
    a.G = c.n_q_heads / c.n_kv_heads;
    a.batch = c.batch;
    a.ntok = kM / a.G;
    a.out_dtype = c.out_dtype;
    a.kv_padded = c.kv_padded;
    const double scale = c.scale > 0.0f ? c.scale : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
    a.c = static_cast<float>(scale * 1.4426950408889634);
    a.q_rows = c.q_rows;
    a.kv_rows = c.kv_rows;
    a.out_row_stride = c.out_row_stride;
    a.out_head_stride = c.out_head_stride;
    a.q_off = q_off;
    a.kv_off = kv_off;
    a.kv_len = kv_len;
    a.out = out;
    a.lse = lse;
    a.err = err;
    const bool f16 = c.in_dtype == RKV_DTYPE_F16;
    using u64 = cuuint64_t;
    alignas(64) CUtensorMap mQ, mK, mV;
    const u64 qd[3] = {static_cast<u64>(c.head_dim), static_cast<u64>(c.n_q_heads), static_cast<u64>(c.q_rows)};
    const u64 qs[2] = {static_cast<u64>(2 * c.q_head_stride), static_cast<u64>(2 * c.q_row_stride)};
    const cuuint32_t qb[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(a.ntok)};
    if (c.kv_rows == 0)
        K = V = q;                             // no row is ever loaded through these maps
    const u64 kd[4] = {static_cast<u64>(c.head_dim), static_cast<u64>(c.kv_rows > 0 ? c.kv_rows : 1),
                       static_cast<u64>(c.n_kv_heads),
                       static_cast<u64>(c.kv_padded ? c.batch : 1)};
    const u64 ks[3] = {static_cast<u64>(2 * c.kv_row_stride), static_cast<u64>(2 * c.kv_head_stride),
                       static_cast<u64>(c.kv_padded ? 2 * c.kv_plane_stride : 2 * c.kv_row_stride)};
    const cuuint32_t kb[4] = {64, kN, 1, 1};
    if (!make_map(&mQ, q, f16, 3, qd, qs, qb) || !make_map(&mK, K, f16, 4, kd, ks, kb) ||
        !make_map(&mV, V, f16, 4, kd, ks, kb))
        return cudaErrorInvalidValue;
    // the tiles are known on the device only: at most one partial tile per sequence
    const int64_t items = (c.q_rows / a.ntok + c.batch) * c.n_kv_heads;
    if (c.head_dim == 128)
        return f16 ? launch_t<128, true>(mQ, mK, mV, a, items, st) : launch_t<128, false>(mQ, mK, mV, a, items, st);
    return f16 ? launch_t<64, true>(mQ, mK, mV, a, items, st) : launch_t<64, false>(mQ, mK, mV, a, items, st);
}

}  // namespace rkv
