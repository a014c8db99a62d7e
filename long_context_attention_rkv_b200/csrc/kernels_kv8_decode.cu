// Attention of one new token per request over the 8-bit block cache.
//
//   out_g = sum_i p_i V_i / sum_i p_i,  p_i = exp(scale q_g . K_i),  K_i = sK_blk codeK_i, V_i = sV_blk codeV_i
//
// The scales stay out of the products: with x_i = scale log2(e) sK_blk (q_g . codeK_i) the kernel keeps,
// over the tokens seen so far, M = max_i (x_i + log2 sV_blk) and
//   L = sum_i t_i,  t_i = 2^15 2^(x_i - M),  O = sum_i w_i codeV_i,  w_i = t_i sV_blk <= 2^15,
// so out = O / L.  Having the V scale in M bounds every w_i whatever the blocks' scales, so
// it can enter the second product as a binary16 number (11 significant bits, rounded to nearest: the same
// or finer than a 16-bit output); the factor 2^15 keeps the weights of a flat context of millions of tokens
// out of binary16's subnormals.  A block whose V scale is 0 counts in M with the smallest scale, 2^-64, and has w_i = 0: it
// neither lifts M over blocks of small scales nor is lost in L.  t_i lies within 2^79 and, for the largest logit,
// above 2^-106; L is scaled by 2^(M - M') in two halves, which alone can fall below fp32's range (scales of 2^-64
// beside 2^80) while the product with L does not.
// M is kept as the two terms of the token that attains it (Top below), and the logits are subtracted from one
// another before anything small is added: x_i + log2 sV_blk, or 15 - M, rounded to 32 bits would be off by 8 and more
// for logits of 2^25 and beyond, past binary16's range and with equal logits weighted by their scales.
//
// Both products run on warp-level tensor-core instructions (m16n8k16, binary16 in, fp32 out): with at most
// 8 query heads per kv-head they have a single narrow column tile, 2 x 128 x 8 multiply-adds per 256 bytes, so
// the kernel is bound by HBM and what counts is that codes go from memory to operand registers without a
// detour.  They do: the order of the channels inside a product is free, so each lane loads 16 consecutive
// bytes of a row and uses them as its operand elements (no shared memory, no shuffles):
//   S^T = K q^T   A = K, 16 tokens x 16 channels.  Lane (g, t) = (lane / 4, lane % 4) holds tokens g and g + 8;
//                 step s takes its channels 16 t + 4 s .. + 3 (s < 4; + 64 for s >= 4).
//   O^T = V^T w   A = V^T, 16 channels x 16 tokens.  Lane (g, t) holds tokens 2t, 2t+1, 2t+8, 2t+9, channels
//                 16 g .. 16 g + 15; row tile i takes channels 16 g + 2 i (rows 0-7) and 16 g + 2 i + 1 (8-15).
//                 w goes from S^T's accumulator layout to the B operand by one 8x8 transpose per 8 tokens.
// (With head_dim 64 a lane's piece is 8 bytes of V, and the K steps stop at 4.)
// int8 codes become binary16 exactly by bytes: 0x6400 | (c + 128) is 1152 + c, minus 1152.  8-bit floats
// have a conversion instruction; binary16 holds them exactly.  q is scaled by a power of two per head so that
// its largest element lies in [2^14, 2^15): every element is then exact or, if tiny, off by at most 2^-40 of
// the largest.
//
// Measured: 4 requests of 131072 tokens, 32 / 8 heads of 128: 172 us in a burst = 6.25 TB/s (0.95 of the measured copy rate), 195 us
// when thousands of calls go on and power lowers the clock; of 64 (half the bytes in flight) 120 us = 4.5 TB/s; 32 / 2 heads
// of 128 (two CTAs per SM) 80 us = 3.3 TB/s.  8 ragged requests of 16384 to 32768, 28 / 4 heads: 47.5 us; 64 of 1024, 32 / 8
// heads: 35.5 us; one of 2049: 7 us, latency.
//
// Work split: units (request, kv-head) are cut into tiles of 64 tokens; a CTA's four warps take 16 tokens of each tile, and
// at the end of a unit their states are merged.  Short rows: a cluster per unit, whose CTAs take equal ranges of its tiles
// and join through their shared memory (cluster_parts says when).  Otherwise the CTAs take equal contiguous ranges of
// all tiles, found from the lengths on the device, and what is not a whole unit is left in the workspace for the join
// kernel, which adds the parts in order.
#include <cuda_fp8.h>

#include <cfloat>
#include <cmath>

#include "kv8_common.cuh"
#include "launchers.h"

namespace rkv {

namespace {

using namespace kv8;

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kTile = 16 * kWarps;     // tokens per CTA step
constexpr int kCtasPerSm = 4;          // at 128 registers; 4 requests of 131072 tokens: 172 us, three 186 us, two 236 us
constexpr int kMaxCtas = 160 * kCtasPerSm;
constexpr float kNone = -FLT_MAX;      // logit before any token
constexpr float kZeroScale = -64.0f;   // log2 of the scale that a scale of 0 has in the maximum (kMinScale)
constexpr float kWeightExp = 15.0f;    // weights are kept times 2^15: binary16 then holds 2^-39 .. 1 of the largest

struct DecodeArgs {
    int32_t Hkv, Hq, G, batch, block_shift, n_blocks, max_blocks, out_dtype;
    float qk;                          // scale * log2(e)
    const uint16_t* q;
    const uint8_t* codes_K;
    const uint8_t* codes_V;
    const float* scale_K;
    const float* scale_V;
    const int32_t* table;
    const int32_t* lengths;
    void* out;
    float* part_o;                     // [2 * CTAs][heads][D]
    float4* part_ml;                   // [2 * CTAs][heads]: M (x, s), L, unused
    int32_t* err;
};

// Tokens of request b that are attended to (its length, clamped to what the table row can hold).
__device__ __forceinline__ int request_len(const DecodeArgs& a, int b)
{
    const int64_t cap = static_cast<int64_t>(a.max_blocks) << a.block_shift;
    return static_cast<int>(min(static_cast<int64_t>(max(a.lengths[b], 0)), cap));
}

// Tiles before each request (all its kv-heads), for the whole CTA: pre[b], b = 0 .. batch.
__device__ __forceinline__ void tile_prefix(const DecodeArgs& a, int64_t* pre)
{
    constexpr int kPer = RKV_MAX_BATCH / kThreads;   // requests per thread, neighbours
    static_assert(kPer * kThreads == RKV_MAX_BATCH, "requests divide over the threads");
    __shared__ int64_t warp_tot[kWarps];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, b0 = threadIdx.x * kPer;
    int64_t n[kPer], sum = 0;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        n[i] = b0 + i < a.batch ? static_cast<int64_t>((request_len(a, b0 + i) + kTile - 1) / kTile) * a.Hkv : 0;
        sum += n[i];
    }
    int64_t v = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t u = __shfl_up_sync(0xffffffffu, v, o);
        v += lane >= o ? u : 0;
    }
    if (lane == 31)
        warp_tot[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w)
        v += warp_tot[w];
    v -= sum;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        v += n[i];
        if (b0 + i < a.batch)
            pre[b0 + i + 1] = v;
    }
    if (threadIdx.x == 0)
        pre[0] = 0;
    __syncthreads();
}

// CTAs that work: at most one per tile, so that none of them has an empty range.
__device__ __forceinline__ int workers(int64_t total, int ctas)
{
    return static_cast<int>(min(total, static_cast<int64_t>(ctas)));
}

// CTA p of P takes tiles [first(p), first(p + 1)).
__device__ __forceinline__ int64_t first_tile(int64_t total, int p, int P) { return total * p / P; }

// The CTA whose range holds tile x.
__device__ __forceinline__ int owner_of(int64_t total, int64_t x, int P)
{
    return static_cast<int>(((x + 1) * P - 1) / total);
}

__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t v)
{
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ float ex2(float x)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// A maximum M = x + s: the logit and the log2 of the value scale of the token that attains it.
struct Top {
    float x, s;
    // log2 of M / other: the difference of logits first, so it is right whatever their size
    __device__ __forceinline__ float over(const Top& other) const { return (x - other.x) + (s - other.s); }
    __device__ __forceinline__ void raise(const Top& other)
    {
        if (other.over(*this) > 0.0f)
            *this = other;
    }
};

constexpr Top kNoTop = {kNone, 0.0f};  // before any token

// The highest of N (a power of two), in m[0] and returned.
template <int N>
__device__ __forceinline__ Top highest(Top (&m)[N])
{
#pragma unroll
    for (int d = N / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < d; ++i)
            m[i].raise(m[i + d]);
    return m[0];
}

// Four codes of a word as two binary16 pairs (bytes 0, 1 and bytes 2, 3), exact.
template <bool kE4M3>
__device__ __forceinline__ void to_half(uint32_t w, uint32_t& lo, uint32_t& hi)
{
    if constexpr (kE4M3) {
        asm("{\n\t.reg .b16 a, b;\n\tmov.b32 {a, b}, %2;\n\tcvt.rn.f16x2.e4m3x2 %0, a;\n\tcvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
            : "=r"(lo), "=r"(hi)
            : "r"(w));
    } else {
        const uint32_t u = w ^ 0x80808080u;                       // c + 128
        const uint32_t p = __byte_perm(u, 0x64646464u, 0x4140), q = __byte_perm(u, 0x64646464u, 0x4342);
        const __half2 off = __halves2half2(__ushort_as_half(0x6480), __ushort_as_half(0x6480));   // 1152
        const __half2 x = __hsub2(*reinterpret_cast<const __half2*>(&p), off);
        const __half2 y = __hsub2(*reinterpret_cast<const __half2*>(&q), off);
        lo = *reinterpret_cast<const uint32_t*>(&x);
        hi = *reinterpret_cast<const uint32_t*>(&y);
    }
}

template <int N>
struct Piece;                                   // N bytes of a code row
template <>
struct Piece<16> {
    uint4 v;
    __device__ __forceinline__ void load(const uint8_t* p) { v = __ldg(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : i == 1 ? v.y : i == 2 ? v.z : v.w; }
};
template <>
struct Piece<8> {
    uint2 v;
    __device__ __forceinline__ void load(const uint8_t* p) { v = __ldg(reinterpret_cast<const uint2*>(p)); }
    __device__ __forceinline__ void zero() { v = make_uint2(0, 0); }
    __device__ __forceinline__ uint32_t word(int i) const { return i == 0 ? v.x : v.y; }
};

// The codes of 16 tokens in one lane's registers, and their block's scales.
template <int D>
struct Codes {
    Piece<16> k[2][D / 64];      // tokens g, g + 8; 64 channels each
    Piece<D / 8> v[4];           // tokens 2t, 2t + 1, 2t + 8, 2t + 9
    float sk, sv;

    // id < 0: a block outside the pool, skipped by its logits; any block of the pool stands in for its rows
    __device__ __forceinline__ void load_k(const DecodeArgs& a, int id, int in_block, int kvh, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        const int64_t unit = static_cast<int64_t>(max(id, 0)) * a.Hkv + kvh;
        const uint8_t* p = a.codes_K + ((unit << a.block_shift) + in_block) * D;
        sk = __ldg(a.scale_K + unit);
        sv = __ldg(a.scale_V + unit);
#pragma unroll
        for (int r = 0; r < 2; ++r)
#pragma unroll
            for (int c = 0; c < D / 64; ++c)
                k[r][c].load(p + (g + 8 * r) * D + 64 * c + 16 * t);
    }

    __device__ __forceinline__ void load_v(const DecodeArgs& a, int id, int in_block, int kvh, int lane)
    {
        const int g = lane >> 2, t = lane & 3;
        const int64_t unit = static_cast<int64_t>(max(id, 0)) * a.Hkv + kvh;
        const uint8_t* p = a.codes_V + ((unit << a.block_shift) + in_block) * D;
#pragma unroll
        for (int r = 0; r < 4; ++r)
            v[r].load(p + (2 * t + (r & 1) + 8 * (r >> 1)) * D + (D / 8) * g);
    }
};

__device__ __forceinline__ void store_out(void* out, int dtype, int64_t e, float v)
{
    if (dtype == RKV_DTYPE_F32)
        static_cast<float*>(out)[e] = v;
    else if (dtype == RKV_DTYPE_F16)
        static_cast<__half*>(out)[e] = __float2half_rn(v);
    else
        static_cast<uint16_t*>(out)[e] = f32_to_bf16_bits(v);
}

// ---- clusters ----

__device__ __forceinline__ int cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return static_cast<int>(r);
}

__device__ __forceinline__ int cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return static_cast<int>(r);
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// A float, or four, of the shared memory of CTA `rank` of the cluster, at this CTA's address p.
__device__ __forceinline__ float peer_float(const float* p, int rank)
{
    uint32_t at;
    float v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(at) : "memory");
    return v;
}

__device__ __forceinline__ float4 peer_float4(const float4* p, int rank)
{
    uint32_t at;
    float4 v;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(at)
                 : "memory");
    return v;
}

constexpr int kMaxParts = 8;           // CTAs of a cluster: the largest portable one

// NT: tiles of 8 query heads (G <= 8 * NT).  kCluster: a cluster per unit, whose CTAs take equal ranges of its tiles and
// join their parts through their shared memory; otherwise equal ranges of all tiles and the workspace.
template <int D, bool kE4M3, bool kF16, int NT, bool kCluster>
__global__ void __launch_bounds__(kThreads, NT == 1 ? kCtasPerSm : 2) kv8_decode_kernel(const DecodeArgs a)
{
    constexpr int kSteps = D / 16;               // K-side products per 16 tokens; also V row tiles
    constexpr int kHeads = 8 * NT;
    __shared__ int64_t pre[kCluster ? 1 : RKV_MAX_BATCH + 1];
    __shared__ float s_part[kCluster ? kHeads * D : 1];                  // this CTA's part
    __shared__ float4 s_part_ml[kHeads], s_ml[kWarps][kHeads];           // the CTA's and the warps' M (x, s), L
    __shared__ float s_o[kWarps][kHeads][D + 4];
    __shared__ float s_qs[kHeads];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g = lane >> 2, t = lane & 3;
    const int p = blockIdx.x;
    int64_t lo = 0, range_lo = 0, hi = 1;
    bool corrupt = false;
    if constexpr (!kCluster) {
        asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
        tile_prefix(a, pre);
        const int64_t total = pre[a.batch];
        const int P = workers(total, gridDim.x);
        lo = range_lo = p < P ? first_tile(total, p, P) : 0;
        hi = p < P ? first_tile(total, p + 1, P) : 0;
        if (p == 0)
            for (int b = tid; b < a.batch; b += kThreads)
                corrupt |= a.lengths[b] != request_len(a, b);
    }

    while (lo < hi) {
        // ---- the unit and this CTA's part of it
        int b, kvh, t_lo, t_hi;
        int64_t u_lo = 0;
        if constexpr (kCluster) {
            const int unit = p / cluster_size();
            b = unit / a.Hkv;
            kvh = unit - b * a.Hkv;
        } else {
            int b0 = 0, b1 = a.batch - 1;
            while (b0 < b1) {
                const int mid = (b0 + b1 + 1) >> 1;
                if (pre[mid] <= lo)
                    b0 = mid;
                else
                    b1 = mid - 1;
            }
            b = b0;
        }
        const int len = request_len(a, b);
        const int nt = (len + kTile - 1) / kTile;
        if constexpr (kCluster) {
            t_lo = nt * cluster_rank() / cluster_size();
            t_hi = nt * (cluster_rank() + 1) / cluster_size();
            corrupt |= a.lengths[b] != len;
        } else {
            kvh = static_cast<int>((lo - pre[b]) / nt);
            u_lo = pre[b] + static_cast<int64_t>(kvh) * nt;
            t_lo = static_cast<int>(lo - u_lo);
            t_hi = static_cast<int>(min(hi, u_lo + nt) - u_lo);
        }
        const int32_t* row = a.table + static_cast<int64_t>(b) * a.max_blocks;
        const uint16_t* qu = a.q + (static_cast<int64_t>(b) * a.Hq + static_cast<int64_t>(kvh) * a.G) * D;

        // This warp's 16 tokens of each tile.  The next tile's K codes are loaded as soon as this one's are in
        // the products, its V codes likewise, and its block id a tile earlier: loads stay in flight all
        // the time without a second set of registers.
        const int tok_mask = (1 << a.block_shift) - 1;
        auto block_id = [&](int ti) {
            const int tok = ti * kTile + warp * 16;
            return tok < len && ti < t_hi ? __ldg(row + (tok >> a.block_shift)) : 0;
        };
        auto checked = [&](int id) {
            const bool bad = id < 0 || id >= a.n_blocks;
            corrupt |= bad;
            return bad ? -1 : id;
        };
        Codes<D> c;
        int id = checked(block_id(t_lo)), next_id = block_id(t_lo + 1);
        c.load_k(a, id, (t_lo * kTile + warp * 16) & tok_mask, kvh, lane);
        c.load_v(a, id, (t_lo * kTile + warp * 16) & tok_mask, kvh, lane);

        // ---- q as B operands: lane (g, t) holds head 8 n + g, the channels of its K pieces
        uint32_t qf[NT][kSteps][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            const int head = 8 * n + g;
            float f[kSteps * 4];
            float top = 0.0f;
#pragma unroll
            for (int c = 0; c < D / 32; ++c) {               // channels 64 (c / 2) + 16 t + 8 (c % 2) .. + 7
                uint4 x = make_uint4(0, 0, 0, 0);
                if (head < a.G)
                    x = __ldg(reinterpret_cast<const uint4*>(qu + head * D + 64 * (c / 2) + 16 * t + 8 * (c % 2)));
                const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                    const uint32_t u = e % 2 ? w[e / 2] >> 16 : w[e / 2] & 0xffffu;
                    float v;
                    if constexpr (kF16)
                        v = __half2float(__ushort_as_half(static_cast<unsigned short>(u)));
                    else
                        v = bf16_bits_to_f32(u);
                    f[8 * c + e] = v;
                    top = fmaxf(top, fabsf(v));
                }
            }
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
            top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
            // q times 2^(15 - e): the largest element in [2^14, 2^15)
            int e = 15;
            if (top > 0.0f && top <= FLT_MAX)
                frexpf(top, &e);
            const float down = ldexpf(1.0f, 15 - max(-100, e));
            if (warp == 0 && t == 0)
                s_qs[head] = a.qk / down;
#pragma unroll
            for (int s = 0; s < kSteps; ++s)
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const __half2 h2 = __floats2half2_rn(f[4 * s + 2 * r] * down, f[4 * s + 2 * r + 1] * down);
                    qf[n][s][r] = *reinterpret_cast<const uint32_t*>(&h2);
                }
        }
        __syncthreads();
        float qs[NT][2];                         // logit factors of heads 8 n + 2t, + 1
#pragma unroll
        for (int n = 0; n < NT; ++n) {
            qs[n][0] = s_qs[8 * n + 2 * t];
            qs[n][1] = s_qs[8 * n + 2 * t + 1];
        }

        float o[NT][kSteps][4];
        Top m[NT][2];
        float l[NT][2];
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int i = 0; i < kSteps; ++i)
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    o[n][i][x] = 0.0f;
            m[n][0] = m[n][1] = kNoTop;
            l[n][0] = l[n][1] = 0.0f;
        }

        for (int ti = t_lo; ti < t_hi; ++ti) {
            const int tok = ti * kTile + warp * 16;
            if (tok >= len)
                break;                           // warp-uniform; only the last tile
            const bool live = id >= 0;
            id = checked(next_id);
            next_id = block_id(ti + 2);
            const int next_row = (tok + kTile) & tok_mask;

            // rows of the block past the request's end may hold anything, NaN codes too; a scale of 0 makes values of 0
            const bool sv_ok = c.sv > 0.0f;
            if (tok + 16 > len || !live || !sv_ok) {
#pragma unroll
                for (int r = 0; r < 4; ++r)
                    if (!live || !sv_ok || tok + 2 * t + (r & 1) + 8 * (r >> 1) >= len)
                        c.v[r].zero();
            }

            // ---- S^T
            float sc[NT][4];
#pragma unroll
            for (int n = 0; n < NT; ++n)
                sc[n][0] = sc[n][1] = sc[n][2] = sc[n][3] = 0.0f;
#pragma unroll
            for (int s = 0; s < kSteps; ++s) {
                uint32_t af[4];
                to_half<kE4M3>(c.k[0][s >> 2].word(s & 3), af[0], af[2]);
                to_half<kE4M3>(c.k[1][s >> 2].word(s & 3), af[1], af[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(sc[n], af, qf[n][s][0], qf[n][s][1]);
            }

            // ---- weights
            const float sk = c.sk, sv = c.sv;
            c.load_k(a, id, next_row, kvh, lane);
            const bool in0 = live && tok + g < len, in1 = live && tok + g + 8 < len;
            const float lsv = sv_ok ? __log2f(sv) : kZeroScale, wsv = sv_ok ? sv : 0.0f;
            uint32_t wf[NT][2];
#pragma unroll
            for (int n = 0; n < NT; ++n) {
                float top[2];
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    const float f = qs[n][x] * sk;
                    sc[n][x] = in0 ? sc[n][x] * f : -INFINITY;
                    sc[n][2 + x] = in1 ? sc[n][2 + x] * f : -INFINITY;
                    top[x] = fmaxf(sc[n][x], sc[n][2 + x]);
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 4));
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 8));
                    top[x] = fmaxf(top[x], __shfl_xor_sync(0xffffffffu, top[x], 16));
                }
                const bool up0 = Top{top[0], lsv}.over(m[n][0]) > 0.0f, up1 = Top{top[1], lsv}.over(m[n][1]) > 0.0f;
                if (__any_sync(0xffffffffu, up0 || up1)) {
                    const Top m0 = up0 ? Top{top[0], lsv} : m[n][0], m1 = up1 ? Top{top[1], lsv} : m[n][1];
                    float r0 = ex2(0.5f * m[n][0].over(m0)), r1 = ex2(0.5f * m[n][1].over(m1));
                    l[n][0] = l[n][0] * r0 * r0;
                    l[n][1] = l[n][1] * r1 * r1;
                    r0 *= r0;
                    r1 *= r1;
#pragma unroll
                    for (int i = 0; i < kSteps; ++i) {
                        o[n][i][0] *= r0;
                        o[n][i][1] *= r1;
                        o[n][i][2] *= r0;
                        o[n][i][3] *= r1;
                    }
                    m[n][0] = m0;
                    m[n][1] = m1;
                }
                const float d0 = kWeightExp - m[n][0].s, d1 = kWeightExp - m[n][1].s;
                const float t00 = ex2((sc[n][0] - m[n][0].x) + d0), t01 = ex2((sc[n][1] - m[n][1].x) + d1);
                const float t10 = ex2((sc[n][2] - m[n][0].x) + d0), t11 = ex2((sc[n][3] - m[n][1].x) + d1);
                l[n][0] += t00 + t10;
                l[n][1] += t01 + t11;
                const __half2 p0 = __floats2half2_rn(t00 * wsv, t01 * wsv), p1 = __floats2half2_rn(t10 * wsv, t11 * wsv);
                wf[n][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p0));
                wf[n][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&p1));
            }

            // ---- O^T: bytes of tokens 2t and 2t + 1 interleaved into pairs, two row tiles per 2 channels
#pragma unroll
            for (int j = 0; j < kSteps / 2; ++j) {
                uint32_t lo4[2], hi4[2];         // channels 4j, 4j+1 and 4j+2, 4j+3 of both tokens of a pair
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    lo4[r] = __byte_perm(c.v[2 * r].word(j), c.v[2 * r + 1].word(j), 0x5140);
                    hi4[r] = __byte_perm(c.v[2 * r].word(j), c.v[2 * r + 1].word(j), 0x7362);
                }
                uint32_t af[4];
                to_half<kE4M3>(lo4[0], af[0], af[1]);
                to_half<kE4M3>(lo4[1], af[2], af[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(o[n][2 * j], af, wf[n][0], wf[n][1]);
                to_half<kE4M3>(hi4[0], af[0], af[1]);
                to_half<kE4M3>(hi4[1], af[2], af[3]);
#pragma unroll
                for (int n = 0; n < NT; ++n)
                    mma16816(o[n][2 * j + 1], af, wf[n][0], wf[n][1]);
            }
            c.load_v(a, id, next_row, kvh, lane);
        }

        // ---- merge the warps
#pragma unroll
        for (int n = 0; n < NT; ++n) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                float v = l[n][x];
                v += __shfl_xor_sync(0xffffffffu, v, 4);
                v += __shfl_xor_sync(0xffffffffu, v, 8);
                v += __shfl_xor_sync(0xffffffffu, v, 16);
                if (g == 0)
                    s_ml[warp][8 * n + 2 * t + x] = make_float4(m[n][x].x, m[n][x].s, v, 0.0f);
#pragma unroll
                for (int i = 0; i < kSteps; ++i) {
                    // rows g and g + 8 of row tile i: channels (D / 8) g + 2 i, + 1
                    s_o[warp][8 * n + 2 * t + x][(D / 8) * g + 2 * i] = o[n][i][x];
                    s_o[warp][8 * n + 2 * t + x][(D / 8) * g + 2 * i + 1] = o[n][i][2 + x];
                }
            }
        }
        __syncthreads();
        const bool whole = t_lo == 0 && t_hi == nt;
        const bool head_part = lo == range_lo && t_lo > 0;   // began in an earlier CTA
        const int64_t part = static_cast<int64_t>(2 * p + (head_part ? 0 : 1)) * a.G;
        for (int x = tid; x < a.G * D; x += kThreads) {
            const int head = x / D, ch = x % D;
            float4 ml[kWarps];
            Top m_[kWarps];
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                ml[w] = s_ml[w][head];
                m_[w] = {ml[w].x, ml[w].y};
            }
            const Top M = highest(m_);
            float L = 0.0f, O = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) {
                const float f = ex2(0.5f * Top{ml[w].x, ml[w].y}.over(M));
                L = fmaf(ml[w].z * f, f, L);
                O = fmaf(s_o[w][head][ch], f * f, O);
            }
            if constexpr (kCluster) {
                s_part[x] = O;
                if (ch == 0)
                    s_part_ml[head] = make_float4(M.x, M.s, L, 0.0f);
            } else if (whole) {
                store_out(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.Hq + kvh * a.G + head) * D + ch,
                          L != 0.0f ? O / L : 0.0f);
            } else {
                a.part_o[(part + head) * D + ch] = O;
                if (ch == 0)
                    a.part_ml[part + head] = make_float4(M.x, M.s, L, 0.0f);
            }
        }
        if constexpr (kCluster) {
            cluster_sync_all();                              // the parts of all CTAs are there
            const int parts = cluster_size();
            for (int x = cluster_rank() * kThreads + tid; x < a.G * D; x += parts * kThreads) {
                const int head = x / D, ch = x % D;
                float4 ml[kMaxParts];
                Top m_[kMaxParts];
                float o_[kMaxParts], L = 0.0f, O = 0.0f;
#pragma unroll
                for (int r = 0; r < kMaxParts; ++r) {
                    ml[r] = r < parts ? peer_float4(&s_part_ml[head], r) : make_float4(kNone, 0.0f, 0.0f, 0.0f);
                    o_[r] = r < parts ? peer_float(&s_part[x], r) : 0.0f;
                    m_[r] = {ml[r].x, ml[r].y};
                }
                const Top M = highest(m_);
#pragma unroll
                for (int r = 0; r < kMaxParts; ++r) {
                    const float f = ex2(0.5f * Top{ml[r].x, ml[r].y}.over(M));
                    L = fmaf(ml[r].z * f, f, L);
                    O = fmaf(o_[r], f * f, O);
                }
                store_out(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.Hq + kvh * a.G + head) * D + ch,
                          L != 0.0f ? O / L : 0.0f);
            }
            __syncthreads();
            cluster_sync_all();                              // no CTA leaves while others read its part
            break;
        } else {
            __syncthreads();
            lo = u_lo + t_hi;
        }
    }
    if (__any_sync(0xffffffffu, corrupt) && lane == 0)
        report(a.err, RKV_ERR_CORRUPT);
}

// Joins the parts of a unit that more than one CTA worked on, in a fixed order; zeros for empty requests.  One CTA
// per query head: the parts' factors first (all their maxima at once), then the weighted sum with a warp per part.
template <int D>
__global__ void __launch_bounds__(kThreads) kv8_join_kernel(const DecodeArgs a, int ctas)
{
    constexpr int kLanes = D / 4;                        // lanes of a row, four channels each
    constexpr int kRows = kThreads / kLanes;             // parts in flight per round
    __shared__ int64_t pre[RKV_MAX_BATCH + 1];
    __shared__ float s_f[kMaxCtas], s_l[kWarps];
    __shared__ float2 s_m[kWarps];
    __shared__ float4 s_o[kRows][kLanes];
    const int b = blockIdx.x, kvh = blockIdx.y / a.G, head = blockIdx.y % a.G, tid = threadIdx.x;
    tile_prefix(a, pre);
    const int64_t total = pre[a.batch];
    const int P = workers(total, ctas);
    const int64_t nt = (pre[b + 1] - pre[b]) / a.Hkv;
    const int64_t u_lo = pre[b] + kvh * nt, u_hi = u_lo + nt;
    const int pa = nt ? owner_of(total, u_lo, P) : 0, pb = nt ? owner_of(total, u_hi - 1, P) : -1;
    const int np = pb - pa + 1;
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (np == 1)
        return;
    // part i: the unit's first CTA left its tail slot, the others their head slots
    auto slot = [&](int i) { return (static_cast<int64_t>(2 * (pa + i)) + (i == 0 ? 1 : 0)) * a.G + head; };
    // the first parts' outputs are on their way while the factors are formed
    constexpr int kAhead = 4;
    const int row = tid / kLanes, col = tid % kLanes;
    float4 first[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const int i = row + k * kRows;
        first[k] = i < np ? __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * D) + col)
                          : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    }
    Top M = kNoTop;
    for (int i = tid; i < np; i += kThreads) {
        const float4 ml = __ldcg(&a.part_ml[slot(i)]);
        M.raise({ml.x, ml.y});
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) {
        const float x = __shfl_down_sync(0xffffffffu, M.x, d), sv = __shfl_down_sync(0xffffffffu, M.s, d);
        M.raise({x, sv});
    }
    if ((tid & 31) == 0)
        s_m[tid >> 5] = make_float2(M.x, M.s);
    __syncthreads();
    M = {s_m[0].x, s_m[0].y};
#pragma unroll
    for (int w = 1; w < kWarps; ++w)
        M.raise({s_m[w].x, s_m[w].y});
    float L = 0.0f;
    for (int i = tid; i < np; i += kThreads) {
        const float4 ml = __ldcg(&a.part_ml[slot(i)]);
        const float f = ex2(0.5f * Top{ml.x, ml.y}.over(M));
        s_f[i] = f * f;
        L = fmaf(ml.z * f, f, L);
    }
    L = warp_sum(L);
    if ((tid & 31) == 0)
        s_l[tid >> 5] = L;
    __syncthreads();
    L = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        L += s_l[w];
    float4 o = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
        const float f = row + k * kRows < np ? s_f[row + k * kRows] : 0.0f;
        o.x = fmaf(first[k].x, f, o.x);
        o.y = fmaf(first[k].y, f, o.y);
        o.z = fmaf(first[k].z, f, o.z);
        o.w = fmaf(first[k].w, f, o.w);
    }
#pragma unroll 4
    for (int i = row + kAhead * kRows; i < np; i += kRows) {
        const float4 v = __ldcg(reinterpret_cast<const float4*>(a.part_o + slot(i) * D) + col);
        const float f = s_f[i];
        o.x = fmaf(v.x, f, o.x);
        o.y = fmaf(v.y, f, o.y);
        o.z = fmaf(v.z, f, o.z);
        o.w = fmaf(v.w, f, o.w);
    }
    s_o[row][col] = o;
    __syncthreads();
    if (tid < D) {
        float v = 0.0f;
#pragma unroll
        for (int r = 0; r < kRows; ++r)
            v += reinterpret_cast<const float*>(s_o[r])[tid];
        store_out(a.out, a.out_dtype, (static_cast<int64_t>(b) * a.Hq + kvh * a.G + head) * D + tid,
                  L != 0.0f ? v / L : 0.0f);
    }
}

template <int D, bool kE4M3, bool kF16, int NT>
cudaError_t launch_cluster(const DecodeArgs& a, int parts, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch * a.Hkv * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_decode_kernel<D, kE4M3, kF16, NT, true>, a);
}

template <int D, bool kE4M3, bool kF16>
cudaError_t launch_t(const DecodeArgs& a, int ctas, int parts, cudaStream_t st)
{
    if (parts > 0)
        return a.G <= 8 ? launch_cluster<D, kE4M3, kF16, 1>(a, parts, st) : launch_cluster<D, kE4M3, kF16, 2>(a, parts, st);
    if (a.G <= 8)
        kv8_decode_kernel<D, kE4M3, kF16, 1, false><<<ctas, kThreads, 0, st>>>(a);
    else
        kv8_decode_kernel<D, kE4M3, kF16, 2, false><<<ctas, kThreads, 0, st>>>(a);
    cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(a.batch, a.Hq);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kv8_join_kernel<D>, a, ctas);
}

template <int D>
cudaError_t launch_d(const DecodeArgs& a, bool e4m3, bool f16, int ctas, int parts, cudaStream_t st)
{
    if (e4m3)
        return f16 ? launch_t<D, true, true>(a, ctas, parts, st) : launch_t<D, true, false>(a, ctas, parts, st);
    return f16 ? launch_t<D, false, true>(a, ctas, parts, st) : launch_t<D, false, false>(a, ctas, parts, st);
}

// CTAs of a cluster per unit, 0 for the form with the workspace and the join kernel.  What the host knows are the units and
// the tiles that a table row can hold, so a cluster is taken where its CTAs have at most 8 tiles even of a full row (one
// long request among short ones then costs little), as many CTAs as run at once.  32 / 8 heads of 128, with join kernel
// and in clusters of 1 / 2 / 4 / 8: 1 request of 512 tokens 6.4 and 9.9 / 6.8 / 5.4 / 4.8 us, of 2049 8.1 and 25 / 14.8 /
// 9.5 / 7.3, of 8192 12.4 and 82 / 43 / 24 / 14.4; 8 of 2049 14.3 and 26 / 15.2 / 11.5 / 11.6; 64 of 1024 35.9 and 32.4 /
// 35.6 / 44 / 62, of 2049 57 and 56 / 59 / 67 / 85.  It also saves the host a launch (2 us).  Rows that could hold much more take
// the other form: with rows of 32768 tokens, one request of 512 6.4 us instead of 4.8, of 2049 8.7 instead of 7.0, 8 of
// 2049 14.3 instead of 11.7.
int cluster_parts(const rkv_kv8_cache& c, int sms)
{
    constexpr int64_t kTiles = 8;
    const int64_t units = static_cast<int64_t>(c.batch) * c.n_kv_heads;
    const int64_t tiles = (static_cast<int64_t>(c.max_blocks) * c.block_size + kTile - 1) / kTile;
    const int64_t at_once = static_cast<int64_t>(sms) * (c.n_q_heads / c.n_kv_heads <= 8 ? kCtasPerSm : 2);
    int parts = 1;
    while (parts < kMaxParts && (tiles > kTiles * parts || units * 2 * parts <= at_once))
        parts *= 2;
    return tiles <= kTiles * parts && (parts == 1 || units * parts <= 2 * at_once) ? parts : 0;
}

// CTAs of a launch: what the SMs hold at once (the NT = 2 form holds two per SM), at most one per tile
// that the table could hold.
int decode_ctas(const rkv_kv8_cache& c, int sms)
{
    const int per_sm = c.n_q_heads / c.n_kv_heads <= 8 ? kCtasPerSm : 2;
    const int64_t tiles = static_cast<int64_t>(c.batch) * c.n_kv_heads *
                          ((static_cast<int64_t>(c.max_blocks) * c.block_size + kTile - 1) / kTile);
    return static_cast<int>(tiles < per_sm * sms ? tiles : per_sm * sms);
}

}  // namespace

uint64_t kv8_decode_ws_bytes(const rkv_kv8_cache& c, int sms)
{
    const uint64_t G = c.n_q_heads / c.n_kv_heads;
    return 2ull * decode_ctas(c, sms) * G * (c.head_dim * 4 + 16);
}

cudaError_t launch_kv8_decode(const rkv_kv8_cache& c, const void* q, const int32_t* table, const int32_t* lengths,
                              void* out, void* workspace, int sms, cudaStream_t st)
{
    DecodeArgs a;
    a.Hkv = c.n_kv_heads;
    a.Hq = c.n_q_heads;
    a.G = c.n_q_heads / c.n_kv_heads;
    a.batch = c.batch;
    a.block_shift = 0;
    while ((1 << a.block_shift) < c.block_size)
        ++a.block_shift;
    a.n_blocks = c.n_blocks;
    a.max_blocks = c.max_blocks;
    a.out_dtype = c.out_dtype;
    const double scale = c.scale > 0.0f ? c.scale : 1.0 / std::sqrt(static_cast<double>(c.head_dim));
    a.qk = static_cast<float>(scale * 1.4426950408889634);
    a.q = static_cast<const uint16_t*>(q);
    a.codes_K = c.codes_K;
    a.codes_V = c.codes_V;
    a.scale_K = c.scale_K;
    a.scale_V = c.scale_V;
    a.table = table;
    a.lengths = lengths;
    a.out = out;
    a.err = c.device_status;
    const bool e4m3 = c.code_type == RKV_KV8_E4M3, f16 = c.in_dtype == RKV_DTYPE_F16;
    const int ctas = decode_ctas(c, sms);
    a.part_o = static_cast<float*>(workspace);
    a.part_ml = reinterpret_cast<float4*>(a.part_o + 2ll * ctas * a.G * c.head_dim);
    const int parts = cluster_parts(c, sms);
    return c.head_dim == 128 ? launch_d<128>(a, e4m3, f16, ctas, parts, st) : launch_d<64>(a, e4m3, f16, ctas, parts, st);
}

}  // namespace rkv
