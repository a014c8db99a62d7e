// Causal attention of packed prompts on the 5th-generation tensor cores.
//
//   o_i = sum_j p_ij v_j / sum_j p_ij,  p_ij = 2^(c q_i.k_j - m_i),  c = scale log2(e),  j <= L - n + i
//
// One pass over the keys in tiles of 64 with the running maximum m_i and sum of each row.  The 128 rows of a query
// tile are tokens x query heads of one kv-head: row r = token r / G, head r % G, so the G heads that share K and V
// share every tile of them, and short prompts fill the rows G times better than one head would.
// S = Q K^T and O += P V are tcgen05 products (M 128, N up to 128, fp32 accumulators in TMEM); P goes back to
// TMEM in the input type as the A operand of the second product.  That rounding (half a step of the
// input type per weight, the sum l taken before it) is no larger than the one of a 16-bit output.
//
// What bounds it: per 128 x 64 tile the two products take 640 cycles of the tensor core at head_dim 128 (S 384: with
// N 64 the reads of Q from shared memory set its pace; P V 256), the 8192 exponentials 512 cycles of the
// special-function unit, and S -> softmax -> P V is one chain of dependent steps with several hundred cycles of
// signalling in it.  So
//   - a CTA works on two query tiles of the same kv-head, each with its own S issuer and softmax warps, and K and
//     V tiles serve both (one ring in shared memory, filled by TMA);
//   - S and P have TMEM columns of their own (that is what tiles of 64 keys buy: two O of 128 columns, two S of 64 and
//     four P of 32 fill the 512): the next S is formed as soon as this one is in the softmax warps' registers, and
//     P V runs beside the next softmax, so neither product is waited for in the steady state;
//   - one thread owns one row (TMEM lane): no shuffles, and the row's maximum and sum never leave registers;
//   - the accumulator is only rescaled when a row's maximum grew by more than 2^8: rare after the first tiles, so
//     almost no step waits for the product before it.  The maximum is kept as one of S, without the factor c, so that
//     differences are exact; where c max is large the weights are formed from them too (kFar);
//   - a share of the exponentials runs on the FMA pipes (exp2_pair below).
//
// Work split: items (sequence, pair of query tiles, kv-head) from those with many keys to those with few (Schedule
// below), taken in snake order by one persistent CTA per SM.  Everything is derived from the offsets on the device, so a
// captured graph follows them.  Few items over many keys (the next tokens of a long request) are split along the
// keys: the CTAs of a cluster each take a range of an item's key tiles and join their parts through their shared memory
// (split_of says when), without a workspace.
//
// Warps: 0 TMA producer, 1 and 2 issue S of query tiles 0 and 1, 3 issues P V of both, 4-7 and 8-11 are their softmax.
//
// Measured: 8192 tokens, 32 query and 8 kv-heads of 128: 445 to 490 us in a burst of ten calls = 1235 to 1120 TFLOP/s, 510 us =
// 1080 TFLOP/s (0.78 of the sustained rate of a plain product) when calls go on and the board's power holds the clock at
// 1.58 GHz; at 1.65 GHz about 1530 cycles per 64 keys of two query tiles, 1280 of them products.  8 ragged prompts of 300
// to 2500 tokens 90 us (burst; 104 us), where the roughly 5000 cycles of an item outside its steps (first loads and S, last product,
// output) count.
//
// Every wait is bounded (2 s); one that gives up records RKV_ERR_TIMEOUT, all roles leave their loops, and copies
// and products in flight are waited for before TMEM is freed.
#include <cudaTypedefs.h>

#include <cfloat>
#include <climits>
#include <cmath>
#include <type_traits>

#include "device_common.cuh"
#include "launchers.h"
#include "sm100_ptx.cuh"

namespace rkv {

namespace {

using namespace sm100;

constexpr int kM = 128;                 // rows of a query tile (TMEM lanes)
constexpr int kN = 64;                  // keys of a tile
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;     // query tile t: S at 128 t, P (two buffers) at 128 t + 64 and + 96, O at 256 + 128 t
constexpr float kNone = -FLT_MAX;       // running maximum (of S) before any key
constexpr int kPoly = 8;                // every kPoly-th pair of exponentials goes to the FMA pipes (0: none); 8192
                                        // tokens: share 0 451 us, 6 % 445, 12 % 447, 25 % 467, 50 % 569 (issue-bound)
constexpr float kLazy = 8.0f;           // the accumulator is rescaled when the maximum grows by 2^8: sums stay far below
                                        // fp32's range, binary16 weights (times 2^kBias) below 2^16
constexpr float kFar = 65536.0f;        // maxima (in units of log 2) from which S - max is formed before the factor c: below, the
                                        // roundings of c max and of the bias' sum with it move an exponent by at most 2^-7;
                                        // from 2^24 on they would move it past binary16's range, from 2^31 past fp32's

// Weights are kept times 2^kBias: binary16 then holds them up to 2^(8 + 7) and down to 2^-32 of the largest
// (a flat row of a million keys stays clear of its smallest step); bf16 has fp32's range.
template <bool kF16>
constexpr float kBias = kF16 ? 7.0f : 0.0f;

struct PrefillArgs {
    int32_t Hq, Hkv, G, batch, ntok, out_dtype, kv_padded;
    int32_t level_keys;                 // whole prompts of at most so many tokens in all are worked on level by level
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

// The largest of three, NaN if one of them is.
__device__ __forceinline__ float max3(float a, float b, float c)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
    return r;
}

// ---- packed pairs of fp32 ---------------------------------------------------------------

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

__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c)
{
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}

__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b)
{
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// 2^x of a pair on the FMA pipes, x <= 2^6: x = n + f with n = rint(x) (taken from the low bits of x + 1.5 2^23),
// 2^f by the degree-5 polynomial of least relative error on [-1/2, 1/2] (found by the Remez exchange; 7.5e-8, with
// fp32 rounding under 2^-22), n added to the exponent field.  x is held at -127, where that leaves 0 or one of the
// smallest subnormal steps: nothing in the weight's 16 bits.
__device__ __forceinline__ void exp2_pair(uint64_t x, float& r0, float& r1)
{
    float a, b;
    unpair(x, a, b);
    x = pair(fmaxf(a, -127.0f), fmaxf(b, -127.0f));
    const uint64_t magic = pair(12582912.0f, 12582912.0f), back = pair(-12582912.0f, -12582912.0f);
    const uint64_t t = add2(x, magic);
    const uint64_t f = fma2(add2(t, back), pair(-1.0f, -1.0f), x);
    uint64_t p = pair(0.0013276471992533984f, 0.0013276471992533984f);
    p = fma2(p, f, pair(0.009675541334453752f, 0.009675541334453752f));
    p = fma2(p, f, pair(0.055507132734978495f, 0.055507132734978495f));
    p = fma2(p, f, pair(0.24022119723839974f, 0.24022119723839974f));
    p = fma2(p, f, pair(0.6931469670647609f, 0.6931469670647609f));
    p = fma2(p, f, pair(1.0000000716546849f, 1.0000000716546849f));
    float t0, t1;
    unpair(t, t0, t1);
    unpair(p, a, b);
    r0 = __uint_as_float(__float_as_uint(a) + (__float_as_uint(t0) << 23));
    r1 = __uint_as_float(__float_as_uint(b) + (__float_as_uint(t1) << 23));
}

// ---- tensor memory, TMA, descriptors -------------------------------------------------------

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

// 32 columns of this warp's TMEM lanes; the values may be used after tmem_arrived on them.
__device__ __forceinline__ void tmem_ld32_async(uint32_t taddr, float* v)
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
                 : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3]), "=f"(v[4]), "=f"(v[5]), "=f"(v[6]), "=f"(v[7]), "=f"(v[8]), "=f"(v[9]), "=f"(v[10]), "=f"(v[11]), "=f"(v[12]), "=f"(v[13]), "=f"(v[14]), "=f"(v[15]), "=f"(v[16]), "=f"(v[17]), "=f"(v[18]), "=f"(v[19]), "=f"(v[20]), "=f"(v[21]), "=f"(v[22]), "=f"(v[23]), "=f"(v[24]), "=f"(v[25]), "=f"(v[26]), "=f"(v[27]), "=f"(v[28]), "=f"(v[29]), "=f"(v[30]), "=f"(v[31])
                 : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld_wait() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

// Orders the uses of v behind the volatile wait above.
__device__ __forceinline__ void tmem_arrived(float* v)
{
    asm volatile("" : "+f"(v[0]), "+f"(v[1]), "+f"(v[2]), "+f"(v[3]), "+f"(v[4]), "+f"(v[5]), "+f"(v[6]), "+f"(v[7]), "+f"(v[8]), "+f"(v[9]), "+f"(v[10]), "+f"(v[11]), "+f"(v[12]), "+f"(v[13]), "+f"(v[14]), "+f"(v[15]), "+f"(v[16]), "+f"(v[17]), "+f"(v[18]), "+f"(v[19]), "+f"(v[20]), "+f"(v[21]), "+f"(v[22]), "+f"(v[23]), "+f"(v[24]), "+f"(v[25]), "+f"(v[26]), "+f"(v[27]), "+f"(v[28]), "+f"(v[29]), "+f"(v[30]), "+f"(v[31]));
}

__device__ __forceinline__ void tmem_st16(uint32_t taddr, const uint32_t* r)
{
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
        "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(taddr),
        "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]),
        "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
        : "memory");
}

__device__ __forceinline__ void tmem_st_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// One lane of a converged warp, in a form that the compiler knows to be a single thread.
__device__ __forceinline__ bool elect_one()
{
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
}

__device__ __forceinline__ void named_sync(int id, int n)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(n) : "memory");
}

__device__ __forceinline__ void named_arrive(int id, int n)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

// 4-D and 3-D tiled TMA loads (no multicast).
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
        : "memory");
}

__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, uint64_t* bar)
{
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
        "[%5];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(smem_addr(bar))
        : "memory");
}

// MN-major operand in the 128-byte swizzle: 64-element blocks of kN rows, 8-key groups 1 KB apart.
__device__ __forceinline__ uint64_t smem_desc_mn(uint32_t start)
{
    return static_cast<uint64_t>((start >> 4) & 0x3fff) | (static_cast<uint64_t>((kN * 128) >> 4) << 16) |
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

// ---- clusters: barriers and shared memory of the other CTAs -----------------------------------

__device__ __forceinline__ uint32_t cluster_rank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ uint32_t cluster_size()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t peer_addr(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ void arrive_at(uint64_t* bar, uint32_t rank)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(peer_addr(smem_addr(bar), rank))
                 : "memory");
}

// mbar_wait for what the threads of other CTAs wrote before they arrived.
__device__ __forceinline__ bool mbar_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort)
{
    if (!mbar_wait(bar, parity, abort))
        return false;
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.test_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_addr(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ float4 peer_float4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

__device__ __forceinline__ float2 peer_float2(uint32_t addr)
{
    float2 v;
    asm volatile("ld.shared::cluster.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
    return v;
}

// ---- work items ------------------------------------------------------------------------------

// Rows and keys of a sequence; ok = false if they leave q or K.
struct Seq {
    int q0, n, kv0, L;
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
    } else {
        const int32_t* off = a.kv_off ? a.kv_off : a.q_off;
        kv0 = off[b];
        L = a.kv_len ? a.kv_len[b] : static_cast<int64_t>(off[b + 1]) - kv0;
    }
    s.ok = s.q0 >= 0 && n >= 0 && s.q0 + n <= a.q_rows && kv0 >= 0 && L >= 0 && kv0 + L <= a.kv_rows;
    s.n = s.ok ? static_cast<int>(n) : 0;
    s.L = s.ok ? static_cast<int>(L) : 0;
    s.kv0 = s.ok ? static_cast<int>(kv0) : 0;
    return s;
}

static_assert(RKV_MAX_BATCH <= kThreads - 32, "make_schedule and the barriers' set-up use other warps");

// Pairs of query tiles in the order in which they are worked on, sequences sorted by their keys.  The order is balanced
// if the work falls from item to item.
//   - Whole prompts (L = n): the keys of a pair grow with its index from the start ("level"), so all sequences' pairs go
//     by level, the highest first: k sequences have the levels between the k-th and the (k + 1)-th one's counts of pairs.
//     8 ragged prompts of 300 to 2500 tokens (28 / 4 heads, 8.4 items per CTA): 99 us sequence by sequence, 92 us so.
//     CTAs that work on different sequences share no K and V, so only where all of it stays in L2 (level_keys: 96 MB):
//     with 92 MB 581 us and 556 us, with 720 MB 16.5 ms and 19.7 ms.
//   - Otherwise (more keys than queries: a sequence's pairs are alike, or too many of them): sequence by sequence, each
//     from its last pair to the first.
struct Schedule {
    Seq seq[RKV_MAX_BATCH];
    int key[RKV_MAX_BATCH];             // keys of sequence b, for the order
    int order[RKV_MAX_BATCH];           // sequences by their keys, most first
    int pairs[RKV_MAX_BATCH + 1];       // pairs before the i-th sequence of that order, or above the i-th one's levels
    int warp_tot[kThreads / 32], warp_keys[kThreads / 32];
    int by_level;
};

__device__ __forceinline__ int pairs_of(const PrefillArgs& a, const Seq& q) { return (q.n + 2 * a.ntok - 1) / (2 * a.ntok); }

// Sorts the sequences and counts their tile pairs (whole CTA).
__device__ __forceinline__ void make_schedule(const PrefillArgs& a, Schedule& s)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    Seq q = {};
    if (tid < a.batch) {
        q = sequence(a, tid);
        s.seq[tid] = q;
        s.key[tid] = q.L;
        if (!q.ok && blockIdx.x == 0)
            report(a.err, RKV_ERR_INVALID_ARG);
    }
    const bool whole = __syncthreads_and(q.L == q.n);
    if (tid < a.batch) {
        int rank = 0;
#pragma unroll 8
        for (int b = 0; b < a.batch; ++b)
            rank += s.key[b] > q.L || (s.key[b] == q.L && b < tid);
        s.order[rank] = tid;
    }
    __syncthreads();
    int v = tid < a.batch ? pairs_of(a, s.seq[s.order[tid]]) : 0;
    const int next = tid + 1 < a.batch ? pairs_of(a, s.seq[s.order[tid + 1]]) : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, v, o);
        v += lane >= o ? n : 0;
    }
    const int keys = __reduce_add_sync(0xffffffffu, min(q.L, 1 << 22));
    if (lane == 31) {
        s.warp_tot[warp] = v;
        s.warp_keys[warp] = keys;
    }
    __syncthreads();
    int all_keys = 0;
    for (int w = 0; w < kThreads / 32; ++w) {
        v += w < warp ? s.warp_tot[w] : 0;
        all_keys += s.warp_keys[w];
    }
    const bool by_level = whole && all_keys <= a.level_keys;
    if (tid < a.batch)
        s.pairs[tid + 1] = by_level ? v - (tid + 1) * next : v;
    if (tid == 0) {
        s.pairs[0] = 0;
        s.by_level = by_level;
    }
    __syncthreads();
}

// One item: query tiles of a pair start at tokens tok0 and tok0 + ntok; query tile t needs the key tiles 0 ..
// nk(t) - 1 (none: the tile is empty or sees no key), of the last of which it sees the first last_width(t) keys, in
// whole groups of 16 (the other tiles are seen whole by its last row).
struct Item {
    int q0, n, kv0, L, kvh, plane, tok0, ntok;
    __device__ __forceinline__ int last_key(int t) const { return L - n + min(tok0 + (t + 1) * ntok, n) - 1; }
    __device__ __forceinline__ int nk(int t) const
    {
        const int last = last_key(t);
        return tok0 + t * ntok < n && last >= 0 ? last / kN + 1 : 0;
    }
    __device__ __forceinline__ int last_width(int t) const { return ((last_key(t) % kN) + 16) & ~15; }
};

// The r-th item of worker p of P (CTAs or clusters): sequence, kv-head and pair; all ones if there is none (with the snake
// order only the last round can lack one).  Out of line: inlined into five places it costs more in instruction fetches
// (all roles run at once) than a call.
constexpr uint64_t kNoItem = ~0ull;
__device__ __noinline__ uint64_t find_item(const Schedule* sc, unsigned batch, unsigned n_kv_heads, unsigned ntok2, unsigned P,
                                           unsigned p, unsigned r)
{
    const unsigned total = static_cast<unsigned>(sc->pairs[batch]) * n_kv_heads;
    const unsigned idx = r * P + ((r & 1) ? P - 1 - p : p);
    if (idx >= total)
        return kNoItem;
    const unsigned pr = idx / n_kv_heads, kvh = idx - pr * n_kv_heads;
    unsigned lo = 0, hi = batch - 1;
    while (lo < hi) {
        const unsigned mid = (lo + hi + 1) >> 1;
        if (static_cast<unsigned>(sc->pairs[mid]) <= pr)
            lo = mid;
        else
            hi = mid - 1;
    }
    const unsigned off = pr - sc->pairs[lo], side = sc->by_level ? lo + 1 : 1, down = off / side;
    const unsigned b = sc->order[sc->by_level ? off - down * side : lo];
    const unsigned pair = (sc->seq[sc->order[lo]].n + ntok2 - 1) / ntok2 - 1 - down;
    return (static_cast<uint64_t>(kvh) << 40) | (static_cast<uint64_t>(b) << 32) | pair;
}

__device__ __forceinline__ bool get_item(const PrefillArgs& a, const Schedule& sc, unsigned P, unsigned p, int r, Item& it)
{
    const uint64_t f = find_item(&sc, a.batch, a.Hkv, 2 * a.ntok, P, p, r);
    if (f == kNoItem)
        return false;
    const int b = static_cast<int>(f >> 32) & 0xff;
    const Seq q = sc.seq[b];
    it.q0 = q.q0;
    it.n = q.n;
    it.kv0 = q.kv0;
    it.L = q.L;
    it.kvh = static_cast<int>(f >> 40);
    it.plane = a.kv_padded ? b : 0;
    it.ntok = a.ntok;
    it.tok0 = static_cast<int>(f) * 2 * a.ntok;
    return true;
}

constexpr uint32_t kMaxParts = 8;       // CTAs that share an item's keys: the largest portable cluster
constexpr int kJoinBar = 9;             // named barrier of the softmax warps (1 to 8: their turns)

// Output staging of a softmax warp: 32 rows of 64 bytes.
constexpr uint32_t kStage = 32 * 64;

template <int D>
struct Layout {
    static constexpr uint32_t qtile = kM * D * 2, tile = kN * D * 2;
    static constexpr int stages = 8;                          // K and V tiles in turn (even: K in the even slots)
    static constexpr uint32_t q = 0, kv = 2 * qtile, stage = kv + stages * tile, bars = stage + 8 * kStage;
    static constexpr uint32_t alloc = bars + 512 + 1024;
};

template <int kStages>
struct Bars {
    uint64_t q_full[2], q_empty[2], kv_full[kStages], kv_empty[kStages];
    uint64_t s_full[2], s_free[2], p_ready[2][2], pv_done[2][2], last[3];   // [query tile][P buffer]
    uint64_t part_full, part_read;   // of a cluster: every CTA's part of an item is there; every CTA has read this one's
    uint32_t tmem;
    int abort;
    int issued;                 // ring slots filled so far (producer, at its end)
    int q_issued[2];
};

template <int D, bool kF16, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    prefill_kernel(const __grid_constant__ CUtensorMap mQ, const __grid_constant__ CUtensorMap mK,
                   const __grid_constant__ CUtensorMap mV, const PrefillArgs a)
{
    using L = Layout<D>;
    constexpr int kHalves = D / 64, kStages = L::stages;
    extern __shared__ unsigned char smem_raw[];
    unsigned char* sm = smem_raw + ((1024 - (smem_addr(smem_raw) & 1023)) & 1023);
    Bars<kStages>* bars = reinterpret_cast<Bars<kStages>*>(sm + L::bars);
    static_assert(sizeof(Bars<kStages>) <= 512, "barrier block");
    __shared__ Schedule sched;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    volatile int* abort = &bars->abort;
    const uint32_t parts = kSplit ? cluster_size() : 1, part = kSplit ? cluster_rank() : 0;
    const unsigned workers = gridDim.x / parts, worker = blockIdx.x / parts;
    auto item_at = [&](int r, Item& it) { return get_item(a, sched, workers, worker, r, it); };
    // this CTA's key tiles of an item that needs n
    auto first_tile = [&](int n) { return kSplit ? static_cast<int>(n * part / parts) : 0; };
    auto end_tile = [&](int n) { return kSplit ? static_cast<int>(n * (part + 1) / parts) : n; };

    if (tid == kThreads - 1) {                                   // make_schedule leaves the last warps idle at first
        for (int t = 0; t < 2; ++t) {
            mbar_init(&bars->q_full[t], 1);
            mbar_init(&bars->q_empty[t], 1);
            mbar_init(&bars->s_full[t], 1);
            mbar_init(&bars->s_free[t], 4);
            for (int b = 0; b < 2; ++b) {
                mbar_init(&bars->p_ready[t][b], 4);
                mbar_init(&bars->pv_done[t][b], 1);
            }
            bars->q_issued[t] = 0;
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&bars->kv_full[i], 1);
            mbar_init(&bars->kv_empty[i], i % 2 == 0 ? 2 : 1);   // K: both S issuers; V: the P V issuer
        }
        mbar_init(&bars->last[0], 1);
        mbar_init(&bars->last[1], 1);
        mbar_init(&bars->last[2], 1);
        if constexpr (kSplit) {
            mbar_init(&bars->part_full, parts + 1);              // the softmax warps of every CTA, and this one's producer
            mbar_init(&bars->part_read, parts);
        }
        bars->abort = 0;
        bars->issued = 0;
        fence_mbar_init();
        prefetch_tensormap(&mQ);
        prefetch_tensormap(&mK);
        prefetch_tensormap(&mV);
    }
    if (warp == 1) {
        tmem_alloc(&bars->tmem, kTmemCols);
        tmem_relinquish();
    }
    make_schedule(a, sched);
    tc_fence_before();
    __syncthreads();
    if constexpr (kSplit)
        cluster_sync_all();                                      // the other CTAs' barriers are there
    tc_fence_after();
    const uint32_t tmem = bars->tmem;
    const uint32_t q_smem = smem_addr(sm + L::q), kv_smem = smem_addr(sm + L::kv);

    if (warp < 4) {
        Item it;
        bool ok = true;
        if (warp == 0 && lane == 0) {
            // ---------------- TMA producer
            const uint32_t q_bytes = static_cast<uint32_t>(a.ntok * a.G * D * 2);
            uint32_t slot = 0, q_use0 = 0, q_use1 = 0;
            auto load_q = [&](int t, uint32_t& use) {
                if (use > 0)
                    ok = ok && mbar_wait_sleep(&bars->q_empty[t], (use - 1) & 1, abort);
                if (!ok)
                    return;
                mbar_arrive_expect_tx(&bars->q_full[t], q_bytes);
#pragma unroll
                for (int x = 0; x < kHalves; ++x)
                    tma_load_3d(q_smem + t * L::qtile + x * (kM * 128), &mQ, 64 * x, it.kvh * a.G, it.q0 + it.tok0 + t * a.ntok,
                                &bars->q_full[t]);
                ++use;
            };
            auto load_kv = [&](const CUtensorMap* m, int j) {
                const uint32_t st = slot % kStages, use = slot / kStages;
                if (use > 0)
                    ok = ok && mbar_wait_sleep(&bars->kv_empty[st], (use - 1) & 1, abort);
                if (!ok)
                    return;
                mbar_arrive_expect_tx(&bars->kv_full[st], L::tile);
#pragma unroll
                for (int x = 0; x < kHalves; ++x)
                    tma_load_4d(kv_smem + st * L::tile + x * (kN * 128), m, 64 * x, it.kv0 + j * kN, it.kvh, it.plane,
                                &bars->kv_full[st]);
                ++slot;
            };
            for (int r = 0; (ok || kSplit) && item_at(r, it); ++r) {
                const int n0 = it.nk(0), n1 = it.nk(1), n = max(n0, n1), jb = first_tile(n), je = end_tile(n);
                if constexpr (kSplit) {
                    // the ring held this CTA's part of the item before.  Arriving here for every item, whatever
                    // happened, keeps this thread within one phase of part_read
                    if (r > 0)
                        ok = ok && mbar_wait_sleep(&bars->part_read, (r - 1) & 1, abort);
                    mbar_arrive(&bars->part_full);
                }
                for (int j = jb; ok && j < je; ++j) {
                    if (j == jb && n0 > jb)
                        load_q(0, q_use0);
                    load_kv(&mK, j);
                    if (j == jb && n1 > jb)
                        load_q(1, q_use1);
                    load_kv(&mV, j);
                }
            }
            if (!ok) {
                if (!*abort)
                    report(a.err, RKV_ERR_TIMEOUT);
                *abort = 1;
            }
            bars->issued = static_cast<int>(slot);
            bars->q_issued[0] = static_cast<int>(q_use0);
            bars->q_issued[1] = static_cast<int>(q_use1);
        } else if (warp > 0 && elect_one()) {
            // ---------------- MMA issuers, one thread each: warps 1 and 2 form S of query tiles 0 and 1, warp 3 P V of both, so
            // that an S whose buffer has become free never stands behind a P that is not ready.  Steps c of a query tile
            // are counted over all items; K_j of an item is ring slot `slot` + 2 j, V_j the next.
            constexpr uint32_t kTileDesc = L::tile >> 4;   // descriptors count 16 bytes
            uint32_t slot = 0;
            auto wait = [&](uint64_t* bar, uint32_t parity) {
                ok = ok && mbar_wait(bar, parity, abort);
                return ok;
            };
            if (warp < 3) {
                const int t = warp - 1;
                const uint64_t q_desc = smem_desc_sw128(q_smem + t * L::qtile), k_desc = smem_desc_sw128(kv_smem);
                const uint32_t tm_s = tmem + 128 * t;
                uint32_t q_use = 0, c = 0;
                for (int r = 0; ok && item_at(r, it); ++r) {
                    const int nk = it.nk(t), n = max(nk, it.nk(1 - t)), jb = first_tile(n), je = end_tile(n);
                    for (int j = jb; j < je; ++j, slot += 2) {
                        const uint32_t ks = slot % kStages;
                        if (!wait(&bars->kv_full[ks], (slot / kStages) & 1))
                            break;
                        if (j >= nk) {
                            mbar_arrive(&bars->kv_empty[ks]);      // the other query tile's alone
                            continue;
                        }
                        if (j == jb && !wait(&bars->q_full[t], q_use++ & 1))
                            break;
                        // P V of step c - 2 has read the P buffer that follows from this S, and S of step c - 1 is in the
                        // softmax warps' registers
                        if (c > 1 && !wait(&bars->pv_done[t][c & 1], ((c - 2) >> 1) & 1))
                            break;
                        if (c > 0 && !wait(&bars->s_free[t], (c - 1) & 1))
                            break;
                        tc_fence_after();
                        // over the 16-key groups that some row sees
                        const uint32_t width = j + 1 < nk ? kN : it.last_width(t);
                        const uint32_t idesc = idesc_f32<kF16>(kM, 0) | ((width >> 3) << 17);
                        const uint64_t kd = k_desc + ks * kTileDesc;
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk)
                            mma_f16(tm_s, q_desc + (kk / 4) * ((kM * 128) >> 4) + (kk % 4) * 2,
                                    kd + (kk / 4) * ((kN * 128) >> 4) + (kk % 4) * 2, idesc, kk > 0 ? 1u : 0u);
                        mma_commit(&bars->s_full[t]);
                        mma_commit(&bars->kv_empty[ks]);
                        if (j + 1 == min(nk, je))
                            mma_commit(&bars->q_empty[t]);
                        ++c;
                    }
                }
            } else {
                constexpr uint32_t idescO = idesc_f32<kF16>(kM, D) | (1u << 16);   // B (= V) MN-major
                const uint64_t v_desc = smem_desc_mn(kv_smem);
                uint32_t c0 = 0, c1 = 0;
                auto issue_pv = [&](int t, uint32_t c, uint64_t vd, int groups, bool first) {
                    if (!wait(&bars->p_ready[t][c & 1], (c >> 1) & 1))
                        return;
                    tc_fence_after();
#pragma unroll
                    for (int kk = 0; kk < kN / 16; ++kk)
                        if (kk < groups)
                            mma_f16_ts(tmem + 256 + 128 * t, tmem + 128 * t + 64 + 32 * (c & 1) + 8 * kk,
                                       vd + kk * (2048 >> 4), idescO, (first && kk == 0) ? 0u : 1u);
                    mma_commit(&bars->pv_done[t][c & 1]);
                };
                for (int r = 0; ok && item_at(r, it); ++r) {
                    const int n0 = it.nk(0), n1 = it.nk(1), n = max(n0, n1), jb = first_tile(n), je = end_tile(n);
                    for (int j = jb; j < je; ++j, slot += 2) {
                        const uint32_t vs = (slot + 1) % kStages;
                        if (!wait(&bars->kv_full[vs], ((slot + 1) / kStages) & 1))
                            break;
                        const uint64_t vd = v_desc + vs * kTileDesc;
                        if (j < n0)
                            issue_pv(0, c0++, vd, (j + 1 < n0 ? kN : it.last_width(0)) / 16, j == jb);
                        if (j < n1)
                            issue_pv(1, c1++, vd, (j + 1 < n1 ? kN : it.last_width(1)) / 16, j == jb);
                        if (!ok)
                            break;
                        mma_commit(&bars->kv_empty[vs]);
                    }
                }
            }
            if (!ok) {
                if (!*abort)
                    report(a.err, RKV_ERR_TIMEOUT);
                *abort = 1;
            }
            // every product that this thread issued has completed before TMEM is released
            volatile int never = 0;
            mma_commit(&bars->last[warp - 1]);
            mbar_wait(&bars->last[warp - 1], 0, &never);
        }
    } else {
        // ---------------- softmax: thread = row of query tile t = TMEM lane
        const int t = (warp - 4) >> 2, row = tid & 127;
        const uint32_t lane_off = static_cast<uint32_t>(32 * (warp & 3)) << 16;
        const uint32_t tm_s = tmem + 128 * t + lane_off, tm_o = tmem + 256 + 128 * t + lane_off;
        const int row_tok = row / a.G, row_head = row - row_tok * a.G;
        // The warps of the two query tiles that share a scheduler take turns at their exponentials: each then has the
        // special-function unit to itself while the other waits for S, finds its maximum or stores.
        const int my_turn = 1 + 2 * (warp & 3) + t, other_turn = 1 + 2 * (warp & 3) + 1 - t;
        uint32_t c = 0, slot = 0;                           // steps of this query tile, ring slots
        bool ok = true;
        Item it, next;
        auto wait = [&](uint64_t* bar, uint32_t parity) {
            const bool got = ok && mbar_wait(bar, parity, abort);
            ok = __all_sync(0xffffffffu, got);
            tc_fence_after();
        };
        if (t == 1)
            named_arrive(other_turn, 64);
        // after a wait gave up the loops go on without work, so that the turns stay matched
        bool more = item_at(0, it);
        for (int r = 0; more; ++r, it = next) {
            const int nk = it.nk(t), tok = it.tok0 + t * a.ntok + row_tok;
            const int lim = it.L - it.n + tok;              // last key that this row sees
            const bool valid = row < a.ntok * a.G && tok < it.n;
            const int n = max(nk, it.nk(1 - t)), jb = first_tile(n), je = end_tile(n), jt = min(nk, je);
            float m = kNone;                                // of S: c m_i is the formula's maximum
            uint64_t sum = pair(0.0f, 0.0f);
            for (int j = jb; j < jt; ++j, ++c) {
                wait(&bars->s_full[t], c & 1);
                float s[64];
                tmem_ld32_async(tm_s, s);
                tmem_ld32_async(tm_s + 32, s + 32);
                tmem_ld_wait();
                tmem_arrived(s);
                tmem_arrived(s + 32);
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars->s_free[t]);          // the next S may be formed
                const int cut = lim - j * kN;               // columns past it are masked
                if (__any_sync(0xffffffffu, cut < kN - 1)) {
#pragma unroll
                    for (int x = 0; x < 64; ++x)
                        s[x] = x <= cut ? s[x] : -INFINITY;
                }
                float t0 = max3(s[0], s[1], s[2]), t1 = max3(s[3], s[4], s[5]), t2 = max3(s[6], s[7], s[8]),
                      t3 = max3(s[9], s[10], s[11]);
#pragma unroll
                for (int x = 12; x + 8 <= 64; x += 8) {
                    t0 = max3(t0, s[x], s[x + 1]);
                    t1 = max3(t1, s[x + 2], s[x + 3]);
                    t2 = max3(t2, s[x + 4], s[x + 5]);
                    t3 = max3(t3, s[x + 6], s[x + 7]);
                }
                t0 = max3(t0, s[60], s[61]);
                t1 = max3(t1, s[62], s[63]);
                t0 = max3(t0, t1, t2);
                // rows that are not stored take no part in what the warp decides together
                const float top = valid ? max3(t0, t0, t3) : -INFINITY;
                // the accumulator keeps its old maximum until the new one is 2^8 larger (the first tile counts as such);
                // a warp rescales together.  A NaN becomes the maximum, and with it every weight of its row
                if (__any_sync(0xffffffffu, !((top - m) * a.c <= kLazy))) {
                    const float was = m;
                    m = (top - m) * a.c <= kLazy ? m : top;
                    const float f = ex2((was - m) * a.c);
                    // the product before this step still adds to O
                    if (j > jb)
                        wait(&bars->pv_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1);
                    float x0, x1;
                    unpair(sum, x0, x1);
                    sum = pair(x0 * f, x1 * f);
#pragma unroll 1
                    for (int x = 0; j > jb && x < D / 16; ++x) {
                        uint32_t w[16];
                        float o[16];
                        tmem_ld16(tm_o + 16 * x, o);
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = __float_as_uint(o[i] * f);
                        tmem_st16(tm_o + 16 * x, w);
                    }
                }
                if (j == n - 1 && (it.L & 15) && n * kN > it.L) {
                    // V rows behind the last key, within its group of 16, meet weights of 0 in the product: they may
                    // hold NaN and are zeroed, by the warps of each query tile before they hand over P
                    const uint32_t vs = slot + 2 * (j - jb) + 1;
                    wait(&bars->kv_full[vs % kStages], (vs / kStages) & 1);
                    const int left = it.L - j * kN;
                    for (int i = row; ok && i < (16 - (left & 15)) * kHalves * 8; i += 128) {
                        const int key = left + i / (kHalves * 8), x = (i >> 3) % kHalves;
                        *reinterpret_cast<uint4*>(sm + L::kv + (vs % kStages) * L::tile + x * (kN * 128) + key * 128 +
                                                  (i & 7) * 16) = make_uint4(0, 0, 0, 0);
                    }
                    fence_proxy_async_smem();
                }
                const uint32_t tm_p = tm_s + 64 + 32 * (c & 1);
                // exponents s c + off; rows without a key so far keep a finite offset whatever c
                float off1 = kBias<kF16> - fmaxf(m * a.c, kNone);
                const bool far = m != kNone && !(fabsf(m * a.c) < kFar);
                if (__any_sync(0xffffffffu, far)) {
                    const float base = far ? m : 0.0f;
#pragma unroll
                    for (int x = 0; x < 64; ++x)
                        s[x] -= base;
                    off1 = far ? kBias<kF16> : off1;
                }
                const uint64_t cc = pair(a.c, a.c), off = pair(off1, off1);
                uint64_t a0 = pair(0.0f, 0.0f), a1 = a0;
                named_sync(my_turn, 64);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    uint32_t w[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const uint64_t e = fma2(pair(s[32 * x + 2 * i], s[32 * x + 2 * i + 1]), cc, off);
                        float u, v;
                        if (kPoly > 0 && i % kPoly == kPoly - 1) {
                            exp2_pair(e, u, v);
                        } else {
                            float e0, e1;
                            unpair(e, e0, e1);
                            u = ex2(e0);
                            v = ex2(e1);
                        }
                        w[i] = pack2<kF16>(u, v);
                        if (i & 1)
                            a1 = add2(a1, pair(u, v));
                        else
                            a0 = add2(a0, pair(u, v));
                    }
                    tmem_st16(tm_p + 16 * x, w);
                }
                named_arrive(other_turn, 64);
                tmem_st_wait();
                tc_fence_before();
                __syncwarp();
                if (lane == 0)
                    mbar_arrive(&bars->p_ready[t][c & 1]);
                sum = add2(sum, add2(a0, a1));
            }
            for (int j = max(jt, jb); j < je; ++j) {        // steps of the other query tile alone
                named_sync(my_turn, 64);
                named_arrive(other_turn, 64);
            }
            // while the last product runs: the next item, and what the rows of this one need
            slot += 2 * (je - jb);
            more = item_at(r + 1, next);
            const bool sees = lim >= 0;
            const int head = it.kvh * a.G + row_head;
            const int64_t q_row = static_cast<int64_t>(it.q0) + tok;
            const int64_t row_at = q_row * a.out_row_stride + head * a.out_head_stride;   // elements
            float l0, l1;
            unpair(sum, l0, l1);
            const float l = l0 + l1, inv_l = sees ? 1.0f / l : 0.0f;
            const float log_sum = sees ? (m * a.c - kBias<kF16> + log2f(l)) * 0.6931471805599453f : -INFINITY;
            if (jt > jb)
                wait(&bars->pv_done[t][(c - 1) & 1], ((c - 1) >> 1) & 1);
            const bool store = ok && valid;
            if constexpr (kSplit) {
                // The parts (m, l, O) of the cluster's CTAs go through the ring, which the item has left, and CTA `part` joins
                // the columns from part * D / parts on: M = max m_x, f_x = 2^(c (m_x - M)), O = sum f_x O_x / sum f_x l_x.
                // Parts without a key tile are (lowest float, 0, 0).
                if (r > 0)
                    wait(&bars->part_read, (r - 1) & 1);
                named_sync(kJoinBar, 256);                       // the products of both query tiles are done
                const uint32_t ml_at = L::stage + (t * kM + row) * 8, o_at = L::kv + t * (kM * D * 4) + row * 16;
                *reinterpret_cast<float2*>(sm + ml_at) = make_float2(m, l);
#pragma unroll 1
                for (int x = 0; x < D / 32; ++x) {
                    float o[32];
                    tmem_ld32(tm_o + 32 * x, o);
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        *reinterpret_cast<float4*>(sm + o_at + (8 * x + i) * (kM * 16)) =
                            jt > jb ? make_float4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3])
                                    : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                }
                tc_fence_before();                               // the next item's first product overwrites O
                fence_proxy_async_smem();                        // later copies into the ring come after these stores
                named_sync(kJoinBar, 256);
                if (warp == 4 && lane < parts)
                    arrive_at(&bars->part_full, lane);
                __syncwarp();
                ok = __all_sync(0xffffffffu, ok && mbar_wait_cluster(&bars->part_full, r & 1, abort));
                // all of a thread's loads from the other CTAs are under way at once
                float2 ml[kMaxParts];
#pragma unroll
                for (uint32_t x = 0; x < kMaxParts; ++x)
                    ml[x] = x < parts ? peer_float2(peer_addr(smem_addr(sm + ml_at), x)) : make_float2(kNone, 0.0f);
                float M = kNone, sum_l = 0.0f;
#pragma unroll
                for (uint32_t x = 0; x < kMaxParts; ++x)
                    M = max3(M, M, ml[x].x);
#pragma unroll
                for (uint32_t x = 0; x < kMaxParts; ++x) {
                    ml[x].x = ex2((ml[x].x - M) * a.c);
                    sum_l = fmaf(ml[x].x, ml[x].y, sum_l);
                }
                const float inv = sees ? 1.0f / sum_l : 0.0f;
                if (store && a.lse && part == 0)
                    a.lse[q_row * a.Hq + head] = sees ? (M * a.c - kBias<kF16> + log2f(sum_l)) * 0.6931471805599453f : -INFINITY;
                const int cols = D / static_cast<int>(parts);
#pragma unroll 1
                for (int col = part * cols; col < static_cast<int>(part + 1) * cols; col += 8) {
                    float4 v[kMaxParts][2];
#pragma unroll
                    for (uint32_t x = 0; x < kMaxParts; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h)
                            v[x][h] = x < parts ? peer_float4(peer_addr(smem_addr(sm + o_at + (col / 4 + h) * (kM * 16)), x))
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    float o[8] = {};
#pragma unroll
                    for (uint32_t x = 0; x < kMaxParts; ++x)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            o[4 * h] = fmaf(ml[x].x, v[x][h].x, o[4 * h]);
                            o[4 * h + 1] = fmaf(ml[x].x, v[x][h].y, o[4 * h + 1]);
                            o[4 * h + 2] = fmaf(ml[x].x, v[x][h].z, o[4 * h + 2]);
                            o[4 * h + 3] = fmaf(ml[x].x, v[x][h].w, o[4 * h + 3]);
                        }
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        o[i] = sees ? o[i] * inv : 0.0f;
                    if (!store)
                        continue;
                    const int64_t at = row_at + col;
                    if (a.out_dtype == RKV_DTYPE_F32) {
                        float4* dst = reinterpret_cast<float4*>(static_cast<float*>(a.out) + at);
                        dst[0] = make_float4(o[0], o[1], o[2], o[3]);
                        dst[1] = make_float4(o[4], o[5], o[6], o[7]);
                    } else {
                        *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at) =
                            make_uint4(pack2<kF16>(o[0], o[1]), pack2<kF16>(o[2], o[3]), pack2<kF16>(o[4], o[5]),
                                       pack2<kF16>(o[6], o[7]));
                    }
                }
                named_sync(kJoinBar, 256);
                if (warp == 4 && lane < parts)
                    arrive_at(&bars->part_read, lane);
                __syncwarp();
                continue;
            }
            if (store && a.lse)
                a.lse[q_row * a.Hq + head] = log_sum;
            // Rows go out through a small staging area of the warp, 64 bytes of each at a time, so that four lanes store
            // neighbouring pieces of one row (a lane storing its own row touches 32 lines per instruction: 4800 cycles
            // an item instead of 2600).  16-byte pieces are swizzled by the row against bank conflicts.
            const uint32_t rows = __ballot_sync(0xffffffffu, store);
            unsigned char* st = sm + L::stage + (warp - 4) * kStage;
            const bool f32 = a.out_dtype == RKV_DTYPE_F32;
            unsigned char* to[4];                           // this lane's pieces: rows 8 i + lane / 4
#pragma unroll
            for (int i = 0; i < 4; ++i)
                to[i] = static_cast<unsigned char*>(a.out) + 16 * (lane & 3) +
                        __shfl_sync(0xffffffffu, row_at, 8 * i + (lane >> 2)) * (f32 ? 4 : 2);
            auto put = [&](const uint32_t (&w)[16], int col_bytes) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    *reinterpret_cast<uint4*>(st + lane * 64 + ((i ^ ((lane >> 1) & 3)) << 4)) =
                        make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
                __syncwarp();
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const int src = 8 * i + (lane >> 2);    // row of the warp
                    const uint4 v = *reinterpret_cast<const uint4*>(st + src * 64 + (((lane & 3) ^ ((src >> 1) & 3)) << 4));
                    if (rows >> src & 1u)
                        *reinterpret_cast<uint4*>(to[i] + col_bytes) = v;
                }
                __syncwarp();
            };
#pragma unroll 1
            for (int x = 0; rows != 0 && x < D; x += 64) {
                float o[64];
                tmem_ld32_async(tm_o + x, o);
                tmem_ld32_async(tm_o + x + 32, o + 32);
                tmem_ld_wait();
                tmem_arrived(o);
                tmem_arrived(o + 32);
                uint32_t w[16];
                if (f32) {
#pragma unroll
                    for (int y = 0; y < 64; y += 16) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = __float_as_uint(sees ? o[y + i] * inv_l : 0.0f);
                        put(w, 4 * (x + y));
                    }
                } else {
#pragma unroll
                    for (int y = 0; y < 64; y += 32) {
#pragma unroll
                        for (int i = 0; i < 16; ++i)
                            w[i] = sees ? pack2<kF16>(o[y + 2 * i] * inv_l, o[y + 2 * i + 1] * inv_l) : 0u;
                        put(w, 2 * (x + y));
                    }
                }
            }
            // the next item's first product overwrites O: it is ordered behind these loads by p_ready
            tc_fence_before();
        }
        if (t == 0)
            named_sync(my_turn, 64);                        // the turn that the other warp still passes on
        if (!ok && lane == 0) {
            if (!*abort)
                report(a.err, RKV_ERR_TIMEOUT);
            *abort = 1;
        }
    }

    // copies that are still in flight (only after an abort) land before the CTA may exit
    __syncthreads();
    if (tid == 0) {
        volatile int never = 0;
        const int n = bars->issued;
        for (int i = n > kStages ? n - kStages : 0; i < n; ++i)
            mbar_wait(&bars->kv_full[i % kStages], (i / kStages) & 1, &never);
        for (int t = 0; t < 2; ++t)
            if (bars->q_issued[t] > 0)
                mbar_wait(&bars->q_full[t], (bars->q_issued[t] - 1) & 1, &never);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmemCols);
    }
    if constexpr (kSplit) {
        __syncwarp();
        cluster_sync_all();                                      // no CTA leaves while others may read its shared memory
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

template <int D, bool kF16, bool kSplit>
cudaError_t launch_t(const CUtensorMap& mQ, const CUtensorMap& mK, const CUtensorMap& mV, const PrefillArgs& a,
                     int workers, int parts, cudaStream_t st)
{
    auto kern = prefill_kernel<D, kF16, kSplit>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, Layout<D>::alloc);
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(workers * parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = Layout<D>::alloc;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = parts;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = kSplit ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, kern, mQ, mK, mV, a);
}

// CTAs that share the keys of an item, as a cluster.  The join costs about as much as 9 key tiles, and a second round
// of items more than a split saves, so: the most CTAs that still run all at once (a GPU Processing Cluster holds
// whole clusters only: 16 clusters of eight CTAs need two rounds, 12 do not, so eight must fit three quarters of the
// SMs) and take at least 10 tiles off a sequence of mean length.  Measured for new tokens over earlier keys, 1 / 2 / 4 / 8
// CTAs: 4 items of 100000 keys (head_dim 64) 903 / 454 / 238 / 127 us; 8 items of 1200 17.1 / 17.0 / 14.9 / 13.9 us, of
// 600 12.6 / 14.4 / 13.2 / 12.7 us; 16 items of 2400 28.3 / 22.4 / 18.0 / 28.4 us; 64 items of 1000 24.6 / 23.1 / 45.4 us.
int split_of(int64_t items, const rkv_prefill_config& c, int sms)
{
    const int64_t tiles = c.kv_rows / kN / (c.kv_padded ? 1 : c.batch);
    int parts = 1;
    for (int p = 2; p <= static_cast<int>(kMaxParts); p *= 2)
        if (items * p <= (p == 8 ? sms * 3 / 4 : sms) && tiles - tiles / p >= 10)
            parts = p;
    return parts;
}

}  // namespace

cudaError_t launch_prefill(const rkv_prefill_config& c, const void* q, const void* K, const void* V,
                           const int32_t* q_off, const int32_t* kv_off, const int32_t* kv_len, void* out, float* lse,
                           int32_t* err, int sms, cudaStream_t st)
{
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
    a.level_keys = static_cast<int>((int64_t(96) << 20) / (4ll * c.head_dim * c.n_kv_heads));   // 96 MB of K and V
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
    // the items are known on the device only: at most one partial pair of tiles per sequence
    const int64_t items = (c.q_rows / (2 * a.ntok) + c.batch) * c.n_kv_heads;
    if (items > INT32_MAX)
        return cudaErrorInvalidValue;
    const int parts = split_of(items, c, sms);
    const int workers = static_cast<int>(items < sms / parts ? items : sms / parts);
    auto launch = [&](auto d, auto half) {
        constexpr int D = decltype(d)::value;
        constexpr bool kF16 = decltype(half)::value;
        return parts > 1 ? launch_t<D, kF16, true>(mQ, mK, mV, a, workers, parts, st)
                         : launch_t<D, kF16, false>(mQ, mK, mV, a, workers, 1, st);
    };
    using D64 = std::integral_constant<int, 64>;
    using D128 = std::integral_constant<int, 128>;
    if (c.head_dim == 128)
        return f16 ? launch(D128{}, std::true_type{}) : launch(D128{}, std::false_type{});
    return f16 ? launch(D64{}, std::true_type{}) : launch(D64{}, std::false_type{});
}

}  // namespace rkv
