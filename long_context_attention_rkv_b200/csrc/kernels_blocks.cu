// Block tables and slot maps of a block cache, kept on the device.
//
// With have_b = ceil(len_b / s) and need_b = ceil((len_b + new_b) / s) blocks of s tokens, request
// b's missing blocks m_b = need_b - have_b come off the top of the free stack in request order:
//   table[b][have_b + i] = free[n_free - 1 - (M_b + i)],  M_b = sum_{c < b} m_c, i < m_b
// and new token t of the packed order (request b, position p = len_b + t - N_b, N_b = sum_{c < b}
// new_c) gets slot table[b][p / s] * s + p % s.  Giving back is the reverse: the blocks of the ended
// requests go on the stack in request order.
//
// Every CTA reads all lengths (at most 256) and forms the prefix sums itself, in shared memory, so nothing is
// handed over between CTAs; they share the output entries.  A token finds its request by a binary search of the
// prefix sums (8 steps in shared memory).  The lengths and the stack's height may be updated in place, so they
// are written when every CTA has read them: by the only CTA of a small call, behind a cluster's barrier
// (giving back), or by a small second launch (prompts).
#include <cooperative_groups.h>

#include "device_common.cuh"
#include "launchers.h"

namespace rkv {

namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 1024;
constexpr int kMaxCtas = 128;
static_assert(kThreads >= RKV_MAX_BATCH, "one thread per request in the prefix sums");

constexpr int kScanWarps = RKV_MAX_BATCH / 32;

// Inclusive sums of x and y over the first RKV_MAX_BATCH threads (the others only meet the barrier).
__device__ __forceinline__ void block_scan(int64_t& x, int64_t& y, int64_t (*tot)[2])
{
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    if (warp < kScanWarps) {
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t nx = __shfl_up_sync(0xffffffffu, x, o), ny = __shfl_up_sync(0xffffffffu, y, o);
            x += lane >= o ? nx : 0;
            y += lane >= o ? ny : 0;
        }
        if (lane == 31) {
            tot[warp][0] = x;
            tot[warp][1] = y;
        }
    }
    __syncthreads();
    if (warp < kScanWarps) {
#pragma unroll
        for (int w = 0; w < kScanWarps; ++w) {
            x += w < warp ? tot[w][0] : 0;
            y += w < warp ? tot[w][1] : 0;
        }
    }
}

// The request whose range [off[b], off[b + 1]) holds x (empty ranges are passed over).
__device__ __forceinline__ int owner(const int* off, int batch, int x)
{
    int lo = 0, hi = batch - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (off[mid] <= x)
            lo = mid;
        else
            hi = mid - 1;
    }
    return lo;
}

constexpr int kNone = INT32_MAX;

struct BlockShared {
    int64_t tot[kScanWarps][2];
    int off[RKV_MAX_BATCH + 1];    // packed new tokens before request b
    int more[RKV_MAX_BATCH + 1];   // blocks taken (given back) before request b
    int have[RKV_MAX_BATCH];       // blocks that the request holds
    int len[RKV_MAX_BATCH];
    int bad;                       // smallest status that forbids the call (kNone: none)
};

// What rkv_blocks_extend does, from the lengths (whole CTA): the prefix sums in s, s.bad, and for its request each
// thread's held and new tokens.  Returns the stack's height.
__device__ __forceinline__ int plan_extend(const rkv_blocks_config& c, int shift, const int32_t* lengths,
                                           const int32_t* new_counts, const int32_t* n_free, int64_t max_new,
                                           BlockShared& s, int64_t& len, int64_t& add)
{
    const int tid = threadIdx.x;
    if (tid == 0)
        s.bad = kNone;
    __syncthreads();
    const int nfree = *n_free;
    int64_t have = 0, more = 0;
    len = add = 0;
    if (tid < c.batch) {
        len = lengths[tid];
        add = new_counts[tid];
        const int64_t m = (1 << shift) - 1;
        const int64_t need = (len + add + m) >> shift;
        have = (len + m) >> shift;
        if (len < 0 || add < 0) {
            atomicMin(&s.bad, RKV_ERR_INVALID_ARG);
            add = have = 0;
        } else if (need > c.max_blocks) {
            atomicMin(&s.bad, RKV_ERR_WORKSPACE);
            add = 0;
        } else {
            more = need - have;
        }
    }
    int64_t tok = add, blk = more;
    block_scan(tok, blk, s.tot);
    if (tid < c.batch) {
        // sums past 31 bits end in `bad` below and are not used
        s.off[tid + 1] = static_cast<int>(tok < INT32_MAX ? tok : INT32_MAX);
        s.more[tid + 1] = static_cast<int>(blk < INT32_MAX ? blk : INT32_MAX);
        s.have[tid] = static_cast<int>(have);
        s.len[tid] = static_cast<int>(len);
    }
    if (tid == 0) {
        s.off[0] = 0;
        s.more[0] = 0;
        if (nfree < 0 || nfree > c.n_blocks)
            atomicMin(&s.bad, RKV_ERR_INVALID_ARG);
    }
    if (tid == c.batch - 1 && (tok > max_new || blk > nfree))
        atomicMin(&s.bad, RKV_ERR_WORKSPACE);
    __syncthreads();   // also: this CTA has read lengths and n_free
    return nfree;
}

// The new lengths and the stack's height (one CTA, after plan_extend).
__device__ __forceinline__ void write_lengths(const rkv_blocks_config& c, const BlockShared& s, int nfree, int64_t len,
                                              int64_t add, int32_t* lengths_out, int32_t* n_free_out, int32_t* err)
{
    const bool ok = s.bad == kNone;
    if (threadIdx.x < c.batch)
        lengths_out[threadIdx.x] = static_cast<int>(ok ? len + add : len);
    if (threadIdx.x == 0) {
        *n_free_out = nfree - (ok ? s.more[c.batch] : 0);
        if (!ok)
            report(err, s.bad);
    }
}

// kPer: neighbouring tokens per thread and round.  Four almost always share a request and a block, so one search
// and one lookup serve them; in a decode step every token is another request's and one per thread keeps the lookups
// side by side.  kAlone: one CTA, which also writes the new lengths; otherwise another launch does that, when
// every CTA of this one has read the old ones.
template <int kPer, bool kAlone>
__global__ void __launch_bounds__(kThreads)
    blocks_extend_kernel(const rkv_blocks_config c, int shift, const int32_t* lengths, const int32_t* new_counts,
                         int32_t* table, const int32_t* __restrict__ free_list, const int32_t* n_free,
                         int32_t* new_off, int32_t* slot_map, int64_t max_new, int32_t* lengths_out,
                         int32_t* n_free_out, int32_t* err)
{
    __shared__ BlockShared s;
    const int tid = threadIdx.x;
    int64_t len, add;
    const int nfree = plan_extend(c, shift, lengths, new_counts, n_free, max_new, s, len, add);
    if constexpr (kAlone)
        write_lengths(c, s, nfree, len, add, lengths_out, n_free_out, err);

    const int gtid = blockIdx.x * kThreads + tid, gsize = gridDim.x * kThreads;
    const bool ok = s.bad == kNone;
    const int total = ok ? s.off[c.batch] : 0, taken = ok ? s.more[c.batch] : 0;
    if (blockIdx.x == 0 && tid <= c.batch)
        new_off[tid] = ok ? s.off[tid] : 0;
    bool corrupt = false;
    for (int i = gtid; i < taken; i += gsize) {
        const int b = owner(s.more, c.batch, i);
        table[static_cast<int64_t>(b) * c.max_blocks + s.have[b] + i - s.more[b]] = free_list[nfree - 1 - i];
    }
    const bool wide = kPer % 4 == 0 && (reinterpret_cast<uintptr_t>(slot_map) & 15) == 0;
    for (int64_t t0 = static_cast<int64_t>(kPer) * gtid; t0 < max_new; t0 += static_cast<int64_t>(kPer) * gsize) {
        int slot[kPer], b = 0, ord = -1, id = -1;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const int64_t t = t0 + i;
            slot[i] = -1;
            if (t >= total)
                continue;
            if (ord < 0 || t >= s.off[b + 1]) {
                b = owner(s.off, c.batch, static_cast<int>(t));
                ord = -1;
            }
            const int p = s.len[b] + static_cast<int>(t) - s.off[b];
            if (ord != p >> shift) {
                ord = p >> shift;
                // a block taken by this call is read from the stack (its table entry is being written)
                id = ord < s.have[b] ? table[static_cast<int64_t>(b) * c.max_blocks + ord]
                                     : free_list[nfree - 1 - (s.more[b] + ord - s.have[b])];
                if (id < 0 || id >= c.n_blocks) {
                    id = -1;
                    corrupt = true;
                }
            }
            if (id >= 0)
                slot[i] = (id << shift) + (p & ((1 << shift) - 1));
        }
        if (wide && t0 + kPer <= max_new) {
#pragma unroll
            for (int i = 0; i + 3 < kPer; i += 4)
                *reinterpret_cast<int4*>(slot_map + t0 + i) = make_int4(slot[i], slot[i + 1], slot[i + 2], slot[i + 3]);
        } else {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (t0 + i < max_new)
                    slot_map[t0 + i] = slot[i];
        }
    }
    if (corrupt)
        report(err, RKV_ERR_CORRUPT);
}

// The new lengths, after the CTAs of blocks_extend_kernel<., false>.
__global__ void __launch_bounds__(kThreads)
    blocks_lengths_kernel(const rkv_blocks_config c, int shift, const int32_t* lengths, const int32_t* new_counts,
                          const int32_t* n_free, int64_t max_new, int32_t* lengths_out, int32_t* n_free_out, int32_t* err)
{
    __shared__ BlockShared s;
    int64_t len, add;
    const int nfree = plan_extend(c, shift, lengths, new_counts, n_free, max_new, s, len, add);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    write_lengths(c, s, nfree, len, add, lengths_out, n_free_out, err);
}

__global__ void __launch_bounds__(kThreads)
    blocks_release_kernel(const rkv_blocks_config c, int shift, const int32_t* lengths, const int32_t* ended,
                          const int32_t* __restrict__ table, int32_t* free_list, const int32_t* n_free,
                          int32_t* lengths_out, int32_t* n_free_out, int32_t* err)
{
    __shared__ BlockShared s;
    const int tid = threadIdx.x;
    if (tid == 0)
        s.bad = kNone;
    __syncthreads();
    const int nfree = *n_free;
    int64_t len = 0, give = 0;
    bool end = false;
    if (tid < c.batch) {
        len = lengths[tid];
        end = ended[tid] != 0;
        const int64_t have = (len + (1 << shift) - 1) >> shift;
        if (len < 0 || have > c.max_blocks)
            atomicMin(&s.bad, RKV_ERR_CORRUPT);
        else
            give = end ? have : 0;
    }
    int64_t sum = give, unused = 0;
    block_scan(sum, unused, s.tot);
    if (tid < c.batch)
        s.more[tid + 1] = static_cast<int>(sum < INT32_MAX ? sum : INT32_MAX);
    if (tid == 0) {
        s.more[0] = 0;
        if (nfree < 0)
            atomicMin(&s.bad, RKV_ERR_CORRUPT);
    }
    if (tid == c.batch - 1 && nfree + sum > c.n_blocks)
        atomicMin(&s.bad, RKV_ERR_CORRUPT);
    cg::this_cluster().sync();   // lengths and n_free have been read by every CTA

    const int total = s.bad != kNone ? 0 : s.more[c.batch];
    if (blockIdx.x == 0) {
        if (tid < c.batch)
            lengths_out[tid] = (end && s.bad == kNone) ? 0 : static_cast<int>(len);
        if (tid == 0) {
            *n_free_out = nfree + total;
            if (s.bad != kNone)
                report(err, s.bad);
        }
    }
    bool corrupt = false;
    for (int i = blockIdx.x * kThreads + tid; i < total; i += gridDim.x * kThreads) {
        const int b = owner(s.more, c.batch, i);
        const int id = table[static_cast<int64_t>(b) * c.max_blocks + i - s.more[b]];
        corrupt |= id < 0 || id >= c.n_blocks;
        free_list[nfree + i] = id;
    }
    if (corrupt)
        report(err, RKV_ERR_CORRUPT);
}

int log2_of(int n)
{
    int s = 0;
    while ((1 << s) < n)
        ++s;
    return s;
}

// CTAs of rkv_blocks_release: the largest portable cluster.  64 requests of up to 16384 tokens in blocks of 16, half of
// them ended: 4.4 us, in one CTA 15.6 us; 16 of up to 4000: 2.9 and 3.3 us.
constexpr int kReleaseCtas = 8;

}  // namespace

cudaError_t launch_blocks_extend(const rkv_blocks_config& c, const int32_t* lengths, const int32_t* new_counts,
                                 int32_t* table, const int32_t* free_list, const int32_t* n_free, int32_t* new_off,
                                 int32_t* slot_map, int64_t max_new, int32_t* lengths_out, int32_t* n_free_out,
                                 int32_t* err, cudaStream_t st)
{
    const int shift = log2_of(c.block_size);
    if (max_new <= 4 * kThreads) {
        // one CTA; up to one token per thread: a decode step (256 tokens: 3.7 us, with four per thread 6.2 us).  4096
        // tokens of 256 requests: 6.8 us, in the form below 8.5 us
        auto kern = max_new <= kThreads ? blocks_extend_kernel<1, true> : blocks_extend_kernel<4, true>;
        kern<<<1, kThreads, 0, st>>>(c, shift, lengths, new_counts, table, free_list, n_free, new_off, slot_map, max_new,
                                     lengths_out, n_free_out, err);
        return cudaGetLastError();
    }
    // one round of 4 tokens per thread, at most kMaxCtas CTAs.  16384 tokens of 256 requests: 8.1 us, in one CTA 13.6 us;
    // 200000 of 8: 5.7 us with both launches, in one cluster of eight CTAs, whose barrier would save the second, 12.3 us
    const int64_t ctas = (max_new + 4 * kThreads - 1) / (4 * kThreads);
    blocks_extend_kernel<4, false><<<static_cast<unsigned>(ctas < kMaxCtas ? ctas : kMaxCtas), kThreads, 0, st>>>(
        c, shift, lengths, new_counts, table, free_list, n_free, new_off, slot_map, max_new, lengths_out, n_free_out, err);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess)
        return e;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(1);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, blocks_lengths_kernel, c, shift, lengths, new_counts, n_free, max_new, lengths_out,
                              n_free_out, err);
}

cudaError_t launch_blocks_release(const rkv_blocks_config& c, const int32_t* lengths, const int32_t* ended,
                                  const int32_t* table, int32_t* free_list, const int32_t* n_free,
                                  int32_t* lengths_out, int32_t* n_free_out, int32_t* err, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(kReleaseCtas);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = kReleaseCtas;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, blocks_release_kernel, c, log2_of(c.block_size), lengths, ended, table, free_list,
                              n_free, lengths_out, n_free_out, err);
}

}  // namespace rkv
