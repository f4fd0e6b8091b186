// Device-side helpers shared by the kernels of libpkv.so: thin wrappers of the
// PTX instructions they use, and the bounded mbarrier wait.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "pkv_internal.h"

namespace pkv {

constexpr uint64_t kWaitLimitNs = 2000000000ull;
constexpr uint32_t kWaitLimitIters = 1u << 30;

// ---------------------------------------------------------------------------
// PTX wrappers

__device__ __forceinline__ uint32_t smem_addr(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

__device__ __forceinline__ void mbar_init(uint32_t bar, uint32_t count)
{
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}

__device__ __forceinline__ void mbar_expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint32_t bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}

__device__ __forceinline__ bool mbar_try_wait(uint32_t bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n"
        " .reg .pred p;\n"
        " mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        " selp.u32 %0, 1, 0, p;\n"
        "}\n"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    return ok != 0;
}

__device__ __forceinline__ uint64_t global_timer_ns()
{
    uint64_t t;
    asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
    return t;
}

// Wait for phase `parity` of an mbarrier, giving up after kWaitLimitNs (or
// kWaitLimitIters polls) with the timeout bit set in the error word (and,
// when host_flags is not NULL, the timeout's flag word set in host memory).
static __device__ __noinline__ bool mbar_wait(uint32_t bar, uint32_t parity, uint32_t *err, uint64_t limit_ns = kWaitLimitNs,
                                       uint32_t *host_flags = nullptr)
{
    if (mbar_try_wait(bar, parity))
        return true;
    const uint64_t t0 = global_timer_ns();
    for (uint32_t i = 1; i < kWaitLimitIters; ++i) {
        if (mbar_try_wait(bar, parity))
            return true;
        if ((i & 255u) == 0 && global_timer_ns() - t0 > limit_ns)
            break;
    }
    atomicOr(err, kErrTimeout);
    if (host_flags)
        *reinterpret_cast<volatile uint32_t *>(host_flags) = 1u;  // bit 0: timeout
    return false;
}

__device__ __forceinline__ uint64_t evict_first_policy()
{
    uint64_t pol;
    asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(pol));
    return pol;
}

// TMA tiled copy of one [1][1][16][64] box of a pool view into shared memory.
__device__ __forceinline__ void tma_load_box(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int d0, int head,
                                             int page, uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5}], [%6], %7;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(d0), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(policy)
        : "memory");
}

// Bulk (non-tensor) async copy global -> shared, completion on an mbarrier.
// Both addresses 16-byte aligned, size a multiple of 16.
__device__ __forceinline__ void bulk_g2s(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar)
{
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Per-thread asynchronous copies global -> shared that bypass L1 (16 or 4
// bytes), and the wait for all of this thread's copies.
__device__ __forceinline__ void cp_async_16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void cp_async_4(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(reinterpret_cast<uint64_t>(src))
                 : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

// Wait until at most the most recently committed group of this thread's
// async copies is still in flight.
__device__ __forceinline__ void cp_async_wait_but_last() { asm volatile("cp.async.wait_group 1;" ::: "memory"); }

__device__ __forceinline__ void cp_async_wait_all()
{
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
}

// Ticket: atomic add with release (orders this block's earlier writes, made
// visible to thread 0 by the preceding __syncthreads) and acquire (the last
// arriver sees every other block's released writes).
__device__ __forceinline__ uint32_t ticket_acq_rel(uint32_t *ctr)
{
    uint32_t prev;
    asm volatile("atom.add.acq_rel.gpu.global.u32 %0, [%1], 1;" : "=r"(prev) : "l"(ctr) : "memory");
    return prev;
}

__device__ __forceinline__ void fence_proxy_async_global()
{
    asm volatile("fence.proxy.async.global;" ::: "memory");
}

// Programmatic dependent launch: wait for the grids this one depends on
// (complete, memory visible); allow dependents to be scheduled.  Both are
// no-ops when the kernel was launched without the PDL attribute.
__device__ __forceinline__ void grid_dependency_wait()
{
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

__device__ __forceinline__ void grid_launch_dependents()
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// Thread-block clusters: rank in the cluster, a full cluster barrier
// (release / acquire), and loads from a peer block's shared memory.
__device__ __forceinline__ uint32_t cluster_ctarank()
{
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}

__device__ __forceinline__ void cluster_sync_all()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t map_shared_rank(uint32_t addr, uint32_t rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
    return r;
}

__device__ __forceinline__ float ld_cluster_f32(uint32_t addr)
{
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// Barrier among the first `threads` threads of the block (named barrier `id`).
__device__ __forceinline__ void named_barrier(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// TMA tiled copy of a whole (page, head) block [d_hi][16 tokens][64 d] of a
// rank-5 pool view (head_dim split as 64 x d_hi) in one instruction.
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap *tm, uint32_t bar, int head, int page,
                                              uint64_t policy)
{
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
        " [%0], [%1, {%2, %3, %4, %5, %6}], [%7], %8;" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(tm)), "r"(0), "r"(0), "r"(0), "r"(head), "r"(page), "r"(bar), "l"(policy)
        : "memory");
}

// Loads that are cached in L2 only (never in L1), for reads of data that a
// kernel still running may be writing: a later load of the same address
// after the dependency wait cannot hit a stale L1 line.
__device__ __forceinline__ int ld_l2_only(const int32_t *ptr)
{
    int v;
    asm volatile("ld.global.cg.s32 %0, [%1];" : "=r"(v) : "l"(ptr));
    return v;
}

__device__ __forceinline__ int4 ld_l2_only(const int4 *ptr)
{
    int4 v;
    asm volatile("ld.global.cg.v4.s32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(ptr));
    return v;
}

__device__ __forceinline__ void prefetch_tensormap(const CUtensorMap *tm)
{
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(tm)) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_smem()
{
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2, uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

__device__ __forceinline__ void ldsm_x4_trans(uint32_t addr, uint32_t &r0, uint32_t &r1, uint32_t &r2,
                                              uint32_t &r3)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
                 : "r"(addr));
}

// D = A * B + D, m16n8k16, bf16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose an 8x8 b16 matrix held one row pair per lane.
__device__ __forceinline__ uint32_t movmatrix_trans(uint32_t x)
{
    uint32_t y;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}

// 2^x on the SFU (ex2.approx: relative error ~2^-22); 2^-inf = +0.
__device__ __forceinline__ float exp2_approx(float x)
{
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi)
{
    __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<uint32_t *>(&v);
}

__device__ __forceinline__ void store_bf16x4(__nv_bfloat16 *dst, float4 v)
{
    uint2 u;
    u.x = pack_bf16(v.x, v.y);
    u.y = pack_bf16(v.z, v.w);
    *reinterpret_cast<uint2 *>(dst) = u;
}

__device__ __forceinline__ float4 fma4(float4 a, float s, float4 b)  // a * s + b
{
    return make_float4(fmaf(a.x, s, b.x), fmaf(a.y, s, b.y), fmaf(a.z, s, b.z), fmaf(a.w, s, b.w));
}

__device__ __forceinline__ float4 scale4(float4 a, float s)
{
    return make_float4(a.x * s, a.y * s, a.z * s, a.w * s);
}

// ---------------------------------------------------------------------------
// Host side: launches, and the weights kernel that the scored decodes share

template <typename P>
cudaError_t launch_kernel(void (*kernel)(P), unsigned grid, unsigned block, size_t smem, cudaStream_t st, bool pdl,
                          const P &params, unsigned cluster = 0)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(block);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (pdl) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n].val.clusterDim.z = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, params);
    return e != cudaSuccess ? e : cudaGetLastError();
}

// cudaFuncSetAttribute(MaxDynamicSharedMemorySize) once per kernel and device (`done`: one per kernel).
template <typename K>
cudaError_t allow_smem(K kernel, int bytes, std::atomic<uint64_t> &done)
{
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = dev < 64 ? (1ull << dev) : 0;
    if (bit && (done.load() & bit))
        return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e == cudaSuccess && bit)
        done.fetch_or(bit);
    return e;
}

inline bool aligned(const void *p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) == 0; }

// The caller's scores: float [row][KV head][token], tokens contiguous, strides in elements.
struct ScoreArgs {
    float *scores;
    int64_t stride_row, stride_head;
};

// The state slots of one (row, KV head): slot(0) = first, slot(i) = base + step * i.
// `count` 0: none.
struct __align__(16) SlotRange {
    int32_t first, count, base, step;
    __device__ int64_t slot(int i) const { return i == 0 ? first : base + (int64_t)step * i; }
};

// What the block of a slot did in THIS call: every block of a scored bf16 decode writes its own slot's, also one that
// refuses its work item or has none (pair -1).  The pairs' ranges and the states lie in a workspace that earlier calls
// filled; only where a pair's records all agree were its states and logits of tokens [tb, te) written by this call.
struct __align__(16) SlotRecord {
    int32_t pair, first, count, tb, te, unused[3];
};

// Arguments of the weights kernel (pkv_scores.cu).
struct WeightParams {
    const float *logits;       // [pair][capacity][logit_heads(G)], log2 domain
    const float *m, *l;        // [slot][G] states: running max (log2 domain) and denominator
    const SlotRange *ranges;   // per pair; the bf16 decode's are of this call only where the records say so
    const SlotRecord *records; // bf16 decode: per slot
    uint32_t *ws_error;
    const int32_t *seq_lens;
    float *scores;
    int64_t stride_row, stride_head;
    int64_t capacity;          // tokens a row can hold
    int64_t n_slots;
    int32_t H_kv, G;
};

// Blocks of the weights kernel: kWeightTokens tokens of one pair each.
constexpr int kWeightThreads = 256;
constexpr int kWeightTokens = 1024;
inline int64_t weight_blocks(int64_t pairs, int64_t capacity) { return pairs * ceil_div(capacity, kWeightTokens); }

// The tokens of a pair, from 0, whose logits this call's bf16 decode wrote, for the whole
// warp: the row's, fewer where the plan covers fewer, 0 where an item was refused or leaves a gap.
__device__ __forceinline__ int attended_end(const WeightParams &p, int pair, const SlotRange &range, int lane)
{
    bool ok = true;
    int end = 0;
    for (int k0 = 0; k0 < range.count; k0 += 32) {
        const int k = k0 + lane;
        int4 r = make_int4(pair, range.first, range.count, 0);
        int te = 0;
        if (k < range.count) {
            const int4 *record = reinterpret_cast<const int4 *>(p.records + range.first + k);
            r = __ldcg(record);
            te = __ldcg(&record[1].x);
        }
        const int above = __shfl_up_sync(0xffffffffu, te, 1);
        ok = ok && r.x == pair && r.y == range.first && r.z == range.count &&
             (k >= range.count || r.w == (lane == 0 ? end : above));  // the tokens follow one another without a gap
        end = __shfl_sync(0xffffffffu, te, min(31, range.count - 1 - k0));
    }
    return __all_sync(0xffffffffu, ok) ? end : 0;
}

// One block's part of the weights kernel, after the kernel before it has
// completed: adds the weights of tokens [chunk * kWeightTokens, + kWeightTokens)
// of a pair to its scores.  LH = logit_heads(G).  The token's logits and
// scores are loaded before the pair's maximum and sum are known, all at once.
// Tokens that the call's decode did not attend to (a refused work item's pair,
// a row that is longer than its plan) keep their scores; so do all on a workspace
// in which a wait ran out.  RECORDS: the bf16 decode's.
template <int LH, bool RECORDS>
__device__ __forceinline__ void add_weights(const WeightParams &p, int pair, int chunk, float *s_m, float *s_inv,
                                            int *s_end)
{
    constexpr int kTokens = kWeightTokens / kWeightThreads;
    const int row = pair / p.H_kv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int64_t t0 = (int64_t)chunk * kWeightTokens + threadIdx.x;
    const SlotRange range = p.ranges[pair];
    const uint32_t error = __ldcg(p.ws_error);
    int64_t n = __ldg(p.seq_lens + row);
    n = n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
    if ((int64_t)chunk * kWeightTokens >= n)
        return;
    float *out = p.scores + (int64_t)row * p.stride_row + (int64_t)(pair % p.H_kv) * p.stride_head;
    const float *x = p.logits + (int64_t)pair * p.capacity * LH;
    float v[kTokens][LH], old[kTokens];
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int64_t t = t0 + k * kWeightThreads;
        old[k] = 0.f;
        if (t < n) {
            old[k] = out[t];
            if constexpr (LH == 2) {
                const float2 a = __ldcg(reinterpret_cast<const float2 *>(x + t * LH));
                v[k][0] = a.x, v[k][1] = a.y;
            } else {
#pragma unroll
                for (int g = 0; g < LH; g += 4) {
                    const float4 a = __ldcg(reinterpret_cast<const float4 *>(x + t * LH + g));
                    v[k][g] = a.x, v[k][g + 1] = a.y, v[k][g + 2] = a.z, v[k][g + 3] = a.w;
                }
            }
        }
    }
    if (range.first < 0 || range.count < 1 || range.first >= p.n_slots || range.slot(range.count - 1) >= p.n_slots) {
        // none, or an earlier call's
        if (RECORDS && chunk == 0 && threadIdx.x == 0)
            atomicOr(p.ws_error, kErrItem);
        return;
    }
    if (error & kErrTimeout)
        return;  // some page never came: states and logits may be missing
    if (RECORDS && warp == kWeightThreads / 32 - 1) {
        const int end = attended_end(p, pair, range, lane);
        if (lane == 0) {
            *s_end = end;
            if (chunk == 0 && end < n)
                atomicOr(p.ws_error, kErrItem);  // the plan does not cover this row
        }
    }
    for (int g = warp; g < LH; g += kWeightThreads / 32) {
        float m = -INFINITY, l = 0.f;
        if (g < p.G) {
            float m0 = -INFINITY, l0 = 0.f;
            if (lane < range.count) {
                m0 = __ldcg(p.m + range.slot(lane) * p.G + g);
                l0 = __ldcg(p.l + range.slot(lane) * p.G + g);
            }
            m = m0;
            for (int k = lane + 32; k < range.count; k += 32)
                m = fmaxf(m, __ldcg(p.m + range.slot(k) * p.G + g));
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1)
                m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
            m = m == -INFINITY ? 0.f : m;
            l = l0 * exp2_approx(m0 - m);
            for (int k = lane + 32; k < range.count; k += 32)
                l = fmaf(__ldcg(p.l + range.slot(k) * p.G + g), exp2_approx(__ldcg(p.m + range.slot(k) * p.G + g) - m), l);
#pragma unroll
            for (int sh = 16; sh > 0; sh >>= 1)
                l += __shfl_xor_sync(0xffffffffu, l, sh);
        }
        if (lane == 0) {
            s_m[g] = m == -INFINITY ? 0.f : m;
            s_inv[g] = l == 0.f ? 0.f : 1.f / l;  // no weight where every logit is -inf; NaN stays NaN
        }
    }
    __syncthreads();
    float w[kTokens] = {};
#pragma unroll
    for (int g = 0; g < LH; ++g) {
        if (g >= p.G)
            break;
        const float m = s_m[g], inv = s_inv[g];
#pragma unroll
        for (int k = 0; k < kTokens; ++k)
            w[k] = fmaf(exp2_approx(v[k][g] - m), inv, w[k]);
    }
    const int64_t end = RECORDS ? min(n, (int64_t)*s_end) : n;
#pragma unroll
    for (int k = 0; k < kTokens; ++k) {
        const int64_t t = t0 + k * kWeightThreads;
        if (t < end)
            out[t] = old[k] + w[k];
    }
}

cudaError_t launch_add_weights(const WeightParams &w, int64_t pairs, cudaStream_t st, bool pdl);

}  // namespace pkv
