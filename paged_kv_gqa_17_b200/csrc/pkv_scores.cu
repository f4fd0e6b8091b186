// Accumulated attention weights: the second kernel of a scored decode.
//
// The decode kernel before it left every valid token's logits x[t][h] (log2
// domain) and each state slot's running max m and denominator l per head.
// With M = max over the pair's slots and L = sum of l 2^(m - M), the weight of
// token t for query head h is 2^(x - M) / L, and
//
//     scores[row][kv head][t] += sum over the G heads of the group.
//
// The weights need the final M and L, which no block of the decode has while
// it streams K, so the logits make one trip through L2 (8 to 64 bytes per
// token against 512 bytes of K and V at D = 128) instead of K being read again.
// Sums run over the heads in ascending order and every score has one writer,
// so results are deterministic.
#include "pkv_device.h"

namespace pkv {

namespace {

constexpr int kWeightThreads = 256;
constexpr int kMaxHeads = 16;

__global__ void __launch_bounds__(kWeightThreads) add_weights_kernel(const WeightParams p)
{
    __shared__ float s_m[kMaxHeads], s_inv[kMaxHeads];
    const int chunks = (int)((p.capacity + kWeightTokens - 1) / kWeightTokens);
    const int pair = blockIdx.x / chunks;
    const int64_t t0 = (int64_t)(blockIdx.x % chunks) * kWeightTokens;
    const int row = pair / p.H_kv;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    grid_dependency_wait();
    grid_launch_dependents();
    int64_t n = __ldg(p.seq_lens + row);
    n = n < 0 ? 0 : (n > p.capacity ? p.capacity : n);
    if (t0 >= n)
        return;
    int2 range = make_int2(pair, 1);
    if (p.slot_range)
        range = p.slot_range[pair];
    // a decode block that refused a malformed work item leaves no usable range
    if (range.x < 0 || range.y < 1 || (int64_t)range.x + range.y > p.n_slots)
        return;
    for (int g = warp; g < p.G; g += kWeightThreads / 32) {
        float m = -INFINITY;
        for (int k = lane; k < range.y; k += 32)
            m = fmaxf(m, p.m[(int64_t)(range.x + k) * p.G + g]);
        for (int sh = 16; sh > 0; sh >>= 1)
            m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
        const float base = m == -INFINITY ? 0.f : m;
        float l = 0.f;
        for (int k = lane; k < range.y; k += 32) {
            const int64_t at = (int64_t)(range.x + k) * p.G + g;
            const float mk = p.m[at];
            if (mk != -INFINITY || p.l[at] != 0.f)
                l = fmaf(p.l[at], exp2_approx(mk - base), l);
        }
        for (int sh = 16; sh > 0; sh >>= 1)
            l += __shfl_xor_sync(0xffffffffu, l, sh);
        if (lane == 0) {
            s_m[g] = base;
            s_inv[g] = l == 0.f ? 0.f : 1.f / l;  // no weight where every logit is -inf; NaN stays NaN
        }
    }
    __syncthreads();
    const int LH = (p.G + 1) & ~1;
    const int64_t t1 = t0 + kWeightTokens < n ? t0 + kWeightTokens : n;
    float *out = p.scores + (int64_t)row * p.stride_row + (int64_t)(pair % p.H_kv) * p.stride_head;
    const float *x = p.logits + (int64_t)pair * p.capacity * LH;
    for (int64_t t = t0 + threadIdx.x; t < t1; t += kWeightThreads) {
        float w = 0.f;
        for (int g = 0; g < LH; g += 2) {
            const float2 v = *reinterpret_cast<const float2 *>(x + t * LH + g);
            w = fmaf(exp2_approx(v.x - s_m[g]), s_inv[g], w);
            if (g + 1 < p.G)
                w = fmaf(exp2_approx(v.y - s_m[g + 1]), s_inv[g + 1], w);
        }
        out[t] += w;
    }
}

}  // namespace

cudaError_t launch_add_weights(const WeightParams &w, int64_t pairs, cudaStream_t st, bool pdl)
{
    return launch_kernel(add_weights_kernel, (unsigned)weight_blocks(pairs, w.capacity), kWeightThreads, 0, st, pdl, w);
}

}  // namespace pkv
