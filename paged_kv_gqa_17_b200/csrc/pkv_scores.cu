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
// Scores outlive the call and decide what an eviction drops, so nothing of an
// earlier call may enter them: the workspace is zeroed once, and a pair's range,
// states and logits count only where every one of its slots' blocks left a
// record of this call.  The check runs beside the loads of the states.
// Sums run over the heads in ascending order and every score has one writer,
// so results are deterministic.
//
// Bound by the launch and one chain of loads (lengths and slots, then logits,
// scores and the slots' maxima at once): 6.4 us more than the decode alone at
// one row of 32768 tokens (28.9 against 22.5 us; 1 MB of scores and 4 MB of
// logits), 4 us of 52 us at eight rows of 533 to 16381 tokens.
#include "pkv_device.h"

namespace pkv {

namespace {

template <int LH>
__global__ void __launch_bounds__(kWeightThreads) add_weights_kernel(const __grid_constant__ WeightParams p)
{
    __shared__ float s_m[LH], s_inv[LH];
    __shared__ int s_end;
    const int chunks = (int)((p.capacity + kWeightTokens - 1) / kWeightTokens);
    grid_dependency_wait();
    grid_launch_dependents();
    add_weights<LH, true>(p, blockIdx.x / chunks, blockIdx.x % chunks, s_m, s_inv, &s_end);
}

}  // namespace

cudaError_t launch_add_weights(const WeightParams &w, int64_t pairs, cudaStream_t st, bool pdl)
{
    const unsigned grid = (unsigned)weight_blocks(pairs, w.capacity);
    switch (logit_heads(w.G)) {
    case 2: return launch_kernel(add_weights_kernel<2>, grid, kWeightThreads, 0, st, pdl, w);
    case 4: return launch_kernel(add_weights_kernel<4>, grid, kWeightThreads, 0, st, pdl, w);
    case 8: return launch_kernel(add_weights_kernel<8>, grid, kWeightThreads, 0, st, pdl, w);
    default: return launch_kernel(add_weights_kernel<16>, grid, kWeightThreads, 0, st, pdl, w);
    }
}

}  // namespace pkv
