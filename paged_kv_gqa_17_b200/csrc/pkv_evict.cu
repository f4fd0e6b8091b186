// Eviction from a paged cache by accumulated attention weight.
//
// For every row longer than `budget` and each of its KV heads: the `recent`
// newest tokens [M, N) stay (M = N - recent), and of the older ones [0, M) the
// A = budget - recent with the highest scores, the lowest slot first among
// equals (a NaN score ranks as -inf).  Slots are refilled in place:
//   - a kept token in a slot < A does not move;
//   - the vacated slots < A ("holes"), in ascending order, receive the kept
//     tokens from slots [A, M) ("movers"), in ascending order: as many, since
//     A are kept in all;
//   - the recent tokens move down to [A, budget), in order.
// Attention does not depend on the order of cached tokens, so only the holes
// are filled instead of everything behind the first one being moved up: for a
// row one page over its budget that is 16 + recent rows instead of nearly all.
//
// One thread-block cluster works on each (row, KV head); its blocks own
// contiguous, ascending shares of [0, M).
//   1. Scores become 32-bit keys in the order of the floats, kept in shared
//      memory (read again from L2 past kMaxKeys per block), and a radix select
//      finds the A-th largest key T in four 8-bit digits: each block counts
//      its keys per digit value, the blocks' counts are added through
//      distributed shared memory, and every block finds the digit itself.
//   2. Each warp counts its segment's keys above T and equal to T; prefix sums
//      over warps and blocks give every key its rank, so which equals stay and
//      which hole meets which mover follow without another sort.  The two
//      ascending lists go to the workspace.
//   3. The moves are copied unit by unit (16 bytes, or less where a row is
//      shorter) over all threads of the cluster.  Their sources lie at or
//      behind A and their destinations before it, so their order is free.
//   4. After a cluster barrier the recent tokens move down: a barrier between
//      a batch's loads and its stores keeps overlapping ranges apart.
// Every write has one writer, so results are deterministic.
#include "pkv_device.h"

#include <climits>
#include <cstring>

namespace pkv {

namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kMaxKeys = 16384;  // keys a block holds in shared memory
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kMaxPlanes = PKV_EVICT_MAX_PLANES;
constexpr int kBatch = 4;        // units a thread copies at once

// One array that moves with the tokens.  Paged: row bytes at
// base + page * s0 + head * s1 + slot_in_page * s2; dense (scores,
// positions): at base + row * s0 + head * s1 + slot * s2.
struct EvictPlane {
    uint8_t *base;
    int64_t s0, s1, s2;
    int32_t unit;   // bytes per copy: 16, 8, 4, 2 or 1
    int32_t first;  // index of its first unit among a token's units
    int32_t dense;
};

struct EvictParams {
    EvictPlane plane[kMaxPlanes + 2];
    int32_t n_planes, units;  // units per token over all planes
    float *scores;
    int64_t score_row, score_head;
    const int32_t *block_table;
    const int32_t *seq_lens;
    int32_t *new_lens;
    int32_t *lists;  // per (row, head): holes [capacity / 2], movers [capacity / 2]
    uint32_t *ws_error;
    int32_t H_kv, max_pages, num_pool_pages, budget, recent;
    int64_t capacity;
};

// A float's bits as an integer in the floats' order; both zeros are equal,
// NaN ranks as -inf.
__device__ __forceinline__ uint32_t score_key(float x)
{
    if (x != x)
        x = -INFINITY;
    const uint32_t u = __float_as_uint(x + 0.f);  // -0 + 0 = +0
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr)
{
    uint32_t v;
    asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
    return v;
}

union Unit {
    uint4 v16;
    uint2 v8;
    uint32_t v4;
    uint16_t v2;
    uint8_t v1;
};

struct EvictShared {
    uint32_t hist[2][kBins];  // by digit parity: a peer may still read one while the other is counted
    uint32_t total[kBins];    // the cluster's counts of this digit
    uint32_t gt[kEvictWarps], eq[kEvictWarps];
    uint32_t block_gt, block_eq;  // read by the peers
    uint32_t moves;               // likewise, from the block that owns slot A
    uint32_t digit, above;        // the chosen digit value and how many keys lie above it
};

// The cluster's barrier: of one block, the block's.
template <int CS>
__device__ __forceinline__ void evict_sync()
{
    if (CS == 1)
        __syncthreads();
    else
        cluster_sync_all();
}

template <int CS>
__global__ void __launch_bounds__(kEvictThreads) evict_kernel(const __grid_constant__ EvictParams p)
{
    extern __shared__ uint32_t s_keys[];
    __shared__ EvictShared sh;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CS == 1 ? 0 : (int)cluster_ctarank();
    const int pair = blockIdx.x / CS;
    const int row = pair / p.H_kv, head = pair % p.H_kv;
    grid_dependency_wait();
    grid_launch_dependents();
    const int N = __ldg(p.seq_lens + row);
    const bool bad_len = N < 0 || N > p.capacity;
    if (bad_len || N <= p.budget) {  // the same for every block of the cluster
        if (head == 0 && rank == 0 && tid == 0) {
            if (bad_len)
                atomicOr(p.ws_error, kErrSeqLen);
            p.new_lens[row] = N < 0 ? 0 : (N > p.capacity ? (int)p.capacity : N);
        }
        return;
    }
    if (head == 0 && rank == 0 && tid == 0)
        p.new_lens[row] = p.budget;
    const int A = p.budget - p.recent;
    const int M = N - p.recent;  // > A
    float *scores = p.scores + (int64_t)row * p.score_row + (int64_t)head * p.score_head;
    const int half = (int)(p.capacity / 2);
    int32_t *holes = p.lists + (int64_t)pair * 2 * half;
    int32_t *movers = holes + half;

    int moves = 0;
    if (A > 0) {
        const int share = (M + CS - 1) / CS;
        const int lo = min(rank * share, M), count = min(lo + share, M) - lo;
        const int held = min(count, kMaxKeys);
        for (int i = tid; i < held; i += kEvictThreads)
            s_keys[i] = score_key(scores[lo + i]);
        auto key_at = [&](int i) { return i < held ? s_keys[i] : score_key(scores[lo + i]); };

        // ---- 1. the A-th largest key ----
        uint32_t prefix = 0, need = (uint32_t)A;  // T's digits so far; its rank among the keys that share them
        for (int shift = 24, d = 0; shift >= 0; shift -= 8, ++d) {
            uint32_t *hist = sh.hist[d & 1];
            for (int i = tid; i < kBins; i += kEvictThreads)
                hist[i] = 0;
            __syncthreads();
            const uint32_t mask = shift == 24 ? 0u : 0xffffffffu << (shift + 8);
            for (int i0 = 0; i0 < count; i0 += kEvictThreads) {
                const int i = i0 + tid;
                uint32_t bin = kBins;  // not counted
                if (i < count) {
                    const uint32_t key = key_at(i);
                    if ((key & mask) == prefix)
                        bin = (key >> shift) & (kBins - 1);
                }
                // equal digits in a whole warp (scores of like size) are one addition
                int same;
                __match_all_sync(0xffffffffu, bin, &same);
                if (same) {
                    if (lane == 0 && bin < kBins)
                        atomicAdd(hist + bin, 32u);
                } else if (bin < kBins) {
                    atomicAdd(hist + bin, 1u);
                }
            }
            evict_sync<CS>();
            if (tid < kBins) {
                uint32_t sum = 0;
                if (CS == 1) {
                    sum = hist[tid];
                } else {
                    const uint32_t at = smem_addr(hist + tid);
#pragma unroll
                    for (int c = 0; c < CS; ++c)
                        sum += ld_cluster_u32(map_shared_rank(at, (uint32_t)c));
                }
                sh.total[tid] = sum;
            }
            __syncthreads();
            if (warp == 0) {
                // lane l holds bins 255 - 8 l down to 248 - 8 l: a prefix sum over lanes counts from the top
                uint32_t sum = 0;
                for (int j = 0; j < 8; ++j)
                    sum += sh.total[kBins - 1 - (lane * 8 + j)];
                uint32_t incl = sum;
                for (int o = 1; o < 32; o <<= 1) {
                    const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o)
                        incl += v;
                }
                uint32_t above = incl - sum;
                if (above < need && need <= incl) {
                    for (int j = 0; j < 8; ++j) {
                        const int bin = kBins - 1 - (lane * 8 + j);
                        const uint32_t c = sh.total[bin];
                        if (need <= above + c) {
                            sh.digit = (uint32_t)bin;
                            sh.above = above;
                            break;
                        }
                        above += c;
                    }
                }
            }
            __syncthreads();
            prefix |= sh.digit << shift;
            need -= sh.above;
        }
        const uint32_t T = prefix;  // `need` >= 1 of the keys equal to T stay, the first ones

        // ---- 2. ranks, and the lists ----
        const int segment = ((count + kEvictWarps - 1) / kEvictWarps + 31) & ~31;  // per warp
        const int s0 = min(warp * segment, count), s1 = min(s0 + segment, count);
        uint32_t gt = 0, eq = 0;
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t key = i < s1 ? key_at(i) : 0u;
            gt += __popc(__ballot_sync(0xffffffffu, i < s1 && key > T));
            eq += __popc(__ballot_sync(0xffffffffu, i < s1 && key == T));
        }
        if (lane == 0) {
            sh.gt[warp] = gt;
            sh.eq[warp] = eq;
        }
        __syncthreads();
        if (tid == 0) {
            uint32_t g = 0, e = 0;
            for (int w = 0; w < kEvictWarps; ++w) {
                const uint32_t gw = sh.gt[w], ew = sh.eq[w];
                sh.gt[w] = g;
                sh.eq[w] = e;
                g += gw;
                e += ew;
            }
            sh.block_gt = g;
            sh.block_eq = e;
        }
        evict_sync<CS>();
        gt = sh.gt[warp];
        eq = sh.eq[warp];
        if (CS > 1) {
            const uint32_t ag = smem_addr(&sh.block_gt), ae = smem_addr(&sh.block_eq);
#pragma unroll
            for (int c = 0; c < CS; ++c)
                if (c < rank) {
                    gt += ld_cluster_u32(map_shared_rank(ag, (uint32_t)c));
                    eq += ld_cluster_u32(map_shared_rank(ae, (uint32_t)c));
                }
        }
        for (int i0 = s0; i0 < s1; i0 += 32) {
            const int i = i0 + lane;
            const uint32_t key = i < s1 ? key_at(i) : 0u;
            const bool is_gt = i < s1 && key > T, is_eq = i < s1 && key == T;
            const uint32_t bg = __ballot_sync(0xffffffffu, is_gt), be = __ballot_sync(0xffffffffu, is_eq);
            const uint32_t below = (1u << lane) - 1u;
            const uint32_t eq_before = eq + __popc(be & below);
            const uint32_t kept_before = gt + __popc(bg & below) + min(eq_before, need);
            if (i < s1) {
                const int slot = lo + i;
                const bool keep = is_gt || (is_eq && eq_before < need);
                if (slot < A && !keep)
                    holes[slot - (int)kept_before] = slot;
                if (slot >= A && keep)
                    movers[A - 1 - (int)kept_before] = slot;  // the j-th mover from the end
                if (slot == A) {
                    // kept_before tokens keep their slots below A: the other slots there are holes
                    for (int c = 0; c < CS; ++c) {
                        const uint32_t at = CS == 1 ? smem_addr(&sh.moves) : map_shared_rank(smem_addr(&sh.moves), (uint32_t)c);
                        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(at), "r"((uint32_t)A - kept_before)
                                     : "memory");
                    }
                }
            }
            gt += __popc(bg);
            eq += __popc(be);
        }
        evict_sync<CS>();
        moves = (int)sh.moves;
    }

    const int32_t *table = p.block_table + (int64_t)row * p.max_pages;
    // The bytes of unit u of the token in `slot`; NULL where its page id is out of range.
    auto unit_at = [&](const EvictPlane &pl, int u, int slot) -> uint8_t * {
        const int64_t in = (int64_t)(u - pl.first) * pl.unit;
        if (pl.dense)
            return pl.base + (int64_t)row * pl.s0 + (int64_t)head * pl.s1 + (int64_t)slot * pl.s2 + in;
        const int page = __ldg(table + slot / kPage);
        if (page < 0 || page >= p.num_pool_pages) {
            atomicOr(p.ws_error, kErrPageId);
            return nullptr;
        }
        return pl.base + (int64_t)page * pl.s0 + (int64_t)head * pl.s1 + (int64_t)(slot % kPage) * pl.s2 + in;
    };
    // Copies the units of `tokens` moves (token j from source(j) to target(j));
    // SEPARATE: a cluster barrier keeps a batch's loads before its stores.
    auto copy = [&](int tokens, auto source, auto target, bool separate) {
        const int64_t all = (int64_t)tokens * p.units;
        const int64_t stride = (int64_t)CS * kEvictThreads;
        for (int64_t b0 = 0; b0 < all; b0 += stride * kBatch) {
            Unit val[kBatch];
            uint8_t *dst[kBatch];
            int size[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int64_t at = b0 + k * stride + rank * kEvictThreads + tid;
                dst[k] = nullptr;
                size[k] = 0;
                if (at < all) {
                    const int j = (int)(at / p.units), u = (int)(at % p.units);
                    int which = 0;
                    while (which + 1 < p.n_planes && u >= p.plane[which + 1].first)
                        ++which;
                    const EvictPlane &pl = p.plane[which];
                    const uint8_t *src = unit_at(pl, u, source(j));
                    dst[k] = unit_at(pl, u, target(j));
                    if (!src)
                        dst[k] = nullptr;
                    if (dst[k]) {
                        size[k] = pl.unit;
                        switch (pl.unit) {
                        case 16: val[k].v16 = *reinterpret_cast<const uint4 *>(src); break;
                        case 8: val[k].v8 = *reinterpret_cast<const uint2 *>(src); break;
                        case 4: val[k].v4 = *reinterpret_cast<const uint32_t *>(src); break;
                        case 2: val[k].v2 = *reinterpret_cast<const uint16_t *>(src); break;
                        default: val[k].v1 = *src; break;
                        }
                    }
                }
            }
            if (separate)
                evict_sync<CS>();
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (!dst[k])
                    continue;
                switch (size[k]) {
                case 16: *reinterpret_cast<uint4 *>(dst[k]) = val[k].v16; break;
                case 8: *reinterpret_cast<uint2 *>(dst[k]) = val[k].v8; break;
                case 4: *reinterpret_cast<uint32_t *>(dst[k]) = val[k].v4; break;
                case 2: *reinterpret_cast<uint16_t *>(dst[k]) = val[k].v2; break;
                default: *dst[k] = val[k].v1; break;
                }
            }
        }
    };
    // ---- 3. holes, then 4. the recent tokens ----
    copy(moves, [&](int j) { return movers[moves - 1 - j]; }, [&](int j) { return holes[j]; }, false);
    evict_sync<CS>();  // every mover has been read: the recent tokens may take their slots
    copy(p.recent, [&](int j) { return M + j; }, [&](int j) { return A + j; }, true);
    // vacated slots start from zero when new tokens take them (all loads lie before a barrier above)
    for (int t = p.budget + rank * kEvictThreads + tid; t < N; t += CS * kEvictThreads)
        scores[t] = 0.f;
}

template <int CS>
cudaError_t launch_evict(const EvictParams &p, int64_t pairs, int keys, cudaStream_t st)
{
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = allow_smem(evict_kernel<CS>, kMaxKeys * 4, configured);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(evict_kernel<CS>, (unsigned)(pairs * CS), kEvictThreads, (size_t)keys * 4, st, true, p, CS);
}

// The largest copy unit that divides a plane's row and all its addresses.
int unit_bytes(const pkv_plane &pl)
{
    const uint64_t all = reinterpret_cast<uintptr_t>(pl.base) | (uint64_t)pl.stride_page | (uint64_t)pl.stride_head |
                         (uint64_t)pl.stride_token | (uint64_t)pl.row_bytes;
    for (int u = 16; u > 1; u >>= 1)
        if (all % u == 0)
            return u;
    return 1;
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_evict_workspace_bytes(const pkv_shape *shape, size_t *bytes)
{
    if (!bytes || check_shape(shape) != PKV_OK)
        return PKV_ERR_INVALID;
    const size_t pairs = (size_t)shape->B * shape->H_kv;
    *bytes = kWsAlign + round_up(pairs * shape->max_pages_per_seq * shape->page_size * 4, kWsAlign);
    return PKV_OK;
}

int pkv_evict_tokens(float *scores, int64_t score_stride_row, int64_t score_stride_head, int32_t *positions,
                     int64_t position_stride_row, int64_t position_stride_head, const pkv_plane *planes,
                     int32_t n_planes, const int32_t *block_table, const int32_t *seq_lens, int32_t budget,
                     int32_t recent, int32_t *new_lens, const pkv_shape *shape, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    if (check_shape(shape) != PKV_OK || budget < 0 || recent < 0 || recent > budget || n_planes < 0 ||
        (n_planes > 0 && !planes))
        return PKV_ERR_INVALID;
    const pkv_shape &s = *shape;
    if (s.page_size != kPage || n_planes > PKV_EVICT_MAX_PLANES)
        return PKV_ERR_UNSUPPORTED;
    if (s.B == 0)
        return PKV_OK;
    if (!scores || !seq_lens || !new_lens || !workspace || !block_table || s.max_pages_per_seq < 1 ||
        s.num_pool_pages < 1 || seq_lens == new_lens)
        return PKV_ERR_INVALID;
    if (!aligned(scores, 4) || (positions && !aligned(positions, 4)) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(new_lens, 4) || !aligned(workspace, 256))
        return PKV_ERR_UNSUPPORTED;
    const int64_t capacity = (int64_t)s.max_pages_per_seq * kPage;
    const int64_t pairs = (int64_t)s.B * s.H_kv;
    if (capacity > INT32_MAX || pairs * kMaxCluster > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    size_t need = 0;
    pkv_evict_workspace_bytes(shape, &need);
    if (workspace_bytes < need)
        return PKV_ERR_CAPACITY;

    EvictParams p;
    std::memset(&p, 0, sizeof p);
    auto add = [&](void *base, int64_t s0, int64_t s1, int64_t s2, int unit, int bytes, int dense) {
        EvictPlane &pl = p.plane[p.n_planes++];
        pl.base = static_cast<uint8_t *>(base);
        pl.s0 = s0;
        pl.s1 = s1;
        pl.s2 = s2;
        pl.unit = unit;
        pl.first = p.units;
        pl.dense = dense;
        p.units += bytes / unit;
    };
    for (int i = 0; i < n_planes; ++i) {
        const pkv_plane &pl = planes[i];
        if (!pl.base || pl.row_bytes < 1 || pl.stride_page < 0 || pl.stride_head < 0 || pl.stride_token < 0)
            return PKV_ERR_INVALID;
        if (pl.row_bytes > PKV_EVICT_MAX_ROW_BYTES)
            return PKV_ERR_UNSUPPORTED;
        add(pl.base, pl.stride_page, pl.stride_head, pl.stride_token, unit_bytes(pl), pl.row_bytes, 0);
    }
    add(scores, score_stride_row * 4, score_stride_head * 4, 4, 4, 4, 1);
    if (positions)
        add(positions, position_stride_row * 4, position_stride_head * 4, 4, 4, 4, 1);
    p.scores = scores;
    p.score_row = score_stride_row;
    p.score_head = score_stride_head;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.new_lens = new_lens;
    p.ws_error = static_cast<uint32_t *>(workspace);
    p.lists = reinterpret_cast<int32_t *>(static_cast<uint8_t *>(workspace) + kWsAlign);
    p.H_kv = s.H_kv;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    p.budget = budget;
    p.recent = recent;
    p.capacity = capacity;

    int cluster = 1;
    while (cluster < kMaxCluster && pairs * cluster * 2 <= 296 && capacity / (cluster * 2) >= 512)
        cluster *= 2;
    const int64_t share = ceil_div(capacity, cluster);
    const int keys = (int)(share < kMaxKeys ? share : kMaxKeys);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = cluster == 8   ? launch_evict<8>(p, pairs, keys, st)
                          : cluster == 4 ? launch_evict<4>(p, pairs, keys, st)
                          : cluster == 2 ? launch_evict<2>(p, pairs, keys, st)
                                         : launch_evict<1>(p, pairs, keys, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
