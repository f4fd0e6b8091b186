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
// One thread-block cluster works on each (row, KV head).
//   1. Scores become 32-bit keys in the order of the floats, held in shared
//      memory, and a radix select finds the A-th largest key T in four 8-bit
//      digits: count the keys per digit value, then every warp finds the digit
//      for itself from the counts (three count buffers in turn, so that one
//      barrier per digit is enough).
//   2. Each warp counts its segment's keys above T and equal to T; prefix sums
//      give every key its rank, so which equals stay and which hole meets which
//      mover follow without another sort.
//   3. The moves are copied over all threads of the cluster, each thread one
//      copy unit (16 bytes, or less where a row is shorter) of a token per
//      step.  A move's source lies at or behind A and its destination before
//      it, so their order is free.
//   4. The recent tokens' first batch is loaded beside the moves; after a
//      cluster barrier (every mover read, every batch loaded) it is stored.
//      Longer windows repeat load, barrier, store.
// Up to kLocalKeys tokens every block of the cluster selects for itself, over
// all keys: a few thousand keys cost less than the cluster barriers that
// sharing them takes (64 pairs of 2064 tokens: 24.4 us with shared selection).
// Above, the blocks own contiguous shares of [0, M), add their counts through
// distributed shared memory and hand the two lists over through the workspace.
// Every write has one writer, so results are deterministic.
#include "pkv_device.h"

#include <algorithm>
#include <climits>
#include <cstring>

namespace pkv {

namespace {

constexpr int kEvictThreads = 512;
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kLocalKeys = 8192;    // capacity up to which every block selects for itself
constexpr int kMaxKeys = 16384;     // shared selection: keys a block holds (the rest is read again)
constexpr int kMaxTable = 2048;     // block-table entries a block holds
constexpr int kMaxCluster = 8;
constexpr int kBins = 256;
constexpr int kMaxPlanes = PKV_EVICT_MAX_PLANES;
constexpr int kBatch = 4;           // units a thread has in flight

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
    int32_t held_keys, held_table;  // keys and block-table entries a block keeps in shared memory
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

struct __align__(16) EvictShared {
    uint32_t hist[3][kBins];
    uint32_t total[kBins];                  // shared selection: the cluster's counts of this digit
    uint32_t gt[kEvictWarps], eq[kEvictWarps];
    uint32_t block_gt, block_eq;            // read by the peers
    uint32_t moves;                         // likewise, written by the block that owns slot A
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

// Which unit of a token a thread copies, and where.
struct UnitAddress {
    uint8_t *base;       // of this (row, head) and unit; NULL: no unit for this thread
    int64_t page, slot;  // strides
    int32_t size, dense;
};

template <int CS, bool LOCAL>
__global__ void __launch_bounds__(kEvictThreads, 2) evict_kernel(const __grid_constant__ EvictParams p)
{
    // [keys][block table][LOCAL: holes, movers as 16-bit slots]
    extern __shared__ uint32_t s_keys[];
    __shared__ EvictShared sh;
    int32_t *s_table = reinterpret_cast<int32_t *>(s_keys + p.held_keys);
    uint16_t *s_holes = reinterpret_cast<uint16_t *>(s_table + p.held_table);
    uint16_t *s_movers = s_holes + p.capacity / 2;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rank = CS == 1 ? 0 : (int)cluster_ctarank();
    const int pair = blockIdx.x / CS;
    const int row = pair / p.H_kv, head = pair - row * p.H_kv;
    const int32_t *table = p.block_table + (int64_t)row * p.max_pages;
    for (int i = tid; i < 3 * kBins; i += kEvictThreads)
        sh.hist[0][i] = 0;
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
    for (int i = tid; i < min(p.held_table, (N + kPage - 1) / kPage); i += kEvictThreads)
        s_table[i] = __ldg(table + i);

    int moves = 0;
    if (A > 0) {
        const int share = LOCAL ? M : (M + CS - 1) / CS;
        const int lo = LOCAL ? 0 : min(rank * share, M), count = min(lo + share, M) - lo;
        const int held = LOCAL ? count : min(count, kMaxKeys);
        for (int i = tid; i < held; i += kEvictThreads)
            s_keys[i] = score_key(scores[lo + i]);
        auto key_at = [&](int i) { return LOCAL || i < held ? s_keys[i] : score_key(scores[lo + i]); };
        evict_sync<CS>();  // no block moves a score that another has yet to read

        // ---- 1. the A-th largest key ----
        uint32_t prefix = 0, need = (uint32_t)A;  // T's digits so far; its rank among the keys that share them
#pragma unroll
        for (int d = 0; d < 4; ++d) {
            const int shift = 24 - 8 * d;
            uint32_t *hist = sh.hist[d % 3];
            if (d == 2)  // every warp, and every peer, is past its reading of the first counts
                for (int i = tid; i < kBins; i += kEvictThreads)
                    sh.hist[0][i] = 0;
            for (int i0 = 0; i0 < count; i0 += kEvictThreads) {
                const int i = i0 + tid;
                uint32_t bin = kBins;  // not counted
                if (i < count) {
                    const uint32_t key = key_at(i);
                    if (d == 0 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
                        bin = (key >> shift) & (kBins - 1);
                }
                if (d == 0) {
                    // scores share their leading bits: one addition per value and warp
                    const uint32_t same = __match_any_sync(0xffffffffu, bin);
                    if (bin < kBins && lane == __ffs(same) - 1)
                        atomicAdd(hist + bin, __popc(same));
                } else if (bin < kBins) {
                    atomicAdd(hist + bin, 1u);
                }
            }
            const uint32_t *total = hist;
            if (LOCAL) {
                __syncthreads();
            } else {
                evict_sync<CS>();
                if (tid < kBins) {
                    uint32_t sum = 0;
                    const uint32_t at = smem_addr(hist + tid);
#pragma unroll
                    for (int c = 0; c < CS; ++c)
                        sum += CS == 1 ? hist[tid] : ld_cluster_u32(map_shared_rank(at, (uint32_t)c));
                    sh.total[tid] = sum;
                }
                __syncthreads();
                total = sh.total;
            }
            // lane l holds bins 255 - 8 l down to 248 - 8 l: a prefix sum over lanes counts from the top
            uint32_t n[8], sum = 0;
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                const uint4 v = *reinterpret_cast<const uint4 *>(total + kBins - 4 - (lane * 8 + j));
                n[j] = v.w, n[j + 1] = v.z, n[j + 2] = v.y, n[j + 3] = v.x;
                sum += v.x + v.y + v.z + v.w;
            }
            uint32_t incl = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const uint32_t v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o)
                    incl += v;
            }
            uint32_t above = incl - sum, digit = 0;
            const bool mine = above < need && need <= incl;
            if (mine) {
                bool found = false;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    found = found || need <= above + n[j];
                    if (!found) {
                        above += n[j];
                        digit = j + 1;
                    }
                }
                digit = kBins - 1 - (lane * 8 + digit);
            }
            const int owner = __ffs(__ballot_sync(0xffffffffu, mine)) - 1;
            prefix |= __shfl_sync(0xffffffffu, digit, owner) << shift;
            need -= __shfl_sync(0xffffffffu, above, owner);
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
        {
            // counts of the warps before this one
            uint32_t g = lane < kEvictWarps ? sh.gt[lane] : 0u, e = lane < kEvictWarps ? sh.eq[lane] : 0u;
            if (!LOCAL && warp == 0) {
                uint32_t all_g = g, all_e = e;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) {
                    all_g += __shfl_xor_sync(0xffffffffu, all_g, o);
                    all_e += __shfl_xor_sync(0xffffffffu, all_e, o);
                }
                if (lane == 0) {
                    sh.block_gt = all_g;
                    sh.block_eq = all_e;
                }
            }
            g = lane < warp ? g : 0u;
            e = lane < warp ? e : 0u;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) {
                g += __shfl_xor_sync(0xffffffffu, g, o);
                e += __shfl_xor_sync(0xffffffffu, e, o);
            }
            gt = g;
            eq = e;
        }
        if (!LOCAL) {
            evict_sync<CS>();
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
            const int kept_before = (int)(gt + __popc(bg & below) + min(eq_before, need));
            if (i < s1) {
                const int slot = lo + i;
                const bool keep = is_gt || (is_eq && eq_before < need);
                if (slot < A && !keep) {
                    if (LOCAL)
                        s_holes[slot - kept_before] = (uint16_t)slot;
                    else
                        holes[slot - kept_before] = slot;
                }
                if (slot >= A && keep) {  // the j-th mover from the end
                    if (LOCAL)
                        s_movers[A - 1 - kept_before] = (uint16_t)slot;
                    else
                        movers[A - 1 - kept_before] = slot;
                }
                if (slot == A) {
                    // kept_before tokens keep their slots below A: the other slots there are holes
                    if (LOCAL || CS == 1)
                        sh.moves = (uint32_t)(A - kept_before);
                    else
                        for (int c = 0; c < CS; ++c)
                            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(
                                             map_shared_rank(smem_addr(&sh.moves), (uint32_t)c)),
                                         "r"((uint32_t)(A - kept_before))
                                         : "memory");
                }
            }
            gt += __popc(bg);
            eq += __popc(be);
        }
        if (LOCAL)
            __syncthreads();
        else
            evict_sync<CS>();
        moves = (int)sh.moves;
    } else {
        __syncthreads();  // the table
    }

    // ---- 3. and 4. the copies ----
    // A token's units lie side by side over the threads; as many tokens at once as fit.
    const int abreast = max(1, kEvictThreads / p.units);
    const int first_token = p.units <= kEvictThreads ? tid / p.units : 0;
    const int first_unit = p.units <= kEvictThreads ? tid - first_token * p.units : tid;
    const int stride = abreast * CS;                          // tokens per step of the cluster
    const int first = first_token < abreast ? rank * abreast + first_token : INT_MAX / 2;
    auto address = [&](int u) {
        UnitAddress t{nullptr, 0, 0, 0, 0};
        if (u >= p.units)
            return t;
        int which = 0;
        while (which + 1 < p.n_planes && u >= p.plane[which + 1].first)
            ++which;
        const EvictPlane &pl = p.plane[which];
        t.dense = pl.dense;
        t.size = pl.unit;
        t.base = pl.base + (int64_t)(u - pl.first) * pl.unit + (int64_t)head * pl.s1;
        if (pl.dense)
            t.base += (int64_t)row * pl.s0;
        t.page = pl.s0;
        t.slot = pl.s2;
        return t;
    };
    // The unit of the token in `slot`; NULL where its page id is out of range.
    auto at = [&](const UnitAddress &t, int slot) -> uint8_t * {
        if (t.dense)
            return t.base + slot * t.slot;
        const int index = slot / kPage;
        const int page = index < p.held_table ? s_table[index] : __ldg(table + index);
        if (page < 0 || page >= p.num_pool_pages) {
            atomicOr(p.ws_error, kErrPageId);
            return nullptr;
        }
        return t.base + page * t.page + (slot % kPage) * t.slot;
    };
    auto load = [&](Unit &v, const uint8_t *src, int size) {
        switch (size) {
        case 16: v.v16 = *reinterpret_cast<const uint4 *>(src); break;
        case 8: v.v8 = *reinterpret_cast<const uint2 *>(src); break;
        case 4: v.v4 = *reinterpret_cast<const uint32_t *>(src); break;
        case 2: v.v2 = *reinterpret_cast<const uint16_t *>(src); break;
        default: v.v1 = *src; break;
        }
    };
    auto store = [&](uint8_t *dst, const Unit &v, int size) {
        switch (size) {
        case 16: *reinterpret_cast<uint4 *>(dst) = v.v16; break;
        case 8: *reinterpret_cast<uint2 *>(dst) = v.v8; break;
        case 4: *reinterpret_cast<uint32_t *>(dst) = v.v4; break;
        case 2: *reinterpret_cast<uint16_t *>(dst) = v.v2; break;
        default: *dst = v.v1; break;
        }
    };
    for (int u = first_unit; u < p.units; u += kEvictThreads) {  // one round unless a token has more units than threads
        const UnitAddress t = address(u);
        for (int j0 = first; j0 < moves; j0 += kBatch * stride) {
            Unit val[kBatch];
            uint8_t *dst[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = j0 + k * stride;
                dst[k] = nullptr;
                if (j < moves) {
                    const uint8_t *src = at(t, LOCAL ? s_movers[moves - 1 - j] : __ldcg(movers + moves - 1 - j));
                    dst[k] = at(t, LOCAL ? s_holes[j] : __ldcg(holes + j));
                    if (!src)
                        dst[k] = nullptr;
                    if (dst[k])
                        load(val[k], src, t.size);
                }
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (dst[k])
                    store(dst[k], val[k], t.size);
        }
    }
    // The recent tokens, in batches: all of a batch is loaded before any of it is stored, everywhere in
    // the cluster; their targets hold movers, which the first barrier has read.  A batch's targets never
    // hold a later batch's sources.
    const int rounds = (p.units + kEvictThreads - 1) / kEvictThreads;
    bool first_batch = true;
    for (int r = 0; r < rounds; ++r) {
        const UnitAddress t = address(first_unit + r * kEvictThreads);
        for (int b0 = 0; b0 < p.recent; b0 += kBatch * stride) {
            Unit val[kBatch];
            uint8_t *dst[kBatch];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                const int j = b0 + first + k * stride;
                dst[k] = nullptr;
                if (t.base && j < p.recent) {
                    const uint8_t *src = at(t, M + j);
                    dst[k] = at(t, A + j);
                    if (!src)
                        dst[k] = nullptr;
                    if (dst[k])
                        load(val[k], src, t.size);
                }
            }
            evict_sync<CS>();
            first_batch = false;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (dst[k])
                    store(dst[k], val[k], t.size);
        }
    }
    if (first_batch)
        evict_sync<CS>();
    // vacated slots start from zero when new tokens take them (all loads lie before a barrier above)
    for (int i = p.budget + rank * kEvictThreads + tid; i < N; i += CS * kEvictThreads)
        scores[i] = 0.f;
}

template <int CS, bool LOCAL>
cudaError_t launch_evict(const EvictParams &p, int64_t pairs, cudaStream_t st)
{
    static std::atomic<uint64_t> configured{0};
    auto kernel = evict_kernel<CS, LOCAL>;
    const cudaError_t e = allow_smem(kernel, (kMaxKeys + kMaxTable) * 4, configured);
    if (e != cudaSuccess)
        return e;
    const size_t smem = (size_t)(p.held_keys + p.held_table) * 4 + (LOCAL ? (size_t)p.capacity * 2 : 0);
    return launch_kernel(kernel, (unsigned)(pairs * CS), kEvictThreads, smem, st, true, p, CS);
}

template <bool LOCAL>
cudaError_t launch_evict_any(int cluster, const EvictParams &p, int64_t pairs, cudaStream_t st)
{
    switch (cluster) {
    case 8: return launch_evict<8, LOCAL>(p, pairs, st);
    case 4: return launch_evict<4, LOCAL>(p, pairs, st);
    case 2: return launch_evict<2, LOCAL>(p, pairs, st);
    default: return launch_evict<1, LOCAL>(p, pairs, st);
    }
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
    if (capacity > INT32_MAX / 4 || pairs * kMaxCluster > INT32_MAX)
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
    while (cluster < kMaxCluster && pairs * cluster * 2 <= 296 && capacity / (cluster * 2) >= 256)
        cluster *= 2;
    const bool local = capacity <= kLocalKeys;
    p.held_keys = (int32_t)(local ? capacity : std::min<int64_t>(ceil_div(capacity, cluster), kMaxKeys));
    p.held_keys = (p.held_keys + 3) & ~3;
    p.held_table = std::min(s.max_pages_per_seq, kMaxTable);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = local ? launch_evict_any<true>(cluster, p, pairs, st)
                                : launch_evict_any<false>(cluster, p, pairs, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
