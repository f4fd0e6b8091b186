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
//      memory, and a radix select finds the A-th largest key T in three digits
//      of 11, 11 and 10 bits: count the keys per digit value, then find the
//      digit from the counts.  Scores of one row share their exponents, so
//      short digits put most keys into few counters, whose atomics then wait
//      for one another.
//   2. Each warp counts its segment's keys above T and equal to T; prefix sums
//      give every key its rank, so which equals stay and which hole meets which
//      mover follow without another sort.
//   3. The moves are copied over all threads of the cluster, each thread one
//      copy unit (16 bytes, or less where a row is shorter) of a token per
//      step.  A move's source lies at or behind A and its destination before
//      it, so their order is free.
//   4. The recent tokens' first batch is loaded beside the selection; after a
//      cluster barrier (every mover read, every batch loaded) it is stored.
//      Longer windows repeat load, barrier, store.
// Where the block table has room for few tokens (kLocalKeys; the lengths are on
// the device) the cluster's first block selects alone and the others read its
// lists through distributed shared memory: a few thousand keys cost less than
// the cluster barriers that sharing them takes.  Above, the blocks own contiguous
// shares of [0, M), add their counts through distributed shared memory, each
// block the values of its slice, and hand the two lists over through the
// workspace.  Alone against shared, us on fresh scores with a cold L2, one page
// over the budget: 64 pairs (clusters of four) 22.5 / 26.6 at 2064 tokens, 28.6 /
// 28.7 at 5120, 34.8 / 30.7 at 8192, 84 / 35 at 16384; 8 pairs (of eight) 20.5 /
// 26.6, 24.6 / 26.6, 30.7 / 26.6, 45 / 31.  A block without peers has no barrier to
// save, only lists that are nearer (kAloneKeys): 152 pairs 28.7 / 36.9 at 2064, 53 /
// 68 at 14336, but 96 / 74 at 16384, where the keys and lists of two blocks no
// longer fit an SM.
// Every write has one writer, so results are deterministic.
//
// What bounds it: one page over the budget, latency (12.7 us for 10 MB that could
// pass in 1.6 us: a dependent chain of loads of scores, three digits, lists,
// page ids and rows); whole prompts, memory (32 rows and heads of 16384 to 32768
// fresh tokens to 8192, with nothing in L2: 81 us, 4.2 TB/s while the rows move).
#include "pkv_device.h"

#include <algorithm>
#include <climits>
#include <cstring>

namespace pkv {

namespace {

constexpr int kEvictThreads = 256;
constexpr int kEvictPerSM = 2;       // blocks an SM holds
constexpr int kEvictWarps = kEvictThreads / 32;
constexpr int kLocalKeys = 6144;    // capacity up to which one block selects for its cluster
constexpr int kAloneKeys = 14336;   // ... for itself where it has no peers; two blocks still fit an SM
constexpr int kMaxKeys = 16384;     // shared selection: keys a block holds (the rest is read again)
constexpr int kMaxTable = 2048;     // block-table entries a block holds
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kMaxPlanes = PKV_EVICT_MAX_PLANES;
constexpr int kWide = 4;            // 16-byte units of recent tokens a thread has in flight
constexpr int kDeep = 6;            // ... and of moves
constexpr int kNarrow = 2;          // smaller ones; with 8 moves or 4 smaller units registers spill (12.7 -> 13.3 us one page over)

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
    int32_t n_planes, wide, units;  // units per token: of 16 bytes, and in all (those of 16 bytes first)
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

__device__ __forceinline__ void st_cluster_u32(uint32_t addr, uint32_t v)
{
    asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ int ld_cluster_u16(uint32_t addr)
{
    uint16_t v;
    asm volatile("ld.shared::cluster.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
    return v;
}

struct __align__(16) EvictShared {
    uint32_t hist[2][kBins];
    uint32_t total[kBins / 2];  // shared selection: the cluster's counts of this block's slice of the values
    uint32_t warp_sum[kEvictWarps], scan[kEvictWarps], slice_sum[kMaxCluster];
    uint32_t digit, above;
    uint32_t gt[kEvictWarps], eq[kEvictWarps];
    uint32_t block_gt, block_eq;  // read by the peers
    uint32_t moves;               // written by the block that owns slot A: to all (shared selection), or read by the peers
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

__device__ __forceinline__ uint32_t inclusive_scan(uint32_t v, int lane)
{
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t up = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o)
            v += up;
    }
    return v;
}

// Adds the block's keys to hist by digit_of(key) (kBins: not counted), four
// keys loaded at a time.  One value may dominate (tokens that no query has met yet all score
// zero), and additions to one address run one by one: the lanes of a warp
// that agree with its first make one addition.
template <typename K, typename V>
__device__ __forceinline__ void count_keys(uint32_t *hist, int count, int tid, K key_at, V digit_of)
{
    const int lane = tid & 31;
    for (int i0 = 0; i0 < count; i0 += 4 * kEvictThreads) {
        uint32_t digit[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int i = i0 + k * kEvictThreads + tid;
            digit[k] = i < count ? digit_of(key_at(i)) : (uint32_t)kBins;
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint32_t first = __shfl_sync(0xffffffffu, digit[k], 0);
            const uint32_t same = __ballot_sync(0xffffffffu, digit[k] == first);
            if (digit[k] < kBins && (lane == 0 || digit[k] != first))
                atomicAdd(hist + digit[k], lane == 0 ? __popc(same) : 1u);
        }
    }
}

// n: this thread's counts of the digit values from top_value down, threads in
// order from the top, `above` keys above all of them: found(digit, keys above
// it) in the thread that holds the digit of the need-th key.
template <int N, typename F>
__device__ __forceinline__ void find_digit(EvictShared &sh, const uint32_t (&n)[N], int top_value, uint32_t above, uint32_t need,
                                           F found)
{
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    uint32_t sum = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
        sum += n[j];
    const uint32_t incl = inclusive_scan(sum, lane);
    if (lane == 31)
        sh.scan[warp] = incl;
    __syncthreads();
    above += incl - sum;
#pragma unroll
    for (int w = 0; w < kEvictWarps; ++w)
        above += w < warp ? sh.scan[w] : 0u;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        if (above < need && need <= above + n[j])
            found((uint32_t)(top_value - j), above);
        above += n[j];
    }
}

// The need-th largest (1 <= need <= all) of the keys of CS blocks (`key_at`
// gives this block's `count`), in three digits of 11, 11 and 10 bits: with
// that many values the first digit splits scores of like size well enough that
// the counting is not serialised on a few addresses.  The blocks' counts are
// added through distributed shared memory.  `need` becomes T's rank among the keys
// equal to it.  sh.hist is zero before.
template <int CS, typename K>
__device__ __forceinline__ uint32_t select_key(EvictShared &sh, K key_at, int count, uint32_t &need)
{
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    constexpr int kPer = kBins / kEvictThreads;  // bins per thread, from the top
    static_assert(kPer == 8, "two 16-byte reads");
    uint32_t prefix = 0;
#pragma unroll
    for (int d = 0; d < 3; ++d) {
        const int shift = d == 0 ? 21 : d == 1 ? 10 : 0;
        const uint32_t mask = d == 2 ? 1023u : 2047u;
        uint32_t *hist = sh.hist[d & 1];
        count_keys(hist, count, tid, key_at, [&](uint32_t key) {
            const bool in = d == 0 || (key >> (d == 1 ? 21 : 10)) == (prefix >> (d == 1 ? 21 : 10));
            return in ? (key >> shift) & mask : (uint32_t)kBins;
        });
        evict_sync<CS>();
        if (CS == 1) {
            const int at = kBins - kPer - tid * kPer;
            const uint4 hi = *reinterpret_cast<const uint4 *>(hist + at + 4);
            const uint4 lo = *reinterpret_cast<const uint4 *>(hist + at);
            const uint32_t n[kPer] = {hi.w, hi.z, hi.y, hi.x, lo.w, lo.z, lo.y, lo.x};  // descending
            find_digit(sh, n, kBins - 1 - tid * kPer, 0u, need, [&](uint32_t digit, uint32_t above) {
                sh.digit = digit;
                sh.above = above;
            });
        } else {
            // Block c adds up the cluster's counts of its slice of the values, slices from the top; the
            // slices' sums tell every block where T's digit lies, and that slice's block finds it.
            constexpr int kSlice = kBins / CS, kMine = kSlice / kEvictThreads;  // per thread: 1, 2 or 4
            const int rank = (int)cluster_ctarank();
            const uint32_t *slice = hist + kBins - (rank + 1) * kSlice;
            uint32_t sum = 0;
#pragma unroll
            for (int h = 0; h < kMine; ++h) {
                const uint32_t mine = smem_addr(slice + tid + h * kEvictThreads);
                uint32_t v[CS], all = 0;
#pragma unroll
                for (int c = 0; c < CS; ++c)
                    v[c] = ld_cluster_u32(map_shared_rank(mine, (uint32_t)c));
#pragma unroll
                for (int c = 0; c < CS; ++c)
                    all += v[c];
                sh.total[tid + h * kEvictThreads] = all;
                sum += all;
            }
            sum = __reduce_add_sync(0xffffffffu, sum);
            if (lane == 0)
                sh.warp_sum[warp] = sum;
            __syncthreads();
            if (tid < CS) {
                uint32_t all = 0;
#pragma unroll
                for (int w = 0; w < kEvictWarps; ++w)
                    all += sh.warp_sum[w];
                st_cluster_u32(map_shared_rank(smem_addr(sh.slice_sum + rank), (uint32_t)tid), all);
            }
            evict_sync<CS>();
            uint32_t above = 0, mine = 0;
#pragma unroll
            for (int c = 0; c < CS; ++c) {
                above += c < rank ? sh.slice_sum[c] : 0u;
                mine = c == rank ? sh.slice_sum[c] : mine;
            }
            if (above < need && need <= above + mine) {  // the same for the whole block
                uint32_t n[kMine];
#pragma unroll
                for (int j = 0; j < kMine; ++j)
                    n[j] = sh.total[kSlice - 1 - tid * kMine - j];
                find_digit(sh, n, kBins - rank * kSlice - 1 - tid * kMine, above, need, [&](uint32_t digit, uint32_t rest) {
                    for (int c = 0; c < CS; ++c) {
                        st_cluster_u32(map_shared_rank(smem_addr(&sh.digit), (uint32_t)c), digit);
                        st_cluster_u32(map_shared_rank(smem_addr(&sh.above), (uint32_t)c), rest);
                    }
                });
            }
            evict_sync<CS>();
        }
        if (d == 1)  // the third digit counts where the first did: every block is past its reading of those
            for (int i = tid; i < kBins; i += kEvictThreads)
                sh.hist[0][i] = 0;
        __syncthreads();
        prefix |= sh.digit << shift;
        need -= sh.above;
    }
    return prefix;
}

// A copy unit of one (row, head)'s tokens: where slot s's lies.
struct UnitAddress {
    uint8_t *base;  // NULL: no unit
    int64_t page, slot;
    int32_t size, dense;
};

template <int CS, bool LOCAL>
__global__ void __launch_bounds__(kEvictThreads, kEvictPerSM) evict_kernel(const __grid_constant__ EvictParams p)
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
    for (int i = tid; i < 2 * kBins; i += kEvictThreads)
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

    __syncthreads();

    // ---- the copies' lanes and addresses; the first recent tokens ----
    // A token's units of one width lie side by side over the threads; as many tokens at once as fit.
    struct Lanes {
        int unit, first, stride;  // this thread's unit (of those of its width), its first token, tokens per step
    };
    auto lanes = [&](int units) {
        Lanes l{tid, rank, CS};
        if (units == 0) {
            l.first = l.stride = INT_MAX / 2;
        } else if (units <= kEvictThreads) {
            const int abreast = kEvictThreads / units, mine = tid / units;
            l.unit = tid - mine * units;
            l.first = mine < abreast ? rank * abreast + mine : INT_MAX / 2;
            l.stride = abreast * CS;
        }
        return l;
    };
    const int narrow_units = p.units - p.wide;
    const Lanes wide = lanes(p.wide), narrow = lanes(narrow_units);
    auto address = [&](int u, int end) {
        UnitAddress t{nullptr, 0, 0, 0, 0};
        if (u >= end)
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
    // The unit of the token in `slot`; ok becomes false where its page id is out of range.
    auto at = [&](const UnitAddress &t, int slot, bool &ok) -> uint8_t * {
        if (t.dense)
            return t.base + slot * t.slot;
        const int index = slot / kPage;
        const int page = index < p.held_table ? s_table[index] : __ldg(table + index);
        const bool good = page >= 0 && page < p.num_pool_pages;
        ok = ok && good;
        return t.base + (good ? page : 0) * t.page + (slot % kPage) * t.slot;
    };
    auto report = [&](bool ok) {
        if (!ok)
            atomicOr(p.ws_error, kErrPageId);
        return ok;
    };
    auto load_small = [&](const uint8_t *src, int size) -> uint2 {
        switch (size) {
        case 8: return *reinterpret_cast<const uint2 *>(src);
        case 4: return make_uint2(*reinterpret_cast<const uint32_t *>(src), 0);
        case 2: return make_uint2(*reinterpret_cast<const uint16_t *>(src), 0);
        default: return make_uint2(*src, 0);
        }
    };
    auto store_small = [&](uint8_t *dst, uint2 v, int size) {
        switch (size) {
        case 8: *reinterpret_cast<uint2 *>(dst) = v; break;
        case 4: *reinterpret_cast<uint32_t *>(dst) = v.x; break;
        case 2: *reinterpret_cast<uint16_t *>(dst) = (uint16_t)v.x; break;
        default: *dst = (uint8_t)v.x; break;
        }
    };
    // The recent tokens go in batches: all of a batch is loaded before any of it
    // is stored, everywhere in the cluster, and a batch's targets never hold a
    // later batch's sources.  The first is loaded here, beside the selection (no move touches
    // its sources), and stored once the movers, whose slots it takes, are read.
    uint4 rw[kWide];
    uint8_t *rw_dst[kWide];
    uint2 rn[kNarrow];
    uint8_t *rn_dst[kNarrow];
    int rn_size = 0;
    auto load_recent = [&](int round, int batch) {
        const UnitAddress tw = address(wide.unit + round * kEvictThreads, p.wide);
#pragma unroll
        for (int k = 0; k < kWide; ++k) {
            const int64_t j = (int64_t)(batch * kWide + k) * wide.stride + wide.first;
            rw_dst[k] = nullptr;
            if (tw.base && j < p.recent) {
                bool ok = true;
                const uint8_t *src = at(tw, M + (int)j, ok);
                uint8_t *dst = at(tw, A + (int)j, ok);
                rw[k] = *reinterpret_cast<const uint4 *>(src);
                rw_dst[k] = report(ok) ? dst : nullptr;
            }
        }
        const UnitAddress tn = address(p.wide + narrow.unit + round * kEvictThreads, p.units);
        rn_size = tn.size;
#pragma unroll
        for (int k = 0; k < kNarrow; ++k) {
            const int64_t j = (int64_t)(batch * kNarrow + k) * narrow.stride + narrow.first;
            rn_dst[k] = nullptr;
            if (tn.base && j < p.recent) {
                bool ok = true;
                const uint8_t *src = at(tn, M + (int)j, ok);
                uint8_t *dst = at(tn, A + (int)j, ok);
                rn[k] = load_small(src, tn.size);
                rn_dst[k] = report(ok) ? dst : nullptr;
            }
        }
    };
    load_recent(0, 0);

    if (A > 0 && (!LOCAL || rank == 0)) {
        const int share = LOCAL ? M : (M + CS - 1) / CS;
        const int lo = LOCAL ? 0 : min(rank * share, M), count = min(lo + share, M) - lo;
        const int held = LOCAL ? count : min(count, kMaxKeys);
#pragma unroll 4
        for (int i = tid; i < held; i += kEvictThreads)
            s_keys[i] = score_key(scores[lo + i]);
        auto key_at = [&](int i) { return LOCAL || i < held ? s_keys[i] : score_key(scores[lo + i]); };
        __syncthreads();

        // ---- 1. the A-th largest key, T: `need` >= 1 of the keys equal to it stay, the first ones ----
        uint32_t need = (uint32_t)A;
        const uint32_t T = select_key<(LOCAL ? 1 : CS)>(sh, key_at, count, need);

        // ---- 2. ranks, and the lists ----
        const int segment = ((count + kEvictWarps - 1) / kEvictWarps + 31) & ~31;  // per warp
        const int s0 = min(warp * segment, count), s1 = min(s0 + segment, count);
        uint32_t gt = 0, eq = 0;
#pragma unroll 4
        for (int i = s0 + lane; i < s1; i += 32) {
            const uint32_t key = key_at(i);
            gt += key > T;
            eq += key == T;
        }
        gt = __reduce_add_sync(0xffffffffu, gt);
        eq = __reduce_add_sync(0xffffffffu, eq);
        if (lane == 0) {
            sh.gt[warp] = gt;
            sh.eq[warp] = eq;
        }
        __syncthreads();
        {
            // counts of the warps before this one
            const uint32_t g = lane < kEvictWarps ? sh.gt[lane] : 0u, e = lane < kEvictWarps ? sh.eq[lane] : 0u;
            if (!LOCAL && warp == 0) {
                const uint32_t all_g = __reduce_add_sync(0xffffffffu, g), all_e = __reduce_add_sync(0xffffffffu, e);
                if (lane == 0) {
                    sh.block_gt = all_g;
                    sh.block_eq = all_e;
                }
            }
            gt = __reduce_add_sync(0xffffffffu, lane < warp ? g : 0u);
            eq = __reduce_add_sync(0xffffffffu, lane < warp ? e : 0u);
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
                    if (CS == 1 || LOCAL)
                        sh.moves = (uint32_t)(A - kept_before);
                    else
                        for (int c = 0; c < CS; ++c)
                            st_cluster_u32(map_shared_rank(smem_addr(&sh.moves), (uint32_t)c),
                                           (uint32_t)(A - kept_before));
                }
            }
            gt += __popc(bg);
            eq += __popc(be);
        }
    }

    // ---- 3. the moves ----
    evict_sync<CS>();  // the lists are there
    int moves = 0;
    uint32_t hole_at = smem_addr(s_holes), mover_at = smem_addr(s_movers);  // of the block that selected
    if (A > 0) {
        if (LOCAL && CS > 1) {
            // The selecting block wrote these in its own shared memory alone: a block's may be touched by others only
            // once it is known to run, and for a local selection the barrier above is the first to say so.
            hole_at = map_shared_rank(hole_at, 0);
            mover_at = map_shared_rank(mover_at, 0);
            moves = (int)ld_cluster_u32(map_shared_rank(smem_addr(&sh.moves), 0));
        } else {
            moves = (int)sh.moves;
        }
    }
    auto mover = [&](int j) { return LOCAL ? ld_cluster_u16(mover_at + 2 * (moves - 1 - j)) : __ldcg(movers + moves - 1 - j); };
    auto hole = [&](int j) { return LOCAL ? ld_cluster_u16(hole_at + 2 * j) : __ldcg(holes + j); };
    for (int u = wide.unit; u < p.wide; u += kEvictThreads) {  // once unless a token has more units than the block threads
        const UnitAddress t = address(u, p.wide);
        // a step's rows are loaded while the next step's places are looked up
        int from[kDeep], to[kDeep];
        auto places = [&](int j0) {
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                const int j = min(j0 + k * wide.stride, moves - 1);
                from[k] = mover(j);
                to[k] = hole(j);
            }
        };
        if (wide.first < moves)
            places(wide.first);
        for (int j0 = wide.first; j0 < moves; j0 += kDeep * wide.stride) {
            uint4 val[kDeep];
            uint8_t *dst[kDeep];
            bool all = true;
#pragma unroll
            for (int k = 0; k < kDeep; ++k) {
                bool ok = true;
                val[k] = *reinterpret_cast<const uint4 *>(at(t, from[k], ok));
                dst[k] = at(t, to[k], ok);
                all = all && ok;
                if (!ok || j0 + k * wide.stride >= moves)
                    dst[k] = nullptr;
            }
            report(all);
            if (moves - j0 > kDeep * wide.stride)
                places(j0 + kDeep * wide.stride);
#pragma unroll
            for (int k = 0; k < kDeep; ++k)
                if (dst[k])
                    *reinterpret_cast<uint4 *>(dst[k]) = val[k];
        }
    }
    for (int u = narrow.unit; u < narrow_units; u += kEvictThreads) {
        const UnitAddress t = address(p.wide + u, p.units);
        for (int j0 = narrow.first; j0 < moves; j0 += 4 * narrow.stride) {
            int from[4], to[4];
            uint2 val[4];
            uint8_t *dst[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int j = min(j0 + k * narrow.stride, moves - 1);
                from[k] = mover(j);
                to[k] = hole(j);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                bool ok = true;
                val[k] = load_small(at(t, from[k], ok), t.size);
                dst[k] = at(t, to[k], ok);
                if (!report(ok) || j0 + k * narrow.stride >= moves)
                    dst[k] = nullptr;
            }
#pragma unroll
            for (int k = 0; k < 4; ++k)
                if (dst[k])
                    store_small(dst[k], val[k], t.size);
        }
    }
    // ---- 4. the recent tokens ----
    const int rounds = (max(p.wide, narrow_units) + kEvictThreads - 1) / kEvictThreads;
    for (int r = 0; r < rounds; ++r) {
        for (int b = 0; b == 0 || (int64_t)b * kWide * wide.stride < p.recent || (int64_t)b * kNarrow * narrow.stride < p.recent;
             ++b) {
            if (r > 0 || b > 0)
                load_recent(r, b);
            evict_sync<CS>();
#pragma unroll
            for (int k = 0; k < kWide; ++k)
                if (rw_dst[k])
                    *reinterpret_cast<uint4 *>(rw_dst[k]) = rw[k];
#pragma unroll
            for (int k = 0; k < kNarrow; ++k)
                if (rn_dst[k])
                    store_small(rn_dst[k], rn[k], rn_size);
        }
    }
    // vacated slots start from zero when new tokens take them (all loads lie before a barrier above)
    for (int i = p.budget + rank * kEvictThreads + tid; i < N; i += CS * kEvictThreads)
        scores[i] = 0.f;
}

template <int CS, bool LOCAL>
cudaError_t launch_evict(const EvictParams &p, int64_t pairs, cudaStream_t st)
{
    static std::atomic<uint64_t> configured{0};
    auto kernel = evict_kernel<CS, LOCAL>;
    const cudaError_t e = allow_smem(kernel, (kMaxKeys + kMaxTable) * 4 + kAloneKeys * 2, configured);
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
        s.num_pool_pages < 1)
        return PKV_ERR_INVALID;
    // the heads of a row read its length while its first one writes the new one
    const uintptr_t before = reinterpret_cast<uintptr_t>(seq_lens), after = reinterpret_cast<uintptr_t>(new_lens);
    if (before < after + 4 * (uintptr_t)s.B && after < before + 4 * (uintptr_t)s.B)
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
        // two planes over one array would move its rows twice at once
        for (int j = 0; j < i; ++j) {
            const uintptr_t a = reinterpret_cast<uintptr_t>(planes[j].base), b = reinterpret_cast<uintptr_t>(pl.base);
            if (a < b + (uintptr_t)pl.row_bytes && b < a + (uintptr_t)planes[j].row_bytes)
                return PKV_ERR_INVALID;
        }
    }
    if (positions && static_cast<const void *>(positions) == static_cast<const void *>(scores))
        return PKV_ERR_INVALID;
    for (int wide = 1; wide >= 0; --wide) {  // planes of 16-byte units first
        for (int i = 0; i < n_planes; ++i) {
            const pkv_plane &pl = planes[i];
            if ((unit_bytes(pl) == 16) == (wide == 1))
                add(pl.base, pl.stride_page, pl.stride_head, pl.stride_token, unit_bytes(pl), pl.row_bytes, 0);
        }
        if (wide)
            p.wide = p.units;
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
    while (cluster < kMaxCluster && pairs * cluster * 2 <= 148 * kEvictPerSM && capacity / (cluster * 2) >= 256)
        cluster *= 2;
    const bool local = capacity <= (cluster > 1 ? kLocalKeys : kAloneKeys);
    p.held_keys = (int32_t)(local ? capacity : std::min<int64_t>(ceil_div(capacity, cluster), kMaxKeys));
    p.held_keys = (p.held_keys + 3) & ~3;
    p.held_table = std::min(s.max_pages_per_seq, kMaxTable);
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = local ? launch_evict_any<true>(cluster, p, pairs, st)
                                : launch_evict_any<false>(cluster, p, pairs, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

}  // extern "C"
