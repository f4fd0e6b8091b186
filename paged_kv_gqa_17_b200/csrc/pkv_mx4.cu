// The 4-bit paged cache: tokens quantised into it, read back, and attended.
//
// Format.  A value is (-1)^s {0, .5, 1, 1.5, 2, 3, 4, 6}[low three bits]
// 2^(scale - 127): e2m1 codes under one power-of-two scale (an exponent byte)
// per 32 dims of a token, 17/64 of bf16's bytes.  A page (16 tokens) of one KV head
// is one record of 17 D bytes, so that one bulk copy stages it:
//     K codes [16][D/2], V codes [16][D/2], K scales [16][D/32], V scales [16][D/32].
// Codes lie in the order in which the tensor-core fragments take them:
//   - K: dim 32 b + 8 c + j in byte c D/8 + 4 b + j/2 of its row.  Lane (r, c) of
//     a warp holds row r of K as the MMA's A operand; its D/8 bytes at c D/8 are
//     eight dims of every scale block, one 16-byte (D = 128) shared load, and a
//     k-step of 16 dims never mixes two scale blocks;
//   - V: dim 32 b + 4 r + j in byte r D/16 + 2 b + j/2.  Lane (r, c) holds dims of
//     row r of V^T for four tokens; the four dims it owns in every block are two
//     bytes, all blocks together one 8-byte load per token.
// (j/2 names the byte, its low four bits the even j.)
#include "pkv_device.h"

#include <algorithm>
#include <cfloat>
#include <climits>
#include <cstring>

#include <cuda_fp16.h>

namespace pkv {

namespace {

// ---------------------------------------------------------------------------
// Record layout

template <int D>
struct Rec {
    static constexpr int kRow = D / 2;        // bytes of a token's codes
    static constexpr int kScaleRow = D / 32;  // bytes of a token's scales
    static constexpr int kV = kPage * kRow;
    static constexpr int kKs = 2 * kPage * kRow;
    static constexpr int kVs = kKs + kPage * kScaleRow;
    static constexpr int kBytes = kVs + kPage * kScaleRow;
    static_assert(kBytes == 17 * D, "record size");
};

// Two e2m1 codes (a byte) to two halves, exactly; the low four bits to the low half.
__device__ __forceinline__ void codes_to_half2(uint32_t w, uint32_t (&out)[4])
{
    asm("{\n"
        " .reg .b8 b0, b1, b2, b3;\n"
        " mov.b32 {b0, b1, b2, b3}, %4;\n"
        " cvt.rn.f16x2.e2m1x2 %0, b0;\n"
        " cvt.rn.f16x2.e2m1x2 %1, b1;\n"
        " cvt.rn.f16x2.e2m1x2 %2, b2;\n"
        " cvt.rn.f16x2.e2m1x2 %3, b3;\n"
        "}\n"
        : "=r"(out[0]), "=r"(out[1]), "=r"(out[2]), "=r"(out[3])
        : "r"(w));
}

// Eight floats to eight e2m1 codes, round to nearest even, saturating at 6;
// x[0] in the lowest four bits.
__device__ __forceinline__ uint32_t floats_to_codes(const float (&x)[8])
{
    uint32_t w;
    asm("{\n"
        " .reg .b8 b0, b1, b2, b3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b0, %2, %1;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b1, %4, %3;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b2, %6, %5;\n"
        " cvt.rn.satfinite.e2m1x2.f32 b3, %8, %7;\n"
        " mov.b32 %0, {b0, b1, b2, b3};\n"
        "}\n"
        : "=r"(w)
        : "f"(x[0]), "f"(x[1]), "f"(x[2]), "f"(x[3]), "f"(x[4]), "f"(x[5]), "f"(x[6]), "f"(x[7]));
    return w;
}

// ---------------------------------------------------------------------------
// Tokens in and out

// Token j of the call belongs to row i with indptr[i] <= j < indptr[i + 1] (to
// row j without an indptr) and lies at seq_lens[i] + j - indptr[i] there.
struct TokenMap {
    const int32_t *block_table;
    const int32_t *seq_lens;
    const int32_t *indptr;
    uint32_t *ws_error;
    int32_t B, max_pages, num_pool_pages;
};

// The record of token j (of head 0) and its slot, or NULL: no row's token, or
// out of its row's pages or the pool (reported).
__device__ __forceinline__ const uint8_t *token_record(const TokenMap &m, const uint8_t *pool, int64_t stride_page, int j,
                                                       bool report, int &slot)
{
    int row = j;
    int64_t at;
    if (m.indptr) {
        int lo = 0, hi = m.B;  // the last row with indptr <= j
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(m.indptr + mid) <= j)
                lo = mid;
            else
                hi = mid;
        }
        row = lo;
        const int begin = __ldg(m.indptr + row);
        if (j < begin || j >= __ldg(m.indptr + row + 1))
            return nullptr;  // behind the last row's tokens
        at = (int64_t)__ldg(m.seq_lens + row) + j - begin;
    } else {
        at = __ldg(m.seq_lens + row);
    }
    if (at < 0 || at >= (int64_t)m.max_pages * kPage) {
        if (report)
            atomicOr(m.ws_error, kErrSeqLen);
        return nullptr;
    }
    const int page = __ldg(m.block_table + (int64_t)row * m.max_pages + at / kPage);
    if (page < 0 || page >= m.num_pool_pages) {
        if (report)
            atomicOr(m.ws_error, kErrPageId);
        return nullptr;
    }
    slot = (int)(at % kPage);
    return pool + (int64_t)page * stride_page;
}

struct WriteParams {
    TokenMap map;
    const __nv_bfloat16 *k, *v;
    int64_t k_token, k_head, v_token, v_head;  // strides in elements
    uint8_t *pool;
    int64_t stride_page, stride_head;
    int32_t n_tokens, H_kv;
};

struct ReadParams {
    TokenMap map;
    __nv_bfloat16 *k, *v;  // [token][head][D]
    const uint8_t *pool;
    int64_t stride_page, stride_head;
    int32_t n_tokens, H_kv;
};

constexpr int kTokenThreads = 256;

// Both token kernels: D/16 lanes take one row (K or V of a token's head), eight
// dims of two neighbouring scale blocks each; a warp takes 256 / D (token, head)
// items at a time, K and V side by side, ROUNDS times over before it uses the
// first, so that the many small rows keep the memory busy.  Meanwhile one lane per
// item finds its record.
template <int D, int ROUNDS>
struct TokenTile {
    static constexpr int kLanes = D / 16;              // per row
    static constexpr int kHeads = 32 / (2 * kLanes);   // items per round: 2 or 4
    static constexpr int kItems = kHeads * ROUNDS;     // per warp and pass
    static_assert(kItems <= 16, "a lane per item and side");
};

// Lane l and l + 16 look after item base + l: its token and head.
struct TokenItem {
    uint32_t j, head;
    bool mine;
};

template <int D, int ROUNDS>
__device__ __forceinline__ TokenItem item_of_lane(uint32_t base, uint32_t items, uint32_t H_kv, int lane)
{
    const uint32_t item = base + (lane & 15);
    TokenItem t;
    t.j = item / H_kv;
    t.head = item - t.j * H_kv;
    t.mine = (lane & 15) < TokenTile<D, ROUNDS>::kItems && item < items;
    return t;
}

// The item's record with its slot in the low four bits (records are 16-byte
// aligned), 0 as token_record's NULL; in lanes below 16.
__device__ __forceinline__ uint64_t locate_item(const TokenItem &t, const TokenMap &m, const uint8_t *pool,
                                                int64_t stride_page, int64_t stride_head, int lane)
{
    if (!t.mine || lane >= 16)
        return 0;
    int slot = 0;
    const uint8_t *rec = token_record(m, pool, stride_page, (int)t.j, t.head == 0, slot);
    return rec ? (uint64_t)(rec + (int64_t)t.head * stride_head) + (uint32_t)slot : 0;
}

// A lane's place in its row's records.  Its two blocks' codes are two words: of
// K, a block each; of V, a row r = 2c and 2c + 1 each, with two bytes per block.
template <int D>
struct TokenLane {
    int is_v, part, dim;     // K or V, item of the round, first dim (the second block's: + 32)
    int code, gap, scale;    // bytes: codes' first word, to the second; the blocks' two scales
    bool has_scale;
    __device__ __forceinline__ explicit TokenLane(int lane)
    {
        using R = Rec<D>;
        constexpr int kLanes = D / 16;
        const int sub = lane % kLanes, two = sub >> 2, c = sub & 3;
        is_v = (lane / kLanes) & 1;
        part = lane / (2 * kLanes);
        dim = 64 * two + 8 * c;
        code = is_v ? R::kV + 2 * c * (D / 16) + 4 * two : c * (D / 8) + 8 * two;
        gap = is_v ? D / 16 : 4;
        scale = (is_v ? R::kVs : R::kKs) + 2 * two;
        has_scale = c == 0;
    }
    // blocks' codes to words, and words to blocks' codes
    __device__ __forceinline__ void exchange(uint32_t (&w)[2]) const
    {
        const uint32_t low = __byte_perm(w[0], w[1], is_v ? 0x5410 : 0x3210);
        w[1] = __byte_perm(w[0], w[1], is_v ? 0x7632 : 0x7654);
        w[0] = low;
    }
};

// Eight bf16 values to codes and their block's scale byte.  The four lanes of a
// block find its largest magnitude by two shuffles; the scale comes from that
// magnitude's exponent field (its largest value lands in [4, 8) and saturates at 6),
// and the products are by a power of two, exact where the code is not zero.
__device__ __forceinline__ uint32_t quantise(const uint4 &raw, uint32_t &scale)
{
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
    // bf16 magnitudes order like their bits, infinities and NaN above every number
    uint32_t top = __vmaxu2(__vmaxu2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                            __vmaxu2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
    top = max(top & 0xffffu, top >> 16);  // bf16 bits of the block's largest magnitude
    const bool bad = top >= 0x7f80u;      // the block reads back as NaN
    const int s = max((int)(top >> 7) - 2, 1);
    const float mul = __uint_as_float((uint32_t)(254 - s) << 23);  // 2^(127 - s)
    scale = bad ? 255u : top == 0 ? 0u : (uint32_t)s;
    float x[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        x[2 * k] = __uint_as_float(w[k] << 16) * mul;
        x[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u) * mul;
    }
    return bad ? 0u : floats_to_codes(x);
}

// Quantises K and V of the new tokens into their slots: 4 D bytes in, 17 D / 8
// out per token and head.  Two blocks to a lane: with one, the lookups, shuffles
// and addresses took as many instructions as the values (29.0 us against 25.4 for 22983
// tokens of 8 heads, D = 128: now 5.7 TB/s, 88 % of the copy rate).
template <int D, int ROUNDS>
__global__ void __launch_bounds__(kTokenThreads) mx4_write_kernel(const __grid_constant__ WriteParams p)
{
    using R = Rec<D>;
    using T = TokenTile<D, ROUNDS>;
    const int lane = threadIdx.x & 31;
    const TokenLane<D> l(lane);
    const uint32_t items = (uint32_t)p.n_tokens * p.H_kv;  // below 2^31 (checked on the host)
    const __nv_bfloat16 *in = (l.is_v ? p.v : p.k) + l.dim;
    // lanes 16 to 31 work out where the items' values lie, the others where their keys do
    const int64_t in_token = lane < 16 ? p.k_token : p.v_token, in_head = lane < 16 ? p.k_head : p.v_head;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t step = gridDim.x * (kTokenThreads / 32) * T::kItems;
    for (uint32_t base = (blockIdx.x * (kTokenThreads / 32) + threadIdx.x / 32) * T::kItems; base < items; base += step) {
        const TokenItem mine = item_of_lane<D, ROUNDS>(base, items, p.H_kv, lane);
        const long long offset = mine.j * in_token + mine.head * in_head;
        uint4 raw[ROUNDS][2];
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const int at = i * T::kHeads + l.part;
            const __nv_bfloat16 *src = in + __shfl_sync(0xffffffffu, offset, 16 * l.is_v + at);
            raw[i][0] = raw[i][1] = make_uint4(0, 0, 0, 0);
            if (base + at < items) {
                raw[i][0] = __ldg(reinterpret_cast<const uint4 *>(src));
                raw[i][1] = __ldg(reinterpret_cast<const uint4 *>(src + 32));
            }
        }
        const unsigned long long found = locate_item(mine, p.map, p.pool, p.stride_page, p.stride_head, lane);
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const unsigned long long to = __shfl_sync(0xffffffffu, found, i * T::kHeads + l.part);
            uint32_t w[2], scale[2];
#pragma unroll
            for (int k = 0; k < 2; ++k)
                w[k] = quantise(raw[i][k], scale[k]);
            l.exchange(w);
            if (to == 0)
                continue;
            uint8_t *rec = reinterpret_cast<uint8_t *>(to & ~15ull);
            const uint32_t slot = (uint32_t)to & 15u;
            *reinterpret_cast<uint32_t *>(rec + slot * R::kRow + l.code) = w[0];
            *reinterpret_cast<uint32_t *>(rec + slot * R::kRow + l.code + l.gap) = w[1];
            if (l.has_scale)
                *reinterpret_cast<uint16_t *>(rec + slot * R::kScaleRow + l.scale) = (uint16_t)(scale[0] | scale[1] << 8);
        }
    }
}

// A scale byte's value: 2^(s - 127), NaN for 255.
__device__ __forceinline__ float scale_value(uint32_t s)
{
    return __uint_as_float(s == 255u ? 0x7fc00000u : s == 0u ? 0x00400000u : s << 23);
}

// The stored values as bf16, exactly (e2m1 has two significant bits): 25.7 us for
// 22983 tokens of 8 heads, D = 128, 5.6 TB/s.
template <int D, int ROUNDS>
__global__ void __launch_bounds__(kTokenThreads) mx4_read_kernel(const __grid_constant__ ReadParams p)
{
    using R = Rec<D>;
    using T = TokenTile<D, ROUNDS>;
    const int lane = threadIdx.x & 31;
    const TokenLane<D> l(lane);
    const uint32_t items = (uint32_t)p.n_tokens * p.H_kv;  // below 2^31 (checked on the host)
    __nv_bfloat16 *out = (l.is_v ? p.v : p.k) + l.dim;
    grid_dependency_wait();
    grid_launch_dependents();
    const uint32_t step = gridDim.x * (kTokenThreads / 32) * T::kItems;
    for (uint32_t base = (blockIdx.x * (kTokenThreads / 32) + threadIdx.x / 32) * T::kItems; base < items; base += step) {
        const TokenItem mine = item_of_lane<D, ROUNDS>(base, items, p.H_kv, lane);
        const unsigned long long found = locate_item(mine, p.map, p.pool, p.stride_page, p.stride_head, lane);
        uint32_t codes[ROUNDS][2], scales[ROUNDS];
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const unsigned long long from = __shfl_sync(0xffffffffu, found, i * T::kHeads + l.part);
            codes[i][0] = codes[i][1] = 0;  // a skipped token reads as zeros
            scales[i] = 127 | 127 << 8;
            if (from) {
                const uint8_t *rec = reinterpret_cast<const uint8_t *>(from & ~15ull);
                const uint32_t slot = (uint32_t)from & 15u;
                codes[i][0] = *reinterpret_cast<const uint32_t *>(rec + slot * R::kRow + l.code);
                codes[i][1] = *reinterpret_cast<const uint32_t *>(rec + slot * R::kRow + l.code + l.gap);
                scales[i] = *reinterpret_cast<const uint16_t *>(rec + slot * R::kScaleRow + l.scale);
            }
        }
#pragma unroll
        for (int i = 0; i < ROUNDS; ++i) {
            const uint32_t item = base + i * T::kHeads + l.part;
            if (item >= items)
                continue;
            l.exchange(codes[i]);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const float s = scale_value((scales[i] >> (8 * k)) & 255u);
                uint32_t h[4], o[4];
                codes_to_half2(codes[i][k], h);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
                    o[j] = pack_bf16(f.x * s, f.y * s);
                }
                __stcs(reinterpret_cast<uint4 *>(out + (int64_t)item * D + 32 * k), make_uint4(o[0], o[1], o[2], o[3]));
            }
        }
    }
}

// ---------------------------------------------------------------------------
// Decode
//
// The (row, KV head) pairs' pages lie end to end, ceil(N_i / 16) per pair; of
// the U pages in all, block b of T owns [floor(b U / T), floor((b + 1) U / T)) and
// its warps split that share the same way, so every warp streams a
// contiguous run of pages, through as many pairs as it takes, and derives it
// from the device lengths alone: one plan, or one captured graph, serves any
// lengths.
//
// A warp stages its pages itself: each page is one bulk copy (17 D bytes) into
// the warp's own ring, completion on an mbarrier, so warps never wait for one
// another while they stream.  Per page:
//   - S^T = K q^T by mma.sync m16n8k16 on f16 (tokens x heads): e2m1 is exact in f16,
//     q is scaled to f16 by a power of two per head (bf16's eight bits fit).
//     Each scale block's partial products, two k-steps, are multiplied by their
//     tokens' scales in fp32;
//   - the softmax runs in the log2 domain against a reference that moves only
//     when a logit exceeds it by 15 (a warp vote), which after the first pages
//     is rare, so most pages need no shuffles and no rescaling;
//   - O^T += V^T P^T: V's scale multiplies P per block of 32 dims, as an exact power of
//     two on packed halves.  Halves cover 2^-24 .. 2^15, so a block's scales are
//     taken relative to a reference exponent; pages whose scales leave the
//     eight steps below it take the same product in bf16, whose exponents
//     reach everywhere.  Two roundings to halves: 2^-11 of a token's weight, or,
//     for tokens that are 2^-(15 + d) or less of the heaviest (d steps up the window),
//     2^-32 of the heaviest's weight times 6 2^(the window's top - 127).  bf16 would
//     keep their leading bits and cost every other token three of its own; such
//     tokens make up an output only where the heavy ones' values are next to nothing.
// Bound by instruction issue before memory: 263 instructions and 446 cycles
// per page and scheduler, 147 of them on the logic pipe at two cycles each (64 are
// the conversions from e2m1, two values at a time).  One row of 32/8
// heads, D = 128: 262144 tokens 65.4 us (4.36 TB/s of 4-bit pages, 67 % of the copy
// rate), 32768 tokens 18.0 to 19.4 us, of which 9 us are pages and the rest the way to
// the first one and the second kernel.
// A pair within one warp's run is finished by the warp; a pair that spans warps
// is merged in shared memory, one that spans blocks by the kernel that
// follows, always in ascending order: results are deterministic.

constexpr int kMaxRows = 4096;       // rows whose page offsets a block keeps in shared memory
constexpr int kMaxBlocks = 1024;
// A pair's P are 2^(logit - m), with the reference m set kPShift below the
// largest logit; they may grow to 2^kPTop, the top of f16's range, before it
// has to move.  Sums of values between warps and blocks are kept times kPUnit,
// 2^-kPShift, so that they reach no further than the values themselves do.
constexpr float kPShift = 8.f, kPTop = 15.f;
constexpr float kPUnit = 0x1p-8f;

struct DecodeParams {
    const __nv_bfloat16 *q;
    __nv_bfloat16 *out;
    const uint8_t *pool;
    int64_t stride_page, stride_head;
    const int32_t *block_table;
    const int32_t *seq_lens;
    // State slots: 2 b and 2 b + 1 hold block b's first and last pair where they reach into other blocks,
    // 2 T + pair (m and l alone, scored decodes) a pair that one block finished.
    float *ws_m, *ws_l, *ws_acc;
    SlotRange *spans;  // [T]: the slots of the pair that begins in block b and reaches beyond it
    int32_t *span_pair;  // [T]: that pair, or -1
    uint32_t *ws_error;
    float *logits;       // scored decode: [pair][max_pages * P][logit_heads(G)]
    SlotRange *ranges;   // scored decode: every pair's slots
    float scale_log2;
    int32_t B, H_q, H_kv, G, max_pages, num_pool_pages, blocks;
};

// One block per SM.  12 warps: 16 (128 registers, some spilled) took 70.5 us
// and 8 69.5 us where 12 took 64.1 us (32 ragged rows, 1.1 M token-heads, G = 8, with scores).
// The 16-head tile's registers allow 8.
template <int D, int NT>
struct DCfg {
    static constexpr int kWarps = NT == 1 ? 12 : 8;
    static constexpr int kThreads = kWarps * 32;
    static constexpr int kMinPages = NT == 1 ? 32 : 16;  // a smaller share costs more in merging than it saves
    static constexpr int kHeads = 8 * NT;
    static constexpr int kState = kHeads * (D + 4) + 2 * kHeads;  // floats: o (rows padded), m, l
    static constexpr int kStages = D == 128 && NT == 1 ? 2 : 3;  // of two pages each
    static constexpr int kStageBytes = 2 * Rec<D>::kBytes;
    static constexpr int kWarpRing = kStages * kStageBytes;
    static_assert(kState * 4 <= kWarpRing, "a warp's last state takes the place of its ring");
    static constexpr int kFirstOff = kWarps * kWarpRing;  // the states of the warps' first runs
    static constexpr int kBarOff = kFirstOff + kWarps * kState * 4;
    static constexpr int kPairOff = kBarOff + kWarps * kStages * 8;  // pair of each of the 2 kWarps states, and
    static constexpr int kScanOff = kPairOff + 4 * kWarps * 4;       // where the n-th of those present lies
    static constexpr int kWeightOff = kScanOff + 64;                // the block's merge: weights, maxima and sums
    static constexpr int kGroupOff = (kWeightOff + 3 * 16 * 32 * 4 + 15) / 16 * 16;  // its pairs
    static constexpr int kPrefixOff = kGroupOff + 32 * 16;                          // int32 [B + 1]
    static_assert(kWarpRing % 16 == 0 && kBarOff % 8 == 0, "alignment of the copies and their barriers");
    static_assert(kPrefixOff + (kMaxRows + 1) * 4 <= 227 * 1024, "shared memory of a block");
};

// [0, U) in T shares of U / T or one more: share b begins at b (U / T) + min(b, U mod T).
struct Shares {
    uint32_t size, more;
    __device__ Shares(uint32_t U, uint32_t T) : size(U / T), more(U - size * T) {}
    __device__ uint32_t begin(uint32_t b) const { return b * size + min(b, more); }
    __device__ uint32_t owner(uint32_t u) const
    {
        const uint32_t split = more * (size + 1);
        return u < split ? u / (size + 1) : more + (u - split) / size;  // size > 0 wherever u >= split
    }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                        uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi)
{
    const __half2 v = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b)
{
    const __half2 v = __hmul2(*reinterpret_cast<const __half2 *>(&a), *reinterpret_cast<const __half2 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&v);
}

// A warp's running state for one pair: heads 8 nt + 2 c + {0, 1}.  o is in units of
// 2^(vref(b) - 127) for its block b of 32 dims.
template <int D, int NT>
struct State {
    uint32_t qf[D / 16][NT][2];  // q as the MMA's B operand
    float sl[NT][2];             // logit = product * sl (log2 domain)
    uint32_t q_exp;              // byte 2 nt + j: the exponent byte of what undoes a head's scaling of q to f16
    float nb[NT][2];             // -m, minus the reference (log2 domain): P is 2^(logit + nb); FLT_MAX: none yet
    float l[NT][2];
    float o[D / 16][NT][4];
    uint32_t vlow;               // per block the lower end of its window of V's scales, 0 .. 247; ~0: none yet
    // the window's top: the scale in whose units o is
    __device__ int vref(int b) const { return (int)((vlow >> (8 * b)) & 255u) + 7; }
};

template <int D, int NT>
__device__ __forceinline__ void load_q(const DecodeParams &p, int pair, int lane, State<D, NT> &st)
{
    const int r = lane >> 2, c = lane & 3;
    const int row = pair / p.H_kv, h = pair % p.H_kv;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        const int g = nt * 8 + r;
        uint4 raw[D / 32];
        uint32_t amax = 0;
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            raw[b] = make_uint4(0, 0, 0, 0);
            if (g < p.G)
                raw[b] = __ldg(reinterpret_cast<const uint4 *>(
                                   p.q + ((int64_t)row * p.H_q + (int64_t)h * p.G + g) * D + 32 * b) + c);
            const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
                amax = max(amax, max((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
        }
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = max(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        // The largest element to [2^13, 2^14): 2^up and its inverse stay normal floats for |up| <= 126.  Elements keep
        // bf16's eight bits down to 2^-30 of it; smaller ones are rounded to multiples of 2^-38 of it, so a logit is
        // off by at most scale 2^-38 max|q| sum |k|.
        const int e = (int)(amax >> 23);
        const int up = e == 255 ? 0 : min(126, 13 + 127 - e);
        const float mul = __uint_as_float((uint32_t)(127 + up) << 23);
#pragma unroll
        for (int b = 0; b < D / 32; ++b) {
            const uint32_t w[4] = {raw[b].x, raw[b].y, raw[b].z, raw[b].w};
            uint32_t f[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                f[i] = pack_f16(__uint_as_float(w[i] << 16) * mul, __uint_as_float(w[i] & 0xffff0000u) * mul);
            st.qf[2 * b][nt][0] = f[0];
            st.qf[2 * b][nt][1] = f[1];
            st.qf[2 * b + 1][nt][0] = f[2];
            st.qf[2 * b + 1][nt][1] = f[3];
        }
        const float inv = p.scale_log2 * __uint_as_float((uint32_t)(127 - up) << 23);
        st.sl[nt][0] = __shfl_sync(0xffffffffu, inv, 8 * c);
        st.sl[nt][1] = __shfl_sync(0xffffffffu, inv, 8 * c + 4);
        const uint32_t both = (uint32_t)__shfl_sync(0xffffffffu, 127 - up, 8 * c) |
                              (uint32_t)__shfl_sync(0xffffffffu, 127 - up, 8 * c + 4) << 8;
        st.q_exp = nt == 0 ? both : st.q_exp | both << 16;
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        // Any logit but -inf, which has no weight (P = 0, where infinity would make NaN of it), outgrows this reference
        st.nb[nt][0] = st.nb[nt][1] = FLT_MAX;
        st.l[nt][0] = st.l[nt][1] = 0.f;
#pragma unroll
        for (int mt = 0; mt < D / 16; ++mt)
            st.o[mt][nt][0] = st.o[mt][nt][1] = st.o[mt][nt][2] = st.o[mt][nt][3] = 0.f;
    }
    st.vlow = ~0u;
}

// Byte b of w as a float's exponent field: 2^(byte - 127), 0 for 0, infinity
// for 255.  Left shifts as products: the integer multiplier is idle here, the
// logic unit is what bounds the kernel.
__device__ __forceinline__ float exponent_float(uint32_t w, int b)
{
    const uint32_t at = w & (0xffu << (8 * b));
    return __uint_as_float(b == 3 ? at >> 1 : at * (1u << (23 - 8 * b)));
}

// Codes of two tokens, interleaved for the tensor cores: nibble pairs (token
// a's, token b's) of the even dims and of the odd dims.
__device__ __forceinline__ void interleave(uint32_t a, uint32_t b, uint32_t &even, uint32_t &odd)
{
    even = (a & 0x0f0f0f0fu) | ((b * 16u) & 0xf0f0f0f0u);
    odd = ((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u);
}

// D = A * B, m16n8k16, f16 operands, fp32 accumulators.
__device__ __forceinline__ void mma_f16_new(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                            uint32_t b0, uint32_t b1)
{
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%10, %10, %10, %10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.f));
}

// The largest scale byte (255 aside) of block b over the valid tokens, for the whole warp.
__device__ __forceinline__ int top_scale(const uint32_t (&vs)[4], int lane, int nvalid, int b)
{
    int top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int e = (vs[i] >> (8 * b)) & 255;
        if (2 * (lane & 3) + (i & 1) + 4 * (i & 2) < nvalid && e < 255)
            top = max(top, e);
    }
    top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
    return max(top, __shfl_xor_sync(0xffffffffu, top, 2));
}

// S^T = K q^T of one page, each block of 32 dims under its tokens' scales:
// rows are tokens r and r + 8, columns heads 8 nt + 2c and 2c + 1.
// Products carry q's scaling to f16, 2^up, which takes them out of fp32 where
// large keys meet small queries although the logits are ordinary.  WIDE undoes
// an up above 0 before the keys' scales, so that only what K q^T itself cannot
// hold overflows (under an up below 0 the product is the smaller one anyway), and takes a
// scale of 255 for the NaN it is; s are logits then.
template <int D, int NT, bool WIDE>
__device__ __forceinline__ void page_products(const uint8_t *rec, int lane, const State<D, NT> &st, float (&s)[NT][4],
                                              float scale_log2 = 0.f)
{
    using R = Rec<D>;
    constexpr int kBlocks = D / 32;
    const int r = lane >> 2, c = lane & 3;
    uint32_t ka[kBlocks], kb[kBlocks], ksa, ksb;
    if constexpr (D == 128) {
        const uint4 a4 = *reinterpret_cast<const uint4 *>(rec + r * R::kRow + c * 16);
        const uint4 b4 = *reinterpret_cast<const uint4 *>(rec + (r + 8) * R::kRow + c * 16);
        ka[0] = a4.x, ka[1] = a4.y, ka[2] = a4.z, ka[3] = a4.w;
        kb[0] = b4.x, kb[1] = b4.y, kb[2] = b4.z, kb[3] = b4.w;
        ksa = *reinterpret_cast<const uint32_t *>(rec + R::kKs + r * 4);
        ksb = *reinterpret_cast<const uint32_t *>(rec + R::kKs + (r + 8) * 4);
    } else {
        const uint2 a2 = *reinterpret_cast<const uint2 *>(rec + r * R::kRow + c * 8);
        const uint2 b2 = *reinterpret_cast<const uint2 *>(rec + (r + 8) * R::kRow + c * 8);
        ka[0] = a2.x, ka[1] = a2.y;
        kb[0] = b2.x, kb[1] = b2.y;
        ksa = *reinterpret_cast<const uint16_t *>(rec + R::kKs + r * 2);
        ksb = *reinterpret_cast<const uint16_t *>(rec + R::kKs + (r + 8) * 2);
    }
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        uint32_t fa[4], fb[4];
        codes_to_half2(ka[b], fa);
        codes_to_half2(kb[b], fb);
        float sa = exponent_float(ksa, b), sb = exponent_float(ksb, b);
        if (WIDE) {
            sa = fmaf(sa, 0.f, sa);
            sb = fmaf(sb, 0.f, sb);
        }
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float part[4];
            mma_f16_new(part, fa[0], fb[0], fa[1], fb[1], st.qf[2 * b][nt][0], st.qf[2 * b][nt][1]);
            mma_f16(part, fa[2], fb[2], fa[3], fb[3], st.qf[2 * b + 1][nt][0], st.qf[2 * b + 1][nt][1]);
            if (WIDE) {
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    part[i] *= fminf(1.f, exponent_float(st.q_exp, 2 * nt + (i & 1)));
            }
#pragma unroll
            for (int i = 0; i < 4; ++i)
                s[nt][i] = b == 0 ? part[i] * (i < 2 ? sa : sb) : fmaf(part[i], i < 2 ? sa : sb, s[nt][i]);
        }
    }
    if (WIDE) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i)  // rounded before the reference comes off, as the weights kernel has them
                s[nt][i] = __fmul_rn(s[nt][i] * scale_log2, fmaxf(1.f, exponent_float(st.q_exp, 2 * nt + (i & 1))));
    }
}

// V codes of tokens 2c, 2c + 1, 2c + 8, 2c + 9 of a page for dims of row r of
// V^T, two tokens side by side (even dims, odd dims), and the tokens' scales.
template <int D>
__device__ __forceinline__ void load_values(const uint8_t *rec, int lane, uint32_t (&ve)[2][D / 64],
                                            uint32_t (&vo)[2][D / 64])
{
    using R = Rec<D>;
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const uint8_t *a = rec + R::kV + (2 * c + 8 * i) * R::kRow + r * (D / 16);
        if constexpr (D == 128) {
            const uint2 x = *reinterpret_cast<const uint2 *>(a), y = *reinterpret_cast<const uint2 *>(a + R::kRow);
            interleave(x.x, y.x, ve[i][0], vo[i][0]);
            interleave(x.y, y.y, ve[i][1], vo[i][1]);
        } else {
            interleave(*reinterpret_cast<const uint32_t *>(a), *reinterpret_cast<const uint32_t *>(a + R::kRow),
                       ve[i][0], vo[i][0]);
        }
    }
}

template <int D>
__device__ __forceinline__ void load_value_scales(const uint8_t *rec, int lane, uint32_t (&vs)[4])
{
    using R = Rec<D>;
    const int c = lane & 3;
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        const uint8_t *a = rec + R::kVs + (2 * c + 4 * i) * R::kScaleRow;
        if constexpr (D == 128) {
            const uint2 s2 = *reinterpret_cast<const uint2 *>(a);
            vs[i] = s2.x, vs[i + 1] = s2.y;
        } else {
            const uint32_t s2 = *reinterpret_cast<const uint32_t *>(a);
            vs[i] = s2 & 0xffffu, vs[i + 1] = s2 >> 16;
        }
    }
}

// O^T += V^T (P V-scale)^T of one page whose scales lie in their windows, d
// steps (a byte per block) above the lower ends: P times 2^(d - 7) in f16.
template <int D, int NT>
__device__ __forceinline__ void add_values(const uint8_t *rec, int lane, State<D, NT> &st, const float (&pr)[NT][4],
                                           const uint32_t (&d)[4])
{
    uint32_t ve[2][D / 64], vo[2][D / 64], pt[NT][2];
    load_values<D>(rec, lane, ve, vo);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
        pt[nt][0] = movmatrix_trans(pack_f16(pr[nt][0], pr[nt][1]));
        pt[nt][1] = movmatrix_trans(pack_f16(pr[nt][2], pr[nt][3]));
    }
#pragma unroll
    for (int w = 0; w < D / 64; ++w) {
        uint32_t e0[4], o0[4], e1[4], o1[4];
        codes_to_half2(ve[0][w], e0);
        codes_to_half2(vo[0][w], o0);
        codes_to_half2(ve[1][w], e1);
        codes_to_half2(vo[1][w], o1);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int b = 2 * w + k;
            // two tokens' steps of block b as the high bytes of two halves (a byte below 128
            // replicates a zero sign into the low ones), then 2^(step - 7) by its exponent field
            const uint32_t sel = (uint32_t)((8 | b) | b << 4 | (8 | 4 | b) << 8 | (4 | b) << 12);
            uint32_t f0, f1;
            asm("prmt.b32 %0, %1, %2, %3;" : "=r"(f0) : "r"(d[0]), "r"(d[1]), "r"(sel));
            asm("prmt.b32 %0, %1, %2, %3;" : "=r"(f1) : "r"(d[2]), "r"(d[3]), "r"(sel));
            f0 = f0 * 4u + 0x20002000u;
            f1 = f1 * 4u + 0x20002000u;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const uint32_t p0 = mul_f16x2(pt[nt][0], f0), p1 = mul_f16x2(pt[nt][1], f1);
                mma_f16(st.o[2 * b][nt], e0[2 * k], o0[2 * k], e1[2 * k], o1[2 * k], p0, p1);
                mma_f16(st.o[2 * b + 1][nt], e0[2 * k + 1], o0[2 * k + 1], e1[2 * k + 1], o1[2 * k + 1], p0, p1);
            }
        }
    }
}

// The same where some scale lies outside its window.  A larger one moves the
// window up; then bf16 takes the product: e2m1 as f16 bits shifted down by
// three is the same value times 2^-112 in bf16, which P 2^(scale - vref + 112) undoes.
template <int D, int NT>
__device__ __forceinline__ void add_values_wide(const uint8_t *rec, int nvalid, int lane, State<D, NT> &st,
                                                const float (&pr)[NT][4], const uint32_t (&vs)[4])
{
    constexpr int kBlocks = D / 32;
    const int r = lane >> 2;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
        const int top_b = top_scale(vs, lane, nvalid, b);
        if (top_b > st.vref(b)) {
            const int up = top_b - st.vref(b);  // 1 .. 247
            const float f = up > 126 ? 0.f : __uint_as_float((uint32_t)(127 - up) << 23);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    st.o[2 * b][nt][i] *= f;
                    st.o[2 * b + 1][nt][i] *= f;
                }
            st.vlow += (uint32_t)up << (8 * b);
        }
    }
    // this lane's rows of P are tokens r and r + 8: their scales, from a lane that holds them
    const uint32_t even_lo = __shfl_sync(0xffffffffu, vs[0], r >> 1), odd_lo = __shfl_sync(0xffffffffu, vs[1], r >> 1);
    const uint32_t even_hi = __shfl_sync(0xffffffffu, vs[2], r >> 1), odd_hi = __shfl_sync(0xffffffffu, vs[3], r >> 1);
    const uint32_t vs_lo = r & 1 ? odd_lo : even_lo, vs_hi = r & 1 ? odd_hi : even_hi;
    uint32_t ve[2][D / 64], vo[2][D / 64];
    load_values<D>(rec, lane, ve, vo);
#pragma unroll
    for (int w = 0; w < kBlocks / 2; ++w) {
        uint32_t a[4][4];
        codes_to_half2(ve[0][w], a[0]);
        codes_to_half2(vo[0][w], a[1]);
        codes_to_half2(ve[1][w], a[2]);
        codes_to_half2(vo[1][w], a[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                a[i][k] = (a[i][k] & 0x80008000u) | ((a[i][k] >> 3) & 0x0fff0fffu);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int b = 2 * w + k;
            auto factor = [&](uint32_t e, bool ok) {
                const int x = (int)e - st.vref(b) + 254;
                return !ok || x <= 0 || e == 0u ? 0.f
                       : e == 255u              ? __uint_as_float(0x7fc00000u)
                                                : __uint_as_float((uint32_t)x << 23);
            };
            const float f0 = factor((vs_lo >> (8 * b)) & 255u, r < nvalid);
            const float f1 = factor((vs_hi >> (8 * b)) & 255u, r + 8 < nvalid);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                // P reaches 2^15: 2^-15 first, then the factor, up to 2^127
                const float q0 = pr[nt][0] * 0x1p-15f * f0, q1 = pr[nt][1] * 0x1p-15f * f0;
                const float q2 = pr[nt][2] * 0x1p-15f * f1, q3 = pr[nt][3] * 0x1p-15f * f1;
                const uint32_t p0 = movmatrix_trans(pack_bf16(q0, q1)), p1 = movmatrix_trans(pack_bf16(q2, q3));
                mma_bf16(st.o[2 * b][nt], a[0][2 * k], a[1][2 * k], a[2][2 * k], a[3][2 * k], p0, p1);
                mma_bf16(st.o[2 * b + 1][nt], a[0][2 * k + 1], a[1][2 * k + 1], a[2][2 * k + 1], a[3][2 * k + 1], p0,
                         p1);
            }
        }
    }
}

// A product's logit (log2 domain).  An infinite product comes of a NaN scale
// (255), or of factors that page_products<WIDE> keeps in range: + 0 * s makes it
// NaN, which sends its page there.
__device__ __forceinline__ float logit(float s, float sl) { return fmaf(s, 0.f, s * sl); }

// The larger of two numbers, NaN if either is.
__device__ __forceinline__ float max_or_nan(float a, float b)
{
    float y;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
    return y;
}

// Moves the references that the largest of these logits outgrew (x: logits,
// nv[h] valid tokens per page), rescaling the state.  Out of line of the common
// path: a pair's first pages come here, later ones only when a logit grows by
// 2^(kPTop - kPShift).
template <int NT, int D>
__device__ __forceinline__ void move_reference(const float (&x)[2][NT][4], const int (&nv)[2], int lane, State<D, NT> &st)
{
    const int r = lane >> 2;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            float mx = -INFINITY;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int k = 0; k < 2; ++k)
                    if (r + 8 * k < nv[h])
                        mx = fmaxf(mx, x[h][nt][2 * k + j]);
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1)
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
            const float old = -st.nb[nt][j];
            float m = old;
            if (mx - old > kPTop) {
                m = mx - kPShift;
                // where floats are further apart than kPShift (logits of 2^27 and more) that may have rounded too far down
                if (mx - m > kPTop)
                    m = mx;
            }
            const float al = exp2_approx(old - m);
            st.nb[nt][j] = -m;
            st.l[nt][j] *= al;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                st.o[mt][nt][j] *= al;
                st.o[mt][nt][2 + j] *= al;
            }
        }
}

// Two neighbouring pages of a stage (records rec and rec + 17 D) into the
// state, nv[h] valid tokens each (0: not this pair's page; whatever the record
// holds is masked).  Two at once share the votes, the loop and its barriers,
// and give the scheduler independent products.  Masks, a moving reference and
// scales outside their windows are branches that whole pages rarely take.
template <int D, int NT, bool SCORED>
__device__ __forceinline__ void attend_pages(const uint8_t *rec, const int (&nv)[2], int lane, State<D, NT> &st,
                                             float scale_log2, float *logits, int logit_heads)
{
    using R = Rec<D>;
    constexpr int kBlocks = D / 32;
    const int r = lane >> 2, c = lane & 3;
    const bool full = nv[0] == kPage && nv[1] == kPage;
    float x[2][NT][4], t[2][NT][4];  // logits, and above the reference
#pragma unroll
    for (int h = 0; h < 2; ++h)
        page_products<D, NT, true>(rec + h * R::kBytes, lane, st, x[h], scale_log2);
    if constexpr (SCORED) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                const int g = 8 * nt + 2 * c;
                if (g < logit_heads) {
                    float *dst = logits + (h * kPage + r) * logit_heads + g;
                    if (r < nv[h])
                        *reinterpret_cast<float2 *>(dst) = make_float2(x[h][nt][0], x[h][nt][1]);
                    if (r + 8 < nv[h])
                        *reinterpret_cast<float2 *>(dst + 8 * logit_heads) = make_float2(x[h][nt][2], x[h][nt][3]);
                }
            }
    }

    // ---- softmax against the reference max ----
    if (st.vlow == ~0u) {
        // the pair's first pages set each block's window of V's scales, from its first token's
        // (any token's would do: what lies outside takes the wide path)
        uint32_t v[4];
        load_value_scales<D>(rec + (nv[0] > 0 ? 0 : R::kBytes), lane, v);
        const uint32_t first = __shfl_sync(0xffffffffu, v[0], 0);
        st.vlow = 0;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
            st.vlow |= (uint32_t)min(max((int)((first >> (8 * b)) & 255u) - 4, 0), 247) << (8 * b);
    }
#pragma unroll 1
    for (int turn = 0;; ++turn) {  // twice where a reference has to move (from none on the pair's first pages)
        float top = -INFINITY;
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    t[h][nt][i] = x[h][nt][i] + st.nb[nt][i & 1];
                    if (!full && r + (i < 2 ? 0 : 8) >= nv[h])
                        t[h][nt][i] = -INFINITY;
                    top = fmaxf(top, t[h][nt][i]);
                }
        if (turn == 1 || !__any_sync(0xffffffffu, top > kPTop))
            break;
        move_reference(x, nv, lane, st);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[h][nt][i] = exp2_approx(t[h][nt][i]);
            st.l[nt][0] += t[h][nt][0] + t[h][nt][2];
            st.l[nt][1] += t[h][nt][1] + t[h][nt][3];
        }

    // ---- the values ----
    // Steps of the tokens' scales above the windows' lower ends, a byte per
    // block: in their windows iff every byte is 0 .. 7.  (A byte below its
    // window borrows, but is itself at least 256 - 247 then.)
    uint32_t d[2][4], out_of = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        load_value_scales<D>(rec + h * R::kBytes, lane, d[h]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            d[h][i] -= st.vlow;
            if (!full && 2 * c + (i & 1) + 4 * (i & 2) >= nv[h])
                d[h][i] = 0;
            out_of |= d[h][i];
        }
    }
    if (!__any_sync(0xffffffffu, (out_of & 0xf8f8f8f8u) != 0)) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
            add_values<D, NT>(rec + h * R::kBytes, lane, st, t[h], d[h]);
    } else {
#pragma unroll 1
        for (int h = 0; h < 2; ++h) {
            float pr[NT][4];
            uint32_t vs[4];
            load_value_scales<D>(rec + h * R::kBytes, lane, vs);
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                    pr[nt][i] = h ? t[1][nt][i] : t[0][nt][i];
            add_values_wide<D, NT>(rec + h * R::kBytes, h ? nv[1] : nv[0], lane, st, pr, vs);
        }
    }
}

// The same for two whole pages whose logits stay in reach of the reference
// max and whose products and V scales lie in theirs, as nearly all do: no masks, no
// rescaling.  False, with the state unchanged, where they do not.  A path of
// its own saves the predicated masks and lets the loads run further ahead:
// 65.4 us against 70.4 us without it at 262144 tokens (one row, 32/8 heads, D = 128).
template <int D, int NT, bool SCORED>
__device__ __forceinline__ bool attend_whole_pages(const uint8_t *rec, int lane, State<D, NT> &st, float *logits,
                                                   int logit_heads)
{
    using R = Rec<D>;
    const int r = lane >> 2, c = lane & 3;
    float t[2][NT][4], top = -INFINITY;
    uint32_t out_of = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        page_products<D, NT, false>(rec + h * R::kBytes, lane, st, t[h]);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            if constexpr (SCORED) {
                // the weights are worked out from the rounded logits, so P is too
#pragma unroll
                for (int i = 0; i < 4; ++i)
                    t[h][nt][i] = logit(t[h][nt][i], st.sl[nt][i & 1]);
                const int g = 8 * nt + 2 * c;
                if (g < logit_heads) {
                    float *dst = logits + (h * kPage + r) * logit_heads + g;
                    *reinterpret_cast<float2 *>(dst) = make_float2(t[h][nt][0], t[h][nt][1]);
                    *reinterpret_cast<float2 *>(dst + 8 * logit_heads) = make_float2(t[h][nt][2], t[h][nt][3]);
                }
            }
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if constexpr (SCORED)
                    t[h][nt][i] += st.nb[nt][i & 1];
                else
                    t[h][nt][i] = fmaf(t[h][nt][i], 0.f, fmaf(t[h][nt][i], st.sl[nt][i & 1], st.nb[nt][i & 1]));
                top = max_or_nan(top, t[h][nt][i]);
            }
        }
        uint32_t vs[4];
        load_value_scales<D>(rec + h * R::kBytes, lane, vs);
        out_of |= (vs[0] - st.vlow) | (vs[1] - st.vlow) | (vs[2] - st.vlow) | (vs[3] - st.vlow);
    }
    if (__any_sync(0xffffffffu, !(top <= kPTop) || (out_of & 0xf8f8f8f8u) != 0))
        return false;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                t[h][nt][i] = exp2_approx(t[h][nt][i]);
            st.l[nt][0] += t[h][nt][0] + t[h][nt][2];
            st.l[nt][1] += t[h][nt][1] + t[h][nt][3];
        }
        uint32_t d[4];
        load_value_scales<D>(rec + h * R::kBytes, lane, d);
#pragma unroll
        for (int i = 0; i < 4; ++i)
            d[i] -= st.vlow;
        add_values<D, NT>(rec + h * R::kBytes, lane, st, t[h], d);
    }
    return true;
}

// A warp's finished state to shared memory: o [head][D + 4] times kPUnit, m, l per head.
template <int D, int NT>
__device__ __forceinline__ void put_state(float *dst, int lane, const State<D, NT> &st)
{
    using C = DCfg<D, NT>;
    const int r = lane >> 2, c = lane & 3;
    float *dm = dst + C::kHeads * (D + 4), *dl = dm + C::kHeads;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = nt * 8 + 2 * c + j;
            float l = st.l[nt][j];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1)
                l += __shfl_xor_sync(0xffffffffu, l, sh);
            if (r == 0) {
                dm[g] = -st.nb[nt][j];
                dl[g] = l;
            }
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                // kPUnit 2^(vref - 127) in two steps, the exponent byte itself the second
                const float f = __uint_as_float((uint32_t)st.vref(b) << 23);
                *reinterpret_cast<float4 *>(dst + g * (D + 4) + 32 * b + 4 * r) =
                    make_float4(st.o[2 * b][nt][j] * kPUnit * f, st.o[2 * b][nt][2 + j] * kPUnit * f,
                                st.o[2 * b + 1][nt][j] * kPUnit * f, st.o[2 * b + 1][nt][2 + j] * kPUnit * f);
            }
        }
}

// The same state of a pair that this warp alone has seen, normalised and written out.
template <int D, int NT, bool SCORED>
__device__ __forceinline__ void write_pair(const DecodeParams &p, int pair, int lane, const State<D, NT> &st)
{
    const int r = lane >> 2, c = lane & 3;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int g = nt * 8 + 2 * c + j;
            float l = st.l[nt][j];
#pragma unroll
            for (int sh = 4; sh < 32; sh <<= 1)
                l += __shfl_xor_sync(0xffffffffu, l, sh);
            if (g >= p.G)
                continue;
            const float inv = l == 0.f ? 0.f : 1.f / l;
            __nv_bfloat16 *dst = p.out + ((int64_t)pair * p.G + g) * D;
#pragma unroll
            for (int b = 0; b < D / 32; ++b) {
                const float f = __uint_as_float((uint32_t)st.vref(b) << 23);
                store_bf16x4(dst + 32 * b + 4 * r,
                             make_float4(st.o[2 * b][nt][j] * inv * f, st.o[2 * b][nt][2 + j] * inv * f,
                                         st.o[2 * b + 1][nt][j] * inv * f, st.o[2 * b + 1][nt][2 + j] * inv * f));
            }
            if (SCORED && r == 0) {
                const int64_t at = (int64_t)(2 * p.blocks + pair) * p.G + g;
                p.ws_m[at] = -st.nb[nt][j];
                p.ws_l[at] = l;
                if (g == 0)
                    p.ranges[pair] = SlotRange{2 * p.blocks + pair, 1, 0, 0};
            }
        }
}

template <int D, int NT, bool SCORED>
__global__ void __launch_bounds__(DCfg<D, NT>::kThreads, 1) mx4_decode_kernel(const __grid_constant__ DecodeParams p)
{
    using C = DCfg<D, NT>;
    using R = Rec<D>;
    constexpr int kWarps = C::kWarps, kThreads = C::kThreads;
    extern __shared__ __align__(128) uint8_t smem[];
    int32_t *state_pair = reinterpret_cast<int32_t *>(smem + C::kPairOff);
    int32_t *scan = reinterpret_cast<int32_t *>(smem + C::kScanOff);
    int32_t *prefix = reinterpret_cast<int32_t *>(smem + C::kPrefixOff);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int64_t capacity = (int64_t)p.max_pages * kPage;
    uint8_t *ring = smem + warp * C::kWarpRing;
    const uint32_t ring_addr = smem_addr(ring);
    const uint32_t bars = smem_addr(smem + C::kBarOff) + warp * C::kStages * 8;
    if (lane == 0) {
        for (int s = 0; s < C::kStages; ++s)
            mbar_init(bars + 8 * s, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (tid < 2 * kWarps)
        state_pair[tid] = -1;
    grid_dependency_wait();

    // ---- page offsets of the rows ----
    auto row_len = [&](int row, bool report) {
        const int n = __ldg(p.seq_lens + row);
        if (n >= 0 && n <= capacity)
            return n;
        if (report)
            atomicOr(p.ws_error, kErrSeqLen);
        return n < 0 ? 0 : (int)capacity;
    };
    if (tid == 0)
        prefix[0] = 0;
    int carry = 0;
    for (int base = 0; base < p.B; base += kThreads) {
        const int row = base + tid;
        int v = row < p.B ? (row_len(row, blockIdx.x == 0) + kPage - 1) / kPage : 0;
        for (int o = 1; o < 32; o <<= 1) {
            const int up = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += up;
        }
        if (lane == 31)
            scan[warp] = v;
        __syncthreads();
        int add = carry;
        for (int w = 0; w < kWarps; ++w) {
            if (w < warp)
                add += scan[w];
            carry += scan[w];
        }
        if (row < p.B)
            prefix[row + 1] = v + add;
        __syncthreads();
    }
    const uint32_t U = (uint32_t)carry * p.H_kv;  // below 2^31 (checked on the host)
    // rows without tokens have no pages: their zeros are dealt out by row
    for (int row = blockIdx.x; row < p.B; row += p.blocks) {
        if (prefix[row + 1] != prefix[row])
            continue;
        uint4 *dst = reinterpret_cast<uint4 *>(p.out + (int64_t)row * p.H_q * D);
        for (int i = tid; i < p.H_q * D / 8; i += kThreads)
            dst[i] = make_uint4(0, 0, 0, 0);
    }
    const uint32_t T = max(1u, min((uint32_t)p.blocks, (U + C::kMinPages - 1) / C::kMinPages));
    if (tid == 0)
        p.span_pair[blockIdx.x] = -1;
    if (blockIdx.x >= T || U == 0)
        return;
    const Shares blocks(U, T);
    const uint32_t u0 = blocks.begin(blockIdx.x), u1 = blocks.begin(blockIdx.x + 1);
    const Shares warps(u1 - u0, kWarps);
    const uint32_t w0 = u0 + warps.begin(warp);
    const int n = (int)(warps.begin(warp + 1) - warps.begin(warp));

    // ---- stream this warp's pages ----
    // lane l holds page 32 k + l of batch k of them: where it lies, for this batch and the next
    const uint8_t *cur_src = nullptr, *next_src = nullptr;
    int cur_pair = -1, next_pair = -1, first_index = 0;
    auto locate = [&](int j, const uint8_t *&src, int &pair) {
        if (j >= n)
            return;
        const uint32_t u = w0 + j;
        int lo = 0, hi = p.B;  // the last row that begins at or before u
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if ((uint32_t)prefix[mid] * p.H_kv <= u)
                lo = mid;
            else
                hi = mid;
        }
        const uint32_t pages = prefix[lo + 1] - prefix[lo];
        const uint32_t in = u - (uint32_t)prefix[lo] * p.H_kv;
        const uint32_t head = in / pages, index = in - head * pages;
        if (j == 0)
            first_index = (int)index;
        pair = lo * p.H_kv + (int)head;
        int phys = __ldg(p.block_table + (int64_t)lo * p.max_pages + index);
        if (phys < 0 || phys >= p.num_pool_pages) {
            atomicOr(p.ws_error, kErrPageId);
            phys = 0;  // read a real page instead; the error bit reports the bad entry
        }
        src = p.pool + (int64_t)phys * p.stride_page + (int64_t)head * p.stride_head;
    };
    // stage s: pages 2 k and 2 k + 1 (the last stage may hold one), each copied by the lane that holds it
    auto issue = [&](const uint8_t *src, int j, int s) {
        if ((j & 1) == 0)
            mbar_expect_tx(bars + 8 * s, j + 1 < n ? C::kStageBytes : R::kBytes);
        bulk_g2s(ring_addr + s * C::kStageBytes + (j & 1) * R::kBytes, src, R::kBytes, bars + 8 * s);
    };
    locate(lane, cur_src, cur_pair);
    __syncwarp();  // the barriers' initialisation
    if (lane < 2 * C::kStages && lane < n)
        issue(cur_src, lane, lane >> 1);
    if (n > 32)
        locate(32 + lane, next_src, next_pair);
    first_index = __shfl_sync(0xffffffffu, first_index, 0);

    // A run of pages that is its whole pair is written out at once; one that the
    // warp's share cuts becomes a state: the warp's first run beside the rings (in
    // use until the warp is done), its last one in the warp's own ring.
    auto state_at = [&](int i) {  // state i = 2 * warp + (0 first, 1 last)
        return reinterpret_cast<float *>(i & 1 ? smem + (i >> 1) * C::kWarpRing
                                               : smem + C::kFirstOff + (i >> 1) * C::kState * 4);
    };
    State<D, NT> st;
    int stage = 0, phase = 0;
    bool ok = true;
    for (int j = 0; j < n && ok;) {  // a pair's run of pages
        const int pair = __shfl_sync(0xffffffffu, cur_pair, j & 31);
        const int row = pair / p.H_kv;
        const int len = row_len(row, false);
        const int pages = prefix[row + 1] - prefix[row];
        const int begin = j == 0 ? first_index : 0;
        const int end = min(pages, begin + n - j);
        const int run = j;
        load_q<D, NT>(p, pair, lane, st);
        for (int index = begin; index < end;) {
            // the stage's first page is index - at; one that begins inside a stage finds it landed already
            const int at = j & 1;
            if (at == 0 || j == run) {
                const uint32_t bar = bars + 8 * stage;
                if (!mbar_try_wait(bar, phase))
                    ok = mbar_wait(bar, phase, p.ws_error);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) {
                    // give up on the pair, but not before the copies in flight had their time to land
                    for (int k = 1; k < C::kStages && (j & ~1) + 2 * k < n; ++k) {
                        stage = stage + 1 == C::kStages ? 0 : stage + 1;
                        phase ^= stage == 0;
                        mbar_wait(bars + 8 * stage, phase, p.ws_error);
                    }
                    break;
                }
            }
            const int take = min(2 - at, end - index);
            const int tokens = len - index * kPage;  // left in the row
            const int nv[2] = {at ? 0 : min(kPage, tokens),
                               at ? min(kPage, tokens) : take == 2 ? min(kPage, tokens - kPage) : 0};
            float *logits = nullptr;
            int heads = 0;
            if constexpr (SCORED) {
                heads = p.G <= 2 ? 2 : p.G <= 4 ? 4 : p.G <= 8 ? 8 : 16;  // logit_heads(G)
                logits = p.logits + ((int64_t)pair * capacity + (int64_t)(index - at) * kPage) * heads;
            }
            const uint8_t *rec = ring + stage * C::kStageBytes;
            if (nv[0] < kPage || nv[1] < kPage || st.vlow == ~0u ||
                !attend_whole_pages<D, NT, SCORED>(rec, lane, st, logits, heads))
                attend_pages<D, NT, SCORED>(rec, nv, lane, st, p.scale_log2, logits, heads);
            index += take;
            j += take;
            if ((j & 1) && j < n)
                continue;  // the stage's second page is another pair's
            __syncwarp();
            // the pages that take this stage's place
            const int k = ((j + 1) & ~1) + 2 * (C::kStages - 1);
            if ((lane & ~1) == (k & 31) && k + (lane & 1) < n)
                issue(((k ^ (j - 1)) & ~31) == 0 ? cur_src : next_src, k + (lane & 1), stage);
            stage = stage + 1 == C::kStages ? 0 : stage + 1;
            phase ^= stage == 0;
            if ((j & 31) == 0) {
                cur_src = next_src;
                cur_pair = next_pair;
                locate(j + 32 + lane, next_src, next_pair);
            }
        }
        if (!ok)
            break;
        if (begin == 0 && end == pages) {
            write_pair<D, NT, SCORED>(p, pair, lane, st);
        } else {
            // the first run where it is not whole begins this warp's share; any other reaches its end
            const int i = 2 * warp + (run > 0 ? 1 : 0);
            put_state<D, NT>(state_at(i), lane, st);
            if (lane == 0)
                state_pair[i] = pair;
        }
    }
    grid_launch_dependents();
    __syncthreads();

    // ---- merge the states of pairs that the warps share ----
    // Lane k of every warp looks at state k: which are there, and where a new
    // pair begins among them (the states of one pair are neighbours).
    constexpr int D4 = D / 4;
    const int G = p.G;
    float *weight = reinterpret_cast<float *>(smem + C::kWeightOff);  // [head][n-th state]
    float *pair_m = weight + 16 * 32, *pair_l = pair_m + 16 * 32;     // [head][n-th state, a pair's first]
    const int my_pair = lane < 2 * kWarps ? state_pair[lane] : -1;
    const uint32_t there = __ballot_sync(0xffffffffu, my_pair >= 0);
    if (there == 0)
        return;
    const uint32_t below = (1u << lane) - 1u;
    const int before = 31 - __clz(there & below);  // the state before this one, or -1
    const int pair_before = __shfl_sync(0xffffffffu, my_pair, before & 31);
    const uint32_t starts = __ballot_sync(0xffffffffu, my_pair >= 0 && (before < 0 || pair_before != my_pair));
    const int nth = __popc(there & below);
    // the states of the pair that begins with state `first`: the n-th to the one before `end`
    auto end_of = [&](int first) {
        const uint32_t later = starts & ~((2u << first) - 1u);
        return __popc(later ? there & ((later & (0u - later)) - 1u) : there);
    };
    const int groups = __popc(starts), group = __popc(starts & below);  // pairs among the states; this lane's, at its start
    // Per pair: {pair, its first state's number, one past its last, state slot}
    int4 *group_at = reinterpret_cast<int4 *>(smem + C::kGroupOff);
    if (warp == 0 && (starts >> lane) & 1u) {
        const int row = my_pair / p.H_kv;
        const uint32_t pages = prefix[row + 1] - prefix[row];
        const uint32_t P0 = (uint32_t)prefix[row] * p.H_kv + (uint32_t)(my_pair - row * p.H_kv) * pages;
        const bool whole = P0 >= u0 && P0 + pages <= u1;
        const int slot = whole ? 2 * p.blocks + my_pair : 2 * (int)blockIdx.x + (P0 > u0 ? 1 : 0);
        group_at[group] = make_int4(my_pair, nth, end_of(lane), slot);
        if (P0 >= u0 && P0 + pages > u1) {
            // the pair begins here and reaches beyond this block
            const SlotRange span{slot, (int)(blocks.owner(P0 + pages - 1) - blockIdx.x) + 1, 2 * (int)blockIdx.x, 2};
            p.spans[blockIdx.x] = span;
            p.span_pair[blockIdx.x] = my_pair;
            if (SCORED)
                p.ranges[my_pair] = span;
        }
        if (SCORED && whole)
            p.ranges[my_pair] = SlotRange{slot, 1, 0, 0};
    }
    if (warp == kWarps - 1 && my_pair >= 0)
        state_pair[2 * kWarps + nth] = (int)(state_at(lane) - reinterpret_cast<float *>(smem));  // where the n-th lies
    // weights: a warp per (head, pair)
    for (int w = warp; w < G * groups; w += kWarps) {
        const int g = w % G, which = w / G;
        const int first = __ffs(__ballot_sync(0xffffffffu, ((starts >> lane) & 1u) != 0 && group == which)) - 1;
        const bool mine = my_pair >= 0 && lane >= first && nth < end_of(first);
        const float *sk = state_at(lane) + C::kHeads * (D + 4) + g;
        const float m = mine ? sk[0] : -INFINITY, l = mine ? sk[C::kHeads] : 0.f;
        float M = m;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
        const float wt = exp2_approx(m - (M == -INFINITY ? 0.f : M));
        float L = mine ? l * wt : 0.f;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            L += __shfl_xor_sync(0xffffffffu, L, o);
        if (mine)
            weight[g * 32 + nth] = wt;
        if (lane == first) {
            pair_m[g * 32 + nth] = M;
            pair_l[g * 32 + nth] = L;
        }
    }
    __syncthreads();
    for (int e = tid; e < groups * G * D4; e += kThreads) {
        const int column = e / D4, d4 = (e % D4) * 4;
        const int which = column / G, g = column - which * G;
        const int4 at = group_at[which];
        const float *col = reinterpret_cast<float *>(smem) + g * (D + 4) + d4;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
        for (int k = at.y; k < at.z; ++k)
            O = fma4(*reinterpret_cast<const float4 *>(col + state_pair[2 * kWarps + k]), weight[g * 32 + k], O);
        const float L = pair_l[g * 32 + at.y];
        const bool whole = at.w >= 2 * p.blocks;
        const int64_t to = (int64_t)at.w * G + g;
        if (whole)
            store_bf16x4(p.out + ((int64_t)at.x * G + g) * D + d4, scale4(O, L == 0.f ? 0.f : 1.f / kPUnit / L));
        else
            *reinterpret_cast<float4 *>(p.ws_acc + to * D + d4) = O;
        if (d4 == 0 && (SCORED || !whole)) {
            p.ws_m[to] = pair_m[g * 32 + at.y];
            p.ws_l[to] = L;
        }
    }
}

// ---------------------------------------------------------------------------
// What follows the decode kernel: one block per (decode block, head) merges the
// pair that begins there and reaches beyond, in ascending order of its blocks;
// with scores, further blocks add the weights.  A launch of its own costs less
// than letting the last of a pair's blocks merge: the tickets alone took that
// kernel 1.3 us, and the merges ran one after another on one SM.

constexpr int kFinishThreads = 256;
static_assert(kFinishThreads == kWeightThreads, "one grid runs both");

struct FinishParams {
    WeightParams w;  // m, l, G; the rest for scores
    const float *acc;
    const SlotRange *spans;
    const int32_t *span_pair;
    __nv_bfloat16 *out;
    int32_t blocks, chunks;
};

// LH = logit_heads(G), 0: no scores.
template <int D, int LH>
__global__ void __launch_bounds__(kFinishThreads) mx4_finish_kernel(const __grid_constant__ FinishParams p)
{
    constexpr int D4 = D / 4, kParts = kFinishThreads / D4;
    __shared__ float4 s_o[kParts][D4];
    __shared__ float s_m[LH > 0 ? LH : 1], s_inv[LH > 0 ? LH : 1];
    const int G = p.w.G;
    grid_dependency_wait();
    grid_launch_dependents();
    if (LH > 0 && (int)blockIdx.x >= p.blocks * G) {
        const int i = blockIdx.x - p.blocks * G;
        add_weights<(LH > 0 ? LH : 2), false>(p.w, i / p.chunks, i % p.chunks, s_m, s_inv, nullptr);
        return;
    }
    const int b = blockIdx.x / G, g = blockIdx.x % G;
    const SlotRange span = p.spans[b];
    const int pair = __ldcg(p.span_pair + b);
    if (pair < 0)
        return;
    const int lane = threadIdx.x & 31, col = threadIdx.x % D4, part = threadIdx.x / D4;
    const int i0 = span.count * part / kParts, i1 = span.count * (part + 1) / kParts;
    // this thread's first states load while the weights are worked out
    constexpr int kAhead = 4;
    float4 ahead[kAhead];
    float m_ahead[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (i0 + k < i1) {
            ahead[k] = __ldcg(reinterpret_cast<const float4 *>(p.acc + (span.slot(i0 + k) * G + g) * D) + col);
            m_ahead[k] = __ldcg(p.w.m + span.slot(i0 + k) * G + g);
        }
    float m0 = -INFINITY, l0 = 0.f;
    if (lane < span.count) {
        m0 = __ldcg(p.w.m + span.slot(lane) * G + g);
        l0 = __ldcg(p.w.l + span.slot(lane) * G + g);
    }
    float M = m0;
    for (int i = lane + 32; i < span.count; i += 32)
        M = fmaxf(M, __ldcg(p.w.m + span.slot(i) * G + g));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    M = M == -INFINITY ? 0.f : M;
    float L = l0 * exp2_approx(m0 - M);
    for (int i = lane + 32; i < span.count; i += 32)
        L = fmaf(__ldcg(p.w.l + span.slot(i) * G + g), exp2_approx(__ldcg(p.w.m + span.slot(i) * G + g) - M), L);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        L += __shfl_xor_sync(0xffffffffu, L, o);
    float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int k = 0; k < kAhead; ++k)
        if (i0 + k < i1)
            O = fma4(ahead[k], exp2_approx(m_ahead[k] - M), O);
    for (int i = i0 + kAhead; i < i1; ++i)
        O = fma4(__ldcg(reinterpret_cast<const float4 *>(p.acc + (span.slot(i) * G + g) * D) + col),
                 exp2_approx(__ldcg(p.w.m + span.slot(i) * G + g) - M), O);
    s_o[part][col] = O;
    __syncthreads();
    if (part != 0)
        return;
#pragma unroll
    for (int k = 1; k < kParts; ++k)
        O = fma4(s_o[k][col], 1.f, O);
    store_bf16x4(p.out + ((int64_t)pair * G + g) * D + col * 4, scale4(O, L == 0.f ? 0.f : 1.f / kPUnit / L));
}

// ---------------------------------------------------------------------------
// Host side

// Workspace of a 4-bit decode plan: the error word, the blocks' states and
// spans and, with PKV_FLAG_SCORES, the pairs' slots and the logits.
struct Mx4Layout {
    size_t m_off, l_off, acc_off, spans_off, span_pair_off, ranges_off, logits_off, total;
    int64_t n_slots;
};

Mx4Layout mx4_layout(const pkv_shape &s, const pkv_plan &p)
{
    Mx4Layout w{};
    const bool scores = (p.flags & PKV_FLAG_SCORES) != 0;
    const size_t pairs = (size_t)s.B * s.H_kv, G = (size_t)(s.H_q / s.H_kv), T = (size_t)p.num_splits;
    w.n_slots = (int64_t)(2 * T + (scores ? pairs : 0));
    size_t off = kWsAlign;
    auto take = [&](size_t bytes) {
        const size_t at = off;
        off += round_up(bytes, kWsAlign);
        return at;
    };
    w.m_off = take((size_t)w.n_slots * G * 4);
    w.l_off = take((size_t)w.n_slots * G * 4);
    w.acc_off = take(2 * T * G * s.head_dim * 4);
    w.spans_off = take(T * sizeof(SlotRange));
    w.span_pair_off = take(T * 4);
    if (scores) {
        w.ranges_off = take(pairs * sizeof(SlotRange));
        w.logits_off = take(pairs * s.max_pages_per_seq * s.page_size * logit_heads((int64_t)G) * 4);
    }
    w.total = off;
    return w;
}

int check_mx4(const pkv_shape &s)
{
    if (s.page_size != kPage || (s.head_dim != 64 && s.head_dim != 128))
        return PKV_ERR_UNSUPPORTED;
    if (s.kv_stride_page <= 0 || s.kv_stride_head <= 0 || s.kv_stride_page % 16 || s.kv_stride_head % 16)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

int check_mx4_plan(const pkv_plan *p)
{
    if (!p || p->mode != PKV_BALANCED || p->num_splits < 1 || p->chunk_pages != 0)
        return PKV_ERR_INVALID;
    if (p->num_splits > kMaxBlocks || (p->flags & ~(PKV_FLAG_SCORES | PKV_FLAG_NO_PDL)))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

template <int D, int NT, bool SCORED>
cudaError_t launch_mx4(const DecodeParams &p, cudaStream_t st, bool pdl)
{
    using C = DCfg<D, NT>;
    auto kernel = mx4_decode_kernel<D, NT, SCORED>;
    const size_t smem = (size_t)C::kPrefixOff + (size_t)(p.B + 1) * 4;
    static std::atomic<uint64_t> configured{0};
    const cudaError_t e = allow_smem(kernel, 227 * 1024, configured);
    if (e != cudaSuccess)
        return e;
    return launch_kernel(kernel, (unsigned)p.blocks, C::kThreads, smem, st, pdl, p);
}

template <int D>
cudaError_t launch_decode(const DecodeParams &p, bool scores, cudaStream_t st, bool pdl)
{
    if (p.G <= 8)
        return scores ? launch_mx4<D, 1, true>(p, st, pdl) : launch_mx4<D, 1, false>(p, st, pdl);
    return scores ? launch_mx4<D, 2, true>(p, st, pdl) : launch_mx4<D, 2, false>(p, st, pdl);
}

template <int D>
cudaError_t launch_finish(const FinishParams &p, bool scores, int64_t grid, cudaStream_t st, bool pdl)
{
    const unsigned n = (unsigned)grid;
    switch (scores ? logit_heads(p.w.G) : 0) {
    case 0: return launch_kernel(mx4_finish_kernel<D, 0>, n, kFinishThreads, 0, st, pdl, p);
    case 2: return launch_kernel(mx4_finish_kernel<D, 2>, n, kFinishThreads, 0, st, pdl, p);
    case 4: return launch_kernel(mx4_finish_kernel<D, 4>, n, kFinishThreads, 0, st, pdl, p);
    case 8: return launch_kernel(mx4_finish_kernel<D, 8>, n, kFinishThreads, 0, st, pdl, p);
    default: return launch_kernel(mx4_finish_kernel<D, 16>, n, kFinishThreads, 0, st, pdl, p);
    }
}

// Pages below which a decode of this tile is one block's: nothing to merge.
int min_pages(int G) { return G <= 8 ? DCfg<128, 1>::kMinPages : DCfg<128, 2>::kMinPages; }

// Rounds of a token kernel: four (enough rows in flight to stream) where one
// would fill three quarters of a full GPU's warps, else one, for the shortest way
// through a few tokens.  Quantising tokens of 8 heads, D = 128, one round against
// four: 1024 tokens 3.1 and 3.4 us, 2048 tokens 4.4 and 4.1, 22983 tokens 30.9 and 25.4.
constexpr int kManyRounds = 4;
constexpr int kTokenBlocks = 148 * 8;  // of 256 threads: a full GPU

bool many_rounds(int64_t rounds) { return rounds >= (int64_t)kTokenBlocks * (kTokenThreads / 32) * 3 / 4; }

template <typename P>
cudaError_t launch_tokens(void (*many)(P), void (*few)(P), int heads, const P &p, cudaStream_t st)
{
    const int64_t items = (int64_t)p.n_tokens * p.H_kv;
    const bool m = many_rounds(ceil_div(items, (int64_t)heads));
    const int64_t blocks = ceil_div(items, (int64_t)heads * (m ? kManyRounds : 1) * (kTokenThreads / 32));
    return launch_kernel(m ? many : few, (unsigned)std::min<int64_t>(blocks, kTokenBlocks), kTokenThreads, 0, st, true, p);
}

int check_tokens(const pkv_shape *shape, const void *pool, const int32_t *block_table, const int32_t *seq_lens,
                 const int32_t *indptr, int32_t n_tokens, const void *workspace)
{
    if (check_shape(shape) != PKV_OK || n_tokens < 0)
        return PKV_ERR_INVALID;
    const int rc = check_mx4(*shape);
    if (rc != PKV_OK)
        return rc;
    if (n_tokens == 0 || shape->B == 0)
        return n_tokens == 0 ? PKV_OK : PKV_ERR_INVALID;
    if (!pool || !block_table || !seq_lens || !workspace || shape->max_pages_per_seq < 1 || shape->num_pool_pages < 1 ||
        (!indptr && n_tokens != shape->B))
        return PKV_ERR_INVALID;
    if ((int64_t)n_tokens * shape->H_kv > INT32_MAX / 2)
        return PKV_ERR_UNSUPPORTED;
    if (!aligned(pool, 16) || !aligned(block_table, 4) || !aligned(seq_lens, 4) || !aligned(indptr, 4) ||
        !aligned(workspace, 4))
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

}  // namespace

}  // namespace pkv

using namespace pkv;

extern "C" {

int pkv_mx4_append(const void *k, const void *v, int64_t k_stride_token, int64_t k_stride_head, int64_t v_stride_token,
                   int64_t v_stride_head, void *pool, const int32_t *block_table, const int32_t *seq_lens,
                   const int32_t *indptr, int32_t n_tokens, const pkv_shape *shape, void *workspace, void *stream)
{
    const int rc = check_tokens(shape, pool, block_table, seq_lens, indptr, n_tokens, workspace);
    if (rc != PKV_OK || n_tokens == 0)
        return rc;
    if (!k || !v)
        return PKV_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16) || (k_stride_token | k_stride_head | v_stride_token | v_stride_head) % 8 ||
        k_stride_token < 0 || k_stride_head < 0 || v_stride_token < 0 || v_stride_head < 0)
        return PKV_ERR_UNSUPPORTED;
    const pkv_shape &s = *shape;
    WriteParams p{};
    p.map = {block_table, seq_lens, indptr, static_cast<uint32_t *>(workspace), s.B, s.max_pages_per_seq, s.num_pool_pages};
    p.k = static_cast<const __nv_bfloat16 *>(k);
    p.v = static_cast<const __nv_bfloat16 *>(v);
    p.k_token = k_stride_token;
    p.k_head = k_stride_head;
    p.v_token = v_stride_token;
    p.v_head = v_stride_head;
    p.pool = static_cast<uint8_t *>(pool);
    p.stride_page = s.kv_stride_page;
    p.stride_head = s.kv_stride_head;
    p.n_tokens = n_tokens;
    p.H_kv = s.H_kv;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = s.head_dim == 128
                              ? launch_tokens(mx4_write_kernel<128, kManyRounds>, mx4_write_kernel<128, 1>, 2, p, st)
                              : launch_tokens(mx4_write_kernel<64, kManyRounds>, mx4_write_kernel<64, 1>, 4, p, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int pkv_mx4_read(const void *pool, const int32_t *block_table, const int32_t *seq_lens, const int32_t *indptr,
                 int32_t n_tokens, void *k, void *v, const pkv_shape *shape, void *workspace, void *stream)
{
    const int rc = check_tokens(shape, pool, block_table, seq_lens, indptr, n_tokens, workspace);
    if (rc != PKV_OK || n_tokens == 0)
        return rc;
    if (!k || !v)
        return PKV_ERR_INVALID;
    if (!aligned(k, 16) || !aligned(v, 16))
        return PKV_ERR_UNSUPPORTED;
    const pkv_shape &s = *shape;
    ReadParams p{};
    p.map = {block_table, seq_lens, indptr, static_cast<uint32_t *>(workspace), s.B, s.max_pages_per_seq, s.num_pool_pages};
    p.k = static_cast<__nv_bfloat16 *>(k);
    p.v = static_cast<__nv_bfloat16 *>(v);
    p.pool = static_cast<const uint8_t *>(pool);
    p.stride_page = s.kv_stride_page;
    p.stride_head = s.kv_stride_head;
    p.n_tokens = n_tokens;
    p.H_kv = s.H_kv;
    const cudaStream_t st = (cudaStream_t)stream;
    const cudaError_t e = s.head_dim == 128
                              ? launch_tokens(mx4_read_kernel<128, kManyRounds>, mx4_read_kernel<128, 1>, 2, p, st)
                              : launch_tokens(mx4_read_kernel<64, kManyRounds>, mx4_read_kernel<64, 1>, 4, p, st);
    return e == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

int pkv_mx4_workspace_bytes(const pkv_shape *shape, const pkv_plan *plan, size_t *bytes)
{
    if (!bytes || check_shape(shape) != PKV_OK)
        return PKV_ERR_INVALID;
    const int rc = check_mx4_plan(plan);
    if (rc != PKV_OK)
        return rc;
    *bytes = mx4_layout(*shape, *plan).total;
    return PKV_OK;
}

int pkv_mx4_decode(const void *q, const void *pool, const int32_t *block_table, const int32_t *seq_lens,
                   int32_t page_size, float scale, void *out, float *scores, int64_t score_stride_row,
                   int64_t score_stride_head, const pkv_shape *shape, const pkv_plan *plan, void *workspace,
                   size_t workspace_bytes, void *stream)
{
    if (check_shape(shape) != PKV_OK || page_size != shape->page_size)
        return PKV_ERR_INVALID;
    int rc = check_mx4_plan(plan);
    if (rc != PKV_OK)
        return rc;
    const pkv_shape &s = *shape;
    if ((rc = check_mx4(s)) != PKV_OK)
        return rc;
    const int G = s.H_q / s.H_kv;
    const int64_t pairs = (int64_t)s.B * s.H_kv, capacity = (int64_t)s.max_pages_per_seq * kPage;
    if (G < 1 || G > 16 || s.B > kMaxRows || pairs * s.max_pages_per_seq > INT32_MAX || capacity > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    // a plan's scores flag sizes its workspace: it goes with scores, and only with them
    if (((plan->flags & PKV_FLAG_SCORES) != 0) != (scores != nullptr))
        return PKV_ERR_UNSUPPORTED;
    if (s.B == 0)
        return PKV_OK;
    if (!q || !pool || !block_table || !seq_lens || !out || !workspace || s.max_pages_per_seq < 1 ||
        s.num_pool_pages < 1)
        return PKV_ERR_INVALID;
    if (!aligned(q, 16) || !aligned(out, 16) || !aligned(pool, 16) || !aligned(block_table, 4) ||
        !aligned(seq_lens, 4) || !aligned(scores, 4) || !aligned(workspace, 256))
        return PKV_ERR_UNSUPPORTED;
    const int64_t merges = (int64_t)plan->num_splits * G;
    if (scores && weight_blocks(pairs, capacity) + merges > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    const Mx4Layout w = mx4_layout(s, *plan);
    if (workspace_bytes < w.total)
        return PKV_ERR_CAPACITY;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    DecodeParams p{};
    p.q = static_cast<const __nv_bfloat16 *>(q);
    p.out = static_cast<__nv_bfloat16 *>(out);
    p.pool = static_cast<const uint8_t *>(pool);
    p.stride_page = s.kv_stride_page;
    p.stride_head = s.kv_stride_head;
    p.block_table = block_table;
    p.seq_lens = seq_lens;
    p.ws_error = reinterpret_cast<uint32_t *>(ws);
    p.ws_m = reinterpret_cast<float *>(ws + w.m_off);
    p.ws_l = reinterpret_cast<float *>(ws + w.l_off);
    p.ws_acc = reinterpret_cast<float *>(ws + w.acc_off);
    p.spans = reinterpret_cast<SlotRange *>(ws + w.spans_off);
    p.span_pair = reinterpret_cast<int32_t *>(ws + w.span_pair_off);
    p.scale_log2 = scale * 1.4426950408889634f;
    p.B = s.B;
    p.H_q = s.H_q;
    p.H_kv = s.H_kv;
    p.G = G;
    p.max_pages = s.max_pages_per_seq;
    p.num_pool_pages = s.num_pool_pages;
    p.blocks = plan->num_splits;
    if (scores) {
        p.ranges = reinterpret_cast<SlotRange *>(ws + w.ranges_off);
        p.logits = reinterpret_cast<float *>(ws + w.logits_off);
    }
    const cudaStream_t st = (cudaStream_t)stream;
    const bool pdl = (plan->flags & PKV_FLAG_NO_PDL) == 0;
    cudaError_t e = s.head_dim == 128 ? launch_decode<128>(p, scores != nullptr, st, pdl)
                                      : launch_decode<64>(p, scores != nullptr, st, pdl);
    if (e != cudaSuccess)
        return PKV_ERR_CUDA;
    // a batch that can never fill one block's share leaves nothing to merge
    if (!scores && (plan->num_splits == 1 || pairs * s.max_pages_per_seq <= min_pages(G)))
        return PKV_OK;
    FinishParams f{};
    f.w.m = p.ws_m;
    f.w.l = p.ws_l;
    f.w.G = G;
    f.acc = p.ws_acc;
    f.spans = p.spans;
    f.span_pair = p.span_pair;
    f.out = p.out;
    f.blocks = p.blocks;
    f.chunks = 1;
    if (scores) {
        f.w.logits = p.logits;
        f.w.ranges = p.ranges;
        f.w.ws_error = p.ws_error;
        f.w.seq_lens = seq_lens;
        f.w.scores = scores;
        f.w.stride_row = score_stride_row;
        f.w.stride_head = score_stride_head;
        f.w.H_kv = s.H_kv;
        f.w.capacity = capacity;
        f.w.n_slots = w.n_slots;
        f.chunks = (int32_t)weight_blocks(1, capacity);
    }
    const int64_t grid = merges + (scores ? weight_blocks(pairs, capacity) : 0);
    e = s.head_dim == 128 ? launch_finish<128>(f, scores != nullptr, grid, st, pdl)
                          : launch_finish<64>(f, scores != nullptr, grid, st, pdl);
    if (e != cudaSuccess)
        return PKV_ERR_CUDA;
    return PKV_OK;
}

}  // extern "C"
