// Internal declarations shared by the host planner (pkv_host.cpp) and the
// CUDA side (pkv_decode.cu) of libpkv.so.  Not part of the C ABI.
#pragma once

#include <cstddef>
#include <cstdint>

#include "pkv.h"

namespace pkv {

constexpr int kPage = 16;          // the fast path's tokens per page
constexpr size_t kWsAlign = 256;   // workspace section alignment

// Device error word bits (pkv_workspace_status).
constexpr uint32_t kErrTimeout = 1;
constexpr uint32_t kErrSeqLen = 2;
constexpr uint32_t kErrPageId = 4;
constexpr uint32_t kErrItem = 8;

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline size_t round_up(size_t x, size_t a) { return (x + a - 1) / a * a; }

// Workspace sections, in bytes from the workspace base.  The error word and
// the counters are zero between calls (each call leaves them so); the
// partial states need no initial value.
struct WsLayout {
    size_t error_off = 0;    // uint32 error word (+ padding)
    size_t counters_off = 0; // uint32 completion counter per (row, kv head) pair
    size_t m_off = 0;        // float m[slot][G]  (running max, log2 domain)
    size_t l_off = 0;        // float l[slot][G]
    size_t acc_off = 0;      // float acc[slot][G][D]
    size_t range_off = 0;    // PKV_FLAG_SCORES: the pair's slots, as int4 (SlotRange)
    size_t record_off = 0;   // PKV_FLAG_SCORES: what each slot's block did, 32 bytes (SlotRecord)
    size_t logits_off = 0;   // PKV_FLAG_SCORES: float logits[pair][max_pages * P][logit_heads(G)]
    size_t total = 0;
    int64_t n_slots = 0;
};

// Heads a token's stored logits are laid out for: the power of two from 2 up that
// holds G, so that they are whole aligned vectors.
inline int32_t logit_heads(int64_t G) { return G <= 2 ? 2 : G <= 4 ? 4 : G <= 8 ? 8 : 16; }

inline WsLayout ws_layout(const pkv_shape &s, const pkv_plan &p, int32_t n_items)
{
    WsLayout w;
    const int64_t pairs = (int64_t)s.B * s.H_kv;
    const int64_t G = s.H_kv > 0 ? s.H_q / s.H_kv : 0;
    if (p.mode == PKV_SPLIT_S)
        w.n_slots = pairs * p.num_splits;
    else if (p.mode == PKV_WORK_QUEUE || p.mode == PKV_BALANCED)
        w.n_slots = n_items;
    const bool scores = (p.flags & PKV_FLAG_SCORES) != 0;
    if (scores && p.mode == PKV_NO_SPLIT)
        w.n_slots = pairs;  // every pair's final state is read back for its weights
    size_t off = kWsAlign;  // error word section
    w.counters_off = off;
    off += round_up((size_t)pairs * 4, kWsAlign);
    w.m_off = off;
    off += round_up((size_t)(w.n_slots * G) * 4, kWsAlign);
    w.l_off = off;
    off += round_up((size_t)(w.n_slots * G) * 4, kWsAlign);
    w.acc_off = off;
    off += round_up((size_t)(w.n_slots * G * s.head_dim) * 4, kWsAlign);
    if (scores) {
        w.range_off = off;
        off += round_up((size_t)pairs * 16, kWsAlign);
        w.record_off = off;
        off += round_up((size_t)w.n_slots * 32, kWsAlign);
        w.logits_off = off;
        off += round_up((size_t)pairs * s.max_pages_per_seq * s.page_size * logit_heads(G) * 4, kWsAlign);
    }
    w.total = off;
    return w;
}

// Shape checks shared by the host entry points; PKV_OK when the shape is
// well formed (fast-path support is checked separately by the decode call).
int check_shape(const pkv_shape *s);

// Balanced queue: block b owns pages [floor(b*U/T), floor((b+1)*U/T)) of
// the U pages of all (row, KV head) pairs laid end to end.
inline int64_t balanced_start(int64_t U, int64_t T, int64_t b) { return (b * U) / T; }

}  // namespace pkv
