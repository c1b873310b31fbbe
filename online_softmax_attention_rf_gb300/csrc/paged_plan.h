// paged_plan.h -- how a step's attention over a paged cache is divided among
// the SMs: the plan that rf_paged_plan writes and rf_attn_paged reads.
//
// Work. A sequence's new tokens are packed with the G = H / Hkv query heads of
// one key head: packed row i * G + j is head j of the group at token i. A tile
// is 128 packed rows (floor(128 / G) tokens); an item is one or two successive
// tiles of one (sequence, key head), which share the keys they read. Items are
// ordered by sequence, key head, first token. An item's key tiles of 128 keys
// are its steps. The plan cuts the sequence of all steps into one contiguous
// span per CTA, of equal cost. An item that a cut falls into is computed in
// parts: each CTA leaves its part's softmax state in the workspace, and the
// merge combines them.
//
// The plan carries the lengths it was made for, so that a call reads one
// consistent set of them.
#pragma once

#include <stdint.h>

namespace rf {

constexpr int kPlanMagic = 0x52465031;
constexpr int kPlanCtas = 152;    // spans; more than the SMs of a GB300 would not be resident
constexpr int kPlanTile = 128;    // packed query rows, and keys, per tile
constexpr int kPlanRows = 2 * kPlanTile;  // packed rows per item

// Where a span starts: step `step` of the item that holds tokens
// [pair * 2 * (128 / G), ...) of (seq, head). seq == B: the end.
struct PlanStart {
  int seq, head, pair, step;
  int row0, row1, kv, pad;  // the sequence's packed rows and cached tokens
};

// An item computed by the CTAs [cta, cta + parts), with `rows` packed rows. The
// merge takes each of its tiles in units of 32 rows, numbered from unit0 on.
struct PlanMerge {
  int seq, head, pair, cta, parts, rows, unit0;
  int row0;  // its first token among the packed tokens
};

struct alignas(16) PlanHeader {
  int magic, B, T, H, Hkv, page, max_pages, causal;
  int ctas;         // spans in use
  int n_merge;      // items in parts
  int merge_units;  // their units of 32 rows
  int pad[5];
  PlanStart start[kPlanCtas + 1];
  PlanMerge merge[kPlanCtas];
  // followed by int32 cu_q[B + 1], kv_len[B] and one word of padding, then
  // int64 cost[B + 1] (prefix sums)
};
static_assert(sizeof(PlanHeader) % 16 == 0 && sizeof(PlanStart) == 32 && sizeof(PlanMerge) == 32,
              "entries are read by 16 bytes; the prefix sums need 8-byte alignment");

__host__ __device__ inline const int32_t* plan_cu_q(const void* plan) {
  return reinterpret_cast<const int32_t*>(static_cast<const PlanHeader*>(plan) + 1);
}
__host__ __device__ inline const int32_t* plan_kv_len(const void* plan, int B) {
  return plan_cu_q(plan) + B + 1;
}
__host__ __device__ inline size_t plan_cost_offset(int B) {
  return sizeof(PlanHeader) + (2 * size_t(B) + 2) * 4;
}
__host__ __device__ inline size_t plan_bytes(int B) {
  const size_t n = plan_cost_offset(B) + (size_t(B) + 1) * 8;
  return (n + 255) / 256 * 256;
}

// Tokens per 128-row tile.
__host__ __device__ inline int plan_tile_tokens(int G) { return kPlanTile / G; }

// Units of 32 rows in tile `tile` of an item of ntok tokens.
__host__ __device__ inline int plan_units(int ntok, int tile, int G) {
  const int tt = plan_tile_tokens(G);
  const int tok = ntok - tile * tt < tt ? ntok - tile * tt : tt;
  return tok > 0 ? (tok * G + 31) / 32 : 0;
}

// Key tiles that hold the first `keys` keys. A cache may have up to 2^31 - 1 of
// them: rounding up by an addition would wrap.
__host__ __device__ inline int plan_steps(int keys) {
  return keys / kPlanTile + (keys % kPlanTile != 0 ? 1 : 0);
}

// Keys that token i of n new ones sees, of kv cached ones.
__host__ __device__ inline int plan_visible(int i, int n, int kv, int causal) {
  if (!causal) return kv;
  const int lim = kv - n + i + 1;
  return lim < 0 ? 0 : lim;
}

}  // namespace rf
