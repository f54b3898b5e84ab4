// Internal declarations of the latent-attention operators (hs_tokens.hip, hs_attend.hip, hs_prompt.hip), shared
// with the C ABI (hs_api.cpp).
#pragma once

#include "hs_internal.h"

namespace hs {

constexpr int kScaleBlock = 32;  // values of an 8-bit row's latent part under one scale

// Where the parts of a row of one format lie, in bytes from its start.
struct RowLayout {
  int32_t latent, rope;  // values of each part
  int32_t mx;            // 1: e4m3 latent values with e8m0 block scales, 0: bf16
  int32_t scales;        // byte offset of the scales (mx)
  int32_t rope_at;       // byte offset of the rope part
  int32_t bytes;         // bytes of a row, a multiple of 16
};

inline RowLayout row_layout(int latent, int rope, bool mx) {
  RowLayout l{latent, rope, mx ? 1 : 0, 0, 0, 0};
  if (mx) {
    l.scales = latent;
    l.rope_at = latent + (int)align16((uint64_t)latent / kScaleBlock);
  } else {
    l.rope_at = 2 * latent;
  }
  l.bytes = l.rope_at + 2 * rope;
  return l;
}

struct MapArgs {
  int32_t R, B, H, T, n;
  const int32_t* fresh;  // [R] new tokens of each request
  const int32_t* len;    // [R] tokens that each request has already
  const int32_t* tail0;  // [R] or nullptr (no tail)
  int32_t* cu;           // [R + 1]
  int32_t* req;          // [n]
  int32_t* pos;          // [n]
  int32_t* slot;         // [n]
  int32_t* status;       // [R] or nullptr
};

struct StoreArgs {
  RowLayout row;
  int32_t R, B, H, T, n;
  int32_t halves;        // 1: the rope part's pairs are (i, i + rope / 2), 0: (2i, 2i + 1)
  float eps;
  int64_t x_stride;      // elements from one token's input row to the next
  const uint16_t* x;     // bf16
  const uint16_t* weight;
  const double* freqs;   // [rope / 2] radians per position, or nullptr (no rotation)
  const int32_t* req;
  const int32_t* pos;
  const int32_t* slot;
  uint16_t* latent;      // [n][latent + rope] bf16, or nullptr
  int32_t* status;       // [R] or nullptr
  char* tail;
  char* hot;
  char* host;            // device address of the pinned pool
  const int32_t* page;
  int32_t* epoch;
};

struct AttendArgs {
  RowLayout row;
  int32_t R, k, B, T, heads;
  int32_t groups;         // groups of 16 heads to a workgroup (1, 2, 4 or 8)
  int32_t splits;         // parts of the selection, each a workgroup's
  float scale;
  const uint16_t* q;      // [R][heads][latent + rope] bf16
  const int32_t* out;     // [R][k] row indices, outside [0, B + T): none
  const char* hot;
  const char* tail;
  const char* gather;     // [R][k] rows, or nullptr (rows from hot and tail)
  uint16_t* o;            // [R][heads][latent] bf16
  float* lse;             // [R][heads] or nullptr
  float* work;            // partial results where splits > 1
};

struct PromptArgs {
  int32_t R, n_q, n_k, heads, nope, rope, value, causal;
  int64_t rope_stride;    // elements
  float scale;
  const uint16_t* q;      // [n_q][heads][nope + rope]
  const uint16_t* kv;     // [n_k][heads][nope + value]
  const uint16_t* krope;  // [n_k] rows of rope values
  const int32_t* cu_q;    // [R + 1]
  const int32_t* cu_k;    // [R + 1]
  uint16_t* o;            // [n_q][heads][value]
  float* lse;             // [n_q][heads] or nullptr
  int32_t sets;           // 128 queries to a workgroup each
  int32_t splits;         // most parts of a query tile's keys
  int32_t items;          // where splits > 1: parts of all tiles to aim at, for a head
  float* work;            // partial results where splits > 1
};

// How hs_attend shares out its work: groups of 16 heads to a workgroup and parts of each selection; and the bytes of the
// parts' results.
struct AttendPlan {
  int groups, splits;
};
AttendPlan attend_plan(int R, int k, int heads, const RowLayout& row);
uint64_t attend_work_bytes(const AttendPlan& plan, int R, int heads, const RowLayout& row);

// The same for hs_attend_prompt.
struct PromptPlan {
  int sets, splits, items;
};
PromptPlan prompt_plan(int R, int n_q, int n_k, int heads, int value);
uint64_t prompt_work_bytes(const PromptPlan& plan, int n_q, int heads, int value);

// Allows the attention kernels the LDS that they take, on the current device.
hipError_t set_attend_lds();
hipError_t set_prompt_lds();

hipError_t launch_map(const MapArgs& a, hipStream_t s);
hipError_t launch_store(const StoreArgs& a, hipStream_t s);
hipError_t launch_attend(const AttendArgs& a, hipStream_t s);
hipError_t launch_prompt(const PromptArgs& a, hipStream_t s);

}  // namespace hs
