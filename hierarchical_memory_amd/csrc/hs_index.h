// Internal declarations of the operators that make a selection (hs_heads.hip, hs_score.hip, hs_select.hip), shared with the C
// ABI (hs_api.cpp).
#pragma once

#include "hs_internal.h"

namespace hs {

constexpr int kMxBlock = 32;  // values under one scale

struct HeadArgs {
  int32_t dim, rope, rope_at;
  int32_t halves;          // 1: the rotated part's pairs are (i, i + rope / 2), 0: (2i, 2i + 1)
  int32_t norm;            // HS_NORM_*
  float eps;
  int32_t heads, n;
  int64_t x_stride, x_head_stride;  // elements
  const uint16_t* x;       // bf16
  const uint16_t* weight;  // [dim] or nullptr
  const uint16_t* bias;    // [dim] or nullptr
  const double* freqs;     // [rope / 2] radians per position, or nullptr (no rotation)
  const int32_t* pos;      // [n] or nullptr
  // rows: bf16 with strides, or (scales given) e4m3 packed
  char* o;
  int64_t o_stride, o_head_stride;  // elements
  uint8_t* scales;
  // the key cache (heads == 1)
  int32_t type;            // HS_KEY_*
  int32_t R, H;
  const int32_t* req;
  char* keys;              // [R][H] values
  uint8_t* key_scales;     // [R][H][dim / 32]
  uint16_t* values;        // [n][dim] bf16 or nullptr
  int32_t* status;         // [R] or nullptr
};

struct ScoreArgs {
  int32_t dim, type, heads, R, H, n;
  const char* keys;
  const uint8_t* key_scales;
  const uint8_t* q;         // e4m3 [n][heads][dim]
  const uint8_t* q_scales;  // [n][heads][dim / 32]
  const float* weights;     // [n][heads]
  const int32_t* req;
  const int32_t* pos;
  float* scores;
  int64_t stride;
};

struct SelectArgs {
  int32_t rows, n, k, recent;
  int64_t columns;
  const float* scores;
  const int32_t* pos;
  const int32_t* cu;  // [rows + 1] or nullptr
  int32_t* topk;      // [rows][k]
  char* work;
};

inline uint64_t key_scales_at(int R, int H, int dim, int type) {  // offset of the scales in the key cache
  return ((uint64_t)R * H * (type ? dim / 2 : dim) + 255) & ~255ull;
}

uint64_t select_work_bytes(int rows, int64_t columns, int k);

hipError_t launch_heads(const HeadArgs& a, hipStream_t s);
hipError_t launch_store_keys(const HeadArgs& a, hipStream_t s);
hipError_t launch_score(const ScoreArgs& a, hipStream_t s);
hipError_t launch_select(const SelectArgs& a, hipStream_t s);

}  // namespace hs
