// Index scores of tokens against the keys of their contexts (gfx950).
//
//   s[t][x] = sum_h w[t][h] * max(0, q[t][h] . key[r][x])
//
// Matrix instructions do the dot products, the queries' heads down the accumulators and the keys across the lanes, so that
// the sum over the heads stays in a lane (and the one 32 away) and 64 scores leave a wave as one store. A wave takes 64 keys at
// a time, from memory straight to its registers and there to bf16, which holds a microscaled value exactly. The instructions
// that take 8- and 4-bit operands as they are would spare that, but they lose of each sum what lies 2^-14 below its largest
// product (normal keys and queries: 1.5e-5 off in 8 bits and 4e-6 in 4, 6e-9 in bf16), and the selection is made of these sums.
// The queries of a workgroup's tokens lie in LDS as the instructions take them, and are read once for every 64 keys.
#include "hs_index.h"
#include "hs_mfma.h"

namespace hs {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWaves = kScoreThreads / 64;
constexpr int kKeys = 64;  // of a wave at a time

// kRows: heads of a token filled up to 16, 32 or 64. kTokens: tokens of a workgroup.
template <int kDim, bool kFour, int kRows, int kTokens>
__global__ __launch_bounds__(kScoreThreads, 2) void score_kernel(ScoreArgs a, int chunk, int chunks) {
  constexpr int kSteps = kDim / 16;                              // of a dot product
  constexpr int kTiles = (kTokens * kRows + 31) / 32;            // of 32 rows
  constexpr int kAcc = kRows < 32 && kTokens == 1 ? 8 : 16;      // accumulators that hold heads
  constexpr int kBlocks = kDim / 64;                             // scales of a lane's half of a key
  constexpr int kRaw = kDim / (kFour ? 64 : 32);                 // 16-byte loads of a lane's half of a key
  constexpr int kKeyBytes = kDim / (kFour ? 2 : 1);
  __shared__ __align__(16) bf8 frag[kTiles * kSteps * 64];       // [tile][step][lane]
  __shared__ __align__(16) float weight[kTiles * 32];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  const int t0 = (int)(blockIdx.x / chunks) * kTokens, part = blockIdx.x % chunks;
  const int lo = part * chunk;
  int req[kTokens], last[kTokens], most = -1;  // last: -1 for a token that is skipped
#pragma unroll
  for (int i = 0; i < kTokens; ++i) {
    const int t = t0 + i < a.n ? t0 + i : a.n - 1;
    const int r = a.req[t], p = a.pos[t];
    const bool there = t0 + i < a.n && r >= 0 && r < a.R && p >= 0 && p < a.H;
    req[i] = r;
    last[i] = there ? p : -1;
    most = last[i] > most ? last[i] : most;
  }
  if (most < lo) return;
  for (int i = tid; i < kTiles * kSteps * 64; i += kScoreThreads) {
    const int row = (i / (kSteps * 64)) * 32 + (i & 31), step = i / 64 % kSteps, t = t0 + row / kRows, h = row % kRows;
    const int d = (i >> 5 & 1) * (kDim / 2) + 8 * step;
    bf2 v[4] = {};
    if (t < a.n && h < a.heads && row < kTokens * kRows) {
      const int64_t at = (int64_t)t * a.heads + h;
      const uint2 x = *(const uint2*)(a.q + at * kDim + d);
      const float scale = __uint_as_float((uint32_t)a.q_scales[at * (kDim / kMxBlock) + d / kMxBlock] << 23);
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, scale, false);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, scale, true);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, scale, false);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, scale, true);
    }
    frag[i] = __builtin_bit_cast(bf8, v);
  }
  for (int i = tid; i < kTiles * 32; i += kScoreThreads) {
    const int t = t0 + i / kRows, h = i % kRows;
    weight[i] = t < a.n && h < a.heads && i < kTokens * kRows ? a.weights[(int64_t)t * a.heads + h] : 0.0f;
  }
  __syncthreads();

  int end = 0;  // of a run of tokens of one request
  for (int begin = 0; begin < kTokens; begin = end) {
    int r = -1, run_last = -1;
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
      if (i == begin) r = req[i];
    bool same = true;
    end = begin;
#pragma unroll
    for (int i = 0; i < kTokens; ++i)
      if (i >= begin) {
        same = same && req[i] == r;
        if (same) {
          end = i + 1;
          run_last = last[i] > run_last ? last[i] : run_last;
        }
      }
    r = __builtin_amdgcn_readfirstlane(r);
    end = __builtin_amdgcn_readfirstlane(end);
    run_last = __builtin_amdgcn_readfirstlane(run_last);
    const int mine = run_last - lo < chunk ? run_last - lo + 1 : chunk;  // keys of this part, from lo on
    if (wave * kKeys >= mine) continue;
    const char* keys = a.keys + ((int64_t)r * a.H + lo) * kKeyBytes + half * (kKeyBytes / 2);
    const uint8_t* scales = a.key_scales + ((int64_t)r * a.H + lo) * (kDim / kMxBlock) + half * kBlocks;
    v4u raw[2][kRaw];
    uint32_t raw_scale[2];
    auto load = [&](int x0) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        int x = x0 + 32 * j + col;
        x = x < mine ? x : mine - 1;
#pragma unroll
        for (int i = 0; i < kRaw; ++i) raw[j][i] = *(const v4u*)(keys + x * kKeyBytes + 16 * i);
        if (kBlocks == 2) raw_scale[j] = *(const uint16_t*)(scales + x * (kDim / kMxBlock));
        else raw_scale[j] = scales[x * (kDim / kMxBlock)];
      }
    };
    load(wave * kKeys);
    for (int x0 = wave * kKeys; x0 < mine; x0 += kScoreWaves * kKeys) {
      bf8 key[2][kSteps];
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int s = 0; s < kSteps; ++s) {
          const float scale = __uint_as_float((raw_scale[j] >> (8 * (s / 4)) & 255u) << 23);
          bf2 v[4];
          if constexpr (kFour) {
            const uint32_t x = raw[j][s / 4][s % 4];
            v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0);
            v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1);
            v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2);
            v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3);
          } else {
            const uint32_t x = raw[j][s / 2][s % 2 * 2], y = raw[j][s / 2][s % 2 * 2 + 1];
            v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, false);
            v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, true);
            v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, false);
            v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, true);
          }
          key[j][s] = __builtin_bit_cast(bf8, v);
        }
      if (x0 + kScoreWaves * kKeys < mine) load(x0 + kScoreWaves * kKeys);
      constexpr int kStride = kRows >= 32 ? kRows / 32 : 1;  // tiles of a token, or of a pair of them
      for (int tile = begin * kRows / 32; tile * 32 < end * kRows; tile += kStride) {
        float sum[2][2] = {};  // [of the pair's tokens][of the key halves]
#pragma unroll
        for (int k = 0; k < kStride; ++k) {
          f16 acc[2] = {};
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const bf8 q = frag[((tile + k) * kSteps + s) * 64 + lane];
            acc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q, key[0][s], acc[0], 0, 0, 0);
            acc[1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q, key[1][s], acc[1], 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < kAcc; ++i) {
            const float w = weight[(tile + k) * 32 + 8 * (i / 4) + 4 * half + i % 4];
            const int of = kRows == 16 && i >= 8;
#pragma unroll
            for (int j = 0; j < 2; ++j)
              sum[of][j] = fmaf(w, __builtin_elementwise_maximum(acc[j][i], 0.0f), sum[of][j]);
          }
        }
#pragma unroll
        for (int k = 0; k < (kRows == 16 && kTokens > 1 ? 2 : 1); ++k) {
          const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum[k][0]), __float_as_uint(sum[k][1]), false, false);
          const float score = __uint_as_float(x[0]) + __uint_as_float(x[1]);
          const int i = kRows == 16 ? tile * 2 + k : tile / kStride;
          int p = -1;
#pragma unroll
          for (int j = 0; j < kTokens; ++j)
            if (j == i) p = last[j];
          if (i >= begin && i < end && x0 + lane <= p - lo) a.scores[(int64_t)(t0 + i) * a.stride + lo + x0 + lane] = score;
        }
      }
    }
  }
}

template <int kDim, bool kFour, int kRows, int kTokens>
hipError_t launch(const ScoreArgs& a, hipStream_t s) {
  const int64_t groups = ((int64_t)a.n + kTokens - 1) / kTokens;
  constexpr int kLeast = kScoreWaves * kKeys;
  int64_t chunk = ((int64_t)a.H * groups / 4096 + kLeast - 1) / kLeast * kLeast;
  chunk = chunk < kLeast ? kLeast : chunk > 4096 ? 4096 : chunk;
  const int chunks = (int)((a.H + chunk - 1) / chunk);
  // (a grid ends below 2^31)
  const int64_t most = ((1ll << 31) - 1) / chunks;
  for (int64_t g0 = 0; g0 < groups; g0 += most) {
    const int64_t t0 = g0 * kTokens, g = groups - g0 < most ? groups - g0 : most;
    ScoreArgs b = a;
    b.n = (int)(a.n - t0);
    b.q += t0 * a.heads * kDim;
    b.q_scales += t0 * a.heads * (kDim / kMxBlock);
    b.weights += t0 * a.heads;
    b.req += t0;
    b.pos += t0;
    b.scores += t0 * a.stride;
    hipLaunchKernelGGL((score_kernel<kDim, kFour, kRows, kTokens>), dim3((uint32_t)(g * chunks)), dim3(kScoreThreads), 0, s, b,
                       (int)chunk, chunks);
  }
  return hipGetLastError();
}

template <int kDim, bool kFour>
hipError_t launch_heads_of(const ScoreArgs& a, hipStream_t s) {
  const bool many = a.n >= 2 * a.R;
  if (a.heads <= 16) return many ? launch<kDim, kFour, 16, 16>(a, s) : launch<kDim, kFour, 16, 1>(a, s);
  if (a.heads <= 32) return many ? launch<kDim, kFour, 32, 8>(a, s) : launch<kDim, kFour, 32, 1>(a, s);
  return many ? launch<kDim, kFour, 64, 4>(a, s) : launch<kDim, kFour, 64, 1>(a, s);
}

}  // namespace

hipError_t launch_score(const ScoreArgs& a, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (a.dim == 64) return a.type ? launch_heads_of<64, true>(a, s) : launch_heads_of<64, false>(a, s);
  return a.type ? launch_heads_of<128, true>(a, s) : launch_heads_of<128, false>(a, s);
}

}  // namespace hs
