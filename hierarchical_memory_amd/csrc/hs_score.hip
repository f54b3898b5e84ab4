// Index scores of tokens against the keys of their contexts (gfx950).
//
//   s[t][x] = sum_h w[t][h] * max(0, q[t][h] . key[r][x])
//
// One thread per key, a token's queries in LDS as 32-bit values.
#include "hs_index.h"

namespace hs {

namespace {

typedef float f2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kScoreThreads = 256;

// byte 255: NaN; byte 0: 2^-127
__device__ __forceinline__ float scale_of(uint32_t byte) {
  return byte == 255 ? __uint_as_float(0x7fc00000u) : byte == 0 ? 0x1p-127f : __uint_as_float(byte << 23);
}

template <int kDim, bool kFour>
__global__ __launch_bounds__(kScoreThreads) void score_kernel(ScoreArgs a) {
  extern __shared__ float q[];  // [heads][kDim]
  const int t = blockIdx.y, tid = threadIdx.x;
  const int r = a.req[t], p = a.pos[t];
  if (r < 0 || r >= a.R || p < 0 || p >= a.H) return;
  if ((int64_t)blockIdx.x * kScoreThreads > p) return;
  for (int i = tid; i < a.heads * kDim; i += kScoreThreads) {
    const int64_t at = (int64_t)t * a.heads * kDim + i;
    const f2 v = __builtin_amdgcn_cvt_pk_f32_fp8((int)a.q[at], false);
    q[i] = v[0] * scale_of(a.q_scales[at / kMxBlock]);
  }
  __syncthreads();
  const int x = blockIdx.x * kScoreThreads + tid;
  if (x > p) return;
  const int64_t row = (int64_t)r * a.H + x;
  float k[kDim];
#pragma unroll
  for (int i = 0; i < kDim; i += 8) {
    const float scale = scale_of(a.key_scales[row * (kDim / kMxBlock) + i / kMxBlock]);
    if (kFour) {
      const uint32_t w = *(const uint32_t*)(a.keys + row * (kDim / 2) + i / 2);
      f2 v[4];
      v[0] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0);
      v[1] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
      v[2] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2);
      v[3] = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
#pragma unroll
      for (int j = 0; j < 8; ++j) k[i + j] = v[j / 2][j % 2] * scale;
    } else {
      const uint2 w = *(const uint2*)(a.keys + row * kDim + i);
      f2 v[4];
      v[0] = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, false);
      v[1] = __builtin_amdgcn_cvt_pk_f32_fp8(w.x, true);
      v[2] = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, false);
      v[3] = __builtin_amdgcn_cvt_pk_f32_fp8(w.y, true);
#pragma unroll
      for (int j = 0; j < 8; ++j) k[i + j] = v[j / 2][j % 2] * scale;
    }
  }
  float s = 0.0f;
  for (int h = 0; h < a.heads; ++h) {
    float d = 0.0f;
#pragma unroll
    for (int i = 0; i < kDim; ++i) d += q[h * kDim + i] * k[i];
    s += a.weights[(int64_t)t * a.heads + h] * __builtin_elementwise_maximum(d, 0.0f);
  }
  a.scores[t * a.stride + x] = s;
}

template <int kDim, bool kFour>
hipError_t launch(const ScoreArgs& a, hipStream_t s) {
  // (a grid's second dimension ends at 65535)
  for (int t0 = 0; t0 < a.n; t0 += 65535) {
    ScoreArgs b = a;
    b.n = a.n - t0 < 65535 ? a.n - t0 : 65535;
    b.q += (int64_t)t0 * a.heads * kDim;
    b.q_scales += (int64_t)t0 * a.heads * (kDim / kMxBlock);
    b.weights += (int64_t)t0 * a.heads;
    b.req += t0;
    b.pos += t0;
    b.scores += t0 * a.stride;
    hipLaunchKernelGGL((score_kernel<kDim, kFour>), dim3((a.H + kScoreThreads - 1) / kScoreThreads, b.n), dim3(kScoreThreads),
                       a.heads * kDim * 4, s, b);
  }
  return hipGetLastError();
}

}  // namespace

hipError_t launch_score(const ScoreArgs& a, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (a.dim == 64) return a.type ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return a.type ? launch<128, true>(a, s) : launch<128, false>(a, s);
}

}  // namespace hs
