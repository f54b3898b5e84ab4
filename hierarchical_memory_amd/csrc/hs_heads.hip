// Heads normed, rotated and rounded in one pass (gfx950): queries in bf16 or 8 bits, index keys into their cache.
#include "hs_index.h"

namespace hs {

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kStatusBad = 1;  // HS_STATUS_BAD_ID
constexpr int kHeadThreads = 256;
constexpr int kMostPer = 4;    // passes of a workgroup over its heads

enum Out { kBf16, kMx8, kCache8, kCache4 };

template <int kLanes, class T>
__device__ __forceinline__ T group_sum(T v) {
#pragma unroll
  for (int d = 1; d < kLanes; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// kLanes lanes have a head, 8 values each (16-byte loads). The turns of a workgroup's tokens are worked out once, into LDS,
// for all of a token's heads.
template <int kLanes, Out kOut>
__global__ __launch_bounds__(kHeadThreads) void heads_kernel(HeadArgs a, int per) {
  constexpr int kUnits = kHeadThreads / kLanes;
  constexpr bool kCache = kOut == kCache8 || kOut == kCache4;
  __shared__ float2 turns[4 * kHeadThreads * kMostPer];  // [tokens][rope / 2] (cosine, sine): at most 4 kLanes for each of kUnits per
  const int tid = threadIdx.x, lane = tid % kLanes, d0 = 8 * lane, P = a.rope / 2;
  const bool has = d0 < a.dim, rotate = a.freqs && P > 0;
  const int j0 = d0 - a.rope_at;  // of the rotated part
  const bool turning = rotate && has && j0 >= 0 && j0 < a.rope;
  float w[8], b[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) w[i] = 1.0f, b[i] = 0.0f;
  if (has && a.weight) {
    const bf8 v = *(const bf8*)(a.weight + d0);
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (float)v[i];
  }
  if (has && a.bias) {
    const bf8 v = *(const bf8*)(a.bias + d0);
#pragma unroll
    for (int i = 0; i < 8; ++i) b[i] = (float)v[i];
  }
  const int64_t units = (int64_t)a.n * a.heads;
  const int span = kUnits * per;
  for (int64_t u0 = (int64_t)blockIdx.x * span; u0 < units; u0 += (int64_t)gridDim.x * span) {
    const int64_t t0 = u0 / a.heads;
    const int h0 = (int)(u0 - t0 * a.heads);
    const int mine = (int)(units - u0 < span ? units - u0 : span);
    if (rotate) {
      __syncthreads();  // the turns before are read
      const int tokens = (h0 + mine - 1) / a.heads + 1;
      for (int i = tid; i < tokens * P; i += kHeadThreads) {
        const int64_t t = t0 + i / P;
        const int x = a.pos[t];
        // the angle in turns, in 64 bits, less its whole turns: what is left of it is exact enough in 32
        const double turn = (double)(x < 0 ? 0 : x) * (a.freqs[i % P] * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
        turns[i] = float2{c, s};
      }
      __syncthreads();
    }
    for (int p = 0; p < per; ++p) {
      const int u = p * kUnits + tid / kLanes;
      const int local = h0 + u, tok = local / a.heads, h = local - tok * a.heads;
      const int64_t t = t0 + tok;
      bool there = u < mine && (!a.pos || a.pos[t] >= 0);
      int64_t row = 0;
      if constexpr (kCache) {
        if (there) {
          const int r = a.req[t], x = a.pos[t];
          if (r < 0 || r >= a.R) {
            there = false;
          } else if (x >= a.H) {
            there = false;
            if (a.status && lane == 0) a.status[r] = kStatusBad;
          } else {
            row = (int64_t)r * a.H + x;
          }
        }
      }
      bf8 v{};
      if (there && has) v = *(const bf8*)(a.x + t * a.x_stride + h * a.x_head_stride + d0);
      float y[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] = (float)v[i];
      if (a.norm != 0) {
        const bool layer = a.norm == 2;
        float sum = 0.0f, sq = 0.0f, mean = 0.0f;
        if (layer) {
#pragma unroll
          for (int i = 0; i < 8; ++i) sum += y[i];
          sum = group_sum<kLanes>(sum);
          mean = sum / (float)a.dim;
          if (has) {
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] -= mean;
          }
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sq += y[i] * y[i];
        sq = group_sum<kLanes>(sq);
        const float inv = 1.0f / sqrtf(sq / (float)a.dim + a.eps);
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] *= inv;
        if (!(sq > 1e-28f && sq < 1e38f)) {  // squares that 32 bits lose (all lanes of a head take this branch, or none)
          double m = 0.0, d = 0.0;
          if (layer) {
#pragma unroll
            for (int i = 0; i < 8; ++i) m += (double)v[i];
            m = group_sum<kLanes>(m) / (double)a.dim;
          }
          double z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            z[i] = has ? (double)v[i] - m : 0.0;
            d += z[i] * z[i];
          }
          d = 1.0 / sqrt(group_sum<kLanes>(d) / (double)a.dim + (double)a.eps);
#pragma unroll
          for (int i = 0; i < 8; ++i) y[i] = (float)(z[i] * d);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = y[i] * w[i] + b[i];
      }
      if (rotate) {
        const float2* cs = turns + tok * P;
        if (a.halves) {
          const bool first = j0 < P;
          const int other = turning ? (first ? lane + P / 8 : lane - P / 8) : lane;
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) z[i] = __shfl(y[i], other, kLanes);
          if (turning) {
            cs += first ? j0 : j0 - P;
#pragma unroll
            for (int i = 0; i < 8; ++i) y[i] = first ? y[i] * cs[i].x - z[i] * cs[i].y : z[i] * cs[i].y + y[i] * cs[i].x;
          }
        } else if (turning) {
          cs += j0 / 2;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float u2 = y[2 * i], q2 = y[2 * i + 1];
            y[2 * i] = u2 * cs[i].x - q2 * cs[i].y;
            y[2 * i + 1] = u2 * cs[i].y + q2 * cs[i].x;
          }
        }
      }
      if constexpr (kOut == kBf16) {
        if (there && has) {
          bf8 o;
#pragma unroll
          for (int i = 0; i < 8; ++i) o[i] = (__bf16)y[i];
          *(bf8*)((uint16_t*)a.o + t * a.o_stride + h * a.o_head_stride + d0) = o;
        }
        continue;
      }
      // the block's largest magnitude m * 2^e, 1 <= m < 2, against the type's largest value, 1.75 * 2^8 or 1.5 * 2^2
      uint32_t top = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t x = __float_as_uint(y[i]) & 0x7fffffffu;
        top = x > top ? x : top;
      }
      for (int d = 1; d < 4; d <<= 1) {
        const uint32_t x = __shfl_xor(top, d);
        top = x > top ? x : top;
      }
      const bool four = kOut == kCache4;
      int expo = (int)(top >> 23) - 127 - (four ? 2 : 8) + ((top & 0x7fffffu) > (four ? 0x400000u : 0x600000u) ? 1 : 0);
      expo = expo < -100 ? -100 : expo;
      const bool number = top < 0x7f800000u;
      const float f = __uint_as_float((uint32_t)(127 - expo) << 23), scale = __uint_as_float((uint32_t)(127 + expo) << 23);
      const uint8_t byte = number ? (uint8_t)(127 + expo) : 255;
      if (!(there && has)) continue;
      if constexpr (kOut == kCache4) {
        uint32_t q = 0;
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[0] * f, y[1] * f, 1.0f, 0);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[2] * f, y[3] * f, 1.0f, 1);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[4] * f, y[5] * f, 1.0f, 2);
        q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, y[6] * f, y[7] * f, 1.0f, 3);
        if (!number) q = 0;
        *(uint32_t*)(a.keys + row * (a.dim / 2) + d0 / 2) = q;
        if (lane % 4 == 0) a.key_scales[row * (a.dim / kMxBlock) + lane / 4] = byte;
        if (a.values) {
          bf2 o[4];
          o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 0);
          o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 1);
          o[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 2);
          o[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(q, scale, 3);
          uint4 u = __builtin_bit_cast(uint4, o);
          if (!number) u = uint4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
          *(uint4*)(a.values + t * a.dim + d0) = u;
        }
      } else {
        uint32_t lo = 0, hi = 0;
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * f, y[1] * f, lo, false);
        lo = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * f, y[3] * f, lo, true);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * f, y[5] * f, hi, false);
        hi = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * f, y[7] * f, hi, true);
        if (!number) lo = hi = 0x7f7f7f7fu;
        const int64_t at = kCache ? row : t * a.heads + h;
        *(uint2*)((kCache ? a.keys : a.o) + at * a.dim + d0) = uint2{lo, hi};
        if (lane % 4 == 0) (kCache ? a.key_scales : a.scales)[at * (a.dim / kMxBlock) + lane / 4] = byte;
        if (kCache && a.values) {
          bf2 o[4];
          o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, false);
          o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, scale, true);
          o[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, false);
          o[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, scale, true);
          uint4 u = __builtin_bit_cast(uint4, o);
          if (!number) u = uint4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
          *(uint4*)(a.values + t * a.dim + d0) = u;
        }
      }
    }
  }
}

template <int kLanes, Out kOut>
hipError_t launch(const HeadArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.n * a.heads;
  if (units <= 0) return hipSuccess;
  constexpr int kUnits = kHeadThreads / kLanes;
  const int per = units > (int64_t)kUnits * 4096 ? kMostPer : 1;
  const int64_t need = (units + kUnits * per - 1) / (kUnits * per);
  hipLaunchKernelGGL((heads_kernel<kLanes, kOut>), dim3((int)(need < (1 << 20) ? need : 1 << 20)), dim3(kHeadThreads), 0, s, a, per);
  return hipGetLastError();
}

template <Out kOut>
hipError_t launch_dim(const HeadArgs& a, hipStream_t s) {
  return a.dim <= 64 ? launch<8, kOut>(a, s) : a.dim <= 128 ? launch<16, kOut>(a, s) : launch<32, kOut>(a, s);
}

}  // namespace

hipError_t launch_heads(const HeadArgs& a, hipStream_t s) {
  return a.scales ? launch_dim<kMx8>(a, s) : launch_dim<kBf16>(a, s);
}

hipError_t launch_store_keys(const HeadArgs& a, hipStream_t s) {
  if (a.type) return a.dim == 64 ? launch<8, kCache4>(a, s) : launch<16, kCache4>(a, s);
  return a.dim == 64 ? launch<8, kCache8>(a, s) : launch<16, kCache8>(a, s);
}

}  // namespace hs
