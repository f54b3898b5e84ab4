// Heads normed, rotated and rounded in one pass (gfx950): queries in bf16 or 8 bits, index keys into their cache.
//
// Four lanes have a head, 8 values of every 32 each: a block under one scale is four lanes', a norm's sum takes two steps over
// them, all of a lane's loads (16 bytes of each block) are on their way at once, and the pairs of a rotated part in halves that
// is a multiple of 64 wide lie in one lane. A workgroup works out the turns (cosine and sine of its tokens' angles) while its
// values come, once for all of a token's heads. Memory bounds many heads (8192 tokens x 16 heads x 192 values 23.7 us, 4.25 TB/s,
// where some of the inputs are still in the last-level cache, 25.9 us, 3.9 TB/s, where none are), one workgroup's chain of reads,
// turns and norm few (256 x 32 x 128 4.7 us) and prompts' keys (41 K of 128 values 10.5 us).
#include "hs_index.h"

namespace hs {

namespace {

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf2 __attribute__((ext_vector_type(2)));

constexpr int kStatusBad = 1;  // HS_STATUS_BAD_ID
constexpr int kHeadThreads = 256;
constexpr int kMostHeadBlocks = 1 << 20;
// Bytes of turns (and exchanged values) of a workgroup: with weight and bias the 64 KiB that a launch takes without a raised
// limit. Only single heads of 256 values that are turned whole pass it in 64s, and go in 32s (40000 of them 27.1 us; with 240
// values turned, in 64s, 26.1).
constexpr size_t kMostTurns = (64 << 10) - 2 * 256 * sizeof(uint16_t);

enum Out { kBf16, kMx8, kCache8, kCache4 };
// How a rotated part in halves finds the other value of a pair, q = rope / 16 pieces of 8 values on: in the lane itself (q a
// multiple of 4), two lanes on in the same block (q = 2), or anywhere (through LDS).
enum Mode { kPairs, kInLane, kTwoLanes, kAnywhere, kStill };

struct HeadPlan {
  int32_t mode;
  uint32_t magic, pair_magic;  // ceil(2^32 / heads), ceil(2^32 / (rope / 2)): (i * magic) >> 32 = i / heads for i < 2^16
  int32_t span;    // heads of a workgroup (its first threads'; all of its threads work out turns)
  int32_t tokens;  // most tokens of a workgroup
};

// Waves to a SIMD: a wave has its C kilobytes on their way, so that four of them keep the memory busy.
constexpr int kWavesOf(int C) { return C <= 1 ? 6 : C <= 2 ? 5 : C <= 4 ? 4 : C <= 6 ? 3 : 2; }

template <class T>
__device__ __forceinline__ T quad_sum(T v) {
  v += __shfl_xor(v, 1);
  v += __shfl_xor(v, 2);
  return v;
}

// kDc: blocks from a value to the other of its pair.
template <int C, int kDc>
__device__ __forceinline__ void turn_in_lane(float (&y)[C][8], int piece0, int q, const float2* cs) {
#pragma unroll
  for (int i = 0; i + kDc < C; ++i) {
    const int p = 4 * i + piece0;  // from the rotated part's begin
    if (p < 0 || p >= q) continue;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float2 t = cs[8 * p + e];
      const float u = y[i][e], v = y[i + kDc][e];
      y[i][e] = u * t.x - v * t.y;
      y[i + kDc][e] = u * t.y + v * t.x;
    }
    __builtin_amdgcn_sched_barrier(0);  // one block's turns in registers at a time
  }
}

// C: blocks of 32 values of a head. kAll: with the ways that few heads are rotated in, halves of other than 16 or 32 values (they
// take registers: 8192 tokens x 32 heads x 128 values in 8 bits 29 us with them in one kernel, 24 without).
template <int C, Out kOut, bool kAll>
__global__ __launch_bounds__(kHeadThreads, kWavesOf(C)) void heads_kernel(HeadArgs a, HeadPlan plan) {
  constexpr bool kCache = kOut == kCache8 || kOut == kCache4;
  __shared__ __align__(16) uint16_t weight[32 * C], bias[32 * C];
  extern __shared__ __align__(16) float2 turns[];  // [tokens][rope / 2] (cosine, sine), then [heads of the workgroup][rope] values
  const int tid = threadIdx.x, lane = tid & 3, span = plan.span;
  const int P = a.rope / 2, q = a.rope / 16, piece0 = lane - a.rope_at / 8;
  const bool rotate = plan.mode != kStill;
  const int64_t units = (int64_t)a.n * a.heads;
  if (a.norm != 0)
    for (int i = tid; i < 32 * C; i += blockDim.x) {
      weight[i] = a.weight ? a.weight[i] : 0x3f80;  // one
      bias[i] = a.bias ? a.bias[i] : 0;
    }
  for (int64_t u0 = (int64_t)blockIdx.x * span; u0 < units; u0 += (int64_t)gridDim.x * span) {
    const int64_t t0 = a.heads == 1 ? u0 : u0 / a.heads;
    const int h0 = (int)(u0 - t0 * a.heads), mine = (int)(units - u0 < span ? units - u0 : span);
    const bool has = tid >> 2 < mine;
    const int u = has ? tid >> 2 : mine - 1, local = h0 + u;  // (lanes behind the last head repeat it, and store nothing)
    const int tok = a.heads == 1 ? local : (int)__umulhi((uint32_t)local, plan.magic), h = local - tok * a.heads;
    const int64_t t = t0 + tok;
    const int position = a.pos ? a.pos[t] : 0;
    bool there = has && position >= 0;
    const uint16_t* in = a.x + t * a.x_stride + h * a.x_head_stride + 8 * lane;
    bf8 v[C];
#pragma unroll
    for (int i = 0; i < C; ++i) v[i] = *(const bf8*)(in + 32 * i);
    int64_t row = 0;
    if constexpr (kCache) {
      const int r = a.req[t];
      const bool known = r >= 0 && r < a.R;
      if (there && known && position >= a.H && a.status && lane == 0) a.status[r] = kStatusBad;
      there = there && known && position < a.H;
      row = (int64_t)r * a.H + position;
    }
    if (rotate) {
      if (u0 != (int64_t)blockIdx.x * span) __syncthreads();  // the turns before are read
      const int tokens = a.heads == 1 ? mine : (int)__umulhi((uint32_t)(h0 + mine - 1), plan.magic) + 1;
      for (int i = tid; i < tokens * P; i += kHeadThreads) {
        const int k = (int)__umulhi((uint32_t)i, plan.pair_magic), pair = i - k * P, x = a.pos[t0 + k];
        // the angle in turns, in 64 bits, less its whole turns: what is left of it is exact enough in 32
        const double turn = (double)(x < 0 ? 0 : x) * (a.freqs[pair] * 0.15915494309189535);
        float s, c;
        sincospif((float)(2.0 * (turn - rint(turn))), &s, &c);
        turns[i] = float2{c, s};
      }
    }
    __syncthreads();
    float y[C][8];
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int e = 0; e < 8; ++e) y[i][e] = (float)v[i][e];
    if (a.norm != 0) {
      const bool layer = a.norm == 2;
      constexpr float kShare = 1.0f / (32 * C);
      if (layer) {
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) sum += y[i][e];
        // The mean as the nearest 32 bits and what they leave of it: of values that hardly differ, next to nothing but that is
        // left behind the mean (rows of equal values are zeros, as by the formula, and no noise over sqrt(eps)).
        constexpr float kCount = 32 * C;
        sum = quad_sum(sum);
        float mean = sum * kShare;
        mean = fmaf(fmaf(-kCount, mean, sum), kShare, mean);
        const float rest = fmaf(-kCount, mean, sum) * kShare;
#pragma unroll
        for (int i = 0; i < C; ++i)
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] = (y[i][e] - mean) - rest;
      }
      float sq = 0.0f;
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) sq += y[i][e] * y[i][e];
      sq = quad_sum(sq);
      const float inv = 1.0f / sqrtf(sq * kShare + a.eps);
#pragma unroll
      for (int i = 0; i < C; ++i)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= inv;
      // squares that 32 bits lose, or their mean and an eps next to the largest (the four lanes take this branch, or none of them)
      if (!(sq > 1e-28f && sq < 1e38f && a.eps < 1e38f)) {
        double m = 0.0, d = 0.0;
        const __bf16* again = (const __bf16*)in;  // (read again: registers are short)
        if (layer) {
#pragma unroll 1
          for (int i = 0; i < 8 * C; ++i) m += (double)(float)again[32 * (i >> 3) + (i & 7)];
          m = quad_sum(m) / (32 * C);
        }
#pragma unroll 1
        for (int i = 0; i < 8 * C; ++i) {
          const double z = (double)(float)again[32 * (i >> 3) + (i & 7)] - m;
          d += z * z;
        }
        d = 1.0 / sqrt(quad_sum(d) / (32 * C) + (double)a.eps);
#pragma unroll
        for (int i = 0; i < C; ++i) {
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] = (float)(((double)(float)again[32 * i + e] - m) * d);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
#pragma unroll
      for (int i = 0; i < C; ++i) {
        const bf8 w = *(const bf8*)(weight + 32 * i + 8 * lane);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[i][e] *= (float)w[e];
        if (layer) {
          const bf8 b = *(const bf8*)(bias + 32 * i + 8 * lane);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[i][e] += (float)b[e];
        }
        __builtin_amdgcn_sched_barrier(0);
      }
    }
    if (rotate) {
      const float2* cs = turns + tok * P;
      if (plan.mode == kPairs) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int p = 4 * i + piece0;
          if (p < 0 || p >= 2 * q) continue;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 z = cs[4 * p + e];
            const float u2 = y[i][2 * e], w2 = y[i][2 * e + 1];
            y[i][2 * e] = u2 * z.x - w2 * z.y;
            y[i][2 * e + 1] = u2 * z.y + w2 * z.x;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else if (plan.mode == kInLane) {
        if (!kAll || q == 4) turn_in_lane<C, 1>(y, piece0, q, cs);
        else if (q == 8) turn_in_lane<C, 2>(y, piece0, q, cs);
        else if (q == 12) turn_in_lane<C, 3>(y, piece0, q, cs);
        else turn_in_lane<C, 4>(y, piece0, q, cs);
      } else if (plan.mode == kTwoLanes) {
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int p = 4 * i + piece0;
          float z[8];
#pragma unroll
          for (int e = 0; e < 8; ++e) z[e] = __shfl_xor(y[i][e], 2);
          if (p < 0 || p >= 4) continue;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 t2 = cs[8 * (p & 1) + e];
            y[i][e] = p < 2 ? y[i][e] * t2.x - z[e] * t2.y : z[e] * t2.y + y[i][e] * t2.x;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      } else if constexpr (kAll) {
        float* part = (float*)(turns + plan.tokens * P) + u * a.rope;  // (the four lanes are of one wave: its LDS accesses stay in order)
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int p = 4 * i + piece0;
          if (p >= 0 && p < 2 * q)
#pragma unroll
            for (int e = 0; e < 8; ++e) part[8 * p + e] = y[i][e];
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int i = 0; i < C; ++i) {
          const int p = 4 * i + piece0;
          if (p < 0 || p >= 2 * q) continue;
          const bool first = p < q;
          const int at = first ? p : p - q;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float2 t2 = cs[8 * at + e];
            const float z = part[8 * (first ? p + q : p - q) + e];
            y[i][e] = first ? y[i][e] * t2.x - z * t2.y : z * t2.y + y[i][e] * t2.x;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if constexpr (kOut == kBf16) {
      if (there) {
        uint16_t* out = (uint16_t*)a.o + t * a.o_stride + h * a.o_head_stride + 8 * lane;
#pragma unroll
        for (int i = 0; i < C; ++i) {
          bf8 o;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] = (__bf16)y[i][e];
          *(bf8*)(out + 32 * i) = o;
        }
      }
    } else {
      const int64_t at = kCache ? row : t * a.heads + h;
      char* const values = (kCache ? a.keys : a.o) + at * (32 * C / (kOut == kCache4 ? 2 : 1));
      uint32_t bytes[(C + 3) / 4] = {};
#pragma unroll
      for (int i = 0; i < C; ++i) {
        // the block's largest magnitude m * 2^e, 1 <= m < 2, against the type's largest value, 1.75 * 2^8 or 1.5 * 2^2
        constexpr bool kFour = kOut == kCache4;
        uint32_t top = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const uint32_t x = __float_as_uint(y[i][e]) & 0x7fffffffu;
          top = x > top ? x : top;
        }
#pragma unroll
        for (int d = 1; d < 4; d <<= 1) {
          const uint32_t x = __shfl_xor(top, d);
          top = x > top ? x : top;
        }
        int expo = (int)(top >> 23) - 127 - (kFour ? 2 : 8) + ((top & 0x7fffffu) > (kFour ? 0x400000u : 0x600000u) ? 1 : 0);
        expo = expo < -100 ? -100 : expo;
        const bool number = top < 0x7f800000u;
        const float f = __uint_as_float((uint32_t)(127 - expo) << 23), scale = __uint_as_float((uint32_t)(127 + expo) << 23);
        bytes[i / 4] |= (number ? (uint32_t)(127 + expo) : 255u) << (8 * (i % 4));
        bf2 o[4];  // as the bytes stand for them
        if constexpr (kFour) {
          uint32_t x = 0;
          x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, y[i][0] * f, y[i][1] * f, 1.0f, 0);
          x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, y[i][2] * f, y[i][3] * f, 1.0f, 1);
          x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, y[i][4] * f, y[i][5] * f, 1.0f, 2);
          x = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(x, y[i][6] * f, y[i][7] * f, 1.0f, 3);
          x = number ? x : 0;
          if (there) *(uint32_t*)(values + 16 * i + 4 * lane) = x;
          o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0);
          o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1);
          o[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2);
          o[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3);
        } else {
          uint2 x{};
          x.x = __builtin_amdgcn_cvt_pk_fp8_f32(y[i][0] * f, y[i][1] * f, x.x, false);
          x.x = __builtin_amdgcn_cvt_pk_fp8_f32(y[i][2] * f, y[i][3] * f, x.x, true);
          x.y = __builtin_amdgcn_cvt_pk_fp8_f32(y[i][4] * f, y[i][5] * f, x.y, false);
          x.y = __builtin_amdgcn_cvt_pk_fp8_f32(y[i][6] * f, y[i][7] * f, x.y, true);
          x = number ? x : uint2{0x7f7f7f7fu, 0x7f7f7f7fu};
          if (there) *(uint2*)(values + 32 * i + 8 * lane) = x;
          o[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, scale, false);
          o[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.x, scale, true);
          o[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, scale, false);
          o[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x.y, scale, true);
        }
        if (kCache && there && a.values) {
          const uint4 bits = __builtin_bit_cast(uint4, o);
          *(uint4*)(a.values + t * (32 * C) + 32 * i + 8 * lane) =
              number ? bits : uint4{0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u, 0x7fc07fc0u};
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      uint8_t* const to = (kCache ? a.key_scales : a.scales) + at * C;
      if (there && lane == 0) {
#pragma unroll
        for (int i = 0; i < C; i += 4) {
          if constexpr (C % 4 == 0) {
            *(uint32_t*)(to + i) = bytes[i / 4];
          } else {
#pragma unroll
            for (int j = i; j < i + 4 && j < C; ++j) to[j] = (uint8_t)(bytes[i / 4] >> (8 * (j - i)));
          }
        }
      }
    }
  }
}

template <int C, Out kOut>
hipError_t launch(const HeadArgs& a, hipStream_t s) {
  const int64_t units = (int64_t)a.n * a.heads;
  if (units <= 0) return hipSuccess;
  const int q = a.rope / 16;
  HeadPlan plan{};
  plan.mode = !a.freqs ? kStill : !a.halves ? kPairs : q % 4 == 0 ? kInLane : q == 2 && a.rope_at % 32 == 0 ? kTwoLanes : kAnywhere;
  plan.magic = a.heads == 1 ? 0 : (uint32_t)(((1ull << 32) + a.heads - 1) / a.heads);
  plan.pair_magic = a.rope ? (uint32_t)(((1ull << 32) + a.rope / 2 - 1) / (a.rope / 2)) : 0;
  // 64 heads to a workgroup (16 where they exchange values through LDS), or as few as leave each thread one turn where there are
  // not 512 workgroups: with single heads, the keys, a workgroup has a token for each of them (256 keys: 6.8 us with 64, 6.3 with 4;
  // 256 tokens with 32 heads: 4.6 with 64, 5.3 with 16)
  int span = plan.mode == kAnywhere ? 16 : kHeadThreads / 4;
  auto tokens = [&] { return a.heads == 1 ? span : (a.heads + span - 2) / a.heads + 1; };
  auto lds = [&] {
    return plan.mode == kStill ? 0 : (size_t)tokens() * a.rope / 2 * sizeof(float2) +
                                         (plan.mode == kAnywhere ? (size_t)span * a.rope * sizeof(float) : 0);
  };
  while (plan.mode != kStill && span > 4 &&
         ((units < (int64_t)span * 512 && tokens() * (a.rope / 2) > kHeadThreads) || lds() > kMostTurns)) span /= 2;
  plan.span = span;
  plan.tokens = tokens();
  const int64_t need = (units + span - 1) / span;
  const dim3 grid((uint32_t)(need < kMostHeadBlocks ? need : kMostHeadBlocks));
  if (plan.mode == kAnywhere || (plan.mode == kInLane && q > 4))
    hipLaunchKernelGGL((heads_kernel<C, kOut, true>), grid, dim3(kHeadThreads), lds(), s, a, plan);
  else
    hipLaunchKernelGGL((heads_kernel<C, kOut, false>), grid, dim3(kHeadThreads), lds(), s, a, plan);
  return hipGetLastError();
}

template <Out kOut>
hipError_t launch_dim(const HeadArgs& a, hipStream_t s) {
  switch (a.dim / 32) {
    case 1: return launch<1, kOut>(a, s);
    case 2: return launch<2, kOut>(a, s);
    case 3: return launch<3, kOut>(a, s);
    case 4: return launch<4, kOut>(a, s);
    case 5: return launch<5, kOut>(a, s);
    case 6: return launch<6, kOut>(a, s);
    case 7: return launch<7, kOut>(a, s);
    default: return launch<8, kOut>(a, s);
  }
}

}  // namespace

hipError_t launch_heads(const HeadArgs& a, hipStream_t s) {
  return a.scales ? launch_dim<kMx8>(a, s) : launch_dim<kBf16>(a, s);
}

hipError_t launch_store_keys(const HeadArgs& a, hipStream_t s) {
  if (a.type) return a.dim == 64 ? launch<2, kCache4>(a, s) : launch<4, kCache4>(a, s);
  return a.dim == 64 ? launch<2, kCache8>(a, s) : launch<4, kCache8>(a, s);
}

}  // namespace hs
