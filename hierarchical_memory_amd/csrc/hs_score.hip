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
// Memory bounds a token for each request (256 x 40960 keys x 32 heads in 4 bits 138 to 146 us, 4.7 to 5.0 TB/s; 32 ragged contexts
// x 20 heads in 8 bits 16.6 us, 4.3 TB/s), the matrix units tokens in groups (4 x 128 tokens behind 3968 to 15872 keys x 32 heads 45
// us, 940 TFLOP/s, 77 % of a large library product; relu and weights take vector instructions between).
#include "hs_index.h"
#include "hs_mfma.h"

namespace hs {

namespace {

constexpr int kScoreThreads = 256;
constexpr int kScoreWaves = kScoreThreads / 64;
constexpr int kJ = 2, kKeys = 32 * kJ;  // of a wave at a time
// Groups whose keys are shared out evenly; more are taken one by one, and the units even them out (32 requests x 16000 keys 15 us
// evenly, 80 one by one; 256 x 4000 24 and 26; 2048 x 500 34 and 28, but there one long context among them would be left alone, as
// it is from 2049 groups on: their starts have to fit LDS).
constexpr int kMostGroups = 2048;
constexpr int kMostBlocks = 1 << 20;

// kRows: heads of a token filled up to 16, 32 or 64. kTokens: tokens of a workgroup.
template <int kDim, bool kFour, int kRows, int kTokens>
__global__ __launch_bounds__(kScoreThreads, 2) void score_kernel(ScoreArgs a, int groups) {
  constexpr int kSteps = kDim / 16;                              // of a dot product
  constexpr int kTiles = (kTokens * kRows + 31) / 32;            // of 32 rows
  constexpr int kAcc = kRows < 32 && kTokens == 1 ? 8 : 16;      // accumulators that hold heads
  constexpr int kBlocks = kDim / 64;                             // scales of a lane's half of a key
  constexpr int kRaw = kDim / (kFour ? 64 : 32);                 // 16-byte loads of a lane's half of a key
  constexpr int kKeyBytes = kDim / (kFour ? 2 : 1);
  constexpr int kAhead = kTokens == 1 && kFour && kRows <= 32 ? 2 : 1;  // steps of a wave whose keys are on their way
  constexpr int kUnit = kTokens == 1 ? kKeys : kScoreWaves * kKeys;     // keys, of which a workgroup has whole numbers
  __shared__ __align__(16) bf8 frag[kTiles * kSteps * 64];       // [tile][step][lane]
  __shared__ __align__(16) float weight[kTiles * 32];
  __shared__ uint32_t start[kMostGroups + 1], sums[kScoreWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int half = lane >> 5, col = lane & 31;
  // the last position of token t, -1 where it is skipped
  auto last_of = [&](int t) {
    const int r = a.req[t], p = a.pos[t];
    return r >= 0 && r < a.R && p >= 0 && p < a.H ? p : -1;
  };
  // this workgroup's share of all groups' keys, in units: from `at` of group g on, `share` of them
  int g = blockIdx.x;
  uint32_t at = 0, share = 0xffffffffu;
  if (groups <= kMostGroups) {
    const int per = (groups + kScoreThreads - 1) / kScoreThreads, g0 = tid * per;
    uint32_t mine = 0;
    for (int i = 0; i < per; ++i)
      if (g0 + i < groups) {
        int most = -1;
#pragma unroll
        for (int j = 0; j < kTokens; ++j) {
          const int t = (g0 + i) * kTokens + j, p = t < a.n ? last_of(t) : -1;
          most = p > most ? p : most;
        }
        start[g0 + i] = mine;  // (of the thread's groups so far)
        mine += (uint32_t)((most >> 31) + 1) * ((uint32_t)most / kUnit + 1);
      }
    uint32_t sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const uint32_t x = __shfl_up(sum, d);
      if (lane >= d) sum += x;
    }
    if (lane == 63) sums[wave] = sum;
    __syncthreads();
    uint32_t before = sum - mine, all = 0;
#pragma unroll
    for (int w = 0; w < kScoreWaves; ++w) {
      if (w < wave) before += sums[w];
      all += sums[w];
    }
    for (int i = 0; i < per; ++i)
      if (g0 + i < groups) start[g0 + i] += before;
    if (tid == 0) start[groups] = all;
    __syncthreads();
    const uint32_t begin = (uint32_t)((uint64_t)all * blockIdx.x / gridDim.x);
    share = (uint32_t)((uint64_t)all * (blockIdx.x + 1) / gridDim.x) - begin;
    int low = 0, high = groups;  // the last group that starts at or before `begin`
    while (high - low > 1) {
      const int mid = (low + high) / 2;
      if (start[mid] <= begin) low = mid;
      else high = mid;
    }
    g = low;
    at = begin - start[g];
  }
  g = __builtin_amdgcn_readfirstlane(g);
  at = __builtin_amdgcn_readfirstlane(at);
  share = __builtin_amdgcn_readfirstlane(share);
  const bool even = groups <= kMostGroups;
  for (; share > 0 && g < groups; g += even ? 1 : (int)gridDim.x, at = 0) {
    const int t0 = g * kTokens;
    int req[kTokens], last[kTokens], most = -1;
#pragma unroll
    for (int i = 0; i < kTokens; ++i) {
      req[i] = t0 + i < a.n ? a.req[t0 + i] : -1;
      last[i] = t0 + i < a.n ? last_of(t0 + i) : -1;
      most = last[i] > most ? last[i] : most;
    }
    const uint32_t units = most < 0 ? 0 : (uint32_t)most / kUnit + 1;
    if (units <= at) continue;
    const uint32_t count = units - at < share ? units - at : share;  // of this group
    if (even) share -= count;
    const int lo = (int)(at * kUnit);                                 // below 2^31: a position is there
    const int64_t chunk = (int64_t)count * kUnit;
    // the queries' pieces of 8 values, kFill of a thread on their way at a time
    constexpr int kPieces = kTiles * kSteps * 64, kFill = kPieces / kScoreThreads < 8 ? kPieces / kScoreThreads : 8;
    auto fill = [&] {
      float w = 0.0f;  // (at most one of a thread)
      static_assert(kTiles * 32 <= kScoreThreads);
      if (tid < kTokens * kRows && t0 + tid / kRows < a.n && tid % kRows < a.heads)
        w = a.weights[(int64_t)(t0 + tid / kRows) * a.heads + tid % kRows];
      for (int i0 = 0; i0 < kPieces; i0 += kFill * kScoreThreads) {
        uint2 x[kFill];
        uint32_t byte[kFill];
#pragma unroll
        for (int j = 0; j < kFill; ++j) {
          const int i = i0 + j * kScoreThreads + tid;
          const int row = (i / (kSteps * 64)) * 32 + (i & 31), step = i / 64 % kSteps, t = t0 + row / kRows, h = row % kRows;
          const int d = (i >> 5 & 1) * (kDim / 2) + 8 * step;
          const bool there = t < a.n && h < a.heads && row < kTokens * kRows;
          const int64_t at = there ? (int64_t)t * a.heads + h : 0;
          x[j] = *(const uint2*)(a.q + at * kDim + d);
          byte[j] = a.q_scales[at * (kDim / kMxBlock) + d / kMxBlock];
          x[j] = there ? x[j] : uint2{};
          byte[j] = there ? byte[j] : 127;
        }
#pragma unroll
        for (int j = 0; j < kFill; ++j) {
          const float scale = __uint_as_float(byte[j] << 23);
          bf2 v[4];
          v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[j].x, scale, false);
          v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[j].x, scale, true);
          v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[j].y, scale, false);
          v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[j].y, scale, true);
          frag[i0 + j * kScoreThreads + tid] = __builtin_bit_cast(bf8, v);
        }
      }
      if (tid < kTiles * 32) weight[tid] = w;
      __syncthreads();
    };

    if (kTokens > 1) fill();
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
      const int mine = (int)(run_last - lo < chunk ? run_last - lo + 1 : chunk);  // keys of this share, from lo on
      const char* keys = a.keys + ((int64_t)r * a.H + lo) * kKeyBytes + half * (kKeyBytes / 2);
      const uint8_t* scales = a.key_scales + ((int64_t)r * a.H + lo) * (kDim / kMxBlock) + half * kBlocks;
      struct Raw { v4u keys[kJ][kRaw]; uint32_t scale[kJ]; };
      auto load = [&](int x0, Raw& raw) {
#pragma unroll
        for (int j = 0; j < kJ; ++j) {
          int x = x0 + 32 * j + col;
          x = x < mine ? x : mine - 1;
#pragma unroll
          for (int i = 0; i < kRaw; ++i) raw.keys[j][i] = *(const v4u*)(keys + (uint64_t)(uint32_t)x * kKeyBytes + 16 * i);
          if (kBlocks == 2) raw.scale[j] = *(const uint16_t*)(scales + (uint64_t)(uint32_t)x * (kDim / kMxBlock));
          else raw.scale[j] = scales[(uint64_t)(uint32_t)x * (kDim / kMxBlock)];
        }
      };
      constexpr int kStep = kScoreWaves * kKeys;
      auto score = [&](int x0, Raw& raw) {  // of the keys in raw, which then holds those kAhead steps on
        bf8 key[kJ][kSteps];
#pragma unroll
        for (int j = 0; j < kJ; ++j)
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const float scale = __uint_as_float((raw.scale[j] >> (8 * (s / 4)) & 255u) << 23);
            bf2 v[4];
            if constexpr (kFour) {
              const uint32_t x = raw.keys[j][s / 4][s % 4];
              v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 0);
              v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 1);
              v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 2);
              v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(x, scale, 3);
            } else {
              const uint32_t x = raw.keys[j][s / 2][s % 2 * 2], y = raw.keys[j][s / 2][s % 2 * 2 + 1];
              v[0] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, false);
              v[1] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, true);
              v[2] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, false);
              v[3] = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(y, scale, true);
            }
            key[j][s] = __builtin_bit_cast(bf8, v);
          }
        if (x0 + kAhead * kStep < mine) load(x0 + kAhead * kStep, raw);
        // the dot products of a tile, and what its accumulators add to the sums
        constexpr int kParts = kRows > 32 ? kRows / 32 : 1;  // tiles of a token
        float sum[2][kJ];                                    // [of a tile's two tokens of 16 heads][of the key halves]
        auto dots = [&](int tile, f16 (&acc)[kJ]) {
#pragma unroll
          for (int j = 0; j < kJ; ++j) acc[j] = f16{};
#pragma unroll
          for (int s = 0; s < kSteps; ++s) {
            const bf8 q = frag[(tile * kSteps + s) * 64 + lane];
#pragma unroll
            for (int j = 0; j < kJ; ++j) acc[j] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q, key[j][s], acc[j], 0, 0, 0);
          }
        };
        auto add = [&](int tile, const f16 (&acc)[kJ]) {
          if (kParts == 1 || tile % kParts == 0)
#pragma unroll
            for (int j = 0; j < kJ; ++j) sum[0][j] = sum[1][j] = 0.0f;
#pragma unroll
          for (int i = 0; i < kAcc; ++i) {
            const float w = weight[tile * 32 + 8 * (i / 4) + 4 * half + i % 4];
            const int of = kRows == 16 && i >= 8;
#pragma unroll
            for (int j = 0; j < kJ; ++j)
              sum[of][j] = fmaf(w, __builtin_elementwise_maximum(acc[j][i], 0.0f), sum[of][j]);
          }
          if (kParts > 1 && tile % kParts != kParts - 1) return;
#pragma unroll
          for (int k = 0; k < (kRows == 16 && kTokens > 1 ? 2 : 1); ++k) {
            const uint32_t u = __float_as_uint(sum[k][0]), v = __float_as_uint(sum[k][kJ - 1]);
            const auto x = __builtin_amdgcn_permlane32_swap(u, v, false, false);
            const float all = __uint_as_float(x[0]) + __uint_as_float(x[1]);
            const int i = kRows == 16 ? tile * 2 + k : tile / kParts;
            int p = -1;
#pragma unroll
            for (int j = 0; j < kTokens; ++j)
              if (j == i) p = last[j];
            if (i >= begin && i < end && lane < kKeys && x0 + lane <= p - lo)
              a.scores[(int64_t)(t0 + i) * a.stride + lo + x0 + lane] = all;
          }
        };
        const int first = kTokens == 1 ? 0 : begin * kRows / 32, stop = kTokens == 1 ? kTiles : (end * kRows + 31) / 32;
        f16 acc[kJ];
#pragma unroll 1
        for (int tile = first; tile < stop; ++tile) {
          int of = tile;
          // (two tiles of one token: their queries are read when they are due, not kept in registers that spill: 256 requests x
          // 2048 keys x 64 heads in 8 bits 24.8 -> 18.8 us)
          if (kRows > 32) asm volatile("" : "+s"(of));
          dots(of, acc);
          if (kRows > 32) __builtin_amdgcn_sched_barrier(0);
          add(of, acc);
        }
      };
      if (kTokens > 1 && wave * kKeys >= mine) continue;
      Raw raw[kAhead];
#pragma unroll
      for (int i = 0; i < kAhead; ++i)
        if (wave * kKeys + i * kStep < mine) load(wave * kKeys + i * kStep, raw[i]);
      if (kTokens == 1) fill();  // (with the first keys on their way)
      for (int x0 = wave * kKeys; x0 < mine; x0 += kAhead * kStep) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          if (x0 + i * kStep < mine) score(x0 + i * kStep, raw[i]);
      }
    }
    if (share > 0) __syncthreads();  // the queries are read, and the next group's may take their place
  }
}

template <int kDim, bool kFour, int kRows, int kTokens>
hipError_t launch(const ScoreArgs& a, hipStream_t s) {
  const int groups = (int)(((int64_t)a.n + kTokens - 1) / kTokens);
  const int64_t units = (int64_t)groups * a.H / kKeys + groups;  // at most
  constexpr int kFull = 2 * 256;  // workgroups that the card holds
  const int blocks = groups > kMostGroups ? (groups < kMostBlocks ? groups : kMostBlocks) : units < kFull ? (int)units : kFull;
  hipLaunchKernelGGL((score_kernel<kDim, kFour, kRows, kTokens>), dim3(blocks), dim3(kScoreThreads), 0, s, a, groups);
  return hipGetLastError();
}

template <int kDim, bool kFour>
hipError_t launch_heads_of(const ScoreArgs& a, hipStream_t s) {
  // Tokens in groups of up to 8, which share their request's keys, where there are two for each of the context's requests (64
  // requests x 8000 keys x 32 heads in 8 bits, us in groups / one by one: 1 token 19.7 / 15.5, 2 20.8 / 24.2, 4 26.4 / 42.8, 8
  // 41.8 / 79.9; a chunk of one request in a context of many pays for that: 128 tokens behind 16000 keys 26 / 41)
  const bool many = a.n >= 2 * a.R;
  if (a.heads <= 16) return many ? launch<kDim, kFour, 16, 8>(a, s) : launch<kDim, kFour, 16, 1>(a, s);
  if (a.heads <= 32) return many ? launch<kDim, kFour, 32, 4>(a, s) : launch<kDim, kFour, 32, 1>(a, s);
  return many ? launch<kDim, kFour, 64, 2>(a, s) : launch<kDim, kFour, 64, 1>(a, s);
}

}  // namespace

hipError_t launch_score(const ScoreArgs& a, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  if (a.dim == 64) return a.type ? launch_heads_of<64, true>(a, s) : launch_heads_of<64, false>(a, s);
  return a.type ? launch_heads_of<128, true>(a, s) : launch_heads_of<128, false>(a, s);
}

}  // namespace hs
