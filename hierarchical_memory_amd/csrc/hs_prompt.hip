// A prompt's latent attention, expanded form, over ragged sequences (gfx950): key j of head h is [kv_j,h nope part | rope
// part of token j], its value the rest of kv_j,h.
//
//   s = scale * q . key,   o = sum_j p_j value_j / sum_j p_j,   p_j = 2^(s_j log2 e - m)   (m a running maximum)
//
// One pass over the keys. A workgroup of four waves takes 256 (128) queries of one sequence and head, 64 (32) to a wave.
// Matrix instructions do both products transposed, so that a query is a lane's column in both and its maximum, sum and
// rescaling stay inside the lane:
//   S^T[key][query]  = K Q^T     A: keys from LDS, B: the queries, kept in registers
//   O^T[dim][query] += V^T P^T   A: values read through the transposing LDS load, B: the weights as S^T left them
// (a lane half h holds the keys 8 i + 4 h + 0..3 of S^T; the second product takes its keys in that order).
// There is one wave to a SIMD, so the two pipes are kept busy from within it: a step of 32 keys computes the next step's
// scores between the exponentials of its own, and takes their maximum between its products with the values.
#include "hs_latent.h"
#include "hs_mfma.h"

#include <utility>

namespace hs {

namespace {

__device__ __align__(16) uint4 zero_key[64];  // what a tile holds behind the last key

// DN, P: nope and rope values of a key, DV: of a value. kSets: column sets of 32 queries of a wave.
template <int DN, int P, int DV, int kSets>
struct PromptShape {
  static constexpr int kWaves = 4;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kPer = DV == 256 ? 1 : 2;      // steps of 32 keys to a tile
  static constexpr int kKeys = 32 * kPer;
  static constexpr int kDepth = kPer == 2 ? 3 : 4;    // tiles in LDS: one or two in use, the others on their way
  static constexpr int kQueries = 32 * kSets * kWaves;
  static constexpr int kSteps = (DN + P) / 16;
  static constexpr int kKeyCols = DN / 64 + 1, kValueCols = DV / 64;  // groups of 64 columns (the last key group: rope)
  static constexpr int kColBytes = kKeys * 128;
  static constexpr int kTileBytes = (kKeyCols + kValueCols) * kColBytes;
  static constexpr int kLoads = kPer * (kKeyCols + kValueCols);  // of a lane, for a tile
  static constexpr uint32_t kLds = kDepth * kTileBytes;
};

// Waits for the oldest of the tiles asked for, `later` of which (kLoads loads each) may still be on their way.
template <int kLoads, int kMost>
__device__ __forceinline__ void wait_tile(int later) {
  if constexpr (kMost > 0) {
    if (later >= kMost) return wait_loads_and_meet<kLoads * kMost>();
    return wait_tile<kLoads, kMost - 1>(later);
  }
  wait_loads_and_meet<0>();
}

__device__ __forceinline__ int cut(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// The sequence of query tile `id` and the tile's number in it: a scan over the sequences' tile counts, one to a thread.
template <int kQueries, int kWaves>
__device__ __forceinline__ bool find_tile(const PromptArgs& a, int id, int* seq, int* tile, int* sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int before = 0;
  for (int r0 = 0; r0 < a.R; r0 += 64 * kWaves) {
    const int r = r0 + tid;
    int c = 0;
    if (r < a.R) {
      const int n = cut(a.cu_q[r + 1], a.n_q) - cut(a.cu_q[r], a.n_q);
      c = n > 0 ? (n + kQueries - 1) / kQueries : 0;
    }
    int x = c;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int y = __shfl_up(x, d);
      if (lane >= d) x += y;
    }
    if (lane == 63) sh[wave] = x;
    if (tid == 0) sh[kWaves] = -1;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) x += sh[w];
      total += sh[w];
    }
    if (id >= before + x - c && id < before + x) {
      sh[kWaves] = r;
      sh[kWaves + 1] = id - (before + x - c);
    }
    __syncthreads();
    const int found = sh[kWaves], at = sh[kWaves + 1];
    __syncthreads();
    if (found >= 0) {
      *seq = __builtin_amdgcn_readfirstlane(found);
      *tile = __builtin_amdgcn_readfirstlane(at);
      return true;
    }
    before += total;
  }
  return false;
}

template <int kBegin, int kGroupBytes, int... G>
__device__ __forceinline__ void load_part(const char* row, uint32_t lds, std::integer_sequence<int, G...>) {
  (load_to_lds<kBegin + 128 * G>(row, lds + G * kGroupBytes), ...);
}

template <int DN, int P, int DV, int kSets>
__global__ __launch_bounds__((PromptShape<DN, P, DV, kSets>::kThreads)) void prompt_kernel(PromptArgs a, int slots) {
  using S = PromptShape<DN, P, DV, kSets>;
  constexpr int kWaves = S::kWaves;
  constexpr int kBlocks = DV / 32;
  extern __shared__ __align__(1024) char smem[];
  __shared__ int sh[kWaves + 2];
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(HS_LDS char*)smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int h = blockIdx.x % a.heads, split = blockIdx.x / a.heads;
  int kat[4], vat[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) kat[i] = col * 128 + (((2 * i + half) ^ swizzle(col)) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) vat[i / 2][i % 2] = across_place(lane, i / 2, 8 * (i % 2)) + S::kKeyCols * S::kColBytes;
  const float scale = scale_of(a.scale);
  const uint32_t sign = a.scale < 0.0f ? kSigns : 0u;

  for (int slot = blockIdx.y; slot < slots; slot += gridDim.y) {
    // the last tiles of a sequence see the most keys, and go first
    int seq, qt;
    if (!find_tile<S::kQueries, kWaves>(a, slots - 1 - slot, &seq, &qt, sh)) continue;
    const int q0 = cut(a.cu_q[seq], a.n_q), nq = cut(a.cu_q[seq + 1], a.n_q) - q0;
    const int k0 = cut(a.cu_k[seq], a.n_k);
    int nk = cut(a.cu_k[seq + 1], a.n_k) - k0;
    if (nk < 0) nk = 0;
    const int first = qt * S::kQueries;
    // keys that the workgroup's last query sees, and its part of their tiles
    const int last_q = first + S::kQueries < nq ? first + S::kQueries - 1 : nq - 1;
    const int end = a.causal ? cut(nk - nq + last_q + 1, nk) : nk;
    const int all = (end + S::kKeys - 1) / S::kKeys;
    const int t0 = (int)((int64_t)all * split / a.splits), t1 = (int)((int64_t)all * (split + 1) / a.splits);

    const int wq = first + wave * 32 * kSets;  // the wave's first query
    int limit[kSets];                           // keys that the lane's queries see
    bf8 q[kSets][S::kSteps];
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
      const int i = wq + 32 * g + col, j = i < nq ? i : nq - 1;
      limit[g] = a.causal ? cut(nk - nq + j + 1, nk) : nk;
      const __bf16* src = (const __bf16*)a.q + ((size_t)(q0 + j) * a.heads + h) * (DN + P) + 8 * half;
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) {
        q[g][s] = turned(*(const v4u*)(src + 16 * s), sign);
      }
    }
#pragma unroll
    for (int g = 0; g < kSets; ++g)
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) asm volatile("" : "+a"(q[g][s]));
    // of the wave: keys that all of its queries see, and that any does
    const int lo = a.causal ? cut(nk - nq + wq + 1, nk) : nk;
    const int hi = a.causal ? cut(nk - nq + wq + 32 * kSets, nk) : nk;

    f16 o[kSets][kBlocks];
    float m[kSets], sum[kSets], rsum[kSets];
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[g][b] = f16{};
      m[g] = -INFINITY;
      sum[g] = rsum[g] = 0.0f;
    }

    // the lane's chunk of one key of every tile
    const int mine = 8 * wave + (lane >> 3), place = (lane & 7) ^ swizzle(mine);
    const char* kv = (const char*)a.kv + ((size_t)k0 * a.heads + h) * (2 * (DN + DV)) + 16 * place;
    const char* kr = (const char*)a.krope + (size_t)k0 * a.rope_stride * 2 + 16 * (P == 64 ? place : place & 3);
    const size_t kv_row = (size_t)a.heads * (2 * (DN + DV)), kr_row = (size_t)a.rope_stride * 2;
    int place_in = 0, place_out = 0;  // of the next tile to load, and to use, of kDepth
    auto load = [&](int t) {
#pragma unroll
      for (int i = 0; i < S::kPer; ++i) {
        const uint32_t to = lds0 + place_in * S::kTileBytes + 4096 * i + 1024 * wave;
        const int j = t * S::kKeys + 32 * i + mine;
        const char* p = j < nk ? kv + j * kv_row : (const char*)zero_key + 16 * place;
        const char* r = j < nk ? kr + j * kr_row : (const char*)zero_key;
        load_part<0, S::kColBytes>(p, to, std::make_integer_sequence<int, DN / 64>());
        load_to_lds<0>(r, to + DN / 64 * S::kColBytes);
        load_part<2 * DN, S::kColBytes>(p, to + S::kKeyCols * S::kColBytes, std::make_integer_sequence<int, DV / 64>());
      }
      place_in = place_in + 1 < S::kDepth ? place_in + 1 : 0;
    };
    // tile t is in LDS for every wave; the one that was used before it is left by all, and loaded anew
    const char* tile = smem;
    auto next_tile = [&](int t) {
      wait_tile<S::kLoads, S::kDepth - 3>(t1 - 1 - t);
      if (t + S::kDepth - 2 < t1) load(t + S::kDepth - 2);
      tile = smem + place_out * S::kTileBytes;
      place_out = place_out + 1 < S::kDepth ? place_out + 1 : 0;
    };

    f16 s[2][kSets];  // scores of two steps
    float top[kSets];
    // what one k-step of the first product of step i adds to its scores
    constexpr int kSet = 4;  // k-steps whose keys are read before the steps before them are multiplied
    bf8 k[2][kSet];
    auto read_keys = [&](const char* at, int from) {
#pragma unroll
      for (int i = 0; i < kSet; ++i)
        if (from + i < S::kSteps) k[from / kSet & 1][i] = *(const bf8*)(at + kat[i] + S::kColBytes * (from / kSet));
    };
    auto score = [&](f16 (&to)[kSets], int j) {
#pragma unroll
      for (int g = 0; g < kSets; ++g)
        to[g] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[j / kSet & 1][j % kSet], q[g][j], to[g], 0, 0, 0);
    };
    // the masked scores of step i, and their maximum so far
    auto mask = [&](f16 (&x)[kSets], int i) {
      if (32 * i + 32 <= lo) return;
#pragma unroll
      for (int g = 0; g < kSets; ++g)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          x[g][e] = 32 * i + 8 * (e / 4) + e % 4 + 4 * half < limit[g] ? x[g][e] : -INFINITY;
    };
    // whether the maximum moves by the scores of a step, and its move
    auto raises = [&]() {
      bool any = false;
#pragma unroll
      for (int g = 0; g < kSets; ++g) {
        top[g] = max_of_halves(top[g]) * scale;
        any |= top[g] > m[g] + kSlack;
      }
      return __any(any);
    };
    auto raise = [&]() {
#pragma unroll
      for (int g = 0; g < kSets; ++g) {
        const float to = top[g] > m[g] + kSlack ? top[g] : m[g];
        const float c = m[g] == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m[g] - to);
        if (__any(m[g] > -INFINITY && c != 1.0f)) {
          sum[g] *= c;
          rsum[g] *= c;
#pragma unroll
          for (int b = 0; b < kBlocks; ++b) o[g][b] *= c;
        }
        m[g] = to;
      }
    };
    const int mine_end = (hi + 31) / 32;  // the wave's steps end here; the others' loads and barriers go on
    // step i with its scores in x; those of step i + 1 go to y
    auto step = [&](int i, f16 (&x)[kSets], f16 (&y)[kSets]) {
      const char* values = tile + 4096 * (i % S::kPer);
      if ((i + 1) % S::kPer == 0 && i + 1 < S::kPer * t1) next_tile((i + 1) / S::kPer);
      if (i >= mine_end) return;
      const char* keys = tile + 4096 * ((i + 1) % S::kPer);
      bf8 p[kSets][2];
      float m0[kSets];
#pragma unroll
      for (int g = 0; g < kSets; ++g) m0[g] = m[g] == -INFINITY ? 0.0f : m[g];
      constexpr int kReads = 3;  // blocks of values that are read before the products of the block before them end
      bf8 v[kReads][2];
      auto read_values = [&](int b) {
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const char* at = values + S::kColBytes * (b >> 1) + 2048 * j;
          v[b % kReads][j] = read_across(at + vat[b & 1][0], at + vat[b & 1][1]);
        }
      };
      const bool more = i + 1 < mine_end && i + 1 < S::kPer * t1;
      if (more) {
        constexpr int kPairs = 8 * kSets, kFirst = kPairs / 4;  // weights, and those before the keys are here
        auto weigh_some = [&](int from, int to) {
          // (the pins keep them between the products around them)
#pragma unroll
          for (int g = 0; g < kSets; ++g) asm volatile("" : "+v"(m0[g]));
#pragma unroll
          for (int e = from; e < to; ++e)
            weigh_pair(x[e / 8][e % 8 * 2], x[e / 8][e % 8 * 2 + 1], scale, m0[e / 8], p[e / 8][e % 8 / 4], e % 4 * 2,
                       sum[e / 8], rsum[e / 8]);
#pragma unroll
          for (int g = 0; g < kSets; ++g) asm volatile("" : "+v"(sum[g]), "+v"(rsum[g]));
          __builtin_amdgcn_sched_barrier(0);
        };
#pragma unroll
        for (int g = 0; g < kSets; ++g) y[g] = f16{};
        read_keys(keys, 0);
        weigh_some(0, kFirst);
#pragma unroll
        for (int j = 0; j < S::kSteps; ++j) {
          if (j % kSet == 0) read_keys(keys, j + kSet);
          if (j == S::kSteps - kSet) read_values(0);
          if (j == S::kSteps - kSet / 2) read_values(1);
          score(y, j);
          weigh_some(kFirst + j * (kPairs - kFirst) / S::kSteps, kFirst + (j + 1) * (kPairs - kFirst) / S::kSteps);
        }
        mask(y, i + 1);
      } else {
        read_values(0);
        read_values(1);
#pragma unroll
        for (int e = 0; e < 8 * kSets; ++e)
          weigh_pair(x[e / 8][e % 8 * 2], x[e / 8][e % 8 * 2 + 1], scale, m0[e / 8], p[e / 8][e % 8 / 4], e % 4 * 2,
                     sum[e / 8], rsum[e / 8]);
      }
      bool up = false;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) {
        if (b + 2 < kBlocks) read_values(b + 2);
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int g = 0; g < kSets; ++g)
            o[g][b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[b % kReads][j], p[g][j], o[g][b], 0, 0, 0);
        // the maximum of the scores (behind the wave's last step they are old ones, and it is not used)
        if (b == 0) {
#pragma unroll
          for (int g = 0; g < kSets; ++g) {
            top[g] = y[g][0];
#pragma unroll
            for (int e = 1; e < 16; ++e) top[g] = fmaxf(top[g], y[g][e]);
            asm volatile("" : "+v"(top[g]));
          }
        }
        if (b == 1) up = raises();
        __builtin_amdgcn_sched_barrier(0);
      }
      if (more && up) raise();
    };

    if (t0 < t1) {
#pragma unroll
      for (int i = 0; i < S::kDepth - 2; ++i)
        if (t0 + i < t1) load(t0 + i);
      next_tile(t0);
      const int begin = S::kPer * t0;
      if (begin < mine_end) {
#pragma unroll
        for (int g = 0; g < kSets; ++g) s[0][g] = f16{};
        const char* keys = tile;
        read_keys(keys, 0);
#pragma unroll
        for (int j = 0; j < S::kSteps; ++j) {
          if (j % kSet == 0) read_keys(keys, j + kSet);
          score(s[0], j);
          __builtin_amdgcn_sched_barrier(0);
        }
        mask(s[0], begin);
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
          top[g] = s[0][g][0];
#pragma unroll
          for (int e = 1; e < 16; ++e) top[g] = fmaxf(top[g], s[0][g][e]);
        }
        if (raises()) raise();
      }
      for (int i = begin; i < S::kPer * t1; i += 2) {
        step(i, s[0], s[1]);
        if (i + 1 < S::kPer * t1) step(i + 1, s[1], s[0]);
      }
    }
    asm volatile("s_barrier" ::: "memory");  // every wave has left the tiles

#pragma unroll
    for (int g = 0; g < kSets; ++g) {
      sum[g] += __shfl_xor(sum[g], 32);
      rsum[g] += __shfl_xor(rsum[g], 32);
      const int i = wq + 32 * g + col;
      if (i >= nq) continue;
      const size_t qh = (size_t)(q0 + i) * a.heads + h;
      if (a.splits == 1) {
        const float f = rsum[g] > 0.0f ? 1.0f / rsum[g] : rsum[g] == 0.0f ? 0.0f : rsum[g];
        __bf16* dst = (__bf16*)a.o + qh * DV + 4 * half;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            bf4 v;
#pragma unroll
            for (int j = 0; j < 4; ++j) v[j] = (__bf16)(o[g][b][4 * c + j] * f);
            *(bf4*)(dst + 32 * b + 8 * c) = v;
          }
        if (a.lse && half == 0)
          a.lse[qh] = sum[g] > 0.0f ? m[g] * kLn2 + logf(sum[g]) : sum[g] == 0.0f ? -INFINITY : sum[g];
        continue;
      }
      // partial results: (m, sum, rsum, -) and the values of every query, head and part
      const size_t ph = qh * a.splits + split;
      if (half == 0) *(f4*)(a.work + ph * 4) = f4{m[g], sum[g], rsum[g], 0.0f};
      float* dst = a.work + (size_t)a.n_q * a.heads * a.splits * 4 + ph * DV + 4 * half;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *(f4*)(dst + 32 * b + 8 * c) = f4{o[g][b][4 * c], o[g][b][4 * c + 1], o[g][b][4 * c + 2], o[g][b][4 * c + 3]};
    }
  }
}

// Joins the parts of each query and head in their order: one wave for both, DV / 64 values a lane.
template <int DV>
__global__ __launch_bounds__(256) void join_prompt_kernel(PromptArgs a) {
  constexpr int kPer = DV / 64;
  const int lane = threadIdx.x & 63;
  // rows behind the last sequence have no parts
  const size_t n = (size_t)cut(a.cu_q[a.R], a.n_q) * a.heads;
  for (size_t qh = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6); qh < n; qh += (size_t)gridDim.x * 4) {
    const f4* st = (const f4*)a.work + qh * a.splits;
    float m = -INFINITY;
    for (int s = 0; s < a.splits; ++s) m = fmaxf(m, st[s][0]);
    const float m0 = m == -INFINITY ? 0.0f : m;
    float sum = 0.0f, rsum = 0.0f, o[kPer] = {};
    const float* src = a.work + (size_t)a.n_q * a.heads * a.splits * 4 + qh * a.splits * DV + lane * kPer;
    for (int s = 0; s < a.splits; ++s) {
      const f4 v = st[s];
      const float c = __builtin_amdgcn_exp2f(v[0] - m0);
      sum += c * v[1];
      rsum += c * v[2];
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] += c * src[(size_t)s * DV + i];
    }
    const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
    __bf16* dst = (__bf16*)a.o + qh * DV + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[i] = (__bf16)(o[i] * f);
    if (a.lse && lane == 0) a.lse[qh] = sum > 0.0f ? m * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
  }
}

constexpr int sets_of(int value) { return value == 256 ? 1 : 2; }

template <int DN, int P, int DV>
hipError_t launch(const PromptArgs& a, hipStream_t s) {
  constexpr int kSets = sets_of(DV);
  using S = PromptShape<DN, P, DV, kSets>;
  constexpr uint32_t lds = S::kLds;
  // every sequence but one may leave a tile part empty
  const int64_t slots = ((int64_t)a.n_q + S::kQueries - 1) / S::kQueries + a.R - 1;
  hipLaunchKernelGGL((prompt_kernel<DN, P, DV, kSets>), dim3(a.heads * a.splits, (int)(slots < 65535 ? slots : 65535)),
                     dim3(S::kThreads), lds, s, a, (int)slots);
  if (a.splits > 1) {
    const uint64_t blocks = ((uint64_t)a.n_q * a.heads + 3) / 4;
    hipLaunchKernelGGL(join_prompt_kernel<DV>, dim3((int)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <int DN, int P, int DV>
hipError_t set_lds() {
  return hipFuncSetAttribute((const void*)prompt_kernel<DN, P, DV, sets_of(DV)>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             (int)PromptShape<DN, P, DV, sets_of(DV)>::kLds);
}

}  // namespace

int prompt_splits(int R, int n_q, int n_k, int heads, int value) {
  const int queries = value == 256 ? 128 : 256;
  const int64_t groups = ((int64_t)n_q + queries - 1) / queries * heads;
  if (groups <= 0) return 1;
  int64_t s = 256 / groups;
  const int64_t most = n_k / R / 512;
  if (s > most) s = most;
  if (s > 16) s = 16;
  return s < 1 ? 1 : (int)s;
}

uint64_t prompt_work_bytes(int R, int n_q, int n_k, int heads, int value) {
  const uint64_t s = (uint64_t)prompt_splits(R, n_q, n_k, heads, value);
  return s == 1 ? 0 : (uint64_t)n_q * heads * s * (16 + 4ull * value);
}

hipError_t set_prompt_lds() {
  for (const auto f : {set_lds<64, 32, 64>, set_lds<64, 64, 64>, set_lds<128, 32, 128>, set_lds<128, 64, 128>,
                       set_lds<192, 32, 256>, set_lds<192, 64, 256>}) {
    const hipError_t e = f();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_prompt(const PromptArgs& a, hipStream_t s) {
  if (a.n_q <= 0) return hipSuccess;
  const bool more = a.rope == 64;
  if (a.value == 64) return more ? launch<64, 64, 64>(a, s) : launch<64, 32, 64>(a, s);
  if (a.value == 128) return more ? launch<128, 64, 128>(a, s) : launch<128, 32, 128>(a, s);
  return more ? launch<192, 64, 256>(a, s) : launch<192, 32, 256>(a, s);
}

}  // namespace hs
