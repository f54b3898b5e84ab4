// A prompt's latent attention, expanded form, over ragged sequences (gfx950): key j of head h is [kv_j,h nope part | rope
// part of token j], its value the rest of kv_j,h.
//
//   s = scale * q . key,   o = sum_j p_j value_j / sum_j p_j,   p_j = 2^(s_j log2 e - m)   (m a running maximum)
//
// One pass over the keys. A workgroup of four waves takes 256 or 128 queries of one sequence and head, 64 or 32 to a wave.
// Matrix instructions do both products transposed, so that a query is a lane's column in both and its maximum, sum and
// rescaling stay inside the lane:
//   S^T[key][query]  = K Q^T     A: keys from LDS, B: the queries, kept in registers
//   O^T[dim][query] += V^T P^T   A: values read through the transposing LDS load, B: the weights as S^T left them
// (a lane half h holds the keys 8 i + 4 h + 0..3 of S^T; the second product takes its keys in that order).
// There are only one or two waves to a SIMD, so the two pipes are kept busy from within a wave: a step of 32 keys computes the
// next step's scores between the exponentials of its own, and takes their maximum between its products with the values.
//
// What bounds it: the matrix units and the card's power. 8192 tokens x 16 heads (128 + 64 / 128 values, causal) take 353 to
// 371 us on different cards, 970 to 925 TFLOP/s, where a plain matrix product of the library reaches 1200; with
// 32 queries to a wave they take 414 (twice the LDS reads for a product). 256 values allow only 32: one prompt of 8192 x 16
// heads takes 600 to 607 us (910 TFLOP/s). 64 values: 257 us for 16 heads, 480 to 487 for 32 (800 and 850 TFLOP/s). 4 chunks of
// 512 tokens behind 4K to 16K x 8 heads x 256 values take 226 to 234 us (740 TFLOP/s): their tiles' keys are cut into 1, 2, 2
// and 3 parts, and the longest part has 6208 keys where an even share is 5216, which alone is 217 us. Short prompts wait for one
// workgroup's chain: the search of its item and its first tiles, about 6 us, and its steps one after another (8 of up to 300
// tokens x 16 heads: 15 us, 7 of them for 300 keys).
#include "hs_latent.h"
#include "hs_mfma.h"

#include <math.h>

#include <utility>

namespace hs {

namespace {

typedef unsigned short us8 __attribute__((ext_vector_type(8)));

constexpr int kLeastKeys = 512;  // keys of a part of a sequence: below, the parts' own costs are more than they save

__device__ __align__(16) uint4 zero_key[64];  // what a tile holds behind the last key

// DN, P: nope and rope values of a key, DV: of a value. kSets: column sets of 32 queries of a wave.
template <int DN, int P, int DV, int kSets>
struct PromptShape {
  static constexpr int kWaves = 4;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kPer = DV == 64 || kSets == 2 ? 2 : 1;  // steps of 32 keys to a tile
  static constexpr int kKeys = 32 * kPer;
  static constexpr int kDepth = DV == 256 ? 4 : 3;    // tiles in LDS: one or two in use, the others on their way
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

// whether bf16 bits are infinite or NaN
__device__ __forceinline__ bool is_odd(unsigned short x) { return (x & 0x7f80) == 0x7f80; }

__device__ __forceinline__ int cut(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// Sums of kN values over the workgroup, in the same order in every workgroup. sh: kN * kWaves values.
template <int kN, int kWaves>
__device__ __forceinline__ void block_sums(float (&x)[kN], float* sh) {
#pragma unroll
  for (int i = 0; i < kN; ++i) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) x[i] += __shfl_xor(x[i], d);
    if ((threadIdx.x & 63) == 0) sh[i * kWaves + (threadIdx.x >> 6)] = x[i];
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kN; ++i) {
    x[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) x[i] += sh[i * kWaves + w];
  }
  __syncthreads();
}

struct Item {  // a workgroup's share: part `part` of the keys of query tile `tile` of a sequence
  int tile, part, parts;
  int q0, nq, k0, nk;  // of the sequence: its first query and key, and how many of both
};

// Item `id` of a head: the sequences from the last to the first, each one's tiles from the last (it sees the most keys) to
// the first, each tile's parts. A sequence's keys are cut into as many parts as makes about a.items of equal length of all
// sequences' tiles, at most a.splits: the finest of four lengths that makes no more (one more would wait for a round of
// its own; 4 chunks of 512 tokens behind 4K to 16K x 8 heads x 256 values 274 -> 227 us against equal counts of parts).
// A scan over the sequences' item counts, one to a thread. sh[4 * kWaves] is 0 behind it.
template <int kQueries, int kWaves>
__device__ __forceinline__ bool find_item(const PromptArgs& a, int id, Item* it, int* sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  struct Sequence {
    int q0, nq, k0, nk, tiles;
  };
  auto sequence = [&](int r) {
    Sequence q{};
    if (r >= 0) {
      const int q1 = a.cu_q[r + 1], k1 = a.cu_k[r + 1];
      q.q0 = cut(a.cu_q[r], a.n_q);
      q.k0 = cut(a.cu_k[r], a.n_k);
      q.nq = cut(q1, a.n_q) - q.q0;
      q.nk = cut(k1, a.n_k) - q.k0;
      q.nk = q.nk > 0 ? q.nk : 0;
      q.tiles = q.nq > 0 ? (q.nq + kQueries - 1) / kQueries : 0;
    }
    return q;
  };
  float per = 0.0f;  // parts to a key
  auto parts_of = [&](int keys, float per) {
    const int parts = (int)((float)keys * fminf(per, 1.0f / kLeastKeys) + 0.5f);
    return parts < 1 ? 1 : parts > a.splits ? a.splits : parts;
  };
  if (a.splits > 1) {
    float all[1] = {};
    for (int r = a.R - 1 - tid; r >= 0; r -= 64 * kWaves) {
      const Sequence q = sequence(r);
      all[0] += (float)q.tiles * (float)q.nk;
    }
    block_sums<1, kWaves>(all, (float*)sh);
    per = (float)a.items / fmaxf(all[0], 1.0f);
    float count[4] = {};
    for (int r = a.R - 1 - tid; r >= 0; r -= 64 * kWaves) {
      const Sequence q = sequence(r);
#pragma unroll
      for (int i = 0; i < 4; ++i) count[i] += (float)q.tiles * (float)parts_of(q.nk, per * (1.1f - 0.1f * i));
    }
    block_sums<4, kWaves>(count, (float*)sh);
    const float most = (float)a.items;
    per *= count[0] <= most ? 1.1f : count[1] <= most ? 1.0f : count[2] <= most ? 0.9f : 0.8f;
  }
  int before = 0;
  for (int r0 = a.R - 1; r0 >= 0; r0 -= 64 * kWaves) {
    const Sequence q = sequence(r0 - tid);
    const int parts = a.splits > 1 ? parts_of(q.nk, per) : 1;
    const int c = q.tiles * parts;
    // inclusive sums over the wave by lane shifts: 1, 2, 4, 8 in each row of 16, then lane 15 into the rows 1 and 3, lane 31
    // into the rows 2 and 3
    int x = c;
    x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false);
    x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false);
    if (lane == 63) sh[wave] = x;
    if (tid == 0) sh[kWaves] = 0;
    __syncthreads();
    int total = 0;
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) x += sh[w];
      total += sh[w];
    }
    if (id >= before + x - c && id < before + x) {
      const int at = id - (before + x - c);
      const int v[7] = {parts, q.tiles - 1 - at / parts, at % parts, q.q0, q.nq, q.k0, q.nk};
      for (int i = 0; i < 7; ++i) sh[kWaves + i] = v[i];
      sh[4 * kWaves] = 0;
    }
    __syncthreads();
    int v[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) v[i] = __builtin_amdgcn_readfirstlane(sh[kWaves + i]);
    __syncthreads();
    if (v[0] > 0) {
      *it = Item{v[1], v[2], v[0], v[3], v[4], v[5], v[6]};
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
  __shared__ int sh[4 * kWaves + 1];
  static_assert(4 * kWaves >= kWaves + 7);
  const uint32_t lds0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(HS_LDS char*)smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const int h = blockIdx.x;
  int kat[4], vat[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) kat[i] = col * 128 + (((2 * i + half) ^ swizzle(col)) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) vat[i / 2][i % 2] = across_place(lane, i / 2, 8 * (i % 2)) + S::kKeyCols * S::kColBytes;
  const float scale = scale_of(a.scale);
  const uint32_t sign = a.scale < 0.0f ? kSigns : 0u;

  for (int slot = blockIdx.y; slot < slots; slot += gridDim.y) {
    Item it;
    if (!find_item<S::kQueries, kWaves>(a, slot, &it, sh)) return;
    const int q0 = it.q0, nq = it.nq, k0 = it.k0, nk = it.nk;
    const int first = it.tile * S::kQueries;
    // keys that the workgroup's last query sees, and its part of their tiles
    const int last_q = first + S::kQueries < nq ? first + S::kQueries - 1 : nq - 1;
    const int end = a.causal ? cut(nk - nq + last_q + 1, nk) : nk;
    const int all = (end + S::kKeys - 1) / S::kKeys;
    const int t0 = (int)((int64_t)all * it.part / it.parts), t1 = (int)((int64_t)all * (it.part + 1) / it.parts);

    const int wq = first + wave * 32 * kSets;  // the wave's first query
    // of the wave: keys that all of its queries see, and that any does
    const int lo = a.causal ? cut(nk - nq + wq + 1, nk) : nk;
    const int hi = a.causal ? cut(nk - nq + wq + 32 * kSets, nk) : nk;

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
    // (128 queries: on their way with the queries, 64 prompts of up to 300 tokens 57 -> 55 us; with 256 the registers that
    // wait for both cost more than they hide, 8192 tokens x 16 heads 360 -> 370)
    auto load_first = [&]() {
#pragma unroll
      for (int i = 0; i < S::kDepth - 2; ++i)
        if (t0 + i < t1) load(t0 + i);
    };
    if constexpr (kSets == 1) load_first();

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
      if (a.scale == 0.0f) zero_scaled(q[g]);
    }
#pragma unroll
    for (int g = 0; g < kSets; ++g)
#pragma unroll
      for (int s = 0; s < S::kSteps; ++s) asm volatile("" : "+a"(q[g][s]));
    f16 o[kSets][kBlocks];
    float m[kSets], sum[kSets], rsum[kSets];
#pragma unroll
    for (int g = 0; g < kSets; ++g) {
#pragma unroll
      for (int b = 0; b < kBlocks; ++b) o[g][b] = f16{};
      m[g] = -INFINITY;
      sum[g] = rsum[g] = 0.0f;
    }

    // An infinite value or a NaN of a key that some of the workgroup's queries see and others do not would reach those too (a
    // weight of zero makes it NaN): the lane takes such ones out of its chunks of the tile, and the queries that see them
    // get them at the end. Only tiles that some query does not see whole are looked through (8192 tokens x 16 heads: no
    // difference; 8 prompts of up to 300 tokens, where all are, 14.5 -> 15.2 us).
    const int all_see = a.causal ? cut(nk - nq + first + 1, nk) : nk;  // keys that every query of the workgroup sees
    auto take_odd = [&](char* at) {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      auto chunk = [&](int i) {
        return (us8*)(at + (S::kKeyCols + i / S::kPer) * S::kColBytes + 4096 * (i % S::kPer) + 1024 * wave + 16 * lane);
      };
      us8 most{};
#pragma unroll
      for (int i = 0; i < S::kPer * S::kValueCols; ++i)
        most = __builtin_elementwise_max(most, *chunk(i) & (unsigned short)0x7fff);
      // 0x7f7f: the largest number; what is above it has another bit
      const v4u m = (v4u)__builtin_elementwise_max(most, us8{} + (unsigned short)0x7f7f);
      if ((m[0] | m[1] | m[2] | m[3]) == 0x7f7f7f7fu) return;
#pragma unroll 1
      for (int i = 0; i < S::kPer * S::kValueCols; ++i) {
        us8 x = *chunk(i);
#pragma unroll
        for (int n = 0; n < 8; ++n) x[n] = is_odd(x[n]) ? 0 : x[n];
        *chunk(i) = x;
      }
      sh[4 * kWaves] = 1;
    };
    // tile t is in LDS for every wave; the one that was used before it is left by all, and loaded anew
    const char* tile = smem;
    auto next_tile = [&](int t) {
      if (S::kKeys * (t + 1) > all_see) take_odd(smem + place_out * S::kTileBytes);
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
        top[g] = max_of_halves(top[g]);
        any |= (top[g] - m[g]) * scale > kSlack;
      }
      return __any(any);
    };
    auto raise = [&]() {
#pragma unroll
      for (int g = 0; g < kSets; ++g) {
        const float to = (top[g] - m[g]) * scale > kSlack ? top[g] : m[g];
        const float c = rebase(m[g], to, scale);
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
    // step i (odd: of a pair's second) with its scores in x; those of step i + 1 go to y
    auto step = [&](auto odd, int i, f16 (&x)[kSets], f16 (&y)[kSets]) {
      constexpr int kAt = odd.value % S::kPer, kNext = (odd.value + 1) % S::kPer;  // place in the tile
      const char* values = tile + 4096 * kAt;
      if (kNext == 0 && i + 1 < S::kPer * t1) next_tile((i + 1) / S::kPer);
      if (i >= mine_end) return;
      const char* keys = tile + 4096 * kNext;
      bf8 p[kSets][2];
      float m0[kSets];
#pragma unroll
      for (int g = 0; g < kSets; ++g) m0[g] = m[g] == -INFINITY ? 0.0f : m[g] * scale;
      bool any_far = false;
#pragma unroll
      for (int g = 0; g < kSets; ++g) any_far |= fabsf(m0[g]) >= kFar;
      if (__any(any_far)) {
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
          const bool far = fabsf(m0[g]) >= kFar;
#pragma unroll
          for (int e = 0; e < 16; ++e) x[g][e] -= far ? m[g] : 0.0f;
          m0[g] = far ? 0.0f : m0[g];
        }
      }
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
      if constexpr (kSets == 2) load_first();
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
        step(std::integral_constant<int, 0>(), i, s[0], s[1]);
        if (i + 1 < S::kPer * t1) step(std::integral_constant<int, 1>(), i + 1, s[1], s[0]);
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
      // (m, sum, rsum, parts) of every query, head and part, and behind them the parts' values
      const size_t ph = qh * a.splits + it.part;
      if (a.splits > 1 && half == 0) *(f4*)(a.work + ph * 4) = f4{m[g], sum[g], rsum[g], (float)it.parts};
      if (it.parts == 1) {
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
          a.lse[qh] = sum[g] > 0.0f ? m[g] * scale * kLn2 + logf(sum[g]) : sum[g] == 0.0f ? -INFINITY : sum[g];
        continue;
      }
      float* dst = a.work + (size_t)a.n_q * a.heads * a.splits * 4 + ph * DV + 4 * half;
#pragma unroll
      for (int b = 0; b < kBlocks; ++b)
#pragma unroll
        for (int c = 0; c < 4; ++c)
          *(f4*)(dst + 32 * b + 8 * c) = f4{o[g][b][4 * c], o[g][b][4 * c + 1], o[g][b][4 * c + 2], o[g][b][4 * c + 3]};
    }
    if (sh[4 * kWaves]) {
      // what was taken out, added to what the lane wrote
      const int from = all_see / S::kKeys > t0 ? all_see / S::kKeys : t0;
      for (int key = S::kKeys * from; key < S::kKeys * t1 && key < hi; ++key) {
        const unsigned short* value = (const unsigned short*)a.kv + ((size_t)(k0 + key) * a.heads + h) * (DN + DV) + DN;
#pragma unroll
        for (int g = 0; g < kSets; ++g) {
          const int i = wq + 32 * g + col;
          if (i >= nq || key >= limit[g]) continue;
          const size_t qh = (size_t)(q0 + i) * a.heads + h;
          __bf16* whole = (__bf16*)a.o + qh * DV;
          float* partial = a.work + (size_t)a.n_q * a.heads * a.splits * 4 + (qh * a.splits + it.part) * DV;
#pragma unroll 1
          for (int d = 4 * half; d < DV; d += d % 4 == 3 ? 5 : 1) {
            if (!is_odd(value[d])) continue;
            const float x = __uint_as_float((uint32_t)value[d] << 16);
            if (it.parts == 1) whole[d] = (__bf16)((float)whole[d] + x);
            else partial[d] += x;
          }
        }
      }
    }
  }
}

// Joins the parts of each query and head in their order: one wave for both, DV / 64 values a lane. What was left in one
// part has its result. Memory bounds it: 2048 queries x 8 heads x 2 parts of 256 values, 34 MB, in 9 us.
template <int DV>
__global__ __launch_bounds__(256) void join_prompt_kernel(PromptArgs a) {
  constexpr int kPer = DV / 64;
  const int lane = threadIdx.x & 63;
  const float scale = scale_of(a.scale);
  // rows before the first sequence and behind the last have no parts
  const size_t n0 = (size_t)cut(a.cu_q[0], a.n_q) * a.heads, n = (size_t)cut(a.cu_q[a.R], a.n_q) * a.heads;
  for (size_t qh = n0 + (size_t)blockIdx.x * 4 + (threadIdx.x >> 6); qh < n; qh += (size_t)gridDim.x * 4) {
    const f4* st = (const f4*)a.work + qh * a.splits;
    const float count = st[0][3];
    const int parts = count >= 2.0f && count <= (float)a.splits ? (int)count : 1;
    if (parts == 1) continue;
    float m = -INFINITY;
    for (int s = 0; s < parts; ++s) m = fmaxf(m, st[s][0]);
    float sum = 0.0f, rsum = 0.0f, o[kPer] = {};
    const float* src = a.work + (size_t)a.n_q * a.heads * a.splits * 4 + qh * a.splits * DV + lane * kPer;
    for (int s = 0; s < parts; ++s) {
      const f4 v = st[s];
      const float c = rebase(v[0], m, scale);
      sum += c * v[1];
      rsum += c * v[2];
#pragma unroll
      for (int i = 0; i < kPer; ++i) o[i] += c * src[(size_t)s * DV + i];
    }
    const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
    __bf16* dst = (__bf16*)a.o + qh * DV + lane * kPer;
#pragma unroll
    for (int i = 0; i < kPer; ++i) dst[i] = (__bf16)(o[i] * f);
    if (a.lse && lane == 0) a.lse[qh] = sum > 0.0f ? m * scale * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
  }
}

constexpr int queries_of(int sets) { return 128 * sets; }

template <int DN, int P, int DV, int kSets>
hipError_t launch(const PromptArgs& a, hipStream_t s) {
  using S = PromptShape<DN, P, DV, kSets>;
  static_assert(S::kQueries == queries_of(kSets));
  constexpr uint32_t lds = S::kLds;
  // every sequence but one may leave a tile part empty; a tile's parts are at most its share of a.items and one more
  int64_t slots = ((int64_t)a.n_q + S::kQueries - 1) / S::kQueries + a.R - 1;
  if (a.splits > 1) slots += a.items + 1;
  hipLaunchKernelGGL((prompt_kernel<DN, P, DV, kSets>), dim3(a.heads, (int)(slots < 65535 ? slots : 65535)),
                     dim3(S::kThreads), lds, s, a, (int)slots);
  if (a.splits > 1) {
    const uint64_t blocks = ((uint64_t)a.n_q * a.heads + 3) / 4;
    hipLaunchKernelGGL(join_prompt_kernel<DV>, dim3((int)(blocks < 4096 ? blocks : 4096)), dim3(256), 0, s, a);
  }
  return hipGetLastError();
}

template <int DN, int P, int DV, int kSets>
hipError_t set_lds() {
  return hipFuncSetAttribute((const void*)prompt_kernel<DN, P, DV, kSets>, hipFuncAttributeMaxDynamicSharedMemorySize,
                             (int)PromptShape<DN, P, DV, kSets>::kLds);
}

}  // namespace

// Queries to a workgroup and parts of the keys, by an estimate of the time for sequences of equal lengths under a causal
// mask. A workgroup's time is its keys' and a start's, the card's that of its longest workgroup or of all of them on 256
// units, and of a longest one's half where they end unevenly (several sequences, two workgroups to a unit). The join
// moves the partial results to memory and back.
// 256 queries to a workgroup (one to a unit) read half as much from LDS for a product as 128 (two to a unit): 8192 tokens x
// 16 heads with 128 values take 374 and 416 us. But 128 fill the card sooner and hide each other's starts: 8 prompts of up
// to 300 tokens x 16 heads take 25 and 16 us, 64 of them 93 and 56. With 64 values they are even (32 heads 507 and 482
// us, 16 heads 258 and 265), and there is one kernel; with 256, the results of 256 queries do not fit into the registers.
// The estimate takes n_q / R queries and n_k / R keys for each of the R sequences. Where most of a context's requests have no
// prompt that is far off: 512 queries behind 15872 keys x 16 heads of 128 take 110 us in a context of 1 or 8 requests and 395 in
// one of 64 or 256 (no parts), and R - 1 workgroups a head begin for nothing (one prompt of 8192 x 16 heads: 352 us in a
// context of one, 356 of 256, 1.5 ms of 4096).
PromptPlan prompt_plan(int R, int n_q, int n_k, int heads, int value) {
  PromptPlan best{1, 1, 0};
  if (n_q <= 0) return best;
  double least = 0.0;
  const double nq = (double)n_q / R, nk = (double)n_k / R;
  const double mean = nq < nk ? nk - nq / 2 : nk / 2;  // keys of a query
  for (int sets = value == 128 ? 2 : 1; sets >= 1; --sets) {
    const bool two = value == 64 || (value == 128 && sets == 1);  // workgroups to a unit
    const double per_key = value == 64 ? 0.0147 : value == 256 ? 0.035 : sets == 2 ? 0.0425 : 0.0235;  // us
    const double tiles = R == 1 ? ceil(nq / queries_of(sets)) : (nq / queries_of(sets) + 0.5) * R, groups = tiles * heads;
    const double start = 6.0 * sets / per_key;  // keys
    const int units = two ? 512 : 256;
    // k = 0: whole; else with one sequence k + 1 parts of each tile, with several k rounds of parts on all units
    for (int k = 0; k < 16; ++k) {
      const double most = tiles * fmin(16.0, nk / kLeastKeys);
      const int items = (int)fmin(R == 1 ? tiles * (k + 1) : (double)k * units / heads, most);
      const double parts = k == 0 ? 1.0 : items / tiles;
      if (k > 0 && (parts < 1.25 || groups * parts > 4096)) continue;
      const double longest = nk / parts + start, each = mean / parts + start, rounds = groups * parts / 256;
      const double all = R > 1 && k > 0 ? 1.15 * rounds * each
                         : R == 1 && !two ? ceil(rounds) * each : rounds * each + longest / 4;
      double t = per_key * (longest > all ? longest : all);
      if (k > 0) t += 5.0 + (double)n_q * heads * parts * (16 + 4 * value) * 2 / 4.5e6;
      if (least == 0.0 || t < least) {
        least = t;
        best.sets = sets;
        best.splits = k == 0 ? 1 : R == 1 ? (int)ceil(parts) : parts <= 8 ? (int)ceil(2 * parts) : 16;
        best.items = k == 0 ? 0 : items;
      }
    }
  }
  return best;
}

uint64_t prompt_work_bytes(const PromptPlan& plan, int n_q, int heads, int value) {
  const uint64_t s = (uint64_t)plan.splits;
  return s == 1 ? 0 : (uint64_t)n_q * heads * s * (16 + 4ull * value);
}

hipError_t set_prompt_lds() {
  for (const auto f : {set_lds<64, 32, 64, 1>, set_lds<64, 64, 64, 1>, set_lds<128, 32, 128, 1>, set_lds<128, 64, 128, 1>,
                       set_lds<128, 32, 128, 2>, set_lds<128, 64, 128, 2>, set_lds<192, 32, 256, 1>,
                       set_lds<192, 64, 256, 1>}) {
    const hipError_t e = f();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_prompt(const PromptArgs& a, hipStream_t s) {
  if (a.n_q <= 0) return hipSuccess;
  const bool more = a.rope == 64;
  if (a.value == 64) return more ? launch<64, 64, 64, 1>(a, s) : launch<64, 32, 64, 1>(a, s);
  if (a.value == 256) return more ? launch<192, 64, 256, 1>(a, s) : launch<192, 32, 256, 1>(a, s);
  if (a.sets == 2) return more ? launch<128, 64, 128, 2>(a, s) : launch<128, 32, 128, 2>(a, s);
  return more ? launch<128, 64, 128, 1>(a, s) : launch<128, 32, 128, 1>(a, s);
}

}  // namespace hs
