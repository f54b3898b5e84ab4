// The k best positions of each row of scores, ascending (gfx950).
//
// A workgroup reads its part of a row once, into registers, 64 consecutive positions to a wave's load. What is selected is kept as
// a mask of each such load, and a thread then writes the positions of one mask: passes over the registers are unrolled code that
// runs once and waits for its own instructions, and three of them are enough (with two more, to count and to write by ballots,
// 256 rows of 40960 took 31 us, with three 20). The k-th best score is found without a sort. It is no lower than the lowest of the
// threads' own best scores (or second best, and so on: as many as make k); what lies above is counted in bins, even in value
// (which keeps a wave's counts apart, where the bits of the scores would share few bins), and the scores of the one bin that the
// k-th lies in, some dozens, are ranked against each other with their positions. A bin of more than kList (few different scores,
// or outliers that stretch the range) is divided further, by the scores' bits, until kList are left or all are equal; the first
// of the equal ones are then taken in order.
// A row of more than kMost positions is cut into parts, whose best k (with their positions, in order) are the row of the next
// launch; ties stay with the lowest positions, as every launch keeps the order. Where that would take a third launch, the first
// one takes the best score of each of some thousand groups instead: the k-th best of those is a bound that k scores reach. A part
// with no more than k of them leaves those (normal scores: 3000 of a million in all), one with more its best k, and one
// workgroup joins them, 48 K at a time. That is for k of up to 4096 (a quarter of a part) and rows of up to 16.7 M (the 1024 parts
// that are joined); others go in as many launches of the first kind as they need.
// Bounded by: a row alone, the instructions and barriers of one workgroup (1 x 4096, k 256, kernel 5.5 to 5.7 us); many rows, the
// vector units, four passes of some instructions to a score (256 x 40960 18.5 to 19 us, 2.2 TB/s); the longest, three launches
// (2 x 1 M 27 us), half of them the join, whose 48 scores to a thread do not fit its registers (66 spilled).
#include "hs_index.h"

#include <algorithm>
#include <type_traits>

namespace hs {

namespace {

constexpr int kSelectThreads = 1024;         // of a workgroup, for rows of more than kShort
constexpr int kShortThreads = 512;
constexpr int kShort = 8 * kShortThreads;
constexpr int kList = 512;                   // scores of a bin that are ranked against each other
constexpr int kMost = 48 * kSelectThreads;   // positions of a workgroup
constexpr int kMiddle = 16 * kSelectThreads; // of one that takes half of the registers
constexpr int kUnits = 256;                  // of the card
constexpr int kTopThreads = 256;
constexpr int kEach = 32;                    // positions of a lane whose best is taken
constexpr int kMostParts = kSelectThreads;   // that are joined

struct SelectLevel {
  const float* in;      // rows of n_in scores
  const int32_t* idx;   // their positions, or nullptr (first launch: their places)
  int64_t n_in;
  int64_t part;         // of a row, to a workgroup
  int64_t row0;         // of the launch
  int32_t parts, parts_in;  // (the latter: joined)
  float* out;           // not the last launch: [row][parts][k] scores, -inf behind the selected, and
  int32_t* out_idx;     // their positions
  // rows under a bound: the best scores of each row's groups, how many of out each part has; out has two more parts for each row
  float* tops;
  int32_t n_tops;
  int32_t* counts;
};

// What launches of the kernel take in and leave: scores by position, parts under a bound (without -inf behind them), such parts.
enum Kind { kPlain, kBounded, kJoin };

// A score's order as 32 bits; of zeros of both signs the same.
__device__ __forceinline__ uint32_t order_of(float x) {
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float score_of(uint32_t order) {
  return __uint_as_float(order & 0x80000000u ? order & 0x7fffffffu : ~order);
}

__device__ __forceinline__ int wave_scan(int v) {  // inclusive
  v += __builtin_amdgcn_update_dpp(0, v, 0x111, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x112, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x114, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x118, 0xf, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x142, 0xa, 0xf, false);
  v += __builtin_amdgcn_update_dpp(0, v, 0x143, 0xc, 0xf, false);
  return v;
}

__device__ __forceinline__ int wave_sum(int v) { return __builtin_amdgcn_readlane(wave_scan(v), 63); }

template <class Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = op(v, __shfl_xor(v, d));
  return v;
}

// f(block) for the first of kMany blocks, one within the other: a way past those that are left out is one jump and not one for each
// (2 rows x 1 M 27 -> 25 us).
template <int kMany, int kFrom = 0, class F>
__device__ __forceinline__ void blocks_of(int blocks, const F& f) {
  if (kFrom < blocks) {
    f(std::integral_constant<int, kFrom>());
    if constexpr (kFrom + 1 < kMany) blocks_of<kMany, kFrom + 1>(blocks, f);
  }
}

// The positions of the row's token, and the row of its scores.
__device__ __forceinline__ int64_t positions_of(const SelectArgs& a, int64_t row, int64_t& from) {
  int64_t t = row;
  if (a.cu) {
    t = a.cu[row + 1] > a.cu[row] ? (int64_t)a.cu[row + 1] - 1 : -1;
    if (t >= a.n) t = -1;
  }
  from = t < 0 ? 0 : t;
  const int64_t m = t < 0 ? 0 : (int64_t)a.pos[t] + 1;
  return m < 0 ? 0 : m < a.columns ? m : a.columns;
}

// The best scores of groups of kEach << shift positions, -inf where there is none: k groups hold k scores that are no lower than
// the k-th best of these. A NaN is left out.
__global__ __launch_bounds__(kTopThreads) void tops_kernel(SelectArgs a, SelectLevel l, int shift) {
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t row = l.row0 + blockIdx.x / l.parts;
  const int64_t chunk = (int64_t)(blockIdx.x % l.parts) * (kTopThreads / 64) + wave;
  if (chunk * (64 >> shift) >= l.n_tops) return;
  int64_t from;
  const int64_t m = positions_of(a, row, from), rivals = m - (m < a.recent ? m : a.recent);
  const int64_t left = rivals - chunk * kEach * 64 - lane;
  const float* in = l.in + from * l.n_in + chunk * kEach * 64 + lane;
  float v[kEach], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) v[i] = left > 64 * i ? in[64 * i] : -INFINITY;
#pragma unroll
  for (int i = 0; i < kEach; ++i) top = fmaxf(top, v[i]);
  for (int d = 0; d < shift; ++d) top = fmaxf(top, __shfl_xor(top, 1 << d));
  if ((lane & ((1 << shift) - 1)) == 0) l.tops[row * l.n_tops + chunk * (64 >> shift) + (lane >> shift)] = top;
}

// kPer: most scores of a thread, kBlock of them in a block: a workgroup passes over as many blocks as its part has.
template <int kThreads, int kPer, Kind kKind>
__global__ __launch_bounds__(kThreads, kPer <= 16 ? 8 : 4) void select_kernel(SelectArgs a, SelectLevel l) {
  constexpr int kWaves = kThreads / 64, kBins = 2 * kThreads;
  // (few scores are joined as a rule, and a lone workgroup takes as long as its instructions do: 3000 of them 4 us less than in 8s)
  constexpr int kBlock = kKind == kJoin ? 4 : 8;
  constexpr int kBest = 2048 / kThreads;  // of a thread's scores, for the bound
  __shared__ int hist[kBins];
  __shared__ uint64_t list[kList];
  __shared__ int rank[kList];
  __shared__ uint64_t masks[kWaves * kPer], ties[kWaves * kPer];  // of the loads, in the order of the positions
  __shared__ int sums[kWaves], tie_sums[kWaves], taken_sums[kWaves], found[4];
  __shared__ uint16_t chosen[kMaxTopK];
  __shared__ float lows[kWaves], highs[kWaves];
  __shared__ int starts[kKind == kJoin ? kMostParts : 1];  // joined: of the parts' scores, one after another
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = l.row0 + blockIdx.x / l.parts;
  const int part = (int)(blockIdx.x % l.parts);
  const bool whole = kKind == kJoin || (kKind == kPlain && l.out == nullptr);
  // the positions that compete, and how many of them are selected
  int64_t from;
  const int64_t m = positions_of(a, row, from);
  if (kKind == kPlain && l.idx) from = row;
  const int recent = m < a.recent ? (int)m : a.recent, k = a.k - recent;
  const int64_t begin = part * l.part;
  int total = 0, done = 0, kept = 0, turn = 0;  // joined: of the parts' scores, those seen, and the best of them so far
  if constexpr (kKind == kJoin) {
    const int mine = tid < l.parts_in ? l.counts[row * l.parts_in + tid] : 0, upto = wave_scan(mine);
    if (lane == 63) sums[wave] = upto;
    __syncthreads();
    int before = upto - mine;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w < wave) before += sums[w];
      total += sums[w];
    }
    starts[tid] = before;
    __syncthreads();
  }
  const int half_parts = kKind == kJoin && l.parts_in > 1 ? 1 << (31 - __builtin_clz(l.parts_in - 1)) : 0;
  // joined: where each i-th lies, of the parts' scores; side by side, as a search waits for LDS at every step
  auto slots_of = [&](const auto& i, auto& slot) {
    constexpr int kMany = sizeof(i) / sizeof(i[0]);
    int p[kMany] = {};
    for (int d = half_parts; d > 0; d >>= 1) {
#pragma unroll
      for (int c = 0; c < kMany; ++c) p[c] += starts[p[c] + d] <= i[c] ? d : 0;
    }
#pragma unroll
    for (int c = 0; c < kMany; ++c) slot[c] = p[c] * a.k + i[c] - starts[p[c]];
  };
  // joined: the row's parts, and behind them two in turn for the best so far
  const int64_t slots = kKind == kJoin ? row * (l.parts_in + 2) * a.k : 0;
  float* const joined = l.out + slots;
  int32_t* const joined_idx = l.out_idx + slots;
  for (;;) {
    int n;
    if constexpr (kKind == kJoin) {
      n = total - done < kMost - kept ? total - done + kept : kMost;
    } else {
      const int64_t rivals = l.idx ? l.n_in : m - recent;
      n = (int)(rivals <= begin ? 0 : rivals - begin < l.part ? rivals - begin : l.part);
    }
    const int per = (n + kThreads - 1) / kThreads, blocks = (per + kBlock - 1) / kBlock;  // of a wave: loads, their blocks
    const int first = wave * per * 64, upto = first + per * 64 < n ? first + per * 64 : n;
    float x[kPer];
    // f(j) for the wave's loads, in their order
    auto each = [&](auto f) {
      blocks_of<kPer / kBlock>(blocks, [&](auto b) {
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
          asm volatile("" : "+v"(x[b * kBlock + i]));  // nothing that a pass works out is kept for the next: registers are short
          f(b * kBlock + i);
        }
      });
    };
    if constexpr (kKind == kJoin) {
      blocks_of<kPer / kBlock>(blocks, [&](auto b) {
        int at[kBlock], slot[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
          at[i] = first + (b * kBlock + i) * 64 + lane;
          at[i] = at[i] < upto ? at[i] : upto - 1;
        }
        int of[kBlock];
#pragma unroll
        for (int i = 0; i < kBlock; ++i) of[i] = done + at[i] - kept;
        slots_of(of, slot);
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
          x[b * kBlock + i] = joined[(uint32_t)(at[i] < kept ? (l.parts_in + turn) * a.k + at[i] : slot[i])];
        __builtin_amdgcn_sched_barrier(0);  // (all on their way before the first is looked at)
#pragma unroll
        for (int i = 0; i < kBlock; ++i)
          if (first + (b * kBlock + i) * 64 + lane >= upto) x[b * kBlock + i] = -INFINITY;
      });
    } else {
      const float* in = l.in + from * l.n_in + begin + first;
      blocks_of<kPer / kBlock>(blocks, [&](auto b) {
        const int left = upto - first - b * kBlock * 64;  // of the wave, from this block on
        if (left >= kBlock * 64) {
#pragma unroll
          for (int i = 0; i < kBlock; ++i) x[b * kBlock + i] = in[(b * kBlock + i) * 64 + lane];
        } else {
#pragma unroll
          for (int i = 0; i < kBlock; ++i) x[b * kBlock + i] = i * 64 + lane < left ? in[(b * kBlock + i) * 64 + lane] : -INFINITY;
        }
      });
    }
    hist[tid] = hist[tid + kThreads] = 0;
    for (int i = tid; i < kList; i += kThreads) rank[i] = 0;
    if (tid == 0) found[3] = 0;
    __syncthreads();
    // the loads' masks of f(j), to LDS
    auto mask_of = [&](uint64_t* to, auto f) {
      uint32_t low = 0, high = 0;
      each([&](int j) {
        const uint64_t mask = __ballot(f(j));
        low = lane == j ? (uint32_t)mask : low;
        high = lane == j ? (uint32_t)(mask >> 32) : high;
      });
      if (lane < per) to[wave * per + lane] = (uint64_t)high << 32 | low;
    };
    // Of the counts, the one that the need-th from the highest on lies in (found[0]), and which of its own that is (found[1]);
    // returns the sum of all
    auto find = [&](int need) {
      const int b = kBins - 2 - 2 * tid, upper = hist[b + 1], both = upper + hist[b], upto = wave_scan(both);
      if (lane == 63) sums[wave] = upto;
      __syncthreads();
      int before = upto - both, all = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sums[w];
        all += sums[w];
      }
      if (before < need && before + both >= need) {  // one thread
        const bool in_upper = before + upper >= need;
        found[0] = in_upper ? b + 1 : b;
        found[1] = in_upper ? need - before : need - before - upper;
      }
      __syncthreads();
      return all;
    };
    const auto lesser = [](float u, float v) { return fminf(u, v); };
    const auto larger = [](float u, float v) { return fmaxf(u, v); };
    int tied = 0;        // of the equal scores in `ties`, those that are selected
    bool every = false;  // what may be selected is
    bool few = false;    // not more than k of the part reach the row's bound: those are left to the next launch
    if constexpr (kKind == kBounded) {
      const float* tops = l.tops + row * l.n_tops;
      float lo = INFINITY, hi = -INFINITY;
      for (int i = tid; i < l.n_tops; i += kThreads) {
        const float v = tops[i];
        lo = fminf(lo, v > -INFINITY ? v : INFINITY);
        hi = fmaxf(hi, v);
      }
      lo = wave_reduce(lo, lesser);
      hi = wave_reduce(hi, larger);
      if (lane == 0) lows[wave] = lo, highs[wave] = hi;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        lo = fminf(lo, lows[w]);
        hi = fmaxf(hi, highs[w]);
      }
      lo = fminf(lo, 3.4028235e38f);
      hi = fminf(hi, 3.4028235e38f);
      const float half_lo = 0.5f * lo, step = fminf((float)(kBins - 1) / (0.5f * hi - half_lo), 3.4028235e38f);
      auto place_of = [&](float v) { return fmaf(v, 0.5f, -half_lo) * step; };
      for (int i = tid; i < l.n_tops; i += kThreads) {
        const float v = tops[i];
        if (v > -INFINITY) atomicAdd(&hist[(uint32_t)fminf(place_of(v), (float)(kBins - 1))], 1);
      }
      __syncthreads();
      if (k > 0 && find(k) >= k) {
        const float least = (float)found[0];
        int reach = 0;
        mask_of(masks, [&](int j) {
          const bool it = place_of(x[j]) >= least;
          reach += it;
          return it;
        });
        reach = wave_sum(reach);
        if (lane == 0) tie_sums[wave] = reach;
        __syncthreads();
        reach = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) reach += tie_sums[w];
        few = reach <= k;
      }
      if (!few) {
        hist[tid] = hist[tid + kThreads] = 0;
        __syncthreads();
      }
    }
    if (!few) {
      // (a median leaves out a NaN, and is one instruction where the larger of two would be two)
      float best[kBest];
#pragma unroll
      for (int i = 0; i < kBest; ++i) best[i] = -INFINITY;
      each([&](int j) {
#pragma unroll
        for (int i = kBest - 1; i >= 0; --i) best[i] = __builtin_amdgcn_fmed3f(x[j], i ? best[i - 1] : INFINITY, best[i]);
      });
      float bound = -INFINITY;  // as many of each thread's as make k
#pragma unroll
      for (int i = 0; i < kBest; ++i)
        if (k > i * kThreads && k <= (i + 1) * kThreads) bound = best[i];
      float hi = wave_reduce(best[0], larger);
      float lo = wave_reduce(bound, lesser);
      if (lane == 0) lows[wave] = lo, highs[wave] = hi;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        lo = fminf(lo, lows[w]);
        hi = fmaxf(hi, highs[w]);
      }
      if (lo == -INFINITY) {
        // too few scores for that bound: the lowest that may be selected, and how many may (a NaN becomes -inf, so that no ballot
        // meets one)
        int valid = 0;
        lo = INFINITY;
        each([&](int j) {
          x[j] = x[j] == x[j] ? x[j] : -INFINITY;
          lo = fminf(lo, x[j] > -INFINITY ? x[j] : INFINITY);
          valid += __popcll(__ballot(x[j] > -INFINITY));
        });
        lo = wave_reduce(lo, lesser);
        __syncthreads();  // the bounds before are read
        if (lane == 0) lows[wave] = lo, sums[wave] = valid;
        __syncthreads();
        valid = 0;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          lo = fminf(lo, lows[w]);
          valid += sums[w];
        }
        every = valid <= k;
      }
      if (k == 0 || every) {
        mask_of(masks, [&](int j) { return every && x[j] > -INFINITY; });
        __syncthreads();
      } else {
        // The bin of a score from lo on: even in value, between halves so that no difference is past 32 bits. The k-th best is lo
        // itself where no k are above it; those that are equal to lo need no count (there may be many: scores of zero).
        lo = fminf(lo, 3.4028235e38f);
        hi = fminf(hi, 3.4028235e38f);
        const float half_lo = 0.5f * lo, step = fminf((float)(kBins - 1) / (0.5f * hi - half_lo), 3.4028235e38f);
        auto place_of = [&](float v) { return fminf(fmaf(v, 0.5f, -half_lo) * step, (float)(kBins - 1)); };
        each([&](int j) {
          if (x[j] > lo) atomicAdd(&hist[(uint32_t)place_of(x[j])], 1);
        });
        __syncthreads();
        const int above = find(k);
        bool equal = above < k;
        const int bin = equal ? 0 : found[0];
        int need = equal ? k - above : found[1], count = equal ? 0 : hist[bin];
        uint32_t from_order = order_of(lo), span = 0xffffffffu;  // of the scores in question
        const float bin_from = (float)bin, bin_to = (float)(bin + 1);
        auto is_in = [&](float v) {
          const float p = place_of(v);
          return v > lo && p >= bin_from && p < bin_to && order_of(v) - from_order <= span;
        };
        auto add_to_list = [&](int j) {
          list[atomicAdd(&found[3], 1)] = (uint64_t)order_of(x[j]) << 32 | (uint32_t)(~(first + j * 64 + lane));
        };
        const bool listed = !equal && count <= kList;
        if (listed) {
          // what lies in the bin or above it; those of the bin that are not selected are taken out below
          mask_of(masks, [&](int j) {
            const float p = place_of(x[j]);
            const bool in_or_above = x[j] > lo && p >= bin_from;
            if (in_or_above && p < bin_to) add_to_list(j);
            return in_or_above;
          });
        }
        while (!equal && count > kList) {
          // the least and largest of them
          uint32_t least_order = 0xffffffffu, most_order = 0;
          each([&](int j) {
            if (is_in(x[j])) {
              const uint32_t u = order_of(x[j]);
              least_order = u < least_order ? u : least_order;
              most_order = u > most_order ? u : most_order;
            }
          });
#pragma unroll
          for (int d = 1; d < 64; d <<= 1) {
            const uint32_t u = __shfl_xor(least_order, d), v = __shfl_xor(most_order, d);
            least_order = u < least_order ? u : least_order;
            most_order = v > most_order ? v : most_order;
          }
          __syncthreads();  // the counts are read, and the bounds before
          if (lane == 0) lows[wave] = __uint_as_float(least_order), highs[wave] = __uint_as_float(most_order);
          hist[tid] = hist[tid + kThreads] = 0;
          __syncthreads();
#pragma unroll
          for (int w = 0; w < kWaves; ++w) {
            const uint32_t u = __float_as_uint(lows[w]), v = __float_as_uint(highs[w]);
            least_order = u < least_order ? u : least_order;
            most_order = v > most_order ? v : most_order;
          }
          from_order = __builtin_amdgcn_readfirstlane(least_order);
          span = __builtin_amdgcn_readfirstlane(most_order) - from_order;
          if (span == 0) {
            equal = true;
            break;
          }
          const int shift = span < (uint32_t)kBins ? 0 : __builtin_clz(kBins - 1) - __builtin_clz(span);  // span >> shift < kBins
          each([&](int j) {
            if (is_in(x[j])) atomicAdd(&hist[(order_of(x[j]) - from_order) >> shift], 1);
          });
          __syncthreads();
          find(need);
          need = found[1];
          count = hist[found[0]];
          const uint32_t begins = (uint32_t)found[0] << shift, width = (1u << shift) - 1;
          span = span - begins < width ? span - begins : width;
          from_order += begins;
        }
        if (equal) {
          const float least = score_of(from_order);
          mask_of(masks, [&](int j) { return x[j] > least; });
          mask_of(ties, [&](int j) { return x[j] == least; });
          tied = need;
          __syncthreads();
        } else {
          if (!listed) {
            mask_of(masks, [&](int j) {
              if (is_in(x[j])) add_to_list(j);
              return x[j] > lo && order_of(x[j]) >= from_order;
            });
          }
          __syncthreads();
          // every wave compares with its share of them
          for (int c = lane; c < count; c += 64) {
            const uint64_t mine = list[c];
            int better = 0;
#pragma unroll 4
            for (int i = wave; i < count; i += kWaves) better += list[i] > mine;
            atomicAdd(&rank[c], better);
          }
          __syncthreads();
          for (int c = tid; c < count; c += kThreads)
            if (rank[c] >= need) {
              const uint32_t i = ~(uint32_t)list[c];
              atomicAnd((uint32_t*)masks + 2 * (i >> 6) + (i >> 5 & 1), ~(1u << (i & 31)));
            }
          __syncthreads();
        }
      }
    }
    auto scan = [&](int v, int* sums, int* total) {  // exclusive
      const int upto = wave_scan(v);
      if (lane == 63) sums[wave] = upto;
      __syncthreads();
      int before = upto - v;
      *total = 0;
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        if (w < wave) before += sums[w];
        *total += sums[w];
      }
      return before;
    };
    // a mask, or where there are fewer of them than threads an equal piece of one, to a thread
    const int loads = kWaves * per, split = loads <= kThreads / 8 ? 3 : loads <= kThreads / 4 ? 2 : loads <= kThreads / 2 ? 1 : 0;
    const int shift = (tid & ((1 << split) - 1)) * (64 >> split);
    const bool has = tid >> split < loads;
    const uint64_t piece = split ? (1ull << (64 >> split)) - 1 : ~0ull;
    uint64_t mask = has ? masks[tid >> split] >> shift & piece : 0;
    int all;
    if (tied > 0) {
      uint64_t tie = has ? ties[tid >> split] >> shift & piece : 0;
      int room = tied - scan(__popcll(tie), tie_sums, &all);
      for (; tie && room > 0; --room) {
        mask |= tie & -tie;
        tie &= tie - 1;
      }
    }
    int at = scan(__popcll(mask), taken_sums, &all);
    // (through LDS, so that a thread's positions need not wait for each other's loads, and stores are whole)
    const int in_part = (tid >> split) * 64 + shift;
    for (; mask; mask &= mask - 1) chosen[at++] = (uint16_t)(in_part + __builtin_ctzll(mask));
    __syncthreads();
    if constexpr (kKind == kJoin) {
      const bool last = done + n - kept == total;
      const int before = (l.parts_in + turn) * a.k, after = (l.parts_in + 1 - turn) * a.k;
      turn ^= 1;
      for (int o = tid; o < all; o += 2 * kThreads) {  // two searches side by side
        const int other = o + kThreads < all ? o + kThreads : o, i[2] = {chosen[o], chosen[other]};
        const int of[2] = {done + i[0] - kept, done + i[1] - kept};
        int slot[2];
        slots_of(of, slot);
#pragma unroll
        for (int c = 0; c < 2; ++c) slot[c] = i[c] < kept ? before + i[c] : slot[c];
        const int32_t id[2] = {joined_idx[slot[0]], joined_idx[slot[1]]};
        if (last) {
          a.topk[row * a.k + o] = id[0];
          a.topk[row * a.k + other] = id[1];
        } else {
          joined[after + o] = joined[slot[0]];
          joined_idx[after + o] = id[0];
          joined[after + other] = joined[slot[1]];
          joined_idx[after + other] = id[1];
        }
      }
      if (!last) {
        done += n - kept;
        kept = all;
        __syncthreads();
        continue;
      }
    } else {
      const int64_t to = whole ? row * a.k : (row * (l.parts + (kKind == kBounded ? 2 : 0)) + part) * a.k;
      for (int o = tid; o < all; o += kThreads) {
        const int64_t i = begin + chosen[o];
        const int32_t id = l.idx ? l.idx[row * l.n_in + i] : (int32_t)i;
        if (whole) {
          a.topk[to + o] = id;
        } else {
          l.out[to + o] = l.in[from * l.n_in + i];
          l.out_idx[to + o] = id;
        }
      }
      if (kKind == kBounded) {
        if (tid == 0) l.counts[row * l.parts + part] = all;
      } else if (!whole) {
        for (int i = all + tid; i < a.k; i += kThreads) l.out[to + i] = -INFINITY;
      }
    }
    if (whole)
      for (int i = all + tid; i < a.k; i += kThreads)
        a.topk[row * a.k + i] = i < all + recent ? (int32_t)(m - recent + i - all) : -1;
    break;
  }
}

template <int kThreads, int kPer, Kind kKind = kPlain>
void launch(const SelectArgs& a, SelectLevel l, hipStream_t s) {
  const int64_t most = std::max<int64_t>(1, (1 << 21) / l.parts);  // rows of a launch (which ends below 2^32 threads)
  for (l.row0 = 0; l.row0 < a.rows; l.row0 += most) {
    const int64_t rows = std::min<int64_t>(most, a.rows - l.row0);
    hipLaunchKernelGGL((select_kernel<kThreads, kPer, kKind>), dim3((uint32_t)(rows * l.parts)), dim3(kThreads), 0, s, a, l);
  }
}

// The part into which a launch cuts rows of more than kMost: one that leaves an eighth of them and runs two workgroups to a unit,
// or, where that would leave more than a quarter, the longest (1 row of 131072, k 2048: 21 us; in parts of 41 K 30).
int64_t part_of(int k) { return 4 * k <= kMiddle ? kMiddle : kMost; }

// Rows whose parts' best would not fit one workgroup are selected under a bound: the groups' best (k of them at least, with a
// quarter to spare), from their k-th best on what a part has, joined. Three launches of which each takes little, against three
// that each select k (2 rows x 1 M, k 2048, 34 -> 25 us, with many ties 40 -> 26; 16 rows x 400000 39 -> 32; 64 x 1 M 152 -> 136);
// against two of those it is no gain (64 x 131072 31 -> 37 us, 1 x 1 M, k 256, 19.7 -> 22.3). A k past a quarter of a part would
// leave too much of each, and parts are counted by a thread of the join each.
struct Bounded {
  int64_t parts, chunks;
  int shift;
  int32_t n_tops;
  bool use;
};
Bounded bounded(int64_t columns, int k) {
  Bounded b{};
  b.parts = (columns + kMiddle - 1) / kMiddle;
  b.chunks = (columns + kEach * 64 - 1) / (kEach * 64);
  while (b.shift < 6 && (b.chunks * (64 >> (b.shift + 1))) * 4 >= (int64_t)k * 5) ++b.shift;
  b.n_tops = (int32_t)(b.chunks * (64 >> b.shift));
  b.use = b.parts * k > kMost && b.parts <= kMostParts && 4 * k <= kMiddle;
  return b;
}

}  // namespace

// Every launch but the last leaves k scores and positions of each part.
uint64_t select_work_bytes(int rows, int64_t columns, int k) {
  uint64_t bytes = 0;
  const Bounded b = bounded(columns, k);
  if (b.use) return ((uint64_t)rows * (8 * (uint64_t)k * (b.parts + 2) + 4 * b.n_tops + 4 * b.parts) + 15) & ~15ull;
  for (int64_t n = columns; n > kMost;) {
    n = (n + part_of(k) - 1) / part_of(k) * k;
    bytes += (uint64_t)rows * n * 8;
  }
  return (bytes + 15) & ~15ull;
}

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  SelectLevel l{};
  l.in = a.scores;
  l.n_in = a.columns;
  const Bounded b = bounded(a.columns, a.k);
  if (b.use) {
    const int64_t slots = a.rows * (b.parts + 2) * a.k;
    l.out = (float*)a.work;
    l.out_idx = (int32_t*)(l.out + slots);
    l.tops = (float*)(l.out_idx + slots);
    l.n_tops = b.n_tops;
    l.counts = (int32_t*)(l.tops + (int64_t)a.rows * b.n_tops);
    l.parts = (int32_t)((b.chunks + kTopThreads / 64 - 1) / (kTopThreads / 64));
    const int64_t most = std::max<int64_t>(1, (1 << 21) / l.parts);
    for (l.row0 = 0; l.row0 < a.rows; l.row0 += most) {
      const int64_t rows = std::min<int64_t>(most, a.rows - l.row0);
      hipLaunchKernelGGL(tops_kernel, dim3((uint32_t)(rows * l.parts)), dim3(kTopThreads), 0, s, a, l, b.shift);
    }
    l.part = kMiddle;
    l.parts = (int32_t)b.parts;
    launch<kSelectThreads, kMiddle / kSelectThreads, kBounded>(a, l, s);
    l.parts_in = l.parts;
    l.parts = 1;
    launch<kSelectThreads, kMost / kSelectThreads, kJoin>(a, l, s);
    return hipGetLastError();
  }
  char* work = a.work;
  for (;;) {
    const bool last = l.n_in <= kMost;
    l.part = last ? kMost : part_of(a.k);
    l.parts = (int32_t)((l.n_in + l.part - 1) / l.part);
    if (l.parts == 0) l.parts = 1;
    const int64_t left = (int64_t)l.parts * a.k, most = l.n_in < l.part ? l.n_in : l.part;  // of a workgroup
    l.out = last ? nullptr : (float*)work;
    l.out_idx = (int32_t*)(work + (uint64_t)a.rows * left * 4);
    // (the smaller kernels where they do: 256 rows of 4096 in 7.5 us, 9.4 with the next, 2048 of 8192 in 45, 60 with the next;
    // but a workgroup that has a unit to itself may as well have all of its registers: 256 rows of 16384 11.4 -> 10.5)
    if (most <= kShort) launch<kShortThreads, kShort / kShortThreads>(a, l, s);
    else if (most <= kMiddle && (int64_t)a.rows * l.parts > kUnits) launch<kSelectThreads, kMiddle / kSelectThreads>(a, l, s);
    else launch<kSelectThreads, kMost / kSelectThreads>(a, l, s);
    if (last) return hipGetLastError();
    work += (uint64_t)a.rows * left * 8;
    l.in = l.out;
    l.idx = l.out_idx;
    l.n_in = left;
  }
}

}  // namespace hs
