// The k best positions of each row of scores, ascending (gfx950).
//
// A workgroup reads its part of a row once, into registers, 64 consecutive positions to a wave's load. What is selected is kept as
// a mask of each such load, and a thread then writes the positions of one mask: passes over the registers are unrolled code that
// runs once and waits for its own instructions, and three of them are enough (with two more, to count and to write by ballots,
// 256 rows of 40960 took 31 us). The k-th best score is found without a sort. It is no lower than the lowest of the threads' own
// best scores (or second best, and so on: as many as make k); what lies above is counted in bins, even in value (which keeps a
// wave's counts apart, where the bits of the scores would share few bins), and the scores of the one bin that the k-th lies in,
// some dozens, are ranked against each other with their positions. A bin of more than kList (few different scores, or outliers
// that stretch the range) is divided further, by the scores' bits, until kList are left or all are equal; the first of the
// equal ones are then taken in order.
// A row of more than kMost positions is cut into parts, whose best k (with their positions, in order) are the row of the next
// launch; ties stay with the lowest positions, as every launch keeps the order.
#include "hs_index.h"

#include <algorithm>

namespace hs {

namespace {

constexpr int kSelectThreads = 1024;         // of a workgroup, for rows of more than kShort
constexpr int kShortThreads = 512;
constexpr int kShort = 8 * kShortThreads;
constexpr int kList = 512;                   // scores of a bin that are ranked against each other
constexpr int kMost = 48 * kSelectThreads;   // positions of a workgroup
constexpr int kMiddle = 16 * kSelectThreads; // up to which a kernel that takes half of the registers is used

struct SelectLevel {
  const float* in;      // rows of n_in scores
  const int32_t* idx;   // their positions, or nullptr (first launch: their places)
  int64_t n_in;
  int64_t part;         // of a row, to a workgroup
  int64_t row0;         // of the launch
  int32_t parts;
  float* out;           // not the last launch: [row][parts][k] scores, -inf behind the selected, and
  int32_t* out_idx;     // their positions
};

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

template <class Op>
__device__ __forceinline__ float wave_reduce(float v, Op op) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = op(v, __shfl_xor(v, d));
  return v;
}

// kPer: most scores of a thread, kBlock of them in a block: a workgroup passes over as many blocks as its part has.
template <int kThreads, int kPer>
__global__ __launch_bounds__(kThreads, kPer <= 16 ? 8 : 4) void select_kernel(SelectArgs a, SelectLevel l) {
  constexpr int kWaves = kThreads / 64, kBins = 2 * kThreads, kBlock = 8;
  constexpr int kBest = 2048 / kThreads;  // of a thread's scores, for the bound
  __shared__ int hist[kBins];
  __shared__ uint64_t list[kList];
  __shared__ int rank[kList];
  __shared__ uint64_t masks[kWaves * kPer], ties[kWaves * kPer];  // of the loads, in the order of the positions
  __shared__ int sums[kWaves], tie_sums[kWaves], taken_sums[kWaves], found[4];
  __shared__ uint16_t chosen[kMaxTopK];
  __shared__ float lows[kWaves], highs[kWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = l.row0 + blockIdx.x / l.parts;
  const int part = (int)(blockIdx.x % l.parts);
  const bool whole = l.out == nullptr;
  // the positions of the row's token, those that compete, and how many of them are selected
  int64_t m, from = row;  // from: row of the scores
  {
    int64_t t = row;
    if (a.cu) {
      t = a.cu[row + 1] > a.cu[row] ? (int64_t)a.cu[row + 1] - 1 : -1;
      if (t >= a.n) t = -1;
    }
    m = t < 0 ? 0 : (int64_t)a.pos[t] + 1;
    m = m < 0 ? 0 : m < a.columns ? m : a.columns;
    if (!l.idx) from = t < 0 ? 0 : t;
  }
  const int recent = m < a.recent ? (int)m : a.recent, k = a.k - recent;
  const int64_t rivals = l.idx ? l.n_in : m - recent, begin = part * l.part;
  const int n = (int)(rivals <= begin ? 0 : rivals - begin < l.part ? rivals - begin : l.part);
  const int blocks = (n + kThreads * kBlock - 1) / (kThreads * kBlock);
  const int first = wave * blocks * kBlock * 64;  // of the wave
  float x[kPer];
  // f(j) for the wave's loads, in their order
  auto each = [&](auto f) {
#pragma unroll
    for (int b = 0; b < kPer / kBlock; ++b)
      if (b < blocks) {
#pragma unroll
        for (int i = 0; i < kBlock; ++i) {
          asm volatile("" : "+v"(x[b * kBlock + i]));  // nothing that a pass works out is kept for the next: registers are short
          f(b * kBlock + i);
        }
      }
  };
  {
    const float* in = l.in + from * l.n_in + begin + first;
#pragma unroll
    for (int b = 0; b < kPer / kBlock; ++b)
      if (b < blocks) {
        const int left = n - first - b * kBlock * 64;  // of the part, from this block on
        if (left >= kBlock * 64) {
#pragma unroll
          for (int i = 0; i < kBlock; ++i) x[b * kBlock + i] = in[(b * kBlock + i) * 64 + lane];
        } else {
#pragma unroll
          for (int i = 0; i < kBlock; ++i) x[b * kBlock + i] = i * 64 + lane < left ? in[(b * kBlock + i) * 64 + lane] : -INFINITY;
        }
      }
  }
  hist[tid] = hist[tid + kThreads] = 0;
  for (int i = tid; i < kList; i += kThreads) rank[i] = 0;
  if (tid == 0) found[3] = 0;
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
  const auto lesser = [](float u, float v) { return fminf(u, v); };
  const auto larger = [](float u, float v) { return fmaxf(u, v); };
  float hi = wave_reduce(best[0], larger);
  float lo = wave_reduce(bound, lesser);
  if (lane == 0) lows[wave] = lo, highs[wave] = hi;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    lo = fminf(lo, lows[w]);
    hi = fmaxf(hi, highs[w]);
  }
  // the loads' masks of f(j), to LDS
  auto mask_of = [&](uint64_t* to, auto f) {
    uint32_t low = 0, high = 0;
    each([&](int j) {
      const uint64_t mask = __ballot(f(j));
      low = lane == j ? (uint32_t)mask : low;
      high = lane == j ? (uint32_t)(mask >> 32) : high;
    });
    if (lane < blocks * kBlock) to[wave * blocks * kBlock + lane] = (uint64_t)high << 32 | low;
  };
  int tied = 0;        // of the equal scores in `ties`, those that are selected
  bool every = false;  // what may be selected is
  if (lo == -INFINITY) {
    // too few scores for that bound: the lowest that may be selected, and how many may (a NaN becomes -infinity, so that no ballot
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
  const int loads = kWaves * blocks * kBlock, split = loads <= kThreads / 8 ? 3 : loads <= kThreads / 4 ? 2 : loads <= kThreads / 2 ? 1 : 0;
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
  const int64_t to = whole ? row * a.k : (row * l.parts + part) * a.k;
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
  if (whole) {
    for (int i = all + tid; i < a.k; i += kThreads) a.topk[to + i] = i < all + recent ? (int32_t)(m - recent + i - all) : -1;
  } else {
    for (int i = all + tid; i < a.k; i += kThreads) l.out[to + i] = -INFINITY;
  }
}

template <int kThreads, int kPer>
void launch(const SelectArgs& a, SelectLevel l, hipStream_t s) {
  const int64_t most = std::max<int64_t>(1, (1 << 21) / l.parts);  // rows of a launch (which ends below 2^32 threads)
  for (l.row0 = 0; l.row0 < a.rows; l.row0 += most) {
    const int64_t rows = std::min<int64_t>(most, a.rows - l.row0);
    hipLaunchKernelGGL((select_kernel<kThreads, kPer>), dim3((uint32_t)(rows * l.parts)), dim3(kThreads), 0, s, a, l);
  }
}

// The part into which a launch cuts rows of more than kMost: one that leaves an eighth of them and runs two workgroups to a unit, or,
// where that would leave more than a quarter, the longest (2 rows of 1 M, k 2048: 62 parts, then 8, then one, 33 us; in parts of 41 K
// 48).
int64_t part_of(int k) { return 4 * k <= kMiddle ? kMiddle : kMost; }

}  // namespace

// Every launch but the last leaves k scores and positions of each part.
uint64_t select_work_bytes(int rows, int64_t columns, int k) {
  uint64_t bytes = 0;
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
  char* work = a.work;
  for (;;) {
    const bool last = l.n_in <= kMost;
    l.part = last ? kMost : part_of(a.k);
    l.parts = (int32_t)((l.n_in + l.part - 1) / l.part);
    if (l.parts == 0) l.parts = 1;
    const int64_t left = (int64_t)l.parts * a.k, most = l.n_in < l.part ? l.n_in : l.part;  // of a workgroup
    l.out = last ? nullptr : (float*)work;
    l.out_idx = (int32_t*)(work + (uint64_t)a.rows * left * 4);
    if (most <= kShort) launch<kShortThreads, kShort / kShortThreads>(a, l, s);
    else if (most <= kMiddle) launch<kSelectThreads, kMiddle / kSelectThreads>(a, l, s);
    else launch<kSelectThreads, kMost / kSelectThreads>(a, l, s);
    if (last) return hipGetLastError();
    work += (uint64_t)a.rows * left * 8;
    l.in = l.out;
    l.idx = l.out_idx;
    l.n_in = left;
  }
}

}  // namespace hs
