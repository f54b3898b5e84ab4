// The k best positions of each row of scores, ascending (gfx950).
//
// A workgroup reads its part of a row once, into registers, 64 consecutive positions to a wave's load, so that what is selected
// leaves in order by ballots. The k-th best score is found without a sort: scores are counted in 2048 bins between the lowest and
// the highest of them, even in value (which keeps a wave's counts apart, where the bits of the scores would share few bins); the
// scores of the one bin that the k-th lies in, some dozens, are ranked against each other with their positions. A bin of more
// than kList (few different scores, or outliers that stretch the range) is divided further by the scores' bits instead, and the
// positions of equal ones are counted in order. The selection is then a comparison with one score and one position.
// A row of more than kMost positions is cut into parts, whose best k (with their positions, in order) are the row of the next
// launch; ties stay with the lowest positions, as every launch keeps the order.
#include "hs_index.h"

namespace hs {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;
constexpr int kBins = 2 * kSelectThreads;
constexpr int kList = 512;                   // scores of a bin that are ranked against each other
constexpr int kMost = 48 * kSelectThreads;   // positions of a workgroup
constexpr int kLeastPart = 8192;             // of a part of a longer row

struct SelectLevel {
  const float* in;      // rows of n_in scores
  const int32_t* idx;   // their positions, or nullptr (first launch: their places)
  int64_t n_in;
  int64_t part;         // of a row, to a workgroup
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

// kPer: most scores of a thread.
template <int kPer>
__global__ __launch_bounds__(kSelectThreads) void select_kernel(SelectArgs a, SelectLevel l) {
  __shared__ int hist[kBins];
  __shared__ uint64_t list[kList];
  __shared__ int sums[kSelectWaves], found[4];
  __shared__ float lows[kSelectWaves], highs[kSelectWaves];
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int64_t row = blockIdx.x / l.parts;
  const int part = (int)(blockIdx.x % l.parts);
  const bool whole = l.out == nullptr;
  // the positions of the row's token, those that compete, and how many of them are selected
  int64_t m, rivals, from = row;  // from: row of the scores
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
  rivals = l.idx ? l.n_in : m - recent;
  const int64_t begin = part * l.part;
  const int n = (int)(rivals <= begin ? 0 : rivals - begin < l.part ? rivals - begin : l.part);
  const float* in = l.in + from * l.n_in + begin;

  const int per = (n + kSelectThreads - 1) / kSelectThreads;  // of a thread
  const int first = wave * per * 64;                          // of the wave
  float x[kPer];
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < per) {
      const int i = first + j * 64 + lane;
      x[j] = i < n ? in[i] : -INFINITY;
    }
  hist[tid] = hist[tid + kSelectThreads] = 0;
  if (tid == 0) found[3] = 0;
  // a NaN becomes -infinity: what is never selected has one form, and no comparison below meets a NaN
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < per) x[j] = x[j] == x[j] ? x[j] : -INFINITY;
  float lo = INFINITY, hi = -INFINITY;
  int valid = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < per) {
      const bool is = x[j] > -INFINITY;
      lo = fminf(lo, is ? x[j] : INFINITY);
      hi = fmaxf(hi, is && x[j] < INFINITY ? x[j] : -INFINITY);
      valid += __popcll(__ballot(is));
    }
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    lo = fminf(lo, __shfl_xor(lo, d));
    hi = fmaxf(hi, __shfl_xor(hi, d));
  }
  if (lane == 0) lows[wave] = lo, highs[wave] = hi, sums[wave] = valid;
  __syncthreads();
  valid = 0;
#pragma unroll
  for (int w = 0; w < kSelectWaves; ++w) {
    lo = fminf(lo, lows[w]);
    hi = fmaxf(hi, highs[w]);
    valid += sums[w];
  }
  // what is selected: a score above `least`, or equal to it up to the position `last`
  float least = -INFINITY;
  int last = -1;
  if (valid > k) {
    // (a range that is zero or past 32 bits puts every finite score, or all but the lowest, into one bin)
    const float step = (float)(kBins - 1) / (hi - lo);
    auto bin_of = [&](float v) {
      const float b = (v - lo) * step;
      return b > 0.0f ? b < (float)(kBins - 1) ? (int)b : kBins - 1 : 0;  // (a NaN: 0)
    };
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (j < per && x[j] > -INFINITY) atomicAdd(&hist[bin_of(x[j])], 1);
    __syncthreads();
    {
      const int b = kBins - 2 - 2 * tid, upper = hist[b + 1], both = upper + hist[b];
      const int upto = wave_scan(both);
      if (lane == 63) sums[wave] = upto;
      __syncthreads();
      int before = upto - both;
#pragma unroll
      for (int w = 0; w < kSelectWaves; ++w)
        if (w < wave) before += sums[w];
      if (before < k && before + both >= k) {  // (one thread; none where k is zero)
        const bool in_upper = before + upper >= k;
        found[0] = in_upper ? b + 1 : b;
        found[1] = in_upper ? k - before : k - before - upper;
      }
      if (k == 0 && tid == 0) found[0] = kBins, found[1] = 0;
    }
    __syncthreads();
    const int bin = found[0];
    int need = found[1];
    const int count = bin < kBins ? hist[bin] : 0;
    if (k == 0) {
      least = INFINITY;
    } else if (count <= kList) {
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j < per && x[j] > -INFINITY && bin_of(x[j]) == bin)
          list[atomicAdd(&found[3], 1)] = (uint64_t)order_of(x[j]) << 32 | (uint32_t)~(first + j * 64 + lane);
      __syncthreads();
      if (tid < count) {
        const uint64_t mine = list[tid];
        int better = 0;
        for (int i = 0; i < count; ++i) better += list[i] > mine;
        if (better == need - 1) {
          found[0] = (int)(mine >> 32);
          found[1] = (int)~(uint32_t)mine;
        }
      }
      __syncthreads();
      least = score_of((uint32_t)found[0]);
      last = found[1];
    } else {
      uint32_t prefix = 0;
#pragma unroll 1
      for (int shift = 24; shift >= 0; shift -= 8) {
        __syncthreads();  // the counts before are read
        if (tid < 256) hist[tid] = 0;
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j < per && x[j] > -INFINITY && bin_of(x[j]) == bin) {
            const uint32_t u = order_of(x[j]);
            if (shift == 24 || u >> (shift + 8) == prefix >> (shift + 8)) atomicAdd(&hist[u >> shift & 255], 1);
          }
        __syncthreads();
        if (wave == 0) {  // a lane has four digits, from the highest on
          const int d = 252 - 4 * lane;
          const int c[4] = {hist[d + 3], hist[d + 2], hist[d + 1], hist[d]};
          const int all = c[0] + c[1] + c[2] + c[3];
          int before = wave_scan(all) - all;
          if (before < need && before + all >= need) {
            int i = 0;
            while (before + c[i] < need) before += c[i++];
            found[0] = d + 3 - i;
            found[1] = need - before;
          }
        }
        __syncthreads();
        prefix |= (uint32_t)found[0] << shift;
        need = found[1];
      }
      least = score_of(prefix);
      // the position of the need-th score that is equal to it
      int equal = 0;
#pragma unroll
      for (int j = 0; j < kPer; ++j)
        if (j < per) equal += __popcll(__ballot(x[j] == least));
      if (lane == 0) sums[wave] = equal;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < wave; ++w) before += sums[w];
      if (before < need && before + equal >= need) {
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (j < per) {
            const uint64_t mask = __ballot(x[j] == least);
            const int rank = before + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
            if (x[j] == least && rank == need - 1) found[2] = first + j * 64 + lane;
            before += __popcll(mask);
          }
      }
      __syncthreads();
      last = found[2];
    }
  }
  int count = 0;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < per) count += __popcll(__ballot(x[j] > least || (x[j] == least && first + j * 64 + lane <= last)));
  __syncthreads();  // what the sums held is read
  if (lane == 0) sums[wave] = count;
  __syncthreads();
  int at = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w < wave) at += sums[w];
    all += sums[w];
  }
  const int64_t to = whole ? row * a.k : (row * l.parts + part) * a.k;
#pragma unroll
  for (int j = 0; j < kPer; ++j)
    if (j < per) {
      const int i = first + j * 64 + lane;
      const bool is = x[j] > least || (x[j] == least && i <= last);
      const uint64_t mask = __ballot(is);
      if (is) {
        const int64_t o = to + at + __builtin_amdgcn_mbcnt_hi((uint32_t)(mask >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)mask, 0));
        const int32_t id = l.idx ? l.idx[row * l.n_in + begin + i] : (int32_t)(begin + i);
        if (whole) {
          a.topk[o] = id;
        } else {
          l.out[o] = x[j];
          l.out_idx[o] = id;
        }
      }
      at += __popcll(mask);
    }
  if (whole) {
    for (int i = all + tid; i < a.k; i += kSelectThreads) a.topk[to + i] = i < all + recent ? (int32_t)(m - recent + i - all) : -1;
  } else {
    for (int i = all + tid; i < a.k; i += kSelectThreads) l.out[to + i] = -INFINITY;
  }
}

template <int kPer>
void launch(const SelectArgs& a, const SelectLevel& l, hipStream_t s) {
  hipLaunchKernelGGL(select_kernel<kPer>, dim3((uint32_t)((int64_t)a.rows * l.parts)), dim3(kSelectThreads), 0, s, a, l);
}

// Positions to a workgroup in a launch over rows of n > kMost: as few as leave the next launch one workgroup to a row, where
// there are such.
int64_t part_of(int64_t n, int k) {
  const int64_t parts = kMost / k, part = (n + parts - 1) / parts;
  return part < kLeastPart ? kLeastPart : part < kMost ? part : kMost;
}

// Scores of a row that it leaves.
int64_t left_of(int64_t n, int k) { return (n + part_of(n, k) - 1) / part_of(n, k) * k; }

}  // namespace

// Every launch but the last leaves k scores and positions of each part.
uint64_t select_work_bytes(int rows, int64_t columns, int k) {
  uint64_t bytes = 0;
  for (int64_t n = columns; n > kMost; n = left_of(n, k)) bytes += (uint64_t)rows * left_of(n, k) * 8;
  return (bytes + 15) & ~15ull;
}

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  SelectLevel l{};
  l.in = a.scores;
  l.n_in = a.columns;
  char* work = a.work;
  while (l.n_in > kMost) {
    const int64_t left = left_of(l.n_in, a.k);
    l.part = part_of(l.n_in, a.k);
    l.parts = (int32_t)(left / a.k);
    l.out = (float*)work;
    l.out_idx = (int32_t*)(work + (uint64_t)a.rows * left * 4);
    launch<kMost / kSelectThreads>(a, l, s);
    work += (uint64_t)a.rows * left * 8;
    l.in = l.out;
    l.idx = l.out_idx;
    l.n_in = left;
  }
  l.part = kMost;
  l.parts = 1;
  l.out = nullptr;
  l.out_idx = nullptr;
  const int64_t per = (l.n_in + kSelectThreads - 1) / kSelectThreads;
  if (per <= 4) launch<4>(a, l, s);
  else if (per <= 16) launch<16>(a, l, s);
  else launch<48>(a, l, s);
  return hipGetLastError();
}

}  // namespace hs
