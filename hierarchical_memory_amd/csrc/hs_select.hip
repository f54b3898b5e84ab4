// The k best positions of each row of scores, ascending (gfx950).
//
// A score's order as 32 bits (0: never selected); the k-th largest is found digit by digit, 8 bits a pass, and the row is then
// read in order: what is larger is selected, and of what is equal as many as there is room for, the lowest first.
#include "hs_index.h"

namespace hs {

namespace {

constexpr int kSelectThreads = 1024;
constexpr int kSelectWaves = kSelectThreads / 64;

__device__ __forceinline__ uint32_t order_of(float x) {
  uint32_t u = __float_as_uint(x);
  if ((u & 0x7fffffffu) > 0x7f800000u || u == 0xff800000u) return 0;
  if (u == 0x80000000u) u = 0;
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive scan of one value per thread, and the total.
__device__ __forceinline__ int block_scan(int v, int* sh, int* total) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int x = v;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int y = __shfl_up(x, d);
    if (lane >= d) x += y;
  }
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSelectWaves; ++w) {
    if (w < wave) before += sh[w];
    all += sh[w];
  }
  __syncthreads();
  *total = all;
  return before + x - v;
}

__global__ __launch_bounds__(kSelectThreads) void select_kernel(SelectArgs a) {
  __shared__ int hist[256], sh[kSelectWaves], found[2];
  const int tid = threadIdx.x;
  const int64_t row = blockIdx.x;
  int64_t t = row;
  if (a.cu) {
    t = a.cu[row + 1] > a.cu[row] ? (int64_t)a.cu[row + 1] - 1 : -1;
    if (t >= a.n) t = -1;
  }
  int64_t m = t < 0 ? 0 : (int64_t)a.pos[t] + 1;  // positions
  m = m < 0 ? 0 : m < a.columns ? m : a.columns;
  const float* s = a.scores + (t < 0 ? 0 : t) * a.columns;
  int32_t* out = a.topk + row * a.k;
  auto order = [&](int64_t i) -> uint32_t { return i >= m ? 0u : i >= m - a.recent ? 0xffffffffu : order_of(s[i]); };
  uint32_t prefix = 0;
  int need = a.k;  // of those with the prefix so far
  bool all = false;
  for (int shift = 24; shift >= 0 && !all; shift -= 8) {
    if (tid < 256) hist[tid] = 0;
    __syncthreads();
    for (int64_t i = tid; i < m; i += kSelectThreads) {
      const uint32_t u = order(i);
      if (u && (shift == 24 || u >> (shift + 8) == prefix >> (shift + 8))) atomicAdd(&hist[u >> shift & 255], 1);
    }
    __syncthreads();
    if (tid == 0) {
      int sum = 0, b = 255;
      for (; b >= 0; --b) {
        if (sum + hist[b] >= need) break;
        sum += hist[b];
      }
      found[0] = b;
      found[1] = need - sum;
    }
    __syncthreads();
    if (found[0] < 0) {  // fewer than k
      all = true;
    } else {
      prefix |= (uint32_t)found[0] << shift;
      need = found[1];
    }
    __syncthreads();
  }
  if (all) prefix = 0, need = 0;
  int at = 0, equal = 0;  // selected, and of those equal to the k-th
  for (int64_t i0 = 0; i0 < m; i0 += kSelectThreads) {
    const int64_t i = i0 + tid;
    const uint32_t u = order(i);
    int total;
    const int rank = equal + block_scan(u && u == prefix, sh, &total);
    equal += total;
    const bool taken = u > prefix || (u && u == prefix && rank < need);
    const int place = at + block_scan(taken, sh, &total);
    at += total;
    if (taken) out[place] = (int32_t)i;
  }
  for (int i = at + tid; i < a.k; i += kSelectThreads) out[i] = -1;
}

}  // namespace

uint64_t select_work_bytes(int, int64_t, int) { return 0; }

hipError_t launch_select(const SelectArgs& a, hipStream_t s) {
  if (a.rows <= 0) return hipSuccess;
  hipLaunchKernelGGL(select_kernel, dim3(a.rows), dim3(kSelectThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hs
