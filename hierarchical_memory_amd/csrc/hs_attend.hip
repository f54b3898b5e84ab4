// One decode step's latent attention over the selected rows (gfx950).
#include "hs_latent.h"

namespace hs {

namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

__device__ __forceinline__ float row_value(const char* row, const RowLayout& l, int d) {
  if (d >= l.latent) return bf(((const uint16_t*)(row + l.rope_at))[d - l.latent]);
  if (!l.mx) return bf(((const uint16_t*)row)[d]);
  const uint32_t q = ((const uint8_t*)row)[d], s = ((const uint8_t*)(row + l.scales))[d / kScaleBlock];
  return __builtin_amdgcn_cvt_f32_fp8(q, 0) * __uint_as_float(s << 23);
}

__device__ __forceinline__ const char* row_of(const AttendArgs& a, int r, int i) {
  const int s = a.out[(size_t)r * a.k + i];
  if (s < 0 || s >= a.B + a.T) return nullptr;
  if (a.gather) return a.gather + ((size_t)r * a.k + i) * a.row.bytes;
  return s < a.B ? a.hot + ((size_t)r * a.B + s) * a.row.bytes : a.tail + ((size_t)r * a.T + s - a.B) * a.row.bytes;
}

constexpr int kAttendThreads = 256;

// One workgroup per request and head: scores by wave, then each thread sums its dimensions.
__global__ __launch_bounds__(kAttendThreads) void attend_kernel(AttendArgs a) {
  extern __shared__ float p[];  // [k]
  __shared__ float red[kAttendThreads];
  const int r = blockIdx.x, h = blockIdx.y, tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int L = a.row.latent, D = L + a.row.rope;
  const uint16_t* q = a.q + ((size_t)r * a.heads + h) * D;
  float m = -INFINITY;
  for (int i = wave; i < a.k; i += kAttendThreads / 64) {
    const char* row = row_of(a, r, i);
    float s = 0.0f;
    if (row)
      for (int d = lane; d < D; d += 64) s += bf(q[d]) * row_value(row, a.row, d);
    for (int d = 1; d < 64; d <<= 1) s += __shfl_xor(s, d);
    s = row ? s * a.scale : -INFINITY;
    if (lane == 0) p[i] = s;
    m = fmaxf(m, s);
  }
  red[tid] = m;
  __syncthreads();
  for (int i = 0; i < kAttendThreads; ++i) m = fmaxf(m, red[i]);
  const float m0 = m == -INFINITY ? 0.0f : m;
  float l = 0.0f;
  for (int i = 0; i < a.k; ++i) l += __expf(p[i] - m0);
  for (int d = tid; d < L; d += kAttendThreads) {
    float o = 0.0f;
    for (int i = 0; i < a.k; ++i) {
      const char* row = row_of(a, r, i);
      if (row) o += __expf(p[i] - m0) * row_value(row, a.row, d);
    }
    o = l > 0.0f ? o / l : o;
    __bf16 b = (__bf16)o;
    a.o[((size_t)r * a.heads + h) * L + d] = __builtin_bit_cast(uint16_t, b);
  }
  if (a.lse && tid == 0) a.lse[(size_t)r * a.heads + h] = m + logf(l);
}

}  // namespace

int attend_splits(int, int, int, const RowLayout&) { return 1; }
uint64_t attend_work_bytes(int, int, int, const RowLayout&) { return 0; }

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  hipLaunchKernelGGL(attend_kernel, dim3(a.R, a.heads), dim3(kAttendThreads), (size_t)a.k * 4, s, a);
  return hipGetLastError();
}

}  // namespace hs
