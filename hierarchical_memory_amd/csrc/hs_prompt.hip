// A prompt's latent attention, expanded form, over ragged sequences (gfx950).
#include "hs_latent.h"

namespace hs {

namespace {

__device__ __forceinline__ float bf(uint16_t v) { return __uint_as_float((uint32_t)v << 16); }

constexpr int kPromptThreads = 256;

__device__ __forceinline__ int cut(int v, int n) { return v < 0 ? 0 : v > n ? n : v; }

// One workgroup per query and head, in tiles of 256 keys.
__global__ __launch_bounds__(kPromptThreads) void prompt_kernel(PromptArgs a) {
  __shared__ float p[kPromptThreads], red[kPromptThreads];
  __shared__ int seq;
  const int tid = threadIdx.x, h = blockIdx.y;
  const int D = a.nope + a.rope, K = a.nope + a.value;
  for (int t = blockIdx.x; t < a.n_q; t += gridDim.x) {
    __syncthreads();
    if (tid == 0) seq = -1;
    __syncthreads();
    for (int r = tid; r < a.R; r += kPromptThreads)
      if (t >= cut(a.cu_q[r], a.n_q) && t < cut(a.cu_q[r + 1], a.n_q)) seq = r;
    __syncthreads();
    if (seq < 0) continue;
    const int q1 = cut(a.cu_q[seq + 1], a.n_q);
    const int k0 = cut(a.cu_k[seq], a.n_k), k1 = cut(a.cu_k[seq + 1], a.n_k);
    int n = k1 - k0;
    if (a.causal) n -= q1 - 1 - t;
    if (n < 0) n = 0;
    const uint16_t* q = a.q + ((size_t)t * a.heads + h) * D;
    float m = -INFINITY, l = 0.0f, o = 0.0f;
    for (int j0 = 0; j0 < n; j0 += kPromptThreads) {
      const int j = j0 + tid;
      float s = -INFINITY;
      if (j < n) {
        const uint16_t* key = a.kv + ((size_t)(k0 + j) * a.heads + h) * K;
        const uint16_t* kr = a.krope + (size_t)(k0 + j) * a.rope_stride;
        s = 0.0f;
        for (int d = 0; d < a.nope; ++d) s += bf(q[d]) * bf(key[d]);
        for (int d = 0; d < a.rope; ++d) s += bf(q[a.nope + d]) * bf(kr[d]);
        s *= a.scale;
      }
      red[tid] = s;
      __syncthreads();
      float top = m;
      for (int i = 0; i < kPromptThreads; ++i) top = fmaxf(top, red[i]);
      const float top0 = top == -INFINITY ? 0.0f : top;
      const float c = __expf(m - top0);
      p[tid] = __expf(s - top0);
      __syncthreads();
      l *= c;
      o *= c;
      for (int i = 0; i < kPromptThreads && j0 + i < n; ++i) {
        l += p[i];
        if (tid < a.value) o += p[i] * bf(a.kv[((size_t)(k0 + j0 + i) * a.heads + h) * K + a.nope + tid]);
      }
      m = top;
      __syncthreads();
    }
    if (tid < a.value) {
      __bf16 b = (__bf16)(l > 0.0f ? o / l : 0.0f);
      a.o[((size_t)t * a.heads + h) * a.value + tid] = __builtin_bit_cast(uint16_t, b);
    }
    if (a.lse && tid == 0) a.lse[(size_t)t * a.heads + h] = m + logf(l);
  }
}

}  // namespace

hipError_t launch_prompt(const PromptArgs& a, hipStream_t s) {
  if (a.n_q <= 0) return hipSuccess;
  hipLaunchKernelGGL(prompt_kernel, dim3(a.n_q < 65536 ? a.n_q : 65536, a.heads), dim3(kPromptThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hs
