// The map of a ragged batch of new tokens and the store of their rows (gfx950).
#include "hs_latent.h"

namespace hs {

namespace {

constexpr int kStatusBad = 1;  // HS_STATUS_BAD_ID

// ---- map ----
//
// Every workgroup scans all requests' counts by itself (4 bytes a request, from L2), so the map is one launch
// without a second pass or any exchange between workgroups, and then fills its own kMapTokens tokens: requests that
// begin inside them leave their number at their first token's place in LDS (no two with tokens begin at the same one),
// and a maximum scan over the places carries it to the tokens behind. Latency bounds it: two rounds of reads (counts, then the
// requests' lengths) and three scans before the first store. 4.7 us for 256 requests with a token each, 10 us for 4096
// requests with 1 M tokens (12.7 MB); 8 requests to a thread, half the rounds, took 15.
constexpr int kMapThreads = 512;
constexpr int kMapWaves = kMapThreads / 64;
constexpr int kMapPer = 4;  // requests a thread takes in a round of the scan, and tokens it fills
constexpr int kMapTokens = kMapThreads * kMapPer;

struct SatAdd {  // sums cut off at cap: associative over values in [0, cap], and below 2^31 for cap <= 2^30
  int cap;
  __device__ int operator()(int a, int b) const {
    const int s = a + b;
    return s < cap ? s : cap;
  }
};
struct MaxOp {
  __device__ int operator()(int a, int b) const { return a > b ? a : b; }
};

// Exclusive scan of one value per thread (0 the neutral element), and the total of all. Inside a wave by lane shifts: 1, 2,
// 4, 8 in each row of 16, then lane 15 into the rows 1 and 3, lane 31 into the rows 2 and 3.
template <class Op>
__device__ __forceinline__ int map_scan(int v, Op op, int* sh, int lane, int wave, int* total) {
  int x = v;
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x111, 0xf, 0xf, false), x);
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x112, 0xf, 0xf, false), x);
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x114, 0xf, 0xf, false), x);
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x118, 0xf, 0xf, false), x);
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x142, 0xa, 0xf, false), x);
  x = op(__builtin_amdgcn_update_dpp(0, x, 0x143, 0xc, 0xf, false), x);
  if (lane == 63) sh[wave] = x;
  __syncthreads();
  int before = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kMapWaves; ++w) {
    const int t = sh[w];
    if (w < wave) before = op(before, t);
    all = op(all, t);
  }
  __syncthreads();  // sh is free again
  const int e = __builtin_amdgcn_update_dpp(0, x, 0x138, 0xf, 0xf, false);  // of the lane before
  *total = all;
  return lane == 0 ? before : op(before, e);
}

__global__ __launch_bounds__(kMapThreads) void map_kernel(MapArgs a) {
  __shared__ int owner[kMapTokens];  // at a request's first token of this workgroup: its number + 1, else 0
  __shared__ int sh[kMapWaves];
  __shared__ int first_start;        // start of the request that holds this workgroup's first token
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int lo = blockIdx.x * kMapTokens;  // below 2^30 + kMapTokens
  const int n = a.n;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) owner[tid + i * kMapThreads] = 0;
  __syncthreads();
  // the requests' own outputs are shared out over the workgroups, as their tokens are
  const int share = (int)(((uint32_t)a.R + gridDim.x - 1) / gridDim.x);
  const int64_t own0 = (int64_t)blockIdx.x * share, own1 = own0 + share;
  int base = 0;
  for (int r0 = 0; r0 < a.R; r0 += kMapThreads * kMapPer) {
    if (base >= lo + kMapTokens && r0 >= own1) break;  // nothing behind is this workgroup's
    int len[kMapPer], raw[kMapPer], sum = 0;
    int had[kMapPer], window[kMapPer];
    bool own[kMapPer];
    const SatAdd add{n};
#pragma unroll
    for (int i = 0; i < kMapPer; ++i) {
      const int r = r0 + tid * kMapPer + i;
      raw[i] = r < a.R ? a.fresh[r] : 0;
      own[i] = r < a.R && r >= own0 && r < own1;
      had[i] = own[i] && a.status ? a.len[r] : 0;
      window[i] = own[i] && a.status && a.T > 0 ? a.tail0[r] : 0;
      const int v = raw[i] < 0 ? 0 : raw[i];
      len[i] = v < n ? v : n;
      sum = add(sum, len[i]);
    }
    int total;
    int at = add(base, map_scan(sum, add, sh, lane, wave, &total));
#pragma unroll
    for (int i = 0; i < kMapPer; ++i) {
      const int r = r0 + tid * kMapPer + i;
      const int end = add(at, len[i]);
      if (r < a.R) {
        if (at < end && end > lo && at < lo + kMapTokens) {
          const int p = at > lo ? at - lo : 0;
          owner[p] = r + 1;
          if (p == 0) first_start = at;
        }
        if (own[i]) {
          a.cu[r] = at;
          if (r == a.R - 1) a.cu[a.R] = end;
          if (a.status) {
            bool bad = raw[i] < 0;
            if (end > at) {
              const int64_t x0 = had[i], x1 = x0 + (end - at) - 1;
              bad |= x0 < 0 || x1 >= a.H || (a.T > 0 && x1 >= (int64_t)window[i] + a.T);
            }
            a.status[r] = bad ? kStatusBad : 0;
          }
        }
      }
      at = end;
    }
    base = add(base, total);
  }
  __syncthreads();
  // the place of the last request start at or before each of the thread's tokens, as place + 1 (0: none)
  int mark[kMapPer], best = 0, unused;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int p = tid * kMapPer + i;
    if (owner[p]) best = p + 1;
    mark[i] = best;
  }
  const int before = map_scan(best, MaxOp(), sh, lane, wave, &unused);
  int req[kMapPer], at[kMapPer], had[kMapPer], window[kMapPer], pos[kMapPer], slot[kMapPer];
  const int t0 = lo + tid * kMapPer;
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int m = mark[i] ? mark[i] : before;
    const bool there = m && t0 + i < base;
    req[i] = there ? owner[m - 1] - 1 : -1;
    at[i] = t0 + i - (m == 1 ? first_start : lo + m - 1);
    had[i] = there ? a.len[req[i]] : 0;
    window[i] = there && a.T > 0 ? a.tail0[req[i]] : 0;
  }
#pragma unroll
  for (int i = 0; i < kMapPer; ++i) {
    const int64_t x = (int64_t)had[i] + at[i];
    bool fine = req[i] >= 0 && x >= 0 && x < a.H;
    slot[i] = -1;
    if (a.T > 0 && x >= window[i]) {
      if (x < (int64_t)window[i] + a.T) slot[i] = a.B + (int)((uint32_t)x % (uint32_t)a.T);
      else fine = false;
    }
    pos[i] = fine ? (int)x : -1;
    slot[i] = fine ? slot[i] : -1;
  }
  if (t0 + kMapPer <= n && (((uintptr_t)a.req | (uintptr_t)a.pos | (uintptr_t)a.slot) & 15) == 0) {
    *(int4*)(a.req + t0) = int4{req[0], req[1], req[2], req[3]};
    *(int4*)(a.pos + t0) = int4{pos[0], pos[1], pos[2], pos[3]};
    *(int4*)(a.slot + t0) = int4{slot[0], slot[1], slot[2], slot[3]};
    return;
  }
#pragma unroll
  for (int i = 0; i < kMapPer; ++i)
    if (t0 + i < n) {
      a.req[t0 + i] = req[i];
      a.pos[t0 + i] = pos[i];
      a.slot[t0 + i] = slot[i];
    }
}

// ---- store ----

typedef __bf16 bf8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

constexpr int kStoreThreads = 256;
constexpr int kStoreWaves = kStoreThreads / 64;

// One wave per token: a lane holds 8 latent values (16-byte loads and stores) and, below rope / 2, one pair of the rope
// part. The 4 lanes of a scale block share its largest magnitude. Memory bounds it: 41 K tokens of 512 + 64 values, 141 MB, in
// 31 us (4.5 TB/s, a copy reaches 4.8); 256 tokens in 3.8 us. Seven waves to a SIMD (72 registers): with six the large call takes
// 32.5 us.
__global__ __launch_bounds__(kStoreThreads, 7) void store_kernel(StoreArgs a) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int L = a.row.latent, P = a.row.rope / 2;
  const bool has = lane * 8 < L, pair = lane < P;
  const int i0 = a.halves ? lane : 2 * lane, i1 = a.halves ? lane + P : 2 * lane + 1;  // of the lane's pair
  bf8 w{};
  if (has) w = *(const bf8*)(a.weight + lane * 8);
  const double freq = pair && a.freqs ? a.freqs[lane] * 0.15915494309189535 : 0.0;  // turns per position
  const int64_t stride = (int64_t)gridDim.x * kStoreWaves;
  for (int64_t t = (int64_t)blockIdx.x * kStoreWaves + wave; t < a.n; t += stride) {
    // the input is on its way with what says where it goes
    const uint16_t* in = a.x + t * a.x_stride;
    bf8 v{};
    if (has) v = *(const bf8*)(in + lane * 8);
    __bf16 z0{}, z1{};
    if (pair) {
      const __bf16* xr = (const __bf16*)(in + L);
      z0 = xr[i0];
      z1 = xr[i1];
    }
    const int r = a.req[t], x = a.pos[t], slot = a.slot[t];
    if (r < 0 || x < 0 || r >= a.R) continue;
    const int ring = slot - a.B;
    const bool in_tail = slot >= a.B && ring < a.T;
    if (x >= a.H || !(in_tail || slot == -1)) {
      if (a.status && lane == 0) a.status[r] = kStatusBad;
      continue;
    }
    float y[8], sq = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = (float)v[i];
      sq += y[i] * y[i];
    }
    sq = wave_sum(sq);
    float inv = 1.0f / sqrtf(sq / (float)L + a.eps);
    if (!(sq > 1e-28f && sq < 1e38f)) {  // squares that 32 bits lose (the whole wave takes this branch, or none)
      double d = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) d += (double)y[i] * (double)y[i];
#pragma unroll
      for (int m = 1; m < 64; m <<= 1) d += __shfl_xor(d, m);
      // (the inverse too may be past 32 bits, 1e40 for the least of bf16's subnormals: the values are lifted first, exactly)
      const float lift = sq < 1.0f ? 0x1p40f : 0x1p-40f;
      inv = (float)(1.0 / sqrt((d / (double)L + (double)a.eps) * ((double)lift * lift)));
#pragma unroll
      for (int i = 0; i < 8; ++i) y[i] *= lift;
    }
    bf8 yb;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      y[i] = y[i] * inv * (float)w[i];
      yb[i] = (__bf16)y[i];
    }
    // the rope part: lane i has pair i
    if (pair) {
      if (a.freqs) {
        // the angle in turns, in 64 bits, less its whole turns: what is left of it is exact enough in 32
        const double turns = (double)x * freq;
        float s, c;
        sincospif((float)(2.0 * (turns - rint(turns))), &s, &c);
        const float u = (float)z0, q = (float)z1;
        z0 = (__bf16)(u * c - q * s);
        z1 = (__bf16)(u * s + q * c);
      }
    }
    // the 8-bit form: the block's largest magnitude m * 2^e, 1 <= m < 2, takes the scale 2^(e - 8), or 2^(e - 7)
    // where m > 1.75 (448 = 1.75 * 2^8)
    uint32_t lo8 = 0, hi8 = 0;
    int expo = 0;
    if (a.row.mx) {
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(y[i]));
      top = fmaxf(top, __shfl_xor(top, 1));
      top = fmaxf(top, __shfl_xor(top, 2));
      const uint32_t b = __float_as_uint(top);
      expo = (int)(b >> 23) - 127 - 8 + ((b & 0x7fffffu) > 0x600000u ? 1 : 0);
      expo = expo < -100 ? -100 : expo;
      const float f = __uint_as_float((uint32_t)(127 - expo) << 23);
      lo8 = __builtin_amdgcn_cvt_pk_fp8_f32(y[0] * f, y[1] * f, lo8, false);
      lo8 = __builtin_amdgcn_cvt_pk_fp8_f32(y[2] * f, y[3] * f, lo8, true);
      hi8 = __builtin_amdgcn_cvt_pk_fp8_f32(y[4] * f, y[5] * f, hi8, false);
      hi8 = __builtin_amdgcn_cvt_pk_fp8_f32(y[6] * f, y[7] * f, hi8, true);
    }
    auto write_row = [&](char* dst) {
      if (a.row.mx) {
        if (has) *(uint2*)(dst + lane * 8) = uint2{lo8, hi8};
        // the scales, and zeros in what fills them up to 16 bytes
        if (lane % 4 == 0 && a.row.scales + lane / 4 < a.row.rope_at)
          dst[a.row.scales + lane / 4] = (char)(has ? 127 + expo : 0);
      } else if (has) {
        *(bf8*)(dst + lane * 16) = yb;
      }
      if (pair) {
        __bf16* d = (__bf16*)(dst + a.row.rope_at);
        d[i0] = z0;
        d[i1] = z1;
      }
    };
    if (a.latent) {
      uint16_t* d = a.latent + t * (L + 2 * P);
      if (has) *(bf8*)(d + lane * 8) = yb;
      if (pair) {
        ((__bf16*)d)[L + i0] = z0;
        ((__bf16*)d)[L + i1] = z1;
      }
    }
    if (in_tail) {
      write_row(a.tail + ((size_t)r * a.T + ring) * a.row.bytes);
    } else {
      write_row(a.host + ((size_t)r * a.H + x) * a.row.bytes);
      const int s = a.page[(size_t)r * a.H + x];
      if (s >= 0 && s < a.B) write_row(a.hot + ((size_t)r * a.B + s) * a.row.bytes);
      if (lane == 0) atomicAdd(a.epoch + r, 1);  // a pending trial of this request is stale now
    }
  }
}

}  // namespace

hipError_t launch_map(const MapArgs& a, hipStream_t s) {
  const int blocks = a.n > 0 ? (int)(((int64_t)a.n + kMapTokens - 1) / kMapTokens) : 1;
  hipLaunchKernelGGL(map_kernel, dim3(blocks), dim3(kMapThreads), 0, s, a);
  return hipGetLastError();
}

hipError_t launch_store(const StoreArgs& a, hipStream_t s) {
  if (a.n <= 0) return hipSuccess;
  const int64_t need = ((int64_t)a.n + kStoreWaves - 1) / kStoreWaves;
  hipLaunchKernelGGL(store_kernel, dim3((int)(need < 8192 ? need : 8192)), dim3(kStoreThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace hs
