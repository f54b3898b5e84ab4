// One decode step's latent attention over the selected rows (gfx950), absorbed form: every head's key is the row, its
// value the row's latent part.
//
//   s = scale * q . row,   o = sum_j p_j latent_j / sum_j p_j,   p_j = 2^(s_j log2 e - m)   (m a running maximum)
//
// One pass over the rows, 32 to a tile. A workgroup of four waves takes a part of one request's selection and 32, 64 or
// 128 of its heads; it reads each row once, whatever the number of heads. Matrix instructions do both products
// transposed, so that a head is a lane's column in both and its maximum, sum and rescaling stay inside the lane:
//   S^T[key][head]  = K Q^T     A: the tile's rows from LDS, B: the queries, kept in registers
//   O^T[dim][head] += V^T P^T   A: the same rows read through the transposing LDS load, B: the weights as S^T left them
// (a lane half h holds the keys 8 i + 4 h + 0..3 of S^T; the second product takes its keys in that order, so the weights
// never change lanes). With w head groups of 32 the other 4 / w waves of a group share out the latent dimensions of the
// second product and each repeat the first.
#include "hs_latent.h"
#include "hs_mfma.h"

#include <climits>
#include <utility>

namespace hs {

namespace {

constexpr int kAttendThreads = 256;
constexpr int kTile = 32;          // rows of a tile
constexpr int kDepth = 4;          // tiles in LDS as memory has them: one in use, the others on their way
constexpr int kListed = 1024;      // rows of the selection whose indices are held in LDS at a time
constexpr int kGroupHeads = 128;   // most heads of one workgroup
__device__ __align__(16) uint4 zero_row[72];  // what a tile holds where there is no row

template <int L, int P, bool kMx>
struct Shape {
  static constexpr int D = L + P;
  static constexpr int kCols = (D + 63) / 64;              // groups of columns of a tile in bf16
  static constexpr int kColBytes = kTile * 128;
  static constexpr int kTileBytes = kCols * kColBytes;
  static constexpr int kSteps = D / 16;                    // of the first product
  // an 8-bit row as memory has it, in groups of 128 bytes and what is left of it (1 or 5 chunks)
  static constexpr int kScales = L, kRope = L + (L / kScaleBlock + 15) / 16 * 16, kRowBytes = kRope + 2 * P;
  static constexpr int kRawCols = kRowBytes / 128, kRawRest = kRowBytes / 16 % 8;
  static constexpr int kRawBytes = kTile * kRowBytes;
  static constexpr int kLoads = kMx ? kRawCols + 1 : kCols;  // of a lane, for a tile
  static constexpr int kAhead = kMx ? kDepth : kDepth - 1;   // tiles asked for before the one in use
  static constexpr uint32_t kLds = (kMx ? 2 * kTileBytes + kDepth * kRawBytes : kDepth * kTileBytes) + 4 * kListed;
  static_assert(!kMx || kRawRest > 0, "the rest is a load of its own");
};

// The loads of one lane for a tile: its chunk of every group of 128 bytes, `row` the address of that chunk in the first.
// bf16 rows of 32 rope values end inside a group: there `last` keeps to the row's end.
template <bool kHalf, int kGroupBytes, int... G>
__device__ __forceinline__ void load_groups(const char* row, const char* last, uint32_t lds,
                                            std::integer_sequence<int, G...>) {
  (load_to_lds<128 * G>(kHalf && G == (int)sizeof...(G) - 1 ? last : row, lds + G * kGroupBytes), ...);
}

struct Part { int r, split, h0, begin, end; };

__device__ __forceinline__ Part part_of(const AttendArgs& a) {
  Part p;
  int b = blockIdx.x;
  const int groups = (a.heads + kGroupHeads - 1) / kGroupHeads;
  p.split = b % a.splits;
  b /= a.splits;
  p.h0 = b % groups * kGroupHeads;
  p.r = b / groups;
  // parts in whole tiles, as even as they come
  const int tiles = (a.k + kTile - 1) / kTile;
  const int per = tiles / a.splits, more = tiles % a.splits;
  const int t0 = p.split * per + (p.split < more ? p.split : more);
  p.begin = t0 * kTile;
  p.end = (t0 + per + (p.split < more)) * kTile;
  if (p.end > a.k) p.end = a.k;
  return p;
}

// A raw tile of 8-bit rows to bf16: thread (row, c) takes 16 values of each 128, their scale's byte from the row, and the
// row's c-th chunk of rope values. Values times a power of two are exact in bf16.
template <int L, int P>
__device__ __forceinline__ void convert_tile(const char* raw, char* tile, int tid) {
  using S = Shape<L, P, true>;
  const int row = tid >> 3, c = tid & 7, f = swizzle(row);
  auto chunk = [&](int q) {  // of the row, which may lie in its rest
    return q < 8 * S::kRawCols ? raw + (q >> 3) * S::kColBytes + row * 128 + (q & 7) * 16
                               : raw + S::kRawCols * S::kColBytes + (row * S::kRawRest + q - 8 * S::kRawCols) * 16;
  };
  const v4u scales = *(const v4u*)chunk(S::kScales / 16);
#pragma unroll
  for (int j = 0; j < L / 128; ++j) {
    const v4u x = *(const v4u*)(raw + j * S::kColBytes + row * 128 + c * 16);
    const float scale = __uint_as_float(((scales[j] >> (8 * (c >> 1))) & 255u) << 23);
    v4u y[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      y[i / 2][i % 2 * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], scale, false));
      y[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x[i], scale, true));
    }
    // the two halves of a row's eight threads write to two groups of columns: in opposite order, to other banks
    char* to = tile + (2 * j + (c >> 2)) * S::kColBytes + row * 128;
    const int first = c >> 2;
    *(v4u*)(to + (((2 * (c & 3) + first) ^ f) << 4)) = first ? y[1] : y[0];
    *(v4u*)(to + (((2 * (c & 3) + 1 - first) ^ f) << 4)) = first ? y[0] : y[1];
  }
  if (c < P / 8) {
    *(v4u*)(tile + L / 64 * S::kColBytes + row * 128 + ((c ^ f) << 4)) = *(const v4u*)chunk(S::kRope / 16 + c);
  }
}

// kGroups: head groups of 32 (1, 2 or 4).
template <int L, int P, bool kMx, int kGroups>
__global__ __launch_bounds__(kAttendThreads, 1) void attend_kernel(AttendArgs a) {
  using S = Shape<L, P, kMx>;
  constexpr int kShare = 4 / kGroups;            // waves that share out a head group's dimensions
  constexpr int kBlocks = L / 32 / kShare;       // blocks of 32 dimensions of a wave
  static_assert(kBlocks % 2 == 0, "a wave's dimensions are whole groups of columns");
  extern __shared__ __align__(1024) char smem[];
  char* raw = smem + (kMx ? 2 * S::kTileBytes : 0);  // tiles as loaded (bf16: the tiles themselves)
  constexpr int kLoadBytes = kMx ? S::kRawBytes : S::kTileBytes;
  int* list = (int*)(raw + kDepth * kLoadBytes);     // row indices of the part, -1: none
  const uint32_t raw0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(HS_LDS char*)raw);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 31, half = lane >> 5;
  const Part part = part_of(a);
  const int head = part.h0 + (wave / kShare) * 32 + col;
  const int share = wave % kShare;
  const int rb = a.row.bytes;
  const int32_t* out = a.out + (size_t)part.r * a.k;
  // row i of the part's list: near + i * rb, or far + i * rb from index `edge` on
  const int edge = a.gather ? INT_MAX : a.B;
  const uintptr_t near = a.gather ? (uintptr_t)(a.gather + (size_t)part.r * a.k * rb)
                                  : (uintptr_t)(a.hot + (size_t)part.r * a.B * rb);
  const uintptr_t far = (uintptr_t)a.tail + ((size_t)part.r * a.T - (size_t)a.B) * rb;
  const uintptr_t none = (uintptr_t)zero_row;

  // the queries, one k-step of 16 values to a register quadruple
  bf8 q[S::kSteps];
  const uint32_t sign = a.scale < 0.0f ? kSigns : 0u;
  {
    const int h = head < a.heads ? head : a.heads - 1;  // columns behind the last head repeat it, and are dropped
    const __bf16* src = (const __bf16*)a.q + ((size_t)part.r * a.heads + h) * S::D + 8 * half;
#pragma unroll
    for (int s = 0; s < S::kSteps; ++s) q[s] = turned(*(const v4u*)(src + 16 * s), sign);
  }
  f16 o[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) o[b] = f16{};
  float m = -INFINITY, sum = 0.0f, rsum = 0.0f;  // rsum: of the weights as rounded for the second product
  const float scale = scale_of(a.scale);

  // LDS places of this lane's reads, but for the tile's start
  int kat[4], vat[2][2];
#pragma unroll
  for (int i = 0; i < 4; ++i) kat[i] = col * 128 + (((2 * i + half) ^ swizzle(col)) << 4);
#pragma unroll
  for (int i = 0; i < 4; ++i) vat[i / 2][i % 2] = across_place(lane, i / 2, 8 * (i % 2)) + S::kColBytes * (kBlocks / 2 * share);

  const int tiles = (part.end - part.begin + kTile - 1) / kTile;
  auto write_list = [&](int from) {  // of the rows [from, from + kListed) of the part
    for (int i = tid; i < kListed; i += kAttendThreads) {
      const int at = part.begin + from + i;
      int s = at < part.end ? out[at] : -1;
      s = s >= 0 && s < a.B + a.T ? (a.gather ? at : s) : -1;
      list[i] = s;
    }
  };
  // asks for tile t (behind the last one: whatever the list holds, so that every tile is the same number of loads) and says
  // which of its rows are there
  const int mine = 8 * wave + (lane >> 3), place = kMx ? lane & 7 : (lane & 7) ^ swizzle(mine);
  const int rest_mine = 8 * wave + lane / S::kRawRest, rest_place = lane % S::kRawRest;  // 8-bit rows: of the row's rest
  auto address = [&](int s) {
    const uintptr_t p = (s < edge ? near : far) + (uint64_t)(uint32_t)s * (uint32_t)rb;
    return (const char*)(s < 0 ? none : p);
  };
  auto load = [&](int t) {
    const int* rows = list + t * kTile % kListed;
    const uint32_t to = raw0 + (t & (kDepth - 1)) * kLoadBytes;
    const char* row = address(rows[mine]);
    if constexpr (kMx) {
      load_groups<false, S::kColBytes>(row + 16 * place, nullptr, to + 1024 * wave,
                                       std::make_integer_sequence<int, S::kRawCols>());
      const char* rest = address(rows[rest_mine & (kTile - 1)]) + 128 * S::kRawCols + 16 * rest_place;
      if (lane < 8 * S::kRawRest) load_to_lds<0>(rest, to + S::kRawCols * S::kColBytes + 128 * S::kRawRest * wave);
    } else {
      load_groups<S::D % 64 != 0, S::kColBytes>(row + 16 * place, row + 16 * (place & 3), to + 1024 * wave,
                                                std::make_integer_sequence<int, S::kCols>());
    }
    return (uint32_t)__ballot(rows[col] >= 0);
  };
  write_list(0);
  // the queries are here before any load to LDS is on its way: a wait for them later would be one for those too
#pragma unroll
  for (int s = 0; s < S::kSteps; ++s) asm volatile("" : "+v"(q[s]));
  __syncthreads();
  uint32_t there[S::kAhead + 1];  // of the tiles asked for, the one in use first
#pragma unroll
  for (int t = 0; t < S::kAhead; ++t) there[t] = load(t);
  if constexpr (kMx) {
    wait_loads_and_meet<S::kLoads * (kDepth - 1)>();
    convert_tile<L, P>(raw, smem, tid);
  }

  for (int t = 0; t < tiles; ++t) {
    wait_loads_and_meet<S::kLoads * (kDepth - 2)>();  // 8-bit rows: for tile t + 1
    if ((t + S::kAhead) * kTile % kListed == 0) {     // every wave has asked for all that the list named
      write_list((t + S::kAhead) * kTile);
      __syncthreads();
    }
    there[S::kAhead] = load(t + S::kAhead);  // into the place that every wave has left
    const char* tile = smem + (kMx ? t & 1 : t & (kDepth - 1)) * S::kTileBytes;
    if constexpr (kMx)
      convert_tile<L, P>(raw + ((t + 1) & (kDepth - 1)) * S::kRawBytes, smem + ((t + 1) & 1) * S::kTileBytes, tid);
    // S^T
    f16 s0{};
    constexpr int kSet = 4;  // k-steps whose rows are read before the steps before them are multiplied
    bf8 k[2][kSet];
#pragma unroll
    for (int i = 0; i < kSet; ++i) k[0][i] = *(const bf8*)(tile + kat[i]);
#pragma unroll
    for (int s = 0; s < S::kSteps; s += kSet) {
#pragma unroll
      for (int i = 0; i < kSet; ++i)
        if (s + kSet + i < S::kSteps)
          k[(s / kSet + 1) & 1][i] = *(const bf8*)(tile + kat[i] + S::kColBytes * ((s + kSet + i) >> 2));
#pragma unroll
      for (int i = 0; i < kSet; ++i)
        if (s + i < S::kSteps)
          s0 = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[(s / kSet) & 1][i], q[s + i], s0, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    // the values' first blocks are on their way during the softmax, the others two blocks ahead of their product
    constexpr int kReads = 3;
    bf8 v[kReads][2];
    auto read_values = [&](int b) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const char* at = tile + S::kColBytes * (b >> 1) + 2048 * j;
        v[b % kReads][j] = read_across(at + vat[b & 1][0], at + vat[b & 1][1]);
      }
    };
    read_values(0);
    read_values(1);
    if (there[0] != 0xffffffffu) {
      const uint32_t mask = there[0] >> (4 * half);
#pragma unroll
      for (int i = 0; i < 16; ++i) s0[i] = (mask >> (8 * (i / 4) + i % 4)) & 1 ? s0[i] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < S::kAhead; ++i) there[i] = there[i + 1];
    float top = s0[0];
#pragma unroll
    for (int i = 1; i < 16; ++i) top = fmaxf(top, s0[i]);
    top = max_of_halves(top) * scale;
    if (__any(top > m + kSlack)) {
      const float to = fmaxf(m, top);
      if (__any(m > -INFINITY)) {
        const float c = m == -INFINITY ? 0.0f : __builtin_amdgcn_exp2f(m - to);
        sum *= c;
        rsum *= c;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= c;
      }
      m = to;
    }
    const float m0 = m == -INFINITY ? 0.0f : m;
    bf8 p[2];
    weigh(s0, scale, m0, p, sum, rsum);
    __builtin_amdgcn_sched_barrier(0);
    // O^T
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (b + 2 < kBlocks) read_values(b + 2);
#pragma unroll
      for (int j = 0; j < 2; ++j) o[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v[b % kReads][j], p[j], o[b], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // the loads behind the last tile write to LDS too
  sum += __shfl_xor(sum, 32);
  rsum += __shfl_xor(rsum, 32);
  if (head >= a.heads) return;
  const size_t rh = (size_t)part.r * a.heads + head;
  if (a.splits == 1) {
    const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
    __bf16* dst = (__bf16*)a.o + rh * L + 32 * kBlocks * share + 4 * half;
#pragma unroll
    for (int b = 0; b < kBlocks; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        bf4 v;
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = (__bf16)(o[b][4 * i + j] * f);
        *(bf4*)(dst + 32 * b + 8 * i) = v;
      }
    if (a.lse && share == 0 && half == 0) a.lse[rh] = sum > 0.0f ? m * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
    return;
  }
  // partial results: [R][heads][splits] of (m, sum, rsum, -) and [R][heads][splits][L]
  const size_t ph = rh * a.splits + part.split;
  const size_t stats = (size_t)a.R * a.heads * a.splits * 4;
  if (share == 0 && half == 0) *(f4*)(a.work + ph * 4) = f4{m, sum, rsum, 0.0f};
  float* dst = a.work + stats + ph * L + 32 * kBlocks * share + 4 * half;
#pragma unroll
  for (int b = 0; b < kBlocks; ++b)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *(f4*)(dst + 32 * b + 8 * i) = f4{o[b][4 * i], o[b][4 * i + 1], o[b][4 * i + 2], o[b][4 * i + 3]};
}

// Joins the parts of one request and head, in their order: one wave per head, eight (four) dimensions a lane.
template <int L>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a) {
  constexpr int kPer = L / 64;
  const size_t rh = (size_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (rh >= (size_t)a.R * a.heads) return;
  const f4* st = (const f4*)a.work + rh * a.splits;
  float m = -INFINITY;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, st[s][0]);
  const float m0 = m == -INFINITY ? 0.0f : m;
  float sum = 0.0f, rsum = 0.0f, o[kPer] = {};
  const float* src = a.work + (size_t)a.R * a.heads * a.splits * 4 + rh * a.splits * L + lane * kPer;
  for (int s = 0; s < a.splits; ++s) {
    const f4 v = st[s];
    const float c = __builtin_amdgcn_exp2f(v[0] - m0);
    sum += c * v[1];
    rsum += c * v[2];
#pragma unroll
    for (int i = 0; i < kPer; i += 4) {
      const f4 x = *(const f4*)(src + (size_t)s * L + i);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[i + j] += c * x[j];
    }
  }
  const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
  __bf16* dst = (__bf16*)a.o + rh * L + lane * kPer;
#pragma unroll
  for (int i = 0; i < kPer; i += 4) {
    bf4 v;
#pragma unroll
    for (int j = 0; j < 4; ++j) v[j] = (__bf16)(o[i + j] * f);
    *(bf4*)(dst + i) = v;
  }
  if (a.lse && lane == 0) a.lse[rh] = sum > 0.0f ? m * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
}

template <int L, int P, bool kMx, int kGroups>
void launch(const AttendArgs& a, hipStream_t s) {
  constexpr uint32_t lds = Shape<L, P, kMx>::kLds;
  const int groups = (a.heads + kGroupHeads - 1) / kGroupHeads;
  hipLaunchKernelGGL((attend_kernel<L, P, kMx, kGroups>), dim3(a.R * groups * a.splits), dim3(kAttendThreads), lds, s, a);
}

template <int L, int P, bool kMx>
hipError_t launch_heads(const AttendArgs& a, hipStream_t s) {
  if (a.heads <= 32) launch<L, P, kMx, 1>(a, s);
  else if (a.heads <= 64) launch<L, P, kMx, 2>(a, s);
  else launch<L, P, kMx, 4>(a, s);
  if (a.splits > 1)
    hipLaunchKernelGGL(join_kernel<L>, dim3((int)(((size_t)a.R * a.heads + 3) / 4)), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int L, int P, bool kMx>
hipError_t set_lds() {
  for (const void* f : {(const void*)attend_kernel<L, P, kMx, 1>, (const void*)attend_kernel<L, P, kMx, 2>,
                        (const void*)attend_kernel<L, P, kMx, 4>}) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<L, P, kMx>::kLds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

int attend_splits(int R, int k, int heads, const RowLayout&) {
  const int groups = (heads + kGroupHeads - 1) / kGroupHeads;
  const int tiles = (k + kTile - 1) / kTile;
  int s = 256 / (R * groups);
  if (s < 1) s = 1;
  if (s > tiles) s = tiles;
  return s;
}

uint64_t attend_work_bytes(int R, int k, int heads, const RowLayout& row) {
  const uint64_t s = (uint64_t)attend_splits(R, k, heads, row);
  return s == 1 ? 0 : (uint64_t)R * heads * s * (16 + 4ull * row.latent);
}

hipError_t set_attend_lds() {
  for (const auto f : {set_lds<512, 64, false>, set_lds<512, 32, false>, set_lds<256, 64, false>, set_lds<256, 32, false>,
                       set_lds<512, 64, true>, set_lds<512, 32, true>, set_lds<256, 64, true>, set_lds<256, 32, true>}) {
    const hipError_t e = f();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

hipError_t launch_attend(const AttendArgs& a, hipStream_t s) {
  const bool wide = a.row.latent == 512, more = a.row.rope == 64;
  if (a.row.mx)
    return wide ? more ? launch_heads<512, 64, true>(a, s) : launch_heads<512, 32, true>(a, s)
                : more ? launch_heads<256, 64, true>(a, s) : launch_heads<256, 32, true>(a, s);
  return wide ? more ? launch_heads<512, 64, false>(a, s) : launch_heads<512, 32, false>(a, s)
              : more ? launch_heads<256, 64, false>(a, s) : launch_heads<256, 32, false>(a, s);
}

}  // namespace hs
