// One decode step's latent attention over the selected rows (gfx950), absorbed form: every head's key is the row, its
// value the row's latent part.
//
//   s = scale * q . row,   o = sum_j p_j latent_j / sum_j p_j,   p_j = 2^(s_j log2 e - m)   (m a running maximum)
//
// One pass over the rows, 32 to a tile. A workgroup of eight waves, two to a SIMD, takes a part of one request's selection
// and up to 128 of its heads, for all of which it reads a row once. Matrix instructions do both products transposed, so that a
// head is a lane's column in both and its maximum, sum and rescaling stay inside four lanes:
//   S^T[key][head]  = K Q^T     A: the tile's rows from LDS, B: the queries, kept in registers
//   O^T[dim][head] += V^T P^T   A: the same rows read through the transposing LDS load, B: the weights as S^T left them
// (lane group g = lane / 16 holds the keys 4 g + 0..3 and 16 + 4 g + 0..3 of S^T; the second product takes its keys in that
// order, so the weights never change lanes). With fewer than eight groups of 16 heads a group has more than one wave: half
// of them take the first 16 keys of each tile, half the others (joined through LDS at the end), and the waves of a half share
// out the latent dimensions of the second product and repeat the first. LDS reads bound it there: with all 32 keys to each
// wave 256 requests x 2048 rows took 130 us for 16 heads and 146 for 64, with halves they take 111 and 124 (604 MB of rows at
// 5.4 and 4.9 TB/s, what memory gives). With 128 heads 170 to 177 us by the card (3.5 TB/s of rows, 850 TFLOP/s): a tile's
// loads alone take 130, and the two products' dependence and the waves' meeting at each tile keep them from hiding all of the
// rest. 8-bit rows are converted to bf16 tiles, so their products cost the same, and a tile passes LDS four times (in, out to be
// converted, in, out to the products): of the bytes that they spare almost nothing shows, 102, 111, 130 and 181 us for 16, 32,
// 64 and 128 heads where bf16 rows take 111, 115, 124 and 171.
#include "hs_latent.h"
#include "hs_mfma.h"

#include <climits>
#include <type_traits>
#include <utility>

namespace hs {

namespace {

constexpr int kAttendThreads = 512;
constexpr int kWavesA = kAttendThreads / 64;
constexpr int kTile = 32;          // rows of a tile
constexpr int kDepth = 4;          // tiles in LDS as memory has them: one in use, the others on their way
constexpr int kListed = 1024;      // rows of the selection whose indices are held in LDS at a time
constexpr int kMostSplits = 64;    // parts of a selection: one to a lane of the wave that joins them
__device__ __align__(16) uint4 zero_row[72];  // what a tile holds where there is no row

// A tile's chunks change places by the row (see hs_mfma.h). LDS answers a 16-byte read in four steps, the first for the lanes
// 0-3, 12-15, 20-23 and 24-27: rows 0-3 and 12-15 at one chunk and rows 4-11 at its neighbour. Those, and 8 rows at two
// neighbouring chunks, meet no bank twice (256 requests x 2048 rows x 128 heads: 185 us with an order that is free of
// conflicts only where all 16 rows are read at one chunk, 172 us with this).
__device__ __forceinline__ int swizzle16(int row) { return (((row >> 1) & 3) << 1) ^ (((row >> 3) & 1) * 5); }

template <int L, int P, bool kMx>
struct Shape {
  static constexpr int D = L + P;
  static constexpr int kCols = (D + 63) / 64;              // groups of columns of a tile in bf16
  static constexpr int kColBytes = kTile * 128;
  static constexpr int kTileBytes = kCols * kColBytes;
  static constexpr int kSteps = D / 32;                    // of the first product
  // an 8-bit row as memory has it, in groups of 128 bytes and what is left of it (1 or 5 chunks)
  static constexpr int kScales = L, kRope = L + (L / kScaleBlock + 15) / 16 * 16, kRowBytes = kRope + 2 * P;
  static constexpr int kRawCols = kRowBytes / 128, kRawRest = kRowBytes / 16 % 8;
  static constexpr int kRawBytes = kTile * kRowBytes;
  // loads of a lane for a tile: the first four waves take its even groups, the others the odd ones and the rest
  static constexpr int kEven = ((kMx ? kRawCols : kCols) + 1) / 2;
  static constexpr int kOdd = (kMx ? kRawCols : kCols) / 2 + (kMx ? 1 : 0);
  static constexpr int kAhead = kMx ? kDepth : kDepth - 1;   // tiles asked for before the one in use
  static constexpr int kLoadBytes = kMx ? kRawBytes : kTileBytes;
  static constexpr uint32_t kLds = (kMx ? 2 * kTileBytes : 0) + kDepth * kLoadBytes + 4 * kListed;
  static_assert(!kMx || kRawRest > 0, "the rest is a load of its own");
  static_assert((kMx ? 2 * kTileBytes : 0) + kDepth * kLoadBytes >= 4 * kTileBytes, "room for the queries of 128 heads");
};

// The loads of one lane for every second group of 128 bytes of a tile from kFirst on: its chunk of each, `row` the address
// of that chunk in the first group. Rows of 32 rope values in bf16 end inside a group: there `last` keeps to the row's end.
template <int kFirst, int kCols, bool kHalf, int kGroupBytes, int... G>
__device__ __forceinline__ void load_groups(const char* row, const char* last, uint32_t lds,
                                            std::integer_sequence<int, G...>) {
  (load_to_lds<128 * (2 * G + kFirst)>(kHalf && 2 * G + kFirst == kCols - 1 ? last : row,
                                       lds + (2 * G + kFirst) * kGroupBytes),
   ...);
}

template <int kCols, bool kHalf, int kGroupBytes>
__device__ __forceinline__ void load_half(bool odd, const char* row, const char* last, uint32_t lds) {
  if (odd)
    load_groups<1, kCols, kHalf, kGroupBytes>(row, last, lds, std::make_integer_sequence<int, kCols / 2>());
  else
    load_groups<0, kCols, kHalf, kGroupBytes>(row, last, lds, std::make_integer_sequence<int, (kCols + 1) / 2>());
}

// All but the last `later` tiles asked for (at most kMost) are in LDS, for every wave.
template <int kMost, class S>
__device__ __forceinline__ void wait_tiles(bool odd, int later) {
  if constexpr (kMost > 0) {
    if (later < kMost) return wait_tiles<kMost - 1, S>(odd, later);
  }
  if (odd) wait_loads_and_meet<S::kOdd * kMost>();
  else wait_loads_and_meet<S::kEven * kMost>();
}

struct Part { int r, split, h0, begin, end; };

// kGroupHeads: heads of a workgroup
template <int kGroupHeads>
__device__ __forceinline__ Part part_of(const AttendArgs& a) {
  Part p;
  const int groups = (a.heads + kGroupHeads - 1) / kGroupHeads;
  // Workgroups go round the eight chiplets in turn. The parts of one request and its queries stay on one, whose cache then
  // gets the queries once: of every eight requests (and head groups) one to a chiplet, those behind the last eight as they come.
  int b = blockIdx.x, u;
  const int whole = a.R * groups / 8 * 8;
  if (b < whole * a.splits) {
    p.split = b / 8 % a.splits;
    u = b / 8 / a.splits * 8 + b % 8;
  } else {
    b -= whole * a.splits;
    p.split = b % a.splits;
    u = whole + b / a.splits;
  }
  p.h0 = u % groups * kGroupHeads;
  p.r = u / groups;
  // parts in whole tiles, as even as they come
  const int tiles = (a.k + kTile - 1) / kTile;
  const int per = tiles / a.splits, more = tiles % a.splits;
  const int t0 = p.split * per + (p.split < more ? p.split : more);
  p.begin = t0 * kTile;
  p.end = (t0 + per + (p.split < more)) * kTile;
  if (p.end > a.k) p.end = a.k;
  return p;
}

// A raw tile of 8-bit rows to bf16: thread (row, c) takes 16 values of each 256, their scale's byte from the row, and the
// row's c-th chunk of rope values. Values times a power of two are exact in bf16 (scale bytes 10 to 246).
template <int L, int P>
struct Converter {
  using S = Shape<L, P, true>;
  v4u values[L / 256], rope;
  uint32_t scales[L / 256];

  static constexpr int kParts = L / 256 + 1;  // of the values, and the rope part's

  __device__ __forceinline__ void read(int part, const char* raw, int tid) {
    const int row = tid >> 4, c = tid & 15;
    auto chunk = [&](int q) {  // of the row, which may lie in its rest
      return q < 8 * S::kRawCols ? raw + (q >> 3) * S::kColBytes + row * 128 + (q & 7) * 16
                                 : raw + S::kRawCols * S::kColBytes + (row * S::kRawRest + q - 8 * S::kRawCols) * 16;
    };
    if (part == kParts - 1) {
      rope = *(const v4u*)chunk(S::kRope / 16 + (c & (P / 8 - 1)));
      return;
    }
    values[part] = *(const v4u*)chunk(16 * part + c);
    scales[part] = ((const uint32_t*)chunk(S::kScales / 16))[2 * part + (c >> 3)];
  }

  __device__ __forceinline__ void write(int part, char* tile, int tid) const {
    const int row = tid >> 4, c = tid & 15, f = swizzle16(row);
    if (part == kParts - 1) {
      if (c < P / 8) *(v4u*)(tile + L / 64 * S::kColBytes + row * 128 + ((c ^ f) << 4)) = rope;
      return;
    }
    const float scale = __uint_as_float(((scales[part] >> (8 * ((c >> 1) & 3))) & 255u) << 23);
    v4u y[2];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = values[part][i];
      y[i / 2][i % 2 * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, false));
      y[i / 2][i % 2 * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(x, scale, true));
    }
    // neighbouring groups of columns in opposite order, to other banks
    char* to = tile + (4 * part + (c >> 2)) * S::kColBytes + row * 128;
    const int first = (c >> 2) & 1;
    *(v4u*)(to + (((2 * (c & 3) + first) ^ f) << 4)) = first ? y[1] : y[0];
    *(v4u*)(to + (((2 * (c & 3) + 1 - first) ^ f) << 4)) = first ? y[0] : y[1];
  }

  __device__ __forceinline__ void read(const char* raw, int tid) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) read(i, raw, tid);
  }
  __device__ __forceinline__ void write(char* tile, int tid) const {
#pragma unroll
    for (int i = 0; i < kParts; ++i) write(i, tile, tid);
  }
};
template <>
struct Converter<0, 0> {
  static constexpr int kParts = 0;
  __device__ __forceinline__ void read(int, const char*, int) {}
  __device__ __forceinline__ void write(int, char*, int) const {}
  __device__ __forceinline__ void read(const char*, int) {}
  __device__ __forceinline__ void write(char*, int) const {}
};

// kGroups: head groups of 16 (1, 2, 4 or 8).
template <int L, int P, bool kMx, int kGroups>
__global__ __launch_bounds__(kAttendThreads) void attend_kernel(AttendArgs a) {
  using S = Shape<L, P, kMx>;
  constexpr int kShare = kWavesA / kGroups;      // waves of a head group
  constexpr int kHalves = kGroups <= 4 ? 2 : 1;  // parts of a tile's keys; the waves of one share out the dimensions
  constexpr int kKeyBlocks = 2 / kHalves;        // blocks of 16 keys of a wave
  constexpr int kBlocks = L / 16 / (kShare / kHalves);  // blocks of 16 dimensions of a wave
  // 8-bit rows and many heads: converted when the first product has left its registers (256 requests x 2048 rows x 128 heads
  // 331 -> 185 us)
  constexpr bool kLate = kMx && kGroups >= 4 && L == 512;
  constexpr int kQueryTiles = (kGroups + 1) / 2; // the queries, as tiles of 32 heads
  extern __shared__ __align__(1024) char smem[];
  char* raw = smem + (kMx ? 2 * S::kTileBytes : 0);  // tiles as loaded (bf16: the tiles themselves)
  int* list = (int*)(raw + kDepth * S::kLoadBytes);  // row indices of the part, -1: none
  const uint32_t smem0 = __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(HS_LDS char*)smem);
  const uint32_t raw0 = smem0 + (uint32_t)(raw - smem);
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, group = lane >> 4;
  const Part part = part_of<16 * kGroups>(a);
  const int head = part.h0 + (wave / kShare) * 16 + col;
  const int share = wave % kShare / kHalves, key_half = wave % kHalves;
  const int rb = a.row.bytes;
  const int32_t* out = a.out + (size_t)part.r * a.k;
  // row i of the part's list: near + i * rb, or far + i * rb from index `edge` on
  const int edge = a.gather ? INT_MAX : a.B;
  const uintptr_t near = a.gather ? (uintptr_t)(a.gather + (size_t)part.r * a.k * rb)
                                  : (uintptr_t)(a.hot + (size_t)part.r * a.B * rb);
  const uintptr_t far = (uintptr_t)a.tail + ((size_t)part.r * a.T - (size_t)a.B) * rb;
  const uintptr_t none = (uintptr_t)zero_row;

  const int tiles = (part.end - part.begin + kTile - 1) / kTile;
  constexpr int kPer = kListed / kAttendThreads;
  auto read_list = [&](int from, int (&s)[kPer]) {  // indices of the rows from `from` on, of the part
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = part.begin + from + i * kAttendThreads + tid;
      s[i] = out[at < part.end ? at : part.end - 1];
    }
  };
  auto write_list = [&](int from, const int (&s)[kPer]) {
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
      const int at = part.begin + from + i * kAttendThreads + tid;
      const bool there = at < part.end && s[i] >= 0 && s[i] < a.B + a.T;
      list[i * kAttendThreads + tid] = there ? (a.gather ? at : s[i]) : -1;
    }
  };
  // asks for tile t and says which of its rows are there
  const bool odd = wave >= kWavesA / 2;
  const int mine = 8 * (wave & 3) + (lane >> 3), place = (lane & 7) ^ swizzle16(mine);
  const int rest_mine = (8 * (wave & 3) + lane / S::kRawRest) & (kTile - 1), rest_place = lane % S::kRawRest;
  auto address = [&](int s) {
    const uintptr_t p = (s < edge ? near : far) + (uint64_t)(uint32_t)s * (uint32_t)rb;
    return (const char*)(s < 0 ? none : p);
  };
  struct Rows { int mine, rest, lane; };  // indices of the rows that this lane loads of a tile, and of row lane % 32
  auto rows_of = [&](int t) {
    const int* rows = list + t * kTile % kListed;
    return Rows{rows[mine], kMx ? rows[rest_mine] : 0, rows[lane & (kTile - 1)]};
  };
  auto load = [&](int t, Rows r) {
    const uint32_t to = raw0 + (t & (kDepth - 1)) * S::kLoadBytes;
    const char* row = address(r.mine);
    if constexpr (kMx) {
      load_half<S::kRawCols, false, S::kColBytes>(odd, row + 16 * (lane & 7), nullptr, to + 1024 * (wave & 3));
      if (odd) {
        const char* rest = address(r.rest) + 128 * S::kRawCols + 16 * rest_place;
        if (lane < 8 * S::kRawRest)
          load_to_lds<0>(rest, to + S::kRawCols * S::kColBytes + 128 * S::kRawRest * (wave & 3));
      }
    } else {
      load_half<S::kCols, S::D % 64 != 0, S::kColBytes>(odd, row + 16 * place, row + 16 * (place & 3),
                                                        to + 1024 * (wave & 3));
    }
    return (uint32_t)__ballot(r.lane >= 0);
  };

  // LDS places of this lane's reads, but for the tile's start
  int kat[2], vat[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) kat[i] = col * 128 + (((4 * i + group) ^ swizzle16(col)) << 4);
  {
    const int row = 4 * group + (col >> 2), x = (lane >> 1) & 1;
#pragma unroll
    for (int i = 0; i < 4; ++i) vat[i] = row * 128 + (((2 * i + x) ^ swizzle16(row)) << 4) + 8 * (lane & 1);
  }

  // The queries go through LDS as tiles of 32 heads (their rows are read whole, and once), in the places of the last tiles;
  // the list of rows is on its way at the same time, and so are then the tiles whose places the queries leave.
  constexpr int kQueryAt = kMx ? 0 : kDepth - kQueryTiles;  // tile place
  constexpr int kEarly = kMx ? (kQueryTiles <= 2 ? S::kAhead : 0) : (kQueryAt < S::kAhead ? kQueryAt : S::kAhead);
  uint32_t there[S::kAhead + 1] = {};  // of the tiles asked for, the one in use first
  bf8 q[S::kSteps];
  {
    int s[kPer];
    read_list(0, s);
#pragma unroll
    for (int i = 0; i < kQueryTiles; ++i) {
      const int h = part.h0 + 32 * i + mine;  // heads behind the last one repeat it, and are dropped
      const char* row = (const char*)a.q + ((size_t)part.r * a.heads + (h < a.heads ? h : a.heads - 1)) * (2 * S::D);
      load_half<S::kCols, S::D % 64 != 0, S::kColBytes>(odd, row + 16 * place, row + 16 * (place & 3),
                                                        smem0 + (kQueryAt + i) * S::kTileBytes + 1024 * (wave & 3));
    }
    write_list(0, s);
    wait_loads_and_meet<0>();
#pragma unroll
    for (int t = 0; t < kEarly; ++t)
      if (t < tiles) there[t] = load(t, rows_of(t));
    const char* tile = smem + (kQueryAt + wave / kShare / 2) * S::kTileBytes + wave / kShare % 2 * 2048;
    const uint32_t sign = a.scale < 0.0f ? kSigns : 0u;
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i)
      q[i] = turned(*(const v4u*)(tile + kat[i & 1] + S::kColBytes * (i >> 1)), sign);
    if (a.scale == 0.0f) zero_scaled(q);
#pragma unroll
    for (int i = 0; i < S::kSteps; ++i) asm volatile("" : "+v"(q[i]));  // read, before others write there
    asm volatile("s_barrier" ::: "memory");
#pragma unroll
    for (int t = kEarly; t < S::kAhead; ++t)
      if (t < tiles) there[t] = load(t, rows_of(t));
  }
  f4 o[kBlocks];
#pragma unroll
  for (int b = 0; b < kBlocks; ++b) o[b] = f4{};
  float m = -INFINITY, sum = 0.0f, rsum = 0.0f;  // rsum: of the weights as rounded for the second product
  const float scale = scale_of(a.scale);
  Converter<kMx ? L : 0, kMx ? P : 0> convert;
  Rows next = rows_of(S::kAhead);
  if constexpr (kMx) {
    wait_tiles<kDepth - 1, S>(odd, tiles - 1);
    convert.read(raw, tid);
    convert.write(smem, tid);
  }

  for (int t = 0; t < tiles; ++t) {
    wait_tiles<kDepth - 2, S>(odd, tiles - 1 - t - (kMx ? 1 : 0));  // (8-bit rows: for tile t + 1)
    const char* tile = smem + (kMx ? t & 1 : t & (kDepth - 1)) * S::kTileBytes;
    const char* keys = tile + 2048 * key_half;
    f4 s[kKeyBlocks] = {};
    constexpr int kSet = kGroups == 8 ? 2 : 4;  // k-steps whose rows are read before the steps before them are multiplied
    bf8 k[2][kSet][kKeyBlocks];
    auto read_keys = [&](int from) {
#pragma unroll
      for (int i = 0; i < kSet; ++i)
#pragma unroll
        for (int b = 0; b < kKeyBlocks; ++b)
          if (from + i < S::kSteps)
            k[from / kSet & 1][i][b] = *(const bf8*)(keys + kat[(from + i) & 1] + S::kColBytes * ((from + i) / 2) + 2048 * b);
    };
    read_keys(0);
    if (t + S::kAhead < tiles) there[S::kAhead] = load(t + S::kAhead, next);  // into the place that every wave has left
    if ((t + S::kAhead + 1) * kTile % kListed == 0 && t + S::kAhead + 1 < tiles) {  // every wave has read all that the list named
      int more[kPer];
      read_list((t + S::kAhead + 1) * kTile, more);
      write_list((t + S::kAhead + 1) * kTile, more);
      __syncthreads();
    }
    next = rows_of(t + S::kAhead + 1);
    const char* converted = raw + ((t + 1) & (kDepth - 1)) * S::kLoadBytes;
    if constexpr (!kLate) convert.read(converted, tid);
    // S^T of 32 keys, 16 to a block
#pragma unroll
    for (int j = 0; j < S::kSteps; ++j) {
      if (j % kSet == 0) read_keys(j + kSet);
#pragma unroll
      for (int b = 0; b < kKeyBlocks; ++b)
        s[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[j / kSet & 1][j % kSet][b], q[j], s[b], 0, 0, 0);
      if (j % kSet == kSet - 1) __builtin_amdgcn_sched_barrier(0);
    }
    // the values' first blocks are on their way during the softmax, the others some blocks ahead of their product
    constexpr int kReads = kGroups == 8 ? 4 : 6;
    std::conditional_t<kHalves == 2, s4, bf8> v[kReads];
    auto read_values = [&](int b) {
      const int d = kBlocks * share + b;  // block of the row; vat is for its place in a group of columns
      const char* at = keys + S::kColBytes * (d >> 2) + (kBlocks % 4 == 0 ? vat[b & 3] : vat[d & 3]);
      if constexpr (kHalves == 2) v[b % kReads] = read_across(at);
      else v[b % kReads] = read_across(at, at + 2048);
    };
    if (kLate && t + 1 < tiles) {
      int at = tid;
      asm volatile("" : "+v"(at));  // places are worked out here, and parts one by one: registers are short
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < convert.kParts; ++i) {
        convert.read(i, converted, at);
        convert.write(i, smem + ((t + 1) & 1) * S::kTileBytes, at);
        __builtin_amdgcn_sched_barrier(0);
      }
    }
#pragma unroll
    for (int b = 0; b < kReads - 1; ++b)
      if (b < kBlocks) read_values(b);
    if constexpr (!kLate) convert.write(smem + ((t + 1) & 1) * S::kTileBytes, tid);
    if (there[0] != 0xffffffffu) {
      const uint32_t mask = there[0] >> (4 * group + 16 * key_half);
#pragma unroll
      for (int i = 0; i < 4 * kKeyBlocks; ++i) s[i / 4][i % 4] = (mask >> (16 * (i / 4) + i % 4)) & 1 ? s[i / 4][i % 4] : -INFINITY;
    }
#pragma unroll
    for (int i = 0; i < S::kAhead; ++i) there[i] = there[i + 1];
    float top = s[0][0];
#pragma unroll
    for (int i = 1; i < 4 * kKeyBlocks; ++i) top = fmaxf(top, s[i / 4][i % 4]);
    top = max_of_quarters(top);
    if (__any((top - m) * scale > kSlack)) {
      const float to = fmaxf(m, top);
      if (__any(m > -INFINITY)) {
        const float c = rebase(m, to, scale);
        sum *= c;
        rsum *= c;
#pragma unroll
        for (int b = 0; b < kBlocks; ++b) o[b] *= c;
      }
      m = to;
    }
    float m0 = m == -INFINITY ? 0.0f : m * scale;
    if (__any(fabsf(m0) >= kFar)) {
      const bool apart = fabsf(m0) >= kFar;
#pragma unroll
      for (int i = 0; i < 4 * kKeyBlocks; ++i) s[i / 4][i % 4] -= apart ? m : 0.0f;
      m0 = apart ? 0.0f : m0;
    }
    bf8 p;
#pragma unroll
    for (int i = 0; i < 4 * kKeyBlocks; i += 2) weigh_pair(s[i / 4][i % 4], s[i / 4][i % 4 + 1], scale, m0, p, i, sum, rsum);
    __builtin_amdgcn_sched_barrier(0);
    // O^T
#pragma unroll
    for (int b = 0; b < kBlocks; ++b) {
      if (b + kReads - 1 < kBlocks) read_values(b + kReads - 1);
      if constexpr (kHalves == 2)
        o[b] = __builtin_amdgcn_mfma_f32_16x16x16bf16_1k(v[b % kReads], __builtin_bit_cast(s8, p).lo, o[b], 0, 0, 0);
      else
        o[b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v[b % kReads], p, o[b], 0, 0, 0);
      if (b % 2 == 1) __builtin_amdgcn_sched_barrier(0);
    }
  }
  wait_loads_and_meet<0>();  // every wave has left the tiles, and what it wrote there
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  rsum += __shfl_xor(rsum, 16);
  rsum += __shfl_xor(rsum, 32);
  constexpr int kOut = kBlocks / kHalves;  // blocks that the wave writes
  f4 out_o[kOut];
  if constexpr (kHalves == 2) {
    // two waves have the same dimensions of both halves of the keys: each joins one half of the blocks, through LDS
    constexpr int kStep = kAttendThreads;
    static_assert((3 + 4 * kOut) * kStep * 4 <= (int)S::kLds);
    float* const given = (float*)smem + wave * 64 + lane;
    const float* const theirs = (const float*)smem + (wave ^ 1) * 64 + lane;
    given[0] = m;
    given[kStep] = sum;
    given[2 * kStep] = rsum;
#pragma unroll
    for (int b = 0; b < kOut; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        out_o[b][j] = key_half ? o[kOut + b][j] : o[b][j];
        given[(3 + 4 * b + j) * kStep] = key_half ? o[b][j] : o[kOut + b][j];
      }
    __syncthreads();
    const float other = theirs[0], to = fmaxf(m, other), c0 = rebase(m, to, scale), c1 = rebase(other, to, scale);
    m = to;
    sum = sum * c0 + theirs[kStep] * c1;
    rsum = rsum * c0 + theirs[2 * kStep] * c1;
#pragma unroll
    for (int b = 0; b < kOut; ++b)
#pragma unroll
      for (int j = 0; j < 4; ++j) out_o[b][j] = out_o[b][j] * c0 + theirs[(3 + 4 * b + j) * kStep] * c1;
  } else {
#pragma unroll
    for (int b = 0; b < kOut; ++b) out_o[b] = o[b];
  }
  if (head >= a.heads) return;
  const size_t rh = (size_t)part.r * a.heads + head;
  const int first = 16 * kOut * (share * kHalves + key_half) + 4 * group;  // of the lane's dimensions: 4 of every 16
  if (a.splits == 1) {
    const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
    __bf16* dst = (__bf16*)a.o + rh * L + first;
#pragma unroll
    for (int b = 0; b < kOut; ++b) {
      bf4 v;
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j] = (__bf16)(out_o[b][j] * f);
      *(bf4*)(dst + 16 * b) = v;
    }
    if (a.lse && wave % kShare == 0 && group == 0)
      a.lse[rh] = sum > 0.0f ? m * scale * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
    return;
  }
  // partial results: [R][heads][splits] of (m, sum, rsum, -) and [R][heads][splits][L]
  const size_t ph = rh * a.splits + part.split;
  const size_t stats = (size_t)a.R * a.heads * a.splits * 4;
  if (wave % kShare == 0 && group == 0) *(f4*)(a.work + ph * 4) = f4{m, sum, rsum, 0.0f};
  float* dst = a.work + stats + ph * L + first;
#pragma unroll
  for (int b = 0; b < kOut; ++b) *(f4*)(dst + 16 * b) = out_o[b];
}

// Joins the parts of one request and head: a workgroup of four waves takes both, each wave every fourth part (all of a wave's
// parts on their way at once), and the waves' sums are added in their order. 32 requests x 16 heads x 8 parts, 8 MB, take
// 4.0 us, 64 x 64 x 4 parts, 34 MB, 8.4.
template <int L>
__global__ __launch_bounds__(256) void join_kernel(AttendArgs a) {
  constexpr int kPer = L / 64, kOnWay = 4;
  __shared__ f4 sums[4][L / 4];
  const size_t rh = blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, splits = a.splits;
  // every lane has one part's figures (there are at most 64 parts)
  f4 v = {-INFINITY, 0.0f, 0.0f, 0.0f};
  if (lane < splits) v = ((const f4*)a.work)[rh * splits + lane];
  const float* src = a.work + (size_t)a.R * a.heads * splits * 4 + rh * splits * L + lane * 4;
  f4 x[kOnWay][kPer / 4], o[kPer / 4] = {};
  auto read = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kOnWay; ++i) {
      const int s = s0 + 4 * i;
#pragma unroll
      for (int j = 0; j < kPer / 4; ++j) x[i][j] = *(const f4*)(src + (size_t)(s < splits ? s : 0) * L + 256 * j);
    }
  };
  read(wave);
  float m = max_of_quarters(v[0]);
#pragma unroll
  for (int d = 1; d < 16; d <<= 1) m = fmaxf(m, __shfl_xor(m, d));
  const float scale = scale_of(a.scale), c = rebase(v[0], m, scale);
  float sum = c * v[1], rsum = c * v[2];
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    sum += __shfl_xor(sum, d);
    rsum += __shfl_xor(rsum, d);
  }
  for (int s0 = wave; s0 < splits; s0 += 4 * kOnWay) {
    if (s0 != wave) read(s0);
#pragma unroll
    for (int i = 0; i < kOnWay; ++i) {
      const int s = s0 + 4 * i;
      const float w = __shfl(c, s < splits ? s : 0);
      if (s < splits)
#pragma unroll
        for (int j = 0; j < kPer / 4; ++j) o[j] += w * x[i][j];
    }
  }
#pragma unroll
  for (int j = 0; j < kPer / 4; ++j) sums[wave][lane + 64 * j] = o[j];
  __syncthreads();
  const int d = threadIdx.x;
  if (d < L / 4) {
    const f4 all = ((sums[0][d] + sums[1][d]) + sums[2][d]) + sums[3][d];
    const float f = rsum > 0.0f ? 1.0f / rsum : rsum == 0.0f ? 0.0f : rsum;
    bf4 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) r[i] = (__bf16)(all[i] * f);
    *(bf4*)((__bf16*)a.o + rh * L + 4 * d) = r;
  }
  if (a.lse && threadIdx.x == 0) a.lse[rh] = sum > 0.0f ? m * scale * kLn2 + logf(sum) : sum == 0.0f ? -INFINITY : sum;
}

template <int L, int P, bool kMx, int kGroups>
void launch(const AttendArgs& a, hipStream_t s) {
  constexpr uint32_t lds = Shape<L, P, kMx>::kLds;
  const int groups = (a.heads + 16 * kGroups - 1) / (16 * kGroups);
  hipLaunchKernelGGL((attend_kernel<L, P, kMx, kGroups>), dim3(a.R * groups * a.splits), dim3(kAttendThreads), lds, s, a);
}

template <int L, int P, bool kMx>
hipError_t launch_heads(const AttendArgs& a, hipStream_t s) {
  if (a.groups == 1) launch<L, P, kMx, 1>(a, s);
  else if (a.groups == 2) launch<L, P, kMx, 2>(a, s);
  else if (a.groups == 4) launch<L, P, kMx, 4>(a, s);
  else launch<L, P, kMx, 8>(a, s);
  if (a.splits > 1)
    hipLaunchKernelGGL(join_kernel<L>, dim3(a.R * a.heads), dim3(256), 0, s, a);
  return hipGetLastError();
}

template <int L, int P, bool kMx>
hipError_t set_lds() {
  for (const void* f : {(const void*)attend_kernel<L, P, kMx, 1>, (const void*)attend_kernel<L, P, kMx, 2>,
                        (const void*)attend_kernel<L, P, kMx, 4>, (const void*)attend_kernel<L, P, kMx, 8>}) {
    const hipError_t e = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, (int)Shape<L, P, kMx>::kLds);
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace

// Heads of a workgroup and parts of each selection: those for which a model of the call's time, in tenths of a microsecond, is
// least. A workgroup takes 5.5 to 9 us to begin and end and 1.7 to 2.7 a tile, by its heads, when all 256 compute units
// stream rows; the join takes 4 us, some more by the parts, and the time that the partial results take to memory and back
// (at 5 TB/s). Measured, in us: 64 requests x 2048 rows x 64 heads (8 bits) in 3, 4, 6, 8 parts 59, 53 (modelled), 73, 69; 32 x
// 2048 x 16 in 6, 8, 12 parts 23, 23 (modelled), 30. Few requests with many heads take fewer heads to a workgroup, which read
// the same rows (from the caches): 128, 64, 32, 16 heads to one: 1 x 2048 x 128 heads 24.8, 20.9, 17.5, 16.0; 4 x 2048 x 128
// 29, 26, 22, 24; 256 x 64 x 128 24, 33, 41, 59.
AttendPlan attend_plan(int R, int k, int heads, const RowLayout& row) {
  const int tiles = (k + kTile - 1) / kTile;
  AttendPlan best{1, 1};
  int64_t least = INT64_MAX;
  for (int g = 8; g >= 1; g /= 2) {
    if (g > 1 && heads <= 8 * g) continue;  // half as many would do
    const int64_t units = (int64_t)R * ((heads + 16 * g - 1) / (16 * g));
    const int tile = g == 8 ? 27 : g == 4 ? 20 : g == 2 ? 18 : 17, start = g == 8 ? 90 : g == 4 ? 70 : g == 2 ? 60 : 55;
    for (int s = 1; s <= tiles && s <= kMostSplits; ++s) {
      const int64_t rounds = (units * s + 255) / 256, per = (tiles + s - 1) / s;
      int64_t t = rounds * (per * tile + start);
      if (s > 1) t += 40 + 4 * s / 5 + (int64_t)R * heads * s * row.latent * 8 / 500000;
      if (t < least) {
        least = t;
        best = AttendPlan{g, s};
      }
    }
  }
  return best;
}

uint64_t attend_work_bytes(const AttendPlan& plan, int R, int heads, const RowLayout& row) {
  const uint64_t s = (uint64_t)plan.splits;
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
