// The experts' products in 8-bit integers on the expand layout for gfx950:
// y[r, n] = x_scales[r] * w_scales[e, n] * sum over k of x[r, k] w[e, n, k].
//
// Mathematics. Sums of products of two 8-bit integers are exact in the matrix cores' 32-bit
// accumulators (32x32x32 and 16x16x64), in any order, and are scaled once at the end.
//
// Experts with more than 32 rows: 256 x 256 tiles, four waves of 128 x 128 results each (all 256 accumulator
// registers), one workgroup a compute unit, which walks over its tiles without a pause: what comes next is loaded
// straight into LDS two steps ahead, also across tiles, in steps of 128 values. What bounds it: the matrix
// cores and the chip's power (1.5 GHz with normally distributed codes; zeros run at 2.3 GHz and are
// no faster than the loads), next to the latency of HBM behind 64 KB of loads a compute unit.
// What the measurements showed, each as the kernel stood:
// - Whole lines. With 64 bytes of a row per load, a compute unit takes in 59 GB/s from L2, with 128 bytes 123 to
//   130 (and 64 experts of 512 rows, 7168 to 4096, 1044 against 994 us).
// - Loads between the products. A wave whose next load waits for the address unit issues no products: two
//   loads for every four products instead of eight in a row, 8192^3 2142 against 2375 TOP/s.
// - Scales through LDS beside the operands, not from memory at the tile's end (25 against 10 us a tile).
// - A tile's blocks of 32 rows alternate between the waves, so that few rows are shared out evenly, and absent
//   ones cost no products.
// Measured on MI355X: 8192^3 461 us (2385 TOP/s; a large library product of the same codes 472), three pairs of
// matrices in turn 484 (480); 64 experts of 512 rows, 7168 to 4096, 890 to 966 by the card, 8 of 2048 rows, 4096 to
// 2048, 127 to 143 (2160 to 1930). Fewer tiles than compute units leave the others idle: one matrix of
// 64 to 128 rows, 7168 to 4096, takes 55 and 57 us, of 256 to 2048 rows 70 to 73, and 4096 to 1024 25 to 45.
//
// Experts with up to 32 rows: their weights are read once, which HBM bounds; see few_rows. 64 experts of
// 8 rows, 7168 to 4096, 314 us (6.0 TB/s), of 32 rows 357; one row 8.3 us with the host's time (the kernel 8.8
// under a trace). The border: 64 experts of 32 rows 355 us there and 380 in tiles, and with up to 128
// rows in parts of 32 496 to 918 us against 386 to 435 in tiles.
#include <type_traits>

#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x16 __attribute__((ext_vector_type(16)));
typedef const __attribute__((address_space(3))) void lds_void;

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr uint32_t kOutside = 0x80000000u;  // an offset outside every descriptor (below 2^30 bytes here)
constexpr uint32_t kBehind = 0x40000000u;   // added to an offset, outside too; to kOutside as well
constexpr int kXcds = 8;
constexpr int kStep = 128;                  // values of the long axis per step: a cache line of a row

// What is the same in every lane, said so: the assembly below takes scalar registers.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  const uint64_t v = (uint64_t)base;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return __builtin_amdgcn_make_buffer_rsrc((void *)((uint64_t)hi << 32 | lo), (short)0,
                                           __builtin_amdgcn_readfirstlane((int)bytes), kRawBufferFlags);
}
// 16 bytes per lane from memory to 1 KB of LDS at `to` (the same in every lane), lane after lane;
// an offset outside the descriptor writes zeros. In assembly, because the compiler waits for every
// load on its way before it reads LDS, whatever place the load writes: the waits are the kernel's own.
// m0 holds the place. It is named as overwritten, so that the compiler keeps no value of its own there; that it
// says that such a register is not restored is what is meant.
#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
__device__ __forceinline__ uint32_t lds_at(const void *p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uintptr_t)(lds_void *)p);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(from)
               : "memory", "m0");
}
// The same with 4 bytes per lane, for scales.
__device__ __forceinline__ void touch(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dword %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(from)
               : "memory", "m0");
}
#pragma clang diagnostic pop
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// A workgroup's tile: 256 rows by 256 channels, a quarter for each of four waves: 128 channels (four
// blocks of 32) and every second block of 32 rows, so that a tile of few rows is shared out evenly.
constexpr int kSide = 256, kBlock = 32, kBlocks = 4;
constexpr int kOperandBytes = kSide * kStep, kStageBytes = 2 * kOperandBytes;  // of a step: x, then w
constexpr int kLineOut = 128, kStrideOut = kLineOut + 16;  // results leave by lines of 32 rows

__device__ __forceinline__ int tiles_of(int rows) { return rows / kSide + (rows % kSide != 0); }

// The rows of expert e inside the buffer: their number, and the first in `begin`.
__device__ __forceinline__ int span_of(const QuantizedMatmulArgs &a, int e, int &begin) {
  if (a.counts == nullptr) {
    begin = 0;
    return (int)a.capacity;
  }
  begin = a.offsets[e];
  const int n = clip_span(begin, a.counts[e], a.capacity);
  return n > 0 ? n : 0;
}

// Tiles of the experts before e, for every e: a workgroup's own prefix sums in LDS.
template <class F>
__device__ __forceinline__ void prefix_tiles(int *before, int *wave_sums, int E, F tiles) {
  const int per = (E + kThreads - 1) / kThreads, first = threadIdx.x * per;
  int own = 0;
  for (int i = 0; i < per; ++i)
    if (first + i < E) own += tiles(first + i);
  const int upto = wave_inclusive_scan(own);
  const int wave = threadIdx.x / kWave;
  if ((threadIdx.x & (kWave - 1)) == kWave - 1) wave_sums[wave] = upto;
  __syncthreads();
  int sum = upto - own;
  for (int w = 0; w < wave; ++w) sum += wave_sums[w];
  for (int i = 0; i < per; ++i)
    if (first + i < E) {
      before[first + i] = sum;
      sum += tiles(first + i);
    }
  if (threadIdx.x == kThreads - 1) before[E] = sum;
  __syncthreads();
}

struct Unit {
  int e, rows, cols, n0;
  int64_t first;  // row of the buffer
};

// The expert whose tiles unit v is among, not before `from`: most often that one or the next.
__device__ __forceinline__ int expert_of(const int *before, int E, int v, int from) {
  if (from + 1 >= E || __builtin_amdgcn_readfirstlane(before[from + 1]) > v) return from;
  int lo = from + 1, hi = E;  // before[lo] <= v < before[hi]
  if (lo + 1 < E && __builtin_amdgcn_readfirstlane(before[lo + 1]) > v) return lo;
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (__builtin_amdgcn_readfirstlane(before[mid]) <= v) lo = mid;
    else hi = mid;
  }
  return lo;
}

// Few rows: a workgroup takes RT * 16 channels of an expert with up to MT * 16 rows, its four waves a
// quarter of the long axis each, through a ring of LDS of their own that no other wave waits for. The
// rings run on from unit to unit, so that HBM never waits; a unit's sums meet in LDS (integers: in any order).
constexpr int kFew = 32;              // rows
constexpr int kRingBytes = 36 * 1024;  // of a wave
constexpr int kScaleSlots = 9;         // units whose scales may be in LDS: one more than a ring has steps, and the one before
struct FewLds {
  char ring[kWaves][kRingBytes];
  int sums[kFew * 64];
  float scales[kScaleSlots][64 + kFew];
  int before[EP_MAX_EXPERTS + 1];
  int wave_sums[kWaves];
};

// Units u0, u0 + by, ... before u1.
template <bool FP32, int RT, int MT>
__device__ __forceinline__ void few_rows(const QuantizedMatmulArgs &a, FewLds &lds, int u0, int u1, int by) {
  constexpr int kChannels = RT * 16, kRows = MT * 16, kLoads = 2 * (RT + MT);
  constexpr int kStepBytes = (kChannels + kRows) * kStep;
  constexpr int kDeep = kRingBytes / kStepBytes < 8 ? kRingBytes / kStepBytes : 8;  // steps in a ring
  static_assert(kDeep < kScaleSlots && (kDeep - 1) * kLoads < 60, "units in flight, and what a wait can count");
  const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int N = a.N, K = a.K;
  const int tiles_n = (N + kChannels - 1) / kChannels, steps = (K + kStep - 1) / kStep;
  prefix_tiles(lds.before, lds.wave_sums, a.E, [&](int e) {
    int b;
    const int n = span_of(a, e, b);
    return n > 0 && n <= kFew ? tiles_n : 0;
  });
  const int s0 = steps * wave / kWaves, own = steps * (wave + 1) / kWaves - s0;  // the last wave has a step at least
  struct Unit {
    int e, rows, n0;
    int64_t first;
  };
  const auto locate = [&](int v, int from) {
    Unit t{expert_of(lds.before, a.E, v, from), 0, 0, 0};
    int begin;
    t.rows = __builtin_amdgcn_readfirstlane(span_of(a, t.e, begin));
    t.first = __builtin_amdgcn_readfirstlane(begin);
    t.n0 = (v - __builtin_amdgcn_readfirstlane(lds.before[t.e])) * kChannels;
    if (t.n0 < 0 || t.n0 >= N || t.rows > kFew) t.rows = 0, t.n0 = 0;  // never for spans of a layout
    return t;
  };
  const auto channels = [&](const Unit &t) { return t.rows == 0 ? 0 : (N - t.n0 < kChannels ? N - t.n0 : kChannels); };
  const int piece = ((lane & 7) ^ (lane >> 4)) * 16;
  const uint32_t off = (uint32_t)(lane >> 3) * (uint32_t)K;
  const uint32_t ring = lds_at(lds.ring[wave]);
  // What is loaded next: a step of a unit ahead of the one that is multiplied.
  int au = u0, as = 0, aslot = 0, aturn = 0;
  Unit at = locate(au, 0);
  const auto rows_of = [&](const Unit &t) { return buffer_of((const char *)a.x + t.first * K, (int64_t)t.rows * K); };
  const auto channels_of = [&](const Unit &t) {
    return buffer_of((const char *)a.w + ((int64_t)t.e * N + t.n0) * K, (int64_t)channels(t) * K);
  };
  __amdgpu_buffer_rsrc_t bx = rows_of(at), bw = channels_of(at);
  const auto load = [&] {
    if (as == 0 && wave == kWaves - 1) {  // a unit's scales, ahead of its steps
      touch(buffer_of(a.w_scales + (int64_t)at.e * N + at.n0, (int64_t)channels(at) * 4), lane * 4u,
            lds_at(lds.scales[aturn]));
      const __amdgpu_buffer_rsrc_t bs =
          buffer_of(a.x_scales + at.first * a.x_scale_cols, (int64_t)at.rows * a.x_scale_cols * 4);
      const uint32_t to = lds_at(lds.scales[aturn] + 64);
      if (lane < kFew) touch(bs, lane * (uint32_t)a.x_scale_cols * 4u, to);  // there is no room for 64
    }
    const uint32_t to = ring + aslot * kStepBytes;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const uint32_t k = (s0 + as) * kStep + (i & 1 ? piece ^ 64 : piece);
      const int block = i < 2 * RT ? i : i - 2 * RT;
      load_to_lds(i < 2 * RT ? bw : bx, off + (uint32_t)(block * 8) * (uint32_t)K + (k < (uint32_t)K ? k : kBehind), to + i * 1024);
    }
    aslot = aslot + 1 < kDeep ? aslot + 1 : 0;
    if (++as == own) {
      as = 0, au += by, aturn = aturn + 1 < kScaleSlots ? aturn + 1 : 0;
      if (au < u1) at = locate(au, at.e);
      else at.rows = 0;
      bx = rows_of(at), bw = channels_of(at);
    }
  };
  if (own > 0)
    for (int i = 0; i < kDeep - 1; ++i) load();
  for (int i = threadIdx.x; i < kRows * kChannels; i += kThreads) lds.sums[i] = 0;
  int slot = 0, turn = 0, e = 0;
  for (int u = u0; u < u1; u += by, turn = turn + 1 < kScaleSlots ? turn + 1 : 0) {
    i32x4 acc[RT][MT];
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int q = 0; q < MT; ++q) acc[p][q] = i32x4{0, 0, 0, 0};
    for (int s = 0; s < own; ++s) {
      // This step's loads are there (those behind it may be on their way: loads return in order), and
      // the last step's operands have been read, whose place the next loads take.
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((kDeep - 2) * kLoads) : "memory");
      __builtin_amdgcn_sched_barrier(0);
      load();
      const char *const from = lds.ring[wave] + slot * kStepBytes + r16 * kStep;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int p16 = ((4 * j + g) ^ (r16 >> 1)) * 16;
        i32x4 w[RT], x[MT];
#pragma unroll
        for (int p = 0; p < RT; ++p) w[p] = *(const i32x4 *)(from + p * 16 * kStep + p16);
#pragma unroll
        for (int q = 0; q < MT; ++q) x[q] = *(const i32x4 *)(from + (kChannels + q * 16) * kStep + p16);
#pragma unroll
        for (int p = 0; p < RT; ++p)
#pragma unroll
          for (int q = 0; q < MT; ++q) acc[p][q] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[p], x[q], acc[p][q], 0, 0, 0);
      }
      slot = slot + 1 < kDeep ? slot + 1 : 0;
    }
    const Unit t = locate(u, e);
    e = t.e;
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");  // the last unit's sums have been read and cleared
#pragma unroll
    for (int p = 0; p < RT; ++p)
#pragma unroll
      for (int q = 0; q < MT; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i) atomicAdd(&lds.sums[(q * 16 + r16) * kChannels + p * 16 + g * 4 + i], acc[p][q][i]);
    asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
    constexpr int kLanes = kChannels / 4;  // four channels a thread
#pragma unroll
    for (int first = 0; first < kRows; first += kThreads / kLanes) {
      const int row = first + threadIdx.x / kLanes, c = threadIdx.x % kLanes * 4;
      if (row >= kRows) continue;
      i32x4 *const from = (i32x4 *)(lds.sums + row * kChannels + c);
      const i32x4 sum = *from;
      *from = i32x4{0, 0, 0, 0};
      if (row >= t.rows || t.n0 + c >= N) continue;
      const float sx = lds.scales[turn][64 + row];
      const f32x4 sw = *(const f32x4 *)(lds.scales[turn] + c);
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = (float)sum[i] * sx * sw[i];
      const int64_t to = (t.first + row) * N + t.n0 + c;
      if constexpr (FP32) *(f32x4 *)((float *)a.y + to) = v;
      else *(u32x2 *)((uint16_t *)a.y + to) = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
    }
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads into this workgroup's LDS
}

// What the experts' rows ask for, found by every workgroup: tiles of the experts with many rows, and
// units of those with few. A unit takes 64 channels where that makes one for every workgroup, else 16
// (7168 to 4096, 4 experts of 20 rows 27 against 34 us, of one row 23 against 26; from two or four on: no better).
// When there are fewer tiles than workgroups, the others take kBeside units of 64 channels each in the
// meantime, and the second launch begins behind those. Top-8 of 64 experts by Zipf, without and with 3, 4, 6, 8 and 10:
//   128 tokens, 7168 -> 4096  378  364 352 340 351 362 us (128 tiles)
//   64 tokens, 7168 -> 4096   381  352 340 331 328 334    (32 to 64 tiles)
//   128 tokens, 2048 -> 7168  224  225 220 229 240 250    (196 to 224 tiles)
//   top-4 of 32 experts, 4096 -> 2048  106  79 68 67 68 68 (32 to 40 tiles)
// Both sides' times grow with the long axis, so the number does not go by it. Both kinds shared out in one launch: 400.
constexpr int kBeside = 6;
struct Plan {
  int tiles, rows, units, early, idle;  // rows: the most of an expert with few
  bool wide;
};
__device__ __forceinline__ Plan plan_of(const QuantizedMatmulArgs &a, int *lds) {
  if (threadIdx.x < 3) lds[threadIdx.x] = 0;
  __syncthreads();
  const int tiles_n = (a.N + kSide - 1) / kSide;
  for (int e = threadIdx.x; e < a.E; e += kThreads) {
    int b;
    const int n = span_of(a, e, b);
    if (n > kFew) atomicAdd(&lds[0], tiles_of(n) * tiles_n);
    else if (n > 0) atomicAdd(&lds[1], 1), atomicMax(&lds[2], n);
  }
  __syncthreads();
  Plan p;
  p.tiles = __builtin_amdgcn_readfirstlane(lds[0]);
  const int active = __builtin_amdgcn_readfirstlane(lds[1]);
  p.rows = __builtin_amdgcn_readfirstlane(lds[2]);
  __syncthreads();
  const int grid = gridDim.x;
  p.wide = (int64_t)active * ((a.N + 63) / 64) >= grid;
  p.units = active * (p.wide ? (a.N + 63) / 64 : (a.N + 15) / 16);
  p.idle = p.tiles > 0 && p.tiles < grid ? grid - p.tiles : 0;
  const int fit = p.idle * (p.wide ? kBeside : 4 * kBeside);
  p.early = fit < p.units ? fit : p.units;
  return p;
}
template <bool FP32>
__device__ __forceinline__ void few_units(const QuantizedMatmulArgs &a, FewLds &lds, const Plan &p, int u0, int u1, int by) {
  if (u0 >= u1) return;
  if (p.wide) {
    if (p.rows <= 16) few_rows<FP32, 4, 1>(a, lds, u0, u1, by);
    else few_rows<FP32, 4, 2>(a, lds, u0, u1, by);
  } else {
    if (p.rows <= 16) few_rows<FP32, 1, 1>(a, lds, u0, u1, by);
    else few_rows<FP32, 1, 2>(a, lds, u0, u1, by);
  }
}

template <bool FP32>
__global__ __launch_bounds__(kThreads, 1) void ep_quantized_matmul_few(const QuantizedMatmulArgs a) {
  __shared__ __attribute__((aligned(1024))) FewLds lds;
  const Plan p = plan_of(a, lds.sums);
  few_units<FP32>(a, lds, p, p.early + blockIdx.x, p.units, gridDim.x);
}

template <bool FP32>
__global__ __launch_bounds__(kThreads, 1) void ep_quantized_matmul_tiles(const QuantizedMatmulArgs a) {
  constexpr int kLoads = kSide / 8 / kWaves;  // of a wave per operand and step: a line of 8 rows each
  constexpr int kElt = FP32 ? 4 : 2;
  __shared__ __attribute__((aligned(1024))) union {
    struct {
      char stages[2 * kStageBytes];
      char lines[kWaves * kBlock * kStrideOut];
      float scales[3][2][kSide];  // of x's rows and of channels, for three units in turn
      int before[EP_MAX_EXPERTS + 1];
      int wave_sums[kWaves];
    };
    FewLds few;
  } lds;
  const int lane = lane_id(), r32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = (wave & 1) * kBlock, wn = (wave >> 1) * (kSide / 2);
  const int N = a.N, K = a.K;
  const int tiles_n = (N + kSide - 1) / kSide, steps = (K + kStep - 1) / kStep;
  const Plan plan = plan_of(a, lds.wave_sums);
  const int units = plan.tiles;
  if (units == 0) return;
  // Workgroup b runs on XCD b % 8: each XCD takes a run of consecutive tiles.
  const int xcd = blockIdx.x % kXcds, group = blockIdx.x / kXcds, groups = (gridDim.x + kXcds - 1 - xcd) / kXcds;
  const int64_t active = gridDim.x < kXcds ? gridDim.x : kXcds;
  const int u1 = (int)(units * (int64_t)(xcd + 1) / active);
  int u = (int)(units * (int64_t)xcd / active) + group;
  if (u >= u1) {
    // Idle workgroups before this one: of the XCDs before, then of its own.
    int idle = u - u1;
    for (int x = 0; x < xcd; ++x) {
      const int have = (gridDim.x + kXcds - 1 - x) / kXcds;
      const int take = (int)(units * (int64_t)(x + 1) / active) - (int)(units * (int64_t)x / active);
      idle += have > take ? have - take : 0;
    }
    if (idle < plan.idle) few_units<FP32>(a, lds.few, plan, idle, plan.early, plan.idle);
    return;
  }
  prefix_tiles(lds.before, lds.wave_sums, a.E, [&](int e) {
    int b;
    const int n = span_of(a, e, b);
    return n > kFew ? tiles_of(n) * tiles_n : 0;
  });
  // Unit v, for an expert that is not before `from`.
  const auto locate = [&](int v, int from) {
    Unit t{expert_of(lds.before, a.E, v, from), 0, 0, 0, 0};
    int begin;
    const int count = __builtin_amdgcn_readfirstlane(span_of(a, t.e, begin)), tiles_m = tiles_of(count);
    const int i = v - __builtin_amdgcn_readfirstlane(lds.before[t.e]);
    if (i < 0 || i >= tiles_m * tiles_n) return t;  // spans that overlap so often that their tiles pass 2^31
    constexpr int kTall = 4;  // row tiles side by side before the next column tile
    const int tall = i / (kTall * tiles_n), left = tiles_m - tall * kTall, width = left < kTall ? left : kTall;
    const int in = i - tall * kTall * tiles_n, m0 = (tall * kTall + in % width) * kSide;
    t.n0 = in / width * kSide;
    t.rows = count - m0 < kSide ? count - m0 : kSide, t.cols = N - t.n0 < kSide ? N - t.n0 : kSide;
    t.first = (int64_t)__builtin_amdgcn_readfirstlane(begin) + m0;
    return t;
  };
  // A unit's operands. A descriptor ends with its last row, so rows behind it read as zeros.
  const auto rows_of = [&](const Unit &t) {
    return buffer_of((const char *)a.x + t.first * K, (int64_t)t.rows * K);
  };
  const auto channels_of = [&](const Unit &t) {
    return buffer_of((const char *)a.w + ((int64_t)t.e * N + t.n0) * K, (int64_t)t.cols * K);
  };
  // A load brings a line of 8 rows. Lane l takes row l / 8 and the 16 bytes (l % 8) ^ (row / 2 % 8) of
  // it, so that the 16 bytes of one place in 16 rows, which are read together, lie in different banks.
  const int piece = ((lane & 7) ^ (lane >> 4)) * 16;  // of even loads; 64 bytes off in odd ones
  uint32_t off[kLoads];
#pragma unroll
  for (int i = 0; i < kLoads; ++i) off[i] = (uint32_t)((wave * kLoads + i) * 8 + (lane >> 3)) * (uint32_t)K;
  const uint32_t stages = lds_at(lds.stages), place = stages + wave * kLoads * 1024;
  const auto load_scales = [&](const Unit &t, int turn) {
    touch(buffer_of(a.x_scales + t.first * a.x_scale_cols, (int64_t)t.rows * a.x_scale_cols * 4),
          threadIdx.x * (uint32_t)a.x_scale_cols * 4u, lds_at(lds.scales[turn][0] + wave * kWave));
    touch(buffer_of(a.w_scales + (int64_t)t.e * N + t.n0, (int64_t)t.cols * 4), threadIdx.x * 4u,
          lds_at(lds.scales[turn][1] + wave * kWave));
  };
  // What is loaded next: a step of a unit that may be ahead of the one that is multiplied.
  struct {
    Unit unit;
    int u, step, turn;
    uint32_t place;
  } ahead{locate(u, 0), u, 0, 0, place};
  __amdgpu_buffer_rsrc_t ahead_x = rows_of(ahead.unit), ahead_w = channels_of(ahead.unit);
  const auto advance = [&](int to) {
    ahead.place = place + to * kStageBytes;
    if (++ahead.step < steps) return;
    ahead.step = 0, ahead.u += groups, ahead.turn = ahead.turn < 2 ? ahead.turn + 1 : 0;
    if (ahead.u < u1) ahead.unit = locate(ahead.u, ahead.unit.e);
    else ahead.unit.rows = ahead.unit.cols = 0;
    ahead_x = rows_of(ahead.unit), ahead_w = channels_of(ahead.unit);
    load_scales(ahead.unit, ahead.turn);
  };
  const auto load = [&](int from, int to) {  // of the 2 kLoads loads of a step and wave, x's first
#pragma unroll
    for (int d = 0; d < 2 * kLoads; ++d) {
      if (d < from || d >= to) continue;
      const int i = d % kLoads;
      const uint32_t at = ahead.step * kStep + (i & 1 ? piece ^ 64 : piece);
      load_to_lds(d < kLoads ? ahead_x : ahead_w, off[i] + (at < (uint32_t)K ? at : kBehind),
                  ahead.place + (d < kLoads ? 0 : kOperandBytes) + i * 1024);
    }
  };
  // A step's loads that are issued by the ends of the last part of the second step before it, and of
  // the parts of the step before it.
  constexpr int kIssued[4] = {8, 16, 16, 16};
  int stage = 0, turn = 0;  // of the step, of the unit
  load_scales(ahead.unit, 0);
  load(0, 2 * kLoads);
  advance(1);
  load(0, kIssued[0]);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(kIssued[0]) : "memory");
  Unit unit{0, 0, 0, 0, 0};

  const auto tile = [&](auto row_blocks) {
    constexpr int Q = decltype(row_blocks)::value;  // of every wave
    i32x16 acc[kBlocks][Q];  // [channels][rows]
#pragma unroll
    for (int p = 0; p < kBlocks; ++p)
#pragma unroll
      for (int q = 0; q < Q; ++q) acc[p][q] = i32x16{};
    struct Operands {
      i32x4 w[kBlocks], x[Q];
    };
    const int turned = r32 >> 1 & 7;
    const char *const at = lds.stages + (wm + r32) * kStep;
    const int to_w = kOperandBytes + (wn - wm) * kStep;
    const auto fetch = [&](int part, int p, Operands &o) {  // the p-th block of both
      const char *const from = at + stage * kStageBytes + ((2 * part + half) ^ turned) * 16;
      o.w[p] = *(const i32x4 *)(from + to_w + p * kBlock * kStep);
      if (p < Q) o.x[p] = *(const i32x4 *)(from + p * 2 * kBlock * kStep);
    };
    // Products of one part of a step, and between them the reads of the next part's operands and the
    // loads [from, to), a few at a time: a wave that waits for the memory path issues no products.
    const auto multiply = [&](const Operands &o, int part, Operands &coming, int from, int to) {
#pragma unroll
      for (int p = 0; p < kBlocks; ++p) {
        fetch(part, p, coming);
        load(from + (to - from) * p / kBlocks, from + (to - from) * (p + 1) / kBlocks);
#pragma unroll
        for (int q = 0; q < Q; ++q)
          acc[p][q] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[p], o.x[q], acc[p][q], 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    Operands even, odd;
#pragma unroll
    for (int p = 0; p < kBlocks; ++p) fetch(0, p, even);
    for (int s = 0; s < steps; ++s) {
      multiply(even, 1, odd, kIssued[0], kIssued[1]);
      multiply(odd, 2, even, kIssued[1], kIssued[2]);
      multiply(even, 3, odd, kIssued[2], kIssued[3]);
      // Before the next step's operands are read its loads have to be there, and every wave has read
      // this step's, whose place the loads of the step behind it take.
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
      advance(stage);
      stage ^= 1;
      multiply(odd, 0, even, 0, kIssued[0]);  // behind the last step: operands that are not used
    }
    // Results leave through LDS as whole lines of 32 rows.
    char *const mine = lds.lines + wave * kBlock * kStrideOut;
    constexpr int kChannels = kLineOut / kElt, kChunks = kSide / 2 / kChannels;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int row0 = wm + q * 2 * kBlock, here = unit.rows - row0 < kBlock ? unit.rows - row0 : kBlock;
      const float sx = lds.scales[turn][0][row0 + r32];
      // a wave whose rows or channels all lie behind the end stores nothing: a descriptor of no bytes
      const __amdgpu_buffer_rsrc_t by =
          buffer_of((const char *)a.y + ((unit.first + row0) * N + unit.n0 + wn) * kElt,
                    here > 0 && wn < unit.cols ? ((int64_t)(here - 1) * N + unit.cols - wn) * kElt : 0);
#pragma unroll
      for (int c = 0; c < kChunks; ++c) {
#pragma unroll
        for (int n = 0; n < kChannels; n += 8) {
          const int p = (c * kChannels + n) / kBlock, i = n / 8 % 4;
          const f32x4 sw = *(const f32x4 *)(lds.scales[turn][1] + wn + c * kChannels + n + half * 4);
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = (float)acc[p][q][i * 4 + j] * sx * sw[j];
          char *const to = mine + r32 * kStrideOut + (n + half * 4) * kElt;
          if constexpr (FP32) *(f32x4 *)to = v;
          else *(u32x2 *)to = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        const int col = wn + c * kChannels + lane % 8 * (16 / kElt);
        uint32_t off_y = col < unit.cols ? (uint32_t)(lane / 8 * N + col - wn) * kElt : kOutside;
#pragma unroll
        for (int i = 0; i < kBlock / 8; ++i) {
          const u32x4 v = *(const u32x4 *)(mine + (i * 8 + lane / 8) * kStrideOut + lane % 8 * 16);
          __builtin_amdgcn_raw_buffer_store_b128(v, by, (int)off_y, 0, 0);
          off_y += (uint32_t)(8 * N) * kElt;
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    }
  };
  for (; u < u1; u += groups, turn = turn < 2 ? turn + 1 : 0) {
    unit = locate(u, unit.e);
    if (unit.rows > 6 * kBlock) tile(std::integral_constant<int, 4>());
    else if (unit.rows > 4 * kBlock) tile(std::integral_constant<int, 3>());
    else if (unit.rows > 2 * kBlock) tile(std::integral_constant<int, 2>());
    else tile(std::integral_constant<int, 1>());
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // loads into this workgroup's LDS
}

}  // namespace

int launch_quantized_matmul(const QuantizedMatmulArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  const unsigned grid = cap > 0 && cap < 256 ? cap : 256;
  const auto run = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, a.stream>>>(a);
    return launch_status();
  };
  // Experts with many rows, then those with few: a buffer of few rows has none of the first, and one
  // expert without routing arrays is of one kind.
  if (a.capacity > kFew) {
    const int rc = a.fp32 ? run(ep_quantized_matmul_tiles<true>) : run(ep_quantized_matmul_tiles<false>);
    if (rc != 0 || a.counts == nullptr) return rc;
  }
  return a.fp32 ? run(ep_quantized_matmul_few<true>) : run(ep_quantized_matmul_few<false>);
}

}  // namespace ep
