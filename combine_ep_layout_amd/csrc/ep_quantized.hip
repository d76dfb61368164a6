// The experts' products in 8-bit integers on the expand layout for gfx950:
// y[r, n] = x_scales[r] * w_scales[e, n] * sum over k of x[r, k] w[e, n, k].
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

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
}
__device__ __forceinline__ const char *uniform(const char *p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return (const char *)((uint64_t)hi << 32 | lo);
}
// 16 bytes per lane from memory to 1 KB of LDS at `to` (the same in every lane), lane after lane;
// an offset outside the descriptor writes zeros. In assembly, because the compiler waits for every
// load on its way before it reads LDS, whatever place the load writes: the waits are the kernel's own.
// Nothing else here uses m0, which holds the place.
__device__ __forceinline__ uint32_t lds_at(const void *p) {
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)(uintptr_t)(lds_void *)p);
}
__device__ __forceinline__ void load_to_lds(__amdgpu_buffer_rsrc_t from, uint32_t off, uint32_t to) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tbuffer_load_dwordx4 %1, %2, 0 offen lds" ::"s"(to), "v"(off), "s"(from)
               : "memory");
}
__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// A wave's tile: 128 rows of x by 128 channels, as 4 x 4 products of 32 x 32.
constexpr int kSide = 128, kBlocks = kSide / 32;

// WM x (4 / WM) waves.
template <int WM>
struct Shape {
  static constexpr int kWN = kWaves / WM;
  static constexpr int kRows = WM * kSide, kCols = kWN * kSide;
  static constexpr int kStageBytes = (kRows + kCols) * kStep;
  static constexpr int kStages = 2;
};

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

template <int WM, bool FP32>
__global__ __launch_bounds__(kThreads, 1) void ep_quantized_matmul_tiles(const QuantizedMatmulArgs a) {
  using S = Shape<WM>;
  constexpr int kXBlocks = S::kRows / 8 / kWaves, kWBlocks = S::kCols / 8 / kWaves;  // per wave, of 8 rows
  constexpr int kLoads = kXBlocks + kWBlocks;
  constexpr int kElt = FP32 ? 4 : 2, kStrideOut = kSide * kElt + 16;
  static_assert(kWaves * 32 * kStrideOut <= S::kStages * S::kStageBytes, "results pass through the stages");
  __shared__ __attribute__((aligned(1024))) char lds[S::kStages * S::kStageBytes];
  __shared__ int before[EP_MAX_EXPERTS + 1];
  __shared__ int wave_sums[kWaves];
  const int lane = lane_id(), r32 = lane & 31, half = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wm = wave % WM * kSide, wn = wave / WM * kSide;
  const int N = a.N, K = a.K;
  const uint32_t stages = lds_at(lds);
  const int tiles_n = (N + S::kCols - 1) / S::kCols, steps = (K + kStep - 1) / kStep;
  const auto span = [&](int e, int &begin) {
    if (a.counts == nullptr) {
      begin = 0;
      return (int)a.capacity;
    }
    begin = a.offsets[e];
    const int n = clip_span(begin, a.counts[e], a.capacity);
    return n > 0 ? n : 0;
  };
  prefix_tiles(before, wave_sums, a.E, [&](int e) {
    int b;
    return (span(e, b) + S::kRows - 1) / S::kRows * tiles_n;
  });
  const int units = __builtin_amdgcn_readfirstlane(before[a.E]);
  // Workgroup b runs on XCD b % 8: each XCD takes a run of consecutive units.
  const int xcd = blockIdx.x % kXcds, group = blockIdx.x / kXcds, groups = (gridDim.x + kXcds - 1 - xcd) / kXcds;
  const int64_t active = gridDim.x < kXcds ? gridDim.x : kXcds;
  const int u1 = (int)(units * (xcd + 1) / active);
  for (int u = (int)(units * xcd / active) + group; u < u1; u += groups) {
    int lo = 0, hi = a.E;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (before[mid] <= u) lo = mid;
      else hi = mid;
    }
    const int e = __builtin_amdgcn_readfirstlane(lo);
    int begin;
    const int count = __builtin_amdgcn_readfirstlane(span(e, begin));
    const int t = u - __builtin_amdgcn_readfirstlane(before[e]), tiles_m = (count + S::kRows - 1) / S::kRows;
    if (t < 0 || t >= tiles_m * tiles_n) continue;  // spans that overlap so often that their tiles pass 2^31
    constexpr int kTall = 4;  // row tiles side by side before the next column tile
    const int tall = t / (kTall * tiles_n), left = tiles_m - tall * kTall, width = left < kTall ? left : kTall;
    const int in = t - tall * kTall * tiles_n;
    const int m0 = (tall * kTall + in % width) * S::kRows, n0 = in / width * S::kCols;
    const int rows = count - m0 < S::kRows ? count - m0 : S::kRows, cols = N - n0 < S::kCols ? N - n0 : S::kCols;
    const int64_t first = (int64_t)begin + m0;
    const __amdgpu_buffer_rsrc_t bx = buffer_of(uniform((const char *)a.x + first * K), (int64_t)rows * K);
    const __amdgpu_buffer_rsrc_t bw =
        buffer_of(uniform((const char *)a.w + ((int64_t)e * N + n0) * K), (int64_t)cols * K);
    // A load brings a line of 8 rows. Lane l takes row l / 8 and the 16 bytes (l % 8) ^ (row / 2 % 8) of
    // it, so that the 16 bytes of one place in 16 rows, which are read together, lie in different banks.
    const int piece = ((lane & 7) ^ (lane >> 4)) * 16;  // of even blocks; 64 bytes off in odd ones
    uint32_t off[kLoads];
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const bool of_x = i < kXBlocks;
      const int row = (of_x ? wave * kXBlocks + i : wave * kWBlocks + i - kXBlocks) * 8 + (lane >> 3);
      off[i] = row < (of_x ? rows : cols) ? (uint32_t)row * (uint32_t)K : kOutside;
    }
    const auto load = [&](int step, int from, int to) {  // the loads [from, to) of a step
      uint32_t k[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t at = step * kStep + (piece ^ i * 64);
        k[i] = at < (uint32_t)K ? at : kBehind;
      }
      const uint32_t place = stages + (step & 1) * S::kStageBytes;
#pragma unroll
      for (int i = 0; i < kLoads; ++i) {
        if (i < from || i >= to) continue;
        const bool of_x = i < kXBlocks;
        const int block = of_x ? wave * kXBlocks + i : S::kRows / 8 + wave * kWBlocks + i - kXBlocks;
        load_to_lds(of_x ? bx : bw, off[i] + k[i & 1], place + block * 1024);
      }
    };
    i32x16 acc[kBlocks][kBlocks];  // [channels][rows]
#pragma unroll
    for (int p = 0; p < kBlocks; ++p)
#pragma unroll
      for (int q = 0; q < kBlocks; ++q) acc[p][q] = i32x16{};
    struct Operands {
      i32x4 w[kBlocks], x[kBlocks];
    };
    const int turn = r32 >> 1 & 7;
    const int at_x = (wm + r32) * kStep, at_w = (S::kRows + wn + r32) * kStep;
    const auto fetch = [&](int step, int part, Operands &o) {
      const char *const from = lds + (step & 1) * S::kStageBytes + (((2 * part + half) ^ turn) * 16);
#pragma unroll
      for (int p = 0; p < kBlocks; ++p) o.w[p] = *(const i32x4 *)(from + at_w + p * 32 * kStep);
#pragma unroll
      for (int q = 0; q < kBlocks; ++q) o.x[q] = *(const i32x4 *)(from + at_x + q * 32 * kStep);
    };
    const auto multiply = [&](const Operands &o) {
#pragma unroll
      for (int p = 0; p < kBlocks; ++p)
#pragma unroll
        for (int q = 0; q < kBlocks; ++q)
          acc[p][q] = __builtin_amdgcn_mfma_i32_32x32x32_i8(o.w[p], o.x[q], acc[p][q], 0, 0, 0);
#pragma unroll
      for (int i = 0; i < 8; ++i) {  // an LDS read, then two products
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
      }
      __builtin_amdgcn_sched_barrier(0);
    };
    // Before a step's operands are read its loads have to be there, and every wave has read the step
    // before it, whose place the next loads take.
    const auto arrive = [&] {
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");
      __builtin_amdgcn_sched_barrier(0);
    };
    __syncthreads();  // the last unit's results have left the stages
    load(0, 0, kLoads);
    Operands even, odd;
    arrive();
    fetch(0, 0, even);
    for (int s = 0; s < steps; ++s) {
      load(s + 1, 0, kLoads / 2);
      fetch(s, 1, odd);
      multiply(even);
      load(s + 1, kLoads / 2, kLoads);
      fetch(s, 2, even);
      multiply(odd);
      fetch(s, 3, odd);
      multiply(even);
      arrive();
      fetch(s + 1, 0, even);  // behind the last step: zeros that are not used
      multiply(odd);
    }
    // Results leave through LDS, 32 rows of a wave's 128 channels at a time, as whole lines.
    const __amdgpu_buffer_rsrc_t bs = buffer_of(uniform((const char *)(a.w_scales + (int64_t)e * N + n0)), (int64_t)cols * 4);
    char *const mine = lds + wave * 32 * kStrideOut;
#pragma unroll
    for (int q = 0; q < kBlocks; ++q) {
      const int row = wm + q * 32 + r32;
      const float sx = row < rows ? a.x_scales[(first + row) * a.x_scale_cols] : 0.f;
#pragma unroll
      for (int p = 0; p < kBlocks; ++p)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int n = p * 32 + i * 8 + half * 4;
          const f32x4 sw = __builtin_bit_cast(f32x4, __builtin_amdgcn_raw_buffer_load_b128(bs, (wn + n) * 4, 0, 0));
          f32x4 v;
#pragma unroll
          for (int j = 0; j < 4; ++j) v[j] = (float)acc[p][q][i * 4 + j] * sx * sw[j];
          char *const to = mine + r32 * kStrideOut + n * kElt;
          if constexpr (FP32) *(f32x4 *)to = v;
          else *(u32x2 *)to = u32x2{pack(v[0], v[1]), pack(v[2], v[3])};
        }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      const int here = rows - wm - q * 32 < 32 ? rows - wm - q * 32 : 32;
      // a wave whose rows or channels all lie behind the end stores nothing: a descriptor of no bytes
      const __amdgpu_buffer_rsrc_t by =
          buffer_of(uniform((const char *)a.y + ((first + wm + q * 32) * N + n0 + wn) * kElt),
                    here > 0 && wn < cols ? ((int64_t)(here - 1) * N + cols - wn) * kElt : 0);
      constexpr int kLanes = kSide * kElt / 16, kPasses = 32 * kLanes / kWave;
      const int c = lane % kLanes * (16 / kElt);
      uint32_t off_y = wn + c < cols ? (uint32_t)(lane / kLanes * N + c) * kElt : kOutside;
#pragma unroll
      for (int i = 0; i < kPasses; ++i) {
        const u32x4 v = *(const u32x4 *)(mine + (i * (kWave / kLanes) + lane / kLanes) * kStrideOut + c * kElt);
        __builtin_amdgcn_raw_buffer_store_b128(v, by, (int)off_y, 0, 0);
        off_y += (uint32_t)(kWave / kLanes * N) * kElt;
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    }
  }
}

}  // namespace

int launch_quantized_matmul(const QuantizedMatmulArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  const unsigned grid = cap > 0 && cap < 256 ? cap : 256;
  if (a.fp32) ep_quantized_matmul_tiles<2, true><<<grid, kThreads, 0, a.stream>>>(a);
  else ep_quantized_matmul_tiles<2, false><<<grid, kThreads, 0, a.stream>>>(a);
  return launch_status();
}

}  // namespace ep
