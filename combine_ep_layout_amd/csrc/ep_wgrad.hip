// The experts' weight gradient on the expand layout for gfx950:
// dW[e] = sum over the rows r of expert e of dy[r]^T x[r] (+ previous).
//
// Mathematics. A product whose summed axis is the rows, which both operands
// have as their slow axis: the matrix instructions (16x16x32 bf16) want eight
// consecutive rows of one column per lane. LDS holds the rows as they come
// (x turned from e4m3 to bf16 on the way), and the transposed LDS reads of
// gfx950 gather the columns: 16 lanes bring four rows' pieces of four columns
// and each leaves with four rows of one column. Row strides keep half a wave's
// pieces in different banks, and x lies in four planes, so that its writes do
// not meet in a few banks either (bank conflicts 24% of the cycles with rows
// as they come, 5% so; 64 experts 2 to 5% faster). Sums in binary32.
//
// What bounds it: with about a hundred rows per expert, writing the gradient
// (64 experts of 4096 x 7168 in bf16: 3.8 GB, 630 us for the stores alone);
// with thousands, the matrix cores. A workgroup of four waves takes 128
// columns of dy by 256 of x (64 x 128 a wave, 128 accumulator registers, two
// workgroups a compute unit); 128 x 128 tiles were slower at both ends (1150
// against 1080 and 392 against 335 us). Steps of 32 rows run three ahead: two
// on their way into registers, one in the other half of LDS, and loads and LDS
// stores are issued between the matrix instructions of a step (all at its
// start: 11% slower).
// Measured on MI355X: 64 experts of 128 e4m3 rows 1080 us (3.6 TB/s), with
// scales that are no powers of two (three products for every one, below) 2340;
// 8 experts of 2048 rows, 4096 by 2048, added to an fp32 gradient, 310 us in
// bf16 (885 TFLOP/s), 312 in e4m3 and 928 with scales of any kind. No kernel
// spills: a register that comes back from memory waits for every load and store
// of its wave (64 experts: 1153 us with one).
#include <type_traits>

#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef short s16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) s16x4 lds_s16x4;

constexpr int kThreads = 256;
constexpr int kTileN = 128, kTileH = 256;  // columns of dy and of x per workgroup
constexpr int kRows = 32;                  // rows of both per step
constexpr int kStrideY = kTileN * 2 + 32;  // LDS bytes per row of dy
// A row of x lies in LDS as four planes: columns 16 i + 4 j to + 3 are the 8 bytes i of plane j.
constexpr int kPlaneX = kTileH / 2 + 8, kStrideX = 4 * kPlaneX + 64;
constexpr int kStrideOut = 64 * 4 + 16;  // 16 rows of 64 results of a wave on their way out
constexpr int kXcds = 8;
constexpr uint32_t kOutside = 0x80000000u;  // an offset outside every descriptor
constexpr int kNonTemporal = 2;             // cache policy of a buffer access

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
}

// The same in every lane, said so: a descriptor that the compiler takes for a lane's own costs a loop
// around every access and registers (8 experts of 2048 bf16 rows 334 us against 310, and spills).
__device__ __forceinline__ const char *uniform(const char *p) {
  const uint64_t v = (uint64_t)p;
  const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)v);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(v >> 32));
  return (const char *)((uint64_t)hi << 32 | lo);
}

__device__ __forceinline__ uint32_t pack(float lo, float hi) {
  const f32x2 f = {lo, hi};
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
}

// Eight rows of one column per lane out of 32 rows in LDS: two transposed
// reads, in each of which the 16 lanes of group g bring four rows' four
// pieces of four columns.
__device__ __forceinline__ bf16x8 column(const char *upper, const char *lower) {
  const s16x4 a = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)upper);
  const s16x4 b = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4 *)lower);
  return __builtin_bit_cast(bf16x8, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

// Values of x = code * scale (e4m3 rows) as the matrix cores take them. Codes
// are exact in bf16, and so are their products with a power of two between
// 2^-64 and 2^64. Any other scale leaves up to 24 bits after the binary32
// product, which are three bf16 parts, each the upper half of what the ones
// before leave; with a product for each part nothing but bits below 2^-133
// (bf16's least step) is lost. Rounding x to bf16 instead would put the
// gradient of 128 rows with scales in [0.01, 1] off by 1.7e-3 where the sum in
// binary32 is off by 2e-7. What the scales are is found on the way: a tile is
// begun with one product, and begun again with three where a scale asks for it.
__device__ __forceinline__ void three_parts(float p, uint32_t (&part)[3]) {  // in the upper halves
#pragma clang fp contract(off)  // p is one rounded value: fused with its product, the parts could come from two
  part[0] = __float_as_uint(p);
  const float rest = p - __uint_as_float(part[0] & 0xFFFF0000u);
  part[1] = __float_as_uint(rest);
  part[2] = __float_as_uint(rest - __uint_as_float(part[1] & 0xFFFF0000u));
  if ((part[0] & 0x7F800000u) == 0x7F800000u) {  // an infinity or NaN is all in the first part
    part[0] |= (part[0] & 0x007FFFFFu) != 0 ? 0x00400000u : 0u;
    part[1] = part[2] = 0;
  }
}
__device__ __forceinline__ uint32_t upper_halves(uint32_t lo, uint32_t hi) { return lo >> 16 | (hi & 0xFFFF0000u); }

// One step's rows on the way from memory to LDS, in a thread's registers: it
// takes the same 16-byte pieces of every step (two of dy, then those of x), at
// offsets from the step's first row that are found once per tile.
template <bool FP8>
struct Stage {
  static constexpr int kPiecesX = FP8 ? 2 : 4, kPieces = 2 + kPiecesX;
  static constexpr int kValues = FP8 ? 16 : 8;  // of x in a piece
  __amdgpu_buffer_rsrc_t by, bx, bs;
  uint32_t off[kPieces], off_s[kPiecesX];
  u32x4 v[2][kPieces];
  float scale[2][kPiecesX];
  bool scaled;
  bool indirect = false;  // this lane has stored a piece whose scale is not for the direct conversion

  static __device__ __forceinline__ int row_y(int i) { return (threadIdx.x + i * kThreads) / (kTileN / 8); }
  static __device__ __forceinline__ int col_y(int i) { return (threadIdx.x + i * kThreads) % (kTileN / 8) * 8; }
  static __device__ __forceinline__ int row_x(int i) { return (threadIdx.x + i * kThreads) / (kTileH / kValues); }
  static __device__ __forceinline__ int col_x(int i) { return (threadIdx.x + i * kThreads) % (kTileH / kValues) * kValues; }

  __device__ __forceinline__ void place(int N, int H, int n0, int h0) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = n0 + col_y(i);
      off[i] = n < N ? ((uint32_t)row_y(i) * N + n) * 2u : kOutside;
    }
#pragma unroll
    for (int i = 0; i < kPiecesX; ++i) {
      const int h = h0 + col_x(i);
      off[2 + i] = h < H ? ((uint32_t)row_x(i) * H + h) * (FP8 ? 1u : 2u) : kOutside;
      if constexpr (FP8) off_s[i] = h < H ? ((uint32_t)row_x(i) * (H / 128) + h / 128) * 4u : kOutside;
    }
  }
  // The next pieces come from `rows` rows at these addresses; rows beyond read as zeros, and no
  // rows (the stream's end) touch no memory.
  __device__ __forceinline__ void aim(const char *y, const char *x, const char *s, int rows, int N,
                                      int H, bool with_scales) {
    rows = __builtin_amdgcn_readfirstlane(rows);
    by = buffer_of(uniform(y), (int64_t)(rows * N) * 2);
    bx = buffer_of(uniform(x), (int64_t)(rows * H) * (FP8 ? 1 : 2));
    if constexpr (FP8) {
      scaled = with_scales;
      bs = buffer_of(uniform(s), scaled ? rows * (H / 128) * 4 : 0);
    }
  }
  __device__ __forceinline__ void load(int set, int i) {
    v[set][i] = __builtin_amdgcn_raw_buffer_load_b128(i < 2 ? by : bx, (int)off[i], 0, 0);
    if constexpr (FP8)
      if (i >= 2) scale[set][i - 2] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(bs, (int)off_s[i - 2], 0, 0));
  }
  // 8 values of row r. In planes, threads that hold 16 consecutive values write 8 consecutive
  // bytes each, and the pieces of eight rows that half a wave reads at once lie in different banks.
  static __device__ __forceinline__ void put_x(char *lx, int r, int h, u32x4 w) {
    char *to = lx + r * kStrideX + (h >> 2 & 3) * kPlaneX + (h >> 4) * 8;
    *(u32x2 *)to = u32x2{w[0], w[1]};
    *(u32x2 *)(to + kPlaneX) = u32x2{w[2], w[3]};
  }
  __device__ __forceinline__ void store(int set, int i, char *ly, char *lx) {
    if (i < 2) {
      *(u32x4 *)(ly + row_y(i) * kStrideY + col_y(i) * 2) = v[set][i];
    } else if constexpr (FP8) {
      // One instruction converts two values: powers of two, and rows behind the end and groups of
      // zeros (codes 0 and a finite scale), which count as scaled by 1. A step with any other scale
      // is noted; its tile is done again.
      const u32x4 c = v[set][i];
      float s = scaled ? scale[set][i - 2] : 1.0f;
      if ((c[0] | c[1] | c[2] | c[3]) == 0 && (__float_as_uint(s) & 0x7F800000u) != 0x7F800000u) s = 1.0f;
      const uint32_t bits = __float_as_uint(s);
      indirect |= (bits & 0x807FFFFFu) != 0 || bits < 0x1F800000u || bits > 0x5F800000u;
      u32x4 w[2];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        w[d >> 1][(d & 1) * 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[d], s, false));
        w[d >> 1][(d & 1) * 2 + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c[d], s, true));
      }
      put_x(lx, row_x(i - 2), col_x(i - 2), w[0]);
      put_x(lx, row_x(i - 2), col_x(i - 2) + 8, w[1]);
    } else {
      put_x(lx, row_x(i - 2), col_x(i - 2), v[set][i]);
    }
  }
  // e4m3 rows: the three parts of x to three places.
  __device__ __forceinline__ void store_parts(int set, int i, char *ly, char *lx) const {
    if (i < 2) {
      *(u32x4 *)(ly + row_y(i) * kStrideY + col_y(i) * 2) = v[set][i];
      return;
    }
    const u32x4 c = v[set][i];
    const float s = scale[set][i - 2];
#pragma unroll
    for (int half = 0; half < 2; ++half) {  // eight values
      u32x4 w[3];
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const f32x2 q = (d & 1) == 0 ? __builtin_amdgcn_cvt_pk_f32_fp8((int)c[2 * half + (d >> 1)], false)
                                     : __builtin_amdgcn_cvt_pk_f32_fp8((int)c[2 * half + (d >> 1)], true);
        uint32_t lo[3], hi[3];
        three_parts(q[0] * s, lo);
        three_parts(q[1] * s, hi);
#pragma unroll
        for (int t = 0; t < 3; ++t) w[t][d] = upper_halves(lo[t], hi[t]);
      }
#pragma unroll
      for (int t = 0; t < 3; ++t) put_x(lx + t * (kRows * kStrideX), row_x(i - 2), col_x(i - 2) + 8 * half, w[t]);
    }
  }
};

template <bool FP8, bool FP32>
__global__ __launch_bounds__(kThreads, 2) void ep_expert_wgrad_tiles(
    const char *__restrict__ dy, const char *__restrict__ x, const float *__restrict__ x_scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int64_t capacity, int N,
    int H, int tiles_h, int tiles, int share, int64_t units, const char *previous, char *dw) {
  using Rows = Stage<FP8>;
  constexpr int kPieces = Rows::kPieces, kElt = FP32 ? 4 : 2;
  constexpr int kTilesQ = kTileH / 32;  // 16-column tiles of x per wave
  constexpr int kStepBytes = kRows * (kStrideY + kStrideX);
  constexpr int kLdsBytes = FP8 ? kRows * (kStrideY + 3 * kStrideX) : 2 * kStepBytes;  // two steps, or one in parts
  static_assert(kLdsBytes >= 2 * kStepBytes && kThreads / kWave * 16 * kStrideOut <= kLdsBytes,
                "every use fits the LDS, two workgroups a compute unit");
  __shared__ __attribute__((aligned(16))) char lds[kLdsBytes];
  const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wn = (wave & 1) * 64, wh = (wave >> 1) * (kTileH / 2);
  // where this lane's pieces of a step's transposed reads lie: row g * 4 + r16 / 4 (and 16 below it)
  const int row = g * 4 + (r16 >> 2);
  const int at_y = row * kStrideY + wn * 2 + (r16 & 3) * 8;
  const int at_x = kRows * kStrideY + row * kStrideX + wh / 2 + (r16 & 1) * 2 * kPlaneX + (r16 >> 1 & 1) * 8;
  // Whether some scale was not for the direct conversion, in the first step and in a later one: two sets
  // in turn, so that one is cleared while no wave can still read or write it.
  __shared__ int indirect[2][2];
  int turn = 0;
  if constexpr (FP8) {
    if (threadIdx.x < 4) indirect[threadIdx.x >> 1][threadIdx.x & 1] = 0;
    __syncthreads();
  }
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    // Workgroup u runs on XCD u % 8: each XCD takes one eighth of every expert's tiles, so what
    // they share of dy and x is in its own L2, whatever the experts' sizes.
    const int64_t k = u / kXcds;
    const int e = (int)(k / share), t = (int)(u % kXcds) * share + (int)(k % share);
    if (t >= tiles) continue;
    const int n0 = t / tiles_h * kTileN, h0 = t % tiles_h * kTileH;
    int64_t begin = 0;
    int count = (int)capacity;
    if (counts != nullptr) {
      int first = __builtin_amdgcn_readfirstlane(offsets[e]);
      count = clip_span(first, __builtin_amdgcn_readfirstlane(counts[e]), capacity);
      begin = first;
    }
    f32x4 acc[4][kTilesQ];
    bool in_parts = false;  // the same in every wave
    if (count > 0) {
      Rows stage;
      stage.place(N, H, n0, h0);
      int left = count;
      const char *from_y = dy + begin * N * 2, *from_x = x + begin * H * (FP8 ? 1 : 2);
      const char *from_s = (const char *)(x_scales != nullptr ? x_scales + begin * (H / 128) : nullptr);
      const auto aim = [&] {  // at the next step
        stage.aim(from_y, from_x, from_s, left <= 0 ? 0 : (left < kRows ? left : kRows), N, H, x_scales != nullptr);
        left -= kRows;
        from_y += (int64_t)kRows * N * 2;
        from_x += (int64_t)kRows * H * (FP8 ? 1 : 2);
        if constexpr (FP8) from_s += (int64_t)kRows * (H / 128) * 4;
      };
      // Three steps ahead of the products: two steps on their way into registers, one in the
      // other half of LDS.
      aim();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) stage.load(0, i);
      aim();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) stage.load(1, i);
      aim();
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        stage.store(0, i, lds, lds + kRows * kStrideY);
        stage.load(0, i);
      }
      int *const seen = indirect[turn];
      if constexpr (FP8)
        if (stage.indirect) seen[0] = 1;
      __syncthreads();
      if constexpr (FP8) {
        turn ^= 1;  // every wave has left the last tile: its set is free
        if (threadIdx.x < 2) indirect[turn][threadIdx.x] = 0;
      }
      const auto step = [&](auto set, auto first) {  // products of the step in lds[set]
        if constexpr (FP8)
          if (stage.indirect) seen[1] = 1;  // in the steps stored so far; the last one stores rows behind the end
        aim();
        const char *sy = lds + set * kStepBytes + at_y, *sx = lds + set * kStepBytes + at_x;
        char *to = lds + (set ^ 1) * kStepBytes;
        // tile q holds, as row 4a + b, column 32 (q / 2) + 8a + 4 (q % 2) + b: two tiles give a
        // lane eight consecutive columns of a row of the gradient
        const auto column_x = [&](int q) {
          const char *at = sx + (q >> 1) * 16 + (q & 1) * kPlaneX;
          return column(at, at + 16 * kStrideX);
        };
        bf16x8 b[4], a[2];
#pragma unroll
        for (int p = 0; p < 4; ++p) b[p] = column(sy + p * 32, sy + p * 32 + 16 * kStrideY);
        a[0] = column_x(0);
#pragma unroll
        for (int q = 0; q < kTilesQ; ++q) {
          if (q < kTilesQ - 1) a[(q + 1) & 1] = column_x(q + 1);
          if (q < kPieces) {
            stage.store(set ^ 1, q, to, to + kRows * kStrideY);
            stage.load(set ^ 1, q);
          }
#pragma unroll
          for (int p = 0; p < 4; ++p)
            acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q & 1], b[p], first ? f32x4{0.f, 0.f, 0.f, 0.f} : acc[p][q], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
        __syncthreads();
      };
      constexpr std::integral_constant<int, 0> even{};
      constexpr std::integral_constant<int, 1> odd{};
      step(even, std::true_type());
      if constexpr (FP8) in_parts = __builtin_amdgcn_readfirstlane(seen[0]) != 0;
      if (!in_parts) {
        for (int rows = count - kRows; rows > 0; rows -= 2 * kRows) {
          step(odd, std::false_type());
          if (rows > kRows) step(even, std::false_type());
        }
        if constexpr (FP8) in_parts = __builtin_amdgcn_readfirstlane(seen[1]) != 0;
      }
    } else {
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < kTilesQ; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
    if constexpr (FP8) {
      if (in_parts) {  // again, with three products for every one: a step's parts of x side by side in LDS
        Rows stage;
        stage.place(N, H, n0, h0);
        int left = count;
        const char *from_y = dy + begin * N * 2, *from_x = x + begin * H;
        const char *from_s = (const char *)(x_scales + begin * (H / 128));
        const auto fetch = [&] {
          stage.aim(from_y, from_x, from_s, left <= 0 ? 0 : (left < kRows ? left : kRows), N, H, true);
#pragma unroll
          for (int i = 0; i < kPieces; ++i) stage.load(0, i);
          left -= kRows;
          from_y += (int64_t)kRows * N * 2;
          from_x += (int64_t)kRows * H;
          from_s += (int64_t)kRows * (H / 128) * 4;
        };
#pragma unroll
        for (int p = 0; p < 4; ++p)
#pragma unroll
          for (int q = 0; q < kTilesQ; ++q) acc[p][q] = f32x4{0.f, 0.f, 0.f, 0.f};
        fetch();
        for (int rows = count; rows > 0; rows -= kRows) {
#pragma unroll
          for (int i = 0; i < kPieces; ++i) stage.store_parts(0, i, lds, lds + kRows * kStrideY);
          __syncthreads();
          fetch();
          bf16x8 b[4];
#pragma unroll
          for (int p = 0; p < 4; ++p) b[p] = column(lds + at_y + p * 32, lds + at_y + p * 32 + 16 * kStrideY);
#pragma unroll 1
          for (int t = 0; t < 3; ++t) {
            const char *sx = lds + at_x + t * (kRows * kStrideX);
#pragma unroll
            for (int q = 0; q < kTilesQ; ++q) {
              const char *at = sx + (q >> 1) * 16 + (q & 1) * kPlaneX;
              const bf16x8 a = column(at, at + 16 * kStrideX);
#pragma unroll
              for (int p = 0; p < 4; ++p)
                acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[p], acc[p][q], 0, 0, 0);
              __builtin_amdgcn_sched_barrier(0);
            }
          }
          __syncthreads();
        }
      }
    }
    // Results leave as whole 128-byte lines: 16 rows of 64 columns at a time pass through LDS
    // (each wave its own part), from where 8 (bf16) or 16 lanes take a row. A wave's LDS accesses
    // keep their order; the fences keep the compiler's, which sees a lane read and write different places.
    char *const mine = lds + wave * 16 * kStrideOut;
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int n = n0 + wn + p * 16, rows = N - n < 16 ? N - n : 16;
      if (rows <= 0) break;
      const int64_t first = ((int64_t)e * N + n) * H * kElt;
      const __amdgpu_buffer_rsrc_t to = buffer_of(dw + first, (int64_t)(rows * H) * kElt);
      const __amdgpu_buffer_rsrc_t old = buffer_of(previous != nullptr ? previous + first : nullptr,
                                                   previous != nullptr ? (int64_t)(rows * H) * kElt : 0);
#pragma unroll
      for (int part = 0; part < kTilesQ / 4; ++part) {
#pragma unroll
        for (int q = 0; q < 4; ++q)
          *(f32x4 *)(mine + r16 * kStrideOut + (q >> 1) * 128 + g * 32 + (q & 1) * 16) = acc[p][part * 4 + q];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        constexpr int kLanes = FP32 ? 16 : 8, kPasses = 16 * kLanes / kWave;
        u32x4 was[kPasses];
        uint32_t off[kPasses];
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const int h = h0 + wh + part * 64 + lane % kLanes * (64 / kLanes);
          off[i] = h < H ? (uint32_t)((i * (kWave / kLanes) + lane / kLanes) * H + h) * kElt : kOutside;
          if (previous != nullptr) was[i] = __builtin_amdgcn_raw_buffer_load_b128(old, (int)off[i], 0, kNonTemporal);
        }
#pragma unroll
        for (int i = 0; i < kPasses; ++i) {
          const char *from = mine + (i * (kWave / kLanes) + lane / kLanes) * kStrideOut + lane % kLanes * (256 / kLanes);
          f32x4 lo = *(const f32x4 *)from;
          u32x4 w;
          if constexpr (FP32) {
            if (previous != nullptr) lo += __builtin_bit_cast(f32x4, was[i]);
            w = __builtin_bit_cast(u32x4, lo);
          } else {
            f32x4 hi = *(const f32x4 *)(from + 16);
            if (previous != nullptr) {
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                lo[2 * j] += __uint_as_float(was[i][j] << 16), lo[2 * j + 1] += __uint_as_float(was[i][j] & 0xFFFF0000u);
                hi[2 * j] += __uint_as_float(was[i][2 + j] << 16), hi[2 * j + 1] += __uint_as_float(was[i][2 + j] & 0xFFFF0000u);
              }
            }
            w = u32x4{pack(lo[0], lo[1]), pack(lo[2], lo[3]), pack(hi[0], hi[1]), pack(hi[2], hi[3])};
          }
          __builtin_amdgcn_raw_buffer_store_b128(w, to, (int)off[i], 0, kNonTemporal);
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      }
    }
    __syncthreads();
  }
}

template <bool FP8, bool FP32>
int wgrad_launch(const ExpertWgradArgs &a) {
  const int cap = stream_workgroup_limit(a.stream);
  const int tn = (a.N + kTileN - 1) / kTileN, th = (a.H + kTileH - 1) / kTileH;
  const int64_t tiles = (int64_t)tn * th;
  if (tiles > INT32_MAX / kXcds) return -2;
  const int share = (int)((tiles + kXcds - 1) / kXcds);
  const int64_t units = (int64_t)a.E * share * kXcds;
  const int64_t most = cap > 0 ? cap : (1 << 23);
  const unsigned blocks = (unsigned)(units < most ? units : most);
  ep_expert_wgrad_tiles<FP8, FP32><<<blocks, kThreads, 0, a.stream>>>(
      (const char *)a.dy, (const char *)a.x, a.x_scales, a.counts, a.offsets, a.capacity, a.N, a.H, th,
      (int)tiles, share, units, (const char *)a.previous, (char *)a.dw);
  return launch_status();
}

}  // namespace

int launch_expert_wgrad(const ExpertWgradArgs &a) {
  if (a.x_fp8) return a.fp32 ? wgrad_launch<true, true>(a) : wgrad_launch<true, false>(a);
  return a.fp32 ? wgrad_launch<false, true>(a) : wgrad_launch<false, false>(a);
}

}  // namespace ep
