// The experts' weight gradient on the expand layout for gfx950:
// dW[e] = sum over the rows r of expert e of dy[r]^T x[r] (+ previous).
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
constexpr int kStrideY = kTileN * 2 + 32, kStrideX = kTileH * 2 + 64;  // LDS bytes per row
constexpr int kXcds = 8;
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
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

// One step's rows on the way from memory to LDS, in a thread's registers.
template <bool FP8>
struct Stage {
  u32x4 y[2], x[FP8 ? 2 : 4];
  float scale[2];

  // rows [row, row + rows) of the buffers (rows beyond read as zeros)
  __device__ __forceinline__ void load(const char *dy, const char *xs, const float *x_scales,
                                       int64_t row, int rows, int N, int H, int n0, int h0) {
    const int tid = threadIdx.x;
    const __amdgpu_buffer_rsrc_t by = buffer_of(dy + row * N * 2, (int64_t)rows * N * 2);
    const __amdgpu_buffer_rsrc_t bx = buffer_of(xs + row * H * (FP8 ? 1 : 2), (int64_t)rows * H * (FP8 ? 1 : 2));
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = tid + i * kThreads, r = c / (kTileN / 8), n = n0 + c % (kTileN / 8) * 8;
      y[i] = __builtin_amdgcn_raw_buffer_load_b128(by, (int)(n < N ? ((uint32_t)r * N + n) * 2u : kOutside), 0, 0);
    }
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = tid + i * kThreads, r = c / (kTileH / 16), h = h0 + c % (kTileH / 16) * 16;
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(bx, (int)(h < H ? (uint32_t)r * H + h : kOutside), 0, 0);
        scale[i] = 1.0f;
        if (x_scales != nullptr) {
          const __amdgpu_buffer_rsrc_t bs = buffer_of(x_scales + row * (H / 128), (int64_t)rows * (H / 128) * 4);
          scale[i] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              bs, (int)(h < H ? ((uint32_t)r * (H / 128) + h / 128) * 4u : kOutside), 0, 0));
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = tid + i * kThreads, r = c / (kTileH / 8), h = h0 + c % (kTileH / 8) * 8;
        x[i] = __builtin_amdgcn_raw_buffer_load_b128(bx, (int)(h < H ? ((uint32_t)r * H + h) * 2u : kOutside), 0, 0);
      }
    }
  }

  // 16 bytes of row r; rows 4 to 7 of eight have their 8-byte halves swapped
  static __device__ __forceinline__ void put_x(char *lx, int r, int h, u32x4 v) {
    if (r & 4) v = __builtin_shufflevector(v, v, 2, 3, 0, 1);
    *(u32x4 *)(lx + r * kStrideX + h * 2) = v;
  }
  __device__ __forceinline__ void store(char *ly, char *lx) const {
    const int tid = threadIdx.x;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int c = tid + i * kThreads;
      *(u32x4 *)(ly + c / (kTileN / 8) * kStrideY + c % (kTileN / 8) * 16) = y[i];
    }
    if constexpr (FP8) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = tid + i * kThreads, r = c / (kTileH / 16), h = c % (kTileH / 16) * 16;
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          u32x4 w;
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i][half * 2 + d], false);
            const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)x[i][half * 2 + d], true);
            w[2 * d] = pack(a[0] * scale[i], a[1] * scale[i]);
            w[2 * d + 1] = pack(b[0] * scale[i], b[1] * scale[i]);
          }
          put_x(lx, r, h + half * 8, w);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int c = tid + i * kThreads;
        put_x(lx, c / (kTileH / 8), c % (kTileH / 8) * 8, x[i]);
      }
    }
  }
};

template <bool FP8, bool FP32>
__global__ __launch_bounds__(kThreads, 2) void ep_expert_wgrad_tiles(
    const char *__restrict__ dy, const char *__restrict__ x, const float *__restrict__ x_scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int64_t capacity, int N,
    int H, int tiles_h, int tiles, int share, int64_t units, const char *previous, char *dw) {
  __shared__ __attribute__((aligned(16))) char ly[2][kRows * kStrideY], lx[2][kRows * kStrideX];
  const int lane = lane_id(), r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int wn = (wave & 1) * 64, wh = (wave >> 1) * 128;
  // where this lane's pieces of a step's transposed reads lie: row g * 4 + r16 / 4 (and 16 below it)
  const int row = g * 4 + (r16 >> 2);
  const int at_y = row * kStrideY + wn * 2 + (r16 & 3) * 8;
  const int at_x = row * kStrideX + wh * 2 + (r16 & 3) * 16, swap = (row & 4) * 2;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int64_t k = u / kXcds;
    const int e = (int)(k / share), t = (int)(u % kXcds) * share + (int)(k % share);
    if (t >= tiles) continue;
    const int n0 = t / tiles_h * kTileN, h0 = t % tiles_h * kTileH;
    int64_t begin = 0, count = capacity;
    if (counts != nullptr) {
      begin = offsets[e];
      count = counts[e];
      if (begin < 0 || begin >= capacity || count < 0) count = 0;
      else if (count > capacity - begin) count = capacity - begin;
    }
    f32x4 acc[4][8] = {};
    Stage<FP8> stage;
    const auto load = [&](int64_t r0) {
      stage.load(dy, x, x_scales, begin + r0, (int)(count - r0 < kRows ? count - r0 : kRows), N, H, n0, h0);
    };
    if (count > 0) load(0);
    int buf = 0;
    __syncthreads();
    for (int64_t r0 = 0; r0 < count; r0 += kRows, buf ^= 1) {
      stage.store(ly[buf], lx[buf]);
      __syncthreads();
      if (r0 + kRows < count) load(r0 + kRows);
      bf16x8 b[4];
#pragma unroll
      for (int p = 0; p < 4; ++p) {
        const char *at = ly[buf] + at_y + p * 32;
        b[p] = column(at, at + 16 * kStrideY);
      }
#pragma unroll
      for (int q = 0; q < 8; ++q) {
        // tile q holds, as row 4a + b, column 32 (q / 2) + 8a + 4 (q % 2) + b: two tiles give a
        // lane eight consecutive columns of a row of the gradient
        const char *at = lx[buf] + at_x + (q >> 1) * 64 + (((q & 1) * 8) ^ swap);
        const bf16x8 a = column(at, at + 16 * kStrideX);
#pragma unroll
        for (int p = 0; p < 4; ++p)
          acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b[p], acc[p][q], 0, 0, 0);
      }
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int n = n0 + wn + p * 16 + r16;
      if (n >= N) continue;
#pragma unroll
      for (int q = 0; q < 4; ++q) {  // eight columns at a time
        const int h = h0 + wh + q * 32 + g * 8;
        if (h >= H) continue;
        const int64_t at = ((int64_t)e * N + n) * H + h;
        f32x4 lo = acc[p][2 * q], hi = acc[p][2 * q + 1];
        if constexpr (FP32) {
          if (previous != nullptr) {
            lo += *(const f32x4 *)(previous + at * 4);
            hi += *(const f32x4 *)(previous + at * 4 + 16);
          }
          *(f32x4 *)(dw + at * 4) = lo;
          *(f32x4 *)(dw + at * 4 + 16) = hi;
        } else {
          if (previous != nullptr) {
            const u32x4 o = *(const u32x4 *)(previous + at * 2);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              lo[2 * i] += __uint_as_float(o[i] << 16), lo[2 * i + 1] += __uint_as_float(o[i] & 0xFFFF0000u);
              hi[2 * i] += __uint_as_float(o[2 + i] << 16), hi[2 * i + 1] += __uint_as_float(o[2 + i] & 0xFFFF0000u);
            }
          }
          const u32x4 v = {pack(lo[0], lo[1]), pack(lo[2], lo[3]), pack(hi[0], hi[1]), pack(hi[2], hi[3])};
          *(u32x4 *)(dw + at * 2) = v;
        }
      }
    }
  }
}

}  // namespace

int launch_expert_wgrad(const ExpertWgradArgs &a) {
  const int cap = stream_workgroup_limit(a.stream);
  const int tn = (a.N + kTileN - 1) / kTileN, th = (a.H + kTileH - 1) / kTileH;
  const int64_t tiles = (int64_t)tn * th;
  if (tiles > INT32_MAX / kXcds) return -2;
  const int share = (int)((tiles + kXcds - 1) / kXcds);
  const int64_t units = (int64_t)a.E * share * kXcds;
  const int64_t most = cap > 0 ? cap : (1 << 23);
  const unsigned blocks = (unsigned)(units < most ? units : most);
  const auto run = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, a.stream>>>((const char *)a.dy, (const char *)a.x, a.x_scales, a.counts,
                                              a.offsets, a.capacity, a.N, a.H, th, (int)tiles, share,
                                              units, (const char *)a.previous, (char *)a.dw);
    return launch_status();
  };
  if (a.x_fp8) return a.fp32 ? run(ep_expert_wgrad_tiles<true, true>) : run(ep_expert_wgrad_tiles<true, false>);
  return a.fp32 ? run(ep_expert_wgrad_tiles<false, true>) : run(ep_expert_wgrad_tiles<false, false>);
}

}  // namespace ep
