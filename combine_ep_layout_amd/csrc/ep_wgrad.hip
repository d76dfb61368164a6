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

constexpr int kThreads = 256;
constexpr int kTileN = 128, kTileH = 128, kRows = 32;
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

template <bool FP8, bool FP32>
__global__ __launch_bounds__(kThreads) void ep_expert_wgrad_tiles(
    const char *__restrict__ dy, const char *__restrict__ x, const float *__restrict__ x_scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int64_t capacity, int N,
    int H, int tiles_n, int tiles_h, int64_t units, const char *previous, char *dw) {
  __shared__ uint16_t ldy[kRows][kTileN + 8], lx[kRows][kTileH + 8];
  const int tid = threadIdx.x, lane = lane_id(), r16 = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid / kWave), wn = (wave & 1) * 64, wh = (wave >> 1) * 64;
  const int per_expert = tiles_n * tiles_h;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = (int)(u / per_expert), t = (int)(u - (int64_t)e * per_expert);
    const int n0 = t / tiles_h * kTileN, h0 = t % tiles_h * kTileH;
    int64_t begin = 0, count = capacity;
    if (counts != nullptr) {
      begin = offsets[e];
      count = counts[e];
      if (begin < 0 || begin >= capacity || count < 0) count = 0;
      else if (count > capacity - begin) count = capacity - begin;
    }
    f32x4 acc[4][4] = {};
    for (int64_t r0 = 0; r0 < count; r0 += kRows) {
      const int rows = (int)(count - r0 < kRows ? count - r0 : kRows);
      const __amdgpu_buffer_rsrc_t by = buffer_of(dy + (begin + r0) * N * 2, (int64_t)rows * N * 2);
      const __amdgpu_buffer_rsrc_t bx = buffer_of(x + (begin + r0) * H * (FP8 ? 1 : 2), (int64_t)rows * H * (FP8 ? 1 : 2));
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int c = tid + i * kThreads, r = c / 16, col = c % 16 * 8;
        const u32x4 v = __builtin_amdgcn_raw_buffer_load_b128(by, (int)(n0 + col < N ? (uint32_t)(r * N + n0 + col) * 2u : kOutside), 0, 0);
        *(u32x4 *)&ldy[r][col] = v;
        u32x4 w;
        if constexpr (FP8) {
          const bool in = h0 + col < H && r < rows;
          const u32x2 q = __builtin_amdgcn_raw_buffer_load_b64(bx, (int)(in ? (uint32_t)(r * H + h0 + col) : kOutside), 0, 0);
          const float s = x_scales != nullptr ? (in ? x_scales[(begin + r0 + r) * (H / 128) + (h0 + col) / 128] : 0.f) : 1.f;
#pragma unroll
          for (int d = 0; d < 2; ++d) {
            const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[d], false);
            const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)q[d], true);
            w[2 * d] = pack(a[0] * s, a[1] * s);
            w[2 * d + 1] = pack(b[0] * s, b[1] * s);
          }
        } else {
          w = __builtin_amdgcn_raw_buffer_load_b128(bx, (int)(h0 + col < H ? (uint32_t)(r * H + h0 + col) * 2u : kOutside), 0, 0);
        }
        *(u32x4 *)&lx[r][col] = w;
      }
      __syncthreads();
      bf16x8 a[4], b[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          // row 4a + b of tile q holds column 16a + 4q + b: a lane's results are then 16
          // consecutive columns of a row of the gradient
          a[q][i] = __builtin_bit_cast(__bf16, lx[g * 8 + i][wh + (r16 >> 2) * 16 + q * 4 + (r16 & 3)]);
          b[q][i] = __builtin_bit_cast(__bf16, ldy[g * 8 + i][wn + q * 16 + r16]);
        }
#pragma unroll
      for (int p = 0; p < 4; ++p)
#pragma unroll
        for (int q = 0; q < 4; ++q)
          acc[p][q] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(a[q], b[p], acc[p][q], 0, 0, 0);
    }
#pragma unroll
    for (int p = 0; p < 4; ++p) {
      const int n = n0 + wn + p * 16 + r16, h = h0 + wh + g * 16;
      if (n >= N) continue;
#pragma unroll
      for (int half = 0; half < 2; ++half) {  // eight columns at a time
        if (h + half * 8 >= H) continue;
        const int64_t at = ((int64_t)e * N + n) * H + h + half * 8;
        f32x4 lo = acc[p][2 * half], hi = acc[p][2 * half + 1];
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
  const int64_t units = (int64_t)a.E * tn * th;
  const int64_t most = cap > 0 ? cap : INT32_MAX;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  const auto run = [&](auto kernel) {
    kernel<<<blocks, kThreads, 0, a.stream>>>((const char *)a.dy, (const char *)a.x, a.x_scales, a.counts,
                                              a.offsets, a.capacity, a.N, a.H, tn, th, units,
                                              (const char *)a.previous, (char *)a.dw);
    return launch_status();
  };
  if (a.x_fp8) return a.fp32 ? run(ep_expert_wgrad_tiles<true, true>) : run(ep_expert_wgrad_tiles<true, false>);
  return a.fp32 ? run(ep_expert_wgrad_tiles<false, true>) : run(ep_expert_wgrad_tiles<false, false>);
}

}  // namespace ep
