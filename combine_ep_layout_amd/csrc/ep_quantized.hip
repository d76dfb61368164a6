// The experts' products in 8-bit integers on the expand layout for gfx950:
// y[r, n] = x_scales[r] * w_scales[e, n] * sum over k of x[r, k] w[e, n, k].
#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kThreads = 256;
constexpr uint32_t kOutside = 0x80000000u;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
}
__device__ __forceinline__ i32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0));
}

// A wave takes 16 rows by 16 channels, four waves 64 channels.
__global__ __launch_bounds__(kThreads) void ep_quantized_matmul_tiles(const QuantizedMatmulArgs a, int tiles_n,
                                                                      int64_t units) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int e = (int)(u / tiles_n), n0 = (int)(u % tiles_n) * 64 + wave * 16;
    int begin = 0, count = (int)a.capacity;
    if (a.counts != nullptr) {
      begin = __builtin_amdgcn_readfirstlane(a.offsets[e]);
      count = clip_span(begin, __builtin_amdgcn_readfirstlane(a.counts[e]), a.capacity);
    }
    const __amdgpu_buffer_rsrc_t w = buffer_of((const char *)a.w + (int64_t)e * a.N * a.K, (int64_t)a.N * a.K);
    const uint32_t wrow = n0 + r < a.N ? (uint32_t)(n0 + r) * (uint32_t)a.K : kOutside;
    for (int m0 = 0; m0 < count; m0 += 16) {
      const int rows = count - m0 < 16 ? count - m0 : 16;
      const int64_t first = (int64_t)begin + m0;
      const __amdgpu_buffer_rsrc_t x = buffer_of((const char *)a.x + first * a.K, (int64_t)rows * a.K);
      i32x4 acc = {0, 0, 0, 0};
      for (int k = 0; k < a.K; k += 64) {
        const bool in = k + g * 16 < a.K;
        const i32x4 av = load16(w, in ? wrow + (uint32_t)(k + g * 16) : kOutside);
        const i32x4 bv = load16(x, in && r < rows ? (uint32_t)r * (uint32_t)a.K + (uint32_t)(k + g * 16) : kOutside);
        acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(av, bv, acc, 0, 0, 0);
      }
      if (r >= rows) continue;
      const float sx = a.x_scales[(first + r) * a.x_scale_cols];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int n = n0 + g * 4 + i;
        if (n >= a.N) continue;
        const float v = (float)acc[i] * sx * a.w_scales[(int64_t)e * a.N + n];
        if (a.fp32) ((float *)a.y)[(first + r) * a.N + n] = v;
        else ((__bf16 *)a.y)[(first + r) * a.N + n] = (__bf16)v;
      }
    }
  }
}

}  // namespace

int launch_quantized_matmul(const QuantizedMatmulArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  const int tiles_n = (a.N + 63) / 64;
  const int64_t units = (int64_t)a.E * tiles_n, most = cap > 0 ? cap : 1 << 22;
  ep_quantized_matmul_tiles<<<(unsigned)(units < most ? units : most), kThreads, 0, a.stream>>>(a, tiles_n, units);
  return launch_status();
}

}  // namespace ep
