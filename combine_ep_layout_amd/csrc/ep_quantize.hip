// Rows to 8-bit integers with one scale per row (ep_quantize_rows), and the
// same of the experts' gated activation (ep_swiglu_quantize), on gfx950.
#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

constexpr int kThreads = 256;
constexpr float kLeast = 0x1p-100f;
constexpr uint32_t kInfBits = 0x7F800000u;

template <bool FP32>
__device__ __forceinline__ float load_one(const void *x, int64_t at) {
  if constexpr (FP32) return ((const float *)x)[at];
  else return __uint_as_float((uint32_t)((const uint16_t *)x)[at] << 16);
}

template <bool FP32, bool GATED>
__device__ __forceinline__ float value(const void *x, int64_t row, int W, int c) {
  if constexpr (!GATED) return load_one<FP32>(x, row * W + c);
  const float g = load_one<FP32>(x, row * 2 * W + c), u = load_one<FP32>(x, row * 2 * W + W + c);
  if (g < kFarGate) return (float)(g * far_sigmoid(g) * u);
  return g * (1.0f / (1.0f + expf(-g))) * u;
}

template <bool FP32, bool GATED>
__global__ __launch_bounds__(kThreads) void ep_quantize(const QuantizeArgs a) {
  __shared__ uint32_t top;
  __shared__ int real;
  for (int64_t row = blockIdx.x; row < a.capacity; row += gridDim.x) {
    __syncthreads();
    if (threadIdx.x == 0) top = 0, real = a.counts == nullptr;
    __syncthreads();
    if (a.counts != nullptr)
      for (int e = threadIdx.x; e < a.E; e += kThreads)
        if (row >= a.offsets[e] && row < (int64_t)a.offsets[e] + a.counts[e]) real = 1;
    __syncthreads();
    if (!real) continue;
    uint32_t most = 0;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const uint32_t bits = __float_as_uint(value<FP32, GATED>(a.x, row, a.width, c)) & 0x7FFFFFFFu;
      most = bits > most ? bits : most;
    }
    atomicMax(&top, most);
    __syncthreads();
    const bool bad = top >= kInfBits;
    const float size = fmaxf(__uint_as_float(bad ? 0 : top), kLeast), by = bad ? 0.f : 127.0f / size;
    for (int c = threadIdx.x; c < a.width; c += kThreads) {
      const float v = bad ? 0.f : value<FP32, GATED>(a.x, row, a.width, c);
      ((int8_t *)a.codes)[row * a.width + c] = (int8_t)__double2int_rn((double)v * (double)by);
    }
    for (int c = threadIdx.x; c < a.scale_cols; c += kThreads)
      a.scales[row * a.scale_cols + c] = bad ? __builtin_nanf("") : size / 127.0f;
  }
}

}  // namespace

int launch_quantize(const QuantizeArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  const int64_t most = cap > 0 ? cap : 1 << 22;
  const unsigned grid = (unsigned)(a.capacity < most ? a.capacity : most);
  const auto run = [&](auto kernel) {
    kernel<<<grid, kThreads, 0, a.stream>>>(a);
    return launch_status();
  };
  if (a.fp32) return a.gated ? run(ep_quantize<true, true>) : run(ep_quantize<true, false>);
  return a.gated ? run(ep_quantize<false, true>) : run(ep_quantize<false, false>);
}

}  // namespace ep
