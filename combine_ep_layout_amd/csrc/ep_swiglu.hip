// The experts' gated activation on the expand layout for gfx950, with an
// 8-bit checkpoint of its input for the backward pass, and that backward pass.
//
// Mathematics. A row is [gate | up], I values each. Forward:
//   h = gate * s(gate) * up,  s(z) = 1 / (1 + exp(-z)),
// and, per 128 values of the row, the checkpoint: the power of two
// scale = 2^p with the smallest p >= -126 that keeps the group's largest
// finite magnitude within 448, and the e4m3 codes of value / scale. With a
// power of two the division is exact and so is the value read back, so the
// codes are the only rounding (half a step, 2^-4 relative; 2^-10 of the scale
// below its smallest normal). An infinity or NaN becomes the code NaN and
// leaves the scale alone: e4m3 has no infinity and a saved 448 would hide it.
// Backward, with gate and up as the checkpoint gives them:
//   d_gate = dh * up * s * (1 + gate * (1 - s)),  d_up = dh * gate * s.
// All arithmetic in binary32, results rounded once.
//
// Measured on MI355X, 32768 rows of 2048 in bf16 with the checkpoint: 101 us
// forward, 126 backward (87 and 113 in the kernel, 5.4 TB/s); the pairs below
// compare two forms of one kernel as they stood when the choice was made.
//
// What bounds both is HBM: 6 to 8 bytes per value pair of bf16 rows and the
// checkpoint's 2.06. So: one pass, a lane takes eight channels (16-byte loads
// of gate and up), 16 lanes hold a scale group and find its maximum with four
// register rotations, no LDS. Which rows are real is known on the device only
// (counts, offsets): a workgroup takes a block of consecutive rows and marks
// its real ones in one 32-bit mask by cutting every expert's span with the
// block, one expert per thread; padding rows are neither read nor written.
#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr int kLane = 8;      // channels per lane
constexpr int kMaxRows = 32;  // rows per block: bits of the mask
constexpr int kCodePolicy = 2 | 16;  // nt, sc1

// 1 / (1 + exp(-z)) for z from kFarGate on. EXACT (binary32 rows) uses the accurate exponential and
// division; bf16 rows the hardware's exp2 and reciprocal, whose error (about
// 2^-22 for |z| below 8, 2^-19 at 80) is far below half a bf16 step.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (EXACT) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

__device__ __forceinline__ float least(const float (&v)[kLane]) {
  float m = v[0];
#pragma unroll
  for (int i = 1; i < kLane; ++i) m = fminf(m, v[i]);
  return m;
}

// Stores are non-temporal, those of 16-byte pieces that fill whole lines at
// device scope as well (95 against 104 us forward, 126 against 138 backward at
// prefill). Binary32 rows leave every second 16 bytes of a line to a second
// store, which device scope would send to memory in halves (50 against 15 us
// at 3000 rows of 1408): not there. Loads are plain (nt: 116 against 110 us).
template <bool FP32>
struct Row {  // eight consecutive values of a row of bf16 or binary32
  static constexpr int kElt = FP32 ? 4 : 2;
  static constexpr int kPolicy = FP32 ? 2 : 2 | 16;  // nt, sc1

  static __device__ __forceinline__ void load(const char *p, float (&v)[kLane]) {
    const u32x4 a = *(const u32x4 *)p;
    if constexpr (FP32) {
      const u32x4 b = *((const u32x4 *)p + 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = __uint_as_float(a[i]), v[4 + i] = __uint_as_float(b[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(a[i] << 16);
        v[2 * i + 1] = __uint_as_float(a[i] & 0xFFFF0000u);
      }
    }
  }
  static __device__ __forceinline__ void store(__amdgpu_buffer_rsrc_t to, uint32_t off,
                                               const float (&v)[kLane]) {
    u32x4 a, b;
    if constexpr (FP32) {
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = __float_as_uint(v[i]), b[i] = __float_as_uint(v[4 + i]);
      __builtin_amdgcn_raw_buffer_store_b128(b, to, (int)off + 16, 0, kPolicy);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const f32x2 f = {v[2 * i], v[2 * i + 1]};
        a[i] = __builtin_bit_cast(uint32_t, __builtin_convertvector(f, bf16x2));
      }
    }
    __builtin_amdgcn_raw_buffer_store_b128(a, to, (int)off, 0, kPolicy);
  }
};

// Rows [r0, r0 + n) of an array of rows of `bytes` bytes.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t rows_of(const void *p, int64_t r0, int n, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc((char *)const_cast<void *>(p) + r0 * bytes, (short)0,
                                           (int)(n * bytes), kRawBufferFlags);
}

__device__ __forceinline__ float row_max(float v) {  // over the 16 lanes of a row
  constexpr int kRowRor = 0x120;
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kRowRor + 8, 0xF, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kRowRor + 4, 0xF, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kRowRor + 2, 0xF, 0xF, false)));
  v = fmaxf(v, __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kRowRor + 1, 0xF, 0xF, false)));
  return v;
}

// Eight e4m3 codes of v / 2^p for the group of the calling lane's 16-lane
// row, and 2^p. p from the maximum m * 2^x (1 <= m < 2): 448 is 1.75 * 2^8,
// so p = x - 8, or x - 7 where m > 1.75 (the added 0x1FFFFF carries into the
// exponent exactly then).
__device__ __forceinline__ u32x2 quantize(const float (&v)[kLane], float &scale) {
  float top = 0.f;
#pragma unroll
  for (int i = 0; i < kLane; ++i) {
    const float a = fabsf(v[i]);
    top = fmaxf(top, a < __builtin_inff() ? a : 0.f);
  }
  top = row_max(top);
  int p = (int)((__float_as_uint(top) + 0x1FFFFFu) >> 23) - 127 - 8;
  p = p < -126 ? -126 : p;
  scale = __uint_as_float((uint32_t)(p + 127) << 23);
  const float back = __uint_as_float((uint32_t)(127 - p) << 23);
  u32x2 codes;
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    float q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      q[i] = fabsf(v[4 * d + i]) < __builtin_inff() ? v[4 * d + i] * back : __builtin_nanf("");
    int c = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
    c = __builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], c, true);
    codes[d] = (uint32_t)c;
  }
  return codes;
}

__device__ __forceinline__ void dequantize(u32x2 codes, float scale, float (&v)[kLane]) {
#pragma unroll
  for (int d = 0; d < 2; ++d) {
    const f32x2 a = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[d], false);
    const f32x2 b = __builtin_amdgcn_cvt_pk_f32_fp8((int)codes[d], true);
    v[4 * d] = a[0] * scale, v[4 * d + 1] = a[1] * scale;
    v[4 * d + 2] = b[0] * scale, v[4 * d + 3] = b[1] * scale;
  }
}

// Bit r set: row r0 + r (r < n <= 32) lies in some expert's span. All threads
// of the workgroup call it.
__device__ __forceinline__ uint32_t real_rows(const int32_t *__restrict__ counts,
                                              const int32_t *__restrict__ offsets, int E, int64_t r0,
                                              int n, uint32_t *lds) {
  const uint32_t all = n == 32 ? ~0u : (1u << n) - 1;
  if (counts == nullptr) return all;
  __syncthreads();
  if (threadIdx.x == 0) *lds = 0;
  __syncthreads();
  for (int e = threadIdx.x; e < E; e += kThreads) {
    const int64_t b = offsets[e], end = b + counts[e];
    const int64_t lo = b > r0 ? b : r0, hi = end < r0 + n ? end : r0 + n;
    if (lo < hi) {
      const int len = (int)(hi - lo);
      atomicOr(lds, (len == 32 ? ~0u : (1u << len) - 1) << (int)(lo - r0));
    }
  }
  __syncthreads();
  return (uint32_t)__builtin_amdgcn_readfirstlane((int)*lds);
}

template <bool FP32, bool SAVE>
__global__ __launch_bounds__(kThreads) void ep_swiglu_rows(
    const char *__restrict__ gate_up, const int32_t *__restrict__ counts,
    const int32_t *__restrict__ offsets, int E, int64_t capacity, int I, int block_rows,
    int64_t blocks, FastDiv by_chunks, char *__restrict__ h, char *__restrict__ codes,
    float *__restrict__ scales) {
  __shared__ uint32_t lds;
  constexpr int kElt = Row<FP32>::kElt;
  const int chunks = I / kLane;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t r0 = b * block_rows;
    const int n = (int)(capacity - r0 < block_rows ? capacity - r0 : block_rows);
    const uint32_t real = real_rows(counts, offsets, E, r0, n, &lds);
    if (real == 0) continue;
    const __amdgpu_buffer_rsrc_t to_h = rows_of(h, r0, n, (int64_t)I * kElt);
    const __amdgpu_buffer_rsrc_t to_codes = SAVE ? rows_of(codes, r0, n, 2 * (int64_t)I) : to_h;
    for (uint32_t c = threadIdx.x; c < (uint32_t)(n * chunks); c += kThreads) {
      const uint32_t r = fast_div_apply(c, by_chunks), i = (c - r * (uint32_t)chunks) * kLane;
      if (!(real >> r & 1)) continue;
      const int64_t row = r0 + r;
      float g[kLane], u[kLane], v[kLane];
      Row<FP32>::load(gate_up + (row * 2 * I + i) * kElt, g);
      Row<FP32>::load(gate_up + (row * 2 * I + I + i) * kElt, u);
#pragma unroll
      for (int q = 0; q < kLane; ++q) v[q] = g[q] * sigmoid<FP32>(g[q]) * u[q];
      if (least(g) < kFarGate) {
#pragma unroll
        for (int q = 0; q < kLane; ++q)
          if (g[q] < kFarGate) v[q] = (float)(g[q] * far_sigmoid(g[q]) * u[q]);
      }
      Row<FP32>::store(to_h, (r * I + i) * kElt, v);
      if constexpr (SAVE) {
        float sg, su;
        const u32x2 cg = quantize(g, sg), cu = quantize(u, su);
        __builtin_amdgcn_raw_buffer_store_b64(cg, to_codes, (int)(r * 2 * I + i), 0, kCodePolicy);
        __builtin_amdgcn_raw_buffer_store_b64(cu, to_codes, (int)(r * 2 * I + I + i), 0, kCodePolicy);
        if ((threadIdx.x & 15) == 0) {
          float *st = scales + row * (2 * I / 128) + i / 128;
          st[0] = sg;
          st[I / 128] = su;
        }
      }
    }
  }
}

// h may be dh, so neither is __restrict__: a thread loads its channels of dh before it stores h there.
template <bool FP32, bool WITH_H>
__global__ __launch_bounds__(kThreads) void ep_swiglu_backward_rows(
    const char *dh, const char *__restrict__ codes, const float *__restrict__ scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int E, int64_t capacity,
    int I, int block_rows, int64_t blocks, FastDiv by_chunks, char *__restrict__ d_gate_up, char *h) {
  __shared__ uint32_t lds;
  constexpr int kElt = Row<FP32>::kElt;
  const int chunks = I / kLane;
  for (int64_t b = blockIdx.x; b < blocks; b += gridDim.x) {
    const int64_t r0 = b * block_rows;
    const int n = (int)(capacity - r0 < block_rows ? capacity - r0 : block_rows);
    const uint32_t real = real_rows(counts, offsets, E, r0, n, &lds);
    if (real == 0) continue;
    const __amdgpu_buffer_rsrc_t to_d = rows_of(d_gate_up, r0, n, 2 * (int64_t)I * kElt);
    const __amdgpu_buffer_rsrc_t to_h = WITH_H ? rows_of(h, r0, n, (int64_t)I * kElt) : to_d;
    for (uint32_t c = threadIdx.x; c < (uint32_t)(n * chunks); c += kThreads) {
      const uint32_t r = fast_div_apply(c, by_chunks), i = (c - r * (uint32_t)chunks) * kLane;
      if (!(real >> r & 1)) continue;
      const int64_t row = r0 + r;
      const char *from = codes + row * 2 * I + i;
      const u32x2 cg = *(const u32x2 *)from;
      const u32x2 cu = *(const u32x2 *)(from + I);
      const float *sc = scales + row * (2 * I / 128) + i / 128;
      float d[kLane], g[kLane], u[kLane], dg[kLane], du[kLane], v[kLane];
      Row<FP32>::load(dh + (row * I + i) * kElt, d);
      dequantize(cg, sc[0], g);
      dequantize(cu, sc[I / 128], u);
      const auto near = [&](int q) {
        const float s = sigmoid<FP32>(g[q]), gs = g[q] * s;
        dg[q] = d[q] * u[q] * (s * (1.0f + g[q] * (1.0f - s)));
        du[q] = d[q] * gs;
        if constexpr (WITH_H) v[q] = gs * u[q];
      };
      const auto far = [&](int q) {
        const double s = far_sigmoid(g[q]), gs = g[q] * s;
        dg[q] = (float)(s * u[q] * d[q] * (1.0 + g[q] * (1.0 - s)));
        du[q] = (float)(gs * d[q]);
        if constexpr (WITH_H) v[q] = (float)(gs * u[q]);
      };
      if (least(g) < kFarGate) {
#pragma unroll
        for (int q = 0; q < kLane; ++q) g[q] < kFarGate ? far(q) : near(q);
      } else {
#pragma unroll
        for (int q = 0; q < kLane; ++q) near(q);
      }
      Row<FP32>::store(to_d, (r * 2 * I + i) * kElt, dg);
      Row<FP32>::store(to_d, (r * 2 * I + I + i) * kElt, du);
      if constexpr (WITH_H) Row<FP32>::store(to_h, (r * I + i) * kElt, v);
    }
  }
}

struct RowGrid {
  int block_rows;
  int64_t blocks;
  unsigned launch;
};
// Rows per block: about two chunks of eight channels for every thread, and an
// odd number, which spreads the blocks that run together over the memory's
// channels (at prefill, rows of 8 KB: 3 rows 88 us forward and 119 backward, 2
// rows 95 and 126, 8 rows 101 and 134), as long as there are still eight
// workgroups for every compute unit.
RowGrid row_grid(int64_t capacity, int chunks, int cap) {
  int64_t rows = 2 * kThreads / chunks | 1;
  if (rows > capacity / 2048) rows = capacity / 2048;
  rows = rows < 1 ? 1 : (rows < kMaxRows ? rows : kMaxRows);
  const int64_t blocks = (capacity + rows - 1) / rows;
  const int64_t most = cap > 0 ? cap : (1 << 22);
  return {(int)rows, blocks, (unsigned)(blocks < most ? blocks : most)};
}

}  // namespace

int launch_swiglu(const SwigluArgs &a) {
  if (a.capacity == 0) return 0;
  const RowGrid g = row_grid(a.capacity, a.I / kLane, stream_workgroup_limit(a.stream));
  const FastDiv by = fast_div((uint32_t)(a.I / kLane));
  const auto run = [&](auto kernel) {
    kernel<<<g.launch, kThreads, 0, a.stream>>>((const char *)a.gate_up, a.counts, a.offsets, a.E,
                                                a.capacity, a.I, g.block_rows, g.blocks, by,
                                                (char *)a.h, (char *)a.codes, a.scales);
    return launch_status();
  };
  if (a.fp32) return a.codes ? run(ep_swiglu_rows<true, true>) : run(ep_swiglu_rows<true, false>);
  return a.codes ? run(ep_swiglu_rows<false, true>) : run(ep_swiglu_rows<false, false>);
}

int launch_swiglu_backward(const SwigluBackwardArgs &a) {
  if (a.capacity == 0) return 0;
  const RowGrid g = row_grid(a.capacity, a.I / kLane, stream_workgroup_limit(a.stream));
  const FastDiv by = fast_div((uint32_t)(a.I / kLane));
  const auto run = [&](auto kernel) {
    kernel<<<g.launch, kThreads, 0, a.stream>>>(
        (const char *)a.dh, (const char *)a.codes, a.scales, a.counts, a.offsets, a.E, a.capacity,
        a.I, g.block_rows, g.blocks, by, (char *)a.d_gate_up, (char *)a.h);
    return launch_status();
  };
  if (a.fp32)
    return a.h ? run(ep_swiglu_backward_rows<true, true>) : run(ep_swiglu_backward_rows<true, false>);
  return a.h ? run(ep_swiglu_backward_rows<false, true>) : run(ep_swiglu_backward_rows<false, false>);
}

}  // namespace ep
