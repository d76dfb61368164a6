// Rows to 8-bit integers with one scale per row (ep_quantize_rows), and the
// same of the experts' gated activation (ep_swiglu_quantize), on gfx950.
//
// Mathematics. With a = max(2^-100, largest |v| of the row): scale a / 127,
// code rint(v * r), r = 127 / a in binary32. fma(v, r, 1.5 * 2^23) rounds the
// exact product once, to an integer with halves to even, and leaves the code
// in its low byte, so the codes are exactly determined. (v / scale, or a product rounded
// first, would put halves, such as half the largest value, on either side.) A
// row with an infinity or NaN, found as an integer maximum of the magnitudes' bits at or above
// infinity's, gets scale NaN and codes 0.
//
// What bounds it is HBM: each value read once, a byte written. So a row stays
// in the registers of one wave (or of four), which has all its loads in flight at
// once and needs no second pass; rows too wide for that are read twice.
// Rows of experts are counted through without their padding, by prefix sums that every workgroup makes for itself.
// Measured on MI355X: 32768 bf16 rows of 7168 for 256 experts 125 us (5.6 TB/s), among as much padding 128
// (workgroups of fixed rows of the buffer, which find out whether these are padding: 124 and 139; 8192 rows
// among four times as much 66 instead of 37), 4096 without experts 14.7; the activation of 32768 rows of 2048
// among padding 61 us (5.5 TB/s).
#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kLane = 8;                     // values of a lane per chunk
constexpr int kChunk = kWave * kLane;        // values of a wave per chunk
constexpr int kMaxRows = 32;                 // rows per block
constexpr float kLeast = 0x1p-100f;
constexpr uint32_t kInfBits = 0x7F800000u;
constexpr int kNonTemporal = 2;  // cache policy of the codes' stores (plain: 5% slower)

// 1 / (1 + exp(-z)) for z from kFarGate on, as ep_swiglu has it.
template <bool EXACT>
__device__ __forceinline__ float sigmoid(float z) {
  if constexpr (EXACT) return 1.0f / (1.0f + expf(-z));
  else return __builtin_amdgcn_rcpf(1.0f + __expf(-z));
}

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *p, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), (short)0, (int)bytes, kRawBufferFlags);
}

// Eight consecutive values of a row as they are in memory; behind the row's end zeros.
template <bool FP32>
struct Raw {
  u32x4 w[FP32 ? 2 : 1];

  __device__ __forceinline__ void load(__amdgpu_buffer_rsrc_t from, uint32_t value) {
    const uint32_t off = value * (FP32 ? 4u : 2u);
    w[0] = __builtin_amdgcn_raw_buffer_load_b128(from, (int)off, 0, 0);
    if constexpr (FP32) w[1] = __builtin_amdgcn_raw_buffer_load_b128(from, (int)off + 16, 0, 0);
  }
  __device__ __forceinline__ float operator[](int i) const {
    if constexpr (FP32) return __uint_as_float(w[i >> 2][i & 3]);
    else return __uint_as_float(i & 1 ? w[0][i >> 1] & 0xFFFF0000u : w[0][i >> 1] << 16);
  }
};

// What a lane keeps of eight values: them, or the activation's.
template <bool FP32, bool GATED>
struct Values;
template <bool FP32>
struct Values<FP32, false> {
  Raw<FP32> v;
  // bits of the largest magnitude so far: two halves of bf16, or one binary32
  __device__ __forceinline__ void top(uint32_t &m) const {
#pragma unroll
    for (int i = 0; i < (FP32 ? 8 : 4); ++i) {
      if constexpr (FP32) {
        const uint32_t b = v.w[i >> 2][i & 3] & 0x7FFFFFFFu;
        m = b > m ? b : m;
      } else {
        const u16x2 b = __builtin_bit_cast(u16x2, v.w[0][i] & 0x7FFF7FFFu);
        m = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(b, __builtin_bit_cast(u16x2, m)));
      }
    }
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) {
    if constexpr (FP32) return m;
    return (m >> 16 > (m & 0xFFFFu) ? m >> 16 : m & 0xFFFFu) << 16;
  }
  __device__ __forceinline__ float operator[](int i) const { return v[i]; }
};
template <bool FP32>
struct Values<FP32, true> {
  float h[kLane];
  __device__ __forceinline__ void set(const Raw<FP32> &g, const Raw<FP32> &u) {
    float least = g[0];
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      h[i] = g[i] * sigmoid<FP32>(g[i]) * u[i];
      least = fminf(least, g[i]);
    }
    if (least < kFarGate) {
#pragma unroll
      for (int i = 0; i < kLane; ++i)
        if (g[i] < kFarGate) h[i] = (float)(g[i] * far_sigmoid(g[i]) * u[i]);
    }
  }
  __device__ __forceinline__ void top(uint32_t &m) const {
#pragma unroll
    for (int i = 0; i < kLane; ++i) {
      const uint32_t b = __float_as_uint(h[i]) & 0x7FFFFFFFu;
      m = b > m ? b : m;
    }
  }
  static __device__ __forceinline__ uint32_t bits(uint32_t m) { return m; }
  __device__ __forceinline__ float operator[](int i) const { return h[i]; }
};

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2) {
    const uint32_t o = (uint32_t)__shfl_xor((int)v, d);
    v = o > v ? o : v;
  }
  return v;
}

// The experts' rows in turn: ends[e] of them belong to experts up to e, and row q of them, if it is e's, is
// row q + shift[e] of the buffer. Returns their number; every workgroup does this for itself.
struct Spans {
  int ends[EP_MAX_EXPERTS], shift[EP_MAX_EXPERTS], wave_sums[kWaves];
};
__device__ __forceinline__ int find_spans(const QuantizeArgs &a, Spans &lds) {
  constexpr int kMost = EP_MAX_EXPERTS / kThreads;
  const int per = (a.E + kThreads - 1) / kThreads, first = threadIdx.x * per;
  int begin[kMost], len[kMost], own = 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    const bool there = i < per && first + i < a.E;
    begin[i] = there ? a.offsets[first + i] : 0, len[i] = there ? a.counts[first + i] : 0;
  }
#pragma unroll
  for (int i = 0; i < kMost; ++i) {
    len[i] = clip_span(begin[i], len[i], a.capacity);
    len[i] = len[i] > 0 ? len[i] : 0, own += len[i];
  }
  const int upto = wave_inclusive_scan(own), wave = threadIdx.x / kWave;
  if (lane_id() == kWave - 1) lds.wave_sums[wave] = upto;
  __syncthreads();
  int sum = upto - own, all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) all += lds.wave_sums[w], sum += w < wave ? lds.wave_sums[w] : 0;
#pragma unroll
  for (int i = 0; i < kMost; ++i)
    if (i < per && first + i < a.E) {
      lds.shift[first + i] = begin[i] - sum;
      sum += len[i];
      lds.ends[first + i] = sum;
    }
  __syncthreads();
  return __builtin_amdgcn_readfirstlane(all);
}

// A row per TEAM waves, C chunks of a wave in registers (C = 0: the row is read twice).
template <bool FP32, bool GATED, int TEAM, int C>
__global__ __launch_bounds__(kThreads) void ep_quantize(const QuantizeArgs a, int block_rows) {
  __shared__ Spans spans;
  __shared__ uint32_t tops[2][kWaves];
  constexpr int kTeams = kWaves / TEAM, kElt = FP32 ? 4 : 2;
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int team = wave / TEAM, member = wave % TEAM, W = a.width;
  const uint32_t lane_value = (uint32_t)(member * kChunk + lane * kLane);
  const int64_t rows = a.counts != nullptr ? find_spans(a, spans) : a.capacity;
  int turn = 0, expert = 0, shift = 0;  // the experts before `expert` have no row left
  int64_t until = a.counts != nullptr ? 0 : rows;  // rows before it are moved by `shift`
  for (int64_t q0 = (int64_t)blockIdx.x * block_rows; q0 < rows; q0 += (int64_t)gridDim.x * block_rows) {
    const int64_t behind = q0 + block_rows < rows ? q0 + block_rows : rows;
    for (int64_t q = q0 + team; q < behind; q += kTeams) {
      if (q >= until) {
        int left = kWave;
        while (left == kWave) {
          left = __builtin_popcountll(ballot(expert + lane < a.E && spans.ends[expert + lane] <= q));
          expert += left;
        }
        if (expert >= a.E) break;  // only if spans overlap
        shift = __builtin_amdgcn_readfirstlane(spans.shift[expert]), until = __builtin_amdgcn_readfirstlane(spans.ends[expert]);
      }
      const int64_t row = q + shift;
      if ((uint64_t)row >= (uint64_t)a.capacity) break;  // so too
      const int64_t bytes = (int64_t)W * kElt;
      const char *const from = (const char *)a.x + row * bytes * (GATED ? 2 : 1);
      const __amdgpu_buffer_rsrc_t first = buffer_of(from, bytes), second = GATED ? buffer_of(from + bytes, bytes) : first;
      const __amdgpu_buffer_rsrc_t to = buffer_of((char *)a.codes + row * W, W);
      Values<FP32, GATED> v[C > 0 ? C : 1];
      const auto load = [&](uint32_t at, Values<FP32, GATED> &x) {
        if constexpr (GATED) {
          Raw<FP32> g, u;
          g.load(first, at), u.load(second, at);
          x.set(g, u);
        } else {
          x.v.load(first, at);
        }
      };
      uint32_t m = 0;
      if constexpr (C > 0) {
        if constexpr (GATED) {
          Raw<FP32> g[C], u[C];
#pragma unroll
          for (int c = 0; c < C; ++c) {
            g[c].load(first, lane_value + c * (TEAM * kChunk));
            u[c].load(second, lane_value + c * (TEAM * kChunk));
          }
#pragma unroll
          for (int c = 0; c < C; ++c) v[c].set(g[c], u[c]);
        } else {
#pragma unroll
          for (int c = 0; c < C; ++c) load(lane_value + c * (TEAM * kChunk), v[c]);
        }
#pragma unroll
        for (int c = 0; c < C; ++c) v[c].top(m);
      } else {
        for (uint32_t at = lane_value; at < (uint32_t)W; at += TEAM * kChunk) {
          load(at, v[0]);
          v[0].top(m);
        }
      }
      m = wave_max(Values<FP32, GATED>::bits(m));
      if constexpr (TEAM > 1) {
        if (lane == 0) tops[turn][member] = m;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < TEAM; ++i) m = tops[turn][i] > m ? tops[turn][i] : m;
        turn ^= 1;  // the other set: a wave may still read this one
      }
      const bool bad = m >= kInfBits;
      const float size = fmaxf(__uint_as_float(m), kLeast);
      const float scale = bad ? __builtin_nanf("") : size / 127.0f, by = 127.0f / size;
      const auto store = [&](uint32_t at, const Values<FP32, GATED> &x) {
        uint32_t q[kLane];
#pragma unroll
        for (int i = 0; i < kLane; ++i) q[i] = __float_as_uint(__builtin_fmaf(x[i], by, 12582912.0f));
        u32x2 codes;
#pragma unroll
        for (int d = 0; d < 2; ++d)
          codes[d] = __builtin_amdgcn_perm(__builtin_amdgcn_perm(q[4 * d + 3], q[4 * d + 2], 0x0C0C0400u),
                                           __builtin_amdgcn_perm(q[4 * d + 1], q[4 * d], 0x0C0C0400u), 0x05040100u);
        if (bad) codes = u32x2{0, 0};
        __builtin_amdgcn_raw_buffer_store_b64(codes, to, (int)at, 0, kNonTemporal);
      };
      if constexpr (C > 0) {
#pragma unroll
        for (int c = 0; c < C; ++c) store(lane_value + c * (TEAM * kChunk), v[c]);
      } else {
        for (uint32_t at = lane_value; at < (uint32_t)W; at += TEAM * kChunk) {
          load(at, v[0]);
          store(at, v[0]);
        }
      }
      for (int c = member * kWave + lane; c < a.scale_cols; c += TEAM * kWave) a.scales[row * a.scale_cols + c] = scale;
    }
  }
}

template <bool FP32, bool GATED, int TEAM, int C>
int quantize_launch(const QuantizeArgs &a) {
  const int cap = stream_workgroup_limit(a.stream);
  // Rows per block: about 8 KB for every team (rows of 14 KB, one or eight: 124 and 135 us at prefill, of 512
  // bytes 17.5 and 13.4 for 65536), as long as there are eight workgroups for every compute unit.
  const int64_t row_bytes = (int64_t)a.width * (FP32 ? 4 : 2) * (GATED ? 2 : 1);
  int64_t rows = (row_bytes >= 8192 ? 1 : (row_bytes <= 1024 ? 8 : 8192 / row_bytes)) * (kWaves / TEAM);
  if (rows > a.capacity / 2048) rows = a.capacity / 2048;
  rows = rows < kWaves / TEAM ? kWaves / TEAM : (rows < kMaxRows ? rows : kMaxRows);
  int64_t blocks = (a.capacity + rows - 1) / rows;
  // With experts, of which the buffer may be half padding, half as many workgroups (as many, a third: 132 and 130
  // instead of 129 us for 32768 rows of 7168 among as much padding; 126, 129 and 126 without any).
  if (a.counts != nullptr && blocks > 2048) blocks = blocks / 2 > 2048 ? blocks / 2 : 2048;
  const int64_t most = cap > 0 ? cap : 1 << 22;
  ep_quantize<FP32, GATED, TEAM, C><<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, a.stream>>>(a, (int)rows);
  return launch_status();
}

// A lane keeps up to 64 registers of a row (as it came, or as binary32 results).
template <bool FP32, bool GATED>
int quantize_type(const QuantizeArgs &a) {
  constexpr int kMost = FP32 || GATED ? 8 : 16;
  const int chunks = (a.width + kChunk - 1) / kChunk;
  if (chunks <= 1) return quantize_launch<FP32, GATED, 1, 1>(a);
  if (chunks <= 2) return quantize_launch<FP32, GATED, 1, 2>(a);
  if (chunks <= 4) return quantize_launch<FP32, GATED, 1, 4>(a);
  if (chunks <= 8) return quantize_launch<FP32, GATED, 1, 8>(a);
  if (chunks <= kMost) return quantize_launch<FP32, GATED, 1, kMost>(a);
  if (chunks <= 4 * 4) return quantize_launch<FP32, GATED, kWaves, 4>(a);
  if (chunks <= 8 * 4) return quantize_launch<FP32, GATED, kWaves, 8>(a);
  if (chunks <= kMost * 4) return quantize_launch<FP32, GATED, kWaves, kMost>(a);
  return quantize_launch<FP32, GATED, kWaves, 0>(a);
}

}  // namespace

int launch_quantize(const QuantizeArgs &a) {
  if (a.capacity == 0) return 0;
  if (a.fp32) return a.gated ? quantize_type<true, true>(a) : quantize_type<true, false>(a);
  return a.gated ? quantize_type<false, true>(a) : quantize_type<false, false>(a);
}

}  // namespace ep
