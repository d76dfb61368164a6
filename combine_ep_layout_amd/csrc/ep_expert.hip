// The experts' products for a few rows on gfx950: per-expert matrix-vector
// products on the expand layout (ep_expert_matvec) and a whole expert layer
// in two launches (ep_moe_layer).
//
// Mathematics. For the rows r of expert e, y[r] = W[e] x[r]; the layer is
// h = silu(G x) * (U x) per (token, k), then out[t] = sum_k w[t, k] D h[t, k].
// Weights are bf16, or e4m3 / e2m1 values with one fp32 scale per 128 values
// of a row; then a group's 128 products are summed first and the sum is
// scaled (the codes are exact in bf16, so no weight is ever rounded).
//
// What bounds it: with a few tokens per expert every weight is used a few
// times, so the time is that of reading the active experts' weights from HBM
// once. The products run on the matrix cores (16x16x32 bf16) all the same: a
// wave takes 16 weight rows per tile as one operand, from memory into registers
// (each row's 64 consecutive bytes go to four lanes), and 16 tokens as the
// other; lanes of absent tokens and rows are given an offset outside the
// buffer descriptor, which reads as 0 and costs no traffic. What carries it:
// loads a whole chunk ahead of the products and held there (the compiler,
// left alone, moves them down to their use: 503 against 355 us for a decode
// batch's fp4 products), 256 consecutive bytes of a row per chunk (64: 351
// against 255 us), the tokens' values through LDS once for four waves, and
// plain loads (non-temporal ones lose 5 to 30%: 53 against 41 us in the second
// launch of one token).
// Measured on MI355X: a bf16 layer of one token, top-8, hidden 7168,
// intermediate 2048 (705 MB of weights) 122 us, 5.8 TB/s; 128 tokens over 197
// active fp4 experts of 256 (4.6 GB) 1015 to 1050 us, 4.5 TB/s; fp4 products of 1024
// rows over 64 experts, 7168 to 4096 (1.0 GB) 212 to 216 us, 4.8 TB/s.
#include <type_traits>

#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset outside every descriptor (below 2^31 bytes)
constexpr int kTile = 16;                   // rows and tokens of one matrix instruction
constexpr int kStep = 128;                  // values of the long axis per step: one scale group
constexpr int kThreads = 256;
constexpr int kComputeUnits = 256;
constexpr int kWideTiles = 2;               // 16-row tiles per wave of the wide kernels

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
}
// The offset where `in`, else one outside every descriptor; arithmetic, because a choice between
// two offsets becomes a branch, and a value loaded in a branch is waited for at its end.
__device__ __forceinline__ uint32_t only(bool in, uint32_t off) { return off | (uint32_t)!in << 31; }
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0);
}
__device__ __forceinline__ float load4(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(b, (int)off, 0, 0));
}

// Value of `v` held by lane `from` (any lane's choice).
__device__ __forceinline__ float lane_value(float v, int from) {
  return __int_as_float(__builtin_amdgcn_ds_bpermute(from * 4, __float_as_int(v)));
}

// How the values of a step's 128 reach the four matrix instructions of the
// step: 16-byte loads per lane and step, and the place inside the step of the
// eight values that lane group g (lane / 16) brings to instruction j. Any
// order does, as long as both operands follow it; this one keeps each weight
// load 16 consecutive bytes.
template <int WT>
struct Weights;
template <>
struct Weights<EP_BF16> {
  static constexpr int kLoads = 4, kStepBytes = 256;
  static constexpr bool kScaled = false;
  static __device__ __forceinline__ int place(int j, int g) { return j * 32 + g * 8; }
  static __device__ __forceinline__ uint32_t load_byte(int l, int g) { return l * 64 + g * 16; }
  static __device__ __forceinline__ bf16x8 operand(const u32x4 (&w)[4], int j) {
    return __builtin_bit_cast(bf16x8, w[j]);
  }
};
template <>
struct Weights<EP_FP8_E4M3> {
  static constexpr int kLoads = 2, kStepBytes = 128;
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ int place(int j, int g) {
    return (j >> 1) * 64 + g * 16 + (j & 1) * 8;
  }
  static __device__ __forceinline__ uint32_t load_byte(int l, int g) { return l * 64 + g * 16; }
  static __device__ __forceinline__ bf16x8 operand(const u32x4 (&w)[2], int j) {
    bf16x8 v;
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const uint32_t c = w[j >> 1][(j & 1) * 2 + d];
      const bf16x2 lo = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, false);
      const bf16x2 hi = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(c, 1.0f, true);
      v[4 * d] = lo[0], v[4 * d + 1] = lo[1], v[4 * d + 2] = hi[0], v[4 * d + 3] = hi[1];
    }
    return v;
  }
};
template <>
struct Weights<EP_FP4X2> {
  static constexpr int kLoads = 1, kStepBytes = 64;
  static constexpr bool kScaled = true;
  static __device__ __forceinline__ int place(int j, int g) { return g * 32 + j * 8; }
  static __device__ __forceinline__ uint32_t load_byte(int, int g) { return g * 16; }
  static __device__ __forceinline__ bf16x8 operand(const u32x4 (&w)[1], int j) {
    const uint32_t c = w[0][j];
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 1);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 2);
    const bf16x2 e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, 1.0f, 3);
    return bf16x8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
  }
};

// One expert's matrix as a wave sees it.
struct Matrix {
  __amdgpu_buffer_rsrc_t w, scales;
  int width;  // values per row
};

template <int WT>
__device__ __forceinline__ Matrix matrix_of(const void *w, const float *scales, int64_t e,
                                            int64_t rows, int width) {
  const int64_t bytes = rows * width * Weights<WT>::kStepBytes / kStep;
  Matrix m;
  m.w = buffer_of((const char *)w + e * bytes, bytes);
  m.width = width;
  if constexpr (Weights<WT>::kScaled) {
    const int64_t n = rows * (width / kStep);
    m.scales = buffer_of(scales + e * n, n * 4);
  } else {
    m.scales = m.w;
  }
  return m;
}

// Byte offsets of the rows row[rt] (negative: absent) in a matrix and in its scales.
template <int WT, int RT>
__device__ __forceinline__ void row_offsets(const Matrix &m, const int (&row)[RT], uint32_t (&wrow)[RT],
                                            uint32_t (&srow)[RT]) {
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const bool in = row[rt] >= 0;
    wrow[rt] = in ? (uint32_t)(((int64_t)row[rt] * m.width * Weights<WT>::kStepBytes) / kStep) : kOutside;
    srow[rt] = in ? (uint32_t)row[rt] * (uint32_t)(m.width / kStep) * 4u : kOutside;
  }
}

// Offset of load l of step s (outside from step s1 on, and behind a row whose
// width is no multiple of 128).
template <int WT>
__device__ __forceinline__ uint32_t weight_at(int width, uint32_t wrow, int s, int s1, int l, int g) {
  using W = Weights<WT>;
  const bool in = s < s1 && (W::kScaled || s * kStep + W::place(l, g) < width);
  return only(in, wrow + (uint32_t)s * W::kStepBytes + W::load_byte(l, g));
}

// 64 consecutive bytes of 16 weight rows, loaded with the lanes as the matrix
// instruction wants them, have neighbouring lanes in 16 different rows: 64
// accesses, one a cycle, for 1 KB (the address units were busy for 81% of the
// launches of a large layer). So four neighbouring lanes load a row's 64 bytes
// (16 accesses) and the values change lanes through 1 KB of LDS of the wave's
// own before their use: 16 bf16 experts of 64 rows, 2048 to 1024, 40 against 51
// us; an fp4 layer's launches 640 and 500 against 680 and 595. The kernels that
// split the long axis are bound by latency and load as the instruction wants
// it. Lane l loads row l / 4 and the 16 bytes (l % 4) ^ (l / 16)
// of it, so that the 16 lanes that read one piece of every row use all banks.
__device__ __forceinline__ int near_row() { return lane_id() >> 2; }
__device__ __forceinline__ int near_piece() { return (lane_id() & 3) ^ (lane_id() >> 4); }
constexpr int kTurnBytes = kWave * 16;  // of LDS per wave
__device__ __forceinline__ u32x4 turn(char *slot, const u32x4 &v) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  *(u32x4 *)(slot + lane * 16) = v;  // a wave's LDS accesses keep their order
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  const u32x4 got = *(const u32x4 *)(slot + (r * 4 + (g ^ (r >> 2))) * 16);
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  return got;
}

// acc[rt] += rows x tokens over steps [s0, s1), a wave on its own. Lane
// (r = lane % 16, g = lane / 16): row[rt] is its weight row (negative:
// absent), tok the byte offset of its token's row in x (kOutside: absent). The
// tokens are the first operand, so a lane's four results are four tokens of
// one weight row and it needs one scale.
template <int WT, int RT>
struct Chunk {  // kSteps steps' operands on their way into registers
  using W = Weights<WT>;
  static constexpr int kSteps = W::kScaled ? 2 : 1;
  u32x4 w[kSteps][RT][W::kLoads], t[kSteps][4];
  float scale[RT];

  // Steps [s, s + kSteps), those from s1 on outside. Lane group g reads the scales of step s + g.
  __device__ __forceinline__ void load(const Matrix &m, const uint32_t (&wrow)[RT],
                                       const uint32_t (&srow)[RT], __amdgpu_buffer_rsrc_t x,
                                       uint32_t tok, int s, int s1) {
    const int g = lane_id() >> 4;
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int l = 0; l < W::kLoads; ++l)
          w[u][rt][l] = load16(m.w, weight_at<WT>(m.width, wrow[rt], s + u, s1, l, g));
    if constexpr (W::kScaled) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
        scale[rt] = load4(m.scales, only(g < kSteps && s + g < s1, srow[rt] + (uint32_t)(s + g) * 4u));
    }
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = (s + u) * kStep + W::place(j, g);
        const bool in = s + u < s1 && (W::kScaled || k < m.width);
        t[u][j] = load16(x, only(in, tok + (uint32_t)k * 2u));
      }
  }

  __device__ __forceinline__ void add(f32x4 (&acc)[RT]) const {
    const int r = lane_id() & 15;
#pragma unroll
    for (int u = 0; u < kSteps; ++u)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        f32x4 sum = acc[rt];
        if constexpr (W::kScaled) sum = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < 4; ++j)
          sum = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, t[u][j]),
                                                        W::operand(w[u][rt], j), sum, 0, 0, 0);
        if constexpr (W::kScaled) {
          const float sc = lane_value(scale[rt], u * 16 + r);
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[rt][i] += sc * sum[i];
        } else {
          acc[rt] = sum;
        }
      }
  }
};

template <int WT, int RT>
__device__ __forceinline__ void multiply(const Matrix &m, const int (&row)[RT],
                                         __amdgpu_buffer_rsrc_t x, uint32_t tok, int s0, int s1,
                                         f32x4 (&acc)[RT]) {
  constexpr int U = Chunk<WT, RT>::kSteps;
  uint32_t wrow[RT], srow[RT];
  row_offsets<WT>(m, row, wrow, srow);
  // Two chunks in turn: one on its way while the other is used. The barriers keep the compiler
  // from moving the loads down to their use to save registers.
  Chunk<WT, RT> a, b;
  a.load(m, wrow, srow, x, tok, s0, s1);
  for (int s = s0; s < s1; s += 2 * U) {
    b.load(m, wrow, srow, x, tok, s + U, s1);
    __builtin_amdgcn_sched_barrier(0);
    a.add(acc);
    __builtin_amdgcn_sched_barrier(0);
    if (s + U >= s1) break;
    a.load(m, wrow, srow, x, tok, s + 2 * U, s1);
    __builtin_amdgcn_sched_barrier(0);
    b.add(acc);
    __builtin_amdgcn_sched_barrier(0);
  }
}

// Sums the waves' partial tiles of one token tile through LDS: after it,
// red_sum(red, waves, RT, rt, tok, row) is the total. Callers synchronise
// before the next put.
template <int RT>
__device__ __forceinline__ void red_put(float *red, int wave, const f32x4 (&acc)[RT]) {
  const int lane = lane_id();
#pragma unroll
  for (int rt = 0; rt < RT; ++rt)
#pragma unroll
    for (int i = 0; i < 4; ++i) red[((wave * RT + rt) * 4 + i) * kWave + lane] = acc[rt][i];
}
template <int RT>
__device__ __forceinline__ float red_sum(const float *red, int waves, int rt, int tok, int row) {
  float v = 0.f;
  for (int w = 0; w < waves; ++w)
    v += red[((w * RT + rt) * 4 + (tok & 3)) * kWave + (tok >> 2) * kTile + row];
  return v;
}

// The same product for a workgroup of four waves with different rows and the
// same tokens, over the whole long axis: the tokens' values come through LDS,
// loaded once for all four waves, a chunk of 256 bytes of every weight row
// ahead of the products. near[rt] is the weight row that this lane loads
// (near_row of the tile; negative: absent).
template <int WT>
struct WideChunk {
  using W = Weights<WT>;
  static constexpr int kSteps = 256 / W::kStepBytes;  // per chunk
  static constexpr int kValues = kSteps * kStep, kPieces = kValues / 8;  // 16-byte pieces of a token
  static constexpr int kTokenBytes = kValues * 2;
};
template <int WT, int MT>
constexpr int wide_lds_bytes() {
  return 2 * MT * kTile * WideChunk<WT>::kTokenBytes + kThreads / kWave * kTurnBytes;
}

template <int WT, int RT, int MT>
__device__ __forceinline__ void multiply_wide(const Matrix &m, const int (&near)[RT],
                                              __amdgpu_buffer_rsrc_t x, const uint32_t *tok_off,
                                              char *lds, f32x4 (&acc)[MT][RT]) {
  using W = Weights<WT>;
  using C = WideChunk<WT>;
  constexpr int kMine = MT * kTile * C::kPieces / kThreads;  // pieces per thread
  const int tid = threadIdx.x, lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int steps = (m.width + kStep - 1) / kStep, chunks = (steps + C::kSteps - 1) / C::kSteps;
  uint32_t wrow[RT], srow[RT];
  row_offsets<WT>(m, near, wrow, srow);
  const int piece_of = near_piece(), step_of = lane & 3;
  char *const slot = lds + 2 * MT * kTile * C::kTokenBytes + tid / kWave * kTurnBytes;
  // A token's pieces are rotated by its number (exclusive or), so that 16 tokens' pieces of the
  // same place, which 16 lanes read at once, lie in different banks.
  uint32_t from[kMine];
  int piece[kMine];
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    const int at = tid + i * kThreads, t = at / C::kPieces;
    piece[i] = (at % C::kPieces) ^ (t & 15);
    from[i] = tok_off[t] + (uint32_t)piece[i] * 16u;
  }
  u32x4 xs[kMine], xs0[kMine], w[2][C::kSteps][RT][W::kLoads];
  float scale[2][RT];
  const auto load_x = [&](u32x4 (&to)[kMine], int c) {
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const bool in = W::kScaled ? c < chunks : c * C::kValues + piece[i] * 8 < m.width;
      to[i] = load16(x, only(in, from[i] + (uint32_t)c * C::kTokenBytes));
    }
  };
  const auto store_x = [&](const u32x4 (&v)[kMine], int c) {
#pragma unroll
    for (int i = 0; i < kMine; ++i)
      *(u32x4 *)(lds + (c & 1) * (MT * kTile * C::kTokenBytes) + (tid + i * kThreads) * 16) = v[i];
  };
  const auto load_w = [&](int c, auto set) {
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int u = 0; u < C::kSteps; ++u)
#pragma unroll
        for (int l = 0; l < W::kLoads; ++l)
          w[set][u][rt][l] = load16(m.w, weight_at<WT>(m.width, wrow[rt], c * C::kSteps + u, steps, l, piece_of));
      if constexpr (W::kScaled) {
        const int s = c * C::kSteps + step_of;
        scale[set][rt] = load4(m.scales, only(step_of < C::kSteps && s < steps, srow[rt] + (uint32_t)s * 4u));
      }
    }
  };
  const auto add = [&](int c, auto set) {
    const char *from_lds = lds + (c & 1) * (MT * kTile * C::kTokenBytes) + r * C::kTokenBytes;
#pragma unroll
    for (int u = 0; u < C::kSteps; ++u) {
      if (u > 0 && c * C::kSteps + u >= steps) break;
      u32x4 turned[RT][W::kLoads];
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int l = 0; l < W::kLoads; ++l) turned[rt][l] = turn(slot, w[set][u][rt][l]);
      f32x4 part[MT][RT];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        bf16x8 t[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          t[mt] = *(const bf16x8 *)(from_lds + mt * kTile * C::kTokenBytes +
                                    (((u * kStep + W::place(j, g)) / 8) ^ r) * 16);
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const bf16x8 b = W::operand(turned[rt], j);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt) {
            if constexpr (W::kScaled)
              part[mt][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                  t[mt], b, j == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : part[mt][rt], 0, 0, 0);
            else
              acc[mt][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t[mt], b, acc[mt][rt], 0, 0, 0);
          }
        }
      }
      if constexpr (W::kScaled) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) {
          const float sc = lane_value(scale[set][rt], r * 4 + u);
#pragma unroll
          for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 4; ++i) acc[mt][rt][i] += sc * part[mt][rt][i];
        }
      }
    }
  };
  constexpr std::integral_constant<int, 0> even{};
  constexpr std::integral_constant<int, 1> odd{};
  // Loads come back in order, so the tokens' are always issued before the weights': the wait for
  // them is then none for the weights of the next chunk (a large fp4 layer: 580 us, 640 with those mixed).
  const auto chunk = [&](int c, auto use, auto fill) {
    store_x(xs, c + 1);
    load_x(xs, c + 2);
    __builtin_amdgcn_sched_barrier(0);
    load_w(c + 1, fill);
    __builtin_amdgcn_sched_barrier(0);
    add(c, use);
    __syncthreads();
  };
  load_x(xs0, 0);
  load_x(xs, 1);
  __builtin_amdgcn_sched_barrier(0);
  load_w(0, even);
  __builtin_amdgcn_sched_barrier(0);
  store_x(xs0, 0);
  __syncthreads();
  for (int c = 0; c < chunks; c += 2) {
    chunk(c, even, odd);
    if (c + 1 >= chunks) break;
    chunk(c + 1, odd, even);
  }
}

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// ------------------------------------------------------------ ep_expert_matvec

// The j-th expert that has rows, found by every wave for itself from the
// counts (a ballot for every 64 experts); absent: e = -1. A span is cut to the
// rows that lie inside the buffer, so no access leaves it whatever the arrays
// hold.
struct Segment {
  int e;
  int64_t begin, count;
};
template <bool ALL = false>  // ALL: also the number of experts that have rows
__device__ __forceinline__ Segment find_segment(int j, const int32_t *__restrict__ counts,
                                                const int32_t *__restrict__ offsets, int E,
                                                int64_t capacity, int *have_rows = nullptr) {
  if (counts == nullptr) return {j == 0 ? 0 : -1, 0, capacity};
  const int lane = lane_id();
  Segment s{-1, 0, 0};
  int total = 0;
  for (int first = 0; first < E && (ALL || s.e < 0); first += 4 * kWave) {
    int begin[4], count[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int e = first + q * kWave + lane;
      begin[q] = e < E ? offsets[e] : 0;
      count[q] = e < E ? counts[e] : 0;
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      count[q] = clip_span(begin[q], count[q], capacity);
      const uint64_t have = ballot(count[q] > 0);
      const int n = __builtin_popcountll(have);
      if (s.e < 0 && j < n) {
        const int at = __builtin_ctzll(ballot((have >> lane & 1) != 0 && count_below(have) == j));
        s = {first + q * kWave + at, read_lane(begin[q], at), read_lane(count[q], at)};
      }
      j -= n;
      total += n;
    }
  }
  if constexpr (ALL) *have_rows = total;
  return s;
}

// Rows of all experts, each one's up to 2^16 of them.
__device__ __forceinline__ int rows_of_all(const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets,
                                           int E, int64_t capacity) {
  int mine = 0;
  for (int e = lane_id(); e < E; e += kWave) {
    int begin = offsets[e];
    const int n = clip_span(begin, counts[e], capacity);
    mine += n < 0 ? 0 : (n < 1 << 16 ? n : 1 << 16);
  }
  return wave_sum(mine);
}

template <int WT, int MT, bool FP32>
__device__ __forceinline__ void matvec_wide_group(const Matrix &m, const uint16_t *x, int64_t row0,
                                                  int rows, int n0, int N, void *y, char *lds,
                                                  uint32_t *tok_off) {
  constexpr int RT = kWideTiles;
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const __amdgpu_buffer_rsrc_t xb = buffer_of(x + row0 * m.width, (int64_t)rows * m.width * 2);
  if (threadIdx.x < MT * kTile)
    tok_off[threadIdx.x] = (int)threadIdx.x < rows ? threadIdx.x * (uint32_t)m.width * 2u : kOutside;
  __syncthreads();
  int row[RT], near[RT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int first = n0 + (wave * RT + rt) * kTile;
    row[rt] = first + r < N ? first + r : -1;
    near[rt] = first + near_row() < N ? first + near_row() : -1;
  }
  f32x4 acc[MT][RT] = {};
  multiply_wide<WT, RT, MT>(m, near, xb, tok_off, lds, acc);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = mt * kTile + g * 4 + i;
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        if (p >= rows || row[rt] < 0) continue;
        const int64_t at = (row0 + p) * (int64_t)N + row[rt];
        if constexpr (FP32) ((float *)y)[at] = acc[mt][rt][i];
        else ((uint16_t *)y)[at] = bf16_bits(acc[mt][rt][i]);
      }
    }
}

// The wide kernel reads x once for 128 rows and walks the whole long axis: right
// where its workgroups take most compute units (24 fp8 experts of 4 rows, 4096
// to 1024, 192 workgroups: 20 against 48 us; one fp4 row to 14336, 112: 23
// against 32; 12 experts of a row, 96: 17 against 19 in fp8, 21 against 20 in
// bf16), or a fifth of them and the split kernel would read every matrix again
// for each 16 of more rows (one bf16 expert of 64 rows, 7168 to 7168, 56
// workgroups: 83 against 114; 3 experts of 29, 39 workgroups: 34 against 35).
// Else waves that share the long axis are faster: one row of an fp4 matrix 7168
// to 4096 (32 workgroups) 10 against 25 us, 40 rows of it in fp8 41 against 60,
// 8 experts of a row, 4096 to 1024 in fp4 (64 workgroups) 11 against 15.
//
// How many experts have rows is known on the device only; the host knows at most
// how many can (no more than there are experts, or rows of the buffer). Where
// that bound is too low for the wide kernel the split kernel runs, else the wide
// kernel, which counts and takes 16 rows at a time itself if they are too few
// (its four waves sharing the long axis). Padding makes that common. At A = 16 or
// 128, one row each for 8 of 256 experts, 4096 to 512 in fp4: 8.8 us against 15.5
// with 128 rows at a time (7.0 at A = 1, where the bound is 8); 4096 to 1024 in
// fp8 14.1 against 18.4; 4 of 64 experts of 4 rows, 7168 to 512 in fp8, 11.0
// against 27. Counting costs full buffers up to 2% (256 fp8 experts of 4 rows,
// 1024 to 2048, 104 against 102).
__host__ __device__ constexpr bool matvec_is_wide(int64_t experts, int64_t rows, int tiles) {
  const int64_t units = experts * tiles;
  return units >= kComputeUnits * 3 / 8 || (units >= kComputeUnits / 5 && rows > kTile * experts);
}

// 16 rows of a matrix for all rows of its expert, the workgroup's waves sharing the long axis.
template <int WT, bool FP32>
__device__ __forceinline__ void matvec_split_unit(const uint16_t *x, const void *w, const float *scales,
                                                  const Segment &seg, int n0, int K, int N, void *y, float *red) {
  const int r = lane_id() & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int steps = (K + kStep - 1) / kStep;
  const Matrix m = matrix_of<WT>(w, scales, seg.e, N, K);
  const int row[1] = {n0 + r < N ? n0 + r : -1};
  for (int64_t p = 0; p < seg.count; p += kTile) {
    const int rows = (int)(seg.count - p < kTile ? seg.count - p : kTile);
    // rows beyond the group lie outside the descriptor
    const __amdgpu_buffer_rsrc_t xb = buffer_of(x + (seg.begin + p) * K, (int64_t)rows * K * 2);
    f32x4 acc[1] = {};
    multiply<WT, 1>(m, row, xb, r < rows ? (uint32_t)r * (uint32_t)K * 2u : kOutside, steps * wave / waves,
                    steps * (wave + 1) / waves, acc);
    red_put<1>(red, wave, acc);
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * kTile; i += blockDim.x) {
      const int c = i % kTile, q = i / kTile;
      if (q < rows && n0 + c < N) {
        const float v = red_sum<1>(red, waves, 0, q, c);
        const int64_t at = (seg.begin + p + q) * (int64_t)N + n0 + c;
        if constexpr (FP32) ((float *)y)[at] = v;
        else ((uint16_t *)y)[at] = bf16_bits(v);
      }
    }
    __syncthreads();
  }
}

// Few tiles: the 4 to 16 waves of a workgroup share 16 rows' long axis.
template <int WT, bool FP32>
__global__ __launch_bounds__(1024) void ep_expert_matvec_split(
    const uint16_t *__restrict__ x, const void *__restrict__ w, const float *__restrict__ scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int E,
    int64_t capacity, int K, int N, int64_t units, int tiles, void *__restrict__ y) {
  extern __shared__ float red[];
  int have_j = -1;
  Segment seg{-1, 0, 0};
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), n0 = (int)(u - (int64_t)j * tiles) * kTile;
    if (j != have_j) seg = find_segment(j, counts, offsets, E, capacity);
    have_j = j;
    if (seg.e < 0) return;  // no further expert has rows
    matvec_split_unit<WT, FP32>(x, w, scales, seg, n0, K, N, y, red);
  }
}

// Many tiles: a workgroup takes 128 rows of one expert's matrix, or where the experts with rows turn out
// to be too few for that, 16 as above.
template <int WT, bool FP32>
__global__ __launch_bounds__(kThreads, 2) void ep_expert_matvec_wide(
    const uint16_t *__restrict__ x, const void *__restrict__ w, const float *__restrict__ scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int E,
    int64_t capacity, int K, int N, int64_t units, int tiles, void *__restrict__ y) {
  __shared__ __attribute__((aligned(16))) char lds[wide_lds_bytes<WT, 2>()];
  __shared__ uint32_t tok_off[2 * kTile];
  int experts = 0;
  int have_j = (int)(blockIdx.x / tiles);
  Segment seg = find_segment<true>(have_j, counts, offsets, E, capacity, &experts);
  if (counts != nullptr && !matvec_is_wide(experts, 0, tiles) &&
      !matvec_is_wide(experts, rows_of_all(counts, offsets, E, capacity), tiles)) {
    const int tiles16 = (N + kTile - 1) / kTile;
    const int64_t units16 = (int64_t)experts * tiles16;
    have_j = -1;
    for (int64_t u = blockIdx.x; u < units16; u += gridDim.x) {
      const int j = (int)(u / tiles16), n0 = (int)(u - (int64_t)j * tiles16) * kTile;
      if (j != have_j) seg = find_segment(j, counts, offsets, E, capacity);
      have_j = j;
      matvec_split_unit<WT, FP32>(x, w, scales, seg, n0, K, N, y, (float *)lds);
    }
    return;
  }
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), n0 = (int)(u - (int64_t)j * tiles) * kWideTiles * kTile * 4;
    if (j != have_j) seg = find_segment(j, counts, offsets, E, capacity);
    have_j = j;
    if (seg.e < 0) return;  // no further expert has rows
    const Matrix m = matrix_of<WT>(w, scales, seg.e, N, K);
    for (int64_t p = 0; p < seg.count;) {
      const int64_t left = seg.count - p;
      const int rows = (int)(left < 2 * kTile ? left : 2 * kTile);
      if (rows > kTile)
        matvec_wide_group<WT, 2, FP32>(m, x, seg.begin + p, rows, n0, N, y, lds, tok_off);
      else
        matvec_wide_group<WT, 1, FP32>(m, x, seg.begin + p, rows, n0, N, y, lds, tok_off);
      p += rows;
    }
  }
}

// ---------------------------------------------------------------- ep_moe_layer
//
// First launch: workgroup (j, tile) finds the j-th expert that occurs in
// topk_idx and its entries by itself (n = T*K <= 1024 ids, no extra launch)
// and computes gate, up and h for 16 or 64 channels; h goes to the workspace
// as a high and a low bf16 part per value (2^-17 relative), so that the second
// product loses nothing to the rounding of h. The workgroups of tile 0 leave
// the list of active experts and their entries behind.
// Second launch: a workgroup owns up to 32 output channels of every token (an
// even share for 256 compute units: 28 of 7168); its waves take (expert, part
// of the long axis) units, the entries' results stay in LDS, and are summed
// with their router weights in k order, so the result is a pure function of
// the inputs. Beyond a few dozen entries h weighs as much as the weights, since
// every workgroup reads it whole: 465 us for 1024 entries over 197 fp4 experts
// (1.5 GB of weights).

struct MoeEntry {  // one active expert, packed: id, first place in the order, entries - 1
  uint32_t v;
  __device__ int e() const { return v & 1023; }
  __device__ int begin() const { return v >> 10 & 1023; }
  __device__ int count() const { return (int)(v >> 20) + 1; }
};

struct FindLds {
  int count[EP_MAX_EXPERTS];
  uint16_t entry[EP_MOE_MAX_ENTRIES];
  int wave_active[4], wave_entries[4];
  int same[EP_MOE_MAX_ENTRIES / kWave];  // entries of the expert in each 64 ids
  int e, before, have, active;
};

// The j-th active expert (first occurrence order for n <= 64, ascending id
// above): e or -1, its `have` entries in f.entry in ascending order (every
// workgroup of an expert has to place them alike), `before` entries of other
// experts ahead of it in the order, and the number of active experts. 256
// threads, ends synchronised.
__device__ __forceinline__ void find_expert(int j, const int32_t *__restrict__ topk_idx, int n, int E,
                                            FindLds &f) {
  const int tid = threadIdx.x, lane = lane_id(), wave = tid / kWave;
  if (n <= kWave) {
    if (wave == 0) {
      const int id = lane < n ? topk_idx[lane] : -1;
      const bool valid = id >= 0 && id < E;
      bool first = valid;
      for (int q = 0; q < n - 1; ++q)
        if (read_lane(id, q) == id && lane > q) first = false;
      const uint64_t firsts = ballot(first);
      const uint64_t at = ballot(first && count_below(firsts) == j);
      int e = -1, before = 0, have = 0;
      if (at != 0) {
        e = read_lane(id, __builtin_ctzll(at));
        const uint64_t same = ballot(id == e);
        if (id == e) f.entry[count_below(same)] = (uint16_t)lane;
        have = __builtin_popcountll(same);
        before = __builtin_popcountll(ballot(valid && id < e));
      }
      if (lane == 0)
        f.e = e, f.before = before, f.have = have, f.active = __builtin_popcountll(firsts);
    }
    __syncthreads();
    return;
  }
  for (int i = tid; i < EP_MAX_EXPERTS; i += kThreads) f.count[i] = 0;
  if (tid == 0) f.e = -1;
  __syncthreads();
  int id[EP_MOE_MAX_ENTRIES / kThreads];
#pragma unroll
  for (int q = 0; q < EP_MOE_MAX_ENTRIES / kThreads; ++q) {
    const int i = tid + q * kThreads;
    id[q] = i < n ? topk_idx[i] : -1;
    if (id[q] >= 0 && id[q] < E) atomicAdd(&f.count[id[q]], 1);
  }
  __syncthreads();
  int act = 0, ent = 0, c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = f.count[tid * 4 + i], act += c[i] > 0, ent += c[i];
  const int act_to = wave_inclusive_scan(act), ent_to = wave_inclusive_scan(ent);
  if (lane == kWave - 1) f.wave_active[wave] = act_to, f.wave_entries[wave] = ent_to;
  __syncthreads();
  int act_before = act_to - act, ent_before = ent_to - ent, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) act_before += f.wave_active[w], ent_before += f.wave_entries[w];
    total += f.wave_active[w];
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (c[i] > 0) {
      if (act_before == j) f.e = tid * 4 + i, f.before = ent_before, f.have = c[i];
      ++act_before;
    }
    ent_before += c[i];
  }
  if (tid == 0) f.active = total;
  __syncthreads();
  const int e = f.e;
  constexpr int kIds = EP_MOE_MAX_ENTRIES / kThreads, kWaves = kThreads / kWave;
  uint64_t same[kIds];
#pragma unroll
  for (int q = 0; q < kIds; ++q) {
    same[q] = ballot(e >= 0 && id[q] == e);
    if (lane == 0) f.same[q * kWaves + wave] = __builtin_popcountll(same[q]);
  }
  __syncthreads();
  int first = 0;
#pragma unroll
  for (int i = 0; i < kIds * kWaves; ++i) {
    if (i % kWaves == wave && (same[i / kWaves] >> lane & 1) != 0)
      f.entry[first + count_below(same[i / kWaves])] = (uint16_t)(tid + i / kWaves * kThreads);
    first += f.same[i];
  }
  __syncthreads();
}

// What the second launch reads: the number of active experts, and the j-th with its entries.
__device__ __forceinline__ void note_expert(int j, int e, const FindLds &f, int32_t *active,
                                            uint32_t *list, uint16_t *order) {
  if (threadIdx.x == 0) {
    if (j == 0) *active = f.active;
    if (e >= 0) list[j] = (uint32_t)e | (uint32_t)f.before << 10 | (uint32_t)(f.have - 1) << 20;
  }
  if (e >= 0)
    for (int i = threadIdx.x; i < f.have; i += kThreads) order[f.before + i] = f.entry[i];
}

// h of one entry and channel as a high and a low bf16 part. The workspace holds
// [I / 8][n][high, low][8] values, the entries in the order of their experts: the
// second launch's lanes, a part of an entry each, then read consecutive pieces of
// 16 bytes.
__device__ __forceinline__ void put_h(uint16_t *h, int n, int at, int c, float gate, float up) {
  // below kFarGate the sigmoid is the square of a = exp(gate / 2), which stays a normal number
  const float a = __expf(0.5f * gate), v = gate < kFarGate ? up * a * gate * a : silu(gate) * up;
  const uint16_t hi = bf16_bits(v);
  uint16_t *to = h + ((int64_t)(c >> 3) * n + at) * 16 + (c & 7);
  to[0] = hi;
  to[8] = (hi & 0x7F80) == 0x7F80 ? 0 : bf16_bits(v - bf16_value(hi));  // an infinity or NaN has no rest
}

// Few units: a workgroup takes 16 channels of one expert, its four waves share the long axis.
template <int WT>
__global__ __launch_bounds__(kThreads) void ep_moe_up_split(
    const uint16_t *__restrict__ x, const int32_t *__restrict__ topk_idx,
    const void *__restrict__ w, const float *__restrict__ scales, int T, int H, int I, int K, int E,
    int64_t units, int tiles, FastDiv by_k, int32_t *__restrict__ active, uint32_t *__restrict__ list,
    uint16_t *__restrict__ order, uint16_t *__restrict__ h) {
  constexpr int waves = kThreads / kWave;
  __shared__ FindLds f;
  __shared__ float red[waves * 2 * 4 * kWave];
  const __amdgpu_buffer_rsrc_t xb = buffer_of(x, (int64_t)T * H * 2);
  const int r = lane_id() & 15, wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int steps = (H + kStep - 1) / kStep;
  int have_j = -1;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), tile = (int)(u - (int64_t)j * tiles);
    if (j != have_j) find_expert(j, topk_idx, T * K, E, f);
    have_j = j;
    const int e = __builtin_amdgcn_readfirstlane(f.e), have = __builtin_amdgcn_readfirstlane(f.have);
    const int before = __builtin_amdgcn_readfirstlane(f.before);
    if (tile == 0) note_expert(j, e, f, active, list, order);
    if (e < 0) return;
    const Matrix m = matrix_of<WT>(w, scales, e, 2 * (int64_t)I, H);
    const int c0 = tile * kTile;
    const int row[2] = {c0 + r < I ? c0 + r : -1, c0 + r < I ? I + c0 + r : -1};
    for (int p0 = 0; p0 < have; p0 += kTile) {
      f32x4 acc[2] = {};
      multiply<WT, 2>(m, row, xb,
                      p0 + r < have ? fast_div_apply(f.entry[p0 + r], by_k) * (uint32_t)H * 2u : kOutside,
                      steps * wave / waves, steps * (wave + 1) / waves, acc);
      red_put<2>(red, wave, acc);
      __syncthreads();
      const int c = threadIdx.x % kTile, q = threadIdx.x / kTile;
      if (p0 + q < have && c0 + c < I)
        put_h(h, T * K, before + p0 + q, c0 + c, red_sum<2>(red, waves, 0, q, c), red_sum<2>(red, waves, 1, q, c));
      __syncthreads();
    }
  }
}

template <int WT, int MT>
__device__ __forceinline__ void up_wide_group(const Matrix &m, __amdgpu_buffer_rsrc_t x, int p0, int have,
                                              const uint16_t *entry, int c0, int I, FastDiv by_k,
                                              int n, int before, uint16_t *h, char *lds, uint32_t *tok_off) {
  const int lane = lane_id(), g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (threadIdx.x < MT * kTile) {
    const int p = p0 + (int)threadIdx.x;
    tok_off[threadIdx.x] = p < have ? fast_div_apply(entry[p], by_k) * (uint32_t)m.width * 2u : kOutside;
  }
  __syncthreads();
  constexpr int RT = kWideTiles, CT = RT / 2;
  int row[CT], near[RT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int first = c0 + (wave * CT + ct) * kTile, c = first + (lane & 15), from = first + near_row();
    row[ct] = c < I ? c : -1;
    near[ct] = from < I ? from : -1;
    near[CT + ct] = from < I ? I + from : -1;
  }
  f32x4 acc[MT][RT] = {};
  multiply_wide<WT, RT, MT>(m, near, x, tok_off, lds, acc);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + mt * kTile + g * 4 + i;
#pragma unroll
      for (int ct = 0; ct < CT; ++ct)
        if (p < have && row[ct] >= 0) put_h(h, n, before + p, row[ct], acc[mt][ct][i], acc[mt][CT + ct][i]);
    }
}

// Many units: a workgroup takes 64 channels (their gate and up rows) of one expert.
template <int WT>
__global__ __launch_bounds__(kThreads, 2) void ep_moe_up_wide(
    const uint16_t *__restrict__ x, const int32_t *__restrict__ topk_idx,
    const void *__restrict__ w, const float *__restrict__ scales, int T, int H, int I, int K, int E,
    int64_t units, int tiles, FastDiv by_k, int32_t *__restrict__ active, uint32_t *__restrict__ list,
    uint16_t *__restrict__ order, uint16_t *__restrict__ h) {
  __shared__ __attribute__((aligned(16))) char lds[wide_lds_bytes<WT, 2>()];
  __shared__ uint32_t tok_off[2 * kTile];
  __shared__ FindLds f;
  const __amdgpu_buffer_rsrc_t xb = buffer_of(x, (int64_t)T * H * 2);
  int have_j = -1;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), tile = (int)(u - (int64_t)j * tiles);
    if (j != have_j) find_expert(j, topk_idx, T * K, E, f);
    have_j = j;
    const int e = __builtin_amdgcn_readfirstlane(f.e), have = __builtin_amdgcn_readfirstlane(f.have);
    const int before = __builtin_amdgcn_readfirstlane(f.before);
    if (tile == 0) note_expert(j, e, f, active, list, order);
    if (e < 0) return;
    const Matrix m = matrix_of<WT>(w, scales, e, 2 * (int64_t)I, H);
    const int c0 = tile * (kWideTiles / 2 * 4 * kTile);
    for (int p = 0; p < have; p += 2 * kTile) {
      if (have - p > kTile) up_wide_group<WT, 2>(m, xb, p, have, f.entry, c0, I, by_k, T * K, before, h, lds, tok_off);
      else up_wide_group<WT, 1>(m, xb, p, have, f.entry, c0, I, by_k, T * K, before, h, lds, tok_off);
    }
    __syncthreads();  // f is rewritten for the next unit
  }
}

// Tokens go in groups of eight: the even rows of the matrix instruction are
// their high parts, the odd rows their low parts, so one instruction and one
// load per lane serve both. An expert with more entries has its rows read again, from
// the L2 that this wave has just filled. NG groups share a pass over the rows.
// A wave's chunks form one stream over all its units, one chunk ahead.
// Waves per workgroup: 8 of up to 256 registers each; with one row tile and
// half the chunk a wave needs half as many, and 16 waves are faster (45 tokens,
// hidden 336: 18 against 21 us). out may be bias, so neither is __restrict__.
constexpr int down_waves(int row_tiles, int groups) { return row_tiles == 1 && groups == 1 ? 16 : 8; }

template <int WT, int RT, int NG>
__global__ __launch_bounds__(down_waves(RT, NG) * kWave) void ep_moe_down(
    const uint16_t *__restrict__ h, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ topk_weights, const uint16_t *bias,
    const void *__restrict__ w, const float *__restrict__ scales, int T, int H, int I, int K, int E,
    int rows, int tiles, int most_parts, const int32_t *__restrict__ active,
    const uint32_t *__restrict__ list, const uint16_t *__restrict__ order, uint16_t *out) {
  using W = Weights<WT>;
  constexpr int kDownWaves = down_waves(RT, NG);
  constexpr int kChunkBytes = NG == 1 ? (RT == 1 ? 128 : 256) : 128;  // of a weight row
  constexpr int U = kChunkBytes / W::kStepBytes > 0 ? kChunkBytes / W::kStepBytes : 1;
  constexpr int kTokens = 8 * NG;
  extern __shared__ float part[];  // [parts][n][RT * 16]
  __shared__ uint32_t experts_lds[EP_MOE_MAX_ENTRIES];
  __shared__ uint16_t order_lds[EP_MOE_MAX_ENTRIES];
  __shared__ __attribute__((aligned(16))) char turn_lds[kDownWaves * kTurnBytes];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  const int piece_of = near_piece(), step_of = lane & 3;
  char *const slot = turn_lds + wave * kTurnBytes;
  const int n = T * K, steps = (I + kStep - 1) / kStep, groups = I / kStep;
  const int experts = __builtin_amdgcn_readfirstlane(*active);
  for (int i = threadIdx.x; i < n; i += kDownWaves * kWave) {
    experts_lds[i] = list[i];
    order_lds[i] = order[i];
  }
  __syncthreads();
  // parts of the long axis: two units for every wave, so that an uneven number of experts does
  // not leave half of the waves without work (one token: 123 against 131 us with one)
  int parts = experts > 0 ? (2 * kDownWaves + experts - 1) / experts : 1;
  parts = parts < most_parts ? parts : most_parts;
  const int units = experts * parts;
  const __amdgpu_buffer_rsrc_t hb = buffer_of(h, (int64_t)n * I * 4);

  struct Place {  // of a chunk in the stream: unit, first entry of the group, step
    int u, p, s, e, begin, have, s0, s1;
  };
  const auto enter = [&](Place &a) {  // the unit a.u; behind the last one a place whose loads lie outside
    a.e = a.begin = a.have = a.p = a.s = a.s0 = a.s1 = 0;
    if (a.u >= units) return;
    const int j = a.u / parts, q = a.u - j * parts;
    const MoeEntry m{(uint32_t)__builtin_amdgcn_readfirstlane((int)experts_lds[j])};
    a.e = m.e(), a.begin = m.begin(), a.have = m.count(), a.p = 0;
    a.s = a.s0 = steps * q / parts, a.s1 = steps * (q + 1) / parts;
  };
  const auto next = [&](const Place &now) {
    Place a = now;
    a.s += U;
    if (a.s >= a.s1) {
      a.s = a.s0;
      a.p += kTokens;
      if (a.p >= a.have) {
        a.u += kDownWaves;
        enter(a);
      }
    }
    return a;
  };

  struct Chunk {
    u32x4 w[U][RT][W::kLoads], t[U][NG][4];
    float scale[RT];
  };
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n0 = tile * rows, here = H - n0 < rows ? H - n0 : rows;
    uint32_t wrow[RT], srow[RT];
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int at = rt * kTile + near_row();
      wrow[rt] = at < here ? (uint32_t)(((int64_t)(n0 + at) * I * W::kStepBytes) / kStep) : kOutside;
      srow[rt] = at < here ? (uint32_t)(n0 + at) * (uint32_t)groups * 4u : kOutside;
    }
    f32x4 acc[NG][RT];
    const auto load = [&](Chunk &c, const Place &a) {
      const Matrix m = matrix_of<WT>(w, scales, a.e, H, I);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int l = 0; l < W::kLoads; ++l)
            c.w[u][rt][l] = load16(m.w, weight_at<WT>(I, wrow[rt], a.s + u, a.s1, l, piece_of));
      if constexpr (W::kScaled) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          c.scale[rt] = load4(m.scales, only(step_of < U && a.s + step_of < a.s1,
                                              srow[rt] + (uint32_t)(a.s + step_of) * 4u));
      }
#pragma unroll
      for (int ng = 0; ng < NG; ++ng) {
        const int p = a.p + ng * 8 + (r >> 1);
        const uint32_t tok = only(p < a.have, (uint32_t)((a.begin + p) * 2 + (r & 1)) * 16u);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int s = a.s + u, k = s * kStep + W::place(j, g);
            const bool in = s < a.s1 && (W::kScaled || k < I);
            c.t[u][ng][j] = load16(hb, only(in, tok + (uint32_t)(k >> 3) * (uint32_t)n * 32u));
          }
      }
    };
    const auto add = [&](const Chunk &c, const Place &a) {
      if (a.s == a.s0)
#pragma unroll
        for (int ng = 0; ng < NG; ++ng)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) acc[ng][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
      // Steps behind the part's end are zeros and not skipped: a load that no use waits for holds
      // up the next one to its registers.
#pragma unroll
      for (int u = 0; u < U; ++u) {
        u32x4 turned[RT][W::kLoads];
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
#pragma unroll
          for (int l = 0; l < W::kLoads; ++l) turned[rt][l] = turn(slot, c.w[u][rt][l]);
        f32x4 sum[NG][RT];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const bf16x8 b = W::operand(turned[rt], j);
#pragma unroll
            for (int ng = 0; ng < NG; ++ng) {
              const bf16x8 t = __builtin_bit_cast(bf16x8, c.t[u][ng][j]);
              if constexpr (W::kScaled)
                sum[ng][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
                    t, b, j == 0 ? f32x4{0.f, 0.f, 0.f, 0.f} : sum[ng][rt], 0, 0, 0);
              else
                acc[ng][rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(t, b, acc[ng][rt], 0, 0, 0);
            }
          }
        if constexpr (W::kScaled) {
#pragma unroll
          for (int rt = 0; rt < RT; ++rt) {
            const float sc = lane_value(c.scale[rt], r * 4 + u);
#pragma unroll
            for (int ng = 0; ng < NG; ++ng)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[ng][rt][i] += sc * sum[ng][rt][i];
          }
        }
      }
      if (a.s + U < a.s1) return;
      // the group's end: a lane's four results are the parts of two entries
      float *const to = part + (int64_t)(a.u % parts) * n * (RT * kTile);
#pragma unroll
      for (int ng = 0; ng < NG; ++ng)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int p = a.p + ng * 8 + g * 2 + i;
          if (p >= a.have) continue;
          const int entry = order_lds[a.begin + p];
#pragma unroll
          for (int rt = 0; rt < RT; ++rt)
            to[entry * (RT * kTile) + rt * kTile + r] = acc[ng][rt][2 * i] + acc[ng][rt][2 * i + 1];
        }
    };
    Place a, b;
    a.u = wave;
    enter(a);
    Chunk ca, cb;
    load(ca, a);
    while (a.u < units) {
      b = next(a);
      load(cb, b);
      __builtin_amdgcn_sched_barrier(0);
      add(ca, a);
      __builtin_amdgcn_sched_barrier(0);
      if (b.u >= units) break;
      a = next(b);
      load(ca, a);
      __builtin_amdgcn_sched_barrier(0);
      add(cb, b);
      __builtin_amdgcn_sched_barrier(0);
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * here; i += kDownWaves * kWave) {
      const int t = i / here, c = i - t * here;
      float sum = 0.f;
      for (int k = 0; k < K; ++k) {
        const int at = t * K + k, id = topk_idx[at];
        if (id < 0 || id >= E) continue;
        float v = 0.f;
        for (int q = 0; q < parts; ++q) v += part[((int64_t)q * n + at) * (RT * kTile) + c];
        sum += (topk_weights != nullptr ? topk_weights[at] : 1.0f) * v;
      }
      const int64_t at = (int64_t)t * H + n0 + c;
      if (bias != nullptr) sum += bf16_value(bias[at]);
      out[at] = bf16_bits(sum);
    }
    __syncthreads();
  }
}

constexpr int64_t kMaxBlocks = (1 << 22) - 1;  // of at most 1024 threads: within the grid limit of 2^32

template <int WT>
int matvec_split_launch(const ExpertMatvecArgs &a, int cap) {
  const int tiles = (a.N + kTile - 1) / kTile;
  const int64_t experts = a.counts == nullptr ? 1 : (a.E < a.capacity ? a.E : a.capacity);
  const int64_t units = experts * tiles;
  const int steps = (a.K + kStep - 1) / kStep;
  const int waves = steps <= 4 ? 4 : (steps <= 8 ? 8 : 16);
  const int64_t most = cap > 0 ? cap : kMaxBlocks;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  const size_t lds = (size_t)waves * 4 * kWave * sizeof(float);
  if (a.fp32)
    ep_expert_matvec_split<WT, true><<<blocks, waves * kWave, lds, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  else
    ep_expert_matvec_split<WT, false><<<blocks, waves * kWave, lds, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  return launch_status();
}

template <int WT>
int matvec_wide_launch(const ExpertMatvecArgs &a, int cap) {
  constexpr int kRows = kWideTiles * 4 * kTile;
  const int tiles = (a.N + kRows - 1) / kRows;
  const int64_t experts = a.counts == nullptr ? 1 : (a.E < a.capacity ? a.E : a.capacity);
  const int64_t units = experts * tiles;
  // Four workgroups for every compute unit, which loop: experts without rows then cost no workgroup each
  // (8 of 256 experts with a row, 2048 to 4096 in fp4 at A = 16: 12.7 us, 31 with a workgroup for every
  // tile that may be; 64 experts of 16 rows, 2048 tiles that all are: 201 us either way).
  const int64_t most = cap > 0 ? cap : 4 * kComputeUnits;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  if (a.fp32)
    ep_expert_matvec_wide<WT, true><<<blocks, kThreads, 0, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  else
    ep_expert_matvec_wide<WT, false><<<blocks, kThreads, 0, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  return launch_status();
}

template <int WT>
int matvec_pick(const ExpertMatvecArgs &a, int cap) {
  const int64_t experts = a.counts == nullptr ? 1 : (a.E < a.capacity ? a.E : a.capacity);
  const int wide_tiles = (a.N + 4 * kWideTiles * kTile - 1) / (4 * kWideTiles * kTile);
  return matvec_is_wide(experts, a.capacity, wide_tiles) ? matvec_wide_launch<WT>(a, cap) : matvec_split_launch<WT>(a, cap);
}

struct MoeWorkspace {
  int32_t *active;
  uint32_t *list;
  uint16_t *order, *h;
};
size_t moe_head_bytes(int64_t n) { return (size_t)((256 + 6 * n + 255) / 256 * 256); }

template <int WT>
int moe_up_split_launch(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap) {
  const int n = a.T * a.K;
  const int tiles = (a.I + kTile - 1) / kTile;
  const int64_t units = (int64_t)(n < a.E ? n : a.E) * tiles;
  const int64_t most = cap > 0 ? cap : kMaxBlocks;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  ep_moe_up_split<WT><<<blocks, kThreads, 0, a.stream>>>(
      (const uint16_t *)a.x, a.topk_idx, a.w_in, a.in_scales, a.T, a.H, a.I, a.K, a.E, units, tiles,
      fast_div((uint32_t)a.K), ws.active, ws.list, ws.order, ws.h);
  return launch_status();
}

template <int WT>
int moe_up_wide_launch(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap) {
  const int n = a.T * a.K;
  constexpr int kChannels = kWideTiles / 2 * 4 * kTile;
  const int tiles = (a.I + kChannels - 1) / kChannels;
  const int64_t units = (int64_t)(n < a.E ? n : a.E) * tiles;
  const int64_t most = cap > 0 ? cap : kMaxBlocks;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  ep_moe_up_wide<WT><<<blocks, kThreads, 0, a.stream>>>(
      (const uint16_t *)a.x, a.topk_idx, a.w_in, a.in_scales, a.T, a.H, a.I, a.K, a.E, units, tiles,
      fast_div((uint32_t)a.K), ws.active, ws.list, ws.order, ws.h);
  return launch_status();
}

template <int WT, int RT, int NG>
int moe_down_launch(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap, int rows) {
  const int n = a.T * a.K;
  const int tiles = (a.H + rows - 1) / rows;
  constexpr int kLdsEntries = 1024;  // parts * entries kept in LDS: 64 or 128 KB
  const int steps = (a.I + kStep - 1) / kStep;
  constexpr int kDownWaves = down_waves(RT, NG);
  int parts = kLdsEntries / n;
  parts = parts < 2 * kDownWaves ? parts : 2 * kDownWaves;
  parts = parts < steps ? parts : steps;
  const unsigned blocks = (unsigned)(cap > 0 && tiles > cap ? cap : tiles);
  const size_t lds = (size_t)parts * n * RT * kTile * sizeof(float);
  ep_moe_down<WT, RT, NG><<<blocks, kDownWaves * kWave, lds, a.stream>>>(
      ws.h, a.topk_idx, a.topk_weights, (const uint16_t *)a.bias, a.w_out, a.out_scales, a.T, a.H, a.I,
      a.K, a.E, rows, tiles, parts, ws.active, ws.list, ws.order, (uint16_t *)a.out);
  return launch_status();
}

// First launch: 64 channels a workgroup where these fill the chip (28 fp8
// entries of 20 experts, hidden 2048, 240 to 336 workgroups: 15 against 20 us;
// 8 bf16 experts of one token, 256 workgroups: 80 us either way), or half of it
// with four entries an expert (128 workgroups in bf16, hidden 4096: 25 against
// 27 us with 4 entries an expert, 28 against 37 with 16), else 16 and the long
// axis shared (8 fp4 experts of one token, 176 workgroups: 16 against 18 us; 4
// fp8 experts of 32 entries, 64: 29 against 38; one bf16 expert, 32: 18 against
// 54). Counted by the experts that the entries could have, not by those that they
// have, which only the device knows: counting there made a few tokens' layer (about
// 18 of 32 fp8 experts active) 37 us instead of 26 and the hot cases 15% slower to
// 20% faster.
// Second launch: two groups of eight tokens a pass where experts have more than
// eight entries on the average (64 fp4 experts, 16 entries each: 255 against
// 266 us; 16 fp8 experts of 64: 191 against 237), else one (197 active fp4
// experts, 5 entries each: 473 against 528). The average is over all experts too: entries
// that all go to 8 of 256 experts (64 tokens, top-8, fp8, 4096 / 512) take 68 us, 62 in a call
// with these 8 experts alone, 64 entries of 4 of 64 bf16 experts (1024 / 512) 19 against 16.
template <int WT>
int moe_pick(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap) {
  const int n = a.T * a.K;
  constexpr int kChannels = kWideTiles / 2 * 4 * kTile;
  const int experts = n < a.E ? n : a.E;
  const int64_t wide_units = (int64_t)experts * ((a.I + kChannels - 1) / kChannels);
  const bool wide = wide_units >= kComputeUnits || (wide_units >= kComputeUnits / 2 && n >= 4 * experts);
  const int rc = wide ? moe_up_wide_launch<WT>(a, ws, cap) : moe_up_split_launch<WT>(a, ws, cap);
  if (rc != 0) return rc;
  // Output rows per workgroup: an even share of the chip's 256 compute units, at most two tiles.
  // Rounded up to two rows, not to a tile: a small layer fills more compute units (whole layers of
  // H 256, 336 and 1152: 36.2, 16.5 and 20.0 us; to four rows 36.4, 17.6, 21.2, to 16 40.4, 25.1, 24.8).
  int rows = (a.H + kComputeUnits - 1) / kComputeUnits;
  rows = (rows + 1) / 2 * 2;
  rows = rows < 2 * kTile ? rows : 2 * kTile;
  const bool many = n > 8 * a.E;
  if (rows <= kTile)
    return many ? moe_down_launch<WT, 1, 2>(a, ws, cap, rows) : moe_down_launch<WT, 1, 1>(a, ws, cap, rows);
  return many ? moe_down_launch<WT, 2, 2>(a, ws, cap, rows) : moe_down_launch<WT, 2, 1>(a, ws, cap, rows);
}

}  // namespace

int launch_expert_matvec(const ExpertMatvecArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  if (a.dtype == EP_BF16) return matvec_pick<EP_BF16>(a, cap);
  if (a.dtype == EP_FP8_E4M3) return matvec_pick<EP_FP8_E4M3>(a, cap);
  return matvec_pick<EP_FP4X2>(a, cap);
}

size_t moe_layer_workspace(int T, int K, int I) {
  const int64_t n = (int64_t)T * K;
  return n == 0 ? 0 : moe_head_bytes(n) + (size_t)n * I * 4;
}

int launch_moe_layer(const MoeLayerArgs &a) {
  if (a.T == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  const int n = a.T * a.K;
  char *p = (char *)a.workspace;
  MoeWorkspace ws{(int32_t *)p, (uint32_t *)(p + 256), (uint16_t *)(p + 256 + 4 * (size_t)n),
                  (uint16_t *)(p + moe_head_bytes(n))};
  if (a.dtype == EP_BF16) return moe_pick<EP_BF16>(a, ws, cap);
  if (a.dtype == EP_FP8_E4M3) return moe_pick<EP_FP8_E4M3>(a, ws, cap);
  return moe_pick<EP_FP4X2>(a, ws, cap);
}

}  // namespace ep
