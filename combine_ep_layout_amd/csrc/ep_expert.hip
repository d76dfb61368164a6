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
// What bounds it: with at most a few tokens per expert every weight is used
// a few times, so the time is that of reading the active experts' weights
// from HBM once. The products run on the matrix cores (16x16x32 bf16) all the
// same: a wave takes 16 weight rows per tile as one operand, straight from
// memory into registers (each row's 64 consecutive bytes go to four lanes:
// nothing is shared between waves, so LDS would only add a trip), and 16
// tokens as the other; lanes of absent tokens and rows are given an offset
// outside the buffer descriptor, which reads as 0 and costs no traffic.
#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

constexpr uint32_t kOutside = 0x80000000u;  // a buffer offset outside every descriptor (below 2^31 bytes)
constexpr int kTile = 16;                   // rows and tokens of one matrix instruction
constexpr int kStep = 128;                  // values of the long axis per step: one scale group
constexpr int kThreads = 256;

__device__ __forceinline__ __amdgpu_buffer_rsrc_t buffer_of(const void *base, int64_t bytes) {
  constexpr int kRawBufferFlags = 0x00020000;
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(base), (short)0, (int)bytes,
                                           kRawBufferFlags);
}
__device__ __forceinline__ u32x4 load16(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 0);
}
// Weights are read once: non-temporal.
__device__ __forceinline__ u32x4 load16_stream(__amdgpu_buffer_rsrc_t b, uint32_t off) {
  return __builtin_amdgcn_raw_buffer_load_b128(b, (int)off, 0, 2);
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

// acc[mt][rt] += rows x tokens over steps [s0, s1). Lane (r = lane % 16,
// g = lane / 16): row[rt] is its weight row (negative: absent), tok[mt] the
// byte offset of its token's row in x (kOutside: absent). The tokens are the
// first operand, so a lane's four results are four tokens of one weight row
// and it needs one scale. SPLIT: each token row is the sum of two bf16 rows,
// low_bytes apart (an fp32 value as high and low part).
template <int WT, int RT, int MT, bool SPLIT>
__device__ __forceinline__ void multiply(const Matrix &m, const int (&row)[RT],
                                         __amdgpu_buffer_rsrc_t x, const uint32_t (&tok)[MT],
                                         uint32_t low_bytes, int s0, int s1,
                                         f32x4 (&acc)[MT][RT]) {
  using W = Weights<WT>;
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  uint32_t wrow[RT], srow[RT];
  const int groups = m.width / kStep;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    wrow[rt] = row[rt] < 0 ? kOutside : (uint32_t)(((int64_t)row[rt] * m.width * W::kStepBytes) / kStep);
    srow[rt] = row[rt] < 0 ? kOutside : (uint32_t)row[rt] * (uint32_t)groups * 4u;
  }
  float ahead[RT];
#pragma unroll 2
  for (int s = s0; s < s1; ++s) {
    u32x4 w[RT][W::kLoads], t[MT][4], low[MT][4];
    if constexpr (W::kScaled) {
      // lane group g reads the scale of the g-th of the next four steps
      if (((s - s0) & 3) == 0) {
#pragma unroll
        for (int rt = 0; rt < RT; ++rt)
          ahead[rt] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(
              m.scales, (int)(s + g < s1 ? srow[rt] + (uint32_t)(s + g) * 4u : kOutside), 0, 0));
      }
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt)
#pragma unroll
      for (int l = 0; l < W::kLoads; ++l) {
        uint32_t off = wrow[rt] + (uint32_t)s * W::kStepBytes + W::load_byte(l, g);
        if constexpr (!W::kScaled)  // the last step of a width that is no multiple of 128
          off = s * kStep + W::place(l, g) < m.width ? off : kOutside;
        w[rt][l] = load16_stream(m.w, off);
      }
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = s * kStep + W::place(j, g);
        uint32_t off = tok[mt] + (uint32_t)k * 2u;
        if constexpr (!W::kScaled) off = k < m.width ? off : kOutside;
        t[mt][j] = load16(x, off);
        if constexpr (SPLIT) low[mt][j] = load16(x, off + low_bytes);
      }
    f32x4 part[MT][RT];
    if constexpr (W::kScaled) {
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) part[mt][rt] = f32x4{0.f, 0.f, 0.f, 0.f};
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const bf16x8 b = W::operand(w[rt], j);
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
          f32x4 &c = W::kScaled ? part[mt][rt] : acc[mt][rt];
          c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, t[mt][j]), b, c, 0, 0, 0);
          if constexpr (SPLIT)
            c = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, low[mt][j]), b, c, 0, 0, 0);
        }
      }
    if constexpr (W::kScaled) {
#pragma unroll
      for (int rt = 0; rt < RT; ++rt) {
        const int from = ((((s - s0) & 3) << 4) | r) << 2;
        const float sc = __int_as_float(__builtin_amdgcn_ds_bpermute(from, __float_as_int(ahead[rt])));
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][rt][i] += sc * part[mt][rt][i];
      }
    }
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

__device__ __forceinline__ float silu(float g) { return g / (1.0f + __expf(-g)); }

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  return __builtin_bit_cast(uint16_t, (__bf16)v);
}
__device__ __forceinline__ float bf16_value(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }

// ------------------------------------------------------------ ep_expert_matvec

// The j-th expert that has rows, by a scan of the counts (1024 at most, four
// per thread of 256); absent: e = -1. A count is cut to the rows that lie
// inside the buffer, so no access leaves it whatever the arrays hold.
struct Segment {
  int e;
  int64_t begin, count;
};
__device__ __forceinline__ int64_t rows_inside(const int32_t *counts, const int32_t *offsets, int e,
                                               int64_t capacity) {
  const int64_t b = offsets[e], c = counts[e];
  return b < 0 || b >= capacity ? 0 : (c < capacity - b ? c : capacity - b);
}
__device__ __forceinline__ Segment find_segment(int j, const int32_t *counts,
                                                const int32_t *offsets, int E, int64_t capacity,
                                                int *lds) {
  if (counts == nullptr) return {j == 0 ? 0 : -1, 0, capacity};
  const int tid = threadIdx.x, wave = tid / kWave;
  int first = tid * 4, have = 0;
  if (tid < kThreads)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (first + i < E && rows_inside(counts, offsets, first + i, capacity) > 0) have |= 1 << i;
  const int mine = __popc(have), upto = wave_inclusive_scan(mine);
  if (tid == 0) lds[16] = -1;
  if (lane_id() == kWave - 1) lds[wave] = upto;
  __syncthreads();
  int before = upto - mine;
  for (int w = 0; w < wave; ++w) before += lds[w];
  if (j >= before && j < before + mine) {
    int skip = j - before;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (have >> i & 1 && skip-- == 0) lds[16] = first + i;
  }
  __syncthreads();
  const int e = __builtin_amdgcn_readfirstlane(lds[16]);
  __syncthreads();
  if (e < 0) return {-1, 0, 0};
  return {e, (int64_t)offsets[e], rows_inside(counts, offsets, e, capacity)};
}

template <int WT, int RT, int MT, bool FP32>
__device__ __forceinline__ void matvec_group(const Matrix &m, const uint16_t *x, int64_t row0,
                                             int rows, int n0, int N, void *y, float *red) {
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  const int waves = blockDim.x / kWave;
  const int steps = (m.width + kStep - 1) / kStep;
  // rows beyond the group lie outside the descriptor
  const __amdgpu_buffer_rsrc_t xb = buffer_of(x + row0 * m.width, (int64_t)rows * m.width * 2);
  int row[RT];
  uint32_t tok[MT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    const int n = n0 + rt * kTile + (lane & 15);
    row[rt] = n < N ? n : -1;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int p = mt * kTile + (lane & 15);
    tok[mt] = p < rows ? (uint32_t)p * (uint32_t)m.width * 2u : kOutside;
  }
  f32x4 acc[MT][RT] = {};
  multiply<WT, RT, MT, false>(m, row, xb, tok, 0, steps * wave / waves, steps * (wave + 1) / waves,
                              acc);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    red_put<RT>(red, wave, acc[mt]);
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * RT * kTile; i += blockDim.x) {
      const int c = i % (RT * kTile), p = i / (RT * kTile);
      const int n = n0 + c;
      if (mt * kTile + p < rows && n < N) {
        const float v = red_sum<RT>(red, waves, c / kTile, p, c % kTile);
        const int64_t at = (row0 + mt * kTile + p) * (int64_t)N + n;
        if constexpr (FP32) ((float *)y)[at] = v;
        else ((uint16_t *)y)[at] = bf16_bits(v);
      }
    }
    __syncthreads();
  }
}

template <int WT, int RT, bool FP32>
__global__ __launch_bounds__(1024) void ep_expert_matvec_tiles(
    const uint16_t *__restrict__ x, const void *__restrict__ w, const float *__restrict__ scales,
    const int32_t *__restrict__ counts, const int32_t *__restrict__ offsets, int E,
    int64_t capacity, int K, int N, int64_t units, int tiles, void *__restrict__ y) {
  extern __shared__ float red[];
  __shared__ int lds[17];
  int have_j = -1;
  Segment seg{-1, 0, 0};
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), n0 = (int)(u - (int64_t)j * tiles) * RT * kTile;
    if (j != have_j) seg = find_segment(j, counts, offsets, E, capacity, lds);
    have_j = j;
    if (seg.e < 0) return;  // no further expert has rows
    const Matrix m = matrix_of<WT>(w, scales, seg.e, N, K);
    for (int64_t p = 0; p < seg.count;) {
      const int64_t left = seg.count - p;
      const int rows = (int)(left < 4 * kTile ? left : 4 * kTile);
      if (rows > 2 * kTile)
        matvec_group<WT, RT, 4, FP32>(m, x, seg.begin + p, rows, n0, N, y, red);
      else if (rows > kTile)
        matvec_group<WT, RT, 2, FP32>(m, x, seg.begin + p, rows, n0, N, y, red);
      else
        matvec_group<WT, RT, 1, FP32>(m, x, seg.begin + p, rows, n0, N, y, red);
      p += rows;
    }
  }
}

// ---------------------------------------------------------------- ep_moe_layer
//
// First launch: workgroup (j, tile) finds the j-th expert that occurs in
// topk_idx and its entries by itself (n = T*K <= 1024 ids, no extra launch),
// its four waves split the long axis of 16 or 32 channels' gate and up rows,
// and h goes to the workspace as a high and a low bf16 part per value, so
// that the second product loses nothing to the rounding of h. The workgroups
// of tile 0 leave the list of active experts and their entries behind.
// Second launch: a workgroup owns up to 32 output channels of every token;
// its waves take (expert, part of the long axis) units, the entries' results
// stay in LDS, and are summed with their router weights in k order, so the
// result is a pure function of the inputs.

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
  int e, before, have, active, next;
};

// The j-th active expert (first occurrence order for n <= 64, ascending id
// above): e or -1, its `have` entries in f.entry, `before` entries of other
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
  if (tid == 0) f.e = -1, f.next = 0;
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
  if (e >= 0) {
#pragma unroll
    for (int q = 0; q < EP_MOE_MAX_ENTRIES / kThreads; ++q)
      if (id[q] == e) f.entry[atomicAdd(&f.next, 1)] = (uint16_t)(tid + q * kThreads);
  }
  __syncthreads();
}

template <int WT, int RT, int MT>
__device__ __forceinline__ void up_group(const Matrix &m, __amdgpu_buffer_rsrc_t x, int p0, int have,
                                         const uint16_t *entry, int c0, int I, int K, FastDiv by_k,
                                         uint16_t *h, float *red) {
  constexpr int CT = RT / 2;  // channel tiles: CT of gate rows, CT of up rows
  const int lane = lane_id(), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  constexpr int waves = kThreads / kWave;
  const int steps = (m.width + kStep - 1) / kStep;
  int row[RT];
  uint32_t tok[MT];
#pragma unroll
  for (int ct = 0; ct < CT; ++ct) {
    const int c = c0 + ct * kTile + (lane & 15);
    row[ct] = c < I ? c : -1;
    row[CT + ct] = c < I ? I + c : -1;
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int p = p0 + mt * kTile + (lane & 15);
    tok[mt] = p < have ? fast_div_apply(entry[p], by_k) * (uint32_t)m.width * 2u : kOutside;
  }
  f32x4 acc[MT][RT] = {};
  multiply<WT, RT, MT, false>(m, row, x, tok, 0, steps * wave / waves, steps * (wave + 1) / waves,
                              acc);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    red_put<RT>(red, wave, acc[mt]);
    __syncthreads();
    for (int i = threadIdx.x; i < kTile * CT * kTile; i += kThreads) {
      const int c = i % (CT * kTile), q = i / (CT * kTile), p = p0 + mt * kTile + q;
      if (p < have && c0 + c < I) {
        const float gate = red_sum<RT>(red, waves, c / kTile, q, c % kTile);
        const float up = red_sum<RT>(red, waves, CT + c / kTile, q, c % kTile);
        const float v = silu(gate) * up;
        const uint16_t hi = bf16_bits(v);
        const float rest = v - bf16_value(hi);
        uint16_t *to = h + (int64_t)entry[p] * 2 * I + c0 + c;
        to[0] = hi;
        to[I] = (hi & 0x7F80) == 0x7F80 ? 0 : bf16_bits(rest);  // an infinity or NaN has no rest
      }
    }
    __syncthreads();
  }
}

template <int WT, int RT, int MTMAX>
__global__ __launch_bounds__(kThreads) void ep_moe_up(
    const uint16_t *__restrict__ x, const int32_t *__restrict__ topk_idx,
    const void *__restrict__ w, const float *__restrict__ scales, int T, int H, int I, int K, int E,
    int64_t units, int tiles, FastDiv by_k, int32_t *__restrict__ active, uint32_t *__restrict__ list,
    uint16_t *__restrict__ order, uint16_t *__restrict__ h) {
  __shared__ FindLds f;
  __shared__ float red[kThreads / kWave * RT * 4 * kWave];
  const __amdgpu_buffer_rsrc_t xb = buffer_of(x, (int64_t)T * H * 2);
  int have_j = -1;
  for (int64_t u = blockIdx.x; u < units; u += gridDim.x) {
    const int j = (int)(u / tiles), tile = (int)(u - (int64_t)j * tiles);
    if (j != have_j) find_expert(j, topk_idx, T * K, E, f);
    have_j = j;
    const int e = __builtin_amdgcn_readfirstlane(f.e), have = f.have;
    if (tile == 0) {
      if (threadIdx.x == 0) {
        if (j == 0) *active = f.active;
        if (e >= 0) list[j] = (uint32_t)e | (uint32_t)f.before << 10 | (uint32_t)(have - 1) << 20;
      }
      if (e >= 0)
        for (int i = threadIdx.x; i < have; i += kThreads) order[f.before + i] = f.entry[i];
    }
    if (e < 0) return;
    const Matrix m = matrix_of<WT>(w, scales, e, 2 * (int64_t)I, H);
    const int c0 = tile * (RT / 2) * kTile;
    for (int p = 0; p < have;) {
      const int left = have - p;
      if (MTMAX > 2 && left > 2 * kTile) {
        up_group<WT, RT, MTMAX>(m, xb, p, have, f.entry, c0, I, K, by_k, h, red);
        p += MTMAX * kTile;
      } else if (MTMAX > 1 && left > kTile) {
        up_group<WT, RT, MTMAX < 2 ? 1 : 2>(m, xb, p, have, f.entry, c0, I, K, by_k, h, red);
        p += 2 * kTile;
      } else {
        up_group<WT, RT, 1>(m, xb, p, have, f.entry, c0, I, K, by_k, h, red);
        p += kTile;
      }
    }
  }
}

template <int WT, int RT, int MT>
__device__ __forceinline__ void down_group(const Matrix &m, __amdgpu_buffer_rsrc_t h, int p0, int have,
                                           const uint16_t *order, int n0, int rows, int I, int s0,
                                           int s1, float *part) {
  const int lane = lane_id(), r = lane & 15, g = lane >> 4;
  int row[RT];
  uint32_t tok[MT];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) row[rt] = rt * kTile + r < rows ? n0 + rt * kTile + r : -1;
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    const int p = p0 + mt * kTile + r;
    tok[mt] = p < have ? (uint32_t)order[p] * (uint32_t)I * 4u : kOutside;
  }
  f32x4 acc[MT][RT] = {};
  multiply<WT, RT, MT, true>(m, row, h, tok, (uint32_t)I * 2u, s0, s1, acc);
#pragma unroll
  for (int mt = 0; mt < MT; ++mt)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int p = p0 + mt * kTile + g * 4 + i;
      if (p < have)
#pragma unroll
        for (int rt = 0; rt < RT; ++rt) part[(int)order[p] * (RT * kTile) + rt * kTile + r] = acc[mt][rt][i];
    }
}

template <int WT, int RT, int MTMAX>
__global__ __launch_bounds__(1024) void ep_moe_down(
    const uint16_t *__restrict__ h, const int32_t *__restrict__ topk_idx,
    const float *__restrict__ topk_weights, const uint16_t *__restrict__ bias,
    const void *__restrict__ w, const float *__restrict__ scales, int T, int H, int I, int K, int E,
    int rows, int tiles, int most_parts, const int32_t *__restrict__ active,
    const uint32_t *__restrict__ list, const uint16_t *__restrict__ order,
    uint16_t *__restrict__ out) {
  extern __shared__ float part[];  // [parts][n][RT * 16]
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), waves = blockDim.x / kWave;
  const int n = T * K;
  const int steps = (I + kStep - 1) / kStep;
  const int experts = __builtin_amdgcn_readfirstlane(*active);
  // parts of the long axis: enough units for every wave
  int parts = experts > 0 ? (waves + experts - 1) / experts : 1;
  parts = parts < most_parts ? parts : most_parts;
  const __amdgpu_buffer_rsrc_t hb = buffer_of(h, (int64_t)n * I * 4);
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int n0 = tile * rows, here = H - n0 < rows ? H - n0 : rows;
    for (int u = wave; u < experts * parts; u += waves) {
      const int j = u / parts, q = u - j * parts;
      const MoeEntry a{(uint32_t)__builtin_amdgcn_readfirstlane((int)list[j])};
      const Matrix m = matrix_of<WT>(w, scales, a.e(), H, I);
      const uint16_t *mine = order + a.begin();
      const int s0 = steps * q / parts, s1 = steps * (q + 1) / parts, have = a.count();
      float *to = part + (int64_t)q * n * (RT * kTile);
      for (int p = 0; p < have;) {
        const int left = have - p;
        if (MTMAX > 1 && left > kTile) {
          down_group<WT, RT, MTMAX>(m, hb, p, have, mine, n0, here, I, s0, s1, to);
          p += MTMAX * kTile;
        } else {
          down_group<WT, RT, 1>(m, hb, p, have, mine, n0, here, I, s0, s1, to);
          p += kTile;
        }
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < T * here; i += blockDim.x) {
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

constexpr int kComputeUnits = 256;

template <int WT, int RT>
int matvec_launch(const ExpertMatvecArgs &a, int cap) {
  const int tiles = (a.N + RT * kTile - 1) / (RT * kTile);
  const int64_t experts = a.counts == nullptr ? 1 : (a.E < a.capacity ? a.E : a.capacity);
  const int64_t units = experts * tiles;
  const int steps = (a.K + kStep - 1) / kStep;
  // few tiles: up to 16 waves share one tile's long axis
  const int waves = units >= 2 * kComputeUnits || steps <= 4 ? 4 : (steps <= 8 ? 8 : 16);
  const int64_t most = cap > 0 ? cap : INT32_MAX;
  const unsigned blocks = (unsigned)(units < most ? units : most);
  const size_t lds = (size_t)waves * RT * 4 * kWave * sizeof(float);
  if (a.fp32)
    ep_expert_matvec_tiles<WT, RT, true><<<blocks, waves * kWave, lds, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  else
    ep_expert_matvec_tiles<WT, RT, false><<<blocks, waves * kWave, lds, a.stream>>>(
        (const uint16_t *)a.x, a.w, a.scales, a.counts, a.offsets, a.E, a.capacity, a.K, a.N, units,
        tiles, a.y);
  return launch_status();
}

template <int WT, int WIDE>
int matvec_pick(const ExpertMatvecArgs &a, int cap) {
  const int64_t experts = a.counts == nullptr ? 1 : (a.E < a.capacity ? a.E : a.capacity);
  const int64_t wide_tiles = (a.N + WIDE * kTile - 1) / (WIDE * kTile);
  return experts * wide_tiles >= 4 * kComputeUnits ? matvec_launch<WT, WIDE>(a, cap)
                                                   : matvec_launch<WT, 1>(a, cap);
}

struct MoeWorkspace {
  int32_t *active;
  uint32_t *list;
  uint16_t *order, *h;
};
size_t moe_head_bytes(int64_t n) { return (size_t)((256 + 6 * n + 255) / 256 * 256); }

template <int WT, int RT, int MTMAX>
int moe_up_launch(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap) {
  const int n = a.T * a.K;
  const int tiles = (a.I + RT / 2 * kTile - 1) / (RT / 2 * kTile);
  const int64_t units = (int64_t)(n < a.E ? n : a.E) * tiles;
  const unsigned blocks = (unsigned)(cap > 0 && units > cap ? cap : units);
  ep_moe_up<WT, RT, MTMAX><<<blocks, kThreads, 0, a.stream>>>(
      (const uint16_t *)a.x, a.topk_idx, a.w_in, a.in_scales, a.T, a.H, a.I, a.K, a.E, units, tiles,
      fast_div((uint32_t)a.K), ws.active, ws.list, ws.order, ws.h);
  return launch_status();
}

template <int WT, int RT, int MTMAX>
int moe_down_launch(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap, int rows) {
  const int n = a.T * a.K;
  const int tiles = (a.H + rows - 1) / rows;
  constexpr int kLdsEntries = 1024;  // parts * entries kept in LDS: 64 or 128 KB
  const int steps = (a.I + kStep - 1) / kStep;
  const int waves = 16;
  int parts = kLdsEntries / n;
  parts = parts < waves ? parts : waves;
  parts = parts < steps ? parts : steps;
  const unsigned blocks = (unsigned)(cap > 0 && tiles > cap ? cap : tiles);
  const size_t lds = (size_t)parts * n * RT * kTile * sizeof(float);
  ep_moe_down<WT, RT, MTMAX><<<blocks, waves * kWave, lds, a.stream>>>(
      ws.h, a.topk_idx, a.topk_weights, (const uint16_t *)a.bias, a.w_out, a.out_scales, a.T, a.H, a.I,
      a.K, a.E, rows, tiles, parts, ws.active, ws.list, ws.order, (uint16_t *)a.out);
  return launch_status();
}

template <int WT, int WIDE>
int moe_pick(const MoeLayerArgs &a, const MoeWorkspace &ws, int cap) {
  const bool few = a.T * a.K <= kTile;  // no expert can have a second token tile
  int rc;
  if (WIDE == 2) {
    rc = few ? moe_up_launch<WT, 2, 1>(a, ws, cap) : moe_up_launch<WT, 2, 4>(a, ws, cap);
  } else {
    const int n = a.T * a.K;
    const int64_t wide_units = (int64_t)(n < a.E ? n : a.E) * ((a.I + 31) / 32);
    const bool wide = wide_units >= 4 * kComputeUnits;
    if (wide) rc = few ? moe_up_launch<WT, WIDE, 1>(a, ws, cap) : moe_up_launch<WT, WIDE, 4>(a, ws, cap);
    else rc = few ? moe_up_launch<WT, 2, 1>(a, ws, cap) : moe_up_launch<WT, 2, 4>(a, ws, cap);
  }
  if (rc != 0) return rc;
  // Output rows per workgroup: an even share of the chip's 256 compute units, at most two tiles.
  int rows = (a.H + kComputeUnits - 1) / kComputeUnits;
  rows = (rows + 3) / 4 * 4;
  rows = rows < 2 * kTile ? rows : 2 * kTile;
  if (rows <= kTile)
    return few ? moe_down_launch<WT, 1, 1>(a, ws, cap, rows) : moe_down_launch<WT, 1, 2>(a, ws, cap, rows);
  return few ? moe_down_launch<WT, 2, 1>(a, ws, cap, rows) : moe_down_launch<WT, 2, 2>(a, ws, cap, rows);
}

}  // namespace

int launch_expert_matvec(const ExpertMatvecArgs &a) {
  if (a.capacity == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  if (a.dtype == EP_BF16) return matvec_pick<EP_BF16, 2>(a, cap);
  if (a.dtype == EP_FP8_E4M3) return matvec_pick<EP_FP8_E4M3, 2>(a, cap);
  return matvec_pick<EP_FP4X2, 4>(a, cap);
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
  if (a.dtype == EP_BF16) return moe_pick<EP_BF16, 2>(a, ws, cap);
  if (a.dtype == EP_FP8_E4M3) return moe_pick<EP_FP8_E4M3, 2>(a, ws, cap);
  return moe_pick<EP_FP4X2, 4>(a, ws, cap);
}

}  // namespace ep
