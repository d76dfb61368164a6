// The router on gfx950: from logits to expert ids, weights, per-expert counts
// and the balance and z losses (ep_router), and the logits' gradient
// (ep_router_backward).
//
// Mathematics. Scores s = softmax(l) or 1 / (1 + exp(-l)), probabilities p = s /
// sum(s). The choice is by l itself (both scorings grow with it) or by s +
// bias. Sigmoids are divided by exp(min(max l, 0)) before they are summed or
// compared with their sum, which keeps rows whose sigmoids all underflow; the
// factor cancels in every quotient. Losses need the sums of p over a sequence's
// tokens: a tile of tokens keeps them in registers and leaves one partial sum
// for each sequence that it meets in slot (tile + sequence), which no other
// pair has, since both only grow; a second launch adds a sequence's slots in order.
#include <type_traits>

#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

template <int L>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int d = 1; d < L; d *= 2) v = fmaxf(v, __shfl_xor(v, d));
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int d = 1; d < L; d *= 2) v += __shfl_xor(v, d);
  return v;
}

__device__ __forceinline__ float bf16_value(uint32_t bits) { return __uint_as_float(bits << 16); }
__device__ __forceinline__ uint32_t bf16_bits(float v) {
  return (uint32_t)__builtin_bit_cast(unsigned short, (__bf16)v);
}

// A row of up to L * V logits held by L lanes. Lane i's j-th value is column
// column(i, j): four neighbours per load where V allows.
template <int L, int V>
__device__ __forceinline__ int column(int i, int j) {
  constexpr int W = V < 4 ? V : 4;
  return j / W * (W * L) + i * W + j % W;
}

// The row's values; -infinity behind its end (and everywhere unless `on`).
template <bool FP32, int L, int V>
__device__ __forceinline__ void load_row(const void *x, int64_t row, int E, int i, bool on, float (&v)[V]) {
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] = -kInf;
  if (!on) return;
  if (V >= 4 && E % 4 == 0) {
#pragma unroll
    for (int j = 0; j < V; j += 4) {
      const int c = column<L, V>(i, j);
      if (c >= E) continue;
      if constexpr (FP32) {
        const f32x4 a = *(const f32x4 *)((const float *)x + row * E + c);
        v[j] = a[0];
        if constexpr (V >= 4) v[j + 1] = a[1], v[j + 2] = a[2], v[j + 3] = a[3];
      } else {
        const u32x2 a = *(const u32x2 *)((const uint16_t *)x + row * E + c);
        v[j] = bf16_value(a[0]);
        if constexpr (V >= 4)
          v[j + 1] = __uint_as_float(a[0] & 0xFFFF0000u), v[j + 2] = bf16_value(a[1]),
                v[j + 3] = __uint_as_float(a[1] & 0xFFFF0000u);
      }
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const int c = column<L, V>(i, j);
      if (c >= E) continue;
      if constexpr (FP32) v[j] = ((const float *)x)[row * E + c];
      else v[j] = bf16_value(((const uint16_t *)x)[row * E + c]);
    }
  }
}

template <bool FP32>
__device__ __forceinline__ float load_one(const void *x, int64_t at) {
  if constexpr (FP32) return ((const float *)x)[at];
  else return bf16_value(((const uint16_t *)x)[at]);
}

// exp(l - ref) for softmax; for sigmoids s(l) * exp(-ref), ref = min(the largest l, 0).
__device__ __forceinline__ float term(bool sigmoid, float l, float ref) {
  if (!sigmoid) return __expf(l - ref);
  return l >= 0.f ? 1.0f / (1.0f + __expf(-l)) : __expf(l - ref) / (1.0f + __expf(l));
}
__device__ __forceinline__ float reference(bool sigmoid, float top) {
  if (top == -kInf) return 0.f;  // nothing is above -infinity: every term is 0
  return sigmoid ? fminf(top, 0.f) : top;
}

// The sequence s with seq[s] <= t < seq[s + 1]: -1 before the first, S behind the last.
__device__ __forceinline__ int sequence_of(const int32_t *seq, int S, int t) {
  if (seq == nullptr) return 0;
  int lo = -1, hi = S + 1;  // seq[lo] <= t < seq[hi]
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    if (seq[mid] <= t) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct Slots {  // partial sums per (tile + sequence), then per sequence
  float *p;      // [slots, E]
  int *counts;   // [slots, E]
  float *z;      // [slots]
  int *tokens;   // [slots]
  double *seq_balance, *seq_z;  // [S]
};

// One row's K ids, by descending key and ascending id; lane i of the L keeps those of places i,
// i + L, ...: ids[b] is place b * L + i.
template <int L, int V, int KB>
__device__ __forceinline__ void choose(double (&key)[V], int i, int K, int (&ids)[KB]) {
#pragma unroll
  for (int b = 0; b < KB; ++b) {
    ids[b] = -1;
    for (int k = b * L; k < K && k < (b + 1) * L; ++k) {
      double best = -(double)kInf;
      int at = 1 << 30;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (key[j] > best) best = key[j], at = column<L, V>(i, j);
#pragma unroll
      for (int d = 1; d < L; d *= 2) {
        const double other = __shfl_xor(best, d);
        const int o = __shfl_xor(at, d);
        if (other > best || (other == best && o < at)) best = other, at = o;
      }
      if (k % L == i && best > -(double)kInf) ids[b] = at;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (column<L, V>(i, j) == at) key[j] = -(double)kInf;
    }
  }
}

template <bool FP32, int L, int V>
__global__ __launch_bounds__(kThreads) void ep_router_rows(const RouterArgs a, int tile_rows, int tiles,
                                                           Slots out) {
  constexpr int KB = 64 / L, kGroups = kThreads / L;
  __shared__ float sums[kGroups * L * V];
  __shared__ int hits[L * V];
  __shared__ float zs[kGroups];
  __shared__ int taken;
  const int i = threadIdx.x % L, group = threadIdx.x / L, E = a.E, K = a.K;
  const bool stats = a.counts != nullptr;
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int last = a.T - tile * tile_rows < tile_rows ? a.T : (tile + 1) * tile_rows;
    for (int pos = tile * tile_rows; pos < last;) {
      int s = 0, end = last;
      if (stats && a.seq != nullptr) {
        s = sequence_of(a.seq, a.S, pos);
        if (s < a.S) end = a.seq[s + 1] < last ? a.seq[s + 1] : last;
      }
      const bool inside = stats && s >= 0 && s < a.S;
      float acc[V], z = 0.f;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
      if (inside) {
        for (int c = threadIdx.x; c < E; c += kThreads) hits[c] = 0;
        if (threadIdx.x == 0) taken = 0;
        __syncthreads();
      }
      for (int first = pos; first < end; first += kGroups) {
        const int row = first + group;
        const bool on = row < end && (a.mask == nullptr || a.mask[row < end ? row : pos] != 0);
        const bool there = row < end;
        float v[V];
        load_row<FP32, L, V>(a.logits, row, E, i, on, v);
        float top = -kInf;
#pragma unroll
        for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
        top = lanes_max<L>(top);
        const float ref = reference(a.sigmoid, top);
        float e[V], total = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) e[j] = term(a.sigmoid, v[j], ref), total += e[j];
        total = lanes_sum<L>(total);
        int ids[KB];
        if (!a.given) {
          double key[V];
          if (a.bias == nullptr) {
#pragma unroll
            for (int j = 0; j < V; ++j) key[j] = v[j];
          } else {
            double sum = 0.0;
            const double m = ref;
#pragma unroll
            for (int j = 0; j < V; ++j) {
              key[j] = a.sigmoid ? 1.0 / (1.0 + exp(-(double)v[j])) : exp((double)v[j] - m);
              sum += key[j];
            }
#pragma unroll
            for (int d = 1; d < L; d *= 2) sum += __shfl_xor(sum, d);
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const int c = column<L, V>(i, j);
              const double bias = c < E ? a.bias[c] : 0.f;
              key[j] = v[j] == -kInf ? -(double)kInf : (a.sigmoid ? key[j] : key[j] / sum) + bias;
            }
          }
          choose<L, V, KB>(key, i, K, ids);
        } else {
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const int k = b * L + i;
            ids[b] = on && k < K ? a.idx[(int64_t)row * K + k] : -1;
            if ((uint32_t)ids[b] >= (uint32_t)E) ids[b] = -1;
          }
        }
        // weights, from the chosen logits
        float l[KB], most = -kInf;
        int any = 0;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          l[b] = ids[b] >= 0 ? load_one<FP32>(a.logits, (int64_t)row * E + ids[b]) : -kInf;
          most = fmaxf(most, l[b]);
          any |= ids[b] >= 0;
        }
        any = lanes_max<L>((float)any) > 0.f;
        if (there && (a.weights != nullptr || !a.given)) {
          const float from = reference(a.sigmoid, lanes_max<L>(most));
          float part = 0.f;
#pragma unroll
          for (int b = 0; b < KB; ++b)
            if (ids[b] >= 0) part += term(a.sigmoid, l[b], from);
          part = lanes_sum<L>(part);
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const int k = b * L + i;
            if (k >= K) continue;
            const int64_t at = (int64_t)row * K + k;
            if (!a.given) a.idx[at] = ids[b];
            if (a.weights == nullptr) continue;
            float w = 0.f;
            if (ids[b] >= 0) {
              if (a.normalize) w = part == 0.f ? 0.f : a.scale * (term(a.sigmoid, l[b], from) / part);
              else if (a.sigmoid) w = a.scale * term(true, l[b], 0.f);
              else w = total == 0.f ? 0.f : a.scale * (term(false, l[b], ref) / total);
            }
            a.weights[at] = w;
          }
        }
        if (inside && there && any) {
          const float by = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += e[j] * by;
          if (i == 0) {
            const float lse = top == -kInf ? 0.f : top + logf(total);
            z += lse * lse;
            atomicAdd(&taken, 1);
          }
#pragma unroll
          for (int b = 0; b < KB; ++b)
            if (ids[b] >= 0) atomicAdd(&hits[ids[b]], 1);
        }
      }
      if (inside) {
#pragma unroll
        for (int j = 0; j < V; ++j) sums[group * (L * V) + column<L, V>(i, j)] = acc[j];
        if (i == 0) zs[group] = z;
        __syncthreads();
        const int64_t slot = tile + s;
        for (int c = threadIdx.x; c < E; c += kThreads) {
          float sum = 0.f;
          for (int g = 0; g < kGroups; ++g) sum += sums[g * (L * V) + c];
          out.p[slot * E + c] = sum;
          out.counts[slot * E + c] = hits[c];
        }
        if (threadIdx.x == 0) {
          float sum = 0.f;
          for (int g = 0; g < kGroups; ++g) sum += zs[g];
          out.z[slot] = sum;
          out.tokens[slot] = taken;
        }
        __syncthreads();
      }
      pos = end;
    }
  }
}

__device__ __forceinline__ double block_sum(double v, double *lds) {
  __syncthreads();
  lds[threadIdx.x] = v;
  __syncthreads();
  for (int d = kThreads / 2; d > 0; d /= 2) {
    if ((int)threadIdx.x < d) lds[threadIdx.x] += lds[threadIdx.x + d];
    __syncthreads();
  }
  return lds[0];
}

// A sequence's slots: its counts, tokens and terms of the losses.
__global__ __launch_bounds__(kThreads) void ep_router_sequences(const RouterArgs a, int tile_rows, Slots in) {
  __shared__ double lds[kThreads];
  for (int s = blockIdx.x; s < a.S; s += gridDim.x) {
    int b = 0, e = a.T;
    if (a.seq != nullptr) {
      b = a.seq[s] < 0 ? 0 : a.seq[s];
      e = a.seq[s + 1] < a.T ? a.seq[s + 1] : a.T;
    }
    const int first = b < e ? b / tile_rows : 0, end = b < e ? (e - 1) / tile_rows + 1 : 0;
    int n = 0;
    double z = 0.0;
    for (int t = first; t < end; ++t) n += in.tokens[t + s], z += in.z[t + s];
    double sum = 0.0;
    for (int c = threadIdx.x; c < a.E; c += kThreads) {
      double p = 0.0;
      int hit = 0;
      for (int t = first; t < end; ++t) {
        const int64_t at = (int64_t)(t + s) * a.E + c;
        p += in.p[at], hit += in.counts[at];
      }
      a.counts[(int64_t)s * a.E + c] = hit;
      sum += hit * p;
    }
    sum = block_sum(sum, lds);
    if (threadIdx.x == 0) {
      a.seq_tokens[s] = n;
      in.seq_balance[s] = n > 0 ? sum * a.E / ((double)a.K * n * n) : 0.0;
      in.seq_z[s] = z;
    }
  }
}

// The losses from the sequences' terms.
__global__ __launch_bounds__(kThreads) void ep_router_losses(const RouterArgs a, Slots in) {
  __shared__ double lds[kThreads];
  double balance = 0.0, z = 0.0, full = 0.0, n = 0.0;
  for (int s = threadIdx.x; s < a.S; s += kThreads) {
    balance += in.seq_balance[s], z += in.seq_z[s];
    n += a.seq_tokens[s], full += a.seq_tokens[s] > 0;
  }
  balance = block_sum(balance, lds), z = block_sum(z, lds);
  n = block_sum(n, lds), full = block_sum(full, lds);
  if (threadIdx.x == 0) {
    a.seq_tokens[a.S] = (int)full, a.seq_tokens[a.S + 1] = (int)n;
    if (a.balance != nullptr) *a.balance = full > 0 ? (float)(balance / full) : 0.f;
    if (a.z != nullptr) *a.z = n > 0 ? (float)(z / n) : 0.f;
  }
}

template <bool FP32, int L, int V>
__global__ __launch_bounds__(kThreads) void ep_router_backward_rows(const RouterBackwardArgs a, int64_t steps) {
  constexpr int KB = 64 / L, kGroups = kThreads / L;
  __shared__ float extra[kGroups][L * V];
  const int i = threadIdx.x % L, group = threadIdx.x / L, E = a.E, K = a.K;
  float *const mine = extra[group];
#pragma unroll
  for (int j = 0; j < V; ++j) mine[column<L, V>(i, j)] = 0.f;
  const float db = a.d_balance != nullptr ? *a.d_balance : 0.f, dz = a.d_z != nullptr ? *a.d_z : 0.f;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t row = step * kGroups + group;
    const bool there = row < a.T;
    float v[V];
    load_row<FP32, L, V>(a.logits, row, E, i, there, v);
    int ids[KB], any = 0;
    float l[KB], dw[KB], most = -kInf;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      const int k = b * L + i;
      const bool in = there && k < K;
      ids[b] = in ? a.idx[row * K + k] : -1;
      if ((uint32_t)ids[b] >= (uint32_t)E) ids[b] = -1;
      l[b] = ids[b] >= 0 ? load_one<FP32>(a.logits, row * E + ids[b]) : -kInf;
      dw[b] = ids[b] >= 0 && a.d_weights != nullptr ? a.scale * a.d_weights[row * K + k] : 0.f;
      most = fmaxf(most, l[b]);
      any |= ids[b] >= 0;
    }
    any = lanes_max<L>((float)any) > 0.f;
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
    top = lanes_max<L>(top);
    const float ref = reference(a.sigmoid, top);
    float p[V], total = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] = term(a.sigmoid, v[j], ref), total += p[j];
    total = lanes_sum<L>(total);
    const float by = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
    for (int j = 0; j < V; ++j) p[j] *= by;
    // what an entry adds: to its logit (normalised weights and sigmoids), or to dp
    float d[KB];
    if (a.normalize) {
      const float from = reference(a.sigmoid, lanes_max<L>(most));
      float part = 0.f, dot = 0.f;
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        d[b] = ids[b] >= 0 ? term(a.sigmoid, l[b], from) : 0.f;
        part += d[b], dot += d[b] * dw[b];
      }
      part = lanes_sum<L>(part), dot = lanes_sum<L>(dot);
      const float share = part == 0.f ? 0.f : 1.0f / part;
#pragma unroll
      for (int b = 0; b < KB; ++b) {
        d[b] *= share * (dw[b] - dot * share);
        if (a.sigmoid) d[b] *= term(true, -l[b], 0.f);  // 1 - s(l) = s(-l)
      }
    } else {
#pragma unroll
      for (int b = 0; b < KB; ++b)
        d[b] = ids[b] < 0 ? 0.f : (a.sigmoid ? dw[b] * term(true, l[b], 0.f) * term(true, -l[b], 0.f) : dw[b]);
    }
    // the entries of an id are added in order, so that an id that occurs twice gets one sum
#pragma unroll
    for (int b = 0; b < KB; ++b)
      for (int k = 0; k < L && b * L + k < K; ++k) {
        if (i == k && ids[b] >= 0) mine[ids[b]] += d[b];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // keeps the lanes' turns apart
      }
    float out[V], dot = 0.f;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      out[j] = mine[column<L, V>(i, j)];
      dot += p[j] * out[j];
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
    for (int b = 0; b < KB; ++b)
      if (ids[b] >= 0) mine[ids[b]] = 0.f;
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (!a.sigmoid && !a.normalize) {
      dot = lanes_sum<L>(dot);
#pragma unroll
      for (int j = 0; j < V; ++j) out[j] = p[j] * (out[j] - dot);
    }
    const int s = a.counts != nullptr && there ? sequence_of(a.seq, a.S, (int)row) : -1;
    if (any && s >= 0 && s < a.S) {
      if (a.d_balance != nullptr) {
        const float n = (float)a.seq_tokens[s], full = (float)a.seq_tokens[a.S];
        const float f = n > 0.f && full > 0.f ? db * ((float)E / ((float)K * n * n * full)) : 0.f;
        float g[V], dot = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int c = column<L, V>(i, j);
          g[j] = c < E ? f * (float)a.counts[(int64_t)s * E + c] : 0.f;
          dot += p[j] * g[j];
        }
        dot = lanes_sum<L>(dot);
#pragma unroll
        for (int j = 0; j < V; ++j)
          out[j] += p[j] * (g[j] - dot) * (a.sigmoid ? term(true, -v[j], 0.f) : 1.0f);
      }
      if (a.d_z != nullptr && top != -kInf) {
        const float n = (float)a.seq_tokens[a.S + 1];
        const float f = n > 0.f ? 2.0f * dz / n * (top + logf(total)) : 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] += f * p[j];
      }
    }
    if (!there) continue;
    if (V >= 4 && E % 4 == 0) {
#pragma unroll
      for (int j = 0; j < V; j += 4) {
        const int c = column<L, V>(i, j);
        if (c >= E) continue;
        if constexpr (V >= 4) {
          if constexpr (FP32) {
            *(f32x4 *)((float *)a.d_logits + row * E + c) = f32x4{out[j], out[j + 1], out[j + 2], out[j + 3]};
          } else {
            *(u32x2 *)((uint16_t *)a.d_logits + row * E + c) =
                u32x2{bf16_bits(out[j]) | bf16_bits(out[j + 1]) << 16, bf16_bits(out[j + 2]) | bf16_bits(out[j + 3]) << 16};
          }
        }
      }
    } else {
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const int c = column<L, V>(i, j);
        if (c >= E) continue;
        if constexpr (FP32) ((float *)a.d_logits)[row * E + c] = out[j];
        else ((uint16_t *)a.d_logits)[row * E + c] = (uint16_t)bf16_bits(out[j]);
      }
    }
  }
}

int tile_rows_of(int) { return 64; }

int64_t slots_of(int T, int S) {
  const int rows = tile_rows_of(T);
  return (int64_t)(T + rows - 1) / rows + S;
}

int64_t up(int64_t n) { return (n + 15) & ~(int64_t)15; }

// f(L, V) for the smallest row of L lanes with V values each that holds E logits.
template <class F>
int for_shape(int E, F f) {
  if (E <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (E <= 32) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
  if (E <= 64) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
  if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
  if (E <= 256) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
  if (E <= 512) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
}

}  // namespace

size_t router_workspace(int T, int E, int S) {
  const int64_t slots = slots_of(T, S);
  return (size_t)(2 * up(slots * E * 4) + 2 * up(slots * 4) + 2 * up((int64_t)S * 8));
}

int launch_router(const RouterArgs &a) {
  const int cap = stream_workgroup_limit(a.stream);
  const int rows = tile_rows_of(a.T), tiles = (a.T + rows - 1) / rows;
  Slots w{};
  if (a.counts != nullptr) {
    const int64_t slots = slots_of(a.T, a.S);
    char *at = (char *)a.workspace;
    const auto take = [&](int64_t bytes) {
      char *p = at;
      at += up(bytes);
      return p;
    };
    w.seq_balance = (double *)take((int64_t)a.S * 8), w.seq_z = (double *)take((int64_t)a.S * 8);
    w.p = (float *)take(slots * a.E * 4), w.counts = (int *)take(slots * a.E * 4);
    w.z = (float *)take(slots * 4), w.tokens = (int *)take(slots * 4);
  }
  if (a.T > 0) {
    const unsigned grid = (unsigned)(cap > 0 && cap < tiles ? cap : tiles);
    const int rc = for_shape(a.E, [&](auto l, auto v) {
      if (a.fp32) ep_router_rows<true, decltype(l)::value, decltype(v)::value><<<grid, kThreads, 0, a.stream>>>(a, rows, tiles, w);
      else ep_router_rows<false, decltype(l)::value, decltype(v)::value><<<grid, kThreads, 0, a.stream>>>(a, rows, tiles, w);
      return launch_status();
    });
    if (rc != 0) return rc;
  }
  if (a.counts == nullptr) return 0;
  ep_router_sequences<<<(unsigned)(cap > 0 && cap < a.S ? cap : a.S), kThreads, 0, a.stream>>>(a, rows, w);
  if (const int rc = launch_status()) return rc;
  ep_router_losses<<<1, kThreads, 0, a.stream>>>(a, w);
  return launch_status();
}

int launch_router_backward(const RouterBackwardArgs &a) {
  if (a.T == 0) return 0;
  const int cap = stream_workgroup_limit(a.stream);
  return for_shape(a.E, [&](auto l, auto v) {
    constexpr int L = decltype(l)::value, V = decltype(v)::value;
    const int64_t steps = ((int64_t)a.T + kThreads / L - 1) / (kThreads / L);
    const int64_t most = cap > 0 ? cap : 1 << 22;
    const unsigned grid = (unsigned)(steps < most ? steps : most);
    if (a.fp32) ep_router_backward_rows<true, L, V><<<grid, kThreads, 0, a.stream>>>(a, steps);
    else ep_router_backward_rows<false, L, V><<<grid, kThreads, 0, a.stream>>>(a, steps);
    return launch_status();
  });
}

}  // namespace ep
