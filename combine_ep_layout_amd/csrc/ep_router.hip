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
//
// A row lies in 16 lanes (up to 256 experts; else in 64), so that a wave works on four at once and a
// maximum over a row takes four DPP steps. What bounds it: for few tokens the launch (128 tokens of 256 experts,
// 7 us under a trace, 8.5 with the host's time); for many the chain of a row's dependent steps, ten maxima of
// which each needs the last, at four waves a SIMD. Measured on MI355X, top-8 of 32768 tokens of 256 experts, fp32
// logits: without statistics 14.7 us (softmax), 20 (with a bias); with them 32 and, in 37 packed sequences, 43 to 47
// (37 and 7 in the two launches), of 1024 experts 96 to 102; of given ids 22. 4096 tokens 15.7. Backward 17 and 20.5
// us, 131072 tokens 58 (4.7 TB/s). Rows by the exact choice cost more: logits that are bf16 values (see Chooser) 46
// us without statistics and 92 with, top-16 of 256 experts 175 and top-32 340 (candidates for 16 lanes only). Steps:
// binary64 keys throughout 57 us for 128 tokens; statistics kept by workgroups of
// 1024 threads, whose registers spill, 144 against 65 us; candidates ranked again one maximum at a time in
// the rare near ties 77 against 20.6 us, since one such row holds up the launch.
#include <type_traits>

#include "ep_device.hpp"
#include "ep_launch.hpp"

namespace ep {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x4_any __attribute__((ext_vector_type(4), aligned(4)));  // a load takes any multiple of 4
typedef int i32x4_any __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kThreads = 256;
constexpr float kInf = __builtin_inff();

// Reductions over a row's L lanes (16 or 64; the same result in each of them). Within 16 lanes by DPP
// rotations, which stay there: all of a row's lanes have to take part, and the four rows of a wave may differ.
template <int N>
__device__ __forceinline__ int rotate(int v) {  // by N within 16 lanes
  constexpr int kRowRor = 0x120;
  return __builtin_amdgcn_update_dpp(0, v, kRowRor + N, 0xF, 0xF, false);
}
template <int L, class F>
__device__ __forceinline__ int over_lanes(int v, F f) {
  v = f(v, rotate<8>(v));
  v = f(v, rotate<4>(v));
  v = f(v, rotate<2>(v));
  v = f(v, rotate<1>(v));
  if constexpr (L == 64) {
    v = f(v, __shfl_xor(v, 16));
    v = f(v, __shfl_xor(v, 32));
  }
  return v;
}
template <int L>
__device__ __forceinline__ float lanes_max(float v) {
  return __int_as_float(over_lanes<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(fmaxf(__int_as_float(a), __int_as_float(b)));
  }));
}
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  return __int_as_float(over_lanes<L>(__float_as_int(v), [](int a, int b) {
    return __float_as_int(__int_as_float(a) + __int_as_float(b));
  }));
}
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  return (uint32_t)over_lanes<L>((int)v, [](int a, int b) { return (uint32_t)a > (uint32_t)b ? a : b; });
}
template <int L>
__device__ __forceinline__ bool lanes_any(bool p) {
  return lanes_max<L>((uint32_t)p) != 0;
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
        const f32x4_any a = *(const f32x4_any *)((const float *)x + row * E + c);
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

// exp(l - ref) for softmax; for sigmoids s(l) * exp(-ref), ref = min(the largest l, 0). Exponentials by
// the exp2 instruction, quotients by the reciprocal: (|l - ref| + 8) * 2^-23 relative at most.
__device__ __forceinline__ float term(bool sigmoid, float l, float ref) {
  if (!sigmoid) return __expf(l - ref);
  const float small = __expf(-fabsf(l)), by = __builtin_amdgcn_rcpf(1.0f + small);
  return l >= 0.f ? by : __expf(l - ref) * by;
}
__device__ __forceinline__ float reference(bool sigmoid, float top) {
  if (top == -kInf) return 0.f;  // nothing is above -infinity: every term is 0
  return sigmoid ? fminf(top, 0.f) : top;
}

// Terms of a row, and their sum in the calling lane. Sigmoids need a second exponential only in rows
// whose logits are all negative.
template <int V>
__device__ __forceinline__ float terms(bool sigmoid, const float (&v)[V], float ref, float (&e)[V]) {
  float total = 0.f;
  if (!sigmoid) {
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = __expf(v[j] - ref), total += e[j];
  } else if (ballot(ref < 0.f) == 0) {
#pragma unroll
    for (int j = 0; j < V; ++j) {
      const float small = __expf(-fabsf(v[j])), by = __builtin_amdgcn_rcpf(1.0f + small);
      e[j] = v[j] >= 0.f ? by : small * by;
      total += e[j];
    }
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) e[j] = term(true, v[j], ref), total += e[j];
  }
  return total;
}

// The sequence s with seq[s] <= t < seq[s + 1]: -1 before the first, S behind the last. L lanes look at L
// of the remaining offsets at a time.
template <int L>
__device__ __forceinline__ int sequence_by_lanes(const int32_t *seq, int S, int t, int i) {
  if (seq == nullptr) return 0;
  int lo = 0, n = S + 1;  // the first lo offsets are at most t, those from lo + n on are not
  while (ballot(n > 0) != 0) {
    const int step = (n + L - 1) / L, at = lo + i * step;
    const bool below = i * step < n && seq[i * step < n ? at : 0] <= t;
    const int found = over_lanes<L>((int)below, [](int a, int b) { return a + b; });
    const int left = n;
    if (found == 0) {
      n = 0;
    } else {
      const int skip = (found - 1) * step + 1;
      lo += skip, n = left - skip < step - 1 ? left - skip : step - 1;
    }
  }
  return lo - 1;
}

struct Slots {  // partial sums per (tile + sequence), then per sequence
  float *p;      // [slots, E]
  int *counts;   // [slots, E]
  float *z;      // [slots]
  int *tokens;   // [slots]
  double *balance;  // [S, parts]: terms of the balance loss
  double *seq_z;    // [S]
  unsigned *done;   // workgroups of the second launch that have left their terms
};

// The order of binary32 numbers as that of integers (-0 has to be +0), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float unordered(uint32_t u) {
  return __uint_as_float(u ^ (u >> 31 ? 0x80000000u : 0xFFFFFFFFu));
}

// Choice of a row's K largest keys, ties by ascending column.
//
// Fast: a key's upper bits and its column (descending) in one 31-bit number, so that a maximum is one integer
// instruction and names its column; x - m, as an unsigned number, puts what is still below the last
// maximum m on top. bf16 logits fit whole. Of binary32 keys the lower bits are lost: then K + 2
// candidates (K + 4 of scores + bias) are taken and ranked by their whole keys, and the choice stands if what
// was left out lies below the K-th whatever its lower bits are. Candidates' scores + bias that differ by no
// more than their rounding errors (one row in a thousand) are ranked again in binary64. With K + 2 of scores + bias
// one batch of 32768 tokens in two has a row that needs the exact choice, which holds up the launch (packed batch
// 44 us without such a row, 56 to 90 with one); K + 4 cost 1 us and left none in 8 batches of drawn logits and
// biases. Keys that are often equal need it more: binary32 logits that hold bf16 values, where three equal ones
// around the last place leave too few candidates although no bits are lost (about 175 of 32768 rows of 256 experts,
// 14.7 -> 46 us; with a bias of zeros 20 -> 37; of bf16 logits, 12.0, and continuous binary32 ones none).
// Exact: binary64 keys, one maximum at a time; for rows where what is left out may reach the K-th (many
// equal keys), for softmax + bias of rows that hold NaN or +infinity, and for more candidates than lanes.
template <int L, int V>
struct Chooser {
  static constexpr int kColumnBits = (L * V <= 16 ? 4 : L * V <= 32 ? 5 : L * V <= 64 ? 6 : L * V <= 128 ? 7 : L * V <= 256 ? 8 : L * V <= 512 ? 9 : 10);
  static constexpr uint32_t kColumns = (1u << kColumnBits) - 1;
  static constexpr int kLost = kColumnBits + 1;  // lower bits of a key

  // The packed number of a key; 0: not to be chosen.
  static __device__ __forceinline__ uint32_t pack(float key, int column) {
    const uint32_t u = ordered(key + 0.0f) >> kLost << kColumnBits | (kColumns - (uint32_t)column);
    return key > -kInf ? u : 0u;
  }
  // The largest C packed numbers: lane k has the k-th (0: none).
  static __device__ __forceinline__ uint32_t largest(const uint32_t (&x)[V], int C, int i) {
    uint32_t last = 0x80000000u, mine = 0;
    for (int k = 0; k < C; ++k) {
      uint32_t t[V];
#pragma unroll
      for (int j = 0; j < V; ++j) t[j] = x[j] - last;
#pragma unroll
      for (int n = V; n > 1; n = (n + 2) / 3) {  // maxima of three
#pragma unroll
        for (int j = 0; j < (n + 2) / 3; ++j) {
          uint32_t m = t[3 * j];
          if (3 * j + 1 < n) m = t[3 * j + 1] > m ? t[3 * j + 1] : m;
          if (3 * j + 2 < n) m = t[3 * j + 2] > m ? t[3 * j + 2] : m;
          t[j] = m;
        }
      }
      const uint32_t best = lanes_max<L>(t[0]) + last;
      if (k == i) mine = best;
      last = best > 1 ? best : 1;
    }
    return mine;
  }
  static __device__ __forceinline__ int column_of(uint32_t packed) { return (int)(kColumns - (packed & kColumns)); }
  // The key, if its lower bits are zeros.
  static __device__ __forceinline__ float whole(uint32_t packed) {
    return __uint_as_float(__float_as_uint(unordered(packed >> kColumnBits << kLost)) >> kLost << kLost);
  }
  // A number that no key with this packed number exceeds.
  static __device__ __forceinline__ float at_most(uint32_t packed) {
    return unordered(packed >> kColumnBits << kLost | ((1u << kLost) - 1));
  }

  // f(key, column) of the row's other candidates.
  template <class T, class F>
  static __device__ __forceinline__ void others(T key, int column, int C, F f) {
    const auto rotated = [](T k, auto n) {
      if constexpr (sizeof(T) == 4) {
        return __int_as_float(rotate<decltype(n)::value>(__float_as_int(k)));
      } else {
        const uint64_t v = __builtin_bit_cast(uint64_t, k);
        const uint32_t lo = (uint32_t)rotate<decltype(n)::value>((int)(uint32_t)v), hi = (uint32_t)rotate<decltype(n)::value>((int)(v >> 32));
        return __builtin_bit_cast(T, (uint64_t)hi << 32 | lo);
      }
    };
    if constexpr (L == 16) {
#define EP_OTHER(N) f(rotated(key, std::integral_constant<int, N>()), rotate<N>(column));
      EP_OTHER(1) EP_OTHER(2) EP_OTHER(3) EP_OTHER(4) EP_OTHER(5) EP_OTHER(6) EP_OTHER(7) EP_OTHER(8)
      EP_OTHER(9) EP_OTHER(10) EP_OTHER(11) EP_OTHER(12) EP_OTHER(13) EP_OTHER(14) EP_OTHER(15)
#undef EP_OTHER
    } else {
      for (int c = 0; c < C; ++c) {
        if constexpr (sizeof(T) == 4) {
          f(read_lane(key, c), read_lane(column, c));
        } else {
          const uint64_t v = __builtin_bit_cast(uint64_t, key);
          const uint32_t lo = (uint32_t)read_lane((int)(uint32_t)v, c), hi = (uint32_t)read_lane((int)(v >> 32), c);
          f(__builtin_bit_cast(T, (uint64_t)hi << 32 | lo), read_lane(column, c));
        }
      }
    }
  }
  // Rank of this lane's (key, column) among the row's lanes, and whether another key is within `near`.
  template <class T>
  static __device__ __forceinline__ int rank(T key, int column, int C, float near, bool &close) {
    int r = 0;
    others(key, column, C, [&](T k, int c) {
      r += k > key || (k == key && c < column);
      if constexpr (sizeof(T) == 4) close |= fabsf(k - key) <= near && c != column;
    });
    return r;
  }

  // Exact: ids[b] of lane i is place b * L + i (-1: none left). Rare, so it reads the row again for every
  // maximum instead of keeping binary64 keys in registers.
  template <bool FP32, int KB>
  static __device__ __forceinline__ void exactly(const RouterArgs &a, int64_t row, bool on, float ref, int i, int (&ids)[KB]) {
    // softmax's term; `ref` is infinite if the row's largest logit is
    const auto part = [&](float l) { return ref == kInf ? (double)(l == kInf) : exp((double)l - (double)ref); };
    double sum = 1.0;
    if (a.bias != nullptr && !a.sigmoid) {
      sum = 0.0;
#pragma unroll 1
      for (int j = 0; j < V; ++j) {
        const int c = column<L, V>(i, j);
        const float l = on && c < a.E ? load_one<FP32>(a.logits, row * a.E + c) : -kInf;
        if (l > -kInf) sum += part(l);
      }
#pragma unroll
      for (int d = 1; d < L; d *= 2) sum += __shfl_xor(sum, d);
    }
    double last = (double)kInf;
    int last_at = -1;
#pragma unroll
    for (int b = 0; b < KB; ++b) {
      ids[b] = -1;
      for (int k = b * L; k < a.K && k < (b + 1) * L; ++k) {
        double best = -(double)kInf;
        int at = 1 << 30;
#pragma unroll 1
        for (int j = 0; j < V; ++j) {
          const int c = column<L, V>(i, j);
          if (!on || c >= a.E) continue;
          const float l = load_one<FP32>(a.logits, row * a.E + c);
          if (!(l > -kInf)) continue;
          double key = l;
          if (a.bias != nullptr)
            key = (a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : part(l) / sum) + (double)a.bias[c];
          // what comes behind the last one, and before the best so far
          if ((key < last || (key == last && c > last_at)) && key > best) best = key, at = c;
        }
#pragma unroll
        for (int d = 1; d < L; d *= 2) {
          const double other = __shfl_xor(best, d);
          const int o = __shfl_xor(at, d);
          if (other > best || (other == best && o < at)) best = other, at = o;
        }
        if (k % L == i && best > -(double)kInf) ids[b] = at;
        last = best, last_at = at;
      }
    }
  }
};

constexpr int kMostOf16 = 256;                // experts of a row in 16 lanes
constexpr int kPerUnit16 = 3, kPerUnit64 = 4;  // workgroups with statistics on a compute unit, as registers allow

template <bool FP32, bool STATS, int L, int V, int KB>
__global__ __launch_bounds__(kThreads, STATS && L == 16 ? kPerUnit16 : kPerUnit64) void ep_router_rows(const RouterArgs a, int tile_rows, int tiles,
                                                              Slots out) {
  using Choice = Chooser<L, V>;
  constexpr int kWaves = kThreads / kWave;
  __shared__ float sums[STATS ? kWaves : 1][STATS ? L * V : 1];
  __shared__ int hits[STATS ? L * V : 1];
  __shared__ float zs[kWaves];
  __shared__ int taken[kWaves];
  const int i = threadIdx.x % L, group = threadIdx.x / L, groups = blockDim.x / L, E = a.E, K = a.K;
  constexpr bool stats = STATS;
  const bool packed_whole = !FP32 && a.bias == nullptr;  // no key bits are lost
  const int wish = a.bias != nullptr && K + 4 <= L ? K + 4 : K + 2;
  const int candidates = packed_whole ? K : (wish < E ? wish : E);
  const bool fast = candidates <= L;
  const bool all_terms = stats || a.bias != nullptr || !(a.normalize || a.sigmoid);
  if (stats && blockIdx.x == 0 && threadIdx.x == 0) *out.done = 0;  // for the next launch
  for (int tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const int last = a.T - tile * tile_rows < tile_rows ? a.T : (tile + 1) * tile_rows;
    for (int pos = tile * tile_rows; pos < last;) {
      int s = 0, end = last;
      if (stats && a.seq != nullptr) {
        s = __builtin_amdgcn_readfirstlane(sequence_by_lanes<L>(a.seq, a.S, pos, i));
        if (s < a.S) end = a.seq[s + 1] < last ? a.seq[s + 1] : last;
        if (end <= pos) end = pos + 1;  // offsets that do not ascend
      }
      const bool inside = STATS && s >= 0 && s < a.S;
      float acc[V], z = 0.f;
      int count = 0;
#pragma unroll
      for (int j = 0; j < V; ++j) acc[j] = 0.f;
      if (STATS && inside) {
        for (int c = threadIdx.x; c < E; c += blockDim.x) hits[c] = 0;
        __syncthreads();
      }
      for (int first = pos; first < end; first += groups) {
        const int row = first + group;
        const bool there = row < end, on = there && (a.mask == nullptr || a.mask[there ? row : pos] != 0);
        float v[V];
        load_row<FP32, L, V>(a.logits, row, E, i, there, v);  // whatever the mask says, which is still on its way
        if (!on) {
#pragma unroll
          for (int j = 0; j < V; ++j) v[j] = -kInf;
        }
        float top = -kInf, total = 0.f, ref = 0.f;
        float e[V];
        if (all_terms) {
#pragma unroll
          for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
          top = lanes_max<L>(top);
          ref = reference(a.sigmoid, top);
          total = lanes_sum<L>(terms(a.sigmoid, v, ref, e));
        }
        int ids[KB], places[KB];  // of this lane
        float chosen = -kInf;     // logit of ids[0], if `known`
        bool known = false;
#pragma unroll
        for (int b = 0; b < KB; ++b) places[b] = b * L + i, ids[b] = -1;
        if (!a.given) {
          const float back = a.sigmoid ? (ref < 0.f ? __expf(ref) : 1.0f) : (total == 0.f ? 0.f : 1.0f / total);
          bool unsure = !fast;
          if (fast) {
            uint32_t x[V];
            if (a.bias == nullptr) {
#pragma unroll
              for (int j = 0; j < V; ++j) x[j] = Choice::pack(v[j], column<L, V>(i, j));
            } else {
              float bias[V];
              load_row<true, L, V>(a.bias, 0, E, i, true, bias);
#pragma unroll
              for (int j = 0; j < V; ++j) x[j] = Choice::pack(v[j] > -kInf ? e[j] * back + bias[j] : -kInf, column<L, V>(i, j));
            }
            const uint32_t mine = Choice::largest(x, candidates, i);
            const bool valid = mine != 0 && i < candidates;
            ids[0] = valid ? Choice::column_of(mine) : -1;
            known = true;
            if (packed_whole) {
              chosen = Choice::whole(mine);
            } else {
              float key = -kInf, near = -1.0f;
              if (valid) {
                key = chosen = load_one<FP32>(a.logits, (int64_t)row * E + ids[0]);
                if (a.bias != nullptr) {
                  // errors of scores: 16 * 2^-23 for sigmoids; 128 * 2^-23 of the largest probability
                  const float most = fabsf(Choice::at_most(mine));
                  near = (a.sigmoid ? 0x1p-19f : 0x1p-16f * back) + 0x1p-21f * most;
                  key = term(a.sigmoid, key, ref) * back + a.bias[ids[0]];
                }
              }
              bool close = false;
              places[0] = Choice::rank(key, valid ? ids[0] : E + i, candidates, near, close);
              // what was left out lies below the last candidate's packed number
              const uint32_t left = (uint32_t)__shfl((int)mine, (int)(threadIdx.x & (kWave - 1)) / L * L + candidates - 1);
              const bool rest = candidates < E && left != 0;
              unsure = valid && rest && places[0] == K - 1 && !(key > Choice::at_most(left) + fmaxf(near, 0.f));
              if (ballot(close && valid && places[0] <= K) != 0) {  // only with a bias: the candidates again, in binary64
                double sum = 1.0;
                if (!a.sigmoid) {
                  sum = 0.0;
#pragma unroll
                  for (int j = 0; j < V; ++j) sum += exp((double)v[j] - (double)ref);
#pragma unroll
                  for (int d = 1; d < L; d *= 2) sum += __shfl_xor(sum, d);
                }
                double exact = -(double)kInf;
                if (valid) {
                  const double l = chosen;
                  exact = (a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)ref) / sum) + (double)a.bias[ids[0]];
                }
                places[0] = Choice::rank(exact, valid ? ids[0] : E + i, candidates, near, close);
              }
              if (places[0] >= K) ids[0] = -1;
              if (a.bias != nullptr && !a.sigmoid) unsure |= total != total;  // NaN or +infinity among the logits: no keys
            }
          }
          unsure = lanes_any<L>(unsure && there);
          if (ballot(unsure) != 0) {
            known = false;
            int exact[KB];
            Choice::template exactly<FP32, KB>(a, row, on, ref, i, exact);
            if (unsure) {
#pragma unroll
              for (int b = 0; b < KB; ++b) ids[b] = exact[b], places[b] = b * L + i;
            }
          }
        } else {
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            const int k = b * L + i;
            if (on && k < K) ids[b] = a.idx[(int64_t)row * K + k];
            if ((uint32_t)ids[b] >= (uint32_t)E) ids[b] = -1;
          }
        }
        // weights, from the chosen logits
        float l[KB], w[KB], most = -kInf;
        bool any = false;
#pragma unroll
        for (int b = 0; b < KB; ++b) {
          if (ids[b] >= 0 && !there) ids[b] = -1;
          l[b] = -kInf;
          if (ids[b] >= 0) l[b] = known && b == 0 ? chosen : load_one<FP32>(a.logits, (int64_t)row * E + ids[b]);
          most = fmaxf(most, l[b]);
          any |= ids[b] >= 0;
        }
        any = lanes_any<L>(any);
        if (a.normalize) {
          const float from = reference(a.sigmoid, lanes_max<L>(most));
          float part = 0.f;
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            w[b] = ids[b] >= 0 ? term(a.sigmoid, l[b], from) : 0.f;
            part += w[b];
          }
          part = lanes_sum<L>(part);
          const float by = part == 0.f ? 0.f : a.scale / part;
#pragma unroll
          for (int b = 0; b < KB; ++b) w[b] = ids[b] >= 0 ? w[b] * by : 0.f;
        } else {
          const float by = a.sigmoid ? a.scale : (total == 0.f ? 0.f : a.scale / total);
#pragma unroll
          for (int b = 0; b < KB; ++b) w[b] = ids[b] >= 0 ? by * term(a.sigmoid, l[b], a.sigmoid ? 0.f : ref) : 0.f;
        }
        if (there) {
#pragma unroll
          for (int b = 0; b < KB; ++b) {
            if (places[b] >= K) continue;
            const int64_t at = (int64_t)row * K + places[b];
            if (!a.given) a.idx[at] = ids[b];
            if (a.weights != nullptr) a.weights[at] = w[b];
          }
        }
        if (STATS && inside && any) {
          const float by = total == 0.f ? 0.f : 1.0f / total;
#pragma unroll
          for (int j = 0; j < V; ++j) acc[j] += e[j] * by;
          const float lse = top == -kInf ? 0.f : top + logf(total);
          z += lse * lse;
          ++count;
#pragma unroll
          for (int b = 0; b < KB; ++b)
            if (ids[b] >= 0) atomicAdd(&hits[ids[b]], 1);
        }
      }
      if (STATS && inside) {
        // a wave's rows first, then the waves in order
        const int wave = threadIdx.x / kWave;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          if constexpr (L == 16) {
            acc[j] += __shfl_xor(acc[j], 16);
            acc[j] += __shfl_xor(acc[j], 32);
          }
          if ((threadIdx.x & (kWave - 1)) < L) sums[wave][column<L, V>(i, j)] = acc[j];
        }
        if constexpr (L == 16) {
          z += __shfl_xor(z, 16), count += __shfl_xor(count, 16);
          z += __shfl_xor(z, 32), count += __shfl_xor(count, 32);
        }
        if ((threadIdx.x & (kWave - 1)) == 0) zs[wave] = z, taken[wave] = count;
        __syncthreads();
        const int64_t slot = tile + s;
        const int waves = blockDim.x / kWave;
        for (int c = threadIdx.x; c < E; c += blockDim.x) {
          float sum = 0.f;
          for (int g = 0; g < waves; ++g) sum += sums[g][c];
          out.p[slot * E + c] = sum;
          out.counts[slot * E + c] = hits[c];
        }
        if (threadIdx.x == 0) {
          float sum = 0.f;
          int n = 0;
          for (int g = 0; g < waves; ++g) sum += zs[g], n += taken[g];
          out.z[slot] = sum;
          out.tokens[slot] = n;
        }
        __syncthreads();
      }
      pos = end;
    }
  }
}

// Sums over a workgroup, in a fixed order.
template <int N>
__device__ __forceinline__ void block_sums(double (&v)[N], double (&lds)[N][kThreads / kWave]) {
#pragma unroll
  for (int d = 1; d < kWave; d *= 2)
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] += __shfl_xor(v[n], d);
  __syncthreads();
  if ((threadIdx.x & (kWave - 1)) == 0)
#pragma unroll
    for (int n = 0; n < N; ++n) lds[n][threadIdx.x / kWave] = v[n];
  __syncthreads();
#pragma unroll
  for (int n = 0; n < N; ++n) {
    v[n] = lds[n][0];
#pragma unroll
    for (int w = 1; w < kThreads / kWave; ++w) v[n] += lds[n][w];
  }
}

// Visible to workgroups of other XCDs, whose L2 is another.
__device__ __forceinline__ void publish(double *p, double v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ void publish(int *p, int v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
template <class T>
__device__ __forceinline__ T published(const T *p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// The slots of a sequence: its counts and tokens, and terms of the losses, `parts` workgroups a sequence with
// LANES columns at a time each. The last workgroup to leave its terms adds them all, in order. The workgroup's
// threads are LANES columns by slots.
template <int LANES>
__global__ __launch_bounds__(kThreads) void ep_router_sequences(const RouterArgs a, int tile_rows, Slots in, int parts) {
  constexpr int kRows = kThreads / LANES, kWaves = kThreads / kWave;
  __shared__ double lds[4][kWaves];
  __shared__ double sums[kWaves][LANES];
  __shared__ int hits[kWaves][LANES];
  __shared__ bool last;
  const int r = threadIdx.x / LANES, i = threadIdx.x % LANES, wave = threadIdx.x / kWave, units = a.S * parts;
  int mine = 0;
  for (int u = blockIdx.x; u < units; u += gridDim.x, ++mine) {
    const int s = u / parts, part = u % parts;
    int b = 0, e = a.T;
    if (a.seq != nullptr) {
      b = a.seq[s] < 0 ? 0 : a.seq[s];
      e = a.seq[s + 1] < a.T ? a.seq[s + 1] : a.T;
    }
    const int first = b < e ? b / tile_rows : 0, end = b < e ? (e - 1) / tile_rows + 1 : 0;
    const int c = part * LANES + i;
    double p = 0.0, n = 0.0, z = 0.0;
    int hit = 0;
    if (c < a.E) {
#pragma unroll 8
      for (int t = first + r; t < end; t += kRows) {
        const int64_t at = (int64_t)(t + s) * a.E + c;
        p += in.p[at], hit += in.counts[at];
      }
    }
    if (part == 0)
      for (int t = first + threadIdx.x; t < end; t += kThreads) n += in.tokens[t + s], z += in.z[t + s];
#pragma unroll
    for (int d = LANES; d < kWave; d *= 2) p += __shfl_xor(p, d), hit += __shfl_xor(hit, d);
    __syncthreads();
    if ((threadIdx.x & (kWave - 1)) < LANES) sums[wave][i] = p, hits[wave][i] = hit;
    __syncthreads();
    double sum = 0.0;
    if (threadIdx.x < LANES && c < a.E) {
#pragma unroll
      for (int w = 1; w < kWaves; ++w) p += sums[w][i], hit += hits[w][i];
      a.counts[(int64_t)s * a.E + c] = hit;
      sum = hit * p;
    }
    double v[4] = {sum, n, z, 0.0};
    block_sums(v, lds);
    if (threadIdx.x == 0) {
      publish(&in.balance[u], v[0]);
      if (part == 0) publish(&in.seq_z[s], v[2]), publish(&a.seq_tokens[s], (int)v[1]);
    }
  }
  if (threadIdx.x == 0) {
    // What this thread has published has left for all when its stores are done, on this chip: relaxed stores of agent
    // scope are written through, and this wait is for them. That is no order of the memory model, and holds for this
    // thread's published values only: a value that the last workgroup is to read from other threads (a.counts, say)
    // needs a release here, with its write-back of L2 (2.7 of 10.3 us for 37 sequences).
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    last = __hip_atomic_fetch_add(in.done, (unsigned)mine, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) + (unsigned)mine == (unsigned)units;
  }
  __syncthreads();
  if (!last) return;
  double v[4] = {0.0, 0.0, 0.0, 0.0};  // balance, z, sequences with tokens, tokens
  for (int u = threadIdx.x; u < units; u += kThreads) {
    const double tokens = published(&a.seq_tokens[u / parts]);
    const double term = published(&in.balance[u]);
    if (tokens > 0) v[0] += term * a.E / (a.K * tokens * tokens);
  }
  for (int s = threadIdx.x; s < a.S; s += kThreads) {
    const int tokens = published(&a.seq_tokens[s]);
    v[1] += published(&in.seq_z[s]), v[2] += tokens > 0, v[3] += tokens;
  }
  block_sums(v, lds);
  if (threadIdx.x == 0) {
    a.seq_tokens[a.S] = (int)v[2], a.seq_tokens[a.S + 1] = (int)v[3];
    if (a.balance != nullptr) *a.balance = v[2] > 0 ? (float)(v[0] / v[2]) : 0.f;
    if (a.z != nullptr) *a.z = v[3] > 0 ? (float)(v[1] / v[3]) : 0.f;
  }
}

// KB: places of a token's ids per lane.
template <bool FP32, int L, int V, int KB>
__global__ __launch_bounds__(kThreads) void ep_router_backward_rows(const RouterBackwardArgs a, int64_t steps) {
  constexpr int kGroups = kThreads / L;
  __shared__ float extra[kGroups][L * V];
  const int i = threadIdx.x % L, group = threadIdx.x / L, E = a.E, K = a.K;
  float *const mine = extra[group];
#pragma unroll
  for (int j = 0; j < V; ++j) mine[column<L, V>(i, j)] = 0.f;
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // other lanes add to these columns
  const float db = a.d_balance != nullptr ? *a.d_balance : 0.f, dz = a.d_z != nullptr ? *a.d_z : 0.f;
  for (int64_t step = blockIdx.x; step < steps; step += gridDim.x) {
    const int64_t row = step * kGroups + group;
    const bool there = row < a.T;
    float v[V];
    load_row<FP32, L, V>(a.logits, row, E, i, there, v);
    const int s = a.counts != nullptr ? sequence_by_lanes<L>(a.seq, a.S, (int)(there ? row : 0), i) : -1;
    int ids[KB];
    bool any = false;
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
    any = lanes_any<L>(any);
    float top = -kInf;
#pragma unroll
    for (int j = 0; j < V; ++j) top = fmaxf(top, v[j]);
    top = lanes_max<L>(top);
    const float ref = reference(a.sigmoid, top);
    float p[V], total = 0.f;
    total = lanes_sum<L>(terms(a.sigmoid, v, ref, p));
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
    // The entries of an id are added by the first of them, in a fixed order.
    if constexpr (KB == 1) {
      float sum = 0.f;
      bool mine_first = true;
      if constexpr (L == 16) {
        const auto with = [&](float v, int id, int lane) {
          if (id != ids[0]) return;
          sum += v;
          mine_first &= lane >= i;
        };
        with(d[0], ids[0], i);
#define EP_WITH(N) with(__int_as_float(rotate<N>(__float_as_int(d[0]))), rotate<N>(ids[0]), rotate<N>(i));
        EP_WITH(1) EP_WITH(2) EP_WITH(3) EP_WITH(4) EP_WITH(5) EP_WITH(6) EP_WITH(7) EP_WITH(8)
        EP_WITH(9) EP_WITH(10) EP_WITH(11) EP_WITH(12) EP_WITH(13) EP_WITH(14) EP_WITH(15)
#undef EP_WITH
      } else {
        for (int k = 0; k < K; ++k) {
          if (read_lane(ids[0], k) != ids[0]) continue;
          sum += read_lane(d[0], k);
          mine_first &= k >= i;
        }
      }
      if (ids[0] >= 0 && mine_first) mine[ids[0]] = sum;
    } else {
#pragma unroll
      for (int b = 0; b < KB; ++b)
        for (int k = 0; k < L && b * L + k < K; ++k) {
          if (i == k && ids[b] >= 0) mine[ids[b]] += d[b];
          __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");  // keeps the lanes' turns apart
        }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
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
      if (any) {  // else out is 0, and p may be of anything: a row of padding
#pragma unroll
        for (int j = 0; j < V; ++j) out[j] = p[j] * (out[j] - dot);
      }
    }
    if (any && s >= 0 && s < a.S) {
      if (a.d_balance != nullptr) {
        const float n = (float)a.seq_tokens[s], full = (float)a.seq_tokens[a.S];
        const float f = n > 0.f && full > 0.f ? db * ((float)E / ((float)K * n * n * full)) : 0.f;
        float g[V], dot = 0.f;
        if (V >= 4 && E % 4 == 0) {
#pragma unroll
          for (int j = 0; j < V; j += 4) {
            const int c = column<L, V>(i, j);
            i32x4_any n = {0, 0, 0, 0};
            if (c < E) n = *(const i32x4_any *)(a.counts + (int64_t)s * E + c);
#pragma unroll
            for (int k = 0; k < 4 && j + k < V; ++k) g[j + k] = f * (float)n[k];
          }
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int c = column<L, V>(i, j);
            g[j] = c < E ? f * (float)a.counts[(int64_t)s * E + c] : 0.f;
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) dot += p[j] * g[j];
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

// Tokens per tile, and so per slot: as few sixteens as leave no more tiles than workgroups run at once, three
// or four a compute unit (powers of two up to 1024 tiles: 32768 tokens of 256 experts 36 us instead of 32.6,
// 131072 95 instead of 85; 768 tiles of 1024 experts 116 instead of 106), and at most 256.
constexpr int kMostSixteens = 16;
int tiles_at_once(int E) { return (E <= kMostOf16 ? kPerUnit16 : kPerUnit64) * 256; }
int tile_rows_of(int T, int E) {
  const int at_once = tiles_at_once(E);
  const int64_t sixteens = ((int64_t)T + 16 * at_once - 1) / (16 * at_once);
  return 16 * (int)(sixteens < 1 ? 1 : (sixteens < kMostSixteens ? sixteens : kMostSixteens));
}

// Columns per workgroup of the second launch: the fewer, the more slots a sequence has.
constexpr int kManySlots = 256, kSomeSlots = 64;
int lanes_of(int64_t tiles, int S) {
  const int64_t slots = tiles / S;
  return slots >= kManySlots ? 4 : (slots >= kSomeSlots ? 16 : 64);
}

struct Sizes {
  int tile_rows, tiles, lanes, parts;
  int64_t slots;
};
Sizes sizes_of(int T, int E, int S) {
  Sizes z;
  z.tile_rows = tile_rows_of(T, E);
  z.tiles = (int)(((int64_t)T + z.tile_rows - 1) / z.tile_rows);
  z.slots = (int64_t)z.tiles + S;
  z.lanes = lanes_of(z.tiles, S);
  z.parts = (E + z.lanes - 1) / z.lanes;
  return z;
}

int64_t up(int64_t n) { return (n + 15) & ~(int64_t)15; }

size_t workspace_of(int64_t slots, int E, int S, int64_t terms) {
  return (size_t)(2 * up(slots * E * 4) + 2 * up(slots * 4) + up(terms * 8) + up((int64_t)S * 8) + up(4));
}

// f(L, V) for the smallest row of L lanes with V values each that holds E logits.
template <class F>
int for_shape(int E, F f) {
  if (E <= 16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 1>());
  if (E <= 32) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 2>());
  if (E <= 64) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 4>());
  if (E <= 128) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 8>());
  if (E <= kMostOf16) return f(std::integral_constant<int, 16>(), std::integral_constant<int, 16>());
  if (E <= 512) return f(std::integral_constant<int, 64>(), std::integral_constant<int, 8>());
  return f(std::integral_constant<int, 64>(), std::integral_constant<int, 16>());
}

}  // namespace

size_t router_workspace(int T, int E, int S) {
  const Sizes z = sizes_of(T, E, S);
  return workspace_of(z.slots, E, S, (int64_t)S * z.parts);
}

// What no call of at most T tokens, E experts and S sequences exceeds. Tiles jump down where their rows go up by
// 16, and terms of the losses where sequences get fewer slots, so a call may need less than a smaller one.
size_t router_workspace_most(int T, int E, int S) {
  const int64_t sixteens = ((int64_t)T + 15) / 16, at_once = tiles_at_once(E);
  const int64_t tall = (sixteens + kMostSixteens - 1) / kMostSixteens, some = at_once > tall ? at_once : tall;
  const int64_t tiles = sixteens < some ? sixteens : some;
  int64_t terms = 0;
  for (const int lanes : {4, 16, 64}) {  // of as many sequences as get so few columns a workgroup
    const int64_t most = lanes == 64 ? S : tiles / (lanes == 4 ? kManySlots : kSomeSlots);
    const int64_t n = (most < S ? most : S) * ((E + lanes - 1) / lanes);
    terms = n > terms ? n : terms;
  }
  return workspace_of(tiles + S, E, S, terms);
}

int launch_router(const RouterArgs &a) {
  const int cap = stream_workgroup_limit(a.stream);
  const Sizes z = sizes_of(a.T, a.E, a.S);
  Slots w{};
  if (a.counts != nullptr) {
    char *at = (char *)a.workspace;
    const auto take = [&](int64_t bytes) {
      char *p = at;
      at += up(bytes);
      return p;
    };
    w.balance = (double *)take((int64_t)a.S * z.parts * 8), w.seq_z = (double *)take((int64_t)a.S * 8);
    w.p = (float *)take(z.slots * a.E * 4), w.counts = (int *)take(z.slots * a.E * 4);
    w.z = (float *)take(z.slots * 4), w.tokens = (int *)take(z.slots * 4);
    w.done = (unsigned *)take(4);
  }
  if (a.T > 0 || a.counts != nullptr) {
    const int rc = for_shape(a.E, [&](auto l, auto v) {
      constexpr int L = decltype(l)::value, V = decltype(v)::value;
      // Without statistics a wave on its own is enough: more workgroups for a few tokens.
      const int threads = a.counts != nullptr || cap > 0 ? kThreads : kWave;
      const int rows = a.counts != nullptr ? z.tile_rows : threads / L;
      const int n = (int)(((int64_t)a.T + rows - 1) / rows), most = cap > 0 ? cap : 1 << 20;
      const unsigned grid = (unsigned)(n < most ? (n > 0 ? n : 1) : most);
      const auto run = [&](auto kernel) {
        kernel<<<grid, threads, 0, a.stream>>>(a, rows, n, w);
        return launch_status();
      };
      const auto with = [&](auto stats, auto places) {
        constexpr bool S = decltype(stats)::value;
        constexpr int KB = decltype(places)::value;
        return a.fp32 ? run(ep_router_rows<true, S, L, V, KB>) : run(ep_router_rows<false, S, L, V, KB>);
      };
      constexpr std::integral_constant<int, 1> one{};
      constexpr std::integral_constant<int, 64 / L> all{};
      if (a.counts != nullptr) return a.K <= L ? with(std::true_type(), one) : with(std::true_type(), all);
      return a.K <= L ? with(std::false_type(), one) : with(std::false_type(), all);
    });
    if (rc != 0) return rc;
  }
  if (a.counts == nullptr) return 0;
  const int64_t units = (int64_t)a.S * z.parts, most = cap > 0 ? cap : 1 << 20;
  const unsigned grid = (unsigned)(units < most ? units : most);
  if (z.lanes == 4) ep_router_sequences<4><<<grid, kThreads, 0, a.stream>>>(a, z.tile_rows, w, z.parts);
  else if (z.lanes == 16) ep_router_sequences<16><<<grid, kThreads, 0, a.stream>>>(a, z.tile_rows, w, z.parts);
  else ep_router_sequences<64><<<grid, kThreads, 0, a.stream>>>(a, z.tile_rows, w, z.parts);
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
    const auto run = [&](auto kernel) {
      kernel<<<grid, kThreads, 0, a.stream>>>(a, steps);
      return launch_status();
    };
    if (a.K <= L) return a.fp32 ? run(ep_router_backward_rows<true, L, V, 1>) : run(ep_router_backward_rows<false, L, V, 1>);
    return a.fp32 ? run(ep_router_backward_rows<true, L, V, 64 / L>) : run(ep_router_backward_rows<false, L, V, 64 / L>);
  });
}

}  // namespace ep
