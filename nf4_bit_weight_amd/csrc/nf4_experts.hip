// Routing to experts, the plan of a choice, and the tokens' rows to and from the
// experts' places (nf4_experts.h).
#include <cmath>

#include "nf4_device.hpp"
#include "nf4_experts.hpp"
#include "nf4_internal.hpp"

namespace nf4 {

namespace {

__device__ __forceinline__ float as_float(uint16_t b) { return __builtin_bit_cast(float, static_cast<uint32_t>(b) << 16); }
__device__ __forceinline__ float value(const float* p) { return *p; }
__device__ __forceinline__ float value(const uint16_t* p) { return as_float(*p); }
__device__ __forceinline__ void store(float* p, float v) { *p = v; }
__device__ __forceinline__ void store(uint16_t* p, float v) { *p = to_bf16(v); }
// value i of 16 bytes
template <typename T>
__device__ __forceinline__ float element(u32x4_t v, int i) {
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(f32x4_t, v)[i];
  else return as_float(static_cast<uint16_t>(v[i / 2] >> (16 * (i & 1))));
}

// LDS written by some lanes of a wave is read by others of the same wave.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// ---- the choice ----------------------------------------------------------------

// Integers in the order of the numbers: a NaN above all, 0 is left for "none".
__device__ __forceinline__ uint32_t rank32(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = x == 0.0f ? 0u : __builtin_bit_cast(uint32_t, x);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ uint64_t rank64(double x) {
  if (x != x) return ~uint64_t{0};
  const uint64_t u = x == 0.0 ? 0u : __builtin_bit_cast(uint64_t, x);
  return u >> 63 ? ~u : u | uint64_t{1} << 63;
}

// An expert in the running.  Where 32 bits order the scores, their rank and the
// index (lower is better) share one word; else the index stands beside it.
template <bool WIDE>
struct Cand;
template <>
struct Cand<false> {
  uint64_t key;
  __device__ __forceinline__ bool over(const Cand& o) const { return key > o.key; }
  __device__ __forceinline__ int index() const { return static_cast<int>(~static_cast<uint32_t>(key)); }
  __device__ __forceinline__ Cand from(int mask) const { return {__shfl_xor(key, mask, 64)}; }
};
template <>
struct Cand<true> {
  uint64_t key;
  int idx;
  __device__ __forceinline__ bool over(const Cand& o) const { return key > o.key || (key == o.key && idx < o.idx); }
  __device__ __forceinline__ int index() const { return idx; }
  __device__ __forceinline__ Cand from(int mask) const { return {__shfl_xor(key, mask, 64), __shfl_xor(idx, mask, 64)}; }
};

template <int PER, bool WIDE>
__device__ __forceinline__ void sort_descending(Cand<WIDE> (&v)[PER]) {
  // odd-even merge sort
#pragma unroll
  for (int p = 1; p < PER; p <<= 1)
#pragma unroll
    for (int q = p; q >= 1; q >>= 1)
#pragma unroll
      for (int j = q % p; j + q < PER; j += 2 * q)
#pragma unroll
        for (int i = 0; i < q; ++i) {
          const int x = i + j, y = i + j + q;
          if (y < PER && x / (2 * p) == y / (2 * p)) {
            const bool swap = v[y].over(v[x]);
            const Cand<WIDE> a = v[x], b = v[y];
            v[x] = swap ? b : a;
            v[y] = swap ? a : b;
          }
        }
}

template <int L, typename V, typename F>
__device__ __forceinline__ V across(V v, F f) {
#pragma unroll
  for (int m = 1; m < L; m <<= 1) v = f(v, __shfl_xor(v, m, 64));
  return v;
}

// e^(l - top) as the softmax takes it: nothing for an expert that is masked out
__device__ __forceinline__ float exp_from(float l, float top) { return l == -INFINITY ? 0.0f : expf(l - top); }

// L lanes of a wave share a token, each holds PER neighbouring experts in
// registers.  Each sorts its own; then k times the best of the L heads is taken
// and its lane moves up.  (A search over all E for each choice costs k (PER + log
// L) steps for every token of the wave, this one a sort and k log L.)
//
// Sums are fp32.  WIDE: what the choice compares (s + bias, sums of two) is computed
// in 64 bits, since 8191 x 256 scores hold several pairs that fp32 rounding would turn round.
template <typename T, int PER, int L, bool WIDE>
__global__ __launch_bounds__(PER == 16 ? 128 : 256) void k_route(RouteArgs a) {
  constexpr int kWaves = PER == 16 ? 2 : 4, kHeld = 64 * PER, kTokens = 64 / L, kOf = L * PER;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane & (L - 1), tk = lane / L, e0 = sub * PER;
  const bool grouped = a.groups > 1;
  char* mine = lds + wave * kHeld * (grouped ? 24 : 8);
  float* s_logit = reinterpret_cast<float*>(mine) + tk * kOf;                         // the token's logits
  int32_t* s_pick = reinterpret_cast<int32_t*>(mine + kHeld * 4) + tk * kOf;          // its choice
  uint64_t* s_score = reinterpret_cast<uint64_t*>(mine + kHeld * 8) + tk * kOf;       // what the groups are judged by
  uint64_t* s_group = reinterpret_cast<uint64_t*>(mine + kHeld * 16) + tk * kOf;      // and the judgement
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens + tk;
  const bool on = t < a.T;

  float l[PER];
  const T* row = static_cast<const T*>(a.logits) + (on ? t * a.stride : 0) + e0;
  constexpr int kVec = 16 / sizeof(T);                                                 // of one load
  if (a.E % kVec == 0 && a.stride % kVec == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < PER; i += kVec) {
      u32x4_t v = {};
      const bool in = on && e0 + i < a.E;
      if (in) v = *reinterpret_cast<const u32x4_t*>(row + i);
#pragma unroll
      for (int j = 0; j < kVec; ++j) {
        l[i + j] = in ? element<T>(v, j) : -INFINITY;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = on && e0 + i < a.E ? value(row + i) : -INFINITY;
  }
#pragma unroll
  for (int i = 0; i < PER; ++i) s_logit[e0 + i] = l[i];

  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = across<L>(top, [](float x, float y) { return fmaxf(x, y); });
  if (top == -INFINITY) top = 0.0f;

  // c, and what orders the experts
  Cand<WIDE> v[PER];
  double c[WIDE ? PER : 1];
  if constexpr (WIDE) {
    double part = 1.0;
    if (!a.sigmoid) {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        c[i] = l[i] == -INFINITY ? 0.0 : exp(static_cast<double>(l[i]) - static_cast<double>(top));
        sum += c[i];
      }
      sum = across<L>(sum, [](double x, double y) { return x + y; });
      part = sum;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      c[i] = a.sigmoid ? 1.0 / (1.0 + exp(-static_cast<double>(l[i]))) : c[i] / part;
      if (a.bias && e0 + i < a.E) c[i] += static_cast<double>(a.bias[e0 + i]);
      const bool live = l[i] != -INFINITY && c[i] != -INFINITY;
      if (!live) c[i] = -INFINITY;
      v[i] = {live ? rank64(a.bias ? c[i] : static_cast<double>(l[i])) : 0, e0 + i};
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = {l[i] == -INFINITY ? 0 : static_cast<uint64_t>(rank32(l[i])) << 32 | static_cast<uint32_t>(~(e0 + i))};
  }

  if (grouped) {
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if constexpr (WIDE) s_score[e0 + i] = a.top2 ? __builtin_bit_cast(uint64_t, c[i]) : v[i].key;
      else s_score[e0 + i] = v[i].key >> 32;
    }
    wave_sync();
    const int size = a.E / a.groups;
    for (int g = sub; g < a.groups; g += L) {
      const uint64_t* s = s_score + g * size;
      uint64_t key = 0;
      if (WIDE && a.top2) {
        double one = -INFINITY, two = -INFINITY;
        bool nan = false;
        for (int i = 0; i < size; ++i) {
          const double x = __builtin_bit_cast(double, s[i]);
          nan |= x != x;
          two = fmax(two, fmin(one, x));
          one = fmax(one, x);
        }
        key = nan ? ~uint64_t{0} : one == -INFINITY ? 0 : rank64(two == -INFINITY ? one : one + two);
      } else {
        for (int i = 0; i < size; ++i) key = s[i] > key ? s[i] : key;
      }
      s_group[g] = key;
    }
    wave_sync();
    for (int g = sub; g < a.groups; g += L) {
      const uint64_t key = s_group[g];
      int before = 0;
      for (int o = 0; o < a.groups; ++o) before += s_group[o] > key || (s_group[o] == key && o < g);
      s_score[g] = before < a.top_groups;
    }
    wave_sync();
    int g = e0 / size, r = e0 - g * size;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      if (e0 + i < a.E && !s_score[g]) v[i].key = 0;
      if (++r == size) r = 0, ++g;
    }
  }

  sort_descending(v);
  for (int j = 0; j < a.k; ++j) {
    Cand<WIDE> best = v[0];
#pragma unroll
    for (int m = 1; m < L; m <<= 1) {
      const Cand<WIDE> o = best.from(m);
      best = o.over(best) ? o : best;
    }
    const bool some = best.key != 0;
    if (sub == 0) s_pick[j] = some ? best.index() : -1;
    if (some && best.index() / PER == sub) {
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) v[i] = v[i + 1];
      v[PER - 1].key = 0;
    }
  }
  wave_sync();

  // Weights.  Renormalised ones are formed from the chosen alone, so that they do not
  // vanish with the scores: softmax from the largest chosen logit, sigmoid (e^l / (1 + e^l)
  // below zero) with all of them scaled up by the best where that is far down.
  float best = -INFINITY, total = 0.0f;
  for (int j = sub; j < a.k; j += L) best = s_pick[j] >= 0 ? fmaxf(best, s_logit[s_pick[j]]) : best;
  best = across<L>(best, [](float x, float y) { return fmaxf(x, y); });
  if (best == -INFINITY || (a.sigmoid && best > 0.0f)) best = 0.0f;
  if (!a.sigmoid && !a.renorm) best = top;
  if (a.sigmoid && !a.renorm) best = 0.0f;
  auto score = [&](float x) {
    if (!a.sigmoid) return expf(x - best);
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - best) / (1.0f + expf(x));
  };
  if (a.renorm) {
    for (int j = sub; j < a.k; j += L) total += s_pick[j] >= 0 ? score(s_logit[s_pick[j]]) : 0.0f;
  } else if (!a.sigmoid) {
#pragma unroll
    for (int i = 0; i < PER; ++i) total += exp_from(l[i], top);
  }
  total = across<L>(total, [](float x, float y) { return x + y; });
  if (a.sigmoid && !a.renorm) total = 1.0f;
  if (!on) return;
  for (int j = sub; j < a.k; j += L) {
    const int e = s_pick[j];
    a.experts[t * a.k + j] = e;
    a.weights[t * a.k + j] = e >= 0 ? a.scale * (score(s_logit[e]) / total) : 0.0f;
  }
}

// grad_logits, with D = sum_j g_j w_j over the chosen:
//   softmax                 [i chosen] g_i w_i - p_i D
//   softmax, renormalised   [i chosen] w_i (g_i - D / scale)
//   sigmoid                 [i chosen] g_i w_i (1 - s_i)
//   sigmoid, renormalised   [i chosen] w_i (1 - s_i) (g_i - D / scale)
// Lanes as in k_route; the token's row is put together in LDS.
template <typename T, int PER, int L>
__global__ __launch_bounds__(PER == 16 ? 128 : 256) void k_route_bwd(RouteArgs a, const float* grad, T* out) {
  constexpr int kWaves = PER == 16 ? 2 : 4, kTokens = 64 / L, kOf = L * PER;
  __shared__ float s_row[kWaves * 64 * PER];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int sub = lane & (L - 1), tk = lane / L;
  float* row = s_row + wave * 64 * PER + tk * kOf;
  const int64_t t = (static_cast<int64_t>(blockIdx.x) * kWaves + wave) * kTokens + tk;
  const bool on = t < a.T;
  const T* logits = static_cast<const T*>(a.logits) + (on ? t * a.stride : 0);
  const int64_t at = on ? t * a.k : 0;

  float D = 0.0f;
  for (int j = sub; j < a.k; j += L)
    if (on && static_cast<uint32_t>(a.experts[at + j]) < static_cast<uint32_t>(a.E)) D += grad[at + j] * a.weights[at + j];
  D = across<L>(D, [](float x, float y) { return x + y; });

  const bool all = !a.sigmoid && !a.renorm;                    // the unchosen have a gradient too
  if (all) {
    float l[PER], top = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int e = sub + i * L;
      l[i] = on && e < a.E ? value(logits + e) : -INFINITY;
      top = fmaxf(top, l[i]);
    }
    top = across<L>(top, [](float x, float y) { return fmaxf(x, y); });
    if (top == -INFINITY) top = 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      l[i] = exp_from(l[i], top);
      sum += l[i];
    }
    sum = across<L>(sum, [](float x, float y) { return x + y; });
    const float f = sum > 0.0f || sum != sum ? -D / sum : 0.0f;
#pragma unroll
    for (int i = 0; i < PER; ++i) row[sub + i * L] = l[i] == 0.0f ? 0.0f : l[i] * f;
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) row[sub + i * L] = 0.0f;
  }
  wave_sync();
  const float mean = a.renorm ? D / a.scale : 0.0f;
  for (int j = sub; j < a.k; j += L) {
    const int e = on ? a.experts[at + j] : -1;
    if (static_cast<uint32_t>(e) >= static_cast<uint32_t>(a.E)) continue;
    float d = a.weights[at + j] * (grad[at + j] - mean);
    if (a.sigmoid) {
      const float x = value(logits + e);                       // 1 - s without the difference
      d *= x >= 0.0f ? expf(-x) / (1.0f + expf(-x)) : 1.0f / (1.0f + expf(x));
    }
    row[e] += d;
  }
  wave_sync();
  if (!on) return;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = sub + i * L;
    if (e < a.E) store(out + t * a.E + e, row[e]);
  }
}

// L and PER for E experts: 8 of them a lane, 16 above 512.
template <typename F>
hipError_t with_lanes(int32_t E, F f) {
  if (E <= 8) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 1>{});
  if (E <= 16) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 2>{});
  if (E <= 32) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 4>{});
  if (E <= 64) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 8>{});
  if (E <= 128) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 16>{});
  if (E <= 256) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 32>{});
  if (E <= 512) return f(std::integral_constant<int, 8>{}, std::integral_constant<int, 64>{});
  return f(std::integral_constant<int, 16>{}, std::integral_constant<int, 64>{});
}

// ---- the plan --------------------------------------------------------------------

// Counting sort of the choices by expert, in three steps: each workgroup counts
// its kPairs-sized run of choices, the counts are summed over the runs, and each
// choice finds its row: the rows of its expert in earlier runs, and those before
// it in its own, from bit masks (one bit a choice, one mask an expert), so that
// the order is the tokens' and no count depends on who comes first.
// A run is 1024 choices, fewer above 256 experts: the masks take E / 8 bytes a choice, 32 KB.
constexpr int plan_pairs(int32_t E) { return E <= 256 ? 1024 : E <= 512 ? 512 : 256; }
int64_t plan_runs(int64_t pairs, int32_t E) { return (pairs + plan_pairs(E) - 1) / plan_pairs(E); }

__global__ __launch_bounds__(256) void k_plan_count(PlanArgs a, int pairs, int32_t* held) {
  extern __shared__ int32_t s_held[];
  for (int e = threadIdx.x; e < a.E; e += 256) s_held[e] = 0;
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * pairs, all = static_cast<int64_t>(a.T) * a.k;
  for (int i = threadIdx.x; i < pairs && first + i < all; i += 256) {
    const int e = a.experts[first + i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E)) atomicAdd(&s_held[e], 1);
  }
  __syncthreads();
  for (int e = threadIdx.x; e < a.E; e += 256) held[static_cast<int64_t>(blockIdx.x) * a.E + e] = s_held[e];
}

// held [runs, E] to the sum over earlier runs, total [E]; a thread an expert.
__global__ __launch_bounds__(64) void k_plan_sum(int32_t* held, int64_t runs, int32_t E, int32_t* total) {
  const int e = blockIdx.x * 64 + threadIdx.x;
  if (e >= E) return;
  int32_t sum = 0;
  for (int64_t r = 0; r < runs; ++r) {
    const int32_t n = held[r * E + e];
    held[r * E + e] = sum;
    sum += n;
  }
  total[e] = sum;
}

__global__ __launch_bounds__(256) void k_plan_place(PlanArgs a, int pairs, const int32_t* held, const int32_t* total) {
  extern __shared__ uint32_t s_mask[];                          // [E][words], then the experts' first rows [E + 1]
  const int words = pairs / 32;
  int32_t* s_first = reinterpret_cast<int32_t*>(s_mask + a.E * words);
  for (int i = threadIdx.x; i < a.E * words; i += 256) s_mask[i] = 0;
  if (threadIdx.x < 64) {                                       // exclusive sums over the experts, by one wave
    int32_t sum = 0;
    for (int e0 = 0; e0 < a.E; e0 += 64) {
      const int e = e0 + threadIdx.x;
      int32_t n = e < a.E ? total[e] : 0, incl = n;
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const int32_t o = __shfl_up(incl, d, 64);
        if (static_cast<int>(threadIdx.x) >= d) incl += o;
      }
      if (e < a.E) s_first[e] = sum + incl - n;
      sum += __shfl(incl, 63, 64);
    }
    if (threadIdx.x == 0) s_first[a.E] = sum;
  }
  __syncthreads();
  const int64_t first = static_cast<int64_t>(blockIdx.x) * pairs, all = static_cast<int64_t>(a.T) * a.k;
  const int n = static_cast<int>(all - first < pairs ? all - first : pairs);
  for (int i = threadIdx.x; i < n; i += 256) {
    const int e = a.experts[first + i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E)) atomicOr(&s_mask[e * words + i / 32], 1u << (i % 32));
  }
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += 256) a.offsets[e] = s_first[e];
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += 256) {
    const int e = a.experts[first + i];
    int32_t row = -1;
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(a.E)) {
      row = s_first[e] + held[static_cast<int64_t>(blockIdx.x) * a.E + e];
      for (int w = 0; w < i / 32; ++w) row += __popc(s_mask[e * words + w]);
      row += __popc(s_mask[e * words + i / 32] & ((1u << (i % 32)) - 1));
      a.tokens[row] = static_cast<int32_t>((first + i) / a.k);
    }
    a.slots[first + i] = row;
    if (first + i >= s_first[a.E]) a.tokens[first + i] = -1;    // a row that belongs to nobody
  }
}

// ---- rows --------------------------------------------------------------------------

// N values of a row as one load: 16 bytes where rows and pointers allow it, else one value.
template <typename T, int N>
struct Vec {
  float f[N];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (N == 1) {
      f[0] = value(p);
    } else {
      const u32x4_t v = *reinterpret_cast<const u32x4_t*>(p);
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = element<T>(v, i);
    }
  }
  __device__ __forceinline__ void put(T* p) const {
    if constexpr (N == 1) {
      store(p, f[0]);
    } else if constexpr (sizeof(T) == 4) {
      *reinterpret_cast<f32x4_t*>(p) = f32x4_t{f[0], f[1], f[2], f[3]};
    } else {
      *reinterpret_cast<u32x4_t*>(p) = u32x4_t{pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                                               pack_bf16x2(f[6], f[7])};
    }
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = 0.0f;
  }
};

__device__ __forceinline__ bool is_row(int32_t slot, const RowsArgs& a) {
  return slot >= 0 && slot < static_cast<int64_t>(a.T) * a.k;
}

// Workgroups: one a token and 256 vectors of its row.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_gather(RowsArgs a, const T* x, int64_t stride, T* rows) {
  const int64_t t = blockIdx.x, h = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * N;
  if (h >= a.H) return;
  Vec<T, N> v;
  v.load(x + t * stride + h);
  for (int j = 0; j < a.k; ++j) {
    const int32_t s = a.slots[t * a.k + j];
    if (is_row(s, a)) v.put(rows + s * a.H + h);
  }
  if (!a.fill) return;
  const int64_t end = *a.end;
  v.zero();
  for (int64_t r = t * a.k; r < (t + 1) * a.k; ++r)
    if (r >= end) v.put(rows + r * a.H + h);
}

// out[t] = sum_j w_j rows[slot_j] (weights NULL: ones)
template <typename T, int N>
__global__ __launch_bounds__(256) void k_combine(RowsArgs a, const T* rows, const float* weights, T* out) {
  const int64_t t = blockIdx.x, h = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * N;
  if (h >= a.H) return;
  Vec<T, N> sum;
  sum.zero();
  for (int j = 0; j < a.k; ++j) {
    const int32_t s = a.slots[t * a.k + j];
    if (!is_row(s, a)) continue;
    const float w = weights ? weights[t * a.k + j] : 1.0f;
    Vec<T, N> v;
    v.load(rows + s * a.H + h);
#pragma unroll
    for (int i = 0; i < N; ++i) sum.f[i] = fmaf(w, v.f[i], sum.f[i]);
  }
  sum.put(out + t * a.H + h);
}

// A workgroup a token.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_combine_bwd(RowsArgs a, const T* grad, int64_t stride, const T* rows, const float* weights,
                                                     T* grad_rows, float* grad_weights) {
  __shared__ float part[4];
  const int64_t t = blockIdx.x;
  const T* g = grad + t * stride;
  for (int j = 0; j < a.k; ++j) {
    const int32_t s = a.slots[t * a.k + j];
    float dot = 0.0f;
    if (is_row(s, a)) {
      const float w = weights[t * a.k + j];
      for (int64_t h = threadIdx.x * N; h < a.H; h += 256 * N) {
        Vec<T, N> gv, v;
        gv.load(g + h);
        if (grad_weights) {
          v.load(rows + s * a.H + h);
#pragma unroll
          for (int i = 0; i < N; ++i) dot = fmaf(gv.f[i], v.f[i], dot);
        }
        if (grad_rows) {
#pragma unroll
          for (int i = 0; i < N; ++i) gv.f[i] *= w;
          gv.put(grad_rows + s * a.H + h);
        }
      }
    }
    if (!grad_weights) continue;
    dot = across<64>(dot, [](float x, float y) { return x + y; });
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = dot;
    __syncthreads();
    if (threadIdx.x == 0) grad_weights[t * a.k + j] = (part[0] + part[1]) + (part[2] + part[3]);
    __syncthreads();
  }
  if (!grad_rows || !a.fill) return;
  const int64_t end = *a.end;
  for (int64_t r = t * a.k; r < (t + 1) * a.k; ++r)
    if (r >= end)
      for (int64_t h = threadIdx.x * N; h < a.H; h += 256 * N) {
        Vec<T, N> z;
        z.zero();
        z.put(grad_rows + r * a.H + h);
      }
}

bool wide(const RowsArgs& a, int64_t stride, std::initializer_list<const void*> pointers) {
  const int64_t n = a.bf16 ? 8 : 4;
  uintptr_t bits = 0;
  for (const void* p : pointers) bits |= reinterpret_cast<uintptr_t>(p);
  return a.H % n == 0 && stride % n == 0 && bits % 16 == 0;
}

template <typename F>
hipError_t with_rows(const RowsArgs& a, bool vec, F f) {
  using std::integral_constant;
  if (a.bf16) return vec ? f(uint16_t{}, integral_constant<int, 8>{}) : f(uint16_t{}, integral_constant<int, 1>{});
  return vec ? f(float{}, integral_constant<int, 4>{}) : f(float{}, integral_constant<int, 1>{});
}
dim3 row_grid(const RowsArgs& a, int n) { return dim3(a.T, static_cast<uint32_t>((a.H + 256 * n - 1) / (256 * n))); }

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  const bool wide = a.bias || (a.groups > 1 && a.top2);
  return with_lanes(a.E, [&](auto per, auto lanes) {
    constexpr int PER = per, L = lanes, kWaves = PER == 16 ? 2 : 4, kTokens = kWaves * (64 / L);
    const size_t bytes = kWaves * 64 * PER * (a.groups > 1 ? 24 : 8);
    const int grid = (a.T + kTokens - 1) / kTokens;
    auto go = [&](auto kernel) {
      kernel<<<grid, 64 * kWaves, bytes, stream>>>(a);
      return hipGetLastError();
    };
    if (a.bf16) return wide ? go(k_route<uint16_t, PER, L, true>) : go(k_route<uint16_t, PER, L, false>);
    return wide ? go(k_route<float, PER, L, true>) : go(k_route<float, PER, L, false>);
  });
}

hipError_t launch_route_bwd(const RouteArgs& a, const float* grad_weights, void* grad_logits, hipStream_t stream) {
  return with_lanes(a.E, [&](auto per, auto lanes) {
    constexpr int PER = per, L = lanes, kWaves = PER == 16 ? 2 : 4, kTokens = kWaves * (64 / L);
    const int grid = (a.T + kTokens - 1) / kTokens;
    if (a.bf16) k_route_bwd<uint16_t, PER, L><<<grid, 64 * kWaves, 0, stream>>>(a, grad_weights, static_cast<uint16_t*>(grad_logits));
    else k_route_bwd<float, PER, L><<<grid, 64 * kWaves, 0, stream>>>(a, grad_weights, static_cast<float*>(grad_logits));
    return hipGetLastError();
  });
}

size_t plan_ws_bytes(int64_t T, int32_t k, int32_t E) { return static_cast<size_t>(plan_runs(T * k, E) + 1) * E * 4; }

hipError_t launch_plan(const PlanArgs& a, void* ws, hipStream_t stream) {
  const int64_t runs = plan_runs(static_cast<int64_t>(a.T) * a.k, a.E);
  const int pairs = plan_pairs(a.E);
  int32_t *total = static_cast<int32_t*>(ws), *held = total + a.E;
  const uint32_t grid = static_cast<uint32_t>(runs);
  if (runs > 0) k_plan_count<<<grid, 256, a.E * 4, stream>>>(a, pairs, held);
  k_plan_sum<<<(a.E + 63) / 64, 64, 0, stream>>>(held, runs, a.E, total);
  // without a choice one workgroup writes the offsets
  k_plan_place<<<grid > 0 ? grid : 1, 256, a.E * (pairs / 8) + (a.E + 1) * 4, stream>>>(a, pairs, held, total);
  return hipGetLastError();
}

hipError_t launch_gather(const RowsArgs& a, const void* x, int64_t stride, void* rows, hipStream_t stream) {
  return with_rows(a, wide(a, stride, {x, rows}), [&](auto type, auto n) {
    using T = decltype(type);
    k_gather<T, n><<<row_grid(a, n), 256, 0, stream>>>(a, static_cast<const T*>(x), stride, static_cast<T*>(rows));
    return hipGetLastError();
  });
}

hipError_t launch_gather_bwd(const RowsArgs& a, const void* grad_rows, void* grad_x, hipStream_t stream) {
  return launch_combine(a, grad_rows, nullptr, grad_x, stream);
}

hipError_t launch_combine(const RowsArgs& a, const void* rows, const float* weights, void* out, hipStream_t stream) {
  return with_rows(a, wide(a, 0, {rows, out}), [&](auto type, auto n) {
    using T = decltype(type);
    k_combine<T, n><<<row_grid(a, n), 256, 0, stream>>>(a, static_cast<const T*>(rows), weights, static_cast<T*>(out));
    return hipGetLastError();
  });
}

hipError_t launch_combine_bwd(const RowsArgs& a, const void* grad_out, int64_t stride, const void* rows, const float* weights,
                              void* grad_rows, float* grad_weights, hipStream_t stream) {
  return with_rows(a, wide(a, stride, {grad_out, rows, grad_rows}), [&](auto type, auto n) {
    using T = decltype(type);
    k_combine_bwd<T, n><<<a.T, 256, 0, stream>>>(a, static_cast<const T*>(grad_out), stride, static_cast<const T*>(rows),
                                                 weights, static_cast<T*>(grad_rows), grad_weights);
    return hipGetLastError();
  });
}

}  // namespace nf4
