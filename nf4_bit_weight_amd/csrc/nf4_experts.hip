// Routing to experts, the plan of a choice, and the tokens' rows to and from the
// experts' places (nf4_experts.h).
#include <cmath>

#include "nf4_attn.hpp"
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
__device__ __forceinline__ float number32(uint32_t r) {       // and back
  return __builtin_bit_cast(float, r & 0x80000000u ? r & 0x7FFFFFFFu : ~r);
}
// (minus infinity is none; x + 0 has no negative zero)
__device__ __forceinline__ uint64_t rank64(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x + 0.0);
  const uint64_t flip = static_cast<uint64_t>(static_cast<int64_t>(u) >> 63) | uint64_t{1} << 63;
  return x != x ? ~uint64_t{0} : (u ^ flip) - 0x000FFFFFFFFFFFFFu;
}

// This lane's value and the one of the lane M further in a butterfly over equal
// values: all M lanes of a block already hold the same, so a mirrored block serves as
// well as a crossed one.  In the vector unit's lane moves (swap16, swap32: one of the two is
// this lane's), a few cycles where a shuffle through LDS takes a hundred.
template <int M>
__device__ __forceinline__ void both(uint32_t v, uint32_t& x, uint32_t& y) {
  static_assert(M == 1 || M == 2 || M == 4 || M == 8 || M == 16 || M == 32, "lanes of a block");
  if constexpr (M <= 8) {
    constexpr int kMove = M == 1 ? 0xB1 : M == 2 ? 0x4E : M == 4 ? 0x141 : 0x140;      // quad_perm, row_half_mirror, row_mirror
    x = v;
    y = static_cast<uint32_t>(__builtin_amdgcn_update_dpp(0, static_cast<int>(v), kMove, 0xF, 0xF, true));
  } else {
    const float f = __builtin_bit_cast(float, v);
    const f32x2_t p = M == 16 ? swap16(f) : swap32(f);
    const float p0 = p[0], p1 = p[1];
    x = __builtin_bit_cast(uint32_t, p0);
    y = __builtin_bit_cast(uint32_t, p1);
  }
}
template <int M>
__device__ __forceinline__ void both(float v, float& x, float& y) {
  uint32_t a, b;
  both<M>(__builtin_bit_cast(uint32_t, v), a, b);
  x = __builtin_bit_cast(float, a);
  y = __builtin_bit_cast(float, b);
}
template <int M>
__device__ __forceinline__ void both(uint64_t v, uint64_t& x, uint64_t& y) {
  uint32_t a[2], b[2];
  both<M>(static_cast<uint32_t>(v), a[0], b[0]);
  both<M>(static_cast<uint32_t>(v >> 32), a[1], b[1]);
  x = static_cast<uint64_t>(a[1]) << 32 | a[0];
  y = static_cast<uint64_t>(b[1]) << 32 | b[0];
}
template <int M>
__device__ __forceinline__ void both(double v, double& x, double& y) {
  uint64_t a, b;
  both<M>(__builtin_bit_cast(uint64_t, v), a, b);
  x = __builtin_bit_cast(double, a);
  y = __builtin_bit_cast(double, b);
}

// f over the L lanes of a token, the same in all of them
template <int L, int M = 1, typename V, typename F>
__device__ __forceinline__ V across(V v, F f) {
  if constexpr (M < L) {
    V x, y;
    both<M>(v, x, y);
    return across<L, 2 * M>(f(x, y), f);
  } else {
    return v;
  }
}

// The largest of the L lanes' values: of the high halves, then of the low halves beside that one.  (Two
// searches of 32 bits, whose maxima take the lane moves with them: a choice takes 43 vector instructions, 54 with
// one search of 64.)
template <int L>
__device__ __forceinline__ uint64_t largest(uint64_t v) {
  auto most = [](uint32_t x, uint32_t y) { return x > y ? x : y; };
  const uint32_t high = static_cast<uint32_t>(v >> 32), top = across<L>(high, most);
  return static_cast<uint64_t>(top) << 32 | across<L>(high == top ? static_cast<uint32_t>(v) : 0u, most);
}
// The lanes of a token's L that stand below `lane`, as a ballot has them.
template <int L>
__device__ __forceinline__ uint64_t lanes_below(int lane) {
  const uint64_t token = ~uint64_t{0} << (lane & ~(L - 1));
  return ((uint64_t{1} << lane) - 1) & token;
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
};
template <>
struct Cand<true> {
  uint64_t key;
  uint32_t idx;
  __device__ __forceinline__ bool over(const Cand& o) const { return key > o.key || (key == o.key && idx < o.idx); }
  __device__ __forceinline__ int index() const { return static_cast<int>(idx); }
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

// e^x for x <= 0 in 64 bits: x = n ln 2 + r, the series of e^r to its 13th term (the next is
// below 2^-57 at |r| = ln 2 / 2), times 2^n, which goes down to the smallest number above zero
// (e^-745.1): scores that differ in 64 bits stay different.  Half of what the library's takes,
// which serves large x too.
__device__ __forceinline__ double exp64(double x) {
  const double y = fmax(x, -746.0);                             // zero from here on; n stays an integer
  const double n = rint(y * 1.4426950408889634074);
  double r = fma(-n, 0.69314718055994530942, y);
  r = fma(-n, 2.3190468138462995e-17, r);                      // ln 2 less its 64-bit value
  double p = 1.0 / 6227020800.0;
  p = fma(p, r, 1.0 / 479001600.0);
  p = fma(p, r, 1.0 / 39916800.0);
  p = fma(p, r, 1.0 / 3628800.0);
  p = fma(p, r, 1.0 / 362880.0);
  p = fma(p, r, 1.0 / 40320.0);
  p = fma(p, r, 1.0 / 5040.0);
  p = fma(p, r, 1.0 / 720.0);
  p = fma(p, r, 1.0 / 120.0);
  p = fma(p, r, 1.0 / 24.0);
  p = fma(p, r, 1.0 / 6.0);
  p = fma(p, r, 0.5);
  p = fma(p, r, 1.0);
  p = fma(p, r, 1.0);
  return x != x ? x : ldexp(p, static_cast<int>(n));
}
// 1 / x for 1 <= x <= 2: the hardware's guess, made good twice
__device__ __forceinline__ double reciprocal64(double x) {
  double r = __builtin_amdgcn_rcp(x);
  r = fma(fma(-x, r, 1.0), r, r);
  return fma(fma(-x, r, 1.0), r, r);
}

// e^(l - top) as the softmax takes it: nothing for an expert that is masked out
__device__ __forceinline__ float exp_from(float l, float top) { return l == -INFINITY ? 0.0f : expf(l - top); }

// This lane's choice (-1: none), the lanes of its wave with the same expert below it, and
// the counts of its wave in s_held [waves][E] (waves: those with choices): the lanes of an expert are found by one ballot for each
// bit of its number.  No count depends on who comes first.
struct Claim {
  int expert;
  int below;
  bool some;
};
__device__ __forceinline__ Claim claim(int e, int32_t E, int waves, int32_t* s_held) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  for (int x = threadIdx.x; x < waves * E; x += blockDim.x) s_held[x] = 0;
  const bool some = static_cast<uint32_t>(e) < static_cast<uint32_t>(E);
  uint64_t same = __ballot(some);
  for (int bit = 1; bit < E; bit <<= 1) {
    const uint64_t set = __ballot((e & bit) != 0);
    same &= (e & bit) != 0 ? set : ~set;
  }
  const int below = __popcll(same & ((uint64_t{1} << lane) - 1));
  __syncthreads();
  if (some && below == 0) s_held[wave * E + e] = __popcll(same);
  __syncthreads();
  return {e, below, some};
}
// s_held to the sums over earlier waves behind `at`; all of it comes back.
__device__ __forceinline__ int32_t sum_waves(int32_t* s_held, int32_t E, int waves, int e, int32_t at) {
  for (int w0 = 0; w0 < waves; w0 += 8) {
    int32_t n[8];
#pragma unroll
    for (int w = 0; w < 8; ++w) n[w] = w0 + w < waves ? s_held[(w0 + w) * E + e] : 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) {
      if (w0 + w < waves) s_held[(w0 + w) * E + e] = at;
      at += n[w];
    }
  }
  return at;
}
__device__ __forceinline__ void settle(const PlanArgs& a, const Claim& c, int32_t row, uint32_t at) {
  if (c.some) a.tokens[row] = static_cast<int32_t>(at / static_cast<uint32_t>(a.k));
  a.slots[at] = c.some ? row : -1;
}

// Rows of the choices [0, n) of `choices` (in LDS or memory) behind s_base, by expert
// and then in order, a workgroup's threads of them at a time; e is this thread's first one.
__device__ __forceinline__ void place(const PlanArgs& a, const int32_t* choices, int e, int n, uint32_t first, int32_t* s_base, int32_t* s_held) {
  const int wave = threadIdx.x >> 6, threads = blockDim.x, waves = (min(n, threads) + 63) / 64;
  for (int c = 0; c < n; c += threads) {
    const int i = c + threadIdx.x;
    if (c > 0) e = i < n ? choices[i] : -1;
    const Claim mine = claim(e, a.E, waves, s_held);
    for (int x = threadIdx.x; x < a.E; x += threads) s_base[x] = sum_waves(s_held, a.E, waves, x, s_base[x]);
    __syncthreads();
    if (i < n) settle(a, mine, mine.some ? s_held[wave * a.E + mine.expert] + mine.below : -1, first + i);
    if (c + threads < n) __syncthreads();
  }
}

// s_first [E + 1] from the experts' counts s_count [E], by the first wave
__device__ __forceinline__ void first_rows(const int32_t* s_count, int32_t E, int32_t* s_first) {
  const int lane = threadIdx.x;
  int32_t sum = 0;
  for (int e0 = 0; e0 < E; e0 += 256) {
    int32_t n[4], incl[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = e0 + 64 * i + lane < E ? s_count[e0 + 64 * i + lane] : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) incl[i] = wave_scan(n[i]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (e0 + 64 * i + lane < E) s_first[e0 + 64 * i + lane] = sum + incl[i] - n[i];
      sum += __builtin_amdgcn_readlane(incl[i], 63);
    }
  }
  if (lane == 0) s_first[E] = sum;
}

// The counts of s_pick's choices [0, n) in s_count [E] (integers: in any order)
__device__ __forceinline__ void count_choices(const int32_t* s_pick, int n, int32_t E, int32_t* s_count) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) s_count[e] = 0;
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += blockDim.x) {
    const int e = s_pick[i];
    if (static_cast<uint32_t>(e) < static_cast<uint32_t>(E)) atomicAdd(&s_count[e], 1);
  }
  __syncthreads();
}

// The run of a workgroup: an `only` run is placed at once, else its counts go to held.
__device__ __forceinline__ void plan_run(const PlanArgs& a, bool only, const int32_t* s_pick, int n, uint32_t first, uint16_t* held, int pitch,
                                         int32_t* s_count, int32_t* s_first, int32_t* s_held) {
  const int threads = blockDim.x;
  const bool once = only && n <= threads;                      // a choice a thread: counted and placed in one pass
  Claim mine{};
  if (once) {
    const int waves = (n + 63) / 64;
    mine = claim(threadIdx.x < n ? s_pick[threadIdx.x] : -1, a.E, waves, s_held);
    for (int e = threadIdx.x; e < a.E; e += threads) s_count[e] = sum_waves(s_held, a.E, waves, e, 0);
    __syncthreads();
  } else {
    count_choices(s_pick, n, a.E, s_count);
  }
  if (!only) {
    uint16_t* mine_held = held + static_cast<int64_t>(blockIdx.x) * pitch;      // (a run has at most 8192 choices)
    for (int e = threadIdx.x; e < pitch; e += threads) mine_held[e] = e < a.E ? static_cast<uint16_t>(s_count[e]) : 0;
    return;
  }
  if (threadIdx.x < 64) first_rows(s_count, a.E, s_first);
  __syncthreads();
  for (int e = threadIdx.x; e <= a.E; e += threads) a.offsets[e] = s_first[e];
  const int32_t end = s_first[a.E];
  for (int r = end + threadIdx.x; r < n; r += threads) a.tokens[r] = -1;      // rows that belong to nobody
  if (once) {
    if (threadIdx.x < n)
      settle(a, mine, mine.some ? s_first[mine.expert] + s_held[(threadIdx.x >> 6) * a.E + mine.expert] + mine.below : -1, first + threadIdx.x);
    return;
  }
  __syncthreads();
  place(a, s_pick, threadIdx.x < n ? s_pick[threadIdx.x] : -1, n, first, s_first, s_held);
}

// L lanes of a wave share a token, each holds PER neighbouring experts in
// registers.  Each sorts its own; then k times the best of the L heads is taken
// and its lane moves up.  (A search over all E for each choice costs k (PER + log
// L) steps for every token of the wave, this one a sort and k log L.)
//
// Sums are fp32.  WIDE: what the choice compares (s + bias, sums of two) is computed
// in 64 bits, since 8191 x 256 scores hold several pairs that fp32 rounding would turn round.
//
// A workgroup's tokens are a run of the plan: it counts their choices for k_plan_place, or,
// as the only one, places them itself (one launch for a batch of new tokens: 5.0 us for one).
//
// What bounds it: 8191 tokens, 256 experts, sigmoid with a bias in 8 groups: 15.7 us alone, 20.7 with the
// plan (23.2 at 1630 vector instructions a wave of two tokens; now 1300, a fifth of them the scores in 64
// bits, a fourth the choices); the bytes take 1.9 us.  Their issue is two thirds of it (20.8k cycles of the
// 32.4k that a compute unit is busy); for the rest one chain of load, scores, sort and choices lies open, since
// all 4096 waves start together, four a SIMD.  16384 tokens, 64 experts, bf16 and
// softmax: 6.3.
template <typename T, int PER, int L, bool WIDE>
__global__ __launch_bounds__(1024) void k_route(RouteArgs a, PlanArgs plan, uint16_t* held, int pitch) {
  constexpr int kTokens = 64 / L, kOf = L * PER;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const int sub = lane & (L - 1), tk = lane / L, e0 = sub * PER;
  int32_t* s_all = reinterpret_cast<int32_t*>(lds);             // the choices of the workgroup
  int32_t* s_pick = s_all + (wave * kTokens + tk) * a.k;        // of the token
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * waves * kTokens, t = t0 + wave * kTokens + tk;
  const bool on = t < a.T;

  float l[PER];
  const T* logits = static_cast<const T*>(a.logits) + (on ? t * a.stride : 0);
  const T* row = logits + e0;
  constexpr int kVec = 16 / sizeof(T);                                                 // of one load
  if (a.E % kVec == 0 && a.stride % kVec == 0 && (reinterpret_cast<uintptr_t>(a.logits) & 15) == 0) {
#pragma unroll
    for (int i = 0; i < PER; i += kVec) {
      u32x4_t v = {};
      const bool in = on && e0 + i < a.E;
      if (in) v = *reinterpret_cast<const u32x4_t*>(row + i);
#pragma unroll
      for (int j = 0; j < kVec; ++j) l[i + j] = in ? element<T>(v, j) : -INFINITY;
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i) l[i] = on && e0 + i < a.E ? value(row + i) : -INFINITY;
  }
  float b[WIDE ? PER : 1] = {};                                 // on its way with the logits
  if constexpr (WIDE) {
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i) b[i] = a.bias[min(e0 + i, a.E - 1)];
    }
  }

  float top = -INFINITY;
#pragma unroll
  for (int i = 0; i < PER; ++i) top = fmaxf(top, l[i]);
  top = across<L>(top, [](float x, float y) { return fmaxf(x, y); });
  if (top == -INFINITY) top = 0.0f;

  // c, and what orders the experts
  Cand<WIDE> v[PER];
  double c[WIDE ? PER : 1];
  if constexpr (WIDE) {
    // (loops without a branch: the experts' 64-bit chains run side by side)
    if (a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        // e^-|l| either way: nothing overflows, and below zero the score is as small as e^l
        const double x = exp64(-static_cast<double>(fabsf(l[i]))), r = reciprocal64(1.0 + x);
        c[i] = l[i] < 0.0f ? x * r : r;
      }
    } else {
      double sum = 0.0;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        const double x = exp64(static_cast<double>(l[i]) - static_cast<double>(top));
        c[i] = l[i] == -INFINITY ? 0.0 : x;
        sum += c[i];
      }
      sum = across<L>(sum, [](double x, double y) { return x + y; });
      const double part = sum > 0.0 ? 1.0 / sum : sum;         // (no expert at all: 0)
#pragma unroll
      for (int i = 0; i < PER; ++i) c[i] *= part;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i) c[i] = l[i] == -INFINITY ? -INFINITY : c[i] + static_cast<double>(b[i]);
    if (a.bias) {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = {rank64(c[i]), static_cast<uint32_t>(e0 + i)};
    } else {
#pragma unroll
      for (int i = 0; i < PER; ++i) v[i] = {rank64(static_cast<double>(l[i])), static_cast<uint32_t>(e0 + i)};
    }
  } else {
#pragma unroll
    for (int i = 0; i < PER; ++i)
      v[i] = {l[i] == -INFINITY ? 0 : static_cast<uint64_t>(rank32(l[i])) << 32 | static_cast<uint32_t>(~(e0 + i))};
  }

  if (a.groups > 1) {
    const int size = a.E / a.groups;
    auto group_rank = [](double one, double two, bool nan) {
      return nan ? ~uint64_t{0} : rank64(two == -INFINITY ? one : one + two);
    };
    if (a.lanes > 0) {
      // a group is a run of `lanes` lanes, a power of two
      uint64_t key = 0;
      if (WIDE && a.top2) {
        double one = -INFINITY, two = -INFINITY;
        uint32_t nan = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          nan |= c[WIDE ? i : 0] != c[WIDE ? i : 0];
          two = fmax(two, fmin(one, c[WIDE ? i : 0]));
          one = fmax(one, c[WIDE ? i : 0]);
        }
        auto merge = [&](auto m) {
          if (m >= L || m >= a.lanes) return;
          double x1, y1, x2, y2;
          uint32_t xn, yn;
          both<m>(one, x1, y1);
          both<m>(two, x2, y2);
          both<m>(nan, xn, yn);
          one = fmax(x1, y1);
          two = fmax(fmin(x1, y1), fmax(x2, y2));
          nan = xn | yn;
        };
        merge(std::integral_constant<int, 1>{});
        merge(std::integral_constant<int, 2>{});
        merge(std::integral_constant<int, 4>{});
        merge(std::integral_constant<int, 8>{});
        merge(std::integral_constant<int, 16>{});
        key = group_rank(one, two, nan != 0);
      } else {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
          const uint64_t x = WIDE ? v[i].key : v[i].key >> 32;
          key = x > key ? x : key;
        }
        auto merge = [&](auto m) {
          if (m >= L || m >= a.lanes) return;
          uint64_t x, y;
          both<m>(key, x, y);
          key = x > y ? x : y;
        };
        merge(std::integral_constant<int, 1>{});
        merge(std::integral_constant<int, 2>{});
        merge(std::integral_constant<int, 4>{});
        merge(std::integral_constant<int, 8>{});
        merge(std::integral_constant<int, 16>{});
      }
      // top_groups times the best of them, of equal ones the lowest: no other of its lanes stands below
      const uint64_t below = lanes_below<L>(lane & ~(a.lanes - 1));
      bool kept = false;
      for (int j = 0; j < a.top_groups; ++j) {
        const bool here = key == largest<L>(key);
        if ((__ballot(here) & below) == 0 && here) kept = true, key = 0;
      }
      if (!kept) {
#pragma unroll
        for (int i = 0; i < PER; ++i) v[i].key = 0;
      }
    } else {
      // any size: through LDS
      uint64_t* s_score = reinterpret_cast<uint64_t*>(lds + a.group_lds) + (wave * kTokens + tk) * 2 * kOf;
      uint64_t* s_group = s_score + kOf;
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if constexpr (WIDE) s_score[e0 + i] = a.top2 ? __builtin_bit_cast(uint64_t, c[i]) : v[i].key;
        else s_score[e0 + i] = v[i].key >> 32;
      }
      wave_sync();
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
          key = group_rank(one, two, nan);
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
  }

  sort_descending(v);
  [[maybe_unused]] const uint64_t below_me = lanes_below<L>(lane);
  uint64_t taken = 0;                                           // the key of choice `sub`
  for (int j = 0; j < a.k; ++j) {
    const uint64_t best = largest<L>(v[0].key);
    if (j == sub) taken = best;
    bool here = best != 0 && v[0].key == best;
    if constexpr (WIDE && L > 1) {
      // the lowest of the lanes that hold it: theirs are the lower experts
      const uint64_t held = __ballot(here);
      here = here && (held & below_me) == 0;
    }
    if (here) s_pick[j] = v[0].index();
    if (sub == 0 && on && best == 0) s_pick[j] = -1;
    if (here) {
#pragma unroll
      for (int i = 0; i + 1 < PER; ++i) v[i] = v[i + 1];
      v[PER - 1].key = 0;
    }
  }
  wave_sync();

  // Weights.  Renormalised ones are formed from the chosen alone, so that they do not
  // vanish with the scores: softmax from the largest chosen logit, sigmoid (e^l / (1 + e^l)
  // below zero) with all of them scaled up by the best where that is far down.
  const int mine = on ? a.k : 0;
  auto logit = [&](int e) { return e < 0 ? -INFINITY : value(logits + e); };
  // a lane has choice `sub` in registers; more where there are more than lanes
  const int first = sub < mine ? s_pick[sub] : -1;
  const float first_logit = !WIDE && first >= 0 ? number32(static_cast<uint32_t>(taken >> 32)) : logit(first);
  float best, total;
  if (a.renorm) {
    best = first_logit;
    for (int j = sub + L; j < mine; j += L) best = fmaxf(best, logit(s_pick[j]));
    best = across<L>(best, [](float x, float y) { return fmaxf(x, y); });
    if (best == -INFINITY || (a.sigmoid && best > 0.0f)) best = 0.0f;
  } else {
    best = a.sigmoid ? 0.0f : top;
  }
  auto score = [&](int e, float x) {
    if (e < 0) return 0.0f;
    if (!a.sigmoid) return expf(x - best);
    return x >= 0.0f ? 1.0f / (1.0f + expf(-x)) : expf(x - best) / (1.0f + expf(x));
  };
  const float first_score = score(first, first_logit);
  if (a.renorm) {
    total = first_score;
    for (int j = sub + L; j < mine; j += L) total += score(s_pick[j], logit(s_pick[j]));
  } else {
    total = 0.0f;
    if (!a.sigmoid) {
#pragma unroll
      for (int i = 0; i < PER; ++i) total += exp_from(l[i], top);
    }
  }
  total = across<L>(total, [](float x, float y) { return x + y; });
  if (a.sigmoid && !a.renorm) total = 1.0f;
  auto write = [&](int j, int e, float s) {
    a.experts[t * a.k + j] = e;
    a.weights[t * a.k + j] = e >= 0 ? a.scale * (s / total) : 0.0f;
  };
  if (sub < mine) write(sub, first, first_score);
  for (int j = sub + L; j < mine; j += L) write(j, s_pick[j], score(s_pick[j], logit(s_pick[j])));
  if (!plan.offsets) return;
  __syncthreads();
  const int n = static_cast<int>(min(static_cast<int64_t>(waves * kTokens), a.T - t0)) * a.k;
  int32_t* s_count = reinterpret_cast<int32_t*>(lds + a.plan_lds);
  plan_run(plan, gridDim.x == 1, s_all, n, static_cast<uint32_t>(t0 * a.k), held, pitch, s_count, s_count + a.E, s_count + 2 * a.E + 1);
}

// grad_logits, with D = sum_j g_j w_j over the chosen:
//   softmax                 [i chosen] g_i w_i - p_i D
//   softmax, renormalised   [i chosen] w_i (g_i - D / scale)
//   sigmoid                 [i chosen] g_i w_i (1 - s_i)
//   sigmoid, renormalised   [i chosen] w_i (1 - s_i) (g_i - D / scale)
// Lanes as in k_route; the token's row is put together in LDS.  (16384 tokens, 64 experts, bf16: 3.8 us.)
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

// A counting sort of the choices by expert.  Runs of tokens are counted (in k_route, or
// here for a choice made elsewhere); then each run's choices find their rows behind
// those of the same expert in earlier runs.  A single run is done in one launch.
__global__ __launch_bounds__(1024) void k_plan_count(PlanArgs a, int run_tokens, uint16_t* held, int pitch) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int32_t* s_pick = reinterpret_cast<int32_t*>(lds);
  const int64_t t0 = static_cast<int64_t>(blockIdx.x) * run_tokens, first = t0 * a.k;
  const int n = static_cast<int>(min(static_cast<int64_t>(run_tokens), a.T - t0)) * a.k;
  for (int i = threadIdx.x; i < n; i += blockDim.x) s_pick[i] = a.experts[first + i];
  int32_t* s_count = s_pick + run_tokens * a.k;
  plan_run(a, gridDim.x == 1, s_pick, n, static_cast<uint32_t>(first), held, pitch, s_count, s_count + a.E, s_count + 2 * a.E + 1);
}

// x of this lane and of the lane M further in lanes whose bit M is clear, y in the others
// (in assembly, and with the wait, as in swap16).
template <int M>
__device__ __forceinline__ int32_t give(int32_t x, int32_t y) {
  static_assert(M == 16 || M == 32, "rows or halves");
  if constexpr (M == 16) asm volatile("s_nop 1\n\tv_permlane16_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  else asm volatile("s_nop 1\n\tv_permlane32_swap_b32 %0, %1" : "+v"(x), "+v"(y));
  return x + y;
}

// Many runs: held [runs, pitch] to sums [runs + 1, pitch] over earlier runs; a wave an expert.
__global__ __launch_bounds__(256) void k_plan_sum(const uint16_t* held, int64_t runs, int pitch, int32_t* sums) {
  const int e = blockIdx.x * 4 + (threadIdx.x >> 6), lane = threadIdx.x & 63;
  int32_t sum = 0;
  for (int64_t r0 = 0; r0 < runs; r0 += 64) {
    const int64_t r = r0 + lane;
    const int32_t n = r < runs ? held[r * pitch + e] : 0, incl = wave_scan(n);
    if (r < runs) sums[r * pitch + e] = sum + incl - n;
    sum += __builtin_amdgcn_readlane(incl, 63);
  }
  if (lane == 0) sums[runs * pitch + e] = sum;
}

// Workgroups place `each` runs.  With sums they are taken from there; else a workgroup sums
// the earlier runs' counts and all of them itself: a thread 8 neighbouring experts of every
// so many runs, then over the lanes and waves.  (8191 tokens, 256 experts: 256 runs, 128 KB of
// counts for each of 128 workgroups, 6.6 us; a third of it the sums, the rest a chain of short steps.)
// LDS: [pitch] of earlier runs, [pitch] of all, [2][16][pitch] partial sums or [16][E] counts of the
// waves, and the experts' first rows [E + 1].
__global__ __launch_bounds__(1024) void k_plan_place(PlanArgs a, int run_tokens, int64_t runs, int each, const uint16_t* held, int pitch,
                                                     const int32_t* sums) {
  extern __shared__ __attribute__((aligned(16))) char lds[];
  int32_t* s_before = reinterpret_cast<int32_t*>(lds);
  int32_t* s_total = s_before + pitch;
  int32_t* s_held = s_total + pitch;
  int32_t* s_first = s_held + (sums ? 16 * a.E : 32 * pitch);
  const int64_t run0 = static_cast<int64_t>(blockIdx.x) * each, t0 = run0 * run_tokens, first = t0 * a.k;
  const int n = static_cast<int>(min(static_cast<int64_t>(run_tokens) * each, a.T - t0)) * a.k;
  const int e0 = threadIdx.x < n ? a.experts[first + threadIdx.x] : -1;
  if (sums) {
    for (int e = threadIdx.x; e < pitch; e += 1024) {
      s_before[e] = sums[run0 * pitch + e];
      s_total[e] = sums[runs * pitch + e];
    }
  } else {
    const int columns = pitch / 8, shift = __ffs(columns) - 1, strips = 1024 >> shift;     // (a power of two)
    const int column = threadIdx.x & (columns - 1), strip = threadIdx.x >> shift;
    // of this thread's runs: [0] in earlier ones, [1] in all.  Two counts a word are added while they
    // fit, four runs of at most 8192 choices each.
    int32_t sum[2][8] = {};
    for (int r0 = strip; r0 < static_cast<int>(runs); r0 += 8 * strips) {
      u32x4_t v[8];                                             // 8 loads on their way at once
#pragma unroll
      for (int b = 0; b < 8; ++b) {
        const int r = r0 + b * strips;
        v[b] = u32x4_t{0, 0, 0, 0};
        if (r < runs) v[b] = *reinterpret_cast<const u32x4_t*>(held + static_cast<int64_t>(r) * pitch + 8 * column);
      }
#pragma unroll
      for (int h = 0; h < 8; h += 4) {
        if (r0 - strip + h * strips >= static_cast<int>(runs)) break;
        u32x4_t of[2] = {};
#pragma unroll
        for (int b = h; b < h + 4; ++b) {
          const uint32_t earlier = r0 + b * strips < run0 ? ~0u : 0u;
          of[0] += v[b] & earlier;
          of[1] += v[b];
        }
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
          for (int i = 0; i < 8; ++i) sum[t][i] += static_cast<int32_t>((of[t][i / 2] >> (16 * (i & 1))) & 0xFFFFu);
      }
    }
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    // Lanes of a wave with the same column.  Across the halves a lane adds up one of two values and
    // leaves the other to its partner: lanes below 32 end with [0], the others with [1]; so again
    // across the rows of 16, for the values [0, 4) and [4, 8).  Inside a row they turn.
    auto turn = [&](auto by) {
      if (columns > by) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[0][i] += lane_move<0x120 + by, 0xF>(sum[0][i]);
    };
    if (columns <= 32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[0][i] = give<32>(sum[0][i], sum[1][i]);
    }
    if (columns <= 16) {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum[0][i] = give<16>(sum[0][i], sum[0][4 + i]);
    }
    turn(std::integral_constant<int, 8>{});
    turn(std::integral_constant<int, 4>{});
    turn(std::integral_constant<int, 2>{});
    turn(std::integral_constant<int, 1>{});
    // waves of the same column: every columns / 64-th, or all
    const int stride = columns > 64 ? columns / 64 : 1, rows = 16 / stride;
    typedef int i32x4 __attribute__((ext_vector_type(4)));
    const i32x4 low{sum[0][0], sum[0][1], sum[0][2], sum[0][3]}, high{sum[0][4], sum[0][5], sum[0][6], sum[0][7]};
    int32_t* part = s_held + (wave / stride) * pitch + 8 * column;
    if (columns > 32) {
      *reinterpret_cast<i32x4*>(part) = low;
      *reinterpret_cast<i32x4*>(part + 4) = high;
      *reinterpret_cast<i32x4*>(part + 16 * pitch) = i32x4{sum[1][0], sum[1][1], sum[1][2], sum[1][3]};
      *reinterpret_cast<i32x4*>(part + 16 * pitch + 4) = i32x4{sum[1][4], sum[1][5], sum[1][6], sum[1][7]};
    } else if (columns == 32) {
      part += (lane >> 5) * 16 * pitch;
      *reinterpret_cast<i32x4*>(part) = low;
      *reinterpret_cast<i32x4*>(part + 4) = high;
    } else if ((lane & 15) < columns) {
      *reinterpret_cast<i32x4*>(part + (lane >> 5) * 16 * pitch + (lane >> 4 & 1) * 4) = low;
    }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * pitch; e += 1024) {       // (s_total follows s_before)
      const int32_t* part = s_held + (e < pitch ? e : e + 15 * pitch);
      int32_t sum = 0;
#pragma unroll 8
      for (int r = 0; r < rows; ++r) sum += part[r * pitch];
      s_before[e] = sum;
    }
  }
  __syncthreads();
  if (threadIdx.x < 64) first_rows(s_total, a.E, s_first);
  __syncthreads();
  const int32_t end = s_first[a.E];
  if (blockIdx.x == 0)
    for (int e = threadIdx.x; e <= a.E; e += 1024) a.offsets[e] = s_first[e];
  for (int e = threadIdx.x; e < a.E; e += 1024) s_before[e] += s_first[e];
  for (int i = threadIdx.x; i < n; i += 1024)
    if (first + i >= end) a.tokens[first + i] = -1;             // a row that belongs to nobody
  __syncthreads();
  place(a, a.experts + first, e0, n, static_cast<uint32_t>(first), s_before, s_held);
}

// ---- rows --------------------------------------------------------------------------

// N values of a row as one load: 16 bytes where rows and pointers allow it, else one value.  (4096 x 8 in
// bf16 of 2047 beside 2048: gather 34 us for 24, combine 91 for 30, its gradients 110 for 52.)
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

// The rows of a token's choices (-1: none), lane j the j-th: one load, where one a step of the
// loop over them would be waited for before each row (48 tokens: 4.1 us so, 2.9 with this).
__device__ __forceinline__ int32_t rows_of(const RowsArgs& a, int64_t t) {
  const int lane = threadIdx.x & 63;
  const int32_t s = lane < a.k ? a.slots[t * a.k + lane] : -1;
  return s < static_cast<int64_t>(a.T) * a.k ? s : -1;
}
__device__ __forceinline__ float lane_value(float x, int lane) {
  return __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, x), lane));
}
constexpr int kAtOnce = 2;   // rows of a token on their way together (8: 33 us for 29 at 4096 x 8 of 2048, 4 the same)

// Workgroups: one a token and 256 vectors of its row, which is read once and written k times.
// What bounds it are the bytes: 4096 tokens x 8 of 2048 in bf16 25.5 us, 5.9 TB/s into the last-level cache.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_gather(RowsArgs a, const T* x, int64_t stride, T* rows) {
  const int64_t t = blockIdx.x, h = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * N;
  const int32_t mine = rows_of(a, t);
  const int64_t end = a.fill ? *a.end : static_cast<int64_t>(a.T) * a.k;
  const bool in = h < a.H;
  Vec<T, N> v;
  if (in) v.load(x + t * stride + h);
  for (int j = 0; j < a.k; ++j) {
    const int32_t s = __builtin_amdgcn_readlane(mine, j);
    if (s >= 0 && in) v.put(rows + s * a.H + h);
  }
  if ((t + 1) * a.k <= end || !in) return;
  v.zero();
  for (int64_t r = t * a.k > end ? t * a.k : end; r < (t + 1) * a.k; ++r) v.put(rows + r * a.H + h);
}

// out[t] = sum_j w_j rows[slot_j] (weights NULL: ones).  Bound by the bytes: 4095 tokens x 8 of 2048
// in bf16 22 us where the last-level cache holds the rows, 40 from memory.
template <typename T, int N>
__global__ __launch_bounds__(256) void k_combine(RowsArgs a, const T* rows, const float* weights, T* out) {
  const int64_t t = blockIdx.x, h = (static_cast<int64_t>(blockIdx.y) * 256 + threadIdx.x) * N;
  const int lane = threadIdx.x & 63;
  const int32_t mine = rows_of(a, t);
  const float w = weights && lane < a.k ? weights[t * a.k + lane] : 1.0f;
  const int64_t at = h < a.H ? h : 0;                           // lanes behind the row's end read its start and write nothing
  Vec<T, N> sum;
  sum.zero();
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    Vec<T, N> v[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      const int32_t s = j0 + j < a.k ? __builtin_amdgcn_readlane(mine, j0 + j) : -1;
      if (s >= 0) v[j].load(rows + s * a.H + at);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if (j0 + j >= a.k || __builtin_amdgcn_readlane(mine, j0 + j) < 0) continue;
      const float wj = lane_value(w, j0 + j);
#pragma unroll
      for (int i = 0; i < N; ++i) sum.f[i] = fmaf(wj, v[j].f[i], sum.f[i]);
    }
  }
  if (h < a.H) sum.put(out + t * a.H + h);
}

// A workgroup a token, kAtOnce of its choices at a time: grad_out is read k / kAtOnce times, from
// the L2.  (4095 x 8 of 2048 in bf16, 285 MB: 48 us, 5.9 TB/s.)
template <typename T, int N>
__global__ __launch_bounds__(256) void k_combine_bwd(RowsArgs a, const T* grad, int64_t stride, const T* rows, const float* weights,
                                                     T* grad_rows, float* grad_weights) {
  __shared__ float s_part[4][kAtOnce];
  const int64_t t = blockIdx.x;
  const int lane = threadIdx.x & 63;
  const T* g = grad + t * stride;
  const int32_t mine = rows_of(a, t);
  const float w = grad_rows && lane < a.k ? weights[t * a.k + lane] : 0.0f;
  for (int j0 = 0; j0 < a.k; j0 += kAtOnce) {
    float dot[kAtOnce] = {};
    for (int64_t h = threadIdx.x * N; h < a.H; h += 256 * N) {
      Vec<T, N> gv, v[kAtOnce];
      gv.load(g + h);
      if (grad_weights) {
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
          const int32_t s = j0 + j < a.k ? __builtin_amdgcn_readlane(mine, j0 + j) : -1;
          if (s >= 0) v[j].load(rows + s * a.H + h);
        }
      }
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) {
        const int32_t s = j0 + j < a.k ? __builtin_amdgcn_readlane(mine, j0 + j) : -1;
        if (s < 0) continue;
        if (grad_weights) {
#pragma unroll
          for (int i = 0; i < N; ++i) dot[j] = fmaf(gv.f[i], v[j].f[i], dot[j]);
        }
        if (grad_rows) {
          const float wj = lane_value(w, j0 + j);
          Vec<T, N> o;
#pragma unroll
          for (int i = 0; i < N; ++i) o.f[i] = gv.f[i] * wj;
          o.put(grad_rows + s * a.H + h);
        }
      }
    }
    if (!grad_weights) continue;
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) dot[j] = across<64>(dot[j], [](float x, float y) { return x + y; });
    if (lane == 0) {
#pragma unroll
      for (int j = 0; j < kAtOnce; ++j) s_part[threadIdx.x >> 6][j] = dot[j];
    }
    __syncthreads();
    const int j = threadIdx.x;
    if (j < kAtOnce && j0 + j < a.k) grad_weights[t * a.k + j0 + j] = (s_part[0][j] + s_part[1][j]) + (s_part[2][j] + s_part[3][j]);
    if (j0 + kAtOnce < a.k) __syncthreads();
  }
  if (!grad_rows || !a.fill) return;
  const int64_t end = *a.end;
  for (int64_t r = t * a.k > end ? t * a.k : end; r < (t + 1) * a.k; ++r)
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

namespace {

// Runs of a plan: the tokens of one workgroup, 4 to 16 waves of them.  One workgroup takes
// all it can hold, which spares a launch; beyond, the smallest that are no more than the
// compute units, so that the waves have a vector unit each.
int lanes_of(int32_t E) { return E <= 8 ? 1 : E <= 16 ? 2 : E <= 32 ? 4 : E <= 64 ? 8 : E <= 128 ? 16 : E <= 256 ? 32 : 64; }
int per_lane(int32_t E) { return E > 512 ? 16 : 8; }
struct Runs {
  int waves, tokens;         // of a workgroup
  int64_t runs;
  int pitch;                 // of the counts
  int64_t each;              // runs of a workgroup of k_plan_place, or 0: the counts are summed first
  size_t held_bytes, bytes;  // of the counts, and with the sums
};
// Every workgroup of k_plan_place reads all counts: fewer workgroups where there are many, so
// that together they read 16 MB (from the L2s mostly), and a launch that sums first where those
// would be too few.
Runs runs_of(int64_t T, int32_t E, int waves) {
  const int of_wave = 64 / lanes_of(E), tokens = waves * of_wave;
  const int64_t needed = (T + of_wave - 1) / of_wave, runs = T > 0 ? (T + tokens - 1) / tokens : 1;
  if (needed < waves) waves = needed > 0 ? static_cast<int>(needed) : 1;
  const int pitch = lanes_of(E) * per_lane(E);
  int64_t each = (runs * runs * pitch * 2 + (int64_t{16} << 20) - 1) >> 24;
  if (each > 8) each = 0;
  const size_t held = static_cast<size_t>(runs) * pitch * 2, sums = each == 0 ? static_cast<size_t>(runs + 1) * pitch * 4 : 0;
  return {waves, tokens, runs, pitch, each, held, held + sums};
}
int waves_for(int64_t T, int32_t E, int most) {
  const int64_t needed = (T + 64 / lanes_of(E) - 1) / (64 / lanes_of(E));
  if (needed <= most) return most;
  int waves = most < 4 ? most : 4;
  while (waves < most && needed > static_cast<int64_t>(waves) * device_cu_count()) waves *= 2;
  return waves;
}
// Waves of a run of a choice with k a token: its choices fit 32 KB of LDS (k_route's always do: k <= E).
int run_waves(int32_t E, int32_t k) {
  int waves = 16;
  while (waves > 1 && waves * (64 / lanes_of(E)) * k * 4 > 32768) waves /= 2;
  return waves;
}

size_t plan_lds(int32_t E, int waves) { return static_cast<size_t>(2 * E + 1 + waves * E) * 4; }

// The second half, behind the counts.
hipError_t launch_place(const PlanArgs& a, const Runs& r, uint16_t* held, hipStream_t stream) {
  allow_lds<k_plan_place>();
  int32_t* sums = nullptr;
  if (r.each == 0) {
    sums = reinterpret_cast<int32_t*>(reinterpret_cast<char*>(held) + r.held_bytes);
    k_plan_sum<<<r.pitch / 4, 256, 0, stream>>>(held, r.runs, r.pitch, sums);
  }
  // (runs of four tokens, of groups that go through LDS, can be more than a launch holds workgroups of 1024)
  const int64_t each = r.each == 0 ? (r.runs >> 21) + 1 : r.each;
  const size_t behind = static_cast<size_t>(r.each == 0 ? 16 * a.E : 32 * r.pitch), lds = (2 * r.pitch + a.E + 1 + behind) * 4;
  k_plan_place<<<static_cast<uint32_t>((r.runs + each - 1) / each), 1024, lds, stream>>>(a, r.tokens, r.runs, static_cast<int>(each), held,
                                                                                        r.pitch, sums);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& args, const PlanArgs& plan, void* ws, hipStream_t stream) {
  RouteArgs a = args;
  const bool wide = a.bias || (a.groups > 1 && a.top2);
  const int size = a.E / a.groups, per = per_lane(a.E), lanes = size / per;
  a.lanes = a.groups > 1 && size % per == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
  const bool through_lds = a.groups > 1 && a.lanes == 0;
  const Runs r = runs_of(a.T, a.E, waves_for(a.T, a.E, through_lds ? 4 : 16));
  size_t bytes = (static_cast<size_t>(r.tokens) * a.k * 4 + 15) / 16 * 16;
  a.group_lds = static_cast<int32_t>(bytes);
  if (through_lds) bytes += static_cast<size_t>(r.waves) * 64 * per * 16;
  a.plan_lds = static_cast<int32_t>(bytes);
  if (plan.offsets) bytes += plan_lds(a.E, r.waves);
  uint16_t* held = static_cast<uint16_t*>(ws);
  const hipError_t e = with_lanes(a.E, [&](auto per_c, auto lanes_c) {
    constexpr int PER = per_c, L = lanes_c;
    auto go = [&](auto kernel) {
      constexpr auto launch = decltype(kernel)::launch;
      allow_lds<launch>();
      launch<<<static_cast<uint32_t>(r.runs), 64 * r.waves, bytes, stream>>>(a, plan, held, r.pitch);
      return hipGetLastError();
    };
    if (a.bf16) return wide ? go(Kernel<k_route<uint16_t, PER, L, true>>{}) : go(Kernel<k_route<uint16_t, PER, L, false>>{});
    return wide ? go(Kernel<k_route<float, PER, L, true>>{}) : go(Kernel<k_route<float, PER, L, false>>{});
  });
  if (e != hipSuccess || !plan.offsets || r.runs == 1) return e;
  return launch_place(plan, r, held, stream);
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

// k_route's shortest runs need the most.
size_t plan_ws_bytes(int64_t T, int32_t k, int32_t E) {
  const int waves = run_waves(E, k);
  const Runs r = runs_of(T, E, waves < 4 ? waves : 4);
  return r.runs == 1 ? 0 : r.bytes;
}

hipError_t launch_plan(const PlanArgs& a, void* ws, hipStream_t stream) {
  const Runs r = runs_of(a.T, a.E, waves_for(a.T, a.E, run_waves(a.E, a.k)));
  uint16_t* held = static_cast<uint16_t*>(ws);
  const size_t lds = static_cast<size_t>(r.tokens) * a.k * 4 + plan_lds(a.E, r.runs == 1 ? 16 : 0);
  allow_lds<k_plan_count>();
  k_plan_count<<<static_cast<uint32_t>(r.runs), 1024, lds, stream>>>(a, r.tokens, held, r.pitch);
  if (r.runs == 1) return hipGetLastError();
  const hipError_t e = hipGetLastError();
  return e != hipSuccess ? e : launch_place(a, r, held, stream);
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
