// Index arithmetic of packed sequences and of the work that is dealt out over
// them.  Plain C++ as well as device code, so that it can be checked on the
// host with offsets that no call should hold: whatever they are, a row belongs
// to a sequence that holds it or to none, and no index leaves its range.
#pragma once

#include <stdint.h>

#ifdef __HIPCC__
#define NF4_HD __host__ __device__ __forceinline__
#else
#define NF4_HD inline
#endif

namespace nf4 {

NF4_HD int smaller(int a, int b) { return a < b ? a : b; }
NF4_HD int larger(int a, int b) { return a > b ? a : b; }

// The rows of sequence b, clamped into 0 .. T whatever the offsets hold.
NF4_HD void seq_rows(const int32_t* offsets, int b, int T, int& first, int& n) {
  if (!offsets) {
    first = b;
    n = b < T ? 1 : 0;
    return;
  }
  const int s = smaller(larger(offsets[b], 0), T), e = smaller(larger(offsets[b + 1], s), T);
  first = s;
  n = e - s;
}

// The sequence of row t, or -1, where `count` of the offsets are <= t: the last
// of them, if it holds the row.  (Of offsets that decrease the last one may
// begin behind it.)
NF4_HD int owner_of(const int32_t* offsets, int B, int t, int count) {
  const int b = count - 1;
  return b >= 0 && b < B && offsets[b] <= t && t < offsets[b + 1] ? b : -1;
}

// `total` steps (or whole units) dealt out to `workers`: the first `extra` take
// one more than the others.
struct Deal {
  int each, extra;
  NF4_HD Deal(int total, int workers) : each(total / workers), extra(total - each * workers) {}
  NF4_HD int begin(int w) const { return w * each + smaller(w, extra); }
  NF4_HD int owner(int i) const {                               // of 0 <= i < total
    const int more = extra * (each + 1);
    return i < more ? i / (each + 1) : extra + (i - more) / larger(each, 1);
  }
};

// Sums over sequences that overlap may pass 32 bits (the host bounds those of
// sequences that do not).  They wrap, and the two calls below then refuse what
// does not fit.
NF4_HD int wrap_add(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) + static_cast<uint32_t>(b)); }
NF4_HD int wrap_sub(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) - static_cast<uint32_t>(b)); }
NF4_HD int wrap_mul(int a, int b) { return static_cast<int>(static_cast<uint32_t>(a) * static_cast<uint32_t>(b)); }

// What a worker does next: unit `u` of a sequence whose `units` units of `share`
// begin at `base`, from..to of its share, for a worker that stands at lo and
// goes to hi.
struct UnitAt {
  int u, from, to;
};
NF4_HD bool unit_at(int lo, int hi, int base, int units, int share, UnitAt& at) {
  if (lo < base) return false;
  const uint32_t d = static_cast<uint32_t>(lo) - static_cast<uint32_t>(base), u = d / static_cast<uint32_t>(share);
  if (u >= static_cast<uint32_t>(units)) return false;
  at.u = static_cast<int>(u);
  at.from = static_cast<int>(d - u * static_cast<uint32_t>(share));
  at.to = smaller(share, at.from + (hi - lo));
  return true;
}

// The workers w0 .. w1 that share unit `u` of a sequence whose units begin at
// `before`, each unit `share` of `total`: `cost` for its start and end, then its
// steps.  u0 is where the unit begins.
struct SharedBy {
  int u0, w0, w1;
};
NF4_HD bool shared_by(int u, int share, int cost, int before, int total, const Deal& deal, SharedBy& s) {
  s.u0 = wrap_add(before, wrap_mul(u, share));
  if (u < 0 || s.u0 < 0 || s.u0 > total - share) return false;
  s.w0 = deal.owner(s.u0 + cost);
  s.w1 = deal.owner(s.u0 + share - 1);
  return true;
}

}  // namespace nf4
