"""The index arithmetic of packed sequences and of the work dealt out over them
(csrc/nf4_deal.hpp), compiled for the host: with offsets that decrease,
overlap or leave the rows, every index that the attention kernels form from it
stays in its range."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "nf4_bit_weight_amd", "csrc")

PROGRAM = r"""
#include <climits>
#include <cstdio>
#include <cstdlib>
#include <vector>
#include "nf4_deal.hpp"
using namespace nf4;

#define NEED(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); std::exit(1); } } while (0)

static int count_of(const std::vector<int>& off, int t) {
  int c = 0;
  for (int o : off) c += o <= t;
  return c;
}

// The sequence that holds a row holds it in the kernels' own clamped rows.
static void owners(const std::vector<int>& off, int T) {
  const int B = static_cast<int>(off.size()) - 1;
  for (int t = 0; t < T; ++t) {
    const int b = owner_of(off.data(), B, t, count_of(off, t));
    NEED(b >= -1 && b < B);
    if (b < 0) continue;
    int first, n;
    seq_rows(off.data(), b, T, first, n);
    NEED(first >= 0 && n >= 0 && first + n <= T);
    NEED(t >= first && t < first + n);
  }
}

// All of a cache attention call: what its workers take and what its join reads.
static void dealt(const std::vector<int>& off, int T, int G, int Hkv, int R, int steps, int cost, int workers, bool sorted) {
  const int B = static_cast<int>(off.size()) - 1;
  std::vector<int> first(B), n(B), tiles(B);
  std::vector<unsigned> before(B + 1, 0);
  const int share = steps + cost;
  for (int b = 0; b < B; ++b) {
    seq_rows(off.data(), b, T, first[b], n[b]);
    tiles[b] = (n[b] * G + R - 1) / R;
    before[b + 1] = before[b] + static_cast<unsigned>(Hkv * tiles[b]) * static_cast<unsigned>(share);
  }
  const int total = static_cast<int>(before[B]);
  const Deal deal(larger(total, 0), workers);
  NEED(deal.begin(0) == 0 && deal.begin(workers) == larger(total, 0));
  long long taken = 0;
  for (int w = 0; w < workers; ++w) {
    for (int b = 0; b < B; ++b) {
      const int units = Hkv * tiles[b], base = static_cast<int>(before[b]), end = static_cast<int>(before[b + 1]);
      for (int lo = larger(deal.begin(w), base); lo < deal.begin(w + 1) && lo < end;) {
        UnitAt at;
        if (!unit_at(lo, deal.begin(w + 1), base, units, share, at)) {
          NEED(!sorted);
          break;
        }
        NEED(at.u >= 0 && at.u < units && at.from >= 0 && at.from < at.to && at.to <= share);
        taken += at.to - at.from;
        lo += at.to - at.from;
      }
    }
  }
  if (sorted) NEED(taken == total);
  for (int t = 0; t < T; ++t) {
    const int b = owner_of(off.data(), B, t, count_of(off, t));
    if (b < 0) continue;
    for (int g = 0; g < G; ++g) {
      const int row = (t - first[b]) * G + g, rt = row / R, rr = row - rt * R;
      NEED(row >= 0 && rr >= 0 && rr < R && rt < tiles[b]);
      for (int h = 0; h < Hkv; ++h) {
        SharedBy by;
        if (!shared_by(rt * Hkv + h, share, cost, static_cast<int>(before[b]), total, deal, by)) {
          NEED(!sorted);
          continue;
        }
        NEED(by.w0 >= 0 && by.w0 <= by.w1 && by.w1 < workers);
        NEED(deal.begin(by.w0) <= by.u0 + cost && by.u0 + share - 1 < deal.begin(by.w1 + 1));
      }
    }
  }
}

int main() {
  // a row before the first sequence whose last offset is small
  const std::vector<int> falling = {5, 10, 0};
  owners(falling, 10);
  dealt(falling, 10, 4, 8, 16, 1024, 2, 512, false);
  std::srand(1);
  for (int round = 0; round < 3000; ++round) {
    const int T = 1 + std::rand() % 40, B = std::rand() % 12;
    std::vector<int> off(B + 1);
    const bool sorted = round % 3 == 0;
    for (auto& o : off) o = sorted ? 0 : std::rand() % (2 * T) - T / 2;
    if (sorted) {
      for (int b = 1; b <= B; ++b) off[b] = smaller(T, off[b - 1] + std::rand() % 5);
    } else if (round % 7 == 0) {
      off[std::rand() % (B + 1)] = round % 2 ? INT_MAX : INT_MIN;
    }
    owners(off, T);
    const int R = 16 << std::rand() % 2;
    dealt(off, T, 1 + std::rand() % 5, 1 + std::rand() % 8, R, 1 + std::rand() % 60, 2, 1 + std::rand() % 512, sorted);
  }
  // counts that pass 32 bits: 200 sequences of the same 30 rows, 2^17 steps each and more
  for (int steps = 1 << 17; steps <= 1 << 20; steps *= 2) {
    std::vector<int> off;
    for (int b = 0; b < 201; ++b) off.push_back(b % 2 ? 30 : 0);
    owners(off, 30);
    dealt(off, 30, 4, 8, 32, steps, 2, 512, false);
  }
  // and bases anywhere
  for (int round = 0; round < 200000; ++round) {
    auto any = [] { return static_cast<int>(static_cast<unsigned>(std::rand()) << 16 ^ static_cast<unsigned>(std::rand())); };
    const int lo = any() & INT_MAX, share = 1 + (any() & 0xFFFF), units = any() & 0x7FFF, base = any();
    const int hi = lo + smaller(INT_MAX - lo, 1 + (any() & 0xFFFF));
    UnitAt at;
    if (hi > lo && unit_at(lo, hi, base, units, share, at))
      NEED(at.u >= 0 && at.u < units && at.from >= 0 && at.from < at.to && at.to <= share);
    const int total = any() & INT_MAX, workers = 1 + (any() & 1023);
    const Deal deal(total, workers);
    SharedBy by;
    if (shared_by(any(), 2 + share, 2, base, total, deal, by)) NEED(by.w0 >= 0 && by.w0 <= by.w1 && by.w1 < workers);
  }
  std::puts("ok");
}
"""


def test_indices_stay_in_range(tmp_path):
    cxx = shutil.which("g++")
    if not cxx:
        pytest.skip("no host compiler")
    src = tmp_path / "deal.cpp"
    src.write_text(PROGRAM)
    exe = tmp_path / "deal"
    subprocess.run([cxx, "-std=c++17", "-O1", "-fsanitize=undefined", "-fno-sanitize-recover=all", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, timeout=120)
    assert r.returncode == 0, r.stdout.decode()
