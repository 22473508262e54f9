// Host-side check of the tensor-core paged decode's work division
// (latent_attention_b200/csrc/paged_slices.cuh): over many random batches every
// chunk of every sequence lies in exactly one unit's segment, a segment is
// "whole" exactly when it holds all chunks, a unit's cursor walks forward, and
// the partial slots of a cut sequence are distinct, inside the unit's two and
// the ones that the combine kernel reads.  Prints "ok <cases>" or the first
// violation (exit status 1).
#include <cstdio>
#include <random>
#include <set>
#include <vector>

#include "paged_slices.cuh"

using namespace mla::pslices;

static int fail(const char* what, int c, int b, int u) {
  std::printf("FAIL case %d seq %d unit %d: %s\n", c, b, u, what);
  return 1;
}

int main() {
  std::mt19937 rng(4321);
  int cases = 0;
  for (int c = 0; c < 4000; ++c) {
    const int kind = c % 5;
    const int B = kind == 0 ? 1 + (int)(rng() % 3) : kind == 1 ? 300 + (int)(rng() % 500)
                                                               : 1 + (int)(rng() % 70);
    const int hi = kind == 0 ? 500000 : kind == 1 ? 300 : 1 + (int)(rng() % 30000);
    std::vector<int> n(B);
    std::vector<int64_t> pre(B + 1);
    for (int b = 0; b < B; ++b) {
      n[b] = (int)(rng() % (hi + 1));
      if (kind == 3 && rng() % 2) n[b] = 0;
      if (kind == 4 && rng() % 10) n[b] = 0;
      if (c % 97 == 0) n[b] = 0;
      pre[b + 1] = pre[b] + charged(n[b]);
    }
    const int units = 1 + (int)(rng() % 148), min_len = 1 + (int)(rng() % 6);
    std::vector<std::vector<int>> seen(B);
    for (int b = 0; b < B; ++b) seen[b].assign((n[b] + CT - 1) / CT, -1);
    std::set<int> slots;
    for (int u = 0; u < units; ++u) {
      const Slice sl = unit_slice(pre.data(), B, u, units, min_len);
      Cursor k;
      k.start(pre.data(), B, sl, u, seq_at(pre.data(), B, sl.r0));
      int last = -1, kk = 0;
      while (!k.done) {
        const Seg s = k.s;
        if (s.b <= last || k.kk != kk || k.j != 0 || s.nch < 1) return fail("walk", c, s.b, u);
        last = s.b;
        for (int j = 0; j < s.nch; ++j) {
          if (s.c0 + j >= (int)seen[s.b].size()) return fail("past the end", c, s.b, u);
          if (seen[s.b][s.c0 + j] != -1) return fail("twice", c, s.b, u);
          seen[s.b][s.c0 + j] = u;
          k.next(pre.data(), B, sl, u);
          if (j + 1 < s.nch && (k.done || k.j != j + 1 || k.s.b != s.b))
            return fail("chunk step", c, s.b, u);
        }
        ++kk;
        const SeqUnits su = seq_units(pre.data(), s.b, B, units, min_len);
        if (s.whole != (s.nch == (int)seen[s.b].size())) return fail("whole", c, s.b, u);
        if (s.whole != (su.u0 == su.u1)) return fail("whole against units", c, s.b, u);
        if (u < su.u0 || u > su.u1) return fail("units", c, s.b, u);
        if (!s.whole) {
          if (s.slot / 2 != u || !slots.insert(s.slot).second) return fail("slot", c, s.b, u);
          if (s.slot != seq_slot(su, u)) return fail("slot of the combine", c, s.b, u);
        }
      }
    }
    for (int b = 0; b < B; ++b) {
      std::set<int> us;
      for (int x : seen[b]) {
        if (x < 0) return fail("chunk not covered", c, b, -1);
        us.insert(x);
      }
      if (n[b]) {
        const SeqUnits su = seq_units(pre.data(), b, B, units, min_len);
        if ((int)us.size() != su.u1 - su.u0 + 1) return fail("a unit without chunks", c, b, -1);
      }
    }
    ++cases;
  }
  std::printf("ok %d\n", cases);
  return 0;
}
