// How the tensor-core paged decode divides its work.  Host and device code,
// shared by the attention kernel, those around it and a host-side check.
//
// A sequence of n > 0 tokens is ceil(n / CT) chunks of CT tokens, and starting
// it is charged kSeqCost chunks.  pre[b] is the number of charged chunks of
// the sequences before b (pre[b + 1] = pre[b] for a sequence without tokens).
// The line of pre[B] charged chunks is cut into slices of L, one per unit.  A
// unit's segment of b is the part of b's chunks in its slice.  A segment that
// holds all of b is written to the output directly; any other leaves a partial
// result in slot 2u (the sequence began in an earlier slice) or 2u + 1 (it
// begins here and goes on), which the output kernel merges.
#pragma once
#include <cstdint>

#if defined(__CUDACC__)
#define MLA_PHD __host__ __device__ __forceinline__
#else
#define MLA_PHD inline
#endif

namespace mla {
namespace pslices {

constexpr int CT = 128;              // tokens per chunk
constexpr int64_t kSeqCost = 2;      // chunks charged per sequence

MLA_PHD int64_t imin(int64_t a, int64_t b) { return a < b ? a : b; }
MLA_PHD int64_t imax(int64_t a, int64_t b) { return a > b ? a : b; }

// Charged chunks of a sequence of n tokens.
MLA_PHD int64_t charged(int64_t n) { return n > 0 ? (n + CT - 1) / CT + kSeqCost : 0; }

MLA_PHD int64_t slice_len(int64_t total, int n_units, int min_len) {
  return imax((total + n_units - 1) / n_units, min_len);
}

struct Slice {
  int64_t r0, r1;                    // charged chunks [r0, r1)
};
MLA_PHD Slice unit_slice(const int64_t* pre, int B, int u, int n_units, int min_len) {
  const int64_t total = pre[B], L = slice_len(total, n_units, min_len);
  Slice s;
  s.r0 = imin(u * L, total);
  s.r1 = imin(s.r0 + L, total);
  return s;
}

// First sequence whose charged chunks reach past r (one with tokens, for
// r < pre[B]).
MLA_PHD int seq_at(const int64_t* pre, int B, int64_t r) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (pre[mid + 1] <= r) lo = mid + 1; else hi = mid;
  }
  return lo;
}

struct Seg {
  int b, c0, nch;      // sequence, first chunk, chunks
  int slot;
  bool whole;          // all chunks of the sequence
};

// Walks a unit's non-empty segments, chunk by chunk.
struct Cursor {
  int kk, j;           // ordinal of the segment, chunk within it
  Seg s;
  bool done;
  MLA_PHD void seek(const int64_t* pre, int B, const Slice& sl, int u, int b) {
    while (true) {
      if (b >= B) { done = true; return; }
      const int64_t p0 = pre[b], p1 = pre[b + 1];
      if (p0 >= sl.r1) { done = true; return; }
      if (p1 == p0) { b = seq_at(pre, B, p0); if (pre[b + 1] == p0) { done = true; return; } continue; }
      const int64_t v0 = p0 + kSeqCost, s0 = imax(sl.r0, v0), s1 = imin(sl.r1, p1);
      if (s1 > s0) {
        s.b = b;
        s.c0 = (int)(s0 - v0);
        s.nch = (int)(s1 - s0);
        s.whole = s0 == v0 && s1 == p1;
        s.slot = 2 * u + (p0 > sl.r0 ? 1 : 0);
        done = false;
        return;
      }
      ++b;
    }
  }
  // b: the sequence at the slice's start, seq_at(pre, B, sl.r0)
  MLA_PHD void start(const int64_t* pre, int B, const Slice& sl, int u, int b) {
    kk = 0; j = 0;
    if (sl.r0 >= sl.r1) { done = true; return; }
    seek(pre, B, sl, u, b);
  }
  // the same from what start() found, kept by another kernel
  MLA_PHD void resume(const Seg& first) {
    kk = 0; j = 0;
    s = first;
    done = first.nch == 0;
  }
  MLA_PHD void next_seg(const int64_t* pre, int B, const Slice& sl, int u) {
    j = 0; ++kk;
    seek(pre, B, sl, u, s.b + 1);
  }
  MLA_PHD void next(const int64_t* pre, int B, const Slice& sl, int u) {
    if (++j == s.nch) next_seg(pre, B, sl, u);
  }
};

// The units u0 .. u1 that hold chunks of sequence b (with tokens), and the
// slot of one's partial.
struct SeqUnits {
  int u0, u1;
  int64_t p0, L;
};
MLA_PHD SeqUnits seq_units(const int64_t* pre, int b, int B, int n_units, int min_len) {
  SeqUnits r;
  r.L = slice_len(pre[B], n_units, min_len);
  r.p0 = pre[b];
  r.u0 = (int)((r.p0 + kSeqCost) / r.L);
  r.u1 = (int)((pre[b + 1] - 1) / r.L);
  return r;
}
MLA_PHD int seq_slot(const SeqUnits& r, int u) { return 2 * u + (r.p0 > u * r.L ? 1 : 0); }

}  // namespace pslices
}  // namespace mla
