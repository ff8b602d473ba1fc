// Softmax attention with a sliding window and a few first tokens that stay
// visible (sinks): the argument block and the visibility rule that its kernels
// share.
//
// Query i of sequence b stands at position p = q_pos[b] + i among that
// sequence's n = lens[b] keys, and key j is visible to it iff
//   0 <= p < n,  j < n,  j <= p + right  and  (j >= p - left  or  j < sinks).
// For a run of queries the visible keys lie in two ranges: the first tokens
// [0, S) and the window [lo, hi), with S <= lo (one range when they touch).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lapnys {

constexpr int kWinUnbounded = 1 << 29;  // a window side without a bound
constexpr int kWinMaxLen = 1 << 28;     // tokens of a sequence (p +- side stays in int32)

struct WinArgs {
  const void* q;      // [B][Hq][Nq][d]
  const void* k;      // [B][Hkv][Nk][d]
  const void* v;
  void* out;          // [B][Hq][Nq][d]
  void* rest;         // like out, bf16 only, or null: what rounding left of out, rounded
  float* lse;         // [B][Hq][Nq]: log2 of the sum of exp over the visible keys; -inf: none
  const int32_t* lens;   // [B] or null (Nk)
  const int32_t* q_pos;  // [B] or null (Nk - Nq)
  int B, Hq, Hkv, g, Nq, Nk, d;
  int left, right, sinks;  // sides as kWinUnbounded when open, all clamped to it
  float scale, scale_log2;  // softmax scale and the same times log2(e)
  // backward
  const void* dout;
  float* D;           // [B][Hq][Nq]: sum_c dout * out
  void* dq;
  void* dk;
  void* dv;
  // The first `stiles` key tiles (those with first tokens, or all where few tiles have many
  // queries each) have their queries cut into `chunks` ranges of chunk_rows
  float* part;        // their fp32 partial dK, dV
  int stiles, chunks, chunk_rows;
};

struct WinSeq {
  int len, qp;
};
__device__ __forceinline__ WinSeq win_seq(const WinArgs& a, int b) {
  WinSeq s;
  s.len = a.lens ? min(max(a.lens[b], 0), a.Nk) : a.Nk;
  s.qp = a.q_pos ? min(max(a.q_pos[b], -kWinMaxLen), kWinMaxLen) : a.Nk - a.Nq;
  return s;
}

// the key ranges that queries [i0, i1) see: first tokens [0, S), window [lo, hi)
struct WinRange {
  int S, lo, hi;
};
__device__ __forceinline__ WinRange win_keys(const WinArgs& a, const WinSeq& s, int i0, int i1) {
  const int p0 = max(s.qp + i0, 0), p1 = min(s.qp + i1, s.len) - 1;
  WinRange r{0, 0, 0};
  if (p0 > p1) return r;
  r.lo = max(0, p0 - a.left);
  r.hi = min(s.len, p1 + a.right + 1);
  if (a.sinks >= r.lo)
    r.lo = 0;
  else
    r.S = a.sinks;
  return r;
}

// the queries [i0, i1) that see some key of [j0, j1)
__device__ __forceinline__ void win_queries(const WinArgs& a, const WinSeq& s, int j0, int j1,
                                            int* i0, int* i1) {
  *i0 = *i1 = 0;
  if (j0 >= s.len || j0 >= j1) return;
  int p0 = max(0, j0 - a.right), p1 = min(s.len, j1 + a.left);
  if (j0 < a.sinks) p1 = s.len;
  p0 = max(p0 - s.qp, 0);
  p1 = min(p1 - s.qp, a.Nq);
  if (p0 < p1) {
    *i0 = p0;
    *i1 = p1;
  }
}

// the keys that one query sees: j in [lo, hi) or j < S (and below hi); none when hi = 0
struct WinRow {
  int lo, hi, S;
};
__device__ __forceinline__ WinRow win_row(const WinArgs& a, const WinSeq& s, int i) {
  const int p = s.qp + i;
  if (i >= a.Nq || p < 0 || p >= s.len) return WinRow{0, 0, 0};
  return WinRow{p - a.left, min(s.len, p + a.right + 1), a.sinks};
}
__device__ __forceinline__ bool win_sees(const WinRow& r, int j) {
  return j < r.hi && (j >= r.lo || j < r.S);
}

}  // namespace lapnys
