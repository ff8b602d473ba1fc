// Windowed softmax attention for a few queries per sequence (single tokens, or
// the few of a step that answers): over plain keys and values (bf16, fp32), or
// over a cache of 8-bit values in blocks with one power-of-two scale per block
// and head (k = k8 * k_scale, v = v8 * v_scale).  Visibility rule: win.cuh.
//
// What bounds it: every visible key and value is read once, for all the query
// heads that share it, and nothing else is large.  So the work is split over the
// keys, evenly and finely: the visible groups of 16 or 32 keys of all rows (a row:
// one sequence, one key head, 16 query rows) are laid end to end, and each warp
// takes one equal stretch, whatever the sequences' lengths are.  Each has a ring of
// TMA copies of its own that runs on across rows, filled by one lane of a fifth
// warp (the working warps spent a third of their time waiting for the copy engine
// to take their requests), and leaves maximum, sum and output of each row that it
// met for k_token_join.  Blocks that shared rows out by themselves lost 8 us a wave to
// their start and end and, on ragged batches, a second wave (32 sequences, 8192
// tokens at the most: 110 us).
// Measured: that batch, 32 heads of 128 on 8: 63 us + 8 for the join, 5.3 TB/s of the
// cache's bytes; 4 sequences up to 131072 tokens, 4 queries of 16 heads on 4: 77 + 10 us;
// 16 sequences of bf16 keys, window 1024: 19 + 8 us, 3.6 TB/s.  fp32 queries: 85, 142 and (fp32
// keys) 35 us, bound by the products of their parts and the registers those take.
//
// Products on the warp-level tensor instruction (m16n8k16), with the contraction's
// order chosen so that no operand is transposed or gathered: a thread's four k of step s
// are four neighbouring features (scores), and column n of output step nt is feature
// n DP / 8 + nt (P V), so keys and values come from shared memory in 16-byte reads
// without bank conflicts (rows of 128 bytes in TMA's 128-byte swizzle).  Rows = (query
// head of the group, query), 16 of them; where there are 8 at most (a token of 4 or 8
// heads a key head) they are the products' columns instead and the keys, the values'
// features their rows: half the products, half the registers for queries and outputs,
// so three blocks of an SM instead of two (84 us for the batch above with 16 rows).  P
// then has to be turned, one movmatrix for 8 keys.
//   - 8-bit: e4m3 -> f16 is exact (one instruction for two; the e4m3 form of the
//     product is no instruction of its own here: it ran as two f16 ones with more
//     conversions, 1576 instructions for 32 keys against about 600).  q is scaled
//     per row by a power of two to fit f16 (features below 2^-38 of the row's
//     largest are lost).  p is kept as 2^10 p (v_scale / reference) in f16, the
//     reference about the row's largest p v_scale so far, so that P V adds up without a
//     product per element; outputs are rescaled when the reference moves.  fp32
//     queries: q and p in two f16 parts (2^-22).
//   - bf16: q, k, v as they are, p rounded to bf16 (2^-8 of each, as the
//     output's own rounding; sums, maxima and outputs are fp32 throughout).
//   - fp32: all operands in three bf16 parts, six products (2^-24 each).
//   With fp32 queries the products of 16 keys are added up by the FP32 pipe: the
//   instruction's own sums are cut off, which 3000 keys a warp made 2e-5 of the output.
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "win_tc.cuh"

namespace lapnys {

namespace {
constexpr int TNW = 4;      // working warps of a block (and one that copies)
constexpr int JNW = 16;     // warps that join a row's parts, at the most
constexpr int kRefMin = -126, kRefMax = 126;   // of the values' scales: range of the reference
constexpr int kRefSlack = 4;                   // 2^10 p, four powers more and a factor below 2: in f16
enum : int { TK_BF16 = 0, TK_E4M3 = 1, TK_E4M3_F32 = 2, TK_F32 = 3 };

template <int KIND>
struct Kind {
  static constexpr int ES = KIND == TK_F32 ? 4 : (KIND == TK_BF16 ? 2 : 1);  // bytes of k, v
  static constexpr bool QF32 = KIND == TK_E4M3_F32 || KIND == TK_F32;
  static constexpr bool F16 = KIND == TK_E4M3 || KIND == TK_E4M3_F32;  // f16 products
  static constexpr int GK = KIND == TK_E4M3 ? 32 : 16;                  // keys of a group
  static constexpr int PARTS = KIND == TK_F32 ? 3 : (KIND == TK_E4M3_F32 ? 2 : 1);
  static constexpr float SHIFT = F16 ? 10.f : 0.f;  // p is held as 2^SHIFT p
};
// ROWS: 16 query rows, or 8 where that is all there are
template <int KIND, int DP, int ROWS>
__host__ __device__ constexpr int ring_stages() {
  return DP < 128 || KIND == TK_E4M3_F32 ? 4 : (ROWS == 8 && KIND != TK_F32 ? 2 : 3);
}
template <int KIND, int DP, int ROWS>
__host__ __device__ constexpr size_t token_smem() {   // rings from a multiple of 1024 bytes on
  return (size_t)TNW * ring_stages<KIND, DP, ROWS>() * 2 * Kind<KIND>::GK * DP * Kind<KIND>::ES + 1024;
}
// blocks of an SM: two (by registers), three of 8 rows, fewer where the rings are that large
template <int KIND, int DP, int ROWS>
__host__ __device__ constexpr int token_blocks() {
  constexpr size_t smem = token_smem<KIND, DP, ROWS>();
  return smem > 113 * 1024 ? 1 : (smem > 74 * 1024 || ROWS == 16 || KIND == TK_E4M3_F32 ? 2 : 3);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// an 8 x 8 tile of 16-bit values, a row's pair 2 t in lane 4 row + t: transposed
__device__ __forceinline__ uint32_t turn(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
// two e4m3 values (low 16 bits) -> two f16, exact
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
// exponent of a magnitude (subnormals and 0 count as the smallest), and 2^e for -127 < e < 128
__device__ __forceinline__ int exponent(float x) { return max((int)(__float_as_uint(x) << 1 >> 24) - 127, kRefMin); }
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// two fp32 as PARTS 16-bit parts, the parts' sum nearest to them
template <int KIND>
__device__ __forceinline__ void split(float x, float y, uint32_t (&w)[Kind<KIND>::PARTS]) {
  if constexpr (KIND == TK_F32) {
    split3_bf16x2(x, y, w);
  } else if constexpr (KIND == TK_BF16) {
    const __nv_bfloat162 h = __floats2bfloat162_rn(x, y);
    w[0] = *reinterpret_cast<const uint32_t*>(&h);
  } else {
#pragma unroll
    for (int p = 0; p < Kind<KIND>::PARTS; ++p) {
      const __half2 h = __floats2half2_rn(x, y);
      w[p] = *reinterpret_cast<const uint32_t*>(&h);
      const float2 f = __half22float2(h);
      x -= f.x;
      y -= f.y;
    }
  }
}

// Byte offset of a row's 16-byte chunk c in a tile of GK rows of RB bytes, as TMA
// leaves it: panels of 128 bytes a row, chunks XORed with the row mod 8 (rows of
// 64 bytes: with half the row mod 4).
// A key row is read at chunks 2 t, 2 t + 1 of each panel (t = lane % 4) and rows
// gid (= lane / 4), a value row at chunk gid and rows 2 t + const: the eight lanes
// of a phase meet eight chunks either way.
template <int RB, int GK>
__device__ __forceinline__ uint32_t tile_off(int row, int c) {
  if constexpr (RB == 64)
    return (uint32_t)(row * 64 + ((c ^ ((row >> 1) & 3)) << 4));
  else
    return (uint32_t)((c >> 3) * (GK * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4));
}
// the chunk of a thread's i-th piece of a key row
template <int RB>
__device__ __forceinline__ int key_chunk(int t, int i) {
  return RB == 64 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
}
}  // namespace

struct TokenMaps {
  CUtensorMap k, v;   // {d, tokens, (batch or block, head)}, boxes of a panel x a copy's rows
};

template <int KIND, int DP, int ROWS>
__global__ void __launch_bounds__(32 * TNW + 32, (token_blocks<KIND, DP, ROWS>())) k_token(const __grid_constant__ TokenMaps mp, const TokenArgs t) {
  using X = Kind<KIND>;
  constexpr int ES = X::ES, RB = DP * ES, NP = X::PARTS, GK = X::GK, NU = GK / 8, NH = GK / 16;
  constexpr int NST = ring_stages<KIND, DP, ROWS>();
  constexpr bool FEW = ROWS == 8;
  constexpr int TILE = GK * RB, SLOT = 2 * TILE;
  constexpr int KS = DP / 16;                  // 16-feature steps of the scores
  constexpr int NT = DP / 8;                   // column steps of P V
  constexpr int PIECE = 16 / ES;               // features of a 16-byte piece
  constexpr int KSP = PIECE / 4;               // steps of a piece, four features a thread each
  constexpr int CH = RB / 16;                  // 16-byte chunks of a row
  constexpr int PANELS = RB == 64 ? 1 : RB / 128;
  constexpr int VP = RB == 64 ? 8 : PIECE;     // features of a thread's piece of a value row
  using TQ = typename std::conditional<X::QF32, float, __nv_bfloat16>::type;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full_s[TNW][NST], empty_s[TNW][NST];  // a ring slot's copies; its reader
  __shared__ int start_s[TNW][4];                         // the stretches: row, group, groups
  __shared__ float scale_s[TNW][NST][4];                  // of its keys, of its values, per 16 keys
  __shared__ int there_s[TNW][NST][2];                    // whether these have a block
  uint8_t* ring = sm_raw + ((1024u - (smem_addr(sm_raw) & 1023u)) & 1023u);
  const WinArgs& a = t.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tq = lane & 3;
  const int R = a.g * a.Nq, heads = a.Hkv * t.rtiles;
  auto seq_of = [&](int b) {
    WinSeq q = win_seq(a, b);
    if (!a.q_pos && t.table) q.qp = q.len - a.Nq;
    return q;
  };
  // the groups of a sequence: first tokens' groups, then the window's
  auto groups_of = [&](const WinRange& r) {
    return (r.S + GK - 1) / GK + (r.hi > r.lo ? (r.hi + GK - 1) / GK - r.lo / GK : 0);
  };
  // ---- this warp's stretch of all groups: `mine` of them from `at` on ----
  const int w = blockIdx.x * TNW + warp, W = gridDim.x * TNW;
  long long total = 0;
  for (int b = lane; b < a.B; b += 32) {
    const int G = groups_of(win_keys(a, seq_of(b), 0, a.Nq));
    total += G;
    if (G == 0 && warp < TNW && b % W == w)   // rows that nobody meets
      for (int h = 0; h < heads; ++h) t.info[b * heads + h] = make_int2(0, -1);
  }
#pragma unroll
  for (int k = 16; k; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  total *= heads;
  const int each = max(2, (int)((total + W - 1) / W));
  const long long at = min(total, (long long)w * each);
  const int mine = (int)min(total - at, (long long)each);
  // where it begins: the sequence (a scan over them), row and group
  int b0 = 0, hr0 = 0, gi0 = 0;
  long long base = 0;
  for (int c = 0; c < a.B; c += 32) {
    const int G = c + lane < a.B ? groups_of(win_keys(a, seq_of(c + lane), 0, a.Nq)) : 0;
    long long upto = (long long)G * heads;
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += x;
    }
    const uint32_t who = __ballot_sync(0xffffffffu, at < base + upto);
    if (who) {
      const int src = __ffs(who) - 1;
      const long long off = at - base - __shfl_sync(0xffffffffu, upto - (long long)G * heads, src);
      const int row_groups = __shfl_sync(0xffffffffu, G, src);
      b0 = c + src;
      hr0 = (int)(off / row_groups);
      gi0 = (int)(off - (long long)hr0 * row_groups);
      break;
    }
    base += __shfl_sync(0xffffffffu, upto, 31);
  }

  auto bar = [](uint64_t* x) { return smem_addr(x); };
  if (warp < TNW && lane == 0) {
    start_s[warp][0] = b0; start_s[warp][1] = hr0; start_s[warp][2] = gi0; start_s[warp][3] = mine;
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(bar(&full_s[warp][i]), 2);     // the copies' request, the scales
      tc::mbar_init(bar(&empty_s[warp][i]), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();

  // a place in the stretch: row (b, hr) and its group gi, and the row's ranges
  struct Cursor {
    int b, hr, gi, G, gs, w0;
    WinSeq sq;
    WinRange kr;
  };
  auto enter = [&](Cursor& c) {        // the row's ranges, from the next row with groups on
    for (;;) {
      c.sq = seq_of(c.b);
      c.kr = win_keys(a, c.sq, 0, a.Nq);
      c.G = groups_of(c.kr);
      if (c.G > 0) break;
      ++c.b;                           // (the stretch ends before the last sequence does)
    }
    c.gs = (c.kr.S + GK - 1) / GK;
    c.w0 = c.kr.lo / GK;
  };
  auto step = [&](Cursor& c) {         // true: another row
    if (++c.gi < c.G) return false;
    c.gi = 0;
    if (++c.hr == heads) {
      c.hr = 0;
      ++c.b;
    }
    return true;
  };

  // first key of the cursor's group and the range of keys that its phase counts
  auto group = [&](const Cursor& c, int* j0, int* jb, int* je) {
    const bool f = c.gi < c.gs;
    *j0 = (f ? c.gi : c.w0 + c.gi - c.gs) * GK;
    *jb = f ? 0 : c.kr.lo;
    *je = f ? c.kr.S : c.kr.hi;
  };
  auto has_keys = [](int j, int jb, int je) { return j < je && j + 16 > jb; };
  // the cache blocks that hold the 16-key parts of a group; only those of parts
  // with keys of the phase are looked up
  auto blocks_of = [&](const Cursor& c, int (&blk)[NH]) {
    int j0, jb, je;
    group(c, &j0, &jb, &je);
#pragma unroll
    for (int h = 0; h < NH; ++h)
      blk[h] = has_keys(j0 + 16 * h, jb, je) ? t.table[(size_t)c.b * t.max_blocks + ((j0 + 16 * h) >> t.Tshift)] : -1;
  };
  if (warp == TNW) {
    // ---- copies: lane i fills the ring of warp i, one box of GK rows for each
    // panel of a group, or one for each half where blocks hold 16 tokens ----
    if (lane >= TNW) return;
    const uint32_t base = smem_addr(ring) + lane * NST * SLOT;
    Cursor c;
    c.b = start_s[lane][0]; c.hr = start_s[lane][1]; c.gi = start_s[lane][2];
    const int n = start_s[lane][3];
    int blk[NH] = {};
    if (n > 0) {
      enter(c);
      if (t.table) blocks_of(c, blk);
    }
    int i = 0;
    for (; i < n; ++i) {
      const int st = i % NST;
      const uint32_t full = bar(&full_s[lane][st]);
      if (!wtc::wait_or_flag(t.err, bar(&empty_s[lane][st]), (uint32_t)(i / NST & 1) ^ 1u)) break;
      int j0, jb, je;
      group(c, &j0, &jb, &je);
      const int hk = c.hr / t.rtiles;
      bool there[NH];
      int bh[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        there[h] = true;
        bh[h] = c.b * a.Hkv + hk;
        if (t.table) {
          there[h] = (unsigned)blk[h] < (unsigned)t.blocks;
          if (!there[h] && has_keys(j0 + 16 * h, jb, je)) atomicOr(t.err, 2);
          bh[h] = (there[h] ? blk[h] : 0) * a.Hkv + hk;
        }
      }
      const uint32_t dst = base + st * SLOT;
      const bool one = NH == 1 || t.table == nullptr || t.Tshift > 4;   // one box
      const bool any = there[0] || there[NH - 1];
      tc::mbar_expect_tx(full, one ? (any ? 2 * TILE : 0) : ((int)there[0] + (int)there[NH - 1]) * TILE);
      const int row = t.table ? j0 & ((1 << t.Tshift) - 1) : j0;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (one ? h > 0 || !any : !there[h]) continue;
        const int src = one && !there[0] ? bh[NH - 1] : bh[h];
#pragma unroll
        for (int p = 0; p < PANELS; ++p) {
          const uint32_t to = dst + p * GK * 128 + h * 16 * (RB == 64 ? 64 : 128);
          wtc::tma3(to, &mp.k, p * (128 / ES), row, src, full);
          wtc::tma3(to + TILE, &mp.v, p * (128 / ES), row, src, full);
        }
      }
      if (i + 1 < n) {
        if (step(c)) enter(c);
        if (t.table) blocks_of(c, blk);
      }
      if (t.table) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          scale_s[lane][st][h] = t.k_scale[bh[h]];
          scale_s[lane][st][2 + h] = t.v_scale[bh[h]];
          there_s[lane][st][h] = there[h];
        }
      }
      wtc::arrive(full);
    }
    // every copy has landed before the block ends, also after an expired wait
    for (int k = i > NST ? i - NST : 0; k < i; ++k)
      wtc::wait_or_flag(t.err, bar(&full_s[lane][k % NST]), (uint32_t)(k / NST) & 1u);
    return;
  }
  if (mine <= 0) return;
  uint8_t* my = ring + warp * NST * SLOT;
  Cursor cu;                           // the group to work on
  cu.b = b0; cu.hr = hr0; cu.gi = gi0;
  enter(cu);
  int left = mine;

  // ---- the row's queries: 16 rows are the products' rows, 8 their columns; row[] and
  // qs[] are those of this thread's scores: rows gid and gid + 8, or columns 2 tq and
  // 2 tq + 1 ----
  constexpr int QR = FEW ? 2 : 4;
  WinRow row[2];
  float qs[2];                         // score factor of the row
  uint32_t qf[NP][KS][QR];
  int free_lo = 0, free_hi = -1;       // keys [free_lo, free_hi) every query sees: no mask
  auto queries = [&](const Cursor& c) {
    const int hk = c.hr / t.rtiles, rt = c.hr - hk * t.rtiles;
    const bool rows_ok = c.sq.qp >= 0 && c.sq.qp + a.Nq <= c.sq.len;
    free_lo = c.sq.qp + a.Nq - 1 - a.left;
    free_hi = rows_ok ? min(c.sq.len, c.sq.qp + a.right + 1) : -1;
#pragma unroll
    for (int r = 0; r < ROWS / 8; ++r) {
      const int rr = rt * 16 + gid + 8 * r;
      const bool ok = rr < R;
      const int e = ok ? rr / a.Nq : 0, i = ok ? rr % a.Nq : 0;
      row[r] = ok ? win_row(a, c.sq, i) : WinRow{0, 0, 0};
      const TQ* q = (const TQ*)a.q + (((size_t)c.b * a.Hq + hk * a.g + e) * a.Nq + i) * a.d;
      float4 x[KS];
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        const int f = key_chunk<RB>(tq, s / KSP) * PIECE + (s % KSP) * 4;
        x[s] = ok && f < a.d ? ld4(q + f) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
      float down = 1.f;
      qs[r] = a.scale_log2;
      if constexpr (X::F16) {
        float mx = 0.f;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[s].x), fabsf(x[s].y)), fmaxf(fabsf(x[s].z), fabsf(x[s].w))));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // the largest feature to [2^13, 2^14)
        const int ex = (int)(__float_as_uint(mx) >> 23) - 127 - 13;
        if (mx > 0.f && mx < INFINITY) {
          const int h = max(-126, min(126, -ex));
          down = __uint_as_float((uint32_t)(h + 127) << 23);
          qs[r] *= __uint_as_float((uint32_t)(127 - h) << 23);
        }
      }
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        uint32_t u[NP];
        split<KIND>(x[s].x * down, x[s].y * down, u);
#pragma unroll
        for (int p = 0; p < NP; ++p) qf[p][s][r] = u[p];
        split<KIND>(x[s].z * down, x[s].w * down, u);
#pragma unroll
        for (int p = 0; p < NP; ++p) qf[p][s][QR / 2 + r] = u[p];
      }
    }
    if constexpr (FEW) {
      const float own = qs[0];
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int rr = 2 * tq + e;
        qs[e] = __shfl_sync(0xffffffffu, own, 4 * rr);
        row[e] = rr < R ? win_row(a, c.sq, rr % a.Nq) : WinRow{0, 0, 0};
      }
    }
  };

  float m[2], l[2];
  // reference of the values' scales by row, below all of them at first: o holds v 2^-vref; and
  // the row's maximum beside which what it holds was some 2^vref
  int vref[2];
  float mref[2];
  constexpr int NO = FEW ? NT / 2 : NT;
  float o[NO][4];                    // 16 rows: [n] is column n; 8: [n] features 2 n, 2 n + 1
  auto clear = [&]() {
    m[0] = m[1] = -INFINITY;
    l[0] = l[1] = 0.f;
    vref[0] = vref[1] = kRefMin;
    mref[0] = mref[1] = -INFINITY;
#pragma unroll
    for (int n = 0; n < NO; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  };
  // the row's share to memory: stretch w of row r is part w + r (unique, since one
  // or the other grows from part to part, and a row's are consecutive)
  const int first_gi = gi0;
  auto leave = [&](const Cursor& c) {
    const int rt = c.hr % t.rtiles, rowid = c.b * heads + c.hr;
    const size_t part = (size_t)(w + rowid) * 16;
    // (the lanes that share a row: 4, or the 8 of a column)
    constexpr int X0 = FEW ? 4 : 1, X1 = FEW ? 16 : 2;
#pragma unroll
    for (int r = 0; r < 2; ++r) {
#pragma unroll
      for (int x = X0; x <= X1; x <<= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], x);
      const int rr = FEW ? 2 * tq + r : gid + 8 * r;
      if (rt * 16 + rr >= R) continue;
      if ((FEW ? gid : tq) == 0) t.part_ml[part + rr] = make_float2(m[r], l[r]);
      float* dst = t.part_o + (part + rr) * a.d;
      const float unit = X::F16 ? pow2(vref[r]) : 1.f;
#pragma unroll
      for (int e = 0; e < (FEW ? 1 : 2); ++e)
#pragma unroll
        for (int n = 0; n < NT; n += 4) {
          const int f = n / VP * (128 / ES) + (FEW ? gid : 2 * tq + e) * VP + n % VP;
          if (f >= a.d) continue;
          float4 y;
          if constexpr (FEW)
            y = make_float4(o[n / 2][r], o[n / 2][2 + r], o[n / 2 + 1][r], o[n / 2 + 1][2 + r]);
          else
            y = make_float4(o[n][2 * r + e], o[n + 1][2 * r + e], o[n + 2][2 * r + e], o[n + 3][2 * r + e]);
          st4(dst + f, make_float4(y.x * unit, y.y * unit, y.z * unit, y.w * unit));
        }
    }
    // the row's first and last parts
    if (lane == 0) {
      const bool whole_start = !(c.b == b0 && c.hr == hr0) || first_gi == 0;
      if (whole_start) t.info[rowid].x = w;
      if (c.gi + 1 >= c.G) t.info[rowid].y = w;
    }
  };
  queries(cu);
  clear();

  int st = 0;
  uint32_t ph = 0;                   // phase of the ring's round
#pragma unroll 1
  for (;;) {
    if (!wtc::wait_warp(t.err, bar(&full_s[warp][st]), ph)) break;
    __syncwarp();
    uint8_t* Kt = my + st * SLOT;
    uint8_t* Vt = Kt + TILE;
    int j0, jb, je;
    group(cu, &j0, &jb, &je);
    float ksc[NH], vsc[NH];
    bool there[NH], all = true;        // a part without a block has no keys
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      ksc[h] = vsc[h] = 1.f;
      there[h] = true;
      if (t.table) {
        ksc[h] = scale_s[warp][st][h];
        vsc[h] = scale_s[warp][st][2 + h];
        there[h] = there_s[warp][st][h] != 0;
        all = all && there[h];
      }
    }
    const bool inside = all && j0 >= jb && j0 + GK <= je;
    if (!inside) {
      // value rows that are no keys of the phase: zeros (0 * anything is not 0)
#pragma unroll 1
      for (int id = lane; id < GK * CH; id += 32) {
        const int r = id / CH, j = j0 + r;
        const bool in = (NH > 1 && r >= 16 ? there[NH - 1] : there[0]) && j >= jb && j < je;
        if (!in) *reinterpret_cast<uint4*>(Vt + tile_off<RB, GK>(r, id % CH)) = make_uint4(0, 0, 0, 0);
      }
      tc::fence_async_smem();
      __syncwarp();
    }
    // ---- scores ----
    // 16 rows: [u] is 8 keys, by row r the values [2 r + e] of keys 2 tq + e; 8: [h] is 16
    // keys, the values [2 (u & 1) + e] of key 8 u + gid and column 2 tq + e
    constexpr int NS = FEW ? NH : NU;
    float s[NS][4];
#pragma unroll
    for (int u = 0; u < NS; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
    // fp32 queries: the instruction cuts its sums off instead of rounding them, so it
    // sums up to 8 products and the FP32 pipe adds those up
    float part[NS][4];
    float (*acc)[4] = NP > 1 ? part : s;
#pragma unroll
    for (int i = 0; i < DP / 4 / PIECE; ++i) {
      uint32_t w[NU][4];
      if constexpr (NP > 1) {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) part[u][e] = 0.f;
      }
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint4 kv = *reinterpret_cast<const uint4*>(Kt + tile_off<RB, GK>(8 * u + gid, key_chunk<RB>(tq, i)));
        w[u][0] = kv.x; w[u][1] = kv.y; w[u][2] = kv.z; w[u][3] = kv.w;
      }
      if constexpr (FEW) {
#pragma unroll
        for (int h = 0; h < NH; ++h) {
          const uint32_t (&lo)[4] = w[2 * h], (&hi)[4] = w[2 * h + 1];   // keys gid, gid + 8
          if constexpr (KIND == TK_F32) {
            uint32_t p[4][3];
            split3_bf16x2(__uint_as_float(lo[0]), __uint_as_float(lo[1]), p[0]);
            split3_bf16x2(__uint_as_float(hi[0]), __uint_as_float(hi[1]), p[1]);
            split3_bf16x2(__uint_as_float(lo[2]), __uint_as_float(lo[3]), p[2]);
            split3_bf16x2(__uint_as_float(hi[2]), __uint_as_float(hi[3]), p[3]);
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
              for (int y = 0; y <= x; ++y) {
                const uint32_t k4[4] = {p[0][x - y], p[1][x - y], p[2][x - y], p[3][x - y]};
                mma_bf(acc[h], k4, qf[y][i][0], qf[y][i][1]);
              }
          } else if constexpr (KIND == TK_BF16) {
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const uint32_t k4[4] = {lo[2 * x], hi[2 * x], lo[2 * x + 1], hi[2 * x + 1]};
              mma_bf(acc[h], k4, qf[0][2 * i + x][0], qf[0][2 * i + x][1]);
            }
          } else {
#pragma unroll
            for (int x = 0; x < 4; ++x) {
              const uint32_t k4[4] = {e4m3x2_f16(lo[x]), e4m3x2_f16(hi[x]), e4m3x2_f16(lo[x] >> 16),
                                      e4m3x2_f16(hi[x] >> 16)};
#pragma unroll
              for (int p = NP - 1; p >= 0; --p) mma_f16(acc[h], k4, qf[p][4 * i + x][0], qf[p][4 * i + x][1]);
            }
          }
        }
      } else if constexpr (KIND == TK_F32) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          uint32_t p0[3], p1[3];
          split3_bf16x2(__uint_as_float(w[u][0]), __uint_as_float(w[u][1]), p0);
          split3_bf16x2(__uint_as_float(w[u][2]), __uint_as_float(w[u][3]), p1);
#pragma unroll
          for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int y = 0; y <= x; ++y) mma_bf(acc[u], qf[y][i], p0[x - y], p1[x - y]);
        }
      } else if constexpr (KIND == TK_BF16) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < NU; ++u) mma_bf(acc[u], qf[0][2 * i + x], w[u][2 * x], w[u][2 * x + 1]);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            const uint32_t b0 = e4m3x2_f16(w[u][x]), b1 = e4m3x2_f16(w[u][x] >> 16);
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) mma_f16(acc[u], qf[p][4 * i + x], b0, b1);
          }
      }
      if constexpr (NP > 1) {
#pragma unroll
        for (int u = 0; u < NS; ++u)
#pragma unroll
          for (int e = 0; e < 4; ++e) s[u][e] += part[u][e];
      }
    }
    // ---- softmax, running maximum and sum ----
    const bool whole = inside && j0 + GK <= free_hi &&
                       (j0 >= free_lo || j0 + GK <= a.sinks);
    // value x of row r: its place, its key, its 16 keys
    constexpr int NV = FEW ? NU : 2 * NU, X0 = FEW ? 4 : 1, X1 = FEW ? 16 : 2;
    const auto at = [](int r, int x) { return FEW ? 2 * (x & 1) + r : 2 * r + (x & 1); };
    const auto key = [&](int x) { return FEW ? 8 * x + gid : 8 * (x >> 1) + 2 * tq + (x & 1); };
    constexpr int PER = FEW ? 2 : 4;
    float p[NS][4];
    bool up = false;
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float qk[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) qk[h] = qs[r] * ksc[h];
      float mx = -INFINITY;
#pragma unroll
      for (int x = 0; x < NV; ++x) s[x >> 1][at(r, x)] *= qk[x / PER];
      if (!whole) {
#pragma unroll
        for (int x = 0; x < NV; ++x) {
          const int j = j0 + key(x);
          if (!(there[x / PER] && j >= jb && j < je && win_sees(row[r], j))) s[x >> 1][at(r, x)] = -INFINITY;
        }
      }
#pragma unroll
      for (int x = 0; x < NV; x += 2) mx = fmaxf(fmaxf(mx, s[x >> 1][at(r, x)]), s[x >> 1][at(r, x + 1)]);
#pragma unroll
      for (int x = X0; x <= X1; x <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      mx = fmaxf(mx, m[r]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      f[r] = exp2f(m[r] - mu);
      up = up || mx > m[r];
      m[r] = mx;
      const float off = X::SHIFT - mu;
      float sum = 0.f;
#pragma unroll
      for (int x = 0; x < NV; ++x) {
        const float y = exp2f(s[x >> 1][at(r, x)] + off);
        p[x >> 1][at(r, x)] = y;
        sum += y;
      }
      l[r] = l[r] * f[r] + sum;
    }
    // ---- the values' scales: p becomes p v_scale 2^-vref ----
    // A row's reference follows the largest p v_scale so far, not v_scale alone: large values of
    // no weight may not push small ones with all the weight out of f16.  It is looked at again
    // where a scale is over 2^kRefSlack above it, or below it by as much in a group that moves
    // the row's maximum.  So p v_scale 2^-vref stays below 2^15 and the row's largest above
    // 2^4, and what f16 cuts off (2^-25) is 2^-29 of that or less.
    if constexpr (X::F16) {
      int ex[NH], hi = kRefMin, lo = kRefMax;
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        ex[h] = there[h] ? exponent(vsc[h]) : kRefMin;
        hi = max(hi, ex[h]);
        if (there[h]) lo = min(lo, ex[h]);
      }
      bool move = false;
#pragma unroll
      for (int r = 0; r < 2; ++r)
        move = move || hi > vref[r] + kRefSlack || (f[r] < 1.f && lo < vref[r] - kRefSlack);
      if (__any_sync(0xffffffffu, move)) {
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          int own = kRefMin;               // the group's largest p v_scale, as a power of two above it
#pragma unroll
          for (int h = 0; h < NH; ++h) {
            float w = 0.f;
#pragma unroll
            for (int x = h * PER; x < (h + 1) * PER; ++x) w = fmaxf(w, p[x >> 1][at(r, x)]);
#pragma unroll
            for (int x = X0; x <= X1; x <<= 1) w = fmaxf(w, __shfl_xor_sync(0xffffffffu, w, x));
            if (w > 0.f) own = max(own, ex[h] + exponent(w) + 1 - (int)X::SHIFT);
          }
          // what o holds was 2^vref beside the maximum mref
          const float held = (float)vref[r] + fmaxf(mref[r] - m[r], -400.f);
          int to = max(own, (int)ceilf(held));
          if (m[r] == -INFINITY) to = hi;  // nothing seen so far
          to = min(max(to, hi - 120), kRefMax);   // (the factors below are finite)
          if (to > vref[r] || to < vref[r] - kRefSlack) {
            f[r] = scalbnf(f[r], vref[r] - to);
            vref[r] = to;
          }
          mref[r] = m[r] + (fmaxf(held, (float)own) - (float)vref[r]);
        }
        up = true;
      } else {
#pragma unroll
        for (int r = 0; r < 2; ++r)
          if (f[r] < 1.f) mref[r] = m[r];
      }
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const float inv = pow2(-vref[r]);
        float to[NH];
#pragma unroll
        for (int h = 0; h < NH; ++h) to[h] = there[h] ? vsc[h] * inv : 0.f;
#pragma unroll
        for (int x = 0; x < NV; ++x) p[x >> 1][at(r, x)] *= to[x / PER];
      }
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int n = 0; n < NO; ++n) {
        o[n][0] *= f[0]; o[n][1] *= f[FEW]; o[n][2] *= f[!FEW]; o[n][3] *= f[1];
      }
    }
    // ---- P V ----
    uint32_t pf[NP][NH][QR];
    if constexpr (FEW) {                   // keys by columns to columns by keys
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        uint32_t w[NP];
        split<KIND>(p[u >> 1][2 * (u & 1)], p[u >> 1][2 * (u & 1) + 1], w);
#pragma unroll
        for (int x = 0; x < NP; ++x) pf[x][u >> 1][u & 1] = turn(w[x]);
      }
    } else {
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t w[NP];
          split<KIND>(p[u][2 * r], p[u][2 * r + 1], w);
#pragma unroll
          for (int x = 0; x < NP; ++x) pf[x][u >> 1][2 * (u & 1) + r] = w[x];
        }
    }
    // adds the values' features n and n + 1 (b: n, c: n + 1; keys 2 tq.. and 8 further)
    const auto add = [&](float (*acc)[4], int x, int g, uint32_t b0, uint32_t b1, uint32_t c0, uint32_t c1) {
      if constexpr (FEW) {
        const uint32_t v4[4] = {b0, c0, b1, c1};
        if constexpr (X::F16) mma_f16(acc[0], v4, pf[x][g][0], pf[x][g][1]);
        else mma_bf(acc[0], v4, pf[x][g][0], pf[x][g][1]);
      } else {
        if constexpr (X::F16) {
          mma_f16(acc[0], pf[x][g], b0, b1);
          mma_f16(acc[1], pf[x][g], c0, c1);
        } else {
          mma_bf(acc[0], pf[x][g], b0, b1);
          mma_bf(acc[1], pf[x][g], c0, c1);
        }
      }
    };
    constexpr int OS = FEW ? 2 : 1;        // features of an o[n]
    // o += what `sum` adds to zeros (fp32 queries), or sum(o)
    const auto into = [&](float (*acc)[4], auto sum) {
      if constexpr (NP > 1) {
        float part[2][4] = {};
        sum(part);
#pragma unroll
        for (int i = 0; i < 2 / OS; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) acc[i][e] += part[i][e];
      } else {
        sum(acc);
      }
    };
#pragma unroll
    for (int g = 0; g < NU / 2; ++g) {     // 16 keys each
      if constexpr (X::F16) {
        constexpr int W = DP / 8 / 4;  // 32-bit words of a thread's piece of a value row
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + tile_off<RB, GK>(rr, gid));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(Vt + tile_off<RB, GK>(rr, gid >> 1) + 8 * (gid & 1));
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          const int sel = (n & 3) | (((n & 3) + 4) << 4), nxt = sel + 0x11;
          const uint32_t b0 = e4m3x2_f16(__byte_perm(v[0][n >> 2], v[1][n >> 2], sel));
          const uint32_t b1 = e4m3x2_f16(__byte_perm(v[2][n >> 2], v[3][n >> 2], sel));
          const uint32_t c0 = e4m3x2_f16(__byte_perm(v[0][n >> 2], v[1][n >> 2], nxt));
          const uint32_t c1 = e4m3x2_f16(__byte_perm(v[2][n >> 2], v[3][n >> 2], nxt));
          into(&o[n / OS], [&](float (*to)[4]) {
#pragma unroll
            for (int x = NP - 1; x >= 0; --x) add(to, x, g, b0, b1, c0, c1);
          });
        }
      } else if constexpr (KIND == TK_BF16) {
#pragma unroll
        for (int h = 0; h < PANELS; ++h) {
          uint32_t v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + tile_off<RB, GK>(rr, 8 * h + gid));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          }
#pragma unroll
          for (int n = 0; n < 8; n += 2)
            add(&o[(8 * h + n) / OS], 0, g, __byte_perm(v[0][n >> 1], v[1][n >> 1], 0x5410),
                __byte_perm(v[2][n >> 1], v[3][n >> 1], 0x5410),
                __byte_perm(v[0][n >> 1], v[1][n >> 1], 0x7632),
                __byte_perm(v[2][n >> 1], v[3][n >> 1], 0x7632));
        }
      } else {
#pragma unroll
        for (int h = 0; h < PANELS; ++h) {
          float v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
            const float4 x = *reinterpret_cast<const float4*>(Vt + tile_off<RB, GK>(rr, 8 * h + gid));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          }
#pragma unroll
          for (int n = 0; n < 4; n += 2) {
            uint32_t b0[3], b1[3], c0[3], c1[3];
            split3_bf16x2(v[0][n], v[1][n], b0);
            split3_bf16x2(v[2][n], v[3][n], b1);
            split3_bf16x2(v[0][n + 1], v[1][n + 1], c0);
            split3_bf16x2(v[2][n + 1], v[3][n + 1], c1);
            into(&o[(4 * h + n) / OS], [&](float (*to)[4]) {
#pragma unroll
              for (int x = 2; x >= 0; --x)
#pragma unroll
                for (int y = 0; y <= x; ++y) add(to, y, g, b0[x - y], b1[x - y], c0[x - y], c1[x - y]);
            });
          }
        }
      }
    }
    __syncwarp();                      // the slot is read
    if (lane == 0) wtc::arrive(bar(&empty_s[warp][st]));
    if (++st == NST) {
      st = 0;
      ph ^= 1u;
    }
    const bool last = --left == 0;
    if (last || cu.gi + 1 >= cu.G) leave(cu);
    if (last) break;
    if (step(cu)) {
      enter(cu);
      queries(cu);
      clear();
    }
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// out = sum over a row's parts: a block a row, its warps take parts in turn
template <typename TQ>
__global__ void __launch_bounds__(32 * JNW) k_token_join(TokenArgs t, float shift) {
  __shared__ __align__(16) float So[JNW][128];
  __shared__ float Sl[JNW];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while k_token still ran
  const int warps = blockDim.x >> 5;
  const WinArgs& a = t.w;
  const long long qrow = blockIdx.x;                     // (b, query head, query)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = 4 * lane;
  const int i = (int)(qrow % a.Nq), hq = (int)(qrow / a.Nq % a.Hq), b = (int)(qrow / a.Nq / a.Hq);
  const int rr = (hq % a.g) * a.Nq + i;
  const size_t rowid = ((size_t)b * a.Hkv + hq / a.g) * t.rtiles + rr / 16;
  const int2 in = t.info[rowid];
  // parts; 0: the row sees nothing (or its warps gave up after an expired wait)
  const int n = in.x >= 0 && in.y < t.grid * TNW && in.y >= in.x ? in.y - in.x + 1 : 0;
  const size_t row0 = (rowid + in.x) * 16 + rr % 16;
  float mx = -INFINITY;
  for (int s = lane; s < n; s += 32) mx = fmaxf(mx, t.part_ml[row0 + (size_t)s * 16].x);
#pragma unroll
  for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = warp; s < n; s += warps) {
    const size_t row = row0 + (size_t)s * 16;
    const float2 x = t.part_ml[row];
    const float f = exp2f(x.x - mu);
    sum = fmaf(x.y, f, sum);
    if (c < a.d) {
      const float4 v = *reinterpret_cast<const float4*>(t.part_o + row * a.d + c);
      acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
    }
  }
  st4(&So[warp][c], acc);
  if (lane == 0) Sl[warp] = sum;
  __syncthreads();
  if (warp) return;
  for (int w = 1; w < warps; ++w) {
    const float4 v = lds4(&So[w][c]);
    sum += Sl[w];
    acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
  }
  const float w = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < a.d) {
    const float4 y = make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w);
    st4((TQ*)a.out + qrow * a.d + c, y);
    if (a.rest)
      *reinterpret_cast<uint2*>((__nv_bfloat16*)a.rest + qrow * a.d + c) =
          make_uint2(wtc::pack_rest(y.x, y.y, wtc::pack(y.x, y.y)), wtc::pack_rest(y.z, y.w, wtc::pack(y.z, y.w)));
  }
  if (a.lse && lane == 0) a.lse[qrow] = sum == 0.f ? -INFINITY : mx + log2f(sum) - shift;
}

namespace {
template <int KIND>
int blocks_of(int d, bool eight) {
  if (d <= 64) return eight ? token_blocks<KIND, 64, 8>() : token_blocks<KIND, 64, 16>();
  return eight ? token_blocks<KIND, 128, 8>() : token_blocks<KIND, 128, 16>();
}
int slots_of(int kind, int d, bool eight) {
  const int sms = 152;   // from the type alone: workspaces do not depend on the device
  switch (kind) {
    case TK_BF16: return sms * blocks_of<TK_BF16>(d, eight);
    case TK_E4M3: return sms * blocks_of<TK_E4M3>(d, eight);
    case TK_E4M3_F32: return sms * blocks_of<TK_E4M3_F32>(d, eight);
    default: return sms * blocks_of<TK_F32>(d, eight);
  }
}
int kind_of(bool cache, bool bf16) {
  return cache ? (bf16 ? TK_E4M3 : TK_E4M3_F32) : (bf16 ? TK_BF16 : TK_F32);
}

template <int KIND, int DP, int ROWS>
cudaError_t go(TokenArgs& t, cudaStream_t st) {
  using TQ = typename std::conditional<Kind<KIND>::QF32, float, __nv_bfloat16>::type;
  constexpr size_t smem = token_smem<KIND, DP, ROWS>();
  static SmemOnce once;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once.allow(k_token<KIND, DP, ROWS>, smem, dev)) != cudaSuccess) return e;
  // a panel's features x the rows of a copy: a group, or a block of 16 tokens
  TokenMaps mp;
  constexpr int ES = Kind<KIND>::ES;
  const WinArgs& a = t.w;
  const int box = t.table && t.Tshift == 4 ? 16 : Kind<KIND>::GK;
  const int N = t.table ? 1 << t.Tshift : a.Nk;
  const long long outer = t.table ? (long long)t.blocks * a.Hkv : (long long)a.B * a.Hkv;
  for (int i = 0; i < 2; ++i)
    if (!encode_tiled_rows(i ? &mp.v : &mp.k, i ? a.v : a.k, ES, a.d, N, outer, DP * ES == 64 ? 64 : 128, box))
      return cudaErrorInvalidValue;
  e = launch("token_attention", k_token<KIND, DP, ROWS>, dim3((unsigned)t.grid), dim3(32 * TNW + 32), smem, st, mp, t);
  if (e != cudaSuccess) return e;
  const long long rows = (long long)t.w.B * t.w.Hq * t.w.Nq;
  // rows of many parts (32 on the average): more warps (4 sequences of 131072 tokens, 76
  // parts: 16.4 us with 4 warps, 10.5 with 16; 32 sequences of 8192, 7 parts: 8.1 and 11.5)
  const long long tiles = (long long)a.B * a.Hkv * t.rtiles;
  const int warps = (long long)t.grid * TNW >= 32 * tiles ? JNW : 4;
  return launch_after("token_join", k_token_join<TQ>, dim3((unsigned)rows), dim3(32 * warps), 0, st, t,
                      Kind<KIND>::SHIFT);
}
}  // namespace

TokenShape token_shape(bool cache, bool bf16, int B, int Hkv, int g, int Nq, int d, long long keys,
                       int left, int right, int sinks) {
  TokenShape s;
  s.rtiles = (g * Nq + 15) / 16;
  // all blocks at once, but no more warps than stretches of two groups
  long long seen = keys;
  if (left < kWinUnbounded && right < kWinUnbounded) {
    const long long w = (long long)left + right + Nq + sinks + 64;
    if (w < seen) seen = w;
  }
  const long long rows = (long long)B * Hkv * s.rtiles, groups = rows * (seen / 16 + 3);
  s.grid = slots_of(kind_of(cache, bf16), d, g * Nq <= 8);
  const long long most = (groups + 2 * TNW - 1) / (2 * TNW);
  if (most < s.grid) s.grid = (int)most;
  const size_t parts = (size_t)rows + (size_t)s.grid * TNW;
  s.o_bytes = parts * 16 * d * 4;
  s.ml_bytes = parts * 16 * 8;
  s.info_bytes = (size_t)rows * 8;
  return s;
}

template <int KIND>
static cudaError_t go_kind(TokenArgs& t, cudaStream_t st) {
  const bool eight = t.w.g * t.w.Nq <= 8;
  if (t.w.d <= 64) return eight ? go<KIND, 64, 8>(t, st) : go<KIND, 64, 16>(t, st);
  return eight ? go<KIND, 128, 8>(t, st) : go<KIND, 128, 16>(t, st);
}
cudaError_t run_token(TokenArgs& t, bool bf16, cudaStream_t st) {
  if (t.table) return bf16 ? go_kind<TK_E4M3>(t, st) : go_kind<TK_E4M3_F32>(t, st);
  return bf16 ? go_kind<TK_BF16>(t, st) : go_kind<TK_F32>(t, st);
}

}  // namespace lapnys
