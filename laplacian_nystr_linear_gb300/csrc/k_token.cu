// Windowed softmax attention for a few queries per sequence (single tokens, or
// the few of a step that answers): over plain keys and values (bf16, fp32), or
// over a cache of 8-bit values in blocks with one power-of-two scale per block
// and head (k = k8 * k_scale, v = v8 * v_scale).  Visibility rule: win.cuh.
//
// What bounds it: every visible key and value is read once, for all the query
// heads that share it, and nothing else is large.  So the work is split over the
// keys: a block takes one (sequence, key head, 16 query rows) and one contiguous
// share of the visible groups of 16 or 32 keys, its warps take groups in turn, each
// with a ring of asynchronous copies of its own (no block barrier in the loop),
// and k_token_join adds the shares.  Shares are cut on the device, from all
// sequences' lengths, so that they are alike in a ragged batch and, where it can
// be, all blocks run at once: a block's start and end (dependent loads of the
// lengths, the table, the queries; the join of its warps) cost 4 us, as much as
// 0.2 MB of cache.
//
// Products on the warp-level tensor instruction (m16n8k16), rows = (query head
// of the group, query), with the contraction's order chosen so that no operand
// is transposed or gathered: a thread's four k of step s are four neighbouring
// features (scores), and column n of output step nt is feature n DP / 8 + nt
// (P V), so both operands come from shared memory in 16-byte reads without bank
// conflicts (the swizzles below).
//   - 8-bit: e4m3 -> f16 is exact (one instruction for two; the e4m3 form of the
//     product is no instruction of its own here: it ran as two f16 ones with more
//     conversions, 1576 instructions for 32 keys against about 600).  q is scaled
//     per row by a power of two to fit f16 (features below 2^-38 of the row's
//     largest are lost).  p is kept as 2^10 p (v_scale / reference) in f16, the
//     reference a scale of the values seen so far, so that P V adds up without a
//     product per element; outputs are rescaled when the reference moves.  fp32
//     queries: q and p in two f16 parts (2^-22).
//   - bf16: q, k, v as they are, p rounded to bf16 (2^-9, below the rounding of
//     the output; sums, maxima and outputs are fp32 throughout).
//   - fp32: all operands in three bf16 parts, six products (2^-24 each).
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "win.cuh"

namespace lapnys {

namespace {
constexpr int TNW = 4;      // warps of a block
enum : int { TK_BF16 = 0, TK_E4M3 = 1, TK_E4M3_F32 = 2, TK_F32 = 3 };

template <int KIND>
struct Kind {
  static constexpr int ES = KIND == TK_F32 ? 4 : (KIND == TK_BF16 ? 2 : 1);  // bytes of k, v
  static constexpr bool QF32 = KIND == TK_E4M3_F32 || KIND == TK_F32;
  static constexpr bool F16 = KIND == TK_E4M3 || KIND == TK_E4M3_F32;  // f16 products
  static constexpr int GK = KIND == TK_E4M3 ? 32 : 16;                  // keys of a group
  static constexpr int PARTS = KIND == TK_F32 ? 3 : (KIND == TK_E4M3_F32 ? 2 : 1);
  static constexpr float SHIFT = F16 ? 10.f : 0.f;  // p is held as 2^SHIFT p
  static constexpr int TRAIL = 32;          // bytes behind a ring slot: scales of the keys, of the
                                            // values, and whether there is a block, per 16 keys
};
template <int KIND, int DP>
__host__ __device__ constexpr int ring_stages() { return DP == 128 && KIND != TK_E4M3_F32 ? 3 : 4; }
template <int KIND, int DP>
__host__ __device__ constexpr size_t token_smem() {
  return (size_t)TNW * ring_stages<KIND, DP>() * (2 * Kind<KIND>::GK * DP * Kind<KIND>::ES + Kind<KIND>::TRAIL);
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
// two e4m3 values (low 16 bits) -> two f16, exact
__device__ __forceinline__ uint32_t e4m3x2_f16(uint32_t v) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)v));
  return r;
}
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

// byte offset of a row's 16-byte chunk in a tile of rows of RB bytes.  A key
// row is read 16 bytes per thread at chunk t + 4 i of rows gid (t = lane % 4,
// gid = lane / 4): odd rows swap their halves.
template <int RB>
__device__ __forceinline__ uint32_t k_off(int row, int c) {
  return (uint32_t)(row * RB + ((RB >= 128 ? c ^ ((row & 1) << 2) : c) << 4));
}
// a value row is read from rows 2 t + const at chunk(s) gid.. : eight lanes of a
// phase hold two gid and four t, spread over the eight chunks of a line
template <int RB>
__device__ __forceinline__ uint32_t v_off(int row, int c) {
  if constexpr (RB == 64) {
    const int line = row >> 1, cc = (((row & 1) << 2) | c) ^ ((line & 3) << 1);
    return (uint32_t)(line * 128 + (cc << 4));
  } else if constexpr (RB == 128) {
    return (uint32_t)(row * RB + ((c ^ (row & 6)) << 4));
  } else if constexpr (RB == 256) {
    return (uint32_t)(row * RB + ((c ^ (((row >> 1) & 1) | (((row >> 2) & 1) << 2))) << 4));
  } else {
    return (uint32_t)(row * RB + ((c ^ ((row >> 1) & 3)) << 4));
  }
}
__device__ __forceinline__ void cp_async4(uint32_t dst, const void* src) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(dst), "l"(src) : "memory");
}
}  // namespace

template <int KIND, int DP>
__global__ void __launch_bounds__(32 * TNW) k_token(TokenArgs t) {
  using X = Kind<KIND>;
  constexpr int ES = X::ES, RB = DP * ES, NP = X::PARTS, GK = X::GK, NU = GK / 8, NH = GK / 16;
  constexpr int NST = ring_stages<KIND, DP>();
  constexpr int TILE = GK * RB, STG = 2 * TILE, SLOT = STG + X::TRAIL;
  constexpr int KS = DP / 16;                  // 16-feature steps of the scores
  constexpr int NT = DP / 8;                   // column steps of P V
  constexpr int PIECE = 16 / ES;               // features of a 16-byte piece
  constexpr int KSP = PIECE / 4;               // steps of a piece, four features a thread each
  constexpr int CH = RB / 16;                  // 16-byte chunks of a row
  constexpr int RPI = 32 / CH;                 // rows that a warp copies at once
  using TQ = typename std::conditional<X::QF32, float, __nv_bfloat16>::type;
  extern __shared__ __align__(128) uint8_t ring[];
  const WinArgs& a = t.w;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tq = lane & 3;
  const int R = a.g * a.Nq, heads = a.Hkv * t.rtiles;
  // the groups of sequence b: first tokens' groups, then the window's
  auto seq_of = [&](int b) {
    WinSeq q = win_seq(a, b);
    if (!a.q_pos && t.table) q.qp = q.len - a.Nq;
    return q;
  };
  auto groups_of = [&](const WinRange& r) {
    return (r.S + GK - 1) / GK + (r.hi > r.lo ? (r.hi + GK - 1) / GK - r.lo / GK : 0);
  };
  // ---- this block's share: every warp goes over the sequences ----
  // shares of at most L groups; L such that all shares run at once where more
  // blocks do than there are rows to share out
  long long total = 0;
  for (int b = lane; b < a.B; b += 32) total += groups_of(win_keys(a, seq_of(b), 0, a.Nq));
#pragma unroll
  for (int k = 16; k; k >>= 1) total += __shfl_xor_sync(0xffffffffu, total, k);
  const int rows = a.B * heads;
  const int want = t.slots > 2 * rows ? t.slots - rows : t.slots;
  const int L = max(2 * TNW, (int)((total * heads + want - 1) / want));
  int base = 0, b = -1, share = 0, shares = 1;
  for (int b0 = 0; b0 < a.B; b0 += 32) {
    const int n = b0 + lane < a.B ? max(1, (groups_of(win_keys(a, seq_of(b0 + lane), 0, a.Nq)) + L - 1) / L) : 0;
    int upto = n;                     // shares of one (head, row tile), up to this sequence
#pragma unroll
    for (int k = 1; k < 32; k <<= 1) {
      const int x = __shfl_up_sync(0xffffffffu, upto, k);
      if (lane >= k) upto += x;
    }
    const bool mine = n > 0 && (int)blockIdx.x >= base + (upto - n) * heads && (int)blockIdx.x < base + upto * heads;
    const uint32_t who = __ballot_sync(0xffffffffu, mine);
    if (who) {
      const int src = __ffs(who) - 1;
      b = b0 + src;
      shares = __shfl_sync(0xffffffffu, n, src);
      share = blockIdx.x - (base + (__shfl_sync(0xffffffffu, upto, src) - shares) * heads);
      break;
    }
    base += __shfl_sync(0xffffffffu, upto, 31) * heads;
  }
  if (b < 0) return;                  // more blocks than shares
  const int sp = share % shares, hr = share / shares;
  const int hk = hr / t.rtiles, rt = hr - hk * t.rtiles;
  const WinSeq sq = seq_of(b);
  const WinRange kr = win_keys(a, sq, 0, a.Nq);
  // keys [free_lo, free_hi) (or first tokens) are seen by every query: no mask
  const bool rows_ok = sq.qp >= 0 && sq.qp + a.Nq <= sq.len;
  const int free_lo = sq.qp + a.Nq - 1 - a.left, free_hi = rows_ok ? min(sq.len, sq.qp + a.right + 1) : -1;
  const int gs = (kr.S + GK - 1) / GK, w0 = kr.lo / GK, G = groups_of(kr);
  const int g0 = (int)((long long)G * sp / shares), g1 = (int)((long long)G * (sp + 1) / shares);
  if (sp == 0 && tid == 0) t.info[b * heads + hr] = make_int2(blockIdx.x, shares);

  uint8_t* my = ring + warp * NST * SLOT;
  const uint32_t my_s = smem_addr(my);
  const size_t plain = ((size_t)b * a.Hkv + hk) * a.Nk;
  // what a lane copies: chunk `lc` of rows lr, lr + RPI, ..
  const int lr = lane / CH, lc = lane % CH;

  // first key of group gi and the range of keys that its phase counts
  auto group = [&](int gi, int* j0, int* jb, int* je) {
    const bool f = gi < gs;
    *j0 = (f ? gi : w0 + gi - gs) * GK;
    *jb = f ? 0 : kr.lo;
    *je = f ? kr.S : kr.hi;
  };
  auto has_keys = [](int j, int jb, int je) { return j < je && j + 16 > jb; };
  // the cache blocks that hold the 16-key parts of group gi; only those of parts
  // with keys of the phase are looked up
  auto blocks_of = [&](int gi, int (&blk)[NH]) {
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
#pragma unroll
    for (int h = 0; h < NH; ++h)
      blk[h] = has_keys(j0 + 16 * h, jb, je) ? t.table[(size_t)b * t.max_blocks + ((j0 + 16 * h) >> t.Tshift)] : -1;
  };
  // copies of group gi into ring slot st
  auto issue = [&](int gi, int st, const int (&blk)[NH]) {
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
    const uint32_t dst = my_s + st * SLOT;
    size_t tok[NH];
    bool there[NH], full = j0 >= jb && j0 + GK <= je && a.d == DP;
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      there[h] = true;
      if (t.table) {
        there[h] = (unsigned)blk[h] < (unsigned)t.blocks;
        if (!there[h] && lane == 0 && has_keys(j0 + 16 * h, jb, je)) atomicOr(t.err, 2);
        const size_t bh = (size_t)(there[h] ? blk[h] : 0) * a.Hkv + hk;
        tok[h] = (bh << t.Tshift) + ((j0 + 16 * h) & ((1 << t.Tshift) - 1));
        if (lane == 0) {
          cp_async4(dst + STG + 4 * h, t.k_scale + bh);
          cp_async4(dst + STG + 8 + 4 * h, t.v_scale + bh);
          *reinterpret_cast<int*>(my + st * SLOT + STG + 16 + 4 * h) = there[h];
        }
      } else {
        tok[h] = plain + j0 + 16 * h;
      }
      full = full && there[h];
    }
    const uint8_t* gk[NH];
    const uint8_t* gv[NH];
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      const size_t off = ((tok[h] + lr) * a.d + lc * PIECE) * ES;
      gk[h] = (const uint8_t*)a.k + off;
      gv[h] = (const uint8_t*)a.v + off;
    }
    if (full) {
#pragma unroll
      for (int u = 0; u < GK / RPI; ++u) {
        constexpr int RH = 16 / RPI;       // copies of a half
        const int off = (u % RH) * RPI * RB;
        cp_async16(dst + k_off<RB>(u * RPI + lr, lc), gk[u / RH] + off, true);
        cp_async16(dst + TILE + v_off<RB>(u * RPI + lr, lc), gv[u / RH] + off, true);
      }
    } else {
#pragma unroll 1
      for (int u = 0; u < GK / RPI; ++u) {
        const int r = u * RPI + lr, h = NH > 1 ? r >> 4 : 0;
        const bool in = NH > 1 && h ? there[NH - 1] : there[0];
        const bool ok = in && lc * PIECE < a.d && j0 + r >= jb && j0 + r < je;
        const size_t off = (size_t)(r % 16 - lr) * a.d * ES;
        const uint8_t* pk = NH > 1 && h ? gk[NH - 1] : gk[0];
        const uint8_t* pv = NH > 1 && h ? gv[NH - 1] : gv[0];
        cp_async16(dst + k_off<RB>(r, lc), ok ? pk + off : (const uint8_t*)a.k, ok);
        cp_async16(dst + TILE + v_off<RB>(r, lc), ok ? pv + off : (const uint8_t*)a.v, ok);
      }
    }
  };

  int gi = g0 + warp, gn = gi;       // group to compute, group to issue
  int blk[NH] = {};
  if (t.table && gn < g1) blocks_of(gn, blk);
#pragma unroll
  for (int st = 0; st < NST - 1; ++st) {
    if (gn < g1) issue(gn, st, blk);
    gn += TNW;
    if (t.table && gn < g1) blocks_of(gn, blk);
    cp_commit();
  }

  // the rows this thread meets: gid and gid + 8 of the tile
  WinRow row[2];
  float qs[2];                       // score factor of the row
  uint32_t qf[NP][KS][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int rr = rt * 16 + gid + 8 * r;
    const bool ok = rr < R;
    const int e = ok ? rr / a.Nq : 0, i = ok ? rr % a.Nq : 0;
    row[r] = ok ? win_row(a, sq, i) : WinRow{0, 0, 0};
    const TQ* q = (const TQ*)a.q + (((size_t)b * a.Hq + hk * a.g + e) * a.Nq + i) * a.d;
    float4 x[KS];
    float mx = 0.f;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      const int c = (tq + 4 * (s / KSP)) * PIECE + (s % KSP) * 4;
      x[s] = ok && c < a.d ? ld4(q + c) : make_float4(0.f, 0.f, 0.f, 0.f);
      mx = fmaxf(mx, fmaxf(fmaxf(fabsf(x[s].x), fabsf(x[s].y)), fmaxf(fabsf(x[s].z), fabsf(x[s].w))));
    }
    float down = 1.f;
    qs[r] = a.scale_log2;
    if constexpr (X::F16) {
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
      uint32_t w[NP];
      split<KIND>(x[s].x * down, x[s].y * down, w);
#pragma unroll
      for (int p = 0; p < NP; ++p) qf[p][s][r] = w[p];
      split<KIND>(x[s].z * down, x[s].w * down, w);
#pragma unroll
      for (int p = 0; p < NP; ++p) qf[p][s][2 + r] = w[p];
    }
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float vref = 1.f;                  // reference of the values' scales: v = vref x what o holds
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  int st = 0;
#pragma unroll 1
  for (; gi < g1; gi += TNW) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();
    // the slot of the group before is free: its copies run under this group's work
    if (gn < g1) issue(gn, st == 0 ? NST - 1 : st - 1, blk);
    gn += TNW;
    if (t.table && gn < g1) blocks_of(gn, blk);
    cp_commit();
    const uint8_t* Kt = my + st * SLOT;
    const uint8_t* Vt = Kt + TILE;
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
    float ksc[NH], vsc[NH];
    bool there[NH], all = true;        // a part without a block has no keys
#pragma unroll
    for (int h = 0; h < NH; ++h) {
      ksc[h] = vsc[h] = 1.f;
      there[h] = true;
      if (t.table) {
        ksc[h] = reinterpret_cast<const float*>(Kt + STG)[h];
        vsc[h] = reinterpret_cast<const float*>(Kt + STG)[2 + h];
        there[h] = reinterpret_cast<const int*>(Kt + STG)[4 + h] != 0;
        all = all && there[h];
      }
    }
    // ---- scores ----
    float s[NU][4];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
#pragma unroll
    for (int i = 0; i < DP / 4 / PIECE; ++i) {
      uint32_t w[NU][4];
#pragma unroll
      for (int u = 0; u < NU; ++u) {
        const uint4 kv = *reinterpret_cast<const uint4*>(Kt + k_off<RB>(8 * u + gid, tq + 4 * i));
        w[u][0] = kv.x; w[u][1] = kv.y; w[u][2] = kv.z; w[u][3] = kv.w;
      }
      if constexpr (KIND == TK_F32) {
#pragma unroll
        for (int u = 0; u < NU; ++u) {
          uint32_t p0[3], p1[3];
          split3_bf16x2(__uint_as_float(w[u][0]), __uint_as_float(w[u][1]), p0);
          split3_bf16x2(__uint_as_float(w[u][2]), __uint_as_float(w[u][3]), p1);
#pragma unroll
          for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int y = 0; y <= x; ++y) mma_bf(s[u], qf[y][i], p0[x - y], p1[x - y]);
        }
      } else if constexpr (KIND == TK_BF16) {
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int u = 0; u < NU; ++u) mma_bf(s[u], qf[0][2 * i + x], w[u][2 * x], w[u][2 * x + 1]);
      } else {
#pragma unroll
        for (int x = 0; x < 4; ++x)
#pragma unroll
          for (int u = 0; u < NU; ++u) {
            const uint32_t b0 = e4m3x2_f16(w[u][x]), b1 = e4m3x2_f16(w[u][x] >> 16);
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) mma_f16(s[u], qf[p][4 * i + x], b0, b1);
          }
      }
    }
    // ---- softmax, running maximum and sum ----
    const bool whole = all && j0 >= jb && j0 + GK <= je && j0 + GK <= free_hi &&
                       (j0 >= free_lo || j0 + GK <= a.sinks);
    float p[NU][4];
    bool up = false;
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float qk[NH];
#pragma unroll
      for (int h = 0; h < NH; ++h) qk[h] = qs[r] * ksc[h];
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) s[u][2 * r + e] *= qk[u / 2];
      if (!whole) {
#pragma unroll
        for (int u = 0; u < NU; ++u)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int j = j0 + 8 * u + 2 * tq + e;
            if (!(there[u / 2] && j >= jb && j < je && win_sees(row[r], j))) s[u][2 * r + e] = -INFINITY;
          }
      }
#pragma unroll
      for (int u = 0; u < NU; ++u) mx = fmaxf(fmaxf(mx, s[u][2 * r]), s[u][2 * r + 1]);
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = fmaxf(mx, m[r]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      f[r] = exp2f(m[r] - mu);
      up = up || mx > m[r];
      m[r] = mx;
      const float off = X::SHIFT - mu;
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < NU; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = exp2f(s[u][2 * r + e] + off);
          p[u][2 * r + e] = x;
          sum += x;
        }
      l[r] = l[r] * f[r] + sum;
    }
    if (__any_sync(0xffffffffu, up)) {
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        o[n][0] *= f[0]; o[n][1] *= f[0]; o[n][2] *= f[1]; o[n][3] *= f[1];
      }
    }
    // ---- P V ----
    if constexpr (X::F16) {
      // p (v_scale / reference): the reference follows a larger scale at once, and
      // a smaller one below 2^-16 of it (one below 2^-64, as of a block of zeros,
      // adds less than fp32 holds beside what it was set for)
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        if (!there[h]) continue;
        const float r = vsc[h] / vref;
        if (r > 1.f || (r < 0x1p-16f && r >= 0x1p-64f)) {
          const float x = vref / vsc[h];
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[n][e] *= x;
          vref = vsc[h];
        }
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) {
        const float r = there[h] ? vsc[h] / vref : 0.f;
        if (r != 1.f) {
#pragma unroll
          for (int u = 2 * h; u < 2 * h + 2; ++u)
#pragma unroll
            for (int e = 0; e < 4; ++e) p[u][e] *= r;
        }
      }
    }
    uint32_t pf[NP][NU / 2][4];
#pragma unroll
    for (int u = 0; u < NU; ++u)
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t w[NP];
        split<KIND>(p[u][2 * r], p[u][2 * r + 1], w);
#pragma unroll
        for (int x = 0; x < NP; ++x) pf[x][u >> 1][2 * (u & 1) + r] = w[x];
      }
#pragma unroll
    for (int g = 0; g < NU / 2; ++g) {     // 16 keys each
      if constexpr (X::F16) {
        constexpr int W = DP / 8 / 4;  // 32-bit words of a thread's piece of a value row
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + v_off<RB>(rr, gid));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(Vt + v_off<RB>(rr, gid >> 1) + 8 * (gid & 1));
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          const int sel = (n & 3) | (((n & 3) + 4) << 4);
          const uint32_t b0 = e4m3x2_f16(__byte_perm(v[0][n >> 2], v[1][n >> 2], sel));
          const uint32_t b1 = e4m3x2_f16(__byte_perm(v[2][n >> 2], v[3][n >> 2], sel));
#pragma unroll
          for (int x = NP - 1; x >= 0; --x) mma_f16(o[n], pf[x][g], b0, b1);
        }
      } else if constexpr (KIND == TK_BF16) {
        constexpr int W = DP / 16;
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
          uint32_t v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + v_off<RB>(rr, gid * (W / 4) + h));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int sel = n & 1 ? 0x7632 : 0x5410;
            mma_bf(o[8 * h + n], pf[0][g], __byte_perm(v[0][n >> 1], v[1][n >> 1], sel),
                   __byte_perm(v[2][n >> 1], v[3][n >> 1], sel));
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < DP / 32; ++h) {
          float v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 16 * g + 2 * tq + (e & 1) + 8 * (e >> 1);
            const float4 x = *reinterpret_cast<const float4*>(Vt + v_off<RB>(rr, gid * (DP / 32) + h));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          }
#pragma unroll
          for (int n = 0; n < 4; ++n) {
            uint32_t b0[3], b1[3];
            split3_bf16x2(v[0][n], v[1][n], b0);
            split3_bf16x2(v[2][n], v[3][n], b1);
#pragma unroll
            for (int x = 2; x >= 0; --x)
#pragma unroll
              for (int y = 0; y <= x; ++y) mma_bf(o[4 * h + n], pf[y][g], b0[x - y], b1[x - y]);
          }
        }
      }
    }
    if (++st == NST) st = 0;
  }
  cp_wait_all();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
    l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
  }

  // ---- the warps' shares joined in shared memory (the rings are free) ----
  __syncthreads();
  float* So = reinterpret_cast<float*>(ring);       // [TNW][16][DP]
  float* Sm = So + TNW * 16 * DP;                   // [TNW][16] maxima, then sums
  float* Sl = Sm + TNW * 16;
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    float* dst = So + (warp * 16 + gid + 8 * r) * DP;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      dst[2 * tq * NT + n] = o[n][2 * r] * vref;
      dst[(2 * tq + 1) * NT + n] = o[n][2 * r + 1] * vref;
    }
    if (tq == 0) {
      Sm[warp * 16 + gid + 8 * r] = m[r];
      Sl[warp * 16 + gid + 8 * r] = l[r];
    }
  }
  __syncthreads();
  constexpr int C4 = DP / 4;
  for (int id = tid; id < 16 * C4; id += 32 * TNW) {
    const int r = id / C4, c = (id % C4) * 4, rr = rt * 16 + r;
    if (rr >= R || c >= a.d) continue;
    float mx = -INFINITY;
#pragma unroll
    for (int w = 0; w < TNW; ++w) mx = fmaxf(mx, Sm[w * 16 + r]);
    const float mu = mx == -INFINITY ? 0.f : mx;
    float sum = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < TNW; ++w) {
      const float f = exp2f(Sm[w * 16 + r] - mu);
      const float4 x = lds4(So + (w * 16 + r) * DP + c);
      sum += Sl[w * 16 + r] * f;
      acc.x = fmaf(x.x, f, acc.x); acc.y = fmaf(x.y, f, acc.y);
      acc.z = fmaf(x.z, f, acc.z); acc.w = fmaf(x.w, f, acc.w);
    }
    const size_t qrow = ((size_t)b * a.Hq + hk * a.g + rr / a.Nq) * a.Nq + rr % a.Nq;
    if (shares == 1) {
      const float w = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      st4((TQ*)a.out + qrow * a.d + c, make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w));
      if (a.lse && c == 0) a.lse[qrow] = sum == 0.f ? -INFINITY : mx + log2f(sum) - X::SHIFT;
    } else {
      const size_t part = (size_t)blockIdx.x * 16 + r;
      st4(t.part_o + part * a.d + c, acc);
      if (c == 0) t.part_ml[part] = make_float2(mx, sum);
    }
  }
}

// out = sum over a row's shares: a block a row, its warps take shares in turn
template <typename TQ>
__global__ void __launch_bounds__(128) k_token_join(TokenArgs t, float shift) {
  __shared__ __align__(16) float So[4][128];
  __shared__ float Sm[4], Sl[4];
  asm volatile("griddepcontrol.wait;" ::: "memory");   // launched while k_token still ran
  const WinArgs& a = t.w;
  const long long qrow = blockIdx.x;                     // (b, query head, query)
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = 4 * lane;
  const int i = (int)(qrow % a.Nq), hq = (int)(qrow / a.Nq % a.Hq), b = (int)(qrow / a.Nq / a.Hq);
  const int rr = (hq % a.g) * a.Nq + i;
  const int2 in = t.info[((size_t)b * a.Hkv + hq / a.g) * t.rtiles + rr / 16];
  if (in.y == 1) return;                                 // written already
  const size_t row0 = (size_t)in.x * 16 + rr % 16;
  float mx = -INFINITY;
  for (int s = lane; s < in.y; s += 32) mx = fmaxf(mx, t.part_ml[row0 + (size_t)s * 16].x);
#pragma unroll
  for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  const float mu = mx == -INFINITY ? 0.f : mx;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = warp; s < in.y; s += 4) {
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
#pragma unroll
  for (int w = 1; w < 4; ++w) {
    const float4 v = lds4(&So[w][c]);
    sum += Sl[w];
    acc.x += v.x; acc.y += v.y; acc.z += v.z; acc.w += v.w;
  }
  const float w = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < a.d)
    st4((TQ*)a.out + qrow * a.d + c, make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w));
  if (a.lse && lane == 0) a.lse[qrow] = sum == 0.f ? -INFINITY : mx + log2f(sum) - shift;
}

namespace {
// blocks of k_token that run at once, by their shared memory (227 KB an SM, 1 KB
// a block for the system)
template <int KIND, int DP>
constexpr int blocks_per_sm() { return (int)(232448 / (token_smem<KIND, DP>() + 1024)); }

int slots_of(int kind, int d) {
  const int sms = 152;   // from the type alone: workspaces do not depend on the device
  switch (kind) {
    case TK_BF16: return sms * (d <= 64 ? blocks_per_sm<TK_BF16, 64>() : blocks_per_sm<TK_BF16, 128>());
    case TK_E4M3: return sms * (d <= 64 ? blocks_per_sm<TK_E4M3, 64>() : blocks_per_sm<TK_E4M3, 128>());
    case TK_E4M3_F32:
      return sms * (d <= 64 ? blocks_per_sm<TK_E4M3_F32, 64>() : blocks_per_sm<TK_E4M3_F32, 128>());
    default: return sms * (d <= 64 ? blocks_per_sm<TK_F32, 64>() : blocks_per_sm<TK_F32, 128>());
  }
}
int kind_of(bool cache, bool bf16) {
  return cache ? (bf16 ? TK_E4M3 : TK_E4M3_F32) : (bf16 ? TK_BF16 : TK_F32);
}

template <int KIND, int DP>
cudaError_t go(TokenArgs& t, cudaStream_t st) {
  using TQ = typename std::conditional<Kind<KIND>::QF32, float, __nv_bfloat16>::type;
  constexpr size_t join = (size_t)TNW * 16 * (DP + 2) * 4;
  constexpr size_t smem = token_smem<KIND, DP>() > join ? token_smem<KIND, DP>() : join;
  static SmemOnce once;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once.allow(k_token<KIND, DP>, smem, dev)) != cudaSuccess) return e;
  e = launch("token_attention", k_token<KIND, DP>, dim3((unsigned)t.grid), dim3(32 * TNW), smem, st, t);
  if (e != cudaSuccess || !t.joined) return e;
  const long long rows = (long long)t.w.B * t.w.Hq * t.w.Nq;
  return launch_after("token_join", k_token_join<TQ>, dim3((unsigned)rows), dim3(128), 0, st, t,
                      Kind<KIND>::SHIFT);
}
}  // namespace

TokenShape token_shape(bool cache, bool bf16, int B, int Hkv, int g, int Nq, int d, long long keys,
                       int left, int right, int sinks) {
  TokenShape s;
  s.rtiles = (g * Nq + 15) / 16;
  s.slots = slots_of(kind_of(cache, bf16), d);
  // groups of a sequence at the most, and so blocks: a share holds at least two
  // groups a warp, shares are at most `slots` beyond one for each row tile
  long long seen = keys;
  if (left < kWinUnbounded && right < kWinUnbounded) {
    const long long w = (long long)left + right + Nq + sinks + 64;
    if (w < seen) seen = w;
  }
  const long long groups = seen / 16 + 3, rows = (long long)B * Hkv * s.rtiles;
  const long long most = (groups + 2 * TNW - 1) / (2 * TNW);
  s.grid = rows * (most < 1 ? 1 : most);
  if (s.grid > rows + s.slots) s.grid = rows + s.slots;
  s.joined = most > 1;
  s.o_bytes = s.joined ? (size_t)s.grid * 16 * d * 4 : 0;
  s.ml_bytes = s.joined ? (size_t)s.grid * 16 * 8 : 0;
  s.info_bytes = (size_t)rows * 8;
  return s;
}

cudaError_t run_token(TokenArgs& t, bool bf16, cudaStream_t st) {
  const bool small = t.w.d <= 64;
  if (t.table) {
    if (bf16) return small ? go<TK_E4M3, 64>(t, st) : go<TK_E4M3, 128>(t, st);
    return small ? go<TK_E4M3_F32, 64>(t, st) : go<TK_E4M3_F32, 128>(t, st);
  }
  if (bf16) return small ? go<TK_BF16, 64>(t, st) : go<TK_BF16, 128>(t, st);
  return small ? go<TK_F32, 64>(t, st) : go<TK_F32, 128>(t, st);
}

}  // namespace lapnys
