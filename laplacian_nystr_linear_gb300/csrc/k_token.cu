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
// and k_token_join adds the shares.  Shares are cut on the device from the
// sequence's own length, so a ragged batch stays even within a sequence.
//
// Products on the warp-level tensor instruction (m16n8k16), rows = (query head
// of the group, query), with the contraction's order chosen so that no operand
// is transposed or gathered: a thread's four k of step s are four neighbouring
// features (scores), and column n of output step nt is feature n DP / 8 + nt
// (P V), so both operands come from shared memory in 16-byte reads without bank
// conflicts (the swizzles below).
//   - 8-bit, bf16 queries: the e4m3 product (m16n8k32) takes the cache's bytes as
//     they are; q and p are the sum of two e4m3 parts each, x = x0 + x1 / 16 with
//     x0 = e4m3(x), x1 = e4m3(16 (x - x0)).  q is scaled per row by a power of two
//     (its 8 bits fit the two parts exactly; features below 2^-14 of the row's
//     largest are off by up to 2^-21 of that), p is kept as 2^8 p (off by 2^-8 of
//     itself like a bf16 rounding, or 2^-22 of the row's largest).  Values are
//     transposed four keys at a time by byte permutes.  Converting the cache to
//     f16 instead costs four instructions per two values: 768 a group of 16 keys
//     in all, 2.8 TB/s.
//   - 8-bit, fp32 queries: e4m3 -> f16 is exact; q (scaled per row) and 2^10 p in
//     two f16 parts (2^-22).
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
  static constexpr bool E4 = KIND == TK_E4M3;       // e4m3 products
  static constexpr bool F16 = KIND == TK_E4M3_F32;  // f16 products
  static constexpr int GK = E4 ? 32 : 16;           // keys of a group
  static constexpr int PARTS = KIND == TK_F32 ? 3 : (E4 || F16 ? 2 : 1);
  static constexpr float SHIFT = E4 ? 8.f : (F16 ? 10.f : 0.f);  // p is held as 2^SHIFT p
  static constexpr int QEXP = E4 ? 7 : 13;  // a row's largest |q| is scaled to [2^QEXP, 2^(QEXP + 1))
  static constexpr int TRAIL = 32;          // bytes behind a ring slot: scales of the keys, of the
                                            // values, and whether there is a block, per 16 keys
};
template <int KIND, int DP>
__host__ __device__ constexpr int ring_stages() { return (KIND == TK_F32 || KIND == TK_E4M3) && DP == 128 ? 3 : 4; }
template <int KIND, int DP>
__host__ __device__ constexpr size_t token_smem() {
  return (size_t)TNW * ring_stages<KIND, DP>() * (2 * Kind<KIND>::GK * DP * Kind<KIND>::ES + Kind<KIND>::TRAIL);
}

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_bf(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_e4(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k32.row.col.f32.e4m3.e4m3.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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
// four values (|x| <= 448) as four e4m3 bytes, and 16 times what those leave as four more
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3) |
         (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3) << 16;
}
__device__ __forceinline__ void split_e4(float a, float b, float c, float d, uint32_t* hi, uint32_t* lo) {
  const uint32_t h = e4m3x4(a, b, c, d);
  const uint32_t w0 = e4m3x2_f16(h), w1 = e4m3x2_f16(h >> 16);
  const float2 x = __half22float2(*reinterpret_cast<const __half2*>(&w0));
  const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w1));
  *hi = h;
  *lo = e4m3x4((a - x.x) * 16.f, (b - x.y) * 16.f, (c - y.x) * 16.f, (d - y.y) * 16.f);
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
  const int sp = blockIdx.x % t.splits;
  const int rt = (blockIdx.x / t.splits) % t.rtiles;
  const int hk = (blockIdx.x / (t.splits * t.rtiles)) % a.Hkv;
  const int b = blockIdx.x / (t.splits * t.rtiles * a.Hkv);
  const int R = a.g * a.Nq;
  WinSeq sq = win_seq(a, b);
  if (!a.q_pos && t.table) sq.qp = sq.len - a.Nq;
  const WinRange kr = win_keys(a, sq, 0, a.Nq);
  // keys [free_lo, free_hi) (or first tokens) are seen by every query: no mask
  const bool rows_ok = sq.qp >= 0 && sq.qp + a.Nq <= sq.len;
  const int free_lo = sq.qp + a.Nq - 1 - a.left, free_hi = rows_ok ? min(sq.len, sq.qp + a.right + 1) : -1;

  // this block's share of the groups: first tokens' groups, then the window's
  const int gs = (kr.S + GK - 1) / GK, w0 = kr.lo / GK;
  const int G = gs + (kr.hi > kr.lo ? (kr.hi + GK - 1) / GK - w0 : 0);
  const int g0 = (int)((long long)G * sp / t.splits), g1 = (int)((long long)G * (sp + 1) / t.splits);

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
      blk[h] = has_keys(j0 + 16 * h, jb, je) ? t.table[(size_t)b * t.max_blocks + (j0 + 16 * h) / t.T] : -1;
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
        tok[h] = bh * t.T + (j0 + 16 * h) % t.T;
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
  uint32_t qf[NP][X::E4 ? DP / 32 : KS][4];
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
    if constexpr (X::F16 || X::E4) {
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      const int ex = (int)(__float_as_uint(mx) >> 23) - 127 - X::QEXP;
      if (mx > 0.f && mx < INFINITY) {
        const int h = max(-126, min(126, -ex));
        down = __uint_as_float((uint32_t)(h + 127) << 23);
        qs[r] *= __uint_as_float((uint32_t)(127 - h) << 23);
      }
    }
    if constexpr (X::E4) {
#pragma unroll
      for (int s = 0; s < KS; ++s)   // step s / 2: its first (a0, a1) or second (a2, a3) four
        split_e4(x[s].x * down, x[s].y * down, x[s].z * down, x[s].w * down,
                 &qf[0][s >> 1][2 * (s & 1) + r], &qf[1][s >> 1][2 * (s & 1) + r]);
    } else {
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
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
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
    if constexpr (NH == 2) {           // (its P is 0: any finite scale will do)
      if (!there[0]) vsc[0] = there[1] ? vsc[1] : 0.f;
      if (!there[1]) vsc[1] = vsc[0];
    } else if (!there[0]) {
      vsc[0] = 0.f;
    }
    // ---- scores ----
    float s[NU][4];
#pragma unroll
    for (int u = 0; u < NU; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
      float s1[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < DP / 4 / PIECE; ++i) {
        const uint4 kv = *reinterpret_cast<const uint4*>(Kt + k_off<RB>(8 * u + gid, tq + 4 * i));
        const uint32_t w[4] = {kv.x, kv.y, kv.z, kv.w};
        if constexpr (KIND == TK_F32) {
          uint32_t p0[3], p1[3];
          split3_bf16x2(__uint_as_float(w[0]), __uint_as_float(w[1]), p0);
          split3_bf16x2(__uint_as_float(w[2]), __uint_as_float(w[3]), p1);
#pragma unroll
          for (int x = 2; x >= 0; --x)
#pragma unroll
            for (int y = 0; y <= x; ++y) mma_bf(s[u], qf[y][i], p0[x - y], p1[x - y]);
        } else if constexpr (KIND == TK_BF16) {
          mma_bf(s[u], qf[0][2 * i], w[0], w[1]);
          mma_bf(s[u], qf[0][2 * i + 1], w[2], w[3]);
        } else if constexpr (X::E4) {
#pragma unroll
          for (int x = 0; x < 2; ++x) {
            mma_e4(s[u], qf[0][2 * i + x], w[2 * x], w[2 * x + 1]);
            mma_e4(s1, qf[1][2 * i + x], w[2 * x], w[2 * x + 1]);
          }
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t b0 = e4m3x2_f16(w[x]), b1 = e4m3x2_f16(w[x] >> 16);
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) mma_f16(s[u], qf[p][4 * i + x], b0, b1);
          }
        }
      }
      if constexpr (X::E4) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[u][e] = fmaf(s1[e], 0.0625f, s[u][e]);
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
    if constexpr (X::E4) {
      // the k of a thread: keys 2 tq, 2 tq + 1 of the group's four runs of 8
      uint32_t pf[2][4];
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int r = 0; r < 2; ++r)
          split_e4(p[2 * h][2 * r], p[2 * h][2 * r + 1], p[2 * h + 1][2 * r], p[2 * h + 1][2 * r + 1],
                   &pf[0][2 * h + r], &pf[1][2 * h + r]);
      // halves of unlike scale (blocks of 16 tokens) go one after the other
      const bool apart = vsc[0] != vsc[1];
#pragma unroll 1
      for (int pass = 0; pass <= (int)apart; ++pass) {
        uint32_t pa[2][4];
#pragma unroll
        for (int x = 0; x < 2; ++x)
#pragma unroll
          for (int e = 0; e < 4; ++e) pa[x][e] = apart && (e >> 1) != pass ? 0u : pf[x][e];
        const float vs = pass ? vsc[1] : vsc[0], vs1 = vs * 0.0625f;
        constexpr int W = DP / 8 / 4;  // 32-bit words of a thread's piece of a value row
        uint32_t v[8][W];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int rr = 8 * (e >> 1) + 2 * tq + (e & 1);
          if constexpr (W == 4) {
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + v_off<RB>(rr, gid));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(Vt + v_off<RB>(rr, gid >> 1) + 8 * (gid & 1));
            v[e][0] = x.x; v[e][1] = x.y;
          }
        }
#pragma unroll
        for (int w = 0; w < W; ++w) {
          uint32_t bt[2][4];           // four keys of each of the word's four columns
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t x0 = __byte_perm(v[4 * h][w], v[4 * h + 1][w], 0x5140);
            const uint32_t x1 = __byte_perm(v[4 * h + 2][w], v[4 * h + 3][w], 0x5140);
            const uint32_t y0 = __byte_perm(v[4 * h][w], v[4 * h + 1][w], 0x7362);
            const uint32_t y1 = __byte_perm(v[4 * h + 2][w], v[4 * h + 3][w], 0x7362);
            bt[h][0] = __byte_perm(x0, x1, 0x5410);
            bt[h][1] = __byte_perm(x0, x1, 0x7632);
            bt[h][2] = __byte_perm(y0, y1, 0x5410);
            bt[h][3] = __byte_perm(y0, y1, 0x7632);
          }
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            float c0[4] = {0.f, 0.f, 0.f, 0.f}, c1[4] = {0.f, 0.f, 0.f, 0.f};
            mma_e4(c0, pa[0], bt[0][x], bt[1][x]);
            mma_e4(c1, pa[1], bt[0][x], bt[1][x]);
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[4 * w + x][e] = fmaf(c0[e], vs, fmaf(c1[e], vs1, o[4 * w + x][e]));
          }
        }
      }
    } else {
      uint32_t pf[NP][4];
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          uint32_t w[NP];
          split<KIND>(p[u][2 * r], p[u][2 * r + 1], w);
#pragma unroll
          for (int x = 0; x < NP; ++x) pf[x][2 * u + r] = w[x];
        }
      if constexpr (KIND == TK_E4M3_F32) {
        constexpr int W = DP / 8 / 4;
        uint32_t v[4][W];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int rr = 2 * tq + (e & 1) + 8 * (e >> 1);
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
          float c[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int x = NP - 1; x >= 0; --x) mma_f16(c, pf[x], b0, b1);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] = fmaf(c[e], vsc[0], o[n][e]);
        }
      } else if constexpr (KIND == TK_BF16) {
        constexpr int W = DP / 16;
#pragma unroll
        for (int h = 0; h < W / 4; ++h) {
          uint32_t v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 2 * tq + (e & 1) + 8 * (e >> 1);
            const uint4 x = *reinterpret_cast<const uint4*>(Vt + v_off<RB>(rr, gid * (W / 4) + h));
            v[e][0] = x.x; v[e][1] = x.y; v[e][2] = x.z; v[e][3] = x.w;
          }
#pragma unroll
          for (int n = 0; n < 8; ++n) {
            const int sel = n & 1 ? 0x7632 : 0x5410;
            mma_bf(o[8 * h + n], pf[0], __byte_perm(v[0][n >> 1], v[1][n >> 1], sel),
                   __byte_perm(v[2][n >> 1], v[3][n >> 1], sel));
          }
        }
      } else {
#pragma unroll
        for (int h = 0; h < DP / 32; ++h) {
          float v[4][4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int rr = 2 * tq + (e & 1) + 8 * (e >> 1);
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
              for (int y = 0; y <= x; ++y) mma_bf(o[4 * h + n], pf[y], b0[x - y], b1[x - y]);
          }
        }
      }
    }
    if (++st == NST) st = 0;
  }
  cp_wait_all();
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
      dst[2 * tq * NT + n] = o[n][2 * r];
      dst[(2 * tq + 1) * NT + n] = o[n][2 * r + 1];
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
    if (t.splits == 1) {
      const float w = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
      st4((TQ*)a.out + qrow * a.d + c, make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w));
      if (a.lse && c == 0) a.lse[qrow] = sum == 0.f ? -INFINITY : mx + log2f(sum) - X::SHIFT;
    } else {
      const size_t part = qrow * t.splits + sp;
      st4(t.part_o + part * a.d + c, acc);
      if (c == 0) t.part_ml[part] = make_float2(mx, sum);
    }
  }
}

// out = sum over a row's shares, one warp a row
template <typename TQ>
__global__ void __launch_bounds__(128) k_token_join(TokenArgs t, float shift) {
  const WinArgs& a = t.w;
  const long long rows = (long long)a.B * a.Hq * a.Nq;
  const long long r = (long long)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (r >= rows) return;
  const float2* ml = t.part_ml + r * t.splits;
  float mx = -INFINITY;
  for (int s = lane; s < t.splits; s += 32) mx = fmaxf(mx, ml[s].x);
#pragma unroll
  for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  const float mu = mx == -INFINITY ? 0.f : mx;
  const int c = 4 * lane;
  float sum = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
  for (int s = 0; s < t.splits; ++s) {
    const float2 x = ml[s];
    const float f = exp2f(x.x - mu);
    sum = fmaf(x.y, f, sum);
    if (c < a.d) {
      const float4 v = ld4(t.part_o + (r * t.splits + s) * a.d + c);
      acc.x = fmaf(v.x, f, acc.x); acc.y = fmaf(v.y, f, acc.y);
      acc.z = fmaf(v.z, f, acc.z); acc.w = fmaf(v.w, f, acc.w);
    }
  }
  const float w = sum > 0.f ? 1.f / sum : (sum == 0.f ? 0.f : sum);
  if (c < a.d)
    st4((TQ*)a.out + r * a.d + c, make_float4(acc.x * w, acc.y * w, acc.z * w, acc.w * w));
  if (a.lse && lane == 0) a.lse[r] = sum == 0.f ? -INFINITY : mx + log2f(sum) - shift;
}

namespace {
// the shares of a row tile's keys: about three blocks for each that fits at once
// (so that short and long sequences of a batch even out), each share at least
// two groups a warp.  From the dimensions alone.
int shares(int blocks, long long keys) {
  const long long most = (keys / 16 + 2 * TNW - 1) / (2 * TNW);
  long long s = (152 * 6 + blocks - 1) / blocks;
  s = s > most ? most : s;
  return (int)(s < 1 ? 1 : (s > 256 ? 256 : s));
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
  const long long n = (long long)t.w.B * t.w.Hkv * t.rtiles * t.splits;
  e = launch("token_attention", k_token<KIND, DP>, dim3((unsigned)n), dim3(32 * TNW), smem, st, t);
  if (e != cudaSuccess || t.splits == 1) return e;
  const long long rows = (long long)t.w.B * t.w.Hq * t.w.Nq;
  return launch("token_join", k_token_join<TQ>, dim3((unsigned)((rows + 3) / 4)), dim3(128), 0, st, t,
                Kind<KIND>::SHIFT);
}
}  // namespace

TokenShape token_shape(int B, int Hkv, int g, int Nq, int d, long long keys, int left, int right,
                       int sinks) {
  TokenShape s;
  s.rtiles = (g * Nq + 15) / 16;
  long long seen = keys;
  if (left < kWinUnbounded && right < kWinUnbounded) {
    const long long w = (long long)left + right + Nq + sinks + 64;
    if (w < seen) seen = w;
  }
  const long long blocks = (long long)B * Hkv * s.rtiles;
  s.splits = shares((int)(blocks < 1 << 20 ? blocks : 1 << 20), seen);
  const size_t rows = (size_t)B * Hkv * g * Nq;
  s.o_bytes = s.splits == 1 ? 0 : rows * s.splits * d * 4;
  s.ml_bytes = s.splits == 1 ? 0 : rows * s.splits * 8;
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
