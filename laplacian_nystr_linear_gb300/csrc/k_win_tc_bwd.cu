// Windowed softmax attention, backward, bf16, on the tcgen05 tensor cores
// (visibility rule: win.cuh; operand tiles: win_tc.cuh; formulas: k_win.cu).
//
// Two kernels, so that every sum has one owner and one order (deterministic, no
// atomics): scores are computed in both, 7 products of 128 x 128 x d per tile of
// pairs instead of 5.
//   k_win_dq_tc   128 queries stay, keys in steps of 128:
//                 S = Q K^T, dP = dO V^T, dS = P (dP - D) as two bf16, dQ += dS K
//   k_win_dkv_tc  128 keys stay, the queries of the group's heads in steps of
//                 128: S^T = K Q^T, dP^T = V dO^T, dV += P^T dO, dK += dS^T Q
// with P = exp2(scale log2(e) s - lse) from the forward's log-sum.  The bf16
// tile that was just computed is the left operand of its product, from tensor
// memory, over the columns it came from; K, Q, dO tiles are read as they lie in
// shared memory both K-major (scores) and MN-major (gradients).
//
//   warps 0-15  elementwise work, one row and a quarter of the columns per thread.
//               Each group of columns writes its bf16 values (16 or 32 columns) over its
//               own 32 columns, so the groups need no barrier and drift apart: one's
//               exponentials run under the others' multiplications, and four warps
//               a scheduler hide the latencies of tensor memory (two of half the
//               columns each: 3700 cycles a step of dkv, the products take 1024);
//   warp 16     TMA (the resident tiles, and two rings);
//   warp 17 (dq: and 18)  one thread issues the products, the bf16 tile's product
//               always before the one that overwrites it, so that their order needs
//               no barrier:
//                 dq:   dQ(j) S(j+2) (S in two buffers)  |  dP(j+1), once dP(j) is
//                       in registers
//                 dkv:  dV(j) S(j+1) dK(j) dP(j+1)
//               (dkv of 2 x 16 heads of 64, 16384 tokens: 450 us; with two threads
//               537; with dS beside P, S in two buffers and dP freed early as in dq
//               478, with two threads 519.  Two blocks an SM with steps of 64: 558,
//               and 393 for dq's 366);
//   warp 18     dkv: log-sum and D of a step's queries into shared memory.
//
// Key tiles with first tokens are seen by all later queries: their queries are
// cut into chunks, one item each, with fp32 partials that k_win_join adds; so are all
// tiles' where there are few with many queries each (wide windows).
// Rows behind a sequence's end are zeroed in shared memory where they are
// summed over (0 * NaN).  Every wait is bounded.
//
// Bound: 16 d flops per visible pair (with dS in two parts) on the tensor pipe, or the
// elementwise warps.  Measured: 16384 tokens, 2 x 16 heads of 64, window 1024: dq 366,
// dkv 450, join 13 us; issue slots 59 % and tensor pipe 41 % busy in dq: the chain of a
// step (scores, exponentials, dS, products) and what stands between items of 9 steps (D,
// the outputs).  8192 tokens, 16 heads of 128 on 4, window 2048: 185, 220 and
// 6 us (0.73 PFLOP/s of the 10 d flops a pair that are needed).
#include <cstring>

#include "internal.h"
#include "win_tc.cuh"

namespace lapnys {

namespace {
using namespace wtc;
constexpr int BT = 128;                 // rows and columns of a tile
constexpr int BEW = 512;                // elementwise threads
constexpr int BTH = BEW + 128;
constexpr int WI = BEW / 32;            // first of the warps that copy and issue
constexpr uint32_t PANEL = BT * 128;
constexpr int NRING1 = 3, NRING2 = 2;   // tiles of the rings (K, V; Q, dO)
template <int NP>
struct BwdShape {
  static constexpr uint32_t TILE = NP * PANEL;
  static constexpr uint32_t SMEM = (2 + NRING1 + NRING2) * TILE + 1024;
};
struct BwdMaps {
  CUtensorMap q, k, v, dout;              // boxes of 64 x 128
  CUtensorMap q16, k16, v16, dout16;      // boxes of 64 x 16 for narrow steps
};
struct BwdGeom {
  int tiles;                              // query tiles (dq); key items of a head (dkv)
  int items;
  int* err;
};

// a tile of w rows (a multiple of 16) from row r0 of head bh
template <int NP>
__device__ __forceinline__ void load_rows(uint32_t dst, const CUtensorMap* wide,
                                          const CUtensorMap* narrow, int r0, int w, int bh,
                                          uint32_t bar) {
#pragma unroll 1
  for (int p = 0; p < NP; ++p) {
    if (w == BT) {
      tma3(dst + p * PANEL, wide, 64 * p, r0, bh, bar);
    } else {
#pragma unroll 1
      for (int r = 0; r < w; r += 16) tma3(dst + p * PANEL + r * 128, narrow, 64 * p, r0 + r, bh, bar);
    }
  }
}
struct Step {
  int r0, re, w;        // rows [r0, re) and the width of the products
};

// dS = P (dP - D) of 32 columns to tensor memory, as 16 columns of bf16 pairs and
// 16 of what their rounding leaves (dS sums to 0 over a row, so what the keys have
// in common cancels in dS K, but not in the roundings: with one bf16 dS, dQ is off
// by 2.9e-3 of its norm for keys of a common part half their spread, with two by
// 1.8e-3, of which the output's rounding is 1.7e-3).  Not whole: only where `bits`
// are set (a select, not a product: what is not seen may be anything).
__device__ __forceinline__ void ds_store(uint32_t dst, const uint32_t (&p)[32],
                                         const uint32_t (&dp)[32], f32x2 minus_D, bool whole,
                                         uint32_t bits) {
  float x[32];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    const float2 y = unpack2(mul2(pack2(__uint_as_float(p[e]), __uint_as_float(p[e + 1])),
                                  add2(pack2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])), minus_D)));
    x[e] = y.x;
    x[e + 1] = y.y;
  }
  if (!whole) {
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1u ? x[e] : 0.f;
  }
  uint32_t o[32];
#pragma unroll
  for (int e = 0; e < 32; e += 2) {
    o[e >> 1] = pack(x[e], x[e + 1]);
    o[16 + (e >> 1)] = pack_rest(x[e], x[e + 1], o[e >> 1]);
  }
  st32(dst, o);
}
}  // namespace

// ---------------------------------------------------------------------------
// dQ
// ---------------------------------------------------------------------------
namespace {
struct DqItem {
  int b, h, i0, i1;
  WinSeq sq;
  WinRange kr;
  int ns, steps;
};
__device__ __forceinline__ DqItem dq_item(const WinArgs& a, const BwdGeom& gm, int it) {
  DqItem r;
  const int heads = a.B * a.Hq;
  const int tile = gm.tiles - 1 - it / heads, h = it % heads;
  r.b = h / a.Hq;
  r.h = h % a.Hq;
  r.i0 = tile * BT;
  r.i1 = min(a.Nq, r.i0 + BT);
  r.sq = win_seq(a, r.b);
  r.kr = win_keys(a, r.sq, r.i0, r.i1);
  r.ns = (r.kr.S + BT - 1) / BT;
  r.steps = r.ns + (r.kr.hi - r.kr.lo + BT - 1) / BT;
  return r;
}
__device__ __forceinline__ Step dq_step(const DqItem& r, int j) {
  Step s;
  const bool first = j < r.ns;
  s.r0 = first ? j * BT : r.kr.lo + (j - r.ns) * BT;
  s.re = min(first ? r.kr.S : r.kr.hi, s.r0 + BT);
  s.w = (s.re - s.r0 + 15) & ~15;
  return s;
}
}  // namespace

template <int NP>
__global__ void __launch_bounds__(BTH, 1) k_win_dq_tc(const __grid_constant__ BwdMaps mp,
                                                      const WinArgs a, const BwdGeom gm) {
  using SH = BwdShape<NP>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t kfull[NRING1], kempty[NRING1], vfull[NRING2], vempty[NRING2];
  __shared__ __align__(8) uint64_t qfull, qempty;       // Q and dO landed; their products done
  __shared__ __align__(8) uint64_t sfull[2], dpfull, dpempty, ofull, oempty, drain[2];
  __shared__ __align__(8) uint64_t dsfull[2];           // (by parity: a step can run ahead)
  __shared__ __align__(8) uint64_t dhfull;              // D written
  __shared__ uint32_t tmem_s;
  __shared__ float Ds[BT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = tc::smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t Qb = base, Ob = Qb + SH::TILE, Kr = Ob + SH::TILE, Vr = Kr + NRING1 * SH::TILE;
  auto bar = [](uint64_t* b) { return tc::smem_u32(b); };
  if (warp == WI) tc::tmem_alloc(&tmem_s, 512);
  if (tid == 0) {
    for (int i = 0; i < NRING1; ++i) {
      tc::mbar_init(bar(&kfull[i]), 1);
      tc::mbar_init(bar(&kempty[i]), 1);
    }
    for (int i = 0; i < NRING2; ++i) {
      tc::mbar_init(bar(&vfull[i]), 1);
      tc::mbar_init(bar(&vempty[i]), 1);
    }
    tc::mbar_init(bar(&qfull), 1);
    tc::mbar_init(bar(&qempty), 2);
    tc::mbar_init(bar(&sfull[0]), 1);
    tc::mbar_init(bar(&sfull[1]), 1);
    tc::mbar_init(bar(&dhfull), WI);
    tc::mbar_init(bar(&dpfull), 1);
    tc::mbar_init(bar(&dpempty), WI);
    tc::mbar_init(bar(&dsfull[0]), WI);
    tc::mbar_init(bar(&dsfull[1]), WI);
    tc::mbar_init(bar(&ofull), 1);
    tc::mbar_init(bar(&oempty), WI);
    tc::mbar_init(bar(&drain[0]), 1);
    tc::mbar_init(bar(&drain[1]), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;
  // tensor memory: S (then dS) in two buffers, dP, dQ
  const uint32_t tS = tmem, tP = tmem + 2 * BT, tO = tmem + 3 * BT;

  if (warp >= WI) {
    if (warp == WI && elect_one()) {
      // ---------------- TMA ----------------
      int n = 0, nq = 0;
      bool bad = false;
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DqItem r = dq_item(a, gm, it);
        if (r.steps == 0) continue;
        if (!wait_or_flag(gm.err, bar(&qempty), (nq & 1) ^ 1u)) break;
        tc::mbar_expect_tx(bar(&qfull), 2 * SH::TILE);
        const int bq = r.b * a.Hq + r.h, bk = r.b * a.Hkv + r.h / a.g;
        load_rows<NP>(Qb, &mp.q, nullptr, r.i0, BT, bq, bar(&qfull));
        load_rows<NP>(Ob, &mp.dout, nullptr, r.i0, BT, bq, bar(&qfull));
        ++nq;
#pragma unroll 1
        for (int j = 0; j < r.steps; ++j, ++n) {
          const Step s = dq_step(r, j);
          const int sk = n % NRING1, sv = n % NRING2;
          if (!wait_or_flag(gm.err, bar(&kempty[sk]), ((n / NRING1) & 1) ^ 1u) ||
              !wait_or_flag(gm.err, bar(&vempty[sv]), ((n / NRING2) & 1) ^ 1u)) {
            bad = true;
            break;
          }
          tc::mbar_expect_tx(bar(&kfull[sk]), (uint32_t)(NP * s.w * 128));
          load_rows<NP>(Kr + sk * SH::TILE, &mp.k, &mp.k16, s.r0, s.w, bk, bar(&kfull[sk]));
          tc::mbar_expect_tx(bar(&vfull[sv]), (uint32_t)(NP * s.w * 128));
          load_rows<NP>(Vr + sv * SH::TILE, &mp.v, &mp.v16, s.r0, s.w, bk, bar(&vfull[sv]));
        }
      }
      // every copy has landed before the block ends, also after an expired wait
#pragma unroll 1
      for (int i = n > NRING1 ? n - NRING1 : 0; i < n; ++i) {
        wait_or_flag(gm.err, bar(&kfull[i % NRING1]), (uint32_t)(i / NRING1) & 1u);
        if (i >= n - NRING2) wait_or_flag(gm.err, bar(&vfull[i % NRING2]), (uint32_t)(i / NRING2) & 1u);
      }
      if (nq) wait_or_flag(gm.err, bar(&qfull), (uint32_t)(nq - 1) & 1u);
    } else if (warp == WI + 1 && elect_one()) {
      // ---------------- scores and dQ ----------------
      int n = 0, nq = 0, no = 0;        // steps, items
      bool bad = false;
      const int ksteps = a.d / 16;
      const uint32_t id = idesc(BT, BT, false), id_q = idesc(BT, a.d, true);
      auto commit = [&](uint64_t* b) { tc::commit(bar(b)); };
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DqItem r = dq_item(a, gm, it);
        if (r.steps == 0) continue;
        if (!wait_or_flag(gm.err, bar(&qfull), (uint32_t)nq++ & 1u)) { bad = true; break; }
        const int n0 = n;
        n += r.steps;
        auto scores = [&](const Step& s, int i) {
          const int sk = i % NRING1;
          const uint32_t K = Kr + sk * SH::TILE;
          if (!wait_or_flag(gm.err, bar(&kfull[sk]), (uint32_t)(i / NRING1) & 1u)) return false;
          if (s.r0 + s.w > r.sq.len && r.sq.len < a.Nk) zero_rows<NP>(K, r.sq.len - s.r0, s.w);
          tc::fence_after();
          mma_features<NP>(tS + (i & 1) * BT, Qb, K, ksteps, s.w == BT ? id : idesc(BT, s.w, false));
          commit(&sfull[i & 1]);
          if (i + 1 == n) commit(&qempty);
          return true;
        };
        Step s = dq_step(r, 0), s1 = dq_step(r, min(1, r.steps - 1));
        if (!scores(s, n0) || (r.steps > 1 && !scores(s1, n0 + 1))) { bad = true; break; }
#pragma unroll 1
        for (int i = n0; i < n; ++i) {
          const int sk = i % NRING1;
          const Step s2 = dq_step(r, min(i - n0 + 2, r.steps - 1));
          if (!wait_or_flag(gm.err, bar(&dsfull[i & 1]), (uint32_t)(i >> 1) & 1u) ||
              (i == n0 && !wait_or_flag(gm.err, bar(&oempty), ((uint32_t)no++ & 1u) ^ 1u))) {
            bad = true;
            break;
          }
          tc::fence_after();
          mma_rows<BT, 32>(tO, tS + (i & 1) * BT, Kr + sk * SH::TILE, s.w / 16, id_q, i > n0);
          mma_rows<BT, 32>(tO, tS + (i & 1) * BT + 16, Kr + sk * SH::TILE, s.w / 16, id_q, true);
          commit(&kempty[sk]);
          if (i + 1 == n) commit(&ofull);
          if (i + 2 < n && !scores(s2, i + 2)) { bad = true; break; }
          s = s1;
          s1 = s2;
        }
      }
      if (bad) {  // what was issued ends before tensor memory is freed
        commit(&drain[0]);
        wait_or_flag(gm.err, bar(&drain[0]), 0);
      }
    } else if (warp == WI + 2 && elect_one()) {
      // ---------------- dP ----------------
      int n = 0, nq = 0;                // steps, items
      bool bad = false;
      const int ksteps = a.d / 16;
      const uint32_t id = idesc(BT, BT, false);
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DqItem r = dq_item(a, gm, it);
        if (r.steps == 0) continue;
        if (!wait_or_flag(gm.err, bar(&qfull), (uint32_t)nq++ & 1u)) { bad = true; break; }
#pragma unroll 1
        for (int j = 0; j < r.steps; ++j, ++n) {
          const int sv = n % NRING2, w = dq_step(r, j).w;
          // (the step before is in registers)
          if (!wait_or_flag(gm.err, bar(&vfull[sv]), (uint32_t)(n / NRING2) & 1u) ||
              !wait_or_flag(gm.err, bar(&dpempty), ((uint32_t)n & 1u) ^ 1u)) {
            bad = true;
            break;
          }
          tc::fence_after();
          mma_features<NP>(tP, Ob, Vr + sv * SH::TILE, ksteps, w == BT ? id : idesc(BT, w, false));
          tc::commit(bar(&dpfull));
          tc::commit(bar(&vempty[sv]));
          if (j + 1 == r.steps) tc::commit(bar(&qempty));
        }
      }
      if (bad) {
        tc::commit(bar(&drain[1]));
        wait_or_flag(gm.err, bar(&drain[1]), 0);
      }
    }
  } else {
    // ---------------- elementwise ----------------
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane, c0 = 32 * grp;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const float c = a.scale_log2;
    int n = 0, no = 0, nd = 0;
    bool bad = false;
    for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
      const DqItem r = dq_item(a, gm, it);
      const int i = r.i0 + row;
      const size_t qrow = ((size_t)r.b * a.Hq + r.h) * a.Nq + i;
      const WinRow wr = win_row(a, r.sq, i);
      // D = dout.(out + rest): 8 rows of a warp, 8 lanes a row
      float D = 0.f, lse = 0.f;
      if (r.steps > 0) {
        if (i < r.i1) lse = a.lse[qrow];
        const int row8 = 8 * warp + (lane >> 3);
        const size_t at = (((size_t)r.b * a.Hq + r.h) * a.Nq + r.i0 + row8) * a.d + 8 * (lane & 7);
        uint4 x[2 * NP], y[2 * NP], z[2 * NP];
#pragma unroll
        for (int e = 0; e < 2 * NP; ++e) {
          const int t = 4 * (e & 1), f = 64 * (e >> 1);      // rows and features further on
          x[e] = y[e] = z[e] = make_uint4(0, 0, 0, 0);
          if (r.i0 + row8 + t < r.i1 && f + 8 * (lane & 7) < a.d) {
            const size_t p = at + (size_t)t * a.d + f;
            x[e] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.dout + p));
            y[e] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.out + p));
            if (a.rest) z[e] = __ldg(reinterpret_cast<const uint4*>((const __nv_bfloat16*)a.rest + p));
          }
        }
        const auto dot = [](uint4 u, uint4 w, float sum) {
          const uint32_t us[4] = {u.x, u.y, u.z, u.w}, ws[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            sum = fmaf(__uint_as_float(us[c] << 16), __uint_as_float(ws[c] << 16), sum);
            sum = fmaf(__uint_as_float(us[c] & 0xffff0000u), __uint_as_float(ws[c] & 0xffff0000u), sum);
          }
          return sum;
        };
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          float sum = 0.f, rest = 0.f;
#pragma unroll
          for (int e = t; e < 2 * NP; e += 2) {
            sum = dot(x[e], y[e], sum);
            rest = dot(x[e], z[e], rest);
          }
          sum += rest;
#pragma unroll
          for (int o = 4; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
          // (written again for the next item only behind `ofull`, for which all have
          // worked through this one's steps)
          if ((lane & 7) == 0) Ds[row8 + 4 * t] = sum;
        }
        arrive_warp(bar(&dhfull));
        if (!wait_warp(gm.err, bar(&dhfull), (uint32_t)nd++ & 1u)) break;
        D = Ds[row];
        if (grp == 0 && i < r.i1) a.D[qrow] = D;
      }

      const int p0 = r.sq.qp + r.i0, p1 = r.sq.qp + r.i1 - 1;
      const bool rows_ok = r.i1 - r.i0 == BT && p0 >= 0 && p1 < r.sq.len;
      const int free_lo = p1 - a.left, free_hi = min(p0 + a.right, r.sq.len - 1);
      const f32x2 c2 = pack2(c, c), o2 = pack2(-lse, -lse), D2 = pack2(-D, -D);
#pragma unroll 1
      for (int j = 0; j < r.steps; ++j, ++n) {
        const Step s = dq_step(r, j);
        const uint32_t S = tS + (n & 1) * BT + lanes + c0, P = tP + lanes + c0;
        if (!wait_warp(gm.err, bar(&sfull[n & 1]), (uint32_t)(n >> 1) & 1u)) { bad = true; break; }
        tc::fence_after();
        uint32_t v[32];
        ld32(S, v);
        ld_wait(v);
#pragma unroll
        for (int e = 0; e < 32; e += 2) {
          const float2 x = unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2, o2));
          v[e] = __float_as_uint(exp2_ftz(x.x));
          v[e + 1] = __float_as_uint(exp2_ftz(x.y));
        }
        if (!wait_warp(gm.err, bar(&dpfull), (uint32_t)n & 1u)) { bad = true; break; }
        tc::fence_after();
        uint32_t dp[32];
        ld32(P, dp);
        const bool whole = rows_ok && s.re - s.r0 == BT && s.r0 + BT - 1 <= free_hi &&
                           (s.r0 >= free_lo || s.re <= a.sinks);
        const int h = min(wr.hi, s.re) - s.r0 - c0, l = wr.lo - s.r0 - c0, z = wr.S - s.r0 - c0;
        ld_wait(dp);
        tc::fence_before();
        arrive_warp(bar(&dpempty));
        ds_store(S, v, dp, D2, whole, whole ? 0u : seen_bits(l, h, z));
        st_wait();
        tc::fence_before();
        arrive_warp(bar(&dsfull[n & 1]));
      }
      if (bad) break;
      if (r.steps > 0) {
        if (!wait_warp(gm.err, bar(&ofull), (uint32_t)no & 1u)) break;
        ++no;
        tc::fence_after();
      }
      // pieces of 32 columns, shared by the groups
      __nv_bfloat16* dst = (__nv_bfloat16*)a.dq + (((size_t)r.b * a.Hq + r.h) * a.Nq + r.i0) * a.d;
#pragma unroll 1
      for (int q = 32 * grp; q < a.d; q += 128) {
        uint32_t o[32];
        if (r.steps > 0) {
          ld32(tO + lanes + q, o);
          ld_wait(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        store_bf16(dst + q, nullptr, a.d, 32 * (warp & 3), r.i1 - r.i0, (a.d - q) / 8, o, a.scale);
      }
      if (r.steps > 0) {
        tc::fence_before();
        arrive_warp(bar(&oempty));
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == WI) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------------------
// dK, dV
// ---------------------------------------------------------------------------
namespace {
struct DkvItem {
  int b, hk, tile, chunk;       // chunk < 0: an ordinary tile
  int j0, j1;                   // keys of the tile, of the sequence
  int i0, i1;                   // queries
  int per, steps;               // steps of one head, of all
  WinSeq sq;
};
__device__ __forceinline__ DkvItem dkv_item(const WinArgs& a, const BwdGeom& gm, int it) {
  DkvItem r;
  const int heads = a.B * a.Hkv;
  const int t = it / heads, h = it % heads;
  r.b = h / a.Hkv;
  r.hk = h % a.Hkv;
  const int nf = a.stiles * a.chunks;
  r.chunk = t < nf ? t % a.chunks : -1;
  r.tile = t < nf ? t / a.chunks : t - nf + a.stiles;
  r.sq = win_seq(a, r.b);
  r.j0 = r.tile * BT;
  r.j1 = min(min(a.Nk, r.j0 + BT), r.sq.len);
  win_queries(a, r.sq, r.j0, r.j1, &r.i0, &r.i1);
  if (r.chunk >= 0) {
    r.i0 = max(r.i0, r.chunk * a.chunk_rows);
    r.i1 = min(r.i1, (r.chunk + 1) * a.chunk_rows);
  }
  r.per = r.i1 > r.i0 ? (r.i1 - r.i0 + BT - 1) / BT : 0;
  r.steps = r.per * a.g;
  return r;
}
// the steps of an item in their order: rows of query head hk g + e
struct StepWalk {
  int e, r0;
  __device__ __forceinline__ Step step(const DkvItem& r) const {
    Step s;
    s.r0 = r0;
    s.re = min(r.i1, r0 + BT);
    s.w = (s.re - r0 + 15) & ~15;
    return s;
  }
  __device__ __forceinline__ void next(const DkvItem& r) {
    r0 += BT;
    if (r0 >= r.i1) {
      r0 = r.i0;
      ++e;
    }
  }
};
__device__ __forceinline__ StepWalk dkv_walk(const DkvItem& r) { return StepWalk{0, r.i0}; }
}  // namespace

template <int NP>
__global__ void __launch_bounds__(BTH, 1) k_win_dkv_tc(const __grid_constant__ BwdMaps mp,
                                                       const WinArgs a, const BwdGeom gm) {
  using SH = BwdShape<NP>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t qfull[NRING1], qempty[NRING1], ofull[NRING2], oempty[NRING2];
  __shared__ __align__(8) uint64_t lfull[2], lempty[2];   // log-sums of a step
  __shared__ __align__(8) uint64_t dfull, dempty;         // D of a step
  __shared__ __align__(8) uint64_t kvfull, kvempty;       // K and V landed; their products done
  __shared__ __align__(8) uint64_t sfull, pfull, dpfull, dsfull, gfull, gempty, drain;
  __shared__ uint32_t tmem_s;
  __shared__ __align__(16) float Ls[2][BT], Ds[BT];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = tc::smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t Kb = base, Vb = Kb + SH::TILE, Qr = Vb + SH::TILE, Or = Qr + NRING1 * SH::TILE;
  auto bar = [](uint64_t* b) { return tc::smem_u32(b); };
  if (warp == WI) tc::tmem_alloc(&tmem_s, 512);
  if (tid == 0) {
    for (int i = 0; i < NRING1; ++i) {
      tc::mbar_init(bar(&qfull[i]), 1);
      tc::mbar_init(bar(&qempty[i]), 1);
    }
    for (int i = 0; i < NRING2; ++i) {
      tc::mbar_init(bar(&ofull[i]), 1);
      tc::mbar_init(bar(&oempty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(bar(&lfull[i]), 32);
      tc::mbar_init(bar(&lempty[i]), BEW);
    }
    tc::mbar_init(bar(&dfull), 32);
    tc::mbar_init(bar(&dempty), BEW);
    tc::mbar_init(bar(&kvfull), 1);
    tc::mbar_init(bar(&kvempty), 1);
    tc::mbar_init(bar(&sfull), 1);
    tc::mbar_init(bar(&pfull), BEW);
    tc::mbar_init(bar(&dpfull), 1);
    tc::mbar_init(bar(&dsfull), BEW);
    tc::mbar_init(bar(&gfull), 1);
    tc::mbar_init(bar(&gempty), BEW);
    tc::mbar_init(bar(&drain), 1);
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;
  // tensor memory: S^T (then P^T), dP^T (then dS^T), dV, dK
  const uint32_t tS = tmem, tP = tmem + BT, tV = tmem + 2 * BT, tK = tmem + 3 * BT;

  if (warp >= WI) {
    if (warp == WI && elect_one()) {
      // ---------------- TMA ----------------
      int n = 0, nk = 0;
      bool bad = false;
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DkvItem r = dkv_item(a, gm, it);
        if (r.steps == 0) continue;
        if (!wait_or_flag(gm.err, bar(&kvempty), (nk & 1) ^ 1u)) break;
        tc::mbar_expect_tx(bar(&kvfull), 2 * SH::TILE);
        const int bk = r.b * a.Hkv + r.hk;
        load_rows<NP>(Kb, &mp.k, nullptr, r.j0, BT, bk, bar(&kvfull));
        load_rows<NP>(Vb, &mp.v, nullptr, r.j0, BT, bk, bar(&kvfull));
        ++nk;
        StepWalk wk = dkv_walk(r);
#pragma unroll 1
        for (int j = 0; j < r.steps; ++j, ++n, wk.next(r)) {
          const Step s = wk.step(r);
          const int bq = r.b * a.Hq + r.hk * a.g + wk.e;
          const int sq = n % NRING1, so = n % NRING2;
          if (!wait_or_flag(gm.err, bar(&qempty[sq]), ((n / NRING1) & 1) ^ 1u) ||
              !wait_or_flag(gm.err, bar(&oempty[so]), ((n / NRING2) & 1) ^ 1u)) {
            bad = true;
            break;
          }
          tc::mbar_expect_tx(bar(&qfull[sq]), (uint32_t)(NP * s.w * 128));
          load_rows<NP>(Qr + sq * SH::TILE, &mp.q, &mp.q16, s.r0, s.w, bq, bar(&qfull[sq]));
          tc::mbar_expect_tx(bar(&ofull[so]), (uint32_t)(NP * s.w * 128));
          load_rows<NP>(Or + so * SH::TILE, &mp.dout, &mp.dout16, s.r0, s.w, bq, bar(&ofull[so]));
        }
      }
#pragma unroll 1
      for (int i = n > NRING1 ? n - NRING1 : 0; i < n; ++i) {
        wait_or_flag(gm.err, bar(&qfull[i % NRING1]), (uint32_t)(i / NRING1) & 1u);
        if (i >= n - NRING2) wait_or_flag(gm.err, bar(&ofull[i % NRING2]), (uint32_t)(i / NRING2) & 1u);
      }
      if (nk) wait_or_flag(gm.err, bar(&kvfull), (uint32_t)(nk - 1) & 1u);
    } else if (warp == WI + 2) {
      // ---------------- log-sums and D of the steps' queries ----------------
      int n = 0;
      bool bad = false;
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DkvItem r = dkv_item(a, gm, it);
        StepWalk wk = dkv_walk(r);
#pragma unroll 1
        for (int j = 0; j < r.steps; ++j, ++n, wk.next(r)) {
          const Step s = wk.step(r);
          const size_t q0 = ((size_t)r.b * a.Hq + r.hk * a.g + wk.e) * a.Nq;
          float x[4], y[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int i = s.r0 + lane + 32 * e;
            x[e] = i < s.re ? a.lse[q0 + i] : INFINITY;
            y[e] = i < s.re ? a.D[q0 + i] : 0.f;
          }
          if (!wait_warp(gm.err, bar(&lempty[n & 1]), ((n >> 1) & 1) ^ 1u)) { bad = true; break; }
#pragma unroll
          for (int e = 0; e < 4; ++e) Ls[n & 1][lane + 32 * e] = x[e];
          arrive(bar(&lfull[n & 1]));
          if (!wait_warp(gm.err, bar(&dempty), ((uint32_t)n & 1u) ^ 1u)) { bad = true; break; }
#pragma unroll
          for (int e = 0; e < 4; ++e) Ds[lane + 32 * e] = y[e];
          arrive(bar(&dfull));
        }
      }
    } else if (warp == WI + 1 && elect_one()) {
      // ---------------- products ----------------
      int n = 0, nk = 0, ng = 0;
      bool bad = false;
      const int ksteps = a.d / 16;
      auto commit = [&](uint64_t* b) { tc::commit(bar(b)); };
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const DkvItem r = dkv_item(a, gm, it);
        if (r.steps == 0) continue;
        if (!wait_or_flag(gm.err, bar(&kvfull), (uint32_t)nk++ & 1u)) { bad = true; break; }
        const int n0 = n;
        n += r.steps;
        // rows behind the sequence's end: zeros
        auto clean = [&](const Step& s, uint32_t tile) {
          const int e = r.sq.len - r.sq.qp - s.r0;
          if (s.w > e && r.sq.len - r.sq.qp < a.Nq) {
            zero_rows<NP>(tile, e, s.w);
          }
        };
        auto scores = [&](const Step& s, int i) {
          const int sq = i % NRING1;
          const uint32_t Q = Qr + sq * SH::TILE;
          if (!wait_or_flag(gm.err, bar(&qfull[sq]), (uint32_t)(i / NRING1) & 1u)) return false;
          clean(s, Q);
          tc::fence_after();
          mma_features<NP>(tS, Kb, Q, ksteps, idesc(BT, s.w, false));
          commit(&sfull);
          return true;
        };
        auto grads = [&](const Step& s, int i) {
          const int so = i % NRING2;
          const uint32_t O = Or + so * SH::TILE;
          if (!wait_or_flag(gm.err, bar(&ofull[so]), (uint32_t)(i / NRING2) & 1u)) return false;
          clean(s, O);
          tc::fence_after();
          mma_features<NP>(tP, Vb, O, ksteps, idesc(BT, s.w, false));
          commit(&dpfull);
          if (i + 1 == n) commit(&kvempty);   // the last product that reads K or V
          return true;
        };
        StepWalk wk = dkv_walk(r);
        Step s = wk.step(r);
        if (!scores(s, n0) || !grads(s, n0)) { bad = true; break; }
#pragma unroll 1
        for (int j = 0; j < r.steps; ++j) {
          const int i = n0 + j, sq = i % NRING1, so = i % NRING2;
          wk.next(r);
          const Step next = wk.step(r);
          if (!wait_or_flag(gm.err, bar(&pfull), (uint32_t)i & 1u) ||
              (j == 0 && !wait_or_flag(gm.err, bar(&gempty), ((uint32_t)ng++ & 1u) ^ 1u))) {
            bad = true;
            break;
          }
          tc::fence_after();
          const uint32_t id = idesc(BT, a.d, true);
          mma_rows<BT, 32>(tV, tS, Or + so * SH::TILE, s.w / 16, id, j > 0);
          commit(&oempty[so]);
          if (j + 1 < r.steps && !scores(next, i + 1)) { bad = true; break; }
          if (!wait_or_flag(gm.err, bar(&dsfull), (uint32_t)i & 1u)) { bad = true; break; }
          tc::fence_after();
          mma_rows<BT, 32>(tK, tP, Qr + sq * SH::TILE, s.w / 16, id, j > 0);
          commit(&qempty[sq]);
          if (j + 1 == r.steps) commit(&gfull);
          if (j + 1 < r.steps && !grads(next, i + 1)) { bad = true; break; }
          s = next;
        }
      }
      if (bad) {  // what was issued ends before tensor memory is freed
        commit(&drain);
        wait_or_flag(gm.err, bar(&drain), 0);
      }
    }
  } else {
    // ---------------- elementwise: rows are keys, columns queries ----------------
    const int grp = warp >> 2, row = 32 * (warp & 3) + lane, c0 = 32 * grp;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S = tS + lanes, P = tP + lanes;
    const float c = a.scale_log2;
    int n = 0, ng = 0;
    bool bad = false;
    for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
      const DkvItem r = dkv_item(a, gm, it);
      const int j = r.j0 + row;
      // positions [pl, ph) see this key
      int pl = j - a.right, ph = j < a.sinks ? r.sq.len : min(r.sq.len, j + a.left + 1);
      if (j >= r.j1) ph = pl = -kWinUnbounded;
      const bool keys_ok = r.j1 - r.j0 == BT;
      const int all_lo = r.j0 + BT - 1 - a.right;
      const int all_hi = r.j0 + BT <= a.sinks ? r.sq.len : min(r.sq.len, r.j0 + a.left + 1);
      const f32x2 c2 = pack2(c, c);
      StepWalk wk = dkv_walk(r);
#pragma unroll 1
      for (int k = 0; k < r.steps; ++k, ++n, wk.next(r)) {
        const Step s = wk.step(r);
        const int ps = r.sq.qp + s.r0;            // position of the step's first query
        const bool whole = keys_ok && s.re - s.r0 == BT && ps >= all_lo && ps + BT <= all_hi;
        const int l = pl - ps - c0, h = min(ph - ps, s.re - s.r0) - c0;
        const uint32_t bits = whole ? 0u : seen_bits(l, h, 0);
        const float* L = &Ls[n & 1][c0];
        const float* D = &Ds[c0];
        const bool ok = wait_or_flag(gm.err, bar(&lfull[n & 1]), (uint32_t)(n >> 1) & 1u);
        if (!wait_warp(gm.err, bar(&sfull), (uint32_t)n & 1u) || !__all_sync(0xffffffffu, ok)) {
          bad = true;
          break;
        }
        tc::fence_after();
        uint32_t v[32], o[16];
        ld32(S + c0, v);
        ld_wait(v);
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 ls = lds4(L + e);
          const float2 x = unpack2(fma2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), c2,
                                        pack2(-ls.x, -ls.y)));
          const float2 y = unpack2(fma2(pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])), c2,
                                        pack2(-ls.z, -ls.w)));
          v[e] = __float_as_uint(exp2_ftz(x.x));
          v[e + 1] = __float_as_uint(exp2_ftz(x.y));
          v[e + 2] = __float_as_uint(exp2_ftz(y.x));
          v[e + 3] = __float_as_uint(exp2_ftz(y.y));
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e)
            if (!(bits >> e & 1u)) v[e] = 0u;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) o[e >> 1] = pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        st16(S + c0, o);
        st_wait();
        tc::fence_before();
        arrive(bar(&pfull));
        arrive(bar(&lempty[n & 1]));

        const bool okd = wait_or_flag(gm.err, bar(&dfull), (uint32_t)n & 1u);
        if (!wait_warp(gm.err, bar(&dpfull), (uint32_t)n & 1u) || !__all_sync(0xffffffffu, okd)) {
          bad = true;
          break;
        }
        tc::fence_after();
        uint32_t dp[32];
        ld32(P + c0, dp);
        ld_wait(dp);
        float x[32];
#pragma unroll
        for (int e = 0; e < 32; e += 4) {
          const float4 ds = lds4(D + e);
          const float2 y = unpack2(mul2(pack2(__uint_as_float(v[e]), __uint_as_float(v[e + 1])),
                                        add2(pack2(__uint_as_float(dp[e]), __uint_as_float(dp[e + 1])),
                                             pack2(-ds.x, -ds.y))));
          const float2 w = unpack2(mul2(pack2(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3])),
                                        add2(pack2(__uint_as_float(dp[e + 2]), __uint_as_float(dp[e + 3])),
                                             pack2(-ds.z, -ds.w))));
          x[e] = y.x; x[e + 1] = y.y; x[e + 2] = w.x; x[e + 3] = w.y;
        }
        if (!whole) {
#pragma unroll
          for (int e = 0; e < 32; ++e) x[e] = bits >> e & 1u ? x[e] : 0.f;
        }
#pragma unroll
        for (int e = 0; e < 32; e += 2) o[e >> 1] = pack(x[e], x[e + 1]);
        st16(P + c0, o);
        st_wait();
        tc::fence_before();
        arrive(bar(&dsfull));
        arrive(bar(&dempty));
      }
      if (bad) break;
      if (r.steps > 0) {
        if (!wait_warp(gm.err, bar(&gfull), (uint32_t)ng & 1u)) break;
        ++ng;
        tc::fence_after();
      }
      // dK by groups 0 and 1, dV by 2 and 3, pieces of 32 columns in turn
      const int which = grp >> 1;
      const uint32_t G = (which ? tV : tK) + lanes;
      const float f = which ? 1.f : a.scale;
      const size_t head = (size_t)r.b * a.Hkv + r.hk;
      __nv_bfloat16* dst = (__nv_bfloat16*)(which ? a.dv : a.dk) + (head * a.Nk + r.j0) * a.d;
      float* part = a.part + (((head * a.stiles + r.tile) * a.chunks + (r.chunk >= 0 ? r.chunk : 0)) * 2 +
                              which) * BT * a.d;
#pragma unroll 1
      for (int q = 32 * (grp & 1); q < a.d; q += 64) {
        uint32_t o[32];
        if (r.steps > 0) {
          ld32(G + q, o);
          ld_wait(o);
        } else {
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = 0;
        }
        if (r.chunk >= 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint4 x[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const uint32_t* p = o + 16 * h + 4 * e;
              x[e] = make_uint4(__float_as_uint(__uint_as_float(p[0]) * f), __float_as_uint(__uint_as_float(p[1]) * f),
                                __float_as_uint(__uint_as_float(p[2]) * f), __float_as_uint(__uint_as_float(p[3]) * f));
            }
            if (q + 16 * h < a.d)
              store_rows(part + q + 16 * h, 4 * (size_t)a.d, 32 * (warp & 3), BT, 4, x);
          }
        } else {
          store_bf16(dst + q, nullptr, a.d, 32 * (warp & 3), a.Nk - r.j0, (a.d - q) / 8, o, f);
        }
      }
      if (r.steps > 0) {
        tc::fence_before();
        arrive(bar(&gempty));
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == WI) tc::tmem_dealloc(tmem, 512);
}

namespace {
template <int NP>
cudaError_t bwd_go(const BwdMaps& mp, const WinArgs& a, int* err, cudaStream_t st) {
  constexpr size_t smem = BwdShape<NP>::SMEM;
  static SmemOnce once_q, once_kv;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once_q.allow(k_win_dq_tc<NP>, smem, dev)) != cudaSuccess ||
      (e = once_kv.allow(k_win_dkv_tc<NP>, smem, dev)) != cudaSuccess)
    return e;
  BwdGeom gm;
  gm.err = err;
  gm.tiles = (a.Nq + BT - 1) / BT;
  gm.items = a.B * a.Hq * gm.tiles;
  e = launch("win_dq_tc", k_win_dq_tc<NP>, dim3((unsigned)(gm.items < sms ? gm.items : sms)),
             dim3(BTH), smem, st, mp, a, gm);
  if (e != cudaSuccess) return e;
  gm.tiles = a.stiles * a.chunks + (a.Nk + BT - 1) / BT - a.stiles;
  gm.items = a.B * a.Hkv * gm.tiles;
  e = launch("win_dkv_tc", k_win_dkv_tc<NP>, dim3((unsigned)(gm.items < sms ? gm.items : sms)),
             dim3(BTH), smem, st, mp, a, gm);
  if (e != cudaSuccess || a.stiles == 0) return e;
  return run_win_join(a, BT, true, st);
}
}  // namespace

int win_tc_tile_rows() { return BT; }

cudaError_t run_win_bwd_tc(const WinArgs& a, cudaStream_t st) {
  int* err = wait_error_address();
  if (err == nullptr) return cudaErrorInvalidSymbol;
  BwdMaps mp;
  const int bq = a.B * a.Hq, bk = a.B * a.Hkv;
  if (!win_map(&mp.q, a.q, bq, a.Nq, a.d, BT) || !win_map(&mp.q16, a.q, bq, a.Nq, a.d, 16) ||
      !win_map(&mp.dout, a.dout, bq, a.Nq, a.d, BT) || !win_map(&mp.dout16, a.dout, bq, a.Nq, a.d, 16) ||
      !win_map(&mp.k, a.k, bk, a.Nk, a.d, BT) || !win_map(&mp.k16, a.k, bk, a.Nk, a.d, 16) ||
      !win_map(&mp.v, a.v, bk, a.Nk, a.d, BT) || !win_map(&mp.v16, a.v, bk, a.Nk, a.d, 16))
    return cudaErrorInvalidValue;
  return a.d <= 64 ? bwd_go<1>(mp, a, err, st) : bwd_go<2>(mp, a, err, st);
}

}  // namespace lapnys
