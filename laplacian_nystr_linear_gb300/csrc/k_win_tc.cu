// Windowed softmax attention, forward, bf16, on the tcgen05 tensor cores
// (visibility rule: win.cuh; operand tiles: win_tc.cuh).
//
// One CTA per SM walks over items of two tiles of 128 query rows that share their
// keys: the same rows of two query heads of a group when the group's size is
// even, else neighbouring rows of one head.  The keys come in steps of at most
// 64: first the steps of the first tokens, then the window's, from its first
// key on (TMA rows start anywhere), a last step as wide as it has to be (a
// multiple of 16), so four first tokens cost a step of 16 keys.
//
//   warps 0-3, 4-7  softmax of tile 0 and of tile 1, one row per thread: scores
//                   from tensor memory, exp2 in fp32, P as bf16 back into the
//                   scores' columns.  The running maximum is only moved when it
//                   grows by more than 2^8 (P <= 2^8: fp32 sums and bf16's
//                   relative rounding are as good there), so the outputs are
//                   rescaled on few steps;
//   warp 8          TMA: K and V tiles through two rings;
//   warps 9, 10     one thread each issues a tile's  S = Q K^T  (both operands in
//                   shared memory) and  O += P V  (P in tensor memory, V as it lies:
//                   MN-major).  A tile has two score buffers, so the scores of the
//                   next step are there when the softmax of this one ends.  Steps of
//                   128 keys leave no room for that beside two outputs of 128 columns:
//                   then softmax, P V and the next Q K^T of a tile follow one another
//                   (a prompt of 32768: 444 us against 426).
//
// Bound: 4 d flops per visible pair on the tensor pipe, or one exponential per
// pair on the special-function pipe, whichever is longer (d = 64: the latter).
// Measured: a prompt of 32768 tokens, 8 heads of 128 on 2, window 4096: 428 us, 1.2
// PFLOP/s; 16384 tokens, 2 x 16 heads of 64, window 1024: 260 us (0.51 PFLOP/s), the
// softmax warps' arithmetic and the steps' latencies; 3136 tokens, 32 heads, windows
// of 225: 35 us.
// Rows of V at and behind the sequence's end are zeroed in shared memory (P is 0
// there, but 0 * NaN is not); rows behind the tensor's are zero by TMA.
// Every wait is bounded, as in the other tensor-core kernels.
#include <cstring>

#include "internal.h"
#include "win_tc.cuh"

namespace lapnys {

namespace {
using namespace wtc;
constexpr int FT = 128;                 // query rows of a tile
constexpr int FK = 64;                  // keys of a step
constexpr int FTH = 352;
constexpr int FNST = 4;                 // tiles of the K ring and of the V ring
template <int NP>
struct FwdShape {
  static constexpr uint32_t QTILE = NP * FT * 128;   // panels of 64 features: rows of 128 bytes
  static constexpr uint32_t TILE = NP * FK * 128;
  static constexpr uint32_t SMEM = 2 * QTILE + 2 * FNST * TILE + 1024;
};
constexpr float kMoveMax = 8.f;         // the maximum moves when it grows by 2^8

struct FwdMaps {
  CUtensorMap q;                        // boxes of 64 x 128
  CUtensorMap k, v;                     // boxes of 64 x 64
  CUtensorMap k16, v16;                 // boxes of 64 x 16 for narrow steps
};
struct FwdGeom {
  int npair;                            // items per (batch, key head): pairs of heads or of tiles
  int by_head;                          // 1: an item's tiles are two heads
  int items;
  int* err;
};

struct FwdItem {
  int b, hk;
  int head[2], i0[2], i1[2];            // query head and rows of both tiles
  WinSeq sq;
  WinRange kr;                          // keys that either tile sees
  WinRange own[2];
  int ns, nw;                           // steps of the first tokens, of the window
};
__device__ __forceinline__ FwdItem fwd_item(const WinArgs& a, const FwdGeom& gm, int it) {
  FwdItem r;
  // the last query tiles first: with an open left side they see the most keys
  const int heads = a.B * a.Hkv * (gm.by_head ? a.g / 2 : a.g);
  const int tq = gm.npair - 1 - it / heads;
  int h = it % heads;
  const int per = gm.by_head ? a.g / 2 : a.g;
  const int e = h % per;
  h /= per;
  r.hk = h % a.Hkv;
  r.b = h / a.Hkv;
  r.sq = win_seq(a, r.b);
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    r.head[s] = r.hk * a.g + (gm.by_head ? 2 * e + s : e);
    r.i0[s] = min(a.Nq, (gm.by_head ? tq : 2 * tq + s) * FT);
    r.i1[s] = min(a.Nq, r.i0[s] + FT);
    r.own[s] = r.i0[s] < r.i1[s] ? win_keys(a, r.sq, r.i0[s], r.i1[s]) : WinRange{0, 0, 0};
  }
  r.kr = win_keys(a, r.sq, r.i0[0], r.i1[1]);
  r.ns = (r.kr.S + FK - 1) / FK;
  r.nw = r.kr.hi > r.kr.lo ? (r.kr.hi - r.kr.lo + FK - 1) / FK : 0;
  return r;
}
// step j of an item: keys [j0, je), and the width of its products
struct FwdStep {
  int j0, je, w;
};
__device__ __forceinline__ FwdStep fwd_step(const FwdItem& r, int j) {
  FwdStep s;
  if (j < r.ns) {
    s.j0 = j * FK;
    s.je = min(r.kr.S, s.j0 + FK);
  } else {
    s.j0 = r.kr.lo + (j - r.ns) * FK;
    s.je = min(r.kr.hi, s.j0 + FK);
  }
  s.w = (s.je - s.j0 + 15) & ~15;
  return s;
}
// The steps that one tile takes part in, as step numbers: those of the first
// tokens, those of the window that it sees, and window steps that still hold first
// tokens (where both ranges are one); and the widths.
struct FwdPlan {
  int ns, steps, head, lo, hi;     // [0, head) and [lo, hi)
  int wS, wW;                      // width of the last step of either kind
  __device__ __forceinline__ bool on(int j) const { return j < head || (j >= lo && j < hi); }
  __device__ __forceinline__ int width(int j) const {
    return j == ns - 1 ? wS : (j == steps - 1 ? wW : FK);
  }
  __device__ __forceinline__ int count() const {
    return max(head, 0) + max(0, hi - max(lo, head));
  }
};
__device__ __forceinline__ FwdPlan fwd_plan(const WinArgs& a, const FwdItem& r, const WinRange& own) {
  FwdPlan p;
  p.ns = r.ns;
  p.steps = r.ns + r.nw;
  p.head = p.lo = p.hi = 0;
  if (own.hi > 0) {
    const int first = min(a.sinks, own.hi);        // first tokens that it may see
    p.head = r.ns + (r.kr.lo < first ? (first - r.kr.lo + FK - 1) / FK : 0);
    p.lo = r.ns + (own.lo - r.kr.lo) / FK;
    p.hi = r.ns + (own.hi - r.kr.lo + FK - 1) / FK;
  }
  p.wS = (r.kr.S - (r.ns - 1) * FK + 15) & ~15;
  p.wW = (r.kr.hi - r.kr.lo - (r.nw - 1) * FK + 15) & ~15;
  return p;
}
}  // namespace

template <int NP>
__global__ void __launch_bounds__(FTH, 1) k_win_fwd_tc(const __grid_constant__ FwdMaps mp,
                                                       const WinArgs a, const FwdGeom gm) {
  using SH = FwdShape<NP>;
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t kfull[FNST], kempty[FNST], vfull[FNST], vempty[FNST];
  __shared__ __align__(8) uint64_t qfull[2], qempty[2];   // Q tile landed; its products done
  __shared__ __align__(8) uint64_t sfull[2][2];           // scores ready, by tile and buffer
  __shared__ __align__(8) uint64_t pfull[2][2];           // P written (128 arrivals)
  // a step's P V done, by tile and parity of the step (a step is only known to have
  // its P V behind it two steps later: one barrier's parity could not tell); O read out
  __shared__ __align__(8) uint64_t pvdone[2][2], oempty[2];
  __shared__ __align__(8) uint64_t drain[2];
  __shared__ uint32_t tmem_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t raw = tc::smem_u32(sm_raw), base = (raw + 1023u) & ~1023u;
  const uint32_t qbuf = base, kring = base + 2 * SH::QTILE, vring = kring + FNST * SH::TILE;
  auto bar = [](uint64_t* b) { return tc::smem_u32(b); };

  if (warp == 9) tc::tmem_alloc(&tmem_s, 512);
  if (tid == 0) {
    for (int i = 0; i < FNST; ++i) {
      tc::mbar_init(bar(&kfull[i]), 1);
      tc::mbar_init(bar(&kempty[i]), 2);
      tc::mbar_init(bar(&vfull[i]), 1);
      tc::mbar_init(bar(&vempty[i]), 2);
    }
    for (int t = 0; t < 2; ++t) {
      tc::mbar_init(bar(&qfull[t]), 1);
      tc::mbar_init(bar(&qempty[t]), 1);
      for (int i = 0; i < 2; ++i) {
        tc::mbar_init(bar(&sfull[t][i]), 1);
        tc::mbar_init(bar(&pfull[t][i]), FT);
        tc::mbar_init(bar(&pvdone[t][i]), 1);
      }
      tc::mbar_init(bar(&oempty[t]), FT);
      tc::mbar_init(bar(&drain[t]), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;
  // tensor memory: the scores' buffers (then P) of both tiles, outputs of both
  const uint32_t tO = tmem + 4 * FK;

  if (warp == 8) {
    // ---------------- TMA ----------------
    if (elect_one()) {
      int n = 0;                       // steps issued
      int nq[2] = {0, 0};              // Q tiles issued
      bool bad = false;
      auto load = [&](const CUtensorMap* wide, const CUtensorMap* narrow, uint32_t dst, const FwdStep& s,
                      int bh, uint32_t full) {
        tc::mbar_expect_tx(full, (uint32_t)(NP * s.w * 128));
#pragma unroll
        for (int p = 0; p < NP; ++p) {
          if (s.w == FK) {
            tma3(dst + p * FK * 128, wide, 64 * p, s.j0, bh, full);
          } else {
#pragma unroll 1
            for (int r = 0; r < s.w; r += 16)
              tma3(dst + p * FK * 128 + r * 128, narrow, 64 * p, s.j0 + r, bh, full);
          }
        }
      };
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const FwdItem r = fwd_item(a, gm, it);
        const int steps = r.ns + r.nw;
#pragma unroll
        for (int t = 0; t < 2; ++t) {
          if (r.own[t].hi == 0) continue;
          if (!wait_or_flag(gm.err, bar(&qempty[t]), (nq[t] & 1) ^ 1u)) { bad = true; break; }
          tc::mbar_expect_tx(bar(&qfull[t]), SH::QTILE);
#pragma unroll
          for (int p = 0; p < NP; ++p)
            tma3(qbuf + t * SH::QTILE + p * FT * 128, &mp.q, 64 * p, r.i0[t], r.b * a.Hq + r.head[t],
                 bar(&qfull[t]));
          ++nq[t];
        }
        const int bh = r.b * a.Hkv + r.hk;
#pragma unroll 1
        for (int j = 0; j < steps && !bad; ++j, ++n) {
          const FwdStep s = fwd_step(r, j);
          const int st = n % FNST;
          const uint32_t ph = (uint32_t)(n / FNST & 1) ^ 1u;
          if (!wait_or_flag(gm.err, bar(&kempty[st]), ph)) { bad = true; break; }
          load(&mp.k, &mp.k16, kring + st * SH::TILE, s, bh, bar(&kfull[st]));
          if (!wait_or_flag(gm.err, bar(&vempty[st]), ph)) { bad = true; break; }
          load(&mp.v, &mp.v16, vring + st * SH::TILE, s, bh, bar(&vfull[st]));
        }
      }
      // every copy has landed before the block ends, also after an expired wait (then
      // K of step n may be one more)
      for (int i = n > FNST ? n - FNST : 0; i < n; ++i) {
        wait_or_flag(gm.err, bar(&kfull[i % FNST]), (uint32_t)(i / FNST) & 1u);
        wait_or_flag(gm.err, bar(&vfull[i % FNST]), (uint32_t)(i / FNST) & 1u);
      }
      if (bad) wait_or_flag(gm.err, bar(&kfull[n % FNST]), (uint32_t)(n / FNST) & 1u);
#pragma unroll
      for (int t = 0; t < 2; ++t)
        if (nq[t]) wait_or_flag(gm.err, bar(&qfull[t]), (uint32_t)(nq[t] - 1) & 1u);
    }
  } else if (warp >= 9) {
    if (elect_one()) {
      // ---------------- products: warp 9 for tile 0, warp 10 for tile 1 ----------------
      const int t = warp - 9;
      int n = 0;                        // steps begun
      int nq = 0, no = 0;               // Q tiles, outputs
      int ks = 0, kp = 0;               // scores, P V issued
      bool bad = false;
      const int ksteps = a.d / 16;
      const uint32_t id_pv = idesc(FT, a.d, true);
      const uint32_t S = tmem + 2 * t * FK, O = tO + t * NP * 64, Q = qbuf + t * SH::QTILE;
      auto commit = [&](uint64_t* b) { tc::commit(bar(b)); };
      for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
        const FwdItem r = fwd_item(a, gm, it);
        const WinRange own = t ? r.own[1] : r.own[0];
        const int steps = r.ns + r.nw;
        if (steps == 0) continue;
        const FwdPlan plan = fwd_plan(a, r, own);
        int todo = plan.count();        // scores still to be issued
        const int clean = r.sq.len < a.Nk ? r.sq.len : kWinUnbounded;   // V rows from here on: zeros
        if (todo > 0 && !wait_or_flag(gm.err, bar(&qfull[t]), (uint32_t)nq++ & 1u)) { bad = true; break; }
        bool begun = false;
        const int n0 = n;
        n += steps;
        // scores of step j; both tiles release the step's K
        auto scores = [&](int j) {
          const int st = (n0 + j) % FNST;
          if (!wait_or_flag(gm.err, bar(&kfull[st]), (uint32_t)((n0 + j) / FNST) & 1u)) return false;
          if (plan.on(j)) {
            tc::fence_after();
            const int i = ks++;
            mma_features<NP, FT, FK>(S + (i & 1) * FK, Q, kring + st * SH::TILE, ksteps,
                                     idesc(FT, plan.width(j), false));
            commit(&sfull[t][i & 1]);
            if (--todo == 0) commit(&qempty[t]);
          }
          commit(&kempty[st]);
          return true;
        };
        if (!scores(0) || (steps > 1 && !scores(1))) { bad = true; break; }
#pragma unroll 1
        for (int j = 0; j < steps; ++j) {
          const int st = (n0 + j) % FNST;
          if (!wait_or_flag(gm.err, bar(&vfull[st]), (uint32_t)((n0 + j) / FNST) & 1u)) { bad = true; break; }
          if (plan.on(j)) {
            const uint32_t V = vring + st * SH::TILE;
            const int w = plan.width(j);
            if (j >= steps - 1 || j == r.ns - 1) {           // the last of either kind may end behind it
              const int j0 = fwd_step(r, j).j0;
              if (j0 + w > clean) zero_rows<NP, FK>(V, clean - j0, w);
            }
            const int i = kp++;
            if (!wait_or_flag(gm.err, bar(&pfull[t][i & 1]), (uint32_t)(i >> 1) & 1u) ||
                (!begun && !wait_or_flag(gm.err, bar(&oempty[t]), ((uint32_t)no++ & 1u) ^ 1u))) {
              bad = true;
              break;
            }
            tc::fence_after();
            mma_rows<FK>(O, S + (i & 1) * FK, V, w / 16, id_pv, begun);
            begun = true;
            commit(&pvdone[t][i & 1]);
          }
          commit(&vempty[st]);
          if (j + 2 < steps && !scores(j + 2)) { bad = true; break; }
        }
      }
      if (bad) {  // what was issued ends before tensor memory is freed
        commit(&drain[t]);
        wait_or_flag(gm.err, bar(&drain[t]), 0);
      }
    }
  } else {
    // ---------------- softmax ----------------
    const int t = warp >> 2;
    const int row = 32 * (warp & 3) + lane;
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t S0 = tmem + 2 * t * FK + lanes, O = tO + t * NP * 64 + lanes;
    const float c = a.scale_log2;
    int k = 0;                            // steps of this tile
    bool bad = false;
    for (int it = blockIdx.x; it < gm.items && !bad; it += gridDim.x) {
      const FwdItem r = fwd_item(a, gm, it);
      // (registers, not an indexed array)
      const WinRange own = t ? r.own[1] : r.own[0];
      const int i0 = t ? r.i0[1] : r.i0[0], i1 = t ? r.i1[1] : r.i1[0];
      const int head = t ? r.head[1] : r.head[0];
      const FwdPlan plan = fwd_plan(a, r, own);
      const int steps = plan.steps, i = i0 + row;
      WinRow wr = win_row(a, r.sq, i);
      if (i >= i1) wr = WinRow{0, 0, 0};
      // keys that every row of the tile sees: no mask
      const int p0 = r.sq.qp + i0, p1 = r.sq.qp + i1 - 1;
      const bool rows_ok = i1 - i0 == FT && p0 >= 0 && p1 < r.sq.len;
      const int free_lo = p1 - a.left, free_hi = min(p0 + a.right, r.sq.len - 1);
      float m = -INFINITY;
      f32x2 ls[2] = {pack2(0.f, 0.f), pack2(0.f, 0.f)};   // sums of the row, four chains
      bool any = false;
#pragma unroll 1
      for (int j = 0; j < steps; ++j) {
        if (!plan.on(j)) continue;
        const FwdStep s = fwd_step(r, j);
        const uint32_t S = S0 + (k & 1) * FK;
        if (!wait_warp(gm.err, bar(&sfull[t][k & 1]), (uint32_t)(k >> 1) & 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
        uint32_t v[2][32];
        ld32(S, v[0]);
        ld32(S + 32, v[1]);
        const bool whole = rows_ok && s.je - s.j0 == FK && s.j0 + FK - 1 <= free_hi &&
                           (s.j0 >= free_lo || s.je <= a.sinks);
        ld_wait(v[0]);
        ld_wait(v[1]);
        if (!whole) {
          const int h = min(wr.hi, s.je) - s.j0, l = wr.lo - s.j0, z = wr.S - s.j0;
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            const uint32_t bits = seen_bits(l - 32 * q, h - 32 * q, z - 32 * q);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(bits >> e & 1u)) v[q][e] = 0xff800000u;   // -inf
          }
        }
        float mq[4];                       // four chains: one is as long as its latencies
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const uint32_t (&x)[32] = v[q >> 1];
          const int e0 = 16 * (q & 1);
          mq[q] = fmaxf(__uint_as_float(x[e0]), __uint_as_float(x[e0 + 1]));
#pragma unroll
          for (int e = 2; e < 16; e += 2)
            mq[q] = fmaxf(fmaxf(mq[q], __uint_as_float(x[e0 + e])), __uint_as_float(x[e0 + e + 1]));
        }
        const float mx = fmaxf(fmaxf(mq[0], mq[1]), fmaxf(mq[2], mq[3]));
        const bool move = (mx - m) * c > kMoveMax || (m == -INFINITY && mx > m);
        const float mn = move ? mx : m;
        if (any && __any_sync(0xffffffffu, move)) {
          const float f = move ? exp2_ftz((m - mn) * c) : 1.f;   // m = -inf: 0
          ls[0] = mul2(ls[0], pack2(f, f));
          ls[1] = mul2(ls[1], pack2(f, f));
          // the step before has been added up (and this one's P V waits for this P)
          if (!wait_warp(gm.err, bar(&pvdone[t][(k - 1) & 1]), (uint32_t)((k - 1) >> 1) & 1u)) {
            bad = true;
            break;
          }
          tc::fence_after();
#pragma unroll 1
          for (int q = 0; q < a.d; q += 16) {
            uint32_t o[16];
            tc::tmem_ld<16>(O + q, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
            st16(O + q, o);
          }
        }
        any = true;
        m = mn;
        const float off = m == -INFINITY ? 0.f : -m * c;
        const f32x2 c2 = pack2(c, c), off2 = pack2(off, off);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          uint32_t p[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float2 x = unpack2(fma2(pack2(__uint_as_float(v[q][e]), __uint_as_float(v[q][e + 1])), c2, off2));
            const float y0 = exp2_ftz(x.x), y1 = exp2_ftz(x.y);
            ls[(e >> 1) & 1] = add2(ls[(e >> 1) & 1], pack2(y0, y1));
            p[e >> 1] = pack(y0, y1);
          }
          st16(S + 16 * q, p);
        }
        st_wait();
        tc::fence_before();
        arrive(bar(&pfull[t][k & 1]));
        ++k;
      }
      if (bad) break;
      const float2 la = unpack2(ls[0]), lb = unpack2(ls[1]);
      const float l = (la.x + la.y) + (lb.x + lb.y);
      if (i < i1 && a.lse)
        a.lse[((size_t)r.b * a.Hq + head) * a.Nq + i] = l == 0.f ? -INFINITY : fmaf(m, c, log2f(l));
      const float w = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      if (any) {
        if (!wait_warp(gm.err, bar(&pvdone[t][(k - 1) & 1]), (uint32_t)((k - 1) >> 1) & 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
      }
      // heads to 64: every lane stores its own row (262 us at 16384 tokens; in turns like the
      // wider heads 274; those 146 us so and 132 in turns, for 16 heads on 4)
      const size_t at = (((size_t)r.b * a.Hq + head) * a.Nq + i0) * a.d;
      __nv_bfloat16* out = (__nv_bfloat16*)a.out + at;
      __nv_bfloat16* rest = a.rest ? (__nv_bfloat16*)a.rest + at : nullptr;
      constexpr int W = NP == 1 ? 16 : 32;
#pragma unroll 1
      for (int q = 0; q < a.d; q += W) {
        uint32_t o[W];
        if (any) {
          tc::tmem_ld<W>(O + q, o);
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) o[e] = 0;
        }
        if constexpr (NP > 1) {
          store_bf16(out + q, rest ? rest + q : nullptr, a.d, 32 * (warp & 3), i1 - i0, (a.d - q) / 8, o, w);
        } else if (i < i1) {
#pragma unroll
          for (int e = 0; e < W; e += 8) {
            float f[8];
            const size_t p = (size_t)row * a.d + q + e;
#pragma unroll
            for (int x = 0; x < 8; ++x) f[x] = __uint_as_float(o[e + x]) * w;
            store8(out + p, rest ? rest + p : nullptr, f);
          }
        }
      }
      if (any) {
        tc::fence_before();
        arrive(bar(&oempty[t]));
      }
    }
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 9) tc::tmem_dealloc(tmem, 512);
}

// [B H][N][d] bf16, boxes of 64 features x `rows` rows
bool win_map(CUtensorMap* t, const void* p, int BH, int N, int d, int rows) {
  const cuuint64_t dim[3] = {(cuuint64_t)d, (cuuint64_t)N, (cuuint64_t)BH};
  const cuuint64_t stride[2] = {(cuuint64_t)d * 2, (cuuint64_t)N * d * 2};
  const cuuint32_t box[3] = {64, (cuuint32_t)rows, 1};
  return encode_tiled_bf16_sw128(t, 3, p, dim, stride, box);
}

namespace {
template <int NP>
cudaError_t fwd_go(const FwdMaps& mp, const WinArgs& a, const FwdGeom& gm, cudaStream_t st) {
  constexpr size_t smem = FwdShape<NP>::SMEM;
  static SmemOnce once;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once.allow(k_win_fwd_tc<NP>, smem, dev)) != cudaSuccess) return e;
  const unsigned grid = (unsigned)(gm.items < sms ? gm.items : sms);
  return launch("win_fwd_tc", k_win_fwd_tc<NP>, dim3(grid), dim3(FTH), smem, st, mp, a, gm);
}
}  // namespace

cudaError_t run_win_fwd_tc(const WinArgs& a, cudaStream_t st) {
  FwdMaps mp;
  FwdGeom gm;
  gm.err = wait_error_address();
  if (gm.err == nullptr) return cudaErrorInvalidSymbol;
  const int qt = (a.Nq + FT - 1) / FT;
  gm.by_head = a.g % 2 == 0;
  gm.npair = gm.by_head ? qt : (qt + 1) / 2;
  gm.items = a.B * a.Hkv * (gm.by_head ? a.g / 2 : a.g) * gm.npair;
  if (!win_map(&mp.q, a.q, a.B * a.Hq, a.Nq, a.d, FT) ||
      !win_map(&mp.k, a.k, a.B * a.Hkv, a.Nk, a.d, FK) ||
      !win_map(&mp.v, a.v, a.B * a.Hkv, a.Nk, a.d, FK) ||
      !win_map(&mp.k16, a.k, a.B * a.Hkv, a.Nk, a.d, 16) ||
      !win_map(&mp.v16, a.v, a.B * a.Hkv, a.Nk, a.d, 16))
    return cudaErrorInvalidValue;
  return a.d <= 64 ? fwd_go<1>(mp, a, gm, st) : fwd_go<2>(mp, a, gm, st);
}

}  // namespace lapnys
