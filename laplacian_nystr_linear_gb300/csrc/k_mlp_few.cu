// The feed-forward block for a few rows (single tokens of some sequences, small batches).
//
// Bound by memory: every weight is read once and used for all rows, so the weights are
// laid out as one stretch of units, 64 k of a block of columns each, block after block,
// and every CTA takes an equal share of it, whatever the sizes are.  A CTA leaves the
// partial sums of each column block that it met; k_mlp_few_join adds a block's parts in
// order and applies bias, gate or the gate's gradient.  Every kernel lets the next one
// start at once and waits for the one before itself, so the second product's CTAs fetch
// weights as soon as the first one's leave their SMs, before the join in between.
//
// The weights are the instruction's left operand, as they lie (MN-major forward, K-major
// in the backward's two products), the rows of x its N, padded to 16.  bf16 (k_mlp_few_tc):
// one thread copies by TMA into a ring of 32 KB slots, one issues, four warps read the
// sums; h and (dg | du) are two bf16 planes (16 bits), the second as further rows of x,
// which costs a call bound by its weights nothing.  16 tokens, 4096 x 10880: 55 us, 5.3 TB/s
// while a product runs.
// fp32, up to 8 rows (k_mlp_few_fma, forward, and k_mlp_few_fma_k, backward): on the FP32
// pipe; a token of 4096 x 10880: 102 us, 5.5 TB/s while a product runs.  9 to 128 rows
// (k_mlp_few_f32): sixteen warps load the weights two units ahead, split them into three bf16
// planes (x comes as three) and write those as operand tiles; six products of planes, a0 b0
// summed over 128 k by the instruction and beyond by the epilogue's registers, as in the large
// products.  148 us at 16 rows (the loading warps' instructions; in two groups with a unit
// each: 169), 216 at 64 (the products of 64 columns); the large products take 464 through
// their packed weights.  More than 64 rows: a second CTA beside, weights out of L2.
#include <cuda.h>

#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "mlp.cuh"
#include "win_tc.cuh"

namespace lapnys {
namespace {

constexpr int FNB = 256, FNF = 128;   // columns of a unit (bf16, fp32)
constexpr int FK = 64;                // k of a unit
constexpr int FEW_BF16 = 64, FEW_F32 = 128, FEW_FMA = 8;   // rows of a call
constexpr int FR = 64;                // rows of an fp32 CTA
constexpr int NTC = 192, NST = 6;     // bf16: threads, slots at the most
constexpr uint32_t A_BYTES = FNB * FK * 2;
// fp32: a warp that issues, three idle beside it, sixteen that load, eight that read the sums
constexpr int LW = 16, EW = 8, NF32 = 32 * (4 + LW + EW), NSF = 3;
constexpr int LP = 128 * 8 / (32 * LW);       // pieces of eight weights a loading thread
constexpr uint32_t PLANE = FNF * FK * 2;      // of the weights' tile
constexpr int KCH = 2;                        // units of an accumulator
// Units of an accumulator, since the instruction cuts its sums off (k_mlp.cu): of bf16 weights
// (a CTA adds the next ones to its slot), and of the smaller products of fp32 ones
constexpr int CUT_BF16 = 256, CUT_F32 = 32;
static_assert(CUT_F32 % KCH == 0, "");

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// the stretch [u0, u1) of a CTA; unit u is k step u % ks of column block u / ks
__device__ __forceinline__ void stretch(const MlpFewArgs& a, int c, int* u0, int* u1) {
  const long long units = (long long)a.nparts * a.nb * a.ks;
  *u0 = (int)(units * c / a.grid);
  *u1 = (int)(units * (c + 1) / a.grid);
}

struct FewMaps {
  CUtensorMap w, x;
};

__device__ __forceinline__ void tma2(uint32_t dst, const CUtensorMap* map, int c0, int c1, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3}], [%4];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(mbar)
      : "memory");
}

__global__ void __launch_bounds__(NTC, 1) k_mlp_few_tc(const __grid_constant__ FewMaps mp, MlpFewArgs a,
                                                        int rows, int nst) {
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[NST], empty[NST], accf[2], acce[2];
  __shared__ uint32_t tmem_s;
  __shared__ int issued_s, consumed_s, bad_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, xrows = a.planes * a.T;
  const uint32_t sm = (tc::smem_u32(sm_raw) + 1023u) & ~1023u;
  const uint32_t b_bytes = (uint32_t)rows * FK * 2, slot = A_BYTES + b_bytes;
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  if (warp == 1) tc::tmem_alloc(&tmem_s, 512);
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(tc::smem_u32(&full[i]), 1);
      tc::mbar_init(tc::smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&accf[i]), 1);
      tc::mbar_init(tc::smem_u32(&acce[i]), 4);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    issued_s = 0;
    consumed_s = 0;
    bad_s = 0;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;
  let_next();      // this block has its tensor memory: no later one holds it back
  if (!(warp == 0 && a.second)) wait_before();

  if (warp == 0) {
    // ---------------- copies ----------------
    if (wtc::elect_one()) {
      int issued = 0;
      bool bad = false;
      auto weights = [&](int u, int st) {
        const int block = u / a.ks, k = u - block * a.ks, part = block / a.nb;
        const uint32_t bar = tc::smem_u32(&full[st]), sa = sm + st * slot;
        const int n = (block - part * a.nb) * FNB;
        tc::mbar_expect_tx(bar, slot);
        if (a.kmajor) {
          const int kp = k >= a.kst ? 1 : 0;
#pragma unroll
          for (int i = 0; i < FNB / 128; ++i)
            wtc::tma3(sa + 16384 * i, &mp.w, (k - kp * a.kst) * FK, kp, n + 128 * i, bar);
        } else {
          // columns of the row of both parts: a part's last block may reach into the next
          // part, whose sums nobody reads
#pragma unroll
          for (int i = 0; i < FNB / 64; ++i) tma2(sa + 8192 * i, &mp.w, part * a.N + n + 64 * i, k * FK, bar);
        }
      };
      // weights are no other kernel's output here: as many as there is room for before
      // the rows are there
      const int head = a.second ? (u1 - u0 < nst ? u1 - u0 : nst) : 0;
      for (int i = 0; i < head; ++i) weights(u0 + i, i);
      if (a.second) wait_before();
      for (int u = u0; u < u1; ++u) {
        const int st = issued % nst, k = u % a.ks, kp = k >= a.kst ? 1 : 0;
        if (issued >= head) {
          if (!wtc::wait_or_flag(a.err, tc::smem_u32(&empty[st]), ((uint32_t)(issued / nst) & 1u) ^ 1u)) {
            bad = true;
            break;
          }
          weights(u, st);
        }
        wtc::tma3(sm + st * slot + A_BYTES, &mp.x, (k - kp * a.kst) * FK, kp, 0, tc::smem_u32(&full[st]));
        ++issued;
      }
      issued_s = issued;
      if (bad) atomicOr(&bad_s, 1);
    }
  } else if (warp == 1) {
    // ---------------- products ----------------
    if (wtc::elect_one()) {
      int consumed = 0, seg = 0;
      bool bad = false;
      const uint32_t id = tc::idesc_bf16(128, rows) | (a.kmajor ? 0u : 1u << 15);
      const uint64_t da0 = a.kmajor ? wtc::desc_k(sm) : wtc::desc_mn(sm, 8192), db0 = wtc::desc_k(sm + A_BYTES);
      const uint64_t step = a.kmajor ? 2 : 128;      // a slice of 16 k
      for (int u = u0; u < u1 && !bad; ++seg) {
        const int end = min(min(u1, (u / a.ks + 1) * a.ks), u + CUT_BF16), first = u;
        if (!wtc::wait_or_flag(a.err, tc::smem_u32(&acce[seg & 1]), ((uint32_t)(seg >> 1) & 1u) ^ 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
        const uint32_t d = tmem + (uint32_t)(seg & 1) * 256;
        for (; u < end; ++u) {
          const int st = consumed % nst;
          if (!wtc::wait_or_flag(a.err, tc::smem_u32(&full[st]), (uint32_t)(consumed / nst) & 1u)) {
            bad = true;
            break;
          }
          tc::fence_after();
          const uint64_t da = da0 + (uint64_t)(st * slot >> 4), db = db0 + (uint64_t)(st * slot >> 4);
#pragma unroll
          for (int k = 0; k < FK / 16; ++k) {
            tc::mma_bf16(d, da + step * k, db + 2 * k, id, u > first || k > 0);
            tc::mma_bf16(d + 128, da + 1024 + step * k, db + 2 * k, id, u > first || k > 0);
          }
          tc::commit(tc::smem_u32(&empty[st]));
          ++consumed;
        }
        if (!bad) tc::commit(tc::smem_u32(&accf[seg & 1]));
      }
      consumed_s = consumed;
      if (bad) atomicOr(&bad_s, 1);
    }
  } else {
    // ---------------- sums ----------------
    const int q = warp & 3;
    bool bad = false;
    for (int u = u0, seg = 0; u < u1 && !bad; ++seg) {
      const int block = u / a.ks;
      const bool more = u > u0 && u > block * a.ks;      // this thread's values are there
      u = min(min(u1, (block + 1) * a.ks), u + CUT_BF16);
      __syncwarp();
      if (!wtc::wait_warp(a.err, tc::smem_u32(&accf[seg & 1]), (uint32_t)(seg >> 1) & 1u)) {
        bad = true;
        break;
      }
      tc::fence_after();
      // one slot for each (column block, CTA) that meet: both only grow
      float* o = a.part + (size_t)(block + blockIdx.x) * xrows * FNB + 32 * q + lane;
      for (int t0 = 0; t0 < rows; t0 += 16)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[16];
          tc::tmem_ld<16>(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)((seg & 1) * 256 + 128 * half + t0), x);
          if (more)
#pragma unroll
            for (int i = 0; i < 16; ++i)
              if (t0 + i < xrows)
                x[i] = __float_as_uint(__uint_as_float(x[i]) + o[(t0 + i) * FNB + 128 * half]);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + i < xrows) o[(t0 + i) * FNB + 128 * half] = __uint_as_float(x[i]);
        }
      tc::fence_before();
      wtc::arrive_warp(tc::smem_u32(&acce[seg & 1]));
    }
    if (bad) atomicOr(&bad_s, 1);
  }
  __syncthreads();
  // after an expired wait: the last products, then the copies that were not consumed
  if (bad_s && tid == 32) {
    const int c = consumed_s, n = issued_s;
    if (c > 0) wtc::wait_or_flag(a.err, tc::smem_u32(&empty[(c - 1) % nst]), (uint32_t)((c - 1) / nst) & 1u);
    for (int k = c; k < n; ++k) wtc::wait_or_flag(a.err, tc::smem_u32(&full[k % nst]), (uint32_t)(k / nst) & 1u);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 1) tc::tmem_dealloc(tmem, 512);
}

// fp32 weights.  WIDE: their rows are whole 16-byte pieces.  Tensor memory: a0 b0 of two
// chunks, 64 columns each; from 128 and from 256 on the smaller products, a0 b1 + a1 b0 and
// a0 b2 + a1 b1 + a2 b0, of a segment: up to CUT_F32 units of a column block.
template <bool WIDE>
__global__ void __launch_bounds__(NF32, 1) k_mlp_few_f32(MlpFewArgs a, int rows) {
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[NSF], empty[NSF], accf[2], acce[2], smalle[2];
  __shared__ uint32_t tmem_s;
  __shared__ int consumed_s, bad_s;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int row0 = blockIdx.y * FR, T = min(FR, a.T - row0);      // rows of this CTA
  const uint32_t sm = (tc::smem_u32(sm_raw) + 1023u) & ~1023u;
  const uint32_t slot = 3 * PLANE + 3 * (uint32_t)rows * 128;
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  if (warp == 0) tc::tmem_alloc(&tmem_s, 512);
  if (tid == 0) {
    for (int i = 0; i < NSF; ++i) {
      tc::mbar_init(tc::smem_u32(&full[i]), LW);
      tc::mbar_init(tc::smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&accf[i]), 1);
      tc::mbar_init(tc::smem_u32(&acce[i]), EW);
      tc::mbar_init(tc::smem_u32(&smalle[i]), EW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    consumed_s = 0;
    bad_s = 0;
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  const uint32_t tmem = tmem_s;
  let_next();      // this block has its tensor memory: no later one holds it back

  if (warp == 0) {
    // ---------------- products ----------------
    if (wtc::elect_one()) {
      int consumed = 0, seg = 0;
      uint32_t ch = 0;                       // chunks so far
      bool bad = false;
      const uint32_t mn = a.kmajor ? 0u : 1u << 15;
      const uint32_t id1 = tc::idesc_bf16(128, rows) | mn, id2 = tc::idesc_bf16(128, 2 * rows) | mn;
      const uint64_t da0 = a.kmajor ? wtc::desc_k(sm) : wtc::desc_mn(sm, 8192);
      const uint64_t db0 = wtc::desc_k(sm + 3 * PLANE);
      const uint64_t step = a.kmajor ? 2 : 128, pa = PLANE >> 4, pb = (uint64_t)rows * 128 >> 4;
      for (int u = u0; u < u1 && !bad; ++seg) {
        const int end = min(min(u1, (u / a.ks + 1) * a.ks), u + CUT_F32), first = u;
        const uint32_t small = tmem + 128 + (uint32_t)(seg & 1) * 128;
        if (!wtc::wait_or_flag(a.err, tc::smem_u32(&smalle[seg & 1]), ((uint32_t)(seg >> 1) & 1u) ^ 1u)) {
          bad = true;
          break;
        }
        for (; u < end && !bad; ++ch) {
          const int stop = min(end, u + KCH), c0 = u;
          if (!wtc::wait_or_flag(a.err, tc::smem_u32(&acce[ch & 1]), ((ch >> 1) & 1u) ^ 1u)) { bad = true; break; }
          tc::fence_after();
          const uint32_t d = tmem + (ch & 1) * 64;
          for (; u < stop; ++u) {
            const int st = consumed % NSF;
            if (!wtc::wait_or_flag(a.err, tc::smem_u32(&full[st]), (uint32_t)(consumed / NSF) & 1u)) {
              bad = true;
              break;
            }
            tc::fence_after();
            const uint64_t da = da0 + (uint64_t)(st * slot >> 4), db = db0 + (uint64_t)(st * slot >> 4);
#pragma unroll
            for (int k = 0; k < FK / 16; ++k) {
              const uint64_t ak = da + step * k, bk = db + 2 * k;
              tc::mma_bf16(d, ak, bk, id1, u > c0 || k > 0);
              tc::mma_bf16(small, ak, bk + pb, id2, u > first || k > 0);     // a0 b1, a0 b2
              tc::mma_bf16(small, ak + pa, bk, id2, 1);                      // a1 b0, a1 b1
              tc::mma_bf16(small + rows, ak + 2 * pa, bk, id1, 1);           // a2 b0
            }
            tc::commit(tc::smem_u32(&empty[st]));
            ++consumed;
          }
          if (!bad) tc::commit(tc::smem_u32(&accf[ch & 1]));
        }
      }
      consumed_s = consumed;
      if (bad) atomicOr(&bad_s, 1);
    }
  } else if (warp >= 4 && warp < 4 + LW) {
    // ---------------- loads ----------------
    const int lt = tid - 128;
    const float* w = (const float*)a.w;
    const size_t ldw = a.kmajor ? (size_t)a.kparts * a.K : (size_t)a.nparts * a.N;
    // Pieces of eight values of a tile's rows: MN-major rows are k in two blocks of 64
    // columns, K-major ones columns.  Of the unit that is fetched next: column block, k step,
    // pointers; divisions once a column block.
    int nu = u0, nk = u0 % a.ks, nblock = u0 / a.ks;
    const float* at[LP];
    int left[LP];                            // values of the row from there (MN-major)
    auto place = [&]() {
      const int part = nblock / a.nb, n0 = (nblock - part * a.nb) * FNF, kp = nk >= a.kst ? 1 : 0;
      const int k0 = (nk - kp * a.kst) * FK;
#pragma unroll
      for (int j = 0; j < LP; ++j) {
        const int r = (lt + 32 * LW * j) >> 3, c = (lt & 7) * 8;
        const int k = a.kmajor ? k0 + c : k0 + (r & 63), n = a.kmajor ? n0 + r : n0 + (r & 64) + c;
        at[j] = a.kmajor ? w + (size_t)n * ldw + (size_t)kp * a.K + k : w + (size_t)k * ldw + (size_t)part * a.N + n;
        left[j] = a.kmajor ? (n < a.N ? a.K : 0) : a.N - n;
      }
    };
    auto fetch = [&](float(&v)[LP][8]) {
      const int k0 = (nk >= a.kst ? nk - a.kst : nk) * FK;
#pragma unroll
      for (int j = 0; j < LP; ++j) {
        const int r = (lt + 32 * LW * j) >> 3, c = (lt & 7) * 8;
        const int m = a.kmajor ? left[j] - k0 - c : (k0 + (r & 63) < a.K ? left[j] : 0);   // of the piece's row
        if constexpr (WIDE) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float4 f = m > 4 * h ? __ldcs(reinterpret_cast<const float4*>(at[j]) + h)
                                       : make_float4(0.f, 0.f, 0.f, 0.f);
            v[j][4 * h] = f.x; v[j][4 * h + 1] = f.y; v[j][4 * h + 2] = f.z; v[j][4 * h + 3] = f.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 8; ++i) v[j][i] = m > i ? __ldcs(at[j] + i) : 0.f;
        }
        at[j] += a.kmajor ? (size_t)FK : FK * ldw;
      }
      ++nu;
      if (++nk == a.ks) {
        nk = 0;
        ++nblock;
        if (nu < u1) place();
      } else if (nk == a.kst) {
        place();                             // K's second part
      }
    };
    // x's three planes of a unit, rows padded with zeros: this thread's pieces
    constexpr int XP = 3 * FR * 8 / (32 * LW);
    const __nv_bfloat16* x = (const __nv_bfloat16*)a.x;
    const __nv_bfloat16* xat[XP];
    uint32_t xto[XP];
    bool xin[XP];
    const int pieces = 3 * rows * 8, xc = (lt & 7) * 8;
#pragma unroll
    for (int i = 0; i < XP; ++i) {
      const int e = lt + 32 * LW * i, rr = e >> 3, plane = rr / rows, t = rr - plane * rows;
      xin[i] = e < pieces && t < T;
      xat[i] = x + ((size_t)plane * a.T + row0 + t) * a.ldx + xc;
      xto[i] = sm + 3 * PLANE + rr * 128 + (((lt & 7) ^ (rr & 7)) << 4);
    }
    int xk = u0 % a.ks;                      // k step of the unit whose rows come next
    auto fetch_x = [&](int st) {
      const int kp = xk >= a.kst ? 1 : 0, k0 = (xk - kp * a.kst) * FK;
      const size_t off = kp * a.xpart + k0;
      const bool in = k0 + xc < ((a.K + 7) & ~7);
#pragma unroll
      for (int i = 0; i < XP; ++i)
        if (lt + 32 * LW * i < pieces)
          cp_async16(xto[i] + st * slot, xin[i] && in ? xat[i] + off : x, xin[i] && in);
      cp_commit();
      if (++xk == a.ks) xk = 0;
    };
    float v0[LP][8], v1[LP][8];
    bool bad = false;
    int n = 0, st = 0;                       // units so far, slot
    // one unit, its weights in v: split, written, and v filled for two units later
    auto work = [&](int u, float(&v)[LP][8]) {
      const int after = st + 1 == NSF ? 0 : st + 1;
      if (u + 1 < u1) {
        // the next unit's slot is free
        if (!wtc::wait_warp(a.err, tc::smem_u32(&empty[after]), ((uint32_t)((n + 1) / NSF) & 1u) ^ 1u)) {
          bad = true;
          return;
        }
        fetch_x(after);
      } else {
        cp_commit();
      }
      const uint32_t base = sm + st * slot;
#pragma unroll
      for (int j = 0; j < LP; ++j) {
        const int r = (lt + 32 * LW * j) >> 3, c = lt & 7;
        uint32_t s[4][3];
#pragma unroll
        for (int i = 0; i < 4; ++i) split3_bf16x2(v[j][2 * i], v[j][2 * i + 1], s[i]);
        const uint32_t to = base + r * 128 + ((c ^ (r & 7)) << 4);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(to + p * PLANE), "r"(s[0][p]), "r"(s[1][p]),
                       "r"(s[2][p]), "r"(s[3][p])
                       : "memory");
      }
      if (u + 2 < u1) fetch(v);
      asm volatile("cp.async.wait_group 1;" ::: "memory");     // this unit's x
      tc::fence_async_smem();
      wtc::arrive_warp(tc::smem_u32(&full[st]));
      ++n;
      st = after;
    };
    if (!a.second) wait_before();
    place();
    fetch(v0);
    if (u0 + 1 < u1) fetch(v1);
    if (a.second) wait_before();             // the weights are no other kernel's output
    fetch_x(0);
    for (int u = u0; u < u1 && !bad; u += 2) {
      work(u, v0);
      if (u + 1 < u1 && !bad) work(u + 1, v1);
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    if (bad) atomicOr(&bad_s, 1);
  } else if (warp >= 4 + LW) {
    // ---------------- sums: half of the rows a warp ----------------
    wait_before();
    constexpr int HR = FR / 2;
    const int q = warp & 3, h0 = warp >= 8 + LW ? HR : 0;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    bool bad = false;
    uint32_t ch = 0;
    int seg = 0;
    for (int u = u0; u < u1 && !bad;) {
      const int block = u / a.ks, end = min(u1, (block + 1) * a.ks);
      int cut = min(end, u + CUT_F32);       // where the segment ends
      float R[HR];
#pragma unroll
      for (int i = 0; i < HR; ++i) R[i] = 0.f;
      for (; u < end; u = min(end, u + KCH), ++ch) {
        __syncwarp();
        if (!wtc::wait_warp(a.err, tc::smem_u32(&accf[ch & 1]), (ch >> 1) & 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
        const bool last = u + KCH >= cut;
        const uint32_t small = tmem + lanes + 128 + (uint32_t)(seg & 1) * 128 + h0;
#pragma unroll
        for (int t0 = 0; t0 < HR; t0 += 16)
          if (h0 + t0 < rows) {
            uint32_t x[16];
            tc::tmem_ld<16>(tmem + lanes + (ch & 1) * 64 + h0 + t0, x);
#pragma unroll
            for (int i = 0; i < 16; ++i) R[t0 + i] += __uint_as_float(x[i]);
            if (last)
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                tc::tmem_ld<16>(small + h * rows + t0, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) R[t0 + i] += __uint_as_float(x[i]);
              }
          }
        tc::fence_before();
        wtc::arrive_warp(tc::smem_u32(&acce[ch & 1]));
        if (last) {
          wtc::arrive_warp(tc::smem_u32(&smalle[seg & 1]));
          ++seg;
          cut = min(end, cut + CUT_F32);
        }
      }
      if (bad) break;
      float* o = a.part + ((size_t)(block + blockIdx.x) * a.T + row0 + h0) * FNF + 32 * q + lane;
#pragma unroll
      for (int t = 0; t < HR; ++t)
        if (h0 + t < T) o[t * FNF] = R[t];
    }
    if (bad) atomicOr(&bad_s, 1);
  }
  __syncthreads();
  if (bad_s && tid == 0) {                   // after an expired wait: the last products
    const int c = consumed_s;
    if (c > 0) wtc::wait_or_flag(a.err, tc::smem_u32(&empty[(c - 1) % NSF]), (uint32_t)((c - 1) / NSF) & 1u);
  }
  tc::fence_before();
  __syncthreads();
  tc::fence_after();
  if (warp == 0) tc::tmem_dealloc(tmem, 512);
}

// fp32, up to 8 rows (TT, padded), on the FP32 pipe: no more than eight multiply-adds a
// weight, which it does as fast as weights come.  x is summed up again from its three planes
// (exactly what it was, or h to 2^-24).  A segment is a CTA's stretch of one column block.
constexpr int FT = 256;               // threads
constexpr int XC = 256;               // k of x in shared memory

// x[t][k0 .. k0 + XC) of K's part kp
template <int TT>
__device__ __forceinline__ void rows_in(const MlpFewArgs& a, int kp, int k0, float* to, int ldt, int ldk) {
  const __nv_bfloat16* x = (const __nv_bfloat16*)a.x + kp * a.xpart + k0;
  const size_t plane = (size_t)a.T * a.ldx;
  for (int e = threadIdx.x; e < XC * TT; e += FT) {
    const int t = e / XC, k = e % XC;
    float v = 0.f;
    if (t < a.T && k0 + k < a.K) {
      const __nv_bfloat16* p = x + (size_t)t * a.ldx + k;
      v = __bfloat162float(p[0]) + (__bfloat162float(p[plane]) + __bfloat162float(p[2 * plane]));
    }
    to[t * ldt + k * ldk] = v;
  }
}

// w [K][nparts][N]: four columns a lane, rows of x in packed pairs; the warps take a
// segment's k in turn and their sums are joined in shared memory, halves of the warps at a
// time, in one order
template <int TT, bool WIDE>
__global__ void __launch_bounds__(FT, 2) k_mlp_few_fma(MlpFewArgs a) {
  __shared__ __align__(16) float xs[XC][TT];
  __shared__ __align__(16) float4 join[4][TT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  let_next();
  wait_before();
  const size_t ld = (size_t)a.nparts * a.N;
  for (int u = u0; u < u1;) {
    const int block = u / a.ks, part = block / a.nb, n = (block - part * a.nb) * FNF + 4 * lane;
    const int end = min(u1, (block + 1) * a.ks);
    const int k0 = (u - block * a.ks) * FK, k1 = min(a.K, (end - block * a.ks) * FK);
    u = end;
    f32x2 acc[4][TT / 2];                   // column, rows 2 t and 2 t + 1
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int t = 0; t < TT / 2; ++t) acc[c][t] = pack2(0.f, 0.f);
    const float* w = (const float*)a.w + (size_t)part * a.N + n;
    for (int kc = k0; kc < k1; kc += XC) {
      const int m = min(XC, k1 - kc);
      __syncthreads();
      rows_in<TT>(a, 0, kc, &xs[0][0], 1, TT);
      __syncthreads();
#pragma unroll 8
      for (int k = warp; k < m; k += FT / 32) {
        const float* p = w + (size_t)(kc + k) * ld;
        float v[4];
        if constexpr (WIDE) {
          const float4 f = n < a.N ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = n + c < a.N ? __ldcs(p + c) : 0.f;
        }
#pragma unroll
        for (int t = 0; t < TT; t += 4) {
          const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&xs[k][t]);
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const f32x2 ww = pack2(v[c], v[c]);
            acc[c][t / 2] = fma2(ww, x.x, acc[c][t / 2]);
            acc[c][t / 2 + 1] = fma2(ww, x.y, acc[c][t / 2 + 1]);
          }
        }
      }
    }
    auto row = [&](int t) {
      float f[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const float2 y = unpack2(acc[c][t / 2]);
        f[c] = t & 1 ? y.y : y.x;
      }
      return make_float4(f[0], f[1], f[2], f[3]);
    };
#pragma unroll
    for (int half = 4; half >= 1; half >>= 1) {
      __syncthreads();
      if (warp >= half && warp < 2 * half)
#pragma unroll
        for (int t = 0; t < TT; ++t) join[warp - half][t][lane] = row(t);
      __syncthreads();
      if (warp < half)
#pragma unroll
        for (int t = 0; t < TT; t += 2) {
          const float4 y = join[warp][t][lane], z = join[warp][t + 1][lane];
          acc[0][t / 2] = wtc::add2(acc[0][t / 2], pack2(y.x, z.x));
          acc[1][t / 2] = wtc::add2(acc[1][t / 2], pack2(y.y, z.y));
          acc[2][t / 2] = wtc::add2(acc[2][t / 2], pack2(y.z, z.z));
          acc[3][t / 2] = wtc::add2(acc[3][t / 2], pack2(y.w, z.w));
        }
    }
    if (warp == 0) {
      float* o = a.part + (size_t)(block + blockIdx.x) * a.T * FNF + 4 * lane;
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < a.T) *reinterpret_cast<float4*>(o + t * FNF) = row(t);
    }
  }
}

// w [N][kparts][K]: a warp takes 16 of a block's columns (rows of w), four at a time, its
// lanes along k; x is read from shared memory once for the four
template <int TT, bool WIDE>
__global__ void __launch_bounds__(FT, 2) k_mlp_few_fma_k(MlpFewArgs a) {
  constexpr int RB = 4;               // rows of w at a time
  __shared__ __align__(16) float xs[TT][XC];
  __shared__ float sums[FNF][TT + 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  let_next();
  wait_before();
  const size_t ld = (size_t)a.kparts * a.K;
  for (int u = u0; u < u1;) {
    const int block = u / a.ks, end = min(u1, (block + 1) * a.ks), n0 = block * FNF + 16 * warp;
    int ku = u - block * a.ks;
    const int kend = end - block * a.ks;
    u = end;
    for (int i = lane; i < 16 * TT; i += 32) sums[16 * warp + i / TT][i % TT] = 0.f;
    while (ku < kend) {
      // as many steps as lie in one part of K and in shared memory
      const int kp = ku >= a.kst ? 1 : 0, k0 = (ku - kp * a.kst) * FK;
      const int steps = min(min(kend, (kp + 1) * a.kst) - ku, XC / FK), m = min(a.K - k0, steps * FK);
      ku += steps;
      __syncthreads();
      rows_in<TT>(a, kp, k0, &xs[0][0], XC, 1);
      __syncthreads();
#pragma unroll 1
      for (int r = 0; r < 16; r += RB) {
        f32x2 acc[RB][TT];
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int t = 0; t < TT; ++t) acc[i][t] = pack2(0.f, 0.f);
        const float* w = (const float*)a.w + (size_t)(n0 + r) * ld + (size_t)kp * a.K + k0 + 4 * lane;
        float4 f[RB][XC / 128];
#pragma unroll
        for (int j = 0; j < XC / 128; ++j)
#pragma unroll
          for (int i = 0; i < RB; ++i) {
            const float* p = w + i * ld + 128 * j;
            const int left = n0 + r + i < a.N ? m - 128 * j - 4 * lane : 0;
            f[i][j] = make_float4(0.f, 0.f, 0.f, 0.f);
            if constexpr (WIDE) {
              if (left > 0) f[i][j] = __ldcs(reinterpret_cast<const float4*>(p));
            } else {
              if (left > 0) f[i][j].x = __ldcs(p);
              if (left > 1) f[i][j].y = __ldcs(p + 1);
              if (left > 2) f[i][j].z = __ldcs(p + 2);
              if (left > 3) f[i][j].w = __ldcs(p + 3);
            }
          }
#pragma unroll
        for (int j = 0; j < XC / 128; ++j)
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const ulonglong2 x = *reinterpret_cast<const ulonglong2*>(&xs[t][128 * j + 4 * lane]);
#pragma unroll
            for (int i = 0; i < RB; ++i) {
              acc[i][t] = fma2(pack2(f[i][j].x, f[i][j].y), x.x, acc[i][t]);
              acc[i][t] = fma2(pack2(f[i][j].z, f[i][j].w), x.y, acc[i][t]);
            }
          }
#pragma unroll
        for (int i = 0; i < RB; ++i)
#pragma unroll
          for (int t = 0; t < TT; ++t) {
            const float2 y = unpack2(acc[i][t]);
            float v = y.x + y.y;
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
            if (lane == 0) sums[16 * warp + r + i][t] += v;
          }
      }
    }
    __syncwarp();
    float* o = a.part + (size_t)(block + blockIdx.x) * a.T * FNF + 16 * warp;
    for (int i = lane; i < 16 * TT; i += 32)
      if (i / 16 < a.T) o[(i / 16) * FNF + i % 16] = sums[16 * warp + i % 16][i / 16];
    __syncwarp();
  }
}

// v as `planes` bf16 values, plane elements apart (infinities leave nothing to the later ones)
__device__ __forceinline__ void put_planes(__nv_bfloat16* o, size_t plane, int planes, float v) {
  for (int i = 0; i < planes; ++i) {
    const __nv_bfloat16 h = __float2bfloat16_rn(v);
    o[i * plane] = h;
    v = isinf(__bfloat162float(h)) && planes == 2 ? 0.f : v - __bfloat162float(h);
  }
}

// a column block (blockIdx.x) of a row (blockIdx.y): its parts in order, then what the mode
// makes of them
template <typename T>
__global__ void __launch_bounds__(256) k_mlp_few_join(MlpFewArgs a) {
  constexpr bool F32 = sizeof(T) == 4;
  constexpr int FN = F32 ? FNF : FNB;
  const int t = blockIdx.y, n = blockIdx.x * FN + threadIdx.x;
  let_next();
  wait_before();
  const long long units = (long long)a.nparts * a.nb * a.ks;
  const int stack = F32 ? 1 : a.planes;      // bf16: the planes' sums lie apart
  const size_t slot = (size_t)stack * a.T * FN;
  float v[2] = {0.f, 0.f};
  for (int p = 0; p < a.nparts; ++p) {
    const long long block = p * a.nb + blockIdx.x, first = block * a.ks, last = first + a.ks - 1;
    // the CTA of unit u: the greatest c with units c / grid <= u
    const int c0 = (int)(((first + 1) * a.grid - 1) / units), c1 = (int)(((last + 1) * a.grid - 1) / units);
    for (int h = stack - 1; h >= 0; --h) {   // the smaller sums first
      const float* s = a.part + (size_t)(block + c0) * slot + ((size_t)h * a.T + t) * FN + threadIdx.x;
      float sum = 0.f;
#pragma unroll 4
      for (int c = c0; c <= c1; ++c, s += slot) sum += *s;
      v[p] += sum;
    }
    if (a.bias && n < a.N) {
      if constexpr (F32)
        v[p] += ((const T*)a.bias)[(size_t)p * a.N + n];
      else
        v[p] += __bfloat162float(((const T*)a.bias)[(size_t)p * a.N + n]);
    }
  }
  const size_t at = (size_t)t * a.N + n;
  if (a.mode == kFewRows) {
    if (n >= a.N) return;
    if constexpr (F32)
      ((T*)a.out)[at] = v[0];
    else
      ((T*)a.out)[at] = __float2bfloat16_rn(v[0]);
    return;
  }
  if (n >= (int)a.ldo) return;
  const bool in = n < a.N;                   // zeros behind the row, as far as its padding goes
  if (a.mode == kFewGlu) {
    float p, s;
    if (a.act == kActSilu)
      mlp_act<F32, kActSilu>(v[0], p, s);
    else if (a.act == kActGelu)
      mlp_act<F32, kActGelu>(v[0], p, s);
    else
      mlp_act<F32, kActGeluTanh>(v[0], p, s);
    if (a.p && in) {
      a.p[at] = p;
      a.q[at] = v[1] * s;
    }
    put_planes((__nv_bfloat16*)a.out + t * a.ldo + n, a.T * a.ldo, a.out_planes, in ? p * v[1] : 0.f);
  } else {
    __nv_bfloat16* o = (__nv_bfloat16*)a.out + 2 * t * a.ldo + n;
    put_planes(o, 2 * a.T * a.ldo, a.out_planes, in ? v[0] * a.q[at] : 0.f);
    put_planes(o + a.ldo, 2 * a.T * a.ldo, a.out_planes, in ? v[0] * a.p[at] : 0.f);
  }
}

// grid and units of a product: a CTA for each SM (two on the FP32 pipe), as far as there are
// units
void shape(MlpFewArgs& a, bool f32) {
  const int fn = f32 ? FNF : FNB;
  a.nb = (a.N + fn - 1) / fn;
  a.kst = (a.K + FK - 1) / FK;
  a.ks = a.kst * a.kparts;
  const long long units = (long long)a.nparts * a.nb * a.ks, most = !f32 ? 152 : a.T <= FEW_FMA ? 304 : 152 / ((a.T + FR - 1) / FR);
  a.grid = (int)(units < most ? units : most);
}

}  // namespace

// Few enough rows to read all weights once; bf16 rows and columns have to be whole 16-byte
// pieces.  (bf16, 4096 x 10880: 73 us at 64 rows, 81 by the large products at 65.  fp32, 3782 x
// 15128, forward + backward: 1452 us at 128 rows, 1531 by the large products at 129.)
bool mlp_few_ok(int T, int C, int F, bool f32) {
  if ((double)C * F >= 1e12) return false;      // units are counted in 32 bits
  return f32 ? T <= FEW_F32 : T <= FEW_BF16 && C % 8 == 0 && F % 8 == 0;
}

size_t mlp_few_bytes(int T, int planes, int N, int nparts, bool f32) {
  const int fn = f32 ? FNF : FNB;
  return ((size_t)nparts * ((N + fn - 1) / fn) + 304) * T * (f32 ? 1 : planes) * fn * 4;
}

template <int TT>
static cudaError_t go_fma(const MlpFewArgs& a, bool wide, cudaStream_t st) {
  auto* k = a.kmajor ? (wide ? k_mlp_few_fma_k<TT, true> : k_mlp_few_fma_k<TT, false>)
                     : (wide ? k_mlp_few_fma<TT, true> : k_mlp_few_fma<TT, false>);
  if (a.second) return launch_after("mlp_few", k, dim3(a.grid), dim3(FT), 0, st, a);
  return launch("mlp_few", k, dim3(a.grid), dim3(FT), 0, st, a);
}

cudaError_t run_mlp_few(MlpFewArgs& a, bool f32, cudaStream_t st) {
  shape(a, f32);
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  a.err = wait_error_address();
  if (a.err == nullptr) return cudaErrorInvalidSymbol;
  const bool pieces = ((uintptr_t)a.w & 15) == 0 && (a.kmajor ? a.K : a.N) % 4 == 0;
  if (f32 && a.T <= FEW_FMA) {
    e = a.T <= 4 ? go_fma<4>(a, pieces, st) : go_fma<8>(a, pieces, st);
  } else if (f32) {
    const int groups = (a.T + FR - 1) / FR, most = a.T < FR ? a.T : FR, rows = (most + 15) / 16 * 16;
    const bool wide = pieces;
    auto* k = wide ? k_mlp_few_f32<true> : k_mlp_few_f32<false>;
    static SmemOnce once[2];
    const size_t smem = NSF * (3 * PLANE + 3 * (size_t)rows * 128) + 1024;
    if ((e = once[wide].allow(k, NSF * (3 * PLANE + 3 * FR * 128) + 1024, dev)) != cudaSuccess) return e;
    const dim3 grid(a.grid, groups);
    e = a.second ? launch_after("mlp_few", k, grid, dim3(NF32), smem, st, a, rows)
                 : launch("mlp_few", k, grid, dim3(NF32), smem, st, a, rows);
  } else {
    const int rows = (a.planes * a.T + 15) / 16 * 16;
    FewMaps mp;
    memset(&mp, 0, sizeof(mp));
    bool ok;
    if (a.kmajor) {
      const cuuint64_t d[3] = {(cuuint64_t)a.K, (cuuint64_t)a.kparts, (cuuint64_t)a.N};
      const cuuint64_t s[2] = {(cuuint64_t)a.K * 2, (cuuint64_t)a.K * a.kparts * 2};
      const cuuint32_t b[3] = {64, 1, 128};
      ok = encode_tiled_bf16_sw128(&mp.w, 3, a.w, d, s, b);
    } else {
      const cuuint64_t d[2] = {(cuuint64_t)a.nparts * a.N, (cuuint64_t)a.K}, s[1] = {d[0] * 2};
      const cuuint32_t b[2] = {64, FK};
      ok = encode_tiled_bf16_sw128(&mp.w, 2, a.w, d, s, b);
    }
    const cuuint64_t d[3] = {(cuuint64_t)a.K, (cuuint64_t)a.kparts, (cuuint64_t)a.planes * a.T};
    const cuuint64_t s[2] = {(cuuint64_t)a.xpart * 2, (cuuint64_t)a.ldx * 2};
    const cuuint32_t b[3] = {64, 1, (cuuint32_t)rows};
    if (!ok || !encode_tiled_bf16_sw128(&mp.x, 3, a.x, d, s, b)) return cudaErrorInvalidValue;
    static SmemOnce once;
    // six slots of up to 32 rows of x, four of more
    const int nst = rows <= 32 ? NST : 4;
    constexpr size_t most = NST * (A_BYTES + 32 * FK * 2) + 1024;
    static_assert(4 * (A_BYTES + 2 * FEW_BF16 * FK * 2) + 1024 <= most, "");
    if ((e = once.allow(k_mlp_few_tc, most, dev)) != cudaSuccess) return e;
    const size_t smem = nst * (A_BYTES + (size_t)rows * FK * 2) + 1024;
    e = a.second ? launch_after("mlp_few", k_mlp_few_tc, dim3(a.grid), dim3(NTC), smem, st, mp, a, rows, nst)
                 : launch("mlp_few", k_mlp_few_tc, dim3(a.grid), dim3(NTC), smem, st, mp, a, rows, nst);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(a.nb, a.T);
  if (f32) return launch_after("mlp_few_join", k_mlp_few_join<float>, grid, dim3(FNF), 0, st, a);
  return launch_after("mlp_few_join", k_mlp_few_join<__nv_bfloat16>, grid, dim3(FNB), 0, st, a);
}

}  // namespace lapnys
