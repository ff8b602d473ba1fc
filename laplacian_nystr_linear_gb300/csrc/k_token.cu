// Windowed softmax attention for a few queries per sequence (single tokens, or
// the few of a step that answers): over plain keys and values (bf16, fp32), or
// over a cache of 8-bit values in blocks with one power-of-two scale per block
// and head (k = k8 * k_scale, v = v8 * v_scale).  Visibility rule: win.cuh.
//
// What bounds it: every visible key and value is read once, for all the query
// heads that share it, and nothing else is large.  So the work is split over the
// keys: a block takes one (sequence, key head, 16 query rows) and one contiguous
// share of the visible groups of 16 keys, its warps take groups in turn, each
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
//   - 8-bit: e4m3 -> f16 is exact; q is scaled per row by a power of two to fit
//     f16 (a row's features below 2^-38 of its largest are lost); p is kept as
//     2^10 p in f16.  fp32 queries: q and p in two f16 parts (2^-22).
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
constexpr int TGK = 16;     // keys of a group
enum : int { TK_BF16 = 0, TK_E4M3 = 1, TK_E4M3_F32 = 2, TK_F32 = 3 };

template <int KIND>
struct Kind {
  static constexpr int ES = KIND == TK_F32 ? 4 : (KIND == TK_BF16 ? 2 : 1);  // bytes of k, v
  static constexpr bool QF32 = KIND == TK_E4M3_F32 || KIND == TK_F32;
  static constexpr bool F16 = KIND == TK_E4M3 || KIND == TK_E4M3_F32;
  static constexpr int PARTS = KIND == TK_F32 ? 3 : (KIND == TK_E4M3_F32 ? 2 : 1);
  static constexpr float SHIFT = F16 ? 10.f : 0.f;  // p is held as 2^SHIFT p
};
template <int KIND, int DP>
__host__ __device__ constexpr int ring_stages() { return KIND == TK_F32 && DP == 128 ? 3 : 4; }
template <int KIND, int DP>
__host__ __device__ constexpr size_t token_smem() {
  return (size_t)TNW * ring_stages<KIND, DP>() * (2 * TGK * DP * Kind<KIND>::ES + 16);
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
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16) mma_f16(d, a, b0, b1); else mma_bf(d, a, b0, b1);
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

// byte offset of a row's 16-byte chunk in a tile of TGK rows of RB bytes.  A key
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
  constexpr int ES = X::ES, RB = DP * ES, NP = X::PARTS;
  constexpr int NST = ring_stages<KIND, DP>();
  constexpr int TILE = TGK * RB, STG = 2 * TILE;
  constexpr int KS = DP / 16;                  // k steps of the scores
  constexpr int NT = DP / 8;                   // column steps of P V
  constexpr int PIECE = 16 / ES;               // features of a 16-byte piece
  constexpr int KSP = PIECE / 4;               // k steps of a piece
  constexpr int CH = RB / 16;                  // 16-byte chunks of a row
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

  // this block's share of the groups: first tokens' groups, then the window's
  const int gs = (kr.S + TGK - 1) / TGK, w0 = kr.lo / TGK;
  const int G = gs + (kr.hi > kr.lo ? (kr.hi + TGK - 1) / TGK - w0 : 0);
  const int g0 = (int)((long long)G * sp / t.splits), g1 = (int)((long long)G * (sp + 1) / t.splits);

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

  uint8_t* my = ring + warp * NST * (STG + 16);
  const uint32_t my_s = smem_addr(my);
  const size_t plain = ((size_t)b * a.Hkv + hk) * a.Nk;

  // first key of group gi and the range of keys that its phase counts
  auto group = [&](int gi, int* j0, int* jb, int* je) {
    const bool f = gi < gs;
    *j0 = (f ? gi : w0 + gi - gs) * TGK;
    *jb = f ? 0 : kr.lo;
    *je = f ? kr.S : kr.hi;
  };
  auto block_of = [&](int gi) -> int {   // the cache block that holds group gi
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
    return t.table[(size_t)b * t.max_blocks + j0 / t.T];
  };
  // copies of group gi into ring slot st
  auto issue = [&](int gi, int st, int blk) {
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
    const uint32_t dst = my_s + st * (STG + 16);
    size_t tok;
    bool there = true;
    if (t.table) {
      there = (unsigned)blk < (unsigned)t.blocks;
      if (!there && lane == 0) atomicOr(t.err, 2);
      const size_t bh = (size_t)(there ? blk : 0) * a.Hkv + hk;
      tok = bh * t.T + j0 % t.T;
      if (lane == 0) {
        cp_async4(dst + STG, t.k_scale + bh);
        cp_async4(dst + STG + 4, t.v_scale + bh);
        *reinterpret_cast<int*>(my + st * (STG + 16) + STG + 8) = there;
      }
    } else {
      tok = plain + j0;
    }
#pragma unroll
    for (int u = 0; u < TGK * CH / 32; ++u) {
      const int id = u * 32 + lane, r = id / CH, c = id % CH;
      const bool ok = there && c * PIECE < a.d && j0 + r >= jb && j0 + r < je;
      const size_t off = ok ? ((tok + r) * a.d + c * PIECE) * ES : 0;
      cp_async16(dst + k_off<RB>(r, c), (const uint8_t*)a.k + off, ok);
      cp_async16(dst + TILE + v_off<RB>(r, c), (const uint8_t*)a.v + off, ok);
    }
  };

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[NT][4];
#pragma unroll
  for (int n = 0; n < NT; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  int gi = g0 + warp, gn = gi;       // group to compute, group to issue
  int blk = t.table && gn < g1 ? block_of(gn) : 0;
#pragma unroll
  for (int st = 0; st < NST - 1; ++st) {
    if (gn < g1) issue(gn, st, blk);
    gn += TNW;
    if (t.table && gn < g1) blk = block_of(gn);
    cp_commit();
  }
  int st = 0;
  for (; gi < g1; gi += TNW) {
    asm volatile("cp.async.wait_group %0;" ::"n"(NST - 2) : "memory");
    __syncwarp();
    const uint8_t* Kt = my + st * (STG + 16);
    const uint8_t* Vt = Kt + TILE;
    int j0, jb, je;
    group(gi, &j0, &jb, &je);
    float ksc = 1.f, vsc = 1.f;
    if (t.table) {
      ksc = *reinterpret_cast<const float*>(Kt + STG);
      vsc = *reinterpret_cast<const float*>(Kt + STG + 4);
      if (!*reinterpret_cast<const int*>(Kt + STG + 8)) je = jb;  // no such block: no keys
    }
    // ---- scores ----
    float s[2][4];
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int e = 0; e < 4; ++e) s[u][e] = 0.f;
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
        } else {
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            const uint32_t b0 = e4m3x2_f16(w[x]), b1 = e4m3x2_f16(w[x] >> 16);
#pragma unroll
            for (int p = NP - 1; p >= 0; --p) mma_f16(s[u], qf[p][4 * i + x], b0, b1);
          }
        }
      }
    }
    // ---- softmax, running maximum and sum ----
    float p[2][4];
    bool up = false;
    float f[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int j = j0 + 8 * u + 2 * tq + e;
          float& x = s[u][2 * r + e];
          x = j >= jb && j < je && win_sees(row[r], j) ? x * (qs[r] * ksc) : -INFINITY;
          mx = fmaxf(mx, x);
        }
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
      mx = fmaxf(mx, m[r]);
      const float mu = mx == -INFINITY ? 0.f : mx;
      f[r] = exp2f(m[r] - mu);
      up = up || mx > m[r];
      m[r] = mx;
      float sum = 0.f;
#pragma unroll
      for (int u = 0; u < 2; ++u)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float x = exp2f(s[u][2 * r + e] - mu + X::SHIFT);
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
    // ---- P V ----
    if constexpr (KIND == TK_E4M3 || KIND == TK_E4M3_F32) {
      constexpr int W = DP / 8 / 4;  // 32-bit words of a thread's value row piece
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
        for (int e = 0; e < 4; ++e) o[n][e] = fmaf(c[e], vsc, o[n][e]);
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
    __syncwarp();
    if (gn < g1) issue(gn, st == 0 ? NST - 1 : st - 1, blk);
    gn += TNW;
    if (t.table && gn < g1) blk = block_of(gn);
    cp_commit();
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
  const long long most = (keys / TGK + 2 * TNW - 1) / (2 * TNW);
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
    const long long w = (long long)left + right + Nq + sinks + 2 * TGK;
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
