// The products of the gated feed-forward block on the tcgen05 tensor cores, by pairs
// of CTAs (cta_group::2), with the activation, its gradient and the biases in the
// epilogues.  T rows, C features, F hidden (sizes M x N x K):
//     forward   g | u = x w_in, h = act(g) u       T x 2 F x C   epilogue: glu
//               y = h w_out                        T x C x F     rows
//     backward  dh = dy w_out^T, dg = dh q,
//               du = dh p                          T x F x C     dglu
//               dx = (dg | du) w_in^T              T x C x 2 F   rows
//               dw_in = x^T (dg | du)              C x 2 F x T   rows or part
//               dw_out = h^T dy                    F x C x T     rows or part
//
// A pair computes 256 x 256 of D = sum_k A(m, k) B(n, k): each CTA copies its 128 rows
// of A and 128 of the 256 rows of B, 32 KB a step of 64 k (a single CTA's 128 x 256 tile
// would take 48 KB for half the work, and L2 gives all SMs about 64 bytes a cycle each
// at the tensor cores' rate).  The leader's one thread issues the products for both.  In
// the glu product the leader's rows of B are the gate's columns, its partner's the
// other half's: both halves of a hidden feature land in one row of tensor memory.
//
// Operands lie as the tensors do, K contiguous (K-major) or not (MN-major), in the
// 128-byte swizzle; maps of four dimensions {inner, part, row, plane} fill what lies
// behind a row, a part (g | u) or the last row with zeros.
//
// The instruction cuts its sums off: 2^-23 of a sum of terms of one sign for every 16 k
// (2^24 rows summed in ranges of 2^19: 4.0e-3 lost, 2^26 rows: 1.2e-2).  So no accumulator of
// bf16 products takes more than 256 steps (16384 k: 2^-13 of the sum, where a bf16 result's own
// rounding is up to 2^-8) but those of g, u and dh, whose K are the features (up to 1024 steps,
// 2^-11); beyond, the epilogue's threads add up to nearest, rows in registers, partial sums where
// they lie, in L2 (LONG; a backward of 131072 rows, 512 x 1408: 858 us, 840 with ranges in one
// accumulator each, 893 with partial sums in registers, which spill).
//
// fp32 operands are three bf16 planes each (24 bits) and a product six of theirs, a0 b0
// apart from the five smaller ones in tensor memory: a0 b0 is summed over two steps there and
// in registers beyond, the others, 2^-7 of the sum at the most, over 32.  A step's planes are
// copied once and read from shared memory by all six.
//
// 640 threads a CTA (384 for dglu): warps 0 and 2 copy (a thread each, A and B, into a ring
// of NST slots), warp 1 issues (leader) and holds the tensor memory, warps 4 to 19 read the
// accumulators, a row a thread, a quarter of the columns each, while the next tile
// accumulates.  Every wait is bounded; a role whose wait expired sets the error word and
// stops issuing, and all threads meet at the cluster barrier before tensor memory is freed.
//
// Measured, bf16: 8192 rows, 8192 x 4096: 1.75 to 1.89 PFLOP/s in every product (the
// library's product of 8192^3: 1.93).  131072 rows, 512 x 1408, forward + backward: 290 +
// 117 + 278 + 214 + 230 + 123 us: the first and third are bound by what passes through L2
// (tiles of K = 512 in, h, p, q, dg and du in and out: 13 TB/s of it), the others run at
// 1.6 to 1.7 PFLOP/s.  fp32, 4096 rows, 1024 x 4096: 250 to 290 TFLOP/s (a sixth of the
// bf16 rate is 320).
#include <cuda_fp16.h>

#include <cstring>

#include "common.cuh"
#include "internal.h"
#include "mlp.cuh"
#include "win_tc.cuh"

namespace lapnys {
namespace {

constexpr int BM = 128;                  // rows of A a CTA
constexpr int BK = kMlpTileK;
// epilogue warps: the gradient of the hidden layer has p and q on their way in registers
// (96 a thread beside sixteen warps, 168 beside eight)
__host__ __device__ constexpr int epilogue_warps(int epi) { return epi == kMlpDglu ? 8 : 16; }
__host__ __device__ constexpr int threads_of(int epi) { return 128 + 32 * epilogue_warps(epi); }
constexpr int GROUP = 8;                 // tiles of M that tiles of N are run over together
constexpr uint32_t BLK64 = 64 * BK * 2;  // 64 rows of an MN-major operand: 8 KB

template <bool F32>
struct Cfg {
  static constexpr int BN = F32 ? 128 : 256;        // columns of a pair's tile
  static constexpr int BNC = BN / 2;                // rows of B a CTA
  static constexpr uint32_t A_BYTES = BM * BK * 2;
  static constexpr uint32_t B_BYTES = BNC * BK * 2;
  static constexpr uint32_t SLOT = A_BYTES + B_BYTES;
  static constexpr int NST = F32 ? 9 : 6;
  static constexpr int PLANES = F32 ? 3 : 1;
  static constexpr int KCH = F32 ? 2 : 256;         // K steps of an accumulator (bf16: LONG)
  static constexpr int KSM = 32;                    // F32: of the smaller products'
  static constexpr uint32_t SMEM = NST * SLOT + 1024;
};

struct Maps {
  CUtensorMap a, b;
};

__device__ __forceinline__ uint32_t rank_of_cta() {
  uint32_t r;
  asm("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
// the leader's copy of a shared-memory address of this CTA
__device__ __forceinline__ uint32_t at_leader(uint32_t addr) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, 0;" : "=r"(r) : "r"(addr));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\nbarrier.cluster.wait.acquire;" ::: "memory");
}
__device__ __forceinline__ void arrive_leader(uint32_t remote) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(remote) : "memory");
}
// a tile into this CTA's shared memory, its bytes counted on the leader's barrier
__device__ __forceinline__ void tma4(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                     int c3, uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "r"(mbar)
      : "memory");
}
__device__ __forceinline__ void mma2(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
// arrives on the barrier of both CTAs when all products issued so far are done
__device__ __forceinline__ void commit2(uint32_t mbar) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
          mbar),
      "h"((uint16_t)3)
      : "memory");
}

// barrier of the epilogue's warps (named barrier 1) that ORs a flag over them
template <int THREADS>
__device__ __forceinline__ bool epilogue_any(bool v) {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.red.or.pred q, 1, %2, p;\n"
      " selp.u32 %0, 1, 0, q;\n}\n"
      : "=r"(r)
      : "r"((uint32_t)v), "n"(THREADS)
      : "memory");
  return r != 0;
}

struct Item {
  int m0, n0, part, ks0, ks1, sp;   // n0: first column of the tile in its part
};
// (32-bit divisions: 64-bit ones took a third of an epilogue's instructions)
template <int TN>
__device__ __forceinline__ Item decode(const MlpGemmArgs& a, int it) {
  Item r;
  const unsigned ntot = a.nt * a.nparts, tiles = a.mt * ntot, all = a.kst * a.kparts * a.kplanes;
  r.sp = 0;
  r.ks0 = 0;
  r.ks1 = (int)all;
  unsigned t = it;
  if (a.splits > 1) {
    r.sp = (int)(t / tiles);
    t -= r.sp * tiles;
    r.ks0 = (int)((unsigned long long)all * r.sp / (unsigned)a.splits);
    r.ks1 = (int)((unsigned long long)all * (r.sp + 1) / (unsigned)a.splits);
  }
  const unsigned g = t / (GROUP * ntot), first = g * GROUP;
  const unsigned gm = min((unsigned)GROUP, a.mt - first);
  const unsigned q = t - g * GROUP * ntot;
  const unsigned n = gm == GROUP ? q / GROUP : q / gm;
  r.m0 = (int)(first + q - n * gm) * (2 * BM);
  r.part = a.nparts > 1 ? (int)(n / a.nt) : 0;
  r.n0 = (int)(n - r.part * a.nt) * TN;
  return r;
}

// sixteen consecutive 16-byte pieces' worth of a lane's row: 32 fp32 values
template <bool ADD = false>
__device__ __forceinline__ void store_f32(float* tile, size_t ld, int first, int rows, int cols,
                                          const float (&v)[32], bool add = false) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint4 c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      c[i] = make_uint4(__float_as_uint(v[16 * h + 4 * i]), __float_as_uint(v[16 * h + 4 * i + 1]),
                        __float_as_uint(v[16 * h + 4 * i + 2]), __float_as_uint(v[16 * h + 4 * i + 3]));
    wtc::store_rows<ADD>(tile + 16 * h, 4 * ld, first, rows, (cols - 16 * h + 3) / 4, c, add);
  }
}
// 32 values of a lane's row as bf16
__device__ __forceinline__ void store_bf16(__nv_bfloat16* tile, size_t ld, int first, int rows, int cols,
                                           const uint32_t (&w)[16]) {
  uint4 c[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) c[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
  wtc::store_rows(tile, 2 * ld, first, rows, (cols + 7) / 8, c);
}
// N (16 or 32) fp32 values of a lane's row as their three planes
template <int N>
__device__ __forceinline__ void store_planes(__nv_bfloat16* tile, size_t ld, size_t plane, int first,
                                             int rows, int cols, const float (&v)[N]) {
  uint32_t w[N / 2][3];
#pragma unroll
  for (int i = 0; i < N / 2; ++i) split3_bf16x2(v[2 * i], v[2 * i + 1], w[i]);
#pragma unroll
  for (int p = 0; p < 3; ++p) {
    uint4 c[4];
#pragma unroll
    for (int i = 0; i < N / 8; ++i)
      c[i] = make_uint4(w[4 * i][p], w[4 * i + 1][p], w[4 * i + 2][p], w[4 * i + 3][p]);
#pragma unroll
    for (int i = N / 8; i < 4; ++i) c[i] = make_uint4(0, 0, 0, 0);
    wtc::store_rows(tile + p * plane, 2 * ld, first, rows, min((cols + 7) / 8, N / 8), c);
  }
}

// the power of two 2^e by which a block row's largest finite value falls into [2^14, 2^15)
__device__ __forceinline__ int row_exponent(float m) {
  const int e = (int)(__float_as_uint(m) >> 23) - 127 - 14;
  return max(e, -126);
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// p and q of a lane's row into a block
template <bool F32>
__device__ __forceinline__ void keep(const MlpKept& k, size_t block, const float (&p)[16],
                                     const float (&q)[16]) {
  const int lane = threadIdx.x & 31;
  if constexpr (F32) {
    uint4* o = reinterpret_cast<uint4*>(k.pq) + block * 8 * 32 + lane;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[i * 32] = make_uint4(__float_as_uint(p[4 * i]), __float_as_uint(p[4 * i + 1]),
                             __float_as_uint(p[4 * i + 2]), __float_as_uint(p[4 * i + 3]));
      o[(4 + i) * 32] = make_uint4(__float_as_uint(q[4 * i]), __float_as_uint(q[4 * i + 1]),
                                   __float_as_uint(q[4 * i + 2]), __float_as_uint(q[4 * i + 3]));
    }
  } else {
    uint4* o = reinterpret_cast<uint4*>(k.pq) + block * 4 * 32 + lane;
    uint32_t word = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float(&v)[16] = h ? q : p;
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 16; i += 2) m = fmaxf(fmaxf(m, fabsf(v[i])), fabsf(v[i + 1]));
      if (m > 3.4e38f) {               // infinities stay themselves: the largest of the others
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) m = fmaxf(m, fabsf(v[i]) <= 3.4e38f ? fabsf(v[i]) : 0.f);
      }
      const int e = row_exponent(m);
      const f32x2 f = pack2(pow2(-e), pow2(-e));
      word |= (uint32_t)(e + 128) << (8 * h);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t w[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 y = unpack2(wtc::mul2(pack2(v[8 * i + 2 * j], v[8 * i + 2 * j + 1]), f));
          const __half2 x = __floats2half2_rn(y.x, y.y);
          w[j] = *reinterpret_cast<const uint32_t*>(&x);
        }
        o[(2 * h + i) * 32] = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
    k.scale[block * 32 + lane] = (uint16_t)word;
  }
}
// p and q of a lane's row as they are kept (bf16 calls)
struct Kept {
  uint4 w[4];
  uint32_t scale;
};
__device__ __forceinline__ void fetch(const MlpKept& k, size_t block, Kept& r) {
  const int lane = threadIdx.x & 31;
  const uint4* o = reinterpret_cast<const uint4*>(k.pq) + block * 4 * 32 + lane;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = o[i * 32];
  r.scale = k.scale[block * 32 + lane];
}
// what the rounding of a pair left (h: the pair as bf16); infinities leave nothing
__device__ __forceinline__ uint32_t rest_of(float a, float b, uint32_t h) {
  uint32_t r = wtc::pack_rest(a, b, h);
  if ((h & 0x7f80u) == 0x7f80u) r &= 0xffff0000u;
  if ((h & 0x7f800000u) == 0x7f800000u) r &= 0x0000ffffu;
  return r;
}
// p (h = 0) or q (h = 1), times x, as bf16 pairs, and (TWO) what their rounding left
template <bool TWO>
__device__ __forceinline__ void times_kept(const Kept& k, int h, const uint32_t (&x)[16], uint32_t* out,
                                           uint32_t* rest) {
  const float s = pow2((int)((k.scale >> (8 * h)) & 0xff) - 128);
  const f32x2 f = pack2(s, s);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const uint4 c = k.w[2 * h + i];
    const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int e = 8 * i + 2 * j;
      const float2 y = __half22float2(*reinterpret_cast<const __half2*>(&w[j]));
      const float2 z = unpack2(wtc::mul2(wtc::mul2(pack2(y.x, y.y), f),
                                         pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1]))));
      out[4 * i + j] = wtc::pack(z.x, z.y);
      if (TWO) rest[4 * i + j] = rest_of(z.x, z.y, out[4 * i + j]);
    }
  }
}
// p (h = 0) or q (h = 1) of a lane's row, fp32 calls
__device__ __forceinline__ void kept_f32(const MlpKept& k, size_t block, int h, float (&v)[16]) {
  const uint4* o = reinterpret_cast<const uint4*>(k.pq) + (block * 2 + h) * 4 * 32 + (threadIdx.x & 31);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint4 w = o[i * 32];
    v[4 * i] = __uint_as_float(w.x);
    v[4 * i + 1] = __uint_as_float(w.y);
    v[4 * i + 2] = __uint_as_float(w.z);
    v[4 * i + 3] = __uint_as_float(w.w);
  }
}

// g becomes p, u becomes q, h = p u
template <bool F32, int KIND>
__device__ __forceinline__ void gate(float (&g)[16], float (&u)[16], float (&h)[16]) {
  if constexpr (!F32 && KIND == kActSilu) {
    const f32x2 one = pack2(1.f, 1.f), minus = pack2(-1.f, -1.f), l2e = pack2(-1.4426950408889634f, -1.4426950408889634f);
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const f32x2 g2 = pack2(g[i], g[i + 1]), u2 = pack2(u[i], u[i + 1]);
      float2 e = unpack2(wtc::mul2(g2, l2e));
      asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.x));
      asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(e.y));
      e = unpack2(wtc::add2(pack2(e.x, e.y), one));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.x));
      asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(e.y));
      const f32x2 s = pack2(e.x, e.y), p = wtc::mul2(g2, s);
      const float2 hh = unpack2(wtc::mul2(p, u2)), pp = unpack2(p);
      const float2 qq = unpack2(wtc::mul2(u2, fma2(p, fma2(s, minus, one), s)));
      h[i] = hh.x; h[i + 1] = hh.y;
      g[i] = pp.x; g[i + 1] = pp.y;
      u[i] = qq.x; u[i + 1] = qq.y;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      float p, s;
      mlp_act<F32, KIND>(g[i], p, s);
      h[i] = p * u[i];
      g[i] = p;
      u[i] *= s;
    }
  }
}
template <bool F32>
__device__ __forceinline__ void gate(int act, float (&g)[16], float (&u)[16], float (&h)[16]) {
  if (act == kActSilu)
    gate<F32, kActSilu>(g, u, h);
  else if (act == kActGelu)
    gate<F32, kActGelu>(g, u, h);
  else
    gate<F32, kActGeluTanh>(g, u, h);
}

// 16 columns of this lane's row, not waited for
__device__ __forceinline__ void ld16(uint32_t taddr, uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15}, [%16];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15])
      : "r"(taddr));
}
// the registers as operands keep their uses behind the wait
__device__ __forceinline__ void wait16(uint32_t (&v)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15])::"memory");
}

// 32 columns of this lane's row; `first`: the warp's first row in the tile, rows: of the
// tile that are in M, m0: the CTA's first row
template <bool F32>
__device__ __forceinline__ void out_rows(const MlpGemmArgs& a, int part, int m0, int n, int first,
                                         int rows, const float* bias, float (&v)[32]) {
  using T = typename std::conditional<F32, float, __nv_bfloat16>::type;
  if (bias)
#pragma unroll
    for (int i = 0; i < 32; ++i) v[i] += bias[i];
  T* tile = (T*)a.out + (size_t)m0 * a.ldo + part * a.part_out + n;
  if (a.wide) {
    if constexpr (F32) {
      store_f32(tile, a.ldo, first, rows, min(32, a.N - n), v);
    } else {
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = wtc::pack(v[2 * i], v[2 * i + 1]);
      store_bf16(tile, a.ldo, first, rows, min(32, a.N - n), w);
    }
    return;
  }
  // rows that are no whole 16-byte pieces: the warp's 32 x 32 values turned, so that its
  // lanes write one row side by side (each writing its own row took 426 us of a gradient of
  // 15128 x 3782, 80 so)
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 16; x > 0; x >>= 1)
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (!(i & x)) {
        const bool upper = lane & x;
        const float got = __shfl_xor_sync(0xffffffffu, upper ? v[i] : v[i | x], x);
        (upper ? v[i] : v[i | x]) = got;
      }
  if (n + lane < a.N) {
    T* o = tile + (size_t)first * a.ldo + lane;
#pragma unroll
    for (int i = 0; i < 32; ++i)
      if (first + i < rows) {
        if constexpr (F32)
          o[i * a.ldo] = v[i];
        else
          o[i * a.ldo] = __float2bfloat16_rn(v[i]);
      }
  }
  __syncwarp();
}

// LONG: bf16 products into rows or partial sums whose ranges are longer than an accumulator's
template <bool F32, int EPI, bool TWO, bool LONG>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(threads_of(EPI), 1)
    k_mlp_gemm(const __grid_constant__ Maps mp, MlpGemmArgs a) {
  using G = Cfg<F32>;
  constexpr int NST = G::NST, BN = G::BN, BNC = G::BNC, TN = EPI == kMlpGlu ? BNC : BN;
  constexpr int PLANES = G::PLANES, KCH = F32 || LONG ? G::KCH : 1 << 30, EPW = epilogue_warps(EPI);
  static_assert(!LONG || (!F32 && (EPI == kMlpRows || EPI == kMlpPart)), "");
  extern __shared__ uint8_t sm_raw[];
  __shared__ __align__(8) uint64_t full[NST];   // leader: both CTAs' copies landed
  __shared__ __align__(8) uint64_t empty[NST];  // a slot's products done
  __shared__ __align__(8) uint64_t accf[2];     // an accumulator's products done
  __shared__ __align__(8) uint64_t acce[2];     // leader: read out by both CTAs' warps
  __shared__ uint32_t tmem_s;
  __shared__ int issued_s[2], consumed_s, bad_s;
  __shared__ float bias_s[2][BN];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = rank_of_cta();
  const uint32_t sm = (tc::smem_u32(sm_raw) + 1023u) & ~1023u;
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;

  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(
                     tc::smem_u32(&tmem_s)),
                 "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < NST; ++i) {
      tc::mbar_init(tc::smem_u32(&full[i]), 2);
      tc::mbar_init(tc::smem_u32(&empty[i]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(tc::smem_u32(&accf[i]), 1);
      tc::mbar_init(tc::smem_u32(&acce[i]), 2 * EPW);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    issued_s[0] = issued_s[1] = 0;
    consumed_s = 0;
    bad_s = 0;
  }
  tc::fence_before();
  __syncthreads();
  cluster_sync();      // the partner's barriers and tensor memory are there too
  tc::fence_after();
  const uint32_t tmem = tmem_s;

  if (warp == 0 || warp == 2) {
    // ---------------- copies: of A by warp 0, of B by warp 2 ----------------
    if (wtc::elect_one()) {
      const bool is_a = warp == 0;
      const CUtensorMap* map = is_a ? &mp.a : &mp.b;
      const bool mn = is_a ? a.amn : a.bmn, two = is_a ? a.two_a : a.two_b;
      const int boxes = mn ? (is_a ? BM : BNC) / 64 : 1;
      const uint32_t bytes = 2 * (is_a ? G::A_BYTES : G::B_BYTES), sm0 = sm + (is_a ? 0 : G::A_BYTES);
      const uint32_t empty0 = tc::smem_u32(&empty[0]), full0 = tc::smem_u32(&full[0]);
      const uint32_t lead0 = at_leader(full0);
      int st = 0, issued = 0;
      uint32_t ph = 0;
      bool bad = false;
      for (int it = pair; it < a.items && !bad; it += pairs) {
        const Item r = decode<TN>(a, it);
        // first row of this CTA, and the operand's part where K does not run over parts
        const int row = is_a ? r.m0 + (int)rank * BM : (EPI == kMlpGlu ? r.n0 : r.n0 + (int)rank * BNC);
        const int part = is_a ? 0 : (EPI == kMlpGlu ? (int)rank : r.part);
        // K step: plane, part of K, k (divisions once a tile: one a step took a sixth of the
        // whole product of dx)
        int pl = 0, kp = 0, kt = r.ks0;
        if (a.kplanes > 1 && kt >= a.kst * a.kparts) {
          pl = 1;
          kt -= a.kst * a.kparts;
        }
        if (a.kparts > 1 && kt >= a.kst) {
          kp = 1;
          kt -= a.kst;
        }
        for (int ks = r.ks0; ks < r.ks1 && !bad; ++ks) {
          const int k0 = kt * BK, pp = a.kparts > 1 ? kp : part;
#pragma unroll 1
          for (int p = 0; p < PLANES; ++p) {
            const int plane = F32 ? p : (two ? pl : 0);
            if (!wtc::wait_or_flag(a.err, empty0 + 8 * st, ph ^ 1u)) { bad = true; break; }
            if (rank == 0) tc::mbar_expect_tx(full0 + 8 * st, bytes);
            const uint32_t dst = sm0 + st * G::SLOT, bar = lead0 + 8 * st;
            if (mn) {
#pragma unroll
              for (int i = 0; i < BM / 64; ++i)
                if (i < boxes) tma4(dst + i * BLK64, map, row + 64 * i, pp, k0, plane, bar);
            } else {
              tma4(dst, map, k0, pp, row, plane, bar);
            }
            ++issued;
            if (++st == NST) { st = 0; ph ^= 1u; }
          }
          if (++kt == a.kst) {
            kt = 0;
            if (++kp == a.kparts) {
              kp = 0;
              ++pl;
            }
          }
        }
      }
      // the products of the last slots are done in both CTAs: their arrivals here come
      // before this CTA ends
      for (int i = 0; i < NST && i < issued && !bad; ++i) {
        const int k = issued - 1 - i;
        bad = !wtc::wait_or_flag(a.err, empty0 + 8 * (k % NST), (uint32_t)(k / NST) & 1u);
      }
      issued_s[is_a ? 0 : 1] = issued;
      if (bad) atomicOr(&bad_s, 1);
    }
  } else if (warp == 1) {
    // ---------------- products, of the leader ----------------
    if (rank == 0 && wtc::elect_one()) {
      int st = 0, consumed = 0;
      uint32_t ph = 0, u = 0;           // u: accumulators used so far
      int si = 0;                       // F32: accumulators of the smaller products
      bool bad = false;
      const uint32_t id = tc::idesc_bf16(2 * BM, BN) | (a.amn ? 1u << 15 : 0u) | (a.bmn ? 1u << 16 : 0u);
      // K slices of 16: 32 bytes on in a K-major row, 16 rows on in an MN-major block
      const uint64_t sta = (a.amn ? 2048 : 32) >> 4, stb = (a.bmn ? 2048 : 32) >> 4;
      const uint64_t da0 = a.amn ? wtc::desc_mn(sm, BLK64) : wtc::desc_k(sm);
      const uint64_t db0 = a.bmn ? wtc::desc_mn(sm + G::A_BYTES, BLK64) : wtc::desc_k(sm + G::A_BYTES);
      for (int it = pair; it < a.items && !bad; it += pairs, ++si) {
        const Item r = decode<TN>(a, it);
        int ks1 = r.ks0;                // F32: first step of the smaller products' accumulator
        for (int k0 = r.ks0; k0 < r.ks1 && !bad; k0 += KCH < r.ks1 - k0 ? KCH : r.ks1 - k0, ++u) {
          const int k1 = KCH < r.ks1 - k0 ? k0 + KCH : r.ks1;
          const int acc = (int)(u & 1);
          if (!wtc::wait_or_flag(a.err, tc::smem_u32(&acce[acc]), ((u >> 1) & 1u) ^ 1u)) { bad = true; break; }
          tc::fence_after();
          const uint32_t d = tmem + (uint32_t)(acc * BN);
          // (the one before last is read out with a chunk that was released before this one)
          if (F32 && k0 - ks1 == G::KSM) {
            ks1 = k0;
            ++si;
          }
          const uint32_t small = tmem + 256 + (uint32_t)(si & 1) * 128;   // F32
          for (int ks = k0; ks < k1; ++ks) {
            uint64_t da[PLANES], db[PLANES];
            int at[PLANES];
            // planes as they come: all products of the planes that are there
#pragma unroll
            for (int p = 0; p < PLANES; ++p) {
              if (!wtc::wait_or_flag(a.err, tc::smem_u32(&full[st]), ph)) { bad = true; break; }
              tc::fence_after();
              at[p] = st;
              da[p] = da0 + (uint64_t)((uint32_t)st * G::SLOT >> 4);
              db[p] = db0 + (uint64_t)((uint32_t)st * G::SLOT >> 4);
              if (p == 0) {
#pragma unroll
                for (int k = 0; k < BK / 16; ++k)
                  mma2(d, da[0] + k * sta, db[0] + k * stb, id, ks > k0 || k > 0);
              } else if (p == 1) {
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                  mma2(small, da[0] + k * sta, db[1 % PLANES] + k * stb, id, ks > ks1 || k > 0);
                  mma2(small, da[1 % PLANES] + k * sta, db[0] + k * stb, id, 1);
                  mma2(small, da[1 % PLANES] + k * sta, db[1 % PLANES] + k * stb, id, 1);
                }
              } else {
#pragma unroll
                for (int k = 0; k < BK / 16; ++k) {
                  mma2(small, da[0] + k * sta, db[2 % PLANES] + k * stb, id, 1);
                  mma2(small, da[2 % PLANES] + k * sta, db[0] + k * stb, id, 1);
                }
              }
              ++consumed;
              if (++st == NST) { st = 0; ph ^= 1u; }
            }
            if (bad) break;
#pragma unroll
            for (int p = 0; p < PLANES; ++p) commit2(tc::smem_u32(&empty[at[p]]));
          }
          if (bad) break;
          commit2(tc::smem_u32(&accf[acc]));
        }
      }
      consumed_s = consumed;
      if (bad) atomicOr(&bad_s, 1);
    }
  } else if (warp >= 4) {
    // ---------------- accumulators ----------------
    const int et = tid - 128, q = warp & 3, sub = (warp - 4) >> 2;
    const uint32_t lanes = (uint32_t)(32 * q) << 16;
    const uint32_t acce0 = at_leader(tc::smem_u32(&acce[0])), acce1 = at_leader(tc::smem_u32(&acce[1]));
    // this warp's columns of a tile (glu: of the gate's, and BNC on those of the other half)
    constexpr int COLS = TN / (EPW / 4);
    const int col0 = sub * COLS;
    uint32_t u = 0;
    int li = 0, si = 0;
    bool bad = false;
    // dglu of bf16 calls: p and q of DEEP blocks, each fetched again for DEEP blocks later
    // as soon as it is used (131072 rows of 1408: 278 us, 5.8 TB/s; read when they were needed,
    // a tile's waits for memory took longer than its products: 491 us)
    constexpr int DEEP = 2;
    Kept kept2[DEEP];
    auto ahead = [&](int tile_m, int n, Kept& k) {
      const int m = tile_m + (int)rank * BM + 32 * q;
      if (m < a.M && n < a.N) fetch(a.kept, (size_t)(m / 32) * a.fblocks + n / 16, k);
    };
    if constexpr (!F32 && EPI == kMlpDglu)
      if (pair < a.items) {
        const Item r = decode<TN>(a, pair);
#pragma unroll
        for (int i = 0; i < DEEP; ++i) ahead(r.m0, r.n0 + col0 + 16 * i, kept2[i]);
      }
    const bool biased = (EPI == kMlpRows || EPI == kMlpGlu) && a.bias != nullptr;
    for (int it = pair; it < a.items && (biased || !bad); it += pairs, ++li, ++si) {
      const Item r = decode<TN>(a, it);
      const int m0 = r.m0 + (int)rank * BM, rows = min(BM, a.M - m0);
      const float* bias = nullptr;
      if (biased) {
        float* bs = bias_s[li & 1];     // the other one may still be read
        if (et < BN) {
          const int half = EPI == kMlpGlu ? et / BNC : r.part, n = r.n0 + (EPI == kMlpGlu ? et % BNC : et);
          const size_t i = (size_t)half * a.N + n;
          bs[et] = n >= a.N ? 0.f : F32 ? ((const float*)a.bias)[i]
                                        : __bfloat162float(((const __nv_bfloat16*)a.bias)[i]);
        }
        // all warps go on, or none
        if (epilogue_any<32 * EPW>(bad)) {
          bad = true;
          break;
        }
        bias = bs;
      }
      const size_t block0 = (size_t)((m0 + 32 * q) / 32) * a.fblocks;   // of p and q
      const bool some = 32 * q < rows;
      // 32 columns of rows or partial sums (add: to those of the chunks before)
      auto plain = [&](int col, float(&v)[32], bool add) {
        const int n = r.n0 + col;
        if (n >= a.N || !some) return;
        if constexpr (EPI == kMlpPart) {
          float* tile = (float*)a.out + ((size_t)r.sp * a.M + m0) * a.ldo + r.part * a.part_out + n;
          store_f32<LONG>(tile, a.ldo, 32 * q, rows, min(32, (a.N - n + 3) & ~3), v, add);
        } else {
          out_rows<F32>(a, r.part, m0, n, 32 * q, rows, bias ? bias + col : nullptr, v);
        }
      };
      // 16 of the gate and of the other half
      auto gated = [&](int col, float(&g)[16], float(&v)[16], float(&h)[16]) {
        if (bias)
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            g[i] += bias[col + i];
            v[i] += bias[BNC + col + i];
          }
        gate<F32>(a.act, g, v, h);
        if (a.kept.pq && some && r.n0 + col < a.N) keep<F32>(a.kept, block0 + (r.n0 + col) / 16, g, v);
      };
      constexpr int NR = EPI == kMlpGlu ? 2 : COLS / 16;
      constexpr bool SUMS = F32 || (LONG && EPI == kMlpRows);
      float R[SUMS ? NR : 1][16];      // the sums so far
      for (int k0 = r.ks0; k0 < r.ks1 && !bad; k0 += KCH < r.ks1 - k0 ? KCH : r.ks1 - k0, ++u) {
        const int acc = (int)(u & 1);
        __syncwarp();
        if (!wtc::wait_warp(a.err, tc::smem_u32(&accf[acc]), (u >> 1) & 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
        const uint32_t d = tmem + lanes + (uint32_t)(acc * BN + col0);
        auto release = [&]() {
          tc::fence_before();
          __syncwarp();
          if (lane == 0) arrive_leader(acc ? acce1 : acce0);
        };
        if constexpr (SUMS) {
          // F32: whether the smaller products' accumulator ends here
          const bool end = F32 && (k0 + KCH >= r.ks1 || (k0 + KCH - r.ks0) % G::KSM == 0);
          const uint32_t sd = tmem + lanes + 256 + (uint32_t)((si & 1) * 128 + col0);
          if (end && k0 + KCH < r.ks1) ++si;
          constexpr uint32_t OTHER = EPI == kMlpGlu ? BNC : 16;
#pragma unroll
          for (int j = 0; j < NR; ++j) {
            uint32_t x[16];
            ld16(d + j * OTHER, x);
            wait16(x);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              R[j][i] = k0 == r.ks0 ? __uint_as_float(x[i]) : R[j][i] + __uint_as_float(x[i]);
            if (end) {
              ld16(sd + j * OTHER, x);
              wait16(x);
#pragma unroll
              for (int i = 0; i < 16; ++i) R[j][i] += __uint_as_float(x[i]);
            }
          }
          release();
        } else if constexpr (EPI == kMlpGlu) {
          uint32_t w[16], rest[TWO ? 16 : 1];
#pragma unroll
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t x[16], y[16];
            ld16(d + 16 * ch, x);
            ld16(d + BNC + 16 * ch, y);
            wait16(x);
            wait16(y);
            if (ch == 1) release();
            float h[16];
            gated(col0 + 16 * ch, reinterpret_cast<float(&)[16]>(x), reinterpret_cast<float(&)[16]>(y), h);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              w[8 * ch + i] = wtc::pack(h[2 * i], h[2 * i + 1]);
              if constexpr (TWO) rest[8 * ch + i] = rest_of(h[2 * i], h[2 * i + 1], w[8 * ch + i]);
            }
          }
          const int n = r.n0 + col0, cols = min(32, (a.N - n + 7) & ~7);
          if (some && n < a.N) {
            __nv_bfloat16* o = (__nv_bfloat16*)a.out + (size_t)m0 * a.ldo + n;
            store_bf16(o, a.ldo, 32 * q, rows, cols, w);
            if constexpr (TWO) store_bf16(o + a.plane_out, a.ldo, 32 * q, rows, cols, rest);
          }
        } else if constexpr (EPI == kMlpDglu) {
          const bool more = it + pairs < a.items;
          int after_m = 0, after_n = 0;
          if (more) {
            const Item after = decode<TN>(a, it + pairs);
            after_m = after.m0;
            after_n = after.n0 + col0;
          }
#pragma unroll 1
          for (int c0 = 0; c0 < COLS; c0 += 16 * DEEP) {
            uint32_t dg[16], du[16], rg[TWO ? 16 : 1], ru[TWO ? 16 : 1];
#pragma unroll
            for (int j = 0; j < DEEP; ++j) {
              const int c = c0 + 16 * j;
              uint32_t x[16];
              ld16(d + c, x);
              wait16(x);
              if (j == DEEP - 1 && c == COLS - 16) release();
              const int o8 = 8 * (j & 1);
              times_kept<TWO>(kept2[j], 1, x, dg + o8, rg + (TWO ? o8 : 0));    // dg = dh q, du = dh p
              times_kept<TWO>(kept2[j], 0, x, du + o8, ru + (TWO ? o8 : 0));
              const bool here = c + 16 * DEEP < COLS;
              if (here || more)
                ahead(here ? r.m0 : after_m, here ? r.n0 + col0 + c + 16 * DEEP : after_n + 16 * j, kept2[j]);
              const int n = r.n0 + col0 + c - 16;
              if ((j & 1) && some && n < a.N) {
                __nv_bfloat16* o = (__nv_bfloat16*)a.out + (size_t)m0 * a.ldo + n;
                const int cols = min(32, (a.N - n + 7) & ~7);
                store_bf16(o, a.ldo, 32 * q, rows, cols, dg);
                store_bf16(o + a.part_out, a.ldo, 32 * q, rows, cols, du);
                if constexpr (TWO) {
                  store_bf16(o + a.plane_out, a.ldo, 32 * q, rows, cols, rg);
                  store_bf16(o + a.plane_out + a.part_out, a.ldo, 32 * q, rows, cols, ru);
                }
              }
            }
          }
        } else {
#pragma unroll 1
          for (int ch = 0; ch < COLS / 32; ++ch) {
            uint32_t x[32];
            wtc::ld32(d + 32 * ch, x);
            wtc::ld_wait(x);
            if (ch == COLS / 32 - 1) release();
            plain(col0 + 32 * ch, reinterpret_cast<float(&)[32]>(x), k0 > r.ks0);
          }
        }
      }
      if constexpr (SUMS && LONG) {
        if (bad) continue;
#pragma unroll
        for (int j = 0; j < NR / 2; ++j) plain(col0 + 32 * j, reinterpret_cast<float(&)[32]>(R[2 * j]), false);
      } else if constexpr (F32) {
        if (bad) continue;
        const int n = r.n0 + col0;
        __nv_bfloat16* o = (__nv_bfloat16*)a.out + (size_t)m0 * a.ldo + n;
        const int cols = (a.N - n + 7) & ~7;
        if constexpr (EPI == kMlpGlu) {
          float h[16];
          gated(col0, R[0], R[1], h);
          if (some && n < a.N) store_planes(o, a.ldo, a.plane_out, 32 * q, rows, cols, h);
        } else if constexpr (EPI == kMlpDglu) {
#pragma unroll
          for (int j = 0; j < NR; ++j)
            if (some && n + 16 * j < a.N)
#pragma unroll
              for (int h = 1; h >= 0; --h) {
                float w[16];
                kept_f32(a.kept, block0 + n / 16 + j, h, w);
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] *= R[j][i];
                store_planes((h ? o : o + a.part_out) + 16 * j, a.ldo, a.plane_out, 32 * q, rows,
                             cols - 16 * j, w);
              }
        } else {
          plain(col0, reinterpret_cast<float(&)[32]>(R), false);
        }
      }
    }
    if (bad) atomicOr(&bad_s, 1);
  }

  // ---- drain and free the tensor memory ----
  // On a healthy run every copy and every product has been waited for.  After an expired
  // wait: the last products (their commit covers all earlier ones), then the copies that
  // were issued and not consumed.
  __syncthreads();
  if (bad_s && rank == 0 && tid == 32) {
    const int c = consumed_s, n = max(issued_s[0], issued_s[1]);
    if (c > 0) wtc::wait_or_flag(a.err, tc::smem_u32(&empty[(c - 1) % NST]), (uint32_t)((c - 1) / NST) & 1u);
    for (int k = c; k < n; ++k) wtc::wait_or_flag(a.err, tc::smem_u32(&full[k % NST]), (uint32_t)(k / NST) & 1u);
  }
  tc::fence_before();
  __syncthreads();
  cluster_sync();
  tc::fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
}

// sums of the ranges in order, + bias, four columns a thread where they are whole
template <typename T>
__global__ void __launch_bounds__(256) k_mlp_reduce(MlpReduceArgs a, int quads) {
  const long long id = (long long)blockIdx.x * 256 + threadIdx.x;
  const long long per = (long long)a.nparts * quads;
  const long long m = id / per;
  if (m >= a.M) return;
  const int q = (int)(id - m * per), part = q / quads, n = (q - part * quads) * 4;
  const float* src = a.part + m * a.ldp + part * a.part_in + n;
  float4 s = *reinterpret_cast<const float4*>(src);
  for (int i = 1; i < a.splits; ++i) {
    const float4 v = *reinterpret_cast<const float4*>(src + i * a.split_stride);
    s.x += v.x; s.y += v.y; s.z += v.z; s.w += v.w;
  }
  float v[4] = {s.x, s.y, s.z, s.w};
  T* o = (T*)a.out + m * a.ldo + part * a.part_out + n;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < a.N) {
      const size_t b = (size_t)part * a.N + n + i;
      if constexpr (sizeof(T) == 4) {
        if (a.bias) v[i] += ((const float*)a.bias)[b];
      } else {
        if (a.bias) v[i] += __bfloat162float(((const __nv_bfloat16*)a.bias)[b]);
      }
    }
  if (n + 4 <= a.N && ((uintptr_t)o & (4 * sizeof(T) - 1)) == 0) {
    st4(o, make_float4(v[0], v[1], v[2], v[3]));
    return;
  }
  for (int i = 0; i < 4 && n + i < a.N; ++i) {
    if constexpr (sizeof(T) == 4)
      o[i] = v[i];
    else
      o[i] = __float2bfloat16_rn(v[i]);
  }
}

template <bool F32>
__global__ void __launch_bounds__(256) k_mlp_pack(MlpPackArgs a) {
  int j = 0;
  while (j + 1 < a.jobs && (long long)blockIdx.x >= a.first[j + 1]) ++j;
  const MlpPackJob& b = a.job[j];
  // eight columns of a row a thread, of the padded row
  const long long id = ((long long)blockIdx.x - a.first[j]) * 256 + threadIdx.x;
  const int per = b.ld / 8;
  const long long row = id / per;
  if (row >= b.rows) return;
  const int c = (int)(id - row * per) * 8;
  __nv_bfloat16* o = b.dst + row * b.ld + c;
  const long long at = row * b.inner + c;
  if constexpr (F32) {
    const float* s = (const float*)b.src + at;
    float v[8];
    if (c + 8 <= b.inner && ((uintptr_t)s & 15) == 0) {
      const float4 x = ld4(s), y = ld4(s + 4);
      v[0] = x.x; v[1] = x.y; v[2] = x.z; v[3] = x.w;
      v[4] = y.x; v[5] = y.y; v[6] = y.z; v[7] = y.w;
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = c + i < b.inner ? s[i] : 0.f;
    }
    uint32_t w[4][3];
#pragma unroll
    for (int i = 0; i < 4; ++i) split3_bf16x2(v[2 * i], v[2 * i + 1], w[i]);
#pragma unroll
    for (int p = 0; p < 3; ++p)
      *reinterpret_cast<uint4*>(o + p * b.rows * b.ld) = make_uint4(w[0][p], w[1][p], w[2][p], w[3][p]);
  } else {
    const __nv_bfloat16* s = (const __nv_bfloat16*)b.src + at;
    __align__(16) __nv_bfloat16 v[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = c + i < b.inner ? s[i] : __nv_bfloat16(0.f);
    *reinterpret_cast<uint4*>(o) = *reinterpret_cast<const uint4*>(v);
  }
}

// rows of range blockIdx.y, 32 columns of blockIdx.x: row y, y + 8, .. by thread y
__global__ void __launch_bounds__(256) k_mlp_colsum(MlpColsumArgs a) {
  __shared__ float s[8][33];
  const int cols = a.parts * a.inner, c = blockIdx.x * 32 + threadIdx.x;
  const int r0 = (int)((long long)a.rows * blockIdx.y / a.ranges);
  const int r1 = (int)((long long)a.rows * (blockIdx.y + 1) / a.ranges);
  float t = 0.f;
  if (c < cols) {
    const int part = c / a.inner;
    const size_t at = (size_t)part * a.pstride + (c - part * a.inner);
#pragma unroll 4
    for (int r = r0 + threadIdx.y; r < r1; r += 8) {
      const size_t i = r * a.ld + at;
      if (a.planes == 0) {
        t += ((const float*)a.src)[i];
      } else {
        const __nv_bfloat16* p = (const __nv_bfloat16*)a.src + i;
        float v = __bfloat162float(p[0]);
        for (int k = 1; k < a.planes; ++k) v += __bfloat162float(p[k * a.plane_stride]);
        t += v;
      }
    }
  }
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    for (int y = 1; y < 8; ++y) t += s[y][threadIdx.x];
    a.part[(size_t)blockIdx.y * cols + c] = t;
  }
}
template <typename T>
__global__ void __launch_bounds__(256) k_mlp_colsum_join(MlpColsumArgs a) {
  __shared__ float s[8][33];
  const int cols = a.parts * a.inner, c = blockIdx.x * 32 + threadIdx.x;
  float t = 0.f;
  if (c < cols)
#pragma unroll 4
    for (int r = threadIdx.y; r < a.ranges; r += 8) t += a.part[(size_t)r * cols + c];
  s[threadIdx.y][threadIdx.x] = t;
  __syncthreads();
  if (threadIdx.y == 0 && c < cols) {
    for (int y = 1; y < 8; ++y) t += s[y][threadIdx.x];
    if constexpr (sizeof(T) == 4)
      ((T*)a.out)[c] = t;
    else
      ((T*)a.out)[c] = __float2bfloat16_rn(t);
  }
}

bool map_view(CUtensorMap* t, const MlpView& v, int box_rows) {
  const cuuint64_t dim[4] = {(cuuint64_t)v.inner, (cuuint64_t)v.parts, (cuuint64_t)v.rows,
                             (cuuint64_t)v.planes};
  const cuuint64_t stride[3] = {(cuuint64_t)v.part_stride * 2, (cuuint64_t)v.row_stride * 2,
                                (cuuint64_t)v.plane_stride * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)box_rows, 1};
  return encode_tiled_bf16_sw128(t, 4, v.p, dim, stride, box);
}

template <bool F32, int EPI, bool TWO = false, bool LONG = false>
cudaError_t go(const char* name, const Maps& mp, const MlpGemmArgs& g, int dev, int sms, cudaStream_t st) {
  static SmemOnce once;
  const cudaError_t e = once.allow(k_mlp_gemm<F32, EPI, TWO, LONG>, Cfg<F32>::SMEM, dev);
  if (e != cudaSuccess) return e;
  const int pairs = g.items < sms / 2 ? g.items : sms / 2;
  return launch(name, k_mlp_gemm<F32, EPI, TWO, LONG>, dim3((unsigned)(2 * pairs)), dim3(threads_of(EPI)), (size_t)Cfg<F32>::SMEM,
                st, mp, g);
}

}  // namespace

int mlp_tile_n(bool f32) { return f32 ? Cfg<true>::BN : Cfg<false>::BN; }

// The ranges that take the least time, by K steps of the longest pair: a tile costs
// about four steps beside its own (its first copies and its last epilogue), a range's
// partial sums are written and read at memory's rate (a step of 64 is 0.27 us in bf16,
// 0.8 us in fp32)
int mlp_splits(long long tiles, int ksteps, double mn, bool f32) {
  const double step = f32 ? 0.8e-6 : 0.27e-6, pairs = 76;
  int best = 1;
  double least = 1e300;
  for (int s = 1; s <= 32 && (s == 1 || ksteps / s >= 4); ++s) {
    const double waves = (double)((tiles * s + (long long)pairs - 1) / (long long)pairs);
    double t = waves * ((ksteps + s - 1) / s + 4) * step;
    if (s > 1) t += 3e-6 + s * mn * 8.0 / 5e12;
    if (t < least) {
      least = t;
      best = s;
    }
  }
  return best;
}

cudaError_t run_mlp_gemm(const char* name, int epi, bool f32, bool two, const MlpView& a, const MlpView& b,
                         MlpGemmArgs& g, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  g.err = wait_error_address();
  if (g.err == nullptr) return cudaErrorInvalidSymbol;
  const int bn = mlp_tile_n(f32), tn = epi == kMlpGlu ? bn / 2 : bn;
  g.mt = (g.M + kMlpTileM - 1) / kMlpTileM;
  g.nt = (g.N + tn - 1) / tn;
  g.kst = ((g.amn ? a.rows : a.inner) + BK - 1) / BK;
  const long long items = (long long)g.mt * g.nt * g.nparts * g.splits;
  if (items >= 1LL << 30) return cudaErrorInvalidValue;   // refused before (check_mlp)
  g.items = (int)items;
  Maps mp;
  memset(&mp, 0, sizeof(mp));
  if (!map_view(&mp.a, a, g.amn ? 64 : BM) || !map_view(&mp.b, b, g.bmn ? 64 : bn / 2))
    return cudaErrorInvalidValue;
  g.two_a = !f32 && a.planes == 2;
  g.two_b = !f32 && b.planes == 2;
  g.kplanes = g.two_a || g.two_b ? 2 : 1;
  if (!f32 && two)
    return epi == kMlpGlu ? go<false, kMlpGlu, true>(name, mp, g, dev, sms, st)
                          : go<false, kMlpDglu, true>(name, mp, g, dev, sms, st);
  if (!f32 && ((long long)g.kst * g.kparts * g.kplanes + g.splits - 1) / g.splits > Cfg<false>::KCH) {
    if (epi == kMlpRows) return go<false, kMlpRows, false, true>(name, mp, g, dev, sms, st);
    if (epi == kMlpPart) return go<false, kMlpPart, false, true>(name, mp, g, dev, sms, st);
  }
#define GO(E) return f32 ? go<true, E>(name, mp, g, dev, sms, st) : go<false, E>(name, mp, g, dev, sms, st)
  switch (epi) {
    case kMlpRows: GO(kMlpRows);
    case kMlpPart: GO(kMlpPart);
    case kMlpGlu: GO(kMlpGlu);
    default: GO(kMlpDglu);
  }
#undef GO
}

cudaError_t run_mlp_reduce(const char* name, const MlpReduceArgs& a, bool bf16, cudaStream_t st) {
  const int quads = (a.N + 3) / 4;
  const long long n = (long long)a.M * a.nparts * quads;
  const dim3 grid((unsigned)((n + 255) / 256));
  if (bf16) return launch(name, k_mlp_reduce<__nv_bfloat16>, grid, dim3(256), 0, st, a, quads);
  return launch(name, k_mlp_reduce<float>, grid, dim3(256), 0, st, a, quads);
}

cudaError_t run_mlp_pack(MlpPackArgs& a, bool bf16, cudaStream_t st) {
  long long n = 0;
  for (int j = 0; j < a.jobs; ++j) {
    a.first[j] = n;
    n += (a.job[j].rows * (a.job[j].ld / 8) + 255) / 256;
  }
  if (n == 0) return cudaSuccess;
  if (n >= 1LL << 31) return cudaErrorInvalidValue;
  if (bf16) return launch("mlp_pack", k_mlp_pack<false>, dim3((unsigned)n), dim3(256), 0, st, a);
  return launch("mlp_pack", k_mlp_pack<true>, dim3((unsigned)n), dim3(256), 0, st, a);
}

// ranges of rows: blocks for four an SM, 64 rows each or more
int mlp_colsum_ranges(int rows, int cols) {
  const int cb = (cols + 31) / 32, want = (608 + cb - 1) / cb, most = (rows + 63) / 64;
  return want < most ? want : most;
}

cudaError_t run_mlp_colsum(const MlpColsumArgs& a, bool bf16, cudaStream_t st) {
  const unsigned cb = (unsigned)((a.parts * a.inner + 31) / 32);
  cudaError_t e = launch("mlp_colsum", k_mlp_colsum, dim3(cb, a.ranges), dim3(32, 8), 0, st, a);
  if (e != cudaSuccess) return e;
  if (bf16) return launch("mlp_colsum_join", k_mlp_colsum_join<__nv_bfloat16>, dim3(cb), dim3(32, 8), 0, st, a);
  return launch("mlp_colsum_join", k_mlp_colsum_join<float>, dim3(cb), dim3(32, 8), 0, st, a);
}

}  // namespace lapnys
