// What the tensor-core kernels of the windowed attention share: tiles by TMA in
// the 128-byte swizzle, products with the left operand in tensor memory, and
// loads and stores of tensor memory without a wait of their own.
//
// A tile of R rows of a [..][d] bf16 tensor is kept as panels of 64 features: R
// rows of 128 bytes each, the row's 16-byte chunks XORed with the row's index
// mod 8.  The same bytes serve as a K-major operand (contraction over features)
// and as an MN-major operand (contraction over rows).
#pragma once
#include <cuda.h>

#include "common.cuh"
#include "tc.cuh"
#include "win.cuh"

namespace lapnys {
namespace wtc {

constexpr uint32_t kSbo = 1024;      // 8 rows of 128 bytes

__device__ __forceinline__ bool wait_or_flag(int* err, uint32_t bar, uint32_t parity) {
  const bool ok = tc::mbar_wait(bar, parity);
  if (!ok) atomicOr(err, 1);
  return ok;
}
// true in one thread of the (converged) warp.  The compiler knows a branch on it
// to hold one thread and keeps what it computes there in uniform registers, which
// is where the products' and copies' descriptors have to be; behind `lane == 0` it
// moves every operand there anew
__device__ __forceinline__ bool elect_one() {
  uint32_t r;
  asm volatile(
      "{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}\n"
      : "=r"(r));
  return r != 0;
}
// wait_or_flag for a whole warp, with one answer
__device__ __forceinline__ bool wait_warp(int* err, uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, wait_or_flag(err, bar, parity));
}
__device__ __forceinline__ void arrive(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// one arrival of the whole warp (the lanes' fences come before the __syncwarp)
__device__ __forceinline__ void arrive_warp(uint32_t bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) arrive(bar);
}
__device__ __forceinline__ void tma3(uint32_t dst, const CUtensorMap* map, int c0, int c1, int c2,
                                     uint32_t mbar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(mbar)
      : "memory");
}
// operand descriptors of a panel tile (layout type 2: 128-byte swizzle); MN-major
// panels are `panel` bytes apart
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
  return tc::desc(saddr, 16, kSbo) | (2ull << 61);
}
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr, uint32_t panel) {
  return tc::desc(saddr, panel, kSbo) | (2ull << 61);
}
// instruction descriptor, bf16 x bf16 -> f32; bmn: B is MN-major
__device__ __forceinline__ uint32_t idesc(int m, int n, bool bmn) {
  return tc::idesc_bf16(m, n) | (bmn ? 1u << 16 : 0u);
}
// D (TMEM) (+)= A (TMEM, packed bf16 pairs) * B (shared)
__device__ __forceinline__ void mma_ts(uint32_t tmem_d, uint32_t tmem_a, uint64_t bdesc, uint32_t id,
                                       uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.b32 p, %4, 0;\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n" ::"r"(tmem_d),
      "r"(tmem_a), "l"(bdesc), "r"(id), "r"(accumulate)
      : "memory");
}

// Products of one tile, issued by one thread.  Consecutive 16-deep slices differ
// by a constant in the descriptors' address field (16-byte units), so the loops
// are unrolled over one base: built anew per slice, the descriptors cost more
// than the product (a prompt of 32768 tokens, heads of 128: 820 us so, 700 unrolled).
// D (+)= A B^T over d features, A and B in shared memory (panels of AR and BR rows)
template <int NP, int AR = 128, int BR = 128>
__device__ __forceinline__ void mma_features(uint32_t d_tmem, uint32_t A, uint32_t B, int ksteps,
                                             uint32_t id) {
  const uint64_t da = desc_k(A), db = desc_k(B);
#pragma unroll
  for (int k = 0; k < 4 * NP; ++k)
    if (k < ksteps)
      tc::mma_bf16(d_tmem, da + (((k >> 2) * AR * 128 + (k & 3) * 32) >> 4),
                   db + (((k >> 2) * BR * 128 + (k & 3) * 32) >> 4), id, k > 0);
}
// D (+)= A B over the `slices` 16-row slices of B, A in tensor memory: two slices
// (16 columns) every PAIR columns
template <int BR = 128, int PAIR = 16>
__device__ __forceinline__ void mma_rows(uint32_t d_tmem, uint32_t A, uint32_t B, int slices,
                                         uint32_t id, bool acc) {
  const uint64_t db = desc_mn(B, BR * 128);
#pragma unroll
  for (int k = 0; k < BR / 16; ++k)
    if (k < slices) mma_ts(d_tmem, A + PAIR * (k >> 1) + 8 * (k & 1), db + 128 * k, id, acc || k > 0);
}

// rows [r0, w) of an NP-panel tile to zero, by the thread that issues the products
template <int NP, int ROWS = 128>
__device__ __forceinline__ void zero_rows(uint32_t tile, int r0, int w) {
#pragma unroll 1
  for (int r = r0; r < w; ++r)
#pragma unroll
    for (int e = 0; e < 8 * NP; ++e)
      asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (e >> 3) * (ROWS * 128) +
                                                                    r * 128 + (e & 7) * 16),
                   "r"(0)
                   : "memory");
  tc::fence_async_smem();
}

// 32 columns of this lane's row, not waited for: ld_wait makes them valid
__device__ __forceinline__ void ld32(uint32_t taddr, uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, "
      "%11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, "
      "%29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]),
        "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]),
        "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(taddr));
}
// the registers as operands keep their uses behind the wait
__device__ __forceinline__ void ld_wait(uint32_t (&v)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]),
                 "+r"(v[7]), "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]),
                 "+r"(v[13]), "+r"(v[14]), "+r"(v[15]), "+r"(v[16]), "+r"(v[17]), "+r"(v[18]),
                 "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]), "+r"(v[23]), "+r"(v[24]),
                 "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]), "+r"(v[30]),
                 "+r"(v[31])::"memory");
}
__device__ __forceinline__ void st32(uint32_t taddr, const uint32_t (&v)[32]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, "
      "%28, %29, %30, %31};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]),
      "r"(v[16]), "r"(v[17]), "r"(v[18]), "r"(v[19]), "r"(v[20]), "r"(v[21]), "r"(v[22]),
      "r"(v[23]), "r"(v[24]), "r"(v[25]), "r"(v[26]), "r"(v[27]), "r"(v[28]), "r"(v[29]),
      "r"(v[30]), "r"(v[31]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st16(uint32_t taddr, const uint32_t* v) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, "
      "%10, %11, %12, %13, %14, %15};" ::"r"(v[0]),
      "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
      "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15]), "r"(taddr)
      : "memory");
}
__device__ __forceinline__ void st_wait() {
  asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ f32x2 add2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f32x2 mul2(f32x2 a, f32x2 b) {
  f32x2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint32_t pack(float a, float b) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// what the rounding of a pair (h = pack(a, b)) leaves, rounded itself
__device__ __forceinline__ uint32_t pack_rest(float a, float b, uint32_t h) {
  float x, y;
  asm("{\n\t.reg .b16 l, u, one;\n\tmov.b32 {l, u}, %4;\n\tmov.b16 one, 0xBF80;\n\t"
      "fma.rn.f32.bf16 %0, l, one, %2;\n\tfma.rn.f32.bf16 %1, u, one, %3;\n\t}"
      : "=f"(x), "=f"(y) : "f"(a), "f"(b), "r"(h));
  return pack(x, y);
}
// Writes 16-byte pieces c of the warp's 32 rows (a row per lane, rows `first`..,
// `stride` bytes apart, only those below `rows`; only `pieces` of 4).  Fours of lanes
// change places first, so that they write 64 bytes of a row: a store then touches 8 rows
// instead of 32, whose lines the load-store unit takes one by one.
__device__ __forceinline__ void store_rows(void* tile, size_t stride, int first, int rows, int pieces,
                                           uint4 (&c)[4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int x = 1; x <= 2; x <<= 1) {
    const bool odd = lane & x;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4& a = c[x == 1 ? 2 * h : h];
      uint4& b = c[x == 1 ? 2 * h + 1 : h + 2];
      const uint4 give = odd ? a : b;
      uint4 got;
      got.x = __shfl_xor_sync(0xffffffffu, give.x, x);
      got.y = __shfl_xor_sync(0xffffffffu, give.y, x);
      got.z = __shfl_xor_sync(0xffffffffu, give.z, x);
      got.w = __shfl_xor_sync(0xffffffffu, give.w, x);
      if (odd)
        a = got;
      else
        b = got;
    }
  }
  const int row = first + (lane & ~3), i = lane & 3;
  uint8_t* dst = (uint8_t*)tile + row * stride + 16 * i;
#pragma unroll
  for (int r = 0; r < 4; ++r)
    if (row + r < rows && i < pieces) *reinterpret_cast<uint4*>(dst + r * stride) = c[r];
}
// 32 columns of the rows, times f, as bf16 to `tile`, and what the rounding leaves to
// `rest` when it is set
__device__ __forceinline__ void store_bf16(__nv_bfloat16* tile, __nv_bfloat16* rest, int d, int first,
                                           int rows, int pieces, const uint32_t (&v)[32], float f) {
  uint4 c[4], z[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float x[8];
    uint32_t h[4];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = __uint_as_float(v[8 * e + i]) * f;
#pragma unroll
    for (int i = 0; i < 4; ++i) h[i] = pack(x[2 * i], x[2 * i + 1]);
    c[e] = make_uint4(h[0], h[1], h[2], h[3]);
    if (rest)
      z[e] = make_uint4(pack_rest(x[0], x[1], h[0]), pack_rest(x[2], x[3], h[1]),
                        pack_rest(x[4], x[5], h[2]), pack_rest(x[6], x[7], h[3]));
  }
  store_rows(tile, 2 * (size_t)d, first, rows, pieces, c);
  if (rest) store_rows(rest, 2 * (size_t)d, first, rows, pieces, z);
}

// eight values of an output row, and what their rounding leaves when `rest` is set
__device__ __forceinline__ void store8(__nv_bfloat16* dst, __nv_bfloat16* rest, const float (&f)[8]) {
  uint32_t h[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = pack(f[2 * i], f[2 * i + 1]);
  *reinterpret_cast<uint4*>(dst) = make_uint4(h[0], h[1], h[2], h[3]);
  if (rest)
    *reinterpret_cast<uint4*>(rest) =
        make_uint4(pack_rest(f[0], f[1], h[0]), pack_rest(f[2], f[3], h[1]),
                   pack_rest(f[4], f[5], h[2]), pack_rest(f[6], f[7], h[3]));
}

// columns [0, 32) of a tile's 32-column piece that a row sees, as bits: columns
// [l, h) and [0, min(z, h)), all relative to the piece
__device__ __forceinline__ uint32_t bits_below(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}
__device__ __forceinline__ uint32_t seen_bits(int l, int h, int z) {
  return bits_below(h) & (~bits_below(l) | bits_below(z));
}

}  // namespace wtc
}  // namespace lapnys
