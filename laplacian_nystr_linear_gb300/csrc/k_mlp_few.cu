// The feed-forward block for a few rows (single tokens of some sequences).
//
// Bound by memory: every weight is read once and used for all rows, so the weights are
// laid out as one stretch of units, 64 k of a block of columns each, block after block,
// and every CTA takes an equal share of it, whatever the sizes are.  A CTA leaves the
// partial sums of each column block that it met; k_mlp_few_join adds a block's parts in
// order and applies bias and gate.  Every kernel lets the next one start at once and
// waits for the one before itself, so the second product's CTAs fill their rings with
// weights as soon as the first one's leave their SMs, before the join in between.
//
// bf16: the weights are the instruction's left operand (256 columns as two times its M,
// MN-major as they lie), the rows of x its N (T padded to 16): one thread copies by TMA
// into a ring of 32 KB slots (about 190 KB in flight an SM), one issues tcgen05 products,
// four warps read the sums.  fp32: on the FP32 pipe, 128 columns a warp, four a lane, rows
// in packed pairs, x from shared memory; 16 rows a CTA, further rows by CTAs beside it that
// read the same weights out of L2.  bf16 calls of up to 32 rows keep h in two bf16 parts, the
// second as further rows of the second product, which is bound by its weights all the same.
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
constexpr int FEW_BF16 = 64, FEW_F32 = 48;   // rows
constexpr int NTC = 192, NST = 6;     // slots at the most
constexpr uint32_t A_BYTES = FNB * FK * 2;
constexpr int NF32 = 256;

__device__ __forceinline__ void wait_before() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }

// the stretch [u0, u1) of a CTA; unit u is k step u % ks of column block u / ks
__device__ __forceinline__ void stretch(const MlpFewArgs& a, int c, int* u0, int* u1) {
  const long long units = (long long)a.parts * a.nb * a.ks;
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
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t sm = (tc::smem_u32(sm_raw) + 1023u) & ~1023u;
  const uint32_t b_bytes = (uint32_t)rows * FK * 2, slot = A_BYTES + b_bytes;
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  let_next();
  if (warp == 1) tc::tmem_alloc(&tmem_s, 256);
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
  if (!(warp == 0 && a.second)) wait_before();

  if (warp == 0) {
    // ---------------- copies ----------------
    if (wtc::elect_one()) {
      int issued = 0;
      bool bad = false;
      auto weights = [&](int u, int st) {
        const int block = u / a.ks, k = u - block * a.ks, part = block / a.nb;
        const uint32_t bar = tc::smem_u32(&full[st]), sa = sm + st * slot;
        // columns of the row of both parts: a part's last block may reach into the next
        // part, whose sums nobody reads
        const int n = part * a.N + (block - part * a.nb) * FNB;
        tc::mbar_expect_tx(bar, slot);
#pragma unroll
        for (int i = 0; i < FNB / 64; ++i) tma2(sa + 8192 * i, &mp.w, n + 64 * i, k * FK, bar);
      };
      // weights are no other kernel's output here: as many as there is room for before
      // the rows are there
      const int head = a.second ? (u1 - u0 < nst ? u1 - u0 : nst) : 0;
      for (int i = 0; i < head; ++i) weights(u0 + i, i);
      if (a.second) wait_before();
      for (int u = u0; u < u1; ++u) {
        const int st = issued % nst, k = u % a.ks;
        if (issued >= head) {
          if (!wtc::wait_or_flag(a.err, tc::smem_u32(&empty[st]), ((uint32_t)(issued / nst) & 1u) ^ 1u)) {
            bad = true;
            break;
          }
          weights(u, st);
        }
        tma2(sm + st * slot + A_BYTES, &mp.x, k * FK, 0, tc::smem_u32(&full[st]));
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
      const uint32_t id = tc::idesc_bf16(128, rows) | (1u << 15);
      const uint64_t da0 = wtc::desc_mn(sm, 8192), db0 = wtc::desc_k(sm + A_BYTES);
      for (int u = u0; u < u1 && !bad; ++seg) {
        const int end = min(u1, (u / a.ks + 1) * a.ks), first = u;
        if (!wtc::wait_or_flag(a.err, tc::smem_u32(&acce[seg & 1]), ((uint32_t)(seg >> 1) & 1u) ^ 1u)) {
          bad = true;
          break;
        }
        tc::fence_after();
        const uint32_t d = tmem + (uint32_t)(seg & 1) * 128;
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
            tc::mma_bf16(d, da + 128 * k, db + 2 * k, id, u > first || k > 0);
            tc::mma_bf16(d + 64, da + 1024 + 128 * k, db + 2 * k, id, u > first || k > 0);
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
      u = min(u1, (block + 1) * a.ks);
      __syncwarp();
      if (!wtc::wait_warp(a.err, tc::smem_u32(&accf[seg & 1]), (uint32_t)(seg >> 1) & 1u)) {
        bad = true;
        break;
      }
      tc::fence_after();
      // one slot for each (column block, CTA) that meet: both only grow
      float* o = a.part + (size_t)(block + blockIdx.x) * a.T * FNB + 32 * q + lane;
      for (int t0 = 0; t0 < rows; t0 += 16)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          uint32_t x[16];
          tc::tmem_ld<16>(tmem + ((uint32_t)(32 * q) << 16) + (uint32_t)((seg & 1) * 128 + 64 * half + t0), x);
#pragma unroll
          for (int i = 0; i < 16; ++i)
            if (t0 + i < a.T) o[(t0 + i) * FNB + 128 * half] = __uint_as_float(x[i]);
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
  if (warp == 1) tc::tmem_dealloc(tmem, 256);
}

// fp32: TT rows from 16 blockIdx.y.  Warps take a segment's k in turn; their sums are
// joined in shared memory, halves of the warps at a time, in one order.
template <int TT, bool WIDE>
__global__ void __launch_bounds__(NF32, 2) k_mlp_few_f32(MlpFewArgs a) {
  constexpr int CH = 128;                   // k of x in shared memory
  __shared__ __align__(16) float xs[CH][TT];
  __shared__ __align__(16) float4 join[4][TT][32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, row0 = blockIdx.y * 16;
  const int rows = min(TT, a.T - row0);
  int u0, u1;
  stretch(a, blockIdx.x, &u0, &u1);
  let_next();
  wait_before();
  const size_t ld = (size_t)a.parts * a.N;
  const float* x0 = (const float*)a.x + (size_t)row0 * a.K;
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
    for (int kc = k0; kc < k1; kc += CH) {
      const int m = min(CH, k1 - kc);
      __syncthreads();
      for (int e = threadIdx.x; e < CH * TT; e += NF32) {
        const int t = e / CH, k = e % CH;
        xs[k][t] = t < rows && k < m ? x0[(size_t)t * a.K + kc + k] : 0.f;
      }
      __syncthreads();
#pragma unroll 8
      for (int k = warp; k < m; k += NF32 / 32) {
        const float* p = w + (size_t)(kc + k) * ld;
        float v[4];
        if constexpr (WIDE) {
          const float4 f = n < a.N ? __ldcs(reinterpret_cast<const float4*>(p)) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) v[c] = n + c < a.N ? __ldg(p + c) : 0.f;
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
    // warps 4 .. 7 into 0 .. 3, then 2, 3 into 0, 1, then 1 into 0
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
      float* o = a.part + ((size_t)(block + blockIdx.x) * a.T + row0) * FNF + 4 * lane;
#pragma unroll
      for (int t = 0; t < TT; ++t)
        if (t < rows) *reinterpret_cast<float4*>(o + t * FNF) = row(t);
    }
  }
}

// a column block of a row (blockIdx.y): its parts in order, then bias and gate
template <typename T>
__global__ void __launch_bounds__(256) k_mlp_few_join(MlpFewArgs a) {
  constexpr int FN = sizeof(T) == 4 ? FNF : FNB;
  const int t = blockIdx.y, n = blockIdx.x * FN + threadIdx.x;
  let_next();
  wait_before();
  const long long units = (long long)a.parts * a.nb * a.ks;
  float v[2] = {0.f, 0.f};
  for (int p = 0; p < a.parts; ++p) {
    const long long block = p * a.nb + blockIdx.x, first = block * a.ks, last = first + a.ks - 1;
    // the CTA of unit u: the greatest c with units c / grid <= u
    const int c0 = (int)(((first + 1) * a.grid - 1) / units), c1 = (int)(((last + 1) * a.grid - 1) / units);
    const float* s = a.part + ((size_t)(block + c0) * a.T + t) * FN + threadIdx.x;
    float lo = 0.f;                   // of the rows that are what rounding left of x
    const bool both = a.T > a.rows;
#pragma unroll 4
    for (int c = c0; c <= c1; ++c, s += (size_t)a.T * FN) {
      v[p] += *s;
      if (both) lo += s[(size_t)a.rows * FN];
    }
    v[p] += lo;
    if (a.bias && n < a.N) {
      if constexpr (sizeof(T) == 4)
        v[p] += ((const T*)a.bias)[(size_t)p * a.N + n];
      else
        v[p] += __bfloat162float(((const T*)a.bias)[(size_t)p * a.N + n]);
    }
  }
  if (n >= a.N) return;
  if (a.act >= 0) {
    constexpr bool EXACT = sizeof(T) == 4;
    float p, s;
    if (a.act == kActSilu)
      mlp_act<EXACT, kActSilu>(v[0], p, s);
    else if (a.act == kActGelu)
      mlp_act<EXACT, kActGelu>(v[0], p, s);
    else
      mlp_act<EXACT, kActGeluTanh>(v[0], p, s);
    v[0] = p * v[1];
  }
  T* o = (T*)a.out + (size_t)t * a.N + n;
  if constexpr (sizeof(T) == 4)
    *o = v[0];
  else {
    *o = __float2bfloat16_rn(v[0]);
    const float hi = __bfloat162float(__float2bfloat16_rn(v[0]));
    if (a.two) o[(size_t)a.rows * a.N] = __float2bfloat16_rn(isinf(hi) ? 0.f : v[0] - hi);
  }
}

// grid and units of a product: a CTA for each SM (fp32: two), as far as there are units
void shape(MlpFewArgs& a, bool f32) {
  const int fn = f32 ? FNF : FNB;
  a.nb = (a.N + fn - 1) / fn;
  a.ks = (a.K + FK - 1) / FK;
  const long long units = (long long)a.parts * a.nb * a.ks, most = f32 ? 304 / ((a.T + 15) / 16) : 152;
  a.grid = (int)(units < most ? units : most);
}

template <int TT>
cudaError_t go_f32(MlpFewArgs& a, cudaStream_t st) {
  const bool wide = a.N % 4 == 0 && ((uintptr_t)a.w & 15) == 0;
  auto* k = wide ? k_mlp_few_f32<TT, true> : k_mlp_few_f32<TT, false>;
  const dim3 grid(a.grid, (a.T + 15) / 16);
  if (a.second) return launch_after("mlp_few", k, grid, dim3(NF32), 0, st, a);
  return launch("mlp_few", k, grid, dim3(NF32), 0, st, a);
}

}  // namespace

// T rows that read all weights once; bf16 rows and columns have to be whole 16-byte
// pieces
bool mlp_few_ok(int T, int C, int F, bool f32) {
  if ((double)C * F >= 1e12) return false;      // units are counted in 32 bits
  return f32 ? T <= FEW_F32 : T <= FEW_BF16 && C % 8 == 0 && F % 8 == 0;
}

// bf16: what rounding leaves of h goes along as further rows of the second product, as far
// as they fit (they cost it nothing: it is bound by the weights)
bool mlp_few_two(int T, bool f32) { return !f32 && 2 * T <= FEW_BF16; }

size_t mlp_few_bytes(int T, int N, int parts) {
  // slots of FNF or FNB columns: as many of the one, half as wide, as are needed of either
  const size_t slots = (size_t)parts * ((N + FNF - 1) / FNF + 1) + 304;
  return slots * T * FNB * 4;
}

cudaError_t run_mlp_few(MlpFewArgs& a, bool f32, cudaStream_t st) {
  shape(a, f32);
  a.err = wait_error_address();
  if (a.err == nullptr) return cudaErrorInvalidSymbol;
  cudaError_t e;
  if (f32) {
    e = a.T <= 4 ? go_f32<4>(a, st) : (a.T <= 8 ? go_f32<8>(a, st) : go_f32<16>(a, st));
  } else {
    int dev = 0, sms = 0;
    if ((e = device_sms(&dev, &sms)) != cudaSuccess) return e;
    const int rows = (a.T + 15) / 16 * 16;
    FewMaps mp;
    memset(&mp, 0, sizeof(mp));
    const cuuint64_t wd[2] = {(cuuint64_t)a.parts * a.N, (cuuint64_t)a.K}, ws[1] = {wd[0] * 2};
    const cuuint64_t xd[2] = {(cuuint64_t)a.K, (cuuint64_t)a.T}, xs[1] = {xd[0] * 2};
    const cuuint32_t wb[2] = {64, FK}, xb[2] = {64, (cuuint32_t)rows};
    if (!encode_tiled_bf16_sw128(&mp.w, 2, a.w, wd, ws, wb) ||
        !encode_tiled_bf16_sw128(&mp.x, 2, a.x, xd, xs, xb))
      return cudaErrorInvalidValue;
    static SmemOnce once;
    // six slots of up to 32 rows of x, five of more
    const int nst = rows <= 32 ? NST : NST - 1;
    constexpr size_t most = NST * (A_BYTES + 32 * FK * 2) + 1024;
    static_assert((NST - 1) * (A_BYTES + FEW_BF16 * FK * 2) + 1024 <= most, "");
    if ((e = once.allow(k_mlp_few_tc, most, dev)) != cudaSuccess) return e;
    const size_t smem = nst * (A_BYTES + (size_t)rows * FK * 2) + 1024;
    e = a.second ? launch_after("mlp_few", k_mlp_few_tc, dim3(a.grid), dim3(NTC), smem, st, mp, a, rows, nst)
                 : launch("mlp_few", k_mlp_few_tc, dim3(a.grid), dim3(NTC), smem, st, mp, a, rows, nst);
  }
  if (e != cudaSuccess) return e;
  const dim3 grid(a.nb, a.rows);
  if (f32) return launch_after("mlp_few_join", k_mlp_few_join<float>, grid, dim3(FNF), 0, st, a);
  return launch_after("mlp_few_join", k_mlp_few_join<__nv_bfloat16>, grid, dim3(FNB), 0, st, a);
}

}  // namespace lapnys
