// The residual of a block with the norms around it:
//
//   h = x + m n(u),  m = gate scale,  n(u) = unit(u) post_weight + post_bias,
//   y = unit(h) weight + bias,        unit(z) = (z - mean) / sqrt(var + eps)
//                                     or  z / sqrt(mean of z^2 + eps).
//
// Backward, with e = dy weight and means over the row's features:
//   dh' = dh + r_h (e - mean(e) - unit(h) mean(e unit(h)))     (no mean(e): root mean square)
//   dx = dh',  du = the same of (dh' m post_weight) through unit(u),
//   dweight = sum dy unit(h), dbias = sum dy, and with S3 = sum dh' unit(u),
//   S4 = sum dh' over a sequence's rows: dpost_weight = sum_b m S3,
//   dpost_bias = sum_b m S4, dgate = scale (post_weight S3 + post_bias S4),
//   dscale = sum_b gate (post_weight S3 + post_bias S4).
//
// Bound by memory: a row is read once, kept in registers and written once; h is formed
// again from x and u in the backward, which reads as much as h would and has no rounding
// in it.  Statistics are of centred values, in fp32.
//
// Backward, up to 6144 features, 8192 without biases (k_norm_bwd_ring): a block an SM takes an
// even stretch of all rows, in tiles of as many rows as its warps work on at once (8 or 16
// features a thread of twelve or sixteen warps), which one thread copies into a ring in shared
// memory (bulk copies; a tile's rows lie side by side).  What a feature is multiplied by is
// laid out there once a sequence, in fp32.  8 x 16384 bf16 rows of 512, both norms, gate and
// scale: 158 us, 5.1 TB/s: sums over a row are what a row waits for, so rows in flight and
// registers count (a warp of its own for the copies costs the registers of four: eight warps
// of 16 features, or sixteen of 8, took 228); loads by the warps themselves beside 255
// registers a thread took 390.  Rows that are no whole 16 bytes lie in the ring as they lie in
// memory and are read from it by pairs or single elements: 1001 features, 428 us for 847 of
// the loads by the threads; 514, 450 for 1425 (2^27 bytes a tensor).  The mean is taken off
// before the product with 1 / deviation, 2 to 4 % of the time: rows of 512 with a mean of 1000
// deviations have weights' gradients as near as 32-bit operations one by one (as one multiply-add:
// 1.5 times as far off), du 1.4 times as far (1.9).
//
// Forward, rows of whole 16 bytes (bf16: or 4), up to 4096 features (k_norm_fwd_rows): threads
// copy their own pieces two rows ahead (cp.async), two blocks an SM: 98 us for the same rows,
// 5.5 TB/s; 32768 rows of 4096, two norms: 198 us, 5.4 TB/s.  (A ring of bulk copies as above:
// 434 us there; registers for the row ahead: 243.)
//
// Rows of up to 128 features (a head's): several to a warp in both directions, 8 features a
// lane. bf16 rows of 64, both layer norms: backward 203 us for 720 with a warp a row, forward
// 123 for 564; of 128: 210 for 367, 132 for 287 (2^27 bytes a tensor).
//
// Other rows (more features, forward of single elements, backward of tensors that start
// anywhere): k_norm_fwd, k_norm_bwd, loads by the threads as they are needed.
//
// The backward's sums over rows stay in registers, are joined over a block's row groups
// in shared memory and over the blocks by k_norm_seq, in one order.
#include "common.cuh"
#include "internal.h"
#include "layer.cuh"
#include "win_tc.cuh"

#include <type_traits>

namespace lapnys {
namespace {

__device__ __forceinline__ float as_f(float x) { return x; }
__device__ __forceinline__ float as_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void from_f(float* p, float x) { *p = x; }
__device__ __forceinline__ void from_f(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// the EPT features of a thread's share of a row: pieces of 16 bytes, `threads`
// pieces apart (WIDE), or single ones
template <typename T, int EPT, bool WIDE>
struct Share {
  static constexpr int V = WIDE ? 16 / (int)sizeof(T) : 1;
  static constexpr int NP = EPT / V;
  struct Raw {
    uint4 w[WIDE ? NP : 1];
    T s[WIDE ? 1 : EPT];
  };
  int t, threads, C;
  __device__ __forceinline__ int col(int j) const { return (j * threads + t) * V; }
  __device__ __forceinline__ Raw raw(const T* p) const {
    Raw r;
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = col(j);
      if constexpr (WIDE)
        r.w[j] = c < C ? *reinterpret_cast<const uint4*>(p + c) : make_uint4(0, 0, 0, 0);
      else
        r.s[j] = c < C ? p[c] : T(0.f);
    }
    return r;
  }
  __device__ __forceinline__ static void open(const Raw& r, float (&v)[EPT]) {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if constexpr (!WIDE) {
        v[j] = as_f(r.s[j]);
      } else if constexpr (sizeof(T) == 4) {
        v[4 * j] = __uint_as_float(r.w[j].x);
        v[4 * j + 1] = __uint_as_float(r.w[j].y);
        v[4 * j + 2] = __uint_as_float(r.w[j].z);
        v[4 * j + 3] = __uint_as_float(r.w[j].w);
      } else {
        const uint32_t w[4] = {r.w[j].x, r.w[j].y, r.w[j].z, r.w[j].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[8 * j + 2 * i] = __uint_as_float(w[i] << 16);
          v[8 * j + 2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
      }
    }
  }
  __device__ __forceinline__ void load(const T* p, float (&v)[EPT]) const { open(raw(p), v); }
  __device__ __forceinline__ void store(T* p, const float (&v)[EPT]) const {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      const int c = col(j);
      if (c >= C) continue;
      if constexpr (!WIDE) {
        from_f(p + c, v[j]);
      } else if constexpr (sizeof(T) == 4) {
        *reinterpret_cast<float4*>(p + c) = make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const __nv_bfloat162 h = __floats2bfloat162_rn(v[8 * j + 2 * i], v[8 * j + 2 * i + 1]);
          w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
        *reinterpret_cast<uint4*>(p + c) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  // whether element i of the share lies in the row
  __device__ __forceinline__ bool in(int i) const { return col(i / V) < C; }
};

// sums over the `warps` warps of a row group: by shuffles, then shared memory; SUB: over the
// `threads` lanes of a row that is less than a warp's
template <bool SUB = false>
struct RowSum {
  float2* slot;     // [2][32] of this group
  int warps, group, threads;
  int turn = 0;
  __device__ __forceinline__ float2 operator()(float2 v) {
    if (SUB || warps == 1) {
#pragma unroll
      for (int o = SUB ? threads >> 1 : 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
      }
      return v;
    }
    // a half of the warp each
    const bool upper = threadIdx.x & 16;
    float t = upper ? v.y : v.x;
    t += __shfl_xor_sync(0xffffffffu, upper ? v.x : v.y, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    float* s = reinterpret_cast<float*>(slot + 32 * turn) + (upper ? 1 : 0);
    turn ^= 1;      // the other half is free again after the next barrier
    const int w = (threadIdx.x >> 5) % warps, i = threadIdx.x & 15;
    if (i == 0) s[2 * w] = t;
    asm volatile("barrier.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    if (warps <= 4) {
      t = s[0];
      for (int j = 1; j < warps; ++j) t += s[2 * j];
    } else {
      t = i < warps ? s[2 * i] : 0.f;
      if (i + 16 < warps) t += s[2 * i + 32];
#pragma unroll
      for (int o = 8; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
    }
    const float z = __shfl_xor_sync(0xffffffffu, t, 16);
    return upper ? make_float2(z, t) : make_float2(t, z);
  }
  __device__ __forceinline__ float operator()(float v) {
#pragma unroll
    for (int o = SUB ? threads >> 1 : 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    if (SUB || warps == 1) return v;
    float* s = reinterpret_cast<float*>(slot + 32 * turn);
    turn ^= 1;
    const int w = (threadIdx.x >> 5) % warps, i = threadIdx.x & 31;
    if (i == 0) s[w] = v;
    asm volatile("barrier.sync %0, %1;" ::"r"(group + 1), "r"(threads) : "memory");
    if (warps <= 4) {
      v = s[0];
      for (int j = 1; j < warps; ++j) v += s[j];
    } else {
      v = i < warps ? s[i] : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    }
    return v;
  }
};

// mean and 1 / deviation of a row's values
template <typename S, int EPT>
__device__ __forceinline__ float2 row_stats(const float (&z)[EPT], int kind, float eps, const S& sh,
                                            RowSum<>& sum) {
  float mean = 0.f;
  const float inv = 1.f / (float)sh.C;
  if (kind == kNormLayer) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < EPT; ++i) t += z[i];       // 0 behind the row
    mean = sum(t) * inv;
  }
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    const float e = sh.in(i) ? z[i] - mean : 0.f;
    q = fmaf(e, e, q);
  }
  return make_float2(mean, rsqrtf(sum(q) * inv + eps));
}

template <typename T, int EPT, bool WIDE>
struct Rows {
  Share<T, EPT, WIDE> sh;
  RowSum<> sum;
  int group, groups;
  __device__ __forceinline__ Rows(const NormArgs& a, int warps, float2 (*slots)[64]) {
    const int warp = threadIdx.x >> 5;
    group = warp / warps;
    groups = (blockDim.x >> 5) / warps;
    sh.threads = 32 * warps;
    sh.t = threadIdx.x - group * sh.threads;
    sh.C = a.C;
    sum.slot = slots[group];
    sum.warps = warps;
    sum.group = group;
    sum.threads = sh.threads;
  }
};

// weight and bias of this thread's features, applied
template <typename S, typename T, int EPT>
__device__ __forceinline__ void affine(const S& sh, const T* w, const T* b, float (&v)[EPT]) {
  float t[EPT];
  if (w) {
    sh.load(w, t);
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] *= t[i];
  }
  if (b) {
    sh.load(b, t);
#pragma unroll
    for (int i = 0; i < EPT; ++i) v[i] += t[i];
  }
}
template <typename S, typename T, int EPT>
__device__ __forceinline__ void times(const S& sh, const T* w, float (&v)[EPT]) {
  affine(sh, w, (const T*)nullptr, v);
}

template <typename T, int EPT, bool WIDE, int TB>
__global__ void __launch_bounds__(TB) k_norm_fwd(NormArgs a, int warps) {
  __shared__ float2 slots[8][64];
  Rows<T, EPT, WIDE> r(a, warps, slots);
  const auto& sh = r.sh;
  const long long rows = (long long)a.B * a.N;
  for (long long row = (long long)blockIdx.x * r.groups + r.group; row < rows;
       row += (long long)gridDim.x * r.groups) {
    const size_t at = (size_t)row * a.C;
    const size_t seq = (size_t)(row / a.N) * a.C;
    float h[EPT];
    float2 su = make_float2(0.f, 0.f), s = make_float2(0.f, 0.f);
    const auto xr = sh.raw((const T*)a.x + at);
    if (a.u) {
      float u[EPT], x[EPT];
      sh.load((const T*)a.u + at, u);
      if (a.post != kNormNone) {
        su = row_stats(u, a.post, a.eps, sh, r.sum);
#pragma unroll
        for (int i = 0; i < EPT; ++i) u[i] = (u[i] - su.x) * su.y;
        affine(sh, (const T*)a.post_weight, (const T*)a.post_bias, u);
      }
      if (a.gate) times(sh, (const T*)a.gate + seq, u);
      times(sh, (const T*)a.scale, u);
      sh.open(xr, x);
#pragma unroll
      for (int i = 0; i < EPT; ++i) h[i] = sh.in(i) ? x[i] + u[i] : 0.f;
      if (a.h) sh.store((T*)a.h + at, h);
    } else {
      sh.open(xr, h);
      if (a.h) sh.store((T*)a.h + at, h);
    }
    if (a.y) {
      s = row_stats(h, a.pre, a.eps, sh, r.sum);
#pragma unroll
      for (int i = 0; i < EPT; ++i) h[i] = (h[i] - s.x) * s.y;
      const size_t of = a.per_seq ? seq : 0;
      affine(sh, a.weight ? (const T*)a.weight + of : nullptr,
             a.bias ? (const T*)a.bias + of : nullptr, h);
      sh.store((T*)a.y + at, h);
    }
    if (a.stats && sh.t == 0)
      reinterpret_cast<float4*>(a.stats)[row] = make_float4(su.x, su.y, s.x, s.y);
  }
}

// A block takes one range of one sequence's rows: blockIdx.x = b * parts + part.
template <typename T, int EPT, bool WIDE, int TB>
__global__ void __launch_bounds__(TB) k_norm_bwd(NormArgs a, int warps) {
  __shared__ float2 slots[8][64];
  extern __shared__ float join[];          // [4][C], where a block has several row groups
  Rows<T, EPT, WIDE> r(a, warps, slots);
  const auto& sh = r.sh;
  const int b = blockIdx.x / a.parts, part = blockIdx.x - b * a.parts;
  const int n0 = (int)((long long)a.N * part / a.parts), n1 = (int)((long long)a.N * (part + 1) / a.parts);
  const size_t seq = (size_t)b * a.C;
  const float inv = 1.f / (float)a.C;
  float A[4][EPT];
#pragma unroll
  for (int k = 0; k < 4; ++k)
#pragma unroll
    for (int i = 0; i < EPT; ++i) A[k][i] = 0.f;
  for (int n = n0 + r.group; n < n1; n += r.groups) {
    const size_t row = (size_t)b * a.N + n, at = row * a.C;
    const float4 st = reinterpret_cast<const float4*>(a.stats)[row];
    float uh[EPT], hh[EPT], d[EPT];
    const auto xr = sh.raw((const T*)a.x + at);
    if (a.u) {
      float t[EPT];
      sh.load((const T*)a.u + at, uh);
      if (a.post != kNormNone)
#pragma unroll
        for (int i = 0; i < EPT; ++i) uh[i] = (uh[i] - st.x) * st.y;
      sh.open(xr, hh);
#pragma unroll
      for (int i = 0; i < EPT; ++i) t[i] = uh[i];
      if (a.post != kNormNone) affine(sh, (const T*)a.post_weight, (const T*)a.post_bias, t);
      if (a.gate) times(sh, (const T*)a.gate + seq, t);
      times(sh, (const T*)a.scale, t);
#pragma unroll
      for (int i = 0; i < EPT; ++i) hh[i] += t[i];
    } else {
      sh.open(xr, hh);
    }
    if (a.dh) {
      sh.load((const T*)a.dh + at, d);
    } else {
#pragma unroll
      for (int i = 0; i < EPT; ++i) d[i] = 0.f;
    }
    if (a.dy) {
      float e[EPT];
      sh.load((const T*)a.dy + at, e);
      float2 m = make_float2(0.f, 0.f);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        hh[i] = (hh[i] - st.z) * st.w;
        A[0][i] = fmaf(e[i], hh[i], A[0][i]);
        A[1][i] += e[i];
      }
      if (a.weight) times(sh, (const T*)a.weight + (a.per_seq ? seq : 0), e);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {     // e is 0 behind the row
        m.x = fmaf(e[i], hh[i], m.x);
        m.y += e[i];
      }
      m = r.sum(m);
      const float m1 = m.x * inv, m0 = a.pre == kNormLayer ? m.y * inv : 0.f;
#pragma unroll
      for (int i = 0; i < EPT; ++i) d[i] = fmaf(st.w, e[i] - m0 - hh[i] * m1, d[i]);
    }
    if (a.dx) sh.store((T*)a.dx + at, d);
    if (a.u) {
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        A[2][i] = fmaf(d[i], uh[i], A[2][i]);
        A[3][i] += d[i];
      }
      if (a.gate) times(sh, (const T*)a.gate + seq, d);
      times(sh, (const T*)a.scale, d);
      if (a.post != kNormNone) {
        times(sh, (const T*)a.post_weight, d);
        float2 m = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const float e = sh.in(i) ? d[i] : 0.f;
          m.x = fmaf(e, uh[i], m.x);
          m.y += e;
        }
        m = r.sum(m);
        const float m1 = m.x * inv, m0 = a.post == kNormLayer ? m.y * inv : 0.f;
#pragma unroll
        for (int i = 0; i < EPT; ++i) d[i] = st.y * (d[i] - m0 - uh[i] * m1);
      }
      if (a.du) sh.store((T*)a.du + at, d);
    }
  }
  if (a.sums == 0) return;
  constexpr int V = Share<T, EPT, WIDE>::V;
  float* out = a.part + (size_t)blockIdx.x * 4 * a.C;
  if (r.groups > 1) {
    for (int g = 0; g < r.groups; ++g) {
      if (r.group == g)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (a.sums >> k & 1)
#pragma unroll
            for (int i = 0; i < EPT; ++i)
              if (sh.in(i)) {
                const int c = k * a.C + sh.col(i / V) + i % V;
                join[c] = g ? join[c] + A[k][i] : A[k][i];
              }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < 4 * a.C; c += blockDim.x)
      if (a.sums >> (c / a.C) & 1) out[c] = join[c];
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (a.sums >> k & 1)
#pragma unroll
        for (int i = 0; i < EPT; ++i)
          if (sh.in(i)) out[k * a.C + sh.col(i / V) + i % V] = A[k][i];
  }
}

// ---------------------------------------------------------------------------
// the backward's rows through a ring in shared memory
// ---------------------------------------------------------------------------
// warps of a block at the most, with E features a thread and KINDS of sums (by their registers)
constexpr int ring_warps(int E, int KINDS) { return E == 8 || KINDS == 2 ? 16 : 12; }
constexpr int RW = ring_warps(8, 4);
constexpr int RING = 6;           // tiles of the ring at the most
constexpr size_t kRingBytes = 216 * 1024;

// shared memory of a block: ring tiles, then vectors, then the join of the sums
struct RingShape {
  int warps, rows, nst;           // warps of a row, rows of a tile, tiles of the ring
  int lanes, workers;             // threads of a row, warps of the block
  uint32_t tensor, tile;          // bytes of a tensor's share of a tile, of a tile
  uint32_t tail;                  // bytes of a tensor behind its last whole 16
  uint32_t vec, join, total;      // bytes: where the vectors and the join start, and in all
};

__device__ __forceinline__ uint4 lds16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
// two or four bytes
template <int BYTES>
__device__ __forceinline__ uint32_t lds_piece(uint32_t addr) {
  uint32_t v;
  if constexpr (BYTES == 4) {
    asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  } else {
    uint16_t h;
    asm volatile("ld.shared.u16 %0, [%1];" : "=h"(h) : "r"(addr));
    v = h;
  }
  return v;
}
// 16 or 4 bytes to shared memory, zeros where `in` is not set
template <int BYTES>
__device__ __forceinline__ void cp_async_piece(uint32_t dst, const void* src, bool in) {
  if constexpr (BYTES == 16)
    cp_async16(dst, src, in);
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}
__device__ __forceinline__ f32x2 pair_of(uint32_t x, uint32_t y) {
  return pack2(__uint_as_float(x), __uint_as_float(y));
}

// The E features of a thread's share of a row, as pairs: pieces of V, `threads` pieces apart.
// FULL: the threads' features are the row's, none behind it.
template <typename T, int V, int E, bool FULL>
struct Pairs {
  static constexpr int NP = E / V, H = E / 2, B = V * (int)sizeof(T);   // pieces, pairs, bytes of a piece
  static constexpr bool WHOLE = B == 16;
  int t, threads, C;
  __device__ __forceinline__ int col(int j) const { return (j * threads + t) * V; }
  __device__ __forceinline__ bool in(int j) const { return FULL || col(j) < C; }
  // pieces in shared memory, the first at `at`, others `apart` bytes on; zeros behind the row
  __device__ __forceinline__ void load(uint32_t at, uint32_t apart, f32x2 (&p)[H]) const {
    if constexpr (WHOLE) {
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        uint4 f = make_uint4(0, 0, 0, 0);
        if (in(j)) f = lds16(at + j * apart);
        if constexpr (V == 4) {
          p[2 * j] = pair_of(f.x, f.y);
          p[2 * j + 1] = pair_of(f.z, f.w);
        } else {
          const uint32_t x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) p[4 * j + i] = pair_of(x[i] << 16, x[i] & 0xffff0000u);
        }
      }
    } else {
      uint32_t f[NP];
#pragma unroll
      for (int j = 0; j < NP; ++j) {
        f[j] = 0;
        if (in(j)) f[j] = lds_piece<B>(at + j * apart);
      }
#pragma unroll
      for (int i = 0; i < H; ++i) {
        if constexpr (V == 2)
          p[i] = pair_of(f[i] << 16, f[i] & 0xffff0000u);
        else if constexpr (sizeof(T) == 2)
          p[i] = pair_of(f[2 * i] << 16, f[2 * i + 1] << 16);
        else
          p[i] = pair_of(f[2 * i], f[2 * i + 1]);
      }
    }
  }
  __device__ __forceinline__ void store(T* o, const f32x2 (&p)[H]) const {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if (!in(j)) continue;
      if constexpr (V == 1) {
        const float2 x = unpack2(p[j / 2]);
        from_f(o + col(j), j & 1 ? x.y : x.x);
      } else if constexpr (V == 2) {
        const float2 x = unpack2(p[j]);
        *reinterpret_cast<uint32_t*>(o + col(j)) = wtc::pack(x.x, x.y);
      } else if constexpr (V == 4) {
        const float2 x = unpack2(p[2 * j]), y = unpack2(p[2 * j + 1]);
        *reinterpret_cast<float4*>(o + col(j)) = make_float4(x.x, x.y, y.x, y.y);
      } else {
        uint32_t w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 x = unpack2(p[4 * j + i]);
          w[i] = wtc::pack(x.x, x.y);
        }
        *reinterpret_cast<uint4*>(o + col(j)) = make_uint4(w[0], w[1], w[2], w[3]);
      }
    }
  }
  // A vector in shared memory, fp32: quarters of whole pieces side by side, others in order.
  // Where feature c of it lies:
  __device__ __forceinline__ int place(int c) const {
    return WHOLE ? (c % V / 4 * (C / V) + c / V) * 4 + c % 4 : c;
  }
  __device__ __forceinline__ void vec(uint32_t base, f32x2 (&p)[H]) const {
#pragma unroll
    for (int j = 0; j < NP; ++j) {
      if constexpr (WHOLE) {
#pragma unroll
        for (int i = 0; i < V / 4; ++i) {
          uint4 f = make_uint4(0, 0, 0, 0);
          if (in(j)) f = lds16(base + (i * (C / V) + j * threads + t) * 16);
          p[(V * j + 4 * i) / 2] = pair_of(f.x, f.y);
          p[(V * j + 4 * i) / 2 + 1] = pair_of(f.z, f.w);
        }
      } else {
        uint32_t f[2] = {0, 0};
        if (V == 2 && in(j)) {
          f[0] = lds_piece<4>(base + 4 * col(j));
          f[1] = lds_piece<4>(base + 4 * col(j) + 4);
        } else if (V == 1 && j % 2 == 0) {
          if (in(j)) f[0] = lds_piece<4>(base + 4 * col(j));
          if (in(j + 1)) f[1] = lds_piece<4>(base + 4 * col(j + 1));
        }
        if (V == 2 || j % 2 == 0) p[V * j / 2] = pair_of(f[0], f[1]);
      }
    }
  }
};

// sequence and first row of a tile, tile by tile
struct Place {
  int b, n;
  __device__ __forceinline__ void next(const NormArgs& a, int rows) {
    n += rows;
    if (n >= a.N) {
      n = 0;
      ++b;
    }
  }
};
__device__ __forceinline__ Place place_of(const NormArgs& a, int u, int rows) {
  const int b = u / a.tiles;
  return {b, (u - b * a.tiles) * rows};
}

// bytes before a tile's first row in its share of the ring: copies start at whole 16 bytes
__device__ __forceinline__ uint32_t ring_skip(const NormArgs& a, const Place& p, uint32_t es) {
  return ((uint32_t)p.b * (uint32_t)a.N + (uint32_t)p.n) * (uint32_t)a.C * es & 15u;
}

// What one thread copies: tile by tile, the tensors that are there and the rows' statistics.
// Rows that are no whole 16 bytes (WHOLE not set): with what lies around them, as far as the
// tensor goes; the last bytes of a tensor one by one.  (It is on the way of every tile: six
// 64-bit multiplications here took 4 % of the kernel.)
template <bool WHOLE>
struct Fill {
  size_t row;                     // the next tile's first
  int n;                          // its place in the sequence
  int st = 0, issued = 0;
  uint32_t ph = 0;
  __device__ __forceinline__ Fill(const NormArgs& a, const Place& at) : row((size_t)at.b * a.N + at.n), n(at.n) {}
  // one tile into the next slot, once all warps are done with what was there
  __device__ __forceinline__ bool tile(const NormArgs& a, const RingShape& s, uint32_t sm, uint64_t* full,
                                       uint64_t* empty, int es, int* err) {
    const void* src[4] = {a.x, a.u, a.dh, a.dy};
    if (!wtc::wait_or_flag(err, tc::smem_u32(&empty[st]), ph ^ 1u)) return false;
    const int rows = min(s.rows, a.N - n);
    const uint32_t bar = tc::smem_u32(&full[st]), base = sm + st * s.tile;
    size_t first = row * (uint32_t)(a.C * es);
    uint32_t bytes = (uint32_t)rows * a.C * es;
    if constexpr (!WHOLE) {
      const uint32_t skip = (uint32_t)first & 15u;
      first -= skip;
      bytes = (skip + bytes + 15u) & ~15u;
      if (first + bytes > (size_t)a.B * a.N * a.C * es) {
        bytes -= 16;
        for (int i = 0; i < 4; ++i)
          if (src[i])
            for (uint32_t o = bytes; o < bytes + s.tail; o += 2) {
              const uint16_t v = *reinterpret_cast<const uint16_t*>((const uint8_t*)src[i] + first + o);
              asm volatile("st.shared.u16 [%0], %1;" ::"r"(base + i * s.tensor + o), "h"(v) : "memory");
            }
      }
    }
    uint32_t all = rows * 16u;
#pragma unroll
    for (int i = 0; i < 4; ++i) all += src[i] ? bytes : 0u;
    tc::mbar_expect_tx(bar, all);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (src[i] && (WHOLE || bytes > 0))
        tc::bulk_g2s(base + i * s.tensor, (const uint8_t*)src[i] + first, bytes, bar);
    tc::bulk_g2s(base + 4 * s.tensor, a.stats + row * 4, rows * 16u, bar);
    row += rows;
    n += rows;
    if (n >= a.N) n = 0;
    ++issued;
    if (++st == s.nst) { st = 0; ph ^= 1u; }
    return true;
  }
};

// SUB: rows of less than a warp's features, several to a warp.
// KINDS: of sums over the rows; two: those through the unit norms alone (no bias's gradient)
template <typename T, int V, int E, int KINDS, bool FULL, bool SUB>
__global__ void __launch_bounds__(32 * ring_warps(E, KINDS), 1)
    k_norm_bwd_ring(NormArgs a, RingShape s, int* err) {
  using P = Pairs<T, V, E, FULL>;
  constexpr int RH = P::H;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 slots[RW][64];
  __shared__ __align__(8) uint64_t full[RING], empty[RING];
  const int workers = s.workers;
  const uint32_t sm = tc::smem_u32(smem);
  if (threadIdx.x == 0)
    for (int i = 0; i < s.nst; ++i) {
      tc::mbar_init(tc::smem_u32(&full[i]), 1);
      tc::mbar_init(tc::smem_u32(&empty[i]), workers);
    }
  asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  __syncthreads();
  const long long units = (long long)a.B * a.tiles;
  const int u0 = (int)(units * blockIdx.x / a.grid), u1 = (int)(units * (blockIdx.x + 1) / a.grid);
  const int threads = s.lanes, group = threadIdx.x / threads, workerst = 32 * workers;
  // thread 0 copies: all slots at first, then one a tile, that of `lag` tiles ago, so that it
  // need not wait for the slowest warp
  Fill<P::WHOLE> fill(a, place_of(a, u0, s.rows));
  bool late = false;
  const int lag = s.nst > 3 ? 2 : 1;
  if (threadIdx.x == 0)
    for (int i = 0; i < s.nst && u0 + i < u1; ++i) late = late || !fill.tile(a, s, sm, full, empty, sizeof(T), err);
  __syncwarp();
  const int t = threadIdx.x - group * threads;
  RowSum<SUB> sum{slots[SUB ? 0 : group], s.warps, group, threads};
  const P sh{t, threads, a.C};
  bool is = true;      // SUB: this thread's row is there
  auto sync = [&]() { __syncthreads(); };
  const float inv = 1.f / (float)a.C;

  // Vectors: weight, m post_weight, m post_bias in fp32, quarters of pieces side by side.
  const bool has_w = a.weight != nullptr && a.dy, has_m = a.u && (a.post != kNormNone || a.gate || a.scale);
  const bool has_b = a.post_bias != nullptr;
  const uint32_t vw = s.vec, vm = vw + (has_w ? 4u * a.C : 0u), vb = vm + (has_m ? 4u * a.C : 0u);
  auto vectors = [&](int b) {
    sync();                                           // nobody reads the last one's
    const size_t seq = (size_t)b * a.C;
    for (int c = threadIdx.x; c < a.C; c += workerst) {
      const int at = sh.place(c);
      float m = 1.f;
      if (a.gate) m *= as_f(((const T*)a.gate)[seq + c]);
      if (a.scale) m *= as_f(((const T*)a.scale)[c]);
      if (has_w) reinterpret_cast<float*>(smem + vw)[at] = as_f(((const T*)a.weight)[a.per_seq ? seq + c : c]);
      if (has_m) reinterpret_cast<float*>(smem + vm)[at] = a.post_weight ? m * as_f(((const T*)a.post_weight)[c]) : m;
      if (has_b) reinterpret_cast<float*>(smem + vb)[at] = m * as_f(((const T*)a.post_bias)[c]);
    }
    sync();
  };
  auto vec = [&](uint32_t base, f32x2(&p)[RH]) { sh.vec(sm + base, p); };
  // this thread's share of a tensor's row in the tile at `tile`
  const uint32_t row_at = (uint32_t)(group * a.C) * sizeof(T) + P::B * t;
  auto share = [&](uint32_t tile, int tensor, f32x2(&p)[RH]) {
    sh.load(tile + tensor * s.tensor + row_at, P::B * threads, p);
    if (SUB && !is)
#pragma unroll
      for (int i = 0; i < RH; ++i) p[i] = pack2(0.f, 0.f);
  };
  auto store = [&](void* base, size_t row, const f32x2(&p)[RH]) { sh.store((T*)base + row * a.C, p); };

  f32x2 A[KINDS][RH];
  constexpr int AT_U = KINDS / 2;     // of dh' unit(u)
  auto clear = [&]() {
#pragma unroll
    for (int k = 0; k < KINDS; ++k)
#pragma unroll
      for (int i = 0; i < RH; ++i) A[k][i] = pack2(0.f, 0.f);
  };
  // The sums of sequence b into this block's slot: half of a kind's pairs at a time side by
  // side in shared memory, [group][pair][thread], and the groups' sums in order.
  // (nvcc 13.0's front end drops the statement behind a loop that is the bare substatement of a
  // discarded constexpr if, in a lambda of a template: no such form in flush, where the join's
  // store was lost to it)
  const int share_of = SUB ? (int)(threadIdx.x >> 5) : group, shares = SUB ? s.workers : s.rows;
  auto flush = [&](int b) {
    constexpr int HP = RH / 2;
    float* out = a.part + ((size_t)b + blockIdx.x) * 4 * a.C;
    float2* join = reinterpret_cast<float2*>(smem + s.join);
    // pair i of thread t of a row
    auto put = [&](int k, int i, int t, float2 v) {
      const int c = ((2 * i / V) * threads + t) * V + 2 * i % V;
      if constexpr (V == 1) {
        if (c < a.C) out[k * a.C + c] = v.x;
        if (c + threads < a.C) out[k * a.C + c + threads] = v.y;
      } else {
        if (c < a.C) *reinterpret_cast<float2*>(out + k * a.C + c) = v;
      }
    };
#pragma unroll
    for (int n = 0; n < KINDS; ++n) {
      const int k = n * (4 / KINDS);
      if (!(a.sums >> k & 1)) continue;
      if (s.rows == 1) {
#pragma unroll
        for (int i = 0; i < RH; ++i) put(k, i, t, unpack2(A[n][i]));
        continue;
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 0; i < HP; ++i) {
          float2 v = unpack2(A[n][h * HP + i]);
          for (int o = SUB ? threads : 32; o < 32; o <<= 1) {     // the rows of a warp
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
          }
          if ((int)(threadIdx.x & 31) < threads) join[(share_of * HP + i) * threads + t] = v;
        }
        sync();
#pragma unroll 1
        for (int e = threadIdx.x; e < HP * threads; e += workerst) {
          float2 v = join[e];
#pragma unroll 4
          for (int g = 1; g < shares; ++g) {
            const float2 y = join[g * HP * threads + e];
            v.x += y.x;
            v.y += y.y;
          }
          put(k, h * HP + e / threads, e % threads, v);
        }
        sync();
      }
    }
  };
  // z becomes (z - mean) / deviation, the mean taken off first as in the forward (z r - mean r
  // would be off by the rounding of mean r, alike in all features)
  auto unit = [](f32x2(&z)[RH], int kind, float mean, float r) {
    const f32x2 rr = pack2(r, r), minus = pack2(-mean, -mean);
    if (kind == kNormLayer)
#pragma unroll
      for (int i = 0; i < RH; ++i) z[i] = wtc::add2(z[i], minus);
#pragma unroll
    for (int i = 0; i < RH; ++i) z[i] = wtc::mul2(z[i], rr);
  };
  // (sum of a b, sum of a) over the row
  auto moments = [&](const f32x2(&x)[RH], const f32x2(&y)[RH]) {
    f32x2 p = wtc::mul2(x[0], y[0]), q = x[0];
#pragma unroll
    for (int i = 1; i < RH; ++i) {
      p = fma2(x[i], y[i], p);
      q = wtc::add2(q, x[i]);
    }
    const float2 v = unpack2(p), w = unpack2(q);
    return sum(make_float2(v.x + v.y, w.x + w.y));
  };

  int st = 0, cur = -1;
  uint32_t ph = 0;
  Place here = place_of(a, u0, s.rows);
  for (int u = u0; u < u1; ++u, here.next(a, s.rows)) {
    const int b = here.b, n = here.n + group;
    if (threadIdx.x == 0 && u - u0 >= lag && u - lag + s.nst < u1)
      late = late || !fill.tile(a, s, sm, full, empty, sizeof(T), err);
    __syncwarp();
    if (b != cur) {
      if (cur >= 0 && a.sums) flush(cur);
      clear();
      if (cur < 0 || a.gate || a.per_seq) vectors(b);
      cur = b;
    }
    // after an expired wait (the error word is set) no other is waited for: every warp goes
    // on to its end, since the sums and the barriers need all
    late = __any_sync(0xffffffffu, late) || !wtc::wait_warp(err, tc::smem_u32(&full[st]), ph);
    is = n < a.N;
    if (SUB ? __any_sync(0xffffffffu, is) : is) {
      const size_t row = (size_t)b * a.N + n;
      const uint32_t tile = sm + st * s.tile + (P::WHOLE ? 0u : ring_skip(a, here, sizeof(T)));
      const uint4 qw = lds16(sm + st * s.tile + 4 * s.tensor + 16 * group);
      float mu = __uint_as_float(qw.x), ru = __uint_as_float(qw.y), mh = __uint_as_float(qw.z),
            rh = __uint_as_float(qw.w);
      if (SUB && !is) mu = ru = mh = rh = 0.f;
      f32x2 uh[RH], d[RH], v[RH];
      if (a.u) {
        share(tile, 1, uh);
        if (a.post != kNormNone) unit(uh, a.post, mu, ru);
      }
      if (a.dh) {
        share(tile, 2, d);
      } else {
#pragma unroll
        for (int i = 0; i < RH; ++i) d[i] = pack2(0.f, 0.f);
      }
      if (a.dy) {
        f32x2 e[RH], hh[RH];
        share(tile, 0, hh);
        share(tile, 3, e);
        if (a.u) {
          if (has_m) {
            vec(vm, v);
#pragma unroll
            for (int i = 0; i < RH; ++i) hh[i] = fma2(uh[i], v[i], hh[i]);
          } else {
#pragma unroll
            for (int i = 0; i < RH; ++i) hh[i] = wtc::add2(uh[i], hh[i]);
          }
          if (has_b) {
            vec(vb, v);
#pragma unroll
            for (int i = 0; i < RH; ++i) hh[i] = wtc::add2(hh[i], v[i]);
          }
        }
        unit(hh, a.pre, mh, rh);
#pragma unroll
        for (int i = 0; i < RH; ++i) {
          A[0][i] = fma2(e[i], hh[i], A[0][i]);
          if constexpr (KINDS == 4) A[1][i] = wtc::add2(e[i], A[1][i]);
        }
        if (has_w) {
          vec(vw, v);
#pragma unroll
          for (int i = 0; i < RH; ++i) e[i] = wtc::mul2(e[i], v[i]);
        }
        const float2 m = moments(e, hh);           // e is 0 behind the row
        const float k1 = -rh * (m.x * inv), k0 = a.pre == kNormLayer ? -rh * (m.y * inv) : 0.f;
        const f32x2 rr = pack2(rh, rh), kk1 = pack2(k1, k1), kk0 = pack2(k0, k0);
#pragma unroll
        for (int i = 0; i < RH; ++i) d[i] = fma2(e[i], rr, fma2(hh[i], kk1, wtc::add2(d[i], kk0)));
      }
      if (a.dx && (!SUB || is)) store(a.dx, row, d);
      if (a.u) {
#pragma unroll
        for (int i = 0; i < RH; ++i) {
          A[AT_U][i] = fma2(d[i], uh[i], A[AT_U][i]);
          if constexpr (KINDS == 4) A[3][i] = wtc::add2(d[i], A[3][i]);
        }
        if (has_m) {
          vec(vm, v);
#pragma unroll
          for (int i = 0; i < RH; ++i) d[i] = wtc::mul2(d[i], v[i]);   // 0 behind the row
        }
        if (a.post != kNormNone) {
          const float2 m = moments(d, uh);
          const float k1 = -ru * (m.x * inv), k0 = a.post == kNormLayer ? -ru * (m.y * inv) : 0.f;
          const f32x2 rr = pack2(ru, ru), kk1 = pack2(k1, k1), kk0 = pack2(k0, k0);
#pragma unroll
          for (int i = 0; i < RH; ++i) d[i] = fma2(d[i], rr, fma2(uh[i], kk1, kk0));
        }
        if (a.du && (!SUB || is)) store(a.du, row, d);
      }
    }
    wtc::arrive_warp(tc::smem_u32(&empty[st]));
    if (++st == s.nst) { st = 0; ph ^= 1u; }
  }
  if (cur >= 0 && a.sums) flush(cur);
  // no copy is in flight when the block ends: all were waited for, but after an expired wait
  if (threadIdx.x == 0 && late)
    for (int i = 0; i < s.nst && i < fill.issued; ++i) {
      const int k = fill.issued - 1 - i;
      wtc::wait_or_flag(err, tc::smem_u32(&full[k % s.nst]), (uint32_t)(k / s.nst) & 1u);
    }
}

// ---------------------------------------------------------------------------
// forward, rows of whole 16-byte pieces
// ---------------------------------------------------------------------------
constexpr int FW = 8;             // warps of a block at the most
constexpr int FD = 3;             // rows of the ring, the one that is worked on among them

// Threads copy their own pieces of a row (cp.async) two rows ahead, so that neither a
// barrier nor registers are needed for them.
template <typename T, int V, int E, bool FULL, bool SUB>
__global__ void __launch_bounds__(32 * FW, 2) k_norm_fwd_rows(NormArgs a, int warps, int rows, int lanes) {
  using P = Pairs<T, V, E, FULL>;
  constexpr int H = P::H;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ float2 slots[FW][64];
  const int group = threadIdx.x / lanes;
  const P sh{(int)threadIdx.x - group * lanes, lanes, a.C};
  RowSum<SUB> sum{slots[SUB ? 0 : group], warps, group, lanes};
  const float inv = 1.f / (float)a.C;
  const uint32_t sm = tc::smem_u32(smem);

  // vectors in fp32: weight, bias, m post_weight, m post_bias
  const bool has_m = a.u && (a.post != kNormNone || a.gate || a.scale);
  const uint32_t part = E * sizeof(T) * blockDim.x, ring = sm;     // a tensor's share of a slot
  const uint32_t size = 4u * a.C, vw = FD * 2 * part, vy = vw + (a.weight ? size : 0), vm = vy + (a.bias ? size : 0),
                 vb = vm + (has_m ? size : 0);
  auto vectors = [&](int b) {
    __syncthreads();
    const size_t seq = (size_t)b * a.C;
    for (int c = threadIdx.x; c < a.C; c += blockDim.x) {
      const int at = sh.place(c);
      const size_t of = a.per_seq ? seq + c : c;
      float m = 1.f;
      if (a.gate) m *= as_f(((const T*)a.gate)[seq + c]);
      if (a.scale) m *= as_f(((const T*)a.scale)[c]);
      if (a.weight) reinterpret_cast<float*>(smem + vw)[at] = as_f(((const T*)a.weight)[of]);
      if (a.bias) reinterpret_cast<float*>(smem + vy)[at] = as_f(((const T*)a.bias)[of]);
      if (has_m) reinterpret_cast<float*>(smem + vm)[at] = a.post_weight ? m * as_f(((const T*)a.post_weight)[c]) : m;
      if (a.post_bias) reinterpret_cast<float*>(smem + vb)[at] = m * as_f(((const T*)a.post_bias)[c]);
    }
    __syncthreads();
  };
  // z becomes its unit norm; returns (mean, 1 / deviation)
  auto unit = [&](f32x2(&z)[H], int kind) {
    float mean = 0.f;
    if (kind == kNormLayer) {
      f32x2 s = z[0];
#pragma unroll
      for (int i = 1; i < H; ++i) s = wtc::add2(s, z[i]);     // 0 behind the row
      const float2 v = unpack2(s);
      mean = sum(v.x + v.y) * inv;
      const f32x2 minus = pack2(-mean, -mean);
#pragma unroll
      for (int i = 0; i < H; ++i) z[i] = wtc::add2(z[i], minus);
    }
    f32x2 q = pack2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < H; ++i)
      if constexpr (V == 1) {
        const float2 v = unpack2(z[i]);
        const f32x2 e = pack2(sh.in(2 * i) ? v.x : 0.f, sh.in(2 * i + 1) ? v.y : 0.f);
        q = fma2(e, e, q);
      } else {
        if (sh.in(2 * i / V)) q = fma2(z[i], z[i], q);
      }
    const float2 v = unpack2(q);
    const float r = rsqrtf(sum(v.x + v.y) * inv + a.eps);
    const f32x2 rr = pack2(r, r);
#pragma unroll
    for (int i = 0; i < H; ++i) z[i] = wtc::mul2(z[i], rr);
    return make_float2(mean, r);
  };

  const long long units = (long long)a.B * a.tiles;
  const int u0 = (int)(units * blockIdx.x / gridDim.x), u1 = (int)(units * (blockIdx.x + 1) / gridDim.x);
  Place here = place_of(a, u0, rows), there = here;
  uint32_t slot_in = ring;
  int left = u1 - u0;                 // tiles that are not on their way
  // this thread's pieces of a row into its own places of a slot (zeros behind the row)
  auto fetch = [&](const T* p, uint32_t slot) {
#pragma unroll
    for (int j = 0; j < P::NP; ++j)
      cp_async_piece<P::B>(slot + (j * blockDim.x + threadIdx.x) * P::B, sh.in(j) ? p + sh.col(j) : p, sh.in(j));
  };
  auto ahead = [&]() {
    const uint32_t slot = slot_in;
    slot_in = slot_in + 2 * part == ring + FD * 2 * part ? ring : slot_in + 2 * part;
    const long long row = (long long)there.b * a.N + there.n + group;
    const bool is = left > 0 && there.n + group < a.N;
    --left;
    there.next(a, rows);
    if (is) {
      fetch((const T*)a.x + row * a.C, slot);
      if (a.u) fetch((const T*)a.u + row * a.C, slot + part);
    }
    cp_commit();
  };
#pragma unroll
  for (int i = 0; i < FD - 1; ++i) ahead();
  int cur = -1;
  uint32_t slot_out = ring;
  for (int u = u0; u < u1; ++u, here.next(a, rows)) {
    const int b = here.b;
    const long long row = here.n + group < a.N ? (long long)b * a.N + here.n + group : -1;
    if (b != cur) {
      if (cur < 0 || a.gate || a.per_seq) vectors(b);
      cur = b;
    }
    ahead();                          // into the slot of the row before
    asm volatile("cp.async.wait_group %0;" ::"n"(FD - 1) : "memory");
    f32x2 h[H], z[H];
    {
      const uint32_t slot = slot_out;
      slot_out = slot_out + 2 * part == ring + FD * 2 * part ? ring : slot_out + 2 * part;
      const uint32_t mine = slot + threadIdx.x * P::B, apart = blockDim.x * P::B;
      sh.load(mine, apart, h);
      if (a.u) sh.load(mine + part, apart, z);
    }
    const bool is = row >= 0;
    if (SUB ? !__any_sync(0xffffffffu, is) : !is) continue;
    float2 su = make_float2(0.f, 0.f), sy = make_float2(0.f, 0.f);
    f32x2 v[H];
    if (a.u) {
      if (a.post != kNormNone) su = unit(z, a.post);
      if (has_m) {
        sh.vec(sm + vm, v);
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = fma2(z[i], v[i], h[i]);     // 0 behind the row
      } else {
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = wtc::add2(z[i], h[i]);
      }
      if (a.post_bias) {
        sh.vec(sm + vb, v);
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = wtc::add2(h[i], v[i]);
      }
      if (a.h && is) sh.store((T*)a.h + row * a.C, h);
    } else if (a.h && is) {
      sh.store((T*)a.h + row * a.C, h);
    }
    if (a.y) {
      sy = unit(h, a.pre);
      if (a.weight) {
        sh.vec(sm + vw, v);
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = wtc::mul2(h[i], v[i]);
      }
      if (a.bias) {
        sh.vec(sm + vy, v);
#pragma unroll
        for (int i = 0; i < H; ++i) h[i] = wtc::add2(h[i], v[i]);
      }
      if (is) sh.store((T*)a.y + row * a.C, h);
    }
    if (a.stats && sh.t == 0 && is) reinterpret_cast<float4*>(a.stats)[row] = make_float4(su.x, su.y, sy.x, sy.y);
  }
}

constexpr int JY = 32;   // threads that share a column of the joins

// seq[b][k][c] = sum over a sequence's slots: `share` threads to a sequence, every one's
// slots, then the threads' sums in order; JY / share sequences a block
__global__ void __launch_bounds__(32 * JY) k_norm_seq(NormArgs a, int share) {
  __shared__ float s[JY][33];
  const int c = blockIdx.x * 32 + threadIdx.x, k = blockIdx.y;
  if (!(a.sums >> k & 1)) return;
  const int y = threadIdx.y % share, some = JY / share;
  for (long long b0 = (long long)blockIdx.z * some; b0 < a.B; b0 += (long long)gridDim.z * some) {
    const long long b = b0 + threadIdx.y / share;
    float t = 0.f;
    if (c < a.C && b < a.B) {
      size_t p0 = (size_t)b * a.parts, p1 = p0 + a.parts;
      if (a.grid > 0) {
        // block of tile u: the greatest c with tiles c / grid <= u
        const long long units = (long long)a.B * a.tiles, first = b * a.tiles;
        p0 = b + ((first + 1) * a.grid - 1) / units;
        p1 = b + ((first + a.tiles) * a.grid - 1) / units + 1;
      }
#pragma unroll 4
      for (size_t p = p0 + y; p < p1; p += share) t += a.part[(p * 4 + k) * a.C + c];
    }
    if (share > 1) {
      __syncthreads();
      s[threadIdx.y][threadIdx.x] = t;
      __syncthreads();
      if (y == 0)
        for (int i = 1; i < share; ++i) t += s[threadIdx.y + i][threadIdx.x];
    }
    if (y == 0 && c < a.C && b < a.B) a.seq[((size_t)b * 4 + k) * a.C + c] = t;
  }
}

// the gradients of the vectors from the sequences' sums: sequences y, y + 32, .. by
// thread y, then the threads' sums in order
template <typename T>
__global__ void __launch_bounds__(32 * JY) k_norm_final(NormArgs a) {
  __shared__ float s[5][JY][33];
  const int c = blockIdx.x * 32 + threadIdx.x, y = threadIdx.y;
  float t[5] = {0.f, 0.f, 0.f, 0.f, 0.f};   // weight, bias, post weight, post bias, scale
  if (c < a.C) {
    auto at = [&](const void* p, size_t i, float none) { return p ? as_f(((const T*)p)[i]) : none; };
    const float pw = at(a.post_weight, c, 1.f), pb = at(a.post_bias, c, 0.f), sc = at(a.scale, c, 1.f);
#pragma unroll 4
    for (int b = y; b < a.B; b += JY) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = a.sums >> k & 1 ? a.seq[((size_t)b * 4 + k) * a.C + c] : 0.f;
      const size_t i = (size_t)b * a.C + c;
      const float g = at(a.gate, i, 1.f), G = pw * v[2] + pb * v[3];
      if (a.per_seq) {
        if (a.dweight) from_f((T*)a.dweight + i, v[0]);
        if (a.dbias) from_f((T*)a.dbias + i, v[1]);
      }
      if (a.dgate) from_f((T*)a.dgate + i, sc * G);
      t[0] += v[0];
      t[1] += v[1];
      t[2] = fmaf(g * sc, v[2], t[2]);
      t[3] = fmaf(g * sc, v[3], t[3]);
      t[4] = fmaf(g, G, t[4]);
    }
  }
#pragma unroll
  for (int k = 0; k < 5; ++k) s[k][y][threadIdx.x] = t[k];
  __syncthreads();
  if (y < 5 && c < a.C) {
    void* out[5] = {a.per_seq ? nullptr : a.dweight, a.per_seq ? nullptr : a.dbias, a.dpost_weight,
                    a.dpost_bias, a.dscale};
    float v = 0.f;
    for (int i = 0; i < JY; ++i) v += s[y][i][threadIdx.x];
    void* o = y == 0 ? out[0] : y == 1 ? out[1] : y == 2 ? out[2] : y == 3 ? out[3] : out[4];
    if (o) from_f((T*)o + c, v);
  }
}

// features a thread, warps a row, row groups a block
struct Shape {
  int ept, warps, groups;
};
Shape shape(int C) {
  Shape s;
  s.ept = C <= 256 ? 8 : 16;
  s.warps = (C + 32 * s.ept - 1) / (32 * s.ept);
  s.groups = s.warps < 8 ? 8 / s.warps : 1;
  return s;
}

// rows without the ring: a block's threads bound its registers (8 features a thread: rows
// of up to 256, eight of them a block)
template <typename T, int EPT, bool WIDE>
cudaError_t go(const NormArgs& a, bool backward, const Shape& s, cudaStream_t st) {
  const int threads = 32 * s.warps * s.groups;
  const dim3 block(threads);
  if (!backward) {
    const long long rows = (long long)a.B * a.N, all = (rows + s.groups - 1) / s.groups;
    const dim3 grid((unsigned)(all < 152 * 64 ? all : 152 * 64));
    if constexpr (!WIDE)
      if (threads <= 256)
        return launch("norm_fwd", k_norm_fwd<T, EPT, WIDE, 256>, grid, block, 0, st, a, s.warps);
    if constexpr (EPT > 8)
      return launch("norm_fwd", k_norm_fwd<T, EPT, WIDE, 1024>, grid, block, 0, st, a, s.warps);
  } else {
    const dim3 grid((unsigned)(a.B * a.parts));
    const size_t smem = s.groups > 1 ? 16 * (size_t)a.C : 0;
    if constexpr (!WIDE)          // whole pieces: beyond the ring's width only
      if (threads <= 256)
        return launch("norm_bwd", k_norm_bwd<T, EPT, WIDE, 256>, grid, block, smem, st, a, s.warps);
    if constexpr (EPT > 8) {
      if (threads <= 512)
        return launch("norm_bwd", k_norm_bwd<T, EPT, WIDE, 512>, grid, block, smem, st, a, s.warps);
      return launch("norm_bwd", k_norm_bwd<T, EPT, WIDE, 1024>, grid, block, smem, st, a, s.warps);
    }
  }
  return cudaErrorInvalidValue;
}

// ranges of a sequence's rows: blocks for two an SM, each group of a block eight rows
// or more
int norm_parts(int B, int N, int C) {
  const Shape s = shape(C);
  const long long most = (N + 8LL * s.groups - 1) / (8LL * s.groups), want = (304 + B - 1) / B;
  const long long p = want < most ? want : most;
  return (int)(p < 1 ? 1 : p);
}

// lanes of a row of 8 features a lane: a power of two; 32 of more than 128 features
int lanes_of(int C) {
  int n = 1;
  while (n < 32 && 8 * n < C) n *= 2;
  return n;
}

// the ring's shape with E features a thread and `vecs` vectors, several rows a warp where
// `sub`; nst 0: rows that do not go through it
RingShape ring_shape(int C, int es, int E, int kinds, int vecs, bool sub = false) {
  RingShape r;
  const int most = ring_warps(E, kinds);
  r.warps = (C + 32 * E - 1) / (32 * E);
  r.rows = r.warps <= most ? most / r.warps : 1;
  r.lanes = 32 * r.warps;
  r.workers = r.warps * r.rows;
  if (sub) {
    r.lanes = lanes_of(C);
    r.rows *= 32 / r.lanes;
  }
  // rows that are no whole 16 bytes: with up to 15 bytes before and behind
  r.tensor = (uint32_t)((r.rows * C * es + (C * es % 16 ? 30 : 0) + 15) & ~15);
  r.tile = 4 * r.tensor + 16 * r.rows;
  r.tail = 0;
  const uint32_t vec = (4u * vecs * C + 15) & ~15u, join = r.rows > 1 ? 64u * r.workers * E : 0u;
  const size_t n = vec + join < kRingBytes ? (kRingBytes - vec - join) / r.tile : 0;
  r.nst = r.warps > most || n < 2 ? 0 : (int)(n < RING ? n : RING);
  r.vec = r.nst * r.tile;
  r.join = r.vec + vec;
  r.total = r.join + join;
  return r;
}

template <typename T, int V, int E, int KINDS, bool SUB = false>
cudaError_t go_ring(NormArgs& a, RingShape r, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  int* err = wait_error_address();
  if (err == nullptr) return cudaErrorInvalidSymbol;
  a.tiles = (a.N + r.rows - 1) / r.rows;
  const long long tiles = (long long)a.B * a.tiles;
  a.grid = (int)(tiles < 152 ? tiles : 152);
  static SmemOnce once[2];
  r.tail = (uint32_t)((size_t)a.B * a.N * a.C * sizeof(T) % 16);
  constexpr bool WHOLE = V * sizeof(T) == 16;
  const bool full = WHOLE && a.C == r.lanes * E;
  auto* k = full ? k_norm_bwd_ring<T, V, E, KINDS, WHOLE, SUB> : k_norm_bwd_ring<T, V, E, KINDS, false, SUB>;
  if ((e = once[full].allow(k, kRingBytes, dev)) != cudaSuccess) return e;
  return launch("norm_bwd", k, dim3(a.grid), dim3(32 * r.workers), r.total, st, a, r, err);
}

template <typename T, int V, int E, bool SUB = false>
cudaError_t go_rows(NormArgs& a, const Shape& s, cudaStream_t st) {
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess) return e;
  static SmemOnce once[2];
  constexpr bool WHOLE = V * sizeof(T) == 16;
  const int lanes = SUB ? lanes_of(a.C) : 32 * s.warps, rows = 32 * s.warps * s.groups / lanes;
  const bool full = WHOLE && a.C == lanes * E;
  auto* k = full ? k_norm_fwd_rows<T, V, E, WHOLE, SUB> : k_norm_fwd_rows<T, V, E, false, SUB>;
  // ring, and the vectors that there are
  const int vecs = (a.weight != nullptr) + (a.bias != nullptr) + (a.post_bias != nullptr) +
                   (a.u && (a.post != kNormNone || a.gate || a.scale));
  const size_t threads = 32 * s.warps * s.groups, smem = FD * 2 * threads * E * sizeof(T) + (size_t)vecs * a.C * 4;
  if ((e = once[full].allow(k, FD * 2 * 32 * FW * E * sizeof(T) + 4 * 32 * FW * E * 4, dev)) != cudaSuccess) return e;
  a.tiles = (a.N + rows - 1) / rows;
  // as many blocks as an SM's shared memory takes (4 KB are static, 1 KB reserved), two at the most
  const long long tiles = (long long)a.B * a.tiles, most = 152LL * (2 * (smem + 5120) <= 228 * 1024 ? 2 : 1);
  const unsigned grid = (unsigned)(tiles < most ? tiles : most);
  return launch("norm_fwd", k, dim3(grid), dim3(32 * s.warps * s.groups), smem, st, a, s.warps, rows, lanes);
}

template <typename T>
cudaError_t pick(NormArgs& a, bool backward, cudaStream_t st) {
  const Shape s = shape(a.C);
  bool wide = a.C % (16 / (int)sizeof(T)) == 0;
  const void* all[] = {a.x, a.u, a.weight, a.bias, a.post_weight, a.post_bias, a.gate, a.scale,
                       a.h, a.y, a.dh, a.dy, a.dx, a.du};
  for (const void* p : all) wide = wide && ((uintptr_t)p & 15) == 0;
  auto al = [](const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; };
  constexpr int V = 16 / (int)sizeof(T);   // features of 16 bytes
  if (backward && al(a.x, 16) && al(a.u, 16) && al(a.dh, 16) && al(a.dy, 16)) {
    const bool whole = a.C % V == 0 && al(a.dx, 16) && al(a.du, 16);
    // fewer sums over the rows leave registers for sixteen warps of 16 features (bf16 rows of
    // 4096, two root mean squares: 170 us, 258 by 8 features; of 8192: 191, 364 by k_norm_bwd);
    // pairs and single elements have none left (rows of 1001: 428 us for 356)
    const bool two = whole && !(a.sums & (kSumDy | kSumDh));
    const int vecs = (a.weight && a.dy) + (a.u && (a.post != kNormNone || a.gate || a.scale)) + (a.post_bias != nullptr);
    const RingShape r = ring_shape(a.C, sizeof(T), 8, 4, vecs),
                    r16 = ring_shape(a.C, sizeof(T), 16, two ? 2 : 4, vecs);
    // 16 features a thread where that works on a third more rows at once and leaves a ring of
    // three tiles, or on twice the rows (bf16 rows of 512, 12 for 8: 173 us for 242; of 1536, 4
    // for 2: 199 for 306; of 640, 6 for 5: 334 for 322; fp32 rows of 512, two tiles: 146 for
    // 139); on two thirds more where only 8 fill their warps (768, 8 for 5: 287 for 255; 1280, 5
    // for 3: 238 for 260); and where 8 do not reach over the row
    const bool only8 = a.C % 256 == 0 && a.C % 512 != 0;
    const bool more = r.nst == 0 || (r16.nst > 2 && 3 * r16.rows >= (only8 ? 5 : 4) * r.rows) ||
                      (r16.nst == 2 && r16.rows >= 2 * r.rows);
    if (!more || r16.nst > 0) {
      // several rows a warp, where a sequence's rows fill half a tile of them
      const RingShape rs = ring_shape(a.C, sizeof(T), 8, 4, vecs, true);
      const bool sub = a.C <= 128 && rs.nst > 0 && 2LL * a.N >= rs.rows;
      auto with = [&](auto v) {
        constexpr int P = decltype(v)::value;
        if (sub) return go_ring<T, P, 8, 4, true>(a, rs, st);
        if (!more) return go_ring<T, P, 8, 4>(a, r, st);
        if constexpr (P == V)
          if (two) return go_ring<T, P, 16, 2>(a, r16, st);
        return go_ring<T, P, 16, 4>(a, r16, st);
      };
      if (whole) return with(std::integral_constant<int, V>{});
      if constexpr (sizeof(T) == 2)
        if (a.C % 2 == 0 && al(a.dx, 4) && al(a.du, 4)) return with(std::integral_constant<int, 2>{});
      return with(std::integral_constant<int, 1>{});
    }
  }
  if (!backward && s.warps <= FW) {
    auto rows = [&](size_t n) { return a.C % (n / sizeof(T)) == 0 && al(a.x, n) && al(a.u, n) && al(a.h, n) && al(a.y, n); };
    // several rows a warp, where a sequence's rows fill half a tile of them
    const bool sub = a.C <= 128 && 2LL * a.N >= 32 * FW / lanes_of(a.C);
    if (rows(16))
      return sub ? go_rows<T, V, 8, true>(a, s, st)
                 : s.ept == 8 ? go_rows<T, V, 8>(a, s, st) : go_rows<T, V, 16>(a, s, st);
    // pairs of bf16 (rows of 514, 2^27 bytes a tensor: 420 us, 552 by k_norm_fwd; single fp32
    // values of rows of 1001 took 245 us for 182)
    if constexpr (sizeof(T) == 2)
      if (rows(4))
        return sub ? go_rows<T, 2, 8, true>(a, s, st)
                   : s.ept == 8 ? go_rows<T, 2, 8>(a, s, st) : go_rows<T, 2, 16>(a, s, st);
  }
  a.parts = norm_parts(a.B, a.N, a.C);
  if (s.ept == 8) return go<T, 8, false>(a, backward, s, st);
  return wide ? go<T, 16, true>(a, backward, s, st) : go<T, 16, false>(a, backward, s, st);
}

}  // namespace

int norm_slots(int B, int N, int C) {
  const long long a = (long long)B * norm_parts(B, N, C), b = (long long)B + 152;
  return (int)(a > b ? a : b);
}

cudaError_t run_norm_fwd(NormArgs& a, bool bf16, cudaStream_t st) {
  return bf16 ? pick<__nv_bfloat16>(a, false, st) : pick<float>(a, false, st);
}

cudaError_t run_norm_bwd(NormArgs& a, bool bf16, cudaStream_t st) {
  a.grid = 0;
  cudaError_t e = bf16 ? pick<__nv_bfloat16>(a, true, st) : pick<float>(a, true, st);
  if (e != cudaSuccess || a.sums == 0) return e;
  const unsigned cols = (unsigned)((a.C + 31) / 32);
  NormArgs f = a;
  if (a.grid == 0 && a.parts == 1) {
    f.seq = a.part;
  } else {
    // about four slots a thread (4096 sequences of a slot or two each: 76 us, 1560 with 32
    // threads to each)
    const long long slots = a.grid > 0 ? (a.grid + a.B - 1) / a.B + 1 : a.parts;
    int share = 1;
    while (share < JY && 4 * share < slots) share *= 2;
    const long long blocks = (a.B + JY / share - 1) / (JY / share);
    e = launch("norm_seq", k_norm_seq, dim3(cols, 4, (unsigned)(blocks < 65535 ? blocks : 65535)),
               dim3(32, JY), 0, st, a, share);
    if (e != cudaSuccess) return e;
  }
  if (bf16) return launch("norm_final", k_norm_final<__nv_bfloat16>, dim3(cols), dim3(32, JY), 0, st, f);
  return launch("norm_final", k_norm_final<float>, dim3(cols), dim3(32, JY), 0, st, f);
}

}  // namespace lapnys
