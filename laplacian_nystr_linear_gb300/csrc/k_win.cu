// Windowed softmax attention of fp32 tensors (visibility rule: win.cuh): forward,
// query gradients, key and value gradients.
//
//   s = scale q.k over the visible keys, P = softmax(s), o = P v
//   D = dout.o, dV = P^T dout, dP = dout V^T, dS = P (dP - D),
//   dQ = scale dS K, dK = scale dS^T Q  (both summed over a group's query heads)
//
// One pass over the keys with the running maximum and sum of each row's softmax;
// the backward recomputes P from the saved log-sum.  Products on the warp-level
// tensor instruction: every operand is three bf16 parts (24 bits) and a product the
// six of their products above 2^-24 (98 TFLOP/s at the instruction's measured rate;
// the FP32 pipe, with operands from shared memory, gave 25 to 30).  The instruction
// cuts its sums off instead of rounding them, so it sums 12 products of a tile at the
// most (scores 6) and the FP32 pipe adds those up: gradients of 700 tokens, heads of
// 128, are off by 3.5e-7 of their norm, with scores summed by the instruction 1.7e-6.
//
// Tiles of 64 rows (queries; keys for dK, dV) x 64 columns, 8 warps: 16 rows and one
// half of the columns each, so a warp's softmax and sums are its own and the halves
// meet once, at the end.  Tiles are split when they are loaded, as three planes of
// shared memory whose 16-byte chunks are XORed with the row (ldmatrix without bank
// conflicts, plain or transposed); P and dS are split in registers.
// Bound by the tensor instruction (4 d operations forward, 14 d backward for each
// visible pair, times six); by its latency where there are few tiles.  Measured: 16 heads
// of 64, 2432 tokens, all visible: 407, 554 and 759 us (60 TFLOP/s of the forward's 4 d,
// 46 of the backward's 10 d); 8 heads of 128: 416, 605 and 790 us.  196 tokens, one head of
// 32: 21, 21 and 24 us.
#include "common.cuh"
#include "internal.h"
#include "win.cuh"

namespace lapnys {

namespace {
constexpr int WT = 64;        // rows and columns of a tile

template <int DP>
struct Planes {
  static constexpr int RB = 2 * DP, PL = WT * RB;   // bytes of a row, of a plane
  static constexpr int BYTES = 3 * PL;
};
template <int DP>
__device__ __forceinline__ uint32_t chunk_at(uint32_t tile, int row, int c) {
  return tile + row * Planes<DP>::RB + ((c ^ (row & 7)) << 4);
}

// Rows [r0, r1) (r1 - r0 <= 64) of a row-major [..][d] matrix as 64 rows x DP features,
// zeros elsewhere: this thread's pieces of 8 features, and from there to a tile's planes.
// All pieces are asked for at once, and for wide heads, where one block fills an SM, before
// the products of the tile before if registers allow it (8 heads of 128, 2432 tokens all
// visible: forward 487 -> 416 us, dQ 653 -> 605 us).
template <int DP>
struct Pieces {
  static constexpr int N = WT * DP / 8 / kThreads;
  float4 x[N], y[N];
  __device__ __forceinline__ void fetch(const float* g, int d, int r0, int r1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = threadIdx.x + i * kThreads, r = r0 + id / (DP / 8), c = id % (DP / 8);
      x[i] = y[i] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (r < r1 && 8 * c < d) {
        const float* p = g + (size_t)r * d + 8 * c;
        x[i] = ld4(p);
        y[i] = ld4(p + 4);
      }
    }
  }
  __device__ __forceinline__ void place(uint32_t tile) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int id = threadIdx.x + i * kThreads;
      uint32_t w[4][3];
      split3_bf16x2(x[i].x, x[i].y, w[0]);
      split3_bf16x2(x[i].z, x[i].w, w[1]);
      split3_bf16x2(y[i].x, y[i].y, w[2]);
      split3_bf16x2(y[i].z, y[i].w, w[3]);
      const uint32_t at = chunk_at<DP>(tile, id / (DP / 8), id % (DP / 8));
#pragma unroll
      for (int q = 0; q < 3; ++q)
        asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at + q * Planes<DP>::PL),
                     "r"(w[0][q]), "r"(w[1][q]), "r"(w[2][q]), "r"(w[3][q])
                     : "memory");
    }
  }
};
template <int DP>
__device__ __forceinline__ void load_planes(uint32_t tile, const float* g, int d, int r0, int r1) {
  Pieces<DP> x;
  x.fetch(g, d, r0, r1);
  x.place(tile);
}

__device__ __forceinline__ void ldm(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void ldm_t(uint32_t (&r)[4], uint32_t at) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(at)
               : "memory");
}
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// two neighbouring tiles of 8 columns: the six products, the smallest first
__device__ __forceinline__ void six(float (&s)[4], float (&t)[4], const uint32_t (&a)[3][4],
                                    const uint32_t (&b)[3][4]) {
#pragma unroll
  for (int x = 2; x >= 0; --x)
#pragma unroll
    for (int y = 0; y <= x; ++y) {
      mma(s, a[y], b[x - y][0], b[x - y][1]);
      mma(t, a[y], b[x - y][2], b[x - y][3]);
    }
}

// s = rows [r0, r0 + 16) of X times rows [c0, c0 + 32) of Y, over d features: value
// [n][2 h + e] is row r0 + lane / 4 + 8 h, column c0 + 8 n + 2 (lane % 4) + e
template <int DP>
__device__ __forceinline__ void dot_rows(uint32_t X, uint32_t Y, int d, int r0, int c0, float (&s)[4][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) s[n][e] = 0.f;
#pragma unroll 2
  for (int k = 0; k < d / 16; ++k) {
    uint32_t x[3][4];
    const uint32_t at = chunk_at<DP>(X, r0 + (lane & 15), 2 * k + (lane >> 4));
#pragma unroll
    for (int q = 0; q < 3; ++q) ldm(x[q], at + q * Planes<DP>::PL);
#pragma unroll
    for (int n = 0; n < 2; ++n) {
      uint32_t y[3][4];
      const uint32_t by = chunk_at<DP>(Y, c0 + 16 * n + (lane & 7) + 8 * (lane >> 4), 2 * k + (lane >> 3 & 1));
#pragma unroll
      for (int q = 0; q < 3; ++q) ldm(y[q], by + q * Planes<DP>::PL);
      float t[2][4];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e >> 2][e & 3] = 0.f;
      six(t[0], t[1], x, y);
#pragma unroll
      for (int e = 0; e < 8; ++e) s[2 * n + (e >> 2)][e & 3] += t[e >> 2][e & 3];
    }
  }
}

// values of dot_rows' layout as the left operand of add_rows
__device__ __forceinline__ void as_left(const float (&p)[4][4], uint32_t (&w)[2][3][4]) {
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      uint32_t u[3];
      split3_bf16x2(p[2 * k + (e >> 1)][2 * (e & 1)], p[2 * k + (e >> 1)][2 * (e & 1) + 1], u);
#pragma unroll
      for (int q = 0; q < 3; ++q) w[k][q][e] = u[q];
    }
}
// o = f o + W Y: W 16 x 32, Y rows [c0, c0 + 32); [n] is 8 features in dot_rows' layout
template <int DP>
__device__ __forceinline__ void add_rows(const uint32_t (&w)[2][3][4], uint32_t Y, int d, int c0,
                                         const float (&f)[2], float (&o)[DP / 8][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DP / 16; ++n) {
    if (16 * n >= d) break;
    float t[2][4];
#pragma unroll
    for (int e = 0; e < 8; ++e) t[e >> 2][e & 3] = 0.f;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t y[3][4];
      const uint32_t at = chunk_at<DP>(Y, c0 + 16 * k + (lane & 15), 2 * n + (lane >> 4));
#pragma unroll
      for (int q = 0; q < 3; ++q) ldm_t(y[q], at + q * Planes<DP>::PL);
      six(t[0], t[1], w[k], y);
    }
#pragma unroll
    for (int e = 0; e < 8; ++e)
      o[2 * n + (e >> 2)][e & 3] = fmaf(o[2 * n + (e >> 2)][e & 3], f[e >> 1 & 1], t[e >> 2][e & 3]);
  }
}

// maximum or sum over the four threads of a row
__device__ __forceinline__ float row_max(float v) {
  v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
  return fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
}
__device__ __forceinline__ float row_sum(float v) {
  v += __shfl_xor_sync(0xffffffffu, v, 1);
  return v + __shfl_xor_sync(0xffffffffu, v, 2);
}

// One half's 16 x DP sums to shared memory for the other's warp of the same rows, and
// from there: rows of DP + 8 floats, a warp's 16 rows from `at` on
template <int DP>
__device__ __forceinline__ void give(float* at, const float (&o)[DP / 8][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h)
      *reinterpret_cast<float2*>(at + ((lane >> 2) + 8 * h) * (DP + 8) + 8 * n + 2 * (lane & 3)) =
          make_float2(o[n][2 * h], o[n][2 * h + 1]);
}
// o = f o + g what was given
template <int DP>
__device__ __forceinline__ void take(const float* at, const float (&f)[2], const float (&g)[2],
                                     float (&o)[DP / 8][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float2 x = *reinterpret_cast<const float2*>(at + ((lane >> 2) + 8 * h) * (DP + 8) + 8 * n + 2 * (lane & 3));
      o[n][2 * h] = fmaf(x.x, g[h], o[n][2 * h] * f[h]);
      o[n][2 * h + 1] = fmaf(x.y, g[h], o[n][2 * h + 1] * f[h]);
    }
}
// a row's share of o, times w, to memory
template <int DP>
__device__ __forceinline__ void put_row(float* dst, int d, int h, float w, const float (&o)[DP / 8][4]) {
  const int tq = threadIdx.x & 3;
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
    if (8 * n < d)
      *reinterpret_cast<float2*>(dst + 8 * n + 2 * tq) = make_float2(o[n][2 * h] * w, o[n][2 * h + 1] * w);
}
}  // namespace

template <int DP>
__global__ void __launch_bounds__(kThreads) k_win_fwd(WinArgs a) {
  extern __shared__ __align__(128) uint8_t smw[];
  using T = Planes<DP>;
  const uint32_t Q = smem_addr(smw), K = Q + T::BYTES, V = K + T::BYTES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tq = lane & 3;
  const int r0 = 16 * (warp & 3), half = warp >> 2, c0 = 32 * half;
  const int qt = (a.Nq + WT - 1) / WT;
  const int h = (blockIdx.x / qt) % a.Hq, b = (blockIdx.x / qt) / a.Hq;
  const int i0 = (blockIdx.x % qt) * WT, i1 = min(a.Nq, i0 + WT);
  const WinSeq sq = win_seq(a, b);
  const WinRange kr = win_keys(a, sq, i0, i1);
  const size_t kv0 = ((size_t)b * a.Hkv + h / a.g) * a.Nk * a.d;
  const size_t q0 = ((size_t)b * a.Hq + h) * a.Nq;
  load_planes<DP>(Q, (const float*)a.q + q0 * a.d, a.d, i0, i1);

  WinRow row[2];
  float m[2], l[2];
  float o[DP / 8][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    row[r] = win_row(a, sq, i0 + r0 + gid + 8 * r);
    m[r] = -INFINITY;
    l[r] = 0.f;
  }
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  constexpr bool AHEAD = DP == 128;
  const int ns = (kr.S + WT - 1) / WT, steps = ns + (kr.hi - kr.lo + WT - 1) / WT;
  Pieces<DP> kp, vp;
  auto fetch = [&](int t) {
    const int j0 = t < ns ? t * WT : kr.lo + (t - ns) * WT, je = min(t < ns ? kr.S : kr.hi, j0 + WT);
    kp.fetch((const float*)a.k + kv0, a.d, j0, je);
    vp.fetch((const float*)a.v + kv0, a.d, j0, je);
  };
  if (AHEAD && steps > 0) fetch(0);
#pragma unroll 1
  for (int t = 0; t < steps; ++t) {
    const int j0 = t < ns ? t * WT : kr.lo + (t - ns) * WT, je = min(t < ns ? kr.S : kr.hi, j0 + WT);
    if (!AHEAD) fetch(t);
    __syncthreads();
    kp.place(K);
    vp.place(V);
    __syncthreads();
    if (AHEAD && t + 1 < steps) fetch(t + 1);
    if (j0 + c0 >= je) continue;
    float s[4][4], f[2];
    dot_rows<DP>(Q, K, a.d, r0, c0, s);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float mx = -INFINITY;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = j0 + c0 + 8 * (e >> 1) + 2 * tq + (e & 1);
        float& x = s[e >> 1][2 * r + (e & 1)];
        x = j < je && win_sees(row[r], j) ? x * a.scale_log2 : -INFINITY;
        mx = fmaxf(mx, x);
      }
      mx = fmaxf(m[r], row_max(mx));
      const float mu = mx == -INFINITY ? 0.f : mx;
      f[r] = exp2f(m[r] - mu);
      m[r] = mx;
      float sum = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float& x = s[e >> 1][2 * r + (e & 1)];
        x = exp2f(x - mu);
        sum += x;
      }
      l[r] = l[r] * f[r] + row_sum(sum);
    }
    uint32_t w[2][3][4];
    as_left(s, w);
    add_rows<DP>(w, V, a.d, c0, f, o);
  }
  __syncthreads();
  // the halves' sums, over the same maximum
  float* buf = reinterpret_cast<float*>(smw) + r0 * (DP + 8);
  float2* ml = reinterpret_cast<float2*>(reinterpret_cast<float*>(smw) + WT * (DP + 8)) + r0;
  if (half) {
    give<DP>(buf, o);
#pragma unroll
    for (int r = 0; r < 2; ++r)
      if (tq == 0) ml[gid + 8 * r] = make_float2(m[r], l[r]);
  }
  __syncthreads();
  if (half) return;
  float f[2], g[2];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const float2 x = ml[gid + 8 * r];
    const float mx = fmaxf(m[r], x.x), mu = mx == -INFINITY ? 0.f : mx;
    f[r] = exp2f(m[r] - mu);
    g[r] = exp2f(x.x - mu);
    l[r] = fmaf(l[r], f[r], x.y * g[r]);
    m[r] = mx;
  }
  take<DP>(buf, f, g, o);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = i0 + r0 + gid + 8 * r;
    if (i >= i1) continue;
    const float w = l[r] > 0.f ? 1.f / l[r] : (l[r] == 0.f ? 0.f : l[r]);
    if (a.lse && tq == 0) a.lse[q0 + i] = l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
    put_row<DP>((float*)a.out + (q0 + i) * a.d, a.d, r, w, o);
  }
}

// dQ of one tile of queries, and D = dout.o of its rows for the kernel below
template <int DP>
__global__ void __launch_bounds__(kThreads) k_win_dq(WinArgs a) {
  extern __shared__ __align__(128) uint8_t smw[];
  using T = Planes<DP>;
  const uint32_t Q = smem_addr(smw), O = Q + T::BYTES, K = O + T::BYTES, V = K + T::BYTES;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tq = lane & 3;
  const int r0 = 16 * (warp & 3), half = warp >> 2, c0 = 32 * half;
  const int qt = (a.Nq + WT - 1) / WT;
  const int h = (blockIdx.x / qt) % a.Hq, b = (blockIdx.x / qt) / a.Hq;
  const int i0 = (blockIdx.x % qt) * WT, i1 = min(a.Nq, i0 + WT);
  const WinSeq sq = win_seq(a, b);
  const WinRange kr = win_keys(a, sq, i0, i1);
  const size_t kv0 = ((size_t)b * a.Hkv + h / a.g) * a.Nk * a.d;
  const size_t q0 = ((size_t)b * a.Hq + h) * a.Nq;
  load_planes<DP>(Q, (const float*)a.q + q0 * a.d, a.d, i0, i1);
  load_planes<DP>(O, (const float*)a.dout + q0 * a.d, a.d, i0, i1);

  WinRow row[2];
  float ls[2], D[2];
  float o[DP / 8][4];
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = i0 + r0 + gid + 8 * r;
    row[r] = win_row(a, sq, i);
    ls[r] = i < i1 ? a.lse[q0 + i] : 0.f;
    float s = 0.f;
    for (int c = 4 * tq; i < i1 && c < a.d; c += 16) {
      const float4 x = ld4((const float*)a.dout + (q0 + i) * a.d + c);
      const float4 y = ld4((const float*)a.out + (q0 + i) * a.d + c);
      s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
    }
    D[r] = row_sum(s);
    if (half == 0 && tq == 0 && i < i1) a.D[q0 + i] = D[r];
  }
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;
  const float one[2] = {1.f, 1.f};
  constexpr bool AHEAD = DP == 128;
  const int ns = (kr.S + WT - 1) / WT, steps = ns + (kr.hi - kr.lo + WT - 1) / WT;
  Pieces<DP> kp, vp;
  auto fetch = [&](int t) {
    const int j0 = t < ns ? t * WT : kr.lo + (t - ns) * WT, je = min(t < ns ? kr.S : kr.hi, j0 + WT);
    kp.fetch((const float*)a.k + kv0, a.d, j0, je);
    vp.fetch((const float*)a.v + kv0, a.d, j0, je);
  };
  if (AHEAD && steps > 0) fetch(0);
#pragma unroll 1
  for (int t = 0; t < steps; ++t) {
    const int j0 = t < ns ? t * WT : kr.lo + (t - ns) * WT, je = min(t < ns ? kr.S : kr.hi, j0 + WT);
    if (!AHEAD) fetch(t);
    __syncthreads();
    kp.place(K);
    vp.place(V);
    __syncthreads();
    if (AHEAD && t + 1 < steps) fetch(t + 1);
    if (j0 + c0 >= je) continue;
    float s[4][4], dp[4][4];
    dot_rows<DP>(Q, K, a.d, r0, c0, s);
    dot_rows<DP>(O, V, a.d, r0, c0, dp);
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int r = e >> 1, j = j0 + c0 + 8 * n + 2 * tq + (e & 1);
        const bool see = j < je && win_sees(row[r], j);
        s[n][e] = see ? exp2f(fmaf(s[n][e], a.scale_log2, -ls[r])) * (dp[n][e] - D[r]) : 0.f;
      }
    uint32_t w[2][3][4];
    as_left(s, w);
    add_rows<DP>(w, K, a.d, c0, one, o);
  }
  __syncthreads();
  float* buf = reinterpret_cast<float*>(smw) + r0 * (DP + 8);
  if (half) give<DP>(buf, o);
  __syncthreads();
  if (half) return;
  take<DP>(buf, one, one, o);
#pragma unroll
  for (int r = 0; r < 2; ++r) {
    const int i = i0 + r0 + gid + 8 * r;
    if (i < i1) put_row<DP>((float*)a.dq + (q0 + i) * a.d, a.d, r, a.scale, o);
  }
}

// dK and dV of one tile of keys, over the queries (and the group's heads) that
// see it.  The first `stiles` tiles (with first tokens, which every later query sees; or all
// of them, where few tiles have many queries each) have their queries cut into `chunks` ranges
// of `chunk_rows`, one block each, whose fp32 partials k_win_join adds in their order.  Heads to 64: two blocks of an SM, at the
// price of some spilled registers (16 heads, 2432 tokens all visible: 890 -> 759 us).
template <int DP>
__global__ void __launch_bounds__(kThreads, DP == 64 ? 2 : 1) k_win_dkv(WinArgs a) {
  extern __shared__ __align__(128) uint8_t smw[];
  using T = Planes<DP>;
  const uint32_t K = smem_addr(smw), V = K + T::BYTES, Q = V + T::BYTES, O = Q + T::BYTES;
  float* Ls = reinterpret_cast<float*>(smw + 4 * T::BYTES);   // log-sum and D of the tile's queries
  float* Ds = Ls + WT;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, gid = lane >> 2, tq = lane & 3;
  const int r0 = 16 * (warp & 3), half = warp >> 2, c0 = 32 * half;
  const int kt = (a.Nk + WT - 1) / WT, items = a.stiles * a.chunks + kt - a.stiles;
  const int it = blockIdx.x % items, hk = (blockIdx.x / items) % a.Hkv, b = (blockIdx.x / items) / a.Hkv;
  const bool first = it < a.stiles * a.chunks;
  const int tile = first ? it / a.chunks : it - a.stiles * (a.chunks - 1);
  const int j0 = tile * WT;
  const WinSeq sq = win_seq(a, b);
  const int j1 = min(min(a.Nk, j0 + WT), sq.len);
  int i0, i1;
  win_queries(a, sq, j0, j1, &i0, &i1);
  if (first) {
    const int c = it % a.chunks;
    i0 = max(i0, c * a.chunk_rows);
    i1 = min(i1, (c + 1) * a.chunk_rows);
  }
  const size_t kv0 = ((size_t)b * a.Hkv + hk) * a.Nk;
  load_planes<DP>(K, (const float*)a.k + kv0 * a.d, a.d, j0, j1);
  load_planes<DP>(V, (const float*)a.v + kv0 * a.d, a.d, j0, j1);
  float dk[DP / 8][4], dv[DP / 8][4];
#pragma unroll
  for (int n = 0; n < DP / 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) dk[n][e] = dv[n][e] = 0.f;
  const float one[2] = {1.f, 1.f};
  for (int e = 0; e < a.g; ++e) {
    const size_t q0 = ((size_t)b * a.Hq + hk * a.g + e) * a.Nq;
#pragma unroll 1
    for (int i = i0; i < i1; i += WT) {
      const int ie = min(i1, i + WT);
      Pieces<DP> qp, op;
      qp.fetch((const float*)a.q + q0 * a.d, a.d, i, ie);
      op.fetch((const float*)a.dout + q0 * a.d, a.d, i, ie);
      __syncthreads();
      qp.place(Q);
      op.place(O);
      if (tid < WT) {
        Ls[tid] = i + tid < ie ? a.lse[q0 + i + tid] : 0.f;
        Ds[tid] = i + tid < ie ? a.D[q0 + i + tid] : 0.f;
      }
      __syncthreads();
      if (i + c0 >= ie) continue;
      float s[4][4], dp[4][4];
      dot_rows<DP>(K, Q, a.d, r0, c0, s);
      uint32_t seen = 0;
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const int ii = c0 + 8 * n + 2 * tq + c;
          const WinRow row = i + ii < ie ? win_row(a, sq, i + ii) : WinRow{0, 0, 0};
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int j = j0 + r0 + gid + 8 * r;
            const bool see = j < j1 && win_sees(row, j);
            seen |= (uint32_t)see << (4 * n + 2 * r + c);
            s[n][2 * r + c] = see ? exp2f(fmaf(s[n][2 * r + c], a.scale_log2, -Ls[ii])) : 0.f;
          }
        }
      uint32_t w[2][3][4];
      as_left(s, w);
      add_rows<DP>(w, O, a.d, c0, one, dv);
      dot_rows<DP>(V, O, a.d, r0, c0, dp);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int x = 0; x < 4; ++x)
          s[n][x] = seen >> (4 * n + x) & 1u ? s[n][x] * (dp[n][x] - Ds[c0 + 8 * n + 2 * tq + (x & 1)]) : 0.f;
      as_left(s, w);
      add_rows<DP>(w, Q, a.d, c0, one, dk);
    }
  }
  __syncthreads();
  // dK is put together by the first half's warps, dV by the other's
  float* mine = reinterpret_cast<float*>(smw) + (size_t)(WT * half + r0) * (DP + 8);
  float* other = reinterpret_cast<float*>(smw) + (size_t)(WT * (1 - half) + r0) * (DP + 8);
  if (half)
    give<DP>(other, dk);
  else
    give<DP>(other, dv);
  __syncthreads();
  float* part = first ? a.part + ((((size_t)b * a.Hkv + hk) * a.stiles + tile) * a.chunks + it % a.chunks) *
                                     2 * WT * a.d
                      : nullptr;
  auto put = [&](float (&g)[DP / 8][4], float* grad, float* to, float f) {
    take<DP>(mine, one, one, g);
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int k = r0 + gid + 8 * r;
      if (first)
        put_row<DP>(to + (size_t)k * a.d, a.d, r, f, g);
      else if (j0 + k < a.Nk)
        put_row<DP>(grad + (kv0 + j0 + k) * a.d, a.d, r, f, g);
    }
  };
  if (half)
    put(dv, (float*)a.dv, part + (size_t)WT * a.d, 1.f);
  else
    put(dk, (float*)a.dk, part, a.scale);
}

// dK and dV of the tiles whose queries were cut: the ranges' partials, added in
// their order and rounded once
template <typename T>
__global__ void __launch_bounds__(256) k_win_join(WinArgs a, int tile_rows) {
  const int d4 = a.d / 4;
  const long long n = (long long)a.B * a.Hkv * a.stiles * 2 * tile_rows * d4;
  for (long long e = (long long)blockIdx.x * blockDim.x + threadIdx.x; e < n;
       e += (long long)gridDim.x * blockDim.x) {
    const int c = (int)(e % d4) * 4;
    const int row = (int)(e / d4 % tile_rows);
    const int which = (int)(e / d4 / tile_rows % 2);
    const long long t = e / d4 / tile_rows / 2;
    const int tile = (int)(t % a.stiles);
    const long long bh = t / a.stiles;
    const int j = tile * tile_rows + row;
    if (j >= a.Nk) continue;
    const float* p = a.part + ((t * a.chunks * 2 + which) * tile_rows + row) * a.d + c;
    float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int k = 0; k < a.chunks; ++k) {
      const float4 x = ld4(p + (size_t)k * 2 * tile_rows * a.d);
      s.x += x.x; s.y += x.y; s.z += x.z; s.w += x.w;
    }
    st4((T*)(which ? a.dv : a.dk) + ((size_t)bh * a.Nk + j) * a.d + c, s);
  }
}

namespace {
template <int DP>
cudaError_t fwd_t(const WinArgs& a, cudaStream_t st) {
  constexpr size_t smem = 3 * Planes<DP>::BYTES;
  static_assert(smem >= (WT * (DP + 8) + 2 * WT) * 4);
  static SmemOnce once;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once.allow(k_win_fwd<DP>, smem, dev)) != cudaSuccess) return e;
  const long long n = (long long)a.B * a.Hq * ((a.Nq + WT - 1) / WT);
  return launch("win_fwd", k_win_fwd<DP>, dim3((unsigned)n), dim3(kThreads), smem, st, a);
}
template <int DP>
cudaError_t bwd_t(const WinArgs& a, cudaStream_t st) {
  constexpr size_t sq = 4 * Planes<DP>::BYTES, sk = sq + 2 * WT * 4;
  static_assert(sq >= 2 * WT * (DP + 8) * 4);
  static SmemOnce once_q, once_kv;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once_q.allow(k_win_dq<DP>, sq, dev)) != cudaSuccess ||
      (e = once_kv.allow(k_win_dkv<DP>, sk, dev)) != cudaSuccess)
    return e;
  const long long nq = (long long)a.B * a.Hq * ((a.Nq + WT - 1) / WT);
  e = launch("win_dq", k_win_dq<DP>, dim3((unsigned)nq), dim3(kThreads), sq, st, a);
  if (e != cudaSuccess) return e;
  const int kt = (a.Nk + WT - 1) / WT;
  const long long nk = (long long)a.B * a.Hkv * (a.stiles * a.chunks + kt - a.stiles);
  e = launch("win_dkv", k_win_dkv<DP>, dim3((unsigned)nk), dim3(kThreads), sk, st, a);
  if (e != cudaSuccess || a.stiles == 0) return e;
  return run_win_join(a, WT, false, st);
}
}  // namespace

cudaError_t run_win_join(const WinArgs& a, int tile_rows, bool bf16, cudaStream_t st) {
  const long long n = (long long)a.B * a.Hkv * a.stiles * 2 * tile_rows * (a.d / 4);
  const unsigned g = (unsigned)((n + 255) / 256 < 4096 ? (n + 255) / 256 : 4096);
  if (bf16)
    return launch("win_join", k_win_join<__nv_bfloat16>, dim3(g), dim3(256), 0, st, a, tile_rows);
  return launch("win_join", k_win_join<float>, dim3(g), dim3(256), 0, st, a, tile_rows);
}

int win_tile_rows() { return WT; }

cudaError_t run_win_fwd(const WinArgs& a, cudaStream_t st) {
  return a.d <= 64 ? fwd_t<64>(a, st) : fwd_t<128>(a, st);
}

cudaError_t run_win_bwd(const WinArgs& a, cudaStream_t st) {
  return a.d <= 64 ? bwd_t<64>(a, st) : bwd_t<128>(a, st);
}

}  // namespace lapnys
