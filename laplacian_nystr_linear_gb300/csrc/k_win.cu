// Windowed softmax attention of fp32 tensors on the FP32 pipe (visibility rule:
// win.cuh): forward, query gradients, key and value gradients.
//
//   s = scale q.k over the visible keys, P = softmax(s), o = P v
//   D = dout.o, dV = P^T dout, dP = dout V^T, dS = P (dP - D),
//   dQ = scale dS K, dK = scale dS^T Q  (both summed over a group's query heads)
//
// One pass over the keys with the running maximum and sum of each row's softmax;
// the backward recomputes P from the saved log-sum.  Tiles of 64 queries x 64
// keys, 256 threads as 16 x 16, each thread 4 x 4 scores and 4 rows x DP / 16
// columns of the outputs in registers; operand tiles in padded shared memory.
// Rows of one tile belong to one half-warp, so P goes through shared memory
// with a warp barrier only.  Bound by the FP32 pipe: 4 d (forward) and 14 d
// (backward, scores recomputed in both kernels) operations per visible pair; by its
// latency where there are few tiles (196 tokens, one head of 32: 32, 35 and 47 us for 4
// blocks of one to two steps, beside 100 us and more of the host's work for the call).
#include "common.cuh"
#include "internal.h"
#include "win.cuh"

namespace lapnys {

namespace {
constexpr int WT = 64;        // queries and keys of a tile
constexpr int WPS = WT + 4;   // row stride of the P tiles

// rows [r0, r1) (r1 - r0 <= 64) of a row-major [..][d] matrix into a padded
// tile of 64 rows x DP columns, zeros elsewhere
template <int DP>
__device__ __forceinline__ void win_load(float* s, const float* g, int d, int r0, int r1) {
  constexpr int C4 = DP / 4;
  for (int id = threadIdx.x; id < WT * C4; id += kThreads) {
    const int r = id / C4, c = (id % C4) * 4;
    float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r0 + r < r1 && c < d) v = ld4(g + (size_t)(r0 + r) * d + c);
    st4(s + r * row_stride(DP) + c, v);
  }
}

// s[r][c] = X[4 ty + r] . Y[tx + 16 c]
template <int DP>
__device__ __forceinline__ void win_dot(const float* Xs, const float* Ys, int ty, int tx,
                                        float (&s)[4][4]) {
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int c = 0; c < 4; ++c) s[r][c] = 0.f;
#pragma unroll 4
  for (int e = 0; e < DP; e += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) x[r] = lds4(Xs + (4 * ty + r) * row_stride(DP) + e);
#pragma unroll
    for (int c = 0; c < 4; ++c) y[c] = lds4(Ys + (tx + 16 * c) * row_stride(DP) + e);
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        s[r][c] = fmaf(x[r].x, y[c].x, s[r][c]);
        s[r][c] = fmaf(x[r].y, y[c].y, s[r][c]);
        s[r][c] = fmaf(x[r].z, y[c].z, s[r][c]);
        s[r][c] = fmaf(x[r].w, y[c].w, s[r][c]);
      }
  }
}

// o[r][..] += sum_j P[4 ty + r][j] Y[j][..]; thread tx owns columns 4 tx + 64 u
template <int DP>
__device__ __forceinline__ void win_acc(const float* Ps, const float* Ys, int ty, int tx,
                                        float4 (&o)[4][DP / 64]) {
#pragma unroll 2
  for (int j = 0; j < WT; j += 4) {
    float4 p[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) p[r] = lds4(Ps + (4 * ty + r) * WPS + j);
#pragma unroll
    for (int e = 0; e < 4; ++e)
#pragma unroll
      for (int u = 0; u < DP / 64; ++u) {
        const float4 y = lds4(Ys + (j + e) * row_stride(DP) + 4 * tx + 64 * u);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const float w = comp(p[r], e);
          o[r][u].x = fmaf(w, y.x, o[r][u].x);
          o[r][u].y = fmaf(w, y.y, o[r][u].y);
          o[r][u].z = fmaf(w, y.z, o[r][u].z);
          o[r][u].w = fmaf(w, y.w, o[r][u].w);
        }
      }
  }
}

// sum or maximum over the 16 threads of a row
__device__ __forceinline__ float row_max(float v) {
#pragma unroll
  for (int k = 8; k; k >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, k));
  return v;
}
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int k = 8; k; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
  return v;
}
}  // namespace

template <int DP>
__global__ void __launch_bounds__(kThreads) k_win_fwd(WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Ks = Qs + WT * row_stride(DP);
  float* Vs = Ks + WT * row_stride(DP);
  float* Ps = Vs + WT * row_stride(DP);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int qt = (a.Nq + WT - 1) / WT;
  const int h = (blockIdx.x / qt) % a.Hq, b = (blockIdx.x / qt) / a.Hq;
  const int i0 = (blockIdx.x % qt) * WT, i1 = min(a.Nq, i0 + WT);
  const WinSeq sq = win_seq(a, b);
  const WinRange kr = win_keys(a, sq, i0, i1);
  const size_t kv0 = ((size_t)b * a.Hkv + h / a.g) * a.Nk * a.d;
  const float* K = (const float*)a.k + kv0;
  const float* V = (const float*)a.v + kv0;
  const size_t q0 = ((size_t)b * a.Hq + h) * a.Nq;
  win_load<DP>(Qs, (const float*)a.q + q0 * a.d, a.d, i0, i1);

  WinRow row[4];
  float m[4], l[4];
  float4 o[4][DP / 64];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    row[r] = win_row(a, sq, i0 + 4 * ty + r);
    m[r] = -INFINITY;
    l[r] = 0.f;
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) o[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  }
  for (int seg = 0; seg < 2; ++seg) {
    const int jb = seg ? kr.lo : 0, je = seg ? kr.hi : kr.S;
    for (int j0 = jb; j0 < je; j0 += WT) {
      __syncthreads();
      win_load<DP>(Ks, K, a.d, j0, min(je, j0 + WT));
      win_load<DP>(Vs, V, a.d, j0, min(je, j0 + WT));
      __syncthreads();
      float s[4][4];
      win_dot<DP>(Qs, Ks, ty, tx, s);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        float mx = -INFINITY;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + tx + 16 * c;
          s[r][c] = j < je && win_sees(row[r], j) ? s[r][c] * a.scale_log2 : -INFINITY;
          mx = fmaxf(mx, s[r][c]);
        }
        mx = fmaxf(m[r], row_max(mx));
        const float mu = mx == -INFINITY ? 0.f : mx;
        const float f = exp2f(m[r] - mu);
        m[r] = mx;
        float sum = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const float p = exp2f(s[r][c] - mu);
          sum += p;
          Ps[(4 * ty + r) * WPS + tx + 16 * c] = p;
        }
        l[r] = l[r] * f + row_sum(sum);
#pragma unroll
        for (int u = 0; u < DP / 64; ++u) {
          o[r][u].x *= f; o[r][u].y *= f; o[r][u].z *= f; o[r][u].w *= f;
        }
      }
      __syncwarp();
      win_acc<DP>(Ps, Vs, ty, tx, o);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    if (i >= i1) continue;
    const float w = l[r] > 0.f ? 1.f / l[r] : (l[r] == 0.f ? 0.f : l[r]);
    if (a.lse && tx == 0) a.lse[q0 + i] = l[r] == 0.f ? -INFINITY : m[r] + log2f(l[r]);
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) {
      const int c = 4 * tx + 64 * u;
      if (c < a.d)
        st4((float*)a.out + (q0 + i) * a.d + c,
            make_float4(o[r][u].x * w, o[r][u].y * w, o[r][u].z * w, o[r][u].w * w));
    }
  }
}

// dQ of one tile of queries, and D = dout.o of its rows for the kernel below
template <int DP>
__global__ void __launch_bounds__(kThreads) k_win_dq(WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Qs = sm;
  float* Os = Qs + WT * row_stride(DP);
  float* Ks = Os + WT * row_stride(DP);
  float* Vs = Ks + WT * row_stride(DP);
  float* Ps = Vs + WT * row_stride(DP);
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int qt = (a.Nq + WT - 1) / WT;
  const int h = (blockIdx.x / qt) % a.Hq, b = (blockIdx.x / qt) / a.Hq;
  const int i0 = (blockIdx.x % qt) * WT, i1 = min(a.Nq, i0 + WT);
  const WinSeq sq = win_seq(a, b);
  const WinRange kr = win_keys(a, sq, i0, i1);
  const size_t kv0 = ((size_t)b * a.Hkv + h / a.g) * a.Nk * a.d;
  const float* K = (const float*)a.k + kv0;
  const float* V = (const float*)a.v + kv0;
  const size_t q0 = ((size_t)b * a.Hq + h) * a.Nq;
  win_load<DP>(Qs, (const float*)a.q + q0 * a.d, a.d, i0, i1);
  win_load<DP>(Os, (const float*)a.dout + q0 * a.d, a.d, i0, i1);

  WinRow row[4];
  float ls[4], D[4];
  float4 o[4][DP / 64];
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    row[r] = win_row(a, sq, i);
    ls[r] = i < i1 ? a.lse[q0 + i] : 0.f;
    float s = 0.f;
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) {
      o[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
      const int c = 4 * tx + 64 * u;
      if (i < i1 && c < a.d) {
        const float4 x = ld4((const float*)a.dout + (q0 + i) * a.d + c);
        const float4 y = ld4((const float*)a.out + (q0 + i) * a.d + c);
        s = fmaf(x.x, y.x, fmaf(x.y, y.y, fmaf(x.z, y.z, fmaf(x.w, y.w, s))));
      }
    }
    D[r] = row_sum(s);
    if (tx == 0 && i < i1) a.D[q0 + i] = D[r];
  }
  for (int seg = 0; seg < 2; ++seg) {
    const int jb = seg ? kr.lo : 0, je = seg ? kr.hi : kr.S;
    for (int j0 = jb; j0 < je; j0 += WT) {
      __syncthreads();
      win_load<DP>(Ks, K, a.d, j0, min(je, j0 + WT));
      win_load<DP>(Vs, V, a.d, j0, min(je, j0 + WT));
      __syncthreads();
      float s[4][4], dp[4][4];
      win_dot<DP>(Qs, Ks, ty, tx, s);
      win_dot<DP>(Os, Vs, ty, tx, dp);
#pragma unroll
      for (int r = 0; r < 4; ++r)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const int j = j0 + tx + 16 * c;
          const bool see = j < je && win_sees(row[r], j);
          Ps[(4 * ty + r) * WPS + tx + 16 * c] =
              see ? exp2f(fmaf(s[r][c], a.scale_log2, -ls[r])) * (dp[r][c] - D[r]) : 0.f;
        }
      __syncwarp();
      win_acc<DP>(Ps, Ks, ty, tx, o);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int i = i0 + 4 * ty + r;
    if (i >= i1) continue;
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) {
      const int c = 4 * tx + 64 * u;
      if (c < a.d)
        st4((float*)a.dq + (q0 + i) * a.d + c,
            make_float4(o[r][u].x * a.scale, o[r][u].y * a.scale, o[r][u].z * a.scale,
                        o[r][u].w * a.scale));
    }
  }
}

// dK and dV of one tile of keys, over the queries (and the group's heads) that
// see it.  A tile that holds first tokens is seen by every later query: its
// queries are cut into `chunks` ranges of `chunk_rows`, one block each, whose
// fp32 partials k_win_join adds in their order.
template <int DP>
__global__ void __launch_bounds__(kThreads) k_win_dkv(WinArgs a) {
  extern __shared__ __align__(16) float sm[];
  float* Ks = sm;
  float* Vs = Ks + WT * row_stride(DP);
  float* Qs = Vs + WT * row_stride(DP);
  float* Os = Qs + WT * row_stride(DP);
  float* Ps = Os + WT * row_stride(DP);
  float* Ss = Ps + WT * WPS;
  float* Ls = Ss + WT * WPS;   // log-sum and D of the tile's queries
  float* Ds = Ls + WT;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
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
  win_load<DP>(Ks, (const float*)a.k + kv0 * a.d, a.d, j0, j1);
  win_load<DP>(Vs, (const float*)a.v + kv0 * a.d, a.d, j0, j1);
  float4 dk[4][DP / 64], dv[4][DP / 64];
#pragma unroll
  for (int r = 0; r < 4; ++r)
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) dk[r][u] = dv[r][u] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int e = 0; e < a.g; ++e) {
    const size_t q0 = ((size_t)b * a.Hq + hk * a.g + e) * a.Nq;
    for (int i = i0; i < i1; i += WT) {
      const int ie = min(i1, i + WT);
      __syncthreads();
      win_load<DP>(Qs, (const float*)a.q + q0 * a.d, a.d, i, ie);
      win_load<DP>(Os, (const float*)a.dout + q0 * a.d, a.d, i, ie);
      if (tid < WT) {
        Ls[tid] = i + tid < ie ? a.lse[q0 + i + tid] : 0.f;
        Ds[tid] = i + tid < ie ? a.D[q0 + i + tid] : 0.f;
      }
      __syncthreads();
      float s[4][4], dp[4][4];
      win_dot<DP>(Ks, Qs, ty, tx, s);
      win_dot<DP>(Vs, Os, ty, tx, dp);
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int ii = tx + 16 * c;
        WinRow row = win_row(a, sq, i + ii);
        if (i + ii >= ie) row = WinRow{0, 0, 0};
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          const int j = j0 + 4 * ty + r;
          const float p =
              j < j1 && win_sees(row, j) ? exp2f(fmaf(s[r][c], a.scale_log2, -Ls[ii])) : 0.f;
          Ps[(4 * ty + r) * WPS + ii] = p;
          Ss[(4 * ty + r) * WPS + ii] = p != 0.f ? p * (dp[r][c] - Ds[ii]) : 0.f;
        }
      }
      __syncwarp();
      win_acc<DP>(Ps, Os, ty, tx, dv);
      win_acc<DP>(Ss, Qs, ty, tx, dk);
    }
  }
#pragma unroll
  for (int r = 0; r < 4; ++r) {
    const int row = 4 * ty + r, j = j0 + row;
#pragma unroll
    for (int u = 0; u < DP / 64; ++u) {
      const int c = 4 * tx + 64 * u;
      if (c >= a.d) continue;
      const float4 x = make_float4(dk[r][u].x * a.scale, dk[r][u].y * a.scale,
                                   dk[r][u].z * a.scale, dk[r][u].w * a.scale);
      if (first) {
        float* p = a.part + (((((size_t)b * a.Hkv + hk) * a.stiles + tile) * a.chunks +
                              it % a.chunks) * 2 * WT + row) * a.d + c;
        st4(p, x);
        st4(p + (size_t)WT * a.d, dv[r][u]);
      } else if (j < a.Nk) {
        st4((float*)a.dk + (kv0 + j) * a.d + c, x);
        st4((float*)a.dv + (kv0 + j) * a.d + c, dv[r][u]);
      }
    }
  }
}

// dK and dV of the tiles that hold first tokens: the chunks' partials, added in
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
  const size_t smem = (size_t)(3 * WT * row_stride(DP) + WT * WPS) * 4;
  static SmemOnce once;
  int dev = 0, sms = 0;
  cudaError_t e = device_sms(&dev, &sms);
  if (e != cudaSuccess || (e = once.allow(k_win_fwd<DP>, smem, dev)) != cudaSuccess) return e;
  const long long n = (long long)a.B * a.Hq * ((a.Nq + WT - 1) / WT);
  return launch("win_fwd", k_win_fwd<DP>, dim3((unsigned)n), dim3(kThreads), smem, st, a);
}
template <int DP>
cudaError_t bwd_t(const WinArgs& a, cudaStream_t st) {
  const size_t sq = (size_t)(4 * WT * row_stride(DP) + WT * WPS) * 4;
  const size_t sk = (size_t)(4 * WT * row_stride(DP) + 2 * WT * WPS + 2 * WT) * 4;
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
