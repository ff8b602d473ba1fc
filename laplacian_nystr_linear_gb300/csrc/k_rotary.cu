// Rotary positions: pairs of features turned by the token's position.
//
//   (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),  t = 2 pi p w_i,
// pair i of rot / 2: features (i, i + rot / 2) in the half layout, (2 i, 2 i + 1)
// interleaved; features from rot on pass unchanged.  w_i is in turns a position, as
// a fraction of 2^64: p w_i modulo 2^64 is the phase to 2^-64 of a turn for every
// 32-bit position, exactly, where 32-bit angles lose all of it (at p = 10^6 a
// rounded fp32 angle is off by 0.03).  The gradient is the turn back, by the same
// factor.
//
// Bound by memory: queries and keys are read and written once.  A thread keeps its
// pairs' cosines and sines in registers over the heads of its token, so they cost a
// few instructions a head; loads of four heads are in flight at once.
#include "common.cuh"
#include "internal.h"
#include "layer.cuh"

namespace lapnys {
namespace {

constexpr int RT = 128;   // threads of a block

// V elements at a time, 16 bytes of them or one
template <typename T, int V>
struct Piece {
  T v[V];
};
template <typename T, int V>
__device__ __forceinline__ Piece<T, V> get(const T* p) {
  Piece<T, V> r;
  if constexpr (V * sizeof(T) == 16)
    *reinterpret_cast<uint4*>(&r) = *reinterpret_cast<const uint4*>(p);
  else
#pragma unroll
    for (int i = 0; i < V; ++i) r.v[i] = p[i];
  return r;
}
template <typename T, int V>
__device__ __forceinline__ void put(T* p, const Piece<T, V>& r) {
  if constexpr (V * sizeof(T) == 16)
    *reinterpret_cast<uint4*>(p) = *reinterpret_cast<const uint4*>(&r);
  else
#pragma unroll
    for (int i = 0; i < V; ++i) p[i] = r.v[i];
}
__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ void of_f(float& o, float x) { o = x; }
__device__ __forceinline__ void of_f(__nv_bfloat16& o, float x) { o = __float2bfloat16_rn(x); }

// A work item is V pairs of a token in the half layout, V features interleaved
// (V / 2 pairs; one pair when V is 1), and last the pieces that are copied.
template <typename T, bool HALF, int V>
__global__ void __launch_bounds__(RT) k_rotary(RotaryArgs a) {
  constexpr bool PAIR = HALF || V == 1;          // two pieces an item, `gap` apart
  constexpr int P = PAIR ? V : V / 2;            // pairs of an item
  constexpr int DEEP = PAIR ? 4 : 8;             // heads in flight
  const long long id = (long long)blockIdx.x * RT + threadIdx.x;
  const long long tokens = (long long)a.B * a.N;
  const long long tok = id / a.units;
  const int unit = (int)(id - tok * a.units);
  if (tok >= tokens) return;
  const int b = (int)(tok / a.N), n = (int)(tok - (long long)b * a.N);
  const int turned = a.rot / (2 * P);
  const bool turn = unit < turned;
  int at, gap;
  bool second = PAIR;
  if (turn) {
    at = HALF ? unit * V : unit * (PAIR ? 2 : V);
    gap = HALF ? a.rot / 2 : 1;
  } else {                                       // copied: two pieces an item as well
    at = a.rot + (unit - turned) * (PAIR ? 2 * V : V);
    gap = V;
    second = PAIR && at + V < a.d;
  }
  float c[P], s[P];
  if (turn) {
    const int32_t p = a.positions ? a.positions[tok] : (a.start ? a.start[b] : 0) + n;
    const uint64_t at_p = (uint64_t)(int64_t)p;
    const int i0 = HALF ? unit * V : unit * P;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const uint64_t phase = at_p * __ldg(a.turns + i0 + i);
      // the upper 32 bits as half turns in [-1, 1)
      float sn, cs;
      sincospif((float)(int32_t)(phase >> 32) * 0x1p-31f, &sn, &cs);
      c[i] = cs * a.factor;
      s[i] = (a.inverse ? -sn : sn) * a.factor;
    }
  }
  const int heads = a.Hq + a.Hkv;
  const int h0 = blockIdx.y * a.heads, h1 = min(heads, h0 + a.heads);
  const size_t row = (size_t)a.d, head = (size_t)a.N * a.d;
  auto from = [&](int h) {
    const T* base = h < a.Hq ? (const T*)a.q + ((size_t)b * a.Hq + h) * head
                             : (const T*)a.k + ((size_t)b * a.Hkv + (h - a.Hq)) * head;
    return base + n * row + at;
  };
  auto to = [&](int h) {
    T* base = h < a.Hq ? (T*)a.q_out + ((size_t)b * a.Hq + h) * head
                       : (T*)a.k_out + ((size_t)b * a.Hkv + (h - a.Hq)) * head;
    return base + n * row + at;
  };
  if (!turn && a.q_out == a.q && a.k_out == a.k) return;   // in place
  for (int h = h0; h < h1; h += DEEP) {
    Piece<T, V> x[DEEP], z[DEEP];
#pragma unroll
    for (int i = 0; i < DEEP; ++i)
      if (h + i < h1) {
        const T* p = from(h + i);
        x[i] = get<T, V>(p);
        if (PAIR && second) z[i] = get<T, V>(p + gap);
      }
#pragma unroll
    for (int i = 0; i < DEEP; ++i)
      if (h + i < h1) {
        T* o = to(h + i);
        if (turn) {
#pragma unroll
          for (int e = 0; e < P; ++e) {
            T& u = PAIR ? x[i].v[e] : x[i].v[(2 * e) % V];
            T& w = PAIR ? z[i].v[e] : x[i].v[(2 * e + 1) % V];
            const float f = to_f(u), g = to_f(w);
            // the same roundings in every variant
            of_f(u, __fmaf_rn(f, c[e], -__fmul_rn(g, s[e])));
            of_f(w, __fmaf_rn(g, c[e], __fmul_rn(f, s[e])));
          }
        }
        put<T, V>(o, x[i]);
        if (PAIR && second) put<T, V>(o + gap, z[i]);
      }
  }
}

template <typename T, bool HALF, int V>
cudaError_t go(RotaryArgs& a, cudaStream_t st) {
  constexpr bool PAIR = HALF || V == 1;
  constexpr int P = PAIR ? V : V / 2;
  const int copied = PAIR ? 2 * V : V;
  a.units = a.rot / (2 * P) + (a.d - a.rot + copied - 1) / copied;
  const long long items = (long long)a.B * a.N * a.units;
  const int heads = a.Hq + a.Hkv;
  // all heads by one thread (its sines once), or fewer where that leaves SMs without
  // threads: half of 152 x 2048
  const long long want = (152LL * 1024 + items - 1) / items;
  int groups = (int)(want < heads ? want : heads);
  a.heads = (heads + groups - 1) / groups;
  groups = (heads + a.heads - 1) / a.heads;
  const long long blocks = (items + RT - 1) / RT;
  if (blocks >= 1LL << 31 || groups > 65535) return cudaErrorInvalidValue;
  return launch("rotary", k_rotary<T, HALF, V>, dim3((unsigned)blocks, groups), dim3(RT), 0, st, a);
}

template <typename T, int V>
cudaError_t pick(RotaryArgs& a, bool half, bool whole, cudaStream_t st) {
  if (half) return whole ? go<T, true, V>(a, st) : go<T, true, 1>(a, st);
  return whole ? go<T, false, V>(a, st) : go<T, false, 1>(a, st);
}

}  // namespace

cudaError_t run_rotary(RotaryArgs& a, bool half, bool bf16, cudaStream_t st) {
  const int v = bf16 ? 8 : 4;
  auto al = [](const void* p) { return ((uintptr_t)p & 15) == 0; };
  // 16-byte pieces where every piece of every row starts on 16 bytes
  const bool whole = al(a.q) && al(a.k) && al(a.q_out) && al(a.k_out) && a.d % v == 0 &&
                     a.rot % v == 0 && (!half || a.rot / 2 % v == 0);
  return bf16 ? pick<__nv_bfloat16, 8>(a, half, whole, st) : pick<float, 4>(a, half, whole, st);
}

}  // namespace lapnys
