// Rotary positions: pairs of features turned by the token's position.
//
//   (a, b) -> factor (a cos t - b sin t, b cos t + a sin t),  t = 2 pi p w_i,
// pair i of rot / 2: features (i, i + rot / 2) in the half layout, (2 i, 2 i + 1)
// interleaved; features from rot on pass unchanged.  w_i is in turns a position, as
// a fraction of 2^64: modulo 2^64 p times that is exact, so the phase is off by p times
// w_i's own rounding, 2^-34 of a turn at p = 2^31, where 32-bit angles lose all of it (at
// p = 10^6 a rounded fp32 angle is off by 0.03).  The gradient is the turn back, by the same
// factor.
//
// Bound by memory: queries and keys are read and written once.  A thread keeps its
// pairs' cosines and sines in registers over the heads of its token, so they cost a
// few instructions a head; loads of four heads are in flight at once.  2 x 8192 tokens,
// 20 heads of 128: 32 us (bf16, 5.3 TB/s; interleaved 30), 55 us (fp32, 6.1 TB/s); pieces
// of 16 bytes of bf16 instead of 8, converted one by one, took 45 and 51 us.  Single
// tokens: the launch.
#include "common.cuh"
#include "internal.h"
#include "layer.cuh"

namespace lapnys {
namespace {

constexpr int RT = 128;   // threads of a block

// V elements as they lie: words of two bf16, single bf16, or fp32
template <typename T, int V>
struct Piece {
  static constexpr int W = V * (int)sizeof(T) >= 4 ? V * (int)sizeof(T) / 4 : 1;
  uint32_t w[W];
  __device__ __forceinline__ void get(const T* p) {
    if constexpr (W == 4) {
      const uint4 x = *reinterpret_cast<const uint4*>(p);
      w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
    } else if constexpr (W == 2) {
      const uint2 x = *reinterpret_cast<const uint2*>(p);
      w[0] = x.x; w[1] = x.y;
    } else if constexpr (sizeof(T) == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void put(T* p) const {
    if constexpr (W == 4)
      *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (W == 2)
      *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (sizeof(T) == 4)
      *reinterpret_cast<uint32_t*>(p) = w[0];
    else
      *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  __device__ __forceinline__ void open(float (&v)[V]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) v[i] = __uint_as_float(w[i]);
    } else if constexpr (V == 1) {
      v[0] = __uint_as_float(w[0] << 16);
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        v[i] = __uint_as_float(w[i / 2] << 16);
        v[i + 1] = __uint_as_float(w[i / 2] & 0xffff0000u);
      }
    }
  }
  __device__ __forceinline__ void close(const float (&v)[V]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < V; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (V == 1) {
      w[0] = __bfloat16_as_ushort(__float2bfloat16_rn(v[0]));
    } else {
#pragma unroll
      for (int i = 0; i < V; i += 2) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(v[i], v[i + 1]);
        w[i / 2] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
  }
};
// (a, b) turned; the same roundings in every variant
__device__ __forceinline__ void turn_pair(float& a, float& b, float c, float s) {
  const float x = __fmaf_rn(a, c, -__fmul_rn(b, s));
  b = __fmaf_rn(b, c, __fmul_rn(a, s));
  a = x;
}

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
    const int64_t p = a.positions ? a.positions[tok] : (int64_t)(a.start ? a.start[b] : 0) + n;
    const uint64_t at_p = (uint64_t)p;
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
  if (!turn && a.q_out == a.q && a.k_out == a.k) return;   // in place
  const int h0 = blockIdx.y * a.heads, h1 = min(a.Hq + a.Hkv, h0 + a.heads);
  const size_t head = (size_t)a.N * a.d, in_head = (size_t)n * a.d + at;
  // heads [lo, hi) of a tensor that has H of them
  auto run = [&](const void* in, void* out, int H, int lo, int hi) {
    if (lo >= hi) return;
    const size_t first = ((size_t)b * H + lo) * head + in_head;
    const T* src = (const T*)in + first;
    T* dst = (T*)out + first;
    for (int left = hi - lo; left > 0; left -= DEEP, src += DEEP * head, dst += DEEP * head) {
      Piece<T, V> x[DEEP], z[DEEP];
#pragma unroll
      for (int i = 0; i < DEEP; ++i)
        if (i < left) {
          x[i].get(src + i * head);
          if (PAIR && second) z[i].get(src + i * head + gap);
        }
#pragma unroll
      for (int i = 0; i < DEEP; ++i)
        if (i < left) {
          if (turn) {
            float f[V], g[V];
            x[i].open(f);
            if constexpr (PAIR) {
              z[i].open(g);
#pragma unroll
              for (int e = 0; e < V; ++e) turn_pair(f[e], g[e], c[e], s[e]);
              z[i].close(g);
            } else {
#pragma unroll
              for (int e = 0; e < P; ++e) turn_pair(f[2 * e], f[2 * e + 1], c[e], s[e]);
            }
            x[i].close(f);
          }
          x[i].put(dst + i * head);
          if (PAIR && second) z[i].put(dst + i * head + gap);
        }
    }
  };
  run(a.q, a.q_out, a.Hq, h0, min(h1, a.Hq));
  run(a.k, a.k_out, a.Hkv, max(h0 - a.Hq, 0), h1 - a.Hq);
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
  // threads: half of 152 x 2048 (twice or four times as many: 31 to 33 us for the 32 above,
  // 16 for 14 at 4096 tokens)
  const long long want = (152LL * 1024 + items - 1) / items;
  int groups = (int)(want < heads ? want : heads);
  groups = groups < 65535 ? groups : 65535;        // the grid's y
  a.heads = (heads + groups - 1) / groups;
  groups = (heads + a.heads - 1) / a.heads;
  const long long blocks = (items + RT - 1) / RT;
  if (blocks >= 1LL << 31) return cudaErrorInvalidValue;
  return launch("rotary", k_rotary<T, HALF, V>, dim3((unsigned)blocks, groups), dim3(RT), 0, st, a);
}

template <typename T, int V>
cudaError_t pick(RotaryArgs& a, bool half, bool whole, cudaStream_t st) {
  if (half) return whole ? go<T, true, V>(a, st) : go<T, true, 1>(a, st);
  return whole ? go<T, false, V>(a, st) : go<T, false, 1>(a, st);
}

}  // namespace

cudaError_t run_rotary(RotaryArgs& a, bool half, bool bf16, cudaStream_t st) {
  const int v = 4;
  auto al = [&](const void* p) { return ((uintptr_t)p & (bf16 ? 7 : 15)) == 0; };
  // pieces of four elements where each of every row starts on its size
  const bool whole = al(a.q) && al(a.k) && al(a.q_out) && al(a.k_out) && a.d % v == 0 &&
                     a.rot % v == 0 && (!half || a.rot / 2 % v == 0);
  return bf16 ? pick<__nv_bfloat16, 4>(a, half, whole, st) : pick<float, 4>(a, half, whole, st);
}

}  // namespace lapnys
