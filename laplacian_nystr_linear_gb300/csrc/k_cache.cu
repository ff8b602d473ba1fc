// Keys and values rounded into a cache of e4m3 blocks with one power-of-two
// scale per block of T tokens and head.
//
//   scale = 2^ceil(log2(amax / 448)) over the finite magnitudes (>= 2^-100),
//   stored = e4m3(x / scale), to nearest, ties to even.
//
// A power of two costs no precision (e4m3 is a floating-point type; the largest
// magnitude still lands in (224, 448]) and makes a later, larger scale harmless:
// the block's earlier tokens are multiplied by the ratio of the scales, exactly,
// unless a value becomes subnormal (below 2^-6 of the new scale: off by at most
// 2^-10 of it more each time the scale grows).  So appending one token at a time gives the
// values of one call, but for those and for infinities: one is stored as 448 of the scale of
// its call, which is a number like any other when the scale grows later.
//
// One block of threads per (sequence, cache block, head, keys or values): the
// new tokens are read once, kept in registers over the reduction and written as
// 8 bytes per 8 values.  Bound by DRAM for prompts (4 of up to 4099 tokens, 8 heads of
// 128, bf16: 23 us, 4.4 TB/s; fp32 31 us,
// 5.4 TB/s), by the launch for one token (7.5 us for 32 sequences).
#include <cuda_fp8.h>

#include "common.cuh"
#include "internal.h"
#include "win.cuh"

namespace lapnys {

namespace {
constexpr int AT = 256;            // threads
constexpr int kMinScaleExp = -100;

// eight values as they lie in memory, and as fp32
template <typename T>
struct Raw8;
template <>
struct Raw8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = ld4(p);
    b = ld4(p + 4);
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
  }
};
template <>
struct Raw8<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) {
    u = __ldg(reinterpret_cast<const uint4*>(p));
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
};
// infinities saturate, NaN stays NaN
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | hi << 16;
}
__device__ __forceinline__ float e4m3(uint32_t byte) {
  const __half_raw h = __nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)byte, __NV_E4M3);
  return __half2float(__half(h));
}
// the smallest power of two s with amax <= 448 s (448 = 1.75 * 2^8)
__device__ __forceinline__ float scale_for(float amax) {
  const uint32_t u = __float_as_uint(amax);
  int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  if (e < kMinScaleExp) e = kMinScaleExp;   // also for 0 and subnormal magnitudes
  return __uint_as_float((uint32_t)(e + 127) << 23);
}
}  // namespace

// AV: vectors of eight values a thread holds (the block's most)
template <typename T, int AV>
__global__ void __launch_bounds__(AT) k_cache_append(AppendArgs a) {
  __shared__ float red[AT / 32];
  const int which = blockIdx.x & 1, h = (blockIdx.x >> 1) % a.Hkv;
  const int x = (blockIdx.x >> 1) / a.Hkv, b = x / a.nt;
  const int start = min(max(a.start[b], -kWinMaxLen), kWinMaxLen);
  const int cap = (int)min((long long)a.max_blocks * a.T, (long long)kWinMaxLen);
  const int end = min(start + a.N, min(a.lens ? max(a.lens[b], 0) : cap, cap));
  const int lb = max(start, 0) / a.T + x % a.nt, P0 = lb * a.T;
  const int fs = max(start, P0) - P0, fe = min(end, P0 + a.T) - P0;   // slots of the new tokens
  if (fs >= fe) return;
  const int held = start > P0 ? fs : 0;   // slots that hold earlier tokens
  const int blk = a.table[(size_t)b * a.max_blocks + lb];
  if ((unsigned)blk >= (unsigned)a.blocks) {
    if (threadIdx.x == 0) atomicOr(a.err, 2);
    return;
  }
  const size_t bh = (size_t)blk * a.Hkv + h;
  const T* src = (const T*)(which ? a.v : a.k) + ((size_t)b * a.Hkv + h) * a.N * a.d +
                 (long long)(P0 + fs - start) * a.d;
  uint8_t* dst = (which ? a.v_cache : a.k_cache) + bh * a.T * a.d;
  float* scp = (which ? a.v_scale : a.k_scale) + bh;
  const int nv = (fe - fs) * a.d / 8;
  Raw8<T> raw[AV];
#pragma unroll
  for (int i = 0; i < AV; ++i) {
    const int id = i * AT + threadIdx.x;
    if (id < nv) raw[i].load(src + (size_t)id * 8);
  }
  const float was = held ? *scp : 0.f;
  float mx = 0.f;
#pragma unroll
  for (int i = 0; i < AV; ++i)
    if (i * AT + (int)threadIdx.x < nv) {
      float v[8];
      raw[i].get(v);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float y = fabsf(v[e]);
        mx = fmaxf(mx, y < INFINITY ? y : 0.f);
      }
    }
#pragma unroll
  for (int k = 16; k; k >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, k));
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = mx;
  __syncthreads();   // also: every thread has read the old scale
#pragma unroll
  for (int w = 0; w < AT / 32; ++w) mx = fmaxf(mx, red[w]);
  const float sc = fmaxf(scale_for(mx), was);
  if (threadIdx.x == 0 && sc != was) *scp = sc;
  const float inv = 1.f / sc;
#pragma unroll
  for (int i = 0; i < AV; ++i) {
    const int id = i * AT + threadIdx.x;
    if (id < nv) {
      float v[8];
      raw[i].get(v);
      *reinterpret_cast<uint2*>(dst + (size_t)fs * a.d + (size_t)id * 8) =
          make_uint2(to_e4m3x4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                     to_e4m3x4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    }
  }
  if (held && sc != was) {
    const float f = was * inv;
    for (int id = threadIdx.x; id < held * a.d / 4; id += AT) {
      uint32_t* p = reinterpret_cast<uint32_t*>(dst) + id;
      const uint32_t u = *p;
      *p = to_e4m3x4(e4m3(u & 255) * f, e4m3(u >> 8 & 255) * f, e4m3(u >> 16 & 255) * f,
                     e4m3(u >> 24) * f);
    }
  }
}

namespace {
template <typename T>
cudaError_t append_go(const AppendArgs& a, cudaStream_t st) {
  const dim3 grid((unsigned)((long long)a.B * a.nt * a.Hkv * 2));
  const int most = a.N < a.T ? a.N : a.T, nv = (most * a.d / 8 + AT - 1) / AT;
  if (nv <= 1) return launch("cache_append", k_cache_append<T, 1>, grid, dim3(AT), 0, st, a);
  if (nv <= 4) return launch("cache_append", k_cache_append<T, 4>, grid, dim3(AT), 0, st, a);
  return launch("cache_append", k_cache_append<T, 8>, grid, dim3(AT), 0, st, a);
}
}  // namespace

cudaError_t run_cache_append(AppendArgs& a, bool bf16, cudaStream_t st) {
  a.nt = (a.N + a.T - 2) / a.T + 1;
  return bf16 ? append_go<__nv_bfloat16>(a, st) : append_go<float>(a, st);
}

}  // namespace lapnys
