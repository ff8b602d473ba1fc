// Argument blocks of what stands around the attentions in a layer: rotary
// positions (k_rotary.cu) and the residual with its norms (k_norm.cu).
#pragma once
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lapnys {

struct RotaryArgs {
  const void* q;             // [B][Hq][N][d]
  const void* k;             // [B][Hkv][N][d]
  void* q_out;               // like q, may be q itself
  void* k_out;
  const uint64_t* turns;     // [rot / 2]: turns a position, in units of 2^-64
  const int32_t* start;      // [B] or null (0)
  const int32_t* positions;  // [B][N] or null
  int B, Hq, Hkv, N, d, rot;
  float factor;              // of the turned features
  int inverse;               // turn back
  // filled by the launcher
  int units, heads;          // work items a token; heads of one
};
cudaError_t run_rotary(RotaryArgs& a, bool half, bool bf16, cudaStream_t st);

enum : int { kNormNone = 0, kNormRms = 1, kNormLayer = 2 };

struct NormArgs {
  const void* x;            // [B][N][C]
  const void* u;            // like x, or null: h = x
  const void* weight;       // [C], or [B][C] with per_seq; null: 1
  const void* bias;         // alike; null: 0
  const void* post_weight;  // [C] or null
  const void* post_bias;    // [C] or null
  const void* gate;         // [B][C] or null
  const void* scale;        // [C] or null
  void* h;                  // may be null (without u)
  void* y;                  // null: no norm of h
  float* stats;             // [B N][4]: mean and 1 / deviation of u, of h; or null
  int B, N, C, per_seq, pre, post;
  float eps;
  // backward
  const void* dh;           // null: 0
  const void* dy;           // null: 0
  void* dx;
  void* du;
  float* part;              // [slots][4][C]: sums over the rows of a part, by kind
  float* seq;               // [B][4][C]: over the rows of a sequence
  void* dweight;            // each may be null
  void* dbias;
  void* dpost_weight;
  void* dpost_bias;
  void* dgate;
  void* dscale;
  int sums;                 // bits of kSum*
  // filled by the launcher: a sequence's parts are slots b * parts .., or, where blocks take
  // even stretches of all tiles, slot b + block for each block that meets it
  int parts, grid, tiles;   // ranges of a sequence; blocks; tiles of a sequence
};
// sums over rows, of dy * (unit norm of h), dy, dh' * (unit norm of u), dh'
enum : int { kSumDyH = 1, kSumDy = 2, kSumDhU = 4, kSumDh = 8 };
constexpr int kNormMaxWidth = 16384;
int norm_slots(int B, int N, int C);     // at the most, of either kind
cudaError_t run_norm_fwd(NormArgs& a, bool bf16, cudaStream_t st);
cudaError_t run_norm_bwd(NormArgs& a, bool bf16, cudaStream_t st);

}  // namespace lapnys
