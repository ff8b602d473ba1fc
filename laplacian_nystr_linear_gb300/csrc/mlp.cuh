// The gated feed-forward block: what its kernels and its host code share.
//
//   z = x w_in + b_in,  (g, u) = the halves of z,  h = act(g) u,  y = h w_out + b_out
//
// with T rows, C features in and out, F hidden.  For the backward the forward keeps
// h and the two factors that the gradient of h is multiplied by,
//   p = act(g)  (of du)   and   q = u act'(g)  (of dg).
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace lapnys {

enum : int { kActSilu = 0, kActGelu = 1, kActGeluTanh = 2 };

// p and q in blocks of 32 rows x 16 features, in the order in which a warp of an
// epilogue (a row a lane) writes and reads them: 16-byte pieces of a row, 32 lanes of a
// piece together.  bf16 calls keep them as f16 times a power of two for each row of a
// block (11 bits: half a step is up to 2^-11 of the value, beside the gradients' own of up to
// 2^-8; below 2^-28 of the block row's largest 2^-39 of that), fp32 calls and few rows in fp32.
constexpr int kMlpBlock = 16;   // features of a block
struct MlpKept {
  uint8_t* pq;        // [ceil(T / 32)][ceil(F / 16)][p, q][pieces][32 lanes] of 16 bytes
  uint16_t* scale;    // [ceil(T / 32)][ceil(F / 16)][32]: exponents of p | q << 8, + 128
};

// values of the activation and its slope
template <bool EXACT>
__device__ __forceinline__ float mlp_sigmoid(float x) {
  if constexpr (EXACT) return 1.f / (1.f + expf(-x));
  float e, r;     // both instructions within 2^-22 of the value
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * -1.4426950408889634f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.f + e));
  return r;
}
template <bool EXACT, int KIND>
__device__ __forceinline__ void mlp_act(float g, float& p, float& slope) {
  if constexpr (KIND == kActSilu) {
    const float s = mlp_sigmoid<EXACT>(g);
    p = g * s;
    slope = fmaf(p, 1.f - s, s);
  } else if constexpr (KIND == kActGelu) {
    const float c = fmaf(0.5f, erff(g * 0.70710678118654752f), 0.5f);
    p = g * c;
    const float e = EXACT ? expf(-0.5f * g * g) : __expf(-0.5f * g * g);
    slope = fmaf(g * 0.39894228040143268f, e, c);
  } else {
    // 0.5 (1 + tanh z) = sigmoid(2 z)
    // (far out both are 0 or 1 long before; bounded, the square stays finite)
    const float g2 = fminf(g * g, 1e18f), k = 1.5957691216057308f;      // 2 sqrt(2 / pi)
    const float s = mlp_sigmoid<EXACT>(k * g * fmaf(0.044715f, g2, 1.f));
    p = g * s;
    slope = fmaf(p * (1.f - s), k * fmaf(3.f * 0.044715f, g2, 1.f), s);
  }
}

// ---- host side -------------------------------------------------------------
// A matrix of bf16 as the products read it: `planes` of `rows` rows of `parts` runs of
// `inner` elements (fp32 values are three planes)
struct MlpView {
  const void* p;
  int inner, parts, rows, planes;
  size_t part_stride, row_stride, plane_stride;   // elements
};

enum : int { kMlpRows = 0, kMlpPart = 1, kMlpGlu = 2, kMlpDglu = 3 };

struct MlpGemmArgs {
  int M, N;              // rows; columns of a part
  int nparts;            // column parts that tiles run over
  int mt, nt;            // tiles of M and of a part's N
  int kst, kparts;       // K steps of a part, parts that K runs over
  int kplanes;           // bf16 calls: 2 where an operand is in two parts (K runs over both)
  int two_a, two_b;      // ... which
  int splits, items;
  int amn, bmn;          // operands stored [k][m], [k][n]
  int act;
  const void* bias;      // [nparts][N] (rows), [2][N] (glu), or null
  void* out;             // rows: [M][ldo], part p of the columns at p * part_out;
                         // part: fp32 [splits][M][ldo]; glu: h; dglu: dg, du [M][2][N padded]
  size_t ldo, part_out, plane_out;
  int wide;              // out takes 16-byte stores
  MlpKept kept;          // glu: written where set; dglu: read
  int fblocks;           // blocks of features
  int* err;
};

// the product of two views: a's rows are M (or its inner, with amn), K the other; two: h,
// or dg and du, of a bf16 call into two planes
cudaError_t run_mlp_gemm(const char* name, int epi, bool f32, bool two, const MlpView& a, const MlpView& b,
                         MlpGemmArgs& g, cudaStream_t st);
// K ranges of a product with `tiles` tiles of `ksteps` steps, M x N of fp32 a range
int mlp_splits(long long tiles, int ksteps, double mn, bool f32);
int mlp_tile_n(bool f32);     // columns of a tile
constexpr int kMlpTileM = 256;
constexpr int kMlpTileK = 64;

// out[m][part][n] = sum over `splits` of part[s][m][part][n] + bias, in order
struct MlpReduceArgs {
  const float* part;
  size_t ldp, part_in, split_stride;
  int splits, M, N, nparts;
  const void* bias;
  void* out;
  size_t ldo, part_out;
};
cudaError_t run_mlp_reduce(const char* name, const MlpReduceArgs& a, bool bf16, cudaStream_t st);

// up to four matrices into planes of bf16 (one of bf16 input, three of fp32)
struct MlpPackJob {
  const void* src;      // [rows][inner]
  __nv_bfloat16* dst;   // planes of [rows][ld]
  long long rows;
  int inner, ld;
};
struct MlpPackArgs {
  MlpPackJob job[4];
  long long first[5];   // first block of each
  int jobs;
};
cudaError_t run_mlp_pack(MlpPackArgs& a, bool bf16, cudaStream_t st);

// sums over rows of planes of bf16 [rows][ld], or of fp32 (no planes), in ranges of rows:
// part [ranges][columns], then out
struct MlpColsumArgs {
  const void* src;
  size_t ld, plane_stride;
  int planes;           // 0: src is fp32
  int rows, inner, parts, pstride;   // columns: `parts` runs of `inner`, `pstride` apart
  float* part;
  int ranges;
  void* out;            // [parts][inner]
};
int mlp_colsum_ranges(int rows, int cols);
cudaError_t run_mlp_colsum(const MlpColsumArgs& a, bool bf16, cudaStream_t st);

// A few rows: out[t][n] = sum_k x[t][k] w[k][n], through fp32 partial sums that a second
// kernel adds and finishes.
//   w: [K][nparts][N], or with kmajor [N][kparts][K] (K runs over the parts);
//   x: bf16 planes of T rows, one after the other, rows ldx apart, K's parts xpart: one or
//      two planes beside bf16 weights, three beside fp32 ones (padded with zeros to 8).
enum : int { kFewRows = 0, kFewGlu = 1, kFewDglu = 2 };
struct MlpFewArgs {
  const void* x;
  const void* w;
  size_t ldx, xpart;
  int T, planes, K, kparts, N, nparts, kmajor;
  float* part;          // [blocks of columns + blocks of the grid][rows][columns of a block]
  bool second;          // x comes from the kernel before, which is one of these
  // the join: rows: out [T][N] + bias; glu: planes of h [T][ldo] with bias [2][N], p and q
  // [T][N] fp32 where set; dglu: planes of (dg | du) [T][2][ldo] from p and q
  int mode, act, out_planes;
  const void* bias;
  void* out;
  size_t ldo;
  float* p;
  float* q;
  // filled by the launcher
  int nb, ks, kst, grid;   // column blocks of a part, K steps (of a part), blocks of the grid
  int* err;
};
// whether a call of T rows goes this way
bool mlp_few_ok(int T, int C, int F, bool f32);
// bytes of the partial sums
size_t mlp_few_bytes(int T, int planes, int N, int nparts, bool f32);
cudaError_t run_mlp_few(MlpFewArgs& a, bool f32, cudaStream_t st);

}  // namespace lapnys
