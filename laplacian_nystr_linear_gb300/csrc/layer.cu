// C ABI of the rotary positions and of the residual with its norms
// (include/lapnys.h has the contract): argument checks and workspaces.
#include <math.h>
#include <string.h>

#include "../../include/lapnys.h"
#include "internal.h"
#include "layer.cuh"

namespace lapnys {
namespace {

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int status(cudaError_t e) { return e == cudaSuccess ? LAPNYS_OK : LAPNYS_ECUDA; }
bool known(int dtype) { return dtype == LAPNYS_F32 || dtype == LAPNYS_BF16; }

int check_norm(NormArgs& a, int B, int N, int C, int per_seq, int pre, int post, float eps) {
  // rows are counted in 32 bits, with room for a tile or the joins' threads behind the last
  if (B <= 0 || N <= 0 || C <= 0 || (long long)B * N > (1LL << 31) - 1024) return LAPNYS_EINVAL;
  if (pre < kNormNone || pre > kNormLayer || post < kNormNone || post > kNormLayer) return LAPNYS_EINVAL;
  if (!(eps >= 0.f) || !isfinite(eps)) return LAPNYS_EINVAL;
  if (C > kNormMaxWidth) return LAPNYS_ENOTSUP;
  a.B = B; a.N = N; a.C = C; a.per_seq = per_seq != 0; a.pre = pre; a.post = post; a.eps = eps;
  return LAPNYS_OK;
}

// without a vector of each sequence all rows are one sequence's
void flatten(NormArgs& a, bool seqs) {
  if (seqs) return;
  a.N *= a.B;
  a.B = 1;
}

struct NormWs {
  size_t part, seq, total;
};
NormWs norm_ws(const NormArgs& a) {
  NormWs w;
  w.part = 0;
  w.seq = align256((size_t)norm_slots(a.B, a.N, a.C) * 4 * a.C * 4);
  w.total = w.seq + align256((size_t)a.B * 4 * a.C * 4);
  return w;
}

// vectors belong to what there is: a norm's to that norm, gate and scale to u
bool fits(const NormArgs& a) {
  if (a.pre == kNormNone && (a.weight || a.bias || a.per_seq || a.y)) return false;
  if (!a.u && (a.post != kNormNone || a.gate || a.scale)) return false;
  return a.post != kNormNone || (!a.post_weight && !a.post_bias);
}

}  // namespace
}  // namespace lapnys

using namespace lapnys;

extern "C" {

int lapnys_rotary(const void* q, const void* k, void* q_out, void* k_out, const uint64_t* turns,
                  const int32_t* start, const int32_t* positions, int B, int Hq, int Hkv, int N,
                  int d, int rot, int layout, float factor, int inverse, cudaStream_t stream,
                  int dtype) {
  NvtxScope nvtx_scope("lapnys_rotary");
  if (B <= 0 || Hq <= 0 || N <= 0 || d <= 0 || rot <= 0 || rot > d || rot % 2 != 0) return LAPNYS_EINVAL;
  if (Hkv < 0 || (k == nullptr) != (Hkv == 0) || (k == nullptr) != (k_out == nullptr))
    return LAPNYS_EINVAL;
  if ((layout != LAPNYS_HALF && layout != LAPNYS_INTERLEAVED) || !known(dtype)) return LAPNYS_EINVAL;
  if (!isfinite(factor) || (start && positions)) return LAPNYS_EINVAL;
  const size_t e = dtype == LAPNYS_BF16 ? 2 : 4;
  if (!q || !q_out || !aligned(q, e) || !aligned(k, e) || !aligned(q_out, e) || !aligned(k_out, e))
    return LAPNYS_EINVAL;
  if (!turns || !aligned(turns, 8) || !aligned(start, 4) || !aligned(positions, 4)) return LAPNYS_EINVAL;
  // one thread for as little as two features
  if (d > 1 << 16 || (long long)Hq + Hkv > 1 << 20 || (long long)B * N > (1LL << 36) / d)
    return LAPNYS_EINVAL;
  RotaryArgs a;
  memset(&a, 0, sizeof(a));
  a.q = q; a.k = k; a.q_out = q_out; a.k_out = k_out;
  a.turns = turns; a.start = start; a.positions = positions;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.N = N; a.d = d; a.rot = rot;
  a.factor = factor; a.inverse = inverse != 0;
  return status(run_rotary(a, layout == LAPNYS_HALF, dtype == LAPNYS_BF16, stream));
}

size_t lapnys_norm_workspace_bytes(int B, int N, int C, int seqs) {
  NormArgs a;
  memset(&a, 0, sizeof(a));
  if (check_norm(a, B, N, C, 0, kNormNone, kNormNone, 0.f) != LAPNYS_OK) return 0;
  flatten(a, seqs != 0);
  return norm_ws(a).total;
}

int lapnys_norm_fwd(const void* x, const void* u, const void* weight, const void* bias,
                    const void* post_weight, const void* post_bias, const void* gate,
                    const void* scale, void* h, void* y, float* stats, int B, int N, int C,
                    int per_seq, int pre, int post, float eps, cudaStream_t stream, int dtype) {
  NvtxScope nvtx_scope("lapnys_norm_fwd");
  NormArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_norm(a, B, N, C, per_seq, pre, post, eps);
  if (rc != LAPNYS_OK) return rc;
  if (!known(dtype)) return LAPNYS_EINVAL;
  a.x = x; a.u = u; a.weight = weight; a.bias = bias; a.post_weight = post_weight;
  a.post_bias = post_bias; a.gate = gate; a.scale = scale; a.h = h; a.y = y; a.stats = stats;
  const void* all[] = {x, u, weight, bias, post_weight, post_bias, gate, scale, h, y};
  for (const void* p : all)
    if (!aligned(p, dtype == LAPNYS_BF16 ? 2 : 4)) return LAPNYS_EINVAL;
  if (!x || !(h || y) || !aligned(stats, 16) || !fits(a) || (pre != kNormNone && !y))
    return LAPNYS_EINVAL;
  flatten(a, gate || a.per_seq);
  return status(run_norm_fwd(a, dtype == LAPNYS_BF16, stream));
}

int lapnys_norm_bwd(const void* x, const void* u, const void* weight, const void* post_weight,
                    const void* post_bias, const void* gate, const void* scale, const float* stats,
                    const void* dh, const void* dy, void* dx, void* du, void* dweight, void* dbias,
                    void* dpost_weight, void* dpost_bias, void* dgate, void* dscale, int B, int N,
                    int C, int per_seq, int pre, int post, cudaStream_t stream, int dtype, void* ws,
                    size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_norm_bwd");
  NormArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_norm(a, B, N, C, per_seq, pre, post, 0.f);
  if (rc != LAPNYS_OK) return rc;
  if (!known(dtype)) return LAPNYS_EINVAL;
  a.x = x; a.u = u; a.weight = weight; a.post_weight = post_weight; a.post_bias = post_bias;
  a.gate = gate; a.scale = scale; a.stats = const_cast<float*>(stats);
  a.dh = dh; a.dy = dy; a.dx = dx; a.du = du; a.dweight = dweight; a.dbias = dbias;
  a.dpost_weight = dpost_weight; a.dpost_bias = dpost_bias; a.dgate = dgate; a.dscale = dscale;
  const void* all[] = {x,  u,  weight, post_weight, post_bias, gate, scale, dh, dy,
                       dx, du, dweight, dbias, dpost_weight, dpost_bias, dgate, dscale};
  for (const void* p : all)
    if (!aligned(p, dtype == LAPNYS_BF16 ? 2 : 4)) return LAPNYS_EINVAL;
  if (!x || !stats || !aligned(stats, 16) || !fits(a)) return LAPNYS_EINVAL;
  if (pre == kNormNone && (dy || dweight || dbias)) return LAPNYS_EINVAL;
  if (!u && (du || dgate || dscale)) return LAPNYS_EINVAL;
  if (post == kNormNone && (dpost_weight || dpost_bias)) return LAPNYS_EINVAL;
  if ((dpost_weight && !post_weight) || (dgate && !gate) || (dscale && !scale)) return LAPNYS_EINVAL;
  a.sums = (dweight ? kSumDyH : 0) | (dbias ? kSumDy : 0) |
           (dpost_weight || dgate || dscale ? kSumDhU : 0) |
           (dpost_bias || ((dgate || dscale) && post_bias) ? kSumDh : 0);
  flatten(a, gate || a.per_seq);
  const NormWs w = norm_ws(a);
  if (a.sums) {
    if (!ws || !aligned(ws, 16)) return LAPNYS_EINVAL;
    if (ws_bytes < w.total) return LAPNYS_ENOSPC;
    a.part = (float*)((uint8_t*)ws + w.part);
    a.seq = (float*)((uint8_t*)ws + w.seq);
  }
  return status(run_norm_bwd(a, dtype == LAPNYS_BF16, stream));
}

}  // extern "C"
