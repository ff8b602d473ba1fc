// C ABI of the windowed attention and of the attention over an 8-bit cache
// (include/lapnys.h has the contract): argument checks, workspaces, and the
// choice of kernel.
#include <math.h>
#include <string.h>

#include "../../include/lapnys.h"
#include "internal.h"
#include "win.cuh"

namespace lapnys {
namespace {

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

// a side of the window: -1 is open; as the kernels take it
bool side(int given, int* out) {
  if (given < -1) return false;
  *out = given < 0 || given > kWinUnbounded ? kWinUnbounded : given;
  return true;
}

int check_mask(WinArgs& a, int left, int right, int sinks, float scale) {
  if (!side(left, &a.left) || !side(right, &a.right) || sinks < 0) return LAPNYS_EINVAL;
  if (!(scale > 0.f) || !isfinite(scale)) return LAPNYS_EINVAL;
  a.sinks = sinks > kWinMaxLen ? kWinMaxLen : sinks;
  a.scale = scale;
  a.scale_log2 = (float)((double)scale * 1.4426950408889634);
  return LAPNYS_OK;
}

int check_dims(WinArgs& a, int B, int Hq, int Hkv, int Nq, int Nk, int d) {
  if (B <= 0 || Hq <= 0 || Hkv <= 0 || Nq <= 0 || Nk <= 0 || d <= 0) return LAPNYS_EINVAL;
  if (Hq % Hkv != 0 || Nq > kWinMaxLen || Nk > kWinMaxLen) return LAPNYS_EINVAL;
  if (d % 16 != 0 || d > 128) return LAPNYS_ENOTSUP;
  a.B = B; a.Hq = Hq; a.Hkv = Hkv; a.g = Hq / Hkv; a.Nq = Nq; a.Nk = Nk; a.d = d;
  // grids are one-dimensional, a block for at least 16 rows or keys
  const long long tiles = (long long)B * Hq * ((Nq + 15LL) / 16 + (Nk + 15LL) / 16);
  return tiles < 1LL << 30 ? LAPNYS_OK : LAPNYS_EINVAL;
}

// Few queries go to the kernel that splits the keys (k_token.cu): it reads the
// keys once for 16 rows (query heads of a group x queries).
bool few(int g, int Nq) { return Nq <= 8 || g * Nq <= 16; }

// a workspace's parts for k_token.cu
size_t token_bytes(const TokenShape& s) {
  return align256(s.o_bytes) + align256(s.ml_bytes) + align256(s.info_bytes);
}
void token_parts(TokenArgs& t, const TokenShape& s, void* ws) {
  uint8_t* p = (uint8_t*)ws;
  t.rtiles = s.rtiles;
  t.grid = s.grid;
  t.part_o = (float*)p;
  t.part_ml = (float2*)(p + align256(s.o_bytes));
  t.info = (int2*)(p + align256(s.o_bytes) + align256(s.ml_bytes));
}

struct WinWs {
  TokenShape tok;               // forward, few queries
  size_t D, part;               // backward
  int stiles, chunks, chunk_rows;
  size_t total;
};

// rows of the backward's key tiles: bf16 by tcgen05, fp32 by the warp-level instruction
int tile_rows(int dtype) { return dtype == LAPNYS_BF16 ? win_tc_tile_rows() : win_tile_rows(); }

WinWs window_ws(const WinArgs& a, bool backward, int dtype) {
  const int tile = tile_rows(dtype);
  WinWs w;
  memset(&w, 0, sizeof(w));
  size_t o = 0;
  if (!backward) {
    if (few(a.g, a.Nq)) {
      w.tok = token_shape(false, dtype == LAPNYS_BF16, a.B, a.Hkv, a.g, a.Nq, a.d, a.Nk, a.left,
                          a.right, a.sinks);
      o = token_bytes(w.tok);
    }
  } else {
    w.D = o; o = align256(o + (size_t)a.B * a.Hq * a.Nq * 4);
    // Key tiles with first tokens that more queries see than an ordinary tile's (twice
    // as many; below that the partials' launch is not worth it): their queries in
    // ranges as long as an ordinary tile's, or longer where enough blocks run anyway
    // (four for each of 152 SMs), which bounds the partials.  As one item, the first
    // tile of 8192 tokens with a window of 2048 runs for 600 us beside 226.  One range would be
    // partials for nothing: then the tiles are like any other.
    const int S = a.sinks < a.Nk ? a.sinks : a.Nk, kt = (a.Nk + tile - 1) / tile;
    const long long reach = (long long)a.left + a.right + tile, BH = (long long)a.B * a.Hkv;
    const long long steps = (long long)a.g * ((a.Nq + tile - 1) / tile);   // of a tile that all see
    if (S > 0 && 2 * reach < a.Nq) {
      const int st = (S + tile - 1) / tile;
      long long n = (a.Nq + reach - 1) / reach;
      const long long most = 608 / (BH * st) + 1;
      n = n < most ? n : most;
      w.chunk_rows = (int)(((a.Nq + n - 1) / n + tile - 1) / tile * tile);
      w.stiles = w.chunk_rows < a.Nq ? st : 0;
    } else if (2 * reach >= a.Nq && (BH * kt < 152 || (BH * kt < 304 && steps >= 64))) {
      // Every tile is seen by half of the queries or more, and there are fewer tiles than
      // SMs, or long ones that fill the SMs once and a little: all tiles' queries in
      // ranges, two items for each of 152 SMs (four of long ones), of four steps (tiles of
      // one head's queries) or more.  fp32, heads of 128, forward + backward: 8 heads on 1,
      // 2 x 1181 tokens, 38 tiles: 2171 us as they are, 1031 cut; 20 on 5, 1986 tokens, 155
      // tiles: 4717 and 3775 us.
      const long long least = (long long)tile * ((3 + a.g) / a.g);
      const long long n = ((steps < 64 ? 304 : 608) + BH * kt - 1) / (BH * kt);
      const long long rows = ((a.Nq + n - 1) / n + tile - 1) / tile * tile;
      w.chunk_rows = (int)(rows > least ? rows : least);
      w.stiles = w.chunk_rows < a.Nq ? kt : 0;
    }
    if (w.stiles > 0) {
      w.chunks = (a.Nq + w.chunk_rows - 1) / w.chunk_rows;
      w.part = o;
      o = align256(o + (size_t)BH * w.stiles * w.chunks * 2 * tile * a.d * 4);
    }
  }
  w.total = o;
  return w;
}

int check_window(WinArgs& a, int B, int Hq, int Hkv, int Nq, int Nk, int d, int left, int right,
                 int sinks, float scale, int dtype) {
  int rc = check_dims(a, B, Hq, Hkv, Nq, Nk, d);
  if (rc != LAPNYS_OK) return rc;
  if ((rc = check_mask(a, left, right, sinks, scale)) != LAPNYS_OK) return rc;
  return dtype == LAPNYS_F32 || dtype == LAPNYS_BF16 ? LAPNYS_OK : LAPNYS_EINVAL;
}

// a cache: `blocks` blocks of `block` tokens, at most max_blocks of them a sequence
int check_cache(WinArgs& a, int B, int Hq, int Hkv, int Nq, int d, int block, int blocks,
                int max_blocks, int dtype) {
  if (block != 16 && block != 32 && block != 64 && block != 128) return LAPNYS_EINVAL;
  if (blocks <= 0 || max_blocks <= 0 || (long long)max_blocks * block > kWinMaxLen)
    return LAPNYS_EINVAL;
  if (Hkv > 0 && (long long)blocks * Hkv >= 1LL << 31) return LAPNYS_EINVAL;
  if (dtype != LAPNYS_F32 && dtype != LAPNYS_BF16) return LAPNYS_EINVAL;
  return check_dims(a, B, Hq, Hkv, Nq, max_blocks * block, d);
}

std::atomic<int> g_sms[64];

int status(cudaError_t e) { return e == cudaSuccess ? LAPNYS_OK : LAPNYS_ECUDA; }

}  // namespace

cudaError_t device_sms(int* dev, int* sms) {
  cudaError_t e = cudaGetDevice(dev);
  if (e != cudaSuccess) return e;
  const int i = *dev;
  *sms = i < 64 ? g_sms[i].load(std::memory_order_relaxed) : 0;
  if (*sms > 0) return cudaSuccess;
  e = cudaDeviceGetAttribute(sms, cudaDevAttrMultiProcessorCount, i);
  if (e == cudaSuccess && i < 64) g_sms[i].store(*sms, std::memory_order_relaxed);
  return e;
}

}  // namespace lapnys

using namespace lapnys;

extern "C" {

size_t lapnys_window_workspace_bytes(int B, int Hq, int Hkv, int Nq, int Nk, int d, int left,
                                     int right, int sinks, int dtype, int backward) {
  WinArgs a;
  memset(&a, 0, sizeof(a));
  if (check_window(a, B, Hq, Hkv, Nq, Nk, d, left, right, sinks, 1.f, dtype) != LAPNYS_OK) return 0;
  return window_ws(a, backward != 0, dtype).total;
}

int lapnys_window_fwd(const void* q, const void* k, const void* v, void* out, float* lse,
                      void* rest, const int32_t* lens, const int32_t* q_pos, int B, int Hq,
                      int Hkv, int Nq, int Nk, int d, int left, int right, int sinks, float scale,
                      cudaStream_t stream, int dtype, void* ws, size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_window_fwd");
  TokenArgs t;
  memset(&t, 0, sizeof(t));
  WinArgs& a = t.w;
  const int rc = check_window(a, B, Hq, Hkv, Nq, Nk, d, left, right, sinks, scale, dtype);
  if (rc != LAPNYS_OK) return rc;
  if (!q || !k || !v || !out || !aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) ||
      !aligned(out, 16) || !aligned(rest, 16) || !aligned(lse, 4) || !aligned(lens, 4) ||
      !aligned(q_pos, 4) || (rest && dtype != LAPNYS_BF16))
    return LAPNYS_EINVAL;
  const WinWs w = window_ws(a, false, dtype);
  if (w.total > 0 && (!ws || !aligned(ws, 16))) return LAPNYS_EINVAL;
  if (ws_bytes < w.total) return LAPNYS_ENOSPC;
  a.q = q; a.k = k; a.v = v; a.out = out; a.lse = lse; a.lens = lens; a.q_pos = q_pos;
  a.rest = rest;
  if (few(a.g, Nq)) {
    token_parts(t, w.tok, ws);
    t.err = wait_error_address();
    if (t.err == nullptr) return LAPNYS_ECUDA;
    return status(run_token(t, dtype == LAPNYS_BF16, stream));
  }
  if (dtype == LAPNYS_BF16) return status(run_win_fwd_tc(a, stream));
  return status(run_win_fwd(a, stream));
}

int lapnys_window_bwd(const void* q, const void* k, const void* v, const void* out,
                      const void* dout, const float* lse, const void* rest, const int32_t* lens,
                      const int32_t* q_pos, void* dq, void* dk, void* dv, int B, int Hq, int Hkv,
                      int Nq, int Nk, int d, int left, int right, int sinks, float scale,
                      cudaStream_t stream, int dtype, void* ws, size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_window_bwd");
  WinArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_window(a, B, Hq, Hkv, Nq, Nk, d, left, right, sinks, scale, dtype);
  if (rc != LAPNYS_OK) return rc;
  const void* all[] = {q, k, v, out, dout, dq, dk, dv, ws};
  for (const void* p : all)
    if (!p || !aligned(p, 16)) return LAPNYS_EINVAL;
  if (!lse || !aligned(rest, 16) || !aligned(lse, 4) || !aligned(lens, 4) || !aligned(q_pos, 4) ||
      (rest && dtype != LAPNYS_BF16))
    return LAPNYS_EINVAL;
  const WinWs w = window_ws(a, true, dtype);
  if (ws_bytes < w.total) return LAPNYS_ENOSPC;
  a.q = q; a.k = k; a.v = v; a.out = const_cast<void*>(out); a.dout = dout;
  a.lse = const_cast<float*>(lse); a.lens = lens; a.q_pos = q_pos;
  a.rest = const_cast<void*>(rest);
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.D = (float*)((uint8_t*)ws + w.D);
  a.part = (float*)((uint8_t*)ws + w.part);
  a.stiles = w.stiles; a.chunks = w.chunks; a.chunk_rows = w.chunk_rows;
  if (dtype == LAPNYS_BF16) return status(run_win_bwd_tc(a, stream));
  return status(run_win_bwd(a, stream));
}

int lapnys_cache_append(const void* k, const void* v, void* k_cache, void* v_cache, float* k_scale,
                        float* v_scale, const int32_t* table, const int32_t* start,
                        const int32_t* lens, int B, int Hkv, int N, int d, int block, int blocks,
                        int max_blocks, cudaStream_t stream, int dtype) {
  NvtxScope nvtx_scope("lapnys_cache_append");
  WinArgs a;
  memset(&a, 0, sizeof(a));
  const int rc = check_cache(a, B, Hkv, Hkv, N, d, block, blocks, max_blocks, dtype);
  if (rc != LAPNYS_OK) return rc;
  const void* all[] = {k, v, k_cache, v_cache};
  for (const void* p : all)
    if (!p || !aligned(p, 16)) return LAPNYS_EINVAL;
  const void* words[] = {k_scale, v_scale, table, start};
  for (const void* p : words)
    if (!p || !aligned(p, 4)) return LAPNYS_EINVAL;
  if (!aligned(lens, 4)) return LAPNYS_EINVAL;
  AppendArgs p;
  memset(&p, 0, sizeof(p));
  p.k = k; p.v = v;
  p.k_cache = (uint8_t*)k_cache; p.v_cache = (uint8_t*)v_cache;
  p.k_scale = k_scale; p.v_scale = v_scale;
  p.table = table; p.start = start; p.lens = lens;
  p.B = B; p.Hkv = Hkv; p.N = N; p.d = d; p.T = block; p.blocks = blocks; p.max_blocks = max_blocks;
  p.err = wait_error_address();
  if (p.err == nullptr) return LAPNYS_ECUDA;
  return status(run_cache_append(p, dtype == LAPNYS_BF16, stream));
}

size_t lapnys_cache_workspace_bytes(int B, int Hq, int Hkv, int Nq, int d, int block, int blocks,
                                    int max_blocks, int left, int right, int sinks, int dtype) {
  WinArgs a;
  memset(&a, 0, sizeof(a));
  if (check_cache(a, B, Hq, Hkv, Nq, d, block, blocks, max_blocks, dtype) != LAPNYS_OK) return 0;
  if (check_mask(a, left, right, sinks, 1.f) != LAPNYS_OK) return 0;
  return token_bytes(token_shape(true, dtype == LAPNYS_BF16, B, Hkv, a.g, Nq, d, a.Nk, a.left,
                                 a.right, a.sinks));
}

int lapnys_cache_attention(const void* q, const void* k_cache, const void* v_cache,
                           const float* k_scale, const float* v_scale, const int32_t* table,
                           const int32_t* lens, const int32_t* q_pos, void* out, int B, int Hq,
                           int Hkv, int Nq, int d, int block, int blocks, int max_blocks, int left,
                           int right, int sinks, float scale, cudaStream_t stream, int dtype,
                           void* ws, size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_cache_attention");
  TokenArgs t;
  memset(&t, 0, sizeof(t));
  WinArgs& a = t.w;
  int rc = check_cache(a, B, Hq, Hkv, Nq, d, block, blocks, max_blocks, dtype);
  if (rc != LAPNYS_OK) return rc;
  if ((rc = check_mask(a, left, right, sinks, scale)) != LAPNYS_OK) return rc;
  const void* all[] = {q, k_cache, v_cache, out};
  for (const void* p : all)
    if (!p || !aligned(p, 16)) return LAPNYS_EINVAL;
  const void* words[] = {k_scale, v_scale, table, lens};
  for (const void* p : words)
    if (!p || !aligned(p, 4)) return LAPNYS_EINVAL;
  if (!aligned(q_pos, 4)) return LAPNYS_EINVAL;
  const TokenShape s = token_shape(true, dtype == LAPNYS_BF16, B, Hkv, a.g, Nq, d, a.Nk, a.left,
                                   a.right, a.sinks);
  const size_t need = token_bytes(s);
  if (need > 0 && (!ws || !aligned(ws, 16))) return LAPNYS_EINVAL;
  if (ws_bytes < need) return LAPNYS_ENOSPC;
  a.q = q; a.k = k_cache; a.v = v_cache; a.out = out; a.lens = lens; a.q_pos = q_pos;
  t.k_scale = k_scale; t.v_scale = v_scale; t.table = table;
  t.Tshift = block == 16 ? 4 : block == 32 ? 5 : block == 64 ? 6 : 7;
  t.blocks = blocks; t.max_blocks = max_blocks;
  token_parts(t, s, ws);
  t.err = wait_error_address();
  if (t.err == nullptr) return LAPNYS_ECUDA;
  return status(run_token(t, dtype == LAPNYS_BF16, stream));
}

}  // extern "C"
