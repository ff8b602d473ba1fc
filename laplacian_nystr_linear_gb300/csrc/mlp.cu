// C ABI of the gated feed-forward block (include/lapnys.h has the contract): argument
// checks, what the forward keeps, workspaces, and the products in their order.
#include <math.h>
#include <string.h>

#include "../../include/lapnys.h"
#include "internal.h"
#include "mlp.cuh"

namespace lapnys {
namespace {

size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }
bool aligned(const void* p, size_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
int status(cudaError_t e) { return e == cudaSuccess ? LAPNYS_OK : LAPNYS_ECUDA; }
int up8(int x) { return (x + 7) & ~7; }

struct Mlp {
  int T, C, F, Cp, Fp;
  bool f32;
  bool few;     // few rows: k_mlp_few.cu
  int planes;   // of packed operands
  int hidden;   // of h and of (dg | du)
  // operands that the products cannot read where they lie: fp32 (three planes), or rows
  // that are not whole 16-byte pieces
  bool pack_c, pack_f;
};

int check_mlp(Mlp& m, int T, int C, int F, int dtype) {
  if (T <= 0 || C <= 0 || F <= 0) return LAPNYS_EINVAL;
  if (dtype != LAPNYS_F32 && dtype != LAPNYS_BF16) return LAPNYS_EINVAL;
  if (T > 1 << 28 || C > 1 << 20 || F > 1 << 20) return LAPNYS_EINVAL;
  // tiles of every product, and their ranges, are counted in 32 bits
  const long long wide = C > F ? C : F, narrow = C > F ? F : C;
  if ((T / kMlpTileM + 1LL) * (wide / 64 + 1) >= 1 << 28 || (wide / 128 + 1) * (narrow / 64 + 1) >= 1 << 24)
    return LAPNYS_EINVAL;
  m.T = T; m.C = C; m.F = F; m.Cp = up8(C); m.Fp = up8(F);
  m.f32 = dtype == LAPNYS_F32;
  m.planes = m.f32 ? 3 : 1;
  m.few = mlp_few_ok(T, C, F, m.f32);
  // what g, u and the gradient of h are summed over in one accumulator (k_mlp.cu)
  if (!m.f32 && !m.few && C > 1 << 16) return LAPNYS_EINVAL;
  // bf16 calls round h and the gradient of (g | u) between the products, which puts the
  // results' errors at 1.4 times their own rounding's, more where few values are summed
  // (1.7 at 4 rows of 64).  Calls of up to 2^28 multiply-adds a product, whose time is
  // launches and latency, keep them in two parts, and the products that read them run over
  // both (16 bits: what is left is the results' own rounding; a training step of 256 rows,
  // 512 x 2048 features: kernels of 112 us for 104, 277 us a step either way).  So do few
  // rows, whose time is the weights' bytes.  Others would take half as long again.
  m.hidden = m.f32 ? 3 : m.few || (double)T * C * F <= 268435456.0 ? 2 : 1;
  m.pack_c = m.f32 || C % 8 != 0;
  m.pack_f = m.f32 || F % 8 != 0;
  return LAPNYS_OK;
}

int feature_blocks(const Mlp& m) { return (m.F + kMlpBlock - 1) / kMlpBlock; }

// ctx: h, then p and q, then their rows' powers of two; of few rows h, then p and q in fp32
// rows
struct Ctx {
  size_t h, pq, scale, total;
};
size_t h_bytes(const Mlp& m) { return align256((size_t)m.hidden * m.T * m.Fp * 2); }
// parts that K runs over beyond the operands' own: the two of h or (dg | du)
int twice(const Mlp& m) { return m.hidden == 2 ? 2 : 1; }
Ctx ctx_of(const Mlp& m) {
  Ctx c;
  const size_t blocks = (size_t)((m.T + 31) / 32) * feature_blocks(m);
  c.h = 0;
  c.pq = h_bytes(m);
  if (m.few) {
    c.scale = 0;
    c.total = c.pq + align256((size_t)2 * m.T * m.F * 4);
    return c;
  }
  c.scale = c.pq + align256(blocks * 2 * 32 * kMlpBlock * (m.f32 ? 4 : 2));
  c.total = c.scale + (m.f32 ? 0 : align256(blocks * 32 * 2));
  return c;
}

// one of the products that may be split over K
struct Split {
  int n;
  size_t bytes;
};
Split split_of(const Mlp& m, int M, int N, int nparts, int K, int kparts) {
  const int bn = mlp_tile_n(m.f32);
  const long long tiles = (long long)((M + kMlpTileM - 1) / kMlpTileM) * ((N + bn - 1) / bn) * nparts;
  const size_t ld = (size_t)up8(N) * nparts;
  Split s;
  s.n = mlp_splits(tiles, (K + kMlpTileK - 1) / kMlpTileK * kparts, (double)M * ld, m.f32);
  s.bytes = s.n > 1 ? align256((size_t)s.n * M * ld * 4) : 0;
  return s;
}

struct Ws {
  size_t x, w_in, w_out, dy, h, dz, part, colsum, total;
};
Ws ws_of(const Mlp& m, bool backward) {
  Ws w;
  memset(&w, 0, sizeof(w));
  size_t o = 0;
  auto room = [&](size_t& at, size_t bytes) {
    at = o;
    o += align256(bytes);
  };
  const size_t two = 2 * (size_t)m.planes;
  room(w.x, m.pack_c ? two * m.T * m.Cp : 0);
  room(w.w_in, m.pack_f && !m.few ? two * m.C * 2 * m.Fp : 0);
  room(w.w_out, m.pack_c && !m.few ? two * m.F * m.Cp : 0);
  size_t part = 0;
  auto most = [&](size_t bytes) { part = bytes > part ? bytes : part; };
  if (!backward) {
    room(w.h, h_bytes(m));
    if (m.few) {
      most(mlp_few_bytes(m.T, m.planes, m.F, 2, m.f32));
      most(mlp_few_bytes(m.T, m.hidden, m.C, 1, m.f32));
    } else {
      most(split_of(m, m.T, m.C, 1, m.F, twice(m)).bytes);
    }
  } else {
    room(w.dy, m.pack_c ? two * m.T * m.Cp : 0);
    room(w.dz, 2 * (size_t)m.hidden * m.T * 2 * m.Fp);
    if (m.few) {
      most(mlp_few_bytes(m.T, m.planes, m.F, 1, m.f32));
      most(mlp_few_bytes(m.T, m.hidden, m.C, 1, m.f32));
    } else {
      most(split_of(m, m.T, m.C, 1, m.F, 2 * twice(m)).bytes);
    }
    most(split_of(m, m.C, m.F, 2, m.T, twice(m)).bytes);
    most(split_of(m, m.F, m.C, 1, m.T, twice(m)).bytes);
    const size_t ci = (size_t)mlp_colsum_ranges(m.T, 2 * m.F) * 2 * m.F * 4;
    const size_t co = (size_t)mlp_colsum_ranges(m.T, m.C) * m.C * 4;
    room(w.colsum, ci > co ? ci : co);
  }
  room(w.part, part);
  w.total = o;
  return w;
}

MlpView view(const void* p, int inner, int parts, int rows, int planes, size_t ld) {
  MlpView v;
  v.p = p; v.inner = inner; v.parts = parts; v.rows = rows; v.planes = planes;
  v.part_stride = ld;
  v.row_stride = ld * parts;
  v.plane_stride = v.row_stride * rows;
  return v;
}

struct Run {
  const Mlp& m;
  uint8_t* ws;
  cudaStream_t st;
  cudaError_t e = cudaSuccess;
  MlpPackArgs pack;

  Run(const Mlp& m_, void* ws_, cudaStream_t st_) : m(m_), ws((uint8_t*)ws_), st(st_) {
    memset(&pack, 0, sizeof(pack));
  }
  // [rows][parts][inner] as the products read it, packed into ws + at where it has to be
  MlpView operand(const void* p, bool packed, size_t at, int rows, int parts, int inner) {
    if (!packed) return view(p, inner, parts, rows, 1, (size_t)inner);
    const int ld = up8(inner);
    MlpPackJob& j = pack.job[pack.jobs++];
    j.src = p;
    j.dst = (__nv_bfloat16*)(ws + at);
    j.rows = (long long)rows * parts;
    j.inner = inner;
    j.ld = ld;
    return view(j.dst, inner, parts, rows, m.planes, (size_t)ld);
  }
  void packs() {
    if (e == cudaSuccess && pack.jobs > 0) e = run_mlp_pack(pack, !m.f32, st);
  }
  // x [T][kparts][K] (planes) times w, few rows
  MlpFewArgs few(const MlpView& x, const void* w, bool kmajor, int N, int nparts, size_t part_at) const {
    MlpFewArgs f;
    memset(&f, 0, sizeof(f));
    f.x = x.p; f.w = w;
    f.ldx = x.row_stride; f.xpart = x.part_stride;
    f.T = m.T; f.planes = x.planes; f.K = x.inner; f.kparts = x.parts; f.N = N; f.nparts = nparts;
    f.kmajor = kmajor;
    f.part = (float*)(ws + part_at);
    return f;
  }
  void run(MlpFewArgs& f) {
    if (e == cudaSuccess) e = run_mlp_few(f, m.f32, st);
  }
  // out[M][nparts][N] = sum over K, split where that is faster
  void rows(const char* name, const MlpView& a, bool amn, const MlpView& b, bool bmn, int M, int N,
            int nparts, int kparts, int K, const void* bias, void* out, size_t part_at) {
    if (e != cudaSuccess) return;
    const Split s = split_of(m, M, N, nparts, K, kparts * twice(m));   // every one reads h or (dg | du)
    MlpGemmArgs g;
    memset(&g, 0, sizeof(g));
    g.M = M; g.N = N; g.nparts = nparts; g.kparts = kparts; g.splits = s.n;
    g.amn = amn; g.bmn = bmn;
    if (s.n == 1) {
      g.bias = bias;
      g.out = out;
      g.ldo = (size_t)nparts * N;
      g.part_out = N;
      g.wide = N % (m.f32 ? 4 : 8) == 0;
      e = run_mlp_gemm(name, kMlpRows, m.f32, false, a, b, g, st);
      return;
    }
    g.out = ws + part_at;
    g.part_out = up8(N);
    g.ldo = g.part_out * nparts;
    e = run_mlp_gemm(name, kMlpPart, m.f32, false, a, b, g, st);
    if (e != cudaSuccess) return;
    MlpReduceArgs r;
    memset(&r, 0, sizeof(r));
    r.part = (const float*)g.out;
    r.ldp = g.ldo;
    r.part_in = g.part_out;
    r.split_stride = (size_t)M * g.ldo;
    r.splits = s.n; r.M = M; r.N = N; r.nparts = nparts;
    r.bias = bias;
    r.out = out;
    r.ldo = (size_t)nparts * N;
    r.part_out = N;
    e = run_mlp_reduce("mlp_reduce", r, !m.f32, st);
  }
  void colsum(const void* src, int planes, size_t ld, size_t plane, int parts, int inner, int pstride,
              void* out, size_t at) {
    if (e != cudaSuccess) return;
    MlpColsumArgs c;
    memset(&c, 0, sizeof(c));
    c.src = src; c.planes = planes; c.ld = ld; c.plane_stride = plane;
    c.rows = m.T; c.inner = inner; c.parts = parts; c.pstride = pstride;
    c.part = (float*)(ws + at);
    c.ranges = mlp_colsum_ranges(m.T, parts * inner);
    c.out = out;
    e = run_mlp_colsum(c, !m.f32, st);
  }
};

MlpKept kept_of(const Mlp& m, void* ctx) {
  MlpKept k = {nullptr, nullptr};
  if (ctx) {
    const Ctx c = ctx_of(m);
    k.pq = (uint8_t*)ctx + c.pq;
    k.scale = (uint16_t*)((uint8_t*)ctx + c.scale);
  }
  return k;
}

}  // namespace
}  // namespace lapnys

using namespace lapnys;

extern "C" {

size_t lapnys_mlp_ctx_bytes(int T, int C, int F, int dtype) {
  Mlp m;
  return check_mlp(m, T, C, F, dtype) == LAPNYS_OK ? ctx_of(m).total : 0;
}

size_t lapnys_mlp_workspace_bytes(int T, int C, int F, int dtype, int backward) {
  Mlp m;
  return check_mlp(m, T, C, F, dtype) == LAPNYS_OK ? ws_of(m, backward != 0).total : 0;
}

int lapnys_mlp_fwd(const void* x, const void* w_in, const void* b_in, const void* w_out,
                   const void* b_out, void* y, int T, int C, int F, int act, cudaStream_t stream,
                   int dtype, void* ctx, size_t ctx_bytes, void* ws, size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_mlp_fwd");
  Mlp m;
  const int rc = check_mlp(m, T, C, F, dtype);
  if (rc != LAPNYS_OK) return rc;
  if (act < LAPNYS_SILU || act > LAPNYS_GELU_TANH) return LAPNYS_EINVAL;
  const void* all[] = {x, w_in, w_out, y};
  for (const void* p : all)
    if (!p || !aligned(p, 16)) return LAPNYS_EINVAL;
  if (!aligned(b_in, 16) || !aligned(b_out, 16) || !aligned(ctx, 16)) return LAPNYS_EINVAL;
  const Ws w = ws_of(m, false);
  if (!ws || !aligned(ws, 16)) return LAPNYS_EINVAL;
  if (ws_bytes < w.total || (ctx && ctx_bytes < ctx_of(m).total)) return LAPNYS_ENOSPC;
  Run r(m, ws, stream);
  const MlpView vx = r.operand(x, m.pack_c, w.x, T, 1, C);
  void* h = ctx ? ctx : r.ws + w.h;
  const MlpView vh = view(h, F, 1, T, m.hidden, m.Fp);
  if (m.few) {
    r.packs();
    MlpFewArgs f = r.few(vx, w_in, false, F, 2, w.part);
    f.mode = kFewGlu; f.act = act; f.out_planes = m.hidden;
    f.bias = b_in; f.out = h; f.ldo = m.Fp;
    if (ctx) {
      f.p = (float*)((uint8_t*)ctx + ctx_of(m).pq);
      f.q = f.p + (size_t)T * F;
    }
    r.run(f);
    f = r.few(vh, w_out, false, C, 1, w.part);
    f.mode = kFewRows; f.second = true;
    f.bias = b_out; f.out = y; f.ldo = C;
    r.run(f);
    return status(r.e);
  }
  const MlpView vi = r.operand(w_in, m.pack_f, w.w_in, C, 2, F);
  const MlpView vo = r.operand(w_out, m.pack_c, w.w_out, F, 1, C);
  r.packs();
  if (r.e == cudaSuccess) {
    MlpGemmArgs g;
    memset(&g, 0, sizeof(g));
    g.M = T; g.N = F; g.nparts = 1; g.kparts = 1; g.splits = 1;
    g.bmn = 1;
    g.act = act;
    g.bias = b_in;
    g.out = h;
    g.ldo = m.Fp;
    g.plane_out = (size_t)T * m.Fp;
    g.kept = kept_of(m, ctx);
    g.fblocks = feature_blocks(m);
    r.e = run_mlp_gemm("mlp_in", kMlpGlu, m.f32, m.hidden == 2, vx, vi, g, stream);
  }
  r.rows("mlp_out", vh, false, vo, true, T, C, 1, 1, F, b_out, y, w.part);
  return status(r.e);
}

int lapnys_mlp_bwd(const void* x, const void* w_in, const void* w_out, const void* dy,
                   const void* ctx, void* dx, void* dw_in, void* db_in, void* dw_out, void* db_out,
                   int T, int C, int F, cudaStream_t stream, int dtype, void* ws, size_t ws_bytes) {
  NvtxScope nvtx_scope("lapnys_mlp_bwd");
  Mlp m;
  const int rc = check_mlp(m, T, C, F, dtype);
  if (rc != LAPNYS_OK) return rc;
  const void* all[] = {x, w_in, w_out, dy, ctx, ws};
  for (const void* p : all)
    if (!p || !aligned(p, 16)) return LAPNYS_EINVAL;
  const void* outs[] = {dx, dw_in, db_in, dw_out, db_out};
  for (const void* p : outs)
    if (!aligned(p, 16)) return LAPNYS_EINVAL;
  const Ws w = ws_of(m, true);
  if (ws_bytes < w.total) return LAPNYS_ENOSPC;
  Run r(m, ws, stream);
  const bool hidden = dx || dw_in || db_in;     // the gradient of z is needed
  MlpView vx, vi, vo, vy;
  if (dw_in) vx = r.operand(x, m.pack_c, w.x, T, 1, C);
  if (dx && !m.few) vi = r.operand(w_in, m.pack_f, w.w_in, C, 2, F);
  if (hidden && !m.few) vo = r.operand(w_out, m.pack_c, w.w_out, F, 1, C);
  if (hidden || dw_out) vy = r.operand(dy, m.pack_c, w.dy, T, 1, C);
  r.packs();
  __nv_bfloat16* dz = (__nv_bfloat16*)(r.ws + w.dz);
  const MlpView vz = view(dz, F, 2, T, m.hidden, m.Fp);
  if (hidden && m.few) {
    MlpFewArgs f = r.few(vy, w_out, true, F, 1, w.part);
    f.mode = kFewDglu; f.out_planes = m.hidden;
    f.out = dz; f.ldo = m.Fp;
    f.p = (float*)((uint8_t*)const_cast<void*>(ctx) + ctx_of(m).pq);
    f.q = f.p + (size_t)T * F;
    r.run(f);
    if (dx) {
      f = r.few(vz, w_in, true, C, 1, w.part);
      f.mode = kFewRows; f.second = true;
      f.out = dx; f.ldo = C;
      r.run(f);
    }
  } else if (hidden && r.e == cudaSuccess) {
    MlpGemmArgs g;
    memset(&g, 0, sizeof(g));
    g.M = T; g.N = F; g.nparts = 1; g.kparts = 1; g.splits = 1;
    g.out = dz;
    g.ldo = 2 * (size_t)m.Fp;
    g.part_out = m.Fp;
    g.plane_out = (size_t)T * 2 * m.Fp;
    g.kept = kept_of(m, const_cast<void*>(ctx));
    g.fblocks = feature_blocks(m);
    r.e = run_mlp_gemm("mlp_dhidden", kMlpDglu, m.f32, m.hidden == 2, vy, vo, g, stream);
  }
  if (dx && !m.few) r.rows("mlp_dx", vz, false, vi, false, T, C, 1, 2, F, nullptr, dx, w.part);
  if (dw_in) r.rows("mlp_dw_in", vx, true, vz, true, C, F, 2, 1, T, nullptr, dw_in, w.part);
  const MlpView vh = view(ctx, F, 1, T, m.hidden, m.Fp);
  if (dw_out) r.rows("mlp_dw_out", vh, true, vy, true, F, C, 1, 1, T, nullptr, dw_out, w.part);
  if (db_in)
    r.colsum(dz, m.hidden, 2 * (size_t)m.Fp, (size_t)T * 2 * m.Fp, 2, F, m.Fp, db_in, w.colsum);
  if (db_out) r.colsum(dy, m.f32 ? 0 : 1, C, 0, 1, C, C, db_out, w.colsum);
  return status(r.e);
}

}  // extern "C"
