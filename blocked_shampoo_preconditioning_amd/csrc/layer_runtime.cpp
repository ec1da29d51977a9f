// Host side of include/shampoo_layer.h: argument checks, the workspace's
// layout and the launches of the feed-forward half of a decoder layer.
#include "../../include/shampoo_layer.h"

#include <cmath>
#include <exception>

#include "layer_kernels.h"
#include "runtime_common.h"

using shp_rt::Carver;
using shp_rt::fail;

namespace {

constexpr int64_t kMaxLd = int64_t(1) << 21;  // 256 rows of an operand stay within 32-bit byte offsets
constexpr int64_t kMaxDim = (int64_t(1) << 31) - 1024;

int64_t round8(int64_t v) { return (v + 7) / 8 * 8; }
bool aligned(const void* p, int64_t a) { return reinterpret_cast<uintptr_t>(p) % a == 0; }

int check_matrix(const char* name, const void* p, int64_t rows, int64_t cols, int64_t ld, int64_t esize, int64_t max_ld) {
  if (rows == 0 || cols == 0) return SHAMPOO_OK;
  if (!p) return fail(SHAMPOO_ERR_INVALID_ARG, std::string(name) + " is NULL");
  if (ld < cols || ld > max_ld)
    return fail(SHAMPOO_ERR_INVALID_ARG, std::string(name) + ": leading dimension " + std::to_string(ld) +
                                             " is not in [" + std::to_string(cols) + ", " + std::to_string(max_ld) + "]");
  if (!aligned(p, esize)) return fail(SHAMPOO_ERR_MISALIGNED, std::string(name) + " is not aligned to its element size");
  return SHAMPOO_OK;
}

int check_dtype(int32_t dtype) {
  if (dtype != SHAMPOO_F32 && dtype != SHAMPOO_BF16)
    return fail(SHAMPOO_ERR_UNSUPPORTED, "dtype must be SHAMPOO_F32 or SHAMPOO_BF16");
  return SHAMPOO_OK;
}

#define RC(expr)                  \
  do {                            \
    if (int rc_ = (expr)) return rc_; \
  } while (0)

// No C++ exception crosses the C boundary.
template <class F>
int guarded(F&& f) {
  try {
    return f();
  } catch (const std::exception& e) {
    return fail(SHAMPOO_ERR_INVALID_ARG, e.what());
  } catch (...) {
    return fail(SHAMPOO_ERR_INVALID_ARG, "unknown C++ exception");
  }
}

// ------------------------------------------------- gated feed-forward block
// Tile and K splits of the products of one launch, by an estimate of its time in
// microseconds. bf16: a K step of 64 takes 1.6 for a 256 tile alone on its CU,
// 0.92 for two 128 tiles on one and 0.72 for one alone, with two sets of waves
// 0.43 on a part of the card and 0.55 on the whole (the L2s' rate), which is what
// is reckoned with. fp32: a K step of 32, six products, takes 2.5 for a 128 x 256
// tile and 1.35 for a 128 tile (2.0 for the gate's, whose four waves are alone on
// the CU). Workgroups of unequal length fill the card about as well as equal ones
// of the same total, but the launch takes at least its longest one's time. Filling
// and emptying costs 5, 3 or 4, a split another launch and its sums' way through
// memory. Measured with the choices left open (a whole step, us): dx of 2048 x
// 2048 x 8192 as 256 tiles in 4 parts 656, as 128 tiles unsplit 709; dWg and dWu
// of 1024 x 768 x 2048 as unsplit 128 tiles 114, in two parts 122, y of that size
// unsplit 124, in 4 parts 118; y of 4096 x 768 x 2048 with one set of waves 159,
// with two 156, its g, u and h as 256 tiles 155, as 128 tiles 161. fp32, first the
// choice, then the other tile's best: 4096 x 768 x 2048 g, u and h 625 as 128 x
// 256 tiles (734), dx with the weights' gradients 639 (665); 300 x 512 x 1024
// those 80 as 128 tiles in 8 parts (90), y 79 (84).
struct Shape {
  int64_t M, N;
  int problems;
  bool gate;
  int64_t steps;
  int32_t splits;
};

double estimate(const Shape* p, int n, shl::TileKind tile, bool f32) {
  double work = 0, longest = 0, extra = 0;
  int64_t groups = 0;
  for (int i = 0; i < n; ++i) {
    if (p[i].M == 0) continue;
    const int64_t tiles = shl::gemm_tiles(p[i].M, p[i].N, p[i].problems, tile, p[i].gate);
    const double each = static_cast<double>((p[i].steps + p[i].splits - 1) / p[i].splits);
    groups += tiles * p[i].splits;
    work += static_cast<double>(tiles * p[i].splits) * each;
    longest = each > longest ? each : longest;
    if (p[i].splits > 1)
      extra += 4 + static_cast<double>(p[i].M) * static_cast<double>(p[i].N) * p[i].problems * (p[i].gate ? 2 : 1) * 6 / 4e6 * p[i].splits;
  }
  const bool big = tile == shl::kTile256 || tile == shl::kTileWide, alone = f32 || tile != shl::kTile128 || groups <= 256;
  const double step = f32 ? big ? 2.5 : p[0].gate ? 2.0 : 1.35 : big ? 1.6 : tile == shl::kTile128x2 ? 0.55 : alone ? 0.72 : 0.92;
  const double slots = alone ? 256 : 512;
  // equal workgroups go in whole rounds; unequal ones about half a round apart
  const double mean = work / static_cast<double>(groups > 0 ? groups : 1);
  double rounds = static_cast<double>(groups) / slots;
  rounds = n == 1 ? static_cast<double>(static_cast<int64_t>(rounds + 0.999)) : rounds < 1 ? 1 : rounds + 0.25;
  double t = rounds * mean * step;
  t = t > longest * step ? t : longest * step;
  return t + (big ? 5 : tile == shl::kTile128x2 ? 4 : 3) * (rounds > 1 ? rounds : 1) + extra;
}

// One product.
constexpr shl::TileKind kTiles[] = {shl::kTile256, shl::kTile128, shl::kTile128x2, shl::kTileWide};

shl::TileKind choose_tile(Shape p, int32_t& splits, bool f32) {
  shl::TileKind tile = shl::kTile128;
  double best = -1;
  for (shl::TileKind t : kTiles) {
    if (!shl::is_tile(t, f32)) continue;
    for (int32_t s = 1; s <= 32 && (s == 1 || s * 4 <= p.steps); ++s) {
      p.splits = s;
      const double us = estimate(&p, 1, t, f32);
      if (best < 0 || us < best) best = us, tile = t, splits = s;
    }
  }
  return tile;
}

// dx (p[0]) with dWd and dWg, dWu (p[1], p[2], whose sums are equally long).
shl::TileKind choose_group(Shape (&p)[3], bool f32) {
  static const int32_t kSplits[] = {1, 2, 3, 4, 6, 8, 12, 16, 24, 32};
  shl::TileKind tile = shl::kTile128;
  double best = -1;
  int32_t a = 1, b = 1;
  for (shl::TileKind t : kTiles) {
    if (!shl::is_tile(t, f32)) continue;
    for (int32_t sa : kSplits) {
      if (sa > 1 && (p[0].M == 0 || sa * 4 > p[0].steps)) break;
      for (int32_t sb : kSplits) {
        if (sb > 1 && (p[1].M + p[2].M == 0 || sb * 4 > p[2].steps)) break;
        p[0].splits = sa, p[1].splits = p[2].splits = sb;
        const double us = estimate(p, 3, t, f32);
        if (best < 0 || us < best) best = us, tile = t, a = sa, b = sb;
      }
    }
  }
  p[0].splits = a, p[1].splits = p[2].splits = b;
  return tile;
}

// A product's operand: its first plane, elements from one plane to the next.
struct Planes {
  const uint16_t* p = nullptr;
  int64_t ld = 0, plane = 0;
};

// One pass over the block's launches: with run = false only the workspace is
// laid out.
struct Ffn {
  const shampoo_ffn_t& a;
  const shl::NormArgs* norm;  // of bf16 x, where g and u are to be taken from it unrounded
  char* ws;
  hipStream_t stream;
  bool run;
  Carver carve{};
  hipError_t err = hipSuccess;
  int64_t N, d, f, fp, e;
  bool f32;
  shl::PackList list{};

  Ffn(const shampoo_ffn_t& a_, const shl::NormArgs* norm_, char* ws_, hipStream_t s, bool run_)
      : a(a_), norm(norm_), ws(ws_), stream(s), run(run_) {
    N = a.tokens, d = a.d_model, f = a.d_hidden, fp = round8(f);
    f32 = a.dtype == SHAMPOO_F32;
    e = f32 ? 4 : 2;
    list.f32 = f32;
  }
  void* take(int64_t bytes) { return ws + carve.take(bytes); }
  void ok(hipError_t x) {
    if (err == hipSuccess) err = x;
  }
  // `saved`: g, u, and h, which fp32 keeps as the planes that its second product
  // reads (as an fp32 array where the forward pass took the few-token kernels).
  int64_t act_bytes() const { return shp_rt::align_up(N * fp * e); }
  int64_t saved_bytes() const { return 2 * act_bytes() + shp_rt::align_up(N * fp * 2 * shl::planes(f32)); }
  char* saved_h() const { return static_cast<char*>(a.saved) + 2 * act_bytes(); }

  // A bf16 operand that loads can take where it is; sums_over_cols: its
  // columns are the product's summation index.
  bool usable(const void* p, int64_t cols, int64_t ld, bool sums_over_cols) const {
    return !f32 && aligned(p, 16) && ld % 8 == 0 && (!sums_over_cols || cols % 8 == 0);
  }
  Planes operand(const void* p, int64_t rows, int64_t cols, int64_t ld, bool sums_over_cols) {
    if (!usable(p, cols, ld, sums_over_cols)) return copied(p, rows, cols, ld);
    return {static_cast<const uint16_t*>(p), ld, 0};
  }
  // h, dg and du as the epilogues write them: what the next products read.
  Planes written(const void* p) const { return {static_cast<const uint16_t*>(p), fp, f32 ? N * fp : 0}; }
  // Puts a copy on the list; flush() makes it.
  Planes copied(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    const int64_t ld_out = round8(cols);
    uint16_t* out = static_cast<uint16_t*>(take(shl::planes(f32) * rows * ld_out * 2));
    if (rows) list.t[list.n++] = shl::PackArgs{p, out, rows, cols, ld, ld_out};
    return {out, ld_out, rows * ld_out};
  }
  // Both weights of the fused products share one leading dimension.
  void operands(const void* p, const void* q, int64_t rows, int64_t cols, int64_t ldp, int64_t ldq, bool sums_over_cols, Planes& x,
                Planes& y) {
    const bool in_place = ldp == ldq && usable(p, cols, ldp, sums_over_cols) && usable(q, cols, ldq, sums_over_cols);
    x = in_place ? operand(p, rows, cols, ldp, sums_over_cols) : copied(p, rows, cols, ldp);
    y = in_place ? operand(q, rows, cols, ldq, sums_over_cols) : copied(q, rows, cols, ldq);
  }
  // Makes the listed copies.
  void flush() {
    if (run) ok(shl::launch_pack(list, stream));
    list.n = 0;
  }

  // Adds a product to the segments of one sum.
  void segment(shl::GemmArgs& g, const Planes& A, const Planes& B, const Planes* B1 = nullptr) {
    g.a[g.nseg] = A.p, g.b[0][g.nseg] = B.p;
    if (B1) g.b[1][g.nseg] = B1->p;
    ++g.nseg;
    g.lda = A.ld, g.ldb = B.ld, g.plane_a = A.plane, g.plane_b = B.plane;
  }

  Shape shape(const shl::GemmArgs& g, bool gate) const {
    return {g.M, g.M ? g.N : 0, g.problems, gate, shl::gemm_steps(g.K, g.nseg, f32), 1};
  }
  void settle(shl::GemmArgs& g, bool gate) {
    g.f32 = f32 ? 1 : 0;
    g.e.act = a.activation;
    if (g.splits > 1)
      g.partial = static_cast<float*>(take(int64_t(4) * g.splits * g.problems * (gate ? 2 : 1) * g.M * g.N));
  }
  void product(shl::GemmArgs& g, bool a_cols, bool b_cols, shl::Epi epi) {
    const bool gate = epi == shl::kGate;
    const shl::TileKind tile = choose_tile(shape(g, gate), g.splits, f32);
    settle(g, gate);
    if (run) ok(shl::launch_gemm(g, tile, a_cols, b_cols, epi, stream));
  }
  void group(shl::GroupArgs& q) {
    Shape p[3] = {shape(q.g[0], false), shape(q.g[1], false), shape(q.g[2], false)};
    const shl::TileKind tile = choose_group(p, f32);
    for (int i = 0; i < 3; ++i) {
      q.g[i].splits = p[i].splits;
      settle(q.g[i], false);
    }
    if (run) ok(shl::launch_group(q, tile, f32, stream));
  }

  // Whether the forward pass takes the few-token kernels. The sizes alone decide,
  // so that results do not go by strides and the backward pass knows in which
  // form fp32 h was kept.
  bool few() const { return N <= shl::decode_tokens(f32) && d >= 2 && f >= 2; }
  // A weight as they read it: bf16 in pairs of columns, so rows that are not 4-byte
  // aligned are copied.
  Planes few_weight(const void* p, int64_t rows, int64_t cols, int64_t ld) {
    if (f32 || (aligned(p, 4) && ld % 2 == 0)) return {static_cast<const uint16_t*>(p), ld, 0};
    return copied(p, rows, cols, ld);
  }
  // The forward products of a few tokens.
  void few_product(shl::DecodeArgs& g, shl::Epi epi) {
    const int64_t groups = shl::decode_groups(g.N), batches = shl::decode_batches(g.K);
    int64_t s = 1;
    if (groups < 192) {
      s = 512 / groups;
      const int64_t most = f32 || N > 16 ? batches / 16 : batches / 32;  // two batches for each wave
      if (s > most) s = most;
      if (s > 32) s = 32;
    }
    g.splits = static_cast<int32_t>(s < 1 ? 1 : s);
    g.e.act = a.activation;
    if (g.splits > 1)
      g.partial = static_cast<float*>(take(int64_t(4) * g.splits * (epi == shl::kGate ? 2 : 1) * g.M * g.N));
    if (run) ok(shl::launch_decode(g, f32, epi, stream));
  }
  void forward_few() {
    char* saved = static_cast<char*>(a.saved);
    void* h = saved ? saved_h() : take(N * fp * e);
    void* rest = f32 ? nullptr : take(N * fp * e);  // the second term of bf16 h
    const Planes wg = few_weight(a.w_gate, d, f, a.ld_gate), wu = few_weight(a.w_up, d, f, a.ld_up);
    const Planes wd = few_weight(a.w_down, f, d, a.ld_down);
    flush();
    shl::DecodeArgs g{};
    g.x = a.x, g.ldx = a.ld_x, g.w[0] = wg.p, g.w[1] = wu.p, g.ldw[0] = wg.ld, g.ldw[1] = wu.ld;
    g.M = static_cast<int32_t>(N), g.N = static_cast<int32_t>(f), g.K = static_cast<int32_t>(d);
    g.e.c[0] = h, g.e.c[1] = rest, g.e.ldc = fp, g.e.ldg = fp, g.e.pad_to = static_cast<int32_t>(fp);
    if (saved) g.e.g = saved, g.e.u = saved + act_bytes();
    few_product(g, shl::kGate);
    shl::DecodeArgs y{};
    y.x = h, y.x_rest = rest, y.ldx = fp, y.w[0] = wd.p, y.ldw[0] = wd.ld;
    y.M = static_cast<int32_t>(N), y.N = static_cast<int32_t>(d), y.K = static_cast<int32_t>(f);
    y.e.c[0] = a.y, y.e.ldc = a.ld_y;
    few_product(y, shl::kStore);
  }

  void forward() {
    if (few() && !norm) return forward_few();
    // With a second term both have the same leading dimension, of whole groups. It
    // doubles the first product (forward of 4096 x 768 x 2048 56 -> 80 us) where one
    // term leaves dx and dWg 2 to 4% wrong; SiLU and GELU are 0.5% off either way.
    const Planes x = !norm || a.ld_x == round8(d) ? operand(a.x, N, d, a.ld_x, true) : copied(a.x, N, d, a.ld_x);
    Planes rest = x;
    if (norm) {
      uint16_t* out = static_cast<uint16_t*>(take(N * x.ld * 2));
      rest.p = out;
      if (run) ok(shl::launch_norm_rest(*norm, out, x.ld, stream));
    }
    Planes wg, wu;
    operands(a.w_gate, a.w_up, d, f, a.ld_gate, a.ld_up, false, wg, wu);
    const Planes wd = operand(a.w_down, f, d, a.ld_down, false);
    flush();
    char* saved = static_cast<char*>(a.saved);
    const Planes h = written(saved ? saved_h() : take(N * fp * 2 * shl::planes(f32)));
    {
      shl::GemmArgs g{};
      if (norm) segment(g, rest, wg, &wu);
      segment(g, x, wg, &wu);
      g.M = static_cast<int32_t>(N), g.N = static_cast<int32_t>(f), g.K = static_cast<int32_t>(round8(d));
      g.k_real = static_cast<int32_t>(d), g.problems = 1;
      g.e.c[0] = const_cast<uint16_t*>(h.p), g.e.ldc = fp, g.e.ldg = fp, g.e.pad_to = static_cast<int32_t>(fp), g.e.plane = h.plane;
      if (saved) g.e.g = saved, g.e.u = saved + act_bytes();
      product(g, false, true, shl::kGate);
    }
    shl::GemmArgs g{};
    segment(g, h, wd);
    g.M = static_cast<int32_t>(N), g.N = static_cast<int32_t>(d), g.K = static_cast<int32_t>(fp);
    g.k_real = static_cast<int32_t>(f), g.problems = 1;
    g.e.c[0] = a.y, g.e.ldc = a.ld_y;
    product(g, false, true, shl::kStore);
  }

  void backward() {
    char* saved = static_cast<char*>(a.saved);
    const bool want_gate = a.dx || a.dw_gate;
    // dy is read by rows for dh and by columns for dWd: one copy serves both
    const Planes dy = operand(a.dy, N, d, a.ld_dy, true);
    Planes wd, h, wg, wu, x;
    if (want_gate) wd = operand(a.w_down, f, d, a.ld_down, true);
    if (a.dw_down) h = f32 && few() ? copied(saved_h(), N, fp, fp) : written(saved_h());
    if (a.dx) operands(a.w_gate, a.w_up, d, f, a.ld_gate, a.ld_up, true, wg, wu);
    if (a.dw_gate) x = operand(a.x, N, d, a.ld_x, false);
    flush();
    Planes pg, pu;
    if (want_gate) {
      pg = written(take(N * fp * 2 * shl::planes(f32)));
      pu = written(take(N * fp * 2 * shl::planes(f32)));
      shl::GemmArgs g{};
      segment(g, dy, wd);
      g.M = static_cast<int32_t>(N), g.N = static_cast<int32_t>(f), g.K = static_cast<int32_t>(round8(d));
      g.k_real = static_cast<int32_t>(d), g.problems = 1;
      g.e.c[0] = const_cast<uint16_t*>(pg.p), g.e.c[1] = const_cast<uint16_t*>(pu.p), g.e.ldc = fp, g.e.plane = pg.plane;
      g.e.g = saved, g.e.u = saved + act_bytes(), g.e.ldg = fp;
      g.e.pad_to = static_cast<int32_t>(fp);
      product(g, false, false, shl::kActBwd);
    }
    shl::GroupArgs q{};
    if (a.dx) {
      shl::GemmArgs& g = q.g[0];
      segment(g, pg, wg);
      segment(g, pu, wu);
      g.M = static_cast<int32_t>(N), g.N = static_cast<int32_t>(d), g.K = static_cast<int32_t>(fp);
      g.k_real = static_cast<int32_t>(f), g.problems = 1;
      g.e.c[0] = a.dx, g.e.ldc = a.ld_dx;
    }
    if (a.dw_down) {
      shl::GemmArgs& g = q.g[1];
      segment(g, h, dy);
      g.M = static_cast<int32_t>(f), g.N = static_cast<int32_t>(d), g.K = g.k_real = static_cast<int32_t>(N), g.problems = 1;
      g.e.c[0] = a.dw_down, g.e.ldc = a.ld_dw_down;
    }
    if (a.dw_gate) {
      shl::GemmArgs& g = q.g[2];
      segment(g, x, pg, &pu);
      g.M = static_cast<int32_t>(d), g.N = static_cast<int32_t>(f), g.K = g.k_real = static_cast<int32_t>(N), g.problems = 2;
      g.e.c[0] = a.dw_gate, g.e.c[1] = a.dw_up, g.e.ldc = a.ld_dw_gate, g.e.ldc1 = a.ld_dw_up;
    }
    group(q);
  }
};

int check_sizes(const shampoo_ffn_t* a) {
  if (!a) return fail(SHAMPOO_ERR_INVALID_ARG, "arguments are NULL");
  if (a->tokens < 0 || a->d_model < 1 || a->d_hidden < 1 || a->tokens > kMaxDim || a->d_model > kMaxLd || a->d_hidden > kMaxLd)
    return fail(SHAMPOO_ERR_INVALID_ARG, "tokens must be in [0, 2^31 - 1024], d_model and d_hidden in [1, 2^21]");
  RC(check_dtype(a->dtype));
  if (a->activation < SHAMPOO_ACT_SILU || a->activation > SHAMPOO_ACT_RELU)
    return fail(SHAMPOO_ERR_UNSUPPORTED, "activation must be one of shampoo_activation_t");
  return SHAMPOO_OK;
}

int check_ffn(const shampoo_ffn_t* a, bool backward) {
  RC(check_sizes(a));
  const int64_t e = a->dtype == SHAMPOO_F32 ? 4 : 2;
  RC(check_matrix("x", a->x, a->tokens, a->d_model, a->ld_x, e, kMaxLd));
  RC(check_matrix("w_gate", a->w_gate, a->d_model, a->d_hidden, a->ld_gate, e, kMaxLd));
  RC(check_matrix("w_up", a->w_up, a->d_model, a->d_hidden, a->ld_up, e, kMaxLd));
  RC(check_matrix("w_down", a->w_down, a->d_hidden, a->d_model, a->ld_down, e, kMaxLd));
  if (a->saved && !aligned(a->saved, 256)) return fail(SHAMPOO_ERR_MISALIGNED, "saved is not aligned to 256 bytes");
  if (!backward) return check_matrix("y", a->y, a->tokens, a->d_model, a->ld_y, e, kMaxLd);
  if (!a->saved && a->tokens) return fail(SHAMPOO_ERR_INVALID_ARG, "saved is NULL: the forward pass has to keep g, u and h");
  RC(check_matrix("dy", a->dy, a->tokens, a->d_model, a->ld_dy, e, kMaxLd));
  if (!a->dw_gate != !a->dw_up) return fail(SHAMPOO_ERR_INVALID_ARG, "dw_gate and dw_up are computed together: give both or none");
  if (a->dx) RC(check_matrix("dx", a->dx, a->tokens, a->d_model, a->ld_dx, e, kMaxLd));
  if (a->dw_gate) {
    RC(check_matrix("dw_gate", a->dw_gate, a->d_model, a->d_hidden, a->ld_dw_gate, e, kMaxLd));
    RC(check_matrix("dw_up", a->dw_up, a->d_model, a->d_hidden, a->ld_dw_up, e, kMaxLd));
  }
  if (a->dw_down) RC(check_matrix("dw_down", a->dw_down, a->d_hidden, a->d_model, a->ld_dw_down, e, kMaxLd));
  return SHAMPOO_OK;
}

int64_t ffn_workspace(const shampoo_ffn_t* a, const shl::NormArgs* norm, bool backward) {
  Ffn p(*a, norm, nullptr, nullptr, false);
  backward ? p.backward() : p.forward();
  return p.carve.o;
}

// The launches of a checked call.
int run_ffn(const shampoo_ffn_t* a, const shl::NormArgs* norm, void* workspace, size_t bytes, void* stream, bool backward) {
  const int64_t need = ffn_workspace(a, norm, backward);
  if (need > 0 && !workspace) return fail(SHAMPOO_ERR_INVALID_ARG, "workspace is NULL");
  if (!aligned(workspace, 256)) return fail(SHAMPOO_ERR_MISALIGNED, "workspace is not aligned to 256 bytes");
  if (bytes < static_cast<size_t>(need))
    return fail(SHAMPOO_ERR_WORKSPACE_TOO_SMALL,
                "workspace has " + std::to_string(bytes) + " bytes, the call needs " + std::to_string(need));
  Ffn p(*a, norm, static_cast<char*>(workspace), static_cast<hipStream_t>(stream), true);
  backward ? p.backward() : p.forward();
  return p.err == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(p.err, backward ? "shampoo_ffn_backward" : "shampoo_ffn_forward");
}

// --------------------------------------------------------- norms and dropout
int make_drop(double p, uint64_t seed, uint32_t offset, shl::DropArgs& d) {
  if (!(p >= 0.0 && p < 1.0)) return fail(SHAMPOO_ERR_INVALID_ARG, "dropout must be in [0, 1)");
  const double t = std::nearbyint(p * 65536.0);
  d.threshold = static_cast<uint32_t>(t > 65535.0 ? 65535.0 : t);
  d.scale = static_cast<float>(65536.0 / (65536.0 - d.threshold));
  d.key0 = static_cast<uint32_t>(seed);
  d.key1 = static_cast<uint32_t>(seed >> 32);
  d.offset = offset;
  return SHAMPOO_OK;
}

constexpr int64_t kAnyLd = int64_t(1) << 40;

int check_vector(const char* name, const void* p, int64_t e) {
  if (p && !aligned(p, e)) return fail(SHAMPOO_ERR_MISALIGNED, std::string(name) + " is not aligned to its element size");
  return SHAMPOO_OK;
}

int check_norm(const shampoo_norm_t* a, bool backward) {
  if (!a) return fail(SHAMPOO_ERR_INVALID_ARG, "arguments are NULL");
  if (a->rows < 0 || a->rows > (int64_t(1) << 40)) return fail(SHAMPOO_ERR_INVALID_ARG, "rows must be in [0, 2^40]");
  if (a->width < 1) return fail(SHAMPOO_ERR_INVALID_ARG, "width must be at least 1");
  if (a->width > shl::kMaxNormWidth)
    return fail(SHAMPOO_ERR_UNSUPPORTED, "width is over " + std::to_string(shl::kMaxNormWidth) + ": a row stays in one workgroup's registers");
  RC(check_dtype(a->dtype));
  for (int32_t k : {a->post_kind, a->next_kind})
    if (k < SHAMPOO_NORM_NONE || k > SHAMPOO_NORM_LAYER)
      return fail(SHAMPOO_ERR_UNSUPPORTED, "norm kinds must be of shampoo_norm_kind_t");
  if (!(a->eps > 0.f) || !std::isfinite(a->eps)) return fail(SHAMPOO_ERR_INVALID_ARG, "eps must be positive and finite");
  if (!std::isfinite(a->residual_scale)) return fail(SHAMPOO_ERR_INVALID_ARG, "residual_scale must be finite");
  if (a->gate && a->rows_per_gate < 1) return fail(SHAMPOO_ERR_INVALID_ARG, "rows_per_gate must be at least 1");
  if (!a->z && a->next_kind == SHAMPOO_NORM_NONE) return fail(SHAMPOO_ERR_INVALID_ARG, "neither z nor a next norm: nothing to compute");
  if (a->post_kind == SHAMPOO_NORM_NONE && (a->post_weight || a->post_bias))
    return fail(SHAMPOO_ERR_INVALID_ARG, "post_weight and post_bias need a post norm");
  if (a->next_kind == SHAMPOO_NORM_NONE && (a->next_weight || a->next_bias))
    return fail(SHAMPOO_ERR_INVALID_ARG, "next_weight and next_bias need a next norm");
  if (!a->z && (a->gate || a->post_weight || a->post_bias))
    return fail(SHAMPOO_ERR_INVALID_ARG, "gate, post_weight and post_bias need z");
  const int64_t e = a->dtype == SHAMPOO_F32 ? 4 : 2, n = a->rows, d = a->width;
  if (a->z) RC(check_matrix("z", a->z, n, d, a->ld_z, e, kAnyLd));
  if (a->gate) RC(check_matrix("gate", a->gate, n ? (n - 1) / a->rows_per_gate + 1 : 0, d, a->ld_gate, e, kAnyLd));
  RC(check_vector("post_weight", a->post_weight, e));
  RC(check_vector("post_bias", a->post_bias, e));
  RC(check_vector("next_weight", a->next_weight, e));
  RC(check_vector("next_bias", a->next_bias, e));
  if (a->stats && !aligned(a->stats, 16)) return fail(SHAMPOO_ERR_MISALIGNED, "stats is not aligned to 16 bytes");
  if (!backward) {
    RC(check_matrix("x", a->x, n, d, a->ld_x, e, kAnyLd));
    if (a->z) RC(check_matrix("r", a->r, n, d, a->ld_r, e, kAnyLd));
    if (a->next_kind != SHAMPOO_NORM_NONE) RC(check_matrix("n", a->n, n, d, a->ld_n, e, kAnyLd));
    return SHAMPOO_OK;
  }
  if (!a->stats && n) return fail(SHAMPOO_ERR_INVALID_ARG, "stats is NULL: the forward pass has to keep them");
  if (a->next_kind != SHAMPOO_NORM_NONE) {
    if (a->z)
      RC(check_matrix("r", a->r, n, d, a->ld_r, e, kAnyLd));
    else
      RC(check_matrix("x", a->x, n, d, a->ld_x, e, kAnyLd));
    RC(check_matrix("dn", a->dn, n, d, a->ld_dn, e, kAnyLd));
  } else if (!a->dr && n) {
    return fail(SHAMPOO_ERR_INVALID_ARG, "dr is NULL and there is no next norm: no gradient comes in");
  }
  if (a->dr) RC(check_matrix("dr", a->dr, n, d, a->ld_dr, e, kAnyLd));
  if (a->dx) RC(check_matrix("dx", a->dx, n, d, a->ld_dx, e, kAnyLd));
  if (a->dz) {
    if (!a->z) return fail(SHAMPOO_ERR_INVALID_ARG, "dz needs z");
    RC(check_matrix("dz", a->dz, n, d, a->ld_dz, e, kAnyLd));
  }
  if (a->d_gate) {
    if (!a->gate) return fail(SHAMPOO_ERR_INVALID_ARG, "d_gate needs gate");
    RC(check_matrix("d_gate", a->d_gate, n ? (n - 1) / a->rows_per_gate + 1 : 0, d, a->ld_d_gate, e, kAnyLd));
  }
  if ((a->d_post_weight || a->d_post_bias) && (!a->z || a->post_kind == SHAMPOO_NORM_NONE))
    return fail(SHAMPOO_ERR_INVALID_ARG, "d_post_weight and d_post_bias need z and a post norm");
  if ((a->d_next_weight || a->d_next_bias) && a->next_kind == SHAMPOO_NORM_NONE)
    return fail(SHAMPOO_ERR_INVALID_ARG, "d_next_weight and d_next_bias need a next norm");
  RC(check_vector("d_post_weight", a->d_post_weight, e));
  RC(check_vector("d_post_bias", a->d_post_bias, e));
  RC(check_vector("d_next_weight", a->d_next_weight, e));
  RC(check_vector("d_next_bias", a->d_next_bias, e));
  return SHAMPOO_OK;
}

int norm_args(const shampoo_norm_t* a, bool backward, shl::NormArgs& k) {
  k = shl::NormArgs{};
  k.z = a->z, k.x = a->x, k.ldz = a->ld_z, k.ldx = a->ld_x;
  k.r = a->r, k.n = a->n, k.ldr = a->ld_r, k.ldn = a->ld_n;
  if (backward && !a->z) k.r = const_cast<void*>(a->x), k.ldr = a->ld_x;
  k.w_post = a->post_weight, k.b_post = a->post_bias, k.gate = a->gate, k.w_next = a->next_weight, k.b_next = a->next_bias;
  k.ld_gate = a->ld_gate, k.stats = a->stats;
  k.dr = a->dr, k.dn = a->dn, k.lddr = a->ld_dr, k.lddn = a->ld_dn;
  k.dx = a->dx, k.dz = a->dz, k.lddx = a->ld_dx, k.lddz = a->ld_dz;
  k.dw_post = a->d_post_weight, k.db_post = a->d_post_bias, k.dgate = a->d_gate, k.dw_next = a->d_next_weight;
  k.db_next = a->d_next_bias, k.ld_dgate = a->ld_d_gate;
  // over the rows it is one gate row for all: the kernels and launches add rows
  // to it, which must not pass 2^63
  k.rows = a->rows, k.rows_per_gate = a->gate && a->rows > 0 ? (a->rows_per_gate < a->rows ? a->rows_per_gate : a->rows) : 1;
  k.d = static_cast<int32_t>(a->width), k.f32 = a->dtype == SHAMPOO_F32 ? 1 : 0;
  k.post_kind = a->post_kind, k.next_kind = a->next_kind;
  // without z nothing is scaled: the norm's input is x itself
  k.eps = a->eps, k.alpha = a->z ? a->residual_scale : 1.f;
  return make_drop(a->dropout, a->seed, a->offset, k.drop);
}

// The norm that made a block's x; `used`: whether the block takes x unrounded (bf16
// with ReLU, whose derivative jumps).
int check_normed(const shampoo_ffn_t* a, const shampoo_norm_t* norm, shl::NormArgs& k, bool& used) {
  RC(check_ffn(a, false));
  if (!norm) return fail(SHAMPOO_ERR_INVALID_ARG, "norm is NULL");
  if (norm->z) return fail(SHAMPOO_ERR_INVALID_ARG, "norm has a z: only a norm alone can be made again");
  RC(check_norm(norm, false));
  if (norm->rows != a->tokens || norm->width != a->d_model || norm->dtype != a->dtype)
    return fail(SHAMPOO_ERR_INVALID_ARG, "norm has another size or dtype than x");
  if (!norm->stats && norm->rows) return fail(SHAMPOO_ERR_INVALID_ARG, "norm's stats are NULL: the norm has to keep them");
  RC(norm_args(norm, false, k));
  // n is x itself, wherever the norm's call left it
  k.n = const_cast<void*>(a->x), k.ldn = a->ld_x;
  used = a->dtype == SHAMPOO_BF16 && a->activation == SHAMPOO_ACT_RELU;
  return SHAMPOO_OK;
}

}  // namespace

extern "C" {

int shampoo_ffn_saved_size(const shampoo_ffn_t* a, size_t* bytes_out) {
  RC(check_sizes(a));
  if (!bytes_out) return fail(SHAMPOO_ERR_INVALID_ARG, "bytes_out is NULL");
  const Ffn p(*a, nullptr, nullptr, nullptr, false);
  *bytes_out = static_cast<size_t>(p.saved_bytes());
  return SHAMPOO_OK;
}

int shampoo_ffn_workspace_size(const shampoo_ffn_t* a, int32_t backward, size_t* bytes_out) {
  return guarded([&]() -> int {
    RC(check_ffn(a, backward != 0));
    if (!bytes_out) return fail(SHAMPOO_ERR_INVALID_ARG, "bytes_out is NULL");
    *bytes_out = static_cast<size_t>(ffn_workspace(a, nullptr, backward != 0));
    return SHAMPOO_OK;
  });
}

int shampoo_ffn_forward(const shampoo_ffn_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_ffn(a, false));
    return run_ffn(a, nullptr, workspace, workspace_bytes, hip_stream, false);
  });
}

int shampoo_ffn_backward(const shampoo_ffn_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_ffn(a, true));
    return run_ffn(a, nullptr, workspace, workspace_bytes, hip_stream, true);
  });
}

int shampoo_ffn_normed_workspace_size(const shampoo_ffn_t* a, const shampoo_norm_t* norm, size_t* bytes_out) {
  return guarded([&]() -> int {
    shl::NormArgs k;
    bool used;
    RC(check_normed(a, norm, k, used));
    if (!bytes_out) return fail(SHAMPOO_ERR_INVALID_ARG, "bytes_out is NULL");
    *bytes_out = static_cast<size_t>(ffn_workspace(a, used ? &k : nullptr, false));
    return SHAMPOO_OK;
  });
}

int shampoo_ffn_forward_normed(const shampoo_ffn_t* a, const shampoo_norm_t* norm, void* workspace, size_t workspace_bytes,
                               void* hip_stream) {
  return guarded([&]() -> int {
    shl::NormArgs k;
    bool used;
    RC(check_normed(a, norm, k, used));
    return run_ffn(a, used ? &k : nullptr, workspace, workspace_bytes, hip_stream, false);
  });
}

int shampoo_norm_workspace_size(const shampoo_norm_t* a, size_t* bytes_out) {
  return guarded([&]() -> int {
    RC(check_norm(a, true));
    if (!bytes_out) return fail(SHAMPOO_ERR_INVALID_ARG, "bytes_out is NULL");
    shl::NormArgs k;
    RC(norm_args(a, true, k));
    *bytes_out = static_cast<size_t>(4 * shl::norm_partial_floats(k));
    return SHAMPOO_OK;
  });
}

int shampoo_norm_forward(const shampoo_norm_t* a, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_norm(a, false));
    shl::NormArgs k;
    RC(norm_args(a, false, k));
    const hipError_t e = shl::launch_norm_forward(k, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_norm_forward");
  });
}

int shampoo_norm_backward(const shampoo_norm_t* a, void* workspace, size_t workspace_bytes, void* hip_stream) {
  return guarded([&]() -> int {
    RC(check_norm(a, true));
    shl::NormArgs k;
    RC(norm_args(a, true, k));
    const int64_t need = 4 * shl::norm_partial_floats(k);
    if (need > 0 && !workspace) return fail(SHAMPOO_ERR_INVALID_ARG, "workspace is NULL");
    if (!aligned(workspace, 256)) return fail(SHAMPOO_ERR_MISALIGNED, "workspace is not aligned to 256 bytes");
    if (workspace_bytes < static_cast<size_t>(need))
      return fail(SHAMPOO_ERR_WORKSPACE_TOO_SMALL,
                  "workspace has " + std::to_string(workspace_bytes) + " bytes, the call needs " + std::to_string(need));
    k.partial = static_cast<float*>(workspace);
    const hipError_t e = shl::launch_norm_backward(k, static_cast<hipStream_t>(hip_stream));
    return e == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(e, "shampoo_norm_backward");
  });
}

int shampoo_dropout(const shampoo_dropout_t* a, void* hip_stream) {
  return guarded([&]() -> int {
    if (!a) return fail(SHAMPOO_ERR_INVALID_ARG, "arguments are NULL");
    if (a->rows < 0 || a->cols < 0 || a->cols > kMaxDim || a->rows > (int64_t(1) << 40))
      return fail(SHAMPOO_ERR_INVALID_ARG, "rows must be in [0, 2^40], cols in [0, 2^31 - 1024]");
    RC(check_dtype(a->dtype));
    const int64_t e = a->dtype == SHAMPOO_F32 ? 4 : 2;
    RC(check_matrix("x", a->x, a->rows, a->cols, a->ld_x, e, kAnyLd));
    RC(check_matrix("y", a->y, a->rows, a->cols, a->ld_y, e, kAnyLd));
    shl::DropoutArgs k{a->x, a->y, a->rows, a->cols, a->ld_x, a->ld_y, a->dtype == SHAMPOO_F32 ? 1 : 0, {}};
    RC(make_drop(a->dropout, a->seed, a->offset, k.drop));
    const hipError_t err = shl::launch_dropout(k, static_cast<hipStream_t>(hip_stream));
    return err == hipSuccess ? SHAMPOO_OK : shp_rt::hip_fail(err, "shampoo_dropout");
  });
}

}  // extern "C"
