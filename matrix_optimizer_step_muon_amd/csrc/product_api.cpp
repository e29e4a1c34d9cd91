// C ABI of the layers' products (include/muon.h): the gated feed-forward block and
// the 8-bit linear product. Validation, the workspace's layout, which tiles a
// product is cut into, and the launches. Nothing is kept between calls.

#include "layer_checks.h"
#include "product_internal.h"

namespace {

using namespace muon::abi;

constexpr int64_t kMaxWidth = int64_t(1) << 22;
constexpr int64_t kMaxUnits = int64_t(1) << 22;
// Row strides, in bytes, up to which 256 rows are within 32-bit offsets; and those of
// what the products' tiles write and add, in elements of up to 4 bytes.
constexpr int64_t kMaxPitch = int64_t(1) << 24, kMaxStride = int64_t(1) << 22;

muon_status check_stride(int64_t ld, const char* name, int item = -1) {
  if (ld > kMaxStride) return fail(MUON_ERR_INVALID_ARG, Views::at(item) + name + ": row stride must be in [cols, 2^22]");
  return MUON_OK;
}

constexpr int64_t kCus = 256;
constexpr double kHbm = 5.2e6;  // bytes per us: what streaming the weights of few rows reaches

// What few_kernels.hip is expected to take for weights of n rows (of each of `ops`)
// of `row` bytes: every CU streams its share of them at 23.5 KB a us, and reads the
// activations once for every share. One MI355X, bf16, 1 and 16 rows: both projections
// of 25600 x 5120 89 and 104 us (estimated 89 and 102; in tiles 109 and 113), of 6144 x
// 2048 10.8 and 11.3 (10.4 and 11.7); one of 5120 x 25600 48 and 60 to 65 (46 and 62; in
// tiles 56 and 57), of 2048 x 6144 7.1 and 11.0 (6.2 and 10.1; in tiles 13.6). Those of 6144
// x 2048 were in the last-level cache both ways; from HBM they take 12.4 and 8.4 (1 row).
double few_us(int64_t n, double row, int ops, int64_t rows) {
  const muon::FewShare f = muon::few_share(n, muon::kFewMost);
  const double weights = double(f.per * ops);
  return 2.0 + double(f.rounds) * weights * row / 23.5e3 * (1.0 + 0.5 * double(rows - 1) / weights);
}

// How a launch is cut up: the tiles, how many of them are one unit each, how many
// pieces the sums of the others are cut into, and what it is expected to take.
struct Choice {
  int tile;
  int64_t whole;
  int splits;
  double us;
};

// What a kind of product costs beside its stages: us that a CU takes to let the sums
// of a tile out (times a factor of the tile's, below), and a stage against one of
// bf16 operands that are both read along K.
struct Cost {
  double leave, stage;
  int first = muon::kPrLarge;  // the largest tile that it has
};
constexpr Cost kGateCost{9.9, 1.0}, kGateGradCost{14.0, 0.99}, kDownCost{3.4, 1.0}, kDxCost{3.4, 0.99}, kLinear8Cost{19.2, 0.96},
    kLinear8F32Cost{19.2, 1.8, muon::kPrMedium};

// For products with t[i] tiles of kind i in all, and `stages` stages of 128 bytes of
// K each, that read `bytes` once. Either all tiles are whole, or all in pieces, or the
// last round, which would leave CUs without work, is in as many pieces as there is
// room for. The constants are fitted to a sweep on one MI355X: 12 sizes from 20 x 2048
// x 6144 to 4096 x 2048 x 6144, six kinds of product, each tile in 1 to 24 pieces, 1014
// times in all. The pick is 1.6% behind the best on average, over 10% in two of 72 (14%,
// where tiles in pieces take more than estimated). At one size each, us of the best cut
// of large, medium and small tiles: 4096 x 6144 x 2048 with both projections 199, 246,
// 408; 2000 x 3200 x 1600 42, 29, 41; 64 x 2048 x 6144 29, 20, 13.
Choice choose(const int64_t t[muon::kPrTiles], int64_t stages, const Cost& cost, double bytes) {
  // Per kind: workgroups per CU; us to fill a tile and to let it out; us per stage
  // with one and with all of a CU's; us per partial tile, written and read.
  static const struct { int per_cu; double fill, leave, one, all, part; } kCost[muon::kPrTiles] = {
      {1, 4.2, 0.3, 1.27, 1.27, 0.077}, {2, 3.2, 0.064, 0.79, 1.05, 0.017}, {2, 0.87, 0.22, 0.27, 0.43, 0.003}};
  Choice best{cost.first, t[cost.first], 1, 1e300};
  for (int i = cost.first; i < muon::kPrTiles; ++i) {
    const auto& c = kCost[i];
    const int64_t round = kCus * c.per_cu;
    const double fixed = c.fill + cost.leave * c.leave;
    auto run = [&](int64_t units, int64_t n) {
      const int64_t full = units / round, rest = units % round;
      const double steps = cost.stage * double(n);
      return double(full) * (fixed + c.all * steps) + (rest ? fixed + (rest <= kCus ? c.one : c.all) * steps : 0.0);
    };
    auto take = [&](int64_t whole, int64_t s) {
      const int64_t pieces = (t[i] - whole) * s;
      if (whole + pieces > kMaxUnits) return;
      double us = 2.0 + run(whole, stages);
      if (pieces) us += run(pieces, ceil_div(stages, s)) + 2.9 + 0.1 * double(s) + c.part * double(pieces);
      const double stream = 4.0 + bytes / kHbm;  // what is the least also counts a little
      us = std::max(us, stream) + 0.15 * std::min(us, stream);
      if (us < best.us) best = {i, whole, int(s), us};
    };
    take(t[i], 1);
    for (const int64_t s : {2, 3, 4, 5, 6, 8, 10, 12, 16, 20, 24, 32, 48, 64}) {
      if (s > stages / 4) break;
      if (t[i] * s <= 4 * round) take(0, s);
      if (t[i] > round && t[i] % round && t[i] % round * s <= 2 * round) take(t[i] / round * round, s);
    }
  }
  return best;
}

// A launch's items laid out: tiles, pieces, and the bytes of partial tiles.
muon_status lay_out(muon::PrArgs& a, bool dual, int elem, const Cost& cost, size_t* bytes, double* us = nullptr) {
  int64_t t[muon::kPrTiles] = {}, stages = 0;
  double moved = 0.0;
  const int pairs = a.parts == 3 ? 6 : 1, bk = 128 / elem;
  for (int i = 0; i < a.n_items; ++i) {
    const muon::PrItem& it = a.item[i];
    moved += double(it.k) * double(it.n + it.m) * elem * it.sums * a.parts * (dual ? 2 : 1);
    for (int j = 0; j < muon::kPrTiles; ++j)
      t[j] += ceil_div(it.m, muon::kPrEdge[j]) * ceil_div(it.n, dual ? muon::kPrEdge[j] / 2 : muon::kPrEdge[j]);
    stages = std::max(stages, ceil_div(it.k, bk) * it.sums * pairs);
  }
  const Choice c = choose(t, stages, cost, moved);
  if (us) *us = c.us;
  a.tile = c.tile;
  const int edge = muon::kPrEdge[c.tile];
  std::fill(a.whole0, a.whole0 + muon::kPrItems, INT32_MAX);
  std::fill(a.piece0, a.piece0 + muon::kPrItems, INT32_MAX);
  int64_t wholes = 0, pieces = 0;
  for (int i = 0; i < a.n_items; ++i) {
    muon::PrItem& it = a.item[i];
    const int64_t mine = ceil_div(it.k, bk) * it.sums * pairs;
    const int64_t tm = ceil_div(it.m, edge), tn = ceil_div(it.n, dual ? edge / 2 : edge);
    if (tm * tn > kMaxUnits) return fail(MUON_ERR_INVALID_ARG, "more than 2^22 tiles in one launch");
    it.tiles_m = int32_t(tm);
    it.tiles_n = int32_t(tn);
    it.splits = int32_t(std::max<int64_t>(1, std::min<int64_t>(c.splits, mine / 2)));
    const int64_t whole = it.splits == 1 ? tm * tn : std::min(tm * tn, std::max<int64_t>(0, c.whole - wholes));
    it.whole = int32_t(whole);
    it.stages = int32_t(mine);
    it.per = int32_t(mine / it.splits);
    a.whole0[i] = int32_t(wholes);
    a.piece0[i] = it.part0 = int32_t(pieces);
    wholes += whole;
    pieces += (tm * tn - whole) * it.splits;
    if (wholes + pieces > kMaxUnits) return fail(MUON_ERR_INVALID_ARG, "more than 2^22 tiles in one launch");
  }
  a.wholes = int32_t(wholes);
  a.pieces = int32_t(pieces);
  *bytes = round256(size_t(pieces) * edge * edge * sizeof(float));
  return MUON_OK;
}

// ------------------------------------------------------------ the gated block

muon_status check_mlp(const muon_mlp& p) {
  MUON_TRY(check_dtype(p.dtype));
  if (p.rows < 0 || p.rows > kMaxRows) return fail(MUON_ERR_INVALID_ARG, "rows must be in [0, 2^30]");
  const struct { int64_t v; const char* name; } sizes[] = {{p.width, "width"}, {p.inner, "inner"}, {p.out, "out"}};
  for (const auto& s : sizes)
    if (s.v < 1 || s.v > kMaxWidth) return fail(MUON_ERR_INVALID_ARG, std::string(s.name) + " must be in [1, 2^22]");
  return MUON_OK;
}

muon_status check_mlp_weights(Views& v, const muon_mlp& p) {
  if (p.act < MUON_ACT_SILU || p.act > MUON_ACT_RELU) return fail(MUON_ERR_UNSUPPORTED, "act must be a muon_act");
  const int e = elem_of(p.dtype);
  MUON_TRY(v.add(p.w_gate, p.inner, p.width, p.width, e, false, "w_gate"));
  MUON_TRY(v.add(p.w_up, p.inner, p.width, p.width, e, false, "w_up"));
  return v.add(p.w_down, p.out, p.inner, p.inner, e, false, "w_down");
}

muon_status check_inner(Views& v, const muon_mlp& p, const muon_q8& q, bool written, const char* name) {
  if (q.rows != p.rows || q.cols != p.inner)
    return fail(MUON_ERR_INVALID_ARG, std::string(name) + " must be a rows x inner checkpoint");
  return check_q8(v, q, written, name);
}

muon_status check_kinds(const muon_mlp& p) {
  const muon_q8* q[] = {&p.a, &p.b, &p.s};
  int kind = -1;
  for (const muon_q8* x : q) {
    if (!x->q) continue;
    if (kind >= 0 && x->kind != kind) return fail(MUON_ERR_INVALID_ARG, "a, b and s must be checkpoints of the same kind");
    kind = x->kind;
  }
  return MUON_OK;
}

// An operand of a product: as the caller gave it, if it is bf16 in 16-byte aligned
// rows of whole 16-byte chunks, else rewritten into the workspace first. A null one
// counts as one to rewrite (where only the workspace's size is asked for).
struct Operand {
  const void* p;
  int64_t rows, cols, ld;
  bool pack;
  size_t at;
};

int64_t pad8(int64_t v) { return (v + 7) / 8 * 8; }
size_t planes_bytes(int64_t rows, int64_t cols, int parts) {
  return round256(size_t(parts) * size_t(rows) * size_t(pad8(cols)) * 2);
}

struct Bump {
  size_t at = 0;
  size_t take(size_t bytes) {
    const size_t here = at;
    at += round256(bytes);
    return here;
  }
};

bool in_place(const void* p, int64_t cols, int64_t ld, int32_t dtype) {
  return dtype == MUON_BF16 && p && reinterpret_cast<uintptr_t>(p) % 16 == 0 && cols % 8 == 0 && ld % 8 == 0 && 2 * ld <= kMaxPitch;
}

Operand operand(Bump& b, bool used, const void* p, int64_t rows, int64_t cols, int64_t ld, int32_t dtype) {
  Operand o{p, rows, cols, ld, used && !in_place(p, cols, ld, dtype), 0};
  if (o.pack) o.at = b.take(planes_bytes(rows, cols, dtype == MUON_F32 ? 3 : 1));
  return o;
}

// One call's products and its workspace.
struct MlpCall {
  Operand ops[4];
  muon::PrArgs first{}, second{};
  bool few_first = false, few_second = false;  // forward: by the kernels for few rows
  char* s = nullptr;                           // forward: s between the two products
  int64_t ld_s = 0, plane_s = 0;               // plane_s: in two planes, so far apart
  size_t bytes = 0;
};

// Two operands of one item share a row stride and a distance of planes: where one
// of two weights of the same shape is rewritten and the other is not, both are bf16
// rows of the same multiple of 8.
void put_operand(muon::PrItem& it, bool is_a, int which, const Operand& o, char* ws, int parts) {
  const uint8_t* p = o.pack ? reinterpret_cast<const uint8_t*>(ws + o.at) : static_cast<const uint8_t*>(o.p);
  const int64_t ld = o.pack ? pad8(o.cols) : o.ld, plane = parts == 3 ? o.rows * ld * 2 : 0;
  (is_a ? it.a : it.b)[which] = p;
  (is_a ? it.lda : it.ldb) = ld * 2;
  (is_a ? it.pa : it.pb) = plane;
}

void start(muon::PrArgs& a, const muon_mlp& p, int64_t m, int64_t n, int64_t k, int sums) {
  a.n_items = 1;
  a.parts = p.dtype == MUON_F32 ? 3 : 1;
  a.f32 = p.dtype == MUON_F32;
  a.item[0].m = int32_t(m);
  a.item[0].n = int32_t(n);
  a.item[0].k = int32_t(k);
  a.item[0].sums = sums;
  a.mlp.act = p.act;
}

// Few rows: a product that reads its weights as they are, once, where that is
// expected to be faster; fp32 always, since tiles would have the weights rewritten
// first. The gate does so only if nothing is kept.
bool few_gate(const muon_mlp& p, double tiles_us) {
  return p.rows <= muon::kFewRows && p.y && !p.a.q && !p.b.q && !p.s.q &&
         (p.dtype == MUON_F32 || few_us(p.inner, double(p.width) * 2, 2, p.rows) <= tiles_us);
}
bool few_down(const muon_mlp& p, double tiles_us) {
  return p.rows <= muon::kFewRows && p.dtype == MUON_BF16 && few_us(p.out, double(p.inner) * 2, 1, p.rows) <= tiles_us;
}

muon_status plan_forward(const muon_mlp& p, MlpCall& c, char* ws) {
  Bump b;
  const int parts = p.dtype == MUON_F32 ? 3 : 1;
  size_t n1 = 0, n2 = 0;
  double us1 = 0.0, us2 = 0.0;
  start(c.first, p, p.rows, p.inner, p.width, 1);
  start(c.second, p, p.rows, p.out, p.inner, 1);
  // fp32 goes through both kernels for few rows or none, and s between them stays fp32
  const bool plain = p.dtype == MUON_F32 && few_gate(p, 0.0);
  c.few_first = c.few_second = plain;
  if (!plain) {
    MUON_TRY(lay_out(c.first, true, 2, kGateCost, &n1, &us1));
    MUON_TRY(lay_out(c.second, false, 2, kDownCost, &n2, &us2));
    c.few_first = few_gate(p, us1);
    c.few_second = few_down(p, us2);
  }
  const bool first = !c.few_first, second = p.y && !c.few_second;  // in tiles
  c.ops[0] = operand(b, first, p.x, p.rows, p.width, p.ld_x, p.dtype);
  c.ops[1] = operand(b, first, p.w_gate, p.inner, p.width, p.width, p.dtype);
  c.ops[2] = operand(b, first, p.w_up, p.inner, p.width, p.width, p.dtype);
  c.ops[3] = operand(b, second, p.w_down, p.out, p.inner, p.inner, p.dtype);
  // and between those kernels bf16 is two planes, for so few rows that it costs 1 or 2%
  const bool two = !plain && p.y && c.few_first && c.few_second && p.rows <= muon::kFewHalves;
  c.ld_s = plain ? p.inner : pad8(p.inner);
  c.plane_s = two ? p.rows * c.ld_s : 0;
  const Operand s{nullptr, p.rows, p.inner, c.ld_s, true,
                  b.take(plain ? size_t(p.rows) * size_t(p.inner) * 4 : planes_bytes(p.rows, p.inner, two ? 2 : parts))};
  c.s = ws + s.at;
  muon::PrItem& f = c.first.item[0];
  put_operand(f, true, 0, c.ops[0], ws, parts);
  put_operand(f, false, 0, c.ops[1], ws, parts);
  put_operand(f, false, 1, c.ops[2], ws, parts);
  muon::PrMlp& e = c.first.mlp;
  e.a = p.a;
  e.b = p.b;
  e.s = p.s;
  e.plane[0] = reinterpret_cast<uint16_t*>(c.s);
  e.ldp = c.ld_s;
  e.pp = p.rows * e.ldp;
  muon::PrItem& g = c.second.item[0];
  put_operand(g, true, 0, s, ws, parts);
  put_operand(g, false, 0, c.ops[3], ws, parts);
  g.out = p.y;
  g.ldo = p.ld_y;
  c.first.partial = c.second.partial = reinterpret_cast<float*>(ws + b.at);
  c.bytes = b.at + std::max(first ? n1 : 0, second ? n2 : 0);
  return MUON_OK;
}

muon_status plan_backward(const muon_mlp& p, const muon_mlp_grads& g, MlpCall& c, char* ws) {
  Bump b;
  const int parts = p.dtype == MUON_F32 ? 3 : 1;
  const bool second = g.d_x != nullptr;
  c.ops[0] = operand(b, true, g.dy, p.rows, p.out, g.ld_dy, p.dtype);
  c.ops[1] = operand(b, true, p.w_down, p.out, p.inner, p.inner, p.dtype);
  c.ops[2] = operand(b, second, p.w_gate, p.inner, p.width, p.width, p.dtype);
  c.ops[3] = operand(b, second, p.w_up, p.inner, p.width, p.width, p.dtype);
  // da and db feed the next product as they are, or from the workspace, both alike
  void* d[2] = {g.d_a, g.d_b};
  const int64_t ld[2] = {g.ld_d_a, g.ld_d_b};
  const bool same = in_place(d[0], p.inner, ld[0], p.dtype) && in_place(d[1], p.inner, ld[1], p.dtype) && ld[0] == ld[1];
  start(c.first, p, p.rows, p.inner, p.out, 1);
  muon::PrItem& f = c.first.item[0];
  put_operand(f, true, 0, c.ops[0], ws, parts);
  put_operand(f, false, 0, c.ops[1], ws, parts);
  muon::PrMlp& e = c.first.mlp;
  e.a = p.a;
  e.b = p.b;
  e.ldp = pad8(p.inner);
  e.pp = p.rows * e.ldp;
  start(c.second, p, p.rows, p.width, p.inner, 2);
  muon::PrItem& s = c.second.item[0];
  for (int i = 0; i < 2; ++i) {
    e.d[i] = d[i];
    e.ldd[i] = ld[i];
    Operand o{d[i], p.rows, p.inner, ld[i], second && !same, 0};
    if (o.pack) {
      o.at = b.take(planes_bytes(p.rows, p.inner, parts));
      e.plane[i] = reinterpret_cast<uint16_t*>(ws + o.at);
    }
    put_operand(s, true, i, o, ws, parts);
    put_operand(s, false, i, c.ops[2 + i], ws, parts);
  }
  s.out = g.d_x;
  s.ldo = g.ld_d_x;
  size_t n1 = 0, n2 = 0;
  MUON_TRY(lay_out(c.first, false, 2, kGateGradCost, &n1));
  MUON_TRY(lay_out(c.second, false, 2, kDxCost, &n2));
  c.first.partial = c.second.partial = reinterpret_cast<float*>(ws + b.at);
  c.bytes = b.at + std::max(n1, second ? n2 : 0);
  return MUON_OK;
}

muon_status launch_few_gate(const muon_mlp& p, const MlpCall& c, hipStream_t stream) {
  muon::FewArgs a{};
  a.a = p.x;
  a.lda = p.ld_x;
  a.b[0] = p.w_gate;
  a.b[1] = p.w_up;
  a.ldb = p.width;
  a.m = int32_t(p.rows);
  a.n = int32_t(p.inner);
  a.k = int32_t(p.width);
  a.act = p.act;
  a.out = c.s;
  a.ldo = c.ld_s;
  a.plane = c.plane_s;
  return hip_status(muon::launch_few(a, p.dtype == MUON_F32, 2, stream));
}

muon_status launch_few_down(const muon_mlp& p, const MlpCall& c, hipStream_t stream) {
  muon::FewArgs a{};
  a.a = c.s;
  a.lda = c.ld_s;
  a.plane = c.plane_s;
  a.b[0] = p.w_down;
  a.ldb = p.inner;
  a.m = int32_t(p.rows);
  a.n = int32_t(p.out);
  a.k = int32_t(p.inner);
  a.out = p.y;
  a.ldo = p.ld_y;
  return hip_status(muon::launch_few(a, p.dtype == MUON_F32, 1, stream));
}

// For the tensors of a pass.
muon_status mlp_workspace(const muon_mlp& p, const muon_mlp_grads* g, size_t* bytes) {
  MUON_TRY(check_mlp(p));
  *bytes = 0;
  if (p.rows == 0) return MUON_OK;
  MlpCall c;
  MUON_TRY(g ? plan_backward(p, *g, c, nullptr) : plan_forward(p, c, nullptr));
  *bytes = c.bytes;
  return MUON_OK;
}

// How an item of a launch is cut up.
void cut_of(const muon::PrArgs& a, const muon::PrItem& it, int32_t* tile, int32_t* whole, int32_t* pieces) {
  *tile = muon::kPrEdge[a.tile];
  *whole = it.whole;
  *pieces = it.whole == it.tiles_m * it.tiles_n ? 1 : it.splits;
}

muon_status mlp_info(const muon_mlp& p, const muon_mlp_grads* g, int32_t* tile, int32_t* whole, int32_t* pieces) {
  MUON_TRY(check_mlp(p));
  for (int i = 0; i < 2; ++i) {
    tile[i] = whole[i] = 0;
    pieces[i] = 1;
  }
  if (p.rows == 0) return MUON_OK;
  MlpCall c;
  MUON_TRY(g ? plan_backward(p, *g, c, nullptr) : plan_forward(p, c, nullptr));
  if (!c.few_first) cut_of(c.first, c.first.item[0], tile, whole, pieces);
  if ((g ? g->d_x : p.y) && !c.few_second) cut_of(c.second, c.second.item[0], tile + 1, whole + 1, pieces + 1);
  return MUON_OK;
}

// The most that either pass takes: everything is wanted, and every operand rewritten.
muon_status mlp_workspace(const muon_mlp& p, size_t* bytes) {
  muon_mlp q = p;
  q.x = q.w_gate = q.w_up = q.w_down = nullptr;
  q.y = q.a.q = &q;
  muon_mlp_grads g{};
  g.d_x = &g;
  size_t forward = 0, backward = 0;
  MUON_TRY(mlp_workspace(q, nullptr, &forward));
  MUON_TRY(mlp_workspace(q, &g, &backward));
  *bytes = std::max(forward, backward);
  return MUON_OK;
}

muon_status check_mlp_workspace(Views& v, const muon_mlp& p, size_t need) {
  if (!need) return MUON_OK;
  if (p.workspace_bytes < need)
    return fail(MUON_ERR_INVALID_ARG, "the workspace has " + std::to_string(p.workspace_bytes) + " bytes, " +
                                          std::to_string(need) + " are needed");
  if (!p.workspace) return fail(MUON_ERR_INVALID_ARG, "workspace is NULL");
  if (reinterpret_cast<uintptr_t>(p.workspace) % 16) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
  return v.add_range(p.workspace, need, "workspace");
}

// The operands that are not in place, rewritten in one launch.
muon_status run_packs(const MlpCall& c, const muon_mlp& p, char* ws, hipStream_t s) {
  muon::PrPacks a{};
  for (const Operand& o : c.ops) {
    if (!o.pack) continue;
    muon::PrPack& d = a.pack[a.n++];
    d.src = o.p;
    d.dst = ws + o.at;
    d.ld = o.ld;
    d.octets = pad8(o.cols) / 8;
    d.rows = int32_t(o.rows);
    d.cols = int32_t(o.cols);
  }
  return hip_status(muon::launch_packs(a, p.dtype == MUON_F32, s));
}

muon_status mlp_forward(const muon_mlp* mlp, void* stream) {
  if (!mlp) return fail(MUON_ERR_INVALID_ARG, "mlp is NULL");
  const muon_mlp& p = *mlp;
  MUON_TRY(check_mlp(p));
  Views v;
  MUON_TRY(check_mlp_weights(v, p));
  const int e = elem_of(p.dtype);
  MUON_TRY(v.add(p.x, p.rows, p.width, p.ld_x, e, false, "x"));
  if (!p.y && !p.a.q && !p.b.q && !p.s.q && p.rows > 0) return fail(MUON_ERR_INVALID_ARG, "y, a, b and s are all NULL");
  if (p.y) {
    MUON_TRY(check_stride(p.ld_y, "y"));
    MUON_TRY(v.add(p.y, p.rows, p.out, p.ld_y, e, true, "y"));
  }
  if (p.a.q) MUON_TRY(check_inner(v, p, p.a, true, "a"));
  if (p.b.q) MUON_TRY(check_inner(v, p, p.b, true, "b"));
  if (p.s.q) MUON_TRY(check_inner(v, p, p.s, true, "s"));
  MUON_TRY(check_kinds(p));
  if (p.rows == 0) return v.disjoint();
  char* ws = static_cast<char*>(p.workspace);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  MlpCall c;
  MUON_TRY(plan_forward(p, c, ws));
  MUON_TRY(check_mlp_workspace(v, p, c.bytes));
  MUON_TRY(v.disjoint());
  MUON_TRY(run_packs(c, p, ws, s));
  if (c.few_first) MUON_TRY(launch_few_gate(p, c, s));
  else MUON_TRY(hip_status(muon::launch_mlp(c.first, muon::kPrGate, false, s)));
  if (!p.y) return MUON_OK;
  if (c.few_second) return launch_few_down(p, c, s);
  return hip_status(muon::launch_mlp(c.second, muon::kPrStore, false, s));
}

muon_status mlp_backward(const muon_mlp* mlp, const muon_mlp_grads* grads, void* stream) {
  if (!mlp || !grads) return fail(MUON_ERR_INVALID_ARG, "mlp or grads is NULL");
  const muon_mlp& p = *mlp;
  const muon_mlp_grads& g = *grads;
  MUON_TRY(check_mlp(p));
  Views v;
  MUON_TRY(check_mlp_weights(v, p));
  const int e = elem_of(p.dtype);
  MUON_TRY(v.add(g.dy, p.rows, p.out, g.ld_dy, e, false, "dy"));
  MUON_TRY(check_inner(v, p, p.a, false, "a"));
  MUON_TRY(check_inner(v, p, p.b, false, "b"));
  if (p.a.kind != p.b.kind) return fail(MUON_ERR_INVALID_ARG, "a and b must be checkpoints of the same kind");
  MUON_TRY(check_stride(g.ld_d_a, "d_a"));
  MUON_TRY(v.add(g.d_a, p.rows, p.inner, g.ld_d_a, e, true, "d_a"));
  MUON_TRY(check_stride(g.ld_d_b, "d_b"));
  MUON_TRY(v.add(g.d_b, p.rows, p.inner, g.ld_d_b, e, true, "d_b"));
  if (g.d_x) {
    MUON_TRY(check_stride(g.ld_d_x, "d_x"));
    MUON_TRY(v.add(g.d_x, p.rows, p.width, g.ld_d_x, e, true, "d_x"));
  }
  if (p.rows == 0) return v.disjoint();
  char* ws = static_cast<char*>(p.workspace);
  MlpCall c;
  MUON_TRY(plan_backward(p, g, c, ws));
  MUON_TRY(check_mlp_workspace(v, p, c.bytes));
  MUON_TRY(v.disjoint());
  const hipStream_t s = static_cast<hipStream_t>(stream);
  MUON_TRY(run_packs(c, p, ws, s));
  MUON_TRY(hip_status(muon::launch_mlp(c.first, muon::kPrGateGrad, true, s)));
  return g.d_x ? hip_status(muon::launch_mlp(c.second, muon::kPrStore, true, s)) : MUON_OK;
}

// ------------------------------------------------------------ the 8-bit product

muon_status check_w8(Views& v, const muon_w8& w, bool q, bool qt, bool written, const char* name, int item = -1) {
  auto bad = [&](muon_status st, const char* what) { return fail(st, Views::at(item) + name + what); };
  if (w.n < 1 || w.n > kMaxCols || w.k < 1 || w.k > kMaxCols) return bad(MUON_ERR_INVALID_ARG, ": n and k must be in [1, 2^24]");
  if (ceil_div(w.n, muon::kBlock) * ceil_div(w.k, muon::kBlock) > (int64_t(1) << 30))
    return bad(MUON_ERR_INVALID_ARG, ": more than 2^30 blocks");
  if (q) {
    if (w.ldq % 16) return bad(MUON_ERR_ALIGN, ": ldq must be a multiple of 16");
    MUON_TRY(v.add(w.q, w.n, (w.k + 15) / 16 * 16, w.ldq, 1, written, name, item, 16));
  }
  if (qt) {
    if (!w.qt) return bad(MUON_ERR_INVALID_ARG, ".qt is NULL");
    if (w.ldqt % 16) return bad(MUON_ERR_ALIGN, ": ldqt must be a multiple of 16");
    MUON_TRY(v.add(w.qt, w.k, (w.n + 15) / 16 * 16, w.ldqt, 1, written, name, item, 16));
  }
  return v.add(w.e, ceil_div(w.n, muon::kBlock), ceil_div(w.k, muon::kBlock), w.lde, 1, written, name, item);
}

muon_status w8_call(const void* w, int64_t ldw, int32_t dtype, const muon_w8* p, bool save, void* stream) {
  return guarded([&]() -> muon_status {
    if (!p) return fail(MUON_ERR_INVALID_ARG, "the 8-bit weight is NULL");
    MUON_TRY(check_dtype(dtype));
    Views v;
    MUON_TRY(check_w8(v, *p, true, save && p->qt, save, "weight"));
    MUON_TRY(v.add(w, p->n, p->k, ldw, elem_of(dtype), !save, "w"));
    MUON_TRY(v.disjoint());
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return hip_status(save ? muon::launch_w8_save(w, ldw, dtype, *p, s)
                           : muon::launch_w8_load(*p, const_cast<void*>(w), ldw, dtype, s));
  });
}

muon_status check_linear8(const muon_linear8_item* items, int32_t n, int32_t dtype, Views& v) {
  if (!items) return fail(MUON_ERR_INVALID_ARG, "items is NULL");
  if (n < 1) return fail(MUON_ERR_INVALID_ARG, "n_items must be >= 1");
  MUON_TRY(check_dtype(dtype));
  const int e = elem_of(dtype);
  for (int32_t i = 0; i < n; ++i) {
    const muon_linear8_item& it = items[i];
    const bool t = it.transposed != 0;
    MUON_TRY(check_q8(v, it.x, false, "x", i));
    if (it.x.kind != MUON_Q8_E4M3) return fail(MUON_ERR_UNSUPPORTED, Views::at(i) + "x must be an e4m3 checkpoint");
    MUON_TRY(check_w8(v, it.w, !t, t, false, "w", i));
    const int64_t k = t ? it.w.n : it.w.k, out = t ? it.w.k : it.w.n;
    if (it.x.cols != k)
      return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "x has " + std::to_string(it.x.cols) + " columns, the weight " + std::to_string(k));
    if (it.w.n > kMaxWidth || it.w.k > kMaxWidth) return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "n and k must be in [1, 2^22]");
    MUON_TRY(check_stride(it.ld_y, "y", i));
    MUON_TRY(v.add(it.y, it.x.rows, out, it.ld_y, e, true, "y", i));
    if (!std::isfinite(it.beta)) return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "beta is not finite");
    if (it.beta != 0.f && it.c == it.y && it.ld_c != it.ld_y)
      return fail(MUON_ERR_INVALID_ARG, Views::at(i) + "c is y, with another row stride");
    if (it.beta != 0.f && it.c != it.y) {
      MUON_TRY(check_stride(it.ld_c, "c", i));
      MUON_TRY(v.add(it.c, it.x.rows, out, it.ld_c, e, false, "c", i));
    }
  }
  return v.disjoint();
}

// Few rows with a bf16 result: a launch of their own, without a workspace. Items
// without rows have nothing to do.
bool few_rows(const muon_linear8_item& it, int32_t dtype) { return it.x.rows <= muon::kFewRows && dtype == MUON_BF16; }
bool in_tiles(const muon_linear8_item& it, int32_t dtype) { return it.x.rows > 0 && !few_rows(it, dtype); }

muon_status few_linear8(const muon_linear8_item& it, hipStream_t s) {
  const bool t = it.transposed != 0;
  muon::FewArgs a{};
  a.a = it.x.q;
  a.lda = it.x.ldq;
  a.ea = static_cast<const uint8_t*>(it.x.e);
  a.lde = it.x.lde;
  a.b[0] = t ? it.w.qt : it.w.q;
  a.ldb = t ? it.w.ldqt : it.w.ldq;
  a.eb = static_cast<const uint8_t*>(it.w.e);
  a.ldeb_n = t ? 1 : it.w.lde;
  a.ldeb_k = t ? it.w.lde : 1;
  a.m = int32_t(it.x.rows);
  a.n = int32_t(t ? it.w.k : it.w.n);
  a.k = int32_t(t ? it.w.n : it.w.k);
  a.out = it.y;
  a.ldo = it.ld_y;
  a.c = it.c;
  a.ldc = it.ld_c;
  a.beta = it.beta;
  return hip_status(muon::launch_few8(a, s));
}

// The launches, of 16 items each, and the workspace of the largest: they follow each
// other on one stream and share it.
muon_status plan_linear8(const muon_linear8_item* items, int32_t n, int32_t dtype, std::vector<muon::PrArgs>& plans, size_t* bytes) {
  *bytes = 0;
  for (int32_t i = 0; i < n; ++i) {
    const muon_linear8_item& it = items[i];
    if (!in_tiles(it, dtype)) continue;
    if (plans.empty() || plans.back().n_items == muon::kPrItems) plans.push_back(muon::PrArgs{});
    muon::PrArgs& a = plans.back();
    muon::PrItem& d = a.item[a.n_items++];
    const bool t = it.transposed != 0;
    a.parts = 1;
    a.f32 = dtype == MUON_F32;
    d.a[0] = static_cast<const uint8_t*>(it.x.q);
    d.lda = it.x.ldq;
    d.ea = static_cast<const uint8_t*>(it.x.e);
    d.lde = it.x.lde;
    d.b[0] = static_cast<const uint8_t*>(t ? it.w.qt : it.w.q);
    d.ldb = t ? it.w.ldqt : it.w.ldq;
    d.eb = static_cast<const uint8_t*>(it.w.e);
    d.ldeb_n = t ? 1 : it.w.lde;
    d.ldeb_k = t ? it.w.lde : 1;
    d.m = int32_t(it.x.rows);
    d.n = int32_t(t ? it.w.k : it.w.n);
    d.k = int32_t(t ? it.w.n : it.w.k);
    d.sums = 1;
    d.out = it.y;
    d.ldo = it.ld_y;
    d.c = it.c;
    d.ldc = it.ld_c;
    d.beta = it.beta;
  }
  for (muon::PrArgs& a : plans) {
    size_t need = 0;
    MUON_TRY(lay_out(a, false, 1, a.f32 ? kLinear8F32Cost : kLinear8Cost, &need));
    *bytes = std::max(*bytes, need);
  }
  return MUON_OK;
}

muon_status linear8(const muon_linear8_item* items, int32_t n, int32_t dtype, void* ws, size_t ws_bytes, void* stream) {
  Views v;
  MUON_TRY(check_linear8(items, n, dtype, v));
  std::vector<muon::PrArgs> plans;
  size_t need = 0;
  MUON_TRY(plan_linear8(items, n, dtype, plans, &need));
  if (need) {
    if (ws_bytes < need)
      return fail(MUON_ERR_INVALID_ARG, "the workspace has " + std::to_string(ws_bytes) + " bytes, " + std::to_string(need) + " are needed");
    if (!ws) return fail(MUON_ERR_INVALID_ARG, "workspace is NULL");
    if (reinterpret_cast<uintptr_t>(ws) % 16) return fail(MUON_ERR_ALIGN, "workspace is not 16-byte aligned");
    MUON_TRY(v.add_range(ws, need, "workspace"));
    MUON_TRY(v.disjoint());
  }
  for (int32_t i = 0; i < n; ++i)
    if (items[i].x.rows > 0 && few_rows(items[i], dtype)) MUON_TRY(few_linear8(items[i], static_cast<hipStream_t>(stream)));
  for (muon::PrArgs& a : plans) {
    a.partial = static_cast<float*>(ws);
    MUON_TRY(hip_status(muon::launch_linear8(a, static_cast<hipStream_t>(stream))));
  }
  return MUON_OK;
}

}  // namespace

extern "C" {

muon_status muon_mlp_forward(const muon_mlp* mlp, void* stream) {
  return guarded([&] { return mlp_forward(mlp, stream); });
}

muon_status muon_mlp_backward(const muon_mlp* mlp, const muon_mlp_grads* grads, void* stream) {
  return guarded([&] { return mlp_backward(mlp, grads, stream); });
}

muon_status muon_mlp_workspace(const muon_mlp* mlp, size_t* bytes) {
  return guarded([&]() -> muon_status {
    if (!mlp || !bytes) return fail(MUON_ERR_INVALID_ARG, "mlp or bytes is NULL");
    return mlp_workspace(*mlp, bytes);
  });
}

muon_status muon_mlp_exact_workspace(const muon_mlp* mlp, const muon_mlp_grads* grads, size_t* bytes) {
  return guarded([&]() -> muon_status {
    if (!mlp || !bytes) return fail(MUON_ERR_INVALID_ARG, "mlp or bytes is NULL");
    return mlp_workspace(*mlp, grads, bytes);
  });
}

muon_status muon_mlp_info(const muon_mlp* mlp, const muon_mlp_grads* grads, int32_t* tile, int32_t* whole, int32_t* pieces) {
  return guarded([&]() -> muon_status {
    if (!mlp || !tile || !whole || !pieces) return fail(MUON_ERR_INVALID_ARG, "mlp, tile, whole or pieces is NULL");
    return mlp_info(*mlp, grads, tile, whole, pieces);
  });
}

muon_status muon_w8_save(const void* w, int64_t ldw, int32_t dtype, const muon_w8* out, void* stream) {
  return w8_call(w, ldw, dtype, out, true, stream);
}

muon_status muon_w8_load(const muon_w8* in, void* w, int64_t ldw, int32_t dtype, void* stream) {
  return w8_call(w, ldw, dtype, in, false, stream);
}

muon_status muon_linear8(const muon_linear8_item* items, int32_t n_items, int32_t dtype, void* workspace, size_t workspace_bytes,
                         void* stream) {
  return guarded([&] { return linear8(items, n_items, dtype, workspace, workspace_bytes, stream); });
}

muon_status muon_linear8_workspace(const muon_linear8_item* items, int32_t n_items, int32_t dtype, size_t* bytes) {
  return guarded([&]() -> muon_status {
    if (!bytes) return fail(MUON_ERR_INVALID_ARG, "bytes is NULL");
    Views v;
    MUON_TRY(check_linear8(items, n_items, dtype, v));
    std::vector<muon::PrArgs> plans;
    return plan_linear8(items, n_items, dtype, plans, bytes);
  });
}

muon_status muon_linear8_info(const muon_linear8_item* items, int32_t n_items, int32_t dtype, int32_t* tile, int32_t* whole,
                              int32_t* pieces) {
  return guarded([&]() -> muon_status {
    if (!tile || !whole || !pieces) return fail(MUON_ERR_INVALID_ARG, "tile, whole or pieces is NULL");
    Views v;
    MUON_TRY(check_linear8(items, n_items, dtype, v));
    std::vector<muon::PrArgs> plans;
    size_t bytes = 0;
    MUON_TRY(plan_linear8(items, n_items, dtype, plans, &bytes));
    int at = 0;  // of the items that go in tiles
    for (int32_t i = 0; i < n_items; ++i) {
      tile[i] = whole[i] = 0;
      pieces[i] = 1;
      if (!in_tiles(items[i], dtype)) continue;
      const muon::PrArgs& a = plans[size_t(at / muon::kPrItems)];
      cut_of(a, a.item[at % muon::kPrItems], tile + i, whole + i, pieces + i);
      ++at;
    }
    return MUON_OK;
  });
}

}  // extern "C"
