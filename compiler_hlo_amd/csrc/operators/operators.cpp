// operators.cpp -- the operators' C ABI: validation, the choice of a kernel
// and its split, the workspace's layout, and the launches.
#include "operators.h"

#include <algorithm>
#include <cmath>
#include <cstring>
#include <memory>
#include <mutex>
#include <new>
#include <string>

#include "../check.h"
#include "../scratch.h"
#include "../ir.h"

namespace hf {
namespace {

struct Buffer {
  std::string name;
  int32_t dtype = HF_F32;
  int rank = 2;
  int64_t rows = 1, cols = 0, ld = 0;  // a vector: one row
  int64_t elem() const {
    switch (dtype) {
      case HF_F32: case HF_S32: return 4;
      case HF_S64: return 8;
      case HF_BF16: case HF_F16: return 2;
    }
    return 1;
  }
  bool empty() const { return rows == 0 || cols == 0; }
  int64_t extent() const { return empty() ? 0 : ((rows - 1) * ld + cols) * elem(); }
  int64_t bytes() const { return rows * cols * elem(); }
};

// One product: its operands as buffers, copied into the workspace first
// where their rows do not start on 16 bytes.
struct Operand {
  int64_t rows = 0, cols = 0, ld = 0;  // as the kernel sees it, in elements
  int64_t pack_at = -1;                // offset of the copy in the workspace
  int64_t src_ld = 0, src_cols = 0;
};
struct Product {
  bool on = false, skinny = false;
  Operand a, b;
  bool gated = false;
  int64_t experts = 0;                 // by expert: b has one weight an expert
  int64_t m = 0, n = 0, k = 0;
  int tile = 0, splits = 1, per_split = 1, waves = 8;
  int64_t tiles_full = 0, part_rows = 0, part_cols = 0;
  int64_t partial_at = 0, ldp = 0;
};

int64_t up(int64_t v, int64_t step) { return (v + step - 1) / step * step; }
int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

}  // namespace
}  // namespace hf

struct hf_operator {
  hf_operator_desc d{};
  int64_t experts = 0, top_k = 0;  // of an extended descriptor
  hf_operator_info info{};
  int device = -1;
  bool plan_only = false;
  hf::Buffer buf[HF_MAX_OPERATOR_BUFFERS];
  int n_params = 0, n_results = 0;
  // buffer numbers of optional operands, -1: none
  int i_scale = -1, i_stream = -1, i_rstd = -1, i_residual = -1, i_a_scale = -1, i_bias = -1, i_z = -1, i_dbias = -1,
      i_offsets = -1, i_weight = -1;
  int64_t ws = 0;
  bool vec = false;
  // gradients of products
  int64_t dz_at = -1, lddz = 0, sums_at = -1;
  int groups = 0;
  hf::Product p1, p2;
};

namespace hf {
namespace {

[[noreturn]] void invalid(const std::string &m) { fail(HF_ERR_INVALID, m); }
[[noreturn]] void unsupported(const std::string &m) { fail(HF_ERR_UNSUPPORTED, m); }

const char *kind_name(int k) {
  static const char *names[] = {"rms_norm",    "rms_norm_grad",   "matmul",         "matmul_grad",         "gated", "gated_grad",
                                "dropout",     "expert_sort",     "expert_dispatch", "expert_combine",
                                "expert_combine_grad", "block_quantize"};
  return names[k];
}

struct Builder {
  hf_operator &op;
  int next = 0;
  int add(const char *name, int32_t dtype, int rank, int64_t rows, int64_t cols) {
    Buffer &b = op.buf[next];
    b.name = name;
    b.dtype = dtype;
    b.rank = rank;
    b.rows = rank == 2 ? rows : 1;
    b.cols = cols;
    const int64_t ld = op.d.row_stride[next];
    if (ld < 0 || (rank == 1 && ld != 0))
      invalid(std::string(name) + ": row stride " + std::to_string(ld) + (rank == 1 ? " of a vector" : ""));
    if (ld > 0 && ld < cols)
      invalid(std::string(name) + ": row stride " + std::to_string(ld) + " is less than its " + std::to_string(cols) +
              " columns");
    b.ld = ld > 0 ? ld : cols;
    int64_t e;
    if (__builtin_mul_overflow(b.rows, b.ld, &e) || e > (int64_t(1) << 56) / 8)
      unsupported(std::string(name) + ": more than 2^56 bytes");
    return next++;
  }
};

constexpr int64_t kBlock = 128;  // of block scales

bool is_half(int t) { return t == HF_BF16 || t == HF_F16; }
bool is_eight(int t) { return t == HF_S8 || t == HF_F8E4M3; }

// Rows that start on 16 bytes (the base pointer does) with whole 16-byte
// vectors, or no second row.
bool aligned16(const Buffer &b) { return b.rows <= 1 || (b.ld * b.elem()) % 16 == 0; }

int64_t take(hf_operator &op, int64_t bytes) {
  const int64_t at = op.ws;
  op.ws = up(op.ws + bytes, 256);
  return at;
}

// The operand as the product kernels take it.  By row, 16-byte chunks of the
// contraction must not run into the next row: the length is padded with zeros
// in a copy where it is no multiple of 16 bytes.  By column, a chunk past the
// last column only feeds sums that are not stored, but it must be aligned.
Operand operand(hf_operator &op, int64_t rows, int64_t cols, int64_t ld, int64_t elem, const char *what) {
  Operand o;
  o.rows = rows;
  o.cols = cols;
  o.ld = o.src_ld = ld;
  o.src_cols = cols;
  if ((cols * elem) % 16 || (rows > 1 && (ld * elem) % 16)) {
    o.cols = o.ld = up(cols, 16 / elem);
    o.pack_at = take(op, rows * o.ld * elem);
  }
  if (o.ld * elem >= (int64_t(8) << 20)) unsupported(std::string(what) + ": rows of 8 MB or more");
  return o;
}

int64_t tiles_of(const Product &p, int64_t tile) { return cdiv(p.m, tile) * cdiv(p.n, p.gated ? tile / 2 : tile); }

// Threads of a product's tiles.
int64_t tile_threads(const Product &p) {
  if (!p.on || p.skinny || p.tile > 1) return 0;
  const int64_t shared = tiles_of(p, p.tile == 0 ? 256 : 128) - p.tiles_full;
  return (p.tiles_full + shared * p.splits) * (p.tile == 0 ? 512 : 256);
}

// The same of products by expert, a gradient's both.
double expert_threads(const hf_operator &op) {
  const Product &p = op.p1, &q = op.p2;
  double n = 0;
  const int64_t rows = p.tile == 0 ? 256 : p.tile == 1 ? 128 : 64, cols = p.tile == 0 ? 256 : 128;
  if (p.on)
    n += p.splits * ((double)expert_tiles(p.m, p.experts, rows, 1) * (double)cdiv(p.n, p.gated ? cols / 2 : cols) + 128);
  // dealt out in whole turns of eight chunks, a 128th of the tiles each at most
  if (q.on) n += q.splits * (1.125 * (double)q.experts * (double)cdiv(q.m, rows) * (double)cdiv(q.n, cols) + 8);
  return n * (p.tile == 1 ? 256 : 512);
}

// The tile (first .. last: 0 the larger, 1 the smaller), and how the last
// tiles are shared: the shortest time by a simple
// account, in microseconds.  A round of tiles (256 of the larger, 512 of the
// smaller, two a compute unit) takes its stages and an end (sums out, the next
// tile's first loads in); sharing costs a launch and the partial sums' way to
// memory and back.  The constants are fits to bf16 and e4m3 products of
// 128 .. 4099 rows with 4096 columns over 4096 .. 16384, all within 10%: a
// stage takes 1.1 (1.35 with the chip full) in the larger tile, 0.6 (0.95 with
// two a compute unit) in the smaller.  What it decides there: 4099 x 4096 x
// 16384 e4m3, 272 large tiles, the last 16 shared by 8 workgroups each, 218
// (303 unshared); 1024 x 4096 x 4096 small tiles, 41 (large 73); 256 x 4096 x
// 4096 small tiles shared by 4, 22 (unshared 37).
double choose_tiles(Product &p, int64_t steps, int first, int last) {
  double best = 1e300;
  for (int tile = first; tile <= last; ++tile) {
    const int64_t t = tile == 0 ? 256 : 128, slots = tile == 0 ? 256 : 512, all = tiles_of(p, t);
    const double full_stage = tile == 0 ? 1.35 : 0.95, end = tile == 0 ? 6.0 : 3.0;
    const auto stage = [&](int64_t groups) { return groups <= slots / 2 ? (tile == 0 ? 1.1 : 0.6) : full_stage; };
    const int64_t full = all / slots * slots, rest = all - full;
    for (int64_t s = 1; s <= 16 && (s == 1 || (rest > 0 && rest * s <= slots && steps >= 2 * s)); ++s) {
      double us = (double)(full / slots) * ((double)steps * full_stage + end);
      if (rest > 0) us += (double)cdiv(steps, s) * stage(rest * s) + end;
      if (s > 1) us += 3.0 + 2.0 * 4.0 * (double)(s * rest * std::min(t, p.m) * t) / 6e6;
      if (us >= best) continue;
      best = us;
      p.tile = tile;
      p.tiles_full = s > 1 ? full : all;
      p.per_split = (int)std::max<int64_t>(1, cdiv(steps, s));
      p.splits = s > 1 ? (int)cdiv(steps, p.per_split) : 1;
      if (p.splits == 1) p.tiles_full = all;
    }
  }
  return best;
}

// Which kernel, which tile and how many parts the contraction is split into.
// m x n are the sums (gated: n gate and n up columns).  Returns the time that
// it accounts for, in microseconds.
double choose(const hf_operator_desc &d, Product &p, int64_t elem) {
  p.on = p.m > 0 && p.n > 0;
  if (!p.on) return 0.0;
  double best = 1e300;
  const int64_t kbytes = p.k * elem;
  p.ldp = p.gated ? 2 * up(p.n, 8) : up(p.n, 8);
  p.skinny = false;
  p.splits = 1;
  // e4m3 widened to 16 bits has no registers to spare for the larger tile or
  // for 16 waves a workgroup
  const bool wide = d.dtype == HF_F8E4M3 && f8_wide(d.out_dtype, p.k);
  const int64_t strips = cdiv(p.n, p.gated ? 64 : 128);
  if (p.m <= 8 && strips <= 64) {
    // Too few strips to fill the chip without sharing the contraction, and so
    // few rows that reading them once for every 16 columns costs little (1 x
    // 4096 x 16384 bf16 26 us, strips 30; 8 x 4096 x 4096 10, strips 12).  With
    // more columns strips are as fast or faster (1 x 22528 x 4096 34 us, skinny
    // 36; 8 rows 34.5 and 43).
    p.skinny = true;
    const int64_t columns = cdiv(p.n, 16), blocks = cdiv(kbytes, 512);
    // As many waves a workgroup as let all workgroups run at once (about 5000
    // waves fit): a second round of workgroups for the last few costs as much
    // as the first.
    p.waves = columns * 16 <= 5120 && !wide ? 16 : 8;
    int64_t s = 1;
    while (columns * s < 256 && blocks >= 2 * s * p.waves) s *= 2;
    p.per_split = (int)cdiv(blocks > 0 ? blocks : 1, s);
    p.splits = blocks > 0 ? (int)cdiv(blocks, p.per_split) : 1;
    best = 4.0 + (double)((p.gated ? 2 : 1) * p.n * kbytes) / 5e6;
  } else if (p.m <= 64) {
    // Shares of the contraction: the shortest time by an account like that of
    // the tiles.  A stage takes its share of the memory's rate, or the latency
    // that four stages in flight leave where there are few workgroups (fits to
    // 16 .. 64 rows, within 20%: 64 x 4096 x 4096 by 4 16 us, unshared 30; 32 x
    // 4096 x 16384 by 8 32 us, unshared 96; 24 x 22528 x 4096 unshared 38).
    p.tile = 2;
    const int64_t steps = cdiv(p.k, 128 / elem);
    for (int64_t s = 1; s <= 32 && (s == 1 || (strips * s <= 256 && steps >= 2 * s)); ++s) {
      const double stage = std::max(0.25 + 0.003 * (double)p.m, 0.00325 * (double)std::min<int64_t>(strips * s, 256));
      double us = (double)cdiv(strips * s, 256) * ((double)cdiv(steps, s) * stage + 3.0);
      if (s > 1) us += 3.5 + 8.0 * (double)(s * p.m * p.ldp) / 5e6;
      if (us >= best) continue;
      best = us;
      p.per_split = (int)std::max<int64_t>(1, cdiv(steps, s));
      p.splits = steps > 0 ? (int)cdiv(steps, p.per_split) : 1;
    }
  } else {
    best = choose_tiles(p, cdiv(p.k, 128 / elem), wide ? 1 : 0, 1);
  }
  return best;
}

// The same for a gradient's two products, which run in one launch with tiles
// of one size.
void choose_gradient(Product &p, Product &q) {
  p.on = p.m > 0 && p.n > 0;
  q.on = q.m > 0 && q.n > 0;
  double best = 1e300;
  const Product p0 = p, q0 = q;
  for (int tile = 0; tile < 2; ++tile) {
    Product x = p0, y = q0;
    double us = 0.0;
    if (x.on) us += choose_tiles(x, cdiv(x.k, 64), tile, tile);
    if (y.on) us += choose_tiles(y, cdiv(y.k, 64), tile, tile);
    if (us >= best) continue;
    best = us;
    p = x;
    q = y;
    p.tile = q.tile = tile;
  }
}

// The partial sums' place, for what choose() chose.
void place_partials(hf_operator &op, Product &p) {
  if (!p.on || p.splits == 1) return;
  const bool tiles = !p.skinny && p.tile < 2;
  const int64_t t = p.tile == 0 ? 256 : 128;
  p.part_rows = std::min(p.m, t);
  p.part_cols = p.gated ? 2 * std::min(t / 2, up(p.n, 8)) : std::min(t, up(p.n, 8));
  const int64_t sums = tiles ? (tiles_of(p, t) - p.tiles_full) * p.part_rows * p.part_cols
                             : p.m * p.ldp;
  p.partial_at = take(op, p.splits * sums * 4);
}

// Products by expert.  How the rows are shared out is not known here, so the
// kernel goes by the rows that an expert has if all have as many (measured with
// the most liked of 8 to 64 experts at two to three times that):
// - up to 24, strips (16 experts of 16 rows, gated 2048 x 4096 e4m3 with block
//   scales 59 us, small tiles 68; 32 of 32 rows, 4096 x 1408 bf16 87 and 76);
// - large tiles from 160 on (8 of 256, gated 4096 x 4096 bf16 176 us, small 210;
//   32 of 96, gated 1408 x 4096 201 and 177), with block scales from 192 on (32
//   of 128, gated 1408 x 4096 120 us, small 107; of 256 135 and 165; 8 of 256,
//   gated 4096 x 4096 113 and 126; of 1024 296 and 358), where they make 128 or
//   more (8 of 256, 512 x 512 bf16 13.8 us, small 11.6);
// - small tiles between.
void choose_experts(const hf_operator &op, Product &p, bool wide) {
  p.on = p.m > 0 && p.n > 0;
  p.experts = op.experts;
  const int64_t rows = p.m / std::max<int64_t>(1, std::min(op.experts, p.m));
  const int64_t from = op.d.flags & HF_OPERATOR_BLOCK_SCALES ? 192 : 160;
  const bool large = !wide && rows >= from && p.m / 256 * cdiv(p.n, p.gated ? 128 : 256) >= 128;
  p.tile = rows <= 24 ? 2 : large ? 0 : 1;
  // The contraction is shared where the tiles are few, by an account of the
  // times as in choose_tiles and choose (a launch more to add the parts counts 4
  // us), for as many tiles as experts with half a tile of rows past their last
  // whole one: 1 row of 8 experts, 2048 x 4096 bf16 by 8 12 us, whole 19; 200 of
  // 4, 512 x 4096 by 16 19 and 36; 1024 of 4, 1024 x 4096 by 3 25 and 37.  8-bit
  // sums whose scales go by the expert's rows stay whole.
  const int64_t steps = std::max<int64_t>(1, cdiv(p.k, 128 / op.buf[0].elem())), size = p.tile == 2 ? 64 : 128;
  const int64_t across = cdiv(p.n, p.gated ? 64 : 128), some = std::min(op.experts, p.m);
  const int64_t groups = std::max<int64_t>(some, p.m / size + some / 2) * across, slots = p.tile == 2 ? 256 : 512;
  p.ldp = p.gated ? 2 * up(p.n, 8) : up(p.n, 8);
  p.per_split = (int)steps;
  const bool whole = p.tile == 0 || (is_eight(op.d.dtype) && !(op.d.flags & HF_OPERATOR_BLOCK_SCALES));
  double best = 1e300;
  for (int64_t s = 1; p.on && s <= 16 && (s == 1 || (!whole && groups * s <= slots && steps >= 2 * s)); ++s) {
    const double stage = p.tile == 2 ? std::max(0.3, 0.00325 * (double)std::min<int64_t>(groups * s, 256))
                                     : groups * s <= 256 ? 0.6 : 0.95;
    double us = (double)cdiv(groups * s, slots) * ((double)cdiv(steps, s) * stage + 3.0);
    if (s > 1) us += 4.0 + 8.0 * (double)(s * p.m * p.ldp) / 5e6;
    if (us >= best) continue;
    best = us;
    p.per_split = (int)cdiv(steps, s);
    p.splits = (int)cdiv(steps, p.per_split);
  }
}

// A gradient by expert: large tiles where db has 128 or more (16 experts of 256
// rows, 4096 x 1408 bf16 173 us, small 189; 8 of 64, 4096 x 4096 168 and 191) that
// hold no more than an eighth more sums than small ones, as every expert's weight
// is rounded up to them (8192 rows of 128 experts, 128 x 128 17.2 us, small 11.8;
// of 64, 384 x 384 37 and 26; 16384 of 60, 640 x 384 60 and 44; as many sums: 8192
// of 200, 136 x 136 24.8 and 27.1).
void choose_experts_gradient(const hf_operator &op, Product &p, Product &q) {
  p.on = p.m > 0 && p.n > 0;
  q.on = q.m > 0 && q.n > 0;
  p.experts = q.experts = op.experts;
  const int64_t large = op.experts * cdiv(q.m, 256) * cdiv(q.n, 256), small = op.experts * cdiv(q.m, 128) * cdiv(q.n, 128);
  p.tile = q.tile = large >= 128 && large * 4 * 8 <= small * 9 ? 0 : 1;
  // Small tiles that leave most of the chip idle share the contractions, by the
  // same account: da's over b's rows, db's over twice the rows that an expert
  // has if all have as many (5549 rows of one expert, 128 x 896 bf16 21 us, whole
  // 61; 12 of 2, 3712 x 320 17 and 36).
  p.ldp = q.ldp = up(q.n, 8);
  const int64_t steps_p = std::max<int64_t>(1, cdiv(p.k, 64)), some = std::max<int64_t>(1, std::min(op.experts, p.m));
  const int64_t steps_q = std::max<int64_t>(1, cdiv(2 * p.m / some, 64)), across = cdiv(q.n, 128);
  const int64_t groups_p = p.on ? std::max<int64_t>(some, p.m / 128 + some / 2) * across : 0;
  const int64_t groups_q = q.on ? op.experts * cdiv(q.m, 128) * across : 0;
  p.per_split = (int)steps_p;
  double best = 1e300;
  for (int64_t s = 1; s <= 16 && (s == 1 || (p.on && p.tile == 1 && steps_p >= 2 * s)); ++s)
    for (int64_t t = 1; t <= 16 && (t == 1 || (q.on && p.tile == 1 && steps_q >= 2 * t)); ++t) {
      const int64_t all = groups_p * s + groups_q * t;
      if ((s > 1 || t > 1) && all > 512) continue;
      const double stage = all <= 256 ? 0.6 : 0.95;
      double us = (double)std::max(p.on ? cdiv(steps_p, s) : 0, q.on ? cdiv(steps_q, t) : 0) * stage;
      if (s > 1) us += 4.0 + 8.0 * (double)(s * p.m * p.ldp) / 5e6;
      if (t > 1) us += 4.0 + 8.0 * (double)(t * op.experts * q.m * q.ldp) / 5e6;
      if (us >= best) continue;
      best = us;
      p.per_split = (int)cdiv(steps_p, s);
      p.splits = (int)cdiv(steps_p, p.per_split);
      q.splits = (int)t;
    }
}

// The partial sums' place of products by expert.
void place_expert_partials(hf_operator &op, Product &p, int64_t rows) {
  if (p.on && p.splits > 1) p.partial_at = take(op, p.splits * rows * p.ldp * 4);
}

void plan_norm(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  Builder b{op};
  b.add("x", d.dtype, 2, d.m, d.n);
  b.add("weight", d.weight_dtype, 1, 1, d.n);
  const bool res = d.flags & HF_OPERATOR_RESIDUAL;
  if (res) op.i_residual = b.add("residual", d.dtype, 2, d.m, d.n);
  op.n_params = b.next;
  b.add("y", d.out_dtype, 2, d.m, d.n);
  if (is_eight(d.out_dtype)) op.i_scale = b.add("scale", HF_F32, 1, 1, d.m);
  if (res) op.i_stream = b.add("stream", d.dtype, 2, d.m, d.n);
  op.i_rstd = b.add("rstd", HF_F32, 1, 1, d.m);
  op.n_results = b.next - op.n_params;
  op.vec = d.n % 8 == 0;
  for (int i = 0; i < b.next; ++i) {
    const Buffer &u = op.buf[i];
    if (u.rank != 2) continue;
    // 8-bit rows take 8-byte stores
    if (u.rows > 1 && (u.ld * u.elem()) % (is_eight(u.dtype) ? 8 : 16)) op.vec = false;
  }
}

void plan_norm_grad(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  Builder b{op};
  b.add("dy", d.dtype, 2, d.m, d.n);
  b.add("h", d.dtype, 2, d.m, d.n);
  b.add("weight", d.weight_dtype, 1, 1, d.n);
  op.i_rstd = b.add("rstd", HF_F32, 1, 1, d.m);
  if (d.flags & HF_OPERATOR_RESIDUAL) op.i_residual = b.add("dstream", d.dtype, 2, d.m, d.n);
  op.n_params = b.next;
  b.add("dx", d.dtype, 2, d.m, d.n);
  b.add("dweight", HF_F32, 1, 1, d.n);
  op.n_results = b.next - op.n_params;
  op.vec = d.n % 8 == 0;
  for (int i = 0; i < b.next; ++i)
    if (op.buf[i].rank == 2 && !aligned16(op.buf[i])) op.vec = false;
  op.groups = norm_grad_groups(d.m, d.n);
  op.sums_at = take(op, (int64_t)op.groups * d.n * 4);
}

void plan_dropout(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  Builder b{op};
  b.add("x", d.dtype, 2, d.m, d.n);
  b.add("state", HF_S64, 1, 1, 2);
  if (d.flags & HF_OPERATOR_RESIDUAL) op.i_residual = b.add("residual", d.dtype, 2, d.m, d.n);
  op.n_params = b.next;
  b.add("y", d.dtype, 2, d.m, d.n);
  op.n_results = 1;
}

void plan_product(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  const bool gated = d.kind == HF_OPERATOR_GATED;
  const int64_t wide = gated ? 2 * d.n : d.n;
  Builder b{op};
  const int64_t weights = op.experts ? op.experts : 1;
  b.add("a", d.dtype, 2, d.m, d.k);
  b.add("b", d.dtype, 2, weights * wide, d.k);
  if (d.flags & HF_OPERATOR_BLOCK_SCALES) {
    const int64_t along = cdiv(d.k, kBlock), high = cdiv(d.n, kBlock);
    op.i_a_scale = b.add("a_scale", HF_F32, 2, along, d.m);
    b.add("b_scale", HF_F32, 2, weights * (gated ? 2 : 1) * high, along);
  } else if (is_eight(d.dtype)) {
    op.i_a_scale = b.add("a_scale", HF_F32, 1, 1, d.m);
    b.add("b_scale", HF_F32, 1, 1, weights * wide);
  }
  if (op.experts) op.i_offsets = b.add("offsets", HF_S32, 1, 1, op.experts + 1);
  if (d.flags & HF_OPERATOR_BIAS) op.i_bias = b.add("bias", d.out_dtype, 1, 1, d.n);
  if (d.flags & HF_OPERATOR_RESIDUAL) op.i_residual = b.add("residual", d.out_dtype, 2, d.m, d.n);
  op.n_params = b.next;
  b.add("d", d.out_dtype, 2, d.m, d.n);
  if (d.flags & HF_OPERATOR_SAVE) op.i_z = b.add("z", d.out_dtype, 2, d.m, wide);
  op.n_results = b.next - op.n_params;
  // the epilogue's accesses of eight elements
  op.vec = !gated || op.i_z < 0 || d.n % 8 == 0;
  for (int i : {op.n_params, op.i_z, op.i_residual})
    if (i >= 0 && op.buf[i].rows > 1 && op.buf[i].ld % 8) op.vec = false;
  // an expert's scales begin at a multiple of 4 of them
  if (op.experts && is_eight(d.dtype) && wide % 4) op.vec = false;
  const int64_t elem = op.buf[0].elem();
  Product &p = op.p1;
  p.m = d.m;
  p.n = d.n;
  p.gated = gated;
  if (p.m > 0 && p.n > 0) {
    p.a = operand(op, d.m, d.k, op.buf[0].ld, elem, "a");
    p.b = operand(op, weights * wide, d.k, op.buf[1].ld, elem, "b");
    p.k = p.a.pack_at >= 0 || p.b.pack_at >= 0 ? up(d.k, 16 / elem) : d.k;
  }
  if (op.experts) {
    choose_experts(op, p, d.dtype == HF_F8E4M3 && f8_wide(d.out_dtype, p.k));
    place_expert_partials(op, p, p.m);
    return;
  }
  const double whole = choose(d, p, elem);
  // A few rows past a multiple of 256 cost a row of tiles; where a strip (or a
  // skinny product) for them is shorter, they get one (4099 x 4096 x 16384
  // e4m3: 222 us with them in tiles, 207 us so).
  const int64_t tail = d.m % 256;
  if (d.m > 256 && tail > 0 && tail <= 64 && p.n > 0) {
    Product body = p, rest = p;
    body.m = d.m - tail;
    body.a.rows = body.m;
    rest.m = rest.a.rows = tail;
    if (choose(d, body, elem) + choose(d, rest, elem) < whole) {
      op.p1 = body;
      op.p2 = rest;
    }
  }
  place_partials(op, op.p1);
  place_partials(op, op.p2);
}

void plan_product_grad(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  const bool gated = d.kind == HF_OPERATOR_GATED_GRAD;
  const int64_t wide = gated ? 2 * d.n : d.n;
  Builder b{op};
  const int64_t weights = op.experts ? op.experts : 1;
  b.add("dd", d.dtype, 2, d.m, d.n);
  b.add("a", d.dtype, 2, d.m, d.k);
  b.add("b", d.dtype, 2, weights * wide, d.k);
  if (gated || d.activation != HF_ACTIVATION_NONE) op.i_z = b.add("z", d.dtype, 2, d.m, wide);
  if (op.experts) op.i_offsets = b.add("offsets", HF_S32, 1, 1, op.experts + 1);
  op.n_params = b.next;
  b.add("da", d.dtype, 2, d.m, d.k);
  b.add("db", d.dtype, 2, weights * wide, d.k);
  if (d.flags & HF_OPERATOR_BIAS) op.i_dbias = b.add("dbias", HF_F32, 1, 1, d.n);
  op.n_results = b.next - op.n_params;
  const int64_t elem = 2;
  op.vec = d.n % 8 == 0 && aligned16(op.buf[0]) && (op.i_z < 0 || aligned16(op.buf[op.i_z]));
  // dz: in the workspace where an activation makes it, or where dd's rows do
  // not start on 16 bytes; rows of a multiple of 8, the tail zero
  op.lddz = up(wide, 8);
  if (wide > 0 && d.m > 0 && (op.i_z >= 0 || !op.vec)) op.dz_at = take(op, d.m * op.lddz * elem);
  const int64_t ldz = op.dz_at >= 0 ? op.lddz : op.buf[0].ld;
  if (ldz * elem >= (int64_t(8) << 20)) unsupported("dd: rows of 8 MB or more");
  op.groups = act_grad_groups(d.m, d.n);
  if (op.i_dbias >= 0) op.sums_at = take(op, (int64_t)op.groups * d.n * 4);
  Operand dz;
  dz.rows = d.m;
  dz.ld = ldz;
  Operand a, w;
  if (d.k > 0 && wide > 0) {
    if (d.m > 0) a = operand(op, d.m, d.k, op.buf[1].ld, elem, "a");
    w = operand(op, weights * wide, d.k, op.buf[2].ld, elem, "b");
  }
  // da [m, k] = dz [m, wide] b [wide, k]
  Product &p = op.p1;
  p.m = d.m;
  p.n = d.k;
  p.k = wide;
  p.a = dz;
  p.a.cols = p.k;
  p.b = w;
  if (op.dz_at >= 0) p.k = op.lddz;  // whole 16-byte chunks; past `wide`, zeros on both sides
  p.a.cols = p.k;
  // db [wide, k] = dz^T [wide, m] a [m, k]
  Product &q = op.p2;
  q.m = wide;
  q.n = d.k;
  q.k = d.m;
  q.a = dz;
  // whole chunks in the last row too: dz's padding is there to be read
  q.a.cols = up(wide, 8);
  q.b = a;
  if (op.experts) {
    choose_experts_gradient(op, p, q);
    place_expert_partials(op, p, p.m);
    place_expert_partials(op, q, op.experts * q.m);
    return;
  }
  choose_gradient(p, q);
  place_partials(op, p);
  place_partials(op, q);
}

void plan_sort(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  Builder b{op};
  b.add("expert", HF_S32, 2, d.m, op.top_k);
  op.n_params = b.next;
  b.add("place", HF_S32, 2, d.m, op.top_k);
  b.add("order", HF_S32, 1, 1, d.m * op.top_k);
  b.add("offsets", HF_S32, 1, 1, op.experts + 1);
  op.n_results = b.next - op.n_params;
  int32_t chunks, per;
  sort_chunks(d.m * op.top_k, &chunks, &per);
  if (chunks > 1) op.sums_at = take(op, (int64_t)chunks * op.experts * 4);
}

void plan_dispatch(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  const int64_t pairs = d.m * op.top_k;
  const bool blocks = d.flags & HF_OPERATOR_BLOCK_SCALES;
  Builder b{op};
  b.add("x", d.dtype, 2, d.m, d.n);
  b.add("place", HF_S32, 2, d.m, op.top_k);
  if (blocks) op.i_a_scale = b.add("x_scale", HF_F32, 2, cdiv(d.n, kBlock), d.m);
  else if (is_eight(d.dtype)) op.i_a_scale = b.add("x_scale", HF_F32, 1, 1, d.m);
  op.n_params = b.next;
  b.add("y", d.dtype, 2, pairs, d.n);
  if (blocks) op.i_scale = b.add("y_scale", HF_F32, 2, cdiv(d.n, kBlock), pairs);
  else if (is_eight(d.dtype)) op.i_scale = b.add("y_scale", HF_F32, 1, 1, pairs);
  op.n_results = b.next - op.n_params;
}

void plan_combine(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  const int64_t pairs = d.m * op.top_k;
  const bool grad = d.kind == HF_OPERATOR_EXPERT_COMBINE_GRAD;
  Builder b{op};
  if (grad) b.add("dd", d.dtype, 2, d.m, d.n);
  b.add("y", d.dtype, 2, pairs, d.n);
  b.add("place", HF_S32, 2, d.m, op.top_k);
  if (grad || (d.flags & HF_OPERATOR_WEIGHTS)) op.i_weight = b.add("weight", HF_F32, 2, d.m, op.top_k);
  if (d.flags & HF_OPERATOR_RESIDUAL) op.i_residual = b.add("residual", d.dtype, 2, d.m, d.n);
  op.n_params = b.next;
  if (grad) {
    b.add("dy", d.dtype, 2, pairs, d.n);
    b.add("dweight", HF_F32, 2, d.m, op.top_k);
  } else {
    b.add("d", d.dtype, 2, d.m, d.n);
  }
  op.n_results = b.next - op.n_params;
  op.vec = d.n % 8 == 0;
  for (int i : {0, grad ? 1 : -1, op.i_residual, op.n_params})
    if (i >= 0 && !aligned16(op.buf[i])) op.vec = false;
}

void plan_quantize(hf_operator &op) {
  const hf_operator_desc &d = op.d;
  Builder b{op};
  b.add("x", d.dtype, 2, d.m, d.n);
  op.n_params = 1;
  b.add("y", HF_F8E4M3, 2, d.m, d.n);
  b.add("scale", HF_F32, 2, cdiv(d.n, kBlock), d.m);
  op.n_results = 2;
  op.vec = d.n % 8 == 0 && aligned16(op.buf[0]) && (op.buf[1].rows <= 1 || op.buf[1].ld % 8 == 0);
}

// The rules that an extended descriptor's fields add.
void check_extended(const hf_operator &op, const std::string &who) {
  const hf_operator_desc &d = op.d;
  const bool product = d.kind >= HF_OPERATOR_MATMUL && d.kind <= HF_OPERATOR_GATED_GRAD;
  const bool grad = d.kind == HF_OPERATOR_MATMUL_GRAD || d.kind == HF_OPERATOR_GATED_GRAD;
  const bool sort = d.kind == HF_OPERATOR_EXPERT_SORT;
  const bool pairs = d.kind >= HF_OPERATOR_EXPERT_SORT && d.kind <= HF_OPERATOR_EXPERT_COMBINE_GRAD;
  if (op.experts < 0 || (sort && op.experts < 1) || (!sort && !product && op.experts))
    invalid(who + ": experts of " + std::to_string(op.experts));
  if (op.experts > HF_MAX_EXPERTS) unsupported(who + ": more than " + std::to_string(HF_MAX_EXPERTS) + " experts");
  if (pairs ? op.top_k < 1 : op.top_k != 0) invalid(who + ": top_k of " + std::to_string(op.top_k));
  int64_t count = 0;
  if (pairs && (__builtin_mul_overflow(d.m, op.top_k, &count) || count > 0x7ff00000 || op.top_k > HF_MAX_EXPERTS))
    unsupported(who + ": too many pairs of a token and an expert");
  if (sort && (d.n || d.k)) invalid(who + ": n and k must be 0");
  if ((d.flags & HF_OPERATOR_BLOCK_SCALES) && (grad || d.dtype != HF_F8E4M3))
    invalid(who + ": block scales are f8e4m3's");
  if (product && op.experts) {
    if (d.flags & (HF_OPERATOR_RESIDUAL | HF_OPERATOR_BIAS)) unsupported(who + ": a bias or a residual by expert");
    if (op.experts * d.n * 2 > (int64_t(1) << 31)) unsupported(who + ": weights of more than 2^31 rows");
  }
}

void make_plan(hf_operator &op, bool extended) {
  const hf_operator_desc &d = op.d;
  if (d.kind < 0 || d.kind > (extended ? HF_OPERATOR_BLOCK_QUANTIZE : HF_OPERATOR_DROPOUT))
    invalid("unknown operator kind " + std::to_string(d.kind));
  const std::string who = kind_name(d.kind);
  const bool product = d.kind >= HF_OPERATOR_MATMUL && d.kind <= HF_OPERATOR_GATED_GRAD;
  const bool grad = d.kind == HF_OPERATOR_MATMUL_GRAD || d.kind == HF_OPERATOR_GATED_GRAD;
  const int64_t most = 0x7fffff00;
  for (int64_t v : {d.m, d.n, d.k})
    if (v < 0) invalid(who + ": a negative size");
  for (int64_t v : {d.m, d.n, d.k})
    if (v > most) unsupported(who + ": a size of 2^31 or more");
  // columns and tiles are counted in 32 bits, with room for a tile's padding
  const int64_t wide_most = int64_t(1) << 30;
  if (d.kind != HF_OPERATOR_DROPOUT && d.n > wide_most) unsupported(who + ": more than 2^30 columns");
  if (product && (d.m > wide_most || d.k > wide_most)) unsupported(who + ": a size of more than 2^30");
  if (!product && d.k != 0) invalid(who + ": k must be 0");
  static const uint32_t allowed[] = {HF_OPERATOR_RESIDUAL, HF_OPERATOR_RESIDUAL,
                                     HF_OPERATOR_RESIDUAL | HF_OPERATOR_BIAS | HF_OPERATOR_SAVE, HF_OPERATOR_BIAS,
                                     HF_OPERATOR_SAVE, 0, HF_OPERATOR_RESIDUAL, 0, HF_OPERATOR_BLOCK_SCALES,
                                     HF_OPERATOR_RESIDUAL | HF_OPERATOR_WEIGHTS, 0, 0};
  const bool forward = d.kind == HF_OPERATOR_MATMUL || d.kind == HF_OPERATOR_GATED;
  if (d.flags & ~(allowed[d.kind] | (extended && forward ? HF_OPERATOR_BLOCK_SCALES : 0))) invalid(who + ": flags it does not take");
  if (d.dtype < HF_F32 || d.dtype > HF_S64 || d.out_dtype < HF_F32 || d.out_dtype > HF_S64)
    invalid(who + ": unknown element type");
  if (d.activation < HF_ACTIVATION_NONE || d.activation > HF_ACTIVATION_SILU || (!product && d.activation))
    invalid(who + ": unknown or misplaced activation");
  if (extended) check_extended(op, who);
  if (d.kind == HF_OPERATOR_EXPERT_SORT) {
  } else if (d.kind == HF_OPERATOR_EXPERT_DISPATCH) {
    if (!is_half(d.dtype) && !is_eight(d.dtype) && d.dtype != HF_F32) unsupported(who + ": this element type");
    if (d.out_dtype != d.dtype) unsupported(who + ": results of this element type");
  } else if (d.kind == HF_OPERATOR_BLOCK_QUANTIZE) {
    if (!is_half(d.dtype) && d.dtype != HF_F32) unsupported(who + ": this element type");
    if (d.out_dtype != HF_F8E4M3) unsupported(who + ": results of this element type");
  } else if (product) {
    const bool ok = grad ? is_half(d.dtype) : is_half(d.dtype) || is_eight(d.dtype);
    if (!ok) unsupported(who + ": operands of this element type");
    if (grad ? d.out_dtype != d.dtype : !is_half(d.out_dtype) && d.out_dtype != HF_F32)
      unsupported(who + ": results of this element type");
    if ((d.kind == HF_OPERATOR_GATED || d.kind == HF_OPERATOR_GATED_GRAD) && 2 * d.n > wide_most)
      unsupported(who + ": 2n of more than 2^30");
    if (d.dtype == HF_S8 && d.k >= (1 << 17)) unsupported(who + ": s8 sums over k >= 2^17 do not fit 32 bits");
  } else {
    if (!is_half(d.dtype) && d.dtype != HF_F32) unsupported(who + ": this element type");
    if (d.kind == HF_OPERATOR_RMS_NORM ? d.out_dtype != d.dtype && !is_eight(d.out_dtype) : d.out_dtype != d.dtype)
      unsupported(who + ": results of this element type");
  }
  if (d.kind == HF_OPERATOR_RMS_NORM || d.kind == HF_OPERATOR_RMS_NORM_GRAD) {
    if (d.n < 1) invalid(who + ": rows of no elements");
    if (d.weight_dtype != d.dtype && d.weight_dtype != HF_F32) invalid(who + ": the weight is of dtype or f32");
    if (!(d.epsilon >= 0) || std::isinf(d.epsilon)) invalid(who + ": epsilon must be finite and >= 0");
  }
  if (d.kind == HF_OPERATOR_DROPOUT && !(d.probability >= 0 && d.probability < 1))
    invalid(who + ": probability must be in [0, 1)");
  switch (d.kind) {
    case HF_OPERATOR_RMS_NORM: plan_norm(op); break;
    case HF_OPERATOR_RMS_NORM_GRAD: plan_norm_grad(op); break;
    case HF_OPERATOR_DROPOUT: plan_dropout(op); break;
    case HF_OPERATOR_MATMUL: case HF_OPERATOR_GATED: plan_product(op); break;
    case HF_OPERATOR_EXPERT_SORT: plan_sort(op); break;
    case HF_OPERATOR_EXPERT_DISPATCH: plan_dispatch(op); break;
    case HF_OPERATOR_EXPERT_COMBINE: case HF_OPERATOR_EXPERT_COMBINE_GRAD: plan_combine(op); break;
    case HF_OPERATOR_BLOCK_QUANTIZE: plan_quantize(op); break;
    default: plan_product_grad(op);
  }
  if (op.experts && product) {
    if (expert_threads(op) >= 4e9) unsupported(who + ": more tiles than a launch holds (2^32 threads)");
  }
  // a gradient's two products share a launch; the last rows' strip has none of these
  else if (tile_threads(op.p1) + tile_threads(op.p2) >= (int64_t(1) << 32))
    unsupported(who + ": more tiles than a launch holds (2^32 threads)");
  for (int i = op.n_params + op.n_results; i < HF_MAX_OPERATOR_BUFFERS; ++i)
    if (d.row_stride[i]) invalid(who + ": a row stride for a buffer it does not have");
  hf_operator_info &f = op.info;
  f.n_params = op.n_params;
  f.n_results = op.n_results;
  f.workspace_bytes = op.ws;
  for (int i = 0; i < op.n_params + op.n_results; ++i) {
    const Buffer &b = op.buf[i];
    f.buffers[i].dtype = b.dtype;
    f.buffers[i].rank = b.rank;
    f.buffers[i].dims[0] = b.rank == 2 ? b.rows : b.cols;
    f.buffers[i].dims[1] = b.rank == 2 ? b.cols : 1;
    f.buffers[i].row_stride = b.rank == 2 ? b.ld : 0;
    f.algorithmic_bytes += b.bytes();
  }
  if (product) {
    const int64_t wide = d.kind == HF_OPERATOR_GATED || d.kind == HF_OPERATOR_GATED_GRAD ? 2 * d.n : d.n;
    f.algorithmic_flops = (grad ? 4 : 2) * d.m * wide * d.k;
    if (op.p1.on) {
      f.tile_rows = op.p1.skinny ? 16 : op.p1.tile == 0 ? 256 : op.p1.tile == 1 ? 128 : 64;
      f.tile_cols = op.p1.skinny ? (op.p1.gated ? 32 : 16) : op.p1.tile == 0 ? 256 : 128;
      f.splits = op.p1.splits;
    }
  }
}

// ---- launches ------------------------------------------------------------

struct Call {
  const hf_operator *op;
  const void *p[HF_MAX_OPERATOR_BUFFERS];
  char *ws;
  hipStream_t stream;
  const void *in(int i) const { return i < 0 ? nullptr : p[i]; }
  void *out(int i) const { return i < 0 ? nullptr : const_cast<void *>(p[i]); }
  int64_t ld(int i) const { return i < 0 ? 0 : op->buf[i].ld; }
};

#define HF_TRY(x)                        \
  do {                                   \
    const hipError_t e_ = (x);           \
    if (e_ != hipSuccess) return e_;     \
  } while (0)

// The operand's address: the caller's, or its copy in the workspace.
hipError_t place(const Call &c, const Operand &o, const void *src, int64_t elem, const void **at) {
  *at = src;
  if (o.pack_at < 0 || o.rows == 0) return hipSuccess;
  void *dst = c.ws + o.pack_at;
  *at = dst;
  return launch_pack(src, o.src_ld * elem, dst, o.ld * elem, o.rows, o.src_cols * elem, c.stream);
}

ProductArgs args_of(const Call &c, const Product &p, const void *a, const void *b, int64_t elem, const Epilogue &e) {
  ProductArgs g{};
  g.dtype = c.op->d.dtype;
  g.tile = p.tile;
  g.splits = 1;
  if (!p.on) return g;
  g.a = a;
  g.b = b;
  g.lda = p.a.ld * elem;
  g.ldb = p.b.ld * elem;
  g.a_bytes = p.a.rows > 0 ? (p.a.rows - 1) * g.lda + p.a.cols * elem : 0;
  g.b_bytes = p.b.rows > 0 ? (p.b.rows - 1) * g.ldb + p.b.cols * elem : 0;
  g.b_half = p.gated ? p.n * g.ldb : 0;
  if (p.experts) {
    const int64_t rows = p.b.rows / p.experts;
    g.b_bytes = rows > 0 ? (rows - 1) * g.ldb + p.b.cols * elem : 0;
    g.b_expert = rows * g.ldb;
    g.offsets = (const int32_t *)c.in(c.op->i_offsets);
    g.experts = (int)p.experts;
  }
  if (c.op->d.flags & HF_OPERATOR_BLOCK_SCALES) {
    const int i = c.op->i_a_scale;
    g.a_scale = (const float *)c.in(i), g.lda_scale = c.ld(i);
    g.b_scale = (const float *)c.in(i + 1), g.ldb_scale = c.ld(i + 1);
    g.b_scale_half = (int)cdiv(p.n, kBlock);
  }
  g.m = (int)p.m;
  g.n = (int)p.n;
  g.k = (int)p.k;
  g.tiles_full = (int)p.tiles_full;
  g.part_rows = (int)p.part_rows;
  g.part_cols = (int)p.part_cols;
  g.splits = p.splits;
  g.k_tiles_per_split = p.per_split;
  g.partial = p.splits > 1 ? (float *)(c.ws + p.partial_at) : nullptr;
  g.ldp = p.ldp;
  g.e = e;
  return g;
}

hipError_t run_product(const Call &c, const Product &p, const void *a, const void *b, int64_t elem, const Epilogue &e,
                       int64_t from = 0) {
  if (!p.on) return hipSuccess;
  ProductArgs g = args_of(c, p, a, b, elem, e);
  if (g.a_scale) g.a_scale += from;  // the first of these rows
  if (p.experts) return launch_experts(g, c.stream);
  if (!p.skinny) return launch_product(g, c.stream);
  SkinnyArgs s{};
  s.p = g;
  s.waves = p.waves;
  s.blocks_per_split = p.per_split;
  return launch_skinny(s, c.stream);
}

hipError_t run_norm(const Call &c) {
  const hf_operator &op = *c.op;
  if (op.d.m == 0) return hipSuccess;
  NormArgs a{};
  a.x = c.in(0), a.ldx = c.ld(0);
  a.weight = c.in(1);
  a.residual = c.in(op.i_residual), a.ldr = c.ld(op.i_residual);
  a.y = c.out(op.n_params), a.ldy = c.ld(op.n_params);
  a.stream = c.out(op.i_stream), a.lds = c.ld(op.i_stream);
  a.scale = (float *)c.out(op.i_scale);
  a.rstd = (float *)c.out(op.i_rstd);
  a.rows = op.d.m;
  a.cols = (int)op.d.n;
  a.dtype = op.d.dtype, a.weight_dtype = op.d.weight_dtype, a.out_dtype = op.d.out_dtype;
  a.eps = (float)op.d.epsilon;
  a.root = (float)std::sqrt(op.d.epsilon);
  a.vec = op.vec;
  return launch_norm(a, c.stream);
}

hipError_t run_norm_grad(const Call &c) {
  const hf_operator &op = *c.op;
  NormGradArgs a{};
  a.dy = c.in(0), a.lddy = c.ld(0);
  a.h = c.in(1), a.ldh = c.ld(1);
  a.weight = c.in(2);
  a.rstd = (const float *)c.in(3);
  a.dstream = c.in(op.i_residual), a.ldds = c.ld(op.i_residual);
  a.dx = c.out(op.n_params), a.lddx = c.ld(op.n_params);
  a.dweight = (float *)c.out(op.n_params + 1);
  a.partial = (float *)(c.ws + op.sums_at);
  a.rows = op.d.m;
  a.cols = (int)op.d.n;
  a.groups = op.groups;
  a.dtype = op.d.dtype, a.weight_dtype = op.d.weight_dtype;
  a.vec = op.vec;
  return launch_norm_grad(a, c.stream);
}

hipError_t run_dropout(const Call &c) {
  const hf_operator &op = *c.op;
  if (op.d.m == 0 || op.d.n == 0) return hipSuccess;
  DropoutArgs a{};
  const int y = op.n_params;
  a.x = c.in(0), a.ldx = c.ld(0);
  a.state = (const int64_t *)c.in(1);
  a.residual = c.in(op.i_residual), a.ldr = c.ld(op.i_residual);
  a.y = c.out(y), a.ldy = c.ld(y);
  a.rows = op.d.m;
  a.cols = op.d.n;
  a.dtype = op.d.dtype;
  const double cut = std::nearbyint(op.d.probability * 65536.0);
  a.cut = (uint32_t)cut;
  a.scale = cut < 65536.0 ? (float)(65536.0 / (65536.0 - cut)) : 0.f;
  const auto dense = [&](int i) { return i < 0 || op.buf[i].rows <= 1 || op.buf[i].ld == op.buf[i].cols; };
  const auto on16 = [&](int i) { return i < 0 || aligned16(op.buf[i]); };
  if (dense(0) && dense(op.i_residual) && dense(y)) {
    a.cols *= a.rows;
    a.rows = 1;
    a.vec = true;
  } else {
    a.vec = op.d.n % 8 == 0 && on16(0) && on16(op.i_residual) && on16(y);
  }
  return launch_dropout(a, c.stream);
}

hipError_t run_product_forward(const Call &c) {
  const hf_operator &op = *c.op;
  const int64_t elem = op.buf[0].elem();
  if (!op.p1.on) return hipSuccess;
  Epilogue e{};
  const int d = op.n_params;
  e.d = c.out(d), e.ldd = c.ld(d);
  e.z = c.out(op.i_z), e.ldz = c.ld(op.i_z);
  e.bias = c.in(op.i_bias);
  e.residual = c.in(op.i_residual), e.ldr = c.ld(op.i_residual);
  if (op.i_a_scale >= 0 && !(op.d.flags & HF_OPERATOR_BLOCK_SCALES)) {
    e.a_scale = (const float *)c.in(op.i_a_scale);
    e.b_scale = (const float *)c.in(op.i_a_scale + 1);
  }
  e.out_dtype = op.d.out_dtype;
  e.act = op.d.activation;
  e.m = (int)op.d.m, e.n = (int)op.d.n;
  e.gated = op.p1.gated;
  e.vec = op.vec;
  const void *a, *b;
  Operand all = op.p1.a;
  all.rows = op.d.m;
  HF_TRY(place(c, all, c.in(0), elem, &a));
  HF_TRY(place(c, op.p1.b, c.in(1), elem, &b));
  e.m = (int)op.p1.m;
  HF_TRY(run_product(c, op.p1, a, b, elem, e));
  if (!op.p2.on) return hipSuccess;
  // the last rows: the same product from their first on
  const int64_t from = op.p1.m, out = op.buf[d].elem();
  a = (const char *)a + from * op.p1.a.ld * elem;
  e.m = (int)op.p2.m;
  e.d = (char *)e.d + from * e.ldd * out;
  if (e.z) e.z = (char *)e.z + from * e.ldz * out;
  if (e.residual) e.residual = (const char *)e.residual + from * e.ldr * out;
  if (e.a_scale) e.a_scale += from;
  return run_product(c, op.p2, a, b, elem, e, from);
}

hipError_t run_product_grad(const Call &c) {
  const hf_operator &op = *c.op;
  const bool gated = op.d.kind == HF_OPERATOR_GATED_GRAD;
  const void *dz = c.in(0);
  if (op.dz_at >= 0) dz = c.ws + op.dz_at;
  if (op.d.n > 0 && (op.dz_at >= 0 || op.i_dbias >= 0)) {
    ActGradArgs g{};
    g.dd = c.in(0), g.lddd = c.ld(0);
    g.z = c.in(op.i_z), g.ldz = c.ld(op.i_z);
    g.dz = op.dz_at >= 0 ? c.ws + op.dz_at : nullptr, g.lddz = op.lddz;
    g.partial = op.i_dbias >= 0 ? (float *)(c.ws + op.sums_at) : nullptr;
    g.m = op.d.m, g.n = (int)op.d.n, g.groups = op.groups;
    g.dtype = op.d.dtype, g.act = op.d.activation;
    g.gated = gated;
    g.vec = op.vec;
    HF_TRY(launch_act_grad(g, c.stream));
    if (op.i_dbias >= 0)
      HF_TRY(launch_column_fold(g.partial, op.groups, op.d.n, (float *)c.out(op.i_dbias), c.stream));
  }
  const void *a = c.in(1), *b = c.in(2);
  if (op.p2.on) HF_TRY(place(c, op.p2.b, c.in(1), 2, &a));
  if (op.p1.on) HF_TRY(place(c, op.p1.b, c.in(2), 2, &b));
  const auto plain = [&](int i, const Product &p) {
    Epilogue e{};
    e.d = c.out(i), e.ldd = c.ld(i);
    e.out_dtype = op.d.dtype;
    e.m = (int)p.m, e.n = (int)p.n;
    e.vec = op.buf[i].rows <= 1 || op.buf[i].ld % 8 == 0;
    return e;
  };
  const ProductArgs da = args_of(c, op.p1, dz, b, 2, plain(op.n_params, op.p1));
  ProductArgs db = args_of(c, op.p2, dz, a, 2, plain(op.n_params + 1, op.p2));
  if (!op.experts) return launch_gradient(da, db, c.stream);
  // a row's bytes: an expert's rows are counted on the GPU
  db.a_bytes = op.p2.a.cols * 2;
  db.b_bytes = op.p2.b.cols * 2;
  return launch_experts_gradient(da, db, c.stream);
}

hipError_t run_sort(const Call &c) {
  const hf_operator &op = *c.op;
  SortArgs a{};
  const int r = op.n_params;
  a.expert = (const int32_t *)c.in(0), a.ld_expert = c.ld(0);
  a.place = (int32_t *)c.out(r), a.ld_place = c.ld(r);
  a.order = (int32_t *)c.out(r + 1);
  a.offsets = (int32_t *)c.out(r + 2);
  a.pairs = (int)(op.d.m * op.top_k);
  a.top_k = (int)op.top_k;
  a.experts = (int)op.experts;
  sort_chunks(a.pairs, &a.chunks, &a.per_chunk);
  if (a.chunks > 1) a.counts = (int32_t *)(c.ws + op.sums_at);
  return launch_sort(a, c.stream);
}

hipError_t run_dispatch(const Call &c) {
  const hf_operator &op = *c.op;
  // rows of no columns still have their scale, where it is a row's
  if (op.d.m == 0 || (op.d.n == 0 && op.i_a_scale < 0)) return hipSuccess;
  DispatchArgs a{};
  const int y = op.n_params;
  const int64_t elem = op.buf[0].elem();
  a.x = c.in(0), a.ldx = c.ld(0) * elem;
  a.y = c.out(y), a.ldy = c.ld(y) * elem;
  a.place = (const int32_t *)c.in(1), a.ld_place = c.ld(1);
  if (op.i_a_scale >= 0) {
    a.x_scale = (const float *)c.in(op.i_a_scale), a.ldx_scale = c.ld(op.i_a_scale);
    a.y_scale = (float *)c.out(op.i_scale), a.ldy_scale = c.ld(op.i_scale);
    a.blocks = (int)op.buf[op.i_a_scale].rows;
  }
  a.tokens = op.d.m;
  a.bytes = op.d.n * elem;
  a.aligned = aligned16(op.buf[y]);
  a.top_k = (int)op.top_k;
  a.pairs = (int)(op.d.m * op.top_k);
  return launch_dispatch(a, c.stream);
}

hipError_t run_combine(const Call &c) {
  const hf_operator &op = *c.op;
  const bool grad = op.d.kind == HF_OPERATOR_EXPERT_COMBINE_GRAD;
  if (op.d.m == 0) return hipSuccess;
  CombineArgs a{};
  const int y = grad ? 1 : 0, r = op.n_params;
  a.y = c.in(y), a.ldy = c.ld(y);
  a.place = (const int32_t *)c.in(y + 1), a.ld_place = c.ld(y + 1);
  a.weight = (const float *)c.in(op.i_weight), a.ld_weight = c.ld(op.i_weight);
  a.residual = c.in(op.i_residual), a.ldr = c.ld(op.i_residual);
  a.tokens = op.d.m;
  a.cols = (int)op.d.n;
  a.top_k = (int)op.top_k;
  a.pairs = (int)(op.d.m * op.top_k);
  a.dtype = op.d.dtype;
  a.vec = op.vec;
  if (grad) {
    a.dd = c.in(0), a.ldd = c.ld(0);
    a.dy = c.out(r), a.lddy = c.ld(r);
    a.dweight = (float *)c.out(r + 1), a.ld_dweight = c.ld(r + 1);
    return launch_combine_grad(a, c.stream);
  }
  if (op.d.n == 0) return hipSuccess;
  a.d = c.out(r), a.ldd = c.ld(r);
  return launch_combine(a, c.stream);
}

hipError_t run_quantize(const Call &c) {
  const hf_operator &op = *c.op;
  if (op.d.m == 0 || op.d.n == 0) return hipSuccess;
  QuantizeArgs a{};
  a.x = c.in(0), a.ldx = c.ld(0);
  a.y = (uint8_t *)c.out(1), a.ldy = c.ld(1);
  a.scale = (float *)c.out(2), a.ld_scale = c.ld(2);
  a.rows = op.d.m;
  a.cols = (int)op.d.n;
  a.dtype = op.d.dtype;
  a.vec = op.vec;
  return launch_quantize(a, c.stream);
}

// Two buffers that share no element.  Column windows of one array (equal row
// strides in bytes, windows that do not meet within a row) are apart though
// their extents cross.
bool apart(const Buffer &x, const void *px, const Buffer &y, const void *py) {
  const uintptr_t x0 = (uintptr_t)px, x1 = x0 + (uintptr_t)x.extent(), y0 = (uintptr_t)py,
                  y1 = y0 + (uintptr_t)y.extent();
  if (x1 <= y0 || y1 <= x0) return true;
  const uintptr_t s = (uintptr_t)(x.ld * x.elem());
  if (x.rows <= 1 || y.rows <= 1 || s != (uintptr_t)(y.ld * y.elem())) return false;
  const uintptr_t off = y0 >= x0 ? (y0 - x0) % s : (s - (x0 - y0) % s) % s;
  return off >= (uintptr_t)(x.cols * x.elem()) && off + (uintptr_t)(y.cols * y.elem()) <= s;
}

hf_status launch_operator(const hf_operator *op, const void *const *params, int32_t n_params, void *const *results,
                          int32_t n_results, void *workspace, bool scratch, void *stream) {
  const auto bad = [](const std::string &m) {
    set_error(m);
    return HF_ERR_INVALID;
  };
  if (!op) return bad("NULL handle");
  if (op->plan_only) return bad("the handle was created plan-only or compile-only");
  if (n_params != op->n_params || n_results != op->n_results || (n_params > 0 && !params) ||
      (n_results > 0 && !results))
    return bad("expected " + std::to_string(op->n_params) + " parameter and " + std::to_string(op->n_results) +
               " result pointers, got " + std::to_string(n_params) + " and " + std::to_string(n_results));
  int dev = -1;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return hip_error(e, "hipGetDevice");
  if (dev != op->device) return bad("the current device differs from the device the operator was created on");
  Call c;
  c.op = op;
  c.stream = (hipStream_t)stream;
  const int all = n_params + n_results;
  for (int i = 0; i < all; ++i) {
    const void *p = i < n_params ? params[i] : results[i - n_params];
    c.p[i] = p;
    const Buffer &b = op->buf[i];
    if (b.empty()) continue;
    if (!p || ((uintptr_t)p & 15)) return bad(b.name + " must be a non-NULL, 16-byte aligned device pointer");
    if (!check_buffer(p, (size_t)b.extent(), op->device, "operator", b.name)) return HF_ERR_INVALID;
  }
  for (int i = n_params; i < all; ++i)
    for (int j = 0; j < i; ++j)
      if (!op->buf[i].empty() && !op->buf[j].empty() && !apart(op->buf[i], c.p[i], op->buf[j], c.p[j]))
        return bad(op->buf[i].name + " overlaps " + op->buf[j].name);
  if (scratch) {
    if (op->ws > (int64_t)HF_SCRATCH_BYTES) {
      set_error("this operator needs " + std::to_string(op->ws) + " bytes of workspace, more than the " +
                std::to_string((long long)HF_SCRATCH_BYTES) +
                " bytes of the library's scratch memory: launch it with hf_operator_launch and a workspace");
      return HF_ERR_UNSUPPORTED;
    }
    workspace = scratch_address(op->device);
    if (op->ws > 0 && !workspace) return bad("no scratch memory was set up on the operator's device");
  } else if (op->ws > 0) {
    const uintptr_t w0 = (uintptr_t)workspace, w1 = w0 + (uintptr_t)op->ws;
    if (!workspace || (w0 & 15))
      return bad("this operator needs a workspace of " + std::to_string(op->ws) +
                 " bytes: a non-NULL, 16-byte aligned device pointer");
    if (!check_buffer(workspace, (size_t)op->ws, op->device, "operator", "the workspace")) return HF_ERR_INVALID;
    for (int i = 0; i < all; ++i) {
      const uintptr_t p0 = (uintptr_t)c.p[i], p1 = p0 + (uintptr_t)op->buf[i].extent();
      if (!op->buf[i].empty() && p0 < w1 && w0 < p1) return bad("the workspace overlaps " + op->buf[i].name);
    }
  }
  c.ws = (char *)workspace;
  switch (op->d.kind) {
    case HF_OPERATOR_RMS_NORM: e = run_norm(c); break;
    case HF_OPERATOR_RMS_NORM_GRAD: e = run_norm_grad(c); break;
    case HF_OPERATOR_DROPOUT: e = run_dropout(c); break;
    case HF_OPERATOR_MATMUL: case HF_OPERATOR_GATED: e = run_product_forward(c); break;
    case HF_OPERATOR_EXPERT_SORT: e = run_sort(c); break;
    case HF_OPERATOR_EXPERT_DISPATCH: e = run_dispatch(c); break;
    case HF_OPERATOR_EXPERT_COMBINE: case HF_OPERATOR_EXPERT_COMBINE_GRAD: e = run_combine(c); break;
    case HF_OPERATOR_BLOCK_QUANTIZE: e = run_quantize(c); break;
    default: e = run_product_grad(c);
  }
  return e == hipSuccess ? HF_OK : hip_error(e, kind_name(op->d.kind));
}

// No exception crosses the C boundary.
template <class F>
hf_status guarded(F f) {
  try {
    return f();
  } catch (const Error &e) {
    set_error(e.msg);
    return e.status;
  } catch (const std::bad_alloc &) {
    set_error("out of host memory");
    return HF_ERR_NOMEM;
  } catch (const std::exception &e) {
    set_error(std::string("internal error: ") + e.what());
    return HF_ERR_INVALID;
  } catch (...) {
    set_error("internal error");
    return HF_ERR_INVALID;
  }
}

// The current device, if it is one that the kernels are compiled for (asked
// once a device: the query takes longer than a launch).
hf_status current_device(int *device) {
  hipError_t e = hipGetDevice(device);
  if (e != hipSuccess) return hip_error(e, "hipGetDevice");
  static std::mutex mu;
  static signed char known[64];
  if (*device < 0 || *device >= 64) {
    set_error("device number out of range");
    return HF_ERR_UNSUPPORTED;
  }
  std::lock_guard<std::mutex> lk(mu);
  if (known[*device]) return HF_OK;
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, *device);
  if (e != hipSuccess) return hip_error(e, "hipGetDeviceProperties");
  if (std::strncmp(prop.gcnArchName, "gfx950", 6) != 0) {
    set_error(std::string("this library targets gfx950 (MI355X); current device is ") + prop.gcnArchName);
    return HF_ERR_UNSUPPORTED;
  }
  std::string err;
  const hf_status st = scratch_prepare(*device, &err);
  if (st != HF_OK) {
    set_error(err);
    return st;
  }
  known[*device] = 1;
  return HF_OK;
}

}  // namespace
}  // namespace hf

namespace hf {
namespace {

// desc as hf_operator_create takes it, or the whole extended one
hf_status create(const hf_operator_desc *desc, const hf_operator_extended_desc *extended, uint32_t flags, hf_operator **out) {
  return guarded([&]() -> hf_status {
    set_error("");
    if (!out) invalid("out is NULL");
    *out = nullptr;
    if (!desc) invalid("desc is NULL");
    if (desc->abi_version != HF_ABI_VERSION)
      invalid("abi_version " + std::to_string(desc->abi_version) + ", expected " + std::to_string(HF_ABI_VERSION));
    if (flags & ~(HF_CREATE_PLAN_ONLY | HF_CREATE_COMPILE_ONLY)) invalid("unknown create flags");
    std::unique_ptr<hf_operator> op(new hf_operator);
    op->d = *desc;
    if (extended) {
      op->experts = extended->experts;
      op->top_k = extended->top_k;
    }
    op->plan_only = flags != 0;
    make_plan(*op, extended != nullptr);
    if (!op->plan_only) {
      const hf_status st = current_device(&op->device);
      if (st != HF_OK) return st;
    }
    *out = op.release();
    return HF_OK;
  });
}

}  // namespace
}  // namespace hf

extern "C" {

hf_status hf_operator_create(const hf_operator_desc *desc, uint32_t flags, hf_operator **out) {
  return hf::create(desc, nullptr, flags, out);
}

hf_status hf_operator_create_extended(const hf_operator_extended_desc *desc, uint32_t flags, hf_operator **out) {
  return hf::create(desc ? &desc->op : nullptr, desc, flags, out);
}

hf_status hf_operator_plan(const hf_operator *op, hf_operator_info *info) {
  return hf::guarded([&]() -> hf_status {
    if (!op || !info) hf::invalid("NULL argument");
    *info = op->info;
    return HF_OK;
  });
}

hf_status hf_operator_launch(const hf_operator *op, const void *const *params, int32_t n_params, void *const *results,
                             int32_t n_results, void *workspace, void *stream) {
  return hf::guarded([&]() -> hf_status {
    return hf::launch_operator(op, params, n_params, results, n_results, workspace, false, stream);
  });
}

hf_status hf_operator_launch_noalloc(const hf_operator *op, const void *const *params, int32_t n_params,
                                     void *const *results, int32_t n_results, void *stream) {
  return hf::guarded([&]() -> hf_status {
    return hf::launch_operator(op, params, n_params, results, n_results, nullptr, true, stream);
  });
}

hf_status hf_operator_destroy(hf_operator *op) {
  delete op;
  return HF_OK;
}

}  // extern "C"
