// operators.h -- between the operators' C ABI (operators.cpp) and their
// kernels (*.hip): launch arguments and launchers.  Plain C++.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "hlofusion.h"

namespace hf {

// ---- row-wise operators (rows.hip) -------------------------------------
struct NormArgs {
  const void *x, *residual, *weight;
  void *y, *stream;
  float *scale, *rstd;
  int64_t ldx, ldr, ldy, lds;  // elements
  int64_t rows;
  int32_t cols;
  int32_t dtype, weight_dtype, out_dtype;
  float eps, root;  // epsilon and its square root, which may be in f32's range alone
  bool vec;  // every row starts on 16 bytes and cols is a multiple of 8
};
hipError_t launch_norm(const NormArgs &a, hipStream_t s);

struct NormGradArgs {
  const void *dy, *h, *weight, *dstream;
  const float *rstd;
  void *dx;
  float *dweight, *partial;    // partial: [groups][cols]
  int64_t lddy, ldh, ldds, lddx;
  int64_t rows;
  int32_t cols, groups;
  int32_t dtype, weight_dtype;
  bool vec;
};
hipError_t launch_norm_grad(const NormGradArgs &a, hipStream_t s);
// The number of row groups whose partial weight gradients are kept apart.
int norm_grad_groups(int64_t rows, int64_t cols);

struct DropoutArgs {
  const void *x, *residual;
  const int64_t *state;
  void *y;
  int64_t ldx, ldr, ldy;
  int64_t rows, cols;
  int32_t dtype;
  uint32_t cut;  // an element is kept if its 16 bits are >= cut
  float scale;
  bool vec;      // 8 elements of one row share a generator call and 16-byte accesses
};
hipError_t launch_dropout(const DropoutArgs &a, hipStream_t s);

// ---- rows by expert (experts.hip) ----------------------------------------
struct SortArgs {
  const int32_t *expert;
  int32_t *place, *order, *offsets;
  int32_t *counts;               // [chunks][experts], chunks > 1
  int64_t ld_expert, ld_place;
  int32_t pairs, top_k, experts;
  int32_t chunks, per_chunk;     // pairs of a workgroup
};
hipError_t launch_sort(const SortArgs &a, hipStream_t s);
// The workgroups of a sort and the pairs of each.
void sort_chunks(int64_t pairs, int32_t *chunks, int32_t *per_chunk);

struct DispatchArgs {
  const void *x;
  void *y;
  const int32_t *place;
  const float *x_scale;          // [blocks][tokens] or NULL
  float *y_scale;
  int64_t ldx, ldy;              // bytes
  int64_t ld_place, ldx_scale, ldy_scale;
  int64_t tokens, bytes;         // of a row
  int32_t top_k, pairs, blocks;
  bool aligned;                  // y's rows start on 16 bytes
};
hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t s);

struct CombineArgs {
  const void *y, *residual, *dd;
  void *d, *dy;
  const int32_t *place;
  const float *weight;           // NULL: ones
  float *dweight;
  int64_t ldy, ldr, ldd, lddy, ld_place, ld_weight, ld_dweight;
  int64_t tokens;
  int32_t cols, top_k, pairs;
  int32_t dtype;
  bool vec;                      // every row starts on 16 bytes and cols is a multiple of 8
};
hipError_t launch_combine(const CombineArgs &a, hipStream_t s);
hipError_t launch_combine_grad(const CombineArgs &a, hipStream_t s);  // ldd: dd's rows

struct QuantizeArgs {
  const void *x;
  uint8_t *y;
  float *scale;
  int64_t ldx, ldy, ld_scale;
  int64_t rows;
  int32_t cols, dtype;
  bool vec;                      // every row starts on 16 (y: 8) bytes and cols is a multiple of 8
};
hipError_t launch_quantize(const QuantizeArgs &a, hipStream_t s);

// out[c] = sum of partial[g][c] over g, in a fixed order.
hipError_t launch_column_fold(const float *partial, int groups, int64_t cols, float *out, hipStream_t s);

// dz = dd * act'(z) (gated: both halves), rounded to dtype, rows of lddz
// elements whose tail past the columns is zero; the column sums' partials if
// wanted.  dz may be NULL (sums only).
struct ActGradArgs {
  const void *dd, *z;
  void *dz;
  float *partial;              // [groups][n] or NULL
  int64_t lddd, ldz, lddz;
  int64_t m;
  int32_t n, groups;
  int32_t dtype, act;
  bool gated, vec;
};
hipError_t launch_act_grad(const ActGradArgs &a, hipStream_t s);
int act_grad_groups(int64_t m, int64_t n);

// dst = src with the tail of every row zero.  In bytes; dst and ld_dst are
// multiples of 16.
hipError_t launch_pack(const void *src, int64_t ld_src, void *dst, int64_t ld_dst, int64_t rows, int64_t bytes,
                       hipStream_t s);

// ---- products (product.hip, skinny.hip) ----------------------------------
// What happens to the sums on their way out (product_epilogue.h): eight
// consecutive ones of a row at a time, four in the skinny product.
struct Epilogue {
  void *d, *z;
  const void *bias, *residual;
  const float *a_scale, *b_scale;
  int64_t ldd, ldz, ldr;
  int32_t out_dtype, act;
  int32_t m, n;       // the extents of d
  bool gated;         // columns n .. 2n-1 of the product are the up half
  bool vec;           // whole groups of d, z and residual are aligned and go in one access
};

struct ProductArgs {
  const void *a, *b;
  int64_t lda, ldb;          // bytes
  int64_t a_bytes, b_bytes;  // from the first to past the last element
  int64_t b_half;            // gated: bytes from a gate row to its up row
  int32_t m, n, k;           // n: columns of d (gated: of one half); k: elements
  int32_t dtype;
  int32_t tile;              // 0: 256 x 256, 1: 128 x 128 (columns of the product), 2: strips, m <= 64
  int32_t tiles_full;        // tiles 0 and 1: so many are one workgroup's, the others `splits` workgroups'
  int32_t splits, k_tiles_per_split;
  // splits > 1: [splits][shared tiles][part_rows][part_cols], the up half's
  // columns after the gate's, or (strips, skinny, by expert) [splits][m][ldp]
  // (db: [splits][experts * m][ldp]); s8: 32-bit integers
  float *partial;
  int32_t part_rows, part_cols;
  int64_t ldp;
  // e4m3 with block scales (else NULL): a_scale [blocks][rows], b_scale [blocks
  // of 128 rows][blocks], in elements; b_scale_half: blocks of rows of n, from a
  // gate block to its up block
  const float *a_scale, *b_scale;
  int64_t lda_scale, ldb_scale;
  int32_t b_scale_half;
  // by expert (else NULL): m rows of a and d, sorted; b_bytes is one weight's,
  // b_expert bytes lie between two
  const int32_t *offsets;
  int32_t experts;
  int32_t piece;             // in a workgroup: which of the splits
  int64_t b_expert;
  Epilogue e;
};
// What a launch of 256 or 512 threads a workgroup takes in tiles by expert.
int64_t expert_tiles(int64_t m, int64_t experts, int64_t size, int64_t per);
hipError_t launch_experts(const ProductArgs &a, hipStream_t s);
// Adds the splits' sums of a.e.m rows (with offsets, of those that are an
// expert's) and runs the epilogue.
hipError_t launch_experts_fold(const ProductArgs &a, const int32_t *offsets, hipStream_t s);
// The gradient by expert: da as above with b's rows as the contraction; db's
// contraction runs over an expert's rows, its a_bytes and b_bytes are a row's,
// its rows m and its results an expert's.
hipError_t launch_experts_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s);
hipError_t launch_product(const ProductArgs &a, hipStream_t s);
// da = dz b (the contraction runs over b's rows) and db = dz^T a (over both
// operands' rows), tiles of one size; one of them may be empty (m or n 0,
// tiles_full 0, splits 1).
hipError_t launch_gradient(const ProductArgs &da, const ProductArgs &db, hipStream_t s);
// Which e4m3 products go through f16 (StepF8Wide).
constexpr bool f8_wide(int out_dtype, int64_t k) { return out_dtype == HF_F32 || k <= 128; }

struct SkinnyArgs {
  ProductArgs p;             // splits: workgroups over k
  int32_t waves;             // of a workgroup: 8 or 16
  int32_t blocks_per_split;  // blocks of 512 contraction bytes
};

hipError_t launch_skinny(const SkinnyArgs &a, hipStream_t s);

// Sum the partials of strips or of skinny products and run the epilogue.
hipError_t launch_product_fold(const ProductArgs &a, hipStream_t s);

}  // namespace hf
