// experts.hip -- rows by expert: (token, choice) pairs sorted by expert, the
// tokens' rows sent to the sorted places and summed up again, and the gradient
// of that sum.
#include "product_epilogue.h"

namespace hf {
namespace {

// ---- sort ----------------------------------------------------------------
// A stable counting sort.  Every wave has a contiguous run of pairs and counts
// its experts in LDS; the counts before a wave's, over the experts, the
// chunks and the waves, are where its first pair of an expert goes.  Then it
// goes through its run again, 64 pairs at a time: pairs of the same expert
// find each other by a ballot for each bit of the expert's number, and their
// rank is the number of them in lower lanes.  No order depends on time.
//
// One workgroup does it all for up to 8192 pairs (192 pairs of 128 experts
// 3.4 us, a launch and a few dependent steps); beyond that each chunk of pairs
// has a workgroup, and a first launch counts by chunk (65528 pairs of 64
// experts 4.6 + 6.2 us; every workgroup of the second adds up the counts of all
// chunks by itself, which a third launch would cost more than).
constexpr int kSortWaves = 16, kSortMost = 1024;  // waves; experts

__device__ __forceinline__ int expert_of(const SortArgs &a, int p) {
  const int e = a.ld_expert == a.top_k ? a.expert[p] : a.expert[(int64_t)(p / a.top_k) * a.ld_expert + p % a.top_k];
  return (uint32_t)e < (uint32_t)a.experts ? e : -1;
}

// This wave's counts of its run, in `count` [experts].
__device__ __forceinline__ void count_run(const SortArgs &a, int from, int to, int *count) {
  for (int p = from + (int)(threadIdx.x % 64); p < to; p += 64) {
    const int e = expert_of(a, p);
    if (e >= 0) atomicAdd(count + e, 1);
  }
}

struct Run {
  int from, to;
  __device__ __forceinline__ explicit Run(const SortArgs &a) {
    const int w = __builtin_amdgcn_readfirstlane(threadIdx.x / 64), per = a.per_chunk / kSortWaves;
    const int64_t at = (int64_t)blockIdx.x * a.per_chunk + (int64_t)w * per;
    from = (int)min(at, (int64_t)a.pairs);
    to = (int)min(at + per, (int64_t)a.pairs);
  }
};

__global__ __launch_bounds__(kSortWaves * 64) void sort_count_kernel(SortArgs a) {
  __shared__ int count[kSortMost];
  for (int e = threadIdx.x; e < a.experts; e += kSortWaves * 64) count[e] = 0;
  __syncthreads();
  const Run r(a);
  count_run(a, r.from, r.to, count);
  __syncthreads();
  for (int e = threadIdx.x; e < a.experts; e += kSortWaves * 64) a.counts[(int64_t)blockIdx.x * a.experts + e] = count[e];
}

__global__ __launch_bounds__(kSortWaves * 64) void sort_kernel(SortArgs a) {
  __shared__ int next[kSortWaves * kSortMost];  // [wave][experts]: counts, then the next free place
  __shared__ int sums[kSortWaves];
  const int t = threadIdx.x, l = t % 64, w = __builtin_amdgcn_readfirstlane(t / 64), experts = a.experts;
  for (int i = t; i < kSortWaves * experts; i += kSortWaves * 64) next[i] = 0;
  __syncthreads();
  const Run r(a);
  count_run(a, r.from, r.to, next + w * experts);
  __syncthreads();
  // an expert a thread: all its pairs, and those of the chunks before this one
  int all = 0, before = 0;
  if (t < experts) {
    if (a.chunks == 1) {
#pragma unroll
      for (int i = 0; i < kSortWaves; ++i) all += next[i * experts + t];
    } else {
#pragma unroll 8
      for (int c = 0; c < a.chunks; ++c) {
        const int n = a.counts[(int64_t)c * experts + t];
        before += c < (int)blockIdx.x ? n : 0;
        all += n;
      }
    }
  }
  int sum = all;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(sum, d);
    sum += l >= d ? o : 0;
  }
  if (l == 63) sums[w] = sum;
  __syncthreads();
  int first = sum - all, total = 0;
#pragma unroll
  for (int i = 0; i < kSortWaves; ++i) {
    const int n = sums[i];
    first += i < w ? n : 0;
    total += n;
  }
  if (t < experts) {
    if (blockIdx.x == 0) a.offsets[t] = first;
    int at = first + before;
#pragma unroll
    for (int i = 0; i < kSortWaves; ++i) {
      const int n = next[i * experts + t];
      next[i * experts + t] = at;
      at += n;
    }
  }
  if (blockIdx.x == 0 && t == 0) a.offsets[experts] = total;
  __syncthreads();
  volatile int *mine = next + w * experts;
  const int bits = 32 - __builtin_clz(experts);
  for (int from = r.from; from < r.to; from += 64) {
    const int p = from + l;
    const int e = p < r.to ? expert_of(a, p) : -1;
    uint64_t same = __ballot(e >= 0);
    for (int b = 0; b < bits; ++b) {
      const bool set = (e >> b) & 1;
      const uint64_t has = __ballot(set);
      same &= set ? has : ~has;
    }
    int place = -1;
    if (e >= 0) place = mine[e] + __popcll(same & ((uint64_t(1) << l) - 1));
    // the places are read before the group's first lane moves them on
    __builtin_amdgcn_wave_barrier();
    if (e >= 0 && __builtin_ctzll(same) == l) mine[e] = place + __popcll(same);
    __builtin_amdgcn_wave_barrier();
    if (p < r.to) {
      a.place[a.ld_place == a.top_k ? p : (int64_t)(p / a.top_k) * a.ld_place + p % a.top_k] = place;
      if (place >= 0) a.order[place] = p;
    }
  }
  // the rows past the last have no pair
  const int64_t chunk = (int64_t)blockIdx.x * a.per_chunk, end = min(chunk + a.per_chunk, (int64_t)a.pairs);
  for (int64_t i = max(chunk, (int64_t)total) + t; i < end; i += kSortWaves * 64) a.order[i] = -1;
}

// ---- dispatch --------------------------------------------------------------
// y[place[t, j]] = x[t], in bytes: a workgroup takes 4 KB of a token's row,
// reads them once and stores them top_k times, in unaligned accesses of 16
// bytes if need be, past the caches where rows are aligned (8191 x 8 rows of
// 4096 bytes, half of them another rank's, with block scales: 31 us, 174 MB,
// 5.6 TB/s; through the caches 45).  Taken by token and not by sorted row, a
// row is read once however many experts it goes to.
// Shorter rows share a workgroup, 2^shift threads each.
constexpr int kPiece = 4096;
template <bool SHORT>
__global__ __launch_bounds__(256) void dispatch_kernel(DispatchArgs a, int64_t scale_groups, int shift) {
  int64_t id = block_number<256>(blockIdx.x, blockIdx.y);
  if (id < scale_groups) {
    // scales: 64 tokens a workgroup, so that their lines are read whole, and
    // four blocks, one a wave
    const int64_t fours = (a.blocks + 3) / 4, group = id / fours, token = group * 64 + threadIdx.x % 64;
    const int64_t b = (id - group * fours) * 4 + threadIdx.x / 64;
    if (token >= a.tokens || b >= a.blocks) return;
    const float scale = a.x_scale[b * a.ldx_scale + token];
    const int32_t *place = a.place + token * a.ld_place;
#pragma unroll 8
    for (int j = 0; j < a.top_k; ++j) {
      const int p = place[j];
      if ((uint32_t)p < (uint32_t)a.pairs) a.y_scale[b * a.ldy_scale + p] = scale;
    }
    return;
  }
  id -= scale_groups;
  const int64_t pieces = SHORT ? 1 : (a.bytes + kPiece - 1) / kPiece;
  const int64_t token = SHORT ? (id << (8 - shift)) + (threadIdx.x >> shift) : id / pieces;
  if (token >= a.tokens) return;
  const int64_t c = SHORT ? (threadIdx.x & ((1 << shift) - 1)) * 16 : (id - token * pieces) * kPiece + threadIdx.x * 16;
  if (c >= a.bytes) return;
  const int left = a.bytes - c < 16 ? (int)(a.bytes - c) : 16;
  const char *x = (const char *)a.x + token * a.ldx + c;
  char *y = (char *)a.y + c;
  const int32_t *place = a.place + token * a.ld_place;
  if (left == 16) {
    u32x4 v;
    __builtin_memcpy(&v, x, 16);
#pragma unroll 8
    for (int j = 0; j < a.top_k; ++j) {
      const int p = place[j];
      if ((uint32_t)p >= (uint32_t)a.pairs) continue;
      if (a.aligned)
        __builtin_nontemporal_store(v, (u32x4 *)(y + p * a.ldy));
      else
        __builtin_memcpy(y + p * a.ldy, &v, 16);
    }
  } else {
    for (int j = 0; j < a.top_k; ++j) {
      const int p = place[j];
      if ((uint32_t)p >= (uint32_t)a.pairs) continue;
      for (int i = 0; i < left; ++i) y[p * a.ldy + i] = x[i];
    }
  }
}

// Threads of a short row: the least power of two that is enough.
int threads_shift(int64_t threads) {
  int s = 0;
  while ((int64_t(1) << s) < threads) ++s;
  return s;
}

// ---- combine ---------------------------------------------------------------
// d[t] = sum_j weight[t, j] y[place[t, j]] + residual[t]: a thread has eight
// columns of a token and asks for up to eight rows before it adds the first.
// Short rows share a workgroup as in the dispatch.  Bound by memory (4099 x 8
// rows of 4096 bf16 and a residual: 61 us, 336 MB, 5.5 TB/s; a single token's
// 8 rows 3.9 us, a launch and two dependent loads).
// Sums are in f32, in the order of j, rounded once.
constexpr int kAtOnce = 8;

template <class E, bool SHORT>
__global__ __launch_bounds__(256) void combine_kernel(CombineArgs a, int shift) {
  const int pieces = SHORT ? 1 : (a.cols + 2047) / 2048;
  const int64_t id = block_number<256>(blockIdx.x, blockIdx.y);
  const int64_t token = SHORT ? (id << (8 - shift)) + (threadIdx.x >> shift) : id / pieces;
  if (token >= a.tokens) return;
  const int c = SHORT ? (threadIdx.x & ((1 << shift) - 1)) * 8 : (int)(id - token * pieces) * 2048 + threadIdx.x * 8;
  const int left = a.cols - c;
  if (left <= 0) return;
  const bool vec = a.vec && left >= 8;
  const int32_t *place = a.place + token * a.ld_place;
  const float *weight = a.weight ? a.weight + token * a.ld_weight : nullptr;
  float sum[8], add[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] = add[i] = 0.f;
  if (a.residual) get_once<E>(a.residual, token * a.ldr + c, left, vec, add);
  for (int j0 = 0; j0 < a.top_k; j0 += kAtOnce) {
    float v[kAtOnce][8], w[kAtOnce];
    int p[kAtOnce];
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      p[j] = j0 + j < a.top_k ? place[j0 + j] : -1;
      w[j] = weight && j0 + j < a.top_k ? weight[j0 + j] : 1.f;
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[j][i] = 0.f;
      if ((uint32_t)p[j] < (uint32_t)a.pairs) get_once<E>(a.y, p[j] * a.ldy + c, left, vec, v[j]);
    }
#pragma unroll
    for (int j = 0; j < kAtOnce; ++j) {
      if ((uint32_t)p[j] >= (uint32_t)a.pairs) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) sum[i] = __builtin_fmaf(w[j], v[j][i], sum[i]);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) sum[i] += add[i];
  put<E, 8>(a.d, token * a.ldd + c, left, vec, sum);
}

// dy[place[t, j]] = weight[t, j] dd[t], dweight[t, j] = <dd[t], y[place[t, j]]>:
// T threads a token, which go through its columns once for every AT choices.
// With 8 elements a thread all loads of a token are in flight before the first
// is used: 8192 x 4 rows of 4096 bf16 take 119 us (604 MB, 5.1 TB/s); with half
// as many threads, twice around, and registers for 8 choices 159 where this form
// took 124, both through the caches.
template <class E, int T, int AT>
__global__ __launch_bounds__(T == 64 ? 256 : T) void combine_grad_kernel(CombineArgs a) {
  __shared__ float part[T == 64 ? 1 : AT][T / 64];
  constexpr int PER = T == 64 ? 4 : 1;
  const int64_t token = block_number<T == 64 ? 256 : T>(blockIdx.x, blockIdx.y) * PER + threadIdx.x / T;
  if (token >= a.tokens) return;  // whole waves, and no barrier follows where PER > 1
  const int t = threadIdx.x % T;
  const int32_t *place = a.place + token * a.ld_place;
  const float *weight = a.weight + token * a.ld_weight;
  for (int j0 = 0; j0 < a.top_k; j0 += AT) {
    float w[AT], dot[AT];
    int p[AT];
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      p[j] = j0 + j < a.top_k ? place[j0 + j] : -1;
      w[j] = j0 + j < a.top_k ? weight[j0 + j] : 0.f;
      dot[j] = 0.f;
    }
    for (int c = t * 8; c < a.cols; c += T * 8) {
      const int left = a.cols - c;
      const bool vec = a.vec && left >= 8;
      float g[8], v[AT][8];
      get<E, 8>(a.dd, token * a.ldd + c, left, vec, g);
#pragma unroll
      for (int j = 0; j < AT; ++j)
        if ((uint32_t)p[j] < (uint32_t)a.pairs) get_once<E>(a.y, p[j] * a.ldy + c, left, vec, v[j]);
#pragma unroll
      for (int j = 0; j < AT; ++j) {
        if ((uint32_t)p[j] >= (uint32_t)a.pairs) continue;
        float o[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          dot[j] = __builtin_fmaf(g[i], v[j][i], dot[j]);
          o[i] = w[j] * g[i];
        }
        put<E, 8>(a.dy, p[j] * a.lddy + c, left, vec, o);
      }
    }
    if (T != 64) __syncthreads();  // the sums of the choices before are read
#pragma unroll
    for (int j = 0; j < AT; ++j) {
      const float s = wave_sum(dot[j]);
      if (T == 64) {
        if (t == 0 && j0 + j < a.top_k) a.dweight[token * a.ld_dweight + j0 + j] = s;
      } else if (threadIdx.x % 64 == 0) {
        part[j][threadIdx.x / 64] = s;
      }
    }
    if (T != 64) {
      __syncthreads();
      if (t < AT && j0 + t < a.top_k) {
        float s = part[t][0];
#pragma unroll
        for (int i = 1; i < T / 64; ++i) s += part[t][i];
        a.dweight[token * a.ld_dweight + j0 + t] = s;
      }
    }
  }
}

template <class E>
hipError_t combine_go(const CombineArgs &a, hipStream_t s) {
  if (a.cols <= 1024) {
    const int shift = threads_shift((a.cols + 7) / 8), per = 256 >> shift;
    return launch(combine_kernel<E, true>, grid_of<256>((a.tokens + per - 1) / per), 256, s, a, shift);
  }
  return launch(combine_kernel<E, false>, grid_of<256>(a.tokens * ((a.cols + 2047) / 2048)), 256, s, a, 8);
}

template <class E, int AT>
hipError_t combine_grad_go(const CombineArgs &a, hipStream_t s) {
  if (a.cols <= 512) return launch(combine_grad_kernel<E, 64, AT>, grid_of<256>((a.tokens + 3) / 4), 256, s, a);
  if (a.cols <= 2048) return launch(combine_grad_kernel<E, 256, AT>, grid_of<256>(a.tokens), 256, s, a);
  return launch(combine_grad_kernel<E, 512, AT>, grid_of<512>(a.tokens), 512, s, a);
}

}  // namespace

void sort_chunks(int64_t pairs, int32_t *chunks, int32_t *per_chunk) {
  const int64_t step = kSortWaves * 64;
  int64_t per = (pairs + step - 1) / step * step;
  if (pairs > 8192) {
    // up to 256 chunks of 2048 pairs or more
    per = ((pairs + 255) / 256 + step - 1) / step * step;
    if (per < 2 * step) per = 2 * step;
  }
  if (per < step) per = step;
  *per_chunk = (int32_t)per;
  *chunks = (int32_t)(pairs > 0 ? (pairs + per - 1) / per : 1);
}

hipError_t launch_sort(const SortArgs &a, hipStream_t s) {
  if (a.chunks > 1) {
    const hipError_t e = launch(sort_count_kernel, dim3((unsigned)a.chunks), kSortWaves * 64, s, a);
    if (e != hipSuccess) return e;
  }
  return launch(sort_kernel, dim3((unsigned)a.chunks), kSortWaves * 64, s, a);
}

hipError_t launch_dispatch(const DispatchArgs &a, hipStream_t s) {
  const int64_t scale_groups = a.x_scale ? (a.tokens + 63) / 64 * ((a.blocks + 3) / 4) : 0;
  if (a.bytes <= kPiece / 2) {
    const int shift = threads_shift((a.bytes + 15) / 16), per = 256 >> shift;
    return launch(dispatch_kernel<true>, grid_of<256>(scale_groups + (a.tokens + per - 1) / per), 256, s, a, scale_groups,
                  shift);
  }
  return launch(dispatch_kernel<false>, grid_of<256>(scale_groups + a.tokens * ((a.bytes + kPiece - 1) / kPiece)), 256, s,
                a, scale_groups, 8);
}

hipError_t launch_combine(const CombineArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return combine_go<BF16>(a, s);
  if (a.dtype == HF_F16) return combine_go<F16>(a, s);
  return combine_go<F32>(a, s);
}

hipError_t launch_combine_grad(const CombineArgs &a, hipStream_t s) {
  if (a.dtype == HF_BF16) return a.top_k <= 4 ? combine_grad_go<BF16, 4>(a, s) : combine_grad_go<BF16, 8>(a, s);
  if (a.dtype == HF_F16) return a.top_k <= 4 ? combine_grad_go<F16, 4>(a, s) : combine_grad_go<F16, 8>(a, s);
  return a.top_k <= 4 ? combine_grad_go<F32, 4>(a, s) : combine_grad_go<F32, 8>(a, s);
}

}  // namespace hf
