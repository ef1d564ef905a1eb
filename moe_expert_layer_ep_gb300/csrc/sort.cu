// Tokens sorted by expert and back, and the gradients of both ways
// (moe_sort_plan, moe_sort_tokens, moe_unsort_tokens,
// moe_unsort_tokens_backward).  No counterpart in the PR reports: the layer's
// quant-scatter and combine are bound to a context's weights, dtype and
// workspace and have no gradient; these work on any rows.
//
//   sort      xs[src2dst[t, j]] = x[t]
//   unsort    out[t] = sum_j w[t, j] * y[src2dst[t, j]]      (w absent: 1)
//   backward of sort    dx[t] = sum_j dxs[src2dst[t, j]]     = unsort without w
//   backward of unsort  dy[src2dst[t, j]] = w[t, j] * dout[t]
//                       dw[t, j] = <dout[t], y[src2dst[t, j]]>
//
// All of them are bound by the bytes of the rows.  A group of threads owns one
// token and walks its columns, so the token's own row is read or written once
// whatever topk is, every sorted row once, and sums over j are taken in j
// order in fp32 registers: nothing is added atomically, the results are the
// same bits every time and at every batch size.
#include <string.h>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kSortThreads = 256;
constexpr int kSortBatch = 4;     // row segments a thread has in flight (sort; element-wide unsort)
constexpr int kJBatch = 8;        // selections handled together

struct SortArgs {
  const void* x;            // sort: x; unsort: sorted rows; backward: dout
  const void* y;            // backward: sorted rows of the forward (NULL: no dw)
  const int32_t* src2dst;   // [T, topk]
  const float* w;           // [T, topk] or NULL
  void* out;                // sort: sorted rows; unsort: out; backward: dy
  float* dw;                // backward
  int64_t T, K, rows;
  int64_t x_ld, y_ld, out_ld;   // elements
  int32_t topk;
  int32_t lanes_log2;       // log2 of the threads that share a token
};

// A thread's share of a row: kVec consecutive elements, as one access.
template <typename E, int kVec>
struct Pack;
template <>
struct Pack<uint16_t, 8> {
  using Raw = uint4;
  __device__ static void open(const Raw& r, float (&f)[8]) {
    const float2 a = unpack_bf16x2(r.x), b = unpack_bf16x2(r.y), c = unpack_bf16x2(r.z), d = unpack_bf16x2(r.w);
    f[0] = a.x; f[1] = a.y; f[2] = b.x; f[3] = b.y; f[4] = c.x; f[5] = c.y; f[6] = d.x; f[7] = d.y;
  }
  __device__ static Raw close(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]),
                      pack_bf16x2(f[6], f[7]));
  }
};
template <>
struct Pack<uint16_t, 2> {
  using Raw = uint32_t;
  __device__ static void open(const Raw& r, float (&f)[2]) {
    const float2 a = unpack_bf16x2(r);
    f[0] = a.x; f[1] = a.y;
  }
  __device__ static Raw close(const float (&f)[2]) { return pack_bf16x2(f[0], f[1]); }
};
template <>
struct Pack<uint16_t, 1> {
  using Raw = uint16_t;
  __device__ static void open(const Raw& r, float (&f)[1]) { f[0] = __uint_as_float(static_cast<uint32_t>(r) << 16); }
  __device__ static Raw close(const float (&f)[1]) { return __bfloat16_as_ushort(__float2bfloat16_rn(f[0])); }
};
template <>
struct Pack<float, 4> {
  using Raw = float4;
  __device__ static void open(const Raw& r, float (&f)[4]) { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
  __device__ static Raw close(const float (&f)[4]) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <>
struct Pack<float, 1> {
  using Raw = float;
  __device__ static void open(const Raw& r, float (&f)[1]) { f[0] = r; }
  __device__ static Raw close(const float (&f)[1]) { return f[0]; }
};

// Each token's destination rows (-1: dropped, or outside the sorted buffer) and
// weights, read once into shared memory by the token's threads.
struct Picks {
  int32_t d[kSortThreads / 32][kMaxTopk];
  float w[kSortThreads / 32][kMaxTopk];
};
// All threads that share a token.
__device__ __forceinline__ void group_sync(int slot, int lanes) {
  if (lanes == 32)
    __syncwarp();
  else
    asm volatile("bar.sync %0, %1;" ::"r"(slot + 1), "r"(lanes) : "memory");
}
__device__ __forceinline__ void load_picks(const SortArgs& a, Picks& s, int64_t t, int slot, int lane, int lanes) {
  if (t < a.T)
    for (int j = lane; j < a.topk; j += lanes) {
      const int32_t d = a.src2dst[t * a.topk + j];
      s.d[slot][j] = d < a.rows ? d : -1;
      s.w[slot][j] = a.w ? a.w[t * a.topk + j] : 1.0f;
    }
  group_sync(slot, lanes);
}

template <typename E, int kVec>
__global__ void __launch_bounds__(kSortThreads) sort_tokens_kernel(SortArgs a) {
  using P = Pack<E, kVec>;
  using Raw = typename P::Raw;
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1);
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kSortThreads >> a.lanes_log2) + (threadIdx.x >> a.lanes_log2);
  __shared__ Picks s;
  const int slot = threadIdx.x >> a.lanes_log2;
  pdl_wait();
  pdl_trigger();
  load_picks(a, s, t, slot, lane, lanes);
  if (t >= a.T) return;
  const E* xrow = static_cast<const E*>(a.x) + t * a.x_ld;
  E* out = static_cast<E*>(a.out);
  const int64_t step = static_cast<int64_t>(lanes) * kVec;
  const int64_t first = static_cast<int64_t>(lane) * kVec + blockIdx.y * kSortBatch * step;
  for (int64_t c0 = first; c0 < a.K; c0 += gridDim.y * kSortBatch * step) {
    Raw v[kSortBatch];
#pragma unroll
    for (int b = 0; b < kSortBatch; ++b)
      if (c0 + b * step < a.K) v[b] = *reinterpret_cast<const Raw*>(xrow + c0 + b * step);
    for (int j = 0; j < a.topk; ++j) {
      const int32_t d = s.d[slot][j];
      if (d < 0) continue;
      E* orow = out + d * a.out_ld + c0;
#pragma unroll
      for (int b = 0; b < kSortBatch; ++b)
        if (c0 + b * step < a.K) *reinterpret_cast<Raw*>(orow + b * step) = v[b];
    }
  }
}

// kJ selections of kSeg row segments per thread at once: eight loads in flight
// whatever topk is.
template <typename E, int kVec, int kJ>
__global__ void __launch_bounds__(kSortThreads) unsort_tokens_kernel(SortArgs a) {
  using P = Pack<E, kVec>;
  using Raw = typename P::Raw;
  constexpr int kSeg = (kVec <= 2 ? 16 : 8) / kJ;
  __shared__ Picks s;
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), slot = threadIdx.x >> a.lanes_log2;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kSortThreads >> a.lanes_log2) + slot;
  pdl_wait();
  pdl_trigger();
  load_picks(a, s, t, slot, lane, lanes);
  if (t >= a.T) return;
  const E* y = static_cast<const E*>(a.x);
  E* orow = static_cast<E*>(a.out) + t * a.out_ld;
  const int64_t step = static_cast<int64_t>(lanes) * kVec;
  const int64_t first = static_cast<int64_t>(lane) * kVec + blockIdx.y * kSeg * step;
  for (int64_t c = first; c < a.K; c += gridDim.y * kSeg * step) {
    float acc[kSeg][kVec];
#pragma unroll
    for (int g = 0; g < kSeg; ++g)
#pragma unroll
      for (int i = 0; i < kVec; ++i) acc[g][i] = 0.0f;
    for (int j0 = 0; j0 < a.topk; j0 += kJ) {
      Raw v[kSeg][kJ];
      // every load of the batch before the first use
#pragma unroll
      for (int jj = 0; jj < kJ; ++jj) {
        const int j = j0 + jj;
        const bool on = j < a.topk && s.d[slot][j] >= 0;
        const E* row = y + (on ? s.d[slot][j] : 0) * a.x_ld + c;
#pragma unroll
        for (int g = 0; g < kSeg; ++g)
          if (on && c + g * step < a.K) v[g][jj] = *reinterpret_cast<const Raw*>(row + g * step);
      }
#pragma unroll
      for (int jj = 0; jj < kJ; ++jj) {
        const int j = j0 + jj;
        if (j >= a.topk || s.d[slot][j] < 0) continue;
        const float w = s.w[slot][j];
#pragma unroll
        for (int g = 0; g < kSeg; ++g) {
          float f[kVec];
          P::open(v[g][jj], f);
#pragma unroll
          for (int i = 0; i < kVec; ++i) acc[g][i] = fmaf(w, f[i], acc[g][i]);
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kSeg; ++g)
      if (c + g * step < a.K) *reinterpret_cast<Raw*>(orow + c + g * step) = P::close(acc[g]);
  }
}

// kBackJ selections' rows in flight per thread.  A token is one short chain of
// loads, stores and a reduction, so it is other tokens on the SM that keep the
// memory busy: a token's threads get two segments of its rows each, or four and
// 128 threads at most where a token has few rows, and rows that are read element
// by element, or few per token, take fewer registers for more CTAs per SM.
// T = 4096, K = 2048, top-8, bf16: 55 us with a CTA per token, 45 us so; T = 8192,
// K = 7168: 306 us with one warp per token, 290 us so, top-2 100 and 99 us.  The
// threads, and with them the order of the dot products' sums, depend on K and the
// rows per token alone, so that a token's results do not depend on the others.
template <typename E, int kVec, int kBackJ>
__global__ void __launch_bounds__(kSortThreads, kBackJ == 8 ? 3 : 4) unsort_backward_kernel(SortArgs a) {
  using P = Pack<E, kVec>;
  using Raw = typename P::Raw;
  constexpr int kSeg = kVec <= 2 ? 2 : 1;
  __shared__ float s_dot[kSortThreads / 32][kJBatch];
  __shared__ Picks s;
  const int lanes = 1 << a.lanes_log2;
  const int lane = threadIdx.x & (lanes - 1), warp = threadIdx.x >> 5, slot = threadIdx.x >> a.lanes_log2;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * (kSortThreads >> a.lanes_log2) + slot;
  pdl_wait();
  pdl_trigger();
  load_picks(a, s, t, slot, lane, lanes);
  const bool live = t < a.T;
  const E* drow = static_cast<const E*>(a.x) + t * a.x_ld;
  const E* y = static_cast<const E*>(a.y);
  E* dy = static_cast<E*>(a.out);
  const int64_t step = static_cast<int64_t>(lanes) * kVec;
  for (int j0 = 0; j0 < a.topk; j0 += kJBatch) {
    float dot[kJBatch];
#pragma unroll
    for (int jj = 0; jj < kJBatch; ++jj) dot[jj] = 0.0f;
    for (int64_t c = static_cast<int64_t>(lane) * kVec; live && c < a.K; c += kSeg * step) {
      Raw rd[kSeg];
#pragma unroll
      for (int i = 0; i < kSeg; ++i)
        if (c + i * step < a.K) rd[i] = *reinterpret_cast<const Raw*>(drow + c + i * step);
#pragma unroll
      for (int h = 0; h < kJBatch; h += kBackJ) {
        Raw v[kSeg][kBackJ];
        int32_t d[kBackJ];
#pragma unroll
        for (int jj = 0; jj < kBackJ; ++jj) {
          d[jj] = j0 + h + jj < a.topk ? s.d[slot][j0 + h + jj] : -1;
          if (y && d[jj] >= 0) {
            const E* row = y + d[jj] * a.y_ld + c;
#pragma unroll
            for (int i = 0; i < kSeg; ++i)
              if (c + i * step < a.K) v[i][jj] = *reinterpret_cast<const Raw*>(row + i * step);
          }
        }
#pragma unroll
        for (int i = 0; i < kSeg; ++i) {
          if (c + i * step >= a.K) continue;
          float g[kVec];
          P::open(rd[i], g);
#pragma unroll
          for (int jj = 0; jj < kBackJ; ++jj) {
            if (d[jj] < 0) continue;
            float f[kVec];
            if (y) {
              P::open(v[i][jj], f);
#pragma unroll
              for (int e = 0; e < kVec; ++e) dot[h + jj] = fmaf(g[e], f[e], dot[h + jj]);
            }
            const float w = s.w[slot][j0 + h + jj];
#pragma unroll
            for (int e = 0; e < kVec; ++e) f[e] = w * g[e];
            *reinterpret_cast<Raw*>(dy + d[jj] * a.out_ld + c + i * step) = P::close(f);
          }
        }
      }
    }
    if (!y) continue;
#pragma unroll
    for (int jj = 0; jj < kJBatch; ++jj)
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) dot[jj] += __shfl_xor_sync(0xFFFFFFFFu, dot[jj], o);
    if ((threadIdx.x & 31) == 0) {
#pragma unroll
      for (int jj = 0; jj < kJBatch; ++jj) s_dot[warp][jj] = dot[jj];
    }
    group_sync(slot, lanes);
    // the group's first threads add its warps' sums in order
    if (live && lane < kJBatch && j0 + lane < a.topk) {
      float sum = 0.0f;
      for (int k = 0; k < lanes / 32; ++k) sum += s_dot[warp + k][lane];
      a.dw[t * a.topk + j0 + lane] = sum;
    }
    group_sync(slot, lanes);
  }
}

using SortKernel = void (*)(SortArgs);
enum SortOp { kOpSort, kOpUnsort, kOpBackward };

template <typename E, int kVec>
SortKernel kernel_of(SortOp op, int topk) {
  if (op == kOpSort) return sort_tokens_kernel<E, kVec>;
  if (op == kOpBackward)
    return kVec <= 2 || topk <= 4 ? unsort_backward_kernel<E, kVec, 4> : unsort_backward_kernel<E, kVec, kVec <= 2 ? 4 : 8>;
  if (topk == 1) return unsort_tokens_kernel<E, kVec, 1>;
  if (topk == 2) return unsort_tokens_kernel<E, kVec, 2>;
  return topk <= 4 ? unsort_tokens_kernel<E, kVec, 4> : unsort_tokens_kernel<E, kVec, 8>;
}

// Row accesses are 16 bytes wide when every row starts on a 16-byte boundary
// and its length is a multiple of 16 bytes, else one element wide, or two bf16
// elements where rows allow it.
moe_status_t launch_sort(SortOp op, SortArgs a, int32_t elem, cudaStream_t s) {
  if (a.T == 0) return MOE_OK;
  const int es = elem == MOE_ELEM_F32 ? 4 : 2;
  const bool has_y = a.y != nullptr;
  const uintptr_t bases = reinterpret_cast<uintptr_t>(a.x) | reinterpret_cast<uintptr_t>(a.out) |
                          (has_y ? reinterpret_cast<uintptr_t>(a.y) : 0);
  const auto fits = [&](int bytes) {
    const int n = bytes / es;
    return bases % bytes == 0 && a.K % n == 0 && a.x_ld % n == 0 && a.out_ld % n == 0 && (!has_y || a.y_ld % n == 0);
  };
  const bool vec = fits(16), two = !vec && es == 2 && fits(4);
  const int64_t units = a.K / (vec ? 16 / es : two ? 2 : 1);
  // segments a thread has in flight, and the threads that cover a row with them
  // (the way back: 128 threads at most.  In us with 128 and with 256, K = 7168,
  // top-8: 4.6 and 5.8 for 128 tokens, 26.6 and 28.8 for 1001, 50.5 and 48.5 for
  // 2000, 161 and 170 for 8192; K = 4096, top-4: 15.5 and 16.8 for 1500, 67 and
  // 77 for 8192; K = 2048 in fp32, top-8: 25.6 and 26.2 for 2000, 49.6 and 47.7
  // for 4000; K = 1001, top-8: 19.1 and 16.6 for 1500, 70.8 and 74.1 for 8192.
  // Where 256 is ahead, its CTAs happen to fill the SMs more evenly.)
  int64_t seg = kSortBatch;
  if (op == kOpUnsort) seg = (vec ? 8 : 16) / (a.topk == 1 ? 1 : a.topk == 2 ? 2 : a.topk <= 4 ? 4 : 8);
  if (op == kOpBackward) seg = vec ? 1 : 2;
  const bool few = a.topk <= 4;
  a.lanes_log2 = 5;
  while (a.lanes_log2 < 8 && (seg << a.lanes_log2) < units &&
         (op != kOpBackward || ((seg << a.lanes_log2) * (few ? 4 : 2) < units && a.lanes_log2 < (few ? 7 : 8))) &&
         (op != kOpUnsort || a.lanes_log2 < 7))
    ++a.lanes_log2;
  const int64_t per_cta = kSortThreads >> a.lanes_log2;
  const int64_t grid = (a.T + per_cta - 1) / per_cta;
  // few tokens: their columns are spread over CTAs too (not in the backward
  // kernel, whose dot products run over a token's whole row)
  int64_t parts = (units + (seg << a.lanes_log2) - 1) / (seg << a.lanes_log2);
  const int64_t room = 1024 / grid;
  if (parts > room) parts = room;
  if (op == kOpBackward || parts < 1) parts = 1;
  SortKernel k;
  if (elem == MOE_ELEM_F32)
    k = vec ? kernel_of<float, 4>(op, a.topk) : kernel_of<float, 1>(op, a.topk);
  else
    k = vec   ? kernel_of<uint16_t, 8>(op, a.topk)
        : two ? kernel_of<uint16_t, 2>(op, a.topk)
              : kernel_of<uint16_t, 1>(op, a.topk);
  return launch_pdl(k, dim3(static_cast<unsigned>(grid), static_cast<unsigned>(parts)), dim3(kSortThreads), 0, s, a) ==
                 cudaSuccess
             ? MOE_OK
             : MOE_ERR_CUDA;
}

bool off(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// Checks that the three row operators share.
moe_status_t check_sort(int64_t T, int32_t topk, int64_t K, int32_t elem, int64_t rows, const int32_t* src2dst,
                        const void* tokens, int64_t tokens_ld, const void* sorted, int64_t sorted_ld) {
  if (T < 0 || topk <= 0 || K <= 0 || rows < 0) return MOE_ERR_INVALID_ARG;
  if (elem != MOE_ELEM_BF16 && elem != MOE_ELEM_F32) return MOE_ERR_INVALID_ARG;
  if (tokens_ld < K || sorted_ld < K) return MOE_ERR_INVALID_ARG;
  if (topk > kMaxTopk || T > 0x7FFFFFFF || rows > 0x7FFFFFFF) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!src2dst || !tokens || (!sorted && rows > 0)) return MOE_ERR_INVALID_ARG;
  const uintptr_t es = elem == MOE_ELEM_F32 ? 4 : 2;
  if (off(src2dst, 4) || off(tokens, es) || off(sorted, es)) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

// ---------------------------------------------------------------------------
// The plan
// ---------------------------------------------------------------------------
// A stable counting sort of the assignments by expert in two kernels.  The
// assignments are cut into at most kPlanParts parts of whole 512s, one CTA
// each.  sort_count leaves each part's experts' counts and every assignment's
// rank among its expert's within the part (warp match, per-warp counts,
// running counts over the part's 512s); sort_place adds the counts of the parts
// before and of the experts before.  Every CTA sums the whole count table
// itself (128 KB at 256 experts, from L2): cheaper than a kernel between the
// two.  Integers only; nothing depends on the order of anything.
constexpr int kPlanThreads = 512;
constexpr int kPlanParts = 128;

struct SortPlanArgs {
  const int32_t* ids;
  int64_t A;
  int32_t E_global, E, first;
  int32_t parts, per_part;   // 512s of a part
  int32_t* status;
  int32_t* hist;             // [parts][E]
  int32_t* rank;             // [A]
  int32_t* src2dst;
  int32_t* start;
  int32_t* counts;
};

// Local expert of assignment i, -1 when it has none.
__device__ __forceinline__ int sort_expert(const SortPlanArgs& p, int64_t i, bool* bad) {
  const int id = p.ids[i];
  *bad = id < -1 || id >= p.E_global;
  const int e = id - p.first;
  return !*bad && id >= 0 && e >= 0 && e < p.E ? e : -1;
}

__global__ void __launch_bounds__(kPlanThreads) sort_count_kernel(SortPlanArgs p) {
  constexpr int kWarps = kPlanThreads / 32;
  __shared__ uint16_t s_warp[kWarps][kMaxLocalExperts];
  __shared__ int32_t s_run[kMaxLocalExperts];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x == 0 && tid < 4) p.status[tid] = 0;   // (only the next kernel sets it)
  for (int e = tid; e < p.E; e += kPlanThreads) s_run[e] = 0;
  for (int r = 0; r < p.per_part; ++r) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * p.per_part + r) * kPlanThreads + tid;
    for (int e = tid; e < p.E; e += kPlanThreads)
#pragma unroll
      for (int w = 0; w < kWarps; ++w) s_warp[w][e] = 0;
    bool bad;
    const int e = i < p.A ? sort_expert(p, i, &bad) : -1;
    __syncthreads();
    const unsigned peers = __match_any_sync(0xFFFFFFFFu, e);
    const int before = __popc(peers & ((1u << lane) - 1u));
    if (e >= 0 && before == 0) s_warp[warp][e] = static_cast<uint16_t>(__popc(peers));
    __syncthreads();
    if (e >= 0) {
      int rank = s_run[e] + before;
      for (int w = 0; w < warp; ++w) rank += s_warp[w][e];
      p.rank[i] = rank;
    }
    __syncthreads();
    for (int x = tid; x < p.E; x += kPlanThreads) {
      int n = 0;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) n += s_warp[w][x];
      s_run[x] += n;
    }
    __syncthreads();
  }
  for (int e = tid; e < p.E; e += kPlanThreads) p.hist[static_cast<int64_t>(blockIdx.x) * p.E + e] = s_run[e];
}

__global__ void __launch_bounds__(kPlanThreads) sort_place_kernel(SortPlanArgs p) {
  __shared__ int32_t s_total[kMaxLocalExperts], s_before[kMaxLocalExperts], s_sum[kPlanThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int e = tid; e < p.E; e += kPlanThreads) s_total[e] = s_before[e] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // few experts: several threads share one, taking every few parts
  int span = 32;
  while (span < p.E && span < kPlanThreads) span <<= 1;
  const int step = kPlanThreads / span;
  for (int e = tid & (span - 1); e < p.E; e += span) {
    int total = 0, before = 0;
#pragma unroll 8
    for (int c = tid / span; c < p.parts; c += step) {
      const int n = p.hist[static_cast<int64_t>(c) * p.E + e];
      total += n;
      if (c < blockIdx.x) before += n;
    }
    if (total) atomicAdd(&s_total[e], total);
    if (before) atomicAdd(&s_before[e], before);
  }
  __syncthreads();
  // experts' first rows: two consecutive experts per thread, scanned
  const int e0 = 2 * tid;
  const int n0 = e0 < p.E ? s_total[e0] : 0, n1 = e0 + 1 < p.E ? s_total[e0 + 1] : 0;
  const int r0 = (n0 + kBlockM - 1) / kBlockM * kBlockM, r1 = (n1 + kBlockM - 1) / kBlockM * kBlockM;
  int x = r0 + r1;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  if (lane == 31) s_sum[warp] = x;
  __syncthreads();
  int row = x - r0 - r1;
  for (int w = 0; w < warp; ++w) row += s_sum[w];
  if (e0 < p.E) s_before[e0] += row;
  if (e0 + 1 < p.E) s_before[e0 + 1] += row + r0;
  if (blockIdx.x == 0) {
    if (e0 < p.E) {
      p.start[e0] = row;
      p.counts[e0] = n0;
    }
    if (e0 + 1 < p.E) {
      p.start[e0 + 1] = row + r0;
      p.counts[e0 + 1] = n1;
    }
  }
  __syncthreads();
  for (int r = 0; r < p.per_part; ++r) {
    const int64_t i = (static_cast<int64_t>(blockIdx.x) * p.per_part + r) * kPlanThreads + tid;
    if (i >= p.A) break;
    bool bad;
    const int e = sort_expert(p, i, &bad);
    if (bad) set_status(p.status, MOE_ERR_EXPERT_ID);
    p.src2dst[i] = e >= 0 ? s_before[e] + p.rank[i] : -1;
  }
}

uint64_t align256(uint64_t x) { return (x + 255) & ~uint64_t(255); }

struct SortWs {
  uint64_t meta, padded, hist, rank, total;
  int32_t parts, per_part;
};
SortWs sort_ws(int64_t A, int32_t E) {
  SortWs w;
  const int64_t blocks = (A + kPlanThreads - 1) / kPlanThreads;
  w.per_part = static_cast<int32_t>((blocks + kPlanParts - 1) / kPlanParts);
  w.parts = w.per_part ? static_cast<int32_t>((blocks + w.per_part - 1) / w.per_part) : 1;
  // (the one-CTA plan uses meta and padded, the two kernels hist and rank)
  w.meta = 256;   // the status word comes first
  w.padded = w.meta + 256;
  w.hist = w.padded + align256(4 * static_cast<uint64_t>(E));
  w.rank = w.hist + align256(4 * static_cast<uint64_t>(w.parts) * E);
  w.total = w.rank + align256(4 * static_cast<uint64_t>(A));
  return w;
}

}  // namespace

}  // namespace moe

extern "C" {

int64_t moe_sort_plan_workspace_size(int64_t T, int32_t topk, int32_t E_local) {
  if (T < 0 || topk <= 0 || E_local <= 0 || T >= (int64_t(1) << 31)) return -1;
  return static_cast<int64_t>(moe::sort_ws(T * topk, E_local).total);
}

moe_status_t moe_sort_plan(const int32_t* topk_ids, int64_t T, int32_t topk, int32_t E_global, int32_t E_local,
                           int32_t expert_start, int32_t* src2dst, int32_t* start, int32_t* counts, void* ws,
                           int64_t ws_bytes, void* stream) {
  if (T < 0 || topk <= 0 || E_global <= 0 || E_local <= 0 || expert_start < 0 ||
      static_cast<int64_t>(E_local) + expert_start > E_global)
    return MOE_ERR_INVALID_ARG;
  if (E_local > moe::kMaxLocalExperts || topk > moe::kMaxTopk || T >= (int64_t(1) << 31) ||
      moe_compact_all_tokens(T * topk, E_local, 128) >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  if ((T > 0 && (!topk_ids || !src2dst)) || !start || !counts || !ws) return MOE_ERR_INVALID_ARG;
  if (moe::off(topk_ids, 4) || moe::off(src2dst, 4) || moe::off(start, 4) || moe::off(counts, 4) || moe::off(ws, 16))
    return MOE_ERR_MISALIGNED;
  const int64_t A = T * topk;
  const moe::SortWs w = moe::sort_ws(A, E_local);
  if (ws_bytes < static_cast<int64_t>(w.total)) return MOE_ERR_BUFFER_TOO_SMALL;
  uint8_t* base = static_cast<uint8_t*>(ws);
  const cudaStream_t cs = static_cast<cudaStream_t>(stream);
  if (moe::plan_is_small(A, E_local)) {   // one CTA: 3.7 us where the two kernels take 6
    moe::PlanArgs p;
    memset(&p, 0, sizeof(p));
    p.topk_ids = topk_ids;
    p.A = A;
    p.E_global = E_global;
    p.E_local = E_local;
    p.expert_start = expert_start;
    p.status = reinterpret_cast<int32_t*>(base);
    p.meta = reinterpret_cast<int32_t*>(base + w.meta);
    p.counts = counts;
    p.padded = reinterpret_cast<int32_t*>(base + w.padded);
    p.start = start;
    p.src2dst = src2dst;
    return moe::launch_plan(p, cs) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  moe::SortPlanArgs p;
  memset(&p, 0, sizeof(p));
  p.ids = topk_ids;
  p.A = A;
  p.E_global = E_global;
  p.E = E_local;
  p.first = expert_start;
  p.parts = w.parts;
  p.per_part = w.per_part;
  p.status = reinterpret_cast<int32_t*>(base);
  p.hist = reinterpret_cast<int32_t*>(base + w.hist);
  p.rank = reinterpret_cast<int32_t*>(base + w.rank);
  p.src2dst = src2dst;
  p.start = start;
  p.counts = counts;
  const dim3 grid(static_cast<unsigned>(w.parts)), block(moe::kPlanThreads);
  if (moe::launch_pdl(moe::sort_count_kernel, grid, block, 0, cs, p) != cudaSuccess ||
      moe::launch_pdl(moe::sort_place_kernel, grid, block, 0, cs, p) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status_t moe_sort_tokens(const void* x, int64_t x_ld, const int32_t* src2dst, int64_t T, int32_t topk, int64_t K,
                             int32_t elem, void* sorted, int64_t sorted_ld, int64_t rows, void* stream) {
  const moe_status_t st = moe::check_sort(T, topk, K, elem, rows, src2dst, x, x_ld, sorted, sorted_ld);
  if (st != MOE_OK) return st;
  moe::SortArgs a;
  memset(&a, 0, sizeof(a));
  a.x = x;
  a.x_ld = x_ld;
  a.src2dst = src2dst;
  a.T = T;
  a.K = K;
  a.topk = topk;
  a.rows = rows;
  a.out = sorted;
  a.out_ld = sorted_ld;
  return moe::launch_sort(moe::kOpSort, a, elem, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_unsort_tokens(const void* sorted, int64_t sorted_ld, int64_t rows, const int32_t* src2dst,
                               const float* topk_weights, int64_t T, int32_t topk, int64_t K, int32_t elem, void* out,
                               int64_t out_ld, void* stream) {
  const moe_status_t st = moe::check_sort(T, topk, K, elem, rows, src2dst, out, out_ld, sorted, sorted_ld);
  if (st != MOE_OK) return st;
  if (moe::off(topk_weights, 4)) return MOE_ERR_MISALIGNED;
  moe::SortArgs a;
  memset(&a, 0, sizeof(a));
  a.x = sorted;
  a.x_ld = sorted_ld;
  a.src2dst = src2dst;
  a.w = topk_weights;
  a.T = T;
  a.K = K;
  a.topk = topk;
  a.rows = rows;
  a.out = out;
  a.out_ld = out_ld;
  return moe::launch_sort(moe::kOpUnsort, a, elem, static_cast<cudaStream_t>(stream));
}

moe_status_t moe_unsort_tokens_backward(const void* dout, int64_t dout_ld, const void* sorted, int64_t sorted_ld,
                                        int64_t rows, const int32_t* src2dst, const float* topk_weights, int64_t T,
                                        int32_t topk, int64_t K, int32_t elem, void* dsorted, int64_t dsorted_ld,
                                        float* dweights, void* stream) {
  moe_status_t st = moe::check_sort(T, topk, K, elem, rows, src2dst, dout, dout_ld, dsorted, dsorted_ld);
  if (st != MOE_OK) return st;
  if ((sorted == nullptr) != (dweights == nullptr) && rows > 0) return MOE_ERR_INVALID_ARG;
  if (sorted && sorted_ld < K) return MOE_ERR_INVALID_ARG;
  if (T > 0 && !topk_weights) return MOE_ERR_INVALID_ARG;
  if (moe::off(topk_weights, 4) || moe::off(dweights, 4) || moe::off(sorted, elem == MOE_ELEM_F32 ? 4 : 2))
    return MOE_ERR_MISALIGNED;
  if (rows == 0) {   // nothing was kept: no rows, and every weight's gradient is 0
    if (T == 0 || !dweights) return MOE_OK;
    return cudaMemsetAsync(dweights, 0, sizeof(float) * T * topk, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? MOE_OK
               : MOE_ERR_CUDA;
  }
  moe::SortArgs a;
  memset(&a, 0, sizeof(a));
  a.x = dout;
  a.x_ld = dout_ld;
  a.y = sorted;
  a.y_ld = sorted_ld;
  a.src2dst = src2dst;
  a.w = topk_weights;
  a.T = T;
  a.K = K;
  a.topk = topk;
  a.rows = rows;
  a.out = dsorted;
  a.out_ld = dsorted_ld;
  a.dw = dweights;
  return moe::launch_sort(moe::kOpBackward, a, elem, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
