// moe_route_backward: the gradient of the router, with its two losses.
//
// For token t with logits z, probabilities p = softmax(z) over all experts,
// l = log sum exp z, and the selection's weights w (softmax over the selected):
//   losses    B = E sum_e f_e P_e,  Z = mean of l^2      (means over the n tokens that
//             f_e = assignments of e / (n k),  P_e = mean of p_e      have an expert)
//   dz_e    = cb (E / n) p_e (f_e - sum_i f_i p_i) + cz (2 / n) l p_e
//             + sum over j with id_j = e of w_j (dw_j - sum_i w_i dw_i)
//             (an assignment that was dropped with its id kept: its dw is 0 and f_e does
//             not count it, but its weight took part in the softmax)
//   dx      = dz W + residual (bf16),   dW = dz^T x (fp32)
//
// Three kernels, and a fourth where dW's sums were split:
//   route_prepare_kernel assignments per expert and tokens that have one; W in fp16, less a
//                        row m that they have in common where that makes an expert's row
//                        clearly smaller, each expert's row times a power of two
//   route_dz_kernel      a warp per token: dz in three bf16 planes whose sum it is (as
//                        moe_router_prepare splits the weights) and, for dx, in fp16
//                        times a power of two, without the weights' own; its sum over the
//                        experts whose rows are less m; zeros behind the
//                        experts up to a multiple of 64; the losses of eight tokens, which
//                        dW's part of the next kernel adds
//   router_products_kernel  both products, dx on some of the CTA pairs and dW on the others:
//     dx                 dz W on the tensor cores in fp16: 11 bits of each factor, so each
//                        term is at most 2^-10 off, for a result that is stored with 8 bits
//                        (over many terms the storing is what is left of the error: 1.66e-3
//                        of the norm, 1.64e-3 with exact factors); three products of bf16
//                        planes cost three times the MMAs (the whole call 132 us, so then 112).
//                        A dz of softmaxes sums to 0, so what the rows of W have in common
//                        cancels, and rounded factors would not (a common row 32 times the
//                        rest: 9.7e-3): hence the rows less m, and dz's sum times m in fp32
//     dW                 dz^T x likewise: x is bf16, so three products per block are dz's
//                        fp32 value times x
//   router_dw_sum_kernel the parts of a split sum, in order
//
// dx.  A tile of 256 tokens x 256 columns on a CTA pair, tokens in lanes, so
// that a thread's columns lie side by side in memory and its power of two is one number.
//
// What bounds it at 8192 x 7168 and 256 experts: the SM's epilogue and shared memory (a tile
// takes 4900 cycles where its MMAs take 2070: operands, residual and result pass through
// shared memory eight times over, 512 KB a tile).
//
// dW.  D = x^T dz, a tile of 256 columns of x by at most 128 experts on a
// CTA pair, both operands MN-major (no transposed copies), the three planes' MMAs on one
// copy of x: 40 KB per SM and 64 tokens for 768 cycles of MMAs.  Experts on the N side cost
// what there are of them, up to a multiple of 32, and put x's columns into lanes, so that a
// warp's stores of an expert are whole lines of dW.
// The tensor cores cut off what does not fit when they add to an fp32 sum (an error that
// grows with the number of steps: 1e-9 of the result per row, 9e-6 after 8192), so a sum
// runs over 256 tokens there, the plane hi in an accumulator of its own, and the segments
// are added in registers, in order.  Bound by its MMAs (the tensor pipe 88 % active).
#include <cuda_fp16.h>
#include <string.h>

#include "internal.h"
#include "pair.cuh"
#include "pairs.h"

namespace moe {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;

// ---------------------------------------------------------------------------
// Counts, and the weights in fp16
// ---------------------------------------------------------------------------
constexpr int kPrepareThreads = 512;
constexpr int kCountCtas = 8;
// m, per column: the middle of the values of four evenly spread experts (of the second and
// third in order), rounded to bf16.  Any row near what rows have in common would do, since
// what is taken off is put back; the middle is not moved by an expert, or a value, unlike the
// others, and each CTA forms it for itself, while the assignments are counted.  (The mean of
// eight took 2.7 us more at 256 experts of 7168, of all, by a kernel before, 4 to 7.)
// An expert's row is taken less m where the sum of its sizes becomes smaller than this share
// of what it was: rows that have nothing in common, whose middle is an accident of the
// drawing, stay as they are.
constexpr float kCentred = 0.7f;

__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }   // |e| <= 126
__device__ __forceinline__ uint32_t pack_half2(float a, float b) {
  const __half2 h = __floats2half2_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, o));
  return v;
}
__device__ __forceinline__ int read_cluster(const int* p, int rank) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(mapa(smem_u32(p), rank)) : "memory");
  return static_cast<int>(v);
}

__device__ __forceinline__ void unpack8(uint4 w, float (&v)[8]) {
  const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 p = unpack_bf16x2(x[j]);
    v[2 * j] = p.x;
    v[2 * j + 1] = p.y;
  }
}

struct PrepareArgs {
  const int32_t* ids;      // [T, topk]
  const uint8_t* kept;     // [T, topk] or null: all
  int64_t T;
  int32_t topk, E;
  int32_t* counts;
  int32_t* tokens;
  int32_t* status;
  const uint4* planes;     // W [3][E][K]
  int64_t row8;            // K / 8
  uint4* common;           // [K] m in bf16
  uint4* half;             // [E][K]
  int32_t* exps;           // [E] the power of two, and 2^16 where the row is less m
};

// What exps holds.
__device__ __forceinline__ int exp_of(int32_t w) { return static_cast<int16_t>(w); }
__device__ __forceinline__ bool is_centred(int32_t w) { return (w >> 16 & 1) != 0; }

// Row e of W, or what is left of it without m, times 2^exp in fp16, its largest
// value in [2^14, 2^15) (exp within +-126).
__device__ __forceinline__ void half_row(const PrepareArgs& g, int e) {
  __shared__ float4 s_part[kPrepareThreads / 32];
  const uint4* hi = g.planes + e * g.row8;
  const uint4* mid = hi + g.E * g.row8;
  const uint4* lo = mid + g.E * g.row8;
  const auto load = [&](const uint4* plane, int64_t i, float (&v)[8]) { unpack8(plane[i], v); };
  const auto load_middle = [&](int64_t i, float (&v)[8]) {   // of the first planes; also its words in bf16
    float w[4][8];
#pragma unroll
    for (int n = 0; n < 4; ++n) load(g.planes + n * g.E / 4 * g.row8, i, w[n]);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float lower = fmaxf(fminf(w[0][j], w[1][j]), fminf(w[2][j], w[3][j]));
      const float upper = fminf(fmaxf(w[0][j], w[1][j]), fmaxf(w[2][j], w[3][j]));
      v[j] = 0.5f * lower + 0.5f * upper;
    }
    const uint4 words = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    unpack8(words, v);
    return words;
  };
  float4 seen = make_float4(0.0f, 0.0f, 0.0f, 0.0f);   // largest and sum, as it is; largest and sum, without m
  for (int64_t i = threadIdx.x; i < g.row8; i += kPrepareThreads) {
    float a[8], b[8], m[8];
    load(hi, i, a);
    load(mid, i, b);
    const uint4 words = load_middle(i, m);
    if (e == 0) g.common[i] = words;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float w = a[j] + b[j], c = fabsf(w - m[j]);
      seen.x = fmaxf(seen.x, fabsf(w));
      seen.y += fabsf(w);
      seen.z = fmaxf(seen.z, c);
      seen.w += c;
    }
  }
  seen = make_float4(warp_max(seen.x), warp_sum(seen.y), warp_max(seen.z), warp_sum(seen.w));
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = seen;
  __syncthreads();
  seen = s_part[0];
#pragma unroll
  for (int w = 1; w < kPrepareThreads / 32; ++w) {
    const float4 p = s_part[w];
    seen = make_float4(fmaxf(seen.x, p.x), seen.y + p.y, fmaxf(seen.z, p.z), seen.w + p.w);
  }
  const bool centred = seen.w < kCentred * seen.y;
  const float most = centred ? seen.z : seen.x;
  const int exp = most > 0.0f ? max(-126, min(126, 141 - static_cast<int>(__float_as_uint(most) >> 23))) : 0;
  const float scale = pow2(exp);
  if (threadIdx.x == 0) g.exps[e] = (exp & 0xFFFF) | (centred ? 1 << 16 : 0);
  for (int64_t i = threadIdx.x; i < g.row8; i += kPrepareThreads) {
    float a[8], b[8];
    load(hi, i, a);
    load(mid, i, b);
#pragma unroll
    for (int j = 0; j < 8; ++j) a[j] += b[j];
    if (centred) {   // (the last plane too: it is 2^-17 of what was common)
      float m[8];
      load(lo, i, b);
      load_middle(i, m);
#pragma unroll
      for (int j = 0; j < 8; ++j) a[j] = a[j] + b[j] - m[j];
    }
    uint32_t o[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = pack_half2(a[2 * j] * scale, a[2 * j + 1] * scale);
    g.half[e * g.row8 + i] = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

// The first cluster counts, its CTAs' histograms meeting in shared memory, so that what it
// writes needs no clearing before (a memset and atomics took 6 us instead of 3, at 65536
// assignments).  The other CTAs take an expert's weights each.
__global__ void __launch_bounds__(kPrepareThreads, 2) route_prepare_kernel(const __grid_constant__ PrepareArgs g) {
  __shared__ int hist[kMaxRouterExperts], s_seen, s_bad;
  pdl_wait();
  pdl_trigger();
  if (blockIdx.x >= kCountCtas) {
    if (static_cast<int>(blockIdx.x) - kCountCtas < g.E) half_row(g, blockIdx.x - kCountCtas);
    return;
  }
  const int rank = static_cast<int>(cluster_ctarank());
  for (int e = threadIdx.x; e < g.E; e += kPrepareThreads) hist[e] = 0;
  if (threadIdx.x == 0) s_seen = s_bad = 0;
  __syncthreads();
  int seen = 0, bad = 0;
  for (int64_t t = rank * kPrepareThreads + threadIdx.x; t < g.T; t += kCountCtas * kPrepareThreads) {
    bool any = false;
    for (int j0 = 0; j0 < g.topk; j0 += 8) {
      int id[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) id[j] = j0 + j < g.topk ? g.ids[t * g.topk + j0 + j] : -1;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (id[j] >= 0 && id[j] < g.E) {
          if (!g.kept || g.kept[t * g.topk + j0 + j]) atomicAdd(&hist[id[j]], 1);
          any = true;
        } else if (id[j] != -1) {
          bad = 1;
        }
      }
    }
    seen += any;
  }
  seen = __reduce_add_sync(kAll, seen);
  bad = __reduce_or_sync(kAll, bad);
  if ((threadIdx.x & 31) == 0) {
    if (seen) atomicAdd(&s_seen, seen);
    if (bad) s_bad = 1;
  }
  cluster_sync();
  for (int e = rank + kCountCtas * threadIdx.x; e < g.E; e += kCountCtas * kPrepareThreads) {
    int n = 0;
#pragma unroll
    for (int r = 0; r < kCountCtas; ++r) n += read_cluster(&hist[e], r);
    g.counts[e] = n;
  }
  if (rank == 0 && threadIdx.x == 0) {
    int n = 0, wrong = 0;
    for (int r = 0; r < kCountCtas; ++r) {
      n += read_cluster(&s_seen, r);
      wrong |= read_cluster(&s_bad, r);
    }
    *g.tokens = n;
    *g.status = wrong ? MOE_ERR_EXPERT_ID : 0;
  }
  cluster_sync();   // no CTA leaves while another may read its shared memory
}

// ---------------------------------------------------------------------------
// Gradient of the logits
// ---------------------------------------------------------------------------
constexpr int kDzWarps = 8;

struct DzArgs {
  const float* logits;
  const int32_t* ids;
  const float* weights;
  const float* dweights;
  const uint8_t* kept;     // [T, topk] or null: all
  int64_t T;
  int32_t E, Ep, topk;     // Ep: E up to a multiple of 64
  float balance, zloss;
  const int32_t* counts;
  const int32_t* tokens;
  const int32_t* exps;     // [E] of the weights' fp16 (PrepareArgs)
  uint16_t* planes;        // [T][3][Ep]
  uint16_t* half;          // [T][Ep] dz 2^-exps, times a power of two of the row, in fp16
  int2* rows;              // [T] 2 to the first's power: what the row's product is multiplied by;
                           // the second, a float: dz's sum over the experts whose rows are less m
  float* dlogits;          // [T, E] or null
  float2* parts;           // [gridDim.x] sums of a CTA's tokens
};

// exp(x) by the hardware's base-2 exponential, 2 ulp and x's rounding; 0 below -87.3.
__device__ __forceinline__ float exp_fast(float x) {
  float e;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.44269504f));
  return e;
}

// A lane holds experts 64 i + 2 lane and the next, i < Q.
template <int Q>
__global__ void __launch_bounds__(32 * kDzWarps, Q <= 2 ? 6 : Q == 4 ? 4 : 2) route_dz_kernel(const DzArgs g) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t t = static_cast<int64_t>(blockIdx.x) * kDzWarps + warp;
  __shared__ float2 s_part[kDzWarps];
  __shared__ float s_row[kDzWarps][64 * Q];
  pdl_wait();
  pdl_trigger();
  float2 part = make_float2(0.0f, 0.0f);
  if (t < g.T) {
    float z[2 * Q];
#pragma unroll
    for (int i = 0; i < 2 * Q; ++i) {
      const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
      z[i] = e < g.E ? g.logits[t * g.E + e] : -INFINITY;
    }
    // this lane's selections, j = lane and lane + 32
    int id[2];
    float wt[2], dw[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int j = lane + 32 * h;
      const bool there = j < g.topk;
      id[h] = there ? g.ids[t * g.topk + j] : -1;
      wt[h] = there ? g.weights[t * g.topk + j] : 0.0f;
      dw[h] = there && (!g.kept || g.kept[t * g.topk + j]) ? g.dweights[t * g.topk + j] : 0.0f;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      if (id[h] >= 0 && id[h] < g.E) continue;
      id[h] = -1;   // no assignment: whatever its weights are
      wt[h] = dw[h] = 0.0f;
    }
    const bool there = __any_sync(kAll, id[0] >= 0 || id[1] >= 0);   // else padding: its logits may be anything
    float top = -INFINITY;
#pragma unroll
    for (int i = 0; i < 2 * Q; ++i) top = fmaxf(top, z[i]);
    if (there) {
      float f[2 * Q];
#pragma unroll
      for (int i = 0; i < 2 * Q; ++i) {
        const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
        f[i] = e < g.E ? static_cast<float>(g.counts[e]) : 0.0f;
      }
      const int n = *g.tokens;
      const float share = 1.0f / (static_cast<float>(n) * static_cast<float>(g.topk));
      top = warp_max(top);
      float total = 0.0f, mixed = 0.0f;
#pragma unroll
      for (int i = 0; i < 2 * Q; ++i) {
        z[i] = exp_fast(z[i] - top);
        f[i] *= share;
        total += z[i];
        mixed += z[i] * f[i];
      }
      total = warp_sum(total);
      const float inv = 1.0f / total;
      mixed = warp_sum(mixed) * inv;   // sum of f p
      const float lse = top + logf(total);
      part = make_float2(mixed, lse * lse);
      const float cb = g.balance * static_cast<float>(g.E) / static_cast<float>(n);
      const float cz = 2.0f * g.zloss / static_cast<float>(n) * lse;
#pragma unroll
      for (int i = 0; i < 2 * Q; ++i) z[i] = z[i] * inv * fmaf(cb, f[i] - mixed, cz);   // dz from here on
      const float mean = warp_sum(wt[0] * dw[0] + wt[1] * dw[1]);
      const float pull0 = wt[0] * (dw[0] - mean), pull1 = wt[1] * (dw[1] - mean);
      // The selections' part, through shared memory: each lane adds its own where all are
      // different experts, else they are added one after another.
      float* row = s_row[warp];
#pragma unroll
      for (int q = 0; q < Q; ++q) *reinterpret_cast<float2*>(row + 64 * q + 2 * lane) = make_float2(z[2 * q], z[2 * q + 1]);
      __syncwarp();
      const unsigned same = __match_any_sync(kAll, id[0] >= 0 ? id[0] : -1 - lane);
      if (g.topk <= 32 && !__any_sync(kAll, same & (same - 1))) {
        if (id[0] >= 0) row[id[0]] += pull0;
      } else {
        for (int j = 0; j < g.topk; ++j) {
          const int e = __shfl_sync(kAll, j < 32 ? id[0] : id[1], j & 31);
          const float pull = __shfl_sync(kAll, j < 32 ? pull0 : pull1, j & 31);
          if (lane == 0 && e >= 0) row[e] += pull;
        }
      }
      __syncwarp();
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const float2 v = *reinterpret_cast<const float2*>(row + 64 * q + 2 * lane);
        z[2 * q] = v.x;
        z[2 * q + 1] = v.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 2 * Q; ++i) z[i] = 0.0f;
    }
    // the row in fp16: W's powers of two taken out again, and one put in that brings the
    // largest of it to at least 2^14, in two factors with W's between them (each product
    // in fp32's range, or nothing beside the largest)
    int we[2 * Q], most = -1000;
    float centred = 0.0f;
    bool any = false;
#pragma unroll
    for (int i = 0; i < 2 * Q; ++i) {
      const int e = 64 * (i >> 1) + 2 * lane + (i & 1);
      const int32_t word = e < g.E ? g.exps[e] : 0;
      we[i] = exp_of(word);
      if (is_centred(word)) centred += z[i];
      any |= is_centred(word);
      if (z[i] != 0.0f) most = max(most, static_cast<int>((__float_as_uint(z[i]) >> 23) & 255u) - 127 - we[i]);
    }
    const int up_by = min(14 - __reduce_max_sync(kAll, most), 252);
    if (__any_sync(kAll, any)) centred = warp_sum(centred);
    if (lane == 0) g.rows[t] = make_int2(-up_by, __float_as_int(centred));
    const float up0 = pow2(up_by / 2), up1 = pow2(up_by - up_by / 2);
    uint32_t* half = reinterpret_cast<uint32_t*>(g.half + t * g.Ep);
#pragma unroll
    for (int q = 0; q < Q; ++q)
      if (64 * q < g.Ep)
        half[32 * q + lane] = pack_half2(z[2 * q] * up0 * pow2(-we[2 * q]) * up1, z[2 * q + 1] * up0 * pow2(-we[2 * q + 1]) * up1);
    uint32_t* row = reinterpret_cast<uint32_t*>(g.planes + t * 3 * g.Ep);
    float* out = g.dlogits ? g.dlogits + t * g.E : nullptr;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int e = 64 * q + 2 * lane;
      if (64 * q >= g.Ep) break;
      float2 v = make_float2(z[2 * q], z[2 * q + 1]);
      if (out) {
        if (e < g.E) out[e] = v.x;
        if (e + 1 < g.E) out[e + 1] = v.y;
      }
#pragma unroll
      for (int p = 0; p < 3; ++p) {   // (each remainder is exact in fp32)
        const uint32_t w = pack_bf16x2(v.x, v.y);
        row[(p * g.Ep + e) >> 1] = w;
        const float2 r = unpack_bf16x2(w);
        v.x -= r.x;
        v.y -= r.y;
      }
    }
  }
  if (lane == 0) s_part[warp] = part;
  __syncthreads();
  if (threadIdx.x == 0) {
    float2 sum = make_float2(0.0f, 0.0f);
    for (int w = 0; w < kDzWarps; ++w) {
      sum.x += s_part[w].x;
      sum.y += s_part[w].y;
    }
    g.parts[blockIdx.x] = sum;
  }
}

// ---------------------------------------------------------------------------
// Gradient of the tokens
// ---------------------------------------------------------------------------
constexpr int kBlock = 64;                       // tokens of a stage of dW
constexpr int kBoxBytes = 64 * 64 * 2;           // an MN-major box of 64 x 64
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;    // producer, MMA, epilogue
constexpr uint32_t kTmemCols = 512;

constexpr int kDxTile = 256;                     // tokens and columns of a pair's tile
constexpr int kDxBlock = 64;                     // experts of a stage
constexpr int kDxPlane = 128 * kDxBlock * 2;     // 16 KB: 128 tokens of dz, or 128 columns of W
constexpr int kDxBox = kDxBlock * 64 * 2;        // an MN-major box of W: 64 experts x 64 columns
constexpr int kDxStage = 2 * kDxPlane;
constexpr int kDxStages = 4;
constexpr int kChunk = 32 * 128;                 // 32 tokens x 64 columns
constexpr int kDxSlots = 3;                      // chunks of an epilogue warp
constexpr int kDxOffSlots = kDxStages * kDxStage;
constexpr int kDxOffBars = kDxOffSlots + kEpiWarps * kDxSlots * kChunk;
constexpr int kDxNumBars = 2 * kDxStages + 5 + kEpiWarps * kDxSlots;
// both parts' holder of the tensor memory's address and their abort flag; dW's part ends
// before it (below)
constexpr int kOffHolder = kDxOffBars + kDxNumBars * 8;
constexpr int kSmem = kOffHolder + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");

struct DxMaps {
  CUtensorMap dz, w, res, out;
};

struct DxArgs {
  int32_t pairs;           // CTA pairs that work on it
  int32_t Ep, e_blocks, t_tiles, k_tiles;
  int64_t T, K;
  const int2* rows;        // [T] (DzArgs)
  const int32_t* exps;     // [E] (PrepareArgs)
  const uint4* common;     // [K] m in bf16 (PrepareArgs)
  int32_t E;
  int32_t residual;
  int32_t* status;
  uint64_t timeout_ns;
};

struct DxItem {
  int t0, k0, n;           // first token, first column, columns of the MMA
};

__device__ __forceinline__ DxItem dx_item(const DxArgs& g, int i) {
  DxItem it;
  const int tt = i / g.k_tiles, kt = i - tt * g.k_tiles;   // (columns innermost: they share dz's rows)
  it.t0 = tt * kDxTile;
  it.k0 = kt * kDxTile;
  it.n = g.K - it.k0 >= kDxTile ? kDxTile : 128;   // (K is a multiple of 128)
  return it;
}

// After an aborted pair: copies may still be on their way into this CTA's shared
// memory, and complete on the other CTA's barrier; they are left ample time.
__device__ __noinline__ void leave_copies_time() {
  const uint64_t now = globaltimer_ns();
  while (globaltimer_ns() - now < 2000000ull) {
  }
}

// A part's barriers, by one thread.
template <int kPartStages>
__device__ __forceinline__ void init_bars(uint64_t* full, uint64_t* empty, uint64_t* tfull, uint64_t* tempty, uint64_t* done) {
  for (int s = 0; s < kPartStages; ++s) {
    mbar_init(&full[s], 1);     // (the even CTA's is used: its producer arrives, both CTAs' copies count)
    mbar_init(&empty[s], 1);
  }
  for (int a = 0; a < 2; ++a) {
    mbar_init(&tfull[a], 1);
    mbar_init(&tempty[a], 2 * kEpiWarps);   // (the even CTA's: both CTAs' epilogue warps)
  }
  mbar_init(done, 1);
}

struct DxBars {
  uint64_t full[kDxStages], empty[kDxStages], tfull[2], tempty[2], done;
  uint64_t arrived[kEpiWarps * kDxSlots];   // of each epilogue warp's chunks: the residual is there
};
static_assert(sizeof(DxBars) == kDxNumBars * 8, "shared memory");

__device__ __forceinline__ void dx_init(uint8_t* smem, const DxMaps& maps) {
  DxBars* b = reinterpret_cast<DxBars*>(smem + kDxOffBars);
  init_bars<kDxStages>(b->full, b->empty, b->tfull, b->tempty, &b->done);
  for (int c = 0; c < kEpiWarps * kDxSlots; ++c) mbar_init(&b->arrived[c], 1);
  prefetch_tensormap(&maps.dz);
  prefetch_tensormap(&maps.w);
  prefetch_tensormap(&maps.out);
}

// kCentredRows: some expert's row is less m, and dz's sums times m are added.
template <bool kCentredRows>
__device__ __forceinline__ void dx_epilogue(uint8_t* smem, const DxMaps& maps, const DxArgs& g, int i0, uint32_t tmem) {
  DxBars* bars = reinterpret_cast<DxBars*>(smem + kDxOffBars);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffHolder + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  uint64_t *tfull = bars->tfull, *tempty = bars->tempty;
  const int items = g.t_tiles * g.k_tiles, i_step = g.pairs;
  // A lane holds a token; a warp takes half of the tile's columns, 64 at a time:
  // whole lines of memory.  The residual is copied to where the result is formed and
  // copied out from, in three places in turn: two chunks are on their way while one is
  // worked on.  (Loads to registers a tile ahead were waited for at the next barrier.)
  const int quad = warp & 3, half = (warp - 2) >> 2;
  uint8_t* slots = smem + kDxOffSlots + (warp - 2) * kDxSlots * kChunk;   // (128-byte rows, 128-byte swizzle)
  uint64_t* arrived = bars->arrived + (warp - 2) * kDxSlots;
  const int row0 = static_cast<int>(rank) * 128 + quad * 32;   // of this warp in a tile
  int next_i = i0;   // the chunk to be copied in next, and its place
  int next_c = 0, next_slot = 0;
  const auto copy_in = [&]() {
    if (!g.residual || next_i >= items) return;
    const DxItem it = dx_item(g, next_i);
    if (lane == 0) {
      mbar_arrive_expect_tx(&arrived[next_slot], kChunk);
      tma_load_3d(slots + next_slot * kChunk, &maps.res, &arrived[next_slot], it.k0 + half * (it.n / 2) + next_c * 64,
                  it.t0 + row0, 0);
    }
    next_slot = next_slot == kDxSlots - 1 ? 0 : next_slot + 1;
    if (++next_c == it.n / 128) {
      next_c = 0;
      next_i += i_step;
    }
  };
  for (int c = 0; c < kDxSlots; ++c) copy_in();
  int slot = 0;
  bool first = true;
  int iter = 0;
  bool ok = true;
  uint32_t phases = 0;   // the places' parities
  for (int i = i0; i < items && ok; i += i_step, ++iter) {
    const DxItem it = dx_item(g, i);
    const int acc = iter & 1;
    // this lane's token: its power of two, in two factors that are numbers of their own
    const int2 of = it.t0 + row0 + lane < g.T ? g.rows[it.t0 + row0 + lane] : make_int2(0, 0);
    const int exp = of.x;
    const float by0 = pow2(exp / 2), by1 = pow2(exp - exp / 2), sum = __int_as_float(of.y);
    ok = __all_sync(kAll, mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag, g.timeout_ns));
    if (!ok) break;
    tc_fence_after();
    const uint32_t taddr = tmem + static_cast<uint32_t>(acc * kDxTile + half * (it.n / 2)) + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
    for (int c = 0; c < it.n / 128; ++c) {
      uint8_t* place = slots + slot * kChunk;
      uint8_t* row = place + lane * 128;
      uint32_t v[2][32];
      tmem_ld_32x32b_x32(taddr + c * 64, v[0]);
      tmem_ld_32x32b_x32(taddr + c * 64 + 32, v[1]);
      uint4 m_words[kCentredRows ? 8 : 1];   // of the 64 columns, the same in every lane
      if constexpr (kCentredRows) {
#pragma unroll
        for (int j = 0; j < 8; ++j) m_words[j] = g.common[(it.k0 + half * (it.n / 2) + c * 64) / 8 + j];
      }
      if (g.residual) {
        ok = __all_sync(kAll, mbar_wait_bounded(&arrived[slot], (phases >> slot) & 1u, abort_flag, g.timeout_ns));
        if (!ok) break;
        phases ^= 1u << slot;
      } else {
        // the place's last store has read it
        if (lane == 0) asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(kDxSlots - 1) : "memory");
        __syncwarp();
      }
      tmem_ld_wait();
      if (c == it.n / 128 - 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint4* at = reinterpret_cast<uint4*>(row + ((j ^ (lane & 7)) << 4));
        const uint4 r = g.residual ? *at : make_uint4(0, 0, 0, 0);
        const uint32_t rw[4] = {r.x, r.y, r.z, r.w};
        uint32_t o[4];
        float common[8];
        if constexpr (kCentredRows) unpack8(m_words[j], common);
#pragma unroll
        for (int m = 0; m < 4; ++m) {
          const float2 f = unpack_bf16x2(rw[m]);
          const int e = 8 * (j & 3) + 2 * m;
          float a = __uint_as_float(v[j >> 2][e]) * by0 * by1, b = __uint_as_float(v[j >> 2][e + 1]) * by0 * by1;
          if constexpr (kCentredRows) {
            a = fmaf(sum, common[2 * m], a);
            b = fmaf(sum, common[2 * m + 1], b);
          }
          o[m] = pack_bf16x2(a + f.x, b + f.y);
        }
        *at = make_uint4(o[0], o[1], o[2], o[3]);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        // (tokens past T are clipped by the map; of some there must be one)
        if (it.t0 + row0 < g.T) tma_store_3d(&maps.out, place, it.k0 + half * (it.n / 2) + c * 64, it.t0 + row0, 0);
        bulk_commit_group();
        // the chunk before has been read by its store: its place is filled again
        if (g.residual && !first) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
      }
      __syncwarp();
      if (!first) copy_in();
      first = false;
      slot = slot == kDxSlots - 1 ? 0 : slot + 1;
    }
  }
  if (!ok) {
    set_status(g.status, MOE_ERR_TIMEOUT);
    *abort_flag = 1;
    leave_copies_time();
  }
  if (lane == 0) bulk_wait_all();   // this warp's stores have completed
}

// (Not inlined: beside the other form in one body it slowed that down, 2 us at 8192 x 7168 and
// 256 experts.  There a call takes 128 us with a common row, 107 without: m passes
// through shared memory's path to the registers too, 512 of a tile's cycles in bf16.)
__device__ __noinline__ void dx_epilogue_centred(uint8_t* smem, const DxMaps& maps, const DxArgs& g, int i0, uint32_t tmem) {
  const DxArgs mine = g;   // (in registers: read again after every barrier they cost 20 us more)
  dx_epilogue<true>(smem, maps, mine, i0, tmem);
}

// The work of CTA pair i0 of g.pairs.
__device__ __forceinline__ void dx_part(uint8_t* smem, const DxMaps& maps, const DxArgs& g, int i0, uint32_t tmem) {
  DxBars* bars = reinterpret_cast<DxBars*>(smem + kDxOffBars);
  uint64_t *full = bars->full, *empty = bars->empty, *tfull = bars->tfull, *tempty = bars->tempty, *done = &bars->done;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffHolder + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int items = g.t_tiles * g.k_tiles;
  const int i_step = g.pairs;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = i0; i < items && ok; i += i_step) {
      const DxItem it = dx_item(g, i);
      const int t = it.t0 + static_cast<int>(rank) * 128;
      const int k = it.k0 + static_cast<int>(rank) * (it.n / 2);
      const bool two = it.n == kDxTile;   // boxes of 64 columns for this CTA's half of W
      const uint32_t bytes = kDxPlane + (two ? 2 : 1) * kDxBox;
      for (int b = 0; b < g.e_blocks; ++b) {
        ok = __all_sync(kAll, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + stage * kDxStage;
        const uint32_t bar = mapa(smem_u32(&full[stage]), 0);
        if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * bytes);
        tma_load_3d_pair(a, &maps.dz, bar, b * kDxBlock, t, 0);
        // (weights' rows past the last expert arrive as zeros)
        tma_load_3d_pair(a + kDxPlane, &maps.w, bar, k, b * kDxBlock, 0);
        if (two) tma_load_3d_pair(a + kDxPlane + kDxBox, &maps.w, bar, k + 64, b * kDxBlock, 0);
        if (++stage == kDxStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {
      if (lane == 0) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      leave_copies_time();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    // (values broadcast from lane 0 are known to be uniform)
    if (__shfl_sync(kAll, rank, 0) == 0) {
      const uint32_t base = __shfl_sync(kAll, smem_u32(smem), 0);
      const uint32_t tm = __shfl_sync(kAll, tmem, 0);
      int stage = 0, iter = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = i0; i < items && ok; i += i_step, ++iter) {
        const DxItem it = dx_item(g, i);
        // D fp32, A and B fp16, B MN-major
        const uint32_t idesc = (1u << 4) | (1u << 16) |
                               (static_cast<uint32_t>(__shfl_sync(kAll, it.n, 0) >> 3) << 17) | ((256u >> 4) << 24);
        const int acc = iter & 1;
        ok = __all_sync(kAll, mbar_wait_cluster_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + static_cast<uint32_t>(acc * kDxTile);
        for (int b = 0; b < g.e_blocks; ++b) {
          ok = __all_sync(kAll, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = base + stage * kDxStage;
          const uint64_t ad = smem_desc(a, 16, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(a + kDxPlane, kDxBox, 1024, kSwizzle128B);
          // (16 experts on: 32 bytes along dz's rows, 16 rows of 128 bytes down W's boxes)
          mma_block_pair(d, ad, bd, 32 >> 4, 2048 >> 4, idesc, b != 0);
          tc_commit_pair(&empty[stage]);
          if (++stage == kDxStages) {
            stage = 0;
            phase ^= 1;
          }
        }
        if (!ok) break;
        tc_commit_pair(&tfull[acc]);
      }
      if (!ok && lane == 0) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // all issued tensor-core work finished before the tensor memory is released
      tc_commit_pair(done);
      const int never = 0;
      mbar_wait_bounded(done, 0, &never, g.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    bool centred = false;   // some expert's row is less m
    for (int e = lane; e < g.E; e += 32) centred |= is_centred(g.exps[e]);
    if (__any_sync(kAll, centred))
      dx_epilogue_centred(smem, maps, g, i0, tmem);
    else
      dx_epilogue<false>(smem, maps, g, i0, tmem);
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weights
// ---------------------------------------------------------------------------
constexpr int kSegment = 256;                    // tokens of a sum in tensor memory
constexpr int kSegBlocks = kSegment / kBlock;
constexpr int kTileK = 256;                      // columns of x of a pair's tile, 128 per CTA
constexpr int kTileE = 128;                      // experts of a tile, at most
constexpr int kStageBytes = 5 * kBoxBytes;       // x: two boxes; each plane of dz: one
constexpr int kStages = 5;
constexpr int kOffBars = kStages * kStageBytes;
constexpr int kNumBars = 2 * kStages + 5;
static_assert(kOffBars + kNumBars * 8 <= kOffHolder, "shared memory");

struct DwMaps {
  CUtensorMap x, dz;
};

struct DwArgs {
  int32_t pairs;           // CTA pairs that work on it
  int32_t E, Ep;
  int64_t K;
  int32_t segments;        // of 256 tokens
  int32_t k_tiles, e_tiles, parts;
  int32_t add;             // one part: dW is added to
  float* out;              // [parts][E][K]
  const float2* losses_of; // [n_losses] the losses' sums over eight tokens each
  int64_t n_losses;
  const int32_t* tokens;
  float* losses;           // [2] or null
  int32_t* status;
  uint64_t timeout_ns;
};

struct DwItem {
  int k0, e0, n;           // first column of x, first expert, experts of the MMA
  int seg0, seg1, part;
};

__device__ __forceinline__ DwItem dw_item(const DwArgs& g, int i) {
  DwItem it;
  const int tiles = g.k_tiles * g.e_tiles;
  it.part = i / tiles;
  const int tile = i - it.part * tiles;
  const int kt = tile / g.e_tiles;   // (experts innermost: they share x's blocks)
  it.k0 = kt * kTileK;
  it.e0 = (tile - kt * g.e_tiles) * kTileE;
  const int left = g.E - it.e0;
  it.n = left >= kTileE ? kTileE : (left + 31) & ~31;
  it.seg0 = static_cast<int>(static_cast<int64_t>(it.part) * g.segments / g.parts);
  it.seg1 = static_cast<int>(static_cast<int64_t>(it.part + 1) * g.segments / g.parts);
  return it;
}

// The losses from their parts, by one warp, in one order.
__device__ __noinline__ void sum_losses(const DwArgs& g, int lane) {
  double b = 0.0, z = 0.0;
  for (int64_t i = lane; i < g.n_losses; i += 32) {
    const float2 v = g.losses_of[i];
    b += v.x;
    z += v.y;
  }
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) {
    b += __shfl_xor_sync(kAll, b, o);
    z += __shfl_xor_sync(kAll, z, o);
  }
  const double n = max(*g.tokens, 1);
  if (lane == 0) {
    g.losses[0] = static_cast<float>(b * g.E / n);
    g.losses[1] = static_cast<float>(z / n);
  }
}

struct DwBars {
  uint64_t full[kStages], empty[kStages], tfull[2], tempty[2], done;
};
static_assert(sizeof(DwBars) == kNumBars * 8, "shared memory");

__device__ __forceinline__ void dw_init(uint8_t* smem, const DwMaps& maps) {
  DwBars* b = reinterpret_cast<DwBars*>(smem + kOffBars);
  init_bars<kStages>(b->full, b->empty, b->tfull, b->tempty, &b->done);
  prefetch_tensormap(&maps.x);
  prefetch_tensormap(&maps.dz);
}

// The work of CTA pair i0 of g.pairs.
__device__ __forceinline__ void dw_part(uint8_t* smem, const DwMaps& maps, const DwArgs& g, int i0, uint32_t tmem) {
  DwBars* bars = reinterpret_cast<DwBars*>(smem + kOffBars);
  uint64_t *full = bars->full, *empty = bars->empty, *tfull = bars->tfull, *tempty = bars->tempty, *done = &bars->done;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffHolder + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();
  const int items = g.k_tiles * g.e_tiles * g.parts;
  const int i_step = g.pairs;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int i = i0; i < items && ok; i += i_step) {
      const DwItem it = dw_item(g, i);
      const int k = it.k0 + static_cast<int>(rank) * 128;
      const int e = it.e0 + static_cast<int>(rank) * (it.n / 2);
      for (int b = it.seg0 * kSegBlocks; b < it.seg1 * kSegBlocks; ++b) {
        ok = __all_sync(kAll, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + stage * kStageBytes;
        const uint32_t bar = mapa(smem_u32(&full[stage]), 0);
        if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * kStageBytes);
        // (rows past T and columns past K arrive as zeros)
        tma_load_3d_pair(a, &maps.x, bar, k, b * kBlock, 0);
        tma_load_3d_pair(a + kBoxBytes, &maps.x, bar, k + 64, b * kBlock, 0);
#pragma unroll
        for (int p = 0; p < 3; ++p)
          tma_load_3d_pair(a + (2 + p) * kBoxBytes, &maps.dz, bar, p * g.Ep + e, b * kBlock, 0);
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok) {
      if (lane == 0) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      leave_copies_time();
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer (even CTA)
    // (values broadcast from lane 0 are known to be uniform)
    if (__shfl_sync(kAll, rank, 0) == 0) {
      const uint32_t base = __shfl_sync(kAll, smem_u32(smem), 0);
      const uint32_t tm = __shfl_sync(kAll, tmem, 0);
      int stage = 0, iter = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int i = i0; i < items && ok; i += i_step) {
        const DwItem it = dw_item(g, i);
        // D fp32, A and B bf16, both MN-major
        const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (1u << 15) | (1u << 16) |
                               (static_cast<uint32_t>(__shfl_sync(kAll, it.n, 0) >> 3) << 17) | ((256u >> 4) << 24);
        for (int s = it.seg0; s < it.seg1 && ok; ++s, ++iter) {
          const int acc = iter & 1;
          ok = __all_sync(kAll, mbar_wait_cluster_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
          if (!ok) break;
          tc_fence_after();
          const uint32_t hi = tm + static_cast<uint32_t>(acc * 2 * kTileE), rest = hi + kTileE;
          for (int b = 0; b < kSegBlocks; ++b) {
            ok = __all_sync(kAll, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
            if (!ok) break;
            tc_fence_after();
            const uint32_t a = base + stage * kStageBytes;
            const uint64_t ad = smem_desc(a, kBoxBytes, 1024, kSwizzle128B);
            const uint64_t bd = smem_desc(a + 2 * kBoxBytes, kBoxBytes, 1024, kSwizzle128B);
            // 16 tokens on: 16 rows of 128 bytes down the boxes
#pragma unroll
            for (int k = 0; k < kBlock / 16; ++k) {
              constexpr uint64_t kStep = 2048 >> 4, kPlane = kBoxBytes >> 4;
              const uint32_t more = !(b == 0 && k == 0);
              mma_bf16_pair(hi, ad + kStep * k, bd + kStep * k, idesc, more);
              mma_bf16_pair(rest, ad + kStep * k, bd + kPlane + kStep * k, idesc, more);
              mma_bf16_pair(rest, ad + kStep * k, bd + 2 * kPlane + kStep * k, idesc, 1u);
            }
            tc_commit_pair(&empty[stage]);
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1;
            }
          }
          if (!ok) break;
          tc_commit_pair(&tfull[acc]);
        }
      }
      if (!ok && lane == 0) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // all issued tensor-core work finished before the tensor memory is released
      tc_commit_pair(done);
      const int never = 0;
      mbar_wait_bounded(done, 0, &never, g.timeout_ns);
    }
  } else {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    const int quad = warp & 3, half = (warp - 2) >> 2;
    int iter = 0;
    bool ok = true;
    // (in the last CTA, which has no more items than any other, while its first MMAs run)
    if (g.losses && i0 == g.pairs - 1 && rank == 1 && warp == 2 + kEpiWarps - 1) sum_losses(g, lane);
    for (int i = i0; i < items && ok; i += i_step) {
      const DwItem it = dw_item(g, i);
      float run[64];   // of this lane's column of x: 64 experts' sums so far
#pragma unroll
      for (int j = 0; j < 64; ++j) run[j] = 0.0f;
      for (int s = it.seg0; s < it.seg1; ++s, ++iter) {
        const int acc = iter & 1;
        ok = __all_sync(kAll, mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag, g.timeout_ns));
        if (!ok) {
          set_status(g.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        if (64 * half < it.n) {
          const uint32_t taddr = tmem + static_cast<uint32_t>(acc * 2 * kTileE + half * 64) +
                                 (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll
          for (int c = 0; c < 2; ++c) {   // (columns past the MMA's hold old sums, which are not stored)
            uint32_t h[32], r[32];
            tmem_ld_32x32b_x32(taddr + c * 32, h);
            tmem_ld_32x32b_x32(taddr + kTileE + c * 32, r);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 32; ++j) run[32 * c + j] += __uint_as_float(h[j]) + __uint_as_float(r[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
      }
      if (!ok) break;
      const int64_t k = it.k0 + static_cast<int64_t>(rank) * 128 + quad * 32 + lane;
      const int e0 = it.e0 + half * 64;
      if (k >= g.K) continue;   // (K is a multiple of 128: whole warps)
      float* dst = g.out + (static_cast<int64_t>(it.part) * g.E + e0) * g.K + k;
#pragma unroll
      for (int j = 0; j < 64; ++j)
        if (e0 + j < g.E) dst[j * g.K] = g.add ? dst[j * g.K] + run[j] : run[j];
    }
  }
}

// dx on the first pairs, dW on the others.  (In launches of their own that ran side by side
// dW's read dz without having waited for it itself.)
__global__ void __launch_bounds__(kThreads, 1)
    router_products_kernel(const __grid_constant__ DxMaps dx_maps, const __grid_constant__ DxArgs dx,
                           const __grid_constant__ DwMaps dw_maps, const __grid_constant__ DwArgs dw) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);
  const int warp = threadIdx.x >> 5, pair = static_cast<int>(blockIdx.x >> 1);
  if (threadIdx.x == 0) {
    if (pair < dx.pairs)
      dx_init(smem, dx_maps);
    else
      dw_init(smem, dw_maps);
    *reinterpret_cast<volatile int*>(holder + 1) = 0;   // the abort flag
    fence_barrier_init();
  }
  if (warp == 1) {
    tmem_alloc_pair(holder, kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *holder;
  if (pair < dx.pairs)
    dx_part(smem, dx_maps, dx, pair, tmem);
  else
    dw_part(smem, dw_maps, dw, pair - dx.pairs, tmem);
  // neither CTA leaves while the other's copies, MMAs or arrivals may reach it
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

__global__ void __launch_bounds__(256) router_dw_sum_kernel(const float4* parts, int n_parts, int64_t n4, int add, float4* dw) {
  pdl_wait();
  pdl_trigger();
  const int64_t i = static_cast<int64_t>(blockIdx.x) * blockDim.x + threadIdx.x;
  if (i >= n4) return;
  float4 sum = add ? dw[i] : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 4
  for (int p = 0; p < n_parts; ++p) {
    const float4 v = parts[p * n4 + i];
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  dw[i] = sum;
}

// ---------------------------------------------------------------------------
// Host
// ---------------------------------------------------------------------------
int64_t up(int64_t n, int64_t to) { return (n + to - 1) / to * to; }
int64_t cuts(int64_t n, int64_t of) { return (n + of - 1) / of; }
int32_t fewer(int32_t pairs, int64_t items) { return items < pairs ? static_cast<int32_t>(items) : pairs; }

// dx and dW run side by side, each on its share of the 76 CTA pairs, dW's MMAs beside dx's
// way through memory and fewer pairs without work at the end of both (4096 tokens, K = 2048,
// 128 experts: 29.1 us after one another, 25.1 so; 8192, 7168, 256: 108.3 and 107.2).  The
// shares follow the cycles of a tile: its MMAs, for dx at least 3200 of its epilogue's, and
// what comes with each (1200 and 200).  dW's sum is cut into as many parts as make its
// rounds' time least, with the parts' way through memory (about 3 KB a cycle, and a
// launch).  All from sizes alone, so that a sum has one order.
constexpr int kPairs = 76;
struct Shares {
  int dx_pairs, dw_pairs, parts;
};
Shares shares(int64_t T, int64_t K, int32_t E) {
  const int64_t dx_tiles = cuts(T, kDxTile) * cuts(K, kDxTile), dx_mma = cuts(E, kDxBlock) * 517;
  const int64_t dx_cycles = (dx_mma > 3200 ? dx_mma : 3200) + 1200;
  const int64_t segments = cuts(T, kSegment), tiles = cuts(K, kTileK) * cuts(E, kTileE);
  const int64_t cycles = kSegBlocks * 6 * (E >= kTileE ? kTileE : up(E, 32)) + 200;
  const double dx_cost = static_cast<double>(dx_tiles) * dx_cycles, dw_cost = static_cast<double>(tiles) * segments * cycles;
  Shares r;
  r.dx_pairs = static_cast<int>(kPairs * dx_cost / (dx_cost + dw_cost) + 0.5);
  r.dx_pairs = r.dx_pairs < 1 ? 1 : r.dx_pairs > kPairs - 1 ? kPairs - 1 : r.dx_pairs;
  r.dw_pairs = kPairs - r.dx_pairs;
  r.parts = 1;
  int64_t least = 0;
  for (int s = 1; s <= 32 && s <= segments; ++s) {
    const int64_t time = cuts(tiles * s, r.dw_pairs) * cuts(segments, s) * cycles + (s > 1 ? 4000 + s * E * K * 8 / 3000 : 0);
    if (s == 1 || time < least) {
      least = time;
      r.parts = s;
    }
  }
  return r;
}

// What the workspace holds, from its start.
struct Places {
  int64_t counts, tokens, exps, parts, common, rows, planes, half, w_half, sums, total;
  Shares shares;
};
Places places(int64_t T, int64_t K, int32_t E) {
  Places p;
  p.tokens = 16;       // (the status word first)
  p.counts = 64;
  p.exps = p.counts + 4 * static_cast<int64_t>(E);
  p.parts = up(p.exps + 4 * static_cast<int64_t>(E), 256);
  p.common = up(p.parts + 8 * cuts(T, kDzWarps), 256);
  p.rows = up(p.common + 2 * K, 256);
  p.planes = up(p.rows + 8 * T, 256);
  p.half = up(p.planes + T * 3 * up(E, 64) * 2, 256);
  p.w_half = up(p.half + T * up(E, 64) * 2, 256);
  p.sums = up(p.w_half + static_cast<int64_t>(E) * K * 2, 256);
  p.shares = shares(T, K, E);
  p.total = p.sums + (p.shares.parts > 1 ? 4 * p.shares.parts * static_cast<int64_t>(E) * K : 0);
  return p;
}

template <int Q>
cudaError_t launch_dz(const DzArgs& g, cudaStream_t s) {
  return launch_pdl(route_dz_kernel<Q>, dim3(static_cast<unsigned>(cuts(g.T, kDzWarps))), dim3(32 * kDzWarps), 0, s, g);
}

bool off(const void* p, uintptr_t by) { return (reinterpret_cast<uintptr_t>(p) & (by - 1)) != 0; }

// [rows][cols] of 16 bits, boxes of box_rows x 64.
moe_status_t box_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, uint32_t box_rows,
                     CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), 1};
  const uint64_t st[2] = {static_cast<uint64_t>(cols) * 2, static_cast<uint64_t>(cols * rows) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_tiled_map(m, p, type, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

#define MOE_TRY(call)                              \
  do {                                             \
    if ((call) != cudaSuccess) return MOE_ERR_CUDA; \
  } while (0)

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int64_t moe_route_backward_workspace_size(int64_t T, int64_t K, int32_t E_global) {
  if (T < 0 || K <= 0 || E_global <= 0) return -1;
  return places(T, K, E_global).total;
}

moe_status_t moe_route_backward(const void* x_bf16, const void* w_planes, const float* logits, const int32_t* topk_ids,
                                const float* topk_weights, const float* dweights, int64_t T, int64_t K,
                                int32_t E_global, int32_t topk, double balance, double zloss, const void* residual,
                                void* dx_bf16, float* dw, int32_t accumulate, float* dlogits, float* losses, void* ws,
                                int64_t ws_bytes, void* stream) {
  return moe_route_backward_kept(x_bf16, w_planes, logits, topk_ids, topk_weights, dweights, nullptr, T, K, E_global, topk,
                                 balance, zloss, residual, dx_bf16, dw, accumulate, dlogits, losses, ws, ws_bytes, stream);
}

moe_status_t moe_route_backward_kept(const void* x_bf16, const void* w_planes, const float* logits,
                                     const int32_t* topk_ids, const float* topk_weights, const float* dweights,
                                     const uint8_t* kept, int64_t T, int64_t K, int32_t E_global, int32_t topk,
                                     double balance, double zloss, const void* residual, void* dx_bf16, float* dw,
                                     int32_t accumulate, float* dlogits, float* losses, void* ws, int64_t ws_bytes,
                                     void* stream) {
  const int32_t E = E_global;
  if (T < 0 || K <= 0 || E <= 0 || topk <= 0) return MOE_ERR_INVALID_ARG;
  if (K % 128 || K > (int64_t(1) << 30) || E > kMaxRouterExperts || topk > kMaxTopk || topk > E || T > (int64_t(1) << 30) ||
      T * topk > 0x7FFFFFFF || cuts(T, kDxTile) * cuts(K, kDxTile) > 0x3FFFFFFF)
    return MOE_ERR_UNSUPPORTED;
  if (!w_planes || !dw || !ws) return MOE_ERR_INVALID_ARG;
  if (T > 0 && (!x_bf16 || !logits || !topk_ids || !topk_weights || !dweights || !dx_bf16)) return MOE_ERR_INVALID_ARG;
  for (const void* p : {x_bf16, w_planes, residual, static_cast<const void*>(dx_bf16), static_cast<const void*>(dw),
                        static_cast<const void*>(ws)})
    if (off(p, 16)) return MOE_ERR_MISALIGNED;
  for (const void* p : {static_cast<const void*>(logits), static_cast<const void*>(topk_ids),
                        static_cast<const void*>(topk_weights), static_cast<const void*>(dweights),
                        static_cast<const void*>(dlogits), static_cast<const void*>(losses)})
    if (off(p, 4)) return MOE_ERR_MISALIGNED;
  const Places at = places(T, K, E);
  if (ws_bytes < at.total) return MOE_ERR_BUFFER_TOO_SMALL;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  uint8_t* base = static_cast<uint8_t*>(ws);
  int32_t* status = reinterpret_cast<int32_t*>(base);
  if (T == 0) {   // no token: no gradient
    MOE_TRY(cudaMemsetAsync(status, 0, 16, s));
    if (!accumulate) MOE_TRY(cudaMemsetAsync(dw, 0, 4 * E * K, s));
    if (losses) MOE_TRY(cudaMemsetAsync(losses, 0, 8, s));
    return MOE_OK;
  }
  const int32_t Ep = static_cast<int32_t>(up(E, 64));
  uint16_t* planes = reinterpret_cast<uint16_t*>(base + at.planes);
  DwMaps maps;
  moe_status_t st;
  if ((st = box_map(&maps.x, x_bf16, T, K, kBlock)) != MOE_OK) return st;
  if ((st = box_map(&maps.dz, planes, T, 3 * Ep, kBlock)) != MOE_OK) return st;
  DxMaps dx_maps;
  uint16_t* half = reinterpret_cast<uint16_t*>(base + at.half);
  uint16_t* w_half = reinterpret_cast<uint16_t*>(base + at.w_half);
  int32_t* exps = reinterpret_cast<int32_t*>(base + at.exps);
  uint4* common = reinterpret_cast<uint4*>(base + at.common);
  int2* rows = reinterpret_cast<int2*>(base + at.rows);
  if ((st = box_map(&dx_maps.dz, half, T, Ep, 128, CU_TENSOR_MAP_DATA_TYPE_FLOAT16)) != MOE_OK) return st;
  if ((st = box_map(&dx_maps.w, w_half, E, K, kDxBlock, CU_TENSOR_MAP_DATA_TYPE_FLOAT16)) != MOE_OK) return st;
  if ((st = box_map(&dx_maps.out, dx_bf16, T, K, 32)) != MOE_OK) return st;
  if ((st = box_map(&dx_maps.res, residual ? residual : dx_bf16, T, K, 32)) != MOE_OK) return st;

  int32_t* counts = reinterpret_cast<int32_t*>(base + at.counts);
  int32_t* tokens = reinterpret_cast<int32_t*>(base + at.tokens);
  const uint4* w = static_cast<const uint4*>(w_planes);
  const PrepareArgs prepare = {topk_ids, kept, T, topk, E, counts, tokens, status, w, K / 8, common,
                               reinterpret_cast<uint4*>(w_half), exps};
  MOE_TRY(launch_pdl_cluster(route_prepare_kernel, dim3(static_cast<unsigned>(kCountCtas + up(E, kCountCtas))),
                             dim3(kPrepareThreads), 0, s, kCountCtas, prepare));
  DzArgs z = {logits, topk_ids, topk_weights, dweights, kept, T, E, Ep, topk, static_cast<float>(balance),
              static_cast<float>(zloss), counts, tokens, exps, planes, half, rows, dlogits,
              reinterpret_cast<float2*>(base + at.parts)};
  MOE_TRY((E <= 64 ? launch_dz<1> : E <= 128 ? launch_dz<2> : E <= 256 ? launch_dz<4> : E <= 512 ? launch_dz<8>
                                                                                            : launch_dz<16>)(z, s));
  DxArgs d;
  memset(&d, 0, sizeof(d));
  d.Ep = Ep;
  d.e_blocks = static_cast<int32_t>(cuts(E, kDxBlock));
  d.t_tiles = static_cast<int32_t>(cuts(T, kDxTile));
  d.k_tiles = static_cast<int32_t>(cuts(K, kDxTile));
  d.T = T;
  d.K = K;
  d.rows = rows;
  d.exps = exps;
  d.common = common;
  d.E = E;
  d.residual = residual != nullptr;
  d.status = status;
  d.timeout_ns = 2000000000ull;
  d.pairs = fewer(at.shares.dx_pairs, static_cast<int64_t>(d.t_tiles) * d.k_tiles);

  DwArgs g;
  memset(&g, 0, sizeof(g));
  g.E = E;
  g.Ep = Ep;
  g.K = K;
  g.segments = static_cast<int32_t>(cuts(T, kSegment));
  g.k_tiles = static_cast<int32_t>(cuts(K, kTileK));
  g.e_tiles = static_cast<int32_t>(cuts(E, kTileE));
  g.parts = at.shares.parts;
  g.add = g.parts == 1 && accumulate;
  g.out = g.parts == 1 ? dw : reinterpret_cast<float*>(base + at.sums);
  g.losses_of = z.parts;
  g.n_losses = cuts(T, kDzWarps);
  g.tokens = tokens;
  g.losses = losses;
  g.status = status;
  g.timeout_ns = 2000000000ull;
  g.pairs = fewer(at.shares.dw_pairs, static_cast<int64_t>(g.k_tiles) * g.e_tiles * g.parts);
  static PerDevice known;
  int resident = 0;   // (no pair waits for another: more than fit run one after another)
  MOE_TRY(on_current_device(known, &resident, [](int* n) { return resident_pairs(router_products_kernel, kThreads, kSmem, n); }));
  MOE_TRY(launch_pdl_cluster(router_products_kernel, dim3(2 * static_cast<unsigned>(d.pairs + g.pairs)), dim3(kThreads), kSmem,
                             s, 2, dx_maps, d, maps, g));
  if (g.parts > 1) {
    const int64_t n4 = static_cast<int64_t>(E) * K / 4;
    MOE_TRY(launch_pdl(router_dw_sum_kernel, dim3(static_cast<unsigned>(cuts(n4, 256))), dim3(256), 0, s,
                       reinterpret_cast<const float4*>(g.out), g.parts, n4, accumulate != 0, reinterpret_cast<float4*>(dw)));
  }
  return MOE_OK;
}

}  // extern "C"
