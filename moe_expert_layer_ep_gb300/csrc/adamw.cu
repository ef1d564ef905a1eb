// One AdamW step over many tensors (moe_adamw_create, moe_adamw_step).  No
// counterpart in the PR reports.
//
//   g' = grad_scale * g
//   m  = beta1 m + (1 - beta1) g'          v = beta2 v + (1 - beta2) g'^2
//   p  = p (1 - lr wd) - lr / (1 - beta1^t) * m / (sqrt(v) / sqrt(1 - beta2^t) + eps)
//
// States in 32 bits, or in 8: each 256 consecutive elements of a tensor share
// two fp32 scales, the largest |m| and the largest v among them.  A code
// holds a root of the value's share of that scale, which spends the 8 bits on
// small values as well as on large ones: m as sgn(m) rn(127 sqrt(|m| / s)),
// 1.6 % apart at the top and down to 6e-5 of it, v as rn(255 (v / s)^(1/4)),
// 1.6 % apart at the top and down to 2e-10.  v > 0 never becomes code 0: a
// second moment rounded to nothing would leave m / eps as the step.  The
// update itself uses the unrounded fp32 m and v of the step.
//
// Bound by memory: every value is read once and written once.  A warp holds
// one 256-element block in registers (two runs of 128 elements, four per
// lane, so every access is a whole contiguous run), finds the block's largest
// values by shuffles and writes codes and scales.  The tensors' table travels
// in the kernel's parameters (up to kMaxTensors of one kind of tensor per
// launch): nothing is copied to the device, and a step can be captured.
#include <math.h>
#include <string.h>

#include <new>
#include <vector>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kAdamThreads = 256;
constexpr int kStateBlock = 256;
constexpr int kMaxTensors = 384;
constexpr int64_t kChunkSmall = 2048;    // elements per CTA: one block per warp
constexpr int64_t kChunkLarge = 8192;

struct AdamTable {
  void* p[kMaxTensors];
  const void* g[kMaxTensors];
  void* m[kMaxTensors];
  void* v[kMaxTensors];
  float* ms[kMaxTensors];
  float* vs[kMaxTensors];
  float* master[kMaxTensors];
  int64_t n[kMaxTensors];
  uint32_t chunk_end[kMaxTensors];   // chunks of tensors 0..i
  uint8_t wide[kMaxTensors];         // every array starts on a boundary of four elements
  int32_t count;
  int32_t chunk;                     // elements
};

struct AdamHyper {
  float b1, omb1, b2, omb2, inv_root, eps, decay, step;
  const float* grad_scale;
};

template <typename T>
__device__ __forceinline__ void load4(const void* base, int64_t i, int64_t n, bool whole, float (&f)[4]);
template <>
__device__ __forceinline__ void load4<float>(const void* base, int64_t i, int64_t n, bool whole, float (&f)[4]) {
  const float* b = static_cast<const float*>(base) + i;
  if (whole) {
    const float4 r = *reinterpret_cast<const float4*>(b);
    f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = i + k < n ? b[k] : 0.0f;
  }
}
template <>
__device__ __forceinline__ void load4<uint16_t>(const void* base, int64_t i, int64_t n, bool whole, float (&f)[4]) {
  const uint16_t* b = static_cast<const uint16_t*>(base) + i;
  if (whole) {
    const uint2 r = *reinterpret_cast<const uint2*>(b);
    const float2 x = unpack_bf16x2(r.x), y = unpack_bf16x2(r.y);
    f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k) f[k] = i + k < n ? __uint_as_float(static_cast<uint32_t>(b[k]) << 16) : 0.0f;
  }
}

template <typename T>
__device__ __forceinline__ void store4(void* base, int64_t i, int64_t n, bool whole, const float (&f)[4]);
template <>
__device__ __forceinline__ void store4<float>(void* base, int64_t i, int64_t n, bool whole, const float (&f)[4]) {
  float* b = static_cast<float*>(base) + i;
  if (whole) {
    *reinterpret_cast<float4*>(b) = make_float4(f[0], f[1], f[2], f[3]);
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) b[k] = f[k];
  }
}
template <>
__device__ __forceinline__ void store4<uint16_t>(void* base, int64_t i, int64_t n, bool whole, const float (&f)[4]) {
  uint16_t* b = static_cast<uint16_t*>(base) + i;
  if (whole) {
    *reinterpret_cast<uint2*>(b) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) b[k] = __bfloat16_as_ushort(__float2bfloat16_rn(f[k]));
  }
}

// Four codes as one word, and back.
__device__ __forceinline__ uint32_t load_codes(const void* base, int64_t i, int64_t n, bool whole) {
  const uint8_t* b = static_cast<const uint8_t*>(base) + i;
  if (whole) return *reinterpret_cast<const uint32_t*>(b);
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    if (i + k < n) w |= static_cast<uint32_t>(b[k]) << (8 * k);
  return w;
}
__device__ __forceinline__ void store_codes(void* base, int64_t i, int64_t n, bool whole, uint32_t w) {
  uint8_t* b = static_cast<uint8_t*>(base) + i;
  if (whole) {
    *reinterpret_cast<uint32_t*>(b) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) b[k] = static_cast<uint8_t>(w >> (8 * k));
  }
}

// Largest of non-negative values over the warp.  As bit patterns, so that a
// NaN (above every number there) is kept: the block's scale then is a NaN and
// so are its states from there on, not silently zero.
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}

// A block's scale from its largest value: at least the smallest normal
// number, so that its reciprocal is finite.
__device__ __forceinline__ float block_scale(float top) { return top > 0.0f ? fmaxf(top, 1.17549435e-38f) : top; }

// P, G: float or uint16_t (bf16).  Rounded operations are written one by one
// (no contraction), so that codes next to a rounding boundary do not depend on
// how the compiler fuses them.
template <typename P, typename G, bool kMaster, bool kCoded>
__global__ void __launch_bounds__(kAdamThreads) adamw_kernel(const __grid_constant__ AdamTable t, const AdamHyper h) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t c = blockIdx.x;
  int lo = 0, hi = t.count - 1;   // first tensor whose chunks end after c
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (t.chunk_end[mid] > c)
      hi = mid;
    else
      lo = mid + 1;
  }
  const uint32_t first = lo ? t.chunk_end[lo - 1] : 0;
  const int64_t n = t.n[lo];
  const bool wide = t.wide[lo] != 0;
  const int64_t begin = static_cast<int64_t>(c - first) * t.chunk;
  const int64_t end = min(begin + t.chunk, n);
  void* p = t.p[lo];
  const void* g = t.g[lo];
  void* m = t.m[lo];
  void* v = t.v[lo];
  float* master = t.master[lo];
  pdl_wait();
  pdl_trigger();
  const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
  for (int64_t b = begin + warp * kStateBlock; b < end; b += kAdamThreads / 32 * kStateBlock) {
    const bool whole = wide && b + kStateBlock <= n;
    float fp[2][4], fg[2][4], fm[2][4], fv[2][4];
    uint32_t cm[2], cv[2];
    float sm = 0.0f, sv = 0.0f;
    if (kCoded) {
      sm = t.ms[lo][b / kStateBlock];
      sv = t.vs[lo][b / kStateBlock];
    }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t i = b + 128 * r + 4 * lane;
      if (kMaster)
        load4<float>(master, i, n, whole, fp[r]);
      else
        load4<P>(p, i, n, whole, fp[r]);
      load4<G>(g, i, n, whole, fg[r]);
      if (kCoded) {
        cm[r] = load_codes(m, i, n, whole);
        cv[r] = load_codes(v, i, n, whole);
      } else {
        load4<float>(m, i, n, whole, fm[r]);
        load4<float>(v, i, n, whole, fv[r]);
      }
    }
    float top_m = 0.0f, top_v = 0.0f;
    float root[2][4];   // sqrt(v)
#pragma unroll
    for (int r = 0; r < 2; ++r)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (kCoded) {
          const float a = __fmul_rn(static_cast<float>(static_cast<int8_t>(cm[r] >> (8 * k))), 1.0f / 127.0f);
          fm[r][k] = __fmul_rn(__fmul_rn(a, fabsf(a)), sm);
          float q = __fmul_rn(static_cast<float>((cv[r] >> (8 * k)) & 0xFFu), 1.0f / 255.0f);
          q = __fmul_rn(q, q);
          fv[r][k] = __fmul_rn(__fmul_rn(q, q), sv);
        }
        const float x = __fmul_rn(fg[r][k], gs);
        fm[r][k] = __fadd_rn(__fmul_rn(fm[r][k], h.b1), __fmul_rn(x, h.omb1));
        fv[r][k] = __fadd_rn(__fmul_rn(fv[r][k], h.b2), __fmul_rn(__fmul_rn(x, x), h.omb2));
        root[r][k] = __fsqrt_rn(fv[r][k]);
        const float denom = __fadd_rn(__fmul_rn(root[r][k], h.inv_root), h.eps);
        fp[r][k] = __fsub_rn(__fmul_rn(fp[r][k], h.decay), __fmul_rn(__fdiv_rn(fm[r][k], denom), h.step));
        if (kCoded) {
          top_m = __uint_as_float(max(__float_as_uint(top_m), __float_as_uint(fabsf(fm[r][k]))));
          top_v = __uint_as_float(max(__float_as_uint(top_v), __float_as_uint(fabsf(fv[r][k]))));
        }
      }
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int64_t i = b + 128 * r + 4 * lane;
      store4<P>(p, i, n, whole, fp[r]);
      if (kMaster) store4<float>(master, i, n, whole, fp[r]);
      if (!kCoded) {
        store4<float>(m, i, n, whole, fm[r]);
        store4<float>(v, i, n, whole, fv[r]);
      }
    }
    if (kCoded) {
      const float nm = block_scale(warp_max(top_m)), nv = block_scale(warp_max(top_v));
      const float im = nm > 0.0f ? __fdiv_rn(1.0f, nm) : 0.0f;
      const float iv = __fsqrt_rn(nv > 0.0f ? __fdiv_rn(1.0f, nv) : 0.0f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        uint32_t wm = 0, wv = 0;
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          int qm = __float2int_rn(__fmul_rn(__fsqrt_rn(__fmul_rn(fabsf(fm[r][k]), im)), 127.0f));
          qm = min(qm, 127);
          if (fm[r][k] < 0.0f) qm = -qm;
          int qv = __float2int_rn(__fmul_rn(__fsqrt_rn(__fmul_rn(root[r][k], iv)), 255.0f));
          qv = min(max(qv, fv[r][k] > 0.0f ? 1 : 0), 255);
          wm |= static_cast<uint32_t>(qm & 0xFF) << (8 * k);
          wv |= static_cast<uint32_t>(qv) << (8 * k);
        }
        const int64_t i = b + 128 * r + 4 * lane;
        store_codes(m, i, n, whole, wm);
        store_codes(v, i, n, whole, wv);
      }
      if (lane == 0) {
        t.ms[lo][b / kStateBlock] = nm;
        t.vs[lo][b / kStateBlock] = nv;
      }
    }
  }
}

using AdamKernel = void (*)(const AdamTable, const AdamHyper);

// kind: bit 0 bf16 parameters, bit 1 bf16 gradients, bit 2 a 32-bit copy, bit 3 states in 8 bits
template <typename P, typename G>
AdamKernel kernel_pg(int kind) {
  constexpr bool kCanMaster = sizeof(P) == 2;
  if (kind & 8)
    return (kind & 4) ? adamw_kernel<P, G, kCanMaster, true> : adamw_kernel<P, G, false, true>;
  return (kind & 4) ? adamw_kernel<P, G, kCanMaster, false> : adamw_kernel<P, G, false, false>;
}
AdamKernel adam_kernel(int kind) {
  if (kind & 1) return (kind & 2) ? kernel_pg<uint16_t, uint16_t>(kind) : kernel_pg<uint16_t, float>(kind);
  return (kind & 2) ? kernel_pg<float, uint16_t>(kind) : kernel_pg<float, float>(kind);
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

}  // namespace

}  // namespace moe

struct moe_adamw {
  struct Launch {
    int kind;
    uint32_t chunks;
    moe::AdamTable table;
  };
  std::vector<Launch> launches;
};

namespace {

moe_status_t check_tensor(const moe_adamw_tensor_t& t) {
  if (t.n < 0) return MOE_ERR_INVALID_ARG;
  if ((t.param_elem != MOE_ELEM_BF16 && t.param_elem != MOE_ELEM_F32) ||
      (t.grad_elem != MOE_ELEM_BF16 && t.grad_elem != MOE_ELEM_F32) || (t.state_bits != 32 && t.state_bits != 8))
    return MOE_ERR_INVALID_ARG;
  if (t.n == 0) return MOE_OK;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return MOE_ERR_INVALID_ARG;
  const bool coded = t.state_bits == 8;
  if (coded != (t.avg_scale != nullptr) || coded != (t.sq_scale != nullptr)) return MOE_ERR_DTYPE_MISMATCH;
  if (t.master && t.param_elem != MOE_ELEM_BF16) return MOE_ERR_DTYPE_MISMATCH;
  const uintptr_t pa = t.param_elem == MOE_ELEM_F32 ? 4 : 2, ga = t.grad_elem == MOE_ELEM_F32 ? 4 : 2;
  if (moe::misaligned(t.param, pa) || moe::misaligned(t.grad, ga) || moe::misaligned(t.master, 4) ||
      moe::misaligned(t.avg_scale, 4) || moe::misaligned(t.sq_scale, 4))
    return MOE_ERR_MISALIGNED;
  if (!coded && (moe::misaligned(t.exp_avg, 4) || moe::misaligned(t.exp_avg_sq, 4))) return MOE_ERR_MISALIGNED;
  return MOE_OK;
}

// Whether every array of the tensor starts on a boundary of four elements.
bool is_wide(const moe_adamw_tensor_t& t) {
  const uintptr_t p = t.param_elem == MOE_ELEM_F32 ? 16 : 8, g = t.grad_elem == MOE_ELEM_F32 ? 16 : 8;
  const uintptr_t s = t.state_bits == 32 ? 16 : 4;
  return !moe::misaligned(t.param, p) && !moe::misaligned(t.grad, g) && !moe::misaligned(t.master, 16) &&
         !moe::misaligned(t.exp_avg, s) && !moe::misaligned(t.exp_avg_sq, s);
}

void add_launch(moe_adamw* a, int kind, const std::vector<const moe_adamw_tensor_t*>& ts) {
  int64_t total = 0;
  for (const auto* t : ts) total += t->n;
  a->launches.emplace_back();
  moe_adamw::Launch& l = a->launches.back();
  memset(&l.table, 0, sizeof(l.table));
  l.kind = kind;
  l.table.count = static_cast<int32_t>(ts.size());
  l.table.chunk = static_cast<int32_t>(total > (int64_t(1) << 23) ? moe::kChunkLarge : moe::kChunkSmall);
  uint32_t end = 0;
  for (size_t i = 0; i < ts.size(); ++i) {
    const moe_adamw_tensor_t& t = *ts[i];
    l.table.p[i] = t.param;
    l.table.g[i] = t.grad;
    l.table.m[i] = t.exp_avg;
    l.table.v[i] = t.exp_avg_sq;
    l.table.ms[i] = t.avg_scale;
    l.table.vs[i] = t.sq_scale;
    l.table.master[i] = t.master;
    l.table.n[i] = t.n;
    l.table.wide[i] = is_wide(t);
    end += static_cast<uint32_t>((t.n + l.table.chunk - 1) / l.table.chunk);
    l.table.chunk_end[i] = end;
  }
  l.chunks = end;
}

}  // namespace

extern "C" {

moe_status_t moe_adamw_create(const moe_adamw_tensor_t* tensors, int32_t count, moe_adamw** out) {
  if (!out) return MOE_ERR_INVALID_ARG;
  *out = nullptr;
  if (count < 0 || (count > 0 && !tensors)) return MOE_ERR_INVALID_ARG;
  for (int32_t i = 0; i < count; ++i) {
    const moe_status_t st = check_tensor(tensors[i]);
    if (st != MOE_OK) return st;
    // chunks of one launch are numbered in 32 bits
    if (tensors[i].n > (int64_t(1) << 40)) return MOE_ERR_UNSUPPORTED;
  }
  try {
    moe_adamw* a = new moe_adamw;
    try {
      for (int kind = 0; kind < 16; ++kind) {
        std::vector<const moe_adamw_tensor_t*> ts;
        int64_t elems = 0;
        for (int32_t i = 0; i < count; ++i) {
          const moe_adamw_tensor_t& t = tensors[i];
          const int k = (t.param_elem == MOE_ELEM_BF16 ? 1 : 0) | (t.grad_elem == MOE_ELEM_BF16 ? 2 : 0) |
                        (t.master ? 4 : 0) | (t.state_bits == 8 ? 8 : 0);
          if (k != kind || t.n == 0) continue;
          if (ts.size() == static_cast<size_t>(moe::kMaxTensors) || (!ts.empty() && elems + t.n > (int64_t(1) << 41))) {
            add_launch(a, kind, ts);
            ts.clear();
            elems = 0;
          }
          ts.push_back(&t);
          elems += t.n;
        }
        if (!ts.empty()) add_launch(a, kind, ts);
      }
    } catch (...) {
      delete a;
      throw;
    }
    *out = a;
  } catch (...) {
    return MOE_ERR_INVALID_ARG;   // host memory
  }
  return MOE_OK;
}

void moe_adamw_destroy(moe_adamw* opt) { delete opt; }

int32_t moe_adamw_launches(const moe_adamw* opt) { return opt ? static_cast<int32_t>(opt->launches.size()) : -1; }

moe_status_t moe_adamw_step(const moe_adamw* opt, const moe_adamw_hyper_t* h, const float* grad_scale, void* stream) {
  if (!opt || !h) return MOE_ERR_INVALID_ARG;
  if (h->step < 1 || !(h->beta1 >= 0.0 && h->beta1 < 1.0) || !(h->beta2 >= 0.0 && h->beta2 < 1.0) ||
      !(h->eps >= 0.0) || !isfinite(h->eps) || !isfinite(h->lr) || !isfinite(h->weight_decay))
    return MOE_ERR_INVALID_ARG;
  if (moe::misaligned(grad_scale, 4)) return MOE_ERR_MISALIGNED;
  moe::AdamHyper a;
  const double t = static_cast<double>(h->step);
  a.b1 = static_cast<float>(h->beta1);
  a.omb1 = static_cast<float>(1.0 - h->beta1);
  a.b2 = static_cast<float>(h->beta2);
  a.omb2 = static_cast<float>(1.0 - h->beta2);
  a.inv_root = static_cast<float>(1.0 / sqrt(1.0 - pow(h->beta2, t)));
  a.eps = static_cast<float>(h->eps);
  a.decay = static_cast<float>(1.0 - h->lr * h->weight_decay);
  a.step = static_cast<float>(h->lr / (1.0 - pow(h->beta1, t)));
  a.grad_scale = grad_scale;
  for (const moe_adamw::Launch& l : opt->launches) {
    const cudaError_t e = moe::launch_pdl(moe::adam_kernel(l.kind), dim3(l.chunks), dim3(moe::kAdamThreads), 0,
                                          static_cast<cudaStream_t>(stream), l.table, a);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
