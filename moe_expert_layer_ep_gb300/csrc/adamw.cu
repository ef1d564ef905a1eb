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
// A gradient whose square is beyond fp32 makes v infinite, and m / inf is no
// step: the parameter only decays, then and later, and in 8 bits so do those of
// its block, whose scale is infinite (code 0 stays v = 0).
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
#include <type_traits>
#include <vector>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

constexpr int kStateBlock = 256;
constexpr int kMaxTensors = 384;
// Threads of a CTA.  Narrow CTAs over short runs of memory suit the 8-bit states,
// whose arithmetic and loads have to overlap across CTAs: 302 M bf16 elements with
// a 32-bit copy took 855 us in CTAs of 128 threads, 822 us in 64 and 717 us in 32
// (28 per SM; the copy bandwidth alone needs 715 us).  With 32-bit states 151 M
// bf16 elements took 501 us in 64 threads and 487 us in 256, of 16 blocks a warp.
__host__ __device__ constexpr int adam_threads(bool coded) { return coded ? 32 : 256; }
// Elements of its chunk: one block per warp, but 16 with 8-bit states (the next
// block is then loaded ahead of this one's arithmetic) from 5 M elements on.  In us
// for one and for 16, 8-bit states with a 32-bit copy: 1 M 5.2 and 13, 4.2 M 18.0
// and 20.2, 5 M 21.3 and 21.6, 8.4 M 34.8 and 29.2, 151 M 598 and 368; without: 5 M
// 21.3 and 20.3, 151 M 598 and 334.  32-bit states: 1 M 5.2 and 15.9, 16.8 M 55.7
// and 67.8, 151 M 470 and 487; with the copy 602 and 623.
__host__ __device__ constexpr int32_t chunk_small(bool coded) { return adam_threads(coded) / 32 * kStateBlock; }
constexpr int32_t chunk_large(bool coded) { return chunk_small(coded) * (coded ? 16 : 1); }
constexpr int64_t kLarge = 5000000;

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
  float b1, omb1, b2, omb2, inv_root, eps, decay, neg_step;
  const float* grad_scale;
};

// Four consecutive elements as loaded, zeros past n.
template <typename T>
struct Raw4;
template <>
struct Raw4<float> {
  float4 r;
  __device__ __forceinline__ void load(const void* base, int32_t i, int32_t n, bool whole) {
    const float* b = static_cast<const float*>(base) + i;
    if (whole)
      r = *reinterpret_cast<const float4*>(b);
    else
      r = make_float4(i < n ? b[0] : 0.0f, i + 1 < n ? b[1] : 0.0f, i + 2 < n ? b[2] : 0.0f, i + 3 < n ? b[3] : 0.0f);
  }
  __device__ __forceinline__ void open(float (&f)[4]) const { f[0] = r.x; f[1] = r.y; f[2] = r.z; f[3] = r.w; }
};
template <>
struct Raw4<uint16_t> {
  uint2 r;
  __device__ __forceinline__ void load(const void* base, int32_t i, int32_t n, bool whole) {
    const uint16_t* b = static_cast<const uint16_t*>(base) + i;
    if (whole) {
      r = *reinterpret_cast<const uint2*>(b);
    } else {
      uint32_t e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = i + k < n ? b[k] : 0u;
      r = make_uint2(e[0] | (e[1] << 16), e[2] | (e[3] << 16));
    }
  }
  __device__ __forceinline__ void open(float (&f)[4]) const {
    const float2 x = unpack_bf16x2(r.x), y = unpack_bf16x2(r.y);
    f[0] = x.x; f[1] = x.y; f[2] = y.x; f[3] = y.y;
  }
};
// Four codes.
template <>
struct Raw4<uint8_t> {
  uint32_t r;
  __device__ __forceinline__ void load(const void* base, int32_t i, int32_t n, bool whole) {
    const uint8_t* b = static_cast<const uint8_t*>(base) + i;
    if (whole) {
      r = *reinterpret_cast<const uint32_t*>(b);
    } else {
      r = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (i + k < n) r |= static_cast<uint32_t>(b[k]) << (8 * k);
    }
  }
};

template <typename T>
__device__ __forceinline__ void store4(void* base, int32_t i, int32_t n, bool whole, const float (&f)[4]);
template <>
__device__ __forceinline__ void store4<float>(void* base, int32_t i, int32_t n, bool whole, const float (&f)[4]) {
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
__device__ __forceinline__ void store4<uint16_t>(void* base, int32_t i, int32_t n, bool whole, const float (&f)[4]) {
  uint16_t* b = static_cast<uint16_t*>(base) + i;
  if (whole) {
    *reinterpret_cast<uint2*>(b) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) b[k] = __bfloat16_as_ushort(__float2bfloat16_rn(f[k]));
  }
}

__device__ __forceinline__ void store_codes(void* base, int32_t i, int32_t n, bool whole, uint32_t w) {
  uint8_t* b = static_cast<uint8_t*>(base) + i;
  if (whole) {
    *reinterpret_cast<uint32_t*>(b) = w;
  } else {
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (i + k < n) b[k] = static_cast<uint8_t>(w >> (8 * k));
  }
}

// Largest of non-negative values over the warp, as bit patterns (NaN is above
// every number there).
__device__ __forceinline__ float warp_max(float x) {
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(x)));
}

constexpr float kTiny = 1.17549435e-38f;   // 2^-126, the smallest normal number
constexpr float kMaxFloat = 3.40282347e+38f;

// A block's scale from its largest value: at least the smallest normal
// number, so that its reciprocal is finite.
__device__ __forceinline__ float block_scale(float top) { return top > 0.0f ? fmaxf(top, kTiny) : top; }

// Square root of a normal number: the hardware's reciprocal root (2 ulp), and
// one Newton step of the root on the residual x - s s, which the fused multiply-add
// forms exactly.  Correctly rounded for every number from 2^-100 up, one ulp off
// in places below (compared with the rounded function over all of them by
// tests/test_gpu_adamw_math.py), in half of that function's instructions.  The codes
// depend on it: next to a rounding boundary an ulp more or less is another code.
// (NaN of infinity, whose reciprocal root is 0.)
__device__ __forceinline__ float sqrt_newton(float x) {
  float y;
  asm("rsqrt.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  const float s = x * y;
  return fmaf(fmaf(-s, s, x), 0.5f * y, s);
}
// The same, of infinity and NaN too.
__device__ __forceinline__ float sqrt_any(float x) {
  const float s = sqrt_newton(x);
  return x <= kMaxFloat ? s : x;
}
// Reciprocal within 2 ulp, of a normal number.
__device__ __forceinline__ float rcp_fast(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// The larger, or NaN if either is one: a block with a NaN gets a NaN scale, and
// its states are NaN from there on, not silently zero.
__device__ __forceinline__ float max_nan(float a, float b) {
  float y;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}

// Byte k of a word of codes as a float less `bias`, without the conversion
// unit: the byte becomes the low mantissa bits of 2^23.
template <int kBias>
__device__ __forceinline__ float byte_value(uint32_t w, int k) {
  return __uint_as_float(__byte_perm(w, 0x4B000000u, 0x7540u + k)) - static_cast<float>(8388608 + kBias);
}
constexpr float kMagic = 12582912.0f;   // 1.5 * 2^23
// Low bytes of four words.  x + kMagic (|x| < 2^22) has the nearest integer to
// x, ties to even, in its low mantissa bits, so these are codes modulo 256.
__device__ __forceinline__ uint32_t low_bytes(float a, float b, float c, float d) {
  const uint32_t lo = __byte_perm(__float_as_uint(a), __float_as_uint(b), 0x0040u);
  const uint32_t hi = __byte_perm(__float_as_uint(c), __float_as_uint(d), 0x0040u);
  return __byte_perm(lo, hi, 0x5410u);
}

// One tensor's arrays, from a chunk's first element.
struct Arrays {
  char *p, *m, *v;
  const char* g;
  float *ms, *vs, *master;
  int32_t n;   // elements of the tensor from there, as far as they matter to the chunk
};

// What a lane loads of the 256-element block at element b of the chunk: twice
// four elements of each array.  kWhole: the block is complete and its arrays
// are aligned, so all accesses are wide; else element by element.
template <typename P, typename G, bool kMaster, bool kCoded, bool kWhole>
struct Block {
  Raw4<typename std::conditional<kMaster, float, P>::type> p[2];
  Raw4<G> g[2];
  Raw4<typename std::conditional<kCoded, uint8_t, float>::type> m[2], v[2];
  float sm, sv;   // kCoded: the block's scales
  __device__ __forceinline__ void load(const Arrays& t, int32_t b, int lane) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int32_t e = b + 128 * r + 4 * lane;
      p[r].load(kMaster ? reinterpret_cast<const char*>(t.master) : t.p, e, t.n, kWhole);
      g[r].load(t.g, e, t.n, kWhole);
      m[r].load(t.m, e, t.n, kWhole);
      v[r].load(t.v, e, t.n, kWhole);
    }
    if (kCoded) {
      sm = t.ms[b / kStateBlock];
      sv = t.vs[b / kStateBlock];
    }
  }
  // The step on this block's values, and its stores.
  __device__ __forceinline__ void step(const Arrays& t, const AdamHyper& h, float gs, int32_t b, int lane) const {
    float top_m = 0.0f, top_v = 0.0f;
    float fm[2][4], fv[2][4], root[2][4];   // root: sqrt(v), of at least the smallest normal number
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float fp[4], fg[4];
      p[r].open(fp);
      g[r].open(fg);
      if constexpr (kCoded) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float a = byte_value<128>(m[r].r ^ 0x80808080u, k) * (1.0f / 127.0f);
          float q = byte_value<0>(v[r].r, k) * (1.0f / 255.0f);
          q = q * q;
          fm[r][k] = a * fabsf(a) * sm;
          fv[r][k] = q * q * sv;
        }
        if (sv > kMaxFloat) {   // (the whole warp; 0 inf is no number, and code 0 no second moment)
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (((v[r].r >> (8 * k)) & 0xFFu) == 0) fv[r][k] = 0.0f;
        }
      } else {
        m[r].open(fm[r]);
        v[r].open(fv[r]);
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        // each product and sum rounded by itself (no contraction), as a
        // step in elementary 32-bit operations does
        const float x = __fmul_rn(fg[k], gs);
        fm[r][k] = __fadd_rn(__fmul_rn(fm[r][k], h.b1), __fmul_rn(x, h.omb1));
        fv[r][k] = __fadd_rn(__fmul_rn(fv[r][k], h.b2), __fmul_rn(__fmul_rn(x, x), h.omb2));
        root[r][k] = sqrt_any(max_nan(fv[r][k], kTiny));
        const float denom = fmaf(root[r][k], h.inv_root, h.eps);
        // (m by the quotient first: m times the step's length may be beyond fp32)
        fp[k] = fmaf(fm[r][k] * rcp_fast(denom), h.neg_step, fp[k] * h.decay);
        if (kCoded) {
          top_m = max_nan(top_m, fabsf(fm[r][k]));
          top_v = max_nan(top_v, fv[r][k]);
        }
      }
      const int32_t i = b + 128 * r + 4 * lane;
      store4<P>(t.p, i, t.n, kWhole, fp);
      if (kMaster) store4<float>(t.master, i, t.n, kWhole, fp);
      if (!kCoded) {
        store4<float>(t.m, i, t.n, kWhole, fm[r]);
        store4<float>(t.v, i, t.n, kWhole, fv[r]);
      }
    }
    if (kCoded) {
      const float nm = block_scale(warp_max(top_m)), nv = block_scale(warp_max(top_v));
      const float im = nm > 0.0f ? __fdiv_rn(1.0f, nm) : 0.0f;
      const float iv = __fsqrt_rn(nv > 0.0f ? __fdiv_rn(1.0f, nv) : 0.0f);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float qm[4], qv[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          qm[k] = __fadd_rn(__fmul_rn(copysignf(sqrt_newton(fmaxf(fabsf(fm[r][k]) * im, kTiny)), fm[r][k]), 127.0f),
                            kMagic);
          // 255 (v / s)^(1/4), at least 1
          const float q = __fadd_rn(fmaxf(__fmul_rn(sqrt_newton(fmaxf(root[r][k] * iv, kTiny)), 255.0f), 1.0f), kMagic);
          qv[k] = fv[r][k] > 0.0f ? q : 0.0f;
        }
        const int32_t i = b + 128 * r + 4 * lane;
        store_codes(t.m, i, t.n, kWhole, low_bytes(qm[0], qm[1], qm[2], qm[3]));
        store_codes(t.v, i, t.n, kWhole, low_bytes(qv[0], qv[1], qv[2], qv[3]));
      }
      if (lane == 0) {
        t.ms[b / kStateBlock] = nm;
        t.vs[b / kStateBlock] = nv;
      }
    }
  }
};

// P, G: float or uint16_t (bf16).
template <typename P, typename G, bool kMaster, bool kCoded>
__global__ void __launch_bounds__(adam_threads(kCoded), kCoded ? 28 : 3)
    adamw_kernel(const __grid_constant__ AdamTable t, const AdamHyper h) {
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
  const int64_t begin = static_cast<int64_t>(c - (lo ? t.chunk_end[lo - 1] : 0)) * t.chunk;
  const int64_t left = t.n[lo] - begin;
  Arrays a;
  a.n = static_cast<int32_t>(left < t.chunk ? left : t.chunk);
  a.p = static_cast<char*>(t.p[lo]) + begin * sizeof(P);
  a.g = static_cast<const char*>(t.g[lo]) + begin * sizeof(G);
  a.m = static_cast<char*>(t.m[lo]) + begin * (kCoded ? 1 : 4);
  a.v = static_cast<char*>(t.v[lo]) + begin * (kCoded ? 1 : 4);
  a.ms = kCoded ? t.ms[lo] + begin / kStateBlock : nullptr;
  a.vs = kCoded ? t.vs[lo] + begin / kStateBlock : nullptr;
  a.master = kMaster ? t.master[lo] + begin : nullptr;
  // complete blocks by wide accesses, the rest (or all, of arrays that do not
  // start on a boundary of four elements) element by element
  const int32_t whole_end = t.wide[lo] ? a.n / kStateBlock * kStateBlock : 0;
  constexpr int32_t kStep = chunk_small(kCoded);
  int32_t b = warp * kStateBlock;
  pdl_wait();
  pdl_trigger();
  const float gs = h.grad_scale ? *h.grad_scale : 1.0f;
  if (kCoded) {
    // states in 8 bits take enough arithmetic that the next block has to be on
    // its way meanwhile; in 32 bits, more warps serve better
    Block<P, G, kMaster, kCoded, true> cur, next;
    if (b < whole_end) cur.load(a, b, lane);
    for (; b < whole_end; b += kStep) {
      if (b + kStep < whole_end) next.load(a, b + kStep, lane);
      cur.step(a, h, gs, b, lane);
      cur = next;
    }
  } else {
    for (; b < whole_end; b += kStep) {
      Block<P, G, kMaster, kCoded, true> cur;
      cur.load(a, b, lane);
      cur.step(a, h, gs, b, lane);
    }
  }
  for (; b < a.n; b += kStep) {
    Block<P, G, kMaster, kCoded, false> cur;
    cur.load(a, b, lane);
    cur.step(a, h, gs, b, lane);
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
  l.table.chunk = total >= moe::kLarge ? moe::chunk_large(kind & 8) : moe::chunk_small(kind & 8);
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
  a.neg_step = static_cast<float>(-h->lr / (1.0 - pow(h->beta1, t)));
  a.grad_scale = grad_scale;
  for (const moe_adamw::Launch& l : opt->launches) {
    const cudaError_t e = moe::launch_pdl(moe::adam_kernel(l.kind), dim3(l.chunks), dim3(moe::adam_threads(l.kind & 8)), 0,
                                          static_cast<cudaStream_t>(stream), l.table, a);
    if (e != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
