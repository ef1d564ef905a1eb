// Dense products of few tiles (a shared expert's on new tokens, a small layer's).
//
// A CTA takes 64 features (M of the MMA; gated: 32 of g and the same 32 of u) of the
// whole reduction and at most 64 rows (its N, 8 to 64): 2048 features are 32 CTAs, where
// tiles of 256 features on CTA pairs are 16, and there is no pair to set up.  The sum of an
// output runs over the reduction in the same steps of the tensor cores as there, so a
// row's bits are those of the larger batches; splitting the reduction over CTAs here alone
// would change them (segments of one length in every dense kernel would not).
//
// What bounds it.  One row of 7168 by 2048 features takes 14 us (those tiles 26.5; the
// weights' bytes 4.3), by 7168 features 18.3 (28.9; 15.1), 2048 by 7168 7.7 (12.5; 4.3).  A
// CTA's 448 MMAs take 49 cycles each, whatever N, whether they add to one accumulator or
// to four, and whatever else is left out: 11.5 us of the first.  Less per MMA: 72 cycles
// where each was issued and each block waited for by itself (19.9 us).  Tiles of 32 or 16
// features (more CTAs, fewer bytes each), and four blocks in one copy, changed nothing.
//
// The accumulator (features in lanes: M = 64 occupies the first 16 lanes of each 32) goes
// through shared memory, from where 128 threads form whole pieces of output rows.
#include "few_rows.h"

#include <string.h>

#include "activation.cuh"

namespace moe {

namespace {

constexpr unsigned kAll = 0xFFFFFFFFu;
constexpr int kBlockK = 64;                      // elements: 128 bytes, one swizzle atom
constexpr int kABytes = 64 * kBlockK * 2;        // 8 KB of weights
constexpr int kGroup = 4;                        // reduction blocks of a stage
constexpr int kMaxStages = 5;
constexpr int kRing = 192 * 1024;                // bytes of all stages, at most
constexpr int kTileFloats = static_cast<int>(kFewRows) * 64;   // a tile's sums, [row][feature]
constexpr int kOffSums = kRing;
constexpr int kOffBars = kOffSums + 2 * kTileFloats * 4;
constexpr int kNumBars = 2 * kMaxStages + 5;
constexpr int kOffHolder = kOffBars + kNumBars * 8;
constexpr int kSmem = kOffHolder + 16 + 1024;
static_assert(kSmem <= 227 * 1024, "shared memory");
constexpr int kEpiThreads = 128;
constexpr int kThreads = 64 + kEpiThreads;       // producer, MMA, epilogue
constexpr uint32_t kTmemCols = 128;              // two accumulators
constexpr int kAhead = 4;                        // output pieces of a thread whose inputs are read at a time

// The four MMAs of a block, issued by a converged warp through one elected lane (see
// pair.cuh): one election for all of them.
__device__ __forceinline__ void mma_block_elect(uint32_t d, uint64_t a, uint64_t b, uint64_t a_step, uint32_t idesc,
                                                uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %5, 0;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t"
      "add.s64 x, %1, %4;\n\tadd.s64 y, %2, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t"
      "add.s64 x, x, %4;\n\tadd.s64 y, y, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t"
      "add.s64 x, x, %4;\n\tadd.s64 y, y, 2;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, 1;\n\t}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "l"(a_step), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit_elect(uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
__device__ __forceinline__ void expect_elect(uint64_t* bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(smem_u32(bar)),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void load_elect(void* dst, const CUtensorMap* map, uint64_t* bar, int32_t c0, int32_t c1) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];\n\t}" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(c0), "r"(c1), "r"(0)
      : "memory");
}
// All epilogue threads' barrier; true where ok is in all of them.
__device__ __forceinline__ bool epilogue_all(bool ok) {
  uint32_t all;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.and.pred q, 1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(all)
      : "r"(static_cast<uint32_t>(ok)), "n"(kEpiThreads)
      : "memory");
  return all != 0;
}

__device__ __forceinline__ float bias_at(const FewRows& g, int64_t i) {
  return g.bias_f32 ? static_cast<const float*>(g.bias)[i]
                    : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(g.bias)[i]) << 16);
}

struct FewMaps {
  CUtensorMap w, x;
};

template <FewWay kWay>
__global__ void __launch_bounds__(kThreads, 1)
    few_rows_kernel(const __grid_constant__ FewMaps maps, const __grid_constant__ FewRows g) {
  constexpr bool kGrad = kWay == kFewGrad || kWay == kFewGradGlu, kGatedFwd = kWay == kFewFwdGlu;
  constexpr int kFeatures = kGatedFwd ? 32 : 64;   // output features of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBars);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffHolder + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < g.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], kEpiThreads / 32);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.x);
  }
  if (warp == 1) {
    tmem_alloc(holder, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  pdl_wait();
  pdl_trigger();
  const uint32_t block_bytes = kABytes + g.n * 128;   // (n is a multiple of 8: whole 1024 bytes)

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    int stage = 0;
    uint32_t phase = 0, issued = 0, parity = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < g.tiles && ok; t += gridDim.x) {
      const int f = t / g.row_tiles * kFeatures, r = t % g.row_tiles * static_cast<int>(kFewRows);
      for (int k0 = 0; k0 < g.k_blocks; k0 += kGroup) {
        const int blocks = min(kGroup, g.k_blocks - k0);
        ok = __all_sync(kAll, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + stage * kGroup * block_bytes;
        expect_elect(&full[stage], blocks * block_bytes);
        for (int kb = k0; kb < k0 + blocks; ++kb, a += block_bytes) {
          if constexpr (kGatedFwd) {
            load_elect(a, &maps.w, &full[stage], kb * kBlockK, f);
            load_elect(a + kABytes / 2, &maps.w, &full[stage], kb * kBlockK, static_cast<int>(g.cols) + f);
          } else if constexpr (kGrad) {
            load_elect(a, &maps.w, &full[stage], f, kb * kBlockK);
          } else {
            load_elect(a, &maps.w, &full[stage], kb * kBlockK, f);
          }
          load_elect(a + kABytes, &maps.x, &full[stage], kb * kBlockK, r);
        }
        issued |= 1u << stage;
        parity = (parity & ~(1u << stage)) | (phase << stage);
        if (++stage == g.stages) {
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
      // never leave the CTA with copies still landing in its shared memory
      const int never = 0;
      for (int s = 0; s < g.stages; ++s)
        if (issued & (1u << s)) mbar_wait_bounded(&full[s], (parity >> s) & 1u, &never, g.timeout_ns);
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    const uint32_t base = __shfl_sync(kAll, smem_u32(smem), 0);
    const uint32_t tm = __shfl_sync(kAll, tmem, 0);
    // D fp32, A and B bf16, M = 64
    const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | (kGrad ? 1u << 15 : 0u) |
                           (static_cast<uint32_t>(g.n >> 3) << 17) | ((64u >> 4) << 24);
    int stage = 0, iter = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < g.tiles && ok; t += gridDim.x, ++iter) {
      const int acc = iter & 1;
      ok = __all_sync(kAll, mbar_wait_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
      if (!ok) break;
      tc_fence_after();
      const uint32_t d = tm + static_cast<uint32_t>(acc * 64);
      for (int k0 = 0; k0 < g.k_blocks; k0 += kGroup) {
        ok = __all_sync(kAll, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t a = base + stage * kGroup * block_bytes;
        // 16 reduction elements on: 32 bytes along a K-major row, 16 rows of 128 bytes
        // down an MN-major box
#pragma unroll
        for (int b = 0; b < kGroup; ++b)
          if (k0 + b < g.k_blocks)
            mma_block_elect(d, smem_desc(a + b * block_bytes, 16, 1024, kSwizzle128B),
                            smem_desc(a + b * block_bytes + kABytes, 16, 1024, kSwizzle128B), (kGrad ? 2048 : 32) >> 4, idesc,
                            k0 + b != 0);
        commit_elect(&empty[stage]);
        if (++stage == g.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
      if (!ok) break;
      commit_elect(&tfull[acc]);
    }
    if (!ok && lane == 0) {
      set_status(g.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    // all issued tensor-core work finished before the tensor memory is released
    commit_elect(done);
    const int never = 0;
    mbar_wait_bounded(done, 0, &never, g.timeout_ns);
  } else {
    // ------------------------------------------------------------------ epilogue
    const int tid = threadIdx.x - 64, quad = warp & 3;
    constexpr int kPairs = kFeatures / 2;                 // a thread's two features, and its first row
    const int pair = tid % kPairs, row0 = tid / kPairs;
    constexpr int kRowStep = kEpiThreads / kPairs;
    float* sums = reinterpret_cast<float*>(smem + kOffSums);
    int iter = 0;
    for (int t = blockIdx.x; t < g.tiles; t += gridDim.x, ++iter) {
      const int acc = iter & 1;
      const int64_t first_row = static_cast<int64_t>(t % g.row_tiles) * kFewRows;   // (row tiles innermost: they share weights)
      const int rows = static_cast<int>(g.rows - first_row < kFewRows ? g.rows - first_row : kFewRows);
      const int64_t col = static_cast<int64_t>(t / g.row_tiles) * kFeatures + 2 * pair;
      const bool there = col < g.cols;   // (cols is a multiple of 8)
      // what is added is read while the MMAs run, the first rows' all of it
      float2 b = make_float2(0.0f, 0.0f), bu = b;
      if constexpr (!kGrad) {
        if (g.bias && there) {
          b = make_float2(bias_at(g, col), bias_at(g, col + 1));
          if constexpr (kGatedFwd) bu = make_float2(bias_at(g, g.cols + col), bias_at(g, g.cols + col + 1));
        }
      }
      uint32_t r[kAhead], z[kAhead], u[kAhead];
      const auto read = [&](int first) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          const int row = first + i * kRowStep;
          r[i] = z[i] = u[i] = 0;
          if (!there || row >= rows) continue;
          const int64_t at = first_row + row;
          if constexpr (kWay == kFewFwd || kWay == kFewGrad)
            if (g.res) r[i] = *reinterpret_cast<const uint32_t*>(g.res + at * g.res_ld + col);
          if constexpr (kGrad)
            if (g.z) z[i] = *reinterpret_cast<const uint32_t*>(g.z + at * g.z_ld + col);
          if constexpr (kWay == kFewGradGlu) u[i] = *reinterpret_cast<const uint32_t*>(g.z + at * g.z_ld + g.cols + col);
        }
      };
      read(row0);
      const bool ok = __all_sync(kAll, mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag,
                                                         g.timeout_ns + static_cast<uint64_t>(g.k_blocks) * 4000u));
      float* tile = sums + acc * kTileFloats;
      if (ok) {
        tc_fence_after();
        const uint32_t taddr = tmem + static_cast<uint32_t>(acc * 64) + (static_cast<uint32_t>(quad * 32) << 16);
        for (int c = 0; c < g.n; c += 32) {
          uint32_t v[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          tmem_ld_wait();
          if (lane < 16) {
#pragma unroll
            for (int j = 0; j < 32; ++j)
              if (c + j < rows) tile[(c + j) * 64 + quad * 16 + lane] = __uint_as_float(v[j]);
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
      // (the tile's other buffer is free again once all threads are here)
      if (!epilogue_all(ok)) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      for (int first = row0; first < rows; first += kAhead * kRowStep) {
        if (first != row0) read(first);
        if (!there) continue;
        with_act(g.act, [&](auto tag) {
          constexpr int kA = decltype(tag)::value;
#pragma unroll
          for (int i = 0; i < kAhead; ++i) {
            const int row = first + i * kRowStep;
            if (row >= rows) break;
            const int64_t at_row = first_row + row;
            float2 s = *reinterpret_cast<const float2*>(tile + row * 64 + 2 * pair);
            uint16_t* out = g.out + at_row * g.out_ld + col;
            if constexpr (kWay == kFewFwdGlu) {
              float2 p = *reinterpret_cast<const float2*>(tile + row * 64 + 32 + 2 * pair);
              if (g.bias) {   // (nothing is added where there is nothing: -0 + 0 is 0)
                s = make_float2(s.x + b.x, s.y + b.y);
                p = make_float2(p.x + bu.x, p.y + bu.y);
              }
              if (g.keep) {
                uint16_t* keep = g.keep + at_row * g.keep_ld + col;
                *reinterpret_cast<uint32_t*>(keep) = pack_bf16x2(s.x, s.y);
                *reinterpret_cast<uint32_t*>(keep + g.cols) = pack_bf16x2(p.x, p.y);
              }
              *reinterpret_cast<uint32_t*>(out) =
                  pack_bf16x2(act_at<kA, false>(s.x, nullptr) * p.x, act_at<kA, false>(s.y, nullptr) * p.y);
            } else if constexpr (kWay == kFewGradGlu) {
              const float2 gate = unpack_bf16x2(z[i]), up = unpack_bf16x2(u[i]);
              float2 slope, value;
              value.x = act_at<kA, true>(gate.x, &slope.x);
              value.y = act_at<kA, true>(gate.y, &slope.y);
              *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(s.x * up.x * slope.x, s.y * up.y * slope.y);
              *reinterpret_cast<uint32_t*>(out + g.cols) = pack_bf16x2(s.x * value.x, s.y * value.y);
            } else {
              if constexpr (kWay == kFewFwd) {
                if (g.bias) s = make_float2(s.x + b.x, s.y + b.y);
                if (g.keep) *reinterpret_cast<uint32_t*>(g.keep + at_row * g.keep_ld + col) = pack_bf16x2(s.x, s.y);
                s = make_float2(act_at<kA, false>(s.x, nullptr), act_at<kA, false>(s.y, nullptr));
              } else if constexpr (kA != MOE_ACT_NONE) {
                const float2 at = unpack_bf16x2(z[i]);
                float2 slope;
                act_at<kA, true>(at.x, &slope.x);
                act_at<kA, true>(at.y, &slope.y);
                s = make_float2(__fmul_rn(s.x, slope.x), __fmul_rn(s.y, slope.y));
              }
              if (g.res) {
                const float2 a = unpack_bf16x2(r[i]);
                s = make_float2(__fadd_rn(s.x, a.x), __fadd_rn(s.y, a.y));
              }
              *reinterpret_cast<uint32_t*>(out) = pack_bf16x2(s.x, s.y);
            }
          }
        });
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// [rows][cols] bf16 with row stride ld, boxes of 64 columns x box_rows.
moe_status_t box_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), 1};
  const uint64_t st[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(ld) * static_cast<uint64_t>(rows) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_tiled_map(m, p, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <FewWay kWay>
cudaError_t launch(const FewMaps& maps, const FewRows& g, cudaStream_t s) {
  static PerDevice known;
  int sms = 0;
  const cudaError_t e = on_current_device(known, &sms, [](int* n) {
    const cudaError_t set = cudaFuncSetAttribute(few_rows_kernel<kWay>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    int device = 0;
    if (set != cudaSuccess) return set;
    const cudaError_t got = cudaGetDevice(&device);
    return got != cudaSuccess ? got : cudaDeviceGetAttribute(n, cudaDevAttrMultiProcessorCount, device);
  });
  if (e != cudaSuccess) return e;
  return launch_pdl(few_rows_kernel<kWay>, dim3(static_cast<unsigned>(g.tiles < sms ? g.tiles : sms)), dim3(kThreads), kSmem, s,
                    maps, g);
}

}  // namespace

moe_status_t launch_few_rows(FewWay way, FewRows g, const void* x, int64_t x_ld, int64_t red, const void* w, void* stream) {
  const bool grad = way == kFewGrad || way == kFewGradGlu;
  const int64_t tile = way == kFewFwdGlu ? 32 : 64;
  g.n = g.rows > kFewRows ? static_cast<int32_t>(kFewRows) : (g.rows + 7) / 8 * 8;
  g.row_tiles = static_cast<int32_t>((g.rows + kFewRows - 1) / kFewRows);
  g.k_blocks = static_cast<int32_t>((red + kBlockK - 1) / kBlockK);
  g.tiles = g.row_tiles * static_cast<int32_t>((g.cols + tile - 1) / tile);
  const int fit = kRing / (kGroup * (kABytes + g.n * 128));
  g.stages = fit < kMaxStages ? fit : kMaxStages;
  g.timeout_ns = 2000000000ull;
  FewMaps maps;
  moe_status_t st = grad ? box_map(&maps.w, w, red, g.cols, g.cols, 64)
                         : box_map(&maps.w, w, way == kFewFwdGlu ? 2 * g.cols : g.cols, red, red, static_cast<uint32_t>(tile));
  if (st != MOE_OK) return st;
  if ((st = box_map(&maps.x, x, g.rows, red, x_ld, static_cast<uint32_t>(g.n))) != MOE_OK) return st;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  switch (way) {
    case kFewFwd: e = launch<kFewFwd>(maps, g, s); break;
    case kFewFwdGlu: e = launch<kFewFwdGlu>(maps, g, s); break;
    case kFewGrad: e = launch<kFewGrad>(maps, g, s); break;
    case kFewGradGlu: e = launch<kFewGradGlu>(maps, g, s); break;
  }
  return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace moe
