// The experts' products on sorted rows and their gradients, on tcgen05 / TMEM
// fed by TMA (moe_expert_gemm and its variants).  No counterpart in the PR
// reports, whose products serve a fixed layer's forward pass only.
//
// For the rows r of expert e (bf16 operands, fp32 sums, one rounding):
//   kFwd          y[r]  = x[r] W_e^T                      W_e [N, C]
//   kFwdSwiglu    [g|u] = x[r] W_e^T, h[r] = silu(g) u    W_e [2I, C]
//   kDgrad        dx[r] = dy[r] W_e
//   kDgradSwiglu  dh    = dy[r] W_e, then with s = 1 / (1 + exp(-g)):
//                 dg = dh u s (1 + g (1 - s)),  du = dh g s
//   kWgrad        dW_e  = sum over r of dy[r]^T x[r]      (0 without rows)
//
// All are 128 x 256 output tiles summed over 64-element blocks of the
// reduction, and differ in which operand's reduction runs along memory rows:
//   kFwd    A = x (K-major)        B = W (K-major)
//   kDgrad  A = dy (K-major)       B = W (MN-major: the output column runs along W's rows)
//   kWgrad  A = dy (MN-major)      B = x (MN-major), reduction over the expert's rows
// A K-major tile is one box of 64 elements x rows; an MN-major tile is one
// 64 x 64 box per 64 output rows / columns, so no operand is ever transposed
// in memory.  Everything is read where the forward pass left it.
//
// An expert's rows are any consecutive rows (start, counts), 128 of them per
// row block.  Rows of a block beyond the expert's are multiplied like the
// others (they only make output rows that are not stored); in kWgrad, where
// rows are summed over, the last reduction block's rows beyond the expert's are
// cleared in shared memory before the product, so whatever lies there, NaN
// included, does not count.
//
// One persistent CTA per SM: warp 0 TMA producer, warp 1 MMA issue, warps 2-5
// epilogue (one per 32 accumulator rows), four stages of 48 KB, two
// accumulators so that a tile's epilogue runs beside the next tile's MMAs.
// The epilogue warps are independent: a warp whose 32 rows all exist stores
// through its own shared-memory tiles and TMA, others row by row.
#include <string.h>

#include <initializer_list>

#include "common.cuh"
#include "internal.h"

namespace moe {

namespace {

enum ExpertOp { kFwd, kFwdSwiglu, kDgrad, kDgradSwiglu, kWgrad };

constexpr int kStages = 4;
constexpr int kTileM = 128;
constexpr int kTileN = 256;
constexpr int kBlockK = 64;                          // elements: 128 bytes, one swizzle atom
constexpr int kABytes = kTileM * kBlockK * 2;        // 16 KB
constexpr int kBBytes = kTileN * kBlockK * 2;        // 32 KB
constexpr int kBoxBytes = 64 * kBlockK * 2;          // an MN-major box: 64 x 64 elements
constexpr int kEpiWarps = 4;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kStgTile = 32 * 64;                    // a store tile: 32 rows x 32 columns
constexpr int kStgPerWarp = 3;
constexpr uint32_t kTmemCols = 512;

constexpr int kOffA = 0;
constexpr int kOffB = kOffA + kStages * kABytes;
constexpr int kOffStg = kOffB + kStages * kBBytes;
constexpr int kOffBar = kOffStg + kEpiWarps * kStgPerWarp * kStgTile;
constexpr int kNumBars = 2 * kStages + 5;            // full, empty; tfull[2], tempty[2]; done
constexpr int kOffHolder = kOffBar + kNumBars * 8;
constexpr int kOffAbort = kOffHolder + 4;
constexpr int kOffScan = kOffAbort + 4;              // warps' sums of the block scan
constexpr int kOffCum = kOffScan + 64;               // row blocks of the experts before e, [E + 1]
constexpr int kSmemBytes = kOffCum + 4 * (kMaxLocalExperts + 1) + 1024;   // + alignment slack
static_assert(kSmemBytes <= 227 * 1024, "shared memory");

constexpr uint32_t kIdesc = (1u << 4)       // D fp32
                            | (1u << 7)     // A bf16
                            | (1u << 10)    // B bf16
                            | (static_cast<uint32_t>(kTileN >> 3) << 17) | (static_cast<uint32_t>(kTileM >> 4) << 24);
constexpr uint32_t kAMnMajor = 1u << 15, kBMnMajor = 1u << 16;

struct ExpertArgs {
  const int32_t* start;     // [E] first row
  const int32_t* counts;    // [E] rows
  int32_t E;
  int64_t rows;             // rows of the sorted buffers
  int32_t n_tiles;          // output column tiles
  int32_t m_tiles;          // kWgrad: output row tiles per expert
  int32_t k_blocks;         // reduction blocks (not kWgrad)
  int64_t n_rows;           // kWgrad: output rows of an expert (N)
  int64_t n_cols;           // output columns (kFwdSwiglu: I)
  uint16_t* out;            // y, gu, dx, dgu or dW
  int64_t out_ld;
  uint16_t* h;              // kFwdSwiglu
  int64_t h_ld;
  const uint16_t* gu;       // kDgradSwiglu
  int64_t gu_ld;
  int32_t* status;
  uint64_t timeout_ns;
};

// One output tile.
struct Tile {
  int expert;
  int64_t row0;   // first sorted row: of the block, or (kWgrad) of the expert
  int valid;      // rows of the block that carry a token
  int mt;         // kWgrad: output row tile
  int nt;         // output column tile
  int kb;         // reduction blocks
  int tail;       // kWgrad: rows of the last reduction block
};

// An expert's rows, none where its numbers do not fit the buffer.
__device__ __forceinline__ int expert_rows(const ExpertArgs& g, int e) {
  const int64_t n = g.counts[e], s = g.start[e];
  return n > 0 && s >= 0 && s + n <= g.rows ? static_cast<int>(n) : 0;
}

template <ExpertOp kOp>
__device__ __forceinline__ Tile tile_at(const ExpertArgs& g, const int32_t* s_cum, int64_t t) {
  Tile r;
  if constexpr (kOp == kWgrad) {
    const int64_t per = static_cast<int64_t>(g.m_tiles) * g.n_tiles;
    r.expert = static_cast<int>(t / per);
    const int64_t i = t - r.expert * per;
    r.mt = static_cast<int>(i / g.n_tiles);
    r.nt = static_cast<int>(i - static_cast<int64_t>(r.mt) * g.n_tiles);
    const int n = expert_rows(g, r.expert);
    r.row0 = g.start[r.expert];
    r.valid = kTileM;
    r.kb = (n + kBlockK - 1) / kBlockK;
    r.tail = n - (r.kb - 1) * kBlockK;
  } else {
    const int64_t b = t / g.n_tiles;
    r.nt = static_cast<int>(t - b * g.n_tiles);
    r.mt = 0;
    int lo = 0, hi = g.E - 1;   // the expert with s_cum[e] <= b < s_cum[e + 1]
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_cum[mid + 1] > b)
        hi = mid;
      else
        lo = mid + 1;
    }
    r.expert = lo;
    const int first = static_cast<int>(b - s_cum[lo]) * kTileM;
    r.row0 = static_cast<int64_t>(g.start[lo]) + first;
    const int left = g.counts[lo] - first;
    r.valid = left < kTileM ? left : kTileM;
    r.kb = g.k_blocks;
    r.tail = kBlockK;
  }
  return r;
}

__device__ __forceinline__ void bulk_wait_read_2() { asm volatile("cp.async.bulk.wait_group.read 2;" ::: "memory"); }

__device__ __forceinline__ void pack32(const float (&f)[32], uint4 (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    o[v] = make_uint4(pack_bf16x2(f[8 * v], f[8 * v + 1]), pack_bf16x2(f[8 * v + 2], f[8 * v + 3]),
                      pack_bf16x2(f[8 * v + 4], f[8 * v + 5]), pack_bf16x2(f[8 * v + 6], f[8 * v + 7]));
}

// This lane's 32 columns of its row into a store tile (64-byte rows, 64-byte
// swizzle: 16-byte piece j of row r at r * 64 + ((j ^ ((r >> 1) & 3)) * 16)).
__device__ __forceinline__ void stage_row(uint8_t* tile, int lane, const uint4 (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v) *reinterpret_cast<uint4*>(tile + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4)) = o[v];
}

// ... or straight to its row in memory, `left` columns from there.
__device__ __forceinline__ void store_row(uint16_t* dst, int64_t left, const uint4 (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    if (8 * v < left) reinterpret_cast<uint4*>(dst)[v] = o[v];
}

// 32 bf16 values of a row, zeros past `left`.
__device__ __forceinline__ void load_row(const uint16_t* src, int64_t left, uint4 (&o)[4]) {
#pragma unroll
  for (int v = 0; v < 4; ++v)
    o[v] = 8 * v < left ? __ldg(reinterpret_cast<const uint4*>(src) + v) : make_uint4(0, 0, 0, 0);
}
__device__ __forceinline__ float bf16_at(const uint4 (&o)[4], int i) {
  const uint4 q = o[i >> 3];
  const uint32_t w = ((i >> 1) & 3) == 0 ? q.x : ((i >> 1) & 3) == 1 ? q.y : ((i >> 1) & 3) == 2 ? q.z : q.w;
  return __uint_as_float((i & 1) ? (w & 0xFFFF0000u) : (w << 16));
}

template <ExpertOp kOp>
__global__ void __launch_bounds__(kThreads, 1)
    expert_gemm_kernel(const __grid_constant__ CUtensorMap map_a, const __grid_constant__ CUtensorMap map_b,
                       const __grid_constant__ CUtensorMap map_out, const __grid_constant__ CUtensorMap map_h,
                       const ExpertArgs g) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kOffBar);
  uint64_t* empty = full + kStages;
  uint64_t* tfull = full + 2 * kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + kOffHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kOffAbort);
  int32_t* s_scan = reinterpret_cast<int32_t*>(smem + kOffScan);
  int32_t* s_cum = reinterpret_cast<int32_t*>(smem + kOffCum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 32 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&map_a);
    prefetch_tensormap(&map_b);
    prefetch_tensormap(&map_out);
  }
  if (warp == 1) {
    tmem_alloc(holder, kTmemCols);
    tmem_relinquish();
  }
  pdl_wait();
  pdl_trigger();
  // row blocks of the experts before each, from the counts: a thread takes
  // consecutive experts, and the threads' sums are scanned
  if constexpr (kOp != kWgrad) {
    const int per = (g.E + kThreads - 1) / kThreads;
    const int e0 = threadIdx.x * per;
    int sum = 0;
    for (int e = e0; e < e0 + per && e < g.E; ++e) sum += (expert_rows(g, e) + kTileM - 1) / kTileM;
    int x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_scan[warp] = x;
    __syncthreads();
    int base = x - sum;
    for (int w = 0; w < warp; ++w) base += s_scan[w];
    for (int e = e0; e < e0 + per && e < g.E; ++e) {
      s_cum[e] = base;
      base += (expert_rows(g, e) + kTileM - 1) / kTileM;
      if (e == g.E - 1) s_cum[g.E] = base;
    }
  }
  if (blockIdx.x == 0)   // numbers that do not fit: reported, and the expert left out
    for (int e = threadIdx.x; e < g.E; e += kThreads)
      if (g.counts[e] != expert_rows(g, e)) set_status(g.status, MOE_ERR_INVALID_ARG);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int64_t n_tiles =
      kOp == kWgrad ? static_cast<int64_t>(g.E) * g.m_tiles * g.n_tiles : static_cast<int64_t>(s_cum[g.E]) * g.n_tiles;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer
    if (lane == 0) {
      int stage = 0;
      uint32_t phase = 0, issued_mask = 0, issued_parity = 0;
      bool ok = true;
      for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
        const Tile tl = tile_at<kOp>(g, s_cum, t);
        for (int kb = 0; kb < tl.kb; ++kb) {
          if (!mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns)) {
            ok = false;
            break;
          }
          uint8_t* a = smem + kOffA + stage * kABytes;
          uint8_t* b = smem + kOffB + stage * kBBytes;
          uint64_t* bar = &full[stage];
          mbar_arrive_expect_tx(bar, kABytes + kBBytes);
          const int k = kb * kBlockK;
          if constexpr (kOp == kWgrad) {
            const int row = static_cast<int>(tl.row0) + k;
#pragma unroll
            for (int i = 0; i < kTileM / 64; ++i)
              tma_load_3d(a + i * kBoxBytes, &map_a, bar, tl.mt * kTileM + 64 * i, row, 0);
#pragma unroll
            for (int i = 0; i < kTileN / 64; ++i)
              tma_load_3d(b + i * kBoxBytes, &map_b, bar, tl.nt * kTileN + 64 * i, row, 0);
          } else {
            tma_load_3d(a, &map_a, bar, k, static_cast<int>(tl.row0), 0);
            if constexpr (kOp == kFwd) {
              tma_load_3d(b, &map_b, bar, k, tl.nt * kTileN, tl.expert);
            } else if constexpr (kOp == kFwdSwiglu) {
              // gate rows, and the up rows I further down
              tma_load_3d(b, &map_b, bar, k, tl.nt * 128, tl.expert);
              tma_load_3d(b + kBBytes / 2, &map_b, bar, k, static_cast<int>(g.n_cols) + tl.nt * 128, tl.expert);
            } else {
#pragma unroll
              for (int i = 0; i < kTileN / 64; ++i)
                tma_load_3d(b + i * kBoxBytes, &map_b, bar, tl.nt * kTileN + 64 * i, k, tl.expert);
            }
          }
          issued_mask |= 1u << stage;
          issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
          if (++stage == kStages) {
            stage = 0;
            phase ^= 1;
          }
        }
      }
      if (!ok) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // never leave the CTA with copies still landing in its shared memory
      for (int s = 0; s < kStages; ++s)
        if (issued_mask & (1u << s)) {
          const int never = 0;
          mbar_wait_bounded(&full[s], (issued_parity >> s) & 1u, &never, g.timeout_ns);
        }
    }
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMA issuer
    constexpr bool kAMn = kOp == kWgrad;
    constexpr bool kBMn = kOp == kDgrad || kOp == kDgradSwiglu || kOp == kWgrad;
    constexpr uint32_t idesc = kIdesc | (kAMn ? kAMnMajor : 0u) | (kBMn ? kBMnMajor : 0u);
    int stage = 0, iter = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = blockIdx.x; t < n_tiles && ok; t += gridDim.x) {
      const Tile tl = tile_at<kOp>(g, s_cum, t);
      if (tl.kb == 0) continue;
      const int acc = iter & 1;
      ok = __all_sync(0xFFFFFFFFu,
                      mbar_wait_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
      if (!ok) break;
      ++iter;
      tc_fence_after();
      const uint32_t d = tmem + static_cast<uint32_t>(acc * kTileN);
      for (int kb = 0; kb < tl.kb; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + kOffA + stage * kABytes;
        uint8_t* b = smem + kOffB + stage * kBBytes;
        int steps = kBlockK / 16;
        if (kOp == kWgrad && kb == tl.kb - 1 && tl.tail < kBlockK) {
          // the expert's last rows: whole steps of 16 rows past its end are
          // left out, the rest of the last step is cleared in both operands
          // (they are consecutive in shared memory as 2 + 4 boxes of
          // 128-byte rows; a row stays in its place under the swizzle)
          steps = (tl.tail + 15) / 16;
          const int clear = steps * 16 - tl.tail;
          for (int i = lane; i < clear * 8 * 6; i += 32) {
            const int box = i / (clear * 8), j = i - box * clear * 8;
            uint8_t* base = box < 2 ? a + box * kBoxBytes : b + (box - 2) * kBoxBytes;
            *reinterpret_cast<uint4*>(base + tl.tail * 128 + j * 16) = make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
          __syncwarp();
        }
        tc_fence_after();
        if (lane == 0) {
          const uint64_t ad = smem_desc(smem_u32(a), kAMn ? kBoxBytes : 16, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(smem_u32(b), kBMn ? kBoxBytes : 16, 1024, kSwizzle128B);
          // 16 reduction elements on: 32 bytes along a K-major row, 16 rows of
          // 128 bytes down an MN-major box
          constexpr uint64_t astep = (kAMn ? 2048 : 32) >> 4, bstep = (kBMn ? 2048 : 32) >> 4;
          for (int k = 0; k < steps; ++k) mma_bf16(d, ad + astep * k, bd + bstep * k, idesc, !(kb == 0 && k == 0));
          tc_commit(&empty[stage]);
          if (kb == tl.kb - 1) tc_commit(&tfull[acc]);
        }
        __syncwarp();
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    if (!ok && lane == 0) {
      set_status(g.status, MOE_ERR_TIMEOUT);
      *abort_flag = 1;
    }
    if (lane == 0) {
      // all issued tensor-core work finished before the TMEM is released
      tc_commit(done);
      const int never = 0;
      mbar_wait_bounded(done, 0, &never, g.timeout_ns);
    }
    __syncwarp();
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3;
    uint8_t* stg = smem + kOffStg + (warp - 2) * kStgPerWarp * kStgTile;
    int iter = 0;
    uint32_t slot = 0;
    for (int64_t t = blockIdx.x; t < n_tiles; t += gridDim.x) {
      const Tile tl = tile_at<kOp>(g, s_cum, t);
      const int acc = iter & 1;
      if (tl.kb > 0) {
        const bool got = mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag, g.timeout_ns);
        if (!__all_sync(0xFFFFFFFFu, got)) {
          set_status(g.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        ++iter;
      }
      const uint32_t taddr = tmem + static_cast<uint32_t>(acc * kTileN) + (static_cast<uint32_t>(quad * 32) << 16);
      if constexpr (kOp == kWgrad) {
        const int64_t r0 = static_cast<int64_t>(tl.mt) * kTileM + quad * 32;
        const int64_t col0 = static_cast<int64_t>(tl.nt) * kTileN;
#pragma unroll 1
        for (int c = 0; c < kTileN / 32; ++c) {
          float f[32];
          if (tl.kb > 0) {
            uint32_t v[32];
            tmem_ld_32x32b_x32(taddr + c * 32, v);
            tmem_ld_wait();
            if (c == kTileN / 32 - 1) {
              tc_fence_before();
              mbar_arrive(&tempty[acc]);
            }
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = 0.0f;
          }
          if (r0 >= g.n_rows || col0 + c * 32 >= g.n_cols) continue;   // warp-uniform
          uint4 o[4];
          pack32(f, o);
          if (lane == 0) bulk_wait_read_2();   // the store from this tile three chunks ago has read it
          __syncwarp();
          uint8_t* tile = stg + slot * kStgTile;
          stage_row(tile, lane, o);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // (rows past N and columns past C are clipped by the map)
            tma_store_3d(&map_out, tile, static_cast<int>(col0) + c * 32, static_cast<int>(r0), tl.expert);
            bulk_commit_group();
          }
          slot = slot == kStgPerWarp - 1 ? 0 : slot + 1;
        }
        continue;
      } else {
        const int r = quad * 32 + lane;
        const bool row_ok = r < tl.valid;
        const bool whole = quad * 32 + 32 <= tl.valid;   // all of this warp's rows exist
        const bool none = quad * 32 >= tl.valid;
        const int64_t row = tl.row0 + r;
        const int row_w = static_cast<int>(tl.row0) + quad * 32;
        constexpr int kChunks = kOp == kFwdSwiglu ? 4 : kTileN / 32;
        const int64_t col0 = static_cast<int64_t>(tl.nt) * (kOp == kFwdSwiglu ? 128 : kTileN);
#pragma unroll 1
        for (int c = 0; c < kChunks; ++c) {
          const int64_t col = col0 + c * 32, left = g.n_cols - col;
          const bool last = c == kChunks - 1;
          const bool skip = none || left <= 0;   // warp-uniform
          uint4 gq[4], uq[4];
          if (kOp == kDgradSwiglu && !skip && row_ok) {
            load_row(g.gu + row * g.gu_ld + col, left, gq);
            load_row(g.gu + row * g.gu_ld + g.n_cols + col, left, uq);
          }
          uint32_t v[32], u[kOp == kFwdSwiglu ? 32 : 1];
          if (!skip) {
            tmem_ld_32x32b_x32(taddr + c * 32, v);
            if constexpr (kOp == kFwdSwiglu) tmem_ld_32x32b_x32(taddr + 128 + c * 32, u);
            tmem_ld_wait();
          }
          if (last) {
            tc_fence_before();
            mbar_arrive(&tempty[acc]);
          }
          if (skip) continue;
          if constexpr (kOp == kFwd || kOp == kDgrad) {
            float f[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) f[i] = __uint_as_float(v[i]);
            uint4 o[4];
            pack32(f, o);
            if (whole) {
              if (lane == 0) bulk_wait_read_2();
              __syncwarp();
              uint8_t* tile = stg + slot * kStgTile;
              stage_row(tile, lane, o);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                tma_store_3d(&map_out, tile, static_cast<int>(col), 0, row_w);
                bulk_commit_group();
              }
              slot = slot == kStgPerWarp - 1 ? 0 : slot + 1;
            } else if (row_ok) {
              store_row(g.out + row * g.out_ld + col, left, o);
            }
          } else {
            // two output halves (g, u or dg, du), and h
            float f0[32], f1[32], f2[kOp == kFwdSwiglu ? 32 : 1];
            if constexpr (kOp == kFwdSwiglu) {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                f0[i] = __uint_as_float(v[i]);
                f1[i] = __uint_as_float(u[i]);
                f2[i] = silu_mul(f0[i], f1[i]);
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i) {
                const float gate = bf16_at(gq, i), up = bf16_at(uq, i), dh = __uint_as_float(v[i]);
                const float s = 1.0f / (1.0f + __expf(-gate));
                f0[i] = dh * up * s * (1.0f + gate * (1.0f - s));
                f1[i] = dh * gate * s;
              }
            }
            uint4 o0[4], o1[4], o2[4];
            pack32(f0, o0);
            pack32(f1, o1);
            if constexpr (kOp == kFwdSwiglu) pack32(f2, o2);
            if (whole) {
              if (lane == 0) bulk_wait_read_all();
              __syncwarp();
              stage_row(stg, lane, o0);
              stage_row(stg + kStgTile, lane, o1);
              if constexpr (kOp == kFwdSwiglu) stage_row(stg + 2 * kStgTile, lane, o2);
              fence_proxy_async_smem();
              __syncwarp();
              if (lane == 0) {
                if (g.out) {
                  tma_store_3d(&map_out, stg, static_cast<int>(col), 0, row_w);
                  tma_store_3d(&map_out, stg + kStgTile, static_cast<int>(col), 1, row_w);
                }
                if constexpr (kOp == kFwdSwiglu)
                  tma_store_3d(&map_h, stg + 2 * kStgTile, static_cast<int>(col), 0, row_w);
                bulk_commit_group();
              }
            } else if (row_ok) {
              if (g.out) {
                store_row(g.out + row * g.out_ld + col, left, o0);
                store_row(g.out + row * g.out_ld + g.n_cols + col, left, o1);
              }
              if constexpr (kOp == kFwdSwiglu) store_row(g.h + row * g.h_ld + col, left, o2);
            }
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's stores have completed
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <ExpertOp kOp>
cudaError_t launch(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& out, const CUtensorMap& h,
                   const ExpertArgs& g, int64_t max_tiles, cudaStream_t s) {
  static bool attr_set = false;
  if (!attr_set) {
    const cudaError_t e =
        cudaFuncSetAttribute(expert_gemm_kernel<kOp>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  int dev = 0, sms = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const int grid = static_cast<int>(max_tiles < sms ? max_tiles : sms);
  return launch_pdl(expert_gemm_kernel<kOp>, dim3(grid), dim3(kThreads), kSmemBytes, s, a, b, out, h, g);
}

constexpr CUtensorMapDataType kBf16 = CU_TENSOR_MAP_DATA_TYPE_BFLOAT16;

// [rows][cols] with row stride ld, boxes of 64 columns x box_rows.
moe_status_t rows_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(rows), 1};
  const uint64_t st[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(ld) * static_cast<uint64_t>(rows) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_tiled_map(m, p, kBf16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// [E][n][c] weights, boxes of 64 columns x box_rows of one expert.
moe_status_t weights_map(CUtensorMap* m, const void* p, int64_t E, int64_t n, int64_t c, uint32_t box_rows) {
  const uint64_t d[3] = {static_cast<uint64_t>(c), static_cast<uint64_t>(n), static_cast<uint64_t>(E)};
  const uint64_t st[2] = {static_cast<uint64_t>(c) * 2, static_cast<uint64_t>(n) * static_cast<uint64_t>(c) * 2};
  const uint32_t box[3] = {64, box_rows, 1};
  return encode_tiled_map(m, p, kBf16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_128B);
}
// [rows][halves][cols] output with row stride ld, stored 32 rows x 32 columns at a time.
moe_status_t out_map(CUtensorMap* m, const void* p, int64_t rows, int64_t halves, int64_t cols, int64_t ld) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), static_cast<uint64_t>(halves), static_cast<uint64_t>(rows)};
  const uint64_t st[2] = {static_cast<uint64_t>(cols) * 2, static_cast<uint64_t>(ld) * 2};
  const uint32_t box[3] = {32, 1, 32};
  return encode_tiled_map(m, p, kBf16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B);
}

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) != 0; }

struct Operand {
  const void* p;
  int64_t ld, cols;
};

// Checks that all variants share; mats: the matrices of sorted rows.
moe_status_t check_expert(int64_t rows, int32_t E, int64_t N, int64_t C, const int32_t* start, const int32_t* counts,
                          const void* status, std::initializer_list<Operand> mats) {
  if (rows < 0 || E <= 0 || N <= 0 || C <= 0) return MOE_ERR_INVALID_ARG;
  if (E > kMaxLocalExperts || N % 8 || C % 8 || rows > 0x7FFFFFFF || N > 0x3FFFFFFF || C > 0x3FFFFFFF)
    return MOE_ERR_UNSUPPORTED;
  if (!start || !counts || !status) return MOE_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(start) | reinterpret_cast<uintptr_t>(counts) | reinterpret_cast<uintptr_t>(status)) &
      3)
    return MOE_ERR_MISALIGNED;
  for (const Operand& o : mats) {
    if (rows > 0 && !o.p) return MOE_ERR_INVALID_ARG;
    if (o.ld < o.cols) return MOE_ERR_INVALID_ARG;
    if (o.ld % 8 || o.ld > (int64_t(1) << 36)) return MOE_ERR_UNSUPPORTED;
    if (off16(o.p)) return MOE_ERR_MISALIGNED;
  }
  return MOE_OK;
}

ExpertArgs expert_args(int64_t rows, int32_t E, const int32_t* start, const int32_t* counts, void* status) {
  ExpertArgs g;
  memset(&g, 0, sizeof(g));
  g.start = start;
  g.counts = counts;
  g.E = E;
  g.rows = rows;
  g.status = static_cast<int32_t*>(status);
  g.timeout_ns = 2000000000ull;
  return g;
}

int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

// Row blocks of any split of `rows` rows among E experts, at most.
int64_t max_blocks(int64_t rows, int32_t E) { return rows / kTileM + E; }

moe_status_t as_status(cudaError_t e) { return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_expert_gemm(const void* x, int64_t x_ld, int64_t rows, const void* w, const int32_t* start,
                             const int32_t* counts, int32_t E, int64_t N, int64_t C, void* y, int64_t y_ld,
                             void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{x, x_ld, C}, {y, y_ld, N}});
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (off16(w)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return MOE_OK;
  CUtensorMap a, b, o;
  if ((st = rows_map(&a, x, rows, C, x_ld, kTileM)) != MOE_OK) return st;
  if ((st = weights_map(&b, w, E, N, C, kTileN)) != MOE_OK) return st;
  if ((st = out_map(&o, y, rows, 1, N, y_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(N, kTileN);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = N;
  g.out = static_cast<uint16_t*>(y);
  g.out_ld = y_ld;
  return as_status(launch<kFwd>(a, b, o, o, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_swiglu(const void* x, int64_t x_ld, int64_t rows, const void* w13, const int32_t* start,
                                    const int32_t* counts, int32_t E, int64_t I, int64_t C, void* gu, int64_t gu_ld,
                                    void* h, int64_t h_ld, void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, I, C, start, counts, status, {{x, x_ld, C}, {h, h_ld, I}});
  if (st != MOE_OK) return st;
  if (!w13) return MOE_ERR_INVALID_ARG;
  if (off16(w13) || off16(gu)) return MOE_ERR_MISALIGNED;
  if (gu && gu_ld < 2 * I) return MOE_ERR_INVALID_ARG;
  if (gu && (gu_ld % 8 || gu_ld > (int64_t(1) << 36))) return MOE_ERR_UNSUPPORTED;
  if (rows == 0) return MOE_OK;
  CUtensorMap a, b, o, hm;
  if ((st = rows_map(&a, x, rows, C, x_ld, kTileM)) != MOE_OK) return st;
  if ((st = weights_map(&b, w13, E, 2 * I, C, 128)) != MOE_OK) return st;
  if ((st = out_map(&hm, h, rows, 1, I, h_ld)) != MOE_OK) return st;
  o = hm;
  if (gu && (st = out_map(&o, gu, rows, 2, I, gu_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, 128);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(gu);
  g.out_ld = gu_ld;
  g.h = static_cast<uint16_t*>(h);
  g.h_ld = h_ld;
  return as_status(
      launch<kFwdSwiglu>(a, b, o, hm, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad(const void* dy, int64_t dy_ld, int64_t rows, const void* w, const int32_t* start,
                                   const int32_t* counts, int32_t E, int64_t N, int64_t C, void* dx, int64_t dx_ld,
                                   void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{dy, dy_ld, N}, {dx, dx_ld, C}});
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (off16(w)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return MOE_OK;
  CUtensorMap a, b, o;
  if ((st = rows_map(&a, dy, rows, N, dy_ld, kTileM)) != MOE_OK) return st;
  if ((st = weights_map(&b, w, E, N, C, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&o, dx, rows, 1, C, dx_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(C, kTileN);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = C;
  g.out = static_cast<uint16_t*>(dx);
  g.out_ld = dx_ld;
  return as_status(launch<kDgrad>(a, b, o, o, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad_swiglu(const void* dy, int64_t dy_ld, int64_t rows, const void* w2, const void* gu,
                                          int64_t gu_ld, const int32_t* start, const int32_t* counts, int32_t E,
                                          int64_t N, int64_t I, void* dgu, int64_t dgu_ld, void* status, void* stream) {
  moe_status_t st =
      check_expert(rows, E, N, I, start, counts, status, {{dy, dy_ld, N}, {gu, gu_ld, 2 * I}, {dgu, dgu_ld, 2 * I}});
  if (st != MOE_OK) return st;
  if (!w2) return MOE_ERR_INVALID_ARG;
  if (off16(w2)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return MOE_OK;
  CUtensorMap a, b, o;
  if ((st = rows_map(&a, dy, rows, N, dy_ld, kTileM)) != MOE_OK) return st;
  if ((st = weights_map(&b, w2, E, N, I, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&o, dgu, rows, 2, I, dgu_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, kTileN);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(dgu);
  g.out_ld = dgu_ld;
  g.gu = static_cast<const uint16_t*>(gu);
  g.gu_ld = gu_ld;
  return as_status(
      launch<kDgradSwiglu>(a, b, o, o, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_wgrad(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int64_t rows,
                                   const int32_t* start, const int32_t* counts, int32_t E, int64_t N, int64_t C,
                                   void* dw, void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{dy, dy_ld, N}, {x, x_ld, C}});
  if (st != MOE_OK) return st;
  if (!dw) return MOE_ERR_INVALID_ARG;
  if (off16(dw)) return MOE_ERR_MISALIGNED;
  if (rows == 0)   // no expert has rows
    return as_status(cudaMemsetAsync(dw, 0, static_cast<size_t>(E) * N * C * 2, static_cast<cudaStream_t>(stream)));
  CUtensorMap a, b, o;
  if ((st = rows_map(&a, dy, rows, N, dy_ld, kBlockK)) != MOE_OK) return st;
  if ((st = rows_map(&b, x, rows, C, x_ld, kBlockK)) != MOE_OK) return st;
  const uint64_t d[3] = {static_cast<uint64_t>(C), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t strides[2] = {static_cast<uint64_t>(C) * 2, static_cast<uint64_t>(N) * static_cast<uint64_t>(C) * 2};
  const uint32_t box[3] = {32, 32, 1};
  if ((st = encode_tiled_map(&o, dw, kBf16, 3, d, strides, box, CU_TENSOR_MAP_SWIZZLE_64B)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(C, kTileN);
  g.m_tiles = ceil_div(N, kTileM);
  g.n_rows = N;
  g.n_cols = C;
  return as_status(launch<kWgrad>(a, b, o, o, g, static_cast<int64_t>(E) * g.m_tiles * g.n_tiles,
                                  static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
