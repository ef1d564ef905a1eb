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
//   kFwdAct(Res)  y[r]  = act(x[r] W_e^T + b_e) (+ res[r])
//   kFwdGlu       [g|u] = x[r] W_e^T + b_e, h[r] = act(g) u
//   kDgradRes     dx[r] = dy[r] W_e + res[r]
//   kDgradAct(Res) dx[r] = act'(z[r]) (dy[r] W_e) (+ res[r])
//   kDgradGlu     dh    = dy[r] W_e, dg = dh u act'(g), du = dh act(g)
//   kWgrad        dW_e  = sum over r of dy[r]^T x[r]      (0 without rows)
// act: activation.cuh.  A dense product is one expert that has all rows; of few tiles it
// goes to few_rows.cu.
//
// Two kernels.
//
// Rows (all but kWgrad).  The sorted rows are few and uneven, the weights' rows
// many and even, so the weights are the M side of the MMA and the tokens its N
// side: D = W X^T, a tile of 256 features x n tokens.  An expert's rows are cut
// into as few blocks of at most 256 as will do (lower ones where those are too few
// for the pairs), equally tall up to a multiple of 32, so uneven experts cost the MMAs of at most 31 rows too many, not of
// half a 128-row block each (which took a sixth to a quarter more at 512 and
// 256 rows per expert).  A tile is worked on by a CTA pair: M = 256 over the
// two, each CTA staging its own 128 weight rows and half of the tokens: 32 KB
// per SM and 64-element block of the reduction, where a 128 x 256 tile on one SM
// needs 48 KB.
//   kFwd    A = W rows (K-major)                  B = x rows (K-major)
//   kDgrad  A = W columns (MN-major: the feature  B = dy rows (K-major)
//           runs along W's memory rows)
// The accumulator holds features in lanes and tokens in columns; the epilogue
// turns it around in registers (lanes exchange with their neighbours, two
// values a shuffle) and in 32-token store tiles, so memory sees whole rows.
// kFwdSwiglu's CTA holds 64 gate rows and the 64 up rows of the same features;
// the warps of a feature's g and of its u hand each other half of a chunk's
// tokens and form h of the other half.
//
// Weights' gradient (kWgrad).  dW = dy^T x, a tile of 256 x at most 256 on a CTA
// pair, both operands MN-major (64 x 64 boxes, no transposed copies), summed
// over the expert's rows 64 at a time.  No other rows are copied, and the last 16
// reduction rows are filled with zeros in both CTAs' shared memory, so whatever
// lies behind the expert's rows, NaN included, does not count.  (In the other
// products such rows only make output rows that are not stored.)
//
// Both: one persistent CTA per SM: warp 0 TMA producer, warp 1 MMA issue, the
// others epilogue (one or two per 32 accumulator lanes, independent of one
// another), two accumulators so that a tile's epilogue runs beside the next
// tile's MMAs.
//
// What bounds it.  A full tile's reduction block takes 517 cycles of the MMA's
// 512, and 32 KB in that time is 63 B per clock, about what an SM gets from L2:
// the two limits coincide, and lower tiles are held by the second (192 tokens:
// 437 cycles for 384).  With all SMs busy the board's power cap then sets the
// clock (1.3 - 1.7 GHz): 8 x 2048 rows of 4096 x 4096 take 291 us forward, 290 us
// for the rows' gradient and 299 us for the weights' in the first milliseconds,
// 331, 331 and 345 us (1664, 1659, 1595 TFLOP/s) when they run on at 1250 W; the
// library's dense product of 16384 x 4096 x 4096 281 and 318 us.  Few rows per
// expert are bound by the weights' bytes (16 tokens on
// 32 experts: 7.3 TB/s), 256 rows per expert nearly so (1536 x 2048 weights:
// 6.1 - 6.6 TB/s), and the weights' gradient by what L2 moves, writes counting
// twice (128 x 1536 x 2048, 256 rows each: 183 us; 133 us without the stores,
// 164 us with the copies of dy left out).
// The activation of other kinds, a bias and a residual (kFwdAct and what follows it) cost
// 8192 rows of 2048 x 2048, 41 us alone: 43 with silu, 46 with gelu, 45 with a residual, 47
// for the rows' gradient through silu, mostly in the last round, whose epilogue no MMAs
// hide (sixteen epilogue warps for it spill: 48 and 70; four: 47 and 64).
// Clusters of four, whose pairs would share their tokens' copies, fit 144 of the
// 152 SMs.  Handing the tall tiles out first, looking up the next tile's numbers
// ahead, or running through the features inside made no difference.
#include <string.h>

#include "activation.cuh"
#include "experts.cuh"
#include "few_rows.h"
#include "internal.h"
#include "pair.cuh"
#include "pairs.h"

namespace moe {

namespace {

enum ExpertOp { kFwd, kFwdSwiglu, kDgrad, kDgradSwiglu, kWgrad, kFwdAct, kFwdActRes, kFwdGlu, kDgradRes, kDgradAct,
                kDgradActRes, kDgradGlu };
// (Res: with a residual.  Kernels of their own, because code that is passed by still costs
// a call of one tile 0.3 to 0.6 us of its 4.5.)
// halves g and u of a gated activation in the weights' rows; gradients of rows
__host__ __device__ constexpr bool gated_fwd(ExpertOp op) { return op == kFwdSwiglu || op == kFwdGlu; }
__host__ __device__ constexpr bool gated_grad(ExpertOp op) { return op == kDgradSwiglu || op == kDgradGlu; }
__host__ __device__ constexpr bool rows_grad(ExpertOp op) { return op == kDgrad || (op >= kDgradRes && op <= kDgradActRes) || gated_grad(op); }
__host__ __device__ constexpr bool adds_rows(ExpertOp op) { return op == kFwdActRes || op == kDgradRes || op == kDgradActRes; }

constexpr int kBlockK = 64;                          // elements: 128 bytes, one swizzle atom
constexpr int kBoxBytes = 64 * kBlockK * 2;          // an MN-major box: 64 x 64 elements
constexpr int kStgTile = 32 * 64;                    // a store tile: 32 rows x 32 columns
constexpr uint32_t kTmemCols = 512;
constexpr int kMaxStages = 6;

// Shared memory: the stages, the epilogue warps' tiles, then the same for all.
constexpr int kNumBars = 3 * kMaxStages + 9;         // full, empty (kWgrad: cleared); tfull[2], tempty[2];
                                                     // done; xchg[4]
constexpr int kTailHolder = kNumBars * 8;
constexpr int kTailAbort = kTailHolder + 4;
constexpr int kTailCum = kTailAbort + 4;             // token blocks of the 32-expert groups before, [33]
constexpr int kTailTry = kTailCum + 33 * 4;          // the groups' token blocks of each height, [4][32]; then the height
constexpr int kTailBytes = kTailTry + 4 * 32 * 4 + 1024;   // + alignment slack

// Epilogue warps and their shared memory, by operator.  The activation and its
// gradient take the epilogue more arithmetic and more bytes than the product
// alone, and the weights' gradient has short sums for a whole output tile: they
// get eight warps, two per 32 lanes.  All get six stages, for which the warps'
// tiles are kept small: with five and larger tiles the activation took 193 us
// instead of 185 (4096 tokens, top-8, 128 experts of 1536 x 2048), its gradient
// 343 us instead of 330 (16384 rows, 32 experts of 7168 x 2048).
template <ExpertOp kOp>
struct Cfg {
  static constexpr int kStages = 6;
  static constexpr int kStage = 32 * 1024;
  static constexpr int kEpiWarps = kOp == kFwd || kOp == kDgrad ? 4 : 8;
  static constexpr int kThreads = 64 + 32 * kEpiWarps + (kOp == kWgrad ? 32 : 0);
  static constexpr int kTiles = kOp == kFwd || kOp == kDgrad ? 3 : 2;   // store tiles of an epilogue warp (kWgrad: one
                                                                        // of twice the size; kFwdSwiglu: one, and
                                                                        // what its warps hand over)
  static constexpr int kStgBytes = kTiles * kStgTile;
  static constexpr int kOffStg = kStages * kStage;
  static constexpr int kOffTail = kOffStg + kEpiWarps * kStgBytes;
  static constexpr int kSmem = kOffTail + kTailBytes;
  static_assert(kSmem <= 227 * 1024 && kStages <= kMaxStages, "shared memory");
};

// D fp32, A and B bf16; M and N are added
constexpr uint32_t kIdesc = (1u << 4) | (1u << 7) | (1u << 10);
__host__ __device__ constexpr uint32_t idesc_mn(int m, int n) {
  return (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}
constexpr uint32_t kAMnMajor = 1u << 15, kBMnMajor = 1u << 16;

struct ExpertArgs {
  const int32_t* start;     // [E] first row
  const int32_t* counts;    // [E] rows
  int32_t E;
  int64_t rows;             // rows of the sorted buffers
  int32_t n_tiles;          // output column (feature) tiles
  int32_t m_tiles;          // kWgrad: output row tiles per expert
  int32_t k_blocks;         // reduction blocks (not kWgrad)
  int64_t n_rows;           // kWgrad: output rows of an expert (N)
  int64_t n_cols;           // output columns (kFwdSwiglu: I)
  int32_t accumulate;       // kWgrad in fp32: dW is added to
  uint16_t* out;            // y, gu, dx or dgu
  int64_t out_ld;
  uint16_t* h;              // kFwdSwiglu
  int64_t h_ld;
  const uint16_t* gu;       // kDgradSwiglu, kDgradGlu; kDgradAct: z
  int64_t gu_ld;
  int32_t act;              // where there is one: moe_act_t
  int32_t bias_f32;         // the bias is fp32, not bf16
  const void* bias;         // kFwdAct, kFwdGlu: [E, weight rows] or null
  const uint16_t* res;      // added to the output; may be the output itself
  int64_t res_ld;
  uint16_t* z;              // kFwdAct: sums before the activation, or null
  int64_t z_ld;
  int32_t* status;
  uint64_t timeout_ns;
};

// All but this thread's last n bulk groups have read their shared memory.
template <int n>
__device__ __forceinline__ void bulk_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(n) : "memory");
}

// The limit of a wait for a whole tile of the tensor core: g.timeout_ns longer than
// its reduction may take, at 4 us a block, which takes 0.1 to 0.7.  (An expert of
// 2^31 rows is a reduction of seconds.)
__device__ __forceinline__ uint64_t tile_limit(const ExpertArgs& g, int blocks) {
  return g.timeout_ns + static_cast<uint64_t>(blocks) * 4000u;
}

// Eight accumulator values as bf16.
__device__ __forceinline__ uint4 pack8(const uint32_t* v) {
  return make_uint4(pack_bf16x2(__uint_as_float(v[0]), __uint_as_float(v[1])),
                    pack_bf16x2(__uint_as_float(v[2]), __uint_as_float(v[3])),
                    pack_bf16x2(__uint_as_float(v[4]), __uint_as_float(v[5])),
                    pack_bf16x2(__uint_as_float(v[6]), __uint_as_float(v[7])));
}

// Two features of a token into a store tile: 64-byte rows, 64-byte swizzle.
__device__ __forceinline__ void put_word(uint8_t* tile, int token, int word, uint32_t w) {
  *reinterpret_cast<uint32_t*>(tile + token * 64 + (((word >> 2) ^ ((token >> 1) & 3)) << 4) + (word & 3) * 4) = w;
}

// A filled store tile of kTok tokens to memory: by TMA when they all exist (the
// map clips features past the end), else each lane copies its token's row
// (dst: the first token's, `left` features from there).  Either way one bulk
// group more, so that the groups count tiles.
template <int kTok>
__device__ __forceinline__ void store_tile(uint8_t* tile, const CUtensorMap* map, int rows, int lane, int c0, int c1,
                                           int c2, uint16_t* dst, int64_t ld, int64_t left) {
  if (rows >= kTok) {
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) tma_store_3d(map, tile, c0, c1, c2);
  } else {
    __syncwarp();
    if (lane < rows) {
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (8 * v < left)
          *reinterpret_cast<uint4*>(dst + lane * ld + 8 * v) =
              *reinterpret_cast<const uint4*>(tile + lane * 64 + ((v ^ ((lane >> 1) & 3)) << 4));
    }
    __syncwarp();
  }
  if (lane == 0) bulk_commit_group();
}

__device__ __forceinline__ void swiglu_grad(float dh, float gate, float up, float* dg, float* du) {
  const float s = sigmoid_fast(gate);
  const float ds = dh * s;
  *dg = ds * up * fmaf(gate, 1.0f - s, 1.0f);
  *du = ds * gate;
}

// ---------------------------------------------------------------------------
// Products of rows
// ---------------------------------------------------------------------------
constexpr int kRowsA = 128 * kBlockK * 2;            // this CTA's 128 features, 16 KB
constexpr int kRowsB = 128 * kBlockK * 2;            // this CTA's half of at most 256 tokens, 16 KB
constexpr int kTokens = 256;                         // tokens of a tile at most

struct RowsTile {
  int expert;
  int64_t row0;   // first sorted row
  int valid;      // tokens
  int n;          // tokens of the MMA: valid rounded up to 32
  int box;        // the map of x that loads half of them: 128 - 32 * box rows
  int ft;         // feature tile
};

// Blocks of at most 256 >> low tokens.
__device__ __forceinline__ int token_blocks(int rows, int low) {
  return static_cast<int>((static_cast<unsigned>(rows) + (kTokens >> low) - 1) >> (8 - low));
}

// How tall tiles may be, 256 >> 0..3 tokens: what makes the time of all rounds
// over the pairs least, at a reduction block's cycles for tiles of those heights
// (what the MMA or L2 needs).  Lower tiles cost more per token, and pay for work
// of a round or two: 1000 rows on one expert of 2048 x 2048 take 13 us instead of
// 16, 2 x 512 rows' gradient on 4096 x 2048 19 instead of 24.5; 8 x 128 rows, for
// which they are no use, 0.3 us more for the choice.
// A converged warp; blocks: [4][32] of the groups of experts.
__device__ __forceinline__ int tile_height(const int32_t* blocks, int n_tiles, int lane) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  const unsigned pairs = gridDim.x >> 1;
  const int64_t tall = static_cast<int64_t>(__reduce_add_sync(kAll, blocks[lane])) * n_tiles;
  if (tall > 2 * pairs) return 0;
  // (lane i: that of 256 >> i)
  unsigned sum = static_cast<unsigned>(tall);
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const unsigned tiles = __reduce_add_sync(kAll, blocks[i * 32 + lane]) * n_tiles;
    if (lane == i) sum = tiles;
  }
  const unsigned cycles = lane == 0 ? 517 : lane == 1 ? 384 : lane == 2 ? 320 : 288;
  const unsigned time = (sum + pairs - 1) / pairs * cycles * 4 + lane;
  return __reduce_min_sync(kAll, lane < 4 ? time : ~0u) & 3;
}

// Tile t, looked up by a whole, converged warp: the group of 32 experts that
// holds it from the groups' sums, then the expert from the counts of the group,
// one per lane.  The same in all lanes.
__device__ __forceinline__ RowsTile rows_tile(const ExpertArgs& g, const int32_t* s_cum, int low, int64_t t, int lane) {
  constexpr unsigned kAll = 0xFFFFFFFFu;
  const bool past = lane * 32 < g.E && static_cast<int64_t>(s_cum[lane + 1]) * g.n_tiles > t;
  const int group = __ffs(__ballot_sync(kAll, past)) - 1;
  const int e = group * 32 + lane;
  const int rows = e < g.E ? expert_rows(g, e) : 0;
  const int start = e < g.E ? expert_start(g, e) : 0;
  const int mine = token_blocks(rows, low);
  int end = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(kAll, end, o);
    if (lane >= o) end += y;
  }
  end += s_cum[group];
  const int at = __ffs(__ballot_sync(kAll, static_cast<int64_t>(end) * g.n_tiles > t)) - 1;
  const int blocks = __shfl_sync(kAll, mine, at), first = __shfl_sync(kAll, end, at) - blocks;
  const int count = __shfl_sync(kAll, rows, at);
  RowsTile r;
  r.expert = group * 32 + at;
  // token blocks innermost: they share a weight tile while it is in L2
  const int i = static_cast<int>(t - static_cast<int64_t>(first) * g.n_tiles);
  r.ft = i / blocks;
  const int b = i - r.ft * blocks;
  const int tall = static_cast<int>(((static_cast<unsigned>(count) + blocks - 1) / blocks + 31) & ~31u);
  r.row0 = static_cast<int64_t>(__shfl_sync(kAll, start, at)) + b * tall;
  const int left = count - b * tall;
  r.valid = left < tall ? left : tall;
  r.n = (r.valid + 31) & ~31;
  r.box = (256 - r.n) / 64;
  return r;
}

// The epilogue's lanes hold one feature of two tokens (a, b); the neighbour
// lane^1 the next (or previous) feature of the same.  After the exchange an
// even lane has both features of the first token, an odd lane of the second.
__device__ __forceinline__ float2 pair_up(float a, float b, bool odd) {
  const float x = __shfl_xor_sync(0xFFFFFFFFu, odd ? a : b, 1);
  return odd ? make_float2(x, b) : make_float2(a, x);
}

// After an aborted pair: copies may still be on their way into this CTA's shared
// memory, and complete on the other CTA's barrier, so they cannot be waited
// for; they are left ample time.
__device__ __noinline__ void leave_copies_time() {
  const uint64_t now = globaltimer_ns();
  while (globaltimer_ns() - now < 2000000ull) {
  }
}

// g and u of chunk c of a tile, arranged as pair_up leaves dh: word i of an even
// (odd) lane holds two features of token 2i (2i + 1).  Zeros where there is none.
__device__ __forceinline__ void load_gate_up(const ExpertArgs& g, const RowsTile& tl, int c, int64_t col, int64_t left,
                                             int lane, uint32_t (&gw)[16], uint32_t (&uw)[16]) {
  const int tok = c * 32 + (lane & 1);
  const bool there = (lane & ~1) < left;
  const uint16_t* src = g.gu + (tl.row0 + tok) * g.gu_ld + col + (lane & ~1);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    gw[i] = uw[i] = 0;
    if (there && tok + 2 * i < tl.valid) {
      gw[i] = __ldg(reinterpret_cast<const uint32_t*>(src + 2 * i * g.gu_ld));
      uw[i] = __ldg(reinterpret_cast<const uint32_t*>(src + 2 * i * g.gu_ld + g.n_cols));
    }
  }
}

// The same of one matrix [rows, >= col + 32] (src).  Plain loads: the matrix may be the
// output, of which each element is read before the same warp writes it.
__device__ __forceinline__ void load_words(const uint16_t* src, int64_t ld, const RowsTile& tl, int c, int64_t col,
                                           int64_t left, int lane, uint32_t (&w)[16]) {
  const int tok = c * 32 + (lane & 1);
  const bool there = (lane & ~1) < left;
  src += (tl.row0 + tok) * ld + col + (lane & ~1);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    w[i] = 0;
    if (there && tok + 2 * i < tl.valid) w[i] = *reinterpret_cast<const uint32_t*>(src + 2 * i * ld);
  }
}

// Element i of a bias.
__device__ __forceinline__ float bias_at(const ExpertArgs& g, int64_t i) {
  return g.bias_f32 ? static_cast<const float*>(g.bias)[i]
                    : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t*>(g.bias)[i]) << 16);
}

// Tensor maps of a rows launch.  x: the tokens in boxes of 128, 96, 64, 32 rows (a
// tile takes the smallest that holds its half of the tokens: one copy per stage,
// as more copies of fewer bytes are slower: 358 us in 32-row boxes, 300 us so,
// at 16384 x 4096 x 4096); out: the output or its first half, out2: its second
// half (kFwdAct: z), h: kFwdSwiglu's third output.
struct RowsMaps {
  CUtensorMap w, x[4], out, out2, h;
};

template <ExpertOp kOp>
__global__ void __launch_bounds__(Cfg<kOp>::kThreads, 1)
    expert_rows_kernel(const __grid_constant__ RowsMaps maps, const ExpertArgs g) {
  using F = Cfg<kOp>;
  constexpr int kRowsStages = F::kStages, kEpiWarps = F::kEpiWarps;
  constexpr bool kGated = gated_fwd(kOp), kGate2 = gated_grad(kOp), kRes = adds_rows(kOp);
  constexpr bool kFwdOne = kOp == kFwdAct || kOp == kFwdActRes;   // one product, with bias and activation
  constexpr bool kZ = kOp == kDgradAct || kOp == kDgradActRes;    // through the activation before it
  constexpr int kFeatures = kGated ? 128 : 256;   // output features of a tile
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::kOffTail);
  uint64_t* empty = full + kRowsStages;
  uint64_t* tfull = empty + kRowsStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint64_t* xchg = done + 1;   // gated: the warps of g and of u
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + F::kOffTail + kTailHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + F::kOffTail + kTailAbort);
  int32_t* s_cum = reinterpret_cast<int32_t*>(smem + F::kOffTail + kTailCum);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kRowsStages; ++s) {
      mbar_init(&full[s], 1);     // (the even CTA's is used: its producer arrives, both CTAs' copies count)
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);   // (the even CTA's: both CTAs' epilogue warps)
    }
    mbar_init(done, 1);
    for (int q = 0; q < 4; ++q) mbar_init(&xchg[q], 64);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.w);
    prefetch_tensormap(&maps.x[0]);
    prefetch_tensormap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc_pair(holder, kTmemCols);
    tmem_relinquish_pair();
  }
  int32_t* s_try = reinterpret_cast<int32_t*>(smem + F::kOffTail + kTailTry);
  if (threadIdx.x < 128) s_try[threadIdx.x] = 0;
  __syncthreads();
  pdl_wait();
  pdl_trigger();
  // token blocks of each group of 32 experts, one warp per group, the tiles'
  // height, and the sums
  for (int k = warp; k < (g.E + 31) / 32; k += F::kThreads / 32) {
    const int e = k * 32 + lane;
    const int rows = e < g.E ? expert_rows(g, e) : 0;
    int blocks = 0;   // (lane i: of height 256 >> i)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int all = __reduce_add_sync(0xFFFFFFFFu, token_blocks(rows, i));
      if (lane == i) blocks = all;
    }
    if (lane < 4) s_try[lane * 32 + k] = blocks;
  }
  __syncthreads();
  if (warp == 0) {
    const int best = tile_height(s_try, g.n_tiles, lane);
    int x = s_try[best * 32 + lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    s_cum[lane + 1] = x;
    if (lane == 0) {
      s_cum[0] = 0;
      s_try[0] = best;
    }
  }
  report_experts(g);
  tc_fence_before();
  // both CTAs' barriers and tensor memory are ready before either is used
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int64_t n_tiles = static_cast<int64_t>(s_cum[32]) * g.n_tiles;
  const int low = s_try[0];
  const int64_t t0 = blockIdx.x >> 1, t_step = gridDim.x >> 1;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (both CTAs)
    const int k_blocks = g.k_blocks;
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int64_t t = t0; t < n_tiles && ok; t += t_step) {
      const RowsTile tl = rows_tile(g, s_cum, low, t, lane);
      const uint32_t bytes = kRowsA + kRowsB / 4 * (4 - tl.box);
      const CUtensorMap* map_x = &maps.x[tl.box];
      const int tok = static_cast<int>(tl.row0) + static_cast<int>(rank) * (tl.n / 2);
      const int f = tl.ft * kFeatures + static_cast<int>(rank) * (kFeatures / 2);
      for (int kb = 0; kb < k_blocks; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + stage * (kRowsA + kRowsB);
        uint8_t* b = a + kRowsA;
        const uint32_t bar = mapa(smem_u32(&full[stage]), 0);
        if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * bytes);
        const int k = kb * kBlockK;
        if constexpr (kOp == kFwd || kFwdOne) {
          tma_load_3d_pair(a, &maps.w, bar, k, f, tl.expert);
        } else if constexpr (kGated) {
          tma_load_3d_pair(a, &maps.w, bar, k, f, tl.expert);
          tma_load_3d_pair(a + kRowsA / 2, &maps.w, bar, k, static_cast<int>(g.n_cols) + f, tl.expert);
        } else {
          tma_load_3d_pair(a, &maps.w, bar, f, k, tl.expert);
          tma_load_3d_pair(a + kBoxBytes, &maps.w, bar, f + 64, k, tl.expert);
        }
        tma_load_3d_pair(b, map_x, bar, k, tok, 0);
        if (++stage == kRowsStages) {
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
    // (values broadcast from lane 0 are known to be uniform: the MMAs' operands
    // and the loops around them stay in uniform registers)
    if (__shfl_sync(0xFFFFFFFFu, rank, 0) == 0) {
      constexpr bool kAMn = rows_grad(kOp);
      const uint32_t base = __shfl_sync(0xFFFFFFFFu, smem_u32(smem), 0);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      const int k_blocks = g.k_blocks;
      int stage = 0, iter = 0;
      uint32_t phase = 0;
      bool ok = true;
      for (int64_t t = t0; t < n_tiles && ok; t += t_step, ++iter) {
        const RowsTile tl = rows_tile(g, s_cum, low, t, lane);
        const uint32_t idesc =
            kIdesc | (kAMn ? kAMnMajor : 0u) | idesc_mn(256, __shfl_sync(0xFFFFFFFFu, tl.n, 0));
        const int acc = iter & 1;
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait_cluster_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        const uint32_t d = tm + static_cast<uint32_t>(acc * kTokens);
        for (int kb = 0; kb < k_blocks; ++kb) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
          if (!ok) break;
          tc_fence_after();
          const uint32_t a = base + stage * (kRowsA + kRowsB);
          const uint64_t ad = smem_desc(a, kAMn ? kBoxBytes : 16, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(a + kRowsA, 16, 1024, kSwizzle128B);
          // 16 reduction elements on: 32 bytes along a K-major row, 16 rows of
          // 128 bytes down an MN-major box
          constexpr uint64_t astep = (kAMn ? 2048 : 32) >> 4, bstep = 32 >> 4;
          mma_block_pair(d, ad, bd, astep, bstep, idesc, kb != 0);
          tc_commit_pair(&empty[stage]);
          if (++stage == kRowsStages) {
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
    const int quad = warp & 3;
    const bool odd = lane & 1;
    const int half = (warp - 2) >> 2;        // eight warps: each takes every other chunk
    uint8_t* stg = smem + F::kOffStg + (warp - 2) * F::kStgBytes;
    int iter = 0;
    uint32_t slot = 0;
    bool ok = true;
    // the warp's next store tile, once the store from it three tiles ago has read it
    auto next_tile = [&]() {
      if (lane == 0) bulk_wait_read<F::kTiles - 1>();
      __syncwarp();
      uint8_t* tile = stg + slot * kStgTile;
      slot = slot == F::kTiles - 1 ? 0 : slot + 1;
      return tile;
    };
    for (int64_t t = t0; t < n_tiles; t += t_step, ++iter) {
      const RowsTile tl = rows_tile(g, s_cum, low, t, lane);
      const int acc = iter & 1;
      // this warp's 32 features, from col (kFwdSwiglu: quads 0 and 1 hold g, 2 and 3 the same features' u)
      const int64_t col = static_cast<int64_t>(tl.ft) * kFeatures + static_cast<int>(rank) * (kFeatures / 2) +
                          (kGated ? quad & 1 : quad) * 32;
      const int64_t left = g.n_cols - col;   // features there are from col
      const int chunks = tl.n / 32;
      constexpr int kStep = kEpiWarps / 4;
      // kDgradSwiglu: g and u as pair_up leaves dh, a chunk ahead of it, the
      // first while the MMAs run (bringing the others into L2 then cost 2 %)
      // (z and the residual likewise)
      uint32_t gw[kGate2 || kZ ? 16 : 1], uw[kGate2 || kRes ? 16 : 1];
      if constexpr (kGate2) load_gate_up(g, tl, half, col, left, lane, gw, uw);
      if constexpr (kZ) load_words(g.gu, g.gu_ld, tl, half, col, left, lane, gw);
      if constexpr (kRes) load_words(g.res, g.res_ld, tl, half, col, left, lane, uw);
      float bias = 0.0f;   // of this lane's feature
      if constexpr (kFwdOne || kOp == kFwdGlu)
        if (g.bias && lane < left) {
          const int64_t wide = kGated ? 2 * g.n_cols : g.n_cols;
          bias = bias_at(g, tl.expert * wide + (kGated && quad >= 2 ? g.n_cols : 0) + col + lane);
        }
      if (!__all_sync(0xFFFFFFFFu, mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag,
                                                     tile_limit(g, g.k_blocks)))) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
      tc_fence_after();
      const uint32_t taddr = tmem + static_cast<uint32_t>(acc * kTokens) + (static_cast<uint32_t>(quad * 32) << 16);
      if (half >= chunks) {   // nothing here for this warp
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
      }
      for (int c = half; c < chunks; c += kStep) {
        const int tok = c * 32;
        const int64_t row = tl.row0 + tok;
        const int rows = min(32, tl.valid - tok);
        uint32_t v[32];
        tmem_ld_32x32b_x32(taddr + tok, v);
        uint32_t ng[kGate2 || kZ ? 16 : 1], nu[kGate2 || kRes ? 16 : 1];
        if constexpr (kGate2) load_gate_up(g, tl, c + kStep, col, left, lane, ng, nu);
        if constexpr (kZ) load_words(g.gu, g.gu_ld, tl, c + kStep, col, left, lane, ng);
        if constexpr (kRes) load_words(g.res, g.res_ld, tl, c + kStep, col, left, lane, nu);
        tmem_ld_wait();
        if (c + kStep >= chunks) {
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
        }
        if (left <= 0) continue;   // warp-uniform
        if constexpr (kFwdOne || kOp == kFwdGlu) {
          if (g.bias) {   // (-0 + 0 is 0: without one nothing is added)
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] = __float_as_uint(__uint_as_float(v[i]) + bias);
          }
        }
        if constexpr (kFwdOne || kZ || kRes) {
          float2 p[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) p[i] = pair_up(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), odd);
          if constexpr (kFwdOne) {
            if (g.z) {
              uint8_t* tile = next_tile();
#pragma unroll
              for (int i = 0; i < 16; ++i) put_word(tile, 2 * i + odd, lane >> 1, pack_bf16x2(p[i].x, p[i].y));
              store_tile<32>(tile, &maps.out2, rows, lane, static_cast<int>(col), 0, static_cast<int>(row),
                             g.z + row * g.z_ld + col, g.z_ld, left);
            }
          }
          const auto apply = [&](auto tag) {
            constexpr int kA = decltype(tag)::value;
            if constexpr (kA != MOE_ACT_NONE) {
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if constexpr (kFwdOne) {
                  p[i].x = act_at<kA, false>(p[i].x, nullptr);
                  p[i].y = act_at<kA, false>(p[i].y, nullptr);
                } else if constexpr (kZ) {
                  const float2 z = unpack_bf16x2(gw[i]);
                  float2 slope;
                  act_at<kA, true>(z.x, &slope.x);
                  act_at<kA, true>(z.y, &slope.y);
                  p[i].x = __fmul_rn(p[i].x, slope.x);
                  p[i].y = __fmul_rn(p[i].y, slope.y);
                }
              }
            }
          };
          if constexpr (kFwdOne || kZ) with_act(g.act, apply);
          uint8_t* tile = next_tile();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            if constexpr (kRes) {
              const float2 r = unpack_bf16x2(uw[i]);
              p[i] = make_float2(__fadd_rn(p[i].x, r.x), __fadd_rn(p[i].y, r.y));
              uw[i] = nu[i];
            }
            if constexpr (kZ) gw[i] = ng[i];
            put_word(tile, 2 * i + odd, lane >> 1, pack_bf16x2(p[i].x, p[i].y));
          }
          store_tile<32>(tile, &maps.out, rows, lane, static_cast<int>(col), 0, static_cast<int>(row),
                         g.out + row * g.out_ld + col, g.out_ld, left);
        } else if constexpr (kOp == kFwd || kOp == kDgrad) {
          uint8_t* tile = next_tile();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const float2 p = pair_up(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), odd);
            put_word(tile, 2 * i + odd, lane >> 1, pack_bf16x2(p.x, p.y));
          }
          store_tile<32>(tile, &maps.out, rows, lane, static_cast<int>(col), 0, static_cast<int>(row),
                     g.out + row * g.out_ld + col, g.out_ld, left);
        } else if constexpr (kGate2) {
          uint32_t dg[16];
          uint8_t* du_tile = next_tile();
          if constexpr (kOp == kDgradSwiglu) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 dh = pair_up(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), odd);
              const float2 gate = unpack_bf16x2(gw[i]), up = unpack_bf16x2(uw[i]);
              float2 g2, u2;
              swiglu_grad(dh.x, gate.x, up.x, &g2.x, &u2.x);
              swiglu_grad(dh.y, gate.y, up.y, &g2.y, &u2.y);
              dg[i] = pack_bf16x2(g2.x, g2.y);
              put_word(du_tile, 2 * i + odd, lane >> 1, pack_bf16x2(u2.x, u2.y));
            }
          } else {
            with_act(g.act, [&](auto tag) {
              constexpr int kA = decltype(tag)::value;
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                const float2 dh = pair_up(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), odd);
                const float2 gate = unpack_bf16x2(gw[i]), up = unpack_bf16x2(uw[i]);
                float2 slope, value;
                value.x = act_at<kA, true>(gate.x, &slope.x);
                value.y = act_at<kA, true>(gate.y, &slope.y);
                dg[i] = pack_bf16x2(dh.x * up.x * slope.x, dh.y * up.y * slope.y);
                put_word(du_tile, 2 * i + odd, lane >> 1, pack_bf16x2(dh.x * value.x, dh.y * value.y));
              }
            });
          }
          uint16_t* dst = g.out + row * g.out_ld + col;
          store_tile<32>(du_tile, &maps.out2, rows, lane, static_cast<int>(col), 0, static_cast<int>(row),
                         dst + g.n_cols, g.out_ld, left);
          uint8_t* dg_tile = next_tile();
#pragma unroll
          for (int i = 0; i < 16; ++i) put_word(dg_tile, 2 * i + odd, lane >> 1, dg[i]);
          store_tile<32>(dg_tile, &maps.out, rows, lane, static_cast<int>(col), 0, static_cast<int>(row), dst, g.out_ld,
                         left);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            gw[i] = ng[i];
            uw[i] = nu[i];
          }
        } else {
          // the g warp forms h of the chunk's first 16 tokens, the u warp of
          // the others: each gives the other its half.  Their barrier takes
          // turns: values written (even phases), values read (odd).  What a
          // warp gave away is where its part of h then goes.
          const bool is_up = quad >= 2;
          uint64_t* meet = &xchg[2 * half + (quad & 1)];
          float* mine = reinterpret_cast<float*>(stg + kStgTile);
          const float* theirs =
              reinterpret_cast<const float*>(smem + F::kOffStg + ((warp - 2) ^ 2) * F::kStgBytes + kStgTile);
          if (lane == 0) bulk_wait_read<0>();   // the chunk before's stores have read the tiles
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 16; ++i) mine[i * 32 + lane] = __uint_as_float(is_up ? v[i] : v[16 + i]);
          mbar_arrive(meet);
          if (g.out) {
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 p = pair_up(__uint_as_float(v[2 * i]), __uint_as_float(v[2 * i + 1]), odd);
              put_word(stg, 2 * i + odd, lane >> 1, pack_bf16x2(p.x, p.y));
            }
            store_tile<32>(stg, is_up ? &maps.out2 : &maps.out, rows, lane, static_cast<int>(col), 0,
                           static_cast<int>(row), g.out + row * g.out_ld + (is_up ? g.n_cols : 0) + col, g.out_ld, left);
          }
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(meet, 0, abort_flag, g.timeout_ns));
          if (!ok) break;
          float x[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = theirs[i * 32 + lane];
          mbar_arrive(meet);
          uint32_t hw[8];
          const auto form_h = [&](auto tag) {
            constexpr int kA = decltype(tag)::value;
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              float hv[2];
#pragma unroll
              for (int j = 0; j < 2; ++j) {
                const int k = 2 * i + j;
                const float gate = is_up ? x[k] : __uint_as_float(v[k]), up = is_up ? __uint_as_float(v[16 + k]) : x[k];
                hv[j] = act_at<kA, false>(gate, nullptr) * up;
              }
              const float2 p = pair_up(hv[0], hv[1], odd);
              hw[i] = pack_bf16x2(p.x, p.y);
            }
          };
          if constexpr (kOp == kFwdGlu)
            with_act(g.act, form_h);
          else
            form_h(ActTag<MOE_ACT_SILU>{});
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(meet, 1, abort_flag, g.timeout_ns));
          if (!ok) break;
          uint8_t* h_tile = stg + kStgTile;
#pragma unroll
          for (int i = 0; i < 8; ++i) put_word(h_tile, 2 * i + odd, lane >> 1, hw[i]);
          const int h0 = is_up ? 16 : 0;
          store_tile<16>(h_tile, &maps.h, rows - h0, lane, static_cast<int>(col), 0, static_cast<int>(row) + h0,
                         g.h + (row + h0) * g.h_ld + col, g.h_ld, left);
        }
      }
      if (!ok) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
        break;
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's stores have completed
  }
  // neither CTA leaves while the other's copies, MMAs or arrivals may reach it
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------------------
// Gradient of the weights
// ---------------------------------------------------------------------------
constexpr int kTileM = 256;                          // dW rows of a pair's tile, 128 per CTA
constexpr int kTileN = 256;                          // dW columns at most

// This CTA pair's tiles, in turn: tile i of expert e.
struct WgradTile {
  int expert, i;
  int64_t row0;   // the expert's first sorted row
  int mt, nt;     // output row and column tile
  int n;          // columns of the MMA: those there are, rounded up to 32
  int kb;         // reduction blocks
  int tail;       // rows of the last one

  // The pair's first tile, and the one `step` tiles on; false past the last expert.
  __device__ __forceinline__ bool first(const ExpertArgs& g, int t) {
    const int per = g.m_tiles * g.n_tiles;
    expert = t / per;
    i = t - expert * per;
    return fill(g);
  }
  __device__ __forceinline__ bool next(const ExpertArgs& g, int step) {
    const int per = g.m_tiles * g.n_tiles;
    i += step;
    while (i >= per) {
      i -= per;
      ++expert;
    }
    return fill(g);
  }
  __device__ __forceinline__ bool fill(const ExpertArgs& g) {
    if (expert >= g.E) return false;
    mt = i / g.n_tiles;
    nt = i - mt * g.n_tiles;
    const int64_t cols = g.n_cols - static_cast<int64_t>(nt) * kTileN;
    n = cols >= kTileN ? kTileN : (static_cast<int>(cols) + 31) & ~31;
    const int rows = expert_rows(g, expert);
    row0 = expert_start(g, expert);
    kb = static_cast<int>((static_cast<unsigned>(rows) + kBlockK - 1) / kBlockK);
    tail = rows - (kb - 1) * kBlockK;
    return true;
  }
};

// Tensor maps of a gradient of the weights.  a: dy, b: x, in boxes of 64 columns
// and wgrad_box_rows(i) rows, so that an expert's last rows are copied as they are,
// in two pieces at most, and what is behind them can be cleared meanwhile.  In us,
// 128 experts of 1536 x 2048 with 225 to 292 rows and with up to 1360, and 16 of
// 700: boxes of 16, 32, 48 and 64 rows, cleared once they have landed, 205, 210 and
// 56; so 196, 206 and 53; a box of every height 191, 199 and 51, but forming 128
// maps takes the host 5 us a call more than four heights do, these 38 one.
constexpr int kBoxes = 19;
struct WgradMaps {
  CUtensorMap a[kBoxes], b[kBoxes], out;
};
__host__ __device__ constexpr int wgrad_box_rows(int i) { return i < 16 ? i + 1 : 16 * (i - 14); }   // 1 .. 16, 32, 48, 64

// kF32: dW in fp32, stored or (g.accumulate) added to what is there.
template <bool kF32>
__global__ void __launch_bounds__(Cfg<kWgrad>::kThreads, 1)
    expert_wgrad_kernel(const __grid_constant__ WgradMaps maps, const ExpertArgs g) {
  using F = Cfg<kWgrad>;
  constexpr int kStages = F::kStages, kEpiWarps = F::kEpiWarps;
  constexpr int kHalf = F::kStage / 2;   // a stage: 64 rows x 128 columns of dy, then of x
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_addr = smem_u32(smem_raw);
  uint8_t* smem = smem_raw + (((raw_addr + 1023u) & ~1023u) - raw_addr);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + F::kOffTail);
  uint64_t* empty = full + kStages;
  uint64_t* cleared = empty + kStages;   // behind an expert's last rows, in both CTAs (the even CTA's)
  uint64_t* tfull = cleared + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* done = tempty + 2;
  uint32_t* holder = reinterpret_cast<uint32_t*>(smem + F::kOffTail + kTailHolder);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + F::kOffTail + kTailAbort);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&cleared[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    mbar_init(done, 1);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&maps.a[kBoxes - 1]);
    prefetch_tensormap(&maps.b[kBoxes - 1]);
    prefetch_tensormap(&maps.out);
  }
  if (warp == 1) {
    tmem_alloc_pair(holder, kTmemCols);
    tmem_relinquish_pair();
  }
  pdl_wait();
  pdl_trigger();
  report_experts(g);
  tc_fence_before();
  cluster_sync();
  tc_fence_after();
  const uint32_t tmem = *holder;
  const int t0 = blockIdx.x >> 1, t_step = gridDim.x >> 1;
  WgradTile tl;

  if (warp == 0) {
    // ------------------------------------------------------------------ producer (both CTAs)
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (bool more = tl.first(g, t0); more && ok; more = tl.next(g, t_step)) {
      const int a0 = tl.mt * kTileM + static_cast<int>(rank) * 128;
      const int b0 = tl.nt * kTileN + static_cast<int>(rank) * (tl.n / 2);
      const bool two = tl.n > 128;   // boxes of 64 columns for this CTA's half of x
      const uint32_t boxes = two ? 4 : 3;
      for (int kb = 0; kb < tl.kb; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        uint8_t* a = smem + stage * F::kStage;
        uint8_t* b = a + kHalf;
        const uint32_t bar = mapa(smem_u32(&full[stage]), 0);
        const int row = static_cast<int>(tl.row0) + kb * kBlockK;
        // a box's rows from row `at` of the block
        const auto copy = [&](int box, int at) {
          tma_load_3d_pair(a + at * 128, &maps.a[box], bar, a0, row + at, 0);
          tma_load_3d_pair(a + at * 128 + kBoxBytes, &maps.a[box], bar, a0 + 64, row + at, 0);
          tma_load_3d_pair(b + at * 128, &maps.b[box], bar, b0, row + at, 0);
          if (two) tma_load_3d_pair(b + at * 128 + kBoxBytes, &maps.b[box], bar, b0 + 64, row + at, 0);
        };
        const int rows = kb == tl.kb - 1 ? tl.tail : kBlockK;
        if (rank == 0) mbar_arrive_expect_tx_elect(&full[stage], 2 * boxes * rows * 128);
        // (pieces start at multiples of 16 rows, and the swizzle's pattern at those of 8)
        if (rows >= 16) copy(rows / 16 + 14, 0);
        if (rows & 15) copy((rows & 15) - 1, rows & 48);
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
    if (rank == 0) {
      // (values broadcast from lane 0 are known to be uniform: the MMAs' operands
      // and the loops around them stay in uniform registers)
      const uint32_t base = __shfl_sync(0xFFFFFFFFu, smem_u32(smem), 0);
      const uint32_t tm = __shfl_sync(0xFFFFFFFFu, tmem, 0);
      int stage = 0, iter = 0;
      uint32_t phase = 0, tails = 0;   // tails: parity of each stage's clearings
      bool ok = true;
      for (bool more = tl.first(g, t0); more && ok; more = tl.next(g, t_step)) {
        const int blocks = __shfl_sync(0xFFFFFFFFu, tl.kb, 0), tail = __shfl_sync(0xFFFFFFFFu, tl.tail, 0);
        if (blocks == 0) continue;
        const uint32_t idesc = kIdesc | kAMnMajor | kBMnMajor | idesc_mn(kTileM, __shfl_sync(0xFFFFFFFFu, tl.n, 0));
        const int acc = iter & 1;
        const uint32_t d = tm + static_cast<uint32_t>(acc * kTileN);
        ok = __all_sync(0xFFFFFFFFu,
                        mbar_wait_cluster_bounded(&tempty[acc], ((iter >> 1) & 1) ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        tc_fence_after();
        ++iter;
        for (int kb = 0; kb < blocks; ++kb) {
          ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&full[stage], phase, abort_flag, g.timeout_ns));
          if (!ok) break;
          int steps = 4;   // MMAs of 16 reduction rows; whole steps past the expert's end are left out
          if (kb == blocks - 1 && tail % 16) {
            ok = __all_sync(0xFFFFFFFFu,
                            mbar_wait_bounded(&cleared[stage], (tails >> stage) & 1u, abort_flag, g.timeout_ns));
            if (!ok) break;
            tails ^= 1u << stage;
          }
          if (kb == blocks - 1) steps = (tail + 15) / 16;
          tc_fence_after();
          // (16 rows of 128 bytes down the boxes)
          const uint32_t a = base + stage * F::kStage;
          const uint64_t ad = smem_desc(a, kBoxBytes, 1024, kSwizzle128B);
          const uint64_t bd = smem_desc(a + kHalf, kBoxBytes, 1024, kSwizzle128B);
          if (steps == 4) {
#pragma unroll
            for (int k = 0; k < 4; ++k)
              mma_bf16_pair(d, ad + (2048 >> 4) * k, bd + (2048 >> 4) * k, idesc, !(kb == 0 && k == 0));
          } else {
            for (int k = 0; k < steps; ++k)
              mma_bf16_pair(d, ad + (2048 >> 4) * k, bd + (2048 >> 4) * k, idesc, !(kb == 0 && k == 0));
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
      if (!ok && lane == 0) {
        set_status(g.status, MOE_ERR_TIMEOUT);
        *abort_flag = 1;
      }
      // all issued tensor-core work finished before the tensor memory is released
      tc_commit_pair(done);
      const int never = 0;
      mbar_wait_bounded(done, 0, &never, g.timeout_ns);
    }
  } else if (warp == kEpiWarps + 2) {
    // ------------------------------------------------------------------ clearing (even CTA)
    // Behind an expert's last rows the rest of their last step of 16 is cleared in
    // all four boxes (a row is 128 consecutive bytes of its box, and stays in its
    // place under the swizzle), while the rows themselves are on their way.  This
    // CTA clears both CTAs' boxes, so that all that orders it is in this CTA: an
    // arrival from the other one would have to be a release at cluster scope, with
    // which experts of up to 1360 rows took 231 us instead of 212.
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (bool more = rank == 0 && tl.first(g, t0); more && ok; more = tl.next(g, t_step)) {
      for (int kb = 0; kb < tl.kb; ++kb) {
        // (of every block, as the producer does: a phase must not be passed by)
        ok = __all_sync(0xFFFFFFFFu, mbar_wait_bounded(&empty[stage], phase ^ 1, abort_flag, g.timeout_ns));
        if (!ok) break;
        if (kb == tl.kb - 1 && tl.tail % 16) {
          const int clear = (16 - tl.tail % 16) * 8;   // 16-byte pieces of a box
          uint8_t* first = smem + stage * F::kStage + tl.tail * 128;
          const uint32_t other = mapa(smem_u32(first), 1);
          for (int i = lane; i < clear; i += 32)
#pragma unroll
            for (int box = 0; box < 4; ++box) clear_remote16(other + box * kBoxBytes + i * 16);
          for (int i = lane; i < clear; i += 32)
#pragma unroll
            for (int box = 0; box < 4; ++box)
              *reinterpret_cast<uint4*>(first + box * kBoxBytes + i * 16) = make_uint4(0, 0, 0, 0);
          // ordered before the MMAs' reads of both CTAs' boxes
          fence_proxy_async_cluster_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(&cleared[stage]);
          __syncwarp();
        }
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
  } else {
    // ------------------------------------------------------------------ epilogue (both CTAs)
    // 64 columns at a time (every other 64 of the tile): two tensor-memory
    // loads, one 32-row x 128-byte store tile (128-byte swizzle: 16-byte piece
    // j of row r at r * 128 + ((j ^ (r & 7)) * 16)), one store of whole lines.
    // fp32: two such tiles of 32 columns.  Sums are added by the copy, in L2:
    // one addition per element, so the results do not depend on the order.
    const int quad = warp & 3, half = (warp - 2) >> 2;
    uint8_t* tile = smem + F::kOffStg + (warp - 2) * F::kStgBytes;
    int iter = 0;
    bool more = tl.first(g, t0);
    while (more) {
      const int acc = iter & 1, n = tl.n, expert = tl.expert;
      const int kb = tl.kb;
      const bool any = kb > 0;
      const int64_t r0 = static_cast<int64_t>(tl.mt) * kTileM + rank * 128 + quad * 32;
      const int64_t col0 = static_cast<int64_t>(tl.nt) * kTileN;
      more = tl.next(g, t_step);   // (its loads are on their way while this tile is waited for)
      if (any) {
        if (!__all_sync(0xFFFFFFFFu,
                        mbar_wait_bounded(&tfull[acc], (iter >> 1) & 1, abort_flag, tile_limit(g, kb)))) {
          set_status(g.status, MOE_ERR_TIMEOUT);
          *abort_flag = 1;
          break;
        }
        tc_fence_after();
        ++iter;
      }
      const uint32_t taddr = tmem + static_cast<uint32_t>(acc * kTileN) + (static_cast<uint32_t>(quad * 32) << 16);
      if (any && 64 * half >= n) {   // nothing here for this warp
        __syncwarp();
        if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
      }
#pragma unroll 1
      for (int c = 64 * half; c < n; c += 64 * (kEpiWarps / 4)) {
        uint4 o[kF32 ? 16 : 8];
        if (any) {
          // (the second 32 columns may lie past the MMA's: loaded all the same,
          // from columns of this accumulator, and clipped by the store)
          uint32_t v[32], u[32];
          tmem_ld_32x32b_x32(taddr + c, v);
          tmem_ld_32x32b_x32(taddr + c + 32, u);
          tmem_ld_wait();
          if (c + 64 * (kEpiWarps / 4) >= n) {
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_remote(mapa(smem_u32(&tempty[acc]), 0));
          }
          if constexpr (kF32) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              o[j] = make_uint4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
              o[8 + j] = make_uint4(u[4 * j], u[4 * j + 1], u[4 * j + 2], u[4 * j + 3]);
            }
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              o[j] = pack8(v + 8 * j);
              o[4 + j] = pack8(u + 8 * j);
            }
          }
        } else {
          if (kF32 && g.accumulate) break;   // nothing to add
#pragma unroll
          for (int j = 0; j < (kF32 ? 16 : 8); ++j) o[j] = make_uint4(0, 0, 0, 0);
        }
        if (r0 >= g.n_rows) continue;        // warp-uniform
#pragma unroll
        for (int h = 0; h < (kF32 ? 2 : 1); ++h) {
          if (kF32 && c + 32 * h >= n) break;   // past the last column
          if (lane == 0) bulk_wait_read<0>();   // the store before has read the tile
          __syncwarp();
#pragma unroll
          for (int j = 0; j < 8; ++j)
            *reinterpret_cast<uint4*>(tile + lane * 128 + ((j ^ (lane & 7)) << 4)) = o[8 * h + j];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            // (rows past N and columns past C are clipped by the map)
            const int col = static_cast<int>(col0) + c + 32 * h;
            if (kF32 && g.accumulate)
              tma_add_3d(&maps.out, tile, col, static_cast<int>(r0), expert);
            else
              tma_store_3d(&maps.out, tile, col, static_cast<int>(r0), expert);
            bulk_commit_group();
          }
        }
      }
    }
    if (lane == 0) bulk_wait_all();   // this warp's stores have completed
  }
  // neither CTA leaves while the other's copies, MMAs or arrivals may reach it
  __syncwarp();
  cluster_sync();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem, kTmemCols);
  }
}

// The status of a call without sorted rows, which no product runs for.
__global__ void report_kernel(const ExpertArgs g) {
  pdl_wait();
  pdl_trigger();
  report_experts(g);
}

// max_tiles: at least the tiles of any split of the rows among the experts.
template <ExpertOp kOp>
cudaError_t launch_rows(const RowsMaps& maps, const ExpertArgs& g, int64_t max_tiles, cudaStream_t s) {
  using F = Cfg<kOp>;
  static PerDevice known;
  int pairs = 0;
  const cudaError_t e = on_current_device(
      known, &pairs, [](int* n) { return resident_pairs(expert_rows_kernel<kOp>, F::kThreads, F::kSmem, n); });
  if (e != cudaSuccess) return e;
  const int grid = 2 * static_cast<int>(max_tiles < pairs ? max_tiles : pairs);
  return launch_pdl_cluster(expert_rows_kernel<kOp>, dim3(grid), dim3(F::kThreads), F::kSmem, s, 2, maps, g);
}

template <bool kF32>
cudaError_t launch_wgrad(const WgradMaps& maps, const ExpertArgs& g, int64_t tiles, cudaStream_t s) {
  using F = Cfg<kWgrad>;
  static PerDevice known;
  int pairs = 0;
  const cudaError_t e = on_current_device(
      known, &pairs, [](int* n) { return resident_pairs(expert_wgrad_kernel<kF32>, F::kThreads, F::kSmem, n); });
  if (e != cudaSuccess) return e;
  const int grid = 2 * static_cast<int>(tiles < pairs ? tiles : pairs);
  return launch_pdl_cluster(expert_wgrad_kernel<kF32>, dim3(grid), dim3(F::kThreads), F::kSmem, s, 2, maps, g);
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
// x of a rows launch: boxes of 128, 96, 64 and 32 rows.
moe_status_t token_maps(RowsMaps* m, const void* p, int64_t rows, int64_t cols, int64_t ld) {
  for (int i = 0; i < 4; ++i) {
    const moe_status_t st = rows_map(&m->x[i], p, rows, cols, ld, 128 - 32 * i);
    if (st != MOE_OK) return st;
  }
  return MOE_OK;
}
// [rows][1][cols] output with row stride ld, stored box_rows rows x 32 columns at a time.
moe_status_t out_map(CUtensorMap* m, const void* p, int64_t rows, int64_t cols, int64_t ld, uint32_t box_rows = 32) {
  const uint64_t d[3] = {static_cast<uint64_t>(cols), 1, static_cast<uint64_t>(rows)};
  const uint64_t st[2] = {static_cast<uint64_t>(ld) * 2, static_cast<uint64_t>(ld) * 2};
  const uint32_t box[3] = {32, 1, box_rows};
  return encode_tiled_map(m, p, kBf16, 3, d, st, box, CU_TENSOR_MAP_SWIZZLE_64B);
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

FewRows few_args(int64_t rows, int64_t cols, void* out, int64_t out_ld, void* status) {
  FewRows g;
  memset(&g, 0, sizeof(g));
  g.rows = static_cast<int32_t>(rows);
  g.cols = cols;
  g.out = static_cast<uint16_t*>(out);
  g.out_ld = out_ld;
  g.status = static_cast<int32_t*>(status);
  return g;
}

// What the products with an epilogue of their own add: a bias, and a matrix of rows
// that may be missing.
moe_status_t check_bias(const void* bias, int32_t elem) {
  if (!bias) return MOE_OK;
  if (elem != MOE_ELEM_BF16 && elem != MOE_ELEM_F32) return MOE_ERR_INVALID_ARG;
  return reinterpret_cast<uintptr_t>(bias) & (elem == MOE_ELEM_F32 ? 3 : 1) ? MOE_ERR_MISALIGNED : MOE_OK;
}
moe_status_t check_optional(const void* p, int64_t ld, int64_t cols) {
  if (!p) return MOE_OK;
  if (ld < cols) return MOE_ERR_INVALID_ARG;
  if (ld % 8 || ld > (int64_t(1) << 36)) return MOE_ERR_UNSUPPORTED;
  return off16(p) ? MOE_ERR_MISALIGNED : MOE_OK;
}
bool is_act(int32_t act) { return act >= MOE_ACT_NONE && act <= MOE_ACT_RELU2; }

int32_t ceil_div(int64_t a, int64_t b) { return static_cast<int32_t>((a + b - 1) / b); }

// Token blocks, of the lowest height, of any split of `rows` rows among E experts, at most.
int64_t max_blocks(int64_t rows, int32_t E) { return rows / (kTokens >> 3) + E; }

// rows == 0: experts that claim some are reported as ever.
moe_status_t no_rows(int32_t E, const int32_t* start, const int32_t* counts, void* status, void* stream) {
  return as_status(launch_pdl(report_kernel, dim3(1), dim3(256), 0, static_cast<cudaStream_t>(stream),
                              expert_args(0, E, start, counts, status)));
}

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
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, N, 64))
    return launch_few_rows(kFewFwd, few_args(rows, N, y, y_ld, status), x, x_ld, C, w, stream);
  RowsMaps m;
  if ((st = token_maps(&m, x, rows, C, x_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w, E, N, C, 128)) != MOE_OK) return st;
  if ((st = out_map(&m.out, y, rows, N, y_ld)) != MOE_OK) return st;
  m.out2 = m.h = m.out;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(N, 256);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = N;
  g.out = static_cast<uint16_t*>(y);
  g.out_ld = y_ld;
  return as_status(launch_rows<kFwd>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
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
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, I, 32)) {
    FewRows f = few_args(rows, I, h, h_ld, status);
    f.act = MOE_ACT_SILU;
    f.keep = static_cast<uint16_t*>(gu);
    f.keep_ld = gu_ld;
    return launch_few_rows(kFewFwdGlu, f, x, x_ld, C, w13, stream);
  }
  RowsMaps m;
  if ((st = token_maps(&m, x, rows, C, x_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w13, E, 2 * I, C, 64)) != MOE_OK) return st;
  if ((st = out_map(&m.h, h, rows, I, h_ld, 16)) != MOE_OK) return st;
  m.out = m.out2 = m.h;
  if (gu && (st = out_map(&m.out, gu, rows, I, gu_ld)) != MOE_OK) return st;
  if (gu && (st = out_map(&m.out2, static_cast<uint16_t*>(gu) + I, rows, I, gu_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, 128);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(gu);
  g.out_ld = gu_ld;
  g.h = static_cast<uint16_t*>(h);
  g.h_ld = h_ld;
  return as_status(
      launch_rows<kFwdSwiglu>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad(const void* dy, int64_t dy_ld, int64_t rows, const void* w, const int32_t* start,
                                   const int32_t* counts, int32_t E, int64_t N, int64_t C, void* dx, int64_t dx_ld,
                                   void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{dy, dy_ld, N}, {dx, dx_ld, C}});
  if (st != MOE_OK) return st;
  if (!w) return MOE_ERR_INVALID_ARG;
  if (off16(w)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, C, 64))
    return launch_few_rows(kFewGrad, few_args(rows, C, dx, dx_ld, status), dy, dy_ld, N, w, stream);
  RowsMaps m;
  if ((st = token_maps(&m, dy, rows, N, dy_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w, E, N, C, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&m.out, dx, rows, C, dx_ld)) != MOE_OK) return st;
  m.out2 = m.h = m.out;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(C, 256);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = C;
  g.out = static_cast<uint16_t*>(dx);
  g.out_ld = dx_ld;
  return as_status(launch_rows<kDgrad>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad_swiglu(const void* dy, int64_t dy_ld, int64_t rows, const void* w2, const void* gu,
                                          int64_t gu_ld, const int32_t* start, const int32_t* counts, int32_t E,
                                          int64_t N, int64_t I, void* dgu, int64_t dgu_ld, void* status, void* stream) {
  moe_status_t st =
      check_expert(rows, E, N, I, start, counts, status, {{dy, dy_ld, N}, {gu, gu_ld, 2 * I}, {dgu, dgu_ld, 2 * I}});
  if (st != MOE_OK) return st;
  if (!w2) return MOE_ERR_INVALID_ARG;
  if (off16(w2)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  RowsMaps m;
  if ((st = token_maps(&m, dy, rows, N, dy_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w2, E, N, I, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&m.out, dgu, rows, I, dgu_ld)) != MOE_OK) return st;
  if ((st = out_map(&m.out2, static_cast<uint16_t*>(dgu) + I, rows, I, dgu_ld)) != MOE_OK) return st;
  m.h = m.out;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, 256);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(dgu);
  g.out_ld = dgu_ld;
  g.gu = static_cast<const uint16_t*>(gu);
  g.gu_ld = gu_ld;
  return as_status(
      launch_rows<kDgradSwiglu>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_act(const void* x, int64_t x_ld, int64_t rows, const void* w, const void* bias,
                                 int32_t bias_elem, int32_t act, const void* residual, int64_t residual_ld,
                                 const int32_t* start, const int32_t* counts, int32_t E, int64_t N, int64_t C, void* z,
                                 int64_t z_ld, void* y, int64_t y_ld, void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{x, x_ld, C}, {y, y_ld, N}});
  if (st != MOE_OK) return st;
  if (!w || !is_act(act)) return MOE_ERR_INVALID_ARG;
  if (off16(w)) return MOE_ERR_MISALIGNED;
  if ((st = check_bias(bias, bias_elem)) != MOE_OK) return st;
  if ((st = check_optional(residual, residual_ld, N)) != MOE_OK) return st;
  if ((st = check_optional(z, z_ld, N)) != MOE_OK) return st;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, N, 64)) {
    FewRows f = few_args(rows, N, y, y_ld, status);
    f.act = act;
    f.bias = bias;
    f.bias_f32 = bias_elem == MOE_ELEM_F32;
    f.res = static_cast<const uint16_t*>(residual);
    f.res_ld = residual_ld;
    f.keep = static_cast<uint16_t*>(z);
    f.keep_ld = z_ld;
    return launch_few_rows(kFewFwd, f, x, x_ld, C, w, stream);
  }
  RowsMaps m;
  if ((st = token_maps(&m, x, rows, C, x_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w, E, N, C, 128)) != MOE_OK) return st;
  if ((st = out_map(&m.out, y, rows, N, y_ld)) != MOE_OK) return st;
  m.out2 = m.h = m.out;
  if (z && (st = out_map(&m.out2, z, rows, N, z_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(N, 256);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = N;
  g.out = static_cast<uint16_t*>(y);
  g.out_ld = y_ld;
  g.act = act;
  g.bias = bias;
  g.bias_f32 = bias_elem == MOE_ELEM_F32;
  g.res = static_cast<const uint16_t*>(residual);
  g.res_ld = residual_ld;
  g.z = static_cast<uint16_t*>(z);
  g.z_ld = z_ld;
  return as_status((residual ? launch_rows<kFwdActRes> : launch_rows<kFwdAct>)(
      m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_glu(const void* x, int64_t x_ld, int64_t rows, const void* w13, const void* bias,
                                 int32_t bias_elem, int32_t act, const int32_t* start, const int32_t* counts, int32_t E,
                                 int64_t I, int64_t C, void* gu, int64_t gu_ld, void* h, int64_t h_ld, void* status,
                                 void* stream) {
  moe_status_t st = check_expert(rows, E, I, C, start, counts, status, {{x, x_ld, C}, {h, h_ld, I}});
  if (st != MOE_OK) return st;
  if (!w13 || !is_act(act)) return MOE_ERR_INVALID_ARG;
  if (off16(w13)) return MOE_ERR_MISALIGNED;
  if ((st = check_bias(bias, bias_elem)) != MOE_OK) return st;
  if ((st = check_optional(gu, gu_ld, 2 * I)) != MOE_OK) return st;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, I, 32)) {
    FewRows f = few_args(rows, I, h, h_ld, status);
    f.act = act;
    f.bias = bias;
    f.bias_f32 = bias_elem == MOE_ELEM_F32;
    f.keep = static_cast<uint16_t*>(gu);
    f.keep_ld = gu_ld;
    return launch_few_rows(kFewFwdGlu, f, x, x_ld, C, w13, stream);
  }
  RowsMaps m;
  if ((st = token_maps(&m, x, rows, C, x_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w13, E, 2 * I, C, 64)) != MOE_OK) return st;
  if ((st = out_map(&m.h, h, rows, I, h_ld, 16)) != MOE_OK) return st;
  m.out = m.out2 = m.h;
  if (gu && (st = out_map(&m.out, gu, rows, I, gu_ld)) != MOE_OK) return st;
  if (gu && (st = out_map(&m.out2, static_cast<uint16_t*>(gu) + I, rows, I, gu_ld)) != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, 128);
  g.k_blocks = ceil_div(C, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(gu);
  g.out_ld = gu_ld;
  g.h = static_cast<uint16_t*>(h);
  g.h_ld = h_ld;
  g.act = act;
  g.bias = bias;
  g.bias_f32 = bias_elem == MOE_ELEM_F32;
  return as_status(launch_rows<kFwdGlu>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad_act(const void* dy, int64_t dy_ld, int64_t rows, const void* w, const void* z,
                                       int64_t z_ld, int32_t act, const void* residual, int64_t residual_ld,
                                       const int32_t* start, const int32_t* counts, int32_t E, int64_t N, int64_t C,
                                       void* dx, int64_t dx_ld, void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{dy, dy_ld, N}, {dx, dx_ld, C}});
  if (st != MOE_OK) return st;
  if (!w || !is_act(act) || (act != MOE_ACT_NONE && !z && rows > 0)) return MOE_ERR_INVALID_ARG;
  if (off16(w)) return MOE_ERR_MISALIGNED;
  if (act == MOE_ACT_NONE) z = nullptr;
  if ((st = check_optional(z, z_ld, C)) != MOE_OK) return st;
  if ((st = check_optional(residual, residual_ld, C)) != MOE_OK) return st;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, C, 64)) {
    FewRows f = few_args(rows, C, dx, dx_ld, status);
    f.act = act;
    f.z = static_cast<const uint16_t*>(z);
    f.z_ld = z_ld;
    f.res = static_cast<const uint16_t*>(residual);
    f.res_ld = residual_ld;
    return launch_few_rows(kFewGrad, f, dy, dy_ld, N, w, stream);
  }
  RowsMaps m;
  if ((st = token_maps(&m, dy, rows, N, dy_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w, E, N, C, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&m.out, dx, rows, C, dx_ld)) != MOE_OK) return st;
  m.out2 = m.h = m.out;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(C, 256);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = C;
  g.out = static_cast<uint16_t*>(dx);
  g.out_ld = dx_ld;
  g.act = act;
  g.gu = static_cast<const uint16_t*>(z);
  g.gu_ld = z_ld;
  g.res = static_cast<const uint16_t*>(residual);
  g.res_ld = residual_ld;
  const auto launch = act == MOE_ACT_NONE ? (residual ? launch_rows<kDgradRes> : launch_rows<kDgrad>)
                                          : (residual ? launch_rows<kDgradActRes> : launch_rows<kDgradAct>);
  return as_status(launch(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_dgrad_glu(const void* dy, int64_t dy_ld, int64_t rows, const void* w2, const void* gu,
                                       int64_t gu_ld, int32_t act, const int32_t* start, const int32_t* counts, int32_t E,
                                       int64_t N, int64_t I, void* dgu, int64_t dgu_ld, void* status, void* stream) {
  moe_status_t st =
      check_expert(rows, E, N, I, start, counts, status, {{dy, dy_ld, N}, {gu, gu_ld, 2 * I}, {dgu, dgu_ld, 2 * I}});
  if (st != MOE_OK) return st;
  if (!w2 || !is_act(act)) return MOE_ERR_INVALID_ARG;
  if (off16(w2)) return MOE_ERR_MISALIGNED;
  if (rows == 0) return no_rows(E, start, counts, status, stream);
  if (few_rows(start, rows, I, 64)) {
    FewRows f = few_args(rows, I, dgu, dgu_ld, status);
    f.act = act;
    f.z = static_cast<const uint16_t*>(gu);
    f.z_ld = gu_ld;
    return launch_few_rows(kFewGradGlu, f, dy, dy_ld, N, w2, stream);
  }
  RowsMaps m;
  if ((st = token_maps(&m, dy, rows, N, dy_ld)) != MOE_OK) return st;
  if ((st = weights_map(&m.w, w2, E, N, I, kBlockK)) != MOE_OK) return st;
  if ((st = out_map(&m.out, dgu, rows, I, dgu_ld)) != MOE_OK) return st;
  if ((st = out_map(&m.out2, static_cast<uint16_t*>(dgu) + I, rows, I, dgu_ld)) != MOE_OK) return st;
  m.h = m.out;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(I, 256);
  g.k_blocks = ceil_div(N, kBlockK);
  g.n_cols = I;
  g.out = static_cast<uint16_t*>(dgu);
  g.out_ld = dgu_ld;
  g.act = act;
  g.gu = static_cast<const uint16_t*>(gu);
  g.gu_ld = gu_ld;
  return as_status(launch_rows<kDgradGlu>(m, g, max_blocks(rows, E) * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

moe_status_t moe_expert_gemm_wgrad(const void* dy, int64_t dy_ld, const void* x, int64_t x_ld, int64_t rows,
                                   const int32_t* start, const int32_t* counts, int32_t E, int64_t N, int64_t C,
                                   void* dw, int32_t dw_elem, int32_t accumulate, void* status, void* stream) {
  moe_status_t st = check_expert(rows, E, N, C, start, counts, status, {{dy, dy_ld, N}, {x, x_ld, C}});
  if (st != MOE_OK) return st;
  if (!dw || (dw_elem != MOE_ELEM_BF16 && dw_elem != MOE_ELEM_F32)) return MOE_ERR_INVALID_ARG;
  const bool f32 = dw_elem == MOE_ELEM_F32;
  if (accumulate && !f32) return MOE_ERR_UNSUPPORTED;
  if (off16(dw)) return MOE_ERR_MISALIGNED;
  const uint64_t size = f32 ? 4 : 2;
  if (rows == 0) {   // no expert has rows
    if (!accumulate) {
      const cudaError_t e = cudaMemsetAsync(dw, 0, size * E * N * C, static_cast<cudaStream_t>(stream));
      if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return no_rows(E, start, counts, status, stream);
  }
  WgradMaps m;
  for (int i = 0; i < kBoxes; ++i) {
    if ((st = rows_map(&m.a[i], dy, rows, N, dy_ld, wgrad_box_rows(i))) != MOE_OK) return st;
    if ((st = rows_map(&m.b[i], x, rows, C, x_ld, wgrad_box_rows(i))) != MOE_OK) return st;
  }
  const uint64_t d[3] = {static_cast<uint64_t>(C), static_cast<uint64_t>(N), static_cast<uint64_t>(E)};
  const uint64_t strides[2] = {C * size, static_cast<uint64_t>(N) * C * size};
  const uint32_t box[3] = {static_cast<uint32_t>(128 / size), 32, 1};
  st = encode_tiled_map(&m.out, dw, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : kBf16, 3, d, strides, box,
                        CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != MOE_OK) return st;
  ExpertArgs g = expert_args(rows, E, start, counts, status);
  g.n_tiles = ceil_div(C, kTileN);
  g.m_tiles = ceil_div(N, kTileM);
  g.n_rows = N;
  g.n_cols = C;
  g.accumulate = accumulate != 0;
  return as_status((f32 ? launch_wgrad<true> : launch_wgrad<false>)(
      m, g, static_cast<int64_t>(E) * g.m_tiles * g.n_tiles, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
