// fathom_kv_attention, many rows (a prompt or a chunk of one): softmax(Q K^T) V
// over the paged cache on the tcgen05 tensor cores.
//
// A unit is 256 (token, head) pairs of one sequence and KV head, as two tiles
// of 128 rows (one, beyond 128 dimensions): the G heads that share a KV head share its keys.  One
// thread block per SM takes a unit through its keys, 128 at a time:
//   S = Q_i K^T        tcgen05.mma, Q and K in shared memory, S in tensor memory
//   P_i = 2^(c S - m_i)     one thread a row, from registers, rounded to bf16, V's type
//   O_i += P_i V       tcgen05.mma, P_i from tensor memory, O_i stays there
// with c = scale * log2 e.  The two tiles alternate, so that the tensor cores
// multiply one while the other's softmax is worked out.  The softmax takes a whole
// row of S into registers at once, so one S serves both tiles and the next scores
// are ready when a softmax ends.  (With an S for each tile, P over its columns, a
// tile's next scores had to wait for its softmax and its product with V: 3700
// clocks for a tile of keys, of which 2600 were softmax.)  A row's reference m
// moves only when its maximum has grown by more than 2^8 (weights up to 2^8 are as
// exact in bf16 and fp32 as those up to 1); then the row of O is rescaled.  The sum of
// the weights is of them before rounding; out is off by 0.0021 of its size, of which
// its own rounding to bf16 is 0.0017.
//
// Bound by the tensor cores and, next to them, by the exponentials: for 256 rows
// and 128 keys 4 products of 128 x 128 x 128 take 2048 clocks of the tensor pipe,
// and 32768 exponentials 2048 clocks of the special-function units.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles, 8 loads K and V by TMA (boxes of
// one page's rows, 128-byte swizzle) into a ring of 4 tiles, 9 issues the MMAs, 10
// and 11 look after V's edges.  An e4m3 cache is widened first, once for all
// units: widen_kernel writes the visible keys' bf16 values (exact, the power-of-two
// scale included) to the workspace, and the units read those.  (Widening inside
// the units, each for itself, held them to 528 TFLOP/s; loads by cp.async from
// four warps held bf16 to 807.)
//
// With 32 query and 8 KV heads, d = 128: 4096 rows over 32768 e4m3 tokens 1.78 ms
// (1160 TFLOP/s, at the board's power limit), 8192 rows with a window of 2048 over
// bf16 309 us (780 TFLOP/s: a unit's 18 tiles of keys do not hide its start and end).
//
// Masks are applied to S, where a tile of keys is not seen whole.  A masked key's
// weight is an exact zero, but 0 * NaN is not.  So in such tiles V's rows that no
// row of the unit sees become zeros, and where a value that some row does not see
// is not finite, the unit is marked and the few-rows kernel (which masks V row by
// row) does it again afterwards.
#include <cuda.h>
#include <cuda_fp8.h>

#include "kv_attention.cuh"
#include "tc_common.cuh"

namespace fathom {

namespace {

constexpr int kSoftWarps = 8;  // 4 for each tile
constexpr int kTmaWarp = 8, kMmaWarp = 9, kEdgeWarp0 = 10, kEdgeWarps = 2;
constexpr int kThreads = 32 * (kEdgeWarp0 + kEdgeWarps);  // 384
constexpr int kEdgeThreads = 32 * kEdgeWarps;
// Registers: 384 threads are launched with 168 each, 64512 in all.  The softmax
// keeps a row of 128 scores in registers; the others give theirs up:
// 256 * 224 + 128 * 56 = 64512.
constexpr int kSoftRegs = 224, kOtherRegs = 56;
static_assert(kSoftRegs * 256 + kOtherRegs * 128 <= 168 * kThreads, "registers of the block");
constexpr int kM = 128;                  // rows of a tile
constexpr int kN = kPromptTile;          // keys of a tile
constexpr int kPanel = kM * 128;         // bytes of 64 dimensions of 128 rows
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.0f;           // a row's reference lags its maximum by less

// A kernel is made for DP = 64, 128 or 256 dimensions, or (not FULL, which costs 3%)
// for fewer than 128 or 256.  (TMA fills the boxes
// past d with zeros; products go over d dimensions alone.)  Up to 128 a unit has
// two row tiles and the ring four places; at 256 tensor memory has room for one O
// and shared memory for one tile of Q and a ring of two.
template <int DP>
struct Size {
  static constexpr int kTiles = DP <= 128 ? 2 : 1;
  static constexpr int kStages = DP <= 128 ? 4 : 2;
  static constexpr int kTileBytes = DP / 64 * kPanel;
  // Q's tiles, then the ring; 1024-byte aligned (the swizzle's period).  More than
  // half an SM's, so that two blocks never share an SM and its tensor memory.
  static constexpr int kBytes = (kTiles + kStages) * kTileBytes + 1024;
  static constexpr int kSmem = kBytes < 120 * 1024 ? 120 * 1024 : kBytes;
};
static_assert(Size<256>::kTiles * 128 == prompt_cols(256) && Size<128>::kTiles * 128 == prompt_cols(128),
              "units as the plan has them");

// 128-byte swizzle.  K-major (Q, K): 8-row groups 1024 bytes apart.  MN-major
// (V, whose rows are the contracted keys): 8-key groups 1024 bytes apart, groups
// of 64 dimensions a panel apart.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t lbo) {
  return (uint64_t)((addr >> 4) & 0x3fffu) | ((uint64_t)((lbo >> 4) & 0x3fffu) << 16) |
         ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

// bf16 operands, fp32 result, M = 128; B K-major or MN-major.
constexpr uint32_t idesc(int n, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(kM >> 4) << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d),
      "l"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d),
      "r"(a), "l"(b), "r"(id), "r"(acc)
      : "memory");
}

__device__ __forceinline__ void proxy_fence() {
  asm volatile("fence.proxy.async.shared::cta;\n" ::: "memory");
}

template <int N>
__device__ __forceinline__ void regs_up() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;\n" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_down() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;\n" ::"n"(N));
}

// 2^x, results below 2^-126 to 0 (hardware; off by 2^-22 of the value).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Two fp32 operations in one.
__device__ __forceinline__ uint64_t pack2(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// mbar_wait with one answer for the whole (converged) warp.
__device__ __forceinline__ bool warp_wait(uint32_t bar, uint32_t parity) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity));
}

__device__ __forceinline__ uint32_t bf16x2(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

// A box of the tensor map from row y and dimension x into shared memory; its bytes
// count towards the barrier.
__device__ __forceinline__ void tma_box(uint32_t dst, const CUtensorMap *map, int x, int y,
                                        uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], "
      "[%1, {%2, %3}], [%4];\n" ::"r"(dst),
      "l"(map), "r"(x), "r"(y), "r"(bar)
      : "memory");
}
__device__ __forceinline__ void mbar_expect(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .b64 st;\n\t"
      "mbarrier.arrive.expect_tx.shared::cta.b64 st, [%0], %1;\n\t}\n" ::"r"(bar),
      "r"(bytes)
      : "memory");
}

// Whether one of two bf16 values is an infinity or a NaN.
__device__ __forceinline__ uint32_t nonfinite2(uint32_t w) {
  return ((w & 0x7f807f80u) + 0x00800080u) & 0x80008000u;
}

// Four e4m3 codes times 2^e as four bf16 values (exact).
__device__ __forceinline__ uint2 widen4(uint32_t w, float f) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h0) : "h"((uint16_t)w));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;\n" : "=r"(h1) : "h"((uint16_t)(w >> 16)));
  const float2 a = __half22float2(*reinterpret_cast<const __half2 *>(&h0));
  const float2 b = __half22float2(*reinterpret_cast<const __half2 *>(&h1));
  return make_uint2(bf16x2(a.x * f, a.y * f), bf16x2(b.x * f, b.y * f));
}

__device__ __forceinline__ void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};\n" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];\n"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

// The low n bits (n may be anything).
__device__ __forceinline__ uint32_t low_bits(int n) {
  return n <= 0 ? 0u : (n >= 32 ? 0xffffffffu : (1u << n) - 1u);
}

// Columns c0 + x of a unit (x < 65536 - G) as rows and heads, without a division each.
struct Columns {
  int row, head, G;
  uint32_t magic;  // 2^32 / G, rounded up
  __device__ __forceinline__ Columns(int c0, int heads) {
    G = heads;
    row = c0 / heads;
    head = c0 - row * heads;
    magic = 0xffffffffu / (uint32_t)heads + 1;  // (0 for G = 1)
  }
  // row (past c0's) and head of column c0 + x; exact while x + head < 2^16, G < 2^16
  __device__ __forceinline__ int row_of(int x) const {
    return G == 1 ? x : (int)__umulhi((uint32_t)(head + x), magic);
  }
  __device__ __forceinline__ int head_of(int x) const { return head + x - row_of(x) * G; }
};

// A thread block's number among a launch's units (those of all KV heads side by
// side) and their splits: units from number tail_from on are divided over `splits`
// blocks each.
struct Unit {
  int unit, split, splits;
};

__device__ __forceinline__ Unit unit_of(const KvAttnParams &a, int x) {
  if (x < a.tail_from) return {x, 0, 1};
  x -= a.tail_from;
  return {a.tail_from + x / a.splits, x % a.splits, a.splits};
}

__host__ __device__ __forceinline__ int unit_blocks(const KvAttnParams &a) {
  const int units = a.units * a.b.h_kv, tail = units > a.tail_from ? units - a.tail_from : 0;
  return units - tail + tail * a.splits;
}

template <int DP, bool FULL>
__global__ void __launch_bounds__(kThreads, 1)
    kv_prompt_kernel(const __grid_constant__ KvAttnParams a, const __grid_constant__ CUtensorMap map_k,
                     const __grid_constant__ CUtensorMap map_v) {
  constexpr int kTile = Size<DP>::kTileBytes, kTiles = Size<DP>::kTiles, kStages = Size<DP>::kStages;
  constexpr int kChunks = DP / 8;  // 16-byte pieces of a row in shared memory
  const int d = FULL ? DP : a.d;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[3 * kStages + 12];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fault;
  grid_dependency_wait();
  allow_dependent_launch();
  if ((int)blockIdx.x == unit_blocks(a)) {  // one more, in the first launch
    write_status(a);
    return;
  }
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const Unit u = unit_of(a, blockIdx.x);
  const int split = u.split;
  const int head = u.unit % a.b.h_kv;
  const KvUnit ku = kv_unit(a, u.unit / a.b.h_kv);
  const int s = ku.s, pair = s * a.b.h_kv + head;
  if (pair < a.pair0 || pair >= a.pair0 + a.pairs) return;  // another launch's
  int *taint = a.taint + (int64_t)u.unit * a.splits + split;
  if (tid < (u.splits == 1 ? a.splits : 1)) taint[tid] = 0;
  const KvSeq q = kv_seq(a.b, s);
  // later rows see more keys: a sequence's last unit comes first
  const int rb = (q.rows * a.G + kM * kTiles - 1) / (kM * kTiles) - 1 - ku.ct;
  if (rb < 0 || !owns(a, q)) return;
  const int c0 = rb * kM * kTiles, c1 = min(c0 + kM * kTiles, q.rows * a.G);
  const int first = q.len - q.rows;  // position of the sequence's first row
  const int p_lo = first + c0 / a.G, p_hi = first + (c1 - 1) / a.G;
  const KvTiles tiles = visible_tiles(a, p_lo, p_hi, kN);
  const int run = u.splits == 1 ? tiles.count : a.tiles_per_split;
  const int i0 = split * run;
  const int nt = min(tiles.count - i0, run);  // tiles of this block
  if (split > 0 && nt <= 0) return;
  const int n_m = c1 - c0 > kM ? 2 : 1;  // tiles of rows
  const Columns cols(c0, a.G);

  // The softmax warps' 32 rows of Q each (zeros behind the last), a row by 8 to 32
  // lanes: 16 loads on their way while the block sets up, looked at afterwards.
  constexpr int kEarly = kChunks < 16 ? kChunks : 16;
  uint4 xq[kEarly];
  auto load_q = [&](int i) {  // a row behind the last: the last; dimensions past d: zeros
    const int x = min(32 * warp + (32 * i + lane) / kChunks, c1 - 1 - c0), ch = lane % kChunks;
    if (8 * ch >= d) return make_uint4(0, 0, 0, 0);
    const uint16_t *e = static_cast<const uint16_t *>(a.q) +
                        (int64_t)(q.row0 + cols.row + cols.row_of(x)) * a.q_stride +
                        (head * a.G + cols.head_of(x)) * d + 8 * ch;
    if (a.q_wide) return __ldg(reinterpret_cast<const uint4 *>(e));
    return make_uint4(e[0] | ((uint32_t)e[1] << 16), e[2] | ((uint32_t)e[3] << 16),
                      e[4] | ((uint32_t)e[5] << 16), e[6] | ((uint32_t)e[7] << 16));
  };
  if (warp < 4 * kTiles && nt > 0)
#pragma unroll
    for (int i = 0; i < kEarly; ++i) xq[i] = load_q(i);

  const uint32_t base = (tc_smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, ring = base + kTiles * kTile;
  const uint32_t bar0 = tc_smem_u32(s_bar);
  auto kv_full = [&](int i) { return bar0 + 8 * i; };                  // TMA's bytes are there
  auto kv_empty = [&](int i) { return bar0 + 8 * (kStages + i); };     // the MMAs are done with it
  auto v_ready = [&](int i) { return bar0 + 8 * (2 * kStages + i); };  // V's edges are in order
  auto q_full = [&](int i) { return bar0 + 8 * (3 * kStages + i); };
  auto s_full = [&](int i) { return bar0 + 8 * (3 * kStages + 2 + i); };
  // half of P_i: its keys 0-63, 64-127
  auto p_full = [&](int i, int half) { return bar0 + 8 * (3 * kStages + 4 + 2 * i + half); };
  auto s_read = [&](int i) { return bar0 + 8 * (3 * kStages + 8 + i); };   // S is in registers
  auto o_done = [&](int i) { return bar0 + 8 * (3 * kStages + 10 + i); };  // O_i += P_i V

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     tc_smem_u32(&s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (warp == kTmaWarp && lane == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kv_full(i), 1);
      mbar_init(kv_empty(i), 1);
      mbar_init(v_ready(i), kEdgeThreads);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(q_full(i), kM);
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i, 0), kM);
      mbar_init(p_full(i, 1), kM);
      mbar_init(s_read(i), kM);
      mbar_init(o_done(i), 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    s_fault = 0;
  }
  // the page of the token `key`, -1 where there is none
  auto page_of = [&](int key) {
    return key < q.len ? kv_page(a.b, s, (int)((unsigned)key / (unsigned)a.b.page_tokens)) : -1;
  };
  // K and V of tile j into the ring, by the TMA warp: a lane per box (box_rows rows of
  // one page, 64 dimensions).  False if the ring's places did not become free.
  const int panels = (d + 63) / 64;
  const int box_row = lane / panels * a.box_rows, box_panel = lane % panels;
  // where the widened copy has the sequence's tiles
  const KvTiles wide = visible_tiles(a, first, q.len - 1, kN);
  auto place = [&](int j) {  // the box's row in the tensor map; -1: nothing to fetch
    const int tile = tiles.at(i0 + j), key = kN * tile + box_row, last = key + a.box_rows - 1;
    if (lane >= kN / a.box_rows * panels || key > p_hi ||
        (last <= p_lo - a.window && key >= a.sinks))
      return -1;
    if (a.n_pad > 0) return (pair - a.pair0) * a.n_pad + kN * wide.index(tile) + box_row;
    const int page = page_of(key);
    if (page < 0) return -1;
    return (page * a.b.h_kv + head) * a.b.page_tokens + key % a.b.page_tokens;
  };
  int next_box = warp == kTmaWarp && nt > 0 ? place(0) : -1;
  auto load = [&](int j) {
    const int at = next_box;
    if (j + 1 < nt) next_box = place(j + 1);
    const uint32_t n = __popc(__ballot_sync(0xffffffffu, at >= 0));
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const int x = 2 * j + side, st = x % kStages;
      if (x >= kStages && !warp_wait(kv_empty(st), (x / kStages - 1) & 1)) return false;
      if (lane == 0) mbar_expect(kv_full(st), n * a.box_rows * 128);
      __syncwarp();
      if (at >= 0)
        tma_box(ring + st * kTile + box_panel * kPanel + box_row * 128, side ? &map_v : &map_k,
                64 * box_panel, at, kv_full(st));
    }
    return true;
  };
  // the first tiles are on their way while the block sets up
  if (warp == kTmaWarp) {
    __syncwarp();
    for (int j = 0; j < kStages / 2 && j < nt; ++j) load(j);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // tensor memory: S (of one tile at a time), P_0, P_1, O_0, O_1
  const uint32_t t_s = tmem;
  auto t_p = [&](int i) { return tmem + kN + kN / 2 * i; };
  auto t_o = [&](int i) { return tmem + 2 * kN + DP * i; };
  // whether some row of the unit sees the key
  auto seen_by_some = [&](int key) {
    return key <= p_hi && (key > p_lo - a.window || key < a.sinks);
  };

  // (nt = 0: no row sees anything; the softmax warps write zeros)
  if (warp < kSoftWarps) {
    // ----------------------------------------------------------- softmax --
    regs_up<kSoftRegs>();
    const int m = warp / 4, r = tid % kM;  // tile and row
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int c = c0 + m * kM + r;
    const int pos = first + cols.row + cols.row_of(min(c, c1 - 1) - c0);
    const float cs = fmaxf(fabsf(a.qscale), 1e-37f);  // (0 would make NaN of a masked score)
    float ref = -INFINITY, l = 0.0f;
    bool live = true;
    if (nt > 0 && m < n_m) {
      const uint32_t flip = a.qscale < 0.0f ? 0x80008000u : 0u;  // makes the scale positive
      auto store_q = [&](int i, uint4 x) {
        const int rr = 32 * (warp & 3) + (32 * i + lane) / kChunks, ch = lane % kChunks;
        x.x ^= flip;
        x.y ^= flip;
        x.z ^= flip;
        x.w ^= flip;
        if (c0 + m * kM + rr >= c1) x = make_uint4(0, 0, 0, 0);
        st_shared16(sq + m * kTile + (ch / 8) * kPanel + rr * 128 + (((ch % 8) ^ (rr & 7)) << 4), x);
      };
#pragma unroll
      for (int i = 0; i < kEarly; ++i) store_q(i, xq[i]);
      if constexpr (kChunks > kEarly) {
#pragma unroll
        for (int i = 0; i < kChunks - kEarly; ++i) xq[i] = load_q(kEarly + i);
#pragma unroll
        for (int i = 0; i < kChunks - kEarly; ++i) store_q(kEarly + i, xq[i]);
      }
      proxy_fence();
      mbar_arrive(q_full(m));
      const int t_lo = first + (c0 + m * kM) / a.G;
      const int t_hi = first + (min(c0 + m * kM + kM, c1) - 1) / a.G;
      // lane b: the page table's entry for block b of 16 keys of tile j.  It is looked at
      // a tile later, so that nothing waits for it.
      auto entry_of = [&](int j) {
        const int key = kN * tiles.at(i0 + j) + kKvBlock * (lane & 7);
        const int at = (int)((unsigned)key / (unsigned)a.b.page_tokens);
        return key < q.len && at < a.b.table_width
                   ? __ldg(a.b.page_table + (int64_t)s * a.b.table_width + at)
                   : -1;
      };
      int entry = entry_of(0);
      for (int j = 0; j < nt; ++j) {
        const int key0 = kN * tiles.at(i0 + j);
        const uint32_t here =
            __ballot_sync(0xffffffffu, entry >= 0 && entry < a.b.num_pages) & 0xffu;
        if (j + 1 < nt) entry = entry_of(j + 1);
        const bool whole = here == 0xffu && sees_all(a, t_lo, t_hi, key0, kN);
        // the keys that this row sees, of 32 from key0 + 32 i
        auto seen = [&](int i) {
          const int k0 = key0 + 32 * i;
          uint32_t b = low_bits(pos - k0 + 1) &
                       (~low_bits(pos - a.window + 1 - k0) | low_bits(a.sinks - k0));
          if (!(here >> (2 * i) & 1)) b &= 0xffff0000u;
          if (!(here >> (2 * i + 1) & 1)) b &= 0x0000ffffu;
          return b;
        };
        if (!warp_wait(s_full(m), j & 1)) {
          live = false;
          break;
        }
        tc_fence_after();
        uint32_t v[kN / 32][32];
#pragma unroll
        for (int i = 0; i < kN / 32; ++i) tc_ld32(t_s + lanes + 32 * i, v[i]);
        tc_wait_ld();
        tc_fence_before();
        mbar_arrive(s_read(m));
        if (!whole) {
#pragma unroll
          for (int i = 0; i < kN / 32; ++i) {
            const uint32_t see = seen(i);
#pragma unroll
            for (int e = 0; e < 32; ++e)
              if (!(see >> e & 1)) v[i][e] = 0xff800000u;  // -inf
          }
        }
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          top[i] = __uint_as_float(v[i][0]);
#pragma unroll
          for (int e = 1; e < 31; e += 2)
            top[i] = fmaxf(top[i], fmaxf(__uint_as_float(v[i][e]), __uint_as_float(v[i][e + 1])));
          top[i] = fmaxf(top[i], __uint_as_float(v[i][31]));
        }
        float mx = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        mx = mx == -INFINITY ? mx : mx * cs;
        // the product with the tile before is complete: O and P may change
        if (j > 0 && !warp_wait(o_done(m), (j - 1) & 1)) {
          live = false;
          break;
        }
        tc_fence_after();
        const bool grow = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float next = grow ? mx : ref;
          const float f = ref == next ? 1.0f : exp2f(ref - next);
          l *= f;
          ref = next;
          if (j > 0) {  // (tile 0 overwrites O)
#pragma unroll
            for (int i = 0; i < DP / 16; ++i) {
              if (16 * i >= d) break;
              uint32_t o[16];
              tc_ld16(t_o(m) + lanes + 16 * i, o);
              tc_wait_ld();
#pragma unroll
              for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
              tc_st16(t_o(m) + lanes + 16 * i, o);
            }
          }
        }
        const float sub = ref == -INFINITY ? 0.0f : ref;
        const uint64_t cs2 = pack2(cs, cs), sub2 = pack2(-sub, -sub);
        uint64_t sum = 0ull, sum2 = 0ull;
#pragma unroll
        for (int i = 0; i < kN / 32; ++i) {
          uint32_t w[16];
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const uint32_t *x = &v[i][e];
            const float2 y = unpack2(fma2(pack2(__uint_as_float(x[0]), __uint_as_float(x[1])), cs2, sub2));
            const float p0 = ex2(y.x), p1 = ex2(y.y);
            if (e & 2)
              sum2 = add2(sum2, pack2(p0, p1));
            else
              sum = add2(sum, pack2(p0, p1));
            w[e / 2] = bf16x2(p0, p1);
          }
          tc_st16(t_p(m) + lanes + 16 * i, w);
          if (i % 2) {  // half of the row: its product can start
            tc_wait_st();
            tc_fence_before();
            mbar_arrive(p_full(m, i / 2));
          }
        }
        const float2 part = unpack2(add2(sum, sum2));
        l += part.x + part.y;
      }
      if (live) live = warp_wait(o_done(m), (nt - 1) & 1);
      if (!live) s_fault = 1;
      tc_fence_after();
    }
    // ---------------------------------------------------------- epilogue --
    if (m < n_m && live) {
      const int row = q.row0 + cols.row + cols.row_of(c - c0), h = head * a.G + cols.head_of(c - c0);
      const int64_t rh = (int64_t)row * a.h_q + h;
      const bool mine = c < c1;
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
      const int64_t part = part_at(a, u.unit, split) + (c - c0);
#pragma unroll
      for (int i = 0; i < DP / 32; ++i) {
        if (32 * i >= d) break;
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
        if (nt > 0) {
          tc_ld32(t_o(m) + lanes + 32 * i, v);
          tc_wait_ld();
        }
        if (u.splits == 1) {
          // by way of the tile's rows of Q, which no product reads any more: a row's
          // 64 bytes here, whole rows to the output below
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              w[z] = bf16x2(l == 0.0f ? 0.0f : __uint_as_float(v[e + 2 * z]) * inv,
                            l == 0.0f ? 0.0f : __uint_as_float(v[e + 2 * z + 1]) * inv);
            const int ch = 4 * i + e / 8;
            st_shared16(sq + m * kTile + (ch / 8) * kPanel + r * 128 + (((ch % 8) ^ (r & 7)) << 4),
                        make_uint4(w[0], w[1], w[2], w[3]));
          }
        } else if (mine) {
          float *out = a.part_o + part * d + 32 * i;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4 *>(out + e) =
                l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                          : make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                        __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        }
      }
      if (u.splits == 1) {
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int rr = 32 * (warp & 3) + (32 * i + lane) / kChunks, ch = lane % kChunks;
          const int x0 = m * kM + rr;
          if (c0 + x0 < c1 && 8 * ch < d) {
            const uint4 x = ld_shared16(sq + m * kTile + (ch / 8) * kPanel + rr * 128 +
                                        (((ch % 8) ^ (rr & 7)) << 4));
            const int64_t at = (int64_t)(q.row0 + cols.row + cols.row_of(x0)) * a.h_q +
                               head * a.G + cols.head_of(x0);
            if (a.out_wide) {
              *reinterpret_cast<uint4 *>(static_cast<uint16_t *>(a.out) + at * d + 8 * ch) = x;
            } else {
              const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
              for (int z = 0; z < 8; ++z)
                static_cast<uint16_t *>(a.out)[at * d + 8 * ch + z] = (uint16_t)(w[z / 2] >> (16 * (z & 1)));
            }
          }
        }
      }
      if (mine) {
        if (u.splits == 1) {
          if (a.lse) a.lse[rh] = lse_of(ref, l, 0.0f);
        } else {
          a.part_ml[part] = make_float2(ref, l);
        }
      }
    }
  } else {
    regs_down<kOtherRegs>();
    if (warp == kTmaWarp && nt > 0) {
      // ----------------------------------------------------------- loads --
      bool live = true;
      for (int j = kStages / 2; j < nt && live; ++j) live = load(j);
      if (!live) s_fault = 1;
    } else if (warp >= kEdgeWarp0 && nt > 0) {
      // ------------------------------------------------------- V's edges --
      const int t = tid - 32 * kEdgeWarp0;
      for (int j = 0; j < nt; ++j) {
        const int x = 2 * j + 1, st = x % kStages;
        const int key0 = kN * tiles.at(i0 + j);
        // a tile that every row sees whole needs nothing, if its pages are there
        const uint32_t there =
            __ballot_sync(0xffffffffu, page_of(key0 + kKvBlock * (lane & 7)) >= 0);
        const bool edge = (there & 0xffu) != 0xffu || !sees_all(a, p_lo, p_hi, key0, kN);
        if (!warp_wait(kv_full(st), (x / kStages) & 1)) {
          s_fault = 1;
          break;
        }
        if (edge) {
          uint32_t bad = 0;
          for (int r = t; r < kN; r += kEdgeThreads) {
            const int key = key0 + r;
            const bool seen = seen_by_some(key) && (there >> (r / kKvBlock) & 1);
            if (seen && sees_all(a, p_lo, p_hi, key, 1)) continue;
            const uint32_t at = ring + st * kTile + r * 128;
#pragma unroll
            for (int i = 0; i < kChunks; ++i) {  // (each lane starts elsewhere: other banks)
              if (64 * (i / 8) >= d) break;  // a panel that is not there
              const uint32_t w = at + (i / 8) * kPanel + 16 * ((i + lane) % 8);
              if (!seen) {
                st_shared16(w, make_uint4(0, 0, 0, 0));
              } else {
                const uint4 v = ld_shared16(w);
                bad |= nonfinite2(v.x) | nonfinite2(v.y) | nonfinite2(v.z) | nonfinite2(v.w);
              }
            }
          }
          if (bad) *taint = kMarkAgain;
          proxy_fence();
        }
        mbar_arrive(v_ready(st));
      }
    } else if (warp == kMmaWarp && nt > 0) {
      // ------------------------------------------------------------ MMAs --
      const uint32_t id_s = idesc(kN, false), id_o = idesc(d, true);
      const bool leader = tc_elect_one();
      bool live = mbar_wait(q_full(0), 0);
      if (n_m == 2 && live) live = mbar_wait(q_full(1), 0);
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (live) live = mbar_wait(bar, parity);
        return live;
      };
      auto mul_s = [&](int m, int stage) {
        if (!leader) return;
#pragma unroll
        for (int k = 0; k < DP / 16; ++k) {
          if (16 * k >= d) break;
          const uint32_t off = (k / 4) * kPanel + (k % 4) * 32;
          mma_ss(t_s, smem_desc(sq + m * kTile + off, 16), smem_desc(ring + stage * kTile + off, 16),
                 id_s, k > 0);
        }
      };
      auto mul_o = [&](int m, int half, int stage, bool acc) {
        if (!leader) return;
#pragma unroll
        for (int k = 4 * half; k < 4 * half + 4; ++k)
          mma_ts(t_o(m), t_p(m) + 8 * k, smem_desc(ring + stage * kTile + k * 2048, kPanel), id_o,
                 acc || k > 0);
      };
      auto commit = [&](uint32_t bar) {
        if (leader) tc_commit(bar);
      };
      // P_m V of tile j, half by half
      auto add_o = [&](int m, int j) {
        const int st = (2 * j + 1) % kStages;
        for (int half = 0; half < 2; ++half) {
          if (!wait(p_full(m, half), j & 1)) return;
          tc_fence_after();
          mul_o(m, half, st, j > 0 || half > 0);
        }
        commit(o_done(m));
      };
      // The next tile's S_0 comes before this one's P_0 V, so that a row tile's next
      // scores wait for its softmax and not the other way round.  There is room for
      // one S: each is multiplied once the softmax has read the one before.
      if (wait(kv_full(0), 0)) {
        tc_fence_after();
        mul_s(0, 0);
        commit(s_full(0));
        if (n_m == 2 && wait(s_read(0), 0)) {
          tc_fence_after();
          mul_s(1, 0);
          commit(s_full(1));
        }
        commit(kv_empty(0));
      }
      for (int j = 0; j < nt && live; ++j) {
        const int st = (2 * j + 2) % kStages;  // K of the next tile
        const bool more = j + 1 < nt;
        if (more) {
          if (!wait(kv_full(st), ((2 * j + 2) / kStages) & 1)) break;
          if (!wait(s_read(n_m - 1), j & 1)) break;
          tc_fence_after();
          mul_s(0, st);
          commit(s_full(0));
          if (n_m == 1) commit(kv_empty(st));
        }
        if (!wait(v_ready((2 * j + 1) % kStages), ((2 * j + 1) / kStages) & 1)) break;
        add_o(0, j);
        if (n_m == 2) {
          if (more) {
            if (!wait(s_read(0), (j + 1) & 1)) break;
            tc_fence_after();
            mul_s(1, st);
            commit(s_full(1));
            commit(kv_empty(st));
          }
          add_o(1, j);
        }
        commit(kv_empty((2 * j + 1) % kStages));
      }
      if (!live) s_fault = 1;
    }
  }

  // The ring's last commits are waited for: then every MMA is complete, and no
  // arrival is pending when the barriers go away.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && nt > 0) {
    for (int i = 0; i < kStages && !s_fault; ++i) {
      const int items = (2 * nt - i + kStages - 1) / kStages;
      if (items > 0 && !mbar_wait(kv_empty(i), (items - 1) & 1)) s_fault = 1;
    }
  }
  __syncthreads();
  if (tid == 0 && s_fault) *taint |= kMarkLate;
  tc_fence_after();
  // Given up halfway: what was issued, products and copies, ends first.  A wait gives up
  // after 2^31 clocks, in which whoever feeds it has stopped too, so the last copy is a
  // second old by now; 2^24 clocks more are a hundred times what one takes.  (Waits on
  // the copies' own barriers here make the compiler spill: 0.8% on every call.)
  if (warp == kMmaWarp && s_fault) {
    const long long t0 = clock64();
    while (clock64() - t0 < (1ll << 24)) {
    }
  }
  __syncwarp();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

// E4M3: the keys that some row sees, K and V, as bf16 in [pair - pair0][n_pad][d].  A
// block per 128 keys of a pair; bound by bytes (1 read, 2 written an element).
constexpr int kWidenThreads = 256;

__global__ void __launch_bounds__(kWidenThreads) widen_kernel(const __grid_constant__ KvAttnParams a,
                                                              uint16_t *wide_k, uint16_t *wide_v) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int d = a.d, pieces = d / 16;
  const int per = a.n_pad / kN;
  const int pair = blockIdx.x / per, tile = blockIdx.x % per;
  const int head = (a.pair0 + pair) % a.b.h_kv, s = (a.pair0 + pair) / a.b.h_kv;
  const KvSeq q = kv_seq(a.b, s);
  if (q.rows == 0 || !owns(a, q)) return;
  const KvTiles tiles = visible_tiles(a, q.len - q.rows, q.len - 1, kN);
  if (tile >= tiles.count) return;
  const int key0 = tiles.at(tile) * kN;
  for (int i = threadIdx.x; i < kN * pieces; i += kWidenThreads) {
    const int r = (int)((unsigned)i / (unsigned)pieces), piece = i - r * pieces, key = key0 + r;
    if (key >= q.len) return;
    const int at = (int)((unsigned)key / (unsigned)a.b.page_tokens);
    const int page = kv_page(a.b, s, at);
    if (page < 0) continue;
    const int slot = key - at * a.b.page_tokens;
    const int64_t h = (int64_t)page * a.b.h_kv + head;
    const int64_t src = (h * a.b.page_tokens + slot) * d + piece * 16;
    const int64_t sc = h * (a.b.page_tokens / kKvBlock) + slot / kKvBlock;
    const int64_t dst = ((int64_t)pair * a.n_pad + tile * kN + r) * d + piece * 16;
#pragma unroll
    for (int side = 0; side < 2; ++side) {
      const uint4 v = __ldg(reinterpret_cast<const uint4 *>(
          static_cast<const uint8_t *>(side ? a.cv : a.ck) + src));
      const float f = exp2i(kv_scale_exp(__ldg((side ? a.v_scale : a.k_scale) + sc)));
      const uint2 w0 = widen4(v.x, f), w1 = widen4(v.y, f), w2 = widen4(v.z, f), w3 = widen4(v.w, f);
      uint4 *out = reinterpret_cast<uint4 *>((side ? wide_v : wide_k) + dst);
      out[0] = make_uint4(w0.x, w0.y, w1.x, w1.y);
      out[1] = make_uint4(w2.x, w2.y, w3.x, w3.y);
    }
  }
}

// ------------------------------------------------------------------ host --

// A [rows][d] bf16 matrix in boxes of box_rows x 64, 128-byte swizzle.
cudaError_t make_map(CUtensorMap *map, const void *ptr, int64_t rows, int d, int box_rows) {
  using Encode = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
  static const Encode encode = []() -> Encode {
    void *fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &fn, cudaEnableDefault, &found) !=
            cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      return nullptr;
    return reinterpret_cast<Encode>(fn);
  }();
  if (!encode) return cudaErrorNotSupported;
  const cuuint64_t dims[2] = {(cuuint64_t)d, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)d * 2};
  const cuuint32_t box[2] = {64, (cuuint32_t)box_rows}, step[2] = {1, 1};
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void *>(ptr), dims,
                            strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

template <int DP, bool FULL>
cudaError_t launch(KvAttnParams a, bool f8, cudaStream_t s) {
  constexpr int smem = Size<DP>::kSmem;
  cudaError_t e = cudaFuncSetAttribute(kv_prompt_kernel<DP, FULL>,
                                       cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  CUtensorMap map_k, map_v;
  const void *k = f8 ? a.wide : a.ck;
  const void *v = f8 ? a.wide + (size_t)a.pairs * a.n_pad * a.d : a.cv;
  const int64_t rows = f8 ? (int64_t)a.pairs * a.n_pad
                          : (int64_t)a.b.num_pages * a.b.h_kv * a.b.page_tokens;
  e = make_map(&map_k, k, rows, a.d, a.box_rows);
  if (e == cudaSuccess) e = make_map(&map_v, v, rows, a.d, a.box_rows);
  const int all = a.b.num_seqs * a.b.h_kv, group = a.pairs;
  for (a.pair0 = 0; a.pair0 < all && e == cudaSuccess; a.pair0 += group) {
    a.pairs = all - a.pair0 < group ? all - a.pair0 : group;
    if (f8)
      e = launch_dependent(widen_kernel, dim3((unsigned)(a.pairs * (a.n_pad / kN))),
                           dim3(kWidenThreads), 0, s, a, const_cast<uint16_t *>(a.wide),
                           static_cast<uint16_t *>(const_cast<void *>(v)));
    if (e == cudaSuccess)
      e = launch_dependent(kv_prompt_kernel<DP, FULL>,
                           dim3((unsigned)(unit_blocks(a) + (a.pair0 == 0 ? a.report : 0))),
                           dim3(kThreads), smem, s, a, map_k, map_v);
  }
  return e;
}

}  // namespace

cudaError_t launch_kv_prompt(const KvAttnParams &a, bool f8, cudaStream_t s) {
  switch (a.d) {
    case 64: return launch<64, true>(a, f8, s);
    case 128: return launch<128, true>(a, f8, s);
    case 256: return launch<256, true>(a, f8, s);
    default: return a.d < 128 ? launch<128, false>(a, f8, s) : launch<256, false>(a, f8, s);
  }
}

}  // namespace fathom
