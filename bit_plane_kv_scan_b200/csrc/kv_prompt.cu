// fathom_kv_attention, many rows (a prompt or a chunk of one): softmax(Q K^T) V
// over the paged cache on the tcgen05 tensor cores.
//
// A unit is 256 (token, head) pairs of one sequence and KV head, as two tiles
// of 128 rows: the G heads that share a KV head share its keys.  One
// thread block per SM takes a unit through its keys, 128 at a time:
//   S_i = Q_i K^T      tcgen05.mma, Q and K in shared memory, S_i in tensor memory
//   P_i = 2^(c S_i - m_i)   one thread a row, rounded to bf16, over S_i's columns
//   O_i += P_i V       tcgen05.mma, P_i from tensor memory, O_i stays there
// with c = scale * log2 e.  The two tiles alternate, so that the tensor cores
// multiply one while the other's softmax is worked out.  A row's reference m
// moves only when its maximum has grown by more than 2^8 (weights up to 2^8 are as
// exact in bf16 and fp32 as those up to 1); then the row of O is rescaled.
//
// Bound by the tensor cores and, next to them, by the exponentials: for 256 rows
// and 128 keys 4 products of 128 x 128 x 128 take 2048 clocks of the tensor pipe,
// and 32768 exponentials 2048 clocks of the special-function units.
//
// Warps: 0-3 and 4-7 the softmax of the two tiles; 8-11 load Q, K and V into
// shared memory, by cp.async (bf16) or through registers (e4m3, which becomes
// bf16 exactly, its power-of-two scale included); 12 issues the MMAs (13-15 are
// there to give up their registers).  K and V go
// through a ring of 4 buffers in 128-byte swizzled rows; pages may be as small as
// 16 tokens.  Keys that no row of the unit sees, and those on bad pages, arrive as
// zeros.
//
// Masks are applied to S, where a tile of keys is not seen whole.  A masked key's
// weight is an exact zero, but 0 * NaN is not: where a value that some row of the
// unit does not see is not finite, the loading warps mark the unit, and the
// few-rows kernel (which masks V row by row) does it again afterwards.
#include <cuda_fp8.h>

#include "kv_attention.cuh"
#include "tc_common.cuh"

namespace fathom {

namespace {

constexpr int kSoftWarps = 8;  // 4 for each tile
constexpr int kLoadWarp0 = kSoftWarps, kLoadWarps = 4;
constexpr int kMmaWarp = kLoadWarp0 + kLoadWarps;
constexpr int kThreads = 32 * (kMmaWarp + 4);  // 512: the MMA warp's group has no other work
// Registers: 512 threads are launched with 128 each, 65536 in all.  The softmax
// keeps a row of 128 scores in registers; the other groups give theirs up:
// 256 * 192 + 128 * 88 + 128 * 40 = 65536.
constexpr int kSoftRegs = 192, kLoadRegs = 88, kMmaRegs = 40;
static_assert(kSoftRegs * 256 + (kLoadRegs + kMmaRegs) * 128 <= 65536, "registers of the block");
constexpr int kLoadThreads = 32 * kLoadWarps;
constexpr int kM = 128;                  // rows of a tile
constexpr int kN = kPromptTile;          // keys of a tile
constexpr int kStages = 4;               // ring of K and V tiles
constexpr int kPanel = kM * 128;         // bytes of 64 dimensions of 128 rows
constexpr uint32_t kTmemCols = 512;
constexpr float kSlack = 8.0f;           // a row's reference lags its maximum by less

template <int D>
constexpr int tile_bytes() { return D / 64 * kPanel; }

// Shared memory: Q's two tiles, then the ring; 1024-byte aligned (the swizzle's
// period).  More than half an SM's, so that two blocks never share an SM and its
// tensor memory.
template <int D>
constexpr int smem_bytes() {
  const int b = (2 + kStages) * tile_bytes<D>() + 1024;
  return b < 120 * 1024 ? 120 * 1024 : b;
}

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

// The loading warps' part: pages of one tile of keys, found by the lanes of
// each warp (lane b: the tile's 16-token block b).
struct TilePages {
  int page, slot, key0;
  bool whole;  // every row of the unit sees every key
};

template <int D, bool F8>
__global__ void __launch_bounds__(kThreads, 1) kv_prompt_kernel(KvAttnParams a) {
  constexpr int kTile = tile_bytes<D>();
  constexpr int kSteps = D / 16;
  extern __shared__ unsigned char smem_raw[];
  __shared__ __align__(8) uint64_t s_bar[2 * kStages + 1 + 4 + 1];
  __shared__ uint32_t s_tmem;
  __shared__ int s_fault;
  if (blockIdx.x == gridDim.x - 1) {
    grid_dependency_wait();
    allow_dependent_launch();
    write_status(a);
    return;
  }
  grid_dependency_wait();
  allow_dependent_launch();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // later rows see more keys: their units come first
  int x = blockIdx.x;
  const int split = x % a.splits;
  x /= a.splits;
  const int hs = x % (a.b.h_kv * a.b.num_seqs);
  const int rb = a.col_tiles - 1 - x / (a.b.h_kv * a.b.num_seqs);
  const int head = hs % a.b.h_kv, s = hs / a.b.h_kv;
  int *taint = a.taint + ((int64_t)(s * a.b.h_kv + head) * a.col_tiles + rb) * a.splits + split;
  if (tid == 0) *taint = 0;
  const KvSeq q = kv_seq(a.b, s);
  const int c0 = rb * kPromptCols, c1 = min(c0 + kPromptCols, q.rows * a.G);
  if (c0 >= c1) return;
  const int first = q.len - q.rows;  // position of the sequence's first row
  const int p_lo = first + c0 / a.G, p_hi = first + (c1 - 1) / a.G;
  const KvTiles tiles = visible_tiles(a, p_lo, p_hi, kN);
  const int i0 = split * a.tiles_per_split;
  const int nt = min(tiles.count - i0, a.tiles_per_split);  // tiles of this block
  if (split > 0 && nt <= 0) return;
  const int n_m = c1 - c0 > kM ? 2 : 1;  // tiles of rows

  const uint32_t base = (tc_smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sq = base, ring = base + 2 * kTile;
  const uint32_t bar0 = tc_smem_u32(s_bar);
  auto kv_full = [&](int i) { return bar0 + 8 * i; };
  auto kv_empty = [&](int i) { return bar0 + 8 * (kStages + i); };
  const uint32_t q_full = bar0 + 8 * (2 * kStages);
  auto s_full = [&](int i) { return bar0 + 8 * (2 * kStages + 1 + i); };
  auto p_full = [&](int i) { return bar0 + 8 * (2 * kStages + 3 + i); };
  const uint32_t o_full = bar0 + 8 * (2 * kStages + 5);

  if (warp == kMmaWarp) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;\n" ::"r"(
                     tc_smem_u32(&s_tmem)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;\n" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      mbar_init(kv_full(i), kLoadThreads);
      mbar_init(kv_empty(i), 1);
    }
    mbar_init(q_full, kLoadThreads);
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full(i), 1);
      mbar_init(p_full(i), kM);
    }
    mbar_init(o_full, 1);
    asm volatile("fence.mbarrier_init.release.cluster;\n" ::: "memory");
    s_fault = 0;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = s_tmem;
  // tensor memory: S_0, S_1 (P_i over their first half), O_0, O_1
  auto t_s = [&](int i) { return tmem + kN * i; };
  auto t_o = [&](int i) { return tmem + 2 * kN + D * i; };

  if (warp < kSoftWarps) {
    // ----------------------------------------------------------- softmax --
    regs_up<kSoftRegs>();
    const int m = warp / 4, r = tid % kM;  // tile and row
    const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
    const int c = c0 + m * kM + r;
    const int pos = first + min(c, c1 - 1) / a.G;
    const float cs = fmaxf(fabsf(a.qscale), 1e-37f);  // (0 would make NaN of a masked score)
    float ref = -INFINITY, l = 0.0f;
    bool live = true;
    if (nt > 0 && m < n_m) {
      const int t_lo = first + (c0 + m * kM) / a.G;
      const int t_hi = first + (min(c0 + m * kM + kM, c1) - 1) / a.G;
      // blocks of 16 keys that are there, of tile j
      auto blocks_of = [&](int j) {
        const int key = kN * tiles.at(i0 + j) + kKvBlock * (lane & 7);
        const bool ok = key < q.len &&
                        kv_page(a.b, s, (int)((unsigned)key / (unsigned)a.b.page_tokens)) >= 0;
        return __ballot_sync(0xffffffffu, ok) & 0xffu;
      };
      uint32_t blocks = blocks_of(0);
      for (int j = 0; j < nt; ++j) {
        const int key0 = kN * tiles.at(i0 + j);
        const uint32_t here = blocks;
        if (j + 1 < nt) blocks = blocks_of(j + 1);
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
        for (int i = 0; i < kN / 32; ++i) tc_ld32(t_s(m) + lanes + 32 * i, v[i]);
        tc_wait_ld();
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
        const bool grow = mx > ref + kSlack;
        if (__any_sync(0xffffffffu, grow)) {
          const float next = grow ? mx : ref;
          const float f = ref == next ? 1.0f : exp2f(ref - next);
          l *= f;
          ref = next;
          if (j > 0) {  // (tile 0 overwrites O)
#pragma unroll
            for (int i = 0; i < D / 16; ++i) {
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
          tc_st16(t_s(m) + lanes + 16 * i, w);
        }
        const float2 part = unpack2(add2(sum, sum2));
        l += part.x + part.y;
        tc_wait_st();
        tc_fence_before();
        mbar_arrive(p_full(m));
      }
      if (live) live = warp_wait(o_full, 0);
      if (!live) s_fault = 1;
      tc_fence_after();
    }
    // ---------------------------------------------------------- epilogue --
    if (m < n_m && live) {
      const int row = q.row0 + c / a.G, h = head * a.G + c % a.G;
      const int64_t rh = (int64_t)row * a.h_q + h;
      const bool mine = c < c1;
      const float inv = l > 0.0f ? 1.0f / l : (l == 0.0f ? 0.0f : l);
      const int64_t part = (int64_t)split * a.b.num_rows * a.h_q + rh;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        uint32_t v[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = 0u;
        if (nt > 0) {
          tc_ld32(t_o(m) + lanes + 32 * i, v);
          tc_wait_ld();
        }
        if (!mine) continue;
        if (a.splits == 1) {
          __nv_bfloat16 *out = static_cast<__nv_bfloat16 *>(a.out) + rh * D + 32 * i;
#pragma unroll
          for (int e = 0; e < 32; e += 2) {
            const float x0 = l == 0.0f ? 0.0f : __uint_as_float(v[e]) * inv;
            const float x1 = l == 0.0f ? 0.0f : __uint_as_float(v[e + 1]) * inv;
            reinterpret_cast<__nv_bfloat162 *>(out)[e / 2] = __floats2bfloat162_rn(x0, x1);
          }
        } else {
          float *out = a.part_o + part * D + 32 * i;
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4 *>(out + e) =
                l == 0.0f ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                          : make_float4(__uint_as_float(v[e]), __uint_as_float(v[e + 1]),
                                        __uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        }
      }
      if (mine) {
        if (a.splits == 1) {
          if (a.lse) a.lse[rh] = lse_of(ref, l, 0.0f);
        } else {
          a.part_ml[part] = make_float2(ref, l);
        }
      }
    }
  } else if (warp < kMmaWarp) {
    // ------------------------------------------------------------- loads --
    // (nt = 0: no row sees anything; the softmax warps write zeros)
    regs_down<kLoadRegs>();
    if (nt > 0) {
    const int t = tid - 32 * kLoadWarp0;
    {  // Q: rows c0 .. c1 - 1, the rest zeros; its sign makes c >= 0
      constexpr int kChunks = D / 8;  // 16-byte pieces of a row
      const uint32_t flip = a.qscale < 0.0f ? 0x80008000u : 0u;
      const uint16_t *qp = static_cast<const uint16_t *>(a.q);
      const bool wide = ((uintptr_t)qp & 15) == 0 && a.q_stride % 8 == 0;
      for (int i = t; i < n_m * kM * kChunks; i += kLoadThreads) {
        const int r = i / kChunks, ch = i % kChunks, c = c0 + r;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (c < c1) {
          const uint16_t *src = qp + (int64_t)(q.row0 + c / a.G) * a.q_stride +
                                (int64_t)(head * a.G + c % a.G) * D + ch * 8;
          if (wide) {
            v = *reinterpret_cast<const uint4 *>(src);
          } else {
            v.x = src[0] | ((uint32_t)src[1] << 16);
            v.y = src[2] | ((uint32_t)src[3] << 16);
            v.z = src[4] | ((uint32_t)src[5] << 16);
            v.w = src[6] | ((uint32_t)src[7] << 16);
          }
          v.x ^= flip;
          v.y ^= flip;
          v.z ^= flip;
          v.w ^= flip;
        }
        const int m = r / kM, rr = r % kM;
        st_shared16(sq + m * kTile + (ch / 8) * kPanel + rr * 128 + (((ch % 8) ^ (rr & 7)) << 4), v);
      }
      proxy_fence();
      mbar_arrive(q_full);
    }
    constexpr int kRow = F8 ? D : 2 * D;            // bytes of a row in the cache
    constexpr int kPer = kRow / 16;                 // 16-byte pieces of a row
    constexpr int kRows = kLoadThreads / kPer;      // rows that the warps load at once
    constexpr int kIter = kN / kRows;               // pieces a thread loads of a tile
    const int piece = t % kPer, r0 = t / kPer;      // this thread's piece of rows r0 + kRows i
    auto pages_of = [&](int j) {
      TilePages p;
      p.key0 = kN * tiles.at(i0 + j);
      const int key = p.key0 + kKvBlock * (lane & 7);
      const int at = (int)((unsigned)key / (unsigned)a.b.page_tokens);
      p.page = key < q.len ? kv_page(a.b, s, at) : -1;
      p.slot = key - at * a.b.page_tokens;
      p.whole = sees_all(a, p_lo, p_hi, p.key0, kN);
      return p;
    };
    // the place of row r0 + kRows i of a tile; NULL where there is nothing, or
    // nothing that a row of the unit sees
    auto row_of = [&](const TilePages &p, const void *cache, int i) -> const uint8_t * {
      const int r = r0 + kRows * i;
      const int page = __shfl_sync(0xffffffffu, p.page, r / kKvBlock);
      const int slot = __shfl_sync(0xffffffffu, p.slot, r / kKvBlock);
      const int key = p.key0 + r;
      if (page < 0 || key > p_hi || (key <= p_lo - a.window && key >= a.sinks)) return nullptr;
      return static_cast<const uint8_t *>(cache) +
             (((int64_t)page * a.b.h_kv + head) * a.b.page_tokens + slot + r % kKvBlock) * kRow +
             piece * 16;
    };
    bool live = true;
    // waits until the ring's buffer of item x is free (every second item is a V)
    auto claim = [&](int x) {
      if (x >= kStages && !warp_wait(kv_empty(x % kStages), (x / kStages - 1) & 1)) {
        live = false;
        s_fault = 1;
      }
      return live;
    };
    if constexpr (!F8) {
      // this thread's piece of row r0 + kRows i sits kRows * 128 bytes after the
      // one before (kRows is a multiple of 8, so the swizzle is the same)
      static_assert(kRows % 8 == 0, "a thread's rows share a swizzle phase");
      const uint32_t my = (piece / 8) * kPanel + r0 * 128 + (((piece % 8) ^ (r0 & 7)) << 4);
      bool pending_check = false;
      // an item whose copies have landed is checked (V) and handed over
      auto finish = [&](int x, bool check) {
        proxy_fence();
        if (check) {
          uint32_t bad = 0;
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            const uint4 v = ld_shared16(ring + (x % kStages) * kTile + my + i * kRows * 128);
            bad |= nonfinite2(v.x) | nonfinite2(v.y) | nonfinite2(v.z) | nonfinite2(v.w);
          }
          if (bad) *taint = 1;
        }
        mbar_arrive(kv_full(x % kStages));
      };
      TilePages p = pages_of(0);
      for (int j = 0; j < nt && live; ++j) {
        const TilePages cur = p;
        if (j + 1 < nt) p = pages_of(j + 1);
#pragma unroll
        for (int side = 0; side < 2; ++side) {
          const int x = 2 * j + side;
          if (!claim(x)) break;
          const uint32_t dst = ring + (x % kStages) * kTile + my;
#pragma unroll
          for (int i = 0; i < kIter; ++i) {
            const uint8_t *src = row_of(cur, side ? a.cv : a.ck, i);
            tc_cp_async16(dst + i * kRows * 128, src ? src : static_cast<const uint8_t *>(a.ck),
                          src ? 16u : 0u);
          }
          tc_cp_async_commit();
          if (x > 0) {
            tc_cp_async_wait<1>();
            finish(x - 1, pending_check);
          }
          pending_check = side && !cur.whole;
        }
      }
      tc_cp_async_wait<0>();
      if (live) finish(2 * nt - 1, pending_check);
    } else {
      // the piece's 16 codes become 32 bytes: dimensions 16 piece .. 16 piece + 15
      static_assert(kRows % 8 == 0 && (kRows <= kKvBlock || kRows % kKvBlock == 0), "");
      const uint32_t my = (piece / 4) * kPanel + r0 * 128;
      const uint32_t o0 = ((piece % 4 * 2) ^ (r0 & 7)) << 4, o1 = ((piece % 4 * 2 + 1) ^ (r0 & 7)) << 4;
      uint4 w[kIter], next[kIter];
      uint32_t exps = 0, exps_next = 0;
      auto fetch = [&](const TilePages &p, int side, uint4 (&v)[kIter], uint32_t &ex) {
        const uint8_t *sc = side ? a.v_scale : a.k_scale;
        ex = p.page < 0 ? 127u
                        : (uint32_t)(kv_scale_exp(__ldg(sc + ((int64_t)p.page * a.b.h_kv + head) *
                                                                (a.b.page_tokens / kKvBlock) +
                                                        p.slot / kKvBlock)) + 127);
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint8_t *src = row_of(p, side ? a.cv : a.ck, i);
          v[i] = make_uint4(0, 0, 0, 0);
          if (src) v[i] = __ldg(reinterpret_cast<const uint4 *>(src));
        }
      };
      TilePages cur = pages_of(0), p = cur;
      fetch(cur, 0, w, exps);
      for (int x = 0; x < 2 * nt && live; ++x) {
        const int side = x & 1;
        if (!side && x + 2 < 2 * nt) p = pages_of(x / 2 + 1);
        // the next item's loads are on their way while this one is widened
        if (x + 1 < 2 * nt) fetch(side ? p : cur, side ^ 1, next, exps_next);
        if (!claim(x)) break;
        const uint32_t dst = ring + (x % kStages) * kTile + my;
        uint32_t bad = 0;
#pragma unroll
        for (int i = 0; i < kIter; ++i) {
          const uint32_t ex = __shfl_sync(0xffffffffu, exps, (r0 + kRows * i) / kKvBlock);
          const float f = __int_as_float((int)ex << 23);
          const uint4 v = w[i];
          const uint2 b0 = widen4(v.x, f), b1 = widen4(v.y, f), b2 = widen4(v.z, f),
                      b3 = widen4(v.w, f);
          st_shared16(dst + i * kRows * 128 + o0, make_uint4(b0.x, b0.y, b1.x, b1.y));
          st_shared16(dst + i * kRows * 128 + o1, make_uint4(b2.x, b2.y, b3.x, b3.y));
          bad |= ((v.x & 0x7f7f7f7fu) + 0x01010101u) | ((v.y & 0x7f7f7f7fu) + 0x01010101u) |
                 ((v.z & 0x7f7f7f7fu) + 0x01010101u) | ((v.w & 0x7f7f7f7fu) + 0x01010101u);
        }
        if (side && !cur.whole && (bad & 0x80808080u)) *taint = 1;
        proxy_fence();
        mbar_arrive(kv_full(x % kStages));
        if (side) cur = p;
        exps = exps_next;
#pragma unroll
        for (int i = 0; i < kIter; ++i) w[i] = next[i];
      }
    }
    }
  } else {
    // -------------------------------------------------------------- MMAs --
    regs_down<kMmaRegs>();
    if (warp == kMmaWarp && nt > 0) {
    constexpr uint32_t kIdS = idesc(kN, false), kIdO = idesc(D, true);
    const bool leader = tc_elect_one();
    bool live = mbar_wait(q_full, 0);
    auto wait = [&](uint32_t bar, uint32_t parity) {
      if (live) live = mbar_wait(bar, parity);
      return live;
    };
    auto mul_s = [&](int m, int stage) {
      if (!leader) return;
#pragma unroll
      for (int k = 0; k < kSteps; ++k) {
        const uint32_t off = (k / 4) * kPanel + (k % 4) * 32;
        mma_ss(t_s(m), smem_desc(sq + m * kTile + off, 16), smem_desc(ring + stage * kTile + off, 16),
               kIdS, k > 0);
      }
    };
    auto mul_o = [&](int m, int stage, bool acc) {
      if (!leader) return;
#pragma unroll
      for (int k = 0; k < kN / 16; ++k)
        mma_ts(t_o(m), t_s(m) + 8 * k, smem_desc(ring + stage * kTile + k * 2048, kPanel), kIdO,
               acc || k > 0);
    };
    auto commit = [&](uint32_t bar) {
      if (leader) tc_commit(bar);
    };
    if (wait(kv_full(0), 0)) {
      tc_fence_after();
      for (int m = 0; m < n_m; ++m) {
        mul_s(m, 0);
        commit(s_full(m));
      }
      commit(kv_empty(0));
    }
    for (int j = 0; j < nt && live; ++j) {
      const int xv = 2 * j + 1, xk = 2 * j + 2;  // ring items: V of this tile, K of the next
      const bool more = j + 1 < nt;
      if (!wait(kv_full(xv % kStages), (xv / kStages) & 1)) break;
      if (more && !wait(kv_full(xk % kStages), (xk / kStages) & 1)) break;
      for (int m = 0; m < n_m; ++m) {
        if (!wait(p_full(m), j & 1)) break;
        tc_fence_after();
        mul_o(m, xv % kStages, j > 0);
        if (m == n_m - 1) commit(kv_empty(xv % kStages));
        if (more) {
          mul_s(m, xk % kStages);
          commit(s_full(m));
        }
      }
      if (more) commit(kv_empty(xk % kStages));
    }
    commit(o_full);
    if (!live) s_fault = 1;
    }
  }
  // Every MMA is complete once o_full has arrived; then the ring's last commits
  // are waited for, so that no arrival is pending when the barriers go away.
  tc_fence_before();
  __syncthreads();
  if (tid == 0 && nt > 0) {
    if (!mbar_wait(o_full, 0)) s_fault = 1;
    for (int i = 0; i < kStages && !s_fault; ++i) {
      const int items = (2 * nt - i + kStages - 1) / kStages;
      if (items > 0 && !mbar_wait(kv_empty(i), (items - 1) & 1)) s_fault = 1;
    }
  }
  __syncthreads();
  if (tid == 0 && s_fault) atomicAdd(&a.status->device_faults, 1u);
  tc_fence_after();
  if (warp == kMmaWarp)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;\n" ::"r"(tmem),
                 "r"(kTmemCols)
                 : "memory");
}

template <int D, bool F8>
cudaError_t launch(const KvAttnParams &a, cudaStream_t s) {
  constexpr int smem = smem_bytes<D>();
  const cudaError_t e = cudaFuncSetAttribute(kv_prompt_kernel<D, F8>,
                                             cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  const int64_t blocks = (int64_t)a.b.num_seqs * a.b.h_kv * a.col_tiles * a.splits + 1;
  return launch_dependent(kv_prompt_kernel<D, F8>, dim3((unsigned)blocks), dim3(kThreads), smem, s, a);
}

}  // namespace

cudaError_t launch_kv_prompt(const KvAttnParams &a, int d, bool f8, cudaStream_t s) {
  if (d == 128) return f8 ? launch<128, true>(a, s) : launch<128, false>(a, s);
  if (d == 64) return f8 ? launch<64, true>(a, s) : launch<64, false>(a, s);
  return cudaErrorInvalidValue;
}

}  // namespace fathom
