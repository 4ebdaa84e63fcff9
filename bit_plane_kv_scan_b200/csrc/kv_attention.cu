// fathom_kv_attention, few rows: the attention of one or a few new tokens of
// each sequence over its paged cache.
//
// Row at position p and query head h: s_j = scale <q, k_j> over the visible j,
// out = sum_j softmax(s)_j v_j, lse = log sum_j exp(s_j).  One pass over K and V
// with a running maximum and sum, 16 keys at a time.
//
// Bound by the bytes of K and V: with G heads a KV head, 4 G operations per
// element.  At 23 bytes a clock and SM that is more than the fp32 units have
// left beside unpacking, so both products run as m16n8k16 MMAs with keys (then
// dimensions) as the 16 rows and up to 8 (token, head) pairs as the 8 columns.
// (The tcgen05 MMAs need 64 rows or more of one operand in shared memory and an
// accumulator in tensor memory; with 8 columns of work their set-up costs more
// than the product.)  The order of the contracted index is free, so lanes read K
// and V from shared memory 16 bytes at a time, just as the rows lie there:
//   S^T = K q^T: lane (g, t) holds, of keys g and g + 8, the pieces t of
//     every four; q's fragments are permuted in the same way.
//   O^T = V^T P^T: lane (g, t) holds, of keys 2t, 2t + 1, 2t + 8, 2t + 9, the
//     pieces g of every eight; byte permutes pair two keys' elements.
//     P^T comes from S^T by movmatrix.
// Each warp takes every fourth 16-key tile of its block's run of tiles, through a
// ring of its own in shared memory that 16-byte asynchronous copies fill 1 or 2
// tiles ahead (no barrier between warps); its lanes look up the pages and scales
// of 32 tiles at once, a batch ahead.  The four warps' results meet in shared
// memory; where a sequence's tiles are split over several blocks, these join their
// results (maximum, sum, output) through the shared memory of a cluster, or, more
// than 16, through the workspace and a second kernel.
//
// E4M3: codes become fp16 exactly (the hardware's conversion).  q is scaled to
// fp16 by a power of two per row and head; a 16-key tile is one scale block, so
// K's scale multiplies S and V's multiplies that tile's product in fp32.
// Softmax weights are rounded to fp16 after a factor 2^15, which keeps weights
// down to 2^-29 of the largest to 11 bits (smaller ones are off by 2^-40 of it).
// bf16: weights are rounded to bf16, since a product's operands have one type and V
// does not fit in fp16's range; out is off by 0.0017 of its size with its own rounding
// to bf16, which alone makes it 0.0017 too.  Their sum is of the weights before that.
// fp32 queries: q and the weights are split into 2 (fp16) or 3 (bf16) terms and
// the products run once for each.
//
// With 32 query and 8 KV heads, d = 128: a row over 1M e4m3 tokens 377 to 402 us by
// board (82 to 87% of the copy rate; the board's power is the limit), 64 rows of
// windows of 4096 bf16 tokens 160 us (84%), a row over 4099 tokens 11 us.  e4m3 MMAs
// for S, q split into two terms, draw more power: 416 us against 391 in a loop.
//
// Masks: only tiles at the edge of what some column sees are masked.  There a V
// row that a token does not see is replaced by zeros for that token, so that
// what it holds (0 * NaN) cannot reach it.
#include <cooperative_groups.h>
#include <cuda_fp8.h>

#include "kv_attention.cuh"
#include "tc_common.cuh"

namespace cg = cooperative_groups;

namespace fathom {

namespace {

constexpr int kWarps = 4;
constexpr int kThreads = 32 * kWarps;
constexpr int kCols = 8;  // (token, head) pairs of a block: the MMA's n
constexpr int kMaxCluster = 16;

template <bool F8>
__device__ __forceinline__ void mma16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0,
                                      uint32_t b1) {
  if constexpr (F8)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
        "{%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t transpose8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;\n" : "=r"(d) : "r"(a));
  return d;
}

// Four e4m3 codes to four fp16 values, exactly.
__device__ __forceinline__ void e4m3_half4(uint32_t four, uint32_t &lo, uint32_t &hi) {
  asm("{\n\t.reg .b16 a, b;\n\t"
      "mov.b32 {a, b}, %2;\n\t"
      "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
      "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(four));
}

// 2^x, results below 2^-126 to 0 (hardware; off by 2^-22 of the value).
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;\n" : "=f"(y) : "f"(x));
  return y;
}

// Two floats as 16-bit terms (a in the low half); what is left goes back.
template <bool F8>
__device__ __forceinline__ uint32_t split16(float &a, float &b) {
  uint32_t r;
  if constexpr (F8) {
    const __half2 h = __floats2half2_rn(a, b);
    r = *reinterpret_cast<const uint32_t *>(&h);
    a -= __low2float(h);
    b -= __high2float(h);
  } else {
    const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
    r = *reinterpret_cast<const uint32_t *>(&h);
    a -= __low2float(h);
    b -= __high2float(h);
  }
  return r;
}

template <int BYTES>
__device__ __forceinline__ void load_bytes(uint32_t p, uint32_t *w) {
  if constexpr (BYTES == 16) {
    asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];\n"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(p));
  } else if constexpr (BYTES == 8) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];\n" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  } else {
    asm volatile("ld.shared.b32 %0, [%1];\n" : "=r"(w[0]) : "r"(p));
  }
}

// Tiles of a warp's ring.  A row of 256 bytes: 2, so that three blocks fit on an SM
// (64 windowed bf16 sessions: 162 us, against 172 with 3 tiles and two blocks).
constexpr int ring_depth(int row_bytes) { return row_bytes == 256 ? 2 : 3; }

template <int D, bool F8>
struct Shape {
  static constexpr int kRow = F8 ? D : 2 * D;                    // bytes of a row
  static constexpr int kKVec = (kRow / 4) % 16 == 0 ? 16 : 8;    // bytes of a K piece
  static constexpr int kVVec = (kRow / 8) % 16 == 0 ? 16 : ((kRow / 8) % 8 == 0 ? 8 : 4);
  static constexpr int kKWords = kRow / 16, kVWords = kRow / 32;  // words a lane has of a row
  static constexpr int kElt = F8 ? 1 : 2;
  // A warp's ring: 16 rows of K, 16 of V, each row 16 bytes longer than it is
  // (an odd number of 16-byte pieces: the pieces that 8 lanes read at once lie
  // in different banks).
  static constexpr int kPitch = kRow + 16, kSide = kKvBlock * kPitch, kStage = 2 * kSide;
  static constexpr int kDepth = ring_depth(kRow);
  static constexpr int kSmem = kWarps * kDepth * kStage;
  // The byte of piece j of the lane's part of a K row: two neighbouring pieces of
  // 128 bytes, so that four lanes' pieces 0 are every second one.
  __device__ static constexpr int k_byte(int j, int t) {
    return kRow % 128 == 0 ? (j >> 1) * 128 + (2 * t + (j & 1)) * 16 : (j * 4 + t) * kKVec;
  }
  __device__ static constexpr int v_byte(int j, int g) { return (j * 8 + g) * kVVec; }
  // the dimension of element e of the lane's part of a K or V row
  __device__ static int k_dim(int e, int t) {
    constexpr int v = kKVec / kElt;
    return k_byte(e / v, t) / kElt + e % v;
  }
  __device__ static int v_dim(int e, int g) {
    constexpr int v = kVVec / kElt;
    return v_byte(e / v, g) / kElt + e % v;
  }
};

// What the lanes of a warp have found out about 32 tiles, one each.
struct Found {
  int page, slot;  // page -1: nothing there
  int scales;      // E4M3: K's byte, V's byte
};

// O^T += V^T P^T for one 16-key tile; with PART only into this lane's columns
// that `mine` names.
template <int D, bool F8, int TERMS, bool PART>
__device__ __forceinline__ void add_pv(float (&o)[D / 16][4], const uint32_t (&v)[4][Shape<D, F8>::kVWords],
                                       float v_scale, const uint32_t (&p0)[TERMS],
                                       const uint32_t (&p1)[TERMS], const bool (&mine)[2]) {
#pragma unroll
  for (int i = 0; i < D / 16; ++i) {
    uint32_t f[4];
    if constexpr (F8) {
      const uint32_t sel = i & 1 ? 0x7362 : 0x5140;
      const uint32_t lo = __byte_perm(v[0][i / 2], v[1][i / 2], sel);
      const uint32_t hi = __byte_perm(v[2][i / 2], v[3][i / 2], sel);
      e4m3_half4(lo, f[0], f[1]);
      e4m3_half4(hi, f[2], f[3]);
    } else {
      f[0] = __byte_perm(v[0][i], v[1][i], 0x5410);
      f[1] = __byte_perm(v[0][i], v[1][i], 0x7632);
      f[2] = __byte_perm(v[2][i], v[3][i], 0x5410);
      f[3] = __byte_perm(v[2][i], v[3][i], 0x7632);
    }
    if constexpr (F8 || PART) {
      float c[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int u = 0; u < TERMS; ++u) mma16<F8>(c, f, p0[u], p1[u]);
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!PART || mine[e & 1]) o[i][e] = fmaf(c[e], F8 ? v_scale : 1.0f, o[i][e]);
    } else {
#pragma unroll
      for (int u = 0; u < TERMS; ++u) mma16<F8>(o[i], f, p0[u], p1[u]);
    }
  }
}

// One thread block's share: column tile ct of sequence s and KV head `head`, which is
// unit `unit`, the split-th run of its keys.
template <int D, bool F8, int TERMS>
__device__ __forceinline__ void attend(const KvAttnParams &a, int s, int head, int ct, int unit,
                                       int split) {
  using S = Shape<D, F8>;
  constexpr int kSteps = D / 16;
  constexpr float kShift = F8 ? 15.0f : 0.0f;
  __shared__ float s_m[kWarps][kCols], s_l[kWarps][kCols];
  extern __shared__ __align__(16) unsigned char s_ring[];
  // the warps' outputs meet where the rings were
  float(*s_o)[kCols][D + 4] = reinterpret_cast<float(*)[kCols][D + 4]>(s_ring);
  // and, of a cluster, this block's result behind them
  float(*s_joined)[D] = reinterpret_cast<float(*)[D]>(s_ring + sizeof(float) * kWarps * kCols * (D + 4));
  __shared__ float2 s_ml[kCols];
  static_assert(sizeof(float) * kCols * (kWarps * (D + 4) + D) <= S::kSmem, "they fit in the rings");
  const KvSeq q = kv_seq(a.b, s);
  // columns of this block (ct may be past the sequence's last)
  const int c1 = (int)min((int64_t)(ct + 1) * kCols, (int64_t)q.rows * a.G), c0 = ct * kCols;
  if (c0 >= c1 || !owns(a, q)) return;
  const int first = q.len - q.rows;  // position of the sequence's first row
  const int p_lo = first + c0 / a.G, p_hi = first + (c1 - 1) / a.G;
  const KvTiles tiles = visible_tiles(a, p_lo, p_hi, kKvBlock);
  const int i0 = split * a.tiles_per_split, i1 = min(i0 + a.tiles_per_split, tiles.count);
  if (split > 0 && i0 >= tiles.count && !a.cluster) return;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;

  // this warp's tiles: number n is tile i0 + warp + kWarps n
  const int mine = i1 - i0 - warp > 0 ? (i1 - i0 - warp + kWarps - 1) / kWarps : 0;
  auto key_of = [&](int n) { return kKvBlock * tiles.at(i0 + warp + kWarps * n); };
  // lane l looks up tile 32 batch + l: page, place and scales, far ahead of use
  auto look = [&](int batch) {
    Found x = {-1, 0, 0};
    const int n = 32 * batch + lane;
    if (n < mine) {
      const int key = key_of(n);
      const int at = (int)((unsigned)key / (unsigned)a.b.page_tokens);
      x.page = kv_page(a.b, s, at);
      x.slot = key - at * a.b.page_tokens;
      if (F8 && x.page >= 0) {
        const int64_t i = ((int64_t)x.page * a.b.h_kv + head) * (a.b.page_tokens / kKvBlock) +
                          x.slot / kKvBlock;
        x.scales = __ldg(a.k_scale + i) | (__ldg(a.v_scale + i) << 8);
      }
    }
    return x;
  };
  Found cur = look(0), next = look(1);
  const uint32_t ring = (uint32_t)__cvta_generic_to_shared(s_ring) + warp * S::kDepth * S::kStage;
  int batch = 0;  // of `cur`
  // starts the copy of tile n (of batch or batch + 1) into its place in the ring
  auto issue = [&](int n) {
    if (n < mine) {
      const bool here = n >> 5 == batch;
      const int page = __shfl_sync(0xffffffffu, here ? cur.page : next.page, n & 31);
      const int slot = __shfl_sync(0xffffffffu, here ? cur.slot : next.slot, n & 31);
      if (page >= 0) {
        const int64_t off = (((int64_t)page * a.b.h_kv + head) * a.b.page_tokens + slot) * S::kRow;
        const uint32_t to = ring + n % S::kDepth * S::kStage;
#pragma unroll
        for (int u = 0; u < S::kRow / 32; ++u) {
          const int i = lane + 32 * u, r = i / (S::kRow / 16), c = i % (S::kRow / 16);
          const uint32_t dst = to + r * S::kPitch + c * 16;
          tc_cp_async16(dst, static_cast<const uint8_t *>(a.ck) + off + i * 16, 16);
          tc_cp_async16(dst + S::kSide, static_cast<const uint8_t *>(a.cv) + off + i * 16, 16);
        }
      }
    }
    tc_cp_async_commit();
  };
  // q: column g, this lane's dimensions.  Its loads and the first tiles' copies are
  // on their way together.
  float qv[4 * kSteps];
  {
    const int c = c0 + g;
    const int64_t at = (int64_t)(q.row0 + c / a.G) * a.q_stride + (int64_t)(head * a.G + c % a.G) * D;
    constexpr int kPiece = S::kKVec / S::kElt;  // dimensions that follow each other
    const bool wide = a.q_wide;
#pragma unroll
    for (int e = 0; e < 4 * kSteps; e += kPiece) {
      const int64_t i = at + S::k_dim(e, t);
#pragma unroll
      for (int w = 0; w < kPiece; ++w) qv[e + w] = 0.0f;
      if (c < c1) {
        if (wide && a.q_bf16) {
#pragma unroll
          for (int w = 0; w < kPiece; w += 8) {
            const uint4 x = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.q) + i + w));
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int z = 0; z < 8; ++z)
              qv[e + w + z] = __uint_as_float(z & 1 ? y[z / 2] & 0xffff0000u : y[z / 2] << 16);
          }
        } else {
#pragma unroll
          for (int w = 0; w < kPiece; ++w) qv[e + w] = load_q(a.q, a.q_bf16, i + w);
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < S::kDepth - 1; ++n) issue(n);

  uint32_t qf[TERMS][kSteps][2];
  float col_scale = a.qscale;  // of column g: softmax scale * log2 e, and q's power of two back
  {
    if constexpr (F8) {
      float big = 0.0f;
#pragma unroll
      for (int e = 0; e < 4 * kSteps; ++e) big = fmaxf(big, fabsf(qv[e]));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 1));
      big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, 2));
      // big to [2^14, 2^15): exact, and 28 binades below stay normal
      const int e = min(max(14 - (((__float_as_int(big) >> 23) & 255) - 127), -120), 120);
      const float f = exp2i(e);
#pragma unroll
      for (int i = 0; i < 4 * kSteps; ++i) qv[i] *= f;
      col_scale *= exp2i(-e);
    }
#pragma unroll
    for (int u = 0; u < TERMS; ++u)
#pragma unroll
      for (int i = 0; i < kSteps; ++i)
#pragma unroll
        for (int w = 0; w < 2; ++w)
          qf[u][i][w] = split16<F8>(qv[4 * i + 2 * w], qv[4 * i + 2 * w + 1]);
  }
  // of this lane's accumulator columns 2t and 2t + 1: scale and position
  float cs[2];
  int pc[2];
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    cs[j] = __shfl_sync(0xffffffffu, col_scale, 4 * (2 * t + j));
    pc[j] = first + min(c0 + 2 * t + j, c1 - 1) / a.G;
  }

  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.0f, 0.0f};
  float o[D / 16][4];
#pragma unroll
  for (int i = 0; i < D / 16; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.0f;

  // the tile of keys key0 .. key0 + 15 in the ring at shared address `at`
  auto fold = [&](int key0, uint32_t at, float k_scale, float v_scale) {
    float sc[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sc2[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    {
      uint32_t k[2][S::kKWords];
#pragma unroll
      for (int r = 0; r < 2; ++r)
#pragma unroll
        for (int j = 0; j < S::kKWords * 4 / S::kKVec; ++j)
          load_bytes<S::kKVec>(at + (g + 8 * r) * S::kPitch + S::k_byte(j, t), &k[r][j * S::kKVec / 4]);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        uint32_t f[4];
        if constexpr (F8) {
          e4m3_half4(k[0][i], f[0], f[2]);
          e4m3_half4(k[1][i], f[1], f[3]);
        } else {
          f[0] = k[0][2 * i];
          f[1] = k[1][2 * i];
          f[2] = k[0][2 * i + 1];
          f[3] = k[1][2 * i + 1];
        }
#pragma unroll
        for (int u = 0; u < TERMS; ++u)  // two sums, so that half as many wait for each other
          mma16<F8>(i & 1 ? sc2 : sc, f, qf[u][i][0], qf[u][i][1]);
      }
    }
    uint32_t xv[4][S::kVWords];
#pragma unroll
    for (int r = 0; r < 4; ++r)
#pragma unroll
      for (int j = 0; j < S::kVWords * 4 / S::kVVec; ++j)
        load_bytes<S::kVVec>(at + S::kSide + (2 * t + (r & 1) + 8 * (r >> 1)) * S::kPitch + S::v_byte(j, g),
                             &xv[r][j * S::kVVec / 4]);
#pragma unroll
    for (int e = 0; e < 4; ++e) sc[e] = (sc[e] + sc2[e]) * (F8 ? cs[e & 1] * k_scale : cs[e & 1]);
    const bool whole = sees_all(a, p_lo, p_hi, key0, kKvBlock);
    if (!whole) {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (!sees(a, pc[e & 1], key0 + g + 8 * (e >> 1))) sc[e] = -INFINITY;
    }
    float corr[2];
    float mn[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float b = fmaxf(sc[j], sc[j + 2]);
      b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 4));
      b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 8));
      b = fmaxf(b, __shfl_xor_sync(0xffffffffu, b, 16));
      mn[j] = fmaxf(m[j], b);
    }
    if (__any_sync(0xffffffffu, mn[0] > m[0] || mn[1] > m[1])) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        corr[j] = mn[j] == -INFINITY ? 1.0f : ex2(m[j] - mn[j]);
        l[j] *= corr[j];
        m[j] = mn[j];
      }
#pragma unroll
      for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= corr[e & 1];
    }
    float p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float ref = m[e & 1] == -INFINITY ? 0.0f : m[e & 1] - kShift;
      p[e] = ex2(sc[e] - ref);
      l[e & 1] += p[e];
    }
    uint32_t p0[TERMS], p1[TERMS];
#pragma unroll
    for (int u = 0; u < TERMS; ++u) {
      p0[u] = transpose8(split16<F8>(p[0], p[1]));
      p1[u] = transpose8(split16<F8>(p[2], p[3]));
    }
    if (whole) {
      add_pv<D, F8, TERMS, false>(o, xv, v_scale, p0, p1, {true, true});
      return;
    }
    // token by token: V rows that the token does not see become zeros, and only
    // its columns take the product
    for (int pos = p_lo; pos <= p_hi; ++pos) {
      uint32_t v[4][S::kVWords];
      const bool mine[2] = {pc[0] == pos, pc[1] == pos};
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const bool see = sees(a, pos, key0 + 2 * t + (r & 1) + 8 * (r >> 1));
#pragma unroll
        for (int w = 0; w < S::kVWords; ++w) v[r][w] = see ? xv[r][w] : 0u;
      }
      add_pv<D, F8, TERMS, true>(o, v, v_scale, p0, p1, mine);
    }
  };

  for (int n = 0; n < mine; ++n) {
    if (n >> 5 != batch) {
      batch = n >> 5;
      cur = next;
      next = look(batch + 1);
    }
    tc_cp_async_wait<S::kDepth - 2>();  // tile n's own copies have landed,
    __syncwarp();                       // and the other lanes'; tile n - 1 has been read
    issue(n + S::kDepth - 1);
    const int page = __shfl_sync(0xffffffffu, cur.page, n & 31);
    const int sc = __shfl_sync(0xffffffffu, cur.scales, n & 31);
    if (page >= 0)
      fold(key_of(n), ring + n % S::kDepth * S::kStage, exp2i(kv_scale_exp(sc & 255)),
           exp2i(kv_scale_exp(sc >> 8)));
  }
  tc_cp_async_wait<0>();
  __syncthreads();  // the rings are free

#pragma unroll
  for (int j = 0; j < 2; ++j) {
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 4);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 8);
    l[j] += __shfl_xor_sync(0xffffffffu, l[j], 16);
    if (g == 0) {
      s_m[warp][2 * t + j] = m[j];
      s_l[warp][2 * t + j] = l[j];
    }
  }
#pragma unroll
  for (int i2 = 0; i2 < D / 16; ++i2)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      s_o[warp][2 * t + (e & 1)][S::v_dim(2 * i2 + (e >> 1), g)] = o[i2][e];
  __syncthreads();
  for (int y = threadIdx.x; y < (c1 - c0) * D; y += kThreads) {
    const int c = y / D, dim = y % D;
    float M = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w][c]);
    float L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w][c] == -INFINITY ? 0.0f : exp2f(s_m[w][c] - M);
      L = fmaf(s_l[w][c], f, L);
      // (a warp that saw nothing has zeros)
      O = fmaf(s_o[w][c][dim], f, O);
    }
    if (a.cluster) {
      s_joined[c][dim] = O;
      if (dim == 0) s_ml[c] = make_float2(M, L);
      continue;
    }
    const int row = q.row0 + (c0 + c) / a.G, h = head * a.G + (c0 + c) % a.G;
    const int64_t rh = (int64_t)row * a.h_q + h;
    if (a.splits == 1) {
      store_out(a, rh * D + dim, L > 0.0f ? O / L : (L == 0.0f ? 0.0f : L));
      if (dim == 0 && a.lse) a.lse[rh] = lse_of(M, L, kShift);
    } else {
      const int64_t part = part_at(a, unit, split) + c;
      a.part_o[part * D + dim] = O;
      if (dim == 0) a.part_ml[part] = make_float2(M, L);
    }
  }
  if (!a.cluster) return;
  // the splits of a unit are a cluster: each block joins its share of the columns'
  // dimensions over all of them
  cg::cluster_group cluster = cg::this_cluster();
  cluster.sync();  // every block's result is in its shared memory
  for (int y = split * kThreads + threadIdx.x; y < (c1 - c0) * D; y += a.splits * kThreads) {
    const int c = y / D, dim = y % D;
    float M = -INFINITY;
    for (int r = 0; r < a.splits; ++r) M = fmaxf(M, cluster.map_shared_rank(&s_ml[c], r)->x);
    float L = 0.0f, O = 0.0f;
    for (int r = 0; r < a.splits; ++r) {
      const float2 ml = *cluster.map_shared_rank(&s_ml[c], r);
      const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : ml.y) : exp2f(ml.x - M);
      L = fmaf(ml.y, f, L);
      O = fmaf(*cluster.map_shared_rank(&s_joined[c][dim], r), f, O);
    }
    const int64_t rh = (int64_t)(q.row0 + (c0 + c) / a.G) * a.h_q + head * a.G + (c0 + c) % a.G;
    store_out(a, rh * D + dim, L > 0.0f ? O / L : (L == 0.0f ? 0.0f : L));
    if (dim == 0 && a.lse) a.lse[rh] = lse_of(M, L, kShift);
  }
  cluster.sync();  // the others have read this block's
}

template <int D, bool F8, int TERMS>
__global__ void __launch_bounds__(kThreads, TERMS > 1 || D > 128 ? 1 : F8 ? 4 : 3)
    kv_attention_kernel(KvAttnParams a) {
  grid_dependency_wait();
  allow_dependent_launch();
  int x = blockIdx.x;
  if (x >= a.units * a.b.h_kv * a.splits) {  // one (cluster) more, if it reports
    if (x == a.units * a.b.h_kv * a.splits) write_status(a);
    return;
  }
  const int split = x % a.splits;
  x /= a.splits;
  const KvUnit u = kv_unit(a, x / a.b.h_kv);
  attend<D, F8, TERMS>(a, u.s, x % a.b.h_kv, u.ct, x, split);
}

// After the many-rows kernel: the units that it marked, column tile by column
// tile, each over all its keys.  Its waits that ran out are added to the status here,
// which is complete by now.
template <int D, bool F8>
__global__ void __launch_bounds__(kThreads) kv_redo_kernel(KvAttnParams a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int per = a.cols / kCols, units = a.units * a.b.h_kv;
  KvAttnParams b = a;
  b.splits = 1;
  b.cluster = 0;
  b.tiles_per_split = 1 << 30;
  for (int x0 = blockIdx.x * kThreads; x0 < units; x0 += gridDim.x * kThreads) {
    // a thread looks at one unit's marks; marked ones are rare
    int marked = 0, late = 0;
    if (x0 + (int)threadIdx.x < units)
      for (int i = 0; i < a.splits; ++i) {
        const int mark = a.taint[(int64_t)(x0 + threadIdx.x) * a.splits + i];
        marked |= mark;
        late += (mark & kMarkLate) != 0;
      }
    if (late) atomicAdd(&a.status->device_faults, (uint32_t)late);
    if (!__syncthreads_or(marked)) continue;
    for (int k = 0; k < kThreads; ++k) {
      if (!__syncthreads_or(marked && (int)threadIdx.x == k)) continue;
      const KvUnit u = kv_unit(a, (x0 + k) / a.b.h_kv);
      const KvSeq q = kv_seq(a.b, u.s);
      const int rb = (q.rows * a.G + a.cols - 1) / a.cols - 1 - u.ct;  // (units come last first)
      for (int ct = 0; ct < per; ++ct) {
        attend<D, F8, 1>(b, u.s, (x0 + k) % a.b.h_kv, rb * per + ct, x0 + k, 0);
        __syncthreads();
      }
    }
  }
}

// One warp's part in joining the splits of one column of a unit, the first split's
// result being number `at`: of n splits those from `from` on, every `step`-th; lane l has dimensions l, l + 32, ...  The splits' maxima
// and sums are read 32 at a time, their outputs 8 at a time, so that their latency
// is not paid split by split.
template <int D>
__device__ __forceinline__ void join_splits(const KvAttnParams &a, int64_t at, int n, int from,
                                            int step, float &m, float &l, float (&o)[D / 32]) {
  constexpr int kPer = D / 32;
  const int lane = threadIdx.x & 31;
  const int mine = n > from ? (n - from + step - 1) / step : 0;
  m = -INFINITY;
  l = 0.0f;
#pragma unroll
  for (int j = 0; j < kPer; ++j) o[j] = 0.0f;
  for (int i0 = 0; i0 < mine; i0 += 32) {
    const int split = from + step * (i0 + lane);
    const float2 ml = split < n ? a.part_ml[at + (int64_t)split * a.part_cols] : make_float2(-INFINITY, 0.0f);
    float big = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
    const float next = fmaxf(m, big);
    const float corr = next == -INFINITY ? 1.0f : exp2f(m - next);
    // (a split that saw nothing has -inf, 0 and zeros; NaN stays NaN)
    const float f = ml.x == -INFINITY ? (ml.y == 0.0f ? 0.0f : ml.y) : exp2f(ml.x - next);
    float sum = ml.y * f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    l = l * corr + sum;
#pragma unroll
    for (int j = 0; j < kPer; ++j) o[j] *= corr;
    m = next;
    const int here = min(32, mine - i0);
    for (int k0 = 0; k0 < here; k0 += 8) {
      float v[8][kPer];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float *po =
            a.part_o + (at + (from + step * (int64_t)(i0 + k0 + k)) * a.part_cols) * D + lane;
#pragma unroll
        for (int j = 0; j < kPer; ++j) v[k][j] = k0 + k < here ? po[32 * j] : 0.0f;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = __shfl_sync(0xffffffffu, f, (k0 + k) & 31);
#pragma unroll
        for (int j = 0; j < kPer; ++j)
          if (k0 + k < here) o[j] = fmaf(v[k][j], w, o[j]);
      }
    }
  }
}

// Few rows: a block joins the splits of one column of a unit, its warps every
// fourth.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_join_kernel(KvAttnParams a, float shift) {
  grid_dependency_wait();
  allow_dependent_launch();
  __shared__ float s_m[kWarps], s_l[kWarps], s_o[kWarps][D];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int x = (int)(blockIdx.x / kCols), head = x % a.b.h_kv;
  const KvUnit u = kv_unit(a, x / a.b.h_kv);
  const KvSeq q = kv_seq(a.b, u.s);
  const int c1 = (int)min((int64_t)(u.ct + 1) * kCols, (int64_t)q.rows * a.G), c0 = u.ct * kCols;
  const int col = c0 + (int)(blockIdx.x % kCols);
  if (col >= c1 || !owns(a, q)) return;
  const int first = q.len - q.rows;
  const int64_t rh = (int64_t)(q.row0 + col / a.G) * a.h_q + head * a.G + col % a.G;
  const KvTiles tiles = visible_tiles(a, first + c0 / a.G, first + (c1 - 1) / a.G, a.tile);
  const int n = max(1, (tiles.count + a.tiles_per_split - 1) / a.tiles_per_split);
  float m, l, o[D / 32];
  join_splits<D>(a, part_at(a, x, 0) + (col - c0), n, warp, kWarps, m, l, o);
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
#pragma unroll
  for (int j = 0; j < D / 32; ++j) s_o[warp][32 * j + lane] = o[j];
  __syncthreads();
  for (int c = threadIdx.x; c < D; c += kThreads) {
    float M = -INFINITY, L = 0.0f, O = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, s_m[w]);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float f = s_m[w] == -INFINITY ? (s_l[w] == 0.0f ? 0.0f : s_l[w]) : exp2f(s_m[w] - M);
      L = fmaf(s_l[w], f, L);
      O = fmaf(s_o[w][c], f, O);
    }
    store_out(a, rh * D + c, L > 0.0f ? O / L : (L == 0.0f ? 0.0f : L));
    if (c == 0 && a.lse) a.lse[rh] = lse_of(M, L, shift);
  }
}

// Many rows: a warp joins the splits of one column of a divided unit.
template <int D>
__global__ void __launch_bounds__(kThreads) kv_join_units_kernel(KvAttnParams a) {
  grid_dependency_wait();
  allow_dependent_launch();
  const int per = a.cols / kWarps, lane = threadIdx.x & 31;  // blocks of a unit
  const int x = a.tail_from + (int)blockIdx.x / per, head = x % a.b.h_kv;
  const KvUnit u = kv_unit(a, x / a.b.h_kv);
  const KvSeq q = kv_seq(a.b, u.s);
  const int rb = (q.rows * a.G + a.cols - 1) / a.cols - 1 - u.ct;  // (units come last first)
  if (rb < 0 || !owns(a, q)) return;
  const int c0 = rb * a.cols, c1 = min(c0 + a.cols, q.rows * a.G), first = q.len - q.rows;
  const int col = c0 + (int)blockIdx.x % per * kWarps + (threadIdx.x >> 5);
  if (col >= c1) return;
  const KvTiles tiles = visible_tiles(a, first + c0 / a.G, first + (c1 - 1) / a.G, a.tile);
  const int n = max(1, (tiles.count + a.tiles_per_split - 1) / a.tiles_per_split);
  const int64_t rh = (int64_t)(q.row0 + col / a.G) * a.h_q + head * a.G + col % a.G;
  float m, l, o[D / 32];
  join_splits<D>(a, part_at(a, x, 0) + (col - c0), n, 0, 1, m, l, o);
#pragma unroll
  for (int j = 0; j < D / 32; ++j)
    store_out(a, rh * D + 32 * j + lane, l > 0.0f ? o[j] / l : (l == 0.0f ? 0.0f : l));
  if (lane == 0 && a.lse) a.lse[rh] = lse_of(m, l, 0.0f);
}

// A call without rows: its status.
__global__ void __launch_bounds__(kThreads) kv_status_kernel(KvAttnParams a) {
  grid_dependency_wait();
  allow_dependent_launch();
  write_status(a);
}

template <int D, bool F8, typename Kernel>
cudaError_t launch_ring(Kernel kernel, int64_t blocks, const KvAttnParams &a, cudaStream_t s) {
  constexpr int smem = Shape<D, F8>::kSmem;
  cudaError_t e = cudaSuccess;
  if (smem > 48 * 1024)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e == cudaSuccess && a.cluster && a.splits > 8)
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  if (!a.cluster) return launch_dependent(kernel, dim3((unsigned)blocks), dim3(kThreads), smem, s, a);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.splits;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

template <int D, bool F8>
cudaError_t launch_redo(const KvAttnParams &a, cudaStream_t s) {
  const int64_t blocks = ((int64_t)a.units * a.b.h_kv + kThreads - 1) / kThreads;
  KvAttnParams b = a;
  b.cluster = 0;
  return launch_ring<D, F8>(kv_redo_kernel<D, F8>, blocks < 296 ? blocks : 296, b, s);
}

template <int D>
cudaError_t launch_d(const KvAttnParams &a, bool f8, cudaStream_t s) {
  const int64_t blocks =
      (int64_t)a.units * a.b.h_kv * a.splits + (a.report ? (a.cluster ? a.splits : 1) : 0);
  const dim3 block(kThreads);
  cudaError_t e;
  if (a.many_rows)
    e = launch_kv_prompt(a, f8, s);
  else if (f8)
    e = a.q_bf16 ? launch_ring<D, true>(kv_attention_kernel<D, true, 1>, blocks, a, s)
                 : launch_ring<D, true>(kv_attention_kernel<D, true, 2>, blocks, a, s);
  else
    e = a.q_bf16 ? launch_ring<D, false>(kv_attention_kernel<D, false, 1>, blocks, a, s)
                 : launch_ring<D, false>(kv_attention_kernel<D, false, 3>, blocks, a, s);
  if (e == cudaSuccess && a.splits > 1 && !a.many_rows && !a.cluster)
    e = launch_dependent(kv_join_kernel<D>, dim3((unsigned)((int64_t)a.units * a.b.h_kv * kCols)),
                         block, 0, s, a, f8 ? 15.0f : 0.0f);
  if constexpr (D >= 64)
    if (e == cudaSuccess && a.splits > 1 && a.many_rows) {
      const int64_t n = ((int64_t)a.units * a.b.h_kv - a.tail_from) * (a.cols / kWarps);
      e = launch_dependent(kv_join_units_kernel<D>, dim3((unsigned)n), block, 0, s, a);
    }
  if constexpr (D >= 64)
    if (e == cudaSuccess && a.many_rows)
      e = f8 ? launch_redo<D, true>(a, s) : launch_redo<D, false>(a, s);
  return e;
}

}  // namespace

// Blocks of the few-rows kernel that the device holds at once, by shared memory
// (228 KB an SM, 1 KB of it for each block).  bf16 queries up to 128 dimensions have
// no more registers than that allows; fp32 queries and more dimensions have up to 255
// a thread, which is two or three blocks an SM where this says three or four, and their
// grids are up to two waves.
static int kv_resident_blocks(int d, bool f8) {
  const int row = f8 ? d : 2 * d;
  const int smem = kWarps * ring_depth(row) * 2 * kKvBlock * (row + 16) + 1280;
  const int per = 228 * 1024 / smem;
  return 148 * (per > 4 ? 4 : per);
}

// The most tiles of `tile` keys that `rows` tokens in a row can see, at least 1.
static int64_t most_tiles(const KvAttnParams &a, int64_t rows, int tile) {
  int64_t most = ((int64_t)a.b.max_len + tile - 1) / tile;
  if (a.window < a.b.max_len) {
    const int64_t w = ((int64_t)a.window + rows - 1 + tile - 2) / tile + 1 +
                      ((int64_t)a.sinks + tile - 1) / tile;
    if (w < most) most = w;
  }
  return most < 1 ? 1 : most;
}

// One launch's plan: of the few-rows or the many-rows kernel, for a.own's sequences.
static void plan_one(KvAttnParams &a, bool f8) {
  const int d = a.d;
  int64_t max_cols = (int64_t)a.b.max_rows * a.G;
  if (a.own == kFewRows && max_cols >= a.many_from) max_cols = a.many_from - 1;
  const int64_t all_pairs = (int64_t)a.b.num_seqs * a.b.h_kv;
  a.pair0 = 0;
  a.pairs = (int)all_pairs;
  a.n_pad = 0;
  a.box_rows = kPromptTile;
  if (a.many_rows && f8) {
    // The widened copy holds as many pairs at a time as fit in 4 GiB, of each the tiles
    // that some row may see.
    a.n_pad = (int)(most_tiles(a, a.b.max_rows, kPromptTile) * kPromptTile);
    const int64_t fit = ((int64_t)4 << 30) / ((int64_t)a.n_pad * d * 4);
    a.pairs = (int)(fit < 1 ? 1 : fit < all_pairs ? fit : all_pairs);
  } else if (a.many_rows) {
    while (a.b.page_tokens % a.box_rows) a.box_rows /= 2;
  }
  a.cols = a.many_rows ? prompt_cols(d) : kCols;
  a.tile = a.many_rows ? kPromptTile : kKvBlock;
  a.part_cols = (int)(max_cols < a.cols ? max_cols : a.cols);
  a.col_tiles = (int)((max_cols + a.cols - 1) / a.cols);
  const int64_t dense = (int64_t)a.b.num_seqs * a.col_tiles;
  const int64_t packed = (int64_t)a.b.num_rows * a.G / a.cols + a.b.num_seqs;
  a.dense = a.b.q_start == nullptr || dense <= packed;
  const int64_t units = a.dense ? dense : packed;
  a.units = (int)(units < INT32_MAX ? units : INT32_MAX);  // (the caller checks the launch's size)
  // the most tiles that one unit's columns can see
  const int64_t tokens = (a.cols + a.G - 2) / a.G + 1;  // tokens that `cols` columns can span
  const int64_t most = most_tiles(a, tokens, a.tile);
  const bool windowed = most < ((int64_t)a.b.max_len + a.tile - 1) / a.tile;
  const int64_t base = units * a.b.h_kv;
  int64_t splits;
  a.tail_from = 0;
  if (a.many_rows) {
    // One block an SM.  Fewer units than SMs: each is divided.  More, of one sequence
    // and about equal length (a chunk over a long context, a window): those that
    // would be left over for a last, partly filled wave are divided to fill it.
    // (Units of a prompt from its start grow with their rows; the short ones come
    // last and fill the gaps.)
    const bool even = windowed || (int64_t)a.b.max_len >= 4 * (int64_t)a.b.max_rows;
    splits = 148 / base;
    if (base > 148 && even && a.b.num_seqs == 1 && a.pairs == all_pairs && base % 148) {
      a.tail_from = (int)(base - base % 148);
      splits = 148 / (base % 148);
    }
    if (splits > most / 8) splits = most / 8;
  } else {
    // Runs of at least 4 tiles a warp, sized by max_len.  Where every sequence goes
    // through about the same number of tiles (a window), as many blocks as the SMs hold
    // at once, rounded up to whole units (64 windowed sessions: 512 on 444 places);
    // where lengths differ from the bound and from each other, smaller runs, so that the
    // SMs end together (24 sessions of 4096 to 65536 tokens: 501 us with one block
    // a place, 357 with 2, 309 with 4, 292 with 8; one session, 64 windowed ones: 1
    // to 4 are within 1%, 8 costs 2 and 6%).
    const int64_t waves = windowed ? 1 : a.b.num_seqs > 1 ? 8 : 4;
    const int64_t want = (waves * kv_resident_blocks(d, f8) + base - 1) / base;
    splits = most / (4 * kWarps);
    if (splits > want) splits = want;
  }
  if (splits < 1) splits = 1;
  a.tiles_per_split = (int)((most + splits - 1) / splits);
  a.splits = (int)((most + a.tiles_per_split - 1) / a.tiles_per_split);
  // Few splits are a cluster and join through its shared memory, without the
  // workspace and a second launch.
  a.cluster = !a.many_rows && a.splits > 1 && a.splits <= kMaxCluster;
}

int plan_kv_attention(const KvAttnParams &a, bool f8, KvAttnParams (&plan)[2]) {
  // The tcgen05 kernel multiplies 256 columns at a time (128 beyond 128 dimensions).
  // It takes sequences of many_from columns or more, if the queries are bf16; its
  // tensor map counts the cache's rows in 31 bits.
  // It reads K and V once for all columns, the few-rows kernel once for every 8; but
  // that one reads e4m3 as it is and divides short runs of keys further.  In us, few
  // against many, 24 sequences of 4096 to 65536 tokens: bf16 16 columns 1256, 780;
  // 32 columns 2178, 818; e4m3 32 columns 1479, 2070; 64 columns 2674, 2068.  64
  // sequences with a window of 4096, bf16, 16 columns: 220, 272.  One of 4099 tokens:
  // 25, 33.
  const bool far = a.b.max_len >= 16384 && a.window >= a.b.max_len;
  const int many_from = f8 ? 64 : far ? 16 : 24;
  const int64_t rows = (int64_t)a.b.num_pages * a.b.h_kv * a.b.page_tokens;
  const bool many = a.q_bf16 && a.d >= 64 && (int64_t)a.b.max_rows * a.G >= many_from &&
                    a.G <= 4096 && (f8 || rows < ((int64_t)1 << 31));
  plan[0] = a;
  plan[0].many_rows = many;
  plan[0].many_from = many_from;
  plan[0].own = kEverySequence;
  plan[0].report = 1;
  // Sequences may have more rows or fewer (a prompt beside decoded tokens): those
  // with few go to the few-rows kernel, which divides a long context among blocks
  // and reads e4m3 as it is.
  const bool both = many && a.b.q_start != nullptr && a.b.num_seqs > 1;
  if (both) {
    plan[1] = plan[0];
    plan[0].own = kManyRows;
    plan[1].own = kFewRows;
    plan[1].many_rows = 0;
    plan[1].report = 0;
    plan_one(plan[1], f8);
  }
  plan_one(plan[0], f8);
  return both ? 2 : 1;
}

cudaError_t launch_kv_status(const KvAttnParams &a, cudaStream_t s) {
  return launch_dependent(kv_status_kernel, dim3(1), dim3(kThreads), 0, s, a);
}

cudaError_t launch_kv_attention(const KvAttnParams &a, bool f8, cudaStream_t s) {
  switch (a.d / 32) {
    case 1: return launch_d<32>(a, f8, s);
    case 2: return launch_d<64>(a, f8, s);
    case 3: return launch_d<96>(a, f8, s);
    case 4: return launch_d<128>(a, f8, s);
    case 5: return launch_d<160>(a, f8, s);
    case 6: return launch_d<192>(a, f8, s);
    case 7: return launch_d<224>(a, f8, s);
    case 8: return launch_d<256>(a, f8, s);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace fathom
