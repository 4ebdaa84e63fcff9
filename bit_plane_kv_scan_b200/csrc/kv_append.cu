// fathom_kv_append: new keys and values into the paged cache, keys and queries
// rotated by their positions on the way.
//
// Row at position p, pair r: angle a = p f_r, (x, y) -> (x cos a - y sin a,
// y cos a + x sin a).  The angle is formed and reduced to [-pi, pi] in fp64 (in
// fp32 a position of a million turns by a wrong 0.06), then sincosf.
//
// A unit is the rows of one sequence that fall into one block of 16 positions.
// Its first thread block takes keys and values, the others `q_heads` query heads
// each; each works out the unit's sines and cosines for itself (1024 of them at
// d = 128, against 32768 elements or more) and keeps them in shared memory.
//
// An E4M3 cache has a power-of-two scale per block of 16 tokens and KV head, so
// a whole block belongs to one warp: it finds the largest new element, raises
// the scale if it must, moves the codes that the block already held, and writes
// the new ones (it reads its rows twice, the second time from L1).  The scale
// comes from the elements before the rotation, which makes it the same whatever
// the sines' last bit, and leaves room for sqrt 2.
//
// Bound by bytes: every element is read and written once.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace fathom {

constexpr int kAppendWarps = 8;
constexpr int kAppendThreads = 32 * kAppendWarps;

struct AppendParams {
  KvBatch b;
  int d, h_q;          // (h_q: 0 without queries)
  int q_heads, parts;  // query heads of a thread block, thread blocks of a unit
  void *ck, *cv;
  uint8_t *k_scale, *v_scale;
  const void *k, *v, *q;
  void *q_out;
  int64_t k_stride, v_stride, q_stride;
  const float *inv_freq;
  int pairs, interleaved;
};

template <typename T>
__device__ __forceinline__ float to_float(T x);
template <>
__device__ __forceinline__ float to_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ float to_float<__nv_bfloat16>(__nv_bfloat16 x) {
  return __bfloat162float(x);
}
template <typename T>
__device__ __forceinline__ T from_float(float x);
template <>
__device__ __forceinline__ float from_float<float>(float x) { return x; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_float<__nv_bfloat16>(float x) {
  return __float2bfloat16_rn(x);
}

// N elements of a row (16-byte aligned when N = 8).
template <typename T, int N>
struct alignas(N == 8 ? 16 : sizeof(T)) Vec {
  T x[N];
};

// cos and sin of p f, the angle in fp64.
__device__ __forceinline__ float2 cos_sin(int p, float f) {
  const double a = (double)p * (double)f;
  const double turns = rint(a * 0.15915494309189535);  // 1 / 2 pi
  double r = fma(-turns, 6.283185307179586, a);
  r = fma(-turns, 2.4492935982947064e-16, r);  // 2 pi less its fp64 value
  float s, c;
  sincosf((float)r, &s, &c);
  return make_float2(c, s);
}

// One row's head, rotated: task t of the head is elements of W pairs, or W
// elements that stay.  `put(dim, Vec)` stores W elements from dimension dim.
template <int W, typename T, typename Put>
__device__ __forceinline__ void rotate_task(const T *head, int t, int d, int pairs, int interleaved,
                                            const float2 *cs, Put put) {
  const int turned = interleaved && W > 1 ? 2 * pairs / W : pairs / W;  // tasks with pairs
  if (t >= turned) {
    const int at = 2 * pairs + (t - turned) * W;
    const Vec<T, W> v = *reinterpret_cast<const Vec<T, W> *>(head + at);
    float o[W];
#pragma unroll
    for (int i = 0; i < W; ++i) o[i] = to_float(v.x[i]);
    put(at, o, o);
    return;
  }
  if (interleaved) {
    if constexpr (W >= 2) {
      const Vec<T, W> v = *reinterpret_cast<const Vec<T, W> *>(head + t * W);
      float o[W], raw[W];
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const float2 c = cs[(t * W + i) / 2];
        const float x = to_float(v.x[i]), y = to_float(v.x[i + 1]);
        raw[i] = x;
        raw[i + 1] = y;
        o[i] = x * c.x - y * c.y;
        o[i + 1] = y * c.x + x * c.y;
      }
      put(t * W, o, raw);
    } else {
      const float2 c = cs[t];
      const float x[1] = {to_float(head[2 * t])}, y[1] = {to_float(head[2 * t + 1])};
      const float ox[1] = {x[0] * c.x - y[0] * c.y}, oy[1] = {y[0] * c.x + x[0] * c.y};
      put(2 * t, ox, x);
      put(2 * t + 1, oy, y);
    }
    return;
  }
  const Vec<T, W> a = *reinterpret_cast<const Vec<T, W> *>(head + t * W);
  const Vec<T, W> b = *reinterpret_cast<const Vec<T, W> *>(head + pairs + t * W);
  float oa[W], ob[W], ra[W], rb[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const float2 c = cs[t * W + i];
    ra[i] = to_float(a.x[i]);
    rb[i] = to_float(b.x[i]);
    oa[i] = ra[i] * c.x - rb[i] * c.y;
    ob[i] = rb[i] * c.x + ra[i] * c.y;
  }
  put(t * W, oa, ra);
  put(pairs + t * W, ob, rb);
}

// Tasks of one head: pairs W at a time, then the elements that stay.
template <int W>
__host__ __device__ __forceinline__ int rotate_tasks(int d, int pairs, int interleaved) {
  return (interleaved && W > 1 ? 2 * pairs / W : pairs / W) + (d - 2 * pairs) / W;
}

template <int W, typename T>
__device__ __forceinline__ void store_vec(T *at, const float *o) {
  Vec<T, W> v;
#pragma unroll
  for (int i = 0; i < W; ++i) v.x[i] = from_float<T>(o[i]);
  *reinterpret_cast<Vec<T, W> *>(at) = v;
}

// The smallest exponent byte whose scale holds |x| <= big within 256.
__device__ __forceinline__ int scale_byte(float big) {
  if (big == 0.0f) return FATHOM_KV_SCALE_MIN;
  int e = ilogbf(big);                        // big = m 2^e, 1 <= m < 2
  if (scalbnf(1.0f, e) != big) ++e;           // smallest power of two >= big
  return min(max(e - 8 + 127, FATHOM_KV_SCALE_MIN), FATHOM_KV_SCALE_MAX);
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b, float c, float e) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, e), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}

__device__ __forceinline__ float e4m3_float(uint32_t code) {
  return __half2float(__half(__nv_cvt_fp8_to_halfraw((__nv_fp8_storage_t)code, __NV_E4M3)));
}

// Rows m of a unit, `heads` heads each of `per` tasks, by the whole thread block:
// fn(row, head, task).
template <typename Fn>
__device__ __forceinline__ void for_tasks(int m, int heads, int per, Fn fn) {
  const int n = m * heads * per;
#pragma unroll 4
  for (int i = threadIdx.x; i < n; i += kAppendThreads) {
    const int t = i % per, rh = i / per;
    fn(rh / heads, rh % heads, t);
  }
}

// A sequence's m rows touch at most m / 16 + 2 blocks of positions, so the units
// of sequence s start at q_start[s] / 16 + 2 s.
template <int W, typename TKV, typename TQ, bool E4M3>
__global__ void __launch_bounds__(kAppendThreads) append_kernel(AppendParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float2 cs[];  // [16][pairs]
  const int d = p.d;
  const int unit = blockIdx.x / p.parts, part = blockIdx.x % p.parts;
  int s = unit, u = 0;
  if (p.b.q_start) {
    auto base = [&](int i) { return (int64_t)(p.b.q_start[i] >> 4) + 2 * (int64_t)i; };
    s = find_seq(p.b.num_seqs, unit, base);
    u = unit - (int)base(s);
  }
  const KvSeq q = kv_seq(p.b, s);
  const int old = q.len - q.rows;  // tokens that the sequence had (< 0: more rows than tokens)
  // this unit's rows: those whose positions fall into one block of 16
  const int blk = (old >> 4) + u;  // floor: positions below 0 have blocks below 0
  const int p0 = max(blk * kKvBlock, old), p1 = min((blk + 1) * kKvBlock, q.len);
  if (u < 0 || p1 <= p0) return;
  const int row0 = q.row0 + (p0 - old), m = p1 - p0;
  for (int i = threadIdx.x; i < m * p.pairs; i += kAppendThreads)
    cs[i] = cos_sin(p0 + i / p.pairs, p.inv_freq[i % p.pairs]);
  __syncthreads();

  if (part > 0) {  // queries
    const int h0 = (part - 1) * p.q_heads, heads = min(p.q_heads, p.h_q - h0);
    const TQ *src = static_cast<const TQ *>(p.q) + (int64_t)row0 * p.q_stride + (int64_t)h0 * d;
    TQ *dst = static_cast<TQ *>(p.q_out) + ((int64_t)row0 * p.h_q + h0) * d;
    for_tasks(m, heads, rotate_tasks<W>(d, p.pairs, p.interleaved), [&](int r, int h, int t) {
      TQ *out = dst + ((int64_t)r * p.h_q + h) * d;
      rotate_task<W>(src + r * p.q_stride + h * d, t, d, p.pairs, p.interleaved, cs + r * p.pairs,
                     [&](int at, const float *o, const float *) { store_vec<W>(out + at, o); });
    });
    return;
  }
  if (blk < 0) return;
  const int page = kv_page(p.b, s, blk * kKvBlock / p.b.page_tokens);
  if (page < 0) return;
  const int held = p0 - blk * kKvBlock;                         // tokens the block has from before
  const int slot0 = blk * kKvBlock % p.b.page_tokens;           // the block's first row in its page
  const int64_t head0 = (int64_t)page * p.b.h_kv;
  const TKV *k = static_cast<const TKV *>(p.k) + (int64_t)row0 * p.k_stride;
  const TKV *v = static_cast<const TKV *>(p.v) + (int64_t)row0 * p.v_stride;
  const int per_k = rotate_tasks<W>(d, p.pairs, p.interleaved), per_v = d / W;

  if constexpr (!E4M3) {
    auto place = [&](void *base, int r, int g) {
      return static_cast<__nv_bfloat16 *>(base) +
             ((head0 + g) * p.b.page_tokens + slot0 + held + r) * d;
    };
    for_tasks(m, p.b.h_kv, per_k, [&](int r, int g, int t) {
      __nv_bfloat16 *out = place(p.ck, r, g);
      rotate_task<W>(k + r * p.k_stride + g * d, t, d, p.pairs, p.interleaved, cs + r * p.pairs,
                     [&](int at, const float *o, const float *) { store_vec<W>(out + at, o); });
    });
    for_tasks(m, p.b.h_kv, per_v, [&](int r, int g, int t) {
      rotate_task<W>(v + r * p.v_stride + g * d, t, d, 0, 0, cs,
                     [&](int at, const float *o, const float *) { store_vec<W>(place(p.cv, r, g) + at, o); });
    });
    return;
  } else {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int i = warp; i < 2 * p.b.h_kv; i += kAppendWarps) {
      const bool is_v = i >= p.b.h_kv;
      const int g = is_v ? i - p.b.h_kv : i;
      const TKV *src = (is_v ? v : k) + g * d;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      const int64_t head = head0 + g;
      uint8_t *scale = (is_v ? p.v_scale : p.k_scale) + head * (p.b.page_tokens / kKvBlock) +
                       slot0 / kKvBlock;
      uint8_t *codes = static_cast<uint8_t *>(is_v ? p.cv : p.ck) + (head * p.b.page_tokens + slot0) * d;
      const int was = held ? kv_scale_exp(*scale) + 127 : 0;
      float big = 0.0f;
#pragma unroll 4
      for (int t = lane; t < m * per_v; t += 32) {
        const int r = t / per_v;
        const Vec<TKV, W> x = *reinterpret_cast<const Vec<TKV, W> *>(src + r * stride + (t - r * per_v) * W);
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float y = fabsf(to_float(x.x[e]));
          if (y < INFINITY) big = fmaxf(big, y);
        }
      }
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) big = fmaxf(big, __shfl_xor_sync(0xffffffffu, big, off));
      int x = scale_byte(big);
      if (held && x > was) {  // the older codes move to the larger scale
        const float f = x - was > 126 ? 0.0f : exp2i(was - x);
        uint32_t *c4 = reinterpret_cast<uint32_t *>(codes);
        for (int t = lane; t < held * d / 4; t += 32) {
          const uint32_t c = c4[t];
          c4[t] = pack_e4m3(e4m3_float(c & 255) * f, e4m3_float((c >> 8) & 255) * f,
                            e4m3_float((c >> 16) & 255) * f, e4m3_float(c >> 24) * f);
        }
      } else if (held) {
        x = was;
      }
      const float f = exp2i(127 - x);
      uint8_t *out = codes + held * d;
      const int per = is_v ? per_v : per_k, pairs = is_v ? 0 : p.pairs;
#pragma unroll 4
      for (int t = lane; t < m * per; t += 32) {
        const int r = t / per;
        rotate_task<W>(src + r * stride, t - r * per, d, pairs, is_v ? 0 : p.interleaved,
                       cs + r * p.pairs, [&](int at, const float *o, const float *) {
                         uint8_t *to = out + r * d + at;
                         if constexpr (W == 8)
                           *reinterpret_cast<uint2 *>(to) =
                               make_uint2(pack_e4m3(o[0] * f, o[1] * f, o[2] * f, o[3] * f),
                                          pack_e4m3(o[4] * f, o[5] * f, o[6] * f, o[7] * f));
                         else
                           *to = (uint8_t)__nv_cvt_float_to_fp8(o[0] * f, __NV_SATFINITE, __NV_E4M3);
                       });
      }
      if (lane == 0) *scale = (uint8_t)x;
    }
  }
}

template <int W, typename TKV, typename TQ>
static cudaError_t launch_append_typed(AppendParams p, bool e4m3, cudaStream_t stream) {
  const int64_t units = p.b.q_start ? p.b.num_rows / kKvBlock + 2 * (int64_t)p.b.num_seqs : p.b.num_seqs;
  // query heads of a thread block: 4 tasks a thread where units have 16 rows
  const int rows = p.b.max_rows < kKvBlock ? p.b.max_rows : kKvBlock;
  const int per = rotate_tasks<W>(p.d, p.pairs, p.interleaved);
  int heads = 4 * kAppendThreads / (rows * per);
  heads = heads < 1 ? 1 : heads > p.h_q ? p.h_q : heads;
  p.q_heads = heads < 1 ? 1 : heads;
  p.parts = 1 + (p.h_q + p.q_heads - 1) / p.q_heads;
  if (units * p.parts > 2147483647) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(units * p.parts)), block(kAppendThreads);
  const size_t smem = sizeof(float2) * kKvBlock * p.pairs;
  return e4m3 ? launch_dependent(append_kernel<W, TKV, TQ, true>, grid, block, smem, stream, p)
              : launch_dependent(append_kernel<W, TKV, TQ, false>, grid, block, smem, stream, p);
}

template <int W>
static cudaError_t launch_append_width(const AppendParams &p, bool e4m3, bool kv_bf16, bool q_bf16,
                                       cudaStream_t s) {
  using B = __nv_bfloat16;
  if (kv_bf16)
    return q_bf16 ? launch_append_typed<W, B, B>(p, e4m3, s) : launch_append_typed<W, B, float>(p, e4m3, s);
  return q_bf16 ? launch_append_typed<W, float, B>(p, e4m3, s)
                : launch_append_typed<W, float, float>(p, e4m3, s);
}

cudaError_t launch_kv_append(const fathom_kv_append_args *a, const KvBatch &b, cudaStream_t stream) {
  AppendParams p;
  p.b = b;
  p.d = a->cache.d;
  p.h_q = a->q ? a->h_q : 0;
  p.ck = a->cache.k;
  p.cv = a->cache.v;
  p.k_scale = a->cache.k_scale;
  p.v_scale = a->cache.v_scale;
  p.k = a->k;
  p.v = a->v;
  p.q = a->q;
  p.q_out = a->q_out;
  p.k_stride = a->k_stride ? a->k_stride : (int64_t)b.h_kv * p.d;
  p.v_stride = a->v_stride ? a->v_stride : (int64_t)b.h_kv * p.d;
  p.q_stride = a->q_stride ? a->q_stride : (int64_t)a->h_q * p.d;
  p.inv_freq = a->inv_freq;
  p.pairs = a->inv_freq ? a->rotary_pairs : 0;
  p.interleaved = p.pairs ? a->interleaved != 0 : 0;
  // 8 elements a thread at a time where every row and every half of the rotated
  // dimensions starts on 16 bytes; else one at a time
  const bool kv_bf16 = a->kv_dtype == FATHOM_BF16, q_bf16 = a->q_dtype == FATHOM_BF16;
  auto wide = [](const void *ptr, int64_t stride, bool bf16) {
    return ((uintptr_t)ptr & 15) == 0 && stride % (bf16 ? 8 : 4) == 0;
  };
  const bool w8 = wide(p.k, p.k_stride, kv_bf16) && wide(p.v, p.v_stride, kv_bf16) &&
                  (!p.q || (wide(p.q, p.q_stride, q_bf16) && wide(p.q_out, 0, q_bf16))) &&
                  (p.interleaved ? p.pairs % 4 == 0 : p.pairs % 8 == 0);
  const bool e4m3 = a->cache.dtype == FATHOM_E4M3;
  return w8 ? launch_append_width<8>(p, e4m3, kv_bf16, q_bf16, stream)
            : launch_append_width<1>(p, e4m3, kv_bf16, q_bf16, stream);
}

}  // namespace fathom
