// fathom_kv_append: new keys and values into the paged cache, keys and queries
// rotated by their positions on the way.
//
// Row at position p, pair r: angle a = p f_r, (x, y) -> (x cos a - y sin a,
// y cos a + x sin a).  The angle is formed and reduced to half a turn in fp64 (in
// fp32 a position of a million turns by a wrong 0.06), then sincospif.
//
// A unit is the rows of one sequence that fall into one block of 16 positions.
// A thread block works out its sines and cosines once (1024 of them at d = 128),
// keeps them in shared memory and turns every head's rows; units of a few rows are
// spread over several blocks.
//
// An E4M3 cache has a power-of-two scale per block of 16 tokens and KV head, so
// a whole block belongs to one warp: it finds the largest new element, raises
// the scale if it must, moves the codes that the block already held, and writes
// the new ones.  The scale
// comes from the elements before the rotation, which makes it the same whatever
// the sines' last bit, and leaves room for sqrt 2.
//
// Bound by bytes: every element is read and written once.  With 32 query and 8 KV
// heads, d = 128: 8192 rows into bf16 pages 42 us (73% of the copy rate), prompts of
// 5003 to 16384 rows into e4m3 pages 160 us (62%), a decoded row 3 us.  A thread has
// one task of 32 bytes on its way; two ahead (177 us) or prefetches into L2 (171)
// are no faster.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include "kv_cache.cuh"

namespace fathom {

constexpr int kAppendWarps = 8;
constexpr int kAppendThreads = 32 * kAppendWarps;

struct AppendParams {
  KvBatch b;
  int d, h_q;          // (h_q: 0 without queries)
  // a unit's work: q_parts of q_heads query heads each, then kv_parts of K and V; on
  // one thread block (parts = 1) or on one for each part
  int parts, q_parts, q_heads, kv_parts;
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

// cos and sin of p f.  The angle is formed in half turns, in fp64 with the
// product's error carried along, and reduced to [-1, 1].
__device__ __forceinline__ float2 cos_sin(int p, float f) {
  constexpr double kInvPi = 0.31830988618379067;       // 1 / pi
  constexpr double kInvPiLow = -1.9678676675182486e-17;  // 1 / pi less that
  // exact below 2^29; from there on 30 and 24 bits may need one more than fp64 has, and
  // the product is off by 2^-24 at most where f is at most 1
  const double a = (double)p * (double)f;
  const double h = a * kInvPi;
  const double low = fma(a, kInvPi, -h) + a * kInvPiLow;
  const double r = (h - 2.0 * rint(0.5 * h)) + low;
  float s, c;
  sincospif((float)r, &s, &c);
  return make_float2(c, s);
}

// A row's cosines and sines in shared memory: two neighbouring pairs of a task as
// (cos, cos, sin, sin), the operands of two-wide arithmetic; the same two of
// neighbouring tasks are neighbours, so that a warp's 16-byte reads hit different
// banks.
struct Turns {
  int per;    // pairs of a task
  int tasks;  // pairs / per
  int row;    // float4s of a row
  __host__ __device__ Turns(int w, int pairs, int interleaved) {
    per = interleaved && w > 1 ? w / 2 : w;
    tasks = pairs / per;
    row = (per + 1) / 2 * tasks;
  }
  __device__ __forceinline__ void put(float4 *cs, int j, float2 c) const {
    float *at = reinterpret_cast<float *>(cs + j % per / 2 * tasks + j / per) + (j % per & 1);
    at[0] = c.x;
    at[2] = c.y;
  }
};

// Two fp32 operations in one.
__device__ __forceinline__ uint64_t two(float x, float y) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};\n" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;\n" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;\n" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ void split2(uint64_t v, float &x, float &y) {
  asm("mov.b64 {%0, %1}, %2;\n" : "=f"(x), "=f"(y) : "l"(v));
}

// One row's head, rotated: task t of the head is W pairs (interleaved: W / 2), or
// W elements that stay.
template <int W, typename T>
struct Task {
  Vec<T, W> a, b;
};

__host__ __device__ __forceinline__ int turned_tasks(int W, int pairs, int interleaved) {
  return interleaved && W > 1 ? 2 * pairs / W : pairs / W;
}

// FULL: every dimension is in a pair of halves (2 pairs = d, not interleaved), the
// usual case, without the branches of the others.
template <int W, bool FULL, typename T>
__device__ __forceinline__ void load_task(Task<W, T> &x, const T *head, int t, int pairs,
                                          int interleaved) {
  auto at = [&](int i) { return *reinterpret_cast<const Vec<T, W> *>(head + i); };
  if constexpr (FULL) {
    x.a = at(t * W);
    x.b = at(pairs + t * W);
    return;
  }
  const int turned = turned_tasks(W, pairs, interleaved);
  if (t >= turned) {
    x.a = at(2 * pairs + (t - turned) * W);
  } else if (interleaved) {
    if constexpr (W > 1) {
      x.a = at(t * W);
    } else {
      x.a = at(2 * t);
      x.b = at(2 * t + 1);
    }
  } else {
    x.a = at(t * W);
    x.b = at(pairs + t * W);
  }
}

// put(dim, W values) stores the task's elements from dimension dim.  Without cs
// (then not interleaved) they stay as they are.
template <int W, bool FULL, typename T, typename Put>
__device__ __forceinline__ void rotate_task(const Task<W, T> &x, int t, int pairs, int interleaved,
                                            const float4 *cs, Put put) {
  const int turned = FULL ? pairs / W : turned_tasks(W, pairs, interleaved);
  float oa[W], ob[W];
#pragma unroll
  for (int i = 0; i < W; ++i) oa[i] = to_float(x.a.x[i]);
  if (!FULL && t >= turned) {
    put(2 * pairs + (t - turned) * W, oa);
    return;
  }
  if constexpr (W > 1 && !FULL) {
    if (interleaved) {
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const float4 c = cs[i / 4 * turned + t];
        const float u = oa[i], v = oa[i + 1], y = oa[i + 2], z = oa[i + 3];
        oa[i] = u * c.x - v * c.z;
        oa[i + 1] = v * c.x + u * c.z;
        oa[i + 2] = y * c.y - z * c.w;
        oa[i + 3] = z * c.y + y * c.w;
      }
      put(t * W, oa);
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) ob[i] = to_float(x.b.x[i]);
  if (cs) {
    if constexpr (W > 1) {
#pragma unroll
      for (int i = 0; i < W; i += 2) {
        const float4 c = cs[i / 2 * turned + t];
        const uint64_t u = two(oa[i], oa[i + 1]), v = two(ob[i], ob[i + 1]), w = two(-ob[i], -ob[i + 1]);
        const uint64_t cc = two(c.x, c.y), ss = two(c.z, c.w);
        split2(fma2(w, ss, mul2(u, cc)), oa[i], oa[i + 1]);
        split2(fma2(u, ss, mul2(v, cc)), ob[i], ob[i + 1]);
      }
    } else {
      const float4 c = cs[t];
      const float u = oa[0], v = ob[0];
      oa[0] = u * c.x - v * c.z;
      ob[0] = v * c.x + u * c.z;
    }
  }
  const bool beside = !FULL && W == 1 && interleaved;
  put(beside ? 2 * t : t * W, oa);
  put(beside ? 2 * t + 1 : pairs + t * W, ob);
}

// Tasks of one head: pairs W at a time, then the elements that stay.
template <int W>
__host__ __device__ __forceinline__ int rotate_tasks(int d, int pairs, int interleaved) {
  return turned_tasks(W, pairs, interleaved) + (d - 2 * pairs) / W;
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

// The tasks of m rows, `heads` heads each of `per` tasks, dealt out to n threads of
// which this is number i: load(task, row, head, t), then store(task, row, head, t).
// The next task's loads are on their way while this one is worked on (the compiler
// may not move a load over a store that could be to the same place), the first
// one's while `meanwhile` runs.
template <int W, typename T, typename Load, typename Store, typename Meanwhile>
__device__ __forceinline__ void for_tasks(int i, int n, int m, int heads, int per, Load load,
                                          Store store, Meanwhile meanwhile) {
  int t = i % per, h = i / per % heads, r = i / per / heads;
  const int dt = n % per, dh = n / per % heads, dr = n / per / heads;
  Task<W, T> x;
  if (r < m) load(x, r, h, t);
  meanwhile();
  while (r < m) {
    int t2 = t + dt, h2 = h + dh, r2 = r + dr;
    if (t2 >= per) {
      t2 -= per;
      ++h2;
    }
    if (h2 >= heads) {
      h2 -= heads;
      ++r2;
    }
    Task<W, T> y;
    if (r2 < m) load(y, r2, h2, t2);
    store(x, r, h, t);
    x = y;
    t = t2;
    h = h2;
    r = r2;
  }
}

// A sequence's m rows touch at most m / 16 + 2 blocks of positions, so the units
// of sequence s start at q_start[s] / 16 + 2 s.
template <int W, typename TKV, typename TQ, bool E4M3, bool FULL>
__global__ void __launch_bounds__(kAppendThreads, 4) append_kernel(AppendParams p) {
  grid_dependency_wait();
  allow_dependent_launch();
  extern __shared__ float4 cs[];  // [16][Turns::row]
  const int d = p.d;
  const int unit = blockIdx.x / p.parts, part0 = blockIdx.x % p.parts;
  int s = unit, u = 0;
  if (p.b.q_start) {
    auto base = [](int i, int row0) { return (int64_t)(row0 >> 4) + 2 * (int64_t)i; };
    s = find_seq(p.b, unit, base);
    u = (int)(unit - base(s, p.b.q_start[s]));
  }
  const KvSeq q = kv_seq(p.b, s);
  if (u < 0 || u > q.rows / kKvBlock + 1) return;
  const int old = q.len - q.rows;  // tokens that the sequence had (< 0: more rows than tokens)
  // this unit's rows: those whose positions fall into one block of 16
  const int blk = (old >> 4) + u;  // floor: positions below 0 have blocks below 0
  const int p0 = max(blk * kKvBlock, old), p1 = min((blk + 1) * kKvBlock, q.len);
  if (p1 <= p0) return;
  const int row0 = q.row0 + (p0 - old), m = p1 - p0;
  const Turns lay(W, p.pairs, p.interleaved);
  bool have = false;
  auto turns = [&]() {  // the unit's cosines and sines, once
    if (have) return;
    have = true;
    for (int i = threadIdx.x; i < m * p.pairs; i += kAppendThreads) {
      const int r = i / p.pairs, j = i - r * p.pairs;
      lay.put(cs + r * lay.row, j, cos_sin(p0 + r, p.inv_freq[j]));
    }
    __syncthreads();
  };
  auto nothing = []() {};

  for (int part = part0; part < p.q_parts; part += p.parts) {  // queries
    const int h0 = part * p.q_heads, heads = min(p.q_heads, p.h_q - h0);
    const TQ *src = static_cast<const TQ *>(p.q) + (int64_t)row0 * p.q_stride + (int64_t)h0 * d;
    TQ *dst = static_cast<TQ *>(p.q_out) + ((int64_t)row0 * p.h_q + h0) * d;
    for_tasks<W, TQ>(
        threadIdx.x, kAppendThreads, m, heads, rotate_tasks<W>(d, p.pairs, p.interleaved),
        [&](Task<W, TQ> &x, int r, int h, int t) {
          load_task<W, FULL>(x, src + r * p.q_stride + h * d, t, p.pairs, p.interleaved);
        },
        [&](const Task<W, TQ> &x, int r, int h, int t) {
          TQ *out = dst + ((int64_t)r * p.h_q + h) * d;
          rotate_task<W, FULL>(x, t, p.pairs, p.interleaved, cs + r * lay.row,
                         [&](int at, const float *o) { store_vec<W>(out + at, o); });
        },
        turns);
  }
  if (blk < 0) return;
  const int page = kv_page(p.b, s, blk * kKvBlock / p.b.page_tokens);
  if (page < 0) return;
  const int held = p0 - blk * kKvBlock;                         // tokens the block has from before
  const int slot0 = blk * kKvBlock % p.b.page_tokens;           // the block's first row in its page
  const int64_t head0 = (int64_t)page * p.b.h_kv;
  const TKV *k = static_cast<const TKV *>(p.k) + (int64_t)row0 * p.k_stride;
  const TKV *v = static_cast<const TKV *>(p.v) + (int64_t)row0 * p.v_stride;
  const int per_k = rotate_tasks<W>(d, p.pairs, p.interleaved);

  const int kv0 = part0 < p.q_parts ? (p.parts == 1 ? 0 : p.kv_parts) : part0 - p.q_parts;
  if constexpr (!E4M3) {
    if (kv0 >= p.kv_parts) return;
    auto place = [&](void *base, int r, int g) {
      return static_cast<__nv_bfloat16 *>(base) +
             ((head0 + g) * p.b.page_tokens + slot0 + held + r) * d;
    };
    for_tasks<W, TKV>(
        threadIdx.x, kAppendThreads, m, p.b.h_kv, per_k,
        [&](Task<W, TKV> &x, int r, int g, int t) {
          load_task<W, FULL>(x, k + r * p.k_stride + g * d, t, p.pairs, p.interleaved);
        },
        [&](const Task<W, TKV> &x, int r, int g, int t) {
          __nv_bfloat16 *out = place(p.ck, r, g);
          rotate_task<W, FULL>(x, t, p.pairs, p.interleaved, cs + r * lay.row,
                         [&](int at, const float *o) { store_vec<W>(out + at, o); });
        },
        turns);
    for_tasks<W, TKV>(
        threadIdx.x, kAppendThreads, m, p.b.h_kv, d / 2 / W,
        [&](Task<W, TKV> &x, int r, int g, int t) {
          load_task<W, true>(x, v + r * p.v_stride + g * d, t, d / 2, 0);
        },
        [&](const Task<W, TKV> &x, int r, int g, int t) {
          __nv_bfloat16 *out = place(p.cv, r, g);
          rotate_task<W, true>(x, t, d / 2, 0, nullptr,
                               [&](int at, const float *o) { store_vec<W>(out + at, o); });
        },
        nothing);
  } else {
    // a warp per KV head and side: keys first, so that most blocks of values need
    // no turns
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    for (int kv_part = kv0; kv_part < p.kv_parts; kv_part += p.parts) {
      if (kv_part * kAppendWarps < p.b.h_kv) turns();
      const int i = kv_part * kAppendWarps + warp;
      if (i >= 2 * p.b.h_kv) break;
      const bool is_v = i >= p.b.h_kv;
      const int g = is_v ? i - p.b.h_kv : i;
      const int64_t stride = is_v ? p.v_stride : p.k_stride;
      const TKV *src = (is_v ? v : k) + g * d;
      const int64_t head = head0 + g;
      uint8_t *scale = (is_v ? p.v_scale : p.k_scale) + head * (p.b.page_tokens / kKvBlock) +
                       slot0 / kKvBlock;
      uint8_t *codes = static_cast<uint8_t *>(is_v ? p.cv : p.ck) + (head * p.b.page_tokens + slot0) * d;
      uint8_t *out = codes + held * d;
      // values go in pairs of halves too, unturned
      const int pairs = is_v ? d / 2 : p.pairs, inter = is_v ? 0 : p.interleaved;
      const int per = rotate_tasks<W>(d, pairs, inter);
      const int turned = FULL ? per : turned_tasks(W, pairs, inter);
      const bool halves = FULL || W == 1 || !inter;  // a turned task has elements in both halves
      const int was = held ? kv_scale_exp(*scale) + 127 : 0;
      float big = 0.0f;
      auto load = [&](Task<W, TKV> &x, int r, int, int t) {
        load_task<W, FULL>(x, src + r * stride, t, pairs, inter);
      };
      // The largest finite element.  bf16: magnitudes are compared as 16-bit integers,
      // two at a time; infinities and NaNs, which lie above, are rare enough to look
      // for a second time.
      uint32_t top = 0;
      auto largest = [&](const Task<W, TKV> &x, int, int, int t) {
        const bool both = FULL || (halves && t < turned);
        if constexpr (W == 8 && sizeof(TKV) == 2) {
          const uint4 a = *reinterpret_cast<const uint4 *>(&x.a), b = *reinterpret_cast<const uint4 *>(&x.b);
          const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
          if (both)
#pragma unroll
            for (int e = 4; e < 8; ++e) top = __vmaxu2(top, w[e] & 0x7fff7fffu);
        } else {
#pragma unroll
          for (int e = 0; e < W; ++e) {
            const float y = fabsf(to_float(x.a.x[e]));
            if (y < INFINITY) big = fmaxf(big, y);
            if (both) {
              const float z = fabsf(to_float(x.b.x[e]));
              if (z < INFINITY) big = fmaxf(big, z);
            }
          }
        }
      };
      auto finite = [&](const Task<W, TKV> &x, int, int, int t) {
#pragma unroll
        for (int e = 0; e < W; ++e) {
          const float y = fabsf(to_float(x.a.x[e]));
          if (y < INFINITY) big = fmaxf(big, y);
          if (halves && t < turned) {
            const float z = fabsf(to_float(x.b.x[e]));
            if (z < INFINITY) big = fmaxf(big, z);
          }
        }
      };
      // a block whose tasks fit into registers is read once
      constexpr int kKeep = sizeof(TKV) == 2 ? 4 : 2;
      Task<W, TKV> keep[kKeep];
      const bool kept = m * per <= 32 * kKeep;
      if (kept) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
          if (lane + 32 * j < m * per) load(keep[j], (lane + 32 * j) / per, 0, (lane + 32 * j) % per);
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
          if (lane + 32 * j < m * per) largest(keep[j], 0, 0, (lane + 32 * j) % per);
      } else {
        for_tasks<W, TKV>(lane, 32, m, 1, per, load, largest, nothing);
      }
      if constexpr (W == 8 && sizeof(TKV) == 2) {
        top = max(top & 0xffffu, top >> 16);
        if (__any_sync(0xffffffffu, top >= 0x7f80u))
          for_tasks<W, TKV>(lane, 32, m, 1, per, load, finite, nothing);
        else
          big = __uint_as_float(top << 16);
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
      auto store = [&](const Task<W, TKV> &y, int r, int, int t) {
        rotate_task<W, FULL>(y, t, pairs, inter, is_v ? nullptr : cs + r * lay.row, [&](int at, const float *o) {
          uint8_t *to = out + r * d + at;
          if constexpr (W == 8)
            *reinterpret_cast<uint2 *>(to) = make_uint2(pack_e4m3(o[0] * f, o[1] * f, o[2] * f, o[3] * f),
                                                        pack_e4m3(o[4] * f, o[5] * f, o[6] * f, o[7] * f));
          else
            *to = (uint8_t)__nv_cvt_float_to_fp8(o[0] * f, __NV_SATFINITE, __NV_E4M3);
        });
      };
      if (kept) {
#pragma unroll
        for (int j = 0; j < kKeep; ++j)
          if (lane + 32 * j < m * per) store(keep[j], (lane + 32 * j) / per, 0, (lane + 32 * j) % per);
      } else {
        for_tasks<W, TKV>(lane, 32, m, 1, per, load, store, nothing);
      }
      __syncwarp();  // every lane has read the older scale
      if (lane == 0) *scale = (uint8_t)x;
    }
  }
}

template <int W, typename TKV, typename TQ>
static cudaError_t launch_append_typed(AppendParams p, bool e4m3, cudaStream_t stream) {
  const int64_t units = p.b.q_start ? p.b.num_rows / kKvBlock + 2 * (int64_t)p.b.num_seqs : p.b.num_seqs;
  // Units of 16 rows keep a thread block busy, which then works out their sines and
  // cosines once; units of a row or a few are spread out, a task a thread.
  const int rows = p.b.max_rows < kKvBlock ? p.b.max_rows : kKvBlock;
  const bool spread = rows < kKvBlock;
  const int per = rotate_tasks<W>(p.d, p.pairs, p.interleaved);
  int heads = spread ? kAppendThreads / (rows * per) : p.h_q;
  heads = heads > p.h_q ? p.h_q : heads;
  p.q_heads = heads < 1 ? 1 : heads;
  p.q_parts = (p.h_q + p.q_heads - 1) / p.q_heads;
  p.kv_parts = e4m3 ? (2 * p.b.h_kv + kAppendWarps - 1) / kAppendWarps : 1;
  p.parts = spread ? p.q_parts + p.kv_parts : 1;
  if (units * p.parts > 2147483647) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)(units * p.parts)), block(kAppendThreads);
  const size_t smem = sizeof(float4) * kKvBlock * Turns(W, p.pairs, p.interleaved).row;
  if (!p.interleaved && 2 * p.pairs == p.d)
    return e4m3 ? launch_dependent(append_kernel<W, TKV, TQ, true, true>, grid, block, smem, stream, p)
                : launch_dependent(append_kernel<W, TKV, TQ, false, true>, grid, block, smem, stream, p);
  return e4m3 ? launch_dependent(append_kernel<W, TKV, TQ, true, false>, grid, block, smem, stream, p)
              : launch_dependent(append_kernel<W, TKV, TQ, false, false>, grid, block, smem, stream, p);
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
