// Attention over the paged cache: parameters and what its kernels share.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace fathom {

// The many-rows kernel's unit: one or two tiles of 128 columns, against 128 keys at
// a time.
constexpr int prompt_cols(int d) { return d <= 128 ? 256 : 128; }
constexpr int kPromptTile = 128;

// From many_from columns (rows times heads of a KV head) on a sequence goes to the
// many-rows kernel.
enum KvOwn { kEverySequence = 0, kFewRows = 1, kManyRows = 2 };

// What a block of the many-rows kernel leaves for the kernel that does units again:
// do this one again, since a value of V that some row does not see is not finite; or
// since a wait ran out, which is a device fault as well.
constexpr int kMarkAgain = 1, kMarkLate = 2;

struct KvAttnParams {
  KvBatch b;
  const void *ck, *cv;
  const uint8_t *k_scale, *v_scale;
  const void *q;
  int64_t q_stride;
  int q_bf16;  // and out's type
  int q_wide, out_wide;  // 16-byte accesses of q's and out's rows are aligned
  int h_q, G, d;
  float qscale;       // softmax scale * log2(e)
  int window, sinks;  // window: above max_len where there is none
  void *out;
  float *lse;
  // The plan (plan_kv_attention) and the workspace.  A unit of work is `cols`
  // (token, head) pairs of one sequence and KV head; it goes through its keys in
  // tiles of `tile`, divided over `splits` thread blocks.
  int many_rows;  // the tcgen05 kernel
  int own;        // 0: every sequence; kFewRows, kManyRows: those with fewer than
                  // many_from columns, the others
  int many_from;
  int report;     // this launch writes the status
  int cols, tile;
  // Units of one KV head: `dense`, col_tiles for each sequence; else sequence s
  // starts at unit q_start[s] G / cols + s (it needs no more than it has there).
  int units, dense, col_tiles;
  int tiles_per_split, splits;
  int cluster;  // few rows: a unit's splits are a cluster
  // many_rows: the (sequence, KV head) pairs of one launch; the units in order of
  // work from which on they are divided (the others are not); the rows of a K or V
  // box; e4m3: keys of a pair in the widened copy, the tiles that its rows see (KvTiles'
  // order) one behind the other (0: there is none)
  int pair0, pairs, tail_from, box_rows, n_pad;
  const uint16_t *wide;  // [2][pairs][n_pad][d] bf16
  WsStatus *status;
  int *taint;       // many_rows: [units * h_kv][splits] marks (kMarkAgain, kMarkLate)
  // of the units from tail_from on, if they are divided and no cluster: [unit]
  // [split][part_cols], part_cols the most columns that a unit has
  int part_cols;
  float2 *part_ml;  // maximum (log2 units), sum
  float *part_o;    // [d] each
};

__device__ __forceinline__ bool owns(const KvAttnParams &a, const KvSeq &q) {
  return a.own == kEverySequence || (q.rows * a.G >= a.many_from) == (a.own == kManyRows);
}

// Unit y of a KV head: its sequence and which of the sequence's units it is.
struct KvUnit {
  int s, ct;
};

__device__ __forceinline__ KvUnit kv_unit(const KvAttnParams &a, int y) {
  if (a.dense) return {y / a.col_tiles, y % a.col_tiles};
  auto base = [&](int i, int row0) { return (int64_t)row0 * a.G / a.cols + i; };
  const int s = find_seq(a.b, y, base);
  const int64_t ct = y - base(s, a.b.q_start[s]);
  return {s, ct < 0 || ct >= a.col_tiles ? a.col_tiles : (int)ct};  // (col_tiles: none)
}

// Where split `split` of unit `unit` (of all KV heads') leaves its result for column 0.
__device__ __forceinline__ int64_t part_at(const KvAttnParams &a, int unit, int split) {
  return ((int64_t)(unit - a.tail_from) * a.splits + split) * a.part_cols;
}

// Whether a row at position p sees token j.
__device__ __forceinline__ bool sees(const KvAttnParams &a, int p, int j) {
  return j <= p && (j > p - a.window || j < a.sinks);
}

// The tiles of `tile` keys that rows at positions p_lo .. p_hi can see: those of
// the first `sinks` tokens, then, `skip` tiles further on, the windows'.
struct KvTiles {
  int count, sink_tiles, skip;
  __device__ __forceinline__ int at(int i) const { return i < sink_tiles ? i : i + skip; }
  // which one tile t is, of these rows' or of some of them alone
  __device__ __forceinline__ int index(int t) const { return t < sink_tiles ? t : t - skip; }
};

__device__ __forceinline__ KvTiles visible_tiles(const KvAttnParams &a, int p_lo, int p_hi,
                                                 int tile) {
  KvTiles x;
  const int end = p_hi < 0 ? 0 : p_hi / tile + 1;
  const int from = max(p_lo - a.window + 1, 0) / tile;
  const int sink = (int)min(((int64_t)a.sinks + tile - 1) / tile, (int64_t)end);
  x.sink_tiles = min(sink, from);
  x.skip = from - x.sink_tiles;
  x.count = max(end - x.skip, 0);
  return x;
}

// Whether every row at positions p_lo .. p_hi sees all of key0 .. key0 + tile - 1.
__device__ __forceinline__ bool sees_all(const KvAttnParams &a, int p_lo, int p_hi, int key0,
                                         int tile) {
  return key0 + tile - 1 <= p_lo && (key0 + tile <= a.sinks || key0 > p_hi - a.window);
}

__device__ __forceinline__ void store_out(const KvAttnParams &a, int64_t at, float x) {
  if (a.q_bf16)
    static_cast<__nv_bfloat16 *>(a.out)[at] = __float2bfloat16_rn(x);
  else
    static_cast<float *>(a.out)[at] = x;
}

// log of the sum of exp(s), from the sum l of 2^(s' - m + shift), s' = s log2 e.
__device__ __forceinline__ float lse_of(float m, float l, float shift) {
  return l == 0.0f ? -INFINITY : (m + log2f(l) - shift) * 0.6931471805599453f;
}

// The last block of a launch counts the sequences that break the batch's
// bounds into the workspace's status.  (Nothing else of that launch may write there:
// its other blocks come before or after this one in no particular order.)
__device__ __forceinline__ void write_status(const KvAttnParams &a) {
  __shared__ int bad;
  if (threadIdx.x == 0) bad = 0;
  __syncthreads();
  int n = 0;
  for (int s = threadIdx.x; s < a.b.num_seqs; s += blockDim.x) n += !kv_seq(a.b, s).valid;
  if (n) atomicAdd(&bad, n);
  __syncthreads();
  if (threadIdx.x == 0) {
    a.status->fallback_heads = 0;
    a.status->device_faults = (uint32_t)bad;
    a.status->max_candidates = 0;
    a.status->union_planes = 0;
  }
}

// kv_attention.cu
cudaError_t launch_kv_status(const KvAttnParams &a, cudaStream_t s);  // a call without rows
cudaError_t launch_kv_attention(const KvAttnParams &a, bool f8, cudaStream_t s);
// The launches of one call, one or two (long and short sequences apart), into plan.
int plan_kv_attention(const KvAttnParams &a, bool f8, KvAttnParams (&plan)[2]);
// kv_prompt.cu: the tcgen05 kernel, and the widening before it
cudaError_t launch_kv_prompt(const KvAttnParams &a, bool f8, cudaStream_t s);

}  // namespace fathom
