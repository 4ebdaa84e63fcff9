// The paged KV cache as the kernels see it: parameters, and the checks of the
// batch's device arrays that every kernel makes in the same way.
#pragma once

#include "fathom_internal.cuh"

namespace fathom {

constexpr int kKvBlock = FATHOM_KV_BLOCK;

struct KvBatch {
  const int32_t *page_table;
  const int32_t *seq_len;
  const int32_t *q_start;  // NULL: row s is sequence s's one row
  int num_seqs, table_width, num_rows, max_rows;
  int max_len;
  int num_pages, page_tokens, h_kv;
};

// One sequence's rows and tokens, as far as they keep the batch's bounds.
struct KvSeq {
  int row0;    // its first row
  int rows;    // new tokens (0 where its rows break the bounds)
  int len;     // tokens in all, the rows included (0 where it breaks the bounds)
  bool valid;  // it kept every bound
};

// Rows r0 .. r1 - 1 keep the batch's bounds.
__device__ __forceinline__ bool kv_rows_ok(const KvBatch &b, int r0, int r1) {
  return r0 >= 0 && r1 >= r0 && r1 <= b.num_rows && r1 - r0 <= b.max_rows;
}

__device__ __forceinline__ KvSeq kv_seq(const KvBatch &b, int s) {
  KvSeq q;
  const int n = b.seq_len[s];
  const bool n_ok = n >= 0 && n <= b.max_len;
  q.len = n_ok ? n : 0;
  q.row0 = s;
  q.rows = 1;
  bool r_ok = true;
  if (b.q_start) {
    const int r0 = b.q_start[s], r1 = b.q_start[s + 1];
    r_ok = kv_rows_ok(b, r0, r1);
    q.row0 = r_ok ? r0 : 0;
    q.rows = r_ok ? r1 - r0 : 0;
  }
  q.valid = n_ok && r_ok;
  return q;
}

// The page of the block of tokens from `token` on; -1 where it holds nothing.
__device__ __forceinline__ int kv_page(const KvBatch &b, int s, int page_at) {
  if (page_at >= b.table_width) return -1;
  const int page = __ldg(b.page_table + (int64_t)s * b.table_width + page_at);
  return page >= 0 && page < b.num_pages ? page : -1;
}

// The exponent of a block's scale.
__device__ __forceinline__ int kv_scale_exp(uint32_t x) {
  return (int)min(max(x, (uint32_t)FATHOM_KV_SCALE_MIN), (uint32_t)FATHOM_KV_SCALE_MAX) - 127;
}

// 2^e for -126 <= e <= 127.
__device__ __forceinline__ float exp2i(int e) { return __int_as_float((e + 127) << 23); }

// The sequence that unit `x` belongs to, where sequence s starts at unit
// start(s, q_start[s]): the last one that starts at x or before, of those whose rows
// keep the bounds.  These start one behind the other as long as their rows do; what the
// others' entries hold does not matter.  The lanes of a warp look at 32 places at once;
// where a place on the way is one of the others, at every sequence in turn.
template <typename Start>
__device__ __forceinline__ int find_seq(const KvBatch &b, int64_t x, Start start) {
  constexpr uint32_t kAll = 0xffffffffu;
  const int lane = threadIdx.x & 31;
  bool ok;
  auto starts_by = [&](int s) {  // (s past the last: no)
    ok = true;
    if (s >= b.num_seqs) return false;
    const int r0 = b.q_start[s], r1 = b.q_start[s + 1];
    ok = kv_rows_ok(b, r0, r1);
    return ok && start(s, r0) <= x;
  };
  int lo = 0, n = b.num_seqs;  // the answer is in [lo, lo + n)
  while (n > 1) {
    const int step = (n + 31) / 32;
    const bool inside = lane * step < n;
    const bool le = starts_by(inside ? lo + lane * step : b.num_seqs);
    if (step > 1 && !__all_sync(kAll, ok)) {
      lo = 0;
      for (int s = 0; s < b.num_seqs; s += 32) {
        const uint32_t m = __ballot_sync(kAll, starts_by(s + lane));
        if (m) lo = s + 31 - __clz((int)m);
      }
      return lo;
    }
    const uint32_t m = __ballot_sync(kAll, le);
    const int last = m ? 31 - __clz((int)m) : 0;
    n = min(step, n - last * step);
    lo += last * step;
  }
  return lo;
}

}  // namespace fathom
