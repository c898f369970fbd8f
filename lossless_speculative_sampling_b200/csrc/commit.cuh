// commit.cuh -- after a verification: the keys and values of the accepted nodes (the root and the
// accepted path; the drafted block's first nodes in a linear batch) of every layer move to the
// end of their request's context in the paged cache.
#pragma once

#include <stdint.h>

#include "psispec.h"

namespace psi {

constexpr int kCommitThreads = 256;
constexpr int kCommitMaxRows = 1024;  // rows of one request (its root and up to 1023 accepted nodes)
constexpr int kCommitBatch = 4;       // 16-byte copies in flight per thread

// One CTA copies one request's rows of one layer, keys (blockIdx.y even) or values. Every row's
// source and destination is checked before any is copied, by every CTA alike, so a request with
// a bad argument is left alone in all layers. Each moved byte is read and written once. Measured on
// a B200: 64 requests, 8 layers, up to 16 rows of 8 heads of 128 bf16 10.8 us, one request 2.7 us, of
// which the checks' chain of dependent loads (offsets, path, pages) is the larger part.
__global__ void __launch_bounds__(kCommitThreads) commit_tree_kernel(const __grid_constant__ psispec_commit_tree_args a) {
  __shared__ int64_t src[kCommitMaxRows], dst[kCommitMaxRows];
  const int b = blockIdx.x, layer = blockIdx.y >> 1, kv = blockIdx.y & 1;
  const int lo = __ldg(a.node_offsets + b), hi = __ldg(a.node_offsets + b + 1);
  const int acc = __ldg(a.accept_len + b), ctx = __ldg(a.context_len + b);
  const int64_t room = int64_t(a.max_pages) * a.page_size;
  const bool first = blockIdx.y == 0 && threadIdx.x == 0;
  bool ok = lo >= 0 && hi >= lo && hi <= a.N && ctx >= 0 && ctx <= room;
  if (ok && acc == -1) {  // the verification reported a data error: nothing was accepted
    if (first) a.out_context_len[b] = ctx;
    return;
  }
  // (the accepted length before what is counted from it: the largest int has no successor)
  ok = ok && acc >= 0 && acc < hi - lo && acc < kCommitMaxRows && (a.path == nullptr || acc <= a.max_depth) &&
       ctx + int64_t(acc) < room;
  const int rows = ok ? acc + 1 : 0;
  if (ok) {
    const int64_t* ns = kv ? a.vn_stride : a.kn_stride;
    const int64_t* cs = kv ? a.vc_stride : a.kc_stride;
    for (int r = threadIdx.x; r < rows; r += kCommitThreads) {
      const int node = r == 0 ? 0 : (a.path ? __ldg(a.path + int64_t(b) * a.max_depth + r - 1) : r);
      const int pos = ctx + r;
      const int page = __ldg(a.page_table + int64_t(b) * a.max_pages + pos / a.page_size);
      const bool good = node >= 0 && node < hi - lo && page >= 0 && page < a.pages;
      ok = ok && good;
      if (good) {
        src[r] = layer * ns[0] + (int64_t(lo) + node) * ns[1];
        dst[r] = layer * cs[0] + page * cs[1] + (pos % a.page_size) * cs[2];
      }
    }
  }
  if (!__syncthreads_and(ok)) {
    if (first) a.out_context_len[b] = -1;
    return;
  }
  const uint16_t* from = static_cast<const uint16_t*>(kv ? a.v_nodes : a.k_nodes);
  uint16_t* to = static_cast<uint16_t*>(kv ? a.v_cache : a.k_cache);
  const int64_t fh = kv ? a.vn_stride[2] : a.kn_stride[2], th = kv ? a.vc_stride[3] : a.kc_stride[3];
  const int per_head = a.D / 8, per_row = a.Hkv * per_head;
  const int total = rows * per_row;
  for (int i0 = threadIdx.x; i0 < total; i0 += kCommitThreads * kCommitBatch) {
    uint4 v[kCommitBatch];
    uint16_t* at[kCommitBatch];
#pragma unroll
    for (int t = 0; t < kCommitBatch; ++t) {
      const int i = i0 + t * kCommitThreads;
      if (i >= total) break;
      const int r = i / per_row, h = (i % per_row) / per_head, c = (i % per_head) * 8;
      v[t] = __ldg(reinterpret_cast<const uint4*>(from + src[r] + h * fh + c));
      at[t] = to + dst[r] + h * th + c;
    }
#pragma unroll
    for (int t = 0; t < kCommitBatch; ++t) {
      if (i0 + t * kCommitThreads >= total) break;
      *reinterpret_cast<uint4*>(at[t]) = v[t];
    }
  }
  if (first) a.out_context_len[b] = ctx + rows;
}

}  // namespace psi
