// Eviction from the cache: which tokens a budget keeps, and their rows moved together.
//
// Selection. A sequence of L tokens falls to L' = L - ceil((L - budget) / span) * span
// (span = dcp * interleave), so every rank drops the same number of tokens and what is
// left lies as a sequence of L' tokens lies. On a rank, m of the tokens between the
// protected head and tail stay: the threshold T, the m-th largest weight, is found by its
// bits from the top, and a token stays if its weight is above T, or equal to T with fewer
// than (m - number above T) equal ones before it.
//
// Compaction. keep_idx ascends, so row i comes from a row at or behind i: in place, a row
// can be written once the rows that come from it or from before it have been read.
#include <algorithm>

#include "common.cuh"

namespace dcpmla {
namespace {

constexpr int kSelThreads = 1024;

// Weights as unsigned keys in their order: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  if (isnan(w)) w = -INFINITY;
  const uint32_t u = __float_as_uint(w + 0.0f);
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Inclusive sum over the block of one value per thread; every thread also gets the total.
__device__ __forceinline__ int block_scan(int v, int* total, int* scratch) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += y;
  }
  if (lane == 31) scratch[warp] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    if (w < warp) before += scratch[w];
    all += scratch[w];
  }
  __syncthreads();
  *total = all;
  return v + before;
}

__global__ void __launch_bounds__(kSelThreads)
evict_select_kernel(int batch, int dcp, int interleave, int max_local_len, int budget, int sink,
                    int recent, int max_keep, int rank_begin,
                    const int32_t* __restrict__ seq_lens, const float* __restrict__ weights,
                    int32_t* __restrict__ keep_idx, int32_t* __restrict__ keep_count,
                    int32_t* __restrict__ new_lens, uint32_t* status) {
  const int b = blockIdx.x, k = blockIdx.y, rank = rank_begin + k;
  __shared__ int hist[256];
  __shared__ int scratch[kSelThreads / 32];
  __shared__ uint32_t s_prefix;
  __shared__ int s_left;
  int64_t L = seq_lens[b];
  const int64_t span = (int64_t)dcp * interleave;
  const int64_t n64 = local_len(L, rank, span, interleave);
  // over the bound on any rank (rank 0 holds the most): the sequence gets no tokens
  if (L < 0 || local_len(L, 0, span, interleave) > max_local_len) {
    if (threadIdx.x == 0)
      raise_status(status, L < 0 ? DCP_STATUS_BAD_SEQ_LEN : DCP_STATUS_LOCAL_OVER_BOUND);
    L = 0;
  }
  const int64_t L2 = L > budget ? L - (L - budget + span - 1) / span * span : L;
  const int n = L > 0 ? (int)n64 : 0;
  const int kept = (int)local_len(L2, rank, span, interleave);
  const float* w = weights + ((int64_t)k * batch + b) * max_local_len;
  int32_t* idx = keep_idx + ((int64_t)k * batch + b) * max_keep;
  if (threadIdx.x == 0) {
    keep_count[(int64_t)k * batch + b] = kept;
    if (k == 0) new_lens[b] = (int32_t)L2;
  }
  for (int i = kept + threadIdx.x; i < max_keep; i += kSelThreads) idx[i] = -1;
  if (kept == n) {
    for (int i = threadIdx.x; i < n; i += kSelThreads) idx[i] = i;
    return;
  }
  const int beg = sink, end = n - recent;
  const int m = kept - sink - recent;  // of the tokens in [beg, end)
  // the m-th largest key, eight bits at a time
  if (threadIdx.x == 0) {
    s_prefix = 0;
    s_left = m;
  }
  for (int shift = 24; shift >= 0; shift -= 8) {
    if (threadIdx.x < 256) hist[threadIdx.x] = 0;
    __syncthreads();
    const uint32_t prefix = s_prefix;
    for (int t = beg + threadIdx.x; t < end; t += kSelThreads) {
      const uint32_t key = weight_key(w[t]);
      if (shift == 24 || (key >> (shift + 8)) == (prefix >> (shift + 8)))
        atomicAdd(&hist[(key >> shift) & 255], 1);
    }
    __syncthreads();
    if (threadIdx.x == 0) {
      int left = s_left, d = 255;
      while (d > 0 && hist[d] < left) left -= hist[d--];
      s_left = left;
      s_prefix = prefix | ((uint32_t)d << shift);
    }
    __syncthreads();
  }
  const uint32_t T = m > 0 ? s_prefix : 0xffffffffu;
  const int equal = m > 0 ? s_left : 0;  // of the tokens at T, the first `equal` stay
  int done = 0, seen = 0;
  for (int t0 = 0; t0 < n; t0 += kSelThreads) {
    const int t = t0 + threadIdx.x;
    bool stay = t < n && (t < beg || t >= end);
    bool at = false;
    if (t >= beg && t < end) {
      const uint32_t key = weight_key(w[t]);
      stay = key > T;
      at = key == T;
    }
    int total;
    const int rank_at = block_scan(at, &total, scratch);
    if (at && seen + rank_at <= equal) stay = true;
    seen += total;
    const int place = block_scan(stay, &total, scratch);
    if (stay) idx[done + place - 1] = t;
    done += total;
  }
}

// ------------------------------------------------------------------ compaction

constexpr int kMoveThreads = 256;
constexpr int kMoveRows = 8;                    // rows per thread and round
constexpr int kMovePieces = 4;                  // 16-byte pieces of a row per CTA
constexpr int kMoveTile = kMoveThreads / kMovePieces * kMoveRows;

// One CTA walks the rows of one (rank, sequence) in order, kMovePieces 16-byte pieces of
// each: a round's rows are all read before the first of them is written, and every later
// round reads behind what this one writes, which is all that in place needs.
__global__ void __launch_bounds__(kMoveThreads)
kv_move_kernel(int batch, int block_size, int max_blocks, int64_t num_blocks, int max_keep,
               int row_pieces, const int32_t* __restrict__ keep_idx,
               const int32_t* __restrict__ keep_count, const int32_t* src_table,
               const int32_t* dst_table, uint4* pool, uint32_t* status) {
  const int b = blockIdx.x, k = blockIdx.y;
  const int piece = blockIdx.z * kMovePieces + threadIdx.x % kMovePieces;
  int n = keep_count[(int64_t)k * batch + b];
  uint32_t bad = 0;
  if (n < 0 || n > max_keep) {
    bad = DCP_STATUS_BAD_PAGE;
    n = 0;
  }
  const bool same = src_table == dst_table;
  const int32_t* idx = keep_idx + ((int64_t)k * batch + b) * max_keep;
  const int32_t* src = src_table + (int64_t)b * max_blocks;
  const int32_t* dst = dst_table + (int64_t)b * max_blocks;
  const int64_t limit = (int64_t)max_blocks * block_size;
  uint4* base = pool + (int64_t)k * num_blocks * block_size * row_pieces;
  for (int r0 = 0; r0 < n; r0 += kMoveTile) {
    uint4 v[kMoveRows];
    int64_t to[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int i = r0 + u * (kMoveThreads / kMovePieces) + threadIdx.x / kMovePieces;
      to[u] = -1;
      if (i >= n || piece >= row_pieces) continue;
      const int64_t t = idx[i];
      if (t < i || t >= limit || i >= limit) {
        bad |= DCP_STATUS_BAD_PAGE;
        continue;
      }
      if (same && t == i) continue;
      const int sb = src[t / block_size], db = dst[i / block_size];
      if (sb < 0 || sb >= num_blocks || db < 0 || db >= num_blocks) {
        bad |= DCP_STATUS_BAD_BLOCK_ID;
        continue;
      }
      v[u] = base[((int64_t)sb * block_size + t % block_size) * row_pieces + piece];
      to[u] = ((int64_t)db * block_size + i % block_size) * row_pieces + piece;
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (to[u] >= 0) base[to[u]] = v[u];
  }
  if (bad) raise_status(status, bad);
}

// The weights of one (rank, sequence), moved the same way.
__global__ void __launch_bounds__(kMoveThreads)
weight_move_kernel(int batch, int max_keep, int max_local_len,
                   const int32_t* __restrict__ keep_idx, const int32_t* __restrict__ keep_count,
                   const float* w_in, float* w_out) {
  const int b = blockIdx.x, k = blockIdx.y;
  const int n = keep_count[(int64_t)k * batch + b];
  if (n < 0 || n > max_keep) return;  // reported by kv_move_kernel
  const int32_t* idx = keep_idx + ((int64_t)k * batch + b) * max_keep;
  const float* from = w_in + ((int64_t)k * batch + b) * max_local_len;
  float* to = w_out + ((int64_t)k * batch + b) * max_local_len;
  for (int r0 = 0; r0 < n; r0 += kMoveThreads * kMoveRows) {
    float v[kMoveRows];
    bool ok[kMoveRows];
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u) {
      const int i = r0 + u * kMoveThreads + threadIdx.x;
      ok[u] = false;
      if (i >= n) continue;
      const int t = idx[i];
      ok[u] = t >= i && t < max_local_len;
      if (ok[u]) v[u] = from[t];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kMoveRows; ++u)
      if (ok[u]) to[r0 + u * kMoveThreads + threadIdx.x] = v[u];
  }
}

}  // namespace

cudaError_t launch_evict_select(const dcp_mla_dims& d, const int32_t* seq_lens,
                                const float* weights, int budget, int sink, int recent,
                                int max_keep, int rank_begin, int num_ranks, int32_t* keep_idx,
                                int32_t* keep_count, int32_t* new_lens, uint32_t* status,
                                cudaStream_t stream) {
  const dim3 grid((unsigned)d.batch, (unsigned)num_ranks);
  evict_select_kernel<<<grid, kSelThreads, 0, stream>>>(
      d.batch, d.dcp, d.interleave, d.max_local_len, budget, sink, recent, max_keep, rank_begin,
      seq_lens, weights, keep_idx, keep_count, new_lens, status);
  return cudaGetLastError();
}

cudaError_t launch_kv_compact(const dcp_mla_dims& d, int row_bytes, const int32_t* keep_idx,
                              const int32_t* keep_count, int max_keep, const int32_t* src_table,
                              const int32_t* dst_table, int num_ranks, void* pool,
                              const float* weights_in, float* weights_out, uint32_t* status,
                              cudaStream_t stream) {
  const int pieces = row_bytes / 16;
  const dim3 grid((unsigned)d.batch, (unsigned)num_ranks,
                  (unsigned)((pieces + kMovePieces - 1) / kMovePieces));
  kv_move_kernel<<<grid, kMoveThreads, 0, stream>>>(
      d.batch, d.block_size, d.max_blocks_per_seq, d.num_blocks, max_keep, pieces, keep_idx,
      keep_count, src_table, dst_table, static_cast<uint4*>(pool), status);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || weights_in == nullptr) return e;
  weight_move_kernel<<<dim3(grid.x, grid.y), kMoveThreads, 0, stream>>>(
      d.batch, max_keep, d.max_local_len, keep_idx, keep_count, weights_in, weights_out);
  return cudaGetLastError();
}

}  // namespace dcpmla
