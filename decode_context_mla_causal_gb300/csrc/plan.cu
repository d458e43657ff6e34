// A step's pages: block tables, free blocks, slots, positions and row offsets from the lengths
// that requests have and are to have.
//
// Latency-bound: a few integers per request and 4 (ranks + 1) bytes per new token. One launch:
// every CTA forms the running sums over the requests (new rows, blocks needed, blocks given
// back) for itself in shared memory, and from there on every table entry, list entry and new
// token is found by a binary search in them, independent of every other. The n-th block handed
// out is the n-th one given back, read from its old table entry (a request that shrinks has no
// entry written), or free_list's n-th from the end (which the call writes only from *free_count
// on), so nothing that is read is written, but lengths and count: the CTA that ends last, by a
// ticket, writes those. Measured: 64 requests with a token each on 8 ranks 7.9 us, 192 requests with
// up to 4096 new tokens each on 4 ranks 11.3 us (floors 0.001 and 0.26): what bounds it is the chain
// of loads, sums over three barriers and searches, and some five 64-bit divisions a request in each
// of four passes.
#include <algorithm>

#include "common.cuh"

namespace dcpmla {
namespace {

constexpr int kPlanThreads = 256;
constexpr int kPlanMaxBatch = 16384;

struct PlanParams {
  const int32_t* targets;
  const int32_t* seq_lens;
  int32_t* new_lens;
  int32_t* block_table;
  int32_t* free_list;
  const int32_t* free_count;
  int32_t* new_count;
  int32_t* slot_mapping;
  int32_t* positions;
  int32_t* cu_rows;
  uint32_t* ticket;
  uint32_t* status;
  int batch, dcp, interleave, block_size, max_blocks, max_local_len, num_blocks, rank_begin,
      num_ranks, max_rows;
};

__device__ __forceinline__ int local0(const PlanParams& p, int g) {
  return (int)local_len(g, 0, (int64_t)p.dcp * p.interleave, p.interleave);
}
__device__ __forceinline__ int blocks_of(const PlanParams& p, int g) {
  return (int)(((int64_t)local0(p, g) + p.block_size - 1) / p.block_size);
}
// What a request asks for: new rows, blocks to take, blocks to give back.
struct Ask {
  int rows, need, freed;
};
__device__ __forceinline__ Ask ask_of(const PlanParams& p, int len, int target, uint32_t& bad) {
  Ask a = {0, 0, 0};
  if (len < 0 || target < 0) {
    bad |= DCP_STATUS_BAD_SEQ_LEN;
  } else if (local0(p, max(len, target)) > p.max_local_len) {
    bad |= DCP_STATUS_LOCAL_OVER_BOUND;
  } else {
    const int d = blocks_of(p, target) - blocks_of(p, len);
    a.rows = max(0, target - len);
    a.need = max(0, d);
    a.freed = max(0, -d);
  }
  return a;
}
// First index whose running sum is above x, of n (n where there is none).
__device__ __forceinline__ int find_end(const int* ends, int n, int x) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (ends[mid] > x) hi = mid;
    else lo = mid + 1;
  }
  return lo;
}

struct Sum3 {
  int64_t rows, need, freed;
};

__global__ void __launch_bounds__(kPlanThreads) plan_kernel(const PlanParams p) {
  extern __shared__ int s_ends[];  // [3][batch]: rows, blocks taken, blocks given back
  __shared__ Sum3 s_warp[kPlanThreads / 32];
  __shared__ int64_t s_most[2][kPlanThreads / 32];
  __shared__ int s_last;
  int* const row_end = s_ends;
  int* const need_end = s_ends + p.batch;
  int* const freed_end = s_ends + 2 * p.batch;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  uint32_t bad = 0;
  int count = *p.free_count;
  if (count < 0 || count > p.num_blocks) {
    bad |= DCP_STATUS_BAD_PAGE;
    count = max(0, min(count, p.num_blocks));
  }
  // running sums: a thread takes `each` requests in a row
  const int each = (p.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(p.batch, tid * each), b1 = min(p.batch, b0 + each);
  Sum3 mine = {0, 0, 0};
  for (int b = b0; b < b1; ++b) {
    const Ask a = ask_of(p, p.seq_lens[b], p.targets[b], bad);
    mine.rows += a.rows;
    mine.need += a.need;
    mine.freed += a.freed;
  }
  Sum3 x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t r = __shfl_up_sync(0xffffffffu, x.rows, o);
    const int64_t n = __shfl_up_sync(0xffffffffu, x.need, o);
    const int64_t f = __shfl_up_sync(0xffffffffu, x.freed, o);
    if (lane >= o) x.rows += r, x.need += n, x.freed += f;
  }
  if (lane == 31) s_warp[warp] = x;
  __syncthreads();
  Sum3 at = {x.rows - mine.rows, x.need - mine.need, x.freed - mine.freed};
  int64_t given_back = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) at.rows += s_warp[w].rows, at.need += s_warp[w].need, at.freed += s_warp[w].freed;
    given_back += s_warp[w].freed;
  }
  const int freed = (int)given_back;  // a table holds them: batch * max_blocks_per_seq < 2^31
  // the requests that fit are those before the first that does not: their last sums
  int64_t rows_most = 0, need_most = 0;
  bool held_back = false;
  {
    Sum3 c = at;
    for (int b = b0; b < b1; ++b) {
      uint32_t again = 0;
      const Ask a = ask_of(p, p.seq_lens[b], p.targets[b], again);
      c.rows += a.rows;
      c.need += a.need;
      c.freed += a.freed;
      if (c.need <= count + given_back && c.rows <= p.max_rows)
        rows_most = c.rows, need_most = c.need;
      else if (a.rows > 0)
        held_back = true;
      freed_end[b] = (int)c.freed;
    }
  }
  if (held_back) bad |= DCP_STATUS_HELD_BACK;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    rows_most = max(rows_most, __shfl_xor_sync(0xffffffffu, rows_most, o));
    need_most = max(need_most, __shfl_xor_sync(0xffffffffu, need_most, o));
  }
  if (lane == 0) s_most[0][warp] = rows_most, s_most[1][warp] = need_most;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    rows_most = max(rows_most, s_most[0][w]);
    need_most = max(need_most, s_most[1][w]);
  }
  const int rows = (int)rows_most, taken = (int)need_most;
  {
    Sum3 c = at;
    for (int b = b0; b < b1; ++b) {
      uint32_t again = 0;
      const Ask a = ask_of(p, p.seq_lens[b], p.targets[b], again);
      c.rows += a.rows;
      c.need += a.need;
      row_end[b] = (int)min(c.rows, rows_most);
      need_end[b] = (int)min(c.need, need_most);
      if (blockIdx.x == 0) p.cu_rows[b + 1] = row_end[b];
    }
  }
  if (blockIdx.x == 0 && tid == 0) p.cu_rows[0] = 0;
  __syncthreads();

  // the n-th block handed out
  auto nth = [&](int n) -> int32_t {
    if (n >= freed) return p.free_list[count - 1 - (n - freed)];
    const int b = find_end(freed_end, p.batch, n);
    const int before = b > 0 ? freed_end[b - 1] : 0;
    return p.block_table[(int64_t)b * p.max_blocks + blocks_of(p, p.targets[b]) + n - before];
  };
  const int step = gridDim.x * kPlanThreads, first = blockIdx.x * kPlanThreads + tid;
  // table entries
  for (int n = first; n < taken; n += step) {
    const int b = find_end(need_end, p.batch, n);
    const int at_block = blocks_of(p, p.seq_lens[b]) + n - (b > 0 ? need_end[b - 1] : 0);
    const int32_t id = nth(n);
    if (id < 0 || id >= p.num_blocks) bad |= DCP_STATUS_BAD_BLOCK_ID;
    p.block_table[(int64_t)b * p.max_blocks + at_block] = id;
  }
  // what is not handed out goes onto the list, the last one first
  for (int i = first; i < freed - taken; i += step) {
    if (count + i >= p.num_blocks) {
      bad |= DCP_STATUS_BAD_PAGE;
      continue;
    }
    const int32_t id = nth(freed - 1 - i);
    if (id < 0 || id >= p.num_blocks) bad |= DCP_STATUS_BAD_BLOCK_ID;
    p.free_list[count + i] = id;
  }
  // new tokens
  for (int t = first; t < p.max_rows; t += step) {
    int owner = -1, pos = 0;
    int32_t slot = -1;
    if (t < rows) {
      const int b = find_end(row_end, p.batch, t);
      const int len = p.seq_lens[b];
      pos = len + t - (b > 0 ? row_end[b - 1] : 0);
      const unsigned chunk = (unsigned)pos / (unsigned)p.interleave;
      const unsigned turn = chunk / (unsigned)p.dcp;
      owner = (int)(chunk - turn * p.dcp) - p.rank_begin;
      const int li = (int)turn * p.interleave + (int)(pos - chunk * p.interleave);
      const int blk = li / p.block_size, held = blocks_of(p, len);
      const int32_t id = blk < held
                             ? p.block_table[(int64_t)b * p.max_blocks + blk]
                             : nth((b > 0 ? need_end[b - 1] : 0) + blk - held);
      if (id >= 0 && id < p.num_blocks) slot = id * p.block_size + (li - blk * p.block_size);
      else bad |= DCP_STATUS_BAD_BLOCK_ID;
    }
    p.positions[t] = pos;
    for (int k = 0; k < p.num_ranks; ++k)
      p.slot_mapping[(int64_t)k * p.max_rows + t] = k == owner ? slot : -1;
  }
  if (bad) raise_status(p.status, bad);

  // lengths and count, which other CTAs may still be reading: by the last one
  __syncthreads();
  if (tid == 0) {
    unsigned ticket = 0;
    if (gridDim.x > 1) {
      __threadfence();
      ticket = atomicAdd(p.ticket, 1u);
    }
    s_last = ticket == gridDim.x - 1;
  }
  __syncthreads();
  if (!s_last) return;
  for (int b = tid; b < p.batch; b += kPlanThreads) {
    uint32_t again = 0;
    const int len = p.seq_lens[b], target = p.targets[b];
    const Ask a = ask_of(p, len, target, again);
    const bool grown = row_end[b] > (b > 0 ? row_end[b - 1] : 0);
    p.new_lens[b] = again == 0 && (a.rows == 0 || grown) ? target : len;
  }
  if (tid == 0) {
    *p.new_count = min(count + freed - taken, p.num_blocks);
    if (gridDim.x > 1) *p.ticket = 0;
  }
}

}  // namespace

int plan_max_batch() { return kPlanMaxBatch; }

cudaError_t launch_kv_plan(const dcp_mla_dims& d, const int32_t* targets, const int32_t* seq_lens,
                           int32_t* new_lens, int32_t* block_table, int32_t* free_list,
                           const int32_t* free_count, int32_t* new_count, int rank_begin,
                           int num_ranks, int max_rows, int32_t* slot_mapping, int32_t* positions,
                           int32_t* cu_rows, uint32_t* workspace, uint32_t* status,
                           cudaStream_t stream) {
  const PlanParams p = {targets,    seq_lens,     new_lens,      block_table,
                        free_list,  free_count,   new_count,     slot_mapping,
                        positions,  cu_rows,      workspace,     status,
                        d.batch,    d.dcp,        d.interleave,  d.block_size,
                        d.max_blocks_per_seq,     d.max_local_len, d.num_blocks,
                        rank_begin, num_ranks,    max_rows};
  const size_t smem = (size_t)3 * d.batch * sizeof(int);
  static bool ready[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             3 * kPlanMaxBatch * (int)sizeof(int));
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  const int grid = (int)std::min<int64_t>(kSms, ((int64_t)max_rows + kPlanThreads - 1) / kPlanThreads);
  plan_kernel<<<grid, kPlanThreads, smem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dcpmla
