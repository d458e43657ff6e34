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
#include "sm103.cuh"

namespace dcpmla {
namespace {

using namespace sm103;

// ------------------------------------------------------------------ selection
//
// A cluster of up to eight CTAs holds the keys of one (rank, sequence) in shared memory:
// the weights are read once. Three passes over 11, 11 and 10 bits count the keys of each
// digit that share the threshold's bits so far. The CTAs add their counts to the first
// CTA's through the cluster's shared memory (few of the 2048 digits occur, so adding takes
// less than reading all counts of all CTAs: 2.5 against 5.5 thousand cycles a pass); that
// CTA finds the digit and tells the others. Keys beyond what shared memory holds are read
// again in every pass. What bounds it is not memory (32 rows of 131072 weights are 3 us of
// it) but the chain of passes: load, three times count, join and tell, count, place; 22.6 us
// for those rows.

constexpr int kSelBins = 2048;
constexpr int kSelPasses = 3;
constexpr int kSelMaxCluster = 8;
constexpr uint32_t kSelAlways = 0xffffffffu;  // above every key: head and tail
constexpr uint32_t kSelMore = 0x80000000u;    // with a digit: more keys have it than are left

// Weights as unsigned keys in their order: NaN as -inf, -0 as 0.
__device__ __forceinline__ uint32_t weight_key(float w) {
  const uint32_t u = __float_as_uint(fmaxf(w, -INFINITY) + 0.0f);  // fmaxf drops a NaN
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}

// Another CTA's shared memory (this CTA's at its own rank).
__device__ __forceinline__ uint2 load_cluster(const void* p, uint32_t rank) {
  uint2 v;
  asm volatile("ld.shared::cluster.v2.u32 {%0, %1}, [%2];"
               : "=r"(v.x), "=r"(v.y)
               : "r"(mapa_shared(smem_u32(p), rank)));
  return v;
}
__device__ __forceinline__ void add_cluster(const void* p, uint32_t rank, uint32_t v) {
  asm volatile("red.relaxed.cluster.shared::cluster.add.u32 [%0], %1;" ::"r"(
                   mapa_shared(smem_u32(p), rank)),
               "r"(v)
               : "memory");
}
__device__ __forceinline__ void store_cluster(const void* p, uint32_t rank, uint32_t a,
                                              uint32_t b) {
  asm volatile("st.shared::cluster.v2.u32 [%0], {%1, %2};" ::"r"(mapa_shared(smem_u32(p), rank)),
               "r"(a), "r"(b)
               : "memory");
}

struct SelectParams {
  const int32_t* seq_lens;
  const float* weights;
  int32_t* keep_idx;
  int32_t* keep_count;
  int32_t* new_lens;
  uint32_t* status;
  int batch, dcp, interleave, max_local_len, budget, sink, recent, max_keep, rank_begin;
  int cluster;   // CTAs of a (rank, sequence)
  int capacity;  // keys a CTA holds
  int wide;      // rows of weights start on 16-byte boundaries and end there
};

template <int kSelThreads>
__global__ void __launch_bounds__(kSelThreads, 1024 / kSelThreads)
    evict_select_kernel(const SelectParams p) {
  constexpr int kSelWarps = kSelThreads / 32;
  extern __shared__ __align__(16) uint32_t keys[];
  __shared__ __align__(8) int hist[kSelPasses][kSelBins];
  __shared__ int warp_sum[kSelWarps];
  __shared__ __align__(8) int counts[2];  // this CTA's keys above the threshold, and at it
  __shared__ int warp_count[2][kSelWarps];
  __shared__ __align__(8) uint32_t found[kSelPasses][2];  // the digit, and what is left there
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = blockIdx.x / p.cluster, me = blockIdx.x % p.cluster;
  const int b = pair % p.batch, k = pair / p.batch, rank = p.rank_begin + k;
  // spans are at most the budget, so everything fits 32 bits
  const int span = p.dcp * p.interleave;
  int L = p.seq_lens[b];
  const bool negative = L < 0;
  if (negative) L = 0;
  const int spans = L / span, rem = L - spans * span;
  // over the bound on any rank (rank 0 holds the most): the sequence gets no tokens
  const bool over = spans * p.interleave + min(rem, p.interleave) > p.max_local_len;
  if (tid == 0 && me == 0 && (negative || over))
    raise_status(p.status, negative ? DCP_STATUS_BAD_SEQ_LEN : DCP_STATUS_LOCAL_OVER_BOUND);
  if (over) L = 0;
  const int cut = L > p.budget ? (L - p.budget - 1) / span + 1 : 0;  // spans to drop
  const int L2 = L - cut * span;
  const int part_of = min(max(rem - rank * p.interleave, 0), p.interleave);
  const int n = L > 0 ? spans * p.interleave + part_of : 0;
  const int kept = n - cut * p.interleave;
  const float* w = p.weights + (int64_t)pair * p.max_local_len;
  int32_t* idx = p.keep_idx + (int64_t)pair * p.max_keep;
  if (tid == 0 && me == 0) {
    p.keep_count[pair] = kept;
    if (k == 0) p.new_lens[b] = L2;
  }
  const int all = p.cluster * kSelThreads, at = me * kSelThreads + tid;
  for (int i = kept + at; i < p.max_keep; i += all) idx[i] = -1;
  if (kept == n) {  // the same for every CTA of the cluster
    for (int i = at; i < n; i += all) idx[i] = i;
    return;
  }
  // this CTA's tokens [t0, t0 + mine), a multiple of 32 * 32 but for the last
  const int part = (n + p.cluster * kSelThreads - 1) / (p.cluster * kSelThreads) * kSelThreads;
  const int t0 = min(n, me * part), mine = min(n, t0 + part) - t0;
  const int tail = n - p.recent;
  auto fresh_key = [&](int i) {
    const int t = t0 + i;
    return t < p.sink || t >= tail ? kSelAlways : weight_key(w[t]);
  };
  // keys i .. i + 3 (i a multiple of 4); 0, below every key, behind the last
  auto keys4 = [&](int i) {
    if (i + 4 <= p.capacity) return *reinterpret_cast<const uint4*>(keys + i);
    uint32_t x[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < mine ? fresh_key(i + e) : 0u;
    return make_uint4(x[0], x[1], x[2], x[3]);
  };
  for (int i = tid; i < kSelPasses * kSelBins; i += kSelThreads) (&hist[0][0])[i] = 0;
  auto sync = [&]() {
    if (p.cluster > 1) cluster_sync_all();
    else __syncthreads();
  };
  __syncthreads();
  if (p.cluster > 1) cluster_arrive();  // counts are zero: the others may add to the first CTA's
  // the first pass counts the keys as they come
  const int padded = (mine + 127) / 128 * 128;
  auto take = [&](int i, uint32_t key) {
    if (key != kSelAlways && i < mine) atomicAdd(&hist[0][key >> 21], 1);
  };
  if (p.wide) {  // 16-byte loads; what they read behind the sequence is in its row's bound
    for (int i0 = 0; i0 < padded; i0 += 16 * kSelThreads) {
      float4 x[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 4 * (u * kSelThreads + tid);
        x[u] = i < mine ? *reinterpret_cast<const float4*>(w + t0 + i)
                        : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int i = i0 + 4 * (u * kSelThreads + tid);
        if (i >= padded) break;
        const float v[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
        uint32_t key[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int t = t0 + i + e;
          key[e] = i + e >= mine                ? 0u
                   : t < p.sink || t >= tail ? kSelAlways
                                             : weight_key(v[e]);
          take(i + e, key[e]);
        }
        if (i < p.capacity)
          *reinterpret_cast<uint4*>(keys + i) = make_uint4(key[0], key[1], key[2], key[3]);
      }
    }
  } else {
    for (int i0 = 0; i0 < padded; i0 += 8 * kSelThreads) {
      uint32_t x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kSelThreads + tid;
        x[u] = i < mine ? fresh_key(i) : 0u;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int i = i0 + u * kSelThreads + tid;
        if (i < padded && i < p.capacity) keys[i] = x[u];
        take(i, x[u]);
      }
    }
  }
  const int m = kept - p.sink - p.recent;  // of the tokens between head and tail
  uint32_t T = 0;                          // the threshold's bits so far
  int left = m;                            // to be taken from the keys that share them
  for (int pass = 0; pass < kSelPasses; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;
    const int bins = pass == 2 ? 1024 : 2048;
    if (pass > 0) {
      // few keys share the threshold's bits (head and tail never do: they lie above +inf)
      const int above = shift + (pass == 1 ? 11 : 10);
      const uint32_t top = T >> above;
      for (int i = 4 * tid; i < padded; i += 4 * kSelThreads) {
        const uint4 q = keys4(i);
        if (q.x >> above == top || q.y >> above == top || q.z >> above == top ||
            q.w >> above == top) {
          const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (x[e] >> above == top) atomicAdd(&hist[pass][x[e] >> shift & (bins - 1)], 1);
        }
      }
    }
    if (pass == 0 && p.cluster > 1) cluster_wait();
    if (me > 0) {
      __syncthreads();
      for (int i = tid; i < bins; i += kSelThreads)
        if (const int c = hist[pass][i]) add_cluster(&hist[pass][i], 0, (uint32_t)c);
    }
    sync();
    if (me == 0) {
      // neighbouring bins per thread, the largest digits first
      constexpr int kPer = kSelBins / kSelThreads;
      const int first = bins - 1 - kPer * tid;
      int c[kPer], sum = 0;
#pragma unroll
      for (int e = 0; e < kPer; e += 2) {
        const int2 two = first >= 0 ? *reinterpret_cast<const int2*>(&hist[pass][first - e - 1])
                                    : make_int2(0, 0);
        c[e] = two.y;
        c[e + 1] = two.x;
        sum += two.x + two.y;
      }
      int incl = sum;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      if (lane == 31) warp_sum[warp] = incl;
      __syncthreads();
      int before =
          incl - sum + __reduce_add_sync(0xffffffffu, lane < warp ? warp_sum[lane] : 0);
      // the digit at which the keys counted from above reach `left`
#pragma unroll
      for (int e = 0; e < kPer; ++e) {
        if (before < left && left <= before + c[e]) {
          const uint32_t more = left < before + c[e] ? kSelMore : 0u;
          for (int r = 0; r < p.cluster; ++r)
            store_cluster(found[pass], r, (uint32_t)(first - e) | more, (uint32_t)(left - before));
        }
        before += c[e];
      }
    }
    sync();
    if (m > 0) {
      T |= (found[pass][0] & ~kSelMore) << shift;
      left = (int)found[pass][1];
    }
  }
  // Keys at T stay as long as fewer than `equal` came before them. As a rule all of them stay,
  // and that is to be above the key below T: half the work of the two loops below.
  const bool ties = m > 0 && (found[kSelPasses - 1][0] & kSelMore) != 0u;
  const int equal = ties ? left : 0;
  // m == 0: no key is above this threshold but the head's and the tail's
  if (!ties) T = m > 0 ? T - 1 : kSelAlways - 1;

  // each warp's run of keys, 128 at a time: how many are above T and at T, then their
  // places in order
  const int run = (padded / 128 + kSelWarps - 1) / kSelWarps * 128;
  const int r0 = min(padded, warp * run), r1 = min(padded, r0 + run);
  int gt = 0, eq = 0;
  for (int i = r0 + 4 * lane; i < r1; i += 128) {
    const uint4 q = keys4(i);
    gt += (q.x > T) + (q.y > T) + (q.z > T) + (q.w > T);
    if (ties) eq += (q.x == T) + (q.y == T) + (q.z == T) + (q.w == T);
  }
  gt = __reduce_add_sync(0xffffffffu, gt);
  eq = __reduce_add_sync(0xffffffffu, eq);
  if (lane == 0) {
    warp_count[0][warp] = gt;
    warp_count[1][warp] = eq;
  }
  __syncthreads();
  if (warp == 0) {
    const int g = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_count[0][lane] : 0);
    const int e = __reduce_add_sync(0xffffffffu, lane < kSelWarps ? warp_count[1][lane] : 0);
    if (lane == 0) {
      counts[0] = g;
      counts[1] = e;
    }
  }
  sync();
  // keys before this warp's run: of the CTAs before this one, and its warps before this one
  const uint2 theirs = lane < me ? load_cluster(counts, lane) : make_uint2(0, 0);
  int above = __reduce_add_sync(
      0xffffffffu, (int)theirs.x + (lane < warp ? warp_count[0][lane] : 0));
  int level = __reduce_add_sync(
      0xffffffffu, (int)theirs.y + (lane < warp ? warp_count[1][lane] : 0));
  const uint32_t earlier = (1u << lane) - 1u;  // lanes
  for (int i0 = r0; i0 < r1; i0 += 128) {
    const int i = i0 + 4 * lane;
    const uint4 q = keys4(i);
    const uint32_t x[4] = {q.x, q.y, q.z, q.w};
    if (!ties) {
      int at = above;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t in = __ballot_sync(0xffffffffu, x[e] > T);
        at += __popc(in & earlier);
        above += __popc(in);
      }
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (x[e] > T) idx[at++] = t0 + i + e;
      continue;
    }
    // both counts of this lane in one word, and of the lanes before it
    int both = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) both += (x[e] > T) + ((x[e] == T) << 16);
    int incl = both;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += y;
    }
    const int excl = incl - both;
    int g = above + (excl & 0xffff), e_seen = level + (excl >> 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const bool is_eq = x[e] == T;
      if (x[e] > T || (is_eq && e_seen < equal)) idx[g + min(e_seen, equal)] = t0 + i + e;
      g += x[e] > T;
      e_seen += is_eq;
    }
    const int last = __shfl_sync(0xffffffffu, incl, 31);
    above += last & 0xffff;
    level += last >> 16;
  }
  if (p.cluster > 1) cluster_sync_all();  // the others may still read this CTA's counts
}

// ------------------------------------------------------------------ compaction
//
// Memory-bound: every moved row is read and written once. A CTA takes a slice of the rows
// of one (rank, sequence) (16-byte pieces [slice * width, ...)) and, when the rows go to
// other blocks, a segment of them. Its pieces pass through a ring of asynchronous copies in
// row order, two rounds in flight, three CTAs to an SM: 302 MB in place 105.0 us (5.8 TB/s read
// and written), 618 MB to other blocks 188.5 us (6.6 TB/s). Two CTAs 105.7 and 192.8 us, four
// 106.0 and 189.0, three rounds in flight 117.2 and 189.8. In place, a round is written when
// all of its own reads have arrived; rounds that are still being read lie behind what it
// writes.

constexpr int kMoveThreads = 256;
constexpr int kMovePer = 4;                             // 16-byte pieces per thread and round
constexpr int kMoveRound = kMoveThreads * kMovePer;     // 16 KB
constexpr int kMoveStages = 3;                          // 48 KB
constexpr int kMoveChunk = 1024;                        // rows looked up together
constexpr int kMoveSmem = kMoveStages * kMoveRound * 16;
constexpr int kWeightPer = 32;                          // weights per thread and round

struct MoveParams {
  const int32_t* keep_idx;
  const int32_t* keep_count;
  const int32_t* src_table;
  const int32_t* dst_table;
  uint4* pool;
  const float* w_in;
  float* w_out;
  uint32_t* status;
  int batch, block_size, max_blocks, num_blocks, max_keep, max_local_len;
  int pieces;        // of a row
  int width;         // pieces of a slice
  int slices;
  int segment_rows;  // rows of a CTA (all of them in place)
  FastDiv block_div, width_div;
};

// The blocks that row t of a sequence comes from and row i goes to, and what is wrong with
// them: such a row stays where it is, and its weight too.
template <bool kInPlace>
__device__ __forceinline__ uint32_t find_blocks(const MoveParams& p, int b, int t, int i,
                                                int& from, int& to) {
  const int32_t* src = p.src_table + (int64_t)b * p.max_blocks;
  const int32_t* dst = p.dst_table + (int64_t)b * p.max_blocks;
  from = src[p.block_div.div(t)];
  to = dst[p.block_div.div(i)];
  if (from < 0 || from >= p.num_blocks || to < 0 || to >= p.num_blocks)
    return DCP_STATUS_BAD_BLOCK_ID;
  // a copy of the source's table: that is in place
  return !kInPlace && to == src[p.block_div.div(i)] ? DCP_STATUS_BAD_PAGE : 0u;
}

// Weights of indices up to `last`; kLook: of rows whose blocks are good. Whether there were
// indices behind `last`.
template <bool kInPlace, bool kLook>
__device__ __forceinline__ bool move_weight_rounds(const MoveParams& p, int b, const int32_t* idx,
                                                   const float* from, float* to, int n,
                                                   int last) {
  bool more = false;
  for (int r0 = 0; r0 < n; r0 += kMoveThreads * kWeightPer) {
    int x[kWeightPer];   // the index, then the weight's bits
    uint32_t valid = 0;  // one bit each
#pragma unroll
    for (int u = 0; u < kWeightPer; ++u) {
      const int i = r0 + u * kMoveThreads + threadIdx.x;
      x[u] = i < n ? idx[i] : -1;
    }
#pragma unroll
    for (int u = 0; u < kWeightPer; ++u) {
      const int i = r0 + u * kMoveThreads + threadIdx.x;
      more |= x[u] > last;
      if (x[u] >= i && x[u] <= last) {
        int sb, db;
        if (!kLook || (kInPlace && x[u] == i) ||
            find_blocks<kInPlace>(p, b, x[u], i, sb, db) == 0)
          valid |= 1u << u;
        x[u] = __float_as_int(from[x[u]]);
      }
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < kWeightPer; ++u)
      if (valid >> u & 1) to[r0 + u * kMoveThreads + threadIdx.x] = __int_as_float(x[u]);
  }
  return more;
}

// The weights of one (rank, sequence), by one CTA: a round is read before it is written.
// Rounds of 8192: with 2048 the rounds' latencies added up (24 us for 24 thousand rows). A row
// with a bad block keeps its weight. As a rule there is none, and the blocks up to the last
// index's are looked over once, not weight by weight (one sequence of 81672 rows to other
// blocks 48 to 52 us, weight by weight 125).
template <bool kInPlace>
__device__ void move_weights(const MoveParams& p, int pair, int b, int n) {
  const int32_t* idx = p.keep_idx + (int64_t)pair * p.max_keep;
  const float* from = p.w_in + (int64_t)pair * p.max_local_len;
  float* to = p.w_out + (int64_t)pair * p.max_local_len;
  const int32_t* src = p.src_table + (int64_t)b * p.max_blocks;
  const int32_t* dst = p.dst_table + (int64_t)b * p.max_blocks;
  const int last = min(n > 0 ? idx[n - 1] : -1, p.max_local_len - 1);
  int odd = last < n - 1;
  if (!odd && n > 0) {
    constexpr int kPer = 8;  // blocks of a thread in flight
    const int from_blocks = p.block_div.div(last) + 1, to_blocks = p.block_div.div(n - 1) + 1;
    for (int k0 = threadIdx.x; k0 < from_blocks; k0 += kPer * kMoveThreads) {
      int x[kPer], y[kPer];
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        const int k = k0 + u * kMoveThreads;
        x[u] = k < from_blocks ? src[k] : 0;
        y[u] = !kInPlace && k < to_blocks ? dst[k] : -1;
      }
#pragma unroll
      for (int u = 0; u < kPer; ++u) {
        odd |= x[u] < 0 || x[u] >= p.num_blocks;
        if (!kInPlace && k0 + u * kMoveThreads < to_blocks)
          odd |= y[u] < 0 || y[u] >= p.num_blocks || y[u] == x[u];
      }
    }
  }
  if (__syncthreads_or(odd)) {
    move_weight_rounds<kInPlace, true>(p, b, idx, from, to, n, p.max_local_len - 1);
  } else if (__syncthreads_or(
                 move_weight_rounds<kInPlace, false>(p, b, idx, from, to, n, last))) {
    // indices out of order: these rows lie behind row n - 1, so none has been written over
    for (int i = threadIdx.x; i < n; i += kMoveThreads) {
      const int t = idx[i];
      int sb, db;
      if (t > last && t < p.max_local_len && find_blocks<kInPlace>(p, b, t, i, sb, db) == 0)
        to[i] = from[t];
    }
  }
}

template <bool kInPlace>
__global__ void __launch_bounds__(kMoveThreads, 3) kv_move_kernel(const MoveParams p) {
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ int2 rows[kMoveChunk];  // from, to; from -1: not moved
  const int pair = blockIdx.x, b = pair % p.batch, k = pair / p.batch;
  int n = p.keep_count[pair];
  if (n < 0 || n > p.max_keep) {
    if (threadIdx.x == 0 && blockIdx.y == 0) raise_status(p.status, DCP_STATUS_BAD_PAGE);
    return;
  }
  // A CTA per (rank, sequence) moves the weights. Before the segments: a long sequence's take
  // as long as many of them (80000 rows of 2 KB on each of two ranks 103 us, behind them
  // 122). In place behind the rows, which take longer (105.1 against 107.5 us).
  int part = blockIdx.y;
  if (p.w_in != nullptr) {
    if (part == (kInPlace ? gridDim.y - 1 : 0)) {
      move_weights<kInPlace>(p, pair, b, n);
      return;
    }
    if (!kInPlace) --part;
  }
  const int slice = part % p.slices, segment = part / p.slices;
  const int first = segment * p.segment_rows;
  n = min(n, first + p.segment_rows);
  const int piece0 = slice * p.width, width = min(p.width, p.pieces - piece0);
  const int32_t* idx = p.keep_idx + (int64_t)pair * p.max_keep;
  const int64_t limit = (int64_t)p.max_blocks * p.block_size;
  uint4* base = p.pool + (int64_t)k * p.num_blocks * p.block_size * p.pieces + piece0;
  const uint32_t my = smem_u32(ring) + threadIdx.x * 16;
  uint32_t bad = 0;
  for (int c0 = first; c0 < n; c0 += kMoveChunk) {
    const int count = min(kMoveChunk, n - c0);
    __syncthreads();
    for (int r = threadIdx.x; r < count; r += kMoveThreads) {
      const int i = c0 + r, t = idx[i];
      int2 row = make_int2(-1, 0);
      if (t < i || t >= limit || i >= limit) {
        bad |= DCP_STATUS_BAD_PAGE;
      } else if (!kInPlace || t != i) {
        int sb, db;
        const uint32_t wrong = find_blocks<kInPlace>(p, b, t, i, sb, db);
        bad |= wrong;
        if (wrong == 0)
          row = make_int2(sb * p.block_size + p.block_div.mod(t),
                          db * p.block_size + p.block_div.mod(i));
      }
      rows[r] = row;
    }
    __syncthreads();
    const int total = count * width, rounds = (total + kMoveRound - 1) / kMoveRound;
    auto place = [&](int f, int& row, int& piece) {
      row = p.width_div.div(f);
      piece = f - row * p.width;
      if (width != p.width) {  // the last slice is narrower
        row = f / width;
        piece = f - row * width;
      }
    };
    auto fetch = [&](int r) {
      if (r < rounds) {
#pragma unroll
        for (int u = 0; u < kMovePer; ++u) {
          const int f = r * kMoveRound + u * kMoveThreads + threadIdx.x;
          if (f >= total) break;
          int row, piece;
          place(f, row, piece);
          const int from = rows[row].x;
          if (from >= 0)
            cp_async16(my + ((r % kMoveStages) * kMoveRound + u * kMoveThreads) * 16,
                       base + (int64_t)from * p.pieces + piece, 16);
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int r = 0; r < kMoveStages - 1; ++r) fetch(r);
    for (int r = 0; r < rounds; ++r) {
      cp_async_wait_group<kMoveStages - 2>();
      if (kInPlace) __syncthreads();  // every thread's reads of this round have arrived
      fetch(r + kMoveStages - 1);
#pragma unroll
      for (int u = 0; u < kMovePer; ++u) {
        const int f = r * kMoveRound + u * kMoveThreads + threadIdx.x;
        if (f >= total) break;
        int row, piece;
        place(f, row, piece);
        if (rows[row].x >= 0)
          base[(int64_t)rows[row].y * p.pieces + piece] = *reinterpret_cast<const uint4*>(
              ring + ((r % kMoveStages) * kMoveRound + u * kMoveThreads + threadIdx.x) * 16);
      }
    }
  }
  if (bad) raise_status(p.status, bad);
}

}  // namespace

cudaError_t launch_evict_select(const dcp_mla_dims& d, const int32_t* seq_lens,
                                const float* weights, int budget, int sink, int recent,
                                int max_keep, int rank_begin, int num_ranks, int32_t* keep_idx,
                                int32_t* keep_count, int32_t* new_lens, uint32_t* status,
                                cudaStream_t stream) {
  constexpr int kMaxKeys = (232448 - 1024 * 32) / 4 / 128 * 128;  // beside the histograms
  SelectParams p;
  p.seq_lens = seq_lens;
  p.weights = weights;
  p.keep_idx = keep_idx;
  p.keep_count = keep_count;
  p.new_lens = new_lens;
  p.status = status;
  p.batch = d.batch;
  p.dcp = d.dcp;
  p.interleave = d.interleave;
  p.max_local_len = d.max_local_len;
  p.budget = budget;
  p.sink = sink;
  p.recent = recent;
  p.max_keep = max_keep;
  p.rank_begin = rank_begin;
  // As many CTAs as give each a few thousand keys, while all are resident. Long rows: 1024
  // threads, one CTA to an SM (32 rows of 131072 weights 22.6 us, with 512 threads 23.8);
  // else 512, two to an SM (8 rows of 2048 7.5 us, with 1024 threads 8.3).
  const int64_t pairs = (int64_t)num_ranks * d.batch;
  const bool many = d.max_local_len > 16384;
  const int threads = many ? 1024 : 512;
  p.cluster = 1;
  while (p.cluster < kSelMaxCluster &&
         (d.max_local_len / p.cluster > kMaxKeys ||
          (d.max_local_len / p.cluster > 4096 && pairs * p.cluster * 2 <= (many ? kSms : 2 * kSms))))
    p.cluster *= 2;
  const int64_t part =
      ((int64_t)d.max_local_len + p.cluster * threads - 1) / (p.cluster * threads) * threads;
  p.capacity = (int)std::min<int64_t>(part, kMaxKeys);
  p.wide = ((uintptr_t)weights & 15) == 0 && d.max_local_len % 4 == 0;
  const int64_t ctas = pairs * p.cluster;
  if (ctas > INT32_MAX) return cudaErrorInvalidConfiguration;
  auto kern = many ? evict_select_kernel<1024> : evict_select_kernel<512>;
  static bool attr_set[2][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[many][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxKeys * 4);
    if (e != cudaSuccess) return e;
    attr_set[many][dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = p.capacity * 4;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = p.cluster;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, p);
}

cudaError_t launch_kv_compact(const dcp_mla_dims& d, int row_bytes, const int32_t* keep_idx,
                              const int32_t* keep_count, int max_keep, const int32_t* src_table,
                              const int32_t* dst_table, int num_ranks, void* pool,
                              const float* weights_in, float* weights_out, uint32_t* status,
                              cudaStream_t stream) {
  constexpr int kWant = 3 * kSms;  // CTAs that fill the device
  const bool in_place = src_table == dst_table;
  const int64_t pairs = (int64_t)num_ranks * d.batch;
  MoveParams p;
  p.keep_idx = keep_idx;
  p.keep_count = keep_count;
  p.src_table = src_table;
  p.dst_table = dst_table;
  p.pool = static_cast<uint4*>(pool);
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.status = status;
  p.batch = d.batch;
  p.block_size = d.block_size;
  p.max_blocks = d.max_blocks_per_seq;
  p.num_blocks = d.num_blocks;
  p.max_keep = max_keep;
  p.max_local_len = d.max_local_len;
  p.pieces = row_bytes / 16;
  p.width = p.pieces;
  p.segment_rows = max_keep;
  if (in_place) {
    // the rows of a (rank, sequence) go in order, so more CTAs can only share their width:
    // down to 32 bytes, a sector of L2 (one sequence cut to 78000 rows of 1 KB on three ranks
    // 104 us, with slices of 64 bytes 136; 8 sequences cut to 16384 rows 87 and 101). Such narrow
    // slices are 2.2 to 5 times the floor: 1024 rows of one are two rounds, so that for every
    // lookup the ring fills and empties behind two dependent loads and two barriers.
    const int64_t want = std::max<int64_t>(1, kWant / pairs);
    p.width = std::max<int>((int)((p.pieces + want - 1) / want), std::min(p.pieces, 2));
    p.width = std::min(p.pieces, (p.width + 1) / 2 * 2);
  } else {
    // enough segments to even out sequences of different lengths
    const int64_t want = std::max<int64_t>(1, 8 * kWant / pairs);
    p.segment_rows = (int)std::max<int64_t>((max_keep + want - 1) / want, 64);
  }
  p.slices = (p.pieces + p.width - 1) / p.width;
  const int segments = (max_keep + p.segment_rows - 1) / p.segment_rows;
  p.block_div = FastDiv::by(d.block_size);
  p.width_div = FastDiv::by(p.width);
  if (pairs > INT32_MAX) return cudaErrorInvalidConfiguration;
  const dim3 grid((unsigned)pairs,
                  (unsigned)(p.slices * segments + (weights_in != nullptr ? 1 : 0)));
  auto kern = in_place ? kv_move_kernel<true> : kv_move_kernel<false>;
  static bool attr_set[2][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[in_place][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMoveSmem);
    if (e != cudaSuccess) return e;
    attr_set[in_place][dev] = true;
  }
  kern<<<grid, kMoveThreads, kMoveSmem, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dcpmla
