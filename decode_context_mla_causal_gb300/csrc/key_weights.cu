// The attention weight that each cached latent row receives from a verify step, added to
// what earlier steps left.
//
// For local token t of (rank, sequence), with the step's merged LSE of every row (j, head),
//   w'_t = [t < n_old] decay * w_t + sum over rows that see t of
//          2^(softmax_scale * kv_scale * log2(e) * (q . k_t) - log2(e) * LSE_row).
// A token's sum needs that token's row and the queries alone, so no token's result
// depends on how the tokens are spread over the machine.
//
// The product S = K Q^T is formed with the tokens as its rows: an accumulator lane is a
// token, and the sum over query rows is a sum over that lane's columns, in one thread's
// registers. Two CTAs share each product (256 tokens, each CTA's own 128 in its shared
// memory and its own accumulator lanes; each holds half of the query rows). The queries of
// one (sequence, row group) stay in shared memory while the tokens stream past:
//   producers  3 warps: TMA copies of 128-byte slices of 128 tokens into a ring, one box per
//              run of a block's tokens. (Copies by threads, 64 bytes a row, need a proxy
//              fence before the tensor core may read them: by the copying threads it drains
//              their copies, 2.4 us a slice; by the issuer it still took 0.6 us a slice,
//              four times the products of 128 rows.)
//   issuer     1 thread of the even CTA: tcgen05.mma of a slice as soon as both CTAs have it
//              (one of the odd CTA passes its arrivals on); both fetch the queries by TMA at
//              the start of a (sequence, row group)
//   epilogue   8 warps, four for each half of the columns: exponentials and sums of the
//              finished tile while the next one is multiplied (two buffers of up to 256
//              columns; one, of four sums, for BF16 products of 65 to 128)
// An FP8 cache's codes enter the tensor cores as they are. q is the sum of an E4M3 term
// (four significant bits) and an E5M2 term for the rest, over a power-of-two scale per row
// that brings the largest element into (224, 448]. bf16 has eight bits, so the rest is 0 to
// 8 units of its last one and E5M2's three bits hold it exactly while the first term is
// normal (elements from 2^-14 of the largest up); below, the sum is off by at most 2^-13
// over 224, under 2^-20 of the largest. Both products run at twice the 16-bit rate, so the
// two cost what one 16-bit product would, and no converted copy of the cache is needed. A
// small kernel forms the terms first (by the epilogue warps of every pair of CTAs it took 8
// us per sequence and pair); the main kernel sets itself up meanwhile.
//
// Work is cut by tiles, not by sequences: the tiles of all sequences are counted from the
// lengths and every pair of CTAs takes an equal, contiguous share, so lengths of any spread
// finish together and the queries change a few times per pair. Each half of a tile, one CTA's
// tokens, has a rank of its own: local lengths are rounded up to half tiles, not to tiles (43
// sequences of up to 1053 tokens on eight ranks, 512 rows: 34.8 us, with whole tiles 45.6). With
// more than 256 rows per sequence the rows are cut into groups; the groups' pairs of CTAs
// walk the same tiles side by side, so that the cache is read from memory once and from L2
// by the others. The groups' sums then go to the workspace, and a second kernel adds them
// in order.
//
// Bound by the tensor cores from about 150 rows on (BF16 290), by memory below. Measured: 4
// sequences of 1048576 tokens, 384 rows, FP8: 1.01 ms, 1.84 PFLOP/s (1.14 ms, 1.63 PFLOP/s, in
// a loop that brings the clock down to 1.5 GHz); 32 sequences of 32768 tokens, 128 rows: BF16
// 189 us, 6.4 TB/s, FP8 114 us, 5.3 TB/s. Blocks of 8 tokens take 16 copies a slice, more than
// three warps issue beside its products: 3 ragged sequences, 480 rows, BF16 112 us, floor 56.
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "sm103.cuh"

namespace dcpmla {
namespace {

using namespace sm103;

constexpr int kTileRows = 256;    // of a product: 128 accumulator lanes in each CTA
constexpr int kMaxCols = 256;     // query rows per product
constexpr int kStageBytes = 128 * 128;  // a slice: 128 bytes of 128 tokens' rows
constexpr int kEpiWarps = 8;      // two groups of four, one for each half of the columns
constexpr int kAhead = 3;         // tiles between reading a token's history and using it
constexpr int kMmaWarp = kEpiWarps;
constexpr int kProdWarp0 = kMmaWarp + 1;
constexpr int kProdWarps = 3;
constexpr int kThreads = 32 * (kProdWarp0 + kProdWarps);
constexpr int kMaxStages = 12;
constexpr uint32_t kTmemCols = 512;
constexpr uint64_t kTimeoutNs = 4000000000ull;
constexpr int kSmemLimit = 232448;
constexpr float kLog2eHi = 1.44269502162933349609375f;  // log2(e), and what it rounds off
constexpr float kLog2eLo = 1.92596299e-8f;

// A latent row in slices of 128 bytes; the last one of an FP8 row is half full.
template <bool kFp8>
struct Shape {
  static constexpr int dims = kFp8 ? 128 : 64;
  static constexpr int slices = kFp8 ? 5 : 9;
  // The tensor cores drop what lies below an accumulator's last bit instead of rounding it, and
  // a score comes out nearer to zero the longer its sum is. So a row's products are added up in
  // several accumulators, and those in 32 bits, rounded to nearest: with one sum of a BF16 row's
  // 36 steps the weights of 7 sequences of up to 4712 tokens (16 rows, no history) are off by
  // 3.0e-6 together, with four by 8.9e-7 (32-bit arithmetic: 8.2e-7); 288 rows: one 1.8e-6, two
  // 9.4e-7. An FP8 row's 36 products have fewer bits: 8 rows without history one sum 1.1e-6, two
  // 5.0e-7 (32-bit arithmetic: 4.5e-7); from 192 rows up one at most 5.7e-7. A CTA has 512 columns
  // of tensor memory: up to 128 columns of a product leave room for four sums (twice up to 64,
  // so that a tile's are read while the next one's are formed), or twice two of FP8. Above, FP8
  // takes one sum, and BF16's two take turns: the epilogue holds the first in registers. BF16, 4
  // sequences of 262144 tokens: 128 rows 184 us with one sum and 185, 256 rows 229 and 235, 1024
  // rows 743 and 760 (four sums 1160); 45 of up to 1041, 64 rows 12.7 and 12.8. FP8, 128 rows or
  // fewer: the same.
  __host__ __device__ static constexpr int sums(int cols) {
    return kFp8 ? (cols > 128 ? 1 : 2) : (cols > 128 ? 2 : 4);
  }
  // Whether a sum ends with slice s.
  __host__ __device__ static constexpr bool ends_sum(int s, int sums) {
    return s == slices - 1 ||
           (sums == 2 ? s == slices / 2 - 1 : sums == 4 && s % 2 == 1 && s < slices - 2);
  }
};

struct KeyWeightParams {
  const int32_t* seq_lens;
  const int32_t* block_table;
  const uint16_t* q;
  const uint8_t* kv;
  const float* kv_scale;
  const float* lse;
  const float* w_in;
  float* w_out;
  float* part;  // [groups][nr][B][max_local_len] sums of the row groups, if there are several
  uint32_t* status;
  float scale_hi, scale_lo;  // softmax_scale * log2(e) in two parts
  float decay;
  int batch, qlen, H, dcp, interleave, block_size, max_blocks, max_local_len, num_blocks, causal,
      rank_begin, num_ranks;
  int groups, group_rows;  // row groups per sequence, rows of each
  int cols;                // group_rows rounded up to a multiple of 32: the product's N
  int stages;
  FastDiv block_div, interleave_div, half_div, pairs_div;
  int page;   // tokens of one copy: a divisor of the block size
  int lanes;  // tokens of a CTA's half tile: the pages that fit 128 lanes
  int rows;   // query rows of a sequence
  const float* q_scale;  // FP8: [B][rows] what the two terms' scale makes of each score
};

// Shared memory of one CTA, in order: half of the queries, the ring, the columns' scales
// and offsets, the next tiles' block ids and histories with the second half columns' sums,
// barriers.
struct Layout {
  int q_bytes, params, tokens, bars, total;
};
__host__ __device__ inline Layout layout_of(int cols, int stages) {
  Layout l;
  l.q_bytes = cols / 2 * kDqk * 2;  // two 8-bit terms, or bf16
  l.params = l.q_bytes + stages * kStageBytes;
  l.tokens = l.params + kMaxCols * 8;
  l.bars = l.tokens + (2 * (kAhead + 1) + 2) * 128 * 4;
  l.total = l.bars + (3 * kMaxStages + 10) * 8 + 64 + 1024;
  return l;
}

// Lengths of one sequence on the call's ranks, from one division.
struct Lengths {
  int whole;  // tokens of complete spans on every rank
  int rem;    // tokens past them
  int old;    // global tokens before the step's own (negative if there are fewer than qlen)
};
__device__ __forceinline__ Lengths lengths_of(const KeyWeightParams& p, int b) {
  int L = p.seq_lens[b];
  Lengths x;
  x.old = (int)max((int64_t)L - p.qlen, (int64_t)INT32_MIN);
  if (L < 0) L = 0;
  const int64_t span = (int64_t)p.dcp * p.interleave;
  // in 32 bits wherever the span fits them
  const int spans = span <= INT32_MAX ? (int)((unsigned)L / (unsigned)span) : 0;
  x.whole = spans * p.interleave;
  x.rem = (int)(L - spans * span);
  return x;
}
__device__ __forceinline__ int rank_len(const KeyWeightParams& p, const Lengths& x, int k) {
  const int64_t r = x.rem - (int64_t)(p.rank_begin + k) * p.interleave;
  const int part = r < 0 ? 0 : (r > p.interleave ? p.interleave : (int)r);
  return min(x.whole + part, p.max_local_len);
}
__device__ __forceinline__ int tiles_of(const KeyWeightParams& p, int n) {
  return n > 0 ? p.half_div.div(n - 1) + 1 : 0;
}

// Tiles of a pair of CTAs that hold a sequence: half a tile, one CTA's tokens, is of one rank.
__device__ __forceinline__ int pair_tiles(const KeyWeightParams& p, const Lengths& x) {
  int halves = 0;
  for (int k = 0; k < p.num_ranks; ++k) halves += tiles_of(p, rank_len(p, x, k));
  return (halves + 1) / 2;
}

// A CTA's walk over the tiles of its pair's share, in the order sequence, rank, half tile. The
// even CTA takes the even halves of a sequence, the odd CTA the odd ones; behind the last one
// it has none (n = 0).
struct Walk {
  int cta, b, k, n, tile, tiles;  // tile: this CTA's half; tiles: halves on rank k
  int here;                       // tiles of the pair in the sequence, from this one on
  int left;                       // and in the share
  Lengths len;
  __device__ __forceinline__ void rank_at(const KeyWeightParams& p) {
    n = rank_len(p, len, k);
    tiles = tiles_of(p, n);
  }
  // from half tile `tile` counted from rank k on to its rank
  __device__ __forceinline__ void settle(const KeyWeightParams& p) {
    while (tile >= tiles) {
      tile -= tiles;
      if (++k == p.num_ranks) {
        n = k = tile = 0;
        return;
      }
      rank_at(p);
    }
  }
  __device__ __forceinline__ void enter(const KeyWeightParams& p, int half) {
    k = 0;
    rank_at(p);
    tile = half;
    settle(p);
  }
  // `share` tiles from tile `skip` of the `of` tiles of sequence b0 on
  __device__ __forceinline__ void start(const KeyWeightParams& p, int cta_, int b0,
                                        const Lengths& x, int skip, int of, int share) {
    cta = cta_;
    b = b0;
    left = share;
    if (share <= 0) return;
    len = x;
    here = of - skip;
    enter(p, 2 * skip + cta);
  }
  // to the next tile; there must be one (left > 1 before)
  __device__ __forceinline__ void advance(const KeyWeightParams& p) {
    --left;
    if (--here > 0) {
      tile += 2;
      settle(p);
      return;
    }
    do {
      ++b;
      len = lengths_of(p, b);
      here = pair_tiles(p, len);
    } while (here == 0);
    enter(p, cta);
  }
};

// Buffers of the accumulators.
__host__ __device__ constexpr int buffers(bool fp8, int cols) {
  return !fp8 && cols > 64 && cols <= 128 ? 1 : 2;
}

struct Barriers {
  uint64_t* full;    // [stages] a slice is in this CTA's ring
  uint64_t* peer;    // [stages] even CTA: it is in the odd CTA's
  uint64_t* empty;   // [stages] the slice has been multiplied
  uint64_t* dfull;   // [2] a buffer holds a tile's sums, or one of its two
  uint64_t* dempty;  // [2] even CTA: both CTAs have read it
  uint64_t* qfull;   // this CTA's half of the queries is here
  uint64_t* qpeer;   // even CTA: the odd CTA's half is there
  uint64_t* qfree;   // every product with the last queries is done
  uint64_t* drain;
  uint32_t* tmem_slot;
  int* abort_flag;
};

// Bounded waits. What other CTAs write into this one arrives through copies and tensor-core
// completions, so no wait needs a cluster-scope acquire (which takes several hundred cycles).
__device__ __noinline__ bool wait_slow(uint32_t a, uint32_t parity, int* abort_flag,
                                       uint32_t* status) {
  const uint64_t t0 = globaltimer_ns();
  for (;;) {
    if (mbar_wait_sleep(a, parity)) return true;
    if (*reinterpret_cast<volatile int*>(abort_flag)) return false;
    if (globaltimer_ns() - t0 > kTimeoutNs) {
      *reinterpret_cast<volatile int*>(abort_flag) = 1;
      raise_status(status, DCP_STATUS_TIMEOUT);
      return false;
    }
  }
}
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, int* abort_flag,
                                         uint32_t* status) {
  const uint32_t a = smem_u32(bar);
  return mbar_try_wait(a, parity) || wait_slow(a, parity, abort_flag, status);
}
// For copies in flight after a timeout: bounded, and whatever the abort flag says.
__device__ __forceinline__ void wait_landed(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_wait_sleep(a, parity) && globaltimer_ns() - t0 < kTimeoutNs) {
  }
}
// Of a converged warp, with a warp-uniform result.
__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, int* abort_flag,
                                         uint32_t* status) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, abort_flag, status));
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats -> 8-bit codes (nearest, saturated), and E4M3 codes back.
__device__ __forceinline__ uint32_t to_f8x2(float lo, float hi, __nv_fp8_interpretation_t type) {
  return __nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, type);
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t c) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)c, __NV_E4M3);
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// ------------------------------------------------------------------ queries of FP8 caches

// One warp per query row: its E4M3 and E5M2 terms (codes [2][B * rows][576]) and what their
// power-of-two scale makes of a score.
constexpr int kSplitWarps = 8;
__global__ void __launch_bounds__(32 * kSplitWarps)
split_queries_kernel(int64_t rows, const uint16_t* __restrict__ q, const float* kv_scale,
                     float scale_hi, float scale_lo, uint8_t* codes, float* q_scale) {
  grid_launch_dependents();  // the main kernel sets itself up and fetches keys meanwhile
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kSplitWarps + (threadIdx.x >> 5);
  if (row >= rows) return;
  constexpr int kLoads = kDqk / 64;
  const uint32_t* src = reinterpret_cast<const uint32_t*>(q + row * kDqk);
  uint32_t x[kLoads];
  float m = 0.f;
#pragma unroll
  for (int s = 0; s < kLoads; ++s) x[s] = src[32 * s + lane];
#pragma unroll
  for (int s = 0; s < kLoads; ++s)
    m = fmaxf(m, fmaxf(fabsf(__uint_as_float(x[s] << 16)),
                       fabsf(__uint_as_float(x[s] & 0xffff0000u))));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  // 2^e brings the largest element into (224, 448]: 135 minus its exponent field makes it
  // [256, 512), halved above 448
  const uint32_t mb = __float_as_uint(m);
  int e = 135 - (int)(mb >> 23) - ((mb & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = m > 0.f ? max(-120, min(120, e)) : 0;
  const float up = __uint_as_float((uint32_t)(127 + e) << 23);
  uint16_t* hi_at = reinterpret_cast<uint16_t*>(codes + row * kDqk);
  uint16_t* lo_at = reinterpret_cast<uint16_t*>(codes + (rows + row) * kDqk);
#pragma unroll
  for (int s = 0; s < kLoads; ++s) {
    const float v0 = __uint_as_float(x[s] << 16) * up;
    const float v1 = __uint_as_float(x[s] & 0xffff0000u) * up;
    const uint32_t hi = to_f8x2(v0, v1, __NV_E4M3);
    const float2 h = from_e4m3x2(hi);
    hi_at[32 * s + lane] = (uint16_t)hi;
    lo_at[32 * s + lane] = (uint16_t)to_f8x2(v0 - h.x, v1 - h.y, __NV_E5M2);
  }
  if (lane == 0) {
    // rounded once: an error of the scale would weigh on every score alike
    const float kv = kv_scale ? *kv_scale : 1.0f;
    q_scale[row] = fmaf(kv, scale_hi, kv * scale_lo) * __uint_as_float((uint32_t)(127 - e) << 23);
  }
}

// This CTA's half of the queries of (sequence b, row group g), by one thread: slices of 128
// bytes of its rows, an FP8 row's last 64 bytes apart. Rows past the sequence's are zeros.
template <bool kFp8>
__device__ __forceinline__ void fetch_queries(const KeyWeightParams& p, const Barriers& bar,
                                              const CUtensorMap* q_map,
                                              const CUtensorMap* q_tail, uint32_t q_base, int b,
                                              int g, int cta) {
  const int half = p.cols / 2, row = g * p.group_rows + cta * half;
  const uint32_t full = smem_u32(bar.qfull);
  mbar_arrive_expect_tx(bar.qfull, (uint32_t)half * kDqk * 2);
  if (kFp8) {
    for (int term = 0; term < 2; ++term) {
      const uint32_t dst = q_base + term * half * kDqk;
      const int z = term * p.batch + b;
#pragma unroll
      for (int s = 0; s < 4; ++s) tma_load_3d(dst + s * half * 128, q_map, 128 * s, row, z, full);
      tma_load_3d(dst + 4 * half * 128, q_tail, 512, row, z, full);
    }
  } else {
    for (int s = 0; s < 9; ++s)
      tma_load_3d(q_base + s * half * 128, q_map, 64 * s, row, b, full);
  }
}

// ------------------------------------------------------------------ producers

// Three warps take the slices in turn (one thread's copies of a slice take longer to issue
// than a slice takes to multiply). Pages without a token, or in a bad block, are not read:
// their accumulator lanes are not used.
template <bool kFp8>
__device__ __forceinline__ void run_producer(const KeyWeightParams& p, const Barriers& bar,
                                             Walk w, const CUtensorMap* map, uint32_t ring,
                                             int turn, int lane) {
  constexpr int kMaxPages = 4;  // per lane: 128 pages of one token
  const int pages = p.lanes / p.page;
  const uint32_t page_bytes = p.page * 128;
  // the blocks of this lane's pages, -1 for none; read a tile ahead
  auto blocks_of = [&](const Walk& at, int (&blk)[kMaxPages]) {
#pragma unroll
    for (int i = 0; i < kMaxPages; ++i) {
      if (32 * i >= pages) break;
      const int pg = lane + 32 * i;
      const int t = at.tile * p.lanes + pg * p.page;
      blk[i] = pg < pages && t < at.n
                   ? p.block_table[(int64_t)at.b * p.max_blocks + p.block_div.div(t)]
                   : -1;
    }
  };
  int blk[kMaxPages];
  if (w.left > 0) blocks_of(w, blk);
  int st = 0;
  uint32_t phase = 0;
  int issued = 0;  // slices so far, the other warps' among them
  while (w.left > 0) {
    int row[kMaxPages], count = 0;  // the pages' first pool rows, -1 for none
#pragma unroll
    for (int i = 0; i < kMaxPages; ++i) {
      if (32 * i >= pages) break;
      const int t = w.tile * p.lanes + (lane + 32 * i) * p.page;
      const bool valid = blk[i] >= 0 && blk[i] < p.num_blocks;
      row[i] = valid ? blk[i] * p.block_size + p.block_div.mod(t) : -1;
      count += valid;
    }
    const uint32_t bytes = __reduce_add_sync(0xffffffffu, count) * page_bytes;
    const int k = w.k;
    if (w.left > 1) {
      w.advance(p);
      blocks_of(w, blk);
    } else {
      w.left = 0;
    }
    for (int s = 0; s < Shape<kFp8>::slices; ++s) {
      if (issued % kProdWarps == turn) {
        if (!wait_bar(&bar.empty[st], phase ^ 1, bar.abort_flag, p.status)) {
          w.left = 0;
          break;
        }
        const uint32_t dst = ring + st * kStageBytes, full = smem_u32(&bar.full[st]);
        const int x = s * Shape<kFp8>::dims;
        if (lane == 0) mbar_arrive_expect_tx(&bar.full[st], bytes);
#pragma unroll
        for (int i = 0; i < kMaxPages; ++i) {
          if (32 * i >= pages) break;
          for (int l = 0; l < min(32, pages - 32 * i); l += 4) {  // lanes past the last: -1
            int r[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) r[u] = __shfl_sync(0xffffffffu, row[i], l + u);
            if (elect_one()) {
#pragma unroll
              for (int u = 0; u < 4; ++u)
                if (r[u] >= 0)
                  tma_load_3d(dst + (l + u + 32 * i) * page_bytes, map, x, r[u], k, full);
            }
            __syncwarp();
          }
        }
      }
      ++issued;
      if (++st == p.stages) {
        st = 0;
        phase ^= 1;
      }
    }
  }
  // After a timeout nothing may be in flight when the CTA ends: the copies that no other warp
  // has waited for are waited for here (bounded).
  if (*reinterpret_cast<volatile int*>(bar.abort_flag) != 0) {
    for (int i = issued > p.stages ? issued - p.stages : 0; i < issued; ++i) {
      if (i % kProdWarps != turn) continue;
      wait_landed(&bar.full[i % p.stages], (uint32_t)(i / p.stages & 1));
    }
  }
}

// The odd CTA's queries, and its word to the issuer that they, and each slice, have arrived.
template <bool kFp8>
__device__ __forceinline__ void run_relay(const KeyWeightParams& p, const Barriers& bar, Walk w,
                                          const CUtensorMap* q_map, const CUtensorMap* q_tail,
                                          uint32_t q_base, int g) {
  const uint32_t peer = mapa_shared(smem_u32(&bar.peer[0]), 0);
  const uint32_t qpeer = mapa_shared(smem_u32(bar.qpeer), 0);
  int st = 0, seg_b = -1;
  uint32_t phase = 0, qphase = 0;
  while (w.left > 0) {
    if (w.b != seg_b) {
      if (seg_b >= 0 && !wait_one(bar.qfree, qphase ^ 1, bar.abort_flag, p.status)) return;
      if (seg_b < 0) {
        grid_dependency_wait();
        fence_proxy_async();
      }
      seg_b = w.b;
      fetch_queries<kFp8>(p, bar, q_map, q_tail, q_base, w.b, g, 1);
      if (!wait_one(bar.qfull, qphase, bar.abort_flag, p.status)) {
        wait_landed(bar.qfull, qphase);
        return;
      }
      qphase ^= 1;
      mbar_arrive_remote_relaxed(qpeer);
    }
    for (int s = 0; s < Shape<kFp8>::slices; ++s) {
      if (!wait_one(&bar.full[st], phase, bar.abort_flag, p.status)) return;
      mbar_arrive_remote_relaxed(peer + 8 * st);
      if (++st == p.stages) {
        st = 0;
        phase ^= 1;
      }
    }
    if (w.left > 1) w.advance(p);
    else w.left = 0;
  }
}

// ------------------------------------------------------------------ issuer

// One thread of the even CTA.
template <bool kFp8, int kBlocks>
__device__ __forceinline__ void run_issuer(const KeyWeightParams& p, const Barriers& bar, Walk w,
                                           const CUtensorMap* q_map, const CUtensorMap* q_tail,
                                           uint32_t q_base, uint32_t ring, uint32_t tbase,
                                           int g) {
  constexpr int kSlices = Shape<kFp8>::slices;
  const uint32_t half = p.cols / 2;
  const uint32_t idesc = kFp8 ? idesc_f8(kTileRows, p.cols, false)
                              : idesc_f16(kTileRows, p.cols, true, false);
  const uint32_t idesc_lo = idesc_f8(kTileRows, p.cols, true);
  // descriptors of the first slices; an address step of n bytes adds n / 16
  const uint64_t ring_desc = smem_desc_sw128(ring, 16, 1024);
  const uint64_t q_desc = smem_desc_sw128(q_base, 16, 1024);
  const uint64_t q_last = smem_desc_sw64(q_base + (kSlices - 1) * half * 128, 512);
  const uint32_t q_step = half * 128 / 16, lo_step = half * kDqk / 16;
  // the sums of a tile side by side in one buffer, or in turn in two
  constexpr int sums = Shape<kFp8>::sums(32 * kBlocks);
  constexpr bool in_turn = !kFp8 && kBlocks > 4;
  const int bufs = buffers(kFp8, p.cols);
  const uint32_t buf_step = kTmemCols / bufs, sum_step = in_turn ? 0 : buf_step / sums;
  int st = 0, buf = 0, seg_b = -1;
  uint32_t phase = 0, dphase = 0, qphase = 0;
  while (w.left > 0) {
    if (w.b != seg_b) {
      if (seg_b >= 0) {
        tc_commit_pair(bar.qfree);
        if (!wait_one(bar.qfree, qphase ^ 1, bar.abort_flag, p.status)) break;
      } else {
        grid_dependency_wait();
        fence_proxy_async();
      }
      seg_b = w.b;
      fetch_queries<kFp8>(p, bar, q_map, q_tail, q_base, w.b, g, 0);
      if (!wait_one(bar.qfull, qphase, bar.abort_flag, p.status)) {
        wait_landed(bar.qfull, qphase);
        break;
      }
      if (!wait_one(bar.qpeer, qphase, bar.abort_flag, p.status)) break;
      qphase ^= 1;
    }
    bool ok = true;
    uint32_t d = 0;
    // unrolled, what the slices' places decide is decided here (FP8, 16 rows: 98.2 us, in a loop
    // 100.4), but not where the sums take turns (BF16, 288 rows: 36.1 us, unrolled 40.4)
#pragma unroll(in_turn ? 1 : kSlices)
    for (int s = 0; s < kSlices; ++s) {
      const bool begins = s == 0 || Shape<kFp8>::ends_sum(s - 1, sums);  // a sum
      const bool enters = s == 0 || (begins && in_turn);                 // a buffer
      ok = (!enters || wait_one(&bar.dempty[buf], dphase ^ 1, bar.abort_flag, p.status)) &&
           wait_one(&bar.full[st], phase, bar.abort_flag, p.status) &&
           wait_one(&bar.peer[st], phase, bar.abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      d = enters ? tbase + buf * buf_step : begins ? d + sum_step : d;
      const uint64_t a = ring_desc + st * (kStageBytes / 16);
      if (!kFp8) {
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_f16_ss_pair(d, a + 2 * kk, q_desc + s * q_step + 2 * kk, idesc, !begins || kk > 0);
      } else if (s < kSlices - 1) {
        const uint64_t q = q_desc + s * q_step;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          mma_f8_ss_pair(d, a + 2 * kk, q + 2 * kk, idesc, !begins || kk > 0);
          mma_f8_ss_pair(d, a + 2 * kk, q + lo_step + 2 * kk, idesc_lo, 1);
        }
      } else {  // the last 64 dims: q's rows are 64 bytes
#pragma unroll
        for (int kk = 0; kk < 2; ++kk) {
          mma_f8_ss_pair(d, a + 2 * kk, q_last + 2 * kk, idesc, 1);
          mma_f8_ss_pair(d, a + 2 * kk, q_last + lo_step + 2 * kk, idesc_lo, 1);
        }
      }
      tc_commit_pair(&bar.empty[st]);
      if (++st == p.stages) {
        st = 0;
        phase ^= 1;
      }
      if (s == kSlices - 1 || (in_turn && Shape<kFp8>::ends_sum(s, sums))) {
        tc_commit_pair(&bar.dfull[buf]);
        if (++buf == bufs) {
          buf = 0;
          dphase ^= 1;
        }
      }
    }
    if (!ok) break;
    if (w.left > 1) w.advance(p);
    else w.left = 0;
  }
  // every product is done before the accumulators are freed and shared memory is left
  tc_commit_pair(bar.drain);
}

// ------------------------------------------------------------------ epilogue

// Scales and negated offsets of the group's columns for the sums of this CTA's tokens: two
// columns are 16 bytes, both scales, then both offsets.
template <bool kFp8>
__device__ __forceinline__ void load_params(const KeyWeightParams& p, int b, int g,
                                            float* params) {
  const int c = threadIdx.x;  // an epilogue thread per column
  if (c >= p.cols) return;
  const int row = g * p.group_rows + c;
  float scale = 0.f, lse = -INFINITY;
  if (c < p.group_rows && row < p.rows) {
    const int64_t at = (int64_t)b * p.rows + row;
    lse = p.lse[at];
    scale = kFp8 ? p.q_scale[at]
                 : (p.kv_scale ? fmaf(*p.kv_scale, p.scale_hi, *p.kv_scale * p.scale_lo)
                               : p.scale_hi);
  }
  params[4 * (c >> 1) + (c & 1)] = scale;
  // a row of -inf LSE attended nothing and adds nothing: 2^(0 - inf)
  params[4 * (c >> 1) + 2 + (c & 1)] =
      lse == -INFINITY ? -INFINITY : -fmaf(lse, kLog2eHi, lse * kLog2eLo);
}

// Two floats in a 64-bit register pair.
__device__ __forceinline__ uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpack2(uint64_t x) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(x));
  return f;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Sum over 16 columns of 2^(r * scale - offset), two at a time; kMasked: of those from
// `first` on.
template <bool kMasked>
__device__ __forceinline__ void add_columns(const uint32_t (&r)[16], const ulonglong2* col,
                                            int first, uint64_t& s0, uint64_t& s1) {
#pragma unroll
  for (int i = 0; i < 16; i += 2) {
    const ulonglong2 ab = col[i / 2];
    const float2 x = unpack2(
        fma2(pack2(__uint_as_float(r[i]), __uint_as_float(r[i + 1])), ab.x, ab.y));
    float e0 = exp2_fast(x.x), e1 = exp2_fast(x.y);
    if (kMasked) {
      e0 = i >= first ? e0 : 0.f;
      e1 = i + 1 >= first ? e1 : 0.f;
    }
    if (i & 2) s1 = add2(s1, pack2(e0, e1));
    else s0 = add2(s0, pack2(e0, e1));
  }
}

template <bool kMasked>
__device__ __forceinline__ float sum_columns(uint32_t trow, const ulonglong2* col, int cols,
                                             int first) {
  uint64_t s0 = 0, s1 = 0;
  uint32_t ra[16], rb[16];  // the next 16 columns load while these are summed
  tmem_ld16(trow, ra);
  for (int c = 0; c < cols; c += 32) {
    tmem_wait_ld16(ra);
    if (c + 16 < cols) tmem_ld16(trow + c + 16, rb);
    add_columns<kMasked>(ra, col + c / 2, first - c, s0, s1);
    if (c + 16 >= cols) break;
    tmem_wait_ld16(rb);
    if (c + 32 < cols) tmem_ld16(trow + c + 32, ra);
    add_columns<kMasked>(rb, col + c / 2 + 8, first - c - 16, s0, s1);
  }
  const float2 a = unpack2(s0), b = unpack2(s1);
  return (a.x + a.y) + (b.x + b.y);
}

__device__ __forceinline__ void add16(uint32_t (&x)[16], const uint32_t (&y)[16]) {
#pragma unroll
  for (int e = 0; e < 16; e += 2) {
    const float2 s = unpack2(add2(pack2(__uint_as_float(x[e]), __uint_as_float(x[e + 1])),
                                  pack2(__uint_as_float(y[e]), __uint_as_float(y[e + 1]))));
    x[e] = __float_as_uint(s.x);
    x[e + 1] = __float_as_uint(s.y);
  }
}
// The same over a tile's sums, `step` columns apart.
template <bool kMasked, int kSums>
__device__ __forceinline__ float sum_side_by_side(uint32_t trow, uint32_t step,
                                                  const ulonglong2* col, int cols, int first) {
  uint64_t s0 = 0, s1 = 0;
  for (int c = 0; c < cols; c += 16) {
    uint32_t r[kSums][16];
#pragma unroll
    for (int i = 0; i < kSums; ++i) tmem_ld16(trow + i * step + c, r[i]);
#pragma unroll
    for (int i = 0; i < kSums; ++i) tmem_wait_ld16(r[i]);
#pragma unroll
    for (int o = 1; o < kSums; o *= 2)
#pragma unroll
      for (int i = 0; i < kSums; i += 2 * o) add16(r[i], r[i + o]);
    add_columns<kMasked>(r[0], col + c / 2, first - c, s0, s1);
  }
  const float2 a = unpack2(s0), b = unpack2(s1);
  return (a.x + a.y) + (b.x + b.y);
}

// And over two sums, the first held in registers until the second is there.
template <int kBlocks>
__device__ __forceinline__ void hold_sum(uint32_t (&held)[kBlocks][16], uint32_t trow, int cols) {
#pragma unroll
  for (int i = 0; i < kBlocks; ++i)
    if (16 * i < cols) tmem_ld16(trow + 16 * i, held[i]);
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) tmem_wait_ld16(held[i]);
}
template <int kBlocks>
__device__ __forceinline__ void add_sum(uint32_t (&held)[kBlocks][16], uint32_t trow, int cols) {
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if (16 * i >= cols) break;
    uint32_t r[16];
    tmem_ld16(trow + 16 * i, r);
    tmem_wait_ld16(r);
    add16(held[i], r);
  }
}
template <bool kMasked, int kBlocks>
__device__ __forceinline__ float sum_held_columns(const uint32_t (&held)[kBlocks][16],
                                                  const ulonglong2* col, int cols, int first) {
  uint64_t s0 = 0, s1 = 0;
#pragma unroll
  for (int i = 0; i < kBlocks; ++i) {
    if (16 * i >= cols) break;
    add_columns<kMasked>(held[i], col + 8 * i, first - 16 * i, s0, s1);
  }
  const float2 a = unpack2(s0), b = unpack2(s1);
  return (a.x + a.y) + (b.x + b.y);
}

// Position of local token t among the step's own tokens: row j sees it from j = place on.
__device__ __forceinline__ int place_of(const KeyWeightParams& p, const Lengths& len, int k,
                                        int t) {
  const int run = p.interleave_div.div(t);
  return (int)(((int64_t)run * p.dcp + p.rank_begin + k) * p.interleave +
               (t - run * p.interleave) - len.old);
}

template <bool kFp8, int kBlocks>
__device__ __forceinline__ void run_epilogue(const KeyWeightParams& p, const Barriers& bar,
                                             Walk w, float* params, float* tokens,
                                             uint32_t tbase, int g, int warp, int lane) {
  const int half = warp >> 2;  // of the columns; the first half's warps write the sums
  const int row = (warp & 3) * 32 + lane;
  int buf = 0, seg_b = -1, slot = 0, odd = 0;
  uint32_t dphase = 0;
  const uint32_t dempty = mapa_shared(smem_u32(&bar.dempty[0]), 0);
  const int cols = p.cols / 2;
  const int bufs = buffers(kFp8, p.cols);
  const uint32_t stride = kTmemCols / bufs;
  // the tiles' block ids and histories of this thread's token, kAhead tiles ahead of their
  // use: behind the copies in flight a load takes several microseconds
  volatile float* history = tokens + row;
  volatile int* block = reinterpret_cast<int*>(tokens) + (kAhead + 1) * 128 + row;
  volatile float* other = tokens + 2 * (kAhead + 1) * 128 + row;
  Walk ahead = w;
  int ahead_slot = 0;
  auto fetch = [&]() {
    if (ahead.left > 0) {
      const int t = ahead.tile * p.lanes + row;
      if (row < p.lanes && t < ahead.n) {
        cp_async4(smem_u32(const_cast<int*>(block + ahead_slot * 128)),
                  p.block_table + (int64_t)ahead.b * p.max_blocks + p.block_div.div(t));
        if (p.groups == 1 && place_of(p, ahead.len, ahead.k, t) < 0)
          cp_async4(smem_u32(const_cast<float*>(history + ahead_slot * 128)),
                    p.w_in + ((int64_t)ahead.k * p.batch + ahead.b) * p.max_local_len + t);
      }
      if (ahead.left > 1) ahead.advance(p);
      else ahead.left = 0;
    }
    cp_async_commit();
    ahead_slot = ahead_slot == kAhead ? 0 : ahead_slot + 1;
  };
  if (half == 0)
    for (int i = 0; i < kAhead; ++i) fetch();
  uint32_t bad = 0;
  while (w.left > 0) {
    if (w.b != seg_b) {
      // the last tile's barrier is behind every warp's sums with the last parameters
      if (seg_b < 0) grid_dependency_wait();
      seg_b = w.b;
      load_params<kFp8>(p, w.b, g, params);
      named_bar_sync(1, 32 * kEpiWarps);
    }
    if (half == 0) fetch();
    const int t = w.tile * p.lanes + row;
    const bool live = row < p.lanes && t < w.n;
    const int place = live ? place_of(p, w.len, w.k, t) : 0;
    // the first column (row of the group) that sees the token
    const int first = p.causal && place > 0 ? place * p.H - g * p.group_rows : 0;
    // After a timeout the loop goes on without waiting, so that both halves' warps come to
    // every barrier below; nothing is written.
    bool ok = true;
    const ulonglong2* col = reinterpret_cast<const ulonglong2*>(params) + half * cols / 2;
    const uint32_t trow = tbase + half * cols + ((uint32_t)((warp & 3) * 32) << 16);
    const bool masked = __any_sync(0xffffffffu, first > half * cols);
    auto wait_sum = [&]() {
      ok = wait_bar(&bar.dfull[buf], dphase, bar.abort_flag, p.status) && ok;
      tc_fence_after();
    };
    auto free_sum = [&]() {
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_remote_relaxed(dempty + 8 * buf);
      if (++buf == bufs) {
        buf = 0;
        dphase ^= 1;
      }
    };
    float sum;
    constexpr int kSums = Shape<kFp8>::sums(32 * kBlocks);
    if (kBlocks == 4) {
      wait_sum();
      const uint32_t at = trow + buf * stride, step = stride / kSums;
      sum = masked ? sum_side_by_side<true, kSums>(at, step, col, cols, first - half * cols)
                   : sum_side_by_side<false, kSums>(at, step, col, cols, 0);
      free_sum();
    } else if (kFp8) {
      wait_sum();
      sum = masked ? sum_columns<true>(trow + buf * stride, col, cols, first - half * cols)
                   : sum_columns<false>(trow + buf * stride, col, cols, 0);
      free_sum();
    } else {
      uint32_t held[kBlocks][16];
      wait_sum();
      hold_sum(held, trow + buf * stride, cols);
      free_sum();
      wait_sum();
      add_sum(held, trow + buf * stride, cols);
      free_sum();
      sum = masked ? sum_held_columns<true>(held, col, cols, first - half * cols)
                   : sum_held_columns<false>(held, col, cols, 0);
    }
    if (half == 1) other[odd * 128] = sum;
    named_bar_sync(1, 32 * kEpiWarps);
    if (half == 0) {
      cp_async_wait_group<kAhead>();
      if (live && ok) {
        sum += other[odd * 128];
        const int blk = block[slot * 128];
        const int64_t at = ((int64_t)w.k * p.batch + w.b) * p.max_local_len + t;
        if (blk < 0 || blk >= p.num_blocks) {
          bad |= DCP_STATUS_BAD_BLOCK_ID;
        } else if (p.groups == 1) {
          p.w_out[at] = place < 0 ? fmaf(p.decay, history[slot * 128], sum) : sum;
        } else {
          p.part[(int64_t)g * p.num_ranks * p.batch * p.max_local_len + at] = sum;
        }
      }
      slot = slot == kAhead ? 0 : slot + 1;
    }
    odd ^= 1;
    if (w.left > 1) w.advance(p);
    else w.left = 0;
  }
  cp_async_wait_all();
  if (bad) raise_status(p.status, bad);
}

// kBlocks: 16 columns each, as many as half of the product has, or more.
template <bool kFp8, int kBlocks>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    key_weights_kernel(const KeyWeightParams p, const __grid_constant__ CUtensorMap map,
                       const __grid_constant__ CUtensorMap q_map,
                       const __grid_constant__ CUtensorMap q_tail) {
  extern __shared__ unsigned char smem_raw[];
  uint8_t* base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  const Layout lay = layout_of(p.cols, p.stages);
  float* params = reinterpret_cast<float*>(base + lay.params);
  Barriers bar;
  bar.full = reinterpret_cast<uint64_t*>(base + lay.bars);
  bar.peer = bar.full + kMaxStages;
  bar.empty = bar.peer + kMaxStages;
  bar.dfull = bar.empty + kMaxStages;
  bar.dempty = bar.dfull + 2;
  bar.qfull = bar.dempty + 2;
  bar.qpeer = bar.qfull + 1;
  bar.qfree = bar.qpeer + 1;
  bar.drain = bar.qfree + 1;
  bar.tmem_slot = reinterpret_cast<uint32_t*>(bar.drain + 1);
  bar.abort_flag = reinterpret_cast<int*>(bar.tmem_slot + 1);
  __shared__ int s_sum[kThreads / 32];
  __shared__ int s_b, s_skip, s_of, s_share;
  __shared__ Lengths s_len;
  const int tid = threadIdx.x, lane = tid & 31;
  const int warp = __shfl_sync(0xffffffffu, tid >> 5, 0);
  const int cta = (int)cluster_ctarank();
  // neighbouring pairs take the row groups of the same tiles
  const int g = (blockIdx.x >> 1) % p.groups;
  const int pair = (blockIdx.x >> 1) / p.groups, pairs = (gridDim.x >> 1) / p.groups;

  if (tid == 0) {
    tma_prefetch_map(&map);
    tma_prefetch_map(&q_map);
    if (kFp8) tma_prefetch_map(&q_tail);
    for (int i = 0; i < p.stages; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.peer[i], 1);
      mbar_init(&bar.empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.dfull[i], 1);
      mbar_init(&bar.dempty[i], 2 * kEpiWarps);
    }
    mbar_init(bar.qfull, 1);
    mbar_init(bar.qpeer, 1);
    mbar_init(bar.qfree, 1);
    mbar_init(bar.drain, 1);
    *bar.abort_flag = 0;
    fence_mbarrier_init_cluster();
  }
  if (warp == kMmaWarp) {
    tmem_alloc_pair(bar.tmem_slot, kTmemCols);
    tmem_relinquish_pair();
  }

  // tiles of every sequence (all ranks), and bad lengths
  auto seq_tiles = [&](int b, Lengths& len) -> int {
    len = lengths_of(p, b);
    if (blockIdx.x == 0) {
      uint32_t bad = 0;
      if (p.seq_lens[b] < 0 || (p.causal && len.old < 0)) bad |= DCP_STATUS_BAD_SEQ_LEN;
      const int64_t r = len.rem - (int64_t)p.rank_begin * p.interleave;
      if (len.whole + min(max(r, (int64_t)0), (int64_t)p.interleave) > p.max_local_len)
        bad |= DCP_STATUS_LOCAL_OVER_BOUND;
      if (bad) raise_status(p.status, bad);
    }
    return pair_tiles(p, len);
  };
  const bool few = p.batch <= 32;  // one warp holds every sequence
  Lengths len = {};
  int mine = 0;
  if (!few || warp == 0)
    for (int b = tid; b < p.batch; b += kThreads) mine += seq_tiles(b, len);
  int sum = mine;
  if (!few) {
    sum = __reduce_add_sync(0xffffffffu, sum);
    if (lane == 0) s_sum[warp] = sum;
    __syncthreads();
    sum = lane < kThreads / 32 ? s_sum[lane] : 0;
  }
  if (warp == 0) {
    sum = __reduce_add_sync(0xffffffffu, sum);
    // equal shares, the first ones a tile longer; and the sequence in which this one begins,
    // 32 sequences at a time
    const int each = p.pairs_div.div(sum), more = sum - each * pairs;
    const int lo = each * pair + min(pair, more);
    int before = 0;
    bool found = false;
    if (lane == 0) s_share = each + (pair < more ? 1 : 0);
    for (int b0 = 0; b0 < p.batch && !found; b0 += 32) {
      const int n = few ? mine : b0 + lane < p.batch ? seq_tiles(b0 + lane, len) : 0;
      int incl = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
      }
      const bool here = before + incl - n <= lo && lo < before + incl;
      if (here) {
        s_b = b0 + lane;
        s_skip = lo - (before + incl - n);
        s_of = n;
        s_len = len;
      }
      found = __any_sync(0xffffffffu, here);
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
  }
  tc_fence_before();
  __syncthreads();
  // this CTA's barriers are ready for the peer; a warp waits for the peer's where it first
  // needs them: the producers never do
  cluster_arrive();
  tc_fence_after();
  const uint32_t tbase = __shfl_sync(0xffffffffu, *bar.tmem_slot, 0);
  Walk w;
  w.start(p, cta, s_b, s_len, s_skip, s_of, s_share);
  const uint32_t q_base = smem_u32(base), ring = q_base + lay.q_bytes;
  if (warp < kEpiWarps) {
    cluster_wait();
    run_epilogue<kFp8, kBlocks>(p, bar, w, params, reinterpret_cast<float*>(base + lay.tokens),
                              tbase, g, warp, lane);
  } else if (warp >= kProdWarp0) {
    run_producer<kFp8>(p, bar, w, &map, ring, warp - kProdWarp0, lane);
    cluster_wait();
  } else if (cta == 0) {
    cluster_wait();
    if (elect_one()) run_issuer<kFp8, kBlocks>(p, bar, w, &q_map, &q_tail, q_base, ring, tbase, g);
    __syncwarp();
  } else {
    cluster_wait();
    if (elect_one()) run_relay<kFp8>(p, bar, w, &q_map, &q_tail, q_base, g);
    __syncwarp();
  }
  if (warp == kMmaWarp) wait_bar(bar.drain, 0, bar.abort_flag, p.status);
  // the kernel that adds the row groups may set itself up beside the last pairs of CTAs
  grid_launch_dependents();
  grid_dependency_wait();  // also where there was no tile: this grid ends after the one before
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();  // the peer no longer touches this CTA's shared memory
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tbase, kTmemCols);
  }
}

// The row groups' sums of every token, in order, onto its history. Four tokens of a thread in
// flight; what does not come from the main kernel is read while that one ends (7 sequences of
// 1549 tokens, 512 rows: 18.5 us together, with a token at a time and no overlap 22.6).
constexpr int kAddThreads = 256, kAddPer = 4;
__global__ void __launch_bounds__(kAddThreads) key_weights_add_kernel(const KeyWeightParams p) {
  const int pair = blockIdx.x, b = pair % p.batch, k = pair / p.batch;
  const Lengths len = lengths_of(p, b);
  const int n = rank_len(p, len, k);
  const int64_t row = (int64_t)pair * p.max_local_len;
  const int64_t step = (int64_t)p.num_ranks * p.batch * p.max_local_len;
  for (int t0 = blockIdx.y * (kAddThreads * kAddPer); t0 < n;
       t0 += gridDim.y * (kAddThreads * kAddPer)) {
    float sum[kAddPer], w[kAddPer];
    bool live[kAddPer];
#pragma unroll
    for (int u = 0; u < kAddPer; ++u) {
      const int t = t0 + u * kAddThreads + threadIdx.x;
      const int blk =
          t < n ? p.block_table[(int64_t)b * p.max_blocks + p.block_div.div(t)] : -1;
      live[u] = blk >= 0 && blk < p.num_blocks;  // others are reported by the main kernel
      w[u] = live[u] && place_of(p, len, k, t) < 0 ? p.w_in[row + t] : 0.f;
      sum[u] = 0.f;
    }
    grid_dependency_wait();
    for (int g = 0; g < p.groups; ++g)
#pragma unroll
      for (int u = 0; u < kAddPer; ++u)
        if (live[u]) sum[u] += p.part[g * step + row + t0 + u * kAddThreads + threadIdx.x];
#pragma unroll
    for (int u = 0; u < kAddPer; ++u)
      if (live[u]) p.w_out[row + t0 + u * kAddThreads + threadIdx.x] = fmaf(p.decay, w[u], sum[u]);
  }
  grid_dependency_wait();  // also where there was no token: this grid ends after the one before
}

// Tensor map over rows of 576 elements [outer][rows], boxes of `width` bytes of `height` rows.
cudaError_t row_map(CUtensorMap* map, const void* base, bool bytes, int64_t rows, int64_t outer,
                    int width, int height) {
  static PFN_cuTensorMapEncodeTiled_v12000 encode = nullptr;
  if (encode == nullptr) {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult found;
    const cudaError_t e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000,
                                                           cudaEnableDefault, &found);
    if (e != cudaSuccess) return e;
    if (found != cudaDriverEntryPointSuccess) return cudaErrorNotSupported;
    encode = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(fn);
  }
  const cuuint64_t row_bytes = bytes ? kDqk : 2 * kDqk;
  const cuuint64_t dims[3] = {kDqk, (cuuint64_t)rows, (cuuint64_t)outer};
  const cuuint64_t strides[2] = {row_bytes, row_bytes * (cuuint64_t)rows};
  const cuuint32_t box[3] = {(cuuint32_t)(bytes ? width : width / 2), (cuuint32_t)height, 1u};
  const cuuint32_t steps[3] = {1, 1, 1};
  const CUresult r =
      encode(map, bytes ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3,
             const_cast<void*>(base), dims, strides, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
             width == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
             CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}

// Tokens of one copy: a run of a block's tokens, so that few copies fill the 128 lanes (a
// copy takes some 200 cycles of a warp to issue, as long as four lanes' share of a slice's
// products takes) and few lanes stay empty: 5 runs of 24 for blocks of 24, 25 of 5 for
// blocks of 5, 4 of 32 for blocks of 96.
int page_tokens(int block_size) {
  int best = 1;
  auto score = [](int d) { return 128 / d * d - 4 * (128 / d); };
  for (int d = 2; d <= std::min(block_size, 128); ++d)
    if (block_size % d == 0 && score(d) > score(best)) best = d;
  return best;
}

int row_groups(const dcp_mla_dims& d) { return (d.qlen * d.num_heads + kMaxCols - 1) / kMaxCols; }

// Workspace: the row groups' sums, then the queries' two terms and scales (FP8 caches).
struct Workspace {
  size_t codes, scales, total;
};
Workspace workspace_of(const dcp_mla_dims& d, int num_ranks) {
  const int groups = row_groups(d);
  const size_t rows = (size_t)d.batch * d.qlen * d.num_heads;
  Workspace w;
  w.codes = groups == 1 ? 0
                        : ((size_t)groups * num_ranks * d.batch * d.max_local_len *
                               sizeof(float) + 127) / 128 * 128;
  w.scales = w.codes + rows * kDqk * 2;
  w.total = (w.scales + rows * sizeof(float) + 15) / 16 * 16;
  return w;
}

}  // namespace

size_t key_weights_workspace_bytes(const dcp_mla_dims& d, int num_ranks) {
  return std::max<size_t>(16, workspace_of(d, num_ranks).total);
}

cudaError_t launch_key_weights(const dcp_mla_dims& d, const int32_t* seq_lens,
                               const int32_t* block_table, const void* q, const void* kv,
                               dcp_kv_dtype kv_dtype, const float* kv_scale, float softmax_scale,
                               const float* lse, float decay, int rank_begin, int num_ranks,
                               const float* weights_in, float* weights_out, void* workspace,
                               uint32_t* status, cudaStream_t stream) {
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3;
  KeyWeightParams p;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.kv_scale = kv_scale;
  p.lse = lse;
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.part = static_cast<float*>(workspace);
  p.status = status;
  const double scale = (double)softmax_scale * 1.4426950408889634;
  p.scale_hi = (float)scale;
  p.scale_lo = (float)(scale - (double)p.scale_hi);
  p.decay = decay;
  p.batch = d.batch;
  p.qlen = d.qlen;
  p.H = d.num_heads;
  p.dcp = d.dcp;
  p.interleave = d.interleave;
  p.block_size = d.block_size;
  p.max_blocks = d.max_blocks_per_seq;
  p.max_local_len = d.max_local_len;
  p.num_blocks = d.num_blocks;
  p.causal = d.causal;
  p.rank_begin = rank_begin;
  p.num_ranks = num_ranks;
  p.groups = row_groups(d);
  p.group_rows = (d.qlen * d.num_heads + p.groups - 1) / p.groups;
  p.cols = (p.group_rows + 31) / 32 * 32;
  const Layout none = layout_of(p.cols, 0);
  p.stages = std::min(kMaxStages, (kSmemLimit - 512 - none.total) / kStageBytes);
  p.page = page_tokens(d.block_size);
  p.lanes = 128 / p.page * p.page;
  p.half_div = FastDiv::by(p.lanes);
  p.rows = d.qlen * d.num_heads;
  p.block_div = FastDiv::by(d.block_size);
  p.interleave_div = FastDiv::by(d.interleave);
  const int smem = layout_of(p.cols, p.stages).total;
  const int pairs_max = partial_concurrent_items();
  if (pairs_max < 1) return cudaErrorInvalidConfiguration;
  const int64_t halves = (int64_t)num_ranks * (((int64_t)d.max_local_len + p.lanes - 1) / p.lanes);
  const int64_t bound = (halves + 1) / 2 * d.batch;
  const int pairs =
      p.groups * (int)std::min<int64_t>(std::max(1, pairs_max / p.groups), bound);
  if (halves > INT32_MAX || bound > INT32_MAX) return cudaErrorInvalidConfiguration;
  p.pairs_div = FastDiv::by(pairs / p.groups);
  // What a thread holds is sized by the columns, as 128 sums do not all stay in its registers
  // (15 sequences of up to 15000 tokens, 288 rows, products of 160 columns: 44.2 us, held as
  // 128 48.3)
  const int which = p.cols <= 128 ? (fp8 ? 0 : 1) : fp8 ? 2 : p.cols <= 192 ? 3 : 4;
  auto kern = which == 0   ? key_weights_kernel<true, 4>
              : which == 1 ? key_weights_kernel<false, 4>
              : which == 2 ? key_weights_kernel<true, 8>
              : which == 3 ? key_weights_kernel<false, 6>
                           : key_weights_kernel<false, 8>;
  static bool attr_set[5][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  if (!attr_set[which][dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemLimit - 512);
    if (e != cudaSuccess) return e;
    attr_set[which][dev] = true;
  }
  const Workspace ws = workspace_of(d, num_ranks);
  uint8_t* codes = static_cast<uint8_t*>(workspace) + ws.codes;
  float* q_scale = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + ws.scales);
  p.q_scale = q_scale;
  CUtensorMap map, q_map, q_tail;
  e = row_map(&map, kv, fp8, (int64_t)d.num_blocks * d.block_size, num_ranks, 128, p.page);
  if (e == cudaSuccess)
    e = row_map(&q_map, fp8 ? static_cast<const void*>(codes) : q, fp8, p.rows,
                fp8 ? 2 * (int64_t)d.batch : d.batch, 128, p.cols / 2);
  q_tail = q_map;
  if (e == cudaSuccess && fp8)
    e = row_map(&q_tail, codes, true, p.rows, 2 * (int64_t)d.batch, 64, p.cols / 2);
  if (e != cudaSuccess) return e;
  if (fp8) {
    const int64_t rows = (int64_t)d.batch * p.rows;
    split_queries_kernel<<<(unsigned)((rows + kSplitWarps - 1) / kSplitWarps), 32 * kSplitWarps,
                           0, stream>>>(rows, p.q, kv_scale, p.scale_hi, p.scale_lo, codes,
                                        q_scale);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  // behind split_queries_kernel, the launch overlaps it
  e = launch_overlapping(fp8, kern, dim3(2 * pairs), dim3(kThreads), smem, stream, p, map, q_map,
                         q_tail);
  if (e != cudaSuccess || p.groups == 1) return e;
  constexpr int kPer = kAddThreads * kAddPer;
  const dim3 grid((unsigned)(num_ranks * d.batch),
                  (unsigned)std::min(1024, (d.max_local_len - 1) / kPer + 1));
  return launch_overlapping(true, key_weights_add_kernel, grid, dim3(kAddThreads), 0, stream, p);
}

}  // namespace dcpmla
