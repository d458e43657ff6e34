// Grouped-head K/V caches: the new tokens' rows into the pools, and the attention of the
// newest tokens over them, split over the cache's length and joined.
//
// For query head h of row (b, j) with K/V head g = h / group, over the tokens t that the
// row sees on the call's ranks,
//   s_t = softmax_scale * k_scale * log2(e) * (q . k_t)          (base 2)
//   O = v_scale * sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m),  LSE = (m + log2 sum) ln 2,
// with a running maximum m. Scores, m, l and O are held in 32 bits. The weights 2^(s - m) are
// rounded to the second product's 16-bit operands, as its matrix instructions take no others
// at this rate: bf16 (half a step, 2^-9 to 2^-8 of each), or f16 beside an FP8 cache's codes,
// which f16 holds exactly. f16 has few exponents, so there the weights, their sum l and O are
// formed 2^15 times as large (the largest f16 is 2^16): from 2^-29 of the largest weight up each
// is off by at most 2^-12 to 2^-11, below by at most 2^-40 of the largest. Without the factor
// weights below 2^-25 would be lost from O, but not from l. A second 16-bit term for what the
// rounding leaves would bring the error of O from 2.1e-3 (BF16; FP8 1.68e-3) to 1.66e-3, which
// is the rounding of the output itself, for 3 to 19% of the time (FP8 9 to 26%).
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"
#include "sm103.cuh"

namespace dcpmla {
namespace {

using namespace sm103;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------ write

// Memory-bound. One warp per row and pool (K or V): it finds the ranks that take the row
// (one, as a rule; a thread per element and rank spends most threads on finding that its
// rank does not: 46 against 33 us for 20000 rows of 1024 elements on four ranks) and copies
// its 16-byte pieces, four in flight (29 us; eight take the registers of half the warps).
// The rows are read once, so their loads leave first what L2 holds of them (26 us; the pools'
// new rows stay for the attention that reads them). Where the call has every rank, some rank
// takes the row, and its first pieces are read while the rank is looked up (24.8 us, 5.0 TB/s;
// with inputs that are in no cache 26.9). The divisions of the FP8 codes are 5 us of that; the
// floor of memory is 18.1 us.
constexpr int kWriteWarps = 4;

template <bool kFp8>
__global__ void __launch_bounds__(32 * kWriteWarps)
gqa_write_kernel(int rows, int num_ranks, int all_ranks, int row_elems, int64_t pool_rows,
                 const int32_t* __restrict__ slot_mapping, const uint16_t* __restrict__ k_new,
                 const uint16_t* __restrict__ v_new, const float* k_scale, const float* v_scale,
                 uint8_t* k_pool, uint8_t* v_pool, uint32_t* status) {
  const int lane = threadIdx.x & 31;
  const int64_t i = (int64_t)blockIdx.x * kWriteWarps + (threadIdx.x >> 5);
  const int row = (int)(i >> 1);
  if (row >= rows) return;
  const bool is_v = i & 1;
  const uint4* src = reinterpret_cast<const uint4*>((is_v ? v_new : k_new) +
                                                    (int64_t)row * row_elems);
  uint8_t* pool = is_v ? v_pool : k_pool;
  const float* scale_at = is_v ? v_scale : k_scale;
  const float scale = kFp8 && scale_at ? *scale_at : 1.0f;
  const int pieces = row_elems / 8;
  uint4 x[4];
  auto load = [&](int c0) {
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (c0 + 32 * u < pieces) x[u] = __ldcs(src + c0 + 32 * u);
  };
  if (all_ranks) load(lane);
  for (int k0 = 0; k0 < num_ranks; k0 += 32) {
    int32_t slot = k0 + lane < num_ranks ? slot_mapping[(int64_t)(k0 + lane) * rows + row] : -1;
    if (slot < -1 || slot >= pool_rows) {
      if (!is_v) raise_status(status, DCP_STATUS_BAD_PAGE);
      slot = -1;
    }
    unsigned owners = __ballot_sync(0xffffffffu, slot >= 0);
    while (owners != 0u) {
      const int r = __ffs(owners) - 1;
      owners &= owners - 1u;
      const int64_t at = ((int64_t)(k0 + r) * pool_rows + __shfl_sync(0xffffffffu, slot, r)) * pieces;
      for (int c0 = lane; c0 < pieces; c0 += 4 * 32) {
        if (pieces > 4 * 32 || !all_ranks) load(c0);
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (c0 + 32 * u >= pieces) break;
          if (kFp8) reinterpret_cast<uint2*>(pool)[at + c0 + 32 * u] = quantize8(x[u], scale);
          else reinterpret_cast<uint4*>(pool)[at + c0 + 32 * u] = x[u];
        }
      }
    }
  }
}

// ------------------------------------------------------------------ decode
//
// Memory-bound for up to 16 query rows per K/V head of 128 dims and enough tokens to fill the
// device: every K and V row is read once, and 4 * 16 * head_dim products per token and K/V head
// are a third of what mma.sync gives at that rate, so the warp-level products serve: a warp's 16
// query rows fill one of their tiles, where a tcgen05 tile would be 128 rows of which the others
// are empty. Beyond that it is bound by instructions: every warp of a team converts the whole
// tile for its own 16 rows (7 sequences of 10915 tokens, FP8: 16 K/V heads with 32 rows 102 us,
// floor 46; 4 K/V heads with 64 rows 60 us, floor 12), and 64 dims have twice the scores and
// exponentials to a byte (26 ragged sequences of up to 10925 tokens, 8 K/V heads with 16 rows:
// FP8 45 us, floor 20; BF16 58 us, floor 40).
//
// A CTA's eight warps share `heads` K/V heads (kWarps / heads warps each) of the same
// tokens, so that the rows of neighbouring heads are read together. A warp keeps its
// queries and its running (m, l, O) in registers and streams K and V tiles of kTok tokens
// through a ring of its own: 16-byte asynchronous copies, three half stages (K, V, next K)
// deep, 16 KB in flight per warp and 128 KB per SM, more than the 45 KB that cover the
// latency of memory at its rate. No warp waits for another but at the end of a sequence,
// where the warps of a head add up. With more than 16 query rows to a K/V head, teams of
// two or four warps with 16 rows each share a ring, and every tile is copied once for the
// team. Measured: 32 sequences of 32768 tokens, 8 K/V heads of 128, FP8: 316 to 324 us, 6.6 to
// 6.8 TB/s; BF16, 24 sequences of 512 to 32768 tokens: 140 us, 6.0 TB/s, of which about 8 us
// are the start, the sequences' ends inside shares and the join. A ring is empty at each end of
// a sequence, which shows where sequences are short: 46 of 6846 tokens, 4 K/V heads with 16
// rows, FP8: 76 us, floor 48.
//
// The tiles of all sequences and ranks are counted from the lengths, and each CTA takes an
// equal, contiguous share: the last tiles of one sequence and the first of the next may
// fall to one CTA. A sequence that lies within one share is finished there; the two that
// may stick out at a share's ends leave (O, m, l) in the workspace, and a second kernel
// joins them in order, so the result does not depend on which share ends first. More and
// smaller shares, dealt as SMs become free, were slower (twice as many: 345 us against 335
// for the FP8 case). Where a sequence's tiles are few (kWholeTiles) a CTA takes whole
// sequences and the second kernel is not launched: 64 sequences of 32 tiles 49 us, in shares
// 55; one sequence of 64 tiles 19 us, in shares 13. The grid is not evened out there: 57
// sequences of up to 1647 tokens, 16 K/V heads, FP8: 67 us, floor 30.

constexpr int kWarps = 8;
constexpr int kRows = 16;        // query rows of a warp
constexpr int kWholeTiles = 32;  // tiles of a sequence over the call's ranks, at the bound

struct GqaParams {
  const int32_t* seq_lens;
  const int32_t* block_table;
  const uint16_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  uint16_t* out;
  float* lse;
  float* part_o;   // [class][CTA][2][heads][16 * team][D], not normalised
  float* part_ml;  // [class][CTA][2][heads][16 * team][2]
  uint32_t* status;
  float softmax_scale;
  int batch, qlen, H, kv_heads, dcp, interleave, block_size, max_blocks, max_local_len,
      num_blocks, causal, rank_begin, num_ranks;
  int group;      // query heads of a K/V head
  int heads;      // K/V heads of a CTA
  int head_sets;  // CTAs that together take all K/V heads
  int team;       // warps of 16 rows each that share a ring
  int row_sets;   // of 16 * team rows of the qlen * group rows of a sequence and K/V head
  int shares;     // CTAs of each (head set, row tile), or 0: one for each sequence
  int join_warps;  // of the second kernel for a (row, query head): 1 or 4
  FastDiv block_div, group_div, shares_div;
};

// Tokens per tile: 8 KB of K (4 KB for 64 dims of FP8).
template <int kD, bool kFp8>
struct Tile {
  static constexpr int kElem = kFp8 ? 1 : 2;
  static constexpr int kTok = kD * kElem == 256 ? 32 : 64;
  static constexpr int kHalf = kTok * kD * kElem;  // bytes of K, or of V
  static constexpr int kChunks = kD * kElem / 16;  // 16-byte chunks of a row
  static constexpr int kRing = 3 * kHalf;          // of a warp
  static constexpr int kSmem = kWarps * kRing;
  static_assert(kRing >= kRows * (kD + 2) * 4, "a warp's ring holds its (O, m, l)");
};

// Lengths of a sequence on the call's ranks.
struct GqaLengths {
  int whole, rem;
};
__device__ __forceinline__ GqaLengths gqa_lengths(const GqaParams& p, int64_t g) {
  const unsigned L = g > 0 ? (unsigned)(g < INT32_MAX ? g : INT32_MAX) : 0u;
  const int64_t span = (int64_t)p.dcp * p.interleave;
  const int spans = span <= INT32_MAX ? (int)(L / (unsigned)span) : 0;
  return {spans * p.interleave, (int)(L - spans * span)};
}
__device__ __forceinline__ int gqa_rank_len(const GqaParams& p, const GqaLengths& x, int k) {
  const int64_t r = x.rem - (int64_t)(p.rank_begin + k) * p.interleave;
  const int part = r < 0 ? 0 : (r > p.interleave ? p.interleave : (int)r);
  return min(x.whole + part, p.max_local_len);
}
template <int kTok>
__device__ __forceinline__ int gqa_tiles(const GqaParams& p, int b) {
  const GqaLengths x = gqa_lengths(p, p.seq_lens[b]);
  int n = 0;
  for (int k = 0; k < p.num_ranks; ++k) n += (gqa_rank_len(p, x, k) + kTok - 1) / kTok;
  return n;
}

__device__ __forceinline__ void ldsm4(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t (&r)[4], uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
// d += a * b, 16 x 8 x 16; f16 operands for FP8 pools, bf16 for BF16 pools.
template <bool kF16>
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                         uint32_t b1) {
  if (kF16)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, "
        "{%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
template <bool kF16>
__device__ __forceinline__ uint32_t pack16(float lo, float hi) {
  uint32_t r;
  if (kF16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Byte offset of a 16-byte chunk of a tile's row: rows kChunks chunks long, the chunks of
// eight neighbouring rows on different banks.
template <int kChunks>
__device__ __forceinline__ uint32_t tile_offset(int row, int chunk) {
  return row * (kChunks * 16) +
         ((kChunks >= 8 ? chunk ^ (row & 7) : chunk ^ ((row >> 1) & 3)) << 4);
}

// The tiles of one sequence that fall to a warp, every `step`-th from `first` of the tiles
// [first, end), numbered through the ranks.
struct TileWalk {
  int k, tile, tiles, n;  // rank, tile on it, its tiles and tokens
  int left;               // tiles of this walk from here on
};

template <int kD, bool kFp8, int kTeam>
__global__ void __launch_bounds__(32 * kWarps, 1) gqa_decode_kernel(const GqaParams p) {
  using T = Tile<kD, kFp8>;
  constexpr int kTeams = kWarps / kTeam;
  constexpr int kHalves = 3 * kTeam;  // of a ring
  constexpr int kTok = T::kTok, kChunks = T::kChunks;
  constexpr int kPairs = kD / 16;    // steps of 16 dims
  constexpr int kNt = kTok / 8;      // n-tiles of the scores
  constexpr int kMine = kTok / 32;   // tokens whose row a lane looks up
  constexpr int kUp = kFp8 ? 15 : 0;  // weights are formed times 2^kUp
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int s_sum[kWarps];
  __shared__ int s_b, s_skip, s_left;
  __shared__ uint64_t s_gone[kWarps][8];  // a warp's tiles in flight: tokens not read
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int q4 = lane & 3, r8 = lane >> 2;
  // neighbouring CTAs take the head sets and row sets of the same tokens
  const int classes = p.head_sets * p.row_sets;
  const int cls = blockIdx.x % classes, share = blockIdx.x / classes;
  const int member = warp % kTeam, team = warp / kTeam;
  const int row_tile = cls % p.row_sets * kTeam + member;
  const int head0 = cls / p.row_sets * p.heads;
  const int heads = min(p.heads, p.kv_heads - head0);

  // tiles of a sequence, and bad lengths
  auto seq_tiles = [&](int i) -> int {
    const int L = p.seq_lens[i];
    const GqaLengths x = gqa_lengths(p, L);
    int n = 0;
    for (int k = 0; k < p.num_ranks; ++k) n += (gqa_rank_len(p, x, k) + kTok - 1) / kTok;
    if (cls == 0 && (p.shares == 0 || share == 0)) {
      uint32_t bad = 0;
      if (L < 0 || (p.causal && L < p.qlen)) bad |= DCP_STATUS_BAD_SEQ_LEN;
      const int64_t r = x.rem - (int64_t)p.rank_begin * p.interleave;
      if (x.whole + min(max(r, (int64_t)0), (int64_t)p.interleave) > p.max_local_len)
        bad |= DCP_STATUS_LOCAL_OVER_BOUND;
      if (bad) raise_status(p.status, bad);
    }
    return n;
  };
  // this CTA's share: `left` tiles from tile `skip` of sequence b on
  int b = share, skip = 0, left;
  if (p.shares == 0) {
    left = seq_tiles(b);
  } else {
    const bool few = p.batch <= 32;  // one warp holds every sequence
    int mine = 0;
    if (!few || warp == 0)
      for (int i = tid; i < p.batch; i += 32 * kWarps) mine += seq_tiles(i);
    int sum = mine;
    if (!few) {
      sum = __reduce_add_sync(0xffffffffu, sum);
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      sum = lane < kWarps ? s_sum[lane] : 0;
    }
    if (warp == 0) {
      sum = __reduce_add_sync(0xffffffffu, sum);
      const int each = p.shares_div.div(sum), more_n = sum - each * p.shares;
      const int lo = each * share + min(share, more_n);
      int before = 0;
      bool found = false;
      if (lane == 0) s_left = each + (share < more_n ? 1 : 0);
      for (int b0 = 0; b0 < p.batch && !found; b0 += 32) {
        const int n = few ? mine : b0 + lane < p.batch ? seq_tiles(b0 + lane) : 0;
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
        }
        found = __any_sync(0xffffffffu, here);
        before += __shfl_sync(0xffffffffu, incl, 31);
      }
    }
    __syncthreads();
    left = s_left;
    if (left == 0) return;
    b = s_b;
    skip = s_skip;
  }

  // warps beyond the last whole set of `heads` have no work
  const int per_head = kTeams / p.heads;
  const int hl = team / per_head, sub = team % per_head;
  if (hl >= heads) return;
  const int head = head0 + hl;
  const int64_t pitch = (int64_t)p.kv_heads * kD * T::kElem;
  const uint32_t ring = smem_u32(smem) + team * (kTeam * T::kRing);
  const float kv_scale = p.k_scale ? *p.k_scale : 1.0f;
  const float base_scale = p.softmax_scale * kv_scale * kLog2e;
  uint32_t bad = 0;
  int edge = 0;  // of the share: its first sequence, and any later one

  for (bool more = true; more; ++b, skip = 0, edge = 1) {
    const int64_t L = p.seq_lens[b];
    const GqaLengths len = gqa_lengths(p, L);
    // what the first row sees: behind it, rows of one tile may see different tokens
    const GqaLengths first = p.causal ? gqa_lengths(p, L - p.qlen + 1) : len;
    int total = 0;
    for (int k = 0; k < p.num_ranks; ++k)
      total += (gqa_rank_len(p, len, k) + kTok - 1) / kTok;
    const int count = min(total - skip, left);  // of this share
    left -= count;
    more = left > 0;
    if (count == 0 && p.shares != 0) continue;  // no token: the second kernel writes it
    const bool whole = count == total;

    float o[kD / 8][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int i = 0; i < kD / 8; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][e] = 0.f;

    // the tile walk of the copies runs ahead of the products'
    TileWalk cw;
    auto start = [&](TileWalk& w) {
      w.left = count > sub ? (count - sub + per_head - 1) / per_head : 0;
      w.k = 0;
      w.n = gqa_rank_len(p, len, 0);
      w.tiles = (w.n + kTok - 1) / kTok;
      w.tile = skip + sub;
      if (w.left > 0)
        while (w.tile >= w.tiles) {
          w.tile -= w.tiles;
          w.n = gqa_rank_len(p, len, ++w.k);
          w.tiles = (w.n + kTok - 1) / kTok;
        }
    };
    auto advance = [&](TileWalk& w) {
      if (--w.left <= 0) return;
      w.tile += per_head;
      while (w.tile >= w.tiles) {
        w.tile -= w.tiles;
        w.n = gqa_rank_len(p, len, ++w.k);
        w.tiles = (w.n + kTok - 1) / kTok;
      }
    };
    // block ids of this lane's tokens of the next tile to copy
    int blk[kMine];
    auto look = [&]() {
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const int t = cw.tile * kTok + lane + 32 * i;
        blk[i] = cw.left > 0 && t < cw.n
                     ? p.block_table[(int64_t)b * p.max_blocks + p.block_div.div(t)]
                     : -1;
      }
    };
    // rows of the tile that is being copied (-1: not read, zeros), and its rank's pools
    int row[kMine];
    int64_t rank_at = 0;
    auto copy_half = [&](const uint8_t* pool, int slot) {
      const uint8_t* from = pool + rank_at + (int64_t)head * (kD * T::kElem);
      const uint32_t to = ring + slot * T::kHalf;
      constexpr int kPer = 32 / kChunks;  // tokens per instruction of the warp
      const int c = lane % kChunks;
      // a team's warps take every kTeam-th instruction (kTeam * kPer divides 32)
#pragma unroll
      for (int i = 0; i < kTok / kPer; i += kTeam) {
        const int t = (i + member) * kPer + lane / kChunks;
        const int r = __shfl_sync(0xffffffffu, row[i * kPer / 32], t & 31);
        cp_async16(to + tile_offset<kChunks>(t, c), from + (int64_t)max(r, 0) * pitch + c * 16,
                   r >= 0 ? 16u : 0u);
      }
    };
    int to = 0;     // the half stage of the next copy
    int tiles = 0;  // copied so far
    auto copy_k = [&]() {  // of the next tile; the copies move on to it
      if (cw.left > 0) {
        uint64_t gone = 0;
#pragma unroll
        for (int i = 0; i < kMine; ++i) {
          const int t = cw.tile * kTok + lane + 32 * i;
          const bool valid = blk[i] >= 0 && blk[i] < p.num_blocks;
          if (!valid && t < cw.n) bad |= DCP_STATUS_BAD_BLOCK_ID;
          row[i] = valid ? blk[i] * p.block_size + p.block_div.mod(t) : -1;
          gone |= (uint64_t)__ballot_sync(0xffffffffu, row[i] < 0) << (32 * i);
        }
        if (lane == 0) s_gone[warp][tiles & 7] = gone;
        ++tiles;
        rank_at = (int64_t)cw.k * p.num_blocks * p.block_size * pitch;
        copy_half(p.k_pool, to);
      }
      to = to + 1 < kHalves ? to + 1 : 0;
      cp_async_commit();
    };
    auto copy_v = [&]() {
      if (cw.left > 0) {
        copy_half(p.v_pool, to);
        advance(cw);
        look();
      }
      to = to + 1 < kHalves ? to + 1 : 0;
      cp_async_commit();
    };
    // A half has arrived. Alone, a warp refills a half stage when it has used it; a team's
    // warps meet here, so the half stage used before this one is free.
    auto arrive = [&](auto copy) {
      if (kTeam == 1) {
        cp_async_wait_group<kHalves - 1>();
        __syncwarp();
      } else {
        cp_async_wait_group<kHalves - 2>();
        named_bar_sync(9 + team, 32 * kTeam);
        copy();
      }
    };
    auto used = [&](auto copy) {
      if (kTeam == 1) {
        __syncwarp();
        copy();
      }
    };

    TileWalk w;
    start(w);
    cw = w;
    look();
    if (kTeam > 1) named_bar_sync(9 + team, 32 * kTeam);  // the ring is free
    copy_k();
#pragma unroll
    for (int i = 1; i < (kTeam == 1 ? kHalves : kHalves - 1); i += 2) {
      copy_v();
      if (i + 1 < (kTeam == 1 ? kHalves : kHalves - 1)) copy_k();
    }
    // while the first tiles are on their way, the queries: 16 rows, row r = (j, query head of
    // the group), in the products' layout; for FP8 pools in f16 over a power of two per row
    // that keeps them in f16's range: exact from 2^-28 of the row's largest element up, off by
    // at most 2^-36 of it below
    uint32_t qa[kPairs][4];
    float scale[2];
    int limit_j[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = row_tile * kRows + r8 + 8 * i;
      const bool live = r < p.qlen * p.group;
      const int j = live ? p.group_div.div(r) : 0;
      const int64_t at = (((int64_t)b * p.qlen + j) * p.H + head * p.group + (r - j * p.group)) * kD;
      limit_j[i] = j;
      scale[i] = base_scale;
      if (kFp8) {
        float m = 0.f;
        uint2 x[kPairs];
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          x[c] = live ? *reinterpret_cast<const uint2*>(p.q + at + 16 * c + 4 * q4)
                      : make_uint2(0, 0);
          m = fmaxf(m, fmaxf(fmaxf(fabsf(__uint_as_float(x[c].x << 16)),
                                   fabsf(__uint_as_float(x[c].x & 0xffff0000u))),
                             fmaxf(fabsf(__uint_as_float(x[c].y << 16)),
                                   fabsf(__uint_as_float(x[c].y & 0xffff0000u)))));
        }
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 1));
        m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, 2));
        // 2^e: the largest element below 2^12
        const int e = m > 0.f ? max(-120, min(120, 138 - (int)(__float_as_uint(m) >> 23))) : 0;
        const float up = __uint_as_float((uint32_t)(127 + e) << 23);
        scale[i] *= __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          qa[c][i] = pack16<true>(__uint_as_float(x[c].x << 16) * up,
                                  __uint_as_float(x[c].x & 0xffff0000u) * up);
          qa[c][i + 2] = pack16<true>(__uint_as_float(x[c].y << 16) * up,
                                      __uint_as_float(x[c].y & 0xffff0000u) * up);
        }
      } else {
#pragma unroll
        for (int c = 0; c < kPairs; ++c) {
          qa[c][i] = live ? *reinterpret_cast<const uint32_t*>(p.q + at + 16 * c + 2 * q4) : 0u;
          qa[c][i + 2] =
              live ? *reinterpret_cast<const uint32_t*>(p.q + at + 16 * c + 8 + 2 * q4) : 0u;
        }
      }
    }

    int slot = 0;  // the half stage in use
    for (int done = 0; w.left > 0; ++done) {
      arrive(copy_v);
      const uint64_t gone_now = s_gone[warp][done & 7];
      float s[kNt][4];
      const uint32_t kb = ring + slot * T::kHalf;
      slot = slot + 1 < kHalves ? slot + 1 : 0;
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        s[nt][0] = s[nt][1] = s[nt][2] = s[nt][3] = 0.f;
#pragma unroll
        for (int c = 0; c < kChunks; c += 4) {
          uint32_t r[4];
          ldsm4(r, kb + tile_offset<kChunks>(8 * nt + (lane & 7), c + (lane >> 3)));
          if (kFp8) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint32_t b0, b1;
              e4m3x4_to_f16x2(r[i], b0, b1);
              mma16816<true>(s[nt], qa[c + i], b0, b1);
            }
          } else {
            mma16816<false>(s[nt], qa[c / 2], r[0], r[1]);
            mma16816<false>(s[nt], qa[c / 2 + 1], r[2], r[3]);
          }
        }
      }
      used(copy_v);

      // masks: rows see their first tokens, bad blocks and what lies behind n are gone
      const int t0 = w.tile * kTok;
      int limit[2] = {kTok, kTok};
      bool masked = false;
      if (gone_now != 0 || t0 + kTok > gqa_rank_len(p, first, w.k)) masked = true;
      if (masked) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int64_t g = L - (p.causal ? p.qlen - 1 - limit_j[i] : 0);
          limit[i] = gqa_rank_len(p, gqa_lengths(p, g), w.k) - t0;
        }
#pragma unroll
        for (int nt = 0; nt < kNt; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int c = 8 * nt + 2 * q4 + (e & 1);
            if (c >= limit[e >> 1] || (gone_now >> c & 1)) s[nt][e] = -INFINITY;
          }
      }

      // running maximum, in the scaled domain (the scales are positive)
      float top[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        top[0] = fmaxf(top[0], fmaxf(s[nt][0], s[nt][1]));
        top[1] = fmaxf(top[1], fmaxf(s[nt][2], s[nt][3]));
      }
      float shift[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 1));
        top[i] = fmaxf(top[i], __shfl_xor_sync(0xffffffffu, top[i], 2));
        top[i] = fmaxf(m[i], top[i] * scale[i]);
        shift[i] = top[i] == -INFINITY ? 0.f : top[i];
      }
      if (__any_sync(0xffffffffu, top[0] > m[0] || top[1] > m[1])) {
        const float a0 = exp2_fast(m[0] - shift[0]), a1 = exp2_fast(m[1] - shift[1]);
        l[0] *= a0;
        l[1] *= a1;
#pragma unroll
        for (int i = 0; i < kD / 8; ++i) {
          o[i][0] *= a0;
          o[i][1] *= a0;
          o[i][2] *= a1;
          o[i][3] *= a1;
        }
        m[0] = top[0];
        m[1] = top[1];
      }
      uint32_t pa[kNt / 2][4];
#pragma unroll
      for (int nt = 0; nt < kNt; ++nt) {
        float e[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
          e[i] = exp2_fast(fmaf(s[nt][i], scale[i >> 1], kUp - shift[i >> 1]));
        l[0] += e[0] + e[1];
        l[1] += e[2] + e[3];
        // rounded to 16 bits for the second product
        pa[nt / 2][2 * (nt & 1)] = pack16<kFp8>(e[0], e[1]);
        pa[nt / 2][2 * (nt & 1) + 1] = pack16<kFp8>(e[2], e[3]);
      }

      arrive(copy_k);
      const uint32_t vb = ring + slot * T::kHalf;
      slot = slot + 1 < kHalves ? slot + 1 : 0;
      // O += P V, steps of 16 tokens and 32 bytes of dims: d[] are the steps' accumulators
      auto step = [&](const uint32_t (&pp)[4], int kk, int c, uint32_t keep0, uint32_t keep1,
                      auto&& d) {
        uint32_t r[4];
        ldsm4_trans(r, vb + tile_offset<kChunks>(16 * kk + (lane & 15), c + (lane >> 4)));
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const uint32_t r0 = r[2 * i] & keep0, r1 = r[2 * i + 1] & keep1;
          if (kFp8) {
            // bytes (token, dim): 00 01 10 11 -> 00 10 01 11
            uint32_t a0, a1, b0, b1;
            e4m3x4_to_f16x2(__byte_perm(r0, 0, 0x3120), a0, b0);
            e4m3x4_to_f16x2(__byte_perm(r1, 0, 0x3120), a1, b1);
            mma16816<true>(d(2 * i), pp, a0, a1);
            mma16816<true>(d(2 * i + 1), pp, b0, b1);
          } else {
            mma16816<false>(d(i), pp, r0, r1);
          }
        }
      };
      constexpr int kD8 = kFp8 ? 2 : 1;  // n-tiles of a chunk
      if (masked && p.causal && p.qlen > 1) {
        // Rows of one tile see different tokens: one pass for each of their boundaries, over
        // the tokens in front of it, kept for the rows of that boundary alone: a token that
        // a row does not see never meets it, whatever its value.
        const int j1 = min(p.qlen - 1, p.group_div.div(row_tile * kRows + kRows - 1));
        for (int j = p.group_div.div(row_tile * kRows); j <= j1; ++j) {
          const int seen = gqa_rank_len(p, gqa_lengths(p, L - (p.qlen - 1 - j)), w.k) - t0;
#pragma unroll
          for (int c = 0; c < kChunks; c += 2) {
            float x[2 * kD8][4];
#pragma unroll
            for (int i = 0; i < 2 * kD8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e) x[i][e] = 0.f;
#pragma unroll
            for (int kk = 0; kk < kTok / 16; ++kk) {
              // tokens 16 kk + 8 h + 2 q4 + {0, 1} of this lane's operands
              uint32_t keep[2];
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                const int t = 16 * kk + 8 * h + 2 * q4;
                keep[h] = (t < seen ? 0xffffu : 0u) | (t + 1 < seen ? 0xffff0000u : 0u);
              }
              step(pa[kk], kk, c, keep[0], keep[1], [&](int i) -> float(&)[4] { return x[i]; });
            }
#pragma unroll
            for (int i = 0; i < 2 * kD8; ++i)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (limit_j[e >> 1] == j) o[kD8 * c + i][e] += x[i][e];
          }
        }
      } else {
#pragma unroll
        for (int kk = 0; kk < kTok / 16; ++kk)
#pragma unroll
          for (int c = 0; c < kChunks; c += 2)
            step(pa[kk], kk, c, 0xffffffffu, 0xffffffffu,
                 [&](int i) -> float(&)[4] { return o[kD8 * c + i]; });
      }
      advance(w);
      used(copy_k);
    }
    cp_async_wait_all();
    __syncwarp();

    // per row: l over the row's four lanes; from here on l and O are over 2^m
    if (kFp8) {
#pragma unroll
      for (int i = 0; i < kD / 8; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][e] *= 1.f / (1 << kUp);
      l[0] *= 1.f / (1 << kUp);
      l[1] *= 1.f / (1 << kUp);
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 1);
      l[i] += __shfl_xor_sync(0xffffffffu, l[i], 2);
    }
    // dims of this lane's accumulators: FP8 16 c + 4 q4 + {0, 1, 2, 3}, BF16 8 c + 2 q4 + {0, 1}
    if (per_head > 1) {
      // the head's warps add up, through the rings (empty now), in order
      float* mine = reinterpret_cast<float*>(smem + warp * T::kRing);
      float* ml = mine + kRows * kD;
      if (kTeam > 1) named_bar_sync(1 + hl, 32 * kTeam * per_head);
      if (sub > 0) {
#pragma unroll
        for (int i = 0; i < kD / 8; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) mine[(4 * i + e) * 32 + lane] = o[i][e];
        if (q4 == 0) {
          ml[2 * r8] = m[0];
          ml[2 * r8 + 1] = l[0];
          ml[2 * r8 + 16] = m[1];
          ml[2 * r8 + 17] = l[1];
        }
      }
      named_bar_sync(1 + hl, 32 * kTeam * per_head);
      if (sub == 0) {
        for (int u = 1; u < per_head; ++u) {
          const float* other = mine + u * (kTeam * T::kRing / 4);
          const float* oml = other + kRows * kD;
          float keep[2], add[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float mo = oml[2 * (r8 + 8 * i)], lo = oml[2 * (r8 + 8 * i) + 1];
            const float mn = fmaxf(m[i], mo), sh = mn == -INFINITY ? 0.f : mn;
            keep[i] = exp2_fast(m[i] - sh);
            add[i] = exp2_fast(mo - sh);
            l[i] = l[i] * keep[i] + lo * add[i];
            m[i] = mn;
          }
#pragma unroll
          for (int i = 0; i < kD / 8; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              o[i][e] = o[i][e] * keep[e >> 1] + other[(4 * i + e) * 32 + lane] * add[e >> 1];
        }
      }
      named_bar_sync(1 + hl, 32 * kTeam * per_head);  // the rings are free for the next sequence
      if (sub > 0) continue;
    }
    if (whole) {
      const float vs = p.v_scale ? *p.v_scale : 1.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = row_tile * kRows + r8 + 8 * i;
        if (r >= p.qlen * p.group) continue;
        const int j = limit_j[i];
        const int64_t rh = ((int64_t)b * p.qlen + j) * p.H + head * p.group + (r - j * p.group);
        const float inv = l[i] == 0.f ? 0.f : vs / l[i];  // no token: 0; NaN stays
        uint16_t* dst = p.out + rh * kD;
        if (kFp8) {
#pragma unroll
          for (int c = 0; c < kD / 16; ++c) {
            const float* a = o[2 * c] + 2 * i;
            const float* d = o[2 * c + 1] + 2 * i;
            *reinterpret_cast<uint2*>(dst + 16 * c + 4 * q4) =
                make_uint2(pack16<false>(a[0] * inv, d[0] * inv),
                           pack16<false>(a[1] * inv, d[1] * inv));
          }
        } else {
#pragma unroll
          for (int c = 0; c < kD / 8; ++c)
            *reinterpret_cast<uint32_t*>(dst + 8 * c + 2 * q4) =
                pack16<false>(o[c][2 * i] * inv, o[c][2 * i + 1] * inv);
        }
        if (q4 == 0) p.lse[rh] = l[i] == 0.f ? -INFINITY : (m[i] + log2f(l[i])) * kLn2;
      }
    } else {
      const int64_t at =
          (((((int64_t)cls * p.shares + share) * 2 + edge) * p.heads + hl) * kTeam + member) *
          kRows;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float* dst = p.part_o + (at + r8 + 8 * i) * kD;
        if (kFp8) {
#pragma unroll
          for (int c = 0; c < kD / 16; ++c)
            *reinterpret_cast<float4*>(dst + 16 * c + 4 * q4) =
                make_float4(o[2 * c][2 * i], o[2 * c + 1][2 * i], o[2 * c][2 * i + 1],
                            o[2 * c + 1][2 * i + 1]);
        } else {
#pragma unroll
          for (int c = 0; c < kD / 8; ++c)
            *reinterpret_cast<float2*>(dst + 8 * c + 2 * q4) =
                make_float2(o[c][2 * i], o[c][2 * i + 1]);
        }
        if (q4 == 0) {
          p.part_ml[(at + r8 + 8 * i) * 2] = m[i];
          p.part_ml[(at + r8 + 8 * i) * 2 + 1] = l[i];
        }
      }
    }
  }
  if (bad) raise_status(p.status, bad);
}

// The rows of a sequence that several shares worked on, joined in their order; and the rows
// of a sequence without a token. A warp per (row, query head), or four where a sequence may
// have many parts: a part's (m, l) per lane, its O over the lanes' dims. What bounds it is the
// latency of its loads, so the first parts' O is on its way with their (m, l), and eight parts
// are in flight at a time. With the first kernel, for 24 ragged sequences (up to 19 parts) a
// warp 140 us, four 144.6 and a CTA with three barriers 144.2; for one sequence of 32768 tokens
// (38 parts) a warp 36.0 us, four 34.2.
constexpr int kJoinThreads = 128;
constexpr int kMaxShares = 512;
template <int kD, int kTok>
__global__ void __launch_bounds__(kJoinThreads) gqa_join_kernel(const GqaParams p) {
  constexpr int kWarpsJ = kJoinThreads / 32;
  constexpr int kV = kD / 32;  // dims of a lane
  __shared__ float s_o[kWarpsJ][kD];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int team = p.join_warps, sub = warp % team;
  const int64_t rh = (int64_t)blockIdx.x * (kWarpsJ / team) + warp / team;
  const bool live = rh < (int64_t)p.batch * p.qlen * p.H;  // a team lives or not as one CTA
  const int row = (int)(rh / p.H), h = (int)(rh - (int64_t)row * p.H);
  const int b = row / p.qlen, j = row - b * p.qlen;
  // tiles of all sequences, of those before this one, and its own
  int all = 0, before = 0, n = 0;
  for (int i = lane; i < p.batch; i += 32) {
    const int tiles = gqa_tiles<kTok>(p, i);
    all += tiles;
    if (i < b) before += tiles;
    if (i == b) n = tiles;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  n = __reduce_add_sync(0xffffffffu, n);
  grid_dependency_wait();
  if (!live) return;
  uint16_t* out = p.out + rh * kD + lane * kV;
  auto store = [&](const float (&y)[kV]) {
    if (kV == 4)
      *reinterpret_cast<uint2*>(out) =
          make_uint2(pack16<false>(y[0], y[1]), pack16<false>(y[kV - 2], y[kV - 1]));
    else
      *reinterpret_cast<uint32_t*>(out) = pack16<false>(y[0], y[1]);
  };
  if (n == 0) {
    const float zero[kV] = {};
    if (sub == 0) store(zero);
    if (sub == 0 && lane == 0) p.lse[rh] = -INFINITY;
    return;
  }
  // the share of a tile: the first `more` shares are a tile longer
  const int each = p.shares_div.div(all), more = all - each * p.shares;
  auto share_of = [&](int x) {
    return x < more * (each + 1) ? x / (each + 1) : more + (x - more * (each + 1)) / max(each, 1);
  };
  const int c0 = share_of(before), parts = share_of(before + n - 1) - c0 + 1;
  if (parts == 1) return;  // finished by its one share
  const int g = h / p.group, r = j * p.group + h % p.group;
  const int set_rows = kRows * p.team;
  const int cls = g / p.heads * p.row_sets + r / set_rows;
  // rows of the parts: a stride apart, but for the first share, whose sequence may be its second
  const int64_t stride = (int64_t)2 * p.heads * set_rows;
  const int64_t first = (((int64_t)cls * p.shares + c0) * 2 * p.heads + g % p.heads) * set_rows +
                        r % set_rows;
  const int edge = before > each * c0 + min(c0, more);  // that share begins before this sequence
  auto part_at = [&](int i) {
    return first + i * stride + (i == 0 && edge ? (int64_t)p.heads * set_rows : 0);
  };
  float x[8][kV];
  auto load = [&](int i0) {  // parts i0, i0 + team, ..
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = i0 + u * team;
      const float* src = p.part_o + part_at(i) * kD + lane * kV;
      if (kV == 4) {
        const float4 v = i < parts ? *reinterpret_cast<const float4*>(src)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        x[u][0] = v.x, x[u][1] = v.y, x[u][kV - 2] = v.z, x[u][kV - 1] = v.w;
      } else {
        const float2 v = i < parts ? *reinterpret_cast<const float2*>(src) : make_float2(0.f, 0.f);
        x[u][0] = v.x, x[u][1] = v.y;
      }
    }
  };
  auto stats = [&](int i) {  // (m, l); m of a part without weight is -inf
    float2 v = i < parts ? *reinterpret_cast<const float2*>(p.part_ml + 2 * part_at(i))
                         : make_float2(-INFINITY, 0.f);
    if (v.y == 0.f) v.x = -INFINITY;
    return v;
  };
  load(sub);
  const float2 mine = stats(lane);
  float m = mine.x;
  for (int i = 32 + lane; i < parts; i += 32) m = fmaxf(m, stats(i).x);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  const float shift = m == -INFINITY ? 0.f : m;
  float l = 0.f, acc[kV] = {};
  for (int i0 = 0; i0 < parts; i0 += 32) {
    const float2 ml = i0 == 0 ? mine : stats(i0 + lane);
    const float weight = ml.y == 0.f ? 0.f : exp2_fast(ml.x - shift);
    l = fmaf(ml.y, weight, l);
    for (int q = 0; q < 32 && i0 + q + sub < parts; q += 8 * team) {
      if (i0 + q > 0) load(i0 + q + sub);
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const float w = __shfl_sync(0xffffffffu, weight, (q + sub + u * team) & 31);
        if (i0 + q + sub + u * team < parts && w != 0.f) {  // weightless parts may hold infinities
#pragma unroll
          for (int e = 0; e < kV; ++e) acc[e] = fmaf(x[u][e], w, acc[e]);
        }
      }
    }
  }
  // the same order of additions in every call
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) l += __shfl_xor_sync(0xffffffffu, l, o);
  if (team > 1) {
#pragma unroll
    for (int e = 0; e < kV; ++e) s_o[warp][lane * kV + e] = acc[e];
    __syncthreads();
    if (sub > 0) return;
    for (int u = 1; u < team; ++u)
#pragma unroll
      for (int e = 0; e < kV; ++e) acc[e] += s_o[warp + u][lane * kV + e];
  }
  const float inv = l == 0.f ? 0.f : (p.v_scale ? *p.v_scale : 1.0f) / l;
#pragma unroll
  for (int e = 0; e < kV; ++e) acc[e] *= inv;
  store(acc);
  if (lane == 0) p.lse[rh] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

// How a call is cut into CTAs.
struct GqaPlan {
  int heads, head_sets, team, row_sets, shares;
  int64_t ctas, tiles;  // tiles: of all sequences, at the bound
};
GqaPlan gqa_plan(const dcp_mla_dims& d, int kv_heads, int head_dim, bool fp8, int num_ranks,
                 int sms) {
  GqaPlan x;
  const int tok = head_dim * (fp8 ? 1 : 2) == 256 ? 32 : 64;
  const int64_t tiles = (int64_t)num_ranks * (((int64_t)d.max_local_len + tok - 1) / tok);
  x.tiles = tiles * d.batch;
  const int row_tiles = (d.qlen * (d.num_heads / kv_heads) + kRows - 1) / kRows;
  x.team = row_tiles >= 3 ? 4 : row_tiles;
  x.row_sets = (row_tiles + x.team - 1) / x.team;
  // Whole sequences: up to eight K/V heads to a CTA, fewer where the CTAs would not fill the
  // device, so that a sequence's tiles spread over a head's warps. Shares: two heads, four
  // warps of each (322 us for 32 x 32768 tokens of FP8, 141 us for 24 ragged sequences of
  // BF16; one head 328 and 149, eight 327 and 145).
  const bool whole = tiles <= kWholeTiles;
  x.heads = std::min({kv_heads, kWarps / x.team, whole ? kWarps : 2});
  const int64_t units = (int64_t)d.batch * x.row_sets * (whole ? 1 : (tiles + 7) / 8);
  while (x.heads > 1 && units * ((kv_heads + x.heads - 1) / x.heads) < sms)
    x.heads = (x.heads + 1) / 2;
  x.head_sets = (kv_heads + x.heads - 1) / x.heads;
  x.heads = (kv_heads + x.head_sets - 1) / x.head_sets;  // evenly
  const int classes = x.head_sets * x.row_sets;
  if (whole) {
    x.shares = 0;
    x.ctas = (int64_t)d.batch * classes;
  } else {
    x.shares = (int)std::max<int64_t>(1, std::min<int64_t>({sms / classes, d.batch * tiles, kMaxShares}));
    x.ctas = (int64_t)x.shares * classes;
  }
  return x;
}

struct GqaKernel {
  void (*kern)(GqaParams);
  int smem;
};
template <int kD, bool kFp8, int kTeam>
constexpr GqaKernel gqa_kernel() {
  return {gqa_decode_kernel<kD, kFp8, kTeam>, Tile<kD, kFp8>::kSmem};
}
const GqaKernel kGqaKernels[4][3] = {
    {gqa_kernel<64, false, 1>(), gqa_kernel<64, false, 2>(), gqa_kernel<64, false, 4>()},
    {gqa_kernel<64, true, 1>(), gqa_kernel<64, true, 2>(), gqa_kernel<64, true, 4>()},
    {gqa_kernel<128, false, 1>(), gqa_kernel<128, false, 2>(), gqa_kernel<128, false, 4>()},
    {gqa_kernel<128, true, 1>(), gqa_kernel<128, true, 2>(), gqa_kernel<128, true, 4>()}};

int gqa_sms() {
  static int cached[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 152;
  if (cached[dev] == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return 152;
    cached[dev] = n;
  }
  return cached[dev];
}

}  // namespace

cudaError_t launch_gqa_kv_write(const dcp_mla_dims& d, int row_elems, const int32_t* slot_mapping,
                                const void* k_new, const void* v_new, dcp_kv_dtype kv_dtype,
                                const float* k_scale, const float* v_scale, int num_ranks,
                                void* k_pool, void* v_pool, uint32_t* status,
                                cudaStream_t stream) {
  const int rows = d.batch * d.qlen;
  const int64_t grid = (2 * (int64_t)rows + kWriteWarps - 1) / kWriteWarps;
  auto kern = kv_dtype == DCP_KV_FP8_E4M3 ? gqa_write_kernel<true> : gqa_write_kernel<false>;
  kern<<<(unsigned)grid, 32 * kWriteWarps, 0, stream>>>(
      rows, num_ranks, num_ranks == d.dcp, row_elems, (int64_t)d.num_blocks * d.block_size, slot_mapping,
      static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new), k_scale, v_scale,
      static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool), status);
  return cudaGetLastError();
}

// Enough for either cache type: (O, m, l) of two sequences for every share.
size_t gqa_workspace_bytes(const dcp_mla_dims& d, int kv_heads, int head_dim, int num_ranks) {
  size_t most = 16;
  for (int fp8 = 0; fp8 < 2; ++fp8) {
    const GqaPlan x = gqa_plan(d, kv_heads, head_dim, fp8 != 0, num_ranks, gqa_sms());
    most = std::max(most, (size_t)x.shares * x.head_sets * x.row_sets * 2 * x.heads * x.team *
                              kRows * (head_dim + 2) * sizeof(float));
  }
  return most;
}

cudaError_t launch_gqa_decode(const dcp_mla_dims& d, int kv_heads, int head_dim,
                              const int32_t* seq_lens, const int32_t* block_table, const void* q,
                              const void* k_pool, const void* v_pool, dcp_kv_dtype kv_dtype,
                              const float* k_scale, const float* v_scale, float softmax_scale,
                              int rank_begin, int num_ranks, void* out, float* lse,
                              void* workspace, uint32_t* status, cudaStream_t stream) {
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3;
  const GqaPlan x = gqa_plan(d, kv_heads, head_dim, fp8, num_ranks, gqa_sms());
  GqaParams p;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.q = static_cast<const uint16_t*>(q);
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.part_o = static_cast<float*>(workspace);
  p.part_ml = p.part_o + (size_t)x.shares * x.head_sets * x.row_sets * 2 * x.heads * x.team *
                             kRows * head_dim;
  p.status = status;
  p.softmax_scale = softmax_scale;
  p.batch = d.batch;
  p.qlen = d.qlen;
  p.H = d.num_heads;
  p.kv_heads = kv_heads;
  p.dcp = d.dcp;
  p.interleave = d.interleave;
  p.block_size = d.block_size;
  p.max_blocks = d.max_blocks_per_seq;
  p.max_local_len = d.max_local_len;
  p.num_blocks = d.num_blocks;
  p.causal = d.causal;
  p.rank_begin = rank_begin;
  p.num_ranks = num_ranks;
  p.group = d.num_heads / kv_heads;
  p.heads = x.heads;
  p.head_sets = x.head_sets;
  p.team = x.team;
  p.row_sets = x.row_sets;
  p.shares = x.shares;
  // a sequence has some shares / batch parts, eight of which a warp reads at a time
  p.join_warps = x.shares > 8 * d.batch ? 4 : 1;
  p.block_div = FastDiv::by(d.block_size);
  p.group_div = FastDiv::by(p.group);
  p.shares_div = FastDiv::by(std::max(1, x.shares));
  if (x.ctas > INT32_MAX || x.tiles > INT32_MAX) return cudaErrorInvalidConfiguration;
  const int dtype_dim = (head_dim == 128 ? 2 : 0) + (fp8 ? 1 : 0);
  const GqaKernel& k = kGqaKernels[dtype_dim][x.team == 4 ? 2 : x.team - 1];
  static bool attr_set[4][3][64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  bool& ready = attr_set[dtype_dim][x.team == 4 ? 2 : x.team - 1][dev];
  if (!ready) {
    e = cudaFuncSetAttribute(k.kern, cudaFuncAttributeMaxDynamicSharedMemorySize, k.smem);
    if (e != cudaSuccess) return e;
    ready = true;
  }
  k.kern<<<(unsigned)x.ctas, 32 * kWarps, k.smem, stream>>>(p);
  e = cudaGetLastError();
  if (e != cudaSuccess || x.shares == 0) return e;
  auto join = head_dim == 64 ? gqa_join_kernel<64, 64>
              : fp8          ? gqa_join_kernel<128, 64>
                             : gqa_join_kernel<128, 32>;
  const int64_t warps = (int64_t)d.batch * d.qlen * d.num_heads * p.join_warps;
  const dim3 grid((unsigned)((warps * 32 + kJoinThreads - 1) / kJoinThreads));
  return launch_overlapping(true, join, grid, dim3(kJoinThreads), 0, stream, p);
}

}  // namespace dcpmla
