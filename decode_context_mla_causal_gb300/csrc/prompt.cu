// Attention of packed prompts: rows of several sequences one behind the other, grouped heads,
// causal or not, with or without tokens in front of the new rows.
//
// Row i of a sequence with n rows and m keys sees the first m - n + 1 + i keys (all m where not
// causal); for query head h with K/V head h / group,
//   s_t = softmax_scale * log2(e) * (q . k_t)                      (base 2)
//   O = sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m),  LSE = (m + log2 sum) ln 2.
// Scores, maxima, sums and O are held in 32 bits; the weights 2^(s - m) are rounded to bf16 for
// the second product, whose matrix instructions take 16-bit operands (half a step, 2^-9 to 2^-8
// of each; their sum is of the unrounded ones).
#include <cuda.h>
#include <cudaTypedefs.h>
#include <cuda_bf16.h>

#include <algorithm>

#include "common.cuh"
#include "sm103.cuh"

namespace dcpmla {
namespace {

using namespace sm103;

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr uint64_t kTimeoutNs = 4000000000ull;

constexpr int kRows = 128;      // of a row tile: tokens x heads of the group
constexpr int kTok = 128;       // keys of a tile
constexpr int kSoftWarps = 8;   // four to a row tile: a thread takes a row
constexpr int kThreads = 32 * kSoftWarps + 128;  // and issuer, copier, cleaner
constexpr int kMaxSeqs = 8192;  // sequences the item kernel holds offsets of
constexpr int kItemThreads = 1024;
constexpr int kMaxCtas = 512;   // of the attention
constexpr int kRoles = kSoftWarps + 3;  // warps that walk over the units
constexpr int kUnitCost = 8;    // key tiles that a unit's start and end take as long as
constexpr int kBuckets = 1024;  // of key tiles, longest items first
constexpr int kFewItems = 128;  // placed by comparing each with the others

// A work item: two row tiles of consecutive tokens of one sequence, for one K/V head.
struct __align__(16) Item {
  int row;    // first row of q
  int rows;   // tokens from there on to the sequence's end, at most those of two tiles
  int key;    // first row of k and v
  int keys;   // of the sequence
  int seen;   // keys that the first token sees, may be < 1
  int tiles;  // key tiles
  int start;  // where its units begin in the row of all units (shares)
  int pad;
};
// Where a CTA's share of that row begins; `tile` may lie behind the unit's last.
struct __align__(16) Start {
  int item, unit, tile, pad;
};
struct __align__(16) Header {
  int items, with_keys;  // of them those with tiles, which stand in front
  int shares, length;    // whether CTAs take equal shares of the row of all units, and its length:
                         // a unit is as long as its tiles and kUnitCost
};

struct PromptParams {
  const Header* header;
  const Start* starts;
  const Item* items;
  int* arrived;  // [CTA][warp of softmax]: pieces of the unit that the CTA's share ends in
  int* ticket;   // whole units that CTAs have taken beside their first
  int* before;   // [unit]: the unit that its CTA took before it, -1: none
  float* parts;  // [CTA][2][row tile][dims, then m, then l][row]
  uint16_t* out;
  float* lse;
  uint32_t* status;
  float scale;  // softmax_scale * log2(e)
  int heads, group, causal;
  int set_heads;    // query heads of a row tile
  int sets;         // row tiles that together take a K/V head's group
  int tile_tokens;  // tokens of a row tile
  FastDiv set_div;
};

struct Bars {
  uint64_t full[12];   // ring slots: filled
  uint64_t empty[12];  // the products with it are done, and the cleaner has passed it
  uint64_t qfull[2], qempty[2];
  uint64_t sfull[2];   // scores of a row tile are in tensor memory
  uint64_t pfull[2];   // its weights are, and V of this tile is there, cleaned (and, where the ring
                       // reaches that far, K of the next)
  uint64_t ofull[2];   // every product of the item's row tile is done
  uint64_t done[2];    // a row tile that had keys is written (second pass)
  uint64_t drain;
  uint64_t want;         // the copier is about to need the next unit
  uint64_t told, heard;  // it is known, and known to all roles
};
struct Rest {
  Bars bar;
  uint32_t tmem;
  int abort_flag;
  int again;              // a row came out with infinities or NaN
  int dirty;              // `first` has entries
  int first[3][128];      // first key with NaN, +inf, -inf in a masked tile's dim
  int unit;               // -1: no more
};

// Shared memory: two row tiles of q, then a ring of slots, each filled by one copy (one thread
// issues a copy in about 200 cycles; with two to four times as many copies to a tile they took
// longer than its products: 480 against 421 us for 2048 rows behind 6144 keys). A tile of K is a
// slot, or three of 64 dims where rows have 192; a tile of V a slot, or there two of 64 keys. They
// pass through the ring in the order in which the products use them up.
template <int kDq, int kDv>
struct Shape {
  static constexpr int kQTile = kRows * kDq * 2;
  static constexpr int kQSlice = kRows * 128;  // bytes of 64 dims
  static constexpr int kKSlots = kDq == 192 ? 3 : 1, kVSlots = kDq == 192 ? 2 : 1;
  static constexpr int kSlot = kTok * kDq * 2 / kKSlots;
  static constexpr int kSlots = kDq == 64 ? 12 : kDq == 128 ? 5 : 8;
  static constexpr int kKSlices = kDq / 64 / kKSlots;  // 64-dim slices of a slot of K
  static constexpr int kVTok = kTok / kVSlots;         // keys of a slot of V
  static constexpr int kRest = 2 * kQTile + kSlots * kSlot;
  static constexpr int kSmem = kRest + (int)sizeof(Rest);
  static_assert(kSmem <= 227 * 1024, "shared memory of a CTA");
  // Whether the ring holds two tiles of K and V: if so, a tile's products are not begun before the
  // next one's K is there (one wait instead of several); else that would hold them up.
  static constexpr bool kAhead = kSlots >= 2 * (kKSlots + kVSlots);
  static_assert(kSlots >= kKSlots + kVSlots, "K of the next tile beside V of this one");
  static_assert(kVTok * kDv * 2 == kSlot, "slots of K and V are alike");
};

__device__ __forceinline__ bool wait_slow(uint32_t a, uint32_t parity, int* abort_flag,
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
// Of a converged warp, with a warp-uniform result.
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, int* abort_flag,
                                          uint32_t* status) {
  return __all_sync(0xffffffffu, wait_one(bar, parity, abort_flag, status));
}
// For copies and products in flight after a timeout: bounded, whatever the abort flag says.
__device__ __forceinline__ void wait_landed(uint64_t* bar, uint32_t parity) {
  const uint32_t a = smem_u32(bar);
  const uint64_t t0 = globaltimer_ns();
  while (!mbar_wait_sleep(a, parity) && globaltimer_ns() - t0 < kTimeoutNs) {
  }
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
// The value, formed here and not kept in registers from before a loop.
__device__ __forceinline__ uint32_t here(uint32_t x) {
  asm volatile("" : "+r"(x));
  return x;
}
// Pairs of floats.
__device__ __forceinline__ uint64_t pack_b32(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t pack_f32(float lo, float hi) {
  return pack_b32(__float_as_uint(lo), __float_as_uint(hi));
}
__device__ __forceinline__ float low_f32(uint64_t x) { return __uint_as_float((uint32_t)x); }
__device__ __forceinline__ float high_f32(uint64_t x) {
  return __uint_as_float((uint32_t)(x >> 32));
}
__device__ __forceinline__ uint64_t fma_f32x2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add_f32x2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// What a CTA works on: whole units (an item and a K/V head's row tile each), longest first (the
// heads of an item side by side; a head's items side by side, so that CTAs read the same keys
// together, was slower: 2614 against 2178 us for four prompts of 128 heads); or an equal share of
// the row of all units, whose first and last unit may be cut. Whole units are dealt in turns, there
// and back through the list, or (kTaken) taken as a CTA comes by them. Every role of the CTA walks
// the same way.
struct Walk {
  Header h;
  Rest& rest;
  uint32_t heard;              // units taken, over both passes
  int round;                   // units dealt in turns, and those without keys beside shares
  int item, unit, tile, left;  // share
  __device__ __forceinline__ Walk(const PromptParams& p, Rest& r) : h(*p.header), rest(r), heard(0) {}
  __device__ __forceinline__ void begin(const PromptParams& p) {  // a pass
    round = 0;
    if (!h.shares) return;
    const Start s = p.starts[blockIdx.x];
    item = s.item, unit = s.unit, tile = s.tile;
    const int each = h.length / (int)gridDim.x, more = h.length - each * (int)gridDim.x;
    left = each + ((int)blockIdx.x < more ? 1 : 0);
  }
  __device__ __forceinline__ int share_of(int x) const {
    const int each = h.length / (int)gridDim.x, more = h.length - each * (int)gridDim.x;
    return x < more * (each + 1) ? x / (each + 1) : more + (x - more * (each + 1)) / each;
  }
  // The CTA's next whole unit, -1: none (or a wait gave up). kAlone: one thread of the warp is
  // here.
  template <bool kAlone>
  __device__ __forceinline__ int take(const PromptParams& p) {
    const uint32_t parity = heard++ & 1;
    if (kAlone) {
      if (!wait_one(&rest.bar.told, parity, &rest.abort_flag, p.status)) return -1;
      const int u = *reinterpret_cast<volatile int*>(&rest.unit);
      mbar_arrive(&rest.bar.heard);
      return u;
    }
    if (!wait_warp(&rest.bar.told, parity, &rest.abort_flag, p.status)) return -1;
    const int u = *reinterpret_cast<volatile int*>(&rest.unit);
    __syncwarp();
    if ((threadIdx.x & 31) == 0) mbar_arrive(&rest.bar.heard);
    return u;
  }
};

// What a unit, or a piece of one, asks of each role. A piece is as a unit whose keys begin at its
// first tile.
struct Work {
  int row, rows, key, keys, seen, head;  // head: first query head of the row tiles
  int kv_head, skipped;                  // keys in front of the piece
  int n[2];   // key tiles of each row tile
  int lo[2];  // keys that the first token of each sees: tiles beyond are masked
  int piece, pieces, first_cta;

  // keys that the token at offset t from the unit's first sees
  __device__ __forceinline__ int sees(const PromptParams& p, int t) const {
    return (p.causal ? max(0, min(keys, seen + t)) : keys) - skipped;
  }
  template <bool kTaken, bool kAlone = false>
  __device__ __forceinline__ bool next(const PromptParams& p, Walk& walk) {
    const int per = p.sets * (p.heads / p.group);
    int at, u, from = 0, take = INT32_MAX;
    piece = 0, pieces = 1, first_cta = blockIdx.x;
    bool found = false;
    while (walk.h.shares && walk.left > 0 && !found) {
      at = walk.item, u = walk.unit, from = walk.tile;
      const int tiles = p.items[at].tiles;
      const int end = min(tiles + kUnitCost, from + walk.left);
      walk.left -= end - from;
      walk.tile = end;
      if (end == tiles + kUnitCost) {
        walk.tile = 0;
        if (++walk.unit == per) walk.unit = 0, ++walk.item;
      }
      take = min(end, tiles) - from;
      found = take > 0;
      if (found && take < tiles) {
        const int begin = p.items[at].start + u * (tiles + kUnitCost);
        first_cta = walk.share_of(begin);
        pieces = walk.share_of(begin + tiles - 1) - first_cta + 1;
        piece = blockIdx.x - first_cta;
      }
    }
    if (!found) {
      take = INT32_MAX, from = 0;
      int index;
      if (kTaken && !walk.h.shares) {
        index = walk.take<kAlone>(p);
      } else {  // beside shares those without keys
        const int grid = gridDim.x, me = blockIdx.x;
        index = walk.round * grid + ((walk.round & 1) ? grid - 1 - me : me) +
                (walk.h.shares ? walk.h.with_keys * per : 0);
        ++walk.round;
      }
      if (index < 0) return false;
      at = index / per;
      if (at >= walk.h.items) return false;
      u = index - at * per;
    }
    kv_head = u / p.sets;
    head = kv_head * p.group + (u - kv_head * p.sets) * p.set_heads;
    const int4 a = reinterpret_cast<const int4*>(p.items + at)[0];
    row = a.x, rows = a.y, key = a.z + from * kTok, keys = a.w;
    seen = p.items[at].seen;
    skipped = from * kTok;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int t0 = i * p.tile_tokens, live = min(p.tile_tokens, rows - t0);
      lo[i] = live > 0 ? sees(p, t0) : 0;
      n[i] = live > 0 ? min(take, max(0, (sees(p, t0 + live - 1) + kTok - 1) / kTok)) : 0;
    }
    return true;
  }
  __device__ __forceinline__ int tiles() const { return max(n[0], n[1]); }
  // The cleaner goes over tile j: rows see different parts of it, or a row tile ends with it before
  // the other does (so that none ends before the cleaner has come to the item).
  __device__ __forceinline__ bool cleaned(int j) const {
    const int end = min(n[0] > 0 ? n[0] : n[1], n[1] > 0 ? n[1] : n[0]);
    return j + 1 == end || (j < n[0] && j >= lo[0] / kTok) || (j < n[1] && j >= lo[1] / kTok);
  }
  // first key of tile j, from its start, that some row of a row tile that takes it may not see
  __device__ __forceinline__ int masked_from(int j) const {
    int x = kTok;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (j < n[i]) x = min(x, max(0, lo[i] - j * kTok));
    return x;
  }
};

// ------------------------------------------------------------------ items

// One CTA: the sequences' items, by the number of their key tiles, longest first; then whether CTAs
// take whole units or equal shares, and where the shares begin. Latency-bound (some 5 us, of which
// the attention's start covers its barriers and tensor memory): a sort in shared memory needs no
// second launch, and the lengths stay on the device.
//
// Whole units are read by neighbouring CTAs at the same time, and nothing is joined; but their ends
// leave SMs idle where there are few of them. Equal shares end together, and cut units are joined
// through the workspace. Whole units against equal shares: 512 units of 49 to 64 tiles (2048 rows
// behind 6144 keys, 64 heads of 128 dims) 340 against 325 us, of 64 dims 297 against 277; behind
// 32768 keys 1537 against 1420; 32 units of 130 tiles (512 rows behind 16384 keys, 16 heads of 192
// dims) 326 against 132. Where units are even enough, whole ones are better: four prompts of 128
// heads 2335 against 3150, 24 ragged prompts 495 against 560, 512 units of 18 to 32 tiles 286
// against 318, one prompt of 1500 rows 33 against 49. The choice goes by the load of units dealt in
// turns, there and back; where CTAs take them as they come by (192 dims) their loads are more even
// than that, so near the border units may be cut that need not be.
__global__ void __launch_bounds__(kItemThreads)
prompt_items_kernel(int batch, int rows, int keys, int causal, int tile_tokens, int max_items,
                    int per, int grid, const int32_t* __restrict__ cu_q,
                    const int32_t* __restrict__ cu_k, Header* header, Start* starts, Item* items,
                    int* arrived, int* ticket, uint32_t* status) {
  __shared__ int s_end[kMaxSeqs];  // items up to and with each sequence
  __shared__ int s_bucket[kBuckets];
  __shared__ int s_warp[32];
  __shared__ int s_before;
  grid_launch_dependents();  // the attention sets itself up meanwhile
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int pair = 2 * tile_tokens;
  // Sequences that overlap could name more items than the rows allow, and more than fit 31 bits:
  // their sums stay at one more than there may be.
  const unsigned cap = (unsigned)max_items + 1u;
  if (tid == 0) s_before = 0;
  s_bucket[tid] = 0;
  __syncthreads();
  for (int b0 = 0; b0 < batch; b0 += kItemThreads) {
    const int b = b0 + tid;
    unsigned n = 0;
    if (b < batch) {
      const int q0 = cu_q[b], q1 = cu_q[b + 1], k0 = cu_k[b], k1 = cu_k[b + 1];
      if (q0 < 0 || q1 < q0 || q1 > rows || k0 < 0 || k1 < k0 || k1 > keys)
        raise_status(status, DCP_STATUS_BAD_SEQ_LEN);
      else
        n = min((unsigned)(q1 - q0 + pair - 1) / pair, cap);
    }
    unsigned x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const unsigned y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x = min(x + y, cap);
    }
    if (lane == 31) s_warp[warp] = (int)x;
    __syncthreads();
    if (warp == 0) {
      unsigned y = s_warp[lane];
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const unsigned z = __shfl_up_sync(0xffffffffu, y, o);
        if (lane >= o) y = min(y + z, cap);
      }
      s_warp[lane] = (int)y;
    }
    __syncthreads();
    const unsigned before = min((unsigned)s_before + (warp > 0 ? s_warp[warp - 1] : 0), cap);
    const int end = (int)min(before + x, cap);
    if (b < batch) s_end[b] = end;
    __syncthreads();
    if (tid == kItemThreads - 1) s_before = end;
    __syncthreads();
  }
  const int total = min(s_before, max_items);
  if (tid == 0 && s_before > max_items) raise_status(status, DCP_STATUS_BAD_SEQ_LEN);
  auto item_of = [&](int i, Item& it) {
    int lo = 0, hi = batch - 1;  // the first sequence that ends behind i
    while (lo < hi) {
      const int mid = (lo + hi) >> 1;
      if (s_end[mid] > i) hi = mid;
      else lo = mid + 1;
    }
    const int at = (i - (lo > 0 ? s_end[lo - 1] : 0)) * pair;
    const int q0 = cu_q[lo], n = cu_q[lo + 1] - q0, k0 = cu_k[lo], m = cu_k[lo + 1] - k0;
    it.row = q0 + at;
    it.rows = min(pair, n - at);
    it.key = k0;
    it.keys = m;
    it.seen = m - n + 1 + at;
    const int most = causal ? max(0, min(m, it.seen + it.rows - 1)) : m;
    it.tiles = (int)(((int64_t)most + kTok - 1) / kTok);
    // those without keys last, and by themselves
    return it.tiles == 0 ? kBuckets - 1 : kBuckets - 1 - min(kBuckets - 1, 1 + it.tiles);
  };
  // Items of one bucket stand in their own order: where shares begin, and so which units are cut and
  // where, goes by the list, and a cut unit is rounded differently. A few items are placed by the
  // number of those in front of them; many by counting the buckets, in which the warps that have
  // items take their places in turn, lanes of one bucket in their order. (One prompt of 200 rows
  // 14.4 us, 15.7 by buckets; 1000 of two rows 261.4, of which the turns are 1.2.)
  Item it;
  int bucket = tid < total ? item_of(tid, it) : -1;
  auto place = [&](int at) {
    reinterpret_cast<int4*>(items + at)[0] = make_int4(it.row, it.rows, it.key, it.keys);
    items[at].seen = it.seen;
    items[at].tiles = it.tiles;
  };
  if (total <= kFewItems) {
    s_bucket[tid] = bucket;
    __syncthreads();
    if (bucket >= 0) {
      int at = 0;
      for (int j = 0; j < total; ++j) {
        const int x = s_bucket[j];
        at += x < bucket || (x == bucket && j < tid);
      }
      place(at);
    }
  } else {
#pragma unroll 1
    for (int pass = 0; pass < 2; ++pass) {  // counted, then placed
#pragma unroll 1
      for (int i0 = 0; i0 < total; i0 += kItemThreads) {
        if (total > kItemThreads) bucket = i0 + tid < total ? item_of(i0 + tid, it) : -1;
        if (pass == 0) {
          if (bucket >= 0) atomicAdd(&s_bucket[bucket], 1);
          continue;
        }
        unsigned peers = 0xffffffffu;
#pragma unroll 1
        for (int k = 1; k <= kBuckets; k <<= 1) {
          const unsigned ones = __ballot_sync(0xffffffffu, bucket & k);
          peers &= bucket & k ? ones : ~ones;
        }
        const int rank = __popc(peers & ((1u << lane) - 1u));
        const int turns = min(kItemThreads / 32, (total - i0 + 31) / 32);
        int at = 0;
#pragma unroll 1
        for (int w = 0; w < turns; ++w) {
          if (w == warp) {
            if (bucket >= 0) at = s_bucket[bucket] + rank;
            __syncwarp();
            if (bucket >= 0 && rank == 0) s_bucket[bucket] += __popc(peers);
          }
          __syncthreads();
        }
        if (bucket >= 0) place(at);
      }
      if (pass == 1) break;
      __syncthreads();
      int x = s_bucket[tid];
      const int own = x;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      if (lane == 31) s_warp[warp] = x;
      __syncthreads();
      int before = 0;
      for (int w = 0; w < warp; ++w) before += s_warp[w];
      s_bucket[tid] = before + x - own;
      __syncthreads();
    }
  }
  for (int i = tid; i < grid * kSoftWarps; i += kItemThreads) arrived[i] = 0;
  if (tid == 0) *ticket = 0;
  __syncthreads();

  // Where the items' units begin in the row of all units.
  __shared__ int64_t s_tiles[32];
  __shared__ int s_keys[32], s_long[32];
  const int each_item = (total + kItemThreads - 1) / kItemThreads;
  const int i0 = min(total, tid * each_item), i1 = min(total, i0 + each_item);
  int64_t mine = 0;
  int with_keys = 0, longest = 0;
  for (int i = i0; i < i1; ++i) {
    const int n = items[i].tiles;
    longest = max(longest, n);
    mine += n > 0 ? (int64_t)(n + kUnitCost) * per : 0;
    with_keys += n > 0;
  }
  int64_t x = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  with_keys = __reduce_add_sync(0xffffffffu, with_keys);
  longest = __reduce_max_sync(0xffffffffu, longest);
  if (lane == 31) s_tiles[warp] = x, s_keys[warp] = with_keys, s_long[warp] = longest;
  __syncthreads();
  int64_t before = x - mine, all = 0;
  with_keys = 0;
  for (int w = 0; w < 32; ++w) {
    if (w < warp) before += s_tiles[w];
    all += s_tiles[w];
    with_keys += s_keys[w];
    longest = max(longest, s_long[w]);
  }
  // Whole units, or equal shares: by what the busiest CTA would have to do. Cutting units costs
  // about kCutCost, and shares lose a twentieth where CTAs no longer read the same keys together.
  constexpr int kCutCost = 20;
  __shared__ int s_most, s_load[kMaxCtas];
  const int64_t in_shares = all / grid * 21 / 20 + kCutCost;
  const unsigned units = (unsigned)with_keys * per;
  const int64_t rounds = (units + grid - 1) / grid;
  bool shares = all <= 1 << 30 && all >= grid && rounds * (longest + kUnitCost) > in_shares;
  if (shares) {  // not ruled out
    if (tid == 0) s_most = 0;
    if (tid < kMaxCtas) s_load[tid] = 0;
    __syncthreads();
    for (unsigned i = tid; i < units; i += kItemThreads) {
      const unsigned r = i / grid, x = i - r * grid;
      atomicAdd(&s_load[(r & 1) ? grid - 1 - x : x], items[i / per].tiles + kUnitCost);
    }
    __syncthreads();
    if (tid < grid) atomicMax(&s_most, s_load[tid]);
    __syncthreads();
    shares = s_most > in_shares;
  }
  if (shares) {
    int64_t at = before;
    const int each = (int)(all / grid), more = (int)(all - (int64_t)each * grid);
    for (int i = i0; i < i1; ++i) {
      const int n = items[i].tiles;
      items[i].start = (int)at;
      const int64_t end = at + (n > 0 ? (int64_t)(n + kUnitCost) * per : 0);
      // the CTAs whose shares begin in this item
      const int64_t longer = (int64_t)more * (each + 1);  // the first `more` shares
      int c = at < longer ? (int)((at + each) / (each + 1))
                          : more + (int)((at - longer + each - 1) / each);
      for (; c < grid; ++c) {
        const int64_t lo = (int64_t)each * c + min(c, more);
        if (lo >= end) break;
        const int in = (int)(lo - at), u = in / (n + kUnitCost);
        starts[c] = Start{i, u, in - u * (n + kUnitCost), 0};
      }
      at = end;
    }
  }
  if (tid == 0)
    *header = Header{total, with_keys, shares ? 1 : 0, (int)min(all, (int64_t)INT32_MAX)};
}

// ------------------------------------------------------------------ attention
//
// Bound by the tensor cores (their pipe is active for 71% of a long chunk's cycles). So two row
// tiles take turns: one's softmax runs beside the other's products. With 64 dims, where half as
// many products stand beside each score, no unit is full (tensor pipe 37%, special functions 37%,
// issue 40%): a row tile's next scores wait until its weights, which stand in their place, are used
// up.
// Scores become weights in the place where they stand, in tensor memory, as the second product's
// first operand; O stays there as well (4 x 128 columns in all), and is touched only where a row's
// maximum jumps (by 2^8). Row tiles hold the heads of a group beside the tokens, so K and V are
// read once for a group.
//
// Measured (64 query heads, 8 K/V heads): 2048 rows behind 6144 keys, 128 dims, 323 us, 1490
// TFLOP/s (without softmax 318: what is left are the starts and ends of the products' chains); 64
// dims 264 to 278 us; behind 32768 keys, 128 dims, 1560 us, 1450 TFLOP/s. 192 and 128 dims (64 K/V
// heads, 2048 rows behind 2048 keys) 265 us: a ring of 128 KB holds one tile of K and V and
// half of the next, and the products wait for copies some 1500 cycles a tile; two CTAs with one
// ring over both of their shared memories would need half the copies each.
template <int kDq, int kDv>
__global__ void __launch_bounds__(kThreads, 1)
prompt_kernel(const PromptParams p, const __grid_constant__ CUtensorMap q_map,
              const __grid_constant__ CUtensorMap k_map,
              const __grid_constant__ CUtensorMap v_map) {
  using T = Shape<kDq, kDv>;
  // Where the ring is short, products wait for memory, for some CTAs a tenth longer than for
  // others: taking units evens that out (2275 to 2138 us for four prompts of 128 heads of 192 dims,
  // 510 to 465 for 4096 rows behind 4096 keys, 32 heads). Elsewhere units are as long as their
  // tiles say, and what is told at each unit's start costs more (482 to 534 us for 24 ragged
  // prompts, 202 to 214 for 4096 rows, 64 heads of 128 dims).
  constexpr bool kTaken = !T::kAhead;
  extern __shared__ __align__(1024) uint8_t smem[];
  Rest& rest = *reinterpret_cast<Rest*>(smem + T::kRest);
  Bars& bar = rest.bar;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const uint32_t base = smem_u32(smem);
  const uint32_t ring = base + 2 * T::kQTile;
  if (tid == 0) {
    for (int i = 0; i < T::kSlots; ++i) {
      mbar_init(&bar.full[i], 1);
      mbar_init(&bar.empty[i], 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bar.qfull[i], 1);
      mbar_init(&bar.qempty[i], 1);
      mbar_init(&bar.sfull[i], 1);
      mbar_init(&bar.pfull[i], kSoftWarps / 2 + 1);
      mbar_init(&bar.ofull[i], 1);
      mbar_init(&bar.done[i], kSoftWarps / 2);
    }
    mbar_init(&bar.drain, 1);
    mbar_init(&bar.want, 1);
    mbar_init(&bar.told, 1);
    mbar_init(&bar.heard, kRoles);
    fence_mbarrier_init_cluster();
    rest.abort_flag = 0;
    rest.again = rest.dirty = 0;
  }
  if (warp == kSoftWarps) tmem_alloc(&rest.tmem, 512);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = rest.tmem;
  // tensor memory columns: scores (and weights, in their place) of both row tiles, then O
  constexpr int kColO = 2 * kTok;
  grid_dependency_wait();  // the items
  int* const abort_flag = &rest.abort_flag;
  // A weight of zero times an infinity or NaN is NaN, and a row's weights for keys that it does not
  // see are zeros. So where a row comes out with either, the CTA goes over its units a second time,
  // and its cleaner over V. (Behind a sequence's last key, where anything may stand, V is zeroed in
  // the first pass already.) Every warp comes here at the end of a pass.
  auto another = [&](int pass) {
    __syncwarp();
    named_bar_sync(1, kThreads);
    return pass == 0 && *reinterpret_cast<volatile int*>(&rest.again) != 0 &&
           *reinterpret_cast<volatile int*>(abort_flag) == 0;
  };

  if (warp < kSoftWarps) {
    // ---------------- softmax: a thread to a row. (Two, with half as many registers, have to tell
    // each other their maxima: 365 us where one takes 348, for 2048 rows behind 6144 keys.)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int side = warp >> 2;
    const int r = tid & 127;  // row of the tile = its tensor memory lane
    const int t = p.set_div.div(r), h = r - t * p.set_heads;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;
    const uint32_t t_s = tmem + lanes + side * kTok, t_o = tmem + lanes + kColO + side * kDv;
    uint32_t sphase = 0, ophase = 0, left = 0;  // left: pieces that this warp has left for joining
    int pass = 0;
    Walk walk(p, rest);
    do {
      walk.begin(p);
      Work w;
      while (w.next<kTaken>(p, walk)) {
        const int token = side * p.tile_tokens + t;
        const int mine = w.sees(p, token);
        float m = -INFINITY, l = 0.f;
        bool ok = true;
        uint32_t x[4][32];
        auto largest = [](const uint32_t(&z)[32]) {
          auto of = [&z](int i) { return __uint_as_float(z[i]); };
          float a = max3(of(0), of(1), of(2)), b = max3(of(3), of(4), of(5));
#pragma unroll
          for (int i = 6; i < 30; i += 4) {
            a = max3(a, of(i), of(i + 1));
            b = max3(b, of(i + 2), of(i + 3));
          }
          return max3(fmaxf(a, b), of(30), of(31));
        };
        for (int j = 0; j < w.n[side]; ++j) {
          ok = wait_warp(&bar.sfull[side], sphase, abort_flag, p.status);
          if (!ok) break;
          sphase ^= 1;
          tc_fence_after();
          // The weights are formed with the maximum so far, which may lag behind the true one by
          // 2^8 (they then reach 2^8, which costs no bits), while the true one is found: nothing
          // waits for it. The first tile begins with the largest of its first 32 scores.
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_ld32(t_s + 32 * c, x[c]);
#pragma unroll
          for (int c = 0; c < 4; ++c) tmem_wait_ld(x[c]);
          const bool masked = (j + 1) * kTok > w.lo[side];
          const int limit = mine - j * kTok;
          if (masked) {
#pragma unroll
            for (int c = 0; c < 4; ++c) {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (32 * c + i >= limit) x[c][i] = 0xff800000u;
            }
          }
          if (j == 0) {
            m = largest(x[0]) * p.scale;
            if (!(m > -INFINITY)) m = -INFINITY;  // NaN as well
          }
          const uint64_t scale2 = pack_f32(p.scale, p.scale);
          float shift = m == -INFINITY ? 0.f : m;
          uint64_t shift2 = pack_f32(-shift, -shift), sum[2] = {0, 0};
          uint32_t pk[64];
          float top[4];
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            top[c] = largest(x[c]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint64_t s2 = fma_f32x2(pack_b32(x[c][2 * i], x[c][2 * i + 1]), scale2, shift2);
              const float a = exp2_fast(low_f32(s2)), b = exp2_fast(high_f32(s2));
              sum[i & 1] = add_f32x2(sum[i & 1], pack_f32(a, b));
              pk[16 * c + i] = pack_bf16(a, b);
            }
          }
          const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]) * p.scale;
          const bool jumps = most > m + 8.f;
          if (!__any_sync(0xffffffffu, jumps)) {
            tmem_st32(t_s, *reinterpret_cast<const uint32_t(*)[32]>(&pk[0]));
            tmem_st32(t_s + 32, *reinterpret_cast<const uint32_t(*)[32]>(&pk[32]));
          } else {
            // Where a row's maximum jumps further (that row's alone: no row depends on those beside
            // it), O is scaled anew and the warp's weights are formed again, in few instructions:
            // this happens once or twice in a unit.
            const float by = jumps ? exp2_fast(m - most) : 1.f;
            m = jumps ? most : m;
            l *= by;
            if (j > 0) {  // the scores' barrier says that the products before them are done
#pragma unroll 1
              for (int c = 0; c < kDv / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(t_o + 32 * c, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * by);
                tmem_st32(t_o + 32 * c, o);
              }
            }
            shift = m == -INFINITY ? 0.f : m;
            shift2 = pack_f32(-shift, -shift);
            sum[0] = sum[1] = 0;
#pragma unroll 1
            for (int c = 0; c < 4; ++c) {  // the weights' columns are of scores read before
              uint32_t z[32], q[16];
              tmem_ld32(t_s + 32 * c, z);
              tmem_wait_ld(z);
#pragma unroll
              for (int i = 0; i < 16; ++i) {
                if (masked && 32 * c + 2 * i >= limit) z[2 * i] = 0xff800000u;
                if (masked && 32 * c + 2 * i + 1 >= limit) z[2 * i + 1] = 0xff800000u;
                const uint64_t s2 = fma_f32x2(pack_b32(z[2 * i], z[2 * i + 1]), scale2, shift2);
                const float a = exp2_fast(low_f32(s2)), b = exp2_fast(high_f32(s2));
                sum[i & 1] = add_f32x2(sum[i & 1], pack_f32(a, b));
                q[i] = pack_bf16(a, b);
              }
              tmem_st16(t_s + 16 * c, q);
            }
          }
          sum[0] = add_f32x2(sum[0], sum[1]);
          l += low_f32(sum[0]) + high_f32(sum[0]);
          tmem_wait_st();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&bar.pfull[side]);
        }
        if (ok && w.n[side] > 0) {
          ok = wait_warp(&bar.ofull[side], ophase, abort_flag, p.status);
          ophase ^= 1;
          tc_fence_after();
        }
        if (!ok) break;
        const bool live = r < p.tile_tokens * p.set_heads && token < w.rows &&
                          w.head + h < (w.kv_head + 1) * p.group;
        const int64_t at = (int64_t)(w.row + token) * p.heads + w.head + h;
        float inv = l == 0.f ? 0.f : 1.f / l;
        const bool cut = w.pieces > 1;
        const int half_warp = side * 4 + (warp & 3);
        auto part_of = [&](int piece) {  // of this unit, this thread's column
          const int cta = w.first_cta + piece;
          const int64_t at = ((int64_t)cta * 2 + (piece == 0 ? 1 : 0)) * 2 + side;
          return p.parts + at * (kDv + 2) * kRows + r;
        };
        float* const part = part_of(w.piece);
        auto store = [&](int c, const float (&y)[32]) {  // 32 dims of the row
          if (!live) return;
          uint16_t* dst = p.out + at * kDv + 32 * c;
          const bool none = l == 0.f;  // no key: 0, whatever O holds
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t z[8];
#pragma unroll
            for (int e = 0; e < 8; ++e)
              z[e] = none ? 0u : pack_bf16(y[16 * i + 2 * e] * inv, y[16 * i + 2 * e + 1] * inv);
            asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(
                             dst + 16 * i),
                         "r"(z[0]), "r"(z[1]), "r"(z[2]), "r"(z[3]), "r"(z[4]), "r"(z[5]),
                         "r"(z[6]), "r"(z[7])
                         : "memory");
          }
        };
        float odd = 0.f;  // NaN where O is not finite
        const bool dirty = *reinterpret_cast<volatile int*>(&rest.dirty) != 0;
#pragma unroll 1
        for (int c = 0; c < kDv / 32; ++c) {
          uint32_t o[32];
          float y[32];
          if (w.n[side] > 0) {
            tmem_ld32(t_o + 32 * c, o);
            tmem_wait_ld(o);
          } else {
            if (cut) break;
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) {
            y[i] = __uint_as_float(o[i]);
            odd = fmaf(y[i], 0.f, odd);
          }
          if (dirty) {
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (rest.first[0][32 * c + i] < mine) y[i] += __uint_as_float(0x7fc00000u);
              if (rest.first[1][32 * c + i] < mine) y[i] += INFINITY;
              if (rest.first[2][32 * c + i] < mine) y[i] -= INFINITY;
            }
          }
          if (cut) {
#pragma unroll
            for (int i = 0; i < 32; ++i) __stcg(part + (32 * c + i) * kRows, y[i]);
          } else {
            store(c, y);
          }
        }
        tc_fence_before();
        if (pass == 0 && __any_sync(0xffffffffu, live && !(odd == 0.f))) {
          if (lane == 0) *reinterpret_cast<volatile int*>(&rest.again) = 1;
          if (cut) continue;  // a piece is left once
        }
        __syncwarp();
        if (pass == 1 && lane == 0 && w.n[side] > 0) mbar_arrive(&bar.done[side]);
        if (cut) {
          const uint32_t which = w.piece == 0 ? 1u : 2u;
          if (left & which) continue;
          left |= which;
          // A unit's pieces are joined, in their order, by the warp that is the last to leave its
          // rows: nobody waits, and the result does not depend on who that is.
          __stcg(part + kDv * kRows, m);
          __stcg(part + (kDv + 1) * kRows, l);
          __threadfence();
          __syncwarp();
          int others = 0;
          if (lane == 0) others = atomicAdd(p.arrived + w.first_cta * kSoftWarps + half_warp, 1);
          if (__shfl_sync(0xffffffffu, others, 0) != w.pieces - 1) continue;
          __threadfence();
          m = -INFINITY;
          for (int k = 0; k < w.pieces; ++k)
            if (__ldcg(part_of(k) + (kDv + 1) * kRows) != 0.f)
              m = fmaxf(m, __ldcg(part_of(k) + kDv * kRows));
          l = 0.f;
          for (int k = 0; k < w.pieces; ++k) {
            const float lk = __ldcg(part_of(k) + (kDv + 1) * kRows);
            if (lk != 0.f) l += lk * exp2_fast(__ldcg(part_of(k) + kDv * kRows) - m);
          }
          inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll 1
          for (int c = 0; c < kDv / 32; ++c) {
            float y[32] = {};
            for (int k = 0; k < w.pieces; ++k) {
              const float* from = part_of(k);
              if (__ldcg(from + (kDv + 1) * kRows) == 0.f) continue;  // O was not written
              const float by = exp2_fast(__ldcg(from + kDv * kRows) - m);
              float z[32];
#pragma unroll
              for (int i = 0; i < 32; ++i) z[i] = __ldcg(from + (32 * c + i) * kRows);
#pragma unroll
              for (int i = 0; i < 32; ++i) y[i] = fmaf(z[i], by, y[i]);
            }
            store(c, y);
          }
        }
        if (live) p.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
      }
    } while (another(pass++));
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == kSoftWarps) {
      // ---------------- issuer: the whole warp waits, one lane issues. What it does between two
      // chains of products is time that the tensor cores stand still: it waits for one barrier to a
      // chain (with one for each slot besides, 421 us where this took 399), and forms nothing
      // between the products of a chain. Two issuers, one to a row tile, interleave their chains,
      // and each then takes as long as both (555 us).
      constexpr uint32_t id_s = idesc_f16(kRows, kTok, true, false);
      constexpr uint32_t id_o = idesc_f16(kRows, kDv, true, true);
      const uint32_t q_desc = (uint32_t)smem_desc_sw128(base, 16, 1024);
      const uint32_t k_desc = (uint32_t)smem_desc_sw128(ring, 16, 1024);
      const uint32_t v_desc = (uint32_t)smem_desc_sw128(ring, T::kVTok * 128, 1024);
      const uint32_t desc_hi = (uint32_t)(smem_desc_sw128(0, 0, 1024) >> 32);
      uint32_t slot = 0, phase = 0, qphase = 0, pphase = 0;  // the latter a bit for each row tile
      bool ok = true;
      auto move = [&](int n) {
        slot += n;
        if (slot >= T::kSlots) slot -= T::kSlots, phase ^= 1;
      };
      auto slot_at = [&](uint32_t s, int c) {
        return s + c < T::kSlots ? s + c : s + c - T::kSlots;
      };
      // Scores of row tile i with the tile of K whose slots begin at s; `ends`: no other row tile
      // uses them after this one; `last`: of the item. Where the ring is short, its slots are
      // waited for one by one, and each is free as soon as its own products are done.
      auto scores = [&](int i, uint32_t s, bool ends, bool last) {
        const uint32_t a = here(q_desc + i * (T::kQTile / 16));
        const uint32_t d = here(tmem + i * kTok);
#pragma unroll
        for (int c = 0; c < T::kKSlots; ++c) {
          const uint32_t at = slot_at(s, c);
          const uint32_t b = k_desc + at * (T::kSlot / 16);
          if (!T::kAhead) {  // (slot, phase) is behind the tile already
            const uint32_t of = at < slot ? phase : phase ^ 1;
            ok = ok && wait_warp(&bar.full[at], of, abort_flag, p.status);
            if (!ok) return;
            tc_fence_after();
          }
          if (elect_one()) {
#pragma unroll
            for (int e = 0; e < T::kKSlices; ++e)
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                mma_f16_ss_lo(d, a + (c * T::kKSlices + e) * (T::kQSlice / 16) + 2 * kk,
                              b + e * (kTok * 128 / 16) + 2 * kk, desc_hi, id_s,
                              c > 0 || e > 0 || kk > 0);
            if (c + 1 == T::kKSlots) tc_commit(&bar.sfull[i]);
            if (ends) tc_commit(&bar.empty[at]);
            if (last && c + 1 == T::kKSlots) tc_commit(&bar.qempty[i]);
          }
          __syncwarp();
        }
      };
      int pass = 0;
      Walk walk(p, rest);
      do {
        walk.begin(p);
        Work w;
        while (ok && w.next<kTaken>(p, walk)) {
          const int tiles = w.tiles();
          if (tiles == 0) continue;
          uint32_t ks = slot;
          move(T::kKSlots);
          if (T::kAhead)
            ok = wait_warp(&bar.full[ks], slot == 0 ? phase ^ 1 : phase, abort_flag, p.status);
          for (int i = 0; i < 2 && ok; ++i) {
            if (w.n[i] == 0) continue;
            ok = wait_warp(&bar.qfull[i], qphase >> i & 1, abort_flag, p.status);
            if (!ok) break;
            qphase ^= 1u << i;
            tc_fence_after();
            scores(i, ks, i == 1 || w.n[1] == 0, w.n[i] == 1);
          }
          for (int j = 0; ok && j < tiles; ++j) {
            const uint32_t vs = slot;
            move(T::kVSlots);
            ks = slot;
            if (j + 1 < tiles) move(T::kKSlots);
            const uint32_t add = j > 0 ? 1u : 0u;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int n = w.n[i];
              if (!ok || j >= n) continue;
              ok = wait_warp(&bar.pfull[i], pphase >> i & 1, abort_flag, p.status);
              if (!ok) continue;
              pphase ^= 1u << i;
              tc_fence_after();
              if (elect_one()) {
                const uint32_t d = here(tmem + kColO + i * kDv), a = here(tmem + i * kTok);
#pragma unroll
                for (int c = 0; c < T::kVSlots; ++c) {
                  const uint32_t at = slot_at(vs, c);
                  const uint32_t b = v_desc + at * (T::kSlot / 16);
#pragma unroll
                  for (int kk = 0; kk < T::kVTok / 16; ++kk)
                    mma_f16_ts_lo(d, a + 8 * (c * (T::kVTok / 16) + kk), b + kk * 128, desc_hi,
                                  id_o, c > 0 || kk > 0 ? 1u : add);
                  if (i == 1 || j >= w.n[1]) tc_commit(&bar.empty[at]);
                }
                if (j + 1 == n) tc_commit(&bar.ofull[i]);
              }
              __syncwarp();
              if (j + 1 < n) scores(i, ks, i == 1 || j + 1 >= w.n[1], j + 2 == n);
            }
          }
        }
      } while (another(pass++));
      // every product is done before tensor memory is freed and shared memory is left
      __syncwarp();
      tc_commit_elect(&bar.drain);
      wait_landed(&bar.drain, 0);
    } else if (warp == kSoftWarps + 1) {
      // ---------------- copier: one thread
      tma_prefetch_map(&q_map);
      tma_prefetch_map(&k_map);
      tma_prefetch_map(&v_map);
      uint32_t slot = 0, phase = 0, qphase = 0, q_issued = 0;  // the latter a bit for each row tile
      int issued = 0;
      bool ok = true;
      int pass = 0;
      Walk walk(p, rest);
      do {
        if (lane == 0) {
          walk.begin(p);
          auto want = [&]() {
            if (kTaken && !walk.h.shares) mbar_arrive(&bar.want);
          };
          want();
          Work w;
          while (ok && w.next<kTaken, true>(p, walk)) {
            const int tiles = w.tiles();
            if (tiles == 0) {
              want();
              continue;
            }
            auto take = [&]() {
              ok = wait_one(&bar.empty[slot], phase ^ 1, abort_flag, p.status);
              if (ok) mbar_arrive_expect_tx(&bar.full[slot], T::kSlot);
              return ok;
            };
            auto moved = [&]() {
              ++issued;
              if (++slot == T::kSlots) slot = 0, phase ^= 1;
            };
            auto queries = [&](int i) {
              if (w.n[i] == 0) return;
              ok = wait_one(&bar.qempty[i], (qphase >> i & 1) ^ 1, abort_flag, p.status);
              if (!ok) return;
              qphase ^= 1u << i;
              q_issued |= 1u << i;
              mbar_arrive_expect_tx(&bar.qfull[i],
                                    (uint32_t)(p.tile_tokens * p.set_heads * kDq * 2));
#pragma unroll
              for (int c = 0; c < kDq / 64; ++c)
                tma_load_3d(base + i * T::kQTile + c * T::kQSlice, &q_map, 64 * c, w.head,
                            w.row + i * p.tile_tokens, smem_u32(&bar.qfull[i]));
            };
            auto keys = [&](int j) {
#pragma unroll
              for (int c = 0; c < T::kKSlots; ++c) {
                if (!take()) return;
                tma_load_4d(ring + slot * T::kSlot, &k_map, 0, w.key + j * kTok, c * T::kKSlices,
                            w.kv_head, smem_u32(&bar.full[slot]));
                moved();
              }
            };
            queries(0);
            if (ok) keys(0);
            if (ok) queries(1);
            for (int j = 0; ok && j < tiles; ++j) {
              if (j > 0) keys(j);
              if (j == max(0, tiles - 2)) want();
#pragma unroll
              for (int c = 0; c < T::kVSlots && ok; ++c) {
                if (!take()) break;
                tma_load_4d(ring + slot * T::kSlot, &v_map, 0, w.key + j * kTok + c * T::kVTok, 0,
                            w.kv_head, smem_u32(&bar.full[slot]));
                moved();
              }
            }
          }
        }
      } while (another(pass++));
      // Nothing may be in flight when the CTA ends: after a timeout the copies that nobody waited
      // for are waited for here (bounded).
      if (lane == 0 && *reinterpret_cast<volatile int*>(abort_flag) != 0) {
        for (int i = max(0, issued - T::kSlots); i < issued; ++i)
          wait_landed(&bar.full[i % T::kSlots], (uint32_t)(i / T::kSlots & 1));
        for (int i = 0; i < 2; ++i)
          if (q_issued >> i & 1) wait_landed(&bar.qfull[i], (qphase >> i & 1) ^ 1);
      }
    } else if (warp == kSoftWarps + 2) {
      // ---------------- cleaner: zeroes V behind the sequence's last key. In a second pass, in
      // tiles that rows see different parts of, infinities and NaN of V become zeros; the first key
      // of each kind and dim is kept, and added to the rows that see it. (In the first pass this
      // held up the end of every unit: 5300 cycles of waiting, now 1900; 348 against 324 us for
      // 2048 rows behind 6144 keys, 682 against 491 for 24 ragged prompts.)
      constexpr int kChunks = kDv / 8;  // 16-byte chunks of a row
      auto reset = [&]() {
        for (int i = lane; i < 3 * 128; i += 32) (&rest.first[0][0])[i] = INT32_MAX;
        __syncwarp();
      };
      reset();
      uint32_t slot = 0, phase = 0, dphase[2] = {0, 0};
      uint32_t gates[2] = {0, 0};  // arrivals at pfull
      bool ok = true, wrote[2] = {false, false};  // row tiles of the last item that had keys
      // Every slot is waited for in turn, and none is refilled before it has been: a parity that
      // was not waited for could be taken for a later one.
      auto used = [&]() {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bar.empty[slot]);
        if (++slot == T::kSlots) slot = 0, phase ^= 1;
      };
      int pass = 0;
      Walk walk(p, rest);
      do {
        const bool clean = pass == 1;
        walk.begin(p);
        Work w;
        while (ok && w.next<kTaken>(p, walk)) {
          const int tiles = w.tiles();
          bool first_clean = true;
          auto keys = [&]() {
            for (int c = 0; ok && c < T::kKSlots; ++c) {
              ok = wait_warp(&bar.full[slot], phase, abort_flag, p.status);
              if (ok) used();
            }
          };
          if (tiles > 0) keys();
          for (int j = 0; ok && j < tiles; ++j) {
            const bool cleaned = clean && w.cleaned(j);
            const int from = clean ? w.masked_from(j) : kTok;
            const int end = min(kTok, w.keys - w.skipped - j * kTok);  // of the sequence
            if (ok && cleaned && first_clean) {  // the last item's rows are written
              first_clean = false;
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                if (ok && wrote[i]) {
                  ok = wait_warp(&bar.done[i], dphase[i], abort_flag, p.status);
                  dphase[i] ^= 1;
                }
                wrote[i] = w.n[i] > 0;
              }
              if (ok && *reinterpret_cast<volatile int*>(&rest.dirty) != 0) {
                reset();
                if (lane == 0) *reinterpret_cast<volatile int*>(&rest.dirty) = 0;
                __syncwarp();
              }
            }
            for (int c = 0; ok && c < T::kVSlots; ++c) {
              ok = wait_warp(&bar.full[slot], phase, abort_flag, p.status);
              if (!ok) break;
              if (end < (c + 1) * T::kVTok) {
                const int first = max(0, end - c * T::kVTok);
                for (int i = lane; i < (T::kVTok - first) * kChunks; i += 32) {
                  const int key = first + i / kChunks, chunk = i % kChunks;
                  asm volatile("st.shared.v4.u32 [%0], {%1, %1, %1, %1};" ::"r"(
                                   ring + slot * T::kSlot + (chunk >> 3) * T::kVTok * 128 +
                                   sw128_offset(key, chunk & 7)),
                               "r"(0)
                               : "memory");
                }
                fence_proxy_async_smem();
              }
              const int first = min(T::kVTok, max(0, from - c * T::kVTok));
              const int pieces = (T::kVTok - first) * kChunks;
#pragma unroll 4
              for (int i = lane; i < pieces; i += 32) {
                const int key = first + i / kChunks, chunk = i % kChunks;
                const uint32_t addr = ring + slot * T::kSlot + (chunk >> 3) * T::kVTok * 128 +
                                      sw128_offset(key, chunk & 7);
                uint32_t y[4];
                asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                             : "=r"(y[0]), "=r"(y[1]), "=r"(y[2]), "=r"(y[3])
                             : "r"(addr));
                uint32_t odd = 0;  // an exponent of ones carries into its half's sign bit
#pragma unroll
                for (int u = 0; u < 4; ++u) odd |= (y[u] & 0x7f807f80u) + 0x00800080u;
                if (odd & 0x80008000u) {
#pragma unroll
                  for (int u = 0; u < 8; ++u) {
                    const uint32_t v = y[u >> 1] >> (16 * (u & 1)) & 0xffffu;
                    if ((v & 0x7f80u) != 0x7f80u) continue;
                    const int kind = (v & 0x7fu) ? 0 : (v & 0x8000u) ? 2 : 1;
                    atomicMin(&rest.first[kind][8 * chunk + u], j * kTok + c * T::kVTok + key);
                    y[u >> 1] &= ~(0xffffu << (16 * (u & 1)));
                  }
                  *reinterpret_cast<volatile int*>(&rest.dirty) = 1;
                  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(y[0]),
                               "r"(y[1]), "r"(y[2]), "r"(y[3])
                               : "memory");
                }
              }
              if (first < T::kVTok) fence_proxy_async_smem();
              used();
            }
            if (T::kAhead && ok && j + 1 < tiles) keys();
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              if (!ok || j >= w.n[i]) continue;
              // not before the last tile's weights are complete: this would count among theirs
              if (gates[i] > 0)
                ok = wait_warp(&bar.pfull[i], (gates[i] - 1) & 1, abort_flag, p.status);
              ++gates[i];
              if (ok && lane == 0) mbar_arrive(&bar.pfull[i]);
            }
            if (!T::kAhead && ok && j + 1 < tiles) keys();
          }
        }
      } while (another(pass++));
    } else {
      // ---------------- units: one thread takes them (kTaken) and tells the others, when the
      // copier is two tiles before its unit's end. In the second pass the CTA goes back over its
      // own.
      const Header h = *p.header;
      const int units = h.shares ? 0 : h.items * p.sets * (p.heads / p.group);
      int last = -1;
      uint32_t told = 0;
      int pass = 0;
      do {
        if (kTaken && lane == 0 && !h.shares) {
          int unit = pass == 0 ? (int)blockIdx.x : last;
          for (bool more = true; more;) {
            if (!wait_one(&bar.want, told & 1, abort_flag, p.status)) break;
            if (pass == 0 && last >= 0) unit = atomicAdd(p.ticket, 1) + (int)gridDim.x;
            more = pass == 0 ? unit < units : unit >= 0;
            if (!wait_one(&bar.heard, (told & 1) ^ 1, abort_flag, p.status)) break;
            *reinterpret_cast<volatile int*>(&rest.unit) = more ? unit : -1;
            mbar_arrive(&bar.told);
            ++told;
            if (!more) break;
            if (pass == 0) {
              __stcg(p.before + unit, last);
              last = unit;
            } else {
              unit = __ldcg(p.before + unit);
            }
          }
        }
      } while (another(pass++));
    }
  }
  __syncwarp();
  __syncthreads();
  if (warp == kSoftWarps) {
    tmem_relinquish();
    tmem_dealloc(tmem, 512);
  }
}

// ------------------------------------------------------------------ host

// Tensor maps of bf16 with boxes of 64 dims: `n` dimensions, sizes, strides in elements (of all but
// the first) and boxes.
cudaError_t make_map(CUtensorMap* map, const void* base, int n, const int64_t* sizes,
                     const int64_t* strides, const int* boxes) {
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
  cuuint64_t size[4], stride[3];
  cuuint32_t box[4], steps[4] = {1, 1, 1, 1};
  for (int i = 0; i < n; ++i) {
    size[i] = (cuuint64_t)sizes[i];
    box[i] = (cuuint32_t)boxes[i];
    if (i > 0) stride[i - 1] = (cuuint64_t)(2 * strides[i - 1]);
  }
  const CUresult r = encode(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, n, const_cast<void*>(base), size,
                            stride, box, steps, CU_TENSOR_MAP_INTERLEAVE_NONE,
                            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  return r == CUDA_SUCCESS ? cudaSuccess : cudaErrorInvalidValue;
}
// Rows of q: boxes of `box_heads` heads of `box_rows` rows.
cudaError_t query_map(CUtensorMap* map, const void* base, int dims, int heads, int rows,
                      int64_t head_stride, int64_t row_stride, int box_heads, int box_rows) {
  const int64_t sizes[3] = {dims, heads, rows}, strides[2] = {head_stride, row_stride};
  const int boxes[3] = {64, box_heads, box_rows};
  return make_map(map, base, 3, sizes, strides, boxes);
}
// Rows of k or v: boxes of `box_slices` slices of 64 dims, each of `box_rows` rows of one head.
cudaError_t key_map(CUtensorMap* map, const void* base, int dims, int heads, int rows,
                    int64_t head_stride, int64_t row_stride, int box_slices, int box_rows) {
  const int64_t sizes[4] = {64, rows, dims / 64, heads}, strides[3] = {row_stride, 64, head_stride};
  const int boxes[4] = {64, box_rows, box_slices, 1};
  return make_map(map, base, 4, sizes, strides, boxes);
}

// How a K/V head's group is laid over the rows of a tile.
struct PromptPlan {
  int set_heads, sets, tile_tokens;
  int64_t max_items;
};
PromptPlan prompt_plan(int rows, int batch, int group) {
  PromptPlan x;
  x.sets = (group + kRows - 1) / kRows;
  x.set_heads = (group + x.sets - 1) / x.sets;  // evenly
  x.tile_tokens = kRows / x.set_heads;
  x.max_items = rows / (2 * x.tile_tokens) + (int64_t)std::min(batch, rows);
  return x;
}

template <int kDq, int kDv>
cudaError_t launch_shape(const dcp_prompt_dims& d, const PromptParams& p, const void* q,
                         const void* k, const void* v, int grid, cudaStream_t stream) {
  using T = Shape<kDq, kDv>;
  CUtensorMap maps[3];
  cudaError_t e = query_map(&maps[0], q, kDq, d.num_heads, d.rows, d.q_head, d.q_row, p.set_heads,
                            p.tile_tokens);
  // without keys nothing is fetched, but a map has to stand over something
  const int keys = std::max(1, d.keys);
  if (e == cudaSuccess)
    e = key_map(&maps[1], k, kDq, d.kv_heads, keys, d.k_head, d.k_row, T::kKSlices, kTok);
  if (e == cudaSuccess)
    e = key_map(&maps[2], v, kDv, d.kv_heads, keys, d.v_head, d.v_row, kDv / 64, T::kVTok);
  if (e != cudaSuccess) return e;
  static bool ready[64] = {};
  int dev = 0;
  e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
  constexpr int smem = Shape<kDq, kDv>::kSmem;
  if (!ready[dev]) {
    e = cudaFuncSetAttribute(prompt_kernel<kDq, kDv>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             smem);
    if (e != cudaSuccess) return e;
    ready[dev] = true;
  }
  return launch_overlapping(true, prompt_kernel<kDq, kDv>, dim3(grid), dim3(kThreads), smem, stream,
                            p, maps[0], maps[1], maps[2]);
}

}  // namespace

int prompt_max_sequences() { return kMaxSeqs; }

namespace {

int prompt_sms() {
  static int cached[64] = {};
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return kSms;
  if (cached[dev] == 0) {
    if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return kSms;
    cached[dev] = std::min(n, kMaxCtas);
  }
  return cached[dev];
}

// Header, starts and arrivals of up to kMaxCtas CTAs, items, units, then the pieces' (O, m, l).
struct PromptWorkspace {
  size_t starts, arrived, ticket, items, before, parts, total;
};
PromptWorkspace prompt_workspace(int64_t max_items, int64_t per, int ctas, int v_dim) {
  PromptWorkspace x;
  x.starts = sizeof(Header);
  x.arrived = x.starts + kMaxCtas * sizeof(Start);
  x.ticket = x.arrived + kMaxCtas * kSoftWarps * sizeof(int);
  x.items = x.ticket + 16;
  x.before = x.items + (size_t)max_items * sizeof(Item);
  x.parts = x.before + ((size_t)(max_items * per) + 3) / 4 * 16;
  x.total = x.parts + (size_t)ctas * 4 * (v_dim + 2) * kRows * sizeof(float);
  return x;
}

}  // namespace

size_t prompt_workspace_bytes(int rows, int batch, int num_heads, int kv_heads, int v_dim) {
  const PromptPlan x = prompt_plan(rows, batch, num_heads / kv_heads);
  return prompt_workspace(x.max_items, (int64_t)x.sets * kv_heads, prompt_sms(), v_dim).total;
}

cudaError_t launch_prompt_attention(const dcp_prompt_dims& d, const int32_t* cu_q,
                                    const int32_t* cu_k, const void* q, const void* k,
                                    const void* v, float softmax_scale, void* out, float* lse,
                                    void* workspace, uint32_t* status, cudaStream_t stream) {
  const int group = d.num_heads / d.kv_heads;
  const PromptPlan x = prompt_plan(d.rows, d.batch, group);
  const int64_t units = x.max_items * x.sets * d.kv_heads;
  if (units > INT32_MAX - 2 * 1024) return cudaErrorInvalidConfiguration;
  // Each unit has a tile for every kTok keys at most.
  const int grid = (int)std::min<int64_t>(prompt_sms(), units * (d.keys / kTok + 1));
  const PromptWorkspace space =
      prompt_workspace(x.max_items, (int64_t)x.sets * d.kv_heads, prompt_sms(), d.v_dim);
  uint8_t* const at = static_cast<uint8_t*>(workspace);
  Header* header = reinterpret_cast<Header*>(at);
  Start* starts = reinterpret_cast<Start*>(at + space.starts);
  int* arrived = reinterpret_cast<int*>(at + space.arrived);
  Item* items = reinterpret_cast<Item*>(at + space.items);
  PromptParams p;
  p.header = header;
  p.starts = starts;
  p.items = items;
  p.arrived = arrived;
  p.ticket = reinterpret_cast<int*>(at + space.ticket);
  p.before = reinterpret_cast<int*>(at + space.before);
  p.parts = reinterpret_cast<float*>(at + space.parts);
  p.out = static_cast<uint16_t*>(out);
  p.lse = lse;
  p.status = status;
  p.scale = softmax_scale * kLog2e;
  p.heads = d.num_heads;
  p.group = group;
  p.causal = d.causal;
  p.set_heads = x.set_heads;
  p.sets = x.sets;
  p.tile_tokens = x.tile_tokens;
  p.set_div = FastDiv::by(x.set_heads);
  prompt_items_kernel<<<1, kItemThreads, 0, stream>>>(
      d.batch, d.rows, d.keys, d.causal, x.tile_tokens, (int)x.max_items, x.sets * d.kv_heads, grid,
      cu_q, cu_k, header, starts, items, arrived, p.ticket, status);
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  if (d.qk_dim == 64) return launch_shape<64, 64>(d, p, q, k, v, grid, stream);
  if (d.qk_dim == 128) return launch_shape<128, 128>(d, p, q, k, v, grid, stream);
  return launch_shape<192, 128>(d, p, q, k, v, grid, stream);
}

}  // namespace dcpmla
