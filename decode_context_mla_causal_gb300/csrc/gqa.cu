// Grouped-head K/V caches: the new tokens' rows into the pools, and the attention of the
// newest tokens over them, split over the cache's length and joined.
//
// For query head h of row (b, j) with K/V head g = h / group, over the tokens t that the
// row sees on the call's ranks,
//   s_t = softmax_scale * k_scale * log2(e) * (q . k_t)          (base 2)
//   O = v_scale * sum_t 2^(s_t - m) v_t / sum_t 2^(s_t - m),  LSE = (m + log2 sum) ln 2,
// with a running maximum m. A rank's tokens of a sequence are cut into pieces whose
// (O, m, l) are joined in rank and piece order, so the result does not depend on which
// piece ends first.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"
#include "fp8.cuh"

namespace dcpmla {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float load_elem(const uint8_t* p, int64_t i, bool fp8) {
  if (fp8) {
    __nv_fp8_e4m3 x;
    x.__x = p[i];
    return float(x);
  }
  return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << 16);
}

// ------------------------------------------------------------------ write

constexpr int kWriteThreads = 128;

// One 8-element piece of a K or V row per thread; the rows of a rank in grid.y.
template <bool kFp8>
__global__ void __launch_bounds__(kWriteThreads)
gqa_write_kernel(int rows, int row_elems, int64_t pool_rows,
                 const int32_t* __restrict__ slot_mapping, const uint16_t* __restrict__ k_new,
                 const uint16_t* __restrict__ v_new, const float* k_scale, const float* v_scale,
                 uint8_t* k_pool, uint8_t* v_pool, uint32_t* status) {
  const int k = blockIdx.y;
  const int per = row_elems / 8;
  const int64_t i = (int64_t)blockIdx.x * kWriteThreads + threadIdx.x;
  if (i >= (int64_t)rows * per) return;
  const int row = (int)(i / per), c = (int)(i % per);
  const int32_t slot = slot_mapping[(int64_t)k * rows + row];
  if (slot < 0 || slot >= pool_rows) {
    if (slot != -1 && c == 0) raise_status(status, DCP_STATUS_BAD_PAGE);
    return;
  }
  const int64_t src = (int64_t)row * row_elems + 8 * c;
  const int64_t dst = ((int64_t)k * pool_rows + slot) * row_elems + 8 * c;
  const uint4 xk = *reinterpret_cast<const uint4*>(k_new + src);
  const uint4 xv = *reinterpret_cast<const uint4*>(v_new + src);
  if (kFp8) {
    *reinterpret_cast<uint2*>(k_pool + dst) = quantize8(xk, k_scale ? *k_scale : 1.0f);
    *reinterpret_cast<uint2*>(v_pool + dst) = quantize8(xv, v_scale ? *v_scale : 1.0f);
  } else {
    *reinterpret_cast<uint4*>(k_pool + 2 * dst) = xk;
    *reinterpret_cast<uint4*>(v_pool + 2 * dst) = xv;
  }
}

// ------------------------------------------------------------------ decode

struct GqaParams {
  const int32_t* seq_lens;
  const int32_t* block_table;
  const uint16_t* q;
  const uint8_t* k_pool;
  const uint8_t* v_pool;
  const float* k_scale;
  const float* v_scale;
  float* part_o;  // [nr][NS][R][H][D]
  float* part_m;  // [nr][NS][R][H]
  float* part_l;
  uint32_t* status;
  float softmax_scale;
  int batch, qlen, H, kv_heads, dcp, interleave, block_size, max_blocks, max_local_len,
      num_blocks, num_splits, causal, rank_begin, num_ranks;
};

// One warp per (rank, piece, row, query head); a lane holds kD / 32 dims.
template <int kD, bool kFp8>
__global__ void __launch_bounds__(128) gqa_partial_kernel(const GqaParams p) {
  constexpr int kE = kD / 32;
  const int lane = threadIdx.x & 31;
  const int R = p.batch * p.qlen;
  const int64_t rh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (rh >= (int64_t)R * p.H) return;
  const int s = blockIdx.y % p.num_splits, k = blockIdx.y / p.num_splits;
  const int row = (int)(rh / p.H), h = (int)(rh % p.H);
  const int b = row / p.qlen, j = row % p.qlen;
  const int g = h / (p.H / p.kv_heads);
  const int rank = p.rank_begin + k;
  const int64_t L = p.seq_lens[b], span = (int64_t)p.dcp * p.interleave;
  int64_t n = local_len(p.causal ? L - p.qlen + 1 + j : L, rank, span, p.interleave);
  uint32_t bad = (L < 0 || (p.causal && L < p.qlen)) ? DCP_STATUS_BAD_SEQ_LEN : 0u;
  if (n > p.max_local_len) {
    bad |= DCP_STATUS_LOCAL_OVER_BOUND;
    n = p.max_local_len;
  }
  const int beg = (int)(n * s / p.num_splits), end = (int)(n * (s + 1) / p.num_splits);
  const float scale = p.softmax_scale * (p.k_scale ? *p.k_scale : 1.0f) * kLog2e;
  float q[kE], acc[kE];
#pragma unroll
  for (int e = 0; e < kE; ++e) {
    q[e] = __uint_as_float((uint32_t)p.q[rh * kD + lane * kE + e] << 16);
    acc[e] = 0.f;
  }
  float m = -INFINITY, l = 0.f;
  for (int t = beg; t < end; ++t) {
    const int blk = p.block_table[(int64_t)b * p.max_blocks + t / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      bad |= DCP_STATUS_BAD_BLOCK_ID;
      continue;
    }
    const int64_t at = ((((int64_t)k * p.num_blocks + blk) * p.block_size + t % p.block_size) *
                            p.kv_heads + g) * kD + lane * kE;
    float x = 0.f;
#pragma unroll
    for (int e = 0; e < kE; ++e) x = fmaf(q[e], load_elem(p.k_pool, at + e, kFp8), x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
    x *= scale;
    const float mn = fmaxf(m, x);
    const float a = exp2f(m - mn), w = exp2f(x - mn);
    m = mn;
    l = l * a + w;
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = fmaf(acc[e], a, w * load_elem(p.v_pool, at + e, kFp8));
  }
  const int64_t at = ((int64_t)k * p.num_splits + s) * R * p.H + rh;
#pragma unroll
  for (int e = 0; e < kE; ++e) p.part_o[at * kD + lane * kE + e] = acc[e];
  if (lane == 0) {
    p.part_m[at] = m;
    p.part_l[at] = l;
    if (bad) raise_status(p.status, bad);
  }
}

// One warp per (row, head) joins the pieces of all ranks in order.
template <int kD>
__global__ void __launch_bounds__(128)
gqa_join_kernel(int64_t rows_heads, int pieces, const float* v_scale,
                const float* __restrict__ part_o, const float* __restrict__ part_m,
                const float* __restrict__ part_l, __nv_bfloat16* __restrict__ out,
                float* __restrict__ lse) {
  constexpr int kE = kD / 32;
  const int lane = threadIdx.x & 31;
  const int64_t rh = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  if (rh >= rows_heads) return;
  float m = -INFINITY, l = 0.f, acc[kE] = {};
  for (int i = 0; i < pieces; ++i) m = fmaxf(m, part_m[i * rows_heads + rh]);
  for (int i = 0; i < pieces; ++i) {
    const int64_t at = i * rows_heads + rh;
    if (part_m[at] == -INFINITY) continue;
    const float w = exp2f(part_m[at] - m);
    l = fmaf(w, part_l[at], l);
#pragma unroll
    for (int e = 0; e < kE; ++e) acc[e] = fmaf(w, part_o[at * kD + lane * kE + e], acc[e]);
  }
  const float inv = l > 0.f ? (v_scale ? *v_scale : 1.0f) / l : 0.f;
#pragma unroll
  for (int e = 0; e < kE; ++e) out[rh * kD + lane * kE + e] = __float2bfloat16_rn(acc[e] * inv);
  if (lane == 0) lse[rh] = l > 0.f ? (m + log2f(l)) * kLn2 : -INFINITY;
}

}  // namespace

cudaError_t launch_gqa_kv_write(const dcp_mla_dims& d, int row_elems, const int32_t* slot_mapping,
                                const void* k_new, const void* v_new, dcp_kv_dtype kv_dtype,
                                const float* k_scale, const float* v_scale, int num_ranks,
                                void* k_pool, void* v_pool, uint32_t* status,
                                cudaStream_t stream) {
  const int rows = d.batch * d.qlen;
  const int64_t n = (int64_t)rows * (row_elems / 8);
  const dim3 grid((unsigned)((n + kWriteThreads - 1) / kWriteThreads), (unsigned)num_ranks);
  auto kern = kv_dtype == DCP_KV_FP8_E4M3 ? gqa_write_kernel<true> : gqa_write_kernel<false>;
  kern<<<grid, kWriteThreads, 0, stream>>>(
      rows, row_elems, (int64_t)d.num_blocks * d.block_size, slot_mapping,
      static_cast<const uint16_t*>(k_new), static_cast<const uint16_t*>(v_new), k_scale, v_scale,
      static_cast<uint8_t*>(k_pool), static_cast<uint8_t*>(v_pool), status);
  return cudaGetLastError();
}

static size_t gqa_parts(const dcp_mla_dims& d, int num_ranks) {
  return (size_t)num_ranks * d.num_splits * d.batch * d.qlen * d.num_heads;
}

size_t gqa_workspace_bytes(const dcp_mla_dims& d, int kv_heads, int head_dim, int num_ranks) {
  (void)kv_heads;
  return (gqa_parts(d, num_ranks) * (head_dim + 2) * sizeof(float) + 15) / 16 * 16;
}

cudaError_t launch_gqa_decode(const dcp_mla_dims& d, int kv_heads, int head_dim,
                              const int32_t* seq_lens, const int32_t* block_table, const void* q,
                              const void* k_pool, const void* v_pool, dcp_kv_dtype kv_dtype,
                              const float* k_scale, const float* v_scale, float softmax_scale,
                              int rank_begin, int num_ranks, void* out, float* lse,
                              void* workspace, uint32_t* status, cudaStream_t stream) {
  const size_t parts = gqa_parts(d, num_ranks);
  GqaParams p;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.q = static_cast<const uint16_t*>(q);
  p.k_pool = static_cast<const uint8_t*>(k_pool);
  p.v_pool = static_cast<const uint8_t*>(v_pool);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.part_o = static_cast<float*>(workspace);
  p.part_m = p.part_o + parts * head_dim;
  p.part_l = p.part_m + parts;
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
  p.num_splits = d.num_splits;
  p.causal = d.causal;
  p.rank_begin = rank_begin;
  p.num_ranks = num_ranks;
  const int64_t rows_heads = (int64_t)d.batch * d.qlen * d.num_heads;
  const dim3 grid((unsigned)((rows_heads + 3) / 4), (unsigned)(num_ranks * d.num_splits));
  const bool fp8 = kv_dtype == DCP_KV_FP8_E4M3;
  auto partial = head_dim == 64 ? (fp8 ? gqa_partial_kernel<64, true> : gqa_partial_kernel<64, false>)
                                : (fp8 ? gqa_partial_kernel<128, true>
                                       : gqa_partial_kernel<128, false>);
  partial<<<grid, 128, 0, stream>>>(p);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  auto join = head_dim == 64 ? gqa_join_kernel<64> : gqa_join_kernel<128>;
  join<<<grid.x, 128, 0, stream>>>(rows_heads, num_ranks * d.num_splits, v_scale, p.part_o,
                                   p.part_m, p.part_l, static_cast<__nv_bfloat16*>(out), lse);
  return cudaGetLastError();
}

}  // namespace dcpmla
