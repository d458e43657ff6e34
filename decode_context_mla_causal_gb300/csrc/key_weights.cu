// The attention weight that each cached latent row receives from a verify step, added to
// what earlier steps left.
//
// For local token t of (rank, sequence), with the step's merged LSE of every row (j, head),
//   w'_t = [t < n_old] decay * w_t + sum over rows with t < n_row of
//          2^(softmax_scale * kv_scale * log2(e) * (q . k_t) - log2(e) * LSE_row).
// A token's sum needs that token's row and the queries alone, so no token's result
// depends on how the tokens are spread over the machine.
#include <cuda_bf16.h>
#include <cuda_fp8.h>

#include <algorithm>

#include "common.cuh"

namespace dcpmla {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kTokens = 64;  // per CTA
constexpr int kWarps = 8;
constexpr int kE = kDqk / 32;

struct KeyWeightParams {
  const int32_t* seq_lens;
  const int32_t* block_table;
  const uint16_t* q;
  const uint8_t* kv;
  const float* kv_scale;
  const float* lse;
  const float* w_in;
  float* w_out;
  uint32_t* status;
  float softmax_scale, decay;
  int batch, qlen, H, dcp, interleave, block_size, max_blocks, max_local_len, num_blocks, causal,
      rank_begin;
};

// One warp per token, a lane holding every 32nd dim of its row.
template <bool kFp8>
__global__ void __launch_bounds__(32 * kWarps) key_weights_kernel(const KeyWeightParams p) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int b = blockIdx.y, k = blockIdx.z, rank = p.rank_begin + k;
  const int64_t L = p.seq_lens[b], span = (int64_t)p.dcp * p.interleave;
  uint32_t bad = (L < 0 || (p.causal && L < p.qlen)) ? DCP_STATUS_BAD_SEQ_LEN : 0u;
  int64_t n = local_len(L, rank, span, p.interleave);
  if (n > p.max_local_len) {
    bad |= DCP_STATUS_LOCAL_OVER_BOUND;
    n = p.max_local_len;
  }
  const int64_t old = local_len(L - p.qlen, rank, span, p.interleave);
  const float scale = p.softmax_scale * (p.kv_scale ? *p.kv_scale : 1.0f) * kLog2e;
  for (int i = warp; i < kTokens; i += kWarps) {
    const int t = blockIdx.x * kTokens + i;
    if (t >= n) break;
    const int blk = p.block_table[(int64_t)b * p.max_blocks + t / p.block_size];
    if (blk < 0 || blk >= p.num_blocks) {
      bad |= DCP_STATUS_BAD_BLOCK_ID;
      continue;
    }
    const int64_t at =
        (((int64_t)k * p.num_blocks + blk) * p.block_size + t % p.block_size) * kDqk;
    float key[kE];
#pragma unroll
    for (int e = 0; e < kE; ++e) {
      if (kFp8) {
        __nv_fp8_e4m3 x;
        x.__x = p.kv[at + 32 * e + lane];
        key[e] = float(x);
      } else {
        key[e] = __uint_as_float(
            (uint32_t)reinterpret_cast<const uint16_t*>(p.kv)[at + 32 * e + lane] << 16);
      }
    }
    float w = 0.f;
    for (int j = 0; j < p.qlen; ++j) {
      int64_t seen =
          local_len(p.causal ? L - p.qlen + 1 + j : L, rank, span, p.interleave);
      if (t >= seen) continue;
      for (int h = 0; h < p.H; ++h) {
        const int64_t row = ((int64_t)b * p.qlen + j) * p.H + h;
        float x = 0.f;
#pragma unroll
        for (int e = 0; e < kE; ++e)
          x = fmaf(key[e], __uint_as_float((uint32_t)p.q[row * kDqk + 32 * e + lane] << 16), x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        const float lse = p.lse[row];
        if (lse != -INFINITY) w += exp2f(fmaf(x, scale, -lse * kLog2e));
      }
    }
    if (lane == 0) {
      const int64_t out = ((int64_t)k * p.batch + b) * p.max_local_len + t;
      p.w_out[out] = t < old ? fmaf(p.decay, p.w_in[out], w) : w;
    }
  }
  if (lane == 0 && bad) raise_status(p.status, bad);
}

}  // namespace

size_t key_weights_workspace_bytes(const dcp_mla_dims& d, int num_ranks) {
  (void)d;
  (void)num_ranks;
  return 16;
}

cudaError_t launch_key_weights(const dcp_mla_dims& d, const Derived& x, const int32_t* seq_lens,
                               const int32_t* block_table, const void* q, const void* kv,
                               dcp_kv_dtype kv_dtype, const float* kv_scale, float softmax_scale,
                               const float* lse, float decay, int rank_begin, int num_ranks,
                               const float* weights_in, float* weights_out, void* workspace,
                               uint32_t* status, cudaStream_t stream) {
  (void)x;
  (void)workspace;
  KeyWeightParams p;
  p.seq_lens = seq_lens;
  p.block_table = block_table;
  p.q = static_cast<const uint16_t*>(q);
  p.kv = static_cast<const uint8_t*>(kv);
  p.kv_scale = kv_scale;
  p.lse = lse;
  p.w_in = weights_in;
  p.w_out = weights_out;
  p.status = status;
  p.softmax_scale = softmax_scale;
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
  const dim3 grid((unsigned)((d.max_local_len + kTokens - 1) / kTokens), (unsigned)d.batch,
                  (unsigned)num_ranks);
  auto kern = kv_dtype == DCP_KV_FP8_E4M3 ? key_weights_kernel<true> : key_weights_kernel<false>;
  kern<<<grid, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace dcpmla
