// Shared definitions of the CUDA library (not shared with the CPU oracle).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/dcp_mla.h"

namespace dcpmla {

constexpr int kDqk = DCP_MLA_QK_DIM;  // 576
constexpr int kDv = DCP_MLA_V_DIM;    // 512

// Host-side derived sizes of a dims struct (validated by check_dims first).
struct Derived {
  int rows;       // R = batch * qlen
  int subpage;    // P
  int ppb;        // subpages per block
  int max_pages;  // MP
};

Derived derive(const dcp_mla_dims& d);

// Record a message for dcp_last_error() and return the status.
dcp_status fail(dcp_status s, const char* fmt, ...);

// Internal launchers (argument checks already done by the API layer).
cudaError_t launch_metadata(const dcp_mla_dims& d, const Derived& x, const int32_t* seq_lens,
                            const int32_t* block_table, int rank_begin, int num_ranks,
                            int32_t* row_len, int32_t* page_ids, int32_t* split_beg,
                            int32_t* split_end, uint32_t* status, cudaStream_t stream);

cudaError_t launch_partial(const dcp_mla_dims& d, const Derived& x, const void* q,
                           const void* kv, dcp_kv_dtype kv_dtype, const float* kv_scale,
                           float softmax_scale, int num_ranks, const int32_t* row_len,
                           const int32_t* page_ids, const int32_t* split_beg,
                           const int32_t* split_end, float* part_o, float* part_m,
                           float* part_l, void* workspace, uint32_t* status,
                           cudaStream_t stream, void* send = nullptr,
                           uint64_t hold_q_ns = 0);

// Device workspace launch_partial uses for the item order (bytes, 16-byte multiple).
size_t partial_workspace_bytes(const dcp_mla_dims& d, int num_ranks);

// Clusters of the partial kernel the current device runs at once (cached per
// device), or a negative value when the query fails.
int partial_concurrent_items();

// Wave balancing reads every (rank, sequence) pair's length in each metadata CTA.
constexpr int kBalanceMaxPairs = 1 << 16;

// Tiles of 64 tokens per work item, the unit of the split plan.
constexpr int kPlanTileTokens = 64;
// Wave balancing cuts no piece below this many tiles.
constexpr int kPlanMinPieceTiles = 8;

cudaError_t launch_merge(const dcp_mla_dims& d, const Derived& x, int num_ranks,
                         const float* part_o, const float* part_m, const float* part_l,
                         void* out, float* lse, float* rank_lse, uint32_t* status,
                         cudaStream_t stream);

cudaError_t launch_slot_mapping(const dcp_mla_dims& d, const int32_t* seq_lens,
                                const int32_t* block_table, int rank_begin, int num_ranks,
                                int32_t* slot_mapping, uint32_t* status, cudaStream_t stream);

cudaError_t launch_kv_write(const dcp_mla_dims& d, const int32_t* slot_mapping, const void* kv_new,
                            dcp_kv_dtype kv_dtype, const float* kv_scale, int num_ranks,
                            void* pool, uint32_t* status, cudaStream_t stream);

int64_t a2a_chunk_words(int R, int Hg, int P);

cudaError_t launch_a2a_pack(const dcp_mla_dims& d, const Derived& x, int num_ranks,
                            const float* part_o, const float* part_m, const float* part_l,
                            void* send, cudaStream_t stream);

cudaError_t launch_a2a_project(const dcp_mla_dims& d, const Derived& x, int num_ranks,
                               const void* send_in, const void* w_v, int payload, void* send,
                               uint32_t* status, cudaStream_t stream);

cudaError_t launch_a2a_combine(const dcp_mla_dims& d, const Derived& x, int payload,
                               const void* recv, int64_t src_stride, int64_t dst_stride,
                               int dst_begin, int num_dst, void* out, float* lse,
                               cudaStream_t stream);

cudaError_t launch_gqa_kv_write(const dcp_mla_dims& d, int row_elems, const int32_t* slot_mapping,
                                const void* k_new, const void* v_new, dcp_kv_dtype kv_dtype,
                                const float* k_scale, const float* v_scale, int num_ranks,
                                void* k_pool, void* v_pool, uint32_t* status,
                                cudaStream_t stream);

size_t gqa_workspace_bytes(const dcp_mla_dims& d, int kv_heads, int head_dim, int num_ranks);

cudaError_t launch_gqa_decode(const dcp_mla_dims& d, int kv_heads, int head_dim,
                              const int32_t* seq_lens, const int32_t* block_table, const void* q,
                              const void* k_pool, const void* v_pool, dcp_kv_dtype kv_dtype,
                              const float* k_scale, const float* v_scale, float softmax_scale,
                              int rank_begin, int num_ranks, void* out, float* lse,
                              void* workspace, uint32_t* status, cudaStream_t stream);

size_t key_weights_workspace_bytes(const dcp_mla_dims& d, int num_ranks);

cudaError_t launch_key_weights(const dcp_mla_dims& d, const int32_t* seq_lens,
                               const int32_t* block_table, const void* q, const void* kv,
                               dcp_kv_dtype kv_dtype, const float* kv_scale, float softmax_scale,
                               const float* lse, float decay, int rank_begin, int num_ranks,
                               const float* weights_in, float* weights_out, void* workspace,
                               uint32_t* status, cudaStream_t stream);

cudaError_t launch_evict_select(const dcp_mla_dims& d, const int32_t* seq_lens,
                                const float* weights, int budget, int sink, int recent,
                                int max_keep, int rank_begin, int num_ranks, int32_t* keep_idx,
                                int32_t* keep_count, int32_t* new_lens, uint32_t* status,
                                cudaStream_t stream);

cudaError_t launch_kv_compact(const dcp_mla_dims& d, int row_bytes, const int32_t* keep_idx,
                              const int32_t* keep_count, int max_keep, const int32_t* src_table,
                              const int32_t* dst_table, int num_ranks, void* pool,
                              const float* weights_in, float* weights_out, uint32_t* status,
                              cudaStream_t stream);

// Local length, on `rank`, of a sequence (or row boundary) of g global tokens ("Support
// Kimi-K3 DCP with DSpark", review thread), unclamped; span = dcp * interleave.
__host__ __device__ __forceinline__ int64_t local_len(int64_t g, int rank, int64_t span,
                                                      int interleave) {
  if (g <= 0) return 0;
  int64_t rem = g % span - (int64_t)rank * interleave;
  rem = rem < 0 ? 0 : (rem > interleave ? interleave : rem);
  return g / span * interleave + rem;
}

// Division of numbers below 2^31 by a divisor known on the host: a multiplication and a
// shift (the multiplier is 2^32 (2^s - d) / d + 1 rounded down, s = ceil(log2 d)).
struct FastDiv {
  uint32_t mul, shift, d;
  static FastDiv by(int32_t divisor) {
    FastDiv f;
    f.d = (uint32_t)divisor;
    f.shift = 0;
    while (((uint64_t)1 << f.shift) < f.d) ++f.shift;
    f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - f.d)) / f.d + 1);
    return f;
  }
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((uint32_t)n, mul) + (uint32_t)n) >> shift);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * (int)d; }
};

// Launch of a kernel that may begin while the one before it in the stream still runs (if
// `overlap`); such a kernel calls grid_dependency_wait() before it uses that one's results.
template <typename... Params, typename... Args>
cudaError_t launch_overlapping(bool overlap, void (*kern)(Params...), dim3 grid, dim3 block,
                               size_t smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = overlap ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kern, args...);
}

__device__ __forceinline__ void raise_status(uint32_t* status, uint32_t bits) {
  if (status != nullptr) atomicOr(status, bits);
}

}  // namespace dcpmla
