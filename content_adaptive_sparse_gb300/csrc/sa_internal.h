// Declarations shared by the translation units of libsa.so (not part of the ABI).
#pragma once
#include <cuda_runtime.h>
#include <stdint.h>

#include "sa_api.h"

namespace sa {

// Device error bits (one error word per translation unit that can raise them).
constexpr unsigned int kErrTimeout = 1u;     // a bounded wait expired
constexpr unsigned int kErrBadIndex = 2u;    // CSR column index out of range (skipped)
constexpr unsigned int kErrCapacity = 4u;    // a device-sized output did not fit its buffer

constexpr int kMaxMaskBlocks = 4096;         // nb limit of the mask builder
constexpr int kMaxRandomBlocks = 64;

// Streaming multiprocessors of the current device (queried per call: a process may drive
// several devices).
inline int current_sm_count() {
  int dev = 0, n = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
      n <= 0)
    n = 1;
  return n;
}

// mask_build.cu
int launch_build_mask(const sa_mask_params& p, const float* d_ratio, int32_t* d_row_ptr, int32_t* d_col_idx,
                      cudaStream_t stream);

// attn_fwd.cu
constexpr int kMaxMasks = 8;       // CSRs per call (head groups)
constexpr int kMaxHeadMap = 256;   // heads with a per-head CSR choice
struct AttnArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int64_t q_strides[3];
  int64_t kv_strides[3];
  int64_t o_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, block, causal, csr_shared;
  int32_t n_masks;
  const int32_t* row_ptr[kMaxMasks];
  const int32_t* col_idx[kMaxMasks];
  uint8_t head_mask[kMaxHeadMap];    // query head -> CSR
  float softmax_scale;
  void* workspace;                   // caller-owned, 256-byte aligned
  size_t workspace_bytes;
};
int launch_attn_fwd(const AttnArgs& a, cudaStream_t stream);
// Workspace bytes of the forward with room for kFwdDefaultSlots split parts (split-row combine).
constexpr int kFwdDefaultSlots = 608;
size_t attn_fwd_workspace_bytes(int64_t batch, int64_t n_tokens, int64_t heads, int head_dim, int64_t csr_batches,
                                int64_t n_masks);
unsigned int attn_read_and_clear_error(cudaStream_t stream);

// offset_attn.cu
constexpr int kMaxOffsets = 64;
constexpr int kMaxWindow = 64;
struct OffsetArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int64_t q_strides[3];
  int64_t kv_strides[3];
  int64_t o_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, window, n_offsets;
  int32_t offsets[kMaxOffsets];
  float softmax_scale;
};
int launch_offset_attn_fwd(const OffsetArgs& a, cudaStream_t stream);
unsigned int offset_read_and_clear_error(cudaStream_t stream);

// offset_interp.cu
constexpr int kMaxInterpRungs = 64;
struct InterpArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;
  float* lse;
  int64_t q_strides[3];
  int64_t kv_strides[3];
  int64_t o_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, window, n_rungs;
  int32_t lo[kMaxInterpRungs];   // floor of the rung distance
  float t[kMaxInterpRungs];      // weight of the farther row
  float softmax_scale;
};
int launch_offset_interp_fwd(const InterpArgs& a, cudaStream_t stream);
unsigned int interp_read_and_clear_error(cudaStream_t stream);

// attn_bwd.cu
struct BwdArgs {
  const void* q;
  const void* k;
  const void* v;
  const void* o;
  const void* d_o;
  const float* lse;
  void* dq;
  void* dk;
  void* dv;
  int64_t q_strides[3];    // q and dq
  int64_t kv_strides[3];   // k, v, dk and dv
  int64_t o_strides[3];    // o and d_o
  int32_t batch, n_tokens, heads, kv_heads, head_dim, block, causal, csr_shared;
  int32_t n_masks;                       // CSRs (head groups); query head h uses head_mask[h]
  const int32_t* row_ptr[kMaxMasks];
  const int32_t* col_idx[kMaxMasks];
  int64_t col_capacity[kMaxMasks];       // entries each CSR may hold (n_masks > 1)
  uint8_t head_mask[kMaxHeadMap];
  float softmax_scale;
  void* workspace;
  size_t workspace_bytes;
};
// Workspace layout of the backward: D = rowsum(dO * O) fp32 [batch][heads][n_tokens],
// the transposed CSRs' col_ptr int32 [n_masks][csr_batches][nb + 1] (csr_batches below counts
// all masks) and row_idx int32 [rest], mask m's entries after those of masks < m.
struct BwdWorkspace {
  size_t dvec_off, col_ptr_off, row_idx_off, bytes;
  int64_t row_idx_capacity;
};
BwdWorkspace bwd_workspace_layout(int64_t batch, int64_t n_tokens, int64_t heads, int64_t block,
                                  int64_t csr_batches, int64_t col_capacity);
int launch_attn_bwd(const BwdArgs& a, cudaStream_t stream);
// Device address of the library's own backward scratch (kBwdStaticScratchBytes, 256-byte
// aligned), used by sa_attn_bwd_noalloc.
constexpr size_t kBwdStaticScratchBytes = size_t(16) << 20;
int bwd_static_scratch(void** ptr);
unsigned int bwd_read_and_clear_error(cudaStream_t stream);

// norm_rope.cu
constexpr int kNormRopeMaxCtas = 2048;   // CTAs of a launch at most (partial weight gradients)
constexpr int kMaxAxes = 8;
struct NormRopeArgs {
  bool backward;
  const void* q;
  const void* k;
  const void* d_q_out;                   // backward
  const void* d_k_out;
  void* q_out;                           // forward: outputs; backward: dq, dk
  void* k_out;
  int64_t q_strides[3], k_strides[3], dy_q_strides[3], dy_k_strides[3], q_out_strides[3], k_out_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, rotary_dim, interleaved;
  const float* q_weight;                 // [head_dim] or null
  const float* k_weight;
  float eps;
  const double* h_inv_freq;              // host, [rotary_dim / 2]
  int32_t n_axes;                        // 0: one position per token
  const int32_t* h_pair_axis;            // host, [rotary_dim / 2], where n_axes > 0
  const int32_t* positions;              // [batch][n_tokens] or null; n_axes > 0: [batch][n_tokens][n_axes]
  float* dq_weight;                      // backward, [head_dim] or null
  float* dk_weight;
  void* workspace;                       // backward: [kNormRopeMaxCtas][2][head_dim] floats
};
int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream);

// sink_attn.cu, sink_bwd.cu
constexpr int kMaxSinks = 128;           // one 128-row key tile
struct SinkArgs {
  const void* q;
  const void* k;
  const void* v;
  void* o;                               // written by the forward, read by the backward
  float* lse;
  const void* d_o;
  void* dq;
  void* dk;
  void* dv;
  int64_t q_strides[3], k_strides[3], v_strides[3], o_strides[3], do_strides[3];
  int64_t dq_strides[3], dk_strides[3], dv_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, window, sinks;
  float softmax_scale;
  void* workspace;
  size_t workspace_bytes;
};
int launch_sink_attn_fwd(const SinkArgs& a, cudaStream_t stream);
unsigned int sink_fwd_read_and_clear_error(cudaStream_t stream);
// Workspace of the backward: -LSE log2(e) and D, fp32 [batch][heads][n_tokens rounded up to 128],
// then the partial sums of the sinks' dK and dV.
struct SinkBwdWorkspace {
  size_t nl2_off, dvec_off, partial_off, bytes;
};
SinkBwdWorkspace sink_bwd_workspace_layout(int64_t batch, int64_t n_tokens, int64_t heads, int64_t kv_heads, int64_t d,
                                           int window, int sinks);
int launch_sink_attn_bwd(const SinkArgs& a, cudaStream_t stream);
unsigned int sink_bwd_read_and_clear_error(cudaStream_t stream);

// sink_decode.cu
struct SinkDecodeArgs {
  const void* q;
  const void* k;                         // bf16 rows, or codes
  const void* v;
  const void* k_scales;                  // 4-bit cache
  const void* v_scales;
  void* o;
  float* lse;
  const int32_t* lengths;
  int64_t q_strides[3], k_strides[3], v_strides[3], o_strides[3];
  int32_t batch, capacity, heads, kv_heads, head_dim, window, sinks;
  bool cache4;
  float softmax_scale;
  int32_t n_parts, part_tiles;           // n_parts > 0: join these partial results of a shared prefix
  const void* part_o;
  const void* part_ml;
  float* scores;                         // not null: add up the rows' weights (workspace of scored_bytes)
  const float* weights_in;
  float* weights_out;
  float decay;
};
// Floats of a row's scores of up to 16 query heads: a power of two.
inline int scored_stride(int heads, int kv_heads) {
  const int group = heads / kv_heads < 16 ? heads / kv_heads : 16;
  int n = 1;
  while (n < group) n *= 2;
  return n;
}
constexpr int kMaxScoredHeads = 128;     // query heads of a key head
int launch_sink_decode(const SinkDecodeArgs& a, cudaStream_t stream);
unsigned int decode_read_and_clear_error(cudaStream_t stream);

// prefix_attn.cu
struct PrefixArgs {
  const void* q;
  const void* k_prefix;
  const void* v_prefix;
  const void* k;                         // own tokens (decode: left to sink_decode.cu)
  const void* v;
  void* o;
  float* lse;
  int64_t q_strides[3], k_prefix_strides[3], v_prefix_strides[3], k_strides[3], v_strides[3], o_strides[3];
  int32_t batch, n_tokens, prefix, heads, kv_heads, head_dim, window;
  bool decode;                           // write the prefix's partial results alone
  float softmax_scale;
  void* workspace;
};
// Workspace: maxima and sums of the partial results, then their O. Decoding: `parts` partial results of every row
// s * group + e of a key head, in blocks (hk * tiles + row / 128) * parts + part (prefix_attn.cu has their layout).
struct PrefixWorkspace {
  int parts, tiles;
  size_t part_o_off, bytes;
};
PrefixWorkspace prefix_workspace(int batch, int n_tokens, int prefix, int heads, int kv_heads, int head_dim, int window,
                                 bool decode);
int launch_prefix_attn(const PrefixArgs& a, cudaStream_t stream);
unsigned int prefix_read_and_clear_error(cudaStream_t stream);

// scored_cache.cu
constexpr int kMaxScoredCapacity = 1 << 20;
struct ScoredArgs {
  const void* k;                         // append: new rows
  const void* v;
  void* k_cache;
  void* v_cache;
  int64_t k_strides[3], v_strides[3], k_cache_strides[3], v_cache_strides[3];
  int32_t batch, n_tokens, kv_heads, head_dim, capacity;
  const int32_t* start;                  // append
  const int32_t* tokens;
  int32_t keep, sinks, recent;           // evict
  const float* weights_in;
  const int32_t* positions_in;
  const int32_t* lengths_in;
  float* weights_out;
  int32_t* positions_out;
  int32_t* lengths_out;
};
int launch_scored_append(const ScoredArgs& a, cudaStream_t stream);
int launch_scored_evict(const ScoredArgs& a, cudaStream_t stream);
unsigned int scored_read_and_clear_error(cudaStream_t stream);

// sink_weights.cu
struct WeightsArgs {
  const void* q;
  const void* k;
  const float* lse;
  int64_t q_strides[3], k_strides[3];
  int32_t batch, n_tokens, heads, kv_heads, head_dim, window, sinks, first_query;
  float softmax_scale;
  float* weights;
  void* workspace;
};
constexpr int kWeightsMaxCtas = 256;     // CTAs of a launch at most
constexpr size_t kWeightsWorkspace = (size_t)kWeightsMaxCtas * 2 * 256 * sizeof(float);
int launch_sink_attn_weights(const WeightsArgs& a, cudaStream_t stream);
unsigned int weights_read_and_clear_error(cudaStream_t stream);

// sink_cache4.cu
struct Cache4Args {
  bool read;
  void* k;                               // rows, [batch][n_tokens][kv_heads][head_dim]
  void* v;
  uint8_t* k_codes;
  void* k_scales;
  uint8_t* v_codes;
  void* v_scales;
  const int32_t* start;
  int64_t k_strides[3], v_strides[3];
  int32_t batch, n_tokens, kv_heads, head_dim, capacity;
};
int launch_cache4(const Cache4Args& a, cudaStream_t stream);
unsigned int cache4_read_and_clear_error(cudaStream_t stream);

}  // namespace sa
