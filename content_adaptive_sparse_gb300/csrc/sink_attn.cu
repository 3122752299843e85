// Causal attention over a token window and a few first tokens ("sinks"), forward: key j is
// visible to query i iff j <= i and (i - j <= window or j < sinks). The kernels are those of the
// block-sparse forward (attn_fwd_pipes.cuh at d = 32 and 64, attn_fwd_wide.cuh at d = 128) on the
// sink-window graph: a 128-query tile's key list is the sinks' 32-key chunks and then the
// window's, so no CSR and no workspace are read, and an item's list is about as long as every
// other's, so items are dealt out in turn.
#include <string.h>

#include "attn_fwd_common.cuh"
#include "attn_fwd_pipes.cuh"
#include "attn_fwd_wide.cuh"

namespace sa {
namespace {

template <int D>
int launch_d(const SinkArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tq, tk, tv, to;
  if (!encode_bhnd_map(&tq, a.q, a.batch, a.n_tokens, a.heads, D, a.q_strides[0], a.q_strides[1], a.q_strides[2],
                       C::CH, kTile, C::TMA_SWZ) ||
      !encode_bhnd_map(&tk, a.k, a.batch, a.n_tokens, a.kv_heads, D, a.k_strides[0], a.k_strides[1], a.k_strides[2],
                       C::CH, 32, C::TMA_SWZ) ||
      !encode_bhnd_map(&tv, a.v, a.batch, a.n_tokens, a.kv_heads, D, a.v_strides[0], a.v_strides[1], a.v_strides[2],
                       C::CH, 32, C::TMA_SWZ))
    return SA_ERR_UNSUPPORTED;
  Params p;
  memset(&p, 0, sizeof(p));
  p.batch = a.batch;
  p.n_tokens = a.n_tokens;
  p.heads = a.heads;
  p.heads_per_kv = a.heads / a.kv_heads;
  p.block = 32;                        // K / V boxes of one 32-key chunk
  p.log2b = 5;
  p.causal = 1;
  p.tiles_per_seq = (a.n_tokens + kTile - 1) / kTile;
  p.n_items = a.batch * a.heads * p.tiles_per_seq;
  p.n_masks = 1;
  p.o = static_cast<__nv_bfloat16*>(a.o);
  memset(&to, 0, sizeof(to));
  p.o_tma = D == 64 && encode_bhnd_map(&to, a.o, a.batch, a.n_tokens, a.heads, D, a.o_strides[0], a.o_strides[1],
                                       a.o_strides[2], C::CH, 32, C::TMA_SWZ)
                ? 1
                : 0;
  p.lse = a.lse;
  p.o_sb = a.o_strides[0];
  p.o_sn = a.o_strides[1];
  p.o_sh = a.o_strides[2];
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.window = a.window;
  p.sinks = a.sinks;
  const auto kern = [] {
    if constexpr (C::WIDE) return attn_fwd_wide_kernel<D, true>;
    else return attn_fwd_kernel<D, true>;
  }();
  // the kernels' register split hands out exactly the launch allocation
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SA_ERR_CUDA;
  if (fa.numRegs != kLaunchRegs) return SA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return SA_ERR_CUDA;
  const int per_cta = C::WIDE ? 1 : 2;
  const int sm_count = current_sm_count();
  const int need = (p.n_items + per_cta - 1) / per_cta;
  kern<<<need < sm_count ? need : sm_count, kThreads, C::SMEM, stream>>>(tq, tk, tv, to, p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

int launch_sink_attn_fwd(const SinkArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_d<32>(a, stream);
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int sink_fwd_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_attn_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
