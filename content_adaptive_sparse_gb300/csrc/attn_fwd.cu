// Block-sparse flash-attention forward for sm_103a (tcgen05 + TMEM + TMA). Head dimensions
// 32 and 64 run the two-pipeline kernel of attn_fwd_pipes.cuh, head dimension 128 the one-stream
// kernel of attn_fwd_wide.cuh. Both take their work items, key tiles and TMA loads from
// attn_fwd_common.cuh, and share the split-row combine (K9) and the launch code below.
#include <string.h>

#include <atomic>

#include "attn_fwd_common.cuh"
#include "attn_fwd_pipes.cuh"
#include "attn_fwd_wide.cuh"

namespace sa {
namespace {

// ------------------------------------------------------------------ split-row combine (K9)
//
// Used when a launch has few work items for the GPU's item streams (see launch_d): a few long
// key lists would then leave SMs idle. fwd_plan_kernel counts the key tiles of every query tile's
// union (one warp per (mask, CSR sequence, query tile)), fwd_schedule_kernel (one CTA) cuts the
// items whose lists are longer than T tiles into parts of T tiles, each with a slot for its
// partial result, and lists the parts first, then the other items; attn_fwd_kernel runs the
// list; fwd_merge_kernel combines the parts of each split item:
//   LSE = ln sum_p exp(LSE_p),  O = sum_p exp(LSE_p - LSE) O_p.

struct SplitHdr {
  int list_len, n_split, part_tiles, n_split_items;
};

constexpr int kPlanWarps = 8;
constexpr int kMinPartTiles = 4;

__global__ void __launch_bounds__(32 * kPlanWarps) fwd_plan_kernel(const __grid_constant__ Params p, int n_groups,
                                                                    int* tiles) {
  __shared__ uint32_t bm[kPlanWarps][kMaxMaskBlocks / 32];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = blockIdx.x * kPlanWarps + warp;
  if (g >= n_groups) return;                         // the whole warp leaves
  const int t = g % p.tiles_per_seq;
  const int cs = (g / p.tiles_per_seq) % p.csr_batches;
  const int m = g / (p.tiles_per_seq * p.csr_batches);
  const int nb = p.nb, nw = (nb + 31) >> 5;
  const int32_t* rp = p.row_ptr[m] + (size_t)cs * (nb + 1);
  const int32_t* ci = p.col_idx[m];
  const int I0 = (t * kTile) >> p.log2b;
  const int nq = min(kTile >> p.log2b, nb - I0);
  for (int w = lane; w < nw; w += 32) bm[warp][w] = 0u;
  __syncwarp();
  for (int r = 0; r < nq; ++r) {
    const int e1 = rp[I0 + r + 1];
    for (int e = rp[I0 + r] + lane; e < e1; e += 32) {
      const int X = ci[e];
      if (X >= 0 && X < nb && (!p.causal || X <= I0 + r)) atomicOr(&bm[warp][X >> 5], 1u << (X & 31));
    }
  }
  __syncwarp();
  int cnt = 0;
  for (int w = lane; w < nw; w += 32) cnt += __popc(bm[warp][w]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) cnt += __shfl_xor_sync(0xffffffffu, cnt, o);
  if (lane == 0) tiles[g] = (cnt * (p.block >> 5) + 3) >> 2;   // 32-key chunks, four per key tile
}

// Block-wide exclusive scan of one int per thread (1024 threads); returns the total too.
__device__ __forceinline__ int block_scan_excl(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += y;
  }
  __syncthreads();
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += y;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  return (warp > 0 ? warp_sums[warp - 1] : 0) + incl - v;
}

// Key tiles of work item k (its query tile's union, from the plan).
__device__ __forceinline__ int item_tiles(const Params& p, const int* tiles, int k) {
  const Item it = decode_item(p, k);
  const int m = p.n_masks > 1 ? p.head_mask[it.h] : 0;
  const int cs = p.csr_shared ? 0 : it.s;
  return tiles[(m * p.csr_batches + cs) * p.tiles_per_seq + it.tile];
}

__global__ void __launch_bounds__(1024) fwd_schedule_kernel(const __grid_constant__ Params p, const int* tiles,
                                                             int slot_cap, int n_pipes, int2* list, int4* split_items,
                                                             SplitHdr* hdr) {
  __shared__ int warp_sums[32];
  __shared__ int s_T;
  const int n = p.n_items;
  const int per = (n + 1023) / 1024;
  const int k0 = min(n, (int)threadIdx.x * per), k1 = min(n, k0 + per);
  // total work, longest item
  long long tot = 0;
  int mx = 0;
  for (int k = k0; k < k1; ++k) {
    const int t = item_tiles(p, tiles, k);
    tot += t;
    mx = max(mx, t);
  }
  // reduce (sum as int: a launch holds far fewer than 2^31 key tiles)
  int total = 0;
  block_scan_excl((int)tot, warp_sums, total);
  int big = mx;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) big = max(big, __shfl_xor_sync(0xffffffffu, big, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) warp_sums[threadIdx.x >> 5] = big;
  __syncthreads();
  if (threadIdx.x == 0) {
    int b = 0;
    for (int w = 0; w < 32; ++w) b = max(b, warp_sums[w]);
    // about two parts of work per item stream (n_pipes: streams of the launch); parts of at
    // least kMinPartTiles key tiles
    int T = max(kMinPartTiles, (total + 2 * n_pipes - 1) / (2 * n_pipes));
    // No split when the longest item is within 1.25x of a stream's even share: the
    // longest-first order then balances the streams about as well, without the partial
    // results and the merge.
    const int share = (total + n_pipes - 1) / n_pipes;
    if (4 * b <= 5 * share) T = max(T, b);
    s_T = T;
    warp_sums[0] = b;
  }
  __syncthreads();
  const int longest = warp_sums[0];
  int T = s_T;
  __syncthreads();
  // the smallest T (doubling) whose parts fit the slots
  for (;;) {
    int need = 0;
    for (int k = k0; k < k1; ++k) {
      const int t = item_tiles(p, tiles, k);
      if (t > T) need += (t + T - 1) / T;
    }
    int need_tot = 0;
    block_scan_excl(need, warp_sums, need_tot);
    if (need_tot <= slot_cap || T >= longest) break;
    T *= 2;
  }
  // positions: split parts first (slot = list position), then the unsplit items
  int n_parts = 0, n_whole = 0, n_si = 0;
  for (int k = k0; k < k1; ++k) {
    const int t = item_tiles(p, tiles, k);
    if (t > T) {
      n_parts += (t + T - 1) / T;
      ++n_si;
    } else {
      ++n_whole;
    }
  }
  int tot_parts = 0, tot_whole = 0, tot_si = 0;
  int pos_p = block_scan_excl(n_parts, warp_sums, tot_parts);
  int pos_w = block_scan_excl(n_whole, warp_sums, tot_whole);
  int pos_s = block_scan_excl(n_si, warp_sums, tot_si);
  pos_w += tot_parts;
  for (int k = k0; k < k1; ++k) {
    const int t = item_tiles(p, tiles, k);
    if (t > T) {
      const int parts = (t + T - 1) / T;
      split_items[pos_s++] = make_int4(k, parts, pos_p, 0);
      for (int q = 0; q < parts; ++q) list[pos_p++] = make_int2(k, q);
    } else {
      list[pos_w++] = make_int2(k, 0);
    }
  }
  if (threadIdx.x == 0) {
    hdr->list_len = tot_parts + tot_whole;
    hdr->n_split = tot_parts;
    hdr->part_tiles = T;
    hdr->n_split_items = tot_si;
  }
}

template <int D>
__global__ void __launch_bounds__(kTile) fwd_merge_kernel(const __grid_constant__ Params p, const int4* split_items,
                                                           const SplitHdr* hdr) {
  const float kNegInf = __int_as_float(0xff800000);
  const int n_si = hdr->n_split_items;
  const int r = threadIdx.x;
  for (int j = blockIdx.x; j < n_si; j += gridDim.x) {
    const int4 si = split_items[j];
    const Item it = decode_item(p, si.x);
    const int qtok = it.tile * kTile + r;
    if (qtok >= p.n_tokens) continue;
    const float* base = p.partial + (size_t)si.z * (kTile * (D + 1));
    float mx = kNegInf;
    for (int q = 0; q < si.y; ++q) mx = fmaxf(mx, base[(size_t)q * (kTile * (D + 1)) + kTile * D + r]);
    __nv_bfloat16* orow = p.o + (int64_t)it.s * p.o_sb + (int64_t)qtok * p.o_sn + (int64_t)it.h * p.o_sh;
    float lse = kNegInf;
    float acc[D];
#pragma unroll
    for (int c = 0; c < D; ++c) acc[c] = 0.f;
    if (mx != kNegInf) {
      float wsum = 0.f;
      for (int q = 0; q < si.y; ++q) {
        const float* part = base + (size_t)q * (kTile * (D + 1));
        const float lq = part[kTile * D + r];
        if (lq == kNegInf) continue;
        const float w = __expf(lq - mx);
        wsum += w;
        const float4* row = reinterpret_cast<const float4*>(part + (size_t)r * D);
#pragma unroll
        for (int c = 0; c < D / 4; ++c) {
          const float4 v = row[c];
          acc[4 * c] += w * v.x;
          acc[4 * c + 1] += w * v.y;
          acc[4 * c + 2] += w * v.z;
          acc[4 * c + 3] += w * v.w;
        }
      }
      const float inv = 1.f / wsum;
#pragma unroll
      for (int c = 0; c < D; ++c) acc[c] *= inv;
      lse = mx + __logf(wsum);
    }
    uint4* dst = reinterpret_cast<uint4*>(orow);
#pragma unroll
    for (int c = 0; c < D / 8; ++c)
      dst[c] = make_uint4(pack_bf16x2(acc[8 * c], acc[8 * c + 1]), pack_bf16x2(acc[8 * c + 2], acc[8 * c + 3]),
                          pack_bf16x2(acc[8 * c + 4], acc[8 * c + 5]), pack_bf16x2(acc[8 * c + 6], acc[8 * c + 7]));
    p.lse[((int64_t)it.s * p.heads + it.h) * p.n_tokens + qtok] = lse;
  }
}

// Workspace of the forward: the work counter, then (split mode) the split header, the plan's
// key-tile counts, the work list, the split items and the partial-result slots, each section
// 256-byte aligned. slot_cap is the number of slots that fit in `bytes`.
struct FwdWorkspace {
  size_t counter_off, hdr_off, tiles_off, list_off, items_off, partial_off, min_bytes, slot_cap;
};

inline size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

FwdWorkspace fwd_workspace_layout(int64_t n_items, int64_t n_groups, int d, size_t bytes) {
  FwdWorkspace w;
  w.counter_off = 0;
  w.hdr_off = 64;
  w.min_bytes = 256;
  w.tiles_off = 256;
  w.list_off = w.tiles_off + up256((size_t)n_groups * 4);
  const size_t slot_bytes = (size_t)kTile * (d + 1) * 4;
  const size_t fixed = w.list_off + up256((size_t)n_items * 8) + 3 * 256;
  // per slot: one list entry (8 B), at most one split item (16 B), the partial (slot_bytes)
  w.slot_cap = bytes > fixed ? (bytes - fixed) / (8 + 16 + slot_bytes) : 0;
  w.items_off = w.list_off + up256((size_t)(n_items + (int64_t)w.slot_cap) * 8);
  w.partial_off = w.items_off + up256(w.slot_cap * 16);
  return w;
}

// The forward kernel of head dimension D.
template <int D>
constexpr auto fwd_kernel() {
  if constexpr (Cfg<D>::WIDE) return attn_fwd_wide_kernel<D, false>;
  else return attn_fwd_kernel<D, false>;
}

template <int D>
int launch_d(const AttnArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tq, tk, tv, to;
  const uint32_t kv_rows = a.block == 32 ? 32u : 64u;
  if (!encode_bhnd_map(&tq, a.q, a.batch, a.n_tokens, a.heads, D, a.q_strides[0], a.q_strides[1], a.q_strides[2],
                       C::CH, kTile, C::TMA_SWZ) ||
      !encode_bhnd_map(&tk, a.k, a.batch, a.n_tokens, a.kv_heads, D, a.kv_strides[0], a.kv_strides[1],
                       a.kv_strides[2], C::CH, kv_rows, C::TMA_SWZ) ||
      !encode_bhnd_map(&tv, a.v, a.batch, a.n_tokens, a.kv_heads, D, a.kv_strides[0], a.kv_strides[1],
                       a.kv_strides[2], C::CH, kv_rows, C::TMA_SWZ))
    return SA_ERR_UNSUPPORTED;
  Params p;
  p.batch = a.batch;
  p.n_tokens = a.n_tokens;
  p.heads = a.heads;
  p.heads_per_kv = a.heads / a.kv_heads;
  p.block = a.block;
  p.log2b = __builtin_ctz((unsigned)a.block);
  p.nb = a.n_tokens / a.block;
  p.causal = a.causal;
  p.csr_shared = a.csr_shared;
  p.tiles_per_seq = (a.n_tokens + kTile - 1) / kTile;
  p.n_items = a.batch * a.heads * p.tiles_per_seq;
  p.n_masks = a.n_masks;
  for (int m = 0; m < kMaxMasks; ++m) {
    p.row_ptr[m] = a.row_ptr[m];
    p.col_idx[m] = a.col_idx[m];
  }
  for (int h = 0; h < kMaxHeadMap; ++h) p.head_mask[h] = a.head_mask[h];
  p.o = static_cast<__nv_bfloat16*>(a.o);
  // d = 64: O leaves through TMA stores of 32-row boxes when its layout allows a tensor map
  // (16-byte aligned base and strides); otherwise, and at other d, through plain stores
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
  p.csr_batches = a.csr_shared ? 1 : a.batch;
  const int n_groups = a.n_masks * p.csr_batches * p.tiles_per_seq;
  const FwdWorkspace ws = fwd_workspace_layout(p.n_items, n_groups, D, a.workspace_bytes);
  if (a.workspace == nullptr || a.workspace_bytes < ws.min_bytes) return SA_ERR_CAPACITY;
  uint8_t* wsb = static_cast<uint8_t*>(a.workspace);
  p.work_counter = reinterpret_cast<unsigned int*>(wsb + ws.counter_off);
  p.work_list = nullptr;
  p.list_hdr = nullptr;
  p.partial = nullptr;
  if (cudaMemsetAsync(p.work_counter, 0, sizeof(unsigned int), stream) != cudaSuccess) return SA_ERR_CUDA;
  const int sm_count = current_sm_count();
  // d <= 64: two pipelines per CTA; d = 128: one item stream per CTA
  auto kern = fwd_kernel<D>();
  // The register split in the kernel hands out exactly the launch allocation: refuse to
  // launch a build whose per-thread register count differs from it.
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SA_ERR_CUDA;
  if (fa.numRegs != kLaunchRegs) return SA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return SA_ERR_CUDA;
  // Split mode when the items are few for the GPU's item streams and the workspace holds
  // partial-result slots: long key lists are then cut into parts (K9), about two per stream.
  // d <= 64 (two streams per SM, each at about half an SM's speed): fewer than two items per
  // stream. d = 128 (one stream per SM at a whole SM's speed, which balances a few long items
  // well in longest-first order): fewer items than SMs. The schedule kernel still keeps the
  // items whole when the longest is within 1.25x of a stream's share.
  const int per_cta = C::WIDE ? 1 : 2;
  const int n_pipes = per_cta * sm_count;
  const bool split = ws.slot_cap >= 2 && p.n_items < (C::WIDE ? 1 : 2) * n_pipes;
  int grid = (p.n_items + per_cta - 1) / per_cta < sm_count ? (p.n_items + per_cta - 1) / per_cta : sm_count;
  if (split) {
    int* tiles = reinterpret_cast<int*>(wsb + ws.tiles_off);
    int2* list = reinterpret_cast<int2*>(wsb + ws.list_off);
    int4* split_items = reinterpret_cast<int4*>(wsb + ws.items_off);
    SplitHdr* hdr = reinterpret_cast<SplitHdr*>(wsb + ws.hdr_off);
    p.partial = reinterpret_cast<float*>(wsb + ws.partial_off);
    fwd_plan_kernel<<<(n_groups + kPlanWarps - 1) / kPlanWarps, 32 * kPlanWarps, 0, stream>>>(p, n_groups, tiles);
    fwd_schedule_kernel<<<1, 1024, 0, stream>>>(p, tiles, (int)ws.slot_cap, n_pipes, list, split_items, hdr);
    if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
    p.work_list = list;
    p.list_hdr = &hdr->list_len;
    grid = sm_count;   // the list is at most n_items + slot_cap entries long
    kern<<<grid, kThreads, C::SMEM, stream>>>(tq, tk, tv, to, p);
    if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
    const int mgrid = (int)(ws.slot_cap < (size_t)(2 * sm_count) ? ws.slot_cap : (size_t)(2 * sm_count));
    fwd_merge_kernel<D><<<mgrid, kTile, 0, stream>>>(p, split_items, hdr);
    return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
  }
  kern<<<grid, kThreads, C::SMEM, stream>>>(tq, tk, tv, to, p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

size_t attn_fwd_workspace_bytes(int64_t batch, int64_t n_tokens, int64_t heads, int head_dim, int64_t csr_batches,
                                int64_t n_masks) {
  const int64_t tiles_per_seq = (n_tokens + kTile - 1) / kTile;
  const int64_t n_items = batch * heads * tiles_per_seq;
  const FwdWorkspace w = fwd_workspace_layout(n_items, n_masks * csr_batches * tiles_per_seq, head_dim, 0);
  const size_t slot_bytes = (size_t)kTile * (head_dim + 1) * 4;
  // room for the default number of split parts (about four per SM of a GB300)
  return w.list_off + up256((size_t)(n_items + kFwdDefaultSlots) * 8) + up256((size_t)kFwdDefaultSlots * 16) +
         (size_t)kFwdDefaultSlots * slot_bytes + 3 * 256;
}

int launch_attn_fwd(const AttnArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_d<32>(a, stream);
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int attn_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_attn_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_attn_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
