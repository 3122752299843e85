// A cache of slots whose rows carry the attention weight that they have gathered: rows go in one behind the
// other, and an eviction keeps `keep` slots of every (sequence, key head): those of the first `sinks` and
// the newest `recent` tokens, then the ones of most weight (ties: the lower slot). Attention does not depend
// on the order of a sequence's keys, so the kept rows stay where they are, and only those at or past slot `keep`
// move, the e-th of them into the e-th freed slot below it: no row that stays is read.
//
// Eviction: one launch, no workspace. A cluster's CTAs take one (sequence, key head); each finds the whole
// selection for itself (8 bytes a slot) and moves its share of the rows (8 D bytes each, there and back):
//   key      32 bits that order like the weight; a protected slot has the largest key
//   select   the keep-th largest key T, eight bits a pass, by histograms in shared memory
//   flags    a bit per slot: freed (below `keep`) or to move (from `keep` on), with counts per 256 slots, so
//            that the e-th set bit is found in a few steps
// The ranks meet before the first write, since outputs may lie over the inputs.
//
// Bound by the bytes of the rows that move, or, where few do, by the selection's latency.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "sa_internal.h"

namespace sa {
namespace {

__device__ unsigned int g_scored_err;

// ------------------------------------------------------------------ append

struct AppendParams {
  const uint4* x[2];                // k, v
  uint4* cache[2];
  int64_t x_sb[2], x_sn[2], x_sh[2], c_sb[2], c_sn[2], c_sh[2];   // 16-byte words
  const int32_t* start;
  const int32_t* tokens;
  float* weights;
  int32_t* positions;
  int n, kv_heads, capacity;
  uint32_t words;                   // 16-byte words of a sequence's keys
};

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  const uint32_t w = blockIdx.x * 256u + threadIdx.x;
  const int s = blockIdx.y >> 1, m = blockIdx.y & 1;
  const int start = p.start ? p.start[s] : 0;
  if (w >= p.words || start < 0) return;
  const int u = (int)(w % (D / 8)), row = (int)(w / (D / 8)), hk = row % p.kv_heads, i = row / p.kv_heads;
  const int64_t slot = (int64_t)start + i;
  if (slot >= p.capacity) {
    if (u == 0 && hk == 0 && m == 0) atomicOr(&g_scored_err, kErrBadIndex);
    return;
  }
  p.cache[m][s * p.c_sb[m] + slot * p.c_sn[m] + hk * p.c_sh[m] + u] = p.x[m][s * p.x_sb[m] + i * p.x_sn[m] + hk * p.x_sh[m] + u];
  if (m == 0 && u == 0) {
    const int64_t at = ((int64_t)s * p.kv_heads + hk) * p.capacity + slot;
    p.weights[at] = 0.f;
    p.positions[at] = p.tokens ? (int32_t)((uint32_t)p.tokens[s] + (uint32_t)i) : (int32_t)slot;
  }
}

// ------------------------------------------------------------------ eviction

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCachedKeys = 16384;     // keys of longer lists are formed anew in every pass
constexpr int kGroup = 256;            // slots per count

struct EvictParams {
  uint4* cache[2];
  int64_t c_sb[2], c_sn[2], c_sh[2];
  const float* w_in;
  const int32_t* pos_in;
  const int32_t* len_in;
  float* w_out;
  int32_t* pos_out;
  int32_t* len_out;                    // null: written by a launch of its own
  int kv_heads, capacity, keep, sinks, recent;
  int cached;                          // keys are kept in shared memory
};

// Orders like the weight; NaN counts as more than infinity, -0 as 0.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sinks, int64_t first_recent) {
  if (pos < sinks || pos >= first_recent) return 0xffffffffu;
  if (w != w) return 0xfffffffeu;
  const uint32_t b = __float_as_uint(w + 0.f);
  return b & 0x80000000u ? ~b : b | 0x80000000u;
}

// Sum over the CTA's threads before this one, and in all (two barriers).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o *= 2) {
    const int y = __shfl_up_sync(0xffffffffu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();                     // the sums of the call before have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  int before = 0;
  all = 0;
#pragma unroll
  for (int k = 0; k < kWarps; ++k) {
    const int y = warp_sums[k];
    before += k < warp ? y : 0;
    all += y;
  }
  return before + x - v;
}

// Slot of the e-th (from 0) set flag.
__device__ __forceinline__ int select_flag(const uint32_t* flags, const int* counts, int groups, int e) {
  int lo = 0, hi = groups - 1;         // counts[g]: flags before group g
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (counts[mid] <= e) lo = mid;
    else hi = mid - 1;
  }
  e -= counts[lo];
  int w = lo * (kGroup / 32);
  for (int n = __popc(flags[w]); e >= n; n = __popc(flags[w])) {
    e -= n;
    ++w;
  }
  uint32_t bits = flags[w];
  int at = 32 * w;
#pragma unroll
  for (int half = 16; half > 0; half /= 2) {
    const int low = __popc(bits & ((1u << half) - 1u));
    if (e >= low) {
      e -= low;
      bits >>= half;
      at += half;
    }
  }
  return at;
}

template <int D>
__global__ void __launch_bounds__(kThreads) evict_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int hist[kWarps][256];
  __shared__ int warp_sums[kWarps];
  __shared__ int found[2];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, ranks = gridDim.x, hk = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = max(0, min(p.len_in[s], p.capacity)), keep = p.keep;
  const int64_t list = ((int64_t)s * p.kv_heads + hk) * p.capacity;
  const float* w_in = p.w_in + list;
  const int32_t* pos_in = p.pos_in + list;
  float* w_out = p.w_out + list;
  int32_t* pos_out = p.pos_out + list;
  if (p.len_out && rank == 0 && hk == 0 && threadIdx.x == 0) p.len_out[s] = min(len, keep);
  if (len <= keep) {                   // the whole cluster
    if (rank == 0)
      for (int j = threadIdx.x; j < len; j += kThreads) {
        w_out[j] = w_in[j];
        pos_out[j] = pos_in[j];
      }
    return;
  }
  const int words = (len + 31) / 32, groups = (len + kGroup - 1) / kGroup;
  int* counts = reinterpret_cast<int*>(smem);
  uint32_t* flags = reinterpret_cast<uint32_t*>(counts + (p.capacity + kGroup - 1) / kGroup);
  uint32_t* keys = flags + (p.capacity + kGroup - 1) / kGroup * (kGroup / 32);
  // ---- the newest token
  int newest = INT32_MIN;
  for (int j = threadIdx.x; j < len; j += kThreads) newest = max(newest, pos_in[j]);
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_sums[warp] = newest;
  __syncthreads();
#pragma unroll
  for (int k = 0; k < kWarps; ++k) newest = max(newest, warp_sums[k]);
  const int64_t first_recent = (int64_t)newest - p.recent + 1;
  const auto form = [&](int j) { return key_of(w_in[j], pos_in[j], p.sinks, first_recent); };
  if (p.cached)
    for (int j = threadIdx.x; j < len; j += kThreads) keys[j] = form(j);
  const auto key = [&](int j) { return p.cached ? keys[j] : form(j); };
  // ---- T, the keep-th largest key: its bits from the top, `left` the rank among the keys that share them
  uint32_t T = 0;
  int left = keep, equal = 0;
#pragma unroll 1
  for (int shift = 24; shift >= 0; shift -= 8) {
    for (int b = threadIdx.x; b < kWarps * 256; b += kThreads) hist[b >> 8][b & 255] = 0;
    __syncthreads();
    for (int j = threadIdx.x; j < len; j += kThreads) {
      const uint32_t k = key(j);
      if (shift == 24 || (k ^ T) >> (shift + 8) == 0) atomicAdd(&hist[warp][(k >> shift) & 255], 1);
    }
    __syncthreads();
    // thread b < 256: keys in bin 255 - b, and in the bins above it
    int n = 0;
    if (threadIdx.x < 256) {
#pragma unroll
      for (int k = 0; k < kWarps; ++k) n += hist[k][255 - threadIdx.x];
    }
    int all;
    const int above = block_scan(n, warp_sums, all);
    if (above < left && left <= above + n) {
      found[0] = 255 - threadIdx.x;
      found[1] = above;
      hist[0][0] = n;
    }
    __syncthreads();
    T |= (uint32_t)found[0] << shift;
    left -= found[1];
    equal = hist[0][0];
    __syncthreads();
  }
  // ---- flags: of the keys equal to T the first `left` stay. A warp takes 32 consecutive slots a time.
  int base = 0;                        // keys equal to T in the slots before, where not all of them stay
#pragma unroll 1
  for (int j0 = 0; j0 < words * 32; j0 += kThreads) {
    const int j = j0 + threadIdx.x;
    const uint32_t k = j < len ? key(j) : 0u;
    const bool same = j < len && k == T;
    bool kept = j < len && k >= T;
    if (left < equal) {
      int all;
      const int before = base + block_scan(same ? 1 : 0, warp_sums, all);
      base += all;
      if (same && before >= left) kept = false;
    }
    const uint32_t bits = __ballot_sync(0xffffffffu, j < len && (j < keep ? !kept : kept));
    if (lane == 0 && j < words * 32) flags[j / 32] = bits;
  }
  for (int w = words + threadIdx.x; w < groups * (kGroup / 32); w += kThreads) flags[w] = 0u;
  __syncthreads();
  // ---- counts before each group, and the freed slots (as many as there are rows to move)
  int total = 0;
#pragma unroll 1
  for (int g0 = 0; g0 < groups; g0 += kThreads) {
    const int g = g0 + threadIdx.x;
    int n = 0;
    if (g < groups)
#pragma unroll
      for (int k = 0; k < kGroup / 32; ++k) n += __popc(flags[g * (kGroup / 32) + k]);
    int all;
    const int before = total + block_scan(n, warp_sums, all);
    if (g < groups) counts[g] = before;
    total += all;
  }
  const int moves = total / 2;
  cluster.sync();                      // every rank has read what the outputs may lie over
  // ---- weights and positions: rank 0
  if (rank == 0) {
    if (w_out != w_in || pos_out != pos_in)
      for (int j = threadIdx.x; j < keep; j += kThreads) {
        if ((flags[j / 32] >> (j & 31)) & 1u) continue;
        w_out[j] = w_in[j];
        pos_out[j] = pos_in[j];
      }
    for (int e = threadIdx.x; e < moves; e += kThreads) {
      const int dst = select_flag(flags, counts, groups, e), src = select_flag(flags, counts, groups, moves + e);
      w_out[dst] = w_in[src];
      pos_out[dst] = pos_in[src];
    }
  }
  // ---- rows: a warp finds 32 moves at a time, then D / 8 lanes copy a row of keys and as many one of values
  constexpr int kLanes = D / 8, kSide = 32 / (2 * kLanes) > 0 ? 32 / (2 * kLanes) : 1;   // moves side by side
  constexpr int kDeep = 8;             // loads of a lane before its first store
  const int m = lane / kLanes & 1, u = lane % kLanes, side = lane / (2 * kLanes);
  uint4* rows = p.cache[m] + s * p.c_sb[m] + hk * p.c_sh[m] + u;
  const int64_t sn = p.c_sn[m];
#pragma unroll 1
  for (int e0 = 32 * (rank * kWarps + warp); e0 < moves; e0 += 32 * ranks * kWarps) {
    int src = 0, dst = 0;
    if (e0 + lane < moves) {
      dst = select_flag(flags, counts, groups, e0 + lane);
      src = select_flag(flags, counts, groups, moves + e0 + lane);
    }
    const int n = min(32, moves - e0);
#pragma unroll 1
    for (int i = 0; i < n; i += kDeep * kSide) {
      uint4 x[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int e = i + k * kSide + side, from = __shfl_sync(0xffffffffu, src, e & 31);
        if (e < n) x[k] = rows[from * sn];
      }
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        const int e = i + k * kSide + side, to = __shfl_sync(0xffffffffu, dst, e & 31);
        if (e < n) rows[to * sn] = x[k];
      }
    }
  }
}

__global__ void cut_lengths_kernel(const int32_t* in, int32_t* out, int n, int capacity, int keep) {
  const int s = blockIdx.x * 256 + threadIdx.x;
  if (s < n) out[s] = max(0, min(min(in[s], capacity), keep));
}

template <int D>
int launch_append(const ScoredArgs& a, cudaStream_t stream) {
  AppendParams p;
  memset(&p, 0, sizeof(p));
  for (int m = 0; m < 2; ++m) {
    const int64_t* x = m ? a.v_strides : a.k_strides;
    const int64_t* c = m ? a.v_cache_strides : a.k_cache_strides;
    p.x[m] = static_cast<const uint4*>(m ? a.v : a.k);
    p.cache[m] = static_cast<uint4*>(m ? a.v_cache : a.k_cache);
    p.x_sb[m] = x[0] / 8;
    p.x_sn[m] = x[1] / 8;
    p.x_sh[m] = x[2] / 8;
    p.c_sb[m] = c[0] / 8;
    p.c_sn[m] = c[1] / 8;
    p.c_sh[m] = c[2] / 8;
  }
  p.start = a.start;
  p.tokens = a.tokens;
  p.weights = a.weights_out;
  p.positions = a.positions_out;
  p.n = a.n_tokens;
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.words = (uint32_t)a.n_tokens * (uint32_t)a.kv_heads * (D / 8);
  append_kernel<D><<<dim3((p.words + 255) / 256, 2 * a.batch), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int D>
int launch_evict(const ScoredArgs& a, cudaStream_t stream) {
  EvictParams p;
  memset(&p, 0, sizeof(p));
  for (int m = 0; m < 2; ++m) {
    const int64_t* c = m ? a.v_cache_strides : a.k_cache_strides;
    p.cache[m] = static_cast<uint4*>(m ? a.v_cache : a.k_cache);
    p.c_sb[m] = c[0] / 8;
    p.c_sn[m] = c[1] / 8;
    p.c_sh[m] = c[2] / 8;
  }
  p.w_in = a.weights_in;
  p.pos_in = a.positions_in;
  p.len_in = a.lengths_in;
  p.w_out = a.weights_out;
  p.pos_out = a.positions_out;
  const bool over = a.lengths_out == a.lengths_in;       // other heads' CTAs may still read them
  p.len_out = over ? nullptr : a.lengths_out;
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.keep = a.keep;
  p.sinks = a.sinks;
  p.recent = a.recent;
  p.cached = a.capacity <= kCachedKeys;
  const int groups = (a.capacity + kGroup - 1) / kGroup;
  const int smem = groups * (4 + kGroup / 8) + (p.cached ? 4 * a.capacity : 0);
  const auto kern = evict_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SA_ERR_CUDA;
  // ranks of a cluster: each with 64 rows to move at least, if every evicted row were replaced, and not more than
  // two CTAs an SM in all
  const int most = a.keep < a.capacity - a.keep ? a.keep : a.capacity - a.keep;
  const int64_t lists = (int64_t)a.batch * a.kv_heads;
  const int sm_count = current_sm_count();
  int ranks = 1;
  while (ranks < 8 && 64 * 2 * ranks <= most && lists * 2 * ranks <= 2 * sm_count) ranks *= 2;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)ranks, (unsigned)a.kv_heads, (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return SA_ERR_CUDA;
  if (over) cut_lengths_kernel<<<(a.batch + 255) / 256, 256, 0, stream>>>(a.lengths_in, a.lengths_out, a.batch, a.capacity, a.keep);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

int launch_scored_append(const ScoredArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_append<32>(a, stream);
    case 64: return launch_append<64>(a, stream);
    case 128: return launch_append<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

int launch_scored_evict(const ScoredArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_evict<32>(a, stream);
    case 64: return launch_evict<64>(a, stream);
    case 128: return launch_evict<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int scored_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_scored_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_scored_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
