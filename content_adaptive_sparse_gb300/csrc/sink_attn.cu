// Causal attention over a token window and a few first tokens ("sinks"), forward, for sm_103a
// (tcgen05 + TMEM + TMA): key j is visible to query i iff j <= i and (i - j <= window or j < sinks).
//
// Work item: 128 queries of one (sequence, head). Its key tiles (128 keys) are those that the window
// meets and, where it does not reach back to it, the first one for the sinks; every role derives
// them from the item's number, so there is no list, no counter and no workspace, and items, of
// nearly equal length, are dealt out in turn to one persistent CTA per SM.
//
// The two 64-key halves of every tile are softmaxes of their own: half h has its running maximum,
// sum and output accumulator O_h = sum P v over its keys, and an item's end joins them:
//   m = max(m_0, m_1),  L = sum_h l_h 2^(m_h - m),  O = sum_h O_h 2^(m_h - m) / L,  LSE = m ln 2 + ln L.
// So no warp waits for another one's row maximum inside a tile (the exchange of half-row maxima was
// the longest wait of a softmax step), and the halves drift apart, one in the exponentials while the
// other is in its loads and stores. The running maximum is followed only when it grows by more than
// 2^8; probabilities are then at most 2^8, rounded to bf16 for the tensor core, and summed in fp32.
//
// TMEM (512 columns): S_b [128 b, +128), b = g % SB, SB = 2 (d = 128) or 3; P of half h over the first 32
// of its own 64 columns of S_b (bf16 pairs), so the PVs' completion frees S_b; then O_0 and O_1.
//
// Warp roles (512 threads; warp w runs on SM sub-partition w % 4):
//   warps 0-7   softmax: query rows 32 (w % 4) .. of the tile, key half w / 4
//   warp 8      lane 0 loads Q, K and V by TMA (V one tile behind K)
//   warp 9      lane 0 issues S_b = Q K^T
//   warps 10, 11  lane 0 issues O_h += P_h V_h (A = P from TMEM, B = V MN-major), h = 0, 1
//   warps 12-15 epilogue: an item's rows through shared memory and TMA stores, under the next item
//
// Measured: 64K tokens, 16 heads of 128, window 4095: 1409-1450 us, 1470-1513 TFLOP/s over the graph's edges, 0.8
// of the library product's rate; what is lost is in whole tiles at the window's two edges (32 of 33 key
// tiles' worth is visible) and in the handshakes of S, P and O between the issuing threads and the
// softmax warps (in a long loop, power-capped, 1570 us). 4 x 8192 tokens, 12 heads of 64, window 511: 92-100
// us, of which the exponentials take 45 at 16 a clock and SM (557 keys a row on average, hidden 32-key chunks
// left out). No pipe is full (issue 51 %, tensor 32 %): an item is 5.8 steps, and at its end both halves'
// warps wait for its last products, the epilogue and the next Q.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "half_softmax.cuh"
#include "ptx_sm100.cuh"
#include "sa_internal.h"
#include "tma_host.h"

namespace sa {
namespace {

struct FParams {
  int batch, n_tokens, heads, heads_per_kv;
  int tiles;                        // 128-row tiles per sequence
  int step_h, step_s, step_tile;    // one item of every CTA, in the items' digits (tile, sequence, head)
  int window, sinks;
  float* lse;
  float scale_log2;
};

// A CTA's items, of all (sequence, head) pairs of one query tile before the next. Step j is key tile 0
// (n_sink = 1, j = 0) or t0 + j - n_sink.
struct Item {
  int s, h, tile, t0, n_sink, steps;
  // The CTA's first item; the next ones are found by additions (64K, d = 128: 1476 -> 1432 us against a
  // division of each item's number in every role). The last tiles come first: they see the most keys.
  __device__ explicit Item(const FParams& p) {
    h = (int)blockIdx.x % p.heads;
    s = (int)blockIdx.x / p.heads % p.batch;
    tile = p.tiles - 1 - (int)blockIdx.x / p.heads / p.batch;
    keys(p);
  }
  __device__ __forceinline__ bool more() const { return tile >= 0; }
  __device__ __forceinline__ void next(const FParams& p) {
    h += p.step_h;
    s += p.step_s;
    tile -= p.step_tile;
    if (h >= p.heads) {
      h -= p.heads;
      ++s;
    }
    if (s >= p.batch) {
      s -= p.batch;
      --tile;
    }
    keys(p);
  }
  __device__ __forceinline__ void keys(const FParams& p) {
    t0 = max(0, tile * kTile - p.window) / kTile;
    n_sink = p.sinks > 0 && t0 > 0 ? 1 : 0;
    steps = n_sink + tile - t0 + 1;
  }
  __device__ __forceinline__ int key_tile(int j) const { return j < n_sink ? 0 : t0 + j - n_sink; }
  // The sink tile's second half is left out when the first holds every sink.
  __device__ __forceinline__ bool one_half(const FParams& p, int j) const { return j < n_sink && p.sinks <= kHalf; }
};

// ------------------------------------------------------------------ loader (warp 8, lane 0)

// One K or V tile into its ring stage: a box of 128 rows, or of 64 (`half`).
template <int D>
__device__ __forceinline__ bool load_tile(int t, const CUtensorMap* whole, const CUtensorMap* part, bool half,
                                          uint8_t* ring, uint64_t* full, uint64_t* empty, int hk, int tok, int s,
                                          volatile int* abort_flag) {
  using C = Cfg<D>;
  const int st = t % C::STAGES;
  if (t >= C::STAGES && !wait_bar(&empty[st], (uint32_t)(t / C::STAGES - 1) & 1u, abort_flag)) return false;
  mbar_arrive_expect_tx(&full[st], half ? C::TILE / 2 : C::TILE);
  const CUtensorMap* map = half ? part : whole;
#pragma unroll
  for (int c = 0; c < C::NCH; ++c)
    tma_load_4d(ring + st * C::TILE + c * C::CHUNK, map, &full[st], c * C::CH, hk, tok, s);
  return true;
}

// The loader is one thread between the softmax warps' instructions; at d = 64 its instructions per
// tile decide how far ahead it gets, so a tile is one box and nothing is divided inside an item.
template <int D>
__device__ void loader(const FParams& p, const CUtensorMap* tq, const CUtensorMap* tk, const CUtensorMap* tv,
                       const CUtensorMap* tkh, const CUtensorMap* tvh, Bars& bars, uint8_t* sQ, uint8_t* sK, uint8_t* sV,
                       volatile int* abort_flag) {
  using C = Cfg<D>;
  int g = 0, gv = 0, n = 0;          // K tiles, V tiles and Q tiles requested
  bool ok = true;
  const bool halved = p.sinks <= kHalf;
  for (Item it(p); ok && it.more(); it.next(p)) {
    const int hk = it.h / p.heads_per_kv;
    const int qb = n & 1;
    if (n >= 2 && !(ok = wait_bar(&bars.q_empty[qb], (uint32_t)(n / 2 - 1) & 1u, abort_flag))) break;
    mbar_arrive_expect_tx(&bars.q_full[qb], C::TILE);
#pragma unroll
    for (int c = 0; c < C::NCH; ++c)
      tma_load_4d(sQ + qb * C::TILE + c * C::CHUNK, tq, &bars.q_full[qb], c * C::CH, it.h, it.tile * kTile, it.s);
    ++n;
    int tok = it.n_sink ? 0 : it.t0 * kTile, before = 0;
    bool half = it.n_sink != 0 && halved, half_before = false;
    for (int j = 0; j <= it.steps; ++j) {              // V one tile behind K
      if (j < it.steps) {
        if (!(ok = load_tile<D>(g, tk, tkh, half, sK, bars.k_full, bars.k_empty, hk, tok, it.s, abort_flag))) break;
        ++g;
      }
      if (j > 0) {
        if (!(ok = load_tile<D>(gv, tv, tvh, half_before, sV, bars.v_full, bars.v_empty, hk, before, it.s, abort_flag)))
          break;
        ++gv;
      }
      before = tok;
      half_before = half;
      tok = j < it.n_sink ? it.t0 * kTile : tok + kTile;
      half = false;
    }
  }
  // every copy of this CTA has landed before it may exit
  for (int i = max(0, n - 2); i < n; ++i) drain_bar(&bars.q_full[i & 1], (uint32_t)(i >> 1) & 1u);
  for (int t = max(0, g - C::STAGES); t < g; ++t) drain_bar(&bars.k_full[t % C::STAGES], (uint32_t)(t / C::STAGES) & 1u);
  for (int t = max(0, gv - C::STAGES); t < gv; ++t) drain_bar(&bars.v_full[t % C::STAGES], (uint32_t)(t / C::STAGES) & 1u);
}

// ------------------------------------------------------------------ softmax (warps 0-7)

// Keys c .. c + 31 that query i sees (bit b: key c + b).
__device__ __forceinline__ uint32_t visible(int i, int c, int window, int sinks) {
  const int lim = i - c, low = lim - window, sk = sinks - c;
  const uint32_t upto = lim >= 31 ? 0xffffffffu : (lim < 0 ? 0u : ((2u << lim) - 1u));
  const uint32_t from = low <= 0 ? 0xffffffffu : (low >= 32 ? 0u : (0xffffffffu << low));
  const uint32_t sink = sk >= 32 ? 0xffffffffu : (sk <= 0 ? 0u : ((1u << sk) - 1u));
  return upto & (from | sink);
}

// Whether some of queries q .. q + 31 sees some of keys k .. k + 31.
__device__ __forceinline__ bool some(int q, int k, int window, int sinks) {
  return q + 31 >= k && (q - (k + 31) <= window || k < sinks);
}
// How they see keys k .. k + 63.
__device__ __forceinline__ int visibility(int q, int k, int window, int sinks) {
  if (q + 31 < k || (q - (k + 63) > window && k >= sinks)) return kNone;
  return q >= k + 63 && (q + 31 - k <= window || k + 63 < sinks) ? kAll : kSome;
}

template <int D>
__device__ void softmax(const FParams& p, Bars& bars, Handoff* hand, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, half = warp >> 2;
  const int row = quarter * 32 + lane;
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
  Softmax<D> W{bars, abort_flag, base + 64u * half, base + C::COL_O + (uint32_t)(D * half), half, lane, p.scale_log2,
               0.f, 0.f};
  int g = 0, n = 0;
  for (Item it(p); it.more(); it.next(p), ++n) {
    const int q0 = it.tile * kTile + 32 * quarter;
    W.m = kLowest;
    W.l = 0.f;
    bool later = false;
    for (int j = 0; j < it.steps; ++j, ++g) {
      const int k0 = it.key_tile(j) * kTile + kHalf * half;
      const int see = visibility(q0, k0, p.window, p.sinks);
      if (!W.done(bars.s_full, g)) return;
      if (half == 1 && it.one_half(p, j)) {            // left out: nothing to store
        if (lane == 0) mbar_arrive(&bars.p_full[1][g % C::SB]);
        continue;
      }
      tc_fence_after();
      bool ok;
      if (see == kAll) ok = W.template tile<kAll>(g, true, true, 0u, 0u, later);
      else if (see == kSome)
        ok = W.template tile<kSome>(g, some(q0, k0, p.window, p.sinks), some(q0, k0 + 32, p.window, p.sinks),
                                    visible(q0 + lane, k0, p.window, p.sinks),
                                    visible(q0 + lane, k0 + 32, p.window, p.sinks), later);
      else ok = W.template tile<kNone>(g, false, false, 0u, 0u, later);
      if (!ok) return;
      later = true;
    }
    // the rows' maxima and sums go to the epilogue
    const int e = n & 1;
    if (n >= 2 && !__all_sync(0xffffffffu, wait_bar(&bars.epi_empty[e], (uint32_t)(n / 2 - 1) & 1u, abort_flag))) return;
    hand[e].m[half][row] = W.m;
    hand[e].l[half][row] = W.l;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.epi_full[e]);
  }
}

// ------------------------------------------------------------------ epilogue (warps 12-15)

template <int D>
__device__ void epilogue(const FParams& p, const CUtensorMap* to, Bars& bars, const Handoff* hand, uint8_t* out,
                         uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
  uint8_t* stage = out + quarter * C::OUT;
  const uint32_t srow = smem_u32(stage) + 64u * lane;
  int n = 0;
  for (Item it(p); it.more(); it.next(p), ++n) {
    const int e = n & 1;
    if (!__all_sync(0xffffffffu, wait_bar(&bars.epi_full[e], (uint32_t)(n >> 1) & 1u, abort_flag))) break;
    const float m0 = hand[e].m[0][row], m1 = hand[e].m[1][row], l0 = hand[e].l[0][row], l1 = hand[e].l[1][row];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.epi_empty[e]);
    const float m = fmaxf(m0, m1);
    float f0 = ex2_approx(m0 - m), f1 = ex2_approx(m1 - m);
    const float L = l0 * f0 + l1 * f1;
    const float inv = L == 0.f ? 0.f : 1.f / L;        // every query sees itself: 0 where its scores are all -inf
    f0 *= inv;
    f1 *= inv;
    const int q0 = it.tile * kTile + 32 * quarter, tok = q0 + lane;
    if (tok < p.n_tokens)
      p.lse[((int64_t)it.s * p.heads + it.h) * p.n_tokens + tok] =
          (m + __log2f(L)) * 0.69314718055994531f;
    if (!__all_sync(0xffffffffu, wait_bar(&bars.o_full, (uint32_t)n & 1u, abort_flag))) break;
    tc_fence_after();
    const uint32_t t0 = base + C::COL_O, t1 = t0 + D;
#pragma unroll 1
    for (int c0 = 0; c0 < D; c0 += 32 * C::BOXES) {
      if (lane == 0) bulk_wait_group_read<0>();          // the staging memory has been read
      __syncwarp();
#pragma unroll
      for (int q = 0; q < 2 * C::BOXES; ++q) {
        uint32_t a[16], b[16];
        tmem_ld_x16(t0 + c0 + 16 * q, a);
        tmem_ld_x16(t1 + c0 + 16 * q, b);
        tmem_ld_wait<16>(a);
        tmem_ld_wait<16>(b);
        uint32_t pk[8];
#pragma unroll
        for (int j = 0; j < 16; j += 2)
          pk[j >> 1] = pack_bf16x2(__uint_as_float(a[j]) * f0 + __uint_as_float(b[j]) * f1,
                                   __uint_as_float(a[j + 1]) * f0 + __uint_as_float(b[j + 1]) * f1);
        // 64-byte rows, 64B swizzle: unit u of row r at u ^ (r / 2) % 4
        const uint32_t x = (uint32_t)(lane >> 1) & 3u, u = 2u * (q & 1), box = srow + 2048u * (q >> 1);
        st_shared_v4(box + ((u ^ x) << 4), pk[0], pk[1], pk[2], pk[3]);
        st_shared_v4(box + (((u + 1u) ^ x) << 4), pk[4], pk[5], pk[6], pk[7]);
      }
      if (c0 + 32 * C::BOXES == D) {
        // the accumulators have been read: the next item's PVs may start
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.o_free);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0 && q0 < p.n_tokens) {                // rows past the sequence are dropped by the store
#pragma unroll
        for (int x = 0; x < C::BOXES; ++x) tma_store_4d(to, stage + 2048 * x, c0 + 32 * x, it.h, q0, it.s);
        bulk_commit_group();
      }
    }
  }
  // this warp's stores are complete before the CTA may exit
  if (lane == 0) bulk_wait_group<0>();
  __syncwarp();
}

// ------------------------------------------------------------------ kernel

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    sink_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap tkh,
                    const __grid_constant__ CUtensorMap tvh, const __grid_constant__ CUtensorMap to,
                    const __grid_constant__ FParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ Handoff hand[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // uniform
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
      mbar_init(&bars.epi_full[i], kSoftmaxWarps);
      mbar_init(&bars.epi_empty[i], kEpilogueWarps);
    }
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.v_full[i], 1);
      mbar_init(&bars.v_empty[i], 2);                    // both halves' issuers
    }
    for (int i = 0; i < C::SB; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.pv_done[i], 2);                    // both halves' issuers
      for (int h = 0; h < 2; ++h) mbar_init(&bars.p_full[h][i], kHalfWarps);
    }
    mbar_init(&bars.o_full, 2);                          // both halves' issuers
    mbar_init(&bars.o_free, kEpilogueWarps);
    for (int i = 0; i < 3; ++i) mbar_init(&bars.drain[i], 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
    tma_prefetch_desc(&to);
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  uint8_t* sQ = sbase;
  uint8_t* sK = sQ + 2 * C::TILE;
  uint8_t* sV = sK + C::STAGES * C::TILE;
  uint8_t* sOut = sV + C::STAGES * C::TILE;
  // The register split's sum is the launch's allocation (checked on the host), so the growth
  // always completes.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;" ::: "memory");
    softmax<D>(p, bars, hand, tmem, &abort_flag);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
    if (warp == 8) {
      if (elect_one()) loader<D>(p, &tq, &tk, &tv, &tkh, &tvh, bars, sQ, sK, sV, &abort_flag);
      __syncwarp();
    } else if (warp == 9) {
      if (elect_one()) qk_issuer<D, Item>(p, bars, sQ, sK, tmem, &abort_flag);
      __syncwarp();
    } else if (warp < 12) {
      if (elect_one()) pv_issuer<D, Item>(p, warp - 10, bars, sV, tmem, &abort_flag);
      __syncwarp();
    } else {
      epilogue<D>(p, &to, bars, hand, sOut, tmem, &abort_flag);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

template <int D>
int launch_d(const SinkArgs& a, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tq, tk, tv, tkh, tvh, to;
  const auto map = [&](CUtensorMap* m, const void* base, int heads, const int64_t st[3], int cols, int rows,
                       CUtensorMapSwizzle swz) {
    return encode_bhnd_map(m, base, a.batch, a.n_tokens, heads, D, st[0], st[1], st[2], cols, rows, swz);
  };
  if (!map(&tq, a.q, a.heads, a.q_strides, C::CH, kTile, C::TMA_SWZ) ||
      !map(&tk, a.k, a.kv_heads, a.k_strides, C::CH, kTile, C::TMA_SWZ) ||
      !map(&tv, a.v, a.kv_heads, a.v_strides, C::CH, kTile, C::TMA_SWZ) ||
      !map(&tkh, a.k, a.kv_heads, a.k_strides, C::CH, kHalf, C::TMA_SWZ) ||
      !map(&tvh, a.v, a.kv_heads, a.v_strides, C::CH, kHalf, C::TMA_SWZ) ||
      !map(&to, a.o, a.heads, a.o_strides, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
    return SA_ERR_UNSUPPORTED;
  FParams p;
  p.batch = a.batch;
  p.n_tokens = a.n_tokens;
  p.heads = a.heads;
  p.heads_per_kv = a.heads / a.kv_heads;
  p.tiles = (a.n_tokens + kTile - 1) / kTile;
  p.window = a.window;
  p.sinks = a.sinks;
  p.lse = a.lse;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  const auto kern = sink_fwd_kernel<D>;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SA_ERR_CUDA;
  if (fa.numRegs != kLaunchRegs) return SA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return SA_ERR_CUDA;
  const int sm_count = current_sm_count();
  const int64_t items = (int64_t)a.batch * a.heads * p.tiles;
  const int grid = items < sm_count ? (int)items : sm_count;
  p.step_h = grid % a.heads;
  p.step_s = grid / a.heads % a.batch;
  p.step_tile = grid / a.heads / a.batch;
  kern<<<grid, kThreads, C::SMEM, stream>>>(tq, tk, tv, tkh, tvh, to, p);
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

unsigned int sink_fwd_read_and_clear_error(cudaStream_t stream) { return fwd_read_and_clear_error(stream); }

}  // namespace sa
