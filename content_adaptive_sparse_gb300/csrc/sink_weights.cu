// The attention weight that every key of the sink-window graph gathers, for sm_103a (tcgen05 + TMEM + TMA):
//   w_j = sum over the query heads of j's key head and the queries i >= first that see j of exp(s_ij - LSE_i).
//
// Scores are taken transposed, S^T = K Q^T: a thread has one key and runs along the queries, so a sum needs no
// exchange, and LSE comes by query from shared memory. A list is 256 keys (two tiles: every tile of
// queries that comes through shared memory then serves twice, 4.7 instead of 9.4 TB/s from L2 at full
// rate) of one (sequence, key head); its steps are the query tiles that see any of them, for every query head.
// Lists are of unequal length (causal, windows, the sinks' keys), so all steps are laid end to end and cut
// evenly between the CTAs; a list that is cut leaves sums in the workspace (at most two per CTA), which a second launch
// adds in their order: the same bits on every run. Where a list begins on that line has a closed form (before()).
//
// Sums: 128 queries a step in four fp32 sums, and the steps' totals with their rounding errors carried along
// (two-term sums), since a key of a long prompt gathers from some 10^5 queries.
//
// Warp roles (384 threads): 0-7 exponentials and sums, key tile w / 4; 8 loads K and Q; 9 issues the products;
// 10 brings LSE.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "f32x2.cuh"
#include "ptx_sm100.cuh"
#include "sa_internal.h"
#include "tma_host.h"

namespace sa {
namespace {

__device__ unsigned int g_weights_err;

constexpr int kTile = 128, kPair = 256;
constexpr int kThreads = 384;
constexpr uint32_t kTmemCols = 512;      // S^T of key tile w in buffer b: 128 columns at 256 b + 128 w

template <int D>
struct Cfg {
  static constexpr int CH = D >= 64 ? 64 : 32;
  static constexpr int NCH = D / CH;
  static constexpr int ROWB = CH * 2;
  static constexpr uint32_t SWZ = ROWB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr CUtensorMapSwizzle TMA_SWZ =
      ROWB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  static constexpr uint32_t ATOM = 8 * ROWB;
  static constexpr int CHUNK = kTile * ROWB;
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int QS = D == 128 ? 2 : 4;          // query tiles in shared memory
  static constexpr int SMEM = 1024 + (4 + QS) * TILE;  // and two lists' keys
  static_assert(SMEM <= 222 * 1024, "shared memory");
};

struct WParams {
  int n, heads, kv_heads, group;
  int tiles, pairs;                 // query tiles, lists of a (sequence, key head)
  int first_tile, reach;            // the first query's tile; query tiles past 2 t that keys of list t reach
  int window, sinks, first;
  int64_t all;                      // steps of one query head of a (sequence, key head)
  int64_t total;                    // steps
  const float* lse;
  float* weights;
  float* partial;                   // [CTA][2][256]
  float scale_log2;
};

__host__ __device__ inline int64_t clamp64(int64_t x, int64_t lo, int64_t hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Query tiles of list t: first and last (none: last < first).
__host__ __device__ inline void span(const WParams& p, int t, int& i0, int& i1) {
  i0 = 2 * t > p.first_tile ? 2 * t : p.first_tile;
  i1 = p.tiles - 1;
  if (!(t == 0 && p.sinks > 0) && 2 * (int64_t)t + p.reach < i1) i1 = 2 * t + p.reach;
}

// Query tiles of the lists before list t, were it not for the sinks: for t' >= a, where the spans begin to hold
// tiles, the sum of min(tiles - 1, 2 t' + reach) - max(first_tile, 2 t') + 1.
__host__ __device__ inline int64_t before_without_sinks(const WParams& p, int64_t t) {
  const int64_t f = p.first_tile, r = p.reach, last = p.tiles - 1;
  int64_t a = f > r ? (f - r + 1) / 2 : 0;
  if (a > t) a = t;
  const int64_t x = clamp64(last >= r ? (last - r) / 2 + 1 : 0, a, t);      // min is 2 t' + r below x
  const int64_t y = clamp64(f / 2 + 1, a, t);                               // max is f below y
  return x * (x - 1) - a * (a - 1) + (x - a) * r + (t - x) * last - (y - a) * f - (t * (t - 1) - y * (y - 1)) + (t - a);
}
__host__ __device__ inline int64_t before(const WParams& p, int64_t t) {
  if (t == 0 || p.sinks == 0) return before_without_sinks(p, t);
  int i0, i1;
  span(p, 0, i0, i1);
  return before_without_sinks(p, t) - before_without_sinks(p, 1) + (i1 - i0 + 1);
}

// The pieces of lists of CTA c of `ctas`: steps [jb, je) of list t of (sequence, key head) sh.
struct Walk {
  int64_t at, end;                  // on the line of all steps
  int sh, t, i0, count;             // the list's first query tile and number of them
  int64_t list;                     // where it begins
  int jb, je;
  __host__ __device__ static int64_t bound(const WParams& p, int c, int ctas) { return p.total * c / ctas; }
  __host__ __device__ Walk(const WParams& p, int c, int ctas) {
    at = bound(p, c, ctas);
    end = bound(p, c + 1, ctas);
    find(p);
  }
  __host__ __device__ Walk(const WParams& p, int64_t x) : at(x), end(x + 1) { find(p); }
  __host__ __device__ bool more() const { return at < end; }
  __host__ __device__ int length(const WParams& p) const { return count * p.group; }
  __host__ __device__ void find(const WParams& p) {
    if (at >= end) return;
    const int64_t per = p.all * p.group;
    sh = (int)(at / per);
    const int64_t r = at % per / p.group;
    int lo = 0, hi = p.pairs - 1;   // the last list that begins at r or before
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (before(p, mid) <= r) lo = mid;
      else hi = mid - 1;
    }
    t = lo;
    list = sh * per + before(p, t) * p.group;
    set(p);
  }
  __host__ __device__ void set(const WParams& p) {
    int i1;
    span(p, t, i0, i1);
    count = i1 - i0 + 1;
    jb = (int)(at - list);
    const int64_t rest = end - list;
    je = rest < length(p) ? (int)rest : length(p);
  }
  __host__ __device__ void next(const WParams& p) {
    at = list + je;
    if (at >= end) return;
    // the next list with steps: only (sequence, key head) starts can be without
    list += length(p);
    if (++t < p.pairs) {
      int a, b;
      span(p, t, a, b);
      if (b >= a) {
        set(p);
        return;
      }
    }
    find(p);
  }
};

// Step j of a list: query head of the group and query tile.
struct Step {
  int e, i;
  __host__ __device__ Step(const Walk& w) : e(w.jb / w.count), i(w.i0 + w.jb % w.count) {}
  __host__ __device__ void next(const Walk& w) {
    if (++i == w.i0 + w.count) {
      i = w.i0;
      ++e;
    }
  }
};

// Whether some query of tile i sees some key of tile k.
__host__ __device__ inline bool tile_seen(const WParams& p, int i, int k) {
  return k * kTile < p.n && i >= k && (i * kTile - (k * kTile + kTile - 1) <= p.window || k * kTile < p.sinks);
}

struct Bars {
  uint64_t k_full[2], k_empty[2];
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2], s_empty[2], lse_full[2];
  uint64_t drain;
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_suspend(bar, parity, abort_flag, &g_weights_err, kErrTimeout);
}
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  int never = 0;
  mbar_wait(bar, parity, &never, &g_weights_err, kErrTimeout);
}

// ------------------------------------------------------------------ loader (warp 8, one lane)

template <int D>
__device__ void loader(const WParams& p, const CUtensorMap* tq, const CUtensorMap* tk, Bars& bars, uint8_t* sK, uint8_t* sQ,
                       volatile int* abort_flag) {
  using C = Cfg<D>;
  int n = 0, g = 0;
  bool ok = true;
  for (Walk w(p, blockIdx.x, gridDim.x); ok && w.more(); w.next(p)) {
    const int s = w.sh / p.kv_heads, hk = w.sh % p.kv_heads;
    const int kb = n & 1;
    if (n >= 2 && !(ok = wait_bar(&bars.k_empty[kb], (uint32_t)(n / 2 - 1) & 1u, abort_flag))) break;
    const int boxes = w.t * kPair + kTile < p.n ? 2 : 1;
    mbar_arrive_expect_tx(&bars.k_full[kb], boxes * C::TILE);
    for (int x = 0; x < boxes; ++x)
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_4d(sK + (2 * kb + x) * C::TILE + c * C::CHUNK, tk, &bars.k_full[kb], c * C::CH, hk, w.t * kPair + x * kTile, s);
    ++n;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const int qb = g % C::QS;
      if (g >= C::QS && !(ok = wait_bar(&bars.q_empty[qb], (uint32_t)(g / C::QS - 1) & 1u, abort_flag))) break;
      mbar_arrive_expect_tx(&bars.q_full[qb], C::TILE);
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_4d(sQ + qb * C::TILE + c * C::CHUNK, tq, &bars.q_full[qb], c * C::CH, hk * p.group + st.e, st.i * kTile, s);
    }
  }
  // every copy of this CTA has landed before it may exit
  for (int i = max(0, n - 2); i < n; ++i) drain_bar(&bars.k_full[i & 1], (uint32_t)(i >> 1) & 1u);
  for (int i = max(0, g - C::QS); i < g; ++i) drain_bar(&bars.q_full[i % C::QS], (uint32_t)(i / C::QS) & 1u);
}

// ------------------------------------------------------------------ products (warp 9, one lane)

template <int D>
__device__ void issuer(const WParams& p, Bars& bars, uint8_t* sK, uint8_t* sQ, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t k0 = make_smem_desc(smem_u32(sK), 16, C::ATOM, C::SWZ);
  const uint64_t q0 = make_smem_desc(smem_u32(sQ), 16, C::ATOM, C::SWZ);
  constexpr uint32_t idesc = make_idesc_bf16(128, 128, 0, 0);
  int n = 0, g = 0;
  bool ok = true;
  for (Walk w(p, blockIdx.x, gridDim.x); ok && w.more(); w.next(p), ++n) {
    const int kb = n & 1;
    if (!(ok = wait_bar(&bars.k_full[kb], (uint32_t)(n >> 1) & 1u, abort_flag))) break;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const int qb = g % C::QS, b = g & 1;
      if (!(ok = wait_bar(&bars.q_full[qb], (uint32_t)(g / C::QS) & 1u, abort_flag))) break;
      if (g >= 2 && !(ok = wait_bar(&bars.s_empty[b], (uint32_t)(g / 2 - 1) & 1u, abort_flag))) break;
      tc_fence_after();
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (!tile_seen(p, st.i, 2 * w.t + x)) continue;
#pragma unroll
        for (int ks = 0; ks < D / 16; ++ks) {
          const uint64_t at = (uint64_t)((((ks * 16) / C::CH) * C::CHUNK + ((ks * 16) % C::CH) * 2) >> 4);
          mma_bf16_ss(tmem + 256u * b + 128u * x, k0 + (uint64_t)(((2 * kb + x) * C::TILE) >> 4) + at,
                      q0 + (uint64_t)((qb * C::TILE) >> 4) + at, idesc, ks > 0 ? 1u : 0u);
        }
      }
      mma_commit(&bars.q_empty[qb]);
      mma_commit(&bars.s_full[b]);
    }
    if (ok) mma_commit(&bars.k_empty[kb]);
  }
  // no MMA of this thread is still at work when the CTA frees its TMEM
  mma_commit(&bars.drain);
  drain_bar(&bars.drain, 0);
}

// ------------------------------------------------------------------ -LSE log2(e) (warp 10)

__device__ void lse_rows(const WParams& p, Bars& bars, float (*nl)[kTile], volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  int g = 0;
  for (Walk w(p, blockIdx.x, gridDim.x); w.more(); w.next(p)) {
    const int s = w.sh / p.kv_heads, hk = w.sh % p.kv_heads;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const float* row = p.lse + ((int64_t)s * p.heads + hk * p.group + st.e) * p.n;
      float v[4];
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const int i = st.i * kTile + 32 * x + lane;
        v[x] = i < p.n ? row[i] * -1.4426950408889634f : 0.f;
      }
      if (g >= 2 && !__all_sync(0xffffffffu, wait_bar(&bars.s_empty[g & 1], (uint32_t)(g / 2 - 1) & 1u, abort_flag))) return;
#pragma unroll
      for (int x = 0; x < 4; ++x) nl[g & 1][32 * x + lane] = v[x];
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.lse_full[g & 1]);
    }
  }
}

// ------------------------------------------------------------------ exponentials and sums (warps 0-7)

// Adds 2^(s c + nl) of 32 queries; SOME: of those whose bit in `see` is set.
template <bool SOME>
__device__ __forceinline__ void add_chunk(const uint32_t* v, uint32_t nl, uint64_t c2, uint32_t see, uint64_t (&sum)[2]) {
#pragma unroll
  for (int j = 0; j < 32; j += 4) {
    uint64_t a, b;
    asm volatile("ld.shared.v2.b64 {%0, %1}, [%2];" : "=l"(a), "=l"(b) : "r"(nl + 4u * j));
    float x[4];
    f2::unpack(f2::fma(f2::pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), c2, a), x[0], x[1]);
    f2::unpack(f2::fma(f2::pack(__uint_as_float(v[j + 2]), __uint_as_float(v[j + 3])), c2, b), x[2], x[3]);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (SOME) x[e] = (see >> (j + e)) & 1u ? x[e] : __int_as_float(0xff800000);
      x[e] = ex2_approx(x[e]);
    }
    sum[0] = f2::add(sum[0], f2::pack(x[0], x[1]));
    sum[1] = f2::add(sum[1], f2::pack(x[2], x[3]));
  }
}

__device__ void sums(const WParams& p, Bars& bars, const float (*nl)[kTile], uint32_t tmem, volatile int* abort_flag) {
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, x = warp >> 2;
  const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + 128u * x;
  const uint64_t c2 = f2::pack(p.scale_log2, p.scale_log2);
  int g = 0;
  for (Walk w(p, blockIdx.x, gridDim.x); w.more(); w.next(p)) {
    const int tile = 2 * w.t + x, k0 = tile * kTile + 32 * quarter, key = k0 + lane;
    // queries that see this thread's key, some key of the warp, every key of the warp (keys past the sequence
    // are not written and count with none)
    const int end = p.n - 1;
    const auto last = [&](int k) { return k < p.sinks || p.window >= end - k ? end : k + p.window; };
    const int lo = max(key, p.first), hi = key < p.n ? last(key) : -1;
    const int any_lo = max(k0, p.first), any_hi = k0 < p.sinks ? end : last(min(k0 + 31, end));
    const int all_lo = max(k0 + 31, p.first), all_hi = k0 < p.sinks && k0 + 31 >= p.sinks ? last(p.sinks) : last(k0);
    float total = 0.f, lost = 0.f;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const int b = g & 1;
      const uint32_t parity = (uint32_t)(g >> 1) & 1u;
      if (!__all_sync(0xffffffffu, wait_bar(&bars.s_full[b], parity, abort_flag) && wait_bar(&bars.lse_full[b], parity, abort_flag)))
        return;
      if (tile_seen(p, st.i, tile)) {
        tc_fence_after();
        const int q0 = st.i * kTile;
        const uint32_t row = smem_u32(nl[b]), at = ts + 256u * b;
        uint64_t sum[2] = {0ull, 0ull};
#pragma unroll 1
        for (int c = 0; c < kTile; c += 64) {
          const int qa = q0 + c, qb = qa + 32;
          const bool on0 = qa + 31 >= any_lo && qa <= any_hi, on1 = qb + 31 >= any_lo && qb <= any_hi;
          uint32_t v[64];
          if (on0) tmem_ld_x32(at + c, v);
          if (on1) tmem_ld_x32(at + c + 32, v + 32);
          tmem_ld_wait<64>(v);
          const auto chunk = [&](int q, const uint32_t* y, uint32_t nl_at) {
            if (q >= all_lo && q + 31 <= all_hi) {
              add_chunk<false>(y, nl_at, c2, 0u, sum);
            } else {
              const int a = lo - q, z = hi - q;
              const uint32_t upto = z >= 31 ? 0xffffffffu : (z < 0 ? 0u : ((2u << z) - 1u));
              const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : (0xffffffffu << a));
              add_chunk<true>(y, nl_at, c2, upto & from, sum);
            }
          };
          if (on0) chunk(qa, v, row + 4u * c);
          if (on1) chunk(qb, v + 32, row + 4u * (c + 32));
        }
        float a, z;
        f2::unpack(f2::add(sum[0], sum[1]), a, z);
        // total += a + z, with the rounding error of the sum carried on
        const float y = (a + z) - lost, t = total + y;
        lost = (t - total) - y;
        total = t;
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_empty[b]);
    }
    const bool whole = w.jb == 0 && w.je == w.length(p);
    if (whole) {
      if (key < p.n) p.weights[(int64_t)w.sh * p.n + key] = total;
    } else {
      p.partial[((int64_t)blockIdx.x * 2 + (w.jb == 0 ? 1 : 0)) * kPair + x * kTile + 32 * quarter + lane] = total;
    }
  }
}

// ------------------------------------------------------------------ kernels

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    sink_weights_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                        const __grid_constant__ WParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ __align__(16) float nl[2][kTile];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // uniform
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.s_empty[i], 8);
      mbar_init(&bars.lse_full[i], 1);
    }
    for (int i = 0; i < C::QS; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
    }
    mbar_init(&bars.drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  uint8_t* sK = sbase;
  uint8_t* sQ = sK + 4 * C::TILE;
  if (warp < 8) {
    sums(p, bars, nl, tmem, &abort_flag);
  } else if (warp == 8) {
    if (elect_one()) loader<D>(p, &tq, &tk, bars, sK, sQ, &abort_flag);
    __syncwarp();
  } else if (warp == 9) {
    if (elect_one()) issuer<D>(p, bars, sK, sQ, tmem, &abort_flag);
    __syncwarp();
  } else if (warp == 10) {
    lse_rows(p, bars, nl, &abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Block c: the list that the bound before CTA c cuts, where that is its first cut: CTA c - 1's sums of it, then
// those of CTA c and on. And zeros for the keys of lists without a query.
__global__ void __launch_bounds__(kPair) sink_weights_join_kernel(const __grid_constant__ WParams p, int ctas, int lists,
                                                                  int first_list, int end_list) {
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  if (c > 0 && c < ctas) {
    const int64_t x = Walk::bound(p, c, ctas);
    const Walk w(p, x);
    if (w.list < x && Walk::bound(p, c - 1, ctas) <= w.list) {
      const int64_t end = w.list + w.length(p);
      float sum = p.partial[((int64_t)(c - 1) * 2 + 1) * kPair + threadIdx.x];
      for (int k = c; Walk::bound(p, k, ctas) < end; ++k) sum += p.partial[(int64_t)k * 2 * kPair + threadIdx.x];
      const int key = w.t * kPair + threadIdx.x;
      if (key < p.n) p.weights[(int64_t)w.sh * p.n + key] = sum;
    }
  }
  const int keys = (end_list - first_list) * kPair;
  for (int64_t i = (int64_t)c * kPair + threadIdx.x; i < (int64_t)lists * keys; i += (int64_t)gridDim.x * kPair)
    p.weights[i / keys * p.n + first_list * kPair + i % keys] = 0.f;
}

template <int D>
int launch(const WeightsArgs& a, WParams& p, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap tq, tk;
  if (!encode_bhnd_map(&tq, a.q, a.batch, a.n_tokens, a.heads, D, a.q_strides[0], a.q_strides[1], a.q_strides[2], C::CH,
                       kTile, C::TMA_SWZ) ||
      !encode_bhnd_map(&tk, a.k, a.batch, a.n_tokens, a.kv_heads, D, a.k_strides[0], a.k_strides[1], a.k_strides[2], C::CH,
                       kTile, C::TMA_SWZ))
    return SA_ERR_UNSUPPORTED;
  const auto kern = sink_weights_kernel<D>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess) return SA_ERR_CUDA;
  int64_t ctas = current_sm_count();
  if (ctas > kWeightsMaxCtas) ctas = kWeightsMaxCtas;
  if (ctas > p.total) ctas = p.total;
  kern<<<(unsigned)ctas, kThreads, C::SMEM, stream>>>(tq, tk, p);
  if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
  // lists without a step: those whose window ends before the first query, but for the sinks'
  const int empty = p.first_tile > p.reach ? (p.first_tile - p.reach + 1) / 2 : 0, from = p.sinks > 0 ? 1 : 0;
  const int end = empty > from ? empty : from;
  if (ctas == 1 && end == from) return SA_OK;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)ctas);
  cfg.blockDim = dim3(kPair);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sink_weights_join_kernel, p, (int)ctas, (int)(a.batch * a.kv_heads), from, end) == cudaSuccess
             ? SA_OK
             : SA_ERR_CUDA;
}

}  // namespace

// Sizes, graph and line of steps of a call.
static WParams params(const WeightsArgs& a) {
  WParams p;
  memset(&p, 0, sizeof(p));
  p.n = a.n_tokens;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.tiles = (a.n_tokens + kTile - 1) / kTile;
  p.pairs = (a.n_tokens + kPair - 1) / kPair;
  p.first_tile = a.first_query / kTile;
  p.reach = (int)(((int64_t)a.window + kPair - 1) / kTile);
  p.window = a.window;
  p.sinks = a.sinks;
  p.first = a.first_query;
  p.all = before(p, p.pairs);
  p.total = p.all * p.group * a.kv_heads * a.batch;
  p.lse = a.lse;
  p.weights = a.weights;
  p.partial = static_cast<float*>(a.workspace);
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  return p;
}

int launch_sink_attn_weights(const WeightsArgs& a, cudaStream_t stream) {
  WParams p = params(a);
  switch (a.head_dim) {
    case 32: return launch<32>(a, p, stream);
    case 64: return launch<64>(a, p, stream);
    case 128: return launch<128>(a, p, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int weights_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_weights_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_weights_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
