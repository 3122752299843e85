// Attention of a batch whose sequences share a prefix, for sm_103a (tcgen05 + TMEM + TMA): query i of a sequence
// sees every row of the prefix and, of its sequence's own tokens, j <= i with i - j <= window.
//
// The prefix is read once for all: the queries of one key head - its G query heads of every token of every
// sequence - are rows of one matrix, row (s n + t) G + e, and a work item is 128 of those rows against a range of
// the prefix's 128-key tiles. A prompt's own keys differ from sequence to sequence, so there an item is 128
// rows t G + e of one sequence. Two plans, whichever a simple count of steps says is cheaper (plan() below):
//   joint    items of all sequences' rows over the prefix, and of each sequence's rows over its own tokens;
//            the partial results (O unnormalised, m, l, in fp32) are joined row by row:
//              M = max m_k,  L = sum l_k 2^(m_k - M),  O = sum O_k 2^(m_k - M) / L,  LSE = M ln 2 + ln L;
//   apart    (long prompts) each sequence's rows over the prefix and its own tokens in one list.
// Few rows leave SMs without work, so a list may be cut into parts, which are joined too. A single token's own
// keys are left to the decoding kernel (sink_decode.cu), which reads them at the copy rate and joins.
//
// The tiles are those of the sink-window forward (half_softmax.cuh), with two differences: rows of Q come
// through cp.async, one row a thread of the epilogue warps (their addresses follow no tensor map), and every row
// has its own interval of visible keys. Warps whose 32 rows are all past the last one only pass
// the barriers.
//
// Measured: the last 8192 tokens of a 64K prompt behind the other 57344, 16 heads of 128 over 4 key heads, window 4095: 2400 to
// 2430 us, 1.69 to 1.67 PFLOP/s, 0.87 of the library product's rate in a burst (2660 to 2730, 0.77, in a long loop, power-capped);
// the tensor pipe is two thirds busy, as in the sink-window forward, with the handshakes of S, P and O between. 32 questions of
// 37 tokens to 16384: 111 us of 82 (148 items of 128 steps on 152 SMs, 0.78 us a step; then one or two own items a CTA, and
// the join, 5 us). 64 tokens behind 32768: 42 us with the decoding launch, of which 19 here, by a CTA's clock in calls that are
// waited for: Q is in after 3.4, the first scores after 4.5 and the second after 6.6 (cold rows and a cold start of every role's
// code), then 0.75 a step (13.5 steps), and 2.3 from the last scores to the results.
//
// Warp roles (512 threads): 0-7 softmax, 8 loader of K and V, 9 S = Q K^T, 10 and 11 O_h += P_h V_h, 12-15 load Q and
// write the results.
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

template <int D>
constexpr int kSmem = 1024 + (2 + 2 * Cfg<D>::STAGES) * Cfg<D>::TILE;

// Rows, lists and parts of a launch. Class 0: rows of all sequences over the prefix. Class 1: rows of one
// sequence over its own tokens, after the prefix where there is no class 0.
struct Layout {
  int batch, n, heads, kv_heads, group;
  int prefix, window;
  int rows, seq_rows;               // of a key head: of all sequences, of one
  int pre_tiles;                    // 128-key tiles of the prefix
  int tiles0, parts0, items0;       // class 0: row tiles of a key head, parts of their lists, items in all
  int tiles1, parts1, items1;       // class 1: row tiles of a sequence and key head, ...
  int row_tiles, slots;             // tiles of `rows`; partial results of a row (0: the items write O and LSE)
  // Partial results lie in blocks of 128 rows of all sequences, `slots` blocks one behind the other: where the
  // first of row r of key head hk has its m and l; the next is 128 places on.
  __device__ int64_t place(int hk, int r) const {
    return (int64_t)(hk * row_tiles + r / kTile) * slots * kTile + r % kTile;
  }
};

struct PParams {
  Layout l;
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                       // [batch][heads][n]
  // O [block][D / 4][128] of four columns each, m (log2 units) and l [block][128]. A warp's 32 rows are neighbours:
  // written row by row they took 2 us.
  float4* part_o;
  float2* part_ml;
  int64_t q_sb, q_sn, q_sh, o_sb, o_sn, o_sh;
  float scale_log2;
};

// A CTA's work: items blockIdx.x, + gridDim.x, ...
struct Item {
  int at;
  bool on;                          // there is such an item
  bool common;                      // class 0
  int s, hk, row0, rows;            // rows row0 .. row0 + rows - 1 of all sequences' (class 0) or of s's
  int pre, begin, steps, own;       // prefix tiles of the whole list; this part of it; first own tile
  int slot;
  __device__ explicit Item(const PParams& p) : at((int)blockIdx.x) { set(p); }
  __device__ __forceinline__ bool more() const { return on; }
  __device__ __forceinline__ void next(const PParams& p) {
    at += (int)gridDim.x;
    set(p);
  }
  // The row tiles of a key head follow one another, so that CTAs at work share its prefix in L2.
  __device__ void set(const PParams& p) {
    const Layout& l = p.l;
    on = at < l.items0 + l.items1;
    if (!on) return;
    common = at < l.items0;
    const int i = common ? at : at - l.items0, parts = common ? l.parts0 : l.parts1;
    const int tiles = common ? l.tiles0 : l.tiles1;
    const int part = i % parts, j = i / parts, tile = j % tiles;
    hk = j / tiles;
    s = 0;
    if (!common) {
      s = hk % l.batch;
      hk /= l.batch;
    }
    row0 = tile * kTile;
    rows = (common ? l.rows : l.seq_rows) - row0;
    if (rows > kTile) rows = kTile;
    pre = common || l.items0 == 0 ? l.pre_tiles : 0;
    int all = pre;
    own = 0;
    if (!common) {
      const int lo = row0 / l.group - l.window;
      own = (lo > 0 ? lo : 0) / kTile;
      all += (row0 + rows - 1) / l.group / kTile - own + 1;
    }
    begin = (int)((int64_t)all * part / parts);
    steps = (int)((int64_t)all * (part + 1) / parts) - begin;
    slot = common || l.items0 == 0 ? part : l.parts0;
  }
  __device__ bool is_prefix(int j) const { return begin + j < pre; }
  __device__ int key_tile(int j) const { return begin + j < pre ? begin + j : own + begin + j - pre; }
  __device__ __forceinline__ bool one_half(const PParams&, int) const { return false; }
  // Row of a key head's matrix (all sequences) of the item's row r.
  __device__ int row(const PParams& p, int r) const { return (common ? 0 : s * p.l.seq_rows) + row0 + r; }
};

// ------------------------------------------------------------------ loader (warp 8, one lane)

template <int D>
__device__ __forceinline__ bool load_tile(int t, const CUtensorMap* map, uint8_t* ring, uint64_t* full, uint64_t* empty,
                                          int hk, int tok, int s, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int st = t % C::STAGES;
  if (t >= C::STAGES && !wait_bar(&empty[st], (uint32_t)(t / C::STAGES - 1) & 1u, abort_flag)) return false;
  mbar_arrive_expect_tx(&full[st], C::TILE);
#pragma unroll
  for (int c = 0; c < C::NCH; ++c)
    tma_load_4d(ring + st * C::TILE + c * C::CHUNK, map, &full[st], c * C::CH, hk, tok, s);
  return true;
}

template <int D>
__device__ void loader(const PParams& p, const CUtensorMap* kp, const CUtensorMap* vp, const CUtensorMap* ko,
                       const CUtensorMap* vo, Bars& bars, uint8_t* sK, uint8_t* sV, volatile int* abort_flag) {
  using C = Cfg<D>;
  int g = 0, gv = 0;                 // K tiles and V tiles requested
  bool ok = true;
  for (Item it(p); ok && it.more(); it.next(p)) {
    for (int j = 0; j <= it.steps; ++j) {              // V one tile behind K
      if (j < it.steps) {
        const bool pre = it.is_prefix(j);
        if (!(ok = load_tile<D>(g, pre ? kp : ko, sK, bars.k_full, bars.k_empty, it.hk, it.key_tile(j) * kTile,
                                pre ? 0 : it.s, abort_flag)))
          break;
        ++g;
      }
      if (j > 0) {
        const bool pre = it.is_prefix(j - 1);
        if (!(ok = load_tile<D>(gv, pre ? vp : vo, sV, bars.v_full, bars.v_empty, it.hk, it.key_tile(j - 1) * kTile,
                                pre ? 0 : it.s, abort_flag)))
          break;
        ++gv;
      }
    }
  }
  // every copy of this CTA has landed before it may exit
  for (int t = max(0, g - C::STAGES); t < g; ++t) drain_bar(&bars.k_full[t % C::STAGES], (uint32_t)(t / C::STAGES) & 1u);
  for (int t = max(0, gv - C::STAGES); t < gv; ++t) drain_bar(&bars.v_full[t % C::STAGES], (uint32_t)(t / C::STAGES) & 1u);
}

// ------------------------------------------------------------------ softmax (warps 0-7)

// Keys c .. c + 31 in [lo, hi] (bit b: key c + b).
__device__ __forceinline__ uint32_t interval(int lo, int hi, int c) {
  const int a = lo - c, b = hi - c;
  const uint32_t upto = b >= 31 ? 0xffffffffu : (b < 0 ? 0u : ((2u << b) - 1u));
  const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : (0xffffffffu << a));
  return upto & from;
}

template <int D>
__device__ void softmax(const PParams& p, Bars& bars, Handoff* hand, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, half = warp >> 2;
  const int row = quarter * 32 + lane;
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
  Softmax<D> W{bars, abort_flag, base + 64u * half, base + C::COL_O + (uint32_t)(D * half), half, lane, p.scale_log2,
               0.f, 0.f};
  int g = 0, n = 0;
  for (Item it(p); it.more(); it.next(p), ++n) {
    const bool absent = 32 * quarter >= it.rows;
    // the tokens of this thread's row and of the warp's first and last (a row past the last one counts as that)
    const int last = it.rows - 1;
    const int t = (it.row0 + min(row, last)) / p.l.group;
    const int ta = __shfl_sync(0xffffffffu, t, 0), tb = __shfl_sync(0xffffffffu, t, 31);
    W.m = kLowest;
    W.l = 0.f;
    bool later = false;
    for (int j = 0; j < it.steps; ++j, ++g) {
      if (!W.done(bars.s_full, g)) return;
      if (absent) {                                    // whatever P and O hold in these rows is not used
        if (lane == 0) mbar_arrive(&bars.p_full[half][g % C::SB]);
        continue;
      }
      const int k0 = it.key_tile(j) * kTile + kHalf * half;
      // the keys that the warp's rows see: some row those of [any_lo, any_hi], every row those of [all_lo, all_hi]
      int lo = 0, hi = p.l.prefix - 1, any_lo = 0, any_hi = hi, all_lo = 0, all_hi = hi;
      if (!it.is_prefix(j)) {
        lo = t - p.l.window;
        hi = t;
        any_lo = ta - p.l.window;
        any_hi = tb;
        all_lo = tb - p.l.window;
        all_hi = ta;
      }
      tc_fence_after();
      bool ok;
      if (k0 >= all_lo && k0 + 63 <= all_hi) ok = W.template tile<kAll>(g, true, true, 0u, 0u, later);
      else if (k0 + 63 >= any_lo && k0 <= any_hi)
        ok = W.template tile<kSome>(g, k0 + 31 >= any_lo && k0 <= any_hi, k0 + 63 >= any_lo && k0 + 32 <= any_hi,
                                    interval(lo, hi, k0), interval(lo, hi, k0 + 32), later);
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

// ------------------------------------------------------------------ Q and the results (warps 12-15)

// Copies this warp's 32 rows of the item's Q into buffer `dst` in the layout of the swizzled TMA boxes (zeros for
// rows past the last one). D / 8 lanes take a row together (a row a lane: 3.5 us, of a cold Q).
template <int D>
__device__ __forceinline__ void load_q(const PParams& p, const Item& it, int quarter, int lane, uint8_t* dst) {
  using C = Cfg<D>;
  constexpr int kLanes = D / 8;
  const bool mine = 32 * quarter + lane < it.rows;
  const int r = it.row(p, mine ? 32 * quarter + lane : 0);
  const int tok = r / p.l.group, e = r - tok * p.l.group, s = tok / p.l.n, t = tok - s * p.l.n;
  const int64_t at = s * p.q_sb + t * p.q_sn + (int64_t)(it.hk * p.l.group + e) * p.q_sh;
  const int u = lane % kLanes, c = u / (C::CH / 8), v = u % (C::CH / 8);
  const uint32_t to = smem_u32(dst) + (uint32_t)(c * C::CHUNK);
#pragma unroll
  for (int k = 0; k < kLanes; ++k) {
    const int from = k * (32 / kLanes) + lane / kLanes, row = 32 * quarter + from;
    const int64_t off = __shfl_sync(0xffffffffu, at, from);
    const uint32_t x = C::ROWB == 128 ? (uint32_t)(row & 7) : (uint32_t)((row >> 1) & 3);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to + (uint32_t)(row * C::ROWB) + (((uint32_t)v ^ x) << 4)),
                 "l"(p.q + off + 8 * u), "r"(row < it.rows ? 16 : 0)
                 : "memory");
  }
}

template <int D>
__device__ void epilogue(const PParams& p, Bars& bars, const Handoff* hand, uint8_t* sQ, uint32_t tmem,
                         volatile int* abort_flag) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;
  const float kNegInf = __int_as_float(0xff800000);
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
  const auto queries = [&](const Item& it, int n) {
    if (!it.more()) return true;
    if (n >= 2 && !__all_sync(0xffffffffu, wait_bar(&bars.q_empty[n & 1], (uint32_t)(n / 2 - 1) & 1u, abort_flag))) return false;
    load_q<D>(p, it, quarter, lane, sQ + (n & 1) * C::TILE);
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.q_full[n & 1]);
    return true;
  };
  int n = 0;
  Item ahead(p);
  if (!queries(ahead, 0)) return;
  for (Item it(p); it.more(); it.next(p), ++n) {
    ahead.next(p);
    if (!queries(ahead, n + 1)) return;                // under this item's products
    const int e = n & 1;
    if (!__all_sync(0xffffffffu, wait_bar(&bars.epi_full[e], (uint32_t)(n >> 1) & 1u, abort_flag))) return;
    const float m0 = hand[e].m[0][row], m1 = hand[e].m[1][row], l0 = hand[e].l[0][row], l1 = hand[e].l[1][row];
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.epi_empty[e]);
    const float m = fmaxf(m0, m1);
    float f0 = ex2_approx(m0 - m), f1 = ex2_approx(m1 - m);
    const float L = l0 * f0 + l1 * f1;
    const bool on = row < it.rows;
    const int r = it.row(p, on ? row : 0);
    const int64_t at = p.l.place(it.hk, r) + (int64_t)it.slot * kTile;
    __nv_bfloat16* o = nullptr;
    if (p.l.slots == 0) {
      const float inv = L == 0.f ? 0.f : 1.f / L;
      f0 *= inv;
      f1 *= inv;
      const int tok = r / p.l.group, h = it.hk * p.l.group + r - tok * p.l.group, s = tok / p.l.n, t = tok - s * p.l.n;
      o = p.o + s * p.o_sb + t * p.o_sn + (int64_t)h * p.o_sh;
      if (on)
        p.lse[((int64_t)s * p.l.heads + h) * p.l.n + t] = L == 0.f ? kNegInf : (m + __log2f(L)) * 0.69314718055994531f;
    } else if (on) {
      p.part_ml[at] = make_float2(m, L);
    }
    if (!__all_sync(0xffffffffu, wait_bar(&bars.o_full, (uint32_t)n & 1u, abort_flag))) return;
    tc_fence_after();
    const uint32_t t0 = base + C::COL_O, t1 = t0 + D;
    float4* part = p.part_o + at / kTile * (D / 4) * kTile + at % kTile;
#pragma unroll 1
    for (int c = 0; c < D; c += 16) {
      uint32_t a[16], b[16];
      tmem_ld_x16(t0 + c, a);
      tmem_ld_x16(t1 + c, b);
      tmem_ld_wait<16>(a);
      tmem_ld_wait<16>(b);
      float v[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) v[j] = __uint_as_float(a[j]) * f0 + __uint_as_float(b[j]) * f1;
      if (!on) continue;
      if (p.l.slots == 0) {
#pragma unroll
        for (int j = 0; j < 16; j += 8)
          *reinterpret_cast<uint4*>(o + c + j) =
              make_uint4(pack_bf16x2(v[j], v[j + 1]), pack_bf16x2(v[j + 2], v[j + 3]), pack_bf16x2(v[j + 4], v[j + 5]),
                         pack_bf16x2(v[j + 6], v[j + 7]));
      } else {
#pragma unroll
        for (int j = 0; j < 16; j += 4) part[(c + j) / 4 * kTile] = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
      }
    }
    // the accumulators have been read: the next item's PVs may start
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.o_free);
  }
}

// ------------------------------------------------------------------ kernels

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    prefix_fwd_kernel(const __grid_constant__ CUtensorMap kp, const __grid_constant__ CUtensorMap vp,
                      const __grid_constant__ CUtensorMap ko, const __grid_constant__ CUtensorMap vo,
                      const __grid_constant__ PParams p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ Handoff hand[2];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // uniform
  // the joining launch may take its place as CTAs leave; it waits for the whole of this one before it joins
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.q_full[i], kEpilogueWarps);
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
  // The register split's sum is the launch's allocation (checked on the host), so the growth
  // always completes.
  if (warp < 8) {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 184;" ::: "memory");
    softmax<D>(p, bars, hand, tmem, &abort_flag);
  } else {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 72;" ::: "memory");
    if (warp == 8) {
      if (elect_one()) loader<D>(p, &kp, &vp, &ko, &vo, bars, sK, sV, &abort_flag);
      __syncwarp();
    } else if (warp == 9) {
      if (elect_one()) qk_issuer<D, Item>(p, bars, sQ, sK, tmem, &abort_flag);
      __syncwarp();
    } else if (warp < 12) {
      if (elect_one()) pv_issuer<D, Item>(p, warp - 10, bars, sV, tmem, &abort_flag);
      __syncwarp();
    } else {
      epilogue<D>(p, bars, hand, sQ, tmem, &abort_flag);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// Joins the partial results of 32 rows of a key head: a lane has a row, a warp every eighth four columns. Rows leave
// through shared memory, so that they are written in runs.
template <int D>
__global__ void __launch_bounds__(256) prefix_join_kernel(const __grid_constant__ PParams p) {
  constexpr int kWarps = 8, kCols = D / 4 / kWarps;        // groups of four columns of a warp
  __shared__ uint2 out[32][D / 4 + 1];
  __shared__ int64_t place[32];
  const float kNegInf = __int_as_float(0xff800000);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hk = blockIdx.y;
  const int r = min((int)blockIdx.x * 32 + lane, p.l.rows - 1);
  const int tok = r / p.l.group, h = hk * p.l.group + r - tok * p.l.group, s = tok / p.l.n, t = tok - s * p.l.n;
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const float2* ml = p.part_ml + p.l.place(hk, r);
  const float4* part = p.part_o + (p.l.place(hk, r) / kTile * (D / 4)) * kTile + r % kTile;
  const int parts = p.l.slots;
  float M = kLowest, L = 0.f;
#pragma unroll 8
  for (int k = 0; k < parts; ++k) M = fmaxf(M, ml[k * kTile].x);
  float4 v[kCols];
#pragma unroll
  for (int c = 0; c < kCols; ++c) v[c] = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 2
  for (int k = 0; k < parts; ++k) {
    const float2 e = ml[k * kTile];
    const float a = ex2_approx(e.x - M);
    L = fmaf(a, e.y, L);
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const float4 x = part[((int64_t)k * (D / 4) + warp + kWarps * c) * kTile];
      v[c].x = fmaf(a, x.x, v[c].x);
      v[c].y = fmaf(a, x.y, v[c].y);
      v[c].z = fmaf(a, x.z, v[c].z);
      v[c].w = fmaf(a, x.w, v[c].w);
    }
  }
  const float inv = L == 0.f ? 0.f : 1.f / L;
#pragma unroll
  for (int c = 0; c < kCols; ++c)
    out[lane][warp + kWarps * c] = make_uint2(pack_bf16x2(v[c].x * inv, v[c].y * inv), pack_bf16x2(v[c].z * inv, v[c].w * inv));
  if (warp == 0) {
    place[lane] = s * p.o_sb + t * p.o_sn + (int64_t)h * p.o_sh;
    if ((int)blockIdx.x * 32 + lane < p.l.rows)
      p.lse[((int64_t)s * p.l.heads + h) * p.l.n + t] = L == 0.f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * (D / 4); i += 256) {
    const int row = i / (D / 4), c = i % (D / 4);
    if ((int)blockIdx.x * 32 + row < p.l.rows) *reinterpret_cast<uint2*>(p.o + place[row] + 4 * c) = out[row][c];
  }
}

// ------------------------------------------------------------------ host

constexpr int kPlanSms = 152;        // a plan must not depend on the device that asks for its workspace

// Rounds of 152 CTAs times an item's steps; an item's start and end cost about three steps (2.3 us). What a CTA's first item costs
// besides, since everything is cold, comes once in every plan.
double cost(int64_t items, double steps) {
  return (double)((items + kPlanSms - 1) / kPlanSms) * (steps + 3.0);
}

// Parts, at most `most`, of each of `lists` lists of `steps` tiles. A part more costs its partial results' way
// to memory and back, about an eighth of a step per row tile and SM.
int parts_of(int64_t lists, double steps, int most) {
  int best = 1;
  double least = cost(lists, steps);
  for (int p = 2; p <= most && lists * p <= 4 * kPlanSms; ++p) {
    const double c = cost(lists * p, steps / p) + 1.0 + 0.125 * (double)(lists * p) / kPlanSms;
    if (c < least) {
      least = c;
      best = p;
    }
  }
  return best;
}

int ceil_div(int64_t a, int64_t b) { return (int)((a + b - 1) / b); }

Layout plan(int batch, int n, int prefix, int heads, int kv_heads, int window, bool decode) {
  Layout l;
  memset(&l, 0, sizeof(l));
  l.batch = batch;
  l.n = n;
  l.heads = heads;
  l.kv_heads = kv_heads;
  l.group = heads / kv_heads;
  l.prefix = prefix;
  l.window = window;
  l.seq_rows = n * l.group;
  l.rows = batch * l.seq_rows;
  l.pre_tiles = ceil_div(prefix, kTile);
  const int joint_tiles = l.row_tiles = ceil_div(l.rows, kTile), seq_tiles = ceil_div(l.seq_rows, kTile);
  const int64_t joint_lists = (int64_t)joint_tiles * kv_heads, seq_lists = (int64_t)batch * seq_tiles * kv_heads;
  // own tiles of a row tile, on average
  const double span = window + (double)kTile / l.group;
  const double own = 1.0 + (span < n / 2.0 ? span : n / 2.0) / kTile;
  const int joint_parts = prefix > 0 ? parts_of(joint_lists, l.pre_tiles, l.pre_tiles < 256 ? l.pre_tiles : 256) : 0;
  const double joint = cost(joint_lists * joint_parts, (double)l.pre_tiles / (joint_parts > 0 ? joint_parts : 1)) +
                       (decode ? 0.0 : cost(seq_lists, own) + 4.0);
  const int apart_parts = parts_of(seq_lists, l.pre_tiles + own, l.pre_tiles < 64 ? l.pre_tiles + 1 : 64);
  const double apart = cost(seq_lists * apart_parts, (l.pre_tiles + own) / apart_parts);
  if (decode || (prefix > 0 && joint < apart)) {
    l.tiles0 = joint_tiles;
    l.parts0 = joint_parts;
    l.items0 = (int)(joint_lists * joint_parts);
    l.parts1 = 1;
    l.slots = joint_parts;
    if (!decode) {
      l.tiles1 = seq_tiles;
      l.items1 = (int)seq_lists;
      l.slots += 1;
    }
  } else {
    l.parts0 = 1;
    l.tiles1 = seq_tiles;
    l.parts1 = apart_parts;
    l.items1 = (int)(seq_lists * apart_parts);
    l.slots = apart_parts > 1 ? apart_parts : 0;
  }
  return l;
}

size_t partial_rows(const Layout& l) { return (size_t)l.kv_heads * l.row_tiles * l.slots * kTile; }

template <int D>
int launch_d(const PrefixArgs& a, const Layout& l, cudaStream_t stream) {
  using C = Cfg<D>;
  CUtensorMap kp, vp, ko, vo;
  memset(&kp, 0, sizeof(kp));
  memset(&vp, 0, sizeof(vp));
  memset(&ko, 0, sizeof(ko));
  memset(&vo, 0, sizeof(vo));
  const auto map = [&](CUtensorMap* m, const void* base, int batch, int tokens, const int64_t st[3]) {
    return encode_bhnd_map(m, base, batch, tokens, a.kv_heads, D, st[0], st[1], st[2], C::CH, kTile, C::TMA_SWZ);
  };
  if (a.prefix > 0 &&
      (!map(&kp, a.k_prefix, 1, a.prefix, a.k_prefix_strides) || !map(&vp, a.v_prefix, 1, a.prefix, a.v_prefix_strides)))
    return SA_ERR_UNSUPPORTED;
  if (l.items1 > 0 &&
      (!map(&ko, a.k, a.batch, a.n_tokens, a.k_strides) || !map(&vo, a.v, a.batch, a.n_tokens, a.v_strides)))
    return SA_ERR_UNSUPPORTED;
  PParams p;
  memset(&p, 0, sizeof(p));
  p.l = l;
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.part_ml = static_cast<float2*>(a.workspace);
  p.part_o = reinterpret_cast<float4*>(static_cast<uint8_t*>(a.workspace) + partial_rows(l) * sizeof(float2));
  p.q_sb = a.q_strides[0];
  p.q_sn = a.q_strides[1];
  p.q_sh = a.q_strides[2];
  p.o_sb = a.o_strides[0];
  p.o_sn = a.o_strides[1];
  p.o_sh = a.o_strides[2];
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  const auto kern = prefix_fwd_kernel<D>;
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kern) != cudaSuccess) return SA_ERR_CUDA;
  if (fa.numRegs != kLaunchRegs) return SA_ERR_UNSUPPORTED;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem<D>) != cudaSuccess) return SA_ERR_CUDA;
  const int items = l.items0 + l.items1, sm_count = current_sm_count();
  kern<<<items < sm_count ? items : sm_count, kThreads, kSmem<D>, stream>>>(kp, vp, ko, vo, p);
  if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
  if (l.slots == 0 || a.decode) return SA_OK;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)((l.rows + 31) / 32), (unsigned)l.kv_heads);
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, prefix_join_kernel<D>, p) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

PrefixWorkspace prefix_workspace(int batch, int n_tokens, int prefix, int heads, int kv_heads, int head_dim, int window,
                                 bool decode) {
  const Layout l = plan(batch, n_tokens, prefix, heads, kv_heads, window, decode);
  PrefixWorkspace w;
  w.parts = l.slots;
  w.tiles = l.row_tiles;
  w.part_o_off = partial_rows(l) * sizeof(float2);
  w.bytes = w.part_o_off + partial_rows(l) * head_dim * sizeof(float);
  if (w.bytes < 256) w.bytes = 256;
  return w;
}

int launch_prefix_attn(const PrefixArgs& a, cudaStream_t stream) {
  const Layout l = plan(a.batch, a.n_tokens, a.prefix, a.heads, a.kv_heads, a.window, a.decode);
  switch (a.head_dim) {
    case 32: return launch_d<32>(a, l, stream);
    case 64: return launch_d<64>(a, l, stream);
    case 128: return launch_d<128>(a, l, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int prefix_read_and_clear_error(cudaStream_t stream) { return fwd_read_and_clear_error(stream); }

}  // namespace sa
