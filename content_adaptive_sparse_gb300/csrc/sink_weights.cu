// The attention weight that every key of the sink-window graph gathers, for sm_103a (tcgen05 + TMEM + TMA):
//   w_j = sum over the query heads of j's key head and the queries i >= first that see j of exp(s_ij - LSE_i).
//
// Scores are taken transposed, S^T = K Q^T: a thread has one key and runs along the queries, so a sum needs no
// exchange. LSE belongs to the queries, the columns: it goes into the product as one more step of it, -LSE / scale in
// three bf16 parts (24 bits) against ones, so that a thread only multiplies and takes 2^x. (Read from shared memory
// instead, where 32 lanes get the same four bytes a cycle, it cost as much of its bandwidth as the products' operands
// do: 259 us for two prompts of 8192 tokens where this takes NNN.) A list is 256 keys (two tiles: every tile of
// queries that comes through shared memory then serves twice, 4.7 instead of 9.4 TB/s from L2 at full
// rate) of one (sequence, key head); its steps are the query tiles that see any of them, for every query head.
// Lists are of unequal length (causal, windows, the sinks' keys), so all steps are laid end to end and cut
// evenly between the CTAs; a list that is cut leaves sums in the workspace (at most two per CTA), which a second launch
// adds in their order: the same bits on every run. Where a list begins on that line has a closed form (before()).
//
// Sums: 64 queries a step in four fp32 sums, and the steps' totals with their rounding errors carried along
// (two-term sums), since a key of a long prompt gathers from some 10^5 queries.
//
// Warp roles (640 threads): 0-15 exponentials and sums (key tile w / 4 % 2, queries 64 (w / 8) .. of the step's); 16 loads K and
// Q; 17 issues the products; 18 brings LSE. The two key tiles have barriers of their own, so that a scheduler's four
// warps are at different places of a step.
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
constexpr int kThreads = 640, kSumWarps = 16;
constexpr uint32_t kTmemCols = 512;      // S^T of key tile w in buffer b: 128 columns at 256 b + 128 w

// The products' last step: tiles of 128 rows of 64 bytes (64-byte swizzle). Ones in the first 32 bytes of one, and -LSE / scale
// of four steps in both halves of two.
constexpr int kSide = kTile * 64;

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
  static constexpr int QS = D == 128 ? 3 : 4;          // query tiles in shared memory
  static constexpr int KS = D == 128 ? 3 : 4;          // key tiles: a list's two, and one or two of the next list
  static constexpr int SMEM = 1024 + (KS + QS) * TILE + 3 * kSide;
  static_assert(SMEM <= 222 * 1024, "shared memory");
};

struct WParams {
  int n, heads, kv_heads, group;
  int tiles, pairs;                 // query tiles, lists of a (sequence, key head)
  int first_tile, reach;            // the first query's tile; query tiles past 2 t that keys of list t reach
  int skip;                         // lists below it have no steps, but for the sinks'
  int window, sinks, first;
  int64_t all;                      // steps of one query head of a (sequence, key head)
  int64_t total;                    // steps
  const float* lse;
  float* weights;
  float* partial;                   // [CTA][2][256]
  float scale_log2, inv_scale;
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

// The last list that begins at r or before, found by all lanes of a warp (one comparison after the other took 5 us of
// 64-bit arithmetic).
struct Search {
  __host__ __device__ int operator()(const WParams& p, int64_t r) const {
    int lo = 0, n = p.pairs;        // it is one of n lists from lo on
#ifdef __CUDA_ARCH__
    const int lane = threadIdx.x & 31;
    while (n > 1) {
      const int step = (n + 31) / 32;
      const unsigned ok = __ballot_sync(0xffffffffu, lane * step < n && before(p, lo + lane * step) <= r);
      const int last = 31 - __clz(ok);         // before(lo) <= r: bit 0 is set
      n = n - last * step < step ? n - last * step : step;
      lo += last * step;
    }
#else
    for (; n > 1 && before(p, lo + 1) <= r; --n) ++lo;
#endif
    return lo;
  }
};

// The pieces of lists of CTA c of `ctas`: steps [jb, je) of list t of (sequence, key head) sh.
struct Walk {
  int64_t at, end;                  // on the line of all steps
  int sh, t, i0, count;             // the list's first query tile and number of them
  int64_t list;                     // where it begins
  int jb, je;
  __host__ __device__ static int64_t bound(const WParams& p, int c, int ctas) { return p.total * c / ctas; }
  // (by all lanes of a warp)
  __host__ __device__ Walk(const WParams& p, int c, int ctas) : Walk(p, bound(p, c, ctas), bound(p, c + 1, ctas)) {}
  __host__ __device__ Walk(const WParams& p, int64_t from, int64_t to) : at(from), end(to) {
    sh = t = i0 = count = jb = je = 0;
    list = 0;
    if (at >= end) return;
    const int64_t per = p.all * p.group;
    sh = (int)(at / per);
    const int64_t r = (at - sh * per) / p.group;
    t = Search()(p, r);
    list = sh * per + before(p, t) * p.group;
    set(p);
  }
  __host__ __device__ bool more() const { return at < end; }
  __host__ __device__ int length(const WParams& p) const { return count * p.group; }
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
    list += length(p);              // the next list with steps
    if (++t < p.skip) t = p.skip;
    if (t >= p.pairs) {
      t = p.sinks > 0 ? 0 : p.skip;
      ++sh;
    }
    set(p);
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
  uint64_t k_full[4], k_empty[4];        // key tile x of the CTA's list n: use 2 n + x of the ring
  uint64_t q_full[4], q_empty[4];
  uint64_t s_full[2][2], s_empty[2][2];  // [key tile][buffer]
  uint64_t lse_full[4], lse_empty[4];
  uint64_t drain;
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_suspend(bar, parity, abort_flag, &g_weights_err, kErrTimeout);
}
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  int never = 0;
  mbar_wait(bar, parity, &never, &g_weights_err, kErrTimeout);
}

// ------------------------------------------------------------------ loader (warp 16, one lane)

template <int D>
__device__ void loader(const WParams& p, Walk w, const CUtensorMap* tq, const CUtensorMap* tk, Bars& bars, uint8_t* sK,
                       uint8_t* sQ, volatile int* abort_flag) {
  using C = Cfg<D>;
  int n = 0, g = 0;                  // key and query tiles asked for
  bool ok = true;
  for (; ok && w.more(); w.next(p)) {
    const int s = w.sh / p.kv_heads, hk = w.sh - s * p.kv_heads;
    const auto keys = [&](int x) {
      const int kb = n % C::KS, tok = w.t * kPair + x * kTile;
      if (n >= C::KS && !wait_bar(&bars.k_empty[kb], (uint32_t)(n / C::KS - 1) & 1u, abort_flag)) return false;
      if (tok < p.n) {
        mbar_arrive_expect_tx(&bars.k_full[kb], C::TILE);
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
          tma_load_4d(sK + kb * C::TILE + c * C::CHUNK, tk, &bars.k_full[kb], c * C::CH, hk, tok, s);
      } else {
        mbar_arrive(&bars.k_full[kb]);                 // no such tile
      }
      ++n;
      return true;
    };
    if (!(ok = keys(0))) break;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const int qb = g % C::QS;
      if (g >= C::QS && !(ok = wait_bar(&bars.q_empty[qb], (uint32_t)(g / C::QS - 1) & 1u, abort_flag))) break;
      mbar_arrive_expect_tx(&bars.q_full[qb], C::TILE);
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_4d(sQ + qb * C::TILE + c * C::CHUNK, tq, &bars.q_full[qb], c * C::CH, hk * p.group + st.e, st.i * kTile, s);
      if (j == w.jb && !(ok = keys(1))) {
        ++g;
        break;
      }
    }
  }
  // every copy of this CTA has landed before it may exit
  for (int i = max(0, n - C::KS); i < n; ++i) drain_bar(&bars.k_full[i % C::KS], (uint32_t)(i / C::KS) & 1u);
  for (int i = max(0, g - C::QS); i < g; ++i) drain_bar(&bars.q_full[i % C::QS], (uint32_t)(i / C::QS) & 1u);
}

// Tile of step g's -LSE / scale; it is in its 32-byte half g % 2.
__device__ __forceinline__ int side_slot(int g) { return (1 + (g >> 1 & 1)) * kSide; }

// ------------------------------------------------------------------ products (warp 17, one lane)

template <int D>
__device__ void issuer(const WParams& p, Walk w, Bars& bars, uint8_t* sK, uint8_t* sQ, uint8_t* sSide, uint32_t tmem,
                       volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t side = make_smem_desc(smem_u32(sSide), 16, 512, kSwizzle64B);     // ones; then -LSE / scale
  const uint64_t k0 = make_smem_desc(smem_u32(sK), 16, C::ATOM, C::SWZ);
  const uint64_t q0 = make_smem_desc(smem_u32(sQ), 16, C::ATOM, C::SWZ);
  constexpr uint32_t idesc = make_idesc_bf16(128, 128, 0, 0);
  int n = 0, g = 0;
  bool ok = true;
  for (; ok && w.more(); w.next(p), n += 2) {
    Step st(w);
    for (int j = w.jb; ok && j < w.je; ++j, ++g, st.next(w)) {
      const int qb = g % C::QS, b = g & 1;
      if (!(ok = wait_bar(&bars.q_full[qb], (uint32_t)(g / C::QS) & 1u, abort_flag))) break;
      if (!(ok = wait_bar(&bars.lse_full[g & 3], (uint32_t)(g >> 2) & 1u, abort_flag))) break;
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        const int kb = (n + x) % C::KS;
        if (j == w.jb && !(ok = wait_bar(&bars.k_full[kb], (uint32_t)((n + x) / C::KS) & 1u, abort_flag))) break;
        if (g >= 2 && !(ok = wait_bar(&bars.s_empty[x][b], (uint32_t)(g / 2 - 1) & 1u, abort_flag))) break;
        tc_fence_after();
        if (tile_seen(p, st.i, 2 * w.t + x)) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t at = (uint64_t)((((ks * 16) / C::CH) * C::CHUNK + ((ks * 16) % C::CH) * 2) >> 4);
            mma_bf16_ss(tmem + 256u * b + 128u * x, k0 + (uint64_t)((kb * C::TILE) >> 4) + at,
                        q0 + (uint64_t)((qb * C::TILE) >> 4) + at, idesc, ks > 0 ? 1u : 0u);
          }
          mma_bf16_ss(tmem + 256u * b + 128u * x, side, side + (uint64_t)((side_slot(g) + 32 * (g & 1)) >> 4), idesc, 1u);
        }
        mma_commit(&bars.s_full[x][b]);
      }
      if (ok) {
        mma_commit(&bars.q_empty[qb]);
        mma_commit(&bars.lse_empty[g & 3]);
      }
    }
    if (ok) {
      mma_commit(&bars.k_empty[n % C::KS]);
      mma_commit(&bars.k_empty[(n + 1) % C::KS]);
    }
  }
  // no MMA of this thread is still at work when the CTA frees its TMEM
  mma_commit(&bars.drain);
  drain_bar(&bars.drain, 0);
}

// ------------------------------------------------------------------ -LSE / scale (warp 18)

// Eight bf16 elements of a row of a tile.
__device__ __forceinline__ uint32_t side_unit(uint8_t* side, int row, int unit) {
  return smem_u32(side) + (uint32_t)(64 * row + ((unit ^ ((row >> 1) & 3)) << 4));
}

// A step's 128 numbers are asked for two steps ahead of their use.
__device__ void lse_rows(const WParams& p, Walk w, Bars& bars, uint8_t* sSide, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  const auto ask = [&](const Walk& at, const Step& st, float (&v)[4]) {
    const int s = at.sh / p.kv_heads, hk = at.sh - s * p.kv_heads;
    const float* row = p.lse + ((int64_t)s * p.heads + hk * p.group + st.e) * p.n;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int i = st.i * kTile + 32 * x + lane;
      v[x] = i < p.n ? row[i] * -p.inv_scale : 0.f;
    }
  };
  // the place of the step that is asked for next
  Step st(w);
  int j = w.jb;
  const auto advance = [&] {
    st.next(w);
    if (++j == w.je) {
      w.next(p);
      if (w.more()) {
        st = Step(w);
        j = w.jb;
      }
    }
  };
  float v[3][4];
  int asked = 0;
#pragma unroll
  for (int k = 0; k < 2; ++k)
    if (w.more()) {
      ask(w, st, v[k]);
      advance();
      ++asked;
    }
  for (int g = 0; g < asked; ++g) {
    if (w.more()) {
      ask(w, st, v[2]);
      advance();
      ++asked;
    }
    if (g >= 4 && !__all_sync(0xffffffffu, wait_bar(&bars.lse_empty[g & 3], (uint32_t)(g / 4 - 1) & 1u, abort_flag))) return;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float y = v[0][x];
      float part[3] = {y, 0.f, 0.f};
      const uint32_t top = __float_as_uint(y) & 0x7f800000u;
      if (top != 0x7f800000u) {                        // numbers: y = part 0 + part 1 + part 2
        part[0] = __bfloat162float(__float2bfloat16_rn(y));
        part[1] = __bfloat162float(__float2bfloat16_rn(y - part[0]));
        part[2] = y - part[0] - part[1];
      }
      st_shared_v4(side_unit(sSide + side_slot(g), 32 * x + lane, 2 * (g & 1)), pack_bf16x2(part[0], part[1]),
                   pack_bf16x2(part[2], 0.f), 0u, 0u);
      v[0][x] = v[1][x];
      v[1][x] = v[2][x];
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.lse_full[g & 3]);
  }
}

// ------------------------------------------------------------------ exponentials and sums (warps 0-15)

// Adds 2^(s c) of 32 queries; SOME: of those whose bit in `see` is set.
template <bool SOME>
__device__ __forceinline__ void add_chunk(const uint32_t* v, uint64_t c2, uint32_t see, uint64_t (&sum)[2]) {
#pragma unroll
  for (int i = 0; i < 32; i += 2) {
    float x0, x1;
    f2::unpack(f2::mul(f2::pack(__uint_as_float(v[i]), __uint_as_float(v[i + 1])), c2), x0, x1);
    if (SOME) {
      x0 = (see >> i) & 1u ? x0 : __int_as_float(0xff800000);
      x1 = (see >> (i + 1)) & 1u ? x1 : __int_as_float(0xff800000);
    }
    sum[i >> 1 & 1] = f2::add(sum[i >> 1 & 1], f2::pack(ex2_approx(x0), ex2_approx(x1)));
  }
}

__device__ void sums(const WParams& p, Walk w, Bars& bars, float (*joint)[kPair], uint32_t tmem, volatile int* abort_flag) {
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, x = warp >> 2 & 1, half = warp >> 3;
  const uint32_t ts = tmem + ((uint32_t)(quarter * 32) << 16) + 128u * x + 64u * half;
  const uint64_t c2 = f2::pack(p.scale_log2, p.scale_log2);
  int g = 0;
  for (int n = 0; w.more(); w.next(p), ++n) {
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
      if (!__all_sync(0xffffffffu, wait_bar(&bars.s_full[x][b], parity, abort_flag))) {
        asm volatile("bar.arrive %0, 64;" ::"r"(1 + (warp & 7)) : "memory");    // the other half may wait for this one
        return;
      }
      const int qa = st.i * kTile + 64 * half, qb = qa + 32;
      const bool on0 = qa + 31 >= any_lo && qa <= any_hi, on1 = qb + 31 >= any_lo && qb <= any_hi;
      if ((on0 || on1) && tile_seen(p, st.i, tile)) {
        tc_fence_after();
        const uint32_t at = ts + 256u * b;
        uint64_t sum[2] = {0ull, 0ull};
        const auto chunk = [&](int q, const uint32_t* y) {
          if (q >= all_lo && q + 31 <= all_hi) {
            add_chunk<false>(y, c2, 0u, sum);
          } else {
            const int a = lo - q, z = hi - q;
            const uint32_t upto = z >= 31 ? 0xffffffffu : (z < 0 ? 0u : ((2u << z) - 1u));
            const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : (0xffffffffu << a));
            add_chunk<true>(y, c2, upto & from, sum);
          }
        };
        uint32_t v[32], u[32];
        tmem_ld_x32(on0 ? at : at + 32, v);
        tmem_ld_wait<32>(v);
        if (on0 && on1) {                              // the second 32 arrive under the first
          tmem_ld_x32(at + 32, u);
          chunk(qa, v);
          tmem_ld_wait<32>(u);
          chunk(qb, u);
        } else {
          chunk(on0 ? qa : qb, v);
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
      if (lane == 0) mbar_arrive(&bars.s_empty[x][b]);
    }
    // the two halves of the queries: warps w and w + 8
    const int mine = x * kTile + 32 * quarter + lane;
    if (half == 1) joint[n & 1][mine] = total;
    asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 7)) : "memory");
    if (half == 1) continue;
    total += joint[n & 1][mine];
    if (w.jb == 0 && w.je == w.length(p)) {
      if (key < p.n) p.weights[(int64_t)w.sh * p.n + key] = total;
    } else {
      p.partial[((int64_t)blockIdx.x * 2 + (w.jb == 0 ? 1 : 0)) * kPair + mine] = total;
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
  __shared__ float joint[2][kPair];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0);   // uniform
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      for (int x = 0; x < 2; ++x) {
        mbar_init(&bars.s_full[x][i], 1);
        mbar_init(&bars.s_empty[x][i], kSumWarps / 2);
      }
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&bars.lse_full[i], 1);
      mbar_init(&bars.lse_empty[i], 1);
    }
    for (int i = 0; i < C::KS; ++i) {
      mbar_init(&bars.k_full[i], 1);
      mbar_init(&bars.k_empty[i], 1);
    }
    for (int i = 0; i < C::QS; ++i) {
      mbar_init(&bars.q_full[i], 1);
      mbar_init(&bars.q_empty[i], 1);
    }
    mbar_init(&bars.drain, 1);
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  uint8_t* sK = sbase;
  uint8_t* sQ = sK + C::KS * C::TILE;
  uint8_t* sSide = sQ + C::QS * C::TILE;
  if (threadIdx.x < 3 * kTile) {
    // ones in the first three columns; zeros everywhere else
    const int m = threadIdx.x / kTile, row = threadIdx.x % kTile;
    const uint32_t one = m == 0 ? 0x3f80u : 0u;
    st_shared_v4(side_unit(sSide + m * kSide, row, 0), one | one << 16, one, 0u, 0u);
    for (int u = 1; u < 4; ++u) st_shared_v4(side_unit(sSide + m * kSide, row, u), 0u, 0u, 0u, 0u);
    fence_proxy_async_smem();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  const Walk w(p, (int)blockIdx.x, (int)gridDim.x);
  if (warp < kSumWarps) {
    sums(p, w, bars, joint, tmem, &abort_flag);
  } else if (warp == 16) {
    if (elect_one()) loader<D>(p, w, &tq, &tk, bars, sK, sQ, &abort_flag);
    __syncwarp();
  } else if (warp == 17) {
    if (elect_one()) issuer<D>(p, w, bars, sK, sQ, sSide, tmem, &abort_flag);
    __syncwarp();
  } else if (warp == 18) {
    lse_rows(p, w, bars, sSide, &abort_flag);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 17) {
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
    const Walk w(p, x, x + 1);
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
  const int from = p.sinks > 0 ? 1 : 0, end = p.skip > from ? p.skip : from;
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
  p.skip = p.first_tile > p.reach ? (p.first_tile - p.reach + 1) / 2 : 0;
  p.all = before(p, p.pairs);
  p.total = p.all * p.group * a.kv_heads * a.batch;
  p.lse = a.lse;
  p.weights = a.weights;
  p.partial = static_cast<float*>(a.workspace);
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.inv_scale = 1.f / a.softmax_scale;
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
