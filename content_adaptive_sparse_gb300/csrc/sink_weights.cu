// The attention weight that every key of the sink-window graph gathers, for sm_103a (tcgen05 + TMEM + TMA):
//   w_j = sum over the query heads of j's key head and the queries i >= first that see j of exp(s_ij - LSE_i).
//
// Scores are taken transposed, S^T = K Q^T: a thread has one key and runs along the queries, so a sum needs no
// exchange. LSE belongs to the queries, the columns: it goes into the product as one more step of it, -LSE / scale in
// three bf16 parts (24 bits) against ones, so that a thread only multiplies and takes 2^x. (Read from shared memory
// instead, where 32 lanes get the same four bytes a cycle, it cost as much of its bandwidth as the products' operands
// do: 259 us for two prompts of 8192 tokens, 205 so.) A list is 256 keys (two tiles: every tile of
// queries that comes through shared memory then serves twice, 4.7 instead of 9.4 TB/s from L2 at full
// rate) of one (sequence, key head); its steps are the query tiles that see any of them, for every query head.
// Lists are of unequal length (causal, windows, the sinks' keys), so all steps are laid end to end and cut
// evenly between the CTAs; a list that is cut leaves sums in the workspace (at most two per CTA), which a second launch
// adds in their order: the same bits on every run. Where a list begins on that line has a closed form (before()).
//
// Products: the keys are the A operand in TMEM, copied there by the summing warps once a list, so that shared memory is
// read for the queries alone (with both operands in it, its bandwidth bound the products: 205 -> 188 us). Three
// buffers of S^T take turns.
//
// Measured: two prompts of 8192 tokens, 16 heads of 128 over 4 key heads, all queries: 190 us, 1.46 PFLOP/s
// (277 GFLOP of visible scores; 210 us in a long loop, power-capped),
// the tensor pipe 72 % busy, the exponentials' 64 %; a step's two products, its sums and the hand-overs between them
// are each near its 1600 cycles. With heads of 64 and 32, where LSE's step is a quarter and a half of the product, 167 and 162 us: there
// the exponentials and hand-overs bound it, not the products. The last 64 queries of 32768: 19 us for 34 MB of keys (18 with
// heads of 64 and 32): 4 us until the first
// scores, 13.5 steps a CTA with a new list every fourth, and the joining launch.
//
// Sums: 64 queries a step in four fp32 sums, and the steps' totals with their rounding errors carried along
// (two-term sums), since a key of a long prompt gathers from some 10^5 queries.
//
// Warp roles (640 threads): 0-15 exponentials and sums (key tile w / 4 % 2, queries 64 (w / 8) .. of the step's); 16 loads K and
// Q; 17 issues the products; 18 and 19 bring LSE. The two key tiles have barriers of their own, so that a scheduler's four
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
// TMEM: three buffers of S^T, 128 columns each, for the products in turn (step g, key tile x: product 2 g + x); then the list's
// two key tiles.
constexpr uint32_t kTmemCols = 512, kColK = 384;
constexpr int kStages = 4;               // query tiles, and numbers -LSE / scale, in shared memory

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
  static constexpr int SMEM = 1024 + (2 + kStages) * TILE + 3 * kSide;   // two key tiles on their way to TMEM
  static_assert(SMEM <= 222 * 1024, "shared memory");
};

struct WParams {
  int n, heads, kv_heads, group;
  int tiles, pairs;                 // query tiles, lists of a (sequence, key head)
  // Query tile i is queries 128 i + shift .., -128 < shift <= 0, so that the first one begins with the first query (the
  // last 64 queries of a prompt are half a tile, not two halves).
  int shift;
  int first_tile, reach;            // the first query's tile; query tiles past 2 t that keys of list t reach
  int skip;                         // lists below it have no steps, but for the sinks'
  int small;                        // all steps are fewer than 2^31
  int window, sinks, first;
  int64_t all;                      // steps of one query head of a (sequence, key head)
  int64_t total;                    // steps: `quota` a CTA, and one more for the first `rest`
  int64_t quota;
  int rest;
  const float* lse;
  float* weights;
  float* partial;                   // [CTA][2][256]
  float scale_log2, inv_scale;
};

__host__ __device__ inline int clamp(int x, int lo, int hi) { return x < lo ? lo : (x > hi ? hi : x); }

// Query tiles of list t: first and last (none: last < first).
__host__ __device__ inline void span(const WParams& p, int t, int& i0, int& i1) {
  i0 = 2 * t > p.first_tile ? 2 * t : p.first_tile;
  i1 = p.tiles - 1;
  if (!(t == 0 && p.sinks > 0) && 2 * (int64_t)t + p.reach < i1) i1 = 2 * t + p.reach;
}

// Query tiles of the lists before list t, were it not for the sinks: for t' >= a, where the spans begin to hold
// tiles, the sum of min(tiles - 1, 2 t' + reach) - max(first_tile, 2 t') + 1. Modulo 2^32 with N = uint32_t, which is enough
// where the steps of all lists are fewer (64-bit products are long chains, and every CTA begins with them).
template <class N>
__host__ __device__ inline N before_without_sinks(const WParams& p, int t) {
  const int f = p.first_tile, r = p.reach, last = p.tiles - 1;
  const int a = p.skip < t ? p.skip : t;
  const int x = clamp(last >= r ? (last - r) / 2 + 1 : 0, a, t);      // min is 2 t' + r below x
  const int y = clamp(f / 2 + 1, a, t);                               // max is f below y
  const N A = a, X = x, Y = y, T = t;
  return X * (X - 1) - A * (A - 1) + (X - A) * (N)r + (T - X) * (N)last - (Y - A) * (N)f - (T * (T - 1) - Y * (Y - 1)) + (T - A);
}
template <class N>
__host__ __device__ inline N before_of(const WParams& p, int t) {
  if (t == 0 || p.sinks == 0) return before_without_sinks<N>(p, t);
  int i0, i1;
  span(p, 0, i0, i1);
  return before_without_sinks<N>(p, t) - before_without_sinks<N>(p, 1) + (N)(i1 - i0 + 1);
}
__host__ __device__ inline int64_t before(const WParams& p, int t) {
  return p.small ? (int64_t)before_of<uint32_t>(p, t) : before_of<int64_t>(p, t);
}

// The last list that begins at r or before, found by all lanes of a warp (one comparison after the other took 5 us of
// 64-bit arithmetic).
__device__ __forceinline__ int list_at(const WParams& p, int64_t r) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = p.pairs;          // it is one of n lists from lo on
  while (n > 1) {
    const int step = (n + 31) / 32;
    const unsigned ok = __ballot_sync(0xffffffffu, lane * step < n && before(p, lo + lane * step) <= r);
    const int last = 31 - __clz(ok);           // before(lo) <= r: bit 0 is set
    n = n - last * step < step ? n - last * step : step;
    lo += last * step;
  }
  return lo;
}

// The pieces of lists of CTA c of `ctas`: steps [jb, je) of list t of (sequence, key head) sh.
struct Walk {
  int64_t at, end;                  // on the line of all steps
  int sh, t, i0, count;             // the list's first query tile and number of them
  int64_t list;                     // where it begins
  int jb, je;
  __device__ static int64_t bound(const WParams& p, int c) { return p.quota * c + (c < p.rest ? c : p.rest); }
  // (by all lanes of a warp)
  __device__ Walk(const WParams& p, int c) : Walk(p, bound(p, c), bound(p, c + 1)) {}
  __device__ Walk(const WParams& p, int64_t from, int64_t to) : at(from), end(to) {
    sh = t = i0 = count = jb = je = 0;
    list = 0;
    if (at >= end) return;
    const int64_t per = p.all * p.group;
    int64_t r;
    if (p.small) {                  // divisions of 64 bits are long
      sh = (int)((uint32_t)at / (uint32_t)per);
      r = (uint32_t)(at - sh * per) / (uint32_t)p.group;
    } else {
      sh = (int)(at / per);
      r = (at - sh * per) / p.group;
    }
    t = list_at(p, r);
    list = sh * per + before(p, t) * p.group;
    set(p);
  }
  __device__ bool more() const { return at < end; }
  __device__ int length(const WParams& p) const { return count * p.group; }
  __device__ void set(const WParams& p) {
    int i1;
    span(p, t, i0, i1);
    count = i1 - i0 + 1;
    jb = (int)(at - list);
    const int64_t rest = end - list;
    je = rest < length(p) ? (int)rest : length(p);
  }
  __device__ void next(const WParams& p) {
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
  __device__ Step(const Walk& w) : e(w.jb / w.count), i(w.i0 + w.jb % w.count) {}
  __device__ void next(const Walk& w) {
    if (++i == w.i0 + w.count) {
      i = w.i0;
      ++e;
    }
  }
};

struct Bars {
  uint64_t k_full[2], k_empty[2];        // key tile x of the CTA's list n, phase n: in shared memory; copied from there
  uint64_t kt_full[2];                   // in TMEM
  uint64_t q_full[kStages], q_empty[kStages];   // step g: stage g % 4, phase g / 4
  uint64_t s_full[2][3];                 // key tile x, step g: [x][g % 3], phase g / 3
  uint64_t s_empty[3];                   // product u: buffer u % 3, phase u / 3
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

// Waits for the last copies: of the keys of list n and of the query tiles before g. (A copy that was never asked for ends
// the wait by its limit; that is after a wait that has already run out.)
__device__ void drain(Bars& bars, int n, int g) {
  if (n >= 0)
    for (int x = 0; x < 2; ++x) drain_bar(&bars.k_full[x], (uint32_t)n & 1u);
  for (int i = max(0, g - kStages); i < g; ++i) drain_bar(&bars.q_full[i % kStages], (uint32_t)(i / kStages) & 1u);
}

template <int D>
__device__ void loader(const WParams& p, Walk w, const CUtensorMap* tq, const CUtensorMap* tk, Bars& bars, uint8_t* sK,
                       uint8_t* sQ, volatile int* abort_flag) {
  using C = Cfg<D>;
  int n = 0, g = 0;                  // lists and query tiles asked for
  bool ok = true;
  for (; ok && w.more(); w.next(p), ++n) {
    const int s = w.sh / p.kv_heads, hk = w.sh - s * p.kv_heads;
    for (int x = 0; ok && x < 2; ++x) {
      const int tok = w.t * kPair + x * kTile;
      if (n > 0 && !(ok = wait_bar(&bars.k_empty[x], (uint32_t)(n - 1) & 1u, abort_flag))) break;
      if (tok < p.n) {
        mbar_arrive_expect_tx(&bars.k_full[x], C::TILE);
#pragma unroll
        for (int c = 0; c < C::NCH; ++c)
          tma_load_4d(sK + x * C::TILE + c * C::CHUNK, tk, &bars.k_full[x], c * C::CH, hk, tok, s);
      } else {
        mbar_arrive(&bars.k_full[x]);                  // no such tile
      }
    }
    if (!ok) break;
    Step st(w);
    for (int j = w.jb; j < w.je; ++j, ++g, st.next(w)) {
      const int qb = g % kStages;
      if (g >= kStages && !(ok = wait_bar(&bars.q_empty[qb], (uint32_t)(g / kStages - 1) & 1u, abort_flag))) break;
      mbar_arrive_expect_tx(&bars.q_full[qb], C::TILE);
#pragma unroll
      for (int c = 0; c < C::NCH; ++c)
        tma_load_4d(sQ + qb * C::TILE + c * C::CHUNK, tq, &bars.q_full[qb], c * C::CH, hk * p.group + st.e, st.i * kTile + p.shift, s);
    }
  }
  // every copy of this CTA has landed before it may exit
  drain(bars, n - 1, g);
  if (!ok) drain(bars, n, 0);
}

// Tile of step g's -LSE / scale; it is in its 32-byte half g % 2.
__device__ __forceinline__ int side_slot(int g) { return (1 + (g >> 1 & 1)) * kSide; }

// ------------------------------------------------------------------ products (warp 17, one lane)

// One thread for both tiles, so that their products, and with them the summing warps, stay half a step apart (with
// a thread for each: 189 -> 212 us). Its instructions are the longest chain of a step, so counters take the
// place of divisions and what a list fixes is worked out once.
template <int D>
__device__ void issuer(const WParams& p, Walk w, Bars& bars, uint8_t* sQ, uint8_t* sSide, uint32_t tmem,
                       volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t ones = make_smem_desc(smem_u32(sSide), 16, 512, kSwizzle64B);
  const uint64_t q0 = make_smem_desc(smem_u32(sQ), 16, C::ATOM, C::SWZ);
  uint32_t g = 0;                    // step
  uint32_t r = 0, buf = 0, used = 0; // g % 3; of the next product: its buffer, and whether that was in use, with the phase
  bool ok = true;
  for (int n = 0; ok && w.more(); w.next(p), ++n) {
    int i0[2], i1[2];                // query tiles that see some of a tile's keys
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int k = 2 * w.t + x;
      i0[x] = k;
      i1[x] = k * kTile < p.sinks ? p.tiles - 1 : (int)(((int64_t)k * kTile + kTile - 1 + p.window - p.shift) / kTile);
      if (k * kTile >= p.n) i1[x] = -1;
      ok = ok && wait_bar(&bars.kt_full[x], (uint32_t)n & 1u, abort_flag);
    }
    int i = w.i0 + w.jb % w.count;
    const int i_end = w.i0 + w.count;
    for (int j = w.jb; ok && j < w.je; ++j, ++g) {
      const uint32_t qb = g % kStages;
      if (!(ok = wait_bar(&bars.q_full[qb], g / kStages & 1u, abort_flag))) break;
      const uint64_t q = q0 + (uint64_t)(qb * (uint32_t)(C::TILE >> 4));
      // the last tile may hold no more than half its queries
      const uint32_t idesc = make_idesc_bf16(128, p.n - i * kTile - p.shift > kTile / 2 ? kTile : kTile / 2, 0, 0);
      const uint64_t side = ones + (uint64_t)((side_slot(g) + 32 * (g & 1)) >> 4);
#pragma unroll
      for (int x = 0; x < 2; ++x) {
        if (used > 0 && !(ok = wait_bar(&bars.s_empty[buf], (used - 1) & 1u, abort_flag))) break;
        tc_fence_after();
        if (i >= i0[x] && i <= i1[x]) {
          const uint32_t s = tmem + 128u * buf, keys = tmem + kColK + (uint32_t)(D / 2) * x;
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            constexpr int kPer = C::CH / 16;
            mma_bf16_ts(s, keys + 8u * ks, q + (uint64_t)(((ks / kPer) * C::CHUNK + (ks % kPer) * 32) >> 4), idesc,
                        ks > 0 ? 1u : 0u);
          }
          mma_bf16_ss(s, ones, side, idesc, 1u);
        }
        mma_commit(&bars.s_full[x][r]);
        if (++buf == 3) {
          buf = 0;
          ++used;
        }
      }
      if (ok) mma_commit(&bars.q_empty[qb]);
      r = r == 2 ? 0 : r + 1;
      if (++i == i_end) i = w.i0;
    }
  }
  // no MMA of this thread is still at work when the CTA frees its TMEM
  mma_commit(&bars.drain);
  drain_bar(&bars.drain, 0);
}

// ------------------------------------------------------------------ -LSE / scale (warps 18, 19)

// Eight bf16 elements of a row of a tile.
__device__ __forceinline__ uint32_t side_unit(uint8_t* side, int row, int unit) {
  return smem_u32(side) + (uint32_t)(64 * row + ((unit ^ ((row >> 1) & 3)) << 4));
}

// Every second step from `which` on (one warp for all was the longest chain of a step). A step's 128 numbers are asked
// for while those of the warp's step before are split.
__device__ void lse_rows(const WParams& p, Walk w, int which, Bars& bars, uint8_t* sSide, volatile int* abort_flag) {
  const int lane = threadIdx.x & 31;
  // the place of the step that is asked for next
  int j = w.jb, i = w.i0 + w.jb % w.count;
  const float* row = nullptr;
  const auto head = [&] {
    const int s = w.sh / p.kv_heads, hk = w.sh - s * p.kv_heads;
    row = p.lse + ((int64_t)s * p.heads + hk * p.group + j / w.count) * p.n;
  };
  const auto advance = [&] {
    if (++i == w.i0 + w.count) {
      i = w.i0;
      row += p.n;
    }
    if (++j < w.je) return;
    w.next(p);
    if (!w.more()) return;
    j = w.jb;
    i = w.i0 + w.jb % w.count;
    head();
  };
  const auto ask = [&](float (&v)[4]) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const int q = i * kTile + p.shift + 32 * x + lane;
      v[x] = q < p.n ? row[q] : 0.f;
    }
    advance();
    if (w.more()) advance();
  };
  head();
  if (which == 1) advance();
  float v[4], ahead[4];
  bool on = w.more();
  if (on) ask(v);
  for (int g = which; on; g += 2) {
    const bool more = w.more();
    if (more) ask(ahead);
    if (g >= kStages && !__all_sync(0xffffffffu, wait_bar(&bars.q_empty[g % kStages], (uint32_t)(g / kStages - 1) & 1u, abort_flag)))
      return;
    uint8_t* tile = sSide + side_slot(g);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      float y = v[x] * -p.inv_scale;
      // for LSE = -inf the largest number: with it scores of -inf, the forward's reason for that LSE, stay so
      if (y == __int_as_float(0x7f800000)) y = __int_as_float(0x7f7fffff);
      float part[3] = {y, 0.f, 0.f};
      const uint32_t top = __float_as_uint(y) & 0x7f800000u;
      if (top != 0x7f800000u) {                        // numbers: y = part 0 + part 1 + part 2
        part[0] = __bfloat162float(__float2bfloat16_rz(y));    // towards 0: the largest numbers have to stay numbers
        part[1] = __bfloat162float(__float2bfloat16_rn(y - part[0]));
        part[2] = y - part[0] - part[1];
      }
      st_shared_v4(side_unit(tile, 32 * x + lane, 2 * (g & 1)), pack_bf16x2(part[0], part[1]), pack_bf16x2(part[2], 0.f), 0u, 0u);
      v[x] = ahead[x];
    }
    fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.q_full[g % kStages]);
    on = more;
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

// This warp's 32 rows of a key tile in shared memory, half of their elements, into TMEM as the products' A operand.
template <int D>
__device__ __forceinline__ void keys_to_tmem(const uint8_t* tile, int quarter, int half, int lane, uint32_t to) {
  using C = Cfg<D>;
  constexpr int kUnits = D / 16;       // 16-byte units of half a row
  const int row = 32 * quarter + lane;
  uint32_t v[4 * kUnits];
#pragma unroll
  for (int k = 0; k < kUnits; ++k) {
    const int unit = kUnits * half + k, c = unit / (C::CH / 8), u = unit % (C::CH / 8);
    const int x = C::ROWB == 128 ? row & 7 : (row >> 1) & 3;
    const uint32_t at = smem_u32(tile) + (uint32_t)(c * C::CHUNK + row * C::ROWB + ((u ^ x) << 4));
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v[4 * k]), "=r"(v[4 * k + 1]), "=r"(v[4 * k + 2]), "=r"(v[4 * k + 3])
                 : "r"(at));
  }
  if constexpr (D == 128) tmem_st_x32(to + 32 * half, v);
  else if constexpr (D == 64) tmem_st_x16(to + 16 * half, v);
  else tmem_st_x8(to + 8 * half, v);
  tmem_st_wait();
}

template <int D>
__device__ void sums(const WParams& p, Walk w, Bars& bars, const uint8_t* sK, float (*joint)[kPair], uint32_t tmem,
                     volatile int* abort_flag) {
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, x = warp >> 2 & 1, half = warp >> 3;
  const uint32_t rows = tmem + ((uint32_t)(quarter * 32) << 16), ts = rows + 64u * half;
  const uint64_t c2 = f2::pack(p.scale_log2, p.scale_log2);
  const auto done = [&](uint64_t* bar, uint32_t parity) {
    if (__all_sync(0xffffffffu, wait_bar(bar, parity & 1u, abort_flag))) return true;
    asm volatile("bar.arrive %0, 64;" ::"r"(1 + (warp & 7)) : "memory");    // the other half may wait for this one
    return false;
  };
  uint32_t r = 0, turn = 0, buf = x;     // step g: g % 3, g / 3; buffer of product 2 g + x
  for (int n = 0; w.more(); w.next(p), ++n) {
    // the products of the list before have all been seen: its keys may go
    if (!done(&bars.k_full[x], (uint32_t)n)) return;
    keys_to_tmem<D>(sK + x * Cfg<D>::TILE, quarter, half, lane, rows + kColK + (uint32_t)(D / 2) * x);
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
      mbar_arrive(&bars.k_empty[x]);
      mbar_arrive(&bars.kt_full[x]);
    }
    const int tile = 2 * w.t + x, k0 = tile * kTile + 32 * quarter, key = k0 + lane;
    // queries that see this thread's key, some key of the warp, every key of the warp (keys past the sequence
    // are not written and count with none)
    const int end = p.n - 1;
    const auto last = [&](int k) { return k < p.sinks || p.window >= end - k ? end : k + p.window; };
    const int lo = max(key, p.first), hi = key < p.n ? last(key) : -1;
    const int any_lo = max(k0, p.first), any_hi = k0 < p.sinks ? end : last(min(k0 + 31, end));
    const int all_lo = max(k0 + 31, p.first), all_hi = k0 < p.sinks && k0 + 31 >= p.sinks ? last(p.sinks) : last(k0);
    float total = 0.f, lost = 0.f;
    int i = w.i0 + w.jb % w.count;
    const int i_end = w.i0 + w.count;
    for (int j = w.jb; j < w.je; ++j) {
      if (!done(&bars.s_full[x][r], turn)) return;
      const int q = i * kTile + p.shift + 64 * half;
      if (k0 < p.n && q + 63 >= any_lo && q <= any_hi) {
        tc_fence_after();
        const uint32_t at = ts + 128u * buf;
        uint64_t sum[2] = {0ull, 0ull};
        uint32_t v[32], u[32];
        if (q >= all_lo && q + 63 <= all_hi) {
          tmem_ld_x32(at, v);
          tmem_ld_wait<32>(v);
          tmem_ld_x32(at + 32, u);                     // arrives under the first 32
          add_chunk<false>(v, c2, 0u, sum);
          tmem_ld_wait<32>(u);
          add_chunk<false>(u, c2, 0u, sum);
        } else {
#pragma unroll 1
          for (int c = 0; c < 64; c += 32) {
            if (q + c + 31 < any_lo || q + c > any_hi) continue;
            tmem_ld_x32(at + c, v);
            tmem_ld_wait<32>(v);
            const int a = lo - q - c, z = hi - q - c;
            const uint32_t upto = z >= 31 ? 0xffffffffu : (z < 0 ? 0u : ((2u << z) - 1u));
            const uint32_t from = a <= 0 ? 0xffffffffu : (a >= 32 ? 0u : (0xffffffffu << a));
            add_chunk<true>(v, c2, upto & from, sum);
          }
        }
        float a, z;
        f2::unpack(f2::add(sum[0], sum[1]), a, z);
        // total += a + z, with the rounding error of the sum carried on (an infinite sum has none)
        const float y = (a + z) - lost, t = total + y;
        lost = t < __int_as_float(0x7f800000) ? (t - total) - y : 0.f;
        total = t;
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_empty[buf]);
      if (++r == 3) {
        r = 0;
        ++turn;
      }
      buf = buf == 0 ? 2 : buf - 1;                    // two products on
      if (++i == i_end) i = w.i0;
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
    for (int x = 0; x < 2; ++x) {
      mbar_init(&bars.k_full[x], 1);
      mbar_init(&bars.k_empty[x], kSumWarps / 2);
      mbar_init(&bars.kt_full[x], kSumWarps / 2);
      for (int i = 0; i < 3; ++i) mbar_init(&bars.s_full[x][i], 1);
    }
    for (int i = 0; i < 3; ++i) mbar_init(&bars.s_empty[i], kSumWarps / 2);
    mbar_init(&bars.drain, 1);
    for (int i = 0; i < kStages; ++i) {
      mbar_init(&bars.q_full[i], 2);                   // the tile, and -LSE / scale
      mbar_init(&bars.q_empty[i], 1);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 17) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  uint8_t* sK = sbase;
  uint8_t* sQ = sK + 2 * C::TILE;
  uint8_t* sSide = sQ + kStages * C::TILE;
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
  const Walk w(p, (int)blockIdx.x);
  if (warp < kSumWarps) {
    sums<D>(p, w, bars, sK, joint, tmem, &abort_flag);
  } else if (warp == 16) {
    if (elect_one()) loader<D>(p, w, &tq, &tk, bars, sK, sQ, &abort_flag);
    __syncwarp();
  } else if (warp == 17) {
    if (elect_one()) issuer<D>(p, w, bars, sQ, sSide, tmem, &abort_flag);
    __syncwarp();
  } else {
    lse_rows(p, w, warp - 18, bars, sSide, &abort_flag);
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
    const int64_t x = Walk::bound(p, c);
    const Walk w(p, x, x + 1);
    if (w.list < x && Walk::bound(p, c - 1) <= w.list) {
      const int64_t end = w.list + w.length(p);
      float sum = p.partial[((int64_t)(c - 1) * 2 + 1) * kPair + threadIdx.x];
      for (int k = c; Walk::bound(p, k) < end; ++k) sum += p.partial[(int64_t)k * 2 * kPair + threadIdx.x];
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
  p.quota = p.total / ctas;
  p.rest = (int)(p.total % ctas);
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
  p.first_tile = (a.first_query + kTile - 1) / kTile;
  p.shift = a.first_query - p.first_tile * kTile;
  p.tiles = p.first_tile + (a.n_tokens - a.first_query + kTile - 1) / kTile;
  p.pairs = (a.n_tokens + kPair - 1) / kPair;
  p.reach = (int)(((int64_t)a.window + kPair - 1 - p.shift) / kTile);
  p.window = a.window;
  p.sinks = a.sinks;
  p.first = a.first_query;
  p.skip = p.first_tile > p.reach ? (p.first_tile - p.reach + 1) / 2 : 0;
  p.all = before(p, p.pairs);        // small is 0 as yet
  p.total = p.all * p.group * a.kv_heads * a.batch;
  p.small = p.total < INT32_MAX;
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
