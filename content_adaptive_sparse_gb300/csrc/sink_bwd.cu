// Backward of the sink-window attention (sink_attn.cu) for sm_103a (tcgen05 + TMEM + TMA).
//
// Gradients of L = sum(dO * O) over the graph "key j is visible to query i iff j <= i and
// (i - j <= window or j < sinks)". With P_ij = exp(s_ij - LSE_i), D_i = sum_d dO_id O_id:
//   dP_ij = <dO_i, v_j>,  dS_ij = P_ij (dP_ij - D_i),
//   dQ_i = c sum_j dS_ij k_j,  dK_j = c sum_i dS_ij q_i,  dV_j = sum_i P_ij dO_i.
// Launches: sink_prep_kernel or, where few keys are seen, sink_few_kernel (D and -LSE log2(e), padded to
// whole tiles), sink_bwd_kernel<D, false> (dQ: query-stationary), sink_bwd_kernel<D, true> (dK and
// dV: key-stationary, all query heads of the key head), and sink_reduce_kernel when the sinks' rows
// were summed in parts. S and dP are taken twice, so every gradient row has one owner: no atomics,
// the same bits every run.
//
// Step: 128 stationary rows (A0, A1) against 128 moving rows (B0, B1) of a ring stage,
//   S = A0 B0^T, dP = A1 B1^T (tcgen05, SS, N = 128), then from the compute warps
//   acc0 += dS B0 and, key-stationary, acc1 += P B1 (A from TMEM as bf16 pairs, B MN-major).
//   dQ: A = Q, dO; B = K, V.  dK / dV: A = K, V; B = Q, dO (S and dP come out transposed).
// A tcgen05.mma costs its issuing thread the same ~67 cycles at N = 64 as at N = 128, hence the
// 128-row steps. P (key-stationary) and dS are stored over the S that they come from, each warp over
// the columns that it alone has read, so that what the issuing threads wait for anyway (P, dS
// stored; products complete) frees the columns: the compute warps neither announce nor wait for
// free columns. S has two buffers (steps alternate), and the next step's S runs under this step's
// exponentials; dP has one, and the next dP runs once this step's dS is stored. Key-stationary at
// d = 128 the accumulators leave room for two buffers in all, which S and dP exchange every step: the
// next S goes where dP lay, once that is read, and the next dP over P and dS, once they are used.
//
// The sinks are seen by every query: the first key tile's items over the queries past the
// window are cut into chunks of query tiles as long as an ordinary item, whose fp32 sums of the
// sinks' rows go to the workspace and are added in a fixed order.
//
// One persistent CTA per SM (20 warps), items dealt out in turn:
//   warp 0      loads the stationary tiles and the rings by TMA
//   warps 1-3   lane 0 issues MMAs (S and dP, dV, dK; or S, dP, dQ); warp 1 owns TMEM
//   warps 4-19  compute: warp w reads TMEM lane quarter w % 4 (one stationary row per thread) and
//               columns 32 c .. 32 c + 31 of a step, c = w / 4 - 1; at an item's end they write
//               its rows. An item's S and dP run under the previous item's output.
//
// Measured: 16321 tokens, 16 / 4 heads of 128, window 2047: 762 us (28 + 295 + 445: 0.84 PFLOP/s over the
// edges, 1.18 with S and dP counted twice; tensor pipe 65 % busy, the rest the chain S, P, dS, product).
// 4 x 8192 tokens, 12 heads of 64, window 511: 290 us (23 + 117 + 160); an item is five steps, and about
// 3000 cycles, of 13000, pass between two items' steps.
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

__device__ unsigned int g_sink_bwd_err;

constexpr int kTile = 128;
constexpr int kCols = 32;              // columns of a step per compute warp
constexpr int kComputeWarps = 4 * kTile / kCols;
constexpr int kIssuers = 3;           // warps whose lane 0 issues MMAs
constexpr int kThreads = 32 * (1 + kIssuers + kComputeWarps);
constexpr int kMaxStages = 3;
constexpr uint32_t kTmemCols = 512;
constexpr float kLog2e = 1.4426950408889634f;

template <int D, bool KV>
struct Cfg {
  static constexpr int CH = D >= 64 ? 64 : 32;         // elements per swizzled row
  static constexpr int NCH = D / CH;
  static constexpr int ROWB = CH * 2;
  static constexpr uint32_t SWZ = ROWB == 128 ? kSwizzle128B : kSwizzle64B;
  static constexpr CUtensorMapSwizzle TMA_SWZ =
      ROWB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  static constexpr uint32_t ATOM = 8 * ROWB;
  static constexpr int CHUNK = kTile * ROWB;           // one d-chunk of a 128-row tile
  static constexpr int TILE = NCH * CHUNK;
  static constexpr int FIX = D == 128 ? 1 : 2;         // buffers of the stationary tiles
  // slots of B0 and of B1
  static constexpr int N0 = D < 128 || !KV ? 3 : 2;
  static constexpr int N1 = D < 128 ? 3 : (KV ? 2 : 1);
  static constexpr int SLOT0 = TILE + (KV ? 1024 : 0);   // B0, then -LSE log2(e) [128] and D [128]
  static constexpr int RING = N0 * SLOT0 + N1 * TILE;
  // then OUT KB per compute warp, from which the outputs leave, 16 OUT columns at a time
  static constexpr int OUT = KV && D == 64 ? 2 : 1;
  static constexpr int SMEM_NEED = 1024 + FIX * 2 * TILE + RING + kComputeWarps * 1024 * OUT;
  // more than half an SM's shared memory: one CTA (and its 512 TMEM columns) per SM
  static constexpr int SMEM = SMEM_NEED > 120 * 1024 ? SMEM_NEED : 120 * 1024;
  // TMEM columns: two buffers of S, dP (SWAP: in the buffer that S leaves free), accumulators. P is
  // stored over the first half of the kCols columns of S that a warp reads, dS over the second half.
  static constexpr bool SWAP = KV && D == 128;
  static constexpr uint32_t COL_ACC0 = SWAP ? 256 : 384;   // dQ or dK
  static constexpr uint32_t COL_ACC1 = COL_ACC0 + D;   // dV
  static_assert(COL_ACC0 + (KV ? 2 : 1) * D <= kTmemCols, "TMEM columns");
  static_assert(kCols == 32, "one visibility word per thread");
  static_assert(N0 <= kMaxStages && N1 <= kMaxStages && SMEM <= 226 * 1024, "shared memory");
};

struct BParams {
  int batch, n_tokens, heads, kv_heads, group;   // group: query heads per key head
  int tiles, pitch;                 // 128-row tiles per sequence; padded tokens = 128 tiles
  int window, sinks;
  // items: (rank, sequence, head of the stationary rows); dK / dV: ranks from `tiles` on are sink chunks
  int ranks;
  int step_head, step_s, step_rank; // one item of every CTA, in these digits
  int chunk_tiles, n_chunks;        // query tiles per sink chunk, sink chunks per (sequence, head)
  int far_tile;                     // first query tile whose window misses key tile 0
  const float* nl2;                 // [batch][heads][pitch]: -LSE log2(e); -inf past the sequence
  float* dvec;                      // [batch][heads][pitch]: D
  __nv_bfloat16* out0;              // dK (the sinks' rows, sink_reduce_kernel)
  __nv_bfloat16* out1;              // dV
  int64_t os_b[2], os_n[2], os_h[2];   // strides of out0, out1
  float* partial;                   // [batch][kv_heads][n_chunks + 1][2][sinks][d]
  float scale, scale_log2;          // of dQ and dK; of the scores
};

struct Bars {
  uint64_t fixed_full[2], fixed_empty[2];               // stationary tiles (items alternate where FIX is 2)
  // ring; [0]: B0 with -LSE and D, for S and the dS product, [1]: B1, for dP and the P product
  uint64_t st_full[2][kMaxStages], st_empty[2][kMaxStages];
  // Steps alternate between two barriers (phase: step / 2) where a wait for one step could meet the
  // next one's completion
  uint64_t s_full[2], dp_full;      // S / dP written
  uint64_t dp_read;                 // SWAP: dP read by the compute warps
  uint64_t p_full[2], ds_full[2];   // P / dS stored by the compute warps
  uint64_t dv_done[2], dk_done[2];  // products of P (dV) and of dS (dK or dQ) complete
  uint64_t acc_full;                // an item's accumulators complete (phase: item)
  uint64_t drain[kIssuers];
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_suspend(bar, parity, abort_flag, &g_sink_bwd_err, kErrTimeout);
}
// The barrier of step g of a pair.
__device__ __forceinline__ bool wait_pair(uint64_t (&bar)[2], int g, volatile int* abort_flag) {
  return wait_bar(&bar[g & 1], (uint32_t)(g >> 1) & 1u, abort_flag);
}
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  int never = 0;
  mbar_wait(bar, parity, &never, &g_sink_bwd_err, kErrTimeout);
}

// Work item: a stationary tile and its moving tiles. Step j (0 .. steps - 1) of a dQ item is key
// tile 0 (n_sink = 1, j = 0) or tile0 + j - n_sink; of a dK / dV item query head head0 + j / per and
// query tile tile0 + j % per.
struct Item {
  int s, head, tile;                // stationary rows: head of Q (dQ) or of K / V
  int steps, per, tile0, n_sink;
  int slot;                         // dK / dV: partial-sum slot of the sinks' rows (-1: none)
};

// A CTA's items in turn, found by additions (the divisions of an item's number took every role some
// hundred cycles between items).
template <bool KV>
struct Walk {
  int head, s, rank;
  __device__ explicit Walk(const BParams& p) {
    const int heads = KV ? p.kv_heads : p.heads, k = blockIdx.x;
    head = k % heads;
    s = k / heads % p.batch;
    rank = k / heads / p.batch;
  }
  __device__ __forceinline__ bool more(const BParams& p) const { return rank < p.ranks; }
  __device__ __forceinline__ void next(const BParams& p) {
    head += p.step_head;
    s += p.step_s;
    rank += p.step_rank;
    if (head >= (KV ? p.kv_heads : p.heads)) {
      head -= KV ? p.kv_heads : p.heads;
      ++s;
    }
    if (s >= p.batch) {
      s -= p.batch;
      ++rank;
    }
  }
  __device__ __forceinline__ Item item(const BParams& p) const {
    Item it;
    it.slot = -1;
    it.head = head;
    it.s = s;
    it.n_sink = 0;
    if constexpr (!KV) {
      it.tile = p.tiles - 1 - rank;                      // the last tiles see the most keys
      it.tile0 = max(0, it.tile * kTile - p.window) / kTile;
      it.n_sink = p.sinks > 0 && it.tile0 > 0 ? 1 : 0;
      it.per = it.tile - it.tile0 + 1;
      it.steps = it.n_sink + it.per;
    } else {
      if (rank < p.tiles) {
        it.tile = rank;
        it.tile0 = rank;
        it.per = min(p.tiles - 1, (rank * kTile + kTile - 1 + p.window) / kTile) - rank + 1;
        if (rank == 0 && p.n_chunks > 0) it.slot = 0;
      } else {
        const int chunk = rank - p.tiles;
        it.tile = 0;
        it.tile0 = p.far_tile + chunk * p.chunk_tiles;
        it.per = min(p.tiles, it.tile0 + p.chunk_tiles) - it.tile0;
        it.slot = 1 + chunk;
      }
      it.steps = it.per * p.group;
    }
    return it;
  }
};

// Moving rows of an item's steps, in order: head and tile.
template <bool KV>
struct Steps {
  int head, tile, last;
  __device__ Steps(const BParams& p, const Item& it) {
    head = KV ? it.head * p.group : it.head / p.group;
    tile = !KV && it.n_sink ? 0 : it.tile0;
    last = it.tile0 + it.per - 1;
  }
  __device__ __forceinline__ void next(const Item& it) {
    if (KV && tile == last) {
      tile = it.tile0;
      ++head;
    } else {
      tile = !KV && tile < it.tile0 ? it.tile0 : tile + 1;
    }
  }
};

// Descriptor offset (bytes >> 4) of k-step ks (16 head-dimension elements) of a K-major tile.
template <int D, bool KV>
__device__ __forceinline__ constexpr uint32_t kstep(int ks) {
  using C = Cfg<D, KV>;
  return (uint32_t)(((ks * 16) / C::CH) * C::CHUNK + ((ks * 16) % C::CH) * 2) >> 4;
}

// ------------------------------------------------------------------ loader (warp 0)

// Requests the moving tile of a ring's g-th step, when the slot is free.
template <int D, bool KV, int B>
__device__ __forceinline__ bool load_slot(const BParams& p, const CUtensorMap* tb, Bars& bars, uint8_t* sRing, int g,
                                          int head, int tile, int s, volatile int* abort_flag) {
  using C = Cfg<D, KV>;
  constexpr int N = B ? C::N1 : C::N0;
  const int st = g % N;
  uint64_t* bar = &bars.st_full[B][st];
  if (g >= N && !wait_bar(&bars.st_empty[B][st], (uint32_t)(g / N - 1) & 1u, abort_flag)) return false;
  uint8_t* slot = sRing + (B ? C::N0 * C::SLOT0 + st * C::TILE : st * C::SLOT0);
  mbar_arrive_expect_tx(bar, B ? C::TILE : C::SLOT0);
#pragma unroll
  for (int c = 0; c < C::NCH; ++c) tma_load_4d(slot + c * C::CHUNK, tb, bar, c * C::CH, head, tile * kTile, s);
  if constexpr (KV && B == 0) {
    const int64_t row = ((int64_t)s * p.heads + head) * p.pitch + (int64_t)tile * kTile;
    bulk_load(slot + C::TILE, p.nl2 + row, 512, bar);
    bulk_load(slot + C::TILE + 512, p.dvec + row, 512, bar);
  }
  return true;
}

// B0: load the stationary tiles and B0's ring; B1: B1's. Where the rings are of one length one lane
// loads both; where they are not, B0 runs ahead, so each has a lane (d = 128, dQ: 339 -> 297 us). Lanes
// cost issue slots (d = 64: 165 -> 169 us), a further warp the compute warps' registers (-> 168 us).
template <int D, bool KV, bool B0, bool B1>
__device__ void loader(const BParams& p, const CUtensorMap* ta0, const CUtensorMap* ta1, const CUtensorMap* tb0,
                       const CUtensorMap* tb1, Bars& bars, uint8_t* sFix, uint8_t* sRing, volatile int* abort_flag) {
  using C = Cfg<D, KV>;
  int g0 = 0, g1 = 0, n = 0;
  bool ok = true;
  for (Walk<KV> walk(p); ok && walk.more(p); walk.next(p), ++n) {
    const Item it = walk.item(p);
    if constexpr (B0) {
      // the S and dP of the item before in this buffer have read its stationary tiles
      const int fb = n % C::FIX;
      if (n >= C::FIX && !(ok = wait_bar(&bars.fixed_empty[fb], (uint32_t)(n / C::FIX - 1) & 1u, abort_flag))) break;
      mbar_arrive_expect_tx(&bars.fixed_full[fb], 2 * C::TILE);
      uint8_t* fix = sFix + fb * 2 * C::TILE;
#pragma unroll
      for (int c = 0; c < C::NCH; ++c) {
        tma_load_4d(fix + c * C::CHUNK, ta0, &bars.fixed_full[fb], c * C::CH, it.head, it.tile * kTile, it.s);
        tma_load_4d(fix + C::TILE + c * C::CHUNK, ta1, &bars.fixed_full[fb], c * C::CH, it.head, it.tile * kTile, it.s);
      }
    }
    Steps<KV> at(p, it);
    for (int j = 0; j < it.steps; ++j, at.next(it)) {
      if (B1 && !(ok = load_slot<D, KV, 1>(p, tb1, bars, sRing, g1, at.head, at.tile, it.s, abort_flag))) break;
      g1 += B1;
      if (B0 && !(ok = load_slot<D, KV, 0>(p, tb0, bars, sRing, g0, at.head, at.tile, it.s, abort_flag))) break;
      g0 += B0;
    }
  }
  // every copy of this lane has landed before the CTA may exit (n counts the items whose stationary
  // tiles were requested, a broken-off one too; g0, g1 the steps requested)
  if constexpr (B0)
    for (int i = max(0, n - C::FIX); i < n; ++i) drain_bar(&bars.fixed_full[i % C::FIX], (uint32_t)(i / C::FIX) & 1u);
  for (int t = max(0, g0 - C::N0); t < g0; ++t) drain_bar(&bars.st_full[0][t % C::N0], (uint32_t)(t / C::N0) & 1u);
  for (int t = max(0, g1 - C::N1); t < g1; ++t) drain_bar(&bars.st_full[1][t % C::N1], (uint32_t)(t / C::N1) & 1u);
}

// TMEM columns of S and dP of step g.
__device__ __forceinline__ constexpr uint32_t col_s(int g) { return 128u * (uint32_t)(g & 1); }
template <bool SWAP>
__device__ __forceinline__ constexpr uint32_t col_dp(int g) {
  return SWAP ? 128u - col_s(g) : 256u;
}

// ------------------------------------------------------------------ MMA issuers (warps 1-3, lane 0)

// One thread issues an MMA every ~67 cycles and spends hundreds more in the waits between products
// (the barriers' shared-memory accesses queue behind the tensor core's operand reads), so the
// products are dealt out to three threads: S and dP, dV, dK; or S, dP, dQ.
template <int D, bool KV>
struct Issuer {
  using C = Cfg<D, KV>;
  Bars& bars;
  uint32_t tmem;
  volatile int* abort_flag;
  uint64_t a0, a1, b0, b1, b0mn, b1mn;

  // descriptor offsets of step g's slots
  __device__ static uint64_t at0(int g) { return (uint64_t)((g % C::N0 * C::SLOT0) >> 4); }
  __device__ static uint64_t at1(int g) { return (uint64_t)((g % C::N1 * C::TILE) >> 4); }
  __device__ __forceinline__ bool landed0(int g) const {
    return wait_bar(&bars.st_full[0][g % C::N0], (uint32_t)(g / C::N0) & 1u, abort_flag);
  }
  __device__ __forceinline__ bool landed1(int g) const {
    return wait_bar(&bars.st_full[1][g % C::N1], (uint32_t)(g / C::N1) & 1u, abort_flag);
  }

  __device__ __forceinline__ void rows_x_rows(uint32_t col, uint64_t a, uint64_t b) const {
    constexpr uint32_t idesc = make_idesc_bf16(128, kTile, 0, 0);
#pragma unroll
    for (int ks = 0; ks < D / 16; ++ks)
      mma_bf16_ss(tmem + col, a + kstep<D, KV>(ks), b + kstep<D, KV>(ks), idesc, ks > 0 ? 1u : 0u);
  }
  // acc (+)= A[128 x 128, bf16 pairs in TMEM] * B[128 x d], the moving tile read MN-major
  __device__ __forceinline__ void pairs_x_tile(uint32_t col, uint32_t a, uint64_t b, bool acc) const {
    constexpr uint32_t idesc = make_idesc_bf16(128, D, 0, 1);
#pragma unroll
    for (int ks = 0; ks < kTile / 16; ++ks)
      mma_bf16_ts(tmem + col, tmem + a + (uint32_t)(kCols * (ks / (kCols / 16)) + 8 * (ks % (kCols / 16))), b + (uint64_t)((16 * ks * C::ROWB) >> 4),
                  idesc, (acc || ks > 0) ? 1u : 0u);
  }
  // S of step g, once what lay in its buffer is used: P and dS of two steps before, or the last dP
  __device__ __forceinline__ bool scores(int g, uint64_t fix) const {
    if constexpr (C::SWAP) {
      if (g > 0 && !wait_bar(&bars.dp_read, (uint32_t)(g - 1) & 1u, abort_flag)) return false;
    } else if (g >= 2) {
      if (KV && !wait_pair(bars.dv_done, g - 2, abort_flag)) return false;
      if (!wait_pair(bars.dk_done, g - 2, abort_flag)) return false;
    }
    if (!landed0(g)) return false;
    tc_fence_after();
    rows_x_rows(col_s(g), a0 + fix, b0 + at0(g));
    mma_commit(&bars.s_full[g & 1]);
    return true;
  }
  // dP, once step g - 1's is read, or its P and dS are used
  __device__ __forceinline__ bool products(int g, uint64_t fix) const {
    if (g > 0) {
      if constexpr (C::SWAP) {
        if (!wait_pair(bars.dv_done, g - 1, abort_flag) || !wait_pair(bars.dk_done, g - 1, abort_flag)) return false;
      } else if (!wait_pair(bars.ds_full, g - 1, abort_flag)) {
        return false;
      }
    }
    if (!landed1(g)) return false;
    tc_fence_after();
    rows_x_rows(col_dp<C::SWAP>(g), a1 + fix, b1 + at1(g));
    mma_commit(&bars.st_empty[1][g % C::N1]);
    mma_commit(&bars.dp_full);
    return true;
  }
  __device__ __forceinline__ bool acc1(int g, bool acc) const {
    if (!landed1(g) || !wait_pair(bars.p_full, g, abort_flag)) return false;
    tc_fence_after();
    pairs_x_tile(C::COL_ACC1, col_s(g), b1mn + at1(g), acc);
    mma_commit(&bars.st_empty[1][g % C::N1]);
    mma_commit(&bars.dv_done[g & 1]);
    return true;
  }
  __device__ __forceinline__ bool acc0(int g, bool acc) const {
    if (!landed0(g) || !wait_pair(bars.ds_full, g, abort_flag)) return false;
    tc_fence_after();
    pairs_x_tile(C::COL_ACC0, col_s(g) + kCols / 2, b0mn + at0(g), acc);
    mma_commit(&bars.st_empty[0][g % C::N0]);
    mma_commit(&bars.dk_done[g & 1]);
    return true;
  }
};

template <int D, bool KV>
__device__ void issuer(const BParams& p, int role, Bars& bars, uint8_t* sFix, uint8_t* sRing, uint32_t tmem,
                       volatile int* abort_flag) {
  using C = Cfg<D, KV>;
  const uint32_t fix = smem_u32(sFix), ring = smem_u32(sRing), ring1 = ring + C::N0 * C::SLOT0;
  const Issuer<D, KV> I{bars, tmem, abort_flag,
                        make_smem_desc(fix, 16, C::ATOM, C::SWZ),
                        make_smem_desc(fix + C::TILE, 16, C::ATOM, C::SWZ),
                        make_smem_desc(ring, 16, C::ATOM, C::SWZ),
                        make_smem_desc(ring1, 16, C::ATOM, C::SWZ),
                        make_smem_desc(ring, C::CHUNK, C::ATOM, C::SWZ),
                        make_smem_desc(ring1, C::CHUNK, C::ATOM, C::SWZ)};
  int g = 0, n = 0;
  bool ok = true;
  for (Walk<KV> walk(p); ok && walk.more(p); walk.next(p), ++n) {
    const int steps = walk.item(p).steps;
    if (role == 2 || (KV && role == 1)) {
      for (int j = 0; ok && j < steps; ++j, ++g) ok = KV && role == 1 ? I.acc1(g, j > 0) : I.acc0(g, j > 0);
      if (ok) mma_commit(&bars.acc_full);
    } else {
      const int fb = n % C::FIX;
      const uint64_t fix = (uint64_t)((fb * 2 * C::TILE) >> 4);
      if (!(ok = wait_bar(&bars.fixed_full[fb], (uint32_t)(n / C::FIX) & 1u, abort_flag))) break;
      for (int j = 0; ok && j < steps; ++j, ++g) {
        if (role == 0) ok = I.scores(g, fix);
        if (ok && role == (KV ? 0 : 1)) ok = I.products(g, fix);
      }
      if (ok) mma_commit(&bars.fixed_empty[fb]);       // the item's last S (and dP) are issued
    }
  }
  // no MMA of this thread is still at work when the CTA frees its TMEM
  mma_commit(&bars.drain[role]);
  drain_bar(&bars.drain[role], 0);
}

// ------------------------------------------------------------------ compute (warps 4-19)

// Bits b in [lo, hi] of 32.
__device__ __forceinline__ uint32_t bit_range(int lo, int hi) {
  const uint32_t from = lo <= 0 ? 0xffffffffu : (lo >= 32 ? 0u : (0xffffffffu << lo));
  const uint32_t upto = hi >= 31 ? 0xffffffffu : (hi < 0 ? 0u : ((2u << hi) - 1u));
  return from & upto;
}

// Visible columns c0 .. c0 + 31 of the thread's row token r. dQ: r is a query, columns are keys;
// dK / dV: r is a key, columns are queries.
template <bool KV>
__device__ __forceinline__ uint32_t visible(int r, int c0, int window, int sinks) {
  if constexpr (KV) return bit_range(r - c0, r < sinks ? 31 : r + window - c0);
  else return bit_range(r - window - c0, r - c0) | (bit_range(0, sinks - 1 - c0) & bit_range(0, r - c0));
}

enum : int { kNone = 0, kAll = 1, kSome = 2 };

// How rows r0 .. r0 + 31 see columns c0 .. c0 + 31 (see `visible`).
template <bool KV>
__device__ __forceinline__ int visibility(int r0, int c0, int window, int sinks) {
  const int q = KV ? c0 : r0, k = KV ? r0 : c0;        // first query, first key
  if (q + 31 < k || (q - (k + 31) > window && k >= sinks)) return kNone;
  return q >= k + 31 && (q + 31 - k <= window || k + 31 < sinks) ? kAll : kSome;
}

// A compute warp.
template <int D, bool KV>
struct Compute {
  using C = Cfg<D, KV>;
  const BParams& p;
  const CUtensorMap* to0;
  const CUtensorMap* to1;
  Bars& bars;
  volatile int* abort_flag;
  uint32_t base;                    // TMEM of this warp's lanes
  int quarter, part, lane;
  uint8_t* out;                     // this warp's staging memory
  uint64_t c2;

  // This warp's TMEM stores are done: one arrival.
  __device__ __forceinline__ void arrive(uint64_t* bar) const {
    tmem_st_wait();
    announce(bar);
  }
  // Its TMEM loads are.
  __device__ __forceinline__ void announce(uint64_t* bar) const {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(bar);
  }

  // An item's rows, this warp's share of the columns: 16 OUT at a time, through OUT KB of shared
  // memory (rows of 32 OUT bytes, swizzled over them) and a TMA store, which drops rows past the
  // sequence. (Stored straight from the registers, 32 rows in 32 lines per instruction, an item's
  // output took as long as two steps; TMA takes a cycle per row whatever its width.)
  __device__ __forceinline__ bool write(const Item& it, int n) const {
    const int tok0 = it.tile * kTile + 32 * quarter, tok = tok0 + lane;
    const bool sum = KV && it.slot >= 0 && tok < p.sinks;   // an fp32 partial sum (its bf16 row is written after)
    const bool rows = it.slot <= 0;                          // a sink chunk has sums only
    const uint32_t srow = smem_u32(out) + 32u * C::OUT * lane;
    const uint32_t turn = C::OUT == 2 ? (uint32_t)(lane >> 1) & 3u : (uint32_t)(lane >> 2) & 1u;
    if (!__all_sync(0xffffffffu, wait_bar(&bars.acc_full, (uint32_t)n & 1u, abort_flag))) return false;
    tc_fence_after();
    constexpr int N = (KV ? 2 : 1) * (D / 16), W = kComputeWarps / 4;   // chunks; warps that share them
#pragma unroll 1
    for (int c0 = C::OUT * part; c0 < N; c0 += C::OUT * W) {
      if (rows) {
        if (lane == 0) bulk_wait_group_read<0>();
        __syncwarp();
      }
      const int m = c0 / (D / 16), col = 16 * (c0 % (D / 16));   // OUT pieces of one tensor
      const float f = m ? 1.f : p.scale;
      uint32_t w[C::OUT][16];
#pragma unroll
      for (int o = 0; o < C::OUT; ++o)
        tmem_ld_x16(base + (m ? C::COL_ACC1 : C::COL_ACC0) + (uint32_t)(col + 16 * o), w[o]);
#pragma unroll
      for (int o = 0; o < C::OUT; ++o) {
        tmem_ld_wait<16>(w[o]);
        if (sum) {
          const int64_t bh = (int64_t)it.s * p.kv_heads + it.head;
          float* prow = p.partial + (((bh * (p.n_chunks + 1) + it.slot) * 2 + m) * p.sinks + tok) * D + col + 16 * o;
#pragma unroll
          for (int e = 0; e < 16; e += 4)
            *reinterpret_cast<float4*>(prow + e) =
                make_float4(__uint_as_float(w[o][e]) * f, __uint_as_float(w[o][e + 1]) * f,
                            __uint_as_float(w[o][e + 2]) * f, __uint_as_float(w[o][e + 3]) * f);
        }
        if (rows) {
          uint32_t pk[8];
#pragma unroll
          for (int e = 0; e < 16; e += 2)
            pk[e >> 1] = pack_bf16x2(__uint_as_float(w[o][e]) * f, __uint_as_float(w[o][e + 1]) * f);
          st_shared_v4(srow + (((2u * o) ^ turn) << 4), pk[0], pk[1], pk[2], pk[3]);
          st_shared_v4(srow + (((2u * o + 1u) ^ turn) << 4), pk[4], pk[5], pk[6], pk[7]);
        }
      }
      if (rows) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0 && tok0 < p.n_tokens) {
          tma_store_4d(m ? to1 : to0, out, col, it.head, tok0, it.s);
          bulk_commit_group();
        }
      }
    }
    return true;
  }

  // A step. Each way of seeing (SEE) has a copy of the code: joined by selects, the mask's
  // instructions would be issued in every step. `prev`: the item before, at an item's first step.
  // `first`: the columns hold every key that the thread's row sees (the first tokens' rows, dQ only), and
  // D goes to *first for dK / dV.
  template <int SEE>
  __device__ __forceinline__ bool step(int g, uint32_t vec, uint32_t see, float nl2, float dval, float* first,
                                       const Item* prev, int n) const {
    const uint32_t tS = base + (uint32_t)(kCols * part) + col_s(g);
    const uint32_t tDP = base + (uint32_t)(kCols * part) + col_dp<C::SWAP>(g);
    if (!__all_sync(0xffffffffu, wait_pair(bars.s_full, g, abort_flag))) return false;
    tc_fence_after();
    // ---- P
    float pr[kCols];
    if constexpr (SEE != kNone) {
      uint32_t v[kCols];
      tmem_ld_x32(tS, v);
      // dK / dV: the stage's -LSE and D have landed with its tiles
      if (KV && !__all_sync(0xffffffffu,
                            wait_bar(&bars.st_full[0][g % C::N0], (uint32_t)(g / C::N0) & 1u, abort_flag)))
        return false;
      tmem_ld_wait<kCols>(v);
#pragma unroll
      for (int e = 0; e < kCols; e += 4) {
        float4 L = make_float4(nl2, nl2, nl2, nl2);
        if constexpr (KV) L = ld_shared_f4(vec + 4 * e);
        const uint64_t s01 = f2::pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1]));
        const uint64_t s23 = f2::pack(__uint_as_float(v[e + 2]), __uint_as_float(v[e + 3]));
        float x[4];
        f2::unpack(f2::fma(s01, c2, f2::pack(L.x, L.y)), x[0], x[1]);
        f2::unpack(f2::fma(s23, c2, f2::pack(L.z, L.w)), x[2], x[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if constexpr (SEE == kSome) x[i] = ((see >> (e + i)) & 1u) ? x[i] : __int_as_float(0xff800000);
          pr[e + i] = ex2_approx(x[i]);
        }
      }
    }
    if constexpr (KV) {
      uint32_t pk[kCols / 2];
#pragma unroll
      for (int e = 0; e < kCols; e += 2) pk[e >> 1] = SEE != kNone ? pack_bf16x2(pr[e], pr[e + 1]) : 0u;
      tmem_st_x16(tS, pk);
    }
    // dQ: the previous item's rows leave after the first exponentials of this one, under which its last
    // product completes (8K training: 132 -> 121 us; for dK / dV, whose registers are full, leaving
    // before them is faster: 163 against 190 us). This item's first product into the accumulators
    // waits for the P or dS that is announced after them.
    if (!KV && prev != nullptr && !write(*prev, n - 1)) return false;
    if constexpr (KV) arrive(&bars.p_full[g & 1]);
    // ---- dS = P (dP - D)
    if (!__all_sync(0xffffffffu, wait_bar(&bars.dp_full, (uint32_t)g & 1u, abort_flag))) return false;
    tc_fence_after();
    uint32_t ds[kCols / 2];
    if constexpr (SEE != kNone) {
      uint32_t v[kCols];
      tmem_ld_x32(tDP, v);
      tmem_ld_wait<kCols>(v);
      if constexpr (C::SWAP) announce(&bars.dp_read);
      if constexpr (!KV && SEE == kSome) {
        if (first != nullptr) {
          dval = 0.f;
#pragma unroll
          for (int e = 0; e < kCols; ++e) dval = fmaf(pr[e], __uint_as_float(v[e]), dval);
          *first = dval;
        }
      }
#pragma unroll
      for (int e = 0; e < kCols; e += 4) {
        float4 L = make_float4(dval, dval, dval, dval);
        if constexpr (KV) L = ld_shared_f4(vec + 512 + 4 * e);
#pragma unroll
        for (int i = 0; i < 4; i += 2) {
          const uint64_t d2 = i ? f2::pack(L.z, L.w) : f2::pack(L.x, L.y);
          const uint64_t dp = f2::pack(__uint_as_float(v[e + i]), __uint_as_float(v[e + i + 1]));
          float y0, y1;
          f2::unpack(f2::mul(f2::pack(pr[e + i], pr[e + i + 1]), f2::sub(dp, d2)), y0, y1);
          ds[(e + i) >> 1] = pack_bf16x2(y0, y1);
        }
      }
    } else {
      if constexpr (C::SWAP) announce(&bars.dp_read);
#pragma unroll
      for (int e = 0; e < kCols / 2; ++e) ds[e] = 0u;
    }
    tmem_st_x16(tS + kCols / 2, ds);
    arrive(&bars.ds_full[g & 1]);
    return true;
  }
};

template <int D, bool KV>
__device__ void compute(const BParams& p, const CUtensorMap* to0, const CUtensorMap* to1, Bars& bars, uint8_t* sRing,
                        uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D, KV>;
  const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;   // warp: uniform
  const int quarter = warp & 3, part = (warp - 1 - kIssuers) >> 2;
  const int row = quarter * 32 + lane;
  const uint32_t ring = smem_u32(sRing);
  const uint32_t base = tmem + ((uint32_t)(quarter * 32) << 16);
  const Compute<D, KV> W{p, to0, to1, bars, abort_flag, base, quarter, part, lane,
                         sRing + C::RING + 1024 * C::OUT * (4 * part + quarter), f2::pack(p.scale_log2, p.scale_log2)};
  int g = 0, n = 0;
  Item it, prev;
  for (Walk<KV> walk(p); walk.more(p); walk.next(p), ++n) {
    prev = it;
    it = walk.item(p);
    const int tok = it.tile * kTile + row;
    float nl2 = 0.f, dval = 0.f;
    float* first = nullptr;
    if constexpr (!KV) {
      const int64_t at = ((int64_t)it.s * p.heads + it.head) * p.pitch + tok;
      nl2 = p.nl2[at];
      dval = p.dvec[at];
      // O is stored in bf16, and in <dO, O> its rounding, 2^-9 of |dO| |O|, goes into every dS of the row
      // alike: into dQ times the mean of the visible keys. That is little where many keys are seen (their
      // mean is short, and dS has a rounding of its own); at two keys it took dQ's error from 0.0024 to
      // 0.0046 of its size, at nine to 0.0027. The first kCols tokens see no other keys than one another, so
      // this warp holds all of their P and dP, and their D is sum P dP. (The time is the same with and
      // without: 4 x 8192 training 384 us; a launch of its own took 11 us in 2 x 200 tokens, 27 against 15.)
      if (it.tile == 0 && quarter == 0 && part == 0) first = p.dvec + at;
    }
    Steps<KV> moving(p, it);
    if (KV && n > 0 && !W.write(prev, n - 1)) return;
    for (int j = 0; j < it.steps; ++j, ++g, moving.next(it)) {
      const int c0 = moving.tile * kTile + kCols * part;
      const uint32_t vec = ring + (uint32_t)((g % C::N0) * C::SLOT0 + C::TILE + 4 * kCols * part);
      const int see = visibility<KV>(it.tile * kTile + 32 * quarter, c0, p.window, p.sinks);
      const Item* before = !KV && j == 0 && n > 0 ? &prev : nullptr;
      bool ok;
      if (see == kAll) ok = W.template step<kAll>(g, vec, 0u, nl2, dval, nullptr, before, n);
      else if (see == kSome)
        ok = W.template step<kSome>(g, vec, visible<KV>(tok, c0, p.window, p.sinks), nl2, dval, first, before, n);
      else ok = W.template step<kNone>(g, vec, 0u, nl2, dval, nullptr, before, n);
      if (!ok) return;
    }
  }
  if (n > 0) W.write(it, n - 1);
}

template <int D, bool KV>
__global__ void __launch_bounds__(kThreads, 1)
    sink_bwd_kernel(const __grid_constant__ CUtensorMap ta0, const __grid_constant__ CUtensorMap ta1,
                    const __grid_constant__ CUtensorMap tb0, const __grid_constant__ CUtensorMap tb1,
                    const __grid_constant__ CUtensorMap to0, const __grid_constant__ CUtensorMap to1,
                    const __grid_constant__ BParams p) {
  using C = Cfg<D, KV>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;
  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::FIX; ++i) {
      mbar_init(&bars.fixed_full[i], 1);
      mbar_init(&bars.fixed_empty[i], KV ? 1 : 2);     // S and dP from one thread, or from two
    }
    for (int i = 0; i < kMaxStages; ++i) {
      for (int b = 0; b < 2; ++b) mbar_init(&bars.st_full[b][i], 1);
      mbar_init(&bars.st_empty[0][i], 1);              // the dS product (S is complete before)
      mbar_init(&bars.st_empty[1][i], KV ? 2 : 1);     // dP, and the P product
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&bars.s_full[i], 1);
      mbar_init(&bars.p_full[i], kComputeWarps);
      mbar_init(&bars.ds_full[i], kComputeWarps);
      mbar_init(&bars.dv_done[i], 1);
      mbar_init(&bars.dk_done[i], 1);
    }
    mbar_init(&bars.dp_full, 1);
    mbar_init(&bars.dp_read, kComputeWarps);
    mbar_init(&bars.acc_full, KV ? 2 : 1);
    for (int i = 0; i < kIssuers; ++i) mbar_init(&bars.drain[i], 1);
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&ta0);
    tma_prefetch_desc(&ta1);
    tma_prefetch_desc(&tb0);
    tma_prefetch_desc(&tb1);
    tma_prefetch_desc(&to0);
    tma_prefetch_desc(&to1);
  }
  if (warp == 1) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;
  uint8_t* sFix = sbase;
  uint8_t* sRing = sFix + C::FIX * 2 * C::TILE;
  if (warp == 0) {
    const int lane = threadIdx.x & 31;
    constexpr bool kOne = C::N0 == C::N1;
    if (lane == 0) loader<D, KV, true, kOne>(p, &ta0, &ta1, &tb0, &tb1, bars, sFix, sRing, &abort_flag);
    if constexpr (!kOne)
      if (lane == 1) loader<D, KV, false, true>(p, &ta0, &ta1, &tb0, &tb1, bars, sFix, sRing, &abort_flag);
    __syncwarp();
  } else if (warp <= kIssuers) {
    if ((threadIdx.x & 31) == 0) issuer<D, KV>(p, warp - 1, bars, sFix, sRing, tmem, &abort_flag);
    __syncwarp();
  } else {
    compute<D, KV>(p, &to0, &to1, bars, sRing, tmem, &abort_flag);
    // this warp's stores are complete before the CTA may exit
    if ((threadIdx.x & 31) == 0) bulk_wait_group<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ------------------------------------------------------------------ D and -LSE log2(e)

struct PrepTensor {
  const __nv_bfloat16* ptr;
  int64_t sb, sn, sh;
};

struct PrepParams {
  PrepTensor q, k, v, o, d_o;
  const float* lse;
  float* nl2;
  float* dvec;
  int batch, n_tokens, heads, group, pitch, window, sinks;
  float scale_log2;
};

// This lane's share of a dot product: 8 elements.
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t av[4] = {a.x, a.y, a.z, a.w}, bv[4] = {b.x, b.y, b.z, b.w};
  float acc = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    acc = fmaf(__uint_as_float(av[e] << 16), __uint_as_float(bv[e] << 16), acc);
    acc = fmaf(__uint_as_float(av[e] & 0xffff0000u), __uint_as_float(bv[e] & 0xffff0000u), acc);
  }
  return acc;
}

template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int w = G / 2; w > 0; w >>= 1) v += __shfl_xor_sync(0xffffffffu, v, w, G);
  return v;
}

// The row `part` of D / 8 threads reads 16 bytes of.
__device__ __forceinline__ uint4 prep_row(const PrepTensor& t, int s, uint32_t i, uint32_t h, int part) {
  return *reinterpret_cast<const uint4*>(t.ptr + s * t.sb + i * t.sn + h * t.sh + 8 * part);
}

// -LSE in log2 units. A query without a finite score (LSE -inf) has no gradient: P is 0, as past the sequence.
__device__ __forceinline__ float minus_lse(float lse) {
  return lse == __int_as_float(0xff800000) ? lse : -lse * kLog2e;
}

// D / 8 consecutive threads per kPrepRows (token, head) rows of a sequence, 16 bytes of O and dO each;
// tokens n .. pitch - 1 get D = 0 and -LSE = -inf, so that their P is 0. (16321 tokens of 16 heads of
// 128: 28 us, 4.8 TB/s; one row a thread 32.)
constexpr int kPrepRows = 2;
template <int D>
__global__ void __launch_bounds__(256) sink_prep_kernel(const __grid_constant__ PrepParams p) {
  constexpr int G = D / 8;
  const int part = threadIdx.x % G;
  const uint32_t heads = (uint32_t)p.heads, n = (uint32_t)p.n_tokens;
  const uint32_t rows = (uint32_t)p.pitch * heads;           // below 2^31 (the host's check)
  const uint32_t r0 = (blockIdx.x * (blockDim.x / G) + threadIdx.x / G) * kPrepRows;
  for (int s = blockIdx.y; s < p.batch; s += gridDim.y) {
    uint4 a[kPrepRows], b[kPrepRows];
#pragma unroll
    for (int u = 0; u < kPrepRows; ++u) {
      const uint32_t i = (r0 + u) / heads, h = (r0 + u) % heads;
      a[u] = b[u] = make_uint4(0u, 0u, 0u, 0u);
      if (i < n) {
        a[u] = prep_row(p.o, s, i, h, part);
        b[u] = prep_row(p.d_o, s, i, h, part);
      }
    }
#pragma unroll
    for (int u = 0; u < kPrepRows; ++u) {
      const uint32_t i = (r0 + u) / heads, h = (r0 + u) % heads;
      const float d = lanes_sum<G>(dot8(a[u], b[u]));
      if (part == 0 && r0 + u < rows) {
        const int64_t bh = (int64_t)s * heads + h;
        p.dvec[bh * p.pitch + i] = d;
        p.nl2[bh * p.pitch + i] = i < n ? minus_lse(p.lse[bh * n + i]) : __int_as_float(0xff800000);
      }
    }
  }
}

// The same with D = sum of P dP (the reason: Compute's `first`) for windows and sinks of which no query sees
// more than kFewKeys keys. (16K tokens of 16 heads of 128 at eight: backward 210 -> 322 us; more would cost more
// than the accuracy that is left to gain.)
constexpr int kFewKeys = 8, kFewStep = 4;
template <int D>
__global__ void __launch_bounds__(256) sink_few_kernel(const __grid_constant__ PrepParams p) {
  constexpr int G = D / 8;
  const int part = threadIdx.x % G;
  const uint32_t heads = (uint32_t)p.heads, n = (uint32_t)p.n_tokens;
  const uint32_t r = blockIdx.x * (blockDim.x / G) + threadIdx.x / G;
  const uint32_t i = r / heads, h = r % heads, hk = h / (uint32_t)p.group;
  const bool in = i < (uint32_t)p.pitch;
  const int lo = max(0, (int)i - p.window), n_sink = min(p.sinks, lo);
  const int keys = in && i < n ? n_sink + (int)i - lo + 1 : 0;
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
  for (int s = blockIdx.y; s < p.batch; s += gridDim.y) {
    const int64_t bh = (int64_t)s * heads + h;
    const uint4 q = keys > 0 ? prep_row(p.q, s, i, h, part) : zero;
    const uint4 g = keys > 0 ? prep_row(p.d_o, s, i, h, part) : zero;
    const float nl2 = keys > 0 ? minus_lse(p.lse[bh * n + i]) : __int_as_float(0xff800000);
    float d = 0.f;
#pragma unroll 1
    for (int e0 = 0; __any_sync(0xffffffffu, e0 < keys); e0 += kFewStep) {
      float sc[kFewStep], dp[kFewStep];
#pragma unroll
      for (int x = 0; x < kFewStep; ++x) {
        const int e = e0 + x;
        const uint32_t j = (uint32_t)(e < n_sink ? e : lo + e - n_sink);
        sc[x] = dot8(q, e < keys ? prep_row(p.k, s, j, hk, part) : zero);
        dp[x] = dot8(g, e < keys ? prep_row(p.v, s, j, hk, part) : zero);
      }
#pragma unroll
      for (int x = 0; x < kFewStep; ++x) {
        sc[x] = lanes_sum<G>(sc[x]);
        dp[x] = lanes_sum<G>(dp[x]);
        if (e0 + x < keys) d = fmaf(ex2_approx(fmaf(sc[x], p.scale_log2, nl2)), dp[x], d);
      }
    }
    if (part == 0 && in) {
      p.dvec[bh * p.pitch + i] = d;
      p.nl2[bh * p.pitch + i] = nl2;
    }
  }
}

// dK, dV of the sinks' rows: the partial sums of the first key tile's items, in slot order.
__global__ void __launch_bounds__(256) sink_reduce_kernel(const __grid_constant__ BParams p, int d) {
  const int quads = d / 4;
  const int64_t gid = (int64_t)blockIdx.x * blockDim.x + threadIdx.x;
  const int e = (int)(gid % quads) * 4;
  int64_t r = gid / quads;
  const int row = (int)(r % p.sinks);
  r /= p.sinks;
  const int m = (int)(r % 2);
  const int64_t bh = r / 2;
  if (bh >= (int64_t)p.batch * p.kv_heads || row >= p.n_tokens) return;
  const float* src = p.partial + (bh * (p.n_chunks + 1) * 2 + m) * (int64_t)p.sinks * d + (int64_t)row * d + e;
  float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c <= p.n_chunks; ++c) {
    const float4 v = *reinterpret_cast<const float4*>(src + (int64_t)c * 2 * p.sinks * d);
    sum.x += v.x;
    sum.y += v.y;
    sum.z += v.z;
    sum.w += v.w;
  }
  __nv_bfloat16* out =
      (m ? p.out1 : p.out0) + (bh / p.kv_heads) * p.os_b[m] + row * p.os_n[m] + (bh % p.kv_heads) * p.os_h[m] + e;
  *reinterpret_cast<uint2*>(out) = make_uint2(pack_bf16x2(sum.x, sum.y), pack_bf16x2(sum.z, sum.w));
}

// ------------------------------------------------------------------ launch

// Chunks of the first key tile's queries past the window (none without sinks).
struct Chunks {
  int far_tile, tiles_each, count;
};

Chunks sink_chunks(int tiles, int window, int sinks) {
  Chunks c;
  c.far_tile = (int)(((int64_t)kTile - 1 + window) / kTile) + 1;
  if (c.far_tile > tiles) c.far_tile = tiles;
  // as long as an ordinary item, and at least 8 tiles, so that their partial sums stay few
  c.tiles_each = c.far_tile > 8 ? c.far_tile : 8;
  c.count = sinks > 0 ? (tiles - c.far_tile + c.tiles_each - 1) / c.tiles_each : 0;
  return c;
}

template <int D, bool KV>
int launch(const SinkArgs& a, BParams p, int ranks, cudaStream_t stream) {
  using C = Cfg<D, KV>;
  CUtensorMap tq, tk, tv, tdo;
  auto map = [&](CUtensorMap* m, const void* base, int heads, const int64_t st[3]) {
    return encode_bhnd_map(m, base, a.batch, a.n_tokens, heads, D, st[0], st[1], st[2], C::CH, kTile, C::TMA_SWZ);
  };
  if (!map(&tq, a.q, a.heads, a.q_strides) || !map(&tk, a.k, a.kv_heads, a.k_strides) ||
      !map(&tv, a.v, a.kv_heads, a.v_strides) || !map(&tdo, a.d_o, a.heads, a.do_strides))
    return SA_ERR_UNSUPPORTED;
  // outputs: boxes of 32 rows by 16 OUT elements
  CUtensorMap to0, to1;
  auto omap = [&](CUtensorMap* m, const void* base, int heads, const int64_t st[3]) {
    return encode_bhnd_map(m, base, a.batch, a.n_tokens, heads, D, st[0], st[1], st[2], 16 * C::OUT, 32,
                           C::OUT == 2 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_32B);
  };
  if (KV ? !omap(&to0, a.dk, a.kv_heads, a.dk_strides) || !omap(&to1, a.dv, a.kv_heads, a.dv_strides)
         : !omap(&to0, a.dq, a.heads, a.dq_strides) || !omap(&to1, a.dq, a.heads, a.dq_strides))
    return SA_ERR_UNSUPPORTED;
  const auto kern = sink_bwd_kernel<D, KV>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return SA_ERR_CUDA;
  const int sm_count = current_sm_count();
  const int heads = KV ? a.kv_heads : a.heads;
  const int64_t items = (int64_t)ranks * a.batch * heads;
  const int grid = items < sm_count ? (int)items : sm_count;
  p.ranks = ranks;
  p.step_head = grid % heads;
  p.step_s = grid / heads % a.batch;
  p.step_rank = grid / heads / a.batch;
  if (KV) kern<<<grid, kThreads, C::SMEM, stream>>>(tk, tv, tq, tdo, to0, to1, p);
  else kern<<<grid, kThreads, C::SMEM, stream>>>(tq, tdo, tk, tv, to0, to1, p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int D>
int launch_d(const SinkArgs& a, const SinkBwdWorkspace& ws, cudaStream_t stream) {
  uint8_t* wsb = static_cast<uint8_t*>(a.workspace);
  BParams p;
  memset(&p, 0, sizeof(p));
  p.batch = a.batch;
  p.n_tokens = a.n_tokens;
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.tiles = (a.n_tokens + kTile - 1) / kTile;
  p.pitch = p.tiles * kTile;
  p.window = a.window;
  p.sinks = a.sinks;
  float* nl2 = reinterpret_cast<float*>(wsb + ws.nl2_off);
  float* dvec = reinterpret_cast<float*>(wsb + ws.dvec_off);
  p.nl2 = nl2;
  p.dvec = dvec;
  p.partial = reinterpret_cast<float*>(wsb + ws.partial_off);
  // Where every query sees one key, P is 1 whatever the scores are: dQ and dK are zero, and dP - D would
  // leave them the rounding of two sums.
  const bool one_key = a.n_tokens == 1 || (a.window == 0 && a.sinks == 0);
  p.scale = one_key ? 0.f : a.softmax_scale;
  p.scale_log2 = a.softmax_scale * kLog2e;
  const auto tensor = [](const void* ptr, const int64_t st[3]) {
    return PrepTensor{static_cast<const __nv_bfloat16*>(ptr), st[0], st[1], st[2]};
  };
  const PrepParams pp{tensor(a.q, a.q_strides), tensor(a.k, a.k_strides), tensor(a.v, a.v_strides),
                      tensor(a.o, a.o_strides), tensor(a.d_o, a.do_strides), a.lse, nl2, dvec,
                      a.batch, a.n_tokens, a.heads, p.group, p.pitch, a.window, a.sinks, p.scale_log2};
  const auto grid = [&](int64_t rows) {                      // of groups of D / 8 threads
    return dim3((unsigned)((rows * (D / 8) + 255) / 256), (unsigned)(a.batch < 65535 ? a.batch : 65535));
  };
  const int64_t rows = (int64_t)p.pitch * a.heads;
  // token i sees min(i, window + sinks) + 1 keys
  if ((int64_t)a.window + a.sinks < kFewKeys) sink_few_kernel<D><<<grid(rows), 256, 0, stream>>>(pp);
  else sink_prep_kernel<D><<<grid((rows + kPrepRows - 1) / kPrepRows), 256, 0, stream>>>(pp);
  if (cudaGetLastError() != cudaSuccess) return SA_ERR_CUDA;
  int st = launch<D, false>(a, p, p.tiles, stream);
  if (st != SA_OK) return st;
  const Chunks c = sink_chunks(p.tiles, a.window, a.sinks);
  p.far_tile = c.far_tile;
  p.chunk_tiles = c.tiles_each;
  p.n_chunks = c.count;
  p.out0 = static_cast<__nv_bfloat16*>(a.dk);
  p.out1 = static_cast<__nv_bfloat16*>(a.dv);
  for (int m = 0; m < 2; ++m) {
    const int64_t* st = m ? a.dv_strides : a.dk_strides;
    p.os_b[m] = st[0];
    p.os_n[m] = st[1];
    p.os_h[m] = st[2];
  }
  st = launch<D, true>(a, p, p.tiles + c.count, stream);
  if (st != SA_OK || c.count == 0) return st;
  const int64_t quads = (int64_t)a.batch * a.kv_heads * 2 * a.sinks * (D / 4);
  sink_reduce_kernel<<<(unsigned)((quads + 255) / 256), 256, 0, stream>>>(p, D);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

SinkBwdWorkspace sink_bwd_workspace_layout(int64_t batch, int64_t n_tokens, int64_t heads, int64_t kv_heads, int64_t d,
                                           int window, int sinks) {
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  const int tiles = (int)((n_tokens + kTile - 1) / kTile);
  const Chunks c = sink_chunks(tiles, window, sinks);
  SinkBwdWorkspace w;
  w.nl2_off = 0;
  w.dvec_off = up((size_t)(batch * heads * tiles) * kTile * 4);
  w.partial_off = 2 * w.dvec_off;
  w.bytes = w.partial_off + (c.count > 0 ? up((size_t)(batch * kv_heads * (c.count + 1)) * 2 * sinks * d * 4) : 0);
  return w;
}

int launch_sink_attn_bwd(const SinkArgs& a, cudaStream_t stream) {
  const SinkBwdWorkspace ws =
      sink_bwd_workspace_layout(a.batch, a.n_tokens, a.heads, a.kv_heads, a.head_dim, a.window, a.sinks);
  if (a.workspace_bytes < ws.bytes) return SA_ERR_CAPACITY;
  switch (a.head_dim) {
    case 32: return launch_d<32>(a, ws, stream);
    case 64: return launch_d<64>(a, ws, stream);
    case 128: return launch_d<128>(a, ws, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int sink_bwd_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_sink_bwd_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_sink_bwd_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
