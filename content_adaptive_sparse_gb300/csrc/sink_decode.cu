// Single-token form of the sink-window attention over a key / value cache: the query is token
// length - 1 of its sequence and sees cache rows j < length with length - 1 - j <= window or
// j < sinks. Cache rows are bf16 (any [batch, capacity, kv_heads, d] strides) or 4-bit codes with
// one bf16 scale per 32 elements (sink_cache4.cu has the layout). Bandwidth bound: each visible
// row is read once for all query heads that share it, and 4-bit rows are read as stored.
//
// A CTA takes one (sequence, key head, up to 16 query heads) and a share of its rows; the CTAs of a
// cluster split the rows of one (sequence, key head) and join their partial results over
// distributed shared memory, so there is one launch, no workspace and no atomics.
//   warp 4      lane 0 fills a ring of stages: 64 rows in 16-row TMA boxes (bf16), or bulk copies of 128
//               contiguous 4-bit rows and their scales
//   warps 0-3   16 rows of every 64 of a stage each, with their own running maximum and sum, on mma.sync
//               m16n8k16 (a tcgen05 tile would need 64 or 128 rows of queries, and the tensor
//               work is small beside the reads)
// Two more forms over bf16 rows: behind a shared prefix, whose partial results (prefix_attn.cu) the join takes
// in beside the cluster's; and with the rows' attention weights added up: a score goes to a workspace as
// it is computed, and after the join, when the heads' maxima and sums are known, each CTA takes its rows'
// probabilities from it (4 bytes per row and query head each way, mostly within L2, where recomputing
// them would read the keys again).
// bf16: S = Q K^T and O += P V with the query heads as the 16 rows.
// 4 bits: S^T = K Q^T and O^T += V^T P^T with the cache rows (the output elements) as the 16 rows and 8
// query heads as the columns, NQ times: what counts here is the instructions spent on unpacking and
// on P, and few heads leave no half-empty tiles this way. Keys: codes n, exact in f16, with Q in f16
// scaled by a power of two; a scale group's sum is multiplied by its scale in fp32. Values: codes n,
// exact in bf16 (P needs its range); the scale belongs to the summed-over row, so it multiplies P (in
// fp32, before P's rounding), and P's 8 x 8 blocks are transposed between the two products (movmatrix). The products' order of
// elements within a row is free, so a lane takes the elements that lie together in the stored
// words, and Q and O use the same order. The running maximum is followed only when a score exceeds
// it by 2^8, which one vote shows.
//
// Measured: 64 sequences of up to 16000 tokens, 16 / 4 heads of 128, window 4095, bf16: 73 us, 6.7 TB/s,
// a plain copy's rate. 32 sequences of 9001 to 32768 tokens, window 16383, 4 bits: 74 us, 3.8 TB/s:
// 46.5 M instructions, mostly to unpack codes (372 per 16 rows), that would take some 40 us at full issue;
// the issue slots are 59 % busy, since the CTAs are unequal and come in 1.7 waves, each with its fill and
// join. One sequence of 700 tokens, 12 heads of 64, window 511: 4.4 us, a launch, one load and the join.
// With weights, 64 sequences of 2049 to 4096 slots, 16 / 4 heads of 128: 77 us, 5.3 TB/s; the CTAs of long sequences
// outlast the others by some 10 us (a CTA's four warps take 64 rows in about half a microsecond, whatever the
// memory could give), and their weights come after that, 4 us. Behind a prefix, 64 sequences of up to 1000 own tokens: 20 us of
// that call's 42, the same end and the join of 19 parts.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "mma_frag.cuh"
#include "ptx_sm100.cuh"
#include "sa_internal.h"
#include "tma_host.h"

namespace sa {
namespace {

using frag::lds128;
using frag::ldsm_x4_t;
using frag::mma16816;
using frag::swz;

__device__ unsigned int g_decode_err;

constexpr int kWarps = 4;               // consumer warps
constexpr int kThreads = 32 * (kWarps + 1);
constexpr int kMaxStages = 8;
constexpr int kMaxCluster = 8;
constexpr int kMaxScoredGroup = kMaxScoredHeads;

// NQ: groups of 8 query heads of a CTA (2 in the bf16 form: one m-tile)
template <int D, bool Q4, int NQ>
struct Cfg {
  static constexpr int Q = 8 * NQ;                     // query heads
  // 16-row tiles of a consumer warp per stage (4 bits: 77 us with two in three stages, 84 with
  // one in six; 74 with the two unrolled)
  static constexpr int TILES = Q4 ? 2 : 1;
  static constexpr int ROWS = 16 * kWarps * TILES;     // cache rows per stage
  static constexpr int CH = D >= 64 ? 64 : 32;         // bf16: elements per swizzled row
  static constexpr int ROWB = CH * 2;
  static constexpr CUtensorMapSwizzle TMA_SWZ =
      ROWB == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B;
  static constexpr int NG = D / 32;                    // scale groups
  static constexpr int CODES = Q4 ? ROWS * D / 2 : ROWS * D * 2;   // K (or V) bytes of a stage
  static constexpr int SCALES = Q4 ? ROWS * NG * 2 : 0;
  static constexpr int STAGE = 2 * (CODES + SCALES);
  static constexpr int STAGES = Q4 ? (D == 128 ? 3 : 4) : (D == 128 ? 3 : (D == 64 ? 4 : 8));
  static constexpr int RING = STAGES * STAGE;
  // after the last stage the ring's memory holds the warps' partial results and the CTA's statistics
  static constexpr int MERGE = (kWarps * (D + 2) + 2) * Q * 4;
  static constexpr int SMEM = 1024 + (RING > MERGE ? RING : MERGE);
  // accumulators of a thread: [D / 8][4], n-tiles of the 16 heads, or [NQ * D / 16][4], m-tiles
  static constexpr int NT = Q4 ? NQ * D / 16 : D / 8;
  static_assert(STAGES <= kMaxStages && SMEM <= 227 * 1024, "shared memory");
};

// What a launch does besides: join the partial results of a shared prefix (prefix_attn.cu), or add up the
// attention weights of the rows.
enum : int { kPlain = 0, kBehindPrefix = 1, kScored = 2 };

struct DParams {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;                       // [batch][heads]
  const int32_t* lengths;
  const uint8_t* kc;                // 4-bit cache, [batch][kv_heads][capacity] rows
  const __nv_bfloat16* ks;
  const uint8_t* vc;
  const __nv_bfloat16* vs;
  int64_t q_sb, q_sh, o_sb, o_sh;
  int heads, kv_heads, group, head_groups, capacity, window, sinks;
  float scale_log2;
  // 0x000f000f, not known to the compiler: (w & mask) | bits is one instruction, but only with one constant
  // in it (4 bits: 220 -> 158 ALU instructions per 16 rows, 86 -> 77 us)
  uint32_t code_mask;
  // kBehindPrefix: n_parts partial results of row s group + e of a key head, in blocks (hk part_tiles + row / 128)
  // n_parts + part
  const float4* part_o;             // [block][D / 4][128]
  const float2* part_ml;            // [block][128]: m (log2 units), l
  int n_parts, part_tiles;
  // kScored
  float* scores;                    // [batch][kv_heads][head_groups][capacity][score_stride], log2 units
  const float* w_in;                // [batch][kv_heads][capacity]
  float* w_out;
  float decay;
  int score_stride;
};

struct Bars {
  uint64_t full[kMaxStages], empty[kMaxStages];
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait(bar, parity, abort_flag, &g_decode_err, kErrTimeout);
}

// The rows that a sequence's query sees, cut into units of 16 rows a warp: first those of the sinks that
// the window does not hold, then the window's, this CTA's share being [begin, end). A stage is up to
// TILES units.
constexpr int kUnit = 16 * kWarps;

template <int TILES, bool Q4>
struct Rows {
  int len, lo, n_sink;              // tokens; first token of the window; sinks before it
  int sink_units, first, begin, end;    // first: token of the window's first unit

  __device__ static Rows of(const DParams& p, int s, int rank, int ranks) {
    Rows r;
    r.len = max(0, min(p.lengths[s], p.capacity));
    r.lo = max(0, r.len - 1 - p.window);
    r.n_sink = min(p.sinks, r.lo);
    r.first = Q4 ? (r.lo & ~7) : r.lo;          // bulk copies start at a multiple of 16 bytes
    r.sink_units = (r.n_sink + kUnit - 1) / kUnit;
    const int total = r.sink_units + (r.len - r.first + kUnit - 1) / kUnit;
    // shares that differ by one unit at most (whole stages of two: 89 us where these take 86)
    r.begin = (int)((int64_t)total * rank / ranks);
    r.end = (int)((int64_t)total * (rank + 1) / ranks);
    return r;
  }
  // The stage that starts at unit j: its first row's token and the tokens [vlo, vhi) of it that are
  // seen; returns the next stage's unit.
  __device__ __forceinline__ int stage(int j, int& tok, int& vlo, int& vhi) const {
    const bool sinks = j < sink_units;
    const int next = TILES == 1 ? j + 1 : min(j + TILES, sinks ? min(sink_units, end) : end);
    if (sinks) {
      tok = j * kUnit;
      vlo = 0;
      vhi = n_sink;
    } else {
      tok = first + (j - sink_units) * kUnit;
      vlo = lo;
      vhi = len;
    }
    vhi = min(vhi, tok + (next - j) * kUnit);
    return next;
  }
};

template <int D, bool Q4, int NQ>
__device__ void producer(const DParams& p, const CUtensorMap* tk, const CUtensorMap* tv, Bars& bars, uint8_t* ring,
                         const Rows<Cfg<D, Q4, NQ>::TILES, Q4>& r, int s, int hk, volatile int* abort_flag) {
  using C = Cfg<D, Q4, NQ>;
  int g = 0;
  for (int j = r.begin; j < r.end; ++g) {
    const int st = g % C::STAGES;
    if (g >= C::STAGES && !wait_bar(&bars.empty[st], (uint32_t)(g / C::STAGES - 1) & 1u, abort_flag)) break;
    int tok, vlo, vhi;
    j = r.stage(j, tok, vlo, vhi);
    uint8_t* stage = ring + st * C::STAGE;
    if constexpr (Q4) {
      const int rows = min(C::ROWS, (vhi - tok + 7) & ~7);          // the capacity is a multiple of 8
      const int64_t row = ((int64_t)s * p.kv_heads + hk) * p.capacity + tok;
      mbar_arrive_expect_tx(&bars.full[st], (uint32_t)(rows * (D + 4 * C::NG)));
      bulk_load(stage, p.kc + row * (D / 2), rows * (D / 2), &bars.full[st]);
      bulk_load(stage + C::CODES, p.ks + row * C::NG, rows * C::NG * 2, &bars.full[st]);
      bulk_load(stage + C::CODES + C::SCALES, p.vc + row * (D / 2), rows * (D / 2), &bars.full[st]);
      bulk_load(stage + 2 * C::CODES + C::SCALES, p.vs + row * C::NG, rows * C::NG * 2, &bars.full[st]);
    } else {
      const int boxes = min(kWarps, (vhi - tok + 15) >> 4);       // tok >= vlo: every earlier box is seen
      mbar_arrive_expect_tx(&bars.full[st], (uint32_t)(boxes * 16 * D * 4));
      for (int b = 0; b < boxes; ++b)
#pragma unroll
        for (int c = 0; c < D / C::CH; ++c) {
          uint8_t* dst = stage + (c * C::ROWS + 16 * b) * C::ROWB;
          tma_load_4d(dst, tk, &bars.full[st], c * C::CH, hk, tok + 16 * b, s);
          tma_load_4d(dst + C::CODES, tv, &bars.full[st], c * C::CH, hk, tok + 16 * b, s);
        }
    }
  }
  // every copy of this CTA has landed before it goes on
  int never = 0;
  for (int t = max(0, g - C::STAGES); t < g; ++t)
    mbar_wait(&bars.full[t % C::STAGES], (uint32_t)(t / C::STAGES) & 1u, &never, &g_decode_err, kErrTimeout);
}

// Shared-memory address of 16-byte unit u of a stage's row (the TMA swizzle undone).
template <int D>
__device__ __forceinline__ uint32_t row_unit(uint32_t base, int row, int u) {
  if constexpr (D == 32) {
    return base + (uint32_t)(row * 64 + ((u ^ ((row >> 1) & 3)) << 4));
  } else {
    return swz(base + (uint32_t)((u >> 3) * Cfg<D, false, 2>::ROWS * 128), row, u & 7);
  }
}

__device__ __forceinline__ void ldsm_x4(uint32_t addr, uint32_t& r0, uint32_t& r1, uint32_t& r2, uint32_t& r3) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r0), "=r"(r1), "=r"(r2), "=r"(r3)
               : "r"(addr));
}

// Codes n + 8 (nibble S of the low and of the high half-word, 1 .. 15) as a bf16 pair of n: over
// the mantissa of 128 they are 136 + n. All exact. low: 0x000f000f.
template <int S>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t low) {
  const uint32_t x = ((w >> (4 * S)) & low) | 0x43004300u;
  const __nv_bfloat162 v = __hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), __floats2bfloat162_rn(136.f, 136.f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// The four pairs of a code word as f16 pairs of n: its ten bits of mantissa take two of the four
// nibbles where they stand, as 1032 + n and 1024 + 16 (n + 8), which one fma turns into n. All exact.
// high: 0x00f000f0.
__device__ __forceinline__ void code_halves(uint32_t w, uint32_t low, uint32_t high, uint32_t (&h)[4]) {
  const __half2 one = __floats2half2_rn(-1032.f, -1032.f), off = __floats2half2_rn(-72.f, -72.f);
  const __half2 sixteenth = __floats2half2_rn(0.0625f, 0.0625f);
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t x = ((k ? w >> 8 : w) & low) | 0x64006400u, y = ((k ? w >> 8 : w) & high) | 0x64006400u;
    const __half2 a = __hadd2(*reinterpret_cast<const __half2*>(&x), one);
    const __half2 b = __hfma2(*reinterpret_cast<const __half2*>(&y), sixteenth, off);
    h[2 * k] = *reinterpret_cast<const uint32_t*>(&a);
    h[2 * k + 1] = *reinterpret_cast<const uint32_t*>(&b);
  }
}

// D += A B in f16 with fp32 sums; FIRST: D = A B.
template <bool FIRST>
__device__ __forceinline__ void mma16816_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             const uint32_t (&b)[2]) {
  if constexpr (FIRST) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
        : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]), "f"(0.f));
  } else {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b[0]), "r"(b[1]));
  }
}

// Transpose of an 8 x 8 matrix of 16-bit elements, row lane / 4, columns 2 (lane % 4) and + 1.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int N>
__device__ __forceinline__ void lds_words(uint32_t addr, uint32_t (&w)[N]) {
  static_assert(N == 1 || N == 2 || N == 4, "words");
  if constexpr (N == 4) {
    const uint4 v = lds128(addr);
    w[0] = v.x; w[1] = v.y; w[2] = v.z; w[3] = v.w;
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(addr));
  } else {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  }
}

// A row's scales.
template <int NG>
__device__ __forceinline__ void load_scales(uint32_t addr, float (&sc)[NG]) {
  uint32_t w[(NG + 1) / 2];
  if constexpr (NG == 1) {
    asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w[0]) : "r"(addr));
  } else {
    lds_words<NG / 2>(addr, w);
  }
#pragma unroll
  for (int c = 0; c < NG; ++c) sc[c] = __uint_as_float(c & 1 ? w[c >> 1] & 0xffff0000u : w[c >> 1] << 16);
}

// 4-bit form. m, l: per query head 8 q + 2 t + e of lane (g, t), m the same in all g, l this lane's rows.
template <int D, int NQ>
__device__ void consumer4(const DParams& p, Bars& bars, uint8_t* ring, const Rows<Cfg<D, true, NQ>::TILES, true>& r, int s,
                          int h0, int n_q, float (&o)[NQ * D / 16][4], float (&m)[2 * NQ], float (&l)[2 * NQ],
                          volatile int* abort_flag) {
  using C = Cfg<D, true, NQ>;
  constexpr int NG = C::NG;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const float kNegInf = __int_as_float(0xff800000);
  // Q^T as f16 B fragments (absent heads are zero). A head's elements are first taken times the power of
  // two that brings the largest to [2^9, 2^10): bf16's 8 bits fit f16's 11, and what falls below
  // f16's last place is 2^-34 of the largest. The power comes back with the softmax scale.
  uint32_t qb[NQ][2 * NG][2];
  float c[2 * NQ], thr[2 * NQ];      // softmax scale of the lane's heads; score beyond which m follows
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const __nv_bfloat16* qr = p.q + (int64_t)s * p.q_sb + (int64_t)(h0 + 8 * q + g) * p.q_sh;
    uint4 w[NG];
    uint32_t top = 0u;
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      w[i] = make_uint4(0u, 0u, 0u, 0u);
      if (8 * q + g < n_q) w[i] = *reinterpret_cast<const uint4*>(qr + 32 * i + 8 * t);
      constexpr uint32_t kAbs = 0x7fff7fffu;
      top = __vmaxu2(top, __vmaxu2(__vmaxu2(w[i].x & kAbs, w[i].y & kAbs), __vmaxu2(w[i].z & kAbs, w[i].w & kAbs)));
    }
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));           // head g
    // exponent field of the largest magnitude (at least that of 2^-90, so that the powers are numbers)
    const int e = max((int)(max(top & 0xffffu, top >> 16) >> 7), 37);
    const float up = __int_as_float((127 + 9 + 127 - e) << 23), back = __int_as_float((e - 9) << 23);
#pragma unroll
    for (int i = 0; i < NG; ++i) {
      const uint32_t v[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const __half2 h = __floats2half2_rn(__uint_as_float(v[k] << 16) * up, __uint_as_float(v[k] & 0xffff0000u) * up);
        qb[q][2 * i + (k >> 1)][k & 1] = *reinterpret_cast<const uint32_t*>(&h);
      }
    }
    // (at least the smallest number: a key that is not seen has the score -inf, and -inf times 0 is NaN)
    const float tiny = __int_as_float(1);
    c[2 * q] = fmaxf(p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t), tiny);
    c[2 * q + 1] = fmaxf(p.scale_log2 * __shfl_sync(0xffffffffu, back, 8 * t + 4), tiny);
    thr[2 * q] = thr[2 * q + 1] = kNegInf;
  }
  // The tile's row x (of both products) is cache row x / 2 + 4 (x % 2) of its half: the value rows of the
  // lanes that load together are then neighbours and conflict in pairs, not all four (94.5 -> 89 us).
  const int gr = (g >> 1) + 4 * (g & 1);
  // this lane's places in a stage: key words, scales of rows g, value words
  const uint32_t ring0 = smem_u32(ring);
  const uint32_t at_k = (uint32_t)((16 * warp + gr) * (D / 2) + t * (D / 8));
  const uint32_t at_s = (uint32_t)(C::CODES + (16 * warp + gr) * NG * 2);
  const uint32_t at_v = (uint32_t)(C::CODES + C::SCALES + (16 * warp + t) * (D / 2) + (g >> 1) * (D / 8));
  const uint32_t sel = g & 1 ? 0x7531u : 0x6420u;
  const uint32_t low = p.code_mask, high = p.code_mask << 4;
  for (int j = r.begin, n = 0; j < r.end; ++n) {
    const int st = n % C::STAGES;
    int tok, vlo, vhi;
    j = r.stage(j, tok, vlo, vhi);
    if (!__all_sync(0xffffffffu, wait_bar(&bars.full[st], (uint32_t)(n / C::STAGES) & 1u, abort_flag))) return;
    const uint32_t stage = ring0 + (uint32_t)(st * C::STAGE);
#pragma unroll
    for (int x = 0; x < C::TILES; ++x) {
      const int t0 = tok + kUnit * x + 16 * warp;
      if (t0 >= vhi || t0 + 16 <= vlo) continue;
      const uint32_t kb = stage + at_k + (uint32_t)(x * kUnit * (D / 2));
      const uint32_t sb = stage + at_s + (uint32_t)(x * kUnit * NG * 2);
      const uint32_t vb = stage + at_v + (uint32_t)(x * kUnit * (D / 2));
      // ---- scores of rows g and g + 8
      uint32_t w0[NG], w1[NG];
      lds_words<NG>(kb, w0);
      lds_words<NG>(kb + 8 * (D / 2), w1);
      float k0[NG], k1[NG];
      load_scales<NG>(sb, k0);
      load_scales<NG>(sb + 16 * NG, k1);
      float sc[NQ][4];
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        uint32_t a[4], b[4];
        code_halves(w0[i], low, high, a);
        code_halves(w1[i], low, high, b);
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          float acc[4];
          mma16816_f16<true>(acc, a[0], b[0], a[1], b[1], qb[q][2 * i]);
          mma16816_f16<false>(acc, a[2], b[2], a[3], b[3], qb[q][2 * i + 1]);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float k = e < 2 ? k0[i] : k1[i];
            sc[q][e] = i == 0 ? acc[e] * k : fmaf(acc[e], k, sc[q][e]);
          }
        }
      }
      float v0[NG], v1[NG];
      load_scales<NG>(sb + C::CODES + C::SCALES, v0);
      load_scales<NG>(sb + C::CODES + C::SCALES + 16 * NG, v1);
      if (t0 < vlo || t0 + 16 > vhi) {
        // rows that are not seen: no score, and zeros for whatever their scales hold
        const bool on0 = t0 + gr >= vlo && t0 + gr < vhi, on1 = t0 + 8 + gr >= vlo && t0 + 8 + gr < vhi;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[q][e] = (e < 2 ? on0 : on1) ? sc[q][e] : kNegInf;
#pragma unroll
        for (int i = 0; i < NG; ++i) {
          v0[i] = on0 ? v0[i] : 0.f;
          v1[i] = on1 ? v1[i] : 0.f;
        }
      }
      // ---- the running maximum: a tile has a row that is seen, so m is a number afterwards
      bool grow = false;
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) grow = grow || sc[q][e] > thr[2 * q + (e & 1)];
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int q = 0; q < NQ; ++q)
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int h = 2 * q + e;
            float mx = fmaxf(sc[q][e], sc[q][e + 2]);
#pragma unroll
            for (int y = 4; y < 32; y *= 2) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, y));
            if (mx > thr[h]) {
              const float a = ex2_approx(m[h] - mx * c[h]);           // 0 from -inf
              m[h] = mx * c[h];
              thr[h] = mx + 8.f / c[h];
              l[h] *= a;
#pragma unroll
              for (int y = 0; y < D / 16; ++y) {
                o[q * (D / 16) + y][e] *= a;
                o[q * (D / 16) + y][e + 2] *= a;
              }
            }
          }
      }
#pragma unroll
      for (int q = 0; q < NQ; ++q)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[q][e] = ex2_approx(fmaf(sc[q][e], c[2 * q + (e & 1)], -m[2 * q + (e & 1)]));
          l[2 * q + (e & 1)] += sc[q][e];
        }
      // ---- values: words (g / 2, i) of the tile's rows 2 t, 2 t + 1, 2 t + 8, 2 t + 9; byte pair g % 2 of each holds
      // this lane's elements 32 i + 4 g + {0, 2, 1, 3} (nibbles 0 .. 3 after the byte selection)
      uint32_t w[4][NG];
#pragma unroll
      for (int k = 0; k < 4; ++k) lds_words<NG>(vb + (uint32_t)(4 * k * (D / 2)), w[k]);
#pragma unroll
      for (int i = 0; i < NG; ++i) {
        const uint32_t x0 = __byte_perm(w[0][i], w[1][i], sel), x1 = __byte_perm(w[2][i], w[3][i], sel);
        const uint32_t a0[4] = {code_pair<0>(x0, low), code_pair<1>(x0, low), code_pair<0>(x1, low), code_pair<1>(x1, low)};
        const uint32_t a1[4] = {code_pair<2>(x0, low), code_pair<3>(x0, low), code_pair<2>(x1, low), code_pair<3>(x1, low)};
#pragma unroll
        for (int q = 0; q < NQ; ++q) {
          const uint32_t b0 = transpose8(pack_bf16x2(sc[q][0] * v0[i], sc[q][1] * v0[i]));
          const uint32_t b1 = transpose8(pack_bf16x2(sc[q][2] * v1[i], sc[q][3] * v1[i]));
          mma16816(o[q * (D / 16) + 2 * i], a0, b0, b1);
          mma16816(o[q * (D / 16) + 2 * i + 1], a1, b0, b1);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.empty[st]);
  }
}

// bf16 form. m, l: per query head g + 8 h of lane (g, t), l this lane's columns.
// kScored: `scores` takes the scores of the CTA's heads, [capacity][score_stride].
template <int D, int MODE>
__device__ void consumer16(const DParams& p, Bars& bars, uint8_t* ring, const Rows<1, false>& r, int s, int h0, int n_q,
                           float* scores, float (&o)[D / 8][4], float (&m)[2], float (&l)[2], volatile int* abort_flag) {
  using C = Cfg<D, false, 2>;
  constexpr int KS = D / 16;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  const float kNegInf = __int_as_float(0xff800000);
  const float c = p.scale_log2;
  // Q as A fragments: rows g and g + 8 (absent heads are zero)
  uint32_t qa[KS][4];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    const int row = g + 8 * half;
    const __nv_bfloat16* qr = p.q + (int64_t)s * p.q_sb + (int64_t)(h0 + row) * p.q_sh;
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      const __nv_bfloat16* at = qr + 16 * k + 2 * t;
      qa[k][half] = row < n_q ? *reinterpret_cast<const uint32_t*>(at) : 0u;
      qa[k][half + 2] = row < n_q ? *reinterpret_cast<const uint32_t*>(at + 8) : 0u;
    }
  }
  const uint32_t ring0 = smem_u32(ring);
  for (int j = r.begin, n = 0; j < r.end; ++n) {
    const int st = n % C::STAGES;
    int tok, vlo, vhi;
    j = r.stage(j, tok, vlo, vhi);
    if (!__all_sync(0xffffffffu, wait_bar(&bars.full[st], (uint32_t)(n / C::STAGES) & 1u, abort_flag))) return;
    const int t0 = tok + 16 * warp;
    if (t0 < vhi && t0 + 16 > vlo) {
      const uint32_t kb = ring0 + (uint32_t)(st * C::STAGE);
      const uint32_t vb = kb + C::CODES + C::SCALES;
      const int row0 = 16 * warp;
      // rows of this lane's score columns: 8 nt + 2 t + e
      bool on[2][2];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = t0 + 8 * nt + 2 * t + e;
          on[nt][e] = at >= vlo && at < vhi;
        }
      float sc[2][4];
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = 0.f;
      {
        const int mi = lane >> 3;
        const int row = row0 + (lane & 7) + ((mi >> 1) << 3);
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4(row_unit<D>(kb, row, 2 * ks + (mi & 1)), b0, b1, b2, b3);
          mma16816(sc[0], qa[ks], b0, b1);
          mma16816(sc[1], qa[ks], b2, b3);
        }
      }
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) sc[nt][e] = on[nt][e & 1] ? sc[nt][e] * c : kNegInf;
      if constexpr (MODE == kScored) {
#pragma unroll
        for (int nt = 0; nt < 2; ++nt)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const int head = g + 8 * (e >> 1);
            if (head < n_q && on[nt][e & 1])
              scores[(int64_t)(t0 + 8 * nt + 2 * t + (e & 1)) * p.score_stride + head] = sc[nt][e];
          }
      }
      // running maximum of rows g (half 0) and g + 8; O and l follow it only when it grows by 2^8
      float mx[2];
      bool grow = false;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        mx[h] = fmaxf(fmaxf(sc[0][2 * h], sc[0][2 * h + 1]), fmaxf(sc[1][2 * h], sc[1][2 * h + 1]));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
        mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
        grow = grow || mx[h] > m[h] + 8.f;
      }
      if (__any_sync(0xffffffffu, grow)) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (mx[h] > m[h] + 8.f) {
            const float a = ex2_approx(m[h] - mx[h]);             // 0 from -inf
            m[h] = mx[h];
            l[h] *= a;
#pragma unroll
            for (int i = 0; i < D / 8; ++i) {
              o[i][2 * h] *= a;
              o[i][2 * h + 1] *= a;
            }
          }
        }
      }
      const float ref[2] = {m[0] == kNegInf ? 0.f : m[0], m[1] == kNegInf ? 0.f : m[1]};
#pragma unroll
      for (int nt = 0; nt < 2; ++nt)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sc[nt][e] = ex2_approx(sc[nt][e] - ref[e >> 1]);
          l[e >> 1] += sc[nt][e];
        }
      {
        const uint32_t pa[4] = {pack_bf16x2(sc[0][0], sc[0][1]), pack_bf16x2(sc[0][2], sc[0][3]),
                                pack_bf16x2(sc[1][0], sc[1][1]), pack_bf16x2(sc[1][2], sc[1][3])};
        const int mi = lane >> 3;
        const int row = row0 + (lane & 7) + ((mi & 1) << 3);
        // rows that are not seen count as zeros, whatever they hold (0 x NaN is NaN)
        const bool whole = t0 >= vlo && t0 + 16 <= vhi;
        const uint32_t k0 = (on[0][0] ? 0xffffu : 0u) | (on[0][1] ? 0xffff0000u : 0u);
        const uint32_t k1 = (on[1][0] ? 0xffffu : 0u) | (on[1][1] ? 0xffff0000u : 0u);
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
          uint32_t b0, b1, b2, b3;
          ldsm_x4_t(row_unit<D>(vb, row, 2 * i + (mi >> 1)), b0, b1, b2, b3);
          if (!whole) {
            b0 &= k0;
            b1 &= k1;
            b2 &= k0;
            b3 &= k1;
          }
          mma16816(o[2 * i], pa, b0, b1);
          mma16816(o[2 * i + 1], pa, b2, b3);
        }
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.empty[st]);
  }
}

// The cluster's partial results (cm, cl, wo of every rank) and the prefix's, for this rank's share of the elements. The
// factors 2^(m_k - M) of all parts come first, a (query head, part) a thread, so that the parts' elements are then
// loaded without a wait between them (64 sequences, 19 parts: 31 us for the launch with a thread walking the parts
// alone).
template <int D>
__device__ __forceinline__ void join_prefix(const DParams& p, cooperative_groups::cluster_group& cluster, float* cm, float* cl,
                                            float* wo, int rank, int ranks, int s, int hk, int hg, int h0, int n_q) {
  constexpr int kQ = 16, kFactors = 32;                    // parts at a time
  const float kNegInf = __int_as_float(0xff800000);
  __shared__ float fm[kQ][kMaxCluster + kFactors];         // maxima, then factors: the ranks', then the parts'
  __shared__ float fl[kQ][kMaxCluster + kFactors];
  __shared__ float top[kQ], sum[kQ];
  const auto block_of = [&](int q, int k) {                 // and the row's place in it
    const int row = s * p.group + hg * kQ + q;
    return make_int2((hk * p.part_tiles + row / 128) * p.n_parts + k, row % 128);
  };
  const int c0 = rank * (D / 4) / ranks, c1 = (rank + 1) * (D / 4) / ranks;    // this rank's columns, four at a time
  const int share = n_q * (c1 - c0);
  constexpr int kEach = (kQ * (D / 4) + kThreads - 1) / kThreads;
  float4 acc[kEach];
#pragma unroll
  for (int x = 0; x < kEach; ++x) acc[x] = make_float4(0.f, 0.f, 0.f, 0.f);
  if (threadIdx.x < kQ) {
    top[threadIdx.x] = kNegInf;
    sum[threadIdx.x] = 0.f;
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");       // the prefix's results
  // several rounds where there are more parts than factors; the ranks' own come with the first
#pragma unroll 1
  for (int k0 = 0; k0 < p.n_parts; k0 += kFactors) {
    const int n = min(kFactors, p.n_parts - k0), own = k0 == 0 ? ranks : 0, all = own + n;
    __syncthreads();
    for (int i = threadIdx.x; i < n_q * all; i += kThreads) {
      const int q = i / all, k = i % all;
      if (k < own) {
        fm[q][k] = *cluster.map_shared_rank(cm + q, k);
        fl[q][k] = *cluster.map_shared_rank(cl + q, k);
      } else {
        const int2 at = block_of(q, k0 + k - own);
        const float2 ml = p.part_ml[(int64_t)at.x * 128 + at.y];
        fm[q][k] = ml.x;
        fl[q][k] = ml.y;
      }
    }
    __syncthreads();
    float back[kEach];                                     // of what has been added up so far
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int q = (threadIdx.x + x * kThreads) % n_q;
      back[x] = 1.f;
      if (k0 > 0) {
        float M = top[q];
        for (int k = 0; k < all; ++k) M = fmaxf(M, fm[q][k]);
        back[x] = ex2_approx(top[q] - M);
      }
    }
    __syncthreads();
    if (threadIdx.x < n_q) {
      const int q = threadIdx.x;
      float M = top[q];
      for (int k = 0; k < all; ++k) M = fmaxf(M, fm[q][k]);
      // M is a number, as the prefix's maxima are (half_softmax.cuh); the ranks' may be -inf
      float L = sum[q] * ex2_approx(top[q] - M);
      for (int k = 0; k < all; ++k) {
        const float a = ex2_approx(fm[q][k] - M);
        fm[q][k] = a;
        L = fmaf(a, fl[q][k], L);
      }
      top[q] = M;
      sum[q] = L;
    }
    __syncthreads();
#pragma unroll
    for (int x = 0; x < kEach; ++x) {
      const int i = threadIdx.x + x * kThreads;
      if (i >= share) continue;
      const int q = i % n_q, col = 4 * (c0 + i / n_q);     // neighbouring rows lie together
      float4 v = acc[x];
      v.x *= back[x];
      v.y *= back[x];
      v.z *= back[x];
      v.w *= back[x];
      const auto add = [&](float a, const float4& y) {
        v.x = fmaf(a, y.x, v.x);
        v.y = fmaf(a, y.y, v.y);
        v.z = fmaf(a, y.z, v.z);
        v.w = fmaf(a, y.w, v.w);
      };
      for (int k = 0; k < own; ++k)
        add(fm[q][k], *reinterpret_cast<const float4*>(cluster.map_shared_rank(wo + q * D + col, k)));
      const int2 it = block_of(q, k0);
      const float4* at = p.part_o + ((int64_t)it.x * (D / 4) + col / 4) * 128 + it.y;
#pragma unroll 8
      for (int k = 0; k < n; ++k) add(fm[q][own + k], at[(int64_t)k * (D / 4) * 128]);
      acc[x] = v;
    }
  }
#pragma unroll
  for (int x = 0; x < kEach; ++x) {
    const int i = threadIdx.x + x * kThreads;
    if (i >= share) continue;
    const int q = i % n_q, col = 4 * (c0 + i / n_q);
    const float L = sum[q], inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint2*>(p.o + (int64_t)s * p.o_sb + (int64_t)(h0 + q) * p.o_sh + col) =
        make_uint2(pack_bf16x2(acc[x].x * inv, acc[x].y * inv), pack_bf16x2(acc[x].z * inv, acc[x].w * inv));
    if (col == 0)
      p.lse[(int64_t)s * p.heads + h0 + q] = L == 0.f ? kNegInf : (top[q] + __log2f(L)) * 0.69314718055994531f;
  }
}

// Weights of rows begin, begin + step, .. below end of a (sequence, key head), whose query heads have maxima hm and inverse
// sums hi. Several rows' scores are loaded at once: one after the other they took a third of the call (64
// sequences of 2049 to 4096 slots).
template <int STRIDE>
__device__ __forceinline__ void add_weights(const DParams& p, int64_t list, int begin, int end, int step, const float* hm,
                                            const float* hi) {
  constexpr int kRows = STRIDE >= 8 ? 32 / STRIDE : 8, kLoad = STRIDE < 4 ? STRIDE : 4;
#pragma unroll 1
  for (int j0 = begin; j0 < end; j0 += kRows * step) {
    float w[kRows], old[kRows];
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      const int j = j0 + x * step;
      w[x] = 0.f;
      old[x] = p.decay != 0.f && j < end ? p.w_in[list * p.capacity + j] : 0.f;
    }
#pragma unroll 1
    for (int g0 = 0; g0 < p.head_groups; ++g0) {
      const float* sc = p.scores + (list * p.head_groups + g0) * p.capacity * STRIDE;
      const int n = min(16, p.group - g0 * 16);
      float v[kRows][STRIDE];
#pragma unroll
      for (int x = 0; x < kRows; ++x) {
        const int j = j0 + x * step;
#pragma unroll
        for (int q = 0; q < STRIDE; q += kLoad) {
          const float* at = sc + (int64_t)j * STRIDE + q;
          if (j >= end) continue;
          if constexpr (kLoad == 4) {
            const float4 y = *reinterpret_cast<const float4*>(at);
            v[x][q] = y.x;
            v[x][q + 1] = y.y;
            v[x][q + 2] = y.z;
            v[x][q + 3] = y.w;
          } else if constexpr (kLoad == 2) {
            const float2 y = *reinterpret_cast<const float2*>(at);
            v[x][q] = y.x;
            v[x][q + 1] = y.y;
          } else {
            v[x][q] = *at;
          }
        }
      }
#pragma unroll
      for (int x = 0; x < kRows; ++x)
#pragma unroll
        for (int q = 0; q < STRIDE; ++q)               // places past the last head were never written
          if (q < n) w[x] = fmaf(ex2_approx(v[x][q] - hm[g0 * 16 + q]), hi[g0 * 16 + q], w[x]);
    }
#pragma unroll
    for (int x = 0; x < kRows; ++x) {
      const int j = j0 + x * step;
      if (j < end) p.w_out[list * p.capacity + j] = fmaf(p.decay, old[x], w[x]);
    }
  }
}

// 4 bits, up to 8 query heads: four CTAs an SM (74 us; three with longer rings 80, five with shorter ones
// and 80 registers 90 to 109).
template <int D, bool Q4, int NQ, int MODE>
__global__ void __launch_bounds__(kThreads, Q4 && NQ == 1 ? 4 : (MODE != kPlain ? 2 : 1)) sink_decode_kernel(const __grid_constant__ CUtensorMap tk,
                                                               const __grid_constant__ CUtensorMap tv,
                                                               const __grid_constant__ DParams p) {
  using C = Cfg<D, Q4, NQ>;
  namespace cg = cooperative_groups;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ Bars bars;
  __shared__ int abort_flag;
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, ranks = gridDim.x;          // the cluster spans the grid's x (and the head groups: kScored)
  const int s = blockIdx.z, hk = blockIdx.y / p.head_groups, hg = blockIdx.y % p.head_groups;
  constexpr int kQ = C::Q;
  const int h0 = hk * p.group + hg * kQ;
  const int n_q = min(kQ, p.group - hg * kQ);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const float kNegInf = __int_as_float(0xff800000);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::STAGES; ++i) {
      mbar_init(&bars.full[i], 1);
      mbar_init(&bars.empty[i], kWarps);
    }
    abort_flag = 0;
    fence_mbar_init();
  }
  __syncthreads();
  const auto r = Rows<C::TILES, Q4>::of(p, s, rank, ranks);
  float o[C::NT][4];
  constexpr int NM = Q4 ? 2 * NQ : 2;                       // query heads of a lane
  float m[NM], l[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    m[i] = kNegInf;
    l[i] = 0.f;
  }
#pragma unroll
  for (int i = 0; i < C::NT; ++i)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[i][e] = 0.f;
  if (warp == kWarps) {
    if (lane == 0) producer<D, Q4, NQ>(p, &tk, &tv, bars, ring, r, s, hk, &abort_flag);
    __syncwarp();
  } else {
    if constexpr (Q4) consumer4<D, NQ>(p, bars, ring, r, s, h0, n_q, o, m, l, &abort_flag);
    else {
      float* scores = nullptr;
      if constexpr (MODE == kScored)
        scores = p.scores + (((int64_t)s * p.kv_heads + hk) * p.head_groups + hg) * p.capacity * p.score_stride;
      consumer16<D, MODE>(p, bars, ring, r, s, h0, n_q, scores, o, m, l, &abort_flag);
    }
  }
  __syncthreads();                                          // the ring is free
  // ---- the warps' partial results: O [warp][query][D], maxima and sums
  float* wo = reinterpret_cast<float*>(ring);
  float* wm = wo + kWarps * kQ * D;
  float* wl = wm + kWarps * kQ;
  if (warp < kWarps) {
    const int g = lane >> 2, t = lane & 3;
#pragma unroll
    for (int h = 0; h < NM; ++h) {
      // the sums over the lanes that share the head; one of them writes
#pragma unroll
      for (int x = Q4 ? 4 : 1; x < (Q4 ? 32 : 4); x *= 2) l[h] += __shfl_xor_sync(0xffffffffu, l[h], x);
      const int row = Q4 ? 8 * (h >> 1) + 2 * t + (h & 1) : g + 8 * h;
      if (row < n_q) {
        if ((Q4 ? g : t) == 0) {
          wm[warp * kQ + row] = m[h];
          wl[warp * kQ + row] = l[h];
        }
        float* dst = wo + (warp * kQ + row) * D;
        if constexpr (Q4) {
          // rows g and g + 8 of m-tile x: elements 32 (x / 2) + 4 g + {0, 2} or {1, 3}
#pragma unroll
          for (int x = 0; x < D / 16; ++x) {
            dst[32 * (x >> 1) + 4 * g + (x & 1)] = o[(h >> 1) * (D / 16) + x][h & 1];
            dst[32 * (x >> 1) + 4 * g + 2 + (x & 1)] = o[(h >> 1) * (D / 16) + x][2 + (h & 1)];
          }
        } else {
#pragma unroll
          for (int i = 0; i < C::NT; ++i) *reinterpret_cast<float2*>(dst + 8 * i + 2 * t) = make_float2(o[i][2 * h], o[i][2 * h + 1]);
        }
      }
    }
  }
  __syncthreads();
  // ---- one partial result per CTA: O in warp 0's place, its maxima and sums behind the warps'
  float* cm = wl + kWarps * kQ;
  float* cl = cm + kQ;
  for (int at = threadIdx.x; at < n_q * (D / 4); at += kThreads) {
    const int row = at / (D / 4), col = 4 * (at % (D / 4));
    float a[kWarps], M = kNegInf, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a[w] = wm[w * kQ + row];
      M = fmaxf(M, a[w]);
    }
    float4 sum = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      a[w] = M != kNegInf ? ex2_approx(a[w] - M) : 1.f;     // without a maximum the sums are zero, or NaN
      const float4 v = *reinterpret_cast<const float4*>(wo + (w * kQ + row) * D + col);
      sum.x = fmaf(a[w], v.x, sum.x);
      sum.y = fmaf(a[w], v.y, sum.y);
      sum.z = fmaf(a[w], v.z, sum.z);
      sum.w = fmaf(a[w], v.w, sum.w);
      L = fmaf(a[w], wl[w * kQ + row], L);
    }
    *reinterpret_cast<float4*>(wo + row * D + col) = sum;
    if (col == 0) {
      cm[row] = M;
      cl[row] = L;
    }
  }
  cluster.sync();
  // ---- the cluster's CTAs join their results: CTA `rank` writes its share of the elements. All the
  // remote loads go out together: one trip's latency, not one per CTA.
  if constexpr (MODE == kBehindPrefix) {
    join_prefix<D>(p, cluster, cm, cl, wo, rank, ranks, s, hk, hg, h0, n_q);
    cluster.sync();                                         // no CTA leaves while another reads its results
    return;
  }
  const int first = MODE == kScored ? hg * ranks : 0;       // this head group's first CTA
  const int pairs = n_q * (D / 2);
  const int p0 = (int)((int64_t)pairs * rank / ranks), p1 = (int)((int64_t)pairs * (rank + 1) / ranks);
  for (int at = p0 + threadIdx.x; at < p1; at += kThreads) {
    const int row = at / (D / 2), col = 2 * (at % (D / 2));
    float mk[kMaxCluster], lk[kMaxCluster];
    float2 v[kMaxCluster];
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      mk[k] = kNegInf;
      lk[k] = 0.f;
      v[k] = make_float2(0.f, 0.f);
      if (k < ranks) {
        mk[k] = *cluster.map_shared_rank(cm + row, first + k);
        lk[k] = *cluster.map_shared_rank(cl + row, first + k);
        v[k] = *reinterpret_cast<const float2*>(cluster.map_shared_rank(wo + row * D + col, first + k));
      }
    }
    float M = kNegInf;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) M = fmaxf(M, mk[k]);
    float x = 0.f, y = 0.f, L = 0.f;
#pragma unroll
    for (int k = 0; k < kMaxCluster; ++k) {
      const float a = M != kNegInf ? ex2_approx(mk[k] - M) : 1.f;
      x = fmaf(a, v[k].x, x);
      y = fmaf(a, v[k].y, y);
      L = fmaf(a, lk[k], L);
    }
    // L is 0 where no key is seen, and NaN where a score that is seen is (no maximum follows a NaN)
    const float inv = L == 0.f ? 0.f : 1.f / L;
    *reinterpret_cast<uint32_t*>(p.o + (int64_t)s * p.o_sb + (int64_t)(h0 + row) * p.o_sh + col) =
        pack_bf16x2(x * inv, y * inv);
    if (col == 0)
      p.lse[(int64_t)s * p.heads + h0 + row] = L == 0.f ? kNegInf : (M + __log2f(L)) * 0.69314718055994531f;
  }
  if constexpr (MODE == kScored) {
    // ---- the weights of this CTA's rows: maxima and sums of all of the key head's query heads, then a row a
    // thread. The head groups' CTAs of one rank have the same rows and share them out.
    __shared__ float hm[kMaxScoredGroup], hi[kMaxScoredGroup];
    for (int q = threadIdx.x; q < p.group; q += kThreads) {
      float M = kNegInf, L = 0.f;
      for (int k = 0; k < ranks; ++k) M = fmaxf(M, *cluster.map_shared_rank(cm + q % kQ, q / kQ * ranks + k));
      for (int k = 0; k < ranks; ++k) {
        const float mk = *cluster.map_shared_rank(cm + q % kQ, q / kQ * ranks + k);
        L = fmaf(M != kNegInf ? ex2_approx(mk - M) : 1.f, *cluster.map_shared_rank(cl + q % kQ, q / kQ * ranks + k), L);
      }
      // a head without a finite score adds nothing, as its O is 0; L is NaN where a score is
      hm[q] = M != kNegInf ? M : 0.f;
      hi[q] = L == 0.f ? 0.f : 1.f / L;
    }
    __syncthreads();
    const int64_t list = (int64_t)s * p.kv_heads + hk;
    const int begin = r.begin * kUnit + hg * kThreads + (int)threadIdx.x, end = min(r.len, r.end * kUnit);
    const int step = p.head_groups * kThreads;
    switch (p.score_stride) {
      case 1: add_weights<1>(p, list, begin, end, step, hm, hi); break;
      case 2: add_weights<2>(p, list, begin, end, step, hm, hi); break;
      case 4: add_weights<4>(p, list, begin, end, step, hm, hi); break;
      case 8: add_weights<8>(p, list, begin, end, step, hm, hi); break;
      default: add_weights<16>(p, list, begin, end, step, hm, hi);
    }
  }
  cluster.sync();                                           // no CTA leaves while another reads its results
}

template <int D, bool Q4, int NQ, int MODE>
int launch(const SinkDecodeArgs& a, cudaStream_t stream) {
  using C = Cfg<D, Q4, NQ>;
  CUtensorMap tk, tv;
  memset(&tk, 0, sizeof(tk));
  memset(&tv, 0, sizeof(tv));
  if (!Q4 &&
      (!encode_bhnd_map(&tk, a.k, a.batch, a.capacity, a.kv_heads, D, a.k_strides[0], a.k_strides[1], a.k_strides[2],
                        C::CH, 16, C::TMA_SWZ) ||
       !encode_bhnd_map(&tv, a.v, a.batch, a.capacity, a.kv_heads, D, a.v_strides[0], a.v_strides[1], a.v_strides[2],
                        C::CH, 16, C::TMA_SWZ)))
    return SA_ERR_UNSUPPORTED;
  DParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const __nv_bfloat16*>(a.q);
  p.o = static_cast<__nv_bfloat16*>(a.o);
  p.lse = a.lse;
  p.lengths = a.lengths;
  if (Q4) {
    p.kc = static_cast<const uint8_t*>(a.k);
    p.ks = static_cast<const __nv_bfloat16*>(a.k_scales);
    p.vc = static_cast<const uint8_t*>(a.v);
    p.vs = static_cast<const __nv_bfloat16*>(a.v_scales);
  }
  p.q_sb = a.q_strides[0];
  p.q_sh = a.q_strides[2];
  p.o_sb = a.o_strides[0];
  p.o_sh = a.o_strides[2];
  p.heads = a.heads;
  p.kv_heads = a.kv_heads;
  p.group = a.heads / a.kv_heads;
  p.head_groups = (p.group + C::Q - 1) / C::Q;
  p.capacity = a.capacity;
  p.window = a.window;
  p.sinks = a.sinks;
  p.scale_log2 = a.softmax_scale * 1.4426950408889634f;
  p.code_mask = 0x000f000fu;
  if (MODE == kBehindPrefix) {
    p.part_o = static_cast<const float4*>(a.part_o);
    p.part_ml = static_cast<const float2*>(a.part_ml);
    p.n_parts = a.n_parts;
    p.part_tiles = a.part_tiles;
  }
  if (MODE == kScored) {
    p.scores = a.scores;
    p.w_in = a.weights_in;
    p.w_out = a.weights_out;
    p.decay = a.decay;
    p.score_stride = scored_stride(a.heads, a.kv_heads);
  }
  const auto kern = sink_decode_kernel<D, Q4, NQ, MODE>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) != cudaSuccess)
    return SA_ERR_CUDA;
  // CTAs per (sequence, key head), while each has a stage of rows when the cache is full: bf16 until
  // there are 1.5 per SM (its loads then saturate the memory; 64 sequences of 4 key heads: 73.8 us
  // with one, 79.6 with two, 88 with four), 4 bits, bound by its instructions, until there are 6 (32
  // sequences of 4 key heads: 107 us with two, 95 with four, 86 with eight; the last two are 3.4
  // and 6.7 per SM).
  const int64_t base = (int64_t)a.batch * a.kv_heads * p.head_groups;
  const int64_t seen = (int64_t)a.window + 1 + a.sinks < a.capacity ? (int64_t)a.window + 1 + a.sinks : a.capacity;
  const int sm_count = current_sm_count();
  int ranks = 1;
  const int most = MODE == kScored ? kMaxCluster / p.head_groups : kMaxCluster;
  while (2 * ranks <= most && 2 * base * ranks < (Q4 ? 12 : 3) * sm_count && seen >= 2 * kUnit * ranks) ranks *= 2;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)ranks, (unsigned)(a.kv_heads * p.head_groups), (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  memset(attr, 0, sizeof(attr));
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = MODE == kScored ? (unsigned)p.head_groups : 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (MODE == kBehindPrefix) {
    // its CTAs may start as the prefix's leave; they read its results after griddepcontrol.wait
    attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[1].val.programmaticStreamSerializationAllowed = 1;
    cfg.numAttrs = 2;
  }
  return cudaLaunchKernelEx(&cfg, kern, tk, tv, p) == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

template <int D>
int launch_d(const SinkDecodeArgs& a, cudaStream_t stream) {
  if (a.n_parts > 0) return launch<D, false, 2, kBehindPrefix>(a, stream);
  if (a.scores) return launch<D, false, 2, kScored>(a, stream);
  if (!a.cache4) return launch<D, false, 2, kPlain>(a, stream);
  return a.heads / a.kv_heads > 8 ? launch<D, true, 2, kPlain>(a, stream) : launch<D, true, 1, kPlain>(a, stream);
}

int launch_sink_decode(const SinkDecodeArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_d<32>(a, stream);
    case 64: return launch_d<64>(a, stream);
    case 128: return launch_d<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int decode_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_decode_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_decode_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
