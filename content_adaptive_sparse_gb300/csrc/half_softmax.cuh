// The forward machinery of dense key tiles that the sink-window and the shared-prefix forward share: the
// two 64-key halves of every 128-key tile are softmaxes of their own (sink_attn.cu has the reasons and
// the figures), with one issuing thread for S and one for each half's O. A kernel brings its own work
// items, loader, epilogue and masks; an Item walks a CTA's work (more / next, steps, one_half).
#pragma once
#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "ptx_sm100.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

__device__ unsigned int g_fwd_err;    // of the including translation unit

constexpr int kTile = 128;            // queries of an item; keys of a tile
constexpr int kHalf = 64;             // keys of a half
constexpr int kThreads = 512;
constexpr int kSoftmaxWarps = 8, kHalfWarps = 4, kEpilogueWarps = 4;
constexpr int kMaxStages = 4, kMaxS = 3;
constexpr uint32_t kTmemCols = 512;
// Register split (setmaxnreg): softmax warpgroups 184, the others 72, of 128 per thread at launch
constexpr int kLaunchRegs = 128;
static_assert(8 * 184 + 8 * 72 == 16 * kLaunchRegs, "register split");

template <int D>
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
  static constexpr int STAGES = D == 128 ? 2 : 4;      // of K and of V
  static constexpr int SB = D == 128 ? 2 : 3;          // S buffers
  static constexpr uint32_t COL_O = 128 * SB;          // O_0; O_1 follows
  static_assert(COL_O + 2 * D <= kTmemCols, "TMEM columns");
  // Staging per epilogue warp, boxes of 32 rows by 32 elements: a whole row at d <= 64, so that the
  // accumulators are free as soon as they are read; a quarter of one at d = 128
  static constexpr int BOXES = D == 128 ? 1 : D / 32;
  static constexpr int OUT = 2048 * BOXES;
  static constexpr int SMEM = 1024 + (2 + 2 * STAGES) * TILE + kEpilogueWarps * OUT;
  static_assert(STAGES <= kMaxStages && SMEM <= 222 * 1024, "shared memory");
};

struct Bars {
  uint64_t q_full[2], q_empty[2];                                 // phase: item / 2
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  // per S buffer (tile g: barrier g % SB, phase g / SB)
  uint64_t s_full[kMaxS];           // S written
  uint64_t p_full[2][kMaxS];        // [half]: P stored
  uint64_t pv_done[kMaxS];          // both halves' PVs complete
  uint64_t o_full, o_free;          // an item's output complete; read
  uint64_t epi_full[2], epi_empty[2];   // maxima and sums handed to the epilogue
  uint64_t drain[3];
};

struct Handoff {
  float m[2][kTile], l[2][kTile];   // per half and row: running maximum (log2 units), sum
};

__device__ __forceinline__ bool wait_bar(uint64_t* bar, uint32_t parity, volatile int* abort_flag) {
  return mbar_wait_suspend(bar, parity, abort_flag, &g_fwd_err, kErrTimeout);
}
// Use n of a ring of N barriers.
template <int N>
__device__ __forceinline__ bool wait_ring(uint64_t* bar, int n, volatile int* abort_flag) {
  return wait_bar(&bar[n % N], (uint32_t)(n / N) & 1u, abort_flag);
}
__device__ __forceinline__ void drain_bar(uint64_t* bar, uint32_t parity) {
  int never = 0;
  mbar_wait(bar, parity, &never, &g_fwd_err, kErrTimeout);
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// ------------------------------------------------------------------ MMA issuers (one thread each)

template <int D>
__device__ __forceinline__ constexpr uint64_t kstep(int ks) {
  using C = Cfg<D>;
  return (uint64_t)((((ks * 16) / C::CH) * C::CHUNK + ((ks * 16) % C::CH) * 2) >> 4);
}

template <int D, class Item, class Params>
__device__ void qk_issuer(const Params& p, Bars& bars, uint8_t* sQ, uint8_t* sK, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t q0 = make_smem_desc(smem_u32(sQ), 16, C::ATOM, C::SWZ);
  const uint64_t k0 = make_smem_desc(smem_u32(sK), 16, C::ATOM, C::SWZ);
  int g = 0, n = 0;
  bool ok = true;
  for (Item it(p); ok && it.more(); it.next(p), ++n) {
    if (!(ok = wait_ring<2>(bars.q_full, n, abort_flag))) break;
    const uint64_t a = q0 + (uint64_t)(((n & 1) * C::TILE) >> 4);
    for (int j = 0; j < it.steps; ++j, ++g) {
      const int st = g % C::STAGES;
      if (!(ok = wait_ring<C::STAGES>(bars.k_full, g, abort_flag))) break;
      // the P of tile g - SB lay over this S
      if (g >= C::SB && !(ok = wait_ring<C::SB>(bars.pv_done, g - C::SB, abort_flag))) break;
      tc_fence_after();
      const uint64_t b = k0 + (uint64_t)((st * C::TILE) >> 4);
      const uint32_t idesc = make_idesc_bf16(128, it.one_half(p, j) ? kHalf : kTile, 0, 0);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_bf16_ss(tmem + 128u * (g % C::SB), a + kstep<D>(ks), b + kstep<D>(ks), idesc, ks > 0 ? 1u : 0u);
      mma_commit(&bars.k_empty[st]);
      mma_commit(&bars.s_full[g % C::SB]);
    }
    if (ok) mma_commit(&bars.q_empty[n & 1]);
  }
  // no MMA of this thread is still at work when the CTA frees its TMEM
  mma_commit(&bars.drain[0]);
  drain_bar(&bars.drain[0], 0);
}

template <int D, class Item, class Params>
__device__ void pv_issuer(const Params& p, int half, Bars& bars, uint8_t* sV, uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t v0 = make_smem_desc(smem_u32(sV), C::CHUNK, C::ATOM, C::SWZ);   // MN-major
  constexpr uint32_t idesc = make_idesc_bf16(128, D, 0, 1);
  int g = 0, n = 0;
  bool ok = true;
  for (Item it(p); ok && it.more(); it.next(p), ++n) {
    bool acc = false;
    for (int j = 0; j < it.steps; ++j, ++g) {
      const int st = g % C::STAGES;
      if (!(ok = wait_ring<C::STAGES>(bars.v_full, g, abort_flag))) break;
      // the item before has been read
      if (j == 0 && n > 0 && !(ok = wait_bar(&bars.o_free, (uint32_t)(n - 1) & 1u, abort_flag))) break;
      if (!(ok = wait_ring<C::SB>(bars.p_full[half], g, abort_flag))) break;
      if (half == 0 || !it.one_half(p, j)) {
        tc_fence_after();
        const uint32_t a = tmem + 128u * (g % C::SB) + 64u * half;
        const uint64_t b = v0 + (uint64_t)((st * C::TILE + half * kHalf * C::ROWB) >> 4);
#pragma unroll
        for (int ks = 0; ks < kHalf / 16; ++ks)
          mma_bf16_ts(tmem + C::COL_O + (uint32_t)(D * half), a + 8u * ks, b + (uint64_t)((16 * ks * C::ROWB) >> 4), idesc,
                      (acc || ks > 0) ? 1u : 0u);
        acc = true;
      }
      mma_commit(&bars.v_empty[st]);
      mma_commit(&bars.pv_done[g % C::SB]);
    }
    if (ok) mma_commit(&bars.o_full);
  }
  mma_commit(&bars.drain[1 + half]);
  drain_bar(&bars.drain[1 + half], 0);
}

// ------------------------------------------------------------------ softmax

// How a warp's 32 rows see the 64 keys of a half.
enum : int { kNone = 0, kAll = 1, kSome = 2 };
__device__ __forceinline__ void mask_chunk(uint32_t* v, uint32_t see) {
#pragma unroll
  for (int j = 0; j < 32; ++j) v[j] = ((see >> j) & 1u) ? v[j] : 0xff800000u;
}
__device__ __forceinline__ void max_chunk(const uint32_t* v, float (&a)[4]) {
#pragma unroll
  for (int j = 0; j < 32; j += 2)
    a[(j >> 1) & 3] = max3(a[(j >> 1) & 3], __uint_as_float(v[j]), __uint_as_float(v[j + 1]));
}
// p = 2^(s c - r) as bf16 pairs; sums into rs
__device__ __forceinline__ void exp_chunk(const uint32_t* v, uint64_t c2, uint64_t r2, uint32_t* pk, uint64_t (&rs)[2]) {
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    float x0, x1;
    f2::unpack(f2::fma(f2::pack(__uint_as_float(v[j]), __uint_as_float(v[j + 1])), c2, r2), x0, x1);
    const float p0 = ex2_approx(x0), p1 = ex2_approx(x1);
    rs[(j >> 1) & 1] = f2::add(rs[(j >> 1) & 1], f2::pack(p0, p1));
    pk[j >> 1] = pack_bf16x2(p0, p1);
  }
}

// Running maximum of a row without a finite score as yet (no key seen, or products past the fp32 range): 2^(s c - m) is 0 for s = -inf,
// where -inf as the maximum would make it NaN.
constexpr float kLowest = -0x1.fffffep127f;

template <int D>
struct Softmax {
  using C = Cfg<D>;
  Bars& bars;
  volatile int* abort_flag;
  uint32_t tS, tO;                  // TMEM of this warp's rows: S_0 (this half's columns), O_h
  int half, lane;
  float c;                          // softmax scale in log2 units
  float m, l;                       // running maximum (log2 units) and sum of this thread's row

  __device__ __forceinline__ bool done(uint64_t* bar, int g) const {
    return __all_sync(0xffffffffu, wait_ring<C::SB>(bar, g, abort_flag));
  }

  // One tile. Each way of seeing has a copy of the code. kSome: see0 / see1 are the keys that the
  // row sees of the two 32-key chunks, any0 / any1 whether some row of the warp sees any (uniform).
  // `later`: O_h holds a sum of this item.
  template <int SEE>
  __device__ __forceinline__ bool tile(int g, bool any0, bool any1, uint32_t see0, uint32_t see1, bool later) {
    const float kNegInf = __int_as_float(0xff800000);
    const uint32_t t = tS + 128u * (g % C::SB);
    uint32_t pk[32];
    if constexpr (SEE == kNone) {
#pragma unroll
      for (int j = 0; j < 32; ++j) pk[j] = 0u;
    } else {
      uint32_t v[64];
      // kSome: a 32-key chunk that no row of the warp sees is not loaded
      const bool on0 = SEE == kAll || any0, on1 = SEE == kAll || any1;
      if (on0) tmem_ld_x32(t, v);
      if (on1) tmem_ld_x32(t + 32, v + 32);
      tmem_ld_wait<64>(v);
      float a[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
      if (on0) {
        if constexpr (SEE == kSome) mask_chunk(v, see0);
        max_chunk(v, a);
      }
      if (on1) {
        if constexpr (SEE == kSome) mask_chunk(v + 32, see1);
        max_chunk(v + 32, a);
      }
      const float mx = fmaxf(max3(a[0], a[1], a[2]), a[3]) * c;          // -inf stays -inf
      const bool need = mx > m + 8.f;
      if (__any_sync(0xffffffffu, need)) {
        // the running maximum grows by more than 2^8: l and O_h follow
        const float alpha = need ? ex2_approx(m - mx) : 1.f;              // 0 from kLowest
        l *= alpha;
        if (need) m = mx;
        if (later) {
          if (!done(bars.pv_done, g - 1)) return false;
          tc_fence_after();
#pragma unroll 1
          for (int ch = 0; ch < D / 16; ++ch) {
            uint32_t o[16];
            tmem_ld_x16(tO + 16 * ch, o);
            tmem_ld_wait<16>(o);
#pragma unroll
            for (int j = 0; j < 16; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * alpha);
            tmem_st_x16(tO + 16 * ch, o);
          }
        }
      }
      const uint64_t c2 = f2::pack(c, c), r2 = f2::pack(-m, -m);
      uint64_t rs[2] = {0ull, 0ull};
      if (on0) {
        exp_chunk(v, c2, r2, pk, rs);
      } else {
#pragma unroll
        for (int j = 0; j < 16; ++j) pk[j] = 0u;
      }
      if (on1) {
        exp_chunk(v + 32, c2, r2, pk + 16, rs);
      } else {
#pragma unroll
        for (int j = 16; j < 32; ++j) pk[j] = 0u;
      }
      float lo, hi;
      f2::unpack(f2::add(rs[0], rs[1]), lo, hi);
      l += lo + hi;
    }
    tmem_st_x32(t, pk);
    tmem_st_wait();
    tc_fence_before();
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.p_full[half][g % C::SB]);
    return true;
  }
};

// Reads and clears the translation unit's device error word.
inline unsigned int fwd_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_fwd_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_fwd_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace
}  // namespace sa
