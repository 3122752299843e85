// Per-head RMS norm of queries and keys with the position rotation in the same pass, forward
// and backward (bandwidth bound: every element is read once and written once).
//
//   xh = x / sqrt(mean(x^2) + eps),  y = xh * w,  (z_a, z_b) = R(angle) (y_a, y_b) per pair;
//   backward with g = R(-angle) dz:  dx = rstd (g w - xh mean(g w xh)),  dw = sum of g xh.
//
// Layout: a row is one (token, head); D / 8 lanes share it and each lane owns four (a, b) pairs,
// so a rotation never leaves its lane. With rotated halves (element p with p + rotary / 2) a
// lane reads two 8-byte runs, interleaved (2p with 2p + 1) one 16-byte run. A warp stays on one
// token and walks its heads in batches of three times the rows that fit it side by side; each
// lane's copies of the next batch into shared memory run under the arithmetic of this one (batch by
// batch through registers: 111 us for the two directions below against 103; two thirds as many rows
// to a batch: 117; a further batch ahead: no gain). The arithmetic is two numbers an instruction,
// and a warp's next place is found by additions (103 -> 91 us). Queries come first, then keys: the
// angles depend on (token, pair) only, each lane takes one of them (two at D = 128), and shuffles
// hand a lane the four that serve it for every head of the token.
//
// Angles: position * frequency is taken modulo one turn in integer arithmetic. The host gives
// frequency / (2 pi) as a 64-bit binary fraction F of a turn; the low 64 bits of position * F
// are the exact phase of F, whatever the position, where a 32-bit product would lose the far
// positions and a 64-bit floating one would run at a small fraction of the GPU's rate. The
// phase's top 32 bits (less than 2^-32 of a turn off) go to sincospif as fp32, half a turn at most, which
// rounds them by 2^-26 of a turn at most.
//
// Measured, 4 x 8192 tokens, 12 + 12 heads of 64: forward 35.2 us (201 MB: 5.7 TB/s), backward with
// the weights' gradients 55.9 us (302 MB: 5.4 TB/s), 0.84 and 0.80 of a plain copy's rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "f32x2.cuh"
#include "ptx_sm100.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

constexpr int kWarps = 8;

struct Tensor {
  const __nv_bfloat16* ptr;
  int64_t sb, sn, sh;
};

struct RopeParams {
  Tensor x[2];              // q, k
  Tensor dy[2];             // backward: gradients of the outputs
  Tensor out[2];            // forward: rotated q, k; backward: dq, dk
  const float* w[2];        // [D], or null: ones
  float* partial;           // backward: [grid][2][D] sums of g xh
  const int32_t* positions; // [batch][n], or null: 0 .. n-1
  int batch, n, heads[2];
  int heads_per_unit, chunks;           // a unit of work: a token and one of `chunks` ranges of its heads
  int step_c, step_i, step_s;           // units of one round of the grid's warps, as (chunk, token, sequence)
  int rotary;
  float eps;
  uint64_t turn[64];        // per pair: frequency / (2 pi) as a fraction of 2^64
};

__device__ __forceinline__ void unpack2(uint32_t v, float& lo, float& hi) {
  lo = __uint_as_float(v << 16);
  hi = __uint_as_float(v & 0xffff0000u);
}

// A lane's 16 bytes of one row on their way to `dst` (shared memory), and as its four (a, b): v[0] and
// v[1] two a elements each, v[2] and v[3] the b elements.
template <bool INTER>
__device__ __forceinline__ void copy_pairs(uint32_t dst, const __nv_bfloat16* row, int lo, int hi) {
  if constexpr (INTER) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(row + lo) : "memory");
  } else {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst), "l"(row + lo) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(dst + 8), "l"(row + hi) : "memory");
  }
}

template <bool INTER>
__device__ __forceinline__ void unpack_pairs(const uint4& r, uint64_t (&v)[4]) {
  float a[4], b[4];
  unpack2(r.x, a[0], a[1]);
  unpack2(r.y, a[2], a[3]);
  unpack2(r.z, b[0], b[1]);
  unpack2(r.w, b[2], b[3]);
  if constexpr (INTER) {                 // r holds a0 b0 a1 b1 ...
    v[0] = f2::pack(a[0], a[2]);
    v[1] = f2::pack(b[0], b[2]);
    v[2] = f2::pack(a[1], a[3]);
    v[3] = f2::pack(b[1], b[3]);
  } else {
    v[0] = f2::pack(a[0], a[1]);
    v[1] = f2::pack(a[2], a[3]);
    v[2] = f2::pack(b[0], b[1]);
    v[3] = f2::pack(b[2], b[3]);
  }
}

template <bool INTER>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* row, int lo, int hi, const uint64_t (&z)[4]) {
  float v[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) f2::unpack(z[e], v[2 * e], v[2 * e + 1]);
  if (INTER) {
    *reinterpret_cast<uint4*>(row + lo) = make_uint4(pack_bf16x2(v[0], v[4]), pack_bf16x2(v[1], v[5]),
                                                     pack_bf16x2(v[2], v[6]), pack_bf16x2(v[3], v[7]));
  } else {
    *reinterpret_cast<uint2*>(row + lo) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
    *reinterpret_cast<uint2*>(row + hi) = make_uint2(pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
}

// Sum over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = LPR / 2; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

template <int D, bool BWD>
struct Cfg {
  static constexpr int LPR = D / 8;      // lanes per row
  static constexpr int RPW = 32 / LPR;   // rows of a warp side by side
  static constexpr int U = 3;            // times RPW rows: a batch
  static constexpr int BATCH = U * 512 * (BWD ? 2 : 1);   // bytes of it
  static constexpr int SMEM = kWarps * 2 * BATCH;         // a warp computes one and requests the next
  static constexpr int CTAS = BWD ? 2 : 3;                // resident CTAs per SM
};

// A warp's place in its work: heads hb .. of q (m = 0) or k (m = 1), below `end`, of token i of
// sequence s, a batch of STEP heads at a time.
template <int STEP>
struct Cursor {
  int s, i, chunk;
  int m, hb, end, k0, k1;
  __device__ __forceinline__ void start(const RopeParams& p, uint32_t unit) {
    const uint32_t tok = unit / (uint32_t)p.chunks;
    chunk = (int)(unit % (uint32_t)p.chunks);
    s = (int)(tok / (uint32_t)p.n);
    i = (int)(tok % (uint32_t)p.n);
    heads(p);
  }
  __device__ __forceinline__ void heads(const RopeParams& p) {
    const int h0 = chunk * p.heads_per_unit, hq = p.heads[0];
    const int h1 = min(hq + p.heads[1], h0 + p.heads_per_unit);
    k0 = max(h0 - hq, 0);
    k1 = h1 - hq;
    m = h0 < hq ? 0 : 1;
    hb = m ? k0 : h0;
    end = m ? k1 : min(h1, hq);
  }
  __device__ __forceinline__ bool more(const RopeParams& p) const { return s < p.batch; }
  __device__ __forceinline__ int64_t token(const RopeParams& p) const { return (int64_t)s * p.n + i; }
  __device__ __forceinline__ void next(const RopeParams& p) {
    hb += STEP;
    if (hb < end) return;
    if (m == 0 && k0 < k1) {
      m = 1;
      hb = k0;
      end = k1;
      return;
    }
    // the next round's unit: the three digits added, without a division
    chunk += p.step_c;
    i += p.step_i;
    s += p.step_s;
    if (chunk >= p.chunks) {
      chunk -= p.chunks;
      ++i;
    }
    if (i >= p.n) {
      i -= p.n;
      ++s;
    }
    heads(p);
  }
};

__device__ __forceinline__ float pair_sum(uint64_t v) {
  float a, b;
  f2::unpack(v, a, b);
  return a + b;
}

// Requests a batch: each lane copies what it will read itself, so no other lane has to wait for it.
template <int D, bool INTER, bool BWD, int STEP>
__device__ __forceinline__ void request(const RopeParams& p, const Cursor<STEP>& c, uint32_t dst, int slot, int lo, int hi) {
  using C = Cfg<D, BWD>;
  if (c.more(p)) {
    const Tensor &x = p.x[c.m], &g = p.dy[c.m];
    const __nv_bfloat16* xp = x.ptr + c.s * x.sb + c.i * x.sn + (c.hb + slot) * x.sh;
    const __nv_bfloat16* gp = BWD ? g.ptr + c.s * g.sb + c.i * g.sn + (c.hb + slot) * g.sh : nullptr;
#pragma unroll
    for (int k = 0; k < C::U; ++k) {
      if (c.hb + k * C::RPW + slot < c.end) {
        copy_pairs<INTER>(dst + 512 * k, xp, lo, hi);
        if constexpr (BWD) copy_pairs<INTER>(dst + 512 * (C::U + k), gp, lo, hi);
      }
      xp += C::RPW * x.sh;
      if constexpr (BWD) gp += C::RPW * g.sh;
    }
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
}

// A batch of q (M = 0) or k (M = 1) that lies in shared memory at `src` (this lane's 16 bytes of its
// first rows); cs / sn / ns are the cosines, sines and negated sines of the lane's angles, w_smem its
// eight weights.
template <int D, bool INTER, bool BWD, int M, int STEP>
__device__ __forceinline__ void batch_rows(const RopeParams& p, const Cursor<STEP>& c, const uint8_t* src, int slot, int lo,
                                           int hi, const uint64_t (&cs)[2], const uint64_t (&sn)[2],
                                           const uint64_t (&ns)[2], const uint64_t* w_smem, uint64_t (&dw)[4]) {
  using C = Cfg<D, BWD>;
  constexpr int LPR = C::LPR;
  __nv_bfloat16* op = const_cast<__nv_bfloat16*>(p.out[M].ptr) + c.s * p.out[M].sb + c.i * p.out[M].sn +
                      (c.hb + slot) * p.out[M].sh;
#pragma unroll
  for (int k = 0; k < C::U; ++k) {
    if (c.hb + k * C::RPW >= c.end) break;           // the whole warp
    const bool on = c.hb + k * C::RPW + slot < c.end;
    // a row past the last head counts as zeros
    const uint4 zero = make_uint4(0u, 0u, 0u, 0u);
    const uint4 xr = on ? *reinterpret_cast<const uint4*>(src + 512 * k) : zero;
    uint64_t x[4], z[4], w[4];
    unpack_pairs<INTER>(xr, x);
#pragma unroll
    for (int e = 0; e < 4; e += 2) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(w_smem + e);
      w[e] = v.x;
      w[e + 1] = v.y;
    }
    const uint64_t ss = f2::fma(x[3], x[3], f2::fma(x[2], x[2], f2::fma(x[1], x[1], f2::mul(x[0], x[0]))));
    const float rstd = rsqrtf(row_sum<LPR>(pair_sum(ss)) * (1.f / D) + p.eps);
    const uint64_t r2 = f2::pack(rstd, rstd);
    if constexpr (!BWD) {
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const uint64_t a = f2::mul(f2::mul(x[e], r2), w[e]), b = f2::mul(f2::mul(x[e + 2], r2), w[e + 2]);
        z[e] = f2::fma(a, cs[e], f2::mul(b, ns[e]));
        z[e + 2] = f2::fma(b, cs[e], f2::mul(a, sn[e]));
      }
    } else {
      uint64_t g[4], gw[4];
      const uint4 gr = on ? *reinterpret_cast<const uint4*>(src + 512 * (C::U + k)) : zero;
      unpack_pairs<INTER>(gr, z);
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        g[e] = f2::fma(z[e], cs[e], f2::mul(z[e + 2], sn[e]));
        g[e + 2] = f2::fma(z[e + 2], cs[e], f2::mul(z[e], ns[e]));
      }
#pragma unroll
      for (int e = 0; e < 4; ++e) gw[e] = f2::mul(g[e], w[e]);
      const uint64_t dot = f2::fma(gw[3], x[3], f2::fma(gw[2], x[2], f2::fma(gw[1], x[1], f2::mul(gw[0], x[0]))));
      const float mean = row_sum<LPR>(pair_sum(dot)) * rstd * (-1.f / D);      // - mean(g w xh)
      const uint64_t m2 = f2::pack(mean, mean);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint64_t xh = f2::mul(x[e], r2);
        dw[e] = f2::fma(g[e], xh, dw[e]);
        z[e] = f2::mul(r2, f2::fma(xh, m2, gw[e]));
      }
    }
    if (on) store_pairs<INTER>(op, lo, hi, z);
    op += C::RPW * p.out[M].sh;
  }
}

// cos, sin and -sin of a lane's four pairs at `pos`: one angle per lane (two at D = 128), handed to the
// lanes whose pair it is.
template <int PPL>
__device__ __forceinline__ void angles(int64_t pos, const uint64_t (&turn)[PPL], int t, uint64_t (&cs)[2],
                                       uint64_t (&sn)[2], uint64_t (&ns)[2]) {
  float my_c[PPL], my_s[PPL];
#pragma unroll
  for (int k = 0; k < PPL; ++k) {
    // phase of a turn in [-2^31, 2^31) / 2^32; sincospif takes half turns
    const int32_t phase = (int32_t)(((uint64_t)pos * turn[k]) >> 32);
    sincospif((float)phase * 4.656612873077393e-10f, &my_s[k], &my_c[k]);   // 2^-31
  }
  float c[4], s[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int from = (4 * t + e) & 31;
    c[e] = __shfl_sync(0xffffffffu, my_c[0], from);
    s[e] = __shfl_sync(0xffffffffu, my_s[0], from);
    if constexpr (PPL == 2) {
      const float c1 = __shfl_sync(0xffffffffu, my_c[PPL - 1], from), s1 = __shfl_sync(0xffffffffu, my_s[PPL - 1], from);
      c[e] = 4 * t >= 32 ? c1 : c[e];
      s[e] = 4 * t >= 32 ? s1 : s[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    cs[e] = f2::pack(c[2 * e], c[2 * e + 1]);
    sn[e] = f2::pack(s[2 * e], s[2 * e + 1]);
    ns[e] = f2::pack(-s[2 * e], -s[2 * e + 1]);
  }
}

template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kWarps, Cfg<D, BWD>::CTAS) norm_rope_kernel(const __grid_constant__ RopeParams p) {
  using C = Cfg<D, BWD>;
  constexpr int LPR = C::LPR;
  constexpr int PAIRS = D / 2;
  constexpr int PPL = (PAIRS + 31) / 32; // pairs whose angles a lane takes
  __shared__ __align__(16) uint64_t w_smem[2][D / 2];     // weights in the lanes' order
  extern __shared__ __align__(16) uint8_t ring[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = lane % LPR, slot = lane / LPR;
  // this lane's pairs are 4t .. 4t+3 of the row's D / 2; those past rotary / 2 are not rotated
  // and hold the elements from `rotary` on
  const int half = p.rotary >> 1;
  const int lo = INTER ? 8 * t : (4 * t < half ? 4 * t : 4 * t + half);
  const int hi = 4 * t < half ? 4 * t + half : 4 * t + D / 2;
  const auto element = [&](int e) { return INTER ? 8 * t + 2 * (e & 3) + (e >> 2) : (e < 4 ? lo + e : hi + e - 4); };
  if (warp < 2 && slot == 0) {
#pragma unroll
    for (int e = 0; e < 8; e += 2)
      w_smem[warp][4 * t + e / 2] =
          p.w[warp] ? f2::pack(p.w[warp][element(e)], p.w[warp][element(e + 1)]) : f2::pack(1.f, 1.f);
  }
  uint64_t turn[PPL];
#pragma unroll
  for (int k = 0; k < PPL; ++k) turn[k] = lane + 32 * k < half ? p.turn[lane + 32 * k] : 0ull;
  __syncthreads();
  uint64_t dw[2][4];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 4; ++e) dw[m][e] = 0ull;
  // this lane's places in its warp's two batches
  uint8_t* mine = ring + warp * 2 * C::BATCH + 16 * lane;
  constexpr int kStep = C::U * C::RPW;
  Cursor<kStep> at, ahead;
  ahead.start(p, blockIdx.x * kWarps + warp);
  request<D, INTER, BWD>(p, ahead, smem_u32(mine), slot, lo, hi);
  int64_t angles_of = -1;
  uint64_t cs[2], sn[2], ns[2];
#pragma unroll 1
  for (int stage = 0; ahead.more(p); stage ^= 1) {
    at = ahead;
    ahead.next(p);
    request<D, INTER, BWD>(p, ahead, smem_u32(mine) + (stage ^ 1) * C::BATCH, slot, lo, hi);
    const int64_t tok = at.token(p);
    if (tok != angles_of) {
      angles_of = tok;
      angles<PPL>(p.positions ? (int64_t)p.positions[tok] : at.i, turn, t, cs, sn, ns);
    }
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    const uint8_t* src = mine + stage * C::BATCH;
    if (at.m == 0) batch_rows<D, INTER, BWD, 0>(p, at, src, slot, lo, hi, cs, sn, ns, &w_smem[0][4 * t], dw[0]);
    else batch_rows<D, INTER, BWD, 1>(p, at, src, slot, lo, hi, cs, sn, ns, &w_smem[1][4 * t], dw[1]);
  }
  if constexpr (BWD) {
    // this CTA's sums of g xh: over the warp's row slots, then over its warps, in a fixed order
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();                                         // the ring is free
    static_assert(kWarps * 2 * D * 4 <= C::SMEM, "the warps' sums");
    float(*red)[2][D] = reinterpret_cast<float(*)[2][D]>(ring);
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float pair[2];
        f2::unpack(dw[m][e >> 1], pair[0], pair[1]);
        float v = pair[e & 1];
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        if (slot == 0) red[warp][m][element(e)] = v;
      }
    __syncthreads();
    for (int e = threadIdx.x; e < 2 * D; e += 32 * kWarps) {
      float v = 0.f;
#pragma unroll
      for (int j = 0; j < kWarps; ++j) v += red[j][e / D][e % D];
      p.partial[(size_t)blockIdx.x * (2 * D) + e] = v;
    }
  }
}

// dw[m][e] = sum over the CTAs' partial sums (fixed order: the result does not vary). One CTA
// per 32 columns, 32 rows of threads.
template <int D>
__global__ void __launch_bounds__(1024) norm_rope_dw_kernel(const float* partial, int n_parts, float* dwq, float* dwk) {
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x;           // column of [2][D]
  float v = 0.f;
  for (int r = threadIdx.y; r < n_parts; r += 32) v += partial[(size_t)r * (2 * D) + col];
  red[threadIdx.y][threadIdx.x] = v;
  __syncthreads();
  if (threadIdx.y == 0) {
    float sum = 0.f;
#pragma unroll
    for (int r = 0; r < 32; ++r) sum += red[r][threadIdx.x];
    float* dst = col < D ? dwq : dwk;
    if (dst) dst[col % D] = sum;
  }
}

Tensor tensor(const void* ptr, const int64_t s[3]) {
  return Tensor{static_cast<const __nv_bfloat16*>(ptr), s[0], s[1], s[2]};
}

template <int D, bool INTER, bool BWD>
int launch(RopeParams& p, const NormRopeArgs& a, cudaStream_t stream) {
  constexpr int RPW = 32 / (D / 8);
  const int all = a.heads + a.kv_heads;
  const int64_t tokens = (int64_t)a.batch * a.n_tokens;
  const int ctas = Cfg<D, BWD>::CTAS * current_sm_count();
  // A warp takes all heads of a token, so that a token's angles are taken once, unless that
  // leaves warps without work: then it takes as few groups of RPW heads as keep them all busy.
  const int groups = (all + RPW - 1) / RPW;
  const int64_t warps = (int64_t)ctas * kWarps;
  int per = (int)((tokens * groups + warps - 1) / warps);
  per = per < groups ? per : groups;
  p.heads_per_unit = per * RPW;
  p.chunks = (groups + per - 1) / per;
  const int64_t units = tokens * p.chunks;             // below 2^31: tokens are below 2^30, and where there are
                                                       // several chunks a token, units are at most warps + tokens
  int64_t grid = (units + kWarps - 1) / kWarps;
  if (grid > ctas) grid = ctas;
  if (grid > kNormRopeMaxCtas) grid = kNormRopeMaxCtas;
  const int64_t round = grid * kWarps;
  p.step_c = (int)(round % p.chunks);
  p.step_i = (int)(round / p.chunks % a.n_tokens);
  p.step_s = (int)(round / p.chunks / a.n_tokens);
  const auto kern = norm_rope_kernel<D, INTER, BWD>;
  constexpr int kSmem = Cfg<D, BWD>::SMEM;
  if (kSmem > 48 * 1024 - 1024 &&
      cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem) != cudaSuccess)
    return SA_ERR_CUDA;
  kern<<<(unsigned)grid, 32 * kWarps, kSmem, stream>>>(p);
  if (BWD && (a.dq_weight || a.dk_weight))
    norm_rope_dw_kernel<D><<<2 * D / 32, dim3(32, 32), 0, stream>>>(p.partial, (int)grid, a.dq_weight, a.dk_weight);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int D>
int launch_d(RopeParams& p, const NormRopeArgs& a, cudaStream_t stream) {
  if (a.backward) return a.interleaved ? launch<D, true, true>(p, a, stream) : launch<D, false, true>(p, a, stream);
  return a.interleaved ? launch<D, true, false>(p, a, stream) : launch<D, false, false>(p, a, stream);
}

}  // namespace

int launch_norm_rope(const NormRopeArgs& a, cudaStream_t stream) {
  RopeParams p;
  p.x[0] = tensor(a.q, a.q_strides);
  p.x[1] = tensor(a.k, a.k_strides);
  p.dy[0] = tensor(a.d_q_out, a.dy_q_strides);
  p.dy[1] = tensor(a.d_k_out, a.dy_k_strides);
  p.out[0] = tensor(a.q_out, a.q_out_strides);
  p.out[1] = tensor(a.k_out, a.k_out_strides);
  p.w[0] = a.q_weight;
  p.w[1] = a.k_weight;
  p.partial = static_cast<float*>(a.workspace);
  p.positions = a.positions;
  p.batch = a.batch;
  p.n = a.n_tokens;
  p.heads[0] = a.heads;
  p.heads[1] = a.kv_heads;
  p.rotary = a.rotary_dim;
  p.eps = a.eps;
  for (int i = 0; i < 64; ++i) {
    // frequencies are below 2 pi (checked), so the fraction is below one turn; the scaling by
    // 2^64 is exact
    const double f = i < a.rotary_dim / 2 ? a.h_inv_freq[i] * 0.15915494309189533576888 : 0.0;
    p.turn[i] = (uint64_t)(f * 18446744073709551616.0);
  }
  switch (a.head_dim) {
    case 32: return launch_d<32>(p, a, stream);
    case 64: return launch_d<64>(p, a, stream);
    case 128: return launch_d<128>(p, a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

}  // namespace sa
