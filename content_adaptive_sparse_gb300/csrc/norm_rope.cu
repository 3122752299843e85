// Per-head RMS norm of queries and keys with the position rotation in the same pass, forward
// and backward (bandwidth bound: every element is read once and written once).
//
//   xh = x / sqrt(mean(x^2) + eps),  y = xh * w,  (z_a, z_b) = R(angle) (y_a, y_b) per pair;
//   backward with g = R(-angle) dz:  dx = rstd (g w - xh mean(g w xh)),  dw = sum of g xh.
//
// Layout: a row is one (token, head); D / 8 lanes share it and each lane owns four (a, b) pairs,
// so a rotation never leaves its lane. With rotated halves (element p with p + rotary / 2) a
// lane reads two 8-byte runs, interleaved (2p with 2p + 1) one 16-byte run. A warp stays on one
// token and walks its heads, queries then keys: the angles depend on (token, pair) only, each lane
// takes one of them (two at D = 128), and shuffles hand a lane the four that serve it for every
// head of the token.
//
// Angles: position * frequency is taken modulo one turn in integer arithmetic. The host gives
// frequency / (2 pi) as a 64-bit binary fraction F of a turn; the low 64 bits of position * F
// are the exact phase of F, whatever the position, where a 32-bit product would lose the far
// positions and a 64-bit floating one would run at a small fraction of the GPU's rate. The
// phase's top 32 bits (2^-33 of a turn off at most) go to sincospif.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

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
  int n, heads[2], heads_per_unit, chunks;
  int64_t units;            // tokens of all sequences x head chunks
  int rotary;
  float eps;
  uint64_t turn[64];        // per pair: frequency / (2 pi) as a fraction of 2^64
};

__device__ __forceinline__ void unpack2(uint32_t v, float& lo, float& hi) {
  lo = __uint_as_float(v << 16);
  hi = __uint_as_float(v & 0xffff0000u);
}

// A lane's 16 bytes of one row, as loaded, and as its four pairs: v[0..3] the a elements, v[4..7]
// the b elements.
template <bool INTER>
__device__ __forceinline__ uint4 load_pairs(const __nv_bfloat16* row, int lo, int hi) {
  if constexpr (INTER) {
    return *reinterpret_cast<const uint4*>(row + lo);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(row + lo);
    const uint2 b = *reinterpret_cast<const uint2*>(row + hi);
    return make_uint4(a.x, a.y, b.x, b.y);
  }
}

template <bool INTER>
__device__ __forceinline__ void unpack_pairs(const uint4& r, float (&v)[8]) {
  if constexpr (INTER) {
    unpack2(r.x, v[0], v[4]);
    unpack2(r.y, v[1], v[5]);
    unpack2(r.z, v[2], v[6]);
    unpack2(r.w, v[3], v[7]);
  } else {
    unpack2(r.x, v[0], v[1]);
    unpack2(r.y, v[2], v[3]);
    unpack2(r.z, v[4], v[5]);
    unpack2(r.w, v[6], v[7]);
  }
}

template <bool INTER>
__device__ __forceinline__ void store_pairs(__nv_bfloat16* row, int lo, int hi, const float (&v)[8]) {
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

// The rows of heads [h0, h1) of q (M = 0) or k (M = 1) of one token, RPW at a time and U times RPW
// rows loaded before the first is written (the outputs may be the inputs, so the compiler cannot
// move a load over a store by itself); s and i are the token's sequence and place, cs / sn the
// lane's angles, w_smem its eight weights.
template <int D, bool INTER, bool BWD, int M>
__device__ __forceinline__ void token_rows(const RopeParams& p, int64_t s, int64_t i, int h0, int h1, int slot, int lo,
                                           int hi, const float (&cs)[4], const float (&sn)[4], const float* w_smem,
                                           float (&dw)[8]) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int U = 3;
  if (h0 >= h1) return;
  const __nv_bfloat16* xp = p.x[M].ptr + s * p.x[M].sb + i * p.x[M].sn + (h0 + slot) * p.x[M].sh;
  const __nv_bfloat16* gp = BWD ? p.dy[M].ptr + s * p.dy[M].sb + i * p.dy[M].sn + (h0 + slot) * p.dy[M].sh : nullptr;
  __nv_bfloat16* op =
      const_cast<__nv_bfloat16*>(p.out[M].ptr) + s * p.out[M].sb + i * p.out[M].sn + (h0 + slot) * p.out[M].sh;
  const int64_t xs = RPW * p.x[M].sh, gs = RPW * p.dy[M].sh, os = RPW * p.out[M].sh;
#pragma unroll 1
  for (int hb = h0; hb < h1; hb += U * RPW) {
    uint4 xr[U], gr[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      xr[k] = make_uint4(0u, 0u, 0u, 0u);            // a row past the last head counts as zeros
      gr[k] = make_uint4(0u, 0u, 0u, 0u);
      if (hb + k * RPW + slot < h1) {
        xr[k] = load_pairs<INTER>(xp, lo, hi);
        if constexpr (BWD) gr[k] = load_pairs<INTER>(gp, lo, hi);
      }
      xp += xs;
      if constexpr (BWD) gp += gs;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (hb + k * RPW >= h1) break;                 // the whole warp
      float x[8], z[8], w[8];
      unpack_pairs<INTER>(xr[k], x);
      *reinterpret_cast<float4*>(w) = *reinterpret_cast<const float4*>(w_smem);
      *reinterpret_cast<float4*>(w + 4) = *reinterpret_cast<const float4*>(w_smem + 4);
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
      if constexpr (!BWD) {
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float a = x[e] * rstd * w[e], b = x[e + 4] * rstd * w[e + 4];
          z[e] = a * cs[e] - b * sn[e];
          z[e + 4] = b * cs[e] + a * sn[e];
        }
      } else {
        float g[8];
        float dot = 0.f;
        unpack_pairs<INTER>(gr[k], z);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          g[e] = z[e] * cs[e] + z[e + 4] * sn[e];
          g[e + 4] = z[e + 4] * cs[e] - z[e] * sn[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) dot += g[e] * w[e] * x[e];
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        const float c = row_sum<LPR>(dot) * rstd * (1.f / D);        // mean(g w xh)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float xh = x[e] * rstd;
          dw[e] += g[e] * xh;
          z[e] = rstd * (g[e] * w[e] - xh * c);
        }
      }
      if (hb + k * RPW + slot < h1) store_pairs<INTER>(op, lo, hi, z);
      op += os;
    }
  }
}

template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kWarps, BWD ? 2 : 4) norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPR = D / 8;             // lanes per row
  constexpr int PAIRS = D / 2;
  constexpr int PPL = (PAIRS + 31) / 32; // pairs whose angles a lane takes
  __shared__ __align__(16) float w_smem[2][D];            // weights in the lanes' order
  __shared__ float red[BWD ? kWarps : 1][2][BWD ? D : 1];
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
    for (int e = 0; e < 8; ++e) w_smem[warp][8 * t + e] = p.w[warp] ? p.w[warp][element(e)] : 1.f;
  }
  uint64_t turn[PPL];
#pragma unroll
  for (int k = 0; k < PPL; ++k) turn[k] = lane + 32 * k < half ? p.turn[lane + 32 * k] : 0ull;
  __syncthreads();
  float dw[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[m][e] = 0.f;
  const int hq = p.heads[0], all = hq + p.heads[1];
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < p.units; u += (int64_t)gridDim.x * kWarps) {
    const int64_t tok = u / p.chunks;
    const int h0 = (int)(u - tok * p.chunks) * p.heads_per_unit;
    const int h1 = min(all, h0 + p.heads_per_unit);
    const int64_t s = tok / p.n, i = tok - s * p.n;
    const int64_t pos = p.positions ? (int64_t)p.positions[tok] : i;
    // one angle per lane (two at D = 128), handed to the lanes whose pair it is
    float my_c[PPL], my_s[PPL], cs[4], sn[4];
#pragma unroll
    for (int k = 0; k < PPL; ++k) {
      // phase of a turn in [-2^31, 2^31) / 2^32; sincospif takes half turns
      const int32_t phase = (int32_t)(((uint64_t)pos * turn[k]) >> 32);
      sincospif((float)phase * 4.656612873077393e-10f, &my_s[k], &my_c[k]);   // 2^-31
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int from = (4 * t + e) & 31;
      cs[e] = __shfl_sync(0xffffffffu, my_c[0], from);
      sn[e] = __shfl_sync(0xffffffffu, my_s[0], from);
      if constexpr (PPL == 2) {
        const float c1 = __shfl_sync(0xffffffffu, my_c[PPL - 1], from), s1 = __shfl_sync(0xffffffffu, my_s[PPL - 1], from);
        cs[e] = 4 * t >= 32 ? c1 : cs[e];
        sn[e] = 4 * t >= 32 ? s1 : sn[e];
      }
    }
    token_rows<D, INTER, BWD, 0>(p, s, i, h0, min(h1, hq), slot, lo, hi, cs, sn, &w_smem[0][8 * t], dw[0]);
    token_rows<D, INTER, BWD, 1>(p, s, i, max(h0 - hq, 0), h1 - hq, slot, lo, hi, cs, sn, &w_smem[1][8 * t], dw[1]);
  }
  if constexpr (BWD) {
    // this CTA's sums of g xh: over the warp's row slots, then over its warps, in a fixed order
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float v = dw[m][e];
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
  const int ctas = 8 * current_sm_count();
  // A warp takes all heads of a token, so that a token's angles are taken once, unless that
  // leaves warps without work: then it takes as few groups of RPW heads as keep them all busy.
  const int groups = (all + RPW - 1) / RPW;
  const int64_t warps = (int64_t)ctas * kWarps;
  int per = (int)((tokens * groups + warps - 1) / warps);
  per = per < groups ? per : groups;
  p.heads_per_unit = per * RPW;
  p.chunks = (groups + per - 1) / per;
  p.units = tokens * p.chunks;
  int64_t grid = (p.units + kWarps - 1) / kWarps;
  if (grid > ctas) grid = ctas;
  if (grid > kNormRopeMaxCtas) grid = kNormRopeMaxCtas;
  norm_rope_kernel<D, INTER, BWD><<<(unsigned)grid, 32 * kWarps, 0, stream>>>(p);
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
