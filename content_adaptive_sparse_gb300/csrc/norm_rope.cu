// Per-head RMS norm of queries and keys with the position rotation in the same pass, forward
// and backward (bandwidth bound: every element is read once and written once).
//
//   xh = x / sqrt(mean(x^2) + eps),  y = xh * w,  (z_a, z_b) = R(angle) (y_a, y_b) per pair;
//   backward with g = R(-angle) dz:  dx = rstd (g w - xh mean(g w xh)),  dw = sum of g xh.
//
// Layout: a row is one (token, head); D / 8 lanes share it and each lane owns four (a, b) pairs,
// so a rotation never leaves its lane. With rotated halves (element p with p + rotary / 2) a
// lane reads two 8-byte runs, interleaved (2p with 2p + 1) one 16-byte run. A warp stays on one
// token and walks its heads, queries then keys: the angles depend on (token, pair) only, and a
// lane's four sines and cosines serve every head of the token.
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

// A lane's four pairs of one row: v[0..3] the a elements, v[4..7] the b elements.
template <bool INTER>
__device__ __forceinline__ void load_pairs(const __nv_bfloat16* row, int lo, int hi, float (&v)[8]) {
  if (INTER) {
    const uint4 r = *reinterpret_cast<const uint4*>(row + lo);
    unpack2(r.x, v[0], v[4]);
    unpack2(r.y, v[1], v[5]);
    unpack2(r.z, v[2], v[6]);
    unpack2(r.w, v[3], v[7]);
  } else {
    const uint2 a = *reinterpret_cast<const uint2*>(row + lo);
    const uint2 b = *reinterpret_cast<const uint2*>(row + hi);
    unpack2(a.x, v[0], v[1]);
    unpack2(a.y, v[2], v[3]);
    unpack2(b.x, v[4], v[5]);
    unpack2(b.y, v[6], v[7]);
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

template <int D, bool INTER, bool BWD>
__global__ void __launch_bounds__(32 * kWarps) norm_rope_kernel(const __grid_constant__ RopeParams p) {
  constexpr int LPR = D / 8;             // lanes per row
  constexpr int RPW = 32 / LPR;          // rows (heads) a warp handles at a time
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = lane % LPR, slot = lane / LPR;
  // this lane's pairs are 4t .. 4t+3 of the row's D / 2; those past rotary / 2 are not rotated
  // and hold the elements from `rotary` on
  const int half = p.rotary >> 1;
  const int lo = INTER ? 8 * t : (4 * t < half ? 4 * t : 4 * t + half);
  const int hi = 4 * t < half ? 4 * t + half : 4 * t + D / 2;
  uint64_t turn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) turn[i] = 4 * t + i < half ? p.turn[4 * t + i] : 0ull;
  float w[2][8];
  float dw[2][8];
#pragma unroll
  for (int m = 0; m < 2; ++m)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int e = INTER ? 8 * t + 2 * (i & 3) + (i >> 2) : (i < 4 ? lo + i : hi + i - 4);
      w[m][i] = p.w[m] ? p.w[m][e] : 1.f;
      dw[m][i] = 0.f;
    }
  const int all = p.heads[0] + p.heads[1];
  for (int64_t u = (int64_t)blockIdx.x * kWarps + warp; u < p.units; u += (int64_t)gridDim.x * kWarps) {
    const int64_t tok = u / p.chunks;
    const int h0 = (int)(u % p.chunks) * p.heads_per_unit;
    const int h1 = min(all, h0 + p.heads_per_unit);
    const int64_t s = tok / p.n;
    const int64_t i0 = tok % p.n;
    const int64_t pos = p.positions ? (int64_t)p.positions[tok] : i0;
    float cs[4], sn[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // phase of a turn in [-2^31, 2^31) / 2^32; sincospif takes half turns
      const int32_t phase = (int32_t)(((uint64_t)pos * turn[i]) >> 32);
      sincospif((float)phase * 4.656612873077393e-10f, &sn[i], &cs[i]);   // 2^-31
    }
#pragma unroll 2
    for (int hb = h0; hb < h1; hb += RPW) {
      const int head = hb + slot;
      const bool on = head < h1;
      const int m = head >= p.heads[0] ? 1 : 0;
      const int64_t h = m ? head - p.heads[0] : head;
      const Tensor& X = p.x[m];
      float x[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = 0.f;
      if (on) load_pairs<INTER>(X.ptr + s * X.sb + i0 * X.sn + h * X.sh, lo, hi, x);
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss += x[i] * x[i];
      if constexpr (!BWD) {
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        float z[8];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float a = x[i] * rstd * (m ? w[1][i] : w[0][i]);
          const float b = x[i + 4] * rstd * (m ? w[1][i + 4] : w[0][i + 4]);
          z[i] = a * cs[i] - b * sn[i];
          z[i + 4] = b * cs[i] + a * sn[i];
        }
        const Tensor& O = p.out[m];
        if (on) store_pairs<INTER>(const_cast<__nv_bfloat16*>(O.ptr) + s * O.sb + i0 * O.sn + h * O.sh, lo, hi, z);
      } else {
        const Tensor& G = p.dy[m];
        float g[8], z[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) z[i] = 0.f;
        if (on) load_pairs<INTER>(G.ptr + s * G.sb + i0 * G.sn + h * G.sh, lo, hi, z);
        float dot = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          g[i] = z[i] * cs[i] + z[i + 4] * sn[i];
          g[i + 4] = z[i + 4] * cs[i] - z[i] * sn[i];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) dot += g[i] * (m ? w[1][i] : w[0][i]) * x[i];
        const float rstd = rsqrtf(row_sum<LPR>(ss) * (1.f / D) + p.eps);
        const float c = row_sum<LPR>(dot) * rstd * (1.f / D);      // mean(g w xh)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float xh = x[i] * rstd;
          const float wi = m ? w[1][i] : w[0][i];
          // a row past the last head adds g xh = 0
          if (m) dw[1][i] += g[i] * xh;
          else dw[0][i] += g[i] * xh;
          z[i] = rstd * (g[i] * wi - xh * c);
        }
        const Tensor& O = p.out[m];
        if (on) store_pairs<INTER>(const_cast<__nv_bfloat16*>(O.ptr) + s * O.sb + i0 * O.sn + h * O.sh, lo, hi, z);
      }
    }
  }
  if constexpr (BWD) {
    // this CTA's sums of g xh: over the warp's row slots, then over its warps, in a fixed order
    __shared__ float red[kWarps][2][D];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float v = dw[m][i];
#pragma unroll
        for (int o = 16; o >= LPR; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        const int e = INTER ? 8 * t + 2 * (i & 3) + (i >> 2) : (i < 4 ? lo + i : hi + i - 4);
        if (slot == 0) red[warp][m][e] = v;
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
