// Key / value cache in 4 bits: writing rows to it and reading them back (bandwidth bound: bf16
// rows one way, 4.5 bits an element the other).
//
// A row is one (token, key head). Each run of 32 elements has the bf16 scale s = amax / 7, and an
// element x the code round(x / s) (ties to even) in -7 .. 7, stored + 8 (s = 0: code 0). The scale is
// the exact quotient rounded once: amax has 8 significant bits and a border between two bf16
// numbers times 7 has 12, so amax / 7 is 2^-13 and more away from the border or on it, and its
// fp32 rounding does not move it across. A run with an infinity or a NaN has the scale NaN and
// reads back as NaN.
//   codes  [batch][kv_heads][capacity][d / 2] bytes: little-endian 32-bit word t * (d / 32) + c holds
//          elements 32 c + 8 t + u, u = 0 .. 7; u = 4 p + i stands at bit 8 p + 4 (i / 2) + 16 (i % 2)
//   scales [batch][kv_heads][capacity][d / 32] bf16
// The word order puts what one lane of the decoding kernel's fragments needs side by side: word
// (t, c) for all c in one load, pairs (2k, 2k + 1) in the two half-words at the same nibble.
//
// One thread per word: 16 bytes of the row, the run's maximum over its four threads by shuffles.
// The rounding takes no division per element: q = x (1 / s) is off by less than 2^-20, while a
// quotient lies on a border (k + 1/2) or 2^-10 and more away from it, so q is first rounded to a
// multiple of 2^-15 (adding 384, whose last place that is, and taking it off again), which puts
// a border's quotient back on the border, and then to the nearest even integer.
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "ptx_sm100.cuh"
#include "sa_internal.h"

namespace sa {
namespace {

__device__ unsigned int g_cache_err;

struct CParams {
  __nv_bfloat16* x[2];              // k, v rows (read by the append, written by the read)
  uint32_t* codes[2];
  __nv_bfloat16* scales[2];
  const int32_t* start;
  int64_t sb[2], sn[2], sh[2];
  int kv_heads, capacity;
  uint32_t words;                   // 32-bit words of one sequence's rows
};

__host__ __device__ constexpr int bit_of(int u) { return 8 * (u >> 2) + 4 * ((u & 3) >> 1) + 16 * (u & 1); }

// Thread's word of sequence s: token i of the call, head h, run c, word t of the run; the cache
// row, or -1 (out of range: reported; start < 0: the sequence is left out, not reported).
template <int D>
struct Place {
  uint32_t c, t, h, i;
  int64_t row;
  __device__ Place(const CParams& p, uint32_t s, uint32_t w) {
    constexpr uint32_t NG = D / 32;
    t = w & 3;
    c = (w >> 2) % NG;
    const uint32_t r = (w >> 2) / NG;
    i = r / (uint32_t)p.kv_heads;
    h = r - i * (uint32_t)p.kv_heads;
    const int start = p.start ? p.start[s] : 0;
    const int64_t slot = (int64_t)start + i;
    row = -1;
    if (start >= 0) {
      if (slot < p.capacity) row = ((int64_t)s * p.kv_heads + h) * p.capacity + slot;
      else if (t == 0 && c == 0) atomicOr(&g_cache_err, kErrBadIndex);
    }
  }
};

// Largest magnitude of a pair's halves as bf16 bits in each half (the order of the bits of
// non-negative bf16 numbers is that of the numbers, infinity and NaN last).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

template <int D>
__global__ void __launch_bounds__(256) cache4_append_kernel(const __grid_constant__ CParams p) {
  constexpr int NG = D / 32;
  const uint32_t w = blockIdx.x * 256u + threadIdx.x;
  const uint32_t s = blockIdx.y >> 1, m = blockIdx.y & 1;
  const bool in = w < p.words;                       // whole runs: four threads in or out together
  const Place<D> at(p, s, in ? w : 0u);
  uint32_t v[4] = {0u, 0u, 0u, 0u};
  if (in) {
    const uint4 r = *reinterpret_cast<const uint4*>(p.x[m] + s * p.sb[m] + at.i * p.sn[m] + at.h * p.sh[m] +
                                                    32 * at.c + 8 * at.t);
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t top = max2(max2(v[0] & kAbs, v[1] & kAbs), max2(v[2] & kAbs, v[3] & kAbs));
  top = max2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t amax = max(top & 0xffffu, top >> 16);             // bf16 bits
  // a run with an infinity or a NaN has the scale NaN
  const __nv_bfloat16 sb =
      __float2bfloat16_rn(amax >= 0x7f80u ? __int_as_float(0x7fc00000) : __fdiv_rn(__uint_as_float(amax << 16), 7.f));
  float sc = __bfloat162float(sb);
  // scales below 2^-64 (the last ones subnormal): 1 / s would overflow, so x and s are taken times
  // 2^70, exactly; and there s = amax / 7 is so coarse that a code can come out past 7
  const bool tiny = sc < 5.421010862427522e-20f;
  const float up = tiny ? 1.1805916207174113e21f : 1.f;
  sc *= up;
  const float inv = sc > 0.f ? __fdiv_rn(1.f, sc) * up : 0.f;      // NaN: 0
  uint32_t word = 0u;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float x = __uint_as_float(u & 1 ? v[u >> 1] & 0xffff0000u : v[u >> 1] << 16);
    float q = x * inv;
    if (tiny) q = fminf(fmaxf(x * up * (sc > 0.f ? __fdiv_rn(1.f, sc) : 0.f), -7.f), 7.f);
    // to a multiple of 2^-15, then to an integer, stored + 8 in the last bits of 1.5 x 2^23 + code
    const float e = __fadd_rn(__fadd_rn(q, 384.f), -384.f);
    word |= (__float_as_uint(__fadd_rn(e, 12582920.f)) & 15u) << bit_of(u);
  }
  if (amax >= 0x7f80u) word = 0x88888888u;
  if (in && at.row >= 0) {
    p.codes[m][at.row * (D / 8) + at.t * NG + at.c] = word;
    if (at.t == 0) p.scales[m][at.row * NG + at.c] = sb;
  }
}

template <int D>
__global__ void __launch_bounds__(256) cache4_read_kernel(const __grid_constant__ CParams p) {
  constexpr int NG = D / 32;
  const uint32_t w = blockIdx.x * 256u + threadIdx.x;
  const uint32_t s = blockIdx.y >> 1, m = blockIdx.y & 1;
  if (w >= p.words) return;
  const Place<D> at(p, s, w);
  uint32_t word = 0x88888888u;                       // rows outside the cache read as zeros
  __nv_bfloat16 sc = __float2bfloat16_rn(0.f);
  if (at.row >= 0) {
    word = p.codes[m][at.row * (D / 8) + at.t * NG + at.c];
    sc = p.scales[m][at.row * NG + at.c];
  }
  // pair k of the word is elements 2k, 2k + 1: 128 + code over the bits of 128, exact, minus 136,
  // times the scale with one rounding
  const __nv_bfloat162 s2 = __halves2bfloat162(sc, sc), off = __floats2bfloat162_rn(136.f, 136.f);
  uint32_t v[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const uint32_t x = ((word >> (4 * k)) & 0x000f000fu) | 0x43004300u;
    const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), off), s2);
    v[k] = *reinterpret_cast<const uint32_t*>(&y);
  }
  *reinterpret_cast<uint4*>(p.x[m] + s * p.sb[m] + at.i * p.sn[m] + at.h * p.sh[m] + 32 * at.c + 8 * at.t) =
      make_uint4(v[0], v[1], v[2], v[3]);
}

template <int D>
int launch(const Cache4Args& a, const CParams& p, cudaStream_t stream) {
  const dim3 grid((p.words + 255u) / 256u, 2 * a.batch);
  if (a.read) cache4_read_kernel<D><<<grid, 256, 0, stream>>>(p);
  else cache4_append_kernel<D><<<grid, 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

int launch_cache4(const Cache4Args& a, cudaStream_t stream) {
  CParams p;
  p.x[0] = static_cast<__nv_bfloat16*>(a.k);
  p.x[1] = static_cast<__nv_bfloat16*>(a.v);
  p.codes[0] = reinterpret_cast<uint32_t*>(a.k_codes);
  p.codes[1] = reinterpret_cast<uint32_t*>(a.v_codes);
  p.scales[0] = static_cast<__nv_bfloat16*>(a.k_scales);
  p.scales[1] = static_cast<__nv_bfloat16*>(a.v_scales);
  p.start = a.start;
  for (int m = 0; m < 2; ++m) {
    const int64_t* st = m ? a.v_strides : a.k_strides;
    p.sb[m] = st[0];
    p.sn[m] = st[1];
    p.sh[m] = st[2];
  }
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.words = (uint32_t)a.n_tokens * a.kv_heads * (a.head_dim / 8);
  switch (a.head_dim) {
    case 32: return launch<32>(a, p, stream);
    case 64: return launch<64>(a, p, stream);
    case 128: return launch<128>(a, p, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int cache4_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_cache_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_cache_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
