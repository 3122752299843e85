// Key / value cache in 4 bits: writing rows to it and reading them back (bandwidth bound: bf16
// rows one way, 4.5 bits an element the other).
//
// A row is one (token, key head). Each run of 32 elements has the bf16 scale s = amax / 7, and an
// element x the code round(x / s) (ties to even) in -7 .. 7, stored + 8 (s = 0: code 0). Both
// divisions are the correctly rounded ones, and neither quotient can come so near a border of
// the next rounding that the first one moves it across: x has 8 significant bits, a border times s
// (or times 7) at most 12, so they are equal or differ by 2^-12 and more. A run with an infinity or
// a NaN gets that scale, and reads back as NaN.
//   codes  [batch][kv_heads][capacity][d / 2] bytes: little-endian 32-bit word t * (d / 32) + c holds
//          elements 32 c + 8 t + u, u = 0 .. 7; u = 4 p + i stands at bit 8 p + 4 (i / 2) + 16 (i % 2)
//   scales [batch][kv_heads][capacity][d / 32] bf16
// The word order puts what one lane of the decoding kernel's fragments needs side by side: word
// (t, c) for all c in one load, pairs (2k, 2k + 1) in the two half-words at the same nibble.
//
// One thread per word: 16 bytes of the row, the run's maximum over its four threads by shuffles.
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
  int n, kv_heads, capacity;
  int64_t words;                    // 32-bit words of all rows
};

__host__ __device__ constexpr int bit_of(int u) { return 8 * (u >> 2) + 4 * ((u & 3) >> 1) + 16 * (u & 1); }

// Thread's word: sequence s, token i of the call, head h, run c, word t of the run; the cache row,
// or -1 (out of range: reported; start < 0: the sequence is left out, not reported).
template <int D>
struct Place {
  int s, i, h, c, t;
  int64_t row;
  __device__ Place(const CParams& p, int64_t w) {
    constexpr int NG = D / 32;
    t = (int)(w & 3);
    c = (int)((w >> 2) % NG);
    const int64_t r = (w >> 2) / NG;
    h = (int)(r % p.kv_heads);
    const int64_t si = r / p.kv_heads;
    i = (int)(si % p.n);
    s = (int)(si / p.n);
    const int start = p.start ? p.start[s] : 0;
    const int64_t slot = (int64_t)start + i;
    row = -1;
    if (start >= 0) {
      if (slot < p.capacity) row = ((int64_t)s * p.kv_heads + h) * p.capacity + slot;
      else if (t == 0 && c == 0) atomicOr(&g_cache_err, kErrBadIndex);
    }
  }
};

template <int D>
__global__ void __launch_bounds__(256) cache4_append_kernel(const __grid_constant__ CParams p) {
  constexpr int NG = D / 32;
  const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int m = blockIdx.y;
  const bool in = w < p.words;                       // whole runs: four threads in or out together
  const Place<D> at(p, in ? w : 0);
  uint32_t v[4] = {0u, 0u, 0u, 0u};
  if (in) {
    const uint4 r = *reinterpret_cast<const uint4*>(p.x[m] + at.s * p.sb[m] + at.i * p.sn[m] + at.h * p.sh[m] +
                                                    32 * at.c + 8 * at.t);
    v[0] = r.x; v[1] = r.y; v[2] = r.z; v[3] = r.w;
  }
  float x[8];
  float amax = 0.f;
  int odd = 0;                                       // an infinity or a NaN in the run
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    x[u] = __uint_as_float(u & 1 ? v[u >> 1] & 0xffff0000u : v[u >> 1] << 16);
    const float a = fabsf(x[u]);
    odd |= a < __int_as_float(0x7f800000) ? 0 : 1;
    amax = fmaxf(amax, a);
  }
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
  amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
  odd |= __shfl_xor_sync(0xffffffffu, odd, 1);
  odd |= __shfl_xor_sync(0xffffffffu, odd, 2);
  const __nv_bfloat16 sb = __float2bfloat16_rn(odd ? __int_as_float(0x7fc00000) : __fdiv_rn(amax, 7.f));
  const float s = __bfloat162float(sb);
  uint32_t word = 0u;
#pragma unroll
  for (int u = 0; u < 8; ++u) {
    const float q = s > 0.f ? rintf(__fdiv_rn(x[u], s)) : 0.f;
    const int code = (int)fminf(fmaxf(q, -7.f), 7.f) + 8;
    word |= (uint32_t)code << bit_of(u);
  }
  if (in && at.row >= 0) {
    p.codes[m][at.row * (D / 8) + at.t * NG + at.c] = word;
    if (at.t == 0) p.scales[m][at.row * NG + at.c] = sb;
  }
}

template <int D>
__global__ void __launch_bounds__(256) cache4_read_kernel(const __grid_constant__ CParams p) {
  constexpr int NG = D / 32;
  const int64_t w = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int m = blockIdx.y;
  if (w >= p.words) return;
  const Place<D> at(p, w);
  uint32_t word = 0x88888888u;                       // rows outside the cache read as zeros
  float s = 0.f;
  if (at.row >= 0) {
    word = p.codes[m][at.row * (D / 8) + at.t * NG + at.c];
    s = __bfloat162float(p.scales[m][at.row * NG + at.c]);
  }
  uint32_t v[4];
#pragma unroll
  for (int u = 0; u < 8; u += 2) {
    const float a = (float)((int)((word >> bit_of(u)) & 15u) - 8) * s;
    const float b = (float)((int)((word >> bit_of(u + 1)) & 15u) - 8) * s;
    v[u >> 1] = pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4*>(p.x[m] + at.s * p.sb[m] + at.i * p.sn[m] + at.h * p.sh[m] + 32 * at.c + 8 * at.t) =
      make_uint4(v[0], v[1], v[2], v[3]);
}

template <int D>
int launch(const Cache4Args& a, const CParams& p, cudaStream_t stream) {
  const dim3 grid((unsigned)((p.words + 255) / 256), 2);
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
  p.n = a.n_tokens;
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.words = (int64_t)a.batch * a.n_tokens * a.kv_heads * (a.head_dim / 8);
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
