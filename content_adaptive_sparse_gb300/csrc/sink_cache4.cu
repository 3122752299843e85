// Key / value cache in 4 bits: writing rows to it and reading them back (bandwidth bound: bf16
// rows one way, 4.5 bits an element the other).
//
// A row is one (token, key head). Each run of 32 elements has the bf16 scale s = amax / 7, and an
// element x the code round(x / s) (ties to even) in -7 .. 7, stored + 8 (s = 0: code 0). A run with an
// infinity or a NaN has the scale NaN and reads back as NaN. amax has 8 significant bits, and a
// border between two bf16 numbers, an odd number of 9 bits, is odd and of 11 bits and more when
// taken 7 times: amax / 7 is never on a border, and 2^-13 of its size or more away from it.
//   codes  [batch][kv_heads][capacity][d / 2] bytes: little-endian 32-bit word t * (d / 32) + c holds
//          elements 32 c + 8 t + u, u = 0 .. 7; u = 4 p + i stands at bit 8 p + 4 (i / 2) + 16 (i % 2)
//   scales [batch][kv_heads][capacity][d / 32] bf16
// The word order puts what one lane of the decoding kernel's fragments needs side by side: word
// (t, c) for all c in one load, pairs (2k, 2k + 1) in the two half-words at the same nibble.
//
// One thread per word at a time: 16 bytes of the row, the run's maximum over its four threads by
// shuffles.
// The rounding takes no division: the approximate q = x (1 / s) is off by less than 2^-19, while a
// quotient lies on a border (k + 1/2) or 2^-10 and more away from it, so q is first rounded to a
// multiple of 2^-15 (by adding 384, whose last place that is), which puts a border's quotient back on
// the border, and then to the nearest even integer. In the same way
// amax times fp32's 1 / 7 rounds to the bf16 number that amax / 7 does.
//
// Measured, K and V of 2 x 16384 tokens, 8 heads of 128 (172 MB): append 30.9 us (5.6 TB/s; 40 with one
// element an instruction and a multiplication per address; bound by its instructions, ~100 a word),
// read 28.0 us (6.1 TB/s).
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "f32x2.cuh"
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
  uint32_t div_m, div_s;            // r / kv_heads = r * div_m >> div_s for r < 2^31
  // 256 words on: step_i tokens and step_h heads, and one token on where that passes the last head;
  // the same in elements of x and in cache rows
  uint32_t step_i, step_h;
  int64_t x_step[2], x_wrap[2], row_step, row_wrap;
};

__host__ __device__ constexpr int bit_of(int u) { return 8 * (u >> 2) + 4 * ((u & 3) >> 1) + 16 * (u & 1); }

// A thread's words: run c and word t of it, the same for all its words (256 words are whole
// rows), and per word token i of the call and head h. Addresses are found by additions.
template <int D, int M, bool WRAP>
struct Place {
  static constexpr uint32_t NG = D / 32;
  uint32_t c, t, h, i;
  __nv_bfloat16* x;                 // the word's elements
  int64_t row;                      // the cache row of slot `start` 0
  __device__ Place(const CParams& p, uint32_t s, uint32_t w) {
    t = w & 3;
    c = (w >> 2) % NG;
    const uint32_t r = (w >> 2) / NG;
    i = (uint32_t)(((uint64_t)r * p.div_m) >> p.div_s);
    h = r - i * (uint32_t)p.kv_heads;
    x = p.x[M] + s * p.sb[M] + i * p.sn[M] + h * p.sh[M] + 32 * c + 8 * t;
    row = ((int64_t)s * p.kv_heads + h) * p.capacity + i;
  }
  __device__ __forceinline__ void next(const CParams& p) {
    i += p.step_i;
    h += p.step_h;
    x += p.x_step[M];
    row += p.row_step;
    if (WRAP && h >= (uint32_t)p.kv_heads) {
      h -= (uint32_t)p.kv_heads;
      ++i;
      x += p.x_wrap[M];
      row += p.row_wrap;
    }
  }
  // whether the word's row is in the cache (past it: reported; start < 0: the sequence is left out, not
  // reported)
  __device__ __forceinline__ bool in(const CParams& p, int start) const {
    if (start < 0) return false;
    if ((uint32_t)start + i < (uint32_t)p.capacity) return true;   // the sum is below 2^32
    if (t == 0 && c == 0) atomicOr(&g_cache_err, kErrBadIndex);
    return false;
  }
};

// Largest magnitude of a pair's halves as bf16 bits in each half (the order of the bits of
// non-negative bf16 numbers is that of the numbers, infinity and NaN last).
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) { return __vmaxu2(a, b); }

__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// The code word of 8 elements (bf16 pairs v), and their run's scale (all 32 lanes call).
__device__ __forceinline__ uint32_t quantise(const uint4& r, __nv_bfloat16& scale) {
  const uint32_t v[4] = {r.x, r.y, r.z, r.w};
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t top = max2(max2(v[0] & kAbs, v[1] & kAbs), max2(v[2] & kAbs, v[3] & kAbs));
  top = max2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint32_t amax = max(top & 0xffffu, top >> 16);             // bf16 bits
  // a run with an infinity or a NaN has the scale NaN
  scale = __float2bfloat16_rn(amax >= 0x7f80u ? __int_as_float(0x7fc00000)
                                              : __uint_as_float(amax << 16) * 0.14285714924335480f);
  const float sc = __bfloat162float(scale);
  uint32_t word = 0u;
  if (!(sc < 5.421010862427522e-20f)) {
    const float inv = rcp_approx(sc);                // NaN: the codes are not used
    // x / s + 384 to a multiple of 2^-15, then, with 8 more, to an integer in the last bits of 1.5 x 2^23;
    // the numbers' low halves are the codes, pair e's at nibble e
    const uint64_t inv2 = f2::pack(inv, inv), grid = f2::pack(384.f, 384.f), last = f2::pack(12582536.f, 12582536.f);
    uint32_t pair[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint64_t x = f2::pack(__uint_as_float(v[e] << 16), __uint_as_float(v[e] & 0xffff0000u));
      float lo, hi;
      f2::unpack(f2::add(f2::fma(x, inv2, grid), last), lo, hi);
      pair[e] = __byte_perm(__float_as_uint(lo), __float_as_uint(hi), 0x5410);
    }
    word = ((pair[3] * 16u + pair[2]) * 16u + pair[1]) * 16u + pair[0];
    if (amax >= 0x7f80u) word = 0x88888888u;
  } else {
    // scales below 2^-64, the last ones subnormal: 1 / s could overflow, and s can be so coarse that
    // a code comes out past 7; the division and the limits then
#pragma unroll 1
    for (int u = 0; u < 8; ++u) {
      const uint32_t pair = u < 4 ? (u < 2 ? v[0] : v[1]) : (u < 6 ? v[2] : v[3]);
      const float x = __uint_as_float(u & 1 ? pair & 0xffff0000u : pair << 16);
      const float q = sc > 0.f ? fminf(fmaxf(rintf(__fdiv_rn(x, sc)), -7.f), 7.f) : 0.f;
      word |= (uint32_t)((int)q + 8) << bit_of(u);
    }
  }
  return word;
}

template <int D, int M, int kWords, bool WRAP>
__device__ __forceinline__ void append_words(const CParams& p, uint32_t s, uint32_t w, int start) {
  constexpr uint32_t NG = D / 32;
  const Place<D, M, WRAP> first(p, s, w);
  uint4 v[kWords];
  Place<D, M, WRAP> at = first;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {                 // whole runs: four threads in or out together
    v[k] = make_uint4(0u, 0u, 0u, 0u);
    if (w + 256u * k < p.words) v[k] = *reinterpret_cast<const uint4*>(at.x);
    at.next(p);
  }
  at = first;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    __nv_bfloat16 scale;
    const uint32_t word = quantise(v[k], scale);
    if (w + 256u * k < p.words && at.in(p, start)) {
      const int64_t row = at.row + start;
      p.codes[M][row * (D / 8) + at.t * NG + at.c] = word;
      if (at.t == 0) p.scales[M][row * NG + at.c] = scale;
    }
    at.next(p);
  }
}

template <int D, int M, int kWords, bool WRAP>
__device__ __forceinline__ void read_words(const CParams& p, uint32_t s, uint32_t w, int start) {
  constexpr uint32_t NG = D / 32;
  const Place<D, M, WRAP> first(p, s, w);
  uint32_t word[kWords];
  __nv_bfloat16 scale[kWords];
  Place<D, M, WRAP> at = first;
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    word[k] = 0x88888888u;                           // rows outside the cache read as zeros
    scale[k] = __float2bfloat16_rn(0.f);
    if (w + 256u * k < p.words && at.in(p, start)) {
      const int64_t row = at.row + start;
      word[k] = p.codes[M][row * (D / 8) + at.t * NG + at.c];
      scale[k] = p.scales[M][row * NG + at.c];
    }
    at.next(p);
  }
  at = first;
  const __nv_bfloat162 off = __floats2bfloat162_rn(136.f, 136.f);
#pragma unroll
  for (int k = 0; k < kWords; ++k) {
    // pair e of the word is elements 2e, 2e + 1: 128 + code over the bits of 128, exact, minus 136,
    // times the scale with one rounding
    const __nv_bfloat162 s2 = __halves2bfloat162(scale[k], scale[k]);
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t x = ((word[k] >> (4 * e)) & 0x000f000fu) | 0x43004300u;
      const __nv_bfloat162 y = __hmul2(__hsub2(*reinterpret_cast<const __nv_bfloat162*>(&x), off), s2);
      v[e] = *reinterpret_cast<const uint32_t*>(&y);
    }
    if (w + 256u * k < p.words) *reinterpret_cast<uint4*>(at.x) = make_uint4(v[0], v[1], v[2], v[3]);
    at.next(p);
  }
}

// One CTA per 256 kWords words of a sequence's keys or values (K and V interleaved in y). The append's
// registers are held to five CTAs an SM (35.0 -> 32.8 us below).
template <int D, bool READ, int kWords>
__global__ void __launch_bounds__(256, READ ? 8 : (kWords > 1 ? 5 : 1)) cache4_kernel(const __grid_constant__ CParams p) {
  const uint32_t w = blockIdx.x * (256u * kWords) + threadIdx.x, s = blockIdx.y >> 1;
  const int start = p.start ? p.start[s] : 0;
  const auto words = [&](auto m, auto wrap) {
    if constexpr (READ) read_words<D, decltype(m)::value, kWords, decltype(wrap)::value>(p, s, w, start);
    else append_words<D, decltype(m)::value, kWords, decltype(wrap)::value>(p, s, w, start);
  };
  using K = std::integral_constant<int, 0>;
  using V = std::integral_constant<int, 1>;
  // where kv_heads divides the rows of 256 words, a thread's words are all of one head (append 33.0 ->
  // 30.9 us)
  if (kWords > 1 && p.step_h == 0) {
    if (blockIdx.y & 1) words(V(), std::false_type());
    else words(K(), std::false_type());
  } else {
    if (blockIdx.y & 1) words(V(), std::true_type());
    else words(K(), std::true_type());
  }
}

template <int D>
int launch(const Cache4Args& a, CParams& p, cudaStream_t stream) {
  const uint32_t rows = 256 / (D / 8);               // rows in 256 words
  p.step_i = rows / (uint32_t)a.kv_heads;
  p.step_h = rows % (uint32_t)a.kv_heads;
  for (int m = 0; m < 2; ++m) {
    p.x_step[m] = p.step_i * p.sn[m] + p.step_h * p.sh[m];
    p.x_wrap[m] = p.sn[m] - a.kv_heads * p.sh[m];
  }
  p.row_step = (int64_t)p.step_h * p.capacity + p.step_i;
  p.row_wrap = 1 - (int64_t)a.kv_heads * p.capacity;
  // Four words a thread, all loaded before the first is worked on, where that still gives every SM
  // several CTAs (K and V of 2 x 16384 tokens: append 49 -> 40 us, read 41 -> 28 us); one word a thread
  // in smaller calls, whose time is one thread's latency (64 sequences of one token: append 3.2 ->
  // 2.0 us).
  const bool many = (int64_t)p.words * 2 * a.batch >= (int64_t)1024 * 4 * current_sm_count();
  const uint32_t per = many ? 1024u : 256u;
  const dim3 grid((p.words + per - 1) / per, 2 * a.batch);
  if (many) {
    if (a.read) cache4_kernel<D, true, 4><<<grid, 256, 0, stream>>>(p);
    else cache4_kernel<D, false, 4><<<grid, 256, 0, stream>>>(p);
  } else {
    if (a.read) cache4_kernel<D, true, 1><<<grid, 256, 0, stream>>>(p);
    else cache4_kernel<D, false, 1><<<grid, 256, 0, stream>>>(p);
  }
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
  // x / d = x * m >> (31 + k), 2^k >= d, m = ceil(2^(31 + k) / d): m d is off 2^(31 + k) by less than
  // d <= 2^k, so x < 2^31 times that stays below 2^(31 + k)
  uint32_t k = 0;
  while ((1u << k) < (uint32_t)a.kv_heads) ++k;
  p.div_s = 31 + k;
  p.div_m = (uint32_t)(((1ull << p.div_s) + a.kv_heads - 1) / a.kv_heads);
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
