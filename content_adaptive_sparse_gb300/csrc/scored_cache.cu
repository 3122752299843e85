// A cache of slots whose rows carry the attention weight that they have gathered: rows go in one behind the
// other, and an eviction keeps `keep` slots of every (sequence, key head): those of the first `sinks` and
// the newest `recent` tokens, then the ones of most weight (ties: the lower slot). Attention does not depend
// on the order of a sequence's keys, so the kept rows stay where they are, and only those at or past slot `keep`
// move, the e-th of them into the e-th freed slot below it: no row that stays is read.
//
// Eviction: one launch, no workspace. A cluster's CTAs take one (sequence, key head); each finds the whole
// selection for itself (8 bytes a slot) and moves its share of the rows (8 D bytes each, there and back):
//   key      32 bits that order like the weight; a protected slot has the largest key
//   select   the keep-th largest key T, by histograms in shared memory of 2048 bins over the range that the keys
//            really have: the bin that holds T is the next range (two rounds mostly, where eight bits a round from the top took
//            four: 16.3 -> 12.1 us for 64 caches)
//   flags    a bit per slot: freed (below `keep`) or to move (from `keep` on), counted so that the e-th freed slot
//            meets the e-th row to move (up to 8192 slots as pairs of slots, longer lists by counts per 256 slots)
// The ranks meet before the first write, since outputs may lie over the inputs.
//
// Measured: 64 caches of 4 key heads of 128 that give up one row of 4097: 7.3 us, latency (loads, three reductions, one row).
// 32 caches of 5001 to 8192 slots cut to 4096: 50 us; the bytes of the rows take 30 at the copy rate,
// the selection comes before any row moves (its instructions, once per rank), the rest is launch and unequal lists.
// Both with outputs elsewhere; in place the lengths are cut by a second launch: 0.8 and 1.1 us more. The form of up to 8192 slots
// spills 16 to 32 bytes a thread at 64 registers, the price of two CTAs an SM.
#include <cooperative_groups.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>
#include <string.h>

#include "key_range.h"
#include "sa_internal.h"

namespace sa {
namespace {

__device__ unsigned int g_scored_err;

// ------------------------------------------------------------------ append

struct AppendParams {
  const uint4* x[2];                // k, v
  uint4* cache[2];
  int64_t x_sb[2], x_sn[2], x_sh[2], c_sb[2], c_sn[2], c_sh[2];   // 16-byte words
  const int32_t* start;
  const int32_t* tokens;
  float* weights;
  int32_t* positions;
  int n, kv_heads, capacity;
  uint32_t words;                   // 16-byte words of a sequence's keys
};

template <int D>
__global__ void __launch_bounds__(256) append_kernel(const __grid_constant__ AppendParams p) {
  const uint32_t w = blockIdx.x * 256u + threadIdx.x;
  const int s = blockIdx.y >> 1, m = blockIdx.y & 1;
  const int start = p.start ? p.start[s] : 0;
  if (w >= p.words || start < 0) return;
  const int u = (int)(w % (D / 8)), row = (int)(w / (D / 8)), hk = row % p.kv_heads, i = row / p.kv_heads;
  const int64_t slot = (int64_t)start + i;
  if (slot >= p.capacity) {
    if (u == 0 && hk == 0 && m == 0) atomicOr(&g_scored_err, kErrBadIndex);
    return;
  }
  p.cache[m][s * p.c_sb[m] + slot * p.c_sn[m] + hk * p.c_sh[m] + u] = p.x[m][s * p.x_sb[m] + i * p.x_sn[m] + hk * p.x_sh[m] + u];
  if (m == 0 && u == 0) {
    const int64_t at = ((int64_t)s * p.kv_heads + hk) * p.capacity + slot;
    p.weights[at] = 0.f;
    p.positions[at] = p.tokens ? (int32_t)((uint32_t)p.tokens[s] + (uint32_t)i) : (int32_t)slot;
  }
}

// ------------------------------------------------------------------ eviction

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kOwn = 16;               // slots of a thread whose keys stay in registers
constexpr int kSmall = kOwn * kThreads;
constexpr int kCachedKeys = 32768;     // longer lists' keys are formed anew in every pass
constexpr int kGroup = 256;            // long lists: slots per count
constexpr uint32_t kSafe = 0xffffffffu;

struct EvictParams {
  uint4* cache[2];
  int64_t c_sb[2], c_sn[2], c_sh[2];
  const float* w_in;
  const int32_t* pos_in;
  const int32_t* len_in;
  float* w_out;
  int32_t* pos_out;
  int32_t* len_out;                    // null: written by a launch of its own
  int kv_heads, capacity, keep, sinks, recent;
  int cached;                          // long lists: keys are kept in shared memory
};

// Orders like the weight; NaN counts as more than infinity, -0 as 0. Protected slots have kSafe.
__device__ __forceinline__ uint32_t key_of(float w, int pos, int sinks, int newest, int recent) {
  const uint32_t b = __float_as_uint(w + 0.f);
  uint32_t k = b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
  if (w != w) k = kSafe - 1;
  if (pos < sinks || (uint32_t)newest - (uint32_t)pos < (uint32_t)recent) k = kSafe;
  return k;
}

// Sum over the CTA's threads before this one, and in all (two barriers).
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& all) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const auto scan = [&](int x) {
#pragma unroll
    for (int o = 1; o < 32; o *= 2) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x;
  };
  const int x = scan(v);
  __syncthreads();                     // the sums of the call before have been read
  if (lane == 31) warp_sums[warp] = x;
  __syncthreads();
  const int y = lane < kWarps ? warp_sums[lane] : 0;
  all = __reduce_add_sync(0xffffffffu, y);
  return __reduce_add_sync(0xffffffffu, lane < warp ? y : 0) + x - v;
}

// Long lists: slot of the e-th (from 0) set flag.
__device__ __forceinline__ int select_flag(const uint32_t* flags, const int* counts, int groups, int e) {
  int lo = 0, hi = groups - 1;         // counts[g]: flags before group g
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (counts[mid] <= e) lo = mid;
    else hi = mid - 1;
  }
  e -= counts[lo];
  int w = lo * (kGroup / 32);
  for (int n = __popc(flags[w]); e >= n; n = __popc(flags[w])) {
    e -= n;
    ++w;
  }
  uint32_t bits = flags[w];
  int at = 32 * w;
#pragma unroll
  for (int half = 16; half > 0; half /= 2) {
    const int low = __popc(bits & ((1u << half) - 1u));
    if (e >= low) {
      e -= low;
      bits >>= half;
      at += half;
    }
  }
  return at;
}

// Shared memory of a list of `capacity` slots: flags, counts and keys (long), or the pairs of slots (SMALL).
__host__ __device__ inline int evict_groups(int capacity) { return (capacity + kGroup - 1) / kGroup; }
inline int evict_smem(int capacity, bool small, bool cached, int moves) {
  return small ? 4 * moves : evict_groups(capacity) * (kGroup / 8 + 4) + (cached ? 4 * capacity : 0);
}

// SMALL: up to 8192 slots. A thread's weights and positions are loaded at once and its keys stay in registers,
// and every move is written out as a pair of 16-bit slots.
template <int D, bool SMALL>
__global__ void __launch_bounds__(kThreads, SMALL ? 2 : 1) evict_kernel(const __grid_constant__ EvictParams p) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ __align__(16) int hist[KeyRange::kBins];
  __shared__ int warp_sums[kWarps];
  __shared__ uint32_t warp_low[kWarps], warp_high[kWarps];
  __shared__ int found[3];
  __shared__ __align__(16) int word_count[SMALL ? kSmall / 32 : 4];
  cg::cluster_group cluster = cg::this_cluster();
  const int rank = blockIdx.x, ranks = gridDim.x, hk = blockIdx.y, s = blockIdx.z;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int len = max(0, min(p.len_in[s], p.capacity)), keep = p.keep;
  const int64_t list = ((int64_t)s * p.kv_heads + hk) * p.capacity;
  const float* w_in = p.w_in + list;
  const int32_t* pos_in = p.pos_in + list;
  float* w_out = p.w_out + list;
  int32_t* pos_out = p.pos_out + list;
  const bool copy = w_out != w_in || pos_out != pos_in;
  if (p.len_out && rank == 0 && hk == 0 && threadIdx.x == 0) p.len_out[s] = min(len, keep);
  if (len <= keep) {                   // the whole cluster
    if (rank == 0 && copy)
      for (int j = threadIdx.x; j < len; j += kThreads) {
        w_out[j] = w_in[j];
        pos_out[j] = pos_in[j];
      }
    return;
  }
  const auto meet = [&] {
    if (ranks > 1) cluster.sync();
    else __syncthreads();
  };
  uint32_t* flags = reinterpret_cast<uint32_t*>(smem);
  const int words = (len + 31) / 32, groups = (len + kGroup - 1) / kGroup;
  int* counts = reinterpret_cast<int*>(flags + evict_groups(p.capacity) * (kGroup / 32));
  uint32_t* keys = reinterpret_cast<uint32_t*>(counts + evict_groups(p.capacity));
  // ---- the newest token
  uint32_t key_own[SMALL ? kOwn : 1];
  int pos_own[SMALL ? kOwn : 1];
  int newest = INT32_MIN;
  if constexpr (SMALL) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = i * kThreads + threadIdx.x;
      pos_own[i] = j < len ? pos_in[j] : INT32_MIN;
      key_own[i] = j < len ? __float_as_uint(w_in[j]) : 0u;          // the weight as yet
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) newest = max(newest, pos_own[i]);
    // outputs elsewhere: the slots below `keep` at once, the ranks' rounds in turn; freed ones are written again
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = i * kThreads + threadIdx.x;
      if (j >= keep || i % ranks != rank) continue;
      if (w_out != w_in) w_out[j] = __uint_as_float(key_own[i]);
      if (pos_out != pos_in) pos_out[j] = pos_own[i];
    }
  } else {
#pragma unroll 8
    for (int j = threadIdx.x; j < len; j += kThreads) newest = max(newest, pos_in[j]);
  }
  newest = __reduce_max_sync(0xffffffffu, newest);
  if (lane == 0) warp_sums[warp] = newest;
  __syncthreads();
  newest = __reduce_max_sync(0xffffffffu, warp_sums[lane % kWarps]);
  const auto form = [&](int j) { return key_of(w_in[j], pos_in[j], p.sinks, newest, p.recent); };
  if constexpr (SMALL) {
#pragma unroll
    for (int i = 0; i < kOwn; ++i) key_own[i] = key_of(__uint_as_float(key_own[i]), pos_own[i], p.sinks, newest, p.recent);
  } else if (p.cached) {
#pragma unroll 4
    for (int j = threadIdx.x; j < len; j += kThreads) keys[j] = form(j);
  }
  reinterpret_cast<int4*>(hist)[threadIdx.x] = make_int4(0, 0, 0, 0);
  // f(slot, key, whether there is such a slot) for this thread's slots; all lanes of a warp at once
  const auto for_slots = [&](auto f) {
    if constexpr (SMALL) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) {
        const int j = i * kThreads + threadIdx.x;
        if (j - lane < len) f(j, key_own[i], j < len);
      }
    } else {
#pragma unroll 1
      for (int j = threadIdx.x; j - lane < len; j += kThreads) {
        const bool on = j < len;
        f(j, on ? (p.cached ? keys[j] : form(j)) : 0u, on);
      }
    }
  };
  // ---- the protected slots, and the range of the others' keys
  int mine = 0;
  uint32_t low = kSafe, high = 0;
  for_slots([&](int, uint32_t k, bool on) {
    const bool safe = k == kSafe;
    mine += on && safe ? 1 : 0;
    low = on ? min(low, k) : low;
    high = on && !safe ? max(high, k) : high;
  });
  mine = __reduce_add_sync(0xffffffffu, mine);
  low = __reduce_min_sync(0xffffffffu, low);
  high = __reduce_max_sync(0xffffffffu, high);
  __syncthreads();                     // warp_sums has been read
  if (lane == 0) {
    warp_sums[warp] = mine;
    warp_low[warp] = low;
    warp_high[warp] = high;
  }
  __syncthreads();
  int equal = __reduce_add_sync(0xffffffffu, lane < kWarps ? warp_sums[lane] : 0), left = keep;
  low = __reduce_min_sync(0xffffffffu, warp_low[lane % kWarps]);
  high = __reduce_max_sync(0xffffffffu, warp_high[lane % kWarps]);
  // ---- One row too many, as in every step of a full cache: it is the highest slot with the lowest key (64 lists of 4097 slots:
  // 10.4 us in a row of launches, 14.5 by the general way).
  int victim = -1;
  if (len == keep + 1) {
    for_slots([&](int j, uint32_t k, bool on) { victim = on && k == low ? max(victim, j) : victim; });
    victim = __reduce_max_sync(0xffffffffu, victim);
    __syncthreads();                   // warp_sums has been read
    if (lane == 0) warp_sums[warp] = victim;
    __syncthreads();
    victim = __reduce_max_sync(0xffffffffu, warp_sums[lane % kWarps]);
    meet();                            // every rank has read what the outputs may lie over, and copied
    if (rank != 0) return;
    if constexpr (!SMALL) {
      for (int j = threadIdx.x; copy && j < keep; j += kThreads) {
        if (j == victim) continue;
        w_out[j] = w_in[j];
        pos_out[j] = pos_in[j];
      }
    }
    if (victim == keep) return;
    if (threadIdx.x == 0) {
      w_out[victim] = w_in[keep];
      pos_out[victim] = pos_in[keep];
    }
    if (threadIdx.x < 2 * (D / 8)) {
      const int m = threadIdx.x / (D / 8);
      uint4* rows = p.cache[m] + s * p.c_sb[m] + hk * p.c_sh[m] + threadIdx.x % (D / 8);
      rows[victim * p.c_sn[m]] = rows[keep * p.c_sn[m]];
    }
    return;
  }
  // ---- T, the keep-th largest key: the keys in [low, high] are counted in up to 2048 equal bins, and the bin that
  // holds it is the next range, until all of a bin's keys are to stay or alike. `left` of the range's
  // `equal` keys are still to be kept.
  uint32_t T = kSafe;
  if (equal < keep) {
    left = keep - equal;
    equal = len - equal;
    KeyRange range{low, high};
    T = low;
#pragma unroll 1
    while (left < equal && range.low < range.high) {
      const int shift = range.shift();
      for_slots([&](int, uint32_t k, bool on) {
        if (on && range.holds(k)) atomicAdd(&hist[range.bin(k, shift)], 1);
      });
      __syncthreads();
      // thread t: four bins from the 4 t-th from the top on
      const int b0 = KeyRange::kBins - 4 - 4 * (int)threadIdx.x;
      const int4 n = *reinterpret_cast<const int4*>(hist + b0);
      *reinterpret_cast<int4*>(hist + b0) = make_int4(0, 0, 0, 0);        // for the next round
      const int count[4] = {n.w, n.z, n.y, n.x};
      int all, above = block_scan(n.x + n.y + n.z + n.w, warp_sums, all);
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (above < left && left <= above + count[k]) {
          found[0] = b0 + 3 - k;
          found[1] = above;
          found[2] = count[k];
        }
        above += count[k];
      }
      __syncthreads();
      range.take((uint32_t)found[0], shift);
      left -= found[1];
      equal = found[2];
      T = range.low;
    }
  }
  // ---- which slots stay. Of the keys equal to T the first `left`: their number before each word of 32 slots
  // goes through shared memory (long lists a chunk of words at a time).
  int base = 0, total = 0;             // keys equal to T, and set flags, in the slots before
  const bool some = left < equal;
  const auto flag_of = [&](int j, uint32_t k, bool on, uint32_t same, int before) {
    bool kept = on && k >= T;
    if (some && on && k == T && before + __popc(same & ((1u << lane) - 1u)) >= left) kept = false;
    return on && (j < keep ? !kept : kept);
  };
  int moves;
  if constexpr (SMALL) {
    // Word 16 i + warp holds the slots of this warp's i-th round. before(): set bits before each of this warp's
    // words. Every warp adds the counts up for itself, eight words a lane (this warp's words are all
    // the warp % 8-th of their lane's).
    static_assert(kWarps == 16 && kOwn == 16, "256 words");
    uint32_t bits[kOwn];
    int before[kOwn];
    const auto count = [&](int& all) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i)
        if (lane == 0) word_count[kWarps * i + warp] = __popc(bits[i]);
      __syncthreads();
      int n[8], sum = 0, mine = 0;
#pragma unroll
      for (int k = 0; k < 8; k += 4) {
        const int4 v = *reinterpret_cast<const int4*>(word_count + 8 * lane + k);
        n[k] = v.x;
        n[k + 1] = v.y;
        n[k + 2] = v.z;
        n[k + 3] = v.w;
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        mine += k < (warp & 7) ? n[k] : 0;
        sum += n[k];
      }
      int x = sum;
#pragma unroll
      for (int o = 1; o < 32; o *= 2) {
        const int y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
      }
      all = __shfl_sync(0xffffffffu, x, 31);
      x += mine - sum;
#pragma unroll
      for (int i = 0; i < kOwn; ++i) before[i] = __shfl_sync(0xffffffffu, x, 2 * i + (warp >> 3));
    };
    if (some) {
#pragma unroll
      for (int i = 0; i < kOwn; ++i) bits[i] = __ballot_sync(0xffffffffu, i * kThreads + (int)threadIdx.x < len && key_own[i] == T);
      count(total);
      __syncthreads();
    }
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = i * kThreads + threadIdx.x;
      bits[i] = __ballot_sync(0xffffffffu, flag_of(j, key_own[i], j < len, some ? bits[i] : 0u, some ? before[i] : 0));
    }
    count(total);
    moves = total / 2;
    // the e-th freed slot and the e-th row to move, 16 bits each
    uint16_t* pairs = reinterpret_cast<uint16_t*>(smem);
#pragma unroll
    for (int i = 0; i < kOwn; ++i) {
      const int j = i * kThreads + threadIdx.x;
      if (bits[i] == 0u) continue;     // the whole warp
      if ((bits[i] >> lane) & 1u) {
        const int e = before[i] + __popc(bits[i] & ((1u << lane) - 1u));
        pairs[j < keep ? 2 * e : 2 * (e - moves) + 1] = (uint16_t)j;
      }
    }
    meet();                            // every rank has read what the outputs may lie over, and copied
    for (int e = rank * kThreads + threadIdx.x; e < moves; e += ranks * kThreads) {
      const int dst = pairs[2 * e], src = pairs[2 * e + 1];
      w_out[dst] = w_in[src];
      pos_out[dst] = pos_in[src];
    }
  } else {
#pragma unroll 1
    for (int j0 = 0; j0 < words * 32; j0 += kThreads) {
      const int j = j0 + threadIdx.x;
      const bool on = j < len;
      const uint32_t k = on ? (p.cached ? keys[j] : form(j)) : 0u;
      const uint32_t same = __ballot_sync(0xffffffffu, on && k == T);
      int before = 0;
      if (some) {
        int all;
        before = block_scan(lane == 0 ? __popc(same) : 0, warp_sums, all);
        before = base + __shfl_sync(0xffffffffu, before, 0);
        base += all;
      }
      const uint32_t bits = __ballot_sync(0xffffffffu, flag_of(j, k, on, same, before));
      if (lane == 0 && j < words * 32) flags[j / 32] = bits;
    }
    for (int w = words + threadIdx.x; w < groups * (kGroup / 32); w += kThreads) flags[w] = 0u;
    __syncthreads();
    // counts before each group, and the freed slots (as many as there are rows to move)
#pragma unroll 1
    for (int g0 = 0; g0 < groups; g0 += kThreads) {
      const int g = g0 + threadIdx.x;
      int n = 0;
      if (g < groups)
#pragma unroll
        for (int k = 0; k < kGroup / 32; ++k) n += __popc(flags[g * (kGroup / 32) + k]);
      int all;
      const int before = total + block_scan(n, warp_sums, all);
      if (g < groups) counts[g] = before;
      total += all;
    }
    moves = total / 2;
    meet();                            // every rank has read what the outputs may lie over
    if (rank == 0) {
      for (int j = threadIdx.x; copy && j < keep; j += kThreads) {
        if ((flags[j / 32] >> (j & 31)) & 1u) continue;
        w_out[j] = w_in[j];
        pos_out[j] = pos_in[j];
      }
      for (int e = threadIdx.x; e < moves; e += kThreads) {
        const int dst = select_flag(flags, counts, groups, e), src = select_flag(flags, counts, groups, moves + e);
        w_out[dst] = w_in[src];
        pos_out[dst] = pos_in[src];
      }
    }
  }
  // ---- rows: a warp takes up to 32 moves at a time, D / 8 lanes a row of keys and as many one of values
  constexpr int kLanes = D / 8, kSide = 32 / (2 * kLanes);   // moves side by side
  constexpr int kDeep = 8;             // loads of a lane before its first store
  constexpr int kTake = kSide * kDeep < 32 ? kSide * kDeep : 32;
  const int m = lane / kLanes & 1, u = lane % kLanes, side = lane / (2 * kLanes);
  uint4* rows = p.cache[m] + s * p.c_sb[m] + hk * p.c_sh[m] + u;
  const int64_t sn = p.c_sn[m];
#pragma unroll 1
  for (int e0 = kTake * (rank * kWarps + warp); e0 < moves; e0 += kTake * ranks * kWarps) {
    int src = 0, dst = 0;
    if (lane < kTake && e0 + lane < moves) {
      if constexpr (SMALL) {
        const uint32_t pair = reinterpret_cast<const uint32_t*>(smem)[e0 + lane];
        dst = (int)(pair & 0xffffu);
        src = (int)(pair >> 16);
      } else {
        dst = select_flag(flags, counts, groups, e0 + lane);
        src = select_flag(flags, counts, groups, moves + e0 + lane);
      }
    }
    const int n = min(kTake, moves - e0);
    uint4 x[kDeep];
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int e = k * kSide + side, from = __shfl_sync(0xffffffffu, src, e & 31);
      if (e < n) x[k] = rows[from * sn];
    }
#pragma unroll
    for (int k = 0; k < kDeep; ++k) {
      const int e = k * kSide + side, to = __shfl_sync(0xffffffffu, dst, e & 31);
      if (e < n) rows[to * sn] = x[k];
    }
  }
}

__global__ void cut_lengths_kernel(const int32_t* in, int32_t* out, int n, int capacity, int keep) {
  const int s = blockIdx.x * 256 + threadIdx.x;
  if (s < n) out[s] = max(0, min(min(in[s], capacity), keep));
}

template <int D>
int launch_append(const ScoredArgs& a, cudaStream_t stream) {
  AppendParams p;
  memset(&p, 0, sizeof(p));
  for (int m = 0; m < 2; ++m) {
    const int64_t* x = m ? a.v_strides : a.k_strides;
    const int64_t* c = m ? a.v_cache_strides : a.k_cache_strides;
    p.x[m] = static_cast<const uint4*>(m ? a.v : a.k);
    p.cache[m] = static_cast<uint4*>(m ? a.v_cache : a.k_cache);
    p.x_sb[m] = x[0] / 8;
    p.x_sn[m] = x[1] / 8;
    p.x_sh[m] = x[2] / 8;
    p.c_sb[m] = c[0] / 8;
    p.c_sn[m] = c[1] / 8;
    p.c_sh[m] = c[2] / 8;
  }
  p.start = a.start;
  p.tokens = a.tokens;
  p.weights = a.weights_out;
  p.positions = a.positions_out;
  p.n = a.n_tokens;
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.words = (uint32_t)a.n_tokens * (uint32_t)a.kv_heads * (D / 8);
  append_kernel<D><<<dim3((p.words + 255) / 256, 2 * a.batch), 256, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

template <int D>
int launch_evict(const ScoredArgs& a, cudaStream_t stream) {
  EvictParams p;
  memset(&p, 0, sizeof(p));
  for (int m = 0; m < 2; ++m) {
    const int64_t* c = m ? a.v_cache_strides : a.k_cache_strides;
    p.cache[m] = static_cast<uint4*>(m ? a.v_cache : a.k_cache);
    p.c_sb[m] = c[0] / 8;
    p.c_sn[m] = c[1] / 8;
    p.c_sh[m] = c[2] / 8;
  }
  p.w_in = a.weights_in;
  p.pos_in = a.positions_in;
  p.len_in = a.lengths_in;
  p.w_out = a.weights_out;
  p.pos_out = a.positions_out;
  const bool over = a.lengths_out == a.lengths_in;       // other heads' CTAs may still read them
  p.len_out = over ? nullptr : a.lengths_out;
  p.kv_heads = a.kv_heads;
  p.capacity = a.capacity;
  p.keep = a.keep;
  p.sinks = a.sinks;
  p.recent = a.recent;
  const bool small = a.capacity <= kSmall;
  p.cached = a.capacity <= kCachedKeys;
  // rows that move at most
  const int most = a.keep < a.capacity - a.keep ? a.keep : a.capacity - a.keep;
  const int smem = evict_smem(a.capacity, small, p.cached, most);
  const auto kern = small ? evict_kernel<D, true> : evict_kernel<D, false>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return SA_ERR_CUDA;
  // ranks of a cluster: each with 64 rows to move at least, if every evicted row were replaced, and not more than
  // two CTAs an SM in all, since each makes the whole selection (32 caches of up to 8192 slots, 4 key heads: 63 us with one rank,
  // 54 with two, 61 with four)
  const int64_t lists = (int64_t)a.batch * a.kv_heads;
  const int sm_count = current_sm_count();
  int ranks = 1;
  while (ranks < 8 && 64 * 2 * ranks <= most && lists * 2 * ranks <= 2 * sm_count) ranks *= 2;
  cudaLaunchConfig_t cfg;
  memset(&cfg, 0, sizeof(cfg));
  cfg.gridDim = dim3((unsigned)ranks, (unsigned)a.kv_heads, (unsigned)a.batch);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr;
  memset(&attr, 0, sizeof(attr));
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = (unsigned)ranks;
  attr.val.clusterDim.y = 1;
  attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kern, p) != cudaSuccess) return SA_ERR_CUDA;
  if (over) cut_lengths_kernel<<<(a.batch + 255) / 256, 256, 0, stream>>>(a.lengths_in, a.lengths_out, a.batch, a.capacity, a.keep);
  return cudaGetLastError() == cudaSuccess ? SA_OK : SA_ERR_CUDA;
}

}  // namespace

int launch_scored_append(const ScoredArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_append<32>(a, stream);
    case 64: return launch_append<64>(a, stream);
    case 128: return launch_append<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

int launch_scored_evict(const ScoredArgs& a, cudaStream_t stream) {
  switch (a.head_dim) {
    case 32: return launch_evict<32>(a, stream);
    case 64: return launch_evict<64>(a, stream);
    case 128: return launch_evict<128>(a, stream);
  }
  return SA_ERR_UNSUPPORTED;
}

unsigned int scored_read_and_clear_error(cudaStream_t stream) {
  unsigned int v = 0, zero = 0;
  cudaMemcpyFromSymbolAsync(&v, g_scored_err, sizeof(v), 0, cudaMemcpyDeviceToHost, stream);
  cudaMemcpyToSymbolAsync(g_scored_err, &zero, sizeof(zero), 0, cudaMemcpyHostToDevice, stream);
  cudaStreamSynchronize(stream);
  return v;
}

}  // namespace sa
