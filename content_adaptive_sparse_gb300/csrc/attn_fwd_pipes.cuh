// Forward at head dimensions 32 and 64: two pipelines per CTA, with 128-key score tiles and one
// full score row per softmax thread: the fixed per-step cost of the softmax (waits, arrivals, TMEM round trips, the
// online-max bookkeeping) covers 128 scores, and no two warps ever exchange a row maximum.
//
// TMEM of pipeline x (256 columns each, two pipelines per CTA): S [256x, +128), P
// [256x + 128, +64) (bf16 pairs), O [256x + 192, +d). P has columns of its own, so the QK of
// key tile j+1 may overwrite S as soon as the softmax has loaded S_j into registers; the
// exponentials of tile j then overlap with QK_{j+1}.
//
// Warp roles (512 threads, 16 warps; warp w runs on SM sub-partition w % 4):
//   warps 0-3   softmax of pipeline 0, warp w reads TMEM lane quarter w (query rows 32w ..)
//   warps 4-7   softmax of pipeline 1
//   warps 14, 15 planners of pipeline 0 / 1: claim items, build the key-block union, publish
//               the item's key tiles into a ring of two batches (up to 16 tiles per entry):
//               the next item's union is built under the current item, and a planner never
//               claims many items ahead of its pipeline
//   warps 8, 11 lane 0 loads Q, K and V of pipeline 0 / 1 by TMA as the batches arrive
//   warps 12, 13 idle (the fourth warpgroup's remainder)
//   warps 9, 10 lane 0 issues the tcgen05 MMAs of pipeline 0 / 1 in the order QK_j, PV_{j-1}:
//                 S = Q K_j^T   (N = keys of the tile, up to 128)
//                 O += P_j V_j  (A = P_j from TMEM, B = V_j MN-major; K = 16 keys per MMA)
//               the next tile's scores are requested as soon as S is free, before the previous
//               tile's probabilities are ready. The commit that frees a K stage also tells the
//               softmax that S is ready, and the one that frees a V stage tells it that P has
//               been read and O written.
#pragma once
#include "attn_fwd_common.cuh"

namespace sa {
namespace {

constexpr int kSoftmaxWarps = 4;      // per pipeline: one per TMEM lane quarter
// Register split of this kernel: softmax warpgroups 192, control warpgroups 64 (8 x 192 + 8 x 64
// = 16 x 128). Measured against 184 / 72: 8K top-16 0.1912-0.1932 -> 0.1911 ms, BigBird 16K
// 0.391-0.395 -> 0.390-0.391 ms; 200 / 56 (control code spills) no better.
constexpr int kPipeSoftmaxRegs = 192;
constexpr int kPipeCtrlRegs = 64;
static_assert(8 * kPipeSoftmaxRegs + 8 * kPipeCtrlRegs == 16 * kLaunchRegs, "register split");
// d = 64: items of at least this many key tiles store O by TMA (measured at 1, 2, 4 and 8:
// 1-4 equal within noise, 8 slower on BigBird 16K; 1 = every item with key tiles)
constexpr int kTmaStoreTiles = 1;
// Of every 16 exponential pairs, these many on the FMA pipe (exp2_fma2). Measured on the 8K
// top-16 workload at 0 / 1 / 2 / 3 / 4 pairs: 193-195 / 197-199 / 199-200 / 211 / 213-215 us:
// in this kernel the exponentials are not held up by the MUFU pipe but by issue slots and
// latency, so the polynomial's extra instructions only add time.
constexpr int kPolyPairs = 0;
constexpr int kMetaConsumers = 2 + kSoftmaxWarps;   // MMA thread, loader, softmax warps
__host__ __device__ constexpr uint32_t col_s(int x) { return 256u * x; }
__host__ __device__ constexpr uint32_t col_p(int x) { return 256u * x + 128u; }
__host__ __device__ constexpr uint32_t col_o(int x) { return 256u * x + 192u; }

struct PipeBars {
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[kMaxStages], k_empty[kMaxStages], v_full[kMaxStages], v_empty[kMaxStages];
  uint64_t m_full[kMetaRing], m_empty[kMetaRing];     // batch ring
  uint64_t s_free;            // the softmax has loaded S_j (phase j)
  uint64_t p_full;            // the softmax has stored P_j (phase j)
  uint64_t drain;
};

// ------------------------------------------------------------------ MMA issuer (warps 9, 10, lane 0)

// O += P_j V_j for the key tile held in ring stage `stage` (its V load was the kt-th),
// after P_j is stored. `o_init` says whether O already holds this item's sum.
template <int D>
__device__ __forceinline__ bool issue_pv(PipeBars& bars, uint32_t tP, uint32_t tO, uint64_t vdesc0, int j, int stage,
                                         int vkt, int nkeys, bool& o_init, volatile int* abort_flag) {
  using C = Cfg<D>;
  if (!wait_bar(&bars.p_full, (uint32_t)j & 1u, abort_flag)) return false;
  if (!wait_bar(&bars.v_full[stage], (uint32_t)(vkt / C::VS) & 1u, abort_flag)) return false;
  tc_fence_after();
  constexpr uint32_t idesc = make_idesc_bf16(128, D, 0, 1);
  const uint64_t b0 = vdesc0 + (uint64_t)((stage * C::KV_BYTES) >> 4);
  if (nkeys == kKeys) {
#pragma unroll
    for (int ks = 0; ks < kKeys / 16; ++ks)
      mma_bf16_ts(tO, tP + 8u * ks, b0 + (uint64_t)((16 * ks * C::ROWB) >> 4), idesc, (o_init || ks > 0) ? 1u : 0u);
  } else {
    for (int ks = 0; ks < nkeys / 16; ++ks)
      mma_bf16_ts(tO, tP + 8u * ks, b0 + (uint64_t)((16 * ks * C::ROWB) >> 4), idesc, (o_init || ks > 0) ? 1u : 0u);
  }
  o_init = true;
  // frees the V stage and tells the softmax that P_j is read and O is written
  mma_commit(&bars.v_empty[stage]);
  return true;
}

template <int D>
__device__ void mma_issuer(int x, PipeBars& bars, const Batch* ring, uint8_t* sQ, uint8_t* sK, uint8_t* sV,
                           uint32_t tmem, volatile int* abort_flag) {
  using C = Cfg<D>;
  const uint64_t qdesc = make_smem_desc(smem_u32(sQ), 16, C::ATOM, C::SWZ);
  const uint64_t kdesc0 = make_smem_desc(smem_u32(sK), 16, C::ATOM, C::SWZ);
  // V is the MN-major B operand of PV: N = d runs across the d-chunks (KV_CHUNK apart)
  const uint64_t vdesc0 = make_smem_desc(smem_u32(sV), C::KV_CHUNK, C::ATOM, C::SWZ);
  const uint32_t tS = tmem + col_s(x), tP = tmem + col_p(x), tO = tmem + col_o(x);
  int g = 0;                // key tiles of this pipeline whose QK is issued (K / V ring position)
  int item_local = -1;
  int qb = 0;
  uint64_t a0 = qdesc;
  bool ok = true;
  bool o_init = false;
  bool pend = false;        // PV of the previous key tile of this item not yet issued
  int p_nkeys = 0;
  for (int mt = 0;; ++mt) {
    int4 hdr;
    if (!(ok = wait_batch(bars, ring, mt, hdr, abort_flag))) break;
    const Batch& e = ring[mt % kMetaRing];
    if (hdr.x == kKindDone) {
      mbar_arrive(&bars.m_empty[mt % kMetaRing]);
      break;
    }
    if (hdr.w & kFirst) {
      ++item_local;
      qb = item_local % C::QB;
      if (!(ok = wait_bar(&bars.q_full[qb], (item_local / C::QB) & 1, abort_flag))) break;
      a0 = qdesc + (uint64_t)((qb * C::Q_BYTES) >> 4);
      o_init = false;
      pend = false;
    }
    const uint4 ncw = ld_shared_u4(&e.nch[0]);
    for (int i = 0; i < hdr.y; ++i) {
      const int nkeys = 32 * (int)((word_of(ncw, i >> 2) >> (8 * (i & 3))) & 0xffu);
      const int stage = g % C::KS;
      if (!(ok = wait_bar(&bars.k_full[stage], (uint32_t)(g / C::KS) & 1u, abort_flag))) break;
      // S is free once the softmax has loaded S_{g-1}
      if (g > 0 && !(ok = wait_bar(&bars.s_free, (uint32_t)(g - 1) & 1u, abort_flag))) break;
      tc_fence_after();
      const uint32_t idesc = make_idesc_bf16(128, (uint32_t)nkeys, 0, 0);
      const uint64_t b0 = kdesc0 + (uint64_t)((stage * C::KV_BYTES) >> 4);
#pragma unroll
      for (int ks = 0; ks < D / 16; ++ks)
        mma_bf16_ss(tS, a0 + kmajor_step<D>(ks, C::Q_CHUNK), b0 + kmajor_step<D>(ks, C::KV_CHUNK), idesc,
                    ks > 0 ? 1u : 0u);
      // frees the K stage and tells the softmax that S_g is ready
      mma_commit(&bars.k_empty[stage]);
      if (pend && !(ok = issue_pv<D>(bars, tP, tO, vdesc0, g - 1, (g - 1) % C::VS, g - 1, p_nkeys, o_init,
                                     abort_flag)))
        break;
      pend = true;
      p_nkeys = nkeys;
      ++g;
    }
    if (!ok) break;
    mbar_arrive(&bars.m_empty[mt % kMetaRing]);
    if (hdr.w & kLast) {
      mma_commit(&bars.q_empty[qb]);   // all QKs of this item issued; arrives when they are done
      // the item's last PV: its completion releases the softmax epilogue
      if (pend && !(ok = issue_pv<D>(bars, tP, tO, vdesc0, g - 1, (g - 1) % C::VS, g - 1, p_nkeys, o_init,
                                     abort_flag)))
        break;
      pend = false;
    }
  }
  // Make sure no MMA of this thread is still writing TMEM when the CTA frees it.
  mma_commit(&bars.drain);
  drain_bar(&bars.drain, 0);
}

// ------------------------------------------------------------------ softmax + epilogue (warps 0-7)

// Rare path of the online max: O *= alpha for this thread's row (O quiescent).
template <int D>
__device__ __forceinline__ void rescale_o(uint32_t tO, float alpha) {
  const uint64_t al2 = f2_pack(alpha, alpha);
#pragma unroll 1
  for (int ch = 0; ch < D / 32; ++ch) {
    uint32_t ov[32];
    tmem_ld_x32(tO + ch * 32, ov);
    tmem_ld_wait<32>(ov);
#pragma unroll
    for (int j = 0; j < 32; j += 2) {
      float lo, hi;
      f2_unpack(f2_mul(f2_pack(__uint_as_float(ov[j]), __uint_as_float(ov[j + 1])), al2), lo, hi);
      ov[j] = __float_as_uint(lo);
      ov[j + 1] = __float_as_uint(hi);
    }
    tmem_st_x32(tO + ch * 32, ov);
  }
  tmem_st_wait();
}

// Softmax and epilogue of pipeline x; this warp handles query rows 32q .. 32q+31 of every
// item (q = its TMEM lane quarter) and all 128 keys of every key tile. At d = 64 (with an
// output tensor map, to) an item's O / l rows are staged, 128B-swizzled, in the item's own Q
// buffer (its QKs are complete) and written by one TMA store per warp; the Q buffer is
// released to the loader (q_empty) once that store has read it.
template <int D, bool WIN>
__device__ void softmax_epilogue(const Params& p, int x, PipeBars& bars, const Batch* ring, uint32_t tmem,
                                 uint8_t* sQ, const CUtensorMap* to, volatile int* abort_flag) {
  using C = Cfg<D>;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quarter = warp & 3;
  const int row = quarter * 32 + lane;               // query row within the tile
  const uint32_t lane_base = (uint32_t)(quarter * 32) << 16;
  const float kNegInf = __int_as_float(0xff800000);
  const float c = p.scale_log2;
  const uint64_t c2 = f2_pack(c, c);
  const uint32_t tS = tmem + col_s(x) + lane_base;
  const uint32_t tP = tmem + col_p(x) + lane_base;
  const uint32_t tO = tmem + col_o(x) + lane_base;

  int g = 0;                // key tiles processed by this pipeline
  int item_local = -1;      // items of this pipeline (Q buffer item_local % QB)
  bool ok = true;
  Item it;
  it.s = it.h = it.tile = 0;
  int qtok = 0;
  float m_use = kNegInf;    // running reference max, log2 units
  float l = 0.f;            // row sum
  int n_item = 0;           // key tiles of the current item
  int slot = -1;            // partial-result slot of a split item's part (-1: write O and LSE)
  for (int mt = 0;; ++mt) {
    int4 hdr;
    ok = __all_sync(0xffffffffu, wait_batch(bars, ring, mt, hdr, abort_flag));
    if (!ok) break;
    const Batch& e = ring[mt % kMetaRing];
    if (hdr.x == kKindDone) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.m_empty[mt % kMetaRing]);
      break;
    }
    if (hdr.w & kFirst) {
      ++item_local;
      it = decode_item(p, hdr.z);
      qtok = it.tile * kTile + row;
      m_use = kNegInf;
      l = 0.f;
      n_item = 0;
      slot = e.slot;
      // Items of at least kTmaStoreTiles key tiles (d = 64, whole items) stage their output in
      // their Q buffer; the others (items without key tiles, split parts, other d) give the
      // buffer up now, and its release then waits only for the item's Q and QKs.
      // An item's first batch holds min(16, its key tiles) tiles, so this test and the one at
      // the item's end, on its tile count, agree.
      if (!(D == 64 && p.o_tma && slot < 0 && hdr.y >= kTmaStoreTiles)) {
        __syncwarp();
        if (lane == 0) mbar_arrive(&bars.q_empty[item_local % C::QB]);
      }
    }
    // this quarter's visibility bytes and the chunk counts of the batch's tiles
    const uint4 vqw = ld_shared_u4(&e.vq[quarter][0]);
    const uint4 ncw = ld_shared_u4(&e.nch[0]);
    for (int i = 0; i < hdr.y; ++i) {
      const int sh = 8 * (i & 3);
      const int vb = (int)((word_of(vqw, i >> 2) >> sh) & 0xffu);
      const int nch = (int)((word_of(ncw, i >> 2) >> sh) & 0xffu);
      const int vis = vb & 15, dch = WIN ? -1 : (vb >> 4) - 1;

      // QK_g done: its commit is the (g / KS)-th completion of K stage g % KS
      ok = __all_sync(0xffffffffu, wait_bar(&bars.k_empty[g % C::KS], (uint32_t)(g / C::KS) & 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
      uint32_t v[128];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) tmem_ld_x32(tS + 32 * ch, v + 32 * ch);
      tmem_ld_wait<128>(v);
      // S may now be overwritten by the next QK
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.s_free);

      if (dch >= 0) {
        // the diagonal chunk starts at this warp's first query: row r sees columns 0 .. r
        const uint32_t kp = (2u << lane) - 1u;       // lane 31: all 32 columns
        switch (dch) {
          case 0: mask_chunk(v, kp); break;
          case 1: mask_chunk(v + 32, kp); break;
          case 2: mask_chunk(v + 64, kp); break;
          default: mask_chunk(v + 96, kp); break;
        }
      }
      if (WIN && (vb >> 4) != 0) {
        // chunks that some of this warp's rows see in part
        const int4 tm = ld_shared_v4(&e.tile[i]);
#pragma unroll
        for (int ch = 0; ch < 4; ++ch)
          if ((vb >> (4 + ch)) & 1)
            mask_chunk(v + 32 * ch, window_bits(qtok, (ch == 0 ? tm.x : ch == 1 ? tm.y : ch == 2 ? tm.z : tm.w) >> 4,
                                                p.window, p.sinks));
      }
      float cm = kNegInf;
#pragma unroll
      for (int ch = 0; ch < 4; ++ch)
        if ((vis >> ch) & 1) cm = chunk_max(v + 32 * ch, cm);
      const float mx = cm * c;                       // -inf stays -inf
      const bool need = mx > m_use + 8.0f;
      float alpha = 1.f;
      bool o_scale = false;
      if (__any_sync(0xffffffffu, need)) {
        // the running max grows by more than 2^8: rescale l now and O before this tile's PV
        alpha = need ? ex2_approx(m_use - mx) : 1.f;   // 0 when m_use = -inf
        o_scale = need && m_use != kNegInf && n_item > 0;
        l *= alpha;
        if (need) m_use = mx;
      }
      // a row of the sink-window graph may have seen no key yet: its scores are all -inf
      const float m_ref = WIN && m_use == kNegInf ? 0.f : m_use;
      const uint64_t negm2 = f2_pack(-m_ref, -m_ref);
      uint64_t rs[2] = {0ull, 0ull};
      // All exponentials of the tile first (P_j packed in registers; the scores' registers
      // are reused as they die): only the stores of P wait for PV_{j-1}, so the tensor
      // core's PV and the next QK run under this tile's exponentials instead of in series
      // with them.
      uint32_t pk[64];
#pragma unroll
      for (int ch = 0; ch < 4; ++ch) {
        if ((vis >> ch) & 1) {
          chunk_exp<kPolyPairs>(v + 32 * ch, c2, negm2, pk + 16 * ch, rs);
        } else {
#pragma unroll
          for (int j = 0; j < 16; ++j) pk[16 * ch + j] = 0u;
        }
      }
      // PV_{g-1} has read P and finished writing O
      if (g > 0) {
        ok = __all_sync(0xffffffffu,
                        wait_bar(&bars.v_empty[(g - 1) % C::VS], (uint32_t)((g - 1) / C::VS) & 1u, abort_flag));
        if (!ok) break;
        tc_fence_after();
      }
      if (__any_sync(0xffffffffu, o_scale)) rescale_o<D>(tO, alpha);
#pragma unroll
      for (int ch = 0; ch < 4; ++ch)
        if (ch < nch) tmem_st_x16(tP + 16 * ch, pk + 16 * ch);
      {
        const uint64_t rs2 = f2_add(rs[0], rs[1]);
        float rs_lo, rs_hi;
        f2_unpack(rs2, rs_lo, rs_hi);
        l += rs_lo + rs_hi;
      }
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.p_full);
      ++g;
      ++n_item;
    }
    if (!ok) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&bars.m_empty[mt % kMetaRing]);
    if (!(hdr.w & kLast)) continue;

    // epilogue: O / l and LSE of this query tile's rows
    if (n_item > 0) {
      ok = __all_sync(0xffffffffu, wait_bar(&bars.v_empty[(g - 1) % C::VS], (uint32_t)((g - 1) / C::VS) & 1u, abort_flag));
      if (!ok) break;
      tc_fence_after();
    }
    const float inv = l > 0.f ? 1.f / l : 0.f;
    const float lse = l > 0.f ? (m_use + __log2f(l)) * 0.69314718055994531f : kNegInf;
    if (slot >= 0) {
      // a part of a split item: O / l of its key range (fp32) and its LSE, merged later
      float* po = p.partial + (size_t)slot * (kTile * (D + 1)) + (size_t)row * D;
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t ov[32];
        if (n_item > 0) {
          tmem_ld_x32(tO + 32 * ch, ov);
          tmem_ld_wait<32>(ov);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        float4* dst = reinterpret_cast<float4*>(po + ch * 32);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          dst[j] = make_float4(__uint_as_float(ov[4 * j]) * inv, __uint_as_float(ov[4 * j + 1]) * inv,
                               __uint_as_float(ov[4 * j + 2]) * inv, __uint_as_float(ov[4 * j + 3]) * inv);
      }
      p.partial[(size_t)slot * (kTile * (D + 1)) + (size_t)kTile * D + row] = lse;
    } else if (D == 64 && p.o_tma && n_item >= kTmaStoreTiles) {
      // Staged in the item's Q buffer (its QKs are complete: the last PV has been waited for):
      // rows of this warp, 128 bytes each, 128B-swizzled (16-byte chunk c of row r at
      // r * 128 + (c ^ (r & 7)) * 16) as the output map's box expects; rows past the sequence
      // end are dropped by the TMA store
      const int qb = item_local % C::QB;
      uint8_t* stg = sQ + qb * C::Q_BYTES + quarter * 32 * 128;
      const uint32_t srow = smem_u32(stg) + (uint32_t)lane * 128u;
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t ov[32];
        if (n_item > 0) {
          tmem_ld_x32(tO + 32 * ch, ov);
          tmem_ld_wait<32>(ov);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        uint32_t pk[16];
#pragma unroll
        for (int j = 0; j < 32; j += 2)
          pk[j >> 1] = pack_bf16x2(__uint_as_float(ov[j]) * inv, __uint_as_float(ov[j + 1]) * inv);
#pragma unroll
        for (int j = 0; j < 4; ++j)
          st_shared_v4(srow + (uint32_t)(((4 * ch + j) ^ (lane & 7)) << 4), pk[4 * j], pk[4 * j + 1], pk[4 * j + 2],
                       pk[4 * j + 3]);
      }
      fence_proxy_async_smem();                      // the staged rows are visible to the TMA store
      __syncwarp();
      if (lane == 0) {
        tma_store_4d(to, stg, 0, it.h, it.tile * kTile + quarter * 32, it.s);
        bulk_commit_group();
      }
      if (qtok < p.n_tokens) p.lse[((int64_t)it.s * p.heads + it.h) * p.n_tokens + qtok] = lse;
      // the buffer goes back to the loader once the store has read it
      if (lane == 0) bulk_wait_group_read<0>();
      __syncwarp();
      if (lane == 0) mbar_arrive(&bars.q_empty[qb]);
    } else {
      const bool store = qtok < p.n_tokens;
      __nv_bfloat16* orow = p.o + (int64_t)it.s * p.o_sb + (int64_t)qtok * p.o_sn + (int64_t)it.h * p.o_sh;
#pragma unroll
      for (int ch = 0; ch < D / 32; ++ch) {
        uint32_t ov[32];
        if (n_item > 0) {
          tmem_ld_x32(tO + 32 * ch, ov);
          tmem_ld_wait<32>(ov);
        } else {
#pragma unroll
          for (int j = 0; j < 32; ++j) ov[j] = 0u;
        }
        if (store) {
          uint32_t pk[16];
#pragma unroll
          for (int j = 0; j < 32; j += 2)
            pk[j >> 1] = pack_bf16x2(__uint_as_float(ov[j]) * inv, __uint_as_float(ov[j + 1]) * inv);
          uint4* dst = reinterpret_cast<uint4*>(orow + ch * 32);
#pragma unroll
          for (int j = 0; j < 4; ++j) dst[j] = make_uint4(pk[4 * j], pk[4 * j + 1], pk[4 * j + 2], pk[4 * j + 3]);
        }
      }
      if (store) p.lse[((int64_t)it.s * p.heads + it.h) * p.n_tokens + qtok] = lse;
    }
    // The next item's first P store follows these O loads in program order, and the MMA
    // thread issues that item's first PV only after the P store: O is not overwritten early.
  }
  // every TMA store of this warp has completed before the CTA may exit
  if (lane == 0) bulk_wait_group<0>();
  __syncwarp();
}

// ------------------------------------------------------------------ kernel

template <int D, bool WIN>
__global__ void __launch_bounds__(kThreads, 1)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                    const __grid_constant__ CUtensorMap tv, const __grid_constant__ CUtensorMap to,
                    const __grid_constant__ Params p) {
  using C = Cfg<D>;
  static_assert(!C::WIDE && 192 + D <= 256, "two-pipeline kernel: head dimension 32 or 64");
  extern __shared__ uint8_t smem_raw[];
  uint8_t* sbase = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  __shared__ PipeBars bars[2];
  __shared__ Batch ring[2][kMetaRing];
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_flag;

  const int warp = threadIdx.x >> 5;
  if (threadIdx.x == 0) {
    for (int x = 0; x < 2; ++x) {
      PipeBars& b = bars[x];
      for (int i = 0; i < 2; ++i) {
        mbar_init(&b.q_full[i], 1);
        // released by the MMA thread (the item's QKs are done) and the softmax warps (at the
        // item's start, or once the item's output store has read the buffer)
        mbar_init(&b.q_empty[i], 1 + kSoftmaxWarps);
      }
      for (int i = 0; i < kMaxStages; ++i) {
        mbar_init(&b.k_full[i], 1);
        mbar_init(&b.k_empty[i], 1);
        mbar_init(&b.v_full[i], 1);
        mbar_init(&b.v_empty[i], 1);
      }
      for (int i = 0; i < kMetaRing; ++i) {
        mbar_init(&b.m_full[i], 1);
        mbar_init(&b.m_empty[i], kMetaConsumers);
      }
      mbar_init(&b.s_free, kSoftmaxWarps);
      mbar_init(&b.p_full, kSoftmaxWarps);
      mbar_init(&b.drain, 1);
    }
    abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tq);
    tma_prefetch_desc(&tk);
    tma_prefetch_desc(&tv);
  }
  if (warp == 9) {
    tmem_alloc(&tmem_slot, kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_slot;

  // Register split: warpgroups 0-1 (softmax) grow, warpgroups 2-3 (control) shrink, at the
  // top of their branches (the compiler budgets the code that follows by it); the sum equals
  // the launch allocation (checked on the host), so the growth always completes.
  static_assert(kPipeSoftmaxRegs == 192 && kPipeCtrlRegs == 64, "register split literals");

  // pipeline 0: softmax warps 0-3, loader 8, MMA 9, planner 14;
  // pipeline 1: softmax warps 4-7, MMA 10, loader 11, planner 15; warps 12, 13 idle
  // (sub-partition w % 4: the planners share 2 and 3 with an MMA thread and a loader, not 0
  // and 1 with both; BigBird 16K 0.395-0.400 -> 0.389-0.392 ms, the rest within noise)
  const int x = warp < 8 ? (warp >> 2) : ((warp == 8 || warp == 9 || warp == 14) ? 0 : 1);
  uint8_t* sQ = sbase + x * C::PIPE_BYTES;
  uint8_t* sK = sQ + C::QB * C::Q_BYTES;
  uint8_t* sV = sK + C::KS * C::KV_BYTES;
  UnionSmem& un = *reinterpret_cast<UnionSmem*>(sV + C::VS * C::KV_BYTES);

  if (warp < 8) {
    // warpgroups 0 and 1: one setmaxnreg instruction for both
    asm volatile("setmaxnreg.inc.sync.aligned.u32 192;" ::: "memory");
    softmax_epilogue<D, WIN>(p, x, bars[x], ring[x], tmem, sQ, &to, &abort_flag);
  } else {
    // warpgroups 2 and 3: one setmaxnreg instruction for both, then the roles
    asm volatile("setmaxnreg.dec.sync.aligned.u32 64;" ::: "memory");
    if (warp == 8 || warp == 11) {
      if ((threadIdx.x & 31) == 0) loader<D>(p, &tq, &tk, &tv, bars[x], ring[x], sQ, sK, sV, &abort_flag);
      __syncwarp();
    } else if (warp == 9 || warp == 10) {
      if ((threadIdx.x & 31) == 0) mma_issuer<D>(x, bars[x], ring[x], sQ, sK, sV, tmem, &abort_flag);
      __syncwarp();
    } else if (warp == 14 || warp == 15) {
      planner<D, WIN>(p, bars[x], ring[x], un, 2 * blockIdx.x + x, 2 * gridDim.x, &abort_flag);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

}  // namespace
}  // namespace sa
