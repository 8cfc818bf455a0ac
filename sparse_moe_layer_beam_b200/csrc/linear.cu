// linear.cu - products of expert-sorted rows with each expert's weights, on
// 5th-generation tensor cores, and their gradients. Rows offsets[e] ..
// offsets[e+1] - 1 belong to expert e (no offsets: one expert has all rows).
//
//   forward   Z = X W_e^T + b_e,  Y = act(Z) + residual       (contraction: in)
//   backward  dZ = dY act'(Z)                                 (elementwise)
//             dX = dZ W_e                                     (contraction: out)
//             dW_e = sum over e's rows of dZ^T X              (contraction: rows)
//             db_e = sum over e's rows of dZ
//
// One kernel does the three products (FWD, DGRAD, WGRAD). A tile is 128 rows
// of D (X rows, or rows of dW_e) times BN columns. None of the operands is
// transposed in memory: W_e in DGRAD and both operands in WGRAD are read by
// TMA as they lie and declared MN-major to the MMA (their contraction runs
// over shared-memory rows instead of columns).
//
//  - Rows of X or dZ beyond the segment of e inside a tile only fill lanes of
//    the accumulator that are not stored. In WGRAD they would be summed, so
//    the last step of a segment zeroes them in shared memory (both operands:
//    0 times a NaN of another expert's row is a NaN) before its MMAs.
//  - Contraction tails (in or out not a multiple of 64) are TMA's zero fill;
//    W is a 3-D map, so that the fill starts at the end of each expert.
//  - Enough tiles for the SMs: persistent CTAs, TMA producer, MMA issuer and
//    four epilogue warps, accumulators double-buffered in TMEM. Fewer: a
//    cluster of up to 8 CTAs splits the contraction of a tile and joins its
//    partial sums through distributed shared memory, in CTA order. Many rows
//    per expert: CTA pairs (linear_pair.cu). Up to four rows: no tiles at all,
//    the weights stream through the CUDA cores (linear_few_kernel). choose()
//    picks the form by estimated time.
//  - Each role is a whole warp whose loops are uniform, one elected lane issuing
//    (see elect_one).
// Every wait is bounded (see sm100.cuh).
#include <string.h>

#include <type_traits>

#include "linear.cuh"
#include "ops.h"

namespace beam {
namespace {

using namespace lin;

constexpr int kThreads = 192;

template <int BN, bool SPLIT>
struct LinCfg {
  static constexpr int kABytes = kM * kK * 2;
  static constexpr int kBBytes = BN * kK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  // persistent: all of shared memory; split: two CTAs per SM, and as many
  // stages (at most 10) as its rows' operand leaves room for
  static constexpr int kRing = SPLIT ? 96 * 1024 : 192 * 1024 / kStageBytes * kStageBytes;
  static constexpr int kStages = SPLIT ? 10 : kRing / kStageBytes;
  static constexpr int kAccStages = SPLIT ? 1 : 2;
  static constexpr int kTmemCols = kAccStages * BN;  // 64, 256 or 512
  static constexpr int kBarBytes = 256;
  static constexpr int kTabBytes = 4 * (3 * kMaxE + 12 + 64);  // and 64 biases (split)
  static constexpr int kSmemBytes = 1024 + kRing + kBarBytes + kTabBytes;
  static_assert(kSmemBytes <= 232448, "dynamic shared memory above the sm_100 limit");
  static_assert(!SPLIT || kRing >= (kM + 1) * BN * 4, "partial tile in the ring");
};

struct Tile {
  int e;
  int row0;   // first row of D: a row of X / dX, or of dW_e
  int rows;   // rows of the tile that exist
  int n0;     // first column
  int k0;     // WGRAD: first row of the segment
  int kcnt;   // WGRAD: rows of the segment
  int nk;     // contraction steps
  bool once;  // the weight tile is read by this tile alone
};

// FWD and DGRAD: an expert's tiles go in groups of 16 row blocks, column tile
// by column tile inside a group, row blocks fastest: the CTAs at work at one
// time share a few weight tiles and at most 16 row blocks through L2.
// WGRAD: row tiles of dW_e fastest in groups of 16 likewise.
template <int MODE, int BN>
__device__ __forceinline__ Tile decode(int t, const LinParams& p, const Segments& s, int bn_out) {
  Tile d;
  int e, m_blks, local;
  if (MODE == kWgrad) {
    const int per = p.m_blk * p.n_blk;
    e = t / per;
    local = t - e * per;
    m_blks = p.m_blk;
  } else {
    e = find_expert(s.rb, p.E, t / p.n_blk);
    local = t - s.rb[e] * p.n_blk;
    m_blks = s.rb[e + 1] - s.rb[e];
  }
  const int g = local / (kRowGroup * p.n_blk);
  const int in_g = min(kRowGroup, m_blks - g * kRowGroup);
  const int rem = local - g * kRowGroup * p.n_blk;
  const int nb = rem / in_g;
  const int mb = g * kRowGroup + rem - nb * in_g;
  d.e = e;
  d.n0 = nb * bn_out;
  d.once = m_blks == 1;
  if (MODE == kWgrad) {
    d.k0 = s.lo[e];
    d.kcnt = s.cnt[e];
    d.nk = (d.kcnt + kK - 1) / kK;
    d.row0 = mb * kM;
    d.rows = min(kM, p.n_w - d.row0);
  } else {
    d.k0 = 0;
    d.kcnt = 0;
    d.nk = p.nk;
    d.row0 = s.lo[e] + mb * kM;
    d.rows = min(kM, s.cnt[e] - mb * kM);
  }
  return d;
}

__device__ __forceinline__ float ld_dsmem_f32(uint32_t addr) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void* p) {
  asm volatile("prefetch.global.L2 [%0];" ::"l"(p));
}

// Four columns n .. n + 3 of one row of D: a (and, for swiglu, the up values
// u). n_out and n_in are multiples of 8, so four columns exist together. bias:
// that of column n, and of its up value `up` floats further.
template <int MODE>
__device__ __forceinline__ void finish4(const LinParams& p, const Tile& t, int r, int n, float* a,
                                        float* u, const float* bias, int up) {
  if (n >= p.cols) return;
  if (MODE == kWgrad) {
    store4(p.out, ((int64_t)t.e * p.n_w + t.row0 + r) * p.n_in + n, a, false, p.fp16);
    return;
  }
  const int64_t row = t.row0 + r;
  if (MODE == kDgrad) {
    store4(p.out, row * p.n_in + n, a, false, p.fp16);
    return;
  }
  const bool glu = p.act == BEAM_MOE_ACT_SWIGLU;
  if (p.bias) {
    const float4 f = *reinterpret_cast<const float4*>(bias);
    a[0] += f.x; a[1] += f.y; a[2] += f.z; a[3] += f.w;
    if (glu) {
      const float4 g = *reinterpret_cast<const float4*>(bias + up);
      u[0] += g.x; u[1] += g.y; u[2] += g.z; u[3] += g.w;
    }
  }
  if (p.z) {
    store4(p.z, row * p.n_w + n, a, false, p.fp16);
    if (glu) store4(p.z, row * p.n_w + p.n_out + n, u, false, p.fp16);
  }
  if (glu) {
    swiglu<4, true>(a, u);
  } else {
    activate<4, true>(p.act, a);
  }
  if (p.residual) {
    float q[4];
    load4(p.residual, row * p.n_out + n, q, p.out32, p.fp16);
#pragma unroll
    for (int j = 0; j < 4; ++j) a[j] += q[j];
  }
  store4(p.out, row * p.n_out + n, a, p.out32, p.fp16);
}

// Sixteen columns from n on of one row, as above; eight of them exist together.
template <int MODE>
__device__ __forceinline__ void finish16(const LinParams& p, const Tile& t, int r, int n, float* a,
                                         const float* u) {
  const int halves = p.cols - n >= 16 ? 2 : 1;
  if (MODE != kFwd) {
    uint16_t* out = static_cast<uint16_t*>(p.out);
    const int64_t at =
        (MODE == kWgrad ? (int64_t)t.e * p.n_w + t.row0 + r : (int64_t)t.row0 + r) * p.n_in + n;
    store8(out, at, a, p.fp16);
    if (halves == 2) store8(out, at + 8, a + 8, p.fp16);
    return;
  }
  const bool glu = p.act == BEAM_MOE_ACT_SWIGLU;
  const int64_t row = t.row0 + r;
  float v[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) v[j] = glu ? u[j] : 0.0f;
  if (p.bias) {
    const float* b = p.bias + (int64_t)t.e * p.n_w + n;
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      if (j >= 8 * halves) break;
      const float4 f = __ldg(reinterpret_cast<const float4*>(b + j));
      a[j] += f.x; a[j + 1] += f.y; a[j + 2] += f.z; a[j + 3] += f.w;
      if (glu) {
        const float4 g = __ldg(reinterpret_cast<const float4*>(b + p.n_out + j));
        v[j] += g.x; v[j + 1] += g.y; v[j + 2] += g.z; v[j + 3] += g.w;
      }
    }
  }
  if (p.z) {
    uint16_t* z = static_cast<uint16_t*>(p.z);
    for (int h = 0; h < halves; ++h) {
      store8(z, row * p.n_w + n + 8 * h, a + 8 * h, p.fp16);
      if (glu) store8(z, row * p.n_w + p.n_out + n + 8 * h, v + 8 * h, p.fp16);
    }
  }
  if (glu) {
    if (p.out32) swiglu<16, true>(a, v);
    else swiglu<16, false>(a, v);
  } else if (p.out32) {
    activate<16, true>(p.act, a);
  } else {
    activate<16, false>(p.act, a);
  }
  const int64_t at = row * p.n_out + n;
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < 16; j += 4) {
      if (j >= 8 * halves) break;
      float q[4];
      load4(p.residual, at + j, q, p.out32, p.fp16);
#pragma unroll
      for (int i = 0; i < 4; ++i) a[j + i] += q[i];
    }
  }
#pragma unroll
  for (int j = 0; j < 16; j += 8) {
    if (j >= 8 * halves) break;
    if (p.out32) {
      store4(p.out, at + j, a + j, true, false);
      store4(p.out, at + j + 4, a + j + 4, true, false);
    } else {
      store8(static_cast<uint16_t*>(p.out), at + j, a + j, p.fp16);
    }
  }
}

// ------------------------------------------------------------------- kernel
// bid: this CTA among those of the product. Split: consecutive groups of
// p.parts CTAs share a tile each (a cluster holds one group or several). LONG
// (WGRAD): segments may be longer than a drain of the accumulators; the split form
// without it is 0.4 us faster (300 x 640 x 640: 15.4 us).
template <int MODE, int BN, bool SPLIT, bool LONG>
__device__ __forceinline__ void linear_body(const CUtensorMap& tm_a, const CUtensorMap& tm_b,
                                            const LinParams& p, int bid) {
  using C = LinCfg<BN, SPLIT>;
  // Split: with few rows the stages of A lie closer together than the 128
  // rows an MMA reads of them; what follows fills lanes that are not stored.
  const int STAGES = SPLIT ? p.stages : C::kStages;
  const int a_stage = SPLIT ? p.a_stage : C::kABytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* ring_b = smem + STAGES * a_stage;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::kRing);
  uint64_t* empty = full + C::kStages;
  uint64_t* tfull = empty + C::kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  int* tab = reinterpret_cast<int*>(smem + C::kRing + C::kBarBytes);
  const Segments seg = {tab, tab + kMaxE, tab + 2 * kMaxE};
  int* scratch = tab + 3 * kMaxE + 4;  // a word per warp, then 64 biases

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t parts = SPLIT ? p.parts : 1;
  const uint32_t rank = SPLIT ? cluster_ctarank() & (parts - 1) : 0;  // in its group
  const uint32_t group0 = SPLIT ? cluster_ctarank() - rank : 0;       // the group's first CTA
  if (threadIdx.x == 0) {
    for (int s = 0; s < STAGES; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 128);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
  }
  if (warp == 0) {
    tmem_alloc(tmem_holder, C::kTmemCols);
    tmem_relinquish();
  }
  if (p.offsets) {
    build_segments<kThreads, kM>(p, seg, scratch);
  } else if (threadIdx.x == 0) {
    seg.lo[0] = seg.rb[0] = 0;
    seg.cnt[0] = p.rows;
    seg.rb[1] = (p.rows + kM - 1) / kM;
  }
  if (p.clear_status && bid == 0) clear_status_area(p);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)*tmem_holder);
  const bool glu = MODE == kFwd && p.act == BEAM_MOE_ACT_SWIGLU;
  const int bn_out = glu ? BN / 2 : BN;
  const int total = MODE == kWgrad ? p.E * p.m_blk * p.n_blk : seg.rb[p.E] * p.n_blk;
  const int first = SPLIT ? bid / (int)parts : bid;
  const int step = SPLIT ? total : gridDim.x;  // split: one tile per cluster
  // this CTA's contraction steps of a tile
  auto k_range = [&](const Tile& t, int& ka, int& kb) {
    ka = SPLIT ? uniform((int)((int64_t)t.nk * rank / parts)) : 0;
    kb = SPLIT ? uniform((int)((int64_t)t.nk * (rank + 1) / parts)) : uniform(t.nk);
  };
  // A wait of the whole warp.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity, uint32_t flag) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, flag));
  };

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    const uint64_t pol_stream = policy_evict_first();
    const uint64_t pol_keep = policy_evict_normal();
    const bool one = elect_one();
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    for (int ti = first; ti < total && ok; ti += step) {
      const Tile t = decode<MODE, BN>(ti, p, seg, bn_out);
      int ka, kb;
      k_range(t, ka, kb);
      const int boxes_a = MODE == kWgrad ? 2 : (t.rows + p.box_a - 1) / p.box_a;
      const uint32_t box_bytes = p.box_a * kK * 2;
      const uint32_t tx = (MODE == kWgrad ? C::kABytes : boxes_a * box_bytes) + C::kBBytes;
      const uint64_t pol_w = t.once ? pol_stream : pol_keep;
      for (int k = ka; k < kb; ++k) {
        if (!warp_wait(&empty[stage], phase ^ 1u, kFlagProducer)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * a_stage;
        uint8_t* sb = ring_b + stage * C::kBBytes;
        uint64_t* bar = &full[stage];
        const int kx = k * kK;
        if (one) {
          mbar_arrive_expect_tx(bar, tx);
          if (MODE == kWgrad) {
#pragma unroll
            for (int b = 0; b < 2; ++b)
              tma_load_2d(sa + b * kBox, &tm_a, bar, t.row0 + b * 64, t.k0 + kx, pol_keep);
#pragma unroll
            for (int b = 0; b < BN / 64; ++b)
              tma_load_2d(sb + b * kBox, &tm_b, bar, t.n0 + b * 64, t.k0 + kx, pol_keep);
          } else {
            if (MODE == kFwd) {
              tma_load_3d(sb, &tm_b, bar, kx, t.n0, t.e, pol_w);
              if (glu)
                tma_load_3d(sb + C::kBBytes / 2, &tm_b, bar, kx, p.n_out + t.n0, t.e, pol_w);
            } else {
#pragma unroll
              for (int b = 0; b < BN / 64; ++b)
                tma_load_3d(sb + b * kBox, &tm_b, bar, t.n0 + b * 64, kx, t.e, pol_w);
            }
            for (int b = 0; b < boxes_a; ++b)
              tma_load_2d(sa + b * box_bytes, &tm_a, bar, kx, t.row0 + b * p.box_a, pol_keep);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == STAGES) {
          stage = 0;
          phase ^= 1u;
        }
      }
    }
    // Let every copy this warp issued land before the CTA can exit.
    if (one)
      for (int64_t i = issued > STAGES ? issued - STAGES : 0; i < issued; ++i)
        mbar_wait(&full[i % STAGES], (uint32_t)((i / STAGES) & 1), nullptr, nullptr, 0u,
                  100000000ull);
    __syncwarp();
  } else if (warp == 1) {
    // ----------------------------------------------------------- MMA issuer
    // (in WGRAD the warp zeroes the rows behind a segment, too)
    const bool one = elect_one();
    const uint32_t sa = smem_addr(smem), sb = smem_addr(ring_b);
    const uint64_t desc_a = MODE == kWgrad ? smem_desc_mn_sw128(sa) : smem_desc_k_sw128(sa);
    const uint64_t desc_b = MODE == kFwd ? smem_desc_k_sw128(sb) : smem_desc_mn_sw128(sb);
    constexpr uint32_t kStepA = MODE == kWgrad ? 2048 >> 4 : 32 >> 4;
    constexpr uint32_t kStepB = MODE == kFwd ? 32 >> 4 : 2048 >> 4;
    int stage = 0;
    uint32_t phase = 0;
    int acc = 0;
    uint32_t acc_phase = 0;
    bool ok = true;
    const uint32_t idesc = idesc_of(p.fp16, MODE == kWgrad, MODE != kFwd, kM, BN);
    for (int ti = first; ti < total && ok; ti += step) {
      const Tile t = decode<MODE, BN>(ti, p, seg, bn_out);
      int ka, kb;
      k_range(t, ka, kb);
      if (ka == kb) continue;  // nothing to add: the epilogue takes zeros
      for (int k0 = ka, k1; k0 < kb && ok; k0 = k1) {  // a drain each
        k1 = LONG ? min(kb, k0 + kDrain) : kb;
        if (!SPLIT || k0 != ka) {
          ok = warp_wait(&tempty[acc], acc_phase ^ 1u, kFlagMma);
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t d = tmem_base + (uint32_t)(acc * BN);
        for (int k = k0; k < k1; ++k) {
          ok = warp_wait(&full[stage], phase, kFlagMma);
          if (!ok) break;
          int k16 = kK / 16;
          if (MODE == kWgrad) {
            const int rem = t.kcnt - k * kK;  // rows of the segment in this step
            if (rem < kK) {
              k16 = (rem + 15) / 16;
              const int dirty = k16 * 16 - rem;  // other rows inside the last MMA
              for (int i = lane; i < dirty * 8 * (2 + BN / 64); i += 32) {
                const int box = i / (dirty * 8), j = i - box * dirty * 8;
                uint8_t* base = box < 2 ? smem + stage * a_stage + box * kBox
                                        : ring_b + stage * C::kBBytes + (box - 2) * kBox;
                reinterpret_cast<uint4*>(base)[rem * 8 + j] = make_uint4(0, 0, 0, 0);
              }
              asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
              __syncwarp();
            }
          }
          tc_fence_after();
          const uint64_t da = desc_a + (uint64_t)(stage * (a_stage >> 4));
          const uint64_t db = desc_b + (uint64_t)(stage * (C::kBBytes >> 4));
          if (one) {
#pragma unroll
            for (int q = 0; q < kK / 16; ++q)
              if (MODE != kWgrad || q < k16)
                umma_bf16(d, da + kStepA * q, db + kStepB * q, idesc, q ? 1u : k != k0);
            umma_commit(&empty[stage]);
          }
          __syncwarp();
          if (++stage == STAGES) {
            stage = 0;
            phase ^= 1u;
          }
        }
        if (!ok) break;
        if (one) umma_commit(&tfull[acc]);
        __syncwarp();
        if (!SPLIT) acc ^= 1;
        if (SPLIT || acc == 0) acc_phase ^= 1u;
      }
    }
    if (one) {
      // Every MMA this warp issued completes before TMEM is released.
      umma_commit(drain);
      mbar_wait(drain, 0, nullptr, nullptr, 0u, 100000000ull);
    }
    __syncwarp();
  } else if (!SPLIT) {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quadrant this warp may access
    const int r = q * 32 + lane;
    float* slot = p.sums + (int64_t)blockIdx.x * kSumFloats;  // WGRAD
    int acc = 0;
    uint32_t acc_phase = 0;
    auto release = [&]() {  // the accumulator is read; on to the other one
      tc_fence_before();
      mbar_arrive(&tempty[acc]);
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    };
    for (int ti = first; ti < total; ti += step) {
      const Tile t = decode<MODE, BN>(ti, p, seg, bn_out);
      const bool none = t.nk == 0;
      const int n_drains = LONG ? drains(t.nk) : 1;
      bool ok = true;
      for (int dr = 0; LONG && dr + 1 < n_drains; ++dr) {  // all but the last
        ok = warp_wait(&tfull[acc], acc_phase, kFlagEpilogue);
        if (!ok) break;
        tc_fence_after();
        for (int c0 = 0; c0 < BN && t.n0 + c0 < p.cols; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN) + c0, v);
          tmem_ld_wait();
          add_drained(slot, c0, r, dr == 0, false, v);
        }
        release();
      }
      if (!ok) break;
      if (!none) {
        if (!warp_wait(&tfull[acc], acc_phase, kFlagEpilogue)) break;
        tc_fence_after();
      }
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * BN);
      for (int c0 = 0; c0 < bn_out && t.n0 + c0 < p.cols; c0 += 16) {
        uint32_t a[16], u[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) a[j] = u[j] = 0u;
        if (!none) {
          tmem_ld16(tb + c0, a);
          if (glu) tmem_ld16(tb + BN / 2 + c0, u);
          tmem_ld_wait();
        }
        if (LONG && n_drains > 1) add_drained(slot, c0, r, false, true, a);
        if (r < t.rows)
          finish16<MODE>(p, t, r, t.n0 + c0, reinterpret_cast<float*>(a),
                         reinterpret_cast<const float*>(u));
      }
      if (!none) release();
    }
  }

  if (SPLIT) {
    // Each CTA leaves its partial sums in its own shared memory (the ring is
    // free: its MMAs are done) and finishes bn_out / parts columns, reading
    // the other parts of them and adding all in CTA order. (Storing them into
    // the finishing CTA instead takes a second barrier before: 1.5 us more.)
    const int q = warp & 3, r = q * 32 + lane;
    constexpr int kLd = kM + 1;  // rows of a column, one off: no bank conflicts below
    float* part = reinterpret_cast<float*>(smem);
    float* s_bias = reinterpret_cast<float*>(scratch + 8);
    const bool have = first < total;
    const int per = bn_out / (int)parts;  // 4 at least
    Tile t;
    if (have) t = decode<MODE, BN>(first, p, seg, bn_out);
    if (warp >= 2 && have) {
      if (MODE == kFwd) {  // what the epilogue reads, on its way before the sums are there
        const int n = t.n0 + rank * per, i = threadIdx.x - 64;
        if (p.residual && i < t.rows && n < p.cols)
          prefetch_l2(static_cast<const uint8_t*>(p.residual) +
                      ((int64_t)(t.row0 + i) * p.n_out + n) * (p.out32 ? 4 : 2));
        if (p.bias && i < (glu ? 2 : 1) * per) {
          const int c = n + (i < per ? i : i - per);
          if (c < p.cols)
            s_bias[i] = __ldg(p.bias + (int64_t)t.e * p.n_w + (i < per ? 0 : p.n_out) + c);
        }
      }
      int ka, kb;
      k_range(t, ka, kb);
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16);
      const int n_drains = LONG ? drains(kb - ka) : 1;
      if (LONG && n_drains > 1) {
        float sum[BN];
#pragma unroll
        for (int j = 0; j < BN; ++j) sum[j] = 0.0f;
        for (int dr = 0; dr < n_drains; ++dr) {
          if (!warp_wait(&tfull[0], dr & 1, kFlagEpilogue)) break;
          tc_fence_after();
#pragma unroll
          for (int c0 = 0; c0 < BN; c0 += 16) {
            uint32_t a[16];
            tmem_ld16(tb + c0, a);
            tmem_ld_wait();
#pragma unroll
            for (int j = 0; j < 16; ++j) sum[c0 + j] += __uint_as_float(a[j]);
          }
          tc_fence_before();
          mbar_arrive(&tempty[0]);
        }
#pragma unroll
        for (int j = 0; j < BN; ++j) part[j * kLd + r] = sum[j];
      } else {
        const bool got = ka < kb && warp_wait(&tfull[0], 0, kFlagEpilogue);
        tc_fence_after();
        for (int c0 = 0; c0 < BN; c0 += 16) {
          uint32_t a[16];
#pragma unroll
          for (int j = 0; j < 16; ++j) a[j] = 0u;
          if (got) {
            tmem_ld16(tb + c0, a);
            tmem_ld_wait();
          }
#pragma unroll
          for (int j = 0; j < 16; ++j) part[(c0 + j) * kLd + r] = __uint_as_float(a[j]);
        }
      }
    }
    cluster_sync();
    if (warp >= 2 && have) {
      // a thread per row and 4 columns, columns fastest; the loads of all
      // parts go out together
      for (int i = threadIdx.x - 64; i < t.rows * (per / 4); i += 128) {
        const int row = i / (per / 4), c = 4 * (i - row * (per / 4));
        const uint32_t mine = smem_addr(part + ((int)rank * per + c) * kLd + row);
        float a[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
        float va[8][4], vu[8][4];
#pragma unroll
        for (uint32_t s = 0; s < 8; ++s) {
          if (s >= parts) break;
          const uint32_t from = mapa_shared(mine, group0 + s);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            va[s][j] = ld_dsmem_f32(from + 4u * kLd * j);
            vu[s][j] = glu ? ld_dsmem_f32(from + 4u * kLd * (BN / 2 + j)) : 0.0f;
          }
        }
#pragma unroll
        for (uint32_t s = 0; s < 8; ++s) {
          if (s >= parts) break;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a[j] += va[s][j];
            u[j] += vu[s][j];
          }
        }
        finish4<MODE>(p, t, row, t.n0 + (int)rank * per + c, a, u, s_bias + c, per);
      }
    }
    cluster_sync();  // no CTA leaves while another reads its part
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 0) {
    tc_fence_after();
    tmem_dealloc(tmem_base, C::kTmemCols);
  }
}

template <int MODE, int BN, bool SPLIT, bool LONG>
__global__ void __launch_bounds__(kThreads, SPLIT ? 2 : 1)
    linear_kernel(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
                  const __grid_constant__ LinParams p) {
  linear_body<MODE, BN, SPLIT, LONG>(tm_a, tm_b, p, blockIdx.x);
}

// ------------------------------------------------------------- a few rows
constexpr int kFewThreads = 128;
constexpr int kFewRows = 4;              // rows of X at most
constexpr int kFewBytes = 40 * 1024;     // of them in shared memory

__device__ __forceinline__ uint4 load_once(const uint16_t* p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.L2::256B.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// The forward for up to four rows (decode): the weights stream through the
// CUDA cores, two weight rows a warp, FP32 FMAs against X in shared memory, the
// next weights' loads in flight meanwhile; lanes' sums are added by a
// shuffle tree. RT rows of a dense layer share the weights; with experts
// (RT = 1) blockIdx.y is the row. One token through 5120 x 5120 11.4 us, 4.6 TB/s,
// a call's fixed part included (tensor cores 17.3 us): bound by the fullest SM of
// one uneven wave (640 CTAs: 5 where the mean is 4.3). Four rows of four experts,
// swiglu, 41 us (58). One weight row a warp with twice
// the loads 13.3 us, four vectors per turn 14.8.
template <int RT, bool GLU>
__global__ void __launch_bounds__(kFewThreads)
    linear_few_kernel(const LinParams p, const uint16_t* __restrict__ x,
                      const uint16_t* __restrict__ w) {
  extern __shared__ uint4 s_x[];  // [RT][n_in / 8]
  if (p.clear_status && blockIdx.x == 0 && blockIdx.y == 0) clear_status_area(p);
  const int lane = threadIdx.x & 31;
  // this warp's weight rows: the gate and up rows of column n, or columns n
  // and n + 1 (n_out is even)
  const int slot = blockIdx.x * (kFewThreads / 32) + (threadIdx.x >> 5);
  const int slots = GLU ? p.n_out : p.n_out / 2;
  const bool live = slot < slots;
  const int n = (GLU ? 1 : 2) * min(slot, slots - 1);
  const int row0 = RT == 1 ? blockIdx.y : 0;
  int e = 0;
  if (p.offsets) {
    // the expert whose segment holds the row; each lane looks at every 32nd
    int found = -1;
    bool bad = false;
#pragma unroll 4
    for (int i = lane; i < p.E; i += 32) {
      int a, b;
      cut_off(p, i, a, b);
      bad |= b < a;
      if (row0 >= a && row0 < b) found = i;
    }
    if (__any_sync(0xffffffffu, bad)) {
      found = -1;
      int end = 0;
#pragma unroll 1
      for (int i = 0; i < p.E; ++i) {
        int a, b, lo, cnt;
        cut_off(p, i, a, b);
        take_segment(a, b, end, lo, cnt);
        if (row0 >= lo && row0 - lo < cnt) found = i;
      }
    }
    e = __reduce_max_sync(0xffffffffu, found);
    if (e < 0) return;  // no expert's row
  }
  const bool fp16 = p.fp16;
  const int nv = p.n_in / 8;  // 16-byte vectors of a row
  const uint16_t* wr = w + ((int64_t)e * p.n_w + n) * p.n_in;
  const int64_t second = GLU ? (int64_t)p.n_out * p.n_in : p.n_in;
  constexpr int U = 2;  // vectors of each row per lane and turn
  uint4 g[2][U], u[2][U];
  auto fetch = [&](int b, int v0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = v0 + 32 * i;
      if (v < nv) {
        g[b][i] = load_once(wr + 8 * v);
        u[b][i] = load_once(wr + second + 8 * v);
      }
    }
  };
  fetch(0, lane);
  const uint4* xr = reinterpret_cast<const uint4*>(x + (int64_t)row0 * p.n_in);
  const int rows = min(RT, p.rows - row0);
  for (int i = threadIdx.x; i < RT * nv; i += kFewThreads)
    s_x[i] = i < rows * nv ? __ldg(xr + i) : make_uint4(0, 0, 0, 0);
  // what the end needs, on its way: lane r finishes row r
  const bool mine = live && lane < rows;
  const int64_t at = (int64_t)(row0 + lane) * p.n_out + n;
  float bias[2] = {0.0f, 0.0f}, residual[2] = {0.0f, 0.0f};
  if (p.bias) {
    bias[0] = __ldg(p.bias + (int64_t)e * p.n_w + n);
    bias[1] = __ldg(p.bias + (int64_t)e * p.n_w + n + (GLU ? p.n_out : 1));
  }
  if (p.residual && mine) {
    residual[0] = load1(p.residual, at, p.out32, fp16);
    if (!GLU) residual[1] = load1(p.residual, at + 1, p.out32, fp16);
  }
  __syncthreads();

  float acc[RT], accu[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = accu[r] = 0.0f;
  auto add = [&](int b, int v0) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      const int v = v0 + 32 * i;
      if (v >= nv) break;
      float wf[8], uf[8];
      unpack8(g[b][i], wf, fp16);
      unpack8(u[b][i], uf, fp16);
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        float xf[8];
        unpack8(s_x[r * nv + v], xf, fp16);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          acc[r] = fmaf(wf[j], xf[j], acc[r]);
          accu[r] = fmaf(uf[j], xf[j], accu[r]);
        }
      }
    }
  };
  constexpr int kTurn = 32 * U;
  for (int v0 = lane; v0 - lane < nv; v0 += 2 * kTurn) {
    fetch(1, v0 + kTurn);
    add(0, v0);
    fetch(0, v0 + 2 * kTurn);
    add(1, v0 + kTurn);
  }
  float v[2] = {0.0f, 0.0f};
#pragma unroll
  for (int r = 0; r < RT; ++r) {
#pragma unroll
    for (int o = 16; o; o >>= 1) {
      acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
      accu[r] += __shfl_xor_sync(0xffffffffu, accu[r], o);
    }
    if (lane == r) {
      v[0] = acc[r] + bias[0];
      v[1] = accu[r] + bias[1];
    }
  }
  if (!mine) return;
  if (p.z) {
    const int64_t zt = (int64_t)(row0 + lane) * p.n_w + n;
    store1(p.z, zt, v[0], false, fp16);
    store1(p.z, zt + (GLU ? p.n_out : 1), v[1], false, fp16);
  }
  if (GLU) {
    swiglu<1, true>(v, v + 1);
    store1(p.out, at, v[0] + residual[0], p.out32, fp16);
  } else {
    activate<2, true>(p.act, v);
    store1(p.out, at, v[0] + residual[0], p.out32, fp16);
    store1(p.out, at + 1, v[1] + residual[1], p.out32, fp16);
  }
}

// ----------------------------------------- dZ and the sums of dZ over rows
constexpr int kActThreads = 256;
constexpr int kActPerSm = 4;
constexpr int kActCols = 256;  // columns of Y per CTA: 32 threads of 8; 8 rows at a time

// g = act'(z) g over 8 values, in FP32 (the choice is made once, see activate).
// Exponentials with __expf: dZ is rounded to 16 bits, and where their error
// counts (25 steps at z = -20) the slope, and with it the term of dbias, is e^-20
// of those near zero. The corrected form cost 6 % (gelu_tanh, 16384 x 5120).
__device__ __forceinline__ void act_grad8(int act, float* g, const float* z) {
  switch (act) {
    case BEAM_MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < 8; ++j) g[j] = z[j] > 0.0f ? g[j] : 0.0f;
      break;
    case BEAM_MOE_ACT_GELU:
#pragma unroll
      for (int j = 0; j < 8; ++j)
        g[j] *= fmaf(z[j], 0.39894228040143268f * __expf(-0.5f * z[j] * z[j]), normal_cdf(z[j]));
      break;
    case BEAM_MOE_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // its slope is s (1 - s) 2 da/dz; from |z| = 100 on s (1 - s) is zero, and the
        // square must not become infinite beside it
        const float s = tanh_gate(z[j]), zz = fminf(z[j] * z[j], 1e4f);
        g[j] *= fmaf(z[j] * s * (1.0f - s),
                     1.59576912160573071f * fmaf(3.0f * 0.044715f, zz, 1.0f), s);
      }
      break;
    case BEAM_MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float s = sigmoid_f(z[j]);
        g[j] *= s * fmaf(z[j], 1.0f - s, 1.0f);
      }
      break;
  }
}

struct ActParams {
  const uint16_t* dy;
  const uint16_t* z;  // NULL: act none
  uint16_t* dz;       // NULL: act none
  float* part;        // [row blocks][n_w] or NULL
};

// BLOCK rows of one expert x 256 columns at a time, CTAs walking the row
// blocks: dZ (rounded to 16 bits, the products' operand type) and the block's
// column sums of the unrounded dZ. Bound by HBM: dY and Z in, dZ out.
template <int BLOCK, bool GLU>
__global__ void __launch_bounds__(kActThreads, kActPerSm)
    act_backward_kernel(const LinParams p, const ActParams a) {
  __shared__ int tab[kMaxE + 1 + 8];
  __shared__ float s_sum[8][GLU ? 2 : 1][kActCols + 8];
  const Segments seg = {nullptr, nullptr, tab};
  const bool ordered = build_segments<kActThreads, BLOCK>(p, seg, tab + kMaxE + 1);
  if (p.clear_status && blockIdx.x == 0 && blockIdx.y == 0) clear_status_area(p);
  const bool fp16 = p.fp16;
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int n = blockIdx.y * kActCols + cl * 8;
  const int total = seg.rb[p.E];
  for (int q = blockIdx.x; q < total; q += gridDim.x) {
    const int e = find_expert(seg.rb, p.E, q);
    int lo, cnt;
    segment(p, e, ordered, lo, cnt);
    const int i0 = (q - seg.rb[e]) * BLOCK;
    const int64_t row0 = lo + i0;
    const int nrows = min(BLOCK, cnt - i0);
    float sum[8], sumu[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) sum[j] = sumu[j] = 0.0f;
    if (n < p.n_out) {
      // the next row's loads are out while this one is worked on
      const uint4* pd = reinterpret_cast<const uint4*>(a.dy + (row0 + rl) * p.n_out + n);
      const uint4* pz = reinterpret_cast<const uint4*>(a.z + (row0 + rl) * p.n_w + n);
      const int64_t sd = p.n_out, sz = p.n_w;  // 8 rows of 2-byte elements, in uint4
      uint4 rd, rz, ru;
      rd = rz = ru = make_uint4(0, 0, 0, 0);
      auto fetch = [&](int r) {
        if (r >= nrows) return;
        rd = *pd;
        if (a.z) {
          rz = *pz;
          if (GLU) ru = pz[p.n_out / 8];
        }
        pd += sd;
        pz += sz;
      };
      fetch(rl);
#pragma unroll 1
      for (int r = rl; r < nrows; r += 8) {
        float g[8], z[8], u[8];
        unpack8(rd, g, fp16);
        if (a.z) {
          unpack8(rz, z, fp16);
          if (GLU) unpack8(ru, u, fp16);
          fetch(r + 8);
          if (GLU) {
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float s = sigmoid_f(z[j]), d = g[j];
              // the slopes first: dY times a half may overflow where dZ does not
              g[j] = d * (u[j] * (s * fmaf(z[j], 1.0f - s, 1.0f)));
              u[j] = d * (z[j] * s);
              sumu[j] += u[j];
            }
          } else {
            act_grad8(p.act, g, z);
          }
          const int64_t at = (row0 + r) * p.n_w + n;
          store8(a.dz, at, g, fp16);
          if (GLU) store8(a.dz, at + p.n_out, u, fp16);
        } else {
          fetch(r + 8);
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] += g[j];
      }
    }
    if (!a.part) continue;
    __syncthreads();  // the last block's sums have been read
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      s_sum[rl][0][cl * 8 + j] = sum[j];
      if (GLU) s_sum[rl][GLU ? 1 : 0][cl * 8 + j] = sumu[j];
    }
    __syncthreads();
    const int c = blockIdx.y * kActCols + threadIdx.x;
    if (c < p.n_out) {
#pragma unroll
      for (int h = 0; h < (GLU ? 2 : 1); ++h) {
        float v = 0.0f;
#pragma unroll
        for (int w = 0; w < 8; ++w) v += s_sum[w][h][threadIdx.x];
        a.part[(int64_t)q * p.n_w + h * p.n_out + c] = v;
      }
    }
  }
}

// dbias[e] = the sums of e's row blocks, 6 interleaved chains joined in order,
// for 32 columns (block bx) and every by-th expert of n_by.
template <int BLOCK>
__device__ __forceinline__ void join_bias(const LinParams& p, const float* __restrict__ part,
                                          float* __restrict__ dbias, int bx, int by, int n_by) {
  __shared__ int tab[kMaxE + 1 + 8];
  __shared__ float s_sum[kThreads / 32][32];
  const Segments seg = {nullptr, nullptr, tab};
  build_segments<kThreads, BLOCK>(p, seg, tab + kMaxE + 1);
  const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
  const int c = bx * 32 + cl;
  for (int e = by; e < p.E; e += n_by) {
    float v = 0.0f;
    if (c < p.n_w)
#pragma unroll 4
      for (int q = seg.rb[e] + rl; q < seg.rb[e + 1]; q += kThreads / 32)
        v += __ldg(part + (int64_t)q * p.n_w + c);
    __syncthreads();
    s_sum[rl][cl] = v;
    __syncthreads();
    if (rl == 0 && c < p.n_w) {
      float t = 0.0f;
#pragma unroll
      for (int w = 0; w < kThreads / 32; ++w) t += s_sum[w][cl];
      dbias[(int64_t)e * p.n_w + c] = t;
    }
  }
}

template <int BLOCK>
__global__ void __launch_bounds__(kThreads)
    bias_join_kernel(const LinParams p, const float* __restrict__ part, float* __restrict__ dbias) {
  join_bias<BLOCK>(p, part, dbias, blockIdx.x, blockIdx.y, gridDim.y);
}

// A small backward's products and bias sums in one launch: they only wait for
// dZ, and each alone leaves SMs idle (39 x 136 x 2872, gelu, dZ included: 14.4 us,
// in launches of their own 23.4; 1000 x 520 x 1320: 27.9 and 39.8).
struct Joint {
  LinParams dx, dw;
  int dx_ctas, dw_ctas;  // whole clusters each; the CTAs behind them join dbias
  int join_x, join_y;
  const float* part;
  float* dbias;
};

template <bool LONG>
__global__ void __launch_bounds__(kThreads, 2)
    linear_joint_kernel(const __grid_constant__ CUtensorMap dx_a,
                        const __grid_constant__ CUtensorMap dx_b,
                        const __grid_constant__ CUtensorMap dw_a,
                        const __grid_constant__ CUtensorMap dw_b, const __grid_constant__ Joint j) {
  const int b = blockIdx.x;
  if (b < j.dx_ctas) {
    linear_body<kDgrad, 64, true, false>(dx_a, dx_b, j.dx, b);
  } else if (b < j.dx_ctas + j.dw_ctas) {
    linear_body<kWgrad, 64, true, LONG>(dw_a, dw_b, j.dw, b - j.dx_ctas);
  } else {
    const int i = b - j.dx_ctas - j.dw_ctas;
    if (i < j.join_x * j.join_y)
      join_bias<32>(j.dx, j.part, j.dbias, i % j.join_x, i / j.join_x, j.join_y);
  }
}

// ------------------------------------------------------------------- launches
template <int MODE, int BN, bool SPLIT, bool LONG>
cudaError_t launch_tiles(const CUtensorMap& ta, const CUtensorMap& tb, const LinParams& p,
                         int64_t tiles, int parts, cudaStream_t st) {
  using C = LinCfg<BN, SPLIT>;
  static PerDevice configured;  // the shared-memory attribute, once per device
  int unused = 0;
  cudaError_t err = per_device(configured, &unused, [](int*) {
    return cudaFuncSetAttribute(linear_kernel<MODE, BN, SPLIT, LONG>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)parts;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 1 : 0;
  const int64_t sms = device_sm_count();
  cfg.gridDim = dim3((unsigned)(SPLIT ? tiles * parts : (tiles < sms ? tiles : sms)));
  return cudaLaunchKernelEx(&cfg, linear_kernel<MODE, BN, SPLIT, LONG>, ta, tb, p);
}

// dZ and the row blocks' sums of it. CTAs for about eight per SM walk the blocks.
template <int BLOCK>
cudaError_t launch_act_blocks(const LinParams& p, const ActParams& a, int64_t blocks,
                              cudaStream_t st) {
  const int64_t cols = (p.n_out + kActCols - 1) / kActCols;
  int64_t gx = (2 * kActPerSm * (int64_t)device_sm_count() + cols - 1) / cols;
  if (gx > blocks) gx = blocks;
  const dim3 grid((unsigned)gx, (unsigned)cols);
  if (p.act == BEAM_MOE_ACT_SWIGLU)
    act_backward_kernel<BLOCK, true><<<grid, kActThreads, 0, st>>>(p, a);
  else
    act_backward_kernel<BLOCK, false><<<grid, kActThreads, 0, st>>>(p, a);
  return cudaGetLastError();
}

// CTAs that join dbias: 32 columns and a share of the experts each.
void join_grid(const LinParams& p, int* x, int* y) {
  *x = (p.n_w + 31) / 32;
  const int want = (8 * device_sm_count() + *x - 1) / *x;
  *y = want < p.E ? want : p.E;
}

cudaError_t launch_bias_join(const LinParams& p, const float* part, int block, float* dbias,
                             cudaStream_t st) {
  int x, y;
  join_grid(p, &x, &y);
  const dim3 grid((unsigned)x, (unsigned)y);
  if (block == 32) bias_join_kernel<32><<<grid, kThreads, 0, st>>>(p, part, dbias);
  else bias_join_kernel<128><<<grid, kThreads, 0, st>>>(p, part, dbias);
  return cudaGetLastError();
}

cudaError_t launch_act_backward(const LinParams& p, const ActParams& a, int block, int64_t blocks,
                                cudaStream_t st) {
  return block == 32 ? launch_act_blocks<32>(p, a, blocks, st)
                     : launch_act_blocks<128>(p, a, blocks, st);
}

// How a product runs: which tile, and on how many CTAs each.
struct Choice {
  int bn;     // columns per tile; 0: CTA pairs
  int parts;  // CTAs that split a tile's contraction (bn = 64)
};

// The four forms by their estimated times, in microseconds: a fixed part and a
// part per contraction step for each turn a CTA takes. The steps' costs are
// measured (16 shapes from 64 x 5120 x 5120 to 16000 x 640 x 640, each form
// forced): a step of 128 x 64, 128 x 128 and 128 x 256 on one CTA 0.37, 0.27
// and 0.48, of 256 x 256 on a pair 0.40. What the estimate decides, for one
// expert and 5120 x 5120: 64 rows split 22.7 (pairs 24.7), 256 rows 128
// columns 28.0 (split 33.4, pairs 37.8), 500 rows pairs 39.8 (128 columns
// 48.0), 800 rows 256 columns 46.3 (pairs 62.7, two turns for 6 of 74), 1500
// rows pairs 64 (256 columns 78). dW on pairs wins whenever they have a tile
// each (64 x 5120 x 5120: 26.8 against 53.1), its stores go out by TMA.
Choice choose(int mode, const LinParams& p, bool glu) {
  const double R = p.rows, E = p.E, sms = device_sm_count();
  auto up = [](double a, double b) { return (double)(int64_t)((a + b - 1) / b); };
  // turns of `slots` workers over t tiles, which are not all full
  auto turns = [](double t, double slots) {
    const double w = t / slots;
    return w <= 1.0 ? 1.0 : 0.5 * (w + (double)(int64_t)(w + 0.999999));
  };
  // row blocks of X: the full ones and the experts' last ones, half of which
  // are taken to be there
  auto row_blocks = [&](double m) { return up(R, m) + (E < R ? E - 1 : R - 1) / 2; };
  const bool dw = mode == kWgrad;
  const double steps = dw ? up(R / E, kK) : up(mode == kFwd ? p.n_in : p.n_w, kK);
  auto tiles = [&](double m, double n) {
    return dw ? E * up(p.n_w, m) * up(p.n_in, n) : row_blocks(m) * up(p.cols, glu ? n / 2 : n);
  };
  Choice best = {64, 1};
  const double t64 = tiles(128, 64);
  // Clusters of up to 1.5 CTAs per SM are resident at once. Each part has two
  // steps at least, four where there are many rows to join (300 x 520 x 1320,
  // dW: 9.4 us against 11.4; one row, 1000 x 520: 6.0 with two, 7.0 with four).
  const double least_steps = !dw && R / E <= 32 ? 2 : 4;
  while (best.parts < 8 && t64 * best.parts * 2 <= 1.5 * sms &&
         steps >= 2 * least_steps * best.parts)
    best.parts *= 2;
  double least = turns(t64 * best.parts, 2 * sms) * (steps / best.parts * 0.37 + 6.0);
  auto consider = [&](int bn, double us) {
    if (us < least) {
      least = us;
      best = {bn, 1};
    }
  };
  const double out = dw ? 3.0 : 0.0;  // dW's stores, which few steps do not hide
  consider(128, turns(tiles(128, 128), sms) * (steps * 0.27 + out) + 9.0);
  consider(256, turns(tiles(128, 256), sms) * (steps * 0.48 + 2 * out) + 12.0);
  // Experts with few rows stream their weights, at the copy bandwidth in either
  // form: 512 rows over 256 experts, 5120 -> 2 x 2560, 1640 us on one CTA a tile
  // and 1615 on pairs, 64 rows 439 and 453, 512 rows 2560 -> 5120 785 and 798.
  if (dw || R / E >= 96) {
    const double t = dw ? tiles(256, 256) : row_blocks(256) * up(p.cols, glu ? 128 : 256);
    consider(0, turns(t, sms / 2) * (steps * 0.40 + 0.7 * out) + 8.0);
  }
  return best;
}

int few_tile(const LinParams& p) { return p.offsets ? 1 : p.rows <= 1 ? 1 : p.rows <= 2 ? 2 : 4; }

// Three and four rows of a dense layer go there while the weights are small
// (640 x 640: 3.1 us, tensor cores 6.1); for 5120 x 5120 the rows' FMAs bound
// it (18.8 us against 16.9).
bool few_rows(const LinParams& p) {
  const int rt = few_tile(p);
  return p.rows <= kFewRows && rt * p.n_in * 2 <= kFewBytes &&
         (rt <= 2 || (int64_t)p.n_w * p.n_in <= (int64_t)8 << 20);
}

cudaError_t launch_few(const LinParams& p, const void* x, const void* w, cudaStream_t st) {
  const bool glu = p.act == BEAM_MOE_ACT_SWIGLU;
  const int rt = few_tile(p);
  const int slots = glu ? p.n_out : p.n_out / 2;
  const dim3 grid((unsigned)((slots + kFewThreads / 32 - 1) / (kFewThreads / 32)),
                  (unsigned)(p.offsets ? p.rows : 1));
  const uint16_t* xx = static_cast<const uint16_t*>(x);
  const uint16_t* ww = static_cast<const uint16_t*>(w);
  auto run = [&](auto rows, auto gated) {
    linear_few_kernel<decltype(rows)::value, decltype(gated)::value>
        <<<grid, kFewThreads, rows.value * p.n_in * 2, st>>>(p, xx, ww);
    return cudaGetLastError();
  };
  using std::integral_constant;
  auto by_rows = [&](auto gated) {
    return rt == 1 ? run(integral_constant<int, 1>(), gated)
                   : rt == 2 ? run(integral_constant<int, 2>(), gated)
                             : run(integral_constant<int, 4>(), gated);
  };
  return glu ? by_rows(std::true_type()) : by_rows(std::false_type());
}

// The one-CTA forms' parameters and tensor maps; *tiles: at most so many.
template <int MODE>
cudaError_t set_up(const LinParams& base, const Choice& c, const void* a, const void* b,
                   LinParams* out, CUtensorMap* ta, CUtensorMap* tb, int64_t* tiles) {
  LinParams p = base;
  const bool glu = MODE == kFwd && p.act == BEAM_MOE_ACT_SWIGLU;
  const int bn = c.bn;
  const int64_t R = p.rows, E = p.E;
  p.parts = c.parts;
  p.n_blk = (p.cols + (glu ? bn / 2 : bn) - 1) / (glu ? bn / 2 : bn);
  p.m_blk = (p.n_w + kM - 1) / kM;
  const int kc = MODE == kFwd ? p.n_in : p.n_w;
  p.nk = (kc + kK - 1) / kK;
  // row blocks: at most this many (every expert may end inside one)
  *tiles = p.n_blk * (MODE == kWgrad ? E * p.m_blk : R / kM + (E < R ? E : R));
  // boxes of the row operand: about an expert's rows, so that few rows cost
  // few bytes; 8 .. 128
  p.box_a = 8;
  while (p.box_a < 128 && p.box_a < 2 * R / E) p.box_a *= 2;
  // split: stages of A hold the rows of the largest possible tile
  p.a_stage = LinCfg<64, true>::kABytes;
  if (MODE != kWgrad && R <= 32) {
    p.box_a = R <= 8 ? 8 : R <= 16 ? 16 : 32;
    p.a_stage = p.box_a * kK * 2;
  }
  p.stages = LinCfg<64, true>::kRing / (p.a_stage + LinCfg<64, true>::kBBytes);
  if (p.stages > LinCfg<64, true>::kStages) p.stages = LinCfg<64, true>::kStages;
  *out = p;
  if (MODE == kWgrad) {
    const cudaError_t err = encode_tmap_2d_bf16(ta, a, p.n_w, R, 64, 64);
    return err != cudaSuccess ? err : encode_tmap_2d_bf16(tb, b, p.n_in, R, 64, 64);
  }
  const cudaError_t err = encode_tmap_2d_bf16(ta, a, kc, R, 64, p.box_a);
  return err != cudaSuccess ? err
                            : encode_tmap_3d_bf16(tb, b, p.n_in, p.n_w, E, 64,
                                                  MODE == kDgrad ? 64 : (glu ? bn / 2 : bn));
}

template <int MODE, bool LONG>
cudaError_t launch_form(const CUtensorMap& ta, const CUtensorMap& tb, const LinParams& p,
                        const Choice& c, int64_t tiles, cudaStream_t st) {
  if (c.bn == 256) return launch_tiles<MODE, 256, false, LONG>(ta, tb, p, tiles, 1, st);
  if (c.bn == 128) return launch_tiles<MODE, 128, false, LONG>(ta, tb, p, tiles, 1, st);
  return launch_tiles<MODE, 64, true, LONG>(ta, tb, p, tiles, c.parts, st);
}

// Whether an expert's rows may be more than a drain of the accumulators takes.
bool long_sums(int64_t rows) { return rows > (int64_t)kDrain * kK; }

template <int MODE>
cudaError_t launch_product(const LinParams& base, const Choice& c, const void* a, const void* b,
                           cudaStream_t st) {
  if (c.bn == 0) {
    if (base.clear_status) {  // the counter has to be zero before the first pair starts
      const cudaError_t e = cudaMemsetAsync(base.status, 0, kStatusWords * 4, st);
      if (e != cudaSuccess) return e;
    }
    return launch_linear_pair(MODE, base, a, b, st);
  }
  LinParams p;
  CUtensorMap ta, tb;
  int64_t tiles;
  const cudaError_t err = set_up<MODE>(base, c, a, b, &p, &ta, &tb, &tiles);
  if (err != cudaSuccess) return err;
  if (MODE == kWgrad && long_sums(p.rows))
    return launch_form<MODE, MODE == kWgrad>(ta, tb, p, c, tiles, st);
  return launch_form<MODE, false>(ta, tb, p, c, tiles, st);
}

int64_t split_ctas(int mode, const LinParams& p, const Choice& c) {
  const int64_t n_blk = (p.cols + 63) / 64, R = p.rows, E = p.E;
  const int64_t m = mode == kWgrad ? E * ((p.n_w + kM - 1) / kM) : R / kM + (E < R ? E : R);
  return n_blk * m * c.parts;
}

// The forms of a backward's products, whichever of its results are asked for
// (so that each comes out the same). True: they can go out in one launch, both
// splitting tiles over clusters and dbias summed over 32-row blocks. Then the
// splits are taken back, those with the fewest steps each first, until all
// CTAs are resident at once (1000 x 520 x 1320, gelu: 36.7 us with 384 CTAs,
// 27.9 with 285; 64 x 2000 x 1000: 21.9 and 17.1).
bool choose_backward(const LinParams& p, int block, Choice* dx, Choice* dw) {
  *dx = choose(kDgrad, p, false);
  *dw = choose(kWgrad, p, false);
  if (dx->bn != 64 || dw->bn != 64 || block != 32) return false;
  int jx, jy;
  join_grid(p, &jx, &jy);
  const int64_t sx = (p.n_w + kK - 1) / kK, sw = (p.rows / p.E + kK - 1) / kK;
  while ((dx->parts > 1 || dw->parts > 1) &&
         split_ctas(kDgrad, p, *dx) + split_ctas(kWgrad, p, *dw) + jx * jy >
             2 * (int64_t)device_sm_count()) {
    Choice* c = dw->parts == 1 || (dx->parts > 1 && sx / dx->parts < sw / dw->parts) ? dx : dw;
    c->parts /= 2;
  }
  return true;
}

template <bool LONG>
cudaError_t launch_joint(const LinParams& base, const Choice& cx, const Choice& cw, const void* dz,
                         const void* x, const void* w, void* dx, void* dw, const float* part,
                         float* dbias, cudaStream_t st) {
  Joint j;
  CUtensorMap xa, xb, wa, wb;
  int64_t tx = 0, tw = 0;
  LinParams p = base;
  p.out = dx;
  cudaError_t err = set_up<kDgrad>(p, cx, dz, w, &j.dx, &xa, &xb, &tx);
  if (err != cudaSuccess) return err;
  p.out = dw;
  err = set_up<kWgrad>(p, cw, dz, x, &j.dw, &wa, &wb, &tw);
  if (err != cudaSuccess) return err;
  const int64_t cluster = cx.parts > cw.parts ? cx.parts : cw.parts;
  auto whole = [&](int64_t n) { return (n + cluster - 1) / cluster * cluster; };
  j.dx_ctas = (int)whole(tx * cx.parts);
  j.dw_ctas = (int)whole(tw * cw.parts);
  j.dw.clear_status = 0;
  j.part = part;
  j.dbias = dbias;
  j.join_x = j.join_y = 0;
  if (dbias) join_grid(base, &j.join_x, &j.join_y);
  using C = LinCfg<64, true>;
  static PerDevice configured;
  int unused = 0;
  err = per_device(configured, &unused, [](int*) {
    return cudaFuncSetAttribute(linear_joint_kernel<LONG>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmemBytes);
  });
  if (err != cudaSuccess) return err;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)cluster;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)(j.dx_ctas + j.dw_ctas + whole((int64_t)j.join_x * j.join_y)));
  return cudaLaunchKernelEx(&cfg, linear_joint_kernel<LONG>, xa, xb, wa, wb, j);
}

struct LinLayout {
  size_t part, dz, sums, total;
  int block;       // rows per block of the dZ kernel
  int64_t blocks;  // row blocks at most
};

// Row blocks of E experts at most: every expert may end inside one.
int64_t most_blocks(int64_t rows, int64_t E, int block) {
  return rows / block + (E < rows ? E : rows);
}

int weight_rows(const beam_moe_linear_cfg& c) {
  return c.act == BEAM_MOE_ACT_SWIGLU ? 2 * c.n_out : c.n_out;
}

LinLayout lin_layout(const beam_moe_linear_cfg& c, int64_t rows, bool backward) {
  LinLayout L;
  const int64_t E = c.n_experts;
  // 32-row blocks while 128-row blocks would leave SMs without work (1000 x
  // 1320, gelu: 34 us with 128 rows)
  const int64_t cols = (c.n_out + kActCols - 1) / kActCols;
  const int64_t wide_from = (512 + cols - 1) / cols * 128;  // rows from which blocks hold 128
  L.block = rows < wide_from ? 32 : 128;
  L.blocks = most_blocks(rows, E, L.block);
  // A workspace serves every smaller number of rows too: the partial sums have
  // room for the most blocks that any of them has.
  int64_t room = L.blocks;
  if (L.block == 128 && most_blocks(wide_from - 1, E, 32) > room)
    room = most_blocks(wide_from - 1, E, 32);
  L.part = 256;
  L.dz = L.part;
  L.sums = L.dz;
  L.total = 256;
  if (backward) {
    const size_t n_w = (size_t)weight_rows(c);
    L.dz = (L.part + (size_t)room * n_w * 4 + 1023) / 1024 * 1024;
    L.sums = L.dz + (c.act == BEAM_MOE_ACT_NONE ? 0 : ((size_t)rows * n_w * 2 + 255) / 256 * 256);
    L.total = L.sums;
    if (long_sums(rows)) L.total += (size_t)device_sm_count() * kSumFloats * 4;
  }
  return L;
}

beam_moe_status check_linear(const beam_moe_linear_cfg* c, int64_t rows) {
  if (!c || rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->n_in <= 0 || c->n_out <= 0 || c->n_experts <= 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->act < BEAM_MOE_ACT_NONE || c->act > BEAM_MOE_ACT_SWIGLU) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->dtype != BEAM_MOE_BF16 && c->dtype != BEAM_MOE_FP16) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->out_fp32 != 0 && c->out_fp32 != 1) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->n_in % 8 || c->n_out % 8 || c->n_in > 65536 || c->n_out > 65536 || c->n_experts > kMaxE)
    return BEAM_MOE_ERR_UNSUPPORTED_SHAPE;
  // (2^22 rows of one expert through one tile: 30 ms, well inside the bounded waits)
  if (rows > (int64_t)1 << 22) return BEAM_MOE_ERR_UNSUPPORTED_SHAPE;
  return BEAM_MOE_OK;
}

beam_moe_status check_linear_ws(const beam_moe_linear_cfg* c, int64_t rows, bool backward,
                                const void* offsets, const void* ws, size_t ws_bytes) {
  if (!ws || (c->n_experts > 1 && !offsets)) return BEAM_MOE_ERR_INVALID_ARG;
  if (reinterpret_cast<uintptr_t>(ws) & 15u) return BEAM_MOE_ERR_ALIGNMENT;
  if (ws_bytes < lin_layout(*c, rows, backward).total) return BEAM_MOE_ERR_WORKSPACE_TOO_SMALL;
  return BEAM_MOE_OK;
}

// A call without rows launches no kernel that clears the status area; the
// status word of a workspace that was given says so all the same.
cudaError_t clear_status(void* ws, size_t ws_bytes, cudaStream_t st) {
  if (!ws || ws_bytes < kStatusWords * 4) return cudaSuccess;
  return cudaMemsetAsync(ws, 0, kStatusWords * 4, st);
}

LinParams lin_params(const beam_moe_linear_cfg& c, int64_t rows, const int32_t* offsets, void* ws) {
  LinParams p;
  memset(&p, 0, sizeof(p));
  p.offsets = offsets;
  p.E = c.n_experts;
  p.rows = (int)rows;
  p.n_in = c.n_in;
  p.n_out = c.n_out;
  p.n_w = weight_rows(c);
  p.act = c.act;
  p.fp16 = c.dtype == BEAM_MOE_FP16;
  p.out32 = c.out_fp32;
  p.status = static_cast<unsigned*>(ws);
  return p;
}

}  // namespace
}  // namespace beam

#define LIN_TRY(expr)                        \
  do {                                       \
    const beam_moe_status s_ = (expr);       \
    if (s_ != BEAM_MOE_OK) return s_;        \
  } while (0)

#define LIN_CUDA(expr)                                          \
  do {                                                          \
    if ((expr) != cudaSuccess) return BEAM_MOE_ERR_CUDA;        \
  } while (0)

extern "C" {

beam_moe_status beam_moe_linear_workspace_size(const beam_moe_linear_cfg* cfg, int64_t rows,
                                               int32_t backward, size_t* bytes) {
  LIN_TRY(beam::check_linear(cfg, rows));
  if (!bytes || (backward != 0 && backward != 1)) return BEAM_MOE_ERR_INVALID_ARG;
  *bytes = beam::lin_layout(*cfg, rows, backward == 1).total;
  return BEAM_MOE_OK;
}

beam_moe_status beam_moe_linear(const beam_moe_linear_cfg* cfg, int64_t rows, const void* x,
                                const void* w, const float* bias, const void* residual,
                                const int32_t* offsets, void* y, void* z, void* ws,
                                size_t ws_bytes, void* stream) {
  LIN_TRY(beam::check_linear(cfg, rows));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (rows == 0) return beam::cuda_status(beam::clear_status(ws, ws_bytes, st));
  LIN_TRY(beam::check_ops_ptrs({x, w, y}, {bias, residual, offsets, z}));
  LIN_TRY(beam::check_linear_ws(cfg, rows, false, offsets, ws, ws_bytes));
  beam::LinParams p = beam::lin_params(*cfg, rows, offsets, ws);
  p.cols = cfg->n_out;
  p.bias = bias;
  p.residual = residual;
  p.z = z;
  p.out = y;
  p.clear_status = 1;
  if (beam::few_rows(p)) {
    LIN_CUDA(beam::launch_few(p, x, w, st));
    return BEAM_MOE_OK;
  }
  const beam::Choice c = beam::choose(beam::kFwd, p, cfg->act == BEAM_MOE_ACT_SWIGLU);
  LIN_CUDA(beam::launch_product<beam::kFwd>(p, c, x, w, st));
  return BEAM_MOE_OK;
}

beam_moe_status beam_moe_linear_backward(const beam_moe_linear_cfg* cfg, int64_t rows,
                                         const void* dy, const void* x, const void* w,
                                         const void* z, const int32_t* offsets, void* dx, void* dw,
                                         float* dbias, void* ws, size_t ws_bytes, void* stream) {
  LIN_TRY(beam::check_linear(cfg, rows));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const size_t n_w = (size_t)beam::weight_rows(*cfg), E = (size_t)cfg->n_experts;
  if (rows == 0) {  // no rows: the sums over rows are zero, dX is empty
    LIN_TRY(beam::check_ops_ptrs({}, {dw, dbias}));
    LIN_CUDA(beam::clear_status(ws, ws_bytes, st));
    if (dw) LIN_CUDA(cudaMemsetAsync(dw, 0, E * n_w * cfg->n_in * 2, st));
    if (dbias) LIN_CUDA(cudaMemsetAsync(dbias, 0, E * n_w * 4, st));
    return BEAM_MOE_OK;
  }
  if (!dx && !dw && !dbias) return BEAM_MOE_ERR_INVALID_ARG;
  if ((dw && !x) || (dx && !w)) return BEAM_MOE_ERR_INVALID_ARG;
  if (cfg->act != BEAM_MOE_ACT_NONE && !z) return BEAM_MOE_ERR_INVALID_ARG;
  LIN_TRY(beam::check_ops_ptrs({dy}, {x, w, z, offsets, dx, dw, dbias}));
  LIN_TRY(beam::check_linear_ws(cfg, rows, true, offsets, ws, ws_bytes));
  const beam::LinLayout L = beam::lin_layout(*cfg, rows, true);
  char* base = static_cast<char*>(ws);
  beam::LinParams p = beam::lin_params(*cfg, rows, offsets, ws);
  const bool acted = cfg->act != BEAM_MOE_ACT_NONE;
  const void* dz = acted ? static_cast<const void*>(base + L.dz) : dy;
  p.clear_status = 1;  // by the first launch
  if (acted || dbias) {
    beam::ActParams a;
    a.dy = static_cast<const uint16_t*>(dy);
    a.z = acted ? static_cast<const uint16_t*>(z) : nullptr;
    a.dz = acted ? reinterpret_cast<uint16_t*>(base + L.dz) : nullptr;
    a.part = dbias ? reinterpret_cast<float*>(base + L.part) : nullptr;
    LIN_CUDA(beam::launch_act_backward(p, a, L.block, L.blocks, st));
    p.clear_status = 0;
  }
  p.cols = cfg->n_in;
  const float* part = reinterpret_cast<const float*>(base + L.part);
  beam::Choice cx, cw;
  const bool joint = beam::choose_backward(p, L.block, &cx, &cw);
  if (joint && dx && dw) {
    LIN_CUDA((beam::long_sums(rows) ? beam::launch_joint<true> : beam::launch_joint<false>)(
        p, cx, cw, dz, x, w, dx, dw, part, dbias, st));
    return BEAM_MOE_OK;
  }
  if (dbias) LIN_CUDA(beam::launch_bias_join(p, part, L.block, dbias, st));
  if (dx) {
    p.out = dx;
    LIN_CUDA(beam::launch_product<beam::kDgrad>(p, cx, dz, w, st));
    p.clear_status = 0;
  }
  if (dw) {
    p.out = dw;
    p.sums = reinterpret_cast<float*>(base + L.sums);
    LIN_CUDA(beam::launch_product<beam::kWgrad>(p, cw, dz, x, st));
  }
  return BEAM_MOE_OK;
}

}  // extern "C"
