// linear_pair.cu - the linear operator's products on CTA pairs (tcgen05
// cta_group::2), for experts with many rows. The same three products as
// linear.cu, as D^T for the first two:
//
//   FWD    D[n][r] = sum_k W_e[n][k] X[r][k]      M: weight rows, N: rows of X
//   DGRAD  D[k][r] = sum_n W_e[n][k] dZ[r][n]     M: weight columns
//   WGRAD  D[n][k] = sum_r dZ[r][n] X[r][k]       M: rows of dW_e
//
// One MMA covers 256 x up to 256; each CTA of the pair holds 128 of M and half
// of N in shared memory and 128 accumulator rows, double-buffered in TMEM, so
// the epilogue of one tile overlaps the MMAs of the next. The rows of X and dZ
// are N in FWD and DGRAD because N may be any multiple of 16: an expert's last
// row block costs what it holds, where as M it would cost 128 rows (measured
// at 8192 rows over 32 experts: a fifth of the tensor work).
//
// swiglu: a CTA's 128 weight rows are gate and up rows of 64 columns in turns
// of 16, so a warp's 32 TMEM lanes hold 16 gate rows and their up rows, which
// lanes exchange with one shuffle.
//
// WGRAD's last step of a segment holds rows of other experts. Each CTA takes
// that step's copies on a barrier of its own; a warp of its own (6) zeroes the
// rows in both operands as soon as they have landed, ahead of the MMAs, and
// releases the step to the MMA thread (done by the MMA warp in turn it cost
// 160 of 1260 us at 512 rows an expert).
//
// Roles, whole warps with one elected lane issuing: warp 0 issues this CTA's TMA
// loads, counted on the even CTA's barriers, and (even CTA) hands out tiles;
// warp 1 of the even CTA issues the pair's MMAs; warps 2-5 of each CTA drain
// their TMEM. No load uses multicast. Every wait is bounded.
//
// Measured: 16384 x 5120 x 5120 dense, Y 585 us, dX 570, dW 595 (1.38 to 1.5
// PFLOP/s, at the rate of a library product under the power limit); 32 experts
// of 509 rows each 677, 674 and 830 us. Bound by the power limit, and dW by
// what it moves through L2 (10 GB).
#include <string.h>

#include "linear.cuh"
#include "ops.h"

namespace beam {
namespace {

using namespace lin;

constexpr int kThreads = 192;   // WGRAD: a warp more, see below
constexpr int kPair = 256;     // M and (most) N of a pair's tile
constexpr int kGroup = 8;      // row blocks that share a sweep over the weights
constexpr int kTileSlots = 8;  // tile indices between the fetching producer and the rest
constexpr int kABytes = 128 * kK * 2;
constexpr int kBBytes = 128 * kK * 2;
constexpr int kStageBytes = kABytes + kBBytes;
constexpr int kStages = 6;
constexpr int kBarBytes = 640;
constexpr int kStoreBytes = 32 * 128;  // a warp's staged 32 x 64 block (WGRAD)

template <int MODE>
struct PairMem {
  static constexpr int kBlock = MODE == kWgrad ? kThreads + 32 : kThreads;
  // behind the ring, WGRAD: 2 staged blocks per warp; else the segment table
  static constexpr int kMore = MODE == kWgrad ? 4 * 2 * kStoreBytes : 4 * (kMaxE + 1 + 7);
  static constexpr int kBytes = 1024 + kStages * kStageBytes + kMore + kBarBytes;
  static_assert(kBytes <= 232448, "dynamic shared memory above the sm_100 limit");
};

// ------------------------------------------------------------- TMA for pairs
__device__ __forceinline__ void tma_load_3d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t c0, int32_t c1, int32_t c2,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_load_4d_pair(void* dst, const CUtensorMap* map, uint32_t bar,
                                                 int32_t c0, int32_t c1, int32_t c2, int32_t c3,
                                                 uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      ".L2::cache_hint [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3),
      "l"(policy)
      : "memory");
}

__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* src, int32_t c0,
                                             int32_t c1, int32_t c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(smem_addr(src)), "r"(c0), "r"(c1), "r"(c2)
      : "memory");
}

// -------------------------------------------------------------------- tiles
// A tile, as it is handed from the even CTA's producer to every role.
struct alignas(16) PairTile {
  int e;        // expert; -1: no tiles left
  int m0;       // first row of M (swiglu: first of 128 columns of Y)
  int n0;       // WGRAD: first column
  int row0;     // first row of X or dZ (WGRAD: of the segment)
  int rows;     // rows of the tile (WGRAD: of the segment)
  int nk;       // contraction steps
  int once;     // the weight tile is read by this tile alone
  int unused;
};
static_assert(sizeof(PairTile) == 32, "two 16-byte pieces");

// FWD, DGRAD: expert by expert, its row blocks in groups of 8; inside a group
// weight tile by weight tile, row blocks fastest. The pairs at work at one time
// then share row blocks and weight tiles through L2, and the weights are read
// from HBM once for up to 2048 rows. (Groups over the experts' row blocks
// alike, to run experts bound by bytes beside experts bound by the tensor
// cores, split experts between groups: 1.4 times the bytes, no faster in a
// short run and slower in a long one, under the power limit.) WGRAD: groups of
// 8 column tiles, row tile by row tile.
template <int MODE>
__device__ __forceinline__ PairTile decode_pair(int t, const LinParams& p, const Segments& s,
                                                bool ordered, int m_step) {
  PairTile d;
  const int m_blk = p.m_blk;
  int blks, local;
  if (MODE == kWgrad) {
    const int per = m_blk * p.n_blk;
    d.e = t / per;
    local = t - d.e * per;
    blks = p.n_blk;
  } else {
    d.e = find_expert(s.rb, p.E, t / m_blk);
    local = t - s.rb[d.e] * m_blk;
    blks = s.rb[d.e + 1] - s.rb[d.e];
  }
  const int g = local / (kGroup * m_blk);
  const int in_g = min(kGroup, blks - g * kGroup);
  const int rem = local - g * kGroup * m_blk;
  const int mb = rem / in_g;
  const int nb = g * kGroup + rem - mb * in_g;
  d.m0 = mb * m_step;
  d.unused = 0;
  if (MODE == kWgrad) {
    segment(p, d.e, ordered, d.row0, d.rows);
    d.nk = (d.rows + kK - 1) / kK;
    d.n0 = nb * kPair;
    d.once = 0;
  } else {
    const int i0 = nb * kPair;
    int lo, cnt;
    segment(p, d.e, ordered, lo, cnt);
    d.row0 = lo + i0;
    d.rows = min(kPair, cnt - i0);
    d.nk = p.nk;
    d.n0 = 0;
    d.once = blks == 1;
  }
  return d;
}

__device__ __forceinline__ void st_cluster_v4(uint32_t addr, int4 v) {
  asm volatile("st.shared::cluster.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y),
               "r"(v.z), "r"(v.w)
               : "memory");
}

template <class T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __half narrow<__half>(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) {
  return __float2bfloat16_rn(v);
}

// n <= N values, one per row, into one column of a row-major matrix. A warp's
// lanes hold neighbouring columns: 64 or 128 bytes of a row per instruction.
template <int N, class T>
__device__ __forceinline__ void store_rows(void* p, int64_t at, int64_t ld, int n, const float* v) {
  T* o = static_cast<T*>(p) + at;
#pragma unroll
  for (int j = 0; j < N; ++j, o += ld)
    if (j < n) *o = narrow<T>(v[j]);
}

template <int N>
__device__ __forceinline__ void store_rows(void* p, int64_t at, int64_t ld, int n, const float* v,
                                           bool f32, bool fp16) {
  if (f32) store_rows<N, float>(p, at, ld, n, v);
  else if (fp16) store_rows<N, __half>(p, at, ld, n, v);
  else store_rows<N, __nv_bfloat16>(p, at, ld, n, v);
}

// N rows (from row r0 of the tile) of one column of Y; v: act(Z). F32: the type
// of Y and the residual.
template <int N, bool F32>
__device__ __forceinline__ void finish_rows(const LinParams& p, const PairTile& t, int col, int r0,
                                            float* v) {
  const int n = min(N, t.rows - r0);
  const int64_t at = (int64_t)(t.row0 + r0) * p.n_out + col;
  if (p.residual) {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < n) v[j] += load1(p.residual, at + (int64_t)j * p.n_out, F32, p.fp16);
  }
  store_rows<N>(p.out, at, p.n_out, n, v, F32, p.fp16);
}

template <int MODE, bool GLU, bool F32>
__global__ void __launch_bounds__(PairMem<MODE>::kBlock, 1)
    linear_pair_kernel(const __grid_constant__ CUtensorMap tm_a,
                       const __grid_constant__ CUtensorMap tm_b,
                       const __grid_constant__ CUtensorMap tm_c, const LinParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                             ~static_cast<uintptr_t>(1023));
  uint8_t* more = smem + kStages * kStageBytes;
  uint64_t* full = reinterpret_cast<uint64_t*>(more + PairMem<MODE>::kMore);
  uint64_t* empty = full + kStages;
  uint64_t* tail = empty + kStages;  // WGRAD: a segment's last step has landed here
  uint64_t* tfull = tail + kStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint64_t* tsfull = drain + 1;             // [kTileSlots] a tile is in the ring
  uint64_t* tsempty = tsfull + kTileSlots;  // [kTileSlots] every reader has it (even CTA)
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(tsempty + kTileSlots);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  PairTile* ring = reinterpret_cast<PairTile*>(  // [kTileSlots]
      (reinterpret_cast<uintptr_t>(tmem_holder + 2) + 15) & ~static_cast<uintptr_t>(15));
  static_assert((3 * kStages + 5 + 2 * kTileSlots) * 8 + 8 + 16 + 32 * kTileSlots <= kBarBytes,
                "barrier area");
  // readers of a tile: the odd CTA's producer, the MMA thread and, of each
  // CTA, the four epilogue warps (WGRAD: and the cleaner)
  constexpr int kTileReaders = 2 + 2 * (MODE == kWgrad ? 5 : 4);
  int* tab = reinterpret_cast<int*>(more);
  const Segments seg = {nullptr, nullptr, tab};

  const int warp = uniform(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_ctarank();  // 0: the CTA that issues MMAs
  const bool leader = rank == 0;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      // WGRAD: a tail step is released by both CTAs' cleaners, the others by
      // the even CTA's producer alone, which arrives twice
      mbar_init(&full[s], MODE == kWgrad ? 2 : 1);
      mbar_init(&empty[s], 1);
      mbar_init(&tail[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * 128);
    }
    mbar_init(drain, 1);
    for (int s = 0; s < kTileSlots; ++s) {
      mbar_init(&tsfull[s], 1);
      mbar_init(&tsempty[s], kTileReaders);
    }
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_a);
    tma_prefetch_desc(&tm_b);
    tma_prefetch_desc(&tm_c);
  }
  if (warp == 1) {
    tmem_alloc_pair(tmem_holder, 512);
    tmem_relinquish_pair();
  }
  const bool ordered = MODE == kWgrad ? offsets_ordered(p)
                                      : build_segments<kThreads, kPair>(p, seg, tab + kMaxE + 1);
  tc_fence_before();
  cluster_sync();  // barriers of both CTAs initialised, TMEM allocated
  tc_fence_after();
  const uint32_t tmem_base = (uint32_t)uniform((int)*tmem_holder);
  const int m_step = GLU ? 128 : kPair;
  const int total = MODE == kWgrad ? p.E * p.m_blk * p.n_blk : seg.rb[p.E] * p.m_blk;

  // Tiles are handed out in order at run time (they differ in rows, and in
  // order their operands stay in L2): the even CTA's producer takes the next
  // index from a counter, works out the tile and publishes it to every role of
  // both CTAs. e = -1: no tiles left, or a wait gave up (the role stops).
  int tslot = 0;
  uint32_t tphase = 0;
  auto next_slot = [&]() {
    if (++tslot == kTileSlots) {
      tslot = 0;
      tphase ^= 1u;
    }
  };
  auto publish_tile = [&](int index) -> PairTile {
    // the readers' arrivals (some from the other CTA) come before the rewrite
    const bool got = mbar_wait(&tsempty[tslot], tphase ^ 1u, abort_flag, p.status, kFlagProducer,
                               1000000000ull, true);
    PairTile t = {-1, 0, 0, 0, 0, 0, 0, 0};
    if (!__all_sync(0xffffffffu, got)) return t;
    if (index < total) t = decode_pair<MODE>(index, p, seg, ordered, m_step);
    if (lane == 0) {
      const int4 a = make_int4(t.e, t.m0, t.n0, t.row0), b = make_int4(t.rows, t.nk, t.once, 0);
      int4* slot = reinterpret_cast<int4*>(&ring[tslot]);
      slot[0] = a;
      slot[1] = b;
      const uint32_t other = mapa_shared(smem_addr(slot), 1);
      st_cluster_v4(other, a);
      st_cluster_v4(other + 16, b);
      mbar_arrive(&tsfull[tslot]);
      mbar_arrive_cluster(mapa_shared(smem_addr(&tsfull[tslot]), 1));
    }
    next_slot();
    return t;
  };
  // All 32 lanes read, lane 0 arrives for them. What the other CTA stored here
  // is acquired at cluster scope.
  auto read_tile = [&](uint32_t flag) -> PairTile {
    const bool got =
        leader ? mbar_wait(&tsfull[tslot], tphase, abort_flag, p.status, flag)
               : mbar_wait(&tsfull[tslot], tphase, abort_flag, p.status, flag, 1000000000ull, true);
    PairTile t = {-1, 0, 0, 0, 0, 0, 0, 0};
    if (!__all_sync(0xffffffffu, got)) return t;
    const int4* slot = reinterpret_cast<const int4*>(&ring[tslot]);
    const int4 a = slot[0], b = slot[1];
    t.e = uniform(a.x);
    t.m0 = a.y;
    t.n0 = a.z;
    t.row0 = a.w;
    t.rows = uniform(b.x);
    t.nk = uniform(b.y);
    t.once = b.z;
    __syncwarp();  // every lane has read the slot
    if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&tsempty[tslot]), 0));
    next_slot();
    return t;
  };
  // A wait of the whole warp.
  auto warp_wait = [&](uint64_t* bar, uint32_t parity, uint32_t flag, bool cluster) -> bool {
    return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, p.status, flag,
                                             1000000000ull, cluster));
  };

  if (warp == 0) {
    // -------------------------------------------------------- TMA producer
    const uint64_t pol_stream = policy_evict_first();
    const uint64_t pol_keep = policy_evict_normal();
    const bool one = elect_one();
    const uint32_t full0 = mapa_shared(smem_addr(full), 0);     // the even CTA's
    const uint32_t tail0 = mapa_shared(smem_addr(tail), rank);  // this CTA's
    int stage = 0;
    uint32_t phase = 0;
    int64_t issued = 0;
    bool ok = true;
    // a tile is published one ahead and its index taken two ahead, so that
    // neither the atomic's latency nor the other CTA's is waited for
    int taken = 0;
    auto take = [&]() {
      if (leader && lane == 0) taken = atomicAdd(p.next_tile, 1);
    };
    take();
    PairTile t = leader ? publish_tile(uniform(taken)) : read_tile(kFlagProducer);
    take();
    PairTile next;
    for (; t.e >= 0 && ok; t = next) {
      if (leader) {
        next = publish_tile(uniform(taken));
        take();
      }
      const int half = ((t.rows + 15) & ~15) >> 1;  // this CTA's rows of N: 8 .. 128
      const bool box64 = half <= 64;
      const CUtensorMap* tmx = box64 ? &tm_c : &tm_b;  // boxes of 64 or 128 rows
      const int xrow = t.row0 + (int)rank * half;
      const uint32_t tx = MODE == kWgrad ? 2 * kStageBytes
                                         : 2u * (kABytes + (box64 ? 64 : 128) * kK * 2);
      const uint64_t pol_w = t.once ? pol_stream : pol_keep;
      const int m0 = t.m0 + (int)rank * (m_step / 2), n0 = t.n0 + (int)rank * 128;
      for (int k = 0; k < t.nk; ++k) {
        if (!warp_wait(&empty[stage], phase ^ 1u, kFlagProducer, false)) {
          ok = false;
          break;
        }
        uint8_t* sa = smem + stage * kStageBytes;
        uint8_t* sb = sa + kABytes;
        uint32_t bar = full0 + 8 * stage;
        const int kx = k * kK;
        if (one) {
          if (MODE == kWgrad) {
            if (t.rows - kx < kK) {  // a segment's last step: the cleaner's
              bar = tail0 + 8 * stage;
              mbar_arrive_expect_tx(&tail[stage], kStageBytes);
            } else if (leader) {
              mbar_arrive_expect_tx(&full[stage], tx);
              mbar_arrive(&full[stage]);
            }
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              tma_load_2d_pair(sa + b * kBox, &tm_a, bar, m0 + b * 64, t.row0 + kx, pol_keep);
              tma_load_2d_pair(sb + b * kBox, &tm_b, bar, n0 + b * 64, t.row0 + kx, pol_keep);
            }
          } else {
            if (leader) mbar_arrive_expect_tx(&full[stage], tx);
            if (MODE == kDgrad) {
#pragma unroll
              for (int b = 0; b < 2; ++b)
                tma_load_3d_pair(sa + b * kBox, &tm_a, bar, m0 + b * 64, kx, t.e, pol_w);
            } else if (GLU) {
#pragma unroll
              for (int b = 0; b < 4; ++b)
                tma_load_4d_pair(sa + b * (kABytes / 4), &tm_a, bar, kx, m0 + b * 16, 0, t.e,
                                 pol_w);
            } else {
              tma_load_3d_pair(sa, &tm_a, bar, kx, m0, t.e, pol_w);
            }
            tma_load_2d_pair(sb, tmx, bar, kx, xrow, pol_keep);
          }
        }
        __syncwarp();
        ++issued;
        if (++stage == kStages) {
          stage = 0;
          phase ^= 1u;
        }
      }
      if (!leader) next = read_tile(kFlagProducer);
    }
    // The even CTA's full barriers count both CTAs' copies: wait for the
    // last ones to land before either CTA can leave.
    if (leader && lane == 0) {
      const int64_t from = issued > kStages ? issued - kStages : 0;
      for (int64_t i = from; i < issued; ++i)
        mbar_wait(&full[i % kStages], (uint32_t)((i / kStages) & 1), nullptr, nullptr, 0u,
                  100000000ull);
    }
    __syncwarp();
  } else if (warp == 1) {
    if (leader) {
      // --------------------------------------------------------- MMA issuer
      const bool one = elect_one();
      const uint32_t smem0 = smem_addr(smem);
      const uint64_t desc_a = MODE == kFwd ? smem_desc_k_sw128(smem0) : smem_desc_mn_sw128(smem0);
      const uint64_t desc_b = MODE == kWgrad ? smem_desc_mn_sw128(smem0 + kABytes)
                                             : smem_desc_k_sw128(smem0 + kABytes);
      constexpr uint32_t kStepA = MODE == kFwd ? 32 >> 4 : 2048 >> 4;
      constexpr uint32_t kStepB = MODE == kWgrad ? 2048 >> 4 : 32 >> 4;
      int stage = 0;
      uint32_t phase = 0;
      int acc = 0;
      uint32_t acc_phase = 0;
      bool ok = true;
      while (ok) {
        const PairTile t = read_tile(kFlagMma);
        if (t.e < 0) break;
        if (t.nk == 0) continue;  // an expert without rows: the epilogue takes zeros
        const uint32_t idesc =
            idesc_of(p.fp16, MODE != kFwd, MODE == kWgrad, kPair,
                     MODE == kWgrad ? kPair : (uint32_t)((t.rows + 15) & ~15));
        for (int k0 = 0, k1; k0 < t.nk && ok; k0 = k1) {  // a drain each
          k1 = MODE == kWgrad ? min(t.nk, k0 + kDrain) : t.nk;
          ok = warp_wait(&tempty[acc], acc_phase ^ 1u, kFlagMma, false);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = tmem_base + (uint32_t)(acc * kPair);
          for (int k = k0; k < k1; ++k) {
            // WGRAD: the other CTA's cleaned rows come with its arrival
            if (!warp_wait(&full[stage], phase, kFlagMma, MODE == kWgrad)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t da = desc_a + (uint64_t)(stage * (kStageBytes >> 4));
            const uint64_t db = desc_b + (uint64_t)(stage * (kStageBytes >> 4));
            const int k16 = MODE == kWgrad ? min(kK / 16, (t.rows - k * kK + 15) / 16) : kK / 16;
            if (one) {
#pragma unroll
              for (int q = 0; q < kK / 16; ++q)
                if (MODE != kWgrad || q < k16)
                  umma_bf16_pair(d, da + kStepA * q, db + kStepB * q, idesc, q ? 1u : k != k0);
              umma_commit_pair(&empty[stage], 0x3);
            }
            __syncwarp();
            if (++stage == kStages) {
              stage = 0;
              phase ^= 1u;
            }
          }
          if (!ok) break;
          if (one) umma_commit_pair(&tfull[acc], 0x3);
          __syncwarp();
          acc ^= 1;
          if (acc == 0) acc_phase ^= 1u;
        }
      }
      // Every MMA of the pair completes before TMEM is released.
      if (one) {
        umma_commit_pair(drain, 0x1);
        mbar_wait(drain, 0, nullptr, nullptr, 0u, 100000000ull);
      }
    }
    __syncwarp();
  } else if (MODE == kWgrad && warp == 6) {
    // ---------------------------------------------------------------- cleaner
    int stage = 0;
    uint32_t phase = 0;  // a bit per stage: its tail barrier is used now and then
    for (;;) {
      const PairTile t = read_tile(kFlagProducer);
      if (t.e < 0) break;
      stage = (stage + t.nk) % kStages;
      const int rem = t.rows % kK;  // rows of the segment in its last step
      if (rem == 0) continue;
      const int at = stage == 0 ? kStages - 1 : stage - 1;
      if (!__all_sync(0xffffffffu, mbar_wait(&tail[at], (phase >> at) & 1u, abort_flag, p.status,
                                             kFlagProducer)))
        break;
      phase ^= 1u << at;
      const int dirty = (16 - rem % 16) % 16;  // other rows inside the last MMA
      uint4* base = reinterpret_cast<uint4*>(smem + at * kStageBytes);
      for (int i = lane; i < dirty * 8 * 4; i += 32) {
        const int box = i / (dirty * 8), j = i - box * dirty * 8;
        base[box * (kBox / 16) + rem * 8 + j] = make_uint4(0, 0, 0, 0);
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(mapa_shared(smem_addr(&full[at]), 0));
    }
  } else {
    // -------------------------------------------------------------- epilogue
    const int q = warp & 3;  // TMEM lane quadrant of this warp
    int acc = 0;
    uint32_t acc_phase = 0;
    float* slot = p.sums + (int64_t)blockIdx.x * kSumFloats;  // WGRAD
    auto release = [&]() {  // the accumulator is read; on to the other one
      tc_fence_before();
      mbar_arrive_cluster(mapa_shared(smem_addr(&tempty[acc]), 0));
      acc ^= 1;
      if (acc == 0) acc_phase ^= 1u;
    };
    int staged = 0;  // WGRAD: the staging block in turn
    for (;;) {
      const PairTile t = read_tile(kFlagEpilogue);
      if (t.e < 0) break;
      const bool none = t.nk == 0;
      const int n_drains = MODE == kWgrad ? drains(t.nk) : 1;
      bool ok = true;
      for (int dr = 0; MODE == kWgrad && dr + 1 < n_drains; ++dr) {  // all but the last
        ok = warp_wait(&tfull[acc], acc_phase, kFlagEpilogue, false);
        if (!ok) break;
        tc_fence_after();
        for (int c0 = 0; c0 < kPair && t.n0 + c0 < p.n_in; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kPair) + c0, v);
          tmem_ld_wait();
          add_drained(slot, c0, q * 32 + lane, dr == 0, false, v);
        }
        release();
      }
      if (!ok) break;
      if (!none) {
        if (!warp_wait(&tfull[acc], acc_phase, kFlagEpilogue, false)) break;
        tc_fence_after();
      }
      const uint32_t tb = tmem_base + ((uint32_t)(q * 32) << 16) + (uint32_t)(acc * kPair);
      if (MODE == kWgrad) {
        // 32 rows x 64 columns at a time: rounded, staged in the 128-byte
        // swizzle TMA expects, stored by TMA (which cuts off what lies behind
        // the matrix). Stores straight from registers touch 32 rows per
        // instruction and bound the kernel when segments are short.
        const int row = t.m0 + (int)rank * 128 + q * 32;
        for (int c0 = 0; c0 < kPair && t.n0 + c0 < p.n_in && row < p.n_w; c0 += 64) {
          uint8_t* buf = more + (q * 2 + staged) * kStoreBytes;
          uint32_t v[4][16];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (none) {
#pragma unroll
              for (int j = 0; j < 16; ++j) v[i][j] = 0u;
            } else {
              tmem_ld16(tb + c0 + i * 16, v[i]);
            }
          }
          if (!none) tmem_ld_wait();
          if (n_drains > 1) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
              add_drained(slot, c0 + i * 16, q * 32 + lane, false, true, v[i]);
          }
          // the store before the last has read its block
          if (lane == 0) asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const float* f = reinterpret_cast<const float*>(&v[i >> 1][(i & 1) * 8]);
            *reinterpret_cast<uint4*>(buf + lane * 128 + ((i ^ (lane & 7)) << 4)) =
                make_uint4(pack16(f[0], f[1], p.fp16), pack16(f[2], f[3], p.fp16),
                           pack16(f[4], f[5], p.fp16), pack16(f[6], f[7], p.fp16));
          }
          asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
          __syncwarp();
          if (lane == 0) {
            tma_store_3d(&tm_c, buf, t.n0 + c0, row, t.e);
            asm volatile("cp.async.bulk.commit_group;" ::: "memory");
          }
          staged ^= 1;
        }
      } else if (GLU) {
        // lanes 0-15: gate rows, 16-31: up rows of 16 columns of Y
        const int col = t.m0 + (int)rank * 64 + q * 16 + (lane & 15);
        const bool live = col < p.n_out;
        const int wrow = (lane < 16 ? 0 : p.n_out) + col;  // this lane's weight row
        const float bias = p.bias && live ? __ldg(p.bias + (int64_t)t.e * p.n_w + wrow) : 0.0f;
        for (int c0 = 0; c0 < t.rows; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(tb + c0, v);
          tmem_ld_wait();
          float* f = reinterpret_cast<float*>(v);
#pragma unroll
          for (int j = 0; j < 16; ++j) f[j] += bias;
          if (p.z && live) {
            store_rows<16>(p.z, (int64_t)(t.row0 + c0) * p.n_w + wrow, p.n_w, t.rows - c0, f,
                           false, p.fp16);
          }
          float g[8], u[8];  // 8 of the 16 rows: the lower half's first 8, the upper's last
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float other = __shfl_xor_sync(0xffffffffu, lane < 16 ? f[8 + j] : f[j], 16);
            g[j] = lane < 16 ? f[j] : other;
            u[j] = lane < 16 ? other : f[8 + j];
          }
          swiglu<8, F32>(g, u);
          if (live) finish_rows<8, F32>(p, t, col, c0 + (lane >> 4) * 8, g);
        }
      } else {
        const int col = t.m0 + (int)rank * 128 + q * 32 + lane;
        const bool live = col < p.cols;
        const float bias =
            MODE == kFwd && p.bias && live ? __ldg(p.bias + (int64_t)t.e * p.n_w + col) : 0.0f;
        for (int c0 = 0; c0 < t.rows; c0 += 16) {
          uint32_t v[16];
          tmem_ld16(tb + c0, v);
          tmem_ld_wait();
          float* f = reinterpret_cast<float*>(v);
          if (!live) continue;
          if (MODE == kDgrad) {
            store_rows<16>(p.out, (int64_t)(t.row0 + c0) * p.n_in + col, p.n_in, t.rows - c0, f,
                           false, p.fp16);
            continue;
          }
          if (MODE == kFwd) {
#pragma unroll
            for (int j = 0; j < 16; ++j) f[j] += bias;
            if (p.z)
              store_rows<16>(p.z, (int64_t)(t.row0 + c0) * p.n_w + col, p.n_w, t.rows - c0, f,
                             false, p.fp16);
            activate<16, F32>(p.act, f);
            finish_rows<16, F32>(p, t, col, c0, f);
          }
        }
      }
      if (!none) release();
    }
    if (MODE == kWgrad && lane == 0) asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync();  // both CTAs done with TMEM and with each other's memory
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

template <int MODE, bool GLU, bool F32>
cudaError_t run_pairs(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& tc,
                      const LinParams& p, cudaStream_t st) {
  // Per device: the shared-memory attribute and the number of CTA pairs that
  // can be resident at once (a pair needs two SMs of one GPC).
  static PerDevice pairs;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 2;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.blockDim = dim3(PairMem<MODE>::kBlock);
  cfg.dynamicSmemBytes = PairMem<MODE>::kBytes;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int resident = 0;
  cudaError_t err = per_device(pairs, &resident, [&cfg](int* v) {
    cudaError_t e =
        cudaFuncSetAttribute(linear_pair_kernel<MODE, GLU, F32>,
                             cudaFuncAttributeMaxDynamicSharedMemorySize, PairMem<MODE>::kBytes);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t probe = cfg;
    probe.gridDim = dim3((unsigned)(device_sm_count() & ~1));
    int clusters = 0;
    e = cudaOccupancyMaxActiveClusters(&clusters, linear_pair_kernel<MODE, GLU, F32>, &probe);
    if (e != cudaSuccess) return e;
    if (clusters < 1) return cudaErrorInvalidConfiguration;
    *v = clusters < device_sm_count() / 2 ? clusters : device_sm_count() / 2;
    return cudaSuccess;
  });
  if (err != cudaSuccess) return err;
  cfg.gridDim = dim3((unsigned)(2 * resident));
  return cudaLaunchKernelEx(&cfg, linear_pair_kernel<MODE, GLU, F32>, ta, tb, tc, p);
}

}  // namespace

cudaError_t launch_linear_pair(int mode, const LinParams& base, const void* a, const void* b,
                               cudaStream_t st) {
  LinParams p = base;
  const uint64_t R = p.rows, E = p.E;
  // words of the status area, zero at the call's start; a launch each
  p.next_tile = reinterpret_cast<int*>(p.status) + kTileCounterWord + mode;
  const bool glu = mode == kFwd && p.act == BEAM_MOE_ACT_SWIGLU;
  CUtensorMap ta, tb, tc;
  cudaError_t err;
  if (mode == kWgrad) {
    p.m_blk = (p.n_w + kPair - 1) / kPair;
    p.n_blk = (p.n_in + kPair - 1) / kPair;
    err = encode_tmap_2d_bf16(&ta, a, p.n_w, R, 64, 64);
    if (err == cudaSuccess) err = encode_tmap_2d_bf16(&tb, b, p.n_in, R, 64, 64);
    if (err == cudaSuccess) err = encode_tmap_3d_bf16(&tc, p.out, p.n_in, p.n_w, E, 64, 32);
    if (err != cudaSuccess) return err;
    return run_pairs<kWgrad, false, false>(ta, tb, tc, p, st);
  }
  // a: rows of X or dZ, b: the weights; on pairs the weights are the A operand
  const uint64_t kc = mode == kFwd ? p.n_in : p.n_w;
  p.nk = (int)((kc + kK - 1) / kK);
  p.m_blk = glu ? (p.n_out + 127) / 128 : (p.cols + kPair - 1) / kPair;
  if (glu)
    err = encode_tmap_glu_bf16(&ta, b, p.n_in, p.n_out, E);
  else
    err = encode_tmap_3d_bf16(&ta, b, p.n_in, p.n_w, E, 64, mode == kDgrad ? 64 : 128);
  if (err == cudaSuccess) err = encode_tmap_2d_bf16(&tb, a, kc, R, 64, 128);
  if (err == cudaSuccess) err = encode_tmap_2d_bf16(&tc, a, kc, R, 64, 64);
  if (err != cudaSuccess) return err;
  if (mode == kDgrad) return run_pairs<kDgrad, false, false>(ta, tb, tc, p, st);
  if (p.out32)
    return glu ? run_pairs<kFwd, true, true>(ta, tb, tc, p, st)
               : run_pairs<kFwd, false, true>(ta, tb, tc, p, st);
  return glu ? run_pairs<kFwd, true, false>(ta, tb, tc, p, st)
             : run_pairs<kFwd, false, false>(ta, tb, tc, p, st);
}

}  // namespace beam
