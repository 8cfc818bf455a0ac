// linear.cuh - shared by the linear operator's kernels (linear.cu,
// linear_pair.cu): parameters, the experts' segments, descriptors, TMA forms
// and the activations.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "sm100.cuh"

namespace beam {
namespace lin {

enum Mode { kFwd, kDgrad, kWgrad };

constexpr int kMaxE = 512;
constexpr int kM = 128;       // rows of D per tile
constexpr int kK = 64;        // contraction per pipeline stage
constexpr int kRowGroup = 16; // row blocks that share a sweep over the columns
constexpr int kBox = 64 * kK * 2;  // bytes of a 64 x 64 box

struct LinParams {
  const int32_t* offsets;  // [E + 1] or NULL
  int E, rows;
  int n_in, n_out, n_w;    // n_w: weight rows per expert (2 n_out for swiglu)
  int cols;                // columns of D that exist (FWD n_out, else n_in)
  int nk;                  // contraction steps (FWD, DGRAD)
  int n_blk, m_blk;        // column tiles; row tiles of dW_e (WGRAD)
  int box_a;               // rows per box of the row operand (FWD, DGRAD)
  int a_stage, stages;     // split: bytes of the row operand per stage, stages
  int parts;               // split: CTAs per tile
  int act, fp16, out32;
  const float* bias;       // [E][n_w] or NULL
  const void* residual;    // [rows][n_out] or NULL
  void* z;                 // [rows][n_w] or NULL
  void* out;
  unsigned* status;
  int clear_status;        // the launch clears the status area (the first of a call)
  int* next_tile;          // CTA pairs: counter of the tiles handed out
  float* sums;             // WGRAD: kSumFloats per CTA, where rows > kDrain kK
};

// The tensor cores cut off as they add to an FP32 accumulator, so a sum whose
// terms have one sign comes out too small by up to 6.8e-9 of itself per term
// (measured; where signs mix 1.6e-9 of the magnitudes and less): fp16's half step,
// 2^-11, at 72,000 rows. dW's sums over rows are therefore taken out of the
// accumulators every 256 steps (16384 rows, 1.1e-4) and added in FP32: one-CTA
// tiles and pairs in a slot of the workspace per CTA, while the other accumulator
// fills; split tiles in registers. 65536 x 2560 x 2560, both products: 1288 us
// without, 1296 every 512 steps, 1311 every 256, 1313 every 128, 1330 every 64.
constexpr int kDrain = 256;            // contraction steps
constexpr int kSumFloats = 128 * 256;  // a CTA's accumulator

__device__ __forceinline__ int drains(int steps) { return (steps + kDrain - 1) / kDrain; }

// v (column c on, row r of the CTA's accumulator) with what the earlier drains
// of the tile left there; kept there unless this one is the last.
__device__ __forceinline__ void add_drained(float* slot, int c, int r, bool first, bool last,
                                            uint32_t (&v)[16]) {
  float* s = slot + c * kM + r;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    float f = __uint_as_float(v[j]);
    if (!first) f += s[j * kM];
    if (last) v[j] = __float_as_uint(f);
    else s[j * kM] = f;
  }
}

constexpr int kStatusWords = 64;

// The status word and the counters of a call, by one CTA of its first launch.
// (The launches after it find them clear; a wait of this launch that gives up
// sets its bit a second from now.)
__device__ __forceinline__ void clear_status_area(const LinParams& p) {
  if (threadIdx.x < kStatusWords) p.status[threadIdx.x] = 0;
}

// ------------------------------------------------------------- the segments
// Whatever the offsets hold, no row has two experts and no row lies outside the
// buffers: expert e's rows are those in [offsets[e], offsets[e + 1]), cut off at
// the rows there are, that lie behind every expert's before it. Offsets that
// ascend (`ordered`) need no look at the experts before; others are walked one
// by one. Row blocks are then at most rows / BLOCK + min(E, rows), which is what
// grids and the workspace are sized for.
__device__ __forceinline__ void cut_off(const LinParams& p, int e, int& a, int& b) {
  a = 0;
  b = p.rows;
  if (p.offsets) {
    a = min(max(__ldg(p.offsets + e), 0), p.rows);
    b = min(max(__ldg(p.offsets + e + 1), 0), p.rows);
  }
}

// The rows [lo, lo + cnt) that expert e gets of its [a, b), and where the rows
// of the experts up to it end.
__device__ __forceinline__ void take_segment(int a, int b, int& end, int& lo, int& cnt) {
  lo = max(a, end);
  cnt = max(b - lo, 0);
  if (b > a) end = max(end, b);
}

__device__ __forceinline__ void segment(const LinParams& p, int e, bool ordered, int& lo,
                                        int& cnt) {
  int a, b, end = 0;
  if (!ordered)
#pragma unroll 1
    for (int i = 0; i < e; ++i) {
      cut_off(p, i, a, b);
      take_segment(a, b, end, lo, cnt);
    }
  cut_off(p, e, a, b);
  take_segment(a, b, end, lo, cnt);
}

// Whether the offsets ascend; all threads of the CTA call it (a barrier).
__device__ __forceinline__ bool offsets_ordered(const LinParams& p) {
  bool bad = false;
  if (p.offsets)
    for (int e = threadIdx.x; e < p.E; e += blockDim.x) {
      int a, b;
      cut_off(p, e, a, b);
      bad |= b < a;
    }
  return !__syncthreads_or(bad);
}

// In shared memory: first row and row count of every expert (unless lo is
// NULL), and the prefix of its BLOCK-row blocks (rb[E]: all of them). THREADS
// threads call it; returns whether the offsets are ordered.
struct Segments {
  int* lo;
  int* cnt;
  int* rb;
};

template <int THREADS, int BLOCK>
__device__ __forceinline__ bool build_segments(const LinParams& p, const Segments& s, int* scratch) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  constexpr int PER = (kMaxE + THREADS - 1) / THREADS;
  int blocks[PER], sum = 0;
  bool bad = false;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    blocks[i] = 0;
    if (e < p.E) {
      int a, b;
      cut_off(p, e, a, b);
      bad |= b < a;
      if (s.lo) {
        s.lo[e] = a;
        s.cnt[e] = b - a;
      }
      blocks[i] = (b - a + BLOCK - 1) / BLOCK;
    }
    sum += blocks[i];
  }
  int inc = sum;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) scratch[warp] = inc;
  if (__syncthreads_or(bad)) {
    if (tid == 0) {
      int end = 0, run = 0;
#pragma unroll 1
      for (int e = 0; e < p.E; ++e) {
        int a, b, lo, cnt;
        cut_off(p, e, a, b);
        take_segment(a, b, end, lo, cnt);
        if (s.lo) {
          s.lo[e] = lo;
          s.cnt[e] = cnt;
        }
        s.rb[e] = run;
        run += (cnt + BLOCK - 1) / BLOCK;
      }
      s.rb[p.E] = run;
    }
    __syncthreads();
    return false;
  }
  int run = inc - sum;
  for (int w = 0; w < warp; ++w) run += scratch[w];
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int e = tid * PER + i;
    if (e < p.E) {
      s.rb[e] = run;
      run += blocks[i];
      if (e == p.E - 1) s.rb[p.E] = run;
    }
  }
  __syncthreads();
  return true;
}

// The expert whose row blocks hold block q (rb[0] <= q < rb[E]).
__device__ __forceinline__ int find_expert(const int* rb, int E, int q) {
  int a = 0, b = E;  // rb[a] <= q < rb[b]
  while (b - a > 1) {
    const int m = (a + b) >> 1;
    if (rb[m] <= q) a = m;
    else b = m;
  }
  return a;
}

// One lane of a converged warp, in the form the compiler knows to be one: the
// loops around it stay uniform, so that descriptors and addresses live in
// uniform registers. Issued from inside an `if (lane == 0)` each MMA cost the
// thread some 70 cycles of register moves, and a step more than its MMAs.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(one));
  return one != 0;
}

__device__ __forceinline__ int uniform(int v) { return __shfl_sync(0xffffffffu, v, 0); }

// -------------------------------------------------------------- descriptors
__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar,
                                            int32_t c0, int32_t c1, int32_t c2, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5}], [%2], %6;" ::"r"(smem_addr(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_addr(bar)), "r"(c0), "r"(c1), "r"(c2),
      "l"(policy)
      : "memory");
}

// MN-major operand, 128-byte swizzle: boxes of 64 (contraction) rows x 64
// elements, 8 KB apart (leading offset), rows in groups of 8 that lie 1 KB
// apart (stride offset). 16 contraction rows further: 2 KB.
__device__ __forceinline__ uint64_t smem_desc_mn_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(kBox >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1u << 46;
  d |= (uint64_t)2u << 61;
  return d;
}

// FP32 sums of bf16 or fp16 products, M x N; an operand is K-major or MN-major.
__device__ __forceinline__ uint32_t idesc_of(bool fp16, bool a_mn, bool b_mn, uint32_t M,
                                             uint32_t N) {
  const uint32_t fmt = fp16 ? 0u : 1u;
  return (1u << 4) | (fmt << 7) | (fmt << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | ((N >> 3) << 17) | ((M >> 4) << 24);
}

// ----------------------------------------------------------------- epilogue
// e^-z. __expf is documented to err by 2 + 1.17 |z| steps: 25 at z = -20. That is
// far below a half step of a 16-bit result, where it is used (FULL false). FULL is
// for FP32 results, and for forms that finish few values: with t the FP32 nearest
// to -z log2 e, e^-z = 2^t e^r, r = -z - t ln 2 (ln 2 in two parts, after Cody and
// Waite), and e^r is 1 + r to first order (r < 1e-5). Used for all results it cost
// 5 % where a short contraction leaves the epilogue as the bound (16384 x 512 x
// 5120, swiglu: 243 and 256 us); expf and a full division there 449 us. z is held
// to +-88, beyond which the quotients below are 0 and 1 either way.
template <bool FULL>
__device__ __forceinline__ float exp_neg(float z) {
  if (!FULL) return __expf(-z);
  z = fminf(fmaxf(z, -88.0f), 88.0f);
  const float t = z * -1.44269504088896341f;
  const float r = fmaf(t, 1.90465429995776787e-9f, fmaf(t, -0.693147182464599609f, -z));
  float p;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
  return fmaf(p, r, p);
}

template <bool FULL = false>
__device__ __forceinline__ float sigmoid_f(float z) {
  return __fdividef(1.0f, 1.0f + exp_neg<FULL>(z));
}

// 1/2 (1 + erf(z / sqrt 2)) as a complement: relative accuracy down the tail.
__device__ __forceinline__ float normal_cdf(float z) {
  return 0.5f * erfcf(z * -0.70710678118654752f);
}

// 1/2 (1 + tanh(a)) = sigmoid(2 a) for a = sqrt(2/pi) (z + 0.044715 z^3).
template <bool FULL = false>
__device__ __forceinline__ float tanh_gate(float z) {
  return sigmoid_f<FULL>(1.59576912160573071f * fmaf(0.044715f * z * z, z, z));
}

template <bool FULL>
__device__ __forceinline__ float silu_f(float z) {
  return __fdividef(z, 1.0f + exp_neg<FULL>(z));
}

// act over N values. The choice is made once for all of them and the longer
// formulas stay rolled: unrolled inside a switch per value they filled the
// instruction cache and bounded the kernel (16384 x 5120 x 5120, act none:
// 885 us against 590).
template <int N, bool FULL>
__device__ __forceinline__ void activate(int act, float* z) {
  switch (act) {
    case BEAM_MOE_ACT_RELU:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = z[j] < 0.0f ? 0.0f : z[j];  // a NaN stays one
      break;
    case BEAM_MOE_ACT_GELU:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] *= normal_cdf(z[j]);
      break;
    case BEAM_MOE_ACT_GELU_TANH:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] *= tanh_gate<FULL>(z[j]);
      break;
    case BEAM_MOE_ACT_SILU:
#pragma unroll
      for (int j = 0; j < N; ++j) z[j] = silu_f<FULL>(z[j]);
      break;
  }
}

// z = silu(z) u over N values.
template <int N, bool FULL>
__device__ __forceinline__ void swiglu(float* z, const float* u) {
#pragma unroll
  for (int j = 0; j < N; ++j) z[j] = silu_f<FULL>(z[j]) * u[j];
}

__device__ __forceinline__ uint32_t pack16(float a, float b, bool fp16) {
  if (fp16) {
    const __half2 h = __floats2half2_rn(a, b);
    return *reinterpret_cast<const uint32_t*>(&h);
  }
  const __nv_bfloat162 h = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack16(uint32_t v, bool fp16) {
  return fp16 ? __half22float2(*reinterpret_cast<const __half2*>(&v))
              : __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(&v));
}

__device__ __forceinline__ float load1(const void* p, int64_t at, bool f32, bool fp16) {
  if (f32) return static_cast<const float*>(p)[at];
  return fp16 ? __half2float(static_cast<const __half*>(p)[at])
              : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[at]);
}

__device__ __forceinline__ void store1(void* p, int64_t at, float v, bool f32, bool fp16) {
  if (f32) static_cast<float*>(p)[at] = v;
  else if (fp16) static_cast<__half*>(p)[at] = __float2half_rn(v);
  else static_cast<__nv_bfloat16*>(p)[at] = __float2bfloat16_rn(v);
}

__device__ __forceinline__ void unpack8(const uint4& u, float* v, bool fp16) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = unpack16(w[i], fp16);
    v[2 * i] = f.x;
    v[2 * i + 1] = f.y;
  }
}

__device__ __forceinline__ void store8(uint16_t* p, int64_t at, const float* v, bool fp16) {
  *reinterpret_cast<uint4*>(p + at) =
      make_uint4(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16), pack16(v[4], v[5], fp16),
                 pack16(v[6], v[7], fp16));
}

// 4 consecutive elements at p (element index at, a multiple of 4).
__device__ __forceinline__ void store4(void* p, int64_t at, const float* v, bool f32, bool fp16) {
  if (f32)
    reinterpret_cast<float4*>(static_cast<float*>(p) + at)[0] = make_float4(v[0], v[1], v[2], v[3]);
  else
    reinterpret_cast<uint2*>(static_cast<uint16_t*>(p) + at)[0] =
        make_uint2(pack16(v[0], v[1], fp16), pack16(v[2], v[3], fp16));
}

__device__ __forceinline__ void load4(const void* p, int64_t at, float* v, bool f32, bool fp16) {
  if (f32) {
    const float4 f = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const uint2 u = *reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(p) + at);
    const float2 a = unpack16(u.x, fp16), b = unpack16(u.y, fp16);
    v[0] = a.x; v[1] = a.y; v[2] = b.x; v[3] = b.y;
  }
}

}  // namespace lin

// The product of one mode on CTA pairs (linear_pair.cu): a, b and p.out as
// for the one-CTA kernel.
cudaError_t launch_linear_pair(int mode, const lin::LinParams& p, const void* a, const void* b,
                               cudaStream_t st);

}  // namespace beam
