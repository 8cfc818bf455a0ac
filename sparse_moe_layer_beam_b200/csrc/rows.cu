// rows.cu - token rows sorted by expert and back, and the gradients of both.
//
//   permute           assignment a = t K + k of expert e goes to row
//                       pos[a] = offsets[e] + |{a' < a : ids[a'] = e}|
//                     (a stable counting sort), xp[pos[a]] = x[t].
//   combine           out[t] = sum_k w[t,k] y[pos[t,k]], k ascending.
//   permute backward  dx[t]  = sum_k dxp[pos[t,k]]: the combine with w = 1.
//   combine backward  dy[pos[t,k]] = w[t,k] dout[t],
//                     dw[t,k] = <dout[t], y[pos[t,k]]>.
//
// An assignment whose id lies outside [0, E) has no row (pos -1) and adds
// nothing anywhere. Sums are chains of FP32 FMAs in a fixed order, rounded to
// a 16-bit output once; nothing depends on the order of atomics (the shared
// memory counters below count, and a count has no order).
//
// All of it is bound by HBM: each row is read or written once.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "ops.h"

namespace beam {
namespace {

constexpr int kMaxE = 512;       // experts
constexpr int kMaxK = 32;        // experts per token
constexpr int kSortChunk = 1024; // assignments per chunk of the three-launch sort
// Up to this many assignments every CTA of the copy counts all ids itself
// (32 KB of L2 reads each) instead of two launches before it.
constexpr int kOneLaunch = 8192;

// ------------------------------------------------------------ element types
template <class T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <class T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32<__half>(float v) { return __float2half_rn(v); }

// N consecutive elements as they sit in memory; loaded and stored in 16-byte
// pieces when N is 8, element by element when it is 1.
template <class T, int N>
struct Pack {
  T v[N];
};

template <class T, int N>
__device__ __forceinline__ Pack<T, N> load_pack(const T* p) {
  Pack<T, N> r;
  if constexpr (N * sizeof(T) >= 16) {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4*>(&r)[i] = __ldg(reinterpret_cast<const uint4*>(p) + i);
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) r.v[i] = p[i];
  }
  return r;
}

template <class T, int N>
__device__ __forceinline__ void store_pack(T* p, const Pack<T, N>& r) {
  if constexpr (N * sizeof(T) >= 16) {
#pragma unroll
    for (int i = 0; i < (int)(N * sizeof(T) / 16); ++i)
      reinterpret_cast<uint4*>(p)[i] = reinterpret_cast<const uint4*>(&r)[i];
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = r.v[i];
  }
}

// ------------------------------------------------------------------ the sort
// Stable rank of every assignment inside its chunk of 1024, and the chunk's
// count of every expert. Warps hold consecutive assignments: a warp's lanes
// with the same expert find each other by match, and the 32 warps' counts are
// summed in warp order.
__global__ void __launch_bounds__(kSortChunk) sort_count_kernel(const int32_t* __restrict__ ids,
                                                                int64_t A, int E,
                                                                uint16_t* __restrict__ rank,
                                                                int32_t* __restrict__ cnt) {
  __shared__ uint16_t w_cnt[32][kMaxE];
  cudaTriggerProgrammaticLaunchCompletion();  // the scan may come on and wait
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  for (int i = lane; i < E; i += 32) w_cnt[warp][i] = 0;
  __syncwarp();
  const int64_t a = (int64_t)blockIdx.x * kSortChunk + tid;
  int e = a < A ? __ldg(ids + a) : -1;
  if (e < 0 || e >= E) e = -1;
  const unsigned same = __match_any_sync(0xffffffffu, e);
  const int before = __popc(same & ((1u << lane) - 1u));
  if (e >= 0 && before == 0) w_cnt[warp][e] = (uint16_t)__popc(same);
  __syncthreads();
  for (int i = tid; i < E; i += kSortChunk) {
    int run = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const int c = w_cnt[w][i];
      w_cnt[w][i] = (uint16_t)run;
      run += c;
    }
    cnt[(size_t)blockIdx.x * E + i] = run;
  }
  __syncthreads();
  if (a < A) rank[a] = e >= 0 ? (uint16_t)(w_cnt[warp][e] + before) : (uint16_t)0;
}

// Exclusive scan over n <= blockDim values, one per thread (all threads call).
__device__ __forceinline__ int block_scan(int v, int* warp_tot, int* total) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nw = blockDim.x >> 5;
  int inc = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int n = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += n;
  }
  if (lane == 31) warp_tot[warp] = inc;
  __syncthreads();
  if (warp == 0) {
    const int w = lane < nw ? warp_tot[lane] : 0;
    int wi = w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int n = __shfl_up_sync(0xffffffffu, wi, o);
      if (lane >= o) wi += n;
    }
    if (lane < nw) warp_tot[lane] = wi - w;
    if (lane == 31) *total = wi;
  }
  __syncthreads();
  return warp_tot[warp] + inc - v;
}

// offsets, and cnt turned from counts into the first row of (chunk, expert).
// A CTA turns 16 experts' columns; each reads all counts once for the totals
// (128 KB from L2 at 131072 assignments to 256 experts: 3 us, where one CTA for
// everything took 10).
constexpr int kScanExperts = 16;

__global__ void __launch_bounds__(1024) sort_scan_kernel(const int32_t* __restrict__ cnt,
                                                         int32_t* __restrict__ base, int nchunks,
                                                         int E, int32_t* __restrict__ offsets) {
  __shared__ int part[1024];
  __shared__ int s_off[kMaxE];
  __shared__ int warp_tot[32], total;
  const int tid = threadIdx.x;
  cudaTriggerProgrammaticLaunchCompletion();  // so may the copy
  cudaGridDependencySynchronize();            // the counts are there
  {
    // thread (j, e) sums the j-th part of expert e's chunks
    const int per_e = 1024 / E;  // E <= 512
    const int e = tid % E, j = tid / E;
    const int len = (nchunks + per_e - 1) / per_e;
    const int c0 = min(nchunks, j * len), c1 = min(nchunks, c0 + len);
    int sum = 0;
    if (j < per_e)
#pragma unroll 8
      for (int c = c0; c < c1; ++c) sum += __ldg(cnt + (size_t)c * E + e);
    part[tid] = sum;
    __syncthreads();
    int tot = 0;
    if (tid < E)
      for (int q = 0; q < per_e; ++q) tot += part[q * E + tid];
    const int off = block_scan(tid < E ? tot : 0, warp_tot, &total);
    if (tid < E) s_off[tid] = off;
    if (blockIdx.x == 0) {
      if (tid < E) offsets[tid] = off;
      if (tid == 0) offsets[E] = total;
    }
    __syncthreads();
  }
  // thread (j, e) turns the j-th of 64 parts of one of this CTA's experts
  const int e = blockIdx.x * kScanExperts + tid % kScanExperts, j = tid / kScanExperts;
  const int len = (nchunks + 63) / 64;
  const int c0 = min(nchunks, j * len), c1 = min(nchunks, c0 + len);
  int sum = 0;
  if (e < E)
#pragma unroll 4
    for (int c = c0; c < c1; ++c) sum += __ldg(cnt + (size_t)c * E + e);
  part[tid] = sum;
  __syncthreads();
  if (e < E) {
    int run = s_off[e];
    for (int q = 0; q < j; ++q) run += part[q * kScanExperts + tid % kScanExperts];
#pragma unroll 4
    for (int c = c0; c < c1; ++c) {
      const int v = __ldg(cnt + (size_t)c * E + e);
      base[(size_t)c * E + e] = run;
      run += v;
    }
  }
}

constexpr int kCopyThreads = 256;

// Copies x[t] to its rows for `tpb` tokens per CTA, a slice of the row per
// blockIdx.y. V: the unit of the copy (16, 4 or 2 bytes; nv of them per row).
// ONE: the positions are counted here, from all ids (A <= kOneLaunch).
template <class V, bool ONE, int U>
__global__ void __launch_bounds__(kCopyThreads)
    permute_rows_kernel(const V* __restrict__ x, int nv, int64_t T, int K, int E, int tpb,
                        const int32_t* __restrict__ ids, const uint16_t* __restrict__ rank,
                        const int32_t* __restrict__ base, int32_t* __restrict__ pos,
                        int32_t* __restrict__ offsets, V* __restrict__ xp) {
  __shared__ int s_pos[kCopyThreads];
  const int tid = threadIdx.x;
  const int64_t t0 = (int64_t)blockIdx.x * tpb;
  const int nt = (int)min((int64_t)tpb, T - t0);
  const int64_t a0 = t0 * K;
  const int na = nt * K;  // <= kCopyThreads
  if constexpr (ONE) {
    __shared__ int s_tot[kMaxE], s_bef[kMaxE];
    __shared__ int warp_tot[32], total;
    const int A = (int)T * K;
    for (int i = tid; i < kMaxE; i += kCopyThreads) s_tot[i] = s_bef[i] = 0;
    __syncthreads();
    for (int a = tid; a < A; a += kCopyThreads) {
      const int e = __ldg(ids + a);
      if (e >= 0 && e < E) {
        atomicAdd(&s_tot[e], 1);
        if (a < a0) atomicAdd(&s_bef[e], 1);
      }
    }
    int e = -1;
    if (tid < na) {
      e = __ldg(ids + a0 + tid);
      if (e < 0 || e >= E) e = -1;
      s_pos[tid] = e;
    }
    __syncthreads();
    const int v0 = s_tot[2 * tid], v1 = s_tot[2 * tid + 1];
    const int off = block_scan(v0 + v1, warp_tot, &total);
    if (blockIdx.x == 0 && blockIdx.y == 0) {
      if (2 * tid < E) offsets[2 * tid] = off;
      if (2 * tid + 1 < E) offsets[2 * tid + 1] = off + v0;
      if (tid == 0) offsets[E] = total;
    }
    s_bef[2 * tid] += off;
    s_bef[2 * tid + 1] += off + v0;
    int p = -1;
    if (e >= 0) {
      p = 0;
      for (int j = 0; j < tid; ++j) p += s_pos[j] == e;
    }
    __syncthreads();
    if (tid < na) {
      if (e >= 0) p += s_bef[e];
      s_pos[tid] = p;
      if (blockIdx.y == 0) pos[a0 + tid] = p;
    }
  } else {
    cudaGridDependencySynchronize();  // the positions' bases are there
    if (tid < na) {
      const int64_t a = a0 + tid;
      const int e = __ldg(ids + a);
      const int p = e >= 0 && e < E
                        ? __ldg(base + (size_t)(a / kSortChunk) * E + e) + (int)__ldg(rank + a)
                        : -1;
      s_pos[tid] = p;
      if (blockIdx.y == 0) pos[a] = p;
    }
  }
  __syncthreads();
  // U units per thread and pass, loaded together
  const int step = gridDim.y * kCopyThreads;
  for (int i = 0; i < nt; ++i) {
    const V* src = x + (t0 + i) * nv;
    for (int v = blockIdx.y * kCopyThreads + tid; v < nv; v += U * step) {
      V d[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u * step < nv) d[u] = __ldg(src + v + u * step);
      for (int k = 0; k < K; ++k) {
        const int p = s_pos[i * K + k];
        if (p < 0) continue;
        V* dst = xp + (size_t)p * nv + v;
#pragma unroll
        for (int u = 0; u < U; ++u)
          if (v + u * step < nv) dst[u * step] = d[u];
      }
    }
  }
}

// --------------------------------------------------- combine and its backward
constexpr int kRowThreads = 128;

// out[t] = sum_k w[t,k] y[pos[t,k]] (w NULL: 1). A CTA per token and slice of
// the row; U packs of N elements per thread and pass, the loads of eight slots
// in flight at once (four, where packs are single elements). 4096 tokens x
// 5120 bf16 x 8 slots: 61 us, 5.75 TB/s; FP32 rows 106 us, 6.7 TB/s. (A warp
// per piece of a row, walking pieces without barriers: 65 to 87 us.)
template <class O, class Y, int N, int U>
__global__ void __launch_bounds__(kRowThreads)
    combine_rows_kernel(const Y* __restrict__ y, int H, int K, int64_t rows,
                        const int32_t* __restrict__ pos, const float* __restrict__ w,
                        O* __restrict__ out) {
  __shared__ int s_pos[kMaxK];
  __shared__ float s_w[kMaxK];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  if (tid < K) {
    const int p = pos[t * K + tid];
    s_pos[tid] = p < rows ? p : -1;
    s_w[tid] = w ? w[t * K + tid] : 1.0f;
  }
  __syncthreads();
  const int nv = H / N, step = gridDim.y * kRowThreads;
  for (int v = blockIdx.y * kRowThreads + tid; v < nv; v += U * step) {
    float acc[U][N];
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int i = 0; i < N; ++i) acc[u][i] = 0.0f;
#pragma unroll(N == 8 ? 8 : 4)
    for (int k = 0; k < K; ++k) {
      const int p = s_pos[k];
      if (p < 0) continue;
      const Y* row = y + (size_t)p * H + (size_t)v * N;
      const float wk = s_w[k];
      Pack<Y, N> r[U];
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (v + u * step < nv) r[u] = load_pack<Y, N>(row + (size_t)u * step * N);
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int i = 0; i < N; ++i) acc[u][i] = fmaf(wk, to_f32(r[u].v[i]), acc[u][i]);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (v + u * step >= nv) break;
      Pack<O, N> o;
#pragma unroll
      for (int i = 0; i < N; ++i) o.v[i] = from_f32<O>(acc[u][i]);
      store_pack<O, N>(out + (size_t)t * H + (size_t)(v + u * step) * N, o);
    }
  }
}

// dy rows and dw of one token's slots, S of them at a time (groups of S from
// blockIdx.y on, gridDim.y groups apart), U packs of N elements per thread and
// pass. A thread's products are added in column order, a warp's by a shuffle
// tree, the warps' in order: the sum has one order whatever runs when.
// 4096 tokens x 5120 bf16 x 8 slots: 122 us, 5.85 TB/s (one slot at a time 145
// us, four 136 us, 256 threads 129 us; FP32 rows want 256 threads).
template <class O, class Y, int N, int S, int U, int THREADS>
__global__ void __launch_bounds__(THREADS)
    combine_bwd_kernel(const O* __restrict__ dout, const Y* __restrict__ y, int H, int K,
                       int64_t rows, const int32_t* __restrict__ pos,
                       const float* __restrict__ w, Y* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float s_sum[kMaxK + S][THREADS / 32];
  __shared__ int s_pos[kMaxK + S];
  __shared__ float s_w[kMaxK + S];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  if (tid < kMaxK + S) {
    const int p = tid < K ? pos[t * K + tid] : -1;
    s_pos[tid] = p < rows ? p : -1;
    s_w[tid] = w && tid < K ? w[t * K + tid] : 1.0f;
  }
  __syncthreads();
  const int nv = H / N;
  const O* d = dout + (size_t)t * H;
  for (int k = S * blockIdx.y; k < K; k += S * gridDim.y) {
    int p[S];
    float wk[S], sum[S];
#pragma unroll
    for (int j = 0; j < S; ++j) {
      p[j] = s_pos[k + j];
      wk[j] = s_w[k + j];
      sum[j] = 0.0f;
    }
    for (int v = tid; v < nv; v += U * THREADS) {
      Pack<Y, N> r[S][U];
      Pack<O, N> g[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t off = (size_t)(v + u * THREADS) * N;
        if (v + u * THREADS >= nv) break;
        if (dw) {
#pragma unroll
          for (int j = 0; j < S; ++j)
            if (p[j] >= 0) r[j][u] = load_pack<Y, N>(y + (size_t)p[j] * H + off);
        }
        g[u] = load_pack<O, N>(d + off);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const size_t off = (size_t)(v + u * THREADS) * N;
        if (v + u * THREADS >= nv) break;
#pragma unroll
        for (int j = 0; j < S; ++j) {
          if (p[j] < 0) continue;
          if (dw) {
#pragma unroll
            for (int i = 0; i < N; ++i)
              sum[j] = fmaf(to_f32(g[u].v[i]), to_f32(r[j][u].v[i]), sum[j]);
          }
          if (dy) {
            Pack<Y, N> o;
#pragma unroll
            for (int i = 0; i < N; ++i) o.v[i] = from_f32<Y>(wk[j] * to_f32(g[u].v[i]));
            store_pack<Y, N>(dy + (size_t)p[j] * H + off, o);
          }
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int j = 0; j < S; ++j) {
#pragma unroll
        for (int o = 16; o; o >>= 1) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], o);
        if ((tid & 31) == 0) s_sum[k + j][tid >> 5] = sum[j];
      }
    }
  }
  if (dw) {
    __syncthreads();
    if (tid < K && tid / S % gridDim.y == blockIdx.y) {
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < THREADS / 32; ++i) sum += s_sum[tid][i];
      dw[t * K + tid] = sum;
    }
  }
}

// ------------------------------------------------------------------- launches
struct SortLayout {
  int nchunks;
  size_t rank, cnt, base, total;
};

SortLayout sort_layout(const beam_moe_rows_cfg& c, int64_t T) {
  SortLayout L;
  const int64_t A = T * c.top_k;
  L.nchunks = (int)((A + kSortChunk - 1) / kSortChunk);
  L.rank = 256;
  const size_t rank_bytes = ((size_t)A * 2 + 255) / 256 * 256;
  L.cnt = L.rank + rank_bytes;
  const size_t cnt_bytes = ((size_t)L.nchunks * c.n_experts * 4 + 255) / 256 * 256;
  L.base = L.cnt + cnt_bytes;
  L.total = A <= kOneLaunch ? 256 : L.base + cnt_bytes;
  return L;
}

template <class V>
cudaError_t run_permute(const beam_moe_rows_cfg& c, int64_t T, const void* x, const int32_t* ids,
                        void* xp, int32_t* pos, int32_t* offsets, char* ws, cudaStream_t st) {
  const SortLayout L = sort_layout(c, T);
  const int K = c.top_k, E = c.n_experts;
  const int64_t A = T * K;
  const int nv = (int)((size_t)c.width * dtype_bytes(c.dtype) / sizeof(V));
  const bool one = A <= kOneLaunch;
  // Positions at hand: a CTA per token (16384 tokens x 5120 to 8 experts each:
  // 257 us; 2, 8 and 16 tokens per CTA: 264, 278 and 302 us). Counted by every
  // CTA: about four CTAs per SM, at most 8 tokens (and 256 assignments) each.
  // With few tokens a row is cut into slices besides.
  const int64_t want = 4 * (int64_t)device_sm_count();
  int tpb = 1;
  if (one) {
    tpb = (int)(T / want < 1 ? 1 : T / want);
    if (tpb > 8) tpb = 8;
    if (tpb * K > kCopyThreads) tpb = kCopyThreads / K;
  }
  const int64_t gx = (T + tpb - 1) / tpb;
  int64_t gy = (want / 2 + gx - 1) / gx;
  const int most = (nv + kCopyThreads - 1) / kCopyThreads;
  if (gy > most) gy = most;
  if (gy < 1) gy = 1;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const V* xv = static_cast<const V*>(x);
  V* xpv = static_cast<V*>(xp);
  constexpr int U = sizeof(V) == 16 ? 1 : 4;
  if (one) {
    permute_rows_kernel<V, true, U><<<grid, kCopyThreads, 0, st>>>(
        xv, nv, T, K, E, tpb, ids, nullptr, nullptr, pos, offsets, xpv);
    return cudaGetLastError();
  }
  uint16_t* rank = reinterpret_cast<uint16_t*>(ws + L.rank);
  int32_t* cnt = reinterpret_cast<int32_t*>(ws + L.cnt);
  int32_t* base = reinterpret_cast<int32_t*>(ws + L.base);
  sort_count_kernel<<<L.nchunks, kSortChunk, 0, st>>>(ids, A, E, rank, cnt);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  // The scan and the copy are launched while the kernel before them still runs
  // and wait for its end on the device: no launch gaps (4096 tokens x 5120 71.7
  // us, 72.5 with them; 4000 x 1003 14.8 and 16.4).
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.stream = st;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  cfg.gridDim = dim3((unsigned)((E + kScanExperts - 1) / kScanExperts));
  cfg.blockDim = dim3(1024);
  err = cudaLaunchKernelEx(&cfg, sort_scan_kernel, (const int32_t*)cnt, base, (int)L.nchunks, E,
                           offsets);
  if (err != cudaSuccess) return err;
  cfg.gridDim = grid;
  cfg.blockDim = dim3(kCopyThreads);
  return cudaLaunchKernelEx(&cfg, permute_rows_kernel<V, false, U>, xv, nv, T, K, E, tpb, ids,
                            (const uint16_t*)rank, (const int32_t*)base, pos, offsets, xpv);
}

template <class O, class Y>
cudaError_t run_combine(const beam_moe_rows_cfg& c, int64_t T, int64_t rows, const void* y,
                        const int32_t* pos, const float* w, void* out, cudaStream_t st) {
  const int H = c.width, K = c.top_k;
  const Y* yy = static_cast<const Y*>(y);
  O* oo = static_cast<O*>(out);
  if (H % 8 == 0) {
    // one pass per thread, however many tokens (4096 tokens: 61 us; all five
    // passes of a row in one CTA 64 us)
    const dim3 grid((unsigned)T, (unsigned)((H / 8 + kRowThreads - 1) / kRowThreads));
    combine_rows_kernel<O, Y, 8, 1><<<grid, kRowThreads, 0, st>>>(yy, H, K, rows, pos, w, oo);
  } else {
    // enough CTAs for eight per SM (4000 tokens x 1003: one CTA per token 11.6
    // us, one pass per thread 13.3 us)
    const int64_t want = (8 * (int64_t)device_sm_count() + T - 1) / T;
    const int64_t most = (H + 4 * kRowThreads - 1) / (4 * kRowThreads);
    const dim3 grid((unsigned)T, (unsigned)(want < most ? want : most));
    combine_rows_kernel<O, Y, 1, 4><<<grid, kRowThreads, 0, st>>>(yy, H, K, rows, pos, w, oo);
  }
  return cudaGetLastError();
}

template <class O, class Y>
cudaError_t run_combine_bwd(const beam_moe_rows_cfg& c, int64_t T, int64_t rows, const void* dout,
                            const void* y, const int32_t* pos, const float* w, void* dy, float* dw,
                            cudaStream_t st) {
  const int H = c.width, K = c.top_k;
  const O* d = static_cast<const O*>(dout);
  const Y* yy = static_cast<const Y*>(y);
  Y* o = static_cast<Y*>(dy);
  const int S = H % 8 == 0 ? 2 : 1;
  int64_t gy = (8 * (int64_t)device_sm_count() + T - 1) / T;  // few tokens: their slots apart
  if (gy > (K + S - 1) / S) gy = (K + S - 1) / S;
  const dim3 grid((unsigned)T, (unsigned)gy);
  constexpr int kThreads = sizeof(Y) == 2 ? 128 : 256;
  if (S == 2)
    combine_bwd_kernel<O, Y, 8, 2, 1, kThreads>
        <<<grid, kThreads, 0, st>>>(d, yy, H, K, rows, pos, w, o, dw);
  else
    combine_bwd_kernel<O, Y, 1, 1, 8, 128>
        <<<grid, 128, 0, st>>>(d, yy, H, K, rows, pos, w, o, dw);
  return cudaGetLastError();
}

// f(O, Y) for the pair of types: the rows' is the configuration's or FP32.
#define BEAM_ROW_TYPES(f, ...)                                                       \
  switch (c.dtype) {                                                                 \
    case BEAM_MOE_FP32: return f<float, float>(__VA_ARGS__);                         \
    case BEAM_MOE_FP16:                                                              \
      return y_dtype == BEAM_MOE_FP32 ? f<__half, float>(__VA_ARGS__)                \
                                      : f<__half, __half>(__VA_ARGS__);              \
    default:                                                                         \
      return y_dtype == BEAM_MOE_FP32 ? f<__nv_bfloat16, float>(__VA_ARGS__)         \
                                      : f<__nv_bfloat16, __nv_bfloat16>(__VA_ARGS__); \
  }

cudaError_t launch_combine_rows(const beam_moe_rows_cfg& c, int64_t T, int64_t rows, const void* y,
                                int32_t y_dtype, const int32_t* pos, const float* w, void* out,
                                cudaStream_t st) {
  BEAM_ROW_TYPES(run_combine, c, T, rows, y, pos, w, out, st)
}

cudaError_t launch_combine_bwd(const beam_moe_rows_cfg& c, int64_t T, int64_t rows,
                               const void* dout, const void* y, int32_t y_dtype,
                               const int32_t* pos, const float* w, void* dy, float* dw,
                               cudaStream_t st) {
  BEAM_ROW_TYPES(run_combine_bwd, c, T, rows, dout, y, pos, w, dy, dw, st)
}

beam_moe_status check_rows(const beam_moe_rows_cfg* c, int64_t T) {
  if (!c || T < 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->width <= 0 || c->n_experts <= 0 || c->top_k <= 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->dtype < BEAM_MOE_BF16 || c->dtype > BEAM_MOE_FP32) return BEAM_MOE_ERR_INVALID_ARG;
  if (c->width > 65536 || c->n_experts > kMaxE || c->top_k > kMaxK)
    return BEAM_MOE_ERR_UNSUPPORTED_SHAPE;
  if (T > ((int64_t)1 << 30) / c->top_k) return BEAM_MOE_ERR_UNSUPPORTED_SHAPE;
  return BEAM_MOE_OK;
}

bool y_type_ok(const beam_moe_rows_cfg* c, int32_t y_dtype) {
  return y_dtype == c->dtype || y_dtype == BEAM_MOE_FP32;
}

}  // namespace
}  // namespace beam

extern "C" {

beam_moe_status beam_moe_permute_workspace_size(const beam_moe_rows_cfg* cfg, int64_t T,
                                                size_t* bytes) {
  const beam_moe_status s = beam::check_rows(cfg, T);
  if (s != BEAM_MOE_OK) return s;
  if (!bytes) return BEAM_MOE_ERR_INVALID_ARG;
  *bytes = beam::sort_layout(*cfg, T).total;
  return BEAM_MOE_OK;
}

beam_moe_status beam_moe_permute(const beam_moe_rows_cfg* cfg, int64_t T, const void* x,
                                 const int32_t* topk_ids, void* xp, int32_t* pos,
                                 int32_t* offsets, void* ws, size_t ws_bytes, void* stream) {
  beam_moe_status s = beam::check_rows(cfg, T);
  if (s != BEAM_MOE_OK) return s;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  s = T == 0 ? beam::check_ops_ptrs({offsets}, {})
             : beam::check_ops_ptrs({x, topk_ids, xp, pos, offsets, ws}, {});
  if (s != BEAM_MOE_OK) return s;
  if (T == 0)  // no rows: every expert's segment is empty
    return beam::cuda_status(cudaMemsetAsync(offsets, 0, 4 * (size_t)(cfg->n_experts + 1), st));
  if (ws_bytes < beam::sort_layout(*cfg, T).total) return BEAM_MOE_ERR_WORKSPACE_TOO_SMALL;
  char* w = static_cast<char*>(ws);
  const size_t row = (size_t)cfg->width * beam::dtype_bytes(cfg->dtype);
  if (row % 16 == 0)
    return beam::cuda_status(
        beam::run_permute<uint4>(*cfg, T, x, topk_ids, xp, pos, offsets, w, st));
  if (row % 4 == 0)
    return beam::cuda_status(
        beam::run_permute<uint32_t>(*cfg, T, x, topk_ids, xp, pos, offsets, w, st));
  return beam::cuda_status(
      beam::run_permute<uint16_t>(*cfg, T, x, topk_ids, xp, pos, offsets, w, st));
}

beam_moe_status beam_moe_permute_backward(const beam_moe_rows_cfg* cfg, int64_t T, int64_t rows,
                                          const void* dxp, const int32_t* pos, void* dx,
                                          void* stream) {
  beam_moe_status s = beam::check_rows(cfg, T);
  if (s != BEAM_MOE_OK) return s;
  if (rows < 0) return BEAM_MOE_ERR_INVALID_ARG;
  if (T == 0) return BEAM_MOE_OK;
  // an empty buffer may have no address
  s = rows == 0 ? beam::check_ops_ptrs({pos, dx}, {dxp}) : beam::check_ops_ptrs({dxp, pos, dx}, {});
  if (s != BEAM_MOE_OK) return s;
  return beam::cuda_status(beam::launch_combine_rows(*cfg, T, rows, dxp, cfg->dtype, pos, nullptr,
                                                     dx, reinterpret_cast<cudaStream_t>(stream)));
}

beam_moe_status beam_moe_combine(const beam_moe_rows_cfg* cfg, int64_t T, int64_t rows,
                                 const void* y, int32_t y_dtype, const int32_t* pos,
                                 const float* w, void* out, void* stream) {
  beam_moe_status s = beam::check_rows(cfg, T);
  if (s != BEAM_MOE_OK) return s;
  if (rows < 0 || !beam::y_type_ok(cfg, y_dtype)) return BEAM_MOE_ERR_INVALID_ARG;
  if (T == 0) return BEAM_MOE_OK;
  s = rows == 0 ? beam::check_ops_ptrs({pos, out}, {y, w}) : beam::check_ops_ptrs({y, pos, out}, {w});
  if (s != BEAM_MOE_OK) return s;
  return beam::cuda_status(beam::launch_combine_rows(*cfg, T, rows, y, y_dtype, pos, w, out,
                                                     reinterpret_cast<cudaStream_t>(stream)));
}

beam_moe_status beam_moe_combine_backward(const beam_moe_rows_cfg* cfg, int64_t T, int64_t rows,
                                          const void* dout, const void* y, int32_t y_dtype,
                                          const int32_t* pos, const float* w, void* dy, float* dw,
                                          void* stream) {
  beam_moe_status s = beam::check_rows(cfg, T);
  if (s != BEAM_MOE_OK) return s;
  if (rows < 0 || !beam::y_type_ok(cfg, y_dtype)) return BEAM_MOE_ERR_INVALID_ARG;
  if (T == 0) return BEAM_MOE_OK;
  // Without rows dy is empty, and y and dy may have no address.
  if (rows != 0 && ((!dy && !dw) || (dw && !y))) return BEAM_MOE_ERR_INVALID_ARG;
  s = beam::check_ops_ptrs({dout, pos}, {y, w, dy, dw});
  if (s != BEAM_MOE_OK) return s;
  if (rows == 0 && !dw) return BEAM_MOE_OK;
  return beam::cuda_status(beam::launch_combine_bwd(*cfg, T, rows, dout, y, y_dtype, pos, w, dy,
                                                    dw, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
