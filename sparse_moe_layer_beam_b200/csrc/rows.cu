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
// One CTA: thread (j, e) sums the j-th part of expert e's chunks.
__global__ void __launch_bounds__(1024) sort_scan_kernel(int32_t* __restrict__ cnt, int nchunks,
                                                         int E, int32_t* __restrict__ offsets) {
  __shared__ int part[1024];
  __shared__ int warp_tot[32], total;
  const int tid = threadIdx.x;
  const int per_e = 1024 / E;  // E <= 512
  const int e = tid % E, j = tid / E;
  const int len = (nchunks + per_e - 1) / per_e;
  const int c0 = min(nchunks, j * len), c1 = min(nchunks, c0 + len);
  const bool act = j < per_e;
  int sum = 0;
  if (act)
#pragma unroll 8
    for (int c = c0; c < c1; ++c) sum += cnt[(size_t)c * E + e];
  part[tid] = sum;
  __syncthreads();
  int tot = 0;
  if (tid < E)
    for (int q = 0; q < per_e; ++q) tot += part[q * E + tid];
  const int off = block_scan(tid < E ? tot : 0, warp_tot, &total);
  if (tid < E) offsets[tid] = off;
  if (tid == 0) offsets[E] = total;
  __syncthreads();
  if (tid < E) {  // part becomes the first row of (part, expert)
    int run = off;
    for (int q = 0; q < per_e; ++q) {
      const int c = part[q * E + tid];
      part[q * E + tid] = run;
      run += c;
    }
  }
  __syncthreads();
  if (act) {
    int run = part[tid];
#pragma unroll 8
    for (int c = c0; c < c1; ++c) {
      const int v = cnt[(size_t)c * E + e];
      cnt[(size_t)c * E + e] = run;
      run += v;
    }
  }
}

constexpr int kCopyThreads = 256;

// Copies x[t] to its rows for `tpb` tokens per CTA, a slice of the row per
// blockIdx.y. V: the unit of the copy (16, 4 or 2 bytes; nv of them per row).
// ONE: the positions are counted here, from all ids (A <= kOneLaunch).
template <class V, bool ONE>
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
  const int step = gridDim.y * kCopyThreads;
  for (int i = 0; i < nt; ++i) {
    const V* src = x + (t0 + i) * nv;
    for (int v = blockIdx.y * kCopyThreads + tid; v < nv; v += step) {
      const V d = __ldg(src + v);
      for (int k = 0; k < K; ++k) {
        const int p = s_pos[i * K + k];
        if (p >= 0) xp[(size_t)p * nv + v] = d;
      }
    }
  }
}

// --------------------------------------------------- combine and its backward
constexpr int kRowThreads = 128;

// out[t] = sum_k w[t,k] y[pos[t,k]] (w NULL: 1). A CTA per token and slice of
// the row; N elements per thread and step.
template <class O, class Y, int N>
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
  const int nv = H / N;
  for (int v = blockIdx.y * kRowThreads + tid; v < nv; v += gridDim.y * kRowThreads) {
    float acc[N];
#pragma unroll
    for (int i = 0; i < N; ++i) acc[i] = 0.0f;
#pragma unroll 4
    for (int k = 0; k < K; ++k) {
      const int p = s_pos[k];
      if (p < 0) continue;
      const Pack<Y, N> r = load_pack<Y, N>(y + (size_t)p * H + (size_t)v * N);
      const float wk = s_w[k];
#pragma unroll
      for (int i = 0; i < N; ++i) acc[i] = fmaf(wk, to_f32(r.v[i]), acc[i]);
    }
    Pack<O, N> o;
#pragma unroll
    for (int i = 0; i < N; ++i) o.v[i] = from_f32<O>(acc[i]);
    store_pack<O, N>(out + (size_t)t * H + (size_t)v * N, o);
  }
}

// dy rows and dw of one token's slots k = blockIdx.y, blockIdx.y + gridDim.y,
// ... A thread's products are added in column order, a warp's by a shuffle
// tree, the four warps' in order: the sum has one order whatever runs when.
template <class O, class Y, int N>
__global__ void __launch_bounds__(kRowThreads)
    combine_bwd_kernel(const O* __restrict__ dout, const Y* __restrict__ y, int H, int K,
                       int64_t rows, const int32_t* __restrict__ pos,
                       const float* __restrict__ w, Y* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float s_sum[kMaxK][kRowThreads / 32];
  const int64_t t = blockIdx.x;
  const int tid = threadIdx.x;
  const int nv = H / N;
  const O* d = dout + (size_t)t * H;
  for (int k = blockIdx.y; k < K; k += gridDim.y) {
    int p = pos[t * K + k];
    if (p >= rows) p = -1;
    float sum = 0.0f;
    if (p >= 0) {
      const float wk = w ? w[t * K + k] : 1.0f;
#pragma unroll 4
      for (int v = tid; v < nv; v += kRowThreads) {
        const Pack<O, N> g = load_pack<O, N>(d + (size_t)v * N);
        const size_t at = (size_t)p * H + (size_t)v * N;
        if (dw) {
          const Pack<Y, N> r = load_pack<Y, N>(y + at);
#pragma unroll
          for (int i = 0; i < N; ++i) sum = fmaf(to_f32(g.v[i]), to_f32(r.v[i]), sum);
        }
        if (dy) {
          Pack<Y, N> o;
#pragma unroll
          for (int i = 0; i < N; ++i) o.v[i] = from_f32<Y>(wk * to_f32(g.v[i]));
          store_pack<Y, N>(dy + at, o);
        }
      }
    }
    if (dw) {
#pragma unroll
      for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
      if ((tid & 31) == 0) s_sum[k][tid >> 5] = sum;
    }
  }
  if (dw) {
    __syncthreads();
    for (int k = blockIdx.y + tid * gridDim.y; k < K; k += kRowThreads * gridDim.y)
      dw[t * K + k] = (s_sum[k][0] + s_sum[k][1]) + (s_sum[k][2] + s_sum[k][3]);
  }
}

// ------------------------------------------------------------------- launches
struct SortLayout {
  int nchunks;
  size_t rank, cnt, total;
};

SortLayout sort_layout(const beam_moe_rows_cfg& c, int64_t T) {
  SortLayout L;
  const int64_t A = T * c.top_k;
  L.nchunks = (int)((A + kSortChunk - 1) / kSortChunk);
  L.rank = 256;
  const size_t rank_bytes = ((size_t)A * 2 + 255) / 256 * 256;
  L.cnt = L.rank + rank_bytes;
  L.total = A <= kOneLaunch ? 256 : L.cnt + ((size_t)L.nchunks * c.n_experts * 4 + 255) / 256 * 256;
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
  // about four CTAs per SM, at most 8 tokens (and 256 assignments) each; with
  // few tokens a row is cut into slices instead
  const int64_t want = 4 * (int64_t)device_sm_count();
  int tpb = (int)(T / want < 1 ? 1 : T / want);
  if (tpb > 8) tpb = 8;
  if (tpb * K > kCopyThreads) tpb = kCopyThreads / K;
  const int64_t gx = (T + tpb - 1) / tpb;
  int64_t gy = (want / 2 + gx - 1) / gx;
  const int most = (nv + kCopyThreads - 1) / kCopyThreads;
  if (gy > most) gy = most;
  if (gy < 1) gy = 1;
  const dim3 grid((unsigned)gx, (unsigned)gy);
  const V* xv = static_cast<const V*>(x);
  V* xpv = static_cast<V*>(xp);
  if (one) {
    permute_rows_kernel<V, true><<<grid, kCopyThreads, 0, st>>>(xv, nv, T, K, E, tpb, ids, nullptr,
                                                                nullptr, pos, offsets, xpv);
    return cudaGetLastError();
  }
  uint16_t* rank = reinterpret_cast<uint16_t*>(ws + L.rank);
  int32_t* cnt = reinterpret_cast<int32_t*>(ws + L.cnt);
  sort_count_kernel<<<L.nchunks, kSortChunk, 0, st>>>(ids, A, E, rank, cnt);
  cudaError_t err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  sort_scan_kernel<<<1, 1024, 0, st>>>(cnt, L.nchunks, E, offsets);
  err = cudaGetLastError();
  if (err != cudaSuccess) return err;
  permute_rows_kernel<V, false><<<grid, kCopyThreads, 0, st>>>(xv, nv, T, K, E, tpb, ids, rank, cnt,
                                                               pos, offsets, xpv);
  return cudaGetLastError();
}

template <class O, class Y>
cudaError_t run_combine(const beam_moe_rows_cfg& c, int64_t T, int64_t rows, const void* y,
                        const int32_t* pos, const float* w, void* out, cudaStream_t st) {
  const int H = c.width, K = c.top_k;
  const Y* yy = static_cast<const Y*>(y);
  O* oo = static_cast<O*>(out);
  if (H % 8 == 0) {
    const dim3 grid((unsigned)T, (unsigned)h_slices(T, H / 8));
    combine_rows_kernel<O, Y, 8><<<grid, kRowThreads, 0, st>>>(yy, H, K, rows, pos, w, oo);
  } else {
    const dim3 grid((unsigned)T, (unsigned)h_slices(T, H));
    combine_rows_kernel<O, Y, 1><<<grid, kRowThreads, 0, st>>>(yy, H, K, rows, pos, w, oo);
  }
  return cudaGetLastError();
}

template <class O, class Y>
cudaError_t run_combine_bwd(const beam_moe_rows_cfg& c, int64_t T, int64_t rows, const void* dout,
                            const void* y, const int32_t* pos, const float* w, void* dy, float* dw,
                            cudaStream_t st) {
  const int H = c.width, K = c.top_k;
  int64_t gy = (4 * (int64_t)device_sm_count() + T - 1) / T;  // few tokens: their slots apart
  if (gy > K) gy = K;
  const dim3 grid((unsigned)T, (unsigned)gy);
  const O* d = static_cast<const O*>(dout);
  const Y* yy = static_cast<const Y*>(y);
  Y* o = static_cast<Y*>(dy);
  if (H % 8 == 0)
    combine_bwd_kernel<O, Y, 8><<<grid, kRowThreads, 0, st>>>(d, yy, H, K, rows, pos, w, o, dw);
  else
    combine_bwd_kernel<O, Y, 1><<<grid, kRowThreads, 0, st>>>(d, yy, H, K, rows, pos, w, o, dw);
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
  if (T * (int64_t)c->top_k > (int64_t)1 << 30) return BEAM_MOE_ERR_UNSUPPORTED_SHAPE;
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
  s = beam::check_ops_ptrs({dxp, pos, dx}, {});
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
  s = beam::check_ops_ptrs({y, pos, out}, {w});
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
  if (!dy && !dw) return BEAM_MOE_ERR_INVALID_ARG;
  if (dw && !y) return BEAM_MOE_ERR_INVALID_ARG;
  if (T == 0) return BEAM_MOE_OK;
  s = beam::check_ops_ptrs({dout, pos}, {y, w, dy, dw});
  if (s != BEAM_MOE_OK) return s;
  return beam::cuda_status(beam::launch_combine_bwd(*cfg, T, rows, dout, y, y_dtype, pos, w, dy,
                                                    dw, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
