// Layer norm over the channels of each row, and its gradients, for sm_103a.
//
//   y = xhat * (offset + weight_g) + bias_g,   xhat = (x - mean) * rstd,
// g the row's group: group_rows consecutive rows share one row of weight and
// bias (one group: the plain layer norm; a group per chunk: the scale and shift
// that a diffusion transformer takes from each chunk's noise level).
// For dy, with t = dy * (offset + weight_g):
//   dx = rstd * (t - mean(t) - xhat * mean(t * xhat)),
//   dweight_g = sum over the group's rows of dy * xhat,  dbias_g = sum of dy.
//
// Both are streams of rows, bound by memory: forward one read and one write of
// a row, backward two reads and one write.  A row lives in registers from its
// one read to its write, so the variance is taken about the mean (a second pass
// over registers, not E[x^2] - mean^2, which loses all digits of rows far off
// centre).  Sums, moments and the weight's gradients are fp32.
#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

using namespace ptx;

// N elements of a row, as one access.  Rows whose channels and strides are
// multiples of 16 bytes go in 16-byte vectors, all others element by element.
template <typename T, bool V>
struct Pack;
template <>
struct Pack<uint16_t, true> {
  static constexpr int N = 8;
  typedef uint4 Raw;
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[N]) {
    const uint32_t w[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) {
    return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Pack<float, true> {
  static constexpr int N = 4;
  typedef float4 Raw;
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[N]) {
    f[0] = r.x, f[1] = r.y, f[2] = r.z, f[3] = r.w;
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) { return make_float4(f[0], f[1], f[2], f[3]); }
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Pack<uint16_t, false> {
  static constexpr int N = 1;
  typedef uint16_t Raw;
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[N]) {
    f[0] = __uint_as_float((uint32_t)r << 16);
  }
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) { return (uint16_t)pack_bf16(f[0], 0.f); }
  static __device__ __forceinline__ Raw zero() { return 0; }
};
template <>
struct Pack<float, false> {
  static constexpr int N = 1;
  typedef float Raw;
  static __device__ __forceinline__ void unpack(const Raw& r, float (&f)[N]) { f[0] = r; }
  static __device__ __forceinline__ Raw pack(const float (&f)[N]) { return f[0]; }
  static __device__ __forceinline__ Raw zero() { return 0.f; }
};

// N consecutive fp32 values of a weight row
template <int N>
__device__ __forceinline__ void load_f32(const float* p, float (&f)[N]) {
  if constexpr (N == 1) {
    f[0] = __ldg(p);
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4) {
      const float4 v = __ldg(reinterpret_cast<const float4*>(p + i));
      f[i] = v.x, f[i + 1] = v.y, f[i + 2] = v.z, f[i + 3] = v.w;
    }
  }
}
template <int N>
__device__ __forceinline__ void store_f32(float* p, const float (&f)[N]) {
  if constexpr (N == 1) {
    *p = f[0];
  } else {
#pragma unroll
    for (int i = 0; i < N; i += 4)
      *reinterpret_cast<float4*>(p + i) = make_float4(f[i], f[i + 1], f[i + 2], f[i + 3]);
  }
}

// A row is shared by `lanes` (a power of two) lanes of a warp, or by all 32 of
// p.warps warps.  Sum of K values over the row's threads; `buf` holds two sets
// of 32 x K floats, taken in turn so that one barrier a sum suffices.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int lanes, int warps, float* buf, int& turn) {
  for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
  if (warps == 1) return;
  float* b = buf + turn * 32 * K;
  turn ^= 1;
  const int warp = threadIdx.x >> 5;
  if ((threadIdx.x & 31) == 0) {
#pragma unroll
    for (int k = 0; k < K; ++k) b[warp * K + k] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
  for (int w = 0; w < warps; ++w)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += b[w * K + k];
}

// One row per group of row threads; NV accesses a thread.
template <typename T, bool V, int NV>
__global__ void __launch_bounds__(V ? 512 : 1024) norm_kernel(const __grid_constant__ NormParams p) {
  using P = Pack<T, V>;
  constexpr int N = P::N;
  __shared__ float buf[2 * 32];
  const int per_row = p.lanes * p.warps;  // threads of a row
  const int slot = threadIdx.x / per_row, me = threadIdx.x - slot * per_row;
  const long long row = (long long)blockIdx.x * (blockDim.x / per_row) + slot;
  const bool live = row < p.rows;
  const int packs = p.C / N;
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  const T* x = static_cast<const T*>(p.x) + (live ? row : 0) * p.x_row;
  typename P::Raw raw[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = me + i * per_row;
    raw[i] = live && j < packs ? reinterpret_cast<const typename P::Raw*>(x)[j] : P::zero();
  }
  float s[1] = {0.f};
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[N];
    P::unpack(raw[i], f);
#pragma unroll
    for (int c = 0; c < N; ++c) s[0] += f[c];
  }
  row_sum<1>(s, p.lanes, p.warps, buf, turn);
  const float mean = s[0] * p.inv_c;
  s[0] = 0.f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    float f[N];
    P::unpack(raw[i], f);
    const bool in = me + i * per_row < packs;
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float d = in ? f[c] - mean : 0.f;
      s[0] = fmaf(d, d, s[0]);
    }
  }
  row_sum<1>(s, p.lanes, p.warps, buf, turn);
  const float rstd = 1.f / sqrtf(fmaf(s[0], p.inv_c, p.eps));
  if (!live) return;
  if (me == 0) {
    if (p.mean != nullptr) p.mean[row] = mean;
    if (p.rstd != nullptr) p.rstd[row] = rstd;
  }
  const long long group = p.group_rows >= p.rows ? 0 : row / p.group_rows;
  const float* w = p.weight != nullptr ? p.weight + group * p.C : nullptr;
  const float* b = p.bias != nullptr ? p.bias + group * p.C : nullptr;
  T* y = static_cast<T*>(p.y) + row * p.y_row;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = me + i * per_row;
    if (j >= packs) break;
    float f[N], wf[N], bf[N];
    P::unpack(raw[i], f);
    if (w != nullptr) load_f32<N>(w + j * N, wf);
    if (b != nullptr) load_f32<N>(b + j * N, bf);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      const float u = (f[c] - mean) * rstd;
      f[c] = fmaf(u, w != nullptr ? p.offset + wf[c] : 1.f, b != nullptr ? bf[c] : 0.f);
    }
    reinterpret_cast<typename P::Raw*>(y)[j] = P::pack(f);
  }
}

// A block takes a range of one group's rows, kRows at a time per group of row
// threads, and keeps its channels' sums of dy * xhat and dy in registers over
// the whole range.  Ranges of a group that several blocks share leave partial
// sums for norm_sums_kernel: no atomics, so the results do not change from
// call to call.
constexpr int kRows = 4;

template <typename T, bool V, int NV>
__global__ void __launch_bounds__(V ? 512 : 1024) norm_back_kernel(const __grid_constant__ NormParams p) {
  using P = Pack<T, V>;
  constexpr int N = P::N;
  extern __shared__ float sm[];  // row sums, or the blocks' channel sums of several row slots
  const int per_row = p.lanes * p.warps;
  const int slots = blockDim.x / per_row;
  const int slot = threadIdx.x / per_row, me = threadIdx.x - slot * per_row;
  const long long group = blockIdx.x / p.splits;
  const int split = (int)(blockIdx.x - group * p.splits);
  const long long g0 = group * p.group_rows;
  const long long g1 = g0 + p.group_rows < p.rows ? g0 + p.group_rows : p.rows;
  const long long r0 = g0 + split * p.split_rows;
  const long long r1 = r0 + p.split_rows < g1 ? r0 + p.split_rows : g1;
  const int packs = p.C / N;
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  float w[NV][N], dw[NV][N], db[NV][N];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = me + i * per_row;
    if (p.weight != nullptr && j < packs) load_f32<N>(p.weight + group * p.C + j * N, w[i]);
#pragma unroll
    for (int c = 0; c < N; ++c) {
      w[i][c] = p.weight != nullptr && j < packs ? w[i][c] + p.offset : 1.f;
      dw[i][c] = db[i][c] = 0.f;
    }
  }
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  for (long long base = r0; base < r1; base += (long long)slots * kRows) {
    typename P::Raw xr[kRows][NV], yr[kRows][NV];
    float mean[kRows], rstd[kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long r = base + slot + (long long)k * slots;
      const bool in = r < r1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = me + i * per_row;
        const bool on = in && j < packs;
        xr[k][i] = on ? reinterpret_cast<const typename P::Raw*>(x + r * p.x_row)[j] : P::zero();
        yr[k][i] = on ? reinterpret_cast<const typename P::Raw*>(dy + r * p.dy_row)[j] : P::zero();
      }
      mean[k] = in ? __ldg(p.mean + r) : 0.f;
      rstd[k] = in ? __ldg(p.rstd + r) : 0.f;
    }
    float s[2 * kRows];
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      s[2 * k] = s[2 * k + 1] = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const bool in = me + i * per_row < packs;  // a missing channel holds 0, not the mean
        float f[N], g[N];
        P::unpack(xr[k][i], f);
        P::unpack(yr[k][i], g);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float u = in ? (f[c] - mean[k]) * rstd[k] : 0.f;
          const float t = g[c] * w[i][c];
          s[2 * k] += t;
          s[2 * k + 1] = fmaf(t, u, s[2 * k + 1]);
          dw[i][c] = fmaf(g[c], u, dw[i][c]);
          db[i][c] += g[c];
        }
      }
    }
    row_sum<2 * kRows>(s, p.lanes, p.warps, sm, turn);
#pragma unroll
    for (int k = 0; k < kRows; ++k) {
      const long long r = base + slot + (long long)k * slots;
      if (r >= r1) break;
      const float mt = s[2 * k] * p.inv_c, mu = s[2 * k + 1] * p.inv_c;
      T* dx = static_cast<T*>(p.y) + r * p.y_row;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = me + i * per_row;
        if (j >= packs) break;
        float f[N], g[N];
        P::unpack(xr[k][i], f);
        P::unpack(yr[k][i], g);
#pragma unroll
        for (int c = 0; c < N; ++c) {
          const float u = (f[c] - mean[k]) * rstd[k];
          f[c] = rstd[k] * (fmaf(g[c], w[i][c], -mt) - u * mu);
        }
        reinterpret_cast<typename P::Raw*>(dx)[j] = P::pack(f);
      }
    }
  }
  if (p.dweight == nullptr && p.dbias == nullptr) return;
  // one range a group: the gradients themselves; several: this range's part
  float* to_w = p.splits == 1 ? (p.dweight != nullptr ? p.dweight + group * p.C : nullptr)
                              : p.part + (long long)blockIdx.x * 2 * p.C;
  float* to_b = p.splits == 1 ? (p.dbias != nullptr ? p.dbias + group * p.C : nullptr) : to_w + p.C;
  if (slots == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = me + i * per_row;
      if (j >= packs) break;
      if (to_w != nullptr) store_f32<N>(to_w + j * N, dw[i]);
      if (to_b != nullptr) store_f32<N>(to_b + j * N, db[i]);
    }
    return;
  }
  // channels of several row slots, added in the slots' order
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = me + i * per_row;
      if (j < packs) {
#pragma unroll
        for (int c = 0; c < N; ++c) sm[slot * p.C + j * N + c] = t == 0 ? dw[i][c] : db[i][c];
      }
    }
    __syncthreads();
    float* to = t == 0 ? to_w : to_b;
    if (to != nullptr)
      for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float a = 0.f;
        for (int k = 0; k < slots; ++k) a += sm[k * p.C + c];
        to[c] = a;
      }
  }
}

// Sum of a group's partial rows: part [groups][splits][2][C].  32 channels x 8
// shares of the splits a block; the shares are added in their order.
__global__ void __launch_bounds__(256) norm_sums_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[8][33];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int blocks = (p.C + 31) / 32;
  const long long unit = blockIdx.x / blocks;  // group and tensor
  const int c = (int)(blockIdx.x - unit * blocks) * 32 + lane;
  const long long group = unit >> 1;
  const int t = (int)(unit & 1);
  float* to = t == 0 ? p.dweight : p.dbias;
  if (to == nullptr) return;
  const float* from = p.part + (group * p.splits * 2 + t) * (long long)p.C + c;
  float a = 0.f;
  if (c < p.C)
#pragma unroll 8
    for (int s = share; s < p.splits; s += 8) a += from[(long long)s * 2 * p.C];
  sm[share][lane] = a;
  __syncthreads();
  if (share == 0 && c < p.C) {
#pragma unroll
    for (int k = 1; k < 8; ++k) a += sm[k][lane];
    to[group * p.C + c] = a;
  }
}

template <typename K>
cudaError_t launch(K kernel, long long blocks, int threads, size_t smem, const NormParams& p, cudaStream_t s) {
  if (blocks < 1 || blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Threads of a row: lanes of one warp while `most` accesses a lane hold the
// row, whole warps from there; returns the accesses a thread.
int row_threads(int packs, int most, NormParams& p) {
  p.lanes = 32;
  p.warps = (packs + 32 * most - 1) / (32 * most);
  if (p.warps == 1)
    while (packs * 2 <= p.lanes) p.lanes /= 2;
  return (packs + p.lanes * p.warps - 1) / (p.lanes * p.warps);
}

template <typename T, bool V>
cudaError_t forward(NormParams& p, cudaStream_t s) {
  const int packs = p.C / Pack<T, V>::N;
  const int nv = row_threads(packs, packs > 6 * 1024 ? 8 : 6, p);
  const int threads = p.warps == 1 ? 256 : 32 * p.warps;
  const int slots = threads / (p.lanes * p.warps);
  const long long blocks = (p.rows + slots - 1) / slots;
  switch (nv) {
    case 1: return launch(norm_kernel<T, V, 1>, blocks, threads, 0, p, s);
    case 2: return launch(norm_kernel<T, V, 2>, blocks, threads, 0, p, s);
    case 3: return launch(norm_kernel<T, V, 3>, blocks, threads, 0, p, s);
    case 4: return launch(norm_kernel<T, V, 4>, blocks, threads, 0, p, s);
    case 5: return launch(norm_kernel<T, V, 5>, blocks, threads, 0, p, s);
    case 6: return launch(norm_kernel<T, V, 6>, blocks, threads, 0, p, s);
    case 7:
    case 8:
      if constexpr (!V) return launch(norm_kernel<T, V, 8>, blocks, threads, 0, p, s);
  }
  return cudaErrorInvalidValue;
}

template <typename T, bool V>
cudaError_t backward(NormParams& p, cudaStream_t s) {
  const int packs = p.C / Pack<T, V>::N;
  const int nv = row_threads(packs, V ? 16 / Pack<T, V>::N : 8, p);
  const int threads = p.warps == 1 ? 256 : 32 * p.warps;
  const int slots = threads / (p.lanes * p.warps);
  const size_t smem = sizeof(float) * (slots > 1 ? (size_t)slots * p.C : 2 * 32 * 2 * kRows);
  const long long blocks = p.groups * p.splits;
  cudaError_t e = cudaErrorInvalidValue;
  switch (nv) {
    case 1: e = launch(norm_back_kernel<T, V, 1>, blocks, threads, smem, p, s); break;
    case 2: e = launch(norm_back_kernel<T, V, 2>, blocks, threads, smem, p, s); break;
    case 3:
    case 4:
      if constexpr (Pack<T, V>::N <= 4) e = launch(norm_back_kernel<T, V, 4>, blocks, threads, smem, p, s);
      break;
    default:
      if constexpr (!V) e = launch(norm_back_kernel<T, V, 8>, blocks, threads, smem, p, s);
  }
  if (e != cudaSuccess || p.splits == 1 || (p.dweight == nullptr && p.dbias == nullptr)) return e;
  return launch(norm_sums_kernel, p.groups * 2 * ((p.C + 31) / 32), 256, 0, p, s);
}

}  // namespace

cudaError_t launch_layer_norm(NormParams& p, bool fp32, bool vec, bool back, cudaStream_t s) {
  if (fp32) {
    if (back) return vec ? backward<float, true>(p, s) : backward<float, false>(p, s);
    return vec ? forward<float, true>(p, s) : forward<float, false>(p, s);
  }
  if (back) return vec ? backward<uint16_t, true>(p, s) : backward<uint16_t, false>(p, s);
  return vec ? forward<uint16_t, true>(p, s) : forward<uint16_t, false>(p, s);
}

}  // namespace sab
