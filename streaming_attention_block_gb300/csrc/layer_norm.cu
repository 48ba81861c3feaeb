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
// 61440 x 1536 bf16 of 40 groups: 63 us, 0.89 of the copy rate, and 103, 0.81;
// 4095 x 1001 fp32, accesses of 4 bytes: 13 and 18 (4.8 and 7.3 at that rate).
#include <algorithm>
#include <atomic>

#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

using namespace ptx;

// Values in registers: pairs in packed fp32 arithmetic, or single ones where an
// access holds one element.
__device__ __forceinline__ float2 vadd(float2 a, float2 b) { return __fadd2_rn(a, b); }
__device__ __forceinline__ float2 vmul(float2 a, float2 b) { return __fmul2_rn(a, b); }
__device__ __forceinline__ float2 vfma(float2 a, float2 b, float2 c) { return __ffma2_rn(a, b, c); }
__device__ __forceinline__ float vadd(float a, float b) { return a + b; }
__device__ __forceinline__ float vmul(float a, float b) { return a * b; }
__device__ __forceinline__ float vfma(float a, float b, float c) { return fmaf(a, b, c); }
__device__ __forceinline__ float both(float2 a) { return a.x + a.y; }
__device__ __forceinline__ float both(float a) { return a; }
template <typename E>
__device__ __forceinline__ E splat(float x);
template <>
__device__ __forceinline__ float2 splat<float2>(float x) {
  return make_float2(x, x);
}
template <>
__device__ __forceinline__ float splat<float>(float x) {
  return x;
}

// N elements of a row, as one access of A bytes: 16 where rows, strides and
// weights allow it, else 4, else (bf16 with an odd stride) one element.  M
// values of type E.
__device__ __forceinline__ float2 wide(uint32_t w) {  // two bf16
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <typename T, int A>
struct Pack;
template <>
struct Pack<uint16_t, 16> {
  static constexpr int N = 8, M = 4;
  typedef uint4 Raw;
  typedef float2 E;
  static __device__ __forceinline__ void unpack(const Raw& r, E (&f)[M]) {
    f[0] = wide(r.x), f[1] = wide(r.y), f[2] = wide(r.z), f[3] = wide(r.w);
  }
  static __device__ __forceinline__ Raw pack(const E (&f)[M]) {
    return make_uint4(pack_bf16(f[0].x, f[0].y), pack_bf16(f[1].x, f[1].y), pack_bf16(f[2].x, f[2].y),
                      pack_bf16(f[3].x, f[3].y));
  }
  static __device__ __forceinline__ Raw zero() { return make_uint4(0u, 0u, 0u, 0u); }
};
template <>
struct Pack<float, 16> {
  static constexpr int N = 4, M = 2;
  typedef float4 Raw;
  typedef float2 E;
  static __device__ __forceinline__ void unpack(const Raw& r, E (&f)[M]) {
    f[0] = make_float2(r.x, r.y), f[1] = make_float2(r.z, r.w);
  }
  static __device__ __forceinline__ Raw pack(const E (&f)[M]) { return make_float4(f[0].x, f[0].y, f[1].x, f[1].y); }
  static __device__ __forceinline__ Raw zero() { return make_float4(0.f, 0.f, 0.f, 0.f); }
};
template <>
struct Pack<uint16_t, 4> {
  static constexpr int N = 2, M = 1;
  typedef uint32_t Raw;
  typedef float2 E;
  static __device__ __forceinline__ void unpack(const Raw& r, E (&f)[M]) { f[0] = wide(r); }
  static __device__ __forceinline__ Raw pack(const E (&f)[M]) { return pack_bf16(f[0].x, f[0].y); }
  static __device__ __forceinline__ Raw zero() { return 0u; }
};
template <>
struct Pack<uint16_t, 2> {
  static constexpr int N = 1, M = 1;
  typedef uint16_t Raw;
  typedef float E;
  static __device__ __forceinline__ void unpack(const Raw& r, E (&f)[M]) { f[0] = __uint_as_float((uint32_t)r << 16); }
  static __device__ __forceinline__ Raw pack(const E (&f)[M]) { return (uint16_t)pack_bf16(f[0], 0.f); }
  static __device__ __forceinline__ Raw zero() { return 0; }
};
template <>
struct Pack<float, 4> {
  static constexpr int N = 1, M = 1;
  typedef float Raw;
  typedef float E;
  static __device__ __forceinline__ void unpack(const Raw& r, E (&f)[M]) { f[0] = r; }
  static __device__ __forceinline__ Raw pack(const E (&f)[M]) { return f[0]; }
  static __device__ __forceinline__ Raw zero() { return 0.f; }
};

// Hides where a raw access came from: what is unpacked after this is unpacked
// anew, instead of held in twice the registers across a barrier.
__device__ __forceinline__ void forget(uint4& r) { asm volatile("" : "+r"(r.x), "+r"(r.y), "+r"(r.z), "+r"(r.w)); }
__device__ __forceinline__ void forget(float4& r) { asm volatile("" : "+f"(r.x), "+f"(r.y), "+f"(r.z), "+f"(r.w)); }
__device__ __forceinline__ void forget(uint32_t& r) { asm volatile("" : "+r"(r)); }
__device__ __forceinline__ void forget(uint16_t& r) { asm volatile("" : "+h"(r)); }
__device__ __forceinline__ void forget(float& r) { asm volatile("" : "+f"(r)); }

// The values of a weight row that belong to an access (plain loads: the kernel
// before this one in the stream may have written them).
__device__ __forceinline__ void load_f32(const float* p, float2 (&f)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w), f[2] = make_float2(b.x, b.y), f[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void load_f32(const float* p, float2 (&f)[2]) {
  const float4 a = *reinterpret_cast<const float4*>(p);
  f[0] = make_float2(a.x, a.y), f[1] = make_float2(a.z, a.w);
}
__device__ __forceinline__ void load_f32(const float* p, float2 (&f)[1]) { f[0] = make_float2(p[0], p[1]); }
__device__ __forceinline__ void load_f32(const float* p, float (&f)[1]) { f[0] = p[0]; }
__device__ __forceinline__ void store_f32(float* p, const float2 (&f)[4]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[2].x, f[2].y, f[3].x, f[3].y);
}
__device__ __forceinline__ void store_f32(float* p, const float2 (&f)[2]) {
  *reinterpret_cast<float4*>(p) = make_float4(f[0].x, f[0].y, f[1].x, f[1].y);
}
__device__ __forceinline__ void store_f32(float* p, const float2 (&f)[1]) { p[0] = f[0].x, p[1] = f[0].y; }
__device__ __forceinline__ void store_f32(float* p, const float (&f)[1]) { *p = f[0]; }

// A row is shared by `lanes` (a power of two) lanes of a warp, or by all 32 of
// `warps` warps.  Sum of K values over the row's threads; `buf` holds two sets
// of 32 x K floats, taken in turn so that one barrier a sum suffices.
template <int K>
__device__ __forceinline__ void row_sum(float (&v)[K], int lanes, int warps, float* buf, int& turn) {
  if (warps == 1) {
    for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], o);
    return;
  }
  // each step halves the lanes of a value or, while there are several, the
  // values of a lane: K + 4 - log2 K exchanges instead of 5 K (K = 8: 9 for 40)
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int idx = 0;
  float t[K];
#pragma unroll
  for (int k = 0; k < K; ++k) t[k] = v[k];
  int left = K, low = 31;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    if (left > 1) {
      left >>= 1;
      const bool up = (lane & o) != 0;
#pragma unroll
      for (int k = 0; k < K / 2; ++k)
        if (k < left) {
          const float give = up ? t[k] : t[k + left];
          t[k] = (up ? t[k + left] : t[k]) + __shfl_xor_sync(0xffffffffu, give, o);
        }
      idx += up ? left : 0;
      low = o - 1;
    } else {
      t[0] += __shfl_xor_sync(0xffffffffu, t[0], o);
    }
  }
  float* b = buf + turn * 32 * K;
  turn ^= 1;
  if ((lane & low) == 0) b[warp * K + idx] = t[0];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = 0.f;
#pragma unroll 4
  for (int w = 0; w < warps; ++w) {
    if constexpr (K % 4 == 0) {
#pragma unroll
      for (int k = 0; k < K; k += 4) {
        const float4 x = *reinterpret_cast<const float4*>(b + w * K + k);
        v[k] += x.x, v[k + 1] += x.y, v[k + 2] += x.z, v[k + 3] += x.w;
      }
    } else {
#pragma unroll
      for (int k = 0; k < K; ++k) v[k] += b[w * K + k];
    }
  }
}

// Where a block works: the rows [r0, r1) of one group, `slots` groups of row
// threads side by side, each K rows at a time.
struct Place {
  int per_row, slots, slot, me, packs;
  long long group, r0, r1;
};
__device__ __forceinline__ Place place(const NormParams& p, int n) {
  Place a;
  a.per_row = p.lanes * p.warps;
  a.slots = blockDim.x / a.per_row;
  a.slot = threadIdx.x / a.per_row;
  a.me = threadIdx.x - a.slot * a.per_row;
  a.packs = p.C / n;
  a.group = blockIdx.x / p.splits;
  const int split = (int)(blockIdx.x - a.group * p.splits);
  const long long g0 = a.group * p.group_rows;
  const long long g1 = min(g0 + p.group_rows, p.rows);
  a.r0 = g0 + split * p.split_rows;
  a.r1 = min(a.r0 + p.split_rows, g1);
  return a;
}

// K rows' accesses of this thread, 0 where there is no row or channel
template <typename P, typename T, int NV, int K>
__device__ __forceinline__ void load_rows(typename P::Raw (&raw)[K][NV], const T* x, long long stride,
                                          const Place& a, long long base) {
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const long long r = base + a.slot + (long long)k * a.slots;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = a.me + i * a.per_row;
      raw[k][i] = r < a.r1 && j < a.packs ? reinterpret_cast<const typename P::Raw*>(x + r * stride)[j] : P::zero();
    }
  }
}

// A thread keeps its channels' weights in registers over all rows of its
// block, and has the next K rows in flight while it works on K.
template <typename T, int A, int NV, int K, int MAXT>
__global__ void __launch_bounds__(MAXT) norm_kernel(const __grid_constant__ NormParams p) {
  using P = Pack<T, A>;
  using E = typename P::E;
  constexpr int N = P::N, M = P::M;
  __shared__ __align__(16) float buf[2 * 32 * K];
  const Place a = place(p, N);
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  const T* x = static_cast<const T*>(p.x);
  typename P::Raw nxt[K][NV];
  load_rows<P>(nxt, x, p.x_row, a, a.r0);
  E w[NV][M], b[NV][M];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = a.me + i * a.per_row;
    const bool in = j < a.packs;
    if (p.weight != nullptr && in) load_f32(p.weight + a.group * p.C + j * N, w[i]);
    if (p.bias != nullptr && in) load_f32(p.bias + a.group * p.C + j * N, b[i]);
#pragma unroll
    for (int c = 0; c < M; ++c) {
      w[i][c] = p.weight != nullptr && in ? vadd(w[i][c], splat<E>(p.offset)) : splat<E>(1.f);
      b[i][c] = p.bias != nullptr && in ? b[i][c] : splat<E>(0.f);
    }
  }
  const long long step = (long long)a.slots * K;
  for (long long base = a.r0; base < a.r1; base += step) {
    typename P::Raw raw[K][NV];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
      for (int i = 0; i < NV; ++i) raw[k][i] = nxt[k][i];
    if (base + step < a.r1) load_rows<P>(nxt, x, p.x_row, a, base + step);
    float s[K], mean[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      E t = splat<E>(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        E f[M];
        P::unpack(raw[k][i], f);
#pragma unroll
        for (int c = 0; c < M; ++c) t = vadd(t, f[c]);
      }
      s[k] = both(t);
    }
    row_sum<K>(s, p.lanes, p.warps, buf, turn);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      mean[k] = s[k] * p.inv_c;
      E t = splat<E>(0.f);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        E f[M];
        forget(raw[k][i]);
        P::unpack(raw[k][i], f);
        if (a.me + i * a.per_row < a.packs) {
#pragma unroll
          for (int c = 0; c < M; ++c) {
            const E d = vadd(f[c], splat<E>(-mean[k]));
            t = vfma(d, d, t);
          }
        }
      }
      s[k] = both(t);
    }
    row_sum<K>(s, p.lanes, p.warps, buf, turn);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long r = base + a.slot + (long long)k * a.slots;
      if (r >= a.r1) break;
      const float rstd = 1.f / sqrtf(fmaf(s[k], p.inv_c, p.eps));
      if (a.me == 0) {
        if (p.mean != nullptr) p.mean[r] = mean[k];
        if (p.rstd != nullptr) p.rstd[r] = rstd;
      }
      T* y = static_cast<T*>(p.y) + r * p.y_row;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = a.me + i * a.per_row;
        if (j >= a.packs) break;
        E f[M];
        forget(raw[k][i]);
        P::unpack(raw[k][i], f);
#pragma unroll
        for (int c = 0; c < M; ++c)
          f[c] = vfma(vmul(vadd(f[c], splat<E>(-mean[k])), splat<E>(rstd)), w[i][c], b[i][c]);
        reinterpret_cast<typename P::Raw*>(y)[j] = P::pack(f);
      }
    }
  }
}

// The same for the gradients, with the sums of dy * xhat and dy of a thread's
// channels in registers over all rows of its block.  Blocks that share a group
// leave partial sums for norm_sums_kernel: no atomics, so the results do not
// change from call to call.
template <typename T, int A, int NV, int K, int MAXT, int MINB>
__global__ void __launch_bounds__(MAXT, MINB) norm_back_kernel(const __grid_constant__ NormParams p) {
  using P = Pack<T, A>;
  using E = typename P::E;
  constexpr int N = P::N, M = P::M;
  extern __shared__ __align__(16) float sm[];  // row sums, or the channel sums of several row slots
  const Place a = place(p, N);
  int turn = 0;
  griddep_launch_dependents();
  griddep_wait();
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  typename P::Raw nx[K][NV], ny[K][NV];
  float nm[K], nr[K];
  auto fetch = [&](long long base) {
    load_rows<P>(nx, x, p.x_row, a, base);
    load_rows<P>(ny, dy, p.dy_row, a, base);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long r = base + a.slot + (long long)k * a.slots;
      nm[k] = r < a.r1 ? ld_global(p.mean + r) : 0.f;
      nr[k] = r < a.r1 ? ld_global(p.rstd + r) : 0.f;
    }
  };
  fetch(a.r0);
  E w[NV][M], dw[NV][M], db[NV][M];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int j = a.me + i * a.per_row;
    const bool in = j < a.packs;
    if (p.weight != nullptr && in) load_f32(p.weight + a.group * p.C + j * N, w[i]);
#pragma unroll
    for (int c = 0; c < M; ++c) {
      w[i][c] = p.weight != nullptr && in ? vadd(w[i][c], splat<E>(p.offset)) : splat<E>(1.f);
      dw[i][c] = db[i][c] = splat<E>(0.f);
    }
  }
  const long long step = (long long)a.slots * K;
  for (long long base = a.r0; base < a.r1; base += step) {
    typename P::Raw xr[K][NV], yr[K][NV];
    float mean[K], rstd[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      mean[k] = nm[k];
      rstd[k] = nr[k];
#pragma unroll
      for (int i = 0; i < NV; ++i) xr[k][i] = nx[k][i], yr[k][i] = ny[k][i];
    }
    if (base + step < a.r1) fetch(base + step);
    float s[2 * K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      E s0 = splat<E>(0.f), s1 = s0;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        E f[M], g[M];
        P::unpack(xr[k][i], f);
        P::unpack(yr[k][i], g);  // 0 where there is no channel: nothing is added there
#pragma unroll
        for (int c = 0; c < M; ++c) {
          const E u = vmul(vadd(f[c], splat<E>(-mean[k])), splat<E>(rstd[k]));
          const E t = vmul(g[c], w[i][c]);
          s0 = vadd(s0, t);
          s1 = vfma(t, u, s1);
          dw[i][c] = vfma(g[c], u, dw[i][c]);
          db[i][c] = vadd(db[i][c], g[c]);
        }
      }
      s[2 * k] = both(s0);
      s[2 * k + 1] = both(s1);
    }
    row_sum<2 * K>(s, p.lanes, p.warps, sm, turn);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const long long r = base + a.slot + (long long)k * a.slots;
      if (r >= a.r1) break;
      const E mt = splat<E>(-s[2 * k] * p.inv_c), mu = splat<E>(-s[2 * k + 1] * p.inv_c);
      T* dx = static_cast<T*>(p.y) + r * p.y_row;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int j = a.me + i * a.per_row;
        if (j >= a.packs) break;
        E f[M], g[M];
        forget(xr[k][i]);
        forget(yr[k][i]);
        P::unpack(xr[k][i], f);
        P::unpack(yr[k][i], g);
#pragma unroll
        for (int c = 0; c < M; ++c) {
          const E u = vmul(vadd(f[c], splat<E>(-mean[k])), splat<E>(rstd[k]));
          f[c] = vmul(splat<E>(rstd[k]), vfma(u, mu, vfma(g[c], w[i][c], mt)));
        }
        reinterpret_cast<typename P::Raw*>(dx)[j] = P::pack(f);
      }
    }
  }
  if (p.dweight == nullptr && p.dbias == nullptr) return;
  // one block a group: the gradients themselves; several: this block's part
  float* to_w = p.splits == 1 ? (p.dweight != nullptr ? p.dweight + a.group * p.C : nullptr)
                              : p.part + (long long)blockIdx.x * 2 * p.C;
  float* to_b = p.splits == 1 ? (p.dbias != nullptr ? p.dbias + a.group * p.C : nullptr) : to_w + p.C;
  if (a.slots == 1) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = a.me + i * a.per_row;
      if (j >= a.packs) break;
      if (to_w != nullptr) store_f32(to_w + j * N, dw[i]);
      if (to_b != nullptr) store_f32(to_b + j * N, db[i]);
    }
    return;
  }
  // channels of several row slots, added in the slots' order
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    __syncthreads();
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int j = a.me + i * a.per_row;
      if (j < a.packs) {
        float* to = sm + a.slot * p.C + j * N;
#pragma unroll
        for (int c = 0; c < M; ++c) *reinterpret_cast<E*>(to + c * (N / M)) = t == 0 ? dw[i][c] : db[i][c];
      }
    }
    __syncthreads();
    float* to = t == 0 ? to_w : to_b;
    if (to != nullptr)
      for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float v = 0.f;
        for (int k = 0; k < a.slots; ++k) v += sm[k * p.C + c];
        to[c] = v;
      }
  }
}

// Sum of a group's partial rows: part [groups][splits][2][C].  32 V channels x S
// shares of the splits a block; the shares are added in their order.
template <int V, int S>
__global__ void __launch_bounds__(32 * S) norm_sums_kernel(const __grid_constant__ NormParams p) {
  __shared__ float sm[S][V][32];
  griddep_launch_dependents();
  griddep_wait();
  const int lane = threadIdx.x & 31, share = threadIdx.x >> 5;
  const int blocks = (p.C + 32 * V - 1) / (32 * V);
  const long long unit = blockIdx.x / blocks;  // group and tensor
  const int c = ((int)(blockIdx.x - unit * blocks) * 32 + lane) * V;
  const long long group = unit >> 1;
  const int t = (int)(unit & 1);
  float* to = t == 0 ? p.dweight : p.dbias;
  if (to == nullptr) return;
  const float* from = p.part + (group * p.splits * 2 + t) * (long long)p.C + c;
  float a[V] = {};
  if (c < p.C)
#pragma unroll 8
    for (int s = share; s < p.splits; s += S) {
      float x[V];
      if constexpr (V == 4)
        *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(from + (long long)s * 2 * p.C);
      else
        x[0] = from[(long long)s * 2 * p.C];
#pragma unroll
      for (int v = 0; v < V; ++v) a[v] += x[v];
    }
#pragma unroll
  for (int v = 0; v < V; ++v) sm[share][v][lane] = a[v];
  __syncthreads();
  if (share < V && c < p.C) {  // warp v adds the v-th of each lane's channels
    float sum = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) sum += sm[k][share][lane];
    to[group * p.C + c + share] = sum;
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

// Cuts every group's rows so that all groups together make one wave of
// `resident` blocks an SM, in ranges of whole steps of `step` rows; at most
// `most` ranges a group.
void cut(NormParams& p, long long step, int resident, int sms, long long most) {
  const long long steps = (p.group_rows + step - 1) / step;
  const long long splits = std::max(1LL, std::min({steps, most, (long long)sms * resident / p.groups}));
  p.split_rows = (steps + splits - 1) / splits * step;
  p.splits = (int)((p.group_rows + p.split_rows - 1) / p.split_rows);
}
template <typename K>
int resident_blocks(K kernel, int threads, size_t smem) {
  int n = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&n, kernel, threads, smem) != cudaSuccess) n = 1;
  return std::max(1, n);
}

// Threads of a row and of a block for NV accesses a thread; `threads` is 256
// where a warp or less holds a row, but no more row slots than a group has
// rows for.
int block_threads(NormParams& p, int packs, int nv, int k) {
  p.lanes = 32;
  p.warps = (packs + 32 * nv - 1) / (32 * nv);
  while (p.warps == 1 && packs * 2 <= p.lanes) p.lanes /= 2;
  if (p.warps > 1) return 32 * p.warps;
  int threads = 256;
  while (threads > 32 && (long long)(threads / 2 / p.lanes) * k >= p.group_rows) threads /= 2;
  return threads;
}

// One instance each: NV accesses a thread, K rows at a time, blocks of at most
// MAXT threads.
template <typename T, int A, int NV, int K, int MAXT>
cudaError_t forward(NormParams& p, int sms, cudaStream_t s) {
  const int threads = block_threads(p, p.C / Pack<T, A>::N, NV, K);
  if (threads > MAXT) return cudaErrorInvalidValue;
  static std::atomic<int> held[33];  // blocks an SM holds, by warps a block
  std::atomic<int>& h = held[threads / 32];
  if (h.load() == 0) h.store(resident_blocks(norm_kernel<T, A, NV, K, MAXT>, threads, 0));
  cut(p, (long long)(threads / (p.lanes * p.warps)) * K, h.load(), sms, p.rows);
  return launch(norm_kernel<T, A, NV, K, MAXT>, p.groups * p.splits, threads, 0, p, s);
}
template <typename T, int A, int NV, int K, int MAXT, int MINB = 0>
cudaError_t backward(NormParams& p, int sms, cudaStream_t s) {
  const auto kernel = norm_back_kernel<T, A, NV, K, MAXT, MINB>;
  const int threads = block_threads(p, p.C / Pack<T, A>::N, NV, K);
  if (threads > MAXT) return cudaErrorInvalidValue;
  const int slots = threads / (p.lanes * p.warps);
  const size_t smem = sizeof(float) * (slots > 1 ? (size_t)slots * p.C : 2 * 32 * 2 * K);
  static std::atomic<int> held[33];
  std::atomic<int>& h = held[threads / 32];
  if (h.load() == 0) h.store(resident_blocks(kernel, threads, 16384));
  cut(p, (long long)slots * K, h.load(), sms, p.splits);
  const cudaError_t e = launch(kernel, p.groups * p.splits, threads, smem, p, s);
  if (e != cudaSuccess || p.splits == 1 || (p.dweight == nullptr && p.dbias == nullptr)) return e;
  // 20000 x 1536 bf16 of one group: 46.3 us with 8 shares, 40.3 with 32; 61440 x 1536
  // of 40 groups, 15 ranges each: 105.4 us with a channel a lane, 103.0 with four
  if (p.splits > 16) return launch(norm_sums_kernel<1, 32>, p.groups * 2 * ((p.C + 31) / 32), 1024, 0, p, s);
  if (p.C % 4 == 0) return launch(norm_sums_kernel<4, 8>, p.groups * 2 * ((p.C + 127) / 128), 256, 0, p, s);
  return launch(norm_sums_kernel<1, 8>, p.groups * 2 * ((p.C + 31) / 32), 256, 0, p, s);
}

// Which instance: what counts is bytes in flight an SM against the cost of a
// barrier, which a thread's work has to cover.  61440 x 1536 bf16, forward, by
// accesses a thread x rows: 1 x 4 77 us, 2 x 4 64, 3 x 2 63, 4 x 2 75, 6 x 1
// 89; backward 1 x 4 111, 2 x 2 105, 3 x 1 112, 6 x 1 156.  61440 x 1024 fp32
// (half the arithmetic a byte): forward 1 x 4 81, 3 x 2 82; backward 1 x 4 119,
// 2 x 2 122.  Wider rows take more accesses a thread, so that 16 warps hold them.
template <typename T, int A>
cudaError_t pick(NormParams& p, bool back, int sms, cudaStream_t s) {
  const int packs = p.C / Pack<T, A>::N;
  constexpr bool kHalf = sizeof(T) == 2;
  if constexpr (A == 16) {
    if (packs <= 32 || (!kHalf && packs <= 256))
      return back ? backward<T, A, 1, 4, 256>(p, sms, s) : forward<T, A, 1, 4, 256>(p, sms, s);
    if (back) {
      if (packs <= 512) return backward<T, A, 2, 2, 256>(p, sms, s);
      if (packs <= 640) return backward<T, A, 2, 1, 320, 2>(p, sms, s);
      if constexpr (kHalf)
        return backward<T, A, 2, 1, 512>(p, sms, s);
      else
        return backward<T, A, 4, 1, 512>(p, sms, s);
    }
    if (packs <= 512 && !kHalf) return forward<T, A, 2, 2, 256>(p, sms, s);
    if (kHalf && packs <= 512) {  // the fewest empty places, 3 accesses a thread where as few
      const int w2 = (packs + 63) / 64 * 64, w3 = (packs + 95) / 96 * 96;
      return w3 <= w2 ? forward<T, A, 3, 2, 256>(p, sms, s) : forward<T, A, 2, 2, 256>(p, sms, s);
    }
    return forward<T, A, 4, 1, 512>(p, sms, s);
  } else {
    if (packs <= 32) return back ? backward<T, A, 1, 4, 256>(p, sms, s) : forward<T, A, 1, 4, 256>(p, sms, s);
    if (packs <= 1024) return back ? backward<T, A, 4, 4, 256>(p, sms, s) : forward<T, A, 4, 4, 256>(p, sms, s);
    if (packs <= 4096) return back ? backward<T, A, 8, 1, 512>(p, sms, s) : forward<T, A, 8, 2, 512>(p, sms, s);
    if constexpr (Pack<T, A>::N == 1)
      return back ? backward<T, A, 16, 1, 512>(p, sms, s) : forward<T, A, 16, 1, 512>(p, sms, s);
    return cudaErrorInvalidValue;
  }
}

}  // namespace

cudaError_t launch_layer_norm(NormParams& p, bool fp32, int access, bool back, int sms, cudaStream_t s) {
  if (fp32) return access == 16 ? pick<float, 16>(p, back, sms, s) : pick<float, 4>(p, back, sms, s);
  if (access == 16) return pick<uint16_t, 16>(p, back, sms, s);
  return access == 4 ? pick<uint16_t, 4>(p, back, sms, s) : pick<uint16_t, 2>(p, back, sms, s);
}

}  // namespace sab
