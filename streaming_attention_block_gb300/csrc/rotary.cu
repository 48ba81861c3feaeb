// Rotary positions of queries and keys, and their gradient (see
// include/sab.h, sab_rotary): an HBM stream, every element read and written
// once, q and k in one launch.
//
// A block takes a few tokens.  Their sines and cosines (one per token and
// pair, shared by every head of q and k) are worked out first into shared
// memory; then every thread moves 16-byte vectors, at a fixed place of the
// head, over the tokens' heads.  The angle of position p is p * f turns
// modulo one turn.  f is a 64-bit fraction of a turn, so the product wraps by
// itself, and its upper 32 bits, as a signed fraction, go to sincospif:
// exact range reduction for any int64 position without fp64 arithmetic.
#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxTokens = 8;   // tokens per block
constexpr int kBatch = 4;       // vectors in flight per thread

__device__ __forceinline__ float bf_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// 16 bytes <-> fp32 values
template <typename T>
struct Vec;
template <>
struct Vec<uint16_t> {  // bf16
  static constexpr int N = 8;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = bf_lo(w[i]);
      x[2 * i + 1] = bf_hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[8]) {
    return make_uint4(ptx::pack_bf16(x[0], x[1]), ptx::pack_bf16(x[2], x[3]), ptx::pack_bf16(x[4], x[5]),
                      ptx::pack_bf16(x[6], x[7]));
  }
  static __device__ __forceinline__ float load(const uint16_t* p) { return bf_lo((uint32_t)*p); }
  static __device__ __forceinline__ void store(uint16_t* p, float x) {
    *p = (uint16_t)(ptx::pack_bf16(x, 0.f) & 0xFFFFu);
  }
};
template <>
struct Vec<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ void unpack(const uint4& v, float (&x)[4]) {
    x[0] = __uint_as_float(v.x);
    x[1] = __uint_as_float(v.y);
    x[2] = __uint_as_float(v.z);
    x[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[4]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float load(const float* p) { return *p; }
  static __device__ __forceinline__ void store(float* p, float x) { *p = x; }
};

__device__ __forceinline__ void turn(float2 cs, float a, float b, float& ra, float& rb) {
  ra = a * cs.x - b * cs.y;
  rb = a * cs.y + b * cs.x;
}

enum Mode { kInterleaved, kHalfVec, kHalfScalar };

// A head's work is cut into `units`, one per thread column:
//   kInterleaved  the head's D / N vectors; a vector holds whole pairs
//   kHalfVec      (dims / 2 a multiple of N) one unit per vector of first
//                 elements together with its vector of second elements, then
//                 one per vector behind `dims`
//   kHalfScalar   one unit per pair, then one per element behind `dims`: the
//                 halves do not start on a 16-byte boundary
template <typename T, Mode M>
__global__ void __launch_bounds__(kMaxThreads) rotary_kernel(const __grid_constant__ RotaryParams p) {
  using V = Vec<T>;
  constexpr int N = V::N;
  __shared__ __align__(16) float2 cs[kMaxTokens * kRotaryMaxPairs];
  ptx::griddep_launch_dependents();
  const int half = p.dims >> 1;
  const long long tokens = (long long)p.B * p.L;
  const long long tok0 = (long long)blockIdx.x * p.tokens;
  const int ntok = (int)min((long long)p.tokens, tokens - tok0);
  const int heads = p.rows[0].heads + p.rows[1].heads;
  const int unit = (int)threadIdx.x % p.units, group = (int)threadIdx.x / p.units;
  const int groups = (int)blockDim.x / p.units;
  ptx::griddep_wait();

  // this thread's rows: (token, head) = (k, h), stepping by `groups` heads
  struct Item {
    const T* in;
    T* out;
    int k;
  };
  int k_next = group / heads, h_next = group - k_next * heads;
  auto next_row = [&]() {
    Item r{nullptr, nullptr, k_next};
    if (k_next < ntok) {
      const long long tok = tok0 + k_next;
      const long long b = p.B == 1 ? 0 : tok / p.L, t = tok - b * p.L;
      const int w = h_next >= p.rows[0].heads;
      const int h = w ? h_next - p.rows[0].heads : h_next;
      const RotaryRows& x = p.rows[w];
      r.in = static_cast<const T*>(x.in) + b * x.in_batch + t * x.in_token + (long long)h * p.D;
      r.out = static_cast<T*>(x.out) + b * x.out_batch + t * x.out_token + (long long)h * p.D;
      h_next += groups;
      while (h_next >= heads) h_next -= heads, ++k_next;
    }
    return r;
  };

  // element offset of the unit's first vector; a kHalfVec pair unit's second
  // vector lies `half` elements further
  const bool pairs = M == kHalfVec && unit < half / N;
  const int e0 = (M == kHalfVec && !pairs) ? unit * N + half : unit * N;
  Item row[kBatch];
  uint4 va[kBatch], vb[kBatch];
  auto fetch = [&]() {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      row[u] = next_row();
      if (M != kHalfScalar && row[u].in != nullptr) {
        va[u] = *reinterpret_cast<const uint4*>(row[u].in + e0);
        if (pairs) vb[u] = *reinterpret_cast<const uint4*>(row[u].in + e0 + half);
      }
    }
  };
  fetch();  // in flight while the angles are worked out

  // sine and cosine of every (token, pair)
  for (int i = threadIdx.x; i < ntok * half; i += blockDim.x) {
    const int k = i / half, j = i - k * half;
    const long long tok = tok0 + k;
    const long long pos = p.positions != nullptr ? __ldg(p.positions + (long long)p.axis[j] * tokens + tok)
                                                 : p.first_position + tok % p.L;
    const unsigned long long turns = (unsigned long long)pos * p.step[j];
    float s, c;
    sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
    cs[k * half + j] = make_float2(c * p.magnitude, s * p.sine);
  }
  __syncthreads();

  while (row[0].in != nullptr) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (row[u].in == nullptr) break;
      const float2* c = cs + row[u].k * half;
      if constexpr (M == kHalfScalar) {
        const T* in = row[u].in;
        T* out = row[u].out;
        if (unit < half) {
          float x, y;
          turn(c[unit], V::load(in + unit), V::load(in + unit + half), x, y);
          V::store(out + unit, x);
          V::store(out + unit + half, y);
        } else {
          out[unit + half] = in[unit + half];
        }
      } else {
        float a[N];
        V::unpack(va[u], a);
        if constexpr (M == kInterleaved) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j)
            if (e0 + 2 * j < p.dims) turn(c[e0 / 2 + j], a[2 * j], a[2 * j + 1], a[2 * j], a[2 * j + 1]);
        } else if (pairs) {
          float b[N];
          V::unpack(vb[u], b);
#pragma unroll
          for (int j = 0; j < N; ++j) turn(c[e0 + j], a[j], b[j], a[j], b[j]);
          *reinterpret_cast<uint4*>(row[u].out + e0 + half) = V::pack(b);
        }
        *reinterpret_cast<uint4*>(row[u].out + e0) = V::pack(a);
      }
    }
    fetch();
  }
}

template <typename T, Mode M>
cudaError_t launch(RotaryParams& p, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int half = p.dims / 2;
  p.units = M == kInterleaved ? p.D / N : M == kHalfVec ? half / N + (p.D - p.dims) / N : half + p.D - p.dims;
  const int threads = p.units > kMaxThreads ? kMaxThreads : kMaxThreads / p.units * p.units;
  const int heads = p.rows[0].heads + p.rows[1].heads, groups = threads / p.units;
  const long long tokens = (long long)p.B * p.L;
  // tokens per block: as few whole batches of rows per thread as leave the
  // fewest idle slots in the last one, but a block for every SM before that
  int best = 1;
  double waste = 2.0;
  for (int t = 1; t <= kMaxTokens && (t == 1 || tokens / t >= 2 * 152); ++t) {
    const int slots = kBatch * groups, rows = t * heads;
    const double w = (double)((rows + slots - 1) / slots * slots) / rows;
    if (w < waste - 0.02) best = t, waste = w;
  }
  p.tokens = best;
  const long long blocks = (tokens + p.tokens - 1) / p.tokens;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)threads, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T, M>, p);
}

template <typename T>
cudaError_t launch_layout(RotaryParams& p, cudaStream_t s) {
  if (!p.half_layout) return launch<T, kInterleaved>(p, s);
  return (p.dims / 2) % Vec<T>::N == 0 ? launch<T, kHalfVec>(p, s) : launch<T, kHalfScalar>(p, s);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams& p, bool fp32, cudaStream_t s) {
  return fp32 ? launch_layout<float>(p, s) : launch_layout<uint16_t>(p, s);
}

}  // namespace sab
