// Rotary positions of queries and keys, and their gradient (see
// include/sab.h, sab_rotary): an HBM stream, every element read and written
// once, q and k in one launch.
//
// A block takes a few tokens.  Their sines and cosines (one per token and
// pair, shared by every head of q and k) are worked out first into shared
// memory, while the first data loads are in flight; then a thread keeps one
// token and one place of the head, holds that place's factors in registers
// and walks over heads, so that the stream, not the issue slots, sets the pace:
// 2 x 30720 tokens of 24 heads of 128 in 112 us, 755 MB at 6.7 TB/s, the copy
// rate (237 us with every vector's factors read from shared memory and its
// place worked out anew).  The angle of position p is
// p * f turns modulo one turn.  f is a 64-bit fraction of a turn, so the
// product wraps by itself, and its upper 32 bits, as a signed fraction, go to
// sincospif: exact range reduction for any int64 position without fp64.
#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kMaxTokens = 8;   // tokens per block

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

// (a, b) turned by cs = (cos, sin): two packed products
__device__ __forceinline__ void turn(float2 cs, float& a, float& b) {
  const float2 r = __ffma2_rn(make_float2(b, a), make_float2(-cs.y, cs.y),
                              __fmul2_rn(make_float2(a, b), make_float2(cs.x, cs.x)));
  a = r.x;
  b = r.y;
}

enum Mode { kInterleaved, kHalfVec, kHalfScalar };
constexpr int kBatch = 4;  // rows in flight per thread

// A head's work is cut into `units`, one per thread column:
//   kInterleaved  the head's D / N vectors; a vector holds whole pairs
//   kHalfVec      (dims / 2 a multiple of N) a vector of first elements with
//                 its vector of second elements; behind `dims`, two vectors
//   kHalfScalar   one pair, or one element behind `dims`: the halves do not
//                 start on a 16-byte boundary.  One element per access and one
//                 pair in flight: 4 x 8191 tokens of 40 heads of 80, 20 rotated,
//                 in 426 us (0.98 TB/s; 32 rotated, kHalfVec: 68 us, 6.2 TB/s)
// A block's columns of `units` threads take one token and every p.splits-th
// head each.
// (Blocks per SM: four of 64 registers for one vector per row, three of 80 for
// two.  Fewer rows in flight cost more than fewer blocks: 4 x 8191 tokens of 32
// heads, 89 us with 4 rows and 2 blocks, 102 us with 2 and 3, 138 us with 1 and
// 4; 81 us with 4 and 3, see kKeep.)
template <typename T, Mode M>
__global__ void __launch_bounds__(kMaxThreads, M == kHalfVec ? 3 : 4)
rotary_kernel(const __grid_constant__ RotaryParams p) {
  using V = Vec<T>;
  constexpr int N = V::N;
  constexpr int kPairs = M == kInterleaved ? N / 2 : M == kHalfVec ? N : 1;  // pairs of a unit
  __shared__ __align__(16) float2 cs[kMaxTokens * kRotaryMaxPairs];
  ptx::griddep_launch_dependents();
  const int half = p.dims >> 1;
  const unsigned tokens = (unsigned)p.B * (unsigned)p.L;  // at most 2^31
  const unsigned tok0 = blockIdx.x * (unsigned)p.tokens;
  const int ntok = (int)min((unsigned)p.tokens, tokens - tok0);
  const int unit = (int)threadIdx.x % p.units, column = (int)threadIdx.x / p.units;
  const int k = column / p.splits;             // token of the block
  const bool active = k < ntok;
  const int heads = p.rows[0].heads + p.rows[1].heads;
  const T *in0 = nullptr, *in1 = nullptr;      // the token's rows of q and k
  T *out0 = nullptr, *out1 = nullptr;
  if (active) {
    const unsigned tok = tok0 + (unsigned)k;
    const long long b = tok / (unsigned)p.L, t = tok - (unsigned)b * (unsigned)p.L;
    in0 = static_cast<const T*>(p.rows[0].in) + b * p.rows[0].in_batch + t * p.rows[0].in_token;
    out0 = static_cast<T*>(p.rows[0].out) + b * p.rows[0].out_batch + t * p.rows[0].out_token;
    in1 = static_cast<const T*>(p.rows[1].in) + b * p.rows[1].in_batch + t * p.rows[1].in_token;
    out1 = static_cast<T*>(p.rows[1].out) + b * p.rows[1].out_batch + t * p.rows[1].out_token;
  }
  // elements e0 .. (first vector or element) and e1 .. (second, if any) of a
  // head, and the number of the unit's pairs that turn
  const bool rot = M == kInterleaved ? unit * N < p.dims : unit < half / (M == kHalfVec ? N : 1);
  int e0 = unit * N, e1 = -1, turns_here = kPairs;
  if constexpr (M == kInterleaved) {
    turns_here = rot ? min(kPairs, half - unit * kPairs) : 0;
  } else if constexpr (M == kHalfVec) {
    // (neighbouring units on neighbouring vectors: whole sectors per access)
    if (!rot) e0 += half;
    e1 = rot ? e0 + half : e0 + (p.units - half / N) * N;
    if (e1 >= p.D) e1 = -1;
  } else {
    e0 = rot ? unit : unit + half;
    e1 = rot ? unit + half : -1;
  }
  ptx::griddep_wait();

  // A row's places: kept from the load to the store, except that kHalfVec works
  // them out anew, which frees the registers for its third block.  (With it 4 x
  // 8191 tokens of 32 heads go from 95 to 87 us, L2 flushed; in kInterleaved 2 x
  // 30720 tokens of 24 heads would go from 117 to 148.)
  constexpr bool kKeep = M != kHalfVec;
  const T* src[kBatch];
  T* dst[kBatch];
  uint4 va[kBatch], vb[kBatch];
  const int hq = p.rows[0].heads;
  int h = active ? column % p.splits : heads;  // next head to fetch
  int first = h;                               // this batch's first
  auto fetch = [&]() {
    if (!kKeep) first = h;
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      dst[u] = nullptr;
      if (h < heads) {
        const bool w = h >= hq;
        const int e = (w ? h - hq : h) * p.D;
        src[u] = (w ? in1 : in0) + e;
        dst[u] = (w ? out1 : out0) + e;
        h += p.splits;
        if constexpr (M != kHalfScalar) {
          va[u] = *reinterpret_cast<const uint4*>(src[u] + e0);
          if (M == kHalfVec && e1 >= 0) vb[u] = *reinterpret_cast<const uint4*>(src[u] + e1);
        }
      }
    }
  };
  fetch();

  // sine and cosine of every (token, pair)
  const int cols = min(half, (int)blockDim.x), lines = (int)blockDim.x / cols, line = (int)threadIdx.x / cols;
  if (line < lines) {
    for (int j = (int)threadIdx.x - line * cols; j < half; j += cols) {
      const unsigned long long step = p.step[j];
      const long long* pos_j = p.positions != nullptr ? p.positions + (long long)p.axis[j] * tokens : nullptr;
      for (int kk = line; kk < ntok; kk += lines) {
        const unsigned tok = tok0 + (unsigned)kk;
        const long long pos = pos_j != nullptr ? __ldg(pos_j + tok) : p.first_position + tok % (unsigned)p.L;
        const unsigned long long turns = (unsigned long long)pos * step;
        float s, c;
        sincospif((float)(int)(turns >> 32) * 0x1p-31f, &s, &c);
        cs[kk * half + j] = make_float2(c * p.magnitude, s * p.sine);
      }
    }
  }
  __syncthreads();
  if (!active) return;
  float2 f[kPairs];
#pragma unroll
  for (int j = 0; j < kPairs; ++j)
    f[j] = rot && j < turns_here ? cs[k * half + unit * kPairs + j] : make_float2(0.f, 0.f);

  while (kKeep ? dst[0] != nullptr : first < heads) {
#pragma unroll
    for (int u = 0; u < kBatch; ++u) {
      if (kKeep ? dst[u] == nullptr : first + u * p.splits >= heads) break;
      T* to = dst[u];
      if (!kKeep) {
        const int hu = first + u * p.splits;
        to = hu < hq ? out0 + hu * p.D : out1 + (hu - hq) * p.D;
      }
      if constexpr (M == kHalfScalar) {
        if (rot) {
          float x = V::load(src[u] + e0), y = V::load(src[u] + e1);
          turn(f[0], x, y);
          V::store(to + e0, x);
          V::store(to + e1, y);
        } else {
          to[e0] = src[u][e0];
        }
      } else {
        if (rot) {
          float x[N], y[N];
          V::unpack(va[u], x);
          if constexpr (M == kInterleaved) {
#pragma unroll
            for (int j = 0; j < kPairs; ++j)
              if (j < turns_here) turn(f[j], x[2 * j], x[2 * j + 1]);
          } else {
            V::unpack(vb[u], y);
#pragma unroll
            for (int j = 0; j < kPairs; ++j) turn(f[j], x[j], y[j]);
            vb[u] = V::pack(y);
          }
          va[u] = V::pack(x);
        }
        *reinterpret_cast<uint4*>(to + e0) = va[u];
        if (M == kHalfVec && e1 >= 0) *reinterpret_cast<uint4*>(to + e1) = vb[u];
      }
    }
    fetch();
  }
}

template <typename T, Mode M>
cudaError_t launch(RotaryParams& p, int sms, cudaStream_t s) {
  constexpr int N = Vec<T>::N;
  const int half = p.dims / 2, rest = p.D - p.dims;
  p.units = M == kInterleaved ? p.D / N : M == kHalfVec ? half / N + (rest / N + 1) / 2 : half + rest;
  const int columns = kMaxThreads / p.units;
  const int heads = p.rows[0].heads + p.rows[1].heads;
  const long long tokens = (long long)p.B * p.L;
  // tokens per block: those that leave the fewest of the threads' batch slots
  // empty, but a block or two for every SM before that
  double best = 0.0;
  for (int t = 1; t <= kMaxTokens && t <= columns && (t == 1 || tokens / t >= 2 * sms); ++t) {
    const int splits = columns / t < heads ? columns / t : heads;
    const int rows = (heads + splits - 1) / splits;  // per thread
    const double used = (double)t * heads / ((double)columns * ((rows + kBatch - 1) / kBatch * kBatch));
    if (t == 1 || used > best + 0.01) best = used, p.tokens = t, p.splits = splits;
  }
  const long long blocks = (tokens + p.tokens - 1) / p.tokens;
  if (blocks > 0x7fffffffLL) return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)blocks, 1, 1);
  cfg.blockDim = dim3((unsigned)(p.tokens * p.splits * p.units), 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, rotary_kernel<T, M>, p);
}

template <typename T>
cudaError_t launch_layout(RotaryParams& p, int sms, cudaStream_t s) {
  if (!p.half_layout) return launch<T, kInterleaved>(p, sms, s);
  return (p.dims / 2) % Vec<T>::N == 0 ? launch<T, kHalfVec>(p, sms, s) : launch<T, kHalfScalar>(p, sms, s);
}

}  // namespace

cudaError_t launch_rotary(RotaryParams& p, bool fp32, int sms, cudaStream_t s) {
  return fp32 ? launch_layout<float>(p, sms, s) : launch_layout<uint16_t>(p, sms, s);
}

}  // namespace sab
