// Decay attention (see include/sab.h, sab_decay_attention): linear attention
// with a decay per head, its single-token form and its gradients.
//
// Per (b, h), with g = exp(log_decay[h]) and a D x D state S:
//   S_t = g S_{t-1} + k_t v_t^T,   o_t = scale q_t S_t.
// The gradients are three runs of the same recurrence on other operands:
//   dq = run(dO, V, K) forward on the transposed state;
//   dv = run(K, Q, dO) and dk = run(V, dO, Q) backward in time, the second on
//   the transposed state; there the state is the gradient of S, and it decays
//   after the token instead of before it.
#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }
__device__ __forceinline__ uint16_t to_bf(float x) { return (uint16_t)(ptx::pack_bf16(x, 0.f) & 0xFFFFu); }

// log of the decay per token, clamped to [-10^4, 0] (NaN stays)
__device__ __forceinline__ float decay_ln(const float* log_decay, int h) {
  const float x = __ldg(log_decay + h);
  return x > 0.f ? 0.f : x < -1e4f ? -1e4f : x;
}
// exp(x) for x <= 0 as a rounded value and the rest.  Multiplying a state by
// the rounded value alone would repeat its error of up to 2^-25 at every token
// (10^4 tokens with a decay near 1: 3e-4).  Above 1/2 the rest is
// (1 - hi) - (1 - exp(x)), the first difference exact; below, the state is
// gone before the error adds up.
struct Decay {
  float hi, lo;
  __device__ __forceinline__ explicit Decay(float x) : hi(expf(x)), lo(0.f) {
    if (hi >= 0.5f) lo = (1.f - hi) + expm1f(x);
  }
  __device__ __forceinline__ float operator()(float s) const { return fmaf(s, hi, s * lo); }
};

// Token-by-token run: one CTA per (b, h) and 32 value columns, the state in
// registers.  A warp owns D / 8 key rows, a lane one value column.
constexpr int kScanTokens = 16;
template <int D>
__global__ void __launch_bounds__(256) decay_scan_kernel(const __grid_constant__ DecayParams p) {
  constexpr int R = D / 8;
  __shared__ float sq[kScanTokens][D], sk[kScanTokens][D], sv[kScanTokens][32];
  __shared__ float part[8][kScanTokens][32];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long bh = blockIdx.x;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int col = blockIdx.y * 32 + lane;
  const int len = p.seq_len != nullptr ? min(max(__ldg(p.seq_len + b), 0), p.L) : p.L;
  const Decay decay(decay_ln(p.log_decay, h));
  float s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    const int row = warp * R + r;
    s[r] = p.state_in == nullptr ? 0.f
                                 : p.state_in[(bh * D + (p.state_t ? col : row)) * D + (p.state_t ? row : col)];
  }
  const long long base = (long long)b * p.L;
  for (int c0 = 0; c0 < len; c0 += kScanTokens) {
    const int n = min(kScanTokens, len - c0);
    auto token = [&](int i) { return p.reverse ? len - 1 - (c0 + i) : c0 + i; };
    __syncthreads();
    for (int i = threadIdx.x; i < n * D; i += 256) {
      const int t = i / D, d = i % D;
      const long long e = ((base + token(t)) * p.H + h) * D + d;
      sq[t][d] = bf(p.q[e]);
      sk[t][d] = bf(p.k[e]) * p.kv_mul;
    }
    for (int i = threadIdx.x; i < n * 32; i += 256)
      sv[i >> 5][i & 31] = bf(p.v[((base + token(i >> 5)) * p.H + h) * D + blockIdx.y * 32 + (i & 31)]);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float v = sv[t][lane];
      float o = 0.f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float x = s[r];
        if (!p.reverse) x = decay(x);
        x = fmaf(sk[t][warp * R + r], v, x);
        o = fmaf(sq[t][warp * R + r], x, o);
        s[r] = p.reverse ? decay(x) : x;
      }
      part[warp][t][lane] = o;
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * 32; i += 256) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) o += part[w][i >> 5][i & 31];
      p.o[((base + token(i >> 5)) * p.H + h) * D + blockIdx.y * 32 + (i & 31)] = to_bf(o * p.o_mul);
    }
  }
  for (int t = len + warp; t < p.L; t += 8) p.o[((base + t) * p.H + h) * D + col] = 0;
  if (p.state_out != nullptr) {
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int row = warp * R + r;
      p.state_out[(bh * D + (p.state_t ? col : row)) * D + (p.state_t ? row : col)] = s[r];
    }
  }
}

// One token: the state passes once through registers.  One CTA per (b, h)
// and W value columns; W / 4 lanes hold a row's columns as 16-byte vectors, so
// a warp reads 128 / W whole row pieces at a time.  Bound by the state's
// bytes (read and written once); W = 32 spreads few heads over the SMs.
template <int D, int W>
__global__ void __launch_bounds__(256) decay_step_kernel(const __grid_constant__ DecayStepParams p) {
  constexpr int kLanes = W / 4;              // lanes per row
  constexpr int kRows = 256 / kLanes;        // rows per pass
  constexpr int kPasses = D / kRows;
  __shared__ float sq[D], sk[D];
  __shared__ float4 part[8][kLanes];
  ptx::griddep_launch_dependents();
  ptx::griddep_wait();
  const long long bh = blockIdx.x;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c4 = tid % kLanes, row0 = tid / kLanes;
  const int col = blockIdx.y * W + 4 * c4;
  const bool on = p.active == nullptr || __ldg(p.active + b) != 0;
  const float* in = p.state_in + bh * D * D;
  float* out = p.state_out + bh * D * D;
  if (!on && p.state_in == p.state_out) {  // nothing moves
    if (tid < kLanes) *reinterpret_cast<uint2*>(p.o + bh * D + col) = make_uint2(0u, 0u);
    return;
  }
  float4 s[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i)
    s[i] = p.state_in == nullptr ? make_float4(0.f, 0.f, 0.f, 0.f)
                                 : *reinterpret_cast<const float4*>(in + (row0 + i * kRows) * D + col);
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  if (on) {
    for (int i = tid; i < D; i += 256) {
      sq[i] = bf(p.q[bh * D + i]) * p.scale;
      sk[i] = bf(p.k[bh * D + i]);
    }
    const uint2 vw = *reinterpret_cast<const uint2*>(p.v + bh * D + col);
    const float v[4] = {__uint_as_float(vw.x << 16), __uint_as_float(vw.x & 0xFFFF0000u), __uint_as_float(vw.y << 16),
                        __uint_as_float(vw.y & 0xFFFF0000u)};
    const Decay decay(decay_ln(p.log_decay, h));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const float k = sk[row0 + i * kRows], q = sq[row0 + i * kRows];
      s[i].x = fmaf(k, v[0], decay(s[i].x));
      s[i].y = fmaf(k, v[1], decay(s[i].y));
      s[i].z = fmaf(k, v[2], decay(s[i].z));
      s[i].w = fmaf(k, v[3], decay(s[i].w));
      acc.x = fmaf(q, s[i].x, acc.x);
      acc.y = fmaf(q, s[i].y, acc.y);
      acc.z = fmaf(q, s[i].z, acc.z);
      acc.w = fmaf(q, s[i].w, acc.w);
    }
  }
#pragma unroll
  for (int i = 0; i < kPasses; ++i) *reinterpret_cast<float4*>(out + (row0 + i * kRows) * D + col) = s[i];
  // sum over the rows: lanes of a warp that share columns, then the warps
#pragma unroll
  for (int o = kLanes; o < 32; o <<= 1) {
    acc.x += __shfl_xor_sync(0xffffffffu, acc.x, o);
    acc.y += __shfl_xor_sync(0xffffffffu, acc.y, o);
    acc.z += __shfl_xor_sync(0xffffffffu, acc.z, o);
    acc.w += __shfl_xor_sync(0xffffffffu, acc.w, o);
  }
  if (lane < kLanes) part[warp][lane] = acc;
  __syncthreads();
  if (tid < kLanes) {
    float4 o = part[0][tid];
#pragma unroll
    for (int w = 1; w < 8; ++w) {
      const float4 a = part[w][tid];
      o.x += a.x;
      o.y += a.y;
      o.z += a.z;
      o.w += a.w;
    }
    *reinterpret_cast<uint2*>(p.o + bh * D + col) = make_uint2(ptx::pack_bf16(o.x, o.y), ptx::pack_bf16(o.z, o.w));
  }
}

template <typename P>
cudaError_t launch(void (*kernel)(P), dim3 grid, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(256, 1, 1);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

}  // namespace

cudaError_t launch_decay_run(const DecayParams& p, cudaStream_t s) {
  const dim3 grid((unsigned)((long long)p.B * p.H), p.D / 32, 1);
  return p.D == 128 ? launch(decay_scan_kernel<128>, grid, p, s) : launch(decay_scan_kernel<64>, grid, p, s);
}

cudaError_t launch_decay_step(const DecayStepParams& p, cudaStream_t s) {
  const long long bh = (long long)p.B * p.H;
  const dim3 grid((unsigned)bh, p.D / 32, 1);
  return p.D == 128 ? launch(decay_step_kernel<128, 32>, grid, p, s) : launch(decay_step_kernel<64, 32>, grid, p, s);
}

}  // namespace sab
