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
#include <atomic>

#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

using namespace ptx;

__device__ __forceinline__ float bf(uint16_t x) { return __uint_as_float((uint32_t)x << 16); }

// log of the decay per token, clamped to [-10^4, 0] (NaN stays)
__device__ __forceinline__ float decay_ln(const float* log_decay, int h) {
  const float x = __ldg(log_decay + h);
  return x > 0.f ? 0.f : x < -1e4f ? -1e4f : x;
}
// Whether a decay of ln per token is 0 in fp32: then, and only then, may a decay
// take an infinity with it (0 * inf is NaN).
__device__ __forceinline__ bool decays_to_zero(float ln) { return expf(ln) == 0.f; }
constexpr float kLeast = 0x1p-149f;  // the smallest positive fp32 number
// exp(x) for x <= 0 as a rounded value and the rest.  Multiplying a state by
// the rounded value alone would repeat its error of up to 2^-25 at every token
// (10^4 tokens with a decay near 1: 3e-4).  Above 1/2 the value is rounded down
// and the rest is (1 - hi) - (1 - exp(x)), the first difference exact; below,
// the state is gone before the error adds up.  Unless the decay is 0 for good
// (`zero`), both are positive, kLeast in place of 0: an infinite state stays
// infinite, and no finite state is moved by more than 1e-6.
struct Decay {
  float hi, lo;
  __device__ __forceinline__ Decay(float x, bool zero) : hi(expf(x)), lo(0.f) {
    if (hi >= 0.5f) {
      const float m = expm1f(x);
      hi = __fadd_rd(1.f, m);
      if (hi >= 0.5f) lo = (1.f - hi) + m;
    }
    if (!zero) {
      if (hi == 0.f) hi = kLeast;
      if (!(lo > 0.f)) lo = kLeast;
    }
  }
  __device__ __forceinline__ float operator()(float s) const { return fmaf(s, hi, s * lo); }
};
// over n tokens
__device__ __noinline__ Decay decay_over(int n, float ln) { return Decay((float)n * ln, decays_to_zero(ln)); }

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
  const long long bh = blockIdx.x / (D / W);
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int c4 = tid % kLanes, row0 = tid / kLanes;
  const int col = (int)(blockIdx.x % (D / W)) * W + 4 * c4;
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
    const float ln = decay_ln(p.log_decay, h);
    const Decay decay(ln, decays_to_zero(ln));
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

// Short runs, token by token in fp32: one CTA per (b, h) and 32 value columns,
// the state in registers (a warp owns D / 8 key rows, a lane one column).  The
// state passes once, a token costs 0.2 us (fp32 multiply-adds and broadcast
// reads), and nothing of the tile kernel's set-up is paid.
constexpr int kShortBatch = 16;  // tokens staged at a time
template <int D>
__global__ void __launch_bounds__(256, D == 128 ? 6 : 8) decay_short_kernel(const __grid_constant__ DecayTileParams p) {
  constexpr int R = D / 8;
  __shared__ __align__(16) float sq[kShortBatch][D], sk[kShortBatch][D], sv[kShortBatch][32];
  __shared__ float part[8][kShortBatch][32];
  griddep_launch_dependents();
  griddep_wait();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const long long bh = blockIdx.x / (D / 32);
  const int b = (int)(bh / p.H), h = (int)(bh % p.H), col0 = (int)(blockIdx.x % (D / 32)) * 32, col = col0 + lane;
  const int len = p.seq_len != nullptr ? min(max(__ldg(p.seq_len + b), 0), p.L) : p.L;
  const float ln = decay_ln(p.log_decay, h);
  const Decay decay(ln, decays_to_zero(ln));
  float s[R];
#pragma unroll
  for (int r = 0; r < R; ++r) s[r] = 0.f;
  if (p.state_in != nullptr) {
    const float* in = p.state_in + bh * D * D;
    if (p.state_t) {
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 x = *reinterpret_cast<const float4*>(in + col * D + warp * R + r);
        s[r] = x.x, s[r + 1] = x.y, s[r + 2] = x.z, s[r + 3] = x.w;
      }
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) s[r] = in[(warp * R + r) * D + col];
    }
  }
  const long long base = (long long)b * p.L;
  for (int c0 = 0; c0 < len; c0 += kShortBatch) {
    const int n = min(kShortBatch, len - c0);
    auto row_of = [&](int i) { return ((base + (p.reverse ? len - 1 - (c0 + i) : c0 + i)) * p.H + h) * D; };
    __syncthreads();
    for (int i = tid; i < n * (D / 8); i += 256) {
      const int t = i / (D / 8), d = i % (D / 8) * 8;
      const long long e = row_of(t) + d;
      const uint4 q = *reinterpret_cast<const uint4*>(p.q + e), k = *reinterpret_cast<const uint4*>(p.k + e);
      const uint32_t qw[4] = {q.x, q.y, q.z, q.w}, kw[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        sq[t][d + 2 * j] = __uint_as_float(qw[j] << 16);
        sq[t][d + 2 * j + 1] = __uint_as_float(qw[j] & 0xFFFF0000u);
        sk[t][d + 2 * j] = __uint_as_float(kw[j] << 16) * p.kv_mul;
        sk[t][d + 2 * j + 1] = __uint_as_float(kw[j] & 0xFFFF0000u) * p.kv_mul;
      }
    }
    for (int i = tid; i < n * 32; i += 256) sv[i >> 5][i & 31] = bf(p.v[row_of(i >> 5) + col0 + (i & 31)]);
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const float v = sv[t][lane];
      float o = 0.f;
#pragma unroll
      for (int r = 0; r < R; r += 4) {
        const float4 k4 = *reinterpret_cast<const float4*>(&sk[t][warp * R + r]);
        const float4 q4 = *reinterpret_cast<const float4*>(&sq[t][warp * R + r]);
        const float k[4] = {k4.x, k4.y, k4.z, k4.w}, q[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x = s[r + j];
          if (!p.reverse) x = decay(x);
          x = fmaf(k[j], v, x);
          o = fmaf(q[j], x, o);
          s[r + j] = p.reverse ? decay(x) : x;
        }
      }
      part[warp][t][lane] = o;
    }
    __syncthreads();
    for (int i = tid; i < n * 32; i += 256) {
      float o = 0.f;
#pragma unroll
      for (int w = 0; w < 8; ++w) o += part[w][i >> 5][i & 31];
      p.o[row_of(i >> 5) + col0 + (i & 31)] = (uint16_t)(pack_bf16(o * p.o_mul, 0.f) & 0xFFFFu);
    }
  }
  for (int t = len + warp; t < p.L; t += 8) p.o[((base + t) * p.H + h) * D + col] = 0;
  if (p.state_out != nullptr) {
    float* out = p.state_out + bh * D * D;
    if (p.state_t) {
#pragma unroll
      for (int r = 0; r < R; r += 4)
        *reinterpret_cast<float4*>(out + col * D + warp * R + r) = make_float4(s[r], s[r + 1], s[r + 2], s[r + 3]);
    } else {
#pragma unroll
      for (int r = 0; r < R; ++r) out[(warp * R + r) * D + col] = s[r];
    }
  }
}

// ---------------------------------------------------------------- tiles
//
// Tokens in tiles of C = 128.  With S the state before a tile of n live
// tokens (forward; reversed in time the exponents are those in brackets):
//   o_i = o_mul ( g^(i+1) q_i S + kv_mul sum_{j <= i} g^(i-j) (q_i.k_j) v_j )
//         [g^(n-1-i),  j >= i,  g^(j-i)]
//   S' = g^n S + kv_mul sum_j g^(n-1-j) k_j v_j^T        [g^(j+1)]
// Four products per tile on tcgen05 (bf16 operands, fp32 accumulators in
// TMEM): scores Q K^T, inter Q S, intra P V, update (W K)^T V.  A tile of a
// head moves 8 D C bytes and costs 4 (C D^2 + C^2 D) multiply-adds at most, so
// the kernel is bound by HBM as long as the element work below stays hidden.
//
// Roundings: P (decay applied in fp32) and the state's copy that multiplies
// q go to bf16, as every tensor-core operand must; the state itself stays in
// fp32 registers.  W K in bf16 would cost the state 8 bits, so it is split into
// TERMS bf16 parts, one product each: three (24 bits) for a state that the
// caller gets, two (16 bits) for one that only feeds bf16 outputs.
//
// One CTA owns a run of tiles of one (b, h).  When B H leaves SMs idle a
// sequence is cut into segments: decay_segment_kernel sums each segment's own
// contribution (reading k and v only), decay_carry_kernel chains them into the
// state before every segment, and the segments then run in parallel.
constexpr int kC = 128;
constexpr uint64_t kTimeoutNs = 2000000000ull;  // 2 s per pipeline wait
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}

// Bounded mbarrier wait: gives up after kTimeoutNs or when another warp of
// the CTA has (see chunk_attn.cu); records the site in the device error word.
// Out of line, as is all rare code here: four roles share the instruction cache.
__device__ __noinline__ bool wait_slow(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned site,
                                       unsigned* err_word) {
  const uint64_t t0 = global_ns();
#pragma unroll 1
  for (uint32_t it = 1;; ++it) {
    if (mbar_try_wait(bar, parity)) return true;
    if ((it & 255u) == 0) {
      if (*abort_flag) return false;
      if (global_ns() - t0 > kTimeoutNs) {
        if (err_word != nullptr) atomicOr(err_word, 1u << site);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned site,
                                             unsigned* err_word) {
  return mbar_try_wait(bar, parity) || wait_slow(bar, parity, abort_flag, site, err_word);
}
__device__ __noinline__ void wait_drain(uint32_t bar, uint32_t parity, unsigned* err_word) {
  const uint64_t t0 = global_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (global_ns() - t0 > kTimeoutNs) {
      if (err_word != nullptr) atomicOr(err_word, 1u << 31);
      return;
    }
  }
}

// Debug builds: the place of a segment's state lies inside the scratch, and the
// block belongs to a sequence.  Uniform over the CTA, before any copy or store.
__device__ __forceinline__ bool in_bounds(const DecayTileParams& p, long long bh, int seg) {
  if constexpr (kDebugBounds) {
    if (bh >= 0 && bh < (long long)p.B * p.H && seg >= 0 && seg < p.nseg &&
        (p.nseg == 1 || bh * p.nseg + seg < p.carry_states))
      return true;
    if (threadIdx.x == 0 && p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
    return false;
  }
  return true;
}

// This block's run, and its index among that run's blocks.
__device__ __forceinline__ const DecayTileParams& pick(const DecayRuns& r, unsigned& block) {
  block = blockIdx.x;
  if (block < r.first) return r.run[0];
  block -= r.first;
  if (r.n == 2) return r.run[1];
  const int i = 1 + (int)(block & 1u);
  block >>= 1;
  return r.run[i];
}

// The tiles [r0, r1) of a segment in run order, and of those the live ones
// [a, b) (tokens inside the sequence).
struct Run {
  int len;      // live tokens of the sequence
  int ntiles;   // tiles of the padded sequence
  int r0, r1, a, b;
  bool rev;
  __device__ __forceinline__ Run(const DecayTileParams& p, int bidx, int seg) : rev(p.reverse != 0) {
    len = p.seq_len != nullptr ? min(max(__ldg(p.seq_len + bidx), 0), p.L) : p.L;
    ntiles = (p.L + kC - 1) / kC;
    r0 = min(seg * p.seg_tiles, ntiles);
    r1 = min(r0 + p.seg_tiles, ntiles);
    const int live = (len + kC - 1) / kC;
    a = rev ? min(max(r0, ntiles - live), r1) : r0;
    b = rev ? r1 : max(min(r1, live), r0);
  }
  __device__ __forceinline__ int tile(int r) const { return rev ? ntiles - 1 - r : r; }
  __device__ __forceinline__ int tokens(int r) const { return min(kC, len - tile(r) * kC); }
  // first token and live tokens of the segment
  __device__ __forceinline__ int first() const { return (rev ? ntiles - b : a) * kC; }
  __device__ __forceinline__ int count() const {
    return a >= b ? 0 : min(len, (rev ? ntiles - a : b) * kC) - first();
  }
};

// Pieces of 16 bytes (8 elements) of a 128-byte swizzled tile of ROWS rows.  A
// row's pieces keep their places, so row-wise work needs no unscrambling.
template <int ROWS>
__device__ __forceinline__ uint32_t piece_off(int row, int c) {
  return (uint32_t)((c >> 3) * (ROWS * 128) + row * 128 + (c & 7) * 16);
}

// Rows of a k tile times f * w[row], as TERMS bf16 parts that add up to it:
// the first in place, the others (the rounded rest of the one before) in tiles
// of `rest_bytes` behind `rest`.  Rows from n on become zero; so do those of
// `v`, if given: they may hold anything, and 0 * NaN would reach every sum.
template <int D, int ROWS, int TERMS, int FROM = 0, int TO = ROWS>
__device__ __forceinline__ void scale_rows(uint8_t* k, uint8_t* rest, uint32_t rest_bytes, uint8_t* v, int tid, int n,
                                           float f, const float* w) {
  constexpr int kPieces = D / 8;             // per row
  constexpr int kStep = 256 / kPieces;       // rows between a thread's pieces
  static_assert(FROM % kStep == 0 && TO % kStep == 0, "whole steps");
  uint32_t off = piece_off<ROWS>(FROM + tid / kPieces, tid % kPieces);
#pragma unroll 2
  for (int row = FROM + tid / kPieces; row < TO; row += kStep, off += kStep * 128) {
    uint32_t part[TERMS][4];
    if (row < n) {
      const float wr = f * w[row];
      const uint4 x = *reinterpret_cast<const uint4*>(k + off);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
      if constexpr (TERMS == 2) {
        // with w = w1 + w2 in bf16: k w1 = hi + e, both bf16 (the product has
        // 16 bits), and the rest is e + k w2: three packed bf16 operations
        const uint32_t w1 = pack_bf16(wr, wr), h1 = w1 & 0xFFFF0000u;
        const float r = wr - __uint_as_float(h1);
        const uint32_t w2 = pack_bf16(r, r);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          part[0][j] = mul_bf16x2(xs[j], w1);
          part[1][j] = fma_bf16x2(xs[j], w2, fma_bf16x2(xs[j], w1, part[0][j] ^ 0x80008000u));
        }
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float2 r = __fmul2_rn(make_float2(__uint_as_float(xs[j] << 16), __uint_as_float(xs[j] & 0xFFFF0000u)),
                                make_float2(wr, wr));
#pragma unroll
          for (int t = 0; t < TERMS; ++t) {
            const uint32_t q = pack_bf16(r.x, r.y);
            part[t][j] = q;
            if (t + 1 < TERMS)
              r = __fadd2_rn(r, make_float2(-__uint_as_float(q << 16), -__uint_as_float(q & 0xFFFF0000u)));
          }
        }
      }
    } else {
#pragma unroll
      for (int t = 0; t < TERMS; ++t)
#pragma unroll
        for (int j = 0; j < 4; ++j) part[t][j] = 0u;
      if (v != nullptr) *reinterpret_cast<uint4*>(v + off) = make_uint4(0u, 0u, 0u, 0u);
    }
    *reinterpret_cast<uint4*>(k + off) = make_uint4(part[0][0], part[0][1], part[0][2], part[0][3]);
#pragma unroll
    for (int t = 1; t < TERMS; ++t)
      *reinterpret_cast<uint4*>(rest + (t - 1) * rest_bytes + off) =
          make_uint4(part[t][0], part[t][1], part[t][2], part[t][3]);
  }
}
template <int D>
__device__ __noinline__ void zero_rows(uint8_t* v, int tid, int n) {
  constexpr int kPieces = D / 8;
#pragma unroll 1
  for (int i = n * kPieces + tid; i < kC * kPieces; i += 256)
    *reinterpret_cast<uint4*>(v + piece_off<kC>(i / kPieces, i % kPieces)) = make_uint4(0u, 0u, 0u, 0u);
}

// One arrival per warp, after its lanes' writes (each lane fences its own).
__device__ __forceinline__ void warp_arrive(uint32_t bar, int lane) {
  __syncwarp();
  if (lane == 0) mbar_arrive(bar);
}

// Carried states are kept as the element threads hold them: 4 columns of a row
// together, the rows of a column group side by side.  Index of (row, col):
// + 1 for the next column of the four, + 4 for the next row, + 8 D for the next
// column group of the same half.
template <int D>
__device__ __forceinline__ int piece_index(int row, int col) {
  const int half = col / (D / 2), c = col % (D / 2);
  return ((c / 4) * 2 * D + half * D + row) * 4 + c % 4;
}

constexpr uint32_t kAMajorMN = 1u << 15;  // instruction descriptor: A is MN-major

// The tile kernel's warps: 0 loads, 1 issues MMAs, 2-9 ("rows") turn scores
// into P and accumulators into output rows, 10-17 ("state") scale k and carry
// the state, 18 stores.  The two element groups work on the same tile at once
// and need each other only through the MMAs.  (One group doing all four steps
// in turn: 198 us for 2 x 30720 tokens of 12 heads of 128; two: 135 us, the
// four roles' code kept small enough for the instruction cache, 222 us before.)
// 608 threads leave 96 registers each; heads of 128 spill 44 bytes of a thread
// (68 and 144 bytes reloaded with two and three parts), heads of 64 up to 8.
// D = 128: a tile's output is staged over its v once the update has read it;
// nothing else is free.  D = 64 has room for an output buffer of its own and
// for two sets of k's parts (kRoomy): the next tile's scores go ahead of the
// update, its k is scaled while the update runs, and the chain from state to
// state is update, state, state product only.
template <int D_, int TERMS_>
struct TileCfg {
  static constexpr int D = D_, TERMS = TERMS_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = kC * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kQStages = D == 128 ? 1 : 2;
  // (D = 64: the update's A operand, M = 128, takes its upper 64 rows from the
  // box behind a k tile; they land in accumulator rows that nothing reads)
  static constexpr uint32_t kKOff = 0;                                       // [kKStages]; scaled in place
  static constexpr bool kRoomy = D == 64;
  static constexpr int kShared = kRoomy ? kC : 80;  // k rows from here on are scaled by the rows' warps
  static constexpr int kKStages = kRoomy ? 3 : 2, kVStages = kRoomy ? 3 : TERMS == 3 ? 1 : 2;
  static constexpr uint32_t kRestOff = kKOff + kKStages * kTileBytes;             // [kRoomy ? 2 : 1][TERMS - 1]
  static constexpr uint32_t kRestBytes = (TERMS - 1) * kTileBytes;
  static constexpr uint32_t kQOff = kRestOff + (kRoomy ? 2 : 1) * kRestBytes;
  static constexpr uint32_t kVOff = kQOff + kQStages * kTileBytes;
  static constexpr uint32_t kOutOff = kVOff + kVStages * kTileBytes;
  static constexpr uint32_t kStOff = kOutOff + (kRoomy ? kTileBytes : 0);   // bf16 state [D][D]
  static constexpr uint32_t kStBoxBytes = D * 128u;
  static constexpr uint32_t kBarOff = kStOff + kBoxes * kStBoxBytes;
  // barriers; those of a slot [3]
  static constexpr int kFullQ = 0, kFullK = 3, kFullV = 6, kEmptyQ = 9, kEmptyK = 12, kEmptyV = 15, kOut = 18;
  static constexpr int kSFull = 21, kPFull = 22, kKwFull = 23, kOFull = 24, kORead = 25, kUFull = 26, kStFull = 27,
                       kDrain = 28, kOutFree = 29, kNumBars = 30;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;               // tmem address, abort flag
  static constexpr uint32_t kTabOff = kMiscOff + 16;                         // decay powers: of P [256], of k [128]
  static constexpr uint32_t kSmemBytes = kTabOff + 4 * (256 + 128) + 1024;
  static constexpr int kThreads = 608;
  static constexpr uint32_t kS = 0, kIntra = 128, kInter = 128 + D, kUpd = 128 + 2 * D;  // TMEM columns
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kTabOff % 4 == 0 && kStOff % 1024 == 0, "alignment");
};

template <int D, int TERMS>
__global__ void __launch_bounds__(TileCfg<D, TERMS>::kThreads, 1)
decay_tile_kernel(const __grid_constant__ DecayRuns runs) {
  using C = TileCfg<D, TERMS>;
  // A run that writes its state (TERMS = 3) has a launch to itself; choosing
  // would cost registers it does not have (1 us of 46 for 8 sequences of up to
  // 2047 tokens, 24 heads of 64).
  unsigned block = blockIdx.x;
  const DecayTileParams& p = TERMS == 3 ? runs.run[0] : pick(runs, block);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  // p_tab[127 + i - j]: factor of the score of row i and column j (0 where
  // masked); w_tab[j]: factor of k row j of a full tile
  float* p_tab = reinterpret_cast<float*>(base + C::kTabOff);
  float* w_tab = p_tab + 256;
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = block % p.nseg;
  int b = (int)(block / p.nseg / p.H);
  const int h = (int)(block / p.nseg % p.H);
  if (!in_bounds(p, block / p.nseg, seg)) return;

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), i == C::kPFull || i == C::kKwFull || i == C::kORead || i == C::kStFull ||
                                (i >= C::kOut && i < C::kOut + 3)
                            ? (i == C::kKwFull && C::kShared < kC ? 16 : 8)
                            : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
    // not before: a dependent on this SM that took TMEM first and then waited
    // for this grid would never give it back
    griddep_launch_dependents();
  }
  // With segments, this kernel follows the ones that sum and chain them.  Those
  // let it start only after their own waits, so that everything before them
  // is complete: all but the carried states may be read, and worked on, now.
  if (p.nseg == 1) griddep_wait();
  if (p.by_length) {
    // more sequences than SMs, of unequal lengths: the longest first, so that
    // the last to start are the shortest (8 sequences of up to 2047 tokens, 24
    // heads of 64, eight draws: 42.3 us on average, 47.6 us in their own order)
    int* lens = reinterpret_cast<int*>(base + C::kTabOff);  // the tables come later
    if ((int)threadIdx.x < p.B) lens[threadIdx.x] = min(max(__ldg(p.seq_len + threadIdx.x), 0), p.L);
    __syncthreads();
    if ((int)threadIdx.x < p.B) {
      int rank = 0;
      for (int i = 0; i < p.B; ++i)
        rank += lens[i] > lens[threadIdx.x] || (lens[i] == lens[threadIdx.x] && i < (int)threadIdx.x);
      if (rank == b) misc[2] = threadIdx.x;
    }
    __syncthreads();
    b = (int)misc[2];
  }
  const long long bh = (long long)b * p.H + h;
  const Run run(p, b, seg);
  const float ln = decay_ln(p.log_decay, h), ld2 = ln * kLog2e;
  if (threadIdx.x < 256) {
    const int d = p.reverse ? 127 - (int)threadIdx.x : (int)threadIdx.x - 127;
    p_tab[threadIdx.x] = d >= 0 ? p.o_mul * p.kv_mul * ex2((float)d * ld2) : 0.f;
  } else if (threadIdx.x < 384) {
    const int j = threadIdx.x - 256;
    w_tab[j] = p.kv_mul * ex2((float)(p.reverse ? j + 1 : 127 - j) * ld2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int nt = run.b - run.a;
  // the state after the last tile is wanted only by state_out
  const int n_upd = p.state_out != nullptr ? nt : nt - 1;
  auto wait = [&](int i, uint32_t parity, unsigned site) {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    if (lane == 0 && nt > 0) {
      int nq = 0, nk = 0, nv = 0;
      // load number n of a stream of `stages` slots
      auto load = [&](const CUtensorMap* m, uint32_t off, int full, int empty, int stages, int& n, int it) {
        const int s = n % stages;
        if (n >= stages && !wait(empty + s, (n / stages - 1) & 1u, 9)) return false;
        mbar_arrive_expect_tx(bar(full + s), C::kTileBytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + off + s * C::kTileBytes + bx * C::kBoxBytes, m, bar(full + s), bx * 64,
                      run.tile(run.a + it) * kC, h, b);
        ++n;
        return true;
      };
      // q first for the first tile, then in the order in which the slots come free
      auto load_q = [&](int it) { return load(&p.q_map, C::kQOff, C::kFullQ, C::kEmptyQ, C::kQStages, nq, it); };
      bool ok = load_q(0);
      for (int it = 0; ok && it < nt; ++it) {
        ok = load(&p.k_map, C::kKOff, C::kFullK, C::kEmptyK, C::kKStages, nk, it) &&
             (it == 0 || C::kVStages > 1 || load_q(it)) &&
             load(&p.v_map, C::kVOff, C::kFullV, C::kEmptyV, C::kVStages, nv, it) &&
             (it == 0 || C::kVStages == 1 || load_q(it));
      }
      if (*abort_flag) {
        auto drain = [&](int full, int stages, int n) {
          for (int i = max(0, n - stages); i < n; ++i)
            wait_drain(bar(full + i % stages), (i / stages) & 1u, p.err_word);
        };
        drain(C::kFullK, C::kKStages, nk);
        drain(C::kFullQ, C::kQStages, nq);
        drain(C::kFullV, C::kVStages, nv);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
    const uint32_t lead = elect_lead();
    constexpr uint32_t id_s = idesc_bf16_f32(128, 128, 0);                 // q . k: both K-major
    constexpr uint32_t id_o = idesc_bf16_f32(128, D, 1);                   // B = v or state, MN-major
    constexpr uint32_t id_u = idesc_bf16_f32(128, D, 1) | kAMajorMN;       // A = scaled k, MN-major
    const uint64_t kmaj = smem_desc_sw128(base_u32, 16, 1024);
    const uint64_t mn = smem_desc_sw128(base_u32, C::kBoxBytes, 1024);
    const uint64_t mn_st = smem_desc_sw128(base_u32, C::kStBoxBytes, 1024);
    auto at = [](uint64_t d, uint32_t off) { return make_desc((uint32_t)d + (off >> 4), (uint32_t)(d >> 32)); };
    auto k_off = [](int kk) { return (uint32_t)((kk >> 2) * C::kBoxBytes + (kk & 3) * 32); };
    auto wait_all = [&](int i, uint32_t parity, unsigned site) {
      const bool r = __all_sync(0xffffffffu, wait(i, parity, site));
      if (r) tc_fence_after();
      return r;
    };
    auto scores = [&](int it) {
      const int s = it % C::kKStages, sq = it % C::kQStages;
      if (!wait_all(C::kFullQ + sq, (it / C::kQStages) & 1u, 10) ||
          !wait_all(C::kFullK + s, (it / C::kKStages) & 1u, 10))
        return false;
      const uint32_t q = C::kQOff + sq * C::kTileBytes, k = C::kKOff + s * C::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_l(lead, tmem + C::kS, at(kmaj, q + k_off(kk)), at(kmaj, k + k_off(kk)), id_s, kk > 0);
      mma_commit_l(lead, bar(C::kSFull));
      return true;
    };
    // A slot is announced free only to a load that waits for it: an arrival that
    // nobody waits for could reach shared memory that the CTA has left.
    bool ok = nt > 0 && scores(0);
    for (int it = 0; ok && it < nt; ++it) {
      const int s = it % C::kKStages, sv = it % C::kVStages, sq = it % C::kQStages;
      const uint32_t q = C::kQOff + sq * C::kTileBytes, k = C::kKOff + s * C::kTileBytes,
                     v = C::kVOff + sv * C::kTileBytes;
      auto state_product = [&]() {
        if (!wait_all(C::kStFull, it & 1u, 11)) return false;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
          mma_ss_l(lead, tmem + C::kInter, at(kmaj, q + k_off(kk)), at(mn_st, C::kStOff + kk * 2048u), id_o, kk > 0);
        if (it + C::kQStages < nt) mma_commit_l(lead, bar(C::kEmptyQ + sq));
        return true;
      };
      // the previous output rows are read
      ok = it == 0 || wait_all(C::kORead, (it - 1) & 1u, 11);
      if (ok && !C::kRoomy) ok = state_product();
      ok = ok && wait_all(C::kPFull, it & 1u, 12) && wait_all(C::kFullV + sv, (it / C::kVStages) & 1u, 10);
      if (!ok) break;
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ts_l(lead, tmem + C::kIntra, tmem + C::kS + (kk >> 2) * 64 + (kk & 3) * 8, at(mn, v + kk * 2048u), id_o,
                 kk > 0);
      if (!C::kRoomy) mma_commit_l(lead, bar(C::kOFull));
      if (it < n_upd && !(ok = wait_all(C::kKwFull, it & 1u, 13))) break;
      if (C::kRoomy) {
        if (it + 1 < nt && !(ok = scores(it + 1))) break;
        if (!(ok = state_product())) break;
        mma_commit_l(lead, bar(C::kOFull));
      }
      if (it < n_upd) {
        const uint32_t rest = C::kRestOff + (C::kRoomy ? (uint32_t)(it & 1) * C::kRestBytes : 0u);
        // the small parts first: an accumulator is cut short at every addition,
        // by up to 2^-23 of what it holds, always towards zero (24 additions at
        // full size lost 6e-7 of the state, 8 lose 1e-7)
#pragma unroll
        for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
          for (int kk = 0; kk < kC / 16; ++kk)
            mma_ss_l(lead, tmem + C::kUpd, at(mn, (t == 0 ? k : rest + (t - 1) * C::kTileBytes) + kk * 2048u),
                     at(mn, v + kk * 2048u), id_u, t < TERMS - 1 || kk > 0);
        mma_commit_l(lead, bar(C::kUFull));
        if (it + C::kKStages < nt) mma_commit_l(lead, bar(C::kEmptyK + s));
        if (C::kRoomy && it + C::kVStages < nt) mma_commit_l(lead, bar(C::kEmptyV + sv));
      }
      if (!C::kRoomy && it + 1 < nt) ok = scores(it + 1);
    }
    if (__any_sync(0xffffffffu, (nt > 0 && !ok) || *abort_flag)) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 18) {
    // --------------------------------------------------------- output store
    if (lane == 0) {
      for (int it = 0; it < nt; ++it) {
        const int so = C::kRoomy ? 0 : it % C::kVStages;  // staging slot
        if (!wait(C::kOut + so, (C::kRoomy ? it : it / C::kVStages) & 1u, 14)) break;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_store_4d(&p.o_map,
                       base_u32 + (C::kRoomy ? C::kOutOff : C::kVOff) + so * C::kTileBytes + bx * C::kBoxBytes, bx * 64,
                       run.tile(run.a + it) * kC, h, b);
        tma_store_commit_and_wait_read();
        mbar_arrive(bar(C::kRoomy ? C::kOutFree : C::kEmptyV + so));
      }
    }
    __syncwarp();
  } else {
    const int quad = warp & 3, hf = ((warp - 2) >> 2) & 1;
    const int row = quad * 32 + lane;  // token of the tile; key dimension of the state
    const uint32_t lane_off = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int kCols = D / 2;       // columns of this thread: [hf D/2, (hf + 1) D/2)
    const bool rev = p.reverse != 0;
    // offset of 16-byte piece c (8 columns) of this thread's row in a swizzled tile
    auto piece = [&](int c, uint32_t box_bytes) {
      const int cc = hf * (kCols / 8) + c;
      return (uint32_t)((cc >> 3) * box_bytes + row * 128 + (((cc & 7) ^ (row & 7)) << 4));
    };
    bool ok = true;
    if (warp < 10) {
      // ------------------------------------------------------------- rows
      const int tid = threadIdx.x - 64;
      // a row's factor of the state: as a Decay, 0 only where the decay is (inf * 0)
      const float f_least = decays_to_zero(ln) ? 0.f : kLeast;
      for (int it = 0; it < nt; ++it) {
        const int n = run.tokens(run.a + it), sv = it % C::kVStages;
        uint8_t* vt = base + C::kVOff + sv * C::kTileBytes;
        // P = decayed, masked scores, bf16, over the scores
        ok = __all_sync(0xffffffffu, wait(C::kSFull, it & 1u, 15));
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int pass = 0; pass < 2; ++pass) {
          const int c0 = hf * 64 + 32 * pass;
          uint32_t pk[16];
          if ((rev ? c0 + 31 < quad * 32 : c0 > quad * 32 + 31) || c0 >= n) {  // nothing visible
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = 0u;
          } else {
            uint32_t x[32];
            tmem_ld32(lane_off + C::kS + c0, x);
            const float* t = p_tab + 127 + row - c0;
            float w[32];
#pragma unroll
            for (int c = 0; c < 32; ++c) w[c] = t[-c];
            tmem_wait_ld();
            if (c0 + 32 > n) {
#pragma unroll
              for (int c = 0; c < 32; ++c)
                if (c0 + c >= n) x[c] = 0u;
            }
#pragma unroll
            for (int c = 0; c < 16; ++c)
              pk[c] = pack_bf16(__uint_as_float(x[2 * c]) * w[2 * c], __uint_as_float(x[2 * c + 1]) * w[2 * c + 1]);
          }
          tmem_st16(lane_off + C::kS + hf * 64 + 16 * pass, pk);
        }
        tmem_wait_st();
        if (n < kC) {  // padding of v must not meet the zeros of P
          ok = __all_sync(0xffffffffu, wait(C::kFullV + sv, (it / C::kVStages) & 1u, 15));
          if (!ok) break;
          zero_rows<D>(vt, tid, n);
          fence_proxy_async_smem();
        }
        tc_fence_before();
        warp_arrive(bar(C::kPFull), lane);
        // a share of k's rows while P V runs (96 sequences of 4096 tokens of heads
        // of 128: 92 us, 97 us with all of them left to the state's warps)
        if (C::kShared < kC && it < n_upd) {
          const int s = it % C::kKStages;
          ok = __all_sync(0xffffffffu, wait(C::kFullK + s, (it / C::kKStages) & 1u, 15));
          if (!ok) break;
          scale_rows<D, kC, TERMS, C::kShared, kC>(base + C::kKOff + s * C::kTileBytes, base + C::kRestOff, C::kTileBytes,
                                                   nullptr, tid, n, 1.f, rev ? w_tab : w_tab + kC - n);
          fence_proxy_async_smem();
          warp_arrive(bar(C::kKwFull), lane);
        }
        // output rows
        const float f = fmaxf(p.o_mul * ex2((float)(rev ? n - 1 - row : row + 1) * ld2), f_least);
        ok = __all_sync(0xffffffffu, wait(C::kOFull, it & 1u, 15));
        if (!ok) break;
        tc_fence_after();
        uint32_t o[kCols / 2];
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 16) {
          uint32_t x[16], y[16];
          tmem_ld16(lane_off + C::kIntra + hf * kCols + c0, x);
          tmem_ld16(lane_off + C::kInter + hf * kCols + c0, y);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            const float2 r = __ffma2_rn(make_float2(__uint_as_float(y[2 * c]), __uint_as_float(y[2 * c + 1])),
                                        make_float2(f, f),
                                        make_float2(__uint_as_float(x[2 * c]), __uint_as_float(x[2 * c + 1])));
            o[c0 / 2 + c] = row < n ? pack_bf16(r.x, r.y) : 0u;
          }
        }
        tc_fence_before();
        warp_arrive(bar(C::kORead), lane);
        // v is free once the update has read it, the own buffer once stored
        if (C::kRoomy ? it > 0 : it < n_upd) {
          ok = __all_sync(0xffffffffu, C::kRoomy ? wait(C::kOutFree, (it - 1) & 1u, 15) : wait(C::kUFull, it & 1u, 15));
          if (!ok) break;
        }
        uint8_t* ot = C::kRoomy ? base + C::kOutOff : vt;
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c)
          *reinterpret_cast<uint4*>(ot + piece(c, C::kBoxBytes)) =
              make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        fence_proxy_async_smem();
        warp_arrive(bar(C::kOut + (C::kRoomy ? 0 : sv)), lane);
      }
      // tiles of the segment without a live token
      for (int r = run.r0; r < run.r1; ++r) {
        if (r >= run.a && r < run.b) continue;
        const int t0 = run.tile(r) * kC, rows = min(kC, p.L - t0);
        for (int i = tid; i < rows * (D / 8); i += 256) {
          const long long e = (((long long)b * p.L + t0 + i / (D / 8)) * p.H + h) * D + i % (D / 8) * 8;
          *reinterpret_cast<uint4*>(p.o + e) = make_uint4(0u, 0u, 0u, 0u);
        }
      }
    } else {
      // ------------------------------------------------------------ state
      const int tid = threadIdx.x - 320;
      float st[kCols];
      auto publish = [&]() {
        if (row < D) {
#pragma unroll
          for (int c = 0; c < kCols / 8; ++c)
            *reinterpret_cast<uint4*>(base + C::kStOff + piece(c, C::kStBoxBytes)) =
                make_uint4(pack_bf16(st[8 * c], st[8 * c + 1]), pack_bf16(st[8 * c + 2], st[8 * c + 3]),
                           pack_bf16(st[8 * c + 4], st[8 * c + 5]), pack_bf16(st[8 * c + 6], st[8 * c + 7]));
        }
        fence_proxy_async_smem();
        tc_fence_before();
        warp_arrive(bar(C::kStFull), lane);
      };
      // the state before the segment
#pragma unroll
      for (int c = 0; c < kCols; ++c) st[c] = 0.f;
      if (p.nseg > 1) {
        griddep_wait();
        const float* in = p.carry + (bh * p.nseg + seg) * D * D;
        if (row < D && p.carry_t) {
          in += piece_index<D>(hf * kCols, row);
#pragma unroll
          for (int c = 0; c < kCols; ++c) st[c] = in[4 * c];
        } else if (row < D) {
          in += piece_index<D>(row, hf * kCols);
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(in + c * 8 * D);
            st[4 * c] = x.x, st[4 * c + 1] = x.y, st[4 * c + 2] = x.z, st[4 * c + 3] = x.w;
          }
        }
      } else if (p.state_in != nullptr && row < D) {
        const float* in = p.state_in + bh * D * D;
        if (p.state_t) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) st[c] = in[(hf * kCols + c) * D + row];
        } else {
#pragma unroll
          for (int c = 0; c < kCols / 4; ++c) {
            const float4 x = *reinterpret_cast<const float4*>(in + row * D + hf * kCols + 4 * c);
            st[4 * c] = x.x, st[4 * c + 1] = x.y, st[4 * c + 2] = x.z, st[4 * c + 3] = x.w;
          }
        }
      }
      if (nt > 0) publish();
      Decay decay = decay_over(kC, ln);
      // the scores have read a tile's k; its scaled form replaces it
      auto scale = [&](int it) {
        const int s = it % C::kKStages, n = run.tokens(run.a + it);
        if (!__all_sync(0xffffffffu, wait(C::kSFull, it & 1u, 8) && wait(C::kFullK + s, (it / C::kKStages) & 1u, 8)))
          return false;
        uint8_t* rest = base + C::kRestOff + (C::kRoomy ? (it & 1) * C::kRestBytes : 0);
        scale_rows<D, kC, TERMS, 0, C::kShared>(base + C::kKOff + s * C::kTileBytes, rest, C::kTileBytes, nullptr, tid, n,
                                                1.f, rev ? w_tab : w_tab + kC - n);
        fence_proxy_async_smem();
        warp_arrive(bar(C::kKwFull), lane);
        return true;
      };
      for (int it = C::kRoomy ? -1 : 0; it < n_upd; ++it) {
        const int next = C::kRoomy ? it + 1 : it;
        if (next < n_upd && !(ok = scale(next))) break;
        if (it < 0) continue;
        const int n = run.tokens(run.a + it);
        ok = __all_sync(0xffffffffu, wait(C::kUFull, it & 1u, 8));
        if (!ok) break;
        tc_fence_after();
        if (n != kC) decay = decay_over(n, ln);
        const float2 hi = make_float2(decay.hi, decay.hi), lo = make_float2(decay.lo, decay.lo);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 16) {
          uint32_t x[16];
          tmem_ld16(lane_off + C::kUpd + hf * kCols + c0, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 16; c += 2) {
            const float2 s2 = make_float2(st[c0 + c], st[c0 + c + 1]);
            const float2 r = __fadd2_rn(__ffma2_rn(s2, hi, __fmul2_rn(s2, lo)),
                                        make_float2(__uint_as_float(x[c]), __uint_as_float(x[c + 1])));
            st[c0 + c] = r.x;
            st[c0 + c + 1] = r.y;
          }
        }
        if (n != kC) decay = decay_over(kC, ln);
        if (it + 1 < nt) publish();
      }
      // an aborted CTA stores no state; its outputs are not valid either
      if (ok && !*abort_flag && p.state_out != nullptr && row < D) {
        float* out = p.state_out + bh * D * D;
        if (p.state_t) {
#pragma unroll
          for (int c = 0; c < kCols; ++c) out[(hf * kCols + c) * D + row] = st[c];
        } else {
#pragma unroll
          for (int c = 0; c < kCols; c += 4)
            *reinterpret_cast<float4*>(out + row * D + hf * kCols + c) =
                make_float4(st[c], st[c + 1], st[c + 2], st[c + 3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A segment's own contribution to the state after it: its tokens' updates with
// the decays to the segment's end, accumulated in TMEM over the segment, 64
// tokens at a time.  Nothing but the loads and the scaling of k runs per
// step, so the loads are kept many steps ahead.  A sum that the caller gets
// (TERMS = 3) is moved to fp32 registers every 256 tokens: an accumulator loses
// 1e-8 of itself at every addition, always towards zero.
template <int D_, int TERMS_>
struct SegCfg {
  static constexpr int D = D_, TERMS = TERMS_;
  static constexpr int kRows = 64;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = kRows * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kStages = TERMS == 3 ? 5 : 6;
  static constexpr uint32_t kStageBytes = 2 * kTileBytes;                   // k (scaled in place), v
  static constexpr uint32_t kRestOff = kStages * kStageBytes;               // [2][TERMS - 1]
  static constexpr uint32_t kRestBytes = (TERMS - 1) * kTileBytes;
  static constexpr uint32_t kPadOff = kRestOff + 2 * kRestBytes;            // D = 64: behind the last A operand
  static constexpr uint32_t kBarOff = kPadOff + (D == 64 ? kTileBytes : 0);
  static constexpr int kFull = 0, kEmpty = kStages, kScaled = 2 * kStages, kFinal = kScaled + 2, kDrain = kFinal + 1,
                       kGroupFull = kDrain + 1 /* [2] */, kGroupFree = kGroupFull + 2 /* [2] */,
                       kNumBars = kGroupFree + 2;
  // TERMS = 3: the sum leaves TMEM for fp32 registers every kGroup steps, first
  // parts and the others apart, two buffers of 2 D columns
  static constexpr int kGroup = 4;
  static constexpr uint32_t kTmemCols = TERMS == 3 ? 4 * D : 128;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kTabOff = kMiscOff + 16;                        // decay powers of k
  static constexpr uint32_t kSmemBytes = kTabOff + 4 * kRows + 1024;
  static constexpr int kThreads = 576;  // loads, MMA, two groups of 8 warps that scale every other step
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

template <int D, int TERMS>
__global__ void __launch_bounds__(SegCfg<D, TERMS>::kThreads, 1)
decay_segment_kernel(const __grid_constant__ DecayRuns runs) {
  using C = SegCfg<D, TERMS>;
  unsigned block;
  const DecayTileParams& p = pick(runs, block);
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrun = p.state_out != nullptr ? p.nseg : p.nseg - 1;  // the last segment's is wanted by state_out only
  const int seg = block % nrun;
  const long long bh = block / nrun;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  if (!in_bounds(p, bh, seg)) return;
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), i == C::kScaled || i == C::kScaled + 1 ? 8 : i >= C::kGroupFree ? 16 : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), C::kTmemCols);
    tmem_relinquish();
  }
  griddep_wait();
  griddep_launch_dependents();  // not before: the tile kernel reads its inputs ahead of its own wait
  const Run run(p, b, seg);
  const float ld2 = decay_ln(p.log_decay, h) * kLog2e;
  float* w_tab = reinterpret_cast<float*>(base + C::kTabOff);  // factor of k row j of a full step next to the end
  if (threadIdx.x < C::kRows) {
    const int n = p.reverse ? (int)threadIdx.x + 1 : C::kRows - 1 - (int)threadIdx.x;
    w_tab[threadIdx.x] = p.kv_mul * ex2((float)n * ld2);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int first = run.first(), count = run.count();
  const int nt = (count + C::kRows - 1) / C::kRows;
  // against the run's order: the tokens it starts with are read last
  auto start = [&](int it) { return (p.reverse ? it : nt - 1 - it) * C::kRows; };
  auto wait = [&](int i, uint32_t parity, unsigned site) {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };
  if (warp == 0) {
    if (lane == 0) {
      // (2 x 30720 tokens of 12 heads: 196 us for the whole call, 202 us with the
      // default policy)
      const uint64_t policy = l2_evict_first();
      int issued = 0;
      for (int it = 0; it < nt; ++it) {
        const int s = it % C::kStages;
        if (it >= C::kStages && !wait(C::kEmpty + s, (it / C::kStages - 1) & 1u, 9)) break;
        mbar_arrive_expect_tx(bar(C::kFull + s), C::kStageBytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx) {
          const uint32_t dst = base_u32 + s * C::kStageBytes + bx * C::kBoxBytes;
          tma_load_4d_hint(dst, &p.k_map_h, bar(C::kFull + s), bx * 64, first + start(it), h, b, policy);
          tma_load_4d_hint(dst + C::kTileBytes, &p.v_map_h, bar(C::kFull + s), bx * 64, first + start(it), h, b,
                           policy);
        }
        ++issued;
      }
      if (*abort_flag)
        for (int i = max(0, issued - C::kStages); i < issued; ++i)
          wait_drain(bar(C::kFull + i % C::kStages), (i / C::kStages) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t lead = elect_lead();
    constexpr uint32_t id_u = idesc_bf16_f32(128, D, 1) | kAMajorMN;
    const uint64_t mn = smem_desc_sw128(base_u32, C::kBoxBytes, 1024);
    auto at = [](uint64_t d, uint32_t off) { return make_desc((uint32_t)d + (off >> 4), (uint32_t)(d >> 32)); };
    bool ok = true;
    for (int it = 0; it < nt; ++it) {
      const int s = it % C::kStages;
      ok = __all_sync(0xffffffffu, wait(C::kScaled + (it & 1), (it / 2) & 1u, 13) &&
                                       wait(C::kFull + s, (it / C::kStages) & 1u, 13));
      if (!ok) break;
      tc_fence_after();
      const uint32_t k = s * C::kStageBytes, v = k + C::kTileBytes, rest = C::kRestOff + (it & 1) * C::kRestBytes;
      if constexpr (TERMS == 3) {
        const int g = it / C::kGroup, buf = g & 1;
        const bool fresh = it % C::kGroup == 0;
        if (fresh && g >= 2) {
          ok = __all_sync(0xffffffffu, wait(C::kGroupFree + buf, (g / 2 - 1) & 1u, 13));
          if (!ok) break;
          tc_fence_after();
        }
        const uint32_t acc = tmem + (uint32_t)buf * 2 * D;
#pragma unroll
        for (int t = TERMS - 1; t >= 0; --t)
#pragma unroll
          for (int kk = 0; kk < C::kRows / 16; ++kk)
            mma_ss_l(lead, t == 0 ? acc : acc + D, at(mn, (t == 0 ? k : rest + (t - 1) * C::kTileBytes) + kk * 2048u),
                     at(mn, v + kk * 2048u), id_u, !fresh || t == 1 || kk > 0);
        if (it % C::kGroup == C::kGroup - 1 || it + 1 == nt) mma_commit_l(lead, bar(C::kGroupFull + buf));
      } else {
#pragma unroll
        for (int t = 0; t < TERMS; ++t)
#pragma unroll
          for (int kk = 0; kk < C::kRows / 16; ++kk)
            mma_ss_l(lead, tmem, at(mn, (t == 0 ? k : rest + (t - 1) * C::kTileBytes) + kk * 2048u),
                     at(mn, v + kk * 2048u), id_u, it > 0 || t > 0 || kk > 0);
      }
      // to the group that scales step it + 2, and to the load of step it +
      // kStages; nobody waits for the last two (see the tile kernel)
      if (it + 2 < nt) mma_commit_l(lead, bar(C::kEmpty + s));
    }
    if (TERMS != 3 && ok) mma_commit_l(lead, bar(C::kFinal));
    if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else {
    const int grp = (warp - 2) >> 3, tid = (threadIdx.x - 64) & 255, hf = ((warp - 2) >> 2) & 1, quad = warp & 3;
    const int row = quad * 32 + lane;
    constexpr int kCols = D / 2;
    // TERMS = 3: this thread's quarter of the row, summed over the groups
    constexpr int kPart = D / 4;
    const int part = ((warp - 2) >> 2) & 3;
    float sum[TERMS == 3 ? kPart : 1];
    int added = 0;  // groups
    auto add_group = [&]() {
      const int buf = added & 1;
      if (!__all_sync(0xffffffffu, wait(C::kGroupFull + buf, (added / 2) & 1u, 15))) return false;
      tc_fence_after();
      const uint32_t src = tmem + ((uint32_t)(quad * 32) << 16) + buf * 2 * D + part * kPart;
#pragma unroll
      for (int c0 = 0; c0 < kPart; c0 += 16) {
        uint32_t x[16], y[16];
        tmem_ld16(src + c0, x);
        tmem_ld16(src + D + c0, y);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 16; ++c) sum[c0 + c] += __uint_as_float(x[c]) + __uint_as_float(y[c]);
      }
      tc_fence_before();
      warp_arrive(bar(C::kGroupFree + buf), lane);
      ++added;
      return true;
    };
    if constexpr (TERMS == 3) {
#pragma unroll
      for (int c = 0; c < kPart; ++c) sum[c] = 0.f;
    }
    bool ok = true;
    for (int it = grp; it < nt; it += 2) {
      const int s = it % C::kStages, t0 = start(it);  // from the segment's first token
      ok = __all_sync(0xffffffffu, wait(C::kFull + s, (it / C::kStages) & 1u, 15));
      // the parts' tiles are free once the group's previous step has been multiplied
      if (ok && it >= 2)
        ok = __all_sync(0xffffffffu, wait(C::kEmpty + (it - 2) % C::kStages, ((it - 2) / C::kStages) & 1u, 15));
      if (!ok) break;
      uint8_t* k = base + s * C::kStageBytes;
      const int after = count - t0 - C::kRows;  // tokens behind the step (forward); missing ones if negative
      scale_rows<D, C::kRows, TERMS>(k, base + C::kRestOff + grp * C::kRestBytes, C::kTileBytes, k + C::kTileBytes, tid,
                                     count - t0, ex2((float)(p.reverse ? t0 : max(after, 0)) * ld2),
                                     p.reverse ? w_tab : w_tab + max(-after, 0));
      fence_proxy_async_smem();
      warp_arrive(bar(C::kScaled + grp), lane);
      if constexpr (TERMS == 3) {  // the group before has been multiplied by now
        if (it % C::kGroup >= 2 && it >= C::kGroup && !(ok = add_group())) break;
      }
    }
    if constexpr (TERMS == 3) {
      while (ok && added * C::kGroup < nt) ok = add_group();
      if (__all_sync(0xffffffffu, ok && !*abort_flag) && row < D) {
        float* out = p.carry + (bh * p.nseg + seg) * D * D + piece_index<D>(row, part * kPart);
#pragma unroll
        for (int c = 0; c < kPart; c += 4)
          *reinterpret_cast<float4*>(out + c * 2 * D) = make_float4(sum[c], sum[c + 1], sum[c + 2], sum[c + 3]);
      }
    } else {
      if (ok && grp == 0) ok = __all_sync(0xffffffffu, wait(C::kFinal, 0, 15));
      ok = ok && grp == 0;
      ok = ok && !*abort_flag;
      if (__all_sync(0xffffffffu, ok)) {
        tc_fence_after();
        float* out = p.carry + (bh * p.nseg + seg) * D * D + piece_index<D>(row, hf * kCols);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t x[32];
          if (nt > 0) {
            tmem_ld32(tmem + ((uint32_t)(quad * 32) << 16) + hf * kCols + c0, x);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) x[c] = 0u;
          }
          if (row < D) {
#pragma unroll
            for (int c = 0; c < 32; c += 4)
              *reinterpret_cast<uint4*>(out + (c0 + c) * 2 * D) = make_uint4(x[c], x[c + 1], x[c + 2], x[c + 3]);
          }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, C::kTmemCols);
  }
}

// Chains the segments' contributions, in place, into the state before every
// segment; the state after the last goes to state_out.  One thread per four
// elements; the contributions are fetched kAhead segments ahead.
constexpr int kMaxSegments = 256;
template <int D>
__global__ void __launch_bounds__(128) decay_carry_kernel(const __grid_constant__ DecayRuns runs) {
  unsigned block;
  const DecayTileParams& p = pick(runs, block);
  constexpr int kAhead = 16, kBlocks = D * D / 512;
  __shared__ float2 decays[kMaxSegments];
  const long long bh = block / kBlocks;
  const int e = ((int)(block % kBlocks) * 128 + threadIdx.x) * 4;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const int nrun = p.state_out != nullptr ? p.nseg : p.nseg - 1;
  if (!in_bounds(p, bh, p.nseg - 1)) return;
  float* c = p.carry + bh * p.nseg * D * D + e;
  // its place in the caller's states, where (row, col) may be held at (col, row)
  const int row = (e / 4) % D, col = (e / (8 * D)) * 4 + ((e / 4) % (2 * D) / D) * (D / 2);
  const long long io = bh * D * D + (p.state_t ? col * D + row : row * D + col);
  griddep_wait();
  griddep_launch_dependents();
  float4 add[kAhead];
  auto fetch = [&](int s0) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (s0 + i < nrun) add[i] = *reinterpret_cast<const float4*>(c + (long long)(s0 + i) * D * D);
  };
  fetch(0);
  const float ln = decay_ln(p.log_decay, h);
  const bool zero = decays_to_zero(ln);
  for (int i = threadIdx.x; i < nrun; i += 128) {
    const Decay d((float)Run(p, b, i).count() * ln, zero);
    decays[i] = make_float2(d.hi, d.lo);
  }
  float4 s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (p.state_in != nullptr)
    s = p.state_t ? make_float4(p.state_in[io], p.state_in[io + D], p.state_in[io + 2 * D], p.state_in[io + 3 * D])
                  : *reinterpret_cast<const float4*>(p.state_in + io);
  __syncthreads();
  for (int s0 = 0; s0 < p.nseg; s0 += kAhead) {
    if (s0 > 0) fetch(s0);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      if (s0 + i < p.nseg) *reinterpret_cast<float4*>(c + (long long)(s0 + i) * D * D) = s;
      if (s0 + i < nrun) {
        const float2 d = decays[s0 + i];
        s.x = fmaf(s.x, d.x, s.x * d.y) + add[i].x;
        s.y = fmaf(s.y, d.x, s.y * d.y) + add[i].y;
        s.z = fmaf(s.z, d.x, s.z * d.y) + add[i].z;
        s.w = fmaf(s.w, d.x, s.w * d.y) + add[i].w;
      }
    }
  }
  if (p.state_out != nullptr) {
    float* out = p.state_out + io;
    if (p.state_t)
      out[0] = s.x, out[D] = s.y, out[2 * D] = s.z, out[3 * D] = s.w;
    else
      *reinterpret_cast<float4*>(out) = s;
  }
}

template <typename P>
cudaError_t launch(void (*kernel)(P), unsigned grid, unsigned threads, size_t smem, const P& p, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid, 1, 1);
  cfg.blockDim = dim3(threads, 1, 1);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Raises a kernel's shared-memory limit, once per device.
template <typename K>
cudaError_t allow_smem(K* kernel, size_t bytes, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev <= 63 && (ready.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev <= 63) ready.fetch_or(1ull << dev);
  return e;
}

template <int D, int TERMS>
cudaError_t launch_segments(DecayRuns& r, cudaStream_t s) {
  using C = SegCfg<D, TERMS>;
  static std::atomic<unsigned long long> ready{0};
  cudaError_t e = allow_smem(decay_segment_kernel<D, TERMS>, C::kSmemBytes, ready);
  if (e != cudaSuccess) return e;
  const unsigned bh = (unsigned)r.run[0].B * r.run[0].H;
  unsigned grid = 0;
  for (int i = 0; i < r.n; ++i) {
    grid += bh * (r.run[i].state_out != nullptr ? r.run[i].nseg : r.run[i].nseg - 1);
    if (i == 0) r.first = grid;
  }
  e = launch(decay_segment_kernel<D, TERMS>, grid, C::kThreads, C::kSmemBytes, r, s);
  if (e != cudaSuccess) return e;
  r.first = bh * (D * D / 512);
  return launch(decay_carry_kernel<D>, r.first * r.n, 128, 0, r, s);
}

template <int D, int TERMS>
cudaError_t launch_tiles(DecayRuns& r, cudaStream_t s) {
  using C = TileCfg<D, TERMS>;
  static std::atomic<unsigned long long> ready{0};
  const cudaError_t e = allow_smem(decay_tile_kernel<D, TERMS>, C::kSmemBytes, ready);
  if (e != cudaSuccess) return e;
  r.first = (unsigned)r.run[0].B * r.run[0].H * r.run[0].nseg;
  return launch(decay_tile_kernel<D, TERMS>, r.first * r.n, C::kThreads, C::kSmemBytes, r, s);
}

bool wants_state(const DecayRuns& r) {
  for (int i = 0; i < r.n; ++i)
    if (r.run[i].state_out != nullptr) return true;
  return false;
}

}  // namespace

// k enters a state that the caller gets as three bf16 parts (24 bits), a state
// that only feeds bf16 outputs as two (16 bits).
cudaError_t launch_decay_segments(DecayRuns& r, cudaStream_t s) {
  if (wants_state(r)) return r.run[0].D == 128 ? launch_segments<128, 3>(r, s) : launch_segments<64, 3>(r, s);
  return r.run[0].D == 128 ? launch_segments<128, 2>(r, s) : launch_segments<64, 2>(r, s);
}

cudaError_t launch_decay_tiles(DecayRuns& r, cudaStream_t s) {
  if (wants_state(r)) {
    if (r.n != 1) return cudaErrorInvalidValue;
    return r.run[0].D == 128 ? launch_tiles<128, 3>(r, s) : launch_tiles<64, 3>(r, s);
  }
  return r.run[0].D == 128 ? launch_tiles<128, 2>(r, s) : launch_tiles<64, 2>(r, s);
}

cudaError_t launch_decay_short(const DecayTileParams& p, cudaStream_t s) {
  const unsigned grid = (unsigned)((long long)p.B * p.H * (p.D / 32));
  return p.D == 128 ? launch(decay_short_kernel<128>, grid, 256, 0, p, s)
                    : launch(decay_short_kernel<64>, grid, 256, 0, p, s);
}

cudaError_t launch_decay_step(const DecayStepParams& p, cudaStream_t s) {
  const long long bh = (long long)p.B * p.H;
  return p.D == 128 ? launch(decay_step_kernel<128, 32>, (unsigned)(bh * 4), 256, 0, p, s)
                    : launch(decay_step_kernel<64, 32>, (unsigned)(bh * 2), 256, 0, p, s);
}

}  // namespace sab
