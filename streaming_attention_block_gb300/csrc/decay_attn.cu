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
// fp32 registers.  W K would lose the state 8 bits, so it is split into a bf16
// part and the bf16 rest, two products: 16 bits.
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
__device__ __forceinline__ bool wait_bounded(uint32_t bar, uint32_t parity, volatile int* abort_flag, unsigned site,
                                             unsigned* err_word) {
  if (mbar_test_wait(bar, parity)) return true;
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
__device__ __forceinline__ void wait_drain(uint32_t bar, uint32_t parity, unsigned* err_word) {
  const uint64_t t0 = global_ns();
#pragma unroll 1
  while (!mbar_try_wait(bar, parity)) {
    if (global_ns() - t0 > kTimeoutNs) {
      if (err_word != nullptr) atomicOr(err_word, 1u << 31);
      return;
    }
  }
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

// k rows of a tile times mul * g^(e0 + sg * row), in place as bf16 with the
// bf16 rest in `rest`; rows from n on become zero.  Both tiles are 128-byte
// swizzled; a row's 16-byte pieces keep their places, so they need no
// unscrambling.  `v`, if given, also loses its rows from n on: they may hold
// anything, and 0 * NaN would reach every output.
template <int D>
__device__ __forceinline__ void scale_rows(uint8_t* k, uint8_t* rest, uint8_t* v, int tid, int n, float mul, float ld2,
                                           int e0, int sg) {
  constexpr int kPieces = D / 8;  // per row
#pragma unroll 4
  for (int i = tid; i < kC * kPieces; i += 256) {
    const int row = i / kPieces, c = i % kPieces;
    const uint32_t off = (uint32_t)((c >> 3) * (kC * 128) + row * 128 + (c & 7) * 16);
    uint32_t hi[4], lo[4];
    if (row < n) {
      const float w = mul * ex2((float)(e0 + sg * row) * ld2);
      const uint4 x = *reinterpret_cast<const uint4*>(k + off);
      const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float a = __uint_as_float(xs[j] << 16) * w, b = __uint_as_float(xs[j] & 0xFFFF0000u) * w;
        hi[j] = pack_bf16(a, b);
        lo[j] = pack_bf16(a - __uint_as_float(hi[j] << 16), b - __uint_as_float(hi[j] & 0xFFFF0000u));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) hi[j] = lo[j] = 0u;
      if (v != nullptr) *reinterpret_cast<uint4*>(v + off) = make_uint4(0u, 0u, 0u, 0u);
    }
    *reinterpret_cast<uint4*>(k + off) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    *reinterpret_cast<uint4*>(rest + off) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
  }
}
template <int D>
__device__ __forceinline__ void zero_rows(uint8_t* v, int tid, int n) {
  constexpr int kPieces = D / 8;
  for (int i = n * kPieces + tid; i < kC * kPieces; i += 256) {
    const int row = i / kPieces, c = i % kPieces;
    *reinterpret_cast<uint4*>(v + (c >> 3) * (kC * 128) + row * 128 + (c & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
  }
}

constexpr uint32_t kAMajorMN = 1u << 15;  // instruction descriptor: A is MN-major

template <int D_>
struct TileCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = kC * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kVStages = D == 128 ? 1 : 2;
  // (D = 64: the update's A operand, M = 128, takes its upper 64 rows from the
  // box behind a k tile; they land in accumulator rows that nothing reads)
  static constexpr uint32_t kQOff = 0;                                   // [2]; the output is staged over q
  static constexpr uint32_t kKOff = kQOff + 2 * kTileBytes;              // [2]; scaled in place
  static constexpr uint32_t kRestOff = kKOff + 2 * kTileBytes;
  static constexpr uint32_t kVOff = kRestOff + kTileBytes;
  static constexpr uint32_t kStOff = kVOff + kVStages * kTileBytes;      // bf16 state [D][D]
  static constexpr uint32_t kStBoxBytes = D * 128u;
  static constexpr uint32_t kBarOff = kStOff + kBoxes * kStBoxBytes;
  static constexpr int kFullQ = 0, kFullK = 2, kFullV = 4;               // [2] each
  static constexpr int kEmptyQ = 6, kEmptyK = 8, kEmptyV = 10;           // [2] each
  static constexpr int kSFull = 12, kPFull = 13, kKwFull = 14, kOFull = 15, kUFull = 16, kStFull = 17, kOut = 18 /* [2] */,
                       kDrain = 20, kNumBars = 21;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;           // tmem address, abort flag
  static constexpr uint32_t kTabOff = (kMiscOff + 16 + 15) & ~15u;        // 32 decay powers, read 16 bytes at a time
  static constexpr uint32_t kSmemBytes = kTabOff + 128 + 1024;
  static constexpr int kThreads = 352;  // producer, MMA, 8 element warps, store
  static constexpr uint32_t kS = 0, kIntra = 128, kInter = 128 + D, kUpd = 128 + 2 * D;  // TMEM columns
  static_assert(kSmemBytes <= 232448, "shared memory budget");
  static_assert(kTabOff % 16 == 0 && kStOff % 1024 == 0, "alignment");
};

template <int D>
__global__ void __launch_bounds__(TileCfg<D>::kThreads, 1)
decay_tile_kernel(const __grid_constant__ DecayTileParams p) {
  using C = TileCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  float* tab = reinterpret_cast<float*>(base + C::kTabOff);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int seg = blockIdx.x % p.nseg;
  const long long bh = blockIdx.x / p.nseg;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);

  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i)
      mbar_init(bar(i), i == C::kPFull || i == C::kKwFull || i == C::kStFull || i == C::kOut || i == C::kOut + 1 ? 256 : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Run run(p, b, seg);
  const float ln = decay_ln(p.log_decay, h), ld2 = ln * kLog2e;
  if (threadIdx.x < 32) tab[lane] = ex2((float)(p.reverse ? lane : 31 - lane) * ld2);
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
      auto load = [&](const CUtensorMap* m, uint32_t off, int fb, int row) {
        mbar_arrive_expect_tx(bar(fb), C::kTileBytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + off + bx * C::kBoxBytes, m, bar(fb), bx * 64, row, h, b);
      };
      int nq = 0, nk = 0, nv = 0;
      bool ok = true;
      for (int it = 0; ok && it < nt; ++it) {
        const int s = it & 1, row = run.tile(run.a + it) * kC, sv = it % C::kVStages;
        if (it >= 2) ok = wait(C::kEmptyK + s, (it / 2 - 1) & 1u, 9);
        if (!ok) break;
        load(&p.k_map, C::kKOff + s * C::kTileBytes, C::kFullK + s, row), ++nk;
        if (it >= 2) ok = wait(C::kEmptyQ + s, (it / 2 - 1) & 1u, 9);
        if (!ok) break;
        load(&p.q_map, C::kQOff + s * C::kTileBytes, C::kFullQ + s, row), ++nq;
        if (it >= C::kVStages) ok = wait(C::kEmptyV + sv, (it / C::kVStages - 1) & 1u, 9);
        if (!ok) break;
        load(&p.v_map, C::kVOff + sv * C::kTileBytes, C::kFullV + sv, row), ++nv;
      }
      if (*abort_flag) {
        for (int i = max(0, nk - 2); i < nk; ++i) wait_drain(bar(C::kFullK + (i & 1)), (i / 2) & 1u, p.err_word);
        for (int i = max(0, nq - 2); i < nq; ++i) wait_drain(bar(C::kFullQ + (i & 1)), (i / 2) & 1u, p.err_word);
        for (int i = max(0, nv - C::kVStages); i < nv; ++i)
          wait_drain(bar(C::kFullV + i % C::kVStages), (i / C::kVStages) & 1u, p.err_word);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ---------------------------------------------------------- MMA issuer
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
    bool ok = true;
    for (int it = 0; ok && it < nt; ++it) {
      const int s = it & 1, sv = it % C::kVStages;
      const uint32_t q = C::kQOff + s * C::kTileBytes, k = C::kKOff + s * C::kTileBytes,
                     v = C::kVOff + sv * C::kTileBytes;
      ok = wait_all(C::kFullQ + s, (it / 2) & 1u, 10) && wait_all(C::kFullK + s, (it / 2) & 1u, 10);
      if (!ok) break;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_e(tmem + C::kS, at(kmaj, q + k_off(kk)), at(kmaj, k + k_off(kk)), id_s, kk > 0);
      mma_commit_e(bar(C::kSFull));
      if (!(ok = wait_all(C::kStFull, it & 1u, 11))) break;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        mma_ss_e(tmem + C::kInter, at(kmaj, q + k_off(kk)), at(mn_st, C::kStOff + kk * 2048u), id_o, kk > 0);
      ok = wait_all(C::kPFull, it & 1u, 12) && wait_all(C::kFullV + sv, (it / C::kVStages) & 1u, 10);
      if (!ok) break;
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ts_e(tmem + C::kIntra, tmem + C::kS + (kk >> 2) * 64 + (kk & 3) * 8, at(mn, v + kk * 2048u), id_o, kk > 0);
      mma_commit_e(bar(C::kOFull));
      if (it >= n_upd) break;
      if (!(ok = wait_all(C::kKwFull, it & 1u, 13))) break;
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ss_e(tmem + C::kUpd, at(mn, k + kk * 2048u), at(mn, v + kk * 2048u), id_u, kk > 0);
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ss_e(tmem + C::kUpd, at(mn, C::kRestOff + kk * 2048u), at(mn, v + kk * 2048u), id_u, 1u);
      mma_commit_e(bar(C::kUFull));
      mma_commit_e(bar(C::kEmptyK + s));
      mma_commit_e(bar(C::kEmptyV + sv));
    }
    if (__any_sync(0xffffffffu, !ok || *abort_flag)) {
      mma_commit_e(bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 10) {
    // --------------------------------------------------------- output store
    if (lane == 0) {
      for (int it = 0; it < nt; ++it) {
        if (!wait(C::kOut + (it & 1), (it / 2) & 1u, 14)) break;
        const int row = run.tile(run.a + it) * kC;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_store_4d(&p.o_map, base_u32 + C::kQOff + (it & 1) * C::kTileBytes + bx * C::kBoxBytes, bx * 64, row, h, b);
        tma_store_commit_and_wait_read();
        mbar_arrive(bar(C::kEmptyQ + (it & 1)));
      }
    }
    __syncwarp();
  } else {
    // -------------------------------------------------------- element work
    const int tid = threadIdx.x - 64;
    const int hf = (warp - 2) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;  // token of the tile; key dimension of the state
    const uint32_t lane_off = tmem + ((uint32_t)(quad * 32) << 16);
    constexpr int kCols = D / 2;       // state and output columns of this thread: [hf D/2, (hf + 1) D/2)
    const bool rev = p.reverse != 0;
    const float p_mul = p.o_mul * p.kv_mul;
    float st[kCols];
    // offset of 16-byte piece c (8 columns) of a row in a swizzled tile
    auto piece = [&](int c, uint32_t box_bytes) {
      const int cc = hf * (kCols / 8) + c;
      return (uint32_t)((cc >> 3) * box_bytes + row * 128 + (((cc & 7) ^ (row & 7)) << 4));
    };
    auto publish_state = [&]() {
      if (row < D) {
#pragma unroll
        for (int c = 0; c < kCols / 8; ++c)
          *reinterpret_cast<uint4*>(base + C::kStOff + piece(c, C::kStBoxBytes)) =
              make_uint4(pack_bf16(st[8 * c], st[8 * c + 1]), pack_bf16(st[8 * c + 2], st[8 * c + 3]),
                         pack_bf16(st[8 * c + 4], st[8 * c + 5]), pack_bf16(st[8 * c + 6], st[8 * c + 7]));
      }
      fence_proxy_async_smem();
      tc_fence_before();
      mbar_arrive(bar(C::kStFull));
    };
    // the state before the segment: carried ones are stored as this run holds
    // them, the caller's possibly transposed
    const float* in = p.nseg > 1 ? p.carry + (bh * p.nseg + seg) * D * D
                                 : p.state_in != nullptr ? p.state_in + bh * D * D : nullptr;
    const bool in_t = p.nseg == 1 && p.state_t;
#pragma unroll
    for (int c = 0; c < kCols; ++c) st[c] = 0.f;
    if (in != nullptr && row < D && nt > 0) {
      if (in_t) {
#pragma unroll
        for (int c = 0; c < kCols; ++c) st[c] = in[(long long)(hf * kCols + c) * D + row];
      } else {
#pragma unroll
        for (int c = 0; c < kCols / 4; ++c) {
          const float4 x = *reinterpret_cast<const float4*>(in + (long long)row * D + hf * kCols + 4 * c);
          st[4 * c] = x.x, st[4 * c + 1] = x.y, st[4 * c + 2] = x.z, st[4 * c + 3] = x.w;
        }
      }
    }
    if (nt > 0) publish_state();
    bool ok = true;
    for (int it = 0; it < nt; ++it) {
      const int s = it & 1, n = run.tokens(run.a + it);
      uint8_t* kt = base + C::kKOff + s * C::kTileBytes;
      uint8_t* vt = base + C::kVOff + (it % C::kVStages) * C::kTileBytes;
      // 1. P = decayed, masked scores, bf16, over the scores
      ok = __all_sync(0xffffffffu, wait(C::kSFull, it & 1u, 15));
      if (!ok) break;
      tc_fence_after();
#pragma unroll
      for (int pass = 0; pass < 2; ++pass) {
        const int c0 = hf * 64 + 32 * pass;
        const uint32_t src = lane_off + C::kS + c0, dst = lane_off + C::kS + hf * 64 + 16 * pass;
        uint32_t pk[16];
        const bool none = (rev ? c0 + 31 < quad * 32 : c0 > quad * 32 + 31) || c0 >= n;
        if (none) {
#pragma unroll
          for (int c = 0; c < 16; ++c) pk[c] = 0u;
        } else {
          uint32_t sv[32];
          tmem_ld32(src, sv);
          tmem_wait_ld();
          if (n == kC && c0 != quad * 32) {
            // whole block on the visible side: g^|i - j| as the distance to the
            // block's near edge times the table's powers, both at most 1
            const float f = p_mul * ex2((float)(rev ? c0 - row : row - c0 - 31) * ld2);
#pragma unroll
            for (int c4 = 0; c4 < 8; ++c4) {
              const float4 t = *reinterpret_cast<const float4*>(tab + 4 * c4);
              pk[2 * c4] = pack_bf16(__uint_as_float(sv[4 * c4]) * (f * t.x), __uint_as_float(sv[4 * c4 + 1]) * (f * t.y));
              pk[2 * c4 + 1] =
                  pack_bf16(__uint_as_float(sv[4 * c4 + 2]) * (f * t.z), __uint_as_float(sv[4 * c4 + 3]) * (f * t.w));
            }
          } else {
            auto one = [&](int c) {
              const int j = c0 + c, d = rev ? j - row : row - j;
              return d >= 0 && j < n ? __uint_as_float(sv[c]) * (p_mul * ex2((float)d * ld2)) : 0.f;
            };
#pragma unroll
            for (int c = 0; c < 16; ++c) pk[c] = pack_bf16(one(2 * c), one(2 * c + 1));
          }
        }
        tmem_st16(dst, pk);
      }
      tmem_wait_st();
      if (n < kC) {  // padding of v must not meet the zeros of P
        ok = __all_sync(0xffffffffu, wait(C::kFullV + it % C::kVStages, (it / C::kVStages) & 1u, 15));
        if (!ok) break;
        zero_rows<D>(vt, tid, n);
        fence_proxy_async_smem();
      }
      tc_fence_before();
      mbar_arrive(bar(C::kPFull));
      // 2. scaled k for the update
      if (it < n_upd) {
        ok = __all_sync(0xffffffffu, wait(C::kFullK + s, (it / 2) & 1u, 15));
        if (!ok) break;
        scale_rows<D>(kt, base + C::kRestOff, nullptr, tid, n, p.kv_mul, ld2, rev ? 1 : n - 1, rev ? 1 : -1);
        fence_proxy_async_smem();
        mbar_arrive(bar(C::kKwFull));
      }
      // 3. output rows, staged over q
      ok = __all_sync(0xffffffffu, wait(C::kOFull, it & 1u, 15));
      if (!ok) break;
      tc_fence_after();
      {
        const float f = p.o_mul * ex2((float)(rev ? n - 1 - row : row + 1) * ld2);
        uint8_t* ot = base + C::kQOff + s * C::kTileBytes;
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t x[32], y[32];
          tmem_ld32(lane_off + C::kIntra + hf * kCols + c0, x);
          tmem_ld32(lane_off + C::kInter + hf * kCols + c0, y);
          tmem_wait_ld();
          uint32_t o[16];
#pragma unroll
          for (int c = 0; c < 16; ++c)
            o[c] = row < n ? pack_bf16(fmaf(__uint_as_float(y[2 * c]), f, __uint_as_float(x[2 * c])),
                                       fmaf(__uint_as_float(y[2 * c + 1]), f, __uint_as_float(x[2 * c + 1])))
                           : 0u;
#pragma unroll
          for (int c = 0; c < 4; ++c)
            *reinterpret_cast<uint4*>(ot + piece(c0 / 8 + c, C::kBoxBytes)) =
                make_uint4(o[4 * c], o[4 * c + 1], o[4 * c + 2], o[4 * c + 3]);
        }
      }
      tc_fence_before();
      fence_proxy_async_smem();
      mbar_arrive(bar(C::kOut + s));
      // 4. the state after the tile
      if (it < n_upd) {
        ok = __all_sync(0xffffffffu, wait(C::kUFull, it & 1u, 15));
        if (!ok) break;
        tc_fence_after();
        const Decay decay((float)n * ln);
#pragma unroll
        for (int c0 = 0; c0 < kCols; c0 += 32) {
          uint32_t x[32];
          tmem_ld32(lane_off + C::kUpd + hf * kCols + c0, x);
          tmem_wait_ld();
#pragma unroll
          for (int c = 0; c < 32; ++c) st[c0 + c] = decay(st[c0 + c]) + __uint_as_float(x[c]);
        }
        if (it + 1 < nt) publish_state();
      }
    }
    // an aborted CTA stores no state; its outputs are not valid either
    if (ok && !*abort_flag && p.state_out != nullptr && row < D) {
      float* out = p.state_out + bh * D * D;
      if (nt == 0 && in != nullptr) {  // nothing live: the state passes through
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          st[c] = in_t ? in[(long long)(hf * kCols + c) * D + row] : in[(long long)row * D + hf * kCols + c];
      }
#pragma unroll
      for (int c = 0; c < kCols; ++c)
        out[p.state_t ? (long long)(hf * kCols + c) * D + row : (long long)row * D + hf * kCols + c] = st[c];
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
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// A segment's own contribution to the state after it: the tiles' updates with
// the decays to the segment's end, accumulated in TMEM over the segment.
template <int D_>
struct SegCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = kC * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kStages = 2;
  static constexpr uint32_t kStageBytes = 3 * kTileBytes;  // k (scaled in place), its rest, v
  static constexpr uint32_t kBarOff = kStages * kStageBytes;
  static constexpr int kFull = 0, kScaled = 2, kEmpty = 4, kFinal = 6, kDrain = 7, kNumBars = 8;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16 + 1024;
  static constexpr int kThreads = 320;
};

template <int D>
__global__ void __launch_bounds__(SegCfg<D>::kThreads, 1)
decay_segment_kernel(const __grid_constant__ DecayTileParams p) {
  using C = SegCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int nrun = p.state_out != nullptr ? p.nseg : p.nseg - 1;  // the last segment's is wanted by state_out only
  const int seg = blockIdx.x % nrun;
  const long long bh = blockIdx.x / nrun;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  if (threadIdx.x == 0) {
    for (int i = 0; i < C::kNumBars; ++i) mbar_init(bar(i), i == C::kScaled || i == C::kScaled + 1 ? 256 : 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 128);
    tmem_relinquish();
  }
  griddep_launch_dependents();
  griddep_wait();
  const Run run(p, b, seg);
  const float ld2 = decay_ln(p.log_decay, h) * kLog2e;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  const int nt = run.b - run.a;
  auto wait = [&](int i, uint32_t parity, unsigned site) {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };
  if (warp == 0) {
    if (lane == 0) {
      int issued = 0;
      for (int it = 0; it < nt; ++it) {
        const int s = it & 1, row = run.tile(run.a + it) * kC;
        if (it >= 2 && !wait(C::kEmpty + s, (it / 2 - 1) & 1u, 9)) break;
        mbar_arrive_expect_tx(bar(C::kFull + s), 2 * C::kTileBytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx) {
          const uint32_t dst = base_u32 + s * C::kStageBytes + bx * C::kBoxBytes;
          tma_load_4d(dst, &p.k_map, bar(C::kFull + s), bx * 64, row, h, b);
          tma_load_4d(dst + 2 * C::kTileBytes, &p.v_map, bar(C::kFull + s), bx * 64, row, h, b);
        }
        ++issued;
      }
      if (*abort_flag)
        for (int i = max(0, issued - 2); i < issued; ++i) wait_drain(bar(C::kFull + (i & 1)), (i / 2) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp == 1) {
    constexpr uint32_t id_u = idesc_bf16_f32(128, D, 1) | kAMajorMN;
    const uint64_t mn = smem_desc_sw128(base_u32, C::kBoxBytes, 1024);
    auto at = [](uint64_t d, uint32_t off) { return make_desc((uint32_t)d + (off >> 4), (uint32_t)(d >> 32)); };
    bool ok = true;
    for (int it = 0; it < nt; ++it) {
      const int s = it & 1;
      ok = __all_sync(0xffffffffu, wait(C::kScaled + s, (it / 2) & 1u, 13) && wait(C::kFull + s, (it / 2) & 1u, 13));
      if (!ok) break;
      tc_fence_after();
      const uint32_t k = s * C::kStageBytes, v = k + 2 * C::kTileBytes;
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ss_e(tmem, at(mn, k + kk * 2048u), at(mn, v + kk * 2048u), id_u, it > 0 || kk > 0);
#pragma unroll
      for (int kk = 0; kk < kC / 16; ++kk)
        mma_ss_e(tmem, at(mn, k + C::kTileBytes + kk * 2048u), at(mn, v + kk * 2048u), id_u, 1u);
      mma_commit_e(bar(C::kEmpty + s));
    }
    mma_commit_e(bar(ok ? C::kFinal : C::kDrain));
    if (!ok && lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    __syncwarp();
  } else {
    const int tid = threadIdx.x - 64, hf = (warp - 2) >> 2, quad = warp & 3, row = quad * 32 + lane;
    constexpr int kCols = D / 2;
    const int first = run.first(), end = first + run.count();
    bool ok = true;
    for (int it = 0; it < nt; ++it) {
      const int s = it & 1, t0 = run.tile(run.a + it) * kC;
      ok = __all_sync(0xffffffffu, wait(C::kFull + s, (it / 2) & 1u, 15));
      if (!ok) break;
      uint8_t* k = base + s * C::kStageBytes;
      scale_rows<D>(k, k + C::kTileBytes, k + 2 * C::kTileBytes, tid, run.tokens(run.a + it), p.kv_mul, ld2,
                    p.reverse ? t0 - first + 1 : end - 1 - t0, p.reverse ? 1 : -1);
      fence_proxy_async_smem();
      mbar_arrive(bar(C::kScaled + s));
    }
    if (ok) ok = __all_sync(0xffffffffu, wait(C::kFinal, 0, 15));
    ok = ok && !*abort_flag;
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      float* out = p.carry + (bh * p.nseg + seg) * D * D + (long long)row * D + hf * kCols;
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
            *reinterpret_cast<uint4*>(out + c0 + c) = make_uint4(x[c], x[c + 1], x[c + 2], x[c + 3]);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 128);
  }
}

// Chains the segments' contributions, in place, into the state before every
// segment; the state after the last goes to state_out.  One thread per element.
template <int D>
__global__ void __launch_bounds__(256) decay_carry_kernel(const __grid_constant__ DecayTileParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const long long bh = blockIdx.x / (D * D / 256);
  const int e = (int)(blockIdx.x % (D * D / 256)) * 256 + threadIdx.x;
  const int b = (int)(bh / p.H), h = (int)(bh % p.H);
  const float ln = decay_ln(p.log_decay, h);
  const int e_io = p.state_t ? (e % D) * D + e / D : e;  // the caller's orientation
  float s = p.state_in != nullptr ? p.state_in[bh * D * D + e_io] : 0.f;
  float* c = p.carry + bh * p.nseg * D * D + e;
  const int nrun = p.state_out != nullptr ? p.nseg : p.nseg - 1;
  float next = nrun > 0 ? c[0] : 0.f;
  for (int seg = 0; seg < p.nseg; ++seg) {
    const float add = next;
    if (seg + 1 < nrun) next = c[(long long)(seg + 1) * D * D];
    c[(long long)seg * D * D] = s;
    if (seg < nrun) s = Decay((float)Run(p, b, seg).count() * ln)(s) + add;
  }
  if (p.state_out != nullptr) p.state_out[bh * D * D + e_io] = s;
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

template <int D>
cudaError_t launch_tiles(const DecayTileParams& p, cudaStream_t s) {
  static std::atomic<unsigned long long> ready{0};  // devices whose kernels have their shared-memory limit raised
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  if (dev > 63 || !(ready.load() >> dev & 1)) {
    e = cudaFuncSetAttribute(decay_tile_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             (int)TileCfg<D>::kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(decay_segment_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)SegCfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    if (dev <= 63) ready.fetch_or(1ull << dev);
  }
  const long long bh = (long long)p.B * p.H;
  DecayTileParams q = p;
  if (p.nseg > 1) {
    const int nrun = p.state_out != nullptr ? p.nseg : p.nseg - 1;
    e = launch(decay_segment_kernel<D>, (unsigned)(bh * nrun), SegCfg<D>::kThreads, SegCfg<D>::kSmemBytes, p, s);
    if (e != cudaSuccess) return e;
    e = launch(decay_carry_kernel<D>, (unsigned)(bh * (D * D / 256)), 256, 0, p, s);
    if (e != cudaSuccess) return e;
    q.state_out = nullptr;  // written by the carry kernel
  }
  return launch(decay_tile_kernel<D>, (unsigned)(bh * p.nseg), TileCfg<D>::kThreads, TileCfg<D>::kSmemBytes, q, s);
}

}  // namespace

cudaError_t launch_decay_tiles(const DecayTileParams& p, cudaStream_t s) {
  return p.D == 128 ? launch_tiles<128>(p, s) : launch_tiles<64>(p, s);
}

cudaError_t launch_decay_step(const DecayStepParams& p, cudaStream_t s) {
  const long long bh = (long long)p.B * p.H;
  return p.D == 128 ? launch(decay_step_kernel<128, 32>, (unsigned)(bh * 4), 256, 0, p, s)
                    : launch(decay_step_kernel<64, 32>, (unsigned)(bh * 2), 256, 0, p, s);
}

}  // namespace sab
