// Gradients of cross attention for sm_103a.  With P recomputed from the
// forward's LSE and delta_i = sum_d dO_id O_id:
//   dV = P^T dO,  dP = dO V^T,  dS = P * (dP - delta),
//   dQ = scale * dS K,  dK = scale * dS^T Q.
// Two kernels.  cross_dq_kernel walks query tiles (persistent, as the forward:
// a query tile meets few key tiles) and works out delta on the way;
// cross_dkv_kernel keeps a key tile and streams all queries that read it: of
// every head of its group and, where the states are shared, of every sequence,
// so that these sums are formed in the accumulators.  Key tiles are few, so the
// queries of one are cut among several blocks, whose parts cross_sum_kernel adds
// in order: no atomics, equal calls give equal bits.  S and dP are formed in both
// kernels: 14 D products a pair for the 10 D of one, whose dQ would go through
// memory in fp32 parts, one for each key tile.
#include <math.h>

#include "cross_common.cuh"

namespace sab {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// What is added to a row's scores for P, from its LSE.  -inf: P is 0, also where
// all scores were -inf (they and an infinity would be no number, and that of every
// key's gradient).
__device__ __forceinline__ float minus_lse(float lse) { return lse == -INFINITY ? -INFINITY : -lse * kLog2e; }

// Where the n-th of a run of tile pairs is, of which one is done with before the
// other (V before K, dO before Q): N pairs of places in turn, the one done with
// last where the other was.
template <int N>
__device__ __forceinline__ int last_slot(int n) {
  return 2 * (n % N) + ((n / N) & 1);
}
template <int N>
__device__ __forceinline__ int first_slot(int n) {
  return last_slot<N>(n) ^ 1;
}

// ------------------------------------------------------------------- dQ, delta

template <int D_>
struct DqCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr uint32_t kQOff = 0, kGOff = kTileBytes;  // Q of an item, dO of two
  static constexpr int kPairs = D == 128 ? 2 : 4;           // of K and V tiles
  static constexpr uint32_t kRingOff = 3 * kTileBytes;
  static constexpr uint32_t kStatOff = kRingOff + 2 * kPairs * kTileBytes;  // [2 items][128] {-LSE log2 e, -delta}
  static constexpr uint32_t kBarOff = kStatOff + 2048;
  static constexpr int kQFull = 0;
  static constexpr int kQFree = 1;            // an item's last scores are done
  static constexpr int kGFull = 2;            // [2 items] dO
  static constexpr int kOut = 4;              // [2] dQ is where dO was
  static constexpr int kSFull = 6;            // S
  static constexpr int kSRead = 7;            // S is read
  static constexpr int kPFull = 8;            // dP
  static constexpr int kGrad = 9;             // dS
  static constexpr int kDone = 10;            // [2 items] the last product
  static constexpr int kRead = 12;            // [2] dQ is taken out
  static constexpr int kStat = 14;            // [2] LSE and delta are there
  static constexpr int kSeen = 16;            // [2] all warps for dS have them
  static constexpr int kMeet = 18;            // [4 quadrants] the two warps of a row
  static constexpr int kDrain = 22;           // [2 warps with products]
  static constexpr int kFull = 24;            // [2 kPairs]
  static constexpr int kEmpty = kFull + 2 * kPairs;  // [2 kPairs]
  static constexpr int kNumBars = kEmpty + 2 * kPairs;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSeqsOff = kMiscOff + 16;  // [kMaxSorted + 1]
  static constexpr uint32_t kSmemBytes = kSeqsOff + (kMaxSorted + 1) * 4;
  // Q, dO, dQ; S; dP and dQ's products; K and V; 8 warps for dS; 4 for delta and dQ
  static constexpr int kThreads = 32 * 16;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// dS of an item with one key tile, for one warp of those for dS (64 keys): delta
// is formed here, from all of its row, as sum_j P_ij dP_ij.  O needs not be read,
// and with few keys its rounding showed in delta (6 keys: error of dQ 2.9e-3 of
// its norm, 2.35e-3 so).  A function of its own: its code would lie in the way of
// the longer items' (2 to 5 % of their time).  2 x 30720 queries over 77 keys, 12
// heads of 128: 280 us for all gradients with O read, 248 so.
template <int D>
__device__ __noinline__ bool one_tile(const CrossBwdParams& p, uint32_t bars, volatile int* abort_flag, float2* stat,
                                      uint32_t n, uint32_t item, uint32_t meets, uint32_t tS, int keys, int b, int hb,
                                      int t0) {
  using C = DqCfg<D>;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, cg = (int)(threadIdx.x >> 7) - 1;
  auto wait = [&](int i, uint32_t parity, unsigned site) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bars + 8u * (uint32_t)i, parity & 1u, abort_flag, site, p.err_word));
  };
  auto arrive = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bars + 8u * (uint32_t)i);
  };
  const uint32_t tG = tS + 128u;
  const int hi = keys - cg * 64;  // this half's keys
  const float lse = stat->x;
  arrive(C::kSeen + (int)(item & 1u));
  if (!wait(C::kSFull, n, 11) || !wait(C::kPFull, n, 12)) return false;
  tc_fence_after();
  // 32 columns of P and dP; zeros past the end, where they may be no numbers
  auto take = [&](int cc, float2 (&pr)[16], uint32_t (&g)[32]) {
    uint32_t v[32];
    tmem_ld32(tS + 32 * cc, v);
    tmem_ld32(tG + 32 * cc, g);
    tmem_wait_ld();
    const int left = hi - 32 * cc;
    if (left < 32) {
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        v[k] = k < left ? v[k] : 0xff800000u;
        g[k] = k < left ? g[k] : 0u;
      }
    }
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])),
                                  make_float2(p.scale_log2, p.scale_log2), make_float2(lse, lse));
      pr[k] = make_float2(ex2(x.x), ex2(x.y));
    }
  };
  float2 pr[16];
  uint32_t g[32];
  float2 acc = make_float2(0.f, 0.f);
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    take(cc, pr, g);
#pragma unroll
    for (int k = 0; k < 16; ++k)
      acc = __ffma2_rn(pr[k], make_float2(__uint_as_float(g[2 * k]), __uint_as_float(g[2 * k + 1])), acc);
  }
  // the halves of a row meet where longer items have LSE and delta, once all have read LSE
  if (!wait(C::kSeen + (int)(item & 1u), item >> 1, 13)) return false;
  float* meet = reinterpret_cast<float*>(stat);
  meet[cg] = acc.x + acc.y;
  arrive(C::kMeet + quad);
  if (!wait(C::kMeet + quad, meets, 16)) return false;
  const float delta = meet[0] + meet[1];
  const float2 nd = make_float2(-delta, -delta);
  const float one = keys == 1 ? 0.f : 1.f;  // one key: P is 1 whatever its score is
#pragma unroll 1
  for (int cc = 0; cc < 2; ++cc) {
    take(cc, pr, g);
    uint32_t o[16];
#pragma unroll
    for (int k = 0; k < 16; ++k) {
      const float2 x = __fmul2_rn(
          __fmul2_rn(pr[k], __fadd2_rn(make_float2(__uint_as_float(g[2 * k]), __uint_as_float(g[2 * k + 1])), nd)),
          make_float2(one, one));
      o[k] = pack_bf16(x.x, x.y);
    }
    tmem_st16(tG + 16 * cc, o);
  }
  tmem_wait_st();
  tc_fence_before();
  arrive(C::kSRead);
  arrive(C::kGrad);
  if (cg == 0) {
    const int row = quad * 32 + lane, row_t = row / p.pack, head = hb * p.pack + row - row_t * p.pack;
    if (row_t < p.tile_tokens && t0 + row_t < p.Lq)
      p.delta[((long long)b * p.H + head) * p.Lq + t0 + row_t] = delta;
  }
  __syncwarp();
  return true;
}

// P stays in registers, so S is free for the next tile as soon as it is read, and
// two warps issue products: one S = Q K^T, the other dP = dO V^T and, once dS is
// over dP, dQ += dS K.  TMEM: S, dP, and dQ of two items, one being taken out.
// SHORT: items may have one key tile; RAGGED: lengths of sequences are given.
template <int D, bool SHORT, bool RAGGED>
__global__ void __launch_bounds__(DqCfg<D>::kThreads, 1) cross_dq_kernel(const __grid_constant__ CrossBwdParams p) {
  using C = DqCfg<D>;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t base_u32 = smem_u32(base);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);  // [0] tmem, [1] abort
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kMiscOff + 4);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  auto wait = [&](int i, uint32_t parity, unsigned site) -> bool {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };
  auto wait_warp = [&](int i, uint32_t parity, unsigned site) -> bool {
    return __all_sync(0xffffffffu, wait(i, parity, site));
  };
  const int warp = uniform<true>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto arrive_warp = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };

  if (threadIdx.x == 0) {
    mbar_init(bar(C::kQFull), 1);
    mbar_init(bar(C::kQFree), 1);
    mbar_init(bar(C::kSFull), 1);
    mbar_init(bar(C::kSRead), 8);
    mbar_init(bar(C::kPFull), 1);
    mbar_init(bar(C::kGrad), 8);
    for (int i = 0; i < 4; ++i) mbar_init(bar(C::kMeet + i), 2);
    for (int i = 0; i < 2 * C::kPairs; ++i) {
      mbar_init(bar(C::kFull + i), 1);
      mbar_init(bar(C::kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kGFull + i), 1);
      mbar_init(bar(C::kOut + i), 4);
      mbar_init(bar(C::kDone + i), 1);
      mbar_init(bar(C::kRead + i), 4);
      mbar_init(bar(C::kStat + i), 4);
      mbar_init(bar(C::kSeen + i), 8);
      mbar_init(bar(C::kDrain + i), 1);
    }
    misc[1] = (base_u32 & 1023u) != 0;  // the tiles' swizzle counts on it
    if (misc[1] != 0 && p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(base_u32 + C::kMiscOff, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform<true>((int)misc[0]);
  griddep_launch_dependents();
  griddep_wait();

  Pass pass;
  pass.first = blockIdx.x;
  pass.step = gridDim.x;
  pass.end = uniform<true>(*abort_flag) ? 0u : p.items;
  pass.list = pass.seqs = nullptr;
  pass.pair = 1;
  pass.split = 0;
  if (RAGGED && p.sorted) {
    uint32_t* seqs = reinterpret_cast<uint32_t*>(base + C::kSeqsOff);
    sort_sequences(p, 1, seqs, reinterpret_cast<uint32_t*>(base + C::kStatOff));
    pass.seqs = seqs;
    const unsigned rounds = ((unsigned)uniform<true>((int)(seqs[p.B] >> 6)) + gridDim.x - 1) / gridDim.x;
    if (pass.end > 0) pass.end = rounds * gridDim.x;
  }
  pass.by = spot_of(p, gridDim.x, 1);

  if (warp == 0) {
    // -------------------------------------------- Q, dO an item ahead, dQ out
    if (RAGGED && !uniform<true>(*abort_flag)) {
      fill_zeros(base + C::kGOff, C::kTileBytes);
      clear_tiles<C::kBoxes>(p, 1, base_u32 + C::kGOff, nullptr);
    }
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(C::kBoxes * p.pack * p.tile_tokens) * 128u;
      int at[2][3];  // where the last two items are
      auto out = [&](int item) -> bool {
        const int buf = item & 1;
        if (!wait(C::kOut + buf, (uint32_t)(item >> 1) & 1u, 0)) return false;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_store_4d(&p.o_map, base_u32 + C::kGOff + buf * C::kTileBytes + bx * C::kBoxBytes, bx * 64, at[0][0],
                       at[0][1], at[0][2]);
        tma_store_commit_and_wait_read();
        return true;
      };
      auto later = [&]() {
#pragma unroll
        for (int i = 0; i < 3; ++i) at[0][i] = at[1][i];
      };
      int item = 0, q_loads = 0;
      bool ok = true;
      Walk<false, RAGGED> c, o;
      o.start(p, pass);
      for (c.start(p, pass); c.more(pass); c.next(p, pass)) {
        const Work& w = c.w;
        if (o.more(pass)) o.next(p, pass);
        if (w.nt == 0) continue;
        const int buf = item & 1;
        if (item >= 2 && !(ok = out(item - 2))) break;
        const int c1 = query_c1(p, w, 0), c2 = query_c2(p, w, 0);
        mbar_arrive_expect_tx(bar(C::kGFull + buf), q_bytes);
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + C::kGOff + buf * C::kTileBytes + bx * C::kBoxBytes, &p.do_map, bar(C::kGFull + buf),
                      bx * 64, c1, c2, w.b);
        ++item;
        later();
        at[1][0] = c1, at[1][1] = c2, at[1][2] = w.b;
        // Q has one place, which the item before still needs, and O of the item
        // after it is loaded by the warps for delta: both are brought near
        for (int bx = 0; bx < C::kBoxes; ++bx) {
          tma_prefetch_4d(&p.q_map, bx * 64, c1, c2, w.b);
          if (o.more(pass) && o.w.nt > (SHORT ? 1 : 0))
            tma_prefetch_4d(&p.of_map, bx * 64, query_c1(p, o.w, 0), query_c2(p, o.w, 0), o.w.b);
        }
        if (item >= 2 && !(ok = wait(C::kQFree, (uint32_t)(item - 2) & 1u, 0))) break;
        mbar_arrive_expect_tx(bar(C::kQFull), q_bytes);
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + C::kQOff + bx * C::kBoxBytes, &p.q_map, bar(C::kQFull), bx * 64, c1, c2, w.b);
        ++q_loads;
      }
      if (item == 1) later();
      for (int k = max(0, item - 2); ok && k < item; ++k) {
        ok = out(k);
        later();
      }
      tma_store_wait_all();
      if (*abort_flag) {  // nothing of this block's copies may land after it
        for (int k = max(0, item - 2); k < item; ++k)
          wait_drain(bar(C::kGFull + (k & 1)), (uint32_t)(k >> 1) & 1u, p.err_word);
        if (q_loads > 0) wait_drain(bar(C::kQFull), (uint32_t)(q_loads - 1) & 1u, p.err_word);
      }
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------------ K, V
    if (lane == 0) {
      int n[2] = {0, 0};  // K and V tiles
      bool ok = true;
      auto load = [&](int which, const CUtensorMap* m, int row, int head, int b) -> bool {
        const int k = n[which];
        const int at = which == 0 ? last_slot<C::kPairs>(k) : first_slot<C::kPairs>(k);
        if (k >= C::kPairs && !wait(C::kEmpty + at, (uint32_t)(k / C::kPairs - 1) & 1u, 1)) return false;
        mbar_arrive_expect_tx(bar(C::kFull + at), C::kTileBytes);
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + C::kRingOff + at * C::kTileBytes + bx * C::kBoxBytes, m, bar(C::kFull + at), bx * 64,
                      row, head, b);
        ++n[which];
        return true;
      };
      Walk<false, RAGGED> c;
      for (c.start(p, pass); ok && c.more(pass); c.next(p, pass)) {
        const Work& w = c.w;
        const int head = w.hb * p.pack / p.group, kb = p.Bk == 1 ? 0 : w.b;
        for (int j = 0; ok && j < w.nt; ++j)
          ok = load(0, &p.k_map, j * kTileN, head, kb) && load(1, &p.v_map, j * kTileN, head, kb);
      }
      if (*abort_flag)
        for (int which = 0; which < 2; ++which)
          for (int k = max(0, n[which] - C::kPairs); k < n[which]; ++k)
            wait_drain(bar(C::kFull + (which == 0 ? last_slot<C::kPairs>(k) : first_slot<C::kPairs>(k))),
                       (uint32_t)(k / C::kPairs) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------ S = Q K^T
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
    const uint64_t dq = smem_desc_sw128(base_u32 + C::kQOff, 16, 1024);
    const uint32_t dk = (uint32_t)smem_desc_sw128(base_u32 + C::kRingOff, 16, 1024), hi = (uint32_t)(dq >> 32);
    const uint32_t lead = elect_lead();
    int n = 0, item = 0;
    bool ok = true;
    Walk<true, RAGGED> c;
    c.start(p, pass);
    c.seek(p, pass);
    while (ok && c.more(pass)) {
      const int nt = c.w.nt;
      c.next(p, pass);  // while the products before run
      c.seek(p, pass);
      if (!(ok = wait_warp(C::kQFull, (uint32_t)item & 1u, 2))) break;
      for (int j = 0; j < nt; ++j, ++n) {
        const int slot = last_slot<C::kPairs>(n);
        // In this order: V of the tile two before was in K's place, and this warp
        // does not wait for V.  Once S of the tile before is read, that V's product
        // is done, and the parity cannot be taken for that of the fill before it.
        if (n > 0 && !(ok = wait_warp(C::kSRead, (n - 1) & 1u, 4))) break;
        if (!(ok = wait_warp(C::kFull + slot, (uint32_t)(n / C::kPairs) & 1u, 3))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_l(lead, tmem, make_desc((uint32_t)dq + off, hi), make_desc(dk + slot * (C::kTileBytes >> 4) + off, hi),
                   idesc_s, kk > 0 ? 1u : 0u);
        }
        mma_commit_l(lead, bar(C::kSFull));
      }
      if (!ok) break;
      mma_commit_l(lead, bar(C::kQFree));
      ++item;
    }
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ---------------------------------------------- dP = dO V^T, dQ += dS K
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
    constexpr uint32_t idesc_q = idesc_bf16_f32(128, D, 1);
    constexpr uint32_t kTile = C::kTileBytes >> 4;
    const uint64_t dg = smem_desc_sw128(base_u32 + C::kGOff, 16, 1024);
    const uint32_t dv = (uint32_t)smem_desc_sw128(base_u32 + C::kRingOff, 16, 1024);
    const uint64_t dm = smem_desc_sw128(base_u32 + C::kRingOff, C::kBoxBytes, 1024);  // as the MN-major operand
    const uint32_t hi_k = (uint32_t)(dg >> 32), hi_mn = (uint32_t)(dm >> 32);
    const uint32_t tG = tmem + 128u;
    const uint32_t lead = elect_lead();
    int n = 0, item = 0;
    bool ok = true;
    Walk<true, RAGGED> c;
    c.start(p, pass);
    c.seek(p, pass);
    while (ok && c.more(pass)) {
      const int nt = c.w.nt, keys = c.w.keys, buf = item & 1;
      const uint32_t tQ = tmem + 256u + (uint32_t)(buf * D), g0 = (uint32_t)dg + (uint32_t)buf * kTile;
      c.next(p, pass);
      c.seek(p, pass);
      if (!(ok = wait_warp(C::kGFull + buf, (uint32_t)(item >> 1) & 1u, 5))) break;
      for (int j = 0; j < nt; ++j, ++n) {
        const int ks = last_slot<C::kPairs>(n), vs = first_slot<C::kPairs>(n), live = keys - j * kTileN;
        if (!(ok = wait_warp(C::kFull + vs, (uint32_t)(n / C::kPairs) & 1u, 6))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_l(lead, tG, make_desc(g0 + off, hi_k), make_desc(dv + vs * kTile + off, hi_k), idesc_s,
                   kk > 0 ? 1u : 0u);
        }
        mma_commit_l(lead, bar(C::kPFull));
        mma_commit_l(lead, bar(C::kEmpty + vs));
        // the item two before has its dQ taken out before this one's goes over it
        if (j == 0 && item >= 2 && !(ok = wait_warp(C::kRead + buf, (uint32_t)((item >> 1) - 1) & 1u, 7))) break;
        if (!(ok = wait_warp(C::kFull + ks, (uint32_t)(n / C::kPairs) & 1u, 8))) break;
        const int steps = min(8, (live + 15) >> 4);  // 16 keys each
        // keys past the sequence's end may hold anything, and 0 * NaN is NaN
        if (__builtin_expect(steps * 16 > live, 0))
          zero_rows<C::kBoxes>(base + C::kRingOff + ks * C::kTileBytes, live, steps * 16);
        if (!(ok = wait_warp(C::kGrad, n & 1u, 9))) break;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          if (kk < steps)
            mma_ts_l(lead, tQ, tG + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8),
                     make_desc((uint32_t)dm + ks * kTile + ((uint32_t)(kk * 16 * 128) >> 4), hi_mn), idesc_q,
                     j + kk > 0 ? 1u : 0u);
        mma_commit_l(lead, bar(C::kEmpty + ks));  // S, of which dS was made, is done too
      }
      if (!ok) break;
      mma_commit_l(lead, bar(C::kDone + buf));
      ++item;
    }
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain + 1));
      if (lane == 0) wait_drain(bar(C::kDrain + 1), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------------------- dS
    const int cg = (warp - 4) >> 2, quad = warp & 3;  // 64 keys each
    const int row = quad * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)cg * 64u, tG = tS + 128u;
    float2* stat = reinterpret_cast<float2*>(base + C::kStatOff) + row;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    int n = 0, item = 0, meets = 0;
    bool ok = true;
    Walk<true, RAGGED> c;
    c.start(p, pass);
    c.seek(p, pass);
    while (ok && c.more(pass)) {
      const int nt = c.w.nt, keys = c.w.keys, b = c.w.b, hb = c.w.hb, t0 = c.w.t0;
      c.next(p, pass);
      c.seek(p, pass);
      if (!(ok = wait_warp(C::kStat + (item & 1), (uint32_t)(item >> 1) & 1u, 10))) break;
      if (SHORT && nt == 1) {
        ok = one_tile<D>(p, base_u32 + C::kBarOff, abort_flag, stat + (item & 1) * 128, (uint32_t)n, (uint32_t)item,
                         (uint32_t)meets, tS, keys, b, hb, t0);
        ++n, ++item, ++meets;
        continue;
      }
      const float2 st = stat[(item & 1) * 128];
      arrive_warp(C::kSeen + (item & 1));
      const float2 nl = make_float2(st.x, st.x), nd = make_float2(st.y, st.y);
      for (int j = 0; j < nt; ++j, ++n) {
        if (!(ok = wait_warp(C::kSFull, n & 1u, 11))) break;
        tc_fence_after();
        float2 pr[32];
        {
          uint32_t v[32], u[32];
          tmem_ld32(tS, v);
          tmem_ld32(tS + 32, u);
          tmem_wait_ld();
          tc_fence_before();
          arrive_warp(C::kSRead);
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc2, nl);
            const float2 y = __ffma2_rn(make_float2(__uint_as_float(u[2 * k]), __uint_as_float(u[2 * k + 1])), sc2, nl);
            pr[k] = make_float2(ex2(x.x), ex2(x.y));
            pr[16 + k] = make_float2(ex2(y.x), ex2(y.y));
          }
        }
        const int hi = keys - j * kTileN - cg * 64;
        if (!(ok = wait_warp(C::kPFull, n & 1u, 12))) break;
        tc_fence_after();
#pragma unroll
        for (int cc = 0; cc < 2; ++cc) {
          uint32_t v[32], o[16];
          tmem_ld32(tG + 32 * cc, v);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = __fmul2_rn(
                pr[16 * cc + k],
                __fadd2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), nd));
            o[k] = pack_bf16(x.x, x.y);
          }
          if (__builtin_expect(hi - 32 * cc < 32, 0)) {  // keys past the end
#pragma unroll
            for (int k = 0; k < 16; ++k) {
              const int left = hi - 32 * cc - 2 * k;
              o[k] = left > 1 ? o[k] : left > 0 ? o[k] & 0xFFFFu : 0u;
            }
          }
          tmem_st16(tG + 16 * cc, o);  // over what this warp has read
        }
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(C::kGrad);
      }
      ++item;
    }
  } else {
    // ------------------------------------------------------------ delta, dQ
    // delta of the next item is formed while this one's products run; O comes
    // from global memory, for there is no room for it beside the tiles of the products.
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tQ = tmem + ((uint32_t)(quad * 32) << 16) + 256u;
    const int row_t = row / p.pack, row_g = row - row_t * p.pack;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of an access
    const uint32_t inv = (65535u + (uint32_t)p.pack) / (uint32_t)p.pack;  // r * inv >> 16 = r / pack below 128
    const int sub = lane / kLanes, col = lane % kLanes;  // 16-byte pieces
    bool ok = true;
    auto alive = [&](const Work& w) { return row_t < w.live && row_t < p.tile_tokens; };
    auto stats = [&](const Work& w, int item) {
      float2* stat = reinterpret_cast<float2*>(base + C::kStatOff) + (item & 1) * 128;
      const bool live = alive(w);
      const long long at = ((long long)w.b * p.H + w.hb * p.pack + row_g) * p.Lq + w.t0 + row_t;
      const float lse = live ? ld_global(p.LSE + at) : INFINITY;
      if (item >= 2 && !wait_warp(C::kSeen + (item & 1), (uint32_t)((item >> 1) - 1) & 1u, 13)) return false;
      if (SHORT && w.nt == 1) {  // delta comes from P and dP
        stat[row].x = live ? minus_lse(lse) : -INFINITY;
        arrive_warp(C::kStat + (item & 1));
        return true;
      }
      const uint16_t* o_base = p.O + w.b * p.o_batch + w.t0 * p.o_token + w.hb * p.pack * p.o_head + col * 8;
      const uint8_t* g_base = base + (item & 1) * C::kTileBytes + C::kGOff + (col >> 3) * C::kBoxBytes;
#pragma unroll 1
      for (int s0 = 0; s0 < kLanes; s0 += 8) {
        uint4 a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = quad * 32 + (s0 + i) * kRows + sub;
          const int rt = (int)((uint32_t)r * inv >> 16), rg = r - rt * p.pack;
          a[i] = make_uint4(0u, 0u, 0u, 0u);
          if (rt < w.live && rt < p.tile_tokens)
            a[i] = *reinterpret_cast<const uint4*>(o_base + rt * p.o_token + rg * p.o_head);
        }
        if (s0 == 0 && !wait_warp(C::kGFull + (item & 1), (uint32_t)(item >> 1) & 1u, 14)) return false;
        float d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = quad * 32 + (s0 + i) * kRows + sub;
          const uint4 g = *reinterpret_cast<const uint4*>(g_base + r * 128 + (((col & 7) ^ (r & 7)) << 4));
          const uint32_t x[4] = {a[i].x, a[i].y, a[i].z, a[i].w}, y[4] = {g.x, g.y, g.z, g.w};
          float2 acc = make_float2(0.f, 0.f);
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc = __ffma2_rn(make_float2(__uint_as_float(x[k] << 16), __uint_as_float(x[k] & 0xFFFF0000u)),
                             make_float2(__uint_as_float(y[k] << 16), __uint_as_float(y[k] & 0xFFFF0000u)), acc);
          d[i] = acc.x + acc.y;
        }
        // sums over a row's lanes, halving the rows a lane holds at each step
        int mine = 0;
#pragma unroll
        for (int n = 4, bit = kLanes / 2; n > 0; n >>= 1, bit >>= 1) {
          const bool up = lane & bit;
          mine = 2 * mine + (up ? 1 : 0);
#pragma unroll
          for (int i = 0; i < n; ++i) {
            const float keep = up ? d[i + n] : d[i], send = up ? d[i] : d[i + n];
            d[i] = keep + __shfl_xor_sync(0xffffffffu, send, bit);
          }
        }
        if (kLanes == 16) d[0] += __shfl_xor_sync(0xffffffffu, d[0], 1);
        if (kLanes == 8 || (lane & 1) == 0) stat[quad * 32 + (s0 + mine) * kRows + sub].y = -d[0];
      }
      __syncwarp();
      const float nd = stat[row].y;
      stat[row] = make_float2(live ? minus_lse(lse) : -INFINITY, live ? nd : 0.f);
      if (live) p.delta[at] = -nd;
      arrive_warp(C::kStat + (item & 1));
      return true;
    };
    Walk<true, RAGGED> c;
    c.start(p, pass);
    c.seek(p, pass);
    bool more = c.more(pass);
    Work w = c.w;
#pragma unroll 1
    for (int item = -1; ok && more; ++item) {
      if (item >= 0) {
        w = c.w;
        c.next(p, pass);
        c.seek(p, pass);
      }
      const bool ahead = c.more(pass);
      if (ahead && !(ok = stats(c.w, item + 1))) break;
      if (item < 0) continue;
      more = ahead;
      const bool live = alive(w);
      uint8_t* out = base + C::kGOff + (item & 1) * C::kTileBytes + row * 128;
      if (!(ok = wait_warp(C::kDone + (item & 1), (uint32_t)(item >> 1) & 1u, 15))) break;
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t v[32];
        tmem_ld32(tQ + (item & 1) * D + cc, v);
        tmem_wait_ld();
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = 8 * i + 2 * k;
            o[k] = live ? pack_bf16(__uint_as_float(v[e]) * p.scale, __uint_as_float(v[e + 1]) * p.scale) : 0u;
          }
          const int k = cc / 8 + i;
          *reinterpret_cast<uint4*>(out + (k >> 3) * C::kBoxBytes + (((k & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
      tc_fence_before();
      arrive_warp(C::kRead + (item & 1));
      fence_proxy_async_smem();
      arrive_warp(C::kOut + (item & 1));
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// -------------------------------------------------------------------- dK, dV

template <int D_>
struct DkvCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kStages = D == 128 ? 2 : 4;
  static constexpr uint32_t kKOff = 0, kVOff = kTileBytes;  // resident
  static constexpr uint32_t kStageOff = 2 * kTileBytes;
  static constexpr uint32_t kStatOff = kStageOff + 2 * kStages * kTileBytes;  // [kStages][2][128] -LSE log2 e, -delta
  static constexpr uint32_t kBarOff = kStatOff + kStages * 1024;
  static constexpr int kRes = 0;
  static constexpr int kStat = 1;                     // [kStages]
  static constexpr int kFull = kStat + kStages;       // [2 kStages] Q and dO tiles
  static constexpr int kEmpty = kFull + 2 * kStages;  // [2 kStages] both streams are done with it
  static constexpr int kSFull = kEmpty + 2 * kStages; // [2 streams] S^T, dP^T
  static constexpr int kPFull = kSFull + 2;       // [2] P^T, dS^T
  static constexpr int kDone = kPFull + 2;        // [2]
  static constexpr int kDrain = kDone + 2;        // [2]
  static constexpr int kNumBars = kDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16;
  // loads; S and dV; dP and dK; a spare; 8 warps for P and dS, and the end
  static constexpr int kThreads = 32 * 12;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// The query tiles of a block: of the sequences, head blocks and tiles that read
// its keys, its share.
struct Stream {
  int i, end;      // tiles
  int iq, hb, b;   // this one's place: tile, head block of the group, sequence
  int live;        // its tokens inside q_len
};

// S^T, dP^T, dV and dK of 128 keys and 128 queries fill TMEM, so the two streams
// that take turns on the tensor cores are S = K Q^T, dV += P^T dO and dP = V dO^T,
// dK += dS^T Q, each with a warp that issues its products: while one's products
// run, the eight warps between turn the other's scores into its operand, P over S
// and dS over dP.  Halves of query tiles as streams took 3090 cycles a tile
// against 2560 of their products, whose 64 columns do not keep up with the reads
// of the other operand; whole ones have 2048.
template <int D>
__global__ void __launch_bounds__(DkvCfg<D>::kThreads, 1) cross_dkv_kernel(const __grid_constant__ CrossBwdParams p) {
  using C = DkvCfg<D>;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t base_u32 = smem_u32(base);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);  // [0] tmem, [1] abort
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kMiscOff + 4);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  auto wait_warp = [&](int i, uint32_t parity, unsigned site) -> bool {
    return __all_sync(0xffffffffu, wait_bounded(bar(i), parity, abort_flag, site, p.err_word));
  };
  const int warp = uniform<true>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  auto arrive_warp = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };
  // key tile, key head, sequence of keys, and share of the queries
  const int key_tiles = (p.Lk + kTileN - 1) / kTileN;
  unsigned u = blockIdx.x;
  const int k0 = (int)(u % (unsigned)key_tiles) * kTileN;
  u /= (unsigned)key_tiles;
  const int hk = (int)(u % (unsigned)p.Hk);
  u /= (unsigned)p.Hk;
  const int kb = (int)(u % (unsigned)p.Bk), share = (int)(u / (unsigned)p.Bk);

  if (threadIdx.x == 0) {
    mbar_init(bar(C::kRes), 1);
    for (int i = 0; i < C::kStages; ++i) mbar_init(bar(C::kStat + i), 1);
    for (int i = 0; i < 2 * C::kStages; ++i) {
      mbar_init(bar(C::kFull + i), 1);
      mbar_init(bar(C::kEmpty + i), 2);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + i), 8);
      mbar_init(bar(C::kDone + i), 1);
      mbar_init(bar(C::kDrain + i), 1);
    }
    misc[1] = (base_u32 & 1023u) != 0 || (kDebugBounds && share >= p.shares);
    if (misc[1] != 0 && p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
    fence_mbar_init();
  }
  // rows that no copy fills (3 heads x 42 tokens leave two) are zeros
  const int rows = p.pack * p.tile_tokens;
  if (rows < kTileM) {
    const int n = (kTileM - rows) * 8;
    for (int i = threadIdx.x; i < C::kStages * 2 * C::kBoxes * n; i += blockDim.x) {
      const int box = i / n, k = i - box * n;
      uint8_t* to = base + C::kStageOff + box * C::kBoxBytes;
      *reinterpret_cast<uint4*>(to + (rows + (k >> 3)) * 128 + (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
    }
  }
  fence_proxy_async_smem();
  if (warp == 1) {
    tmem_alloc(base_u32 + C::kMiscOff, 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = (uint32_t)uniform<true>((int)misc[0]);
  griddep_launch_dependents();
  griddep_wait();
  const int keys = length_of<true>(p.kv_len, kb, p.Lk) - k0;  // of this tile, from 128 on whole
  const bool dead = keys <= 0 || uniform<true>(*abort_flag) != 0;

  const int blocks = p.group / p.pack, seqs = p.Bk == 1 ? p.B : 1;
  // every shares-th tile, so that each share has its part of every sequence
  Stream first;
  first.i = share;
  first.end = dead ? first.i : (int)((long long)seqs * blocks * p.n_qtiles);
  const int by_r = p.shares / p.n_qtiles;
  const int by_iq = p.shares - by_r * p.n_qtiles, by_b = by_r / blocks, by_hb = by_r - by_b * blocks;
  {
    const int r = share / p.n_qtiles;
    first.iq = share - r * p.n_qtiles;
    first.b = (p.Bk == 1 ? 0 : kb) + r / blocks;
    first.hb = r % blocks;
  }
  auto advance = [&](Stream& s) {
    s.i += p.shares;
    s.iq += by_iq;
    s.hb += by_hb;
    s.b += by_b;
    if (s.iq >= p.n_qtiles) s.iq -= p.n_qtiles, ++s.hb;
    if (s.hb >= blocks) s.hb -= blocks, ++s.b;
  };
  // the next tile with a live query, from this one on
  auto seek = [&](Stream& s) {
    for (; s.i < s.end; advance(s)) {
      if constexpr (kDebugBounds) {
        if (s.b >= p.B || s.hb >= blocks || s.iq >= p.n_qtiles) {
          if (p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
          *abort_flag = 1;
          s.i = s.end;
          return;
        }
      }
      s.live = min(p.tile_tokens, length_of<true>(p.q_len, s.b, p.Lq) - s.iq * p.tile_tokens);
      if (s.live > 0) return;
    }
  };
  auto next = [&](Stream& s) {
    advance(s);
    seek(s);
  };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool any = first.i < first.end;
    if (lane == 0 && any) {
      mbar_arrive_expect_tx(bar(C::kRes), 2 * C::kTileBytes);
#pragma unroll
      for (int bx = 0; bx < C::kBoxes; ++bx) {
        tma_load_4d(base_u32 + C::kKOff + bx * C::kBoxBytes, &p.k_map, bar(C::kRes), bx * 64, k0, hk, kb);
        tma_load_4d(base_u32 + C::kVOff + bx * C::kBoxBytes, &p.v_map, bar(C::kRes), bx * 64, k0, hk, kb);
      }
    }
    const uint32_t tile_bytes = (uint32_t)(C::kBoxes * rows) * 128u;
    // four rows a lane: place within the tile's heads and tokens
    int tok[4], hd[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = lane + 32 * i;
      tok[i] = r / p.pack;
      hd[i] = r - tok[i] * p.pack;
    }
    Stream s = first;
    seek(s);
    float ls[4], dl[4];
    bool has[4];  // of the tile to be loaded next, requested one tile ahead
    auto fetch = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = s.iq * p.tile_tokens + tok[i], head = hk * p.group + s.hb * p.pack + hd[i];
        const long long at = ((long long)s.b * p.H + head) * p.Lq + t;
        has[i] = tok[i] < s.live && lane + 32 * i < rows;
        ls[i] = dl[i] = 0.f;
        if (has[i]) ls[i] = ld_global(p.LSE + at), dl[i] = ld_global(p.delta + at);
      }
    };
    if (s.i < s.end) fetch();
    int loads[2] = {0, 0};  // Q and dO tiles
    auto load = [&](int which, const CUtensorMap* m) -> bool {
      const int k = loads[which], at = which == 0 ? last_slot<C::kStages>(k) : first_slot<C::kStages>(k);
      if (k >= C::kStages && !wait_warp(C::kEmpty + at, (uint32_t)(k / C::kStages - 1) & 1u, 0)) return false;
      if (lane == 0) {
        const int head = hk * p.group + s.hb * p.pack, t = s.iq * p.tile_tokens;
        const int c1 = p.pack == 1 ? t : head, c2 = p.pack == 1 ? head : t;
        const uint32_t full = bar(C::kFull + at);
        mbar_arrive_expect_tx(full, tile_bytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + C::kStageOff + at * C::kTileBytes + bx * C::kBoxBytes, m, full, bx * 64, c1, c2, s.b);
      }
      __syncwarp();
      ++loads[which];
      return true;
    };
    bool ok = true;
    while (s.i < s.end) {
      const int st = loads[0] % C::kStages;
      if (!(ok = load(0, &p.q_map) && load(1, &p.do_map))) break;
      float* stat = reinterpret_cast<float*>(base + C::kStatOff + st * 1024);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        stat[lane + 32 * i] = has[i] ? minus_lse(ls[i]) : -INFINITY;
        stat[128 + lane + 32 * i] = -dl[i];
      }
      arrive_warp(C::kStat + st);
      next(s);
      if (s.i < s.end) fetch();
    }
    if (lane == 0 && *abort_flag) {
      if (any) wait_drain(bar(C::kRes), 0, p.err_word);
      for (int which = 0; which < 2; ++which)
        for (int k = max(0, loads[which] - C::kStages); k < loads[which]; ++k)
          wait_drain(bar(C::kFull + (which == 0 ? last_slot<C::kStages>(k) : first_slot<C::kStages>(k))),
                     (uint32_t)(k / C::kStages) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------- products of a stream
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 128, 0);
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, D, 1);
    constexpr uint32_t kTile = C::kTileBytes >> 4;
    const int h = warp - 1;  // 0: S, dV; 1: dP, dK
    const uint32_t dk = (uint32_t)smem_desc_sw128(base_u32 + C::kKOff, 16, 1024) + (uint32_t)h * kTile;
    const uint64_t ds = smem_desc_sw128(base_u32 + C::kStageOff, 16, 1024);
    const uint64_t dm = smem_desc_sw128(base_u32 + C::kStageOff, C::kBoxBytes, 1024);  // as the MN-major operand
    const uint32_t hi_k = (uint32_t)(ds >> 32), hi_mn = (uint32_t)(dm >> 32);
    const uint32_t tS = tmem + 128u * (uint32_t)h, tA = tmem + 256u + (uint32_t)(h * D);
    const uint32_t lead = elect_lead();
    Stream s = first;
    seek(s);
    bool ok = first.i >= first.end || wait_warp(C::kRes, 0, 1);  // also where no query turns out live
    int n = 0;
    for (; ok && s.i < s.end; ++n) {
      const uint32_t parity = (uint32_t)(n / C::kStages) & 1u;
      const int qs = last_slot<C::kStages>(n), gs = first_slot<C::kStages>(n);
      const int own = h == 0 ? qs : gs, other = h == 0 ? gs : qs;  // of the scores, of the sums
      if (!(ok = wait_warp(C::kFull + own, parity, 2))) break;
      const bool part = p.q_len != nullptr && s.live < p.tile_tokens;
      const int live = s.live * p.pack;
      // queries past the sequence's end may hold anything, and 0 * NaN is NaN
      if (__builtin_expect(part, 0))
        zero_rows<C::kBoxes>(base + C::kStageOff + own * C::kTileBytes, live, kTileM);
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
        mma_ss_l(lead, tS, make_desc(dk + off, hi_k), make_desc((uint32_t)ds + own * kTile + off, hi_k), idesc_s,
                 kk > 0 ? 1u : 0u);
      }
      mma_commit_l(lead, bar(C::kSFull + h));
      mma_commit_l(lead, bar(C::kEmpty + own));
      next(s);
      if (!(ok = wait_warp(C::kFull + other, parity, 2))) break;
      if (__builtin_expect(part, 0))  // by both streams, whichever comes first
        zero_rows<C::kBoxes>(base + C::kStageOff + other * C::kTileBytes, live, kTileM);
      if (!(ok = wait_warp(C::kPFull + h, (uint32_t)n & 1u, 3))) break;
      tc_fence_after();
#pragma unroll
      for (int kk = 0; kk < 8; ++kk)
        mma_ts_l(lead, tA, tS + (uint32_t)((kk >> 2) * 64 + (kk & 3) * 8),
                 make_desc((uint32_t)dm + other * kTile + ((uint32_t)(kk * 16 * 128) >> 4), hi_mn), idesc_acc,
                 n + kk > 0 ? 1u : 0u);
      mma_commit_l(lead, bar(C::kEmpty + other));
    }
    if (ok && n > 0) mma_commit_l(lead, bar(C::kDone + h));
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain + h));
      if (lane == 0) wait_drain(bar(C::kDrain + h), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------- P^T, dS^T; the end
    const int hf = (warp - 4) >> 2, quad = warp & 3;  // 64 queries each
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)hf * 64u, tG = tS + 128u;
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    Stream s = first;
    seek(s);
    bool ok = true;
    int n = 0;
    for (; ok && s.i < s.end; ++n, next(s)) {
      const float* stat = reinterpret_cast<const float*>(base + C::kStatOff + (n % C::kStages) * 1024) + hf * 64;
      if (!(ok = wait_warp(C::kStat + n % C::kStages, (uint32_t)(n / C::kStages) & 1u, 7))) break;
      float2 pr[32];
      if (!(ok = wait_warp(C::kSFull, (uint32_t)n & 1u, 4))) break;
      tc_fence_after();
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t v[32], o[16];
        tmem_ld32(tS + 32 * cc, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 nl = *reinterpret_cast<const float2*>(stat + 32 * cc + 2 * k);
          const float2 x = __ffma2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), sc2, nl);
          const float2 e = make_float2(ex2(x.x), ex2(x.y));
          pr[16 * cc + k] = e;
          o[k] = pack_bf16(e.x, e.y);
        }
        tmem_st16(tS + 16 * cc, o);  // over the scores that this warp has read
      }
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(C::kPFull);
      if (!(ok = wait_warp(C::kSFull + 1, (uint32_t)n & 1u, 5))) break;
      tc_fence_after();
#pragma unroll
      for (int cc = 0; cc < 2; ++cc) {
        uint32_t v[32], o[16];
        tmem_ld32(tG + 32 * cc, v);
        tmem_wait_ld();
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const float2 nd = *reinterpret_cast<const float2*>(stat + 128 + 32 * cc + 2 * k);
          const float2 x = __fmul2_rn(
              pr[16 * cc + k],
              __fadd2_rn(make_float2(__uint_as_float(v[2 * k]), __uint_as_float(v[2 * k + 1])), nd));
          o[k] = pack_bf16(x.x, x.y);
        }
        tmem_st16(tG + 16 * cc, o);
      }
      tmem_wait_st();
      tc_fence_before();
      arrive_warp(C::kPFull + 1);
    }
    if (ok && n > 0) ok = wait_warp(C::kDone + hf, 0, 6);
    ok = ok && !uniform<true>(*abort_flag);
    const int key = k0 + row;
    if (ok && key - row < p.Lk) {  // half 0 has dV, half 1 dK
      tc_fence_after();
      const bool live = row < keys && n > 0 && (hf == 0 || keys + k0 > 1);  // one key's softmax has no gradient
      const float mul = hf == 0 ? 1.f : p.scale;
      const uint32_t from = tmem + lane_off + 256u + (uint32_t)hf * D;
      // one share: the gradients; several: this share's part
      uint16_t* out = hf == 0 ? p.dV + kb * p.dv_batch + key * p.dv_token + hk * p.dv_head
                              : p.dK + kb * p.dk_batch + key * p.dk_token + hk * p.dk_head;
      float* part = p.part + ((long long)blockIdx.x * 2 + hf) * (kTileN * D) + (long long)row * 4;
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t v[32];
        if (n > 0) {
          tmem_ld32(from + cc, v);
          tmem_wait_ld();
        }
#pragma unroll
        for (int k = 0; k < 32; ++k) v[k] = live ? __float_as_uint(__uint_as_float(v[k]) * mul) : 0u;
        if (p.shares == 1) {
          if (key < p.Lk)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              reinterpret_cast<uint4*>(out + cc)[i] = make_uint4(
                  pack_bf16(__uint_as_float(v[8 * i]), __uint_as_float(v[8 * i + 1])),
                  pack_bf16(__uint_as_float(v[8 * i + 2]), __uint_as_float(v[8 * i + 3])),
                  pack_bf16(__uint_as_float(v[8 * i + 4]), __uint_as_float(v[8 * i + 5])),
                  pack_bf16(__uint_as_float(v[8 * i + 6]), __uint_as_float(v[8 * i + 7])));
        } else {  // [D / 4][128 keys] of four columns: a warp's rows are 512 contiguous bytes
#pragma unroll
          for (int i = 0; i < 8; ++i)
            *reinterpret_cast<uint4*>(part + (long long)(cc / 4 + i) * (kTileN * 4)) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
        __syncwarp();
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

// The shares' parts of a key tile's dV (even blocks) or dK, added in their order.
template <int D>
__global__ void __launch_bounds__(256) cross_sum_kernel(const __grid_constant__ CrossBwdParams p) {
  griddep_launch_dependents();
  griddep_wait();
  const int key_tiles = (p.Lk + kTileN - 1) / kTileN;
  const unsigned units = (unsigned)key_tiles * (unsigned)p.Hk * (unsigned)p.Bk;
  constexpr unsigned kPieces = D / 4 * kTileN / 256;  // 256 places of four columns a block
  const unsigned blk = blockIdx.x / kPieces, piece = blockIdx.x % kPieces;
  const unsigned unit = blk >> 1;
  const int which = (int)(blk & 1u);
  unsigned u = unit;
  const int k0 = (int)(u % (unsigned)key_tiles) * kTileN;
  u /= (unsigned)key_tiles;
  const int hk = (int)(u % (unsigned)p.Hk), kb = (int)(u / (unsigned)p.Hk);
  const int at = (int)piece * 256 + (int)threadIdx.x, row = at & (kTileN - 1), c4 = at / kTileN;
  const int key = k0 + row;
  if (key >= p.Lk) return;
  float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
  if (key < length_of<false>(p.kv_len, kb, p.Lk)) {
    const float4* from =
        reinterpret_cast<const float4*>(p.part) + ((long long)unit * 2 + which) * (kTileN * D / 4) + at;
#pragma unroll 4
    for (int s = 0; s < p.shares; ++s) {
      const float4 x = __ldcg(from + (long long)s * units * 2 * (kTileN * D / 4));
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
  }
  uint16_t* out = which == 0 ? p.dV + kb * p.dv_batch + key * p.dv_token + hk * p.dv_head
                             : p.dK + kb * p.dk_batch + key * p.dk_token + hk * p.dk_head;
  *reinterpret_cast<uint2*>(out + 4 * c4) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
}

template <typename K>
cudaError_t launch(K* kernel, unsigned blocks, int threads, size_t smem, std::atomic<unsigned long long>& ready,
                   const CrossBwdParams& p, cudaStream_t s) {
  const cudaError_t e = allow_smem(kernel, smem, ready);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks, 1, 1);
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

template <int D>
cudaError_t backward(const CrossBwdParams& p, int sms, cudaStream_t s) {
  static std::atomic<unsigned long long> dq_ready[3], dkv_ready, sum_ready;
  const unsigned blocks = p.items < (unsigned)sms ? p.items : (unsigned)sms;
  const int kind = p.q_len != nullptr || p.kv_len != nullptr ? 2 : p.Lk <= kTileN ? 1 : 0;
  cudaError_t e = launch(kind == 2   ? cross_dq_kernel<D, true, true>
                         : kind == 1 ? cross_dq_kernel<D, true, false>
                                     : cross_dq_kernel<D, false, false>,
                         blocks, DqCfg<D>::kThreads, DqCfg<D>::kSmemBytes, dq_ready[kind], p, s);
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)((p.Lk + kTileN - 1) / kTileN) * (unsigned)p.Hk * (unsigned)p.Bk;
  e = launch(cross_dkv_kernel<D>, units * (unsigned)p.shares + p.forged, DkvCfg<D>::kThreads, DkvCfg<D>::kSmemBytes, dkv_ready, p,
             s);
  if (e != cudaSuccess || p.shares == 1) return e;
  return launch(cross_sum_kernel<D>, units * 2 * (D / 4 * kTileN / 256), 256, 0, sum_ready, p, s);
}

}  // namespace

cudaError_t launch_cross_backward(const CrossBwdParams& p, int sms, cudaStream_t s) {
  return p.D == 128 ? backward<128>(p, sms, s) : backward<64>(p, sms, s);
}

}  // namespace sab
