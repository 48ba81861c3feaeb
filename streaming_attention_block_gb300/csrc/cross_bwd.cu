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
// kernels (14 D products a pair for the 10 D of one), which costs less than
// sending dQ's parts, one for each key tile, through memory.
#include <math.h>

#include "cross_common.cuh"

namespace sab {
namespace {

constexpr float kLog2e = 1.4426950408889634f;

// ------------------------------------------------------------------- dQ, delta

template <int D_>
struct DqCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr uint32_t kHalfBox = kBoxBytes / 2, kHalfBytes = kTileBytes / 2;
  static constexpr int kSlots = D == 128 ? 3 : 8;  // of a stream: halves of V and K tiles in turn
  static constexpr uint32_t kQOff = 0, kGOff = kTileBytes;  // Q, dO of an item; two items
  static constexpr uint32_t kRingOff = 4 * kTileBytes;
  static constexpr uint32_t kStatOff = kRingOff + 2 * kSlots * kHalfBytes;  // [2 items][128] {-LSE log2 e, -delta}
  static constexpr uint32_t kBarOff = kStatOff + 2048;
  static constexpr int kQFull = 0;                     // [2 items]
  static constexpr int kOut = 2;                       // [2] dQ is where Q was
  static constexpr int kFull = 4;                      // [2 streams][kSlots]
  static constexpr int kEmpty = kFull + 2 * kSlots;    // [2][kSlots]
  static constexpr int kSFull = kEmpty + 2 * kSlots;   // [2 streams]
  static constexpr int kPFull = kSFull + 2;            // [2]
  static constexpr int kDone = kPFull + 2;             // [2] an item's last product
  static constexpr int kRead = kDone + 2;              // [2] dQ is taken out
  static constexpr int kStat = kRead + 2;              // [2 items] LSE and delta are there
  static constexpr int kSeen = kStat + 2;              // [2] all warps for dS have them
  static constexpr int kDrain = kSeen + 2;             // [2 streams]
  static constexpr int kNumBars = kDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16;
  // Q and dO; products of keys [0, 64) and [64, 128); K and V; 8 warps for dS; 4
  // for delta and dQ
  static constexpr int kThreads = 32 * 16;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// S and dP of a key tile (128 columns each) and dQ do not fit in TMEM twice, so
// the two halves of every key tile are the streams that take turns on the tensor
// cores: each with its scores, its dP (dS goes over the scores), its part of dQ
// and a warp that issues its products, in the order S, dP, dQ, S, dP ...
template <int D>
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
    for (int s = 0; s < 2 * C::kSlots; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kQFull + i), 1);
      mbar_init(bar(C::kOut + i), 4);
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + i), 8);
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
  pass.list = nullptr;
  pass.pair = 1;
  pass.split = 0;
  pass.by = spot_of(p, gridDim.x, 1);

  if (warp == 0) {
    // ------------------------------------------------------------ Q and dO an item ahead, dQ out
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(2 * C::kBoxes * p.pack * p.tile_tokens) * 128u;
      int at[2][3];  // where the items in the buffers are
      auto out = [&](int item) -> bool {
        const int buf = item & 1;
        if (!wait(C::kOut + buf, (uint32_t)(item >> 1) & 1u, 0)) return false;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_store_4d(&p.o_map, base_u32 + buf * 2 * C::kTileBytes + bx * C::kBoxBytes, bx * 64, at[0][0], at[0][1],
                       at[0][2]);
        tma_store_commit_and_wait_read();
        return true;
      };
      int item = 0;
      bool ok = true;
      Walk<false> c, o;
      o.start(p, pass);
      for (c.start(p, pass); c.more(pass); c.next(p, pass)) {
        const Work& w = c.w;
        if (o.more(pass)) o.next(p, pass);
        if (w.nt == 0) continue;
        const int buf = item & 1;
        if (item >= 2 && !(ok = out(item - 2))) break;
        mbar_arrive_expect_tx(bar(C::kQFull + buf), q_bytes);
        const int c1 = query_c1(p, w, 0), c2 = query_c2(p, w, 0);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx) {
          const uint32_t to = base_u32 + buf * 2 * C::kTileBytes + bx * C::kBoxBytes;
          tma_load_4d(to + C::kGOff, &p.do_map, bar(C::kQFull + buf), bx * 64, c1, c2, w.b);
          tma_load_4d(to + C::kQOff, &p.q_map, bar(C::kQFull + buf), bx * 64, c1, c2, w.b);
        }
        // O of the item after it, which the warps for delta load themselves
        if (o.more(pass) && o.w.nt > 0) {
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_prefetch_4d(&p.of_map, bx * 64, query_c1(p, o.w, 0), query_c2(p, o.w, 0), o.w.b);
        }
#pragma unroll
        for (int i = 0; i < 3; ++i) at[0][i] = at[1][i];
        at[1][0] = c1, at[1][1] = c2, at[1][2] = w.b;
        ++item;
      }
      if (item == 1) {
#pragma unroll
        for (int i = 0; i < 3; ++i) at[0][i] = at[1][i];
      }
      for (int k = max(0, item - 2); ok && k < item; ++k) {
        ok = out(k);
#pragma unroll
        for (int i = 0; i < 3; ++i) at[0][i] = at[1][i];
      }
      tma_store_wait_all();
      if (*abort_flag)  // nothing of this block's copies may land after it
        for (int k = max(0, item - 2); k < item; ++k)
          wait_drain(bar(C::kQFull + (k & 1)), (uint32_t)(k >> 1) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp == 3) {
    // ------------------------------------------------------------- V, K, each stream its half
    if (lane == 0) {
      int loads[2] = {0, 0};
      Ring<C::kSlots> r[2];
      bool ok = true;
      Walk<false> c;
      for (c.start(p, pass); ok && c.more(pass); c.next(p, pass)) {
        const Work& w = c.w;
        const int head = w.hb * p.pack / p.group, kb = p.Bk == 1 ? 0 : w.b;
        for (int j = 0; ok && j < w.nt; ++j) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (w.keys - j * kTileN <= 64 * h) break;  // the tile ends before this half
#pragma unroll 1
            for (int k = 0; ok && k < 2; ++k) {  // V before K: V's slot is free first
              const CUtensorMap* m = k == 0 ? &p.v_map : &p.k_map;
              const int at = h * C::kSlots + r[h].slot;
              if (loads[h] >= C::kSlots && !(ok = wait(C::kEmpty + at, r[h].parity ^ 1u, 1))) break;
              mbar_arrive_expect_tx(bar(C::kFull + at), C::kHalfBytes);
#pragma unroll
              for (int bx = 0; bx < C::kBoxes; ++bx)
                tma_load_4d(base_u32 + C::kRingOff + at * C::kHalfBytes + bx * C::kHalfBox, m, bar(C::kFull + at),
                            bx * 64, j * kTileN + 64 * h, head, kb);
              r[h].next();
              ++loads[h];
            }
            if (!ok) break;
          }
        }
      }
      if (*abort_flag)
        for (int h = 0; h < 2; ++h)
          for (int k = max(0, loads[h] - C::kSlots); k < loads[h]; ++k)
            wait_drain(bar(C::kFull + h * C::kSlots + k % C::kSlots), (uint32_t)(k / C::kSlots) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp < 3) {
    // ------------------------------------------------------------- products
    const int h = warp - 1;  // keys [64 h, 64 h + 64) of every tile
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, 0);
    constexpr uint32_t idesc_q = idesc_bf16_f32(128, D, 1);
    constexpr uint32_t kStep = C::kHalfBytes >> 4;
    const uint32_t ring = C::kRingOff + (uint32_t)h * C::kSlots * C::kHalfBytes;
    const uint64_t dq = smem_desc_sw128(base_u32 + C::kQOff, 16, 1024);
    const uint64_t dk = smem_desc_sw128(base_u32 + ring, 16, 1024);
    const uint64_t dm = smem_desc_sw128(base_u32 + ring, C::kHalfBox, 1024);  // as the MN-major operand
    const uint32_t hi_k = (uint32_t)(dq >> 32), hi_mn = (uint32_t)(dm >> 32);
    const uint32_t tS = tmem + (uint32_t)h * 128u, tQ = tmem + 256u + (uint32_t)h * D;
    const uint32_t full = C::kFull + h * C::kSlots, empty = C::kEmpty + h * C::kSlots;
    const uint32_t lead = elect_lead();
    Ring<C::kSlots> r;
    uint32_t p_parity = 0;
    int used = 0, item = 0;
    bool ok = true;
    auto scores = [&](uint32_t to, uint32_t a_lo, uint32_t b_lo) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t a = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4, b = ((kk >> 2) * C::kHalfBox + (kk & 3) * 32) >> 4;
        mma_ss_l(lead, to, make_desc(a_lo + a, hi_k), make_desc(b_lo + b, hi_k), idesc_s, kk > 0 ? 1u : 0u);
      }
    };
    Walk<true> c;
    c.start(p, pass);
    c.seek(p, pass);
    while (ok && c.more(pass)) {
      const int buf = item & 1, keys = c.w.keys - 64 * h, steps_n = (keys + 127) >> 7;  // tiles with keys in this half
      if (!(ok = wait_warp(C::kQFull + buf, (uint32_t)(item >> 1) & 1u, 2))) break;
      const uint32_t q0 = (uint32_t)dq + buf * (2 * C::kTileBytes >> 4);
      for (int j = 0; j < steps_n; ++j) {
        const int live = keys - j * kTileN;
        const int vs = r.slot;
        if (!(ok = wait_warp(full + vs, r.parity, 3))) break;
        r.next();
        tc_fence_after();
        scores(tS + 64u, q0 + (C::kTileBytes >> 4), (uint32_t)dk + vs * kStep);  // dP = dO V^T
        mma_commit_l(lead, bar(empty + vs));
        const int ks = r.slot;
        if (!(ok = wait_warp(full + ks, r.parity, 3))) break;
        r.next();
        scores(tS, q0, (uint32_t)dk + ks * kStep);  // S = Q K^T
        mma_commit_l(lead, bar(C::kSFull + h));
        const int steps = min(4, (live + 15) >> 4);  // 16 keys each
        // keys past the sequence's end may hold anything, and 0 * NaN is NaN
        if (__builtin_expect(steps * 16 > live, 0))
          zero_rows<C::kBoxes, C::kHalfBox>(base + ring + ks * C::kHalfBytes, live, steps * 16);
        // the item before has its dQ taken out before this one's goes over it
        if (__builtin_expect(j == 0 && used > 0, 0) && !(ok = wait_warp(C::kRead + h, (uint32_t)(used - 1) & 1u, 4)))
          break;
        if (!(ok = wait_warp(C::kPFull + h, p_parity, 5))) break;
        p_parity ^= 1u;
        tc_fence_after();
        const uint32_t m0 = (uint32_t)dm + ks * kStep;
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)  // dQ += dS K
          if (kk < steps)
            mma_ts_l(lead, tQ, tS + (uint32_t)(kk >> 1) * 32u + (uint32_t)(kk & 1) * 8u,
                     make_desc(m0 + ((uint32_t)(kk * 16 * 128) >> 4), hi_mn), idesc_q, j + kk > 0 ? 1u : 0u);
        mma_commit_l(lead, bar(empty + ks));
      }
      if (!ok) break;
      if (steps_n > 0) {
        mma_commit_l(lead, bar(C::kDone + h));
        ++used;
      }
      ++item;
      c.next(p, pass);
      c.seek(p, pass);
    }
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain + h));
      if (lane == 0) wait_drain(bar(C::kDrain + h), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp < 12) {
    // ------------------------------------------------------------------- dS
    // Eight warps to a step, 32 columns each: half the time of four from scores
    // to dS, which is what a stream waits for.
    const int cg = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t tS = tmem + ((uint32_t)(quad * 32) << 16) + (uint32_t)cg * 32u;
    const float2* stat = reinterpret_cast<const float2*>(base + C::kStatOff);
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    uint32_t parity[2] = {0u, 0u};
    int item = 0;
    bool ok = true;
    Walk<true> c;
    c.start(p, pass);
    c.seek(p, pass);
    while (ok && c.more(pass)) {
      const int nt = c.w.nt, keys = c.w.keys;
      if (!(ok = wait_warp(C::kStat + (item & 1), (uint32_t)(item >> 1) & 1u, 6))) break;
      const float2 st = stat[(item & 1) * 128 + row];
      arrive_warp(C::kSeen + (item & 1));
      const float2 nl = make_float2(st.x, st.x), nd = make_float2(st.y, st.y);
      for (int j = 0; ok && j < nt; ++j) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int live = keys - j * kTileN - h * 64;
          if (live <= 0) break;  // only an item's last tile ends before a half
          if (!(ok = wait_warp(C::kSFull + h, parity[h], 7))) break;
          parity[h] ^= 1u;
          tc_fence_after();
          uint32_t s[32], g[32], o[16];
          tmem_ld32(tS + 128 * h, s);
          tmem_ld32(tS + 128 * h + 64, g);
          tmem_wait_ld();
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * k]), __uint_as_float(s[2 * k + 1])), sc2, nl);
            const float2 pr = make_float2(ex2(x.x), ex2(x.y));
            const float2 ds =
                __fmul2_rn(pr, __fadd2_rn(make_float2(__uint_as_float(g[2 * k]), __uint_as_float(g[2 * k + 1])), nd));
            o[k] = pack_bf16(ds.x, ds.y);
          }
          const int hi = live - cg * 32;
          if (__builtin_expect(hi < 32, 0)) {  // keys past the end
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = 2 * k + 1 < hi ? o[k] : 2 * k < hi ? o[k] & 0xFFFFu : 0u;
          }
          tmem_st16(tS + 128 * h, o);  // over the first half of the scores read
          tmem_wait_st();
          tc_fence_before();
          arrive_warp(C::kPFull + h);
        }
      }
      ++item;
      c.next(p, pass);
      c.seek(p, pass);
    }
  } else {
    // ------------------------------------------------------------ delta, dQ
    // delta of the next item is formed while this one's products run; O comes
    // from global memory, for there is no room for it beside two items' Q and dO.
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t tQ = tmem + ((uint32_t)(quad * 32) << 16) + 256u;
    const int row_t = row / p.pack, row_g = row - row_t * p.pack;
    constexpr int kLanes = D / 8, kRows = 32 / kLanes;  // lanes of a row, rows of an access
    const uint32_t inv = (65535u + (uint32_t)p.pack) / (uint32_t)p.pack;  // r * inv >> 16 = r / pack below 128
    const int sub = lane / kLanes, col = lane % kLanes;  // 16-byte pieces
    int used[2] = {0, 0};
    bool ok = true;
    auto alive = [&](const Work& w) { return row_t < w.live && row_t < p.tile_tokens; };
    auto stats = [&](const Work& w, int item) {
      float2* stat = reinterpret_cast<float2*>(base + C::kStatOff) + (item & 1) * 128;
      const bool live = alive(w);
      const long long at = ((long long)w.b * p.H + w.hb * p.pack + row_g) * p.Lq + w.t0 + row_t;
      const float lse = live ? __ldg(p.LSE + at) : INFINITY;
      if (item >= 2 && !wait_warp(C::kSeen + (item & 1), (uint32_t)((item >> 1) - 1) & 1u, 10)) return false;
      const uint16_t* o_base = p.O + w.b * p.o_batch + w.t0 * p.o_token + w.hb * p.pack * D + col * 8;
      const uint8_t* g_base = base + (item & 1) * 2 * C::kTileBytes + C::kGOff + (col >> 3) * C::kBoxBytes;
#pragma unroll 1
      for (int s0 = 0; s0 < kLanes; s0 += 8) {
        uint4 a[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int r = quad * 32 + (s0 + i) * kRows + sub;
          const int rt = (int)((uint32_t)r * inv >> 16), rg = r - rt * p.pack;
          a[i] = rt < w.live && rt < p.tile_tokens ? *reinterpret_cast<const uint4*>(o_base + rt * p.o_token + rg * D)
                                                   : make_uint4(0u, 0u, 0u, 0u);
        }
        if (s0 == 0 && !wait_warp(C::kQFull + (item & 1), (uint32_t)(item >> 1) & 1u, 8)) return false;
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
      stat[row] = make_float2(live ? -lse * kLog2e : -INFINITY, live ? nd : 0.f);
      if (live) p.delta[at] = -nd;
      arrive_warp(C::kStat + (item & 1));
      return true;
    };
    Walk<true> c;
    auto seek = [&]() {
      while (c.more(pass) && c.w.nt == 0) {  // no query or no key
        if (row_t < p.tile_tokens && c.w.t0 + row_t < p.Lq) {
          uint4* out = reinterpret_cast<uint4*>(p.dQ + c.w.b * p.dq_batch + (c.w.t0 + row_t) * p.dq_token +
                                                (c.w.hb * p.pack + row_g) * D);
#pragma unroll 1
          for (int i = 0; i < D / 8; ++i) out[i] = make_uint4(0u, 0u, 0u, 0u);
        }
        c.next(p, pass);
      }
    };
    c.start(p, pass);
    seek();
    bool more = c.more(pass);
    Work w = c.w;
#pragma unroll 1
    for (int item = -1; ok && more; ++item) {
      if (item >= 0) {
        w = c.w;
        c.next(p, pass);
        seek();
      }
      const bool ahead = c.more(pass);
      if (ahead && !(ok = stats(c.w, item + 1))) break;
      if (item < 0) continue;
      more = ahead;
      const bool live = alive(w);
      uint8_t* out = base + (item & 1) * 2 * C::kTileBytes + C::kQOff + row * 128;
      // dQ: the halves' parts
      const bool two = w.keys > 64;
      if (!(ok = wait_warp(C::kDone, (uint32_t)used[0] & 1u, 9))) break;
      ++used[0];
      if (two) {
        if (!(ok = wait_warp(C::kDone + 1, (uint32_t)used[1] & 1u, 9))) break;
        ++used[1];
      }
      tc_fence_after();
#pragma unroll 1
      for (int cc = 0; cc < D; cc += 32) {
        uint32_t a[32], b[32];
        tmem_ld32(tQ + cc, a);
        if (two) tmem_ld32(tQ + D + cc, b);
        tmem_wait_ld();
        if (cc + 32 == D) {
          tc_fence_before();
          arrive_warp(C::kRead);
          if (two) arrive_warp(C::kRead + 1);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int e = 8 * i + 2 * k;
            float2 x = make_float2(__uint_as_float(a[e]), __uint_as_float(a[e + 1]));
            if (two) x = __fadd2_rn(x, make_float2(__uint_as_float(b[e]), __uint_as_float(b[e + 1])));
            x = __fmul2_rn(x, make_float2(p.scale, p.scale));
            o[k] = live ? pack_bf16(x.x, x.y) : 0u;
          }
          const int k = cc / 8 + i;
          *reinterpret_cast<uint4*>(out + (k >> 3) * C::kBoxBytes + (((k & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[0], o[1], o[2], o[3]);
        }
      }
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
  // a stage: Q, dO, then 128 of -LSE log2 e and 128 of -delta
  static constexpr uint32_t kStageBytes = 2 * kTileBytes + 1024;
  static constexpr uint32_t kBarOff = kStageOff + kStages * kStageBytes;
  static constexpr int kRes = 0;
  static constexpr int kFull = 1;                       // [kStages][2 halves]
  static constexpr int kEmpty = kFull + 2 * kStages;    // [kStages][2]
  static constexpr int kSFull = kEmpty + 2 * kStages;   // [2 halves]
  static constexpr int kPFull = kSFull + 2;             // [2]
  static constexpr int kTaken = kPFull + 2;             // [2] P and dS are read
  static constexpr int kDone = kTaken + 2;
  static constexpr int kDrain = kDone + 1;              // [2]
  static constexpr int kNumBars = kDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16;
  // loads; scores; accumulations; a spare; 8 warps for P and dS, and the end
  static constexpr int kThreads = 32 * 12;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// The query tiles of a block, in two halves of h_tokens tokens x h_pack heads
// (at most 64 rows): of the block's share of the sequences, head blocks and
// tiles that read its keys.
struct Stream {
  int i, end;      // tiles
  int iq, hb, b;   // this one's place: tile, head block of the group, sequence
  int live;        // its tokens inside q_len
};

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
    for (int i = 0; i < 2 * C::kStages; ++i) {
      mbar_init(bar(C::kFull + i), 2);  // copies, LSE and delta
      mbar_init(bar(C::kEmpty + i), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + i), 8);
      mbar_init(bar(C::kTaken + i), 1);
      mbar_init(bar(C::kDrain + i), 1);
    }
    mbar_init(bar(C::kDone), 1);
    misc[1] = (base_u32 & 1023u) != 0;
    if (misc[1] != 0 && p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
    fence_mbar_init();
  }
  // rows of a half that no copy fills (3 heads x 21 tokens leave one) are zeros
  if (p.h_pack * p.h_tokens < 64) {
    const int first = p.h_pack * p.h_tokens, n = (64 - first) * 8;
    for (int i = threadIdx.x; i < C::kStages * 2 * C::kBoxes * 2 * n; i += blockDim.x) {
      const int blk = i / n, k = i - blk * n;  // box, half
      const int st = blk / (4 * C::kBoxes), rest = blk - st * 4 * C::kBoxes;
      uint8_t* to = base + C::kStageOff + st * C::kStageBytes + (rest >> 1) * C::kBoxBytes + (rest & 1) * (C::kBoxBytes / 2);
      *reinterpret_cast<uint4*>(to + (first + (k >> 3)) * 128 + (k & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
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

  const int blocks = p.group / p.h_pack, seqs = p.Bk == 1 ? p.B : 1;
  const long long all = (long long)seqs * blocks * p.h_qtiles;
  Stream first;
  first.i = (int)(all * share / p.shares);
  first.end = dead ? first.i : (int)(all * (share + 1) / p.shares);
  {
    const int r = first.i / p.h_qtiles;
    first.iq = first.i - r * p.h_qtiles;
    first.b = (p.Bk == 1 ? 0 : kb) + r / blocks;
    first.hb = r % blocks;
  }
  // the next tile with a live query, from this one on
  auto seek = [&](Stream& s) {
    for (; s.i < s.end; ++s.i) {
      s.live = min(2 * p.h_tokens, length_of<true>(p.q_len, s.b, p.Lq) - s.iq * 2 * p.h_tokens);
      if (s.live > 0) return;
      if (++s.iq == p.h_qtiles) {
        s.iq = 0;
        if (++s.hb == blocks) s.hb = 0, ++s.b;
      }
    }
  };
  auto next = [&](Stream& s) {
    ++s.i;
    if (++s.iq == p.h_qtiles) {
      s.iq = 0;
      if (++s.hb == blocks) s.hb = 0, ++s.b;
    }
    seek(s);
  };
  // rows of half h that hold live queries
  auto rows_of = [&](const Stream& s, int h) { return min(max(s.live - h * p.h_tokens, 0), p.h_tokens) * p.h_pack; };

  if (warp == 0) {
    // ---------------------------------------------------------------- loads
    const bool any = first.i < first.end;
    if (lane == 0 && any) {
      mbar_arrive_expect_tx(bar(C::kRes), 2 * C::kTileBytes);
#pragma unroll
      for (int bx = 0; bx < C::kBoxes; ++bx) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint32_t to = base_u32 + bx * C::kBoxBytes + h * (C::kBoxBytes / 2);
          tma_load_4d(to + C::kKOff, &p.k_map, bar(C::kRes), bx * 64, k0 + 64 * h, hk, kb);
          tma_load_4d(to + C::kVOff, &p.v_map, bar(C::kRes), bx * 64, k0 + 64 * h, hk, kb);
        }
      }
    }
    const uint32_t half_bytes = (uint32_t)(2 * C::kBoxes * p.h_pack * p.h_tokens) * 128u;
    // two rows of each half a lane: place within the tile's heads and tokens
    int tok[2], hd[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = lane + 32 * i;
      tok[i] = r / p.h_pack;
      hd[i] = r - tok[i] * p.h_pack;
    }
    Stream s = first;
    seek(s);
    float ls[4], dl[4];
    bool has[4];  // of the tile to be loaded next, requested one tile ahead
    auto fetch = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int h = i >> 1, r = lane + 32 * (i & 1);
        const bool in = r < rows_of(s, h);
        const int t = s.iq * 2 * p.h_tokens + h * p.h_tokens + tok[i & 1];
        const int head = hk * p.group + s.hb * p.h_pack + hd[i & 1];
        const long long at = ((long long)s.b * p.H + head) * p.Lq + t;
        ls[i] = dl[i] = 0.f;
        if (in) ls[i] = __ldg(p.LSE + at), dl[i] = __ldg(p.delta + at);
        has[i] = in;
      }
    };
    if (s.i < s.end) fetch();
    int n = 0, halves = 0;
    bool ok = true;
    while (ok && s.i < s.end) {
      const int st = n % C::kStages;
      const uint32_t so = C::kStageOff + st * C::kStageBytes;
      const int head = hk * p.group + s.hb * p.h_pack, t0 = s.iq * 2 * p.h_tokens;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (n >= C::kStages &&
            !(ok = wait_warp(C::kEmpty + 2 * st + h, (uint32_t)(n / C::kStages - 1) & 1u, 0)))
          break;
        const uint32_t full = bar(C::kFull + 2 * st + h);
        if (lane == 0) {
          const int t = t0 + h * p.h_tokens;
          const int c1 = p.h_pack == 1 ? t : head, c2 = p.h_pack == 1 ? head : t;
          mbar_arrive_expect_tx(full, half_bytes);
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx) {
            const uint32_t to = base_u32 + so + bx * C::kBoxBytes + h * (C::kBoxBytes / 2);
            tma_load_4d(to, &p.q_map_h, full, bx * 64, c1, c2, s.b);
            tma_load_4d(to + C::kTileBytes, &p.do_map_h, full, bx * 64, c1, c2, s.b);
          }
        }
        float* stat = reinterpret_cast<float*>(base + so + 2 * C::kTileBytes) + 64 * h;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          stat[lane + 32 * i] = has[2 * h + i] ? -ls[2 * h + i] * kLog2e : -INFINITY;
          stat[128 + lane + 32 * i] = -dl[2 * h + i];
        }
        arrive_warp(C::kFull + 2 * st + h);
        ++halves;
      }
      if (!ok) break;
      ++n;
      next(s);
      if (s.i < s.end) fetch();
    }
    if (lane == 0 && *abort_flag) {
      if (any) wait_drain(bar(C::kRes), 0, p.err_word);
      for (int k = max(0, halves - 2 * C::kStages); k < halves; ++k)
        wait_drain(bar(C::kFull + 2 * ((k >> 1) % C::kStages) + (k & 1)), (uint32_t)((k >> 1) / C::kStages) & 1u,
                   p.err_word);
    }
    __syncwarp();
  } else if (warp == 1) {
    // --------------------------------------- S^T = K Q^T, dP^T = V dO^T
    constexpr uint32_t idesc_s = idesc_bf16_f32(128, 64, 0);
    constexpr uint32_t kStep = C::kStageBytes >> 4;
    constexpr uint32_t kHalf = (64u * 128u) >> 4;
    const uint64_t dk = smem_desc_sw128(base_u32 + C::kKOff, 16, 1024);
    const uint64_t dv = smem_desc_sw128(base_u32 + C::kVOff, 16, 1024);
    const uint64_t ds = smem_desc_sw128(base_u32 + C::kStageOff, 16, 1024);
    const uint32_t hi_k = (uint32_t)(dk >> 32);
    const uint32_t lead = elect_lead();
    auto scores = [&](uint32_t to, uint32_t a_lo, uint32_t b_lo) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
        mma_ss_l(lead, to, make_desc(a_lo + off, hi_k), make_desc(b_lo + off, hi_k), idesc_s, kk > 0 ? 1u : 0u);
      }
    };
    Stream s = first;
    seek(s);
    bool ok = first.i >= first.end || wait_warp(C::kRes, 0, 1);  // also where no query turns out live
    for (int n = 0; ok && s.i < s.end; ++n, next(s)) {
      const int st = n % C::kStages;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(ok = wait_warp(C::kFull + 2 * st + h, (uint32_t)(n / C::kStages) & 1u, 2))) break;
        const int rows = rows_of(s, h);
        if (__builtin_expect(p.q_len != nullptr && rows < p.h_pack * p.h_tokens, 0)) {
          // queries past the sequence's end may hold anything, and 0 * NaN is NaN
          uint8_t* q = base + C::kStageOff + st * C::kStageBytes + h * (C::kBoxBytes / 2);
          zero_rows<C::kBoxes>(q, rows, 64);
          zero_rows<C::kBoxes>(q + C::kTileBytes, rows, 64);
        }
        if (n > 0 && !(ok = wait_warp(C::kTaken + h, (uint32_t)(n - 1) & 1u, 3))) break;
        tc_fence_after();
        const uint32_t q0 = (uint32_t)ds + st * kStep + h * kHalf;
        scores(tmem + 128u * h, (uint32_t)dk, q0);
        scores(tmem + 128u * h + 64u, (uint32_t)dv, q0 + (C::kTileBytes >> 4));
        mma_commit_l(lead, bar(C::kSFull + h));
      }
    }
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 2) {
    // --------------------------------------- dV += P^T dO, dK += dS^T Q
    constexpr uint32_t idesc_acc = idesc_bf16_f32(128, D, 1);
    constexpr uint32_t kStep = C::kStageBytes >> 4;
    const uint64_t dm = smem_desc_sw128(base_u32 + C::kStageOff, C::kBoxBytes, 1024);
    const uint32_t hi_mn = (uint32_t)(dm >> 32);
    const uint32_t lead = elect_lead();
    Stream s = first;
    seek(s);
    bool ok = true, any = false;
    for (int n = 0; ok && s.i < s.end; ++n, next(s)) {
      const int st = n % C::kStages;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(ok = wait_warp(C::kPFull + h, (uint32_t)n & 1u, 4))) break;
        tc_fence_after();
        const uint32_t q0 = (uint32_t)dm + st * kStep + ((uint32_t)(h * 64 * 128) >> 4);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_l(lead, tmem + 256, tmem + 128u * h + (kk >> 1) * 32 + (kk & 1) * 8,
                   make_desc(q0 + ((C::kTileBytes + kk * 16 * 128) >> 4), hi_mn), idesc_acc,
                   n + h + kk > 0 ? 1u : 0u);
#pragma unroll
        for (int kk = 0; kk < 4; ++kk)
          mma_ts_l(lead, tmem + 256 + D, tmem + 128u * h + 64u + (kk >> 1) * 32 + (kk & 1) * 8,
                   make_desc(q0 + ((uint32_t)(kk * 16 * 128) >> 4), hi_mn), idesc_acc, n + h + kk > 0 ? 1u : 0u);
        mma_commit_l(lead, bar(C::kTaken + h));
        mma_commit_l(lead, bar(C::kEmpty + 2 * st + h));
        any = true;
      }
    }
    if (ok && any) mma_commit_l(lead, bar(C::kDone));
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain + 1));
      if (lane == 0) wait_drain(bar(C::kDrain + 1), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp >= 4) {
    // ---------------------------------------------------- P^T, dS^T; the end
    const int hf = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tS = tmem + lane_off + (uint32_t)hf * 32u;  // eight warps to a half's step, 32 queries each
    const float2 sc2 = make_float2(p.scale_log2, p.scale_log2);
    Stream s = first;
    seek(s);
    bool ok = true;
    int n = 0;
    for (; ok && s.i < s.end; ++n, next(s)) {
      const float* stat = reinterpret_cast<const float*>(base + C::kStageOff + (n % C::kStages) * C::kStageBytes +
                                                         2 * C::kTileBytes) + hf * 32;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!(ok = wait_warp(C::kSFull + h, (uint32_t)n & 1u, 5))) break;
        tc_fence_after();
        uint32_t sv[32], gv[32], po[16], so[16];
        tmem_ld32(tS + 128 * h, sv);
        tmem_ld32(tS + 128 * h + 64, gv);
        tmem_wait_ld();
#pragma unroll
        for (int c4 = 0; c4 < 8; ++c4) {
          const float4 nl = *reinterpret_cast<const float4*>(stat + 64 * h + 4 * c4);
          const float4 nd = *reinterpret_cast<const float4*>(stat + 128 + 64 * h + 4 * c4);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            const int k = 2 * c4 + e;
            const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[2 * k]), __uint_as_float(sv[2 * k + 1])), sc2,
                                        e ? make_float2(nl.z, nl.w) : make_float2(nl.x, nl.y));
            const float2 pr = make_float2(ex2(x.x), ex2(x.y));
            const float2 g = __fadd2_rn(make_float2(__uint_as_float(gv[2 * k]), __uint_as_float(gv[2 * k + 1])),
                                        e ? make_float2(nd.z, nd.w) : make_float2(nd.x, nd.y));
            const float2 d = __fmul2_rn(pr, g);
            po[k] = pack_bf16(pr.x, pr.y);
            so[k] = pack_bf16(d.x, d.y);
          }
        }
        tmem_st16(tS + 128 * h, po);  // over the first half of what this warp has read
        tmem_st16(tS + 128 * h + 64, so);
        tmem_wait_st();
        tc_fence_before();
        arrive_warp(C::kPFull + h);
      }
      if (!ok) break;
    }
    if (ok && n > 0) ok = wait_warp(C::kDone, 0, 6);
    ok = ok && !uniform<true>(*abort_flag);
    const int key = k0 + row;
    if (ok && key - row < p.Lk) {  // half 0 has dV, half 1 dK
      tc_fence_after();
      const bool live = row < keys && n > 0;
      const float mul = hf == 0 ? 1.f : p.scale;
      const uint32_t from = tmem + lane_off + 256u + (uint32_t)hf * D;
      // one share: the gradients; several: this share's part
      uint16_t* out = hf == 0 ? p.dV + kb * p.dv_batch + key * p.dv_token + hk * D
                              : p.dK + kb * p.dk_batch + key * p.dk_token + hk * D;
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
    const float4* from = reinterpret_cast<const float4*>(p.part) + ((long long)unit * 2 + which) * (kTileN * D / 4) + at;
#pragma unroll 4
    for (int s = 0; s < p.shares; ++s) {
      const float4 x = __ldcg(from + (long long)s * units * 2 * (kTileN * D / 4));
      a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
    }
  }
  uint16_t* out = which == 0 ? p.dV + kb * p.dv_batch + key * p.dv_token + hk * D
                             : p.dK + kb * p.dk_batch + key * p.dk_token + hk * D;
  *reinterpret_cast<uint2*>(out + 4 * c4) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
}

template <typename K>
cudaError_t launch(K kernel, unsigned blocks, int threads, size_t smem, const CrossBwdParams& p, cudaStream_t s) {
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
  static bool set = false;
  if (!set) {
    cudaError_t e = cudaFuncSetAttribute(cross_dq_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)DqCfg<D>::kSmemBytes);
    if (e == cudaSuccess)
      e = cudaFuncSetAttribute(cross_dkv_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                               (int)DkvCfg<D>::kSmemBytes);
    if (e != cudaSuccess) return e;
    set = true;
  }
  cudaError_t e = launch(cross_dq_kernel<D>, p.items < (unsigned)sms ? p.items : (unsigned)sms, DqCfg<D>::kThreads,
                         DqCfg<D>::kSmemBytes, p, s);
  if (e != cudaSuccess) return e;
  const unsigned units = (unsigned)((p.Lk + kTileN - 1) / kTileN) * (unsigned)p.Hk * (unsigned)p.Bk;
  e = launch(cross_dkv_kernel<D>, units * (unsigned)p.shares, DkvCfg<D>::kThreads, DkvCfg<D>::kSmemBytes, p, s);
  if (e != cudaSuccess || p.shares == 1) return e;
  return launch(cross_sum_kernel<D>, units * 2 * (D / 4 * kTileN / 256), 256, 0, p, s);
}

}  // namespace

cudaError_t launch_cross_backward(const CrossBwdParams& p, int sms, cudaStream_t s) {
  return p.D == 128 ? backward<128>(p, sms, s) : backward<64>(p, sms, s);
}

}  // namespace sab
