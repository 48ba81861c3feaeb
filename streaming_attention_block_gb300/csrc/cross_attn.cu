// Cross attention: one sequence's queries over another's keys and values (an
// encoder's states), forward and backward, for sm_103a.
//
// For query row i of head h and the first kv_len[b] keys of head h / (H / Hk):
//   s_ij = scale * q_i.k_j,  O_i = sum_j softmax_j(s_ij) v_j,
//   LSE_i = ln sum_j exp(s_ij).
// Rows are queries of several heads where heads share keys: a tile of 128 rows
// holds `pack` heads of 128 / pack tokens, so that a few tokens fill it and
// keys are read once for all of them.
//
// What is particular to it: an encoder's states are short (a prompt), the
// queries many, so a tile of queries meets only a handful of key tiles.  The
// work on a tile of queries is then mostly its beginning and end, and the
// kernels below run one block per SM over a list of such tiles with the
// pipeline never drained between them: keys, queries and products of the next
// tile are under way while the softmax of this one ends.
//
// Every mbarrier wait is bounded: on expiry the kernel records the wait site
// in the library's error word, raises a block-wide abort flag, drains its own
// copies and products, frees TMEM and returns.
#include <math.h>

#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

using namespace ptx;

constexpr uint64_t kTimeoutNs = 2000000000ull;
constexpr float kLn2 = 0.6931471805599453f;
constexpr float kLog2e = 1.4426950408889634f;
// P = 2^(s - m) in bf16 has fp32's exponents and is summed in fp32, so the
// reference m need not be the row's maximum: any m within 2^40 of it gives the
// same digits.  Rows start with m = 0 and move it only when a score leaves this
// range, which scores of normalised or random queries never do: no tile then
// waits for its maximum, and O is never rescaled.
constexpr float kRange = 40.0f;

__device__ __forceinline__ uint64_t global_ns() {
  uint64_t t;
  asm volatile("mov.u64 %0, %%globaltimer;" : "=l"(t));
  return t;
}
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

// A place in a ring of N slots: the slot and the parity of its current round.
template <int N>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void next() {
    if (++slot == N) slot = 0, parity ^= 1u;
  }
};

// ------------------------------------------------------------------ forward

// One tile of queries: `pack` heads from head hb * pack on, tile_tokens tokens
// from t0 on, and the key tiles [first, first + nt) of its sequence.
struct Work {
  int b, hb, t0;
  int live;         // tokens of the tile inside q_len
  int first, nt;
  int keys;         // keys of the range
};
__device__ __forceinline__ int length_of(const int* lens, int b, int most) {
  return lens == nullptr ? most : min(max(__ldg(lens + b), 0), most);
}
__device__ __forceinline__ Work work_at(const CrossParams& p, unsigned item, int split) {
  Work w;
  const unsigned r = item / (unsigned)p.n_qtiles;
  w.t0 = (int)(item - r * (unsigned)p.n_qtiles) * p.tile_tokens;
  w.b = (int)(r / (unsigned)p.head_blocks);
  w.hb = (int)(r - (unsigned)w.b * (unsigned)p.head_blocks);
  w.live = min(p.tile_tokens, length_of(p.q_len, w.b, p.Lq) - w.t0);
  const int kl = w.live > 0 ? length_of(p.kv_len, p.Bk == 1 ? 0 : w.b, p.Lk) : 0;
  const int total = (kl + kTileN - 1) / kTileN;
  w.first = (int)((long long)total * split / p.splits);
  const int last = (int)((long long)total * (split + 1) / p.splits);
  w.nt = last - w.first;
  w.keys = min(kl, last * kTileN) - w.first * kTileN;
  if constexpr (kDebugBounds) {
    if (w.b >= p.B || w.hb >= p.head_blocks || w.t0 >= p.Lq || w.first < 0 || last * kTileN - kTileN >= p.Lk) {
      if (p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
      w.nt = w.live = 0;
    }
  }
  return w;
}
// The blocks' tiles in order, tile by tile of keys.
struct Cursor {
  unsigned item;
  Work w;
  int j;
  bool more;
  // first item of this block that has keys
  __device__ __forceinline__ void start(const CrossParams& p, unsigned first, unsigned step, int split) {
    item = first;
    seek(p, step, split);
  }
  __device__ __forceinline__ void seek(const CrossParams& p, unsigned step, int split) {
    j = 0;
    for (; item < p.items; item += step) {
      w = work_at(p, item, split);
      if (w.nt > 0) {
        more = true;
        return;
      }
    }
    more = false;
  }
  __device__ __forceinline__ void next(const CrossParams& p, unsigned step, int split) {
    if (++j < w.nt) return;
    item += step;
    seek(p, step, split);
  }
};

template <int D_>
struct FwdCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kSlots = D == 128 ? 5 : 10;          // K and V tiles in the order of their use
  static constexpr uint32_t kQOff = 0;                      // two tiles: Q, then its O on the way out
  static constexpr uint32_t kRingOff = 2 * kTileBytes;
  static constexpr uint32_t kBarOff = kRingOff + kSlots * kTileBytes;
  static constexpr int kQFull = 0;                          // [2]
  static constexpr int kQFree = 2;                          // [2] O has left the tile
  static constexpr int kFull = 4;                           // [kSlots]
  static constexpr int kEmpty = kFull + kSlots;             // [kSlots]
  static constexpr int kSFull = kEmpty + kSlots;            // [2 buffers]
  static constexpr int kPFull = kSFull + 2;                 // [2 buffers][2 halves]
  static constexpr int kPVDone = kPFull + 4;
  static constexpr int kODone = kPVDone + 1;                // a query tile's last product
  static constexpr int kOReady = kODone + 1;                // O staged for its store
  static constexpr int kDrain = kOReady + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kSmemBytes = kMiscOff + 16 + 1024;
  // producer, products, 8 softmax warps, the store of O
  static constexpr int kThreads = 32 * 11;
  static constexpr uint32_t kTmemO = 256;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// One block per SM walks its query tiles (SPLIT: one tile, its keys cut among
// the blocks of a cluster, see the end).  Scores of a key tile are in one of
// two TMEM buffers; the keys [0, 64) and [64, 128) of every tile are two halves
// with four softmax warps, a reference m, a sum l and an accumulator O each, so
// that they meet only when a query tile is done.  The products are issued in
// the order PV(g), S(g + 2) over all tiles of the block, also from one query
// tile to the next.
template <int D, bool SPLIT>
__global__ void __launch_bounds__(FwdCfg<D>::kThreads, 1) cross_fwd_kernel(const __grid_constant__ CrossParams p) {
  using C = FwdCfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_u32 = smem_u32(smem_raw);
  const uint32_t base_u32 = (raw_u32 + 1023u) & ~1023u;
  uint8_t* base = smem_raw + (base_u32 - raw_u32);
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);  // [0] tmem, [1] abort
  volatile int* abort_flag = reinterpret_cast<volatile int*>(misc + 1);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  auto wait = [&](int i, uint32_t parity, unsigned site) -> bool {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };
  auto wait_warp = [&](int i, uint32_t parity, unsigned site) -> bool {
    return __all_sync(0xffffffffu, wait(i, parity, site));
  };
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int split = SPLIT ? (int)(blockIdx.x % (unsigned)p.splits) : 0;
  const unsigned first_item = SPLIT ? blockIdx.x / (unsigned)p.splits : blockIdx.x;
  const unsigned step = SPLIT ? p.items : gridDim.x;  // SPLIT: one item a block

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kQFull + i), 1);
      mbar_init(bar(C::kQFree + i), 1);
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + 2 * i), 128);
      mbar_init(bar(C::kPFull + 2 * i + 1), 128);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    mbar_init(bar(C::kPVDone), 1);
    mbar_init(bar(C::kODone), 1);
    mbar_init(bar(C::kOReady), 256);
    mbar_init(bar(C::kDrain), 1);
    misc[1] = 0;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(misc), 512);
    tmem_relinquish();
  }
  if (warp == 0 && lane == 0) {
    prefetch_tmap(&p.q_map);
    prefetch_tmap(&p.k_map);
    prefetch_tmap(&p.v_map);
    prefetch_tmap(&p.o_map);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = misc[0];
  griddep_launch_dependents();
  griddep_wait();

  if (warp == 0) {
    // ------------------------------------------------------------- producer
    if (lane == 0) {
      const uint32_t q_bytes = (uint32_t)(C::kBoxes * p.pack * p.tile_tokens) * 128u;
      Ring<C::kSlots> r;
      int loads = 0, tiles = 0;  // K and V tiles, query tiles requested
      bool ok = true;
      // one K or V tile into the next slot
      auto load = [&](const CUtensorMap* m, int row, int head, int b) -> bool {
        if (loads >= C::kSlots && !wait(C::kEmpty + r.slot, r.parity ^ 1u, 0)) return false;
        const uint32_t full = bar(C::kFull + r.slot);
        mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_load_4d(base_u32 + C::kRingOff + r.slot * C::kTileBytes + bx * C::kBoxBytes, m, full, bx * 64, row, head,
                      b);
        r.next();
        ++loads;
        return true;
      };
      Cursor c;
      c.start(p, first_item, step, split);
      int v_row = -1, v_head = 0, v_b = 0;  // the V tile that is still to be requested
      while (c.more) {
        const int head = c.w.hb * p.pack / p.group, kb = p.Bk == 1 ? 0 : c.w.b;
        const int row = (c.w.first + c.j) * kTileN;
        if (c.j == 0) {
          const int qb = tiles & 1;
          if (tiles >= 2 && !(ok = wait(C::kQFree + qb, (uint32_t)(tiles / 2 - 1) & 1u, 1))) break;
          mbar_arrive_expect_tx(bar(C::kQFull + qb), q_bytes);
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_4d(base_u32 + C::kQOff + qb * C::kTileBytes + bx * C::kBoxBytes, &p.q_map, bar(C::kQFull + qb),
                        bx * 64, c.w.hb * p.pack, c.w.t0, c.w.b);
          ++tiles;
        }
        if (!(ok = load(&p.k_map, row, head, kb))) break;
        if (v_row >= 0 && !(ok = load(&p.v_map, v_row, v_head, v_b))) break;
        v_row = row, v_head = head, v_b = kb;
        c.next(p, step, split);
      }
      if (ok && v_row >= 0) load(&p.v_map, v_row, v_head, v_b);
      if (*abort_flag) {  // nothing of this block's copies may land after it
        for (int k = max(0, tiles - 2); k < tiles; ++k)
          wait_drain(bar(C::kQFull + (k & 1)), (uint32_t)(k / 2) & 1u, p.err_word);
        for (int k = max(0, loads - C::kSlots); k < loads; ++k)
          wait_drain(bar(C::kFull + k % C::kSlots), (uint32_t)(k / C::kSlots) & 1u, p.err_word);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTileN, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
    const uint64_t dq = smem_desc_sw128(base_u32 + C::kQOff, 16, 1024);
    const uint64_t dk = smem_desc_sw128(base_u32 + C::kRingOff, 16, 1024);
    const uint64_t dv = smem_desc_sw128(base_u32 + C::kRingOff, C::kBoxBytes, 1024);
    const uint32_t kq_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
    constexpr uint32_t kStep = C::kTileBytes >> 4;
    const uint32_t lead = elect_lead();
    Ring<C::kSlots> r;
    bool ok = true;
    Cursor cs, cv;  // the tile whose scores, and whose values, come next
    cs.start(p, first_item, step, split);
    cv = cs;
    int gs = 0, gv = 0, tiles = 0;
    auto issue_s = [&]() -> bool {  // S(gs) = Q K^T
      if (cs.j == 0) {
        if (!wait_warp(C::kQFull + (tiles & 1), (uint32_t)(tiles >> 1) & 1u, 2)) return false;
        ++tiles;
      }
      if (!wait_warp(C::kFull + r.slot, r.parity, 3)) return false;
      tc_fence_after();
      const uint32_t a0 = (uint32_t)dq + (uint32_t)((tiles - 1) & 1) * kStep, b0 = (uint32_t)dk + r.slot * kStep;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
        mma_ss_l(lead, tmem + (uint32_t)(gs & 1) * 128u, make_desc(a0 + off, kq_hi), make_desc(b0 + off, kq_hi),
                 idesc_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit_l(lead, bar(C::kSFull + (gs & 1)));
      mma_commit_l(lead, bar(C::kEmpty + r.slot));
      r.next();
      ++gs;
      cs.next(p, step, split);
      return true;
    };
    auto issue_pv = [&]() -> bool {  // O_half += P_half V_half
      if (!wait_warp(C::kFull + r.slot, r.parity, 3)) return false;
      const int valid = min(kTileN, cv.w.keys - cv.j * kTileN);
      const int steps = (valid + 15) >> 4;  // 16 keys each
      if (valid & 15) {
        // keys past the sequence's end may hold anything, and 0 * NaN is NaN:
        // the values of the last step's are zeroed (later steps are left out)
        uint8_t* v = base + C::kRingOff + r.slot * C::kTileBytes;
        const int n = (16 * steps - valid) * 8;  // 16-byte pieces a box
        for (int i = lane; i < n * C::kBoxes; i += 32) {
          const int bx = i >= n ? 1 : 0, k = i - bx * n;
          *reinterpret_cast<uint4*>(v + bx * C::kBoxBytes + (valid + (k >> 3)) * 128 + (k & 7) * 16) =
              make_uint4(0u, 0u, 0u, 0u);
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      const uint32_t b0 = (uint32_t)dv + r.slot * kStep;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {
        if (!wait_warp(C::kPFull + 2 * (gv & 1) + hf, (uint32_t)(gv >> 1) & 1u, 4 + hf)) return false;
        tc_fence_after();
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          if (hf * 4 + kk < steps)
            mma_ts_l(lead, tmem + C::kTmemO + hf * D, tmem + (uint32_t)(gv & 1) * 128u + hf * 64u + kk * 8,
                     make_desc(b0 + (((hf * 4 + kk) * 16 * 128) >> 4), v_hi), idesc_pv,
                     kk > 0 || cv.j > 0 ? 1u : 0u);
        }
      }
      mma_commit_l(lead, bar(C::kPVDone));
      if (cv.j + 1 == cv.w.nt) mma_commit_l(lead, bar(C::kODone));
      mma_commit_l(lead, bar(C::kEmpty + r.slot));
      r.next();
      ++gv;
      cv.next(p, step, split);
      return true;
    };
    if (cs.more) ok = issue_s();
    if (ok && cs.more) ok = issue_s();
    while (ok && cv.more) {
      ok = issue_pv();
      if (ok && cs.more) ok = issue_s();
    }
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp < 10) {
    // ---------------------------------------------------- softmax, epilogue
    const int hf = (warp - 2) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tSh = tmem + lane_off + (uint32_t)hf * 64u;  // + buffer * 128
    const uint32_t tO = tmem + lane_off + C::kTmemO + (uint32_t)hf * D;
    const int row_t = row / p.pack, row_g = row - row_t * p.pack;
    const int warp_t = (quad * 32) / p.pack;  // first token of the warp's rows
    const float sl = p.scale_log2;
    int g = 0, tiles = 0;
    bool ok = true;
    for (unsigned item = first_item; ok && item < p.items; item += step) {
      const Work w = work_at(p, item, split);
      const int t = w.t0 + row_t;
      const bool stored = row_t < p.tile_tokens && t < p.Lq;  // this row has an O and an LSE
      const bool live = row_t < w.live;
      const long long lse_at = ((long long)w.b * p.H + w.hb * p.pack + row_g) * p.Lq + t;
      if (!SPLIT && w.nt == 0) {  // no query or no key: zeros, and -inf
        if (stored) {
          uint16_t* o = p.O + w.b * p.o_batch + t * p.o_token + (w.hb * p.pack + row_g) * D + hf * (D / 2);
#pragma unroll
          for (int i = 0; i < D / 16; ++i) reinterpret_cast<uint4*>(o)[i] = make_uint4(0u, 0u, 0u, 0u);
          if (hf == 0 && p.LSE != nullptr) p.LSE[lse_at] = -INFINITY;
        }
        continue;
      }
      const bool busy = warp_t < w.live;  // some row of the warp is live
      float m_run = 0.f, l_run = 0.f;
      for (int j = 0; j < w.nt; ++j, ++g) {
        if (!(ok = wait_warp(C::kSFull + (g & 1), (uint32_t)(g >> 1) & 1u, 6 + hf))) break;
        const int hi = w.keys - j * kTileN - hf * 64;  // visible columns of this half
        if (busy && hi > 0) {
          tc_fence_after();
          const uint32_t tS = tSh + (uint32_t)(g & 1) * 128u;
          uint32_t s0[32], s1[32], pk[32];
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          auto mask = [&](uint32_t (&sv)[32], int cb) {
            if (hi < 64) {
#pragma unroll
              for (int c = 0; c < 32; ++c) sv[c] = cb + c < hi ? sv[c] : 0xff800000u;
            }
          };
          auto max32 = [&](const uint32_t (&sv)[32]) -> float {
            float pm[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float m = fmax3(__uint_as_float(sv[k]), __uint_as_float(sv[k + 4]), __uint_as_float(sv[k + 8]));
              m = fmax3(m, __uint_as_float(sv[k + 12]), __uint_as_float(sv[k + 16]));
              m = fmax3(m, __uint_as_float(sv[k + 20]), __uint_as_float(sv[k + 24]));
              pm[k] = fmaxf(m, __uint_as_float(sv[k + 28]));
            }
            return fmax3(fmaxf(pm[0], pm[1]), pm[2], pm[3]);
          };
          const float2 sl2 = make_float2(sl, sl);
          auto exps32 = [&](const uint32_t (&sv)[32], float m, uint32_t* pko, float2& ps) {
            const float2 m2 = make_float2(-m, -m);
#pragma unroll
            for (int c = 0; c < 16; ++c) {
              const float2 x =
                  __ffma2_rn(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sl2, m2);
              const float e0 = ex2(x.x), e1 = ex2(x.y);
              ps = __fadd2_rn(ps, make_float2(e0, e1));
              pko[c] = pack_bf16(e0, e1);
            }
          };
          float2 psa = make_float2(0.f, 0.f), psb = make_float2(0.f, 0.f);
          tmem_wait_ld();
          mask(s0, 0);
          float mx = max32(s0);
          exps32(s0, m_run, pk, psa);
          mask(s1, 32);
          mx = fmaxf(mx, max32(s1)) * sl;
          exps32(s1, m_run, pk + 16, psb);
          // above the range at any time; below it on the first tile, where a
          // low maximum may be the row's
          const bool need = mx > m_run + kRange || (j == 0 && mx < -kRange && mx > -INFINITY);
          if (__any_sync(0xffffffffu, need)) {
            float alpha = 1.f;
            if (need) {
              if (j > 0) alpha = ex2(m_run - mx);
              l_run *= alpha;
              m_run = mx;
            }
            if (j > 0) {
              // S(g) is there, so PV(g - 2) is done: PV(g - 1) is this phase or the last
              if (!(ok = wait_warp(C::kPVDone, (uint32_t)(g - 1) & 1u, 8))) break;
              tc_fence_after();
#pragma unroll 1
              for (int cc = 0; cc < D; cc += 32) {
                uint32_t o[32];
                tmem_ld32(tO + cc, o);
                tmem_wait_ld();
#pragma unroll
                for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * alpha);
                tmem_st32(tO + cc, o);
              }
            }
            psa = psb = make_float2(0.f, 0.f);
            exps32(s0, m_run, pk, psa);
            exps32(s1, m_run, pk + 16, psb);
          }
          tmem_st32(tS, pk);
          l_run += (psa.x + psa.y) + (psb.x + psb.y);
          tmem_wait_st();
          tc_fence_before();
        }
        mbar_arrive(bar(C::kPFull + 2 * (g & 1) + hf));
      }
      if (!ok) break;
      // ---------------------------------------------------------- epilogue
      // the halves meet: (m, l) through the query tile, which is read no more
      // (the other half may be a tile behind, so a barrier of query tiles, whose
      // every phase is waited for, says when: not that of key tiles)
      if (w.nt > 0 && !(ok = wait_warp(C::kODone, (uint32_t)tiles & 1u, 9))) break;
      tc_fence_after();
      uint8_t* stage = base + C::kQOff + (tiles & 1) * C::kTileBytes;
      float2* xch = reinterpret_cast<float2*>(stage);
      xch[hf * 128 + row] = make_float2(m_run, l_run);
      named_bar_sync(1, 256);
      const float2 other = xch[(1 - hf) * 128 + row];
      const float m0 = hf == 0 ? m_run : other.x, l0 = hf == 0 ? l_run : other.y;
      const float m1 = hf == 0 ? other.x : m_run, l1 = hf == 0 ? other.y : l_run;
      // a sum of 0 has no say; NaN has
      const bool on0 = live && l0 != 0.f, on1 = live && l1 != 0.f;
      const float M = fmaxf(on0 ? m0 : -INFINITY, on1 ? m1 : -INFINITY);
      const float e0 = on0 ? ex2(m0 - M) : 0.f, e1 = on1 ? ex2(m1 - M) : 0.f;
      const float L = (on0 ? l0 * e0 : 0.f) + (on1 ? l1 * e1 : 0.f);
      constexpr int kCols = D / 2;
      const uint32_t tO0 = tmem + lane_off + C::kTmemO + (uint32_t)(hf * kCols);
      // columns cc .. cc + 31 of this half's share of O, weighted; what a half
      // without keys left in TMEM is no number to count on
      auto join32 = [&](int cc, float f0, float f1, float (&v)[32]) {
        uint32_t oa[32], ob[32];
        if (w.nt > 0) {
          tmem_ld32(tO0 + cc, oa);
          tmem_ld32(tO0 + D + cc, ob);
          tmem_wait_ld();
        }
#pragma unroll
        for (int c = 0; c < 32; ++c)
          v[c] = (on0 ? __uint_as_float(oa[c]) * f0 : 0.f) + (on1 ? __uint_as_float(ob[c]) * f1 : 0.f);
      };
      if constexpr (!SPLIT) {
        const float inv = on0 || on1 ? 1.f / L : 0.f;
        const float f0 = e0 * inv, f1 = e1 * inv;
        uint32_t o[kCols / 2];
#pragma unroll
        for (int cc = 0; cc < kCols; cc += 32) {
          float v[32];
          join32(cc, f0, f1, v);
#pragma unroll
          for (int c = 0; c < 16; ++c) o[cc / 2 + c] = pack_bf16(v[2 * c], v[2 * c + 1]);
        }
        tc_fence_before();
        named_bar_sync(1, 256);  // O and the exchange are read: both may be written again
#pragma unroll
        for (int i = 0; i < kCols / 8; ++i) {
          const int k = hf * (kCols / 8) + i;
          *reinterpret_cast<uint4*>(stage + (k >> 3) * C::kBoxBytes + row * 128 + (((k & 7) ^ (row & 7)) << 4)) =
              make_uint4(o[4 * i], o[4 * i + 1], o[4 * i + 2], o[4 * i + 3]);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(C::kOReady));
        if (hf == 0 && stored && p.LSE != nullptr)
          p.LSE[lse_at] = on0 || on1 ? (M + __log2f(L)) * kLn2 : -INFINITY;
      } else {
        // ------------------------- the cluster's blocks join their key ranges
        // This block's (M, L) of every row where its cluster reads them; then
        // O, weighted, to the block that sums its columns (D / splits each).
        constexpr uint32_t kStat = 4096;  // past the exchange
        if (hf == 0)
          *reinterpret_cast<float2*>(stage + kStat + row * 8) =
              make_float2(on0 || on1 ? M : -INFINITY, *abort_flag ? -1.f : L);
        cluster_sync_all();
        float top = -INFINITY;
        bool bad = false;
        const uint32_t stat = base_u32 + C::kQOff + kStat + (uint32_t)row * 8u;
        float2 part[8];
#pragma unroll
        for (int c = 0; c < 8; ++c) {
          if (c < p.splits) {
            const uint32_t at = mapa(stat, (uint32_t)c);
            part[c] = make_float2(ld_dsmem_f32(at), ld_dsmem_f32(at + 4u));
            bad = bad || part[c].y == -1.f;
            top = fmaxf(top, part[c].x);
          }
        }
        float total = 0.f;
#pragma unroll
        for (int c = 0; c < 8; ++c)
          if (c < p.splits && part[c].x > -INFINITY) total += part[c].y * ex2(part[c].x - top);
        const bool any = top > -INFINITY;
        const float inv = any ? 1.f / total : 0.f;
        const float f0 = on0 ? ex2(m0 - top) * inv : 0.f, f1 = on1 ? ex2(m1 - top) * inv : 0.f;
        const int per = D / p.splits;  // columns of a block's sum
#pragma unroll 1
        for (int cc = 0; cc < kCols; cc += 32) {
          float v[32];
          join32(cc, f0, f1, v);
          if (!stored) continue;
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int col = hf * kCols + cc + 4 * i, to = col / per;
            st_dsmem_v4(mapa(base_u32 + C::kRingOff + (uint32_t)((split * 128 + row) * per + col - to * per) * 4u,
                             (uint32_t)to),
                        v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
          }
        }
        cluster_sync_all();
        if (stored && !bad) {
          const float* sum = reinterpret_cast<const float*>(base + C::kRingOff) + row * per;
          uint16_t* o = p.O + w.b * p.o_batch + t * p.o_token + (w.hb * p.pack + row_g) * D + split * per;
          for (int cc = 4 * hf; cc < per; cc += 8) {  // the halves take four columns in turn
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < p.splits; ++c) {
              const float4 x = *reinterpret_cast<const float4*>(sum + c * 128 * per + cc);
              a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
            }
            *reinterpret_cast<uint2*>(o + cc) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
          }
          if (split == 0 && hf == 0 && p.LSE != nullptr) p.LSE[lse_at] = any ? (top + __log2f(total)) * kLn2 : -INFINITY;
        }
      }
      if (w.nt > 0) ++tiles;
    }
    if (SPLIT && !ok) {  // the cluster still meets twice
      if (hf == 0) *reinterpret_cast<float2*>(base + C::kQOff + 4096 + row * 8) = make_float2(-INFINITY, -1.f);
      cluster_sync_all();
      cluster_sync_all();
    }
  } else if (!SPLIT) {
    // ------------------------------------------------------- the store of O
    if (lane == 0) {
      int tiles = 0;
      Cursor c;
      for (c.start(p, first_item, step, split); c.more; ++tiles) {
        const int qb = tiles & 1;
        if (!wait(C::kOReady, (uint32_t)tiles & 1u, 10) || *abort_flag) break;
#pragma unroll
        for (int bx = 0; bx < C::kBoxes; ++bx)
          tma_store_4d(&p.o_map, base_u32 + C::kQOff + qb * C::kTileBytes + bx * C::kBoxBytes, bx * 64,
                       c.w.hb * p.pack, c.w.t0, c.w.b);
        tma_store_commit_and_wait_read();
        mbar_arrive(bar(C::kQFree + qb));
        c.item += step;
        c.seek(p, step, split);
      }
    }
    __syncwarp();
  }
  if (SPLIT && (warp < 2 || warp >= 10)) {
    cluster_sync_all();
    cluster_sync_all();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool SPLIT>
cudaError_t launch_fwd(const CrossParams& p, int sms, cudaStream_t s) {
  using C = FwdCfg<D>;
  static bool attr_set = false;
  if (!attr_set) {
    cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<D, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::kSmemBytes);
    if (e == cudaSuccess && SPLIT)
      e = cudaFuncSetAttribute(cross_fwd_kernel<D, SPLIT>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    attr_set = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(SPLIT ? p.items * (unsigned)p.splits : (p.items < (unsigned)sms ? p.items : (unsigned)sms), 1, 1);
  cfg.blockDim = dim3(C::kThreads, 1, 1);
  cfg.dynamicSmemBytes = C::kSmemBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)p.splits;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = SPLIT ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D, SPLIT>, p);
}

}  // namespace

cudaError_t launch_cross_forward(const CrossParams& p, int sms, cudaStream_t s) {
  if (p.D == 128) return p.splits > 1 ? launch_fwd<128, true>(p, sms, s) : launch_fwd<128, false>(p, sms, s);
  return p.splits > 1 ? launch_fwd<64, true>(p, sms, s) : launch_fwd<64, false>(p, sms, s);
}

}  // namespace sab
