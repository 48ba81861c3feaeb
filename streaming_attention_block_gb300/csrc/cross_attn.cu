// Cross attention: one sequence's queries over another's keys and values (an
// encoder's states), for sm_103a.
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

#include <type_traits>

#include "cross_common.cuh"

namespace sab {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
// P = 2^(s - m) in bf16 has fp32's exponents and is summed in fp32, so the
// reference m need not be the row's maximum: any m that keeps the row's sum l from
// 2^-24 to 2^80 gives the same digits.  Nothing overflows below; a key whose P ftz
// drops has less than 2^-102 of the sum, and products P V below 2^-126 lose at most
// 2^-126 a key of O (a least sum of 2^-80 lost values of 2^-60 and below).  Rows
// take m = 0, without looking for a maximum; their sums are in that range where the
// largest score is between -16.6 and 55.4 - ln(keys).  A tile with a row whose l is
// not, or whose O is not finite, is done again with its running maxima, two tiles
// an item one by one.  2 x 30720 queries over 512 keys, 12 heads of 128: 142 us, with
// a row of it in every seventh tile 235, with all tiles done again 472; one chunk of
// 1536 queries 11 and 22; 16384 over 8192 keys, 8 heads, 331, 554 and 1265.
constexpr float kLeastSum = 0x1p-24f, kMostSum = 0x1p80f;
constexpr float kRescale = 8.0f;  // running maxima: O is rescaled when one grows by more than 2^8
constexpr int kRedoList = 64;     // query tiles a block remembers

// The number of a query tile, counted one by one.
__device__ __forceinline__ uint32_t tile_of(const CrossParams& p, const Spot& s, int st, int pair) {
  const uint32_t column = (uint32_t)s.b * (uint32_t)p.head_blocks + (uint32_t)s.hb;
  return column * (uint32_t)p.n_qtiles + (uint32_t)(s.iq * pair + st);
}

// ------------------------------------------------------------------ forward

// Scores of columns from hi on do not exist.
__device__ __forceinline__ void mask_from(uint32_t (&s)[32], int hi) {
  if (__builtin_expect(hi < 32, 0)) {
#pragma unroll
    for (int c = 0; c < 32; ++c) s[c] = c < hi ? s[c] : 0xff800000u;
  }
}
// P = 2^(s * sl - m) of 32 scores, as 16 columns of bf16 pairs to TMEM; sums by
// pairs into ps.
__device__ __forceinline__ void exps32(const uint32_t (&s)[32], float sl, float m, float2& ps, uint32_t to) {
  const float2 sl2 = make_float2(sl, sl), m2 = make_float2(-m, -m);
  uint32_t pk[16];
#pragma unroll
  for (int c = 0; c < 16; ++c) {
    const float2 x = __ffma2_rn(make_float2(__uint_as_float(s[2 * c]), __uint_as_float(s[2 * c + 1])), sl2, m2);
    const float e0 = ex2(x.x), e1 = ex2(x.y);
    ps = __fadd2_rn(ps, make_float2(e0, e1));
    pk[c] = pack_bf16(e0, e1);
  }
  tmem_st16(to, pk);
}

// One step with the running maximum, the same for the row's two halves: their
// warps meet twice, and exchange through columns of the scores that P leaves
// free.  tS: the step's scores of these lanes; tO: this half's columns of O.  At
// the last step half 0 returns the row's sum, half 1 its maximum, as l.  A call:
// its code would lie in the way of the fast steps'.
struct SlowSum {
  float m, l;
  bool ok;
};
__device__ __noinline__ SlowSum slow_step(const CrossParams& p, uint32_t meet, volatile int* abort_flag,
                                          uint32_t parity, uint32_t tS, uint32_t tO, int cols, int hf, int hi,
                                          bool first, bool last, float m, float l) {
  const int lane = threadIdx.x & 31;
  auto meet_pair = [&](uint32_t par) -> bool {
    __syncwarp();
    if (lane == 0) mbar_arrive(meet);
    return __all_sync(0xffffffffu, wait_bounded(meet, par, abort_flag, 13, p.err_word));
  };
  const uint32_t tX = tS + 32u;
  tS += (uint32_t)hf * 64u;
  uint32_t s0[32], s1[32];
  float own = -INFINITY;
  tc_fence_after();
  tmem_ld32(tS, s0);
  tmem_ld32(tS + 32, s1);
  tmem_wait_ld();
  mask_from(s0, hi);
  mask_from(s1, hi - 32);
#pragma unroll
  for (int k = 0; k < 32; ++k) own = fmax3(own, __uint_as_float(s0[k]), __uint_as_float(s1[k]));
  tmem_st1(tX + (uint32_t)hf * 64u, __float_as_uint(own));
  tmem_wait_st();
  tc_fence_before();
  if (!meet_pair(parity)) return SlowSum{m, l, false};
  tc_fence_after();
  const float top = fmaxf(own, __uint_as_float(tmem_ld1(tX + (uint32_t)(1 - hf) * 64u))) * p.scale_log2;
  float alpha = 1.f;
  if (first) {
    m = top > -INFINITY ? top : 0.f;
    l = 0.f;
  } else if (top > m + kRescale) {
    alpha = ex2(m - top);
    m = top;
  }
  if (!first && __any_sync(0xffffffffu, alpha != 1.f)) {
    // the scores are there, so the stream's products before them are done
#pragma unroll 1
    for (int cc = 0; cc < cols; cc += 16) {
      uint32_t v[16];
      tmem_ld16(tO + (uint32_t)cc, v);
      tmem_wait_ld();
#pragma unroll
      for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
      tmem_st16(tO + (uint32_t)cc, v);
    }
  }
  float2 ps = make_float2(0.f, 0.f);
  exps32(s0, p.scale_log2, m, ps, tS);
  exps32(s1, p.scale_log2, m, ps, tS + 16);
  l = l * alpha + (ps.x + ps.y);
  if (last) tmem_st1(tX + (uint32_t)hf * 64u + 1u, __float_as_uint(l));
  tmem_wait_st();
  tc_fence_before();
  if (!meet_pair(parity ^ 1u)) return SlowSum{m, l, false};  // both halves of O are rescaled, the maxima read
  if (last) {
    tc_fence_after();
    l = hf == 0 ? l + __uint_as_float(tmem_ld1(tX + 64u + 1u)) : m;
    tc_fence_before();
  }
  return SlowSum{m, l, true};
}

// Puts a query tile on the list of those to be done again; called by each of its
// rows that wants it (see the kernel for misc).
__device__ __noinline__ void again_later(const CrossParams& p, uint32_t* misc, uint32_t* list, unsigned end,
                                         unsigned item, const uint32_t* seqs, int st, int pair) {
  if (atomicMax(&misc[4], end) >= end) return;  // another row has
  const uint32_t n = atomicAdd(&misc[2], 1u);
  if (n < kRedoList) {
    const Spot s = seqs != nullptr ? sorted_spot(p, seqs, item) : spot_of(p, item, pair);
    list[n] = tile_of(p, s, st, pair);
  } else {
    atomicMin(&misc[3], item);
  }
}

template <int D_, bool PAIR>
struct FwdCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kQTiles = PAIR ? 2 : 1;
  static constexpr int kSlots = D == 128 ? (PAIR ? 4 : 5) : 10;  // K and V tiles in turn
  static constexpr uint32_t kOOff = 0;                           // O on its way out
  static constexpr uint32_t kQOff = kTileBytes;
  static constexpr uint32_t kRingOff = (1 + kQTiles) * kTileBytes;
  static constexpr uint32_t kSumOff = kRingOff + kSlots * kTileBytes;  // [2 streams][2][128]
  static constexpr uint32_t kBarOff = kSumOff + 2048;
  static constexpr int kQFull = 0;                          // [2 query tiles]
  static constexpr int kQFree = 2;                          // [2] the tile's last scores are done
  static constexpr int kFull = 4;                           // [kSlots]
  static constexpr int kEmpty = kFull + kSlots;             // [kSlots]
  static constexpr int kSFull = kEmpty + kSlots;            // [2 streams]
  static constexpr int kPFull = kSFull + 2;                 // [2]
  static constexpr int kODone = kPFull + 2;                 // [2] a query tile's last product
  static constexpr int kLReady = kODone + 2;                // [2] its sums
  static constexpr int kORead = kLReady + 2;                // [2] both are read
  static constexpr int kPairMeet = kORead + 2;              // [4 quadrants] running maxima only
  static constexpr int kOReady = kPairMeet + 4;             // O staged for its store
  static constexpr int kOFree = kOReady + 1;                // and read by it
  static constexpr int kDrain = kOFree + 1;                 // [2 streams]
  static constexpr int kNumBars = kDrain + 2;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kListOff = kMiscOff + 32;
  static constexpr uint32_t kSeqsOff = kListOff + kRedoList * 4;  // [kMaxSorted + 1]
  static constexpr uint32_t kSmemBytes = kSeqsOff + (kMaxSorted + 1) * 4;
  // K, V and Q; products of stream 0; the store of O; products of stream 1;
  // 8 softmax warps; 4 that end tiles
  static constexpr int kThreads = 32 * 16;
  static constexpr uint32_t kTmemO = 256;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// One block per SM walks its items.  An item's work is two streams of steps
// that take turns: two query tiles over the same key tiles (PAIR, which halves
// the traffic of K and V from L2), or one query tile over every other key tile
// each.  A stream has its own scores S (P goes over them), its own accumulator O
// and its own warp that issues the products, in the order S, PV, S, PV ...: with
// one warp for both, which has to ask some four barriers a step, the tensor cores
// waited for that warp (1800 cycles a step for 1024 of products; 1270 with two).
// Softmax: the keys [0, 64) and [64, 128) of a tile are two halves with four
// warps and a sum l each.  Four more warps take a finished O out while the next
// tile's steps go on.  SPLIT: one item a block, its keys cut among the blocks of
// a cluster (see the end).
template <int D, bool PAIR, bool SPLIT, bool RAGGED>
__global__ void __launch_bounds__(FwdCfg<D, PAIR>::kThreads, 1)
cross_fwd_kernel(const __grid_constant__ CrossParams p) {
  using C = FwdCfg<D, PAIR>;
  extern __shared__ __align__(1024) uint8_t base[];
  const uint32_t base_u32 = smem_u32(base);
  // [0] tmem, [1] abort, [2] tiles to be done again, [3] item at which the list
  // was full, [4] the end of a query tile that was last put on it
  uint32_t* misc = reinterpret_cast<uint32_t*>(base + C::kMiscOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(base + C::kMiscOff + 4);
  uint32_t* list = reinterpret_cast<uint32_t*>(base + C::kListOff);
  auto bar = [&](int i) -> uint32_t { return base_u32 + C::kBarOff + 8u * (uint32_t)i; };
  auto wait = [&](int i, uint32_t parity, unsigned site) -> bool {
    return wait_bounded(bar(i), parity, abort_flag, site, p.err_word);
  };
  auto wait_warp = [&](int i, uint32_t parity, unsigned site) -> bool {
    return __all_sync(0xffffffffu, wait(i, parity, site));
  };
  const int warp = uniform<true>(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const int split = SPLIT ? (int)(blockIdx.x % (unsigned)p.splits) : 0;
  auto arrive_warp = [&](int i) {  // one arrival for the warp
    __syncwarp();
    if (lane == 0) mbar_arrive(bar(i));
  };

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(C::kQFull + i), 1);
      mbar_init(bar(C::kQFree + i), PAIR ? 1 : 2);
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + i), 8);
      mbar_init(bar(C::kODone + i), 1);
      mbar_init(bar(C::kLReady + i), 8);
      mbar_init(bar(C::kORead + i), 4);
      mbar_init(bar(C::kDrain + i), 1);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 2);
    }
    for (int i = 0; i < 4; ++i) mbar_init(bar(C::kPairMeet + i), 2);
    mbar_init(bar(C::kOReady), 4);
    mbar_init(bar(C::kOFree), 1);
    misc[1] = (base_u32 & 1023u) != 0;  // the tiles' swizzle counts on it
    if (misc[1] != 0 && p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
    misc[2] = misc[4] = 0;
    misc[3] = 0xffffffffu;
    fence_mbar_init();
    fence_proxy_async_smem();
  }
  if (warp == 1) {
    tmem_alloc(base_u32 + C::kMiscOff, 512);
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
  const uint32_t tmem = (uint32_t)uniform<true>((int)misc[0]);
  griddep_launch_dependents();
  griddep_wait();

  Pass pass;
  pass.first = SPLIT ? blockIdx.x / (unsigned)p.splits : blockIdx.x;
  pass.step = SPLIT ? p.items : gridDim.x;
  pass.end = uniform<true>(*abort_flag) ? 0u : p.items;
  pass.list = pass.seqs = nullptr;
  pass.pair = PAIR ? 2 : 1;
  pass.split = split;
  if (RAGGED && p.sorted) {
    uint32_t* seqs = reinterpret_cast<uint32_t*>(base + C::kSeqsOff);
    sort_sequences(p, pass.pair, seqs, reinterpret_cast<uint32_t*>(base + C::kSumOff));
    pass.seqs = seqs;
    const unsigned rounds = ((unsigned)uniform<true>((int)(seqs[p.B] >> 6)) + gridDim.x - 1) / gridDim.x;
    if (pass.end > 0) pass.end = rounds * gridDim.x;
  }
  const unsigned all = pass.end;
  pass.by = SPLIT ? Spot{0, 0, 0} : spot_of(p, gridDim.x, pass.pair);
  // To the next pass, after all roles are through with this one; false: done.
  auto next_pass = [&](int& number) -> bool {
    if (SPLIT) return false;  // running maxima from the start
    __syncwarp();
    named_bar_sync(2, C::kThreads);
    if (uniform<true>(*abort_flag)) return false;
    const uint32_t n = (uint32_t)uniform<true>(min((int)misc[2], kRedoList));
    const uint32_t over = (uint32_t)uniform<true>((int)misc[3]);
    if (number == 0 && n > 0) {
      number = 1;
      pass.first = 0;
      pass.step = 1;
      pass.end = n;
      pass.list = list;
      pass.pair = 1;
      return true;
    }
    if (number < 2 && over != 0xffffffffu) {
      number = 2;
      pass.first = over;
      pass.step = gridDim.x;
      pass.end = all;
      pass.list = nullptr;
      pass.pair = PAIR ? 2 : 1;
      return true;
    }
    return false;
  };
  int number = 0;
  int steps_before = 0;  // of the block's items so far: in turn, steps go to stream 0 and 1 (not PAIR)
  // whether a stream has steps in an item of nt key tiles, and (not PAIR) the first
  auto first_tile = [&](int s) -> int { return (s ^ steps_before) & 1; };
  auto has_steps = [&](int s, int nt, int streams) -> bool { return PAIR ? s < streams : first_tile(s) < nt; };

  if (warp == 0) {
    // ----------------------------------------------------------- K, V and Q
    Ring<C::kSlots> r;
    int loads = 0, asked[2] = {0, 0};
    do {
      if (lane == 0) {
        const uint32_t q_bytes = (uint32_t)(C::kBoxes * p.pack * p.tile_tokens) * 128u;
        // one tile into the next slot
        auto load = [&](const CUtensorMap* m, int row, int head, int b) -> bool {
          if (loads >= C::kSlots && !wait(C::kEmpty + r.slot, r.parity ^ 1u, 0)) return false;
          const uint32_t full = bar(C::kFull + r.slot);
          mbar_arrive_expect_tx(full, C::kTileBytes);
#pragma unroll
          for (int bx = 0; bx < C::kBoxes; ++bx)
            tma_load_4d(base_u32 + C::kRingOff + r.slot * C::kTileBytes + bx * C::kBoxBytes, m, full, bx * 64, row,
                        head, b);
          r.next();
          ++loads;
          return true;
        };
        bool ok = true;
        Walk<false, RAGGED> c;
        for (c.start(p, pass); ok && c.more(pass); c.next(p, pass)) {
          const Work& w = c.w;
          if (w.nt == 0) continue;
          const int head = w.hb * p.pack / p.group, kb = p.Bk == 1 ? 0 : w.b;
          for (int j = 0; ok && j < w.nt; ++j) {
            if (!(ok = load(&p.k_map, (w.first + j) * kTileN, head, kb))) break;
            // there is room for the first keys before there is for the queries,
            // which the item before reads to its end
            if (j == 0) {
#pragma unroll
              for (int t = 0; t < C::kQTiles; ++t) {
                if (t >= w.streams) break;
                if (asked[t] > 0 && !(ok = wait(C::kQFree + t, (uint32_t)(asked[t] - 1) & 1u, 1))) break;
                ++asked[t];
                mbar_arrive_expect_tx(bar(C::kQFull + t), q_bytes);
#pragma unroll
                for (int bx = 0; bx < C::kBoxes; ++bx)
                  tma_load_4d(base_u32 + C::kQOff + t * C::kTileBytes + bx * C::kBoxBytes, &p.q_map, bar(C::kQFull + t),
                              bx * 64, query_c1(p, w, t), query_c2(p, w, t), w.b);
              }
            }
            ok = ok && load(&p.v_map, (w.first + j) * kTileN, head, kb);
          }
        }
      }
    } while (next_pass(number));
    if (lane == 0 && *abort_flag) {  // nothing of this block's copies may land after it
      for (int k = max(0, loads - C::kSlots); k < loads; ++k)
        wait_drain(bar(C::kFull + k % C::kSlots), (uint32_t)(k / C::kSlots) & 1u, p.err_word);
#pragma unroll
      for (int t = 0; t < C::kQTiles; ++t)
        if (asked[t] > 0) wait_drain(bar(C::kQFull + t), (uint32_t)(asked[t] - 1) & 1u, p.err_word);
    }
    __syncwarp();
  } else if (warp == 1 || warp == 3) {
    // ------------------------------------------------------------- products
    const int s = warp == 3 ? 1 : 0;  // the stream
    const int qt = PAIR ? s : 0;
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTileN, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
    constexpr uint32_t kStep = C::kTileBytes >> 4;
    const uint64_t dq = smem_desc_sw128(base_u32 + C::kQOff + qt * C::kTileBytes, 16, 1024);
    const uint64_t dk = smem_desc_sw128(base_u32 + C::kRingOff, 16, 1024);
    const uint64_t dv = smem_desc_sw128(base_u32 + C::kRingOff, C::kBoxBytes, 1024);
    const uint32_t q_lo = (uint32_t)dq, k_lo = (uint32_t)dk, v_lo = (uint32_t)dv;
    const uint32_t kq_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
    const uint32_t tS = tmem + (uint32_t)s * 128u, tO = tmem + C::kTmemO + (uint32_t)s * D;
    const uint32_t lead = elect_lead();
    Ring<C::kSlots> r;  // place of the key tile; its values are one on
    uint32_t q_parity = 0, p_parity = 0;
    int used = 0;  // query tiles in this accumulator so far
    bool ok = true;
    auto scores = [&]() -> bool {  // S = Q K^T
      if (!wait_warp(C::kFull + r.slot, r.parity, 3)) return false;
      tc_fence_after();
      const uint32_t b0 = k_lo + r.slot * kStep;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
        mma_ss_l(lead, tS, make_desc(q_lo + off, kq_hi), make_desc(b0 + off, kq_hi), idesc_qk, kk > 0 ? 1u : 0u);
      }
      mma_commit_l(lead, bar(C::kSFull + s));
      mma_commit_l(lead, bar(C::kEmpty + r.slot));
      return true;
    };
    // Past a key tile that only the other stream works on.  Its slots are waited
    // for and freed all the same: a parity tells two rounds of a slot apart, so
    // no warp may be a round behind another.
    auto pass_by = [&]() -> bool {
      for (int i = 0; i < 2; ++i) {
        if (!wait_warp(C::kFull + r.slot, r.parity, 3)) return false;
        arrive_warp(C::kEmpty + r.slot);
        r.next();
      }
      return true;
    };
    do {
      Walk<true, RAGGED> ahead;  // the next item is looked up while the softmax works on this one
      ahead.start(p, pass);
      ahead.seek(p, pass);
      while (ahead.more(pass)) {
        const struct {
          int nt, streams, keys;
        } c = {ahead.w.nt, ahead.w.streams, ahead.w.keys};
        if (!has_steps(s, c.nt, c.streams)) {
          ahead.next(p, pass);
          ahead.seek(p, pass);
          if (!PAIR) {
            if (!(ok = wait_warp(C::kQFull, q_parity, 2))) break;
            q_parity ^= 1u;
            arrive_warp(C::kQFree);
          }
          for (int j = 0; ok && j < c.nt; ++j) ok = pass_by();
          if (!ok) break;
          steps_before += c.nt;
          continue;
        }
        if (!(ok = wait_warp(C::kQFull + qt, q_parity, 2))) break;
        q_parity ^= 1u;
        constexpr int kBy = PAIR ? 1 : 2;  // key tiles from step to step
        int j = PAIR ? 0 : first_tile(s);
        if (j > 0 && !(ok = pass_by())) break;
        if (!(ok = scores())) break;
        ahead.next(p, pass);
        ahead.seek(p, pass);
        bool begun = false;
        for (;;) {
          const bool more = j + kBy < c.nt;
          if (!more) mma_commit_l(lead, bar(C::kQFree + qt));
          // O += P V
          const int keys = c.keys - j * kTileN, steps = min(8, (keys + 15) >> 4);  // 16 keys each
          Ring<C::kSlots> v = r;
          v.next();
          if (!(ok = wait_warp(C::kFull + v.slot, v.parity, 3))) break;
          // keys past the sequence's end may hold anything, and 0 * NaN is NaN:
          // the values of the last step's are zeroed (later steps are left out)
          if (__builtin_expect(steps * 16 > keys, 0))
            zero_rows<C::kBoxes>(base + C::kRingOff + v.slot * C::kTileBytes, keys, steps * 16);
          // the first product of a query tile overwrites what the accumulator held
          if (__builtin_expect(!begun && used > 0, 0) &&
              !(ok = wait_warp(C::kORead + s, (uint32_t)(used - 1) & 1u, 4)))
            break;
          if (!(ok = wait_warp(C::kPFull + s, p_parity, 5))) break;
          p_parity ^= 1u;
          tc_fence_after();
          const uint32_t b0 = v_lo + v.slot * kStep;
          // P of keys 64 .. 127 starts 64 columns after that of the first 64
          auto product = [&](int kk) {
            mma_ts_l(lead, tO, tS + (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u,
                     make_desc(b0 + ((uint32_t)(kk * 16 * 128) >> 4), v_hi), idesc_pv, kk > 0 || begun ? 1u : 0u);
          };
          if (__builtin_expect(steps == 8, 1)) {
#pragma unroll
            for (int kk = 0; kk < 8; ++kk) product(kk);
          } else {
#pragma unroll 1
            for (int kk = 0; kk < steps; ++kk) product(kk);
          }
          begun = true;
          mma_commit_l(lead, bar(C::kEmpty + v.slot));
          r.next();
          r.next();
          if (!PAIR && j + 1 < c.nt && !(ok = pass_by())) break;
          if (!more) break;
          j += kBy;
          if (!(ok = scores())) break;
        }
        if (!ok) break;
        mma_commit_l(lead, bar(C::kODone + s));
        ++used;
        steps_before += c.nt;
      }
    } while (next_pass(number) && ok);
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain + s));
      if (lane == 0) wait_drain(bar(C::kDrain + s), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------- the store of O
    int tile = 0;
    if (RAGGED && !uniform<true>(*abort_flag)) {
      fill_zeros(base + C::kOOff, C::kTileBytes);
      clear_tiles<C::kBoxes>(p, pass.pair, base_u32 + C::kOOff, p.LSE);
    }
    if (!SPLIT && lane == 0) mbar_arrive(bar(C::kOFree));
    do {
      if (lane == 0 && !SPLIT) {
        bool ok = true;
        Walk<false, RAGGED> c;
        for (c.start(p, pass); ok && c.more(pass); c.next(p, pass)) {
          const Work& w = c.w;
          if (w.nt == 0) continue;
          for (int t = 0; t < w.streams; ++t, ++tile) {
            if (!(ok = wait(C::kOReady, (uint32_t)tile & 1u, 10) && !*abort_flag)) break;
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_store_4d(&p.o_map, base_u32 + C::kOOff + bx * C::kBoxBytes, bx * 64, query_c1(p, w, t),
                           query_c2(p, w, t), w.b);
            tma_store_commit_and_wait_read();
            mbar_arrive(bar(C::kOFree));
          }
        }
        tma_store_wait_all();  // a later pass may write the same rows
      }
    } while (next_pass(number));
    __syncwarp();
  } else if (warp < 12) {
    // -------------------------------------------------------------- softmax
    const int hf = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tSh = tmem + lane_off + (uint32_t)hf * 64u;  // + stream * 128
    const int warp_t = (quad * 32) / p.pack;  // first token of the warp's rows
    int used[2] = {0, 0};
    uint32_t s_parity[2] = {0u, 0u};
    bool ok = true;
    // one step of stream S of an item
    float m_s[2] = {0.f, 0.f}, l_s[2] = {0.f, 0.f};
    uint32_t pair_parity = 0;  // of the two warps' meetings: two a step, so it stays 0 between steps
    auto step = [&](auto stream, bool slow, int keys, int rows_live, int tile, bool first, bool last) -> bool {
      constexpr int S = decltype(stream)::value;
      if (!wait_warp(C::kSFull + S, s_parity[S], 6 + hf)) return false;
      s_parity[S] ^= 1u;
      const int hi = keys - tile * kTileN - hf * 64;                            // visible columns of this half
      const bool busy = (PAIR ? S * p.tile_tokens : 0) + warp_t < rows_live;  // some row of the warp is live
      const uint32_t tS = tSh + (uint32_t)S * 128u;
      float& l = l_s[S];
      float& m = m_s[S];
      if (__builtin_expect(!slow, 1)) {
        if (__builtin_expect(busy && hi > 0, 1)) {
          tc_fence_after();
          uint32_t s0[32], s1[32];
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          tmem_wait_ld();
          float2 ps = make_float2(0.f, 0.f);
          mask_from(s0, hi);
          exps32(s0, p.scale_log2, 0.f, ps, tS);
          tmem_wait_ld();
          mask_from(s1, hi - 32);
          exps32(s1, p.scale_log2, 0.f, ps, tS + 16);
          l += ps.x + ps.y;
          tmem_wait_st();
          tc_fence_before();
        }
      } else {
        const SlowSum x = slow_step(p, bar(C::kPairMeet + quad), abort_flag, pair_parity, tmem + lane_off + (uint32_t)S * 128u,
                                    tmem + lane_off + C::kTmemO + (uint32_t)(S * D + hf * (D / 2)), D / 2, hf, hi,
                                    first, last, m, l);
        if (!x.ok) return false;
        m = x.m;
        l = x.l;
      }
      arrive_warp(C::kPFull + S);
      if (__builtin_expect(last, 0)) {
        // the sums of a query tile: two halves, or (running maxima) sum and maximum
        if (used[S] > 0 && !wait_warp(C::kORead + S, (uint32_t)(used[S] - 1) & 1u, 9)) return false;
        reinterpret_cast<float*>(base + C::kSumOff)[(S * 2 + hf) * 128 + row] = l;
        arrive_warp(C::kLReady + S);
        ++used[S];
        l = 0.f;
      }
      return true;
    };
    const std::integral_constant<int, 0> zero;
    const std::integral_constant<int, 1> one;
    do {
      const bool slow = SPLIT || number > 0;
      Walk<true, RAGGED> c;
      c.start(p, pass);
      c.seek(p, pass);
      while (ok && c.more(pass)) {
        const int nt = c.w.nt, streams = c.w.streams, keys = c.w.keys, live = c.w.live;
        if (PAIR) {
          for (int j = 0; ok && j < nt; ++j) {
            ok = step(zero, slow, keys, live, j, j == 0, j + 1 == nt);
            if (ok && streams == 2) ok = step(one, slow, keys, live, j, j == 0, j + 1 == nt);
          }
        } else {
          for (int j = -(steps_before & 1); ok && j < nt; j += 2) {
            if (j >= 0) ok = step(zero, slow, keys, live, j, j < 2, j + 2 >= nt);
            if (ok && j + 1 < nt) ok = step(one, slow, keys, live, j + 1, j < 1, j + 3 >= nt);
          }
          steps_before += nt;
        }
        c.next(p, pass);
        c.seek(p, pass);
      }
    } while (next_pass(number) && ok);
  } else {
    // ------------------------------------------------------- ends of tiles
    const int quad = warp & 3, row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const int row_t = row / p.pack, row_g = row - row_t * p.pack;
    const float* sums = reinterpret_cast<const float*>(base + C::kSumOff);
    uint8_t* stage = base + C::kOOff;
    bool ok = pass.end > 0;
    int used[2] = {0, 0}, tiles = 0;
    auto finish = [&](const Work& w, unsigned item, int st) -> bool {
      if (kDebugBounds && w.b < 0) return false;  // a part of a cluster: none of its blocks stores
      const int t = w.t0 + st * p.tile_tokens + row_t;
      const bool stored = row_t < p.tile_tokens && t < p.Lq;  // this row has an O and an LSE
      const bool live = row_t < p.tile_tokens && st * p.tile_tokens + row_t < w.live;
      const long long lse_at = ((long long)w.b * p.H + w.hb * p.pack + row_g) * p.Lq + t;
      // the streams' sums and products
      bool on[2] = {false, false}, has[2];
      float m[2] = {0.f, 0.f}, l[2] = {0.f, 0.f};
#pragma unroll
      for (int o = 0; o < 2; ++o) {
        has[o] = PAIR ? o == st : has_steps(o, w.nt, 1);
        if (!has[o]) continue;
        if (!wait_warp(C::kLReady + o, (uint32_t)used[o] & 1u, 12)) return false;
        const float x = sums[(o * 2) * 128 + row], y = sums[(o * 2 + 1) * 128 + row];
        l[o] = SPLIT || number > 0 ? x : x + y;
        m[o] = SPLIT || number > 0 ? y : 0.f;
        on[o] = live && l[o] != 0.f;  // a sum of 0 has no say; NaN has
        if (!wait_warp(C::kODone + o, (uint32_t)used[o] & 1u, 9)) return false;
        ++used[o];
      }
      tc_fence_after();
      const float top_own = fmaxf(on[0] ? m[0] : -INFINITY, on[1] ? m[1] : -INFINITY);
      const float sum = (on[0] ? l[0] * ex2(m[0] - top_own) : 0.f) + (on[1] ? l[1] * ex2(m[1] - top_own) : 0.f);
      const bool any_own = on[0] || on[1];
      const uint32_t tO = tmem + lane_off + C::kTmemO;
      // columns cc .. cc + 31 of O: the streams' weighted (what a stream without
      // keys left in TMEM is no number to count on)
      auto take = [&](int cc, const float (&f)[2], float2 (&x)[16]) {
#pragma unroll
        for (int c = 0; c < 16; ++c) x[c] = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < (PAIR ? 1 : 2); ++i) {
          const int o = PAIR ? st : i;
          if (!PAIR && !has[i]) continue;
          uint32_t v[32];
          tmem_ld32(tO + (uint32_t)(o * D + cc), v);
          tmem_wait_ld();
          if (cc + 32 == D) {
            tc_fence_before();
            arrive_warp(C::kORead + o);
          }
          const float w = o ? f[1] : f[0];
          const float2 g = make_float2(w, w);
          if (o ? on[1] : on[0]) {
#pragma unroll
            for (int c = 0; c < 16; ++c)
              x[c] = __ffma2_rn(make_float2(__uint_as_float(v[2 * c]), __uint_as_float(v[2 * c + 1])), g, x[c]);
          }
        }
      };
      if constexpr (!SPLIT) {
        const float inv = any_own ? 1.f / sum : 0.f;
        const float f[2] = {on[0] ? ex2(m[0] - top_own) * inv : 0.f, on[1] ? ex2(m[1] - top_own) * inv : 0.f};
        if (!wait_warp(C::kOFree, (uint32_t)tiles & 1u, 11)) return false;
        ++tiles;
        float2 sound = make_float2(0.f, 0.f);  // stays 0 unless some value is not finite
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float2 x[16];
          take(cc, f, x);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              sound = __ffma2_rn(x[4 * i + c], make_float2(0.f, 0.f), sound);
              w4[c] = pack_bf16(x[4 * i + c].x, x[4 * i + c].y);
            }
            const int k = cc / 8 + i;
            *reinterpret_cast<uint4*>(stage + (k >> 3) * C::kBoxBytes + row * 128 + (((k & 7) ^ (row & 7)) << 4)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
        }
        const bool again =
            number == 0 && live && !(sum >= kLeastSum && sum <= kMostSum && sound.x == 0.f && sound.y == 0.f);
        if (__builtin_expect(again, 0)) again_later(p, misc, list, (unsigned)tiles, item, pass.seqs, st, pass.pair);
        fence_proxy_async_smem();
        arrive_warp(C::kOReady);
        if (stored && p.LSE != nullptr) p.LSE[lse_at] = any_own ? (top_own + __log2f(sum)) * kLn2 : -INFINITY;
      } else {
        // ------------------------- the cluster's blocks join their key ranges
        // This block's maximum and sum of every row where its cluster reads them;
        // then O, weighted, to the block that sums its columns (D / splits each).
        *reinterpret_cast<float2*>(stage + row * 8) =
            make_float2(any_own ? top_own : -INFINITY, *abort_flag ? -1.f : sum);
        cluster_sync_all();
        float top = -INFINITY;
        bool bad = false;
        const uint32_t stat = base_u32 + C::kOOff + (uint32_t)row * 8u;
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
        const float f[2] = {on[0] ? ex2(m[0] - top) / total : 0.f, on[1] ? ex2(m[1] - top) / total : 0.f};
        const int per = D / p.splits;  // columns of a block's sum
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 32) {
          float2 x[16];
          take(cc, f, x);
          if (stored) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int col = cc + 4 * i, to = col / per;
              st_dsmem_v4(mapa(base_u32 + C::kRingOff + (uint32_t)((split * 128 + row) * per + col - to * per) * 4u,
                               (uint32_t)to),
                          x[2 * i].x, x[2 * i].y, x[2 * i + 1].x, x[2 * i + 1].y);
            }
          }
          __syncwarp();
        }
        cluster_sync_all();
        if (stored && !bad) {
          const float* all = reinterpret_cast<const float*>(base + C::kRingOff) + row * per;
          uint16_t* out = p.O + w.b * p.o_batch + t * p.o_token + (w.hb * p.pack + row_g) * p.o_head + split * per;
          for (int cc = 0; cc < per; cc += 4) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < p.splits; ++c) {
              const float4 x = *reinterpret_cast<const float4*>(all + c * 128 * per + cc);
              a.x += x.x, a.y += x.y, a.z += x.z, a.w += x.w;
            }
            *reinterpret_cast<uint2*>(out + cc) = make_uint2(pack_bf16(a.x, a.y), pack_bf16(a.z, a.w));
          }
          if (split == 0 && p.LSE != nullptr) p.LSE[lse_at] = any ? (top + __log2f(total)) * kLn2 : -INFINITY;
        }
      }
      return true;
    };
    do {
      Walk<true, RAGGED> c;
      for (c.start(p, pass); ok && c.more(pass); c.next(p, pass)) {
        const Work& w = c.w;
        if (!SPLIT && w.nt == 0) continue;
#pragma unroll 1
        for (int st = 0; ok && st < w.streams; ++st) ok = finish(w, c.at, st);
        steps_before += w.nt;
      }
    } while (next_pass(number) && ok);
    if (SPLIT && !ok) {  // the cluster still meets twice
      *reinterpret_cast<float2*>(stage + row * 8) = make_float2(-INFINITY, -1.f);
      cluster_sync_all();
      cluster_sync_all();
    }
  }
  if (SPLIT && warp < 12) {
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

template <int D, bool PAIR, bool SPLIT, bool RAGGED>
cudaError_t launch_fwd(const CrossParams& p, int sms, cudaStream_t s) {
  using C = FwdCfg<D, PAIR>;
  static std::atomic<unsigned long long> ready;
  const cudaError_t e = allow_smem(cross_fwd_kernel<D, PAIR, SPLIT, RAGGED>, C::kSmemBytes, ready);
  if (e != cudaSuccess) return e;
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
  return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D, PAIR, SPLIT, RAGGED>, p);
}

template <int D>
cudaError_t forward(const CrossParams& p, int sms, cudaStream_t s) {
  if (p.splits > 1) return launch_fwd<D, false, true, false>(p, sms, s);
  if (p.q_len != nullptr || p.kv_len != nullptr)
    return p.pair == 2 ? launch_fwd<D, true, false, true>(p, sms, s) : launch_fwd<D, false, false, true>(p, sms, s);
  return p.pair == 2 ? launch_fwd<D, true, false, false>(p, sms, s) : launch_fwd<D, false, false, false>(p, sms, s);
}

}  // namespace

cudaError_t launch_cross_forward(const CrossParams& p, int sms, cudaStream_t s) {
  return p.D == 128 ? forward<128>(p, sms, s) : forward<64>(p, sms, s);
}

}  // namespace sab
