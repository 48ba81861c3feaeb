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
// reference m need not be the row's maximum: any m that keeps the sum l within
// 2^80 of 1 gives the same digits (nothing overflows, and what ftz drops is
// below 2^-46 of the sum).  Rows take m = 0, without looking for a maximum, which
// scores below 55 in size never need; a tile with a row whose l leaves the range,
// or whose O is not finite, is done again with its running maxima.
constexpr float kLeastSum = 0x1p-80f, kMostSum = 0x1p80f;
constexpr float kRescale = 8.0f;  // running maxima: O is rescaled when one grows by more than 2^8
constexpr int kRedoList = 64;     // query tiles a block remembers

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

// The number of a query tile, counted one by one, from its item and stream.
__device__ __forceinline__ uint32_t tile_of(const CrossParams& p, unsigned item, int st, int pair) {
  const unsigned n = (unsigned)(p.n_qtiles + pair - 1) / (unsigned)pair;
  const unsigned r = item / n;
  return r * (unsigned)p.n_qtiles + (item - r * n) * (unsigned)pair + (unsigned)st;
}

// ------------------------------------------------------------------ forward

// kUniform: the whole warp asks, and the answer is told the compiler to be one
// value for all lanes (the operands of the products live in uniform registers;
// what it does not know to be uniform it moves there lane by lane, every time).
template <bool kUniform>
__device__ __forceinline__ int uniform(int x) {
  return kUniform ? __shfl_sync(0xffffffffu, x, 0) : x;
}
template <bool kUniform>
__device__ __forceinline__ int length_of(const int* lens, int b, int most) {
  return lens == nullptr ? most : uniform<kUniform>(min(max(__ldg(lens + b), 0), most));
}

// One or two query tiles (`streams`) of `pack` heads from head hb * pack on,
// tile_tokens tokens each from t0 on, and the key tiles [first, first + nt).
struct Work {
  int b, hb, t0;
  int live;         // tokens from t0 on that are inside q_len
  int streams;
  int first, nt;
  int keys;         // keys of the range
};
template <bool kUniform>
__device__ __forceinline__ Work work_at(const CrossParams& p, unsigned item, int split, int pair) {
  Work w;
  const unsigned n = (unsigned)(p.n_qtiles + pair - 1) / (unsigned)pair;
  const unsigned r = item / n;
  w.t0 = (int)(item - r * n) * pair * p.tile_tokens;
  w.b = (int)(r / (unsigned)p.head_blocks);
  w.hb = (int)(r - (unsigned)w.b * (unsigned)p.head_blocks);
  w.live = length_of<kUniform>(p.q_len, w.b, p.Lq) - w.t0;
  w.streams = pair == 2 && w.live > p.tile_tokens ? 2 : 1;
  const int kl = w.live > 0 ? length_of<kUniform>(p.kv_len, p.Bk == 1 ? 0 : w.b, p.Lk) : 0;
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

// What a block works through.  Pass 0: every step-th item.  Pass 1: the query
// tiles of the list, one by one.  Pass 2: the items of pass 0 from the one on at
// which the list was full.
struct Pass {
  unsigned first, step, end;  // items, or places of the list
  const uint32_t* list;       // or null
  int pair, split;
};
// Steps of a pass in order: each key tile of an item, for each of its streams.
template <bool kUniform>
struct Cursor {
  unsigned at, item;
  Work w;
  int j, st;
  bool more;
  __device__ __forceinline__ void start(const CrossParams& p, const Pass& a) {
    at = a.first;
    seek(p, a);
  }
  __device__ __forceinline__ void seek(const CrossParams& p, const Pass& a) {
    j = st = 0;
    for (; at < a.end; at += a.step) {
      item = a.list != nullptr ? (unsigned)uniform<kUniform>((int)a.list[at]) : at;
      w = work_at<kUniform>(p, item, a.split, a.pair);
      if (w.nt > 0) {
        more = true;
        return;
      }
    }
    more = false;
  }
  __device__ __forceinline__ void skip(const CrossParams& p, const Pass& a) {
    at += a.step;
    seek(p, a);
  }
  __device__ __forceinline__ bool last() const { return j + 1 == w.nt; }
  // the next step; true where it has another key tile
  __device__ __forceinline__ bool next(const CrossParams& p, const Pass& a) {
    if (++st < w.streams) return false;
    st = 0;
    if (++j == w.nt) skip(p, a);
    return true;
  }
};

template <int D_, bool PAIR>
struct FwdCfg {
  static constexpr int D = D_;
  static constexpr int kBoxes = D / 64;
  static constexpr uint32_t kBoxBytes = 128u * 128u;
  static constexpr uint32_t kTileBytes = kBoxBytes * kBoxes;
  static constexpr int kStreams = PAIR ? 2 : 1;
  static constexpr int kSlots = D == 128 ? (PAIR ? 4 : 5) : 10;  // K and V tiles in turn
  static constexpr uint32_t kOOff = 0;                           // O on its way out
  static constexpr uint32_t kQOff = kTileBytes;                  // a query tile of each stream
  static constexpr uint32_t kRingOff = (1 + kStreams) * kTileBytes;
  static constexpr uint32_t kSumOff = kRingOff + kSlots * kTileBytes;  // [2 accumulators][2][128]
  static constexpr uint32_t kBarOff = kSumOff + 2048;
  static constexpr int kQFull = 0;                          // [2 streams]
  static constexpr int kQFree = 2;                          // [2] the tile's last scores are done
  static constexpr int kFull = 4;                           // [kSlots]
  static constexpr int kEmpty = kFull + kSlots;             // [kSlots]
  static constexpr int kSFull = kEmpty + kSlots;            // [2 buffers]
  static constexpr int kPFull = kSFull + 2;                 // [2 buffers]
  static constexpr int kODone = kPFull + 2;                 // [2 accumulators] a query tile's last product
  static constexpr int kLReady = kODone + 2;                // [2] its sums
  static constexpr int kORead = kLReady + 2;                // [2] both are read
  static constexpr int kPVDone = kORead + 2;                // running maxima only
  static constexpr int kPairMeet = kPVDone + 1;             // [4 quadrants] running maxima only
  static constexpr int kOReady = kPairMeet + 4;             // O staged for its store
  static constexpr int kOFree = kOReady + 1;                // and read by it
  static constexpr int kDrain = kOFree + 1;
  static constexpr int kNumBars = kDrain + 1;
  static constexpr uint32_t kMiscOff = kBarOff + kNumBars * 8;
  static constexpr uint32_t kListOff = kMiscOff + 32;
  static constexpr uint32_t kSmemBytes = kListOff + kRedoList * 4;
  // K and V, products, the store of O, Q; 8 softmax warps; 4 that end tiles
  static constexpr int kThreads = 32 * 16;
  static constexpr uint32_t kTmemO = 256;
  static_assert(kSmemBytes <= 232448, "shared memory budget");
};

// One block per SM walks its items: one query tile, or two that share their
// key tiles (PAIR), which halves the traffic of K and V from L2.  SPLIT: one
// item a block, its keys cut among the blocks of a cluster (see the end).
// Scores of a step (a key tile and a stream) are in one of two TMEM buffers; the
// keys [0, 64) and [64, 128) of a tile are two halves with four softmax warps
// and a sum l each.  Products are issued in the order PV(g), S(g + 2) over all
// steps of the block, also from one query tile to the next, and there are two
// accumulators O (of the two streams, or of every other query tile): four warps
// of their own take a finished one out while the next tile's steps go on.
template <int D, bool PAIR, bool SPLIT>
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
      mbar_init(bar(C::kQFree + i), 1);
      mbar_init(bar(C::kSFull + i), 1);
      mbar_init(bar(C::kPFull + i), 8);
      mbar_init(bar(C::kODone + i), 1);
      mbar_init(bar(C::kLReady + i), 8);
      mbar_init(bar(C::kORead + i), 4);
    }
    for (int s = 0; s < C::kSlots; ++s) {
      mbar_init(bar(C::kFull + s), 1);
      mbar_init(bar(C::kEmpty + s), 1);
    }
    mbar_init(bar(C::kPVDone), 1);
    for (int i = 0; i < 4; ++i) mbar_init(bar(C::kPairMeet + i), 2);
    mbar_init(bar(C::kOReady), 4);
    mbar_init(bar(C::kOFree), 1);
    mbar_init(bar(C::kDrain), 1);
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
  pass.list = nullptr;
  pass.pair = PAIR ? 2 : 1;
  pass.split = split;
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
      pass.end = p.items;
      pass.list = nullptr;
      pass.pair = PAIR ? 2 : 1;
      return true;
    }
    return false;
  };
  int number = 0;
  // The accumulator of a query tile, and how often each has been used: of the
  // tile's stream in PAIR, else in turn.
  int used[2] = {0, 0}, tiles = 0;
  auto accumulator = [&](int st) -> int { return PAIR ? st : tiles & 1; };
  auto uses = [&](int o) -> int { return o ? used[1] : used[0]; };
  auto use = [&](int o) {
    ++tiles;
    if (o) ++used[1];
    else ++used[0];
  };

  if (warp == 0) {
    // -------------------------------------------------------------- K and V
    Ring<C::kSlots> r;
    int loads = 0;
    do {
      if (lane == 0) {
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
        Cursor<false> c;
        for (c.start(p, pass); c.more;) {
          const int head = c.w.hb * p.pack / p.group, kb = p.Bk == 1 ? 0 : c.w.b;
          const int row = (c.w.first + c.j) * kTileN;
          if (!load(&p.k_map, row, head, kb) || !load(&p.v_map, row, head, kb)) break;
          while (!c.next(p, pass)) {
          }
        }
      }
    } while (next_pass(number));
    if (lane == 0 && *abort_flag)  // nothing of this block's copies may land after it
      for (int k = max(0, loads - C::kSlots); k < loads; ++k)
        wait_drain(bar(C::kFull + k % C::kSlots), (uint32_t)(k / C::kSlots) & 1u, p.err_word);
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------- products
    // Shared memory feeds the products at its full rate, so a barrier's answer
    // takes this warp some 200 cycles: the next one is asked in the middle of
    // the products before it.
    constexpr uint32_t idesc_qk = idesc_bf16_f32(128, kTileN, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(128, D, 1);
    const uint64_t dq = smem_desc_sw128(base_u32 + C::kQOff, 16, 1024);
    const uint64_t dk = smem_desc_sw128(base_u32 + C::kRingOff, 16, 1024);
    const uint64_t dv = smem_desc_sw128(base_u32 + C::kRingOff, C::kBoxBytes, 1024);
    const uint32_t kq_hi = (uint32_t)(dq >> 32), v_hi = (uint32_t)(dv >> 32);
    constexpr uint32_t kStep = C::kTileBytes >> 4;
    const uint32_t lead = elect_lead();
    Ring<C::kSlots> rk, rv;  // the places of the two cursors' tiles
    rv.next();
    int gs = 0, gv = 0;
    uint32_t q_parity[2] = {0u, 0u};
    bool ok = true, p_there = false, k_there = false;  // asked ahead
    auto ask = [&](int i, uint32_t parity) -> bool {
      return __all_sync(0xffffffffu, mbar_test_wait(bar(i), parity));
    };
    do {
      Cursor<true> cs, cv;  // the step whose scores, and whose values, come next
      cs.start(p, pass);
      cv = cs;
      auto issue_s = [&]() -> bool {  // S(gs) = Q K^T
        const int st = PAIR ? cs.st : 0;
        if (cs.j == 0) {
          if (!wait_warp(C::kQFull + st, st ? q_parity[1] : q_parity[0], 2)) return false;
          if (st) q_parity[1] ^= 1u;
          else q_parity[0] ^= 1u;
        }
        if (st == 0 && !k_there && !wait_warp(C::kFull + rk.slot, rk.parity, 3)) return false;
        k_there = false;
        tc_fence_after();
        const uint32_t a0 = (uint32_t)dq + (uint32_t)st * kStep, b0 = (uint32_t)dk + rk.slot * kStep;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = ((kk >> 2) * C::kBoxBytes + (kk & 3) * 32) >> 4;
          mma_ss_l(lead, tmem + (uint32_t)(gs & 1) * 128u, make_desc(a0 + off, kq_hi), make_desc(b0 + off, kq_hi),
                   idesc_qk, kk > 0 ? 1u : 0u);
          if (kk == D / 32) p_there = ask(C::kPFull + (gv & 1), (uint32_t)(gv >> 1) & 1u);
        }
        mma_commit_l(lead, bar(C::kSFull + (gs & 1)));
        if (cs.last()) mma_commit_l(lead, bar(C::kQFree + st));
        const int slot = rk.slot;
        ++gs;
        if (cs.next(p, pass)) {
          mma_commit_l(lead, bar(C::kEmpty + slot));
          rk.next();
          rk.next();
        }
        return true;
      };
      auto issue_pv = [&]() -> bool {  // O += P V
        const int st = PAIR ? cv.st : 0, o = accumulator(st);
        const int valid = min(kTileN, cv.w.keys - cv.j * kTileN);
        const int steps = (valid + 15) >> 4;  // 16 keys each
        if (st == 0) {
          if (!wait_warp(C::kFull + rv.slot, rv.parity, 3)) return false;
          if (valid & 15) {
            // keys past the sequence's end may hold anything, and 0 * NaN is
            // NaN: the values of the last step's are zeroed (later steps are
            // left out)
            uint8_t* v = base + C::kRingOff + rv.slot * C::kTileBytes;
            const int n = (16 * steps - valid) * 8;  // 16-byte pieces a box
            for (int i = lane; i < n * C::kBoxes; i += 32) {
              const int bx = i >= n ? 1 : 0, k = i - bx * n;
              *reinterpret_cast<uint4*>(v + bx * C::kBoxBytes + (valid + (k >> 3)) * 128 + (k & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        // the first product of a query tile overwrites what the accumulator held
        if (cv.j == 0 && uses(o) > 0 && !wait_warp(C::kORead + o, (uint32_t)(uses(o) - 1) & 1u, 4)) return false;
        if (!p_there && !wait_warp(C::kPFull + (gv & 1), (uint32_t)(gv >> 1) & 1u, 5)) return false;
        p_there = false;
        tc_fence_after();
        const uint32_t b0 = (uint32_t)dv + rv.slot * kStep, d0 = tmem + C::kTmemO + (uint32_t)o * D;
        const uint32_t a0 = tmem + (uint32_t)(gv & 1) * 128u;
        // P of keys 64 .. 127 starts 64 columns after that of the first 64
        auto product = [&](int kk) {
          mma_ts_l(lead, d0, a0 + (uint32_t)(kk >> 2) * 64u + (uint32_t)(kk & 3) * 8u,
                   make_desc(b0 + ((uint32_t)(kk * 16 * 128) >> 4), v_hi), idesc_pv, kk > 0 || cv.j > 0 ? 1u : 0u);
        };
        if (steps == 8) {
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            product(kk);
            if (kk == 4 && cs.more && cs.st == 0) k_there = ask(C::kFull + rk.slot, rk.parity);
          }
        } else {
#pragma unroll 1
          for (int kk = 0; kk < steps; ++kk) product(kk);
        }
        if (SPLIT || number > 0) mma_commit_l(lead, bar(C::kPVDone));
        if (cv.last()) {
          mma_commit_l(lead, bar(C::kODone + o));
          use(o);
        }
        const int slot = rv.slot;
        ++gv;
        if (cv.next(p, pass)) {
          mma_commit_l(lead, bar(C::kEmpty + slot));
          rv.next();
          rv.next();
        }
        return true;
      };
      while (ok && cv.more) {
        while (ok && cs.more && gs < gv + 2) {
          // a query tile that is not there yet does not hold up the products
          // of the one before
          if (cs.j == 0 && gs > gv && !ask(C::kQFull + (PAIR ? cs.st : 0), PAIR && cs.st ? q_parity[1] : q_parity[0]))
            break;
          ok = issue_s();
        }
        ok = ok && issue_pv();
      }
    } while (next_pass(number) && ok);
    if (!ok) {
      mma_commit_l(lead, bar(C::kDrain));
      if (lane == 0) wait_drain(bar(C::kDrain), 0, p.err_word);
    }
    __syncwarp();
  } else if (warp == 2) {
    // ------------------------------------------------------- the store of O
    int tile = 0;
    do {
      if (lane == 0 && !SPLIT) {
        Cursor<false> c;
        bool ok = true;
        for (c.start(p, pass); ok && c.more; c.skip(p, pass)) {
          for (int st = 0; st < c.w.streams; ++st, ++tile) {
            if (!(ok = wait(C::kOReady, (uint32_t)tile & 1u, 10) && !*abort_flag)) break;
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_store_4d(&p.o_map, base_u32 + C::kOOff + bx * C::kBoxBytes, bx * 64, c.w.hb * p.pack,
                           c.w.t0 + st * p.tile_tokens, c.w.b);
            tma_store_commit_and_wait_read();
            mbar_arrive(bar(C::kOFree));
          }
        }
        tma_store_wait_all();  // a later pass may write the same rows
      }
    } while (next_pass(number));
    __syncwarp();
  } else if (warp == 3) {
    // -------------------------------------------------------------------- Q
    int asked[2] = {0, 0};
    do {
      if (lane == 0) {
        const uint32_t bytes = (uint32_t)(C::kBoxes * p.pack * p.tile_tokens) * 128u;
        Cursor<false> c;
        bool ok = true;
        for (c.start(p, pass); ok && c.more; c.skip(p, pass)) {
#pragma unroll
          for (int st = 0; st < C::kStreams; ++st) {
            if (st >= c.w.streams) break;
            if (asked[st] > 0 && !(ok = wait(C::kQFree + st, (uint32_t)(asked[st] - 1) & 1u, 1))) break;
            ++asked[st];
            mbar_arrive_expect_tx(bar(C::kQFull + st), bytes);
#pragma unroll
            for (int bx = 0; bx < C::kBoxes; ++bx)
              tma_load_4d(base_u32 + C::kQOff + st * C::kTileBytes + bx * C::kBoxBytes, &p.q_map, bar(C::kQFull + st),
                          bx * 64, c.w.hb * p.pack, c.w.t0 + st * p.tile_tokens, c.w.b);
          }
        }
      }
    } while (next_pass(number));
    if (lane == 0 && *abort_flag)
      for (int st = 0; st < C::kStreams; ++st)
        if (asked[st] > 0) wait_drain(bar(C::kQFull + st), (uint32_t)(asked[st] - 1) & 1u, p.err_word);
    __syncwarp();
  } else if (warp < 12) {
    // -------------------------------------------------------------- softmax
    const int hf = (warp - 4) >> 2, quad = warp & 3;
    const int row = quad * 32 + lane;
    const uint32_t lane_off = (uint32_t)(quad * 32) << 16;
    const uint32_t tSh = tmem + lane_off + (uint32_t)hf * 64u;  // + buffer * 128
    const int warp_t = (quad * 32) / p.pack;  // first token of the warp's rows
    const float sl = p.scale_log2;
    int g = 0;
    bool ok = true;
    auto mask = [&](uint32_t (&sv)[32], int hi) {  // columns from hi on do not exist
      if (hi < 32) {
#pragma unroll
        for (int c = 0; c < 32; ++c) sv[c] = c < hi ? sv[c] : 0xff800000u;
      }
    };
    auto exps = [&](const uint32_t (&sv)[32], float m, float2& ps, uint32_t to) {
      const float2 sl2 = make_float2(sl, sl), m2 = make_float2(-m, -m);
      uint32_t pk[16];
#pragma unroll
      for (int c = 0; c < 16; ++c) {
        const float2 x = __ffma2_rn(make_float2(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1])), sl2, m2);
        const float e0 = ex2(x.x), e1 = ex2(x.y);
        ps = __fadd2_rn(ps, make_float2(e0, e1));
        pk[c] = pack_bf16(e0, e1);
      }
      tmem_st16(to, pk);
    };
    int done_before = -1;  // steps of the first pass, whose products PVDone does not count
    uint32_t pair_parity = 0;
    auto meet_pair = [&]() -> bool {  // the two warps of a quadrant
      arrive_warp(C::kPairMeet + quad);
      pair_parity ^= 1u;
      return wait_warp(C::kPairMeet + quad, pair_parity ^ 1u, 13);
    };
    do {
      const bool slow = SPLIT || number > 0;
      if (slow && done_before < 0) done_before = g;
      float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;
      Cursor<true> c;
      for (c.start(p, pass); c.more; c.next(p, pass), ++g) {
        const int st = PAIR ? c.st : 0, o = accumulator(st);
        if (!(ok = wait_warp(C::kSFull + (g & 1), (uint32_t)(g >> 1) & 1u, 6 + hf))) break;
        const int hi = c.w.keys - c.j * kTileN - hf * 64;          // visible columns of this half
        const bool busy = st * p.tile_tokens + warp_t < c.w.live;  // some row of the warp is live
        const uint32_t tS = tSh + (uint32_t)(g & 1) * 128u;
        float m_last = 0.f;
        if (!slow) {
          if (busy && hi > 0) {
            tc_fence_after();
            uint32_t s0[32], s1[32];
            tmem_ld32(tS, s0);
            tmem_wait_ld();
            tmem_ld32(tS + 32, s1);  // on its way while the first 32 are worked on
            float2 ps = make_float2(0.f, 0.f);
            mask(s0, hi);
            exps(s0, 0.f, ps, tS);
            tmem_wait_ld();
            mask(s1, hi - 32);
            exps(s1, 0.f, ps, tS + 16);
            if (st) l1 += ps.x + ps.y;
            else l0 += ps.x + ps.y;
            tmem_wait_st();
            tc_fence_before();
          }
        } else {
          // running maxima, the same for the row's two halves: they meet at
          // every step, in columns of the scores that P leaves free
          const uint32_t tX = tmem + lane_off + (uint32_t)(g & 1) * 128u + 32u;
          uint32_t s0[32], s1[32];
          float own = -INFINITY;
          tc_fence_after();
          tmem_ld32(tS, s0);
          tmem_ld32(tS + 32, s1);
          tmem_wait_ld();
          mask(s0, hi);
          mask(s1, hi - 32);
#pragma unroll
          for (int k = 0; k < 32; ++k) own = fmax3(own, __uint_as_float(s0[k]), __uint_as_float(s1[k]));
          tmem_st1(tX + (uint32_t)hf * 64u, __float_as_uint(own));
          tmem_wait_st();
          tc_fence_before();
          if (!(ok = meet_pair())) break;
          tc_fence_after();
          const float top = fmaxf(own, __uint_as_float(tmem_ld1(tX + (uint32_t)(1 - hf) * 64u))) * sl;
          const float m_old = st ? m1 : m0;
          float m_new = m_old, alpha = 1.f;
          if (c.j == 0) m_new = top > -INFINITY ? top : 0.f;
          else if (top > m_old + kRescale) m_new = top, alpha = ex2(m_old - top);
          if (c.j > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
            // S(g) is there, so PV(g - 2) is done; with one stream the last
            // product into this O is PV(g - 1): this phase or the last
            if (c.w.streams == 1 && !(ok = wait_warp(C::kPVDone, (uint32_t)(g - 1 - done_before) & 1u, 8))) break;
            tc_fence_after();
#pragma unroll 1
            for (int cc = 0; cc < D / 2; cc += 16) {  // half of the columns each
              uint32_t v[16];
              const uint32_t tO = tmem + lane_off + C::kTmemO + (uint32_t)(o * D + hf * (D / 2) + cc);
              tmem_ld16(tO, v);
              tmem_wait_ld();
#pragma unroll
              for (int k = 0; k < 16; ++k) v[k] = __float_as_uint(__uint_as_float(v[k]) * alpha);
              tmem_st16(tO, v);
            }
          }
          float2 ps = make_float2(0.f, 0.f);
          exps(s0, m_new, ps, tS);
          exps(s1, m_new, ps, tS + 16);
          float& l = st ? l1 : l0;
          l = l * alpha + (ps.x + ps.y);
          if (st) m1 = m_new;
          else m0 = m_new;
          m_last = m_new;
          if (c.last()) tmem_st1(tX + (uint32_t)hf * 64u + 1u, __float_as_uint(l));
          tmem_wait_st();
          tc_fence_before();
          if (!(ok = meet_pair())) break;  // both halves of O are rescaled, the maxima read
          if (c.last()) {                  // half 0 takes the sum, half 1 the maximum
            tc_fence_after();
            l = hf == 0 ? l + __uint_as_float(tmem_ld1(tX + 64u + 1u)) : m_last;
            tc_fence_before();
          }
        }
        arrive_warp(C::kPFull + (g & 1));
        if (c.last()) {
          // the sums of a query tile: two halves, or (running maxima) sum and maximum
          if (uses(o) > 0 && !(ok = wait_warp(C::kORead + o, (uint32_t)(uses(o) - 1) & 1u, 9))) break;
          reinterpret_cast<float*>(base + C::kSumOff)[(o * 2 + hf) * 128 + row] = st ? l1 : l0;
          arrive_warp(C::kLReady + o);
          use(o);
          if (st) l1 = 0.f;
          else l0 = 0.f;
        }
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
    // zeros and -inf for a query tile without a query or without a key
    auto clear = [&](const Work& w, int t0) {
      const int t = t0 + row_t, head = w.hb * p.pack + row_g;
      if (row_t < p.tile_tokens && t < p.Lq) {
        uint16_t* o = p.O + w.b * p.o_batch + t * p.o_token + head * D;
#pragma unroll
        for (int i = 0; i < D / 8; ++i) reinterpret_cast<uint4*>(o)[i] = make_uint4(0u, 0u, 0u, 0u);
        if (p.LSE != nullptr) p.LSE[((long long)w.b * p.H + head) * p.Lq + t] = -INFINITY;
      }
    };
    auto finish = [&](const Work& w, unsigned item, int st) -> bool {
      const int o = accumulator(st);
      const int t = w.t0 + st * p.tile_tokens + row_t;
      const bool stored = row_t < p.tile_tokens && t < p.Lq;  // this row has an O and an LSE
      const bool live = row_t < p.tile_tokens && st * p.tile_tokens + row_t < w.live;
      const long long lse_at = ((long long)w.b * p.H + w.hb * p.pack + row_g) * p.Lq + t;
      const uint32_t tO = tmem + lane_off + C::kTmemO + (uint32_t)(o * D);
      if constexpr (!SPLIT) {
        if (!wait_warp(C::kLReady + o, (uint32_t)uses(o) & 1u, 12)) return false;
        const float a = sums[(o * 2) * 128 + row], b = sums[(o * 2 + 1) * 128 + row];
        const float m = number > 0 ? b : 0.f, l = number > 0 ? a : a + b;
        const bool on = live && l != 0.f;  // a sum of 0 has no say; NaN has
        const float inv = on ? 1.f / l : 0.f;
        if (!wait_warp(C::kODone + o, (uint32_t)uses(o) & 1u, 9)) return false;
        tc_fence_after();
        if (tiles > 0 && !wait_warp(C::kOFree, (uint32_t)(tiles - 1) & 1u, 11)) return false;
        use(o);
        float2 sound = make_float2(0.f, 0.f);  // stays 0 unless some value is not finite
#pragma unroll
        for (int cc = 0; cc < D; cc += 32) {
          uint32_t v[32];
          tmem_ld32(tO + cc, v);
          tmem_wait_ld();
          if (cc + 32 == D) {
            tc_fence_before();
            arrive_warp(C::kORead + o);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            uint32_t w4[4];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int k = 8 * i + 2 * c;
              const float2 x = on ? __fmul2_rn(make_float2(__uint_as_float(v[k]), __uint_as_float(v[k + 1])),
                                               make_float2(inv, inv))
                                  : make_float2(0.f, 0.f);
              sound = __ffma2_rn(x, make_float2(0.f, 0.f), sound);
              w4[c] = pack_bf16(x.x, x.y);
            }
            const int k = cc / 8 + i;
            *reinterpret_cast<uint4*>(stage + (k >> 3) * C::kBoxBytes + row * 128 + (((k & 7) ^ (row & 7)) << 4)) =
                make_uint4(w4[0], w4[1], w4[2], w4[3]);
          }
        }
        const bool again =
            number == 0 && live && !(l >= kLeastSum && l <= kMostSum && sound.x == 0.f && sound.y == 0.f);
        if (again && atomicMax(&misc[4], (uint32_t)tiles) < (uint32_t)tiles) {  // the tile's first such row
          const uint32_t n = atomicAdd(&misc[2], 1u);
          if (n < kRedoList) list[n] = tile_of(p, item, st, pass.pair);
          else atomicMin(&misc[3], item);
        }
        fence_proxy_async_smem();
        arrive_warp(C::kOReady);
        if (stored && p.LSE != nullptr) p.LSE[lse_at] = on ? (m + __log2f(l)) * kLn2 : -INFINITY;
      } else {
        // ------------------------- the cluster's blocks join their key ranges
        // This block's (m, l) of every row where its cluster reads them; then
        // O, weighted, to the block that sums its columns (D / splits each).
        float m = -INFINITY, l = 0.f;
        if (w.nt > 0) {
          if (!wait_warp(C::kLReady, 0u, 12) || !wait_warp(C::kODone, 0u, 9)) return false;
          tc_fence_after();
          l = sums[row];
          m = sums[128 + row];
        }
        const bool on = live && l != 0.f;
        *reinterpret_cast<float2*>(stage + row * 8) = make_float2(on ? m : -INFINITY, *abort_flag ? -1.f : l);
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
        const float f = on ? ex2(m - top) / total : 0.f;
        const int per = D / p.splits;  // columns of a block's sum
#pragma unroll 1
        for (int cc = 0; cc < D; cc += 16) {
          uint32_t v[16];
          if (w.nt > 0) {
            tmem_ld16(tO + cc, v);
            tmem_wait_ld();
          }
          if (stored) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int col = cc + 4 * i, to = col / per;
              // what a block without keys left in TMEM is no number to count on
              st_dsmem_v4(mapa(base_u32 + C::kRingOff + (uint32_t)((split * 128 + row) * per + col - to * per) * 4u,
                               (uint32_t)to),
                          on ? __uint_as_float(v[4 * i]) * f : 0.f, on ? __uint_as_float(v[4 * i + 1]) * f : 0.f,
                          on ? __uint_as_float(v[4 * i + 2]) * f : 0.f, on ? __uint_as_float(v[4 * i + 3]) * f : 0.f);
            }
          }
          __syncwarp();
        }
        cluster_sync_all();
        if (stored && !bad) {
          const float* sum = reinterpret_cast<const float*>(base + C::kRingOff) + row * per;
          uint16_t* out = p.O + w.b * p.o_batch + t * p.o_token + (w.hb * p.pack + row_g) * D + split * per;
          for (int cc = 0; cc < per; cc += 4) {
            float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
            for (int c = 0; c < p.splits; ++c) {
              const float4 x = *reinterpret_cast<const float4*>(sum + c * 128 * per + cc);
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
      for (unsigned at = pass.first; ok && at < pass.end; at += pass.step) {
        const unsigned item = pass.list != nullptr ? (unsigned)uniform<true>((int)pass.list[at]) : at;
        const Work w = work_at<true>(p, item, split, pass.pair);
        if (!SPLIT) {
          if (w.nt == 0) clear(w, w.t0);
          if (pass.pair == 2 && (w.nt == 0 || w.streams == 1) && w.t0 + p.tile_tokens < p.Lq)
            clear(w, w.t0 + p.tile_tokens);
          if (w.nt == 0) continue;
        }
#pragma unroll 1
        for (int st = 0; ok && st < w.streams; ++st) ok = finish(w, item, st);
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

template <int D, bool PAIR, bool SPLIT>
cudaError_t launch_fwd(const CrossParams& p, int sms, cudaStream_t s) {
  using C = FwdCfg<D, PAIR>;
  static bool attr_set = false;
  if (!attr_set) {
    cudaError_t e = cudaFuncSetAttribute(cross_fwd_kernel<D, PAIR, SPLIT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)C::kSmemBytes);
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
  return cudaLaunchKernelEx(&cfg, cross_fwd_kernel<D, PAIR, SPLIT>, p);
}

}  // namespace

cudaError_t launch_cross_forward(const CrossParams& p, int sms, cudaStream_t s) {
  if (p.splits > 1) return p.D == 128 ? launch_fwd<128, false, true>(p, sms, s) : launch_fwd<64, false, true>(p, sms, s);
  if (p.pair == 2) return p.D == 128 ? launch_fwd<128, true, false>(p, sms, s) : launch_fwd<64, true, false>(p, sms, s);
  return p.D == 128 ? launch_fwd<128, false, false>(p, sms, s) : launch_fwd<64, false, false>(p, sms, s);
}

}  // namespace sab
