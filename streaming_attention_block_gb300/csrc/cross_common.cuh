// What the cross-attention kernels share: bounded waits, ring places, lengths.
#pragma once

#include "ptx.cuh"
#include "sab_internal.h"

namespace sab {
namespace {

using namespace ptx;

constexpr uint64_t kTimeoutNs = 2000000000ull;

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
  return __builtin_expect(mbar_try_wait(bar, parity), 1) || wait_slow(bar, parity, abort_flag, site, err_word);
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

// Zero the rows [from, to) of a tile in shared memory (whole warp).
template <int BOXES, int BOX_BYTES = 128 * 128>
__device__ __noinline__ void zero_rows(uint8_t* tile, int from, int to) {
  const int lane = threadIdx.x & 31, n = (to - from) * 8;  // 16-byte pieces a box of 64 columns
  for (int i = lane; i < n * BOXES; i += 32) {
    const int bx = i >= n ? 1 : 0, k = i - bx * n;
    *reinterpret_cast<uint4*>(tile + bx * BOX_BYTES + (from + (k >> 3)) * 128 + (k & 7) * 16) =
        make_uint4(0u, 0u, 0u, 0u);
  }
  fence_proxy_async_smem();
  __syncwarp();
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

// Where an item is: its query tiles, head block and sequence.
struct Spot {
  int iq, hb, b;
};
__device__ __noinline__ Spot spot_of(const CrossParams& p, unsigned item, int pair) {
  const unsigned n = (unsigned)(p.n_qtiles + pair - 1) / (unsigned)pair;
  const unsigned r = item / n;
  Spot s;
  s.iq = (int)(item - r * n);
  s.b = (int)(r / (unsigned)p.head_blocks);
  s.hb = (int)(r - (unsigned)s.b * (unsigned)p.head_blocks);
  return s;
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
__device__ __forceinline__ Work work_at(const CrossParams& p, const Spot& s, int split, int pair) {
  Work w;
  w.t0 = s.iq * pair * p.tile_tokens;
  w.b = s.b;
  w.hb = s.hb;
  w.live = length_of<kUniform>(p.q_len, w.b, p.Lq) - w.t0;
  w.streams = pair == 2 && w.live > p.tile_tokens ? 2 : 1;
  const int kl = w.live > 0 ? length_of<kUniform>(p.kv_len, p.Bk == 1 ? 0 : w.b, p.Lk) : 0;
  const int total = (kl + kTileN - 1) / kTileN;
  int last = total;
  w.first = 0;
  if (p.splits > 1) {
    w.first = (int)((long long)total * split / p.splits);
    last = (int)((long long)total * (split + 1) / p.splits);
  }
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

// Coordinates of a query tile in its maps: head and token, or (one head a tile)
// token and head.  The copy engine takes a plane of the first two axes at a
// time: 128 planes of one row each took 3500 cycles a tile, one plane 1500.
__device__ __forceinline__ int query_c1(const CrossParams& p, const Work& w, int t) {
  return p.pack == 1 ? w.t0 + t * p.tile_tokens : w.hb * p.pack;
}
__device__ __forceinline__ int query_c2(const CrossParams& p, const Work& w, int t) {
  return p.pack == 1 ? w.hb : w.t0 + t * p.tile_tokens;
}

// What a block works through.  Pass 0: every step-th item.  Pass 1: the query
// tiles of the list, one by one.  Pass 2: the items of pass 0 from the one on at
// which the list was full.
struct Pass {
  unsigned first, step, end;  // items, or places of the list
  const uint32_t* list;       // or null
  int pair, split;
  Spot by;                    // `step` items on
};
// The items of a pass in order.  Every role walks them by itself, by additions:
// the divisions that find an item's place took 2000 cycles between two items.
template <bool kUniform>
struct Walk {
  unsigned at;
  Spot spot;
  Work w;
  __device__ __forceinline__ unsigned item(const Pass& a) const {
    return a.list != nullptr ? (unsigned)uniform<kUniform>((int)a.list[at]) : at;
  }
  __device__ __forceinline__ void start(const CrossParams& p, const Pass& a) {
    at = a.first;
    if (at < a.end) place(p, a, spot_of(p, item(a), a.pair));
  }
  __device__ __forceinline__ void place(const CrossParams& p, const Pass& a, const Spot& s) {
    spot = s;
    w = work_at<kUniform>(p, spot, a.split, a.pair);
  }
  __device__ __forceinline__ bool more(const Pass& a) const { return at < a.end; }
  __device__ __forceinline__ void next(const CrossParams& p, const Pass& a) {
    at += a.step;
    if (at >= a.end) return;
    if (__builtin_expect(a.list != nullptr, 0)) {
      place(p, a, spot_of(p, item(a), a.pair));
      return;
    }
    const int n = (p.n_qtiles + a.pair - 1) >> (a.pair - 1);
    Spot s = {spot.iq + a.by.iq, spot.hb + a.by.hb, spot.b + a.by.b};
    if (s.iq >= n) s.iq -= n, ++s.hb;
    if (s.hb >= p.head_blocks) s.hb -= p.head_blocks, ++s.b;
    place(p, a, s);
  }
  // the next one that has keys
  __device__ __forceinline__ void seek(const CrossParams& p, const Pass& a) {
    while (more(a) && w.nt == 0) next(p, a);
  }
};

}  // namespace
}  // namespace sab
