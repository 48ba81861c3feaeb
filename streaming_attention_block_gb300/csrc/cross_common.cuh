// What the cross-attention kernels share: bounded waits, ring places, lengths,
// the order of the work.
#pragma once

#include <atomic>

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
template <int BOXES>
__device__ __noinline__ void zero_rows(uint8_t* tile, int from, int to) {
  const int lane = threadIdx.x & 31, n = (to - from) * 8;  // 16-byte pieces a box of 64 columns
  for (int i = lane; i < n * BOXES; i += 32) {
    const int bx = i >= n ? 1 : 0, k = i - bx * n;
    *reinterpret_cast<uint4*>(tile + bx * 128 * 128 + (from + (k >> 3)) * 128 + (k & 7) * 16) =
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
  return lens == nullptr ? most : uniform<kUniform>(min(max(ld_global(lens + b), 0), most));
}

// A kernel's shared memory limit, set once for each device.
template <typename K>
cudaError_t allow_smem(K* kernel, size_t bytes, std::atomic<unsigned long long>& ready) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev <= 63 && (ready.load() >> dev & 1))) return e;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
  if (e == cudaSuccess && dev <= 63) ready.fetch_or(1ull << dev);
  return e;
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
// Items in the order of their key tiles, the most first, where lengths differ: a
// block's items are every so many of them, so that in the order of the sequences
// some blocks met the long ones and some the empty.  Means of five draws of
// lengths, in the order of the sequences and in this one: 8 x 1023 queries over 777
// keys, 24/4 heads of 64, 40.5 and 30.6 us; 64 x 1 over 4095, 24/8 heads of 128,
// 103.8 and 95.4 us.  Up to 64 sequences, which is what the table holds; more are
// taken as they come, which costs 13 to 19 % forward and 9 to 22 % in the gradients
// (65 to 128 x up to 512 over up to 777 keys against 64 of them), and 30, 14 and 5 %
// for 65, 80 and 128 x 1 over up to 4095, 24/4 heads of 64.
//
// seqs[i]: number of the first item of the i-th sequence in that order << 6 | the
// sequence; seqs[B]: all items << 6.  For all threads of a block; scratch: 128
// words.
constexpr int kMaxSorted = 64;
__device__ __noinline__ void sort_sequences(const CrossParams& p, int pair, uint32_t* seqs, uint32_t* scratch) {
  const int t = threadIdx.x;
  int nt = 0, tiles = 0;
  if (t < p.B) {
    const int ql = length_of<false>(p.q_len, t, p.Lq), kl = length_of<false>(p.kv_len, p.Bk == 1 ? 0 : t, p.Lk);
    if (ql > 0 && kl > 0) {
      nt = (kl + kTileN - 1) / kTileN;
      tiles = (ql + pair * p.tile_tokens - 1) / (pair * p.tile_tokens);
    }
  }
  if (t < kMaxSorted) {
    scratch[t] = (uint32_t)nt;
    scratch[kMaxSorted + t] = (uint32_t)tiles;
  }
  __syncthreads();
  if (t < p.B) {
    int rank = 0;
    uint32_t before = 0;
    auto count = [&](int u, uint32_t other, uint32_t its) {
      if ((int)other > nt || ((int)other == nt && u < t)) ++rank, before += its;
    };
#pragma unroll 2
    for (int u = 0; u < p.B; u += 4) {
      const uint4 a = *reinterpret_cast<const uint4*>(scratch + u);
      const uint4 c = *reinterpret_cast<const uint4*>(scratch + kMaxSorted + u);
      count(u, a.x, c.x);
      count(u + 1, a.y, c.y);
      count(u + 2, a.z, c.z);
      count(u + 3, a.w, c.w);
    }
    seqs[rank] = (before * (uint32_t)p.head_blocks) << 6 | (uint32_t)t;
    if (rank == p.B - 1) seqs[p.B] = ((before + (uint32_t)tiles) * (uint32_t)p.head_blocks) << 6;
  }
  __syncthreads();
}
// The item of a place of a block's walk, whose every other round of gridDim.x
// items goes backwards: who has the longest of one has the shortest of the next.
// b < 0: there is none (the last round is not full).
__device__ __noinline__ Spot sorted_spot(const CrossParams& p, const uint32_t* seqs, unsigned at) {
  const unsigned round = at / gridDim.x, by = at - round * gridDim.x;
  const unsigned item = round & 1u ? at - by + (gridDim.x - 1u - by) : at;
  if (item >= seqs[p.B] >> 6) return Spot{0, 0, -1};
  int lo = 0, hi = p.B;  // the last sequence that begins at the item or before it
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if ((seqs[mid] >> 6) <= item) lo = mid;
    else hi = mid;
  }
  const unsigned start = seqs[lo] >> 6, per = ((seqs[lo + 1] >> 6) - start) / (unsigned)p.head_blocks;
  Spot s;
  s.hb = (int)((item - start) / per);
  s.iq = (int)(item - start - (unsigned)s.hb * per);
  s.b = (int)(seqs[lo] & 63u);
  return s;
}

// One or two query tiles (`streams`) of `pack` heads from head hb * pack on,
// tile_tokens tokens each from t0 on, and the key tiles [first, first + nt).
struct Work {
  int b, hb, t0;    // b < 0: an index that a debug build has refused
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
  w.live = 0;
  w.streams = 1;
  w.first = w.nt = w.keys = 0;
  // (a refused item has nothing, and its rows are not taken for dead ones)
  if constexpr (kDebugBounds) {
    if ((unsigned)w.b >= (unsigned)p.B || (unsigned)w.hb >= (unsigned)p.head_blocks ||
        (unsigned)w.t0 >= (unsigned)p.Lq) {
      if (p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
      w.b = -1;
      return w;
    }
  }
  w.live = length_of<kUniform>(p.q_len, w.b, p.Lq) - w.t0;
  w.streams = pair == 2 && w.live > p.tile_tokens ? 2 : 1;
  const int kl = w.live > 0 ? length_of<kUniform>(p.kv_len, p.Bk == 1 ? 0 : w.b, p.Lk) : 0;
  const int total = (kl + kTileN - 1) / kTileN;
  int last = total;
  if (p.splits > 1) {
    w.first = (int)((long long)total * split / p.splits);
    last = (int)((long long)total * (split + 1) / p.splits);
  }
  w.nt = last - w.first;
  w.keys = min(kl, last * kTileN) - w.first * kTileN;
  if constexpr (kDebugBounds) {
    if (w.first < 0 || last * kTileN - kTileN >= p.Lk) {
      if (p.err_word != nullptr) atomicOr(p.err_word, kErrBoundsBit);
      w.nt = w.live = 0;
      w.b = -1;
    }
  }
  return w;
}

// Zeros for the rows of the block's share of query tiles without a query or
// without a key: from `zeros`, a tile in shared memory that holds them, through
// the copy engine (stores of 16 bytes a row took longer than the products of a
// full tile: 8 x 2000 x 777 tokens, 12 heads of 128, half of the queries padding:
// 55 us against 47 without padding).  lse: -inf for them, or null.  Whole warp.
template <int BOXES>
__device__ __noinline__ void clear_tiles(const CrossParams& p, int pair, uint32_t zeros, float* lse) {
  const int lane = threadIdx.x & 31;
  for (unsigned i = blockIdx.x; i < p.items; i += gridDim.x) {
    const Work w = work_at<false>(p, spot_of(p, i, pair), 0, pair);
    if (kDebugBounds && w.b < 0) continue;
    for (int t = w.nt == 0 ? 0 : w.streams; t < pair; ++t) {
      const int t0 = w.t0 + t * p.tile_tokens;
      if (t0 >= p.Lq) break;
      if (lane == 0) {
        for (int bx = 0; bx < BOXES; ++bx)
          tma_store_4d(&p.o_map, zeros + bx * 128u * 128u, bx * 64, p.pack == 1 ? t0 : w.hb * p.pack,
                       p.pack == 1 ? w.hb : t0, w.b);
      }
      const int tokens = min(p.tile_tokens, p.Lq - t0);
      for (int g = 0; lse != nullptr && g < p.pack; ++g)
        for (int k = lane; k < tokens; k += 32)
          lse[((long long)w.b * p.H + w.hb * p.pack + g) * p.Lq + t0 + k] = -INFINITY;
    }
  }
  if (lane == 0) tma_store_commit_and_wait_read();
  __syncwarp();
}
// Such a tile (whole warp).
__device__ __noinline__ void fill_zeros(uint8_t* tile, int bytes) {
  for (int i = (threadIdx.x & 31) * 16; i < bytes; i += 512)
    *reinterpret_cast<uint4*>(tile + i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Coordinates of a query tile in its maps: head and token, or (one head a tile)
// token and head.
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
  const uint32_t* seqs;       // sorted sequences, or null
  int pair, split;
  Spot by;                    // `step` items on
};
// The items of a pass in order.  Every role walks them by itself, by additions
// where their order is that of the tiles.
template <bool kUniform, bool kRagged>
struct Walk {
  unsigned at;
  Spot spot;
  Work w;
  __device__ __forceinline__ unsigned item(const Pass& a) const {
    return a.list != nullptr ? (unsigned)uniform<kUniform>((int)a.list[at]) : at;
  }
  __device__ __forceinline__ void start(const CrossParams& p, const Pass& a) {
    at = a.first;
    if (at < a.end) place(p, a, find(p, a));
  }
  __device__ __forceinline__ Spot find(const CrossParams& p, const Pass& a) const {
    if (!kRagged || a.list != nullptr || a.seqs == nullptr) return spot_of(p, item(a), a.pair);
    Spot s = sorted_spot(p, a.seqs, at);
    s.iq = uniform<kUniform>(s.iq);
    s.hb = uniform<kUniform>(s.hb);
    s.b = uniform<kUniform>(s.b);
    return s;
  }
  __device__ __forceinline__ void place(const CrossParams& p, const Pass& a, const Spot& s) {
    spot = s;
    if (kRagged && s.b < 0) {
      w.nt = w.live = 0;
      return;
    }
    w = work_at<kUniform>(p, spot, a.split, a.pair);
  }
  __device__ __forceinline__ bool more(const Pass& a) const { return at < a.end; }
  __device__ __forceinline__ void next(const CrossParams& p, const Pass& a) {
    at += a.step;
    if (at >= a.end) return;
    if ((kRagged && a.seqs != nullptr) || __builtin_expect(a.list != nullptr, 0)) {
      place(p, a, find(p, a));
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
