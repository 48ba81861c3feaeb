// Host side of libsab.so: ring handle, argument validation, key-set planner,
// TMA tensor-map encoding and kernel launches.  No call allocates device
// memory or synchronises the host (except sab_get_last_device_error).
#include <cuda.h>
#include <cuda_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include <algorithm>
#include <atomic>
#include <new>
#include <vector>

#include "../../include/sab.h"
#include "sab_internal.h"

using namespace sab;

namespace {

constexpr size_t kAlign = 256;
constexpr unsigned kRotaryMagic = 0x53524f54u;  // a plan that sab_rotary_plan_init filled

// Debug builds: the kind of launch whose next instance carries a forged index
// (sab_debug_inject_bounds_error); 0 when none is pending.
std::atomic<int> g_inject{0};
bool take_injection(int what) {
  if (!kDebugBounds) return false;
  int expect = what;
  return g_inject.compare_exchange_strong(expect, 0);
}
size_t align_up(size_t x, size_t a) { return (x + a - 1) / a * a; }
bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

typedef CUresult (*EncodeTiledFn)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                  const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                  CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                  CUtensorMapFloatOOBfill);

EncodeTiledFn encode_fn() {
  static EncodeTiledFn fn = nullptr;
  if (fn == nullptr) {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) ==
            cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<EncodeTiledFn>(p);
  }
  return fn;
}

// 4-D bf16 map with coordinates (d, row, h, b) and a 64 x 128 box, 128-byte swizzle.
bool encode_map(CUtensorMap* m, const void* ptr, int D, long long rows, int H, int B, size_t s_row,
                size_t s_h, size_t s_b, int box_rows = kTileN) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)s_row, (cuuint64_t)s_h, (cuuint64_t)s_b};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Head-major [B, H, rows, D] E4M3 codes: plain (unswizzled) 128-row boxes of
// whole D-byte rows, expanded to bf16 inside the attention kernel.
bool encode_head_major_u8(CUtensorMap* m, const void* ptr, int B, int H, long long rows, int D,
                          bool swizzle128 = false) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)rows, (cuuint64_t)H, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)D, (cuuint64_t)rows * D, (cuuint64_t)H * rows * D};
  const cuuint32_t box[4] = {(cuuint32_t)D, (cuuint32_t)kTileN, 1, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void*>(ptr), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_NONE,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// Token-major [B, L, H, D] bf16.
bool encode_token_major(CUtensorMap* m, const void* ptr, int B, int L, int H, int D, int box_rows = kTileN) {
  const size_t e = 2;
  return encode_map(m, ptr, D, L, H, B, (size_t)H * D * e, (size_t)D * e, (size_t)L * H * D * e, box_rows);
}

// Head-major [B, H, rows, D] bf16.
bool encode_head_major(CUtensorMap* m, const void* ptr, int B, int H, long long rows, int D) {
  const size_t e = 2;
  return encode_map(m, ptr, D, rows, H, B, (size_t)D * e, (size_t)rows * D * e, (size_t)H * rows * D * e);
}

bool valid_desc(const sab_ring_desc* d) {
  if (d == nullptr) return false;
  if (d->num_layers < 1 || d->batch < 1 || d->heads < 1 || d->chunk_tokens < 1 || d->ring_slots < 1)
    return false;
  if (d->head_dim != 64 && d->head_dim != 128) return false;
  if (d->has_sink != 0 && d->has_sink != 1) return false;
  if (d->kv_dtype != SAB_KV_BF16 && d->kv_dtype != SAB_KV_FP8_E4M3 && d->kv_dtype != SAB_KV_INT8K_FP8V)
    return false;
  const long long rows = (long long)(d->has_sink + d->ring_slots) * d->chunk_tokens;
  if (rows > (1LL << 30)) return false;
  if ((long long)d->batch * d->heads * rows * d->head_dim > (1LL << 40)) return false;
  return true;
}

struct Geometry {
  long long rows;       // rows per (b, h)
  size_t codes_bytes;   // one tensor (K or V) of one layer, aligned
  size_t scale_bytes;   // one tensor's scales of one layer, aligned (FP8)
  size_t layer_bytes;
};

Geometry geometry(const sab_ring_desc& d) {
  Geometry g;
  g.rows = (long long)(d.has_sink + d.ring_slots) * d.chunk_tokens;
  const size_t esize = d.kv_dtype == SAB_KV_BF16 ? 2 : 1;
  g.codes_bytes = align_up((size_t)d.batch * d.heads * g.rows * d.head_dim * esize, kAlign);
  g.scale_bytes = d.kv_dtype != SAB_KV_BF16
                      ? align_up((size_t)d.batch * d.heads * (d.has_sink + d.ring_slots) * sizeof(float), kAlign)
                      : 0;
  g.layer_bytes = 2 * g.codes_bytes + 2 * g.scale_bytes;
  return g;
}

// Split workspace: one arrival counter per (b, h, query tile), then the
// fp32 partial rows [S][B*H][n_qtiles*128][D] and partial LSEs [S][B*H][n_qtiles*128].
struct WsLayout {
  size_t count_off, o_off, lse_off, total;
};
WsLayout ws_layout(int BH, int Lq, int D, int splits) {
  WsLayout w{0, 0, 0, 0};
  if (splits <= 1) return w;
  const size_t n_qtiles = (size_t)(Lq + kTileM - 1) / kTileM;
  const size_t lq_pad = n_qtiles * kTileM;
  w.count_off = 0;
  w.o_off = align_up((size_t)BH * n_qtiles * sizeof(unsigned), kAlign);
  w.lse_off = w.o_off + align_up((size_t)splits * BH * lq_pad * D * sizeof(float), kAlign);
  w.total = w.lse_off + align_up((size_t)splits * BH * lq_pad * sizeof(float), kAlign);
  return w;
}

constexpr int kMaxSplits = 256;
constexpr int kMaxAutoSplits = 8;

int device_sms() {
  static int n = 0;
  if (n == 0) {
    int dev = 0, v = 0;
    if (cudaGetDevice(&dev) == cudaSuccess &&
        cudaDeviceGetAttribute(&v, cudaDevAttrMultiProcessorCount, dev) == cudaSuccess && v > 0)
      n = v;
    else
      return 148;
  }
  return n;
}

// num_splits == 0: the KV split count S (1..8) that minimises the modelled
// time of one call, in key-tile periods.  CTAs (one query tile x one split)
// run one per SM, so the call takes ceil(tiles * S / SMs) waves of
// ceil(kv_tiles / S) key tiles each; every wave after the first also pays a
// CTA's set-up and epilogue (about 5 key tiles: the first wave's overlaps the
// previous kernel), and S > 1 adds the partial-tile write and the merge (about
// 1 + 0.4 S key tiles).
int auto_splits(long long q_tiles, int kv_tiles) {
  const long long sms = device_sms();
  int best = 1;
  double best_cost = 0.0;
  for (int s = 1; s <= kMaxAutoSplits && (s == 1 || s <= kv_tiles / 2); ++s) {
    const long long waves = (q_tiles * s + sms - 1) / sms;
    double cost = (double)waves * ((kv_tiles + s - 1) / s) + 5.0 * (double)(waves - 1);
    if (s > 1) cost += 1.0 + 0.4 * s;
    if (s == 1 || cost < best_cost) {
      best_cost = cost;
      best = s;
    }
  }
  return best;
}

}  // namespace

struct sab_ring {
  sab_ring_desc d;
  uint8_t* mem;
  Geometry g;
  std::vector<long long> newest;
  std::vector<int> held;
  std::vector<int> sink_set;
  std::vector<CUtensorMap> kmap, vmap;  // per layer, BF16 rings

  uint8_t* layer_base(int l) const { return mem + (size_t)l * g.layer_bytes; }
  void* k(int l) const { return layer_base(l); }
  void* v(int l) const { return layer_base(l) + g.codes_bytes; }
  float* ks(int l) const {
    return g.scale_bytes ? reinterpret_cast<float*>(layer_base(l) + 2 * g.codes_bytes) : nullptr;
  }
  float* vs(int l) const {
    return g.scale_bytes ? reinterpret_cast<float*>(layer_base(l) + 2 * g.codes_bytes + g.scale_bytes) : nullptr;
  }
};

extern "C" {

size_t sab_kv_ring_bytes(const sab_ring_desc* desc) {
  if (!valid_desc(desc)) return 0;
  return geometry(*desc).layer_bytes * (size_t)desc->num_layers;
}

sab_status sab_kv_ring_create(const sab_ring_desc* desc, void* dev_mem, size_t bytes, void* stream,
                              sab_ring** out) {
  if (out == nullptr || !valid_desc(desc) || dev_mem == nullptr) return SAB_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(dev_mem) % kAlign) != 0) return SAB_ERR_INVALID_ARG;
  const size_t need = sab_kv_ring_bytes(desc);
  if (bytes < need) return SAB_ERR_INVALID_ARG;
  sab_ring* r = new (std::nothrow) sab_ring();
  if (r == nullptr) return SAB_ERR_INVALID_ARG;
  r->d = *desc;
  r->mem = static_cast<uint8_t*>(dev_mem);
  r->g = geometry(*desc);
  r->newest.assign(desc->num_layers, -1);
  r->held.assign(desc->num_layers, 0);
  r->sink_set.assign(desc->num_layers, 0);
  r->kmap.resize(desc->num_layers);
  r->vmap.resize(desc->num_layers);
  const bool fp8 = desc->kv_dtype != SAB_KV_BF16;  // one byte per element
  for (int l = 0; l < desc->num_layers; ++l) {
    const int B = desc->batch, H = desc->heads, D = desc->head_dim;
    const bool okm = fp8 ? (encode_head_major_u8(&r->kmap[l], r->k(l), B, H, r->g.rows, D) &&
                            encode_head_major_u8(&r->vmap[l], r->v(l), B, H, r->g.rows, D))
                         : (encode_head_major(&r->kmap[l], r->k(l), B, H, r->g.rows, D) &&
                            encode_head_major(&r->vmap[l], r->v(l), B, H, r->g.rows, D));
    if (!okm) {
      delete r;
      return SAB_ERR_CUDA;
    }
  }
  if (cudaMemsetAsync(dev_mem, 0, need, static_cast<cudaStream_t>(stream)) != cudaSuccess) {
    delete r;
    return SAB_ERR_CUDA;
  }
  *out = r;
  return SAB_OK;
}

sab_status sab_kv_ring_destroy(sab_ring* ring) {
  delete ring;
  return SAB_OK;
}

sab_status sab_kv_ring_get_desc(const sab_ring* ring, sab_ring_desc* desc) {
  if (ring == nullptr || desc == nullptr) return SAB_ERR_INVALID_ARG;
  *desc = ring->d;
  return SAB_OK;
}

sab_status sab_kv_ring_layer_ptrs(const sab_ring* ring, int layer, void** k, void** v, float** k_scale,
                                  float** v_scale) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  if (k) *k = ring->k(layer);
  if (v) *v = ring->v(layer);
  if (k_scale) *k_scale = ring->ks(layer);
  if (v_scale) *v_scale = ring->vs(layer);
  return SAB_OK;
}

static sab_status write_chunk(sab_ring* r, int layer, int slot_row0, int scale_idx, const void* K, const void* V,
                              void* stream, const long long* d_chunk = nullptr) {
  AppendParams p;
  memset(&p, 0, sizeof(p));
  p.src[0] = static_cast<const uint16_t*>(K);
  p.src[1] = static_cast<const uint16_t*>(V);
  p.dst[0] = r->k(layer);
  p.dst[1] = r->v(layer);
  p.scale[0] = r->ks(layer);
  p.scale[1] = r->vs(layer);
  p.B = r->d.batch;
  p.H = r->d.heads;
  p.D = r->d.head_dim;
  p.Lc = r->d.chunk_tokens;
  p.rows = (int)r->g.rows;
  p.slot_row0 = slot_row0;
  p.scale_idx = scale_idx;
  p.scale_stride = r->d.has_sink + r->d.ring_slots;
  p.k_int8 = r->d.kv_dtype == SAB_KV_INT8K_FP8V ? 1 : 0;
  p.d_chunk = d_chunk;
  p.ring_slots = r->d.ring_slots;
  p.has_sink = r->d.has_sink;
  p.err_word = device_error_word();
  if (d_chunk == nullptr && take_injection(SAB_DEBUG_INJECT_APPEND_SLOT)) {
    p.slot_row0 = p.rows;  // one slot past the (b, h) block
    p.scale_idx = p.scale_stride;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  const cudaError_t e = r->d.kv_dtype == SAB_KV_BF16 ? launch_append_bf16(p, s) : launch_append_fp8(p, s);
  return e == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

sab_status sab_kv_ring_set_sink(sab_ring* ring, int layer, const void* K, const void* V, void* stream) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr || !aligned16(K) || !aligned16(V)) return SAB_ERR_INVALID_ARG;
  if (!ring->d.has_sink) return SAB_ERR_UNSUPPORTED;
  const sab_status st = write_chunk(ring, layer, 0, 0, K, V, stream);
  if (st == SAB_OK) ring->sink_set[layer] = 1;
  return st;
}

sab_status sab_kv_ring_append(sab_ring* ring, int layer, long long chunk, const void* K, const void* V,
                              void* stream) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr || !aligned16(K) || !aligned16(V)) return SAB_ERR_INVALID_ARG;
  if (chunk < 0) return SAB_ERR_OUT_OF_RANGE;
  const long long newest = ring->newest[layer];
  if (newest >= 0 && chunk != newest && chunk != newest + 1) return SAB_ERR_OUT_OF_RANGE;
  const int R = ring->d.ring_slots;
  const int slot = (int)(chunk % R);
  const int row0 = (ring->d.has_sink + slot) * ring->d.chunk_tokens;
  const sab_status st = write_chunk(ring, layer, row0, ring->d.has_sink + slot, K, V, stream);
  if (st != SAB_OK) return st;
  if (newest < 0) {
    ring->held[layer] = 1;
  } else if (chunk == newest + 1) {
    ring->held[layer] = std::min(R, ring->held[layer] + 1);
  }
  ring->newest[layer] = chunk;
  return SAB_OK;
}

sab_status sab_kv_ring_slot_of(const sab_ring* ring, int layer, long long chunk, int* slot) {
  if (ring == nullptr || slot == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  const long long newest = ring->newest[layer];
  if (newest < 0 || chunk > newest || chunk <= newest - ring->held[layer]) return SAB_ERR_OUT_OF_RANGE;
  *slot = (int)(chunk % ring->d.ring_slots);
  return SAB_OK;
}

sab_status sab_kv_ring_get_state(const sab_ring* ring, long long* newest_chunk, int* held, int* sink_set) {
  if (ring == nullptr) return SAB_ERR_INVALID_ARG;
  for (int l = 0; l < ring->d.num_layers; ++l) {
    if (newest_chunk) newest_chunk[l] = ring->newest[l];
    if (held) held[l] = ring->held[l];
    if (sink_set) sink_set[l] = ring->sink_set[l];
  }
  return SAB_OK;
}

sab_status sab_kv_ring_set_state(sab_ring* ring, const long long* newest_chunk, const int* held,
                                 const int* sink_set) {
  if (ring == nullptr || newest_chunk == nullptr || held == nullptr || sink_set == nullptr)
    return SAB_ERR_INVALID_ARG;
  for (int l = 0; l < ring->d.num_layers; ++l) {
    const long long n = newest_chunk[l];
    const int h = held[l];
    if (n < -1 || h < 0 || h > ring->d.ring_slots || (long long)h > n + 1 || ((n == -1) != (h == 0)))
      return SAB_ERR_INVALID_ARG;
    if (sink_set[l] != 0 && sink_set[l] != 1) return SAB_ERR_INVALID_ARG;
    if (sink_set[l] && !ring->d.has_sink) return SAB_ERR_INVALID_ARG;
  }
  for (int l = 0; l < ring->d.num_layers; ++l) {
    ring->newest[l] = newest_chunk[l];
    ring->held[l] = held[l];
    ring->sink_set[l] = sink_set[l];
  }
  return SAB_OK;
}

size_t sab_chunk_attention_workspace(const sab_ring* ring, int num_splits) {
  if (ring == nullptr || num_splits < 0 || num_splits > kMaxSplits) return 0;
  if (num_splits == 0) num_splits = kMaxAutoSplits;
  return ws_layout(ring->d.batch * ring->d.heads, ring->d.chunk_tokens, ring->d.head_dim, num_splits).total;
}

static sab_status launch_attention(AttnParams& p, int Lq, int splits, void* workspace, size_t ws_bytes,
                                   void* stream) {
  if ((long long)p.B * p.H > 65535) return SAB_ERR_UNSUPPORTED;
  // One CTA per (128-query tile, (b, h), KV split), key-half softmax.  Splits
  // (explicit, or chosen on auto to fill the SMs) merge their partial rows by
  // log-sum-exp through the workspace.
  const int n_qtiles = (Lq + kTileM - 1) / kTileM;
  if (splits == 0) {
    // block-causal: a query tile sees at most (window + 1) chunks plus one straddled tile
    const int tiles = p.mode == kModeStreaming
                          ? p.plan.total_tiles
                          : ((p.window + 1) * p.chunk_tokens + 2 * kTileN - 1) / kTileN;
    splits = auto_splits((long long)n_qtiles * p.B * p.H, tiles);
  }
  p.Lq = Lq;
  p.n_qtiles = n_qtiles;
  p.splits = splits;
  if (splits > 1) {
    const WsLayout w = ws_layout(p.B * p.H, Lq, p.D, splits);
    if (workspace == nullptr || ws_bytes < w.total) return SAB_ERR_WORKSPACE;
    if ((reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0) return SAB_ERR_INVALID_ARG;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    p.ws_count = reinterpret_cast<unsigned*>(ws + w.count_off);
    p.ws_o = reinterpret_cast<float*>(ws + w.o_off);
    p.ws_lse = reinterpret_cast<float*>(ws + w.lse_off);
    p.ws_tiles = (long long)((w.lse_off - w.o_off) / ((size_t)kTileM * p.D * sizeof(float)));
    if (take_injection(SAB_DEBUG_INJECT_WS_TILE)) p.ws_tiles -= 1;  // the last tile "past" the workspace
  }
  if (p.mode == kModeStreaming && p.d_chunk == nullptr && p.plan.nseg > 0 &&
      take_injection(SAB_DEBUG_INJECT_KEY_ROW)) {
    KvSegment& sg = p.plan.seg[p.plan.nseg - 1];
    sg.row0 += p.src_rows[sg.src];  // the last key run moved past the end of its source
  }
  return launch_chunk_attention_kh(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

// Validation and key-set planning shared by both chunk-attention entry points.
// Validation and parameters common to host-planned and graph-mode calls
// (everything but the chunk index).
static sab_status plan_common(const sab_ring* ring, int layer, const void* Q, const void* K_cur, const void* V_cur,
                              int window, int use_sink, int num_splits, float softmax_scale, void* O, float* LSE,
                              AttnParams& p) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  if (Q == nullptr || O == nullptr || !aligned16(Q) || !aligned16(O)) return SAB_ERR_INVALID_ARG;
  if ((K_cur == nullptr) != (V_cur == nullptr)) return SAB_ERR_INVALID_ARG;
  if (K_cur != nullptr && (!aligned16(K_cur) || !aligned16(V_cur))) return SAB_ERR_INVALID_ARG;
  if (LSE != nullptr && (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0) return SAB_ERR_INVALID_ARG;
  if (window < 0 || num_splits < 0 || num_splits > kMaxSplits) return SAB_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return SAB_ERR_INVALID_ARG;
  if (use_sink != 0 && use_sink != 1) return SAB_ERR_INVALID_ARG;
  const sab_ring_desc& d = ring->d;
  if (use_sink && !d.has_sink) return SAB_ERR_INVALID_ARG;
  if (use_sink && !ring->sink_set[layer]) return SAB_ERR_OUT_OF_RANGE;
  const bool kcur = K_cur != nullptr;
  const bool fp8 = d.kv_dtype != SAB_KV_BF16;
  // The 8-bit cache path expands 128-byte code rows in place (D = 128), reads
  // every key from the ring (the current chunk is appended first) and needs
  // chunks of at least 128 tokens (a key tile spans at most two chunks).
  if (fp8 && (kcur || d.head_dim != 128 || d.chunk_tokens < kTileN)) return SAB_ERR_UNSUPPORTED;
  const int Lc = d.chunk_tokens;
  memset(&p, 0, sizeof(p));
  p.mode = kModeStreaming;
  p.fp8 = fp8 ? 1 : 0;
  p.k_int8 = d.kv_dtype == SAB_KV_INT8K_FP8V ? 1 : 0;
  p.k_scale = ring->ks(layer);
  p.v_scale = ring->vs(layer);
  p.scale_stride = d.has_sink + d.ring_slots;
  p.chunk_tokens = d.chunk_tokens;
  p.B = d.batch;
  p.H = d.heads;
  p.D = d.head_dim;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.O = static_cast<uint16_t*>(O);
  p.LSE = LSE;
  p.window = window;
  p.ring_slots = d.ring_slots;
  p.has_sink = d.has_sink;
  p.use_sink = use_sink;
  p.kcur = kcur ? 1 : 0;
  p.src_rows[0] = (int)ring->g.rows;
  p.src_rows[1] = kcur ? Lc : 0;
  p.k_map[0] = ring->kmap[layer];
  p.v_map[0] = ring->vmap[layer];
  p.k_map[1] = ring->kmap[layer];
  p.v_map[1] = ring->vmap[layer];
  if (kcur) {
    if (!encode_token_major(&p.k_map[1], K_cur, d.batch, Lc, d.heads, d.head_dim) ||
        !encode_token_major(&p.v_map[1], V_cur, d.batch, Lc, d.heads, d.head_dim))
      return SAB_ERR_CUDA;
  }
  if (!encode_token_major(&p.q_map, Q, d.batch, Lc, d.heads, d.head_dim) ||
      !encode_token_major(&p.o_map, O, d.batch, Lc, d.heads, d.head_dim))
    return SAB_ERR_CUDA;
  return SAB_OK;
}

// Validation and key-set planning of a host-planned call (chunk known here).
static sab_status plan_chunk_attention(const sab_ring* ring, int layer, long long chunk, const void* Q,
                                       const void* K_cur, const void* V_cur, int window, int use_sink,
                                       int num_splits, float softmax_scale, void* O, float* LSE, AttnParams& p) {
  const sab_status st =
      plan_common(ring, layer, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  if (chunk < 0) return SAB_ERR_OUT_OF_RANGE;
  // ring chunks needed: [need_lo, need_hi], all held by the ring
  const long long need_lo = std::max(0LL, chunk - window);
  const long long need_hi = p.kcur ? chunk - 1 : chunk;
  if (need_hi >= need_lo) {
    const long long newest = ring->newest[layer];
    const long long oldest = newest - ring->held[layer] + 1;
    if (newest < 0 || need_hi > newest || need_lo < oldest) return SAB_ERR_OUT_OF_RANGE;
  }
  plan_key_runs(chunk, window, p.ring_slots, p.chunk_tokens, p.has_sink, use_sink, p.kcur, p.plan);
  return SAB_OK;
}

sab_status sab_chunk_attention(const sab_ring* ring, int layer, long long chunk, const void* Q, const void* K_cur,
                               const void* V_cur, int window, int use_sink, int num_splits, float softmax_scale,
                               void* O, float* LSE, void* workspace, size_t ws_bytes, void* stream) {
  AttnParams p;
  const sab_status st =
      plan_chunk_attention(ring, layer, chunk, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  return launch_attention(p, ring->d.chunk_tokens, num_splits, workspace, ws_bytes, stream);
}

sab_status sab_chunk_attention_fp8mma(const sab_ring* ring, int layer, long long chunk, const void* Q, int window,
                                      int use_sink, int num_splits, float softmax_scale, void* O, float* LSE,
                                      void* workspace, size_t ws_bytes, void* stream) {
  if (ring == nullptr) return SAB_ERR_INVALID_ARG;
  if (ring->d.kv_dtype != SAB_KV_FP8_E4M3) return SAB_ERR_UNSUPPORTED;
  AttnParams p;
  const sab_status st = plan_chunk_attention(ring, layer, chunk, Q, nullptr, nullptr, window, use_sink, num_splits,
                                             softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  p.f8mma = 1;
  // the tensor cores read the code tiles as K-major / MN-major operands in
  // the 128-byte-swizzled layout (D = 128 codes = one swizzle row)
  const sab_ring_desc& d = ring->d;
  if (!encode_head_major_u8(&p.k_map[0], ring->k(layer), d.batch, d.heads, ring->g.rows, d.head_dim, true) ||
      !encode_head_major_u8(&p.v_map[0], ring->v(layer), d.batch, d.heads, ring->g.rows, d.head_dim, true))
    return SAB_ERR_CUDA;
  return launch_attention(p, ring->d.chunk_tokens, num_splits, workspace, ws_bytes, stream);
}

sab_status sab_chunk_attention_dev(const sab_ring* ring, int layer, const long long* d_chunk, const void* Q,
                                   const void* K_cur, const void* V_cur, int window, int use_sink, int num_splits,
                                   float softmax_scale, void* O, float* LSE, void* workspace, size_t ws_bytes,
                                   void* stream) {
  if (d_chunk == nullptr || (reinterpret_cast<uintptr_t>(d_chunk) & 7u) != 0) return SAB_ERR_INVALID_ARG;
  AttnParams p;
  const sab_status st =
      plan_common(ring, layer, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  // every window the stream can ask for must fit in the ring
  if (window > (p.kcur ? p.ring_slots : p.ring_slots - 1)) return SAB_ERR_OUT_OF_RANGE;
  p.d_chunk = d_chunk;
  // the host plan of a full window sizes the split choice; the kernels plan
  // the actual chunk on the device
  plan_key_runs((long long)window + p.ring_slots, window, p.ring_slots, p.chunk_tokens, p.has_sink, use_sink,
                p.kcur, p.plan);
  return launch_attention(p, ring->d.chunk_tokens, num_splits, workspace, ws_bytes, stream);
}

sab_status sab_qk_norm_rope(sab_ring* ring, int layer, long long chunk, const void* Q, const void* K, const void* V,
                            const float* gamma_q, const float* gamma_k, const sab_rope_desc* rope, void* Q_out,
                            void* K_out, void* V_out, int append, void* stream) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers || rope == nullptr) return SAB_ERR_INVALID_ARG;
  const sab_ring_desc& d = ring->d;
  if (Q == nullptr || K == nullptr || V == nullptr || Q_out == nullptr) return SAB_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(Q_out)) return SAB_ERR_INVALID_ARG;
  if ((K_out && !aligned16(K_out)) || (V_out && !aligned16(V_out))) return SAB_ERR_INVALID_ARG;
  if ((gamma_q && (reinterpret_cast<uintptr_t>(gamma_q) & 3u)) || (gamma_k && (reinterpret_cast<uintptr_t>(gamma_k) & 3u)))
    return SAB_ERR_INVALID_ARG;
  if (append != 0 && append != 1) return SAB_ERR_INVALID_ARG;
  if (rope->frames < 1 || rope->height < 1 || rope->width < 1 ||
      (long long)rope->frames * rope->height * rope->width != d.chunk_tokens)
    return SAB_ERR_INVALID_ARG;
  if (rope->band_t < 0 || rope->band_h < 0 || rope->band_w < 0 || (rope->band_t | rope->band_h | rope->band_w) & 1 ||
      rope->band_t + rope->band_h + rope->band_w != d.head_dim)
    return SAB_ERR_INVALID_ARG;
  if (!(rope->base > 1.f) || !isfinite(rope->base) || !(rope->eps > 0.f) || !isfinite(rope->eps))
    return SAB_ERR_INVALID_ARG;
  if (chunk < 0) return SAB_ERR_OUT_OF_RANGE;
  const bool bf16_ring = d.kv_dtype == SAB_KV_BF16;
  // an 8-bit ring quantises per (batch, head) block: K', V go through K_out,
  // V_out and the ring's own quantiser
  if (append && !bf16_ring && (K_out == nullptr || V_out == nullptr)) return SAB_ERR_INVALID_ARG;
  const long long newest = ring->newest[layer];
  if (append && newest >= 0 && chunk != newest && chunk != newest + 1) return SAB_ERR_OUT_OF_RANGE;
  const int R = d.ring_slots, slot = (int)(chunk % R);
  RopeParams rp;
  memset(&rp, 0, sizeof(rp));
  rp.q_in = static_cast<const uint16_t*>(Q);
  rp.k_in = static_cast<const uint16_t*>(K);
  rp.v_in = static_cast<const uint16_t*>(V);
  rp.gamma_q = gamma_q;
  rp.gamma_k = gamma_k;
  rp.q_out = static_cast<uint16_t*>(Q_out);
  rp.k_out = static_cast<uint16_t*>(K_out);
  rp.v_out = static_cast<uint16_t*>(V_out);
  if (append && bf16_ring) {
    rp.ring_k = static_cast<uint16_t*>(ring->k(layer));
    rp.ring_v = static_cast<uint16_t*>(ring->v(layer));
  }
  rp.B = d.batch;
  rp.H = d.heads;
  rp.D = d.head_dim;
  rp.Lc = d.chunk_tokens;
  rp.rows = (int)ring->g.rows;
  rp.slot_row0 = (d.has_sink + slot) * d.chunk_tokens;
  rp.err_word = device_error_word();
  if (rp.ring_k != nullptr && take_injection(SAB_DEBUG_INJECT_APPEND_SLOT)) rp.slot_row0 = rp.rows;
  rp.chunk = chunk;
  rp.F = rope->frames;
  rp.Hp = rope->height;
  rp.Wp = rope->width;
  rp.bt = rope->band_t;
  rp.bh = rope->band_h;
  rp.bw = rope->band_w;
  rp.log2_base = log2f(rope->base);
  rp.eps = rope->eps;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (launch_qk_rope(rp, s) != cudaSuccess) return SAB_ERR_CUDA;
  if (!append) return SAB_OK;
  if (!bf16_ring) {
    const sab_status st = write_chunk(ring, layer, rp.slot_row0, d.has_sink + slot, K_out, V_out, stream);
    if (st != SAB_OK) return st;
  }
  if (newest < 0) {
    ring->held[layer] = 1;
  } else if (chunk == newest + 1) {
    ring->held[layer] = std::min(R, ring->held[layer] + 1);
  }
  ring->newest[layer] = chunk;
  return SAB_OK;
}

sab_status sab_kv_ring_append_dev(sab_ring* ring, int layer, const long long* d_chunk, const void* K,
                                  const void* V, void* stream) {
  if (ring == nullptr || layer < 0 || layer >= ring->d.num_layers) return SAB_ERR_INVALID_ARG;
  if (K == nullptr || V == nullptr || !aligned16(K) || !aligned16(V)) return SAB_ERR_INVALID_ARG;
  if (d_chunk == nullptr || (reinterpret_cast<uintptr_t>(d_chunk) & 7u) != 0) return SAB_ERR_INVALID_ARG;
  return write_chunk(ring, layer, 0, 0, K, V, stream, d_chunk);
}

sab_status sab_chunk_counter_add(long long* d_chunk, long long delta, void* stream) {
  if (d_chunk == nullptr || (reinterpret_cast<uintptr_t>(d_chunk) & 7u) != 0) return SAB_ERR_INVALID_ARG;
  return launch_counter_add(d_chunk, delta, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK
                                                                                            : SAB_ERR_CUDA;
}

// Allocation-free variant: the split merge goes through the library's own
// device scratch (a file-scope array of the attention kernel's translation
// unit) instead of a caller workspace.  Not a counterpart of anything in the
// method; see include/sab.h.
sab_status sab_chunk_attention_noalloc(const sab_ring* ring, int layer, long long chunk, const void* Q,
                                       const void* K_cur, const void* V_cur, int window, int use_sink,
                                       int num_splits, float softmax_scale, void* O, float* LSE, void* stream) {
  if (num_splits < 1) return SAB_ERR_INVALID_ARG;
  AttnParams p;
  const sab_status st =
      plan_chunk_attention(ring, layer, chunk, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  if (num_splits == 1) return launch_attention(p, ring->d.chunk_tokens, 1, nullptr, 0, stream);
  const WsLayout w = ws_layout(ring->d.batch * ring->d.heads, ring->d.chunk_tokens, ring->d.head_dim, num_splits);
  void* scratch = nullptr;
  size_t cap = 0;
  if (noalloc_scratch(&scratch, &cap) != cudaSuccess) return SAB_ERR_CUDA;
  if (w.total > cap) return SAB_ERR_WORKSPACE;
  // the arrival counters must start at zero; the partial rows are fully rewritten
  if (cudaMemsetAsync(scratch, 0, w.o_off, static_cast<cudaStream_t>(stream)) != cudaSuccess) return SAB_ERR_CUDA;
  return launch_attention(p, ring->d.chunk_tokens, num_splits, scratch, cap, stream);
}

size_t sab_block_causal_attention_workspace(int B, int L, int H, int D, int num_splits) {
  if (B < 1 || L < 1 || H < 1 || (D != 64 && D != 128) || num_splits < 0 || num_splits > kMaxSplits) return 0;
  if (num_splits == 0) num_splits = kMaxAutoSplits;
  return ws_layout(B * H, L, D, num_splits).total;
}

sab_status sab_block_causal_attention(const void* Q, const void* K, const void* V, int B, int L, int H, int D,
                                      int chunk_tokens, int window, int num_splits, float softmax_scale, void* O,
                                      float* LSE, void* workspace, size_t ws_bytes, void* stream) {
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return SAB_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return SAB_ERR_INVALID_ARG;
  if (LSE != nullptr && (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0) return SAB_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || H < 1 || (D != 64 && D != 128) || chunk_tokens < 1 || window < 0) return SAB_ERR_INVALID_ARG;
  if (num_splits < 0 || num_splits > kMaxSplits) return SAB_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return SAB_ERR_INVALID_ARG;
  if ((long long)L > (1LL << 30)) return SAB_ERR_INVALID_ARG;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.mode = kModeBlockCausal;
  p.B = B;
  p.H = H;
  p.D = D;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.chunk_tokens = chunk_tokens;
  p.window = window;
  p.Lk = L;
  p.src_rows[0] = L;
  p.O = static_cast<uint16_t*>(O);
  p.LSE = LSE;
  if (!encode_token_major(&p.q_map, Q, B, L, H, D) || !encode_token_major(&p.k_map[0], K, B, L, H, D) ||
      !encode_token_major(&p.v_map[0], V, B, L, H, D) || !encode_token_major(&p.o_map, O, B, L, H, D))
    return SAB_ERR_CUDA;
  p.k_map[1] = p.k_map[0];
  p.v_map[1] = p.v_map[0];
  return launch_attention(p, L, num_splits, workspace, ws_bytes, stream);
}

sab_status sab_memory_prefix_attention(const void* Q, const void* K, const void* V, int B, int L, int H, int D,
                                       int mem_pad, const int* mem_len, int chunk_tokens, int window,
                                       float softmax_scale, void* O, float* LSE, void* stream) {
  if (Q == nullptr || K == nullptr || V == nullptr || O == nullptr) return SAB_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K) || !aligned16(V) || !aligned16(O)) return SAB_ERR_INVALID_ARG;
  if (LSE != nullptr && (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0) return SAB_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || H < 1 || (D != 64 && D != 128) || chunk_tokens < 1 || window < 0) return SAB_ERR_INVALID_ARG;
  if (mem_pad < 0 || mem_pad > L) return SAB_ERR_INVALID_ARG;
  if (mem_pad > 0 && (mem_len == nullptr || (reinterpret_cast<uintptr_t>(mem_len) & 3u) != 0))
    return SAB_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return SAB_ERR_INVALID_ARG;
  if ((long long)L > (1LL << 30)) return SAB_ERR_INVALID_ARG;
  AttnParams p;
  memset(&p, 0, sizeof(p));
  p.mode = mem_pad > 0 ? kModeMemPrefix : kModeBlockCausal;
  p.B = B;
  p.H = H;
  p.D = D;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.chunk_tokens = chunk_tokens;
  p.window = window;
  p.Lk = L;
  p.src_rows[0] = L;
  p.mem_pad = mem_pad;
  p.mem_len = mem_len;
  p.O = static_cast<uint16_t*>(O);
  p.LSE = LSE;
  if (!encode_token_major(&p.q_map, Q, B, L, H, D) || !encode_token_major(&p.k_map[0], K, B, L, H, D) ||
      !encode_token_major(&p.v_map[0], V, B, L, H, D) || !encode_token_major(&p.o_map, O, B, L, H, D))
    return SAB_ERR_CUDA;
  p.k_map[1] = p.k_map[0];
  p.v_map[1] = p.v_map[0];
  // one query tile per CTA, unsplit: the key runs are planned per CTA
  return launch_attention(p, L, 1, nullptr, 0, stream);
}

size_t sab_block_causal_attention_backward_workspace(int B, int L, int H) {
  if (B < 1 || L < 1 || H < 1) return 0;
  return align_up((size_t)B * H * L * sizeof(float), kAlign);
}

static sab_status attention_backward(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                     const float* LSE, int B, int L, int H, int D, int mem_pad, const int* mem_len,
                                     int chunk_tokens, int window, float softmax_scale, void* dQ, void* dK, void* dV,
                                     void* workspace, size_t ws_bytes, void* stream) {
  const void* ins[] = {Q, K, V, O, dO, dQ, dK, dV};
  for (const void* x : ins)
    if (x == nullptr || !aligned16(x)) return SAB_ERR_INVALID_ARG;
  if (LSE == nullptr || (reinterpret_cast<uintptr_t>(LSE) & 3u) != 0) return SAB_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || H < 1 || (D != 64 && D != 128) || chunk_tokens < 1 || window < 0) return SAB_ERR_INVALID_ARG;
  if (mem_pad < 0 || mem_pad > L) return SAB_ERR_INVALID_ARG;
  if (mem_pad > 0 && (mem_len == nullptr || (reinterpret_cast<uintptr_t>(mem_len) & 3u) != 0))
    return SAB_ERR_INVALID_ARG;
  if (!(softmax_scale > 0.f) || !isfinite(softmax_scale)) return SAB_ERR_INVALID_ARG;
  if ((long long)L > (1LL << 30) || (long long)B * H > 65535) return SAB_ERR_INVALID_ARG;
  if (workspace == nullptr || ws_bytes < sab_block_causal_attention_backward_workspace(B, L, H) ||
      (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
    return SAB_ERR_WORKSPACE;
  BwdParams p;
  memset(&p, 0, sizeof(p));
  p.O = static_cast<const uint16_t*>(O);
  p.dO = static_cast<const uint16_t*>(dO);
  p.LSE = LSE;
  p.delta = static_cast<float*>(workspace);
  p.dQ = static_cast<uint16_t*>(dQ);
  p.dK = static_cast<uint16_t*>(dK);
  p.dV = static_cast<uint16_t*>(dV);
  p.B = B;
  p.H = H;
  p.D = D;
  p.L = L;
  p.chunk_tokens = chunk_tokens;
  p.window = window;
  p.mem_pad = mem_pad;
  p.mem_len = mem_pad > 0 ? mem_len : nullptr;
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  if (!encode_token_major(&p.q_map, Q, B, L, H, D) || !encode_token_major(&p.k_map, K, B, L, H, D) ||
      !encode_token_major(&p.v_map, V, B, L, H, D) || !encode_token_major(&p.do_map, dO, B, L, H, D) ||
      !encode_token_major(&p.q_map_h, Q, B, L, H, D, 64) || !encode_token_major(&p.k_map_h, K, B, L, H, D, 64) ||
      !encode_token_major(&p.v_map_h, V, B, L, H, D, 64) || !encode_token_major(&p.do_map_h, dO, B, L, H, D, 64))
    return SAB_ERR_CUDA;
  return launch_attention_backward(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

sab_status sab_block_causal_attention_backward(const void* Q, const void* K, const void* V, const void* O,
                                               const void* dO, const float* LSE, int B, int L, int H, int D,
                                               int chunk_tokens, int window, float softmax_scale, void* dQ,
                                               void* dK, void* dV, void* workspace, size_t ws_bytes,
                                               void* stream) {
  return attention_backward(Q, K, V, O, dO, LSE, B, L, H, D, 0, nullptr, chunk_tokens, window, softmax_scale, dQ, dK,
                            dV, workspace, ws_bytes, stream);
}

sab_status sab_memory_prefix_attention_backward(const void* Q, const void* K, const void* V, const void* O,
                                                const void* dO, const float* LSE, int B, int L, int H, int D,
                                                int mem_pad, const int* mem_len, int chunk_tokens, int window,
                                                float softmax_scale, void* dQ, void* dK, void* dV, void* workspace,
                                                size_t ws_bytes, void* stream) {
  return attention_backward(Q, K, V, O, dO, LSE, B, L, H, D, mem_pad, mem_len, chunk_tokens, window, softmax_scale,
                            dQ, dK, dV, workspace, ws_bytes, stream);
}

// x^(num/den) within 2^-51 of it.  The quotient's rounding, up to 2^-53 of it,
// would grow by ln(x^(num/den)) (2^-50.4 for base 10^4 and 44 dimensions), so its
// exact remainder goes into a first-order factor.
static double power_of_quotient(double x, int num, int den) {
  const double e = (double)num / den;
  const double rest = fma(-e, (double)den, (double)num) / den;
  const double f = pow(x, e);
  return fma(f, rest * log(x), f);
}

sab_status sab_rotary_plan_init(const sab_rotary_desc* desc, sab_rotary_plan* plan) {
  if (desc == nullptr || plan == nullptr) return SAB_ERR_INVALID_ARG;
  const sab_rotary_desc& d = *desc;
  if (d.layout != SAB_ROTARY_INTERLEAVED && d.layout != SAB_ROTARY_HALF) return SAB_ERR_INVALID_ARG;
  if (d.axes < 1 || d.axes > 3) return SAB_ERR_INVALID_ARG;
  long long dims = 0;
  for (int a = 0; a < d.axes; ++a) {
    if (d.band[a] < 2 || (d.band[a] & 1)) return SAB_ERR_INVALID_ARG;
    dims += d.band[a];
  }
  if (dims > SAB_ROTARY_MAX_DIMS) return SAB_ERR_INVALID_ARG;
  if (!(d.base > 1.0) || !isfinite(d.base) || !((float)d.magnitude > 0.f) || !isfinite((float)d.magnitude))
    return SAB_ERR_INVALID_ARG;
  double s = 1.0;
  if (d.scaling != SAB_ROTARY_SCALE_NONE) {
    if (d.scaling < 0 || d.scaling > SAB_ROTARY_SCALE_RAMP) return SAB_ERR_INVALID_ARG;
    if (!(d.factor >= 1.0) || !isfinite(d.factor)) return SAB_ERR_INVALID_ARG;
    s = d.factor;
  }
  if (d.scaling == SAB_ROTARY_SCALE_RAMP &&
      (!(d.original_context > 0.0) || !isfinite(d.original_context) || !isfinite(d.ramp_fast) ||
       !isfinite(d.ramp_slow) || !(d.ramp_slow < d.ramp_fast)))
    return SAB_ERR_INVALID_ARG;
  if (d.scaling == SAB_ROTARY_SCALE_BASE)
    for (int a = 0; a < d.axes; ++a)
      if (d.band[a] == 2) return SAB_ERR_INVALID_ARG;
  constexpr double kTwoPi = 6.283185307179586476925286766559;
  memset(plan, 0, sizeof(*plan));
  int j = 0;
  for (int a = 0; a < d.axes; ++a) {
    const int n = d.band[a];
    if (d.scaling == SAB_ROTARY_SCALE_BASE && !isfinite(d.base * pow(s, n / (n - 2.0)))) return SAB_ERR_INVALID_ARG;
    for (int i = 0; i < n / 2; ++i, ++j) {
      double f = power_of_quotient(d.base, -2 * i, n);
      // (base s^(n/(n-2)))^(-2i/n)
      if (d.scaling == SAB_ROTARY_SCALE_BASE) f *= power_of_quotient(s, -2 * i, n - 2);
      if (d.scaling == SAB_ROTARY_SCALE_LINEAR) f /= s;
      if (d.scaling == SAB_ROTARY_SCALE_RAMP) {
        const double w = (d.original_context * f / kTwoPi - d.ramp_slow) / (d.ramp_fast - d.ramp_slow);
        const double keep = w < 0.0 ? 0.0 : w > 1.0 ? 1.0 : w;
        f *= keep + (1.0 - keep) / s;
      }
      // f <= 1 radian per position, so below 1/6 of a turn
      plan->axis[j] = (unsigned char)a;
      plan->step[j] = (unsigned long long)(ldexp(f / kTwoPi, 64) + 0.5);
    }
  }
  plan->layout = d.layout;
  plan->axes = d.axes;
  plan->dims = (int)dims;
  plan->magnitude = (float)d.magnitude;
  plan->magic = kRotaryMagic;
  return SAB_OK;
}

// Rows of one rotary tensor: pointers, strides, and that no two output
// tokens share an element.
static bool rotary_rows_ok(const sab_rotary_rows* r, int B, int L, int D, int esize) {
  if (r->in == nullptr || r->out == nullptr || !aligned16(r->in) || !aligned16(r->out) || r->heads < 1) return false;
  if ((long long)r->heads * D > (1LL << 30)) return false;
  const long long st[4] = {r->in_batch, r->in_token, r->out_batch, r->out_token};
  for (long long x : st)
    if (x < 0 || x > (1LL << 40) || (x * esize) % 16 != 0) return false;
  if (r->in == r->out && (r->in_batch != r->out_batch || r->in_token != r->out_token) && (long long)B * L > 1)
    return false;
  const long long row = (long long)r->heads * D;
  // whole extents within 2^47 elements, more than a device can address: what is
  // formed from the strides below and in the kernel stays within 64 bits
  constexpr long long kMost = 1LL << 47;
  for (int i = 0; i < 4; i += 2) {
    if (B > 1 && st[i] > kMost / (B - 1)) return false;
    if (L > 1 && st[i + 1] > kMost / (L - 1)) return false;
  }
  const bool token_apart = L == 1 || r->out_token >= row, batch_apart = B == 1 || r->out_batch >= row;
  const bool token_inner = B == 1 || r->out_batch >= (L - 1) * r->out_token + row;
  const bool batch_inner = L == 1 || r->out_token >= (B - 1) * r->out_batch + row;
  return token_apart && batch_apart && (token_inner || batch_inner);
}

static sab_status rotary(const sab_rotary_plan* plan, const sab_rotary_rows* q, const sab_rotary_rows* k,
                         const long long* positions, long long first_position, int B, int L, int D, int dtype,
                         bool backward, void* stream) {
  if (plan == nullptr || plan->magic != kRotaryMagic || q == nullptr) return SAB_ERR_INVALID_ARG;
  if (plan->axes < 1 || plan->axes > 3 || plan->dims < 2 || plan->dims > SAB_ROTARY_MAX_DIMS || plan->dims % 2 != 0)
    return SAB_ERR_INVALID_ARG;
  for (int j = 0; j < plan->dims / 2; ++j)
    if (plan->axis[j] >= plan->axes) return SAB_ERR_INVALID_ARG;
  if (dtype != SAB_DTYPE_BF16 && dtype != SAB_DTYPE_FP32) return SAB_ERR_INVALID_ARG;
  if (B < 1 || L < 1 || L > (1 << 30) || (long long)B * L > (1LL << 31) || D < 8 || D % 8 != 0 ||
      D > SAB_ROTARY_MAX_DIMS || plan->dims > D)
    return SAB_ERR_INVALID_ARG;
  if (positions == nullptr ? plan->axes != 1 : (reinterpret_cast<uintptr_t>(positions) & 7u) != 0)
    return SAB_ERR_INVALID_ARG;
  const int esize = dtype == SAB_DTYPE_BF16 ? 2 : 4;
  if (!rotary_rows_ok(q, B, L, D, esize) || (k != nullptr && !rotary_rows_ok(k, B, L, D, esize)))
    return SAB_ERR_INVALID_ARG;
  // one tensor's rows turned twice, or turned while the other is read
  if (k != nullptr && (k->out == q->out || k->out == q->in || q->out == k->in)) return SAB_ERR_INVALID_ARG;
  RotaryParams p;
  memset(&p, 0, sizeof(p));
  for (int w = 0; w < 2; ++w) {
    const sab_rotary_rows* r = w == 0 ? q : k;
    if (r != nullptr)
      p.rows[w] = RotaryRows{r->in, r->out, r->heads, r->in_batch, r->in_token, r->out_batch, r->out_token};
  }
  p.positions = positions;
  p.first_position = first_position;
  p.B = B;
  p.L = L;
  p.D = D;
  p.dims = plan->dims;
  p.half_layout = plan->layout == SAB_ROTARY_HALF;
  p.magnitude = plan->magnitude;
  p.sine = backward ? -plan->magnitude : plan->magnitude;
  memcpy(p.axis, plan->axis, sizeof(p.axis));
  memcpy(p.step, plan->step, sizeof(p.step));
  const cudaError_t e = launch_rotary(p, dtype == SAB_DTYPE_FP32, device_sms(), static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

sab_status sab_rotary(const sab_rotary_plan* plan, const sab_rotary_rows* q, const sab_rotary_rows* k,
                      const long long* positions, long long first_position, int B, int L, int D, int dtype,
                      void* stream) {
  return rotary(plan, q, k, positions, first_position, B, L, D, dtype, false, stream);
}

sab_status sab_rotary_backward(const sab_rotary_plan* plan, const sab_rotary_rows* dq, const sab_rotary_rows* dk,
                               const long long* positions, long long first_position, int B, int L, int D,
                               int dtype, void* stream) {
  return rotary(plan, dq, dk, positions, first_position, B, L, D, dtype, true, stream);
}

// Arguments common to the decay attention calls.
static bool decay_shape_ok(int B, int L, int H, int D) {
  return B >= 1 && L >= 1 && H >= 1 && (D == 64 || D == 128) && L <= (1 << 30) && (long long)B * H <= (1LL << 24) &&
         (long long)B * L <= (1LL << 38) / ((long long)H * D);
}
static bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

// Runs of up to so many tokens go token by token in fp32, with 32 value columns a
// CTA; longer ones in tiles.  Measured, us, token by token against tiles:
//   forward, heads of 128, 16 tokens: 12 heads 4.7 / 5.2, with states 5.3 / 11.0;
//     96 heads 13.6 / 5.5 and 15.9 / 12.5; 768 heads 56.6 / 30.4 and 60.5 / 66.4.
//     40 tokens of 12 heads 10.1 / 5.4 and 10.6 / 11.1; 4 tokens of 96 heads 5.1 /
//     5.4 and 7.7 / 12.3.  Heads of 64, 16 tokens: 12, 192 and 768 heads 3.5 / 4.4,
//     7.3 / 8.6 and 18.7 / 24.6, with states 3.8 / 5.7, 7.7 / 11.1 and 21.0 / 34.1.
//   gradients (three launches token by token, shared ones in tiles), heads of 128:
//     12 tokens of 12 heads 11.5 / 5.3, with states 13.4 / 14.3; of 48 heads 34.4 /
//     5.5 and 43.4 / 16.2; 4 tokens of 192 heads 18.1 / 20.3 and 31.3 / 36.9.  Heads
//     of 64: 8 tokens of 12 heads 8.1 / 4.5 and 8.8 / 9.8; 12 tokens of 304 heads
//     18.6 / 26.6 and 23.3 / 31.5.
// So: longer runs while the CTAs fit the SMs once, shorter ones beside tiles that
// need one wave, longer ones beside tiles that write states or need several waves.
static int decay_short_tokens(long long bh, int D, bool state, bool gradients) {
  const long long sms = device_sms();
  const bool once = bh * (D / 32) <= sms;
  if (!gradients) return D == 64 ? 16 : once ? (state ? 40 : 16) : (state ? 12 : 4);
  const long long waves = (3 * bh + sms - 1) / sms;  // of the tiles
  if (waves >= 3) return D == 128 ? 4 : 12;
  if (D == 128) return once && state ? 12 : 0;
  return waves == 2 ? 2 : state ? 8 : 0;
}

// How a call cuts its sequences.  A CTA takes a sequence's head as a whole, or,
// when B * H of them leave SMs idle, segments of it; the states before the
// segments then cost a pass over k and v and two launches.  Chosen by modelled
// times, in us, for T tiles in a row (whole) or `per` tiles a segment with a
// share f of the SMs at work.
struct DecayCut {
  int nseg, seg_tiles;
};

// One run, one segment per SM.  Measured, whole against cut, without and with
// state_out, heads of 128: 2 sequences of 2 tiles 8.2 / 11.3 and 16.0 / 11.9; 24
// of 4 tiles 14.2 / 13.0 and 23.9 / 15.0; 72 of 12 tiles 38.6 / 40.8 and 54.8 /
// 47.8; 24 of 32 tiles 95 / 37 and 127 / 43.  (More segments than SMs lose: 156
// of 12 tiles 76.7 / 101.6.)
static DecayCut decay_cut_forward(int tiles, long long bh, int D, bool state) {
  const long long most = std::min<long long>(device_sms() / bh, tiles);
  if (most < 2) return {1, tiles};
  const int per = (int)((tiles + most - 1) / most), n = (tiles + per - 1) / per;
  const double f = (double)(bh * n) / device_sms();
  const double whole =
      D == 128 ? (state ? 8.5 + 3.8 * tiles : 3.0 + 2.9 * tiles) : (state ? 3.6 + 2.15 * tiles : 2.5 + 2.03 * tiles);
  const double cut = D == 128 ? 7.0 + 4.3 * per + 4.5 * f + (state ? 1.0 + 0.5 * per + 2.5 * f : 0.0)
                              : 6.2 + 2.95 * per + 1.7 * f + (state ? 0.6 + 0.3 * per + f : 0.0);
  return n > 1 && cut < whole ? DecayCut{n, per} : DecayCut{1, tiles};
}

// Three runs that share launches: one CTA a segment and run, in waves over the
// SMs, so fewer and longer segments than one per SM.  Fitted to 300 calls (1
// to 96 heads, 4 to 240 tiles, 1 to 152 segments) to 3 %; the choice was never
// 2 % slower than the best.  Heads of 128, without state, us by segments: 12
// of 12 tiles 41 (whole), 40 (2), 30 (4), 38 (6), 44 (12); 24 of 240 tiles 664,
// 513 (2), 464 (4), 490 (6); 48 of 32 tiles 104, 142 (2), 163 (4).
static DecayCut decay_cut_gradients(int tiles, long long bh, int D, bool state) {
  const long long sms = device_sms(), most = std::min<long long>(sms / bh, tiles);
  auto waves = [&](long long ctas) { return (double)((ctas + sms - 1) / sms); };
  double best = D == 128 ? (state ? waves(2 * bh) * (6.3 + 2.8 * tiles) + waves(bh) * (10.0 + 3.65 * tiles)
                                  : waves(3 * bh) * (8.0 + 2.8 * tiles))
                         : (state ? waves(2 * bh) * (7.0 + 2.15 * tiles) + waves(bh) * (4.3 + 2.22 * tiles)
                                  : 4.6 + waves(3 * bh) * (3.4 + 2.15 * tiles));
  DecayCut how{1, tiles};
  for (int n = 2, last = tiles; n <= most; ++n) {  // the fewest segments of each length
    const int per = (tiles + n - 1) / n;
    if (per == last) continue;
    last = per;
    const double f = (double)(bh * n) / sms, sums = waves(bh * (2 * n - 2 + state)) * per, wt = waves(3 * bh * n);
    const double t = D == 128 ? (state ? 11.3 : 10.0) + 0.05 * n + 24.0 * f + (state ? 1.5 : 0.9) * sums +
                                    wt * (0.9 + 3.1 * per)
                              : 9.6 + 0.05 * n + 13.0 * f + (state ? 1.4 : 0.9) * sums + wt * (0.6 + 2.1 * per);
    if (t < best) best = t, how = {n, per};
  }
  return how;
}

static DecayCut decay_cut(int B, int L, int H, int D, bool state, bool gradients) {
  const int tiles = (L + kTileM - 1) / kTileM;
  return gradients ? decay_cut_gradients(tiles, (long long)B * H, D, state)
                   : decay_cut_forward(tiles, (long long)B * H, D, state);
}
static size_t decay_workspace(int B, int L, int H, int D, bool gradients) {
  if (!decay_shape_ok(B, L, H, D)) return 0;
  const int n = std::max(decay_cut(B, L, H, D, false, gradients).nseg, decay_cut(B, L, H, D, true, gradients).nseg);
  return n == 1 ? 0 : (gradients ? 2 : 1) * align_up((size_t)B * H * n * D * D * sizeof(float), kAlign);
}

size_t sab_decay_attention_workspace(int B, int L, int H, int D) { return decay_workspace(B, L, H, D, false); }

// One run of the recurrence.  carry: the part of the workspace that holds the
// states before the segments; carry_t: run 1's, transposed.
struct DecayRun {
  const void *q, *k, *v;
  void* o;
  const float* in;
  float* out;
  int reverse, state_t;
  float kv_mul, o_mul;
  int carry, carry_t;
};
// Up to three runs, of which the third, if any, reads the second's carried
// states.  Runs share their launches, except that whole sequences whose state
// is wanted go by themselves: they multiply more, and may write a state that
// another run reads.
static sab_status decay_runs(const DecayRun* runs, int n, const DecayCut& cut, const float* log_decay,
                             const int* seq_len, int B, int L, int H, int D, void* workspace, size_t ws_bytes,
                             void* stream) {
  DecayRuns all;
  memset(&all, 0, sizeof(all));
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  bool state = false;
  for (int i = 0; i < n; ++i) state = state || runs[i].out != nullptr;
  const bool is_short = L <= decay_short_tokens((long long)B * H, D, state, n > 1), cut_up = cut.nseg > 1;
  const size_t states = cut_up ? (size_t)B * H * cut.nseg : 0, held = ws_bytes / ((size_t)D * D * sizeof(float));
  for (int i = 0; i < n; ++i) {
    const DecayRun& r = runs[i];
    DecayTileParams& p = all.run[i];
    p.seg_tiles = cut.seg_tiles;
    p.nseg = cut.nseg;
    p.q = static_cast<const uint16_t*>(r.q);
    p.k = static_cast<const uint16_t*>(r.k);
    p.v = static_cast<const uint16_t*>(r.v);
    p.o = static_cast<uint16_t*>(r.o);
    p.log_decay = log_decay;
    p.seq_len = seq_len;
    p.state_in = r.in;
    p.state_out = r.out;
    p.carry = static_cast<float*>(workspace) + r.carry * states * D * D;
    p.carry_t = r.carry_t;
    p.carry_states = (long long)held - (long long)(r.carry * states);
    p.B = B;
    p.L = L;
    p.H = H;
    p.D = D;
    p.by_length = seq_len != nullptr && p.nseg == 1 && B > 1 && B <= kMaxByLength && (long long)B * H > device_sms();
    p.reverse = r.reverse;
    p.state_t = r.state_t;
    p.kv_mul = r.kv_mul;
    p.o_mul = r.o_mul;
    p.err_word = device_error_word();
    if (is_short) {
      if (launch_decay_short(p, s) != cudaSuccess) return SAB_ERR_CUDA;
      continue;
    }
    const bool sums = cut_up && !r.carry_t;
    if (!encode_token_major(&p.q_map, r.q, B, L, H, D) || !encode_token_major(&p.k_map, r.k, B, L, H, D) ||
        !encode_token_major(&p.v_map, r.v, B, L, H, D) || !encode_token_major(&p.o_map, r.o, B, L, H, D) ||
        (sums && (!encode_token_major(&p.k_map_h, r.k, B, L, H, D, 64) ||
                  !encode_token_major(&p.v_map_h, r.v, B, L, H, D, 64))))
      return SAB_ERR_CUDA;
  }
  if (is_short) return SAB_OK;
  if (cut_up) {
    all.n = std::min(n, 2);
    if (launch_decay_segments(all, s) != cudaSuccess) return SAB_ERR_CUDA;
    for (int i = 0; i < n; ++i) all.run[i].state_out = nullptr;  // written with the segments' states
  }
  const bool apart = n > 1 && all.run[n - 1].state_out != nullptr;
  all.n = apart ? n - 1 : n;
  if (launch_decay_tiles(all, s) != cudaSuccess) return SAB_ERR_CUDA;
  if (apart) {
    all.run[0] = all.run[n - 1];
    all.n = 1;
    if (launch_decay_tiles(all, s) != cudaSuccess) return SAB_ERR_CUDA;
  }
  return SAB_OK;
}

sab_status sab_decay_attention(const void* Q, const void* K, const void* V, const float* log_decay,
                               const int* seq_len, const float* state_in, int B, int L, int H, int D, float scale,
                               void* O, float* state_out, void* workspace, size_t ws_bytes, void* stream) {
  const void* ptrs[] = {Q, K, V, O};
  for (const void* x : ptrs)
    if (x == nullptr || !aligned16(x)) return SAB_ERR_INVALID_ARG;
  if (O == Q || O == K || O == V) return SAB_ERR_INVALID_ARG;
  if (log_decay == nullptr || !aligned4(log_decay) || !aligned4(seq_len) || !aligned16(state_in) ||
      !aligned16(state_out))
    return SAB_ERR_INVALID_ARG;
  if (!decay_shape_ok(B, L, H, D) || !(scale > 0.f) || !isfinite(scale)) return SAB_ERR_INVALID_ARG;
  const size_t need = sab_decay_attention_workspace(B, L, H, D);
  if (need > 0 && (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0))
    return SAB_ERR_WORKSPACE;
  const DecayRun run = {Q, K, V, O, state_in, state_out, 0, 0, 1.f, scale, 0, 0};
  return decay_runs(&run, 1, decay_cut(B, L, H, D, state_out != nullptr, false), log_decay, seq_len, B, L, H, D,
                    workspace, ws_bytes, stream);
}

sab_status sab_decay_attention_step(const void* Q, const void* K, const void* V, const float* log_decay,
                                    const int* active, const float* state_in, int B, int H, int D, float scale,
                                    void* O, float* state_out, void* stream) {
  const void* ptrs[] = {Q, K, V, O, state_out};
  for (const void* x : ptrs)
    if (x == nullptr || !aligned16(x)) return SAB_ERR_INVALID_ARG;
  if (O == Q || O == K || O == V) return SAB_ERR_INVALID_ARG;
  if (log_decay == nullptr || !aligned4(log_decay) || !aligned4(active) || !aligned16(state_in))
    return SAB_ERR_INVALID_ARG;
  if (!decay_shape_ok(B, 1, H, D) || !(scale > 0.f) || !isfinite(scale)) return SAB_ERR_INVALID_ARG;
  DecayStepParams p;
  memset(&p, 0, sizeof(p));
  p.q = static_cast<const uint16_t*>(Q);
  p.k = static_cast<const uint16_t*>(K);
  p.v = static_cast<const uint16_t*>(V);
  p.o = static_cast<uint16_t*>(O);
  p.log_decay = log_decay;
  p.active = active;
  p.state_in = state_in;
  p.state_out = state_out;
  p.B = B;
  p.H = H;
  p.D = D;
  p.scale = scale;
  return launch_decay_step(p, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

size_t sab_decay_attention_backward_workspace(int B, int L, int H, int D) { return decay_workspace(B, L, H, D, true); }

sab_status sab_decay_attention_backward(const void* Q, const void* K, const void* V, const void* dO,
                                        const float* log_decay, const int* seq_len, const float* state_in,
                                        const float* d_state_out, int B, int L, int H, int D, float scale, void* dQ,
                                        void* dK, void* dV, float* d_state_in, void* workspace, size_t ws_bytes,
                                        void* stream) {
  const void* ptrs[] = {Q, K, V, dO, dQ, dK, dV};
  for (int i = 0; i < 7; ++i) {
    if (ptrs[i] == nullptr || !aligned16(ptrs[i])) return SAB_ERR_INVALID_ARG;
    for (int j = 4; j < 7; ++j)
      if (j != i && ptrs[i] == ptrs[j]) return SAB_ERR_INVALID_ARG;
  }
  if (log_decay == nullptr || !aligned4(log_decay) || !aligned4(seq_len) || !aligned16(state_in) ||
      !aligned16(d_state_out) || !aligned16(d_state_in))
    return SAB_ERR_INVALID_ARG;
  if (d_state_in != nullptr && d_state_in == state_in) return SAB_ERR_INVALID_ARG;
  if (!decay_shape_ok(B, L, H, D) || !(scale > 0.f) || !isfinite(scale)) return SAB_ERR_INVALID_ARG;
  const size_t need = sab_decay_attention_backward_workspace(B, L, H, D);
  if (need > 0 && (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0))
    return SAB_ERR_WORKSPACE;
  // dV and dK share one chain of states (dK's run holds them transposed).
  // d_state_in, which may be d_state_out, is written by the last to read
  // d_state_out: the chain, or else dK's run.
  const DecayCut how = decay_cut(B, L, H, D, d_state_in != nullptr, true);
  const bool cut = how.nseg > 1;
  const DecayRun runs[3] = {{dO, V, K, dQ, state_in, nullptr, 0, 1, 1.f, scale, 0, 0},
                            {K, Q, dO, dV, d_state_out, cut ? d_state_in : nullptr, 1, 0, scale, 1.f, 1, 0},
                            {V, dO, Q, dK, d_state_out, cut ? nullptr : d_state_in, 1, 1, scale, 1.f, 1, 1}};
  return decay_runs(runs, 3, how, log_decay, seq_len, B, L, H, D, workspace, ws_bytes, stream);
}

// ------------------------------------------------------------ cross attention

static bool cross_shape_ok(const sab_cross_desc* d) {
  if (d == nullptr || d->batch < 1 || d->q_tokens < 1 || d->kv_tokens < 1 || d->heads < 1 || d->kv_heads < 1)
    return false;
  if (d->head_dim != 64 && d->head_dim != 128) return false;
  if (d->heads % d->kv_heads != 0 || d->heads / d->kv_heads > kTileM) return false;
  if (d->kv_batch != 1 && d->kv_batch != d->batch) return false;
  // a query tile over 2^26 keys takes up to 1.1 s (2.2 us a key tile with running
  // maxima); its end is waited for 2 s at most
  if (d->q_tokens > (1 << 30) || d->kv_tokens > (1 << 26) || d->heads > (1 << 20)) return false;
  return (long long)d->batch * d->heads * ((d->q_tokens + 31) / 32) <= (1LL << 30) &&
         (long long)d->kv_batch * d->kv_heads * ((d->kv_tokens + 31) / 32) <= (1LL << 30);
}
// The kernels' scale, of exponents to base 2, has to be finite too: with an
// infinite one a score of 0 is no number.
static bool cross_scale_ok(float scale) { return scale > 0.f && isfinite(scale * 1.4426950408889634f); }
// Rows of one [B, L, H, D] tensor: pointer and strides that a tensor map takes;
// heads and tokens apart from one another, and sequences too where the tensor is
// written.  Strides of axes of one entry say nothing.
static long long head_of(const sab_token_rows* r, int H, int D) { return H > 1 && r->head != 0 ? r->head : D; }
static long long token_of(const sab_token_rows* r, int L, int H, int D) { return L > 1 ? r->token : (long long)H * D; }
static long long batch_of(const sab_token_rows* r, int B, int H, int D) { return B > 1 ? r->batch : (long long)H * D; }
static bool token_rows_ok(const sab_token_rows* r, int B, int L, int H, int D, bool out) {
  if (r == nullptr || r->data == nullptr || !aligned16(r->data)) return false;
  constexpr long long kMost = 1LL << 38;  // elements: a tensor map's strides are below 2^40 bytes
  struct Axis {
    long long stride, n;
  } axes[3] = {{head_of(r, H, D), H}, {r->token, L}, {r->batch, B}};
  for (const Axis& a : axes)
    if (a.n > 1 && (a.stride < D || a.stride > kMost || a.stride % 8 != 0)) return false;
  // sequences that are only read may share tokens, as windows of one run do
  const int nested = out ? 3 : 2;
  for (int i = 0; i < nested; ++i)  // by stride
    for (int k = 0; k + 1 < nested; ++k)
      if (axes[k].stride > axes[k + 1].stride) {
        const Axis a = axes[k];
        axes[k] = axes[k + 1];
        axes[k + 1] = a;
      }
  long long extent = D;
  for (int i = 0; i < nested; ++i) {
    if (axes[i].n == 1) continue;
    if (axes[i].stride < extent) return false;
    extent += (axes[i].n - 1) * axes[i].stride;
  }
  return true;
}

// Query rows: a map of tiles of `pack` heads x `tokens` tokens.
static bool encode_query_rows(CUtensorMap* m, const sab_token_rows* r, int B, int L, int H, int D, int pack,
                              int tokens) {
  EncodeTiledFn fn = encode_fn();
  if (fn == nullptr) return false;
  const size_t head = (size_t)head_of(r, H, D) * 2, token = (size_t)token_of(r, L, H, D) * 2;
  const size_t batch = (size_t)batch_of(r, B, H, D) * 2;
  if (pack == 1)  // tokens before heads
    return encode_map(m, r->data, D, L, H, B, token, head, batch, tokens);
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)L, (cuuint64_t)B};
  const cuuint64_t strides[3] = {head, token, batch};
  const cuuint32_t box[4] = {64, (cuuint32_t)pack, (cuuint32_t)tokens, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, r->data, dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}
static bool encode_key_rows(CUtensorMap* m, const sab_token_rows* r, int B, int L, int H, int D) {
  return encode_map(m, r->data, D, L, H, B, (size_t)token_of(r, L, H, D) * 2, (size_t)head_of(r, H, D) * 2,
                    (size_t)batch_of(r, B, H, D) * 2);
}

// Heads of one tile of `rows` query rows: the number, among those that divide
// the heads of a key head, with the fewest tiles; of equals the largest, whose
// tiles share their keys.
static int cross_pack(int q_tokens, int group, int rows) {
  int best = 1;
  long long least = 0;
  for (int k = 1; k <= group && k <= rows; ++k) {
    if (group % k != 0) continue;
    const int tokens = rows / k;
    const long long tiles = (long long)((q_tokens + tokens - 1) / tokens) * (group / k);
    if (k == 1 || tiles <= least) best = k, least = tiles;
  }
  return best;
}

// Blocks among which the keys of a query tile are cut: as many (a power of two,
// at most 8) as the SMs that the query tiles leave idle, each with a key tile.
static int cross_splits(unsigned items, int key_tiles) {
  int n = 1;
  while (n < 8 && 2LL * n * items <= device_sms() && 2 * n <= key_tiles) n *= 2;
  return n;
}

// Query tiles of a call whose sequences may differ in length: 2^26 at most.  A
// block first clears its rows without a query or key, in 1.1 (gradients 1.6) us a
// tile of one token (measured up to 2^20), and its other warps wait for that 2 s at
// most.  On 152 SMs 2^26 tiles make 0.5 (0.7) s, 2^28 would 1.9 (2.8).
static bool cross_tiles_ok(const sab_cross_desc& d, const int* q_len, const int* kv_len, long long tiles) {
  return (q_len == nullptr && kv_len == nullptr) || d.batch * tiles <= (1LL << 26);
}

// More than one item a block, of sequences that may differ in length; 64 of them
// and 2^26 items at most (what the kernels' table of them holds).
static int cross_sorted(const sab_cross_desc& d, const int* q_len, const int* kv_len, unsigned items) {
  return (q_len != nullptr || kv_len != nullptr) && d.batch > 1 && d.batch <= 64 && (long long)items > device_sms() &&
         items < (1u << 26);
}

// Debug builds: the items of a sequence past the last.
static bool forge_items(CrossParams& p) {
  if (!take_injection(SAB_DEBUG_INJECT_CROSS_ITEM)) return false;
  p.items += (unsigned)(p.head_blocks * ((p.n_qtiles + p.pair - 1) / p.pair));
  return true;
}

sab_status sab_cross_attention(const sab_cross_desc* desc, const sab_token_rows* Q, const sab_token_rows* K,
                               const sab_token_rows* V, const int* q_len, const int* kv_len, float softmax_scale,
                               const sab_token_rows* O, float* LSE, void* stream) {
  if (!cross_shape_ok(desc) || !cross_scale_ok(softmax_scale)) return SAB_ERR_INVALID_ARG;
  const sab_cross_desc& d = *desc;
  const int D = d.head_dim;
  if (!token_rows_ok(Q, d.batch, d.q_tokens, d.heads, D, false) ||
      !token_rows_ok(K, d.kv_batch, d.kv_tokens, d.kv_heads, D, false) ||
      !token_rows_ok(V, d.kv_batch, d.kv_tokens, d.kv_heads, D, false) ||
      !token_rows_ok(O, d.batch, d.q_tokens, d.heads, D, true))
    return SAB_ERR_INVALID_ARG;
  if (O->data == Q->data || O->data == K->data || O->data == V->data || !aligned4(q_len) || !aligned4(kv_len) ||
      !aligned16(LSE))
    return SAB_ERR_INVALID_ARG;
  CrossParams p;
  memset(&p, 0, sizeof(p));
  p.q_len = q_len;
  p.kv_len = kv_len;
  p.O = static_cast<uint16_t*>(O->data);
  p.o_batch = batch_of(O, d.batch, d.heads, D);
  p.o_token = token_of(O, d.q_tokens, d.heads, D);
  p.o_head = head_of(O, d.heads, D);
  p.LSE = LSE;
  p.B = d.batch;
  p.Bk = d.kv_batch;
  p.Lq = d.q_tokens;
  p.Lk = d.kv_tokens;
  p.H = d.heads;
  p.D = d.head_dim;
  p.group = d.heads / d.kv_heads;
  p.pack = cross_pack(d.q_tokens, p.group, kTileM);
  p.tile_tokens = kTileM / p.pack;
  p.n_qtiles = (d.q_tokens + p.tile_tokens - 1) / p.tile_tokens;
  p.head_blocks = d.heads / p.pack;
  if (!cross_tiles_ok(d, q_len, kv_len, (long long)p.head_blocks * p.n_qtiles)) return SAB_ERR_INVALID_ARG;
  // Two query tiles an item, unless that takes the SMs over a third more tile
  // times.  Measured alone and in pairs, 128 columns a head, 512 keys: one wave of
  // tiles against two 11.4 and 13.2 us, two and two 16.9 and 14.4, three and four
  // 22.2 and 21.3, eight and eight 48.7 and 37.4 (64 columns, 1500 keys: three and
  // four 33.3 and 36.2, eight and eight 79.0 and 69.7).
  const long long columns = (long long)d.batch * p.head_blocks, sms = device_sms();
  const long long waves1 = (columns * p.n_qtiles + sms - 1) / sms;
  const long long waves2 = 2 * ((columns * ((p.n_qtiles + 1) / 2) + sms - 1) / sms);
  p.pair = 3 * waves2 <= 4 * waves1 ? 2 : 1;
  p.items = (unsigned)(columns * ((p.n_qtiles + p.pair - 1) / p.pair));
  p.splits = p.pair == 2 ? 1 : cross_splits(p.items, (d.kv_tokens + kTileN - 1) / kTileN);
  p.sorted = cross_sorted(d, q_len, kv_len, p.items);
  forge_items(p);
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.err_word = device_error_word();
  if (!encode_query_rows(&p.q_map, Q, d.batch, d.q_tokens, d.heads, d.head_dim, p.pack, p.tile_tokens) ||
      !encode_query_rows(&p.o_map, O, d.batch, d.q_tokens, d.heads, d.head_dim, p.pack, p.tile_tokens) ||
      !encode_key_rows(&p.k_map, K, d.kv_batch, d.kv_tokens, d.kv_heads, d.head_dim) ||
      !encode_key_rows(&p.v_map, V, d.kv_batch, d.kv_tokens, d.kv_heads, d.head_dim))
    return SAB_ERR_CUDA;
  return launch_cross_forward(p, device_sms(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK
                                                                                              : SAB_ERR_CUDA;
}

// Blocks among which the queries of a key tile are cut: those that take the
// fewest waves of blocks times tiles, where a block begins and ends in about the
// time of 3 tiles and parts that have to be added cost 4 more.
static int cross_shares(long long units, long long tiles) {
  const long long sms = device_sms();
  int best = 1;
  double least = 0.0;
  for (int n = 1; n <= 64 && n <= tiles; ++n) {
    const double cost =
        (double)((units * n + sms - 1) / sms) * (double)((tiles + n - 1) / n + 3) + (n > 1 ? 4.0 + 0.05 * n : 0.0);
    if (n == 1 || cost < least) best = n, least = cost;
  }
  return best;
}
struct CrossBackPlan {
  int pack, tile_tokens, n_qtiles, shares;
  long long units;
  size_t delta_bytes, part_bytes;
};
static CrossBackPlan cross_back_plan(const sab_cross_desc& d) {
  CrossBackPlan b;
  const int group = d.heads / d.kv_heads;
  b.pack = cross_pack(d.q_tokens, group, kTileM);
  b.tile_tokens = kTileM / b.pack;
  b.n_qtiles = (d.q_tokens + b.tile_tokens - 1) / b.tile_tokens;
  b.units = (long long)((d.kv_tokens + kTileN - 1) / kTileN) * d.kv_heads * d.kv_batch;
  const long long tiles = (long long)(d.batch / d.kv_batch) * (group / b.pack) * b.n_qtiles;
  b.shares = cross_shares(b.units, tiles);
  b.delta_bytes = align_up((size_t)d.batch * d.heads * d.q_tokens * sizeof(float), kAlign);
  b.part_bytes =
      b.shares == 1 ? 0 : align_up((size_t)b.shares * b.units * 2 * kTileN * d.head_dim * sizeof(float), kAlign);
  return b;
}

size_t sab_cross_attention_backward_workspace(const sab_cross_desc* desc) {
  if (!cross_shape_ok(desc)) return 0;
  const CrossBackPlan b = cross_back_plan(*desc);
  return b.delta_bytes + b.part_bytes;
}

sab_status sab_cross_attention_backward(const sab_cross_desc* desc, const sab_token_rows* Q, const sab_token_rows* K,
                                        const sab_token_rows* V, const sab_token_rows* O, const sab_token_rows* dO,
                                        const float* LSE, const int* q_len, const int* kv_len, float softmax_scale,
                                        const sab_token_rows* dQ, const sab_token_rows* dK, const sab_token_rows* dV,
                                        void* workspace, size_t ws_bytes, void* stream) {
  if (!cross_shape_ok(desc) || !cross_scale_ok(softmax_scale)) return SAB_ERR_INVALID_ARG;
  const sab_cross_desc& d = *desc;
  const int B = d.batch, L = d.q_tokens, H = d.heads, Hk = d.kv_heads, D = d.head_dim;
  const sab_token_rows* in[] = {Q, O, dO, K, V};
  const sab_token_rows* out[] = {dQ, dK, dV};
  for (int i = 0; i < 5; ++i)
    if (!(i < 3 ? token_rows_ok(in[i], B, L, H, D, false)
                : token_rows_ok(in[i], d.kv_batch, d.kv_tokens, Hk, D, false)))
      return SAB_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i) {
    if (!(i < 1 ? token_rows_ok(out[i], B, L, H, D, true)
                : token_rows_ok(out[i], d.kv_batch, d.kv_tokens, Hk, D, true)))
      return SAB_ERR_INVALID_ARG;
    for (const sab_token_rows* x : in)
      if (x->data == out[i]->data) return SAB_ERR_INVALID_ARG;
    for (int k = 0; k < i; ++k)
      if (out[k]->data == out[i]->data) return SAB_ERR_INVALID_ARG;
  }
  if (LSE == nullptr || !aligned16(LSE) || !aligned4(q_len) || !aligned4(kv_len)) return SAB_ERR_INVALID_ARG;
  const CrossBackPlan b = cross_back_plan(d);
  if (!cross_tiles_ok(d, q_len, kv_len, (long long)(H / b.pack) * b.n_qtiles)) return SAB_ERR_INVALID_ARG;
  if (workspace == nullptr || ws_bytes < b.delta_bytes + b.part_bytes ||
      (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0)
    return SAB_ERR_WORKSPACE;
  CrossBwdParams p;
  memset(&p, 0, sizeof(p));
  p.q_len = q_len;
  p.kv_len = kv_len;
  p.LSE = const_cast<float*>(LSE);
  p.B = d.batch;
  p.Bk = d.kv_batch;
  p.Lq = d.q_tokens;
  p.Lk = d.kv_tokens;
  p.H = d.heads;
  p.Hk = d.kv_heads;
  p.D = d.head_dim;
  p.group = d.heads / d.kv_heads;
  p.pack = b.pack;
  p.tile_tokens = b.tile_tokens;
  p.n_qtiles = b.n_qtiles;
  p.head_blocks = d.heads / p.pack;
  p.pair = 1;
  p.items = (unsigned)((long long)d.batch * p.head_blocks * p.n_qtiles);
  p.splits = 1;
  p.sorted = cross_sorted(d, q_len, kv_len, p.items);
  p.forged = forge_items(p) ? 1 : 0;
  p.shares = b.shares;
  p.scale = softmax_scale;
  p.scale_log2 = softmax_scale * 1.4426950408889634f;
  p.delta = static_cast<float*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + b.delta_bytes);
  p.O = static_cast<uint16_t*>(O->data);  // read
  p.o_batch = batch_of(O, d.batch, d.heads, D);
  p.o_token = token_of(O, d.q_tokens, d.heads, D);
  p.o_head = head_of(O, d.heads, D);
  p.dK = static_cast<uint16_t*>(dK->data);
  p.dV = static_cast<uint16_t*>(dV->data);
  p.dk_batch = batch_of(dK, d.kv_batch, Hk, D);
  p.dk_token = token_of(dK, d.kv_tokens, Hk, D);
  p.dk_head = head_of(dK, Hk, D);
  p.dv_batch = batch_of(dV, d.kv_batch, Hk, D);
  p.dv_token = token_of(dV, d.kv_tokens, Hk, D);
  p.dv_head = head_of(dV, Hk, D);
  p.err_word = device_error_word();
  if (!encode_query_rows(&p.q_map, Q, B, L, H, D, p.pack, p.tile_tokens) ||
      !encode_query_rows(&p.do_map, dO, B, L, H, D, p.pack, p.tile_tokens) ||
      !encode_query_rows(&p.of_map, O, B, L, H, D, p.pack, p.tile_tokens) ||
      !encode_query_rows(&p.o_map, dQ, B, L, H, D, p.pack, p.tile_tokens) ||
      !encode_key_rows(&p.k_map, K, d.kv_batch, d.kv_tokens, d.kv_heads, D) ||
      !encode_key_rows(&p.v_map, V, d.kv_batch, d.kv_tokens, d.kv_heads, D))
    return SAB_ERR_CUDA;
  return launch_cross_backward(p, device_sms(), static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK
                                                                                               : SAB_ERR_CUDA;
}

// ------------------------------------------------------------------ layer norm

// The most row ranges of a group whose sums a layer norm's gradients may keep
// apart (the launcher takes one wave of blocks or fewer): about ten blocks for
// every SM over all groups, none of fewer than 8 rows.
struct NormCut {
  long long groups;
  int splits;
};
static NormCut norm_cut(long long rows, long long group_rows) {
  NormCut n;
  if (group_rows > rows) group_rows = rows;
  n.groups = (rows + group_rows - 1) / group_rows;
  n.splits = (int)std::max(1LL, std::min(10LL * device_sms() / n.groups, group_rows / 8));
  return n;
}
static bool norm_shape_ok(long long rows, int channels, long long group_rows) {
  return rows >= 1 && rows <= 0x7fffffffLL && channels >= 1 && channels <= SAB_NORM_MAX_CHANNELS && group_rows >= 1;
}
static bool norm_stride_ok(long long stride, long long rows, int channels, bool out) {
  if (stride < 0 || (rows > 1 && stride > (1LL << 47) / rows)) return false;
  return !out || rows == 1 || stride >= channels;
}

// What the two directions share; `io` are the tensors of the rows' type.
static sab_status norm_common(const sab_norm_desc* d, const void* const* io, const long long* strides, int n,
                              const void* const* f32, int nf, NormParams& p, int& access) {
  if (d == nullptr || !norm_shape_ok(d->rows, d->channels, d->group_rows)) return SAB_ERR_INVALID_ARG;
  if (d->dtype != SAB_DTYPE_BF16 && d->dtype != SAB_DTYPE_FP32) return SAB_ERR_INVALID_ARG;
  if (!(d->eps > 0.f) || !isfinite(d->eps) || !isfinite(d->weight_offset)) return SAB_ERR_INVALID_ARG;
  const uintptr_t es = d->dtype == SAB_DTYPE_BF16 ? 2 : 4;
  uintptr_t low = d->channels * es;  // its lowest bits, or-ed together: what all divide
  for (int i = 0; i < n; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(io[i]);
    if (a == 0 || a % es != 0 || !norm_stride_ok(strides[i], d->rows, d->channels, i == n - 1))
      return SAB_ERR_INVALID_ARG;
    low |= a | (uintptr_t)strides[i] * es;
  }
  for (int i = 0; i + 1 < n; ++i)  // in place: the same rows
    if (io[i] == io[n - 1] && strides[i] != strides[n - 1] && d->rows > 1) return SAB_ERR_INVALID_ARG;
  for (int i = 0; i < nf; ++i) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(f32[i]);
    if (a % 4 != 0) return SAB_ERR_INVALID_ARG;
    low |= a;
  }
  access = low % 16 == 0 ? 16 : low % 4 == 0 ? 4 : 2;
  memset(&p, 0, sizeof(p));
  const NormCut cut = norm_cut(d->rows, d->group_rows);
  p.rows = d->rows;
  p.group_rows = std::min(d->group_rows, d->rows);
  p.groups = cut.groups;
  p.splits = cut.splits;
  p.C = d->channels;
  p.inv_c = 1.f / (float)d->channels;
  p.eps = d->eps;
  p.offset = d->weight_offset;
  return SAB_OK;
}

sab_status sab_layer_norm(const sab_norm_desc* desc, const void* X, long long x_stride, const float* weight,
                          const float* bias, void* Y, long long y_stride, float* mean, float* rstd, void* stream) {
  const void* io[] = {X, Y};
  const long long strides[] = {x_stride, y_stride};
  const void* f32[] = {weight, bias};
  NormParams p;
  int access = 0;
  const sab_status st = norm_common(desc, io, strides, 2, f32, 2, p, access);
  if (st != SAB_OK) return st;
  if (!aligned4(mean) || !aligned4(rstd)) return SAB_ERR_INVALID_ARG;
  p.x = X;
  p.x_row = x_stride;
  p.y = Y;
  p.y_row = y_stride;
  p.weight = weight;
  p.bias = bias;
  p.mean = mean;
  p.rstd = rstd;
  const cudaError_t e = launch_layer_norm(p, desc->dtype == SAB_DTYPE_FP32, access, false, device_sms(),
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

size_t sab_layer_norm_backward_workspace(long long rows, int channels, long long group_rows) {
  if (!norm_shape_ok(rows, channels, group_rows)) return 0;
  const NormCut n = norm_cut(rows, group_rows);
  return n.splits == 1 ? 0 : align_up((size_t)n.groups * n.splits * 2 * channels * sizeof(float), kAlign);
}

sab_status sab_layer_norm_backward(const sab_norm_desc* desc, const void* X, long long x_stride, const void* dY,
                                   long long dy_stride, const float* weight, const float* mean, const float* rstd,
                                   void* dX, long long dx_stride, float* dweight, float* dbias, void* workspace,
                                   size_t ws_bytes, void* stream) {
  const void* io[] = {X, dY, dX};
  const long long strides[] = {x_stride, dy_stride, dx_stride};
  const void* f32[] = {weight, dweight, dbias};
  NormParams p;
  int access = 0;
  const sab_status st = norm_common(desc, io, strides, 3, f32, 3, p, access);
  if (st != SAB_OK) return st;
  if (mean == nullptr || rstd == nullptr || !aligned4(mean) || !aligned4(rstd)) return SAB_ERR_INVALID_ARG;
  if (dweight != nullptr && dweight == dbias) return SAB_ERR_INVALID_ARG;
  const bool sums = dweight != nullptr || dbias != nullptr;
  const size_t need = sums ? sab_layer_norm_backward_workspace(desc->rows, desc->channels, desc->group_rows) : 0;
  if (need > 0 && (workspace == nullptr || ws_bytes < need || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0))
    return SAB_ERR_WORKSPACE;
  p.x = X;
  p.x_row = x_stride;
  p.dy = dY;
  p.dy_row = dy_stride;
  p.y = dX;
  p.y_row = dx_stride;
  p.weight = weight;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dweight = dweight;
  p.dbias = dbias;
  p.part = static_cast<float*>(workspace);
  const cudaError_t e = launch_layer_norm(p, desc->dtype == SAB_DTYPE_FP32, access, true, device_sms(),
                                          static_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? SAB_OK : SAB_ERR_CUDA;
}

sab_status sab_selftest_split_abort(const sab_ring* ring, int layer, long long chunk, const void* Q,
                                    const void* K_cur, const void* V_cur, int window, int use_sink, int num_splits,
                                    float softmax_scale, void* O, float* LSE, void* workspace, size_t ws_bytes,
                                    int abort_split, void* stream) {
  if (num_splits < 2 || num_splits > kMaxSplits) return SAB_ERR_INVALID_ARG;
  if (abort_split < 0 || abort_split >= num_splits) return SAB_ERR_INVALID_ARG;
  AttnParams p;
  const sab_status st =
      plan_chunk_attention(ring, layer, chunk, Q, K_cur, V_cur, window, use_sink, num_splits, softmax_scale, O, LSE, p);
  if (st != SAB_OK) return st;
  p.inject_abort = abort_split + 1;
  return launch_attention(p, ring->d.chunk_tokens, num_splits, workspace, ws_bytes, stream);
}

sab_status sab_selftest_bounded_wait(unsigned long long timeout_ns, void* stream) {
  if (timeout_ns < 1000000ull || timeout_ns > 2000000000ull) return SAB_ERR_INVALID_ARG;
  return launch_wait_timeout_probe(timeout_ns, static_cast<cudaStream_t>(stream)) == cudaSuccess ? SAB_OK
                                                                                                : SAB_ERR_CUDA;
}

sab_status sab_get_last_device_error(void* stream) {
  if (cudaStreamSynchronize(static_cast<cudaStream_t>(stream)) != cudaSuccess) return SAB_ERR_CUDA;
  unsigned v = 0;
  if (read_and_clear_device_error(&v) != cudaSuccess) return SAB_ERR_CUDA;
  if (v & kErrBoundsBit) return SAB_ERR_BOUNDS;
  return v ? SAB_ERR_TIMEOUT : SAB_OK;
}

int sab_debug_bounds_enabled(void) { return kDebugBounds ? 1 : 0; }

sab_status sab_debug_inject_bounds_error(int what) {
  if (!kDebugBounds) return SAB_ERR_UNSUPPORTED;
  if (what < 0 || what > SAB_DEBUG_INJECT_CROSS_ITEM) return SAB_ERR_INVALID_ARG;
  g_inject.store(what);
  return SAB_OK;
}

const char* sab_status_string(sab_status status) {
  switch (status) {
    case SAB_OK: return "SAB_OK";
    case SAB_ERR_INVALID_ARG: return "SAB_ERR_INVALID_ARG";
    case SAB_ERR_UNSUPPORTED: return "SAB_ERR_UNSUPPORTED";
    case SAB_ERR_OUT_OF_RANGE: return "SAB_ERR_OUT_OF_RANGE";
    case SAB_ERR_WORKSPACE: return "SAB_ERR_WORKSPACE";
    case SAB_ERR_CUDA: return "SAB_ERR_CUDA";
    case SAB_ERR_TIMEOUT: return "SAB_ERR_TIMEOUT";
    case SAB_ERR_BOUNDS: return "SAB_ERR_BOUNDS";
  }
  return "SAB_ERR_UNKNOWN";
}

const char* sab_version(void) { return "sab 0.1.0 (sm_103a)"; }

}  // extern "C"
