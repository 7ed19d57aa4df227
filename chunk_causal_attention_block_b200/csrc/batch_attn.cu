// wf_batch_attn: attention of a batch of requests that share a prefix, over a
// paged K/V pool (bf16, head_dim 64 or 128, tcgen05 + TMEM + TMA).
//
// Row (t, h) of request b, key head h / group, sees the prefix's keys and b's
// own keys [0, min(len_b, (x / G + 1) G)) for own position x and block G
// (1: token-causal; the chunk length: chunk-causal):
//   O = softmax(q K^T * scale) V,  LSE = ln sum exp(q K^T * scale).
//
// Work.  A unit is up to two 128-row tiles (tokens x group rows of one key
// head, so a K/V tile is read once for a whole group) against a list of
// 128-key tiles.  Rows of a request that fill half a tile or more run the
// prefix's tiles and their own in one unit.  Rows of smaller requests are
// packed across requests for the prefix (each prefix key is then read once
// for the whole batch) and run their own keys in units of their own.  The
// units of all heads form one line of costs (the work list of
// wf_batch_tables) that is cut into equal shares, one per CTA, wherever the
// cut falls; parts of a row's keys leave normalised fp32 rows and their LSE
// in the workspace and batch_combine_kernel merges them in a fixed order.
//
// Pipeline.  The kernel runs a sequence of subtiles (row tile, key tile), the
// m-th on stream m mod 2.  A stream is a softmax warpgroup with its own S and
// O in TMEM.  Two-tile units alternate their row tiles over the same K/V
// tile; one-tile units alternate key tiles, so that short shares keep both
// streams busy too, also across units.  Step m of the MMA thread issues
// PV(m-2) and S(m), both on stream m mod 2; the commit that announces S(m)
// covers PV(m-2), so the softmax owns O when it sees S.  The online softmax
// is the one of attn_sm100.cu (log2 domain, reference raised only when a
// row's maximum grows by more than 2^8).
//
// Warp roles (384 threads; registers as in attn_sm100.cu):
//   warps 0-3, 4-7  softmax of stream 0 and 1
//   warp  8   MMA issue (lane 0), TMEM allocation
//   warp  9   TMA producer: Q tiles (ring of two), K/V pages (ring of kStages)
//   warp 10   scheduler: walks this CTA's share and publishes items
//   warp 11   zeroes the V rows behind a list's last key, whatever the page
//             holds there (0 * NaN would reach O), before the PV MMA
//
// Every wait is bounded; on expiry the status word is set, all roles return,
// the producer waits for its copies in flight, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cmath>
#include <cstdint>
#include <cstdlib>

#include "sm100_ptx.cuh"
#include "wf_batch.h"

namespace wf {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kSoftmaxRegs = 224;
constexpr uint32_t kControlRegs = 56;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs == kThreads * 168, "register split must match launch");
constexpr int kHalfBytes = 128 * 128;  // 128 rows x 64 bf16, 128-byte swizzled
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kItems = 4;

enum Dest { kDirect = 0, kMainOwn = 1, kMainPrefix = 2, kCutHead = 3, kCutTail = 4 };

// One share of a unit for one key head, published by the scheduler.
struct Item {
  int32_t j0, j1;   // key tiles; j1 = 0: no more items
  int32_t head;     // key head
  int32_t req, tok0, ntok, ptiles, cbase, pos0, len;  // of the unit (ptiles >= 0)
  int32_t parity;   // stream of the item's first subtile
  int32_t dest;
};
static_assert(sizeof(Item) == 48, "item layout");

struct Params {
  const wf_batch_hdr* hdr;
  const wf_batch_unit* units;
  const int64_t* pre;
  const int32_t* ctok;
  const int32_t* table;
  const int32_t* prefix_table;
  __nv_bfloat16* out;
  float* lse;
  wf_dev_status* status;
  float* main_o;
  float* cut_o;
  float* main_lse;
  float* cut_lse;
  uint64_t fingerprint;
  uint64_t timeout_ns;
  float scale_log2;
  int32_t H, kv_heads, group, tile_tokens;
  int32_t cols, page_shift, block_tokens, max_tokens, max_ctok;
};

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kHalfBytes;
  static constexpr int kStages = D == 128 ? 5 : 8;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
  // barriers
  static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6, kOFull = 8, kItemFull = 10;
  static constexpr int kItemEmpty = kItemFull + kItems;
  static constexpr int kMmaDone = kItemEmpty + kItems;
  static constexpr int kKVFull = kMmaDone + 1;
  static constexpr int kKVEmpty = kKVFull + kStages;
  static constexpr int kVRaw = kKVEmpty + kStages;  // a V tile has landed whose last rows are still to be zeroed
  static constexpr int kNumBars = kVRaw + kStages;
  static constexpr int kTail = 8 * kNumBars + 16 + kItems * int(sizeof(Item));
  static constexpr int kSmemBytes = 1024 + (2 + kStages) * kTile + (kTail + 127) / 128 * 128;
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};
// softmax warps (8), MMA, producer, zeroing warp
constexpr uint32_t kItemReaders = 11;

struct Shared {
  uint8_t* base;  // two Q tiles, then the K/V stages; 1024-aligned
  uint64_t* bars;
  uint32_t* tmem_slot;
  int32_t* abort_flag;
  Item* items;
};

template <int D>
__device__ __forceinline__ Shared carve_smem(uint8_t* raw) {
  Shared s;
  s.base = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023));
  uint8_t* tail = s.base + (2 + Cfg<D>::kStages) * Cfg<D>::kTile;
  s.items = reinterpret_cast<Item*>(tail);
  s.bars = reinterpret_cast<uint64_t*>(tail + kItems * sizeof(Item));
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.bars + Cfg<D>::kNumBars);
  s.abort_flag = reinterpret_cast<int32_t*>(s.tmem_slot + 1);
  return s;
}

template <int D>
__device__ __forceinline__ uint8_t* q_tile(const Shared& s, int slot) {
  return s.base + slot * Cfg<D>::kTile;
}
template <int D>
__device__ __forceinline__ uint8_t* kv_tile(const Shared& s, int st) {
  return s.base + (2 + st) * Cfg<D>::kTile;
}

// Bounded wait; false if the CTA is aborting.  The first expiry records where.
__device__ __forceinline__ bool wait_bar(const Shared& sh, const Params& p, int bar, uint32_t parity, int where) {
  const uint32_t addr = smem_u32(sh.bars + bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  for (;;) {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(addr, parity)) return true;
    if (*reinterpret_cast<volatile int32_t*>(sh.abort_flag)) return false;
    if (global_timer_ns() - t0 > p.timeout_ns) {
      *reinterpret_cast<volatile int32_t*>(sh.abort_flag) = 1;
      if (atomicCAS(&p.status->code, 0, int32_t(WF_ERR_DEVICE_TIMEOUT)) == 0) {
        p.status->where = where;
        p.status->block = int32_t(blockIdx.x);
        p.status->thread = int32_t(threadIdx.x);
        __threadfence();
      }
      return false;
    }
  }
}

__device__ __forceinline__ bool warp_wait(const Shared& sh, const Params& p, int bar, uint32_t parity, int where) {
  return __all_sync(0xffffffffu, wait_bar(sh, p, bar, parity, where));
}

// ---------------------------------------------------------------- shares of the line of costs
__device__ __forceinline__ int64_t share_begin(int c, int64_t total, int ctas) { return int64_t(c) * total / ctas; }

// The share that holds cost position x.
__device__ __forceinline__ int share_of(int64_t x, int64_t total, int ctas) {
  return int(((x + 1) * ctas + total - 1) / total) - 1;
}

// Key tiles of a unit at cost position s (cost w per tile) that start inside [lo, hi).
__device__ __forceinline__ void share_tiles(int64_t s, int32_t w, int32_t ktiles, int64_t lo, int64_t hi, int32_t& j0,
                                            int32_t& j1) {
  const int64_t a = lo <= s ? 0 : (lo - s + w - 1) / w, b = hi <= s ? 0 : (hi - s + w - 1) / w;
  j0 = int32_t(a < ktiles ? a : ktiles);
  j1 = int32_t(b < ktiles ? b : ktiles);
}

__device__ __forceinline__ int32_t tile_cost(int32_t ntok, int32_t tile_tokens) {
  return ntok > tile_tokens ? WF_BATCH_PAIR_COST : WF_BATCH_SINGLE_COST;
}

// Whether rows of this unit run no other key tiles than the unit's, and on one
// stream: an uncut unit then writes its output rows itself.
__device__ __forceinline__ bool unit_direct(const wf_batch_unit& u, int32_t tile_tokens) {
  return u.req >= 0 && u.ptiles >= 0 && (u.ntok > tile_tokens || u.ktiles == 1);
}

// ---------------------------------------------------------------- item ring
// Copies item `it` and gives its slot back; false at the end (or on an abort).
// Called by whole warps, and with kLane by one lane alone.
template <int D, bool kLane = false>
__device__ __forceinline__ bool take_item(const Shared& sh, const Params& p, int it, Item& x, int where) {
  const int bar = Cfg<D>::kItemFull + it % kItems;
  const uint32_t parity = (it / kItems) & 1;
  if (!(kLane ? wait_bar(sh, p, bar, parity, where) : warp_wait(sh, p, bar, parity, where))) return false;
  x = sh.items[it % kItems];
  if (!kLane) __syncwarp();
  if (kLane || (threadIdx.x & 31) == 0) mbar_arrive(smem_u32(sh.bars + Cfg<D>::kItemEmpty + it % kItems));
  return x.j1 > 0;
}

template <int D>
__device__ __forceinline__ void scheduler(const Shared& sh, const Params& p) {
  const int lane = threadIdx.x & 31;
  int it = 0;
  int32_t parity = 0;
  const wf_batch_hdr* h = p.hdr;
  const int64_t head_cost = h->head_cost, total = head_cost * p.kv_heads;
  const int ctas = h->ctas, units = h->units;
  const int c = int(blockIdx.x);
  if (h->fingerprint == p.fingerprint && total > 0 && c < ctas) {
    const int64_t lo = share_begin(c, total, ctas), hi = share_begin(c + 1, total, ctas);
    int32_t head = int32_t(lo / head_cost);
    // first unit: the last one that starts at or before lo, found 32 probes at a time
    const int64_t rem = lo - int64_t(head) * head_cost;
    int32_t a = 0, b = units;
    while (b - a > 1) {
      const int32_t step = (b - a + 31) / 32, probe = a + lane * step;
      const uint32_t le = __ballot_sync(0xffffffffu, probe < b && __ldg(p.pre + probe) <= rem);
      const int k = 31 - __clz(le);  // lane 0 always holds: pre[a] <= rem
      a = a + k * step;
      b = min(b, a + step);
    }
    int32_t u = a;
    bool more = true;
    while (more) {
      // 32 units at a time, one per lane
      const int32_t mine = u + lane;
      wf_batch_unit r{};
      int64_t s = 0;
      if (mine < units) {
        const int4* src = reinterpret_cast<const int4*>(p.units + mine);
        reinterpret_cast<int4*>(&r)[0] = __ldg(src);
        reinterpret_cast<int4*>(&r)[1] = __ldg(src + 1);
        s = int64_t(head) * head_cost + __ldg(p.pre + mine);
      }
      int32_t j0 = 0, j1 = 0;
      const int32_t w = tile_cost(r.ntok, p.tile_tokens);
      if (mine < units) share_tiles(s, w, r.ktiles, lo, hi, j0, j1);
      const uint32_t live = __ballot_sync(0xffffffffu, mine < units && j0 < j1);
      more = __all_sync(0xffffffffu, mine >= units || s < hi);
      uint32_t todo = live;
      while (todo) {
        const int src = __ffs(todo) - 1;
        todo &= todo - 1;
        const int32_t n = __shfl_sync(0xffffffffu, (j1 - j0) * (r.ntok > p.tile_tokens ? 2 : 1), src);
        if (!warp_wait(sh, p, Cfg<D>::kItemEmpty + it % kItems, ((it / kItems) & 1) ^ 1, 40)) return;
        if (lane == src) {
          Item x;
          x.j0 = j0;
          x.j1 = j1;
          x.head = head;
          x.req = r.req;
          x.tok0 = r.tok0;
          x.ntok = r.ntok;
          x.ptiles = r.ptiles < 0 ? 0 : r.ptiles;
          x.cbase = r.cbase;
          x.pos0 = r.pos0;
          x.len = r.len;
          x.parity = parity;
          x.dest = j0 > 0                          ? kCutHead
                   : j1 < r.ktiles                 ? kCutTail
                   : unit_direct(r, p.tile_tokens) ? kDirect
                   : r.req < 0                     ? kMainPrefix
                                                   : kMainOwn;
          sh.items[it % kItems] = x;
          mbar_arrive(smem_u32(sh.bars + Cfg<D>::kItemFull + it % kItems));
        }
        __syncwarp();
        parity = (parity + n) & 1;
        ++it;
      }
      u += 32;
      if (u >= units) {
        u = 0;
        if (++head >= p.kv_heads) more = false;
        // the next head's first unit starts where this head ends
        if (int64_t(head) * head_cost >= hi) more = false;
      }
    }
  }
  if (!warp_wait(sh, p, Cfg<D>::kItemEmpty + it % kItems, ((it / kItems) & 1) ^ 1, 41)) return;
  if (lane == 0) {
    Item x{};
    sh.items[it % kItems] = x;
    mbar_arrive(smem_u32(sh.bars + Cfg<D>::kItemFull + it % kItems));
  }
}

// ---------------------------------------------------------------- K/V tiles
// Key tile j of an item: where its pages are listed and how many keys it holds.
struct KeyTile {
  int32_t head;
  int32_t valid;   // keys, at most 128
  int32_t own;     // 1: block table, 0: prefix table
  int64_t entry;   // first page's entry there
};

__device__ __forceinline__ KeyTile key_tile(const Params& p, const Item& x, int32_t j, int32_t prefix_len) {
  KeyTile k;
  k.head = x.head;
  k.own = j >= x.ptiles;
  const int32_t base = (k.own ? j - x.ptiles : j) * 128;
  const int32_t left = (k.own ? x.len : prefix_len) - base;
  k.valid = left < 128 ? left : 128;
  k.entry = (k.own ? int64_t(x.req) * p.cols : 0) + (base >> p.page_shift);
  return k;
}

// The whole warp copies a tile's pages, one (page, 64-column half) per lane and
// round; only pages that hold keys are read.
template <int D>
__device__ __forceinline__ void load_tile(const Shared& sh, const Params& p, const CUtensorMap* tm, const KeyTile& k,
                                          int st, int bar_index) {
  const int lane = threadIdx.x & 31;
  const int pages = (k.valid + (1 << p.page_shift) - 1) >> p.page_shift;
  const uint32_t page_bytes = 128u << p.page_shift;  // of one half
  const uint32_t bar = smem_u32(sh.bars + bar_index);
  if (lane == 0) mbar_arrive_expect_tx(bar, uint32_t(pages) * page_bytes * Cfg<D>::kHalves);
  __syncwarp();
  const int32_t* list = k.own ? p.table : p.prefix_table;
  const uint32_t dst = smem_u32(kv_tile<D>(sh, st));
  for (int i = lane; i < pages * Cfg<D>::kHalves; i += 32) {
    const int pg = i / Cfg<D>::kHalves, half = i % Cfg<D>::kHalves;
    // an entry outside the pool reads zeros, not memory: the map's bounds hold
    const int64_t tok = int64_t(__ldg(list + k.entry + pg)) << p.page_shift;
    const int32_t at = tok < 0 || tok > 0x7FFFFF00 ? 0x7FFFFF00 : int32_t(tok);
    tma_load_3d(dst + half * kHalfBytes + pg * page_bytes, tm, bar, 64 * half, k.head, at);
  }
}

// The K/V ring is filled and used in one order, which the producer, the MMA
// thread and the zeroing warp each follow: at step m the V tile of subtile m-2
// (if that subtile is the first on its tile), then the K tile of subtile m
// (likewise).
template <int D>
__device__ __forceinline__ void producer(const Shared& sh, const Params& p, const CUtensorMap* tm_q,
                                         const CUtensorMap* tm_k, const CUtensorMap* tm_v) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int32_t prefix_len = p.hdr->prefix_len;
  int kv_it = 0, q_it = 0;
  uint32_t raw_phase = 0, raw_last = 0;  // per stage: parity of the next raw fill; last fill was raw
  bool ok = true;
  KeyTile v1{}, v2{};                    // V tiles of the last and the second last subtile
  bool has1 = false, has2 = false;
  const uint32_t q_bytes = uint32_t(p.tile_tokens * p.group) * 128 * C::kHalves;

  auto fill = [&](const CUtensorMap* tm, const KeyTile& k, bool is_v) -> bool {
    const int st = kv_it % C::kStages;
    if (!warp_wait(sh, p, C::kKVEmpty + st, ((kv_it / C::kStages) & 1) ^ 1, 2)) return false;
    const bool raw = is_v && k.valid < 128;
    load_tile<D>(sh, p, tm, k, st, raw ? C::kVRaw + st : C::kKVFull + st);
    raw_last = raw ? raw_last | (1u << st) : raw_last & ~(1u << st);
    if (raw) raw_phase ^= 1u << st;
    ++kv_it;
    return true;
  };

  int it = 0;
  Item x;
  for (; ok && take_item<D>(sh, p, it, x, 1); ++it) {
    const int tiles = x.ntok > p.tile_tokens ? 2 : 1;
    for (int s = 0; s < tiles && ok; ++s, ++q_it) {
      const int slot = q_it & 1;
      if (!warp_wait(sh, p, C::kQEmpty + slot, ((q_it >> 1) & 1) ^ 1, 3)) { ok = false; break; }
      const uint32_t bar = smem_u32(sh.bars + C::kQFull + slot);
      if (lane == 0) mbar_arrive_expect_tx(bar, q_bytes);
      __syncwarp();
      if (lane < C::kHalves)
        tma_load_3d(smem_u32(q_tile<D>(sh, slot)) + lane * kHalfBytes, tm_q, bar, 64 * lane, x.head * p.group,
                    x.tok0 + s * p.tile_tokens);
    }
    for (int j = x.j0; j < x.j1 && ok; ++j) {
      const KeyTile k = key_tile(p, x, j, prefix_len);
      for (int s = 0; s < tiles && ok; ++s) {
        if (has2 && !fill(tm_v, v2, true)) ok = false;
        if (ok && s == 0 && !fill(tm_k, k, false)) ok = false;
        v2 = v1;
        has2 = has1;
        v1 = k;
        has1 = s == 0;
      }
    }
  }
  for (int e = 0; e < 2 && ok && !*reinterpret_cast<volatile int32_t*>(sh.abort_flag); ++e) {
    if (has2 && !fill(tm_v, v2, true)) ok = false;
    v2 = v1;
    has2 = has1;
    has1 = false;
  }
  // The CTA must not exit with copies still landing in its shared memory: wait
  // for the last fill of every stage and Q slot, whoever gave up since.
  for (int st = 0; st < C::kStages; ++st) {
    if (kv_it <= st) continue;
    const bool raw = (raw_last >> st) & 1;
    uint32_t parity = uint32_t((kv_it - 1 - st) / C::kStages) & 1;
    if (raw) parity = ((raw_phase >> st) & 1) ^ 1;
    const uint32_t addr = smem_u32(sh.bars + (raw ? C::kVRaw : C::kKVFull) + st);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(addr, parity) && global_timer_ns() - t0 < p.timeout_ns) {
    }
  }
  for (int b = 0; b < 2; ++b) {
    if (q_it <= b) continue;
    const uint32_t parity = uint32_t((q_it - 1 - b) >> 1) & 1;
    const uint32_t addr = smem_u32(sh.bars + C::kQFull + b);
    const uint64_t t0 = global_timer_ns();
    while (!mbar_try_wait(addr, parity) && global_timer_ns() - t0 < p.timeout_ns) {
    }
  }
}

// Zero the rows behind the last key of ragged V tiles.  Row r of a 64-column
// half is the 128 bytes at r * 128 (the swizzle permutes 16-byte pieces inside
// a row only).
template <int D>
__device__ __forceinline__ void zero_role(const Shared& sh, const Params& p) {
  using C = Cfg<D>;
  const int lane = threadIdx.x & 31;
  const int32_t prefix_len = p.hdr->prefix_len;
  int kv_it = 0;
  uint32_t raw_phase = 0;
  int32_t v1 = 0, v2 = 0;  // valid keys of the V tiles of the last two subtiles; 0: no new tile
  auto pass_v = [&](int32_t valid) -> bool {
    if (valid > 0 && valid < 128) {
      const int st = kv_it % C::kStages;
      if (!warp_wait(sh, p, C::kVRaw + st, (raw_phase >> st) & 1, 50)) return false;
      raw_phase ^= 1u << st;
      const uint32_t base = smem_u32(kv_tile<D>(sh, st));
      const int words = (128 - valid) * 8;  // 16-byte pieces per half
#pragma unroll
      for (int half = 0; half < C::kHalves; ++half)
        for (int i = lane; i < words; i += 32) st_shared_v4(base + half * kHalfBytes + valid * 128 + i * 16, 0, 0, 0, 0);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(sh.bars + C::kKVFull + st));
    }
    kv_it += valid > 0;
    return true;
  };
  Item x;
  for (int it = 0; take_item<D>(sh, p, it, x, 51); ++it) {
    const int tiles = x.ntok > p.tile_tokens ? 2 : 1;
    for (int j = x.j0; j < x.j1; ++j) {
      const int32_t valid = key_tile(p, x, j, prefix_len).valid;
      for (int s = 0; s < tiles; ++s) {
        if (!pass_v(v2)) return;
        kv_it += s == 0;
        v2 = v1;
        v1 = s == 0 ? valid : 0;
      }
    }
  }
  if (*reinterpret_cast<volatile int32_t*>(sh.abort_flag)) return;
  if (!pass_v(v2)) return;
  pass_v(v1);
}

// ---------------------------------------------------------------- MMA issue
// Descriptor offsets as immediates, fully unrolled (attn_sm100.cu measures why).
template <int D, int kk>
__device__ __forceinline__ void issue_s_slice(uint32_t s_tmem, uint64_t qd, uint64_t kd) {
  constexpr uint32_t off = uint32_t(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
  mma_ss_off<off, off>(s_tmem, qd, kd, Cfg<D>::kIdescQK, kk > 0 ? 1u : 0u);
  if constexpr (kk + 1 < D / 16) issue_s_slice<D, kk + 1>(s_tmem, qd, kd);
}

template <int D, int kk>
__device__ __forceinline__ void issue_pv_slice(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t acc0) {
  mma_ts_off<kk * 8, uint32_t((kk * 2048) >> 4)>(o_tmem, p_tmem, vd, Cfg<D>::kIdescPV, kk > 0 ? 1u : acc0);
  if constexpr (kk < 7) issue_pv_slice<D, kk + 1>(o_tmem, p_tmem, vd, acc0);
}

// What a pending PV product needs to know of its subtile.
constexpr uint32_t kPvLive = 1, kPvFirst = 2, kPvLast = 4, kPvOpens = 8, kPvCloses = 16;

template <int D>
__device__ __forceinline__ void mma_issuer(const Shared& sh, const Params& p, uint32_t tmem) {
  using C = Cfg<D>;
  int kv_it = 0, q_it = 0;
  uint32_t p_phase = 0;  // bit t: parity of stream t's next P
  uint32_t m = 0;        // subtile
  uint32_t pv1 = 0, pv2 = 0;
  int vst = 0;
  bool ok = true;

  // PV of subtile m-2, on stream m & 1
  auto issue_pv = [&](uint32_t pv) -> bool {
    const uint32_t t = m & 1;
    if (pv & kPvOpens) {
      vst = kv_it % C::kStages;
      if (!wait_bar(sh, p, C::kKVFull + vst, (kv_it / C::kStages) & 1, 12)) return false;
      ++kv_it;
    }
    if (!wait_bar(sh, p, C::kPFull + t, (p_phase >> t) & 1, 14 + t)) return false;
    p_phase ^= 1u << t;
    tc_fence_after();
    issue_pv_slice<D, 0>(tmem + 256 + 128 * t, tmem + 128 * t,
                         smem_desc_sw128(smem_u32(kv_tile<D>(sh, vst)), kHalfBytes, 1024), pv & kPvFirst ? 0u : 1u);
    if (pv & kPvLast) mma_commit(smem_u32(sh.bars + C::kOFull + t));
    if (pv & kPvCloses) mma_commit(smem_u32(sh.bars + C::kKVEmpty + vst));
    return true;
  };

  Item x;
  for (int it = 0; ok && take_item<D, true>(sh, p, it, x, 10); ++it) {
    const int tiles = x.ntok > p.tile_tokens ? 2 : 1;
    const int n = x.j1 - x.j0;
    int kst = 0;
    for (int j = 0; j < n && ok; ++j) {
      for (int s = 0; s < tiles; ++s, ++m) {
        const uint32_t t = m & 1;
        if ((pv2 & kPvLive) && !issue_pv(pv2)) { ok = false; break; }
        if (s == 0) {
          kst = kv_it % C::kStages;
          if (!wait_bar(sh, p, C::kKVFull + kst, (kv_it / C::kStages) & 1, 13)) { ok = false; break; }
          ++kv_it;
        }
        const int slot = (q_it + s) & 1;
        if (j == 0 && !wait_bar(sh, p, C::kQFull + slot, ((q_it + s) >> 1) & 1, 11)) { ok = false; break; }
        tc_fence_after();
        issue_s_slice<D, 0>(tmem + 128 * t, smem_desc_sw128(smem_u32(q_tile<D>(sh, slot)), 16, 1024),
                            smem_desc_sw128(smem_u32(kv_tile<D>(sh, kst)), 16, 1024));
        mma_commit(smem_u32(sh.bars + C::kSFull + t));
        if (s == tiles - 1) mma_commit(smem_u32(sh.bars + C::kKVEmpty + kst));
        if (j == n - 1) mma_commit(smem_u32(sh.bars + C::kQEmpty + slot));
        pv2 = pv1;
        // first and last subtile of its stream in this item
        const int step = tiles == 2 ? 1 : 2;
        pv1 = kPvLive | (j < step ? kPvFirst : 0u) | (j + step >= n ? kPvLast : 0u) | (s == 0 ? kPvOpens : 0u) |
              (s == tiles - 1 ? kPvCloses : 0u);
      }
    }
    q_it += tiles;
  }
  for (int e = 0; e < 2 && ok && !*reinterpret_cast<volatile int32_t*>(sh.abort_flag); ++e, ++m) {
    if ((pv2 & kPvLive) && !issue_pv(pv2)) ok = false;
    pv2 = pv1;
    pv1 = 0;
  }
  // all issued MMAs complete before TMEM is released
  mma_commit(smem_u32(sh.bars + C::kMmaDone));
  const uint32_t addr = smem_u32(sh.bars + C::kMmaDone);
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(addr, 0) && global_timer_ns() - t0 < p.timeout_ns) {
  }
}

// ---------------------------------------------------------------- softmax
// exp2(s * sl2 - m) as bf16 pairs into TMEM; returns the fp32 row sum (taken
// before the rounding; P in bf16 feeds the tensor cores).
__device__ __forceinline__ float exp_to_p(const float (&s)[128], float sl2, float m_ref, uint32_t s_tm) {
  const float2 sl2x2 = make_float2(sl2, sl2);
  const float2 negm2 = make_float2(-m_ref, -m_ref);
  float2 ls[4] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
#pragma unroll
  for (int q4 = 0; q4 < 4; ++q4) {
    uint32_t pk[16];
#pragma unroll
    for (int x = 0; x < 16; ++x) {
      const int pi = 16 * q4 + x;
      const float2 v = __ffma2_rn(make_float2(s[2 * pi], s[2 * pi + 1]), sl2x2, negm2);
      const float2 pr = make_float2(fast_exp2(v.x), fast_exp2(v.y));
      ls[x & 3] = __fadd2_rn(ls[x & 3], pr);
      pk[x] = pack_bf16x2(pr.x, pr.y);
    }
    tmem_st16(s_tm + 16 * q4, pk);
  }
  const float2 l01 = __fadd2_rn(ls[0], ls[1]), l23 = __fadd2_rn(ls[2], ls[3]);
  const float2 lt = __fadd2_rn(l01, l23);
  return lt.x + lt.y;
}

template <int D>
__device__ __forceinline__ void softmax_role(const Shared& sh, const Params& p, uint32_t tmem, int t) {
  using C = Cfg<D>;
  const int warp = (threadIdx.x / 32) % 4;
  const int row = warp * 32 + int(threadIdx.x & 31);
  const uint32_t lane_off = uint32_t(warp * 32) << 16;
  const uint32_t s_tm = tmem + lane_off + uint32_t(128 * t);
  const uint32_t o_tm = tmem + lane_off + uint32_t(256 + 128 * t);
  const int32_t prefix_len = p.hdr->prefix_len;
  const int32_t row_tok = row / p.group, row_head = row - row_tok * p.group;
  uint32_t s_phase = 0, o_phase = 0;
  Item x;
  for (int it = 0; take_item<D>(sh, p, it, x, 20 + t); ++it) {
    const bool pair = x.ntok > p.tile_tokens;
    const int32_t tile = pair ? t ^ x.parity : 0;               // row tile of this stream
    const int32_t tok_i = tile * p.tile_tokens + row_tok;        // token inside the unit
    const bool live = row_tok < p.tile_tokens && tok_i < x.ntok;
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int32_t pos = x.pos0 + tok_i;
    // own keys that this row sees
    const int64_t seen = (int64_t(pos) / p.block_tokens + 1) * p.block_tokens;
    const int32_t limit = seen < x.len ? int32_t(seen) : x.len;
    const int step = pair ? 1 : 2;
    float m_ref = -INFINITY;  // reference max (log2 units)
    float l = 0.f;
    bool first = true;
    for (int j = x.j0 + (pair ? 0 : t ^ x.parity); j < x.j1; j += step) {
      if (!warp_wait(sh, p, C::kSFull + t, s_phase, 22 + t)) return;
      s_phase ^= 1;
      if (warp_live) {
        tc_fence_after();
        const int32_t visible = j < x.ptiles ? prefix_len - j * 128 : limit - (j - x.ptiles) * 128;
        float s[128];
        float mxs[8];
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          uint32_t r[32];
          tmem_ld32(s_tm + 32 * q4, r);
#pragma unroll
          for (int c = 0; c < 32; ++c) s[32 * q4 + c] = __uint_as_float(r[c]);
        }
        tmem_wait_ld();
        if (visible < 128) {
#pragma unroll
          for (int c = 0; c < 128; ++c)
            if (c >= visible) s[c] = -INFINITY;
        }
#pragma unroll
        for (int c = 0; c < 8; ++c) mxs[c] = fmaxf(s[c], s[c + 8]);
#pragma unroll
        for (int k = 16; k < 128; k += 16) {
#pragma unroll
          for (int c = 0; c < 8; ++c) mxs[c] = max3f(mxs[c], s[k + c], s[k + 8 + c]);
        }
        const float mx = fmaxf(max3f(mxs[0], mxs[1], mxs[2]), max3f(mxs[3], max3f(mxs[4], mxs[5], mxs[6]), mxs[7]));
        const float m_new = fmaxf(m_ref, mx * p.scale_log2);
        if (first) {
          m_ref = m_new;
        } else {
          const bool need = m_new > m_ref + kRescaleThreshold;
          if (__any_sync(0xffffffffu, need)) {
            const float alpha = need ? fast_exp2(m_ref - m_new) : 1.0f;
#pragma unroll
            for (int q = 0; q < D / 32; ++q) {
              uint32_t r[32];
              tmem_ld32(o_tm + 32 * q, r);
              tmem_wait_ld();
#pragma unroll
              for (int c = 0; c < 32; ++c) r[c] = __float_as_uint(__uint_as_float(r[c]) * alpha);
              tmem_st32(o_tm + 32 * q, r);
            }
            tmem_wait_st();
            if (need) {
              l *= alpha;
              m_ref = m_new;
            }
          }
        }
        // a row that has seen no key yet: every exponent is -inf, P = 0
        l += exp_to_p(s, p.scale_log2, m_ref == -INFINITY ? 0.f : m_ref, s_tm);
        tmem_wait_st();
        tc_fence_before();
      }
      first = false;
      mbar_arrive(smem_u32(sh.bars + C::kPFull + t));
    }
    // epilogue
    const int32_t head = x.head * p.group + row_head;
    const int32_t tok = x.tok0 + tok_i;
    const int32_t part = pair ? tile : t;  // row tile or key parity: which half of a partial slot
    if (first) {
      // no key tile of this item on this stream: a direct item's row is the other stream's
      if (!live || x.dest == kDirect) continue;
    } else {
      if (!warp_wait(sh, p, C::kOFull + t, o_phase, 24 + t)) return;
      o_phase ^= 1;
      tc_fence_after();
    }
    if (!warp_live) continue;
    const float inv_l = l > 0.f ? 1.0f / l : 0.f;
    const float lse_row = l > 0.f ? (m_ref + __log2f(l)) * kLn2 : -INFINITY;
    if (x.dest == kDirect) {
      uint4* dst = reinterpret_cast<uint4*>(p.out + (int64_t(tok) * p.H + head) * D);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t r[32];
        tmem_ld32(o_tm + 32 * q, r);
        tmem_wait_ld();
        if (live) {
#pragma unroll
          for (int v = 0; v < 4; ++v) {
            uint4 w;
            w.x = pack_bf16x2(__uint_as_float(r[8 * v + 0]) * inv_l, __uint_as_float(r[8 * v + 1]) * inv_l);
            w.y = pack_bf16x2(__uint_as_float(r[8 * v + 2]) * inv_l, __uint_as_float(r[8 * v + 3]) * inv_l);
            w.z = pack_bf16x2(__uint_as_float(r[8 * v + 4]) * inv_l, __uint_as_float(r[8 * v + 5]) * inv_l);
            w.w = pack_bf16x2(__uint_as_float(r[8 * v + 6]) * inv_l, __uint_as_float(r[8 * v + 7]) * inv_l);
            dst[4 * q + v] = w;
          }
        }
      }
      if (live && p.lse) p.lse[int64_t(head) * p.max_tokens + tok] = lse_row;
      continue;
    }
    // partial row: normalised O and LSE
    float* po;
    float* pl;
    bool store = live;
    if (x.dest == kMainOwn || x.dest == kMainPrefix) {
      int32_t ct = x.cbase + tok_i;
      if (x.dest == kMainPrefix) ct = live ? __ldg(p.ctok + tok) : -1;
      store = live && ct >= 0;  // a larger request's row in a shared tile has its prefix elsewhere
      const int32_t key_half = pair ? 0 : t;
      const int64_t prow = (int64_t((x.dest == kMainOwn ? 2 : 0) + key_half) * p.max_ctok + (store ? ct : 0)) * p.H + head;
      po = p.main_o + prow * D;
      pl = p.main_lse + prow;
    } else {
      const int64_t prow = ((int64_t(blockIdx.x) * 2 + (x.dest == kCutTail)) * 2 + part) * 128 + row;
      po = p.cut_o + prow * D;
      pl = p.cut_lse + prow;
    }
    if (!first) {
      float4* dst = reinterpret_cast<float4*>(po);
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
        uint32_t r[32];
        tmem_ld32(o_tm + 32 * q, r);
        tmem_wait_ld();
        if (store) {
#pragma unroll
          for (int v = 0; v < 8; ++v)
            dst[8 * q + v] = make_float4(__uint_as_float(r[4 * v]) * inv_l, __uint_as_float(r[4 * v + 1]) * inv_l,
                                         __uint_as_float(r[4 * v + 2]) * inv_l, __uint_as_float(r[4 * v + 3]) * inv_l);
        }
      }
    }
    if (store) *pl = lse_row;
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    batch_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                      const __grid_constant__ CUtensorMap tm_v, const Params p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const Shared sh = carve_smem<D>(smem_raw);
  const int warp = threadIdx.x / 32;
  const int lane = threadIdx.x % 32;

  if (warp == 9 && lane == 0) {
    for (int b = 0; b < C::kNumBars; ++b) {
      uint32_t count = 1;
      if (b == C::kPFull || b == C::kPFull + 1) count = 128;  // a stream's softmax threads
      if (b >= C::kItemEmpty && b < C::kItemEmpty + kItems) count = kItemReaders;
      mbar_init(smem_u32(sh.bars + b), count);
    }
    *sh.abort_flag = 0;
    fence_barrier_init();
    fence_proxy_async_smem();
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.hdr->fingerprint != p.fingerprint)
    p.status->code = WF_ERR_PLAN;  // not built, or for another description: the scheduler finds no work
  if (warp == 8) {
    tmem_alloc(smem_u32(sh.tmem_slot), kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *sh.tmem_slot;

  if (warp < 8) {
    regs_increase<kSoftmaxRegs>();
    softmax_role<D>(sh, p, tmem, warp / 4);
  } else {
    regs_decrease<kControlRegs>();
    if (warp == 8) {
      if (lane == 0) mma_issuer<D>(sh, p, tmem);
      __syncwarp();
    } else if (warp == 9)
      producer<D>(sh, p, &tm_q, &tm_k, &tm_v);
    else if (warp == 10)
      scheduler<D>(sh, p);
    else
      zero_role<D>(sh, p);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- merging parts
// One warp per row at a time.  A row's parts, in this order: its own unit's
// shares, then (rows of small requests) the shares of the prefix unit that
// holds its token.
struct Merge {
  float m, l;
  float acc[4];
};

template <int D>
__device__ __forceinline__ void merge_part(Merge& g, const float* o, const float* lse, int lane) {
  const float x = *lse;
  if (x == -INFINITY) return;  // saw no key; its O row is not written
  constexpr int V = D / 32;
  float v[V];
  if constexpr (V == 4) {
    const float4 f = reinterpret_cast<const float4*>(o)[lane];
    v[0] = f.x; v[1] = f.y; v[2] = f.z; v[3] = f.w;
  } else {
    const float2 f = reinterpret_cast<const float2*>(o)[lane];
    v[0] = f.x; v[1] = f.y;
  }
  const float m = fmaxf(g.m, x);
  const float a = g.m == -INFINITY ? 0.f : expf(g.m - m), b = expf(x - m);
  g.l = g.l * a + b;
#pragma unroll
  for (int k = 0; k < V; ++k) g.acc[k] = g.acc[k] * a + b * v[k];
  g.m = m;
}

template <int D>
__device__ __forceinline__ void merge_unit(Merge& g, const Params& p, const wf_batch_unit& u, int64_t s, int64_t total,
                                           int ctas, int32_t tok_i, int32_t row_head, int32_t ct, int32_t head, int lane) {
  const bool pair = u.ntok > p.tile_tokens;
  const int32_t w = tile_cost(u.ntok, p.tile_tokens);
  const int c0 = share_of(s, total, ctas), c1 = share_of(s + int64_t(u.ktiles - 1) * w, total, ctas);
  if (c0 == c1) {
    const int64_t prow = (int64_t(u.req < 0 ? 0 : 2) * p.max_ctok + ct) * p.H + head;
    merge_part<D>(g, p.main_o + prow * D, p.main_lse + prow, lane);
    if (!pair) {
      const int64_t odd = prow + int64_t(p.max_ctok) * p.H;
      merge_part<D>(g, p.main_o + odd * D, p.main_lse + odd, lane);
    }
    return;
  }
  const int32_t tile = tok_i / p.tile_tokens;
  const int32_t row = (tok_i - tile * p.tile_tokens) * p.group + row_head;
  for (int c = c0; c <= c1; ++c) {
    int32_t j0, j1;
    share_tiles(s, w, u.ktiles, share_begin(c, total, ctas), share_begin(c + 1, total, ctas), j0, j1);
    if (j0 >= j1) continue;
    const int64_t slot = (int64_t(c) * 2 + (j0 == 0)) * 2;
    for (int k = pair ? tile : 0; k <= (pair ? tile : 1); ++k) {
      const int64_t prow = (slot + k) * 128 + row;
      merge_part<D>(g, p.cut_o + prow * D, p.cut_lse + prow, lane);
    }
  }
}

constexpr int kCombineThreads = 256;

template <int D>
__global__ void __launch_bounds__(kCombineThreads) batch_combine_kernel(const Params p) {
  const wf_batch_hdr* h = p.hdr;
  const int64_t head_cost = h->head_cost, total = head_cost * p.kv_heads;
  if (h->fingerprint != p.fingerprint || total == 0) return;
  const int lane = threadIdx.x & 31;
  const int ctas = h->ctas, np = h->prefix_units, own = h->units - np;
  const int subs = h->max_rows < 32 ? h->max_rows : 32;  // warps that share a unit's rows
  const int64_t tasks = int64_t(own) * p.kv_heads * subs;
  const int64_t warps = int64_t(gridDim.x) * (kCombineThreads / 32);
  for (int64_t k = int64_t(blockIdx.x) * (kCombineThreads / 32) + (threadIdx.x >> 5); k < tasks; k += warps) {
    const int32_t sub = int32_t(k % subs), kv = int32_t(k / subs % p.kv_heads), ui = np + int32_t(k / subs / p.kv_heads);
    const wf_batch_unit u = p.units[ui];
    const int64_t s = int64_t(kv) * head_cost + p.pre[ui];
    if (unit_direct(u, p.tile_tokens)) {
      const int64_t last = s + int64_t(u.ktiles - 1) * tile_cost(u.ntok, p.tile_tokens);
      if (share_of(s, total, ctas) == share_of(last, total, ctas)) continue;  // written by the attention
    }
    for (int32_t r = sub; r < u.ntok * p.group; r += subs) {
      const int32_t tok_i = r / p.group, row_head = r - tok_i * p.group;
      const int32_t tok = u.tok0 + tok_i, head = kv * p.group + row_head;
      Merge g;
      g.m = -INFINITY;
      g.l = 0.f;
      for (int x = 0; x < 4; ++x) g.acc[x] = 0.f;
      const int32_t ct = u.cbase + tok_i;
      merge_unit<D>(g, p, u, s, total, ctas, tok_i, row_head, ct, head, lane);
      if (u.ptiles < 0) {
        const int32_t pu = tok / (2 * p.tile_tokens);
        const wf_batch_unit q = p.units[pu];
        merge_unit<D>(g, p, q, int64_t(kv) * head_cost + p.pre[pu], total, ctas, tok - q.tok0, row_head, ct, head, lane);
      }
      const float inv = g.l > 0.f ? 1.0f / g.l : 0.f;
      __nv_bfloat16* dst = p.out + (int64_t(tok) * p.H + head) * D;
      if constexpr (D == 128) {
        uint2 o;
        o.x = pack_bf16x2(g.acc[0] * inv, g.acc[1] * inv);
        o.y = pack_bf16x2(g.acc[2] * inv, g.acc[3] * inv);
        reinterpret_cast<uint2*>(dst)[lane] = o;
      } else {
        reinterpret_cast<uint32_t*>(dst)[lane] = pack_bf16x2(g.acc[0] * inv, g.acc[1] * inv);
      }
      if (lane == 0 && p.lse) p.lse[int64_t(head) * p.max_tokens + tok] = g.l > 0.f ? g.m + logf(g.l) : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// [tokens, heads, D] with boxes of 64 dims x box_heads x box_tokens.
bool make_tmap(CUtensorMap* tm, const void* base, int64_t tokens, int32_t heads, int32_t dim, int32_t box_heads,
               int32_t box_tokens) {
  auto encode = get_encode();
  if (!encode) return false;
  cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(tokens)};
  cuuint64_t strides[2] = {cuuint64_t(dim) * 2, cuuint64_t(heads) * cuuint64_t(dim) * 2};
  cuuint32_t box[3] = {64, cuuint32_t(box_heads), cuuint32_t(box_tokens)};
  cuuint32_t estr[3] = {1, 1, 1};
  return encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box, estr,
                CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
wf_status launch(const wf_batch_desc* d, const BatchLayout& L, const Params& p, const void* q, const void* k_pool,
                 const void* v_pool, cudaStream_t stream) {
  static int attr_done[64] = {0};
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return WF_ERR_CUDA;
  if (dev < 0 || dev >= 64) return WF_ERR_UNSUPPORTED;
  if (!attr_done[dev]) {
    if (cudaFuncSetAttribute(batch_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, Cfg<D>::kSmemBytes) !=
        cudaSuccess) {
      cudaGetLastError();
      return WF_ERR_CUDA;
    }
    attr_done[dev] = 1;
  }
  const int64_t pool = int64_t(d->pool_pages) * d->page_tokens;
  CUtensorMap tq, tk, tv;
  if (!make_tmap(&tq, q, d->max_tokens, d->num_heads, D, L.group, L.tile_tokens) ||
      !make_tmap(&tk, k_pool, pool, d->num_kv_heads, D, 1, d->page_tokens) ||
      !make_tmap(&tv, v_pool, pool, d->num_kv_heads, D, 1, d->page_tokens))
    return WF_ERR_CUDA;
  batch_attn_kernel<D><<<L.ctas, kThreads, Cfg<D>::kSmemBytes, stream>>>(tq, tk, tv, p);
  if (cudaGetLastError() != cudaSuccess) return WF_ERR_CUDA;
  // as many warps as rows at most
  const int64_t rows = int64_t(d->max_tokens) * d->num_heads;
  const int64_t blocks = (rows + kCombineThreads / 32 - 1) / (kCombineThreads / 32);
  const int64_t most = int64_t(L.ctas) * 8;
  batch_combine_kernel<D><<<unsigned(blocks < most ? blocks : most), kCombineThreads, 0, stream>>>(p);
  return cudaGetLastError() == cudaSuccess ? WF_OK : WF_ERR_CUDA;
}

bool misaligned(const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) % 16 != 0; }

// Limit of every bounded wait (WF_WAIT_TIMEOUT_MS, default 2000 ms), read at each launch.
uint64_t wait_timeout_ns() {
  const char* env = std::getenv("WF_WAIT_TIMEOUT_MS");
  long ms = env ? std::atol(env) : 2000;
  if (ms < 1) ms = 1;
  return uint64_t(ms) * 1000000ull;
}

}  // namespace
}  // namespace wf

extern "C" wf_status wf_batch_attn(const wf_batch_desc* desc, const void* plan, const int32_t* block_table,
                                   const int32_t* prefix_table, const void* q, const void* k_pool, const void* v_pool,
                                   void* out, float* lse, float softmax_scale, void* workspace, size_t workspace_bytes,
                                   wf_stream_t stream) {
  const wf::BatchLayout L = wf::batch_layout(desc);
  if (L.error != WF_OK) return L.error;
  if (!plan || !block_table || !q || !k_pool || !v_pool || !out || !workspace) return WF_ERR_INVALID_ARG;
  if (desc->max_prefix_pages > 0 && !prefix_table) return WF_ERR_INVALID_ARG;
  if (wf::misaligned(plan) || wf::misaligned(q) || wf::misaligned(k_pool) || wf::misaligned(v_pool) ||
      wf::misaligned(out) || wf::misaligned(workspace) || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(block_table) % 4 || reinterpret_cast<uintptr_t>(prefix_table) % 4)
    return WF_ERR_ALIGNMENT;
  if (workspace_bytes < L.workspace_bytes) return WF_ERR_WORKSPACE;
  if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale)) return WF_ERR_INVALID_ARG;
  const double scale = softmax_scale == 0.f ? 1.0 / std::sqrt(double(desc->head_dim)) : double(softmax_scale);

  wf::Params p{};
  const uint8_t* pl = static_cast<const uint8_t*>(plan);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hdr = reinterpret_cast<const wf_batch_hdr*>(pl);
  p.units = reinterpret_cast<const wf_batch_unit*>(pl + L.off_units);
  p.pre = reinterpret_cast<const int64_t*>(pl + L.off_pre);
  p.ctok = reinterpret_cast<const int32_t*>(pl + L.off_ctok);
  p.table = block_table;
  p.prefix_table = prefix_table;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = reinterpret_cast<wf_dev_status*>(ws);
  p.main_o = reinterpret_cast<float*>(ws + WF_ATTN_STATUS_BYTES);
  p.cut_o = reinterpret_cast<float*>(ws + L.off_cut_o);
  p.main_lse = reinterpret_cast<float*>(ws + L.off_main_lse);
  p.cut_lse = reinterpret_cast<float*>(ws + L.off_cut_lse);
  p.fingerprint = L.fingerprint;
  p.timeout_ns = wf::wait_timeout_ns();
  p.scale_log2 = float(scale * 1.4426950408889634);
  p.H = desc->num_heads;
  p.kv_heads = desc->num_kv_heads;
  p.group = L.group;
  p.tile_tokens = L.tile_tokens;
  p.cols = desc->max_request_pages;
  while ((1 << p.page_shift) < desc->page_tokens) ++p.page_shift;
  p.block_tokens = desc->block_tokens;
  p.max_tokens = desc->max_tokens;
  p.max_ctok = int32_t(L.max_ctok);
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  return desc->head_dim == 128 ? wf::launch<128>(desc, L, p, q, k_pool, v_pool, s)
                               : wf::launch<64>(desc, L, p, q, k_pool, v_pool, s);
}
