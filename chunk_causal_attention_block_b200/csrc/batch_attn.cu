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
// 128-key tiles.  Rows of a request with more tokens than a row tile holds run
// the prefix's tiles and their own in one unit.  Rows of smaller requests are
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
// Narrow items (at most 32 rows: a single token or a short proposal's own keys)
// would leave three of a stream's four warps idle.  Their Q rows lie four
// times in the Q tile, one copy for each warp; a warp takes 32 of the tile's
// 128 keys, P goes to shared memory and the MMA forms O^T = V^T P^T, 32
// columns wide.
//
// What bounds it.  Many single tokens: HBM (96 requests, up to 4000 own keys
// each, 32760 shared, 12 heads, 1.50 GB: 278 us, 5.4 TB/s, on other pages every
// time; 250 us, 6.0 TB/s, on the same ones again).  Chunks of rows: the
// exponentials and MMAs of the two streams, which are busy 57% of the time
// each, under the power limit (2 x 4680 tokens over 42120 keys, 12 heads: 2.37
// ms, 1.02 PFLOP/s of visible pairs with other inputs every time; 2.05-2.4 ms on
// the same ones).  The stream attention (attn_sm100.cu) takes 7% less on a round
// that both can run (18720 rows over up to 51480 keys, 12 heads, in turn on one
// box: 5.1 and 5.5 ms); what makes the difference has not been measured.  A few
// rows: latency (one token over 334 keys: 10 us, 4 of them the merging's).
//
// Precision.  Scores, maxima, sums, O and merged parts are fp32.  P is rounded
// to bf16 for the product with V, since one tcgen05.mma takes both operands in
// one 16-bit type and V is bf16: a relative error over a case of 0.0018-0.0024
// against 64 bits, where an fp32 form that rounds O alone has 0.0016-0.0017.
//
// Warp roles (384 threads):
//   warps 0-3, 4-7  softmax of stream 0 and 1
//   warp  8   MMA issue (one elected lane), TMEM allocation
//   warp  9   TMA producer of Q tiles (ring of two) and K pages
//   warp 10   scheduler: walks this CTA's share and publishes items
//   warp 11   TMA producer of V pages (K and V share a ring of kStages tiles)
//
// Every wait is bounded; on expiry the status word is set, all roles return,
// copies in flight are waited for, and TMEM is freed.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <algorithm>
#include <atomic>
#include <cmath>
#include <cstddef>
#include <cstdint>
#include <cstdlib>
#include <mutex>

#include "sm100_ptx.cuh"
#include "wf_batch.h"

namespace wf {
namespace {

constexpr int kThreads = 384;
constexpr uint32_t kSoftmaxRegs = 208;
constexpr uint32_t kControlRegs = 88;
static_assert(2 * 128 * kSoftmaxRegs + 128 * kControlRegs == kThreads * 168, "register split must match launch");
constexpr int kHalfBytes = 128 * 128;  // 64-column half of a Q tile: 128 rows x 64 bf16, 128-byte swizzled
constexpr int kAtom = 8 * 128;         // 8 rows of 64 bf16: the swizzle's unit
constexpr uint32_t kTmemCols = 512;
constexpr float kRescaleThreshold = 8.0f;
constexpr float kLn2 = 0.69314718055994531f;
constexpr int kItems = 8;
constexpr int kNarrow = 32;  // rows up to which an item is narrow

enum Dest { kDirect = 0, kMainOwn = 1, kMainPrefix = 2, kCut = 3 };

// One share of a unit for one key head, published by the scheduler.
struct Item {
  int32_t j0, j1;   // key tiles; j1 = 0: no more items
  int32_t head;     // key head << 1 | narrow (at most kNarrow rows)
  int32_t dest;
  int32_t req, tok0, ntok, ptiles, pos0, len;  // of the unit (ptiles >= 0)
  int32_t parity;   // stream of the item's first subtile
  int32_t tile0;    // key tiles of this CTA before the item's first
  int64_t row0;     // output or partial row of the item's first row (stream or row tile 0)
  int64_t lse0;     // direct: of its LSE
};
static_assert(sizeof(Item) == 64, "item layout");

// A two-tile unit whose first cut is the beginning of the CTA's share.
struct Cut {
  int64_t s;        // cost position of the unit
  int32_t head, tok0, ntok, ktiles;
  int32_t c0, n;    // shares c0 .. c0+n-1 hold its tiles; n = 0: none
};
static_assert(sizeof(Cut) == WF_BATCH_CUT_BYTES, "cut record layout");

struct Params {
  const wf_batch_hdr* hdr;
  const wf_batch_start* starts;
  const wf_batch_unit* units;
  const int64_t* pre;
  const int32_t* ctok;
  const wf_batch_ctok* ctok_list;
  const int32_t* table;
  const int32_t* prefix_table;
  __nv_bfloat16* out;
  float* lse;
  wf_dev_status* status;
  // partial rows: [prefix, own][key parity][ctok][H], then [CTA][head, tail][row tile or key parity][128]
  float* part_o;
  float* part_lse;
  Cut* cuts;        // per CTA
  int64_t main_rows;
  uint64_t fingerprint;
  uint64_t timeout_ns;
  float scale_log2;
  int32_t H, kv_heads, group, tile_tokens;
  uint32_t group_inv;  // ceil(2^16 / group)
  int32_t cols, page_shift, block_tokens, max_tokens, max_ctok;
  int32_t stall_first_load;  // test hook: CTA 0 never issues its first K tile
};

__device__ __forceinline__ void tmem_ld4(uint32_t taddr, uint32_t (&r)[4]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(taddr));
}

constexpr int kXchBytes = 128 * 8;    // per stream: what its warps tell one another of narrow items' rows
constexpr int kStageRows = 32 * 128;  // per softmax warp: 128 bytes of each of its rows, on their way out

template <int D>
struct Cfg {
  static constexpr int kHalves = D / 64;
  static constexpr int kTile = kHalves * kHalfBytes;
  // K/V tiles hold 8-key groups one after another, in each the atoms of its
  // 64-column halves: a page's rows are then one block, whatever its size, and
  // one copy brings both halves.  (A copy takes about 60 cycles + 4 per
  // 128-byte row: with 16-token pages and a copy per half, 3970 cycles for a K
  // and a V tile, where HBM delivers them in 2950.)
  static constexpr int kGroup = kHalves * kAtom;
  static constexpr int kStages = D == 128 ? 4 : 8;
  static constexpr uint32_t kIdescQK = idesc_bf16_f32(128, 128, 0);
  static constexpr uint32_t kIdescPV = idesc_bf16_f32(128, D, 1);
  // narrow items: O^T = V^T P^T, A (V) MN-major, B (P) K-major
  static constexpr uint32_t kIdescOT = idesc_bf16_f32(128, kNarrow, 0) | (1u << 15);
  // barriers
  static constexpr int kQFull = 0, kQEmpty = 2, kSFull = 4, kPFull = 6, kOFull = 8, kItemFull = 10;
  static constexpr int kItemEmpty = kItemFull + kItems;
  static constexpr int kMmaDone = kItemEmpty + kItems;
  static constexpr int kXch = kMmaDone + 1;  // + stream: its warps exchange row maxima or sums
  static constexpr int kKVFull = kXch + 2;
  static constexpr int kKVEmpty = kKVFull + kStages;
  static constexpr int kNumBars = kKVEmpty + kStages;
  // the small parts come first, then the tiles from the next 1024-byte boundary on
  static constexpr int kSmall = kItems * int(sizeof(Item)) + 2 * kXchBytes + 8 * kNumBars + 8 + 2 * kStages * 4;
  static constexpr int kTiles = (2 + kStages) * kTile + 8 * kStageRows;
  static constexpr int kSmemBytes = (kSmall + 1023) / 1024 * 1024 + kTiles;
  static_assert(kSmemBytes <= 232448, "shared memory per block");
};
// softmax warps (8), MMA, two producers
constexpr uint32_t kItemReaders = 11;

// Shared memory by 32-bit addresses: items, exchange, barriers, TMEM address
// and abort flag at `base`, two Q tiles, the K/V stages and outgoing rows at
// `tiles`.  (Generic pointers cost a conversion at every use.)
template <int D>
struct Shared {
  using C = Cfg<D>;
  static constexpr int kXchAt = kItems * int(sizeof(Item));
  static constexpr int kBarsAt = kXchAt + 2 * kXchBytes;
  static constexpr int kTmemAt = kBarsAt + 8 * C::kNumBars;
  static constexpr int kAbortAt = kTmemAt + 4;
  static constexpr int kFillsAt = kAbortAt + 4;
  static constexpr int kRowsAt = (2 + C::kStages) * C::kTile;

  uint32_t base, tiles;

  __device__ __forceinline__ uint32_t q_tile(int slot) const { return tiles + slot * C::kTile; }
  __device__ __forceinline__ uint32_t kv_tile(int st) const { return tiles + (2 + st) * C::kTile; }
  __device__ __forceinline__ uint32_t out_rows(int warp) const { return tiles + kRowsAt + warp * kStageRows; }
  // narrow items: a stream's P (two halves of 64 keys, kNarrow rows), in its warps' outgoing rows
  __device__ __forceinline__ uint32_t p_tile(int t) const { return tiles + kRowsAt + t * 4 * kStageRows; }
  __device__ __forceinline__ uint32_t xch(int t) const { return base + kXchAt + t * kXchBytes; }
  __device__ __forceinline__ uint32_t item(int it) const { return base + it % kItems * int(sizeof(Item)); }
  __device__ __forceinline__ uint32_t bar(int b) const { return base + kBarsAt + 8 * b; }
  __device__ __forceinline__ uint32_t fills(int producer, int st) const {
    return base + kFillsAt + 4 * (producer * C::kStages + st);
  }
  __device__ __forceinline__ bool aborting() const { return ld_shared_u32(base + kAbortAt) != 0; }
};

__device__ __forceinline__ void st_shared_u32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}

__device__ __forceinline__ void st_shared_f32x2(uint32_t addr, float a, float b) {
  asm volatile("st.shared.v2.f32 [%0], {%1, %2};" ::"r"(addr), "f"(a), "f"(b) : "memory");
}

__device__ __forceinline__ float2 ld_shared_f32x2(uint32_t addr) {
  float2 v;
  asm volatile("ld.shared.v2.f32 {%0, %1}, [%2];" : "=f"(v.x), "=f"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ int64_t ld_shared_s64(uint32_t addr) {
  int64_t v;
  asm volatile("ld.shared.s64 %0, [%1];" : "=l"(v) : "r"(addr) : "memory");
  return v;
}

// Bounded wait; false if the CTA is aborting.  An expiry records where in one
// 16-byte store.  Kept short: it is instantiated at every wait, and calls of
// small items wait for the instruction cache.
template <int D>
__device__ __forceinline__ bool wait_bar(const Shared<D>& sh, const Params& p, int bar, uint32_t parity, int where) {
  const uint32_t addr = sh.bar(bar);
  if (mbar_try_wait(addr, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  do {
#pragma unroll 1
    for (int i = 0; i < 64; ++i)
      if (mbar_try_wait(addr, parity)) return true;
    if (sh.aborting()) return false;
  } while (global_timer_ns() - t0 <= p.timeout_ns);
  st_shared_u32(sh.base + Shared<D>::kAbortAt, 1);
  *reinterpret_cast<int4*>(p.status) =
      make_int4(WF_ERR_DEVICE_TIMEOUT, where, int32_t(blockIdx.x), int32_t(threadIdx.x));
  return false;
}

// The same without giving up for others (the end of a role): false after the limit.
__device__ __forceinline__ bool wait_alone(uint32_t bar, uint32_t parity, uint64_t timeout_ns) {
  const uint64_t t0 = global_timer_ns();
  while (!mbar_try_wait(bar, parity))
    if (global_timer_ns() - t0 > timeout_ns) return false;
  return true;
}

template <int D>
__device__ __forceinline__ bool warp_wait(const Shared<D>& sh, const Params& p, int bar, uint32_t parity, int where) {
  return __all_sync(0xffffffffu, wait_bar(sh, p, bar, parity, where));
}

// The scheduler's wait for a slot of the item ring.  It lasts as long as the
// oldest item runs (a million key tiles take 1 s), so it gives up only when no
// K tile has been asked for within the limit: a role that is stuck expires by
// itself and ends this wait too.
template <int D>
__device__ __forceinline__ bool wait_slot(const Shared<D>& sh, const Params& p, int it, int where) {
  using C = Cfg<D>;
  const uint32_t addr = sh.bar(C::kItemEmpty + it % kItems), parity = ((it / kItems) & 1) ^ 1;
  const int lane = threadIdx.x & 31;
  uint32_t seen = ~0u;  // (no count of fills)
  uint64_t since = 0;
#pragma unroll 1
  while (!__all_sync(0xffffffffu, mbar_try_wait(addr, parity))) {
    if (__any_sync(0xffffffffu, sh.aborting())) return false;
    const uint32_t fill = lane < C::kStages ? ld_shared_u32(sh.fills(0, lane)) : 0;
    const uint64_t now = global_timer_ns();
    if (__any_sync(0xffffffffu, fill != seen)) {
      seen = fill;
      since = now;
    } else if (__any_sync(0xffffffffu, now - since > p.timeout_ns)) {
      if (lane == 0) {
        st_shared_u32(sh.base + Shared<D>::kAbortAt, 1);
        *reinterpret_cast<int4*>(p.status) =
            make_int4(WF_ERR_DEVICE_TIMEOUT, where, int32_t(blockIdx.x), int32_t(threadIdx.x));
      }
      return false;
    }
  }
  return true;
}

// ---------------------------------------------------------------- shares of the line of costs
// Equal shares of `size` (the last one shorter).
struct Line {
  int64_t head_cost, total, size;
  double rcp;  // 1 / size
};

__device__ __forceinline__ Line line_of(const Params& p) {
  const wf_batch_hdr* h = p.hdr;
  Line x;
  x.head_cost = h->head_cost;
  x.total = h->head_cost * p.kv_heads;
  x.size = h->share;
  x.rcp = h->share_rcp;
  return x;
}

__device__ __forceinline__ int64_t share_begin(const Line& x, int c) {
  const int64_t b = c * x.size;
  return b < x.total ? b : x.total;
}

// The share that holds cost position s < total: at most 256 of them, so the
// fp64 product is off by far less than one.
__device__ __forceinline__ int share_of(const Line& x, int64_t s) {
  int c = int(double(s) * x.rcp);
  c -= c * x.size > s;
  c += (c + 1) * x.size <= s;
  return c;
}

// Key tiles of a unit at cost position s (1 << w per tile) that start inside [lo, hi).
__device__ __forceinline__ void share_tiles(int64_t s, int32_t w, int32_t ktiles, int64_t lo, int64_t hi, int32_t& j0,
                                            int32_t& j1) {
  const int64_t up = (int64_t(1) << w) - 1;
  const int64_t a = lo <= s ? 0 : (lo - s + up) >> w, b = hi <= s ? 0 : (hi - s + up) >> w;
  j0 = int32_t(a < ktiles ? a : ktiles);
  j1 = int32_t(b < ktiles ? b : ktiles);
}

__device__ __forceinline__ int32_t tile_shift(int32_t ntok, int32_t tile_tokens) {
  return ntok > tile_tokens ? WF_BATCH_PAIR_SHIFT : WF_BATCH_SINGLE_SHIFT;
}

// Whether rows of this unit run no other key tiles than the unit's, and on one
// stream: an uncut unit then writes its output rows itself.
__device__ __forceinline__ bool unit_direct(const wf_batch_unit& u, int32_t tile_tokens) {
  return u.req >= 0 && u.ptiles >= 0 && (u.ntok > tile_tokens || u.ktiles == 1);
}

// Indices of partial rows.
__device__ __forceinline__ int64_t main_row(const Params& p, bool own, int key_parity, int32_t ctok, int32_t head) {
  return (int64_t((own ? 2 : 0) + key_parity) * p.max_ctok + ctok) * p.H + head;
}
__device__ __forceinline__ int64_t cut_row(const Params& p, int cta, bool tail, int half, int32_t row) {
  return p.main_rows + ((int64_t(cta) * 2 + tail) * 2 + half) * 128 + row;
}

// ---------------------------------------------------------------- item ring
// Copies item `it` and gives its slot back; false at the end (or on an abort).
// The fields come through a shuffle from lane 0, which tells the compiler that
// they are the same in all lanes: what the MMA and the producer warp derive
// from them (loop counts, ring positions, descriptors) then stays in uniform
// registers, as tcgen05.mma and TMA instructions need it.  Without that each
// MMA took 136 cycles to issue instead of 64 (its operands moved from ordinary
// registers one by one).
template <int D>
__device__ __forceinline__ bool take_item(const Shared<D>& sh, const Params& p, int it, Item& x, int where) {
  if (!warp_wait(sh, p, Cfg<D>::kItemFull + it % kItems, (it / kItems) & 1, where)) return false;
  const uint32_t src = sh.item(it);
  int32_t* dst = reinterpret_cast<int32_t*>(&x);
#pragma unroll
  for (int k = 0; k < int(sizeof(Item) / 16); ++k) {
    uint32_t v[4];
    ld_shared_v4(src + 16 * k, v);
#pragma unroll
    for (int i = 0; i < 4; ++i) dst[4 * k + i] = __shfl_sync(0xffffffffu, int32_t(v[i]), 0);
  }
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(sh.bar(Cfg<D>::kItemEmpty + it % kItems));
  return x.j1 > 0;
}

// True in one lane of the (converged) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t yes;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(yes));
  return yes != 0;
}

template <int D>
__device__ __forceinline__ void put_item(const Shared<D>& sh, int it, const Item& x) {
  const uint32_t dst = sh.item(it);
  const uint32_t* src = reinterpret_cast<const uint32_t*>(&x);
#pragma unroll
  for (int k = 0; k < int(sizeof(Item) / 16); ++k)
    st_shared_v4(dst + 16 * k, src[4 * k], src[4 * k + 1], src[4 * k + 2], src[4 * k + 3]);
}

__device__ __forceinline__ int32_t item_field(uint32_t item, uint32_t offset) {
  return int32_t(ld_shared_u32(item + offset));
}
__device__ __forceinline__ int64_t item_field64(uint32_t item, uint32_t offset) { return ld_shared_s64(item + offset); }

// The whole warp is done with item `it`.
template <int D>
__device__ __forceinline__ void release_item(const Shared<D>& sh, int it) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(sh.bar(Cfg<D>::kItemEmpty + it % kItems));
}

// What the scheduler reads before anything else, while the block is set up:
// its share of the line of costs, and lane i's of the first 32 units.
struct Share {
  int64_t head_cost, lo, hi;
  int32_t units, head, unit;  // units 0: nothing to do
};

__device__ __forceinline__ Share first_share(const Params& p) {
  const wf_batch_hdr* h = p.hdr;
  const int c = int(blockIdx.x);
  const wf_batch_start at = p.starts[c];  // (not written if c is beyond the shares)
  const Line line = line_of(p);
  Share x;
  x.head_cost = line.head_cost;
  x.lo = share_begin(line, c);
  x.hi = share_begin(line, c + 1);
  x.units = h->fingerprint == p.fingerprint && x.lo < x.hi ? h->units : 0;
  x.head = x.units > 0 ? at.head : 0;
  x.unit = x.units > 0 ? at.unit : 0;
  return x;
}

// A lane's unit and its cost position.
__device__ __forceinline__ bool load_unit(const Params& p, const Share& x, int32_t head, int32_t unit, wf_batch_unit& r,
                                          int64_t& s) {
  if (unit >= x.units) return false;
  const int4* src = reinterpret_cast<const int4*>(p.units + unit);
  reinterpret_cast<int4*>(&r)[0] = src[0];
  reinterpret_cast<int4*>(&r)[1] = src[1];
  s = int64_t(head) * x.head_cost + p.pre[unit];
  return true;
}

template <int D>
__device__ __forceinline__ void scheduler(const Shared<D>& sh, const Params& p, const Share& x, wf_batch_unit r,
                                          int64_t s) {
  const int lane = threadIdx.x & 31;
  int it = 0;
  int32_t parity = 0, tile0 = 0;
  int32_t head = x.head, u = x.unit;
  bool have = u + lane < x.units, more = x.units > 0, start = true;
  while (more) {
    // 32 units at a time, one per lane
    int32_t j0 = 0, j1 = 0;
    const int32_t w = tile_shift(r.ntok, p.tile_tokens);
    if (have) share_tiles(s, w, r.ktiles, x.lo, x.hi, j0, j1);
    more = __all_sync(0xffffffffu, !have || s < x.hi);
    if (start && lane == 0) {
      // for the merging: whether the share begins with the first cut of a two-tile unit (written before any
      // wait can give up: the merging kernel reads it all the same)
      const Line line = line_of(p);
      Cut k{};
      if (j0 > 0 && j0 < j1 && r.req >= 0 && r.ntok > p.tile_tokens) {
        k.c0 = share_of(line, s);
        if (share_of(line, s + (int64_t(j0 - 1) << w)) == k.c0) {
          k.s = s;
          k.head = head;
          k.tok0 = r.tok0;
          k.ntok = r.ntok;
          k.ktiles = r.ktiles;
          k.n = share_of(line, s + (int64_t(r.ktiles - 1) << w)) - k.c0 + 1;
        }
      }
      p.cuts[blockIdx.x] = k;
    }
    start = false;
    uint32_t todo = __ballot_sync(0xffffffffu, j0 < j1);
    while (todo) {
      const int src = __ffs(todo) - 1;
      todo &= todo - 1;
      const int32_t n = __shfl_sync(0xffffffffu, j1 - j0, src);
      const bool pair = __shfl_sync(0xffffffffu, r.ntok, src) > p.tile_tokens;
      if (!wait_slot<D>(sh, p, it, 40)) return;
      if (lane == src) {
        Item y;
        y.j0 = j0;
        y.j1 = j1;
        y.head = head << 1 | (r.ntok * p.group <= kNarrow);
        y.req = r.req;
        y.tok0 = r.tok0;
        y.ntok = r.ntok;
        y.ptiles = r.ptiles < 0 ? 0 : r.ptiles;
        y.pos0 = r.pos0;
        y.len = r.len;
        y.parity = parity;
        y.tile0 = tile0;
        const int32_t head0 = head * p.group;
        y.lse0 = int64_t(head0) * p.max_tokens + r.tok0;
        if (j0 > 0 || j1 < r.ktiles) {
          y.dest = kCut;
          y.row0 = cut_row(p, int(blockIdx.x), j0 == 0, 0, 0);
        } else if (unit_direct(r, p.tile_tokens)) {
          y.dest = kDirect;
          y.row0 = int64_t(r.tok0) * p.H + head0;
        } else if (r.req < 0) {
          y.dest = kMainPrefix;  // the rows' tokens have partial rows of their own
          y.row0 = head0;
        } else {
          y.dest = kMainOwn;
          y.row0 = main_row(p, true, 0, r.cbase, head0);
        }
        put_item<D>(sh, it, y);
        mbar_arrive(sh.bar(Cfg<D>::kItemFull + it % kItems));
      }
      __syncwarp();
      parity ^= pair ? 0 : n & 1;
      tile0 += n;
      ++it;
    }
    u += 32;
    if (u >= x.units) {
      // the next head's first unit starts where this head ends
      u = 0;
      ++head;
      more = more && head < p.kv_heads && int64_t(head) * x.head_cost < x.hi;
    }
    if (more) have = load_unit(p, x, head, u + lane, r, s);
  }
  if (!wait_slot<D>(sh, p, it, 41)) return;
  if (lane == 0) {
    put_item<D>(sh, it, Item{});
    mbar_arrive(sh.bar(Cfg<D>::kItemFull + it % kItems));
  }
}

// ---------------------------------------------------------------- K/V tiles
// Key tile j of an item.  Lane i of the producer holds
// the tile's i-th page (16 at most): read from the table once, a tile ahead of
// its use, for K and V both.
struct KeyTile {
  int32_t head_valid;  // key head << 8 | keys (at most 128)
  int32_t page;        // this lane's page (as loaded: used a tile later)
};

__device__ __forceinline__ int32_t tile_keys(const Item& x, int32_t j, int32_t prefix_len) {
  const int32_t left = j >= x.ptiles ? x.len - (j - x.ptiles) * 128 : prefix_len - j * 128;
  return left < 128 ? left : 128;
}

__device__ __forceinline__ KeyTile key_tile(const Params& p, const Item& x, int32_t j, int32_t prefix_len) {
  KeyTile k;
  const int32_t valid = tile_keys(x, j, prefix_len);
  k.head_valid = x.head >> 1 << 8 | valid;
  const bool own = j >= x.ptiles;
  const int32_t pg = int32_t(threadIdx.x & 31);
  const int32_t* list = own ? p.table + x.req * p.cols : p.prefix_table;
  const int32_t first = ((own ? j - x.ptiles : j) * 128) >> p.page_shift;
  k.page = pg << p.page_shift < valid ? list[first + pg] : 0;
  return k;
}

// One page's rows of one key head: coordinates (dim in half, key in group, half,
// group, head).
__device__ __forceinline__ void tma_load_page(uint32_t dst, const CUtensorMap* tmap, uint32_t bar, int32_t head,
                                              int32_t group) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %3, %3, %4, %5}], "
      "[%2];" ::"r"(dst),
      "l"(tmap), "r"(bar), "r"(0), "r"(group), "r"(head)
      : "memory");
}

// Copies a tile; only pages that hold keys are read.  The pages go round by
// shuffle and one lane issues all copies (32 lanes issuing one each serialise,
// at about 85 cycles a copy).
template <int D>
__device__ __forceinline__ void load_tile(const Shared<D>& sh, const Params& p, const CUtensorMap* tm, const KeyTile& k,
                                          int st, int bar_index) {
  const int head = k.head_valid >> 8, valid = k.head_valid & 255;
  const int pages = (valid + (1 << p.page_shift) - 1) >> p.page_shift;
  const uint32_t page_bytes = uint32_t(Cfg<D>::kHalves * 128) << p.page_shift;
  const uint32_t bar = sh.bar(bar_index);
  uint32_t dst = sh.kv_tile(st);
  // in 8-token groups; an entry outside the pool reads zeros, not memory: the map's bounds hold
  const int64_t mine = int64_t(k.page) << (p.page_shift - 3);
  const int32_t at = mine < 0 || mine > 0x0FFFFFF0 ? 0x0FFFFFF0 : int32_t(mine);
  if (elect_one()) mbar_arrive_expect_tx(bar, uint32_t(pages) * page_bytes);
  // four pages at a time: their positions first, then the copies back to back
#pragma unroll 1
  for (int pg = 0; pg < pages; pg += 4) {
    int32_t a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = __shfl_sync(0xffffffffu, at, pg + i);
    if (elect_one()) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (pg + i < pages) tma_load_page(dst + i * page_bytes, tm, bar, head, a[i]);
    }
    dst += 4 * page_bytes;
  }
}

// The K/V ring is used in one order, which its two producers and the MMA warp
// each follow: at step m the V tile of subtile m-2 (if that subtile is the
// first on its tile), then the K tile of subtile m (likewise).  Q and K come
// from one warp, V from another: with small pages, what a tile costs is the
// issue of its copies.
//
// Subtile by subtile, with the steps of the last two V tiles at the end.
struct Walk {
  Item x{};
  int it = 0, j = 0, s = 0, tiles = 1, left = 2;
  bool more = true;

  // Whether the current item is used up and another has to be taken.
  __device__ __forceinline__ bool at_item() const { return more && j == x.j1; }
  __device__ __forceinline__ void begin(const Params& p) {
    ++it;
    j = x.j0;
    tiles = x.ntok > p.tile_tokens ? 2 : 1;
  }
  // Whether this step has a place for a K tile in the ring.  (The step behind a
  // last one-row-tile subtile has, too: V tile n of the CTA then has fill 2n+2
  // in one-tile items and 2n+1 in two-tile ones, wherever it stands.)
  __device__ __forceinline__ bool opens_k() const { return more ? s == 0 : left == 2 && tiles == 1; }
  // To the next subtile; false behind the last step.
  __device__ __forceinline__ bool next() {
    if (!more) return --left > 0;
    if (++s == tiles) {
      s = 0;
      ++j;
    }
    return true;
  }
};

// What a producer leaves behind for a CTA that gives up: its last fill of each stage.
template <int D>
__device__ __forceinline__ void note_fill(const Shared<D>& sh, int producer, int st, int fill) {
  if (elect_one()) st_shared_u32(sh.fills(producer, st), uint32_t(fill + 1));
}

template <int D>
__device__ __forceinline__ void k_producer(const Shared<D>& sh, const Params& p, const CUtensorMap* tm_q,
                                           const CUtensorMap* tm_narrow, const CUtensorMap* tm_k) {
  using C = Cfg<D>;
  const int32_t prefix_len = p.hdr->prefix_len;
  int kv_it = 0, q_it = 0;
  KeyTile next{};
  uint32_t opened = 0;  // bit 0, 1: the last and the second last subtile were the first on their tiles
  Walk w;
  for (;;) {
    if (w.at_item()) {
      w.more = take_item<D>(sh, p, w.it, w.x, 1);
      if (!w.more) break;  // no K tile is left
      w.begin(p);
      next = key_tile(p, w.x, w.j, prefix_len);
    }
    kv_it += (opened >> 1) & 1;  // the V tile's stage
    if (w.s == 0) {
      const KeyTile k = next;
      if (w.j + 1 < w.x.j1) next = key_tile(p, w.x, w.j + 1, prefix_len);
      const int st = kv_it % C::kStages;
      if (!warp_wait(sh, p, C::kKVEmpty + st, ((kv_it / C::kStages) & 1) ^ 1, 2)) break;
      // failure-detection test: this fill's barrier is never armed, so that
      // the MMA warp's bounded wait on it must expire
      if (!(p.stall_first_load && blockIdx.x == 0 && kv_it == 0)) {
        load_tile<D>(sh, p, tm_k, k, st, C::kKVFull + st);
        note_fill(sh, 0, st, kv_it);
      }
      ++kv_it;
    }
    // An item's Q tiles follow its first K tile: their slots come free only
    // with the last scores of the item before.
    if (w.s == 0 && w.j == w.x.j0) {
      bool ok = true;
#pragma unroll 1
      for (int i = 0; i < w.tiles; ++i, ++q_it) {
        const int slot = q_it & 1;
        ok = warp_wait(sh, p, C::kQEmpty + slot, ((q_it >> 1) & 1) ^ 1, 3);
        if (!ok) break;
        const uint32_t bar = sh.bar(C::kQFull + slot);
        const bool narrow = w.x.head & 1;
        const CUtensorMap* tm = narrow ? tm_narrow : tm_q;
        const int lanes = narrow ? kNarrow : 128, rows = lanes / p.group * p.group;  // a box holds the latter
        if (elect_one()) {
          mbar_arrive_expect_tx(bar, uint32_t(rows * (128 / lanes)) * 128 * C::kHalves);
#pragma unroll 1
          for (int at = 0; at < 128; at += lanes)
#pragma unroll
            for (int half = 0; half < C::kHalves; ++half)
              tma_load_3d(sh.q_tile(slot) + half * kHalfBytes + at * 128, tm, bar, 64 * half, (w.x.head >> 1) * p.group,
                          w.x.tok0 + i * p.tile_tokens);
        }
        __syncwarp();
      }
      if (!ok) break;
    }
    opened = opened << 1 | (w.s == 0);
    w.next();
  }
  // Copies in flight end before the CTA does: by their use, or here if it gives up.
  if (sh.aborting())
#pragma unroll 1
    for (int b = 0; b < 2 && b < q_it; ++b)
      wait_alone(sh.bar(C::kQFull + b), uint32_t((q_it - 1 - b) >> 1) & 1, p.timeout_ns);
}

template <int D>
__device__ __forceinline__ void v_producer(const Shared<D>& sh, const Params& p, const CUtensorMap* tm_v) {
  using C = Cfg<D>;
  const int32_t prefix_len = p.hdr->prefix_len;
  int kv_it = 0;
  KeyTile next{}, v1{}, v2{};  // of the coming, the last and the second last subtile; head_valid 0: no tile of its own
  Walk w;
  for (;;) {
    if (w.at_item()) {
      w.more = take_item<D>(sh, p, w.it, w.x, 51);
      if (!w.more && sh.aborting()) return;
      if (w.more) {
        w.begin(p);
        next = key_tile(p, w.x, w.j, prefix_len);
      }
    }
    if (v2.head_valid != 0) {
      const int st = kv_it % C::kStages;
      if (!warp_wait(sh, p, C::kKVEmpty + st, ((kv_it / C::kStages) & 1) ^ 1, 4)) return;
      load_tile<D>(sh, p, tm_v, v2, st, C::kKVFull + st);
      note_fill(sh, 1, st, kv_it);
      ++kv_it;
    }
    kv_it += w.opens_k();
    v2 = v1;
    v1 = KeyTile{};
    if (w.more && w.s == 0) {
      v1 = next;
      if (w.j + 1 < w.x.j1) next = key_tile(p, w.x, w.j + 1, prefix_len);
    }
    if (!w.next()) return;
  }
}

// ---------------------------------------------------------------- MMA issue
// Descriptor offsets as immediates, fully unrolled (attn_sm100.cu measures why).
template <int D, int kk>
__device__ __forceinline__ void issue_s_slice(uint32_t s_tmem, uint64_t qd, uint64_t kd) {
  constexpr uint32_t q_off = uint32_t(((kk >> 2) * kHalfBytes + (kk & 3) * 32) >> 4);
  constexpr uint32_t k_off = uint32_t(((kk >> 2) * kAtom + (kk & 3) * 32) >> 4);
  mma_ss_off<q_off, k_off>(s_tmem, qd, kd, Cfg<D>::kIdescQK, kk > 0 ? 1u : 0u);
  if constexpr (kk + 1 < D / 16) issue_s_slice<D, kk + 1>(s_tmem, qd, kd);
}

template <int D, int kk>
__device__ __forceinline__ void issue_pv_slice(uint32_t o_tmem, uint32_t p_tmem, uint64_t vd, uint32_t acc0) {
  mma_ts_off<kk * 8, uint32_t((kk * 2 * Cfg<D>::kGroup) >> 4)>(o_tmem, p_tmem, vd, Cfg<D>::kIdescPV, kk > 0 ? 1u : acc0);
  if constexpr (kk < 7) issue_pv_slice<D, kk + 1>(o_tmem, p_tmem, vd, acc0);
}

// Narrow: O^T (lanes: dims, columns: rows) += V^T P^T.  With 64 dims, lanes 64
// to 127 repeat the next 8-key group's and are not looked at.
template <int D, int kk>
__device__ __forceinline__ void issue_ot_slice(uint32_t o_tmem, uint64_t vd, uint64_t pd, uint32_t acc0) {
  mma_ss_off<uint32_t((kk * 2 * Cfg<D>::kGroup) >> 4), uint32_t(((kk >> 2) * kNarrow * 128 + (kk & 3) * 32) >> 4)>(
      o_tmem, vd, pd, Cfg<D>::kIdescOT, kk > 0 ? 1u : acc0);
  if constexpr (kk < 7) issue_ot_slice<D, kk + 1>(o_tmem, vd, pd, acc0);
}

// What a pending PV product needs to know of its subtile.
constexpr uint32_t kPvLive = 1, kPvFirst = 2, kPvLast = 4, kPvOpens = 8, kPvCloses = 16, kPvNarrow = 32;

template <int D>
__device__ __forceinline__ void mma_issuer(const Shared<D>& sh, const Params& p, uint32_t tmem) {
  using C = Cfg<D>;
  int kv_it = 0, q_it = 0;
  uint32_t p_phase = 0;        // bit t: parity of stream t's next P
  uint32_t ot = 0;             // bit t: which of its two O^T stream t's narrow item has
  uint32_t pv1 = 0, pv2 = 0;   // flags of the last and the second last subtile
  int vst = 0, kst = 0;

  // One step per subtile, then two more for the last PV products.
  Item x{};
  int it = 0, j = 0, n = 0, s = 0, tiles = 1, left = 2;
  bool more = true;
  for (uint32_t m = 0;; ++m) {
    if (more && j == n) {
      q_it += n > 0 ? tiles : 0;
      more = take_item<D>(sh, p, it, x, 10);
      if (!more && sh.aborting()) break;
      if (more) {
        ++it;
        j = 0;
        n = x.j1 - x.j0;
        tiles = x.ntok > p.tile_tokens ? 2 : 1;
      }
    }
    const uint32_t t = m & 1;
    if (pv2 & kPvLive) {
      if (pv2 & kPvOpens) {
        vst = kv_it % C::kStages;
        if (!warp_wait(sh, p, C::kKVFull + vst, (kv_it / C::kStages) & 1, 12)) break;
        ++kv_it;
      }
      if (!warp_wait(sh, p, C::kPFull + t, (p_phase >> t) & 1, 14 + t)) break;
      p_phase ^= 1u << t;
      tc_fence_after();
      const uint64_t vd = smem_desc_sw128(sh.kv_tile(vst), kAtom, C::kGroup);
      if ((pv2 & kPvNarrow) && (pv2 & kPvFirst)) ot ^= 1u << t;
      if (elect_one()) {
        const uint32_t acc = pv2 & kPvFirst ? 0u : 1u;
        if (pv2 & kPvNarrow)
          issue_ot_slice<D, 0>(tmem + 256 + 128 * t + kNarrow * ((ot >> t) & 1), vd,
                               smem_desc_sw128(sh.p_tile(t), 16, kAtom), acc);
        else
          issue_pv_slice<D, 0>(tmem + 256 + 128 * t, tmem + 128 * t, vd, acc);
        if (pv2 & kPvLast) mma_commit(sh.bar(C::kOFull + t));
        if (pv2 & kPvCloses) mma_commit(sh.bar(C::kKVEmpty + vst));
      }
      __syncwarp();
    }
    pv2 = pv1;
    if (!more) {
      kv_it += left == 2 && tiles == 1;  // (see Walk)
      pv1 = 0;
      if (--left == 0) break;
      continue;
    }
    if (s == 0) {
      kst = kv_it % C::kStages;
      if (!warp_wait(sh, p, C::kKVFull + kst, (kv_it / C::kStages) & 1, 13)) break;
      ++kv_it;
    }
    const int slot = (q_it + s) & 1;
    if (j == 0 && !warp_wait(sh, p, C::kQFull + slot, ((q_it + s) >> 1) & 1, 11)) break;
    tc_fence_after();
    const uint64_t qd = smem_desc_sw128(sh.q_tile(slot), 16, kAtom);
    const uint64_t kd = smem_desc_sw128(sh.kv_tile(kst), 16, C::kGroup);
    if (elect_one()) {
      issue_s_slice<D, 0>(tmem + 128 * t, qd, kd);
      mma_commit(sh.bar(C::kSFull + t));
      if (s == tiles - 1) mma_commit(sh.bar(C::kKVEmpty + kst));
      if (j == n - 1) mma_commit(sh.bar(C::kQEmpty + slot));
    }
    __syncwarp();
    // first and last subtile of its stream in this item
    const int step = tiles == 2 ? 1 : 2;
    pv1 = kPvLive | (j < step ? kPvFirst : 0u) | (j + step >= n ? kPvLast : 0u) | (s == 0 ? kPvOpens : 0u) |
          (s == tiles - 1 ? kPvCloses : 0u) | (x.head & 1 ? kPvNarrow : 0u);
    if (++s == tiles) {
      s = 0;
      ++j;
    }
  }
  // all issued MMAs complete before TMEM is released
  if (elect_one()) mma_commit(sh.bar(C::kMmaDone));
  __syncwarp();
  wait_alone(sh.bar(C::kMmaDone), 0, p.timeout_ns);
}

// ---------------------------------------------------------------- softmax
// exp2(s * sl2 - m) as bf16 pairs into TMEM; returns the fp32 row sum (taken
// before the rounding, so that the errors of single weights average out instead
// of moving the whole row).
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

// O * scale of the warp's 32 rows to their destinations (nullptr: none), as
// bf16 or fp32.  A thread holds a row, but rows lie far apart in memory: stored
// from registers, a 16-byte piece of each at a time, the two tiles of a unit
// took 8000 cycles.  So 128 bytes of every row at a time go through shared
// memory (the warp's own, 16-byte pieces swizzled by row) and leave as full
// lines, eight lanes to a row.
template <int D>
__device__ __forceinline__ void store_rows(const Shared<D>& sh, uint32_t o_tm, uint8_t* dst, bool as_bf16, float scale) {
  const int lane = threadIdx.x & 31;
  const uint32_t buf = sh.out_rows(threadIdx.x / 32);
  const uint32_t mine = buf + lane * 128;
  const uint32_t rows = __ballot_sync(0xffffffffu, dst != nullptr);
  const int chunks = D * (as_bf16 ? 2 : 4) / 128;
#pragma unroll 1
  for (int c = 0; c < chunks; ++c) {
    uint32_t r[32];
    if (as_bf16) {
      uint32_t r2[32];
      tmem_ld32(o_tm + 64 * c, r);
      tmem_ld32(o_tm + 64 * c + 32, r2);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 16; ++x) {
        r[x] = pack_bf16x2(__uint_as_float(r[2 * x]) * scale, __uint_as_float(r[2 * x + 1]) * scale);
        r2[x] = pack_bf16x2(__uint_as_float(r2[2 * x]) * scale, __uint_as_float(r2[2 * x + 1]) * scale);
      }
#pragma unroll
      for (int x = 0; x < 16; ++x) r[16 + x] = r2[x];
    } else {
      tmem_ld32(o_tm + 32 * c, r);
      tmem_wait_ld();
#pragma unroll
      for (int x = 0; x < 32; ++x) r[x] = __float_as_uint(__uint_as_float(r[x]) * scale);
    }
#pragma unroll
    for (int v = 0; v < 8; ++v)
      st_shared_v4(mine + ((v ^ (lane & 7)) << 4), r[4 * v], r[4 * v + 1], r[4 * v + 2], r[4 * v + 3]);
    __syncwarp();
    // 16 rows at a time, their loads all before their stores: one warp a sub-partition hides no latency
#pragma unroll 1
    for (uint32_t left = rows, r0 = lane >> 3; left != 0; left >>= 16, r0 += 16) {
      uint64_t to[4];
      uint32_t w[4][4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = r0 + 4 * i;
        to[i] = __shfl_sync(0xffffffffu, reinterpret_cast<uint64_t>(dst), row);
        ld_shared_v4(buf + row * 128 + (((lane & 7) ^ (row & 7)) << 4), w[i]);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (to[i] != 0)
          *reinterpret_cast<uint4*>(to[i] + 128 * c + (lane & 7) * 16) = make_uint4(w[i][0], w[i][1], w[i][2], w[i][3]);
    }
    __syncwarp();
  }
}

// The stream's four warps have all come here (and what they wrote to shared
// memory can be read).
template <int D>
__device__ __forceinline__ bool stream_sync(const Shared<D>& sh, const Params& p, int t, uint32_t& phase) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(sh.bar(Cfg<D>::kXch + t));
  const bool ok = warp_wait(sh, p, Cfg<D>::kXch + t, phase, 28 + t);
  phase ^= 1;
  return ok;
}

// The maximum of `a` and the sum of `b` over the stream's warps, lane by lane.
template <int D>
__device__ __forceinline__ bool exchange(const Shared<D>& sh, const Params& p, int t, float a, float b, float& a_max,
                                         float& b_sum, uint32_t& phase) {
  const uint32_t at = sh.xch(t) + (threadIdx.x & 31) * 8;
  st_shared_f32x2(at + ((threadIdx.x >> 5) & 3) * 256, a, b);
  if (!stream_sync<D>(sh, p, t, phase)) return false;
  float2 v[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) v[w] = ld_shared_f32x2(at + w * 256);
  a_max = fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x));
  b_sum = (v[0].y + v[1].y) + (v[2].y + v[3].y);
  return true;
}

// One key tile of a narrow item.  Its rows stand four times in the 128 lanes
// of S, once for each warp, which takes 32 of the tile's keys: the exp2 of few
// rows spread over all four sub-partitions instead of 128 in a row on one
// (2300 cycles a tile).  The warps agree on the rows' maxima, P goes to shared
// memory as the B operand of O^T = V^T P^T, and O^T, with a dim per lane and a
// row per column, needs no merging and leaves in coalesced stores.  Along with
// the maxima the warps exchange `extra`, which comes back summed.
template <int D>
__device__ __forceinline__ bool narrow_tile(const Shared<D>& sh, const Params& p, int t, uint32_t s_tm, uint32_t o_tm,
                                            int32_t visible, bool first, float& m_ref, float& l, float& extra,
                                            uint32_t& x_phase) {
  const int lane = threadIdx.x & 31, warp = (threadIdx.x >> 5) & 3;
  float s[32];
  {
    uint32_t r[32];
    tmem_ld32(s_tm + 32 * warp, r);
    tmem_wait_ld();
#pragma unroll
    for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(r[c]);
  }
  visible -= 32 * warp;
  if (visible < 32) {
    const uint32_t bits = visible <= 0 ? 0u : (1u << visible) - 1u;
#pragma unroll
    for (int c = 0; c < 32; ++c)
      if (!(bits >> c & 1)) s[c] = -INFINITY;
  }
  float mx[4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
    mx[c] = max3f(max3f(s[c], s[c + 4], s[c + 8]), max3f(s[c + 12], s[c + 16], s[c + 20]), fmaxf(s[c + 24], s[c + 28]));
  const float mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * p.scale_log2;
  float row_max;
  if (!exchange<D>(sh, p, t, mine, extra, row_max, extra, x_phase)) return false;
  const float m_new = fmaxf(m_ref, row_max);
  if (first) {
    m_ref = m_new;
  } else {
    const bool need = m_new > m_ref + kRescaleThreshold;  // the same in all four warps
    if (__any_sync(0xffffffffu, need)) {
      const float alpha = need ? fast_exp2(m_ref - m_new) : 1.0f;
      uint32_t o[32];
      tmem_ld32(o_tm, o);
      tmem_wait_ld();
#pragma unroll
      for (int c = 0; c < 32; ++c) o[c] = __float_as_uint(__uint_as_float(o[c]) * __shfl_sync(0xffffffffu, alpha, c));
      tmem_st32(o_tm, o);
      tmem_wait_st();
      if (need) {
        l *= alpha;
        m_ref = m_new;
      }
    }
  }
  const float neg = m_ref == -INFINITY ? 0.f : -m_ref;  // a row that has seen no key yet: every exponent is -inf
  const uint32_t row = sh.p_tile(t) + (warp >> 1) * (kNarrow * 128) + lane * 128;
  float sum[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t w[4];
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float a = fast_exp2(fmaf(s[8 * k + 2 * x], p.scale_log2, neg));
      const float b = fast_exp2(fmaf(s[8 * k + 2 * x + 1], p.scale_log2, neg));
      sum[x] += a + b;
      w[x] = pack_bf16x2(a, b);
    }
    st_shared_v4(row + ((((warp & 1) * 4 + k) ^ (lane & 7)) << 4), w[0], w[1], w[2], w[3]);
  }
  l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
  fence_proxy_async_smem();  // for the tensor cores
  return true;
}

// A narrow item's rows out of O^T: lane = dim, so a warp stores 32 dims of a
// row at once.  row: output or partial row of the lane's row (-1: none; no
// memory holds 2^31 of them); scale likewise.
template <int D>
__device__ __forceinline__ void store_columns(const Params& p, uint32_t o_tm, int32_t row, bool direct, float scale,
                                              int rows) {
  const int dim = threadIdx.x & 127;
  if (dim >= D) return;  // (whole warps)
#pragma unroll 1
  for (int c = 0; c < rows; c += 4) {
    uint32_t r[4];
    int32_t to[4];
    float o[4];
    tmem_ld4(o_tm + c, r);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      to[i] = __shfl_sync(0xffffffffu, row, c + i);
      o[i] = __shfl_sync(0xffffffffu, scale, c + i);
    }
    tmem_wait_ld();
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] *= __uint_as_float(r[i]);
    if (direct) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (to[i] >= 0) p.out[int64_t(to[i]) * D + dim] = __float2bfloat16_rn(o[i]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (to[i] >= 0) p.part_o[int64_t(to[i]) * D + dim] = o[i];
    }
  }
}

// Zeroes the rows of a V tile behind its `valid` keys, whatever their page
// holds there (0 * NaN would reach O): by the stream whose P is the first to
// meet the tile, before it hands P over.  (The swizzle permutes 16-byte pieces
// inside a row's 128 bytes only.)
template <int D>
__device__ __forceinline__ bool zero_tail(const Shared<D>& sh, const Params& p, int fill, int32_t valid) {
  using C = Cfg<D>;
  const int st = fill % C::kStages, th = threadIdx.x & 127;
  if (!warp_wait(sh, p, C::kKVFull + st, (fill / C::kStages) & 1, 26)) return false;
  const uint32_t base = sh.kv_tile(st) + (th & 7) * 16;
#pragma unroll 1
  for (int row = valid + (th >> 3); row < 128; row += 16) {
#pragma unroll
    for (int half = 0; half < C::kHalves; ++half)
      st_shared_v4(base + (row >> 3) * C::kGroup + half * kAtom + (row & 7) * 128, 0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  return true;
}

// A narrow item whose last key tile is under way.  Its rows are stored after the
// stream's next item has handed over its first P: O^T of the two lie apart, so
// neither the product nor the stores hold the other stream's MMAs up.
struct Pending {
  bool on = false;
  float m, l;
  int64_t row, lse;  // of the lane's row: output or partial row (-1: none), LSE
  int32_t rows;
  bool direct;
};

// Softmax statistics to LSE and scale of one row, and the row's destination.
template <int D>
__device__ __forceinline__ uint8_t* row_out(const Params& p, bool direct, int64_t row, int64_t lse, float m, float l,
                                            bool writes_lse, bool has_o) {
  if (row < 0) return nullptr;
  if (writes_lse) {
    const float x = l != 0.f ? (m + __log2f(l)) * kLn2 : -INFINITY;  // (a row's NaN stays one)
    if (!direct)
      p.part_lse[row] = x;
    else if (p.lse)
      p.lse[lse] = x;
  }
  if (!has_o) return nullptr;
  return direct ? reinterpret_cast<uint8_t*>(p.out + row * D) : reinterpret_cast<uint8_t*>(p.part_o + row * D);
}

template <int D>
__device__ __forceinline__ void softmax_role(const Shared<D>& sh, const Params& p, uint32_t tmem, int t) {
  using C = Cfg<D>;
  const int warp = (threadIdx.x / 32) % 4;
  const uint32_t lane_off = uint32_t(warp * 32) << 16;
  const uint32_t s_tm = tmem + lane_off + uint32_t(128 * t);
  const uint32_t o_tm = tmem + lane_off + uint32_t(256 + 128 * t);
  const int32_t prefix_len = p.hdr->prefix_len;
  const int64_t half_rows = int64_t(p.max_ctok) * p.H;
  uint32_t s_phase = 0, o_phase = 0, x_phase = 0, ot = 0;
  Pending pend;
  auto store_pending = [&](float sum) {
    row_out<D>(p, pend.direct, pend.row, pend.lse, pend.m, sum, warp == 0, true);
    store_columns<D>(p, o_tm + kNarrow * (ot ^ 1), int32_t(pend.row), pend.direct, sum != 0.f ? __frcp_rn(sum) : 0.f,
                     pend.rows);
    pend.on = false;
  };
  for (int it = 0;; ++it) {
    // The item stays in shared memory until its last use and is read again
    // there: held in registers across the key tiles it made ptxas spill.
    if (!warp_wait(sh, p, C::kItemFull + it % kItems, (it / kItems) & 1, 20 + t)) return;
    const uint32_t item = sh.item(it);
    const int32_t j1 = item_field(item, offsetof(Item, j1));
    const bool narrow = item_field(item, offsetof(Item, head)) & 1;
    if (pend.on && !narrow) {
      // nothing to overlap it with (the end), or an item that uses all of O
      // (between tiles, S(m) separates one exchange from the next; here the stream meets before and after)
      float none, sum;
      if (!stream_sync<D>(sh, p, t, x_phase)) return;
      if (!exchange<D>(sh, p, t, 0.f, pend.l, none, sum, x_phase)) return;
      if (!stream_sync<D>(sh, p, t, x_phase)) return;
      if (!warp_wait(sh, p, C::kOFull + t, o_phase, 24 + t)) return;
      o_phase ^= 1;
      tc_fence_after();
      ot ^= 1;
      store_pending(sum);
      ot ^= 1;
    }
    if (j1 == 0) return;
    const int32_t row = threadIdx.x & (narrow ? kNarrow - 1 : 127);
    const int32_t row_tok = int32_t(uint32_t(row) * p.group_inv >> 16);  // row / group, exact below 2^8
    const bool pair = item_field(item, offsetof(Item, ntok)) > p.tile_tokens;
    const int32_t other = t ^ item_field(item, offsetof(Item, parity));
    const int32_t tok_i = (pair && other ? p.tile_tokens : 0) + row_tok;  // token inside the unit
    const bool live = row_tok < p.tile_tokens && tok_i < item_field(item, offsetof(Item, ntok));
    const bool warp_live = __any_sync(0xffffffffu, live);
    const int32_t ptiles = item_field(item, offsetof(Item, ptiles));
    const int32_t len = item_field(item, offsetof(Item, len));
    int32_t limit;  // own keys that this row sees
    {
      const uint32_t pos = uint32_t(item_field(item, offsetof(Item, pos0)) + tok_i), block = uint32_t(p.block_tokens);
      const uint32_t seen = block == 1 ? pos + 1 : (pos / block + 1) * block;  // at most pos + block: below 2^32
      limit = int32_t(seen < uint32_t(len) ? seen : uint32_t(len));
    }
    // two row tiles: every key tile for one of them; one: every second key tile
    const int32_t j0 = item_field(item, offsetof(Item, j0)), tile0 = item_field(item, offsetof(Item, tile0)) - j0;
    int32_t j = j0 + (pair ? 0 : other);
    const int32_t step = pair ? 1 : 2;
    float m_ref = -INFINITY;  // reference max (log2 units)
    float l = 0.f;
    bool first = true;
    for (; j < j1; j += step) {
      if (!warp_wait(sh, p, C::kSFull + t, s_phase, 22 + t)) return;
      s_phase ^= 1;
      const int32_t visible = j < ptiles ? prefix_len - j * 128 : limit - (j - ptiles) * 128;
      const int32_t keys = j < ptiles ? visible : len - (j - ptiles) * 128;  // of the tile, behind which rows are zeroed
      const bool ragged = keys < 128 && !(pair && other);
      const int32_t fill = 2 * (tile0 + j) + (pair ? 1 : 2);
      if (narrow) {
        tc_fence_after();
        if (first) ot ^= 1;
        float sum = pend.on ? pend.l : 0.f;
        if (!narrow_tile<D>(sh, p, t, s_tm, o_tm + kNarrow * ot, visible, first, m_ref, l, sum, x_phase)) return;
        first = false;
        if (ragged && !zero_tail<D>(sh, p, fill, keys)) return;
        // (before P is handed over: the item's own last product must not pass the one waited for)
        if (pend.on) {
          if (!warp_wait(sh, p, C::kOFull + t, o_phase, 24 + t)) return;
          o_phase ^= 1;
          tc_fence_after();
        }
        tc_fence_before();
        mbar_arrive(sh.bar(C::kPFull + t));
        if (pend.on) store_pending(sum);
        continue;
      }
      if (warp_live) {
        tc_fence_after();
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
          // bit c of word w: column 32 w + c is seen
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int32_t n = visible - 32 * w;
            const uint32_t bits = n >= 32 ? 0xffffffffu : n <= 0 ? 0u : (1u << n) - 1u;
#pragma unroll
            for (int c = 0; c < 32; ++c)
              if (!(bits >> c & 1)) s[32 * w + c] = -INFINITY;
          }
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
#pragma unroll 1
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
      if (ragged && !zero_tail<D>(sh, p, fill, keys)) return;
      mbar_arrive(sh.bar(C::kPFull + t));
    }
    const int32_t dest = item_field(item, offsetof(Item, dest));
    int64_t out_row = item_field64(item, offsetof(Item, row0)), lse = item_field64(item, offsetof(Item, lse0));
    const int32_t rows = item_field(item, offsetof(Item, ntok)) * p.group;
    const int32_t tok = item_field(item, offsetof(Item, tok0)) + tok_i;
    release_item<D>(sh, it);
    const int32_t row_head = row - row_tok * p.group;
    lse += int64_t(row_head) * p.max_tokens + tok_i;
    if (dest == kCut) {
      out_row += (pair ? other : t) * 128 + row;
    } else if (dest == kMainPrefix) {
      const int32_t ct = live ? p.ctok[tok] : -1;
      // a larger request's row in a shared tile has its prefix elsewhere
      out_row = ct < 0 ? -1 : out_row + (pair ? 0 : t * half_rows) + int64_t(ct) * p.H + row_head;
    } else {
      out_row += int64_t(tok_i) * p.H + row_head + (dest == kMainOwn ? t * half_rows : 0);
    }
    // no key tile of this item on this stream: a direct item's rows are the other stream's
    if (!live || (first && dest == kDirect)) out_row = -1;
    if (narrow && !first) {
      pend.on = true;
      pend.m = m_ref;
      pend.l = l;
      pend.row = out_row;
      pend.lse = lse;
      pend.rows = rows;
      pend.direct = dest == kDirect;
      continue;
    }
    if (!first) {
      if (!warp_wait(sh, p, C::kOFull + t, o_phase, 24 + t)) return;
      o_phase ^= 1;
      tc_fence_after();
    }
    uint8_t* dst = row_out<D>(p, dest == kDirect, out_row, lse, m_ref, l, !narrow || warp == 0, !first);
    if (!first && warp_live) store_rows<D>(sh, o_tm, dst, dest == kDirect, l != 0.f ? __frcp_rn(l) : 0.f);
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    batch_attn_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_narrow,
                      const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                      const Params p) {
  using C = Cfg<D>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const Shared<D> sh{raw, (raw + C::kSmall + 1023) & ~1023u};
  if (sh.tiles + C::kTiles > raw + C::kSmemBytes) {  // dynamic shared memory not on a 1024-byte boundary: never seen
    cudaGridDependencySynchronize();
    if (threadIdx.x == 0) p.status->code = WF_ERR_ALIGNMENT;
    return;
  }
  const int warp = __shfl_sync(0xffffffffu, int(threadIdx.x) / 32, 0);
  const int lane = threadIdx.x % 32;

  Share share{};
  wf_batch_unit unit{};
  int64_t unit_at = 0;
  if (warp == 9) {
    for (int b = lane; b < C::kNumBars; b += 32) {
      uint32_t count = 1;
      if (b == C::kPFull || b == C::kPFull + 1) count = 128;  // a stream's softmax threads
      if (b >= C::kItemEmpty && b < C::kItemEmpty + kItems) count = kItemReaders;
      if (b == C::kXch || b == C::kXch + 1) count = 4;  // a stream's warps
      mbar_init(sh.bar(b), count);
    }
    if (lane == 0) st_shared_u32(sh.base + Shared<D>::kAbortAt, 0);
    if (lane < 2 * C::kStages) st_shared_u32(sh.fills(0, 0) + 4 * lane, 0);
    fence_barrier_init();
    fence_proxy_async_smem();
    if (lane == 0) {
      tma_prefetch_desc(&tm_q);
      tma_prefetch_desc(&tm_k);
      tma_prefetch_desc(&tm_v);
    }
  } else if (warp == 8) {
    tmem_alloc(sh.base + Shared<D>::kTmemAt, kTmemCols);
    tmem_relinquish();
  }
  // Launched while the stream's previous kernel may still run: nothing before
  // this line reads or writes global memory.
  cudaGridDependencySynchronize();
  // The merging kernel may come onto this SM as soon as this block leaves it.
  // (Behind the wait: it reads the plan before it waits itself.)
  cudaTriggerProgrammaticLaunchCompletion();
  if (warp == 10) {
    share = first_share(p);
    load_unit(p, share, share.head, share.unit + lane, unit, unit_at);
  }
  if (blockIdx.x == 0 && threadIdx.x == 0 && p.hdr->fingerprint != p.fingerprint)
    p.status->code = WF_ERR_PLAN;  // not built, or for another description: the scheduler finds no work
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = ld_shared_u32(sh.base + Shared<D>::kTmemAt);

  if (warp < 8) {
    regs_increase<kSoftmaxRegs>();
    softmax_role<D>(sh, p, tmem, warp / 4);
  } else {
    regs_decrease<kControlRegs>();
    if (warp == 8)
      mma_issuer<D>(sh, p, __shfl_sync(0xffffffffu, tmem, 0));
    else if (warp == 9)
      k_producer<D>(sh, p, &tm_q, &tm_narrow, &tm_k);
    else if (warp == 10)
      scheduler<D>(sh, p, share, unit, unit_at);
    else
      v_producer<D>(sh, p, &tm_v);
  }
  tc_fence_before();
  __syncthreads();
  if (sh.aborting() && warp == 9 && lane < C::kStages) {
    const uint32_t k = ld_shared_u32(sh.fills(0, lane)), v = ld_shared_u32(sh.fills(1, lane)), last = k > v ? k : v;
    if (last > 0) wait_alone(sh.bar(C::kKVFull + lane), ((last - 1) / C::kStages) & 1, p.timeout_ns);
  }
  if (warp == 8) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemCols);
  }
}

// ---------------------------------------------------------------- merging parts
// Eight lanes a row, four rows a warp.  A row's parts, in this order: its own
// unit's shares, then (requests that share the prefix) the shares of the
// prefix unit that holds its token.  Eight parts at a time: lane i finds part
// i's row and LSE, the eight their maximum and weights, and the O rows are then
// summed, D / 8 dims per lane.  (A warp a row spent most of its instructions on
// finding the parts: 690 a row, 24 us for 22500 rows.)
struct Parts {
  int64_t s;      // cost position of the unit
  int32_t shift, ktiles;
  int c0, n;      // first share; parts
  bool pair, cut, own;
  int32_t half, row;  // of a two-tile unit: the row's tile; the row in its tile
};

__device__ __forceinline__ Parts parts_of(const Params& p, const Line& line, const wf_batch_unit& u, int64_t s,
                                          int32_t tok_i, int32_t row_head) {
  Parts q;
  q.s = s;
  q.pair = u.ntok > p.tile_tokens;
  q.shift = tile_shift(u.ntok, p.tile_tokens);
  q.ktiles = u.ktiles;
  q.c0 = share_of(line, s);
  const int c1 = u.ktiles == 1 ? q.c0 : share_of(line, s + (int64_t(u.ktiles - 1) << q.shift));
  q.cut = c1 > q.c0;
  q.own = u.req >= 0;
  q.n = (c1 - q.c0 + 1) * (q.pair ? 1 : 2);
  q.half = tok_i >= p.tile_tokens;
  q.row = (tok_i - q.half * p.tile_tokens) * p.group + row_head;
  return q;
}

// Row index of part i, or -1 if that share holds none of the unit's tiles.
__device__ __forceinline__ int64_t part_row(const Params& p, const Line& line, const Parts& q, int i, int32_t ct,
                                            int32_t head) {
  const int half = q.pair ? q.half : i & 1;
  if (!q.cut) return main_row(p, q.own, q.pair ? 0 : half, ct, head);
  const int c = q.c0 + (q.pair ? i : i >> 1);
  int32_t j0, j1;
  share_tiles(q.s, q.shift, q.ktiles, share_begin(line, c), share_begin(line, c + 1), j0, j1);
  return j0 < j1 ? cut_row(p, c, j0 == 0, half, q.row) : -1;
}

// Merges the row of this lane's group of eight (`on`: there is one) and stores
// it.  ct, head: where parts of uncut units lie.
template <int D>
__device__ __forceinline__ void merge_row(const Params& p, const Line& line, bool on, const Parts& a, const Parts& b,
                                          int32_t ct, int32_t head, int32_t tok) {
  constexpr int Q = D / 32;  // float4s per lane: dims 4 (g + 8 q) .. + 3
  constexpr int kAhead = 16 / Q;  // parts whose loads are in flight
  const int g = threadIdx.x & 7, group = threadIdx.x & 24;
  float m = -INFINITY, l = 0.f;
  float4 acc[Q];
#pragma unroll
  for (int q = 0; q < Q; ++q) acc[q] = make_float4(0.f, 0.f, 0.f, 0.f);
  const int n = on ? a.n + b.n : 0, most = __reduce_max_sync(0xffffffffu, n);
#pragma unroll 1
  for (int base = 0; base < most; base += 8) {
    const int i = base + g;
    int64_t row = -1;
    if (i < n) row = i < a.n ? part_row(p, line, a, i, ct, head) : part_row(p, line, b, i - a.n, ct, head);
    const float x = row >= 0 ? p.part_lse[row] : -INFINITY;
    // the first O rows are on their way before their weights are known: one latency instead of two
    float4 o[kAhead][Q];
    auto load = [&](int k) {
#pragma unroll
      for (int c = 0; c < kAhead; ++c) {
        const int64_t r = __shfl_sync(0xffffffffu, row, group + k + c);
        const float4* src = reinterpret_cast<const float4*>(p.part_o + r * D) + g;
#pragma unroll
        for (int q = 0; q < Q; ++q) o[c][q] = r >= 0 ? __ldcs(src + 8 * q) : make_float4(0.f, 0.f, 0.f, 0.f);
      }
    };
    load(0);
    float mx = x;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    const float m_new = fmaxf(m, mx);
    const float old = m == -INFINITY ? 0.f : __expf(m - m_new);
    const float w = x == -INFINITY ? 0.f : __expf(x - m_new);
    float ws = w;
#pragma unroll
    for (int off = 4; off > 0; off >>= 1) ws += __shfl_xor_sync(0xffffffffu, ws, off);
    l = l * old + ws;
    m = m_new;
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      acc[q].x *= old; acc[q].y *= old; acc[q].z *= old; acc[q].w *= old;
    }
#pragma unroll 1
    for (int k = 0; k < 8 && base + k < most; k += kAhead) {
      if (k > 0) load(k);
#pragma unroll
      for (int c = 0; c < kAhead; ++c) {
        const float wk = __shfl_sync(0xffffffffu, w, group + k + c);
        // (a part that saw no key has no O row: whatever lies there is not used)
#pragma unroll
        for (int q = 0; q < Q; ++q)
          if (wk != 0.f) {
            acc[q].x = fmaf(wk, o[c][q].x, acc[q].x);
            acc[q].y = fmaf(wk, o[c][q].y, acc[q].y);
            acc[q].z = fmaf(wk, o[c][q].z, acc[q].z);
            acc[q].w = fmaf(wk, o[c][q].w, acc[q].w);
          }
      }
    }
  }
  if (!on) return;
  const float inv = l != 0.f ? __frcp_rn(l) : 0.f;
  uint2* dst = reinterpret_cast<uint2*>(p.out + (int64_t(tok) * p.H + head) * D) + g;
#pragma unroll
  for (int q = 0; q < Q; ++q)
    dst[8 * q] = make_uint2(pack_bf16x2(acc[q].x * inv, acc[q].y * inv), pack_bf16x2(acc[q].z * inv, acc[q].w * inv));
  if (g == 0 && p.lse) p.lse[int64_t(head) * p.max_tokens + tok] = l != 0.f ? m + logf(l) : -INFINITY;
}

constexpr int kCombineThreads = 128;
constexpr int kCombineRows = kCombineThreads / 8;  // a block at a time

// Launched while the attention still runs (programmatic dependent launch): what
// does not depend on its results is read first.
template <int D>
__global__ void __launch_bounds__(kCombineThreads, 4) batch_combine_kernel(const Params p) {
  const wf_batch_hdr* h = p.hdr;
  const Line line = line_of(p);
  if (h->fingerprint != p.fingerprint || line.total == 0) {
    cudaGridDependencySynchronize();  // what follows on the stream waits for this kernel alone
    return;
  }
  const int np = h->prefix_units, ctas = h->ctas;
  const int sub = threadIdx.x >> 3;
  const Parts none{};
  bool waited = false;
  // rows of one-tile units
  const int64_t rows = int64_t(h->ctoks) * p.H;  // at most 2^20 tokens x 2^12 heads
#pragma unroll 1
  for (int64_t k0 = int64_t(blockIdx.x) * kCombineRows; k0 < rows; k0 += int64_t(gridDim.x) * kCombineRows) {
    const uint32_t k = uint32_t(k0 + sub);  // (rows fit 32 bits)
    const uint32_t ct = k / uint32_t(p.H);
    const int32_t head = int32_t(k - ct * uint32_t(p.H)), kv = head / p.group, row_head = head - kv * p.group;
    bool on = k < rows;
    Parts a = none, b = none;
    int32_t tok = 0;
    if (on) {
      const wf_batch_ctok at = p.ctok_list[ct];
      tok = at.tok;
      const int32_t pu = tok / (2 * p.tile_tokens), pi = pu < np ? pu : at.unit;
      const wf_batch_unit u = p.units[at.unit], q = p.units[pi];
      const int64_t s0 = int64_t(kv) * line.head_cost, su = s0 + p.pre[at.unit], sq = s0 + p.pre[pi];
      on = !unit_direct(u, p.tile_tokens);  // a single tile, never cut
      a = parts_of(p, line, u, su, tok - u.tok0, row_head);
      if (u.ptiles < 0) b = parts_of(p, line, q, sq, tok - q.tok0, row_head);
    }
    if (!waited) cudaGridDependencySynchronize();
    waited = true;
    merge_row<D>(p, line, on, a, b, int32_t(ct), head, tok);
  }
  if (!waited) cudaGridDependencySynchronize();
  // rows of two-tile units that were cut; a unit is taken up at its first cut
  if (p.max_tokens <= p.tile_tokens) return;
  constexpr int kBlocks = 256 / kCombineRows;
#pragma unroll 1
  for (int k = blockIdx.x; k < ctas * kBlocks; k += gridDim.x) {
    const int r = k % kBlocks * kCombineRows + sub, half = r >> 7, row = r & 127;
    const Cut cut = p.cuts[k / kBlocks];
    if (cut.n == 0) continue;
    const bool on = row < (half ? cut.ntok - p.tile_tokens : p.tile_tokens) * p.group;
    Parts a;
    a.s = cut.s;
    a.shift = WF_BATCH_PAIR_SHIFT;
    a.ktiles = cut.ktiles;
    a.c0 = cut.c0;
    a.n = cut.n;
    a.pair = a.cut = a.own = true;
    a.half = half;
    a.row = row;
    const int32_t ti = row / p.group;
    merge_row<D>(p, line, on, a, none, 0, cut.head * p.group + (row - ti * p.group),
                 cut.tok0 + (half ? p.tile_tokens : 0) + ti);
  }
}

// ---------------------------------------------------------------- host
PFN_cuTensorMapEncodeTiled_v12000 get_encode() {
  static std::atomic<PFN_cuTensorMapEncodeTiled_v12000> known{nullptr};
  PFN_cuTensorMapEncodeTiled_v12000 fn = known.load(std::memory_order_relaxed);
  if (!fn) {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &ptr, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess) {
      cudaGetLastError();
      return nullptr;
    }
    fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
    known.store(fn, std::memory_order_relaxed);
  }
  return fn;
}

bool encode_map(CUtensorMap* tm, const void* base, int rank, const cuuint64_t* dims, const cuuint64_t* strides,
                const cuuint32_t* box) {
  auto encode = get_encode();
  const cuuint32_t ones[5] = {1, 1, 1, 1, 1};
  return encode && encode(tm, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, cuuint32_t(rank), const_cast<void*>(base), dims, strides,
                          box, ones, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                          CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// q [tokens, heads, D]: boxes of 64 dims x group heads x tile_tokens tokens.
bool make_q_map(CUtensorMap* tm, const void* base, int64_t tokens, int32_t heads, int32_t dim, int32_t group,
                int32_t tile_tokens) {
  const cuuint64_t row = cuuint64_t(dim) * 2;
  const cuuint64_t dims[3] = {cuuint64_t(dim), cuuint64_t(heads), cuuint64_t(tokens)};
  const cuuint64_t strides[2] = {row, row * heads};
  const cuuint32_t box[3] = {64, cuuint32_t(group), cuuint32_t(tile_tokens)};
  return encode_map(tm, base, 3, dims, strides, box);
}

// A pool [tokens, heads, D] as (64 dims, 8 tokens, halves, groups of 8 tokens,
// heads); a box is one head's rows of a page.
bool make_pool_map(CUtensorMap* tm, const void* base, int64_t tokens, int32_t heads, int32_t dim, int32_t page) {
  const cuuint64_t row = cuuint64_t(dim) * 2, token = row * heads;
  const cuuint64_t dims[5] = {64, 8, cuuint64_t(dim / 64), cuuint64_t(tokens / 8), cuuint64_t(heads)};
  const cuuint64_t strides[4] = {token, 128, 8 * token, row};
  const cuuint32_t box[5] = {64, 8, cuuint32_t(dim / 64), cuuint32_t(page / 8), 1};
  return encode_map(tm, base, 5, dims, strides, box);
}

// Held while a call's two kernels are launched, so that they stand right behind
// one another: on a stream and workspace that two threads use, another call's
// parts would otherwise come between these and their merging.  One of several
// locks by workspace, for calls that share nothing to seldom meet (about 20 ns).
std::mutex& between_kernels(const void* workspace) {
  static std::mutex locks[64];
  return locks[(reinterpret_cast<uintptr_t>(workspace) >> 8) % 64];
}

template <int D>
wf_status launch(const wf_batch_desc* d, const BatchLayout& L, const Params& p, const void* q, const void* k_pool,
                 const void* v_pool, cudaStream_t stream) {
  static std::atomic<int> attr_done[64];  // (threads may find out the same at once)
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
  CUtensorMap tq, tn, tk, tv;
  // (a group of more than kNarrow heads has no narrow items)
  if (!make_q_map(&tq, q, d->max_tokens, d->num_heads, D, L.group, L.tile_tokens) ||
      !make_q_map(&tn, q, d->max_tokens, d->num_heads, D, L.group, std::max(1, kNarrow / L.group)) ||
      !make_pool_map(&tk, k_pool, pool, d->num_kv_heads, D, d->page_tokens) ||
      !make_pool_map(&tv, v_pool, pool, d->num_kv_heads, D, d->page_tokens))
    return WF_ERR_CUDA;
  const std::lock_guard<std::mutex> both(between_kernels(p.status));
  const wf_status launched =
      launch_early(batch_attn_kernel<D>, unsigned(L.ctas), kThreads, Cfg<D>::kSmemBytes, stream, tq, tn, tk, tv, p);
  if (launched != WF_OK) return launched;
  // as many blocks as the rows that may have to be merged fill, or as run at once a few times over
  const int64_t rows = std::max(L.max_ctok * d->num_heads, d->max_tokens > L.tile_tokens ? int64_t(L.ctas) * 256 : 0);
  const int64_t blocks = (rows + kCombineRows - 1) / kCombineRows, most = int64_t(L.ctas) * 16;
  return launch_early(batch_combine_kernel<D>, unsigned(blocks < most ? blocks : most), kCombineThreads, 0, stream, p);
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
  // other blocks still read what one of them would write over
  constexpr size_t kBf16 = 2;
  const size_t T = size_t(desc->max_tokens), H = size_t(desc->num_heads), D = size_t(desc->head_dim);
  const size_t pool_bytes = size_t(desc->pool_pages) * size_t(desc->page_tokens) * size_t(desc->num_kv_heads) * D * kBf16;
  const wf::Span in[] = {
      {plan, L.plan_bytes}, {q, T * H * D * kBf16}, {k_pool, pool_bytes}, {v_pool, pool_bytes},
      {block_table, size_t(desc->max_requests) * size_t(desc->max_request_pages) * sizeof(int32_t)},
      {prefix_table, size_t(desc->max_prefix_pages) * sizeof(int32_t)}};
  const wf::Span results[] = {{out, T * H * D * kBf16}, {lse, T * H * sizeof(float)}, {workspace, L.workspace_bytes}};
  if (wf::written_over(results, in)) return WF_ERR_INVALID_ARG;
  if (wf::misaligned(plan) || wf::misaligned(q) || wf::misaligned(k_pool) || wf::misaligned(v_pool) ||
      wf::misaligned(out) || wf::misaligned(workspace) || reinterpret_cast<uintptr_t>(lse) % 4 ||
      reinterpret_cast<uintptr_t>(block_table) % 4 || reinterpret_cast<uintptr_t>(prefix_table) % 4)
    return WF_ERR_ALIGNMENT;
  if (workspace_bytes < L.workspace_bytes) return WF_ERR_WORKSPACE;
  if (!(softmax_scale >= 0.f) || !std::isfinite(softmax_scale)) return WF_ERR_INVALID_ARG;
  if (!wf::on_current_device(plan)) return WF_ERR_INVALID_ARG;
  const double scale = softmax_scale == 0.f ? 1.0 / std::sqrt(double(desc->head_dim)) : double(softmax_scale);

  wf::Params p{};
  const uint8_t* pl = static_cast<const uint8_t*>(plan);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  p.hdr = reinterpret_cast<const wf_batch_hdr*>(pl);
  p.starts = reinterpret_cast<const wf_batch_start*>(pl + L.off_starts);
  p.units = reinterpret_cast<const wf_batch_unit*>(pl + L.off_units);
  p.pre = reinterpret_cast<const int64_t*>(pl + L.off_pre);
  p.ctok = reinterpret_cast<const int32_t*>(pl + L.off_ctok);
  p.ctok_list = reinterpret_cast<const wf_batch_ctok*>(pl + L.off_ctok_list);
  p.table = block_table;
  p.prefix_table = prefix_table;
  p.out = static_cast<__nv_bfloat16*>(out);
  p.lse = lse;
  p.status = reinterpret_cast<wf_dev_status*>(ws);
  p.part_o = reinterpret_cast<float*>(ws + WF_ATTN_STATUS_BYTES);
  p.part_lse = reinterpret_cast<float*>(ws + L.off_lse);
  p.cuts = reinterpret_cast<wf::Cut*>(ws + L.off_cuts);
  p.main_rows = L.main_rows;
  p.fingerprint = L.fingerprint;
  p.timeout_ns = wf::wait_timeout_ns();
  p.scale_log2 = float(scale * 1.4426950408889634);
  const char* stall = std::getenv("WF_DEBUG_STALL_FIRST_LOAD");
  p.stall_first_load = stall && stall[0] == '1';
  p.H = desc->num_heads;
  p.kv_heads = desc->num_kv_heads;
  p.group = L.group;
  p.group_inv = uint32_t((65536 + L.group - 1) / L.group);
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
