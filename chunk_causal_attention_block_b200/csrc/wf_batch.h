// Internal layout of the batch plan: the device buffer that wf_batch_tables
// fills from request lengths on the GPU and that wf_batch_append and
// wf_batch_attn read.  Nothing of it is known to the host, which only sizes
// it from the capacities of wf_batch_desc.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "wf.h"
#include "wf_plan.h"

// Key tiles are shared out to CTAs by cost.  A tile against two row tiles
// (256 rows) costs 1 << WF_BATCH_PAIR_SHIFT, against one 1 <<
// WF_BATCH_SINGLE_SHIFT, and every unit WF_BATCH_UNIT_COST more for filling
// and draining the pipeline.  (A single tile at the cost of a pair: 64 decoding
// requests 54 -> 67 us, a round of two branches 2.1 -> 2.6 ms.  A unit at 1, 2,
// 3 or 8 instead of 4: within 6% both ways, as the cuts happen to fall.)
#define WF_BATCH_PAIR_SHIFT 3
#define WF_BATCH_SINGLE_SHIFT 2
#define WF_BATCH_UNIT_COST 4
#define WF_BATCH_CUT_BYTES 32  // workspace per CTA beside its partial rows

// One work unit of the attention, for one key head: up to two 128-row tiles of
// queries (tokens tok0 .. tok0+ntok-1, each with the key head's query heads)
// against ktiles 128-key tiles, the first ptiles of them the prefix's.
struct wf_batch_unit {
  int32_t req;     // request, or -1: rows of all requests against the prefix alone
  int32_t tok0;    // first new token (row of q)
  int32_t ntok;    // new tokens; more than a tile's tokens: two row tiles
  int32_t ktiles;  // key tiles; 0: nothing to do
  int32_t ptiles;  // prefix tiles at the front; -1: none, the rows' prefix part comes from a req -1 unit
  int32_t cbase;   // partial-row index of token tok0 (units of one row tile), else -1
  int32_t pos0;    // own position (without the prefix) of token tok0
  int32_t len;     // own tokens of the request, cached and new
};
static_assert(sizeof(wf_batch_unit) == 32, "unit record layout");

struct wf_batch_hdr {
  wf_dev_status status;   // 0: what the table builder found wrong with the lengths (all zero: nothing)
  uint64_t fingerprint;   // 16: of the description that the plan was built for
  int32_t tokens;         // 24: new tokens of the step
  int32_t units;          // 28: records in the unit list
  int32_t prefix_units;   // 32: of them, the leading ones with req = -1
  int32_t prefix_len;     // 36
  int32_t ctas;           // 40: CTAs that get a share
  int32_t ctoks;          // 44: tokens of one-tile units
  int64_t head_cost;      // 48: cost of one key head's units
  int64_t share;          // 56: cost of a CTA's share of all heads'
  double share_rcp;       // 64: 1 / share
  int32_t pad[46];
};

// Where a CTA's share of the work begins.
struct wf_batch_start {
  int32_t head, unit;
};

// A token of a one-tile unit: its rows may have to be merged from parts.
struct wf_batch_ctok {
  int32_t tok, unit;
};
static_assert(sizeof(wf_batch_hdr) == 256, "batch plan header layout");

// What a call reads of any plan, before it knows whether it was built for its
// own description: the header and its CTAs' starts.  Every plan has room for
// the most CTAs, so that another description's, however small, can be read.
#define WF_BATCH_MAX_CTAS 256
#define WF_BATCH_PLAN_HEAD (sizeof(wf_batch_hdr) + WF_BATCH_MAX_CTAS * sizeof(wf_batch_start))

namespace wf {

// Sizes and offsets that follow from a description (valid if ok).
struct BatchLayout {
  wf_status error;
  int32_t group;         // query heads per key head
  int32_t tile_tokens;   // tokens of a 128-row tile: floor(128 / group)
  int32_t ctas;
  int32_t max_units;
  int64_t max_ctok;      // capacity of partial-row tokens
  size_t off_starts, off_units, off_pre, off_ctok, off_ctok_list, plan_bytes;
  int64_t main_rows;     // partial rows of uncut units; those of the CTAs' cuts follow
  size_t off_cuts, off_lse, workspace_bytes;  // partial O first, after the status block
  uint64_t fingerprint;
};

BatchLayout batch_layout(const wf_batch_desc* d);

// Memory that a call may touch, [lo, hi); no pointer or no bytes: none.
struct Span {
  uintptr_t lo, hi;
  const void* ptr;
  Span(const void* p, size_t bytes) : ptr(p) {
    lo = p && bytes ? reinterpret_cast<uintptr_t>(p) : 0;
    hi = lo == 0 ? 0 : bytes > ~lo ? ~uintptr_t(0) : lo + bytes;
  }
};

inline bool overlap(const Span& a, const Span& b) { return (a.lo < b.hi) & (b.lo < a.hi); }

// Whether an output shares memory with an input or with another output: blocks
// of one call read and write without any order between them.
template <size_t N, size_t M>
inline bool written_over(const Span (&out)[N], const Span (&in)[M]) {
  bool any = false;  // (all pairs without a branch: 0.05 us of a call)
  for (size_t o = 0; o < N; ++o) {
    for (size_t i = 0; i < M; ++i) any |= overlap(out[o], in[i]);
    for (size_t i = 0; i < o; ++i) any |= overlap(out[o], out[i]);
  }
  return any;
}

// Whether ptr is memory of the current device: elsewhere a kernel would fault on it.
bool on_current_device(const void* ptr);

#ifdef __CUDACC__
// Launches a kernel that may start while the kernel before it in the stream
// still runs, and that touches no global memory before it has called
// cudaGridDependencySynchronize (but what older kernels than that one wrote).
// Such kernels read with plain loads: __ldg is for data that nobody writes while
// the kernel runs, which here begins before the wait ends.
// Saves the gap between two kernels, 1.5 to 2 us: one token's attention 12.3 ->
// 10.7 us a call, 64 decoding requests 53.7 -> 51.7 us.
template <typename... Params, typename... Args>
wf_status launch_early(void (*kernel)(Params...), unsigned blocks, unsigned threads, size_t smem, cudaStream_t stream,
                       const Args&... args) {
  cudaLaunchAttribute early{};
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  if (cudaLaunchKernelEx(&cfg, kernel, Params(args)...) == cudaSuccess) return WF_OK;
  cudaGetLastError();
  return WF_ERR_CUDA;
}
#endif

}  // namespace wf
