// wf_batch_tables: block tables, slot maps and the attention's work list of a
// batch of requests, built on the GPU from the requests' lengths, so that one
// captured graph serves steps of any lengths and the host never waits for
// them.
//
// With c_b cached and f_b new tokens of request b, pages of P tokens and
// exclusive sums written E[.]:
//   token_start_b = E[f]_b
//   pages held h_b (given, or ceil(c_b / P)); needed n_b = max(h_b, ceil((c_b + f_b) / P))
//   table[b][i] = free_pages[free_head + E[n - h]_b + i - h_b]   for h_b <= i < n_b
//   new token i of b: local position x = c_b + i, position prefix_len + x,
//   slot table[b][x / P] * P + x mod P
//
// One launch without any exchange between blocks: every block sums all
// requests' lengths itself (one block-wide scan; a few KB from L2), block 0
// writes the per-request results and the work list, the others each take a
// share of the new tokens and find a token's request by bisection in shared
// memory.  A thread whose token opens a page writes that page's table entry,
// so nobody reads an entry that somebody else writes.  All sums are 64-bit; what
// does not fit voids the whole step (no tokens, no work, tables untouched) and
// is recorded in the plan.
//
// Not bound by its few bytes: up to about 1000 requests by latency (launch, scan,
// bisection; a call in a graph 4.5 us for 5 and 64 requests, 6.1 for 512, 7.8 for
// 1024), beyond that by block 0, which makes all units and finds where all
// shares begin (10.9 us for 2048, 22 for 4096, 51 for 8192).
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "wf_batch.h"

namespace {

struct TablesParams {
  const int32_t* cached;
  const int32_t* fresh;
  const int32_t* prefix_len;
  const int32_t* held;
  const int32_t* free_pages;
  const int32_t* free_head;
  int32_t* free_head_out;
  int32_t* held_out;
  int32_t* table;
  int32_t* token_start;
  int32_t* slot_map;
  int32_t* positions;
  wf_batch_hdr* hdr;
  wf_batch_start* starts;  // [max_ctas]
  wf_batch_unit* units;
  int64_t* pre;    // exclusive sums of unit costs
  int32_t* ctok;   // partial-row index of each token, -1 for none
  wf_batch_ctok* ctok_list;  // and the tokens by that index
  int32_t B, max_tokens, cols, max_prefix, num_free, pool_pages;
  int32_t page, page_shift, tile_tokens, block_tokens, kv_heads, max_ctas;
  uint64_t fingerprint;
};

// Exclusive block-wide sums of N 64-bit values per thread; totals in `total`.
// scratch: N * (warps + 1) values.
template <int N, int kThreads>
__device__ void block_scan(int64_t (&v)[N], int64_t (&total)[N], int64_t* scratch) {
  constexpr int kWarps = kThreads / 32;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int64_t inc[N];
#pragma unroll
  for (int k = 0; k < N; ++k) {
    inc[k] = v[k];
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, inc[k], off);
      if (lane >= off) inc[k] += o;
    }
    if (lane == 31) scratch[k * (kWarps + 1) + warp] = inc[k];
  }
  __syncthreads();
  // one warp per value turns the warps' sums into exclusive ones
  if (warp < N) {
    int64_t* row = scratch + warp * (kWarps + 1);
    const int64_t own = lane < kWarps ? row[lane] : 0;
    int64_t w = own;
#pragma unroll
    for (int off = 1; off < kWarps; off <<= 1) {
      const int64_t o = __shfl_up_sync(0xffffffffu, w, off);
      if (lane >= off) w += o;
    }
    if (lane < kWarps) row[lane] = w - own;
    if (lane == kWarps - 1) row[kWarps] = w;
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) {
    v[k] = inc[k] - v[k] + scratch[k * (kWarps + 1) + warp];
    total[k] = scratch[k * (kWarps + 1) + kWarps];
  }
  __syncthreads();  // scratch may be used again
}

// What a request adds to the sums, packed in three words so that the scan
// (64-bit shuffles, the block's main instruction load at 1024 requests) stays
// short: new tokens; new pages << 24 | tokens of one-tile units; own units <<
// 16 | small requests.  With f <= 2^22, at most 2^24 pages a request and 2^13
// requests no field reaches its neighbour (2^20 one-tile tokens, 2^13 small).
struct Sums {
  int64_t w[3];
  __device__ __forceinline__ void add(int32_t f, int32_t new_pages, int32_t tile_tokens) {
    const int32_t tiles = f <= tile_tokens ? f > 0 : (f + tile_tokens - 1) / tile_tokens;  // (mostly no division)
    w[0] += f;
    w[1] += (int64_t(new_pages) << 24) + ((tiles & 1) ? f - (tiles - 1) * tile_tokens : 0);
    w[2] += (int64_t((tiles + 1) / 2) << 16) + (f > 0 && f <= tile_tokens);
  }
};
__device__ __forceinline__ int64_t sum_tokens(const int64_t (&w)[3]) { return w[0]; }
__device__ __forceinline__ int64_t sum_pages(const int64_t (&w)[3]) { return w[1] >> 24; }
__device__ __forceinline__ int32_t sum_ctok(const int64_t (&w)[3]) { return int32_t(w[1] & 0xffffff); }
__device__ __forceinline__ int64_t sum_units(const int64_t (&w)[3]) { return w[2] >> 16; }
__device__ __forceinline__ int32_t sum_small(const int64_t (&w)[3]) { return int32_t(w[2] & 0xffff); }

// Last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int32_t* a, int n, int32_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (a[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

__device__ __forceinline__ int32_t ceil_shift(int64_t x, int s) { return int32_t((x + (int64_t(1) << s) - 1) >> s); }

__device__ __forceinline__ int64_t unit_cost(const TablesParams& p, int32_t ntok, int32_t ktiles) {
  const int shift = ntok > p.tile_tokens ? WF_BATCH_PAIR_SHIFT : WF_BATCH_SINGLE_SHIFT;
  return ktiles > 0 ? (int64_t(ktiles) << shift) + WF_BATCH_UNIT_COST : 0;
}

// Returns the unit's cost.  (Stored field by field, 1024 units took 8000 cycles.)
__device__ __forceinline__ int64_t store_unit(const TablesParams& p, int u, const wf_batch_unit& r) {
  int4* dst = reinterpret_cast<int4*>(p.units + u);
  dst[0] = make_int4(r.req, r.tok0, r.ntok, r.ktiles);
  dst[1] = make_int4(r.ptiles, r.cbase, r.pos0, r.len);
  return unit_cost(p, r.ntok, r.ktiles);
}

template <int kThreads>
__global__ void __launch_bounds__(kThreads) batch_tables_kernel(const TablesParams p) {
  extern __shared__ int32_t sm[];
  int32_t* s_start = sm;                // [B + 1] first token of each request
  int32_t* s_first = s_start + p.B + 1; // [B] first new page of each request, from free_head
  int32_t* s_ctok = s_first + p.B;      // [B] first partial-row token
  int32_t* s_unit = s_ctok + p.B;       // [B + 1] first own unit
  __shared__ int64_t scratch[3 * (kThreads / 32 + 1)];

  cudaGridDependencySynchronize();
  const int tid = threadIdx.x;
  const int per = (p.B + kThreads - 1) / kThreads;
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  const int Tt = p.tile_tokens;
  const int32_t prefix = p.prefix_len ? *p.prefix_len : 0;
  const int32_t head = *p.free_head;

  Sums v{};
  int64_t total[3];
  int bad = 0;  // 1: invalid, 2: does not fit
  for (int b = b0; b < b1; ++b) {
    const int32_t c = p.cached[b], f = p.fresh[b];
    const int32_t least = c < 0 ? 0 : ceil_shift(c, p.page_shift);
    const int32_t h = p.held ? p.held[b] : least;
    if (c < 0 || f < 0 || h < least) {
      bad |= 1;
      continue;
    }
    const int32_t n = max(h, ceil_shift(int64_t(c) + f, p.page_shift));
    if (n > p.cols || f > p.max_tokens) {
      bad |= 2;
      continue;
    }
    v.add(f, n - h, Tt);
  }
  block_scan<3, kThreads>(v.w, total, scratch);
  if (prefix < 0 || head < 0) bad |= 1;
  if (prefix > p.max_prefix || sum_tokens(total) > p.max_tokens || head + sum_pages(total) > p.num_free) bad |= 2;
  if (__syncthreads_or(bad)) {
    bad = __syncthreads_or(bad & 1);
    if (blockIdx.x == 0) {
      for (int b = tid; b <= p.B; b += kThreads) p.token_start[b] = 0;
      if (p.held_out)
        for (int b = tid; b < p.B; b += kThreads) p.held_out[b] = p.held[b];
      if (tid == 0) {
        *p.free_head_out = head;
        wf_batch_hdr h{};
        h.status.code = bad ? WF_ERR_INVALID_ARG : WF_ERR_CAPACITY;
        h.fingerprint = p.fingerprint;
        *p.hdr = h;
        p.pre[0] = 0;
      }
    }
    return;
  }

  // Requests of at most a row tile share their prefix tiles (see batch_attn.cu).
  // (With half a tile as the limit, 48 requests of 1 to 20 tokens, 5 heads to a
  // key head, took 133 us on a prefix of 4680: the larger ones read it alone.)
  const bool shared = prefix > 0 && sum_small(total) >= 2;
#pragma unroll 1
  for (int b = b0; b < b1; ++b) {
    const int32_t c = p.cached[b], f = p.fresh[b];
    const int32_t h = p.held ? p.held[b] : ceil_shift(c, p.page_shift);
    const int32_t n = max(h, ceil_shift(int64_t(c) + f, p.page_shift));
    s_start[b] = int32_t(sum_tokens(v.w));
    s_first[b] = int32_t(sum_pages(v.w));
    s_ctok[b] = sum_ctok(v.w);
    s_unit[b] = int32_t(sum_units(v.w));
    if (blockIdx.x == 0) {
      p.token_start[b] = s_start[b];
      if (p.held_out) p.held_out[b] = n;
    }
    v.add(f, n - h, Tt);
  }
  const int32_t tokens = int32_t(sum_tokens(total));
  if (tid == 0) {
    s_start[p.B] = tokens;
    s_unit[p.B] = int32_t(sum_units(total));
    if (blockIdx.x == 0) {
      p.token_start[p.B] = tokens;
      *p.free_head_out = head + int32_t(sum_pages(total));
    }
  }
  __syncthreads();

  const int32_t pair_tokens = 2 * Tt;
  const int32_t np = shared ? (tokens + pair_tokens - 1) / pair_tokens : 0;  // prefix units
  if (blockIdx.x > 0) {
    for (int64_t t64 = int64_t(blockIdx.x - 1) * kThreads + tid; t64 < tokens; t64 += int64_t(gridDim.x - 1) * kThreads) {
      const int32_t t = int32_t(t64);
      const int b = last_not_above(s_start, p.B, t);
      const int32_t i = t - s_start[b], c = p.cached[b], f = s_start[b + 1] - s_start[b];
      const int32_t h = p.held ? p.held[b] : ceil_shift(c, p.page_shift);
      const int32_t x = c + i, pi = x >> p.page_shift, in_page = x & (p.page - 1);
      int32_t* entry = p.table + int64_t(b) * p.cols + pi;
      int32_t pg;
      if (pi >= h) {
        pg = p.free_pages[head + s_first[b] + (pi - h)];
        if (in_page == 0) *entry = pg;
      } else {
        pg = *entry;
      }
      // a page outside the pool gets no slot: the append skips it
      p.slot_map[t] = pg >= 0 && pg < p.pool_pages ? pg * p.page + in_page : -1;
      p.positions[t] = prefix + x;
      const int32_t tiles = (f + Tt - 1) / Tt, tail = (tiles - 1) * Tt;
      const int32_t ct = (tiles & 1) && i >= tail ? s_ctok[b] + i - tail : -1;
      p.ctok[t] = ct;
      if (ct >= 0) p.ctok_list[ct] = {t, np + s_unit[b + 1] - 1};
    }
    return;
  }

  // ---- block 0: the attention's units (prefix units, then own ones) and the
  // running sum of their costs.  A thread makes consecutive units of each kind,
  // so that one scan does whatever their number, and keeps the first's cost.
  const int32_t ptiles = (prefix + 127) >> 7;
  const int32_t units = np + s_unit[p.B];
  int32_t first[2], behind[2];  // units of each kind that this thread makes
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    const int32_t begin = kind ? np : 0, end = kind ? units : np;
    const int32_t n = (end - begin + kThreads - 1) / kThreads;
    first[kind] = min(begin + tid * n, end);
    behind[kind] = min(first[kind] + n, end);
  }
  int64_t sum[2] = {0, 0}, all_costs[2], cost0[2] = {0, 0};
  for (int u = first[0]; u < behind[0]; ++u) {
    const int32_t tok0 = u * pair_tokens, ntok = min(pair_tokens, tokens - tok0);
    // it runs only if it holds a token of a small request (of its larger ones, a few at most, none is empty)
    int32_t ktiles = 0;
    for (int32_t t = tok0; t < tok0 + ntok && ktiles == 0;) {
      const int i = last_not_above(s_start, p.B, t);
      if (s_start[i + 1] - s_start[i] <= Tt) ktiles = ptiles;
      t = s_start[i + 1];
    }
    const int64_t cost = store_unit(p, u, {-1, tok0, ntok, ktiles, ptiles, -1, 0, 0});
    if (u == first[0]) cost0[0] = cost;
    sum[0] += cost;
  }
  int b = -1;
#pragma unroll 1
  for (int u = first[1]; u < behind[1]; ++u) {
    const int32_t w = u - np;
    if (b < 0 || s_unit[b + 1] <= w) {
      // a step of single tokens has one unit for each request
      const bool same = w < p.B && s_unit[w] == w && s_unit[w + 1] > w;
      b = same ? w : last_not_above(s_unit, p.B, w);
    }
    const int32_t c = p.cached[b], f = s_start[b + 1] - s_start[b], i0 = (w - s_unit[b]) * pair_tokens;
    const int32_t ntok = min(pair_tokens, f - i0), pos0 = c + i0, len = c + f;
    const bool small = shared && f <= Tt;
    const uint32_t last = uint32_t(pos0 + ntok - 1), G = uint32_t(p.block_tokens);
    const uint32_t seen = G == 1 ? last + 1 : (last / G + 1) * G;  // at most last + G
    const int32_t end = int32_t(min(uint32_t(len), seen));
    const int64_t cost = store_unit(p, u, {b, s_start[b] + i0, ntok, ((end + 127) >> 7) + (small ? 0 : ptiles),
                                           small ? -1 : ptiles, ntok <= Tt ? s_ctok[b] : -1, pos0, len});
    if (u == first[1]) cost0[1] = cost;
    sum[1] += cost;
  }
  block_scan<2, kThreads>(sum, all_costs, scratch);
  const int64_t carry = all_costs[0] + all_costs[1];
  sum[1] += all_costs[0];
#pragma unroll
  for (int kind = 0; kind < 2; ++kind) {
    int64_t at = sum[kind];
    for (int u = first[kind]; u < behind[kind]; ++u) {
      p.pre[u] = at;
      at += u == first[kind] ? cost0[kind] : unit_cost(p, p.units[u].ntok, p.units[u].ktiles);
    }
  }
  __shared__ int64_t s_share;
  __shared__ double s_rcp;
  if (tid == 0) {
    p.pre[units] = carry;
    wf_batch_hdr h{};
    h.fingerprint = p.fingerprint;
    h.tokens = tokens;
    h.units = units;
    h.prefix_units = np;
    h.prefix_len = prefix;
    h.ctoks = sum_ctok(total);
    h.head_cost = carry;
    // Equal shares, rounded up: a quotient in fp64, put right (64-bit divisions took 1 us of a small call).
    // No share is smaller than two single tiles: shorter ones cost more in merging than they save.
    const int64_t all = carry * p.kv_heads;
    int64_t share = int64_t(double(all) / p.max_ctas);
    while (share * p.max_ctas < all) ++share;
    h.share = max(share, int64_t(2) << WF_BATCH_SINGLE_SHIFT);
    h.share_rcp = 1.0 / double(h.share);
    int ctas = int(double(all) * h.share_rcp);
    while (ctas > 0 && (ctas - 1) * h.share >= all) --ctas;
    while (ctas * h.share < all) ++ctas;
    h.ctas = ctas;
    *p.hdr = h;
    s_share = h.share;
    s_rcp = h.share_rcp;
  }
  __syncthreads();
  // the unit that holds the beginning of each share, found from the units' side
  const int64_t share = s_share;
  const double rcp = s_rcp;
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    int64_t end = kind ? sum[1] : sum[0];
    for (int u = kind ? first[1] : first[0]; u < (kind ? behind[1] : behind[0]); ++u) {
      const int64_t at = end;
      end = p.pre[u + 1];
      for (int h = 0; h < p.kv_heads; ++h) {
        const int64_t s = h * carry + at, e = h * carry + end;
        int c = int(double(s) * rcp);  // first share that begins at or behind s: within one of the quotient
        while (c > 0 && (c - 1) * share >= s) --c;
        while (c * share < s) ++c;
        for (; c * share < e; ++c) p.starts[c] = {h, u};
      }
    }
  }
}

template <int kThreads>
wf_status launch_tables(const TablesParams& p, cudaStream_t stream) {
  const size_t smem = sizeof(int32_t) * (4 * size_t(p.B) + 2);
  if (smem > 40 * 1024) {
    static std::atomic<int> attr_done[64];  // (threads may find out the same at once)
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return WF_ERR_CUDA;
    if (dev < 0 || dev >= 64) return WF_ERR_UNSUPPORTED;
    if (!attr_done[dev]) {
      constexpr int kMost = int(sizeof(int32_t)) * (4 * 8192 + 2);
      static_assert(kMost <= 220 * 1024, "lengths in shared memory");
      if (cudaFuncSetAttribute(batch_tables_kernel<kThreads>, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost) !=
          cudaSuccess) {
        cudaGetLastError();
        return WF_ERR_CUDA;
      }
      attr_done[dev] = 1;
    }
  }
  const int token_blocks = (p.max_tokens + kThreads - 1) / kThreads;
  const int most = 147 * (1024 / kThreads);
  const int blocks = 1 + (token_blocks < most ? token_blocks : most);
  return wf::launch_early(batch_tables_kernel<kThreads>, blocks, kThreads, smem, stream, p);
}

// SM count of the current device, asked for once per device.
int sm_count() {
  static std::atomic<int> known[64];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) {
    cudaGetLastError();
    return 0;
  }
  if (known[dev] == 0) {
    int sms = 0;
    if (cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) {
      cudaGetLastError();
      return 0;
    }
    known[dev] = sms;
  }
  return known[dev];
}

}  // namespace

namespace wf {

bool on_current_device(const void* ptr) {
  int dev = 0;
  cudaPointerAttributes a;
  if (cudaGetDevice(&dev) != cudaSuccess || cudaPointerGetAttributes(&a, ptr) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  return (a.type == cudaMemoryTypeDevice || a.type == cudaMemoryTypeManaged) && a.device == dev;
}

BatchLayout batch_layout(const wf_batch_desc* d) {
  BatchLayout L{};
  L.error = WF_ERR_INVALID_ARG;
  if (!d) return L;
  const int64_t H = d->num_heads, K = d->num_kv_heads, P = d->page_tokens;
  if (H < 1 || K < 1 || H % K != 0 || d->pool_pages < 1 || d->max_requests < 1 || d->max_tokens < 1 ||
      d->max_request_pages < 1 || d->max_prefix_pages < 0 || d->block_tokens < 1 || d->num_ctas < 0 || d->head_dim < 1)
    return L;
  if (d->dtype != WF_BF16 && d->dtype != WF_F32) return L;
  if (P != 8 && P != 16 && P != 32 && P != 64 && P != 128) return L;
  L.error = WF_ERR_UNSUPPORTED;
  if (d->dtype != WF_BF16 || (d->head_dim != 64 && d->head_dim != 128) || H / K > 128) return L;
  L.error = WF_ERR_CAPACITY;
  // the work list's 64-bit cost arithmetic, int32 token and page indices
  const int64_t kMaxKeys = int64_t(1) << 27;
  if (K > 256 || H > 4096 || d->max_requests > 8192 || d->max_tokens > (1 << 22) || d->num_ctas > WF_BATCH_MAX_CTAS ||
      d->pool_pages * P > 0x7FFFFFFF || int64_t(d->max_requests) * d->max_request_pages > 0x7FFFFFFF ||
      d->max_request_pages * P > kMaxKeys || d->max_prefix_pages * P > kMaxKeys)
    return L;
  L.ctas = d->num_ctas;
  if (L.ctas == 0) {
    const int sms = sm_count();
    if (sms < 1) {
      L.error = WF_ERR_CUDA;
      return L;
    }
    L.ctas = sms < WF_BATCH_MAX_CTAS ? sms : WF_BATCH_MAX_CTAS;
  }
  L.group = int32_t(H / K);
  L.tile_tokens = 128 / L.group;
  const int64_t pair = 2 * L.tile_tokens;
  // own units: each request's tokens in pairs of tiles; prefix units: all tokens in pairs of tiles
  L.max_units = int32_t(d->max_requests + d->max_tokens / pair + (d->max_tokens + pair - 1) / pair + 1);
  const int64_t ctok = int64_t(d->max_requests) * L.tile_tokens;
  L.max_ctok = ctok < d->max_tokens ? ctok : d->max_tokens;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  L.off_starts = sizeof(wf_batch_hdr);
  L.off_units = up(WF_BATCH_PLAN_HEAD);
  L.off_pre = up(L.off_units + size_t(L.max_units) * sizeof(wf_batch_unit));
  L.off_ctok = up(L.off_pre + size_t(L.max_units + 1) * sizeof(int64_t));
  L.off_ctok_list = up(L.off_ctok + size_t(d->max_tokens) * sizeof(int32_t));
  L.plan_bytes = up(L.off_ctok_list + size_t(L.max_ctok) * sizeof(wf_batch_ctok));
  // partial rows: [prefix, own][key parity][ctok][H], then [ctas][head, tail][tile or key parity][128]
  L.main_rows = 4 * L.max_ctok * H;
  const size_t rows = size_t(L.main_rows) + size_t(L.ctas) * 4 * 128;
  L.off_lse = up(WF_ATTN_STATUS_BYTES + rows * size_t(d->head_dim) * sizeof(float));
  L.off_cuts = up(L.off_lse + rows * sizeof(float));
  L.workspace_bytes = up(L.off_cuts + size_t(L.ctas) * WF_BATCH_CUT_BYTES);
  uint64_t f = 0xcbf29ce484222325ull;  // FNV-1a over the description's words
  const int32_t words[] = {d->num_heads, d->num_kv_heads, d->head_dim, d->dtype, d->page_tokens, d->pool_pages,
                           d->max_requests, d->max_tokens, d->max_request_pages, d->max_prefix_pages,
                           d->block_tokens, L.ctas};
  for (int32_t w : words)
    for (int k = 0; k < 4; ++k) f = (f ^ uint64_t((uint32_t(w) >> (8 * k)) & 255)) * 0x100000001b3ull;
  L.fingerprint = f | 1;  // never the zero of a plan that was not built
  L.error = WF_OK;
  return L;
}

}  // namespace wf

extern "C" size_t wf_batch_plan_bytes(const wf_batch_desc* desc) {
  const wf::BatchLayout L = wf::batch_layout(desc);
  return L.error == WF_OK ? L.plan_bytes : 0;
}

extern "C" size_t wf_batch_workspace_bytes(const wf_batch_desc* desc) {
  const wf::BatchLayout L = wf::batch_layout(desc);
  return L.error == WF_OK ? L.workspace_bytes : 0;
}

extern "C" wf_status wf_batch_tables(const wf_batch_desc* desc, const int32_t* cached, const int32_t* fresh,
                                     const int32_t* prefix_len, const int32_t* held, const int32_t* free_pages,
                                     int32_t num_free, const int32_t* free_head, int32_t* free_head_out,
                                     int32_t* held_out, int32_t* block_table, int32_t* token_start, int32_t* slot_map,
                                     int32_t* positions, void* plan, size_t plan_bytes, wf_stream_t stream) {
  const wf::BatchLayout L = wf::batch_layout(desc);
  if (L.error != WF_OK) return L.error;
  if (!cached || !fresh || (!free_pages && num_free > 0) || !free_head || !free_head_out || !block_table ||
      !token_start || !slot_map || !positions || !plan || num_free < 0)
    return WF_ERR_INVALID_ARG;
  if (desc->max_prefix_pages > 0 && !prefix_len) return WF_ERR_INVALID_ARG;
  if ((held == nullptr) != (held_out == nullptr)) return WF_ERR_INVALID_ARG;
  // every block reads the lengths while block 0 writes: no output may lie in an input
  constexpr size_t kWord = sizeof(int32_t);
  const size_t B = size_t(desc->max_requests), T = size_t(desc->max_tokens);
  const wf::Span in[] = {{cached, B * kWord}, {fresh, B * kWord}, {prefix_len, kWord}, {held, B * kWord},
                         {free_pages, size_t(num_free) * kWord}, {free_head, kWord}};
  const wf::Span out[] = {{free_head_out, kWord}, {held_out, B * kWord},
                          {block_table, B * size_t(desc->max_request_pages) * kWord}, {token_start, (B + 1) * kWord},
                          {slot_map, T * kWord}, {positions, T * kWord}, {plan, L.plan_bytes}};
  if (wf::written_over(out, in)) return WF_ERR_INVALID_ARG;
  for (const wf::Span& x : in)
    if (reinterpret_cast<uintptr_t>(x.ptr) % kWord) return WF_ERR_ALIGNMENT;
  for (const wf::Span& x : out)
    if (reinterpret_cast<uintptr_t>(x.ptr) % kWord) return WF_ERR_ALIGNMENT;
  if (reinterpret_cast<uintptr_t>(plan) % 16) return WF_ERR_ALIGNMENT;
  if (plan_bytes < L.plan_bytes) return WF_ERR_WORKSPACE;
  if (!wf::on_current_device(plan)) return WF_ERR_INVALID_ARG;

  TablesParams p{};
  p.cached = cached;
  p.fresh = fresh;
  p.prefix_len = desc->max_prefix_pages > 0 ? prefix_len : nullptr;
  p.held = held;
  p.free_pages = free_pages;
  p.free_head = free_head;
  p.free_head_out = free_head_out;
  p.held_out = held_out;
  p.table = block_table;
  p.token_start = token_start;
  p.slot_map = slot_map;
  p.positions = positions;
  uint8_t* pl = static_cast<uint8_t*>(plan);
  p.hdr = reinterpret_cast<wf_batch_hdr*>(pl);
  p.starts = reinterpret_cast<wf_batch_start*>(pl + L.off_starts);
  p.units = reinterpret_cast<wf_batch_unit*>(pl + L.off_units);
  p.pre = reinterpret_cast<int64_t*>(pl + L.off_pre);
  p.ctok = reinterpret_cast<int32_t*>(pl + L.off_ctok);
  p.ctok_list = reinterpret_cast<wf_batch_ctok*>(pl + L.off_ctok_list);
  p.B = desc->max_requests;
  p.max_tokens = desc->max_tokens;
  p.cols = desc->max_request_pages;
  p.max_prefix = desc->max_prefix_pages * desc->page_tokens;
  p.num_free = num_free;
  p.pool_pages = desc->pool_pages;
  p.page = desc->page_tokens;
  while ((1 << p.page_shift) < p.page) ++p.page_shift;
  p.tile_tokens = L.tile_tokens;
  p.block_tokens = desc->block_tokens;
  p.kv_heads = desc->num_kv_heads;
  p.max_ctas = L.ctas;
  p.fingerprint = L.fingerprint;

  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  // Blocks of 256 or 1024 threads.  A small block starts and scans sooner, a
  // large one has a thread for every request (a call in a graph): 5 requests 4.5
  // us with 256 and 5.5 us with 1024, 256 requests 5.1 and 6.2 us, 512 6.5 and
  // 6.8 us, 1024 9.8 and 8.0 us, 8192 115 and 51 us.
  return p.B <= 512 ? launch_tables<256>(p, st) : launch_tables<1024>(p, st);
}

extern "C" wf_status wf_batch_status(const void* plan, wf_stream_t stream, int32_t* detail) {
  return wf_attn_workspace_status(plan, stream, detail);  // the plan begins with the same status block
}
