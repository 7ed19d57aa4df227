// wf_batch_append: writes the new tokens' K and V rows into the paged pool at
// their slots, and, given a table of angles, rotates Q and K on the way:
//   x' = x c - y s,  y' = x s + y c   for every interleaved pair (x, y) of a
// row, with (c, s) the token's fp32 table entry of that pair; in fp32, rounded
// once to bf16.
//
// HBM-bound: each row is read once and written once.  A thread owns one
// 16-byte column of a token's rows (Q heads, K heads, V heads), so that it
// loads that column's four (cos, sin) pairs once, and four of the rows, whose
// loads are all in flight before the first is used.  The block is as many
// threads as one token's rows or a few tokens' need, none idle: bytes in
// flight are what the speed depends on (2.25 loads a thread in fixed blocks of
// 256 reached 5.75 TB/s on 37440 tokens of 12 + 24 rows of 128, and 3.0 TB/s on
// 16 + 2 rows of 64, where 14 of 32 row slots idled; now 5.9 TB/s, 121 us, on
// the former with other inputs every time, 6.3 TB/s, 112 us, on the same ones
// again).  Neighbouring threads cover whole rows: coalesced.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cstdint>

#include "wf_batch.h"

namespace {

constexpr int kMaxThreads = 384;
constexpr int kInFlight = 4;

struct AppendParams {
  const wf_batch_hdr* hdr;
  const int32_t* slot_map;
  const float4* rope;  // [tokens][D / 4]: two (cos, sin) pairs each; nullptr: K as given, Q not touched
  const uint4* q;
  const uint4* k;
  const uint4* v;
  uint4* q_rot;
  uint4* k_pool;
  uint4* v_pool;
  uint64_t fingerprint;
  int64_t pool_tokens;
  int32_t H, kv_heads;
  int32_t slots;  // threads of a token in one column: rows are slots apart
};

__device__ __forceinline__ uint32_t rotate_bf16x2(uint32_t xy, float c, float s) {
  const float x = __uint_as_float(xy << 16), y = __uint_as_float(xy & 0xffff0000u);
  const __nv_bfloat162 r = __floats2bfloat162_rn(x * c - y * s, x * s + y * c);
  return *reinterpret_cast<const uint32_t*>(&r);
}

// kVec: 16-byte columns of a row (D / 8).
template <int kVec, bool kRope>
__global__ void __launch_bounds__(kMaxThreads, 3) batch_append_kernel(const AppendParams p) {
  cudaGridDependencySynchronize();
  if (p.hdr->fingerprint != p.fingerprint) return;
  const int tokens = p.hdr->tokens;
  const int col = threadIdx.x % kVec, line = threadIdx.x / kVec;
  const int sub = line / p.slots, first = line - sub * p.slots;  // token of the block, first row
  const int per_block = blockDim.x / (kVec * p.slots);
  const int nq = kRope ? p.H : 0, rows = nq + 2 * p.kv_heads;
  for (int64_t t = int64_t(blockIdx.x) * per_block + sub; t < tokens; t += int64_t(gridDim.x) * per_block) {
    const int64_t slot = p.slot_map[t];
    const bool in_pool = slot >= 0 && slot < p.pool_tokens;
    float4 cs0, cs1;
    if (kRope) {
      const float4* r = p.rope + (t * kVec + col) * 2;
      cs0 = r[0];
      cs1 = r[1];
    }
    for (int r0 = first; r0 < rows; r0 += p.slots * kInFlight) {
      uint4 x[kInFlight];
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * p.slots;
        if (r < rows) {
          const uint4* src = r < nq                ? p.q + (t * p.H + r) * kVec
                             : r < nq + p.kv_heads ? p.k + (t * p.kv_heads + (r - nq)) * kVec
                                                   : p.v + (t * p.kv_heads + (r - nq - p.kv_heads)) * kVec;
          x[i] = __ldcs(src + col);
        }
      }
#pragma unroll
      for (int i = 0; i < kInFlight; ++i) {
        const int r = r0 + i * p.slots;
        if (r >= rows) continue;
        if (kRope && r < nq + p.kv_heads) {
          x[i].x = rotate_bf16x2(x[i].x, cs0.x, cs0.y);
          x[i].y = rotate_bf16x2(x[i].y, cs0.z, cs0.w);
          x[i].z = rotate_bf16x2(x[i].z, cs1.x, cs1.y);
          x[i].w = rotate_bf16x2(x[i].w, cs1.z, cs1.w);
        }
        if (r < nq) {
          __stcs(p.q_rot + (t * p.H + r) * kVec + col, x[i]);
        } else if (in_pool) {
          const bool is_k = r < nq + p.kv_heads;
          const int h = r - nq - (is_k ? 0 : p.kv_heads);
          __stcs((is_k ? p.k_pool : p.v_pool) + (slot * p.kv_heads + h) * kVec + col, x[i]);
        }
      }
    }
  }
}

bool misaligned(const void* ptr) { return reinterpret_cast<uintptr_t>(ptr) % 16 != 0; }

}  // namespace

extern "C" wf_status wf_batch_append(const wf_batch_desc* desc, const void* plan, const int32_t* slot_map,
                                     const float* rope, const void* q, const void* k, const void* v, void* q_rot,
                                     void* k_pool, void* v_pool, wf_stream_t stream) {
  const wf::BatchLayout L = wf::batch_layout(desc);
  if (L.error != WF_OK) return L.error;
  if (!plan || !slot_map || !k || !v || !k_pool || !v_pool) return WF_ERR_INVALID_ARG;
  // Q only turns: without angles there is nothing to do
  if (rope ? (!q || !q_rot) : (q || q_rot)) return WF_ERR_INVALID_ARG;
  // nothing that other threads still read is written over (a Q row is turned by the threads that read it)
  constexpr size_t kBf16 = 2;
  const size_t T = size_t(desc->max_tokens), D = size_t(desc->head_dim);
  const size_t q_bytes = T * size_t(desc->num_heads) * D * kBf16, kv_bytes = T * size_t(desc->num_kv_heads) * D * kBf16;
  const size_t pool_bytes = size_t(desc->pool_pages) * size_t(desc->page_tokens) * size_t(desc->num_kv_heads) * D * kBf16;
  const wf::Span in[] = {{k, kv_bytes}, {v, kv_bytes}, {rope, T * D * sizeof(float)}, {slot_map, T * sizeof(int32_t)},
                         {plan, L.plan_bytes}, {q != q_rot ? q : nullptr, q_bytes}};
  const wf::Span out[] = {{q_rot, q_bytes}, {k_pool, pool_bytes}, {v_pool, pool_bytes}};
  if (wf::written_over(out, in)) return WF_ERR_INVALID_ARG;
  if (misaligned(plan) || misaligned(rope) || misaligned(q) || misaligned(k) || misaligned(v) || misaligned(q_rot) ||
      misaligned(k_pool) || misaligned(v_pool) || reinterpret_cast<uintptr_t>(slot_map) % 4)
    return WF_ERR_ALIGNMENT;
  if (!wf::on_current_device(plan)) return WF_ERR_INVALID_ARG;
  AppendParams p{};
  p.hdr = static_cast<const wf_batch_hdr*>(plan);
  p.slot_map = slot_map;
  p.rope = reinterpret_cast<const float4*>(rope);
  p.q = static_cast<const uint4*>(q);
  p.k = static_cast<const uint4*>(k);
  p.v = static_cast<const uint4*>(v);
  p.q_rot = static_cast<uint4*>(q_rot);
  p.k_pool = static_cast<uint4*>(k_pool);
  p.v_pool = static_cast<uint4*>(v_pool);
  p.fingerprint = L.fingerprint;
  p.pool_tokens = int64_t(desc->pool_pages) * desc->page_tokens;
  p.H = desc->num_heads;
  p.kv_heads = desc->num_kv_heads;
  const int vec = desc->head_dim / 8;
  const int rows = (rope ? desc->num_heads : 0) + 2 * desc->num_kv_heads;
  p.slots = std::min((rows + kInFlight - 1) / kInFlight, kMaxThreads / vec);
  const int per_block = std::max(1, 128 / (vec * p.slots));
  const int threads = vec * p.slots * per_block;
  const unsigned blocks = unsigned(std::min((desc->max_tokens + per_block - 1) / per_block, L.ctas * 32));
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  void (*kernel)(AppendParams);
  if (desc->head_dim == 128)
    kernel = rope ? batch_append_kernel<16, true> : batch_append_kernel<16, false>;
  else
    kernel = rope ? batch_append_kernel<8, true> : batch_append_kernel<8, false>;
  return wf::launch_early(kernel, blocks, unsigned(threads), 0, s, p);
}
