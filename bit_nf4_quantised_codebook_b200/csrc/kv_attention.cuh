// kv_attention.cuh — what the two attention kernels over the 4-bit cache share: their
// arguments, the table lookup that turns two codes into two fp16 levels, and the kernel
// that joins the parts of an item (one sequence, key/value head and tile of query rows)
// that several workers shared.
#pragma once
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include "internal.h"
#include "kv_common.cuh"
#include "launch.cuh"

namespace qlora {

constexpr float kLift = 6.0f;          // a new largest contribution to a block gets the fp16 weight 2^kLift
constexpr float kMostWeight = 16384.0f;  // a weight past this renews the scales
constexpr float kMostSum = 0x1p100f;   // and so does a sum past this
constexpr float kFloor = -3.0e38f;     // "no maximum yet": finite, so that differences stay defined

struct KvAttnArgs {
  KvBatch kb;
  const uint16_t *Q;
  int64_t q_token_stride, q_head_stride;
  uint16_t *out;
  const uint8_t *k_codes, *v_codes;
  const uint16_t *k_absmax, *v_absmax;
  int heads, group;   // key/value heads; query heads of each
  float scale_log2;   // scale * log2(e) / unit
  float v_unit;       // 1 / unit: levels are stored times `unit`
  int causal, window;
  int few_rows;       // sequences with more rows (tokens x group) than this go to the many-row kernel
  int32_t *again;     // [batch] those that it leaves to the few-row kernel all the same (with few_rows only)
  __half levels[16];
  // workspace
  float *part_o;      // [workers][2][rows of a tile][D] normalised partial outputs
  float *part_lse;    // [workers][2][rows of a tile] log2 of their weights' sum
  struct KvPart *parts;  // [workers][2]
};

// A worker's part of an item that it shares with others (slot 0: the item its range
// starts in; slot 1: the one it ends in).
struct alignas(16) KvPart {
  int present;
  int joins;      // 1: the second part of its item, whose CTA joins them all
  int g0, last;   // the item's first and last worker
  int head_slot;  // slot of the first worker's part
  int row0;       // first token row of the sequence
  int head, tile;
  int rows;       // of the tile
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float lg2(float x) {
  float y;
  asm("lg2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}
// Table entry of byte I of w (lane address `tab`: table base | lane * 4).
template <int I>
__device__ __forceinline__ uint32_t lookup(uint32_t w, uint32_t tab) {
  return lds32(prmt(w, tab, 0x7604u | (I << 4)));
}
__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
// 16 bytes from global to shared memory, past the first-level cache.
__device__ __forceinline__ void copy16(uint32_t dst, const void *src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copies_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>  // all but the last N groups of this thread's copies have landed
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
// Joins the items that several workers shared.  CTA (k, y): 8 / SPLIT rows, SPLIT warps to each, of
// the item that the range of worker k starts inside of, when worker k holds the item's second
// part.  The first parts are loaded together with all the weights.
constexpr int kMaxWorkers = 1024;
template <int D, int ROWS, int SPLIT>
__global__ void __launch_bounds__(256) k_kv_join(const __grid_constant__ KvAttnArgs a) {
  constexpr int V = D / 32;  // channels per lane
  constexpr int U = SPLIT > 1 || ROWS < 128 ? 4 : 2;  // parts loaded at once (those of the long items of prompts are two or three)
  __shared__ float s_acc[SPLIT > 1 ? 8 * D : 1];
  pdl_wait();
  pdl_launch_dependents();
  const int k = static_cast<int>(blockIdx.x) + 1;
  const KvPart p = a.parts[k * 2];
  if (!p.joins) return;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = warp % SPLIT;
  const int r = static_cast<int>(blockIdx.y) * (8 / SPLIT) + warp / SPLIT;
  const bool live = r < p.rows;
  if (SPLIT == 1 && !live) return;
  const int n = live ? p.last - p.g0 + 1 : 0;
  auto part_of = [&](int i) { return static_cast<int64_t>(p.g0 + i) * 2 + (i == 0 ? p.head_slot : 0); };
  auto lse_of = [&](int i) {
    const int64_t part = part_of(i);
    return a.parts[part].present ? a.part_lse[part * ROWS + r] : -INFINITY;  // workers without steps
  };
  // this warp's parts: share, share + SPLIT, ...
  const int mine = (n - share + SPLIT - 1) / SPLIT;
  float2 v[U][V / 2];
  auto load = [&](int j0) {
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const int i = share + min(j0 + j, mine - 1) * SPLIT;
      const float *src = a.part_o + (part_of(i) * ROWS + r) * D + lane * V;
#pragma unroll
      for (int x = 0; x < V / 2; ++x) v[j][x] = *reinterpret_cast<const float2 *>(src + 2 * x);
    }
  };
  if (mine > 0) load(0);
  float top = -INFINITY;
  for (int i = lane; i < n; i += 32) top = fmaxf(top, lse_of(i));
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
  float sum = 0.0f, acc[V] = {};
  for (int i = lane; i < n; i += 32) {
    const float lse = lse_of(i);
    sum += lse == -INFINITY ? 0.0f : ex2(lse - top);
  }
  float weight = 0.0f;
  for (int j0 = 0; j0 < mine; j0 += U) {
    if ((j0 & 31) == 0 && j0 + lane < mine) {  // (what lanes past the last part hold is not used)
      const float lse = lse_of(share + (j0 + lane) * SPLIT);
      weight = lse == -INFINITY ? 0.0f : ex2(lse - top);
    }
#pragma unroll
    for (int j = 0; j < U; ++j) {
      const float f = __shfl_sync(0xFFFFFFFFu, weight, (j0 + j) & 31);
      if (j0 + j < mine && f != 0.0f) {  // an absent part holds anything
#pragma unroll
        for (int x = 0; x < V / 2; ++x) {
          acc[2 * x] = fmaf(f, v[j][x].x, acc[2 * x]);
          acc[2 * x + 1] = fmaf(f, v[j][x].y, acc[2 * x + 1]);
        }
      }
    }
    if (j0 + U < mine) load(j0 + U);
  }
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
  if (SPLIT > 1) {  // the row's warps, in order
#pragma unroll
    for (int x = 0; x < V; ++x) s_acc[warp * D + lane * V + x] = acc[x];
    __syncthreads();
    if (share != 0 || !live) return;
#pragma unroll
    for (int w = 1; w < SPLIT; ++w)
#pragma unroll
      for (int x = 0; x < V; ++x) acc[x] += s_acc[(warp + w) * D + lane * V + x];
  }
  const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
  const int rr = p.tile * ROWS + r, i = rr / a.group, h = rr - i * a.group;
  uint16_t *dst = a.out + ((static_cast<int64_t>(p.row0 + i) * a.heads + p.head) * a.group + h) * D + lane * V;
#pragma unroll
  for (int x = 0; x < V / 2; ++x)
    *reinterpret_cast<uint32_t *>(dst + 2 * x) = pack_bf16x2(acc[2 * x] * inv, acc[2 * x + 1] * inv);
}

// kv_prefill.cu
size_t kv_prefill_workspace(int head_dim, int group, int batch, int64_t tokens, int num_sms);
cudaError_t launch_kv_prefill(const KvAttnArgs &a, int head_dim, void *ws, int num_sms, unsigned long long timeout_ns,
                              cudaStream_t st);

}  // namespace qlora
