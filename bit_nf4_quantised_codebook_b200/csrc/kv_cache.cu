// kv_cache.cu — writing keys and values into the 4-bit paged cache and reading
// them back: the block quantisation of "QLoRA: Efficient Finetuning of Quantized
// LLMs" (intuitivepapers.ai, §Quantize in blocks, §NormalFloat) with blocks of 64
// channels and the block's absmax kept, in bfloat16, where it is exact.
//
// Both kernels stream: a token's key and value of every head are a row of 8-channel
// units (16 bytes of bfloat16, 4 bytes of codes); a CTA takes up to 1024 units - whole
// token rows, or a piece of one - finds the cache slot of each of its token rows once
// (binary search over token_start, then the page table), and each thread then moves
// four units, their loads issued together.
// Bound by HBM for prompts (2 + 17/32 bytes per element each way) and by the chain of
// dependent loads token_start -> kv_len -> page_table -> data for single tokens.
//
// Code of one element.  The code is #{i : float32(x / c) >= t_i}.  x and c are
// bfloat16, so x / c is one of the ratios a / b * 2^-k of integers a < 256, b < 256,
// and between two ratios that the definition codes differently there is a gap of at
// least 2^-19 of their size around each threshold (checked over all of them when the
// table is built, and by a test that runs every ratio).  x * rcp(c), within 2^-22, is
// therefore compared with a float32 placed inside that gap, and no exact quotient is
// needed.  The gap also leaves the threshold's four lowest mantissa bits free: they
// carry the code below it, so that one 32-bit word per bucket of x / c holds both, the
// 32 words of the table lie in 32 different banks, and a lookup never conflicts.
#include <cmath>
#include <cstdint>
#include <cstring>
#include <cuda_runtime.h>
#include "internal.h"
#include "kv_common.cuh"
#include "launch.cuh"
#include "nf4_decode.cuh"

namespace qlora {
namespace {

constexpr int kKvThreads = 256;
constexpr int kKvUnitsPerThread = 4;
constexpr int kKvSpan = kKvThreads * kKvUnitsPerThread;  // units of one CTA
constexpr int kKvMaxTokens = kKvSpan / 8;                // token rows of one CTA (>= 8 units each)

struct KvCodeTable {
  uint32_t e[32];
};

struct KvRows {
  const uint16_t *src[2];  // append: K, V (strided)
  int64_t token_stride[2], head_stride[2];
  uint16_t *dst[2];        // read: K_out, V_out (contiguous; nullable)
  uint8_t *codes[2];
  uint16_t *absmax[2];
  int heads;
  int head_shift;       // a head is 1 << head_shift units
  int per_side;         // units of a token's keys: heads << head_shift
  int per_token;        // per_side, times 2 unless one output is not wanted
  int tokens_per_cta;   // whole token rows of a CTA; 1 when a row is split over blockIdx.y
  uint32_t magic;       // ceil(2^32 / per_token): w / per_token = umulhi(w, magic) for w * per_token < 2^32
};

// Unit v of this CTA: its token row (counted from the CTA's first), side, head and
// place in the head.  False when there is no such unit.
struct KvUnit {
  int t, side, head, sub;
};
__device__ __forceinline__ bool kv_unit(const KvRows &r, int v, int rows, KvUnit &u) {
  const int w = static_cast<int>(blockIdx.y) * kKvSpan + v;
  u.t = static_cast<int>(__umulhi(static_cast<uint32_t>(w), r.magic));
  const int x = w - u.t * r.per_token;
  u.side = x >= r.per_side ? 1 : 0;
  const int y = x - u.side * r.per_side;
  u.head = y >> r.head_shift;
  u.sub = y - (u.head << r.head_shift);
  return u.t < rows;
}

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Slot index page * page_size + slot (a 64-bit value) of token row t, or -1 when no
// sequence owns the row or its position or page is out of range.
__device__ __forceinline__ int64_t row_slot(const KvBatch &kb, int t) {
  int lo = 0, hi = kb.batch;  // last b in [0, batch) with token_start[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(kb.token_start + mid) <= t) lo = mid;
    else hi = mid;
  }
  const KvSeq q = kv_seq(kb, lo);
  const int i = t - q.row0;
  if (i < 0 || i >= q.n) return -1;
  const int p = q.pos0() + i;
  const int page = p < 0 ? -1 : kv_page(kb, lo, p);
  if (page < 0) {
    kv_error(kb);
    return -1;
  }
  return (static_cast<int64_t>(page) << kb.page_shift) | (p & ((1 << kb.page_shift) - 1));
}

// The slots of this CTA's token rows, into shared memory; returns how many rows.
__device__ __forceinline__ int load_slots(const KvBatch &kb, int t0, int per_cta, int64_t *slots) {
  const int rows = min(per_cta, kb.tokens - t0);
  for (int i = threadIdx.x; i < rows; i += kKvThreads) slots[i] = row_slot(kb, t0 + i);
  __syncthreads();
  return rows;
}

// Flat index of a slot and head in the cache's [page][head][slot] order.
__device__ __forceinline__ int64_t cache_row(const KvBatch &kb, int64_t slot, int head, int heads) {
  const int64_t page = slot >> kb.page_shift;
  const int in_page = static_cast<int>(slot) & ((1 << kb.page_shift) - 1);
  return ((page * heads + head) << kb.page_shift) + in_page;
}

// LOG: buckets by sign and exponent (E3M0, one threshold per binade); otherwise 31
// equal buckets over [-1, 1].  SKIP8: the code book holds zero twice (codes 7 and 8)
// and uses 7.
template <bool LOG, bool SKIP8>
__device__ __forceinline__ uint32_t kv_code(float x, const uint32_t *tab) {
  uint32_t b;
  if (LOG) {
    const uint32_t bits = __float_as_uint(x);
    const int e = min(max(static_cast<int>((bits >> 23) & 255u) - 119, 0), 8);
    b = static_cast<uint32_t>(e) | ((bits >> 27) & 16u);
  } else {
    // 2^23 + 16 + 15 x, rounded to nearest: the bucket (1 .. 31) in the low mantissa bits
    b = __float_as_uint(__fmaf_rn(x, 15.0f, 8388608.0f + 16.0f)) & 31u;
  }
  const uint32_t e = tab[b];
  const uint32_t c = (e & 15u) + (x >= __uint_as_float(e) ? 1u : 0u);
  return SKIP8 && c == 8u ? 9u : c;
}

template <bool LOG, bool SKIP8>
__global__ void __launch_bounds__(kKvThreads) k_kv_append(const __grid_constant__ KvBatch kb,
                                                           const __grid_constant__ KvRows r,
                                                           const __grid_constant__ KvCodeTable table) {
  __shared__ uint32_t s_tab[32];
  __shared__ int64_t s_slot[kKvMaxTokens];
  if (threadIdx.x < 32) s_tab[threadIdx.x] = table.e[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * r.tokens_per_cta;
  const int rows = load_slots(kb, t0, r.tokens_per_cta, s_slot);

  uint4 raw[kKvUnitsPerThread];
  int64_t row[kKvUnitsPerThread];
  int side[kKvUnitsPerThread], sub[kKvUnitsPerThread];
#pragma unroll
  for (int k = 0; k < kKvUnitsPerThread; ++k) {
    KvUnit u;
    row[k] = -1;
    raw[k] = make_uint4(0, 0, 0, 0);
    if (kv_unit(r, k * kKvThreads + threadIdx.x, rows, u) && s_slot[u.t] >= 0) {
      row[k] = cache_row(kb, s_slot[u.t], u.head, r.heads);
      raw[k] = ld_stream(r.src[u.side] + static_cast<int64_t>(t0 + u.t) * r.token_stride[u.side] +
                         static_cast<int64_t>(u.head) * r.head_stride[u.side] + u.sub * 8);
    }
    side[k] = u.side;
    sub[k] = u.sub;
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < kKvUnitsPerThread; ++k) {
    const uint32_t wd[4] = {raw[k].x, raw[k].y, raw[k].z, raw[k].w};
    // largest magnitude of the 8 elements, as bfloat16 bits: those of non-negative
    // values order like integers, infinities and NaN above every finite one
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) m = __vmaxu2(m, wd[i] & 0x7FFF7FFFu);
    m = max(m >> 16, m & 0xFFFFu);
    // the 8 threads of a block are consecutive lanes (units come in whole heads)
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
    m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
    const bool finite = m < 0x7F80u;
    float c = __uint_as_float(m << 16), scale = 1.0f;
    // very small and very large blocks are scaled by 2^96 or 2^-96, exactly, so that the
    // reciprocal is a normal number
    if (m < (31u << 7)) scale = 0x1p96f;
    if (m >= (223u << 7)) scale = 0x1p-96f;
    c *= scale;
    const float rc = c > 0.0f && finite ? __frcp_rn(c) : 0.0f;  // zero and non-finite blocks: every ratio 0
    uint32_t packed = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float lo = __uint_as_float(wd[i] << 16), hi = __uint_as_float(wd[i] & 0xFFFF0000u);
      lo = finite ? __fmul_rn(__fmul_rn(lo, scale), rc) : 0.0f;
      hi = finite ? __fmul_rn(__fmul_rn(hi, scale), rc) : 0.0f;
      packed |= ((kv_code<LOG, SKIP8>(lo, s_tab) << 4) | kv_code<LOG, SKIP8>(hi, s_tab)) << (8 * i);
    }
    if (row[k] >= 0) {
      const int s = side[k];
      reinterpret_cast<uint32_t *>(r.codes[s])[(row[k] << r.head_shift) + sub[k]] = packed;
      if ((sub[k] & 7) == 0)
        r.absmax[s][(row[k] << (r.head_shift - 3)) + (sub[k] >> 3)] = static_cast<uint16_t>(finite ? m : 0x7FC0u);
      bad |= !finite;
    }
  }
  if (bad && kb.dev_err) atomicOr(kb.dev_err, QLORA_DEVERR_NONFINITE);
}

__global__ void __launch_bounds__(kKvThreads) k_kv_read(const __grid_constant__ KvBatch kb,
                                                         const __grid_constant__ KvRows r,
                                                         const __grid_constant__ Nf4Levels lv) {
  __shared__ float s_level[16];  // 16 words in 16 banks: a lookup never conflicts
  __shared__ int64_t s_slot[kKvMaxTokens];
  if (threadIdx.x < 16) s_level[threadIdx.x] = lv.q[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * r.tokens_per_cta;
  const int rows = load_slots(kb, t0, r.tokens_per_cta, s_slot);

  uint32_t codes[kKvUnitsPerThread], amax[kKvUnitsPerThread];
  uint16_t *dst[kKvUnitsPerThread];
#pragma unroll
  for (int k = 0; k < kKvUnitsPerThread; ++k) {
    KvUnit u;
    dst[k] = nullptr;
    codes[k] = amax[k] = 0;
    if (kv_unit(r, k * kKvThreads + threadIdx.x, rows, u) && s_slot[u.t] >= 0) {
      const int64_t row = cache_row(kb, s_slot[u.t], u.head, r.heads);
      codes[k] = __ldg(reinterpret_cast<const uint32_t *>(r.codes[u.side]) + (row << r.head_shift) + u.sub);
      amax[k] = __ldg(r.absmax[u.side] + (row << (r.head_shift - 3)) + (u.sub >> 3));
      dst[k] = r.dst[u.side] + (((static_cast<int64_t>(t0 + u.t) * r.heads + u.head) << r.head_shift) + u.sub) * 8;
    }
  }
#pragma unroll
  for (int k = 0; k < kKvUnitsPerThread; ++k) {
    const float c = __uint_as_float(amax[k] << 16);
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      o[i] = pack_bf16x2(__fmul_rn(s_level[(codes[k] >> (8 * i + 4)) & 15u], c),
                         __fmul_rn(s_level[(codes[k] >> (8 * i)) & 15u], c));
    if (dst[k]) *reinterpret_cast<uint4 *>(dst[k]) = make_uint4(o[0], o[1], o[2], o[3]);
  }
}

KvRows cache_rows(const qlora_kv_cache &c, int sides) {
  KvRows r = {};
  r.codes[0] = c.k_codes;
  r.codes[1] = c.v_codes;
  r.absmax[0] = c.k_absmax;
  r.absmax[1] = c.v_absmax;
  r.heads = c.heads;
  r.head_shift = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
  r.per_side = c.heads << r.head_shift;
  r.per_token = sides * r.per_side;
  r.tokens_per_cta = r.per_token < kKvSpan ? kKvSpan / r.per_token : 1;
  r.magic = static_cast<uint32_t>(((1ull << 32) + r.per_token - 1) / r.per_token);
  return r;
}

dim3 rows_grid(const KvRows &r, int64_t tokens) {
  return dim3(static_cast<unsigned>((tokens + r.tokens_per_cta - 1) / r.tokens_per_cta),
              static_cast<unsigned>((r.per_token + kKvSpan - 1) / kKvSpan));
}

}  // namespace

KvBatch kv_device_batch(const qlora_kv_cache &c, const qlora_kv_batch &b, int *dev_err) {
  KvBatch k;
  k.token_start = b.token_start;
  k.kv_len = b.kv_len;
  k.page_table = b.page_table;
  k.batch = b.batch;
  k.max_pages = b.max_pages;
  k.num_pages = static_cast<int>(c.num_pages);
  k.page_shift = 0;
  while ((1 << k.page_shift) < c.page_size) ++k.page_shift;
  k.tokens = static_cast<int>(b.tokens);
  k.dev_err = dev_err;
  return k;
}

// The 32 words of the code lookup.  Around each threshold lie the largest ratio that
// the definition codes below it and the smallest that it codes above; a float32 between
// the two, at least 2^-22 of its size from either (the error of x * rcp(c) is smaller),
// with the code below it in its four lowest bits, goes into the bucket it falls in.
bool build_kv_code_table(int codebook, uint32_t table[32]) {
  float levels[16], thr[15];
  if (!build_format_codebook_f32(codebook, levels, thr)) return false;
  const bool log_buckets = codebook == QLORA_CB_FP4_E3M0;
  float bound[15];
  for (int i = 0; i < 15; ++i) {
    bound[i] = 2.0f;  // a threshold above every ratio (Int4's lowest level is never met: its threshold lies below)
    if (i > 0 && thr[i] == thr[i - 1]) {
      bound[i] = bound[i - 1];
      continue;
    }
    double below = -2.0, above = 2.0;
    for (int sign = -1; sign <= 1; sign += 2)
      for (int k = 0; k <= 20; ++k)
        for (int b = 128; b < 256; ++b) {
          // the ratios sign * a / (b * 2^k) nearest to the threshold on this grid
          const double unit = 1.0 / (static_cast<double>(b) * (1 << k));
          const double near = std::floor(sign * static_cast<double>(thr[i]) / unit);
          for (double a = near - 2; a <= near + 2; ++a) {
            if (a < 0 || a > 255 || a * unit > 1.0) continue;
            const double ratio = sign * a * unit;
            const float q = static_cast<float>(sign * a) / (static_cast<float>(b) * static_cast<float>(1 << k));
            if (q >= thr[i]) above = std::fmin(above, ratio);
            else below = std::fmax(below, ratio);
          }
        }
    if (below == -2.0) {  // no ratio is coded below it
      bound[i] = -2.0f;
      continue;
    }
    const double lo = below + std::fabs(below) * 0x1p-22, hi = above - std::fabs(above) * 0x1p-22;
    // the float32 nearest the middle with the code below (for the upper of two equal
    // thresholds, that of the lower one) in its low bits
    const float mid = static_cast<float>((lo + hi) * 0.5);
    uint32_t bits;
    std::memcpy(&bits, &mid, 4);
    bool found = false;
    for (int step = -1; step <= 1 && !found; ++step) {
      const uint32_t cand = ((bits & ~15u) + static_cast<uint32_t>(step * 16)) | static_cast<uint32_t>(i);
      float f;
      std::memcpy(&f, &cand, 4);
      if (f > lo && f < hi) {
        bound[i] = f;
        found = true;
      }
    }
    if (!found) return false;
  }
  for (int b = 0; b < 32; ++b) {
    // the ratios of bucket b lie in [lo, hi]; widened by far more than the rounding of its index
    float lo, hi;
    if (log_buckets) {
      const int e = (b & 15) > 8 ? 8 : (b & 15);
      const float inner = e == 0 ? 0.0f : std::ldexp(1.0f, e - 8), outer = std::ldexp(1.0f, e - 7);
      lo = b & 16 ? -outer : inner;
      hi = b & 16 ? -inner : outer;
    } else {
      lo = (static_cast<float>(b) - 16.5f - 0x1p-10f) / 15.0f;
      hi = (static_cast<float>(b) - 15.5f + 0x1p-10f) / 15.0f;
    }
    uint32_t base = 0, inside = 0;
    float in = 0.0f;
    for (int i = 0; i < 15; ++i) {
      if (bound[i] < lo) {
        base = static_cast<uint32_t>(i) + 1;
      } else if (bound[i] <= hi) {
        if (inside && bound[i] != in) return false;  // two thresholds in one bucket
        if (!inside) in = bound[i];
        inside = 1;
      }
    }
    if (inside) std::memcpy(&table[b], &in, 4);
    else table[b] = 0x40000000u | base;  // 2.0 and the code in its low bits: never reached
  }
  return true;
}

cudaError_t launch_kv_append(const qlora_kv_cache &c, const KvBatch &kb, const uint16_t *K, int64_t k_token_stride,
                             int64_t k_head_stride, const uint16_t *V, int64_t v_token_stride, int64_t v_head_stride,
                             const uint32_t table[32], cudaStream_t st) {
  KvRows r = cache_rows(c, 2);
  r.src[0] = K;
  r.src[1] = V;
  r.token_stride[0] = k_token_stride;
  r.token_stride[1] = v_token_stride;
  r.head_stride[0] = k_head_stride;
  r.head_stride[1] = v_head_stride;
  KvCodeTable t;
  std::memcpy(t.e, table, sizeof(t.e));
  const dim3 grid = rows_grid(r, kb.tokens);
  switch (c.codebook) {
    case QLORA_CB_FP4_E3M0: return launch_k(k_kv_append<true, true>, grid, dim3(kKvThreads), 0, st, 1, kb, r, t);
    case QLORA_CB_FP4_E2M1: return launch_k(k_kv_append<false, true>, grid, dim3(kKvThreads), 0, st, 1, kb, r, t);
    default: return launch_k(k_kv_append<false, false>, grid, dim3(kKvThreads), 0, st, 1, kb, r, t);
  }
}

cudaError_t launch_kv_read(const qlora_kv_cache &c, const KvBatch &kb, uint16_t *K_out, uint16_t *V_out,
                           const float levels[16], cudaStream_t st) {
  KvRows r = cache_rows(c, K_out && V_out ? 2 : 1);
  r.dst[0] = K_out;
  r.dst[1] = V_out;
  if (!K_out) {  // the values alone
    r.dst[0] = V_out;
    r.codes[0] = c.v_codes;
    r.absmax[0] = c.v_absmax;
  }
  Nf4Levels lv;
  std::memcpy(lv.q, levels, sizeof(lv.q));
  return launch_k(k_kv_read, rows_grid(r, kb.tokens), dim3(kKvThreads), 0, st, 1, kb, r, lv);
}

}  // namespace qlora
