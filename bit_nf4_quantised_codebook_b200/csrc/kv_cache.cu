// kv_cache.cu — writing keys and values into the 4-bit paged cache and reading
// them back: the block quantisation of "QLoRA: Efficient Finetuning of Quantized
// LLMs" (intuitivepapers.ai, §Quantize in blocks, §NormalFloat) with blocks of 64
// channels and the block's absmax kept, in bfloat16, where it is exact.
//
// Both kernels stream: a token's row is a run of 8-channel units (16 bytes of bfloat16, 4
// bytes of codes), the same for its key and its value.  A CTA takes up to 128 or 256 units - whole
// token rows, or a piece of one - finds the cache row of each of its tokens once (one guess,
// or a binary search over token_start, then the page table), and each thread then moves one or
// two units of both sides, all loads issued together.
// Bound by HBM for prompts (2 + 17/32 bytes per element each way) and by the chain of
// dependent loads token_start -> kv_len -> page_table -> data for single tokens.  Measured:
// in a replayed graph, reading 60000 tokens of 8 heads of 128 takes 57 us (5.4 TB/s, 0.84 of the
// measured copy rate); appending 8000 such tokens 13 us (2.1 times its floor: 25 instructions per element)
// and that and reading them back 25 us; a step of 16 tokens of 32 heads 5 us for both.
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

constexpr int kKvThreads = 128;
constexpr int kKvMaxTokens = kKvThreads * 2 / 8;  // token rows of a CTA (8 units or more each)
constexpr uint32_t kNoRow = 0xFFFFFFFFu;

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
  int per_token;        // units of a token: heads << head_shift
  int span;             // units of a CTA
  int tokens_per_cta;   // whole token rows of a CTA; 1 when a row is split over blockIdx.y
  uint32_t magic;       // ceil(2^32 / per_token): w / per_token = umulhi(w, magic) for w * per_token < 2^32
};

// Unit v of this CTA: its token row (counted from the CTA's first), and place in it.
// False when there is no such unit.
struct KvUnit {
  int t, in_row, head, sub;
};
__device__ __forceinline__ bool kv_unit(const KvRows &r, int v, int rows, KvUnit &u) {
  const int w = static_cast<int>(blockIdx.y) * r.span + v;
  u.t = static_cast<int>(__umulhi(static_cast<uint32_t>(w), r.magic));
  u.in_row = w - u.t * r.per_token;
  u.head = u.in_row >> r.head_shift;
  u.sub = u.in_row - (u.head << r.head_shift);
  return u.t < rows;
}

__device__ __forceinline__ uint4 ld_stream(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

// Cache row of head 0 of token row t (rows count (page, head, slot) in that order: below
// 2^31), or kNoRow when no sequence owns the row or its position or page is out of range.
__device__ __forceinline__ uint32_t token_row(const KvBatch &kb, int heads, int t) {
  // the sequence: with one token each it is t; else the last one with token_start <= t
  int lo = min(t, kb.batch - 1);
  if (!(__ldg(kb.token_start + lo) <= t && t < __ldg(kb.token_start + lo + 1))) {
    lo = 0;
    for (int hi = kb.batch; hi - lo > 1;) {
      const int mid = (lo + hi) >> 1;
      if (__ldg(kb.token_start + mid) <= t) lo = mid;
      else hi = mid;
    }
  }
  const KvSeq q = kv_seq(kb, lo);
  const int i = t - q.row0;
  if (i < 0 || i >= q.n) return kNoRow;
  const int p = q.pos0() + i;
  const int page = p < 0 ? -1 : kv_page(kb, lo, p);
  if (page < 0) {
    kv_error(kb);
    return kNoRow;
  }
  return ((static_cast<uint32_t>(page) * heads) << kb.page_shift) + (p & ((1 << kb.page_shift) - 1));
}

// The CTAs behind the last token row, launched where there is an error word: the first checks every
// sequence, those too that no row leads to (beside the others: a step of 16 tokens takes as long as without).
__device__ __forceinline__ bool checks_batch(const KvBatch &kb, int t0) {
  if (t0 < kb.tokens) return false;
  if (blockIdx.y == 0)
    for (int b = threadIdx.x; b < kb.batch; b += kKvThreads) kv_seq(kb, b);
  return true;
}

// The cache rows of this CTA's tokens, into shared memory; returns how many tokens.
__device__ __forceinline__ int load_rows(const KvBatch &kb, const KvRows &r, int t0, uint32_t *rows) {
  const int n = min(r.tokens_per_cta, kb.tokens - t0);
  for (int i = threadIdx.x; i < n; i += kKvThreads) rows[i] = token_row(kb, r.heads, t0 + i);
  __syncthreads();
  return n;
}

// LOG: buckets by sign and exponent (E3M0, one threshold per binade); otherwise 31
// equal buckets over [-1, 1].  SKIP8: the code book holds zero twice (codes 7 and 8)
// and uses 7.  Appends the code of the ratio x to `packed` (its four lowest bits).
template <bool LOG, bool SKIP8>
__device__ __forceinline__ void kv_code(float x, const uint32_t *tab, uint32_t &packed) {
  uint32_t b;  // byte offset of the bucket's word
  if (LOG) {
    const uint32_t bits = __float_as_uint(x);
    const int e = min(max(static_cast<int>((bits >> 23) & 255u) - 119, 0), 8);
    b = (static_cast<uint32_t>(e) | ((bits >> 27) & 16u)) * 4u;
  } else {
    // 2^23 + 64 + 60 x, rounded to nearest: four times the bucket (1 .. 31), and a remainder
    b = __float_as_uint(__fmaf_rn(x, 60.0f, 8388608.0f + 64.0f)) & 0x7Cu;
  }
  const uint32_t e = *reinterpret_cast<const uint32_t *>(reinterpret_cast<const uint8_t *>(tab) + b);
  const bool above = x >= __uint_as_float(e);
  if (SKIP8) {
    const uint32_t c = (e & 15u) + (above ? 1u : 0u);
    packed = packed * 16u + (c == 8u ? 9u : c);
  } else {
    packed = packed * 16u + (e & 15u);
    if (above) ++packed;
  }
}

// Codes of the 8 elements of `raw`, whose block the 8 neighbouring lanes share; `m` becomes the
// block's absmax as bfloat16 bits.
template <bool LOG, bool SKIP8>
__device__ __forceinline__ uint32_t kv_encode(const uint4 &raw, const uint32_t *tab, uint32_t &m) {
  const uint32_t wd[4] = {raw.x, raw.y, raw.z, raw.w};
  // the bits of non-negative values order like integers, infinities and NaN above every finite one
  m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = __vmaxu2(m, wd[i] & 0x7FFF7FFFu);
  m = max(m >> 16, m & 0xFFFFu);
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
  float x[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    x[2 * i] = __uint_as_float(wd[i] << 16);
    x[2 * i + 1] = __uint_as_float(wd[i] & 0xFFFF0000u);
  }
  float c = __uint_as_float(m << 16);
  if (m < (31u << 7) || m >= (223u << 7)) {
    // very small and very large blocks are scaled by 2^96 or 2^-96, exactly, so that the
    // reciprocal is a normal number
    const float scale = m < (31u << 7) ? 0x1p96f : 0x1p-96f;
    c *= scale;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= scale;
  }
  float rc;  // within 2^-23
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(rc) : "f"(c));
  if (m == 0) rc = 0.0f;  // a zero block: every ratio 0
  uint32_t packed = 0;
#pragma unroll
  for (int i = 3; i >= 0; --i) {  // the even element of each byte in the high nibble, byte 0 lowest
    kv_code<LOG, SKIP8>(__fmul_rn(x[2 * i], rc), tab, packed);
    kv_code<LOG, SKIP8>(__fmul_rn(x[2 * i + 1], rc), tab, packed);
  }
  return packed;
}

template <bool LOG, bool SKIP8, int UNITS>
__global__ void __launch_bounds__(kKvThreads) k_kv_append(const __grid_constant__ KvBatch kb,
                                                           const __grid_constant__ KvRows r,
                                                           const __grid_constant__ KvCodeTable table) {
  __shared__ uint32_t s_tab[32];
  __shared__ uint32_t s_row[kKvMaxTokens];
  if (threadIdx.x < 32) s_tab[threadIdx.x] = table.e[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * r.tokens_per_cta;
  if (checks_batch(kb, t0)) return;
  const int n = load_rows(kb, r, t0, s_row);
  uint4 raw[UNITS][2];
  uint32_t row[UNITS], sub[UNITS];
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    KvUnit u;
    row[k] = kNoRow;
    raw[k][0] = raw[k][1] = make_uint4(0, 0, 0, 0);
    if (kv_unit(r, k * kKvThreads + threadIdx.x, n, u) && s_row[u.t] != kNoRow) {
      row[k] = s_row[u.t] + (static_cast<uint32_t>(u.head) << kb.page_shift);
#pragma unroll
      for (int s = 0; s < 2; ++s)
        raw[k][s] = ld_stream(r.src[s] + static_cast<int64_t>(t0 + u.t) * r.token_stride[s] +
                              static_cast<int64_t>(u.head) * r.head_stride[s] + u.sub * 8);
    }
    sub[k] = u.sub;
  }
  bool bad = false;
#pragma unroll
  for (int k = 0; k < UNITS; ++k)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      uint32_t m;  // (units come in whole heads: 8 lanes share a block)
      const uint32_t packed = kv_encode<LOG, SKIP8>(raw[k][s], s_tab, m);
      if (row[k] != kNoRow) {
        reinterpret_cast<uint32_t *>(r.codes[s])[(static_cast<uint64_t>(row[k]) << r.head_shift) + sub[k]] = packed;
        const bool finite = m < 0x7F80u;
        if ((sub[k] & 7) == 0)
          r.absmax[s][(static_cast<uint64_t>(row[k]) << (r.head_shift - 3)) + (sub[k] >> 3)] =
              static_cast<uint16_t>(finite ? m : 0x7FC0u);
        bad |= !finite;
      }
    }
  if (bad && kb.dev_err) atomicOr(kb.dev_err, QLORA_DEVERR_NONFINITE);
}

// KEYS, VALUES: which sides are wanted.
template <bool KEYS, bool VALUES, int UNITS>
__global__ void __launch_bounds__(kKvThreads) k_kv_read(const __grid_constant__ KvBatch kb,
                                                         const __grid_constant__ KvRows r,
                                                         const __grid_constant__ Nf4Levels lv) {
  __shared__ float s_level[16];  // 16 words in 16 banks: a lookup never conflicts
  __shared__ uint32_t s_row[kKvMaxTokens];
  if (threadIdx.x < 16) s_level[threadIdx.x] = lv.q[threadIdx.x];
  pdl_wait();
  pdl_launch_dependents();
  const int t0 = static_cast<int>(blockIdx.x) * r.tokens_per_cta;
  if (checks_batch(kb, t0)) return;
  const int n = load_rows(kb, r, t0, s_row);
  uint32_t codes[UNITS][2], amax[UNITS][2];
  int64_t dst[UNITS];  // unit of the outputs, or -1
#pragma unroll
  for (int k = 0; k < UNITS; ++k) {
    KvUnit u;
    dst[k] = -1;
    codes[k][0] = codes[k][1] = amax[k][0] = amax[k][1] = 0;
    if (kv_unit(r, k * kKvThreads + threadIdx.x, n, u) && s_row[u.t] != kNoRow) {
      const uint64_t row = s_row[u.t] + (static_cast<uint32_t>(u.head) << kb.page_shift);
      const uint64_t at = (row << r.head_shift) + u.sub, block = (row << (r.head_shift - 3)) + (u.sub >> 3);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (!(s == 0 ? KEYS : VALUES)) continue;
        codes[k][s] = __ldg(reinterpret_cast<const uint32_t *>(r.codes[s]) + at);
        amax[k][s] = __ldg(r.absmax[s] + block);
      }
      dst[k] = static_cast<int64_t>(t0 + u.t) * r.per_token + u.in_row;
    }
  }
#pragma unroll
  for (int k = 0; k < UNITS; ++k)
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      if (!(s == 0 ? KEYS : VALUES)) continue;
      const float c = __uint_as_float(amax[k][s] << 16);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        o[i] = pack_bf16x2(__fmul_rn(s_level[(codes[k][s] >> (8 * i + 4)) & 15u], c),
                           __fmul_rn(s_level[(codes[k][s] >> (8 * i)) & 15u], c));
      if (dst[k] >= 0)
        __stcs(reinterpret_cast<uint4 *>(r.dst[s]) + dst[k], make_uint4(o[0], o[1], o[2], o[3]));
    }
}

// Units per thread: two, which read more at once; one while that leaves fewer CTAs than the GPU
// holds at once (16 tokens of 32 heads of 128: 5.2 us against 6.5 for an append and a read back;
// 60000 tokens of 8 heads: a read of 71 us against 56).
int units_per_thread(const qlora_kv_cache &c, int64_t tokens) {
  return tokens * c.heads * (c.head_dim / 8) <= 148 * 8 * kKvThreads ? 1 : 2;
}

KvRows cache_rows(const qlora_kv_cache &c, int units) {
  KvRows r = {};
  r.codes[0] = c.k_codes;
  r.codes[1] = c.v_codes;
  r.absmax[0] = c.k_absmax;
  r.absmax[1] = c.v_absmax;
  r.heads = c.heads;
  r.head_shift = c.head_dim == 64 ? 3 : c.head_dim == 128 ? 4 : 5;
  r.per_token = c.heads << r.head_shift;
  r.span = kKvThreads * units;
  r.tokens_per_cta = r.per_token < r.span ? r.span / r.per_token : 1;
  r.magic = static_cast<uint32_t>(((1ull << 32) + r.per_token - 1) / r.per_token);
  return r;
}

dim3 rows_grid(const KvRows &r, const KvBatch &kb) {
  return dim3(static_cast<unsigned>((static_cast<int64_t>(kb.tokens) + r.tokens_per_cta - 1) / r.tokens_per_cta) +
                  (kb.dev_err ? 1u : 0u),
              static_cast<unsigned>((r.per_token + r.span - 1) / r.span));
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
      lo = (static_cast<float>(b) - 16.125f - 0x1p-10f) / 15.0f;
      hi = (static_cast<float>(b) - 15.125f + 0x1p-10f) / 15.0f;
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
  const int units = units_per_thread(c, kb.tokens);
  KvRows r = cache_rows(c, units);
  r.src[0] = K;
  r.src[1] = V;
  r.token_stride[0] = k_token_stride;
  r.token_stride[1] = v_token_stride;
  r.head_stride[0] = k_head_stride;
  r.head_stride[1] = v_head_stride;
  KvCodeTable t;
  std::memcpy(t.e, table, sizeof(t.e));
  const dim3 grid = rows_grid(r, kb);
  auto go = [&](auto kern1, auto kern2) {
    return units == 1 ? launch_k(kern1, grid, dim3(kKvThreads), 0, st, 1, kb, r, t)
                      : launch_k(kern2, grid, dim3(kKvThreads), 0, st, 1, kb, r, t);
  };
  switch (c.codebook) {
    case QLORA_CB_FP4_E3M0: return go(k_kv_append<true, true, 1>, k_kv_append<true, true, 2>);
    case QLORA_CB_FP4_E2M1: return go(k_kv_append<false, true, 1>, k_kv_append<false, true, 2>);
    default: return go(k_kv_append<false, false, 1>, k_kv_append<false, false, 2>);
  }
}

cudaError_t launch_kv_read(const qlora_kv_cache &c, const KvBatch &kb, uint16_t *K_out, uint16_t *V_out,
                           const float levels[16], cudaStream_t st) {
  const int units = units_per_thread(c, kb.tokens);
  KvRows r = cache_rows(c, units);
  r.dst[0] = K_out;
  r.dst[1] = V_out;
  Nf4Levels lv;
  std::memcpy(lv.q, levels, sizeof(lv.q));
  const dim3 grid = rows_grid(r, kb);
  auto go = [&](auto kern1, auto kern2) {
    return units == 1 ? launch_k(kern1, grid, dim3(kKvThreads), 0, st, 1, kb, r, lv)
                      : launch_k(kern2, grid, dim3(kKvThreads), 0, st, 1, kb, r, lv);
  };
  if (!K_out) return go(k_kv_read<false, true, 1>, k_kv_read<false, true, 2>);
  if (!V_out) return go(k_kv_read<true, false, 1>, k_kv_read<true, false, 2>);
  return go(k_kv_read<true, true, 1>, k_kv_read<true, true, 2>);
}

}  // namespace qlora
