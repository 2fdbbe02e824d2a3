// kv_attention.cu — softmax attention of a call's token rows over the 4-bit paged
// cache, without writing a dequantised key or value anywhere.
//
//   s_ij = scale * sum_b cK[j,b] * (sum_{d in b} q_id * levelK_jd)     b: blocks of 64 channels
//   o_id = sum_j softmax(s_i)_j * cV[j,b] * levelV_jd
//
// The constants c multiply sums and weights, never single elements: an element costs
// one byte-permute and one shared-memory lookup per pair of codes.  A table of 256
// half2 entries (both levels of a byte), one copy per lane, is laid out so that the
// permute that picks the byte out of a code word builds the lookup's address in the
// same instruction (entry stride 256 bytes, table at a multiple of 64 KiB) and 32 lanes
// never share a bank.  The products run on mma.sync m16n8k16: with a handful of query
// rows per key/value head the tensor pipe is not what bounds this kernel (22 % busy), and
// its operands' register layouts let decoded pairs be used as they come:
//   S^T (16 tokens x 8 rows) = K (A operand: token rows, codes decoded in place) * Q^T
//   O^T (16 channels x 8 rows) += V^T (A operand: pairs of tokens of one channel per
//        register, formed by merging the nibbles of two tokens' words) * P^T
// P^T is S^T's accumulator transposed with movmatrix.
//
// Numbers.  Levels are held in fp16: exactly for the integer and float grids (stored as
// the small integers they are multiples of), within 2^-11 for NF4, at a scale where their
// errors cancel on average (see launch_kv_attention).  Each query row is
// scaled by a power of two to a largest magnitude in [2^13, 2^14) and is then exact in
// fp16 down to 2^-30 of it, and rounded to 2^-38 of it below.  The softmax keeps a reference m per row (its running maximum
// when last renewed) and float32 weights P = 2^(s - m) and their sum.  Into the second
// product go w = P * cV * F_b in fp16 (within 2^-12), F_b a scale per row and block that
// gives the largest contribution so far a w of 2^6 when last renewed.  m and F_b are renewed
// when some w passes 2^14 or the sum 2^100, which after the first tokens is rare: the usual
// step needs no maximum and no rescaling.  What is below 2^-31 of the largest contribution to
// a block is lost, whatever the constants' range, and so is a weight below 2^-126 of the
// row's largest, which is 0 in float32.  All accumulators are float32.
//
// Work.  An item is one sequence x row tile (8 * NT rows: tokens x the query heads of one
// key/value head) x key/value head, cut into steps of 128 tokens.  The steps of all items
// form one line that is cut evenly among all warp groups (4 warps; one CTA per SM), so
// sequences of any mix of lengths finish together.  Inside a step every warp takes 32
// tokens with its own running statistics; a group joins its four warps through shared
// memory at the end of its part of an item.  An item that several groups shared is joined
// from their normalised parts, in order, by a second small kernel.
//
// Bound by the decoding's instructions and their latencies together, no unit being full: 2.9
// instructions per element (one of them the lookup and permute of a pair's half, a quarter the
// copies and the softmax), issue slots 64 %, load/store pipe 68 % and integer pipe 49 % busy with the
// 16 warps that the registers allow, which wait for fixed latencies first of all.  64 sequences of 1
// to 8192 tokens, 64 query and 8 key/value heads of 128: 81 us in a replayed graph (86 call by call),
// 3.72 TB/s of codes and constants (0.58 of the measured copy rate); one sequence of 131071: 50 us.
// Codes loaded straight into registers took 62 us for the latter (one 32-byte sector per request),
// registers spilled beside a full shared memory 4 us.  The tiles of 16 rows and the heads of 256 spill
// all the same (88 bytes a thread with heads of 128, 32 with 64 and 256); what that costs them is not measured.
#include <atomic>
#include <climits>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include "internal.h"
#include "kv_attention.cuh"
#include "kv_common.cuh"
#include "launch.cuh"

namespace qlora {
namespace {

constexpr int kStepTokens = 128;     // tokens of one step of a group (4 warps x 32)
// What starting and ending an item costs a group, in steps: its place on the line is that much
// longer than its steps, so that a group with many short items gets fewer of them.
constexpr int kItemOverhead = 3;  // 64 uneven sequences: 106 us without, 92, 81, 81, 83 us with 1, 2, 3, 5
__device__ __forceinline__ void mma16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                         uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
// The same with a zero accumulator.
__device__ __forceinline__ void mma16816_zero(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=f"(c[0]), "=f"(c[1]), "=f"(c[2]), "=f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(0.0f));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
template <int NB>
__device__ __forceinline__ void ld_consts(const uint8_t *p, uint32_t (&c)[(NB + 1) / 2]) {
  if (NB == 1) c[0] = *reinterpret_cast<const uint16_t *>(p);
  if (NB == 2) c[0] = *reinterpret_cast<const uint32_t *>(p);
  if (NB == 4) {
    const uint2 v = *reinterpret_cast<const uint2 *>(p);
    c[0] = v.x;
    c[(NB + 1) / 2 - 1] = v.y;
  }
}
template <int NB>
__device__ __forceinline__ float const_of(const uint32_t (&c)[(NB + 1) / 2], int b) {
  return __uint_as_float(b & 1 ? c[b / 2] & 0xFFFF0000u : c[b / 2] << 16);
}

// log2 of the scale F of a block's weights, for the reference m and the largest
// contribution mv.
__device__ __forceinline__ float weight_exponent(float m, float mv) {
  return fminf(fmaxf(kLift + (m - mv), -126.0f), 126.0f);
}

// Steps, row tiles and first token of a sequence's items.
struct KvSpan {
  KvSeq q;
  int tiles;   // row tiles per key/value head (0: no rows)
  int steps;   // steps of each item (at least 1 where there are rows)
  int lo;      // first cached token that a row may see, rounded down to 32
  __device__ __forceinline__ int64_t units(int heads) const {
    return static_cast<int64_t>(tiles) * heads * (steps + kItemOverhead);
  }
};
__device__ __forceinline__ KvSpan kv_span(const KvAttnArgs &a, int b, int tile_rows) {
  KvSpan s;
  s.q = kv_seq(a.kb, b);
  const int rows = s.q.n * a.group;
  // (written by an earlier kernel of this call, maybe after this one started: from the second-level cache)
  s.tiles = rows > a.few_rows && __ldcg(a.again + b) == 0 ? 0 : (rows + tile_rows - 1) / tile_rows;
  int lo = 0;
  if (a.window > 0) lo = max(0, min(s.q.len, s.q.pos0() - a.window + 1)) & ~31;
  s.lo = lo;
  s.steps = max(1, (s.q.len - lo + kStepTokens - 1) / kStepTokens);
  return s;
}

// What a warp needs again after the steps of a part.  Kept in shared memory meanwhile: with
// little first-level cache beside it, a spilled register would be a second-level cache access
// in every step.
struct WarpState {
  int64_t at, stop, begin, total, seq_start, first, end;
  int b, head, tile, step0, step1, row0, n, len, tiles, steps, lo;
};

template <int D_, int NT_, int GROUPS_>
struct AttnCfg {
  static constexpr int D = D_;
  static constexpr int NT = NT_;          // tiles of 8 query rows
  static constexpr int ROWS = 8 * NT;
  static constexpr int NB = D / 64;       // blocks of 64 channels
  static constexpr int GROUPS = GROUPS_;  // warp groups per CTA
  static constexpr int THREADS = GROUPS * 128;
  static constexpr int T = D * NT > 128 ? 1 : 2;  // tiles of 16 tokens in one part of a warp's work
  static constexpr int PARTS = 2 / T;         // parts of a warp's 32 tokens of a step
  static constexpr int CW = (NB + 1) / 2;     // words of a token's constants
  // shared memory: a ring of parts per warp, the first FRONT of them before the table
  static constexpr int CODES = T * 16 * (D / 2), CONSTS = T * 16 * NB * 2;  // bytes of a part's keys (values the same)
  static constexpr int PART_BYTES = 2 * (CODES + CONSTS);
  static constexpr int STAGES = 8704 / PART_BYTES;  // 2 or 4
  static constexpr int RING = STAGES * PART_BYTES;
  static constexpr int WARPS = 4 * GROUPS;
  static constexpr int FRONT = 7;
  static constexpr int LSE_BYTES = WARPS * ROWS * 4;
  static constexpr int SMEM_BYTES = 0x20000 + (WARPS - FRONT) * RING + LSE_BYTES + (THREADS + 1) * 8 + WARPS * sizeof(WarpState);
  static_assert(ROWS * D * 4 <= RING, "a warp's outputs are joined in its ring");
  static_assert(RING % 128 == 0 && FRONT * RING <= 0x10000 - 0x400, "rings before the table");
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
};

// The token of a tile that index i < 8 of a product's token axis stands for (i + 8: 8 more).
// A lane's value tokens, indices 2t and 2t + 1, are then t and 4 + (t ^ 2): with the swizzle
// below, neither the key loads (lane (g, t): index g, 8 bytes) nor the value loads (lane
// (g, t): indices 2t and 2t + 1, 4 bytes at 4g) of a warp meet in a bank.
__device__ __forceinline__ int token_of(int i) { return i & 1 ? 4 + ((i >> 1) ^ 2) : i >> 1; }
// 32-byte blocks of a token's codes are stored at block k ^ swizzle(token).
template <int NB>
__device__ __forceinline__ int swizzle(int token) {
  return NB == 4 ? token & 3 : NB == 2 ? (token >> 1) & 1 : 0;
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) k_kv_attention(const __grid_constant__ KvAttnArgs a) {
  constexpr int D = C::D, NT = C::NT, NB = C::NB, T = C::T, CW = C::CW, ROWS = C::ROWS, S = C::STAGES;
  extern __shared__ __align__(1024) uint8_t smem[];
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t table = (smem_base + 0xFFFFu) & ~0xFFFFu;  // 64 KiB at a multiple of 64 KiB
  uint8_t *tail = smem + (table - smem_base) + 0x10000u;    // rings, the joins' sums, the line's prefix sums
  float *lse = reinterpret_cast<float *>(tail + (C::WARPS - C::FRONT) * C::RING);
  int64_t *prefix = reinterpret_cast<int64_t *>(tail + (C::WARPS - C::FRONT) * C::RING + C::LSE_BYTES);
  volatile WarpState *state = reinterpret_cast<WarpState *>(prefix + C::THREADS + 1) + (threadIdx.x >> 5);
  __shared__ int64_t s_warp_sum[C::THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gq = warp >> 2, gw = warp & 3;  // group in the CTA, warp in the group
  const int g = lane >> 2, t = lane & 3;
  auto build_table = [&] {
    for (int i = tid; i < 256 * 32; i += C::THREADS) {
      const int byte = i >> 5;
      const __half2 h = __halves2half2(a.levels[byte >> 4], a.levels[byte & 15]);
      *reinterpret_cast<__half2 *>(smem + (table - smem_base) + byte * 256 + (i & 31) * 4) = h;
    }
  };
  // beside the many-row kernel there is often nothing to do here, and no kernel before this one
  // leaves room to build the table while it runs
  const bool alone = a.few_rows == INT_MAX;
  if (alone) build_table();
  pdl_wait();
  pdl_launch_dependents();
  if (table - smem_base < C::FRONT * C::RING) {  // cannot happen while shared memory starts low
    if (tid < C::GROUPS * 2) a.parts[blockIdx.x * C::GROUPS * 2 + tid].joins = 0;
    kv_error(a.kb);
    return;
  }

  // ---------------------------------------------------------------- the line of steps
  // each thread sums a run of sequences; prefix[i] is where run i starts
  const int run = (a.kb.batch + C::THREADS - 1) / C::THREADS;
  {
    const int b0 = min(a.kb.batch, tid * run), b1 = min(a.kb.batch, b0 + run);
    int64_t sum = 0;
    for (int b = b0; b < b1; ++b) sum += kv_span(a, b, ROWS).units(a.heads);
    int64_t x = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) s_warp_sum[warp] = x;
    __syncthreads();
    int64_t at = x - sum;
    for (int w = 0; w < warp; ++w) at += s_warp_sum[w];
    prefix[tid] = at;
    if (tid == C::THREADS - 1) prefix[C::THREADS] = at + sum;
    __syncthreads();
  }
  int64_t total = prefix[C::THREADS];
  if (!alone && total > 0) {
    build_table();
    __syncthreads();
  }
  const int workers = gridDim.x * C::GROUPS, me = blockIdx.x * C::GROUPS + gq;
  int64_t at = me * total / workers;
  int64_t stop = static_cast<int64_t>(me + 1) * total / workers;
  int64_t begin = at;
  const uint32_t tab = table | (lane * 4);
  auto ring_of = [&](int w) { return w < C::FRONT ? smem + w * C::RING : tail + (w - C::FRONT) * C::RING; };
  uint8_t *ring = ring_of(warp);
  // this lane's place in a part's codes: keys of index g and values of index 2t, by block
  int koff[NB], voff[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    koff[k] = token_of(g) * (D / 2) + 32 * (k ^ swizzle<NB>(token_of(g))) + 8 * t;
    voff[k] = C::CODES + t * (D / 2) + 32 * (k ^ swizzle<NB>(t)) + 4 * g;
  }
  const int vodd = (4 + (t ^ 2) - t) * (D / 2);  // from index 2t to 2t + 1 (whose swizzle differs by NB / 2)
  const int coff = 2 * C::CODES + token_of(g) * NB * 2;
  // and in its copies: 16-byte chunk `lane` of each 512 bytes of codes, and one chunk of constants
  constexpr int CH = D / 32;                 // chunks of a token
  constexpr int CC = C::CONSTS / 16;         // chunks of a part's key constants
  const int copy_dst = (lane / CH) * (D / 2) + (((lane % CH) ^ (swizzle<NB>(lane / CH) << 1)) << 4);
  const uint16_t *const_src = (lane < CC ? a.k_absmax : a.v_absmax) + (lane % (2 * NB)) * 8;
  const bool one_tile_pages = a.kb.page_shift < 5;  // pages of 16: a part's two tiles lie apart
  const bool const_second = T == 2 && (lane % CC) >= CC / 2;  // of the part's second tile
  const uint32_t ring_addr = smem_u32(ring);
  if (gw == 0 && lane < 2) {  // no part yet
    a.parts[me * 2 + lane].present = 0;
    a.parts[me * 2 + lane].joins = 0;
  }

  int b = 0;
  int64_t seq_start = 0;
  KvSpan sp = {};
  if (at < stop) {
    int lo = 0, hi = C::THREADS;  // last run that starts at or before `at` (empty ones follow the one that holds it)
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (prefix[mid] <= at) lo = mid;
      else hi = mid;
    }
    b = lo * run;
    seq_start = prefix[lo];
    sp = kv_span(a, b, ROWS);
  }
  while (at < stop) {
    while (seq_start + sp.units(a.heads) <= at) {  // on to the sequence that holds step `at`
      seq_start += sp.units(a.heads);
      sp = kv_span(a, ++b, ROWS);
    }
    const int64_t rel = at - seq_start;
    const int units = sp.steps + kItemOverhead;  // the item's place on the line: its overhead, then its steps
    const int item = static_cast<int>(rel / units);
    int head = item % a.heads, tile = item / a.heads;
    int64_t first = seq_start + static_cast<int64_t>(item) * units, end = first + units;
    int step0 = max(0, static_cast<int>(at - first) - kItemOverhead);
    int step1 = (stop < end ? static_cast<int>(stop - first) : units) - kItemOverhead;
    if (step1 <= step0) {  // this range ends before the item's first step
      at = stop;
      break;
    }
    if (lane == 0) {
      state->at = at;
      state->stop = stop;
      state->begin = begin;
      state->total = total;
      state->seq_start = seq_start;
      state->first = first;
      state->end = end;
      state->b = b;
      state->head = head;
      state->tile = tile;
      state->step0 = step0;
      state->step1 = step1;
      state->row0 = sp.q.row0;
      state->n = sp.q.n;
      state->len = sp.q.len;
      state->tiles = sp.tiles;
      state->steps = sp.steps;
      state->lo = sp.lo;
    }
    __syncwarp();
    int row_limit = sp.q.n * a.group - tile * ROWS;  // rows of the tile that exist

    // ------------------------------------------------------------ query rows -> B operand
    uint32_t q[NT][NB][4][2];
    float qs[NT][2];       // factor of the scores of rows 2t, 2t + 1
    int see_lo[NT][2], see_hi[NT][2];
    int all_lo = 0, all_hi = 0x7FFFFFFF;  // tokens that every row sees
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int r = n * 8 + g;
      const bool live = r < row_limit;
      const int rr = tile * ROWS + r;
      const int i = live ? rr / a.group : 0;
      const int h = live ? rr - i * a.group : 0;
      const uint16_t *src = a.Q + static_cast<int64_t>(sp.q.row0 + i) * a.q_token_stride +
                            static_cast<int64_t>(head * a.group + h) * a.q_head_stride + 16 * t;
      uint32_t raw[NB][8];
      uint32_t m = 0;
#pragma unroll
      for (int k = 0; k < NB; ++k) {
        uint4 u = make_uint4(0, 0, 0, 0), v = u;
        if (live) {
          u = __ldg(reinterpret_cast<const uint4 *>(src + 64 * k));
          v = __ldg(reinterpret_cast<const uint4 *>(src + 64 * k + 8));
        }
        raw[k][0] = u.x, raw[k][1] = u.y, raw[k][2] = u.z, raw[k][3] = u.w;
        raw[k][4] = v.x, raw[k][5] = v.y, raw[k][6] = v.z, raw[k][7] = v.w;
#pragma unroll
        for (int x = 0; x < 8; ++x) m = __vmaxu2(m, raw[k][x] & 0x7FFF7FFFu);
      }
      m = max(m >> 16, m & 0xFFFFu);
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
      m = max(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
      // q * 2^-e has its largest magnitude in [2^13, 2^14); e within what float32 powers hold
      int e = static_cast<int>(m >> 7) - 127 - 13;
      if (m == 0 || m >= 0x7F80u) e = 0;
      e = max(e, -120);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int x = 0; x < 8; ++x)
          q[n][k][x >> 1][x & 1] = pack_half2(__uint_as_float(raw[k][x] << 16) * down,
                                              __uint_as_float(raw[k][x] & 0xFFFF0000u) * down);
      float up = __uint_as_float(static_cast<uint32_t>(127 + e) << 23) * a.scale_log2;
      if (m >= 0x7F80u) up = __uint_as_float(0x7FC00000u);  // a non-finite query: its row is NaN throughout
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        qs[n][c] = __shfl_sync(0xFFFFFFFFu, up, (2 * t + c) * 4);
        const int ic = __shfl_sync(0xFFFFFFFFu, i, (2 * t + c) * 4);
        const int lc = __shfl_sync(0xFFFFFFFFu, live ? 1 : 0, (2 * t + c) * 4);
        const int pos = sp.q.pos0() + ic;
        see_hi[n][c] = a.causal ? min(sp.q.len, pos + 1) : sp.q.len;
        see_lo[n][c] = a.window > 0 ? max(0, pos - a.window + 1) : 0;
        if (lc) {
          all_lo = max(all_lo, see_lo[n][c]);
          all_hi = min(all_hi, see_hi[n][c]);
        }
      }
    }
    all_lo = __reduce_max_sync(0xFFFFFFFFu, all_lo);
    all_hi = __reduce_min_sync(0xFFFFFFFFu, all_hi);

    float o[NT][NB][4][4];
    float l[NT][2], mx[NT][2];            // sum and reference of rows 2t, 2t + 1
    float mv[NT][NB][2], fv[NT][NB][2];   // largest s + log2 cV when last renewed, and F = weight_scale(mx - mv)
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        l[n][c] = 0.0f;
        mx[n][c] = kFloor;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          mv[n][k][c] = kFloor;
          fv[n][k][c] = 1.0f;
        }
      }
#pragma unroll
      for (int k = 0; k < NB; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[n][k][i][c] = 0.0f;
    }

    // ------------------------------------------------------------ the steps
    // This warp's 32-token chunks lie 128 apart; a chunk is worked off in parts of T tiles of
    // 16 tokens, copied STAGES - 1 parts ahead into this warp's ring.  A tile lies inside one
    // page, so its 16 slots can be copied whether or not the sequence ends among them; what
    // lies past the end is masked like what a row does not see.
    const int parts = (step1 - step0) * C::PARTS;
    auto base_of = [&](int u) {
      return sp.lo + (step0 + u / C::PARTS) * kStepTokens + gw * 32 + (u % C::PARTS) * (T * 16);
    };
    // The page of each tile is loaded a part before it is used, and checked then.
    const int32_t *pages = a.kb.page_table + static_cast<int64_t>(b) * a.kb.max_pages;
    bool bad_page = false;
    auto load_pages = [&](int u, int (&page)[T]) {
      const int tok = base_of(u);
      page[0] = __ldg(pages + min(tok >> a.kb.page_shift, a.kb.max_pages - 1));
      if (T == 2 && one_tile_pages) page[T - 1] = __ldg(pages + min((tok + 16) >> a.kb.page_shift, a.kb.max_pages - 1));
    };
    // cache row of the token `tok` on `page`; row 0 for tiles without a page
    auto row_of = [&](int tok, int page) -> uint32_t {
      const bool bad = static_cast<unsigned>(page) >= static_cast<unsigned>(a.kb.num_pages);
      bad_page |= bad && tok < sp.q.len;
      const uint32_t row = ((static_cast<uint32_t>(page) * a.heads + head) << a.kb.page_shift) +
                           (tok & ((1 << a.kb.page_shift) - 1));
      return bad ? 0 : row;
    };
    auto copy_codes = [&](uint32_t dst, const uint8_t *ks, const uint8_t *vs, int bytes) {
#pragma unroll
      for (int j = 0; j < C::CODES; j += 512)  // 512 bytes each
        if (j < bytes) {
          copy16(dst + j, ks + j);
          copy16(dst + C::CODES + j, vs + j);
        }
    };
    auto copy_part = [&](int u, const int (&page)[T]) {
      const uint32_t dst = ring_addr + (u % S) * C::PART_BYTES;
      const int tok = base_of(u);
      const uint32_t row = row_of(tok, page[0]);
      const uint64_t at = static_cast<uint64_t>(row) * (D / 2) + lane * 16;
      uint32_t const_row = row;
      if (T == 1 || !one_tile_pages) {  // the part's rows lie side by side
        copy_codes(dst + copy_dst, a.k_codes + at, a.v_codes + at, C::CODES);
        if (T == 2 && const_second) const_row += 16;
      } else {
        const uint32_t row1 = row_of(tok + 16, page[T - 1]);
        const uint64_t at1 = static_cast<uint64_t>(row1) * (D / 2) + lane * 16;
        copy_codes(dst + copy_dst, a.k_codes + at, a.v_codes + at, 8 * D);
        copy_codes(dst + copy_dst + 8 * D, a.k_codes + at1, a.v_codes + at1, 8 * D);
        if (const_second) const_row = row1;
      }
      if (lane < 2 * CC) copy16(dst + 2 * C::CODES + lane * 16, const_src + static_cast<uint64_t>(const_row) * NB);
    };
    int page[T];
    {
      int first_pages[S][T];
#pragma unroll
      for (int j = 0; j < S; ++j) load_pages(j, first_pages[j]);
      load_pages(S, page);
#pragma unroll
      for (int j = 0; j < S; ++j) {
        if (j < parts) copy_part(j, first_pages[j]);
        copies_commit();
      }
    }
    for (int u = 0; u < parts; ++u) {
      const int tok0 = base_of(u);
      copies_wait<S - 1>();
      __syncwarp();  // every lane's copies of this part are there
      const uint8_t *part = ring + (u % S) * C::PART_BYTES;
      // products of the scores: s[i][n][0..3] = (token g, row 2t), (g, 2t + 1), (g + 8, 2t), (g + 8, 2t + 1)
      float s[T][NT][4];
#pragma unroll
      for (int i = 0; i < T; ++i) {
        uint32_t kcon[2][CW];
        ld_consts<NB>(part + coff + i * 32 * NB, kcon[0]);
        ld_consts<NB>(part + coff + i * 32 * NB + 16 * NB, kcon[1]);
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          float acc[NT][4];
          const uint2 w0 = *reinterpret_cast<const uint2 *>(part + i * 8 * D + koff[k]);
          const uint2 w1 = *reinterpret_cast<const uint2 *>(part + i * 8 * D + 4 * D + koff[k]);
          {
            const uint32_t a0 = lookup<0>(w0.x, tab), a1 = lookup<0>(w1.x, tab), a2 = lookup<1>(w0.x, tab),
                           a3 = lookup<1>(w1.x, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816_zero(acc[n], a0, a1, a2, a3, q[n][k][0][0], q[n][k][0][1]);
          }
          {
            const uint32_t a0 = lookup<2>(w0.x, tab), a1 = lookup<2>(w1.x, tab), a2 = lookup<3>(w0.x, tab),
                           a3 = lookup<3>(w1.x, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(acc[n], a0, a1, a2, a3, q[n][k][1][0], q[n][k][1][1]);
          }
          {
            const uint32_t a0 = lookup<0>(w0.y, tab), a1 = lookup<0>(w1.y, tab), a2 = lookup<1>(w0.y, tab),
                           a3 = lookup<1>(w1.y, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(acc[n], a0, a1, a2, a3, q[n][k][2][0], q[n][k][2][1]);
          }
          {
            const uint32_t a0 = lookup<2>(w0.y, tab), a1 = lookup<2>(w1.y, tab), a2 = lookup<3>(w0.y, tab),
                           a3 = lookup<3>(w1.y, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(acc[n], a0, a1, a2, a3, q[n][k][3][0], q[n][k][3][1]);
          }
          const float c0 = const_of<NB>(kcon[0], k), c1 = const_of<NB>(kcon[1], k);
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const float cc = c < 2 ? c0 : c1;
              s[i][n][c] = k == 0 ? cc * acc[n][c] : fmaf(cc, acc[n][c], s[i][n][c]);
            }
        }
      }
      uint32_t vcon[T][2][CW];
#pragma unroll
      for (int i = 0; i < T; ++i) {
        ld_consts<NB>(part + coff + C::CONSTS + i * 32 * NB, vcon[i][0]);
        ld_consts<NB>(part + coff + C::CONSTS + i * 32 * NB + 16 * NB, vcon[i][1]);
      }
      // scores, with what a row does not see at -inf: only where some row does not see the whole part
      const bool masked = tok0 < all_lo || tok0 + T * 16 > all_hi;
#pragma unroll
      for (int i = 0; i < T; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) s[i][n][c] *= qs[n][c & 1];
      if (masked) {
#pragma unroll
        for (int i = 0; i < T; ++i)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              const int j = tok0 + 16 * i + token_of(g) + 8 * (c >> 1);
              if (j >= see_hi[n][c & 1] || j < see_lo[n][c & 1]) s[i][n][c] = -INFINITY;
            }
      }
      // weights, in fp16 pairs (rows 2t, 2t + 1) for each block, and the new sums
      uint32_t p[T][NT][NB][2];
      float sum[NT][2];
      auto weights = [&](bool hide) -> bool {
        float most = 0.0f;
        bool over = false;
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          sum[n][0] = l[n][0];
          sum[n][1] = l[n][1];
#pragma unroll
          for (int i = 0; i < T; ++i)
#pragma unroll
            for (int x = 0; x < 2; ++x) {
              const float s0 = s[i][n][2 * x], s1 = s[i][n][2 * x + 1];
              const float p0 = ex2(s0 - mx[n][0]), p1 = ex2(s1 - mx[n][1]);
              sum[n][0] += p0;
              sum[n][1] += p1;
#pragma unroll
              for (int k = 0; k < NB; ++k) {
                const float cv = const_of<NB>(vcon[i][x], k);
                // (in this order: a scale times a constant may pass float32, and 0 * inf would stay)
                float w0 = p0 * cv * fv[n][k][0], w1 = p1 * cv * fv[n][k][1];
                if (hide) {  // a token that a row does not see adds nothing, whatever its value's constant
                  w0 = s0 == -INFINITY ? 0.0f : w0;
                  w1 = s1 == -INFINITY ? 0.0f : w1;
                }
                most = fmaxf(most, fmaxf(w0, w1));
                p[i][n][k][x] = pack_half2(w0, w1);
              }
            }
          over |= sum[n][0] > kMostSum || sum[n][1] > kMostSum;
        }
        return over || most > kMostWeight;
      };
      const bool over = masked ? weights(true) : weights(false);
      if (__any_sync(0xFFFFFFFFu, over)) {
        // renew: references to the maximum of the scores so far, scales to the largest contributions
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            float top = mx[n][c];
#pragma unroll
            for (int i = 0; i < T; ++i) top = fmaxf(top, fmaxf(s[i][n][c], s[i][n][c + 2]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, d));
            const float old = mx[n][c];
            l[n][c] *= ex2(old - top);
            mx[n][c] = top;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              float tv = mv[n][k][c];
#pragma unroll
              for (int i = 0; i < T; ++i)
#pragma unroll
                for (int x = 0; x < 2; ++x)
                  tv = fmaxf(tv, s[i][n][c + 2 * x] + lg2(const_of<NB>(vcon[i][x], k)));
#pragma unroll
              for (int d = 4; d < 32; d <<= 1) tv = fmaxf(tv, __shfl_xor_sync(0xFFFFFFFFu, tv, d));
              // accumulated so far in units of 2^-(m + log2 F)
              const float e = weight_exponent(top, tv);
              const float f = ex2((old - top) + (e - weight_exponent(old, mv[n][k][c])));
              mv[n][k][c] = tv;
              fv[n][k][c] = ex2(e);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                o[n][k][i][c] *= f;
                o[n][k][i][c + 2] *= f;
              }
            }
          }
        weights(true);
      }
      // the second product
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        l[n][0] = sum[n][0];
        l[n][1] = sum[n][1];
      }
#pragma unroll
      for (int i = 0; i < T; ++i) {
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            p[i][n][k][0] = movmatrix(p[i][n][k][0]);
            p[i][n][k][1] = movmatrix(p[i][n][k][1]);
          }
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          // even channels of indices 2t, 2t + 1 in one byte (x), odd ones in another (y)
          auto word = [&](int offset) { return *reinterpret_cast<const uint32_t *>(part + i * 8 * D + offset); };
          const uint32_t v0 = word(voff[k]), v1 = word(voff[k ^ (NB / 2)] + vodd);
          const uint32_t v2 = word(voff[k] + 4 * D), v3 = word(voff[k ^ (NB / 2)] + 4 * D + vodd);
          const uint32_t x0 = (v0 & 0xF0F0F0F0u) | ((v1 >> 4) & 0x0F0F0F0Fu);
          const uint32_t y0 = ((v0 << 4) & 0xF0F0F0F0u) | (v1 & 0x0F0F0F0Fu);
          const uint32_t x1 = (v2 & 0xF0F0F0F0u) | ((v3 >> 4) & 0x0F0F0F0Fu);
          const uint32_t y1 = ((v2 << 4) & 0xF0F0F0F0u) | (v3 & 0x0F0F0F0Fu);
          {
            const uint32_t a0 = lookup<0>(x0, tab), a1 = lookup<0>(y0, tab), a2 = lookup<0>(x1, tab),
                           a3 = lookup<0>(y1, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][k][0], a0, a1, a2, a3, p[i][n][k][0], p[i][n][k][1]);
          }
          {
            const uint32_t a0 = lookup<1>(x0, tab), a1 = lookup<1>(y0, tab), a2 = lookup<1>(x1, tab),
                           a3 = lookup<1>(y1, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][k][1], a0, a1, a2, a3, p[i][n][k][0], p[i][n][k][1]);
          }
          {
            const uint32_t a0 = lookup<2>(x0, tab), a1 = lookup<2>(y0, tab), a2 = lookup<2>(x1, tab),
                           a3 = lookup<2>(y1, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][k][2], a0, a1, a2, a3, p[i][n][k][0], p[i][n][k][1]);
          }
          {
            const uint32_t a0 = lookup<3>(x0, tab), a1 = lookup<3>(y0, tab), a2 = lookup<3>(x1, tab),
                           a3 = lookup<3>(y1, tab);
#pragma unroll
            for (int n = 0; n < NT; ++n) mma16816(o[n][k][3], a0, a1, a2, a3, p[i][n][k][0], p[i][n][k][1]);
          }
        }
      }
      __syncwarp();  // every lane has read this part
      if (u + S < parts) copy_part(u + S, page);
      copies_commit();
      load_pages(u + S + 1, page);
    }
    copies_wait<0>();
    if (bad_page) kv_error(a.kb);
    at = state->at;
    stop = state->stop;
    begin = state->begin;
    total = state->total;
    seq_start = state->seq_start;
    first = state->first;
    end = state->end;
    b = state->b;
    head = state->head;
    tile = state->tile;
    step0 = state->step0;
    step1 = state->step1;
    sp.q.row0 = state->row0;
    sp.q.n = state->n;
    sp.q.len = state->len;
    sp.tiles = state->tiles;
    sp.steps = state->steps;
    sp.lo = state->lo;
    row_limit = sp.q.n * a.group - tile * ROWS;

    // ------------------------------------------------------------ join the group's warps
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        float sum = l[n][c];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, d);
        const int r = n * 8 + 2 * t + c;
        const float inv = sum > 0.0f || sum != sum ? a.v_unit / sum : 0.0f;
        if (g == 0) lse[warp * ROWS + r] = sum > 0.0f || sum != sum ? mx[n][c] + lg2(sum) : -INFINITY;
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          // channels 8g .. 8g + 7 of block k, without the weights' scale (a power of two that may
          // pass float32's exponents: applied as two halves)
          const float f = ex2(-0.5f * weight_exponent(mx[n][c], mv[n][k][c]));
          const float fi = f * inv;
          float *dst = reinterpret_cast<float *>(ring) + r * D + 64 * k + 8 * g;
          *reinterpret_cast<float4 *>(dst) = make_float4(o[n][k][0][c] * fi * f, o[n][k][0][c + 2] * fi * f,
                                                         o[n][k][1][c] * fi * f, o[n][k][1][c + 2] * fi * f);
          *reinterpret_cast<float4 *>(dst + 4) = make_float4(o[n][k][2][c] * fi * f, o[n][k][2][c + 2] * fi * f,
                                                             o[n][k][3][c] * fi * f, o[n][k][3][c + 2] * fi * f);
        }
      }
    named_barrier(1 + gq, 128);
    const float *my_lse = lse + gq * 4 * ROWS;
    const bool whole = step0 == 0 && step1 == sp.steps;
    const int slot = at == begin ? 0 : 1;
    const int64_t part = static_cast<int64_t>(me) * 2 + slot;
    const int tl = tid & 127;
    for (int x = tl; x < ROWS * (D / 8); x += 128) {
      const int r = x / (D / 8), ch = (x % (D / 8)) * 8;
      float top = my_lse[r], wsum = 0.0f;
#pragma unroll
      for (int w = 1; w < 4; ++w) top = fmaxf(top, my_lse[w * ROWS + r]);
      float acc[8] = {};
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const float x = my_lse[w * ROWS + r];
        const float f = x == -INFINITY ? 0.0f : ex2(x - top);
        wsum += f;
        const float *src = reinterpret_cast<const float *>(ring_of(gq * 4 + w)) + r * D + ch;
        const float4 u = *reinterpret_cast<const float4 *>(src);
        const float4 v = *reinterpret_cast<const float4 *>(src + 4);
        acc[0] = fmaf(f, u.x, acc[0]);
        acc[1] = fmaf(f, u.y, acc[1]);
        acc[2] = fmaf(f, u.z, acc[2]);
        acc[3] = fmaf(f, u.w, acc[3]);
        acc[4] = fmaf(f, v.x, acc[4]);
        acc[5] = fmaf(f, v.y, acc[5]);
        acc[6] = fmaf(f, v.z, acc[6]);
        acc[7] = fmaf(f, v.w, acc[7]);
      }
      const float inv = wsum == 0.0f ? 0.0f : 1.0f / wsum;
#pragma unroll
      for (int i = 0; i < 8; ++i) acc[i] *= inv;
      if (!whole) {
        float *dst = a.part_o + (part * ROWS + r) * D + ch;
        *reinterpret_cast<float4 *>(dst) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        *reinterpret_cast<float4 *>(dst + 4) = make_float4(acc[4], acc[5], acc[6], acc[7]);
        if (ch == 0) a.part_lse[part * ROWS + r] = wsum == 0.0f ? -INFINITY : top + lg2(wsum);
      } else if (r < row_limit) {
        const int rr = tile * ROWS + r, i = rr / a.group, h = rr - i * a.group;
        uint16_t *dst = a.out +
                        (static_cast<int64_t>(sp.q.row0 + i) * a.heads * a.group + head * a.group + h) * D + ch;
        *reinterpret_cast<uint4 *>(dst) = make_uint4(pack_bf16x2(acc[0], acc[1]), pack_bf16x2(acc[2], acc[3]),
                                                     pack_bf16x2(acc[4], acc[5]), pack_bf16x2(acc[6], acc[7]));
      }
    }
    if (!whole && tl == 0) {
      // the group that holds step u is the largest g with g * total / workers <= u
      auto group_of = [&](int64_t u) { return static_cast<int>(((u + 1) * workers - 1) / total); };
      KvPart p;
      p.present = 1;
      p.row0 = sp.q.row0;
      p.head = head;
      p.tile = tile;
      p.rows = row_limit;
      p.g0 = group_of(first + kItemOverhead);  // holds the item's first step
      p.last = group_of(end - 1);
      p.head_slot = p.g0 * total / workers >= first ? 0 : 1;
      p.joins = step0 > 0 && at == (p.g0 + 1) * total / workers ? 1 : 0;
      a.parts[part] = p;
    }
    named_barrier(1 + gq, 128);  // the rings are free again
    at = first + kItemOverhead + step1;
  }
}

using Cfg64x1 = AttnCfg<64, 1, 4>;
using Cfg64x2 = AttnCfg<64, 2, 4>;
using Cfg128x1 = AttnCfg<128, 1, 4>;
using Cfg128x2 = AttnCfg<128, 2, 3>;
using Cfg256x1 = AttnCfg<256, 1, 3>;

constexpr int kManyParts = 8;
template <class C>
cudaError_t run_attention(KvAttnArgs a, void *ws, int num_sms, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void *>(k_kv_attention<C>), C::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  if (num_sms * C::GROUPS > kMaxWorkers) num_sms = kMaxWorkers / C::GROUPS;
  const int workers = num_sms * C::GROUPS;
  uint8_t *w = static_cast<uint8_t *>(ws);
  a.parts = reinterpret_cast<KvPart *>(w);
  w += static_cast<size_t>(workers) * 2 * sizeof(KvPart);
  a.part_lse = reinterpret_cast<float *>(w);
  w += static_cast<size_t>(workers) * 2 * C::ROWS * 4;
  a.part_o = reinterpret_cast<float *>(w);
  e = launch_k(k_kv_attention<C>, dim3(num_sms), dim3(C::THREADS), C::SMEM_BYTES, st, 1, a);
  if (e != cudaSuccess) return e;
  // Four warps to a row where an item has many parts (one sequence of 131071 tokens, 74 parts to
  // an item: 49 against 54 us); one where it has a few, in a quarter of the CTAs, most of which find
  // nothing to join (24 sequences of drafts: 22 against 27 us).  With the many-row kernel in the
  // call there is usually nothing at all.
  if (a.few_rows == INT_MAX && workers > kManyParts * static_cast<int64_t>(a.kb.batch) * a.heads)
    return launch_k(k_kv_join<C::D, C::ROWS, 4>, dim3(workers - 1, C::ROWS / 2), dim3(256), 0, st, 1, a);
  return launch_k(k_kv_join<C::D, C::ROWS, 1>, dim3(workers - 1, C::ROWS / 8), dim3(256), 0, st, 1, a);
}

template <class C>
size_t workspace_of(int num_sms) {
  return static_cast<size_t>(num_sms) * C::GROUPS * 2 * (sizeof(KvPart) + C::ROWS * 4 + C::ROWS * C::D * 4);
}

}  // namespace

namespace {
size_t few_workspace(int head_dim, int num_sms) {
  switch (head_dim) {
    case 64: return workspace_of<Cfg64x2>(num_sms);
    case 128: return workspace_of<Cfg128x2>(num_sms);
    default: return workspace_of<Cfg256x1>(num_sms);
  }
}
// Sequences with more rows (tokens x query heads per key/value head) than this go to the
// many-row kernel.
constexpr int kFewRows = 64;
// The host knows a call's totals, not how its rows are spread.  The many-row kernels are launched
// where the sequences have more than kFewRows on average (one sequence over 16384 cached tokens, 8
// key/value heads: 132 rows 54 us against 74 in the few-row kernel, 68 rows 48 against 49; over 2048
// tokens 32 against 27 and 28 against 23), or where one of them may have many: if each has one token or
// more, none has more rows than its first token's and those above one token each.  Up to kSpreadRows
// of those, the few-row kernel takes the whole call (right for any number of rows, each 16 of
// them decoding the cache anew): the launches cost a call without use for them 11 us (16 sequences of
// 4096 tokens, 40 rows each: 107 against 96 us).  Sequences without rows are taken for ones with a
// token here, since totals do not tell a prompt among empty slots from a batch of single tokens: 256
// tokens over 8192 take 78 us alone or among 64 slots, 246 among 256 (the header says so).
// Single tokens stay in the few-row kernel for any number of query heads: with 128 of them on one
// key/value head, one sequence of 32768 tokens takes 32 us (many-row kernel: 71), 16 of 4096 48 us
// (45); only 64 of 2048 would be better off there (81 against 59 us).
constexpr int64_t kSpreadRows = 512;
bool may_have_many_rows(int64_t tokens, int batch, int group) {
  const int64_t more = (tokens - batch) * group;
  return more > kSpreadRows || (more > 0 && tokens * group > static_cast<int64_t>(kFewRows) * batch);
}
size_t again_bytes(int batch) { return (static_cast<size_t>(batch) * 4 + 15) / 16 * 16; }
}  // namespace

size_t kv_attention_workspace(int head_dim, int group, int batch, int64_t tokens, int num_sms) {
  size_t bytes = (few_workspace(head_dim, num_sms) + 15) / 16 * 16;
  if (may_have_many_rows(tokens, batch, group))
    bytes += again_bytes(batch) + kv_prefill_workspace(head_dim, group, batch, tokens, num_sms);
  return bytes;
}

cudaError_t launch_kv_attention(const qlora_kv_cache &c, const KvBatch &kb, const uint16_t *Q, int q_heads,
                                int64_t q_token_stride, int64_t q_head_stride, float scale, int causal, int window,
                                uint16_t *out, void *ws, const float levels[16], int num_sms,
                                unsigned long long timeout_ns, cudaStream_t st) {
  KvAttnArgs a = {};
  a.kb = kb;
  a.Q = Q;
  a.q_token_stride = q_token_stride;
  a.q_head_stride = q_head_stride;
  a.out = out;
  a.k_codes = c.k_codes;
  a.v_codes = c.v_codes;
  a.k_absmax = c.k_absmax;
  a.v_absmax = c.v_absmax;
  a.heads = c.heads;
  a.group = q_heads / c.heads;
  // Levels are held in fp16 times a unit.  The integer grid and E2M1 are (halves of) small
  // integers at their unit, and exact; so is E3M0.  NF4's levels are rounded, within 2^-11 at any
  // unit; what counts over a long cache, where random errors average out, is the sum of the
  // rounding errors weighted by how often each level is met.  Of two million units in [1, 2) this
  // one leaves the smallest: 2e-6 of the values' root mean square or less for values that are
  // Gaussian, Laplace, uniform, Student's t or have strong channels (unit 1: up to 5e-5, which over
  // 131071 tokens of random signs was an error of 0.003 of the output).
  const float unit = c.codebook == QLORA_CB_NF4        ? 1.458608f
                     : c.codebook == QLORA_CB_INT4     ? 7.0f
                     : c.codebook == QLORA_CB_FP4_E2M1 ? 6.0f
                                                       : 1.0f;
  for (int i = 0; i < 16; ++i) {
    float v = levels[i] * unit;
    if (c.codebook == QLORA_CB_INT4 || c.codebook == QLORA_CB_FP4_E2M1)
      v = static_cast<float>(static_cast<int>(v * 2.0f + (v < 0 ? -0.5f : 0.5f))) * 0.5f;
    a.levels[i] = __float2half_rn(v);
  }
  a.scale_log2 = scale * 1.4426950408889634f / unit;
  a.v_unit = 1.0f / unit;
  a.causal = causal;
  a.window = window;
  a.few_rows = INT_MAX;
  if (may_have_many_rows(kb.tokens, kb.batch, a.group)) {
    a.few_rows = kFewRows;
    uint8_t *more = static_cast<uint8_t *>(ws) + (few_workspace(c.head_dim, num_sms) + 15) / 16 * 16;
    a.again = reinterpret_cast<int32_t *>(more);
    const cudaError_t e =
        launch_kv_prefill(a, c.head_dim, more + again_bytes(kb.batch), num_sms, timeout_ns, st);
    if (e != cudaSuccess) return e;
  }
  // 16-row tiles once a sequence has on average more than 8 rows per key/value head (a
  // tile's rows share the decoding of every key and value)
  const bool wide = static_cast<int64_t>(kb.tokens) * a.group > 8 * static_cast<int64_t>(kb.batch);
  switch (c.head_dim) {
    case 64: return wide ? run_attention<Cfg64x2>(a, ws, num_sms, st) : run_attention<Cfg64x1>(a, ws, num_sms, st);
    case 128: return wide ? run_attention<Cfg128x2>(a, ws, num_sms, st) : run_attention<Cfg128x1>(a, ws, num_sms, st);
    default: return run_attention<Cfg256x1>(a, ws, num_sms, st);
  }
}

}  // namespace qlora
