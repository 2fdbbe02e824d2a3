// kv_prefill.cu — attention over the 4-bit cache for sequences with many query rows
// (prompt chunks): the same definition as kv_attention.cu, on the tensor cores of sm_100a.
//
// An item is one sequence x key/value head x tile of 256 query rows (tokens x the query
// heads of that key/value head; 128 rows with 256 channels), cut into steps of 128 cached
// tokens (64 with 256 channels).  The steps of all items form one line, cut evenly among
// one CTA per SM; parts of items that CTAs share are joined by k_kv_join.
//
// A CTA's roles:
//   warps 0-3, 4-7  softmax of 128 rows each, one row per thread: while one half works on its
//                   scores the tensor cores serve the other
//   warps 8-11      decode the step's keys from codes to fp16 in the 128-byte swizzled operand
//                   layout, once for all 256 rows
//   warp 12         issues the MMAs
//   warps 13-15     decode the step's values
// S = Q K^T (Q and K in shared memory) lands in TMEM; the softmax warps read it, replace it
// in place by fp16 weights, and those are the A operand, from TMEM, of O += P V.
//
// The blocks' constants.  Where the constants of a step lie within a few binades of one
// another (every step of ordinary data) they are multiplied into the fp16 levels, relative to
// one exponent for the step's keys and one for its values.  Where they do not - a constant far
// from the others, a value's that is zero, or one not finite - the step is "wide": each token's keys have an exponent of
// their own that multiplies its scores, the values stay levels, and their constants multiply
// the weights, one set of weights and one product per block of 64 channels.  So a value that a
// row does not see can be of any size, or NaN, and leaves the row as it is.
//
// Numbers.  As in kv_attention.cu: levels and weights in fp16 (2^-11 each), everything else
// float32; and one more rounding of level x constant to fp16 (2^-11) for NF4.  A row's
// weights are 2^(s - r), r renewed when one passes 2^14: the largest then weighs 2^6, and what
// is 2^-31 of it vanishes (its value can be 2^8 times another's of the step: 2^-23).
// The weights carry their step's exponent, and so does their sum, which is brought to the
// row's maximum before it is added: where a step's values are so small beside what the row has
// seen that the sum would lose terms (kFar), the sequence is marked in `again`, and the few-row kernel,
// launched behind this one, whose sums know nothing of the values, computes it anew.  So is one where a
// block's largest contribution to a row weighs less than 2^kLeast, because another block's or a token
// whose values are zero set the row's only reference: the few-row kernel has one per block.  And so is one with
// a key whose blocks lie more than 2^kNearBlocks apart: there, constants multiply float32 sums.  (Marked for
// one block of 2^31, 4096 over 8192 takes 4.4 ms in place of 0.57.)
//
// Measured (4096 tokens x 4 query heads over 8192 cached, 8 key/value heads of 128): 0.58 ms,
// 715 TFLOP/s of the visible pairs (0.55 without the guards of sums and references, which the
// compiler schedules some 3 % worse; folding them into other steps changed nothing).  A step takes 5700
// clocks, of which the tensor cores work 2100: no unit is near its limit (three chunks of 1400 tokens
// together: issue slots 39 %, tensor pipe 28 %, ex2 unit 29 % busy), it is bound by the chain from one
// step of a row tile to the next (softmax, the two products and their hand-overs) and by the decoding of
// the values between two products that use them (2400).  An item starts and ends in 15000 clocks
// (queries, first keys, outputs), the kernel in 10000.  With heads of 256 (68 bytes of registers
// spilled a thread), 2048 tokens x 4 query heads over 4096, 4 key/value heads, take 0.26 ms.  Tried without gain: values in two stages (more decoding next to the softmax slows it as
// much), scores in two halves (products of 64 columns), 20 warps, two passes of the softmax between
// checks (spills, and with shared memory full a spilled register is a second-level cache access),
// outputs turned through shared memory (the stores are faster, the steps slower).
#include <atomic>
#include <cstdint>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include "internal.h"
#include "kv_attention.cuh"
#include "kv_common.cuh"
#include "launch.cuh"
#include "ptx.cuh"

namespace qlora {
namespace {

template <int D_>
struct PreCfg {
  static constexpr int D = D_;
  static constexpr int NB = D / 64;               // blocks of 64 channels
  static constexpr int MT = D == 256 ? 1 : 2;     // tiles of 128 rows
  static constexpr int ROWS = 128 * MT;
  static constexpr int N = D == 256 ? 64 : 128;   // cached tokens of a step
  static constexpr int TW = N / 4;                // tokens of one decoding warp = columns of one softmax pass
  static constexpr int Q_BYTES = 128 * D * 2;     // one row tile
  static constexpr int KV_BYTES = N * D * 2;
  static constexpr int P_COL = D == 256 ? 64 : 0; // where the weights go, from the scores' first column
  static constexpr int SP_COLS = D == 256 ? 192 : 128;
  static constexpr int O_COL = MT * SP_COLS;
  static constexpr int TMEM_COLS = 512;
  static constexpr int THREADS = 16 * 32;
  // registers of a thread: softmax and the others; together what the CTA starts with
  static constexpr int REGS_SOFTMAX = 136, REGS_OTHERS = 120;
  static_assert(256 * REGS_SOFTMAX + 256 * REGS_OTHERS == 128 * THREADS, "register split");
  static constexpr int BARS = 19;
  static constexpr int MISC_FLOATS = 2 * N + 2 * NB * N;
  static constexpr int MISC_BYTES = MISC_FLOATS * 4 + 4 * 8 + 2 * 7 * 8 + BARS * 8 + 48;
  static constexpr int SMEM_BYTES = 0x20000 + KV_BYTES + MT * Q_BYTES + ROWS * NB * 4;
  static_assert(SMEM_BYTES <= 227 * 1024, "shared memory of one CTA");
  static_assert(O_COL + MT * D <= TMEM_COLS, "TMEM columns");
};

// Binades between the largest and the smallest constant of a step up to which they are folded
// into the fp16 operands: keys keep all their bits (fp16 has 25 binades below 2^12), and a
// weight that vanishes in fp16 (2^-31 of the largest) can have a value 2^8 times another's.
constexpr int kNearKeys = 12, kNearValues = 8;
// Binades between the blocks of one key up to which the smaller ones keep their bits in fp16 (the largest is
// held below 2^12, levels are 2^-7 of it or more).
constexpr int kNearBlocks = 16;
// What starting and ending an item costs a CTA, in steps: part of its place on the line.
constexpr int kItemOverhead = 2;  // three chunks, 1400 tokens together: 152, 146, 148, 146 us with 1, 2, 3, 4
// Binades between the unit of a step's sum and the row's largest weight: of 126 in float32, so that what is
// lost is 2^-62 of that weight or less.  Ordinary steps stay below 10.
constexpr float kFar = 64.0f;
constexpr float kMostTotal = 0x1p120f;  // a row's sum past this may have overflowed
// A block's largest contribution must weigh at least 2^kLeast: what vanishes beside it is then 2^-23 of it.
constexpr float kLeast = -2.0f;
constexpr float kSeen = -1.0e38f;  // a contribution of unknown size
constexpr unsigned long long kDrainNs = 1000000000ull;  // bound on the wait for the MMAs in flight at the end

// How a step's keys and values were written (by the decoding warps, for the others).  Where
// the constants of a step lie close together they are folded into the fp16 operands; where
// they do not (wide) they multiply the scores (cs) and the weights (cv), token by token.
struct StepInfo {
  float scale;  // keys: factor of the scores; values: the exponent that constants are relative to
  int wide;
};
struct KvEntry {  // a row tile of a sequence; its heads follow one another on the line
  int b, tile;
  int lo;     // first cached token of its first step
  int steps;  // at least 1
};

struct PrefillArgs {
  KvAttnArgs a;
  KvEntry *entries;
  int64_t *prefix;  // [entries + 1]: where each entry's steps start on the line
  int *count;       // entries
  int max_entries;  // room for them
  unsigned long long timeout_ns;
};

// Instruction descriptor, kind::f16: float32 accumulator, fp16 A and B.
constexpr uint32_t idesc_f16(int m, int n, bool b_mn_major) {
  return (1u << 4) | ((b_mn_major ? 1u : 0u) << 16) | (static_cast<uint32_t>(n >> 3) << 17) |
         (static_cast<uint32_t>(m >> 4) << 24);
}

// ---------------------------------------------------------------- the line of steps
// One CTA lists the row tiles of the sequences that have many rows.
constexpr int kPlanThreads = 1024;
template <class C>
__global__ void __launch_bounds__(kPlanThreads) k_kv_plan(const __grid_constant__ PrefillArgs p) {
  __shared__ int s_off[QLORA_KV_MAX_BATCH + 1];
  __shared__ int64_t s_sum[kPlanThreads / 32];
  const KvAttnArgs &a = p.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_wait();
  pdl_launch_dependents();
  // inclusive scan of one value per thread over the CTA
  auto scan = [&](int64_t v) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t y = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += y;
    }
    __syncthreads();  // s_sum is free
    if (lane == 31) s_sum[warp] = v;
    __syncthreads();
    for (int w = 0; w < warp; ++w) v += s_sum[w];
    return v;
  };
  const int run = (a.kb.batch + kPlanThreads - 1) / kPlanThreads;
  const int b0 = min(a.kb.batch, tid * run), b1 = min(a.kb.batch, b0 + run);
  int tiles[QLORA_KV_MAX_BATCH / kPlanThreads];
  int64_t sum = 0;
#pragma unroll
  for (int i = 0; i < QLORA_KV_MAX_BATCH / kPlanThreads; ++i) {
    tiles[i] = 0;
    if (b0 + i < b1) {
      a.again[b0 + i] = 0;
      const int rows = kv_seq(a.kb, b0 + i).n * a.group;
      if (rows > a.few_rows) tiles[i] = (rows + C::ROWS - 1) / C::ROWS;
    }
    sum += tiles[i];
  }
  const int64_t incl = scan(sum);
  // (sequences that share rows, an error, may list any number: held below what an int holds)
  constexpr int64_t kMost = 1 << 30;
  int off = static_cast<int>(min(incl - sum, kMost));
#pragma unroll
  for (int i = 0; i < QLORA_KV_MAX_BATCH / kPlanThreads; ++i) {
    if (b0 + i < b1) s_off[b0 + i] = off;
    off += tiles[i];
  }
  if (tid == kPlanThreads - 1) s_off[a.kb.batch] = static_cast<int>(min(incl, kMost));
  __syncthreads();
  // ... and more than there is room for
  const int count = min(s_off[a.kb.batch], p.max_entries);
  if (count < s_off[a.kb.batch] && tid == 0) kv_error(a.kb);
  int64_t carry = 0;
  for (int base = 0; base < count; base += kPlanThreads) {
    const int e = base + tid;
    int64_t units = 0;
    if (e < count) {
      int lo = 0, hi = a.kb.batch;  // last b with s_off[b] <= e: the one with tiles among equals
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_off[mid] <= e) lo = mid;
        else hi = mid;
      }
      const KvSeq q = kv_seq(a.kb, lo);
      KvEntry t;
      t.b = lo;
      t.tile = e - s_off[lo];
      const int i0 = t.tile * C::ROWS / a.group;
      const int i1 = min(q.n - 1, (t.tile * C::ROWS + C::ROWS - 1) / a.group);
      const int see = a.causal ? min(q.len, q.pos0() + i1 + 1) : q.len;
      t.lo = a.window > 0 ? max(0, min(q.len, q.pos0() + i0 - a.window + 1)) & ~31 : 0;
      t.steps = max(1, (see - t.lo + C::N - 1) / C::N);
      p.entries[e] = t;
      units = static_cast<int64_t>(t.steps + kItemOverhead) * a.heads;
    }
    const int64_t upto = scan(units);
    if (e < count) p.prefix[e] = carry + upto - units;
    __syncthreads();
    for (int w = 0; w < kPlanThreads / 32; ++w) carry += s_sum[w];
  }
  if (tid == 0) {
    p.prefix[count] = carry;
    *p.count = count;
  }
}

// ---------------------------------------------------------------- a worker's part of an item
struct Segment {
  int b, head, tile;
  KvSeq q;
  int lo;            // first cached token of step 0
  int step0, step1;  // its steps
  int rows;          // rows of the tile that exist (at most ROWS: the second half stays idle with one row tile)
  bool whole;        // the item is this worker's alone
  int slot;
  int used;          // of the line
  int64_t first, end, at;  // the item's place on the line, and where this part begins
};

// This worker's parts, in order.  A role keeps two integers between its parts, and reads
// and computes the rest again when it needs it: state kept through the steps would be
// spilled, and with all of shared memory in use a spilled value is a second-level cache
// access away.
template <class C>
__device__ __forceinline__ bool next_part(const PrefillArgs &p, const volatile int64_t *my_line, int &e, int done, Segment &s) {
  const int64_t begin = my_line[0], stop = my_line[1], at = begin + done;  // done: of the line
  if (at >= stop) return false;
  KvEntry t = p.entries[e];
  int64_t base = p.prefix[e], after = p.prefix[e + 1];
  while (at >= after) {
    ++e;
    t = p.entries[e];
    base = after;
    after = p.prefix[e + 1];
  }
  const int64_t rel = at - base;
  s.b = t.b;
  s.tile = t.tile;
  s.lo = t.lo;
  const int units = t.steps + kItemOverhead;
  s.head = static_cast<int>(rel / units);
  s.first = base + static_cast<int64_t>(s.head) * units;
  s.end = s.first + units;
  s.step0 = max(0, static_cast<int>(at - s.first) - kItemOverhead);
  s.step1 = (stop < s.end ? static_cast<int>(stop - s.first) : units) - kItemOverhead;
  if (s.step1 <= s.step0) return false;  // the range ends before the item's first step
  s.used = static_cast<int>(s.first + kItemOverhead + s.step1 - at);
  s.whole = s.step0 == 0 && s.step1 == t.steps;
  s.slot = at == begin ? 0 : 1;
  s.at = at;
  s.q = kv_seq(p.a.kb, s.b);
  s.rows = min(s.q.n * p.a.group - s.tile * C::ROWS, C::ROWS);
  return true;
}

// MMAs and commits by one elected lane of a converged warp (always the same one).
__device__ __forceinline__ void mma_f16_ss(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
      "l"(ad), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void mma_f16_ts(uint32_t d, uint32_t at, uint64_t bd, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
      "r"(at), "l"(bd), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void commit(uint64_t *bar) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xFFFFFFFF;\n\t"
      "@e tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(smem_u32(bar))
      : "memory");
}
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const uint32_t (&v)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(v[0]),
               "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7])
               : "memory");
}
// Two float32 in one 64-bit register, and the paired arithmetic of sm_100.
__device__ __forceinline__ uint64_t pair_bits(uint32_t lo, uint32_t hi) {
  uint64_t d;
  asm("mov.b64 %0, {%1, %2};" : "=l"(d) : "r"(lo), "r"(hi));
  return d;
}
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return pair_bits(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ float low(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x)); }
__device__ __forceinline__ float high(uint64_t x) { return __uint_as_float(static_cast<uint32_t>(x >> 32)); }
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ void st_global_v8(float *p, const float *f) {  // 32-byte aligned
  asm volatile("st.global.v8.f32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "f"(f[0]), "f"(f[1]), "f"(f[2]),
               "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7])
               : "memory");
}
__device__ __forceinline__ float pow2(int e) { return __uint_as_float(static_cast<uint32_t>(127 + e) << 23); }
__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&w)[4]) { ld_shared_v4(addr, w[0], w[1], w[2], w[3]); }

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1) k_kv_prefill(const __grid_constant__ PrefillArgs p) {
  constexpr int D = C::D, NB = C::NB, N = C::N, TW = C::TW, MT = C::MT;
  extern __shared__ __align__(1024) uint8_t smem[];
  const KvAttnArgs &a = p.a;
  const uint32_t smem_base = smem_u32(smem);
  const uint32_t table = (smem_base + 0xFFFFu) & ~0xFFFFu;  // 64 KiB at a multiple of 64 KiB
  // before the table: keys, constants, barriers; in its gaps (the upper half of each 256
  // bytes): two stages of codes; after it: values, queries and [NB][ROWS] each row's largest
  // contribution to each block in wide steps, as a logarithm
  const uint32_t k_smem = (smem_base + 1023u) & ~1023u;
  const uint32_t v_smem = table + 0x10000u, q_smem = v_smem + C::KV_BYTES;
  float *largest = reinterpret_cast<float *>(smem + (q_smem - smem_base) + MT * C::Q_BYTES);
  float *cs = reinterpret_cast<float *>(smem + (k_smem - smem_base) + C::KV_BYTES);  // [2][N] score factors
  float *cv = cs + 2 * N;                                                            // [2][NB][N] value constants
  StepInfo *kinfo = reinterpret_cast<StepInfo *>(cv + 2 * NB * N), *vinfo = kinfo + 2;  // [2] each
  int2 *ranges = reinterpret_cast<int2 *>(vinfo + 2);                                // [2][7] of the decoding warps
  uint64_t *bars = reinterpret_cast<uint64_t *>(ranges + 14);
  uint64_t *kfull = bars, *kempty = bars + 1, *vfull = bars + 2, *vempty = bars + 3, *cfull = bars + 4,
           *sfull = bars + 6, *pfull = bars + 8, *opv = bars + 10, *qfull = bars + 12, *drain = bars + 14, *krange = bars + 15, *vrange = bars + 17;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::BARS);
  volatile int *abort_flag = reinterpret_cast<volatile int *>(tmem_slot + 1);
  int *s_entry = reinterpret_cast<int *>(tmem_slot + 2);
  volatile int64_t *my_line = reinterpret_cast<int64_t *>(tmem_slot + 4);  // this worker's steps on the line

  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  if (table - smem_base < C::KV_BYTES + 1024 + C::MISC_BYTES) {  // cannot happen while shared memory starts low
    pdl_wait();
    if (tid < 2) p.a.parts[blockIdx.x * 2 + tid].joins = 0;
    kv_error(a.kb);
    return;
  }
  if (tid == 0) {
    mbar_init(kfull, 4);
    mbar_init(kempty, 1);
    mbar_init(vfull, 3);
    mbar_init(vempty, 1);
    mbar_init(drain, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&cfull[i], 7);
      mbar_init(&krange[i], 4);
      mbar_init(&vrange[i], 3);
      mbar_init(&sfull[i], 1);
      mbar_init(&pfull[i], 4);
      mbar_init(&opv[i], 1);
      mbar_init(&qfull[i], 4);
    }
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 12) {
    tmem_alloc(tmem_slot, C::TMEM_COLS);
    tmem_relinquish();
  }
  for (int i = tid; i < 256 * 32; i += C::THREADS) {
    const int byte = i >> 5;
    const __half2 h = __halves2half2(a.levels[byte >> 4], a.levels[byte & 15]);
    *reinterpret_cast<__half2 *>(smem + (table - smem_base) + byte * 256 + (i & 31) * 4) = h;
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == 0) {  // the entry that holds this worker's first step: 32 probes at a time
    const int count = *p.count;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * p.prefix[count] / gridDim.x;
    int lo = 0, hi = count;
    while (hi - lo > 1) {
      const int stride = (hi - lo + 31) / 32;
      const int probe = lo + lane * stride;
      const unsigned below = __ballot_sync(0xFFFFFFFFu, probe < hi && p.prefix[min(probe, hi - 1)] <= at);
      const int last = 31 - __clz(static_cast<int>(below));  // lane 0's probe is lo, at or below `at`
      const int nlo = lo + last * stride;
      hi = min(hi, nlo + stride);
      lo = nlo;
    }
    if (lane == 0) {
      *s_entry = lo;
      my_line[0] = at;
      my_line[1] = static_cast<int64_t>(blockIdx.x + 1) * p.prefix[count] / gridDim.x;
    }
  }
  if (tid == 0)
    for (int i = 0; i < 2; ++i) {
      a.parts[blockIdx.x * 2 + i].present = 0;
      a.parts[blockIdx.x * 2 + i].joins = 0;
    }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xFFFFFFFFu, *tmem_slot, 0);
  int entry = *s_entry, done_steps = 0;  // where this role is on the line
  auto wait = [&](uint64_t *bar, uint32_t parity) {
    return mbar_wait_bounded(bar, parity, abort_flag, a.kb.dev_err, p.timeout_ns);
  };

  if (warp < 8) {
    regs_inc<C::REGS_SOFTMAX>();
    // ================================================================ softmax: one row per thread
    const int m = warp >> 2;
    const int r = tid & 127;
    const uint32_t lanes = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_tmem = lanes + m * C::SP_COLS, p_tmem = s_tmem + C::P_COL, o_tmem = lanes + C::O_COL + m * D;
    uint32_t steps_done = 0;  // of this row tile
    uint32_t all_steps = 0;   // of the CTA
    bool ok = true;
    while (ok) {
      int nsteps, tok0, see_lo, see_hi;
      float qs = 0.0f;
      {
      Segment sg;
      if (!next_part<C>(p, my_line, entry, done_steps, sg)) break;
      nsteps = sg.step1 - sg.step0;
      if (m * 128 >= sg.rows) {  // no row in this half
        all_steps += nsteps;
        done_steps += sg.used;
        continue;
      }
      // ---- the query row: scaled to fp16, into the swizzled operand
      const int row = m * 128 + r;
      const bool live = row < sg.rows;
      const int rr = sg.tile * C::ROWS + row;
      const int tok = live ? rr / a.group : 0, h = live ? rr - tok * a.group : 0;
      {
        // A warp reads its 32 rows four at a time, 128 bytes of each by eight lanes (a row per lane
        // touches 32 lines with every load: 6000-10000 clocks against 4000-6000).
        const int64_t from = static_cast<int64_t>(sg.q.row0 + tok) * a.q_token_stride +
                             static_cast<int64_t>(sg.head * a.group + h) * a.q_head_stride;
        const unsigned there = __ballot_sync(0xFFFFFFFFu, live);
        constexpr int BATCH = NB == 4 ? 4 : 8;  // loads in flight: of this many rows
        auto exponent_of = [](uint32_t mag) {     // largest magnitude in [2^13, 2^14)
          const int x = mag == 0 || mag >= 0x7F80u ? 0 : static_cast<int>(mag >> 7) - 127 - 13;
          return max(x, -120);
        };
        uint32_t mag = 0;
#pragma unroll 1
        for (int g0 = 0; g0 < 8; g0 += BATCH) {
          uint4 raw[BATCH][NB];
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int x = (g0 + i) * 4 + (lane >> 3);
            const uint16_t *src = a.Q + __shfl_sync(0xFFFFFFFFu, from, x) + (lane & 7) * 8;
#pragma unroll
            for (int k = 0; k < NB; ++k)
              raw[i][k] = there >> x & 1 ? __ldg(reinterpret_cast<const uint4 *>(src + 64 * k)) : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int i = 0; i < BATCH; ++i) {
            const int x = (g0 + i) * 4 + (lane >> 3);
            uint32_t most = 0;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              most = __vmaxu2(__vmaxu2(most, raw[i][k].x & 0x7FFF7FFFu), raw[i][k].y & 0x7FFF7FFFu);
              most = __vmaxu2(__vmaxu2(most, raw[i][k].z & 0x7FFF7FFFu), raw[i][k].w & 0x7FFF7FFFu);
            }
            most = max(most >> 16, most & 0xFFFFu);
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
            most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 4));
            const float down = pow2(-exponent_of(most));
            const uint32_t dst = q_smem + m * C::Q_BYTES + ((warp & 3) * 32 + x) * 128 + (((lane & 7) ^ (x & 7)) << 4);
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              const uint32_t in[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
              uint32_t o[4];
#pragma unroll
              for (int y = 0; y < 4; ++y)
                o[y] = pack_half2(__uint_as_float(in[y] << 16) * down, __uint_as_float(in[y] & 0xFFFF0000u) * down);
              st_shared_v4(dst + k * 16384, o[0], o[1], o[2], o[3]);
            }
            const uint32_t of_row = __shfl_sync(0xFFFFFFFFu, most, (lane & 3) * 8);  // of row 4 (g0 + i) + lane % 4
            if (lane >> 2 == g0 + i) mag = of_row;
          }
        }
        const int e = exponent_of(mag);
        qs = pow2(e) * a.scale_log2;
        if (mag >= 0x7F80u) qs = __uint_as_float(0x7FC00000u);  // a non-finite query: its row is NaN throughout
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&qfull[m]);
      }
      const int pos = sg.q.pos0() + tok;
      see_hi = !live ? 0x7FFFFFFF : a.causal ? min(sg.q.len, pos + 1) : sg.q.len;
      see_lo = live && a.window > 0 ? max(0, pos - a.window + 1) : 0;
      tok0 = sg.lo + sg.step0 * N;
      }

      float ref = kFloor, mx = kFloor, rv = kFloor, l = 0.0f, far = kFloor;
      float folded = kFloor;  // largest contribution in steps that are not wide, when last renewed
      bool apart = false;     // there was a wide step
      for (int step = 0; step < nsteps; ++step, ++steps_done, ++all_steps, tok0 += N) {
        const int st = all_steps & 1;
        // The scores first: while this half sat out items, phases of cfull passed that it did not wait
        // for, and a parity alone does not tell them apart.  With this step's scores there, the phase
        // of two steps ago is over (the products of its values were issued before them).
        ok = wait(&sfull[m], steps_done & 1) && wait(&cfull[st], (all_steps >> 1) & 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const bool hide = __any_sync(0xFFFFFFFFu, tok0 < see_lo || tok0 + N > see_hi);
        const StepInfo hk = kinfo[st], hv = vinfo[st];
        const bool kwide = hk.wide != 0, vwide = hv.wide != 0;
        const float e_c = hv.scale;
        const float *csr = cs + st * N, *cvr = cv + st * NB * N;
        const float factor = hk.scale * qs;
        auto unit_of_sums = [&] { return ref - e_c - mx; };  // in binades above the row's maximum
        far = fmaxf(far, unit_of_sums());
        if (!vwide) {
          if (tok0 < see_hi && tok0 + N > see_lo) folded = fmaxf(folded, kSeen);
        } else if (!apart) {
          apart = true;
#pragma unroll
          for (int k = 0; k < NB; ++k) largest[k * C::ROWS + m * 128 + r] = kFloor;
        }
        // The usual pass over TW columns: v holds their products, w receives the weights; two
        // columns per instruction where there is a paired one.  With `masked` the columns that the row
        // does not see weigh nothing (their constants, folded into the operands, are finite).
        const uint32_t sees = static_cast<uint32_t>(max(see_hi - see_lo, 0));
        auto seen = [&](int c, int j) { return static_cast<uint32_t>(tok0 + c * TW + j - see_lo) < sees; };
        auto plain = [&](const bool masked, int c, const uint32_t (&v)[TW], uint32_t (&w)[TW / 2], float &sum) -> bool {
          auto shown = [&](float x, int j) { return !masked || seen(c, j) ? x : -INFINITY; };
          const uint64_t f2 = pair(factor, factor), shift2 = pair(e_c - ref, e_c - ref);
          uint64_t total0 = 0, total1 = 0;
          __half2 most = __float2half2_rn(0.0f);
#pragma unroll
          for (int j = 0; j < TW; j += 4) {
            const uint64_t x0 = fma2(pair_bits(v[j], v[j + 1]), f2, shift2);
            const uint64_t x1 = fma2(pair_bits(v[j + 2], v[j + 3]), f2, shift2);
            const float p0 = ex2(shown(low(x0), j)), p1 = ex2(shown(high(x0), j + 1)), p2 = ex2(shown(low(x1), j + 2)),
                        p3 = ex2(shown(high(x1), j + 3));
            total0 = add2(total0, pair(p0, p1));
            total1 = add2(total1, pair(p2, p3));
            w[j / 2] = pack_half2(p0, p1);
            w[j / 2 + 1] = pack_half2(p2, p3);
            most = __hmax2(most, __hmax2(*reinterpret_cast<const __half2 *>(&w[j / 2]),
                                         *reinterpret_cast<const __half2 *>(&w[j / 2 + 1])));
          }
          total0 = add2(total0, total1);
          sum = low(total0) + high(total0);
          return __low2float(most) > kMostWeight || __high2float(most) > kMostWeight;
        };
        // The reference moves: to the largest score and the largest contribution so far, with `top` and
        // `big` of this pass (an earlier step's score says nothing of contributions in this step's
        // exponent).  What was accumulated, and weighed in the passes of this step before this one, follows.
        auto renew = [&](int c, float top, float big) {
          rv = fmaxf(rv, big);
          if (!vwide) folded = fmaxf(folded, big);
          const float next = ceilf(fmaxf(rv - kLift, top + e_c - 100.0f));
          const float f = next > ref ? ex2(ref - next) : 1.0f;  // a power of two
          ref = fmaxf(ref, next);
          const float highest = fmaxf(mx, top);
          l *= ex2(mx - highest);
          mx = highest;
          far = fmaxf(far, unit_of_sums());
          tmem_st_wait();
          auto rescale = [&](uint32_t from, int cols, auto scale) {
#pragma unroll 1
            for (int k = 0; k < cols; k += 16) {
              uint32_t o[16];
              tmem_ld16(from + k, o);
              tmem_ld_wait();
#pragma unroll
              for (int j = 0; j < 16; ++j) o[j] = scale(o[j]);
              tmem_st16(from + k, o);
            }
          };
          if (step > 0)
            rescale(o_tmem, D, [&](uint32_t x) { return __float_as_uint(__uint_as_float(x) * f); });
          // the weights of the passes before this one (and whatever else those columns hold)
          // (by two factors: below 2^-24 one would be 0 in fp16, with weights of 2^14 before it)
          const __half2 f2 = __float2half2_rn(fmaxf(f, 0x1p-24f)), rest = __float2half2_rn(f < 0x1p-24f ? f * 0x1p24f : 1.0f);
          rescale(p_tmem, c * 32, [&](uint32_t x) {
            const __half2 y = __hmul2(__hmul2(*reinterpret_cast<__half2 *>(&x), f2), rest);
            return *reinterpret_cast<const uint32_t *>(&y);
          });
          tmem_st_wait();
        };
        // A pass where constants multiply the scores or the weights: three times the usual one's time.
        // (Three chunks, 1400 tokens together, took 176 us when masked steps went through it as well.)
        auto careful = [&](int c, const uint32_t (&v)[TW], uint32_t (&w)[NB * TW / 2], float &sum) {
          float s[TW];
          float top = -INFINITY, big = -INFINITY;
          float block_most[NB];
#pragma unroll
          for (int j = 0; j < TW; ++j) {
            const int t = tok0 + c * TW + j;
            s[j] = __uint_as_float(v[j]) * (kwide ? csr[c * TW + j] : hk.scale) * qs;
            if (t >= see_hi || t < see_lo) s[j] = -INFINITY;
          }
#pragma unroll 1
          for (int pass = 0; pass < 2; ++pass) {
            sum = 0.0f;
#pragma unroll
            for (int k = 0; k < NB; ++k) block_most[k] = 0.0f;
#pragma unroll
            for (int j = 0; j < TW; j += 2) {
              const float p0 = ex2(s[j] - (ref - e_c)), p1 = ex2(s[j + 1] - (ref - e_c));
              sum += p0 + p1;
#pragma unroll
              for (int k = 0; k < NB; ++k) {
                if (k > 0 && !vwide) continue;
                const float c0 = vwide ? cvr[k * N + c * TW + j] : 1.0f, c1 = vwide ? cvr[k * N + c * TW + j + 1] : 1.0f;
                // a token that a row does not see adds nothing, whatever its value's constant; one that it
                // sees is zero in block_most only if the constant is
                const float w0 = s[j] == -INFINITY ? 0.0f : (p0 + 0x1p-120f) * c0,
                            w1 = s[j + 1] == -INFINITY ? 0.0f : (p1 + 0x1p-120f) * c1;
                block_most[k] = fmaxf(block_most[k], fmaxf(w0, w1));
                w[k * (TW / 2) + j / 2] = pack_half2(w0, w1);
              }
            }
            float most = block_most[0];
#pragma unroll
            for (int k = 1; k < NB; ++k) most = fmaxf(most, block_most[k]);
            if (pass == 1 || !__any_sync(0xFFFFFFFFu, most > kMostWeight || sum > kMostSum)) break;
#pragma unroll
            for (int j = 0; j < TW; ++j) {
              top = fmaxf(top, s[j]);
              if (!vwide) continue;
#pragma unroll
              for (int k = 0; k < NB; ++k) big = fmaxf(big, s[j] + lg2(cvr[k * N + c * TW + j]) + e_c);
            }
            if (!vwide) big = top + e_c;
            renew(c, top, big);
          }
          if (vwide) {
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              float &mine = largest[k * C::ROWS + m * 128 + r];
              mine = fmaxf(mine, ref + lg2(block_most[k]));
            }
          }
        };
#pragma unroll 1
        for (int c = 0; c < 4; ++c) {
          uint32_t v[TW], w[NB * TW / 2];
          float sum;
          if constexpr (TW == 32) tmem_ld32(s_tmem + c * TW, v);
          else tmem_ld16(s_tmem + c * TW, v);
          tmem_ld_wait();
          auto &usual = reinterpret_cast<uint32_t(&)[TW / 2]>(w);
          if (kwide || vwide) {
            careful(c, v, w, sum);
          } else if (__any_sync(0xFFFFFFFFu, hide ? plain(true, c, v, usual, sum) : plain(false, c, v, usual, sum))) {
            float most = -INFINITY;
#pragma unroll
            for (int j = 0; j < TW; ++j)
              if (!hide || seen(c, j)) most = fmaxf(most, __uint_as_float(v[j]));
            most *= factor;
            renew(c, most, most + e_c);
            plain(true, c, v, usual, sum);
          }
          l = fmaf(sum, ex2(unit_of_sums()), l);
          const uint32_t to = p_tmem + c * 32;  // over the scores just read, or apart from them
          if (!vwide) {
            if constexpr (TW == 32) tmem_st16(to, reinterpret_cast<const uint32_t(&)[16]>(w));
            else tmem_st8(to, reinterpret_cast<const uint32_t(&)[8]>(w));
          } else {
            if constexpr (NB == 1) tmem_st16(to, w);
            else tmem_st32(to, w);
          }
        }
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&pfull[m]);
      }
      if (!ok) break;
      // ---- the outputs of this part of the item
      ok = wait(&opv[m], (steps_done - 1) & 1);
      if (!__all_sync(0xFFFFFFFFu, ok)) {
        ok = false;
        break;
      }
      tc_fence_after();
      Segment sg;
      next_part<C>(p, my_line, entry, done_steps, sg);
      done_steps += sg.used;
      const int row = m * 128 + r, rr = sg.tile * C::ROWS + row;
      const bool live = row < sg.rows;
      const int tok = live ? rr / a.group : 0, h = live ? rr - tok * a.group : 0;
      bool lost = far > kFar || l > kMostTotal;
      if (apart && l > 0.0f) {
        // What a step that is not wide contributes reaches every block, within 2^kNearValues; it is enough where the
        // reference is its own (the largest then weighs 2^(kLift - 1) or more).
#pragma unroll
        for (int k = 0; k < NB; ++k) {
          const float top = fmaxf(largest[k * C::ROWS + row], folded - (kLift - 1.0f - kLeast));
          lost |= top > kFloor && top - ref < kLeast;
        }
      }
      if (live && lost) a.again[sg.b] = 1;
      const bool any = l > 0.0f || l != l;
      const float half_unit = ex2(0.5f * (ref - mx));  // applied twice: it may pass float32's exponents
      const float inv = any ? a.v_unit / l * half_unit : 0.0f;
      const int64_t part = static_cast<int64_t>(blockIdx.x) * 2 + sg.slot;
      uint16_t *dst = a.out + ((static_cast<int64_t>(sg.q.row0 + tok) * a.heads + sg.head) * a.group + h) * D;
      float *dst_part = a.part_o + (part * C::ROWS + row) * D;
#pragma unroll 1
      for (int k = 0; k < D; k += 32) {
        uint32_t v[32];
        tmem_ld32(o_tmem + k, v);
        tmem_ld_wait();
        if (live) {
          float f[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) f[j] = __uint_as_float(v[j]) * inv * half_unit;
          if (sg.whole) {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              *reinterpret_cast<uint4 *>(dst + k + j) =
                  make_uint4(pack_bf16x2(f[j], f[j + 1]), pack_bf16x2(f[j + 2], f[j + 3]),
                             pack_bf16x2(f[j + 4], f[j + 5]), pack_bf16x2(f[j + 6], f[j + 7]));
          } else {
#pragma unroll
            for (int j = 0; j < 32; j += 8)
              st_global_v8(dst_part + k + j, f + j);  // whole sectors
          }
        }
      }
      tc_fence_before();
      if (!sg.whole) {
        if (live) a.part_lse[part * C::ROWS + row] = any ? mx + lg2(l) : -INFINITY;
        if (tid == 0) {
          const int64_t total = p.prefix[*p.count];
          const int64_t workers = gridDim.x;
          // the worker that holds step u is the largest g with g * total / workers <= u
          auto worker_of = [&](int64_t u) { return static_cast<int>(((u + 1) * workers - 1) / total); };
          KvPart kp;
          kp.present = 1;
          kp.row0 = sg.q.row0;
          kp.head = sg.head;
          kp.tile = sg.tile;
          kp.rows = sg.rows;
          kp.g0 = worker_of(sg.first + kItemOverhead);  // holds the item's first step
          kp.last = worker_of(sg.end - 1);
          kp.head_slot = kp.g0 * total / workers >= sg.first ? 0 : 1;
          kp.joins = sg.step0 > 0 && sg.at == (kp.g0 + 1) * total / workers ? 1 : 0;
          a.parts[part] = kp;
        }
      }
    }
  } else {
    regs_dec<C::REGS_OTHERS>();
    if (warp != 12) {
    // ================================================================ decoding: codes -> fp16 operands
    // Four warps for the keys, three for the values.  A unit is a tile of 16 tokens (inside one
    // page): two lanes per token.
    const bool keys = warp < 12;
    const int dw = keys ? warp - 8 : warp - 13, warps = keys ? 4 : 3;
    constexpr int TILES = N / 16, MINE = (TILES + 2) / 3;  // tiles dw, dw + warps, ...: at most MINE
    constexpr int PASSES = D / 64;                         // 16-byte pieces of codes per lane and tile
    const int sub = lane & 1, tok = lane >> 1;
    const uint32_t tab = table | (lane * 4);
    const uint8_t *codes = keys ? a.k_codes : a.v_codes;
    const uint16_t *absmax = keys ? a.k_absmax : a.v_absmax;
    uint64_t *full = keys ? kfull : vfull, *empty = keys ? kempty : vempty, *range = keys ? krange : vrange;
    const uint32_t operand = keys ? k_smem : v_smem;
    int2 *my_ranges = ranges + (keys ? 0 : 4);
    const int near = keys ? kNearKeys : kNearValues;
    // raw codes, in the table's gaps: 128 bytes of every 256
    auto gap = [&](int stage, int off) {
      return table + 128u + static_cast<uint32_t>(stage) * 32768u + (keys ? 0u : 16384u) +
             static_cast<uint32_t>((off >> 7) * 256 + (off & 127));
    };
    uint32_t n = 0;  // steps of the CTA so far
    bool ok = true;
    while (ok) {
      int b, lo, nsteps, head, len;
      const int32_t *pages;
      {
        Segment sg;
        if (!next_part<C>(p, my_line, entry, done_steps, sg)) break;
        b = sg.b;
        nsteps = sg.step1 - sg.step0;
        lo = sg.lo + sg.step0 * N;
        head = sg.head;
        len = sg.q.len;
        pages = a.kb.page_table + static_cast<int64_t>(sg.b) * a.kb.max_pages;
        done_steps += sg.used;
      }
      bool bad_page = false;
      auto tile_of = [&](int i) { return dw + i * warps; };
      auto load_pages = [&](int step, int (&page)[MINE]) {
#pragma unroll
        for (int i = 0; i < MINE; ++i)
          page[i] = __ldg(pages + min((lo + step * N + 16 * tile_of(i)) >> a.kb.page_shift, a.kb.max_pages - 1));
      };
      uint32_t con[MINE][(NB + 1) / 2];  // constants of this lane's tokens, as loaded for the step to come
      auto fetch = [&](int step, const int (&page)[MINE], int stage) {
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          if (tile_of(i) >= TILES) continue;
          const int t = lo + step * N + 16 * tile_of(i);
          const bool bad = static_cast<unsigned>(page[i]) >= static_cast<unsigned>(a.kb.num_pages);
          bad_page |= bad && t < len;
          const uint32_t row = bad ? 0
                                   : ((static_cast<uint32_t>(page[i]) * a.heads + head) << a.kb.page_shift) +
                                         (t & ((1 << a.kb.page_shift) - 1));
          const uint8_t *src = codes + static_cast<uint64_t>(row) * (D / 2) + lane * 16;
#pragma unroll
          for (int x = 0; x < D / 64; ++x)  // 8 D bytes of codes per tile
            copy16(gap(stage, tile_of(i) * 8 * D + x * 512 + lane * 16), src + x * 512);
          const uint16_t *pc = absmax + (static_cast<uint64_t>(row) + tok) * NB;
          if constexpr (NB == 1) con[i][0] = __ldg(pc);
          if constexpr (NB == 2) con[i][0] = __ldg(reinterpret_cast<const uint32_t *>(pc));
          if constexpr (NB == 4) {
            const uint2 u = __ldg(reinterpret_cast<const uint2 *>(pc));
            con[i][0] = u.x;
            con[i][(NB + 1) / 2 - 1] = u.y;
          }
        }
        copies_commit();
      };
      int page[MINE];
      load_pages(0, page);
      fetch(0, page, n & 1);
      load_pages(1, page);
      for (int step = 0; step < nsteps; ++step, ++n) {
        const int st = n & 1;
        // ---- the range of the step's constants
        uint32_t bits[MINE][NB];
        // least: without keys of zero (they wrap past all others); 0xFFFF where there is none
        uint32_t most = 0, least = 0xFFFFu;
        const uint32_t wrap = keys ? 1u : 0u;
#pragma unroll
        for (int i = 0; i < MINE; ++i)
#pragma unroll
          for (int k = 0; k < NB; ++k) {
            const uint32_t c = k & 1 ? con[i][k / 2] >> 16 : con[i][k / 2] & 0xFFFFu;
            // no tile, or behind the sequence: anything, and masked
            const bool none = tile_of(i) >= TILES || lo + step * N + 16 * tile_of(i) + tok >= len;
            bits[i][k] = none ? 0 : c;
            most = max(most, bits[i][k]);
            // (a value of zero is far from all others: it contributes nothing, and folded in, with a high
            // score, it would set the weights' reference)
            least = min(least, none ? 0xFFFFu : c - wrap);
          }
        if (step + 1 < nsteps) {
          fetch(step + 1, page, st ^ 1);
          load_pages(step + 2, page);
          copies_wait<1>();
        } else {
          copies_wait<0>();
        }
        most = __reduce_max_sync(0xFFFFFFFFu, most);
        least = __reduce_min_sync(0xFFFFFFFFu, least);
        if (lane == 0) {
          my_ranges[st * 7 + dw] = make_int2(most, least);
          mbar_arrive(&range[st]);
        }
        ok = wait(&range[st], (n >> 1) & 1);
        // (the factors of the scores are rewritten: no one may still read those of two steps ago)
        if (ok && keys && n > 0) ok = wait(empty, (n - 1) & 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        for (int i = 0; i < warps; ++i) {
          const int2 o = my_ranges[st * 7 + i];
          most = max(most, static_cast<uint32_t>(o.x));
          least = min(least, static_cast<uint32_t>(o.y));
        }
        // ---- constants: folded into the operands (keys below 2^12, values below 2), or apart
        auto exponent = [](uint32_t b) { return static_cast<int>(b >> 7) - 127; };
        const int e = most ? exponent(most) : 0;
        const bool wide = most >= 0x7F80u || e < -100 || e > 110 ||
                          (least != 0xFFFFu && e - exponent(least + wrap) > near);
        __half2 hc[MINE][NB];
        if (!wide) {
          const float f = pow2(keys ? 11 - e : -e);
#pragma unroll
          for (int i = 0; i < MINE; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k) hc[i][k] = __float2half2_rn(__uint_as_float(bits[i][k] << 16) * f);
          if (dw == 0 && lane == 0) {
            if (keys) kinfo[st] = StepInfo{pow2(e - 11), 0};
            else vinfo[st] = StepInfo{static_cast<float>(e), 0};
          }
        } else if (keys) {
          // each token's keys relative to their own exponent
#pragma unroll
          for (int i = 0; i < MINE; ++i) {
            uint32_t top = 0, low = 0xFFFFu;
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              top = max(top, bits[i][k]);
              if (bits[i][k] != 0) low = min(low, bits[i][k]);
            }
            if (NB > 1 && top < 0x7F80u && exponent(top) - exponent(low) > kNearBlocks) a.again[b] = 1;
            const int te = max(exponent(top), -110);
            const bool bad = top >= 0x7F80u;
#pragma unroll
            for (int k = 0; k < NB; ++k)
              hc[i][k] = __float2half2_rn(bad ? 0.0f : __uint_as_float(bits[i][k] << 16) * pow2(11 - te));
            if (sub == 0 && tile_of(i) < TILES)
              cs[st * N + 16 * tile_of(i) + tok] = bad ? __uint_as_float(0x7FC00000u) : pow2(te - 11);
          }
          if (dw == 0 && lane == 0) kinfo[st] = StepInfo{1.0f, 1};
        } else {
          // levels alone; the constants, as float32, multiply the weights
          const int top = most >= 0x7F80u ? 0 : e;
          const int base = top > 80 ? top - 80 : top < -100 ? max(top, -126) : 0;
#pragma unroll
          for (int i = 0; i < MINE; ++i)
#pragma unroll
            for (int k = 0; k < NB; ++k) {
              hc[i][k] = __float2half2_rn(1.0f);
              if (sub == 0 && tile_of(i) < TILES)
                cv[(st * NB + k) * N + 16 * tile_of(i) + tok] = bits[i][k] >= 0x7F80u
                                                                    ? __uint_as_float(0x7FC00000u)
                                                                    : __uint_as_float(bits[i][k] << 16) * pow2(-base);
            }
          if (dw == 0 && lane == 0) vinfo[st] = StepInfo{static_cast<float>(base), 1};
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&cfull[st]);
        if (!keys && n > 0) ok = wait(empty, (n - 1) & 1);
        if (!__all_sync(0xFFFFFFFFu, ok)) {
          ok = false;
          break;
        }
        // ---- codes: 16 bytes (32 channels) of a token at a time, in an order of pieces and words
        // that keeps eight neighbouring lanes (4 tokens) out of each other's banks
#pragma unroll
        for (int i = 0; i < MINE; ++i) {
          if (tile_of(i) >= TILES) continue;
          const int tr = 16 * tile_of(i) + tok;
#pragma unroll
          for (int it = 0; it < PASSES; ++it) {
            const int q = NB == 1 ? sub : NB == 2 ? 2 * sub + (it ^ ((tr >> 1) & 1)) : 4 * sub + (it ^ (tr & 3));
            uint32_t w[4];
            lds128(gap(st, tr * (D / 2) + q * 16), w);
            constexpr int SWAP = NB == 1 ? 0 : NB == 2 ? 2 : 1;
            const int swap = sub * SWAP;
            if constexpr (SWAP != 0) {
#pragma unroll
              for (int j = 0; j < 4; ++j)
                if (j < (j ^ SWAP)) {
                  const uint32_t x = w[j], y = w[j ^ SWAP];
                  w[j] = sub ? y : x;
                  w[j ^ SWAP] = sub ? x : y;
                }
            }
            __half2 f = hc[i][0];
#pragma unroll
            for (int k = 1; k < NB; ++k)
              if ((q >> 1) == k) f = hc[i][k];
            const uint32_t out = operand + (q >> 1) * (N * 128) + tr * 128;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              uint32_t o[4] = {lookup<0>(w[j], tab), lookup<1>(w[j], tab), lookup<2>(w[j], tab), lookup<3>(w[j], tab)};
#pragma unroll
              for (int x = 0; x < 4; ++x) {
                const __half2 y = __hmul2(*reinterpret_cast<__half2 *>(&o[x]), f);
                o[x] = *reinterpret_cast<const uint32_t *>(&y);
              }
              st_shared_v4(out + ((((q & 1) * 4 + (j ^ swap)) ^ (tr & 7)) << 4), o[0], o[1], o[2], o[3]);
            }
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(full);
      }
      copies_wait<0>();
      __syncwarp();
      if (bad_page) kv_error(a.kb);
    }
    } else {
    // all lanes run the loop, so that addresses stay in uniform registers; one issues
    // ================================================================ MMA issue
    constexpr uint32_t idesc_s = idesc_f16(128, N, false), idesc_o = idesc_f16(128, D, true),
                       idesc_ob = idesc_f16(128, 64, true);
    uint32_t n = 0;                 // steps of the CTA
    uint32_t done[2] = {0, 0};      // P V products of each row tile
    uint32_t queries[2] = {0, 0};
    bool ok = true;
    auto wait_all = [&](uint64_t *bar, uint32_t parity) { return __all_sync(0xFFFFFFFFu, wait(bar, parity)) != 0; };
    const uint64_t q_desc = smem_desc_sw128(q_smem, 16, 1024), k_desc = smem_desc_sw128(k_smem, 16, 1024),
                   v_desc = smem_desc_sw128(v_smem, N * 128, 1024);
    auto scores = [&](int m) {  // S_m = Q_m K^T
#pragma unroll
      for (int k = 0; k < D / 16; ++k)
        mma_f16_ss(tmem + m * C::SP_COLS, q_desc + ((m * C::Q_BYTES + (k >> 2) * 16384 + (k & 3) * 32) >> 4),
                   k_desc + (((k >> 2) * (N * 128) + (k & 3) * 32) >> 4), idesc_s, k > 0 ? 1u : 0u);
    };
    auto outputs = [&](int m, bool first, bool wide) {  // O_m += P_m V, or O_m,b += P_m,b V_b block by block
      const uint32_t d = tmem + C::O_COL + m * D, pt = tmem + m * C::SP_COLS + C::P_COL;
      if (!wide) {
#pragma unroll
        for (int k = 0; k < N / 16; ++k)
          mma_f16_ts(d, pt + (TW == 32 ? 32 * (k >> 1) + 8 * (k & 1) : 32 * k), v_desc + (k * 2048 >> 4), idesc_o,
                     !first || k > 0 ? 1u : 0u);
      } else {
#pragma unroll 1
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int k = 0; k < N / 16; ++k) {
            const int at = TW == 32 ? 32 * (k >> 1) + 16 * b + 8 * (k & 1) : 32 * k + 8 * b;
            mma_f16_ts(d + 64 * b, pt + at, v_desc + ((b * (N * 128) + k * 2048) >> 4), idesc_ob,
                       !first || k > 0 ? 1u : 0u);
          }
      }
    };
    while (ok) {
      int tiles, nsteps;
      {
        Segment sg;
        if (!next_part<C>(p, my_line, entry, done_steps, sg)) break;
        tiles = MT == 2 && sg.rows > 128 ? 2 : 1;
        nsteps = sg.step1 - sg.step0;
        done_steps += sg.used;
      }
      for (int m = 0; m < tiles && ok; ++m) ok = wait_all(&qfull[m], queries[m]++ & 1);
      if (ok) ok = wait_all(kfull, n & 1);
      if (!ok) break;
      tc_fence_after();
      // the previous item's outputs have been waited for by its softmax warps, which then
      // announced these queries
      for (int m = 0; m < tiles; ++m) {
        scores(m);
        commit(&sfull[m]);
      }
      commit(kempty);
      for (int i = 0; i < nsteps && ok; ++i) {
        ok = wait_all(vfull, n & 1);
        const bool wide = __shfl_sync(0xFFFFFFFFu, vinfo[n & 1].wide, 0) != 0;
        for (int m = 0; m < tiles && ok; ++m) {
          ok = wait_all(&pfull[m], done[m] & 1);
          if (!ok) break;
          tc_fence_after();
          outputs(m, i == 0, wide);
          commit(&opv[m]);
          if (m == tiles - 1) commit(vempty);
          if (i + 1 < nsteps) {
            // the next scores overwrite the weights this product reads
            if (m == 0) ok = wait_all(kfull, (n + 1) & 1);
            ok = ok && wait_all(&opv[m], done[m] & 1);
            if (!ok) break;
            tc_fence_after();
            scores(m);
            commit(&sfull[m]);
            if (m == tiles - 1) commit(kempty);
          }
          ++done[m];
        }
        ++n;
      }
    }
    // after a wait that gave up too, nothing may still write TMEM or read shared memory
    // when the CTA leaves
    int unused = 0;
    commit(drain);
    mbar_wait_bounded(drain, 0, &unused, nullptr, kDrainNs);
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 12) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
}

template <class C>
size_t entries_of(int group, int batch, int64_t tokens) {
  return static_cast<size_t>(tokens * group / C::ROWS + batch);
}

template <class C>
size_t workspace_of(int group, int batch, int64_t tokens, int num_sms) {
  const size_t e = entries_of<C>(group, batch, tokens);
  return 48 + e * sizeof(KvEntry) + (e + 2) / 2 * 16 +
         static_cast<size_t>(num_sms) * 2 * (sizeof(KvPart) + C::ROWS * 4 + static_cast<size_t>(C::ROWS) * C::D * 4);
}

template <class C>
cudaError_t run_prefill(const KvAttnArgs &args, void *ws, int num_sms, unsigned long long timeout_ns, cudaStream_t st) {
  static std::atomic<uint64_t> attr_done{0};
  cudaError_t e = smem_attr_once(reinterpret_cast<const void *>(k_kv_prefill<C>), C::SMEM_BYTES, attr_done);
  if (e != cudaSuccess) return e;
  if (num_sms > kMaxWorkers) num_sms = kMaxWorkers;
  PrefillArgs p;
  p.a = args;
  p.timeout_ns = timeout_ns;
  const size_t n = entries_of<C>(args.group, args.kb.batch, args.kb.tokens);
  p.max_entries = static_cast<int>(n);
  uint8_t *w = static_cast<uint8_t *>(ws);
  p.count = reinterpret_cast<int *>(w);
  w += 16;
  p.entries = reinterpret_cast<KvEntry *>(w);
  w += n * sizeof(KvEntry);
  p.prefix = reinterpret_cast<int64_t *>(w);
  w += (n + 2) / 2 * 16;
  p.a.parts = reinterpret_cast<KvPart *>(w);
  w += static_cast<size_t>(num_sms) * 2 * sizeof(KvPart);
  p.a.part_lse = reinterpret_cast<float *>(w);
  w += static_cast<size_t>(num_sms) * 2 * C::ROWS * 4;
  p.a.part_o = reinterpret_cast<float *>((reinterpret_cast<uintptr_t>(w) + 31) & ~static_cast<uintptr_t>(31));  // for 32-byte stores
  if ((e = launch_k(k_kv_plan<C>, dim3(1), dim3(kPlanThreads), 0, st, 1, p)) != cudaSuccess) return e;
  if ((e = launch_k(k_kv_prefill<C>, dim3(num_sms), dim3(C::THREADS), C::SMEM_BYTES, st, 1, p)) != cudaSuccess) return e;
  return launch_k(k_kv_join<C::D, C::ROWS, 1>, dim3(num_sms - 1, C::ROWS / 8), dim3(256), 0, st, 1, p.a);
}

}  // namespace

size_t kv_prefill_workspace(int head_dim, int group, int batch, int64_t tokens, int num_sms) {
  switch (head_dim) {
    case 64: return workspace_of<PreCfg<64>>(group, batch, tokens, num_sms);
    case 128: return workspace_of<PreCfg<128>>(group, batch, tokens, num_sms);
    default: return workspace_of<PreCfg<256>>(group, batch, tokens, num_sms);
  }
}

cudaError_t launch_kv_prefill(const KvAttnArgs &a, int head_dim, void *ws, int num_sms, unsigned long long timeout_ns,
                              cudaStream_t st) {
  switch (head_dim) {
    case 64: return run_prefill<PreCfg<64>>(a, ws, num_sms, timeout_ns, st);
    case 128: return run_prefill<PreCfg<128>>(a, ws, num_sms, timeout_ns, st);
    default: return run_prefill<PreCfg<256>>(a, ws, num_sms, timeout_ns, st);
  }
}

}  // namespace qlora
