// Attention of one new token per request over the paged INT4 key/value cache.
//
//   s_i = scale q . k_i,  m = max s_i,  l = sum exp(s_i - m),
//   y = (sum exp(s_i - m) v_i) / l,   k_i, v_i = code * scale
//
// The floor is one read of the cache: 132 bytes per token and key-value head
// against 4 * 128 operations per query head, so the work is a stream of pages
// with the arithmetic hidden under it.  At the measured 6.55 TB/s an SM has
// about 5.7 cycles per token and head, i.e. some 23 warp instructions; this kernel
// executes as many, and with the four warps that a scheduler's registers hold issues in 59 % of the
// cycles, waiting for products and their results: 64 requests of 8 heads and 14200
// tokens on average (eight queries a head) take 232 us, 4.1 TB/s.
//
// Division.  The turns (32 tokens of one request and key-value head) of all
// requests form one sequence, request-major; every CTA takes an equal contiguous
// part of it and every warp an equal contiguous part of that, found on the GPU from the lengths, so
// ragged batches load every SM alike and a captured launch follows the lengths
// of its replay.  A warp's part is a run of segments (one request and head each) that it
// streams on its own, with 16-byte asynchronous copies one turn ahead.  A segment that
// covers its whole request leaves as output at once; a first one that continues an earlier warp's
// goes to shared memory, a last one that is cut off stays in registers, and when all
// warps are done the pieces are added in order.  What still lacks pieces of other CTAs
// goes to the workspace as (sum, m, l), and the CTA that arrives last adds these in
// their fixed order (the sums come out the same whichever CTA that is).  With one
// join of the warps per CTA instead of one per segment, ragged batches lost a third of their time.
//
// Products.  mma.sync, whose operands are registers: the codes are unpacked into them and used at once.  The tensor-memory
// path takes 128 rows, which could be tokens (scores) and dims (sums), and would read the unpacked codes from shared
// or tensor memory: in 8 bits 256 bytes written and read again per token and head, some 4 of the 5.7 cycles at
// 128 bytes a cycle.  It has not been built or measured.
//  - scores, up to four query heads: m16n8k32 in integers, A = 16 tokens x 128 dims of K codes (nibbles shifted to
//    the top of a byte: 16 code, one logic operation per four), B = the queries as whole multiples of 2^-22 of the
//    power of two above their head's largest value, in three signed bytes: an fp16 value of at least 2^-11 of
//    the largest is such a multiple, a smaller one is off by at most 2^-22 of the largest.  The sums are exact, so
//    three float32 roundings are all else that a score has.  The tile's other four columns take the second byte.
//  - scores, more query heads: m16n8k16, A = 16 tokens x 128 dims of K codes as fp16 numbers (as the values', below), B =
//    the queries as they are; a sum's 128 terms are cut off at 2^-23 of the largest or finer.  With three bytes and integers
//    16 query heads took 39.1 instead of 35.7 us (33 requests of 64/4 heads and 4096 tokens), 64 long
//    requests of 64/8 heads 229 instead of 232; with this way for four query heads too 12 x 32/32 heads took 35.0 instead of 32.9.
//    With queries in two bytes (half a step of max|q| / 32639) a query channel 30 (100) times the others left errors of
//    1.4 to 1.8 (2.9 to 6.2) times the output's own rounding, scores of standard deviation 14 up to 1.19 times;
//    now it is 1.0 everywhere.  A lane reads 16 consecutive bytes of a token's row; the order of the dims inside
//    the product is free, so the queries are arranged once per segment to match the nibbles.
//  - sum: m16n8k16, A = 128 dims x 16 tokens of V codes (exact; a logic operation makes a subnormal
//    fp16 number of a nibble, a multiply-add the code), B = the weights, taken from the scores' layout by
//    movmatrix.  A lane reads 8 bytes of each of its 4 tokens and pairs two tokens' nibbles by byte permutation.  A turn's
//    32 tokens are added up in the tensor core, which cuts every term off at 2^-23 of the largest or finer; the
//    running sums are rounded float32 adds (added after every 16 tokens, attention took 2 to 6 % longer).
//    With the subnormal numbers as operands, and -8 sum(w) added by one more product, long caches took 2 % less
//    time, but the tensor core aligns its terms by a subnormal operand's exponent, 2^6 times the number's own, and
//    the terms were cut off that much earlier: 10 to 18 % of the outputs came out rounded to the wrong side, now 0.2 %.
// Weights: w = exp2(s - m) * (v scale), times 2^8 over the head's largest w so far, enters as two fp16 numbers, its
// rounding and what that left (2^-22 relative, or 2^-33 of that largest where the second is
// subnormal).  Taken relative to the largest v scale instead, they were lost beside a token of no weight with a much
// larger v scale: errors of 1.05, 5, 21 and 170 times the output's own rounding at 2^14, 2^18, 2^20 and 2^23 times
// theirs, at the same speed.  With the rounding alone an earlier version was 14 % faster on long caches (188 us instead of 217), but
// left 1.5 times the error of the output's own rounding.  The second product joins the turn's sums: added to the running
// ones directly, whose sum it cuts off at 2^-23 once per 16 tokens, it took 2 % less time, but a warp's part of 227
// thousand tokens came out 8e-5 too small, and longer ones by more.
// m and the largest w are references that move only when a weight passes one by 2^7 (checked with one vote
// per 32 tokens), so the sums are rarely rescaled.
#include <cuda_fp16.h>

#include <algorithm>

#include "fq_device.cuh"
#include "fq_host.h"
#include "kv_cache.cuh"

namespace fq {

size_t sync_block_bytes();

namespace {

constexpr int kStep = 32;           // tokens per turn, taken as two halves of 16
constexpr int kStepV = kStep * kKvRowBytes, kStepKs = 2 * kStepV, kStepVs = kStepKs + 2 * kStep;
constexpr int kStepBytes = kStepVs + 2 * kStep;  // K codes, V codes, K scales, V scales
constexpr int kDepth = 2;           // turns of a warp in shared memory: one taken, one under way
// What a request and head costs besides its turns, in turns.  With 1, 2, 3 and 4: 17 ragged requests of 32/8 heads to
// 8192 tokens 29.4, 26.2, 26.3, 25.9 us, 48 of 16/16 heads to 4000 60.3, 54.0, 53.3, 53.3, one of 4000 tokens 13.6,
// 13.9, 12.5, 12.5, 64 even ones of 64/8 heads and 14200 228.4, 228.4, 228.7, 229.1.
constexpr int kItemCost = 3;
// Little work: a part shorter than kMinUnits, or a request and head in more than kMaxParts parts, costs
// more in the join than it saves.  One request of 8 heads and 4000 tokens took 12.4 us with parts of 8, 16.0 us
// with 24, 17.4 us with 40; one head of 16384 tokens 14.6 us in 64 parts, 12.9 us in 32.
constexpr int kMinUnits = 8, kMaxParts = 32;
// Where every request and head can have a CTA, none is divided unless the largest has kJoinUnits (the cost of the
// join) more than an equal part.  33 requests of 40/8 heads and 1300 tokens took 23.4 us divided, 19.4 whole, of
// 2048 29.5 and 26.2; 8 heads of 1000 tokens 12.0 and 11.6, of 4000 12.2 and 23.6; 33 of 0 to 2000 tokens 22.7 and 24.8.
constexpr int kJoinUnits = 28;
constexpr int kWarps = 8;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kMaxAttnR = 16384;
constexpr float kSlack = 128.0f;    // how far a weight may pass its reference
constexpr float kLowest = -1e30f;   // the reference before the first score
constexpr float kWeightScale = 256.0f;
constexpr float kLeastWeight = 0x1p-100f;  // largest weights below this count as this: far from any that an output shows
constexpr float kRound = 12582912.0f;  // 1.5 * 2^23: adding it leaves a rounded integer in the low bits
constexpr int kRoundBits = 0x4B400000;

struct AttnParams {
  const __half* Q;
  long long ldq;
  int R, Hq, G, chunks;             // chunks of at most 8 NT query heads per key-value head
  const int32_t* len;
  const int32_t* table;
  int max_pages;
  KvView kv;
  float scale_log2;
  int window;
  __half* Y;
  float* part;                      // [2 * CTAs][8 NT][130]: sums, m, l
  unsigned* count;                  // one counter per CTA
};

// A warp's walk over its part, and the segment it is at: turns [ta, ta + turns) of the nt turns of a request
// and key-value head's chunk of query heads.  Kept in shared memory, since the turns leave no register for it.
struct WarpWalk {
  long long pos, last;  // units still to be taken
  long long before;     // units before request r
  long long item0;      // the first unit of the segment's request and head
  int next, r, head, chunk, nt, ta;
};

struct AttnSmem {
  long long pre[kAttnThreads + 1];  // units of one head before each thread's run of requests
  long long wsum[kWarps];
  int wmax[kWarps];
  long long part[2], total;         // this CTA's units, all units
  int ctas;                         // CTAs that share them
  // pieces of requests and heads: 0 a warp's first segment, if it continues an earlier warp's, 1 its last
  // one, if it is cut off.  item: the first unit of the request and head, -1: no piece
  long long item[kWarps][2];
  WarpWalk walk[kWarps];
  int ends;                         // bit w: piece 0 of warp w reaches the end of its request
  int row[kWarps][2], heads[kWarps][2], turns[kWarps][2];  // its first row of Y, heads, turns of the whole
  float m[kWarps][2][16], l[kWarps][2][16];
  int join[2], left[2];             // parts this CTA has left and is the last to: 0 continued, 1 started here
};

// Turns [t0, t1) and tokens [lo, hi) of request r.
struct Span {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int r) {
  const long long cap = static_cast<long long>(p.max_pages) << p.kv.page_shift;
  Span s;
  s.hi = int(min(static_cast<long long>(max(p.len[r], 0)), cap));
  s.lo = p.window > 0 ? max(0, s.hi - p.window) : 0;
  s.t0 = s.lo / kStep;
  s.t1 = s.hi > s.lo ? (s.hi - 1) / kStep + 1 : s.t0;
  return s;
}

// a / b of non-negative numbers, in 32 bits where they fit.
__device__ __forceinline__ long long divide(long long a, long long b) {
  if (((a | b) >> 32) == 0) return uint32_t(a) / uint32_t(b);
  return a / b;
}

// 2^x within 2^-22 of itself; results below 2^-126 are 0.  That is what two float32 roundings of the argument leave
// as well, and nothing beside the output's 2^-11.
__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1, const float (&c)[4]) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%11,%12,%13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]), "f"(c[3]));
}

__device__ __forceinline__ void mma_s8(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                       uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+r"(c[0]), "+r"(c[1]), "+r"(c[2]), "+r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The first product of a sum, which starts from kRound's bits: below 2^22 in magnitude, the sum is then a float32 number's
// mantissa, and whole_numbers() takes it out without a conversion.
__device__ __forceinline__ void mma_s8_first(int (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                             uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k32.row.col.s32.s8.s8.s32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%10,%10,%10,%10};"
      : "=r"(c[0]), "=r"(c[1]), "=r"(c[2]), "=r"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "r"(kRoundBits));
}
__device__ __forceinline__ float2 whole_numbers(int a, int b) {
  return fadd2(make_float2(__int_as_float(a), __int_as_float(b)), make_float2(-kRound, -kRound));
}

__device__ __forceinline__ void add4(float (&a)[4], const float (&b)[4]) {
  const float2 x = fadd2(make_float2(a[0], a[1]), make_float2(b[0], b[1]));
  const float2 y = fadd2(make_float2(a[2], a[3]), make_float2(b[2], b[3]));
  a[0] = x.x;
  a[1] = x.y;
  a[2] = y.x;
  a[3] = y.y;
}

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// The same byte of four words, by a byte selection of two words at a time.
__device__ __forceinline__ uint32_t bytes4(const uint32_t (&v)[4], uint32_t sel) {
  return __byte_perm(__byte_perm(v[0], v[1], sel), __byte_perm(v[2], v[3], sel), 0x5410);
}

// Nibbles u of each half word at bits 0-3 and 4-7 -> the fp16 numbers q 2^-10, u = q + 8: the codes' top bits are flipped
// beforehand (here, in the same operation, took 4 % longer).  A nibble is the mantissa of the subnormal number u 2^-24
// or u 2^-20, and one exact multiply-add takes it to q 2^-10.
__device__ __forceinline__ uint32_t codes_from(uint32_t u, uint16_t factor) {
  const __half2 q = __hfma2(*reinterpret_cast<const __half2*>(&u), __half2half2(__ushort_as_half(factor)),
                            __half2half2(__ushort_as_half(0xA000)));  // -8 2^-10
  return *reinterpret_cast<const uint32_t*>(&q);
}
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return codes_from(w & 0x000F000Fu, 0x7400); }  // 2^14
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return codes_from(w & 0x00F000F0u, 0x6400); }  // 2^10

// The token of score row i (0..15): rows 2t, 2t + 1 of one lane's weights.  Bit 0
// alternates within a row pair (score reads of two rows hit different banks)
// and with t (the four lanes of a value read hit two bank halves).
__device__ __forceinline__ int token_of_row(int i) {
  const int t = (i >> 1) & 3, b = i & 1;
  return (b ^ (t & 1)) | ((t & 1) << 1) | ((t >> 1) << 2) | (i & 8);
}

// Where value k (of 4) of product i (of 8) of a lane lies in a kept piece: lanes write consecutive
// words, and the lanes of a warp that read one head's values (see the adding of pieces) find 32 banks.
constexpr int kPieceFloats = 32 * 32 + 4;
__device__ __forceinline__ int piece_offset(int i, int k, int lane) { return (4 * i + k) * 32 + lane + (i >> 1); }

template <int TO = 0, int FROM = 0>
__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(TO), "n"(FROM)
               : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The CTA whose part holds unit x of the sequence: parts are [total c / C, total (c + 1) / C).
__device__ __forceinline__ int cta_of_unit(long long x, long long total, int C) {
  return int(divide((x + 1) * C - 1, total));
}

// The parts of one request and head, left by CTAs c_first .. c_first + parts - 1, added in that
// order and written as `heads` rows of Y.  A warp takes one head, or, with four heads or
// fewer, one head's every second (fourth, eighth) part; the loads of eight parts
// are under way at a time.
template <int HB>
__device__ __noinline__ void join_parts(const float* all, int c_first, int parts, int heads, float* sums, __half* Y) {
  constexpr size_t kSlot = static_cast<size_t>(HB) * (kHeadDim + 2);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub_n = heads <= 1 ? 8 : heads <= 2 ? 4 : heads <= 4 ? 2 : 1;
  auto slot = [&](int c) { return all + (2 * static_cast<size_t>(c_first + c) + (c == 0)) * kSlot; };
  for (int hh = warp / sub_n; hh < heads; hh += kWarps / sub_n) {
    const int sub = warp % sub_n;
    float mx = kLowest;
    for (int c = lane; c < parts; c += 32) mx = fmaxf(mx, __ldcg(slot(c) + HB * kHeadDim + hh));
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float ls = 0.f;
    for (int c0 = sub; c0 < parts; c0 += 8 * sub_n) {
      float4 v[8];
      float mc[8], lc[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int c = c0 + k * sub_n;
        const float* src = slot(min(c, parts - 1));
        mc[k] = c < parts ? __ldcg(src + HB * kHeadDim + hh) : kLowest;
        lc[k] = c < parts ? __ldcg(src + HB * kHeadDim + HB + hh) : 0.f;
        v[k] = c < parts ? __ldcg(reinterpret_cast<const float4*>(src + hh * kHeadDim) + lane)
                         : make_float4(0.f, 0.f, 0.f, 0.f);
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float f = exp2_approx(mc[k] - mx);
        ls += lc[k] * f;
        acc.x += v[k].x * f;
        acc.y += v[k].y * f;
        acc.z += v[k].z * f;
        acc.w += v[k].w * f;
      }
    }
    if (sub_n > 1) {  // at most one head per warp: every warp comes here once or not at all
      float* mine = sums + warp * (kHeadDim + 4);
      *reinterpret_cast<float4*>(mine + 4 * lane) = acc;
      if (lane == 0) mine[kHeadDim] = ls;
      named_barrier(1 + hh, 32 * sub_n);
      if (sub != 0) continue;
      acc = make_float4(0.f, 0.f, 0.f, 0.f);
      ls = 0.f;
      for (int k = 0; k < sub_n; ++k) {
        const float* other = sums + (warp + k) * (kHeadDim + 4);
        const float4 v = *reinterpret_cast<const float4*>(other + 4 * lane);
        acc.x += v.x;
        acc.y += v.y;
        acc.z += v.z;
        acc.w += v.w;
        ls += other[kHeadDim];
      }
    }
    const float inv = ls > 0.f ? 1.0f / ls : 0.f;
    const __half2 a = __floats2half2_rn(acc.x * inv, acc.y * inv);
    const __half2 b = __floats2half2_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(Y + hh * kHeadDim + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
}

// NT: tiles of 8 query heads; TWICE: at most 4 query heads, which also take columns 4-7 of the tile: there
// the weights are what the rounding of those in columns 0-3 left, so one product does both; P16: pages of 16
// tokens, so that a turn spans two.
template <int NT, bool TWICE, bool P16>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 2 : 1) kv_attn_kernel(const AttnParams p) {
  constexpr int HB = 8 * NT;
  // the warps' turns, then each warp's continued segment, [32 NT values][32 lanes]
  extern __shared__ __align__(128) uint8_t dyn[];
  float* sums = reinterpret_cast<float*>(dyn + kWarps * kDepth * kStepBytes);
  __shared__ AttnSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, HC = p.kv.H * p.chunks;
  pdl_launch_dependents();
  pdl_wait();

  // ---- the sequence: each thread's run of requests, summed (the requests that have tokens counted in
  // the upper bits)
  const int run = (p.R + kAttnThreads - 1) / kAttnThreads;
  const int ra = min(p.R, tid * run), rb = min(p.R, ra + run);
  constexpr int kCountBit = 44;
  long long mine = 0;
  int largest = 0;  // units of a request and head
  for (int r = ra; r < rb; ++r) {
    const Span s = span_of(p, r);
    if (s.t1 > s.t0) {
      mine += (s.t1 - s.t0) + kItemCost + (1ll << kCountBit);
      largest = max(largest, (s.t1 - s.t0) + kItemCost);
    }
  }
  largest = __reduce_max_sync(0xffffffffu, largest);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.wsum[warp] = incl, sm.wmax[warp] = largest;
  if (lane < 2) sm.item[warp][lane] = -1;
  if (tid == 0) sm.ends = sm.join[0] = sm.join[1] = 0;
  __syncthreads();
  long long all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) incl += sm.wsum[w];
    all += sm.wsum[w];
    largest = max(largest, sm.wmax[w]);
  }
  constexpr long long kUnits = (1ll << kCountBit) - 1;
  sm.pre[tid] = (incl - mine) & kUnits;
  const long long total = (all & kUnits) * HC;
  const long long items = (all >> kCountBit) * HC;
  int C = int(min(static_cast<long long>(gridDim.x), max(min(items * kMaxParts, total / kMinUnits), items)));
  const bool whole = items <= gridDim.x && static_cast<long long>(largest - kJoinUnits) * C <= total;
  if (whole) {
    C = int(items);
    // request number cta / HC of those with tokens, head cta % HC
    int n = cta / HC - int((incl - mine) >> kCountBit);
    if (n >= 0 && n < int(mine >> kCountBit)) {
      long long before = sm.pre[tid];
      for (int r = ra; r < rb; ++r) {
        const Span s = span_of(p, r);
        if (s.t1 == s.t0) continue;
        const int units = s.t1 - s.t0 + kItemCost;
        if (n-- == 0) {
          sm.part[0] = before * HC + static_cast<long long>(cta % HC) * units;
          sm.part[1] = sm.part[0] + units;
        }
        before += units;
      }
    }
  }
  for (int r = cta; r < p.R; r += gridDim.x) {  // requests without tokens
    const Span s = span_of(p, r);
    if (s.t1 == s.t0)
      for (int i = tid; i < p.Hq * kHeadDim / 8; i += kAttnThreads)
        reinterpret_cast<uint4*>(p.Y + static_cast<size_t>(r) * p.Hq * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
  }
  if (cta >= C) return;
  if (tid == 0) {
    if (!whole) {
      sm.part[0] = divide(total * cta, C);
      sm.part[1] = divide(total * (cta + 1), C);
    }
    sm.total = total;
    sm.ctas = C;
  }
  __syncthreads();
  // this CTA's part, this warp's part of it, and the request that one starts in
  const long long units = sm.part[1] - sm.part[0];
  WarpWalk& walk = sm.walk[warp];
  {
    const long long first = sm.part[0] + units * warp / kWarps;
    const int b8 = 8 * (__popc(__ballot_sync(0xffffffffu, sm.pre[8 * lane] * HC <= first)) - 1);
    const int t = b8 + __popc(__ballot_sync(0xffffffffu, lane < 8 && sm.pre[b8 + (lane & 7)] * HC <= first)) - 1;
    if (lane == 0) {
      walk.pos = first;
      walk.last = sm.part[0] + units * (warp + 1) / kWarps;
      walk.next = t * run;
      walk.before = sm.pre[t] * HC;
    }
    __syncwarp();
  }

  const int ps = p.kv.page_shift;
  const int g = lane >> 2, t4 = lane & 3;
  // what this lane copies of a turn: every 32nd 16-byte piece of the K and of the V codes, and lanes
  // 0-7 (pages of 16: 0-3 of each page) a piece of the scales
  constexpr int kHalves = P16 ? 2 : 1;
  constexpr int kScalePieces = P16 ? 2 : 4;   // 16-byte pieces of one kind of scales per page taken
  const uint32_t my_ring = smem_u32(dyn) + uint32_t(warp * kDepth * kStepBytes + lane * 16);
  // its scales from and to, less the 16 lane of the codes
  const int sc_src = (2 * kKvRowBytes << ps) + (lane % kScalePieces) * 16 + (lane / kScalePieces & 1) * (2 << ps) - lane * 16;
  const uint32_t sc_dst = kStepKs + (lane % kScalePieces) * 16 + (lane / kScalePieces & 1) * (2 * kStep) - lane * 16;
  const int v_src = kKvRowBytes << ps, page_mask = (1 << ps) - 1;
  const uint32_t page_bytes = uint32_t(p.kv.H) * uint32_t(p.kv.block_bytes());  // of all heads: 2.2 MB at most
  // byte offsets inside a turn of this lane's operands
  const int row0 = token_of_row(g);           // score rows g and g + 8 of a half: tokens row0, row0 + 8
  const uint8_t* ring = dyn + warp * kDepth * kStepBytes;
  const int k_off = row0 * kKvRowBytes + t4 * 16;
  const int va_off = kStepV + token_of_row(2 * t4) * kKvRowBytes + 8 * g;
  const int vb_off = kStepV + token_of_row(2 * t4 + 1) * kKvRowBytes + 8 * g;
  // The segment under way: its first token, turns, tokens, block table and cache.
  struct Seg {
    int tok0, turns, lo, hi;
    const int32_t* row;
    const uint8_t* cache;  // its head in page 0, this lane's 16 bytes of codes
  };
  auto next_segment = [&](Seg& q) {
    WarpWalk k = walk;
    __syncwarp();  // read by every lane
    while (k.pos < k.last) {
      const Span s = span_of(p, k.next);
      const int nt = s.t1 - s.t0, units = nt ? nt + kItemCost : 0;
      const long long len_r = static_cast<long long>(units) * HC;
      if (k.pos >= k.before + len_r) {
        k.before += len_r;
        ++k.next;
        continue;
      }
      const int hc = int(divide(k.pos - k.before, units));
      k.item0 = k.before + static_cast<long long>(hc) * units;
      k.ta = max(0, int(k.pos - k.item0) - kItemCost);
      const int tb = int(min(static_cast<long long>(units), k.last - k.item0)) - kItemCost;
      k.pos = min(k.item0 + units, k.last);
      if (tb <= k.ta) continue;
      k.r = k.next;
      k.head = p.chunks == 1 ? hc : hc / p.chunks;
      k.chunk = hc - k.head * p.chunks;
      k.nt = nt;
      if (lane == 0) walk = k;
      __syncwarp();
      q.turns = tb - k.ta;
      q.lo = s.lo;
      q.hi = s.hi;
      q.tok0 = (s.t0 + k.ta) * kStep;
      q.row = p.table + static_cast<size_t>(k.r) * p.max_pages;
      q.cache = p.kv.block(0, k.head) + lane * 16;
      return true;
    }
    return false;
  };
  struct Ids {
    int id[kHalves];
  };
  auto page_ids = [&](const Seg& q, int i) {
    Ids v;
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      const int t = q.tok0 + i * kStep + 16 * h;
      // a half may lie before or behind the request's tokens
      const bool in = i < q.turns && (!P16 || (t + 16 > q.lo && t < q.hi));
      v.id[h] = in ? __ldg(q.row + (t >> ps)) : -1;
    }
    return v;
  };
  // Copies of turn i into ring slot `to`; returns which halves have their tokens (bits 0, 1).
  auto fetch = [&](const Seg& q, int i, const Ids& ids, int to) {
    uint32_t got = 0;
    const uint32_t dst = my_ring + uint32_t(to * kStepBytes);
#pragma unroll
    for (int h = 0; h < kHalves; ++h) {
      if (uint32_t(ids.id[h]) < uint32_t(p.kv.num_pages)) {
        const uint32_t off = P16 ? 0 : (q.tok0 + i * kStep) & page_mask;
        const uint8_t* page = q.cache + static_cast<uint64_t>(uint32_t(ids.id[h])) * page_bytes;
        const uint8_t* k = page + static_cast<uint64_t>(off) * kKvRowBytes;
        const uint8_t* v = k + v_src;
        const uint32_t d = dst + h * 1024;
        copy16<0, 0>(d, k);
        copy16<512, 512>(d, k);
        copy16<kStepV, 0>(d, v);
        copy16<kStepV + 512, 512>(d, v);
        if (!P16) {
          copy16<1024, 1024>(d, k);
          copy16<1536, 1536>(d, k);
          copy16<kStepV + 1024, 1024>(d, v);
          copy16<kStepV + 1536, 1536>(d, v);
        }
        if (lane < 2 * kScalePieces) copy16(dst + sc_dst + h * 32, page + static_cast<uint64_t>(off) * 2 + sc_src);
        got |= P16 ? 1u << h : 3u;
      }
    }
    copy_commit();
    return got;
  };
  // Query heads of a segment: heads [q0, q0 + heads)
  auto first_head = [&]() { return walk.head * p.G + walk.chunk * HB; };
  auto head_count = [&]() { return min(HB, p.G - walk.chunk * HB); };
  const int col = TWICE ? g & 3 : g;
  uint4 raw[NT][4];  // lane (g, t4): the head of column g, dims [32 t4, 32 t4 + 32)
  auto load_queries = [&]() {
    const __half* src = p.Q + static_cast<long long>(walk.r) * p.ldq + (first_head() + col) * kHeadDim + 32 * t4;
    const int heads = head_count();
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
      for (int j = 0; j < 4; ++j)
        raw[nn][j] = nn * 8 + col < heads ? *reinterpret_cast<const uint4*>(src + nn * 8 * kHeadDim + 8 * j)
                                        : make_uint4(0, 0, 0, 0);
  };

  constexpr uint32_t kFlip = 0x88888888u;  // code -> code + 8
  Seg seg;
  int slot = 0;         // ring slot of the turn to be taken
  float o[NT][8][4];
  float m[NT][2], l[NT][2];
  float winv[NT][2];             // 2^8 over the largest weight p * (v scale) so far
  bool held = false;             // the last segment is cut off and stays in registers
  static_assert(NT * kPieceFloats * 4 <= kDepth * kStepBytes, "a piece fits a warp's turns");
  auto in_units = [&]() {  // the registers hold 2^-10 of the sums, times winv
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float f = 0x1p10f / winv[nn][k];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          o[nn][i][k] *= f;
          o[nn][i][k + 2] *= f;
        }
      }
    if (TWICE) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[0][i][k] += __shfl_xor_sync(0xffffffffu, o[0][i][k], 2);
    }
  };
  // piece 0 of a warp lies behind the turns, piece 1 takes the warp's own turns' bytes
  auto piece = [&](int w, int which) {
    return which ? reinterpret_cast<float*>(dyn + w * kDepth * kStepBytes) : sums + w * NT * kPieceFloats;
  };
  auto keep = [&](int which) {
    float* dst = piece(warp, which);
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) dst[nn * kPieceFloats + piece_offset(i, k, lane)] = o[nn][i][k];
#pragma unroll
      for (int k = 0; k < 2; ++k)
        if (g == 0) {
          sm.m[warp][which][nn * 8 + 2 * t4 + k] = m[nn][k];
          sm.l[warp][which][nn * 8 + 2 * t4 + k] = l[nn][k];
        }
    }
    if (lane == 0) {
      sm.item[warp][which] = walk.item0;
      sm.row[warp][which] = walk.r * p.Hq + first_head();
      sm.heads[warp][which] = head_count();
      sm.turns[warp][which] = walk.nt;
    }
  };
  auto write_heads = [&](int r, int q0, int heads) {
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const int hh = nn * 8 + 2 * t4 + k;
        if (hh >= heads) continue;
        const float inv = l[nn][k] > 0.f ? 1.0f / l[nn][k] : 0.f;
        uint32_t v[8];  // dims 16 g + 2 j, 16 g + 2 j + 1
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const __half2 x = __floats2half2_rn(o[nn][j][k] * inv, o[nn][j][k + 2] * inv);
          v[j] = *reinterpret_cast<const uint32_t*>(&x);
        }
        uint4* dst = reinterpret_cast<uint4*>(p.Y + (static_cast<size_t>(r) * p.Hq + q0 + hh) * kHeadDim + 16 * g);
        dst[0] = make_uint4(v[0], v[1], v[2], v[3]);
        dst[1] = make_uint4(v[4], v[5], v[6], v[7]);
      }
  };
  while (next_segment(seg)) {
    load_queries();
    Ids next_ids = page_ids(seg, 0);
    // queries of this segment as the products' second operands
    uint32_t qf[NT][16];
    float unit[2];     // of the sums of heads 2 t4, 2 t4 + 1, times the score's scale
    uint32_t most[NT];  // bits of the largest value of column g's head, as float32: at least 0x7F800000 if it is not finite
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
      __half2 m2 = __float2half2_rn(0.f);  // NaN stays
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2* h2 = reinterpret_cast<const __half2*>(&raw[nn][j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) m2 = __hmax2_nan(m2, __habs2(h2[k]));
      }
      uint32_t mb = __float_as_uint(__half2float(__hmax_nan(__low2half(m2), __high2half(m2))));
      mb = max(mb, __shfl_xor_sync(0xffffffffu, mb, 1));  // of numbers without sign, NaN the largest
      most[nn] = max(mb, __shfl_xor_sync(0xffffffffu, mb, 2));
    }
    if (TWICE) {
      // three signed bytes of multiples of 2^(E-22), 2^E the power of two above the head's largest value: q =
      // 2^(E-22) (65536 hi + 256 mid + lo), |hi| <= 64; the even dims of 8 in one word, the odd ones in the next.  The
      // first product's columns 0-3 hold hi and 4-7 mid, the second's lo and 0.
      const uint32_t mb = most[0];
      // the largest value is 0 or has the float32 exponent mb >> 23 in [103, 142] (fp16's range); E = (mb >> 23) - 126
      const bool finite = mb < 0x7F800000u;
      const float inv = mb && finite ? __uint_as_float((275u - (mb >> 23)) << 23) : 0.f;
      const bool upper = g < 4;
      const uint32_t sel = upper ? 0x6262u : 0x5151u, flip = upper ? 0u : 0x80808080u;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2* h2 = reinterpret_cast<const __half2*>(&raw[0][j]);
        uint32_t ev[4], od[4];  // round(q inv) + 128 * 256 + 128: byte 2 is hi, byte 1 mid + 128, byte 0 lo + 128
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __half22float2(h2[k]);
          ev[k] = __float_as_uint(__fmaf_rn(f.x, inv, kRound)) - uint32_t(kRoundBits - 32896);
          od[k] = __float_as_uint(__fmaf_rn(f.y, inv, kRound)) - uint32_t(kRoundBits - 32896);
        }
        qf[0][2 * j] = bytes4(ev, sel) ^ flip;
        qf[0][2 * j + 1] = bytes4(od, sel) ^ flip;
        qf[0][8 + 2 * j] = upper ? bytes4(ev, 0x4040u) ^ 0x80808080u : 0u;
        qf[0][8 + 2 * j + 1] = upper ? bytes4(od, 0x4040u) ^ 0x80808080u : 0u;
      }
      // 2^(E-22) scale / 16 (a nibble is taken 16-fold); a head with an infinity or NaN is NaN
      const float u = !finite ? NAN : mb ? __uint_as_float(((mb >> 23) - 21u) << 23) * (p.scale_log2 / 16.0f) : 0.f;
      unit[0] = __shfl_sync(0xffffffffu, u, 8 * t4);
      unit[1] = __shfl_sync(0xffffffffu, u, 8 * t4 + 4);
    } else {
      // as they are, dims d and d + 4 of 8 in a word, as the nibbles lie; a head with an infinity or NaN is NaN
#pragma unroll
      for (int nn = 0; nn < NT; ++nn)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint4 nan = make_uint4(0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu, 0x7FFF7FFFu);
          const uint4 r = most[nn] < 0x7F800000u ? raw[nn][j] : nan;
          qf[nn][4 * j] = __byte_perm(r.x, r.z, 0x5410);
          qf[nn][4 * j + 1] = __byte_perm(r.x, r.z, 0x7632);
          qf[nn][4 * j + 2] = __byte_perm(r.y, r.w, 0x5410);
          qf[nn][4 * j + 3] = __byte_perm(r.y, r.w, 0x7632);
        }
      unit[0] = unit[1] = p.scale_log2 * 0x1p10f;  // codes are taken as multiples of 2^-10
    }
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nn][i][k] = 0.f;
      m[nn][0] = m[nn][1] = kLowest;
      l[nn][0] = l[nn][1] = 0.f;
      winv[nn][0] = winv[nn][1] = kWeightScale / kLeastWeight;
    }

    uint32_t coming = 0;  // halves of the turn under way
    for (int i = -1; i < seg.turns; ++i) {
      __syncwarp();  // every lane is done with the last turn, whose bytes the next one takes
      const uint32_t have = coming;
      {
        const Ids ids = next_ids;
        next_ids = page_ids(seg, i + 2);
        coming = fetch(seg, i + 1, ids, slot ^ 1);
      }
      const uint8_t* sp = ring + slot * kStepBytes;
      slot ^= 1;
      if (have == 0u) continue;  // nothing there, or the first copies have just been sent
      copy_wait<1>();
      __syncwarp();  // every lane's copies of this turn
      // scores of the 32 tokens: rows g, g + 8 of both halves
      float sc[2][NT][4], ks[2][2], vs[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(sp + k_off + h * 1024);
        const uint4 k1 = *reinterpret_cast<const uint4*>(sp + k_off + h * 1024 + 8 * kKvRowBytes);
        const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
        if (TWICE) {
          int a[2][4];  // sums of the products with hi and mid, and with lo
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t e0, d0, e1, d1;  // 16 q of the even and odd dims of rows g and g + 8
            unpack8_hi(kw0[j], e0, d0);
            unpack8_hi(kw1[j], e1, d1);
#pragma unroll
            for (int b = 0; b < 2; ++b) {
              if (j == 0)
                mma_s8_first(a[b], e0, e1, d0, d1, qf[0][8 * b], qf[0][8 * b + 1]);
              else
                mma_s8(a[b], e0, e1, d0, d1, qf[0][8 * b + 2 * j], qf[0][8 * b + 2 * j + 1]);
            }
          }
#pragma unroll
          for (int k = 0; k < 4; k += 2) {
            // 65536 hi + lo, and 256 mid of the same heads four columns on
            const float c = t4 < 2 ? 65536.0f : 256.0f;
            float2 s = ffma2(whole_numbers(a[0][k], a[0][k + 1]), make_float2(c, c), whole_numbers(a[1][k], a[1][k + 1]));
            s = fadd2(s, make_float2(__shfl_xor_sync(0xffffffffu, s.x, 2), __shfl_xor_sync(0xffffffffu, s.y, 2)));
            s = fmul2(s, make_float2(unit[0], unit[1]));
            sc[h][0][k] = s.x;
            sc[h][0][k + 1] = s.y;
          }
        } else {
          float a[NT][4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint32_t x0 = kw0[j] ^ kFlip, x1 = kw1[j] ^ kFlip, z0 = x0 >> 8, z1 = x1 >> 8;
            const uint32_t e0 = codes_lo(x0), e1 = codes_lo(x1), d0 = codes_hi(x0), d1 = codes_hi(x1);
            const uint32_t f0 = codes_lo(z0), f1 = codes_lo(z1), g0 = codes_hi(z0), g1 = codes_hi(z1);
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
              const float zero[4] = {0.f, 0.f, 0.f, 0.f};
              if (j == 0)
                mma_f16(a[nn], e0, e1, d0, d1, qf[nn][0], qf[nn][1], zero);
              else
                mma_f16(a[nn], e0, e1, d0, d1, qf[nn][4 * j], qf[nn][4 * j + 1], a[nn]);
              mma_f16(a[nn], f0, f1, g0, g1, qf[nn][4 * j + 2], qf[nn][4 * j + 3], a[nn]);
            }
          }
#pragma unroll
          for (int nn = 0; nn < NT; ++nn)
#pragma unroll
            for (int k = 0; k < 4; ++k) sc[h][nn][k] = a[nn][k] * unit[k & 1];
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ks[h][k] = __half2float(*reinterpret_cast<const __half*>(sp + kStepKs + 2 * (row0 + 16 * h + 8 * k)));
          vs[h][k] = __half2float(*reinterpret_cast<const __half*>(sp + kStepVs + 2 * (row0 + 16 * h + 8 * k)));
        }
      }
      const int at = seg.tok0 + i * kStep;
      if (__builtin_expect(at < seg.lo || at + kStep > seg.hi || (P16 && have != 3u), 0)) {
        // what is masked scores -inf and weighs 0, whatever its scales hold
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = at + row0 + 16 * h + 8 * k;
            const bool ok = t >= seg.lo && t < seg.hi && ((have >> h) & 1u);
            ks[h][k] = ok ? ks[h][k] : 1.0f;
            vs[h][k] = ok ? vs[h][k] : 0.0f;
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
              sc[h][nn][2 * k] = ok ? sc[h][nn][2 * k] : -INFINITY;
              sc[h][nn][2 * k + 1] = ok ? sc[h][nn][2 * k + 1] : -INFINITY;
            }
          }
      }
      // log2 of the weights before the v scale, and whether one of them passes its reference, or a weight the largest
      // so far, by too much: 2^top > 2^7 or 2^top vtop winv > 2^15, in one comparison (vtop and top may be of
      // two tokens of the lane, so this asks a little early)
      const float vtop = fmaxf(fmaxf(fabsf(vs[0][0]), fabsf(vs[0][1])), fmaxf(fabsf(vs[1][0]), fabsf(vs[1][1])));
      float x[2][NT][4], far = 0.f;
#pragma unroll
      for (int nn = 0; nn < NT; ++nn)
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          float top = -INFINITY;
#pragma unroll
          for (int h = 0; h < 2; ++h)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              x[h][nn][2 * i + k] = __fmaf_rn(sc[h][nn][2 * i + k], ks[h][i], -m[nn][k]);
              top = fmaxf(top, x[h][nn][2 * i + k]);
            }
          far = fmaxf(far, exp2_approx(top) * fmaxf(vtop * winv[nn][k], kWeightScale));
        }
      if (__any_sync(0xffffffffu, far > kWeightScale * kSlack)) {
        // new references: the largest score of each head, the largest weight
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            float mx = m[nn][k];
#pragma unroll
            for (int h = 0; h < 2; ++h)
              mx = fmaxf(mx, fmaxf(sc[h][nn][k] * ks[h][0], sc[h][nn][k + 2] * ks[h][1]));
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
            const float f = exp2_approx(m[nn][k] - mx);
            m[nn][k] = mx;
            float wm = kLeastWeight;
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                x[h][nn][2 * i + k] = __fmaf_rn(sc[h][nn][2 * i + k], ks[h][i], -mx);
                wm = fmaxf(wm, exp2_approx(x[h][nn][2 * i + k]) * fabsf(vs[h][i]));
              }
#pragma unroll
            for (int d = 4; d < 32; d <<= 1) wm = fmaxf(wm, __shfl_xor_sync(0xffffffffu, wm, d));
            // the largest weight so far, by the new reference
            wm = fmaxf(wm, f * (kWeightScale / winv[nn][k]));
            const float wi = kWeightScale / wm, fw = f * (wi / winv[nn][k]);
            winv[nn][k] = wi;
            l[nn][k] *= f;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[nn][i8][k] *= fw;
              o[nn][i8][k + 2] *= fw;
            }
          }
      }
      constexpr int kW = TWICE ? 1 : 2;
      uint32_t w[2][kW][NT][2];  // of both halves: weights and what their rounding left, as operands
#pragma unroll
      for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
          const float p0 = exp2_approx(x[h][nn][0]), p1 = exp2_approx(x[h][nn][1]);
          const float p2 = exp2_approx(x[h][nn][2]), p3 = exp2_approx(x[h][nn][3]);
          l[nn][0] += p0 + p2;
          l[nn][1] += p1 + p3;
          const float2 wi = make_float2(winv[nn][0], winv[nn][1]);
          const float2 wa = fmul2(make_float2(p0, p1), fmul2(make_float2(vs[h][0], vs[h][0]), wi));
          const float2 wb = fmul2(make_float2(p2, p3), fmul2(make_float2(vs[h][1], vs[h][1]), wi));
          __half2 a = __float22half2_rn(wa), b = __float22half2_rn(wb);
          const float2 ra = __half22float2(a), rb = __half22float2(b);
          const float take = TWICE && t4 < 2 ? 0.f : 1.f;  // columns 0-3 keep the weight itself
          const __half2 al = __floats2half2_rn(__fmaf_rn(-take, ra.x, wa.x), __fmaf_rn(-take, ra.y, wa.y));
          const __half2 bl = __floats2half2_rn(__fmaf_rn(-take, rb.x, wb.x), __fmaf_rn(-take, rb.y, wb.y));
          w[h][kW - 1][nn][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&al));
          w[h][kW - 1][nn][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&bl));
          if (!TWICE) {
            w[h][0][nn][0] = transpose8x8(*reinterpret_cast<const uint32_t*>(&a));
            w[h][0][nn][1] = transpose8x8(*reinterpret_cast<const uint32_t*>(&b));
          }
        }
      }
      // values: lane (g, t4) holds dims [16 g, 16 g + 16) of its four tokens of a half
#pragma unroll
      for (int jj = 0; jj < 2; ++jj) {
        uint32_t xw[2][4];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          xw[h][0] = *reinterpret_cast<const uint32_t*>(sp + va_off + h * 1024 + 4 * jj) ^ kFlip;
          xw[h][1] = *reinterpret_cast<const uint32_t*>(sp + vb_off + h * 1024 + 4 * jj) ^ kFlip;
          xw[h][2] = *reinterpret_cast<const uint32_t*>(sp + va_off + h * 1024 + 8 * kKvRowBytes + 4 * jj) ^ kFlip;
          xw[h][3] = *reinterpret_cast<const uint32_t*>(sp + vb_off + h * 1024 + 8 * kKvRowBytes + 4 * jj) ^ kFlip;
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const int t = 2 * (2 * jj + j);
          float d[NT][2][4];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t y0 = __byte_perm(xw[h][0], xw[h][1], sel);
            const uint32_t y1 = __byte_perm(xw[h][2], xw[h][3], sel);
            const uint32_t z0 = y0 >> 8, z1 = y1 >> 8;
            const uint32_t a0 = codes_lo(y0), a1 = codes_hi(y0), a2 = codes_lo(y1), a3 = codes_hi(y1);
            const uint32_t b0 = codes_lo(z0), b1 = codes_hi(z0), b2 = codes_lo(z1), b3 = codes_hi(z1);
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
              if (h == 0) {
                const float zero[4] = {0.f, 0.f, 0.f, 0.f};
                mma_f16(d[nn][0], a0, a1, a2, a3, w[h][0][nn][0], w[h][0][nn][1], zero);
                mma_f16(d[nn][1], b0, b1, b2, b3, w[h][0][nn][0], w[h][0][nn][1], zero);
              } else {
                mma_f16(d[nn][0], a0, a1, a2, a3, w[h][0][nn][0], w[h][0][nn][1], d[nn][0]);
                mma_f16(d[nn][1], b0, b1, b2, b3, w[h][0][nn][0], w[h][0][nn][1], d[nn][1]);
              }
              if (!TWICE) {
                mma_f16(d[nn][0], a0, a1, a2, a3, w[h][kW - 1][nn][0], w[h][kW - 1][nn][1], d[nn][0]);
                mma_f16(d[nn][1], b0, b1, b2, b3, w[h][kW - 1][nn][0], w[h][kW - 1][nn][1], d[nn][1]);
              }
            }
          }
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            add4(o[nn][t], d[nn][0]);
            add4(o[nn][t + 1], d[nn][1]);
          }
        }
      }
    }
    __syncwarp();
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) l[nn][k] += __shfl_xor_sync(0xffffffffu, l[nn][k], d);
    const int ta = walk.ta;
    const bool to_end = ta + seg.turns == walk.nt;
    in_units();
    if (ta == 0 && to_end) {
      write_heads(walk.r, first_head(), head_count());
    } else if (ta > 0) {
      keep(0);
      if (lane == 0 && to_end) atomicOr(&sm.ends, 1 << warp);
    } else {
      held = true;  // cut off: this warp's last segment, kept when its turns' bytes are free
    }
  }
  copy_wait<0>();
  __syncwarp();
  if (held) keep(1);
  __syncthreads();

  // ---- pieces of one request and head, added in the order of the warps.  A group is led by a piece 1, or
  // by the first piece 0 when that continues an earlier CTA's; a warp takes one head of it.  Lane
  // 2 w + which knows of piece (w, which).
  const long long my_item = lane < 2 * kWarps ? sm.item[lane >> 1][lane & 1] : -1;
  const bool from_before = (lane & 1) == 0 && my_item >= 0 && my_item + kItemCost < sm.part[0];
  const uint32_t before_mask = __ballot_sync(0xffffffffu, from_before);
  // all pieces 0 from before are of one request and head: the first leads
  uint32_t leads = __ballot_sync(0xffffffffu, (lane & 1) && my_item >= 0) | (before_mask & -before_mask);
  const int my_ends = sm.ends;
#pragma unroll 1
  for (; leads; leads &= leads - 1) {
    const int lead = __ffs(leads) - 1, lw = lead >> 1, which = lead & 1;
    const long long item0 = __shfl_sync(0xffffffffu, my_item, lead);
    const bool member = my_item == item0 && ((lane & 1) ? lane == lead : lane >= lead);
    const uint32_t members = __ballot_sync(0xffffffffu, member);
    const bool complete = which && __any_sync(0xffffffffu, member && !(lane & 1) && ((my_ends >> (lane >> 1)) & 1));
    const int heads = sm.heads[lw][which], row = sm.row[lw][which];
    float* part = p.part + static_cast<size_t>(2 * cta + which) * HB * (kHeadDim + 2);
#pragma unroll 1
    for (int hh = warp; hh < heads; hh += kWarps) {
      const float mo = member ? sm.m[lane >> 1][lane & 1][hh] : kLowest;
      float mx = mo;
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, d));
      mx = __shfl_sync(0xffffffffu, mx, 0);
      const float f = member ? exp2_approx(mo - mx) : 0.f;
      float ls = member ? sm.l[lane >> 1][lane & 1][hh] * f : 0.f;
#pragma unroll
      for (int d = 1; d < 16; d <<= 1) ls += __shfl_xor_sync(0xffffffffu, ls, d);
      ls = __shfl_sync(0xffffffffu, ls, 0);
      const int gg = lane & 7, q = lane >> 3;  // dims 16 gg + 4 q + 0..3
      const int at = (hh >> 3) * kPieceFloats + piece_offset(2 * q, hh & 1, 4 * gg + ((hh & 7) >> 1));
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int w = -1; w < kWarps; ++w) {  // the lead's piece 1, then the pieces 0
        const int src_lane = w < 0 ? lead : 2 * w;
        const float fw = __shfl_sync(0xffffffffu, f, src_lane);
        if (!((members >> src_lane) & 1u) || (w < 0 && !which)) continue;
        const float* src = (w < 0 ? piece(lw, 1) : piece(w, 0)) + at;
        acc[0] += src[0] * fw;
        acc[1] += src[64] * fw;  // rows g + 8 of the same instruction
        acc[2] += src[128] * fw;
        acc[3] += src[192] * fw;
      }
      const int dim = 16 * gg + 4 * q;
      if (complete) {
        const float inv = ls > 0.f ? 1.0f / ls : 0.f;
        const __half2 a = __floats2half2_rn(acc[0] * inv, acc[1] * inv);
        const __half2 b = __floats2half2_rn(acc[2] * inv, acc[3] * inv);
        *reinterpret_cast<uint2*>(p.Y + (static_cast<size_t>(row) + hh) * kHeadDim + dim) =
            make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
      } else {
        *reinterpret_cast<float4*>(part + hh * kHeadDim + dim) = make_float4(acc[0], acc[1], acc[2], acc[3]);
        if (lane == 0) {
          part[HB * kHeadDim + hh] = mx;
          part[HB * kHeadDim + HB + hh] = ls;
        }
      }
    }
    if (!complete && tid == 0) sm.left[which] = lw, sm.join[which] = 1;
  }
  __syncthreads();
  if (tid < 2 && sm.join[tid]) {
    // counted, once every thread's share of the part is written
    const int lw = sm.left[tid];
    const long long t0 = sm.item[lw][tid] + kItemCost;
    const int c_first = cta_of_unit(t0, sm.total, sm.ctas);
    const int parts = cta_of_unit(t0 + sm.turns[lw][tid] - 1, sm.total, sm.ctas) - c_first + 1;
    __threadfence();
    sm.join[tid] = atomicInc(&p.count[c_first], unsigned(parts - 1)) == unsigned(parts - 1);
    sm.turns[lw][tid] = parts;
    sm.item[lw][tid] = c_first;
  }
  __syncthreads();
  for (int which = 0; which < 2; ++which)
    if (sm.join[which]) {
      // the CTA that arrived last joins the parts, in the order of the CTAs
      const int lw = sm.left[which];
      __threadfence();
      join_parts<HB>(p.part, int(sm.item[lw][which]), sm.turns[lw][which], sm.heads[lw][which], sums,
                     p.Y + static_cast<size_t>(sm.row[lw][which]) * kHeadDim);
      __syncthreads();
    }
}

// CTAs of a launch: two per SM with one tile of 8 queries, one with two (their
// registers hold 16 queries' sums).
int attn_nt(int G) { return G > 8 ? 2 : 1; }
int attn_grid(int nt) { return sm_count() * (nt == 1 ? 2 : 1); }

template <int NT, bool TWICE, bool P16>
fq_status launch_attn(const AttnParams& p, cudaStream_t stream) {
  auto kern = kv_attn_kernel<NT, TWICE, P16>;
  constexpr size_t smem = size_t(kWarps) * (kDepth * kStepBytes + NT * kPieceFloats * sizeof(float));
  static std::atomic<uint64_t> allowed{0};
  if (!allow_smem(kern, smem, allowed))
    return fail(FQ_ERR_CUDA, "cannot reserve %zu bytes of shared memory", smem);
  launch_pdl(kern, dim3(attn_grid(NT)), dim3(kAttnThreads), smem, stream, p);
  return check_launch("kv_attn_kernel");
}

}  // namespace
}  // namespace fq

extern "C" {

size_t fq_kv_attn_workspace_size(int R, int Hq, int H) {
  if (R < 1 || R > fq::kMaxAttnR || H < 1 || H > 128 || Hq < H || Hq % H || Hq > 1024) return 0;
  const int nt = fq::attn_nt(Hq / H);
  return fq::sync_block_bytes() + size_t(2) * fq::attn_grid(nt) * 8 * nt * (fq::kHeadDim + 2) * sizeof(float);
}

fq_status fq_kv_attn(const uint16_t* Q, long long ldq, int R, int Hq, const int32_t* len, const int32_t* block_table,
                     int max_pages, const fq_kv_cache* cache, float scale, int window, uint16_t* Y, void* workspace,
                     size_t ws_bytes, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_kv_cache(cache);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(R >= 1 && R <= fq::kMaxAttnR, "R = %d must lie in [1, %d]", R, fq::kMaxAttnR);
  FQ_CHECK_ARG(Hq >= cache->H && Hq % cache->H == 0 && Hq <= 1024,
               "Hq = %d must be a multiple of H = %d, at most 1024", Hq, cache->H);
  FQ_CHECK_ARG(Q && Y && fq::aligned(Q, 16) && fq::aligned(Y, 16), "Q and Y must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(ldq >= static_cast<long long>(Hq) * fq::kHeadDim && ldq % 8 == 0,
               "ldq = %lld must be a multiple of 8 and at least Hq * 128 = %d", ldq, Hq * fq::kHeadDim);
  FQ_CHECK_ARG(len && block_table && fq::aligned(len, 4) && fq::aligned(block_table, 4),
               "len and block_table must be non-NULL and 4-byte aligned");
  FQ_CHECK_ARG(max_pages >= 1 && static_cast<long long>(max_pages) * cache->page_size < (1ll << 31),
               "max_pages = %d: at least 1, and fewer than 2^31 tokens", max_pages);
  FQ_CHECK_ARG(window >= 0, "window = %d must not be negative", window);
  FQ_CHECK_ARG(scale >= -65536.0f && scale <= 65536.0f, "scale = %g must lie in [-65536, 65536]", double(scale));
  const size_t need = fq_kv_attn_workspace_size(R, Hq, cache->H);
  if (!workspace || ws_bytes < need || !fq::aligned(workspace, 256))
    return fq::fail(FQ_ERR_INVALID, "workspace of %zu bytes (256-byte aligned) required, got %zu", need, ws_bytes);
  fq::AttnParams p{};
  p.Q = reinterpret_cast<const __half*>(Q);
  p.ldq = ldq;
  p.R = R;
  p.Hq = Hq;
  p.G = Hq / cache->H;
  const int nt = fq::attn_nt(p.G);
  p.chunks = (p.G + 8 * nt - 1) / (8 * nt);
  p.len = len;
  p.table = block_table;
  p.max_pages = max_pages;
  p.kv = fq::kv_view(cache);
  p.scale_log2 = scale * 1.4426950408889634f;
  p.window = window;
  p.Y = reinterpret_cast<__half*>(Y);
  p.count = static_cast<unsigned*>(workspace) + fq::kJoinCounters;
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + fq::sync_block_bytes());
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool p16 = cache->page_size == 16;
  if (nt == 2) return p16 ? fq::launch_attn<2, false, true>(p, cs) : fq::launch_attn<2, false, false>(p, cs);
  if (p.G > 4) return p16 ? fq::launch_attn<1, false, true>(p, cs) : fq::launch_attn<1, false, false>(p, cs);
  return p16 ? fq::launch_attn<1, true, true>(p, cs) : fq::launch_attn<1, true, false>(p, cs);
}

}  // extern "C"
