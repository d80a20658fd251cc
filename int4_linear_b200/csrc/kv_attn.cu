// Attention of one new token per request over the paged INT4 key/value cache.
//
//   s_i = scale q . k_i,  m = max s_i,  l = sum exp(s_i - m),
//   y = (sum exp(s_i - m) v_i) / l,   k_i, v_i = code * scale
//
// The floor is one read of the cache: 132 bytes per token and key-value head
// against 4 * 128 operations per query head, so the work is a stream of pages
// with the arithmetic hidden under it.  At the measured 6.55 TB/s an SM has
// about 5.7 cycles per token and head, i.e. some 23 warp instructions; turning
// 256 nibbles into operands alone takes 10, so the layout below moves no operand
// through shuffles or a second pass of shared memory.
//
// Division.  The tiles (64 tokens of one request and key-value head) of all
// requests form one sequence, request-major; every CTA takes an equal contiguous
// part of it, found on the GPU from the lengths, so ragged batches load every SM
// alike and a captured launch follows the lengths of its replay.  A part is a run of
// segments (one request and head each).  A segment that covers its whole
// request is finished by its CTA; otherwise the CTA leaves (sum, m, l) in the
// workspace, and the CTA that arrives last adds the parts in their fixed order
// (the sums come out the same whichever CTA that is).
//
// In a CTA eight warps take 16 tokens each in turn, each with its own m, l and sum,
// joined per segment through shared memory.  A warp brings its own tokens
// with 16-byte asynchronous copies several turns ahead and waits for nobody else's.
//
// Products: mma.m16n8k16 (fp16, float32 sums).  The tensor-memory path needs
// 128 rows of queries, and a request has G = Hq / H <= 16 of them per head, so its
// staging of operands would cost more than the product.
//  - scores: A = 16 tokens x 128 dims of K codes, B = 8 queries.  A lane reads 16
//    consecutive bytes of a token's row; the order of the dims inside the product is
//    free, so the queries are arranged once per segment to match the nibbles.  A nibble
//    becomes the fp16 number 64 + (code + 8) by one logic operation; the constant
//    72 sum(q) is taken off through the accumulator's initial value (an error of
//    72 sum|q| 2^-24, 2^-15 of a logit at most for queries and keys of unit size).
//  - sum: A = 128 dims x 16 tokens of V codes (exact), B = the weights, taken
//    from the scores' layout by movmatrix.  A lane reads 8 bytes of each of its 4
//    tokens and pairs two tokens' nibbles by byte permutation.
// Weights: w = exp2(s - m) * (v scale / largest v scale so far) * 2^8 is
// rounded to fp16 (2^-11 relative, independent errors that the sum averages; weights below
// 2^-22 of the largest lose bits, 2^-33 of it at most each).  m is a
// reference that moves only when a score passes it by 2^7 (checked with one vote
// per 16 tokens), so the sums are rarely rescaled.
#include <cuda_fp16.h>

#include <algorithm>

#include "fq_device.cuh"
#include "fq_host.h"
#include "kv_cache.cuh"

namespace fq {

size_t sync_block_bytes();

namespace {

constexpr int kTile = 64;           // tokens per tile of the division
constexpr int kStep = 32;           // tokens per warp and turn, taken as two halves of 16
constexpr int kStepV = kStep * kKvRowBytes, kStepKs = 2 * kStepV, kStepVs = kStepKs + 2 * kStep;
constexpr int kStepBytes = kStepVs + 2 * kStep;  // K codes, V codes, K scales, V scales
constexpr int kDepth = 3;           // turns in flight per warp
constexpr int kWarps = 8;
constexpr int kAttnThreads = kWarps * 32;
constexpr int kHeadPad = 164;       // floats of one head's sums in shared memory (see sum_offset)
constexpr int kMaxAttnR = 16384;
constexpr float kSlack = 7.0f;      // log2 of how far a score may pass the reference
constexpr float kLowest = -1e30f;   // the reference before the first score
constexpr float kWeightScale = 256.0f;

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

struct AttnSmem {
  int r0;                           // the request this CTA starts in, and the tiles before that request
  long long before;
  long long wsum[kWarps];
  float m[kWarps][16], l[kWarps][16];
  int join;
};

// Tiles [t0, t1) and tokens [lo, hi) of request r.
struct Span {
  int lo, hi, t0, t1;
};
__device__ __forceinline__ Span span_of(const AttnParams& p, int r) {
  const long long cap = static_cast<long long>(p.max_pages) << p.kv.page_shift;
  Span s;
  s.hi = int(min(static_cast<long long>(max(p.len[r], 0)), cap));
  s.lo = p.window > 0 ? max(0, s.hi - p.window) : 0;
  s.t0 = s.lo / kTile;
  s.t1 = s.hi > s.lo ? (s.hi - 1) / kTile + 1 : s.t0;
  return s;
}

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

__device__ __forceinline__ uint32_t transpose8x8(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

// (a & b) ^ c in one logic operation.
__device__ __forceinline__ uint32_t and_xor(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(d) : "r"(a), "r"(b), "r"(c));
  return d;
}
// Nibbles of each half word (two's complement codes q) at bits 0-3 and 4-7 -> the fp16 numbers
// (q + 8) 2^-24 and (q + 8) 2^-20 (subnormal: the nibble is the mantissa).
__device__ __forceinline__ uint32_t codes_lo(uint32_t w) { return and_xor(w, 0x000F000Fu, 0x00080008u); }
__device__ __forceinline__ uint32_t codes_hi(uint32_t w) { return and_xor(w, 0x00F000F0u, 0x00800080u); }

// The token of score row i (0..15): rows 2t, 2t + 1 of one lane's weights.  Bit 0
// alternates within a row pair (score reads of two rows hit different banks)
// and with t (the four lanes of a value read hit two bank halves).
__device__ __forceinline__ int token_of_row(int i) {
  const int t = (i >> 1) & 3, b = i & 1;
  return (b ^ (t & 1)) | ((t & 1) << 1) | ((t >> 1) << 2) | (i & 8);
}

// Where dim 16 g + d of a head's sums lies in shared memory: lanes with
// consecutive g write, and lanes with consecutive (d / 4, g) read, distinct banks.
__device__ __forceinline__ int sum_offset(int g, int d) { return d * 8 + (d >> 2) * 8 + g; }

__device__ __forceinline__ void copy16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// The CTA whose part holds tile x of the sequence: parts are [total c / C, total (c + 1) / C).
__device__ __forceinline__ int cta_of_tile(long long x, long long total, int C) {
  return int(((x + 1) * C - 1) / total);
}

// NT: tiles of 8 query heads; P16: pages of 16 tokens, so that a turn spans two.
template <int NT, bool P16>
__global__ void __launch_bounds__(kAttnThreads, NT == 1 ? 2 : 1) kv_attn_kernel(const AttnParams p) {
  constexpr int HB = 8 * NT;
  // the warps' turns in flight; between segments the eight warps' sums, [warps][8][kHeadPad]
  extern __shared__ __align__(128) uint8_t dyn[];
  float* sums = reinterpret_cast<float*>(dyn);
  __shared__ AttnSmem sm;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = blockIdx.x, HC = p.kv.H * p.chunks;
  pdl_launch_dependents();
  pdl_wait();

  // ---- this CTA's part: tiles of each thread's run of requests, summed
  const int run = (p.R + kAttnThreads - 1) / kAttnThreads;
  const int ra = min(p.R, tid * run), rb = min(p.R, ra + run);
  long long mine = 0;
  for (int r = ra; r < rb; ++r) {
    const Span s = span_of(p, r);
    mine += s.t1 - s.t0;
  }
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long u = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += u;
  }
  if (lane == 31) sm.wsum[warp] = incl;
  __syncthreads();
  long long base = 0, all = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) base += sm.wsum[w];
    all += sm.wsum[w];
  }
  const long long total = all * HC;
  // few tiles: fewer CTAs, so that a part is worth its join
  const int C = int(min(static_cast<long long>(gridDim.x), (total + 1) / 2));
  // requests without tokens
  for (int r = cta; r < p.R; r += gridDim.x) {
    const Span s = span_of(p, r);
    if (s.t1 == s.t0)
      for (int i = tid; i < p.Hq * kHeadDim / 8; i += kAttnThreads)
        reinterpret_cast<uint4*>(p.Y + static_cast<size_t>(r) * p.Hq * kHeadDim)[i] = make_uint4(0, 0, 0, 0);
  }
  if (cta >= C) return;
  const long long first = total * cta / C, last = total * (cta + 1) / C;
  {
    const long long e0 = (base + incl - mine) * HC, e1 = (base + incl) * HC;
    if (e0 <= first && first < e1) {
      long long acc = e0;
      for (int r = ra; r < rb; ++r) {
        const Span s = span_of(p, r);
        const long long n = static_cast<long long>(s.t1 - s.t0) * HC;
        if (first < acc + n) {
          sm.r0 = r;
          sm.before = acc;
          break;
        }
        acc += n;
      }
    }
  }
  __syncthreads();

  int r = sm.r0;
  long long pos = first, before = sm.before;  // next tile; tiles before request r
  const int ps = p.kv.page_shift;
  const int g = lane >> 2, t4 = lane & 3;
  // what this lane copies of a turn: every 32nd 16-byte piece of the K and of the V codes, and lanes
  // 0-7 (pages of 16: 0-3 of each page) a piece of the scales
  constexpr int kHalves = P16 ? 2 : 1;
  constexpr int kPieces = P16 ? 2 : 4;        // 512-byte pieces of one kind of codes per page taken
  constexpr int kScalePieces = P16 ? 2 : 4;   // 16-byte pieces of one kind of scales per page taken
  const uint32_t my_ring = smem_u32(dyn) + uint32_t(warp * kDepth * kStepBytes);
  const int sc_src = (2 * kKvRowBytes << ps) + (lane % kScalePieces) * 16 + (lane / kScalePieces & 1) * (2 << ps);
  const uint32_t sc_dst = kStepKs + (lane % kScalePieces) * 16 + (lane / kScalePieces & 1) * (2 * kStep);
  // byte offsets inside a turn of this lane's operands
  const int row0 = token_of_row(g);           // score rows g and g + 8 of a half: tokens row0, row0 + 8
  const uint8_t* ring = dyn + warp * kDepth * kStepBytes;
  const int k_off = row0 * kKvRowBytes + t4 * 16;
  const int va_off = kStepV + token_of_row(2 * t4) * kKvRowBytes + 8 * g;
  const int vb_off = kStepV + token_of_row(2 * t4 + 1) * kKvRowBytes + 8 * g;
  while (pos < last) {
    const Span s = span_of(p, r);
    const int nt = s.t1 - s.t0;
    const long long len_r = static_cast<long long>(nt) * HC;
    if (pos >= before + len_r) {
      before += len_r;
      ++r;
      continue;
    }
    const int hc = int((pos - before) / nt), ta = int((pos - before) % nt);
    const int tb = int(min(static_cast<long long>(nt), ta + (last - pos)));
    const int head = hc / p.chunks, q0 = head * p.G + (hc % p.chunks) * HB;  // first query head
    const int heads = min(HB, p.G - (hc % p.chunks) * HB);

    // ---- this warp's turns: 32 tokens at tok0 + 256 i
    const int tok0 = (s.t0 + ta) * kTile + warp * kStep;
    const int tok_end = min(s.hi, (s.t0 + tb) * kTile);
    const int turns = tok0 < tok_end ? (tok_end - 1 - tok0) / (kWarps * kStep) + 1 : 0;
    const int32_t* row = p.table + static_cast<size_t>(r) * p.max_pages;
    struct Ids {
      int id[kHalves];
    };
    auto page_ids = [&](int i) {
      Ids v;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        const int t = tok0 + i * (kWarps * kStep) + 16 * h;
        const bool in = i < turns && t + (P16 ? 16 : kStep) > s.lo && t < tok_end;
        v.id[h] = in ? __ldg(row + (t >> ps)) : -1;
      }
      return v;
    };
    uint32_t loaded = 0;  // bits 2 j, 2 j + 1: the halves of the turn fetched j turns ago have their tokens
    auto fetch = [&](int i, const Ids& ids, int slot) {
      loaded <<= 2;
#pragma unroll
      for (int h = 0; h < kHalves; ++h) {
        if (ids.id[h] >= 0 && ids.id[h] < p.kv.num_pages) {
          const int off = P16 ? 0 : (tok0 + i * (kWarps * kStep)) & ((1 << ps) - 1);
          const uint8_t* src = p.kv.block(ids.id[h], head);
          const uint32_t dst = my_ring + uint32_t(slot * kStepBytes);
          const uint8_t* k = src + off * kKvRowBytes + lane * 16;
          const uint8_t* v = k + (kKvRowBytes << ps);
          const uint32_t d = dst + h * 1024 + lane * 16;
#pragma unroll
          for (int c = 0; c < kPieces; ++c) {
            copy16(d + 512 * c, k + 512 * c);
            copy16(d + kStepV + 512 * c, v + 512 * c);
          }
          if (lane < 2 * kScalePieces) copy16(dst + sc_dst + h * 32, src + sc_src + 2 * off);
          loaded |= P16 ? 1u << h : 3u;
        }
      }
      copy_commit();
    };
    Ids next_ids;
    {
      Ids ids[kDepth - 1];
#pragma unroll
      for (int i = 0; i < kDepth - 1; ++i) ids[i] = page_ids(i);
      next_ids = page_ids(kDepth - 1);
#pragma unroll
      for (int i = 0; i < kDepth - 1; ++i) fetch(i, ids[i], i);
    }

    // queries of this segment in 16-bit fixed point, two signed bytes: q = unit (256 hi + lo).  Lane
    // (g, t4) holds head g, dims [32 t4, 32 t4 + 32): the even dims of 8 in one word, the odd ones in the next
    uint32_t qf[NT][2][8];
    float unit[NT][2];  // of heads 2 t4, 2 t4 + 1, times the score's scale and 1/16 (a nibble is taken 16-fold)
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
      uint4 w[4];
      __half2 m2 = __float2half2_rn(0.f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        w[j] = make_uint4(0, 0, 0, 0);
        if (nn * 8 + g < heads)
          w[j] = *reinterpret_cast<const uint4*>(p.Q + static_cast<long long>(r) * p.ldq +
                                                 (q0 + nn * 8 + g) * kHeadDim + 32 * t4 + 8 * j);
        const __half2* h2 = reinterpret_cast<const __half2*>(&w[j]);
#pragma unroll
        for (int k = 0; k < 4; ++k) m2 = __hmax2(m2, __habs2(h2[k]));
      }
      float mq = __half2float(__hmax(__low2half(m2), __high2half(m2)));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 1));
      mq = fmaxf(mq, __shfl_xor_sync(0xffffffffu, mq, 2));
      const float inv = mq > 0.f ? 32639.0f / mq : 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const __half2* h2 = reinterpret_cast<const __half2*>(&w[j]);
        uint32_t hi[2] = {0, 0}, lo[2] = {0, 0};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __half22float2(h2[k]);
          const int ev = __float2int_rn(f.x * inv), od = __float2int_rn(f.y * inv);
          const int eh = (ev + 128) >> 8, oh = (od + 128) >> 8;
          hi[0] |= (uint32_t(eh) & 255u) << (8 * k);
          hi[1] |= (uint32_t(oh) & 255u) << (8 * k);
          lo[0] |= (uint32_t(ev) & 255u) << (8 * k);
          lo[1] |= (uint32_t(od) & 255u) << (8 * k);
        }
        qf[nn][0][2 * j] = hi[0];
        qf[nn][0][2 * j + 1] = hi[1];
        qf[nn][1][2 * j] = lo[0];
        qf[nn][1][2 * j + 1] = lo[1];
      }
      const float u = mq * (p.scale_log2 / (16.0f * 32639.0f));
      unit[nn][0] = __shfl_sync(0xffffffffu, u, 8 * t4);
      unit[nn][1] = __shfl_sync(0xffffffffu, u, 8 * t4 + 4);
    }
    float o[NT][8][4];
    float m[NT][2], l[NT][2];
    float vcap = 0.f, vinv = 0.f;  // largest v scale so far, and 2^8 over it
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) o[nn][i][k] = 0.f;
      m[nn][0] = m[nn][1] = kLowest;
      l[nn][0] = l[nn][1] = 0.f;
    }

    int slot = 0;
    for (int i = 0; i < turns; ++i) {
      copy_wait<kDepth - 2>();
      __syncwarp();  // every lane's copies of this turn, and every lane is done with the last one
      {
        const Ids ids = next_ids;
        next_ids = page_ids(i + kDepth);
        fetch(i + kDepth - 1, ids, slot == 0 ? kDepth - 1 : slot - 1);
      }
      const uint8_t* sp = ring + slot * kStepBytes;
      slot = slot == kDepth - 1 ? 0 : slot + 1;
      const uint32_t have = (loaded >> (2 * (kDepth - 1))) & 3u;
      if (have == 0u) continue;
      // scores of the 32 tokens: rows g, g + 8 of both halves
      float sc[2][NT][4], ks[2][2], vs[2][2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 k0 = *reinterpret_cast<const uint4*>(sp + k_off + h * 1024);
        const uint4 k1 = *reinterpret_cast<const uint4*>(sp + k_off + h * 1024 + 8 * kKvRowBytes);
        const uint32_t kw0[4] = {k0.x, k0.y, k0.z, k0.w}, kw1[4] = {k1.x, k1.y, k1.z, k1.w};
        int ah[NT][4], al[NT][4];
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
          for (int k = 0; k < 4; ++k) ah[nn][k] = al[nn][k] = 0;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t e0, d0, e1, d1;  // 16 q of the even and odd dims of rows g and g + 8
          unpack8_hi(kw0[j], e0, d0);
          unpack8_hi(kw1[j], e1, d1);
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            mma_s8(ah[nn], e0, e1, d0, d1, qf[nn][0][2 * j], qf[nn][0][2 * j + 1]);
            mma_s8(al[nn], e0, e1, d0, d1, qf[nn][1][2 * j], qf[nn][1][2 * j + 1]);
          }
        }
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
          for (int k = 0; k < 4; ++k) sc[h][nn][k] = float(ah[nn][k] * 256 + al[nn][k]) * unit[nn][k & 1];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          ks[h][k] = __half2float(*reinterpret_cast<const __half*>(sp + kStepKs + 2 * (row0 + 16 * h + 8 * k)));
          vs[h][k] = __half2float(*reinterpret_cast<const __half*>(sp + kStepVs + 2 * (row0 + 16 * h + 8 * k)));
        }
      }
      const int at = tok0 + i * (kWarps * kStep);
      if (at < s.lo || at + kStep > s.hi || have != 3u) {
        // what is masked scores -inf and weighs 0, whatever its scales hold
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int t = at + row0 + 16 * h + 8 * k;
            const bool ok = t >= s.lo && t < s.hi && ((have >> h) & 1u);
            ks[h][k] = ok ? ks[h][k] : 1.0f;
            vs[h][k] = ok ? vs[h][k] : 0.0f;
#pragma unroll
            for (int nn = 0; nn < NT; ++nn) {
              sc[h][nn][2 * k] = ok ? sc[h][nn][2 * k] : -INFINITY;
              sc[h][nn][2 * k + 1] = ok ? sc[h][nn][2 * k + 1] : -INFINITY;
            }
          }
      }
      // log2 of the weights before the v scale, and whether one passes its reference by too much
      const float vtop = fmaxf(fmaxf(vs[0][0], vs[0][1]), fmaxf(vs[1][0], vs[1][1]));
      float x[2][NT][4], top = -INFINITY;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int nn = 0; nn < NT; ++nn)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            x[h][nn][k] = __fmaf_rn(sc[h][nn][k], ks[h][k >> 1], -m[nn][k & 1]);
            top = fmaxf(top, x[h][nn][k]);
          }
      if (__any_sync(0xffffffffu, top > kSlack || vtop > vcap)) {
        // new references: the largest score of each head, the largest v scale
        float vm = fmaxf(vtop, vcap);
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) vm = fmaxf(vm, __shfl_xor_sync(0xffffffffu, vm, d));
        const float vf = vm > 0.f ? vcap / vm : 0.f;
        vcap = vm;
        vinv = vm > 0.f ? kWeightScale / vm : 0.f;
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
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
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              x[h][nn][k] = __fmaf_rn(sc[h][nn][k], ks[h][0], -mx);
              x[h][nn][k + 2] = __fmaf_rn(sc[h][nn][k + 2], ks[h][1], -mx);
            }
            l[nn][k] *= f;
#pragma unroll
            for (int i8 = 0; i8 < 8; ++i8) {
              o[nn][i8][k] *= f * vf;
              o[nn][i8][k + 2] *= f * vf;
            }
          }
        }
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t w0[NT], w1[NT];
        float c8[NT][4];  // -8 sum(w): rows g in the units of codes_lo, rows g + 8 of codes_hi
        const float v0 = vs[h][0] * vinv, v1 = vs[h][1] * vinv;
#pragma unroll
        for (int nn = 0; nn < NT; ++nn) {
          const float p0 = exp2_approx(x[h][nn][0]), p1 = exp2_approx(x[h][nn][1]);
          const float p2 = exp2_approx(x[h][nn][2]), p3 = exp2_approx(x[h][nn][3]);
          l[nn][0] += p0 + p2;
          l[nn][1] += p1 + p3;
          const __half2 a = __floats2half2_rn(p0 * v0, p1 * v0), b = __floats2half2_rn(p2 * v1, p3 * v1);
          w0[nn] = transpose8x8(*reinterpret_cast<const uint32_t*>(&a));
          w1[nn] = transpose8x8(*reinterpret_cast<const uint32_t*>(&b));
          const float zero[4] = {0.f, 0.f, 0.f, 0.f};
          // -2^-21 = -8 2^-24 and -2^-17 = -8 2^-20 as fp16
          mma_f16(c8[nn], 0x80088008u, 0x80808080u, 0x80088008u, 0x80808080u, w0[nn], w1[nn], zero);
        }
        // values: lane (g, t4) holds dims [16 g, 16 g + 16) of its four tokens
        const uint2 x0 = *reinterpret_cast<const uint2*>(sp + va_off + h * 1024);
        const uint2 x1 = *reinterpret_cast<const uint2*>(sp + vb_off + h * 1024);
        const uint2 x2 = *reinterpret_cast<const uint2*>(sp + va_off + h * 1024 + 8 * kKvRowBytes);
        const uint2 x3 = *reinterpret_cast<const uint2*>(sp + vb_off + h * 1024 + 8 * kKvRowBytes);
#pragma unroll
        for (int j = 0; j < 4; ++j) {  // four dims: half word j of the 16 dims
          const uint32_t sel = (j & 1) ? 0x7632u : 0x5410u;
          const uint32_t y0 = __byte_perm(j < 2 ? x0.x : x0.y, j < 2 ? x1.x : x1.y, sel);
          const uint32_t y1 = __byte_perm(j < 2 ? x2.x : x2.y, j < 2 ? x3.x : x3.y, sel);
          const uint32_t z0 = y0 >> 8, z1 = y1 >> 8;
          // dims 4 j (rows g, in units of 2^-24), 4 j + 1 (rows g + 8, 2^-20); 4 j + 2, 4 j + 3
          const uint32_t a0 = codes_lo(y0), a1 = codes_hi(y0), a2 = codes_lo(y1), a3 = codes_hi(y1);
          const uint32_t b0 = codes_lo(z0), b1 = codes_hi(z0), b2 = codes_lo(z1), b3 = codes_hi(z1);
#pragma unroll
          for (int nn = 0; nn < NT; ++nn) {
            float d[4];
            mma_f16(d, a0, a1, a2, a3, w0[nn], w1[nn], c8[nn]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nn][2 * j][k] += d[k];
            mma_f16(d, b0, b1, b2, b3, w0[nn], w1[nn], c8[nn]);
#pragma unroll
            for (int k = 0; k < 4; ++k) o[nn][2 * j + 1][k] += d[k];
          }
        }
      }
    }
    copy_wait<0>();

    // ---- the eight warps' parts of the segment
#pragma unroll
    for (int nn = 0; nn < NT; ++nn)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float v = l[nn][k];
#pragma unroll
        for (int d = 4; d < 32; d <<= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
        if (g == 0) {
          sm.m[warp][nn * 8 + 2 * t4 + k] = m[nn][k];
          sm.l[warp][nn * 8 + 2 * t4 + k] = v;
        }
      }
    __syncthreads();  // also: every warp is done with its turns, whose bytes the sums take
    const long long item0 = before + static_cast<long long>(hc) * nt;  // the request and head's tiles in the sequence
    const bool whole = ta == 0 && tb == nt;
    const int c_first = cta_of_tile(item0, total, C);
    const int parts = cta_of_tile(item0 + nt - 1, total, C) - c_first + 1;
    float* part = p.part + static_cast<size_t>(2 * cta + (ta == 0 ? 1 : 0)) * HB * (kHeadDim + 2);
#pragma unroll
    for (int nn = 0; nn < NT; ++nn) {
      // 1. every warp's sums at the common reference
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        float mx = kLowest;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) mx = fmaxf(mx, sm.m[w][nn * 8 + 2 * t4 + k]);
        const float f = exp2_approx(m[nn][k] - mx) * (vcap * (1.0f / kWeightScale));
        const float flo = f * 0x1p24f, fhi = f * 0x1p20f;  // rows g hold 2^-24, rows g + 8 2^-20 of the sums
        float* dst = sums + (warp * 8 + 2 * t4 + k) * kHeadPad;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = 4 * (i >> 1) + 2 * (i & 1);
          dst[sum_offset(g, d)] = o[nn][i][k] * flo;
          dst[sum_offset(g, d + 1)] = o[nn][i][k + 2] * fhi;
        }
      }
      __syncthreads();
      // 2. added over the warps: this thread takes head `warp`, dims 16 (lane % 8) + 4 (lane / 8) + 0..3
      const int hh = nn * 8 + warp;
      const int gg = lane & 7, d4 = lane >> 3;
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
      float mx = kLowest, ls = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const float* src = sums + (w * 8 + warp) * kHeadPad;
#pragma unroll
        for (int k = 0; k < 4; ++k) acc[k] += src[sum_offset(gg, 4 * d4 + k)];
        mx = fmaxf(mx, sm.m[w][hh]);
      }
#pragma unroll
      for (int w = 0; w < kWarps; ++w) ls += sm.l[w][hh] * exp2_approx(sm.m[w][hh] - mx);
      if (hh < heads) {
        const int dim = 16 * gg + 4 * d4;
        if (whole) {
          const float inv = ls > 0.f ? 1.0f / ls : 0.f;
          const __half2 a = __floats2half2_rn(acc[0] * inv, acc[1] * inv);
          const __half2 b = __floats2half2_rn(acc[2] * inv, acc[3] * inv);
          *reinterpret_cast<uint2*>(p.Y + (static_cast<size_t>(r) * p.Hq + q0 + hh) * kHeadDim + dim) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        } else {
          *reinterpret_cast<float4*>(part + hh * kHeadDim + dim) = make_float4(acc[0], acc[1], acc[2], acc[3]);
          if (lane == 0) {
            part[HB * kHeadDim + hh] = mx;
            part[HB * kHeadDim + HB + hh] = ls;
          }
        }
      }
      if (nn + 1 < NT) __syncthreads();
    }
    if (!whole) {
      // 3. the CTA that arrives last joins the parts, in the order of the CTAs
      __threadfence();
      __syncthreads();
      if (tid == 0) sm.join = atomicInc(&p.count[c_first], unsigned(parts - 1)) == unsigned(parts - 1);
      __syncthreads();
      if (sm.join) {
        __threadfence();
        const size_t stride = static_cast<size_t>(HB) * (kHeadDim + 2);
        for (int hh = warp; hh < heads; hh += kWarps) {
          float mx = kLowest;
          for (int c = 0; c < parts; ++c)
            mx = fmaxf(mx, __ldcg(p.part + (2 * (c_first + c) + (c == 0)) * stride + HB * kHeadDim + hh));
          float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
          float ls = 0.f;
          for (int c = 0; c < parts; ++c) {
            const float* src = p.part + (2 * (c_first + c) + (c == 0)) * stride;
            const float f = exp2_approx(__ldcg(src + HB * kHeadDim + hh) - mx);
            ls += __ldcg(src + HB * kHeadDim + HB + hh) * f;
            const float4 v = __ldcg(reinterpret_cast<const float4*>(src + hh * kHeadDim) + lane);
            acc.x += v.x * f;
            acc.y += v.y * f;
            acc.z += v.z * f;
            acc.w += v.w * f;
          }
          const float inv = ls > 0.f ? 1.0f / ls : 0.f;
          const __half2 a = __floats2half2_rn(acc.x * inv, acc.y * inv);
          const __half2 b = __floats2half2_rn(acc.z * inv, acc.w * inv);
          *reinterpret_cast<uint2*>(p.Y + (static_cast<size_t>(r) * p.Hq + q0 + hh) * kHeadDim + 4 * lane) =
              make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
        }
      }
    }
    pos += tb - ta;
    // the next segment's copies and writes to sm follow every warp's reads above
    __syncthreads();
  }
}

constexpr size_t kAttnSmem = size_t(kWarps) * kDepth * kStepBytes;
static_assert(kAttnSmem >= size_t(kWarps) * 8 * kHeadPad * sizeof(float), "the sums take the turns' bytes");

// CTAs of a launch: two per SM with one tile of 8 queries, one with two (their
// registers hold 16 queries' sums).
int attn_nt(int G) { return G > 8 ? 2 : 1; }
int attn_grid(int nt) { return sm_count() * (nt == 1 ? 2 : 1); }

template <int NT, bool P16>
fq_status launch_attn(const AttnParams& p, cudaStream_t stream) {
  auto kern = kv_attn_kernel<NT, P16>;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, int(kAttnSmem)) != cudaSuccess)
    return fail(FQ_ERR_CUDA, "cannot reserve %zu bytes of shared memory", kAttnSmem);
  launch_pdl(kern, dim3(attn_grid(NT)), dim3(kAttnThreads), kAttnSmem, stream, p);
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
  FQ_CHECK_ARG(scale == scale && scale - scale == 0.f, "scale must be finite");
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
  p.count = static_cast<unsigned*>(workspace);
  p.part = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + fq::sync_block_bytes());
  cudaStream_t cs = static_cast<cudaStream_t>(stream);
  const bool p16 = cache->page_size == 16;
  if (nt == 1) return p16 ? fq::launch_attn<1, true>(p, cs) : fq::launch_attn<1, false>(p, cs);
  return p16 ? fq::launch_attn<2, true>(p, cs) : fq::launch_attn<2, false>(p, cs);
}

}  // extern "C"
