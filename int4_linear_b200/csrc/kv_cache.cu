// The paged INT4 key/value cache: block tables and slots of a step, new keys
// and values into their pages, cached tokens back to fp16.
#include <cuda_fp16.h>

#include <algorithm>

#include "fq_device.cuh"
#include "fq_host.h"
#include "kv_cache.cuh"

namespace fq {

fq_status check_kv_cache(const fq_kv_cache* c) {
  FQ_CHECK_ARG(c != nullptr, "cache is NULL");
  FQ_CHECK_ARG(c->pool && aligned(c->pool, 16), "the cache pool must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(c->page_size == 16 || c->page_size == 32 || c->page_size == 64 || c->page_size == 128,
               "page_size = %d must be 16, 32, 64 or 128", c->page_size);
  FQ_CHECK_ARG(c->H >= 1 && c->H <= 128, "H = %d must lie in [1, 128]", c->H);
  FQ_CHECK_ARG(c->num_pages >= 1 && static_cast<long long>(c->num_pages) * c->page_size < (1ll << 31),
               "num_pages = %d of %d tokens: at least 1, and fewer than 2^31 tokens", c->num_pages, c->page_size);
  return FQ_OK;
}

KvView kv_view(const fq_kv_cache* c) {
  KvView v;
  v.pool = c->pool;
  v.num_pages = c->num_pages;
  v.page_shift = c->page_size == 16 ? 4 : c->page_size == 32 ? 5 : c->page_size == 64 ? 6 : 7;
  v.H = c->H;
  return v;
}

namespace {

// ------------------------------------------------------------------ block tables and slots

constexpr int kPlanThreads = 1024;
constexpr int kPlanMaxR = 16384;

struct PlanParams {
  const int32_t *len, *fresh, *free_pages, *used;
  int32_t *table, *len_out, *start, *slots, *used_out;
  int R, page_shift, max_pages, num_free, max_tokens;
};

// Inclusive sum of v over the block's threads; `total` is the block's sum.
// Every thread calls it; `part` holds 33 words.
__device__ __forceinline__ int block_inclusive_sum(int v, int* part, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, o);
    if (lane >= o) v += u;
  }
  if (lane == 31) part[warp] = v;
  __syncthreads();
  if (warp == 0) {
    int w = part[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int u = __shfl_up_sync(0xffffffffu, w, o);
      if (lane >= o) w += u;
    }
    part[lane] = w;
  }
  __syncthreads();
  total = part[31];
  const int base = warp ? part[warp - 1] : 0;
  __syncthreads();  // part is free again
  return base + v;
}

// Last index i in [0, n) with a[i] <= x (a ascending, a[0] <= x).
__device__ __forceinline__ int last_not_above(const int* a, int n, int x) {
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

// Two exclusive sums over the requests (rows of the step's batch, then pages
// asked for) in every CTA, then one thread per row of the batch and per fresh
// page, which finds its request by bisection.  Bound by latency: two dependent
// loads (lengths, then a table or free-list entry), a few barriers.  The CTAs of a
// cluster repeat the sums, which cost less than passing them on, and share the
// rows; the cluster barrier between the last read of the lengths and the first
// write lets len_out be len and pages_used_out be pages_used.  64 requests of one new token each: 3.9 us.
__global__ void __launch_bounds__(kPlanThreads) kv_plan_kernel(const PlanParams p) {
  extern __shared__ int sm[];
  int* s_start = sm;            // [R] first row of each request
  int* s_first = sm + p.R;      // [R] pages asked for before it
  int* s_len = sm + 2 * p.R;    // [R] tokens held; ~held when the request is refused
  __shared__ int part[33];
  const int tid = threadIdx.x;
  const int rank = int(blockIdx.x), ncta = int(gridDim.x);
  const int page = 1 << p.page_shift;
  pdl_launch_dependents();
  pdl_wait();
  const int used = max(*p.used, 0);
  const int avail = p.num_free - used;
  int tok0 = 0, ask0 = 0, taken = 0;
  for (int base = 0; base < p.R; base += kPlanThreads) {
    const int r = base + tid;
    int ln = 0, nw = 0;
    if (r < p.R) {
      ln = max(p.len[r], 0);
      nw = max(p.fresh[r], 0);
    }
    int total;
    const int end = tok0 + block_inclusive_sum(nw, part, total);
    tok0 += total;
    const int held = int((static_cast<long long>(ln) + page - 1) >> p.page_shift);
    const long long want = (static_cast<long long>(ln) + nw + page - 1) >> p.page_shift;
    const bool fits = want <= p.max_pages && end <= p.max_tokens;
    const int need = fits ? int(want) - held : 0;
    const int asked = ask0 + block_inclusive_sum(need, part, total);
    ask0 += total;
    const bool granted = fits && (need == 0 || asked <= avail);
    if (r < p.R) {
      s_start[r] = end - nw;
      s_first[r] = asked - need;
      s_len[r] = granted ? ln : ~ln;
    }
    // the granted requests that need pages come first in asking order
    int grant_end = granted && need ? asked : 0;
#pragma unroll
    for (int o = 16; o; o >>= 1) grant_end = max(grant_end, __shfl_xor_sync(0xffffffffu, grant_end, o));
    if ((tid & 31) == 0) part[tid >> 5] = grant_end;
    __syncthreads();
    grant_end = part[tid & 31];
#pragma unroll
    for (int o = 16; o; o >>= 1) grant_end = max(grant_end, __shfl_xor_sync(0xffffffffu, grant_end, o));
    taken = max(taken, grant_end);
    __syncthreads();
  }
  if (ncta > 1)
    cluster_sync();
  else
    __syncthreads();
  const int tokens = tok0;
  // per request
  for (int r = rank * kPlanThreads + tid; r < p.R; r += ncta * kPlanThreads) {
    const int l = s_len[r];
    const int nw = (r + 1 < p.R ? s_start[r + 1] : tokens) - s_start[r];
    p.len_out[r] = l >= 0 ? l + nw : ~l;
    p.start[r] = s_start[r];
  }
  if (rank == 0 && tid == 0) {
    p.start[p.R] = tokens;
    *p.used_out = used + taken;
  }
  // per fresh page
  for (int j = rank * kPlanThreads + tid; j < taken; j += ncta * kPlanThreads) {
    const int r = last_not_above(s_first, p.R, j);
    const int held = (s_len[r] + page - 1) >> p.page_shift;
    p.table[size_t(r) * p.max_pages + held + (j - s_first[r])] = p.free_pages[used + j];
  }
  // per row of the batch, four at a time so that their searches and loads overlap; a page that this
  // step takes is read from the free list, so that no CTA waits for another's table entries
  const int stride = ncta * kPlanThreads;
  for (int i0 = rank * kPlanThreads + tid; i0 < p.max_tokens; i0 += 4 * stride) {
    int lo[4], hi[4], slot[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      lo[u] = 0;
      hi[u] = p.R;
    }
    while (hi[0] - lo[0] > 1) {  // the same number of halvings for all, give or take one
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int mid = (lo[u] + hi[u]) >> 1;
        if (s_start[mid] <= i0 + u * stride)
          lo[u] = mid;
        else
          hi[u] = mid;
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int i = i0 + u * stride;
      while (hi[u] - lo[u] > 1) {
        const int mid = (lo[u] + hi[u]) >> 1;
        if (s_start[mid] <= i)
          lo[u] = mid;
        else
          hi[u] = mid;
      }
      slot[u] = -1;
      const int r = lo[u], l = s_len[r];
      if (i < tokens && l >= 0) {
        const int pos = l + (i - s_start[r]);
        const int pi = pos >> p.page_shift, held = (l + page - 1) >> p.page_shift;
        const int id = pi < held ? p.table[size_t(r) * p.max_pages + pi] : p.free_pages[used + s_first[r] + pi - held];
        if (uint32_t(id) < 1u << (31 - p.page_shift)) slot[u] = id * page + (pos & (page - 1));  // no page of any cache otherwise
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (i0 + u * stride < p.max_tokens) p.slots[i0 + u * stride] = slot[u];
  }
}

// ------------------------------------------------------------------ into and out of the pages

constexpr int kRowThreads = 256;

// Codes clamp(round-half-even(v / s), -8, 7) of eight fp16 values and an fp16 scale s > 0, packed.
// v and s have 11 bits each, so v / s is a tie (k + 1/2) or at least 2^-12 from one.  v * inv, off by
// less than 2^-18, is therefore first rounded to a multiple of 2^-13 (by adding 1.5 * 2^10), which makes a tie
// exact and moves nothing else across one, then to an integer (by adding 1.5 * 2^23), ties to even:
// two float32 operations where an IEEE division and its rounding take some fifteen.  Quotients lie in [-8.25, 7.25].
__device__ __forceinline__ uint32_t codes8(const __half2 (&v)[4], float inv) {
  constexpr float kFine = 1536.0f, kWhole = 12582912.0f;
  uint32_t even[4], odd[4];  // codes in the low bits
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = __half22float2(v[j]);
    const float2 a = ffma2(f, make_float2(inv, inv), make_float2(kFine, kFine));
    const float2 q = fadd2(a, make_float2(kWhole - kFine, kWhole - kFine));
    even[j] = __float_as_uint(q.x);
    odd[j] = __float_as_uint(q.y);
  }
  const uint32_t e = __byte_perm(__byte_perm(even[0], even[1], 0x0040), __byte_perm(even[2], even[3], 0x0040), 0x5410);
  const uint32_t o = __byte_perm(__byte_perm(odd[0], odd[1], 0x0040), __byte_perm(odd[2], odd[3], 0x0040), 0x5410);
  return (e & 0x0F0F0F0Fu) | ((o << 4) & 0xF0F0F0F0u);
}

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// Token, head and kind (0 key, 1 value) of a head vector, a token's vectors being its H keys, then its H values.
struct KvVec {
  long long t;
  int h, which;
};
// What the vectors of one thread, a grid apart, are apart in tokens and in a token's vectors.
struct KvStep {
  long long vecs, tokens;
  int rest;
};
// A thread's vectors: one division to begin with instead of one per vector.
struct KvWalk {
  long long t, dt;
  int r, dr, H;
  __device__ __forceinline__ KvWalk(long long vec, const KvStep& step, int heads)
      : dt(step.tokens), dr(step.rest), H(heads) {
    const uint32_t per = 2u * uint32_t(H);
    t = (vec >> 32) == 0 ? uint32_t(vec) / per : vec / per;
    r = int(vec - t * per);
  }
  __device__ __forceinline__ KvVec next() {
    const int which = r >= H;
    const KvVec v{t, which ? r - H : r, which};
    t += dt;
    r += dr;
    if (r >= 2 * H) {
      r -= 2 * H;
      ++t;
    }
    return v;
  }
};

// One head vector per 8 lanes, each with the 8 values at 8 sub and at 64 + 8 sub (whole sectors per load and
// store), two vectors per turn, read before their slots are known so that the loads overlap.  Bound by HBM
// (256 bytes read, 66 written per vector) and by the loads that an SM has under way: at 48 registers five CTAs fit, of the
// eight per SM that the grid has.  16384 tokens of 8 heads 16.9 us, 5.0 TB/s; an earlier version took 16.5, with five or
// six CTAs per SM in the grid 17.1, with one or three vectors per turn 17.5 and 17.1, with every value
// clamped 17.8, with a division per vector for its token 19.5.  Codes 0 beside a scale of NaN would cost 0.5 us.
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(const __half* __restrict__ K, long long ldk,
                                                               const __half* __restrict__ V, long long ldv, int T,
                                                               const int32_t* __restrict__ slots, float alpha_k,
                                                               float alpha_v, KvView c, KvStep step) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kVecs = 2;
  const int sub = threadIdx.x & 7;
  const int limit = c.num_pages << c.page_shift;
  const long long total = 2ll * T * c.H;
  // every lane of a warp takes the same number of turns (the shuffles below)
  const long long first = static_cast<long long>(blockIdx.x) * (kRowThreads / 8) + (threadIdx.x >> 3);
  KvWalk walk(first, step, c.H);
  for (long long base = first - ((threadIdx.x >> 3) & 3); base < total; base += kVecs * step.vecs) {
    const long long vec0 = base + ((threadIdx.x >> 3) & 3);
    KvVec v[kVecs];
    uint4 raw[kVecs][2];
    int slot[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      raw[u][0] = raw[u][1] = make_uint4(0, 0, 0, 0);
      slot[u] = -1;
      v[u] = walk.next();
      if (vec0 + u * step.vecs < total) {
        const uint4* src =
            reinterpret_cast<const uint4*>((v[u].which ? V + v[u].t * ldv : K + v[u].t * ldk) + v[u].h * kHeadDim) + sub;
        raw[u][0] = src[0];
        raw[u][1] = src[8];
        slot[u] = slots[v[u].t];
      }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      __half2(&h2)[8] = reinterpret_cast<__half2(&)[8]>(raw[u]);
      __half2 m2 = __habs2(h2[0]);
#pragma unroll
      for (int j = 1; j < 8; ++j) m2 = __hmax2_nan(m2, __habs2(h2[j]));
      float m = __half2float(__hmax_nan(__low2half(m2), __high2half(m2)));
#pragma unroll
      for (int o = 4; o; o >>= 1) m = max_nan(m, __shfl_xor_sync(0xffffffffu, m, o));
      if (slot[u] < 0 || slot[u] >= limit) continue;
      m = __fmaf_rn(m, 0.0f, m);  // an infinity becomes NaN
      const float alpha = v[u].which ? alpha_v : alpha_k;
      const __half sh = __float2half_rn(__fdiv_rn(__fmul_rn(m, alpha), 7.0f));  // NaN: 0x7FFF
      const float s = __half2float(sh);
      const float inv = s > 0.f ? __fdividef(1.0f, s) : 0.f;  // s = 0: codes 0
      if (alpha < 1.0f || s < 0x1p-14f) {
        // values may pass the clamp: cut to 7.25 s and -8.25 s, which round to 7 and -8 (otherwise s is the largest
        // magnitude / 7, at most 2^-11 off, and none does)
        const __half2 top = __float2half2_rn(7.25f * s), bottom = __float2half2_rn(-8.25f * s);
#pragma unroll
        for (int j = 0; j < 8; ++j) h2[j] = __hmax2(__hmin2(h2[j], top), bottom);
      }
      const uint32_t w0 = codes8(reinterpret_cast<const __half2(&)[4]>(h2[0]), inv);
      const uint32_t w1 = codes8(reinterpret_cast<const __half2(&)[4]>(h2[4]), inv);
      uint8_t* page = c.block(slot[u] >> c.page_shift, v[u].h);
      const int off = slot[u] & ((1 << c.page_shift) - 1);
      uint32_t* row = reinterpret_cast<uint32_t*>(page + c.codes(v[u].which) + off * kKvRowBytes) + sub;
      row[0] = w0;
      row[8] = w1;
      if (sub == 0) *reinterpret_cast<__half*>(page + c.scales(v[u].which) + 2 * off) = sh;
    }
  }
}

// Codes and scales as fq_quant_kv wrote them: four lanes per head vector.  66 bytes read and written; 16384 tokens of 8
// heads 7.2 us (they stay in L2), 65536 26 us, 2.6 TB/s of reads and as much of writes.
__global__ void __launch_bounds__(kRowThreads) kv_store_kernel(const uint8_t* __restrict__ Kq,
                                                               const __half* __restrict__ Ks,
                                                               const uint8_t* __restrict__ Vq,
                                                               const __half* __restrict__ Vs, int T,
                                                               const int32_t* __restrict__ slots, KvView c,
                                                               KvStep step) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 3;
  const int limit = c.num_pages << c.page_shift;
  const long long total = 2ll * T * c.H;
  const long long first = static_cast<long long>(blockIdx.x) * (kRowThreads / 4) + (threadIdx.x >> 2);
  KvWalk walk(first, step, c.H);
  for (long long vec = first; vec < total; vec += step.vecs) {
    const KvVec v = walk.next();
    const long long t = v.t;
    const int h = v.h, which = v.which;
    const int slot = slots[t];
    if (slot < 0 || slot >= limit) continue;
    const long long row = t * c.H + h;
    uint8_t* base = c.block(slot >> c.page_shift, h);
    const int off = slot & ((1 << c.page_shift) - 1);
    const uint4 q = reinterpret_cast<const uint4*>((which ? Vq : Kq) + row * kKvRowBytes)[sub];
    reinterpret_cast<uint4*>(base + c.codes(which) + off * kKvRowBytes)[sub] = q;
    if (sub == 0) *reinterpret_cast<__half*>(base + c.scales(which) + 2 * off) = (which ? Vs : Ks)[row];
  }
}

// One head vector per 8 lanes, each with the 8 values at 8 sub and at 64 + 8 sub (whole sectors per load and
// store), four vectors per turn so that their slots and codes are loaded together.  One rounding: the fp16 product.  Bound by
// HBM (66 bytes read, 256 written per vector): 16384 tokens of 8 heads 14.1 us, 6.0 TB/s.
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const int32_t* __restrict__ slots, int T,
                                                              __half* __restrict__ K, __half* __restrict__ V,
                                                              KvView c, KvStep step) {
  pdl_launch_dependents();
  pdl_wait();
  constexpr int kVecs = 4;
  const int sub = threadIdx.x & 7;
  const int limit = c.num_pages << c.page_shift;
  const long long total = 2ll * T * c.H;
  const long long first = static_cast<long long>(blockIdx.x) * (kRowThreads / 8) + (threadIdx.x >> 3);
  KvWalk walk(first, step, c.H);
  for (long long vec = first; vec < total; vec += kVecs * step.vecs) {
    KvVec v[kVecs];
    int slot[kVecs];
    uint2 w[kVecs];
    __half s[kVecs];
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      slot[u] = -1;
      v[u] = walk.next();
      if (vec + u * step.vecs < total) slot[u] = slots[v[u].t];
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      w[u] = make_uint2(0, 0);
      s[u] = __ushort_as_half(0);
      if (slot[u] >= 0 && slot[u] < limit) {
        const uint8_t* page = c.block(slot[u] >> c.page_shift, v[u].h);
        const int off = slot[u] & ((1 << c.page_shift) - 1);
        const uint32_t* row = reinterpret_cast<const uint32_t*>(page + c.codes(v[u].which) + off * kKvRowBytes) + sub;
        w[u] = make_uint2(row[0], row[8]);
        s[u] = *reinterpret_cast<const __half*>(page + c.scales(v[u].which) + 2 * off);
      }
    }
#pragma unroll
    for (int u = 0; u < kVecs; ++u) {
      if (vec + u * step.vecs >= total) break;
      uint4 out[2];
      __half2* o2 = reinterpret_cast<__half2*>(out);
      const __half2 s2 = __half2half2(s[u]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // byte j's two nibbles q as the fp16 numbers 1032 + q, less 1032, times the scale
        const uint32_t word = j < 4 ? w[u].x : w[u].y;
        const uint32_t pair = __byte_perm(word, word >> 4, 0x0400u + 0x0101u * (j & 3));
        uint32_t h;
        asm("lop3.b32 %0, %1, %2, %3, 0x6a;" : "=r"(h) : "r"(pair), "r"(0x000F000Fu), "r"(0x64086408u));
        const __half2 q = __hsub2(*reinterpret_cast<const __half2*>(&h), __half2half2(__ushort_as_half(0x6408)));
        o2[j] = __hmul2(q, s2);
      }
      uint4* dst = reinterpret_cast<uint4*>((v[u].which ? V : K) + (v[u].t * c.H + v[u].h) * kHeadDim) + sub;
      dst[0] = out[0];
      dst[8] = out[1];
    }
  }
}

// CTAs for 2 T H head vectors of `lanes` lanes each, and the step that they make.
int row_grid(int T, int H, int lanes, KvStep& step) {
  const long long vectors = 2ll * T * H, want = (vectors * lanes + kRowThreads - 1) / kRowThreads;
  const int grid = int(std::min<long long>(std::max<long long>(want, 1), static_cast<long long>(sm_count()) * 8));
  step.vecs = static_cast<long long>(grid) * (kRowThreads / lanes);
  step.tokens = step.vecs / (2 * H);
  step.rest = int(step.vecs % (2 * H));
  return grid;
}

}  // namespace
}  // namespace fq

extern "C" {

fq_status fq_kv_plan(const int32_t* len, const int32_t* new_tokens, int R, int page_size, int32_t* block_table,
                     int max_pages, const int32_t* free_pages, int num_free, const int32_t* pages_used,
                     int32_t* len_out, int32_t* token_start, int32_t* slots, int max_tokens,
                     int32_t* pages_used_out, void* stream) {
  fq::clear_error();
  FQ_CHECK_ARG(R >= 1 && R <= fq::kPlanMaxR, "R = %d must lie in [1, %d]", R, fq::kPlanMaxR);
  FQ_CHECK_ARG(page_size == 16 || page_size == 32 || page_size == 64 || page_size == 128,
               "page_size = %d must be 16, 32, 64 or 128", page_size);
  FQ_CHECK_ARG(max_pages >= 1 && static_cast<long long>(max_pages) * page_size < (1ll << 31),
               "max_pages = %d: at least 1, and fewer than 2^31 tokens", max_pages);
  FQ_CHECK_ARG(num_free >= 0 && max_tokens >= 0 && max_tokens <= (1 << 30),
               "num_free = %d must not be negative, max_tokens = %d lie in [0, 2^30]", num_free, max_tokens);
  FQ_CHECK_ARG(len && new_tokens && block_table && pages_used && len_out && token_start && pages_used_out &&
                   (free_pages || num_free == 0) && (slots || max_tokens == 0),
               "a pointer is NULL");
  for (const void* q : {static_cast<const void*>(len), static_cast<const void*>(new_tokens),
                        static_cast<const void*>(block_table), static_cast<const void*>(free_pages),
                        static_cast<const void*>(pages_used), static_cast<const void*>(len_out),
                        static_cast<const void*>(token_start), static_cast<const void*>(slots),
                        static_cast<const void*>(pages_used_out)})
    FQ_CHECK_ARG(fq::aligned(q, 4), "pointers must be 4-byte aligned");
  fq::PlanParams p{};
  p.len = len;
  p.fresh = new_tokens;
  p.free_pages = free_pages;
  p.used = pages_used;
  p.table = block_table;
  p.len_out = len_out;
  p.start = token_start;
  p.slots = slots;
  p.used_out = pages_used_out;
  p.R = R;
  p.page_shift = page_size == 16 ? 4 : page_size == 32 ? 5 : page_size == 64 ? 6 : 7;
  p.max_pages = max_pages;
  p.num_free = num_free;
  p.max_tokens = max_tokens;
  const size_t smem = size_t(R) * 3 * sizeof(int);
  if (smem > 47 * 1024 &&
      cudaFuncSetAttribute(fq::kv_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, int(smem)) != cudaSuccess)
    return fq::fail(FQ_ERR_CUDA, "cannot reserve %zu bytes of shared memory", smem);
  // more CTAs only where there are rows for them: the cluster barrier costs more than it saves below
  const unsigned ncta = max_tokens > 4 * fq::kPlanThreads ? 8 : 1;
  if (ncta == 1)
    fq::launch_pdl(fq::kv_plan_kernel, dim3(1), dim3(fq::kPlanThreads), smem, static_cast<cudaStream_t>(stream), p);
  else
    fq::launch_pdl_cluster(fq::kv_plan_kernel, dim3(ncta), dim3(fq::kPlanThreads), smem,
                           static_cast<cudaStream_t>(stream), ncta, p);
  return fq::check_launch("kv_plan_kernel");
}

fq_status fq_kv_write(const uint16_t* K, long long ldk, const uint16_t* V, long long ldv, int T,
                      const int32_t* slots, float alpha_k, float alpha_v, const fq_kv_cache* cache, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_kv_cache(cache);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(T >= 1, "T = %d must be >= 1", T);
  FQ_CHECK_ARG(K && V && fq::aligned(K, 16) && fq::aligned(V, 16), "K and V must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(slots && fq::aligned(slots, 4), "slots must be non-NULL and 4-byte aligned");
  const long long row = static_cast<long long>(cache->H) * fq::kHeadDim;
  FQ_CHECK_ARG(ldk >= row && ldv >= row && ldk % 8 == 0 && ldv % 8 == 0,
               "row strides %lld and %lld must be multiples of 8 and at least H * 128 = %lld", ldk, ldv, row);
  FQ_CHECK_ARG(alpha_k > 0.f && alpha_k <= 1.f && alpha_v > 0.f && alpha_v <= 1.f, "alpha must lie in (0, 1]");
  fq::KvStep step;
  const int grid = fq::row_grid(T, cache->H, 8, step);
  fq::launch_pdl(fq::kv_write_kernel, dim3(grid), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), reinterpret_cast<const __half*>(K), ldk,
                 reinterpret_cast<const __half*>(V), ldv, T, slots, alpha_k, alpha_v, fq::kv_view(cache), step);
  return fq::check_launch("kv_write_kernel");
}

fq_status fq_kv_store(const uint8_t* Kq, const uint16_t* Ks, const uint8_t* Vq, const uint16_t* Vs, int T,
                      const int32_t* slots, const fq_kv_cache* cache, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_kv_cache(cache);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(T >= 1, "T = %d must be >= 1", T);
  FQ_CHECK_ARG(Kq && Vq && fq::aligned(Kq, 16) && fq::aligned(Vq, 16),
               "Kq and Vq must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(Ks && Vs && fq::aligned(Ks, 2) && fq::aligned(Vs, 2), "Ks and Vs must be non-NULL and aligned");
  FQ_CHECK_ARG(slots && fq::aligned(slots, 4), "slots must be non-NULL and 4-byte aligned");
  fq::KvStep step;
  const int grid = fq::row_grid(T, cache->H, 4, step);
  fq::launch_pdl(fq::kv_store_kernel, dim3(grid), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), Kq, reinterpret_cast<const __half*>(Ks), Vq,
                 reinterpret_cast<const __half*>(Vs), T, slots, fq::kv_view(cache), step);
  return fq::check_launch("kv_store_kernel");
}

fq_status fq_kv_read(const fq_kv_cache* cache, const int32_t* slots, int T, uint16_t* K, uint16_t* V, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_kv_cache(cache);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(T >= 1, "T = %d must be >= 1", T);
  FQ_CHECK_ARG(K && V && fq::aligned(K, 16) && fq::aligned(V, 16), "K and V must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(slots && fq::aligned(slots, 4), "slots must be non-NULL and 4-byte aligned");
  fq::KvStep step;
  const int grid = fq::row_grid(T, cache->H, 8, step);
  fq::launch_pdl(fq::kv_read_kernel, dim3(grid), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), slots, T, reinterpret_cast<__half*>(K),
                 reinterpret_cast<__half*>(V), fq::kv_view(cache), step);
  return fq::check_launch("kv_read_kernel");
}

}  // extern "C"
