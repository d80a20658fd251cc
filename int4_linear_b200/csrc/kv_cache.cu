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
// write lets len_out be len and pages_used_out be pages_used.
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
  const int used = *p.used;
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
#pragma unroll 1
    for (int w = 0; w < kPlanThreads / 32; ++w) taken = max(taken, part[w]);
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
  // per row of the batch; a page that this step takes is read from the free
  // list, so that no CTA waits for another's table entries
  for (int i = rank * kPlanThreads + tid; i < p.max_tokens; i += ncta * kPlanThreads) {
    int slot = -1;
    if (i < tokens) {
      const int r = last_not_above(s_start, p.R, i);
      const int l = s_len[r];
      if (l >= 0) {
        const int pos = l + (i - s_start[r]);
        const int pi = pos >> p.page_shift, held = (l + page - 1) >> p.page_shift;
        const int id = pi < held ? p.table[size_t(r) * p.max_pages + pi] : p.free_pages[used + s_first[r] + pi - held];
        slot = id * page + (pos & (page - 1));
      }
    }
    p.slots[i] = slot;
  }
}

// ------------------------------------------------------------------ into and out of the pages

constexpr int kRowThreads = 256;

// clamp(round-half-even(v / s), -8, 7) for fp16 values v and an fp16 scale s > 0
// (both widened), inv ~ 1 / s.  v / s differs from a tie (k + 1/2) by at least
// 2^-12 unless it is one, since v and s have 11 bits each, so the nearest integer of
// v * inv is right except on a tie; there |v - q s| = s / 2 exactly, and q moves to
// the even neighbour.
__device__ __forceinline__ int code_f16(float v, float s, float inv) {
  float q = rintf(__fmul_rn(v, inv));
  const float e = __fmaf_rn(-q, s, v);
  int c = int(q);
  if (fabsf(e) + fabsf(e) == s && (c & 1)) c += e > 0.f ? 1 : -1;
  return min(max(c, -8), 7);
}

// One head vector per 8 lanes: 32 bytes in, 8 bytes of codes out per lane.
// Bound by HBM (256 bytes read, 66 written per vector).
__global__ void __launch_bounds__(kRowThreads) kv_write_kernel(const __half* __restrict__ K, long long ldk,
                                                               const __half* __restrict__ V, long long ldv, int T,
                                                               const int32_t* __restrict__ slots, float alpha_k,
                                                               float alpha_v, KvView c) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 7;
  const long long nvec = 2ll * T * c.H;
  const int limit = c.num_pages << c.page_shift;
  const long long step = static_cast<long long>(gridDim.x) * (kRowThreads / 8);
  // every lane of a warp takes the same number of turns (the shuffles below)
  const long long first = static_cast<long long>(blockIdx.x) * (kRowThreads / 8) + (threadIdx.x >> 3);
  const long long turns = (nvec - (first - ((threadIdx.x >> 3) & 3)) + step - 1) / step;
  for (long long it = 0; it < turns; ++it) {
    const long long vec = first + it * step;
    int slot = -1, h = 0, which = 0;
    long long t = 0;
    if (vec < nvec) {
      h = int(vec % c.H);
      const long long tw = vec / c.H;
      which = int(tw & 1);
      t = tw >> 1;
      slot = slots[t];
    }
    const bool ok = slot >= 0 && slot < limit;
    uint4 raw[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (ok) {
      const uint4* src = reinterpret_cast<const uint4*>((which ? V + t * ldv : K + t * ldk) + h * kHeadDim) + 2 * sub;
      raw[0] = src[0];
      raw[1] = src[1];
    }
    const __half2* h2 = reinterpret_cast<const __half2*>(raw);
    __half2 m2 = __habs2(h2[0]);
#pragma unroll
    for (int j = 1; j < 8; ++j) m2 = __hmax2(m2, __habs2(h2[j]));
    float m = __half2float(__hmax(__low2half(m2), __high2half(m2)));
#pragma unroll
    for (int o = 4; o; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    const __half sh = __float2half_rn(__fdiv_rn(__fmul_rn(m, which ? alpha_v : alpha_k), 7.0f));
    const float s = __half2float(sh);
    const float inv = s > 0.f ? __fdividef(1.0f, s) : 0.f;
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float2 f = __half22float2(h2[j]);
      w[j >> 2] |= (uint32_t(code_f16(f.x, s, inv)) & 15u) << (8 * (j & 3));
      w[j >> 2] |= (uint32_t(code_f16(f.y, s, inv)) & 15u) << (8 * (j & 3) + 4);
    }
    if (ok) {
      uint8_t* base = c.block(slot >> c.page_shift, h);
      const int off = slot & ((1 << c.page_shift) - 1);
      *reinterpret_cast<uint2*>(base + c.codes(which) + off * kKvRowBytes + 8 * sub) = make_uint2(w[0], w[1]);
      if (sub == 0) *reinterpret_cast<__half*>(base + c.scales(which) + 2 * off) = sh;
    }
  }
}

// Codes and scales as fq_quant_kv wrote them: four lanes per head vector.
__global__ void __launch_bounds__(kRowThreads) kv_store_kernel(const uint8_t* __restrict__ Kq,
                                                               const __half* __restrict__ Ks,
                                                               const uint8_t* __restrict__ Vq,
                                                               const __half* __restrict__ Vs, int T,
                                                               const int32_t* __restrict__ slots, KvView c) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 3;
  const long long nvec = 2ll * T * c.H;
  const int limit = c.num_pages << c.page_shift;
  for (long long vec = static_cast<long long>(blockIdx.x) * (kRowThreads / 4) + (threadIdx.x >> 2); vec < nvec;
       vec += static_cast<long long>(gridDim.x) * (kRowThreads / 4)) {
    const int h = int(vec % c.H);
    const long long tw = vec / c.H;
    const int which = int(tw & 1);
    const long long t = tw >> 1;
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

// One head vector per 8 lanes: 8 bytes of codes in, 32 bytes out per lane.
// The product of a 4-bit code and an 11-bit scale is exact in float32, so
// there is one rounding, to fp16.
__global__ void __launch_bounds__(kRowThreads) kv_read_kernel(const int32_t* __restrict__ slots, int T,
                                                              __half* __restrict__ K, __half* __restrict__ V,
                                                              KvView c) {
  pdl_launch_dependents();
  pdl_wait();
  const int sub = threadIdx.x & 7;
  const long long nvec = 2ll * T * c.H;
  const int limit = c.num_pages << c.page_shift;
  for (long long vec = static_cast<long long>(blockIdx.x) * (kRowThreads / 8) + (threadIdx.x >> 3); vec < nvec;
       vec += static_cast<long long>(gridDim.x) * (kRowThreads / 8)) {
    const int h = int(vec % c.H);
    const long long tw = vec / c.H;
    const int which = int(tw & 1);
    const long long t = tw >> 1;
    const int slot = slots[t];
    uint4 out[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (slot >= 0 && slot < limit) {
      const uint8_t* base = c.block(slot >> c.page_shift, h);
      const int off = slot & ((1 << c.page_shift) - 1);
      const uint2 w = *reinterpret_cast<const uint2*>(base + c.codes(which) + off * kKvRowBytes + 8 * sub);
      const float s = __half2float(*reinterpret_cast<const __half*>(base + c.scales(which) + 2 * off));
      __half2* o2 = reinterpret_cast<__half2*>(out);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int b = int(((j < 4 ? w.x : w.y) >> (8 * (j & 3))) & 255u);
        const int lo = (b << 28) >> 28, hi = (b << 24) >> 28;
        o2[j] = __floats2half2_rn(float(lo) * s, float(hi) * s);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>((which ? V : K) + (t * c.H + h) * kHeadDim) + 2 * sub;
    dst[0] = out[0];
    dst[1] = out[1];
  }
}

int row_grid(long long vectors, int lanes) {
  const long long want = (vectors * lanes + kRowThreads - 1) / kRowThreads;
  return int(std::min<long long>(std::max<long long>(want, 1), static_cast<long long>(sm_count()) * 8));
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
  FQ_CHECK_ARG(num_free >= 0 && max_tokens >= 0, "num_free = %d and max_tokens = %d must not be negative", num_free,
               max_tokens);
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
  if (fq::launch_pdl_cluster(fq::kv_plan_kernel, dim3(ncta), dim3(fq::kPlanThreads), smem,
                             static_cast<cudaStream_t>(stream), ncta, p) != cudaSuccess)
    return fq::check_launch("kv_plan_kernel");
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
  fq::launch_pdl(fq::kv_write_kernel, dim3(fq::row_grid(2ll * T * cache->H, 8)), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), reinterpret_cast<const __half*>(K), ldk,
                 reinterpret_cast<const __half*>(V), ldv, T, slots, alpha_k, alpha_v, fq::kv_view(cache));
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
  fq::launch_pdl(fq::kv_store_kernel, dim3(fq::row_grid(2ll * T * cache->H, 4)), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), Kq, reinterpret_cast<const __half*>(Ks), Vq,
                 reinterpret_cast<const __half*>(Vs), T, slots, fq::kv_view(cache));
  return fq::check_launch("kv_store_kernel");
}

fq_status fq_kv_read(const fq_kv_cache* cache, const int32_t* slots, int T, uint16_t* K, uint16_t* V, void* stream) {
  fq::clear_error();
  const fq_status st = fq::check_kv_cache(cache);
  if (st != FQ_OK) return st;
  FQ_CHECK_ARG(T >= 1, "T = %d must be >= 1", T);
  FQ_CHECK_ARG(K && V && fq::aligned(K, 16) && fq::aligned(V, 16), "K and V must be non-NULL and 16-byte aligned");
  FQ_CHECK_ARG(slots && fq::aligned(slots, 4), "slots must be non-NULL and 4-byte aligned");
  fq::launch_pdl(fq::kv_read_kernel, dim3(fq::row_grid(2ll * T * cache->H, 8)), dim3(fq::kRowThreads), 0,
                 static_cast<cudaStream_t>(stream), slots, T, reinterpret_cast<__half*>(K),
                 reinterpret_cast<__half*>(V), fq::kv_view(cache));
  return fq::check_launch("kv_read_kernel");
}

}  // extern "C"
