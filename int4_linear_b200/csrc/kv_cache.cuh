// Where a page of the INT4 key/value cache keeps what (see fq_kv_cache in fq.h).
#pragma once

#include <cstddef>
#include <cstdint>

#include "../../include/fq.h"

namespace fq {

constexpr int kHeadDim = 128;
constexpr int kKvRowBytes = kHeadDim / 2;                 // packed codes of one head vector
constexpr int kKvTokenBytes = 2 * kKvRowBytes + 2 * 2;    // K and V codes, two fp16 scales

struct KvView {
  uint8_t* pool;
  int num_pages;
  int page_shift;  // log2 of the page size
  int H;
  __host__ __device__ int block_bytes() const { return kKvTokenBytes << page_shift; }
  // the bytes of one page and head (the pool may pass 2^32 bytes)
  __host__ __device__ uint8_t* block(int page, int head) const {
    return pool + (static_cast<size_t>(page) * H + head) * static_cast<size_t>(block_bytes());
  }
  __host__ __device__ int codes(int which) const { return (kKvRowBytes * which) << page_shift; }
  __host__ __device__ int scales(int which) const { return (2 * kKvRowBytes + 2 * which) << page_shift; }
};

// FQ_OK, or the error of a cache description outside fq.h's ranges.
fq_status check_kv_cache(const fq_kv_cache* c);
KvView kv_view(const fq_kv_cache* c);

}  // namespace fq
