// The paged key-value cache (bfly_cache.hip, bfly_attend.hip): its layout and
// the launch parameters shared by the C-ABI layer and the kernels.
#pragma once

#include "bfly_internal.h"

namespace bfly {

// Formats of a cache's rows, as bfly_kv.
enum CacheFormat : int { kCacheBF16 = 0, kCacheInt8 = 1, kCacheE4M3 = 2, kCacheInt4 = 3 };

// Bytes that n elements of a row take.
__host__ __device__ constexpr int cache_bytes(int format, int n) {
  return format == kCacheBF16 ? 2 * n : format == kCacheInt4 ? n / 2 : n;
}

// Keys and values: pages [pages][kv_heads][page_size][head_dim], scales
// [pages][kv_heads][page_size] (not for bf16).  A head's part of a page is one
// contiguous run, so that whatever reads a sequence's tokens of one head reads
// page_size rows at a time.
struct CacheParams {
  const void* k;             // [tokens] rows of kv_heads * head_dim elements, k_stride apart
  const void* v;
  int64_t k_stride, v_stride;
  void* k_cache;
  void* v_cache;
  uint16_t* k_scales;
  uint16_t* v_scales;
  const int32_t* slots;      // [tokens]: page * page_size + place; outside the cache: none
  int64_t tokens;
  int32_t pages, kv_heads, page_shift, head_dim, format;
  int32_t x_bf16;            // type of k and v
};
hipError_t launch_cache_write(const CacheParams& p, hipStream_t s);
hipError_t launch_cache_read(const CacheParams& p, hipStream_t s);  // k, v are written

constexpr int kCacheMaxPage = 65536;

struct AttendParams {
  const void* q;             // [rows] rows of heads * head_dim elements, q_stride apart
  int64_t q_stride;
  const void* k_cache;
  const void* v_cache;
  const uint16_t* k_scales;
  const uint16_t* v_scales;
  const int32_t* tables;     // [rows][table_width] pages; one outside [0, pages): none
  const int32_t* lens;       // [rows]
  void* y;                   // [rows][heads][head_dim]
  float* lse;                // [rows][heads] or nullptr
  float* partials;           // attend_workspace_bytes
  int64_t rows;
  int32_t heads, kv_heads, head_dim, pages, page_shift, table_width, max_len, window, format;
  int32_t q_bf16, y_bf16;
  float scale;
};
hipError_t launch_attend(const AttendParams& p, hipStream_t s);

}  // namespace bfly
