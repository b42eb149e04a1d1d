// The 4-bit key/value cache's format (spec_verify.h describes it) as the
// kernels address it, and the argument checks its entry points share.
#pragma once

#include "spec_verify.h"

#include "common.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace sv {

constexpr int kNaNScale = 255;   // the scale byte of a block that reads back as NaN

// Offsets inside the record of one page and head.  D numbers per vector, P
// tokens per page.
template <int D>
struct Format {
  static constexpr int kBlocks = D / 32;    // scales per vector
  static constexpr int kRow = D / 2;        // bytes of a key's codes
  static constexpr int kPiece = D / 32;     // bytes of one token's codes in a value piece (D / 16 codes)
  static constexpr int kTileV = 8 * D;      // bytes of 16 tokens' value codes
  __device__ static int record(int P) { return P * (D + D / 16); }
  __device__ static int keys(int r) { return r * kRow; }
  __device__ static int key_scales(int P, int r) { return P * D + r * kBlocks; }
  // Token r's first number of lane share i (numbers i * D/16 on).
  __device__ static int values(int P, int r, int i) {
    return P * kRow + (r >> 4) * kTileV + ((r >> 2) & 3) * (2 * D) + i * (4 * kPiece) + (r & 3) * kPiece;
  }
  __device__ static int value_scale(int P, int r, int blk) {
    return P * D + P * kBlocks + (r >> 4) * (D / 2) + blk * 16 + (r & 15);
  }
};

// A cache and its call's positions, as the kernels take them.
struct CacheView {
  uint8_t* data;
  const int32_t* table;
  const int32_t* len;
  const int32_t* count;
  int pages, heads, page_log2, table_len;
  int B, n, lag;
};

struct Span {   // one sequence's tokens in a call
  int pos;      // position of token 0
  int count;    // tokens, or -1 after a range error
};

__device__ __forceinline__ Span span_from(const CacheView& c, int64_t pos, int count) {
  const int64_t room = (int64_t)c.table_len << c.page_log2;
  if (count < 0 || count > c.n || (count > 0 && (pos < 0 || pos + count > room))) return {0, -1};
  return {count > 0 ? (int)pos : 0, count};
}
__device__ __forceinline__ Span span_of(const CacheView& c, int b) {
  return span_from(c, (int64_t)(c.len ? c.len[b] : 0) - c.lag, c.count ? c.count[b] : c.n);
}

// An entry of an array that the kernel does not write, through the scalar cache: the address is the wave's.
__device__ __forceinline__ int scalar_at(const int32_t* p, int at) {
  return ((const __attribute__((address_space(4))) int32_t*)(uintptr_t)p)[at];
}

// Eight numbers of a row whose first lies anywhere its type's alignment allows.
struct __attribute__((packed, aligned(2))) Bf16x8 { uint32_t w[4]; };
struct __attribute__((packed, aligned(4))) F32x8 { float v[8]; };

template <int DT>
__device__ __forceinline__ void load_row8(const void* row, int64_t j, float (&x)[8]) {
  if constexpr (DT == kBF16) {
    const Bf16x8 t = *reinterpret_cast<const Bf16x8*>(static_cast<const uint16_t*>(row) + j);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = bf16_lo(t.w[e]);
      x[2 * e + 1] = bf16_hi(t.w[e]);
    }
  } else {
    const F32x8 t = *reinterpret_cast<const F32x8*>(static_cast<const float*>(row) + j);
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = t.v[e];
  }
}

// 2^(e - 127).  Codes of a block with e = 255 are not used.
__device__ __forceinline__ float scale_of(unsigned e) { return __uint_as_float(e << 23); }

inline int page_log2_of(int page) {
  return page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : page == 256 ? 8 : -1;
}
inline bool dim_ok(int dim) { return dim == 64 || dim == 128 || dim == 256; }
inline bool off16(const void* p) { return ((uintptr_t)p & 15) != 0; }

// What every entry point checks of its cache and sizes.
inline int check_cache(const spec_cache* c, int lag, int B, int n, int dtype) {
  if (!c || page_log2_of(c->page) < 0 || !dim_ok(c->dim) || c->heads < 1 || c->pages < 0 || c->table_len < 0 ||
      lag < 0 || lag > 1 || B < 0 || n < 1)
    return SPEC_EINVAL;
  if ((int64_t)c->table_len * c->page > ((int64_t)1 << 30) || (int64_t)B * n > ((int64_t)1 << 24)) return SPEC_EINVAL;
  const int64_t most = ((int64_t)1 << 34) / c->dim;   // B * n * heads * dim <= 2^34, without overflow
  if (B > 0 && c->heads > most / ((int64_t)B * n)) return SPEC_EINVAL;
  if (dtype != SPEC_F32 && dtype != SPEC_BF16) return SPEC_EDTYPE;
  return SPEC_OK;
}
inline int check_buffers(const spec_cache* c) {
  // An empty pool or table needs no storage: every token is then an error found on the device.
  if ((c->pages > 0 && !c->data) || (c->table_len > 0 && !c->table) || off16(c->data)) return SPEC_EINVAL;
  return SPEC_OK;
}
inline CacheView view_of(const spec_cache* c, const int32_t* len, int lag, const int32_t* count, int B, int n) {
  return {static_cast<uint8_t*>(c->data), c->table, len, count, c->pages, c->heads, page_log2_of(c->page), c->table_len, B, n, lag};
}

}  // namespace sv
