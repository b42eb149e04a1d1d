// Writing keys and values into the 4-bit cache, and reading them back
// (spec_verify.h describes the format and the entry points).
#include "format.h"

#include <float.h>

namespace sv {
namespace {

// The page of position t, or -1.
__device__ __forceinline__ int page_of(const CacheView& c, int b, int t) {
  const int p = c.table[(int64_t)b * c.table_len + (t >> c.page_log2)];
  return (p >= 0 && p < c.pages) ? p : -1;
}

// status[b]: 0, 1 after a range error, 2 if some token's page is bad.
__device__ void report(const CacheView& c, int b, int32_t* status) {
  const Span s = span_of(c, b);
  int bad = 0;
  if (s.count > 0) {
    const int p0 = s.pos >> c.page_log2, p1 = (s.pos + s.count - 1) >> c.page_log2;
    for (int p = p0 + (int)threadIdx.x; p <= p1; p += kThreads) bad |= page_of(c, b, p << c.page_log2) < 0;
  }
  bad = __syncthreads_or(bad);
  if (threadIdx.x == 0) status[b] = s.count < 0 ? 1 : bad ? 2 : 0;
}

// A wave takes a tile of 16 positions of one sequence and head, its keys and
// its values, as the attention's waves read them: lane (g, i) holds 4 tokens,
// 4 g to 4 g + 3, of D / 16 numbers from i * D / 16 on.  The values' codes of
// a lane then lie side by side in the record, every access of a row is
// contiguous over 16 lanes, and what depends on the sequence is scalar.
struct TileArgs {
  CacheView c;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  void* out_k;
  void* out_v;
  int32_t* status;
  int tiles;    // that n tokens of a sequence can touch
  int blocks;   // work-groups; those behind write the status
};

struct Tile {
  int b, h, token0, r0, page;   // token0: the call's token at the tile's first position (may be negative)
  int count;                    // tokens of the sequence, -1 after a range error
};

// Tile number `wave`; false if there is none.
__device__ __forceinline__ bool tile_of(const TileArgs& a, unsigned wave, Tile& t) {
  const CacheView& c = a.c;
  const unsigned row = wave / (unsigned)c.heads, seq = row / (unsigned)a.tiles;
  if (seq >= (unsigned)c.B) return false;
  t.b = (int)seq;
  t.h = (int)(wave - row * (unsigned)c.heads);
  const int tile = (int)(row - seq * (unsigned)a.tiles);
  const int64_t pos = (int64_t)(c.len ? scalar_at(c.len, t.b) : 0) - c.lag;
  const Span s = span_from(c, pos, c.count ? scalar_at(c.count, t.b) : c.n);
  t.count = s.count;
  const int start = (s.pos & ~15) + 16 * tile;
  t.token0 = start - s.pos;
  if (t.token0 >= (s.count < 0 ? c.n : s.count)) return false;
  t.r0 = start & ((1 << c.page_log2) - 1);
  t.page = -1;
  if (s.count >= 0) {
    const int page = scalar_at(c.table + (int64_t)t.b * c.table_len, start >> c.page_log2);
    if (page >= 0 && page < c.pages) t.page = page;
  }
  return true;
}

// op over the lanes that hold a block of 32 numbers.
template <int D, class V, class Op>
__device__ __forceinline__ V over_block(V x, Op op) {
  x = op(x, dpp<kDppQuad1032>(x, x));
  if constexpr (D <= 128) x = op(x, dpp<kDppQuad2301>(x, x));
  if constexpr (D == 64) x = op(x, dpp<kDppRowHalfMirror>(x, x));
  return x;
}

// D / 16 numbers of a row whose first lies anywhere its type's alignment allows.
template <int N>
struct __attribute__((packed, aligned(2))) Bf16xN { uint16_t w[N]; };
template <int N>
struct __attribute__((packed, aligned(4))) F32xN { float v[N]; };
template <int DT, int N>
__device__ __forceinline__ void load_row(const void* row, int64_t j, float (&x)[N]) {
  if constexpr (DT == kBF16) {
    const Bf16xN<N> t = *reinterpret_cast<const Bf16xN<N>*>(static_cast<const uint16_t*>(row) + j);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = __uint_as_float((uint32_t)t.w[e] << 16);
  } else {
    const F32xN<N> t = *reinterpret_cast<const F32xN<N>*>(static_cast<const float*>(row) + j);
#pragma unroll
    for (int e = 0; e < N; ++e) x[e] = t.v[e];
  }
}

// The codes of a lane's N numbers of one token, and the scale byte of their block.
template <int D, int N>
__device__ __forceinline__ unsigned quantise(const float (&x)[N], uint32_t (&w)[(N + 7) / 8]) {
  float m = 0.0f;
  int odd = 0;   // a NaN or an infinity
#pragma unroll
  for (int e = 0; e < N; ++e) {
    m = fmaxf(m, fabsf(x[e]));
    odd |= !(fabsf(x[e]) <= FLT_MAX);
  }
  m = over_block<D>(m, [](float u, float v) { return fmaxf(u, v); });
  odd = over_block<D>(odd, [](int u, int v) { return u | v; });
  // a = f 2^(E - 127), 1 <= f < 2: the smallest power of two s with a <= 7 s
  // is 2^(E - 129) up to f = 1.75 and 2^(E - 128) above.  Below the normal
  // range E = 0 and the clamp decides.
  const unsigned bits = __float_as_uint(m);
  int e = (int)(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 3 ? 3 : e > 252 ? 252 : e;
  const float scale = scale_of((unsigned)e);
#pragma unroll
  for (int q = 0; q < (N + 7) / 8; ++q) {
    uint32_t y = 0;
    y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[8 * q], x[8 * q + 1], scale, 0);
    y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[8 * q + 2], x[8 * q + 3], scale, 1);
    if constexpr (N > 4) {
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[8 * q + 4], x[8 * q + 5], scale, 2);
      y = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(y, x[8 * q + 6], x[8 * q + 7], scale, 3);
    }
    w[q] = odd ? 0 : y;
  }
  return odd ? (unsigned)kNaNScale : (unsigned)e;
}

// Codes of N numbers at p: N / 2 bytes.
template <int N>
__device__ __forceinline__ void store_codes(uint8_t* p, const uint32_t (&w)[(N + 7) / 8]) {
  if constexpr (N == 4) {
    *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  } else if constexpr (N == 8) {
    *reinterpret_cast<uint32_t*>(p) = w[0];
  } else {
    *reinterpret_cast<uint64_t*>(p) = (uint64_t)w[1] << 32 | w[0];
  }
}
template <int N>
__device__ __forceinline__ void load_codes(const uint8_t* p, uint32_t (&w)[(N + 7) / 8]) {
  if constexpr (N == 4) {
    w[0] = *reinterpret_cast<const uint16_t*>(p);
  } else if constexpr (N == 8) {
    w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else {
    const uint64_t t = *reinterpret_cast<const uint64_t*>(p);
    w[0] = (uint32_t)t;
    w[1] = (uint32_t)(t >> 32);
  }
}

// Bound by memory where there is much: a number in, 4 bits and a 32nd of a
// byte out; else by the chain of loads (length, page, numbers), so a wave
// takes the keys or the values of its tile, and asks for them before it looks
// at the page.  Three prompts of 8191 tokens at most, float32, written and read
// back: 196 MB in 28 + 21 us.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void append_kernel(TileArgs a) {
  using F = Format<D>;
  constexpr int N = D / 16;
  const CacheView& c = a.c;
  if ((int)blockIdx.x >= a.blocks) return report(c, (int)blockIdx.x - a.blocks, a.status);
  const unsigned wave = blockIdx.x * kWaves + (unsigned)uni((int)(threadIdx.x >> 6));
  const bool values = wave & 1;
  Tile t;
  if (!tile_of(a, wave >> 1, t)) return;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, P = 1 << c.page_log2;
  const void* src = values ? a.v : a.k;
  const int64_t stride = values ? a.v_stride : a.k_stride;
  const int64_t first = (int64_t)t.b * c.n + t.token0 + 4 * g, in = (int64_t)t.h * D + i * N;
  float x[4][N];
  bool live[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {   // lanes of one token leave or stay together
    const int token = t.token0 + 4 * g + j;
    live[j] = token >= 0 && token < t.count;
#pragma unroll
    for (int e = 0; e < N; ++e) x[j][e] = 0.0f;
    if (live[j]) load_row<DT, N>(src, (first + j) * stride + in, x[j]);
  }
  if (t.page < 0) return;
  uint8_t* rec = c.data + ((int64_t)t.page * c.heads + t.h) * F::record(P);
  const bool scales = i % (32 / N) == 0;   // the block's first lane writes its scale
  uint32_t w[4][(N + 7) / 8];
  unsigned sc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) sc[j] = quantise<D, N>(x[j], w[j]);
  const int r = t.r0 + 4 * g;
  if (!values) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!live[j]) continue;
      store_codes<N>(rec + F::keys(r + j) + i * (N / 2), w[j]);
      if (scales) rec[F::key_scales(P, r + j) + i / (32 / N)] = (uint8_t)sc[j];
    }
  } else if (live[0] && live[1] && live[2] && live[3]) {
    uint32_t* at = reinterpret_cast<uint32_t*>(rec + F::values(P, r, i));
    if constexpr (N == 4) {
      at[0] = w[0][0] | w[1][0] << 16;
      at[1] = w[2][0] | w[3][0] << 16;
    } else {
#pragma unroll
      for (int q = 0; q < N / 8; ++q)
        reinterpret_cast<u32x4*>(at)[q] = N == 8 ? u32x4{w[0][0], w[1][0], w[2][0], w[3][0]}
                                                 : u32x4{w[2 * q][0], w[2 * q][N / 8 - 1], w[2 * q + 1][0], w[2 * q + 1][N / 8 - 1]};
    }
    if (scales)
      *reinterpret_cast<uint32_t*>(rec + F::value_scale(P, r, i / (32 / N))) = sc[0] | sc[1] << 8 | sc[2] << 16 | sc[3] << 24;
  } else {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      if (!live[j]) continue;
      store_codes<N>(rec + F::values(P, r + j, i), w[j]);
      if (scales) rec[F::value_scale(P, r + j, i / (32 / N))] = (uint8_t)sc[j];
    }
  }
}

typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));

// A token's N numbers to its row.  In bfloat16 they are exact: 2 significant
// bits, and the scale keeps them in the normal range.
template <int DT, int N>
__device__ __forceinline__ void store_row(void* out, int64_t at, const uint32_t (&w)[(N + 7) / 8], unsigned e) {
  const float scale = scale_of(e);
  if constexpr (DT == kBF16) {
    uint32_t y[N / 2];
#pragma unroll
    for (int q = 0; q < (N + 7) / 8; ++q) {
      y[4 * q] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], scale, 0));
      y[4 * q + 1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], scale, 1));
      if constexpr (N > 4) {
        y[4 * q + 2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], scale, 2));
        y[4 * q + 3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w[q], scale, 3));
      }
    }
    if (e == kNaNScale) {
#pragma unroll
      for (int q = 0; q < N / 2; ++q) y[q] = 0x7FC07FC0u;
    }
    uint16_t* p = static_cast<uint16_t*>(out) + at;
    if constexpr (N == 4) {
      *reinterpret_cast<uint64_t*>(p) = (uint64_t)y[1] << 32 | y[0];
    } else {
#pragma unroll
      for (int q = 0; q < N / 8; ++q) {
        const u32x4 o = {y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
        if constexpr (N == 8) {   // neighbouring lanes fill whole lines: nothing to keep in the cache
          __builtin_nontemporal_store(o, reinterpret_cast<u32x4*>(p) + q);
        } else {
          reinterpret_cast<u32x4*>(p)[q] = o;
        }
      }
    }
  } else {
    float y[N];
#pragma unroll
    for (int q = 0; q < (N + 7) / 8; ++q) {
      const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], scale, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], scale, 1);
      y[8 * q] = a.x; y[8 * q + 1] = a.y; y[8 * q + 2] = b.x; y[8 * q + 3] = b.y;
      if constexpr (N > 4) {
        const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], scale, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w[q], scale, 3);
        y[8 * q + 4] = c.x; y[8 * q + 5] = c.y; y[8 * q + 6] = d.x; y[8 * q + 7] = d.y;
      }
    }
    if (e == kNaNScale) {
#pragma unroll
      for (int q = 0; q < N; ++q) y[q] = __uint_as_float(0x7FC00000u);
    }
#pragma unroll
    for (int q = 0; q < N / 4; ++q)
      reinterpret_cast<f32x4*>(static_cast<float*>(out) + at)[q] = f32x4{y[4 * q], y[4 * q + 1], y[4 * q + 2], y[4 * q + 3]};
  }
}

// Bound by memory: the rows that it writes, 256 contiguous bytes (dim 128,
// bfloat16) for each token and head.  32 prefixes of up to 8192 positions: 732
// MB in 131 us, 5.6 TB/s; one thread for 8 numbers wherever they lie took 305.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void read_kernel(TileArgs a) {
  using F = Format<D>;
  constexpr int N = D / 16, W = (N + 7) / 8;
  const CacheView& c = a.c;
  if ((int)blockIdx.x >= a.blocks) return report(c, (int)blockIdx.x - a.blocks, a.status);
  Tile t;
  if (!tile_of(a, blockIdx.x * kWaves + (unsigned)uni((int)(threadIdx.x >> 6)), t)) return;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4, P = 1 << c.page_log2;
  const uint8_t* rec = c.data + ((int64_t)max(t.page, 0) * c.heads + t.h) * F::record(P);
  const int live = t.count < 0 ? c.n : t.count, r = t.r0 + 4 * g, blk = i / (32 / N);
  const int64_t row0 = ((int64_t)t.b * c.n + t.token0 + 4 * g) * c.heads + t.h;
  uint32_t k[4][W], v[4][W];
  unsigned ks[4], vs[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
#pragma unroll
    for (int q = 0; q < W; ++q) k[j][q] = v[j][q] = 0;
    ks[j] = vs[j] = kNaNScale;
  }
  if (t.page >= 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      load_codes<N>(rec + F::keys(r + j) + i * (N / 2), k[j]);
      ks[j] = rec[F::key_scales(P, r + j) + blk];
    }
    const uint32_t* at = reinterpret_cast<const uint32_t*>(rec + F::values(P, r, i));
    if constexpr (N == 4) {
      const uint64_t x = *reinterpret_cast<const uint64_t*>(at);
#pragma unroll
      for (int j = 0; j < 4; ++j) v[j][0] = (uint32_t)(x >> (16 * j)) & 0xFFFFu;
    } else {
#pragma unroll
      for (int q = 0; q < N / 8; ++q) {
        const u32x4 x = reinterpret_cast<const u32x4*>(at)[q];
#pragma unroll
        for (int y = 0; y < 4; ++y) v[(4 * q + y) / W][(4 * q + y) % W] = x[y];
      }
    }
    const uint32_t s4 = *reinterpret_cast<const uint32_t*>(rec + F::value_scale(P, r, blk));
#pragma unroll
    for (int j = 0; j < 4; ++j) vs[j] = s4 >> (8 * j) & 255;
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int token = t.token0 + 4 * g + j;
    if (token < 0 || token >= live) continue;
    const int64_t to = (row0 + (int64_t)j * c.heads) * D + i * N;
    store_row<DT, N>(a.out_k, to, k[j], ks[j]);
    store_row<DT, N>(a.out_v, to, v[j], vs[j]);
  }
}

template <class Launch>
int by_dim_and_type(int dim, int dtype, Launch launch) {
  (void)hipGetLastError();
  const bool bf = dtype == SPEC_BF16;
  switch (dim) {
    case 64: bf ? launch(std::integral_constant<int, 64>{}, std::integral_constant<int, kBF16>{}) : launch(std::integral_constant<int, 64>{}, std::integral_constant<int, kF32>{}); break;
    case 128: bf ? launch(std::integral_constant<int, 128>{}, std::integral_constant<int, kBF16>{}) : launch(std::integral_constant<int, 128>{}, std::integral_constant<int, kF32>{}); break;
    default: bf ? launch(std::integral_constant<int, 256>{}, std::integral_constant<int, kBF16>{}) : launch(std::integral_constant<int, 256>{}, std::integral_constant<int, kF32>{}); break;
  }
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}

// Tiles of 16 positions that n tokens can touch, and work-groups for B
// sequences' tiles: at most B * n * heads tiles, which check_cache keeps within 28 bits.
int tiles_of(int n) { return (n + 14) / 16 + 1; }
int blocks_for(const spec_cache* c, int B, int n, int waves_per_tile) {
  return (int)(((int64_t)B * tiles_of(n) * c->heads * waves_per_tile + kWaves - 1) / kWaves);
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_cache_page_bytes(int page, int dim) {
  return sv::page_log2_of(page) < 0 || !sv::dim_ok(dim) ? 0 : (size_t)page * (size_t)(dim + dim / 16);
}

extern "C" int spec_cache_append(const spec_cache* cache, const void* k, const void* v, int dtype,
                                 int64_t k_stride, int64_t v_stride, const int32_t* len, int lag,
                                 const int32_t* count, int B, int n, int32_t* status, void* stream) {
  using namespace sv;
  if (const int st = check_cache(cache, lag, B, n, dtype)) return st;
  if (k_stride < 0 || v_stride < 0) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  if (const int st = check_buffers(cache)) return st;
  const uintptr_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!k || !v || ((uintptr_t)k % es) || ((uintptr_t)v % es)) return SPEC_EINVAL;
  const int blocks = blocks_for(cache, B, n, 2);
  const TileArgs a{view_of(cache, len, lag, count, B, n), k, v, k_stride, v_stride, nullptr, nullptr, status, tiles_of(n), blocks};
  const dim3 grid(blocks + (status ? B : 0));
  return by_dim_and_type(cache->dim, dtype, [&](auto d, auto t) {
    hipLaunchKernelGGL((append_kernel<decltype(d)::value, decltype(t)::value>), grid, dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), a);
  });
}

extern "C" int spec_cache_read(const spec_cache* cache, const int32_t* len, int lag, const int32_t* count,
                               int B, int n, void* out_k, void* out_v, int dtype, int32_t* status,
                               void* stream) {
  using namespace sv;
  if (const int st = check_cache(cache, lag, B, n, dtype)) return st;
  if (B == 0) return SPEC_OK;
  if (const int st = check_buffers(cache)) return st;
  if (!out_k || !out_v || off16(out_k) || off16(out_v)) return SPEC_EINVAL;
  const int blocks = blocks_for(cache, B, n, 1);
  const TileArgs a{view_of(cache, len, lag, count, B, n), nullptr, nullptr, 0, 0, out_k, out_v, status, tiles_of(n), blocks};
  const dim3 grid(blocks + (status ? B : 0));
  return by_dim_and_type(cache->dim, dtype, [&](auto d, auto t) {
    hipLaunchKernelGGL((read_kernel<decltype(d)::value, decltype(t)::value>), grid, dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), a);
  });
}
