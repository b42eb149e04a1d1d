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

struct AppendArgs {
  CacheView c;
  const void* k;
  const void* v;
  int64_t k_stride, v_stride;
  int32_t* status;
  int blocks;   // work-groups per half (keys, values); those behind write the status
};

// One thread per 8 numbers; the 4 threads of a block of 32 are neighbours in
// a wave and share its largest magnitude through two quad permutes.  Bound by
// memory: 8 numbers in, 4 bytes and a quarter of a scale out.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void append_kernel(AppendArgs a) {
  using F = Format<D>;
  const CacheView& c = a.c;
  if ((int)blockIdx.x >= 2 * a.blocks) return report(c, (int)blockIdx.x - 2 * a.blocks, a.status);
  const bool values = (int)blockIdx.x >= a.blocks;
  const unsigned per_token = (unsigned)c.heads * (D / 8);
  const unsigned unit = ((unsigned)blockIdx.x - (values ? a.blocks : 0)) * kThreads + threadIdx.x;
  const unsigned token = unit / per_token, in_token = unit - token * per_token;
  // per_token is a multiple of 8, so the four threads of a block leave together.
  if (token >= (unsigned)c.B * (unsigned)c.n) return;
  const int b = token / (unsigned)c.n, i = token - b * c.n;
  const Span s = span_of(c, b);
  if (i >= s.count) return;
  const int t = s.pos + i;
  const int page = page_of(c, b, t);
  if (page < 0) return;
  const int h = in_token / (D / 8), d0 = (in_token % (D / 8)) * 8;

  float x[8];
  load_row8<DT>(values ? a.v : a.k, (int64_t)token * (values ? a.v_stride : a.k_stride) + h * D + d0, x);
  float m = 0.0f;
  int odd = 0;   // a NaN or an infinity
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    m = fmaxf(m, fabsf(x[e]));
    odd |= !(fabsf(x[e]) <= FLT_MAX);
  }
  m = fmaxf(m, dpp<kDppQuad1032>(m, m));
  m = fmaxf(m, dpp<kDppQuad2301>(m, m));
  odd |= dpp<kDppQuad1032>(odd, odd);
  odd |= dpp<kDppQuad2301>(odd, odd);
  // a = f 2^(E - 127), 1 <= f < 2: the smallest power of two s with a <= 7 s
  // is 2^(E - 129) up to f = 1.75 and 2^(E - 128) above.  Below the normal
  // range E = 0 and the clamp decides.
  const unsigned bits = __float_as_uint(m);
  int e = (int)(bits >> 23) - 2 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  e = e < 3 ? 3 : e > 252 ? 252 : e;
  const float scale = scale_of((unsigned)e);
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
  if (odd) w = 0;

  const int P = 1 << c.page_log2, r = t & (P - 1);
  uint8_t* rec = c.data + ((int64_t)page * c.heads + h) * F::record(P);
  if (!values) {
    *reinterpret_cast<uint32_t*>(rec + F::keys(r) + d0 / 2) = w;
    if ((d0 & 31) == 0) rec[F::key_scales(P, r) + d0 / 32] = (uint8_t)(odd ? kNaNScale : e);
  } else {
    const int share = d0 / (D / 16);
    uint8_t* at = rec + F::values(P, r, share);
    if constexpr (D == 64) {   // two shares of 4 numbers
      *reinterpret_cast<uint16_t*>(at) = (uint16_t)w;
      *reinterpret_cast<uint16_t*>(at + 4 * F::kPiece) = (uint16_t)(w >> 16);
    } else {
      *reinterpret_cast<uint32_t*>(at + (d0 % (D / 16)) / 2) = w;
    }
    if ((d0 & 31) == 0) rec[F::value_scale(P, r, d0 / 32)] = (uint8_t)(odd ? kNaNScale : e);
  }
}

struct ReadArgs {
  CacheView c;
  void* out_k;
  void* out_v;
  int32_t* status;
  int blocks;
};

typedef float f32x2 __attribute__((ext_vector_type(2)));

// One thread per 8 numbers, as append.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void read_kernel(ReadArgs a) {
  using F = Format<D>;
  const CacheView& c = a.c;
  if ((int)blockIdx.x >= 2 * a.blocks) return report(c, (int)blockIdx.x - 2 * a.blocks, a.status);
  const bool values = (int)blockIdx.x >= a.blocks;
  const unsigned per_token = (unsigned)c.heads * (D / 8);
  const unsigned unit = ((unsigned)blockIdx.x - (values ? a.blocks : 0)) * kThreads + threadIdx.x;
  const unsigned token = unit / per_token, in_token = unit - token * per_token;
  if (token >= (unsigned)c.B * (unsigned)c.n) return;
  const int b = token / (unsigned)c.n, i = token - b * c.n;
  const Span s = span_of(c, b);
  if (s.count >= 0 && i >= s.count) return;
  const int h = in_token / (D / 8), d0 = (in_token % (D / 8)) * 8;
  const int t = s.pos + i;
  const int page = s.count < 0 ? -1 : page_of(c, b, t);
  float x[8];
  unsigned e = kNaNScale;
  uint32_t w = 0;
  if (page >= 0) {
    const int P = 1 << c.page_log2, r = t & (P - 1);
    const uint8_t* rec = c.data + ((int64_t)page * c.heads + h) * F::record(P);
    if (!values) {
      w = *reinterpret_cast<const uint32_t*>(rec + F::keys(r) + d0 / 2);
      e = rec[F::key_scales(P, r) + d0 / 32];
    } else {
      const uint8_t* at = rec + F::values(P, r, d0 / (D / 16));
      if constexpr (D == 64) {
        w = *reinterpret_cast<const uint16_t*>(at) | (uint32_t)*reinterpret_cast<const uint16_t*>(at + 4 * F::kPiece) << 16;
      } else {
        w = *reinterpret_cast<const uint32_t*>(at + (d0 % (D / 16)) / 2);
      }
      e = rec[F::value_scale(P, r, d0 / 32)];
    }
  }
  const float scale = scale_of(e);
  const f32x2 y0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 0);
  const f32x2 y1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 1);
  const f32x2 y2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 2);
  const f32x2 y3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, scale, 3);
  x[0] = y0.x; x[1] = y0.y; x[2] = y1.x; x[3] = y1.y;
  x[4] = y2.x; x[5] = y2.y; x[6] = y3.x; x[7] = y3.y;
  if (e == kNaNScale) {
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(0x7FC00000u);
  }
  void* out = values ? a.out_v : a.out_k;
  const int64_t at = (int64_t)unit * 8;
  if constexpr (DT == kBF16) {
    // Exact: 2 significant bits, and the scale keeps it in the normal range.
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = (__float_as_uint(x[2 * j]) >> 16) | (__float_as_uint(x[2 * j + 1]) & 0xFFFF0000u);
    *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(out) + at) = o;
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
    p[0] = f32x4{x[0], x[1], x[2], x[3]};
    p[1] = f32x4{x[4], x[5], x[6], x[7]};
  }
}

template <class Args, class Launch>
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

// Work-groups for B * n tokens' keys (or values).  check_cache keeps the units within 31 bits.
int blocks_for(const spec_cache* c, int B, int n) {
  const int64_t units = (int64_t)B * n * c->heads * (c->dim / 8);
  return (int)((units + kThreads - 1) / kThreads);
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
  const int blocks = blocks_for(cache, B, n);
  const AppendArgs a{view_of(cache, len, lag, count, B, n), k, v, k_stride, v_stride, status, blocks};
  const dim3 grid(2 * blocks + (status ? B : 0));
  return by_dim_and_type<AppendArgs>(cache->dim, dtype, [&](auto d, auto t) {
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
  const int blocks = blocks_for(cache, B, n);
  const ReadArgs a{view_of(cache, len, lag, count, B, n), out_k, out_v, status, blocks};
  const dim3 grid(2 * blocks + (status ? B : 0));
  return by_dim_and_type<ReadArgs>(cache->dim, dtype, [&](auto d, auto t) {
    hipLaunchKernelGGL((read_kernel<decltype(d)::value, decltype(t)::value>), grid, dim3(kThreads), 0,
                       static_cast<hipStream_t>(stream), a);
  });
}
