// Attention of a round's new tokens over the 4-bit key/value cache
// (spec_verify.h describes the format, the visibility rule and the errors).
#include "format.h"

#include <math.h>

namespace sv {
namespace {

struct AttentionArgs {
  CacheView c;
  const void* q;
  int64_t q_stride;
  int heads_q, group;   // query heads, query heads per key/value head
  float scale;
  int window;
  const uint64_t* mask;
  void* out;
  float* lse;
};

template <int DT>
__device__ __forceinline__ void store_one(void* out, int64_t j, float v) {
  if constexpr (DT == kBF16) {
    static_cast<__bf16*>(out)[j] = (__bf16)v;
  } else {
    static_cast<float*>(out)[j] = v;
  }
}

// Number d of token r's key (value) in a record; NaN for a NaN block.
template <int D>
__device__ __forceinline__ float code_value(unsigned byte, int d, unsigned e) {
  const unsigned code = (d & 1) ? byte >> 4 : byte & 15;
  const unsigned m = code & 7;
  const float mag = m < 2 ? 0.5f * m : (1.0f + 0.5f * (m & 1)) * (float)(1u << ((m >> 1) - 1));
  return e == kNaNScale ? __uint_as_float(0x7FC00000u) : ((code & 8) ? -mag : mag) * scale_of(e);
}

// The plain kernel: one work-group per query row, 256 keys at a time; each
// thread scores one key, then the threads split the numbers of the output.
// m and l are the running maximum and sum of the softmax.
template <int D, int DT>
__global__ __launch_bounds__(kThreads) void attention_kernel(AttentionArgs a) {
  using F = Format<D>;
  constexpr int kParts = kThreads / D;
  __shared__ float qs[D], ps[kThreads], red[kWaves], accs[kThreads];
  const CacheView& c = a.c;
  const int64_t row = (int64_t)blockIdx.x;
  const int hq = row % a.heads_q, token = row / a.heads_q;
  const int b = token / c.n, i = token % c.n, h = hq / a.group;
  const Span s = span_of(c, b);
  const int tid = threadIdx.x, d = tid % D, part = tid / D;
  if (s.count >= 0 && i >= s.count) return;
  const float nan = __uint_as_float(0x7FC00000u);
  if (s.count < 0) {
    if (part == 0) store_one<DT>(a.out, row * D + d, nan);
    if (a.lse && tid == 0) a.lse[row] = nan;
    return;
  }
  if (tid < D) qs[tid] = load_one<DT>(a.q, token * a.q_stride + (int64_t)hq * D + tid);
  const int at = s.pos + i;
  const int hi = a.mask ? s.pos + s.count : at + 1;
  const int lo = a.window > 0 && at - a.window + 1 > 0 ? at - a.window + 1 : 0;
  const uint64_t bits = a.mask ? a.mask[(int64_t)b * c.n + i] : 0;
  const int P = 1 << c.page_log2;
  float m = -INFINITY, l = 0.0f, acc = 0.0f;
  int nan_row = 0;
  for (int t0 = lo; t0 < hi; t0 += kThreads) {
    __syncthreads();
    const int t = t0 + tid;
    bool sees = t < hi;
    if (sees && a.mask && t >= s.pos) sees = (bits >> (t - s.pos)) & 1;
    float x = -INFINITY;
    if (sees) {
      const int page = c.table[(int64_t)b * c.table_len + (t >> c.page_log2)];
      if (page < 0 || page >= c.pages) {
        nan_row = 1;
      } else {
        const int r = t & (P - 1);
        const uint8_t* rec = c.data + ((int64_t)page * c.heads + h) * F::record(P);
        float dot = 0.0f;
        for (int j = 0; j < D; ++j)
          dot += qs[j] * code_value<D>(rec[F::keys(r) + j / 2], j, rec[F::key_scales(P, r) + j / 32]);
        x = dot * a.scale;
        for (int j = 0; j < F::kBlocks; ++j)
          nan_row |= rec[F::value_scale(P, r, j)] == kNaNScale || rec[F::key_scales(P, r) + j] == kNaNScale;
        nan_row |= x != x;
      }
    }
    float top = x;
    for (int off = 32; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    if ((tid & 63) == 0) red[tid >> 6] = top;
    __syncthreads();
    top = fmaxf(fmaxf(fmaxf(red[0], red[1]), fmaxf(red[2], red[3])), m);
    const float safe = top == -INFINITY ? 0.0f : top;
    const float alpha = expf(m - safe);
    ps[tid] = sees ? expf(x - safe) : 0.0f;
    m = top;
    l = l * alpha;
    acc *= alpha;
    __syncthreads();
    for (int k = 0; k < kThreads; ++k) l += ps[k];
    for (int k = part; k < kThreads; k += kParts) {
      const float p = ps[k];
      if (p == 0.0f) continue;
      const int tk = t0 + k, r = tk & (P - 1);
      const int page = c.table[(int64_t)b * c.table_len + (tk >> c.page_log2)];
      if (page < 0 || page >= c.pages) continue;
      const uint8_t* rec = c.data + ((int64_t)page * c.heads + h) * F::record(P);
      const int share = d / (D / 16);
      acc += p * code_value<D>(rec[F::values(P, r, share) + d % (D / 16) / 2], d, rec[F::value_scale(P, r, d / 32)]);
    }
  }
  nan_row = __syncthreads_or(nan_row);
  accs[tid] = acc;
  __syncthreads();
  if (part == 0) {
    for (int p = 1; p < kParts; ++p) acc += accs[p * D + d];
    store_one<DT>(a.out, row * D + d, nan_row ? nan : l > 0.0f ? acc / l : 0.0f);
  }
  if (a.lse && tid == 0) a.lse[row] = nan_row ? nan : m + logf(l);
}

int check_attention(int B, int n, int heads_q, int heads, int dim) {
  if (B < 0 || n < 1 || heads < 1 || heads_q < heads || heads_q % heads || !dim_ok(dim)) return SPEC_EINVAL;
  if ((int64_t)B * n > ((int64_t)1 << 24)) return SPEC_EINVAL;
  if (B > 0 && heads_q > (((int64_t)1 << 34) / dim) / ((int64_t)B * n)) return SPEC_EINVAL;
  const int64_t groups = ((int64_t)n * (heads_q / heads) + 15) / 16;
  if (B > 0 && groups * heads > ((int64_t)1 << 24) / B) return SPEC_EINVAL;
  return SPEC_OK;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_cache_attention_workspace_bytes(int B, int n, int heads_q, int heads, int dim) {
  return B == 0 || sv::check_attention(B, n, heads_q, heads, dim) ? 0 : 256;
}

extern "C" int spec_cache_attention(const spec_cache* cache, const void* q, int dtype, int64_t q_stride,
                                    int heads_q, const int32_t* len, int lag, const int32_t* count, int B,
                                    int n, float scale, int window, const uint64_t* mask, void* out,
                                    float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  using namespace sv;
  if (const int st = check_cache(cache, lag, B, n, dtype)) return st;
  if (const int st = check_attention(B, n, heads_q, cache->heads, cache->dim)) return st;
  if (q_stride < 0 || window < 0 || !isfinite(scale) || (mask && n > 64)) return SPEC_EINVAL;
  if (B == 0) return SPEC_OK;
  if (const int st = check_buffers(cache)) return st;
  const uintptr_t es = dtype == SPEC_BF16 ? 2 : 4;
  if (!q || ((uintptr_t)q % es) || !out || off16(out)) return SPEC_EINVAL;
  if (!workspace || workspace_bytes < spec_cache_attention_workspace_bytes(B, n, heads_q, cache->heads, cache->dim))
    return SPEC_EWORKSPACE;
  const AttentionArgs a{view_of(cache, len, lag, count, B, n), q, q_stride, heads_q, heads_q / cache->heads, scale, window, mask, out, lse};
  (void)hipGetLastError();
  const dim3 grid((unsigned)B * (unsigned)n * (unsigned)heads_q);
  const hipStream_t st = static_cast<hipStream_t>(stream);
#define SV_LAUNCH(D)                                                                                         \
  if (dtype == SPEC_BF16)                                                                                    \
    hipLaunchKernelGGL((attention_kernel<D, kBF16>), grid, dim3(kThreads), 0, st, a);                        \
  else                                                                                                       \
    hipLaunchKernelGGL((attention_kernel<D, kF32>), grid, dim3(kThreads), 0, st, a)
  switch (cache->dim) {
    case 64: SV_LAUNCH(64); break;
    case 128: SV_LAUNCH(128); break;
    default: SV_LAUNCH(256); break;
  }
#undef SV_LAUNCH
  return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;
}
