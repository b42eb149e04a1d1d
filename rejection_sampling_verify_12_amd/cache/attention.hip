// Attention of a round's new tokens over the 4-bit key/value cache
// (spec_verify.h describes the format, the visibility rule and the errors).
//
// The query rows of one sequence that share a key/value head (n tokens times
// heads_q / heads) are cut into groups of RT tiles of 16.  A work-group takes
// a group and a run of keys; each of its 4 waves takes blocks of 32 keys, 4
// blocks (a unit of 128 keys) at a time, with no shared memory in the loop:
//
//   S^T = K Q^T       16x16x32 products: rows = 16 keys, columns = 16 queries.
//   P = 2^(c S - m)   c = |scale| log2 e; a lane holds 8 keys of one query.
//   O^T += V^T P^T    rows = 16 numbers of the vector, columns = 16 queries,
//                     summed over the 32 keys.
//
// Both products accept any order of their summed index as long as both
// operands use the same.  That is used twice: a lane's 16 (at dim 128) bytes
// of keys are contiguous and share one scale, and the lane that holds 8 weights of
// a query after the first product needs exactly those 8 keys in the second, so
// the weights never move between lanes.  Column = query in both products, so
// the softmax's maximum, sum and rescaling are one register per lane.
#include "format.h"

#include <float.h>
#include <math.h>

namespace sv {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;               // keys per wave and step
constexpr int kUnitKeys = kWaves * kBlock;   // keys per work-group and step
constexpr int kCUs = 256;                // MI355X

struct AttentionArgs {
  CacheView c;
  const void* q;
  int64_t q_stride;
  int heads_q, group;   // query heads, query heads per key/value head
  int groups;           // row groups per sequence and key/value head
  float c2;             // |scale| log2(e)
  int flip, zero;       // scale < 0; scale == 0 (or too small for a float): the queries are taken as 0
  int window;
  const uint64_t* mask;
  void* out;
  float* lse;
  unsigned* arrivals;   // [B * groups * heads]: parts of an item that are in the workspace
  float* parts;         // [2 * grid]: a part's sums [rows][D], maxima [rows], sums [rows]
};

template <int DT>
constexpr int kTerms = DT == kBF16 ? 1 : 3;   // bfloat16 parts that a query or a weight is cut into

// Waves per SIMD the registers of a variant leave room for.
constexpr int waves_for(int D, int dt, int rt) {
  const int terms = dt == kBF16 ? 1 : 3;
  const int regs = rt * (D / 4 + terms * D / 8) + 96;
  return regs <= 160 ? 3 : regs <= 250 ? 2 : 1;
}
// Row tiles of a group, at most.
constexpr int max_tiles(int D, int dt) { return dt == kBF16 ? (D == 256 ? 2 : 4) : (D == 256 ? 1 : 2); }
// Row tiles per group for rows of one sequence and head: as many groups as the
// largest tile count needs, the tiles spread evenly over them.
inline int tiles_for(int D, int dt, int64_t rows) {
  const int64_t tiles = (rows + 15) / 16, groups = (tiles + max_tiles(D, dt) - 1) / max_tiles(D, dt);
  return (int)((tiles + groups - 1) / groups);
}

// The keys a row group looks at.
struct Item {
  Span s;
  int tok0, tok1;   // its first and last token
  int lo, hi;       // positions, lo on a block's border
  int units;        // 0: no row of the group is in use
};

__device__ __forceinline__ Item item_of(const AttentionArgs& a, int b, int rg, int rows) {
  Item it;
  it.s = span_of(a.c, b);
  const int used = it.s.count < 0 ? a.c.n : it.s.count;
  it.tok0 = rg * rows / a.group;
  it.tok1 = min((rg * rows + rows - 1) / a.group, used - 1);
  if (it.tok0 >= used) {
    it.units = 0;
    return it;
  }
  if (it.s.count < 0) {   // one unit that writes NaN
    it.units = 1;
    it.lo = it.hi = 0;
    return it;
  }
  it.hi = a.mask ? it.s.pos + it.s.count : it.s.pos + it.tok1 + 1;
  it.lo = a.window > 0 ? max(0, it.s.pos + it.tok0 + 1 - a.window) & ~(kBlock - 1) : 0;
  it.units = (it.hi - it.lo + kUnitKeys - 1) / kUnitKeys;
  return it;
}

// A lane's share of a block: codes and scales of 2 tiles of 16 keys.
template <int D>
struct Codes {
  uint32_t k[2][D / 32], v[2][D / 32];
  uint32_t ks[2], vs[2];
};

template <int D>
__device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[D / 32]) {
  if constexpr (D == 64) {
    const u32x2 t = *reinterpret_cast<const u32x2*>(p);
    w[0] = t.x; w[1] = t.y;
  } else {
#pragma unroll
    for (int x = 0; x < D / 128; ++x) {
      const u32x4 t = reinterpret_cast<const u32x4*>(p)[x];
      w[4 * x] = t.x; w[4 * x + 1] = t.y; w[4 * x + 2] = t.z; w[4 * x + 3] = t.w;
    }
  }
}

// Block of keys p .. p + 31 of one page; page < 0: NaN blocks.
template <int D>
__device__ __forceinline__ void load_codes(const AttentionArgs& a, int page, int h, int p, int lane, Codes<D>& x) {
  using F = Format<D>;
  const int i = lane & 15, g = lane >> 4;
  if (page >= 0) {
    const int P = 1 << a.c.page_log2, r = p & (P - 1);
    const uint8_t* rec = a.c.data + ((int64_t)page * a.c.heads + h) * F::record(P);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      load_words<D>(rec + F::keys(r + 16 * t) + (i * F::kRow + g * (D / 8)), x.k[t]);
      const uint8_t* ks = rec + F::key_scales(P, r + 16 * t) + i * F::kBlocks;
      if constexpr (D == 256) {
        x.ks[t] = *reinterpret_cast<const uint16_t*>(ks + 2 * g);
      } else {
        x.ks[t] = ks[D == 128 ? g : g >> 1];
      }
    }
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      load_words<D>(rec + F::values(P, r + 16 * t, 0) + (g * (2 * D) + i * (D / 8)), x.v[t]);
      x.vs[t] = *reinterpret_cast<const uint32_t*>(rec + F::value_scale(P, r + 16 * t, 0) + (i * (D / 16) / 32 * 16 + 4 * g));
    }
  } else {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int c = 0; c < D / 32; ++c) x.k[t][c] = x.v[t][c] = 0;
      x.ks[t] = D == 256 ? 0xFFFFu : 0xFFu;
      x.vs[t] = 0xFFFFFFFFu;
    }
  }
}

// Some byte of w is 255.
__device__ __forceinline__ uint32_t has_ff(uint32_t w) {
  return ((w & 0x7F7F7F7Fu) + 0x01010101u) & w & 0x80808080u;
}

__device__ __forceinline__ uint32_t cvt_pair(uint32_t w, float scale, int byte) {
  switch (byte) {   // the selector is an immediate
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
}
__device__ __forceinline__ bf16x8 as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(bf16x8, u32x4{a, b, c, d});
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, bf16x2{(__bf16)a, (__bf16)b});
}
// x as TERMS bfloat16 parts, each the rounded rest of the ones before (to nearest even).
template <int TERMS>
__device__ __forceinline__ void split8(const float (&x)[8], bf16x8 (&out)[TERMS]) {
  float rest[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) rest[e] = x[e];
#pragma unroll
  for (int t = 0; t < TERMS; ++t) {
    uint32_t w[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) w[e] = pack_bf16(rest[2 * e], rest[2 * e + 1]);
    out[t] = as_bf16x8(w[0], w[1], w[2], w[3]);
    if (t + 1 < TERMS) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        rest[2 * e] -= bf16_lo(w[e]);
        rest[2 * e + 1] -= bf16_hi(w[e]);
      }
    }
  }
}

template <int D, int DT, int RT>
struct State {   // one wave's running result; a lane holds query (lane & 15) of each tile
  f32x4 o[RT][D / 16];
  float m[RT], l[RT];   // maximum (base 2), and the sum over the lane's own keys
};

template <int D, int DT, int RT>
struct Rows {   // the group's queries
  bf16x8 q[RT][D / 32][kTerms<DT>];
  int token[RT];
};

template <int D, int DT, int RT>
__device__ __forceinline__ void attend_block(const AttentionArgs& a, const Item& it, int b, int p, int lane,
                                             Codes<D>& x, const Rows<D, DT, RT>& rows, State<D, DT, RT>& st) {
  constexpr int T = kTerms<DT>;
  const int g = lane >> 4;
  const f32x4 zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const bool full = p + kBlock - 1 <= (a.mask ? it.s.pos - 1 : it.s.pos + it.tok0) &&
                    (a.window == 0 || p > it.s.pos + it.tok1 - a.window);
  // Keys with a NaN block (rare): bit 16 t + key of the tile.
  uint32_t nan_keys = 0;
  if (__any((int)(has_ff(x.ks[0]) | has_ff(x.ks[1]) | has_ff(x.vs[0]) | has_ff(x.vs[1])))) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      uint64_t k = __ballot(has_ff(x.ks[t]) != 0);
      k |= k >> 32;
      uint32_t keys = (uint32_t)(k | k >> 16) & 0xFFFFu;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        const bool bad = (x.vs[t] >> (8 * jj) & 255) == 255;
        const uint64_t v = __ballot(bad);
#pragma unroll
        for (int gg = 0; gg < 4; ++gg) keys |= (v >> (16 * gg) & 0xFFFF) ? 1u << (4 * gg + jj) : 0u;
        // The row's weight says NaN; the value itself must not reach other rows.
        if (bad) x.vs[t] = (x.vs[t] & ~(255u << (8 * jj))) | 127u << (8 * jj);
      }
      nan_keys |= keys << (16 * t);
    }
  }
  if (!full) {
    // Places behind the last token hold anything: no scale of theirs may give an infinity.
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) {
        if ((x.vs[t] >> (8 * jj) & 255) > 252) x.vs[t] = (x.vs[t] & ~(255u << (8 * jj))) | 127u << (8 * jj);
      }
    }
  }

  f32x4 s[RT][2];
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    const float s0 = scale_of(x.ks[t] & 255), s1 = D == 256 ? scale_of(x.ks[t] >> 8) : s0;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) s[rt][t] = zero;
#pragma unroll
    for (int c = 0; c < D / 32; ++c) {
      const uint32_t w = x.k[t][c];
      const float sc = (D == 256 && c >= 4) ? s1 : s0;
      const bf16x8 k = as_bf16x8(cvt_pair(w, sc, 0), cvt_pair(w, sc, 1), cvt_pair(w, sc, 2), cvt_pair(w, sc, 3));
#pragma unroll
      for (int rt = 0; rt < RT; ++rt)
#pragma unroll
        for (int e = T - 1; e >= 0; --e)
          s[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, rows.q[rt][c][e], s[rt][t], 0, 0, 0);
    }
  }

  bf16x8 w[RT][T];
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    if (!full || nan_keys) {
      const int at = it.s.pos + rows.token[rt];
      const int last = a.mask ? it.s.pos - 1 : at;
      const uint64_t bits = (a.mask && rows.token[rt] < it.s.count) ? a.mask[(int64_t)b * a.c.n + rows.token[rt]] : 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int key = p + 16 * (e >> 2) + 4 * g + (e & 3);
        bool sees = key <= last && rows.token[rt] < it.s.count;
        if (a.mask && key >= it.s.pos && key < it.s.pos + it.s.count) sees = bits >> (key - it.s.pos) & 1;
        if (a.window > 0) sees = sees && key > at - a.window;
        const float v = (nan_keys >> (16 * (e >> 2) + 4 * g + (e & 3)) & 1) ? __uint_as_float(0x7FC00000u) : s[rt][e >> 2][e & 3];
        s[rt][e >> 2][e & 3] = sees ? v : -INFINITY;
      }
    }
    const f32x4 x0 = s[rt][0], x1 = s[rt][1];
    float top = fmaxf(fmaxf(fmaxf(x0[0], x0[1]), fmaxf(x0[2], x0[3])), fmaxf(fmaxf(x1[0], x1[1]), fmaxf(x1[2], x1[3])));
    const auto max2 = [](float u, float v) { return fmaxf(u, v); };
    top = swap_combine<16>(top, max2);
    top = swap_combine<32>(top, max2) * a.c2;
    const float m = fmaxf(st.m[rt], top);
    const float safe = m == -INFINITY ? 0.0f : m;
    if (__any(m > st.m[rt])) {
      const float alpha = exp2_fast(st.m[rt] - safe);
      st.l[rt] *= alpha;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) st.o[rt][d] *= alpha;
      st.m[rt] = m;
    }
    float pr[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) pr[e] = exp2_fast(fmaf(s[rt][e >> 2][e & 3], a.c2, -safe));
    st.l[rt] += ((pr[0] + pr[1]) + (pr[2] + pr[3])) + ((pr[4] + pr[5]) + (pr[6] + pr[7]));
    split8<T>(pr, w[rt]);
  }

  float vsc[2][4];
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) vsc[t][jj] = scale_of(x.vs[t] >> (8 * jj) & 255);
  // Numbers 2 d and 2 d + 1 of the lane's D / 16, for its 8 keys.  Token jj's
  // codes are bytes jj * D/32 on of the lane's share.
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int byte = (e & 3) * (D / 32) + d;
      y[e] = cvt_pair(x.v[e >> 2][byte / 4], vsc[e >> 2][e & 3], byte % 4);
    }
    uint32_t even[4], odd[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      even[e] = __builtin_amdgcn_perm(y[2 * e + 1], y[2 * e], 0x05040100u);
      odd[e] = __builtin_amdgcn_perm(y[2 * e + 1], y[2 * e], 0x07060302u);
    }
    const bf16x8 v0 = as_bf16x8(even[0], even[1], even[2], even[3]), v1 = as_bf16x8(odd[0], odd[1], odd[2], odd[3]);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int e = T - 1; e >= 0; --e) {
        st.o[rt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, w[rt][e], st.o[rt][2 * d], 0, 0, 0);
        st.o[rt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, w[rt][e], st.o[rt][2 * d + 1], 0, 0, 0);
      }
    }
  }
}

// D / 16 numbers of a row of the output.
template <int D, int DT>
__device__ __forceinline__ void store_row(void* out, int64_t at, const float (&v)[D / 16]) {
  if constexpr (DT == kBF16) {
    uint32_t w[D / 32];
#pragma unroll
    for (int e = 0; e < D / 32; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at);
    if constexpr (D == 64) {
      *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int e = 0; e < D / 128; ++e) reinterpret_cast<u32x4*>(p)[e] = u32x4{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]};
    }
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int e = 0; e < D / 64; ++e) p[e] = f32x4{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
  }
}

__device__ __forceinline__ float ld_dev_f(const float* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void st_dev_f(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Work-groups take equal runs of units: run w is [w U / W, (w + 1) U / W) of all
// U units, ordered by sequence, row group, key/value head and key.  An item
// (all keys of one group and head) that lies in one run is written at once;
// otherwise each run's part goes to the workspace, and the last to arrive
// joins the parts in order.  A run has at most two such parts, its first and its last.
template <int D, int DT, int RT>
__global__ __launch_bounds__(kThreads, waves_for(D, DT, RT)) void attention_kernel(AttentionArgs a) {
  constexpr int R = 16 * RT, S = D / 16, kPart = R * (D + 2);
  __shared__ float sums[kWaves][16][D + 4];
  __shared__ float tops[kWaves][R], totals[kWaves][R];
  __shared__ int64_t scan[kWaves];
  __shared__ int64_t found_start;
  __shared__ int found_entry, is_last;
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int heads = a.c.heads, entries = a.c.B * a.groups;

  // Units before this thread's entries, and in all.
  const int per = (entries + kThreads - 1) / kThreads;
  const int e0 = min(tid * per, entries), e1 = min(e0 + per, entries);
  int64_t mine = 0;
  for (int e = e0; e < e1; ++e) mine += item_of(a, e / a.groups, e % a.groups, R).units;
  int64_t before = mine;
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t o = __shfl_up((long long)before, off);
    if (lane >= off) before += o;
  }
  if (lane == 63) scan[wave] = before;
  __syncthreads();
  before -= mine;
  int64_t all = 0;
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) before += scan[w];
    all += scan[w];
  }
  const int64_t U = all * heads;
  const int64_t W = U < (int64_t)gridDim.x ? U : (int64_t)gridDim.x;
  const int64_t run = blockIdx.x;
  if (run >= W) return;   // the whole work-group
  int64_t u = run * U / W;
  const int64_t u1 = (run + 1) * U / W, u_begin = u;
  if (before * heads <= u && u < (before + mine) * heads) {
    int64_t start = before * heads;
    for (int e = e0; e < e1; ++e) {
      const int64_t units = (int64_t)item_of(a, e / a.groups, e % a.groups, R).units * heads;
      if (u < start + units) {
        found_entry = e;
        found_start = start;
        break;
      }
      start += units;
    }
  }
  __syncthreads();
  int entry = uni(found_entry);
  int64_t entry_start = (int64_t)uni((uint64_t)found_start);

  while (u < u1) {
    const int b = entry / a.groups, rg = entry % a.groups;
    const Item it = item_of(a, b, rg, R);
    const int64_t entry_units = (int64_t)it.units * heads;
    if (u >= entry_start + entry_units) {
      entry_start += entry_units;
      ++entry;
      continue;
    }
    const int h = (int)((u - entry_start) / it.units);
    const int64_t u0 = entry_start + (int64_t)h * it.units;   // the item's first unit
    const int k0 = (int)(u - u0);
    const int k1 = (int)((u1 < u0 + it.units ? u1 : u0 + it.units) - u0);

    if (it.s.count < 0) {
      float nan[S];
#pragma unroll
      for (int d = 0; d < S; ++d) nan[d] = __uint_as_float(0x7FC00000u);
      for (int r = tid >> 4; r < R; r += 16) {
        const int row = rg * R + r, token = row / a.group, head = h * a.group + row % a.group;
        if (token >= a.c.n) break;
        const int64_t at = ((int64_t)b * a.c.n + token) * a.heads_q + head;
        store_row<D, DT>(a.out, at * D + (tid & 15) * S, nan);
        if (a.lse && (tid & 15) == 0) a.lse[at] = nan[0];
      }
      u += 1;
      continue;
    }

    Rows<D, DT, RT> rows;
    State<D, DT, RT> st;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = rg * R + rt * 16 + i, token = row / a.group, head = h * a.group + row % a.group;
      rows.token[rt] = token;
      const bool used = token < it.s.count && !a.zero;
      const int64_t at = ((int64_t)b * a.c.n + token) * a.q_stride + (int64_t)head * D + g * (D / 4);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (used) load_row8<DT>(a.q, at + 8 * c, x);
        if (a.flip) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = -x[e];
        }
        split8<kTerms<DT>>(x, rows.q[rt][c]);
      }
      st.m[rt] = -INFINITY;
      st.l[rt] = 0.0f;
#pragma unroll
      for (int d = 0; d < S; ++d) st.o[rt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }

    // The wave's blocks p = lo + 128 k + 32 wave below hi; codes are loaded one
    // block ahead, page numbers two.
    const int32_t* table = a.c.table + (int64_t)b * a.c.table_len;
    const int p1 = min(it.hi, it.lo + kUnitKeys * k1);
    int p = it.lo + kUnitKeys * k0 + kBlock * wave;
    const auto page_at = [&](int pos) {
      if (pos >= p1) return -1;
      const int page = table[pos >> a.c.page_log2];
      return (page >= 0 && page < a.c.pages) ? page : -1;
    };
    if (p < p1) {
      Codes<D> x, y;
      int next = uni(page_at(p));
      load_codes<D>(a, next, h, p, lane, x);
      next = uni(page_at(p + kUnitKeys));
      for (; p < p1; p += kUnitKeys) {
        if (p + kUnitKeys < p1) load_codes<D>(a, next, h, p + kUnitKeys, lane, y);
        next = uni(page_at(p + 2 * kUnitKeys));
        attend_block<D, DT, RT>(a, it, b, p, lane, x, rows, st);
        x = y;
      }
    }

    // Join the waves.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const auto add2 = [](float v, float w) { return v + w; };
      st.l[rt] = swap_combine<32>(swap_combine<16>(st.l[rt], add2), add2);
      if (g == 0) {
        tops[wave][rt * 16 + i] = st.m[rt];
        totals[wave][rt * 16 + i] = st.l[rt];
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == it.units;
    float* part = a.parts + (2 * run + (u == u_begin ? 0 : 1)) * kPart;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt > 0) __syncthreads();   // sums is read by the tile before
      {
        float m = tops[0][rt * 16 + i];
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][rt * 16 + i]);
        const float f = exp2_fast(st.m[rt] - (m == -INFINITY ? 0.0f : m));
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int d = 0; d < S; ++d) sums[wave][i][(4 * g + r) * S + d] = st.o[rt][d][r] * f;
      }
      __syncthreads();
      const int row16 = tid >> 4, share = tid & 15;
      float m = tops[0][rt * 16 + row16], l = 0.0f, v[S];
      for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][rt * 16 + row16]);
      const float safe = m == -INFINITY ? 0.0f : m;
      for (int w = 0; w < kWaves; ++w) l += totals[w][rt * 16 + row16] * exp2_fast(tops[w][rt * 16 + row16] - safe);
#pragma unroll
      for (int d = 0; d < S; ++d)
        v[d] = (sums[0][row16][share * S + d] + sums[1][row16][share * S + d]) + (sums[2][row16][share * S + d] + sums[3][row16][share * S + d]);
      if (whole) {
        const int row = rg * R + rt * 16 + row16, token = row / a.group, head = h * a.group + row % a.group;
        if (token < it.s.count) {
          const int64_t at = ((int64_t)b * a.c.n + token) * a.heads_q + head;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
          for (int d = 0; d < S; ++d) v[d] *= inv;
          store_row<D, DT>(a.out, at * D + share * S, v);
          if (a.lse && share == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
        }
      } else {
#pragma unroll
        for (int d = 0; d < S; ++d) st_dev_f(part + (rt * 16 + row16) * D + share * S + d, v[d]);
        if (share == 0) {
          st_dev_f(part + R * D + rt * 16 + row16, m);
          st_dev_f(part + R * D + R + rt * 16 + row16, l);
        }
      }
    }
    if (!whole) {
      const int64_t first = ((u0 + 1) * W - 1) / U, last = ((u0 + it.units) * W - 1) / U;   // runs with a part
      unsigned* arrived = a.arrivals + (int64_t)entry * heads + h;
      wait_mem();
      __syncthreads();
      if (tid == 0) {
        const unsigned was = __hip_atomic_fetch_add(arrived, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        is_last = was == (unsigned)(last - first);
        if (is_last) __hip_atomic_store(arrived, 0u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
      }
      __syncthreads();
      if (uni(is_last)) {
        // The first run's part is its second one unless the item starts that run.
        const int64_t side0 = first * U / W < u0 ? 1 : 0;
        for (int rt = 0; rt < RT; ++rt) {
          const int row16 = tid >> 4, share = tid & 15;
          float m = -INFINITY, l = 0.0f, v[S];
#pragma unroll
          for (int d = 0; d < S; ++d) v[d] = 0.0f;
#pragma unroll 2
          for (int64_t w = first; w <= last; ++w) {
            const float* q = a.parts + (2 * w + (w == first ? side0 : 0)) * kPart;
            const float pm = ld_dev_f(q + R * D + rt * 16 + row16), pl = ld_dev_f(q + R * D + R + rt * 16 + row16);
            float pv[S];
#pragma unroll
            for (int d = 0; d < S; ++d) pv[d] = ld_dev_f(q + (rt * 16 + row16) * D + share * S + d);
            const float top = fmaxf(m, pm), safe = top == -INFINITY ? 0.0f : top;
            const float f0 = exp2_fast(m - safe), f1 = exp2_fast(pm - safe);
            m = top;
            l = l * f0 + pl * f1;
#pragma unroll
            for (int d = 0; d < S; ++d) v[d] = v[d] * f0 + pv[d] * f1;
          }
          const int row = rg * R + rt * 16 + row16, token = row / a.group, head = h * a.group + row % a.group;
          if (token < it.s.count) {
            const int64_t at = ((int64_t)b * a.c.n + token) * a.heads_q + head;
            const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
            for (int d = 0; d < S; ++d) v[d] *= inv;
            store_row<D, DT>(a.out, at * D + share * S, v);
            if (a.lse && share == 0) a.lse[at] = l == 0.0f ? -INFINITY : (m + log2f(l)) * 0.6931471805599453f;
          }
        }
      }
    }
    __syncthreads();
    u = u0 + k1;
  }
}

int check_attention(int B, int n, int heads_q, int heads, int dim) {
  if (B < 0 || n < 1 || heads < 1 || heads_q < heads || heads_q % heads || !dim_ok(dim)) return SPEC_EINVAL;
  if ((int64_t)B * n > ((int64_t)1 << 24)) return SPEC_EINVAL;
  if (B > 0 && heads_q > (((int64_t)1 << 34) / dim) / ((int64_t)B * n)) return SPEC_EINVAL;
  const int64_t groups = ((int64_t)n * (heads_q / heads) + 15) / 16;
  if (B > 0 && groups * heads > ((int64_t)1 << 24) / B) return SPEC_EINVAL;
  return SPEC_OK;
}

constexpr int grid_for(int D, int dt, int rt) { return kCUs * waves_for(D, dt, rt); }

// Bytes of the arrival counters: one for every item a call of these sizes can
// have, whatever its tiles.
size_t arrival_bytes(int B, int n, int heads_q, int heads) {
  const int64_t groups = ((int64_t)n * (heads_q / heads) + 15) / 16;
  return ((size_t)B * groups * heads * sizeof(unsigned) + 255) / 256 * 256;
}

}  // namespace
}  // namespace sv

extern "C" size_t spec_cache_attention_workspace_bytes(int B, int n, int heads_q, int heads, int dim) {
  using namespace sv;
  if (B == 0 || check_attention(B, n, heads_q, heads, dim)) return 0;
  // The largest over the variants of calls with as many rows or fewer.
  size_t parts = 0;
  for (int dt : {(int)kF32, (int)kBF16}) {
    const int64_t tiles = ((int64_t)n * (heads_q / heads) + 15) / 16;
    for (int rt = 1; rt <= max_tiles(dim, dt) && rt <= tiles; ++rt) {
      const size_t need = (size_t)2 * grid_for(dim, dt, rt) * 16 * rt * (dim + 2) * sizeof(float);
      parts = need > parts ? need : parts;
    }
  }
  return arrival_bytes(B, n, heads_q, heads) + (parts + 255) / 256 * 256;
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
  if (!workspace || off16(workspace) ||
      workspace_bytes < spec_cache_attention_workspace_bytes(B, n, heads_q, cache->heads, cache->dim))
    return SPEC_EWORKSPACE;
  AttentionArgs a;
  a.c = view_of(cache, len, lag, count, B, n);
  a.q = q;
  a.q_stride = q_stride;
  a.heads_q = heads_q;
  a.group = heads_q / cache->heads;
  const float c2 = fabsf(scale) * 1.4426950408889634f;
  a.zero = c2 < FLT_MIN;
  a.c2 = a.zero ? 1.0f : c2;
  a.flip = scale < 0.0f;
  a.window = window;
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  a.arrivals = static_cast<unsigned*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + arrival_bytes(B, n, heads_q, cache->heads));
  const int64_t rows = (int64_t)n * a.group;
  const int dt = dtype == SPEC_BF16 ? (int)kBF16 : (int)kF32, rt = tiles_for(cache->dim, dt, rows);
  a.groups = (int)((rows + 16 * rt - 1) / (16 * rt));
  (void)hipGetLastError();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // No more work-groups than units the call can have at most.
  const int64_t most = (int64_t)B * a.groups * cache->heads * (((int64_t)cache->table_len * cache->page + kUnitKeys - 1) / kUnitKeys + 1);
#define SV_LAUNCH(D, DT, RT)                                                                                       \
  if (cache->dim == D && dt == (int)DT && rt == RT) {                                                              \
    const int grid = (int)(most < grid_for(D, DT, RT) ? most : grid_for(D, DT, RT));                               \
    hipLaunchKernelGGL((attention_kernel<D, DT, RT>), dim3(grid), dim3(kThreads), 0, st, a);                       \
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;                                               \
  }
  SV_LAUNCH(64, kBF16, 1) SV_LAUNCH(64, kBF16, 2) SV_LAUNCH(64, kBF16, 3) SV_LAUNCH(64, kBF16, 4)
  SV_LAUNCH(128, kBF16, 1) SV_LAUNCH(128, kBF16, 2) SV_LAUNCH(128, kBF16, 3) SV_LAUNCH(128, kBF16, 4)
  SV_LAUNCH(256, kBF16, 1) SV_LAUNCH(256, kBF16, 2)
  SV_LAUNCH(64, kF32, 1) SV_LAUNCH(64, kF32, 2)
  SV_LAUNCH(128, kF32, 1) SV_LAUNCH(128, kF32, 2)
  SV_LAUNCH(256, kF32, 1)
#undef SV_LAUNCH
  return SPEC_EINVAL;
}
