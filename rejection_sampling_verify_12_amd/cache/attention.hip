// Attention of a round's new tokens over the 4-bit key/value cache
// (spec_verify.h describes the format, the visibility rule and the errors).
//
// The query rows of one sequence that share a key/value head (n tokens times
// heads_q / heads) are cut into groups of RT tiles of 16.  A work-group takes
// a group and a run of keys; each of its 4 waves takes blocks of 32 keys, 4
// blocks (a unit of 128 keys) at a time; only the queries are in shared memory:
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
//
// What bounds it.  Few rows (plain decoding): reading the cache.  64
// sequences of 2000 to 33000 positions, 8 heads of 128, 8 query rows each:
// 777 MB in 130 us, 6.0 TB/s in all and 6.9 TB/s in the loop, where a plain
// read reaches 7.2.  Many rows (verification, prompts): the vector
// instructions and the latency between dependent ones.  A block of 32 keys at
// dim 128 takes 112 of them to turn the codes into bfloat16 (a value's codes
// come in pairs along the vector and are needed in pairs along the keys: one
// v_perm per pair, as each token has its own scale), and about 45 and 17 matrix
// products of 16 cycles for each tile of 16 queries.  256 sequences of 300 to
// 6000 positions, 36 rows per head: 568 MB in 159 us, against 79 us at the
// read rate.  Measured and left: key codes straight into the scaled 4-bit
// by 8-bit matrix product (the queries as two 8-bit parts) saves 34
// instructions a block, but its sums keep only about 17 bits below the largest term.
#include "format.h"

#include <float.h>
#include <math.h>

#include <type_traits>

namespace sv {
namespace {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef unsigned u32x2 __attribute__((ext_vector_type(2)));

constexpr int kBlock = 32;               // keys per wave and step
constexpr int kUnitKeys = kWaves * kBlock;   // keys per work-group and step
// What an item weighs besides its units when the work is divided: queries in,
// waves joined and results out take about as long as these units.
constexpr int kItemUnits = 6;            // measured 3, 4, 6: 181, 174, 167 us for 256 sequences of 300 to 6000 positions
constexpr int kCUs = 256;                // MI355X
constexpr int kSpans = 512;              // sequences whose positions a work-group keeps in shared memory

struct AttentionArgs {
  CacheView c;
  const void* q;
  int64_t q_stride;
  int heads_q, group;   // query heads, query heads per key/value head
  unsigned by_group;    // ceil(2^32 / group): row / group = the upper half of row * by_group
  int groups;           // row groups per sequence and key/value head
  float c2;             // |scale| log2(e)
  int flip, zero;       // scale < 0; scale == 0 (or too small for a float): the queries are taken as 0
  int window;
  const uint64_t* mask;
  void* out;
  float* lse;
  struct Join* joins;   // [grid]
  float* parts;         // [2 * grid]: a part's numbers [rows][D], references [rows], sums to divide by [rows], sums for lse [rows]
};

// An item that several runs hold, written by the second of them (parts = 0 by
// every other run): run `run` - 1 has its first part, in its second place if `side` is set.
struct Join {
  int b, row0, h, used, parts, side;
};

template <int DT>
constexpr int kTerms = DT == kBF16 ? 1 : 3;   // bfloat16 parts that a query or a weight is cut into

// Waves per SIMD the registers of a variant leave room for (a fit to what the
// compiler needs).  Holding every variant to two or more pays although the
// largest two keep some of what surrounds the loop in scratch memory: prompt pieces of 2048
// tokens 95 us against 126 with one wave.
constexpr int waves_for(int D, int dt, int rt) {
  const int regs = rt * (D / 4 + 16) + D / 2 + 42;
  return regs <= 128 ? 4 : regs <= 168 ? 3 : 2;
}
// Row tiles of a group, at most: the codes are turned into numbers once for
// all of them.  (Three at dim 128 instead of four: 95 against 92 us for prompt
// pieces; one at dim 256 instead of two: 62 against 53 us for trees of 24 tokens.)
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

__device__ __forceinline__ int token_of(const AttentionArgs& a, int row) {
  return a.group == 1 ? row : (int)__umulhi((unsigned)row, a.by_group);
}

__device__ __forceinline__ Item item_of(const AttentionArgs& a, Span span, int rg, int rows) {
  Item it;
  it.s = span;
  const int used = it.s.count < 0 ? a.c.n : it.s.count;
  it.tok0 = token_of(a, rg * rows);
  it.tok1 = min(token_of(a, rg * rows + rows - 1), used - 1);
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

// A lane's share of a block of 32 keys: codes and scales of 2 tiles of 16
// keys.  Scales are loaded as the 4 bytes that hold the lane's and cut out
// where they are used: a load of 1 or 2 bytes is widened by an instruction
// that waits for it, right behind the load.
template <int D>
struct Half {   // of the keys, or of the values
  uint32_t w[2][D / 32];
  uint32_t sc[2];
};

// Cache policies: nontemporal where one row group has all of a sequence's
// queries, so that a key is read once (64 sequences of 2000 to 33000 positions:
// 173 us, 177 without); otherwise kept for the other groups (trees of 24 tokens at
// dim 256, four groups: 49 us, 56 nontemporal).
constexpr int kOnce = 2, kAgain = 0;
template <int D, int POLICY>
__device__ __forceinline__ void load_words(__amdgpu_buffer_rsrc_t rs, int voff, int soff, uint32_t (&w)[D / 32]) {
  if constexpr (D == 64) {
    const u32x2 t = __builtin_amdgcn_raw_buffer_load_b64(rs, voff, soff, POLICY);
    w[0] = t.x; w[1] = t.y;
  } else {
#pragma unroll
    for (int x = 0; x < D / 128; ++x) {
      const u32x4 t = __builtin_amdgcn_raw_buffer_load_b128(rs, voff + 16 * x, soff, POLICY);
      w[4 * x] = t.x; w[4 * x + 1] = t.y; w[4 * x + 2] = t.z; w[4 * x + 3] = t.w;
    }
  }
}

// Where a lane's share lies in a record; the block's own place is scalar.
template <int D>
struct Places {
  int k, v, ks, vs;
  int kbit;   // where the lane's key scales (8 bits, 16 at dim 256) start in their 32
  __device__ __forceinline__ Places(int P, int lane) {
    using F = Format<D>;
    const int i = lane & 15, g = lane >> 4;
    k = i * F::kRow + g * (D / 8);
    v = F::values(P, 0, 0) + g * (2 * D) + i * (D / 8);
    const int scale = i * F::kBlocks + (D == 256 ? 2 * g : D == 128 ? g : g >> 1);
    ks = F::key_scales(P, 0) + (scale & ~3);
    kbit = 8 * (scale & 3);
    vs = F::value_scale(P, 0, 0) + i * (D / 16) / 32 * 16 + 4 * g;
  }
};

// The record of one page and one head of it, or no bytes for a page outside the pool.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t record_rsrc(const uint8_t* head, int64_t page_bytes, int page, int bytes) {
  return chunk_rsrc(head + max(page, 0) * page_bytes, page < 0 ? 0 : bytes);
}
template <int D, int POLICY>
__device__ __forceinline__ void load_keys(__amdgpu_buffer_rsrc_t rs, int r, const Places<D>& at, Half<D>& x) {
  using F = Format<D>;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    load_words<D, POLICY>(rs, at.k + 16 * t * F::kRow, r * F::kRow, x.w[t]);
    x.sc[t] = __builtin_amdgcn_raw_buffer_load_b32(rs, at.ks + 16 * t * F::kBlocks, r * F::kBlocks, 0);
  }
}
template <int D, int POLICY>
__device__ __forceinline__ void load_values(__amdgpu_buffer_rsrc_t rs, int r, const Places<D>& at, Half<D>& x) {
  using F = Format<D>;
  // 16 tokens take as many bytes of values (scales) as of keys (scales).
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    load_words<D, POLICY>(rs, at.v + 16 * t * F::kRow, r * F::kRow, x.w[t]);
    x.sc[t] = __builtin_amdgcn_raw_buffer_load_b32(rs, at.vs + 16 * t * F::kBlocks, r * F::kBlocks, 0);
  }
}

// The upper bits of bytes from 192 on: scales of 2^65 and NaN blocks, told apart by find_nan_keys.
__device__ __forceinline__ uint32_t suspect(uint32_t w) { return w & (w << 1); }
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

// Powers of two that a weight may pass 1 by before the row's reference moves:
// float32 and bfloat16 lose nothing to it, and T keys of it are far from their largest numbers.
constexpr float kSlack = 16.0f;
constexpr float kNone = -FLT_MAX;

template <int D, int DT, int RT>
struct State {   // one wave's running result; a lane holds query (lane & 15) of each tile
  f32x4 o[RT][D / 16];
  float m[RT];   // reference (base 2; kNone before the first key)
  float l[RT];   // sum of the weights over the lane's own keys; bf16: only if lse is wanted
  // bf16: sum of the rounded weights over all keys, by a product with ones.
  // Dividing by it rather than by l cancels the part of the roundings that
  // the weights have in common (all of it where one weight carries the row).
  f32x4 r[DT == kBF16 ? RT : 1];
};

template <int RT>
struct Rows {   // the group's queries
  const u32x4* q;   // in shared memory: [D / 32][RT][terms][64 lanes]
  int token[RT];
};

// Scores of a block: rows = keys, columns = queries.  rt's tile t holds keys
// 16 t + 4 (lane / 16) + 0 .. 3 of query lane % 16.
template <int D, int DT, int RT>
__device__ __forceinline__ void score_block(const Half<D>& x, const uint32_t (&ks)[2], const Rows<RT>& rows, int lane, f32x4 (&s)[RT][2]) {
  constexpr int T = kTerms<DT>;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) s[rt][0] = s[rt][1] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < D / 32; ++c) {
    bf16x8 k[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const float sc = scale_of(D == 256 ? (c < 4 ? ks[t] & 255 : ks[t] >> 8) : ks[t]);
      const uint32_t w = x.w[t][c];
      k[t] = as_bf16x8(cvt_pair(w, sc, 0), cvt_pair(w, sc, 1), cvt_pair(w, sc, 2), cvt_pair(w, sc, 3));
    }
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
#pragma unroll
      for (int e = T - 1; e >= 0; --e) {
        const bf16x8 q = __builtin_bit_cast(bf16x8, rows.q[((c * RT + rt) * T + e) * 64 + lane]);
#pragma unroll
        for (int t = 0; t < 2; ++t) s[rt][t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k[t], q, s[rt][t], 0, 0, 0);
      }
    }
  }
}

// Keys of the block with a NaN block, bit 16 t + key of tile t (rare).  The
// row's weight will say NaN; the value itself must not reach other rows, so
// its scale is replaced.
template <int D>
__device__ __forceinline__ uint32_t find_nan_keys(uint32_t k0, uint32_t k1, uint32_t (&v)[2]) {
  uint32_t found = 0;
#pragma unroll
  for (int t = 0; t < 2; ++t) {
    uint64_t k = __ballot(has_ff(t ? k1 : k0) != 0);
    k |= k >> 32;
    uint32_t keys = (uint32_t)(k | k >> 16) & 0xFFFFu;
#pragma unroll
    for (int jj = 0; jj < 4; ++jj) {
      const bool bad = (v[t] >> (8 * jj) & 255) == 255;
      const uint64_t m = __ballot(bad);
#pragma unroll
      for (int gg = 0; gg < 4; ++gg) keys |= (m >> (16 * gg) & 0xFFFF) ? 1u << (4 * gg + jj) : 0u;
      if (bad) v[t] = (v[t] & ~(255u << (8 * jj))) | 127u << (8 * jj);
    }
    found |= keys << (16 * t);
  }
  return found;
}

// Bit k: the row whose token is at position `at` sees key p + k.
__device__ __forceinline__ uint32_t seen_keys(const AttentionArgs& a, const Item& it, int b, int at, int p) {
  const auto below = [](int n) { return n >= 32 ? ~0u : n <= 0 ? 0u : (1u << n) - 1; };   // bits 0 .. n - 1
  const int token = at - it.s.pos;
  if (token >= it.s.count) return 0;
  uint32_t sees = below(at + 1 - p);
  if (a.mask) {
    const int first = it.s.pos - p;   // of the new tokens, in the block
    uint64_t bits = a.mask[(int64_t)b * a.c.n + token];
    bits &= it.s.count >= 64 ? ~0ull : (1ull << it.s.count) - 1;
    sees = below(first) | (uint32_t)(first >= 32 || first <= -64 ? 0 : first >= 0 ? bits << first : bits >> -first);
  }
  return a.window > 0 ? sees & ~below(at - a.window + 1 - p) : sees;
}

// Weights of a block and the running maximum and sum.  `masked`: some row does not see some key.
template <int D, int DT, int RT>
__device__ __forceinline__ void weigh_block(const AttentionArgs& a, const Item& it, int b, int p, int lane, bool masked,
                                            uint32_t nan_keys, float c2, bool lse, const Rows<RT>& rows, f32x4 (&s)[RT][2],
                                            State<D, DT, RT>& st, bf16x8 (&w)[RT][kTerms<DT>]) {
  const int g = lane >> 4;
#pragma unroll
  for (int rt = 0; rt < RT; ++rt) {
    float x[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = s[rt][e >> 2][e & 3];
    if (masked || nan_keys) {
      int at = it.s.pos + rows.token[rt], g4 = 4 * g;
      asm volatile("" : "+v"(at), "+v"(g4));   // computed here, not kept over the loop
      const uint32_t sees = seen_keys(a, it, b, at, p);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int in = 16 * (e >> 2) + (e & 3);
        if (nan_keys) x[e] = nan_keys >> (in + g4) & 1 ? __uint_as_float(0x7FC00000u) : x[e];
        x[e] = sees >> (in + g4) & 1 ? x[e] : -INFINITY;
      }
    }
    // The reference m only has to keep 2^(x - m) in range, so it moves when a
    // score passes it by more than kSlack: most blocks need neither the
    // exchange between lanes nor the rescaling.  (A NaN moves nothing: its own
    // weight says NaN.)
    const auto max2 = [](float u, float v) { return __builtin_elementwise_maximum(u, v); };
    float top = max2(max2(max2(x[0], x[1]), x[2]), max2(max2(x[3], x[4]), max2(max2(x[5], x[6]), x[7])));
    if (__any(top * c2 > st.m[rt] + kSlack)) {
      const auto maxf = [](float u, float v) { return fmaxf(u, v); };
      top = swap_combine<32>(swap_combine<16>(top, maxf), maxf) * c2;
      const float m = fmaxf(st.m[rt], top), alpha = exp2_fast(st.m[rt] - m);
      st.l[rt] *= alpha;
      if constexpr (DT == kBF16) st.r[rt] *= alpha;
#pragma unroll
      for (int d = 0; d < D / 16; ++d) st.o[rt][d] *= alpha;
      st.m[rt] = m;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = exp2_fast(fmaf(x[e], c2, -st.m[rt]));
    if (DT == kF32 || lse) st.l[rt] += ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
    split8<kTerms<DT>>(x, w[rt]);
  }
}

// O^T += V^T P^T.  Numbers 2 d and 2 d + 1 of the lane's D / 16, for its 8 keys; token jj's codes are bytes
// jj * D/32 on of the lane's share.
template <int D, int DT, int RT>
__device__ __forceinline__ void gather_block(const Half<D>& x, const bf16x8 (&w)[RT][kTerms<DT>], State<D, DT, RT>& st) {
  constexpr int T = kTerms<DT>;
  if constexpr (DT == kBF16) {
    const bf16x8 ones = as_bf16x8(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) st.r[rt] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ones, w[rt][0], st.r[rt], 0, 0, 0);
  }
  float sc[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sc[e] = scale_of(__builtin_amdgcn_ubfe(x.sc[e >> 2], 8 * (e & 3), 8));
#pragma unroll
  for (int d = 0; d < D / 32; ++d) {
    uint32_t y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int byte = (e & 3) * (D / 32) + d;
      y[e] = cvt_pair(x.w[e >> 2][byte / 4], sc[e], byte % 4);
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

// N numbers of a row of the output.
template <int D, int DT, int N>
__device__ __forceinline__ void store_numbers(void* out, int64_t at, const float (&v)[N]) {
  if constexpr (DT == kBF16) {
    uint32_t w[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) w[e] = pack_bf16(v[2 * e], v[2 * e + 1]);
    uint32_t* p = reinterpret_cast<uint32_t*>(static_cast<uint16_t*>(out) + at);
    if constexpr (N == 4) {
      *reinterpret_cast<u32x2*>(p) = u32x2{w[0], w[1]};
    } else {
#pragma unroll
      for (int e = 0; e < N / 8; ++e) reinterpret_cast<u32x4*>(p)[e] = u32x4{w[4 * e], w[4 * e + 1], w[4 * e + 2], w[4 * e + 3]};
    }
  } else {
    f32x4* p = reinterpret_cast<f32x4*>(static_cast<float*>(out) + at);
#pragma unroll
    for (int e = 0; e < N / 4; ++e) p[e] = f32x4{v[4 * e], v[4 * e + 1], v[4 * e + 2], v[4 * e + 3]};
  }
}

// Units in W equal runs (the first U % W have one more): the first unit of
// run w, and the run of unit u.
struct Runs {
  int q, rem;
  __device__ __forceinline__ Runs(int U, int W) : q(U / W), rem(U - U / W * W) {}
  __device__ __forceinline__ int start(int w) const { return w * q + min(w, rem); }
  __device__ __forceinline__ int of(int u) const {
    const int wide = rem * (q + 1);
    return u < wide ? u / (q + 1) : rem + (u - wide) / q;
  }
};

// Inclusive prefix sum over the wave (every lane active).
__device__ __forceinline__ int inclusive_scan(int v) {
  int s = v + dpp<kDppRowShr + 1, 0xF, 0xF, true>(v, 0);
  s += dpp<kDppRowShr + 2, 0xF, 0xF, true>(v, 0);
  s += dpp<kDppRowShr + 3, 0xF, 0xF, true>(v, 0);   // rows: sums of 4
  s += dpp<kDppRowShr + 4, 0xF, 0xE>(s, 0);         // lanes 4..15 of a row
  s += dpp<kDppRowShr + 8, 0xF, 0xC>(s, 0);         // lanes 8..15
  s += dpp<kDppRowBcast15, 0xA>(s, 0);              // rows 1, 3
  s += dpp<kDppRowBcast31, 0xC>(s, 0);              // rows 2, 3
  return s;
}

// A scalar that the loop keeps, rather than loading it from the arguments for each block.
template <class V>
__device__ __forceinline__ V pin(V x) {
  asm volatile("" : "+s"(x));
  return x;
}

// Work-groups take equal runs of units, ordered by sequence, row group,
// key/value head and key.  An item (all keys of one group and head) that lies
// in one run is written at once; otherwise each run's part goes to the
// workspace, for join_kernel.  A run has at most two such parts, its first
// and its last.
template <int D, int DT, int RT, int POLICY>
__global__ __launch_bounds__(kThreads, waves_for(D, DT, RT)) void attention_kernel(AttentionArgs) {
  const AttentionArgs& a = kernel_arg0<AttentionArgs>();
  constexpr int R = 16 * RT, S = D / 16, kPart = R * (D + 3), T = kTerms<DT>;
  constexpr int kSums = kWaves * 16 * (D + 4) * 4, kQ = R * D * 2 * T;
  __shared__ __align__(16) char space[kSums > kQ ? kSums : kQ];   // the queries, then the waves' results
  __shared__ float tops[kWaves][R], totals[kWaves][R], exacts[kWaves][R];   // references, sums to divide by, sums for lse
  __shared__ Span spans[kSpans];
  float (&sums)[kWaves][16][D + 4] = *reinterpret_cast<float (*)[kWaves][16][D + 4]>(space);
  const int tid = threadIdx.x, lane = tid & 63, wave = uni(tid >> 6);
  const int i = lane & 15, g = lane >> 4;
  const int heads = a.c.heads, entries = a.c.B * a.groups;

  // Every wave finds its run by itself (each writes the same positions and
  // reads its own), so the work-group starts without a barrier.
  {
    int len[kSpans / 64], count[kSpans / 64];   // all loads before the first use
#pragma unroll
    for (int q = 0; q < kSpans / 64; ++q) {
      const int b = min(lane + 64 * q, a.c.B - 1);
      if (64 * q >= a.c.B) break;
      len[q] = a.c.len ? a.c.len[b] : 0;
      count[q] = a.c.count ? a.c.count[b] : a.c.n;
    }
#pragma unroll
    for (int q = 0; q < kSpans / 64; ++q) {
      if (64 * q >= a.c.B) break;
      if (lane + 64 * q < a.c.B) spans[lane + 64 * q] = span_from(a.c, (int64_t)len[q] - a.c.lag, count[q]);
    }
  }
  const auto span_at = [&](int b) { return b < kSpans ? spans[b] : span_of(a.c, b); };
  const auto units_at = [&](int entry) {
    const int b = entry / a.groups;
    return item_of(a, span_at(b), entry - b * a.groups, R).units;
  };
  // Units of one head before this lane's entries, and in all (the host keeps
  // them within 31 bits).  Where there is a work-group for every unit, items
  // weigh their units alone.
  const int per = (entries + 63) / 64;
  const int e0 = min(lane * per, entries), e1 = min(e0 + per, entries);
  int units = 0, items = 0;
  for (int e = e0; e < e1; ++e) {
    const int x = units_at(e);
    units += x;
    items += x > 0;
  }
  const int units_through = inclusive_scan(units), items_through = inclusive_scan(items);
  const int extra = __builtin_amdgcn_readlane(units_through, 63) * heads <= (int)gridDim.x ? 0 : kItemUnits;
  const int mine = units + extra * items, through = units_through + extra * items_through, before = through - mine;
  const int U = __builtin_amdgcn_readlane(through, 63) * heads, W = min(U, (int)gridDim.x), run = blockIdx.x;
  if (tid == 0) a.joins[run].parts = 0;
  if (run >= W) return;   // the whole work-group
  const Runs runs(U, W);
  int u = runs.start(run);
  const int u1 = runs.start(run + 1), u_begin = u;
  int found = 0, start = before * heads;
  const bool here = start <= u && u < through * heads;
  if (here) {
    for (int e = e0; e < e1; ++e) {
      const int x = units_at(e), weight = (x + (x > 0 ? extra : 0)) * heads;
      found = e;
      if (u < start + weight) break;
      start += weight;
    }
  }
  const int at = __ffsll((unsigned long long)__ballot(here)) - 1;   // one lane's entries hold the run's start
  int entry = __builtin_amdgcn_readlane(found, at), entry_start = __builtin_amdgcn_readlane(start, at);
  const Places<D> places(1 << a.c.page_log2, lane);

  while (u < u1 && entry < entries) {
    const int b = entry / a.groups, rg = entry - b * a.groups;
    const Span span = span_at(b);
    const Item it = item_of(a, {uni(span.pos), uni(span.count)}, rg, R);
    const int weight = it.units > 0 ? it.units + extra : 0;
    if (u >= entry_start + weight * heads) {
      entry_start += weight * heads;
      ++entry;
      continue;
    }
    const int h = (u - entry_start) / weight;
    const int u0 = entry_start + h * weight;   // the item's first unit; its last `extra` have no keys
    const int k0 = u - u0, k1 = min(u1 - u0, weight);
    const int row0 = rg * R;
    // Rows in use; all n tokens' after a range error.
    const int used = min(R, (it.s.count < 0 ? a.c.n : it.s.count) * a.group - row0);
    const auto place_of = [&](int r) {   // row r of the group in q and out, in rows of D
      const int row = row0 + r, token = token_of(a, row);
      return ((int64_t)b * a.c.n + token) * a.heads_q + h * a.group + (row - token * a.group);
    };

    if (it.s.count < 0) {
      float nan[S];
#pragma unroll
      for (int d = 0; d < S; ++d) nan[d] = __uint_as_float(0x7FC00000u);
      for (int r = tid >> 4; r < used && k0 == 0; r += 16) {
        const int64_t at = place_of(r);
        store_numbers<D, DT, S>(a.out, at * D + (tid & 15) * S, nan);
        if (a.lse && (tid & 15) == 0) a.lse[at] = nan[0];
      }
      u = u0 + k1;
      continue;
    }

    // The wave's blocks p = lo + 128 k + 32 wave below hi.  The next block is
    // loaded when this one's keys have been used, its page number a block
    // earlier; the first one, before the queries.
    const int32_t* table = a.c.table + (int64_t)b * a.c.table_len;
    const int log2 = pin(a.c.page_log2), P = 1 << log2, record = Format<D>::record(P), pages = pin(a.c.pages);
    const uint8_t* head = pin(a.c.data + (int64_t)h * record);
    const int64_t page_bytes = (int64_t)heads * record;
    const float c2 = pin(a.c2);
    const bool lse = a.lse != nullptr;
    const int p1 = min(it.hi, it.lo + kUnitKeys * k1);
    int p = it.lo + kUnitKeys * k0 + kBlock * wave;
    // Blocks from whole0 to whole1 are seen by every row as a whole.
    const int whole0 = a.window > 0 ? it.s.pos + it.tok1 - a.window + 1 : 0;
    const int whole1 = (a.mask ? it.s.pos - 1 : it.s.pos + it.tok0) - (kBlock - 1);
    const auto page_at = [&](int pos) {   // positions behind the run read the run's last page
      const int page = scalar_at(table, min(pos, p1 - 1) >> log2);
      return (page >= 0 && page < pages) ? page : -1;
    };
    Half<D> k, v[2];
    int page = -1, next = -1;
    __amdgpu_buffer_rsrc_t rec;
    if (p < p1) {
      page = page_at(p);
      next = page_at(p + kUnitKeys);
      rec = record_rsrc(head, page_bytes, page, record);
      load_keys<D, POLICY>(rec, p & (P - 1), places, k);
      load_values<D, POLICY>(rec, p & (P - 1), places, v[0]);
    }

    Rows<RT> rows;
    State<D, DT, RT> st;
    rows.q = reinterpret_cast<const u32x4*>(space);
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const int row = row0 + rt * 16 + i, token = token_of(a, row), head = h * a.group + (row - token * a.group);
      rows.token[rt] = token;
      const bool live = token < it.s.count && !a.zero;
      const int64_t at = ((int64_t)b * a.c.n + token) * a.q_stride + (int64_t)head * D + g * (D / 4);
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        if ((rt * (D / 32) + c) % kWaves != wave) continue;   // the waves share the work
        float x[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
        if (live) load_row8<DT>(a.q, at + 8 * c, x);
        if (a.flip) {
#pragma unroll
          for (int e = 0; e < 8; ++e) x[e] = -x[e];
        }
        bf16x8 q[T];
        split8<T>(x, q);
#pragma unroll
        for (int e = 0; e < T; ++e)
          reinterpret_cast<u32x4*>(space)[((c * RT + rt) * T + e) * 64 + lane] = __builtin_bit_cast(u32x4, q[e]);
      }
      st.m[rt] = kNone;
      st.l[rt] = 0.0f;
      if constexpr (DT == kBF16) st.r[rt] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int d = 0; d < S; ++d) st.o[rt][d] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
    __syncthreads();

    if (p < p1) {
      // One block, values in v0; the next one's go to v1.  False after the last.
      const auto step = [&](Half<D>& v0, Half<D>& v1) __attribute__((always_inline)) {
        const int pn = p + kUnitKeys;
        const bool more = pn < p1;
        f32x4 s[RT][2];
        bf16x8 w[RT][T];
        uint32_t ks[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) ks[t] = __builtin_amdgcn_ubfe(k.sc[t], places.kbit, D == 256 ? 16 : 8);
        if (page < 0) {
          ks[0] = ks[1] = D == 256 ? 0xFFFFu : 0xFFu;
          v0.sc[0] = v0.sc[1] = 0xFFFFFFFFu;
        }
        const bool masked = p < whole0 || p > whole1;
        score_block<D, DT, RT>(k, ks, rows, lane, s);
        __builtin_amdgcn_sched_barrier(0);
        // A wave that feeds the matrix cores goes before one that works on its
        // weights: 256 sequences of 300 to 6000 positions 165 -> 159 us.
        __builtin_amdgcn_s_setprio(0);
        rec = record_rsrc(head, page_bytes, more ? next : -1, record);
        load_keys<D, POLICY>(rec, pn & (P - 1), places, k);
        load_values<D, POLICY>(rec, pn & (P - 1), places, v1);
        page = next;
        next = page_at(pn + kUnitKeys);
        uint32_t nan_keys = 0;
        const uint32_t both = ks[0] | ks[1] << (D == 256 ? 16 : 8);
        if (__any((int)((suspect(both) | suspect(v0.sc[0]) | suspect(v0.sc[1])) & 0x80808080u)))
          nan_keys = find_nan_keys<D>(ks[0], ks[1], v0.sc);
        if (masked) {
          // Places behind the last token hold anything: no scale of theirs may give an infinity.
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            uint32_t& x = v0.sc[e >> 2];
            if ((x >> (8 * (e & 3)) & 255) > 252) x = (x & ~(255u << (8 * (e & 3)))) | 127u << (8 * (e & 3));
          }
        }
        weigh_block<D, DT, RT>(a, it, b, p, lane, masked, nan_keys, c2, lse, rows, s, st, w);
        __builtin_amdgcn_sched_barrier(0);
        __builtin_amdgcn_s_setprio(1);
        gather_block<D, DT, RT>(v0, w, st);
        __builtin_amdgcn_sched_barrier(0);
        p = pn;
        return more;
      };
      while (step(v[0], v[1]) && step(v[1], v[0])) {
      }
      __builtin_amdgcn_s_setprio(0);
    }

    // Join the waves.
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      const auto add2 = [](float x, float y) { return x + y; };
      st.l[rt] = swap_combine<32>(swap_combine<16>(st.l[rt], add2), add2);
      if (g == 0) {
        tops[wave][rt * 16 + i] = st.m[rt];
        totals[wave][rt * 16 + i] = DT == kBF16 ? st.r[rt][0] : st.l[rt];
        exacts[wave][rt * 16 + i] = st.l[rt];
      }
    }
    __syncthreads();
    const bool whole = k0 == 0 && k1 == weight;
    float* part = a.parts + (int64_t)(2 * run + (u == u_begin ? 0 : 1)) * kPart;
#pragma unroll
    for (int rt = 0; rt < RT; ++rt) {
      if (rt > 0) __syncthreads();   // sums is read by the tile before
      {
        float m = tops[0][rt * 16 + i];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][rt * 16 + i]);
        const float f = exp2_fast(st.m[rt] - m);
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int d = 0; d < S; ++d) sums[wave][i][(4 * g + r) * S + d] = st.o[rt][d][r] * f;
      }
      __syncthreads();
      const int row16 = tid >> 4, share = tid & 15, r = rt * 16 + row16;
      if (r < used) {
        float m = tops[0][r], l = 0.0f, exact = 0.0f, v[S];
#pragma unroll
        for (int w = 1; w < kWaves; ++w) m = fmaxf(m, tops[w][r]);
#pragma unroll
        for (int w = 0; w < kWaves; ++w) {
          const float f = exp2_fast(tops[w][r] - m);
          l += totals[w][r] * f;
          exact += exacts[w][r] * f;
        }
#pragma unroll
        for (int d = 0; d < S; ++d)
          v[d] = (sums[0][row16][share * S + d] + sums[1][row16][share * S + d]) + (sums[2][row16][share * S + d] + sums[3][row16][share * S + d]);
        if (whole) {
          const int64_t at = place_of(r);
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
#pragma unroll
          for (int d = 0; d < S; ++d) v[d] *= inv;
          store_numbers<D, DT, S>(a.out, at * D + share * S, v);
          if (a.lse && share == 0) a.lse[at] = exact == 0.0f ? -INFINITY : (m + log2f(exact)) * 0.6931471805599453f;
        } else {
#pragma unroll
          for (int d = 0; d < S; d += 4) *reinterpret_cast<f32x4*>(part + r * D + share * S + d) = f32x4{v[d], v[d + 1], v[d + 2], v[d + 3]};
          if (share == 0) {
            part[R * D + r] = m;
            part[R * D + R + r] = l;
            part[R * D + 2 * R + r] = exact;
          }
        }
      }
    }
    if (tid == 0 && k0 > 0) {
      const int first = runs.of(u0), last = runs.of(u0 + weight - 1);   // the runs with a part
      if (first == run - 1) a.joins[run] = {b, row0, h, used, last - first + 1, runs.start(first) < u0 ? 1 : 0};
    }
    __syncthreads();
    u = u0 + k1;
  }
}

// Joins the parts of the items that several runs hold, in order.  A wave takes
// kRows rows, a lane 4 numbers of every (256 / D)-th part; where an item has
// many parts the waves of a work-group share them, and the work-group takes
// kRows rows.  A kernel of its own spreads the rows over the chip: with the
// last work-group to arrive joining its item alone, 5 tokens over 200000
// positions took 72 us and now take 51.
template <int D, int DT, int RT>
__global__ __launch_bounds__(kThreads) void join_kernel(AttentionArgs) {
  const AttentionArgs& a = kernel_arg0<AttentionArgs>();
  constexpr int R = 16 * RT, kPart = R * (D + 3), kLanes = D / 4, kSplit = 64 / kLanes, kAhead = 4, kRows = 4;
  static_assert(kRows == kWaves, "a wave joins one row of a shared item");
  __shared__ f32x4 numbers[kWaves][kRows][kLanes];
  __shared__ float sums[kWaves][kRows][3];
  const int* at = reinterpret_cast<const int*>(a.joins + blockIdx.x);
  const Join j = {scalar_at(at, 0), scalar_at(at, 1), scalar_at(at, 2), scalar_at(at, 3), scalar_at(at, 4), scalar_at(at, 5)};
  const bool shared = j.parts > 4 * kSplit;
  const int lane = threadIdx.x & 63, wave = uni((int)(threadIdx.x >> 6)), rows = shared ? kRows : kRows * kWaves;
  if (j.parts == 0 || (int)blockIdx.y * rows >= j.used) return;   // the whole work-group
  const int r0 = (int)blockIdx.y * rows + (shared ? 0 : wave * kRows), first = (int)blockIdx.x - 1;
  const int mine = lane / kLanes + (shared ? wave * kSplit : 0), step = shared ? kWaves * kSplit : kSplit, d = lane % kLanes * 4;
  struct Sum {
    float m, l, exact;
    f32x4 v;
    __device__ __forceinline__ void add(float pm, float pl, float pe, f32x4 pv) {
      const float top = fmaxf(m, pm), f0 = exp2_fast(m - top), f1 = exp2_fast(pm - top);
      m = top;
      l = l * f0 + pl * f1;
      exact = exact * f0 + pe * f1;
      v = v * f0 + pv * f1;
    }
  };
  Sum sum[kRows];
#pragma unroll
  for (int n = 0; n < kRows; ++n) sum[n] = {kNone, 0.0f, 0.0f, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
  for (int x = mine; x < j.parts; x += step * kAhead) {
    float pm[kAhead][kRows], pl[kAhead][kRows], pe[kAhead][kRows];
    f32x4 pv[kAhead][kRows];
#pragma unroll
    for (int y = 0; y < kAhead; ++y) {
      const int z = x + y * step;
      const float* p = a.parts + (int64_t)(2 * (first + z) + (z == 0 ? j.side : 0)) * kPart;
#pragma unroll
      for (int n = 0; n < kRows; ++n) {
        const int r = r0 + n;
        pm[y][n] = kNone;
        pl[y][n] = pe[y][n] = 0.0f;
        pv[y][n] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
        if (z < j.parts && r < j.used) {
          pm[y][n] = p[R * D + r];
          pl[y][n] = p[R * D + R + r];
          pe[y][n] = p[R * D + 2 * R + r];
          pv[y][n] = *reinterpret_cast<const f32x4*>(p + r * D + d);
        }
      }
    }
#pragma unroll
    for (int y = 0; y < kAhead; ++y)
#pragma unroll
      for (int n = 0; n < kRows; ++n) sum[n].add(pm[y][n], pl[y][n], pe[y][n], pv[y][n]);
  }
  const auto join2 = [](Sum& s, auto swap) {   // with the lane that has the row's other parts
    const auto max2 = [](float x, float y) { return fmaxf(x, y); };
    const auto add2 = [](float x, float y) { return x + y; };
    constexpr int kSwap = decltype(swap)::value;
    const float top = swap_combine<kSwap>(s.m, max2), f = exp2_fast(s.m - top);
    s.m = top;
    s.l = swap_combine<kSwap>(s.l * f, add2);
    s.exact = swap_combine<kSwap>(s.exact * f, add2);
#pragma unroll
    for (int e = 0; e < 4; ++e) s.v[e] = swap_combine<kSwap>(s.v[e] * f, add2);
  };
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    if constexpr (kSplit == 4) join2(sum[n], std::integral_constant<int, 16>{});
    if constexpr (kSplit >= 2) join2(sum[n], std::integral_constant<int, 32>{});
  }
  const auto write = [&](int r, const Sum& s) {
    const int row = j.row0 + r, token = token_of(a, row);
    const int64_t to = ((int64_t)j.b * a.c.n + token) * a.heads_q + j.h * a.group + (row - token * a.group);
    const float inv = s.l == 0.0f ? 0.0f : 1.0f / s.l;
    const float o[4] = {s.v[0] * inv, s.v[1] * inv, s.v[2] * inv, s.v[3] * inv};
    store_numbers<D, DT, 4>(a.out, to * D + d, o);
    if (a.lse && d == 0) a.lse[to] = s.exact == 0.0f ? -INFINITY : (s.m + log2f(s.exact)) * 0.6931471805599453f;
  };
  if (!shared) {
#pragma unroll
    for (int n = 0; n < kRows; ++n)
      if (lane < kLanes && r0 + n < j.used) write(r0 + n, sum[n]);
    return;
  }
#pragma unroll
  for (int n = 0; n < kRows; ++n) {
    if (lane < kLanes) numbers[wave][n][lane] = sum[n].v;
    if (lane == 0) {
      sums[wave][n][0] = sum[n].m;
      sums[wave][n][1] = sum[n].l;
      sums[wave][n][2] = sum[n].exact;
    }
  }
  __syncthreads();
  if (lane < kLanes && r0 + wave < j.used) {
    Sum s = {kNone, 0.0f, 0.0f, f32x4{0.0f, 0.0f, 0.0f, 0.0f}};
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s.add(sums[w][wave][0], sums[w][wave][1], sums[w][wave][2], numbers[w][wave][lane]);
    write(r0 + wave, s);
  }
}

int check_attention(int B, int n, int heads_q, int heads, int dim) {
  if (B < 0 || n < 1 || heads < 1 || heads_q < heads || heads_q % heads || !dim_ok(dim)) return SPEC_EINVAL;
  if ((int64_t)B * n > ((int64_t)1 << 24)) return SPEC_EINVAL;
  if (B > 0 && heads_q > (((int64_t)1 << 34) / dim) / ((int64_t)B * n)) return SPEC_EINVAL;
  const int64_t groups = ((int64_t)n * (heads_q / heads) + 15) / 16;
  if (B > 0 && groups * heads > ((int64_t)1 << 24) / B) return SPEC_EINVAL;
  // row / group by a multiplication needs rows * group < 2^32 (with room for a last group's rows)
  if (((int64_t)n * (heads_q / heads) + 64) * (heads_q / heads) >= ((int64_t)1 << 32)) return SPEC_EINVAL;
  return SPEC_OK;
}

constexpr int grid_for(int D, int dt, int rt) { return kCUs * waves_for(D, dt, rt); }

constexpr size_t kJoinBytes = (size_t)kCUs * 4 * sizeof(Join);   // at most 4 waves per SIMD

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
      const size_t need = (size_t)2 * grid_for(dim, dt, rt) * 16 * rt * (dim + 3) * sizeof(float);
      parts = need > parts ? need : parts;
    }
  }
  return (kJoinBytes + parts + 255) / 256 * 256;
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
  if (!isfinite(c2)) return SPEC_EINVAL;
  a.zero = c2 < FLT_MIN;
  a.c2 = a.zero ? 1.0f : c2;
  a.flip = scale < 0.0f;
  a.window = window < 1 << 30 ? window : 0;   // positions are below 2^30
  a.mask = mask;
  a.out = out;
  a.lse = lse;
  a.joins = static_cast<Join*>(workspace);
  a.parts = reinterpret_cast<float*>(static_cast<char*>(workspace) + kJoinBytes);
  const int64_t rows = (int64_t)n * a.group;
  a.by_group = (unsigned)((((uint64_t)1 << 32) + a.group - 1) / a.group);
  const int dt = dtype == SPEC_BF16 ? (int)kBF16 : (int)kF32, rt = tiles_for(cache->dim, dt, rows);
  a.groups = (int)((rows + 16 * rt - 1) / (16 * rt));
  (void)hipGetLastError();
  const hipStream_t st = static_cast<hipStream_t>(stream);
  // No more work-groups than units the call can have at most.
  const int64_t most = (int64_t)B * a.groups * cache->heads * (((int64_t)cache->table_len * cache->page + kUnitKeys - 1) / kUnitKeys + 1 + kItemUnits);
  if (most > INT_MAX) return SPEC_EINVAL;
  const unsigned row_chunks = (unsigned)((rows < 16 * rt ? rows : 16 * rt) + kWaves - 1) / kWaves;
  const int policy = a.groups == 1 ? kOnce : kAgain;
#define SV_LAUNCH(D, DT, RT, POLICY)                                                                               \
  if (cache->dim == D && dt == (int)DT && rt == RT && policy == POLICY) {                                          \
    const int grid = (int)(most < grid_for(D, DT, RT) ? most : grid_for(D, DT, RT));                               \
    hipLaunchKernelGGL((attention_kernel<D, DT, RT, POLICY>), dim3(grid), dim3(kThreads), 0, st, a);               \
    hipLaunchKernelGGL((join_kernel<D, DT, RT>), dim3(grid, row_chunks), dim3(kThreads), 0, st, a);                \
    return hipGetLastError() == hipSuccess ? SPEC_OK : SPEC_ELAUNCH;                                               \
  }
  SV_LAUNCH(64, kBF16, 1, kOnce) SV_LAUNCH(64, kBF16, 2, kOnce) SV_LAUNCH(64, kBF16, 3, kOnce) SV_LAUNCH(64, kBF16, 4, kOnce)
  SV_LAUNCH(128, kBF16, 1, kOnce) SV_LAUNCH(128, kBF16, 2, kOnce) SV_LAUNCH(128, kBF16, 3, kOnce) SV_LAUNCH(128, kBF16, 4, kOnce)
  SV_LAUNCH(256, kBF16, 1, kOnce) SV_LAUNCH(256, kBF16, 2, kOnce)
  SV_LAUNCH(64, kF32, 1, kOnce) SV_LAUNCH(64, kF32, 2, kOnce)
  SV_LAUNCH(128, kF32, 1, kOnce) SV_LAUNCH(128, kF32, 2, kOnce)
  SV_LAUNCH(256, kF32, 1, kOnce)
  // Several groups have as many tiles as the rows spread over them: more than half of the most.
  SV_LAUNCH(64, kBF16, 3, kAgain) SV_LAUNCH(64, kBF16, 4, kAgain)
  SV_LAUNCH(128, kBF16, 3, kAgain) SV_LAUNCH(128, kBF16, 4, kAgain)
  SV_LAUNCH(256, kBF16, 2, kAgain)
  SV_LAUNCH(64, kF32, 2, kAgain) SV_LAUNCH(128, kF32, 2, kAgain) SV_LAUNCH(256, kF32, 1, kAgain)
#undef SV_LAUNCH
  return SPEC_EINVAL;
}
