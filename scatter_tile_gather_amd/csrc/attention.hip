// Attention of one new token per sequence over a paged key-value cache.
//
// Every cached key and value is read once, so HBM bounds the call; the design
// keeps all else off that path.
//  - A workgroup takes one cache head of one sequence over a part of its
//    tokens, for up to 16 of the query heads that share it.  Its four waves
//    walk over blocks of 32 tokens.
//  - Scores are computed transposed, S^T = K Q^T (v_mfma 16x16x32): a lane then
//    holds, for query l % 16, the scores of 8 of the 32 tokens -- just the
//    elements that the second product wants as its left operand P, so
//    probabilities never cross lanes.  The 8 tokens that lane group g = l / 16
//    holds are 4g .. 4g+3 and 16+4g .. 16+4g+3; the sum over tokens may take
//    them in any order as long as V is fed in the same one.
//  - K rows go from memory to the matrix unit as they are (a lane's 16 bytes
//    are its operand).  V is wanted with 8 tokens of one dimension in a lane
//    but lies with 8 dimensions of one token in 16 bytes: a lane loads 8 x 8
//    elements and transposes them with byte permutes in its own registers.
//    Nothing of K or V passes through LDS, and there is no barrier in the loop.
//  - One pass, with a running maximum that is raised only when a score exceeds
//    it by 2^8: until then p = 2^(s - m) <= 2^8 fits, and the usual iteration
//    needs no exchange between lanes and no rescaling.
//  - P is fed to the matrix unit as two 16-bit terms, the rounded value and the
//    rounded rest, so that its rounding (2^-9 of a term in bf16) does not add
//    to the output's; the product is far from being the bound.
#include <type_traits>

#include "stg_internal.h"

namespace stg {
namespace {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

constexpr int kWaves = 4;
constexpr int kThreads = 64 * kWaves;
constexpr int kBlock = 32;    // tokens of a wave's iteration
constexpr int kSpan = 1024;   // tokens whose addresses are in LDS at a time
constexpr float kRaise = 8.f; // log2 of how far a score may exceed the running maximum
constexpr int kQueries = 16;  // query heads of a workgroup

struct Args {
  const char* q;
  const char* k;
  const char* v;
  char* out;
  int64_t q_row, q_head, o_row, o_head;  // bytes
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // bytes
  const int32_t* table;
  int64_t table_stride;
  const int32_t* lens;
  const float* k_scale;
  const float* v_scale;
  float* lse;
  float* part;   // (rows, q_heads, splits, depth): sums relative to the part's maximum
  float2* stat;  // (rows, q_heads, splits): maximum (log2) and sum
  float scale_log2;
  int32_t rows, width, pages, slots;
  int32_t heads, group, tiles, depth, splits;
  int64_t window;
};

struct BF16 {
  typedef __bf16 x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t put(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
  static __device__ __forceinline__ float get(uint32_t b) { return __uint_as_float(b << 16); }
  // two e4m3 codes (the low or the high half of w); bf16 holds every code exactly
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.f, HIGH));
  }
};
struct F16 {
  typedef _Float16 x8 __attribute__((ext_vector_type(8)));
  static __device__ __forceinline__ f32x4 mma(u32x4 a, u32x4 b, f32x4 c) {
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(x8, a), __builtin_bit_cast(x8, b), c, 0, 0, 0);
  }
  static __device__ __forceinline__ uint32_t put(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
  static __device__ __forceinline__ float get(uint32_t b) { return (float)__builtin_bit_cast(_Float16, (uint16_t)b); }
  template <bool HIGH>
  static __device__ __forceinline__ uint32_t from_e4m3(uint32_t w) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.f, HIGH));
  }
};

// Eight elements moved down by n (0 .. 8) places of 16 bits, zeros above.
__device__ __forceinline__ u32x4 drop16(u32x4 v, int n) {
  uint64_t lo = v[0] | (uint64_t)v[1] << 32, hi = v[2] | (uint64_t)v[3] << 32;
  if (n >= 8) {
    lo = hi = 0;
  } else if (n >= 4) {
    lo = hi >> (16 * (n - 4));
    hi = 0;
  } else if (n > 0) {
    lo = lo >> (16 * n) | hi << (64 - 16 * n);
    hi >>= 16 * n;
  }
  return u32x4{(uint32_t)lo, (uint32_t)(lo >> 32), (uint32_t)hi, (uint32_t)(hi >> 32)};
}

// The tokens of row b that are attended, [begin, end), and this split's share.
struct Range {
  int32_t begin, end;
};
__host__ __device__ __forceinline__ int64_t split_tokens(int64_t n, int32_t splits) {
  return ((n + splits - 1) / splits + kBlock - 1) / kBlock * kBlock;
}
__device__ __forceinline__ Range attended(const Args& a, int32_t b) {
  const int64_t room = int64_t(a.width) * a.slots;
  const int64_t len = a.lens[b] < 0 ? 0 : a.lens[b] > room ? room : a.lens[b];
  const int64_t begin = a.window > 0 && len > a.window ? len - a.window : 0;
  return Range{(int32_t)begin, (int32_t)len};
}

// DS: depth in steps of 32 (rounded up); E4M3: the caches hold e4m3 codes.
template <class T, int DS, bool E4M3>
struct Geometry {
  static constexpr int kSteps = DS;
  // a lane's share of a value row, in dimensions: chunks of 8 over 128
  // dimensions, one chunk of 4 for a rest of 64
  static constexpr int kDims = DS <= 2 ? 4 : DS <= 4 ? 8 : DS <= 6 ? 12 : 16;
  static constexpr int kEights = kDims / 8;
  static constexpr int kFours = kDims % 8 / 4;
};

// 8 dimensions of a K or V row as 16-bit elements.
template <class T, bool E4M3>
struct Raw8 {
  using type = std::conditional_t<E4M3, u32x2, u32x4>;
  static __device__ __forceinline__ type load(const char* p) {
    type v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
  }
  static __device__ __forceinline__ u32x4 wide(type v) {
    if constexpr (E4M3)
      return u32x4{T::template from_e4m3<false>(v[0]), T::template from_e4m3<true>(v[0]),
                   T::template from_e4m3<false>(v[1]), T::template from_e4m3<true>(v[1])};
    else
      return v;
  }
};
template <class T, bool E4M3>
struct Raw4 {
  using type = std::conditional_t<E4M3, uint32_t, u32x2>;
  static __device__ __forceinline__ type load(const char* p) {
    type v;
    __builtin_memcpy(&v, p, sizeof(v));
    return v;
  }
  static __device__ __forceinline__ u32x2 wide(type v) {
    if constexpr (E4M3) return u32x2{T::template from_e4m3<false>(v), T::template from_e4m3<true>(v)};
    else return v;
  }
};

// Elements 2w and 2w+1 of eight rows -> the two operands that hold one
// dimension of the eight tokens each.
__device__ __forceinline__ void transpose_pair(const uint32_t (&r)[8], u32x4& even, u32x4& odd) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    even[i] = __builtin_amdgcn_perm(r[2 * i + 1], r[2 * i], 0x05040100u);
    odd[i] = __builtin_amdgcn_perm(r[2 * i + 1], r[2 * i], 0x07060302u);
  }
}

template <class T, int DS, bool E4M3>
__global__ __launch_bounds__(kThreads) void paged_attention_kernel(Args a) {
  using G = Geometry<T, DS, E4M3>;
  using R8 = Raw8<T, E4M3>;
  using R4 = Raw4<T, E4M3>;
  constexpr int kElem = E4M3 ? 1 : 2;
  // token addresses during the loop, the waves' sums after it
  __shared__ union {
    struct {
      int64_t k[kSpan], v[kSpan];
    } at;
    float sums[kWaves][kQueries][128];
  } lds;
  __shared__ float2 stats[kWaves][kQueries];

  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int col = lane & 15, grp = lane >> 4;
  uint32_t id = blockIdx.x;
  const int h = id % a.heads;
  id /= a.heads;
  const int tile = id % a.tiles;
  id /= a.tiles;
  const int split = id % a.splits;
  const int b = id / a.splits;

  const Range all = attended(a, b);
  const int64_t share = split_tokens(all.end - all.begin, a.splits);
  const int64_t begin = all.begin + split * share;
  const int64_t end = begin + share < all.end ? begin + share : all.end;
  if (begin >= end && split > 0) return;  // the join knows which parts exist

  // queries: operand column `col`, dimensions 8 grp + 32 step ..
  const int head0 = h * a.group + tile * kQueries;
  const int queries = a.group - tile * kQueries < kQueries ? a.group - tile * kQueries : kQueries;
  u32x4 qf[G::kSteps];
  {
    const char* q = a.q + b * a.q_row + (head0 + (col < queries ? col : 0)) * a.q_head;
#pragma unroll
    for (int s = 0; s < G::kSteps; ++s) {
      const int d = 8 * grp + 32 * s;
      const int from = d < a.depth - 8 ? d : a.depth - 8;
      u32x4 x;
      __builtin_memcpy(&x, q + 2 * from, 16);
      qf[s] = col < queries ? drop16(x, d - from < 8 ? d - from : 8) : u32x4{0, 0, 0, 0};
    }
  }
  const float c = a.scale_log2 * (a.k_scale ? a.k_scale[h] : 1.f);
  const char* kbase = a.k + h * a.k_head;
  const char* vbase = a.v + h * a.v_head;
  // where this lane's K chunks and V chunks begin; a chunk that would pass the
  // row's end is read further down, so every load stays inside the row
  int kd[G::kSteps];
#pragma unroll
  for (int s = 0; s < G::kSteps; ++s) {
    const int d = 8 * grp + 32 * s;
    kd[s] = d < a.depth - 8 ? d : a.depth - 8;
  }
  int vd8[G::kEights ? G::kEights : 1], vd4 = 0;
#pragma unroll
  for (int i = 0; i < G::kEights; ++i) {
    const int d = 128 * i + 8 * col;
    vd8[i] = d < a.depth - 8 ? d : a.depth - 8;
  }
  if constexpr (G::kFours > 0) {
    const int d = 128 * G::kEights + 4 * col;
    vd4 = d < a.depth - 4 ? d : a.depth - 4;
  }
  const bool ragged = a.depth != 32 * DS;

  f32x4 o[G::kDims];
#pragma unroll
  for (int e = 0; e < G::kDims; ++e) o[e] = f32x4{0.f, 0.f, 0.f, 0.f};
  float m = -INFINITY, sum = 0.f;

  for (int64_t s0 = begin; s0 < end; s0 += kSpan) {
    const int n = end - s0 < kSpan ? (int)(end - s0) : kSpan;
    const int blocks = (n + kBlock - 1) / kBlock;
    __syncthreads();
    for (int i = threadIdx.x; i < blocks * kBlock; i += kThreads) {
      int64_t ka = -1, va = -1;
      if (i < n) {
        const int32_t j = (int32_t)(s0 + i), entry = j / a.slots;
        const int32_t page = a.table[b * a.table_stride + entry];
        if ((uint32_t)page < (uint32_t)a.pages) {
          const int64_t slot = j - entry * a.slots;
          ka = page * a.k_page + slot * a.k_slot;
          va = page * a.v_page + slot * a.v_slot;
        }
      }
      lds.at.k[i] = ka;
      lds.at.v[i] = va;
    }
    __syncthreads();
    for (int blk = wave; blk < blocks; blk += kWaves) {
      const int i0 = blk * kBlock;
      // scores of tokens 16 t + 4 grp + r for query `col`
      f32x4 s[2];
#pragma unroll
      for (int t = 0; t < 2; ++t) {
        const int64_t at = lds.at.k[i0 + 16 * t + col];
        const char* row = kbase + (at < 0 ? 0 : at);
        u32x4 kf[G::kSteps];
#pragma unroll
        for (int st = 0; st < G::kSteps; ++st) kf[st] = R8::wide(R8::load(row + kd[st] * kElem));
        if (ragged) {
#pragma unroll
          for (int st = 0; st < G::kSteps; ++st) {
            const int over = 8 * grp + 32 * st - kd[st];
            kf[st] = drop16(kf[st], over < 8 ? over : 8);
          }
        }
        s[t] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int st = 0; st < G::kSteps; ++st) s[t] = T::mma(kf[st], qf[st], s[t]);
      }
      int64_t va[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) va[i] = lds.at.v[i0 + 16 * (i >> 2) + 4 * grp + (i & 3)];
      float x[8], top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        x[i] = va[i] < 0 ? -INFINITY : s[i >> 2][i & 3] * c;
        top = fmaxf(top, x[i]);
      }
      if (__ballot(top > m + kRaise)) {
        top = fmaxf(top, __shfl_xor(top, 16));
        top = fmaxf(top, __shfl_xor(top, 32));
        const float to = fmaxf(m, top);
        const float f = m == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(m - to);
        m = to;
        sum *= f;
        float fr[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) fr[r] = __shfl(f, 4 * grp + r);
#pragma unroll
        for (int e = 0; e < G::kDims; ++e)
#pragma unroll
          for (int r = 0; r < 4; ++r) o[e][r] *= fr[r];
      }
      const float base = m == -INFINITY ? 0.f : m;
      u32x4 hi, lo;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = __builtin_amdgcn_exp2f(x[2 * i] - base), p1 = __builtin_amdgcn_exp2f(x[2 * i + 1] - base);
        sum += p0 + p1;
        const uint32_t h0 = T::put(p0), h1 = T::put(p1);
        hi[i] = h0 | h1 << 16;
        lo[i] = T::put(p0 - T::get(h0)) | T::put(p1 - T::get(h1)) << 16;
      }
      bool holes = false;
#pragma unroll
      for (int i = 0; i < 8; ++i) holes |= va[i] < 0;
      const bool any_hole = __ballot(holes) != 0;
#pragma unroll
      for (int g8 = 0; g8 < G::kEights; ++g8) {
        u32x4 rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[i] = R8::wide(R8::load(vbase + (va[i] < 0 ? 0 : va[i]) + vd8[g8] * kElem));
        if (any_hole) {  // what lies in a hole may be NaN, and 0 * NaN is not 0
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (va[i] < 0) rows[i] = u32x4{0, 0, 0, 0};
        }
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          uint32_t r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = rows[i][w];
          u32x4 even, odd;
          transpose_pair(r, even, odd);
          f32x4& oe = o[8 * g8 + 2 * w];
          f32x4& oo = o[8 * g8 + 2 * w + 1];
          oe = T::mma(lo, even, T::mma(hi, even, oe));
          oo = T::mma(lo, odd, T::mma(hi, odd, oo));
        }
      }
      if constexpr (G::kFours > 0) {
        u32x2 rows[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) rows[i] = R4::wide(R4::load(vbase + (va[i] < 0 ? 0 : va[i]) + vd4 * kElem));
        if (any_hole) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            if (va[i] < 0) rows[i] = u32x2{0, 0};
        }
#pragma unroll
        for (int w = 0; w < 2; ++w) {
          uint32_t r[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) r[i] = rows[i][w];
          u32x4 even, odd;
          transpose_pair(r, even, odd);
          f32x4& oe = o[8 * G::kEights + 2 * w];
          f32x4& oo = o[8 * G::kEights + 2 * w + 1];
          oe = T::mma(lo, even, T::mma(hi, even, oe));
          oo = T::mma(lo, odd, T::mma(hi, odd, oo));
        }
      }
    }
  }

  // the four waves' parts, joined: thread (query, col) takes a chunk of the sums
  sum += __shfl_xor(sum, 16);
  sum += __shfl_xor(sum, 32);
  if (grp == 0) stats[wave][col] = make_float2(m, sum);
  const int jq = threadIdx.x >> 4;
  const int64_t head = int64_t(b) * a.heads * a.group + head0 + jq;  // (row, query head)
  float f[kWaves], top = -INFINITY, total = 0.f;
#pragma unroll
  for (int piece = 0; piece < G::kEights + G::kFours; ++piece) {
    const int n = piece < G::kEights ? 8 : 4;
    __syncthreads();  // the loop's addresses, or the last piece, are read
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (e < n)
#pragma unroll
        for (int r = 0; r < 4; ++r) lds.sums[wave][4 * grp + r][col * n + e] = o[8 * piece + e < G::kDims ? 8 * piece + e : 0][r];
    __syncthreads();
    if (piece == 0) {
#pragma unroll
      for (int w = 0; w < kWaves; ++w) top = fmaxf(top, stats[w][jq].x);
#pragma unroll
      for (int w = 0; w < kWaves; ++w) {
        f[w] = stats[w][jq].y == 0.f ? 0.f : __builtin_amdgcn_exp2f(stats[w][jq].x - top);
        total += f[w] * stats[w][jq].y;
      }
    }
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = 0.f;
      if (e < n)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) y[e] += f[w] * lds.sums[w][jq][col * n + e];
    }
    if (jq >= queries) continue;
    int d = 128 * piece + n * col;
    d = d < a.depth - n ? d : a.depth - n;
    if (a.splits == 1) {
      const float g = total == 0.f ? 0.f : (a.v_scale ? a.v_scale[h] : 1.f) / total;
      uint16_t z[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) z[e] = (uint16_t)T::put(total == 0.f ? 0.f : y[e] * g);
      char* dst = a.out + b * a.o_row + (head0 + jq) * a.o_head + 2 * d;
      if (n == 8) __builtin_memcpy(dst, z, 16);
      else __builtin_memcpy(dst, z, 8);
      if (piece == 0 && col == 0 && a.lse)
        a.lse[head] = total == 0.f ? -INFINITY : (top + __log2f(total)) * 0.69314718056f;
    } else {
      const int64_t p = head * a.splits + split;
      float* dst = a.part + p * a.depth + d;
      if (n == 8) __builtin_memcpy(dst, y, 32);
      else __builtin_memcpy(dst, y, 16);
      if (piece == 0 && col == 0) a.stat[p] = make_float2(top, total);
    }
  }
}

// One workgroup per row and query head: its parts, weighted by their maxima.
template <class T>
__global__ __launch_bounds__(64) void join_kernel(Args a) {
  const int hq = a.heads * a.group;
  const int b = blockIdx.x / hq, h = blockIdx.x - b * hq;
  const Range all = attended(a, b);
  const int64_t n = all.end - all.begin, share = split_tokens(n, a.splits);
  const int parts = n > 0 ? (int)((n + share - 1) / share) : 1;
  const float2* stat = a.stat + int64_t(blockIdx.x) * a.splits;
  const float* part = a.part + int64_t(blockIdx.x) * a.splits * a.depth;
  float top = -INFINITY;
  for (int i = 0; i < parts; ++i) top = fmaxf(top, stat[i].x);
  float total = 0.f, y[4] = {0.f, 0.f, 0.f, 0.f};
  for (int i = 0; i < parts; ++i) {
    const float f = stat[i].y == 0.f ? 0.f : __builtin_amdgcn_exp2f(stat[i].x - top);
    total += f * stat[i].y;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int d = threadIdx.x + 64 * e;
      if (d < a.depth) y[e] += f * part[int64_t(i) * a.depth + d];
    }
  }
  const float g = total == 0.f ? 0.f : (a.v_scale ? a.v_scale[h / a.group] : 1.f) / total;
  char* dst = a.out + b * a.o_row + h * a.o_head;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const int d = threadIdx.x + 64 * e;
    if (d < a.depth) ((uint16_t*)dst)[d] = (uint16_t)T::put(total == 0.f ? 0.f : y[e] * g);
  }
  if (threadIdx.x == 0 && a.lse) a.lse[blockIdx.x] = total == 0.f ? -INFINITY : (top + __log2f(total)) * 0.69314718056f;
}

// ---- host -------------------------------------------------------------------

constexpr int64_t kWantGroups = 4096;  // workgroups that fill the chip and balance long against short rows
constexpr int64_t kLeastShare = 256;   // tokens of a split, at least

int check_query(const char* what, const stg_tensor* t, const char* name) {
  if (int rc = check_tensor(t, name)) return rc;
  if (t->dtype != STG_BF16 && t->dtype != STG_F16)
    return fail(STG_ERR_UNSUPPORTED, "%s: %s must be bf16 or f16", what, name);
  if (t->rank != 3 || (t->shape[2] > 1 && t->stride[2] != 1))
    return fail(STG_ERR_INVALID, "%s: %s must be (rows, heads, depth) with unit depth stride", what, name);
  return STG_OK;
}

// Splits of a sequence, from the sizes that the host knows.
int64_t splits_for(int64_t groups, int64_t longest) {
  if (groups < 1 || longest < 1) return 1;
  int64_t n = (kWantGroups + groups - 1) / groups;
  const int64_t most = (longest + kLeastShare - 1) / kLeastShare;
  n = n < most ? n : most;
  return n < 1 ? 1 : n > 1024 ? 1024 : n;
}

int plan(const char* what, const stg_tensor* q, const stg_tensor* k_cache, const stg_tensor* page_table, int64_t window,
         int64_t max_len, int64_t* tiles, int64_t* splits, int64_t* bytes) {
  if (int rc = check_query(what, q, "q")) return rc;
  if (int rc = check_paged_cache(what, k_cache, k_cache, page_table)) return rc;
  const int64_t heads = k_cache->shape[2], depth = q->shape[2];
  if (k_cache->dtype != q->dtype && k_cache->dtype != STG_U8)
    return fail(STG_ERR_INVALID, "%s: caches must be of q's dtype or u8 (e4m3 codes)", what);
  if (k_cache->shape[3] != depth) return fail(STG_ERR_INVALID, "%s: q and the caches differ in depth", what);
  if (depth < 8 || depth > 256) return fail(STG_ERR_UNSUPPORTED, "%s: depth must be in [8, 256]", what);
  if (page_table->shape[0] != q->shape[0]) return fail(STG_ERR_INVALID, "%s: page_table needs a row per query", what);
  if (heads ? q->shape[1] % heads != 0 : q->shape[1] != 0)
    return fail(STG_ERR_INVALID, "%s: query heads must be a multiple of the cache's heads", what);
  if (q->shape[1] > 65536 || heads > 65536) return fail(STG_ERR_RANGE, "%s: more than 65536 heads", what);
  if (window < 0 || max_len < 0) return fail(STG_ERR_INVALID, "%s: negative window or max_len", what);
  const int64_t group = heads ? q->shape[1] / heads : 0;
  *tiles = (group + kQueries - 1) / kQueries;
  int64_t groups;
  if (__builtin_mul_overflow(q->shape[0], heads * *tiles, &groups) || groups > (int64_t(1) << 31) - 1)
    return fail(STG_ERR_RANGE, "%s: too many rows and heads", what);
  int64_t longest = page_table->shape[1] * k_cache->shape[1];  // each below 2^31
  if (max_len && max_len < longest) longest = max_len;
  if (window && window < longest) longest = window;
  *splits = splits_for(groups, longest);
  *bytes = 0;
  if (*splits > 1) {
    const int64_t parts = q->shape[0] * q->shape[1] * *splits;
    *bytes = parts * (8 + depth * 4);
  }
  return STG_OK;
}

template <class T, bool E4M3>
void launch_attention(const Args& a, uint32_t grid, hipStream_t st) {
  const auto go = [&](auto kernel) {
    launch_kernel("paged_attention", kernel, dim3(grid), dim3(kThreads), 0, st, a);
  };
  const int steps = (a.depth + 31) / 32;
  if (steps <= 2) go(paged_attention_kernel<T, 2, E4M3>);
  else if (steps == 3) go(paged_attention_kernel<T, 3, E4M3>);
  else if (steps == 4) go(paged_attention_kernel<T, 4, E4M3>);
  else if (steps <= 6) go(paged_attention_kernel<T, 6, E4M3>);
  else go(paged_attention_kernel<T, 8, E4M3>);
}

}  // namespace
}  // namespace stg

using namespace stg;

extern "C" int64_t paged_attention_workspace(const stg_tensor* q, const stg_tensor* k_cache,
                                             const stg_tensor* page_table, int64_t window, int64_t max_len) {
  clear_error();
  int64_t tiles, splits, bytes;
  if (int rc = plan("paged_attention_workspace", q, k_cache, page_table, window, max_len, &tiles, &splits, &bytes))
    return -rc;
  return bytes;
}

extern "C" int paged_attention(const stg_tensor* q, const stg_tensor* k_cache, const stg_tensor* v_cache,
                               const stg_tensor* page_table, const int32_t* seq_lens, const float* k_scale,
                               const float* v_scale, float scale, int64_t window, int64_t max_len,
                               const stg_tensor* out, float* lse, void* workspace, int64_t workspace_bytes,
                               void* stream) {
  clear_error();
  const char* what = "paged_attention";
  int64_t tiles, splits, bytes;
  if (int rc = plan(what, q, k_cache, page_table, window, max_len, &tiles, &splits, &bytes)) return rc;
  if (int rc = check_paged_cache(what, k_cache, v_cache, page_table)) return rc;
  if (int rc = check_query(what, out, "out")) return rc;
  if (out->dtype != q->dtype) return fail(STG_ERR_INVALID, "%s: out has another dtype than q", what);
  for (int d = 0; d < 3; ++d)
    if (out->shape[d] != q->shape[d]) return fail(STG_ERR_INVALID, "%s: out has another shape than q", what);
  if (k_cache->dtype != STG_U8 && (k_scale || v_scale))
    return fail(STG_ERR_INVALID, "%s: scales are for u8 (e4m3) caches", what);
  if (!q->shape[0] || !q->shape[1]) return STG_OK;
  if (!seq_lens) return fail(STG_ERR_INVALID, "%s: null seq_lens", what);
  if (bytes) {
    if (!workspace || workspace_bytes < bytes)
      return fail(STG_ERR_INVALID, "%s: needs a workspace of %lld bytes", what, (long long)bytes);
    if ((uintptr_t)workspace & 255) return fail(STG_ERR_INVALID, "%s: workspace must be 256-byte aligned", what);
  }
  Args a;
  const int64_t es = dtype_size(k_cache->dtype);
  a.q = (const char*)q->data;
  a.k = (const char*)k_cache->data;
  a.v = (const char*)v_cache->data;
  a.out = (char*)out->data;
  a.q_row = q->stride[0] * 2;
  a.q_head = q->stride[1] * 2;
  a.o_row = out->stride[0] * 2;
  a.o_head = out->stride[1] * 2;
  a.k_page = k_cache->stride[0] * es;
  a.k_slot = k_cache->stride[1] * es;
  a.k_head = k_cache->stride[2] * es;
  a.v_page = v_cache->stride[0] * es;
  a.v_slot = v_cache->stride[1] * es;
  a.v_head = v_cache->stride[2] * es;
  a.table = (const int32_t*)page_table->data;
  a.table_stride = page_table->stride[0];
  a.lens = seq_lens;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.lse = lse;
  a.scale_log2 = scale * 1.44269504089f;
  a.rows = (int32_t)q->shape[0];
  a.width = (int32_t)page_table->shape[1];
  a.pages = (int32_t)k_cache->shape[0];
  a.slots = (int32_t)k_cache->shape[1];
  if (!a.pages || !a.slots) {  // a cache without a slot holds no token, and nothing is read from it
    a.width = 0;
    a.slots = 1;
  }
  a.heads = (int32_t)k_cache->shape[2];
  a.group = (int32_t)(q->shape[1] / k_cache->shape[2]);
  a.tiles = (int32_t)tiles;
  a.depth = (int32_t)q->shape[2];
  a.splits = (int32_t)splits;
  a.window = window;
  const int64_t parts = q->shape[0] * q->shape[1] * splits;
  a.stat = (float2*)workspace;
  a.part = (float*)workspace + 2 * parts;
  int64_t grid;
  if (__builtin_mul_overflow(int64_t(a.rows) * a.heads * a.tiles, splits, &grid) || grid > (int64_t(1) << 31) - 1 ||
      q->shape[0] * q->shape[1] > (int64_t(1) << 31) - 1)
    return fail(STG_ERR_RANGE, "%s: too many rows and heads", what);
  const hipStream_t st = as_stream(stream);
  const bool e4m3 = k_cache->dtype == STG_U8;
  if (q->dtype == STG_BF16) {
    if (e4m3) launch_attention<BF16, true>(a, (uint32_t)grid, st);
    else launch_attention<BF16, false>(a, (uint32_t)grid, st);
  } else {
    if (e4m3) launch_attention<F16, true>(a, (uint32_t)grid, st);
    else launch_attention<F16, false>(a, (uint32_t)grid, st);
  }
  if (int rc = check_launch(what)) return rc;
  if (splits == 1) return STG_OK;
  const dim3 rows((uint32_t)(q->shape[0] * q->shape[1]));
  if (q->dtype == STG_BF16) launch_kernel("paged_attention/join", join_kernel<BF16>, rows, dim3(64), 0, st, a);
  else launch_kernel("paged_attention/join", join_kernel<F16>, rows, dim3(64), 0, st, a);
  return check_launch("paged_attention/join");
}
