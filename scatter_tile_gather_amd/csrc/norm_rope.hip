// Norms of query and key heads with the rotation by position in the same pass:
// forward, forward into the pages of a cache, and backward.
//
// A head's x (depth D) becomes y = x w / sqrt(mean(x^2) + eps), and the pair
// (y_a, y_b) of frequency f turns by the angle t = position f.  Every element
// is read once and written once, so HBM bounds large calls and launch latency
// small ones; all else is kept to what fits beside the memory traffic:
//  - a head is held by L lanes, L the power of two that covers ceil(D / 16):
//    two chunks of 8 elements a lane, loaded as 16 bytes each (bf16, f16).
//    The sum of squares is then a reduction over L lanes.
//  - in the half layout a lane holds chunks i and i + R/16, so both elements
//    of its pairs are its own; interleaved pairs lie inside a chunk.  Only a
//    half layout whose R / 2 is not a multiple of 8 exchanges elements, through
//    LDS.
//  - cosine and sine depend on the token and the pair alone: the wave that
//    owns a token computes them once, into LDS, for all heads.
#include <math.h>

#include <cmath>
#include <type_traits>

#include "stg_internal.h"

namespace stg {
namespace {

constexpr int kWaves = 4;  // waves per workgroup; each works alone until the end
constexpr int kThreads = 64 * kWaves;

enum Mode { kHalfInLane = 0, kInterleaved = 1, kHalfExchange = 2 };
enum CacheKind { kNoCache = 0, kSameCache = 1, kE4m3Cache = 2 };

struct Rows {  // (tokens, heads, depth), strides in elements
  char* data;
  int64_t token, head;
};

struct Turn {
  const float* inv_freq;
  const void* wq;
  const void* wk;
  int32_t weight_f32;  // weights are fp32, else of the tensors' type
  int32_t norm;
  float gain, eps;
  int32_t rotary;  // R
};

struct Shape {
  int64_t tokens;
  int32_t q_heads, k_heads, depth;
  int32_t lanes;        // L
  int32_t wave_tokens;  // tokens whose heads a wave takes at a time
};

struct Cache {
  char* k;
  char* v;
  int64_t k_page, k_slot, k_head, v_page, v_slot, v_head;  // elements
  const int32_t* table;
  int64_t table_stride;
  int32_t rows, width, pages;
  int32_t slots;
  const int32_t* token_rows;
  const float* k_scale;
  const float* v_scale;
};

// Orders a wave's LDS accesses against each other: the LDS unit runs one
// wave's instructions in order, so only the compiler has to be held.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_wave_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

struct BF16 {
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float get(uint32_t bits) { return __uint_as_float(bits << 16); }
  static __device__ __forceinline__ uint32_t put(float x) {
    return __builtin_bit_cast(uint16_t, (__bf16)x);
  }
};
struct F16 {
  static constexpr int kBytes = 2;
  static __device__ __forceinline__ float get(uint32_t bits) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)bits);
  }
  static __device__ __forceinline__ uint32_t put(float x) { return __builtin_bit_cast(uint16_t, (_Float16)x); }
};
struct F32 {
  static constexpr int kBytes = 4;
};

template <class T>
__device__ __forceinline__ float load_one(const char* p) {
  if constexpr (T::kBytes == 4) return *(const float*)p;
  else return T::get(*(const uint16_t*)p);
}
template <class T>
__device__ __forceinline__ void store_one(char* p, float x) {
  if constexpr (T::kBytes == 4) *(float*)p = x;
  else *(uint16_t*)p = (uint16_t)T::put(x);
}

// n (<= 8, may be <= 0) elements at p; the others are 0.
template <class T>
__device__ __forceinline__ void load_chunk(const char* p, int n, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = 0.f;
  if (n >= 8) {
    if constexpr (T::kBytes == 4) {
      const u32x4 a = ld16(p), b = ld16(p + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[i] = __uint_as_float(a[i]);
        x[4 + i] = __uint_as_float(b[i]);
      }
    } else {
      const u32x4 a = ld16(p);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        x[2 * i] = T::get(a[i] & 0xFFFFu);
        x[2 * i + 1] = T::get(a[i] >> 16);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) x[i] = load_one<T>(p + i * T::kBytes);
  }
}

template <class T>
__device__ __forceinline__ void store_chunk(char* p, int n, const float (&x)[8]) {
  if (n >= 8) {
    if constexpr (T::kBytes == 4) {
      u32x4 a, b;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        a[i] = __float_as_uint(x[i]);
        b[i] = __float_as_uint(x[4 + i]);
      }
      st16(p, a);
      st16(p + 16, b);
    } else {
      u32x4 a;
#pragma unroll
      for (int i = 0; i < 4; ++i) a[i] = T::put(x[2 * i]) | T::put(x[2 * i + 1]) << 16;
      st16(p, a);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) store_one<T>(p + i * T::kBytes, x[i]);
  }
}

// x / scale rounded to the nearest e4m3 code, ties to even, saturated at 448;
// NaN passes the comparisons and stays NaN.
__device__ __forceinline__ void store_e4m3(char* p, int n, const float (&x)[8], float scale) {
  float y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float v = x[i] / scale;
    y[i] = v > 448.f ? 448.f : v < -448.f ? -448.f : v;
  }
  int w[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i], y[4 * i + 1], 0, false);
    w[i] = __builtin_amdgcn_cvt_pk_fp8_f32(y[4 * i + 2], y[4 * i + 3], w[i], true);
  }
  if (n >= 8) {
    __builtin_memcpy(p, w, 8);
  } else {
#pragma unroll
    for (int i = 0; i < 7; ++i)
      if (i < n) p[i] = (char)(w[i >> 2] >> (8 * (i & 3)));
  }
}

// Sum over the L lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lanes) {
  for (int d = 1; d < lanes; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

// The two chunks of 8 elements that lane `sub` of a head holds.
struct Chunks {
  int a, b;    // first elements
  int na, nb;  // elements of the chunk inside the head (<= 0: none)
};
template <int MODE>
__device__ __forceinline__ Chunks chunks_of(int sub, int depth, int rotary) {
  Chunks c;
  const int count = (depth + 7) >> 3;
  int a = sub, b = sub + ((count + 1) >> 1);
  if (sub >= (count + 1) >> 1) a = b = count;  // more lanes than pairs of chunks
  if constexpr (MODE == kHalfInLane) {
    const int h = rotary >> 4;
    a = sub < h ? sub : 2 * sub;  // past the turning chunks, two neighbours: 2h + 2 (sub - h)
    b = sub < h ? sub + h : 2 * sub + 1;
  }
  c.a = a * 8;
  c.b = b * 8;
  c.na = depth - c.a;
  c.nb = depth - c.b;
  return c;
}

// cos and sin (times gain) of a token's angles -> cs[0 .. R/2).  position *
// inv_freq is exact in fp64 up to 2^29 positions and is reduced to one turn
// there, so fp32 sees an angle of at most pi whatever the position.
__device__ __forceinline__ void angles_of(const Turn& t, int32_t position, float2* cs) {
  const double kInvTurn = 0.15915494309189533577, kTurnHi = 6.28318530717958623200, kTurnLo = 2.44929359829470641e-16;
  for (int i = threadIdx.x & 63; i < t.rotary >> 1; i += 64) {
    const double a = (double)position * (double)t.inv_freq[i];
    const double n = rint(a * kInvTurn);
    const float r = (float)fma(-n, kTurnLo, fma(-n, kTurnHi, a));
    float s, c;
    sincosf(r, &s, &c);
    cs[i] = make_float2(c * t.gain, s * t.gain);
  }
}

// Turns a lane's chunks in place; sign -1 turns back.  `swap` is this wave's
// LDS for exchanged elements, indexed by head group.
template <int MODE>
__device__ __forceinline__ void turn(float (&a)[8], float (&b)[8], const Chunks& c, const float2* cs, int rotary,
                                     float sign, float* swap) {
  if constexpr (MODE == kHalfInLane) {
    if (c.a < rotary >> 1) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float2 z = cs[c.a + i];
        const float s = sign * z.y, x = a[i], y = b[i];
        a[i] = x * z.x - y * s;
        b[i] = y * z.x + x * s;
      }
    }
  } else if constexpr (MODE == kInterleaved) {
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      if (c.a + i < rotary) {
        const float2 z = cs[(c.a + i) >> 1];
        const float s = sign * z.y, x = a[i], y = a[i + 1];
        a[i] = x * z.x - y * s;
        a[i + 1] = y * z.x + x * s;
      }
      if (c.b + i < rotary) {
        const float2 z = cs[(c.b + i) >> 1];
        const float s = sign * z.y, x = b[i], y = b[i + 1];
        b[i] = x * z.x - y * s;
        b[i + 1] = y * z.x + x * s;
      }
    }
  } else {
    const int h = rotary >> 1;
    wave_sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (c.a + i < rotary) swap[c.a + i] = a[i];
      if (c.b + i < rotary) swap[c.b + i] = b[i];
    }
    wave_sync();
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int da = c.a + i, db = c.b + i;
      if (da < rotary) {
        const float2 z = cs[da < h ? da : da - h];
        const float s = sign * z.y;
        a[i] = da < h ? a[i] * z.x - swap[da + h] * s : a[i] * z.x + swap[da - h] * s;
      }
      if (db < rotary) {
        const float2 z = cs[db < h ? db : db - h];
        const float s = sign * z.y;
        b[i] = db < h ? b[i] * z.x - swap[db + h] * s : b[i] * z.x + swap[db - h] * s;
      }
    }
  }
}

template <class T>
__device__ __forceinline__ void load_weight(const void* w, int f32, int at, int n, float (&x)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  } else if (f32) {
    load_chunk<F32>((const char*)w + at * 4, n, x);
  } else {
    load_chunk<T>((const char*)w + int64_t(at) * T::kBytes, n, x);
  }
}

// LDS of one wave, in floats: cos and sin of its tokens, then the exchange.
__host__ __device__ inline int wave_floats(int rotary, int wave_tokens, int mode) {
  return wave_tokens * rotary + (mode == kHalfExchange ? 1024 : 0);
}

// A wave takes wave_tokens tokens and blockIdx.y's share of their heads; each
// group of L lanes one head at a time: query heads, then key heads, then (into
// a cache) value heads.
template <class T, int MODE, int CACHE>
__global__ __launch_bounds__(kThreads) void forward_kernel(Rows q, Rows k, Rows v, const int32_t* positions, Turn t,
                                                           Shape sh, Rows q_out, Rows k_out, Cache cache) {
  extern __shared__ float lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float2* cs = (float2*)(lds + wave * wave_floats(t.rotary, sh.wave_tokens, MODE));
  const int64_t first = (int64_t(blockIdx.x) * kWaves + wave) * sh.wave_tokens;
  if (first >= sh.tokens) return;
  const int tokens = sh.tokens - first < sh.wave_tokens ? (int)(sh.tokens - first) : sh.wave_tokens;
  const int L = sh.lanes, sub = lane & (L - 1), group = lane / L, groups = 64 / L;
  float* swap = (float*)cs + sh.wave_tokens * t.rotary + group * L * 16;
  const Chunks c = chunks_of<MODE>(sub, sh.depth, t.rotary);
  float wqa[8], wqb[8], wka[8], wkb[8];
  load_weight<T>(t.wq, t.weight_f32, c.a, c.na, wqa);
  load_weight<T>(t.wq, t.weight_f32, c.b, c.nb, wqb);
  load_weight<T>(t.wk, t.weight_f32, c.a, c.na, wka);
  load_weight<T>(t.wk, t.weight_f32, c.b, c.nb, wkb);
  for (int i = 0; i < tokens; ++i) angles_of(t, positions[first + i], cs + i * (t.rotary >> 1));
  wave_sync();
  const int heads = sh.q_heads + sh.k_heads * (CACHE == kNoCache ? 1 : 2);
  for (int item = blockIdx.y * groups + group; item - group < tokens * heads; item += groups * gridDim.y) {
    const bool live = item < tokens * heads;
    const int i = live ? item / heads : 0;
    int h = live ? item - i * heads : 0;
    const int64_t tok = first + i;
    const int role = h < sh.q_heads ? 0 : h < sh.q_heads + sh.k_heads ? 1 : 2;
    h -= role == 0 ? 0 : role == 1 ? sh.q_heads : sh.q_heads + sh.k_heads;
    const Rows& in = role == 0 ? q : role == 1 ? k : v;
    const char* src = in.data + (tok * in.token + h * in.head) * T::kBytes;
    float a[8], b[8];
    load_chunk<T>(src + int64_t(c.a) * T::kBytes, live ? c.na : 0, a);
    load_chunk<T>(src + int64_t(c.b) * T::kBytes, live ? c.nb : 0, b);
    float va[8], vb[8];  // a value's elements pass as they are
    if constexpr (CACHE != kNoCache) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        va[e] = a[e];
        vb[e] = b[e];
      }
    }
    if (t.norm) {
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
      const float r = 1.f / sqrtf(head_sum(ss, L) / (float)sh.depth + t.eps);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        a[e] *= r * (role == 0 ? wqa[e] : wka[e]);
        b[e] *= r * (role == 0 ? wqb[e] : wkb[e]);
      }
    }
    turn<MODE>(a, b, c, cs + i * (t.rotary >> 1), t.rotary, 1.f, swap);
    if (!live) continue;
    if (CACHE == kNoCache || role == 0) {
      const Rows& o = role == 0 ? q_out : k_out;
      char* dst = o.data + (tok * o.token + h * o.head) * T::kBytes;
      store_chunk<T>(dst + int64_t(c.a) * T::kBytes, c.na, a);
      store_chunk<T>(dst + int64_t(c.b) * T::kBytes, c.nb, b);
      continue;
    }
    if constexpr (CACHE != kNoCache) {
      const int64_t row = cache.token_rows ? cache.token_rows[tok] : tok;
      const int32_t pos = positions[tok];
      if (row < 0 || row >= cache.rows || pos < 0) continue;
      const int32_t entry = pos / cache.slots;
      if (entry >= cache.width) continue;
      const int32_t page = cache.table[row * cache.table_stride + entry];
      if ((uint32_t)page >= (uint32_t)cache.pages) continue;
      const int64_t slot = pos - entry * cache.slots;
      if (role == 2) {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          a[e] = va[e];
          b[e] = vb[e];
        }
      }
      const int64_t at = role == 1 ? page * cache.k_page + slot * cache.k_slot + h * cache.k_head
                                   : page * cache.v_page + slot * cache.v_slot + h * cache.v_head;
      char* base = role == 1 ? cache.k : cache.v;
      if constexpr (CACHE == kSameCache) {
        store_chunk<T>(base + (at + c.a) * T::kBytes, c.na, a);
        store_chunk<T>(base + (at + c.b) * T::kBytes, c.nb, b);
      } else {
        const float* scales = role == 1 ? cache.k_scale : cache.v_scale;
        const float scale = scales ? scales[h] : 1.f;
        store_e4m3(base + at + c.a, c.na, a, scale);
        store_e4m3(base + at + c.b, c.nb, b, scale);
      }
    }
  }
}

// ---- backward ---------------------------------------------------------------

struct Gradient {  // queries or keys
  Rows dy, x, dx;
  const void* w;
  int32_t heads;
  int32_t groups;   // workgroups on it
  float* partial;   // (groups, depth) or null
};

// Workgroups 0 .. dq.groups-1 take queries, the others keys; a workgroup's
// waves walk over its tokens, summing u x' for the weight in registers.
template <class T, int MODE>
__global__ __launch_bounds__(kThreads) void backward_kernel(Gradient dq, Gradient dk, const int32_t* positions, Turn t,
                                                            Shape sh) {
  extern __shared__ float lds[];
  const bool keys = (int)blockIdx.x >= dq.groups;
  const Gradient g = keys ? dk : dq;
  const int group_id = keys ? blockIdx.x - dq.groups : blockIdx.x;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  float2* cs = (float2*)(lds + wave * wave_floats(t.rotary, sh.wave_tokens, MODE));
  const int L = sh.lanes, sub = lane & (L - 1), group = lane / L, groups = 64 / L;
  float* swap = (float*)cs + sh.wave_tokens * t.rotary + group * L * 16;
  const Chunks c = chunks_of<MODE>(sub, sh.depth, t.rotary);
  float wa[8], wb[8], sa[8], sb[8];
  load_weight<T>(g.w, t.weight_f32, c.a, c.na, wa);
  load_weight<T>(g.w, t.weight_f32, c.b, c.nb, wb);
#pragma unroll
  for (int e = 0; e < 8; ++e) sa[e] = sb[e] = 0.f;
  const float inv_depth = 1.f / (float)sh.depth;
  for (int64_t first = (int64_t(group_id) * kWaves + wave) * sh.wave_tokens; first < sh.tokens;
       first += int64_t(g.groups) * kWaves * sh.wave_tokens) {
    const int tokens = sh.tokens - first < sh.wave_tokens ? (int)(sh.tokens - first) : sh.wave_tokens;
    wave_sync();
    for (int i = 0; i < tokens; ++i) angles_of(t, positions[first + i], cs + i * (t.rotary >> 1));
    wave_sync();
    for (int item = group; item - group < tokens * g.heads; item += groups) {
      const bool live = item < tokens * g.heads;
      const int i = live ? item / g.heads : 0;
      const int h = live ? item - i * g.heads : 0;
      const int64_t tok = first + i;
      const char* dy = g.dy.data + (tok * g.dy.token + h * g.dy.head) * T::kBytes;
      float ua[8], ub[8];
      load_chunk<T>(dy + int64_t(c.a) * T::kBytes, live ? c.na : 0, ua);
      load_chunk<T>(dy + int64_t(c.b) * T::kBytes, live ? c.nb : 0, ub);
      float xa[8], xb[8];
      if (t.norm) {
        const char* x = g.x.data + (tok * g.x.token + h * g.x.head) * T::kBytes;
        load_chunk<T>(x + int64_t(c.a) * T::kBytes, live ? c.na : 0, xa);
        load_chunk<T>(x + int64_t(c.b) * T::kBytes, live ? c.nb : 0, xb);
      }
      turn<MODE>(ua, ub, c, cs + i * (t.rotary >> 1), t.rotary, -1.f, swap);
      if (t.norm) {
        // with r = 1 / sqrt(mean(x^2) + eps): dx = r u w - x r^3 mean(u w x)
        float ss = 0.f, sd = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss += xa[e] * xa[e] + xb[e] * xb[e];
          sd += ua[e] * wa[e] * xa[e] + ub[e] * wb[e] * xb[e];
        }
        ss = head_sum(ss, L);
        sd = head_sum(sd, L);
        const float r = 1.f / sqrtf(ss * inv_depth + t.eps);
        const float back = r * sd * inv_depth;  // mean(u w x')
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xa[e] *= r;
          xb[e] *= r;
          if (live) {
            sa[e] += ua[e] * xa[e];
            sb[e] += ub[e] * xb[e];
          }
          ua[e] = r * (ua[e] * wa[e] - xa[e] * back);
          ub[e] = r * (ub[e] * wb[e] - xb[e] * back);
        }
      }
      if (live) {
        char* dx = g.dx.data + (tok * g.dx.token + h * g.dx.head) * T::kBytes;
        store_chunk<T>(dx + int64_t(c.a) * T::kBytes, c.na, ua);
        store_chunk<T>(dx + int64_t(c.b) * T::kBytes, c.nb, ub);
      }
    }
  }
  if (!g.partial) return;  // the same for all waves of the workgroup
  for (int d = L; d < 64; d <<= 1) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      sa[e] += __shfl_xor(sa[e], d);
      sb[e] += __shfl_xor(sb[e], d);
    }
  }
  __syncthreads();  // LDS is free of angles
  if (group == 0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      if (e < c.na) lds[wave * sh.depth + c.a + e] = sa[e];
      if (e < c.nb) lds[wave * sh.depth + c.b + e] = sb[e];
    }
  }
  __syncthreads();
  for (int d = threadIdx.x; d < sh.depth; d += kThreads) {
    float s = 0.f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) s += lds[w * sh.depth + d];
    g.partial[int64_t(group_id) * sh.depth + d] = s;
  }
}

// dw[d] = sum of the workgroups' partial sums; 64 columns a workgroup, 16 rows
// at a time.  blockIdx.y: queries, keys.
template <class T>
__global__ __launch_bounds__(1024) void weight_kernel(const float* pq, int nq, void* dwq, const float* pk, int nk,
                                                      void* dwk, int depth, int f32) {
  __shared__ float sums[16][64];
  const float* p = blockIdx.y ? pk : pq;
  const int n = blockIdx.y ? nk : nq;
  void* dw = blockIdx.y ? dwk : dwq;
  if (!dw) return;
  const int col = threadIdx.x & 63, row = threadIdx.x >> 6, d = blockIdx.x * 64 + col;
  float s = 0.f;
  if (d < depth)
    for (int i = row; i < n; i += 16) s += p[int64_t(i) * depth + d];
  sums[row][col] = s;
  __syncthreads();
  if (row == 0 && d < depth) {
    float all = 0.f;
#pragma unroll
    for (int i = 0; i < 16; ++i) all += sums[i][col];
    if (f32) ((float*)dw)[d] = all;
    else store_one<T>((char*)dw + int64_t(d) * T::kBytes, all);
  }
}

// ---- host -------------------------------------------------------------------


int check_rows(const char* what, const stg_tensor* t, const char* name) {
  if (int rc = check_tensor(t, name)) return rc;
  if (t->dtype != STG_BF16 && t->dtype != STG_F16 && t->dtype != STG_F32)
    return fail(STG_ERR_UNSUPPORTED, "%s: %s must be bf16, f16 or f32", what, name);
  if (t->rank != 3 || (t->shape[2] > 1 && t->stride[2] != 1))
    return fail(STG_ERR_INVALID, "%s: %s must be (tokens, heads, depth) with unit depth stride", what, name);
  return STG_OK;
}

int check_like(const char* what, const stg_tensor* t, const char* name, const stg_tensor* like) {
  if (int rc = check_rows(what, t, name)) return rc;
  if (t->dtype != like->dtype) return fail(STG_ERR_INVALID, "%s: %s has another dtype", what, name);
  for (int d = 0; d < 3; ++d)
    if (t->shape[d] != like->shape[d]) return fail(STG_ERR_INVALID, "%s: %s has another shape", what, name);
  return STG_OK;
}

Rows rows_of(const stg_tensor* t) { return Rows{(char*)t->data, t->stride[0], t->stride[1]}; }

// Checks q, k and how; fills the kernel's shape and mode.
int check_call(const char* what, const stg_tensor* q, const stg_tensor* k, const int32_t* positions,
               const stg_norm_rope* how, Shape* sh, Turn* t, int* mode) {
  if (int rc = check_rows(what, q, "q")) return rc;
  if (int rc = check_rows(what, k, "k")) return rc;
  if (q->dtype != k->dtype) return fail(STG_ERR_INVALID, "%s: q and k have different dtypes", what);
  if (q->shape[0] != k->shape[0] || q->shape[2] != k->shape[2])
    return fail(STG_ERR_INVALID, "%s: q and k differ in tokens or depth", what);
  if (!how) return fail(STG_ERR_INVALID, "%s: null stg_norm_rope", what);
  const int64_t depth = q->shape[2];
  if (depth < 1 || depth > 1024) return fail(STG_ERR_UNSUPPORTED, "%s: depth must be in [1, 1024]", what);
  if (q->shape[1] > 65536 || k->shape[1] > 65536) return fail(STG_ERR_RANGE, "%s: more than 65536 heads", what);
  if (how->rotary_dim < 0 || how->rotary_dim > depth || how->rotary_dim % 2)
    return fail(STG_ERR_INVALID, "%s: rotary_dim must be even, 0 .. depth", what);
  if (how->rotary_dim && !how->inv_freq) return fail(STG_ERR_INVALID, "%s: null inv_freq", what);
  if (!how->norm && (how->q_weight || how->k_weight)) return fail(STG_ERR_INVALID, "%s: weights without norm", what);
  if ((how->q_weight || how->k_weight) && how->weight_dtype != STG_F32 && how->weight_dtype != q->dtype)
    return fail(STG_ERR_UNSUPPORTED, "%s: weights must be f32 or of q's dtype", what);
  if (how->norm && !(how->eps >= 0.f)) return fail(STG_ERR_INVALID, "%s: eps must be >= 0", what);
  if (q->shape[0] && how->rotary_dim && !positions) return fail(STG_ERR_INVALID, "%s: null positions", what);
  t->inv_freq = how->inv_freq;
  t->wq = how->q_weight;
  t->wk = how->k_weight;
  t->weight_f32 = how->weight_dtype == STG_F32;
  t->norm = how->norm != 0;
  t->gain = how->rope_scale;
  t->eps = how->eps;
  t->rotary = how->rotary_dim;
  sh->tokens = q->shape[0];
  sh->q_heads = (int32_t)q->shape[1];
  sh->k_heads = (int32_t)k->shape[1];
  sh->depth = (int32_t)depth;
  int lanes = 1;
  while (lanes * 16 < depth) lanes *= 2;
  sh->lanes = lanes;
  sh->wave_tokens = 1;
  // nothing turns, or pairs lie in a chunk: no partner in another lane
  *mode = how->interleaved || !how->rotary_dim ? kInterleaved : how->rotary_dim % 16 == 0 ? kHalfInLane : kHalfExchange;
  return STG_OK;
}

template <class F>
void with_mode(int mode, F&& f) {
  if (mode == kHalfInLane) f(std::integral_constant<int, kHalfInLane>{});
  else if (mode == kInterleaved) f(std::integral_constant<int, kInterleaved>{});
  else f(std::integral_constant<int, kHalfExchange>{});
}
template <class F>
void with_type(int32_t dtype, F&& f) {
  if (dtype == STG_BF16) f(BF16{});
  else if (dtype == STG_F16) f(F16{});
  else f(F32{});
}

// Tokens that a wave takes at a time: enough that its groups of lanes have
// four heads each, as far as 4 KiB of angles a wave allow.
int32_t wave_tokens_for(const Shape& sh, int heads, int rotary) {
  const int groups = 64 / sh.lanes;
  int n = heads > 0 ? (4 * groups + heads - 1) / heads : 1;
  if (rotary && n > 1024 / rotary) n = 1024 / rotary;
  return n < 1 ? 1 : n > 64 ? 64 : n;
}

template <int CACHE>
int launch_forward(const char* what, int32_t dtype, int mode, const Rows& q, const Rows& k, const Rows& v,
                   const int32_t* positions, const Turn& t, Shape sh, const Rows& q_out, const Rows& k_out,
                   const Cache& cache, hipStream_t st) {
  const int heads = sh.q_heads + sh.k_heads * (CACHE == kNoCache ? 1 : 2);
  if (!sh.tokens || !heads) return STG_OK;
  const int groups = 64 / sh.lanes;
  sh.wave_tokens = wave_tokens_for(sh, heads, t.rotary);
  // few tokens: a token's heads go to several workgroups, so that a step of
  // one token is spread over more than one compute unit
  while (sh.wave_tokens > 1 && sh.tokens < 1024 * sh.wave_tokens) sh.wave_tokens = (sh.wave_tokens + 1) / 2;
  const int64_t blocks = (sh.tokens + int64_t(kWaves) * sh.wave_tokens - 1) / (int64_t(kWaves) * sh.wave_tokens);
  if (blocks > (int64_t(1) << 31) - 1) return fail(STG_ERR_RANGE, "%s: too many tokens", what);
  const int rounds = (int)((int64_t(sh.wave_tokens) * heads + groups - 1) / groups);
  int shares = 1;
  while (shares < rounds && blocks * kWaves * shares < 1024) shares *= 2;
  const dim3 grid((uint32_t)blocks, (uint32_t)(shares < rounds ? shares : rounds));
  const uint32_t shmem = kWaves * wave_floats(t.rotary, sh.wave_tokens, mode) * 4;
  with_type(dtype, [&](auto type) {
    with_mode(mode, [&](auto m) {
      using T = decltype(type);
      if constexpr (CACHE == kNoCache || T::kBytes == 2)
        launch_kernel(what, forward_kernel<T, decltype(m)::value, CACHE>, grid, dim3(kThreads), shmem, st, q, k, v,
                      positions, t, sh, q_out, k_out, cache);
    });
  });
  return check_launch(what);
}

// Workgroups that sum a weight gradient: enough to fill the chip, each with
// a few tokens at least.
int32_t sum_groups(int64_t tokens, int32_t wave_tokens, int64_t most) {
  const int64_t n = (tokens + int64_t(kWaves) * wave_tokens - 1) / (int64_t(kWaves) * wave_tokens);
  return (int32_t)(n < 1 ? 1 : n > most ? most : n);
}
constexpr int64_t kSumGroups = 1024;

// (query workgroups, key workgroups): shared out by heads
void split_groups(const Shape& sh, int32_t* nq, int32_t* nk) {
  const int64_t heads = sh.q_heads + sh.k_heads;
  int64_t q = heads ? kSumGroups * sh.q_heads / heads : 0;
  q = q < 1 ? 1 : q > kSumGroups - 1 ? kSumGroups - 1 : q;
  *nq = sum_groups(sh.tokens, sh.wave_tokens, q);
  *nk = sum_groups(sh.tokens, sh.wave_tokens, kSumGroups - q);
}

}  // namespace
}  // namespace stg

using namespace stg;

extern "C" int rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor, double original_len,
                                double beta_fast, double beta_slow, float* inv_freq, float* rope_scale) {
  clear_error();
  const char* what = "rope_frequencies";
  if (rotary_dim < 0 || rotary_dim % 2) return fail(STG_ERR_INVALID, "%s: rotary_dim must be even and >= 0", what);
  if (rotary_dim && !inv_freq) return fail(STG_ERR_INVALID, "%s: null inv_freq", what);
  if (!(base > 1.0) || !std::isfinite(base)) return fail(STG_ERR_INVALID, "%s: base must be finite and > 1", what);
  if (scaling < STG_ROPE_NONE || scaling > STG_ROPE_YARN) return fail(STG_ERR_INVALID, "%s: unknown scaling", what);
  if (scaling != STG_ROPE_NONE && (!(factor >= 1.0) || !std::isfinite(factor)))
    return fail(STG_ERR_INVALID, "%s: factor must be finite and >= 1", what);
  const double d = rotary_dim, kTurn = 6.283185307179586;
  double gain = 1.0, low = 0.0, high = 0.0;
  if (scaling == STG_ROPE_YARN) {
    if (!(original_len >= 1.0) || !(beta_slow > 0.0) || !(beta_fast > beta_slow) || !std::isfinite(beta_fast) ||
        !std::isfinite(original_len))
      return fail(STG_ERR_INVALID, "%s: needs original_len >= 1 and beta_fast > beta_slow > 0", what);
    gain = 0.1 * log(factor) + 1.0;
    // the index whose frequency makes `turns` turns over original_len
    auto index = [&](double turns) { return d * log(original_len / (turns * kTurn)) / (2.0 * log(base)); };
    low = floor(index(beta_fast));
    high = ceil(index(beta_slow));
    low = low < 0.0 ? 0.0 : low;
    high = high > d - 1.0 ? d - 1.0 : high;
  }
  if (scaling == STG_ROPE_NTK && rotary_dim > 2) base *= pow(factor, d / (d - 2.0));
  for (int i = 0; i < rotary_dim / 2; ++i) {
    double f = pow(base, -2.0 * i / d);
    if (scaling == STG_ROPE_LINEAR) f /= factor;
    if (scaling == STG_ROPE_YARN) {
      const double span = high - low > 0.001 ? high - low : 0.001;
      double ramp = (i - low) / span;
      ramp = ramp < 0.0 ? 0.0 : ramp > 1.0 ? 1.0 : ramp;
      f = f * (1.0 - ramp) + f / factor * ramp;
    }
    inv_freq[i] = (float)f;
  }
  if (rope_scale) *rope_scale = (float)gain;
  return STG_OK;
}

extern "C" int qk_norm_rope(const stg_tensor* q, const stg_tensor* k, const int32_t* positions,
                            const stg_norm_rope* how, const stg_tensor* q_out, const stg_tensor* k_out, void* stream) {
  clear_error();
  const char* what = "qk_norm_rope";
  Shape sh;
  Turn t;
  int mode;
  if (int rc = check_call(what, q, k, positions, how, &sh, &t, &mode)) return rc;
  if (int rc = check_like(what, q_out, "q_out", q)) return rc;
  if (int rc = check_like(what, k_out, "k_out", k)) return rc;
  return launch_forward<kNoCache>(what, q->dtype, mode, rows_of(q), rows_of(k), Rows{}, positions, t, sh,
                                  rows_of(q_out), rows_of(k_out), Cache{}, as_stream(stream));
}

extern "C" int qk_norm_rope_append(const stg_tensor* q, const stg_tensor* k, const stg_tensor* v,
                                   const int32_t* positions, const stg_norm_rope* how, const int32_t* rows,
                                   const stg_tensor* k_cache, const stg_tensor* v_cache, const stg_tensor* page_table,
                                   const float* k_scale, const float* v_scale, const stg_tensor* q_out, void* stream) {
  clear_error();
  const char* what = "qk_norm_rope_append";
  Shape sh;
  Turn t;
  int mode;
  if (int rc = check_call(what, q, k, positions, how, &sh, &t, &mode)) return rc;
  if (q->dtype == STG_F32) return fail(STG_ERR_UNSUPPORTED, "%s: q must be bf16 or f16", what);
  if (int rc = check_like(what, v, "v", k)) return rc;
  if (int rc = check_like(what, q_out, "q_out", q)) return rc;
  if (sh.tokens && !positions) return fail(STG_ERR_INVALID, "%s: null positions", what);
  if (int rc = check_paged_cache(what, k_cache, v_cache, page_table)) return rc;
  if (k_cache->dtype != q->dtype && k_cache->dtype != STG_U8)
    return fail(STG_ERR_INVALID, "%s: the cache must be of q's dtype or u8 (e4m3 codes)", what);
  if (k_cache->shape[2] != k->shape[1] || k_cache->shape[3] != k->shape[2])
    return fail(STG_ERR_INVALID, "%s: cache and k differ in heads or depth", what);
  if (k_cache->dtype != STG_U8 && (k_scale || v_scale))
    return fail(STG_ERR_INVALID, "%s: scales are for u8 (e4m3) caches", what);
  Cache c;
  c.k = (char*)k_cache->data;
  c.v = (char*)v_cache->data;
  c.k_page = k_cache->stride[0];
  c.k_slot = k_cache->stride[1];
  c.k_head = k_cache->stride[2];
  c.v_page = v_cache->stride[0];
  c.v_slot = v_cache->stride[1];
  c.v_head = v_cache->stride[2];
  c.table = (const int32_t*)page_table->data;
  c.table_stride = page_table->stride[0];
  c.rows = (int32_t)page_table->shape[0];
  c.width = (int32_t)page_table->shape[1];
  // a cache without slots holds no page: nothing is written
  c.pages = k_cache->shape[1] ? (int32_t)k_cache->shape[0] : 0;
  c.slots = k_cache->shape[1] ? (int32_t)k_cache->shape[1] : 1;
  c.token_rows = rows;
  c.k_scale = k_scale;
  c.v_scale = v_scale;
  if (k_cache->dtype == STG_U8)
    return launch_forward<kE4m3Cache>(what, q->dtype, mode, rows_of(q), rows_of(k), rows_of(v), positions, t, sh,
                                      rows_of(q_out), Rows{}, c, as_stream(stream));
  return launch_forward<kSameCache>(what, q->dtype, mode, rows_of(q), rows_of(k), rows_of(v), positions, t, sh,
                                    rows_of(q_out), Rows{}, c, as_stream(stream));
}

extern "C" int64_t qk_norm_rope_backward_workspace(const stg_tensor* q, const stg_tensor* k) {
  clear_error();
  const char* what = "qk_norm_rope_backward_workspace";
  if (int rc = check_rows(what, q, "q")) return -rc;
  if (int rc = check_rows(what, k, "k")) return -rc;
  if (q->shape[2] != k->shape[2]) return -fail(STG_ERR_INVALID, "%s: q and k differ in depth", what);
  if (q->shape[2] > 1024) return -fail(STG_ERR_UNSUPPORTED, "%s: depth must be in [1, 1024]", what);
  return kSumGroups * q->shape[2] * 4;
}

extern "C" int qk_norm_rope_backward(const stg_tensor* dq_out, const stg_tensor* dk_out, const stg_tensor* q,
                                     const stg_tensor* k, const int32_t* positions, const stg_norm_rope* how,
                                     const stg_tensor* dq, const stg_tensor* dk, void* dq_weight, void* dk_weight,
                                     void* workspace, int64_t workspace_bytes, void* stream) {
  clear_error();
  const char* what = "qk_norm_rope_backward";
  Shape sh;
  Turn t;
  int mode;
  if (int rc = check_call(what, q, k, positions, how, &sh, &t, &mode)) return rc;
  if (int rc = check_like(what, dq_out, "dq_out", q)) return rc;
  if (int rc = check_like(what, dk_out, "dk_out", k)) return rc;
  if (int rc = check_like(what, dq, "dq", q)) return rc;
  if (int rc = check_like(what, dk, "dk", k)) return rc;
  const bool sums = dq_weight || dk_weight;
  if (sums && !t.norm) return fail(STG_ERR_INVALID, "%s: weight gradients without norm", what);
  if (sums && how->weight_dtype != STG_F32 && how->weight_dtype != q->dtype)
    return fail(STG_ERR_UNSUPPORTED, "%s: weight gradients must be f32 or of q's dtype", what);
  if (sums) {
    const int64_t need = kSumGroups * sh.depth * 4;
    if (!workspace || workspace_bytes < need)
      return fail(STG_ERR_INVALID, "%s: needs a workspace of %lld bytes", what, (long long)need);
    if ((uintptr_t)workspace & 255) return fail(STG_ERR_INVALID, "%s: workspace must be 256-byte aligned", what);
  }
  const int heads = sh.q_heads < sh.k_heads ? sh.q_heads : sh.k_heads;
  sh.wave_tokens = wave_tokens_for(sh, heads, t.rotary);
  while (sh.wave_tokens > 1 && sh.tokens < 1024 * sh.wave_tokens) sh.wave_tokens = (sh.wave_tokens + 1) / 2;
  int32_t nq, nk;
  split_groups(sh, &nq, &nk);
  float* pq = (float*)workspace;
  float* pk = pq + int64_t(nq) * sh.depth;
  const Gradient gq{rows_of(dq_out), rows_of(q), rows_of(dq), t.wq, sh.q_heads, nq, dq_weight ? pq : nullptr};
  const Gradient gk{rows_of(dk_out), rows_of(k), rows_of(dk), t.wk, sh.k_heads, nk, dk_weight ? pk : nullptr};
  const hipStream_t st = as_stream(stream);
  uint32_t shmem = kWaves * wave_floats(t.rotary, sh.wave_tokens, mode) * 4;
  if (shmem < kWaves * (uint32_t)sh.depth * 4) shmem = kWaves * sh.depth * 4;
  if (!sh.tokens && !sums) return STG_OK;
  with_type(q->dtype, [&](auto type) {
    with_mode(mode, [&](auto m) {
      launch_kernel(what, backward_kernel<decltype(type), decltype(m)::value>, dim3(nq + nk), dim3(kThreads), shmem, st,
                    gq, gk, positions, t, sh);
    });
  });
  if (int rc = check_launch(what)) return rc;
  if (!sums) return STG_OK;
  with_type(q->dtype, [&](auto type) {
    launch_kernel("qk_norm_rope_backward/weights", weight_kernel<decltype(type)>, dim3((sh.depth + 63) / 64, 2),
                  dim3(1024), 0, st, (const float*)pq, (int)nq, dq_weight, (const float*)pk, (int)nk, dk_weight,
                  (int)sh.depth, (int)t.weight_f32);
  });
  return check_launch("qk_norm_rope_backward/weights");
}
