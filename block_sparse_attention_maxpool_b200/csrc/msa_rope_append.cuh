// Cache append with the position rotation applied on the way, and the append
// into an 8-bit cache with one scale per (128-token block, group).
//
// Rotation of a row x at position p: pair i of the first 2 * half dims turns
// by p * inv_freq[i]: (x0, x1) -> (x0 c - x1 s, x1 c + x0 s), pair i being
// dims (i, i + half) or, interleaved, (2i, 2i + 1); later dims are copied.
// p * inv_freq is formed in float64 and reduced to a fraction of a turn
// there: in float32 the angle of position 131071 would be off by up to 0.008
// rad.  c and s are float32 (one table of 64 values per warp in shared
// memory, filled once for all rows of the warp's position), the turn is
// float32 arithmetic, and one rounding to the stored type follows.
//
// Everything here is bound by its bytes (a prompt) or by launch latency (a
// decode step).  In the bf16 append one warp owns a (token, group) or a (query, group): a
// token's K and V rows and its indexer key are one load each per lane, a
// query's 16 heads are eight 16-byte loads per lane, all in flight before
// the first is used.  16384 tokens with 64 query heads and indexer rows (738
// MB): 130 us, 5.7 TB/s, 0.86 of the measured copy rate; 32 tokens: 5.4 us.
#pragma once

#include <cuda_fp16.h>

#include "msa_common.cuh"

namespace msa {
namespace rope {

struct Rope {
  const double* inv_freq;   // [half]; null: no rotation (half = 0)
  int half;                 // rotated pairs, a multiple of 8, at most 64
  int interleaved;
};

// cos and sin of the `half` angles of position p, into the warp's table.
__device__ __forceinline__ void fill_table(const Rope& r, int p, float* cs, float* sn, int lane) {
  for (int i = lane; i < r.half; i += 32) {
    double t = static_cast<double>(p) * __ldg(r.inv_freq + i) * 0.15915494309189535;   // turns
    t -= rint(t);
    float s, c;
    sincospif(2.f * static_cast<float>(t), &s, &c);
    cs[i] = c;
    sn[i] = s;
  }
  __syncwarp();
}

// Lane j of n lanes sharing a row of 128 (two vectors of W = 64 / n elements
// each): where its two vectors start.  Rotated lanes (j < half / W) hold the
// pairs j * W .. j * W + W - 1, whichever dims these are; the others copy.
template <int W>
__device__ __forceinline__ void vector_dims(const Rope& r, int j, int& d0, int& d1) {
  const bool split = j * W < r.half && !r.interleaved;
  d0 = split ? j * W : 2 * j * W;
  d1 = split ? j * W + r.half : 2 * j * W + W;
}

// Turn the lane's two vectors in place.
template <int W>
__device__ __forceinline__ void turn(const Rope& r, int j, float (&a)[W], float (&b)[W], const float* cs,
                                     const float* sn) {
  if (j * W >= r.half) return;
  float c[W], s[W];
#pragma unroll
  for (int i = 0; i < W; i += 4) {
    const float4 x = *reinterpret_cast<const float4*>(cs + j * W + i);
    const float4 y = *reinterpret_cast<const float4*>(sn + j * W + i);
    c[i] = x.x; c[i + 1] = x.y; c[i + 2] = x.z; c[i + 3] = x.w;
    s[i] = y.x; s[i + 1] = y.y; s[i + 2] = y.z; s[i + 3] = y.w;
  }
  if (!r.interleaved) {
#pragma unroll
    for (int i = 0; i < W; ++i) {
      const float x0 = a[i], x1 = b[i];
      a[i] = x0 * c[i] - x1 * s[i];
      b[i] = x1 * c[i] + x0 * s[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < W / 2; ++i) {
      const float x0 = a[2 * i], x1 = a[2 * i + 1];
      a[2 * i] = x0 * c[i] - x1 * s[i];
      a[2 * i + 1] = x1 * c[i] + x0 * s[i];
      const float y0 = b[2 * i], y1 = b[2 * i + 1];
      b[2 * i] = y0 * c[W / 2 + i] - y1 * s[W / 2 + i];
      b[2 * i + 1] = y1 * c[W / 2 + i] + y0 * s[W / 2 + i];
    }
  }
}

__device__ __forceinline__ void unpack8(const uint4& v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = __uint_as_float(w[i] << 16);
    f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}

__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
}

// A bf16 row's two 16-byte vectors (8 lanes per row), turned.  Copying lanes
// write back the bits they read.
__device__ __forceinline__ void turn_bf16(const Rope& r, int j, uint4& va, uint4& vb, const float* cs,
                                          const float* sn) {
  if (j * 8 >= r.half) return;
  float a[8], b[8];
  unpack8(va, a);
  unpack8(vb, b);
  turn<8>(r, j, a, b, cs, sn);
  va = pack8(a);
  vb = pack8(b);
}

struct AppendParams {
  Rope rope;
  __nv_bfloat16* k_cache;        // null: no K/V rows in this call
  __nv_bfloat16* v_cache;
  const __nv_bfloat16* k_new;    // [n_tok][G][128]
  const __nv_bfloat16* v_new;
  void* idx_cache;               // null: no indexer keys
  int idx_f16;
  const float* idx_new;          // [n_tok][G][128]
  const int32_t* tok_stream;
  const int32_t* tok_pos;
  int n_tok;
  const __nv_bfloat16* q;        // [n_q][16 G][128], null: no queries
  __nv_bfloat16* q_out;          // may be q
  const float* idx_q;            // [n_q][G][128], null: none
  float* idx_q_out;              // may be idx_q
  const int32_t* q_pos;
  int n_q;
  int n_streams, G, capacity;
  KvPages pages;
};

constexpr int kWarps = 8;

// An F32 row of 128 by 16 lanes (two vectors of four each), turned.
__device__ __forceinline__ void turn_f32_row(const Rope& r, int j, const float* src, float (&a)[4], float (&b)[4],
                                             int& d0, int& d1, const float* cs, const float* sn) {
  vector_dims<4>(r, j, d0, d1);
  const float4 x = *reinterpret_cast<const float4*>(src + d0);
  const float4 y = *reinterpret_cast<const float4*>(src + d1);
  a[0] = x.x; a[1] = x.y; a[2] = x.z; a[3] = x.w;
  b[0] = y.x; b[1] = y.y; b[2] = y.z; b[3] = y.w;
  turn<4>(r, j, a, b, cs, sn);
}

__global__ void __launch_bounds__(kWarps * 32) rope_append_kernel(const AppendParams P) {
  __shared__ __align__(16) float table[kWarps][2][64];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  float* cs = table[threadIdx.x >> 5][0];
  float* sn = table[threadIdx.x >> 5][1];
  const long long unit = static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5);
  const long long tok_units = static_cast<long long>(P.n_tok) * P.G;
  const int j = lane & 7;
  const int row4 = lane >> 3;                 // which of four rows this lane works on
  int d0, d1;
  vector_dims<8>(P.rope, j, d0, d1);
  if (unit < tok_units) {
    const int t = static_cast<int>(unit / P.G);
    const int g = static_cast<int>(unit - static_cast<long long>(t) * P.G);
    const int s = P.tok_stream[t];
    const int p = P.tok_pos[t];
    if (s < 0 || s >= P.n_streams || p < 0 || p >= P.capacity) {
      if (g == 0 && lane == 0) raise_error(MSA_DEVERR_TOKEN_RANGE);
      return;
    }
    const long long blk = kv_block_row(P.pages, s, g, p / 128, P.G, P.capacity);
    if (blk < 0) {
      if (lane == 0) raise_error(MSA_DEVERR_PAGE_RANGE);
      return;
    }
    fill_table(P.rope, p, cs, sn, lane);
    const size_t dst = (static_cast<size_t>(blk) + (p & 127)) * 128;
    const size_t src = (static_cast<size_t>(t) * P.G + g) * 128;
    if (lane < 16) {                          // lanes 0-7: the K row, 8-15: the V row (copied as it is)
      if (P.k_cache != nullptr) {
        const bool is_k = row4 == 0;
        const __nv_bfloat16* from = (is_k ? P.k_new : P.v_new) + src;
        __nv_bfloat16* to = (is_k ? P.k_cache : P.v_cache) + dst;
        uint4 a = *reinterpret_cast<const uint4*>(from + d0);
        uint4 b = *reinterpret_cast<const uint4*>(from + d1);
        if (is_k) turn_bf16(P.rope, j, a, b, cs, sn);
        *reinterpret_cast<uint4*>(to + d0) = a;
        *reinterpret_cast<uint4*>(to + d1) = b;
      }
    } else if (P.idx_cache != nullptr) {      // lanes 16-31: the indexer key
      float a[4], b[4];
      int e0, e1;
      turn_f32_row(P.rope, lane - 16, P.idx_new + src, a, b, e0, e1, cs, sn);
      if (P.idx_f16) {
        __half* to = static_cast<__half*>(P.idx_cache) + dst;
        __half2 h[4] = {__floats2half2_rn(a[0], a[1]), __floats2half2_rn(a[2], a[3]), __floats2half2_rn(b[0], b[1]),
                        __floats2half2_rn(b[2], b[3])};
        *reinterpret_cast<uint2*>(to + e0) = *reinterpret_cast<uint2*>(&h[0]);
        *reinterpret_cast<uint2*>(to + e1) = *reinterpret_cast<uint2*>(&h[2]);
      } else {
        float* to = static_cast<float*>(P.idx_cache) + dst;
        *reinterpret_cast<float4*>(to + e0) = make_float4(a[0], a[1], a[2], a[3]);
        *reinterpret_cast<float4*>(to + e1) = make_float4(b[0], b[1], b[2], b[3]);
      }
    }
    return;
  }
  const long long qu = unit - tok_units;
  if (qu >= static_cast<long long>(P.n_q) * P.G) return;
  const int i = static_cast<int>(qu / P.G);
  const int g = static_cast<int>(qu - static_cast<long long>(i) * P.G);
  const int p = P.q_pos[i];
  if (p < 0 || p >= P.capacity) {
    if (g == 0 && lane == 0) raise_error(MSA_DEVERR_QUERY_RANGE);
    return;
  }
  uint4 a[4], b[4];
  const size_t row0 = (static_cast<size_t>(i) * P.G + g) * 16;
  if (P.q != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const __nv_bfloat16* from = P.q + (row0 + 4 * k + row4) * 128;
      a[k] = *reinterpret_cast<const uint4*>(from + d0);
      b[k] = *reinterpret_cast<const uint4*>(from + d1);
    }
  }
  fill_table(P.rope, p, cs, sn, lane);
  if (P.idx_q != nullptr && lane >= 16) {
    float x[4], y[4];
    int e0, e1;
    const size_t row = (static_cast<size_t>(i) * P.G + g) * 128;
    turn_f32_row(P.rope, lane - 16, P.idx_q + row, x, y, e0, e1, cs, sn);
    *reinterpret_cast<float4*>(P.idx_q_out + row + e0) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(P.idx_q_out + row + e1) = make_float4(y[0], y[1], y[2], y[3]);
  }
  if (P.q != nullptr) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      turn_bf16(P.rope, j, a[k], b[k], cs, sn);
      __nv_bfloat16* to = P.q_out + (row0 + 4 * k + row4) * 128;
      *reinterpret_cast<uint4*>(to + d0) = a[k];
      *reinterpret_cast<uint4*>(to + d1) = b[k];
    }
  }
}

// ---- 8-bit cache ----------------------------------------------------------------
// Rows are e4m3; a (block, group) of K or V has one scale, the power of two
// that leaves its largest finite value at or below 448 (the largest e4m3).
// A power of two costs no accuracy against amax / 448 (e4m3 is a floating-
// point type: a value's relative rounding does not depend on the scale until
// it is 2^-14 of the largest) and makes growing the scale harmless: dividing
// a stored row by a power of two rounds only values that become subnormal.
// What a call does to a touched (block, group): after = max(before, need),
// need from the call's tokens; rows already there are requantised once, from
// before to after; the call's rows are quantised once, with after.  A token
// at the block's first slot starts the block anew (a recycled page), before
// counts as empty then.

struct BlockNeed {      // per (stream, block, group), zeroed before the call's first kernel
  unsigned int k, v;    // bits of the scale the call's tokens need; 0: not touched
  unsigned int fresh;   // the call writes the block's first slot
  unsigned int pad;
};

struct Fp8Params {
  Rope rope;
  uint8_t* k_cache;
  uint8_t* v_cache;
  float* k_scale;                // [S][G][nblk], or [n_pages][G]
  float* v_scale;
  const __nv_bfloat16* k_new;    // [n_tok][G][128]
  const __nv_bfloat16* v_new;
  const int32_t* tok_stream;
  const int32_t* tok_pos;
  int n_tok;
  int n_streams, G, capacity;
  KvPages pages;
  BlockNeed* need;               // [S * nblk * G]
};

constexpr int kMinExp = -100;    // scale of a block of zeros: 2^-100

// Bits of the smallest power of two 2^e, e >= kMinExp, with amax <= 448 * 2^e
// (448 = 1.75 * 2^8).
__device__ __forceinline__ unsigned int scale_bits(float amax) {
  const unsigned int b = __float_as_uint(amax);
  int e = static_cast<int>(b >> 23) - 127 - ((b & 0x7fffffu) <= 0x600000u ? 8 : 7);
  e = max(e, kMinExp);
  return static_cast<unsigned int>(e + 127) << 23;
}

__device__ __forceinline__ float finite_abs(float x) {
  x = fabsf(x);
  return x <= 3.402823466e38f ? x : 0.f;      // NaN and infinities do not set the scale
}

// Four floats to e4m3, nearest even; beyond +-448 saturates, NaN stays NaN.
__device__ __forceinline__ uint32_t to_e4m3x4(float a, float b, float c, float d) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(b), "f"(a));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(d), "f"(c));
  return static_cast<uint32_t>(lo) | (static_cast<uint32_t>(hi) << 16);
}

__device__ __forceinline__ float2 from_e4m3x2(uint16_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(v));
  return __half22float2(*reinterpret_cast<__half2*>(&h));
}

__device__ __forceinline__ uint32_t requantise4(uint32_t w, float ratio) {
  const float2 a = from_e4m3x2(static_cast<uint16_t>(w & 0xffffu));
  const float2 b = from_e4m3x2(static_cast<uint16_t>(w >> 16));
  return to_e4m3x4(a.x * ratio, a.y * ratio, b.x * ratio, b.y * ratio);
}

// One token's K row (lanes 0-15) or V row (lanes 16-31): the lane's two
// vectors of four values and where they start.
__device__ __forceinline__ void load_kv(const Fp8Params& P, size_t src, int lane, float (&a)[4], float (&b)[4],
                                        int& d0, int& d1) {
  vector_dims<4>(P.rope, lane & 15, d0, d1);
  const __nv_bfloat16* from = (lane < 16 ? P.k_new : P.v_new) + src;
  const uint2 x = *reinterpret_cast<const uint2*>(from + d0);
  const uint2 y = *reinterpret_cast<const uint2*>(from + d1);
  a[0] = __uint_as_float(x.x << 16); a[1] = __uint_as_float(x.x & 0xffff0000u);
  a[2] = __uint_as_float(x.y << 16); a[3] = __uint_as_float(x.y & 0xffff0000u);
  b[0] = __uint_as_float(y.x << 16); b[1] = __uint_as_float(y.x & 0xffff0000u);
  b[2] = __uint_as_float(y.y << 16); b[3] = __uint_as_float(y.y & 0xffff0000u);
}

// Largest finite magnitude of the half-warp's row.
__device__ __forceinline__ float row_amax(const float (&a)[4], const float (&b)[4]) {
  float m = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) m = fmaxf(m, fmaxf(finite_abs(a[i]), finite_abs(b[i])));
#pragma unroll
  for (int o = 8; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
  return m;
}

// Where token t of group g goes: the first row of its block, or -1 (and the
// error bit) when it names no slot.
__device__ __forceinline__ long long fp8_block(const Fp8Params& P, int t, int g, int& s, int& p, int lane,
                                               bool report) {
  s = P.tok_stream[t];
  p = P.tok_pos[t];
  if (s < 0 || s >= P.n_streams || p < 0 || p >= P.capacity) {
    if (report && g == 0 && lane == 0) raise_error(MSA_DEVERR_TOKEN_RANGE);
    return -1;
  }
  const long long blk = kv_block_row(P.pages, s, g, p / 128, P.G, P.capacity);
  if (blk < 0 && report && lane == 0) raise_error(MSA_DEVERR_PAGE_RANGE);
  return blk;
}

// 1 of 3: the scale every touched block needs (integer maxima: the order in
// which tokens arrive does not matter).  One warp per token: the table of its
// angles serves all groups, four groups' rows are in flight at a time.
__global__ void __launch_bounds__(kWarps * 32, 4) fp8_need_kernel(const Fp8Params P) {
  __shared__ __align__(16) float table[kWarps][2][64];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= P.n_tok) return;
  float a[4][4], b[4][4];
  int d0, d1;
  auto load4 = [&](int g0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_kv(P, (static_cast<size_t>(t) * P.G + min(g0 + i, P.G - 1)) * 128, lane, a[i], b[i], d0, d1);
  };
  load4(0);                                    // does not depend on where the token goes
  int s, p;
  if (fp8_block(P, t, 0, s, p, lane, true) < 0) return;
  float* cs = table[threadIdx.x >> 5][0];
  float* sn = table[threadIdx.x >> 5][1];
  fill_table(P.rope, p, cs, sn, lane);
  BlockNeed* e = P.need + (static_cast<size_t>(s) * (P.capacity / 128) + p / 128) * P.G;
  for (int g0 = 0; g0 < P.G; g0 += 4) {
    if (g0 > 0) load4(g0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (lane < 16) turn<4>(P.rope, lane & 15, a[i], b[i], cs, sn);
      const unsigned int bits = scale_bits(row_amax(a[i], b[i]));
      if (g0 + i < P.G && (lane & 15) == 0) {
        atomicMax(lane == 0 ? &e[g0 + i].k : &e[g0 + i].v, bits);
        if (lane == 0 && (p & 127) == 0) e[g0 + i].fresh = 1u;
      }
    }
  }
}

// Requantise `rows` of 128 e4m3 values by `ratio` (n threads, thread i).
__device__ __forceinline__ void requantise_block(uint8_t* cache, long long row, float ratio, int i, int n) {
  uint4* v = reinterpret_cast<uint4*>(cache + static_cast<size_t>(row) * 128);
  for (int k = i; k < 128 * 128 / 16; k += n) {
    uint4 x = v[k];
    x.x = requantise4(x.x, ratio);
    x.y = requantise4(x.y, ratio);
    x.z = requantise4(x.z, ratio);
    x.w = requantise4(x.w, ratio);
    v[k] = x;
  }
}

// New scale of a touched block from the old one; `grow`: the old rows' ratio
// when they have to be requantised, else 0 (a ratio that float32 cannot hold
// is taken as 2^-126, which makes zeros of any e4m3 as well).
__device__ __forceinline__ float next_scale(float held, bool fresh, unsigned int need_bits, float& grow) {
  const float before = !fresh && held > 0.f ? held : 0.f;
  const float need = __uint_as_float(need_bits);
  const float after = fmaxf(before, need);
  grow = before > 0.f && after > before ? fmaxf(before / after, 1.17549435e-38f) : 0.f;
  return after;
}

// 2 of 3: the touched blocks' scales, and their older rows requantised.  One
// table entry per lane; the warp then works on the blocks that have to be
// requantised one after the other.
__global__ void __launch_bounds__(kWarps * 32) fp8_scale_kernel(const Fp8Params P) {
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int nblk = P.capacity / 128;
  const long long n = static_cast<long long>(P.n_streams) * nblk * P.G;
  const long long e = (static_cast<long long>(blockIdx.x) * kWarps + (threadIdx.x >> 5)) * 32 + lane;
  long long row = -1;
  float gk = 0.f, gv = 0.f;
  if (e < n) {
    const uint4 need = *reinterpret_cast<const uint4*>(P.need + e);
    if (need.x != 0u) {
      const int g = static_cast<int>(e % P.G);
      const long long sb = e / P.G;
      row = kv_block_row(P.pages, static_cast<int>(sb / nblk), g, static_cast<int>(sb % nblk), P.G, P.capacity);
      if (row >= 0) {
        P.k_scale[row / 128] = next_scale(P.k_scale[row / 128], need.z != 0u, need.x, gk);
        P.v_scale[row / 128] = next_scale(P.v_scale[row / 128], need.z != 0u, need.y, gv);
      }
    }
  }
  unsigned int todo = __ballot_sync(0xffffffffu, gk != 0.f || gv != 0.f);
  while (todo != 0u) {
    const int l = __ffs(todo) - 1;
    todo &= todo - 1u;
    const long long r = __shfl_sync(0xffffffffu, row, l);
    const float fk = __shfl_sync(0xffffffffu, gk, l), fv = __shfl_sync(0xffffffffu, gv, l);
    if (fk != 0.f) requantise_block(P.k_cache, r, fk, lane, 32);
    if (fv != 0.f) requantise_block(P.v_cache, r, fv, lane, 32);
  }
}

// Quantise one row with its block's scale (a product where the scale is a
// normal power of two, as this call makes them: its reciprocal is exact; a
// caller's other scales are divided by).
__device__ __forceinline__ void store_e4m3(uint8_t* row, const float (&a)[4], const float (&b)[4], int d0, int d1,
                                           float scale) {
  const uint32_t e = __float_as_uint(scale);
  if ((e & 0x807fffffu) == 0u && e - (1u << 23) < (252u << 23)) {
    const float inv = __uint_as_float((254u << 23) - e);
    *reinterpret_cast<uint32_t*>(row + d0) = to_e4m3x4(a[0] * inv, a[1] * inv, a[2] * inv, a[3] * inv);
    *reinterpret_cast<uint32_t*>(row + d1) = to_e4m3x4(b[0] * inv, b[1] * inv, b[2] * inv, b[3] * inv);
  } else {
    *reinterpret_cast<uint32_t*>(row + d0) = to_e4m3x4(a[0] / scale, a[1] / scale, a[2] / scale, a[3] / scale);
    *reinterpret_cast<uint32_t*>(row + d1) = to_e4m3x4(b[0] / scale, b[1] / scale, b[2] / scale, b[3] / scale);
  }
}

// 3 of 3: the call's rows.
__global__ void __launch_bounds__(kWarps * 32, 4) fp8_store_kernel(const Fp8Params P) {
  __shared__ __align__(16) float table[kWarps][2][64];
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (t >= P.n_tok) return;
  float a[4][4], b[4][4];
  int d0, d1;
  auto load4 = [&](int g0) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      load_kv(P, (static_cast<size_t>(t) * P.G + min(g0 + i, P.G - 1)) * 128, lane, a[i], b[i], d0, d1);
  };
  load4(0);
  int s, p;
  const long long blk0 = fp8_block(P, t, 0, s, p, lane, false);
  if (blk0 < 0) return;
  // group g's block lies g blocks (pool) or g regions (contiguous cache) on
  const long long step = P.pages.table != nullptr ? 128 : P.capacity;
  const float* scales = lane < 16 ? P.k_scale : P.v_scale;
  uint8_t* cache = lane < 16 ? P.k_cache : P.v_cache;
  // lane 16 i + g holds the K (i = 0) or V scale of group g (G <= 16)
  float mine = 0.f;
  if ((lane & 15) < P.G) mine = scales[(blk0 + (lane & 15) * step) / 128];
  float* cs = table[threadIdx.x >> 5][0];
  float* sn = table[threadIdx.x >> 5][1];
  fill_table(P.rope, p, cs, sn, lane);
  for (int g0 = 0; g0 < P.G; g0 += 4) {
    if (g0 > 0) load4(g0);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float scale = __shfl_sync(0xffffffffu, mine, (lane & 16) + ((g0 + i) & 15));
      if (lane < 16) turn<4>(P.rope, lane & 15, a[i], b[i], cs, sn);
      if (g0 + i < P.G)
        store_e4m3(cache + (static_cast<size_t>(blk0 + (g0 + i) * step) + (p & 127)) * 128, a[i], b[i], d0, d1, scale);
    }
  }
}

// The three steps in one launch, for calls of at most kSmallTokens tokens (a
// decode step, a few drafted tokens): one CTA per (token, group).  The CTA of
// the first token in the list that names a block looks the list over for the
// others of that block and does all of them; the CTAs of the others leave.
// With three launches and a cleared table 32 tokens took 28.8 us a call, and
// the work of one launch is bound by its chain of dependent loads; the search
// grows with the square of the tokens, so it is kept to short lists.
constexpr int kSmallTokens = 256;
constexpr int kSmallWarps = 4;

__global__ void __launch_bounds__(kSmallWarps * 32) fp8_append_small_kernel(const Fp8Params P) {
  __shared__ __align__(16) float table[kSmallWarps][2][64];
  __shared__ unsigned int need_k, need_v, fresh, later;
  pdl_trigger();
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int t = blockIdx.x / P.G;
  const int g = blockIdx.x - t * P.G;
  int s, p;
  const long long blk = fp8_block(P, t, g, s, p, threadIdx.x, true);
  if (blk < 0) return;
  if (threadIdx.x == 0) {
    need_k = need_v = 0u;
    fresh = later = 0u;
  }
  // this thread's two tokens of the list: do they lie in the same block
  static_assert(kSmallTokens == 2 * kSmallWarps * 32, "two tokens of the list per thread");
  int pos[2];
  bool same[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int u = i * kSmallWarps * 32 + threadIdx.x;
    pos[i] = u < P.n_tok ? P.tok_pos[u] : -1;
    same[i] = u < P.n_tok && P.tok_stream[u] == s && pos[i] >= 0 && pos[i] / 128 == p / 128;
  }
  const float held_k = P.k_scale[blk / 128], held_v = P.v_scale[blk / 128];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (same[i] && i * kSmallWarps * 32 + static_cast<int>(threadIdx.x) < t) later = 1u;
  __syncthreads();
  if (later != 0u) return;                     // an earlier token's CTA does this block
  float* cs = table[warp][0];
  float* sn = table[warp][1];
  float a[4], b[4];
  int d0 = 0, d1 = 0, last = -1;
  // each warp does the tokens that its threads found, one after the other
  auto each = [&](auto&& fn) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      unsigned int todo = __ballot_sync(0xffffffffu, same[i]);
      while (todo != 0u) {
        const int l = __ffs(todo) - 1;
        todo &= todo - 1u;
        const int u = i * kSmallWarps * 32 + warp * 32 + l;
        const int q = __shfl_sync(0xffffffffu, pos[i], l);
        if (u != last) {                       // (kept from the first pass where a warp has one token)
          load_kv(P, (static_cast<size_t>(u) * P.G + g) * 128, lane, a, b, d0, d1);
          __syncwarp();
          fill_table(P.rope, q, cs, sn, lane);
          if (lane < 16) turn<4>(P.rope, lane & 15, a, b, cs, sn);
          last = u;
        }
        fn(q);
      }
    }
  };
  each([&](int q) {
    const unsigned int bits = scale_bits(row_amax(a, b));
    if (lane == 0) atomicMax(&need_k, bits);
    if (lane == 16) atomicMax(&need_v, bits);
    if (lane == 0 && (q & 127) == 0) fresh = 1u;
  });
  __syncthreads();
  float gk, gv;
  const float sk = next_scale(held_k, fresh != 0u, need_k, gk);
  const float sv = next_scale(held_v, fresh != 0u, need_v, gv);
  if (gk != 0.f) requantise_block(P.k_cache, blk, gk, threadIdx.x, kSmallWarps * 32);
  if (gv != 0.f) requantise_block(P.v_cache, blk, gv, threadIdx.x, kSmallWarps * 32);
  if (threadIdx.x == 0) {
    P.k_scale[blk / 128] = sk;
    P.v_scale[blk / 128] = sv;
  }
  __syncthreads();                             // the old rows are requantised before the new ones land
  each([&](int q) {
    store_e4m3((lane < 16 ? P.k_cache : P.v_cache) + (static_cast<size_t>(blk) + (q & 127)) * 128, a, b, d0, d1,
               lane < 16 ? sk : sv);
  });
}

}  // namespace rope
}  // namespace msa
