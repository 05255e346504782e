// Expansion of an 8-bit cache to bf16, ahead of a prefill call's attention.
//
// A prompt's tiles read a block many times (every 16 queries of a window read
// it again, 8 queries of a selection share it at best), so the e4m3 values
// are converted once per call, by a kernel of their own, into caches in the
// caller's workspace, which the bf16 prefill kernels read: bf16(scale * e4m3),
// exact when the scale is a power of two, as the append writes it.  Only blocks
// that some query of the call can see are touched.  Small caches and pools
// expand in place: the copy has their layout, and the same page table serves
// both.  Of a large one the visible blocks go, stream by stream, into a pool of
// `room` pages behind a table of the call's own.  What the queries see only the
// device knows (the positions are there, and a captured call is replayed with
// others), so where it matters the last CTA of the range kernel adds the blocks
// up and chooses: the tiles, or the cluster kernel that reads the 8-bit cache
// itself, where the blocks do not fit, the queries come from too many streams or
// a selection over many blocks takes less time there.  The kernels of the side
// that was not chosen return at once (2048 queries: 9 to 26 us in all).  Bound by
// bytes: 128 read and 256 written per row.  (Converted inside the attention kernel by four warps of
// its own, block by block, the 2048-query selection on 16384 tokens took 1.04
// ms instead of 0.66: the conversion of a block, about 4000 cycles next to the
// softmax warps, paced the loop.)
#pragma once

#include <cuda_fp16.h>

#include "msa_common.cuh"

namespace msa {
namespace expand {

// Selected blocks: whether the union tiles take less time than the cluster
// kernel, for n_q queries that see `total` blocks, `top` at most in one stream.
// A tile of 8 queries reads the union of their selections, about
// top (1 - (1 - 15 / top)^8) blocks where queries choose apart from one another,
// one microsecond a block on 148 SMs, behind the expansion of all that is seen
// (96 KB of traffic per block and group); the cluster kernel reads each query's
// 16 blocks, 0.085 us for a (query, group).  Measured, 4 groups, one stream
// (tiles / cluster, us, back to back), by the tokens that the queries see:
//
//   queries     1024         4096         16384         65536
//       256    36 /  59     68 /  89    123 /   89    179 /   91
//       512    48 / 103    107 / 171    193 /  171    277 /  174
//      1024    68 / 174    181 / 336    334 /  336    469 /  341
//      2048                267 / 666    579 /  668    774 /  672
//      4096                391 / 1119  1101 / 1329   1502 / 1331
//
// and 1920 queries of 30 streams on 2048 tokens 244 / 635, on 4096 422 / 635, on
// 16384 927 / 636.
__host__ __device__ inline bool selection_tiles_pay(int n_q, int G, int top, long long total, int sms) {
  const float blocks = static_cast<float>(top), pairs = static_cast<float>(n_q) * G;
  const float miss = 1.f - fminf(1.f, 15.f / blocks), miss2 = miss * miss, miss4 = miss2 * miss2;
  const float rounds = ceilf(ceilf(n_q / 8.f) * G / sms);
  const float tiles = 40.f + rounds * blocks * (1.f - miss4 * miss4) + 0.023f * static_cast<float>(total) * G;
  return tiles < 10.f + 0.085f * (148.f / sms) * pairs * fminf(blocks, 16.f) / 16.f;
}

struct Params {
  const uint8_t* k_cache;
  const uint8_t* v_cache;
  const float* k_scale;       // scale of cache row r: k_scale[r / 128]
  const float* v_scale;
  uint4* k_out;               // bf16, rows as in k_cache or in the pages of `table`
  uint4* v_out;
  int32_t* range;             // [S][2], zeroed: highest position + 1, capacity - lowest slot seen
  int32_t* ctl;               // [2]: CTAs of the range kernel that are done (zeroed), the choice (kTiles); null: neither
  int32_t* base;              // [S]: first page of the stream's blocks
  int32_t* table;             // [S][capacity / 128]: the call's own pages; null: laid out as the 8-bit cache
  long long room;             // pages behind `table`
  const int32_t* q_stream;
  const int32_t* q_pos;
  int n_q, G, n_streams, capacity;
  int window, n_sink;         // selection form: window = capacity, n_sink = 0
  bool clean;                 // selection form: NaN in V rows that the stream's queries do not see becomes zero
  int share;                  // queries per stream that the tiles want; 0: the host has seen to it
  int sms;                    // selection form that the device chooses by what is seen; else 0
  KvPages pages;
};

constexpr int32_t kCluster = 0, kTiles = 1;      // ctl[1]

// The blocks that a stream's queries see: the sinks' that lie before the window's first, then the window's on.
struct Visible {
  int sinks, win, n;
  __device__ Visible(const Params& P, int hi, int lo) {
    const int first = P.capacity - lo;
    win = first / 128;
    sinks = min((P.n_sink + 127) / 128, win);
    n = hi == 0 ? 0 : sinks + (hi - 1) / 128 - win + 1;
  }
  __device__ int block(int i) const { return i < sinks ? i : win + i - sinks; }
};

// The choice, and where each stream's blocks go (one CTA of 256 threads, the
// ranges complete).
__device__ void choose(const Params& P) {
  __shared__ long long before[8];
  __shared__ int top, streams;
  if (threadIdx.x == 0) top = streams = 0;
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long total = 0;
  for (int s0 = 0; s0 < P.n_streams; s0 += 256) {
    const int s = s0 + threadIdx.x;
    const long long n = s < P.n_streams ? Visible(P, __ldcg(P.range + 2 * s), __ldcg(P.range + 2 * s + 1)).n : 0;
    if (n > 0) {
      atomicMax(&top, static_cast<int>(n));
      atomicAdd(&streams, 1);
    }
    long long sum = n;                             // inclusive over the warp, then over the warps
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, sum, o);
      if (lane >= o) sum += x;
    }
    if (lane == 31) before[warp] = sum;
    __syncthreads();
    long long at = total + sum - n;
    for (int w = 0; w < 8; ++w) {
      if (w < warp) at += before[w];
      total += before[w];
    }
    __syncthreads();
    if (s < P.n_streams && P.table != nullptr) P.base[s] = static_cast<int32_t>(min(at, P.room));
  }
  if (threadIdx.x != 0) return;
  bool tiles = (P.table == nullptr || total <= P.room) && P.n_q >= static_cast<long long>(P.share) * streams;
  if (tiles && P.sms > 0 && total > 0) tiles = selection_tiles_pay(P.n_q, P.G, top, total, P.sms);
  P.ctl[1] = tiles ? kTiles : kCluster;
}

// The slots that each stream's queries can see.
__global__ void __launch_bounds__(256) expand_range_kernel(const Params P) {
  pdl_trigger();
  pdl_wait();
  const int i = blockIdx.x * 256 + threadIdx.x;
  int s = -1, p = 0;
  if (i < P.n_q) {
    s = P.q_stream[i];
    p = P.q_pos[i];
    if (s < 0 || s >= P.n_streams || p < 0 || p >= P.capacity) s = -1;
  }
  const unsigned same = __match_any_sync(0xffffffffu, s);
  const unsigned hi = __reduce_max_sync(same, static_cast<unsigned>(p + 1));
  const unsigned lo = __reduce_max_sync(same, static_cast<unsigned>(P.capacity - max(0, p - P.window + 1)));
  if (s >= 0 && (threadIdx.x & 31) == __ffs(same) - 1) {
    atomicMax(P.range + 2 * s, static_cast<int>(hi));
    atomicMax(P.range + 2 * s + 1, static_cast<int>(lo));
  }
  if (P.ctl == nullptr) return;
  __shared__ bool last;
  __threadfence();
  __syncthreads();
  if (threadIdx.x == 0) last = atomicAdd(P.ctl, 1) == static_cast<int>(gridDim.x) - 1;
  __syncthreads();
  if (!last) return;
  __threadfence();
  choose(P);
}

// 16 e4m3 values times `f`, as bf16.
__device__ __forceinline__ void expand16(const uint4& x, float f, uint4& a, uint4& b) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  uint32_t r[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(w[i >> 1] >> ((i & 1) * 16))));
    const float2 v = __half22float2(*reinterpret_cast<__half2*>(&h));
    r[i] = pack_bf16(v.x * f, v.y * f);
  }
  a = make_uint4(r[0], r[1], r[2], r[3]);
  b = make_uint4(r[4], r[5], r[6], r[7]);
}

// The NaN codes (0x7f, 0xff) of four e4m3 values set to zero.
__device__ __forceinline__ uint32_t without_nan(uint32_t w) {
  const uint32_t nan = ((w & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;   // bit 7 of each such byte
  return w & ~((nan >> 7) * 0xffu);
}

// CTA (stream, group, z): blocks z, z + gridDim.z, ... of those that the
// stream's queries see.
__global__ void __launch_bounds__(256) expand_kernel(const Params P) {
  pdl_trigger();
  pdl_wait();
  const int s = blockIdx.x, g = blockIdx.y;
  if (P.ctl != nullptr && __ldcg(P.ctl + 1) != kTiles) return;
  const int hi = P.range[2 * s];
  const Visible seen(P, hi, P.range[2 * s + 1]);
  const int base = P.table != nullptr ? P.base[s] : 0;
  for (int i = blockIdx.z; i < seen.n; i += gridDim.z) {
    const int b = seen.block(i);
    const long long row = kv_block_row(P.pages, s, g, b, P.G, P.capacity);
    if (P.table != nullptr && g == 0 && threadIdx.x == 0)
      P.table[static_cast<size_t>(s) * (P.capacity / 128) + b] = row < 0 ? -1 : base + i;
    if (row < 0) continue;                       // the attention kernel reports it
    const long long dst = P.table != nullptr ? (static_cast<long long>(base + i) * P.G + g) * 128 : row;
    const float ks = __ldcg(P.k_scale + row / 128), vs = __ldcg(P.v_scale + row / 128);
    const uint4* k = reinterpret_cast<const uint4*>(P.k_cache + row * 128);
    const uint4* v = reinterpret_cast<const uint4*>(P.v_cache + row * 128);
    uint4* ko = P.k_out + dst * 16;
    uint4* vo = P.v_out + dst * 16;
    uint4 x[4], y[4];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      x[c] = __ldcs(k + threadIdx.x + 256 * c);
      y[c] = __ldcs(v + threadIdx.x + 256 * c);
    }
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      // V rows past every query of the stream may hold NaN, which times a weight
      // of zero would still be NaN in the union tiles (the window tiles clear
      // what they do not see; streams that share the page write the same
      // values, but for such a NaN)
      if (P.clean && b * 128 + static_cast<int>(threadIdx.x + 256 * c) / 8 >= hi)
        y[c] = make_uint4(without_nan(y[c].x), without_nan(y[c].y), without_nan(y[c].z), without_nan(y[c].w));
      const int at = (threadIdx.x + 256 * c) * 2;
      uint4 a, d;
      expand16(x[c], ks, a, d);
      ko[at] = a;
      ko[at + 1] = d;
      expand16(y[c], vs, a, d);
      vo[at] = a;
      vo[at + 1] = d;
    }
  }
}

}  // namespace expand
}  // namespace msa
