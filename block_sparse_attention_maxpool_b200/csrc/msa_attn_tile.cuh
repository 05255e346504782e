// GQA attention of batches of many queries (prefill) on the tensor cores:
// over the last `window` slots and the first `n_sink` ones, or over selected
// blocks, read from a bf16 cache or from an e4m3 cache with one scale per
// (128-token block, group).  The mathematics is that of msa_attn_cluster.cuh.
//
// Bound by the two products (4 * 128 FLOP per query head and visible slot) and
// by the exponentials: a 128 x 128 tile of scores is 1024 cycles of MMA (S and
// P V) and 1024 cycles of the special-function units, so the aim is to keep
// both busy at once.  A CTA works on two tiles of 8 queries x 16 heads = 128
// rows, A and B, which share every K and V block it loads; while the softmax
// warps of one tile work, the tensor pipe works for the other.
//
//   S = Q K^T    M = 128 rows, N = 128 keys (tensor memory, f32)
//   P = exp2(f S - m) as bf16 pairs over S's columns, one thread per row
//   O += P V     A from tensor memory, B = V from shared memory
//
// A row's reference m is raised (and its O rescaled in tensor memory) only
// when a block's maximum passes it by more than 8 (log2 units), so rescaling
// is rare and P stays below 2^8.  The row sum adds the rounded P values.
//
// Warps: 0 plans the tile's blocks and loads K, 1 loads Q and issues S, 2 loads V,
// 3 issues P V, 4-7 and 8-11 are the softmax of A and B (a TMEM lane quarter
// each), 12-15 (e4m3) convert K and V to bf16.  The planner evaluates 32
// candidate blocks at a time, one per lane: which of the 16 queries see the
// block.  A block that some query sees becomes a record (block, 16-bit query
// mask, scales) in a ring that every role reads; a record without a query
// ends the tile.  So the other roles need no plan in global memory, tiles
// may mix streams and positions at will (queries of one stream after the
// other), and a tile's softmax skips blocks its queries do not see.
// Selected blocks are gathered through a bitmap of 512 blocks at a time.
//
// e4m3: the converters write K unscaled (its scale is a factor of the score)
// and V times its scale's power of two, both exact in bf16; what is left of
// the V scale, a factor in [1, 2), goes into P through the exponent and out
// of the row sum again.
//
// V rows of a block that no query of the tile sees become zeros (they may
// hold NaN): by the V loader after the copy landed, or while converting.
// Only blocks that no single query sees whole are looked at: the diagonal,
// the window's first block, a cut sink block.
#pragma once

#include <cuda_fp16.h>

#include "msa_attn_prefill_union.cuh"
#include "msa_common.cuh"

namespace msa {
namespace tattn {

using uattn::add_bf16x2_f32;
using uattn::cvt_bf16x2;
using uattn::ex2_approx;
using uattn::ffma2;
using uattn::fmax3;

constexpr int kD = 128;
constexpr int kBlock = 128;
constexpr int kHpg = 16;
constexpr int kTopK = 16;
constexpr int kTileQ = 16;                          // queries of a CTA's two tiles
constexpr uint32_t kHalf = 128 * 128;               // [128 rows][64 bf16]
constexpr uint32_t kTile = 2 * kHalf;
constexpr int kRing = 2;                            // K and V stages
constexpr int kRecs = 8;
constexpr int kMapBlocks = 512;
constexpr uint32_t kTmemCols = 512;                 // S_A, S_B, O_A, O_B: 128 columns each
constexpr uint32_t kOCol = 256;
constexpr uint32_t kIdescS = umma_idesc_bf16_f32(128, 128, false, false);
constexpr uint32_t kIdescPV = umma_idesc_bf16_f32(128, 128, false, true);
constexpr float kRescale = 8.f;

template <bool kF8>
struct Cfg {
  static constexpr int kThreads = kF8 ? 512 : 384;
  static constexpr int kRecReaders = kF8 ? 15 : 11;  // S, V, P V, 8 softmax warps, 4 converter warps
};

struct Rec {
  int32_t block;
  uint32_t mask;      // queries 0-7 (A) and 8-15 (B) that see the block; 0: the tile ends
  int32_t row;        // first cache row
  int32_t fix;        // some rows are seen by no query
  float ks;           // e4m3: K scale
  float v2;           // e4m3: V scale = v2 * vm, v2 +- a power of two,
  float vm;           // vm in [1, 2)
  int32_t pad;
};

template <bool kF8>
struct Layout {
  static constexpr uint32_t kQOff = 0;                                   // A, B
  static constexpr uint32_t kKOff = 2 * kTile;
  static constexpr uint32_t kVOff = kKOff + kRing * kTile;
  static constexpr uint32_t kStageOff = kVOff + kRing * kTile;           // e4m3: a K and a V block as loaded
  static constexpr uint32_t kRecOff = kStageOff + (kF8 ? 2 * kHalf : 0);
  static constexpr uint32_t kMapOff = kRecOff + kRecs * sizeof(Rec);
  static constexpr uint32_t kBarOff = kMapOff + kMapBlocks * 2;
  static constexpr uint32_t kEnd = kBarOff + 56 * 8;
  static constexpr size_t kBytes = kEnd + 1024;
};
static_assert(Layout<true>::kBytes <= 232448, "shared memory budget");

struct Params {
  const int32_t* q_stream;
  const int32_t* q_pos;
  const int32_t* sel;         // selection form: [n_q][G][16]
  const float* k_scale;
  const float* v_scale;
  __nv_bfloat16* out;         // [n_q][16 G][128]
  int n_q, G, n_streams, capacity, n_tiles;
  int window, n_sink;
  float scale_log2;
  KvPages pages;
};

struct Bars {
  uint64_t *q_full, *q_empty, *rec_full, *rec_empty, *kfull, *kempty, *vland, *vready, *vempty;
  uint64_t *s_full, *p_full, *pv_done, *o_empty, *st_full, *st_empty, *mma_done;
  uint32_t* tmem_slot;
  __device__ explicit Bars(uint8_t* base) {
    uint64_t* b = reinterpret_cast<uint64_t*>(base);
    q_full = b;
    q_empty = b + 1;
    rec_full = b + 2;              // [kRecs]
    rec_empty = rec_full + kRecs;
    kfull = rec_empty + kRecs;     // [kRing]: the bf16 K block is in shared memory
    kempty = kfull + kRing;
    vland = kempty + kRing;        // [kRing]: the V copy landed (or was converted)
    vready = vland + kRing;        // [kRing]: rows that nobody sees are zero
    vempty = vready + kRing;
    s_full = vempty + kRing;       // [2]: S of the tile is in tensor memory
    p_full = s_full + 2;           // [2]: its P is written (4 softmax warps)
    pv_done = p_full + 2;          // [2]: its P V finished
    o_empty = pv_done + 2;         // [2]: O was read (4 softmax warps)
    st_full = o_empty + 2;         // [2]: e4m3 K, V landed
    st_empty = st_full + 2;        // [2]: converted (4 warps)
    mma_done = st_empty + 2;       // [2]: the issuers' last MMAs
    tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  }
};
static_assert(2 + 2 * kRecs + 5 * kRing + 7 * 2 + 1 <= 56, "barrier slots");

// Tile t -> (group, first query); group-major, so that CTAs running at the
// same time share K and V in L2; the last queries (the longest lists of a
// causal batch) come first.
__device__ __forceinline__ void tile_coords(const Params& P, int t, int& g, int& q0) {
  g = t / P.n_tiles;
  q0 = (P.n_tiles - 1 - (t - g * P.n_tiles)) * kTileQ;
}

// Query `lane` (0 .. 15) of the tile: its position, or -1 without a valid query.
__device__ __forceinline__ int tile_query(const Params& P, int q0, int lane, int& stream, bool& bad) {
  const int qi = q0 + lane;
  stream = -1;
  bad = false;
  if (lane >= kTileQ || qi >= P.n_q) return -1;
  const int s = __ldg(P.q_stream + qi);
  const int p = __ldg(P.q_pos + qi);
  if (s < 0 || s >= P.n_streams || p < 0 || p >= P.capacity) {
    bad = true;
    return -1;
  }
  stream = s;
  return p;
}

// Row r of block b is seen by query position p.
template <bool kWin>
__device__ __forceinline__ bool sees(const Params& P, int p, int j) {
  return j <= p && (!kWin || j > p - P.window || j < P.n_sink);
}

// Whether any query of `mask` sees slot j (pos: lane q holds query q's position).
template <bool kWin>
__device__ __forceinline__ bool anyone_sees(const Params& P, uint32_t mask, int pos, int j) {
  bool any = false;
#pragma unroll
  for (int q = 0; q < kTileQ; ++q) {
    const int p = __shfl_sync(0xffffffffu, pos, q);
    any |= ((mask >> q) & 1u) != 0u && sees<kWin>(P, p, j);
  }
  return any;
}

template <bool kF8, bool kWin>
struct Planner {
  const Params& P;
  uint8_t* smem;
  const Bars& B;
  int lane;
  int rec = 0, ring = 0;       // records and K blocks so far
  bool ok = true;

  // Append the records of 32 candidates (one per lane) to the ring, and load
  // their K blocks.
  __device__ void emit(const CUtensorMap* tm_k, int block, uint32_t mask, bool whole, int s, int g) {
    int row = -1;
    float ks = 0.f, vs = 0.f;
    if (mask != 0u) {
      const long long r = kv_block_row(P.pages, s, g, block, P.G, P.capacity);
      if (r < 0) {
        raise_error(MSA_DEVERR_PAGE_RANGE);
      } else {
        row = static_cast<int>(r);
        if (kF8) {
          ks = __ldg(P.k_scale + r / kBlock);
          vs = __ldg(P.v_scale + r / kBlock);
        }
      }
    }
    uint32_t todo = __ballot_sync(0xffffffffu, row >= 0);
    while (todo != 0u && ok) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1u;
      Rec in;
      in.block = __shfl_sync(0xffffffffu, block, l);
      in.mask = __shfl_sync(0xffffffffu, mask, l);
      in.row = __shfl_sync(0xffffffffu, row, l);
      in.fix = __shfl_sync(0xffffffffu, whole ? 0 : 1, l);
      in.ks = __shfl_sync(0xffffffffu, ks, l);
      const float v = __shfl_sync(0xffffffffu, vs, l);
      const uint32_t vb = __float_as_uint(v);
      const bool normal = (vb & 0x7f800000u) != 0u && (vb & 0x7f800000u) != 0x7f800000u;
      in.v2 = normal ? __uint_as_float(vb & 0xff800000u) : v;
      in.vm = normal ? __uint_as_float((vb & 0x007fffffu) | 0x3f800000u) : 1.f;
      in.pad = 0;
      push(in);
      if (ok && lane == 0) {
        if (kF8) {
          if (ring > 0) ok = mbar_wait(&B.st_empty[0], (ring - 1) & 1);
          if (ok) {
            mbar_arrive_expect_tx(&B.st_full[0], kHalf);
            tma_load_2d(smem + Layout<kF8>::kStageOff, tm_k, 0, in.row, &B.st_full[0]);
          }
        } else {
          const int st = ring % kRing, use = ring / kRing;
          if (use > 0) ok = mbar_wait(&B.kempty[st], (use - 1) & 1);
          if (ok) {
            uint8_t* dst = smem + Layout<kF8>::kKOff + st * kTile;
            mbar_arrive_expect_tx(&B.kfull[st], kTile);
            tma_load_2d(dst, tm_k, 0, in.row, &B.kfull[st]);
            tma_load_2d(dst + kHalf, tm_k, 64, in.row, &B.kfull[st]);
          }
        }
      }
      ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
      ++ring;
    }
  }

  __device__ void push(const Rec& in) {
    if (lane == 0) {
      const int at = rec % kRecs, use = rec / kRecs;
      if (use > 0) ok = mbar_wait(&B.rec_empty[at], (use - 1) & 1);
      if (ok) {
        reinterpret_cast<Rec*>(smem + Layout<kF8>::kRecOff)[at] = in;
        mbar_arrive(&B.rec_full[at]);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    ++rec;
  }
};

// Four e4m3 values as two bf16 pairs, times `f` (exact when f is a power of two).
template <bool kScale>
__device__ __forceinline__ uint2 e4m3x4_to_bf16(uint32_t w, float f) {
  uint32_t h0, h1;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h0) : "h"(static_cast<uint16_t>(w & 0xffffu)));
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h1) : "h"(static_cast<uint16_t>(w >> 16)));
  float2 a = __half22float2(*reinterpret_cast<__half2*>(&h0));
  float2 b = __half22float2(*reinterpret_cast<__half2*>(&h1));
  if (kScale) {
    a.x *= f;
    a.y *= f;
    b.x *= f;
    b.y *= f;
  }
  return make_uint2(cvt_bf16x2(a.x, a.y), cvt_bf16x2(b.x, b.y));
}

// Row r of a staged e4m3 block to the two bf16 halves of dst.
template <bool kScale>
__device__ __forceinline__ void convert_row(const uint8_t* src, uint8_t* dst, int r, float f, bool zero) {
#pragma unroll
  for (int c = 0; c < 8; ++c) {
    uint4 x = *reinterpret_cast<const uint4*>(src + swz128(r, c));
    if (kScale && zero) x = make_uint4(0u, 0u, 0u, 0u);
    const uint2 a = e4m3x4_to_bf16<kScale>(x.x, f), b = e4m3x4_to_bf16<kScale>(x.y, f);
    const uint2 d = e4m3x4_to_bf16<kScale>(x.z, f), e = e4m3x4_to_bf16<kScale>(x.w, f);
    uint8_t* half = dst + (c >> 2) * kHalf;
    *reinterpret_cast<uint4*>(half + swz128(r, (c & 3) * 2)) = make_uint4(a.x, a.y, b.x, b.y);
    *reinterpret_cast<uint4*>(half + swz128(r, (c & 3) * 2 + 1)) = make_uint4(d.x, d.y, e.x, e.y);
  }
}

template <bool kF8, bool kWin>
__global__ void __launch_bounds__(Cfg<kF8>::kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Params P) {
  using L = Layout<kF8>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars B(smem + L::kBarOff);
  const Rec* recs = reinterpret_cast<const Rec*>(smem + L::kRecOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int n_tasks = P.G * P.n_tiles;

  if (threadIdx.x == 0) {
    mbar_init(B.q_full, 1);
    mbar_init(B.q_empty, 1);
    for (int i = 0; i < kRecs; ++i) {
      mbar_init(&B.rec_full[i], 1);
      mbar_init(&B.rec_empty[i], Cfg<kF8>::kRecReaders);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&B.kfull[i], kF8 ? 4 : 1);
      mbar_init(&B.kempty[i], 1);
      mbar_init(&B.vland[i], kF8 ? 4 : 1);
      mbar_init(&B.vready[i], 1);
      mbar_init(&B.vempty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.pv_done[i], 1);
      mbar_init(&B.o_empty[i], 4);
      mbar_init(&B.st_full[i], 1);
      mbar_init(&B.st_empty[i], 4);
      mbar_init(&B.mma_done[i], 1);
    }
    mbar_fence_init();
  }
  if (warp == 1) tmem_alloc(B.tmem_slot, kTmemCols);
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *B.tmem_slot;
  pdl_trigger();
  pdl_wait();

  // The next record (every role keeps its own count of records read).
  auto next_rec = [&](int r, Rec& in) {
    if (!mbar_wait(&B.rec_full[r % kRecs], (r / kRecs) & 1)) return false;
    in = recs[r % kRecs];
    return true;
  };
  auto done_rec = [&](int r) { mbar_arrive(&B.rec_empty[r % kRecs]); };

  // The softmax rows need registers that the other roles do not.  The shares
  // of the warpgroups add up to the launch's: 88 + 2 * 208 = 3 * 168, and
  // 72 + 2 * 184 + 72 = 4 * 128.
  if (warp < 4) {
    if constexpr (kF8) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    else asm volatile("setmaxnreg.dec.sync.aligned.u32 88;");
    if (warp == 0) {
      // ------------------------- planner and K loader -------------------------
      Planner<kF8, kWin> pl{P, smem, B, lane};
      for (int t = blockIdx.x; t < n_tasks && pl.ok; t += gridDim.x) {
        int g, q0, stream;
        bool bad;
        tile_coords(P, t, g, q0);
        const int pos = tile_query(P, q0, lane, stream, bad);
        if (bad && g == 0) raise_error(MSA_DEVERR_QUERY_RANGE);
        uint32_t left = __ballot_sync(0xffffffffu, pos >= 0);
        while (left != 0u && pl.ok) {
          // the queries of one stream
          const int s = __shfl_sync(0xffffffffu, stream, __ffs(left) - 1);
          const uint32_t seg = __ballot_sync(0xffffffffu, pos >= 0 && stream == s);
          left &= ~seg;
          const bool here = ((seg >> lane) & 1u) != 0u;
          const int pmax = static_cast<int>(__reduce_max_sync(0xffffffffu, here ? static_cast<unsigned>(pos) : 0u));
          if (kWin) {
            const int a = here ? max(0, pos - P.window + 1) : P.capacity;
            const int first = static_cast<int>(__reduce_min_sync(0xffffffffu, static_cast<unsigned>(a))) / kBlock;
            const int sinks = min((P.n_sink + kBlock - 1) / kBlock, first);
            const int n = sinks + pmax / kBlock - first + 1;
            for (int base = 0; base < n && pl.ok; base += 32) {
              const int i = base + lane;
              const int b = i < sinks ? i : first + i - sinks;
              uint32_t mask = 0u;
              bool whole = false;
  #pragma unroll
              for (int q = 0; q < kTileQ; ++q) {
                const int p = __shfl_sync(0xffffffffu, pos, q);
                const int j0 = b * kBlock, j1 = j0 + kBlock - 1;
                const bool some = ((seg >> q) & 1u) != 0u && j0 <= p && (j1 > p - P.window || j0 < P.n_sink);
                if (some) {
                  mask |= 1u << q;
                  whole |= j1 <= p && (j0 > p - P.window || j1 < P.n_sink);
                }
              }
              pl.emit(&tm_k, b, i < n ? mask : 0u, whole, s, g);
            }
          } else {
            // lane 2q + h holds entries 8h .. 8h + 7 of query q
            const int q = lane >> 1;
            const int pq = __shfl_sync(0xffffffffu, pos, q);
            const bool mine = ((seg >> q) & 1u) != 0u;
            int e[8];
  #pragma unroll
            for (int i = 0; i < 8; ++i) e[i] = -1;
            if (mine) {
              const int4* src = reinterpret_cast<const int4*>(P.sel + (static_cast<size_t>(q0 + q) * P.G + g) * kTopK) + (lane & 1) * 2;
              const int4 x = __ldg(src), y = __ldg(src + 1);
              e[0] = x.x; e[1] = x.y; e[2] = x.z; e[3] = x.w;
              e[4] = y.x; e[5] = y.y; e[6] = y.z; e[7] = y.w;
  #pragma unroll
              for (int i = 0; i < 8; ++i) {
                if (e[i] > pq / kBlock) {
                  raise_error(MSA_DEVERR_SEL_RANGE);
                  e[i] = -1;
                }
              }
            }
            uint32_t* map = reinterpret_cast<uint32_t*>(smem + L::kMapOff);
            for (int wb = 0; wb <= pmax / kBlock && pl.ok; wb += kMapBlocks) {
              for (int i = lane; i < kMapBlocks / 2; i += 32) map[i] = 0u;
              __syncwarp();
  #pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int o = e[i] - wb;
                if (e[i] >= 0 && o >= 0 && o < kMapBlocks) atomicOr(&map[o >> 1], (1u << q) << ((o & 1) * 16));
              }
              __syncwarp();
              const int n = min(kMapBlocks, pmax / kBlock + 1 - wb);
              for (int base = 0; base < n && pl.ok; base += 32) {
                const int i = base + lane, b = wb + i;
                const uint32_t mask = i < n ? (map[i >> 1] >> ((i & 1) * 16)) & 0xffffu : 0u;
                bool whole = false;
  #pragma unroll
                for (int k = 0; k < kTileQ; ++k) {
                  const int p = __shfl_sync(0xffffffffu, pos, k);
                  whole |= ((mask >> k) & 1u) != 0u && b * kBlock + kBlock - 1 <= p;
                }
                pl.emit(&tm_k, b, mask, whole, s, g);
              }
              __syncwarp();
            }
          }
        }
        if (pl.ok) pl.push(Rec{0, 0u, 0, 0, 0.f, 0.f, 1.f, 0});
      }
      // no copy may still be landing when the CTA exits
      if (lane == 0) {
        if (kF8) {
          if (pl.ring > 0) mbar_wait(&B.st_full[0], (pl.ring - 1) & 1);
        } else {
          for (int j = max(0, pl.ring - kRing); j < pl.ring; ++j) mbar_wait(&B.kfull[j % kRing], (j / kRing) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 2) {
      // --------------------------------- V loader ---------------------------------
      int r = 0, ring = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < n_tasks && ok; t += gridDim.x) {
        int g, q0, stream;
        bool bad;
        tile_coords(P, t, g, q0);
        const int pos = tile_query(P, q0, lane, stream, bad);
        for (;; ++r) {
          Rec in;
          ok = next_rec(r, in);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (in.mask == 0u) {
            __syncwarp();
            if (lane == 0) done_rec(r);
            ++r;
            break;
          }
          const int st = ring % kRing, use = ring / kRing;
          if (kF8) {
            if (lane == 0) {
              if (ring > 0) ok = mbar_wait(&B.st_empty[1], (ring - 1) & 1);
              if (ok) {
                mbar_arrive_expect_tx(&B.st_full[1], kHalf);
                tma_load_2d(smem + L::kStageOff + kHalf, &tm_v, 0, in.row, &B.st_full[1]);
              }
            }
          } else {
            uint8_t* dst = smem + L::kVOff + st * kTile;
            if (lane == 0) {
              if (use > 0) ok = mbar_wait(&B.vempty[st], (use - 1) & 1);
              if (ok) {
                mbar_arrive_expect_tx(&B.vland[st], kTile);
                tma_load_2d(dst, &tm_v, 0, in.row, &B.vland[st]);
                tma_load_2d(dst + kHalf, &tm_v, 64, in.row, &B.vland[st]);
              }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (ok && in.fix != 0) {
              ok = mbar_wait(&B.vland[st], use & 1);
              ok = __all_sync(0xffffffffu, ok);
              for (int i = 0; i < kBlock && ok; i += 32) {
                const int row = i + lane;
                if (!anyone_sees<kWin>(P, in.mask, pos, in.block * kBlock + row)) {
  #pragma unroll
                  for (int c = 0; c < 8; ++c) {
                    *reinterpret_cast<uint4*>(dst + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                    *reinterpret_cast<uint4*>(dst + kHalf + row * 128 + c * 16) = make_uint4(0u, 0u, 0u, 0u);
                  }
                }
              }
              fence_proxy_async_smem();
            }
            __syncwarp();
            if (lane == 0 && ok) mbar_arrive(&B.vready[st]);
          }
          ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
          if (!ok) break;
          ++ring;
          if (lane == 0) done_rec(r);
        }
      }
      if (lane == 0) {
        if (kF8) {
          if (ring > 0) mbar_wait(&B.st_full[1], (ring - 1) & 1);
        } else {
          for (int j = max(0, ring - kRing); j < ring; ++j) mbar_wait(&B.vland[j % kRing], (j / kRing) & 1);
        }
      }
      __syncwarp();
    } else if (warp == 1) {
      // --------------------------- S issuer: S = Q K^T (lane 0) ---------------------------
      // S and P V come from two issuing threads: the tensor pipe drains when one
      // thread switches operand configuration, not when two threads interleave.
      if (lane == 0) {
        const uint32_t q_base = smem_addr(smem + L::kQOff);
        const uint32_t k_base = smem_addr(smem + L::kKOff);
        int r = 0, ring = 0, tiles = 0, n[2] = {0, 0};
        bool ok = true;
        for (int t = blockIdx.x; t < n_tasks && ok; t += gridDim.x, ++tiles) {
          // this tile's Q, once the previous tile's S MMAs are done with theirs
          // (the planner and the other loads run ahead meanwhile)
          if (tiles > 0) ok = mbar_wait(B.q_empty, (tiles - 1) & 1);
          if (!ok) break;
          int g, q0;
          tile_coords(P, t, g, q0);
          const int nq = min(kTileQ, P.n_q - q0);
          mbar_arrive_expect_tx(B.q_full, static_cast<uint32_t>(nq) * (kHpg * kD * 2));
          for (int i = 0; i < nq; ++i) {
            const int row = (q0 + i) * (P.G * kHpg) + g * kHpg;           // q viewed as [n_q * Hq][128]
            uint8_t* dst = smem + L::kQOff + (i >> 3) * kTile + (i & 7) * (kHpg * 128);
            tma_load_2d(dst, &tm_q, 0, row, B.q_full);
            tma_load_2d(dst + kHalf, &tm_q, 64, row, B.q_full);
          }
          ok = mbar_wait(B.q_full, tiles & 1);
          tc_fence_after();
          for (; ok; ++r) {
            Rec in;
            ok = next_rec(r, in);
            if (!ok) break;
            done_rec(r);
            if (in.mask == 0u) {
              umma_commit(B.q_empty);
              ++r;
              break;
            }
            const int st = ring % kRing;
            ok = mbar_wait(&B.kfull[st], (ring / kRing) & 1);
            const uint32_t kb = k_base + st * kTile;
  #pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (((in.mask >> (8 * x)) & 0xffu) == 0u || !ok) continue;
              // the tile's previous P V is done: its S columns are free
              if (n[x] > 0) ok = mbar_wait(&B.pv_done[x], (n[x] - 1) & 1);
              if (!ok) break;
              ++n[x];
              tc_fence_after();
  #pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t off = (kk >> 2) * kHalf + (kk & 3) * 32;
                umma_f16_ss(tmem_base + x * 128, umma_desc_sw128(q_base + x * kTile + off), umma_desc_sw128(kb + off), kIdescS,
                            kk != 0);
              }
              umma_commit(&B.s_full[x]);
            }
            umma_commit(&B.kempty[st]);
            ++ring;
          }
        }
        umma_commit(&B.mma_done[0]);
        mbar_wait(&B.mma_done[0], 0);
      }
      __syncwarp();
    } else if (warp == 3) {
      // --------------------------- P V issuer: O (+)= P V (lane 0) ---------------------------
      if (lane == 0) {
        const uint32_t v_base = smem_addr(smem + L::kVOff);
        int r = 0, ring = 0, n[2] = {0, 0}, outs[2] = {0, 0};
        bool ok = true;
        for (int t = blockIdx.x; t < n_tasks && ok; t += gridDim.x) {
          bool begun[2] = {false, false};
          for (; ok; ++r) {
            Rec in;
            ok = next_rec(r, in);
            if (!ok) break;
            done_rec(r);
            if (in.mask == 0u) {
              ++r;
              break;
            }
            const int st = ring % kRing, use = ring / kRing;
            const uint32_t vb = v_base + st * kTile;
  #pragma unroll
            for (int x = 0; x < 2; ++x) {
              if (((in.mask >> (8 * x)) & 0xffu) == 0u || !ok) continue;
              ok = mbar_wait(&B.p_full[x], n[x] & 1);
              if (ok && !begun[x] && outs[x] > 0) ok = mbar_wait(&B.o_empty[x], (outs[x] - 1) & 1);
              if (ok) ok = mbar_wait(&B.vland[st], use & 1);
              if (ok && !kF8) ok = mbar_wait(&B.vready[st], use & 1);
              if (!ok) break;
              ++n[x];
              tc_fence_after();
  #pragma unroll
              for (int kk = 0; kk < 8; ++kk)
                umma_f16_ts(tmem_base + kOCol + x * 128, tmem_base + x * 128 + kk * 8, umma_desc_sw128_mn(vb + kk * 2048, kHalf),
                            kIdescPV, (!begun[x] && kk == 0) ? 0u : 1u);
              umma_commit(&B.pv_done[x]);
              if (!begun[x]) ++outs[x];
              begun[x] = true;
            }
            umma_commit(&B.vempty[st]);
            ++ring;
          }
        }
        umma_commit(&B.mma_done[1]);
        mbar_wait(&B.mma_done[1], 0);
      }
      __syncwarp();
    }
  } else if (warp < 12) {
    // ---------------- softmax and output: one thread per (query, head) row ----------------
    if constexpr (kF8) asm volatile("setmaxnreg.inc.sync.aligned.u32 184;");
    else asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    const int x = (warp - 4) >> 2;                     // tile
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;               // TMEM lane = MMA row
    const int q = x * 8 + row / kHpg;                  // query of the CTA's 16
    const uint32_t wq = 3u << (x * 8 + quarter * 2);   // this warp's two queries
    const uint32_t lane_addr = static_cast<uint32_t>(quarter * 32) << 16;
    const uint32_t sbuf = tmem_base + lane_addr + x * 128;
    const uint32_t obuf = tmem_base + lane_addr + kOCol + x * 128;
    int r = 0, n = 0;
    bool ok = true;
    for (int t = blockIdx.x; t < n_tasks && ok; t += gridDim.x) {
      int g, q0;
      tile_coords(P, t, g, q0);
      const int qi = q0 + q;
      int pq = -1;
      if (qi < P.n_q) pq = __ldg(P.q_pos + qi);
      const int aq = kWin ? pq - P.window + 1 : 0;     // first slot of the window
      float m_ref = -INFINITY, l = 0.f;
      bool begun = false;
      for (;; ++r) {
        Rec in;
        ok = next_rec(r, in);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        __syncwarp();
        if (lane == 0) done_rec(r);
        if (in.mask == 0u) {
          ++r;
          break;
        }
        if (((in.mask >> (8 * x)) & 0xffu) == 0u) continue;
        const bool mine = ((in.mask >> q) & 1u) != 0u;
        const bool active = (in.mask & wq) != 0u;
        const int j0 = in.block * kBlock;
        const int hi = mine ? pq - j0 : -1;            // columns lo .. hi and those below `sink` are visible
        const int lo = aq - j0;
        const int sink = kWin ? P.n_sink - j0 : 0;
        const bool cut = mine && (hi < kBlock - 1 || (kWin && lo > 0 && sink < min(lo, kBlock)));
        float f = kF8 ? P.scale_log2 * in.ks : P.scale_log2;
        ok = mbar_wait(&B.s_full[x], n & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++n;
        tc_fence_after();
        if (active) {
          float s[kBlock];
          {
            float v0[32], v1[32], v2[32], v3[32];
            tmem_ld32(sbuf, v0);
            tmem_ld32(sbuf + 32, v1);
            tmem_ld32(sbuf + 64, v2);
            tmem_ld32(sbuf + 96, v3);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              s[i] = v0[i];
              s[32 + i] = v1[i];
              s[64 + i] = v2[i];
              s[96 + i] = v3[i];
            }
          }
          if (f < 0.f) {                               // the maximum below is of f s
            f = -f;
#pragma unroll
            for (int c = 0; c < kBlock; ++c) s[c] = -s[c];
          }
          if (f == 0.f) f = 1.17549435e-38f;           // -inf (masked) times 0 would be NaN
          if (__any_sync(0xffffffffu, cut)) {
#pragma unroll
            for (int c = 0; c < kBlock; ++c)
              s[c] = c <= hi && (!kWin || c >= lo || c < sink) ? s[c] : -INFINITY;
          }
          // the row maximum: four chains of three-input maxima
          float m4[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmax3(s[i], s[4 + i], s[8 + i]);
#pragma unroll
          for (int c = 12; c < kBlock - 4; c += 8)
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], s[c + i], s[c + 4 + i]);
#pragma unroll
          for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], s[kBlock - 4 + i]);
          const float mb = mine ? fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * f : -INFINITY;
          const bool raise = mb > m_ref + kRescale;
          const bool rescale = raise && begun && m_ref != -INFINITY;
          if (__any_sync(0xffffffffu, rescale)) {
            // S came after the tile's previous P V, so O is at rest
            const float fo = rescale ? ex2_approx(m_ref - mb) : 1.f;
            l *= fo;
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              float v[32];
              tmem_ld32(obuf + c * 32, v);
              tmem_ld_wait();
#pragma unroll
              for (int i = 0; i < 32; ++i) v[i] *= fo;
              tmem_st32(obuf + c * 32, v);
            }
          }
          if (raise) m_ref = mb;
          float neg_m = -m_ref;
          if (kF8) neg_m += __log2f(in.vm);
          const float2 f2 = make_float2(f, f), nm2 = make_float2(neg_m, neg_m);
          float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float pk[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              const float2 y = ffma2(make_float2(s[h * 64 + 2 * i], s[h * 64 + 2 * i + 1]), f2, nm2);
              // a row whose query does not see the block keeps nothing of it
              const uint32_t pp = mine ? cvt_bf16x2(ex2_approx(y.x), ex2_approx(y.y)) : 0u;
              acc[i & 3] = add_bf16x2_f32(pp, acc[i & 3]);
              pk[i] = __uint_as_float(pp);
            }
            tmem_st32(sbuf + h * 32, pk);
          }
          const float sum = (acc[0] + acc[1]) + (acc[2] + acc[3]);
          l += kF8 ? __fdividef(sum, in.vm) : sum;
        } else {
          float z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0.f;
          tmem_st32(sbuf, z);
          tmem_st32(sbuf + 32, z);
        }
        begun = true;
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.p_full[x]);
      }
      if (!ok) break;
      __nv_bfloat16* dst = P.out + (static_cast<size_t>(qi) * (P.G * kHpg) + g * kHpg + (row % kHpg)) * kD;
      if (begun) {
        ok = mbar_wait(&B.pv_done[x], (n - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          float v[32];
          tmem_ld32(obuf + c * 32, v);
          tmem_ld_wait();
          if (qi < P.n_q) {
#pragma unroll
            for (int i = 0; i < 32; i += 8) {
              uint4 w = make_uint4(pack_bf16(v[i] * inv, v[i + 1] * inv), pack_bf16(v[i + 2] * inv, v[i + 3] * inv),
                                   pack_bf16(v[i + 4] * inv, v[i + 5] * inv), pack_bf16(v[i + 6] * inv, v[i + 7] * inv));
              if (l == 0.f) w = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(dst + c * 32 + i) = w;
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.o_empty[x]);
      } else if (qi < P.n_q) {
#pragma unroll
        for (int i = 0; i < kD; i += 8) *reinterpret_cast<uint4*>(dst + i) = make_uint4(0u, 0u, 0u, 0u);
      }
    }
  } else {
    // ----------------------------- converters (e4m3) -----------------------------
    if constexpr (kF8) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
      const int row = (warp - 12) * 32 + lane;
      int r = 0, ring = 0;
      bool ok = true;
      for (int t = blockIdx.x; t < n_tasks && ok; t += gridDim.x) {
        int g, q0, stream;
        bool bad;
        tile_coords(P, t, g, q0);
        const int pos = tile_query(P, q0, lane, stream, bad);
        for (;; ++r) {
          Rec in;
          ok = next_rec(r, in);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          __syncwarp();
          if (lane == 0) done_rec(r);
          if (in.mask == 0u) {
            ++r;
            break;
          }
          const int st = ring % kRing, use = ring / kRing;
          // K
          ok = mbar_wait(&B.st_full[0], ring & 1);
          if (ok && use > 0) ok = mbar_wait(&B.kempty[st], (use - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          convert_row<false>(smem + L::kStageOff, smem + L::kKOff + st * kTile, row, 1.f, false);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&B.st_empty[0]);
            mbar_arrive(&B.kfull[st]);
          }
          // V
          bool zero = false;
          if (in.fix != 0) zero = !anyone_sees<kWin>(P, in.mask, pos, in.block * kBlock + row);
          ok = mbar_wait(&B.st_full[1], ring & 1);
          if (ok && use > 0) ok = mbar_wait(&B.vempty[st], (use - 1) & 1);
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          convert_row<true>(smem + L::kStageOff + kHalf, smem + L::kVOff + st * kTile, row, in.v2, zero);
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) {
            mbar_arrive(&B.st_empty[1]);
            mbar_arrive(&B.vland[st]);
          }
          ++ring;
        }
      }
    }
  }
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tmem_base, kTmemCols);
  }
}

}  // namespace tattn
}  // namespace msa
