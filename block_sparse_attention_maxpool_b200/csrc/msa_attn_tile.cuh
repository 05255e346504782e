// Sliding-window GQA attention of batches of many queries (prefill) on the
// tensor cores: over the last `window` slots and the first `n_sink` ones of a
// bf16 cache.  The mathematics is that of msa_attn_cluster.cuh.
//
// Bound by the two products (4 * 128 FLOP per query head and visible slot) and
// by the exponentials: a 128 x 128 tile of scores is 1024 cycles of MMA (S and
// P V) and 1024 cycles of the special-function units, so the aim is to keep
// both busy at once.  A CTA works on two tiles of 8 queries x 16 heads = 128
// rows, A and B, which share every K and V block it loads; while the softmax
// warps of one tile work, the tensor pipe works for the other.
//
//   S = Q K^T    M = 128 rows, N = 64 keys (tensor memory, f32)
//   P = exp2(f S - m) as bf16 pairs over S's columns, one thread per row
//   O += P V     A from tensor memory, B = V from shared memory
//
// Tensor memory holds O of both tiles (128 columns each) and, per tile, two
// buffers of 64 columns: the halves of a block.  While the softmax of one half
// runs, the other half's P V and the next block's S run, so a tile's chain of
// MMA, softmax, MMA with a barrier crossing each (about 230 cycles) is hidden.
// With one buffer of 128 columns per tile, S of the next block had to wait
// for P V of the whole last one: 952 us instead of 854 us for an 8192-token
// prompt, window 4096, 64 heads, although an MMA of 64 columns costs 69 cycles
// where one of 128 costs 64 to 77 (both read the 128 rows of Q).
//
// A row's reference m is raised (and its O rescaled in tensor memory) only
// when a half's maximum passes it by more than 8 (log2 units), so rescaling
// is rare and P stays below 2^8.  The row sum adds the rounded P values.
//
// Warps: 0 plans the tile's blocks and loads K, 1 loads Q and issues S, 2
// loads V, 3 issues P V, 4-7 and 8-11 are the softmax of A and B (a TMEM lane
// quarter each).  The planner evaluates 32 candidate blocks at a time, one
// per lane: which of the 16 queries see the block.  A block that some query
// sees becomes a record (block, 16-bit query mask) in a ring that every role
// reads; a record without a query ends the tile.  So the other roles need no
// plan in global memory, tiles may mix streams and positions at will (the
// queries of one stream after the other), and a tile's softmax skips blocks
// that its queries do not see.
//
// V rows of a block that no query of the tile sees become zeros (they may
// hold NaN) once their copy has landed.  Only blocks that no single query
// sees whole are looked at: the diagonal, the window's first block, a cut
// sink block.
//
// Hot code is kept short and the rare paths (a masked block, a raised
// reference) out of line: with twelve warps in five roles the instruction
// cache decides.  With the rare paths inside loops unrolled over 128 columns
// the same prompt took 1.37 ms.  Measured for it now: 0.76 ms in a single replay,
// 1.08 PFLOP/s of visible products (0.66 of cuBLAS's measured burst); back to
// back, at the card's power limit, 0.89 ms (0.57).  Per block (both tiles)
// the S issuer spends about 2150 cycles issuing and the P V issuer 900, so the
// tensor pipe is what the loop comes closest to; exponentials take about 1750
// of a softmax warp's 3600.  Measured and not kept: every fourth exponential on
// the FMA pipes (no change), the two tiles taking turns at the special-
// function units (slower by a quarter), P through shared memory (slower by a
// tenth), reading the next record ahead (no change).
#pragma once

#include "msa_attn_prefill_union.cuh"
#include "msa_common.cuh"

namespace msa {
namespace tattn {

using uattn::cvt_bf16x2;
using uattn::ex2_approx;
using uattn::ffma2;
using uattn::fmax3;

constexpr int kD = 128;
constexpr int kBlock = 128;
constexpr int kHpg = 16;
constexpr int kTileQ = 16;                          // queries of a CTA's two tiles
constexpr uint32_t kHalf = 128 * 128;               // [128 rows][64 bf16]
constexpr uint32_t kTile = 2 * kHalf;
constexpr int kRing = 2;                            // K and V stages
constexpr int kRecs = 8;
constexpr uint32_t kTmemCols = 512;                 // S_A, S_B, O_A, O_B: 128 columns each
constexpr uint32_t kOCol = 256;
constexpr int kPart = 64;                           // keys whose P is handed over at once
constexpr int kParts = kBlock / kPart;
constexpr uint32_t kIdescS = umma_idesc_bf16_f32(128, kPart, false, false);
constexpr uint32_t kIdescPV = umma_idesc_bf16_f32(128, 128, false, true);
constexpr float kRescale = 8.f;

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.u32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0u;
}

constexpr int kThreads = 12 * 32;
constexpr int kRecReaders = 11;                     // S, V and P V warps, 8 softmax warps

struct Rec {
  int32_t block;
  uint32_t mask;      // queries 0-7 (A) and 8-15 (B) that see the block; 0: the tile ends
  int32_t row;        // first cache row
  int32_t fix;        // 0: a query sees every row; else some row may be seen by none (kFix*)
  int32_t lo, hi;     // kFixRange: rows lo .. hi are seen, and those below the sinks' end
  int32_t pad[2];
};
constexpr int32_t kFixRange = 1;   // the queries' windows overlap
constexpr int32_t kFixExact = 2;   // they may leave gaps: every row is checked against every query

struct Layout {
  static constexpr uint32_t kQOff = 0;                                   // A, B
  static constexpr uint32_t kKOff = 2 * kTile;
  static constexpr uint32_t kVOff = kKOff + kRing * kTile;
  static constexpr uint32_t kOutOff = kVOff + kRing * kTile;             // 32 rows x 64 dims per softmax warp
  static constexpr uint32_t kRecOff = kOutOff + 8 * 32 * 128;
  static constexpr uint32_t kBarOff = kRecOff + kRecs * sizeof(Rec);
  static constexpr uint32_t kEnd = kBarOff + 48 * 8;
  static constexpr size_t kBytes = kEnd + 1024;
};
static_assert(Layout::kBytes <= 232448, "shared memory budget");

struct Params {
  const int32_t* q_stream;
  const int32_t* q_pos;
  __nv_bfloat16* out;         // [n_q][16 G][128]
  int n_q, G, n_streams, capacity, n_tiles;
  int window, n_sink;
  float scale_log2;
  KvPages pages;
  Gate gate;
};

struct Bars {
  uint64_t *q_full, *q_empty, *rec_full, *rec_empty, *kfull, *kempty, *vland, *vready, *vempty;
  uint64_t *s_full, *p_full, *pv_done, *o_empty, *mma_done;
  uint32_t* tmem_slot;
  __device__ explicit Bars(uint8_t* base) {
    uint64_t* b = reinterpret_cast<uint64_t*>(base);
    q_full = b;
    q_empty = b + 1;
    rec_full = b + 2;              // [kRecs]
    rec_empty = rec_full + kRecs;
    kfull = rec_empty + kRecs;     // [kRing]: the bf16 K block is in shared memory
    kempty = kfull + kRing;
    vland = kempty + kRing;        // [kRing]: the V copy landed
    vready = vland + kRing;        // [kRing]: rows that nobody sees are zero
    vempty = vready + kRing;
    s_full = vempty + kRing;       // [2 * 2]: S of the (tile, half block) is in tensor memory
    p_full = s_full + 4;           // [2 * 2]: its P is written (4 softmax warps)
    pv_done = p_full + 4;          // [2 * 2]: its P V finished
    o_empty = pv_done + 4;         // [2]: O was read (4 softmax warps)
    mma_done = o_empty + 2;        // [2]: the issuers' last MMAs
    tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 2);
  }
};
static_assert(2 + 2 * kRecs + 5 * kRing + 3 * 4 + 2 * 2 + 1 <= 48, "barrier slots");

// Task t -> (group, first query).  The last queries (the longest lists of a
// causal batch) come first, the groups of a tile next to each other, and
// every other round of tasks runs over the CTAs backwards, so that the sums
// of the CTAs' tasks come out even (the busiest CTA of an 8192-token prompt
// had 14 % more than the average in plain group-major order).
__device__ __forceinline__ void tile_coords(const Params& P, int t, int& g, int& q0) {
  const int tile = t / P.G;
  g = t - tile * P.G;
  q0 = (P.n_tiles - 1 - tile) * kTileQ;
}
__device__ __forceinline__ int task_at(int k) {
  const int c = (k & 1) != 0 ? static_cast<int>(gridDim.x - 1 - blockIdx.x) : static_cast<int>(blockIdx.x);
  return k * static_cast<int>(gridDim.x) + c;
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

// Store 16 consecutive fp32 columns of this thread's TMEM lane.
__device__ __forceinline__ void tmem_st16(uint32_t taddr, const float (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(__float_as_uint(v[0])), "r"(__float_as_uint(v[1])), "r"(__float_as_uint(v[2])),
      "r"(__float_as_uint(v[3])), "r"(__float_as_uint(v[4])), "r"(__float_as_uint(v[5])),
      "r"(__float_as_uint(v[6])), "r"(__float_as_uint(v[7])), "r"(__float_as_uint(v[8])),
      "r"(__float_as_uint(v[9])), "r"(__float_as_uint(v[10])), "r"(__float_as_uint(v[11])),
      "r"(__float_as_uint(v[12])), "r"(__float_as_uint(v[13])), "r"(__float_as_uint(v[14])),
      "r"(__float_as_uint(v[15]))
      : "memory");
}

// Columns c0 .. c0 + 63 of a row: those outside lo .. hi and not below `sink`
// become -inf.
__device__ __forceinline__ void mask_part(float (&v)[kPart], int c0, int lo, int hi, int sink) {
  const auto below = [](int n) {                       // bits 0 .. n - 1
    return n <= 0 ? 0ull : (n >= 64 ? ~0ull : (1ull << n) - 1ull);
  };
  const unsigned long long seen = below(hi + 1 - c0) & (~below(lo - c0) | below(sink - c0));
  const uint32_t w[2] = {static_cast<uint32_t>(seen), static_cast<uint32_t>(seen >> 32)};
#pragma unroll
  for (int c = 0; c < kPart; ++c) v[c] = (w[c >> 5] & (1u << (c & 31))) != 0u ? v[c] : -INFINITY;
}

// Slot j is seen by query position p.
__device__ __forceinline__ bool sees(const Params& P, int p, int j) {
  return j <= p && (j > p - P.window || j < P.n_sink);
}

// Whether any query of `mask` sees slot j (pos: lane q holds query q's position).
__device__ __forceinline__ bool anyone_sees(const Params& P, uint32_t mask, int pos, int j) {
  bool any = false;
#pragma unroll
  for (int q = 0; q < kTileQ; ++q) {
    const int p = __shfl_sync(0xffffffffu, pos, q);
    any |= ((mask >> q) & 1u) != 0u && sees(P, p, j);
  }
  return any;
}

struct Planner {
  const Params& P;
  uint8_t* smem;
  const Bars& B;
  int lane;
  int rec = 0, ring = 0;       // records and K blocks so far
  bool ok = true;

  // Append the records of 32 candidates (one per lane) to the ring, and load
  // their K blocks.
  __device__ void emit(const CUtensorMap* tm_k, int block, uint32_t mask, bool whole, int pmin, int pmax, int s,
                       int g) {
    int row = -1;
    if (mask != 0u) {
      row = static_cast<int>(kv_block_row(P.pages, s, g, block, P.G, P.capacity));
      if (row < 0) raise_error(MSA_DEVERR_PAGE_RANGE);
    }
    uint32_t todo = __ballot_sync(0xffffffffu, row >= 0);
    while (todo != 0u && ok) {
      const int l = __ffs(todo) - 1;
      todo &= todo - 1u;
      Rec in;
      in.block = __shfl_sync(0xffffffffu, block, l);
      in.mask = __shfl_sync(0xffffffffu, mask, l);
      in.row = __shfl_sync(0xffffffffu, row, l);
      // pmin, pmax: the positions of all of the stream's queries in the tile
      in.fix = __shfl_sync(0xffffffffu, whole ? 0 : (pmax - pmin < P.window ? kFixRange : kFixExact), l);
      in.lo = pmin - P.window + 1 - in.block * kBlock;
      in.hi = pmax - in.block * kBlock;
      in.pad[0] = in.pad[1] = 0;
      push(in);
      if (ok && lane == 0) {
        const int st = ring % kRing, use = ring / kRing;
        if (use > 0) ok = mbar_wait(&B.kempty[st], (use - 1) & 1);
        if (ok) {
          uint8_t* dst = smem + Layout::kKOff + st * kTile;
          mbar_arrive_expect_tx(&B.kfull[st], kTile);
          tma_load_2d(dst, tm_k, 0, in.row, &B.kfull[st]);
          tma_load_2d(dst + kHalf, tm_k, 64, in.row, &B.kfull[st]);
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
        reinterpret_cast<Rec*>(smem + Layout::kRecOff)[at] = in;
        mbar_arrive(&B.rec_full[at]);
      }
    }
    ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
    ++rec;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
    attn_tile_kernel(const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const Params P) {
  using L = Layout;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const Bars B(smem + L::kBarOff);
  const Rec* recs = reinterpret_cast<const Rec*>(smem + L::kRecOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(B.q_full, 1);
    mbar_init(B.q_empty, 1);
    for (int i = 0; i < kRecs; ++i) {
      mbar_init(&B.rec_full[i], 1);
      mbar_init(&B.rec_empty[i], kRecReaders);
    }
    for (int i = 0; i < kRing; ++i) {
      mbar_init(&B.kfull[i], 1);
      mbar_init(&B.kempty[i], 1);
      mbar_init(&B.vland[i], 1);
      mbar_init(&B.vready[i], 1);
      mbar_init(&B.vempty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&B.s_full[i], 1);
      mbar_init(&B.p_full[i], 4);
      mbar_init(&B.pv_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&B.o_empty[i], 4);
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
  const int n_tasks = gate_open(P.gate) ? P.G * P.n_tiles : 0;

  // The next record (every role keeps its own count of records read).
  auto next_rec = [&](int r, Rec& in) {
    if (!mbar_wait(&B.rec_full[r % kRecs], (r / kRecs) & 1)) return false;
    in = recs[r % kRecs];
    return true;
  };
  auto done_rec = [&](int r) { mbar_arrive(&B.rec_empty[r % kRecs]); };

  if (warp < 4) {
    if (warp == 0) {
      // ------------------------- planner and K loader -------------------------
      Planner pl{P, smem, B, lane};
      for (int k = 0, t = task_at(0); t < n_tasks && pl.ok; t = task_at(++k)) {
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
          const int pmin = static_cast<int>(__reduce_min_sync(0xffffffffu, here ? static_cast<unsigned>(pos) : 0x7fffffffu));
          const int first = max(0, pmin - P.window + 1) / kBlock;
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
            pl.emit(&tm_k, b, i < n ? mask : 0u, whole, pmin, pmax, s, g);
          }
        }
        if (pl.ok) pl.push(Rec{0, 0u, 0, 0, 0, 0, {0, 0}});
      }
      // no copy may still be landing when the CTA exits
      if (lane == 0) {
        for (int j = max(0, pl.ring - kRing); j < pl.ring; ++j) mbar_wait(&B.kfull[j % kRing], (j / kRing) & 1);
      }
      __syncwarp();
    } else if (warp == 2) {
      // --------------------------------- V loader ---------------------------------
      // A block whose rows are not all seen is finished (its unseen rows set to
      // zero) after the next block's copy has been issued.
      int r = 0, ring = 0;
      bool ok = true;
      Rec todo{0, 0u, 0, 0, 0, 0, {0, 0}};
      int todo_ring = -1;
      for (int k = 0, t = task_at(0); t < n_tasks && ok; t = task_at(++k)) {
        int g, q0, stream;
        bool bad;
        tile_coords(P, t, g, q0);
        const int pos = tile_query(P, q0, lane, stream, bad);
        auto finish = [&]() {
          if (todo_ring < 0) return;
          const int st = todo_ring % kRing;
          uint8_t* dst = smem + L::kVOff + st * kTile;
          ok = __all_sync(0xffffffffu, mbar_wait(&B.vland[st], (todo_ring / kRing) & 1));
#pragma unroll 1
          for (int i = 0; i < kBlock && ok; i += 32) {
            const int row = i + lane;
            const bool seen = todo.fix == kFixRange
                                  ? row <= todo.hi && (row >= todo.lo || todo.block * kBlock + row < P.n_sink)
                                  : anyone_sees(P, todo.mask, pos, todo.block * kBlock + row);
            if (!seen) {
#pragma unroll
              for (int c = 0; c < 8; ++c) {
                const int at = row * 128 + (c ^ (lane & 7)) * 16;      // (eight lanes, eight bank groups)
                *reinterpret_cast<uint4*>(dst + at) = make_uint4(0u, 0u, 0u, 0u);
                *reinterpret_cast<uint4*>(dst + kHalf + at) = make_uint4(0u, 0u, 0u, 0u);
              }
            }
          }
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0 && ok) mbar_arrive(&B.vready[st]);
          todo_ring = -1;
        };
        for (;; ++r) {
          Rec in;
          ok = __all_sync(0xffffffffu, next_rec(r, in));
          if (!ok) break;
          if (in.mask != 0u) {
            const int st = ring % kRing, use = ring / kRing;
            if (lane == 0) {
              if (use > 0) ok = mbar_wait(&B.vempty[st], (use - 1) & 1);
              if (ok) {
                uint8_t* dst = smem + L::kVOff + st * kTile;
                mbar_arrive_expect_tx(&B.vland[st], kTile);
                tma_load_2d(dst, &tm_v, 0, in.row, &B.vland[st]);
                tma_load_2d(dst + kHalf, &tm_v, 64, in.row, &B.vland[st]);
                if (in.fix == 0) mbar_arrive(&B.vready[st]);
              }
            }
            ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
            if (!ok) break;
          }
          finish();
          if (!ok) break;
          __syncwarp();
          if (lane == 0) done_rec(r);
          if (in.mask == 0u) {
            ++r;
            break;
          }
          if (in.fix != 0) {
            todo = in;
            todo_ring = ring;
          }
          ++ring;
        }
      }
      if (lane == 0)
        for (int j = max(0, ring - kRing); j < ring; ++j) mbar_wait(&B.vland[j % kRing], (j / kRing) & 1);
      __syncwarp();
    } else if (warp == 1) {
      // ------------------- Q loads and the S issuer: S = Q K^T -------------------
      // S and P V come from two issuing threads: the tensor pipe drains when one
      // thread switches operand configuration, not when two threads interleave.
      // The whole warp walks the loop in step (barriers, counters and
      // descriptors stay uniform), one lane issues.
      const uint64_t q_desc = umma_desc_sw128(smem_addr(smem + L::kQOff));
      const uint64_t k_desc = umma_desc_sw128(smem_addr(smem + L::kKOff));
      // a negative score factor: the MMA negates q (bit 13 of the descriptor)
      const uint32_t idesc = kIdescS | (P.scale_log2 < 0.f ? 1u << 13 : 0u);
      int r = 0, ring = 0, tiles = 0, n0 = 0, n1 = 0;
      bool ok = true;
      for (int k = 0, t = task_at(0); t < n_tasks && ok; t = task_at(++k), ++tiles) {
        // this tile's Q, once the previous tile's S MMAs are done with theirs
        // (the planner and the other loads run ahead meanwhile)
        if (tiles > 0) ok = __all_sync(0xffffffffu, mbar_wait(B.q_empty, (tiles - 1) & 1));
        if (!ok) break;
        int g, q0;
        tile_coords(P, t, g, q0);
        const int nq = min(kTileQ, P.n_q - q0);
        if (lane == 0) mbar_arrive_expect_tx(B.q_full, static_cast<uint32_t>(nq) * (kHpg * kD * 2));
        __syncwarp();
        if (lane < nq) {
          const int row = (q0 + lane) * (P.G * kHpg) + g * kHpg;        // q viewed as [n_q * Hq][128]
          uint8_t* dst = smem + L::kQOff + (lane >> 3) * kTile + (lane & 7) * (kHpg * 128);
          tma_load_2d(dst, &tm_q, 0, row, B.q_full);
          tma_load_2d(dst + kHalf, &tm_q, 64, row, B.q_full);
        }
        __syncwarp();
        ok = __all_sync(0xffffffffu, mbar_wait(B.q_full, tiles & 1));
        for (; ok; ++r) {
          ok = __all_sync(0xffffffffu, mbar_wait(&B.rec_full[r % kRecs], (r / kRecs) & 1));
          if (!ok) break;
          const uint32_t mask = __shfl_sync(0xffffffffu, recs[r % kRecs].mask, 0);
          if (elect_one()) {
            done_rec(r);
            if (mask == 0u) umma_commit(B.q_empty);
          }
          if (mask == 0u) {
            ++r;
            break;
          }
          const int st = ring % kRing;
          ok = __all_sync(0xffffffffu, mbar_wait(&B.kfull[st], (ring / kRing) & 1));
          const uint64_t kd = k_desc + static_cast<uint64_t>(st) * (kTile >> 4);
#pragma unroll 1
          for (int i = 0; i < 2 * kParts; ++i) {
            const int h = i >> 1, x = i & 1;
            const int n = x == 0 ? n0 : n1;
            if (((mask >> (8 * x)) & 0xffu) == 0u || !ok) continue;
            // the half's previous P V is done: its S columns are free
            if (n > 0) ok = __all_sync(0xffffffffu, mbar_wait(&B.pv_done[2 * x + h], (n - 1) & 1));
            tc_fence_after();
            if (elect_one()) {
              const uint64_t qd = q_desc + x * (kTile >> 4), kh = kd + h * kPart * 8;
              const uint32_t d = tmem_base + x * 128 + h * kPart;
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint64_t off = ((kk >> 2) * kHalf + (kk & 3) * 32) >> 4;
                umma_f16_ss(d, qd + off, kh + off, idesc, kk != 0);
              }
              umma_commit(&B.s_full[2 * x + h]);
            }
          }
          n0 += (mask & 0xffu) != 0u ? 1 : 0;
          n1 += (mask >> 8) != 0u ? 1 : 0;
          if (elect_one()) umma_commit(&B.kempty[st]);
          ++ring;
        }
      }
      if (elect_one()) umma_commit(&B.mma_done[0]);
      mbar_wait(&B.mma_done[0], 0);
      __syncwarp();
    } else if (warp == 3) {
      // -------------------------- P V issuer: O (+)= P V --------------------------
      const uint64_t v_desc = umma_desc_sw128_mn(smem_addr(smem + L::kVOff), kHalf);
      int r = 0, ring = 0, n0 = 0, n1 = 0, outs0 = 0, outs1 = 0;
      bool ok = true;
      for (int k = 0, t = task_at(0); t < n_tasks && ok; t = task_at(++k)) {
        uint32_t begun = 0u;                               // bit x: the tile has its first P V
        for (; ok; ++r) {
          ok = __all_sync(0xffffffffu, mbar_wait(&B.rec_full[r % kRecs], (r / kRecs) & 1));
          if (!ok) break;
          const uint32_t mask = __shfl_sync(0xffffffffu, recs[r % kRecs].mask, 0);
          if (elect_one()) done_rec(r);
          if (mask == 0u) {
            ++r;
            break;
          }
          const int st = ring % kRing, use = ring / kRing;
          const uint64_t vd = v_desc + static_cast<uint64_t>(st) * (kTile >> 4);
          ok = __all_sync(0xffffffffu, mbar_wait(&B.vland[st], use & 1));
          if (ok) ok = __all_sync(0xffffffffu, mbar_wait(&B.vready[st], use & 1));
#pragma unroll 1
          for (int i = 0; i < 2 * kParts; ++i) {
            const int h = i >> 1, x = i & 1;
            const int n = x == 0 ? n0 : n1, outs = x == 0 ? outs0 : outs1;
            if (((mask >> (8 * x)) & 0xffu) == 0u || !ok) continue;
            const bool first = ((begun >> x) & 1u) == 0u;
            ok = __all_sync(0xffffffffu, mbar_wait(&B.p_full[2 * x + h], n & 1));
            if (ok && first && outs > 0) ok = __all_sync(0xffffffffu, mbar_wait(&B.o_empty[x], (outs - 1) & 1));
            tc_fence_after();
            if (elect_one()) {
              // P: bf16 pairs over the first half of the half's columns
              const uint32_t d = tmem_base + kOCol + x * 128, pa = tmem_base + x * 128 + h * kPart;
              const uint64_t vh = vd + h * (kPart / 16) * (2048 >> 4);
#pragma unroll
              for (int kk = 0; kk < kPart / 16; ++kk)
                umma_f16_ts(d, pa + kk * 8, vh + kk * (2048 >> 4), kIdescPV, kk == 0 && first ? 0u : 1u);
              umma_commit(&B.pv_done[2 * x + h]);
            }
            if (first) {
              if (x == 0) ++outs0;
              else ++outs1;
            }
            begun |= 1u << x;
          }
          n0 += (mask & 0xffu) != 0u ? 1 : 0;
          n1 += (mask >> 8) != 0u ? 1 : 0;
          if (elect_one()) umma_commit(&B.vempty[st]);
          ++ring;
        }
      }
      if (elect_one()) umma_commit(&B.mma_done[1]);
      mbar_wait(&B.mma_done[1], 0);
      __syncwarp();
    }
  } else if (warp < 12) {
    // ---------------- softmax and output: one thread per (query, head) row ----------------
    // the S issuer negates q where the factor is negative; -inf (masked) times
    // a zero factor would be NaN
    const float f = fmaxf(fabsf(P.scale_log2), 1.17549435e-38f);
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
    for (int k = 0, t = task_at(0); t < n_tasks && ok; t = task_at(++k)) {
      int g, q0;
      tile_coords(P, t, g, q0);
      const int qi = q0 + q;
      int pq = -1;
      if (qi < P.n_q) pq = __ldg(P.q_pos + qi);
      const int aq = pq - P.window + 1;                // first slot of the window
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
        const int sink = P.n_sink - j0;
        const bool cut = mine && (hi < kBlock - 1 || (lo > 0 && sink < min(lo, kBlock)));
        const bool any_cut = __any_sync(0xffffffffu, cut);
#pragma unroll 1
        for (int h = 0; h < kParts; ++h) {
          ok = __all_sync(0xffffffffu, mbar_wait(&B.s_full[2 * x + h], n & 1));
          if (!ok) break;
          tc_fence_after();
          const uint32_t sb = sbuf + h * kPart;
          if (active) {
            float s[kPart];
            tmem_ld64(sb, s);
            tmem_ld_wait();
            if (__builtin_expect(any_cut, 0)) mask_part(s, h * kPart, lo, hi, sink);
            // the row maximum: four chains of three-input maxima
            float m4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmax3(s[i], s[4 + i], s[8 + i]);
#pragma unroll
            for (int c = 12; c < kPart - 4; c += 8)
#pragma unroll
              for (int i = 0; i < 4; ++i) m4[i] = fmax3(m4[i], s[c + i], s[c + 4 + i]);
#pragma unroll
            for (int i = 0; i < 4; ++i) m4[i] = fmaxf(m4[i], s[kPart - 4 + i]);
            const float mb = mine ? fmaxf(fmax3(m4[0], m4[1], m4[2]), m4[3]) * f : -INFINITY;
            const bool raise = mb > m_ref + kRescale;
            const bool rescale = raise && begun && m_ref != -INFINITY;
            if (__builtin_expect(__any_sync(0xffffffffu, rescale), 0)) {
              // O is at rest once the P V of the half before has finished
              const int before = h == 0 ? n - 1 : n;   // count of that half's earlier steps
              ok = __all_sync(0xffffffffu, mbar_wait(&B.pv_done[2 * x + (h ^ 1)], before & 1));
              if (!ok) break;
              tc_fence_after();
              const float fo = rescale ? ex2_approx(m_ref - mb) : 1.f;
              l *= fo;
#pragma unroll 1
              for (int c = 0; c < 8; ++c) {
                float v[16];
                tmem_ld16(obuf + c * 16, v);
                tmem_ld_wait();
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] *= fo;
                tmem_st16(obuf + c * 16, v);
              }
            }
            if (raise) m_ref = mb;
            const float neg_m = m_ref == -INFINITY ? 0.f : -m_ref;       // nothing visible yet
            const float2 f2 = make_float2(f, f), nm2 = make_float2(neg_m, neg_m);
            // (the row sum adds the rounded values, two at a time)
            const float2 one2 = make_float2(1.f, 1.f);
            float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
            float pk[kPart / 2];
#pragma unroll
            for (int i = 0; i < kPart / 2; ++i) {
              const float2 y = ffma2(make_float2(s[2 * i], s[2 * i + 1]), f2, nm2);
              // a row whose query does not see the block keeps nothing of it
              const uint32_t pp = mine ? cvt_bf16x2(ex2_approx(y.x), ex2_approx(y.y)) : 0u;
              acc[i & 1] = ffma2(make_float2(__uint_as_float(pp << 16), __uint_as_float(pp & 0xffff0000u)), one2, acc[i & 1]);
              pk[i] = __uint_as_float(pp);
            }
            tmem_st32(sb, pk);
            l += (acc[0].x + acc[0].y) + (acc[1].x + acc[1].y);
          } else {
            float z[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) z[i] = 0.f;
            tmem_st16(sb, z);
            tmem_st16(sb + 16, z);
          }
          begun = true;
          tmem_st_wait();
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&B.p_full[2 * x + h]);
        }
        if (!ok) break;
        ++n;
      }
      if (!ok) break;
      __nv_bfloat16* dst = P.out + (static_cast<size_t>(qi) * (P.G * kHpg) + g * kHpg + (row % kHpg)) * kD;
      if (begun) {
        ok = mbar_wait(&B.pv_done[2 * x + kParts - 1], (n - 1) & 1);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        const float inv = l != 0.f ? 1.f / l : 0.f;
        // through shared memory, 64 dims at a time, so that a store covers whole
        // 128-byte lines (a row per lane took 2 us more a task)
        uint8_t* stage = smem + L::kOutOff + (warp - 4) * (32 * 128);
#pragma unroll 1
        for (int half = 0; half < 2; ++half) {
#pragma unroll 1
          for (int c = 0; c < 2; ++c) {
            float v[32];
            tmem_ld32(obuf + half * 64 + c * 32, v);
            tmem_ld_wait();
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              uint4 w = make_uint4(pack_bf16(v[8 * i] * inv, v[8 * i + 1] * inv), pack_bf16(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                                   pack_bf16(v[8 * i + 4] * inv, v[8 * i + 5] * inv), pack_bf16(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
              if (l == 0.f) w = make_uint4(0u, 0u, 0u, 0u);
              *reinterpret_cast<uint4*>(stage + swz128(lane, c * 4 + i)) = w;
            }
          }
          __syncwarp();
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int rr = i * 4 + (lane >> 3);        // row of the warp's 32
            const int qr = q0 + x * 8 + quarter * 2 + rr / kHpg;
            const uint4 w = *reinterpret_cast<const uint4*>(stage + swz128(rr, lane & 7));
            if (qr < P.n_q)
              *reinterpret_cast<uint4*>(P.out + (static_cast<size_t>(qr) * (P.G * kHpg) + g * kHpg + rr % kHpg) * kD + half * 64 +
                                        (lane & 7) * 8) = w;
          }
          __syncwarp();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&B.o_empty[x]);
      } else if (qi < P.n_q) {
#pragma unroll
        for (int i = 0; i < kD; i += 8) *reinterpret_cast<uint4*>(dst + i) = make_uint4(0u, 0u, 0u, 0u);
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
