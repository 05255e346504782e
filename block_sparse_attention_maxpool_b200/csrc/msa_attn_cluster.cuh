// GQA attention of single queries, a thread-block cluster per (query, group):
// over the last `window` tokens and the first `n_sink` ones, or over selected
// blocks, read from a bf16 cache or from an e4m3 cache with one scale per
// (128-token block, group).
//
//   out = sum_j p_j v_j / sum_j p_j,  p_j = exp2(c q . k_j - m),
//   c = softmax_scale * log2 e, m the largest exponent, j over the visible
//   slots: j <= p and (j > p - window or j < n_sink), or j <= p in the
//   selected blocks.
//
// Bound by the K and V bytes of the visible rows.  A pair's rows are cut into
// units (64 bf16 or 128 e4m3 rows of one block: 32 KB of K and V) and the
// units into equal shares, one per CTA of the pair's cluster (1 to 16 CTAs,
// chosen by the host so that the grid fills the SMs).  A CTA streams its
// share through a three-stage TMA ring; two CTAs fit an SM, so one's prologue
// and merge overlap the other's loads.  Four consumer warps take a quarter of
// a unit's rows each, with the 16 heads as the rows of an m16n8k16 MMA, and
// keep their own running maximum, sum and O in registers; the four are merged
// in shared memory and the CTAs of a cluster through distributed shared
// memory, each CTA writing a slice of the output.  So nothing goes through
// global memory between CTAs: no workspace, no flags, no order of arrival,
// the same result every time.
//
// O and the sum of the p have references (the exponent that counts as 2^0)
// that are raised only when a unit passes them by a few powers of two, so O
// is hardly ever rescaled.
//
// e4m3 rows: K and V values are converted exactly to fp16, and the MMAs take
// fp16.  q keeps its 8 significant bits in fp16 after a power-of-two scaling
// of each head's row to a largest magnitude in [2^14, 2^15) (elements more
// than 2^29 below it lose bits); the block's K scale, the head's scaling and
// c are one float32 factor of the score.  The V scale joins the exponent: p vs
// is what O adds up, rounded to fp16 (11 bits, normal down to 2^-24 of the
// reference) with a reference of its own, which follows the largest p vs; the
// p are summed in float32, unrounded.  bf16 rows: p is rounded to bf16, the
// row sum adds the rounded values.
//
// Measured: bf16, 32 queries x 4 groups, window 4096 in shuffled pages: 49.7
// us, 5.4 TB/s (0.83 of the measured copy rate).  e4m3: window 32768, 8
// queries x 4 groups: 58 us, 4.6 TB/s; 16 selected blocks, 32 queries x 4
// groups: 21.8 us, 3.1 TB/s.  Loads, start and merge alone take 82 to 88 % of
// those two; with thousands of pairs the units' arithmetic is the larger part
// (about 1460 SM cycles per e4m3 unit, bound by dependent latencies with eight
// consumer warps per SM: 128 conversions, 64 MMAs and 32 byte regroupings per
// warp).  Three CTAs per SM (two stages, 128
// registers) took 6 % less on thousands of pairs and 8 % more on a decode
// batch; eight warps of 16 rows per CTA took 40 % more; clusters of 9 or 13
// CTAs, which would spread 32 pairs evenly over 148 SMs, took 1.4 times as long
// as 8 (they do not pack into the GPCs), so the size is a power of two.  With
// the products on tcgen05 (a block's 128 rows as M, the heads' q in two e4m3
// and p in four e5m2 pieces as N) 2048 queries took 870 us instead of 710 and a
// decode call 2 us more; the tensor core also aligned the tiny weights beside
// a dominating one to it where the latter's V is zero.
//
// ldmatrix moves 16-bit pairs, so on e4m3 tiles it hands a thread four
// consecutive dims of a K row, or two dims of two V rows.  The MMA's k index
// of the scores is only summed over, so K's dims 4t .. 4t + 3 serve as k =
// 2t, 2t + 1, 2t + 8, 2t + 9 and q is loaded in the same order; for V the
// byte pairs are regrouped so that one n tile holds the even and the next the
// odd dims of 16.
//
// Rows a mask cuts off inside a unit: their scores become -inf, and their V
// values 0 (a cache may hold anything there, NaN included).
#pragma once

#include <cuda_fp16.h>

#include "msa_common.cuh"

namespace msa {
namespace cattn {

constexpr int kD = 128;
constexpr int kBlock = 128;
constexpr int kHpg = 16;
constexpr int kTopK = 16;
constexpr int kWarps = 4;                        // consumer warps
constexpr int kThreads = (kWarps + 1) * 32;      // and the producer warp
constexpr uint32_t kStageBytes = 32768;          // K and V of one unit
constexpr uint32_t kHalfStage = kStageBytes / 2;
constexpr int kMaxCluster = 16;
constexpr int kOStride = kD + 4;                 // padded row of the merge buffer

template <bool kF8>
struct Unit {
  static constexpr int kRows = kF8 ? 128 : 64;
  static constexpr int kWarpRows = kRows / kWarps;
  static constexpr int kStages = 3;
  static constexpr int kCtas = 2;     // CTAs per SM
};

// What the producer tells the consumers about the unit in a stage.
struct UnitInfo {
  int32_t data;       // the unit's rows landed (else nothing to attend in it)
  int32_t lo, hi;     // rows lo .. hi of the unit are visible,
  int32_t sink;       // and rows below `sink`
  float ks, vs;       // e4m3: scales of the block
  int32_t pad[2];
};

template <bool kF8>
struct Layout {
  static constexpr int kStages = Unit<kF8>::kStages;
  static constexpr uint32_t kMergeOff = 0;                                       // [4][16][kOStride], over the ring
  static constexpr uint32_t kMergeMlOff = kWarps * kHpg * kOStride * 4;          // [4][16][4], over the ring
  static constexpr uint32_t kOutOff = kStages * kStageBytes;                     // the CTA's merged O [16][128]
  static constexpr uint32_t kMlOff = kOutOff + kHpg * kD * 4;                    // and its references, sum [16][4]
  static constexpr uint32_t kInfoOff = kMlOff + kHpg * 4 * 4;
  static constexpr uint32_t kBarOff = kInfoOff + kStages * sizeof(UnitInfo);
  static constexpr uint32_t kEnd = kBarOff + 2 * kStages * 8;
  static constexpr size_t kBytes = kEnd + 1024;
};
static_assert(Layout<true>::kMergeMlOff + kWarps * kHpg * 4 * 4 <= 2 * kStageBytes, "merge buffer fits the ring");
static_assert(2 * (Layout<true>::kBytes + 1024) <= 228 * 1024 && 2 * (Layout<false>::kBytes + 1024) <= 228 * 1024,
              "CTAs per SM");

struct Params {
  const __nv_bfloat16* q;     // [n_q][16 G][128]
  const int32_t* q_stream;
  const int32_t* q_pos;
  const int32_t* sel;         // selection form: [n_q][G][16]
  const float* k_scale;       // e4m3: scale of cache row r is k_scale[r / 128]
  const float* v_scale;
  __nv_bfloat16* out;         // [n_q][16 G][128]
  int n_q, G, n_streams, capacity;
  int window, n_sink;         // window form
  float scale_log2;
  KvPages pages;
  Gate gate;
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ void mma_f16_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
      "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Two e4m3 values (the low and the high byte of v) as fp16, exactly.
__device__ __forceinline__ uint32_t e4m3_to_f16x2(uint32_t v) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(v)));
  return h;
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// Address of this CTA's shared-memory address `addr` in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t map_rank(uint32_t addr, uint32_t rank) {
  uint32_t d;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(d) : "r"(addr), "r"(rank));
  return d;
}

__device__ __forceinline__ void ld_cluster4(uint32_t addr, float (&v)[4]) {
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];"
               : "=f"(v[0]), "=f"(v[1]), "=f"(v[2]), "=f"(v[3])
               : "r"(addr)
               : "memory");
}

// The units of query position p: n of them; unit i covers the slots from
// first(i) on.  Window form: the sink units that lie wholly before the
// window's first unit, then the window's.
template <bool kF8, bool kWin>
struct Units {
  static constexpr int kRows = Unit<kF8>::kRows;
  int n, n_sink_units, win_unit;
  __device__ Units(const Params& P, int p) {
    if (kWin) {
      const int first = max(0, p - P.window + 1);
      win_unit = first / kRows;
      n_sink_units = min((P.n_sink + kRows - 1) / kRows, win_unit);
      n = n_sink_units + p / kRows - win_unit + 1;
    } else {
      win_unit = n_sink_units = 0;
      n = kTopK * (kBlock / kRows);
    }
  }
  // window form: first slot of unit i
  __device__ int first(int i) const { return (i < n_sink_units ? i : win_unit + i - n_sink_units) * kRows; }
};

template <bool kF8, bool kWin>
__global__ void __launch_bounds__(kThreads, Unit<kF8>::kCtas)
    attn_cluster_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_v,
                        const Params P, const int cluster) {
  using Layout = cattn::Layout<kF8>;
  constexpr int kStages = Unit<kF8>::kStages;
  constexpr int kRows = Unit<kF8>::kRows;
  constexpr int kWarpRows = Unit<kF8>::kWarpRows;
  constexpr int kSub = kWarpRows / 16;                 // 16-row steps of a warp's share of a unit
  // O's reference m_o is raised only when a unit passes it by more than
  // kRaise (log2 units); p is held as 2^kLift p, at most 2^14 in fp16
  constexpr float kRaise = kF8 ? 4.f : 8.f;
  constexpr float kLift = kF8 ? 10.f : 0.f;
  constexpr float kRaiseSum = 32.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + Layout::kBarOff);
  uint64_t* empty = full + kStages;
  UnitInfo* info = reinterpret_cast<UnitInfo*>(smem + Layout::kInfoOff);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int rank = cluster > 1 ? static_cast<int>(cluster_rank()) : 0;
  const long long pair = blockIdx.x / cluster;

  if (threadIdx.x == kWarps * 32) {
    prefetch_tensormap(&tm_k);
    prefetch_tensormap(&tm_v);
    for (int st = 0; st < kStages; ++st) {
      mbar_init(&full[st], 1);
      mbar_init(&empty[st], kWarps);
    }
    mbar_fence_init();
  }
  __syncthreads();
  pdl_trigger();
  pdl_wait();
  if (!gate_open(P.gate)) return;                      // (the whole grid)

  const int qi = static_cast<int>(pair / P.G);
  const int g = static_cast<int>(pair - static_cast<long long>(qi) * P.G);
  // the producer's selection is on its way with the query's place
  int picked = -1;
  if (!kWin && warp == kWarps) picked = __ldcg(P.sel + pair * kTopK + (lane & (kTopK - 1)));
  const int s = P.q_stream[qi];
  const int p = P.q_pos[qi];
  const bool valid_q = s >= 0 && s < P.n_streams && p >= 0 && p < P.capacity;
  if (!valid_q && g == 0 && rank == 0 && threadIdx.x == 0) raise_error(MSA_DEVERR_QUERY_RANGE);
  const Units<kF8, kWin> units(P, valid_q ? p : 0);
  const int n_units = valid_q ? units.n : 0;
  const int u0 = static_cast<int>(static_cast<long long>(n_units) * rank / cluster);
  const int u1 = static_cast<int>(static_cast<long long>(n_units) * (rank + 1) / cluster);

  if (warp == kWarps) {
    // ------------- producer: 32 units resolved at a time, one per lane -------------
    // a block that the selection names again counts once
    if (!kWin && (__match_any_sync(0xffffffffu, picked) & ((1u << (lane & (kTopK - 1))) - 1u)) != 0u) picked = -1;
    int k = 0;
    bool ok = true;
    for (int base = u0; base < u1 && ok; base += 32) {
      int row = -1, lo = 0, hi = -1, sink = 0;
      float ks = 0.f, vs = 0.f;
      const int block = kWin ? 0 : __shfl_sync(0xffffffffu, picked, ((base + lane) / (kBlock / kRows)) & (kTopK - 1));
      if (base + lane < u1) {
        const int u = base + lane;
        int first;
        bool any = true;
        if (kWin) {
          first = units.first(u);
          lo = max(0, p - P.window + 1 - first);
          sink = P.n_sink - first;
        } else {
          const int b = block;
          any = b >= 0 && b <= p / kBlock;
          if (b > p / kBlock) raise_error(MSA_DEVERR_SEL_RANGE);
          first = b * kBlock + (u % (kBlock / kRows)) * kRows;
        }
        hi = min(p - first, kRows - 1);
        if (any && hi >= 0) {
          const long long blk = kv_block_row(P.pages, s, g, first / kBlock, P.G, P.capacity);
          if (blk < 0) {
            raise_error(MSA_DEVERR_PAGE_RANGE);
          } else {
            row = static_cast<int>(blk) + first % kBlock;   // the host checks that every row fits 31 bits
            if (kF8) {
              ks = __ldcg(P.k_scale + blk / kBlock);      // (the append before may have written them)
              vs = __ldcg(P.v_scale + blk / kBlock);
            }
          }
        }
      }
      const int count = min(32, u1 - base);
      for (int i = 0; i < count; ++i, ++k) {
        const int r = __shfl_sync(0xffffffffu, row, i);
        const int l = __shfl_sync(0xffffffffu, lo, i), h = __shfl_sync(0xffffffffu, hi, i);
        const int sk = __shfl_sync(0xffffffffu, sink, i);
        const int st = k % kStages;
        if (lane == 0 && ok) {
          if (k >= kStages) ok = mbar_wait(&empty[st], (k / kStages - 1) & 1);
          if (ok && r >= 0) {
            uint8_t* dst = smem + st * kStageBytes;
            if (kF8) {
              tma_load_2d(dst, &tm_k, 0, r, &full[st]);
              tma_load_2d(dst + kHalfStage, &tm_v, 0, r, &full[st]);
            } else {
              tma_load_2d(dst, &tm_k, 0, r, &full[st]);
              tma_load_2d(dst + kHalfStage / 2, &tm_k, 64, r, &full[st]);
              tma_load_2d(dst + kHalfStage, &tm_v, 0, r, &full[st]);
              tma_load_2d(dst + kHalfStage + kHalfStage / 2, &tm_v, 64, r, &full[st]);
            }
          }
        }
        // the scales arrive behind the copies (the record's arrival closes the
        // phase, so the copies may be announced after they were issued)
        const float fk = __shfl_sync(0xffffffffu, ks, i), fv = __shfl_sync(0xffffffffu, vs, i);
        if (lane == 0 && ok) {
          UnitInfo& in = info[st];
          in.data = r >= 0;
          in.lo = l;
          in.hi = h;
          in.sink = sk;
          in.ks = fk;
          in.vs = fv;
          mbar_arrive_expect_tx(&full[st], r >= 0 ? kStageBytes : 0u);
        }
        ok = __shfl_sync(0xffffffffu, ok ? 1 : 0, 0) != 0;
        if (!ok) break;
      }
    }
    // no copy may still be landing when the ring is reused
    if (lane == 0)
      for (int j = max(0, k - kStages); j < k; ++j) mbar_wait(&full[j % kStages], (j / kStages) & 1);
    __syncwarp();
  } else {
    // -------------------------------- consumers --------------------------------
    const int gr = lane >> 2, tq = lane & 3;
    const int mi = lane >> 3, l7 = lane & 7;
    uint32_t qa[8][4];
    float qf[2] = {P.scale_log2, P.scale_log2};        // score factors of heads gr and gr + 8
    {
      const __nv_bfloat16* q0 = P.q + (static_cast<size_t>(pair) * kHpg + gr) * kD;
      const __nv_bfloat16* q1 = q0 + 8 * kD;
      if (!kF8) {
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qa[ks][0] = *reinterpret_cast<const uint32_t*>(q0 + 16 * ks + 2 * tq);
          qa[ks][1] = *reinterpret_cast<const uint32_t*>(q1 + 16 * ks + 2 * tq);
          qa[ks][2] = *reinterpret_cast<const uint32_t*>(q0 + 16 * ks + 8 + 2 * tq);
          qa[ks][3] = *reinterpret_cast<const uint32_t*>(q1 + 16 * ks + 8 + 2 * tq);
        }
      } else {
        uint2 x[2][8];
        float top[2] = {0.f, 0.f};
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          x[0][ks] = *reinterpret_cast<const uint2*>(q0 + 16 * ks + 4 * tq);
          x[1][ks] = *reinterpret_cast<const uint2*>(q1 + 16 * ks + 4 * tq);
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            const uint32_t w[2] = {x[h][ks].x, x[h][ks].y};
#pragma unroll
            for (int i = 0; i < 2; ++i)
              top[h] = fmaxf(top[h], fmaxf(fabsf(__uint_as_float(w[i] << 16)), fabsf(__uint_as_float(w[i] & 0xffff0000u))));
          }
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 1));
          top[h] = fmaxf(top[h], __shfl_xor_sync(0xffffffffu, top[h], 2));
          // 2^(14 - e), e the exponent of the largest magnitude
          int e = static_cast<int>(__float_as_uint(top[h]) >> 23) - 127;
          e = top[h] > 0.f ? max(e, -100) : 14;
          const float up = __uint_as_float(static_cast<uint32_t>(127 + 14 - e) << 23);
          qf[h] *= __uint_as_float(static_cast<uint32_t>(127 - 14 + e) << 23);
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            qa[ks][h] = pack_f16(__uint_as_float(x[h][ks].x << 16) * up, __uint_as_float(x[h][ks].x & 0xffff0000u) * up);
            qa[ks][2 + h] = pack_f16(__uint_as_float(x[h][ks].y << 16) * up, __uint_as_float(x[h][ks].y & 0xffff0000u) * up);
          }
        }
      }
    }
    float o[16][4];
#pragma unroll
    for (int n = 0; n < 16; ++n) o[n][0] = o[n][1] = o[n][2] = o[n][3] = 0.f;
    float m_o[2] = {-INFINITY, -INFINITY}, m_l[2] = {-INFINITY, -INFINITY}, l_run[2] = {0.f, 0.f};
    const int wr = warp * kWarpRows;
    bool ok = true;
    for (int k = 0; k < u1 - u0; ++k) {
      const int st = k % kStages;
      if (ok) ok = mbar_wait(&full[st], (k / kStages) & 1);
      ok = __all_sync(0xffffffffu, ok);                // warp-uniform: the MMAs below take the whole warp
      if (!ok) break;
      const UnitInfo in = info[st];
      // rows of this warp that the masks leave
      const bool cut = in.hi < wr + kWarpRows - 1 || (in.lo > wr && in.sink < min(in.lo, wr + kWarpRows));
      const bool none = wr > in.hi || (in.lo > min(in.hi, wr + kWarpRows - 1) && in.sink <= wr);
      if (in.data != 0 && !none) {
        const uint32_t kbase = smem_addr(smem + st * kStageBytes);
        const uint32_t vbase = kbase + kHalfStage;
        float sc[2 * kSub][4];                         // scores: n tiles of 8 rows
#pragma unroll
        for (int t = 0; t < 2 * kSub; ++t) sc[t][0] = sc[t][1] = sc[t][2] = sc[t][3] = 0.f;
        if (kF8) {
          // one x4: 8 rows x 64 dims, i.e. four k-steps of one n tile; the n
          // tiles take turns, so that successive MMAs do not wait for each other
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            uint32_t b[2 * kSub][4];
#pragma unroll
            for (int t = 0; t < 2 * kSub; ++t) ldmatrix_x4(b[t], kbase + swz128(wr + t * 8 + l7, half * 4 + mi));
#pragma unroll
            for (int i = 0; i < 4; ++i)
#pragma unroll
              for (int t = 0; t < 2 * kSub; ++t)
                mma_f16_16816(sc[t], qa[half * 4 + i], e4m3_to_f16x2(b[t][i]), e4m3_to_f16x2(b[t][i] >> 16));
          }
        } else {
#pragma unroll
          for (int ks = 0; ks < 8; ++ks) {
            uint32_t b[4];
            ldmatrix_x4(b, kbase + (ks >> 2) * (kHalfStage / 2) + swz128(wr + (mi >> 1) * 8 + l7, (ks & 3) * 2 + (mi & 1)));
            mma_bf16_16816(sc[0], qa[ks], b[0], b[1]);
            mma_bf16_16816(sc[1], qa[ks], b[2], b[3]);
          }
        }
        const float f0 = kF8 ? qf[0] * in.ks : qf[0], f1 = kF8 ? qf[1] * in.ks : qf[1];
        float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
        for (int t = 0; t < 2 * kSub; ++t) {
#pragma unroll
          for (int e = 0; e < 4; ++e) sc[t][e] *= e < 2 ? f0 : f1;
        }
        if (cut) {
#pragma unroll
          for (int t = 0; t < 2 * kSub; ++t) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const int r = wr + t * 8 + tq * 2 + (e & 1);
              if (r > in.hi || (r < in.lo && r >= in.sink)) sc[t][e] = -INFINITY;
            }
          }
        }
#pragma unroll
        for (int t = 0; t < 2 * kSub; ++t)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e >> 1] = fmaxf(mx[e >> 1], sc[t][e]);
        // log2 of the V scale: a unit's rows weigh p * vs in O
        const float lvs = kF8 ? __log2f(fabsf(in.vs)) : 0.f;
        bool up[2];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 1));
          mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], 2));
          up[h] = mx[h] + lvs > m_o[h] + kRaise;
        }
        if (__any_sync(0xffffffffu, up[0] || up[1])) {
          float alpha[2];
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float m_new = up[h] ? mx[h] + lvs : m_o[h];
            alpha[h] = m_o[h] == m_new ? 1.f : ex2(m_o[h] - m_new);      // 0 the first time
            m_o[h] = m_new;
            if (!kF8) l_run[h] *= alpha[h];
          }
#pragma unroll
          for (int n = 0; n < 16; ++n) {
            o[n][0] *= alpha[0];
            o[n][1] *= alpha[0];
            o[n][2] *= alpha[1];
            o[n][3] *= alpha[1];
          }
        }
        // e4m3: the sum of the p has a reference of its own, raised rarely
        // (float32 has room)
        if (kF8 && __any_sync(0xffffffffu, mx[0] > m_l[0] + kRaiseSum || mx[1] > m_l[1] + kRaiseSum)) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            if (mx[h] > m_l[h]) {
              l_run[h] *= ex2(m_l[h] - mx[h]);
              m_l[h] = mx[h];
            }
          }
        }
        uint32_t pa[kSub][4];
        float rs[2] = {0.f, 0.f};
        // (m_o still -inf: everything masked, or a V scale of zero)
        const float off[2] = {m_o[0] == -INFINITY ? -INFINITY : lvs - m_o[0] + kLift,
                              m_o[1] == -INFINITY ? -INFINITY : lvs - m_o[1] + kLift};
        const float off_l[2] = {m_l[0] == -INFINITY ? 0.f : -m_l[0], m_l[1] == -INFINITY ? 0.f : -m_l[1]};
        const uint32_t sign = kF8 && in.vs < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int t = 0; t < 2 * kSub; ++t) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const float x = ex2(sc[t][2 * h] + off[h]), y = ex2(sc[t][2 * h + 1] + off[h]);
            uint32_t w;
            if (kF8) {
              w = pack_f16(x, y) ^ sign;
              rs[h] += ex2(sc[t][2 * h] + off_l[h]) + ex2(sc[t][2 * h + 1] + off_l[h]);
            } else {
              w = pack_bf16(x, y);
              rs[h] += __uint_as_float(w << 16) + __uint_as_float(w & 0xffff0000u);
            }
            pa[t >> 1][(t & 1) * 2 + h] = w;
          }
        }
        l_run[0] += rs[0];
        l_run[1] += rs[1];
        // V rows that the masks cut off count as zeros
        uint32_t keep[kSub][2];
        if (cut) {
#pragma unroll
          for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              const int r = wr + u * 16 + i * 8 + tq * 2;
              const bool a = r <= in.hi && (r >= in.lo || r < in.sink);
              const bool b = r + 1 <= in.hi && (r + 1 >= in.lo || r + 1 < in.sink);
              keep[u][i] = (a ? 0x0000ffffu : 0u) | (b ? 0xffff0000u : 0u);
            }
          }
        }
        if (kF8) {
          // 16 dims at a time: tile n the even ones, n + 1 the odd ones
#pragma unroll
          for (int c = 0; c < 8; ++c) {
            uint32_t v[4];                             // rows 0-7, 8-15, 16-23, 24-31 of the warp's 32
            ldmatrix_x4_trans(v, vbase + swz128(wr + mi * 8 + l7, c));
            if (cut) {
#pragma unroll
              for (int u = 0; u < 2 * kSub; ++u) v[u] &= keep[u >> 1][u & 1];
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
              const uint32_t x2 = __byte_perm(v[2 * u], 0u, 0x3120), y2 = __byte_perm(v[2 * u + 1], 0u, 0x3120);
              mma_f16_16816(o[2 * c], pa[u], e4m3_to_f16x2(x2), e4m3_to_f16x2(y2));
              mma_f16_16816(o[2 * c + 1], pa[u], e4m3_to_f16x2(x2 >> 16), e4m3_to_f16x2(y2 >> 16));
            }
          }
        } else {
#pragma unroll
          for (int jn = 0; jn < 8; ++jn) {
            uint32_t v[4];
            ldmatrix_x4_trans(v, vbase + (jn >> 2) * (kHalfStage / 2) + swz128(wr + (mi & 1) * 8 + l7, (jn & 3) * 2 + (mi >> 1)));
            if (cut) {
              v[0] &= keep[0][0];
              v[1] &= keep[0][1];
              v[2] &= keep[0][0];
              v[3] &= keep[0][1];
            }
            mma_bf16_16816(o[2 * jn], pa[0], v[0], v[1]);
            mma_bf16_16816(o[2 * jn + 1], pa[0], v[2], v[3]);
          }
        }
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&empty[st]);
    }
    // the warp's state goes to the merge buffer once the ring is idle
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 1);
      l_run[h] += __shfl_xor_sync(0xffffffffu, l_run[h], 2);
    }
    named_barrier_sync(1, kWarps * 32);
    float* so = reinterpret_cast<float*>(smem + Layout::kMergeOff) + warp * kHpg * kOStride;
    float* sml = reinterpret_cast<float*>(smem + Layout::kMergeMlOff) + warp * kHpg * 4;
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      if (kF8) {
        // tile 2c column x: dim 16c + 2x, tile 2c + 1: the dim after it
        const int d = 16 * c + 4 * tq;
        *reinterpret_cast<float4*>(so + gr * kOStride + d) = make_float4(o[2 * c][0], o[2 * c + 1][0], o[2 * c][1], o[2 * c + 1][1]);
        *reinterpret_cast<float4*>(so + (gr + 8) * kOStride + d) = make_float4(o[2 * c][2], o[2 * c + 1][2], o[2 * c][3], o[2 * c + 1][3]);
      } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int n = 2 * c + i, d = 8 * n + 2 * tq;
          *reinterpret_cast<float2*>(so + gr * kOStride + d) = make_float2(o[n][0], o[n][1]);
          *reinterpret_cast<float2*>(so + (gr + 8) * kOStride + d) = make_float2(o[n][2], o[n][3]);
        }
      }
    }
    if (tq == 0) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float4*>(sml + (gr + 8 * h) * 4) = make_float4(m_o[h], kF8 ? m_l[h] : m_o[h], l_run[h], 0.f);
    }
    named_barrier_sync(1, kWarps * 32);
    // the CTA's state: thread (head, 16 dims)
    const int tid = threadIdx.x;
    const int head = tid >> 3, dd = (tid & 7) * 16;
    const float* all = reinterpret_cast<const float*>(smem + Layout::kMergeOff);
    const float* allml = reinterpret_cast<const float*>(smem + Layout::kMergeMlOff);
    float acc[16];
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.f;
    float Mo = -INFINITY, Ml = -INFINITY, L = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      Mo = fmaxf(Mo, allml[(w * kHpg + head) * 4]);
      Ml = fmaxf(Ml, allml[(w * kHpg + head) * 4 + 1]);
    }
    const float uo = Mo == -INFINITY ? 0.f : Mo, ul = Ml == -INFINITY ? 0.f : Ml;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 ml = *reinterpret_cast<const float4*>(allml + (w * kHpg + head) * 4);
      const float f = ex2(ml.x - uo);
      L += ml.z * ex2(ml.y - ul);
#pragma unroll
      for (int i = 0; i < 16; i += 4) {
        const float4 v = *reinterpret_cast<const float4*>(all + (w * kHpg + head) * kOStride + dd + i);
        acc[i] += v.x * f;
        acc[i + 1] += v.y * f;
        acc[i + 2] += v.z * f;
        acc[i + 3] += v.w * f;
      }
    }
    if (cluster == 1) {
      const float inv = L != 0.f ? ex2(uo - ul - kLift) / L : 0.f;
      uint32_t w[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = pack_bf16(acc[2 * i] * inv, acc[2 * i + 1] * inv);
      uint4* dst = reinterpret_cast<uint4*>(P.out + (static_cast<size_t>(pair) * kHpg + head) * kD + dd);
      dst[0] = make_uint4(w[0], w[1], w[2], w[3]);
      dst[1] = make_uint4(w[4], w[5], w[6], w[7]);
    } else {
      float* mine = reinterpret_cast<float*>(smem + Layout::kOutOff) + head * kD + dd;
#pragma unroll
      for (int i = 0; i < 16; i += 4)
        *reinterpret_cast<float4*>(mine + i) = make_float4(acc[i], acc[i + 1], acc[i + 2], acc[i + 3]);
      if ((tid & 7) == 0) {
        *reinterpret_cast<float4*>(smem + Layout::kMlOff + head * 16) = make_float4(Mo, Ml, L, 0.f);
      }
    }
  }
  if (cluster == 1) return;
  __syncwarp();
  cluster_sync();                                      // every CTA's state is in its shared memory
  if (warp < kWarps) {
    // rank r writes heads r, r + cluster, ...: a quarter of a warp's lanes per
    // 32 dims, four dims a lane
    for (int head = rank + warp * cluster; head < kHpg; head += kWarps * cluster) {
      const uint32_t obase = smem_addr(smem + Layout::kOutOff) + (head * kD + lane * 4) * 4;
      // lane c < cluster holds rank c's references and sum
      float ml[4] = {-INFINITY, -INFINITY, 0.f, 0.f};
      if (lane < cluster) ld_cluster4(map_rank(smem_addr(smem + Layout::kMlOff) + head * 16, lane), ml);
      float Mo = ml[0], Ml = ml[1];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        Mo = fmaxf(Mo, __shfl_xor_sync(0xffffffffu, Mo, o));
        Ml = fmaxf(Ml, __shfl_xor_sync(0xffffffffu, Ml, o));
      }
      const float uo = Mo == -INFINITY ? 0.f : Mo, ul = Ml == -INFINITY ? 0.f : Ml;
      const float fc = ex2(ml[0] - uo);
      float L = lane < cluster ? ml[2] * ex2(ml[1] - ul) : 0.f;
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
      float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 4
      for (int c = 0; c < cluster; ++c) {
        float v[4];
        ld_cluster4(map_rank(obase, c), v);
        const float f = __shfl_sync(0xffffffffu, fc, c);
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[i] += v[i] * f;
      }
      const float inv = L != 0.f ? ex2(uo - ul - kLift) / L : 0.f;
      *reinterpret_cast<uint2*>(P.out + (static_cast<size_t>(pair) * kHpg + head) * kD + lane * 4) =
          make_uint2(pack_bf16(acc[0] * inv, acc[1] * inv), pack_bf16(acc[2] * inv, acc[3] * inv));
    }
  }
  __syncwarp();
  cluster_sync();                                      // no CTA leaves while another reads its shared memory
}

}  // namespace cattn
}  // namespace msa
