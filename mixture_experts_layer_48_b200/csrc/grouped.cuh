// Matrix products grouped by expert, ragged sizes, forward and backward.
//
// R rows lie in expert order: expert e owns rows [offsets[e], offsets[e+1]) (what moe_route and
// moe_permute produce).  W is [E, K, N], bf16; all sums are fp32 in tensor memory.
//
//   product            y[r, :] = x[r, :] W[e]          x [R, K] -> y [R, N]       (forward)
//   transposed         y[r, :] = x[r, :] W[e]^T        x [R, N] -> y [R, K]       (gradient of x)
//   weight gradient    dW[e]   = sum_r x[r, :]^T dy[r, :]   over e's rows         [E, K, N]
//
// Three kernel shapes, persistent and warp-specialised (TMA producer warp, MMA issuer warp, four or
// eight epilogue warps) around a ring of 128-byte-swizzled shared-memory stages of 64 reduction
// elements (128 where a tile has few rows):
//
//   grouped_cols_kernel   few rows per expert, bound by reading each touched expert's weights
//                         once from HBM: 128 weight columns are the M operand, the rows N, and a
//                         cluster of S CTAs can split the reduction of one tile (each sends its
//                         partial sums to the rank that owns the column, over distributed shared
//                         memory; they are added in rank order, so results do not depend on timing)
//   grouped_rows_kernel   many rows per expert, bound by the tensor cores: 256 rows x 256 columns
//                         per CTA pair (tcgen05 cta_group::2)
//   grouped_wgrad_kernel  256 x 256 tiles of dW[e] per CTA pair, the expert's rows are the
//                         reduction; both operands are MN-major
//
// Measured (one B200; copy bandwidth 6.46 TB/s, bf16 1.63 PFLOP/s in a burst and 1.38 sustained).  The
// two long ones as a burst of 12 calls, and after 3 s of calls, when the power cap holds the clock at
// 1.1 to 1.5 GHz:
//   grouped_cols_kernel   64 rows over 32 experts, 2880 x 5760: 144 us, 6.5 TB/s; one token on 128
//                         experts, 2880 x 2880, fp32: 18.7 us, 3.6 TB/s (about 5 us of it start-up)
//   grouped_rows_kernel   131,072 skewed rows, 2880 x 5760: 3.0 ms, 1.43 PFLOP/s, and 3.5 ms, 1.23;
//                         tensor pipe 85 to 88 % busy, the rest is hand-over and the experts' padded last
//                         chunks.  fp32 results cost 5 to 15 % more (32,768 rows, 2880 x 2880: 489 us for
//                         440)
//   grouped_wgrad_kernel  32,768 rows, 2880 x 5760: 0.97 ms, 1.12 PFLOP/s, and 1.12 ms, 0.97; tensor pipe
//                         65 % busy (16 stages a tile, each with a ragged end); fp32 1.15 to 1.22 ms; 512
//                         rows over 128 experts, 2880 x 2880: 462 to 700 us, 3.0 to 4.6 TB/s of writes
//
// The segments are read on the device: every CTA checks the E + 1 offsets and scans them in
// shared memory, so there is no work-list kernel, no workspace and no host sync.  Offsets that
// are negative, decrease or pass R give empty segments and set the status word.  Rows outside
// every segment are neither used nor written.
//
// Sums: the tensor cores add into fp32 accumulators with truncation, an error that grows with the
// reduction: by about 1.1e-9 of the result per element on values of random signs (measured: 3.0e-6
// at 2880, 6.3e-6 at 5760, 1.9e-5 at 16384), by 7e-9 where all terms have one sign (2.9e-2 at 4
// million).  fp32 results therefore come from pieces of 640 elements, added in the epilogue's
// registers with round to nearest (2.7e-7 ... 7e-7 in all on random signs, 4.5e-6 on one).  bf16
// results, whose rounding is 3.9e-3, take one piece per reduction of a product (at most 32768
// elements, 2.3e-4), and pieces of 65536 rows in the weight gradient (4.6e-4), whose reductions have
// no such bound.
#pragma once

#include "common.cuh"
#include "ep.cuh"
#include "expert_gemm_mx.cuh"
#include "gemm.cuh"

namespace moe {

constexpr int kGrMaxE = 256;
constexpr int kGrBK = 64;           // reduction elements of one 128-byte swizzle row (a stage, mostly)
constexpr int kGrPieceStages = 10;  // stages per accumulator of an fp32 result (640 elements)
constexpr int kGrPieceRowsBf16 = 65536;   // rows per accumulator of a bf16 weight gradient

MOE_DEVINL void tma_load_3d(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2,
                            uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(bar))
      : "memory");
}
MOE_DEVINL void tma_load_3d_pair(void* smem_dst, const CUtensorMap* map, int c0, int c1, int c2,
                                 uint32_t bar_cluster_addr) {
  asm volatile(
      "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(c2), "r"(bar_cluster_addr)
      : "memory");
}
// Wait that also orders the reads after writes of the other CTAs of the cluster.
MOE_DEVINL bool mbar_try_wait_cluster(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}
MOE_DEVINL bool wait_or_abort_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                      uint32_t* status) {
  if (mbar_try_wait_cluster(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (*abort_flag) return false;
    if (mbar_try_wait_cluster(bar, parity)) return true;
    if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}
// For a thread whose event may lie any time ahead, as the work before it is not its own: the limit
// starts anew whenever *progress changes.
MOE_DEVINL bool wait_or_abort_while(uint64_t* bar, uint32_t parity, const volatile uint32_t* progress,
                                    volatile int* abort_flag, uint32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  uint64_t t0 = globaltimer_ns();
  uint32_t seen = *progress;
  while (true) {
    if (*abort_flag) return false;
    if (mbar_try_wait(bar, parity)) return true;
    const uint32_t now = *progress;
    if (now != seen) {
      seen = now;
      t0 = globaltimer_ns();
    } else if (globaltimer_ns() - t0 > kWaitLimitNs) {
      atomicOr(status, kStatusTimeout);
      *abort_flag = 1;
      return false;
    }
  }
}
// The same answer for every lane, so that a warp leaves its loop as one (the tensor-memory loads
// and barriers that follow are collective).
MOE_DEVINL bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                          uint32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort(bar, parity, abort_flag, status));
}
MOE_DEVINL bool warp_wait_cluster(uint64_t* bar, uint32_t parity, volatile int* abort_flag,
                                  uint32_t* status) {
  return __all_sync(0xffffffffu, wait_or_abort_cluster(bar, parity, abort_flag, status));
}
// Named barrier over nthreads threads that also answers whether `ok` held for all of them.
MOE_DEVINL bool named_bar_and(int id, int nthreads, bool ok) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(nthreads), "r"((uint32_t)ok)
      : "memory");
  return r != 0;
}
// sum[i] += column taddr + i of this warp's 32 TMEM lanes (lane = thread), 8 columns at a time so
// that the loaded values need few registers beside the sums.
MOE_DEVINL void tmem_add32(uint32_t taddr, float (&sum)[32]) {
#pragma unroll
  for (int h = 0; h < 32; h += 8) {
    uint32_t r[8];
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]),
          "=r"(r[7])
        : "r"(taddr + h)
        : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
    for (int i = 0; i < 8; ++i) sum[h + i] += __uint_as_float(r[i]);
  }
}
// The two halves of cluster_sync_all, for whole warps.
MOE_DEVINL void cluster_arrive() {
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
MOE_DEVINL void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
// 16 bytes to another CTA's shared memory, counted on that CTA's barrier when they have arrived.
MOE_DEVINL void st_async_f4(uint32_t to, float x, float y, float z, float w, uint32_t bar) {
  asm volatile(
      "st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.f32 [%0], {%1, %2, %3, %4}, "
      "[%5];" ::"r"(to),
      "f"(x), "f"(y), "f"(z), "f"(w), "r"(bar)
      : "memory");
}

// Expert segments in shared memory: expert e owns rows [beg[e], beg[e] + cnt[e]); its row chunks
// are number base[e] .. base[e + 1] - 1 of the call's.
struct Segments {
  int32_t beg[kGrMaxE];
  int32_t cnt[kGrMaxE];
  int32_t base[kGrMaxE + 1];
};

// Every thread of the block; the caller synchronises the block afterwards.  Only warp 0 writes
// base, after a barrier inside.
MOE_DEVINL void load_segments(Segments& s, const int32_t* __restrict__ offsets, int E, int R,
                              int chunk, uint32_t* status) {
  for (int e = threadIdx.x; e < E; e += blockDim.x) {
    const int b = offsets[e], n = offsets[e + 1];
    const bool ok = b >= 0 && n >= b && n <= R;
    if (!ok) atomicOr(status, kStatusBadCounts);
    s.beg[e] = ok ? b : 0;
    s.cnt[e] = ok ? n - b : 0;
  }
  __syncthreads();
  if (threadIdx.x < 32) {
    const int lane = threadIdx.x;
    int run = 0;
    for (int e0 = 0; e0 < E; e0 += 32) {
      const int e = e0 + lane;
      const int c = e < E ? (s.cnt[e] + chunk - 1) / chunk : 0;
      int inc = c;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (e < E) s.base[e] = run + inc - c;
      run += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (lane == 0) s.base[E] = run;
  }
}

// The expert that owns tile t when an expert with c chunks has c * per tiles: the last e with
// base[e] * per <= t.  t < base[E] * per.
MOE_DEVINL int find_expert(const Segments& s, int E, int per, int t) {
  const int c = t / per;
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s.base[mid] <= c) lo = mid;
    else hi = mid;
  }
  return lo;
}

struct GroupedArgs {
  const int32_t* offsets;  // [E + 1]
  int E, R;
  int Kred;                // reduction length (row length of x; rows of a segment for dW)
  int Ncols;               // columns of the result
  int M;                   // rows of one dW[e] (weight gradient only)
  void* out;               // [R, Ncols], or [E, M, Ncols] for the weight gradient
  uint32_t* status;
};

// Writes 4 fp32 values as fp32 or bf16 to 4 consecutive columns.
template <bool F32>
MOE_DEVINL void store4(void* out, size_t idx, float4 v) {
  if constexpr (F32) {
    *reinterpret_cast<float4*>(static_cast<float*>(out) + idx) = v;
  } else {
    *reinterpret_cast<uint2*>(static_cast<uint16_t*>(out) + idx) =
        make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
  }
}

// ------------------------------------------------------------------------------------------------
// Few rows per expert: weight columns as the M operand, rows as N.
//
// ROWS: rows per tile (largest MMA N).  NM: 128-column MMAs per tile.
//   <32, 1>   a cluster of S CTAs splits a tile's reduction (S = 1: one CTA per tile)
//   <128, 2>  one CTA per tile of 256 columns: the rows are loaded once for both MMAs
// ------------------------------------------------------------------------------------------------
template <int ROWS, int NM>
struct ColsCfg {
  static constexpr bool kSplit = NM == 1;
  // Reduction elements per stage: a 128-column tile takes 128 (32 KB of weights; with 64 it streamed
  // 47 GB/s per SM instead of 64: one token down 20.0 against 18.7 us).
  static constexpr int kK = kSplit ? 2 * kGrBK : kGrBK;
  static constexpr int kABytes = NM * 128 * kK * 2;
  static constexpr int kBHalf = ROWS * kGrBK * 2;           // 64 elements of every row
  static constexpr int kBBytes = ROWS * kK * 2;
  static constexpr int kStageBytes = kABytes + kBBytes;
  static constexpr int kStages = 4;
  // Rows per TMA box: the MMAs take the rows rounded up to 16; a 128-row tile copies 64 at a time
  // (8 experts of 128 rows, 2880 x 2880: 30.1 us against 37.1 with boxes of 16).
  static constexpr int kRowBox = kSplit ? 16 : 64;
  static constexpr int kAccBufs = 2;
  static constexpr int kTmemCols = kAccBufs * NM * ROWS;    // 64, 256, 512: powers of two
  static constexpr int kEpiWarps = 4 * NM;                  // four per 128-column MMA
  static constexpr int kThreads = 64 + 32 * kEpiWarps;
  // split: two buffers of partial sums [source rank][column of this rank][row]; else rows staged
  // for the stores
  static constexpr int kPitch = kSplit ? ROWS + 4 : 33;     // floats
  static constexpr int kEpiBytes = kSplit ? 2 * 128 * kPitch * 4 : kEpiWarps * 16 * kPitch * 4;
  static constexpr int kSmem = 1024 + kStages * kStageBytes + 256 + kEpiBytes;
  static_assert(kStageBytes % 1024 == 0, "128-byte swizzle atoms");
  static_assert(kSmem + (int)sizeof(Segments) + 64 <= 227 * 1024, "shared memory");
};

template <int ROWS, int NM, bool TRANS, bool F32>
__global__ void __launch_bounds__(ColsCfg<ROWS, NM>::kThreads, 1)
    grouped_cols_kernel(const GroupedArgs a, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap, const int S) {
  using C = ColsCfg<ROWS, NM>;
  constexpr int kStages = C::kStages, kBufs = C::kAccBufs;
  constexpr int TW = 128 * NM;                       // output columns per tile
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* ring = align1k(smem_raw);
  uint64_t* bars = reinterpret_cast<uint64_t*>(ring + kStages * C::kStageBytes);
  uint64_t* full = bars;
  uint64_t* empty = full + kStages;
  uint64_t* acc_full = empty + kStages;
  uint64_t* acc_empty = acc_full + kBufs;
  uint64_t* drain = acc_empty + kBufs;
  uint64_t* part_full = drain + 1;       // the cluster's partial sums of this rank's columns are here
  uint64_t* part_empty = part_full + 2;  // every rank has added the sums this CTA sent it
  float* epi = reinterpret_cast<float*>(ring + kStages * C::kStageBytes + 256);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = C::kSplit ? (int)cluster_ctarank() : 0;

  if (warp == 1) {
    tmem_alloc(&s_tmem, C::kTmemCols);
    tmem_relinquish();
  }
  if (tid == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < kBufs; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 32 * C::kEpiWarps);
    }
    mbar_init(drain, 1);
    for (int b = 0; b < 2; ++b) {
      mbar_init(&part_full[b], 1);
      mbar_init(&part_empty[b], S);
    }
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
  pdl_wait();  // offsets, rows and weights may come from the previous kernels
  pdl_launch_next();
  load_segments(seg, a.offsets, a.E, a.R, ROWS, a.status);
  tc_fence_before();
  __syncthreads();
  // the other CTAs' barriers are only needed once sums are sent: the copies start before that
  if (C::kSplit) cluster_arrive();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;

  const int NT = (a.Ncols + TW - 1) / TW;
  const int tiles = seg.base[a.E] * NT;
  const int nk_all = (a.Kred + C::kK - 1) / C::kK;
  const int piece = F32 ? kGrPieceStages * kGrBK / C::kK : nk_all;
  const int group = C::kSplit ? (int)blockIdx.x / S : (int)blockIdx.x;
  const int groups = C::kSplit ? (int)gridDim.x / S : (int)gridDim.x;
  volatile int* abort_flag = &s_abort;

  // Tile t: the chunks of one expert and column block are neighbours, so an expert with more
  // than one chunk re-reads its weight block from L2.
  struct Tile { int e, row0, rows, n0; };
  auto tile_at = [&](int t) {
    Tile w;
    w.e = find_expert(seg, a.E, NT, t);
    const int chunks = seg.base[w.e + 1] - seg.base[w.e];
    const int local = t - seg.base[w.e] * NT;
    const int ch = local % chunks;
    w.n0 = local / chunks * TW;
    w.row0 = seg.beg[w.e] + ch * ROWS;
    w.rows = min(ROWS, seg.cnt[w.e] - ch * ROWS);
    return w;
  };
  // This CTA's stages of tile t: an even split over the cluster, the remainder rotated from tile
  // to tile so that every rank streams the same bytes in the long run.
  auto k_range = [&](int t, int& k0, int& k1) {
    if (!C::kSplit) {
      k0 = 0;
      k1 = nk_all;
      return;
    }
    const int q = nk_all / S, rem = nk_all - q * S;
    const int p = (rank + t / groups) % S;
    k0 = p * q + min(p, rem);
    k1 = k0 + q + (p < rem ? 1 : 0);
  };

  if (warp == 0) {
    // ------------------------------ TMA producer ------------------------------
    if (lane == 0) {
      uint32_t issued = 0, ph = 0;
      int slot = 0;
      bool ok = true;
      for (int t = group; ok && t < tiles && !*abort_flag; t += groups) {
        const Tile w = tile_at(t);
        int k0, k1;
        k_range(t, k0, k1);
        const int nrb = (w.rows + C::kRowBox - 1) / C::kRowBox;
        const uint32_t bytes = C::kABytes + (uint32_t)nrb * C::kRowBox * C::kK * 2;
        for (int k = k0 * C::kK; k < k1 * C::kK; k += C::kK) {
          if (!wait_or_abort(&empty[slot], ph ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&full[slot], bytes);
          uint8_t* st = ring + slot * C::kStageBytes;
          // weight boxes past the matrix's edges are zero-filled (each expert is a plane of the
          // map, so an edge never reads the next expert)
          if (TRANS) {  // [columns of y, reduction]: 128 x 64 boxes, K-major
#pragma unroll
            for (int m = 0; m < NM; ++m)
#pragma unroll
              for (int h = 0; h < C::kK / kGrBK; ++h)
                tma_load_3d(st + (m + h) * 128 * kGrBK * 2, &wmap, k + h * kGrBK, w.n0 + 128 * m, w.e,
                            &full[slot]);
          } else {      // [reduction, columns of y]: kK x 64 boxes, MN-major
#pragma unroll
            for (int b = 0; b < 2 * NM; ++b)
              tma_load_3d(st + b * 64 * C::kK * 2, &wmap, w.n0 + 64 * b, k, w.e, &full[slot]);
          }
#pragma unroll
          for (int h = 0; h < C::kK / kGrBK; ++h)
            for (int r = 0; r < nrb; ++r)
              tma_load_2d(st + C::kABytes + h * C::kBHalf + r * (C::kRowBox * kGrBK * 2), &xmap,
                          k + h * kGrBK, w.row0 + r * C::kRowBox, &full[slot]);
          ++issued;
          if (++slot == kStages) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      // never leave the CTA with copies in flight
      for (uint32_t j = issued - min(issued, (uint32_t)kStages); j < issued; ++j)
        if (!mbar_wait_bounded(&full[j % kStages], (j / kStages) & 1u, kWaitLimitNs))
          atomicOr(a.status, kStatusTimeout);
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer ------------------------------
    if (lane == 0) {
      const uint32_t ring_s = smem_u32(ring);
      // descriptors of slot 0; a slot / K-step offset only moves the 14-bit start address
      const uint64_t adesc0 = TRANS ? smem_desc_sw128(ring_s, 16, 1024)
                                    : smem_desc_sw128(ring_s, 64 * C::kK * 2, 1024);
      const uint64_t bdesc0 = smem_desc_sw128(ring_s + C::kABytes, 16, 1024);
      int slot = 0, unit = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = group; ok && t < tiles && !*abort_flag; t += groups) {
        const Tile w = tile_at(t);
        int k0, k1;
        k_range(t, k0, k1);
        const int N = (w.rows + 15) / 16 * 16;
        const uint32_t idesc = idesc_bf16_f32(128, N, !TRANS, false);
        for (int p0 = k0; ok && p0 < k1; p0 += piece, ++unit) {
          const int p1 = min(k1, p0 + piece);
          const int buf = unit % kBufs;
          const uint32_t aph = (unit / kBufs) & 1u;
          if (!wait_or_abort(&acc_empty[buf], aph ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * NM * ROWS;
          uint32_t acc = 0;
          for (int kst = p0; kst < p1; ++kst) {
            if (!wait_or_abort(&full[slot], ph, abort_flag, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t soff = (uint64_t)((slot * C::kStageBytes) >> 4);
#pragma unroll
            for (int k16 = 0; k16 < C::kK / 16; ++k16) {
              // K-major: 64 elements a box, 32 bytes a step; MN-major: 16 rows of 128 bytes a step
              const int kmaj = (k16 % 4) * 32;
              const uint64_t ak =
                  adesc0 + soff + ((TRANS ? k16 / 4 * 128 * kGrBK * 2 + kmaj : k16 * 2048) >> 4);
              const uint64_t bk = bdesc0 + soff + ((k16 / 4 * C::kBHalf + kmaj) >> 4);
#pragma unroll
              for (int m = 0; m < NM; ++m)
                tc_mma_bf16(d + m * ROWS, ak + ((m * 128 * kGrBK * 2) >> 4), bk, idesc, acc | k16);
            }
            tc_commit(&empty[slot]);
            acc = issued = 1;
            if (++slot == kStages) {
              slot = 0;
              ph ^= 1u;
            }
          }
          if (ok) tc_commit(&acc_full[buf]);
        }
      }
      if (issued) {  // all MMAs complete before the tensor memory is freed
        tc_commit(drain);
        if (!mbar_wait_bounded(drain, 0, kWaitLimitNs)) atomicOr(a.status, kStatusTimeout);
      }
    }
  } else {
    // ------------------------------ epilogue ------------------------------
    // One TMEM lane (one weight column) per thread; the tile's rows are TMEM columns.  An fp32
    // result's pieces are added in sum[][].
    constexpr int kChunks = ROWS / 32;
    const int q = warp & 3, m = (warp - 2) >> 2;
    const uint32_t lane_base = tmem_base + ((uint32_t)(32 * q) << 16) + m * ROWS;
    int unit = 0, ti = 0;
    bool ok = true;
    Tile prev{};
    const int share = 128 / S;
    if (C::kSplit) cluster_wait();
    // Adds the S partial sums of this rank's columns of tile number i in rank order and writes
    // them, 4 columns of a row per thread; the same answer for all four warps.
    auto add_parts = [&](const Tile& w, int i, bool good) {
      const int pb = i & 1;
      if (good)
        good = warp_wait_cluster(&part_full[pb], (i >> 1) & 1u, abort_flag, a.status);
      const float* part = epi + pb * 128 * C::kPitch;
      for (int j = tid - 64; good && j < w.rows * (share / 4); j += 128) {
        const int r = j % w.rows, c4 = 4 * (j / w.rows), col = w.n0 + rank * share + c4;
        if (col >= a.Ncols) continue;
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int s = 0; s < S; ++s) {
          const float* p = part + (s * share + c4) * C::kPitch + r;
          v.x += p[0];
          v.y += p[C::kPitch];
          v.z += p[2 * C::kPitch];
          v.w += p[3 * C::kPitch];
        }
        store4<F32>(a.out, (size_t)(w.row0 + r) * a.Ncols + col, v);
      }
      good = named_bar_and(1, 128, good);
      if (good && tid - 64 < S)
        mbar_arrive_cluster(mapa_shared(smem_u32(&part_empty[pb]), tid - 64));
      return good;
    };
    for (int t = group; ok && t < tiles; t += groups, ++ti) {
      const Tile w = tile_at(t);
      int k0, k1;
      k_range(t, k0, k1);
      float sum[F32 ? kChunks : 1][32];
      if constexpr (F32) {
#pragma unroll
        for (int c = 0; c < kChunks; ++c)
#pragma unroll
          for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
        for (int p0 = k0; p0 < k1; p0 += piece, ++unit) {
          const int buf = unit % kBufs;
          ok = warp_wait(&acc_full[buf], (unit / kBufs) & 1u, abort_flag, a.status);
          if (!ok) break;
          tc_fence_after();
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (32 * c < w.rows) tmem_add32(lane_base + buf * NM * ROWS + 32 * c, sum[c]);
          tc_fence_before();
          mbar_arrive(&acc_empty[buf]);
        }
      }
      // rows 32 c .. 32 c + 31 of this thread's column
      const int buf = unit % kBufs;
      const bool any = !F32 && k1 > k0;   // one piece, still in tensor memory
      auto chunk = [&](int c, float (&v)[32]) {
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = sum[c][i];
        } else if (any) {
          tmem_ld32(lane_base + buf * NM * ROWS + 32 * c, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.f;
        }
      };
      if (ok && any) {
        ok = warp_wait(&acc_full[buf], (unit / kBufs) & 1u, abort_flag, a.status);
        tc_fence_after();
      }
      if constexpr (C::kSplit) {
        // Each rank adds and writes 128 / S of the tile's columns: every thread sends the rows of
        // its column to that column's rank.
        const int pb = ti & 1;
        if (ok)
          ok = warp_wait_cluster(&part_empty[pb], ((ti >> 1) & 1u) ^ 1u, abort_flag, a.status);
        if (ok) {
          if (tid == 64) mbar_arrive_expect_tx(&part_full[pb], 128u * 4u * ((w.rows + 3) & ~3));
          const int col = 32 * q + lane, dest = col / share;
          const uint32_t to = mapa_shared(
              smem_u32(epi + ((pb * S + rank) * share + col % share) * C::kPitch), dest);
          const uint32_t bar = mapa_shared(smem_u32(&part_full[pb]), dest);
#pragma unroll
          for (int c = 0; c < kChunks; ++c)
            if (32 * c < w.rows) {
              float v[32];
              chunk(c, v);
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                if (32 * c + i < w.rows)
                  st_async_f4(to + 4 * (32 * c + i), v[i], v[i + 1], v[i + 2], v[i + 3], bar);
            }
          if (any) {
            tc_fence_before();
            mbar_arrive(&acc_empty[buf]);
            ++unit;
          }
        }
        // a tile is added up after the next one's sums have left; either way the four warps agree
        // on going on (they meet at the same barriers)
        ok = ti > 0 ? add_parts(prev, ti - 1, ok) : named_bar_and(1, 128, ok);
        prev = w;
        if (!ok) break;
      } else if (ok) {
        float* stage = epi + (warp - 2) * 16 * C::kPitch;
        const int col0 = w.n0 + 128 * m + 32 * q;
#pragma unroll
        for (int c = 0; c < kChunks; ++c) {
          if (32 * c >= w.rows || col0 >= a.Ncols) continue;  // warp-uniform
          float v[32];
          chunk(c, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {   // 16 rows at a time
#pragma unroll
            for (int i = 0; i < 16; ++i) stage[i * C::kPitch + lane] = v[16 * h + i];
            __syncwarp();
            // 8 lanes cover the 32 columns of a row
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int r = 4 * i + (lane >> 3), row = 32 * c + 16 * h + r, cc = 4 * (lane & 7);
              const float* sp = stage + r * C::kPitch + cc;
              if (row < w.rows && col0 + cc < a.Ncols)
                store4<F32>(a.out, (size_t)(w.row0 + row) * a.Ncols + col0 + cc,
                            make_float4(sp[0], sp[1], sp[2], sp[3]));
            }
            __syncwarp();
          }
        }
        if (any) {
          tc_fence_before();
          mbar_arrive(&acc_empty[buf]);
          ++unit;
        }
      }
    }
    if (C::kSplit && ok && ti > 0) ok = add_parts(prev, ti - 1, true);
    if (C::kSplit && !ok) {
      // gave up: let what was sent to the other CTAs land before they may leave
      const uint64_t t0 = globaltimer_ns();
      while (globaltimer_ns() - t0 < 100000) {
      }
    }
  }

  if (C::kSplit && warp < 2) {
    __syncwarp();
    cluster_wait();
  }
  tc_fence_before();
  __syncthreads();
  if (C::kSplit) cluster_sync_all();  // no CTA leaves while another reads its sums
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem_base, C::kTmemCols);
}

// ------------------------------------------------------------------------------------------------
// CTA pairs: 256 x 256 result tiles.  Shared by the many-row product and the weight gradient.
//
// The even CTA issues the MMAs, so it has to learn when both CTAs have read an accumulator.  Its own
// epilogue threads arrive on acc_empty; the odd CTA's arrive on their CTA's `drained`, and that
// CTA's otherwise idle MMA lane passes each completed phase on.  (An arrival across the cluster
// releases at cluster scope, which waits for the arriving thread's global stores: from the
// epilogue threads it cost 1.3 us a tile.)
// ------------------------------------------------------------------------------------------------
constexpr int kPairStages = 6;
constexpr int kPairHalf = 128;                                 // rows and columns staged per CTA
constexpr int kPairABytes = kPairHalf * kGrBK * 2;             // 16 KB
constexpr int kPairStageBytes = 2 * kPairABytes;               // 32 KB per CTA
constexpr int kPairEpiWarps = 8;                               // two per TMEM lane quarter
constexpr int kPairEpiPitch = 36;                              // 32-bit words per staged row of 32
constexpr int kPairEpiBytes = kPairEpiWarps * 16 * kPairEpiPitch * 4;
constexpr int kPairSmem = 1024 + kPairStages * kPairStageBytes + 256 + kPairEpiBytes;
constexpr int kPairThreads = 64 + 32 * kPairEpiWarps;
constexpr int kWgradThreads = kPairThreads + 64;   // + warps that mask ragged ends and report it
static_assert(kPairSmem + (int)sizeof(Segments) + 64 <= 227 * 1024, "shared memory");
static_assert(128 * 260 * 4 <= kPairStages * kPairStageBytes, "exchange of a split tile");

// Half of the columns of a matrix's last 256-column block, rounded up to 16: what each CTA stages of
// it, so that the block's MMAs cover no more columns than it holds (2880 columns end in a block of
// 64).  The block of tile t is t % NT in both kernels.
MOE_DEVINL int last_half(int ncols, int NT) { return (ncols - 256 * (NT - 1) + 31) / 32 * 16; }

// Arrives on the barrier at this offset in both CTAs of the pair (mask: their bits) when the
// tcgen05 operations that this thread issued have completed.
MOE_DEVINL void commit_pair(uint64_t* bar, uint16_t mask) {
  asm volatile(
      "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], "
      "%1;" ::"r"(smem_u32(bar)),
      "h"(mask)
      : "memory");
}

// One warp's 32 rows x 128 bytes (32 words w per lane, lane = row) to columns col0 .. of `out` (row
// stride ld, first row row0), 16 rows at a time through shared memory so that eight lanes write
// one whole 128-byte line (64 bytes a row ran at half HBM's write rate).  rows_ok: valid rows of
// the 32.
template <bool F32>
MOE_DEVINL void pair_store(const uint32_t* w, uint32_t* stage, int lane, void* out, size_t row0,
                           int rows_ok, int col0, int ld) {
  const int col = col0 + (lane & 7) * (F32 ? 4 : 8);
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (lane >> 4 == h) {
      uint4* mine = reinterpret_cast<uint4*>(stage + (lane & 15) * kPairEpiPitch);
#pragma unroll
      for (int i = 0; i < 8; ++i)
        mine[i] = make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int r = 4 * i + (lane >> 3);
      const uint4 v = *reinterpret_cast<const uint4*>(stage + r * kPairEpiPitch + 4 * (lane & 7));
      if (16 * h + r < rows_ok && col < ld)
        *reinterpret_cast<uint4*>(static_cast<uint8_t*>(out) +
                                  ((row0 + 16 * h + r) * ld + col) * (F32 ? 4 : 2)) = v;
    }
    __syncwarp();
  }
}

// Odd CTA, one lane: passes the completed phases of `drained` for the accumulators unit ..
// unit + pieces - 1 on to the acc_empty of the even CTA, number `even` of the cluster.
MOE_DEVINL bool pair_relay(int pieces, int& unit, uint64_t* drained, uint64_t* acc_empty, int even,
                           volatile int* abort_flag, uint32_t* status) {
  for (int p = 0; p < pieces; ++p, ++unit) {
    const int buf = unit & 1;
    if (!wait_or_abort(&drained[buf], (unit >> 1) & 1u, abort_flag, status)) return false;
    mbar_arrive_cluster(mapa_shared(smem_u32(&acc_empty[buf]), even));
  }
  return true;
}

// Adds the `pieces` accumulators of a tile (32 rows x 128 columns of this warp) up in sum[][].
// mine: whether this warp's part is wanted.  Returns false when a wait gave up.
MOE_DEVINL bool pair_collect(uint32_t taddr, int pieces, int& unit, uint64_t* acc_full,
                             uint64_t* acc_read, bool mine, float (&sum)[4][32],
                             volatile int* abort_flag, uint32_t* status) {
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int i = 0; i < 32; ++i) sum[c][i] = 0.f;
  for (int p = 0; p < pieces; ++p, ++unit) {
    const int buf = unit & 1;
    if (!warp_wait(&acc_full[buf], (unit >> 1) & 1u, abort_flag, status)) return false;
    tc_fence_after();
    if (mine) {
#pragma unroll
      for (int c = 0; c < 4; ++c) tmem_add32(taddr + buf * 256 + 32 * c, sum[c]);
    }
    tc_fence_before();
    mbar_arrive(&acc_read[buf]);
  }
  return true;
}

// The epilogue of one tile for one warp: 32 rows (TMEM lanes of its quarter) x 128 columns, from
// `pieces` accumulators in turn.  taddr: this warp's lanes and first column in buffer 0.  unit: the
// accumulators handed over so far.  rows_ok <= 0: nothing to write, the hand-over only.
// pieces = 0 writes zeros.  acc_read: this CTA's acc_empty or drained.  Returns false when a wait
// gave up.  PIECES: whether a bf16 result may have more than one accumulator, and is summed as an
// fp32 one.
template <bool F32, bool PIECES>
MOE_DEVINL bool pair_epilogue(uint32_t taddr, int pieces, int& unit, uint64_t* acc_full,
                              uint64_t* acc_read, uint32_t* stage, int lane, void* out,
                              size_t row0, int rows_ok, int col0, int ld, volatile int* abort_flag,
                              uint32_t* status) {
  const bool mine = rows_ok > 0 && col0 < ld;   // warp-uniform
  if constexpr (F32) {
    float sum[4][32];
    if (!pair_collect(taddr, pieces, unit, acc_full, acc_read, mine, sum, abort_flag, status))
      return false;
    if (!mine) return true;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = __float_as_uint(sum[c][i]);
      pair_store<true>(w, stage, lane, out, row0, rows_ok, col0 + 32 * c, ld);
    }
  } else if constexpr (PIECES) {
    float sum[4][32];
    if (!pair_collect(taddr, pieces, unit, acc_full, acc_read, mine, sum, abort_flag, status))
      return false;
    if (!mine) return true;
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i)
        w[i] = cvt_bf16x2(sum[2 * c + i / 16][2 * (i % 16)], sum[2 * c + i / 16][2 * (i % 16) + 1]);
      pair_store<false>(w, stage, lane, out, row0, rows_ok, col0 + 64 * c, ld);
    }
  } else {
    const int buf = unit & 1;
    if (pieces > 0) {
      if (!warp_wait(&acc_full[buf], (unit >> 1) & 1u, abort_flag, status)) return false;
      tc_fence_after();
    }
    // all 128 columns into registers first: the accumulator is free while they are stored
    uint32_t w[2][32];
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (mine && pieces > 0) {
        float v[32];
        tmem_ld32(taddr + buf * 256 + 32 * c, v);
#pragma unroll
        for (int i = 0; i < 16; ++i) w[c / 2][16 * (c % 2) + i] = cvt_bf16x2(v[2 * i], v[2 * i + 1]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[c / 2][16 * (c % 2) + i] = 0u;
      }
    }
    if (pieces > 0) {
      tc_fence_before();
      mbar_arrive(&acc_read[buf]);
      ++unit;
    }
    if (mine) {
#pragma unroll
      for (int c = 0; c < 2; ++c)
        pair_store<false>(w[c], stage, lane, out, row0, rows_ok, col0 + 64 * c, ld);
    }
  }
  return true;
}

// Many rows per expert.  Tile: 256 rows of one expert x 256 columns; each CTA of the pair stages
// its 128 rows of x (K-major) and 128 of the weight columns (MN-major, or K-major for the
// transposed product), the even CTA issues MMAs over both, and each CTA's tensor memory receives
// its 128 rows x 256 columns.  Rows of a chunk past the segment's end are computed (they are
// other experts' rows, or zero past R) and never stored.
template <bool TRANS, bool F32>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kPairThreads, 1)
    grouped_rows_kernel(const GroupedArgs a, const __grid_constant__ CUtensorMap wmap,
                        const __grid_constant__ CUtensorMap xmap) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  uint8_t* ring = align1k(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kPairStages * kPairStageBytes);
  uint64_t* empty = full + kPairStages;
  uint64_t* acc_full = empty + kPairStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;   // odd CTA: its epilogue has read the accumulator
  uint64_t* drain = drained + 2;
  uint32_t* epi = reinterpret_cast<uint32_t*>(ring + kPairStages * kPairStageBytes + 256);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int rank = (int)cluster_ctarank();
  const bool leader = rank == 0;

  if (warp == 1) {
    tmem_alloc_2sm(&s_tmem, 512);
    tmem_relinquish_2sm();
  }
  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 32 * kPairEpiWarps + 1);   // even CTA's threads, odd CTA's relay
      mbar_init(&drained[b], 32 * kPairEpiWarps);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    fence_barrier_init();
    tma_prefetch_desc(&wmap);
    tma_prefetch_desc(&xmap);
  }
  pdl_wait();  // offsets, rows and weights may come from the previous kernels
  pdl_launch_next();
  load_segments(seg, a.offsets, a.E, a.R, 256, a.status);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;

  const int NT = (a.Ncols + 255) / 256;
  const int tiles = seg.base[a.E] * NT;
  const int nk = (a.Kred + kGrBK - 1) / kGrBK;
  const int piece = F32 ? kGrPieceStages : nk;
  const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
  volatile int* abort_flag = &s_abort;

  // Tile t: the column blocks of one chunk are neighbours, so the pairs that run together share
  // a few chunks of rows and one expert's weights in L2.
  struct Tile { int e, row0, rows, n0; };
  auto tile_at = [&](int t) {
    Tile w;
    w.e = find_expert(seg, a.E, NT, t);
    const int local = t - seg.base[w.e] * NT;
    const int ch = local / NT;
    w.n0 = (local - ch * NT) * 256;
    w.row0 = seg.beg[w.e] + ch * 256;
    w.rows = min(256, seg.cnt[w.e] - ch * 256);
    return w;
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------------------
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), 0);   // the even CTA's full[0]
      uint32_t issued = 0, ph = 0;
      int slot = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles && !*abort_flag; t += npairs) {
        const Tile w = tile_at(t);
        const int half = t % NT == NT - 1 ? last_half(a.Ncols, NT) : kPairHalf;
        const int row0 = w.row0 + rank * kPairHalf, col0 = w.n0 + rank * half;
        const bool two = !TRANS && half > 64;   // 64-column boxes
        const uint32_t bytes = kPairABytes + (TRANS || two ? kPairABytes : kPairABytes / 2);
        for (int k = 0; k < a.Kred; k += kGrBK) {
          if (!wait_or_abort(&empty[slot], ph ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          const uint32_t bar = full0 + 8 * slot;
          if (leader) mbar_arrive_expect_tx(&full[slot], 2 * bytes);
          uint8_t* st = ring + slot * kPairStageBytes;
          tma_load_2d_pair(st, &xmap, k, row0, bar);
          if (TRANS) {
            tma_load_3d_pair(st + kPairABytes, &wmap, k, col0, w.e, bar);
          } else {
            tma_load_3d_pair(st + kPairABytes, &wmap, col0, k, w.e, bar);
            if (two)
              tma_load_3d_pair(st + kPairABytes + 64 * kGrBK * 2, &wmap, col0 + 64, k, w.e, bar);
          }
          ++issued;
          if (++slot == kPairStages) {
            slot = 0;
            ph ^= 1u;
          }
        }
      }
      // the even CTA's full barriers count both CTAs' copies: drain them before the pair exits
      if (leader)
        for (uint32_t j = issued - min(issued, (uint32_t)kPairStages); j < issued; ++j)
          if (!mbar_wait_bounded(&full[j % kPairStages], (j / kPairStages) & 1u, kWaitLimitNs))
            atomicOr(a.status, kStatusTimeout);
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (even CTA) ------------------------------
    if (leader && lane == 0) {
      constexpr uint32_t idesc_all = idesc_bf16_f32(256, 256, false, !TRANS);
      const uint32_t idesc_last = idesc_bf16_f32(256, 2 * last_half(a.Ncols, NT), false, !TRANS);
      const uint32_t ring_s = smem_u32(ring);
      const uint64_t adesc0 = smem_desc_sw128(ring_s, 16, 1024);
      const uint64_t bdesc0 = TRANS ? smem_desc_sw128(ring_s + kPairABytes, 16, 1024)
                                    : smem_desc_sw128(ring_s + kPairABytes, 64 * kGrBK * 2, 1024);
      constexpr int kBStep = TRANS ? 32 : 16 * 128;
      // slot and phase are counted, not divided out: this lane's instructions bound the rate
      int slot = 0, unit = 0;
      uint32_t ph = 0, issued = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles && !*abort_flag; t += npairs) {
        const uint32_t idesc = t % NT == NT - 1 ? idesc_last : idesc_all;
        for (int p0 = 0; ok && p0 < nk; p0 += piece, ++unit) {
          const int p1 = min(nk, p0 + piece);
          const int buf = unit & 1;
          if (!wait_or_abort(&acc_empty[buf], ((unit >> 1) & 1u) ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * 256;
          uint32_t acc = 0;
          for (int kst = p0; kst < p1; ++kst) {
            if (!wait_or_abort(&full[slot], ph, abort_flag, a.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t soff = (uint64_t)((slot * kPairStageBytes) >> 4);
#pragma unroll
            for (int k16 = 0; k16 < kGrBK / 16; ++k16)
              tc_mma_bf16_2sm(d, adesc0 + soff + ((k16 * 32) >> 4),
                              bdesc0 + soff + ((k16 * kBStep) >> 4), idesc, acc | k16);
            commit_pair(&empty[slot], 3);
            acc = issued = 1;
            if (++slot == kPairStages) {
              slot = 0;
              ph ^= 1u;
            }
          }
          if (ok) {
            commit_pair(&acc_full[buf], 3);
          }
        }
      }
      if (issued) {  // all MMAs complete before the tensor memory is freed
        tc_commit_2sm(smem_u32(drain));
        if (!mbar_wait_bounded(drain, 0, kWaitLimitNs)) atomicOr(a.status, kStatusTimeout);
      }
    }
    if (!leader && lane == 0) {
      const int pieces = (nk + piece - 1) / piece;
      int unit = 0;
      for (int t = pair; t < tiles; t += npairs)
        if (!pair_relay(pieces, unit, drained, acc_empty, 0, abort_flag, a.status)) break;
    }
  } else {
    // ------------------------------ epilogue (both CTAs) ------------------------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + 128 * half;
    uint32_t* stage = epi + (warp - 2) * 16 * kPairEpiPitch;
    uint64_t* acc_read = leader ? acc_empty : drained;
    const int pieces = (nk + piece - 1) / piece;
    const int r0 = rank * kPairHalf + 32 * q;   // this warp's first row of a tile
    int unit = 0;
    for (int t = pair; t < tiles; t += npairs) {
      const Tile w = tile_at(t);
      if (!pair_epilogue<F32, false>(taddr, pieces, unit, acc_full, acc_read, stage, lane, a.out,
                                     (size_t)w.row0 + r0, w.rows - r0, w.n0 + 128 * half, a.Ncols,
                                     abort_flag, a.status))
        break;
    }
  }

  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_2sm(tmem_base, 512);
}

// Rows per accumulator of a weight-gradient tile (whole stages), and the accumulators that cnt rows
// take.
template <bool F32>
MOE_DEVINL constexpr int wgrad_piece() { return F32 ? kGrPieceStages * kGrBK : kGrPieceRowsBf16; }
template <bool F32>
MOE_DEVINL int wgrad_pieces(int cnt) { return (cnt + wgrad_piece<F32>() - 1) / wgrad_piece<F32>(); }

// Weight gradient.  Tile: 256 x 256 of dW[e]; the reduction runs over e's rows, 64 per stage,
// from x [R, M] and dy [R, Ncols] as they lie (both MN-major: 64 x 64 boxes).  A segment's last
// stage may hold rows of the next expert: a warp of each CTA overwrites them with zeros in both
// operands (zeroing one would let a NaN or an infinity of the other through) before the MMAs
// read them, up to the next multiple of 16; the MMAs stop there.  Such a stage's copies complete
// on a barrier of their own CTA; then the even CTA's warp completes the stage's `full` phase, the
// odd CTA's its `masked` phase, which a lane of a warp of its own passes on, and the MMA lane
// waits for both.  No thread that writes memory arrives across the cluster, and ordinary stages take no
// arrival from the odd CTA: the release waits for the thread's writes (0.45 us a stage from the
// producer lane, half the kernel's rate; 0.5 us a tile from the masking warp).
// Experts without rows get zeros.  The masking and reporting warps skip tiles without a ragged end, so
// they may wait for their next one through most of a call, and a call can outlast the limit of a wait
// (1.6 million rows of 32768 x 32768): their limit counts from the producer's last copies.
//
// SPLIT: where the tiles are too few for the GPU, a cluster of `pairs` (2 or 4) CTA pairs takes one
// tile, each pair a run of the segment's stages.  Afterwards every CTA holds partial sums of its
// 128 rows of the tile; CTA (pair p, half h) gets those of its 128 / pairs rows from the other
// pairs' CTAs of half h through distributed shared memory (the rings, idle by then), adds them in
// pair order and writes them.
//
// PIECES: calls whose segments may be longer than one bf16 accumulator takes (the host knows R
// only).  Both ways in one kernel spilled, and cost the calls without such segments 3 %; summing
// always costs them 2 % (8192 tokens, 2880 x 2880: 489 us, 503-514, 497-501).
template <bool F32, bool SPLIT, bool PIECES>
__global__ void __launch_bounds__(kWgradThreads, 1)
    grouped_wgrad_kernel(const GroupedArgs a, const __grid_constant__ CUtensorMap xmap,
                         const __grid_constant__ CUtensorMap dymap, const int pairs) {
  extern __shared__ __align__(128) uint8_t smem_raw[];
  __shared__ Segments seg;
  __shared__ uint32_t s_tmem;
  __shared__ int s_abort;
  __shared__ uint32_t s_progress;   // changes as the producer goes round the ring
  uint8_t* ring = align1k(smem_raw);
  uint64_t* full = reinterpret_cast<uint64_t*>(ring + kPairStages * kPairStageBytes);
  uint64_t* empty = full + kPairStages;
  uint64_t* ragged = empty + kPairStages;   // this CTA's copies of a stage that gets masked
  uint64_t* masked = ragged + kPairStages;       // odd CTA: it has masked its part of a stage
  uint64_t* peer_masked = masked;                // even CTA: the odd CTA has
  uint64_t* acc_full = masked + kPairStages;
  uint64_t* acc_empty = acc_full + 2;
  uint64_t* drained = acc_empty + 2;   // odd CTA: its epilogue has read the accumulator
  uint64_t* drain = drained + 2;
  uint32_t* epi = reinterpret_cast<uint32_t*>(ring + kPairStages * kPairStageBytes + 256);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int cta = (int)cluster_ctarank();
  const int rank = cta & 1, even = cta & ~1;   // half of the pair, its even CTA
  const bool leader = rank == 0;

  if (warp == 1) {
    tmem_alloc_2sm(&s_tmem, 512);
    tmem_relinquish_2sm();
  }
  if (tid == 0) {
    for (int s = 0; s < kPairStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
      mbar_init(&ragged[s], 1);
      mbar_init(&masked[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&acc_full[b], 1);
      mbar_init(&acc_empty[b], 32 * kPairEpiWarps + 1);   // even CTA's threads, odd CTA's relay
      mbar_init(&drained[b], 32 * kPairEpiWarps);
    }
    mbar_init(drain, 1);
    s_abort = 0;
    s_progress = 0;
    fence_barrier_init();
    tma_prefetch_desc(&xmap);
    tma_prefetch_desc(&dymap);
  }
  pdl_wait();  // offsets and rows may come from the previous kernels
  pdl_launch_next();
  load_segments(seg, a.offsets, a.E, a.R, 1, a.status);
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  const uint32_t tmem_base = s_tmem;

  const int NT = (a.Ncols + 255) / 256, MT = (a.M + 255) / 256;
  const int per = NT * MT, tiles = a.E * per;
  // SPLIT: one tile per cluster; else the pairs walk the tiles
  const int pair = SPLIT ? (int)blockIdx.x / (2 * pairs) : (int)blockIdx.x >> 1;
  const int npairs = SPLIT ? tiles : (int)gridDim.x >> 1;
  volatile int* abort_flag = &s_abort;
  volatile uint32_t* progress = &s_progress;
  // This pair's rows [r0, r1) of an expert's cnt.
  struct Range { int r0, r1; };
  auto range_of = [&](int cnt) {
    if (!SPLIT) return Range{0, cnt};
    const long long stages = (cnt + kGrBK - 1) / kGrBK;
    const int p = cta >> 1;
    return Range{min(cnt, (int)(stages * p / pairs) * kGrBK),
                 min(cnt, (int)(stages * (p + 1) / pairs) * kGrBK)};
  };

  if (warp == 0) {
    // ------------------------------ TMA producer (both CTAs) ------------------------------
    if (lane == 0) {
      const uint32_t full0 = mapa_shared(smem_u32(full), even);   // the even CTA's full[0]
      uint32_t issued = 0, ph = 0;
      uint32_t ragged_ph = 0;     // bit s: parity of the next masked stage in slot s
      uint32_t last_ragged = 0;   // bit s: slot s's last stage was a masked one
      int slot = 0;
      bool ok = true;
      for (int t = pair; ok && t < tiles && !*abort_flag; t += npairs) {
        const int e = t / per, l = t - e * per;
        const int half = t % NT == NT - 1 ? last_half(a.Ncols, NT) : kPairHalf;
        const int m0 = l / NT * 256 + rank * kPairHalf, n0 = l % NT * 256 + rank * half;
        const bool two = half > 64;   // 64-column boxes
        const uint32_t bytes = kPairABytes + (two ? kPairABytes : kPairABytes / 2);
        const int beg = seg.beg[e], cnt = seg.cnt[e];
        const Range rg = range_of(cnt);
        for (int r = rg.r0; r < rg.r1; r += kGrBK) {
          if (!wait_or_abort(&empty[slot], ph ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          uint8_t* st = ring + slot * kPairStageBytes;
          constexpr int kBox = 64 * kGrBK * 2;
          if (cnt - r >= kGrBK) {
            const uint32_t bar = full0 + 8 * slot;
            if (leader) mbar_arrive_expect_tx(&full[slot], 2 * bytes);
            tma_load_2d_pair(st, &xmap, m0, beg + r, bar);
            tma_load_2d_pair(st + kBox, &xmap, m0 + 64, beg + r, bar);
            tma_load_2d_pair(st + 2 * kBox, &dymap, n0, beg + r, bar);
            if (two) tma_load_2d_pair(st + 3 * kBox, &dymap, n0 + 64, beg + r, bar);
            last_ragged &= ~(1u << slot);
          } else {
            mbar_arrive_expect_tx(&ragged[slot], bytes);
            tma_load_2d(st, &xmap, m0, beg + r, &ragged[slot]);
            tma_load_2d(st + kBox, &xmap, m0 + 64, beg + r, &ragged[slot]);
            tma_load_2d(st + 2 * kBox, &dymap, n0, beg + r, &ragged[slot]);
            if (two) tma_load_2d(st + 3 * kBox, &dymap, n0 + 64, beg + r, &ragged[slot]);
            last_ragged |= 1u << slot;
            ragged_ph ^= 1u << slot;
          }
          ++issued;
          if (++slot == kPairStages) {
            slot = 0;
            ph ^= 1u;
            *progress = issued;
          }
        }
      }
      // drain: a masked stage's copies are this CTA's own, the others are counted on the even
      // CTA's full barriers
      for (uint32_t j = issued - min(issued, (uint32_t)kPairStages); j < issued; ++j) {
        const int s = j % kPairStages;
        bool done = true;
        if ((last_ragged >> s) & 1u)
          done = mbar_wait_bounded(&ragged[s], ((ragged_ph >> s) & 1u) ^ 1u, kWaitLimitNs);
        if (leader) done = mbar_wait_bounded(&full[s], (j / kPairStages) & 1u, kWaitLimitNs) && done;
        if (!done) atomicOr(a.status, kStatusTimeout);
      }
    }
  } else if (warp == 1) {
    // ------------------------------ MMA issuer (even CTA) ------------------------------
    if (leader && lane == 0) {
      constexpr uint32_t idesc_all = idesc_bf16_f32(256, 256, true, true);
      const uint32_t idesc_last = idesc_bf16_f32(256, 2 * last_half(a.Ncols, NT), true, true);
      const uint32_t ring_s = smem_u32(ring);
      const uint64_t adesc0 = smem_desc_sw128(ring_s, 64 * kGrBK * 2, 1024);
      const uint64_t bdesc0 = smem_desc_sw128(ring_s + kPairABytes, 64 * kGrBK * 2, 1024);
      int slot = 0, unit = 0;
      uint32_t ph = 0, issued = 0, masked_ph = 0;   // bit s: parity of the next masked stage in slot s
      bool ok = true;
      for (int t = pair; ok && t < tiles && !*abort_flag; t += npairs) {
        const int cnt = seg.cnt[t / per];
        const uint32_t idesc = t % NT == NT - 1 ? idesc_last : idesc_all;
        const Range rg = range_of(cnt);
        constexpr int piece = wgrad_piece<F32>();
        for (int p0 = rg.r0; ok && p0 < rg.r1; p0 += piece, ++unit) {
          const int p1 = min(rg.r1, p0 + piece);
          const int buf = unit & 1;
          if (!wait_or_abort(&acc_empty[buf], ((unit >> 1) & 1u) ^ 1u, abort_flag, a.status)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t d = tmem_base + buf * 256;
          uint32_t acc = 0;
          for (int r = p0; r < p1; r += kGrBK) {
            if (!wait_or_abort(&full[slot], ph, abort_flag, a.status)) {
              ok = false;
              break;
            }
            const uint64_t ak = adesc0 + ((slot * kPairStageBytes) >> 4);
            const uint64_t bk = bdesc0 + ((slot * kPairStageBytes) >> 4);
            if (cnt - r >= kGrBK) {
              tc_fence_after();
#pragma unroll
              for (int k16 = 0; k16 < kGrBK / 16; ++k16)
                tc_mma_bf16_2sm(d, ak + ((k16 * 2048) >> 4), bk + ((k16 * 2048) >> 4), idesc, acc | k16);
            } else {
              const uint32_t mph = (masked_ph >> slot) & 1u;
              masked_ph ^= 1u << slot;
              if (!wait_or_abort_cluster(&peer_masked[slot], mph, abort_flag, a.status)) {
                ok = false;
                break;
              }
              tc_fence_after();
              for (int k16 = 0; k16 < (cnt - r + 15) / 16; ++k16)
                tc_mma_bf16_2sm(d, ak + ((k16 * 2048) >> 4), bk + ((k16 * 2048) >> 4), idesc, acc | k16);
            }
            commit_pair(&empty[slot], (uint16_t)(3 << even));
            acc = issued = 1;
            if (++slot == kPairStages) {
              slot = 0;
              ph ^= 1u;
            }
          }
          if (ok) {
            commit_pair(&acc_full[buf], (uint16_t)(3 << even));
          }
        }
      }
      if (issued) {  // all MMAs complete before the tensor memory is freed
        tc_commit_2sm(smem_u32(drain));
        if (!mbar_wait_bounded(drain, 0, kWaitLimitNs)) atomicOr(a.status, kStatusTimeout);
      }
    }
    if (!leader && lane == 0) {
      int unit = 0;
      for (int t = pair; t < tiles; t += npairs) {
        const Range rg = range_of(seg.cnt[t / per]);
        if (!pair_relay(wgrad_pieces<F32>(rg.r1 - rg.r0), unit, drained, acc_empty, even, abort_flag,
                        a.status))
          break;
      }
    }
  } else if (warp == 2 + kPairEpiWarps) {
    // ------------------------------ masking of ragged ends (both CTAs) ------------------------
    uint32_t it = 0, ragged_ph = 0;
    for (int t = pair; t < tiles; t += npairs) {
      const Range rg = range_of(seg.cnt[t / per]);   // r0 is a multiple of a stage
      const int rem = rg.r1 % kGrBK;
      it += (rg.r1 - rg.r0 + kGrBK - 1) / kGrBK;
      if (rg.r1 == rg.r0 || rem == 0) continue;
      const int slot = (it - 1) % kPairStages;
      const uint32_t ph = (ragged_ph >> slot) & 1u;
      ragged_ph ^= 1u << slot;
      if (!__all_sync(0xffffffffu, wait_or_abort_while(&ragged[slot], ph, progress, abort_flag, a.status)))
        break;
      // a row of a 64 x 64 box is 128 contiguous bytes (the swizzle permutes inside them)
      uint8_t* st = ring + slot * kPairStageBytes;
      const int pad = (16 - rem % 16) % 16;
      for (int i = lane; i < pad * 4 * 8; i += 32) {
        const int box = i / (pad * 8), j = i % (pad * 8);
        *reinterpret_cast<uint4*>(st + box * (64 * kGrBK * 2) + (rem + j / 8) * 128 + (j % 8) * 16) =
            make_uint4(0, 0, 0, 0);
      }
      if (pad > 0) fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(leader ? &full[slot] : &masked[slot]);
    }
  } else if (warp == 3 + kPairEpiWarps) {
    // ------------------------------ masked stages reported (odd CTA) ------------------------------
    if (!leader && lane == 0) {
      uint32_t it = 0, masked_ph = 0;
      for (int t = pair; t < tiles; t += npairs) {
        const Range rg = range_of(seg.cnt[t / per]);
        it += (rg.r1 - rg.r0 + kGrBK - 1) / kGrBK;
        if (rg.r1 == rg.r0 || rg.r1 % kGrBK == 0) continue;
        const int slot = (it - 1) % kPairStages;
        if (!wait_or_abort_while(&masked[slot], (masked_ph >> slot) & 1u, progress, abort_flag, a.status))
          break;
        masked_ph ^= 1u << slot;
        mbar_arrive_cluster(mapa_shared(smem_u32(&peer_masked[slot]), even));
      }
    }
  } else if (!SPLIT) {
    // ------------------------------ epilogue (both CTAs) ------------------------------
    const int q = warp & 3, half = (warp - 2) >> 2;
    const uint32_t taddr = tmem_base + ((uint32_t)(32 * q) << 16) + 128 * half;
    uint32_t* stage = epi + (warp - 2) * 16 * kPairEpiPitch;
    uint64_t* acc_read = leader ? acc_empty : drained;
    int unit = 0;
    for (int t = pair; t < tiles; t += npairs) {
      const int e = t / per, l = t - e * per;
      const int m0 = l / NT * 256 + rank * kPairHalf + 32 * q, n0 = l % NT * 256 + 128 * half;
      const int cnt = seg.cnt[e];
      if (!pair_epilogue<F32, PIECES>(taddr, wgrad_pieces<F32>(cnt), unit, acc_full, acc_read, stage, lane,
                                      a.out, (size_t)e * a.M + m0, a.M - m0, n0, a.Ncols, abort_flag,
                                      a.status))
        break;
    }
  }

  if constexpr (SPLIT) {
    // ------------------------------ exchange (tile `pair`, every warp) ------------------------
    const bool epi_warp = warp >= 2 && warp < 2 + kPairEpiWarps;
    const int q = warp & 3, half = (warp - 2) >> 2;
    const int e = pair / per, l = pair - e * per;
    const int m0 = l / NT * 256 + rank * kPairHalf, n0 = l % NT * 256;
    const int share = kPairHalf / pairs;           // rows of the tile that this CTA writes
    constexpr int kPitch = 260;                    // floats per row of 256 in the exchange
    float sum[4][32];
    if (epi_warp) {
      const Range rg = range_of(seg.cnt[e]);
      int unit = 0;
      pair_collect(tmem_base + ((uint32_t)(32 * q) << 16) + 128 * half,
                   wgrad_pieces<F32>(rg.r1 - rg.r0), unit, acc_full, leader ? acc_empty : drained,
                   true, sum, abort_flag, a.status);
    }
    __syncwarp();
    cluster_sync_all();   // no CTA of the cluster has copies or MMAs on its ring any more
    if (epi_warp) {
      const int row = 32 * q + lane;
      const uint32_t to = mapa_shared(
          smem_u32(ring) + 4u * (((cta >> 1) * share + row % share) * kPitch + 128 * half),
          2 * (row / share) + rank);
#pragma unroll
      for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int i = 0; i < 32; i += 4)
          asm volatile("st.shared::cluster.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(
                           to + 4 * (32 * c + i)),
                       "f"(sum[c][i]), "f"(sum[c][i + 1]), "f"(sum[c][i + 2]), "f"(sum[c][i + 3])
                       : "memory");
    }
    __syncwarp();
    cluster_sync_all();   // every CTA has the sums of its rows
    if (epi_warp) {
      const float* part = reinterpret_cast<const float*>(ring);
      const int row0 = m0 + (cta >> 1) * share;
      for (int i = tid - 64; i < share * 64; i += 32 * kPairEpiWarps) {
        const int r = i / 64, c4 = 4 * (i % 64);
        if (row0 + r >= a.M || n0 + c4 >= a.Ncols) continue;
        float4 v = *reinterpret_cast<const float4*>(part + r * kPitch + c4);
        for (int p = 1; p < pairs; ++p) {
          const float4 o = *reinterpret_cast<const float4*>(part + (p * share + r) * kPitch + c4);
          v = make_float4(v.x + o.x, v.y + o.y, v.z + o.z, v.w + o.w);
        }
        store4<F32>(a.out, ((size_t)e * a.M + row0 + r) * a.Ncols + n0 + c4, v);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  cluster_sync_all();
  tc_fence_after();
  if (warp == 1) tmem_dealloc_2sm(tmem_base, 512);
}

}  // namespace moe
