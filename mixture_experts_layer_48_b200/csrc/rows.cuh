// Row-wise operators around the expert products, all bound by HBM: SwiGLU on rows [gate | up]
// with its backward pass, and the RMS norms before and after the block fused with its gate and
// residual scale, with their backward pass.
//
// One row is spread over TPR threads, VPT vectors of 4 (or 8) consecutive elements each, and
// stays in registers between the passes over it, so every input is read once and every output
// written once.  All arithmetic and every sum is fp32.  Sums over rows (the gradients of the norm
// weights and the gate) are kept in registers per thread over all rows of a persistent block,
// written as one partial row per row group and added in a fixed order by a second kernel: results
// do not depend on timing.
//
// Measured (graph replay, one B200, copy bandwidth 6.46 TB/s; rows of 2880): SwiGLU of 32,768 rows
// 86 us forward, 138 us backward (6.6 and 6.8 TB/s); norms of 8189 rows, bf16 residual and fp32
// block output, 42 us forward (5.6 TB/s: issue slots and row sums), of 32,768 rows backward 281 us with
// an fp32 residual (6.7 TB/s) and 237 us with a bf16 one (5.6 TB/s).
#pragma once

#include "common.cuh"
#include "grouped.cuh"
#include "ring.h"

namespace moe {

MOE_DEVINL float4 load4(const float* p) { return *reinterpret_cast<const float4*>(p); }
MOE_DEVINL float4 load4(const uint16_t* p) {
  const uint2 v = *reinterpret_cast<const uint2*>(p);
  return make_float4(bf16lo(v.x), bf16hi(v.x), bf16lo(v.y), bf16hi(v.y));
}
MOE_DEVINL void save4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
MOE_DEVINL void save4(uint16_t* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(cvt_bf16x2(v.x, v.y), cvt_bf16x2(v.z, v.w));
}
// v as the type of p holds it.
MOE_DEVINL float4 as_stored(const float*, float4 v) { return v; }
MOE_DEVINL float4 as_stored(const uint16_t*, float4 v) {
  const uint32_t a = cvt_bf16x2(v.x, v.y), b = cvt_bf16x2(v.z, v.w);
  return make_float4(bf16lo(a), bf16hi(a), bf16lo(b), bf16hi(b));
}

MOE_DEVINL float4 operator*(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
MOE_DEVINL float4 operator*(float4 a, float b) { return make_float4(a.x * b, a.y * b, a.z * b, a.w * b); }
MOE_DEVINL float4 fma4(float4 a, float4 b, float4 c) {
  return make_float4(fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y), fmaf(a.z, b.z, c.z),
                     fmaf(a.w, b.w, c.w));
}
MOE_DEVINL float4 fma4(float4 a, float b, float4 c) {
  return make_float4(fmaf(a.x, b, c.x), fmaf(a.y, b, c.y), fmaf(a.z, b, c.z), fmaf(a.w, b, c.w));
}
MOE_DEVINL float dot4(float4 a, float4 b) { return a.x * b.x + a.y * b.y + a.z * b.z + a.w * b.w; }

// How a row of n4 vectors lies on TPR threads: thread l holds vectors l, l + TPR, ... (VPT of
// them).  The launch picks (TPR, VPT) so that the first kFull of a thread's vectors exist for
// every thread; only the last ones are tested against the row's end.
template <int TPR, int VPT>
struct RowCfg {
  static constexpr int kThreads = TPR < 128 ? 128 : TPR;
  static constexpr int kRows = kThreads / TPR;   // rows per block
  static constexpr int kFull = VPT <= 4 ? VPT - 1 : VPT == 6 ? 4 : 6;
  static_assert(VPT <= 4 || VPT == 6 || VPT == 8, "by_row_length");
};

// Sum over the TPR threads of a row, the same value in each of them.  `red` has a word per warp
// of the block; every thread of the block takes part.  Calls in a row alternate between two such
// arrays, so that a call's words are read before the next but one overwrites them.
template <int TPR>
MOE_DEVINL float row_sum(float v, float* red) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xffffffffu, v, d);
  if constexpr (TPR > 32) {
    constexpr int W = TPR / 32;
    const int warp = threadIdx.x >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const float* mine = red + warp / W * W;
    v = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) v += mine[i];
  }
  return v;
}

// ---- norms around the block ---------------------------------------------------------------------
struct NormArgs {
  int T, H;
  float eps, scale;
  const void *resid, *y;                    // y null: no block output to add
  const float *w_post, *gate, *w_next;      // null: no norm after / no gate / no norm before
  void* resid_out;
  uint16_t* x;
  float *rstd_post, *rstd_next;             // forward: written
  // backward
  const void* dresid;                       // null: nothing flows into the new residual itself
  const uint16_t* dx;
  const float *c_rstd_post, *c_rstd_next;
  void *dresid_out, *dy;
  int dy_f32;
  float *part_y, *part_x;                   // [row groups, H] partial column sums, or null
  int stages, stage_bytes;                  // the ring of the staged kernels
  int lose_row;                             // rows from here on count as not arrived (self-test)
  uint32_t* status;
};

// scale * gate * w_post, all that either pass needs of the three.
MOE_DEVINL float4 post_factor(const NormArgs& a, int v) {
  float4 p = make_float4(a.scale, a.scale, a.scale, a.scale);
  if (a.gate != nullptr) p = p * load4(a.gate + 4 * v);
  if (a.w_post != nullptr) p = p * load4(a.w_post + 4 * v);
  return p;
}

// Blocks per SM of the staged kernels, by the registers that a thread's vectors take: forward 1024
// threads (64 registers) with three vectors a thread, 1280 (51) with fewer; backward 512 (128), 768
// (85) and 1024 (64).  A backward row on 512 threads with two vectors takes two blocks of 64
// registers, some of them spilled (16,000 rows of 4096: 199 us, 217 with one block).  More vectors:
// one block.  Rows of over 6144 spill there, backward, up to 744 bytes a thread with eight vectors: fp32
// residual and block output, 2^26 elements, 4.8 TB/s at rows of 8192 (282 us), 3.1 at 16384 (439 us);
// forward 5.4 and 4.8.
template <int TPR, int VPT>
constexpr int norm_forward_blocks() {
  return VPT > 3 ? 1 : (VPT == 3 ? 1024 : 1280) / RowCfg<TPR, VPT>::kThreads;
}
template <int TPR, int VPT>
constexpr int norm_backward_blocks() {
  return VPT > 3 ? 1 : (VPT == 3 ? 512 : VPT == 2 && TPR < 512 ? 768 : 1024) / RowCfg<TPR, VPT>::kThreads;
}
constexpr int kRowRingMax = 4;

// Thread 0: `rows` rows of row_bytes from g (null: none) to a stage, counted on its barrier.
MOE_DEVINL void ring_copy(uint8_t* to, const void* g, size_t row0, int rows, int row_bytes,
                          uint64_t* bar) {
  if (g != nullptr)
    bulk_g2s(to, static_cast<const uint8_t*>(g) + row0 * row_bytes, rows * row_bytes, bar);
}

// Thread 0, after a wait that gave up at row `lost` of a block's rows t, t + step, ... < T: waits for the
// copies that are still on their way, so that none lands in shared memory that another block has by
// then.
MOE_DEVINL void ring_drain(uint64_t* full, int stages, int t, int step, int T, int lost) {
  const int issued = ring_issued((lost - t) / step, stages, (T - t + step - 1) / step);
  for (int j = ring_oldest(issued, stages); j < issued; ++j)
    mbar_wait_bounded(&full[ring_slot(j, stages)], ring_parity(j, stages), kWaitLimitNs);
}

// r' = r + scale * gate * norm(y);  x = norm(r').  RT, YT: float or uint16_t (bf16).  One row a
// block (or kRows) from global memory; STAGED: persistent blocks that work as the backward kernel's.
template <int TPR, int VPT, typename RT, typename YT, bool STAGED>
__global__ void __launch_bounds__(RowCfg<TPR, VPT>::kThreads,
                                  STAGED ? norm_forward_blocks<TPR, VPT>() : 1)
    block_norm_kernel(const NormArgs a) {
  using C = RowCfg<TPR, VPT>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][C::kThreads / 32];
  __shared__ uint64_t full[kRowRingMax];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int n4 = a.H / 4;
  const float inv_h = 1.f / (float)a.H;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const int r_bytes = a.H * (int)sizeof(RT), y_bytes = a.H * (int)sizeof(YT);
  const int step = gridDim.x * C::kRows;
  auto fetch = [&](int t0, int slot) {   // thread 0
    const int rows = min(C::kRows, a.T - t0);
    uint64_t* bar = &full[slot];
    mbar_arrive_expect_tx(bar, rows * (r_bytes + (a.y != nullptr ? y_bytes : 0)));
    uint8_t* stage = ring + slot * a.stage_bytes;
    ring_copy(stage, a.resid, t0, rows, r_bytes, bar);
    ring_copy(stage + C::kRows * r_bytes, a.y, t0, rows, y_bytes, bar);
  };
  if (STAGED && threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_next();
  if (STAGED) {
    __syncthreads();
    if (threadIdx.x == 0)
      for (int s = 0, t0 = blockIdx.x * C::kRows; s < a.stages && t0 < a.T; ++s, t0 += step)
        fetch(t0, s);
  }
  constexpr int kHeld = STAGED ? VPT : 1;
  float4 w_next[kHeld], w_post[kHeld];
  if (STAGED) {
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = i * TPR + lane;
      w_next[i] = a.w_next != nullptr && v < n4 ? load4(a.w_next + 4 * v) : zero;
      w_post[i] = v < n4 ? post_factor(a, v) : zero;
    }
  }
  auto next_factor = [&](int i) { return STAGED ? w_next[i] : load4(a.w_next + 4 * (i * TPR + lane)); };
  auto y_factor = [&](int i) { return STAGED ? w_post[i] : post_factor(a, i * TPR + lane); };

  int slot = 0, turn = 0;
  uint32_t phase = 0;
  int lost = -1;          // first row whose copy this thread did not see arrive
  int t0 = blockIdx.x * C::kRows;
  do {
    const int t = t0 + sub;
    const bool live = C::kRows == 1 || t < a.T;
    auto ok = [&](int i) { return live && (i < C::kFull || i * TPR + lane < n4); };
    const size_t base = (size_t)t * a.H + 4 * lane;
    const RT* resid = static_cast<const RT*>(a.resid) + base;
    const YT* yrow = static_cast<const YT*>(a.y) + base;
    if (STAGED) {
      if (lost < 0 &&
          (t0 >= a.lose_row || !mbar_wait_bounded(&full[slot], phase, kWaitLimitNs))) {
        atomicOr(a.status, kStatusTimeout);
        lost = t0;
      }
      const uint8_t* stage = ring + slot * a.stage_bytes;
      const int at = sub * a.H + 4 * lane;
      resid = reinterpret_cast<const RT*>(stage) + at;
      yrow = reinterpret_cast<const YT*>(stage + C::kRows * r_bytes) + at;
    }
    bool refilled = !STAGED;
    auto refill = [&]() {   // after a barrier that follows the loads
      if (refilled) return;
      refilled = true;
      if (threadIdx.x == 0 && lost < 0 && t0 + (long long)a.stages * step < a.T)
        fetch(t0 + a.stages * step, slot);
      if (++slot == a.stages) {
        slot = 0;
        phase ^= 1u;
      }
    };
    float4 r[VPT], y[VPT];
#pragma unroll
    for (int i = 0; i < VPT; ++i) r[i] = ok(i) ? load4(resid + 4 * i * TPR) : zero;
    if (a.y != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) y[i] = ok(i) ? load4(yrow + 4 * i * TPR) : zero;
      float s = 1.f;
      if (a.w_post != nullptr) {
        float ss = 0.f;
#pragma unroll
        for (int i = 0; i < VPT; ++i) ss += dot4(y[i], y[i]);
        s = rsqrtf(row_sum<TPR>(ss, red[turn]) * inv_h + a.eps);
        turn ^= 1;
        if (STAGED && TPR == 32) __syncthreads();
        refill();
        if (live && lane == 0) a.rstd_post[t] = s;
      }
      RT* out = static_cast<RT*>(a.resid_out) + base;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (ok(i)) {
          const float4 q = fma4(y[i] * s, y_factor(i), r[i]);
          save4(out + 4 * i * TPR, q);
          r[i] = as_stored(out, q);   // the next norm reads what a reader of r' would
        }
    }
    if (a.x != nullptr) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i) ss += dot4(r[i], r[i]);
      const float s = rsqrtf(row_sum<TPR>(ss, red[turn]) * inv_h + a.eps);
      turn ^= 1;
      if (STAGED && TPR == 32) __syncthreads();
      refill();
      if (live && lane == 0) a.rstd_next[t] = s;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (ok(i)) save4(a.x + base + 4 * i * TPR, r[i] * s * next_factor(i));
    }
    if (STAGED && a.w_post == nullptr && a.x == nullptr) {
      __syncthreads();
      refill();
    }
    t0 += step;
  } while (STAGED && t0 < a.T);
  if (STAGED && lost >= 0 && threadIdx.x == 0)
    ring_drain(full, a.stages, blockIdx.x * C::kRows, step, a.T, lost);
}

// Backward.  With rh = r' * rstd_next and t = dx * w_next:
//   dr = dresid + rstd_next * (t - rh * mean(t * rh))                 gradient of r' and of r
// with yh = y * rstd_post (or y without the norm after) and d = scale * gate * dr * w_post:
//   dy = rstd_post * (d - yh * mean(d * yh))                          (or scale * gate * dr)
// column sums: part_x = sum dx * rh (dw_next), part_y = sum dr * yh (dw_post and dgate follow).
//
// Persistent blocks: the column sums stay in registers over all rows of a block.  STAGED: a
// block's next rows are on their way while it works on one, a bulk copy per operand into a ring
// of shared-memory stages, read into registers at the start of a step and refilled after the
// step's first block-wide barrier; the vectors are then held in registers too (the ring leaves
// too little L1 for them: loaded again for every row they cost more time than the row itself).
// Rows too long for a ring and those registers come straight from global memory.
template <int TPR, int VPT, typename RT, typename YT, bool STAGED>
__global__ void __launch_bounds__(RowCfg<TPR, VPT>::kThreads, norm_backward_blocks<TPR, VPT>())
    block_norm_backward_kernel(const NormArgs a) {
  using C = RowCfg<TPR, VPT>;
  extern __shared__ __align__(128) uint8_t ring[];
  __shared__ float red[2][C::kThreads / 32];
  __shared__ uint64_t full[kRowRingMax];
  const int lane = threadIdx.x % TPR, sub = threadIdx.x / TPR;
  const int n4 = a.H / 4;
  const float inv_h = 1.f / (float)a.H;
  const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
  const int r_bytes = a.H * (int)sizeof(RT), y_bytes = a.H * (int)sizeof(YT), x_bytes = a.H * 2;
  const int step = gridDim.x * C::kRows;
  auto fetch = [&](int t0, int slot) {   // thread 0
    const int rows = min(C::kRows, a.T - t0);
    uint64_t* bar = &full[slot];
    mbar_arrive_expect_tx(bar, rows * ((a.dresid != nullptr ? r_bytes : 0) +
                                       (a.dx != nullptr ? x_bytes + r_bytes : 0) +
                                       (a.y != nullptr ? y_bytes : 0)));
    uint8_t* stage = ring + slot * a.stage_bytes;
    ring_copy(stage, a.dresid, t0, rows, r_bytes, bar);
    ring_copy(stage + C::kRows * r_bytes, a.dx != nullptr ? a.resid : nullptr, t0, rows, r_bytes, bar);
    ring_copy(stage + 2 * C::kRows * r_bytes, a.dx, t0, rows, x_bytes, bar);
    ring_copy(stage + C::kRows * (2 * r_bytes + x_bytes), a.y, t0, rows, y_bytes, bar);
  };
  if (STAGED && threadIdx.x == 0) {
    for (int s = 0; s < a.stages; ++s) mbar_init(&full[s], 1);
    fence_barrier_init();
  }
  pdl_wait();
  pdl_launch_next();
  if (STAGED) {
    __syncthreads();
    if (threadIdx.x == 0)
      for (int s = 0, t0 = blockIdx.x * C::kRows; s < a.stages && t0 < a.T; ++s, t0 += step)
        fetch(t0, s);
  }
  constexpr int kHeld = STAGED ? VPT : 1;
  float4 w_next[kHeld], w_post[kHeld];
  float4 sum_x[VPT], sum_y[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + lane;
    sum_x[i] = sum_y[i] = zero;
    if (STAGED) {
      w_next[i] = a.w_next != nullptr && v < n4 ? load4(a.w_next + 4 * v) : zero;
      w_post[i] = v < n4 ? post_factor(a, v) : zero;
    }
  }
  auto next_factor = [&](int i) { return STAGED ? w_next[i] : load4(a.w_next + 4 * (i * TPR + lane)); };
  auto y_factor = [&](int i) { return STAGED ? w_post[i] : post_factor(a, i * TPR + lane); };

  // every thread of the block takes every step (the row sums are block-wide)
  int slot = 0, turn = 0;
  uint32_t phase = 0;
  int lost = -1;   // first row whose copy this thread did not see arrive: the status word says so, the
                   // rest is not waited for
  for (int t0 = blockIdx.x * C::kRows; t0 < a.T; t0 += step) {
    const int t = t0 + sub;
    const bool live = C::kRows == 1 || t < a.T;
    auto ok = [&](int i) { return live && (i < C::kFull || i * TPR + lane < n4); };
    const size_t base = (size_t)t * a.H + 4 * lane;
    float4 dr[VPT], dx[VPT], r[VPT], y[VPT];
    const RT* dres = static_cast<const RT*>(a.dresid) + base;
    const RT* res = static_cast<const RT*>(a.resid) + base;
    const uint16_t* dxrow = a.dx + base;
    const YT* yrow = static_cast<const YT*>(a.y) + base;
    if (STAGED) {
      if (lost < 0 &&
          (t0 >= a.lose_row || !mbar_wait_bounded(&full[slot], phase, kWaitLimitNs))) {
        atomicOr(a.status, kStatusTimeout);
        lost = t0;
      }
      const uint8_t* stage = ring + slot * a.stage_bytes;
      const int at = sub * a.H + 4 * lane;
      dres = reinterpret_cast<const RT*>(stage) + at;
      res = reinterpret_cast<const RT*>(stage + C::kRows * r_bytes) + at;
      dxrow = reinterpret_cast<const uint16_t*>(stage + 2 * C::kRows * r_bytes) + at;
      yrow = reinterpret_cast<const YT*>(stage + C::kRows * (2 * r_bytes + x_bytes)) + at;
    }
    // A barrier after the loads: the stage may be refilled.  The first row sum of a step is one.
    auto refill = [&]() {
      if (STAGED) {
        if (threadIdx.x == 0 && lost < 0 && t0 + (long long)a.stages * step < a.T)
          fetch(t0 + a.stages * step, slot);
        if (++slot == a.stages) {
          slot = 0;
          phase ^= 1u;
        }
      }
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) dr[i] = a.dresid != nullptr && ok(i) ? load4(dres + 4 * i * TPR) : zero;
    if (a.y != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) y[i] = ok(i) ? load4(yrow + 4 * i * TPR) : zero;
    }
    if (a.dx != nullptr) {
#pragma unroll
      for (int i = 0; i < VPT; ++i) {
        dx[i] = ok(i) ? load4(dxrow + 4 * i * TPR) : zero;
        r[i] = ok(i) ? load4(res + 4 * i * TPR) : zero;
      }
      const float s = live ? a.c_rstd_next[t] : 0.f;
      float c = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (ok(i)) {
          r[i] = r[i] * s;
          sum_x[i] = fma4(dx[i], r[i], sum_x[i]);
          dx[i] = dx[i] * next_factor(i);
          c += dot4(dx[i], r[i]);
        }
      c = row_sum<TPR>(c, red[turn]) * inv_h;
      turn ^= 1;
      if (TPR == 32) __syncthreads();
      refill();
#pragma unroll
      for (int i = 0; i < VPT; ++i) dr[i] = fma4(fma4(r[i], -c, dx[i]), s, dr[i]);
    } else {
      __syncthreads();
      refill();
    }
    RT* out = static_cast<RT*>(a.dresid_out) + base;
#pragma unroll
    for (int i = 0; i < VPT; ++i)
      if (ok(i)) save4(out + 4 * i * TPR, dr[i]);
    if (a.dy != nullptr) {
      const float s = a.w_post != nullptr && live ? a.c_rstd_post[t] : 1.f;
      float c = 0.f;
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (ok(i)) {
          if (a.y != nullptr) {
            y[i] = y[i] * s;
            sum_y[i] = fma4(dr[i], y[i], sum_y[i]);
          }
          dr[i] = dr[i] * y_factor(i);
          if (a.w_post != nullptr) c += dot4(dr[i], y[i]);
        }
      if (a.w_post != nullptr) {
        c = row_sum<TPR>(c, red[turn]) * inv_h;
        turn ^= 1;
#pragma unroll
        for (int i = 0; i < VPT; ++i) dr[i] = fma4(y[i], -c, dr[i]) * s;
      }
#pragma unroll
      for (int i = 0; i < VPT; ++i)
        if (ok(i)) {
          if (a.dy_f32) save4(static_cast<float*>(a.dy) + base + 4 * i * TPR, dr[i]);
          else save4(static_cast<uint16_t*>(a.dy) + base + 4 * i * TPR, dr[i]);
        }
    }
  }
  if (STAGED && lost >= 0 && threadIdx.x == 0)
    ring_drain(full, a.stages, blockIdx.x * C::kRows, step, a.T, lost);
  const size_t row = (size_t)(blockIdx.x * C::kRows + sub) * a.H;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + lane;
    if (v < n4) {
      if (a.part_x != nullptr) save4(a.part_x + row + 4 * v, sum_x[i]);
      if (a.part_y != nullptr) save4(a.part_y + row + 4 * v, sum_y[i]);
    }
  }
}

// dw_next[h] = sum_p part_x[p, h]; with S[h] = sum_p part_y[p, h]: dw_post = scale * gate * S and
// dgate = scale * w_post * S.  block 1024 = 32 columns x 32 slices of the partial rows, each slice
// added in row order, then the slices in order.  grid (ceil(H / 32), 2).
__global__ void __launch_bounds__(1024)
    block_norm_colsum_kernel(const float* __restrict__ part_x, const float* __restrict__ part_y,
                             int parts, int H, float scale, const float* __restrict__ gate,
                             const float* __restrict__ w_post, float* __restrict__ dw_next,
                             float* __restrict__ dw_post, float* __restrict__ dgate) {
  __shared__ float acc[32][33];
  pdl_wait();
  pdl_launch_next();
  const float* part = blockIdx.y == 0 ? part_x : part_y;
  if (part == nullptr) return;
  const int lane = threadIdx.x & 31, slice = threadIdx.x >> 5;
  const int h = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (h < H) {
    const int per = (parts + 31) / 32, p1 = min(parts, (slice + 1) * per);
#pragma unroll 4
    for (int p = slice * per; p < p1; ++p) s += part[(size_t)p * H + h];
  }
  acc[slice][lane] = s;
  __syncthreads();
  if (slice != 0 || h >= H) return;
#pragma unroll
  for (int i = 1; i < 32; ++i) s += acc[i][lane];
  if (blockIdx.y == 0) {
    dw_next[h] = s;
    return;
  }
  s *= scale;
  if (dw_post != nullptr) dw_post[h] = gate != nullptr ? s * gate[h] : s;
  if (dgate != nullptr) dgate[h] = w_post != nullptr ? s * w_post[h] : s;
}

// ---- SwiGLU on rows [gate | up] -----------------------------------------------------------------
MOE_DEVINL float sigmoid_f32(float z) { return __fdividef(1.f, 1.f + __expf(-z)); }

// h[r, :] = row_w[r] * silu(gu[r, :I]) * gu[r, I:] (row_w null: 1).  One thread per 8 elements.
__global__ void __launch_bounds__(256)
    swiglu_rows_kernel(const uint16_t* __restrict__ gu, const float* __restrict__ row_w,
                       uint16_t* __restrict__ h, int R, int I) {
  pdl_wait();
  pdl_launch_next();
  const int nv = I / 8;
  const long long n = (long long)R * nv;
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < n; i += (long long)gridDim.x * 256) {
    const int r = (int)(i / nv), v = (int)(i - (long long)r * nv);
    const uint16_t* row = gu + (size_t)r * 2 * I + 8 * v;
    const uint4 g = *reinterpret_cast<const uint4*>(row);
    const uint4 u = *reinterpret_cast<const uint4*>(row + I);
    const float w = row_w != nullptr ? row_w[r] : 1.f;
    auto one = [&](uint32_t a, uint32_t b) {
      const float g0 = bf16lo(a), g1 = bf16hi(a);
      return cvt_bf16x2(w * (g0 * sigmoid_f32(g0) * bf16lo(b)), w * (g1 * sigmoid_f32(g1) * bf16hi(b)));
    };
    *reinterpret_cast<uint4*>(h + (size_t)r * I + 8 * v) =
        make_uint4(one(g.x, u.x), one(g.y, u.y), one(g.z, u.z), one(g.w, u.w));
  }
}

// With s = sigmoid(g): du = w dh g s;  dg = w dh u s (1 + g (1 - s));  dw = sum dh g s u.
template <int TPR, int VPT>
__global__ void __launch_bounds__(RowCfg<TPR, VPT>::kThreads)
    swiglu_rows_backward_kernel(const uint16_t* __restrict__ dh, const uint16_t* __restrict__ gu,
                                const float* __restrict__ row_w, uint16_t* __restrict__ dgu,
                                float* __restrict__ drow_w, int R, int I) {
  constexpr int kRows = RowCfg<TPR, VPT>::kRows;
  __shared__ float red[RowCfg<TPR, VPT>::kThreads / 32];
  const int lane = threadIdx.x % TPR;
  const int r = blockIdx.x * kRows + threadIdx.x / TPR;
  const bool live = r < R;
  const int nv = live ? I / 8 : 0;
  pdl_wait();
  pdl_launch_next();
  const uint16_t* drow = dh + (size_t)r * I;
  const uint16_t* row = gu + (size_t)r * 2 * I;
  uint4 d[VPT], g[VPT], u[VPT];
  const uint4 zero = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + lane;
    d[i] = v < nv ? *reinterpret_cast<const uint4*>(drow + 8 * v) : zero;
    g[i] = v < nv ? *reinterpret_cast<const uint4*>(row + 8 * v) : zero;
    u[i] = v < nv ? *reinterpret_cast<const uint4*>(row + I + 8 * v) : zero;
  }
  const float w = row_w != nullptr && live ? row_w[r] : 1.f;
  float sum = 0.f;
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = i * TPR + lane;
    if (v >= nv) continue;
    uint32_t* dp = reinterpret_cast<uint32_t*>(&d[i]);
    uint32_t* gp = reinterpret_cast<uint32_t*>(&g[i]);
    uint32_t* up = reinterpret_cast<uint32_t*>(&u[i]);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float dg[2], du[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float dd = k ? bf16hi(dp[j]) : bf16lo(dp[j]);
        const float gg = k ? bf16hi(gp[j]) : bf16lo(gp[j]);
        const float uu = k ? bf16hi(up[j]) : bf16lo(up[j]);
        const float s = sigmoid_f32(gg), a = gg * s;
        sum = fmaf(dd * uu, a, sum);
        const float wd = w * dd;
        du[k] = wd * a;
        dg[k] = wd * uu * fmaf(a, 1.f - s, s);
      }
      gp[j] = cvt_bf16x2(dg[0], dg[1]);
      up[j] = cvt_bf16x2(du[0], du[1]);
    }
    uint16_t* out = dgu + (size_t)r * 2 * I + 8 * v;
    *reinterpret_cast<uint4*>(out) = g[i];
    *reinterpret_cast<uint4*>(out + I) = u[i];
  }
  if (drow_w != nullptr) {
    sum = row_sum<TPR>(sum, red);
    if (live && lane == 0) drow_w[r] = sum;
  }
}

}  // namespace moe
