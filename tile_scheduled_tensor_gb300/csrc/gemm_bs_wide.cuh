// Block-scaled FP8 GEMM, 128 x 256 tiles of D, one scale of B per 128 columns and k-block: the
// conditions and the sum of gemm_bs_tile.cuh, for problems with tiles enough for every SM.
//
// A 128 x 128 tile brings 32 KB into shared memory per k-block of 128, 512 cycles at the 64 bytes a
// cycle that an SM takes in by TMA (measured; with nothing added to the sums the 128-column kernel
// still takes 550 cycles), against 256 of tensor-core work.  Twice the columns bring 48 KB for twice
// the work: 384 cycles per 128 x 128.  Four stages of 48 KB, two partials of 256 TMEM columns, and
// 128 sums per accumulating thread, for which the role warpgroup gives registers up:
//   warps 0-3   producer, MMA issuers 0 and 1 (k-blocks of even and odd count, each into its own
//               partial, so that one waits while the other's MMAs run), and a warp that fills the
//               group table
//   warps 4-11  accumulate: two per TMEM quadrant, 128 columns each, 16 at a time with the next 16's
//               load in flight (32 and 32 spill: 640 cycles per 64 columns against 170)
// 16384 rows over 16 experts of 4096 x 4096 (550 GFLOP): 255 us with one set of inputs over and over, 0.56
// of twice the measured BF16 rate, and 270 to 279 with inputs in turn, at the clocks that the power cap
// then leaves; 330 with 128 x 128 tiles.  What bounds it now is the accumulating warps' chain per k-block (750
// cycles: 340 adding, the rest waiting, handing over and storing) before the 768 of its loads.
#pragma once
#include "gemm_bs_tile.cuh"

namespace tst {

struct WideCfg {
  static constexpr int A_BYTES = 128 * 128;
  static constexpr int B_BYTES = 256 * 128;
  static constexpr int STAGES = 4;
  static constexpr int STAGING_OFFSET = STAGES * (A_BYTES + B_BYTES);
  static constexpr int WALK_OFFSET = STAGING_OFFSET + 8 * kTileStaging;
  static constexpr int BAR_OFFSET = (WALK_OFFSET + kWalkBytes + 7) / 8 * 8;
  static constexpr int STAT_OFFSET = BAR_OFFSET + (2 * STAGES + 2 * 2 + 1) * 8;   // the accumulating warps' counters (debug)
  static constexpr int MISC_OFFSET = STAT_OFFSET + 3 * 8;
  static constexpr int SMEM_BYTES = 1024 + MISC_OFFSET + 16;
  static_assert(SMEM_BYTES <= kSmemLimit, "fits an SM");
};
constexpr int kWideRoleRegs = 56, kWideSumRegs = 224;
static_assert(128 * kWideRoleRegs + 256 * kWideSumRegs <= kBsTileThreads * kTileLaunchRegs, "the split fits the launch");

// MMA issuer r, one thread: the k-blocks whose count over this CTA's tiles has parity r, each into
// partial r.  Each stage has one reader, which commits EMPTY.  PEMPTY is waited for before FULL: it shows
// that every k-block up to q - 2 has landed, without which a ring of three stages could take FULL's
// parity for an earlier use's.
__device__ __forceinline__ void wide_mma(const KernelParams& p, const Ctx& c, Walk walk, uint32_t r, uint32_t tmem_base,
                                         uint32_t smem_a, uint32_t smem_b, uint32_t bar_full, uint32_t bar_empty,
                                         uint32_t bar_pfull, uint32_t bar_pempty, uint32_t bar_drain) {
  const uint32_t idesc = ptx::make_idesc(0u, kBlockM, 256) | p.fmt_ab;
  const uint64_t a_desc0 = ptx::sw128_kmajor_desc(smem_a);
  const uint64_t b_desc0 = ptx::sw128_kmajor_desc(smem_b);
  const uint32_t d = tmem_base + r * 256u;
  int stage = 0;
  uint32_t phase = 0, q = 0;
  bool ok = true;
  long long wait_full = 0, wait_pempty = 0;   // role-cycle counters (debug)
  const bool stats = p.stats != nullptr && r == 0;
  const int nkb = p.sched.kt;
  while (ok && walk.skip()) {
    for (int kb = 0; kb < nkb; ++kb, ++q) {
      if ((q & 1u) == r) {
        const long long t0 = stats ? clock64() : 0;
        if (!wait_phase<1>(p, c, bar_pempty + 8 * r, ((q >> 1) & 1u) ^ 1u, ROLE_MMA)) { ok = false; break; }
        const long long t1 = stats ? clock64() : 0;
        if (!wait_phase<1>(p, c, bar_full + 8 * stage, phase, ROLE_MMA)) { ok = false; break; }
        if (stats) { wait_pempty += t1 - t0; wait_full += clock64() - t1; }
        ptx::tc_fence_after();
        const uint64_t a_desc = a_desc0 + static_cast<uint64_t>(stage * (WideCfg::A_BYTES >> 4));
        const uint64_t b_desc = b_desc0 + static_cast<uint64_t>(stage * (WideCfg::B_BYTES >> 4));
#pragma unroll
        for (int i = 0; i < 4; ++i)   // 32 bytes of K per MMA; the first overwrites
          ptx::mma_f8(d, a_desc + 2 * i, b_desc + 2 * i, idesc, i != 0);
        ptx::mma_commit(bar_empty + 8 * stage);
        ptx::mma_commit(bar_pfull + 8 * r);
      }
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
  }
  if (stats) {
    p.stats[blockIdx.x * kStatSlots + STAT_MMA_WAIT_FULL] = wait_full;
    p.stats[blockIdx.x * kStatSlots + STAT_MMA_WAIT_TEMPTY] = wait_pempty;   // partials
    p.stats[blockIdx.x * kStatSlots + STAT_KBLOCKS] = q;                     // both issuers'
  }
  // every MMA this issuer issued completes before TMEM is released (the drain barrier counts both)
  ptx::mma_commit(bar_drain);
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar_drain, 0)) {
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      raise_error<1>(p, c, ST_TIMEOUT, ROLE_MMA);
      break;
    }
  }
}

template <int OUT>
__device__ __forceinline__ void run_epilogue_wide(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base,
                                                  uint32_t bar_pfull, uint32_t bar_pempty, uint8_t* staging,
                                                  long long* counters) {
  const int warp = (threadIdx.x >> 5) - 4;   // 0-7 among the accumulating warps
  const int lane = threadIdx.x & 31;
  const int group = warp >> 2;               // which 128 columns of the tile
  const int quad = warp & 3;                 // TMEM lane quadrant this warp may access
  uint8_t* const stage = staging + warp * kTileStaging;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(group * 128);
  uint32_t q = 0;   // k-blocks of this CTA so far: k-block q is in partial q & 1
  bool ok = true;
  const bool stat_thread = p.stats != nullptr && threadIdx.x == 128;   // warp 4, lane 0
  // debug counters in shared memory: {waiting, in tiles, tiles}; registers are short here
  if (stat_thread) counters[0] = counters[1] = counters[2] = 0;
  auto wait_partial = [&] {
    const long long t0 = stat_thread ? clock64() : 0;
    ok = wait_phase_warp(p, c, bar_pfull + 8 * (q & 1u), (q >> 1) & 1u, ROLE_EPILOGUE);
    if (stat_thread) counters[0] += clock64() - t0;
    ptx::tc_fence_after();
  };
  auto release = [&] {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar_pempty + 8 * (q & 1u));
  };
  const int nkb = p.sched.kt;
  const int32_t ncols = p.N;
  Tile w;
  while (ok && walk.next_warp(w)) {
    const int32_t row0 = w.row0 + quad * 32, col0 = w.n * 256 + group * 128;
    if (row0 >= w.row_end || col0 >= ncols) {   // this warp has nothing of the tile
      for (int i = 0; i < nkb && ok; ++i, ++q) {
        wait_partial();
        if (ok && lane == 0) ptx::mbar_arrive(bar_pempty + 8 * (q & 1u));
      }
      continue;
    }
    if (stat_thread) counters[1] -= clock64();
    const int32_t row = row0 + lane < p.M ? row0 + lane : p.M - 1;   // rows past the end are not stored
    const float* sa_row = p.bs_a + static_cast<int64_t>(row / p.bs_rows) * p.bs_kblocks;
    const float* sb_row = p.bs_b + (static_cast<int64_t>(w.group) * p.bs_group_rows + col0 / p.bs_rows_b) * p.bs_kblocks;
    float na = __ldg(sa_row), nb = __ldg(sb_row);   // the next k-block's scales
    float r[128];
#pragma unroll
    for (int j = 0; j < 128; ++j) r[j] = 0.0f;
#pragma unroll 1
    for (int kb = 0; kb < nkb; ++kb) {
      const float s = na * nb;
      const int32_t kn = kb + 1 < nkb ? kb + 1 : kb;
      na = __ldg(sa_row + kn);   // in flight until the next k-block
      nb = __ldg(sb_row + kn);
      wait_partial();
      if (!ok) break;
      const uint32_t taddr = taddr0 + (q & 1u) * 256u;
      uint32_t va[16], vb[16];
      auto fold = [&](const uint32_t (&v)[16], float* sum) {
#pragma unroll
        for (int i = 0; i < 16; i += 2) ptx::fma_f32x2_after(sum[i], sum[i + 1], s, v[i], v[i + 1]);
      };
      ptx::tmem_load_16cols_async(taddr, va);
#pragma unroll
      for (int chunk = 0; chunk < 8; chunk += 2) {
        ptx::tmem_wait_loads();
        ptx::tmem_load_16cols_async(taddr + static_cast<uint32_t>(16 * (chunk + 1)), vb);
        fold(va, r + 16 * chunk);
        ptx::tmem_wait_loads();
        if (chunk < 6) ptx::tmem_load_16cols_async(taddr + static_cast<uint32_t>(16 * (chunk + 2)), va);
        else release();   // the partial's last columns are in registers
        fold(vb, r + 16 * (chunk + 1));
      }
      ++q;
    }
    if (ok) {
      // the basic epilogue on the block-scaled sum: alpha, column bias, ReLU, cast, store
      float alpha = p.alpha;
      if (p.use_scales) alpha = alpha * __ldg(p.scales) * __ldg(p.scales + 1);
      if (p.has_bias) {
#pragma unroll
        for (int i = 0; i < 128; ++i) r[i] = fmaf(alpha, r[i], col0 + i < ncols ? __ldg(p.bias + col0 + i) : 0.0f);
      } else {
#pragma unroll
        for (int i = 0; i < 128; ++i) r[i] = fmaf(alpha, r[i], 0.0f);
      }
      if (p.relu) {
#pragma unroll
        for (int i = 0; i < 128; ++i) r[i] = fmaxf(r[i], 0.0f);
      }
      constexpr int PIECE = OUT == OUT_BF16 ? 32 : 16;
      const bool whole_rows = ncols % (OUT == OUT_BF16 ? 8 : 4) == 0;
#pragma unroll
      for (int i = 0; i < 128; i += PIECE) {
        if (whole_rows && col0 + i + PIECE <= ncols) {
          store_rows<OUT>(p, stage, lane, row0, w.row_end, ncols, col0 + i, r + i);
        } else if (row0 + lane < w.row_end) {
          const int64_t at = static_cast<int64_t>(row0 + lane) * ncols + col0 + i;
#pragma unroll
          for (int k = 0; k < PIECE; ++k)
            if (col0 + i + k < ncols) {
              if (OUT == OUT_BF16) reinterpret_cast<__nv_bfloat16*>(p.C)[at + k] = __float2bfloat16_rn(r[i + k]);
              else reinterpret_cast<float*>(p.C)[at + k] = r[i + k];
            }
        }
      }
    }
    if (stat_thread) {
      counters[1] += clock64();
      counters[2] += 1;
    }
  }
  if (stat_thread) {
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_WAIT_TFULL] = counters[0];
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_BUSY] = counters[1] - counters[0];
    p.stats[blockIdx.x * kStatSlots + STAT_ITEMS] = counters[2];
  }
}

template <int OUT>
__global__ void __launch_bounds__(kBsTileThreads, 1) gemm_bs_wide_kernel(const __grid_constant__ KernelParams p) {
  using Cfg = WideCfg;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_a = ptx::smem_addr(smem);
  const uint32_t smem_b = smem_a + Cfg::STAGES * Cfg::A_BYTES;
  const uint32_t bar_full = smem_a + Cfg::BAR_OFFSET;
  const uint32_t bar_empty = bar_full + 8 * Cfg::STAGES;
  const uint32_t bar_pfull = bar_empty + 8 * Cfg::STAGES;
  const uint32_t bar_pempty = bar_pfull + 8 * 2;
  const uint32_t bar_drain = bar_pempty + 8 * 2;
  const GroupTable table(smem + Cfg::WALK_OFFSET);
  SharedCtl* ctl = reinterpret_cast<SharedCtl*>(smem + Cfg::MISC_OFFSET);
  const int warp = threadIdx.x >> 5;
  const long long t_start = clock64();

  Ctx c;
  c.abort = &ctl->abort;
  c.abort_addr = ptx::smem_addr(&ctl->abort);
  c.rank = 0;
  c.rank_m = 0;
  c.rank_n = 0;
  c.csize = 1;
  c.unit = static_cast<int32_t>(blockIdx.x);

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::STAGES; ++s) {
      ptx::mbar_init(bar_full + 8 * s, 1);
      ptx::mbar_init(bar_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2; ++b) {
      ptx::mbar_init(bar_pfull + 8 * b, 1);
      ptx::mbar_init(bar_pempty + 8 * b, kBsWarps);
    }
    ptx::mbar_init(bar_drain, 2);
    ctl->abort = 0;
    ctl->ep_ok = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_a);
    ptx::prefetch_tmap(&p.tmap_b);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), 512);
    ptx::tmem_relinquish();
  }
  if (warp == 3 && p.sched.groups > 0) fill_group_table(p.sched, table);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const Walk walk(p.sched, table, c.unit);

  if (warp < 4) {
    ptx::setmaxnreg_dec<kWideRoleRegs>();
    if (warp == 0) {
      if (ptx::elect_one())
        bs_producer<128, 256>(p, c, walk, smem_a, Cfg::A_BYTES, smem_b, Cfg::B_BYTES, bar_full, bar_empty);
    } else if (warp < 3) {
      if (ptx::elect_one())
        wide_mma(p, c, walk, static_cast<uint32_t>(warp - 1), tmem_base, smem_a, smem_b, bar_full, bar_empty, bar_pfull,
                 bar_pempty, bar_drain);
    }
    __syncwarp();
  } else {
    ptx::setmaxnreg_inc<kWideSumRegs>();
    run_epilogue_wide<OUT>(p, c, walk, tmem_base, bar_pfull, bar_pempty, smem + Cfg::STAGING_OFFSET,
                           reinterpret_cast<long long*>(smem + Cfg::STAT_OFFSET));
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (p.stats && threadIdx.x == 0) p.stats[blockIdx.x * kStatSlots + STAT_TOTAL] = clock64() - t_start;
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace tst
