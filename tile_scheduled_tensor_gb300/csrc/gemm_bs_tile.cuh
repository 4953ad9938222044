// Block-scaled FP8 GEMM where a 128 x 128 tile of D meets one scale of B per k-block: k-blocks of
// 128 and B's scale tiles a multiple of 128 rows high (1 x 128 tiles of A with 128 x 128 of B,
// 128 x 128 of both, ...).  The sum, the tile, the ring, the partials in Tensor Memory and the
// two issuers are those of gemm_blockscale.cuh; the accumulating warps are simpler and faster:
//
//   - the factor of a k-block is one number per row, s = sA[row][kb] sB[kb], so a thread needs 4
//     of them per window of 4 k-blocks.  It reads them from global memory into registers a window
//     ahead: no scales in shared memory, and no barrier among the warps, which each run at their
//     own pace;
//   - a warp whose 32 rows are past the end of its group loads and adds nothing;
//   - grouped plans find their tiles in a table (group_walk.cuh);
//   - single-thread roles run under elect.sync: a barrier wait costs the thread that issues MMAs
//     130 cycles there, 266 under a test of the lane number (measured; the 4 MMAs of a k-block
//     are 256 cycles of tensor-core work).
//
// 8192 x 8192 x 8192 in 536 us, 0.54 of twice the measured BF16 rate (the general form: 789).  Bound by the
// 32 KB per k-block that come in by TMA, 512 cycles, and the handshakes that the accumulation adds.
#pragma once
#include "gemm_blockscale.cuh"
#include "group_walk.cuh"

namespace tst {

// TMA producer by one thread: A_ROWS x 128 bytes of A and B_ROWS x 128 of B per stage, at smem_a and
// smem_b + stage * their strides.
template <int A_ROWS, int B_ROWS = 128>
__device__ __forceinline__ void bs_producer(const KernelParams& p, const Ctx& c, Walk walk, uint32_t smem_a, uint32_t stride_a,
                                            uint32_t smem_b, uint32_t stride_b, uint32_t bar_full, uint32_t bar_empty) {
  constexpr uint32_t STAGE_BYTES = (A_ROWS + B_ROWS) * 128;
  int stage = 0;
  uint32_t phase = 0, issued = 0, issued_parity = 0;
  bool ok = true;
  int32_t seq = 0;
  long long wait_empty = 0;
  const bool hint = p.l2_hint != 0;
  uint64_t pol_a = 0, pol_b = 0;
  if (hint) {
    const uint64_t keep = ptx::l2_policy_evict_last(), normal = ptx::l2_policy_evict_normal();
    pol_a = p.l2_hint == 1 ? keep : normal;
    pol_b = p.l2_hint == 1 ? normal : keep;
  }
  const int32_t nkb = p.sched.kt;
  Tile w;
  while (ok && walk.next(w)) {
    if (p.trace != nullptr && seq < p.max_items) {
      int32_t* rec = p.trace + (static_cast<int64_t>(c.unit) * p.max_items + seq) * 8;
      rec[0] = c.unit; rec[1] = seq; rec[2] = w.index; rec[3] = w.m;
      rec[4] = w.n; rec[5] = 0; rec[6] = nkb; rec[7] = ITEM_FINAL | (w.clamped ? ITEM_CLAMPED : 0);
    }
    if (w.clamped) record_status(p, ST_DEVICE_CHECK, ROLE_PRODUCER);
    const int32_t b_row0 = w.group * p.sched.group_b_rows + w.n * B_ROWS;
    for (int32_t kb = 0; kb < nkb; ++kb) {
      const long long t0 = p.stats ? clock64() : 0;
      if (!wait_phase<1>(p, c, bar_empty + 8 * stage, phase ^ 1u, ROLE_PRODUCER)) { ok = false; break; }
      if (p.stats) wait_empty += clock64() - t0;
      const uint32_t bar = bar_full + 8 * stage, da = smem_a + stage * stride_a, db = smem_b + stage * stride_b;
      ptx::mbar_arrive_expect_tx(bar, STAGE_BYTES);
      if (!((p.debug_flags & DBG_SKIP_LOAD) && seq == 0 && kb == 0)) {
        if (hint) {
          ptx::tma_load_2d_hint(db, &p.tmap_b, bar, kb * 128, b_row0, pol_b);
          ptx::tma_load_2d_hint(da, &p.tmap_a, bar, kb * 128, w.row0, pol_a);
        } else {
          ptx::tma_load_2d(db, &p.tmap_b, bar, kb * 128, b_row0);
          ptx::tma_load_2d(da, &p.tmap_a, bar, kb * 128, w.row0);
        }
      }
      issued |= 1u << stage;
      issued_parity = (issued_parity & ~(1u << stage)) | (phase << stage);
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
    }
    ++seq;
  }
  if (p.stats) p.stats[blockIdx.x * kStatSlots + STAT_PROD_WAIT_EMPTY] = wait_empty;
  if (!ok) {   // aborting: wait (bounded) until the loads already issued have landed
    const uint64_t t0 = ptx::globaltimer();
    for (int s = 0; s < p.stages; ++s) {
      if (!(issued & (1u << s))) continue;
      while (!ptx::mbar_try_wait(bar_full + 8 * s, (issued_parity >> s) & 1u))
        if (ptx::globaltimer() - t0 > p.timeout_ns) break;
    }
  }
}

// the issuers' view of the walk: every tile takes the whole K
struct WalkK {
  Walk walk;
  int32_t kt;
  __device__ __forceinline__ bool next() { return walk.skip(); }
  __device__ __forceinline__ int32_t k_count() const { return kt; }
};

// wait_phase for a converged warp, which follows one verdict
__device__ __forceinline__ bool wait_phase_warp(const KernelParams& p, const Ctx& c, uint32_t bar, uint32_t parity,
                                                uint32_t role) {
  return __all_sync(0xFFFFFFFFu, wait_phase<1>(p, c, bar, parity, role));
}

constexpr int kTileWindow = 4;   // k-blocks whose scales a thread holds (8 spilled 280 bytes)

// The scales of one row for k-blocks kb .. kb + 3 (past the last: the last again).
__device__ __forceinline__ void load_scales(const float* row, int32_t kb, int32_t kblocks, bool whole, float (&v)[kTileWindow]) {
  if (whole) {   // 16-byte loads where the rows of scales are whole multiples of them
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + kb));
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
  } else {
#pragma unroll
    for (int i = 0; i < kTileWindow; ++i) v[i] = __ldg(row + (kb + i < kblocks ? kb + i : kblocks - 1));
  }
}

// Warps 4-11 accumulate: two per TMEM quadrant, 64 columns each.
constexpr int kTileLaunchRegs = 168; // 65536 / 384, in steps of 8: what the block is launched with
constexpr int kTileRoleRegs = 56, kTileSumRegs = 216;
static_assert(128 * kTileRoleRegs + 256 * kTileSumRegs <= kBsTileThreads * kTileLaunchRegs, "the split fits the launch");
constexpr int kTileStaging = 2048;   // per accumulating warp: 32 rows x 64 bytes of D

// A warp's 32 x 64-byte piece of D (32 BF16 or 16 FP32 columns; lane = row, 16-byte chunk q of row r
// at q ^ ((r >> 1) & 3)) through shared memory, so that four lanes store the 64 adjacent bytes of a
// row: whole 32-byte sectors, where a row per lane writes halves of 32 different ones.
template <int OUT>
__device__ __forceinline__ void store_rows(const KernelParams& p, uint8_t* stage, int lane, int32_t row0, int32_t row_end,
                                           int32_t ncols, int32_t col0, const float* z) {
  constexpr int EB = OUT == OUT_BF16 ? 2 : 4;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    uint4 pk;
    if (OUT == OUT_BF16) {
      uint32_t* u = reinterpret_cast<uint32_t*>(&pk);
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        __nv_bfloat162 two = __floats2bfloat162_rn(z[8 * q + 2 * h], z[8 * q + 2 * h + 1]);
        u[h] = *reinterpret_cast<uint32_t*>(&two);
      }
    } else {
      pk = make_uint4(__float_as_uint(z[4 * q]), __float_as_uint(z[4 * q + 1]), __float_as_uint(z[4 * q + 2]),
                      __float_as_uint(z[4 * q + 3]));
    }
    *reinterpret_cast<uint4*>(stage + lane * 64 + ((q ^ ((lane >> 1) & 3)) << 4)) = pk;
  }
  __syncwarp();
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = i * 8 + (lane >> 2), q = lane & 3;
    const uint4 pk = *reinterpret_cast<const uint4*>(stage + r * 64 + ((q ^ ((r >> 1) & 3)) << 4));
    if (row0 + r < row_end)
      *reinterpret_cast<uint4*>(static_cast<uint8_t*>(p.C) + (static_cast<int64_t>(row0 + r) * ncols + col0) * EB + q * 16) = pk;
  }
  __syncwarp();   // the piece is read before the next one is written
}

template <int OUT>
__device__ __forceinline__ void run_epilogue_tile(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base,
                                                  uint32_t bar_pfull, uint32_t bar_pempty, uint8_t* staging) {
  const int warp = (threadIdx.x >> 5) - 4;   // 0-7 among the accumulating warps
  const int lane = threadIdx.x & 31;
  const int group = warp >> 2;               // which 64 columns of the tile
  const int quad = warp & 3;                 // TMEM lane quadrant this warp may access
  const int row_in_tile = quad * 32 + lane;
  uint8_t* const stage = staging + warp * kTileStaging;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(group * 64);
  const bool whole = (p.bs_kblocks & 3) == 0 && ((reinterpret_cast<uintptr_t>(p.bs_a) | reinterpret_cast<uintptr_t>(p.bs_b)) & 15u) == 0;
  float alpha = p.alpha;
  if (p.use_scales) alpha = alpha * __ldg(p.scales) * __ldg(p.scales + 1);
  uint32_t q = 0;   // pairs of k-blocks of this CTA so far: pair q uses slot q & 1
  bool ok = true;
  const bool stat_thread = p.stats != nullptr && threadIdx.x == 128;   // warp 4, lane 0
  long long wait_pfull = 0, busy = 0, items = 0;
  // the scales of an item: this thread's row of A, the tile's row of B
  auto scale_rows = [&](const Tile& w, const float*& sa, const float*& sb) {
    const int32_t row = w.row0 + row_in_tile < p.M ? w.row0 + row_in_tile : p.M - 1;   // rows past the end are not stored
    sa = p.bs_a + static_cast<int64_t>(row / p.bs_rows) * p.bs_kblocks;
    sb = p.bs_b + (static_cast<int64_t>(w.group) * p.bs_group_rows + w.n * 128 / p.bs_rows_b) * p.bs_kblocks;
  };
  auto wait_pair = [&](uint32_t pair) {
    const long long t0 = stat_thread ? clock64() : 0;
    ok = wait_phase_warp(p, c, bar_pfull + 8 * (pair & 1u), (pair >> 1) & 1u, ROLE_EPILOGUE);
    if (stat_thread) wait_pfull += clock64() - t0;
    ptx::tc_fence_after();
  };
  auto release = [&](uint32_t pair) {
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar_pempty + 8 * (pair & 1u));
  };
  // 32 columns of the pair's k-block k, half h, left in flight
  auto load = [&](uint32_t pair, int k, int h, uint32_t (&v)[32]) {
    ptx::tmem_load_32cols_async(taddr0 + (2 * (pair & 1u) + static_cast<uint32_t>(k)) * 128u + static_cast<uint32_t>(32 * h), v);
  };
  auto fold = [&](float s, const uint32_t (&v)[32], float* r) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) ptx::fma_f32x2_after(r[i], r[i + 1], s, v[i], v[i + 1]);
  };
  Tile w, wn;
  bool have = walk.next_warp(w);
  const int nkb = p.sched.kt;
  const float *sa_row = nullptr, *sb_row = nullptr;
  float na[kTileWindow], nb[kTileWindow];   // the next window's scales
  if (have) {
    scale_rows(w, sa_row, sb_row);
    load_scales(sa_row, 0, p.bs_kblocks, whole, na);
    load_scales(sb_row, 0, p.bs_kblocks, whole, nb);
  }
  while (have && ok) {
    const bool have_next = walk.next_warp(wn);
    if (w.row0 + quad * 32 >= w.row_end) {   // this warp has no rows of the tile
      for (int i = 0; i < nkb && ok; i += 2, ++q) {
        wait_pair(q);
        if (ok && lane == 0) ptx::mbar_arrive(bar_pempty + 8 * (q & 1u));
      }
      if (have_next) {
        scale_rows(wn, sa_row, sb_row);
        load_scales(sa_row, 0, p.bs_kblocks, whole, na);
        load_scales(sb_row, 0, p.bs_kblocks, whole, nb);
      }
    } else {
      const long long t1 = stat_thread ? clock64() : 0;
      // half a k-block's columns at a time, the next half's load in flight while one is added: va
      // takes the first halves, vb the second
      float r[64];
      uint32_t va[32], vb[32];
#pragma unroll
      for (int j = 0; j < 64; ++j) r[j] = 0.0f;
      wait_pair(q);
      if (ok) load(q, 0, 0, va);
      for (int kb = 0; kb < nkb && ok; kb += kTileWindow) {
        float s[kTileWindow];
#pragma unroll
        for (int i = 0; i < kTileWindow; ++i) s[i] = na[i] * nb[i];
        // the next window's scales fly while this one is added
        int32_t kn = kb + kTileWindow;
        if (kn >= nkb) {
          kn = 0;
          if (have_next) scale_rows(wn, sa_row, sb_row);
        }
        load_scales(sa_row, kn, p.bs_kblocks, whole, na);
        load_scales(sb_row, kn, p.bs_kblocks, whole, nb);
#pragma unroll
        for (int j = 0; j < kTileWindow; j += 2) {
          const int left = nkb - kb - j;   // k-blocks from this pair on; an odd last one is alone
          if (left <= 0 || !ok) break;
          ptx::tmem_wait_loads();
          load(q, 0, 1, vb);
          fold(s[j], va, r);
          ptx::tmem_wait_loads();
          if (left > 1) {
            load(q, 1, 0, va);
            fold(s[j], vb, r + 32);
            ptx::tmem_wait_loads();
            load(q, 1, 1, vb);
            fold(s[j + 1], va, r);
            ptx::tmem_wait_loads();
          }
          release(q);   // the slot's last partials are in registers
          ++q;
          if (left > 2) {
            wait_pair(q);
            if (ok) load(q, 0, 0, va);
          }
          fold(left > 1 ? s[j + 1] : s[j], vb, r + 32);
        }
      }
      if (ok) {
        // the basic epilogue on the block-scaled sum: alpha, column bias, ReLU, cast, store
        const int32_t col0 = w.n * 128 + group * 64, row0 = w.row0 + quad * 32, ncols = p.N;
        if (p.has_bias) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            r[i] = fmaf(alpha, r[i], col0 + i < ncols ? __ldg(p.bias + col0 + i) : 0.0f);
        } else {
#pragma unroll
          for (int i = 0; i < 64; ++i) r[i] = fmaf(alpha, r[i], 0.0f);
        }
        if (p.relu) {
#pragma unroll
          for (int i = 0; i < 64; ++i) r[i] = fmaxf(r[i], 0.0f);
        }
        constexpr int PIECE = OUT == OUT_BF16 ? 32 : 16;
        if (col0 + 64 <= ncols && ncols % (OUT == OUT_BF16 ? 8 : 4) == 0) {
#pragma unroll
          for (int i = 0; i < 64; i += PIECE)
            store_rows<OUT>(p, stage, lane, row0, w.row_end, ncols, col0 + i, r + i);
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            float z[32];
#pragma unroll
            for (int i = 0; i < 32; ++i) z[i] = r[32 * h + i];
            store_chunk<OUT>(p.C, ncols, row0 + lane, w.row_end, col0 + 32 * h, z);
          }
        }
      }
      if (stat_thread) busy += clock64() - t1;
    }
    items += 1;
    w = wn;
    have = have_next;
  }
  if (stat_thread) {
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_WAIT_TFULL] = wait_pfull;
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_BUSY] = busy - wait_pfull;
    p.stats[blockIdx.x * kStatSlots + STAT_ITEMS] = items;
  }
}

template <int OUT>
__global__ void __launch_bounds__(kBsTileThreads, 1) gemm_bs_tile_kernel(const __grid_constant__ KernelParams p) {
  using Cfg = TileCfg<128, 1, 1>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t smem_a = ptx::smem_addr(smem);
  const uint32_t smem_b = smem_a + Cfg::STAGES * Cfg::A_BYTES;
  const uint32_t bar_full = smem_a + Cfg::BAR_OFFSET;
  const uint32_t bar_empty = bar_full + 8 * Cfg::STAGES;
  const uint32_t bar_pfull = bar_empty + 8 * Cfg::STAGES;
  const uint32_t bar_pempty = bar_pfull + 8 * kBsBuffers;
  const uint32_t bar_drain = bar_pempty + 8 * kBsBuffers;
  // the ring's last stage (p.stages < Cfg::STAGES) holds the group table and the staging of D
  static_assert(kWalkBytes <= Cfg::A_BYTES && 8 * kTileStaging <= Cfg::B_BYTES, "the last stage holds table and staging");
  const GroupTable table(smem + (Cfg::STAGES - 1) * Cfg::A_BYTES);
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
      ptx::mbar_init(bar_empty + 8 * s, 1);   // one issuer reads each stage
    }
    for (int b = 0; b < kBsPairSlots; ++b) {
      ptx::mbar_init(bar_pfull + 8 * b, 2);   // both issuers
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

  if (warp < 4) {   // one warpgroup: the producer, the issuers and a warp that has done its part
    ptx::setmaxnreg_dec<kTileRoleRegs>();
    if (warp == 0) {
      if (ptx::elect_one())
        bs_producer<128>(p, c, walk, smem_a, Cfg::A_BYTES, smem_b, Cfg::B_BYTES, bar_full, bar_empty);
    } else if (warp < 3) {
      if (ptx::elect_one())
        run_mma_bs<4>(p, c, WalkK{walk, p.sched.kt}, warp - 1, tmem_base, smem_a, smem_b, bar_full, bar_empty, bar_pfull, bar_pempty, bar_drain);
    }
    __syncwarp();
  } else {
    ptx::setmaxnreg_inc<kTileSumRegs>();
    run_epilogue_tile<OUT>(p, c, walk, tmem_base, bar_pfull, bar_pempty, smem + Cfg::STAGES * Cfg::A_BYTES + (Cfg::STAGES - 1) * Cfg::B_BYTES);
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
