// Block-scaled FP8 grouped GEMM for groups of few rows (a decoding step's tokens, fine-grained
// experts): the same sum as gemm_blockscale.cuh,
//
//   D[i][j] = epilogue( sum_kb sA[i][kb] sB[j][kb] sum_{k in kb} a_ik b_jk ),
//
// with the operands' places exchanged.  A 128-row tensor-core tile over a group of a few rows
// would hold mostly rows of other groups; here the 128 rows (TMEM lanes) are 128 columns of D,
// i.e. rows of B, and the instruction's N are NT = 16 or 32 rows of the group.  What bounds
// such groups is reading B once, so the ring holds little of A and the promotion adds NT sums per
// thread and k-block instead of 64 per thread of twice as many threads.
//
// Roles, 192 threads, two CTAs per SM (so that one's epilogue and start overlap the other's stream),
// persistent over the groups' NT x 128 tiles of D, k-blocks of 128:
//   warp 0     TMA producer: 128 x 128 bytes of B and NT x 128 of A per stage
//   warp 1     MMA issuer: per k-block wait for a free partial and the stage, four K = 32 MMAs
//              into the partial (the first overwriting), commit to EMPTY and PFULL
//   warps 2-5  a thread per column of D: per k-block load the NT partials of its lane, release the
//              buffer, add factor * partial; at the end alpha, bias, ReLU, cast, store.
// Where B's scale tiles are a multiple of 128 rows high (SHARED) the factor of a row and k-block,
// sA sB, is the same for all columns: the warps multiply them once into a table in shared memory,
// a window of 8 k-blocks at a time from values loaded a window before; else the table holds sA and
// each thread its column's sB.  Every wait is bounded as in the 128-row kernel.
// 64 rows over 32 experts of 4096 x 4096: 537 MB of B in 85 us, 0.93 of the copy rate (the general form: 130).
#pragma once
#include "gemm_bs_tile.cuh"

namespace tst {

template <int NT>
struct NarrowCfg {
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_BYTES = NT * 128;
  static constexpr int STAGE_BYTES = W_BYTES + X_BYTES;
  static constexpr int BUFS = 8;                            // k-block partials in TMEM
  static constexpr int TMEM_COLS = BUFS * NT;
  static constexpr int WINDOW_BYTES = kBsWindow * NT * 4;
  static constexpr int LIMIT = (228 * 1024 - 2 * 1024) / 2;   // dynamic shared memory of one of two CTAs per SM
  static constexpr int FIXED = 1024 + 2 * WINDOW_BYTES + kWalkBytes + 512;
  static constexpr int STAGES = (LIMIT - FIXED) / STAGE_BYTES;
  static constexpr int WINDOW_OFFSET = STAGES * STAGE_BYTES;
  static constexpr int WALK_OFFSET = WINDOW_OFFSET + 2 * WINDOW_BYTES;
  static constexpr int BAR_OFFSET = (WALK_OFFSET + kWalkBytes + 7) / 8 * 8;
  static constexpr int MISC_OFFSET = BAR_OFFSET + (2 * STAGES + 2 * BUFS + 1) * 8;
  static constexpr int SMEM_BYTES = 1024 + MISC_OFFSET + 16;
  static_assert(STAGE_BYTES % 1024 == 0 && SMEM_BYTES <= LIMIT, "swizzled tiles start on 1024 bytes; two CTAs fit an SM");
};

template <int NT>
__device__ __forceinline__ void narrow_mma(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, uint32_t smem,
                                           uint32_t bar_full, uint32_t bar_empty, uint32_t bar_pfull, uint32_t bar_pempty,
                                           uint32_t bar_drain) {
  using Cfg = NarrowCfg<NT>;
  // the exchanged operands exchange their formats too: the plan's A format is in bits 7-9, B's in 10-12
  const uint32_t fmt = ((p.fmt_ab >> 3) & (7u << 7)) | ((p.fmt_ab & (7u << 7)) << 3);
  const uint32_t idesc = ptx::make_idesc(0u, 128, NT) | fmt;
  const uint64_t w_desc0 = ptx::sw128_kmajor_desc(smem);
  const uint64_t x_desc0 = ptx::sw128_kmajor_desc(smem + Cfg::W_BYTES);
  int stage = 0, buf = 0;
  uint32_t phase = 0, buf_phase = 0;
  bool ok = true;
  long long wait_full = 0, wait_pempty = 0, kblocks = 0;
  while (ok && walk.skip()) {
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      const long long t0 = p.stats ? clock64() : 0;
      if (!wait_phase<1>(p, c, bar_pempty + 8 * buf, buf_phase ^ 1u, ROLE_MMA)) { ok = false; break; }
      const long long t1 = p.stats ? clock64() : 0;
      if (!wait_phase<1>(p, c, bar_full + 8 * stage, phase, ROLE_MMA)) { ok = false; break; }
      if (p.stats) { wait_pempty += t1 - t0; wait_full += clock64() - t1; ++kblocks; }
      ptx::tc_fence_after();
      const uint64_t w_desc = w_desc0 + static_cast<uint64_t>(stage * (Cfg::STAGE_BYTES >> 4));
      const uint64_t x_desc = x_desc0 + static_cast<uint64_t>(stage * (Cfg::STAGE_BYTES >> 4));
      const uint32_t d = tmem_base + static_cast<uint32_t>(buf * NT);
#pragma unroll
      for (int i = 0; i < 4; ++i)   // 32 bytes of K per MMA; the first overwrites
        ptx::mma_f8(d, w_desc + 2 * i, x_desc + 2 * i, idesc, i != 0);
      ptx::mma_commit(bar_empty + 8 * stage);
      ptx::mma_commit(bar_pfull + 8 * buf);
      if (++stage == p.stages) { stage = 0; phase ^= 1u; }
      if (++buf == Cfg::BUFS) { buf = 0; buf_phase ^= 1u; }
    }
  }
  if (p.stats) {
    p.stats[blockIdx.x * kStatSlots + STAT_MMA_WAIT_FULL] = wait_full;
    p.stats[blockIdx.x * kStatSlots + STAT_MMA_WAIT_TEMPTY] = wait_pempty;
    p.stats[blockIdx.x * kStatSlots + STAT_KBLOCKS] = kblocks;
  }
  // every MMA issued completes before TMEM is released
  ptx::mma_commit(bar_drain);
  const uint64_t t0 = ptx::globaltimer();
  while (!ptx::mbar_try_wait(bar_drain, 0)) {
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      raise_error<1>(p, c, ST_TIMEOUT, ROLE_MMA);
      break;
    }
  }
}

// r[q] += f[q] * v[q], or with one scale of B per column (f[q] * sb) * v[q]: the scales' product first,
// as in the other forms, since either scale times a partial may leave FP32's range where the product does
// not.  f is read by broadcast four at a time.
template <int N, bool SHARED>
__device__ __forceinline__ void narrow_fold(const float* f, float sb, const float (&v)[N], float* r) {
#pragma unroll
  for (int q = 0; q < N; q += 4) {
    float4 a = *reinterpret_cast<const float4*>(f + q);
    if constexpr (!SHARED) {
      ptx::mul_f32x2(a.x, a.y, sb, sb, a.x, a.y);
      ptx::mul_f32x2(a.z, a.w, sb, sb, a.z, a.w);
    }
    ptx::fma_f32x2(r[q], r[q + 1], a.x, a.y, v[q], v[q + 1]);
    ptx::fma_f32x2(r[q + 2], r[q + 3], a.z, a.w, v[q + 2], v[q + 3]);
  }
}

template <int NT, int OUT, bool SHARED>
__device__ __forceinline__ void narrow_epilogue(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base,
                                                uint32_t bar_pfull, uint32_t bar_pempty, float* win_ptr) {
  using Cfg = NarrowCfg<NT>;
  constexpr int EP_THREADS = 128;
  constexpr int PER = kBsWindow * NT / EP_THREADS;     // table entries per thread and window
  const int lane = threadIdx.x & 31;
  const int e = static_cast<int>(threadIdx.x) - 64;    // among the accumulating threads
  const int quad = (threadIdx.x >> 5) & 3;             // TMEM lane quadrant this warp may access
  const int col_in_tile = quad * 32 + lane;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  float alpha = p.alpha;
  if (p.use_scales) alpha = alpha * __ldg(p.scales) * __ldg(p.scales + 1);
  int buf = 0;
  uint32_t buf_phase = 0;
  bool ok = true;
  const bool stat_thread = p.stats != nullptr && threadIdx.x == 64;   // warp 2, lane 0
  long long wait_pfull = 0, busy = 0, items = 0;
  // table entry i of this thread: row (e + i EP_THREADS) / 8 of the tile, k-block of the window % 8
  const int entry_kb = e % kBsWindow;
  float na[PER], nb[SHARED ? 1 : kBsWindow];           // the next window's scales
  const int32_t nkb = p.sched.kt;
  auto load_window = [&](const Tile& w, int32_t kb0) {
    const int32_t last = p.bs_kblocks - 1;             // k-blocks past K are not folded
    const int32_t kb = kb0 + entry_kb < last ? kb0 + entry_kb : last;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const int32_t at = w.row0 + (e + i * EP_THREADS) / kBsWindow;
      const int32_t row = at < p.M ? at : p.M - 1;     // rows past the group are not stored
      na[i] = __ldg(p.bs_a + static_cast<int64_t>(row / p.bs_rows) * p.bs_kblocks + kb);
    }
    const int64_t first = static_cast<int64_t>(w.group) * p.bs_group_rows;
    if constexpr (SHARED) {
      nb[0] = __ldg(p.bs_b + (first + w.n * 128 / p.bs_rows_b) * p.bs_kblocks + kb);
    } else {
      const int32_t at = w.n * 128 + col_in_tile, col = at < p.N ? at : p.N - 1;
      const float* sb = p.bs_b + (first + col / p.bs_rows_b) * p.bs_kblocks;
#pragma unroll
      for (int i = 0; i < kBsWindow; ++i) nb[i] = __ldg(sb + (kb0 + i < last ? kb0 + i : last));
    }
  };
  Tile w, wn;
  // every warp walks the same items and windows and meets the same barriers, after a failed wait too
  bool have = walk.next_warp(w);
  uint32_t g = 0;   // windows begun so far: window g uses table g & 1
  if (have) load_window(w, 0);
  while (have) {
    const bool have_next = walk.next_warp(wn);
    float r[NT];
#pragma unroll
    for (int j = 0; j < NT; ++j) r[j] = 0.0f;
    for (int kb = 0; kb < nkb; kb += kBsWindow, ++g) {
      float* win = win_ptr + (g & 1u) * (Cfg::WINDOW_BYTES / 4);
#pragma unroll
      for (int i = 0; i < PER; ++i)
        win[entry_kb * NT + (e + i * EP_THREADS) / kBsWindow] = SHARED ? na[i] * nb[0] : na[i];
      float sb[SHARED ? 1 : kBsWindow];
      if constexpr (!SHARED) {
#pragma unroll
        for (int i = 0; i < kBsWindow; ++i) sb[i] = nb[i];
      }
      ptx::named_bar_sync(kBsBarrier, EP_THREADS);   // table g is in place; table g - 1 is read
      if (kb + kBsWindow < nkb) load_window(w, kb + kBsWindow);
      else if (have_next) load_window(wn, 0);
#pragma unroll(SHARED ? 1 : kBsWindow)
      for (int j = 0; j < kBsWindow; ++j) {
        if (ok && kb + j < nkb) {
          const long long t0 = stat_thread ? clock64() : 0;
          ok = wait_phase_warp(p, c, bar_pfull + 8 * buf, buf_phase, ROLE_EPILOGUE);
          if (ok) {
            const long long t1 = stat_thread ? clock64() : 0;
            if (stat_thread) wait_pfull += t1 - t0;
            ptx::tc_fence_after();
            float v[NT];
            if constexpr (NT == 16) ptx::tmem_load_16cols(taddr0 + static_cast<uint32_t>(buf * NT), v);
            else ptx::tmem_load_32cols(taddr0 + static_cast<uint32_t>(buf * NT), v);
            ptx::tc_fence_before();
            __syncwarp();
            if (lane == 0) ptx::mbar_arrive(bar_pempty + 8 * buf);   // the partials are in registers
            narrow_fold<NT, SHARED>(win + j * NT, SHARED ? 1.0f : sb[j], v, r);
            if (++buf == Cfg::BUFS) { buf = 0; buf_phase ^= 1u; }
            if (stat_thread) busy += clock64() - t1;
          }
        }
      }
    }
    const int32_t col = w.n * 128 + col_in_tile;
    if (ok && col < p.N) {
      // the basic epilogue: alpha, column bias, ReLU, cast; a warp stores 32 adjacent columns of each row
      const float b = p.has_bias ? __ldg(p.bias + col) : 0.0f;
#pragma unroll
      for (int i = 0; i < NT; ++i) {
        const int32_t row = w.row0 + i;
        if (row >= w.row_end) break;
        float z = fmaf(alpha, r[i], b);
        if (p.relu) z = fmaxf(z, 0.0f);
        const int64_t at = static_cast<int64_t>(row) * p.N + col;
        if (OUT == OUT_BF16) reinterpret_cast<__nv_bfloat16*>(p.C)[at] = __float2bfloat16_rn(z);
        else reinterpret_cast<float*>(p.C)[at] = z;
      }
    }
    items += 1;
    w = wn;
    have = have_next;
  }
  if (stat_thread) {
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_WAIT_TFULL] = wait_pfull;
    p.stats[blockIdx.x * kStatSlots + STAT_EPI_BUSY] = busy;
    p.stats[blockIdx.x * kStatSlots + STAT_ITEMS] = items;
  }
}

template <int NT, int OUT, bool SHARED>
__global__ void __launch_bounds__(kBsNarrowThreads, 2) gemm_bs_narrow_kernel(const __grid_constant__ KernelParams p) {
  using Cfg = NarrowCfg<NT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_addr(smem);
  const uint32_t bar_full = base + Cfg::BAR_OFFSET;
  const uint32_t bar_empty = bar_full + 8 * Cfg::STAGES;
  const uint32_t bar_pfull = bar_empty + 8 * Cfg::STAGES;
  const uint32_t bar_pempty = bar_pfull + 8 * Cfg::BUFS;
  const uint32_t bar_drain = bar_pempty + 8 * Cfg::BUFS;
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
    for (int b = 0; b < Cfg::BUFS; ++b) {
      ptx::mbar_init(bar_pfull + 8 * b, 1);
      ptx::mbar_init(bar_pempty + 8 * b, 4);   // the accumulating warps
    }
    ptx::mbar_init(bar_drain, 1);
    ctl->abort = 0;
    ctl->ep_ok = 0;
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_a);
    ptx::prefetch_tmap(&p.tmap_b);
  }
  if (warp == 1) {
    ptx::tmem_alloc(ptx::smem_addr(&ctl->tmem_base), Cfg::TMEM_COLS);
    ptx::tmem_relinquish();
  }
  const GroupTable table(smem + Cfg::WALK_OFFSET);
  if (warp == 2) fill_group_table(p.sched, table);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const Walk walk(p.sched, table, c.unit);

  if (warp == 0) {
    if (ptx::elect_one())
      bs_producer<NT>(p, c, walk, base + Cfg::W_BYTES, Cfg::STAGE_BYTES, base, Cfg::STAGE_BYTES, bar_full, bar_empty);
    __syncwarp();
  } else if (warp == 1) {
    if (ptx::elect_one())
      narrow_mma<NT>(p, c, walk, tmem_base, base, bar_full, bar_empty, bar_pfull, bar_pempty, bar_drain);
    __syncwarp();
  } else {
    narrow_epilogue<NT, OUT, SHARED>(p, c, walk, tmem_base, bar_pfull, bar_pempty,
                                     reinterpret_cast<float*>(smem + Cfg::WINDOW_OFFSET));
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (p.stats && threadIdx.x == 0) p.stats[blockIdx.x * kStatSlots + STAT_TOTAL] = clock64() - t_start;
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, Cfg::TMEM_COLS);
  }
}

}  // namespace tst
