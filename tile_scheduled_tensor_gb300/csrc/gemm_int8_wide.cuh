// The int8 GEMM (gemm_int8.cuh: the same sums, in the same way) for many tokens: CTA pairs that share one
// 256-channel x NT-token MMA (tcgen05 cta_group::2), and tokens that a first kernel has made FP16.
//
// Every weight is converted for a tile of its own, so its conversion is paid once per NT tokens and hides
// behind the MMAs.  The tokens' would be paid once per 256 channels, and cost more there: through shared
// memory it is a read and a twice as wide write beside the MMA's own reads.  int8_widen_kernel makes it
// once per call, into the plan's workspace (3 bytes of traffic per element), and TMA brings FP16 tiles.
//
// Roles, 512 threads per CTA, one CTA per SM, persistent over 256 x NT tiles; each CTA of a pair holds 128
// channels and half of the tokens' tile:
//   warp 0      TMA: 128 x 128 bytes of B per k-block, into the byte ring
//   warp 1      MMA issuer (the leader's): four K = 16 MMAs per half k-block; every eighth k-block a new
//               accumulator, of two
//   warp 2      TMA: this CTA's half of the tokens, FP16, two 64-element atoms per k-block
//   warps 4-7   weights: a thread per channel, 64 bytes -> 32 columns of Tensor Memory per half k-block
//   warps 8-15  a thread per channel and half of the tokens: accumulator -> integer sums; store
#pragma once
#include "gemm_int8.cuh"

namespace tst {

constexpr int kInt8WideThreads = 512;
constexpr int kInt8WideRegs = 128, kInt8RoleRegs = 56, kInt8ConvertRegs = 88, kInt8SumRegs = 184;
static_assert(kInt8RoleRegs + kInt8ConvertRegs + 2 * kInt8SumRegs <= 4 * kInt8WideRegs, "the split fits the launch");

template <int NT_>
struct Int8WideCfg {
  static constexpr int NT = NT_;
  static constexpr int XR = NT / 2;                          // tokens per CTA
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_ATOM = XR * 128;
  static constexpr int X_BYTES = 2 * X_ATOM;
  static constexpr int BUFS = NT <= 192 ? 2 : 1;
  static constexpr int A_COL = BUFS * NT;
  static constexpr int CV = (512 - A_COL) / 32;              // converted half k-blocks
  static constexpr int FIXED = 1024 + kWalkBytes + 512;
  static constexpr int XS = 5;                               // tokens' ring
  static constexpr int WS = (kSmemLimit - FIXED - XS * X_BYTES) / W_BYTES;
  static constexpr int X_OFFSET = WS * W_BYTES;
  static constexpr int WALK_OFFSET = X_OFFSET + XS * X_BYTES;
  static constexpr int BAR_OFFSET = (WALK_OFFSET + kWalkBytes + 7) / 8 * 8;
  static constexpr int BARS = 2 * WS + 2 * XS + 2 * CV + 2 * BUFS + 1;
  static constexpr int MISC_OFFSET = BAR_OFFSET + BARS * 8;
  static constexpr int SMEM_BYTES = 1024 + MISC_OFFSET + 16;
  static_assert(X_ATOM % 1024 == 0 && SMEM_BYTES <= kSmemLimit && WS >= 3 && CV >= 2 && CV <= 32, "fits an SM");
};

template <class Cfg>
struct Int8WideBars {
  uint32_t w_full, w_empty, x_full, x_empty, cv_full, cv_empty, acc_full, acc_empty, drain;
  __device__ __forceinline__ explicit Int8WideBars(uint32_t base)
      : w_full(base), w_empty(w_full + 8 * Cfg::WS), x_full(w_empty + 8 * Cfg::WS), x_empty(x_full + 8 * Cfg::XS),
        cv_full(x_empty + 8 * Cfg::XS), cv_empty(cv_full + 8 * Cfg::CV), acc_full(cv_empty + 8 * Cfg::CV),
        acc_empty(acc_full + 8 * Cfg::BUFS), drain(acc_empty + 8 * Cfg::BUFS) {}
};

// wait_phase for a pair's warp, which follows one verdict (suspended waits, as in the kernel of single CTAs, cost 3 %
// here, where few warps wait)
__device__ __forceinline__ bool int8_wait_pair(const KernelParams& p, const Ctx& c, uint32_t bar, uint32_t parity, uint32_t role) {
  return __all_sync(0xFFFFFFFFu, wait_phase<2>(p, c, bar, parity, role));
}

template <class Cfg>
__device__ __forceinline__ void int8_wide_weight_loads(const KernelParams& p, const Ctx& c, Walk walk, uint32_t smem, const Int8WideBars<Cfg>& bar) {
  RingAt<Cfg::WS> r;
  uint32_t issued = 0, parity = 0;
  bool ok = true;
  Tile w;
  while (ok && walk.next(w)) {
    if (w.clamped && c.rank == 0) record_status(p, ST_DEVICE_CHECK, ROLE_PRODUCER);
    const int32_t b_row0 = w.group * p.sched.group_b_rows + w.n * 256 + static_cast<int32_t>(c.rank) * 128;
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      if (!wait_phase<2>(p, c, bar.w_empty + 8 * r.at, r.phase ^ 1u, ROLE_PRODUCER)) { ok = false; break; }
      ptx::mbar_arrive_expect_tx(bar.w_full + 8 * r.at, Cfg::W_BYTES);
      ptx::tma_load_2d(smem + r.at * Cfg::W_BYTES, &p.tmap_b, bar.w_full + 8 * r.at, kb * 128, b_row0);
      issued |= 1u << r.at;
      parity = (parity & ~(1u << r.at)) | (r.phase << r.at);
      r.next();
    }
  }
  int8_land<Cfg::WS>(p, bar.w_full, issued, parity);
}

// Both CTAs' tokens arrive on the leader's barrier.  peer_issued: a word of each CTA, 0 at first.
template <class Cfg>
__device__ __forceinline__ void int8_wide_token_loads(const KernelParams& p, const Ctx& c, Walk walk, uint32_t smem, const Int8WideBars<Cfg>& bar,
                                                      volatile uint32_t* peer_issued) {
  RingAt<Cfg::XS> r;
  uint32_t issued = 0, parity = 0, count = 0;
  bool ok = true;
  auto mark = [&] {
    issued |= 1u << r.at;
    parity = (parity & ~(1u << r.at)) | (r.phase << r.at);
    r.next();
  };
  Tile w;
  ptx::griddep_wait();   // the FP16 tokens are the kernel's before
  while (ok && walk.next(w)) {
    const int32_t row0 = w.row0 + static_cast<int32_t>(c.rank) * Cfg::XR;
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      if (!wait_phase<2>(p, c, bar.x_empty + 8 * r.at, r.phase ^ 1u, ROLE_PRODUCER)) { ok = false; break; }
      const uint32_t full = bar.x_full + 8 * r.at, dst = smem + r.at * Cfg::X_BYTES;
      if (c.rank == 0) ptx::mbar_arrive_expect_tx(full, 2 * Cfg::X_BYTES);
      const uint32_t leader = ptx::mapa(full, 0);
      ptx::tma_load_2d_pair(dst, &p.tmap_a, leader, kb * 128, row0);
      ptx::tma_load_2d_pair(dst + Cfg::X_ATOM, &p.tmap_a, leader, kb * 128 + 64, row0);
      mark();
      ++count;
    }
  }
  // The leader waits for both CTAs' copies; the peer's own land before the cluster's last barrier lets it go, which the
  // leader reaches only after its wait here.  Where waits ran out the peer may have issued more (at most its ring), onto
  // phases that the leader has not opened: the peer tells how many, and the leader opens them for the peer's half.
  if (c.rank != 0) {
    ptx::st_cluster_u32(ptx::mapa(ptx::smem_addr(const_cast<uint32_t*>(peer_issued)), 0), 2u * count + 1u);
    return;
  }
  const uint64_t t0 = ptx::globaltimer(), limit = int8_end_limit(p);
  uint32_t told = 0;
  while ((told = *peer_issued) == 0u)
    if (ptx::globaltimer() - t0 > limit) break;
  // the difference of the counts, each modulo 2^31
  const int32_t more = told != 0u ? static_cast<int32_t>((told - 1u) - 2u * count) / 2 : 0;
  for (int32_t i = 0; i < more && i < Cfg::XS; ++i) {
    ptx::mbar_arrive_expect_tx(bar.x_full + 8 * r.at, Cfg::X_BYTES);
    mark();
  }
  int8_land<Cfg::XS>(p, bar.x_full, issued, parity);
}

template <class Cfg>
__device__ __forceinline__ void int8_wide_mma(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, uint32_t xs,
                                              const Int8WideBars<Cfg>& bar) {
  const uint32_t idesc = ptx::make_idesc(0u, 256, Cfg::NT);   // FP16 operands
  const uint64_t x_desc0 = ptx::sw128_kmajor_desc(xs);
  RingAt<Cfg::XS> r;
  RingAt<Cfg::CV> t;
  RingAt<Cfg::BUFS> acc;
  bool ok = true;
  while (ok && walk.skip()) {
    for (int32_t kb = 0; ok && kb < p.sched.kt; ++kb) {
      const int32_t in_fold = kb % kInt8Fold;
      if (in_fold == 0 && !wait_phase<2>(p, c, bar.acc_empty + 8 * acc.at, acc.phase ^ 1u, ROLE_MMA)) { ok = false; break; }
      if (!wait_phase<2>(p, c, bar.x_full + 8 * r.at, r.phase, ROLE_MMA)) { ok = false; break; }
      const uint32_t d = tmem_base + static_cast<uint32_t>(acc.at * Cfg::NT);
      const uint64_t x = x_desc0 + static_cast<uint64_t>(r.at * (Cfg::X_BYTES >> 4));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (!wait_phase<2>(p, c, bar.cv_full + 8 * t.at, t.phase, ROLE_MMA)) { ok = false; break; }
        ptx::tc_fence_after();
        const uint32_t a = tmem_base + static_cast<uint32_t>(Cfg::A_COL + t.at * 32);
#pragma unroll
        for (int i = 0; i < 4; ++i)   // 16 of K: 8 TMEM columns, 32 bytes of an atom
          ptx::mma_f16_ts_pair(d, a + 8 * i, x + h * (Cfg::X_ATOM >> 4) + i * 2, idesc, in_fold != 0 || h != 0 || i != 0);
        ptx::mma_commit_pair_mc(bar.cv_empty + 8 * t.at, 3);
        t.next();
      }
      if (!ok) break;
      ptx::mma_commit_pair_mc(bar.x_empty + 8 * r.at, 3);
      r.next();
      if (in_fold == kInt8Fold - 1 || kb == p.sched.kt - 1) {
        ptx::mma_commit_pair_mc(bar.acc_full + 8 * acc.at, 3);
        acc.next();
      }
    }
  }
  // every MMA issued completes before TMEM is released
  ptx::mma_commit_pair(bar.drain);
  int8_drain<2>(p, c, bar.drain);
}

template <class Cfg>
__device__ __forceinline__ void int8_wide_weights(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, const uint8_t* smem,
                                                  const Int8WideBars<Cfg>& bar) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const uint8_t* const src0 = smem + (quad * 32 + lane) * 128;
  const int sub = lane & 7;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::A_COL;
  const uint32_t cv_full = ptx::mapa(bar.cv_full, 0);   // the leader's
  RingAt<Cfg::WS> r;
  RingAt<Cfg::CV> t;
  while (walk.skip()) {
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      if (!int8_wait_pair(p, c, bar.w_full + 8 * r.at, r.phase, ROLE_EPILOGUE)) return;
      const uint8_t* const src = src0 + r.at * Cfg::W_BYTES;
      uint4 v[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(src + ((q ^ sub) << 4));
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t f[32];
#pragma unroll
        for (int q = 0; q < 4; ++q) int8_to_half(v[q], f + 8 * q);
        if (h == 0) {
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const uint4*>(src + (((4 + q) ^ sub) << 4));
        } else {
          __syncwarp();
          if (lane == 0) ptx::mbar_arrive(bar.w_empty + 8 * r.at);   // the bytes are in registers
        }
        if (!int8_wait_pair(p, c, bar.cv_empty + 8 * t.at, t.phase ^ 1u, ROLE_EPILOGUE)) return;
        ptx::tc_fence_after();
        ptx::tmem_store_32cols(taddr0 + static_cast<uint32_t>(t.at * 32), f);
        ptx::tmem_wait_stores();
        ptx::tc_fence_before();
        __syncwarp();
        if (lane == 0) ptx::mbar_arrive_remote(cv_full + 8 * t.at);
        t.next();
      }
      r.next();
    }
  }
}

template <class Cfg, int OUT>
__device__ __forceinline__ void int8_wide_epilogue(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, const Int8WideBars<Cfg>& bar) {
  constexpr int HALF = Cfg::NT / 2;
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3, half = (threadIdx.x >> 5) >= 12;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(half * HALF);
  const uint32_t acc_empty = ptx::mapa(bar.acc_empty, 0);
  RingAt<Cfg::BUFS> acc;
  Tile w;
  while (walk.next_warp(w)) {
    RowScales<HALF> scale;
    scale.load(p, w.row0 + half * HALF);
    int32_t sum[HALF];
    for (int32_t kb = 0; kb < p.sched.kt; kb += kInt8Fold) {
      if (!int8_wait_pair(p, c, bar.acc_full + 8 * acc.at, acc.phase, ROLE_EPILOGUE)) return;
      ptx::tc_fence_after();
#pragma unroll
      for (int q = 0; q < HALF; q += 16) {
        float v[16];
        ptx::tmem_load_16cols(taddr0 + static_cast<uint32_t>(acc.at * Cfg::NT + q), v);
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int32_t x = __float2int_rn(v[i]);   // a whole number already
          sum[q + i] = kb == 0 ? x : sum[q + i] + x;
        }
      }
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive_remote(acc_empty + 8 * acc.at);
      acc.next();
    }
    int8_store<HALF, OUT>(p, w, w.row0 + half * HALF, w.n * 256 + static_cast<int32_t>(c.rank) * 128 + quad * 32 + lane, sum,
                          scale);
  }
}

template <class Cfg, int OUT>
__global__ void __launch_bounds__(kInt8WideThreads, 1) gemm_int8_wide_kernel(const __grid_constant__ KernelParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_addr(smem);
  const Int8WideBars<Cfg> bar(base + Cfg::BAR_OFFSET);
  SharedCtl* ctl = reinterpret_cast<SharedCtl*>(smem + Cfg::MISC_OFFSET);
  const int warp = threadIdx.x >> 5;

  Ctx c;
  c.abort = &ctl->abort;
  c.abort_addr = ptx::smem_addr(&ctl->abort);
  c.rank = ptx::cluster_ctarank();
  c.rank_m = c.rank;
  c.rank_n = 0;
  c.csize = 2;
  c.unit = static_cast<int32_t>(blockIdx.x) / 2;

  if (threadIdx.x == 0) {
    for (int s = 0; s < Cfg::WS; ++s) {
      ptx::mbar_init(bar.w_full + 8 * s, 1);
      ptx::mbar_init(bar.w_empty + 8 * s, 4);
    }
    for (int s = 0; s < Cfg::XS; ++s) {
      ptx::mbar_init(bar.x_full + 8 * s, 1);
      ptx::mbar_init(bar.x_empty + 8 * s, 1);
    }
    for (int s = 0; s < Cfg::CV; ++s) {
      ptx::mbar_init(bar.cv_full + 8 * s, 8);    // the converting warps of both CTAs
      ptx::mbar_init(bar.cv_empty + 8 * s, 1);
    }
    for (int b = 0; b < Cfg::BUFS; ++b) {
      ptx::mbar_init(bar.acc_full + 8 * b, 1);
      ptx::mbar_init(bar.acc_empty + 8 * b, 16);
    }
    ptx::mbar_init(bar.drain, 1);
    ctl->abort = 0;
    ctl->ep_ok = 0;
    ctl->pad = 0;   // the peer's k-blocks of tokens, as int8_wide_token_loads tells them
    ptx::fence_mbar_init();
    ptx::prefetch_tmap(&p.tmap_a);
    ptx::prefetch_tmap(&p.tmap_b);
  }
  if (warp == 1) {
    ptx::tmem_alloc_pair(ptx::smem_addr(&ctl->tmem_base), 512);
    ptx::tmem_relinquish_pair();
  }
  const GroupTable table(smem + Cfg::WALK_OFFSET);
  if (warp == 2) fill_group_table(p.sched, table);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::cluster_sync();   // the other CTA's barriers exist before anyone signals them
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const Walk walk(p.sched, table, c.unit);

  if (warp < 4) {
    ptx::setmaxnreg_dec<kInt8RoleRegs>();
    if (warp == 0) {
      if (ptx::elect_one()) int8_wide_weight_loads<Cfg>(p, c, walk, base, bar);
    } else if (warp == 1) {
      if (c.rank == 0 && ptx::elect_one()) int8_wide_mma<Cfg>(p, c, walk, tmem_base, base + Cfg::X_OFFSET, bar);
    } else if (warp == 2) {
      if (ptx::elect_one()) int8_wide_token_loads<Cfg>(p, c, walk, base + Cfg::X_OFFSET, bar, &ctl->pad);
    }
    __syncwarp();
  } else if (warp < 8) {
    ptx::setmaxnreg_dec<kInt8ConvertRegs>();
    int8_wide_weights<Cfg>(p, c, walk, tmem_base, smem, bar);
  } else {
    ptx::setmaxnreg_inc<kInt8SumRegs>();
    int8_wide_epilogue<Cfg, OUT>(p, c, walk, tmem_base, bar);
  }

  ptx::tc_fence_before();
  __syncthreads();
  // no CTA leaves (nor frees TMEM) while the other may still signal its barriers or the leader's MMAs use its memory
  ptx::cluster_sync();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc_pair(tmem_base, 512);
  }
}

// A (rows x K bytes) as FP16, the groups' rows only: bound by its traffic of 3 bytes per element.
constexpr int kInt8WidenThreads = 256;
struct Int8WidenParams {
  const int8_t* a;
  uint32_t* out;               // rows x K FP16
  const int32_t* group_rows;   // groups, or null: all rows
  int64_t units;               // of 16 elements: rows * K / 16
  int32_t groups, units_per_row;
};
__global__ void __launch_bounds__(kInt8WidenThreads) int8_widen_kernel(const Int8WidenParams p) {
  ptx::griddep_launch_dependents();
  int64_t most = p.units;
  if (p.group_rows != nullptr) {
    __shared__ unsigned long long used;
    if (threadIdx.x == 0) used = 0ull;
    __syncthreads();
    unsigned long long mine = 0;
    for (int g = threadIdx.x; g < p.groups; g += kInt8WidenThreads) mine += p.group_rows[g] > 0 ? p.group_rows[g] : 0;
    if (mine != 0) atomicAdd(&used, mine);
    __syncthreads();
    const int64_t rows = static_cast<int64_t>(used) * p.units_per_row;
    most = rows < most ? rows : most;
  }
  constexpr int PER = 4;
  const int64_t step = static_cast<int64_t>(gridDim.x) * kInt8WidenThreads;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kInt8WidenThreads + threadIdx.x; i < most; i += PER * step) {
    uint4 v[PER];
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (i + u * step < most) v[u] = __ldg(reinterpret_cast<const uint4*>(p.a) + i + u * step);
#pragma unroll
    for (int u = 0; u < PER; ++u)
      if (i + u * step < most) {
        uint32_t h[8];
        int8_to_half(v[u], h);
        uint4* const out = reinterpret_cast<uint4*>(p.out) + 2 * (i + u * step);
        out[0] = make_uint4(h[0], h[1], h[2], h[3]);
        out[1] = make_uint4(h[4], h[5], h[6], h[7]);
      }
  }
}

}  // namespace tst
