// GEMM of 8-bit integers with a scale per token (row of A) and per channel (row of B):
//
//   D[i][j] = cast( relu?( float(sum_k a_ik b_jk) ra_i cb_j + bias_j ) ),   the sum exact,
//
// dense, or grouped with one N x K matrix, one row of scales and one of biases per group.
//
// sm_103a's tcgen05 has no integer kind.  Every int8 value is an FP16 value, a product of two is an
// integer of at most 2^14, and a sum of 1024 of them is at most 2^24: the FP32 accumulator of
// kind::f16 holds it exactly, in any order.  So the operands travel as bytes (HBM, L2, TMA, the
// shared-memory ring), become FP16 on their way to the tensor core, and every 1024 of K the
// accumulator is added to 32-bit integer sums in registers.
//
// The operands are exchanged as in gemm_bs_narrow.cuh: the 128 rows of the MMA (TMEM lanes) are
// channels, rows of B, and its N are NT tokens, rows of A.  Few tokens then waste no tensor-core
// rows, and the bulk of the bytes to convert, the weights, goes from registers straight into Tensor
// Memory, which holds the MMA's first operand: no second pass through shared memory.
//
// A byte x becomes FP16 as 0x6400 | (x ^ 0x80), which is 1024 + (x + 128), less 1152: for four bytes
// one exclusive or, two byte permutes, two packed subtractions.
//
// The tokens, far fewer bytes, are made FP16 once per call by int8_widen_kernel, into the plan's workspace,
// and come by TMA.  (Two warps that converted them beside the weights took 1400 cycles per k-block of 64
// tokens, and 450 of 16, most of it waiting for their writes to be seen by the tensor core.)
//
// Roles, 640 threads (of 128 tokens: 512), one CTA per SM, persistent over NT x 128 tiles of D, k-blocks
// of 128:
//   warp 0      TMA: 128 x 128 bytes of B per stage of the byte ring
//   warps 1, 3  MMA issuers of every second k-block, into accumulators of their own: eight K = 16 MMAs,
//               which one thread issues in about 64 cycles each, however few tokens they have; every
//               eighth k-block of theirs into a new accumulator
//   warp 2      TMA: NT tokens, FP16, two 64-element atoms per k-block
//   warps 8-11  a thread per channel: accumulators -> integer sums; scales, bias, ReLU, cast, store
//   the others  weights: a thread per channel, 128 bytes -> 64 columns of Tensor Memory.  One k-block
//               takes a warpgroup 800 to 1000 cycles, most of them latencies, where its 16 KB come in
//               700 at the copy rate: three warpgroups (of 128 tokens: two) take k-blocks in turn.  A
//               fourth is in the others' way: 16 tokens x 8192 x 8192 in 22.9 us with it, 22.0 without
// What bounds it: the copy rate while each weight is read once (64 rows over 32 experts of 4096 x 4096 in
// 85 us, 0.93 of it).  Where tiles of several tokens' rows read it again, from L2 (512 x 9728 x 4096: 72 us in
// tiles of 32 tokens, 49 of 64, 40 of 128), a k-block takes 460, 610 and 910 cycles, in which all SMs take in
// 16 TB/s of bytes and FP16 tokens; half of the MMAs left out changes that by 1 to 5 %, the conversion left out
// by 10 to 20.  2047 ragged rows over 60 experts of 1416 x 2064 take 55 us: six tiles of 17 k-blocks an SM.
// Every wait is bounded as in the other kernels.
#pragma once
#include "gemm_bs_tile.cuh"
#include "int8_params.h"
#include "ptx_int8.cuh"

namespace tst {

constexpr int kInt8Fold = 8;   // k-blocks of 128 per accumulator: 1024 products of at most 2^14

template <int NT_>
struct Int8Cfg {
  static constexpr int NT = NT_;
  static constexpr int WSETS = NT == 128 ? 2 : 3;          // warpgroups that convert weights, k-blocks in turn
  static constexpr int THREADS = 256 + 128 * WSETS;
  static constexpr int W_BYTES = 128 * 128;
  static constexpr int X_ATOM = NT * 128;                  // 64 elements of the tokens' tile
  static constexpr int X_BYTES = 2 * X_ATOM;
  static constexpr int BUFS = NT >= 64 ? 1 : 2;            // accumulators per issuer
  static constexpr int A_COL = 2 * BUFS * NT;              // first TMEM column of the weights
  static constexpr int CV = (512 - A_COL) / 128 * 2;       // converted k-blocks of weights: 64 TMEM columns each
  static constexpr int XS = NT == 128 ? 4 : NT == 32 ? 8 : 6;   // k-blocks of tokens
  static constexpr int FIXED = 1024 + XS * X_BYTES + kWalkBytes + 512;
  // A warpgroup that converts weights meets every WSETS-th k-block alone, an issuer every second one, and
  // loads land and warpgroups finish in any order.  A wait tells a phase only from the one before it, so a
  // stage is always the same warpgroup's (STAGES a multiple of WSETS) and the same issuer's (CV and XS even),
  // and so many converted k-blocks are there that the one two turns ago is used up (CV >= WSETS).
  static constexpr int STAGES = (kSmemLimit - FIXED) / W_BYTES / WSETS * WSETS;
  static constexpr int X_OFFSET = STAGES * W_BYTES;
  static constexpr int WALK_OFFSET = X_OFFSET + XS * X_BYTES;
  static constexpr int BAR_OFFSET = (WALK_OFFSET + kWalkBytes + 7) / 8 * 8;
  static constexpr int BARS = 2 * STAGES + 2 * CV + 2 * XS + 4 * BUFS + 1;
  static constexpr int MISC_OFFSET = BAR_OFFSET + BARS * 8;
  static constexpr int SMEM_BYTES = 1024 + MISC_OFFSET + 16;
  static_assert(X_ATOM % 1024 == 0, "swizzled tiles start on 1024 bytes");
  static_assert(SMEM_BYTES <= kSmemLimit && STAGES >= 4 && STAGES <= 32, "fits an SM");
  static_assert(STAGES % WSETS == 0 && CV >= WSETS && CV % 2 == 0 && XS % 2 == 0, "phases are told apart");
  // registers per thread of the warpgroups: roles, weights, sums
  static constexpr int LAUNCH_REGS = NT == 128 ? 128 : 96;
  static constexpr int ROLE_REGS = 56, WEIGHT_REGS = 88, SUM_REGS = NT == 128 ? 184 : 160;
  static_assert(ROLE_REGS + WSETS * WEIGHT_REGS + SUM_REGS <= (2 + WSETS) * LAUNCH_REGS, "the split fits the launch");
};

// 16 int8 values -> 8 pairs of FP16, in their order.  (Shifts and masks for the permutes: 10 % slower tiles of
// 16 and 32 tokens.)
__device__ __forceinline__ void int8_to_half(const uint4& v, uint32_t* h) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = w[i] ^ 0x80808080u;
    const uint32_t lo = __byte_perm(u, 0x64646464u, 0x4140), hi = __byte_perm(u, 0x64646464u, 0x4342);
    asm("sub.f16x2 %0, %1, %2;" : "=r"(h[2 * i]) : "r"(lo), "r"(0x64806480u));
    asm("sub.f16x2 %0, %1, %2;" : "=r"(h[2 * i + 1]) : "r"(hi), "r"(0x64806480u));
  }
}

template <int OUT>
struct OutOf { using T = float; };
template <>
struct OutOf<OUT_BF16> { using T = __nv_bfloat16; };

// The shared addresses of the barriers: byte ring, converted k-blocks, tokens, each issuer's accumulators.
template <class Cfg>
struct Int8Bars {
  uint32_t full, empty, cv_full, cv_empty, x_full, x_empty, acc_full, acc_empty, drain;
  __device__ __forceinline__ explicit Int8Bars(uint32_t base)
      : full(base), empty(full + 8 * Cfg::STAGES), cv_full(empty + 8 * Cfg::STAGES), cv_empty(cv_full + 8 * Cfg::CV),
        x_full(cv_empty + 8 * Cfg::CV), x_empty(x_full + 8 * Cfg::XS), acc_full(x_empty + 8 * Cfg::XS),
        acc_empty(acc_full + 16 * Cfg::BUFS), drain(acc_empty + 16 * Cfg::BUFS) {}
};

// wait_phase with the waiting thread suspended.  Many warps wait here beside those that work, and tries that
// return at once take their places in the queue to shared memory.
constexpr uint32_t kInt8Suspend = 1000;   // ns
template <int CG>
__device__ __forceinline__ bool int8_wait(const KernelParams& p, const Ctx& c, uint32_t bar, uint32_t parity, uint32_t role) {
  if (ptx::mbar_try_wait_for(bar, parity, kInt8Suspend)) return true;
  const uint64_t t0 = ptx::globaltimer();
  while (true) {
    if (ptx::mbar_try_wait_for(bar, parity, kInt8Suspend)) return true;
    if (*c.abort) return false;
    if (ptx::globaltimer() - t0 > p.timeout_ns) {
      raise_error<CG>(p, c, ST_TIMEOUT, role);
      return false;
    }
  }
}
template <int CG>
__device__ __forceinline__ bool int8_wait_warp(const KernelParams& p, const Ctx& c, uint32_t bar, uint32_t parity, uint32_t role) {
  return __all_sync(0xFFFFFFFFu, int8_wait<CG>(p, c, bar, parity, role));
}

// position in a ring of N
template <int N>
struct RingAt {
  int at = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next() {
    if (++at == N) { at = 0; phase ^= 1u; }
  }
};

// What a CTA has in flight, copies and MMAs, ends before the CTA does, also where a wait of another role ran out: limits of
// a plan may be shorter than a copy takes, so these waits have at least 100 ms.
__device__ __forceinline__ uint64_t int8_end_limit(const KernelParams& p) {
  constexpr uint64_t kLeast = 100ull * 1000 * 1000;
  return p.timeout_ns > kLeast ? p.timeout_ns : kLeast;
}

// bounded wait until the copies of a producer have landed: of every one that leaves, as the roles that would wait for them
// may have given up
template <int N>
__device__ __forceinline__ void int8_land(const KernelParams& p, uint32_t full, uint32_t issued, uint32_t parity) {
  const uint64_t t0 = ptx::globaltimer(), limit = int8_end_limit(p);
  for (int s = 0; s < N; ++s) {
    if (!(issued & (1u << s))) continue;
    while (!ptx::mbar_try_wait(full + 8 * s, (parity >> s) & 1u))
      if (ptx::globaltimer() - t0 > limit) break;
  }
}

// The same for the MMAs, which a commit to `drain` follows.
template <int CG>
__device__ __forceinline__ void int8_drain(const KernelParams& p, const Ctx& c, uint32_t drain) {
  const uint64_t t0 = ptx::globaltimer(), limit = int8_end_limit(p);
  while (!ptx::mbar_try_wait(drain, 0)) {
    if (ptx::globaltimer() - t0 > limit) {
      raise_error<CG>(p, c, ST_TIMEOUT, ROLE_MMA);
      break;
    }
  }
}

template <class Cfg>
__device__ __forceinline__ void int8_producer(const KernelParams& p, const Ctx& c, Walk walk, uint32_t smem, const Int8Bars<Cfg>& bar) {
  RingAt<Cfg::STAGES> r;
  uint32_t issued = 0, issued_parity = 0;
  bool ok = true;
  Tile w;
  while (ok && walk.next(w)) {
    if (w.clamped) record_status(p, ST_DEVICE_CHECK, ROLE_PRODUCER);
    const int32_t b_row0 = w.group * p.sched.group_b_rows + w.n * 128;
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      if (!int8_wait<1>(p, c, bar.empty + 8 * r.at, r.phase ^ 1u, ROLE_PRODUCER)) { ok = false; break; }
      const uint32_t full = bar.full + 8 * r.at, dst = smem + r.at * Cfg::W_BYTES;
      ptx::mbar_arrive_expect_tx(full, Cfg::W_BYTES);
      ptx::tma_load_2d(dst, &p.tmap_b, full, kb * 128, b_row0);
      issued |= 1u << r.at;
      issued_parity = (issued_parity & ~(1u << r.at)) | (r.phase << r.at);
      r.next();
    }
  }
  int8_land<Cfg::STAGES>(p, bar.full, issued, issued_parity);
}

// NT rows of two 64-element atoms per k-block.
template <class Cfg>
__device__ __forceinline__ void int8_token_loads(const KernelParams& p, const Ctx& c, Walk walk, uint32_t xs, const Int8Bars<Cfg>& bar) {
  RingAt<Cfg::XS> r;
  uint32_t issued = 0, issued_parity = 0;
  bool ok = true;
  Tile w;
  ptx::griddep_wait();   // they are the kernel's before
  while (ok && walk.next(w)) {
    for (int32_t kb = 0; kb < p.sched.kt; ++kb) {
      if (!int8_wait<1>(p, c, bar.x_empty + 8 * r.at, r.phase ^ 1u, ROLE_PRODUCER)) { ok = false; break; }
      const uint32_t full = bar.x_full + 8 * r.at, dst = xs + r.at * Cfg::X_BYTES;
      ptx::mbar_arrive_expect_tx(full, Cfg::X_BYTES);
      ptx::tma_load_2d(dst, &p.tmap_a, full, kb * 128, w.row0);
      ptx::tma_load_2d(dst + Cfg::X_ATOM, &p.tmap_a, full, kb * 128 + 64, w.row0);
      issued |= 1u << r.at;
      issued_parity = (issued_parity & ~(1u << r.at)) | (r.phase << r.at);
      r.next();
    }
  }
  int8_land<Cfg::XS>(p, bar.x_full, issued, issued_parity);
}

// issuer: of the two that take the k-blocks in turn, each into its own accumulators
template <class Cfg>
__device__ __forceinline__ void int8_mma(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, uint32_t xs, int issuer,
                                         const Int8Bars<Cfg>& bar) {
  const uint32_t idesc = ptx::make_idesc(0u, 128, Cfg::NT);   // FP16 operands
  const uint64_t x_desc0 = ptx::sw128_kmajor_desc(xs);
  const int32_t blocks = p.sched.kt;
  const uint32_t acc_full = bar.acc_full + 8 * Cfg::BUFS * issuer, acc_empty = bar.acc_empty + 8 * Cfg::BUFS * issuer;
  RingAt<Cfg::CV> r;
  RingAt<Cfg::XS> x;
  RingAt<Cfg::BUFS> acc;
  bool ok = true;
  uint32_t count = 0;   // k-blocks so far, of all tiles: a tile's first is either issuer's
  while (ok && walk.skip()) {
    for (int32_t i = 0; i < blocks; ++i, ++count, r.next(), x.next()) {
      if ((count & 1u) != static_cast<uint32_t>(issuer)) continue;
      const int32_t in_fold = (i >> 1) % kInt8Fold;
      if (in_fold == 0 && !int8_wait<1>(p, c, acc_empty + 8 * acc.at, acc.phase ^ 1u, ROLE_MMA)) { ok = false; break; }
      if (!int8_wait<1>(p, c, bar.x_full + 8 * x.at, x.phase, ROLE_MMA)) { ok = false; break; }
      if (!int8_wait<1>(p, c, bar.cv_full + 8 * r.at, r.phase, ROLE_MMA)) { ok = false; break; }
      ptx::tc_fence_after();
      const uint32_t d = tmem_base + static_cast<uint32_t>((issuer * Cfg::BUFS + acc.at) * Cfg::NT);
      const uint32_t a = tmem_base + static_cast<uint32_t>(Cfg::A_COL + r.at * 64);
      const uint64_t xd = x_desc0 + static_cast<uint64_t>(x.at * (Cfg::X_BYTES >> 4));
#pragma unroll
      for (int q = 0; q < 8; ++q)   // 16 of K: 8 TMEM columns, 32 bytes of an atom
        ptx::mma_f16_ts(d, a + 8 * q, xd + (q >> 2) * (Cfg::X_ATOM >> 4) + (q & 3) * 2, idesc, in_fold != 0 || q != 0);
      ptx::mma_commit(bar.cv_empty + 8 * r.at);
      ptx::mma_commit(bar.x_empty + 8 * x.at);
      if (in_fold == kInt8Fold - 1 || i + 2 >= blocks) {
        ptx::mma_commit(acc_full + 8 * acc.at);
        acc.next();
      }
    }
  }
  // every MMA issued completes before TMEM is released
  ptx::mma_commit(bar.drain);
  int8_drain<1>(p, c, bar.drain);
}

// set: of WSETS that take the k-blocks in turn.
template <class Cfg>
__device__ __forceinline__ void int8_weights(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, const uint8_t* smem,
                                             int set, const Int8Bars<Cfg>& bar) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const uint8_t* const src0 = smem + (quad * 32 + lane) * 128;
  const int sub = lane & 7;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + Cfg::A_COL;
  int64_t blocks = 0;   // k-blocks of this CTA
  while (walk.skip()) blocks += p.sched.kt;
  RingAt<Cfg::STAGES> r;
  RingAt<Cfg::CV> t;
  for (int i = 0; i < set; ++i) { r.next(); t.next(); }
  for (int64_t i = set; i < blocks; i += Cfg::WSETS) {
    if (!int8_wait_warp<1>(p, c, bar.full + 8 * r.at, r.phase, ROLE_EPILOGUE)) return;
    const uint8_t* const src = src0 + r.at * Cfg::W_BYTES;
    uint4 v[8];
#pragma unroll
    for (int q = 0; q < 8; ++q) v[q] = *reinterpret_cast<const uint4*>(src + ((q ^ sub) << 4));
    if (!int8_wait_warp<1>(p, c, bar.cv_empty + 8 * t.at, t.phase ^ 1u, ROLE_EPILOGUE)) return;
    ptx::tc_fence_after();
#pragma unroll
    for (int half = 0; half < 2; ++half) {   // 64 of K: 32 columns
      uint32_t h[32];
#pragma unroll
      for (int q = 0; q < 4; ++q) int8_to_half(v[4 * half + q], h + 8 * q);
      ptx::tmem_store_32cols(taddr0 + static_cast<uint32_t>(t.at * 64 + half * 32), h);
    }
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar.empty + 8 * r.at);   // every lane has its bytes
    ptx::tmem_wait_stores();
    ptx::tc_fence_before();
    __syncwarp();
    if (lane == 0) ptx::mbar_arrive(bar.cv_full + 8 * t.at);
#pragma unroll
    for (int s = 0; s < Cfg::WSETS; ++s) { r.next(); t.next(); }
  }
}

// The row scales of N rows from row0 on, a row per lane: fetched by a whole warp while a tile is summed
template <int N>
struct RowScales {
  static constexpr int V = (N + 31) / 32;
  float v[V];
  __device__ __forceinline__ void load(const KernelParams& p, int32_t row0) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int32_t row = row0 + i * 32 + static_cast<int32_t>(threadIdx.x & 31);
      v[i] = __ldg(p.ext.row_scale + (row < p.M ? row : p.M - 1));   // rows past the end are not stored
    }
  }
  __device__ __forceinline__ float of(int i) const { return __shfl_sync(0xFFFFFFFFu, v[i >> 5], i & 31); }
};

__device__ __forceinline__ float relu_nan(float z) {   // a NaN stays
  float r;
  asm("max.NaN.f32 %0, %1, 0f00000000;" : "=f"(r) : "f"(z));
  return r;
}

// A thread's column of a tile: rows row0 .. row0 + N - 1 of D from their integer sums.  A warp holds 32
// adjacent columns.  FP32 rows are stored 128 bytes at once.  BF16, where rows and D are whole 4-byte
// words: neighbouring lanes exchange a value, so that each has two adjacent columns of one of two rows,
// and a store takes two rows of 64 bytes, half as many of them (8192 x 8192 x 1024, bound by this code:
// 144 us with a store per row).
template <int N, int OUT>
__device__ __forceinline__ void int8_store(const KernelParams& p, const Tile& w, int32_t row0, int32_t col, const int32_t (&sum)[N],
                                           const RowScales<N>& scale) {
  const bool on = col < p.N;
  const int64_t channel = static_cast<int64_t>(w.group) * p.N + (on ? col : 0);
  const float cb = __ldg(p.ext.col_scale + channel);
  const float b = p.has_bias ? __ldg(p.bias + channel) : 0.0f;
  const int32_t rows = w.row_end - row0;
  auto value = [&](int i) {
    const float z = fmaf(__int2float_rn(sum[i]) * scale.of(i), cb, b);
    return p.relu ? relu_nan(z) : z;
  };
  if constexpr (OUT == OUT_BF16) {
    if (p.tma_store) {   // whole words
      const bool odd = (threadIdx.x & 1) != 0;
      __nv_bfloat16* dst = static_cast<__nv_bfloat16*>(p.C) + static_cast<int64_t>(row0 + (odd ? 1 : 0)) * p.N + (col & ~1);
      const int64_t step = 2 * static_cast<int64_t>(p.N);
      const int32_t mine = on ? rows - (odd ? 1 : 0) : 0;
#pragma unroll
      for (int i = 0; i < N; i += 2, dst += step) {
        const float z0 = value(i), z1 = value(i + 1);
        const float other = __shfl_xor_sync(0xFFFFFFFFu, odd ? z0 : z1, 1);
        const __nv_bfloat162 two = __floats2bfloat162_rn(odd ? other : z0, odd ? z1 : other);
        if (i < mine) *reinterpret_cast<__nv_bfloat162*>(dst) = two;
      }
      return;
    }
  }
  using Out = typename OutOf<OUT>::T;
  Out* dst = static_cast<Out*>(p.C) + static_cast<int64_t>(row0) * p.N + col;
  const int32_t mine = on ? rows : 0;
#pragma unroll
  for (int i = 0; i < N; ++i, dst += p.N) {
    const float z = value(i);
    if (i < mine) *dst = static_cast<Out>(z);
  }
}

template <class Cfg, int OUT>
__device__ __forceinline__ void int8_epilogue(const KernelParams& p, const Ctx& c, Walk walk, uint32_t tmem_base, const Int8Bars<Cfg>& bar) {
  const int lane = threadIdx.x & 31, quad = (threadIdx.x >> 5) & 3;
  const uint32_t taddr0 = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
  RingAt<Cfg::BUFS> acc0, acc1;   // the issuers'
  uint32_t count = 0;             // k-blocks of the tiles before
  Tile w;
  while (walk.next_warp(w)) {
    RowScales<Cfg::NT> scale;
    scale.load(p, w.row0);
    int32_t sum[Cfg::NT];
    bool first = true;
    for (int32_t i = 0; i < p.sched.kt; i += (i & 1) ? 2 * kInt8Fold - 1 : 1) {   // the first k-block of each accumulator
      const int issuer = static_cast<int>((count + static_cast<uint32_t>(i)) & 1u), at = issuer * Cfg::BUFS + (issuer ? acc1.at : acc0.at);
      if (!int8_wait_warp<1>(p, c, bar.acc_full + 8 * at, issuer ? acc1.phase : acc0.phase, ROLE_EPILOGUE)) return;
      ptx::tc_fence_after();
#pragma unroll
      for (int q = 0; q < Cfg::NT; q += 16) {
        float v[16];
        ptx::tmem_load_16cols(taddr0 + static_cast<uint32_t>(at * Cfg::NT + q), v);
#pragma unroll
        for (int j = 0; j < 16; ++j) {
          const int32_t x = __float2int_rn(v[j]);   // a whole number already
          sum[q + j] = first ? x : sum[q + j] + x;
        }
      }
      first = false;
      ptx::tc_fence_before();
      __syncwarp();
      if (lane == 0) ptx::mbar_arrive(bar.acc_empty + 8 * at);
      if (issuer) acc1.next();
      else acc0.next();
    }
    count += static_cast<uint32_t>(p.sched.kt);
    int8_store<Cfg::NT, OUT>(p, w, w.row0, w.n * 128 + quad * 32 + lane, sum, scale);
  }
}

template <class Cfg, int OUT>
__global__ void __launch_bounds__(Cfg::THREADS, 1) gemm_int8_kernel(const __grid_constant__ KernelParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const uint32_t base = ptx::smem_addr(smem);
  const Int8Bars<Cfg> bar(base + Cfg::BAR_OFFSET);
  SharedCtl* ctl = reinterpret_cast<SharedCtl*>(smem + Cfg::MISC_OFFSET);
  const int warp = threadIdx.x >> 5;

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
      ptx::mbar_init(bar.full + 8 * s, 1);
      ptx::mbar_init(bar.empty + 8 * s, 4);      // the warpgroup that converts it
    }
    for (int s = 0; s < Cfg::CV; ++s) {
      ptx::mbar_init(bar.cv_full + 8 * s, 4);
      ptx::mbar_init(bar.cv_empty + 8 * s, 1);
    }
    for (int s = 0; s < Cfg::XS; ++s) {
      ptx::mbar_init(bar.x_full + 8 * s, 1);
      ptx::mbar_init(bar.x_empty + 8 * s, 1);
    }
    for (int b = 0; b < 2 * Cfg::BUFS; ++b) {
      ptx::mbar_init(bar.acc_full + 8 * b, 1);
      ptx::mbar_init(bar.acc_empty + 8 * b, 4);
    }
    ptx::mbar_init(bar.drain, 2);                 // both issuers
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
  const GroupTable table(smem + Cfg::WALK_OFFSET);
  if (warp == 2) fill_group_table(p.sched, table);
  ptx::tc_fence_before();
  __syncthreads();
  ptx::tc_fence_after();
  const uint32_t tmem_base = ctl->tmem_base;
  const Walk walk(p.sched, table, c.unit);

  if (warp < 4) {
    ptx::setmaxnreg_dec<Cfg::ROLE_REGS>();
    if (warp == 0) {
      if (ptx::elect_one()) int8_producer<Cfg>(p, c, walk, base, bar);
    } else if (warp == 2) {
      if (ptx::elect_one()) int8_token_loads<Cfg>(p, c, walk, base + Cfg::X_OFFSET, bar);
    } else if (ptx::elect_one()) {
      int8_mma<Cfg>(p, c, walk, tmem_base, base + Cfg::X_OFFSET, warp >> 1, bar);
    }
    __syncwarp();
  } else if (warp < 8 || warp >= 12) {
    if constexpr (Cfg::WEIGHT_REGS < Cfg::LAUNCH_REGS) ptx::setmaxnreg_dec<Cfg::WEIGHT_REGS>();
    int8_weights<Cfg>(p, c, walk, tmem_base, smem, warp < 8 ? 0 : (warp >> 2) - 2, bar);
  } else {
    ptx::setmaxnreg_inc<Cfg::SUM_REGS>();
    int8_epilogue<Cfg, OUT>(p, c, walk, tmem_base, bar);
  }

  ptx::tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    ptx::tc_fence_after();
    ptx::tmem_dealloc(tmem_base, 512);
  }
}

}  // namespace tst
