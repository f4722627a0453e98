// Packed-sequence attention, backward, on the Blackwell tensor cores (bf16 in,
// fp32 accumulate).
//
//   P = 2^(c S - L),  c = tau log2 e,  L = lse log2 e,   dP = dout v^T,
//   dS = P (dP - delta),  delta_i = dout_i . out_i = sum_j P_ij dP_ij,
//   dq = tau dS k,   dk = tau dS^T q,   dv = P^T dout,
// dk and dv summed over the query heads that share the key/value head.
//
// Two kernels, each recomputing S and dP, so that every sum stays in one CTA's
// tensor memory and no atomics enter it (seven products instead of five, and the
// same bits from run to run):
//   * k_seq_dq: a CTA per (128 query rows, head), over the key tiles; it also
//     writes delta and L for the second kernel;
//   * k_seq_dkdv: a CTA per (128 keys, key/value head), over the query heads of
//     the group and their query tiles, with S and dP transposed (lane = key), so
//     that P^T and dS^T are the first operands in tensor memory.
//
// delta is dout . out from the rounded out where a row sees more than one key
// tile; where one tile holds all its keys (short sequences, the first rows of a
// causal one) it is sum P dP / sum P in fp32.  There few keys share the weight,
// dP - delta cancels, and the rounding of out would be as large as dS (measured:
// dq 0.9% off in sequences of a few tokens, 0.25% with the sum).
//
// Warps 0-7: elementwise (warp w: lanes 32 (w % 4).., columns of half w / 4);
// warp 8: MMAs (one elected lane); warp 9: TMA; warp 10 (dk/dv): statistics of the
// query tiles and zeros behind the sequence's end.  P and dS are rounded to bf16
// and written over the S and dP columns that the same warp has read.
//
// Rows behind a sequence's end are set to zero in every operand whose rows are
// contracted, and their weights are 0 (L = +inf, or a select), so nothing that
// stands there enters a sum.  Every wait is bounded.
//
// Measured: two causal sequences of 8,192 tokens, 16 heads on 4, d 128, 1.57 ms in a
// burst of five calls (dq 0.69, dk/dv 0.87 each under the profiler; 1,230 TFLOP/s
// issued, 880 of the five products' count), 1.62 over 30 calls and 1.79 over 300, as
// power lowers the clock; 2,090 and 3,130 cycles per tile against 1,610 and 2,140 of
// tensor work (d 96: 1,950 and 2,930 against 1,200 and 1,600).  Bound by the
// arithmetic warps: 64 exponentials a thread and tile keep the special-function unit
// busy for 1,024 cycles, and loads, products and stores of P and dS follow in the
// same warps.
#include <cuda.h>
#include <math.h>

#include "seq_tc.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int MMA_WARP = 8, TMA_WARP = 9, STAT_WARP = 10, NT = 384;
constexpr uint32_t TMEM_COLS = 512;

template <int HD>
struct Cfg {
  static constexpr int NSEG = HD > 64 ? 2 : 1;
  static constexpr uint32_t TILE = NSEG * SEG;
  // streamed tiles in flight: what 227 KB hold beside the two resident tiles (dk/dv:
  // whole pairs, and the statistics)
  static constexpr int NST = HD > 64 ? 5 : 8, NSTK = HD > 64 ? 4 : 8;
};

// 64 columns of P or dS (two bf16 per word) into tensor memory.
__device__ __forceinline__ void store_half(uint32_t taddr, const uint32_t (&p)[32]) {
  tmem_st32(taddr, p);
  tmem_wait_st();
}

// The HD channels of a warp's 32 accumulator rows in pieces of 32, shared between
// the two warps of the rows (three pieces at HD = 96: two and one).
template <int HD>
__device__ __forceinline__ void store_acc(uint32_t taddr, float f, __nv_bfloat16* dst,
                                          int64_t stride, int live, int half, int d, int lane) {
  constexpr int N = HD / 32, FIRST = (N + 1) / 2;
#pragma unroll
  for (int c = 0; c < FIRST; ++c) {
    const int piece = half * FIRST + c;
    if (piece >= N) break;
    uint32_t o[32];
    tmem_ld32(taddr + 32 * piece, o);
    tmem_wait_ld();
    store_rows32(o, f, dst, stride, live, 32 * piece, d, lane);
  }
}

// ---- dq -------------------------------------------------------------------------------

template <int HD>
struct SmemQ {
  uint8_t q[Cfg<HD>::TILE], dout[Cfg<HD>::TILE];
  uint8_t kv[Cfg<HD>::NST][Cfg<HD>::TILE];  // ring: k_0, v_0, k_1, v_1, ...
  float part[2][ROWS];                      // halves of row sums
  uint64_t q_full, do_full;
  uint64_t o_full, o_read;  // out in the ring's last slot, before that is a ring slot
  uint64_t full[Cfg<HD>::NST], empty[Cfg<HD>::NST];
  uint64_t s_full[2], dp_full, ds_full;
  uint64_t k_fixed, done, drain;
  uint32_t tmem_base;
  int32_t abort;
};

struct MapsB {
  CUtensorMap q, k, v, dout, out;
};

// Tensor memory: S (two buffers, dS over the columns read), dP, dq.
constexpr uint32_t QCOL_S = 0, QCOL_DP = 256, QCOL_ACC = 384;

template <int HD>
__global__ void __launch_bounds__(NT, 1)
    k_seq_dq(SeqGeo g, Strides st, pack3d_seq_index ix, const __grid_constant__ MapsB maps,
             const float* lse, float* delta, float* lse2, __nv_bfloat16* dq) {
  using C = Cfg<HD>;
  constexpr int NSEG = C::NSEG, NST = C::NST;
  overlapped_start();
  const int h = blockIdx.x % g.Hq;
  const Tile t = load_tile_entry(ix.query, blockIdx.x / g.Hq);
  const int64_t window = (int64_t)(blockIdx.x / g.Hq) * ROWS;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  if (unused_rows(g, now.rows, window, ROWS))
    zero_unused(g, now.rows, window, ROWS, dq + (int64_t)h * g.d, st.dq);
  if (t.len == 0) return;
  extern __shared__ uint8_t smem_raw[];
  SmemQ<HD>& sm = *reinterpret_cast<SmemQ<HD>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~(uintptr_t)1023);
  volatile int32_t* abort_flag = &sm.abort;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  const int n = ((g.causal ? min(t.len, t.off + ROWS) : t.len) + ROWS - 1) / ROWS;
  const bool fix = n * ROWS > t.len;

  if (tid == 0) {
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.do_full, 1);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_read, 8);  // one arrival per elementwise warp (one key tile: their sums)
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.s_full[0], 1);
    mbar_init(&sm.s_full[1], 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.ds_full, 8);  // one arrival per elementwise warp
    mbar_init(&sm.k_fixed, 1);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == TMA_WARP && lane == 0) {
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
    tma_prefetch_map(&maps.dout);
    tma_prefetch_map(&maps.out);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;

  if (warp == TMA_WARP) {
    const int hk = h / g.G, row0 = t.start + t.off;
    int issued = 0;
    if (lane == 0) {
      bool ok = true;
      mbar_arrive_expect_tx(&sm.q_full, C::TILE);
      load_tile_tma<NSEG>(sm.q, &maps.q, h, row0, &sm.q_full);
      for (int i = 0; i < 2 * n && ok; ++i) {
        const int s = i % NST, round = i / NST;
        if (round > 0 &&
            !(ok = mbar_wait_or_abort(&sm.empty[s], (round - 1) & 1, WAIT_LIMIT, abort_flag)))
          break;
        if (i == NST - 1 && !(ok = mbar_wait_or_abort(&sm.o_read, 0, WAIT_LIMIT, abort_flag)))
          break;
        mbar_arrive_expect_tx(&sm.full[s], C::TILE);
        load_tile_tma<NSEG>(sm.kv[s], (i & 1) ? &maps.v : &maps.k, hk, t.start + (i / 2) * ROWS,
                            &sm.full[s]);
        if (i == 0) {
          mbar_arrive_expect_tx(&sm.do_full, C::TILE);
          load_tile_tma<NSEG>(sm.dout, &maps.dout, h, row0, &sm.do_full);
          if (n > 1) {
            mbar_arrive_expect_tx(&sm.o_full, C::TILE);
            load_tile_tma<NSEG>(sm.kv[NST - 1], &maps.out, h, row0, &sm.o_full);
          }
        }
        issued = i + 1;
      }
    }
    issued = __shfl_sync(0xffffffffu, issued, 0);
    if (fix && issued == 2 * n) {
      // key rows behind the end: zero before dS k contracts them
      const int i = 2 * n - 2, s = i % NST;
      if (warp_wait(&sm.full[s], (i / NST) & 1, abort_flag)) {
        zero_rows<NSEG>(sm.kv[s], t.len - (n - 1) * ROWS, lane);
        if (lane == 0) mbar_arrive(&sm.k_fixed);
      }
    }
    if (lane == 0) {  // copies in flight land before the CTA ends (bounded)
      mbar_wait(&sm.q_full, 0, WAIT_LIMIT);
      if (issued > 0) mbar_wait(&sm.do_full, 0, WAIT_LIMIT);
      if (issued > 0 && n > 1) mbar_wait(&sm.o_full, 0, WAIT_LIMIT);
      for (int i = max(0, issued - NST); i < issued; ++i)
        mbar_wait(&sm.full[i % NST], (i / NST) & 1, WAIT_LIMIT);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    constexpr uint32_t idesc_s = idesc_bf16(ROWS, ROWS, false);
    constexpr uint32_t idesc_o = idesc_bf16(ROWS, HD, true);
    const uint64_t qd = sdesc_sw128(smem_u32(sm.q)), dod = sdesc_sw128(smem_u32(sm.dout));
    const uint64_t kvd = sdesc_sw128(smem_u32(sm.kv[0]));
    auto slot = [&](int i) { return kvd + (uint64_t)(((i % NST) * C::TILE) >> 4); };
    auto wait_item = [&](int i) {
      return warp_wait(&sm.full[i % NST], (i / NST) & 1, abort_flag);
    };
    auto issue_s = [&](int j) -> bool {
      if (!wait_item(2 * j)) return false;
      if (fix && j == n - 1 && !warp_wait(&sm.k_fixed, 0, abort_flag)) return false;
      tc_fence_after();
      const uint64_t b = slot(2 * j);
#pragma unroll
      for (int s = 0; s < HD / 16; ++s)
        mma_ss_warp(tbase + QCOL_S + ROWS * (j & 1), qd + k_step(s), b + k_step(s), idesc_s, s > 0);
      mma_commit_warp(&sm.s_full[j & 1]);
      return true;
    };
    auto issue_dp = [&](int j) -> bool {
      if (!wait_item(2 * j + 1)) return false;
      tc_fence_after();
      const uint64_t b = slot(2 * j + 1);
#pragma unroll
      for (int s = 0; s < HD / 16; ++s)
        mma_ss_warp(tbase + QCOL_DP, dod + k_step(s), b + k_step(s), idesc_s, s > 0);
      mma_commit_warp(&sm.dp_full);
      mma_commit_warp(&sm.empty[(2 * j + 1) % NST]);
      return true;
    };
    bool ok = warp_wait(&sm.q_full, 0, abort_flag) && issue_s(0) &&
              warp_wait(&sm.do_full, 0, abort_flag) && issue_dp(0) && (n < 2 || issue_s(1));
    for (int j = 0; j < n && ok; ++j) {
      if (!(ok = warp_wait(&sm.ds_full, j & 1, abort_flag))) break;
      tc_fence_after();
      // dP of the next tile first: the elementwise warps wait for it
      if (j + 1 < n && !(ok = issue_dp(j + 1))) break;
      const uint32_t a = tbase + QCOL_S + ROWS * (j & 1);
      const uint64_t b = slot(2 * j);
#pragma unroll
      for (int s = 0; s < ROWS / 16; ++s)
        mma_ts_warp(tbase + QCOL_ACC, a + (s >> 2) * 64 + (s & 3) * 8, b + row_step(s), idesc_o,
                    (j > 0 || s > 0) ? 1u : 0u);
      mma_commit_warp(&sm.empty[(2 * j) % NST]);
      if (j == n - 1) mma_commit_warp(&sm.done);
      if (j + 2 < n) ok = issue_s(j + 2);
    }
    __syncwarp();
  } else if (warp < 8) {
    const int half = warp >> 2, r = tid & (ROWS - 1);
    const int pos = t.off + r;
    const bool live = pos < t.len;
    const int64_t row = (int64_t)t.start + pos;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const float c2 = g.tau * LOG2E;
    const float L = live ? lse[(int64_t)h * g.N + row] * LOG2E : 0.f;
    float dl = 0.f;
    bool ok = true;
    if (n > 1) {
      // delta = dout . out from shared memory, half the channels per thread (16-byte
      // piece c of row r stands at c ^ (r % 8): no bank conflicts).  Read from global
      // memory the two tiles took 8,000 cycles, past the little L1 cache that the
      // shared memory leaves.
      ok = warp_wait(&sm.do_full, 0, abort_flag) && warp_wait(&sm.o_full, 0, abort_flag);
      float x = 0.f;
#pragma unroll
      for (int c = 0; c < HD / 16; ++c) {
        const int ch = half * (HD / 16) + c;
        const uint32_t at = (ch >> 3) * SEG + r * 128 + (((ch & 7) ^ (r & 7)) << 4);
        const uint4 u = *reinterpret_cast<const uint4*>(sm.kv[NST - 1] + at);
        const uint4 w = *reinterpret_cast<const uint4*>(sm.dout + at);
        const uint32_t uu[4] = {u.x, u.y, u.z, u.w}, ww[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float2 y = unpack_bf16x2(uu[e]), z = unpack_bf16x2(ww[e]);
          x = fmaf(y.x, z.x, x);
          x = fmaf(y.y, z.y, x);
        }
      }
      sm.part[half][r] = x;
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.o_read);
      // (an mbarrier: its wait is bounded, that of a block barrier is not)
      if (ok) ok = warp_wait(&sm.o_read, 0, abort_flag);
      dl = sm.part[0][r] + sm.part[1][r];
    }
    for (int j = 0; j < n && ok; ++j) {
      const uint32_t tS = tbase + lane_base + QCOL_S + ROWS * (j & 1) + 64 * half;
      const uint32_t tP = tbase + lane_base + QCOL_DP + 64 * half;
      if (!(ok = warp_wait(&sm.s_full[j & 1], (j >> 1) & 1, abort_flag))) break;
      tc_fence_after();
      uint32_t s[64], d[64];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(s + 32 * c));
      tmem_wait_ld();
      const float2 cc = make_float2(c2, c2), ll = make_float2(-L, -L);
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float2 x = f2_fma(
            make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])), cc, ll);
        s[2 * e] = __float_as_uint(ex2(x.x));
        s[2 * e + 1] = __float_as_uint(ex2(x.y));
      }
      const bool masked = j == n - 1 && (g.causal || fix);
      // last column of this half that the row sees
      const int end = min(g.causal ? pos : t.len - 1, t.len - 1) - j * ROWS - 64 * half;
      if (!(ok = warp_wait(&sm.dp_full, j & 1, abort_flag))) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(tP + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(d + 32 * c));
      tmem_wait_ld();
      if (masked) {
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c > end) s[c] = d[c] = 0u;
      }
      if (n == 1) {
        // every key of the row is here: delta = sum P dP / sum P
        float a = 0.f, b = 0.f;
#pragma unroll
        for (int c = 0; c < 64; ++c) {
          a = fmaf(__uint_as_float(s[c]), __uint_as_float(d[c]), a);
          b += __uint_as_float(s[c]);
        }
        // (one key tile leaves the ring's last slot unused)
        float2* sum = reinterpret_cast<float2*>(sm.kv[NST - 1]);
        sum[half * ROWS + r] = make_float2(a, b);
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.o_read);
        if (!(ok = warp_wait(&sm.o_read, 0, abort_flag))) break;
        const float2 x = sum[r], y = sum[ROWS + r];
        dl = (x.x + y.x) / (x.y + y.y);
      }
      const float2 dd = make_float2(-dl, -dl);
      uint32_t p[32];
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float2 x = f2_add(make_float2(__uint_as_float(d[2 * e]), __uint_as_float(d[2 * e + 1])), dd);
        x = f2_mul(x, make_float2(__uint_as_float(s[2 * e]), __uint_as_float(s[2 * e + 1])));
        p[e] = pack_bf16x2(x.x, x.y);
      }
      if (masked) {
        // a row without a finite delta (behind the end) passes nothing on either
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          if (2 * e > end) p[e] = 0u;
          if (2 * e == end) p[e] &= 0xffffu;
        }
      }
      store_half(tS, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ds_full);
    }
    if (ok && half == 0 && live) {
      delta[(int64_t)h * g.N + row] = dl;
      lse2[(int64_t)h * g.N + row] = L;
    }
    if (ok) ok = warp_wait(&sm.done, 0, abort_flag);
    if (ok) {
      tc_fence_after();
      const int base = pos - lane;  // the warp's first row
      store_acc<HD>(tbase + lane_base + QCOL_ACC, g.tau,
                    dq + ((int64_t)t.start + base) * st.dq + (int64_t)h * g.d, st.dq, t.len - base,
                    half, g.d, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (sm.abort && tid == 0) atomicOr(&ix.err[0], ERR_TIMEOUT_BIT);
  if (warp == MMA_WARP) {
    if (sm.abort) {  // products in flight land before the columns are freed
      mma_commit_warp(&sm.drain);
      if (lane == 0) mbar_wait(&sm.drain, 0, WAIT_LIMIT);
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

// ---- dk, dv ----------------------------------------------------------------------------

template <int HD>
struct SmemK {
  uint8_t k[Cfg<HD>::TILE], v[Cfg<HD>::TILE];
  uint8_t qd[Cfg<HD>::NSTK][Cfg<HD>::TILE];  // ring: q_0, dout_0, q_1, dout_1, ...
  alignas(16) float stat[Cfg<HD>::NSTK][2][ROWS];  // L and delta of the query tile in the slot
  uint64_t k_full, v_full;
  uint64_t full[Cfg<HD>::NSTK], ready[Cfg<HD>::NSTK], empty[Cfg<HD>::NSTK];
  uint64_t s_full, dp_full, p_full, ds_full;
  uint64_t done, drain;
  uint32_t tmem_base;
  int32_t abort;
};

// Tensor memory: S^T (P over it), dP^T (dS over it), dk, dv.
constexpr uint32_t KCOL_S = 0, KCOL_DP = 128, KCOL_DK = 256;

template <int HD>
__global__ void __launch_bounds__(NT, 1)
    k_seq_dkdv(SeqGeo g, Strides st, pack3d_seq_index ix, const __grid_constant__ MapsB maps,
               const float* delta, const float* lse2, __nv_bfloat16* dk, __nv_bfloat16* dv) {
  using C = Cfg<HD>;
  constexpr int NSEG = C::NSEG, NST = C::NSTK;
  constexpr uint32_t KCOL_DV = KCOL_DK + HD;
  overlapped_start();
  const int hk = blockIdx.x % g.Hk;
  const Tile t = load_tile_entry(ix.key, blockIdx.x / g.Hk);
  const int64_t window = (int64_t)(blockIdx.x / g.Hk) * ROWS;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  if (unused_rows(g, now.rows, window, ROWS)) {
    zero_unused(g, now.rows, window, ROWS, dk + (int64_t)hk * g.d, st.dk);
    zero_unused(g, now.rows, window, ROWS, dv + (int64_t)hk * g.d, st.dv);
  }
  if (t.len == 0) return;
  extern __shared__ uint8_t smem_raw[];
  SmemK<HD>& sm = *reinterpret_cast<SmemK<HD>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                                ~(uintptr_t)1023);
  volatile int32_t* abort_flag = &sm.abort;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // query tiles of a head that see these keys, and all steps (heads of the group
  // one after the other)
  const int first = g.causal ? t.off / ROWS : 0;
  const int per = (t.len + ROWS - 1) / ROWS - first, n = per * g.G;
  const bool ragged = (t.len & (ROWS - 1)) != 0;

  if (tid == 0) {
    mbar_init(&sm.k_full, 1);
    mbar_init(&sm.v_full, 1);
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.ready[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.p_full, 8);  // one arrival per elementwise warp
    mbar_init(&sm.ds_full, 8);
    mbar_init(&sm.done, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == TMA_WARP && lane == 0) {
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
    tma_prefetch_map(&maps.dout);
  }
  if (warp == MMA_WARP) {
    tmem_alloc(&sm.tmem_base, TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tbase = sm.tmem_base;

  if (warp >= 8) {
    regs_dec<OTHER_REGS>();
  if (warp == TMA_WARP) {
    int issued = 0;
    if (lane == 0) {
      bool ok = true;
      const int key0 = t.start + t.off;
      mbar_arrive_expect_tx(&sm.k_full, C::TILE);
      load_tile_tma<NSEG>(sm.k, &maps.k, hk, key0, &sm.k_full);
      int h = hk * g.G, qt = first;
      for (int i = 0; i < 2 * n && ok; ++i) {
        const int s = i % NST, round = i / NST;
        if (round > 0 &&
            !(ok = mbar_wait_or_abort(&sm.empty[s], (round - 1) & 1, WAIT_LIMIT, abort_flag)))
          break;
        mbar_arrive_expect_tx(&sm.full[s], C::TILE);
        load_tile_tma<NSEG>(sm.qd[s], (i & 1) ? &maps.dout : &maps.q, h, t.start + qt * ROWS,
                            &sm.full[s]);
        if (i == 0) {
          mbar_arrive_expect_tx(&sm.v_full, C::TILE);
          load_tile_tma<NSEG>(sm.v, &maps.v, hk, key0, &sm.v_full);
        }
        issued = i + 1;
        if ((i & 1) && ++qt == first + per) {
          qt = first;
          ++h;
        }
      }
      // copies in flight land before the CTA ends (bounded)
      mbar_wait(&sm.k_full, 0, WAIT_LIMIT);
      if (issued > 0) mbar_wait(&sm.v_full, 0, WAIT_LIMIT);
      for (int i = max(0, issued - NST); i < issued; ++i)
        mbar_wait(&sm.full[i % NST], (i / NST) & 1, WAIT_LIMIT);
    }
    __syncwarp();
  } else if (warp == STAT_WARP) {
    // Statistics of each query tile, and zeros behind the sequence's end: every
    // streamed tile becomes `ready` here.
    int h = hk * g.G, qt = first;
    for (int i = 0; i < 2 * n; ++i) {
      const int s = i % NST;
      float L[4], dl[4];
      if (!(i & 1)) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int pos = qt * ROWS + 4 * lane + e;
          const int64_t at = (int64_t)h * g.N + t.start + pos;
          // a weight of 0 behind the end
          L[e] = pos < t.len ? lse2[at] : INFINITY;
          dl[e] = pos < t.len ? delta[at] : 0.f;
        }
      }
      // (the slot's last readers are done: its copy was issued after `empty`)
      if (!warp_wait(&sm.full[s], (i / NST) & 1, abort_flag)) break;
      if (!(i & 1)) {
        *reinterpret_cast<float4*>(&sm.stat[s][0][4 * lane]) =
            make_float4(-L[0], -L[1], -L[2], -L[3]);
        *reinterpret_cast<float4*>(&sm.stat[s][1][4 * lane]) =
            make_float4(-dl[0], -dl[1], -dl[2], -dl[3]);
      }
      if (ragged && qt == first + per - 1) zero_rows<NSEG>(sm.qd[s], t.len & (ROWS - 1), lane);
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ready[s]);
      if ((i & 1) && ++qt == first + per) {
        qt = first;
        ++h;
      }
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    constexpr uint32_t idesc_s = idesc_bf16(ROWS, ROWS, false);
    constexpr uint32_t idesc_o = idesc_bf16(ROWS, HD, true);
    const uint64_t kd = sdesc_sw128(smem_u32(sm.k)), vd = sdesc_sw128(smem_u32(sm.v));
    const uint64_t ring = sdesc_sw128(smem_u32(sm.qd[0]));
    auto slot = [&](int i) { return ring + (uint64_t)(((i % NST) * C::TILE) >> 4); };
    auto wait_item = [&](int i) {
      return warp_wait(&sm.ready[i % NST], (i / NST) & 1, abort_flag);
    };
    auto issue_first = [&](int item, uint64_t a, uint32_t col, uint64_t* bar) -> bool {
      if (!wait_item(item)) return false;
      tc_fence_after();
      const uint64_t b = slot(item);
#pragma unroll
      for (int s = 0; s < HD / 16; ++s)
        mma_ss_warp(tbase + col, a + k_step(s), b + k_step(s), idesc_s, s > 0);
      mma_commit_warp(bar);
      return true;
    };
    auto issue_acc = [&](int item, uint32_t col, uint32_t acc, bool add) {
      const uint64_t b = slot(item);
#pragma unroll
      for (int s = 0; s < ROWS / 16; ++s)
        mma_ts_warp(tbase + acc, tbase + col + (s >> 2) * 64 + (s & 3) * 8, b + row_step(s),
                    idesc_o, (add || s > 0) ? 1u : 0u);
      mma_commit_warp(&sm.empty[item % NST]);
    };
    bool ok = warp_wait(&sm.k_full, 0, abort_flag) && issue_first(0, kd, KCOL_S, &sm.s_full) &&
              warp_wait(&sm.v_full, 0, abort_flag) && issue_first(1, vd, KCOL_DP, &sm.dp_full);
    for (int i = 0; i < n && ok; ++i) {
      if (!(ok = warp_wait(&sm.p_full, i & 1, abort_flag))) break;
      tc_fence_after();
      issue_acc(2 * i + 1, KCOL_S, KCOL_DV, i > 0);  // dv += P^T dout
      if (i + 1 < n && !(ok = issue_first(2 * i + 2, kd, KCOL_S, &sm.s_full))) break;
      if (!(ok = warp_wait(&sm.ds_full, i & 1, abort_flag))) break;
      tc_fence_after();
      issue_acc(2 * i, KCOL_DP, KCOL_DK, i > 0);  // dk += dS^T q
      if (i + 1 < n)
        ok = issue_first(2 * i + 3, vd, KCOL_DP, &sm.dp_full);
      else
        mma_commit_warp(&sm.done);
    }
    __syncwarp();
  }
  } else {
    regs_inc<ARITH_REGS>();
    const int half = warp >> 2, r = tid & (ROWS - 1);
    const int pos = t.off + r;
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_base + KCOL_S + 64 * half;
    const uint32_t tP = tbase + lane_base + KCOL_DP + 64 * half;
    const float c2 = g.tau * LOG2E;
    const float2 cc = make_float2(c2, c2);
    bool ok = true;
    int qt = first;
    for (int i = 0; i < n; ++i) {
      const int s = (2 * i) % NST;
      if (!(ok = warp_wait(&sm.ready[s], ((2 * i) / NST) & 1, abort_flag))) break;
      const float4* stat = reinterpret_cast<const float4*>(sm.stat[s][0] + 64 * half);
      float4 v[16];  // -L, then -delta of this half's columns
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = stat[e];
      if (!(ok = warp_wait(&sm.s_full, i & 1, abort_flag))) break;
      tc_fence_after();
      uint32_t x[64], p[32];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(x + 32 * c));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        const float2 y = f2_fma(
            make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), cc,
            e & 1 ? make_float2(v[e / 2].z, v[e / 2].w) : make_float2(v[e / 2].x, v[e / 2].y));
        x[2 * e] = __float_as_uint(ex2(y.x));
        x[2 * e + 1] = __float_as_uint(ex2(y.y));
      }
      if (g.causal && qt == first) {
        // the diagonal tile: query column c sees key row r where c >= r
        const int from = r - 64 * half;
#pragma unroll
        for (int c = 0; c < 64; ++c)
          if (c < from) x[c] = 0u;
      }
#pragma unroll
      for (int e = 0; e < 32; ++e)
        p[e] = pack_bf16x2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1]));
      store_half(tS, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.p_full);
#pragma unroll
      for (int e = 0; e < 16; ++e) v[e] = stat[ROWS / 4 + e];
      if (!(ok = warp_wait(&sm.dp_full, i & 1, abort_flag))) break;
      tc_fence_after();
      uint32_t y[64];
#pragma unroll
      for (int c = 0; c < 2; ++c)
        tmem_ld32(tP + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(y + 32 * c));
      tmem_wait_ld();
#pragma unroll
      for (int e = 0; e < 32; ++e) {
        float2 z = f2_add(
            make_float2(__uint_as_float(y[2 * e]), __uint_as_float(y[2 * e + 1])),
            e & 1 ? make_float2(v[e / 2].z, v[e / 2].w) : make_float2(v[e / 2].x, v[e / 2].y));
        z = f2_mul(z, make_float2(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])));
        p[e] = pack_bf16x2(z.x, z.y);
      }
      store_half(tP, p);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.ds_full);
      if (++qt == first + per) qt = first;
    }
    if (ok) ok = warp_wait(&sm.done, 0, abort_flag);
    if (ok) {
      tc_fence_after();
      const int base = pos - lane;  // the warp's first row
      const int64_t row = (int64_t)t.start + base;
      store_acc<HD>(tbase + lane_base + KCOL_DK, g.tau, dk + row * st.dk + (int64_t)hk * g.d, st.dk,
                    t.len - base, half, g.d, lane);
      store_acc<HD>(tbase + lane_base + KCOL_DV, 1.f, dv + row * st.dv + (int64_t)hk * g.d, st.dv,
                    t.len - base, half, g.d, lane);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (sm.abort && tid == 0) atomicOr(&ix.err[0], ERR_TIMEOUT_BIT);
  if (warp == MMA_WARP) {
    if (sm.abort) {
      mma_commit_warp(&sm.drain);
      if (lane == 0) mbar_wait(&sm.drain, 0, WAIT_LIMIT);
      __syncwarp();
    }
    tc_fence_after();
    tmem_dealloc(tbase, TMEM_COLS);
  }
}

template <int HD>
int backward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const void* q,
             const void* k, const void* v, const void* out, const float* lse, const void* dout,
             void* dq, void* dk, void* dv, float* delta, float* lse2, cudaStream_t s) {
  MapsB maps;
  if (!encode_rows(&maps.q, q, g.d, g.Hq, g.N, st.q, ROWS) ||
      !encode_rows(&maps.k, k, g.d, g.Hk, g.N, st.k, ROWS) ||
      !encode_rows(&maps.v, v, g.d, g.Hk, g.N, st.v, ROWS) ||
      !encode_rows(&maps.dout, dout, g.d, g.Hq, g.N, st.dout, ROWS) ||
      !encode_rows(&maps.out, out, g.d, g.Hq, g.N, st.out, ROWS))
    return PACK3D_ERR_CUDA;
  constexpr size_t bq = sizeof(SmemQ<HD>) + 1024, bk = sizeof(SmemK<HD>) + 1024;
  static_assert(bq <= 232448 && bk <= 232448, "shared memory of a CTA");
  if (!allow_smem<k_seq_dq<HD>>(bq) || !allow_smem<k_seq_dkdv<HD>>(bk)) return PACK3D_ERR_CUDA;
  using B = __nv_bfloat16;
  count_launches(2);
  const int rc = launch_overlapped(k_seq_dq<HD>, (unsigned)(g.n_rows * g.Hq), NT, bq, s, g, st, *ix,
                                   maps, lse, delta, lse2, (B*)dq);
  if (rc) return rc;
  return launch_overlapped(k_seq_dkdv<HD>, (unsigned)(g.n_rows * g.Hk), NT, bk, s, g, st, *ix, maps,
                           (const float*)delta, (const float*)lse2, (B*)dk, (B*)dv);
}

}  // namespace

int launch_backward_tc(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                       const void* q, const void* k, const void* v, const void* out,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv,
                       float* delta, float* lse2, cudaStream_t s) {
#define P3D_ARGS g, st, ix, q, k, v, out, lse, dout, dq, dk, dv, delta, lse2, s
  if (g.d <= 64) return backward<64>(P3D_ARGS);
  if (g.d <= 96) return backward<96>(P3D_ARGS);
  return backward<128>(P3D_ARGS);
#undef P3D_ARGS
}

}  // namespace seq
}  // namespace p3d
