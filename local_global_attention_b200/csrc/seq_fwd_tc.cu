// Packed-sequence attention, forward, on the Blackwell tensor cores (bf16 in,
// fp32 accumulate).
//
//   S_ij = tau q_i . k_j over the row's own sequence (j <= i when causal),
//   out_i = sum_j exp(S_ij - lse_i) v_j,  lse_i = ln sum_j exp S_ij,
// in one pass over the keys with a running maximum m and sum l: per key tile
//   P = 2^(c S - m),  l += row sum of P,  O += P v,   c = tau log2 e,
// and out = O / l.  m moves only when a row's maximum grows by more than 8
// (log2 units), so O, in tensor memory, is rarely rescaled; P then stays below
// 2^8, which bf16 holds as precisely as values below 1.  l sums the unrounded P
// in fp32; P is rounded to bf16 as the operand of the product with v.
//
// One CTA per (256 query rows of a sequence, head): two tiles of 128 rows that
// share every key/value tile loaded, which halves the L2 reads per product (a
// 128-row CTA would need 64 bytes per clock and SM at head_dim 128, about twice
// what L2 gives).  Roles:
//   * warps 0-3 and 4-7: the softmax of tile 0 and of tile 1, a row per thread;
//   * warp 8: the MMAs (one elected lane), ordered
//       S0(0) S1(0) | PV0(j) S0(j+1) PV1(j) S1(j+1) | ...
//     so one tile's products run while the other tile's softmax works;
//   * warp 9: TMA loads of q, k and v, and zeros over the v rows behind the
//     sequence's end in its last tile.
// Tensor memory: S0, S1 (128 columns of fp32 each; P as bf16 over the first 64),
// O0, O1.  The products of one tile are issued in order, so S(j+1) over P(j)
// needs no wait for PV(j), and a softmax warp that sees S(j) complete knows that
// PV(j-1) is too, when it rescales O.
//
// Masked logits are set to -inf by a select in the tiles that need it: the
// diagonal one, and the last one of a sequence whose length is no multiple of
// 128.  Every wait is bounded; a CTA that gives up sets the timeout bit of the
// index's error word.
//
// Measured: a causal sequence of 32,768 tokens, 16 heads on 2, d 128, 3.65-3.87 ms
// (1,140-1,200 TFLOP/s, 0.69-0.73 of the measured burst rate; at 990 W the clock falls
// to 1.57 GHz); 16,384 tokens not causal, 8 heads, d 96, 0.97-1.01 ms.  Bound by the
// chain S - softmax - P v of a tile (3,230 cycles a step of both tiles at d 128,
// 2,960 at d 96, against 2,140 and 1,610 of tensor work) and, in long runs, by
// power.  Short sequences pay about 7,000 cycles per CTA for set-up, first loads
// and output.
#include <cuda.h>
#include <math.h>

#include "seq_tc.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int MMA_WARP = 8, TMA_WARP = 9, NT = 384;
constexpr uint32_t TMEM_COLS = 512, COL_S = 0, COL_O = 256;
constexpr float RESCALE_THRESHOLD = 8.0f;
// P is handed to its product in two halves (whole: 920, quarters: 939 against
// 884 us at 16,384 tokens, d 96, not causal, on a cool GPU).
constexpr int PARTS = 2;

template <int HD>
struct Cfg {
  static constexpr int NSEG = HD > 64 ? 2 : 1;
  static constexpr uint32_t TILE = NSEG * SEG;
  // key and value tiles in flight: what 227 KB hold beside the two query tiles
  static constexpr int NST = HD > 64 ? 5 : 8;
};

template <int HD>
struct Smem {
  uint8_t q[2][Cfg<HD>::TILE];
  uint8_t kv[Cfg<HD>::NST][Cfg<HD>::TILE];  // ring: k_0, v_0, k_1, v_1, ...
  uint64_t q_full[2];
  uint64_t full[Cfg<HD>::NST], empty[Cfg<HD>::NST];
  uint64_t s_full[2];     // S of the tile's next key tile computed
  uint64_t p_full[2][PARTS];  // a part of P's columns written
  uint64_t o_done[2];     // every product of the tile done
  uint64_t v_fixed;       // rows behind the sequence's end are zero
  uint64_t drain;
  uint32_t tmem_base;
  int32_t abort;
};

struct Maps {
  CUtensorMap q, k, v;
  CUtensorMap out;  // boxes of 32 rows
};

// P = 2^(S c - m) of 32 keys into 16 words; returns the sum.
__device__ __forceinline__ float exp_pack(const uint32_t* sv, float c2, float mneg, uint32_t* p) {
  float2 acc[2] = {make_float2(0.f, 0.f), make_float2(0.f, 0.f)};
  const float2 cc = make_float2(c2, c2), mm = make_float2(mneg, mneg);
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const float2 a = f2_fma(make_float2(__uint_as_float(sv[2 * i]), __uint_as_float(sv[2 * i + 1])),
                            cc, mm);
    const float2 e = make_float2(ex2(a.x), ex2(a.y));
    acc[i & 1] = f2_add(acc[i & 1], e);
    p[i] = pack_bf16x2(e.x, e.y);
  }
  const float2 t = f2_add(acc[0], acc[1]);
  return t.x + t.y;
}

template <int HD>
__global__ void __launch_bounds__(NT, 1)
    k_seq_forward_tc(SeqGeo g, int64_t stride_out, pack3d_seq_index ix,
                     const __grid_constant__ Maps maps, __nv_bfloat16* out, float* lse) {
  using C = Cfg<HD>;
  constexpr int NSEG = C::NSEG, NST = C::NST;
  overlapped_start();
  const int h = blockIdx.x % g.Hq;
  const Tile t = load_tile_entry(ix.pair, blockIdx.x / g.Hq);
  const int64_t window = (int64_t)(blockIdx.x / g.Hq) * PAIR;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  if (unused_rows(g, now.rows, window, PAIR)) {
    zero_unused(g, now.rows, window, PAIR, out + (int64_t)h * g.d, stride_out);
    const int64_t row = window + threadIdx.x;
    if (threadIdx.x < PAIR && row >= now.rows && row < g.N) lse[(int64_t)h * g.N + row] = 0.f;
  }
  if (t.len == 0) return;
  extern __shared__ uint8_t smem_raw[];
  Smem<HD>& sm = *reinterpret_cast<Smem<HD>*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) &
                                              ~(uintptr_t)1023);
  volatile int32_t* abort_flag = &sm.abort;
  const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
  // key tiles that each query tile visits (the second one may have no rows)
  auto tiles_of = [&](int i) {
    const int first = t.off + i * ROWS;
    if (first >= t.len) return 0;
    return ((g.causal ? min(t.len, first + ROWS) : t.len) + ROWS - 1) / ROWS;
  };
  const int n0 = tiles_of(0), n1 = tiles_of(1), n = max(n0, n1);
  const bool fix = n * ROWS > t.len;  // the last key tile ends behind the sequence

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&sm.q_full[i], 1);
      mbar_init(&sm.s_full[i], 1);
      for (int p = 0; p < PARTS; ++p)
        mbar_init(&sm.p_full[i][p], 4);  // one arrival per softmax warp
      mbar_init(&sm.o_done[i], 1);
    }
    for (int s = 0; s < NST; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    mbar_init(&sm.v_fixed, 1);
    mbar_init(&sm.drain, 1);
    sm.abort = 0;
    fence_barrier_init();
  }
  if (warp == TMA_WARP && lane == 0) {
    tma_prefetch_map(&maps.q);
    tma_prefetch_map(&maps.k);
    tma_prefetch_map(&maps.v);
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

  if (warp >= 8) {
    regs_dec<OTHER_REGS>();
  if (warp == TMA_WARP) {
    // ================= TMA producer (lane 0) =================
    const int hk = h / g.G, row0 = t.start + t.off;
    int issued = 0;
    if (lane == 0) {
      bool ok = true;
      mbar_arrive_expect_tx(&sm.q_full[0], C::TILE);
      load_tile_tma<NSEG>(sm.q[0], &maps.q, h, row0, &sm.q_full[0]);
      for (int i = 0; i < 2 * n && ok; ++i) {
        const int s = i % NST, round = i / NST;
        if (round > 0 &&
            !(ok = mbar_wait_or_abort(&sm.empty[s], (round - 1) & 1, WAIT_LIMIT, abort_flag)))
          break;
        mbar_arrive_expect_tx(&sm.full[s], C::TILE);
        load_tile_tma<NSEG>(sm.kv[s], (i & 1) ? &maps.v : &maps.k, hk, t.start + (i / 2) * ROWS,
                            &sm.full[s]);
        if (i == 0 && n1 > 0) {
          mbar_arrive_expect_tx(&sm.q_full[1], C::TILE);
          load_tile_tma<NSEG>(sm.q[1], &maps.q, h, row0 + ROWS, &sm.q_full[1]);
        }
        issued = i + 1;
      }
    }
    issued = __shfl_sync(0xffffffffu, issued, 0);
    if (fix && issued == 2 * n) {
      const int i = 2 * n - 1, s = i % NST;
      if (warp_wait(&sm.full[s], (i / NST) & 1, abort_flag)) {
        zero_rows<NSEG>(sm.kv[s], t.len - (n - 1) * ROWS, lane);
        if (lane == 0) mbar_arrive(&sm.v_fixed);
      }
    }
    // Copies still in flight must land before the CTA ends (bounded).
    if (lane == 0) {
      mbar_wait(&sm.q_full[0], 0, WAIT_LIMIT);
      if (n1 > 0 && issued > 0) mbar_wait(&sm.q_full[1], 0, WAIT_LIMIT);
      for (int i = max(0, issued - NST); i < issued; ++i)
        mbar_wait(&sm.full[i % NST], (i / NST) & 1, WAIT_LIMIT);
    }
    __syncwarp();
  } else if (warp == MMA_WARP) {
    // ================= MMA issue (the whole warp, converged; one lane issues) =================
    constexpr uint32_t idesc_s = idesc_bf16(ROWS, ROWS, false);
    constexpr uint32_t idesc_o = idesc_bf16(ROWS, HD, true);
    const uint64_t qd = sdesc_sw128(smem_u32(sm.q[0])), kvd = sdesc_sw128(smem_u32(sm.kv[0]));
    auto wait_item = [&](int i) {
      return warp_wait(&sm.full[i % NST], (i / NST) & 1, abort_flag);
    };
    auto issue_s = [&](int i, int j) {
      const uint32_t dS = tbase + COL_S + ROWS * i;
      const uint64_t a = qd + (uint64_t)((i * C::TILE) >> 4);
      const uint64_t b = kvd + (uint64_t)((((2 * j) % NST) * C::TILE) >> 4);
#pragma unroll
      for (int st = 0; st < HD / 16; ++st)
        mma_ss_warp(dS, a + k_step(st), b + k_step(st), idesc_s, st > 0);
      mma_commit_warp(&sm.s_full[i]);
    };
    auto issue_pv = [&](int i, int j, int part) {
      const uint32_t pS = tbase + COL_S + ROWS * i;
      const uint64_t b = kvd + (uint64_t)((((2 * j + 1) % NST) * C::TILE) >> 4);
#pragma unroll
      for (int x = 0; x < 8 / PARTS; ++x) {
        const int st = part * (8 / PARTS) + x;
        mma_ts_warp(tbase + COL_O + HD * i, pS + 8 * st, b + row_step(st), idesc_o,
                    (j > 0 || st > 0) ? 1u : 0u);
      }
    };
    bool ok = warp_wait(&sm.q_full[0], 0, abort_flag) && wait_item(0);
    if (ok) {
      tc_fence_after();
      issue_s(0, 0);
      if (n1 > 0 && (ok = warp_wait(&sm.q_full[1], 0, abort_flag))) {
        tc_fence_after();
        issue_s(1, 0);
      }
      mma_commit_warp(&sm.empty[0]);
    }
    for (int j = 0; j < n && ok; ++j) {
      if (!(ok = wait_item(2 * j + 1))) break;
      if (fix && j == n - 1 && !(ok = warp_wait(&sm.v_fixed, 0, abort_flag))) break;
      if (j + 1 < n && !(ok = wait_item(2 * j + 2))) break;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int ni = i ? n1 : n0;
        if (j >= ni || !ok) continue;
#pragma unroll
        for (int part = 0; part < PARTS; ++part) {
          if (!(ok = warp_wait(&sm.p_full[i][part], j & 1, abort_flag))) break;
          tc_fence_after();
          issue_pv(i, j, part);
        }
        if (!ok) break;
        if (j + 1 < ni)
          issue_s(i, j + 1);
        else
          mma_commit_warp(&sm.o_done[i]);
      }
      mma_commit_warp(&sm.empty[(2 * j + 1) % NST]);
      if (j + 1 < n) mma_commit_warp(&sm.empty[(2 * j + 2) % NST]);
    }
    __syncwarp();
  }
  } else {
    regs_inc<ARITH_REGS>();
    // ================= softmax (one query row per thread) =================
    const int i = warp >> 2, ni = i ? n1 : n0;
    const int r = tid & (ROWS - 1);
    const int pos = t.off + i * ROWS + r;  // position in the sequence
    const uint32_t lane_base = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tbase + lane_base + COL_S + ROWS * i;
    const uint32_t tO = tbase + lane_base + COL_O + HD * i;
    const float c2 = g.tau * LOG2E;
    float m_run = -INFINITY, l_run = 0.f;
    bool ok = true;
    for (int j = 0; j < ni; ++j) {
      if (!(ok = warp_wait(&sm.s_full[i], j & 1, abort_flag))) break;
      tc_fence_after();
      uint32_t sv[ROWS];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        tmem_ld32(tS + 32 * c, *reinterpret_cast<uint32_t(*)[32]>(sv + 32 * c));
      tmem_wait_ld();
      // the diagonal tile, or the end of the sequence
      const bool masked = j == ni - 1 && (g.causal || fix);
      const int last = min(g.causal ? pos : t.len - 1, t.len - 1) - j * ROWS;
      if (masked) {
#pragma unroll
        for (int c = 0; c < ROWS; ++c)
          if (c > last) sv[c] = 0xff800000u;
      }
      float mx[4];
#pragma unroll
      for (int c = 0; c < 4; ++c)
        mx[c] = fmaxf(__uint_as_float(sv[2 * c]), __uint_as_float(sv[2 * c + 1]));
#pragma unroll
      for (int c = 8; c < ROWS; c += 2)
        mx[(c / 2) & 3] = max3(mx[(c / 2) & 3], __uint_as_float(sv[c]), __uint_as_float(sv[c + 1]));
      const float top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * c2;
      float corr = 1.f;
      if (top > m_run + RESCALE_THRESHOLD) {
        corr = ex2(m_run - top);
        l_run *= corr;
        m_run = top;
      }
      if (j > 0 && __any_sync(0xffffffffu, corr != 1.f)) {
        // (Unrolled at 64 and 128; at 96 the compiler then spills 52 bytes in the row
        // loop: 40.9 against 38.7 us for a ragged batch.  Rolled at 128: 3.89
        // against 3.72 ms for 32,768 tokens.)
        constexpr int UNROLL = HD == 96 ? 1 : HD / 32;
#pragma unroll UNROLL
        for (int c = 0; c < HD / 32; ++c) {
          uint32_t o[32];
          tmem_ld32(tO + 32 * c, o);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * corr);
          tmem_st32(tO + 32 * c, o);
        }
      }
      // a row of -inf logits only (none of finite inputs has one) stays at weight 0
      const float mneg = m_run == -INFINITY ? 0.f : -m_run;
#pragma unroll
      for (int part = 0; part < PARTS; ++part) {
        constexpr int W = ROWS / PARTS / 2;  // words of a part
        uint32_t p[W];
#pragma unroll
        for (int c = 0; c < W / 16; ++c)
          l_run += exp_pack(sv + 2 * W * part + 32 * c, c2, mneg, p + 16 * c);
#pragma unroll
        for (int c = 0; c < W / 16; ++c)
          tmem_st16(tS + W * part + 16 * c, *reinterpret_cast<uint32_t(*)[16]>(p + 16 * c));
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[i][part]);
      }
    }
    if (ok && ni > 0) ok = warp_wait(&sm.o_done[i], 0, abort_flag);
    if (ok && ni > 0) {
      tc_fence_after();
      const float inv = 1.f / l_run;
      const int64_t row = (int64_t)t.start + pos;
      if (pos < t.len) lse[(int64_t)h * g.N + row] = (m_run + log2f(l_run)) * LN2;
      // Out through the query tile's shared memory (every product that read it is
      // done), in the layout the query came in, by TMA where the warp's 32 rows are
      // all the sequence's, else by pieces of 128 bytes.  Straight from registers, a
      // row per lane, the stores took 2,600 cycles at 128 channels (shortest training
      // step at d 96: forward 9.9 against 8.2 us).
      uint8_t* tile = sm.q[i];
#pragma unroll 1
      for (int c0 = 0; c0 < HD; c0 += 32) {
        uint32_t o[32];
        tmem_ld32(tO + c0, o);
        tmem_wait_ld();
        uint8_t* to = tile + (c0 >> 6) * SEG + r * 128;
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t w[4];
#pragma unroll
          for (int x = 0; x < 4; ++x)
            w[x] = pack_bf16x2(__uint_as_float(o[8 * c + 2 * x]) * inv,
                               __uint_as_float(o[8 * c + 2 * x + 1]) * inv);
          *reinterpret_cast<uint4*>(to + ((((c0 & 32) >> 3) + c) ^ (r & 7)) * 16) =
              make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      const int first = pos - lane, live = t.len - first;  // the warp's first row, its rows
      tile += (r - lane) * 128;
      if (live >= 32) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
#pragma unroll
          for (int s = 0; s < NSEG; ++s)
            tma_store_3d(&maps.out, tile + s * SEG, 64 * s, h, t.start + first);
          tma_store_wait();
        }
      } else {
        __syncwarp();
        __nv_bfloat16* dst = out + (row - lane) * stride_out + (int64_t)h * g.d;
        for (int x = lane; x < live * 8 * NSEG; x += 32) {
          const int rr = x / (8 * NSEG), c = x % (8 * NSEG);
          if (8 * c < g.d)
            *reinterpret_cast<uint4*>(dst + rr * stride_out + 8 * c) =
                *reinterpret_cast<const uint4*>(tile + (c >> 3) * SEG + rr * 128 +
                                                (((c & 7) ^ (rr & 7)) << 4));
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (sm.abort && tid == 0) atomicOr(&ix.err[0], ERR_TIMEOUT_BIT);
  if (warp == MMA_WARP) {
    // A CTA that gave up may still have products in flight: they land before
    // the columns are freed (bounded).
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
int forward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const void* q,
            const void* k, const void* v, void* out, float* lse, cudaStream_t s) {
  Maps maps;
  if (!encode_rows(&maps.q, q, g.d, g.Hq, g.N, st.q, ROWS) ||
      !encode_rows(&maps.k, k, g.d, g.Hk, g.N, st.k, ROWS) ||
      !encode_rows(&maps.v, v, g.d, g.Hk, g.N, st.v, ROWS) ||
      !encode_rows(&maps.out, out, g.d, g.Hq, g.N, st.out, 32))
    return PACK3D_ERR_CUDA;
  constexpr size_t bytes = sizeof(Smem<HD>) + 1024;  // + alignment slack
  static_assert(bytes <= 232448, "shared memory of a CTA");
  if (!allow_smem<k_seq_forward_tc<HD>>(bytes)) return PACK3D_ERR_CUDA;
  count_launches(1);
  return launch_overlapped(k_seq_forward_tc<HD>, (unsigned)(g.n_pair * g.Hq), NT, bytes, s, g, st.out,
                           *ix, maps, (__nv_bfloat16*)out, lse);
}

}  // namespace

int launch_forward_tc(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                      const void* q, const void* k, const void* v, void* out, float* lse,
                      cudaStream_t s) {
  if (g.d <= 64) return forward<64>(g, st, ix, q, k, v, out, lse, s);
  if (g.d <= 96) return forward<96>(g, st, ix, q, k, v, out, lse, s);
  return forward<128>(g, st, ix, q, k, v, out, lse, s);
}

}  // namespace seq
}  // namespace p3d
