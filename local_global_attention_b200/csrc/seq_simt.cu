// Packed-sequence attention on the CUDA cores in fp32 throughout (the fp32 mode).
//
//   S_ij = tau q_i . k_j, P = softmax over the row's own sequence, out = P v,
//   lse = ln sum exp S;   delta_i = dout_i . out_i,  dS = P (dout v^T - delta),
//   dq_i = tau sum_j dS_ij k_j,  dk_j = tau sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i,
//   dk and dv summed over the query heads that share the key/value head.
//
// A block of 128 threads owns 32 rows (queries, or keys for dk and dv) and streams
// tiles of 64 columns; a thread holds 4 x 4 values of S (rows 4 ty + i, columns
// tx + 16 j) and 4 rows of the accumulators.  Operands stand in shared memory as
// rows with four floats of padding (a quarter warp's 16-byte reads of consecutive
// rows then meet no bank twice); a row of P is written and read by one half warp,
// so it needs no block barrier.  The forward keeps one pass over the keys with the
// running maximum and sum; the backward recomputes P from lse, once by query tile
// (dq) and once by key tile, where S is formed transposed, so no sum crosses blocks.
//
// Bound by fp32 FMA and the shared-memory reads that feed it (2.5 reads of a warp
// per 12 FMA in the accumulation; pairs of FMA in one instruction), and at the
// sizes of the fp32 workloads by the latency of the longest row of tiles: a
// training step of 2,000 tokens in four sequences, 4 heads, d 48, takes 0.27 ms
// (7.2 TFLOP/s; 0.29 with single FMA).  64-row blocks of 256 threads without the
// double buffer took 0.41 ms, 32-row ones 0.37; 2 x 4 values per thread and 256
// threads 0.34 (more reads per FMA).
#include <math.h>

#include "seq_internal.cuh"
#include "tc_primitives.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int TR = 32, TC = 64, NT = 128, PAD = 4, PS = TC + 4;
constexpr int SUB = ROWS / TR;  // blocks per entry of the 128-row tile lists
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// `rows` rows of d channels into an N x HD tile by asynchronous copies; missing
// rows and channels are zero.
template <int HD, int N>
__device__ __forceinline__ void load_tile(float* dst, const float* src, int64_t stride, int rows,
                                          int d) {
  constexpr int C4 = HD / 4;
  for (int i = threadIdx.x; i < N * C4; i += NT) {
    const int r = i / C4, c = (i % C4) * 4;
    if (r < rows && c < d)
      tc::cp_async16(dst + r * (HD + PAD) + c, src + r * stride + c);
    else
      tc::cp_async16_zero(dst + r * (HD + PAD) + c, src);
  }
}

// Two tiles streamed together, double-buffered: while one pair is worked on the
// next one is on its way (its latency, exposed, was two thirds of the time).
template <int HD>
struct Stream {
  static constexpr int TILE = TC * (HD + PAD);
  float* base;  // [2 buffers][2 tiles][TC][HD + PAD]
  __device__ __forceinline__ float* tile(int step, int which) const {
    return base + ((step & 1) * 2 + which) * TILE;
  }
  __device__ __forceinline__ void request(int step, const float* a, int64_t sa, const float* b,
                                          int64_t sb, int rows, int d) const {
    load_tile<HD, TC>(tile(step, 0), a, sa, rows, d);
    load_tile<HD, TC>(tile(step, 1), b, sb, rows, d);
  }
};

// s[i][j] = a_row(4 ty + i) . b_row(tx + 16 j)
template <int HD>
__device__ __forceinline__ void dot_tile(float (&s)[4][4], const float* a, const float* b, int tx,
                                         int ty) {
  float2 acc[4][4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[i][j] = make_float2(0.f, 0.f);
#pragma unroll 6
  for (int c = 0; c < HD; c += 4) {
    float4 x[4], y[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      x[i] = *reinterpret_cast<const float4*>(a + (4 * ty + i) * (HD + PAD) + c);
#pragma unroll
    for (int j = 0; j < 4; ++j)
      y[j] = *reinterpret_cast<const float4*>(b + (tx + 16 * j) * (HD + PAD) + c);
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        acc[i][j] = tc::f2_fma(make_float2(x[i].x, x[i].y), make_float2(y[j].x, y[j].y), acc[i][j]);
        acc[i][j] = tc::f2_fma(make_float2(x[i].z, x[i].w), make_float2(y[j].z, y[j].w), acc[i][j]);
      }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = acc[i][j].x + acc[i][j].y;
}

// Four rows of an accumulator: channels 2 tx + 32 j + {0, 1}, and 32 N2 + tx where
// HD is an odd multiple of 16.
template <int HD>
struct Acc {
  static constexpr int N2 = HD / 32, N1 = (HD % 32) / 16;
  float2 two[4][N2];
  float one[4][N1 ? N1 : 1];

  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < N2; ++j) two[i][j] = make_float2(0.f, 0.f);
      one[i][0] = 0.f;
    }
  }
  __device__ __forceinline__ void scale(int i, float f) {
#pragma unroll
    for (int j = 0; j < N2; ++j) {
      two[i][j].x *= f;
      two[i][j].y *= f;
    }
    one[i][0] *= f;
  }
  // row i += sum_k p[4 ty + i][k] b_row(k)
  __device__ __forceinline__ void add(const float* p, const float* b, int tx, int ty) {
#pragma unroll 4
    for (int k = 0; k < TC; k += 4) {
      float4 w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = *reinterpret_cast<const float4*>(p + (4 * ty + i) * PS + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        const float* row = b + (k + kk) * (HD + PAD);
        auto f = [&](int i) {
          return kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
        };
#pragma unroll
        for (int j = 0; j < N2; ++j) {
          const float2 y = *reinterpret_cast<const float2*>(row + 2 * tx + 32 * j);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            two[i][j] = tc::f2_fma(make_float2(f(i), f(i)), y, two[i][j]);
          }
        }
        if (N1) {
          const float y = row[32 * N2 + tx];
#pragma unroll
          for (int i = 0; i < 4; ++i) one[i][0] = fmaf(f(i), y, one[i][0]);
        }
      }
    }
  }
  __device__ __forceinline__ void store(float* dst, int64_t stride, const float (&f)[4], int rows,
                                        int d, int tx, int ty) const {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (4 * ty + i >= rows) continue;
      float* row = dst + (4 * ty + i) * stride;
#pragma unroll
      for (int j = 0; j < N2; ++j) {
        const int c = 2 * tx + 32 * j;
        if (c < d)
          *reinterpret_cast<float2*>(row + c) = make_float2(two[i][j].x * f[i], two[i][j].y * f[i]);
      }
      if (N1 && 32 * N2 + tx < d) row[32 * N2 + tx] = one[i][0] * f[i];
    }
  }
};

// This block's rows: the tile of its list entry, the first row in the sequence.
__device__ __forceinline__ bool own_rows(const int32_t* list, Tile& t, int& off, int& rows) {
  t = load_tile_entry(list, blockIdx.x / SUB);
  off = t.off + (blockIdx.x % SUB) * TR;
  rows = min(TR, t.len - off);
  return off < t.len;
}

template <int HD>
__global__ void __launch_bounds__(NT)
    k_seq_forward_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const float* __restrict__ q,
                       const float* __restrict__ k, const float* __restrict__ v,
                       float* __restrict__ out, float* __restrict__ lse) {
  Tile t;
  int off, rows;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  const int64_t window = (int64_t)blockIdx.x * TR;
  if (unused_rows(g, now.rows, window, TR)) {
    zero_unused(g, now.rows, window, TR, out + (int64_t)blockIdx.y * g.d, st.out);
    const int64_t row = window + threadIdx.x;
    if (threadIdx.x < TR && row >= now.rows && row < g.N)
      lse[(int64_t)blockIdx.y * g.N + row] = 0.f;
  }
  if (!own_rows(ix.query, t, off, rows)) return;
  extern __shared__ float sm[];
  float* sq = sm;
  const Stream<HD> kv = {sq + TR * (HD + PAD)};
  float* sp = kv.base + 4 * Stream<HD>::TILE;
  const int h = blockIdx.y, hk = h / g.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t row0 = (int64_t)t.start + off;
  load_tile<HD, TR>(sq, q + row0 * st.q + (int64_t)h * g.d, st.q, rows, g.d);
  Acc<HD> o;
  o.clear();
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
  }
  const float c2 = g.tau * LOG2E;
  const int end = g.causal ? min(t.len, off + TR) : t.len, steps = (end + TC - 1) / TC;
  auto request = [&](int i) {
    if (i < steps) {
      const int64_t key0 = (int64_t)t.start + i * TC;
      kv.request(i, k + key0 * st.k + (int64_t)hk * g.d, st.k, v + key0 * st.v + (int64_t)hk * g.d,
                 st.v, min(TC, t.len - i * TC), g.d);
    }
    tc::cp_async_commit();
  };
  request(0);
  for (int it = 0; it < steps; ++it) {
    const int k0 = it * TC, keys = min(TC, t.len - k0);
    const float *sk = kv.tile(it, 0), *sv = kv.tile(it, 1);
    request(it + 1);
    tc::cp_async_wait_group<1>();
    __syncthreads();
    float s[4][4];
    dot_tile<HD>(s, sq, sk, tx, ty);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int last = g.causal ? min(keys - 1, off + 4 * ty + i - k0) : keys - 1;
      float top = m[i];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[i][j] = tx + 16 * j <= last ? s[i][j] * c2 : -INFINITY;
        top = fmaxf(top, s[i][j]);
      }
#pragma unroll
      for (int w = 1; w < 16; w *= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      const float base = top == -INFINITY ? 0.f : top;
      const float corr = exp2f(m[i] - base);
      m[i] = top;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float e = exp2f(s[i][j] - base);
        sum += e;
        sp[(4 * ty + i) * PS + tx + 16 * j] = e;
      }
      l[i] = l[i] * corr + sum;
      o.scale(i, corr);
    }
    __syncwarp();
    o.add(sp, sv, tx, ty);
    __syncthreads();  // the buffers are read; the next request overwrites them
  }
  float f[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
#pragma unroll
    for (int w = 1; w < 16; w *= 2) l[i] += __shfl_xor_sync(0xffffffffu, l[i], w);
    f[i] = 1.f / l[i];
    if (tx == 0 && 4 * ty + i < rows)
      lse[(int64_t)h * g.N + row0 + 4 * ty + i] = (m[i] + log2f(l[i])) * LN2;
  }
  o.store(out + row0 * st.out + (int64_t)h * g.d, st.out, f, rows, g.d, tx, ty);
}

// delta[h][i] = dout_i . out_i: one warp per (row, head).
__global__ void __launch_bounds__(NT)
    k_seq_delta(SeqGeo g, Strides st, pack3d_seq_index ix, const float* __restrict__ out,
                const float* __restrict__ dout, float* __restrict__ delta) {
  if (ix.err[0]) return;
  const int64_t w = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32;
  const int64_t row = w / g.Hq;
  const int h = (int)(w % g.Hq), lane = threadIdx.x % 32;
  if (row >= g.N || ix.pos[row] < 0) return;
  float x = 0.f;
  for (int c = lane; c < g.d; c += 32)
    x = fmaf(out[row * st.out + (int64_t)h * g.d + c], dout[row * st.dout + (int64_t)h * g.d + c], x);
  for (int o = 16; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0) delta[(int64_t)h * g.N + row] = x;
}

// dq: the block's rows are queries, the columns keys.
template <int HD>
__global__ void __launch_bounds__(NT)
    k_seq_dq_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const float* __restrict__ q,
                  const float* __restrict__ k, const float* __restrict__ v,
                  const float* __restrict__ lse, const float* __restrict__ delta,
                  const float* __restrict__ dout, float* __restrict__ dq) {
  Tile t;
  int off, rows;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  const int64_t window = (int64_t)blockIdx.x * TR;
  if (unused_rows(g, now.rows, window, TR))
    zero_unused(g, now.rows, window, TR, dq + (int64_t)blockIdx.y * g.d, st.dq);
  if (!own_rows(ix.query, t, off, rows)) return;
  extern __shared__ float sm[];
  float *sq = sm, *sdo = sq + TR * (HD + PAD);
  const Stream<HD> kv = {sdo + TR * (HD + PAD)};
  float* ss = kv.base + 4 * Stream<HD>::TILE;
  const int h = blockIdx.y, hk = h / g.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t row0 = (int64_t)t.start + off;
  load_tile<HD, TR>(sq, q + row0 * st.q + (int64_t)h * g.d, st.q, rows, g.d);
  load_tile<HD, TR>(sdo, dout + row0 * st.dout + (int64_t)h * g.d, st.dout, rows, g.d);
  const float c2 = g.tau * LOG2E;
  float L[4], dl[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const bool live = 4 * ty + i < rows;
    L[i] = live ? lse[(int64_t)h * g.N + row0 + 4 * ty + i] * LOG2E : 0.f;
    dl[i] = live ? delta[(int64_t)h * g.N + row0 + 4 * ty + i] : 0.f;
  }
  Acc<HD> o;
  o.clear();
  const int end = g.causal ? min(t.len, off + TR) : t.len, steps = (end + TC - 1) / TC;
  auto request = [&](int i) {
    if (i < steps) {
      const int64_t key0 = (int64_t)t.start + i * TC;
      kv.request(i, k + key0 * st.k + (int64_t)hk * g.d, st.k, v + key0 * st.v + (int64_t)hk * g.d,
                 st.v, min(TC, t.len - i * TC), g.d);
    }
    tc::cp_async_commit();
  };
  request(0);
  for (int it = 0; it < steps; ++it) {
    const int k0 = it * TC, keys = min(TC, t.len - k0);
    const float *sk = kv.tile(it, 0), *sv = kv.tile(it, 1);
    request(it + 1);
    tc::cp_async_wait_group<1>();
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<HD>(s, sq, sk, tx, ty);
    dot_tile<HD>(dp, sdo, sv, tx, ty);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int last = g.causal ? min(keys - 1, off + 4 * ty + i - k0) : keys - 1;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        ss[(4 * ty + i) * PS + c] =
            c <= last ? exp2f(fmaf(s[i][j], c2, -L[i])) * (dp[i][j] - dl[i]) : 0.f;
      }
    }
    __syncwarp();
    o.add(ss, sk, tx, ty);
    __syncthreads();
  }
  const float f[4] = {g.tau, g.tau, g.tau, g.tau};
  o.store(dq + row0 * st.dq + (int64_t)h * g.d, st.dq, f, rows, g.d, tx, ty);
}

// dk, dv: the block's rows are keys, the columns the queries of the group's heads.
template <int HD>
__global__ void __launch_bounds__(NT)
    k_seq_dkdv_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const float* __restrict__ q,
                    const float* __restrict__ k, const float* __restrict__ v,
                    const float* __restrict__ lse, const float* __restrict__ delta,
                    const float* __restrict__ dout, float* __restrict__ dk,
                    float* __restrict__ dv) {
  Tile t;
  int off, rows;
  const State now = load_state(ix);
  if (block_failed(now)) return;
  const int64_t window = (int64_t)blockIdx.x * TR;
  if (unused_rows(g, now.rows, window, TR)) {
    zero_unused(g, now.rows, window, TR, dk + (int64_t)blockIdx.y * g.d, st.dk);
    zero_unused(g, now.rows, window, TR, dv + (int64_t)blockIdx.y * g.d, st.dv);
  }
  if (!own_rows(ix.key, t, off, rows)) return;
  extern __shared__ float sm[];
  float *sk = sm, *sv = sk + TR * (HD + PAD);
  const Stream<HD> qd = {sv + TR * (HD + PAD)};
  float *sp = qd.base + 4 * Stream<HD>::TILE, *ss = sp + TR * PS;
  const int hk = blockIdx.y, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int64_t key0 = (int64_t)t.start + off;
  load_tile<HD, TR>(sk, k + key0 * st.k + (int64_t)hk * g.d, st.k, rows, g.d);
  load_tile<HD, TR>(sv, v + key0 * st.v + (int64_t)hk * g.d, st.v, rows, g.d);
  const float c2 = g.tau * LOG2E;
  Acc<HD> ok, ov;
  ok.clear();
  ov.clear();
  const int begin = g.causal ? off / TC * TC : 0;  // the tile that holds the first key's row
  const int per = (t.len - begin + TC - 1) / TC, steps = per * g.G;
  auto request = [&](int i) {
    if (i < steps) {
      const int h = hk * g.G + i / per, q0 = begin + i % per * TC;
      const int64_t row0 = (int64_t)t.start + q0;
      qd.request(i, q + row0 * st.q + (int64_t)h * g.d, st.q,
                 dout + row0 * st.dout + (int64_t)h * g.d, st.dout, min(TC, t.len - q0), g.d);
    }
    tc::cp_async_commit();
  };
  request(0);
  int h = hk * g.G, q0 = begin;
  for (int it = 0; it < steps; ++it) {
    const int queries = min(TC, t.len - q0);
    const int64_t row0 = (int64_t)t.start + q0;
    const float *sq = qd.tile(it, 0), *sdo = qd.tile(it, 1);
    float L[4], dl[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = tx + 16 * j;
      L[j] = c < queries ? lse[(int64_t)h * g.N + row0 + c] * LOG2E : 0.f;
      dl[j] = c < queries ? delta[(int64_t)h * g.N + row0 + c] : 0.f;
    }
    request(it + 1);
    tc::cp_async_wait_group<1>();
    __syncthreads();
    float s[4][4], dp[4][4];
    dot_tile<HD>(s, sk, sq, tx, ty);
    dot_tile<HD>(dp, sv, sdo, tx, ty);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      // queries from the key's own position on
      const int first = g.causal ? off + 4 * ty + i - q0 : 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = tx + 16 * j;
        const bool seen = c >= first && c < queries;
        const float e = seen ? exp2f(fmaf(s[i][j], c2, -L[j])) : 0.f;
        sp[(4 * ty + i) * PS + c] = e;
        ss[(4 * ty + i) * PS + c] = seen ? e * (dp[i][j] - dl[j]) : 0.f;
      }
    }
    __syncwarp();
    ov.add(sp, sdo, tx, ty);
    ok.add(ss, sq, tx, ty);
    __syncthreads();
    if ((q0 += TC) >= t.len) {
      q0 = begin;
      ++h;
    }
  }
  const float fk[4] = {g.tau, g.tau, g.tau, g.tau}, fv[4] = {1.f, 1.f, 1.f, 1.f};
  ok.store(dk + key0 * st.dk + (int64_t)hk * g.d, st.dk, fk, rows, g.d, tx, ty);
  ov.store(dv + key0 * st.dv + (int64_t)hk * g.d, st.dv, fv, rows, g.d, tx, ty);
}

// `own` tiles of TR rows, two buffers of two streamed ones of TC rows, `weights` squares of P or dS.
template <int HD>
constexpr size_t smem_bytes(int own, int weights) {
  return sizeof(float) * ((size_t)(own * TR + 4 * TC) * (HD + PAD) + (size_t)weights * TR * PS);
}

template <int HD>
int forward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const float* q,
            const float* k, const float* v, float* out, float* lse, cudaStream_t s) {
  constexpr size_t bytes = smem_bytes<HD>(1, 1);
  if (!allow_smem<k_seq_forward_simt<HD>>(bytes)) return PACK3D_ERR_CUDA;
  k_seq_forward_simt<HD>
      <<<dim3(SUB * g.n_rows, g.Hq), NT, bytes, s>>>(g, st, *ix, q, k, v, out, lse);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

template <int HD>
int backward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const float* q,
             const float* k, const float* v, const float* out, const float* lse, const float* dout,
             float* dq, float* dk, float* dv, float* delta, cudaStream_t s) {
  constexpr size_t b_dq = smem_bytes<HD>(2, 1), b_kv = smem_bytes<HD>(2, 2);
  if (!allow_smem<k_seq_dq_simt<HD>>(b_dq) || !allow_smem<k_seq_dkdv_simt<HD>>(b_kv))
    return PACK3D_ERR_CUDA;
  const int64_t warps = (int64_t)g.N * g.Hq;
  k_seq_delta<<<(unsigned)((warps + NT / 32 - 1) / (NT / 32)), NT, 0, s>>>(g, st, *ix, out, dout,
                                                                          delta);
  k_seq_dq_simt<HD><<<dim3(SUB * g.n_rows, g.Hq), NT, b_dq, s>>>(g, st, *ix, q, k, v, lse, delta,
                                                                dout, dq);
  k_seq_dkdv_simt<HD><<<dim3(SUB * g.n_rows, g.Hk), NT, b_kv, s>>>(g, st, *ix, q, k, v, lse, delta,
                                                                  dout, dk, dv);
  count_launches(3);
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_forward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                        const void* q, const void* k, const void* v, void* out, float* lse,
                        cudaStream_t s) {
  using F = const float*;
#define P3D_ARGS g, st, ix, (F)q, (F)k, (F)v, (float*)out, lse, s
  if (g.d <= 48) return forward<48>(P3D_ARGS);
  if (g.d <= 64) return forward<64>(P3D_ARGS);
  if (g.d <= 96) return forward<96>(P3D_ARGS);
  return forward<128>(P3D_ARGS);
#undef P3D_ARGS
}

int launch_backward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                         const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv,
                         float* delta, cudaStream_t s) {
  using F = const float*;
#define P3D_ARGS                                                                                 \
  g, st, ix, (F)q, (F)k, (F)v, (F)out, lse, (F)dout, (float*)dq, (float*)dk, (float*)dv, delta, s
  if (g.d <= 48) return backward<48>(P3D_ARGS);
  if (g.d <= 64) return backward<64>(P3D_ARGS);
  if (g.d <= 96) return backward<96>(P3D_ARGS);
  return backward<128>(P3D_ARGS);
#undef P3D_ARGS
}

}  // namespace seq
}  // namespace p3d
