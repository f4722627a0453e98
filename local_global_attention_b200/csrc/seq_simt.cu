// Packed-sequence attention on the CUDA cores, fp32 arithmetic throughout.
//
//   S_ij = tau q_i . k_j, P = softmax over the row's own sequence, out = P v,
//   lse = ln sum exp S;   delta_i = dout_i . out_i,  dS = P (dout v^T - delta),
//   dq_i = tau sum_j dS_ij k_j,  dk_j = tau sum_i dS_ij q_i,  dv_j = sum_i P_ij dout_i,
//   dk and dv summed over the query heads that share the key/value head.
//
// 64 x 64 tiles of S, 256 threads, 4 x 4 values each (rows 4 ty + i, columns
// tx + 16 j), operands as fp32 rows in shared memory with four floats of padding
// (a quarter warp's 16-byte reads of consecutive rows then meet no bank twice).
// The forward keeps one pass over the keys with the running maximum and sum;
// the backward recomputes P from lse, in one kernel by query tile for dq and
// one by key tile for dk and dv, so no sum crosses blocks and no atomics are
// needed.  Bound by fp32 FMA and the shared-memory reads that feed it.
#include <math.h>

#include "seq_internal.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int T = 64, NT = 256, PAD = 4, PS = T + 4;
constexpr float LOG2E = 1.4426950408889634f, LN2 = 0.6931471805599453f;

// `rows` rows of d channels (row pitch `stride` elements) into a 64 x HD tile;
// missing rows and channels are zero.
template <typename E, int HD>
__device__ __forceinline__ void load_tile(float* dst, const E* src, int64_t stride, int rows,
                                          int d) {
  constexpr int C4 = HD / 4;
  for (int i = threadIdx.x; i < T * C4; i += NT) {
    const int r = i / C4, c = (i % C4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows && c < d) {
      const E* p = src + r * stride + c;
      x = make_float4(to_f32<E>(p[0]), to_f32<E>(p[1]), to_f32<E>(p[2]), to_f32<E>(p[3]));
    }
    *reinterpret_cast<float4*>(dst + r * (HD + PAD) + c) = x;
  }
}

// s[i][j] = a_row(4 ty + i) . b_row(tx + 16 j)
template <int HD>
__device__ __forceinline__ void dot_tile(float (&s)[4][4], const float* a, const float* b, int tx,
                                         int ty) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) s[i][j] = 0.f;
#pragma unroll 4
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
        s[i][j] = fmaf(x[i].x, y[j].x, s[i][j]);
        s[i][j] = fmaf(x[i].y, y[j].y, s[i][j]);
        s[i][j] = fmaf(x[i].z, y[j].z, s[i][j]);
        s[i][j] = fmaf(x[i].w, y[j].w, s[i][j]);
      }
  }
}

// o[i][..] += sum_k p[4 ty + i][k] b_row(k): channels 2 tx + 32 jj + {0, 1}
template <int HD>
__device__ __forceinline__ void acc_tile(float2 (&o)[4][HD / 32], const float* p, const float* b,
                                         int tx, int ty) {
#pragma unroll 2
  for (int k = 0; k < T; k += 4) {
    float4 w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(p + (4 * ty + i) * PS + k);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
#pragma unroll
      for (int jj = 0; jj < HD / 32; ++jj) {
        const float2 y =
            *reinterpret_cast<const float2*>(b + (k + kk) * (HD + PAD) + 2 * tx + 32 * jj);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float f = kk == 0 ? w[i].x : kk == 1 ? w[i].y : kk == 2 ? w[i].z : w[i].w;
          o[i][jj].x = fmaf(f, y.x, o[i][jj].x);
          o[i][jj].y = fmaf(f, y.y, o[i][jj].y);
        }
      }
  }
}

// As acc_tile with the transpose of p: o[i] += sum_k p[k][4 ty + i] b_row(k).
template <int HD>
__device__ __forceinline__ void acc_tile_t(float2 (&o)[4][HD / 32], const float* p, const float* b,
                                           int tx, int ty) {
#pragma unroll 4
  for (int k = 0; k < T; ++k) {
    const float4 w = *reinterpret_cast<const float4*>(p + k * PS + 4 * ty);
#pragma unroll
    for (int jj = 0; jj < HD / 32; ++jj) {
      const float2 y = *reinterpret_cast<const float2*>(b + k * (HD + PAD) + 2 * tx + 32 * jj);
      o[0][jj].x = fmaf(w.x, y.x, o[0][jj].x);
      o[0][jj].y = fmaf(w.x, y.y, o[0][jj].y);
      o[1][jj].x = fmaf(w.y, y.x, o[1][jj].x);
      o[1][jj].y = fmaf(w.y, y.y, o[1][jj].y);
      o[2][jj].x = fmaf(w.z, y.x, o[2][jj].x);
      o[2][jj].y = fmaf(w.z, y.y, o[2][jj].y);
      o[3][jj].x = fmaf(w.w, y.x, o[3][jj].x);
      o[3][jj].y = fmaf(w.w, y.y, o[3][jj].y);
    }
  }
}

template <typename E, int HD>
__device__ __forceinline__ void store_rows(E* dst, int64_t stride, const float2 (&o)[4][HD / 32],
                                           const float (&f)[4], int rows, int d, int tx, int ty) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (4 * ty + i >= rows) continue;
    E* row = dst + (4 * ty + i) * stride;
#pragma unroll
    for (int jj = 0; jj < HD / 32; ++jj) {
      const int c = 2 * tx + 32 * jj;
      if (c < d) {
        row[c] = from_f32<E>(o[i][jj].x * f[i]);
        row[c + 1] = from_f32<E>(o[i][jj].y * f[i]);
      }
    }
  }
}

// Block (x: 2 x 128-row tile + half, y: head).  The lists hold 128-row tiles;
// each is two blocks here.
template <typename E, int HD>
__global__ void __launch_bounds__(NT)
    k_seq_forward_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const E* __restrict__ q,
                       const E* __restrict__ k, const E* __restrict__ v, E* __restrict__ out,
                       float* __restrict__ lse) {
  if (ix.err[0]) return;
  const Tile t = reinterpret_cast<const Tile*>(ix.query)[blockIdx.x >> 1];
  const int off = t.off + (blockIdx.x & 1) * T;
  if (off >= t.len) return;
  extern __shared__ float sm[];
  constexpr int TILE = T * (HD + PAD);
  float *sq = sm, *sk = sm + TILE, *sv = sm + 2 * TILE, *sp = sm + 3 * TILE;
  const int h = blockIdx.y, hk = h / g.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int rows = min(T, t.len - off);
  const int64_t row0 = (int64_t)t.start + off;
  load_tile<E, HD>(sq, q + row0 * st.q + (int64_t)h * g.d, st.q, rows, g.d);
  float2 o[4][HD / 32];
  float m[4], l[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    m[i] = -INFINITY;
    l[i] = 0.f;
#pragma unroll
    for (int jj = 0; jj < HD / 32; ++jj) o[i][jj] = make_float2(0.f, 0.f);
  }
  const float c2 = g.tau * LOG2E;
  const int end = g.causal ? min(t.len, off + T) : t.len;
  for (int k0 = 0; k0 < end; k0 += T) {
    const int keys = min(T, t.len - k0);
    const int64_t key0 = (int64_t)t.start + k0;
    __syncthreads();
    load_tile<E, HD>(sk, k + key0 * st.k + (int64_t)hk * g.d, st.k, keys, g.d);
    load_tile<E, HD>(sv, v + key0 * st.v + (int64_t)hk * g.d, st.v, keys, g.d);
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
#pragma unroll
      for (int jj = 0; jj < HD / 32; ++jj) {
        o[i][jj].x *= corr;
        o[i][jj].y *= corr;
      }
    }
    __syncwarp();  // a row of sp is written and read by the same half warp
    acc_tile<HD>(o, sp, sv, tx, ty);
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
  store_rows<E, HD>(out + row0 * st.out + (int64_t)h * g.d, st.out, o, f, rows, g.d, tx, ty);
}

// delta[h][i] = dout_i . out_i: one warp per (row, head).
template <typename E>
__global__ void __launch_bounds__(NT)
    k_seq_delta(SeqGeo g, Strides st, pack3d_seq_index ix, const E* __restrict__ out,
                const E* __restrict__ dout, float* __restrict__ delta) {
  if (ix.err[0]) return;
  const int64_t w = (int64_t)blockIdx.x * (NT / 32) + threadIdx.x / 32;
  const int64_t row = w / g.Hq;
  const int h = (int)(w % g.Hq), lane = threadIdx.x % 32;
  if (row >= g.N || ix.pos[row] < 0) return;
  float x = 0.f;
  for (int c = lane; c < g.d; c += 32)
    x = fmaf(to_f32<E>(out[row * st.out + (int64_t)h * g.d + c]),
             to_f32<E>(dout[row * st.dout + (int64_t)h * g.d + c]), x);
  for (int o = 16; o; o /= 2) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0) delta[(int64_t)h * g.N + row] = x;
}

// P and dS of one tile into sp (when given) and ss, from S and dP products.
template <int HD>
__device__ __forceinline__ void grad_tile(const SeqGeo& g, const float* sq, const float* sdo,
                                          const float* sk, const float* sv, float* sp, float* ss,
                                          const float* row_lse, const float* row_delta, int rows,
                                          int keys, int q0, int k0, int tx, int ty) {
  float s[4][4], dp[4][4];
  dot_tile<HD>(s, sq, sk, tx, ty);
  dot_tile<HD>(dp, sdo, sv, tx, ty);
  const float c2 = g.tau * LOG2E;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = 4 * ty + i;
    const int last = r >= rows ? -1 : g.causal ? min(keys - 1, q0 + r - k0) : keys - 1;
    const float lse2 = r < rows ? row_lse[r] * LOG2E : 0.f, dl = r < rows ? row_delta[r] : 0.f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int c = tx + 16 * j;
      const float e = c <= last ? exp2f(fmaf(s[i][j], c2, -lse2)) : 0.f;
      const float ds = c <= last ? e * (dp[i][j] - dl) : 0.f;
      if (sp) sp[r * PS + c] = e;
      ss[r * PS + c] = ds;
    }
  }
}

template <typename E, int HD>
__global__ void __launch_bounds__(NT)
    k_seq_dq_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const E* __restrict__ q,
                  const E* __restrict__ k, const E* __restrict__ v, const float* __restrict__ lse,
                  const float* __restrict__ delta, const E* __restrict__ dout,
                  E* __restrict__ dq) {
  if (ix.err[0]) return;
  const Tile t = reinterpret_cast<const Tile*>(ix.query)[blockIdx.x >> 1];
  const int off = t.off + (blockIdx.x & 1) * T;
  if (off >= t.len) return;
  extern __shared__ float sm[];
  constexpr int TILE = T * (HD + PAD);
  float *sq = sm, *sdo = sm + TILE, *sk = sm + 2 * TILE, *sv = sm + 3 * TILE, *ss = sm + 4 * TILE;
  const int h = blockIdx.y, hk = h / g.G, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int rows = min(T, t.len - off);
  const int64_t row0 = (int64_t)t.start + off;
  load_tile<E, HD>(sq, q + row0 * st.q + (int64_t)h * g.d, st.q, rows, g.d);
  load_tile<E, HD>(sdo, dout + row0 * st.dout + (int64_t)h * g.d, st.dout, rows, g.d);
  float2 o[4][HD / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < HD / 32; ++jj) o[i][jj] = make_float2(0.f, 0.f);
  const int end = g.causal ? min(t.len, off + T) : t.len;
  for (int k0 = 0; k0 < end; k0 += T) {
    const int keys = min(T, t.len - k0);
    const int64_t key0 = (int64_t)t.start + k0;
    __syncthreads();
    load_tile<E, HD>(sk, k + key0 * st.k + (int64_t)hk * g.d, st.k, keys, g.d);
    load_tile<E, HD>(sv, v + key0 * st.v + (int64_t)hk * g.d, st.v, keys, g.d);
    __syncthreads();
    grad_tile<HD>(g, sq, sdo, sk, sv, nullptr, ss, lse + (int64_t)h * g.N + row0,
                  delta + (int64_t)h * g.N + row0, rows, keys, off, k0, tx, ty);
    __syncwarp();
    acc_tile<HD>(o, ss, sk, tx, ty);
  }
  const float f[4] = {g.tau, g.tau, g.tau, g.tau};
  store_rows<E, HD>(dq + row0 * st.dq + (int64_t)h * g.d, st.dq, o, f, rows, g.d, tx, ty);
}

template <typename E, int HD>
__global__ void __launch_bounds__(NT)
    k_seq_dkdv_simt(SeqGeo g, Strides st, pack3d_seq_index ix, const E* __restrict__ q,
                    const E* __restrict__ k, const E* __restrict__ v,
                    const float* __restrict__ lse, const float* __restrict__ delta,
                    const E* __restrict__ dout, E* __restrict__ dk, E* __restrict__ dv) {
  if (ix.err[0]) return;
  const Tile t = reinterpret_cast<const Tile*>(ix.key)[blockIdx.x >> 1];
  const int off = t.off + (blockIdx.x & 1) * T;
  if (off >= t.len) return;
  extern __shared__ float sm[];
  constexpr int TILE = T * (HD + PAD);
  float *sq = sm, *sdo = sm + TILE, *sk = sm + 2 * TILE, *sv = sm + 3 * TILE;
  float *sp = sm + 4 * TILE, *ss = sp + T * PS;
  const int hk = blockIdx.y, tx = threadIdx.x % 16, ty = threadIdx.x / 16;
  const int keys = min(T, t.len - off);
  const int64_t key0 = (int64_t)t.start + off;
  load_tile<E, HD>(sk, k + key0 * st.k + (int64_t)hk * g.d, st.k, keys, g.d);
  load_tile<E, HD>(sv, v + key0 * st.v + (int64_t)hk * g.d, st.v, keys, g.d);
  float2 ok[4][HD / 32], ov[4][HD / 32];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int jj = 0; jj < HD / 32; ++jj) ok[i][jj] = ov[i][jj] = make_float2(0.f, 0.f);
  for (int h = hk * g.G; h < (hk + 1) * g.G; ++h)
    for (int q0 = g.causal ? off : 0; q0 < t.len; q0 += T) {
      const int rows = min(T, t.len - q0);
      const int64_t row0 = (int64_t)t.start + q0;
      __syncthreads();
      load_tile<E, HD>(sq, q + row0 * st.q + (int64_t)h * g.d, st.q, rows, g.d);
      load_tile<E, HD>(sdo, dout + row0 * st.dout + (int64_t)h * g.d, st.dout, rows, g.d);
      __syncthreads();
      grad_tile<HD>(g, sq, sdo, sk, sv, sp, ss, lse + (int64_t)h * g.N + row0,
                    delta + (int64_t)h * g.N + row0, rows, keys, q0, off, tx, ty);
      __syncthreads();
      acc_tile_t<HD>(ov, sp, sdo, tx, ty);
      acc_tile_t<HD>(ok, ss, sq, tx, ty);
    }
  const float fk[4] = {g.tau, g.tau, g.tau, g.tau}, fv[4] = {1.f, 1.f, 1.f, 1.f};
  store_rows<E, HD>(dk + key0 * st.dk + (int64_t)hk * g.d, st.dk, ok, fk, keys, g.d, tx, ty);
  store_rows<E, HD>(dv + key0 * st.dv + (int64_t)hk * g.d, st.dv, ov, fv, keys, g.d, tx, ty);
}

template <int HD>
constexpr size_t smem_bytes(int tiles, int squares) {
  return sizeof(float) * ((size_t)tiles * T * (HD + PAD) + (size_t)squares * T * PS);
}

template <typename K>
bool allow_smem(K kernel, size_t bytes) {
  return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) ==
         cudaSuccess;
}

template <typename E, int HD>
int forward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const void* q,
            const void* k, const void* v, void* out, float* lse, cudaStream_t s) {
  constexpr size_t bytes = smem_bytes<HD>(3, 1);
  if (!allow_smem(k_seq_forward_simt<E, HD>, bytes)) return PACK3D_ERR_CUDA;
  k_seq_forward_simt<E, HD><<<dim3(2 * g.n_rows, g.Hq), NT, bytes, s>>>(
      g, st, *ix, (const E*)q, (const E*)k, (const E*)v, (E*)out, lse);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

template <typename E, int HD>
int backward(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix, const void* q,
             const void* k, const void* v, const void* out, const float* lse, const void* dout,
             void* dq, void* dk, void* dv, float* delta, cudaStream_t s) {
  constexpr size_t b_dq = smem_bytes<HD>(4, 1), b_kv = smem_bytes<HD>(4, 2);
  if (!allow_smem(k_seq_dq_simt<E, HD>, b_dq) || !allow_smem(k_seq_dkdv_simt<E, HD>, b_kv))
    return PACK3D_ERR_CUDA;
  const int64_t warps = (int64_t)g.N * g.Hq;
  k_seq_delta<E><<<(unsigned)((warps + NT / 32 - 1) / (NT / 32)), NT, 0, s>>>(
      g, st, *ix, (const E*)out, (const E*)dout, delta);
  k_seq_dq_simt<E, HD><<<dim3(2 * g.n_rows, g.Hq), NT, b_dq, s>>>(
      g, st, *ix, (const E*)q, (const E*)k, (const E*)v, lse, delta, (const E*)dout, (E*)dq);
  k_seq_dkdv_simt<E, HD><<<dim3(2 * g.n_rows, g.Hk), NT, b_kv, s>>>(
      g, st, *ix, (const E*)q, (const E*)k, (const E*)v, lse, delta, (const E*)dout, (E*)dk,
      (E*)dv);
  count_launches(3);
  return cuda_status(cudaGetLastError());
}

}  // namespace

int launch_forward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                        const void* q, const void* k, const void* v, void* out, float* lse,
                        cudaStream_t s) {
  if (g.d <= 64) return forward<float, 64>(g, st, ix, q, k, v, out, lse, s);
  if (g.d <= 96) return forward<float, 96>(g, st, ix, q, k, v, out, lse, s);
  return forward<float, 128>(g, st, ix, q, k, v, out, lse, s);
}

int launch_backward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                         const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv,
                         float* delta, cudaStream_t s) {
#define P3D_ARGS g, st, ix, q, k, v, out, lse, dout, dq, dk, dv, delta, s
  if (g.d <= 64) return backward<float, 64>(P3D_ARGS);
  if (g.d <= 96) return backward<float, 96>(P3D_ARGS);
  return backward<float, 128>(P3D_ARGS);
#undef P3D_ARGS
}

}  // namespace seq
}  // namespace p3d
