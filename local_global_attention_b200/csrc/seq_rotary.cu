// Rotary positions of queries and keys on a packed sequence.
//
// Pair j of a head turns by the angle f = position * theta_j:
//   (x1, x2) -> a (x1 cos f - x2 sin f, x1 sin f + x2 cos f),
// pairs (j, j + r/2) in the half layout, (2j, 2j + 1) in the interleaved one, j <
// r/2; channels from r on are copied.  The gradient is the transpose: the same
// with -f.  a is the amplitude that some long-context scalings bring.
//
// The angle is kept in turns as a 64-bit binary fraction, theta_j / (2 pi) 2^64
// rounded once on the host: position * fraction modulo 2^64 is exact, so the
// angle of position 10^6 is as good as that of position 1 (2^-64 of a turn per
// position, then 2^-32 of a turn where its upper half becomes a float for
// sincospi).  An fp32 product position * theta would be off by 0.03 rad there.
//
// Memory bound: every element is read and written once, 8 bytes or so of index
// per row.  A thread owns one group of VEC pairs of a token and walks over
// HEADS heads with the same cosines and sines in registers, so their ~40
// instructions a pair are shared; consecutive threads cover a head's channels,
// then the next heads of the same token, so a warp's accesses are whole rows.
// VEC is the widest power of two (16 bytes at most) that divides the pair
// segments, so odd rotated widths run with narrower accesses.
#include <math.h>

#include <algorithm>

#include "seq_internal.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int NT = 256;
constexpr int MAX_PAIRS = 128;  // head_dim <= 256

struct RotArgs {
  uint64_t freq[MAX_PAIRS];  // theta_j / (2 pi), 64-bit binary fraction
  float amp, sense;          // sense -1: the transpose
  int half, r, d, n;         // pairs, rotated channels, head dim, rows
  int Hq, Hk;
  int units;                 // threads of one (row, head group): pair groups, then copied groups
  int pair_units;
  int splits;                // head groups of a row
  int rows;                  // rows of a block
  int64_t sq, sk, soq, sok;  // elements between rows
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T x[VEC];
};

// HEADS: heads per thread.
template <typename T, int VEC, int LAYOUT, int HEADS>
__global__ void __launch_bounds__(NT)
    k_rotary(const __grid_constant__ RotArgs a, const int32_t* __restrict__ pos, const T* q,
             const T* k, T* qo, T* ko) {
  const int cols = a.units * a.splits;
  const int col = blockIdx.y * NT + threadIdx.x;
  // cols <= NT: rows of a block side by side; else a block covers NT columns of one row
  const int row_in = cols <= NT ? threadIdx.x / cols : 0;
  const int c = cols <= NT ? threadIdx.x % cols : col;
  const int64_t row = (int64_t)blockIdx.x * a.rows + row_in;
  if (row_in >= a.rows || c >= cols || row >= a.n) return;
  const int p = pos[row];
  if (p < 0) return;  // a row behind the last sequence: left as it was
  const int u = c % a.units, h0 = c / a.units;
  using V = Vec<T, VEC>;
  const int H = a.Hq + a.Hk;
  auto src = [&](int h) {
    return h < a.Hq ? q + row * a.sq + (int64_t)h * a.d : k + row * a.sk + (int64_t)(h - a.Hq) * a.d;
  };
  auto dst = [&](int h) {
    return h < a.Hq ? qo + row * a.soq + (int64_t)h * a.d
                    : ko + row * a.sok + (int64_t)(h - a.Hq) * a.d;
  };
  if (u >= a.pair_units) {  // channels that are not rotated
    const int ch = a.r + (u - a.pair_units) * VEC;
#pragma unroll
    for (int i = 0; i < HEADS; ++i) {
      const int h = h0 + i * a.splits;
      if (h < H && src(h) != dst(h))
        *reinterpret_cast<V*>(dst(h) + ch) = *reinterpret_cast<const V*>(src(h) + ch);
    }
    return;
  }
  constexpr int NP = LAYOUT == PACK3D_ROTARY_HALF ? VEC : VEC / 2;  // pairs of a thread
  const int j0 = u * NP;
  float cs[NP], sn[NP];
#pragma unroll
  for (int i = 0; i < NP; ++i) {
    const uint64_t turn = (uint64_t)p * a.freq[j0 + i];
    const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
    sincospif(x, &sn[i], &cs[i]);
    cs[i] *= a.amp;
    sn[i] *= a.amp * a.sense;
  }
  V lo[HEADS], hi[HEADS];
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i * a.splits;
    if (h < H) {
      if (LAYOUT == PACK3D_ROTARY_HALF) {
        lo[i] = *reinterpret_cast<const V*>(src(h) + j0);
        hi[i] = *reinterpret_cast<const V*>(src(h) + j0 + a.half);
      } else {
        lo[i] = *reinterpret_cast<const V*>(src(h) + 2 * j0);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < HEADS; ++i) {
    const int h = h0 + i * a.splits;
    if (h >= H) continue;
#pragma unroll
    for (int e = 0; e < NP; ++e) {
      T& r1 = LAYOUT == PACK3D_ROTARY_HALF ? lo[i].x[e] : lo[i].x[2 * e];
      T& r2 = LAYOUT == PACK3D_ROTARY_HALF ? hi[i].x[e] : lo[i].x[2 * e + 1];
      const float x1 = to_f32<T>(r1), x2 = to_f32<T>(r2);
      r1 = from_f32<T>(x1 * cs[e] - x2 * sn[e]);
      r2 = from_f32<T>(x1 * sn[e] + x2 * cs[e]);
    }
    if (LAYOUT == PACK3D_ROTARY_HALF) {
      *reinterpret_cast<V*>(dst(h) + j0) = lo[i];
      *reinterpret_cast<V*>(dst(h) + j0 + a.half) = hi[i];
    } else {
      *reinterpret_cast<V*>(dst(h) + 2 * j0) = lo[i];
    }
  }
}

template <typename T, int VEC, int LAYOUT>
int launch(RotArgs a, const int32_t* pos, const void* q, const void* k, void* qo, void* ko,
           cudaStream_t s) {
  const int H = a.Hq + a.Hk;
  a.pair_units = LAYOUT == PACK3D_ROTARY_HALF ? a.half / VEC : a.r / VEC;
  a.units = a.pair_units + (a.d - a.r) / VEC;
  // Four heads per thread where that still fills the GPU (148 SMs x 2048
  // threads); one head per thread for few rows, where the length of a thread's
  // chain is what a call takes.
  const bool wide = (int64_t)a.n * a.units * H >= (int64_t)148 * 2048 * 4;
  a.splits = wide ? (H + 3) / 4 : H;
  const int cols = a.units * a.splits;
  a.rows = std::max(1, NT / cols);
  const dim3 grid((unsigned)((a.n + a.rows - 1) / a.rows), (unsigned)((cols + NT - 1) / NT));
  if (wide)
    k_rotary<T, VEC, LAYOUT, 4><<<grid, NT, 0, s>>>(a, pos, (const T*)q, (const T*)k, (T*)qo,
                                                    (T*)ko);
  else
    k_rotary<T, VEC, LAYOUT, 1><<<grid, NT, 0, s>>>(a, pos, (const T*)q, (const T*)k, (T*)qo,
                                                    (T*)ko);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

template <typename T>
int launch_type(const RotArgs& a, int layout, const int32_t* pos, const void* q, const void* k,
                void* qo, void* ko, cudaStream_t s) {
  const int seg = layout == PACK3D_ROTARY_HALF ? a.half : a.r;
  constexpr int TOP = 16 / sizeof(T);
  int vec = 1;
  while (vec < TOP && seg % (2 * vec) == 0) vec *= 2;
  if (layout == PACK3D_ROTARY_HALF) {
    switch (vec) {
      case 8: return launch<T, TOP, PACK3D_ROTARY_HALF>(a, pos, q, k, qo, ko, s);
      case 4: return launch<T, 4, PACK3D_ROTARY_HALF>(a, pos, q, k, qo, ko, s);
      case 2: return launch<T, 2, PACK3D_ROTARY_HALF>(a, pos, q, k, qo, ko, s);
      default: return launch<T, 1, PACK3D_ROTARY_HALF>(a, pos, q, k, qo, ko, s);
    }
  }
  switch (vec) {
    case 8: return launch<T, TOP, PACK3D_ROTARY_INTERLEAVED>(a, pos, q, k, qo, ko, s);
    case 4: return launch<T, 4, PACK3D_ROTARY_INTERLEAVED>(a, pos, q, k, qo, ko, s);
    default: return launch<T, 2, PACK3D_ROTARY_INTERLEAVED>(a, pos, q, k, qo, ko, s);
  }
}

// theta_j of the r/2 pairs, and the default amplitude of the scaling.
int frequencies(const pack3d_rotary_params* p, double* theta, double* amp) {
  const double two_pi = 6.283185307179586476925286766559;
  const int r = p->rot_dim, half = r / 2;
  const double f = p->factor;
  double base = p->base;
  *amp = 1.0;
  if (p->scaling == PACK3D_ROTARY_BASE && r > 2) base *= pow(f, (double)r / (r - 2));
  for (int j = 0; j < half; ++j) theta[j] = pow(base, -2.0 * j / r);
  if (p->scaling == PACK3D_ROTARY_LINEAR)
    for (int j = 0; j < half; ++j) theta[j] /= f;
  if (p->scaling == PACK3D_ROTARY_BANDS)
    for (int j = 0; j < half; ++j) {
      const double turns = p->original_length * theta[j] / two_pi;
      const double m = std::min(1.0, std::max(0.0, (turns - p->low) / ((double)p->high - p->low)));
      theta[j] = m * theta[j] + (1.0 - m) * theta[j] / f;
    }
  if (p->scaling == PACK3D_ROTARY_RAMP) {
    auto pair_of = [&](double turns) {
      return r * log(p->original_length / (two_pi * turns)) / (2.0 * log(base));
    };
    const double lo = std::max(floor(pair_of(p->high)), 0.0);
    const double hi = std::min(ceil(pair_of(p->low)), (double)(r - 1));
    for (int j = 0; j < half; ++j) {
      const double m = std::min(1.0, std::max(0.0, (j - lo) / std::max(hi - lo, 0.001)));
      theta[j] = (1.0 - m) * theta[j] + m * theta[j] / f;
    }
    *amp = 0.1 * log(f) + 1.0;
  }
  for (int j = 0; j < half; ++j)
    if (!isfinite(theta[j])) return PACK3D_ERR_ARG;
  return PACK3D_OK;
}

int check_params(const pack3d_rotary_params* p) {
  if (!p) return PACK3D_ERR_ARG;
  if (p->n_tokens < 0 || p->Hq < 1 || p->Hk < 0 || p->Hq > 65536 || p->Hk > 65536)
    return PACK3D_ERR_ARG;
  if (p->n_tokens > (1 << 30)) return PACK3D_ERR_ARG;
  if (p->head_dim < 1 || p->rot_dim < 2 || (p->rot_dim & 1) || p->rot_dim > p->head_dim)
    return PACK3D_ERR_ARG;
  if (p->dtype != PACK3D_BF16 && p->dtype != PACK3D_FP32) return PACK3D_ERR_ARG;
  if (p->layout != PACK3D_ROTARY_HALF && p->layout != PACK3D_ROTARY_INTERLEAVED)
    return PACK3D_ERR_ARG;
  if (!(p->base > 0.f) || !isfinite(p->base)) return PACK3D_ERR_ARG;
  if (!isfinite(p->amplitude) || p->amplitude < 0.f) return PACK3D_ERR_ARG;
  switch (p->scaling) {
    case PACK3D_ROTARY_NONE: break;
    case PACK3D_ROTARY_RAMP:
      // its pair numbers need a base that shrinks the frequencies
      if (!(p->base > 1.f)) return PACK3D_ERR_ARG;
      // fall through: the same turn counts
    case PACK3D_ROTARY_BANDS:
      if (p->original_length < 1 || !(p->low > 0.f) || !(p->high > p->low) || !isfinite(p->high))
        return PACK3D_ERR_ARG;
      // fall through: the same factor
    case PACK3D_ROTARY_LINEAR:
    case PACK3D_ROTARY_BASE:
      if (!(p->factor >= 1.f) || !isfinite(p->factor)) return PACK3D_ERR_ARG;
      break;
    default: return PACK3D_ERR_ARG;
  }
  if (p->head_dim % 8 || p->head_dim > 256) return PACK3D_ERR_UNSUPPORTED;
  return PACK3D_OK;
}

int rotary(const pack3d_rotary_params* p, const int32_t* pos, const void* q, const void* k,
           void* qo, void* ko, float sense, cudaStream_t s) {
  int rc = check_params(p);
  if (rc) return rc;
  RotArgs a;
  double theta[MAX_PAIRS], amp;
  if ((rc = frequencies(p, theta, &amp))) return rc;
  a.half = p->rot_dim / 2;
  for (int j = 0; j < MAX_PAIRS; ++j) {
    long double f = 0.0L;
    if (j < a.half) {
      f = (long double)theta[j] / 6.283185307179586476925286766559L;
      f -= floorl(f);
    }
    // 2^64 f, rounded; a fraction that rounds up to 1 is 0 turns
    const long double x = roundl(ldexpl(f, 64));
    a.freq[j] = x >= 18446744073709551616.0L ? 0ull : (uint64_t)x;
  }
  a.amp = p->amplitude > 0.f ? p->amplitude : (float)amp;
  a.sense = sense;
  a.r = p->rot_dim;
  a.d = p->head_dim;
  a.n = p->n_tokens;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.units = a.pair_units = a.splits = a.rows = 0;
  const int64_t cq = (int64_t)p->Hq * p->head_dim, ck = (int64_t)p->Hk * p->head_dim;
  a.sq = p->stride_q ? p->stride_q : cq;
  a.sk = p->stride_k ? p->stride_k : ck;
  a.soq = p->stride_q_out ? p->stride_q_out : cq;
  a.sok = p->stride_k_out ? p->stride_k_out : ck;
  if (a.sq < cq || a.soq < cq || a.sk < ck || a.sok < ck || a.sq % 8 || a.sk % 8 || a.soq % 8 ||
      a.sok % 8)
    return PACK3D_ERR_ARG;
  if (p->n_tokens == 0) return PACK3D_OK;
  if (!pos || !q || !qo || (p->Hk && (!k || !ko))) return PACK3D_ERR_ARG;
  if (((uintptr_t)pos & 3) || (((uintptr_t)q | (uintptr_t)qo) & 15) ||
      (p->Hk && (((uintptr_t)k | (uintptr_t)ko) & 15)))
    return PACK3D_ERR_ARG;
  // In place means the same rows: another pitch would write rows not read yet.
  if ((q == qo && a.sq != a.soq) || (p->Hk && k == ko && a.sk != a.sok)) return PACK3D_ERR_ARG;
  return p->dtype == PACK3D_BF16
             ? launch_type<__nv_bfloat16>(a, p->layout, pos, q, k, qo, ko, s)
             : launch_type<float>(a, p->layout, pos, q, k, qo, ko, s);
}

}  // namespace

}  // namespace seq
}  // namespace p3d

extern "C" {

int pack3d_rotary(const pack3d_rotary_params* p, const int32_t* positions, const void* q,
                  const void* k, void* q_out, void* k_out, pack3d_stream_t stream) {
  return p3d::seq::rotary(p, positions, q, k, q_out, k_out, 1.f, (cudaStream_t)stream);
}

int pack3d_rotary_backward(const pack3d_rotary_params* p, const int32_t* positions,
                           const void* dq_out, const void* dk_out, void* dq, void* dk,
                           pack3d_stream_t stream) {
  return p3d::seq::rotary(p, positions, dq_out, dk_out, dq, dk, -1.f, (cudaStream_t)stream);
}

}  // extern "C"
