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
// Memory bound: every element is read and written once, 4 bytes of index per
// row.  A thread keeps one place of a row (a head's VEC pairs, or VEC channels
// that are only copied) and walks over rows; per group of rows a block first
// issues its loads, then computes the rows' cosines and sines once, one pair per
// thread, into shared memory, where all heads of a row find them, then turns and
// stores.  Consecutive threads cover a head, then the next heads, so a warp's
// accesses are whole rows.  VEC is the widest power of two (16 bytes at most)
// that divides the pair segments, so odd rotated widths run with narrower
// accesses.  Measured at 65,536 rows x 16 heads x 96 (402 MB): 78 us, 5.2 TB/s,
// 0.79 of the copy bandwidth; with cosines per thread, shared by four heads
// only, and loads after them 126 us.
#include <math.h>

#include <algorithm>

#include "seq_internal.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int NT = 256;
constexpr int MAX_PAIRS = 128;   // head_dim <= 256
constexpr int MAX_HEADS = 65536; // of q and k together
constexpr int CS_ENTRIES = 2048; // (cos, sin) pairs of a group of rows in shared memory

struct RotArgs {
  uint64_t freq[MAX_PAIRS];  // theta_j / (2 pi), 64-bit binary fraction
  float amp, sense;          // sense -1: the transpose
  int zero;                  // rows of a negative position become zero
  int half, r, d, n;         // pairs, rotated channels, head dim, rows
  int Hq, Hk;
  int units;                 // threads of a head: VEC pairs or channels turned, then copied
  int pair_units;
  int cols, slots;           // threads of a row; rows side by side in a block
  int64_t sq, sk, soq, sok;  // elements between rows
};

template <typename T, int VEC>
struct alignas(sizeof(T) * VEC) Vec {
  T x[VEC];
};

// VEC values moved by one access of their whole width.
template <int BYTES>
struct Word;
template <>
struct Word<16> {
  using type = uint4;
};
template <>
struct Word<8> {
  using type = uint2;
};
template <>
struct Word<4> {
  using type = uint32_t;
};
template <>
struct Word<2> {
  using type = uint16_t;
};
template <typename T, int VEC>
__device__ __forceinline__ void load(Vec<T, VEC>& v, const T* src) {
  using W = typename Word<sizeof(T) * VEC>::type;
  *reinterpret_cast<W*>(&v) = *reinterpret_cast<const W*>(src);
}
template <typename T, int VEC>
__device__ __forceinline__ void store(T* dst, const Vec<T, VEC>& v) {
  using W = typename Word<sizeof(T) * VEC>::type;
  *reinterpret_cast<W*>(dst) = *reinterpret_cast<const W*>(&v);
}

// ROWS_T: rows of a thread per group.
template <typename T, int VEC, int LAYOUT, int ROWS_T>
__global__ void __launch_bounds__(NT)
    k_rotary(const __grid_constant__ RotArgs a, const int32_t* __restrict__ pos, const T* q,
             const T* k, T* qo, T* ko) {
  constexpr bool HALF = LAYOUT == PACK3D_ROTARY_HALF;
  constexpr int NP = HALF ? VEC : VEC / 2;  // pairs of a thread
  using V = Vec<T, VEC>;
  extern __shared__ float2 cs_all[];  // two of [rows of a group][pairs]
  __shared__ uint64_t freq[MAX_PAIRS];
  for (int j = threadIdx.x; j < a.half; j += blockDim.x) freq[j] = a.freq[j];
  // this thread's row slot, head and channels
  const int slot = a.slots == 1 ? 0 : threadIdx.x / a.cols;
  const int col = blockIdx.y * NT + threadIdx.x - slot * a.cols;
  const int h = col / a.units, u = col - h * a.units;
  const bool turned = u < a.pair_units;
  const int ch = turned ? u * VEC : a.r + (u - a.pair_units) * VEC;
  const bool is_k = h >= a.Hq;
  const int64_t si = is_k ? a.sk : a.sq, so = is_k ? a.sok : a.soq;
  const T* src = is_k ? k + (int64_t)(h - a.Hq) * a.d + ch : q + (int64_t)h * a.d + ch;
  T* dst = is_k ? ko + (int64_t)(h - a.Hq) * a.d + ch : qo + (int64_t)h * a.d + ch;
  // in place, the copied channels are there already
  const bool mine = col < a.cols && (turned || src != dst || a.zero);
  const int entry = HALF ? ch : ch / 2;
  const int rows = a.slots * ROWS_T;  // of a group
  int side = 0;
  __syncthreads();
  for (int64_t row0 = (int64_t)blockIdx.x * rows; row0 < a.n;
       row0 += (int64_t)gridDim.x * rows, side ^= 1) {
    const int live = (int)min((int64_t)rows, a.n - row0);
    V lo[ROWS_T], hi[HALF ? ROWS_T : 1];
    // loads that wait for nothing (rows that will be left alone are read as well)
#pragma unroll
    for (int i = 0; i < ROWS_T; ++i) {
      const int r = slot + i * a.slots;
      if (mine && r < live) {
        const T* p = src + (row0 + r) * si;
        load(lo[i], p);
        if (HALF && turned) load(hi[HALF ? i : 0], p + a.half);
      }
    }
    // (two halves in turn: the barrier below also ends the reads of two groups ago)
    float2* cs = cs_all + side * rows * a.half;
    for (int e = threadIdx.x; e < live * a.half; e += blockDim.x) {
      const int r = e / a.half, j = e - r * a.half;
      const uint64_t turn = (uint64_t)(int64_t)pos[row0 + r] * freq[j];
      const float x = (float)(int32_t)(turn >> 32) * 4.656612873077393e-10f;  // 2^-31: half turns
      float sn, c;
      sincospif(x, &sn, &c);
      cs[e] = make_float2(c * a.amp, sn * a.amp * a.sense);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < ROWS_T; ++i) {
      const int r = slot + i * a.slots;
      if (!mine || r >= live) continue;
      T* p = dst + (row0 + r) * so;
      if (pos[row0 + r] < 0) {  // behind the last sequence
        if (a.zero) {
          store(p, V{});
          if (HALF && turned) store(p + a.half, V{});
        }
        continue;
      }
      if (turned) {
        const float2* c = cs + r * a.half + entry;
#pragma unroll
        for (int e = 0; e < NP; ++e) {
          T& r1 = HALF ? lo[i].x[e] : lo[i].x[2 * e];
          T& r2 = HALF ? hi[HALF ? i : 0].x[e] : lo[i].x[2 * e + 1];
          const float x1 = to_f32<T>(r1), x2 = to_f32<T>(r2);
          r1 = from_f32<T>(x1 * c[e].x - x2 * c[e].y);
          r2 = from_f32<T>(x1 * c[e].y + x2 * c[e].x);
        }
        if (HALF) store(p + a.half, hi[HALF ? i : 0]);
      }
      store(p, lo[i]);
    }
  }
}

template <typename T, int VEC, int LAYOUT>
int launch(RotArgs a, const int32_t* pos, const void* q, const void* k, void* qo, void* ko,
           cudaStream_t s) {
  a.pair_units = LAYOUT == PACK3D_ROTARY_HALF ? a.half / VEC : a.r / VEC;
  a.units = a.pair_units + (a.d - a.r) / VEC;
  a.cols = (a.Hq + a.Hk) * a.units;
  a.slots = std::max(1, NT / a.cols);
  // Four vectors in flight per thread (two rows in the half layout, whose pairs are
  // two vectors: 36 against 39 us with four rows at 16,411 x 20 x 128; four rows
  // interleaved: 75 against 90 us with two at 65,536 x 16 x 96) where that still
  // gives every SM its 2,048 threads; one row where there are few, and the length
  // of a thread's chain is what a call takes.
  constexpr int WIDE = LAYOUT == PACK3D_ROTARY_HALF ? 2 : 4;
  const bool wide = (int64_t)a.n * a.cols >= (int64_t)148 * 2048 * WIDE;
  const int rows = wide ? WIDE : 1;
  // the cosines of two groups fit into the shared memory every block may have
  a.slots = std::min(a.slots, std::max(1, CS_ENTRIES / (rows * a.half)));
  const int threads = a.cols < NT ? a.slots * a.cols : NT;
  const int64_t parts = (a.cols + NT - 1) / NT;
  // Blocks that stay (sixteen per SM) and walk over groups of rows: a thread's own
  // frequency comes from the kernel's parameters, which a warp reads one address
  // at a time, so it is copied to shared memory once per block.
  const int64_t groups = ((int64_t)a.n + rows * a.slots - 1) / (rows * a.slots);
  const dim3 grid((unsigned)std::min<int64_t>(groups, std::max<int64_t>(1, 148 * 16 / parts)),
                  (unsigned)parts);
  const size_t bytes = 2 * sizeof(float2) * rows * a.slots * a.half;
  if (wide)
    k_rotary<T, VEC, LAYOUT, WIDE><<<grid, threads, bytes, s>>>(
        a, pos, (const T*)q, (const T*)k, (T*)qo, (T*)ko);
  else
    k_rotary<T, VEC, LAYOUT, 1><<<grid, threads, bytes, s>>>(a, pos, (const T*)q, (const T*)k,
                                                             (T*)qo, (T*)ko);
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

// theta_j of the r/2 pairs, and the default amplitude of the scaling.  The powers
// base^(-2j/r) are products of one factor in 64-bit mantissas (128 products are
// off by 2^-57 at most), which takes a call 1 us less of host time than as many
// powers.  With a base below 1 the frequencies grow, and a relative error of one is as
// many times more of a turn: there every power is taken by itself (2^-61 relative),
// and pairs of MAX_TURNS turns per position or more are refused, whose fraction would
// keep too few bits (below it the angle of position 2^31 is off by 2^-26 of a turn at
// most).
constexpr long double MAX_TURNS = 16.0L;
int frequencies(const pack3d_rotary_params* p, long double* theta, double* amp) {
  const long double two_pi = 6.283185307179586476925286766559L;
  const int r = p->rot_dim, half = r / 2;
  const long double f = p->factor, L = p->original_length;
  long double base = p->base;
  *amp = 1.0;
  if (p->scaling == PACK3D_ROTARY_BASE && r > 2) base *= powl(f, (long double)r / (r - 2));
  const long double step = powl(base, -2.0L / r);
  theta[0] = 1.0L;
  for (int j = 1; j < half; ++j)
    theta[j] = base < 1.0L ? powl(base, -2.0L * j / r) : theta[j - 1] * step;
  if (p->scaling == PACK3D_ROTARY_LINEAR)
    for (int j = 0; j < half; ++j) theta[j] /= f;
  if (p->scaling == PACK3D_ROTARY_BANDS)
    for (int j = 0; j < half; ++j) {
      const long double turns = L * theta[j] / two_pi;
      const long double m =
          std::min(1.0L, std::max(0.0L, (turns - p->low) / ((long double)p->high - p->low)));
      theta[j] = m * theta[j] + (1.0L - m) * theta[j] / f;
    }
  if (p->scaling == PACK3D_ROTARY_RAMP) {
    auto pair_of = [&](double turns) {
      return r * log(p->original_length / ((double)two_pi * turns)) / (2.0 * log(p->base));
    };
    const double lo = std::max(floor(pair_of(p->high)), 0.0);
    const double hi = std::min(ceil(pair_of(p->low)), (double)(r - 1));
    for (int j = 0; j < half; ++j) {
      const double m = std::min(1.0, std::max(0.0, (j - lo) / std::max(hi - lo, 0.001)));
      theta[j] = (1.0L - m) * theta[j] + m * theta[j] / f;
    }
    *amp = 0.1 * log((double)f) + 1.0;
  }
  // (the last pair is the fastest where the base is below 1, and at most 1 elsewhere)
  return theta[half - 1] < MAX_TURNS * two_pi ? PACK3D_OK : PACK3D_ERR_ARG;
}

int check_params(const pack3d_rotary_params* p) {
  if (!p) return PACK3D_ERR_ARG;
  if (p->n_tokens < 0 || p->Hq < 1 || p->Hk < 0 || (int64_t)p->Hq + p->Hk > MAX_HEADS)
    return PACK3D_ERR_ARG;
  if (p->n_tokens > (1 << 30)) return PACK3D_ERR_ARG;
  if (p->head_dim < 1 || p->rot_dim < 2 || (p->rot_dim & 1) || p->rot_dim > p->head_dim)
    return PACK3D_ERR_ARG;
  const int dtype = p->dtype & ~PACK3D_ZERO_UNUSED_ROWS;
  if (dtype != PACK3D_BF16 && dtype != PACK3D_FP32) return PACK3D_ERR_ARG;
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
  long double theta[MAX_PAIRS];
  double amp;
  if ((rc = frequencies(p, theta, &amp))) return rc;
  a.half = p->rot_dim / 2;
  for (int j = 0; j < a.half; ++j) {
    // the turn's fraction as 64 bits; one that rounds up to a whole turn is 0
    long double f = theta[j] * (1.0L / 6.283185307179586476925286766559L);
    if (f >= 1.0L) f -= floorl(f);
    const long double x = f * 18446744073709551616.0L + 0.5L;
    a.freq[j] = x >= 18446744073709551616.0L ? 0ull : (uint64_t)x;
  }
  a.amp = p->amplitude > 0.f ? p->amplitude : (float)amp;
  a.sense = sense;
  a.zero = (p->dtype & PACK3D_ZERO_UNUSED_ROWS) != 0;
  a.r = p->rot_dim;
  a.d = p->head_dim;
  a.n = p->n_tokens;
  a.Hq = p->Hq;
  a.Hk = p->Hk;
  a.units = a.pair_units = a.cols = a.slots = 0;
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
  return (p->dtype & ~PACK3D_ZERO_UNUSED_ROWS) == PACK3D_BF16
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
