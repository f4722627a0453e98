// Internal declarations of the packed-sequence operators: dense attention over
// sequences of different lengths packed one behind the other, and rotary
// positions.
#pragma once

#include <atomic>

#include "pack3d_internal.cuh"

namespace p3d {
namespace seq {

constexpr int ROWS = 128;  // rows of one attention tile (the M of one tcgen05 MMA)
constexpr int PAIR = 256;  // query rows of one forward CTA: two tiles share each key/value load
constexpr int MAX_DIM = 128;
// Bits of the index's error word.
constexpr int ERR_LENGTHS_BIT = 1, ERR_TIMEOUT_BIT = 4;

// Shape derived once on the host from pack3d_seq_params and passed by value.
struct SeqGeo {
  int B, N;                // sequences, rows of the packed tensors
  int Hq, Hk, G, d;        // G = Hq / Hk query heads share a key/value head
  int causal;
  float tau;               // softmax scale
  int dtype;
  int zero;                // outputs' rows of no sequence become zero
  int n_pair, n_rows;      // entries of the 256-row and of the 128-row tile lists
};

// Elements between two tokens of each tensor.
struct Strides {
  int64_t q, k, v, out, dout, dq, dk, dv;
};

// One tile of a sequence, as the lists hold it: the sequence's first row and
// length, and the tile's first row in the sequence.  An unused entry has
// length 0.
struct Tile {
  int start, len, off, pad;
};

// (A plain load: a read-only one may be moved ahead of the wait for the kernel
// that wrote the list.)
__device__ __forceinline__ Tile load_tile_entry(const int32_t* list, int i) {
  const int4 x = reinterpret_cast<const int4*>(list)[i];
  return Tile{x.x, x.y, x.z, x.w};
}

// The index's error word and the rows that its sequences hold (cu[n_seqs]).  A block
// decides once whether the index holds an error: another block, of this launch or of
// one on another stream, may set the timeout bit between the loads of two warps, and
// warps that went on without those that left would wait on barriers and use tensor
// memory that nobody has set up.  (The barrier takes 0.1 us of a kernel's 6 to 9.)
struct State {
  int err, rows;
};
__device__ __forceinline__ State load_state(const pack3d_seq_index& ix) {
  const int2 x = *reinterpret_cast<const int2*>(ix.err);
  return State{x.x, x.y};
}

__device__ __forceinline__ bool block_failed(const State& now) {
  return __syncthreads_or(now.err) != 0;
}

// Zeros into those of the rows [first, first + n) of one head that belong to no
// sequence (`rows` of them do), by one block.  Block b of a launch over the tile
// lists takes the rows [b T, b T + T), whatever tile it has: a list has at least
// ceil(N / T) entries.
__device__ __forceinline__ bool unused_rows(const SeqGeo& g, int rows, int64_t first, int n) {
  // (unlikely: the zeroing then stands behind the kernel's way through its code)
  return __builtin_expect(g.zero && first < g.N && rows < min((int64_t)g.N, first + n), 0);
}
template <typename T>
__device__ __forceinline__ void zero_unused(const SeqGeo& g, int rows, int64_t first, int n,
                                            T* head, int64_t stride) {
  constexpr int E = 16 / sizeof(T);
  const int pieces = g.d / E;
  const int64_t from = max((int64_t)rows, first), end = min((int64_t)g.N, first + n);
  for (int i = threadIdx.x; i < (int)(end - from) * pieces; i += blockDim.x)
    *reinterpret_cast<uint4*>(head + (from + i / pieces) * stride + i % pieces * E) =
        make_uint4(0, 0, 0, 0);
}

// Let KERNEL use `bytes` of dynamic shared memory on the current device (asked for
// once per device: the runtime call costs as much host time as a tensor map).
template <auto KERNEL>
inline bool allow_smem(size_t bytes) {
  static std::atomic<uint64_t> done{0};  // a bit per device
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) !=
      cudaSuccess)
    return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

int make_geo(const pack3d_seq_params* p, SeqGeo* g);
int make_strides(const SeqGeo& g, const pack3d_seq_strides* s, Strides* out);

int launch_build_index(const SeqGeo& g, const int32_t* cu, const pack3d_seq_index* ix,
                       cudaStream_t s);
int launch_forward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                        const void* q, const void* k, const void* v, void* out, float* lse,
                        cudaStream_t s);
int launch_forward_tc(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                      const void* q, const void* k, const void* v, void* out, float* lse,
                      cudaStream_t s);
int launch_backward_simt(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                         const void* q, const void* k, const void* v, const void* out,
                         const float* lse, const void* dout, void* dq, void* dk, void* dv,
                         float* delta, cudaStream_t s);
int launch_backward_tc(const SeqGeo& g, const Strides& st, const pack3d_seq_index* ix,
                       const void* q, const void* k, const void* v, const void* out,
                       const float* lse, const void* dout, void* dq, void* dk, void* dv,
                       float* delta, float* lse2, cudaStream_t s);

}  // namespace seq
}  // namespace p3d
