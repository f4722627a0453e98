// Pieces shared by the tensor-core kernels of packed-sequence attention: the
// 128-byte-swizzled operand tiles, their descriptors and tensor maps, and the
// converged-warp forms of waits.
//
// An operand tile is ROWS rows of one head, in segments of 64 channels: segment
// s is [ROWS][128 bytes] with the 128-byte swizzle, the form in which a TMA box
// of {64 channels, 1 head, ROWS rows} lands and which the MMAs read K-major
// (channels contracted) or MN-major (rows contracted).  Channels from head_dim
// on and rows behind the tensor are filled with zeros by the copy.
#pragma once

#include "seq_internal.cuh"
#include "tc_attn_common.cuh"

namespace p3d {
namespace seq {

using namespace tc;

constexpr uint32_t SEG = ROWS * 128;  // bytes of one 64-channel segment of a tile
constexpr uint32_t WAIT_LIMIT = 1u << 20;
constexpr float LOG2E = 1.4426950408889634f;
constexpr float LN2 = 0.6931471805599453f;

// Matrix descriptor with the 128-byte swizzle (layout type 2): 8 rows of 128
// bytes per swizzle atom, so the stride byte offset is 1024; the leading byte
// offset is the distance of two 64-channel segments for an MN-major operand
// (not read for a K-major one).
__device__ __forceinline__ uint64_t sdesc_sw128(uint32_t saddr) {
  uint64_t d = 0;
  d |= (uint64_t)((saddr >> 4) & 0x3FFFu);
  d |= (uint64_t)(SEG >> 4) << 16;
  d |= (uint64_t)(1024u >> 4) << 32;
  d |= (uint64_t)1 << 46;
  d |= (uint64_t)2 << 61;
  return d;
}

// Descriptor offset (16-byte units) of channel step st (16 channels) of a
// K-major tile, and of row step st (16 rows) of an MN-major one.
__host__ __device__ constexpr uint32_t k_step(int st) {
  return ((st >> 2) * SEG + (st & 3) * 32) >> 4;
}
__host__ __device__ constexpr uint32_t row_step(int st) { return (uint32_t)(st * 16 * 128) >> 4; }

// Move registers between warpgroups (all four warps of one execute the same
// call): the kernel is launched with 168 registers per thread, 384 threads; two
// warpgroups take ARITH_REGS each, the third keeps OTHER_REGS.
constexpr int ARITH_REGS = 208, OTHER_REGS = 80;
static_assert(2 * ARITH_REGS + OTHER_REGS <= 3 * 168, "registers of the launch");
template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}

// Launches that overlap the end of the kernel before them in the stream: the next
// kernel's blocks may be placed once every block of this one has started and SMs
// come free; the first thing they do is to wait until this one is complete and
// its writes are visible, so an order of launches means what it always does.
// What it saves is the launch latency between the kernels of one call (and of
// calls in a row).  Global memory that an earlier kernel wrote is read through
// plain pointers in these kernels (no __restrict__, no read-only loads): the
// compiler may move read-only loads ahead of the wait.
__device__ __forceinline__ void overlapped_start() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");
}
template <typename... P, typename... A>
inline int launch_overlapped(void (*kernel)(P...), unsigned blocks, unsigned threads, size_t smem,
                             cudaStream_t s, A... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(blocks);
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cuda_status(cudaLaunchKernelEx(&cfg, kernel, P(args)...));
}

// A wait of a whole converged warp: true once the phase is complete, false when
// some role of the CTA has given up or the poll limit is reached.  The vote keeps
// the branch uniform: a wait on a completed phase takes 48 cycles, against 155
// with a loop of its own per lane and one vote behind it.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity,
                                          volatile int32_t* abort) {
  if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
  for (uint32_t i = 0; i < WAIT_LIMIT; ++i) {
    if (__all_sync(0xffffffffu, mbar_try_wait(bar, parity))) return true;
    if (__any_sync(0xffffffffu, *abort)) return false;
  }
  *abort = 1;
  return false;
}

// Maximum of three values in one instruction.
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Rows [from, ROWS) of a tile set to zero by one warp, visible to the tensor
// core once the warp has arrived on a barrier: what stands behind the last row
// of a sequence (the next sequence, or anything) must not enter a product that
// contracts rows, where even a weight of zero passes a NaN on.
template <int NSEG>
__device__ __forceinline__ void zero_rows(uint8_t* tile, int from, int lane) {
  for (int i = from * 8 + lane; i < ROWS * 8; i += 32)
#pragma unroll
    for (int s = 0; s < NSEG; ++s)
      *reinterpret_cast<uint4*>(tile + s * SEG + i * 16) = make_uint4(0, 0, 0, 0);
  fence_proxy_async_smem();
  __syncwarp();
}

// One box of a 3-D tensor map from shared memory to global memory (what lies
// outside the tensor is not written), and the wait until this thread's boxes are
// written.
__device__ __forceinline__ void tma_store_3d(const void* map, const void* src, int c0, int c1,
                                             int c2) {
  asm volatile(
      "cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%1, %2, %3}], [%4];" ::"l"(
          reinterpret_cast<uint64_t>(map)),
      "r"(c0), "r"(c1), "r"(c2), "r"(smem_u32(src))
      : "memory");
}
__device__ __forceinline__ void tma_store_wait() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}

// 32 channels [c0, c0 + 32) of a warp's 32 accumulator rows (lane = row), scaled
// and rounded to bf16, into rows `stride` elements apart from dst on: rows below
// `live`, channels below d.  Four lanes first exchange their 16-byte pieces, so
// that they store 64 contiguous bytes of one row: an access of a warp then meets 8
// lines instead of 32 (an epilogue of 128 channels took 2,600 cycles with a row
// per lane).
__device__ __forceinline__ void store_rows32(const uint32_t (&o)[32], float f, __nv_bfloat16* dst,
                                             int64_t stride, int live, int c0, int d, int lane) {
  uint32_t w[4][4];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      const float2 y = f2_mul(make_float2(__uint_as_float(o[8 * c + 2 * x]),
                                          __uint_as_float(o[8 * c + 2 * x + 1])),
                              make_float2(f, f));
      w[c][x] = pack_bf16x2(y.x, y.y);
    }
  // transpose (lane of the four) x (piece), one bit at a time
#pragma unroll
  for (int bit = 1; bit <= 2; bit *= 2) {
    const bool upper = lane & bit;
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (c & bit) continue;
#pragma unroll
      for (int x = 0; x < 4; ++x) {
        const uint32_t got =
            __shfl_xor_sync(0xffffffffu, upper ? w[c][x] : w[c | bit][x], bit);
        if (upper)
          w[c][x] = got;
        else
          w[c | bit][x] = got;
      }
    }
  }
  const int ch = c0 + 8 * (lane & 3);
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    const int row = (lane & ~3) + s;
    if (row < live && ch < d)
      *reinterpret_cast<uint4*>(dst + row * stride + ch) =
          make_uint4(w[s][0], w[s][1], w[s][2], w[s][3]);
  }
}

// Tensor map of a packed tensor [N][H][d] (tokens `stride` elements apart):
// boxes of {64 channels, 1 head, `rows` rows}.
inline bool encode_rows(CUtensorMap* m, const void* base, int d, int H, int N, int64_t stride,
                        int rows) {
  tca::EncodeTiled fn = tca::encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)N};
  const cuuint64_t strides[2] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[3] = {64, 1, (cuuint32_t)rows}, step[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(base), dims, strides, box,
            step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) ==
         CUDA_SUCCESS;
}

// One tile (all segments) of a head by TMA; returns nothing, signals `bar`.
template <int NSEG>
__device__ __forceinline__ void load_tile_tma(uint8_t* dst, const CUtensorMap* map, int head,
                                              int row, uint64_t* bar) {
#pragma unroll
  for (int s = 0; s < NSEG; ++s) tma_load_3d(dst + s * SEG, map, 64 * s, head, row, bar);
}

}  // namespace seq
}  // namespace p3d
