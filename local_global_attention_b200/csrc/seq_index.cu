// The index of a pack of sequences: per-row positions and sequence numbers, and
// the tile lists of the attention kernels, from the prefix sums of the lengths.
//
// A sequence of length n has ceil(n / T) tiles of T rows.  Tile t of sequence s
// gets the slot floor(cu[s] / T) + s + t: floor(a + b) >= floor(a) + floor(b) and
// ceil(b) <= floor(b) + 1, so the slots of two sequences never meet, and there
// are at most floor(N / T) + B of them.  Every slot finds its sequence by
// bisection of that sum, so nothing is scanned over the sequences.
//
// Each list is then ordered by cost (columns the tile has to visit), the most
// expensive first, by a counting sort over 1024 cost classes in one block, so
// that the hardware's block scheduler fills the end of a launch with small
// tiles.  Only the order inside a class varies from run to run; no result
// depends on the order of the tiles.
//
// Latency bound (a few MB at most, kept in L2): one memset and one kernel, the
// lists by three blocks and the rows by the others: 8.3 us for 64 sequences of
// 65,536 tokens, 63 us for 2,000 sequences of a million.
#include <algorithm>

#include "seq_internal.cuh"

namespace p3d {
namespace seq {

namespace {

constexpr int NT = 1024, CLASSES = 1024;

// Last s with floor(cu[s] / T) + s <= slot (T = 1: cu[s] <= slot, no + s), for
// s in [0, B).
template <bool TILES>
__device__ __forceinline__ int find_seq(const int32_t* cu, int B, int T, int64_t slot) {
  int lo = 0, hi = B - 1;
  while (lo < hi) {
    const int mid = (int)(((int64_t)lo + hi + 1) >> 1);
    const int64_t key = TILES ? (int64_t)(cu[mid] / T) + mid : (int64_t)cu[mid];
    if (key <= slot)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

enum { LIST_PAIR = 0, LIST_QUERY = 1, LIST_KEY = 2, N_LISTS = 3 };

__global__ void __launch_bounds__(NT)
    k_seq_index(SeqGeo g, const int32_t* __restrict__ cu_in, pack3d_seq_index ix) {
  __shared__ int32_t hist[CLASSES];
  __shared__ int32_t part[32];
  __shared__ int32_t bad;
  const int tid = threadIdx.x;
  if (blockIdx.x >= N_LISTS) {
    // one row per thread: position in its sequence and the sequence's number,
    // -1 behind the last one
    const int64_t i = (int64_t)(blockIdx.x - N_LISTS) * NT + tid;
    if (i >= g.N) return;
    // the last s with cu[s] <= i is not empty; rows at or behind cu[B] have none
    int s = -1, pos = -1;
    if (i < cu_in[g.B] && i >= cu_in[0]) {
      s = find_seq<false>(cu_in, g.B, 1, i);
      pos = (int)(i - cu_in[s]);
    }
    ix.pos[i] = pos;
    ix.seq[i] = s;
    return;
  }
  const int list = blockIdx.x;
  // the prefix sums start at 0, never fall and end inside the tensors
  if (tid == 0) bad = cu_in[0] != 0 || cu_in[g.B] > g.N;
  __syncthreads();
  for (int s = tid; s < g.B; s += NT)
    if (cu_in[s + 1] < cu_in[s] || cu_in[s] < 0 || cu_in[s] > g.N) bad = 1;
  for (int i = tid; i < CLASSES; i += NT) hist[i] = 0;
  __syncthreads();
  Tile* out = reinterpret_cast<Tile*>(list == LIST_PAIR ? ix.pair : list == LIST_QUERY ? ix.query
                                                                                      : ix.key);
  const int slots = list == LIST_PAIR ? g.n_pair : g.n_rows;
  if (bad) {
    if (tid == 0) atomicOr(&ix.err[0], ERR_LENGTHS_BIT);
    for (int i = tid; i < slots; i += NT) out[i] = Tile{0, 0, 0, 0};
    return;
  }
  if (list == 0 && tid == 0) ix.err[1] = cu_in[g.B];
  const int T = list == LIST_PAIR ? PAIR : ROWS;
  int shift = 0;  // cost classes of 2^shift tiles of 128 columns
  while (((g.N / ROWS + 1) >> shift) >= CLASSES) ++shift;
  // the tile of a slot, and its cost class (0: the most expensive)
  auto tile_at = [&](int slot, Tile& t) -> int {
    const int s = find_seq<true>(cu_in, g.B, T, slot);
    const int c0 = cu_in[s];
    const int64_t off = ((int64_t)slot - (c0 / T + s)) * T;
    t = Tile{c0, cu_in[s + 1] - c0, (int)off, 0};
    if (off >= t.len) return -1;
    const int64_t cols = !g.causal            ? t.len
                         : list == LIST_KEY ? t.len - t.off
                                            : min((int64_t)t.len, (int64_t)t.off + T);
    return CLASSES - 1 - (int)((cols / ROWS) >> shift);
  };
  for (int i = tid; i < slots; i += NT) {
    Tile t;
    const int c = tile_at(i, t);
    if (c >= 0) atomicAdd(&hist[c], 1);
  }
  __syncthreads();
  // exclusive scan of the 1024 classes, one per thread
  {
    const int lane = tid & 31, warp = tid >> 5;
    const int mine = hist[tid];
    int x = mine;
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) part[warp] = x;
    __syncthreads();
    if (warp == 0) {
      int p = part[lane];
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += y;
      }
      part[lane] = p;
    }
    __syncthreads();
    hist[tid] = x - mine + (warp ? part[warp - 1] : 0);
  }
  const int used = part[31];
  __syncthreads();
  for (int i = tid; i < slots; i += NT) {
    Tile t;
    const int c = tile_at(i, t);
    if (c >= 0) out[atomicAdd(&hist[c], 1)] = t;
  }
  for (int i = used + tid; i < slots; i += NT) out[i] = Tile{0, 0, 0, 0};
}

}  // namespace

int launch_build_index(const SeqGeo& g, const int32_t* cu, const pack3d_seq_index* ix,
                       cudaStream_t s) {
  if (cudaMemsetAsync(ix->err, 0, 2 * sizeof(int32_t), s) != cudaSuccess) return PACK3D_ERR_CUDA;
  const int blocks = N_LISTS + (g.N + NT - 1) / NT;
  k_seq_index<<<blocks, NT, 0, s>>>(g, cu, *ix);
  count_launches(1);
  return cuda_status(cudaGetLastError());
}

}  // namespace seq
}  // namespace p3d
