// C ABI of the packed-sequence attention: argument checks, buffer sizing and
// launches.  Every entry point returns a status code and never throws; nothing
// here allocates or frees device memory.
#include <math.h>

#include "seq_internal.cuh"

namespace p3d {
namespace seq {

int make_geo(const pack3d_seq_params* p, SeqGeo* g) {
  if (!p || !g) return PACK3D_ERR_ARG;
  if (p->n_seqs < 1 || p->n_seqs > (1 << 30) || p->n_tokens < 0 || p->n_tokens > (1 << 30))
    return PACK3D_ERR_ARG;
  if (p->Hq < 1 || p->Hk < 1 || p->Hq > 65535 || p->Hq % p->Hk || p->head_dim < 1)
    return PACK3D_ERR_ARG;
  if (!isfinite(p->scale)) return PACK3D_ERR_ARG;
  const int dtype = p->dtype & ~PACK3D_ZERO_UNUSED_ROWS;
  if (dtype != PACK3D_BF16 && dtype != PACK3D_FP32) return PACK3D_ERR_ARG;
  if (p->head_dim % 8 || p->head_dim > MAX_DIM) return PACK3D_ERR_UNSUPPORTED;
  g->B = p->n_seqs;
  g->N = p->n_tokens;
  g->Hq = p->Hq;
  g->Hk = p->Hk;
  g->G = p->Hq / p->Hk;
  g->d = p->head_dim;
  g->causal = p->causal != 0;
  g->tau = p->scale > 0.f ? p->scale : 1.0f / sqrtf((float)p->head_dim);
  g->dtype = dtype;
  g->zero = dtype != p->dtype;
  // a sequence of n rows has at most floor(n / T) + 1 tiles of T rows, no more
  // than n of them not empty
  const int64_t B = p->n_seqs, N = p->n_tokens;
  const int64_t pair = N / PAIR + B, rows = N / ROWS + B;
  // launches have at most four blocks per (tile, head), and at most 2^31 - 1 blocks
  if (4 * rows * p->Hq >= (int64_t)1 << 31) return PACK3D_ERR_ARG;
  g->n_pair = (int)pair;
  g->n_rows = (int)rows;
  return PACK3D_OK;
}

int make_strides(const SeqGeo& g, const pack3d_seq_strides* s, Strides* out) {
  const int64_t cq = (int64_t)g.Hq * g.d, ck = (int64_t)g.Hk * g.d;
  const pack3d_seq_strides none = {0, 0, 0, 0, 0, 0, 0, 0};
  if (!s) s = &none;
  auto one = [](int64_t given, int64_t least, int64_t* to) {
    *to = given ? given : least;
    // below 2^37 elements a tensor map's byte stride stays below 2^40
    return *to >= least && *to % 8 == 0 && *to < (int64_t)1 << 37;
  };
  const bool ok = one(s->q, cq, &out->q) & one(s->k, ck, &out->k) & one(s->v, ck, &out->v) &
                  one(s->out, cq, &out->out) & one(s->dout, cq, &out->dout) &
                  one(s->dq, cq, &out->dq) & one(s->dk, ck, &out->dk) & one(s->dv, ck, &out->dv);
  return ok ? PACK3D_OK : PACK3D_ERR_ARG;
}

namespace {

inline size_t align256(size_t x) { return (x + 255) & ~(size_t)255; }

struct Layout {
  size_t pos, seq, pair, query, key, err, total;
};

Layout index_layout(const SeqGeo& g) {
  Layout L;
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o += align256(bytes);
    return at;
  };
  L.pos = take(sizeof(int32_t) * (size_t)g.N);
  L.seq = take(sizeof(int32_t) * (size_t)g.N);
  L.pair = take(sizeof(Tile) * (size_t)g.n_pair);
  L.query = take(sizeof(Tile) * (size_t)g.n_rows);
  L.key = take(sizeof(Tile) * (size_t)g.n_rows);
  L.err = take(2 * sizeof(int32_t));
  L.total = o;
  return L;
}

int check_index(const SeqGeo& g, const pack3d_seq_index* ix) {
  if (!ix || !ix->pos || !ix->seq || !ix->pair || !ix->query || !ix->key || !ix->err)
    return PACK3D_ERR_ARG;
  // the buffer was sized for these
  return ix->n_pair == g.n_pair && ix->n_rows == g.n_rows && ix->n_seqs == g.B &&
                 ix->n_tokens == g.N
             ? PACK3D_OK
             : PACK3D_ERR_ARG;
}

// Tensors start on 16-byte boundaries (the tensor maps and the vector accesses).
template <typename... P>
bool aligned(const P*... p) {
  return (((uintptr_t)p | ...) & 15) == 0;
}

size_t backward_bytes(const SeqGeo& g) {
  return 2 * align256(sizeof(float) * (size_t)g.Hq * g.N);
}

}  // namespace

}  // namespace seq
}  // namespace p3d

using namespace p3d;
using namespace p3d::seq;

extern "C" {

size_t pack3d_seq_index_bytes(const pack3d_seq_params* p) {
  SeqGeo g;
  if (make_geo(p, &g)) return 0;
  return index_layout(g).total;
}

int pack3d_seq_index_init(const pack3d_seq_params* p, void* buffer, size_t bytes,
                          pack3d_seq_index* out) {
  SeqGeo g;
  int rc = make_geo(p, &g);
  if (rc) return rc;
  if (!buffer || !out || ((uintptr_t)buffer & 255)) return PACK3D_ERR_ARG;
  const Layout L = index_layout(g);
  if (bytes < L.total) return PACK3D_ERR_ARG;
  char* base = (char*)buffer;
  out->pos = (int32_t*)(base + L.pos);
  out->seq = (int32_t*)(base + L.seq);
  out->pair = (int32_t*)(base + L.pair);
  out->query = (int32_t*)(base + L.query);
  out->key = (int32_t*)(base + L.key);
  out->err = (int32_t*)(base + L.err);
  out->n_pair = g.n_pair;
  out->n_rows = g.n_rows;
  out->n_seqs = g.B;
  out->n_tokens = g.N;
  return PACK3D_OK;
}

int pack3d_seq_build_index(const pack3d_seq_params* p, const int32_t* cu_seqlens,
                           pack3d_seq_index* idx, pack3d_stream_t stream) {
  SeqGeo g;
  int rc = make_geo(p, &g);
  if (rc) return rc;
  if (!cu_seqlens || ((uintptr_t)cu_seqlens & 3)) return PACK3D_ERR_ARG;
  if ((rc = check_index(g, idx))) return rc;
  return launch_build_index(g, cu_seqlens, idx, (cudaStream_t)stream);
}

int pack3d_seq_index_check(const pack3d_seq_index* idx, pack3d_stream_t stream) {
  if (!idx || !idx->err) return PACK3D_ERR_ARG;
  int32_t err[2] = {0, 0};
  if (cudaMemcpyAsync(err, idx->err, sizeof(err), cudaMemcpyDeviceToHost, (cudaStream_t)stream) !=
      cudaSuccess)
    return PACK3D_ERR_CUDA;
  if (cudaStreamSynchronize((cudaStream_t)stream) != cudaSuccess) return PACK3D_ERR_CUDA;
  if (err[0] & ERR_LENGTHS_BIT) return PACK3D_ERR_LENGTHS;
  return err[0] ? PACK3D_ERR_TIMEOUT : PACK3D_OK;
}

int pack3d_seq_forward(const pack3d_seq_params* p, const pack3d_seq_index* idx,
                       const pack3d_seq_strides* strides, const void* q, const void* k,
                       const void* v, void* out, float* lse, pack3d_stream_t stream) {
  SeqGeo g;
  Strides st;
  int rc = make_geo(p, &g);
  if (rc) return rc;
  if ((rc = check_index(g, idx)) || (rc = make_strides(g, strides, &st))) return rc;
  if (g.N == 0) return PACK3D_OK;  // every sequence is empty
  if (!q || !k || !v || !out || !lse || !aligned(q, k, v, out) || ((uintptr_t)lse & 3))
    return PACK3D_ERR_ARG;
  if (g.dtype == PACK3D_BF16)
    return launch_forward_tc(g, st, idx, q, k, v, out, lse, (cudaStream_t)stream);
  return launch_forward_simt(g, st, idx, q, k, v, out, lse, (cudaStream_t)stream);
}

size_t pack3d_seq_backward_workspace_bytes(const pack3d_seq_params* p) {
  SeqGeo g;
  if (make_geo(p, &g)) return 0;
  return backward_bytes(g);
}

int pack3d_seq_backward(const pack3d_seq_params* p, const pack3d_seq_index* idx,
                        const pack3d_seq_strides* strides, const void* q, const void* k,
                        const void* v, const void* out, const float* lse, const void* dout,
                        void* dq, void* dk, void* dv, void* workspace, size_t workspace_bytes,
                        pack3d_stream_t stream) {
  SeqGeo g;
  Strides st;
  int rc = make_geo(p, &g);
  if (rc) return rc;
  if ((rc = check_index(g, idx)) || (rc = make_strides(g, strides, &st))) return rc;
  if (g.N == 0) return PACK3D_OK;
  if (!q || !k || !v || !out || !lse || !dout || !dq || !dk || !dv || !workspace)
    return PACK3D_ERR_ARG;
  if (!aligned(q, k, v, out, dout, dq, dk, dv) || ((uintptr_t)lse & 3)) return PACK3D_ERR_ARG;
  if (((uintptr_t)workspace & 255) || workspace_bytes < backward_bytes(g)) return PACK3D_ERR_ARG;
  float* delta = (float*)workspace;
  if (g.dtype == PACK3D_FP32)
    return launch_backward_simt(g, st, idx, q, k, v, out, lse, dout, dq, dk, dv, delta,
                                (cudaStream_t)stream);
  float* lse2 = (float*)((char*)workspace + backward_bytes(g) / 2);
  return launch_backward_tc(g, st, idx, q, k, v, out, lse, dout, dq, dk, dv, delta, lse2,
                            (cudaStream_t)stream);
}

}  // extern "C"
