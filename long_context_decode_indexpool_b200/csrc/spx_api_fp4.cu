// C ABI of the 4-bit latent cache: host-side validation and launches (rules
// as in spx_api.cu: every check runs before the first launch of a call).
#include "spx.h"
#include "spx_internal.h"

using namespace spx;

namespace {

inline bool al(const void* p, unsigned n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

spx_status cuda_status(cudaError_t e) { return e == cudaSuccess ? SPX_OK : SPX_ERR_CUDA; }

// Token positions fit 31 bits and sequences 16, so that byte offsets into a
// cache stay far below 2^63.
constexpr int64_t kMaxTok = kFp4MaxTok;
constexpr int32_t kMaxSeqs = 65535;
constexpr int64_t kMaxRows = int64_t(1) << 33;  // rows of one write or read: 8 TiB

// The checks the two attention calls share, after the shape of their rows.
spx_status attn_fp4(const spx_dims* d, int32_t rows, int32_t per_seq, const void* q,
                    const void* codes, const void* scales, int64_t seq_tok, int64_t cap_tok,
                    bool sparse, const int32_t* idx, const int32_t* count, const int64_t* n_vis,
                    int64_t max_len, void* out, float* lse, void* ws, size_t ws_bytes,
                    spx_stream stream) {
  if (!q || !codes || !scales || !n_vis || !out || (sparse && (!idx || !count)))
    return SPX_ERR_INVALID_ARG;
  if (!al(q, 16) || !al(codes, 16) || !al(scales, 16) || !al(out, 16) || !al(n_vis, 8) ||
      (lse && !al(lse, 4)) || (sparse && (!al(idx, 4) || !al(count, 4))))
    return SPX_ERR_INVALID_ARG;
  // the plan's bound on the lengths is the one that the kernel clamps them to
  const int64_t len_cap = max_len < cap_tok ? max_len : cap_tok;
  const AttnFp4Plan p = plan_attn_fp4(rows, per_seq, d->heads, sparse, len_cap, device_sm_count());
  if (p.tiles > 0x7fffffff) return SPX_ERR_UNSUPPORTED;
  if (p.ws_bytes > 0 && (!ws || ws_bytes < p.ws_bytes || !al(ws, 16))) return SPX_ERR_WORKSPACE;
  AttnFp4Args a{};
  a.per_seq = per_seq;
  a.heads = d->heads;
  a.q = q;
  a.codes = static_cast<const uint8_t*>(codes);
  a.scales = static_cast<const uint8_t*>(scales);
  a.seq_tok = seq_tok;
  a.len_cap = len_cap;
  a.idx = sparse ? idx : nullptr;
  a.count = sparse ? count : nullptr;
  a.n_vis = n_vis;
  a.sm_scale = d->sm_scale;
  a.out = out;
  a.lse = lse;
  a.ws = ws;
  return cuda_status(launch_attn_fp4(p, a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // namespace

extern "C" {

spx_status spx_latent_append_fp4(int32_t B, const void* latent, int64_t n_new, const int32_t* n_add,
                                 void* codes, void* scales, int64_t cap_tok, const int64_t* len_dev,
                                 int64_t max_len, void* stored, spx_stream stream) {
  if (B < 1 || B > kMaxSeqs || n_new < 0 || n_new > kMaxTok || cap_tok < 1 || cap_tok > kMaxTok || max_len < 0 ||
      max_len > cap_tok)
    return SPX_ERR_SHAPE;
  if (n_new == 0) return SPX_OK;
  if (B * n_new > kMaxRows) return SPX_ERR_SHAPE;
  if (!latent || !codes || !scales || !len_dev) return SPX_ERR_INVALID_ARG;
  if (!al(latent, 16) || !al(codes, 16) || !al(scales, 16) || !al(len_dev, 8) ||
      (n_add && !al(n_add, 4)) || (stored && !al(stored, 16)))
    return SPX_ERR_INVALID_ARG;
  return cuda_status(launch_latent_append_fp4(
      B, latent, n_new, n_add, static_cast<uint8_t*>(codes), static_cast<uint8_t*>(scales), cap_tok,
      len_dev, max_len, stored, reinterpret_cast<cudaStream_t>(stream)));
}

spx_status spx_latent_read_fp4(int32_t B, const void* codes, const void* scales, int64_t cap_tok,
                               const int64_t* pos, int64_t m, const int64_t* n_vis, void* out,
                               spx_stream stream) {
  if (B < 1 || B > kMaxSeqs || m < 0 || m > kMaxTok || cap_tok < 1 || cap_tok > kMaxTok) return SPX_ERR_SHAPE;
  if (m == 0) return SPX_OK;
  if (B * m > kMaxRows) return SPX_ERR_SHAPE;
  if (!codes || !scales || !n_vis || !out) return SPX_ERR_INVALID_ARG;
  if (!al(codes, 16) || !al(scales, 16) || !al(n_vis, 8) || !al(out, 16) || (pos && !al(pos, 8)))
    return SPX_ERR_INVALID_ARG;
  return cuda_status(launch_latent_read_fp4(
      B, static_cast<const uint8_t*>(codes), static_cast<const uint8_t*>(scales), cap_tok, pos, m,
      n_vis, out, reinterpret_cast<cudaStream_t>(stream)));
}

spx_status spx_attn_fp4_workspace_size(const spx_dims* d, int32_t rows, int64_t max_len,
                                       size_t* bytes) {
  spx_status st = check_dims(d);
  if (st != SPX_OK) return st;
  if (!bytes) return SPX_ERR_INVALID_ARG;
  if (rows < 1 || rows > 65535 || max_len < 0) return SPX_ERR_SHAPE;
  *bytes = plan_attn_fp4(rows, 1, d->heads, true, max_len, device_sm_count()).ws_bytes;
  return SPX_OK;
}

spx_status spx_sparse_mla_attn_fp4(const spx_dims* d, int32_t rows, const void* q,
                                   const void* codes, const void* scales, int64_t seq_stride,
                                   int64_t cap_tok, const int32_t* idx, const int32_t* count,
                                   const int64_t* n_vis, int64_t max_len, void* out, float* lse,
                                   void* ws, size_t ws_bytes, spx_stream stream) {
  spx_status st = check_dims(d);
  if (st != SPX_OK) return st;
  if (rows < 1 || rows > 65535 || max_len < 0 || cap_tok < 1 || cap_tok > kMaxTok ||
      seq_stride < 0)
    return SPX_ERR_SHAPE;
  if (seq_stride != 0 && (seq_stride / kLatent < cap_tok || seq_stride % kLatent != 0))
    return SPX_ERR_SHAPE;
  return attn_fp4(d, rows, 1, q, codes, scales, seq_stride / kLatent, cap_tok, true, idx, count,
                  n_vis, max_len, out, lse, ws, ws_bytes, stream);
}

spx_status spx_latent_attn_fp4_workspace_size(const spx_dims* d, int32_t rows,
                                              int32_t rows_per_seq, int64_t max_len,
                                              size_t* bytes) {
  spx_status st = check_dims(d);
  if (st != SPX_OK) return st;
  if (!bytes) return SPX_ERR_INVALID_ARG;
  if (rows < 1 || rows > 65535 || max_len < 0) return SPX_ERR_SHAPE;
  if (rows_per_seq < 1 || rows % rows_per_seq != 0) return SPX_ERR_SHAPE;
  *bytes = plan_attn_fp4(rows, rows_per_seq, d->heads, false, max_len, device_sm_count()).ws_bytes;
  return SPX_OK;
}

spx_status spx_latent_attn_fp4(const spx_dims* d, int32_t rows, int32_t rows_per_seq,
                               const void* q, const void* codes, const void* scales,
                               int64_t cap_tok, const int64_t* n_vis, int64_t max_len, void* out,
                               float* lse, void* ws, size_t ws_bytes, spx_stream stream) {
  spx_status st = check_dims(d);
  if (st != SPX_OK) return st;
  if (rows < 1 || rows > 65535 || max_len < 0 || cap_tok < 1 || cap_tok > kMaxTok)
    return SPX_ERR_SHAPE;
  if (rows_per_seq < 1 || rows % rows_per_seq != 0) return SPX_ERR_SHAPE;
  return attn_fp4(d, rows, rows_per_seq, q, codes, scales, cap_tok, cap_tok, false, nullptr,
                  nullptr, n_vis, max_len, out, lse, ws, ws_bytes, stream);
}

}  // extern "C"
