// Latent attention over a cache held in 4 bits (format: latent_fp4.cuh):
//   out[h] = sum_t softmax_t(sm_scale * q_h . c_t) c_t   over a token set S,
// S either the tokens of the row's selected blocks and its partial tail, or
// every token the row sees.
//
// One CTA takes one row and 16 heads: tiles of 32 tokens are dequantised into
// shared memory (fp32), the running maximum and sum of each head are kept in
// fp32, and each thread owns two dims of every head's output.
#include "latent_fp4.cuh"
#include "spx_device.cuh"
#include "spx_internal.h"

namespace spx {

namespace {

constexpr int kThreads = 256;
constexpr int kTile = 32;
constexpr int kHeads = 16;
constexpr int kSmem = (kTile * kLatent + kHeads * kLatent) * 4;

__global__ void __launch_bounds__(kThreads) k_attn_fp4(const AttnFp4Args a) {
  extern __shared__ float sm[];
  float* c_s = sm;                    // [kTile][512]
  float* q_s = sm + kTile * kLatent;  // [16][512]
  __shared__ float z_s[kHeads][kTile], corr_s[kHeads], m_s[kHeads], l_s[kHeads];
  __shared__ int64_t pos_s[kTile];
  const int r = blockIdx.x, h0 = blockIdx.y * kHeads, tid = threadIdx.x;
  int64_t n = a.n_vis[r];
  n = n < 0 ? 0 : (n > a.len_cap ? a.len_cap : n);
  const int64_t nblk = n / kPool;
  int64_t S = n;
  int cnt = 0;
  if (a.idx) {
    cnt = min(max(a.count[r], 0), kTopK);
    if (cnt > nblk) cnt = static_cast<int>(nblk);
    S = cnt * kPool + (n - nblk * kPool);
  }
  const int64_t base = static_cast<int64_t>(r / a.per_seq) * a.seq_tok;
  const __nv_bfloat16* q = static_cast<const __nv_bfloat16*>(a.q) +
                           (static_cast<int64_t>(r) * a.heads + h0) * kLatent;
  for (int i = tid; i < kHeads * kLatent; i += kThreads) q_s[i] = __bfloat162float(q[i]);
  if (tid < kHeads) {
    m_s[tid] = -INFINITY;
    l_s[tid] = 0.f;
  }
  float o[kHeads][2];
  for (int h = 0; h < kHeads; ++h) o[h][0] = o[h][1] = 0.f;
  for (int64_t t0 = 0; t0 < S; t0 += kTile) {
    __syncthreads();
    if (tid < kTile) {
      int64_t p = -1;
      if (t0 + tid < S) {
        p = t0 + tid;
        if (a.idx) {
          if (p < cnt * kPool) {
            const int b = a.idx[static_cast<int64_t>(r) * kTopK + (p >> 2)];
            p = b < 0 || b >= nblk ? -1 : static_cast<int64_t>(b) * kPool + (p & 3);
          } else {
            p = nblk * kPool + (p - cnt * kPool);
          }
        }
      }
      pos_s[tid] = p;
    }
    __syncthreads();
    for (int i = tid; i < kTile * (kLatent / 2); i += kThreads) {
      const int t = i / (kLatent / 2), j = i % (kLatent / 2);
      float2 f = make_float2(0.f, 0.f);
      if (pos_s[t] >= 0) {
        const int64_t at = base + pos_s[t];
        const float s = fp4_scale(a.scales[at * kFp4Groups + j / 16]);
        f = __half22float2(fp4x2_to_half2(a.codes[at * kFp4CodeBytes + j]));
        f.x *= s;
        f.y *= s;
      }
      c_s[t * kLatent + 2 * j] = f.x;
      c_s[t * kLatent + 2 * j + 1] = f.y;
    }
    __syncthreads();
    for (int i = tid; i < kHeads * kTile; i += kThreads) {
      const int h = i / kTile, t = i % kTile;
      float s = 0.f;
      for (int d = 0; d < kLatent; ++d) {
        const int k = (d + t) & (kLatent - 1);  // lanes on different banks
        s += q_s[h * kLatent + k] * c_s[t * kLatent + k];
      }
      z_s[h][t] = pos_s[t] >= 0 ? s * a.sm_scale : -INFINITY;
    }
    __syncthreads();
    if (tid < kHeads) {
      float m = m_s[tid];
      for (int t = 0; t < kTile; ++t) m = fmaxf(m, z_s[tid][t]);
      const float corr = m_s[tid] == -INFINITY ? 0.f : expf(m_s[tid] - m);
      float l = l_s[tid] * corr;
      for (int t = 0; t < kTile; ++t) {
        const float p = z_s[tid][t] == -INFINITY ? 0.f : expf(z_s[tid][t] - m);
        z_s[tid][t] = p;
        l += p;
      }
      m_s[tid] = m;
      l_s[tid] = l;
      corr_s[tid] = corr;
    }
    __syncthreads();
    for (int h = 0; h < kHeads; ++h) {
      o[h][0] *= corr_s[h];
      o[h][1] *= corr_s[h];
      for (int t = 0; t < kTile; ++t) {
        o[h][0] += z_s[h][t] * c_s[t * kLatent + 2 * tid];
        o[h][1] += z_s[h][t] * c_s[t * kLatent + 2 * tid + 1];
      }
    }
  }
  __syncthreads();
  for (int h = 0; h < kHeads; ++h) {
    const float l = l_s[h], inv = l != 0.f ? 1.f / l : 0.f;
    __nv_bfloat162* out = reinterpret_cast<__nv_bfloat162*>(
        static_cast<__nv_bfloat16*>(a.out) + (static_cast<int64_t>(r) * a.heads + h0 + h) * kLatent);
    out[tid] = __floats2bfloat162_rn(o[h][0] * inv, o[h][1] * inv);
    if (tid == 0 && a.lse)
      a.lse[static_cast<int64_t>(r) * a.heads + h0 + h] = l != 0.f ? m_s[h] + logf(l) : -INFINITY;
  }
}

}  // namespace

AttnFp4Plan plan_attn_fp4(int rows, int per_seq, int heads, bool sparse, int64_t max_len,
                          int num_sms) {
  (void)rows, (void)per_seq, (void)heads, (void)sparse, (void)max_len, (void)num_sms;
  return AttnFp4Plan{0};
}

cudaError_t launch_attn_fp4(const AttnFp4Plan& p, const AttnFp4Args& a, cudaStream_t stream) {
  (void)p;
  if (cudaError_t e = cudaFuncSetAttribute(k_attn_fp4, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                           kSmem))
    return e;
  k_attn_fp4<<<dim3(a.rows, a.heads / kHeads), kThreads, kSmem, stream>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace spx
