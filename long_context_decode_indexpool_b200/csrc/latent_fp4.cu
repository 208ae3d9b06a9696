// 4-bit latent cache: quantising write and read back (format: latent_fp4.cuh).
//
// [W1] "GLM-5.3-Flash: 하이브리드 희소·선형 어텐션과 IndexPool·EPD로 1M 컨텍스트를
// 오픈 소스로 서빙하는 방법", section "양자화: W8A8와 혼합 캐시", keeps cache
// entries in 8 bits; the 4-bit form is this library's own step further, 272
// bytes a token instead of 1024 (bf16) or 516 (FP8).
//
// Both kernels give a row to a warp; lane l holds dims 8l..8l+7 and
// 256+8l..256+8l+7, so that every 16-byte load and 4-byte code store of the
// warp is contiguous, and a group of 32 dims is four lanes.
#include "latent_fp4.cuh"
#include "spx_device.cuh"
#include "spx_internal.h"

namespace spx {

namespace {

constexpr int kThreads = 256;  // 8 rows per CTA

// Exponents from the bits of a largest magnitude: with |x| = 1.f * 2^X the
// smallest e with |x| <= 6 * 2^e = 1.5 * 2^(e + 2) is X - 2, or X - 1 when
// f > 0.5, i.e. when adding 63 carries out of the 7 fraction bits.  Zeros and
// subnormals give at most -128, below every clamp.
__device__ __forceinline__ int nat_exponent(uint32_t bits) {
  return static_cast<int>((bits + 63u) >> 7) - 129;
}

// bf16 bits of the two values of a code byte times 2^e (exact: two
// significant bits).
__device__ __forceinline__ uint32_t dequant2(uint32_t byte, float scale) {
  const float2 f = __half22float2(fp4x2_to_half2(byte));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * scale, f.y * scale);
  return *reinterpret_cast<const uint32_t*>(&b);
}

// One row a warp.  Two or four rows a warp, their loads first, were slower
// (49,000 rows of a padded batch: 23.7 us, 24.2 and 25.2).
__global__ void __launch_bounds__(kThreads)
    k_latent_append_fp4(const uint4* lat, int64_t rows, int64_t n_new, const int32_t* __restrict__ n_add,
                        uint8_t* __restrict__ codes, uint8_t* __restrict__ scales, int64_t cap_tok,
                        const int64_t* __restrict__ len, int64_t max_len, uint4* stored) {
  const int lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5);
  if (row >= rows) return;  // uniform per warp, as every branch below
  const int64_t b = row / n_new, i = row - b * n_new;
  if (n_add && i >= n_add[b]) return;
  const int64_t p0 = len[b];
  if (p0 < 0 || p0 >= max_len - i) return;
  const uint4 u[2] = {lat[row * 64 + lane], lat[row * 64 + 32 + lane]};
  uint32_t big[2];  // bits of the group's largest magnitude
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t m = 0x7FFF7FFFu;
    const uint32_t v = __vmaxu2(__vmaxu2(u[h].x & m, u[h].y & m), __vmaxu2(u[h].z & m, u[h].w & m));
    big[h] = max(v & 0xFFFFu, v >> 16);
#pragma unroll
    for (int o = 1; o < 4; o <<= 1) big[h] = max(big[h], __shfl_xor_sync(0xffffffffu, big[h], o));
  }
  const bool nan[2] = {big[0] > 0x7F80u, big[1] > 0x7F80u};
  const uint32_t top =
      __reduce_max_sync(0xffffffffu, max(nan[0] ? 0u : big[0], nan[1] ? 0u : big[1]));
  const int E = min(max(nat_exponent(top), -kFp4MaxExp), kFp4MaxExp);
  const int64_t at = b * cap_tok + p0 + i;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int e = min(max(nat_exponent(big[h]), E - kFp4Spread), E);
    const uint32_t byte = nan[h] ? kFp4NanByte : static_cast<uint32_t>(e + 127);
    const float inv = __int_as_float((127 - e) << 23);  // 2^-e
    const uint32_t w[4] = {u[h].x, u[h].y, u[h].z, u[h].w};
    uint32_t c = 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      // x * 2^-e is exact; one rounding to E2M1, nearest even, saturating
      const float2 f = make_float2(__uint_as_float(w[k] << 16) * inv,
                                   __uint_as_float(w[k] & 0xFFFF0000u) * inv);
      c |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(f, __NV_E2M1, cudaRoundNearest)) << (8 * k);
    }
    if (nan[h]) c = 0;
    reinterpret_cast<uint32_t*>(codes + at * kFp4CodeBytes)[32 * h + lane] = c;
    if ((lane & 3) == 0) scales[at * kFp4Groups + 8 * h + (lane >> 2)] = static_cast<uint8_t>(byte);
    if (stored) {
      const float s = fp4_scale(byte);
      stored[row * 64 + 32 * h + lane] = make_uint4(dequant2(c, s), dequant2(c >> 8, s),
                                                    dequant2(c >> 16, s), dequant2(c >> 24, s));
    }
  }
}

// A warp takes kRows rows in a row, all of whose loads it issues first: 1 where
// there are few rows, 4 where there are many (many_rows below).
template <int kRows>
__global__ void __launch_bounds__(kThreads)
    k_latent_read_fp4(const uint8_t* __restrict__ codes, const uint8_t* __restrict__ scales,
                      int64_t cap_tok, const int64_t* __restrict__ pos, int64_t rows, int64_t m,
                      const int64_t* __restrict__ n_vis, uint4* __restrict__ out) {
  const int lane = threadIdx.x & 31;
  const int64_t row0 =
      (static_cast<int64_t>(blockIdx.x) * (kThreads / 32) + (threadIdx.x >> 5)) * kRows;
  if (row0 >= rows) return;
  int64_t b = row0 / m, i = row0 - b * m;
  uint32_t c[kRows][2], s[kRows][2];
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    c[r][0] = c[r][1] = 0;  // zeros where there is no such token
    s[r][0] = s[r][1] = 127;
    if (row0 + r < rows) {
      const int64_t p = pos ? pos[row0 + r] : i;
      if (p >= 0 && p < min(n_vis[b], cap_tok)) {
        const int64_t at = b * cap_tok + p;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          c[r][h] = reinterpret_cast<const uint32_t*>(codes + at * kFp4CodeBytes)[32 * h + lane];
          s[r][h] = scales[at * kFp4Groups + 8 * h + (lane >> 2)];
        }
      }
      if (++i == m) {
        i = 0;
        ++b;
      }
    }
  }
#pragma unroll
  for (int r = 0; r < kRows; ++r) {
    if (row0 + r >= rows) break;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float f = fp4_scale(s[r][h]);
      const uint32_t x = c[r][h];
      out[(row0 + r) * 64 + 32 * h + lane] =
          make_uint4(dequant2(x, f), dequant2(x >> 8, f), dequant2(x >> 16, f), dequant2(x >> 24, f));
    }
  }
}

// Whether a warp reads 4 rows: from as many on as give half of the device's warps
// (64 an SM) work then.  Measured, one row a warp / four, on 148 SMs (18,944 rows),
// in us, rows from the front: 4,096 rows 2.7 / 3.0, 16,384 6.5 / 6.7, 24,576
// 8.4 / 8.1, 131,072 32.1 / 29.0; scattered rows: 4,096 2.9 / 3.4, 16,384 7.0 /
// 6.9, 24,576 8.8 / 8.4, 131,072 35.8 / 27.3.
bool many_rows(int64_t rows) { return rows >= int64_t(2) * 64 * device_sm_count(); }

cudaError_t grid_for(int64_t rows, int per_warp, unsigned* grid) {
  const int64_t per = kThreads / 32 * per_warp;
  const int64_t blocks = (rows + per - 1) / per;
  if (blocks > 0x7fffffff) return cudaErrorInvalidValue;
  *grid = static_cast<unsigned>(blocks);
  return cudaSuccess;
}

}  // namespace

cudaError_t launch_latent_append_fp4(int B, const void* lat, int64_t n_new, const int32_t* n_add,
                                     uint8_t* codes, uint8_t* scales, int64_t cap_tok,
                                     const int64_t* len_dev, int64_t max_len, void* stored,
                                     cudaStream_t stream) {
  const int64_t rows = B * n_new;
  if (rows <= 0) return cudaSuccess;
  unsigned grid = 0;
  if (cudaError_t e = grid_for(rows, 1, &grid)) return e;
  k_latent_append_fp4<<<grid, kThreads, 0, stream>>>(
      static_cast<const uint4*>(lat), rows, n_new, n_add, codes, scales, cap_tok, len_dev, max_len,
      static_cast<uint4*>(stored));
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_latent_read_fp4(int B, const uint8_t* codes, const uint8_t* scales,
                                   int64_t cap_tok, const int64_t* pos, int64_t m,
                                   const int64_t* n_vis, void* out, cudaStream_t stream) {
  const int64_t rows = B * m;
  if (rows <= 0) return cudaSuccess;
  const bool many = many_rows(rows);
  unsigned grid = 0;
  if (cudaError_t e = grid_for(rows, many ? 4 : 1, &grid)) return e;
  auto* kernel = many ? k_latent_read_fp4<4> : k_latent_read_fp4<1>;
  kernel<<<grid, kThreads, 0, stream>>>(codes, scales, cap_tok, pos, rows, m, n_vis,
                                        static_cast<uint4*>(out));
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace spx
