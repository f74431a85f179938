// Latent attention of new tokens over the paged 8-bit cache (paged_cache.cuh).
//
//   S[h,s]   = scale 2^k_s (q_lat[h] . code_s + q_rope[h] . rope_s)
//   o_lat[h] = sum_s softmax_s(S[h,:]) 2^k_s code_s,   lse[h] = log sum_s exp S[h,s]
//
// over every position the token sees, or over its selected positions.
//
// One warp per (query row, head), one key at a time with a running maximum and
// sum: lane l holds latent dims 16 l .. 16 l + 15 and rope dims 2 l, 2 l + 1.
#pragma once
#include <cuda_bf16.h>

#include "internal.h"
#include "paged_cache.cuh"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kPagedThreads = 256;

__global__ void __launch_bounds__(kPagedThreads)
    paged_mla_kernel(const uint16_t* __restrict__ q, int T, const int32_t* __restrict__ cu_q,
                     const int32_t* __restrict__ seq_len, const int32_t* __restrict__ idx, int topk, PagedCache c,
                     float scale_log2, __nv_bfloat16* __restrict__ o_lat, float* __restrict__ lse) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x >> 3, h = (blockIdx.x & 7) * 8 + (threadIdx.x >> 5);
  const int b = owner_of(cu_q, c.batch, t);
  if (b >= c.batch) return;
  const int seen = seen_by(c, cu_q, seq_len, b, t);
  const uint16_t* qh = q + ((long long)t * 64 + h) * 576;
  float ql[16], qr[2];
#pragma unroll
  for (int i = 0; i < 16; ++i) ql[i] = bf16_bits_to_float(qh[16 * lane + i]) * scale_log2;
  qr[0] = bf16_bits_to_float(qh[512 + 2 * lane]) * scale_log2;
  qr[1] = bf16_bits_to_float(qh[512 + 2 * lane + 1]) * scale_log2;
  float m = -INFINITY, l = 0.f, o[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) o[i] = 0.f;
  const int n = idx ? topk : seen;
  for (int j = 0; j < n; ++j) {
    int s = j;
    if (idx) {
      s = idx[(long long)t * topk + j];
      if (s < 0) continue;
      if (s >= seen) {
        raise_status(kStatusBadRow);
        continue;
      }
    }
    const int row = cache_row(c, b, s);
    if (row < 0) continue;
    const uint8_t* kp = c.kv8 + (long long)row * kRow8;
    const uint4 w = *reinterpret_cast<const uint4*>(kp + 16 * lane);
    const float2 r = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(kp + 512 + 4 * lane));
    const float f = c.kv_scale[row];
    const uint32_t ww[4] = {w.x, w.y, w.z, w.w};
    float k[16];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const __half2_raw hr =
          __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(ww[i >> 1] >> (16 * (i & 1))), __NV_E4M3);
      const float2 p = __half22float2(__half2(hr));
      k[2 * i] = p.x * f;
      k[2 * i + 1] = p.y * f;
    }
    float x = qr[0] * (r.x * f) + qr[1] * (r.y * f);
#pragma unroll
    for (int i = 0; i < 16; ++i) x = fmaf(ql[i], k[i], x);
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float mn = x > m ? x : m;
    const float al = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(x - mn);
    m = mn;
    l = l * al + p;
#pragma unroll
    for (int i = 0; i < 16; ++i) o[i] = fmaf(p, k[i], o[i] * al);
  }
  __nv_bfloat16* dst = o_lat + ((long long)t * 64 + h) * 512 + 16 * lane;
#pragma unroll
  for (int i = 0; i < 16; ++i) dst[i] = __float2bfloat16(l == 0.f ? 0.f : o[i] / l);
  if (lse && lane == 0) lse[(long long)t * 64 + h] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

}  // namespace

cudaError_t launch_paged_mla(const PagedMlaLaunch& p) {
  return launch_pdl(paged_mla_kernel, dim3(unsigned(p.T) * 8u), dim3(kPagedThreads), 0, p.stream, 1, p.q, p.T, p.cu_q,
                    p.seq_len, p.idx, p.topk, p.cache, p.scale * 1.4426950408889634f,
                    reinterpret_cast<__nv_bfloat16*>(p.o_lat), p.lse);
}

}  // namespace dsa
