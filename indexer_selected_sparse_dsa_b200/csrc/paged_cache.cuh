// The paged 8-bit latent cache: quantising rows as they are written, and
// reading them back to flat bf16 rows.
//
// A cache row stands for 512 latent and 64 rope values, all times one power of
// two:  c_kv = 2^k code,  k_rope = 2^k rope,  k the smallest whole number with
// max |c_kv| <= 448 2^k (448: e4m3's largest value), held to -60 .. 60.  Since
// the factor is a power of two, nothing but the e4m3 code is ever rounded: the
// rope half is exact, a code times 2^k is exact in bf16 (4 significant bits),
// and a kernel may take codes and rope as they are and apply 2^k to the sum.
// One factor per row is enough for a floating-point code: e4m3 keeps 3 bits of
// fraction over 2^15, so a value 2^14 below its row's largest is no worse off.
#pragma once
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "internal.h"
#include "ptx.cuh"

namespace dsa {

namespace {

constexpr int kRow8 = 640;       // bytes of a cache row: 512 codes, 64 bf16
constexpr int kExpMin = -60, kExpMax = 60;
constexpr int kCacheThreads = 256;

// The page of its sequence that position s lies in (an integer division takes some 20 instructions).
__device__ __forceinline__ int page_index(const PagedCache& c, int s) {
  return int((unsigned long long)unsigned(s) * c.page_mul >> c.page_shift);
}

// The row of the flattened cache that holds position s of sequence b, or -1
// (and the status bit) where the page table points outside the cache.
__device__ __forceinline__ int cache_row(const PagedCache& c, int b, int s) {
  const int p = page_index(c, s);
  const int page = c.page_table[(long long)b * c.max_pages + p];
  if (page < 0 || page >= c.n_pages) {
    raise_status(kStatusBadRow);
    return -1;
  }
  return page * c.page_size + (s - p * c.page_size);
}

// Longest sequence the page table can describe.
__device__ __forceinline__ long long max_positions(const PagedCache& c) { return (long long)c.max_pages * c.page_size; }

// Sequence that owns query row t (all lanes of a warp, same t): the number of
// cu_q[1 .. batch] that are <= t, found 32 ways at a time.
__device__ __forceinline__ int owner_of(const int32_t* __restrict__ cu_q, int batch, int t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = (lane + 1) * step;
    const bool le = i <= n && cu_q[lo + i] <= t;
    const int c = __popc(__ballot_sync(0xffffffffu, le));
    lo += c * step;
    n = min(step - 1, n - c * step);
  }
  return lo;
}

// Positions that query row t of sequence b sees: 0 .. seen - 1, its own the last.
// 0 (and the status bit) where cu_q, T, seq_len and the page table do not describe it.
__device__ __forceinline__ int seen_by(const PagedCache& c, const int32_t* __restrict__ cu_q,
                                       const int32_t* __restrict__ seq_len, int T, int b, int t) {
  const int q0 = cu_q[b], q1 = cu_q[b + 1], len = seq_len[b];
  const long long seen = (long long)len - ((long long)q1 - t) + 1;
  if (q0 < 0 || t < q0 || t >= q1 || q1 > T || seen < 1 || len > max_positions(c)) {
    raise_status(kStatusBadRow);
    return 0;
  }
  return int(seen);
}

// Exponent k of a row whose largest finite |c_kv| has the fp32 pattern `bits`.
__device__ __forceinline__ int row_exponent(uint32_t bits) {
  const int e = int(bits >> 23) - 127;  // amax = 1.m 2^e; 448 = 1.75 2^8
  const int k = e - 8 + ((bits & 0x7fffffu) > 0x600000u ? 1 : 0);
  return bits < 0x00800000u ? kExpMin : min(max(k, kExpMin), kExpMax);
}

__device__ __forceinline__ float pow2f(int k) { return __uint_as_float(uint32_t(k + 127) << 23); }

// What has to move is 1152 bytes in and 644 out a row: 37913 rows take 15.7 us from HBM (4.3 TB/s, 0.66 of the measured
// copy rate, at which they would take 10.4 us), 13.6 us again and again where they stay in L2; 13 rows 2.0 us, a launch.
// One warp per row, so that the row's largest value is one warp reduction; four rows a warp, for more loads in flight, took
// 15.8 us where one took 13.9, from L2 (from HBM it was not tried).  Lane l holds latent
// values 8 l .. 8 l + 7, 256 + 8 l .. + 7 and rope values 2 l, 2 l + 1, so every load and store is whole lines.
__global__ void __launch_bounds__(kCacheThreads)
    cache_write_kernel(const uint16_t* __restrict__ rows, long long rows_ld, int T, const int32_t* __restrict__ cu_q,
                       const int32_t* __restrict__ seq_len, PagedCache c) {
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31;
  const int t = blockIdx.x * (kCacheThreads / 32) + (threadIdx.x >> 5);
  if (t >= T) return;
  const uint16_t* src = rows + t * rows_ld;
  const uint4 x0 = *reinterpret_cast<const uint4*>(src + 8 * lane);
  const uint4 x1 = *reinterpret_cast<const uint4*>(src + 256 + 8 * lane);
  const uint32_t xr = *reinterpret_cast<const uint32_t*>(src + 512 + 2 * lane);

  const int b = owner_of(cu_q, c.batch, t);
  if (b >= c.batch || (b == 0 && t < cu_q[0])) return;  // behind the last sequence, or before the first
  const int seen = seen_by(c, cu_q, seq_len, T, b, t);
  const int row = seen > 0 ? cache_row(c, b, seen - 1) : -1;
  if (row < 0) return;

  const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
  float v[16];
  uint32_t amax = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    const uint32_t a = __float_as_uint(v[i]) & 0x7fffffffu;
    if (a < 0x7f800000u) amax = max(amax, a);
    else v[i] = __uint_as_float(0x7fc00000u);  // an infinity is stored as NaN, not as some finite value
  }
  amax = __reduce_max_sync(0xffffffffu, amax);
  const int k = row_exponent(amax);
  const float inv = pow2f(-k);
  uint32_t code[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i] * inv, v[4 * i + 1] * inv), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(v[4 * i + 2] * inv, v[4 * i + 3] * inv), __NV_SATFINITE, __NV_E4M3);
    code[i] = lo | (hi << 16);
  }
  uint8_t* dst = c.kv8 + (long long)row * kRow8;
  *reinterpret_cast<uint2*>(dst + 8 * lane) = make_uint2(code[0], code[1]);
  *reinterpret_cast<uint2*>(dst + 256 + 8 * lane) = make_uint2(code[2], code[3]);
  const __nv_bfloat162 r2 =
      __floats2bfloat162_rn(__uint_as_float(xr << 16) * inv, __uint_as_float(xr & 0xffff0000u) * inv);
  *reinterpret_cast<__nv_bfloat162*>(dst + 512 + 4 * lane) = r2;
  if (lane == 0) c.kv_scale[row] = pow2f(k);
}

// Two e4m3 codes (low 16 bits) times s, as two bf16.
__device__ __forceinline__ uint32_t codes_to_bf16x2(uint32_t codes, float s) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(codes & 0xffffu), __NV_E4M3);
  const float2 f = __half22float2(__half2(h));
  const __nv_bfloat162 o = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t*>(&o);
}

// Length of sequence b as the reader takes it: 0 (and the status bit, once) where
// the table or the flat rows cannot hold it.
__device__ __forceinline__ int read_len(const PagedCache& c, const int32_t* seq_len, const int64_t* kv_start,
                                        long long cache_rows, int b, bool report) {
  const int n = seq_len[b];
  const long long k0 = kv_start[b];
  if (n == 0) return 0;
  if (n < 0 || n > max_positions(c) || k0 < 0 || k0 + n > cache_rows) {
    if (report) raise_status(kStatusBadRow);
    return 0;
  }
  return n;
}

// The rows of all sequences, in order, are cut into equal shares, one per CTA.
// Each CTA finds the sequence its share starts in with one scan over the
// lengths; from there its warps walk on, one row per warp at a time.  1796 bytes
// a row have to move: 64850 rows of 16 ragged sequences take 24.4 us from HBM (0.73
// of the measured copy rate, at which they would take 17.8 us), 20.2 us with part of
// them in L2; one sequence of 777 rows 4.2 us, of which the chain length, table,
// page, row is most (four rows at a time per warp made that 5.4 us).
__global__ void __launch_bounds__(kCacheThreads)
    cache_read_kernel(PagedCache c, const int32_t* __restrict__ seq_len, const int64_t* __restrict__ kv_start,
                      uint16_t* __restrict__ kv, long long cache_rows) {
  __shared__ long long warp_sum[kCacheThreads / 32];
  __shared__ int start_b;
  __shared__ long long start_off;
  pdl_wait();
  pdl_trigger();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  constexpr int kWarps = kCacheThreads / 32;

  const int per = (c.batch + kCacheThreads - 1) / kCacheThreads;
  const int b0 = min(int(threadIdx.x) * per, c.batch), b1 = min(b0 + per, c.batch);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += read_len(c, seq_len, kv_start, cache_rows, b, blockIdx.x == 0);
  long long incl = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, o);
    if (lane >= o) incl += up;
  }
  if (lane == 31) warp_sum[warp] = incl;
  __syncthreads();
  long long before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sum[w];
    total += warp_sum[w];
  }
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long g0 = share * blockIdx.x, g1 = min(g0 + share, total);
  if (g0 >= g1) return;  // the same for the whole CTA
  long long at = before + incl - mine;
  if (g0 >= at && g0 < at + mine) {
    int b = b0;
    for (;; ++b) {
      const int n = read_len(c, seq_len, kv_start, cache_rows, b, false);
      if (g0 < at + n) break;
      at += n;
    }
    start_b = b;
    start_off = g0 - at;
  }
  __syncthreads();
  int b = start_b;
  long long s = start_off + warp;
  int n = read_len(c, seq_len, kv_start, cache_rows, b, false);
  for (long long g = g0 + warp; g < g1; g += kWarps, s += kWarps) {
    while (s >= n) {
      s -= n;
      n = read_len(c, seq_len, kv_start, cache_rows, ++b, false);
    }
    const int row = cache_row(c, b, int(s));
    if (row < 0) continue;
    const uint8_t* src = c.kv8 + (long long)row * kRow8;
    const uint2 q0 = *reinterpret_cast<const uint2*>(src + 8 * lane);
    const uint2 q1 = *reinterpret_cast<const uint2*>(src + 256 + 8 * lane);
    const __nv_bfloat162 r = *reinterpret_cast<const __nv_bfloat162*>(src + 512 + 4 * lane);
    const float f = c.kv_scale[row];
    uint16_t* dst = kv + (kv_start[b] + s) * 576;
    *reinterpret_cast<uint4*>(dst + 8 * lane) = make_uint4(codes_to_bf16x2(q0.x, f), codes_to_bf16x2(q0.x >> 16, f),
                                                           codes_to_bf16x2(q0.y, f), codes_to_bf16x2(q0.y >> 16, f));
    *reinterpret_cast<uint4*>(dst + 256 + 8 * lane) = make_uint4(codes_to_bf16x2(q1.x, f), codes_to_bf16x2(q1.x >> 16, f),
                                                                 codes_to_bf16x2(q1.y, f), codes_to_bf16x2(q1.y >> 16, f));
    *reinterpret_cast<__nv_bfloat162*>(dst + 512 + 2 * lane) =
        __floats2bfloat162_rn(__low2float(r) * f, __high2float(r) * f);
  }
}

}  // namespace

cudaError_t launch_cache_write(const CacheWriteLaunch& p) {
  const unsigned rows = kCacheThreads / 32;
  return launch_pdl(cache_write_kernel, dim3((unsigned(p.T) + rows - 1) / rows), dim3(kCacheThreads), 0, p.stream, 1,
                    p.rows, (long long)p.rows_ld, p.T, p.cu_q, p.seq_len, p.cache);
}

cudaError_t launch_cache_read(const CacheReadLaunch& p) {
  return launch_pdl(cache_read_kernel, dim3(unsigned(p.sm_count) * 8u), dim3(kCacheThreads), 0, p.stream, 1, p.cache,
                    p.seq_len, p.kv_start, p.kv, (long long)p.cache_rows);
}

}  // namespace dsa
