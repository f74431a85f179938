// Latent attention of new tokens over the paged 8-bit cache (paged_cache.cuh).
//
//   S[h,s]   = scale 2^k_s (q_lat[h] . code_s + q_rope[h] . rope_s)
//   o_lat[h] = sum_s softmax_s(S[h,:]) 2^k_s code_s,   lse[h] = log sum_s exp S[h,s]
//
// over every position the token sees, or over its selected positions.
//
// Scores straight from the codes.  The query of a head is split once into
// q = 2^e (hi + lo / 16), both e4m3 (4 + 4 significant bits: exact for values
// within 2^13 of the head's largest, as lo's smallest step, 2^-9, is 2^-13 of 1 in
// hi's units, where that value is 224 to 448; below, off by half of it, 2^-21.8 of
// the largest at most), so
// the 8-bit tensor path multiplies the cache's codes as they lie in memory:
// M = 128 rows, 64 of hi and 64 of lo.  The rope half follows in bf16 on top: half
// of the query on the hi rows and eight times it on the lo rows, both exact.  (Zero
// lo rows would make NaN of an infinite rope value, where a head's -inf is weight 0;
// hi rows alone, M = 64, took 1.5% more time for a chunk.)  2^k_s, 2^e and the scale
// are applied to the fp32 sums.
//
// Values as fp16.  A code is exact in fp16, and a probability rounded to fp16
// (2^-11) is eight times closer than one in bf16.  The row's 2^k goes into the
// probability: with y = S log2(e) + k_s, u_s = 2^(y - m + 28) where m follows
// the maximum of y in whole numbers, at most 11 behind.  sum 2^-24 u code is the
// numerator: 2^-24 u is at most 2^15, and what fp16 cannot hold of it is 2^-29 of
// the largest.  sum u 2^-k_s (fp32, u before rounding) is the denominator, where a
// row of the smallest scale may weigh as much as one of the largest with a u
// 2^-120 of its: fp32 holds u down to 2^-126, 2^-154 of the largest, so what is
// lost of the denominator is below 2^-34 of it a key.
//
// Shared memory carries no query: hi and lo lie in tensor memory as the A operand
// (lanes 0..15 of each quarter the hi codes of 16 heads, lanes 16..31 their lo
// codes), the keys are the B operand, and S comes out with a lane per head.  One
// 16x32bx2 load then hands a thread the hi sums of its head, another the lo sums
// of the same keys: maximum, sum and scale of a head are registers, not a reduction
// over threads.
//
// What bounds it: per 128-key tile the tensor pipe is busy for 2300 cycles by its
// counter (2900 by the steps' measured times: 1024 codes, 260 rope, 1600 values at
// M = 128, N = 64), and shared memory moves 80 KB of codes in and 96 KB of operands
// out for S, 128 KB of widened values in and 192 KB out for O, 16 KB of P and 32 KB
// of the softmax's tables: 544 KB, 4350 cycles at 128 bytes each, against 3500 that a
// tile's 82 KB take from HBM.  Measured 5500 cycles a tile (a chunk of 148 rows,
// start and results included).  64 sequences of 2K to 16K positions, one token: 130
// us (3.3 TB/s, 0.50 of the measured copy rate; 147-157 us in a long run, with the
// clock at 1.6 GHz under the power cap); 778 tokens of two prompts' chunks, 512 of
// them over 8192 positions: 0.77-0.85 ms (760 to 840 TFLOP/s, 0.47 to 0.52 of the
// measured bf16 rate); 64 x 2048 selected rows: 49 us.
//
// The batch's 128-key tiles are shared out over the CTAs (paged_share.cuh), a CTA
// walking query row after query row; a row that ends in another CTA leaves partial
// sums that paged_mla_merge_kernel joins.  20 warps:
//  * warp 3 finds each key's cache row and 2^k, up to four tiles ahead;
//  * warps 0 and 1 copy the tile's rows with cp.async, four chunks of 128 codes and
//    the rope chunk, each 128 bytes of 128 keys;
//  * warps 4..11 read the codes again (they are in L2 by then), widen them to
//    fp16 and store them for the value product, three slots of 128 keys x 128 dims;
//    at the end of a row they write its result;
//  * warps 12..19 are the softmax (a thread: one head, 32 keys) and prepare the
//    next row's query while the last value product of a row runs;
//  * warp 2 issues S = Q K^T (M = 64 heads x (hi, lo), N = 128 keys) one tile
//    ahead of O^T += V^T P^T (M = 128 dims x 4, N = 64 heads).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <algorithm>

#include "internal.h"
#include "paged_cache.cuh"
#include "paged_share.cuh"
#include "ptx.cuh"
#include "sparse_mla.cuh"

namespace dsa {

namespace {

constexpr int kPgThreads = 640;       // five warps per scheduler: 96 registers a thread
constexpr int kPgMma = 2, kPgAddr = 3, kPgVWarp = 4, kPgSoft = 12;  // first warp of each role (keys: 0)
constexpr int kPgSlot = 16384;        // 128 keys x 128 bytes, 128B-swizzled
constexpr int kPgKSlots = 5;          // the five chunks of a tile, each in a place of its own
constexpr int kPgKGroups = 3;         // waited for together: codes 0..255, codes 256..511, rope
constexpr int kPgVSlots = 3;          // of 128 dims: one product runs, one is ready, one is being widened
constexpr int kPgRows = 4;            // tiles whose keys are described
constexpr unsigned long long kPgBriefNs = 8000;  // wait limits below it are brief: two failing tries
constexpr float kPgShift = 28.f;      // log2 of u at the running maximum ...
constexpr float kPgLazy = 11.f;       // ... which a score may pass by this much ...
constexpr float kPgHalf = 1.f / (1 << 24);  // ... and u's factor in the value product (fp16 ends at 2^16)

constexpr int kPgQR = 0;                                     // the query's rope half: 128 rows (1/2 and 8 times it) x 64 bf16
constexpr int kPgP = kPgQR + kPgSlot;                        // 2 chunks of 64 heads x 64 keys fp16
constexpr int kPgK = kPgP + kPgSlot;
constexpr int kPgV = kPgK + kPgKSlots * kPgSlot;             // a slot: two chunks of 128 keys x 64 dims fp16
constexpr int kPgKeyOff = kPgV + kPgVSlots * 2 * kPgSlot;    // of 128 keys: int row, float 2^k scale log2(e), k, 2^-k
constexpr int kPgRedOff = kPgKeyOff + kPgRows * 2048;        // float red[2][64]
constexpr int kPgMOff = kPgRedOff + 512;                     // float alpha[64], 1 / l [64], 2^-e[64]
constexpr int kPgStageOff = kPgMOff + 768;                   // codes of 64 dims on their way to tensor memory: 128 rows x 64
constexpr int kPgBarOff = kPgStageOff + 8192;
enum PgBar {
  kBarQFull, kBarQEmpty, kBarPFull, kBarPFree, kBarOFree, kBarCodes, kBarSFull, kBarSFree, kBarLFull, kBarDrain,
  kBarKFull, kBarKEmpty = kBarKFull + kPgKGroups, kBarVFull = kBarKEmpty + kPgKGroups,
  kBarVEmpty = kBarVFull + kPgVSlots, kBarRowFull = kBarVEmpty + kPgVSlots, kBarRowEmpty = kBarRowFull + kPgRows,
  kPgBars = kBarRowEmpty + kPgRows
};
constexpr int kPgTailOff = kPgBarOff + 8 * kPgBars;          // tmem address, start (b, t, tile), share, tiles before start and end
constexpr int kPgSmem = kPgTailOff + 64;
constexpr int kPgSmemAlloc = kPgSmem + 1024;
constexpr uint32_t kPgQCol = 128, kPgOCol = 256;             // S: 128 columns; Q: 128 (512 codes); O^T: 4 x 64

// ln(2^(m - kPgShift) l), -inf for l = 0.  m and l may be far from 1 in opposite directions (by a row's 2^k): whole
// exponents are added first, so that the sum is rounded at its own size.
__device__ __forceinline__ float log_sum(float m, float l) {
  const uint32_t bits = __float_as_uint(l);
  if (l == 0.f) return -INFINITY;
  if (bits - 0x00800000u >= 0x7f000000u) return (m - kPgShift + log2f(l)) * 0.69314718055994531f;  // not a normal number
  const float e = float(int(bits >> 23) - 127), f = __uint_as_float((bits & 0x007fffffu) | 0x3f800000u);
  return ((m - kPgShift + e) + log2f(f)) * 0.69314718055994531f;
}

// Query rows of sequence b: 0 (and the status bit) where cu_q is not in order.
__device__ __forceinline__ int seq_rows(const int32_t* __restrict__ cu_q, int T, int b, int& q0, bool report) {
  q0 = cu_q[b];
  const int q1 = cu_q[b + 1];
  if (q0 < 0 || q1 < q0 || q1 > T) {
    if (report) raise_status(kStatusBadRow);
    return 0;
  }
  return q1 - q0;
}

// The batch's tiles as every role of a CTA walks them, in order: row t of
// sequence b, tile `tile` of the row's `ntiles`, `left` tiles until the CTA's end.
struct TileWalk {
  const PagedCache& c;
  const int32_t* __restrict__ cu_q;
  const int32_t* __restrict__ seq_len;
  int T;
  int topk_tiles;  // 0: dense
  int b, t, tile, ntiles, seen, row_end;
  int left;

  __device__ __forceinline__ void enter_row() {
    const int len = seq_len[b];
    const long long n = (len > max_positions(c)) ? 0 : (long long)len - (row_end - t) + 1;
    seen = n < 1 ? 0 : int(n);
    ntiles = topk_tiles ? topk_tiles : max(1, int((unsigned(seen) + 127u) >> 7));
  }
  __device__ __forceinline__ void start(const int* at, int tiles) {
    b = at[0];
    t = at[1];
    tile = at[2];
    left = tiles;
    row_end = cu_q[b + 1];
    enter_row();
  }
  // the tiles of this CTA in the current row
  __device__ __forceinline__ int segment() const { return min(ntiles - tile, left); }
  // step over n <= segment() tiles
  __device__ __forceinline__ void advance(int n) {
    left -= n;
    tile += n;
    if (left > 0 && tile == ntiles) {
      tile = 0;
      if (++t == row_end) {
        int q0 = 0, nq = 0;
        while (nq == 0 && b + 1 < c.batch) nq = seq_rows(cu_q, T, ++b, q0, false);
        t = q0;
        row_end = q0 + nq;
      }
      enter_row();
    }
  }
};

// Sixteen codes of each of a thread's four keys; zeros where the tile has no key at all.
__device__ __forceinline__ void load_codes(uint4 (&w)[4], const uint8_t* const (&src)[4], int col, bool any) {
#pragma unroll
  for (int j = 0; j < 4; ++j) w[j] = make_uint4(0, 0, 0, 0);
  if (any) {
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = *reinterpret_cast<const uint4*>(src[j] + col);
  }
}

// Sixteen codes as fp16, into two 16-byte segments.
__device__ __forceinline__ void store_fp16(uint8_t* s0, uint8_t* s1, const uint4& x) {
  const uint32_t xs[4] = {x.x, x.y, x.z, x.w};
  uint32_t f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, l;\n\tcvt.rn.f16x2.e4m3x2 %1, h;\n\t}"
        : "=r"(f[2 * i]), "=r"(f[2 * i + 1])
        : "r"(xs[i]));
  *reinterpret_cast<uint4*>(s0) = make_uint4(f[0], f[1], f[2], f[3]);
  *reinterpret_cast<uint4*>(s1) = make_uint4(f[4], f[5], f[6], f[7]);
}

// The largest magnitudes of eight bf16, even and odd ones apart (as patterns: they order like the values).
__device__ __forceinline__ uint32_t max_abs_bf16(const uint4& x) {
  return __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu), __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
}
// 2^-e with max |q| <= 448 2^e, from the largest magnitude's fp32 pattern.  NaN where that is infinite or NaN (codes have
// no infinity): all of the head's codes become NaN.
__device__ __forceinline__ float query_scale(uint32_t a) {
  const int e = max(int(a >> 23) - 135 + ((a & 0x7fffffu) > 0x600000u ? 1 : 0), -100);
  return a < 0x7f800000u ? pow2f(-e) : __uint_as_float(0x7fc00000u);
}
__device__ __forceinline__ uint32_t scale_bf16x2(uint32_t w, f32x2 inv) {
  float a, b;
  f2_unpack(f2_mul(f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u)), inv), a, b);
  const __nv_bfloat162 o = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&o);
}
__device__ __forceinline__ uint4 scale_bf16x8(const uint4& x, f32x2 inv) {
  return make_uint4(scale_bf16x2(x.x, inv), scale_bf16x2(x.y, inv), scale_bf16x2(x.z, inv), scale_bf16x2(x.w, inv));
}

// Four query values (two words of bf16 pairs) times inv as hi codes and lo codes: v = hi + lo / 16.  v goes through
// fp16, exact but for what is 2^-33 of 448.
__device__ __forceinline__ void split_codes(uint32_t w0, uint32_t w1, f32x2 inv, uint32_t& hi, uint32_t& lo) {
  const uint32_t w[2] = {w0, w1};
  uint32_t c[2], d[2];
  const __half2 n16 = __half2half2(__ushort_as_half(0xcc00)), p16 = __half2half2(__ushort_as_half(0x4c00));  // -16, 16
#pragma unroll
  for (int p = 0; p < 2; ++p) {
    float a, b;
    f2_unpack(f2_mul(f2_pack(__uint_as_float(w[p] << 16), __uint_as_float(w[p] & 0xffff0000u)), inv), a, b);
    const __half2 v = __floats2half2_rn(a, b);
    c[p] = __nv_cvt_halfraw2_to_fp8x2(v, __NV_SATFINITE, __NV_E4M3);
    const __half2 f(__nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(c[p]), __NV_E4M3));
    d[p] = __nv_cvt_halfraw2_to_fp8x2(__hfma2(f, n16, __hmul2(v, p16)), __NV_SATFINITE, __NV_E4M3);
  }
  hi = __byte_perm(c[0], c[1], 0x5410);
  lo = __byte_perm(d[0], d[1], 0x5410);
}

template <bool kSparse, bool kBrief>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_mla_kernel(const uint16_t* __restrict__ q, int T, const int32_t* __restrict__ cu_q,
                     const int32_t* __restrict__ seq_len, const int32_t* __restrict__ idx, int topk,
                     const __grid_constant__ PagedCache c, float scale_log2, __nv_bfloat16* __restrict__ o_lat,
                     float* __restrict__ lse, int2* __restrict__ meta, float* __restrict__ part_out, WaitLimit lim) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kPgBarOff + 8u * i; };
  auto keys_of = [&](int n) { return smem + kPgKeyOff + (n % kPgRows) * 2048; };  // the table of the CTA's tile n
  float* alpha_s = reinterpret_cast<float*>(smem + kPgMOff);
  float* linv_s = alpha_s + 64;
  float* qinv_s = alpha_s + 128;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kPgTailOff);
  int* start_s = reinterpret_cast<int*>(smem + kPgTailOff + 8);  // b, t, tile where this CTA begins; a share
  long long* ends_s = reinterpret_cast<long long*>(smem + kPgTailOff + 24);  // the batch's tiles before it, and before the next
  // (by a shuffle, so that the compiler knows it to be the same in all lanes: the roles' addresses and descriptors
  // then live in uniform registers)
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const int topk_tiles = kSparse ? (topk + 127) >> 7 : 0;

  if (threadIdx.x == 0) {
    mbar_init(bar(kBarQFull), 8);  // one arrival per warp of the role, where several arrive
    mbar_init(bar(kBarQEmpty), 1);
    mbar_init(bar(kBarPFull), 8);
    mbar_init(bar(kBarPFree), 1);
    mbar_init(bar(kBarOFree), 8);
    mbar_init(bar(kBarCodes), 1);
    mbar_init(bar(kBarSFull), 1);
    mbar_init(bar(kBarSFree), 8);
    mbar_init(bar(kBarLFull), 8);
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < kPgKGroups; ++i) {
      mbar_init(bar(kBarKFull + i), 64);  // every copying thread
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < kPgVSlots; ++i) {
      mbar_init(bar(kBarVFull + i), 8);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    for (int i = 0; i < kPgRows; ++i) {
      mbar_init(bar(kBarRowFull + i), 1);
      mbar_init(bar(kBarRowEmpty + i), 18);  // the key, value and softmax warps
    }
    fence_mbar_init();
  }
  if (warp == kPgMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();

  // ---------------------------------------------------------------- this CTA's share
  // (paged_share.cuh.)  Rows split with the cost of their start counted, against equal shares of tiles alone: 16 sequences
  // of up to six drafted tokens 69 -> 62 us, 64 x 2048 selected rows 52.5 -> 49.6 us, 300 positions 16.6 -> 17.2 us (two
  // sums to scan).  A cost of 1 or 3 tiles: 64 and 62 us, 52 and 51 us.
  {
    longlong2* sums = reinterpret_cast<longlong2*>(smem);  // the warps' sums, in the rope half's room
    int* longest_s = reinterpret_cast<int*>(sums + 32);
    const int per = (c.batch + kPgThreads - 1) / kPgThreads;
    const int b0 = min(int(threadIdx.x) * per, c.batch), b1 = min(b0 + per, c.batch);
    auto tiles = [&](int b, int& q0, int& nq, long long& len, bool report) {
      nq = seq_rows(cu_q, T, b, q0, report);
      len = seq_len[b];
      if (len < 0 || len > max_positions(c)) len = -1;
      if (report && nq > 0 && len < nq) raise_status(kStatusBadRow);
      return tiles_of(nq, len, topk_tiles, nq);
    };
    auto scan = [&](longlong2 v) {  // inclusive, over the lanes
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const longlong2 up = make_longlong2(__shfl_up_sync(0xffffffffu, v.x, o), __shfl_up_sync(0xffffffffu, v.y, o));
        if (lane >= o) v = make_longlong2(v.x + up.x, v.y + up.y);
      }
      return v;
    };
    int q0, nq;
    long long len;
    longlong2 mine = make_longlong2(0, 0);  // tiles, rows
    int longest = 0;                        // tiles of a row
    for (int b = b0; b < b1; ++b) {
      mine.x += tiles(b, q0, nq, len, blockIdx.x == 0);
      mine.y += nq;
      if (nq > 0) longest = max(longest, topk_tiles ? topk_tiles : int((max(len, 1ll) + 127) >> 7));
    }
    const longlong2 incl = scan(mine);
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
      sums[warp] = incl;
      longest_s[warp] = longest;
    }
    __syncthreads();
    longest = __reduce_max_sync(0xffffffffu, lane < kPgThreads / 32 ? longest_s[lane] : 0);
    const longlong2 all = scan(lane < kPgThreads / 32 ? sums[lane] : make_longlong2(0, 0));
    const long long all_tiles = __shfl_sync(0xffffffffu, all.x, 31);
    const long long all_rows = __shfl_sync(0xffffffffu, all.y, 31);
    const int wb = max(warp - 1, 0);
    const longlong2 before = make_longlong2(__shfl_sync(0xffffffffu, all.x, wb), __shfl_sync(0xffffffffu, all.y, wb));
    const PagedShares sh = paged_shares(all_tiles, all_rows, longest, int(gridDim.x));
    if (threadIdx.x == 64) start_s[3] = int(min(sh.share, 1ll << 30));  // (a row has less than 2^24 tiles)
    const long long x0 = incl.x - mine.x + (warp ? before.x : 0), y0 = incl.y - mine.y + (warp ? before.y : 0);
#pragma unroll 1
    for (int e = 0; e < 2; ++e) {  // where the share begins, and where it ends
      const long long g = sh.begin(int(blockIdx.x) + e);
      long long x = x0, at = sh.line(x0, y0);
      if (g < at || g >= at + sh.line(mine.x, mine.y)) continue;
      for (int b = b0;; ++b) {
        const long long n = per == 1 ? mine.x : tiles(b, q0, nq, len, false);  // (one sequence: its numbers are at hand)
        if (g < at + sh.line(n, nq)) {
          long long first;
          int tile;
          const int row = sh.cut(nq, len, topk_tiles, g - at, first, tile);
          if (e == 0) {
            start_s[0] = b;
            start_s[1] = q0 + row;
            start_s[2] = tile;
          }
          ends_s[e] = x + first + tile;  // tiles before g
          break;
        }
        x += n;
        at += sh.line(n, nq);
      }
    }
    const long long end = sh.line(all_tiles, all_rows);
    if (threadIdx.x == 0 && sh.begin(int(blockIdx.x) + 1) >= end) ends_s[1] = all_tiles;
    if (threadIdx.x == 32 && sh.begin(int(blockIdx.x)) >= end) ends_s[0] = all_tiles;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  constexpr uint32_t tmem = 0;  // all 512 columns: the allocation starts at 0
  TileWalk walk{c, cu_q, seq_len, T, topk_tiles, 0, 0, 0, 0, 0, 0, 0};
  const int own_tiles = int(ends_s[1] - ends_s[0]);
  const bool busy = own_tiles > 0;
  if (busy) walk.start(start_s, own_tiles);
  else if (threadIdx.x == 0) meta[blockIdx.x] = make_int2(-1, 0);

  // A bounded wait of a whole warp; the lanes agree on its outcome.  A try that fails comes back after 4 us (measured, with
  // any time hint), so a limit below two of them takes the kernel that looks without suspending.  The time is the SM's
  // cycles at 2 a ns (its clock is at most 1.965 GHz): globaltimer in each of the 18 waits costs 0.9% of a chunk.  Who gives
  // up leaves its loop; the roles that wait for it run into their own limits.
  const long long limit = 2 * (long long)min(lim.ns, 1ull << 60);
  auto warp_wait = [&](uint32_t b, uint32_t parity) {
    const long long t0 = clock64();
    bool done;
#pragma unroll 1
    do done = __all_sync(0xffffffffu, kBrief ? mbar_test_wait(b, parity) : mbar_try_wait(b, parity)) != 0;
    while (!done && !__any_sync(0xffffffffu, clock64() - t0 >= limit));
    return done;
  };
  // The same for the softmax: one warp tries, and a barrier hands all 256 threads the outcome, so that they leave
  // together if they have to.
  auto group_wait = [&](uint32_t b, uint32_t parity) {
    const bool done = warp == kPgSoft ? warp_wait(b, parity) : true;
    return bar_red_or(1, 256, done ? 0 : 1) == 0;
  };
  // --- the first row's query, by the value and softmax warps together: eight lanes to a head keep it in registers, and its
  // codes go through the room of the value slots in one step, where a later row's (below) go in eight through a small one
  // (one row over 300 positions: 17.4 -> 15.3 us against the softmax warps alone by that way).
  if (busy && warp >= kPgVWarp) {
    const int l8 = lane & 7, h = 4 * (warp - kPgVWarp) + (lane >> 3), row = 32 * (h >> 4) + (h & 15);
    const uint4* src = reinterpret_cast<const uint4*>(q + ((long long)walk.t * 64 + h) * 576) + l8;
    uint4 x[9];
#pragma unroll
    for (int i = 0; i < 9; ++i) x[i] = src[8 * i];
    uint32_t a = 0;
#pragma unroll
    for (int i = 0; i < 9; ++i) a = __vmaxu2(a, max_abs_bf16(x[i]));
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) a = __vmaxu2(a, __shfl_xor_sync(0xffffffffu, a, o));
    const float inv1 = query_scale(max(a << 16, a & 0xffff0000u));
    if (l8 == 0) qinv_s[h] = inv1;
    const f32x2 inv = f2_pack(inv1, inv1);
    // 16-byte units of a row of 512 bytes: two neighbouring rows in different halves of 128 bytes, eight all apart
    uint8_t* stage = smem + kPgV;
    auto unit = [](int r, int u) { return r * 512 + ((u ^ (4 * (r & 1) + ((r >> 1) & 3))) << 4); };
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      uint2 hi, lo;
      split_codes(x[i].x, x[i].y, inv, hi.x, lo.x);
      split_codes(x[i].z, x[i].w, inv, hi.y, lo.y);
      uint8_t* to = stage + unit(row, 4 * i + (l8 >> 1)) + 8 * (l8 & 1);  // (the swizzle is the same 16 rows on)
      *reinterpret_cast<uint2*>(to) = hi;
      *reinterpret_cast<uint2*>(to + 16 * 512) = lo;
    }
    uint8_t* rope = smem + kPgQR + row * 128 + ((l8 ^ (row & 7)) << 4);
    *reinterpret_cast<uint4*>(rope) = scale_bf16x8(x[8], f2_pack(0.5f * inv1, 0.5f * inv1));
    *reinterpret_cast<uint4*>(rope + 16 * 128) = scale_bf16x8(x[8], f2_pack(8.f * inv1, 8.f * inv1));
    named_bar_sync(2, 512);
    const int own = 32 * (warp & 3) + lane, piece = (warp >> 2) - 1;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float w[16];
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float4 y = *reinterpret_cast<const float4*>(stage + unit(own, 8 * piece + 4 * j + k));
        w[4 * k] = y.x, w[4 * k + 1] = y.y, w[4 * k + 2] = y.z, w[4 * k + 3] = y.w;
      }
      tmem_st16(tmem + (uint32_t(32 * (warp & 3)) << 16) + kPgQCol + 32 * piece + 16 * j, w);
    }
    tmem_wait_st();
    tc_fence_before();
    fence_proxy_async_smem();
    named_bar_sync(2, 512);
    if (warp >= kPgSoft && lane == 0) mbar_arrive(bar(kBarQFull));
  }
  if (!busy) {
    // nothing to do
  } else if (warp < kPgMma) {
    // ---------------------------------------------------------------- keys
    const int g = threadIdx.x & 7, r0 = threadIdx.x >> 3;  // segment g of rows r0 + 8 j
    const uint32_t dst = sbase + kPgK + uint32_t(r0 * 128 + ((g ^ r0) << 4));
    const uint8_t* base = c.kv8 + 16 * g;
    bool ok = true;
    for (int n = 0; n < walk.left && ok; ++n) {
      const int rb = n % kPgRows;
      if (!(ok = warp_wait(bar(kBarRowFull + rb), uint32_t(n / kPgRows) & 1u))) break;
      const int* row_s = reinterpret_cast<const int*>(keys_of(n)) + r0;
      const bool none = row_s[0] < 0;
      const uint8_t* src[16];
#pragma unroll
      for (int j = 0; j < 16; ++j) src[j] = base + (long long)max(row_s[8 * j], 0) * kRow8;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarRowEmpty + rb));
#pragma unroll
      for (int gr = 0; gr < kPgKGroups; ++gr) {
        if (!(ok = warp_wait(bar(kBarKEmpty + gr), (uint32_t(n) & 1u) ^ 1u))) break;
#pragma unroll
        for (int ch = 2 * gr; ch < min(2 * gr + 2, kPgKSlots); ++ch)
#pragma unroll
          for (int j = 0; j < 16; ++j)
            cp_async_16_or_zero(dst + ch * kPgSlot + j * 1024, src[j] + 128 * ch, none);
        cp_async_arrive_noinc(bar(kBarKFull + gr));
      }
    }
    if (!ok && lane == 0) raise_status(kStatusTimeout);
    cp_async_wait_all();
  } else if (warp == kPgAddr) {
    // ---------------------------------------------------------------- addresses
    // Keys lane + 32 i of each tile.  Position, page and scale are three loads
    // that follow from each other; each is made one tile after the one before it,
    // so that none is waited for.
    const int total = walk.left;
    int s2[4], s1[4], page1[4], row0[4], b2, seen2 = 0;
    float sc0[4];
    int seen_row = walk.t;  // (the first row's query is being read already)
    auto position = [&]() {  // of the walk's next tile (-1: none); then step on
      b2 = walk.b;
      if (walk.left > 0 && walk.t != seen_row) {  // a new row: its query is wanted soon
        seen_row = walk.t;
        const char* qr = reinterpret_cast<const char*>(q + (long long)walk.t * 64 * 576);
        for (int i = lane; i < 64 * 576 * 2 / 128; i += 32) prefetch_l2(qr + 128 * i);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int j = walk.tile * 128 + lane + 32 * i;
        int s = -1;
        if (walk.left > 0) {
          if (!kSparse) {
            s = j < walk.seen ? j : -1;
          } else if (j < topk) {
            s = idx[(long long)walk.t * topk + j];  // (looked at a step later)
          }
        }
        s2[i] = s;
      }
      seen2 = walk.seen;
      if (walk.left > 0) walk.advance(1);
    };
    auto page = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (kSparse && s2[i] >= seen2) {
          raise_status(kStatusBadRow);
          s2[i] = -1;
        }
        s1[i] = s2[i];
        page1[i] = s2[i] >= 0 ? c.page_table[(long long)b2 * c.max_pages + page_index(c, s2[i])] : 0;
      }
    };
    auto scale = [&]() {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        int y = -1;
        if (s1[i] >= 0) {
          if (page1[i] >= 0 && page1[i] < c.n_pages) y = page1[i] * c.page_size + (s1[i] - page_index(c, s1[i]) * c.page_size);
          else raise_status(kStatusBadRow);
        }
        row0[i] = y;
        sc0[i] = y >= 0 ? c.kv_scale[y] : 0.f;
      }
    };
    position();
    page();
    position();
    scale();
    page();
    position();
    for (int n = 0; n < total; ++n) {
      const int rb = n % kPgRows;
      if (!warp_wait(bar(kBarRowEmpty + rb), (uint32_t(n / kPgRows) & 1u) ^ 1u)) {
        if (lane == 0) raise_status(kStatusTimeout);
        break;
      }
      int* row_s = reinterpret_cast<int*>(keys_of(n)) + lane;
      float* cs_s = reinterpret_cast<float*>(row_s) + 128;
      // A place without a key takes the row of one that has: its score gets -inf added, and what other rows of the cache
      // hold (NaN perhaps) is not read.  -1 throughout where the tile has no key.
      const int some = __reduce_max_sync(0xffffffffu, max(max(row0[0], row0[1]), max(row0[2], row0[3])));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int e = int(__float_as_uint(sc0[i]) >> 23);  // k + 127
        const bool has = row0[i] >= 0;
        row_s[32 * i] = has ? row0[i] : some;
        cs_s[32 * i] = has ? sc0[i] * scale_log2 : 0x1p-24f;  // (any factor but 0, which times an infinite score is NaN)
        cs_s[128 + 32 * i] = has ? float(e - 127) : -INFINITY;
        cs_s[256 + 32 * i] = has ? pow2f(127 - e) : 0.f;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarRowFull + rb));
      scale();
      page();
      position();
    }
  } else if (warp == kPgMma) {
    // ---------------------------------------------------------------- MMA issuer
    const uint32_t el = elect_one();
    const uint32_t idesc_k = idesc_e4m3(128, 128);
    const uint32_t idesc_r = idesc_bf16(128, 128, 0, 0);
    const uint32_t idesc_v = idesc_f16(128, 64, 1, 0);
    const uint64_t qr_desc = smem_desc(sbase + kPgQR, 16, 1024, kSwizzle128B);
    const uint64_t k_desc = smem_desc(sbase + kPgK, 16, 1024, kSwizzle128B);
    const uint64_t p_desc = smem_desc(sbase + kPgP, 16, 1024, kSwizzle128B);
    const uint64_t v_desc = smem_desc(sbase + kPgV, kPgSlot, 1024, kSwizzle128B);
    int n = 0, seg = 0;  // tiles whose scores are issued, rows begun
    bool ok = true;
    // The keys' places are fixed by the chunk, and all that addresses are made of is the same in all lanes, so descriptors
    // stay in uniform registers: it is this warp's instructions, one in some ten cycles beside the other roles, that
    // bound the tile otherwise.
    int vs = 0;
    uint32_t vp = 0;
    auto values = [&](int m, uint32_t add) {  // 128 dims of the value product
      if (!warp_wait(bar(kBarVFull + vs), vp)) return false;
      tc_fence_after();
      const uint64_t vd = v_desc + vs * (2 * kPgSlot >> 4);
#pragma unroll
      for (int k = 0; k < 8; ++k)
        mma_f16_ss_in(el, tmem + kPgOCol + 64 * m, vd + 128 * k, p_desc + (k >> 2) * 512 + 2 * (k & 3), idesc_v,
                      k ? 1u : add);
      mma_commit_in(el, bar(kBarVEmpty + vs));
      if (++vs == kPgVSlots) {
        vs = 0;
        vp ^= 1u;
      }
      return true;
    };
    while (ok && walk.left > 0) {
      const int nt = __shfl_sync(0xffffffffu, walk.segment(), 0);
      if (!(ok = warp_wait(bar(kBarQFull), uint32_t(seg & 1)))) break;
      tc_fence_after();
#pragma unroll 1
      for (int t = -1; t < nt; ++t) {  // scores of tile t + 1, values of tile t
        const bool more = t + 1 < nt;
        const uint32_t np = uint32_t(n) & 1u;
        if (more) {
          // S of the codes; the buffer is free once the softmax has read the tile before
          if (n > 0 && !(ok = warp_wait(bar(kBarSFree), np ^ 1u))) break;
#pragma unroll
          for (int gr = 0; gr < 2; ++gr) {
            if (!(ok = warp_wait(bar(kBarKFull + gr), np))) break;
            fence_proxy_async_smem();
            tc_fence_after();
#pragma unroll
            for (int k = 8 * gr; k < 8 * gr + 8; ++k)
              mma_f8_ts_in(el, tmem, tmem + kPgQCol + 8 * k, k_desc + (k >> 2) * (kPgSlot >> 4) + 2 * (k & 3), idesc_k,
                           k ? 1u : 0u);
            mma_commit_in(el, bar(kBarKEmpty + gr));
          }
          if (!ok) break;
          mma_commit_in(el, bar(kBarCodes));
        } else {
          mma_commit_in(el, bar(kBarQEmpty));
        }
        if (t >= 0) {
          if (!(ok = warp_wait(bar(kBarPFull), np ^ 1u))) break;
          if (t == 0 && seg > 0 && !(ok = warp_wait(bar(kBarOFree), uint32_t(seg - 1) & 1u))) break;
          if (!(ok = values(0, t > 0 ? 1u : 0u))) break;
        }
        if (more) {
          // The rope half on top of the codes' sums.  Only products of one shape are ordered by their issue; these two
          // differ in the depth of a step, so a barrier stands between them (a part of the value product fills it).
          if (!(ok = warp_wait(bar(kBarCodes), np))) break;
          if (!(ok = warp_wait(bar(kBarKFull + 2), np))) break;
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            mma_f16_ss_in(el, tmem, qr_desc + 2 * k, k_desc + 4 * (kPgSlot >> 4) + 2 * k, idesc_r, 1u);
          mma_commit_in(el, bar(kBarKEmpty + 2));
          mma_commit_in(el, bar(kBarSFull));
          ++n;
        }
        if (t >= 0) {
          if (!(ok = values(1, t > 0 ? 1u : 0u)) || !(ok = values(2, t > 0 ? 1u : 0u)) ||
              !(ok = values(3, t > 0 ? 1u : 0u)))
            break;
          mma_commit_in(el, bar(kBarPFree));
        }
      }
      walk.advance(nt);
      ++seg;
    }
    if (!ok && lane == 0) raise_status(kStatusTimeout);
    // every product issued above must be complete before tensor memory is released
    mma_commit_in(el, bar(kBarDrain));
    mbar_drain(bar(kBarDrain), 0);
  } else if (warp < kPgSoft) {
    // ---------------------------------------------------------------- values
    const int vt = threadIdx.x - 32 * kPgVWarp;
    // Codes 16 g .. 16 g + 15 of rows r0 + 32 j: segments 2 (g % 4) and the next of
    // chunk g / 4 of the widened row.  Eight lanes take the first chunk of a row and
    // the second of its neighbour: with the swizzle, their stores fill all banks.
    const int g = vt & 7, r0 = (vt >> 3) ^ (g >> 2);
    const uint32_t voff = uint32_t((g >> 2) * kPgSlot + r0 * 128);
    const uint32_t seg0 = uint32_t(((2 * (g & 3)) ^ (r0 & 7)) << 4), seg1 = seg0 ^ 16u;
    const uint8_t* base = c.kv8 + 16 * g;
    uint8_t* const dst = smem + kPgV + voff;
    const int total = walk.left;
    int seg = 0, i = 0;  // rows begun, half tiles (256 dims) done
    if (vt == 0) meta[blockIdx.x] = make_int2(-1, 0);
    bool ok = true, any = false;
    const uint8_t* src[4];
    auto rows = [&](int n) {
      const int rb = n % kPgRows;
      if (!warp_wait(bar(kBarRowFull + rb), uint32_t(n / kPgRows) & 1u)) return false;
      const int* row_s = reinterpret_cast<const int*>(keys_of(n)) + r0;
      any = row_s[0] >= 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) src[j] = base + (long long)max(row_s[32 * j], 0) * kRow8;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarRowEmpty + rb));
      return true;
    };
    int vs = 0;
    uint32_t vp = 0;
    auto widen = [&](const uint4 (&w)[4]) {  // into the next slot
      if (!warp_wait(bar(kBarVEmpty + vs), vp ^ 1u)) return false;
      uint8_t* d = dst + vs * 2 * kPgSlot;
#pragma unroll
      for (int j = 0; j < 4; ++j) store_fp16(d + j * 4096 + seg0, d + j * 4096 + seg1, w[j]);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarVFull + vs));
      if (++vs == kPgVSlots) {
        vs = 0;
        vp ^= 1u;
      }
      return true;
    };
    // The codes of a slot are loaded two slots ahead, across tiles and rows.
    uint4 w0[4], w1[4];
    if ((ok = rows(0))) {
      load_codes(w0, src, 0, any);
      load_codes(w1, src, 128, any);
    }
    while (ok && walk.left > 0) {
      const int nt = walk.segment(), row = walk.t, tile = walk.tile;
      const bool whole = nt == walk.ntiles;
      if (!whole && tile == 0) {
        const int rest = walk.ntiles - nt, share = start_s[3];
        if (vt == 0) meta[blockIdx.x] = make_int2(row, 1 + (rest + share - 1) / share);
      }
      walk.advance(nt);
      const int end = i + 2 * nt;
#pragma unroll 1
      for (; i < end; ++i) {
        if (!(ok = widen(w0))) break;
        const bool more = i + 1 < 2 * total;
        const int col = (i & 1) ? 0 : 256;
        if (more) {
          if ((i & 1) && !(ok = rows((i + 1) >> 1))) break;
          load_codes(w0, src, col, any);
        }
        if (!(ok = widen(w1))) break;
        if (more) load_codes(w1, src, col + 128, any);
      }
      // --- the row's result, or this part's.  O^T: a lane per dim, a column per head.
      if (!ok || !(ok = warp_wait(bar(kBarLFull), uint32_t(seg & 1)))) break;
      if (!(ok = warp_wait(bar(kBarPFree), uint32_t((end >> 1) - 1) & 1u))) break;
      tc_fence_after();
      const int quarter = warp & 3, h0 = 32 * ((warp - kPgVWarp) >> 2), odd = lane & 1;
      // a CTA leaves at most two partial results: of the row it starts inside (0) and of the row it ends inside (1)
      float* prow = part_out + (long long)(2 * blockIdx.x + (tile == 0 ? 1 : 0)) * kPartFloats + h0 * 512 + 32 * quarter + lane;
      __nv_bfloat16* orow = o_lat + ((long long)row * 64 + h0 + odd) * 512 + 32 * quarter + (lane - odd);
#pragma unroll 1
      for (int mm = 0; mm < 4; ++mm) {
        float ov[32];
        tmem_ld32_sync((uint32_t(quarter * 32) << 16) + kPgOCol + 64 * mm + h0, ov);
        if (whole) {
          // two neighbouring lanes trade, so that each stores two dims of one head
#pragma unroll
          for (int h = 0; h < 32; h += 2) {
            const float2 li = *reinterpret_cast<const float2*>(linv_s + h0 + h);
            const float a = ov[h] * li.x, b = ov[h + 1] * li.y;
            const float got = __shfl_xor_sync(0xffffffffu, odd ? a : b, 1);
            *reinterpret_cast<__nv_bfloat162*>(orow + h * 512 + 128 * mm) =
                __floats2bfloat162_rn(odd ? got : a, odd ? b : got);
          }
        } else {
#pragma unroll
          for (int h = 0; h < 32; ++h) prow[h * 512 + 128 * mm] = ov[h];
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarOFree));
      ++seg;
    }
    if (!ok && vt == 0) meta[blockIdx.x] = make_int2(-1, 0);
    if (!ok && lane == 0) raise_status(kStatusTimeout);
  } else {
    // ---------------------------------------------------------------- softmax and queries
    const int st = threadIdx.x - 32 * kPgSoft;
    const int sw = warp - kPgSoft, quarter = warp & 3, w2 = sw >> 2;
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16);
    const int part = lane >> 4;
    const int head = 16 * quarter + (lane & 15);  // this thread's head, and its keys: key0 .. key0 + 31 of a tile
    const int key0 = 64 * part + 32 * w2;
    const int h0 = 32 * w2;                       // of O^T: lanes are dims, and this warp takes heads h0 .. h0 + 31
    float* red = reinterpret_cast<float*>(smem + kPgRedOff);
    bool ok = true;

    int n = 0, seg = 0, nt = 0;  // tiles done, rows begun before this one
    float g = qinv_s[head];           // 2^e of the head's query
    // the head's running maximum m of y (a whole number) and sum (two keys side by side); the row they are of
    float m = -INFINITY;
    f32x2 l2 = 0ull;
    int row = 0;
    bool whole = false, head_part = false;
    g = g == g ? 1.f / g : 1.f;
    named_bar_sync(1, 256);  // (the next row's scale goes to the same place)
    for (;; ++seg) {  // (`ok` is the same in all threads of the role)
      const bool more = walk.left > 0;
      if (seg > 0) {
        // --- the sum of the row before: its reciprocal for the value role, which writes the result
        if (!ok || (seg > 1 && !(ok = group_wait(bar(kBarOFree), uint32_t(seg) & 1u)))) break;
        float l, l1;
        f2_unpack(l2, l, l1);
        l += l1;
        l += __shfl_xor_sync(0xffffffffu, l, 16);
        if (part == 0) red[64 * w2 + head] = l;
        named_bar_sync(1, 256);
        if (sw < 4 && part == 0) {  // (l is 0 or NaN where there is no m)
          l = red[head] + red[64 + head];
          linv_s[head] = l == 0.f ? 0.f : 1.f / (l * kPgHalf);
          if (!whole) {
            float* prow = part_out + (long long)(2 * blockIdx.x + (head_part ? 1 : 0)) * kPartFloats + 64 * 512;
            prow[head] = m;
            prow[64 + head] = l;
          } else if (lse) {
            lse[(long long)row * 64 + head] = log_sum(m, l);
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarLFull));
        if (more && !(ok = group_wait(bar(kBarQEmpty), uint32_t(seg - 1) & 1u))) break;
        if (!more) break;
        // --- the query's codes into tensor memory (lane = row of the A operand): 128 dims at a time, through shared memory
        // in two halves of 64, then the rope half into shared memory.  Eight lanes read 128 bytes of a head.
        named_bar_sync(1, 256);
        const float own = qinv_s[head];
        g = own == own ? 1.f / own : 1.f;
        {
          const int hd = 8 * sw + (lane >> 3);  // and hd + 4
          const uint4* src = reinterpret_cast<const uint4*>(q + ((long long)walk.t * 64 + hd) * 576) + (lane & 7);
          const float i0 = qinv_s[hd], i1 = qinv_s[hd + 4];
          const f32x2 inv[2] = {f2_pack(i0, i0), f2_pack(i1, i1)};
          const int own_row = 32 * quarter + lane;
          uint8_t* stage = smem + kPgStageOff;
          uint4 x[4], nx[4];  // dims 128 i .. + 63 of the two heads, then the next 64
#pragma unroll
          for (int k = 0; k < 4; ++k) x[k] = src[8 * (k >> 1) + 288 * (k & 1)];
#pragma unroll 1
          for (int i = 0; i < 4; ++i) {
#pragma unroll
            for (int k = 0; k < 4; ++k) nx[k] = src[min(16 * (i + 1), 56) + 8 * (k >> 1) + 288 * (k & 1)];
            uint2 hi[4], lo[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              split_codes(x[k].x, x[k].y, inv[k & 1], hi[k].x, lo[k].x);
              split_codes(x[k].z, x[k].w, inv[k & 1], hi[k].y, lo[k].y);
            }
#pragma unroll
            for (int d = 0; d < 2; ++d) {
#pragma unroll
              for (int k = 0; k < 2; ++k) {
                const int h = hd + 4 * k, row = 32 * (h >> 4) + (h & 15);
                const int at = 16 * (((lane & 7) >> 1) ^ ((row >> 1) & 3)) + 8 * (lane & 1);  // (of row + 16 too)
                *reinterpret_cast<uint2*>(stage + row * 64 + at) = hi[2 * d + k];
                *reinterpret_cast<uint2*>(stage + (row + 16) * 64 + at) = lo[2 * d + k];
              }
              named_bar_sync(1, 256);
              uint4 c[2];
#pragma unroll
              for (int k = 0; k < 2; ++k)
                c[k] = *reinterpret_cast<const uint4*>(stage + own_row * 64 + 16 * ((2 * w2 + k) ^ ((own_row >> 1) & 3)));
              tmem_st8(lane_addr + kPgQCol + 32 * i + 16 * d + 8 * w2, reinterpret_cast<const uint32_t*>(c));
              named_bar_sync(1, 256);
            }
#pragma unroll
            for (int k = 0; k < 4; ++k) x[k] = nx[k];
          }
          // (the last "next" is dims 448 .. 511 and, 64 further, the rope half)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const int h = hd + 4 * k, row = 32 * (h >> 4) + (h & 15);
            uint8_t* to = smem + kPgQR + row * 128 + (((lane & 7) ^ (row & 7)) << 4);
            *reinterpret_cast<uint4*>(to) = scale_bf16x8(x[2 + k], f2_mul(inv[k], f2_pack(0.5f, 0.5f)));
            *reinterpret_cast<uint4*>(to + 16 * 128) = scale_bf16x8(x[2 + k], f2_mul(inv[k], f2_pack(8.f, 8.f)));
          }
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarQFull));
      }
      nt = walk.segment();
      row = walk.t;
      whole = nt == walk.ntiles;
      head_part = walk.tile == 0;
      walk.advance(nt);
      // --- the next row's scale, while this one's first scores are made: eight heads a warp
      if (walk.left > 0) {
        uint32_t amax[8];
        const uint16_t* qw = q + ((long long)walk.t * 64 + 8 * sw) * 576;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint4 x0 = *reinterpret_cast<const uint4*>(qw + 576 * i + 8 * lane);
          const uint4 x1 = *reinterpret_cast<const uint4*>(qw + 576 * i + 256 + 8 * lane);
          const uint32_t xr = *reinterpret_cast<const uint32_t*>(qw + 576 * i + 512 + 2 * lane);
          amax[i] = __vmaxu2(__vmaxu2(max_abs_bf16(x0), max_abs_bf16(x1)), xr & 0x7fff7fffu);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const uint32_t a = __reduce_max_sync(0xffffffffu, max(amax[i] << 16, amax[i] & 0xffff0000u));
          if (lane == 0) qinv_s[8 * sw + i] = query_scale(a);
        }
      }
      // --- the row's tiles
      const f32x2 g2 = f2_pack(g, g);
      float off = 0.f, most = -INFINITY;  // kPgShift - m, and the x that asks for a new m
      m = -INFINITY;
      l2 = 0ull;
      for (int t = 0; t < nt; ++t, ++n) {
        // Of this head and 32 keys: x = y + off = y - m + kPgShift, y = S log2(e) + k (-inf where there is no key).  k and
        // m are whole numbers, so x takes one rounding, of its own size (before there is an m, off is -k of the tile's
        // first key).  Some x above kPgShift + kPgLazy, or a first maximum: the heads' maxima give a new m.
        if (!(ok = group_wait(bar(kBarSFull), uint32_t(n) & 1u))) break;
        tc_fence_after();
        const float* cs_s = reinterpret_cast<const float*>(keys_of(n)) + 128 + key0;
        if (m == -INFINITY) {
          const float k0 = reinterpret_cast<const float*>(keys_of(n))[256];
          off = k0 > -INFINITY ? -k0 : 0.f;
        }
        const f32x2 off2 = f2_pack(off, off), c16 = f2_pack(0.0625f, 0.0625f);
        f32x2 x[16];
        float top = -INFINITY;
#pragma unroll
        for (int i0 = 0; i0 < 16; i0 += 4) {
          float hi[8], lo[8];
          tmem_ld_halves8x2_sync<64>(lane_addr + h0 + 2 * i0, lane_addr + (16u << 16) + h0 + 2 * i0, hi, lo);
#pragma unroll
          for (int i = 0; i < 4; i += 2) {
            const ulonglong2 cs = *reinterpret_cast<const ulonglong2*>(cs_s + 2 * (i0 + i));
            const ulonglong2 kk = *reinterpret_cast<const ulonglong2*>(cs_s + 128 + 2 * (i0 + i));
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int k = i + e;
              const f32x2 d = f2_fma(f2_pack(lo[2 * k], lo[2 * k + 1]), c16, f2_pack(hi[2 * k], hi[2 * k + 1]));
              x[i0 + k] = f2_fma(d, f2_mul(e ? cs.y : cs.x, g2), f2_add(e ? kk.y : kk.x, off2));
              float a0, a1;
              f2_unpack(x[i0 + k], a0, a1);
              top = fmaxf(top, fmaxf(a0, a1));
            }
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarSFree));
        if (reinterpret_cast<const int*>(keys_of(n))[0] < 0) {  // no key in the tile: whatever the query holds
#pragma unroll
          for (int i = 0; i < 16; ++i) x[i] = f2_pack(-INFINITY, -INFINITY);
          top = -INFINITY;
        }
        int resc = 0;
        if (bar_red_or(1, 256, top > most)) {
          top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 16));
          if (part == 0) red[64 * w2 + head] = top;
          named_bar_sync(1, 256);
          const float mt = floorf(fmaxf(red[head], red[64 + head]) - off);
          // The sum takes 2^(m - mt) in two factors: rows of unlike scales may leave more than fp32's exponents between
          // the maxima, and less between the sums.
          float al = 1.f, al2 = 1.f;
          if (mt > m && (m == -INFINITY || mt >= m + kPgLazy)) {
            const float e = floorf(0.5f * (m - mt));
            al = m == -INFINITY ? 0.f : fast_exp2(e);
            al2 = m == -INFINITY ? 0.f : fast_exp2(m - mt - e);
            const float d = kPgShift - mt - off;
            const f32x2 d2 = f2_pack(d, d);
#pragma unroll
            for (int i = 0; i < 16; ++i) x[i] = f2_add(x[i], d2);
            m = mt;
            off = kPgShift - mt;
            most = kPgShift + kPgLazy;
          }
          l2 = f2_mul(f2_mul(l2, f2_pack(al, al)), f2_pack(al2, al2));
          al *= al2;
          if (sw < 4 && part == 0) alpha_s[head] = al;
          resc = bar_red_or(1, 256, t > 0 && al != 1.f);  // also publishes alpha_s
        }
        // u = 2^x; 2^-24 u rounded to fp16 for the value product; the sum takes it unrounded
        uint32_t w[16];
#pragma unroll
        for (int i0 = 0; i0 < 16; i0 += 2) {
          const ulonglong2 inv = *reinterpret_cast<const ulonglong2*>(cs_s + 256 + 2 * i0);
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            float a0, a1;
            f2_unpack(x[i0 + e], a0, a1);
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            const f32x2 u = f2_pack(a0, a1);
            l2 = f2_fma(u, e ? inv.y : inv.x, l2);
            f2_unpack(f2_mul(u, f2_pack(kPgHalf, kPgHalf)), a0, a1);
            const __half2 p = __floats2half2_rn(a0, a1);
            w[i0 + e] = *reinterpret_cast<const uint32_t*>(&p);
          }
        }
        // P and O are free once the previous value product is done
        if (t > 0 && !(ok = group_wait(bar(kBarPFree), uint32_t(n - 1) & 1u))) break;
        if (resc) {
          tc_fence_after();
          // O^T (lane = dim, column = head) *= alpha[head], where a head of these 16 asks for it
          const uint32_t ask = __ballot_sync(0xffffffffu, alpha_s[h0 + lane] != 1.f);
#pragma unroll 1
          for (int hh = 0; hh < 32; hh += 16) {
            if (!((ask >> hh) & 0xffffu)) continue;
#pragma unroll 1
            for (int mm = 0; mm < 4; ++mm) {
              float ov[16];
              const uint32_t a = lane_addr + kPgOCol + 64 * mm + h0 + hh;
              tmem_ld16_sync(a, ov);
#pragma unroll
              for (int h = 0; h < 16; ++h) ov[h] *= alpha_s[h0 + hh + h];
              tmem_st16(a, ov);
            }
          }
          tmem_wait_st();
        }
        uint8_t* prow = smem + kPgP + part * 8192 + head * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *reinterpret_cast<uint4*>(prow + (((4 * w2 + i) ^ (head & 7)) << 4)) =
              make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(bar(kBarRowEmpty + n % kPgRows));
          mbar_arrive(bar(kBarPFull));
        }
      }
    }
    if (!ok && st == 0) raise_status(kStatusTimeout);
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPgMma) {
    __syncwarp();
    tmem_dealloc(*tmem_slot, 512);
  }
}

// Rows split over CTAs: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M - 24) l_i.  The row that CTA c of the
// attention ended inside: its own partial result 1, then partial result 0 of the CTAs behind it.  Every block lists the
// split rows; a warp takes 128 dims of one head of one of them at a time, with eight partial results in flight.
constexpr int kMergeThreads = 256;
__global__ void __launch_bounds__(kMergeThreads) paged_mla_merge_kernel(const int2* __restrict__ meta, int ctas,
                                                                        const float* __restrict__ part,
                                                                        __nv_bfloat16* __restrict__ o_lat,
                                                                        float* __restrict__ lse) {
  __shared__ int3 list[kPgMaxGrid];  // CTA, row, parts
  __shared__ int warp_count[kMergeThreads / 32];
  pdl_wait();
  pdl_trigger();
  static_assert(kPgMaxGrid <= kMergeThreads, "a thread looks at one CTA");
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int2 mine = int(threadIdx.x) < ctas ? meta[threadIdx.x] : make_int2(-1, 0);
  const uint32_t votes = __ballot_sync(0xffffffffu, mine.x >= 0);
  if (lane == 0) warp_count[warp] = __popc(votes);
  __syncthreads();
  int before = 0, rows = 0;
#pragma unroll
  for (int w = 0; w < kMergeThreads / 32; ++w) {
    before += w < warp ? warp_count[w] : 0;
    rows += warp_count[w];
  }
  if (mine.x >= 0) list[before + __popc(votes & ((1u << lane) - 1u))] = make_int3(threadIdx.x, mine.x, mine.y);
  __syncthreads();
  for (int u = blockIdx.x * (kMergeThreads / 32) + warp; u < rows * 256; u += gridDim.x * (kMergeThreads / 32)) {
    const int h = (u >> 2) & 63, d = 128 * (u & 3) + 4 * lane;
    const int3 sp = list[u >> 8];
    const int parts = sp.z;
    auto at = [&](int i) { return part + (long long)(i == 0 ? 2 * sp.x + 1 : 2 * (sp.x + i)) * kPartFloats; };
    // lane i holds the weight of part i0 + i (0 behind the last); the parts' own loads do not wait for it
    float4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const float4*>(at(min(k, parts - 1)) + h * 512 + d);
    float m = -INFINITY, l = 0.f;
    if (lane < parts) {
      m = at(lane)[64 * 512 + h];
      l = at(lane)[64 * 512 + 64 + h];
    }
    float M = m;
    for (int i = 32 + lane; i < parts; i += 32) M = fmaxf(M, at(i)[64 * 512 + h]);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
    const float M0 = M == -INFINITY ? 0.f : M;
    float den = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < parts; i0 += 32) {
      const bool has = i0 + lane < parts;
      if (i0 > 0 && has) {
        m = at(i0 + lane)[64 * 512 + h];
        l = at(i0 + lane)[64 * 512 + 64 + h];
      }
      const float w = has ? fast_exp2(m - M0) : 0.f;
      const float e = floorf(0.5f * (m - M0));  // (in two factors: 2^(m - M0) may pass fp32's exponents where l makes up for it)
      den += !has ? 0.f : m == -INFINITY ? w * l : l * fast_exp2(e) * fast_exp2(m - M0 - e);
      const int n = min(32, parts - i0);
      for (int j = 0; j < n; j += 8) {
        if (i0 + j > 0) {
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = *reinterpret_cast<const float4*>(at(i0 + min(j + k, n - 1)) + h * 512 + d);
        }
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float wk = __shfl_sync(0xffffffffu, w, (j + k) & 31);
          if (j + k < n) {
            acc.x = fmaf(wk, x[k].x, acc.x);
            acc.y = fmaf(wk, x[k].y, acc.y);
            acc.z = fmaf(wk, x[k].z, acc.z);
            acc.w = fmaf(wk, x[k].w, acc.w);
          }
        }
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) den += __shfl_xor_sync(0xffffffffu, den, o);
    const float inv = den == 0.f ? 0.f : 1.f / (den * kPgHalf);
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc.x * inv, acc.y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc.z * inv, acc.w * inv);
    *reinterpret_cast<uint2*>(o_lat + ((long long)sp.y * 64 + h) * 512 + d) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
    if (lse && (u & 3) == 0 && lane == 0)
      lse[(long long)sp.y * 64 + h] = log_sum(M0, den);
  }
}

}  // namespace

// Room for every CTA's two partial results, behind the CTAs' split rows.
inline int paged_mla_grid(int T, int64_t max_keys, int sm_count) {
  const int64_t tiles = int64_t(T) * ((std::min<int64_t>(max_keys, INT32_MAX) + 127) / 128);  // (a length is an int32)
  const int64_t most = sm_count < kPgMaxGrid ? sm_count : kPgMaxGrid;
  return int(tiles < most ? tiles : most);
}
constexpr size_t kPgMetaBytes = (kPgMaxGrid * sizeof(int2) + 255) / 256 * 256;
inline size_t paged_mla_ws_bytes(int T, int64_t max_keys) {
  return kPgMetaBytes + size_t(2 * paged_mla_grid(T, max_keys, kPgMaxGrid)) * kPartFloats * 4;
}

cudaError_t prepare_paged_mla() {
  static_assert(kPgSmemAlloc <= 232448, "paged MLA shared memory exceeds the per-CTA limit");
  for (auto* kernel : {paged_mla_kernel<false, false>, paged_mla_kernel<false, true>, paged_mla_kernel<true, false>,
                       paged_mla_kernel<true, true>}) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmemAlloc);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

cudaError_t launch_paged_mla(const PagedMlaLaunch& p) {
  const int64_t max_keys = p.idx ? p.topk : int64_t(p.cache.max_pages) * p.cache.page_size;
  const unsigned grid = unsigned(paged_mla_grid(p.T, max_keys, p.sm_count));
  int2* meta = static_cast<int2*>(p.ws);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kPgMetaBytes);
  auto* o = reinterpret_cast<__nv_bfloat16*>(p.o_lat);
  const bool brief = p.wait_ns < kPgBriefNs;
  auto* kernel = p.idx ? (brief ? paged_mla_kernel<true, true> : paged_mla_kernel<true, false>)
                       : (brief ? paged_mla_kernel<false, true> : paged_mla_kernel<false, false>);
  cudaError_t e = launch_pdl(kernel, dim3(grid), dim3(kPgThreads), kPgSmemAlloc, p.stream, 1, p.q, p.T, p.cu_q, p.seq_len,
                             p.idx, p.topk, p.cache, p.scale * 1.4426950408889634f, o, p.lse, meta, part,
                             WaitLimit{p.wait_ns});
  if (e != cudaSuccess || grid == 1) return e;
  // at most one split row per CTA, 32 blocks' worth of warps each
  const unsigned blocks = grid * 32u < 4u * unsigned(p.sm_count) ? grid * 32u : 4u * unsigned(p.sm_count);
  return launch_pdl(paged_mla_merge_kernel, dim3(blocks), dim3(kMergeThreads), 0, p.stream, 1, meta, int(grid), part, o,
                    p.lse);
}

}  // namespace dsa
