// Latent attention of new tokens over the paged 8-bit cache (paged_cache.cuh).
//
//   S[h,s]   = scale 2^k_s (q_lat[h] . code_s + q_rope[h] . rope_s)
//   o_lat[h] = sum_s softmax_s(S[h,:]) 2^k_s code_s,   lse[h] = log sum_s exp S[h,s]
//
// over every position the token sees, or over its selected positions.
//
// Scores straight from the codes.  The query of a head is split once into
// q = 2^e (hi + lo / 16), both e4m3 (4 + 4 significant bits: exact for values
// within 2^5 of the head's largest, never off by more than 2^-22 of it), so
// the 8-bit tensor path multiplies the cache's codes as they lie in memory:
// N = 128 columns, 64 of hi and 64 of lo.  The rope half follows in bf16 into
// the hi columns.  2^k_s, 2^e and the scale are applied to the fp32 sums.
//
// Values as fp16.  A code is exact in fp16, and a probability rounded to fp16
// (2^-11) is eight times closer than one in bf16.  The row's 2^k goes into the
// probability: with y = S log2(e) + k_s, u_s = 2^(y - m + 6) where m follows
// the running maximum of y in whole numbers, so u is at most 2^14 (see kLazyRescale) and what
// fp16 cannot hold is 2^-31 of the largest; sum u code is the numerator,
// sum u 2^-k_s (fp32, u before rounding) the denominator.
//
// One CTA walks an equal share of all 128-key tiles of the batch, query row
// after query row; a row that ends in another CTA leaves partial sums that
// paged_mla_merge_kernel joins.  16 warps:
//  * warp 3 finds each key's cache row and 2^k, up to four tiles ahead;
//  * warps 0 and 1 copy the tile's rows (four chunks of 128 codes, then
//    the rope chunk) into a ring of 16 KB slots, 128 bytes of 128 keys each, with cp.async;
//  * warps 4..7 read the codes again (they are in L2 by then), widen them to
//    fp16 and store them for the value product: two slots of 128 keys x 128
//    dims; at the start of a query row they prepare the query;
//  * warps 8..15 are the softmax, two groups of 32 heads: a thread owns a key;
//  * warp 2 issues S^T = K Q^T (M = 128 keys) one tile ahead of
//    O^T += V^T P^T (M = 128 dims x 4, N = 64 heads).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "internal.h"
#include "paged_cache.cuh"
#include "ptx.cuh"
#include "sparse_mla.cuh"

namespace dsa {

namespace {

constexpr int kPgThreads = 512;
constexpr int kPgMma = 2, kPgAddr = 3, kPgVWarp = 4, kPgSoft = 8;  // first warp of each role (keys: 0)
constexpr int kPgRegs = 128;  // registers a thread at launch; then by warpgroup:
constexpr int kPgRegs0 = 72, kPgRegsV = 136, kPgRegsS = 152;
static_assert(kPgThreads * kPgRegs <= 65536 && 128 * (kPgRegs0 + kPgRegsV + 2 * kPgRegsS) <= kPgThreads * kPgRegs,
              "the warpgroups' registers must not exceed the block's");
constexpr int kPgSlot = 16384;        // 128 keys x 128 bytes, 128B-swizzled
constexpr int kPgKSlots = 4;
constexpr int kPgVSlots = 2;
constexpr int kPgRows = 4;            // tiles whose row numbers are held
constexpr int kPgMaxGrid = 160;       // CTAs at most (the workspace is sized for it)
constexpr float kPgShift = 6.f;       // log2 of the probability at the running maximum
constexpr float kPgNone = 1e30f;      // shift of a head without a maximum yet: any finite score sets one

constexpr int kPgQ8 = 0;                                     // 4 chunks of 128 rows (hi heads, lo heads) x 128 codes
constexpr int kPgQR = kPgQ8 + 4 * kPgSlot;                   // 64 heads x 64 bf16
constexpr int kPgP = kPgQR + 8192;                           // 128 keys x 64 heads fp16
constexpr int kPgK = kPgP + kPgSlot;
constexpr int kPgV = kPgK + kPgKSlots * kPgSlot;             // a slot: two chunks of 128 keys x 64 dims fp16
constexpr int kPgRowOff = kPgV + kPgVSlots * 2 * kPgSlot;    // int row[kPgRows][128]
constexpr int kPgScaleOff = kPgRowOff + kPgRows * 512;       // float 2^k[kPgRows][128]
constexpr int kPgRedOff = kPgScaleOff + kPgRows * 512;       // float red[2][4][32]
constexpr int kPgMOff = kPgRedOff + 1024;                    // float m[64], alpha[64], l[64], 2^e[2][64], kPgShift - m [64]
constexpr int kPgBarOff = kPgMOff + 1536;
enum PgBar {
  kBarQFull, kBarQEmpty, kBarPFull, kBarPFree, kBarOFree, kBarCodes, kBarDrain, kBarSFull,  // s_full x2
  kBarKFull = kBarSFull + 2, kBarKEmpty = kBarKFull + kPgKSlots, kBarVFull = kBarKEmpty + kPgKSlots,
  kBarVEmpty = kBarVFull + kPgVSlots, kBarRowFull = kBarVEmpty + kPgVSlots, kBarRowEmpty = kBarRowFull + kPgRows,
  kPgBars = kBarRowEmpty + kPgRows
};
constexpr int kPgTailOff = kPgBarOff + 8 * kPgBars;          // tmem address, abort flag, start (b, t, tile), share
constexpr int kPgSmem = kPgTailOff + 64;
constexpr int kPgSmemAlloc = kPgSmem + 1024;
constexpr uint32_t kPgOCol = 256;                            // S^T: two buffers of 128 columns; O^T: 4 x 64

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

// sum of ceil(i / 128) over i = 1 .. n
__device__ __forceinline__ long long tiles_below(long long n) {
  const long long q = n >> 7, r = n & 127;
  return 64 * q * (q + 1) + r * (q + 1);
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
    ntiles = topk_tiles ? topk_tiles : max(1, (seen + 127) >> 7);
  }
  __device__ __forceinline__ void start(const int* at) {
    b = at[0];
    t = at[1];
    tile = at[2];
    left = at[3];
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

// Tiles of the first j query rows of a sequence with nq rows and length len (len < 0: a bad one, rows that see nothing).
__device__ __forceinline__ long long tiles_of(int nq, long long len, int topk_tiles, int j) {
  if (topk_tiles) return (long long)j * topk_tiles;
  if (len < 0) return j;
  const long long base = len - nq;                    // positions before the first query row
  const long long none = min((long long)j, max(0ll, -base));  // rows that see nothing: one (empty) tile each
  return none + tiles_below(max(0ll, base + j)) - tiles_below(max(0ll, base));
}

// Lane L of the warp gets the reduction of v[L % 16] over the 32 lanes.
template <bool kMax>
__device__ __forceinline__ float reduce_scatter16(float (&v)[16]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int w = 8; w >= 1; w >>= 1) {
#pragma unroll
    for (int i = 0; i < w; ++i) {
      const float mine = (lane & w) ? v[w + i] : v[i], give = (lane & w) ? v[i] : v[w + i];
      const float got = __shfl_xor_sync(0xffffffffu, give, w);
      v[i] = kMax ? fmaxf(mine, got) : mine + got;
    }
  }
  const float got = __shfl_xor_sync(0xffffffffu, v[0], 16);
  return kMax ? fmaxf(v[0], got) : v[0] + got;
}

// Codes 16 g .. 16 g + 15 (+ col) of a thread's eight keys; zeros where there is no key.
__device__ __forceinline__ void load_codes(uint4 (&w)[8], const int (&y)[8], const uint8_t* base, int col) {
#pragma unroll
  for (int j = 0; j < 8; ++j)
    w[j] = y[j] >= 0 ? *reinterpret_cast<const uint4*>(base + (long long)y[j] * kRow8 + col) : make_uint4(0, 0, 0, 0);
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

template <bool kSparse>
__global__ void __launch_bounds__(kPgThreads, 1)
    paged_mla_kernel(const uint16_t* __restrict__ q, int T, const int32_t* __restrict__ cu_q,
                     const int32_t* __restrict__ seq_len, const int32_t* __restrict__ idx, int topk,
                     const __grid_constant__ PagedCache c, float scale_log2, __nv_bfloat16* __restrict__ o_lat,
                     float* __restrict__ lse, int2* __restrict__ meta, float* __restrict__ part, WaitLimit lim) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const uint32_t sbase = smem_u32(smem);
  auto bar = [&](int i) { return sbase + kPgBarOff + 8u * i; };
  int* row_s = reinterpret_cast<int*>(smem + kPgRowOff);
  float* scale_s = reinterpret_cast<float*>(smem + kPgScaleOff);
  float* m_s = reinterpret_cast<float*>(smem + kPgMOff);
  float* alpha_s = m_s + 64;
  float* l_s = m_s + 128;
  float* g_s = m_s + 192;  // two rows' worth: the next row's query is prepared while this one's scores are still read
  float* off_s = m_s + 320;  // what a score is shifted by before 2^x: kPgShift - m, kPgNone before there is an m
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + kPgTailOff);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + kPgTailOff + 4);
  int* start_s = reinterpret_cast<int*>(smem + kPgTailOff + 8);  // b, t, tile, tiles of this CTA, tiles of a share
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int topk_tiles = kSparse ? (topk + 127) >> 7 : 0;

  if (threadIdx.x == 0) {
    mbar_init(bar(kBarQFull), 128);
    mbar_init(bar(kBarQEmpty), 1);
    mbar_init(bar(kBarPFull), 256);
    mbar_init(bar(kBarPFree), 1);
    mbar_init(bar(kBarOFree), 256);
    mbar_init(bar(kBarCodes), 1);
    mbar_init(bar(kBarDrain), 1);
    for (int i = 0; i < 2; ++i) mbar_init(bar(kBarSFull + i), 1);
    for (int i = 0; i < kPgKSlots; ++i) {
      mbar_init(bar(kBarKFull + i), 64);
      mbar_init(bar(kBarKEmpty + i), 1);
    }
    for (int i = 0; i < kPgVSlots; ++i) {
      mbar_init(bar(kBarVFull + i), 128);
      mbar_init(bar(kBarVEmpty + i), 1);
    }
    for (int i = 0; i < kPgRows; ++i) {
      mbar_init(bar(kBarRowFull + i), 1);
      mbar_init(bar(kBarRowEmpty + i), 14);  // one per warp of the key, value and softmax roles
    }
    *abort_flag = 0;
    start_s[3] = 0;
    fence_mbar_init();
  }
  if (warp == kPgMma) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  pdl_wait();

  // ---------------------------------------------------------------- this CTA's share
  {
    long long* sums = reinterpret_cast<long long*>(smem);  // the warps' sums, in the query's room
    const int per = (c.batch + kPgThreads - 1) / kPgThreads;
    const int b0 = min(int(threadIdx.x) * per, c.batch), b1 = min(b0 + per, c.batch);
    auto weight = [&](int b, int& q0, int& nq, long long& len, bool report) {
      nq = seq_rows(cu_q, T, b, q0, report);
      len = seq_len[b];
      if (len < 0 || len > max_positions(c)) len = -1;
      if (report && nq > 0 && len < nq) raise_status(kStatusBadRow);
      return tiles_of(nq, len, topk_tiles, nq);
    };
    int q0, nq;
    long long len, mine = 0;
    for (int b = b0; b < b1; ++b) mine += weight(b, q0, nq, len, blockIdx.x == 0);
    long long incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long up = __shfl_up_sync(0xffffffffu, incl, o);
      if (lane >= o) incl += up;
    }
    if (lane == 31) sums[warp] = incl;
    __syncthreads();
    long long before = 0, total = 0;
    for (int w = 0; w < kPgThreads / 32; ++w) {
      if (w < warp) before += sums[w];
      total += sums[w];
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x;
    const long long g0 = share * blockIdx.x, g1 = min(g0 + share, total);
    long long at = before + incl - mine;
    if (g0 < g1 && g0 >= at && g0 < at + mine) {
      for (int b = b0;; ++b) {
        const long long w = weight(b, q0, nq, len, false);
        if (g0 < at + w) {
          int lo = 0, hi = nq;  // the last row j with tiles_of(j) <= g0 - at
          while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (tiles_of(nq, len, topk_tiles, mid) <= g0 - at) lo = mid;
            else hi = mid;
          }
          start_s[0] = b;
          start_s[1] = q0 + lo;
          start_s[2] = int(g0 - at - tiles_of(nq, len, topk_tiles, lo));
          start_s[3] = int(g1 - g0);
          start_s[4] = int(share);
          break;
        }
        at += w;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  TileWalk walk{c, cu_q, seq_len, T, topk_tiles, 0, 0, 0, 0, 0, 0, 0};
  const bool busy = start_s[3] > 0;
  if (busy) walk.start(start_s);
  else if (threadIdx.x == 0) meta[blockIdx.x] = make_int2(-1, 0);

  if (!busy) {
    // nothing to do
  } else if (warp < kPgVWarp) {
    reg_dec<kPgRegs0>();
    if (warp < kPgMma) {
      // ---------------------------------------------------------------- keys
      const int g = threadIdx.x & 7, r0 = threadIdx.x >> 3;  // segment g of rows r0 + 8 j
      const uint32_t off = uint32_t(r0 * 128 + ((g ^ r0) << 4));
      const uint8_t* base = c.kv8 + 16 * g;
      int slot = 0;
      uint32_t sphase = 0;
      bool ok = true;
      for (int n = 0; n < walk.left && ok; ++n) {
        const int rb = n % kPgRows;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(kBarRowFull + rb), uint32_t(n / kPgRows) & 1u, lim, abort_flag));
        if (!ok) break;
        int y[16];
#pragma unroll
        for (int j = 0; j < 16; ++j) y[j] = row_s[rb * 128 + r0 + 8 * j];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarRowEmpty + rb));
        for (int ch = 0; ch < 5; ++ch) {
          if (!(ok = mbar_wait(bar(kBarKEmpty + slot), sphase ^ 1u, lim, abort_flag))) break;
          const uint32_t dst = sbase + kPgK + slot * kPgSlot + off;
#pragma unroll
          for (int j = 0; j < 16; ++j)
            cp_async_16_or_zero(dst + j * 1024, base + (long long)max(y[j], 0) * kRow8 + 128 * ch, y[j] < 0);
          cp_async_arrive_noinc(bar(kBarKFull + slot));
          if (++slot == kPgKSlots) {
            slot = 0;
            sphase ^= 1u;
          }
        }
        ok = __all_sync(0xffffffffu, ok);
      }
      cp_async_wait_all();
    } else if (warp == kPgAddr) {
      // ---------------------------------------------------------------- addresses
      // Keys lane + 32 i of each tile.  Position, page and scale are three loads
      // that follow from each other; each is made one tile after the one before it,
      // so that none is waited for.
      const int total = walk.left;
      int s2[4], s1[4], page1[4], row0[4], b2;
      float sc0[4];
      auto position = [&]() {  // of the walk's next tile (-1: none); then step on
        b2 = walk.b;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int j = walk.tile * 128 + lane + 32 * i;
          int s = -1;
          if (walk.left > 0) {
            if (!kSparse) {
              s = j < walk.seen ? j : -1;
            } else if (j < topk) {
              s = idx[(long long)walk.t * topk + j];
              if (s >= walk.seen) {
                raise_status(kStatusBadRow);
                s = -1;
              }
            }
          }
          s2[i] = s;
        }
        if (walk.left > 0) walk.advance(1);
      };
      auto page = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          s1[i] = s2[i];
          page1[i] = s2[i] >= 0 ? c.page_table[(long long)b2 * c.max_pages + int(unsigned(s2[i]) / unsigned(c.page_size))] : 0;
        }
      };
      auto scale = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          int y = -1;
          if (s1[i] >= 0) {
            if (page1[i] >= 0 && page1[i] < c.n_pages) y = page1[i] * c.page_size + int(unsigned(s1[i]) % unsigned(c.page_size));
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
        const bool ok = __all_sync(
            0xffffffffu, mbar_wait(bar(kBarRowEmpty + rb), (uint32_t(n / kPgRows) & 1u) ^ 1u, lim, abort_flag));
        if (!ok) break;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          row_s[rb * 128 + lane + 32 * i] = row0[i];
          scale_s[rb * 128 + lane + 32 * i] = sc0[i];
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarRowFull + rb));
        scale();
        page();
        position();
      }
    } else {
      // ---------------------------------------------------------------- MMA issuer
      {
        const bool el = elect_one();
        const uint32_t idesc_k = idesc_e4m3(128, 128);
        const uint32_t idesc_r = idesc_bf16(128, 64, 0, 0);
        const uint32_t idesc_v = idesc_f16(128, 64, 1, 1);
        int kslot = 0, vslot = 0, n = 0, seg = 0;  // n: the row's first tile
        uint32_t kphase = 0, vphase = 0, cphase = 0;
        bool ok = true;
        auto warp_wait = [&](uint32_t b, uint32_t parity) {
          return __all_sync(0xffffffffu, mbar_wait(b, parity, lim, abort_flag)) != 0;
        };
        auto next_k = [&]() {
          if (el) mma_commit(bar(kBarKEmpty + kslot));
          if (++kslot == kPgKSlots) {
            kslot = 0;
            kphase ^= 1u;
          }
        };
        // S^T of the codes (N = 128, first) into buffer `buf`
        auto codes = [&](int buf) {
          for (int ch = 0; ch < 4; ++ch) {
            if (!(ok = warp_wait(bar(kBarKFull + kslot), kphase))) return;
            fence_proxy_async_smem();
            tc_fence_after();
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (el) mma_f8_ss(tmem + 128 * buf, smem_desc(sbase + kPgK + kslot * kPgSlot + 32 * k, 16, 1024, kSwizzle128B),
                        smem_desc(sbase + kPgQ8 + ch * kPgSlot + 32 * k, 16, 1024, kSwizzle128B), idesc_k,
                        (ch | k) ? 1u : 0u);
            next_k();
          }
          if (el) mma_commit(bar(kBarCodes));
        };
        // ... and of the rope half into the hi columns on top of it.  Only products of one shape and kind are ordered by
        // their issue: a barrier stands between these two (and other work is queued meanwhile).
        auto rope = [&](int buf) {
          if (!(ok = warp_wait(bar(kBarCodes), cphase))) return;
          cphase ^= 1u;
          if (!(ok = warp_wait(bar(kBarKFull + kslot), kphase))) return;
          fence_proxy_async_smem();
          tc_fence_after();
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (el) mma_bf16_ss(tmem + 128 * buf, smem_desc(sbase + kPgK + kslot * kPgSlot + 32 * k, 16, 1024, kSwizzle128B),
                        smem_desc(sbase + kPgQR + 32 * k, 16, 1024, kSwizzle128B), idesc_r, 1u);
          next_k();
          if (el) mma_commit(bar(kBarSFull + buf));
        };
        while (ok && walk.left > 0) {
          const int nt = walk.segment();
          if (!(ok = warp_wait(bar(kBarQFull), uint32_t(seg & 1)))) break;
          codes(n & 1);
          for (int s = 0; s <= nt && ok; ++s) {
            // scores of tile s, codes of tile s + 1, values of tile s - 1
            if (s < nt) {
              rope((n + s) & 1);
              if (!ok) break;
              if (s == nt - 1 && el) mma_commit(bar(kBarQEmpty));
            }
            if (s >= 1 && !(ok = warp_wait(bar(kBarPFull), uint32_t(n + s - 1) & 1u))) break;
            // tile s + 1 takes the buffer of tile s - 1, whose probabilities are there
            if (s + 1 < nt) codes((n + s + 1) & 1);
            if (!ok || s == 0) continue;
            if (s == 1 && seg > 0 && !(ok = warp_wait(bar(kBarOFree), uint32_t(seg - 1) & 1u))) break;
            tc_fence_after();
            for (int m = 0; m < 4; ++m) {
              if (!(ok = warp_wait(bar(kBarVFull + vslot), vphase))) break;
              tc_fence_after();
#pragma unroll
              for (int k = 0; k < 8; ++k)
                if (el)
                  mma_bf16_ss(tmem + kPgOCol + 64 * m,
                            smem_desc(sbase + kPgV + vslot * 2 * kPgSlot + k * 2048, kPgSlot, 1024, kSwizzle128B),
                            smem_desc(sbase + kPgP + k * 2048, kPgSlot, 1024, kSwizzle128B), idesc_v,
                            (s > 1 || k > 0) ? 1u : 0u);
              if (el) mma_commit(bar(kBarVEmpty + vslot));
              if (++vslot == kPgVSlots) {
                vslot = 0;
                vphase ^= 1u;
              }
            }
            if (ok && el) mma_commit(bar(kBarPFree));
          }
          n += nt;
          walk.advance(nt);
          ++seg;
        }
        if (el) mma_commit(bar(kBarDrain));
        mbar_drain(bar(kBarDrain), 0);
      }
      __syncwarp();
    }
  } else if (warp < kPgSoft) {
    reg_inc<kPgRegsV>();
    // ---------------------------------------------------------------- queries and values
    const int vt = threadIdx.x - 32 * kPgVWarp;
    const int vw = warp - kPgVWarp;
    // Codes 16 g .. 16 g + 15 of rows r0 + 16 j: segments 2 (g % 4) and the next of
    // chunk g / 4 of the widened row.  Eight lanes take the first chunk of a row and
    // the second of its neighbour: with the swizzle, their stores fill all banks.
    const int g = vt & 7, r0 = (vt >> 3) ^ (g >> 2);
    const uint32_t voff = uint32_t((g >> 2) * kPgSlot + r0 * 128);
    const uint32_t seg0 = uint32_t(((2 * (g & 3)) ^ (r0 & 7)) << 4), seg1 = seg0 ^ 16u;
    const int total = walk.left;
    int slot = 0, seg = 0, row_tiles = 0;
    uint32_t sphase = 0;
    bool ok = true;
    auto wait = [&](uint32_t b, uint32_t parity) {
      return __all_sync(0xffffffffu, mbar_wait(b, parity, lim, abort_flag)) != 0;
    };
    // The codes of a slot are loaded two slots ahead, across tiles and rows.
    const uint8_t* base = c.kv8 + 16 * g;
    int y[8];
    auto rows = [&](int n) {
      const int rb = n % kPgRows;
      if (!(ok = wait(bar(kBarRowFull + rb), uint32_t(n / kPgRows) & 1u))) return;
#pragma unroll
      for (int j = 0; j < 8; ++j) y[j] = row_s[rb * 128 + r0 + 16 * j];
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(kBarRowEmpty + rb));
    };
    uint4 w0[8], w1[8];
    auto widen = [&](const uint4 (&w)[8]) {  // into the next slot
      if (!wait(bar(kBarVEmpty + slot), sphase ^ 1u)) return false;
      uint8_t* dst = smem + kPgV + slot * 2 * kPgSlot + voff;
#pragma unroll
      for (int j = 0; j < 8; ++j) store_fp16(dst + j * 2048 + seg0, dst + j * 2048 + seg1, w[j]);
      fence_proxy_async_smem();
      mbar_arrive(bar(kBarVFull + slot));
      if (++slot == kPgVSlots) {
        slot = 0;
        sphase ^= 1u;
      }
      return true;
    };
    rows(0);
    if (ok) {
      load_codes(w0, y, base, 0);
      load_codes(w1, y, base, 128);
    }
    for (int n = 0; n < total && ok; ++n) {
      if (row_tiles == 0) {
        // --- the query row: hi and lo codes and the scaled rope half
        if (!(ok = wait(bar(kBarQEmpty), uint32_t(seg & 1) ^ 1u))) break;
#pragma unroll 2
        for (int i = 0; i < 16; ++i) {
          const int h = vw * 16 + i;
          const uint16_t* qh = q + ((long long)walk.t * 64 + h) * 576;
          const uint4 x0 = *reinterpret_cast<const uint4*>(qh + 16 * lane);
          const uint4 x1 = *reinterpret_cast<const uint4*>(qh + 16 * lane + 8);
          const uint32_t xr = *reinterpret_cast<const uint32_t*>(qh + 512 + 2 * lane);
          const uint32_t w[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
          uint32_t amax = 0;
          auto see = [&](uint32_t bits) {
            bits &= 0x7fffffffu;
            if (bits < 0x7f800000u) amax = max(amax, bits);
          };
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            see(w[j] << 16);
            see(w[j] & 0xffff0000u);
          }
          see(xr << 16);
          see(xr & 0xffff0000u);
          amax = __reduce_max_sync(0xffffffffu, amax);
          // 2^e with max |q| <= 448 2^e
          const int e0 = int(amax >> 23) - 135 + ((amax & 0x7fffffu) > 0x600000u ? 1 : 0);
          const int e = max(e0, -100);
          const float inv = pow2f(-e);
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float v[4] = {__uint_as_float(w[2 * j] << 16), __uint_as_float(w[2 * j] & 0xffff0000u),
                          __uint_as_float(w[2 * j + 1] << 16), __uint_as_float(w[2 * j + 1] & 0xffff0000u)};
            uint32_t hh = 0, ll = 0;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              float a = v[2 * p] * inv, bb = v[2 * p + 1] * inv;
              // an infinite value is taken as NaN (codes have no infinity): so is every score with it
              if (isinf(a)) a = __uint_as_float(0x7fc00000u);
              if (isinf(bb)) bb = __uint_as_float(0x7fc00000u);
              const __nv_fp8x2_storage_t c2 = __nv_cvt_float2_to_fp8x2(make_float2(a, bb), __NV_SATFINITE, __NV_E4M3);
              const float2 f = __half22float2(__half2(__nv_cvt_fp8x2_to_halfraw2(c2, __NV_E4M3)));
              const __nv_fp8x2_storage_t d2 =
                  __nv_cvt_float2_to_fp8x2(make_float2((a - f.x) * 16.f, (bb - f.y) * 16.f), __NV_SATFINITE, __NV_E4M3);
              hh |= uint32_t(c2) << (16 * p);
              ll |= uint32_t(d2) << (16 * p);
            }
            hi[j] = hh;
            lo[j] = ll;
          }
          // lane holds codes 16 lane ..: chunk lane / 8, segment lane % 8
          uint8_t* dst = smem + kPgQ8 + (lane >> 3) * kPgSlot + h * 128 + (((lane & 7) ^ (h & 7)) << 4);
          *reinterpret_cast<uint4*>(dst) = make_uint4(hi[0], hi[1], hi[2], hi[3]);
          *reinterpret_cast<uint4*>(dst + 64 * 128) = make_uint4(lo[0], lo[1], lo[2], lo[3]);
          *reinterpret_cast<__nv_bfloat162*>(smem + kPgQR + h * 128 + (((lane >> 2) ^ (h & 7)) << 4) + (lane & 3) * 4) =
              __floats2bfloat162_rn(__uint_as_float(xr << 16) * inv, __uint_as_float(xr & 0xffff0000u) * inv);
          if (lane == 0) g_s[64 * (seg & 1) + h] = pow2f(e);
        }
        fence_proxy_async_smem();
        mbar_arrive(bar(kBarQFull));
        row_tiles = walk.segment();
        walk.advance(row_tiles);
        ++seg;
      }
      --row_tiles;
      if (!(ok = widen(w0))) break;
      load_codes(w0, y, base, 256);
      if (!(ok = widen(w1))) break;
      load_codes(w1, y, base, 384);
      if (!(ok = widen(w0))) break;
      const bool more = n + 1 < total;
      if (more) {
        rows(n + 1);
        if (!ok) break;
        load_codes(w0, y, base, 0);
      }
      if (!(ok = widen(w1))) break;
      if (more) load_codes(w1, y, base, 128);
    }
  } else {
    reg_inc<kPgRegsS>();
    // ---------------------------------------------------------------- softmax
    const int half = (warp - kPgSoft) >> 2;   // heads 32 half .. 32 half + 31
    const int quarter = warp & 3;             // TMEM lanes of this warp
    const int r = quarter * 32 + lane;        // its key of the tile, its dim of O^T
    const int st = threadIdx.x - 32 * (kPgSoft + 4 * half);
    const int bar_id = 1 + half;
    const uint32_t lane_addr = tmem + (uint32_t(quarter * 32) << 16);
    float* red = reinterpret_cast<float*>(smem + kPgRedOff) + half * 128;
    const int h0 = 32 * half;
    auto wait_all = [&](uint32_t b, uint32_t parity) {
      const bool mine = st == 0 ? mbar_wait(b, parity, lim, abort_flag) : true;
      return bar_red_or(bar_id, 128, mine ? 0 : 1) == 0;
    };
    bool ok = true;
    int n = 0, seg = 0;
    int2 split = make_int2(-1, 0);
    while (ok && walk.left > 0) {
      const int nt = walk.segment();
      f32x2 l_acc[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) l_acc[i] = 0ull;
      if (st < 32) {
        m_s[h0 + st] = -INFINITY;
        off_s[h0 + st] = kPgNone;
      }
      for (int t = 0; t < nt && ok; ++t, ++n) {
        // (the barrier in here also publishes m_s; the scores' barrier follows the query's, so 2^e is there too)
        if (!(ok = wait_all(bar(kBarSFull + (n & 1)), uint32_t(n >> 1) & 1u))) break;
        tc_fence_after();
        const int rb = n % kPgRows;
        const bool valid = row_s[rb * 128 + r] >= 0;
        const float sc = scale_s[rb * 128 + r];
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(kBarRowEmpty + rb));
        // Of this key (-inf without one) and 32 heads: x = y - m + kPgShift, y = S log2(e) + k.  k and m are whole
        // numbers, so x takes one rounding, of its own size.  Above kPgShift + kLazyRescale for some head of some key
        // (pass 0): the maxima of y (pass 1) give new m, and x is taken again (pass 2).
        const float cs = sc * scale_log2;
        const float kf = valid ? float(int(__float_as_uint(sc) >> 23) - 127) : -INFINITY;
        const f32x2 cs2 = f2_pack(cs, cs), kf2 = f2_pack(kf, kf), c16 = f2_pack(0.0625f, 0.0625f);
        const uint32_t sa = lane_addr + 128 * (n & 1) + h0;
        const ulonglong2* g4 = reinterpret_cast<const ulonglong2*>(g_s + 64 * (seg & 1) + h0);
        const ulonglong2* off4 = reinterpret_cast<const ulonglong2*>(off_s + h0);
        f32x2 x[16];
        int resc = 0;
#pragma unroll 1
        for (int pass = 0; pass < 3; ++pass) {
          float top = -INFINITY;
#pragma unroll
          for (int i0 = 0; i0 < 16; i0 += 4) {
            float hi[8], lo[8];
            tmem_ld8x2_sync(sa + 2 * i0, sa + 64 + 2 * i0, hi, lo);
#pragma unroll
            for (int i = 0; i < 4; i += 2) {
              const ulonglong2 g = g4[(i0 + i) >> 1];
              ulonglong2 off = off4[(i0 + i) >> 1];
              if (pass == 1) off = make_ulonglong2(0ull, 0ull);
#pragma unroll
              for (int e = 0; e < 2; ++e) {
                const int k = i + e;
                const f32x2 d = f2_fma(f2_pack(lo[2 * k], lo[2 * k + 1]), c16, f2_pack(hi[2 * k], hi[2 * k + 1]));
                x[i0 + k] = f2_fma(d, f2_mul(e ? g.y : g.x, cs2), f2_add(kf2, e ? off.y : off.x));
                float a0, a1;
                f2_unpack(x[i0 + k], a0, a1);
                top = fmaxf(top, fmaxf(a0, a1));
              }
            }
          }
          if (pass == 0 && !bar_red_or(bar_id, 128, top > kPgShift + kLazyRescale ? 1 : 0)) break;
          if (pass == 1) {
#pragma unroll
            for (int i0 = 0; i0 < 16; i0 += 8) {
              float v[16];
#pragma unroll
              for (int i = 0; i < 8; ++i) f2_unpack(x[i0 + i], v[2 * i], v[2 * i + 1]);
              const float mx = reduce_scatter16<true>(v);
              if (lane < 16) red[quarter * 32 + 2 * i0 + lane] = mx;
            }
            named_bar_sync(bar_id, 128);
            int mine = 0;
            if (st < 32) {
              const float mt = floorf(fmaxf(fmaxf(red[st], red[32 + st]), fmaxf(red[64 + st], red[96 + st])));
              const float mu = m_s[h0 + st];
              float al = 1.f;
              if (mt >= mu + kLazyRescale && mt > mu) {
                al = mu == -INFINITY ? 0.f : fast_exp2(mu - mt);
                m_s[h0 + st] = mt;
                off_s[h0 + st] = kPgShift - mt;
                mine = t > 0;
              }
              alpha_s[h0 + st] = al;
            }
            resc = bar_red_or(bar_id, 128, mine);  // also publishes m_s, off_s and alpha_s
          }
        }
        // P and O are free once the previous value product is done
        if (t > 0 && !(ok = wait_all(bar(kBarPFree), uint32_t(n - 1) & 1u))) break;
        if (resc) {
          tc_fence_after();
#pragma unroll 1
          for (int m = 0; m < 4; ++m) {
            float o[32];
            const uint32_t a = lane_addr + kPgOCol + 64 * m + h0;
            tmem_ld32_sync(a, o);
#pragma unroll
            for (int h = 0; h < 32; ++h) o[h] *= alpha_s[h0 + h];
            tmem_st16(a, o);
            tmem_st16(a + 16, o + 16);
          }
          tmem_wait_st();
#pragma unroll
          for (int i = 0; i < 16; ++i) l_acc[i] = f2_mul(l_acc[i], *reinterpret_cast<const f32x2*>(&alpha_s[h0 + 2 * i]));
        }
        // u = 2^x, rounded to fp16 for the value product; the sums take it unrounded
        const float inv = valid ? pow2f(127 - int(__float_as_uint(sc) >> 23)) : 0.f;
        const f32x2 inv2 = f2_pack(inv, inv);
        uint8_t* prow = smem + kPgP + r * 128;
#pragma unroll
        for (int i0 = 0; i0 < 16; i0 += 4) {
          uint32_t w[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            float a0, a1;
            f2_unpack(x[i0 + i], a0, a1);
            a0 = fast_exp2(a0);
            a1 = fast_exp2(a1);
            l_acc[i0 + i] = f2_fma(f2_pack(a0, a1), inv2, l_acc[i0 + i]);
            const __half2 p = __floats2half2_rn(a0, a1);
            w[i] = *reinterpret_cast<const uint32_t*>(&p);
          }
          *reinterpret_cast<uint4*>(prow + ((((h0 >> 3) + (i0 >> 2)) ^ (r & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(kBarPFull));
      }
      if (!ok) break;
      // --- the row's (or the segment's) result
      if (!(ok = wait_all(bar(kBarPFree), uint32_t(n - 1) & 1u))) break;
      tc_fence_after();
#pragma unroll
      for (int i0 = 0; i0 < 16; i0 += 8) {
        float v[16];
#pragma unroll
        for (int i = 0; i < 8; ++i) f2_unpack(l_acc[i0 + i], v[2 * i], v[2 * i + 1]);
        const float l = reduce_scatter16<false>(v);
        if (lane < 16) red[quarter * 32 + 2 * i0 + lane] = l;
      }
      named_bar_sync(bar_id, 128);
      if (st < 32) l_s[h0 + st] = red[st] + red[32 + st] + red[64 + st] + red[96 + st];
      named_bar_sync(bar_id, 128);
      const bool whole = nt == walk.ntiles;
      // a CTA leaves at most two partial results: of the row it starts inside (0) and of the row it ends inside (1)
      float* prow = part + (long long)(2 * blockIdx.x + (walk.tile == 0 ? 1 : 0)) * kPartFloats;
#pragma unroll 1
      for (int m = 0; m < 4; ++m) {
        float o[32];
        tmem_ld32_sync(lane_addr + kPgOCol + 64 * m + h0, o);
        const int d = 128 * m + r;
#pragma unroll
        for (int h = 0; h < 32; ++h) {
          if (whole) {
            const float l = l_s[h0 + h];
            o_lat[((long long)walk.t * 64 + h0 + h) * 512 + d] = __float2bfloat16(l == 0.f ? 0.f : o[h] / l);
          } else {
            prow[(h0 + h) * 512 + d] = o[h];
          }
        }
      }
      tc_fence_before();
      mbar_arrive(bar(kBarOFree));
      if (st < 32) {
        const float l = l_s[h0 + st], m = m_s[h0 + st];  // (l is 0 or NaN where there is no m)
        if (!whole) {
          prow[64 * 512 + h0 + st] = m;
          prow[64 * 512 + 64 + h0 + st] = l;
        } else if (lse) {
          lse[(long long)walk.t * 64 + h0 + st] = l == 0.f ? -INFINITY : (m - kPgShift + log2f(l)) * 0.69314718055994531f;
        }
      }
      if (!whole && walk.tile == 0) {
        const int rest = walk.ntiles - nt, share = start_s[4];
        split = make_int2(walk.t, 1 + (rest + share - 1) / share);
      }
      named_bar_sync(bar_id, 128);  // l_s, m_s are rewritten for the next row
      walk.advance(nt);
      ++seg;
    }
    if (half == 0 && st == 0) meta[blockIdx.x] = ok ? split : make_int2(-1, 0);
  }
  pdl_trigger();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kPgMma) {
    __syncwarp();
    tmem_dealloc(tmem, 512);
  }
}

// Rows split over CTAs: with M = max m_i, o = sum 2^(m_i - M) O_i / sum 2^(m_i - M) l_i.  The row that CTA
// blockIdx.x of the attention ended inside: its own partial result 1, then partial result 0 of the CTAs behind it.
// Grid (attention CTAs, 8): eight heads a block, one per warp.
__global__ void __launch_bounds__(256) paged_mla_merge_kernel(const int2* __restrict__ meta,
                                                              const float* __restrict__ part,
                                                              __nv_bfloat16* __restrict__ o_lat,
                                                              float* __restrict__ lse) {
  pdl_wait();
  pdl_trigger();
  const int2 sp = meta[blockIdx.x];
  if (sp.x < 0) return;
  const int lane = threadIdx.x & 31, h = blockIdx.y * 8 + (threadIdx.x >> 5);
  auto at = [&](int i) {
    return part + (long long)(i == 0 ? 2 * blockIdx.x + 1 : 2 * (blockIdx.x + i)) * kPartFloats;
  };
  float M = -INFINITY;
  for (int i = lane; i < sp.y; i += 32) M = fmax_(M, at(i)[64 * 512 + h]);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmax_(M, __shfl_xor_sync(0xffffffffu, M, o));
  const float M0 = M == -INFINITY ? 0.f : M;
  float den = 0.f;
  float4 acc[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) acc[k] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i = 0; i < sp.y; ++i) {
    const float* p = at(i);
    const float w = fast_exp2(p[64 * 512 + h] - M0);
    den = fmaf(w, p[64 * 512 + 64 + h], den);
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float4 x = *reinterpret_cast<const float4*>(p + h * 512 + 128 * k + 4 * lane);
      acc[k].x = fmaf(w, x.x, acc[k].x);
      acc[k].y = fmaf(w, x.y, acc[k].y);
      acc[k].z = fmaf(w, x.z, acc[k].z);
      acc[k].w = fmaf(w, x.w, acc[k].w);
    }
  }
  const float inv = den == 0.f ? 0.f : 1.f / den;
  __nv_bfloat16* dst = o_lat + ((long long)sp.x * 64 + h) * 512;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const __nv_bfloat162 a = __floats2bfloat162_rn(acc[k].x * inv, acc[k].y * inv);
    const __nv_bfloat162 b = __floats2bfloat162_rn(acc[k].z * inv, acc[k].w * inv);
    *reinterpret_cast<uint2*>(dst + 128 * k + 4 * lane) =
        make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
  }
  if (lse && lane == 0)
    lse[(long long)sp.x * 64 + h] = den == 0.f ? -INFINITY : (M0 - kPgShift + log2f(den)) * 0.69314718055994531f;
}

}  // namespace

// Room for every CTA's two partial results, behind the CTAs' split rows.
inline int paged_mla_grid(int T, int64_t max_keys, int sm_count) {
  const int64_t tiles = int64_t(T) * ((max_keys + 127) / 128);
  const int64_t most = sm_count < kPgMaxGrid ? sm_count : kPgMaxGrid;
  return int(tiles < most ? tiles : most);
}
constexpr size_t kPgMetaBytes = (kPgMaxGrid * sizeof(int2) + 255) / 256 * 256;
inline size_t paged_mla_ws_bytes(int T, int64_t max_keys) {
  return kPgMetaBytes + size_t(2 * paged_mla_grid(T, max_keys, kPgMaxGrid)) * kPartFloats * 4;
}

cudaError_t prepare_paged_mla() {
  static_assert(kPgSmemAlloc <= 232448, "paged MLA shared memory exceeds the per-CTA limit");
  cudaError_t e = cudaFuncSetAttribute(paged_mla_kernel<false>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmemAlloc);
  if (e != cudaSuccess) return e;
  return cudaFuncSetAttribute(paged_mla_kernel<true>, cudaFuncAttributeMaxDynamicSharedMemorySize, kPgSmemAlloc);
}

cudaError_t launch_paged_mla(const PagedMlaLaunch& p) {
  const int64_t max_keys = p.idx ? p.topk : int64_t(p.cache.max_pages) * p.cache.page_size;
  const unsigned grid = unsigned(paged_mla_grid(p.T, max_keys, p.sm_count));
  int2* meta = static_cast<int2*>(p.ws);
  float* part = reinterpret_cast<float*>(static_cast<uint8_t*>(p.ws) + kPgMetaBytes);
  auto* o = reinterpret_cast<__nv_bfloat16*>(p.o_lat);
  cudaError_t e = launch_pdl(p.idx ? paged_mla_kernel<true> : paged_mla_kernel<false>, dim3(grid), dim3(kPgThreads),
                             kPgSmemAlloc, p.stream, 1, p.q, p.T, p.cu_q, p.seq_len, p.idx, p.topk, p.cache,
                             p.scale * 1.4426950408889634f, o, p.lse, meta, part, WaitLimit{p.wait_ns});
  if (e != cudaSuccess || grid == 1) return e;
  return launch_pdl(paged_mla_merge_kernel, dim3(grid, 8), dim3(256), 0, p.stream, 1, meta, part, o, p.lse);
}

}  // namespace dsa
