// lmhead_logits.cu -- the lm_head's logits of 1 to 16 rows, bit for bit those
// of the argmax kernels: lane l of a warp owns elements 256 j + 8 l + i and
// accumulates them in element order, the 32 lane sums are added in xor rounds
// 16, 8, 4, 2, 1.
//
// What bounds it: that order leaves the products to the FP32 units (K H V
// multiply-adds at 128 an SM and clock: 131 us at K 16, H 2048, V 151,936,
// where the weights' own bytes take 92, and it takes 212; at K 8 it takes 125,
// at K 16, H 1024 and V 32,003 31, where the products take 14).  So the other
// instructions have to be few:
//  * a warp takes eight vocab rows and two rows of x at a time: one
//    fma.rn.f32x2 (two correctly rounded multiply-adds, so the same bits) per
//    pair of rows, with the weight in both halves; x, its rows' bf16 side by
//    side in a word, is unpacked once for eight rows (four rows and half as
//    many registers, twelve warps: 262 us; rows apart: 233);
//  * eight warps hold the sums of 16 or 12 rows, twelve those of 8 or 4 (K 8: 144 us with
//    eight; ten, uneven over the four schedulers, 151; an earlier form);
//  * slots of 512 columns (of 256: 287 us), counted without divisions (221 and
//    235 us, an earlier form);
//  * the xor rounds of 32 (row, vocab) sums together: in each round a lane
//    hands over the half of its sums that its partner keeps, 31 shuffles for
//    32 sums instead of 160 (a + b = b + a, so again the same bits), and lane
//    b ends with sum b.
// Each warp streams its own weights through two 8 KB slots (one bulk copy a
// row) and waits for no other warp.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kLlSlots = 2;
constexpr int kLlRows = 8;      // vocab rows of a warp's step
constexpr int kLlCols = 512;    // columns of a slot
constexpr int kLlSlotBytes = kLlRows * kLlCols * 2;
constexpr uint64_t kLlDrainNs = 2000000000ull;

// The warps of an SM, by the registers of their KR x kLlRows sums.
__host__ __device__ constexpr int ll_warps(int KR) { return KR <= 8 ? 12 : 8; }

struct LlTable {
  uint64_t full[12][kLlSlots];
  int abort;
};

__device__ __forceinline__ unsigned long long ll_pair(float lo, float hi) {
  unsigned long long p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(lo), "f"(hi));
  return p;
}

__device__ __forceinline__ void ll_fma2(unsigned long long& d, unsigned long long a, unsigned long long b) {
  asm("fma.rn.f32x2 %0, %1, %2, %0;" : "+l"(d) : "l"(a), "l"(b));
}

__device__ __forceinline__ float ll_el(const uint4& v, int i) {
  const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
  return (i & 1) ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}

// The xor-round sums of 32 values: lane b returns the sum of v[b].
__device__ __forceinline__ float ll_reduce32(float (&v)[32], int lane) {
#pragma unroll
  for (int d = 16; d >= 1; d >>= 1) {
    const bool up = lane & d;
#pragma unroll
    for (int k = 0; k < d; ++k) {
      const float keep = up ? v[k + d] : v[k], give = up ? v[k] : v[k + d];
      v[k] = __fadd_rn(keep, __shfl_xor_sync(0xffffffffu, give, d));
    }
  }
  return v[0];
}

}  // namespace

template <int KR>
__global__ void __launch_bounds__(ll_warps(KR) * 32, 1) k_lmhead_logits(const __grid_constant__ LmHeadArgs a) {
  constexpr int kLlWarps = ll_warps(KR);
  extern __shared__ __align__(128) unsigned char smem[];
  const int K = a.K, H = a.H, V = a.V;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  unsigned char* ring = smem + (size_t)warp * kLlSlots * kLlSlotBytes;
  uint4* xs = reinterpret_cast<uint4*>(smem + (size_t)kLlWarps * kLlSlots * kLlSlotBytes);  // [KR][H] bf16
  LlTable& T = *reinterpret_cast<LlTable*>(reinterpret_cast<unsigned char*>(xs) + (size_t)KR * H * 2);
  const int nblk = (H + kLlCols - 1) / kLlCols;
  const int ngrp = (V + kLlRows - 1) / kLlRows, step = gridDim.x * kLlWarps;
  const int g0 = warp * gridDim.x + blockIdx.x;  // this warp's groups of rows: g0, g0 + step, ...
  const int nst = g0 < ngrp ? ((ngrp - 1 - g0) / step + 1) * nblk : 0;
  volatile int* abort = &T.abort;
  // stage s: column block s % nblk of the group g0 + (s / nblk) step, asked for
  // in order, by the whole warp, a row a lane
  const uint64_t pol = policy_evict_first();
  int grp = g0, c0 = 0;
  auto issue = [&](int s) {
    const uint32_t bytes = (uint32_t)min(kLlCols, H - c0) * 2u;
    const int nr = min(kLlRows, V - grp * kLlRows);
    uint64_t* bar = &T.full[warp][s % kLlSlots];
    if (lane == 0) mbar_arrive_expect_tx(bar, bytes * nr);
    __syncwarp();
    if (lane < nr)
      bulk_load(ring + (size_t)(s % kLlSlots) * kLlSlotBytes + lane * (kLlCols * 2),
                a.W + (size_t)(grp * kLlRows + lane) * H + c0, bytes, bar, pol);
    if ((c0 += kLlCols) >= H) {
      c0 = 0;
      grp += step;
    }
  };
  if (lane == 0) {
    for (int i = 0; i < kLlSlots; ++i) mbar_init(&T.full[warp][i], 1);
    if (warp == 0) T.abort = 0;
    fence_mbar_init();
  }
  __syncthreads();
  for (int s = 0; s < min(nst, kLlSlots); ++s) issue(s);
  pdl_launch_dependents();
  // x in planes [pair of rows][256 columns][first or second half of a lane's
  // eight][lane][4 words {row 2p, row 2p + 1}]: a warp's 16-byte reads are consecutive
  for (int i = threadIdx.x; i < KR / 2 * H / 8; i += blockDim.x) {
    const int p = i / (H / 8), c = i - p * (H / 8);
    const uint4 z = make_uint4(0u, 0u, 0u, 0u);
    const uint4* x = reinterpret_cast<const uint4*>(a.x) + (size_t)2 * p * (H / 8) + c;
    const uint4 u = 2 * p < K ? __ldcg(x) : z, v = 2 * p + 1 < K ? __ldcg(x + H / 8) : z;
    uint4* at = xs + (size_t)(i >> 5) * 64 + (i & 31);
    at[0] = make_uint4(__byte_perm(u.x, v.x, 0x5410), __byte_perm(u.x, v.x, 0x7632), __byte_perm(u.y, v.y, 0x5410),
                       __byte_perm(u.y, v.y, 0x7632));
    at[32] = make_uint4(__byte_perm(u.z, v.z, 0x5410), __byte_perm(u.z, v.z, 0x7632), __byte_perm(u.w, v.w, 0x5410),
                        __byte_perm(u.w, v.w, 0x7632));
  }
  __syncthreads();

  unsigned long long acc[kLlRows][KR / 2];  // {row 2p, row 2p + 1} of vocab row q
  int s = 0, blk = 0, v0 = g0 * kLlRows;
  for (; s < nst; ++s) {
    bool ok = !*abort && mbar_wait_bounded(&T.full[warp][s % kLlSlots], (uint32_t)(s / kLlSlots) & 1u, a.wait_ns, abort);
    if (!__all_sync(0xffffffffu, ok)) {
      *abort = 1;
      break;
    }
    if (blk == 0) {
#pragma unroll
      for (int q = 0; q < kLlRows; ++q)
#pragma unroll
        for (int p = 0; p < KR / 2; ++p) acc[q][p] = 0ull;
    }
    const uint4* ws = reinterpret_cast<const uint4*>(ring + (size_t)(s % kLlSlots) * kLlSlotBytes);
    const int nj = min(kLlCols, H - blk * kLlCols) / 256;
#pragma unroll 1
    for (int j = 0; j < nj; ++j) {
      uint4 w[kLlRows];
#pragma unroll
      for (int q = 0; q < kLlRows; ++q) w[q] = ws[q * (kLlCols / 8) + j * 32 + lane];
      const uint4* xj = xs + (blk * (kLlCols / 256) + j) * 64 + lane;
#pragma unroll
      for (int hf = 0; hf < 2; ++hf) {  // elements 0-3, 4-7 of the lane's eight
        unsigned long long ww[kLlRows][4];
#pragma unroll
        for (int q = 0; q < kLlRows; ++q)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float f = ll_el(w[q], 4 * hf + i);
            ww[q][i] = ll_pair(f, f);
          }
#pragma unroll
        for (int p = 0; p < KR / 2; ++p) {
          const uint4 x = xj[p * (H / 4) + 32 * hf];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t u = i == 0 ? x.x : i == 1 ? x.y : i == 2 ? x.z : x.w;
            const unsigned long long xx = ll_pair(__uint_as_float(u << 16), __uint_as_float(u & 0xFFFF0000u));
#pragma unroll
            for (int q = 0; q < kLlRows; ++q) ll_fma2(acc[q][p], ww[q][i], xx);
          }
        }
      }
    }
    __syncwarp();
    if (s + kLlSlots < nst) issue(s + kLlSlots);
    if (++blk < nblk) continue;
    blk = 0;
    // sums b = q + kLlRows r of 32 / kLlRows rows of x at a time, one a lane
    constexpr int RB = 32 / kLlRows;
#pragma unroll
    for (int h = 0; h < KR / RB; ++h) {
      float v[32];
#pragma unroll
      for (int b = 0; b < 32; ++b) {
        const int r = RB * h + b / kLlRows;
        float lo, hi;
        asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(acc[b % kLlRows][r >> 1]));
        v[b] = (r & 1) ? hi : lo;
      }
      const float l = ll_reduce32(v, lane);
      const int r = RB * h + lane / kLlRows, q = lane % kLlRows;
      if (r < K && v0 + q < V) a.logits[(size_t)r * V + v0 + q] = l;
    }
    v0 += step * kLlRows;
  }
  if (*abort && s < nst) {
    // this warp's copies still in flight (those of stage s on) land before it leaves
    if (lane == 0) {
      for (int i = s; i < min(nst, s + kLlSlots); ++i)
        mbar_wait_drain(&T.full[warp][i % kLlSlots], (uint32_t)(i / kLlSlots) & 1u, kLlDrainNs);
      if (a.err) atomicCAS(a.err, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
    }
  }
}

template <int KR>
static cudaError_t launch_lmhead_logits_t(const LmHeadArgs& a, cudaStream_t s) {
  constexpr int kLlWarps = ll_warps(KR);
  const size_t sm = (size_t)kLlWarps * kLlSlots * kLlSlotBytes + (size_t)KR * a.H * 2 + sizeof(LlTable);
  constexpr int most = kLlWarps * kLlSlots * kLlSlotBytes + KR * 2048 * 2 + (int)sizeof(LlTable);
  const cudaError_t e = prepare_kernel<k_lmhead_logits<KR>>(most);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms());
  cfg.blockDim = dim3(kLlWarps * 32);
  cfg.dynamicSmemBytes = sm;
  cfg.stream = s;
  // an ordinary launch: the weights are read before the dependency wait
  return cudaLaunchKernelEx(&cfg, k_lmhead_logits<KR>, a);
}

// Rows are padded to 4, 8, 12 (172 us where 16 take 207) or 16.  Up to 4 the weights' bytes bound it, and K 1
// takes what K 4 takes: 97 and 100 us at H 2048, V 151,936 (92 at the copy's
// bandwidth), 15 at H 1024, V 32,003 (10).
cudaError_t launch_lmhead_logits(const LmHeadArgs& a, cudaStream_t s) {
  return a.K <= 4   ? launch_lmhead_logits_t<4>(a, s)
         : a.K <= 8  ? launch_lmhead_logits_t<8>(a, s)
         : a.K <= 12 ? launch_lmhead_logits_t<12>(a, s)
                     : launch_lmhead_logits_t<16>(a, s);
}

}  // namespace moe
