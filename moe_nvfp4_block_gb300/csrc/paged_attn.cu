// paged_attn.cu -- attention of verify rows over a paged KV cache.
//
// For row t of sequence b (position pos = kv_len[b] + i) and query head h:
//   s_p = score(q . k_p),  o = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m)
// over the visible positions p, in one pass with a running maximum m.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;

// The score of q . k = x at distance dist = p - pos, times log2 e.
// tanh(z) = 1 - 2 / (e^2z + 1): its error is absolute (one FP32 rounding of
// 1), which is what a score needs.
__device__ __forceinline__ float score_log2(const PagedAttnArgs& a, float x, float slope, int dist) {
  float s = x * a.scale;
  if (a.softcap > 0.f) s = a.softcap * (1.f - 2.f / (exp2f(2.f * kLog2e * (s / a.softcap)) + 1.f));
  return (s + slope * (float)dist) * kLog2e;
}

}  // namespace

// CTA (row t, head h): four warps take every fourth position, a lane four
// dims; the warps' (m, l, o) are merged in shared memory.
__global__ void __launch_bounds__(128) k_paged_attn_rows(const __grid_constant__ PagedAttnArgs a) {
  __shared__ float s_m[4], s_l[4], s_o[4][128];
  const PagedRows& P = a.p;
  pdl_wait();
  pdl_launch_dependents();
  const int t = blockIdx.y, h = blockIdx.x, kvh = h / a.group;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  int b = -1;
  for (int i = 0; i < P.n_seqs; ++i)
    if (P.start[i] <= t && t < P.start[i + 1]) b = i;
  if (b < 0) return;
  const int r0 = P.start[b], n = P.start[b + 1] - r0, len = P.kv_len[b];
  int e = 0;
  if (r0 < 0 || n > a.max_rows || P.start[b + 1] > P.T || len < 0) e = MOE_ERR_INVALID_ARG;
  else if ((long long)len + n > (long long)P.max_pages << P.lps) e = MOE_ERR_CAPACITY;
  if (e) {
    if (threadIdx.x == 0) atomicCAS(P.err, 0, e);
    return;
  }
  const int pos = len + t - r0;
  const int first = a.first ? min(max(0, a.first[b]), pos + 1) : 0, prefix = a.prefix ? a.prefix[b] : 0;
  const uint2 qv = *reinterpret_cast<const uint2*>(a.q + t * a.qs + h * 128 + 4 * lane);
  const float q0 = bf16_bits_to_float(qv.x & 0xffff), q1 = __uint_as_float(qv.x & 0xffff0000u);
  const float q2 = bf16_bits_to_float(qv.y & 0xffff), q3 = __uint_as_float(qv.y & 0xffff0000u);
  const float slope = a.slopes ? a.slopes[h] : 0.f;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int p = first + warp; p <= pos; p += 4) {
    if (a.window > 0 && p <= pos - a.window && p >= prefix) continue;
    int page = P.table[(size_t)b * P.max_pages + (p >> P.lps)];
    if (page < 0 || page >= P.n_pages) {
      if (lane == 0) atomicCAS(P.err, 0, (int)MOE_ERR_INVALID_ARG);
      page = 0;
    }
    const size_t at = ((((size_t)page * P.nkv + kvh) << P.lps) + (p & ((1 << P.lps) - 1))) * 128 + 4 * lane;
    const uint2 kk = *reinterpret_cast<const uint2*>(P.kp + at);
    const uint2 vv = *reinterpret_cast<const uint2*>(P.vp + at);
    float x = q0 * bf16_bits_to_float(kk.x & 0xffff) + q1 * __uint_as_float(kk.x & 0xffff0000u) +
              q2 * bf16_bits_to_float(kk.y & 0xffff) + q3 * __uint_as_float(kk.y & 0xffff0000u);
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x += __shfl_xor_sync(0xffffffffu, x, d);
    const float s = score_log2(a, x, slope, p - pos);
    const float mx = fmaxf(m, s), ref = mx == -INFINITY ? 0.f : mx;
    const float al = exp2f(m - ref), w = exp2f(s - ref);
    m = mx;
    l = l * al + w;
    o[0] = o[0] * al + w * bf16_bits_to_float(vv.x & 0xffff);
    o[1] = o[1] * al + w * __uint_as_float(vv.x & 0xffff0000u);
    o[2] = o[2] * al + w * bf16_bits_to_float(vv.y & 0xffff);
    o[3] = o[3] * al + w * __uint_as_float(vv.y & 0xffff0000u);
  }
  if (lane == 0) {
    s_m[warp] = m;
    s_l[warp] = l;
  }
  for (int i = 0; i < 4; ++i) s_o[warp][4 * lane + i] = o[i];
  __syncthreads();
  const float M = fmaxf(fmaxf(s_m[0], s_m[1]), fmaxf(s_m[2], s_m[3])), ref = M == -INFINITY ? 0.f : M;
  float L = 0.f, O = 0.f;
  for (int w = 0; w < 4; ++w) {
    const float f = exp2f(s_m[w] - ref);
    L += s_l[w] * f;
    O += s_o[w][threadIdx.x] * f;
  }
  a.o[t * a.os + h * 128 + threadIdx.x] = float_to_bf16_bits(L == 0.f ? 0.f : O / L);
  if (threadIdx.x == 0 && a.lse) a.lse[(size_t)t * a.nq + h] = L == 0.f ? -INFINITY : (ref + log2f(L)) * 0.6931471805599453f;
}

cudaError_t launch_paged_attention(const PagedAttnArgs& a, cudaStream_t s) {
  max_carveout(k_paged_attn_rows);
  k_paged_attn_rows<<<dim3(a.nq, a.p.T), 128, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace moe
