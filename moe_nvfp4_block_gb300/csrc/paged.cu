// paged.cu -- the append of verify rows to a paged KV cache, with the rotary
// embedding of their queries and keys.
//
// Row t of a call belongs to the sequence b with start[b] <= t < start[b + 1]
// and has position p = kv_len[b] + (t - start[b]).  With the pair (x, y) =
// (dims i, i + rd / 2) of a head and the angle a = p * freq[i]:
//   x' = x cos a - y sin a,   y' = y cos a + x sin a.
// The rotated key and the value go to slot p % page_size of page
// table[b][p / page_size], the rotated query to q_out.
//
// What bounds it: (nq + 2 nkv) * 512 bytes read and written a row; the angles'
// double-precision reduction (rd / 2 a row, shared by the row's heads) is the
// only arithmetic that counts, so a CTA takes whole rows.  8061 rows of 64
// heads with 64 rotary dims: 56 us, 4.8 TB/s read and written; 5967 rows of 10
// heads with 128: 17 us where the bytes take 5, the angles' doubles the rest.
#include "internal.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kApThreads = 256;
constexpr int kApRows = 4;  // most rows of a CTA

}  // namespace

// CTA j: rows [rows j, rows (j + 1)): one, or as many as leave one wave, up to 4
// (1696 rows of 20 heads: 7.6 us where a CTA a row takes 9.9).  The CTA copies the row starts, finds
// its rows' sequences and slots, takes the angles' sines and cosines (thread
// per pair), then walks its rows' heads.
// VEC (rd / 2 a multiple of 8): eight lanes a head, each with two 16-byte
// pieces.  The first rd / 16 lanes have a piece of the first half of the
// rotary dims and its partner in the second, so a pair's four products need no
// other lane and its sines and cosines serve both; the other lanes pass two
// pieces on.  Two heads a lane are in flight, the first two from before
// anything else is known.  The arithmetic is 3 instructions an element (one
// piece a lane, its partner by shuffles, one float at a time: 12, which bound
// the kernel: 74 us against 56 for 8061 rows of 64 heads).  With 16 heads or
// fewer a CTA works on two or four rows side by side (5967 rows of 10: 16 us
// against 21 for one after another).
// Else: 16 lanes a head, each element's partner loaded.
// NORM: the queries and keys of each head are divided by the root of their mean
// square (over the head's lanes by shuffles) and multiplied by the gain (in
// shared memory: in registers, 16 dims a lane, fewer CTAs fit), before they turn;
// all in FP32.  8247 rows of 80 heads: 85 us, 4.0 TB/s read and written (a step's
// two heads are used as soon as loaded: waits for loads are the first stall, then
// instructions, 53% of the issue slots); 160 verify rows of 48 heads 4.5 us.
// Widths whose half is no multiple of 8 cost twice: 8240 rows of 64 heads with 60
// rotary dims 117 us, with 64 57 (norms: 118, 63).
template <bool VEC, bool NORM>
__global__ void __launch_bounds__(kApThreads, NORM ? 4 : 0) k_paged_append(const __grid_constant__ PagedAppendArgs a) {
  constexpr int U = 2;
  __shared__ int s_start[kPagedMaxSeqs + 1];
  __shared__ int s_pos[kApRows];
  __shared__ long long s_slot[kApRows];  // element of head 0, dim 0 of the row's slot, or -1
  __shared__ __align__(16) float s_cos[kApRows][64], s_sin[kApRows][64];
  __shared__ uint4 s_gain[NORM ? 32 : 1];  // of the queries, of the keys
  const PagedRows& P = a.p;
  const int t0 = blockIdx.x * a.rows, ps = 1 << P.lps;
  const int nqu = a.q ? a.nq : 0, units = nqu + 2 * P.nkv, half = a.rd >> 1;
  // VEC: this lane's pieces of a head, and whether they turn
  constexpr int HS = kApThreads / (VEC ? 8 : 16);  // heads side by side: G of a row, HS / G rows
  const int G = !VEC || units > 16 ? HS : units > 8 ? 16 : 8;
  const int hl = half >> 3, l8 = threadIdx.x & 7, hs = threadIdx.x / (VEC ? 8 : 16), h0 = hs & (G - 1), r0 = hs / G;
  const bool turns = VEC && l8 < hl;
  const int d0 = 8 * (turns ? l8 : 2 * l8), d1 = turns ? d0 + half : d0 + 8;
  auto source = [&](int t, int u) {
    return u < nqu ? a.q + t * a.qs + u * 128
           : u < nqu + P.nkv ? a.k + t * a.ks + (u - nqu) * 128 : a.v + t * a.vs + (u - nqu - P.nkv) * 128;
  };
  uint4 x[U], y[U];
  auto load = [&](int t, int u0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + k * G + h0;
      if (t >= P.T || u >= units) continue;
      const uint16_t* src = source(t, u);
      x[k] = *reinterpret_cast<const uint4*>(src + d0);
      y[k] = *reinterpret_cast<const uint4*>(src + d1);
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  if (VEC && r0 < a.rows) load(t0 + r0, 0);
  if (NORM && threadIdx.x < 32) {
    const uint16_t* g = threadIdx.x < 16 ? a.qg : a.kg;
    s_gain[threadIdx.x] = g ? reinterpret_cast<const uint4*>(g)[threadIdx.x & 15]
                            : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  }
  bool wrong = false;
  for (int i = threadIdx.x; i <= P.n_seqs; i += kApThreads) {
    const int s0 = P.start[i], s1 = P.start[min(i + 1, P.n_seqs)];
    s_start[i] = s0;
    wrong |= wrong_rows(s0, s1, P.T);
  }
  wrong = __syncthreads_or(wrong);
  if (wrong && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(P.err, 0, (int)MOE_ERR_INVALID_ARG);
  if (threadIdx.x < a.rows) {
    const int t = t0 + threadIdx.x;
    const int b = t < P.T ? seq_of(s_start, P.n_seqs, t, P.T, wrong) : -1;
    long long slot = -1;
    int pos = -1;
    if (b >= 0) {
      const int len = P.kv_len[b];
      const long long p = (long long)len + (t - s_start[b]);
      int e = 0;
      if (len < 0) {
        e = MOE_ERR_INVALID_ARG;
      } else if (p >= (long long)P.max_pages << P.lps) {
        e = MOE_ERR_CAPACITY;
      } else {
        const int page = P.table[(size_t)b * P.max_pages + (size_t)(p >> P.lps)];
        if (page < 0 || page >= P.n_pages) e = MOE_ERR_INVALID_ARG;
        else slot = (((long long)page * P.nkv << P.lps) + (p & (ps - 1))) * 128;
      }
      if (e) atomicCAS(P.err, 0, e);
      pos = (int)(p < 0 ? 0 : p > 0x7fffffff ? 0x7fffffff : p);
    }
    s_pos[threadIdx.x] = pos;
    s_slot[threadIdx.x] = slot;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < a.rows * half; i += kApThreads) {
    const int r = i / half, j = i - r * half;
    if (s_pos[r] >= 0) rope_cs(s_pos[r], a.freq[j], s_cos[r][j], s_sin[r][j]);
  }
  __syncthreads();
  for (int r = r0; r < a.rows; r += HS / G) {
    const int t = t0 + r;
    if (s_pos[r] < 0) continue;  // no sequence's row
    const long long slot = s_slot[r];
    auto target = [&](int u) {
      const bool isk = u < nqu + P.nkv;
      return u < nqu ? a.qo + t * a.qos + u * 128
             : slot >= 0 ? (isk ? P.kp : P.vp) + slot + ((long long)(u - nqu - (isk ? 0 : P.nkv)) << P.lps) * 128 : nullptr;
    };
    if constexpr (VEC) {
      f2 c2[4], s2[4], n2[4];  // cosines, sines, minus the sines of dims d0 .. d0 + 7
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = *reinterpret_cast<const float2*>(&s_cos[r][d0 + 2 * i]);
          const float2 s = *reinterpret_cast<const float2*>(&s_sin[r][d0 + 2 * i]);
          c2[i] = make_f2(c.x, c.y);
          s2[i] = make_f2(s.x, s.y);
          n2[i] = make_f2(-s.x, -s.y);
        }
      }
      for (int u0 = 0; u0 < units; u0 += U * G) {
        if (r > r0 || u0 > 0) load(t, u0);
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int u = u0 + k * G + h0;
          if (u >= units) continue;
          if constexpr (NORM) {
            if (u < nqu + P.nkv) {  // (the eight lanes of a head take the same way)
              const unsigned lanes = 0xFFu << (threadIdx.x & 24);
              f2 ss = make_f2(0.f, 0.f);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const f2 lo = unpack2(word(x[k], i)), hi = unpack2(word(y[k], i));
                ss = fma2(hi, hi, fma2(lo, lo, ss));
              }
              float sq = sum2(ss);
              sq += __shfl_xor_sync(lanes, sq, 1);
              sq += __shfl_xor_sync(lanes, sq, 2);
              sq += __shfl_xor_sync(lanes, sq, 4);
              const float inv = inv_sqrt(__fmaf_rn(sq, 1.f / 128.f, a.eps));
              const f2 inv2 = make_f2(inv, inv);
              const uint4* gain = s_gain + (u < nqu ? 0 : 16);
              uint4 g[2] = {gain[d0 >> 3], gain[d1 >> 3]};
              f2 lo[4], hi[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                lo[i] = mul2(mul2(unpack2(word(x[k], i)), inv2), unpack2(word(g[0], i)));
                hi[i] = mul2(mul2(unpack2(word(y[k], i)), inv2), unpack2(word(g[1], i)));
              }
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                word(x[k], i) = pack2(turns ? add2(mul2(lo[i], c2[i]), mul2(hi[i], n2[i])) : lo[i]);
                word(y[k], i) = pack2(turns ? add2(mul2(hi[i], c2[i]), mul2(lo[i], s2[i])) : hi[i]);
              }
            }
          } else if (turns && u < nqu + P.nkv) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f2 lo = unpack2(word(x[k], i)), hi = unpack2(word(y[k], i));
              word(x[k], i) = pack2(add2(mul2(lo, c2[i]), mul2(hi, n2[i])));
              word(y[k], i) = pack2(add2(mul2(hi, c2[i]), mul2(lo, s2[i])));
            }
          }
          uint16_t* dst = target(u);
          if (dst) {
            *reinterpret_cast<uint4*>(dst + d0) = x[k];
            *reinterpret_cast<uint4*>(dst + d1) = y[k];
          }
        }
      }
    } else {
      for (int u0 = 0; u0 < units; u0 += HS) {  // a warp's lanes stay together: q_out may be q
        const int u = u0 + h0, e0 = 8 * (threadIdx.x & 15);
        const bool live = u < units, turn = u < nqu + P.nkv && e0 < a.rd, normed = NORM && u < nqu + P.nkv;
        const uint16_t* src = source(t, live ? u : 0);
        uint4 w = *reinterpret_cast<const uint4*>(src + e0);
        float partner[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = e0 + i;
          partner[i] = turn && d < a.rd ? bf16_bits_to_float(src[d < half ? d + half : d - half]) : 0.f;
        }
        __syncwarp();  // every lane has read its head
        float inv = 1.f;
        if constexpr (NORM) {
          float sq = 0.f;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float lo = __uint_as_float(word(w, i) << 16), hi = __uint_as_float(word(w, i) & 0xFFFF0000u);
            sq = __fmaf_rn(hi, hi, __fmaf_rn(lo, lo, sq));
          }
#pragma unroll
          for (int d = 1; d < 16; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
          inv = inv_sqrt(__fmaf_rn(sq, 1.f / 128.f, a.eps));
        }
        if (turn || normed) {
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = e0 + i, j = d < half ? d : d - half;
            const uint32_t pair = word(w, i >> 1);
            z[i] = (i & 1) ? __uint_as_float(pair & 0xFFFF0000u) : __uint_as_float(pair << 16);
            if constexpr (NORM) {
              const uint32_t gw = reinterpret_cast<const uint32_t*>(s_gain + (u < nqu ? 0 : 16))[4 * (threadIdx.x & 15) + (i >> 1)];
              z[i] = __fmul_rn(__fmul_rn(z[i], inv), (i & 1) ? __uint_as_float(gw & 0xFFFF0000u) : __uint_as_float(gw << 16));
              if (d < a.rd) {
                const uint16_t* g = reinterpret_cast<const uint16_t*>(s_gain + (u < nqu ? 0 : 16));
                partner[i] = __fmul_rn(__fmul_rn(partner[i], inv), bf16_bits_to_float(g[d < half ? d + half : d - half]));
              }
            }
            if (turn && d < a.rd) {
              const float xc = __fmul_rn(z[i], s_cos[r][j]), ys = __fmul_rn(partner[i], s_sin[r][j]);
              z[i] = d < half ? __fsub_rn(xc, ys) : __fadd_rn(xc, ys);
            }
          }
          w = make_uint4(pack_bf16(z[0], z[1]), pack_bf16(z[2], z[3]), pack_bf16(z[4], z[5]), pack_bf16(z[6], z[7]));
        }
        uint16_t* dst = live ? target(u) : nullptr;
        if (dst) *reinterpret_cast<uint4*>(dst + e0) = w;
      }
    }
  }
}

cudaError_t launch_paged_append(const PagedAppendArgs& a0, cudaStream_t s) {
  PagedAppendArgs a = a0;
  const int wave = 4 * num_sms();
  a.rows = a.p.T >= kApRows * wave ? kApRows : (a.p.T + wave - 1) / wave;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.p.T + a.rows - 1) / a.rows);
  cfg.blockDim = dim3(kApThreads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern, cudaError_t e) { return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, a) : e; };
  const bool vec = (a.rd / 2) % 8 == 0;
  if (a.norm)
    return vec ? run(k_paged_append<true, true>, prepare_kernel<k_paged_append<true, true>>(0))
               : run(k_paged_append<false, true>, prepare_kernel<k_paged_append<false, true>>(0));
  return vec ? run(k_paged_append<true, false>, prepare_kernel<k_paged_append<true, false>>(0))
             : run(k_paged_append<false, false>, prepare_kernel<k_paged_append<false, false>>(0));
}

}  // namespace moe
