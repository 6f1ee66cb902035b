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
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kApThreads = 256;
constexpr int kApRows = 4;  // most rows of a CTA

// A sequence's rows [s0, s1) that are none of a call's T rows (no rows: anywhere).
__device__ __forceinline__ bool wrong_rows(int s0, int s1, int T) { return s0 != s1 && (s0 < 0 || s1 < s0 || s1 > T); }

// Row t's sequence: the last b with start[b] <= t, or -1.  With `wrong` rows
// somewhere the starts need not rise: the last right sequence that has t.
__device__ __forceinline__ int seq_of(const int* start, int n, int t, int T, bool wrong) {
  if (wrong) {
    for (int b = n - 1; b >= 0; --b)
      if (!wrong_rows(start[b], start[b + 1], T) && start[b] <= t && t < start[b + 1]) return b;
    return -1;
  }
  int lo = 0, hi = n + 1;  // start[lo - 1] <= t < start[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1 < n ? lo - 1 : -1;
}

// Two floats, and two correctly rounded operations at a time.
typedef unsigned long long f2;
__device__ __forceinline__ f2 make_f2(float x, float y) {
  f2 p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ f2 unpack2(uint32_t w) { return make_f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u)); }
__device__ __forceinline__ uint32_t pack2(f2 p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return pack_bf16(x, y);
}
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}

__device__ __forceinline__ uint32_t& word(uint4& v, int i) { return reinterpret_cast<uint32_t*>(&v)[i]; }

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
template <bool VEC>
__global__ void __launch_bounds__(kApThreads) k_paged_append(const __grid_constant__ PagedAppendArgs a) {
  constexpr int U = 2;
  __shared__ int s_start[kPagedMaxSeqs + 1];
  __shared__ int s_pos[kApRows];
  __shared__ long long s_slot[kApRows];  // element of head 0, dim 0 of the row's slot, or -1
  __shared__ __align__(16) float s_cos[kApRows][64], s_sin[kApRows][64];
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
          if (turns && u < nqu + P.nkv) {
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
        const bool live = u < units, turn = u < nqu + P.nkv && e0 < a.rd;
        const uint16_t* src = source(t, live ? u : 0);
        uint4 w = *reinterpret_cast<const uint4*>(src + e0);
        float partner[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int d = e0 + i;
          partner[i] = turn && d < a.rd ? bf16_bits_to_float(src[d < half ? d + half : d - half]) : 0.f;
        }
        __syncwarp();  // every lane has read its head
        if (turn) {
          float z[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            const int d = e0 + i, j = d < half ? d : d - half;
            const uint32_t pair = word(w, i >> 1);
            z[i] = (i & 1) ? __uint_as_float(pair & 0xFFFF0000u) : __uint_as_float(pair << 16);
            if (d < a.rd) {
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
  return (a.rd / 2) % 8 == 0 ? run(k_paged_append<true>, prepare_kernel<k_paged_append<true>>(0))
                             : run(k_paged_append<false>, prepare_kernel<k_paged_append<false>>(0));
}

}  // namespace moe
