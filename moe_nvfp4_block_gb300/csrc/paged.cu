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
// only arithmetic that counts, so a CTA takes whole rows.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kApThreads = 256;
constexpr int kApRows = 4;  // most rows of a CTA

// Row t's sequence: the last b with start[b] <= t, or -1.
__device__ __forceinline__ int seq_of(const int* start, int n, int t) {
  int lo = 0, hi = n + 1;  // start[lo - 1] <= t < start[hi]
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= t) lo = mid + 1;
    else hi = mid;
  }
  return lo - 1 < n ? lo - 1 : -1;
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float unpack(const uint4& v, int i) {
  const uint32_t w = i < 4 ? (i < 2 ? v.x : v.y) : (i < 6 ? v.z : v.w);
  return (i & 1) ? __uint_as_float(w & 0xFFFF0000u) : __uint_as_float(w << 16);
}

}  // namespace

// CTA j: rows [rows j, rows (j + 1)).  The CTA copies the row starts, finds
// its rows' sequences and slots, takes the angles' sines and cosines (thread
// per pair), then walks its rows' heads, 16 lanes a head, 16 bytes a lane,
// four heads in flight; the first four are loaded before anything else is
// known, and a lane's sines and cosines are read once a row (one head at a
// time, its angles element by element: 74 us against 55 for 8061 rows of 64
// heads).
// VEC: rd / 2 is a multiple of 8, so a piece's partner is one whole piece of
// the same head (a shuffle); else each element's partner is loaded.
template <bool VEC>
__global__ void __launch_bounds__(kApThreads) k_paged_append(const __grid_constant__ PagedAppendArgs a) {
  constexpr int U = 4;
  __shared__ int s_start[kPagedMaxSeqs + 1];
  __shared__ int s_pos[kApRows];
  __shared__ long long s_slot[kApRows];  // element of head 0, dim 0 of the row's slot, or -1
  __shared__ float s_cos[kApRows][64], s_sin[kApRows][64];
  const PagedRows& P = a.p;
  const int t0 = blockIdx.x * a.rows, ps = 1 << P.lps;
  const int nqu = a.q ? a.nq : 0, units = nqu + 2 * P.nkv;
  const int lane16 = threadIdx.x & 15, d0 = 8 * lane16, h0 = threadIdx.x >> 4;
  constexpr int HS = kApThreads / 16;  // heads side by side
  // this thread's piece of head u0 + k HS + h0: where it is read at row t0
  const uint16_t* src[U];
  uint4 x[U];
  auto place = [&](int u0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + k * HS + h0;
      src[k] = (u < nqu ? a.q + t0 * a.qs + u * 128
                : u < nqu + P.nkv ? a.k + t0 * a.ks + (u - nqu) * 128 : a.v + t0 * a.vs + (u - nqu - P.nkv) * 128) + d0;
    }
  };
  auto load = [&](int t, int u0) {
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + k * HS + h0;
      x[k] = make_uint4(0u, 0u, 0u, 0u);
      if (t < P.T && u < units) x[k] = *reinterpret_cast<const uint4*>(src[k]);
    }
  };
  pdl_wait();
  pdl_launch_dependents();
  place(0);
  load(t0, 0);
  for (int i = threadIdx.x; i <= P.n_seqs; i += kApThreads) s_start[i] = P.start[i];
  __syncthreads();
  if (threadIdx.x < a.rows) {
    const int t = t0 + threadIdx.x;
    const int b = t < P.T ? seq_of(s_start, P.n_seqs, t) : -1;
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
  const int half = a.rd >> 1;
  for (int i = threadIdx.x; i < a.rows * half; i += kApThreads) {
    const int r = i / half, j = i - r * half;
    if (s_pos[r] >= 0) rope_cs(s_pos[r], a.freq[j], s_cos[r][j], s_sin[r][j]);
  }
  __syncthreads();
  // the lane's eight angles: dims d0 .. d0 + 7 are pairs j0 .. j0 + 7, with
  // the sine's sign by the half they lie in (VEC: a lane is in one half)
  const int j0 = d0 < half ? d0 : d0 - half;
  const bool turns = VEC && d0 < a.rd;
  for (int u0 = 0; u0 < units; u0 += U * HS) {
    if (u0 > 0) place(u0);
    for (int r = 0; r < a.rows; ++r) {
      const int t = t0 + r;
      if (s_pos[r] >= 0) {  // else no sequence's row
        if (r > 0 || u0 > 0) load(t, u0);
        const long long slot = s_slot[r];
        float c8[8], s8[8];
        if (turns) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            c8[i] = s_cos[r][j0 + i];
            s8[i] = d0 < half ? -s_sin[r][j0 + i] : s_sin[r][j0 + i];
          }
        }
#pragma unroll
        for (int k = 0; k < U; ++k) {
          const int u = u0 + k * HS + h0;
          const bool isq = u < nqu, isk = !isq && u < nqu + P.nkv, live = u < units;
          if (VEC) {
            const int hl = half >> 3;  // lanes of half the rotary width
            const int from = (threadIdx.x & 16) | (lane16 < hl ? lane16 + hl : lane16 < 2 * hl ? lane16 - hl : lane16);
            uint4 o;
            o.x = __shfl_sync(0xffffffffu, x[k].x, from);
            o.y = __shfl_sync(0xffffffffu, x[k].y, from);
            o.z = __shfl_sync(0xffffffffu, x[k].z, from);
            o.w = __shfl_sync(0xffffffffu, x[k].w, from);
            if (turns && (isq || isk)) {
              float z[8];
#pragma unroll
              for (int i = 0; i < 8; ++i)
                z[i] = __fadd_rn(__fmul_rn(unpack(x[k], i), c8[i]), __fmul_rn(unpack(o, i), s8[i]));
              x[k] = make_uint4(pack2(z[0], z[1]), pack2(z[2], z[3]), pack2(z[4], z[5]), pack2(z[6], z[7]));
            }
          } else {
            const bool turn = live && (isq || isk) && d0 < a.rd;
            float y[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const int d = d0 + i;
              y[i] = turn && d < a.rd ? bf16_bits_to_float(src[k][d < half ? i + half : i - half]) : 0.f;
            }
            __syncwarp();  // q_out may be q: every lane has read its head
            if (turn) {
              float z[8];
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                const int d = d0 + i, j = d < half ? d : d - half;
                z[i] = unpack(x[k], i);
                if (d < a.rd) {
                  const float xc = __fmul_rn(z[i], s_cos[r][j]), ys = __fmul_rn(y[i], s_sin[r][j]);
                  z[i] = d < half ? __fsub_rn(xc, ys) : __fadd_rn(xc, ys);
                }
              }
              x[k] = make_uint4(pack2(z[0], z[1]), pack2(z[2], z[3]), pack2(z[4], z[5]), pack2(z[6], z[7]));
            }
          }
          if (!live) continue;
          const int h = isq ? u : isk ? u - nqu : u - nqu - P.nkv;
          uint16_t* dst = isq ? a.qo + t * a.qos + h * 128
                          : slot >= 0 ? (isk ? P.kp : P.vp) + slot + ((long long)h << P.lps) * 128 : nullptr;
          if (dst) *reinterpret_cast<uint4*>(dst + d0) = x[k];
        }
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int u = u0 + k * HS + h0;
        src[k] += u < nqu ? a.qs : u < nqu + P.nkv ? a.ks : a.vs;
      }
    }
  }
}

cudaError_t launch_paged_append(const PagedAppendArgs& a0, cudaStream_t s) {
  PagedAppendArgs a = a0;
  a.rows = a.p.T >= kApRows * 2 * num_sms() ? kApRows : 1;
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
