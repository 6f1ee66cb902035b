// paged8.cu -- the append of rows to a paged KV cache of 8 bits: norms of
// queries and keys for each head, rotary embedding, E4M3 codes and a scale for
// each 16 positions and KV head.
//
// With y = x / sqrt(mean(x^2) + eps) * gain turned as in paged.cu, a block's
// scale is s = 2^e, the smallest with max |y| <= 448 s over the block's new rows
// (and the block's own if it has committed positions and that is more), and a
// code is e4m3(y / s).  A power of two, so that dividing is exact, a scale that
// grows moves the committed codes' exponents only (exact above 2^-6 s), and the
// attention's products can take it in a float's exponent.
//
// What bounds it: nq * 512 + 2 nkv * (256 + 128) bytes a row.  A block's scale
// needs all of its rows, so the unit of work is a block of a sequence: the CTA
// that has its first new row (the leader) takes the block's rows, which may
// reach past the CTA's own.  Its tasks (two queries a lane in flight; a KV head's
// keys or values of the block) are dealt over the warps.  Where a CTA
// has one row, two share its tasks.
//
// Measured: 8247 rows of 48 query and 8 KV heads, normed, 64 rotary dims: 75 us
// (3.4 TB/s read and written): a block's trip is its loads, the norms' sums over
// 16 lanes, its largest value, the codes (38% of the issue slots, waits for
// loads first, 128 registers: two CTAs an SM).  160 verify rows of 64 sequences
// 7.4 us, one row 4.2.  Rotary widths whose half is no multiple of 8 (rows through
// shared memory): 8240 rows with 60 rotary dims 194 us, with 64 80.
#include <cfloat>

#include "internal.h"
#include "paged_rows.cuh"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kA8Threads = 256;
constexpr int kA8Warps = kA8Threads / 32;
constexpr int kA8Block = 16;  // positions of a scale; rows of a CTA at most
constexpr int kA8Rows = 8;    // most rows of a CTA (leaders are looked for among them)
constexpr int kA8Pairs = 2;   // queries of a lane in flight

// A block of a sequence that gets rows: the first of them (the leader) and its
// position; the rows, whose bits `own` are set (all up to n, unless sequences'
// rows overlap); the block's committed positions; the slot (row of 128 codes,
// of head 0) of the leader, or -1.
struct A8Block {
  int t, n, pos, com;
  uint32_t own;
  long long slot;
};

__device__ __forceinline__ uint32_t e4m3_codes(f2 a, f2 b, f2 inv) {
  float x, y, z, w;
  const f2 p = mul2(a, inv), q = mul2(b, inv);
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  asm("mov.b64 {%0, %1}, %2;" : "=f"(z), "=f"(w) : "l"(q));
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(y), "f"(x));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(w), "f"(z));
  return (uint32_t)lo | (uint32_t)hi << 16;
}

// Codes (four) times f, rounded.
__device__ __forceinline__ uint32_t e4m3_times(uint32_t w, float f) {
  uint32_t r = 0;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)(w >> (16 * i))));
    const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&h));
    uint16_t c;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(c) : "f"(v.y * f), "f"(v.x * f));
    r |= (uint32_t)c << (16 * i);
  }
  return r;
}

__device__ __forceinline__ float max2(float m, f2 p) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return fmaxf(m, fmaxf(fabsf(x), fabsf(y)));
}
__device__ __forceinline__ float finite_or(float x, float other) { return fabsf(x) <= FLT_MAX ? x : other; }
__device__ __forceinline__ f2 finite2(f2 p, float other) {
  float x, y;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
  return make_f2(finite_or(x, other), finite_or(y, other));
}

}  // namespace

// CTA j: the blocks whose leaders are rows [rows j, rows (j + 1)).  Eight lanes
// take a head's row, 16 dims each; with VEC (rd / 2 a multiple of 8) a lane that
// turns has eight dims of the first half of the rotary dims and their partners
// in the second, else a row's normed values go through shared memory.
// A warp's four groups of lanes take: queries, four (row, head) pairs; keys and
// values, with one row four heads, two rows two heads, else four rows of one
// head at a time, up to 16 kept in registers until the block's maximum is known.
template <bool VEC, bool NORM>
__global__ void __launch_bounds__(kA8Threads, 2) k_paged_append8(const __grid_constant__ PagedAppend8Args A) {
  const PagedAppendArgs& a = A.a;
  const PagedRows& P = a.p;
  __shared__ int s_start[kPagedMaxSeqs + 1];
  __shared__ A8Block s_block[kA8Block];
  __shared__ int s_n;
  __shared__ uint4 s_gain[32];  // of the queries, of the keys
  __shared__ __align__(16) float s_cos[kA8Block][64], s_sin[kA8Block][64];
  __shared__ __align__(16) float s_head[VEC ? 1 : kA8Warps][4][128];
  const int t0 = blockIdx.x * a.rows, ps = 1 << P.lps, half = a.rd >> 1;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, grp = lane >> 3, l8 = lane & 7;
  const int nqu = a.q ? a.nq : 0;
  const bool turns = VEC && l8 < (half >> 3);
  const int d0 = VEC ? 8 * (turns ? l8 : 2 * l8) : 16 * l8, d1 = turns ? d0 + half : d0 + 8;

  pdl_wait();
  pdl_launch_dependents();
  if (NORM && threadIdx.x < 32) {  // (in registers, 16 more than there are)
    const uint16_t* g = threadIdx.x < 16 ? a.qg : a.kg;
    s_gain[threadIdx.x] = g ? reinterpret_cast<const uint4*>(g)[threadIdx.x & 15]
                            : make_uint4(0x3F803F80u, 0x3F803F80u, 0x3F803F80u, 0x3F803F80u);
  }
  bool wrong = false;
  for (int i = threadIdx.x; i <= P.n_seqs; i += kA8Threads) {
    const int s0 = P.start[i], s1 = P.start[min(i + 1, P.n_seqs)];
    s_start[i] = s0;
    wrong |= wrong_rows(s0, s1, P.T);
  }
  wrong = __syncthreads_or(wrong);
  if (wrong && blockIdx.x == 0 && threadIdx.x == 0) atomicCAS(P.err, 0, (int)MOE_ERR_INVALID_ARG);
  if (warp == 0) {  // the CTA's leaders, in order
    const int t = t0 + lane;
    A8Block B{t, 0, 0, 0, 0u, -1};
    if (lane < a.rows && t < P.T) {
      const int b = seq_of(s_start, P.n_seqs, t, P.T, wrong);
      if (b >= 0) {
        const int i = t - s_start[b], len = P.kv_len[b];
        const long long p = (long long)len + i;
        const int o = (int)(p & (kA8Block - 1));
        bool leads = i == 0 || o == 0;
        if (wrong) {  // rows of the block before this one may be another sequence's
          leads = true;
          for (int j = max(t - o, s_start[b]); j < t; ++j) leads = leads && seq_of(s_start, P.n_seqs, j, P.T, true) != b;
        }
        if (leads) {
          int e = 0;
          if (len < 0) {
            e = MOE_ERR_INVALID_ARG;
          } else if (p >= (long long)P.max_pages << P.lps) {
            e = MOE_ERR_CAPACITY;
          } else {
            const int page = P.table[(size_t)b * P.max_pages + (size_t)(p >> P.lps)];
            if (page < 0 || page >= P.n_pages) e = MOE_ERR_INVALID_ARG;
            else B.slot = ((long long)page * P.nkv << P.lps) + (p & (ps - 1));
          }
          if (e) atomicCAS(P.err, 0, e);
          B.pos = (int)(p < 0 ? 0 : p > 0x7fffffff ? 0x7fffffff : p);
          B.n = min(kA8Block - o, s_start[b + 1] - t);
          B.com = max(0, o - i);
          B.own = (1u << B.n) - 1;
          for (int j = 1; wrong && j < B.n; ++j)
            if (seq_of(s_start, P.n_seqs, t + j, P.T, true) != b) B.own &= ~(1u << j);
        }
      }
    }
    const unsigned who = __ballot_sync(0xffffffffu, B.n > 0);
    if (B.n > 0) s_block[__popc(who & ((1u << lane) - 1))] = B;
    if (lane == 0) s_n = __popc(who);
  }
  __syncthreads();

  // What a head's row is multiplied by (over its eight lanes; 1 without norms).
  auto norm = [&](const uint4& x0, const uint4& y0) {
    if constexpr (!NORM) return 1.f;
    uint4 x = x0, y = y0;
    f2 ss = make_f2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f2 lo = unpack2(word(x, i)), hi = unpack2(word(y, i));
      ss = fma2(hi, hi, fma2(lo, lo, ss));
    }
    float sq = sum2(ss);
#pragma unroll
    for (int d = 1; d < 8; d <<= 1) sq += __shfl_xor_sync(0xffffffffu, sq, d);
    return inv_sqrt(__fmaf_rn(sq, 1.f / 128.f, a.eps));
  };
  // A head's row: normed, turned; into v (dims d0 .., d1 ..).
  auto make = [&](const uint4& x0, const uint4& y0, float inv, int r, bool q, f2 (&v)[8]) {
    uint4 x = x0, y = y0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = unpack2(word(x, i));
      v[4 + i] = unpack2(word(y, i));
    }
    if constexpr (NORM) {
      const f2 inv2 = make_f2(inv, inv);
      const uint4* gain = s_gain + (q ? 0 : 16);
      uint4 g0 = gain[d0 >> 3], g1 = gain[d1 >> 3];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[i] = mul2(mul2(v[i], inv2), unpack2(word(g0, i)));
        v[4 + i] = mul2(mul2(v[4 + i], inv2), unpack2(word(g1, i)));
      }
    }
    if constexpr (VEC) {
      if (turns) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float2 c = *reinterpret_cast<const float2*>(&s_cos[r][d0 + 2 * i]);
          const float2 s = *reinterpret_cast<const float2*>(&s_sin[r][d0 + 2 * i]);
          const f2 c2 = make_f2(c.x, c.y), lo = v[i], hi = v[4 + i];
          v[i] = add2(mul2(lo, c2), mul2(hi, make_f2(-s.x, -s.y)));
          v[4 + i] = add2(mul2(hi, c2), mul2(lo, make_f2(s.x, s.y)));
        }
      }
    } else {
      float* row = s_head[warp][grp];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) *reinterpret_cast<f2*>(row + 16 * l8 + 2 * i) = v[i];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 16 * l8 + i, j = d < half ? d : d - half;
        if (d < a.rd) {
          const float xc = __fmul_rn(row[d], s_cos[r][j]), ys = __fmul_rn(row[d < half ? d + half : j], s_sin[r][j]);
          const float z = d < half ? __fsub_rn(xc, ys) : __fadd_rn(xc, ys);
          float u, w;
          asm("mov.b64 {%0, %1}, %2;" : "=f"(u), "=f"(w) : "l"(v[i >> 1]));
          v[i >> 1] = i & 1 ? make_f2(u, z) : make_f2(z, w);
        }
      }
    }
  };
  const uint4 zero = make_uint4(0u, 0u, 0u, 0u);

  for (int k = 0; k < s_n; ++k) {
    const A8Block B = s_block[k];
    for (int i = threadIdx.x; i < B.n * half; i += kA8Threads) {
      const int r = i / half, j = i - r * half;
      rope_cs_fine(B.pos + r, a.freq[j], s_cos[r][j], s_sin[r][j]);
    }
    __syncthreads();

    // The block's tasks: keys and values of `heads` heads (with `per` groups of
    // lanes a head), and 16 (row, head) pairs of queries.  They are dealt over
    // the warps of all CTAs of the block.
    const int per = B.n == 1 ? 1 : B.n == 2 ? 2 : 4, heads = 4 / per, pairs = B.n * nqu;
    const int n_kv = B.slot >= 0 ? (2 * P.nkv + heads - 1) / heads : 0, n_q = (pairs + 4 * kA8Pairs - 1) / (4 * kA8Pairs);
    for (int task = warp * gridDim.y + blockIdx.y; task < n_kv + n_q; task += kA8Warps * gridDim.y) {
      if (task >= n_kv) {
        uint4 x[kA8Pairs], y[kA8Pairs];
        int r[kA8Pairs], h[kA8Pairs];
        bool live[kA8Pairs];
#pragma unroll
        for (int i = 0; i < kA8Pairs; ++i) {
          const int u = ((task - n_kv) * kA8Pairs + i) * 4 + grp;
          r[i] = min(u, pairs - 1) / nqu;
          h[i] = u - r[i] * nqu;
          live[i] = u < pairs && (B.own >> r[i] & 1);
          x[i] = y[i] = zero;
          if (live[i]) {
            const uint16_t* src = a.q + (B.t + r[i]) * a.qs + h[i] * 128;
            x[i] = *reinterpret_cast<const uint4*>(src + d0);
            y[i] = *reinterpret_cast<const uint4*>(src + d1);
          }
        }
#pragma unroll
        for (int i = 0; i < kA8Pairs; ++i) {
          f2 v[8];
          make(x[i], y[i], norm(x[i], y[i]), r[i], true, v);
          if (!live[i]) continue;
          uint16_t* dst = a.qo + (B.t + r[i]) * a.qos + h[i] * 128;
          *reinterpret_cast<uint4*>(dst + d0) = make_uint4(pack2(v[0]), pack2(v[1]), pack2(v[2]), pack2(v[3]));
          *reinterpret_cast<uint4*>(dst + d1) = make_uint4(pack2(v[4]), pack2(v[5]), pack2(v[6]), pack2(v[7]));
        }
        continue;
      }
      const int hu = task * heads + grp / per;
      const bool isv = hu >= P.nkv, live = hu < 2 * P.nkv;
      const int h = isv ? hu - P.nkv : hu;
      uint4 x[4], y[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (grp & (per - 1)) + 4 * i;
        x[i] = y[i] = zero;
        if (live && (B.own >> r & 1)) {
          const uint16_t* src = isv ? a.v + (B.t + r) * a.vs + h * 128 : a.k + (B.t + r) * a.ks + h * 128;
          x[i] = *reinterpret_cast<const uint4*>(src + d0);
          y[i] = *reinterpret_cast<const uint4*>(src + d1);
        }
      }
      const long long slot = B.slot + ((long long)h << P.lps);
      uint8_t* scale = (isv ? A.vs : A.ks) + (slot >> 4);
      const int old = live && B.com > 0 ? *scale : 0;
      const bool keys = task * heads < P.nkv;  // some lane of the warp has a key
      f2 v[4][8];
      float m = 0.f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (4 * i >= B.n) continue;
        const int r = (grp & (per - 1)) + 4 * i;
        if (keys) make(x[i], y[i], norm(x[i], y[i]), r < B.n ? r : 0, false, v[i]);  // (a row that is not the block's: zeros)
        if (isv) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            v[i][j] = unpack2(word(x[i], j));
            v[i][4 + j] = unpack2(word(y[i], j));
          }
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max2(m, v[i][j]);
      }
      auto over = [&](float z) {
        for (int d = 1; d < 8 * per; d <<= 1) z = fmaxf(z, __shfl_xor_sync(0xffffffffu, z, d));
        return z;
      };
      m = over(m);
      if (__any_sync(0xffffffffu, m > FLT_MAX)) {  // an infinity: the largest of the others; its code is NaN
        m = 0.f;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (4 * i >= B.n) continue;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            m = max2(m, finite2(v[i][j], 0.f));
            v[i][j] = finite2(v[i][j], __int_as_float(0x7fffffff));
          }
        }
        m = over(m);
      }
      // 448 = 1.75 * 2^8
      const uint32_t mb = __float_as_uint(m);
      const int want = max(1, (int)(mb >> 23) - ((mb & 0x7fffffu) <= 0x600000u ? 8 : 7)), now = max(want, old);
      const float by = now == 255 ? __int_as_float(0x7fffffff) : now == 254 ? 0x1p-127f : __uint_as_float((uint32_t)(254 - now) << 23);
      const f2 by2 = make_f2(by, by);
      uint8_t* codes = (isv ? A.vc : A.kc) + slot * 128;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = (grp & (per - 1)) + 4 * i;
        if (!live || !(B.own >> r & 1)) continue;
        *reinterpret_cast<uint2*>(codes + r * 128 + d0) = make_uint2(e4m3_codes(v[i][0], v[i][1], by2), e4m3_codes(v[i][2], v[i][3], by2));
        *reinterpret_cast<uint2*>(codes + r * 128 + d1) = make_uint2(e4m3_codes(v[i][4], v[i][5], by2), e4m3_codes(v[i][6], v[i][7], by2));
      }
      if (!live) continue;
      if (B.com > 0 && now > old) {  // the committed positions' codes move with the scale
        const int e = 127 + old - now;
        const float f = now == 255 ? __int_as_float(0x7fffffff) : e > 0 ? __uint_as_float((uint32_t)e << 23) : 0.f;
        uint8_t* begin = codes - (B.pos & (kA8Block - 1)) * 128;
        for (int r = (grp & (per - 1)); r < B.com; r += per) {
          uint4* c = reinterpret_cast<uint4*>(begin + r * 128) + l8;
          uint4 w = *c;
#pragma unroll
          for (int j = 0; j < 4; ++j) word(w, j) = e4m3_times(word(w, j), f);
          *c = w;
        }
      }
      if (l8 == 0 && (grp & (per - 1)) == 0) *scale = (uint8_t)now;
    }
    __syncthreads();  // the angles are free
  }
}

cudaError_t launch_paged_append8(const PagedAppend8Args& a0, cudaStream_t s) {
  PagedAppend8Args a = a0;
  const int wave = 2 * num_sms(), rows = (a.a.p.T + wave - 1) / wave;
  a.a.rows = rows < kA8Rows ? rows : kA8Rows;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.a.p.T + a.a.rows - 1) / a.a.rows, rows == 1 ? 2 : 1);
  cfg.blockDim = dim3(kA8Threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern, cudaError_t e) { return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, a) : e; };
  const bool vec = (a.a.rd / 2) % 8 == 0;
  if (a.a.norm)
    return vec ? run(k_paged_append8<true, true>, prepare_kernel<k_paged_append8<true, true>>(0))
               : run(k_paged_append8<false, true>, prepare_kernel<k_paged_append8<false, true>>(0));
  return vec ? run(k_paged_append8<true, false>, prepare_kernel<k_paged_append8<true, false>>(0))
             : run(k_paged_append8<false, false>, prepare_kernel<k_paged_append8<false, false>>(0));
}

}  // namespace moe
