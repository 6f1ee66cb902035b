// logits.cu -- the rules of a batch of rows on their logits (penalties for
// repeated tokens, biases, grammar masks) and each row's argmax, in one pass.
//
// CTA (tile, row) owns `tile` consecutive tokens of a row.  Tiles of up to 4096
// count their repeated tokens in a table with a place for each, and the walk
// over the logits (penalty, bias, mask, store, running maximum) looks there.
// Longer tiles turn the history into a short list: a bit map of the tile, the
// number of bits before each of its words, and, by a second look at the
// history, the tokens' counts at their places in the list; the penalties (a
// division among them) are taken once per listed token, the walk holds listed
// tokens at -inf, and the list's own pass behind it stores and compares them,
// in the list's rising order, so that a warp's 32 lie near one another.  More
// than kLgList listed tokens are worked on a stretch of the tile at a time.
// The row's last CTA (a ticket) takes the best of the tiles.
//
// (A short tile by the list takes five more waits: 8.1 us against 6.1 for one
// row of 151,936 with a history of 700.  A long one by the table would leave
// its threads too little to do between two looks at the history.)
//
// What bounds it: the logits read and written once, and above that the
// instructions of the walk and the looks at the history.  256 rows of 128,003
// bf16 tokens (131 MB in all: 19 us at a copy's bandwidth) take 25 us without
// rules, 39 with biases and masks, 58 with histories of 4000 as well.  So:
//  * tiles are as long as leaves the SMs evenly filled, since every tile looks
//    through its row's whole history: 65 us where tiles of 65,536 took 70;
//  * lines come by cp.async, kLgRing ahead a thread, asked for before the look
//    at the history (25 us without rules, 37 with plain loads two ahead);
//  * a thread's 16-byte line of 4 or 8 tokens is one step: one shifted word of
//    the bit map and one of the mask, whole 16-byte loads of the bias, one
//    maximum, and the index is searched only in a line that beats the warp's
//    best (listed tokens picked up inside the walk: 65 us against 59);
//  * lines over an end of the row take a step of their own.
//
// Rows start anywhere (an odd vocabulary): a row's elements are grouped by
// the 16-byte lines of its input, element j = v + phase with phase the row's
// offset from a line; whole lines inside the row take one 16-byte load.
#include <type_traits>

#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ bool lg_better(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

// f[i] += the i-th of the N biases that start MIS floats into b.
template <int N, int MIS>
__device__ __forceinline__ void lg_add(const float4 (&b)[N / 4 + 1], float (&f)[N]) {
  float w[N + 4];
#pragma unroll
  for (int i = 0; i < N / 4 + 1; ++i) {
    w[4 * i] = b[i].x;
    w[4 * i + 1] = b[i].y;
    w[4 * i + 2] = b[i].z;
    w[4 * i + 3] = b[i].w;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = __fadd_rn(f[i], w[i + MIS]);
}

}  // namespace

constexpr int kLgList = 4096;
constexpr int kLgRing = 4;  // lines a thread has asked for ahead of the one it works on

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_logits(const __grid_constant__ LogitArgs a) {
  constexpr int N = 16 / sizeof(T);  // elements of a line
  constexpr bool DENSE = THREADS == 256;  // a count for every token of the tile, no list
  extern __shared__ __align__(16) uint4 s_ring[];  // [kLgRing][THREADS] lines of x
  unsigned* s_bits = reinterpret_cast<unsigned*>(s_ring + kLgRing * THREADS);  // [tile / 32] bit map
  __shared__ float s_bv[THREADS / 32];
  __shared__ int s_bi[THREADS / 32];
  const moe_logit_rules& R = a.rules;
  const int r = blockIdx.y, V = a.V, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nw = a.tile / 32;
  int* s_pre = reinterpret_cast<int*>(s_bits + nw);                          // [nw] bits before the word
  int* s_cnt = DENSE ? reinterpret_cast<int*>(s_bits) : s_pre + nw;          // [kLgList] counts, then values
  int* s_tok = s_cnt + kLgList;                                              // [kLgList] elements of the tile
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(a.x) + r * a.xs;
  T* out = a.out ? static_cast<T*>(a.out) + r * a.os : nullptr;
  const int phase = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const bool same = out && (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(x) & 15);
  // this CTA's elements start at j0: element e of the tile is token e + j0 - phase
  const int j0 = blockIdx.x * a.tile;
  const int e_lo = max(0, phase - j0), e_hi = min(a.tile, V + phase - j0);  // the row's elements
  const T* xt = x + (j0 - phase);
  // line k of this thread is at element (k THREADS + tid) N; the first ones are
  // on their way while the history is looked at
  auto fetch = [&](int k) {
    const int e = (k * THREADS + tid) * N;
    if (e >= e_lo && e + N <= e_hi) cp_async_16(&s_ring[k % kLgRing * THREADS + tid], xt + e);
    cp_async_commit();
  };
#pragma unroll
  for (int k = 0; k < kLgRing; ++k) fetch(k);
  auto load = [](T e) {
    if constexpr (sizeof(T) == 4) return (float)e;
    else return bf16_bits_to_float(e);
  };
  auto store = [](float f) {
    if constexpr (sizeof(T) == 4) return (T)f;
    else return (T)float_to_bf16_bits(f);
  };

  // the row's parameters, all asked for before the first wait
  const int brow = R.bias ? R.bias_row[r] : -1, arow = R.allow ? R.allow_row[r] : -1;
  const float* bias = brow >= 0 && brow < R.n_bias ? R.bias + (size_t)brow * V + (j0 - phase) : nullptr;
  const uint32_t* allow = arow >= 0 && arow < R.n_allow ? R.allow + (size_t)arow * ((V + 31) / 32) : nullptr;
  // where the tile's lines start in the bias: the same for all of them
  const int bias_mis = (int)((reinterpret_cast<uintptr_t>(bias) >> 2) & 3);
  const float rep = R.tokens && R.repetition ? R.repetition[r] : 1.f;
  const float pres = R.tokens && R.presence ? R.presence[r] : 0.f;
  const float freq = R.tokens && R.frequency ? R.frequency[r] : 0.f;
  int h0 = 0, h1 = 0, n = 0;  // the history; listed tokens of the tile (DENSE: whether it has any)
  // f(e) for every token of the history that is element e of the tile
  auto history = [&](auto f) {
    auto one = [&](int v) {
      const int e = v + phase - j0;
      if (v >= 0 && v < V && e >= 0 && e < a.tile) f(e);
    };
    // aligned groups of four, and the tokens before and after them
    const int mis = (int)((reinterpret_cast<uintptr_t>(R.tokens + h0) >> 2) & 3);
    const int g0 = min(h1, h0 + ((4 - mis) & 3)), g1 = g0 + ((h1 - g0) & ~3);
    if (tid < g0 - h0) one(R.tokens[h0 + tid]);
    if (tid < h1 - g1) one(R.tokens[g1 + tid]);
    for (int i = g0 + 4 * tid; i < g1; i += 4 * THREADS) {
      const int4 t = __ldg(reinterpret_cast<const int4*>(R.tokens + i));
      one(t.x);
      one(t.y);
      one(t.z);
      one(t.w);
    }
  };
  if (R.tokens) {
    h0 = max(0, R.begin[r]);
    h1 = min(R.n_tokens, R.end[r]);
    if (DENSE && h0 < h1) {
      for (int i = tid; i < a.tile / 4; i += THREADS) reinterpret_cast<uint4*>(s_cnt)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      history([&](int e) { atomicAdd(&s_cnt[e], 1); });
      __syncthreads();
      n = 1;
    }
    if (!DENSE && h0 < h1) {
      for (int i = tid; i < nw / 4; i += THREADS) reinterpret_cast<uint4*>(s_bits)[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      history([&](int e) { atomicOr(&s_bits[e >> 5], 1u << (e & 31)); });
      __syncthreads();
      // bits before each word: thread t has words [t k, (t + 1) k)
      const int k = (nw + THREADS - 1) / THREADS;
      int own = 0;
      for (int i = tid * k; i < min(nw, tid * k + k); ++i) own += __popc(s_bits[i]);
      int inc = own;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const int o = __shfl_up_sync(0xffffffffu, inc, d);
        if (lane >= d) inc += o;
      }
      if (lane == 31) s_bi[warp] = inc;
      __syncthreads();
      int before = inc - own;
      for (int w = 0; w < THREADS / 32; ++w) {
        const int c = s_bi[w];
        if (w < warp) before += c;
        n += c;
      }
      for (int i = tid * k; i < min(nw, tid * k + k); ++i) {
        s_pre[i] = before;
        before += __popc(s_bits[i]);
      }
      __syncthreads();
    }
  }
  auto penalise = [&](float f, int c) {
    f = f > 0.f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
    return __fsub_rn(f, __fadd_rn(pres, __fmul_rn((float)c, freq)));
  };

  float bv = -INFINITY;
  int bi = -1, k = 0;
  float wmax = -INFINITY;  // of the warp's lanes' bv
  auto warp_max = [](float x) {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, d));
    return x;
  };
  // The warp's lines of step k: bias, mask, store, maximum.  A listed token is
  // stored and compared behind the walk, and is -inf here.  EDGE: lines or
  // their bias may reach over an end of the row.
  auto step = [&](int k, auto edge) {
    constexpr bool EDGE = decltype(edge)::value;
    const int e0 = (k * THREADS + tid) * N, v = e0 + j0 - phase;
    const bool whole = !EDGE || (e0 >= e_lo && e0 + N <= e_hi);
    unsigned in = (1u << N) - 1u;  // which tokens of the line are the row's
    if (EDGE && !whole) {
      in = 0;
#pragma unroll
      for (int i = 0; i < N; ++i) in |= e0 + i >= e_lo && e0 + i < e_hi ? 1u << i : 0u;
    }
    // what comes from memory besides the ring, asked for before any is used
    float4 b[N / 4 + 1];
    uint32_t bits = in;
    const bool wide = bias && (!EDGE || (v >= 4 && v + N + 4 <= V));  // whole lines of the bias: 3 floats more on a side
    if (wide) {
      const float4* p = reinterpret_cast<const float4*>(bias + e0 - bias_mis);
#pragma unroll
      for (int i = 0; i < N / 4 + 1; ++i) b[i] = __ldg(p + i);
    }
    if (allow && in) {
      const int v0 = EDGE ? max(v, 0) : v, v1 = EDGE ? min(v + N, V) - 1 : v + N - 1;
      bits = __funnelshift_r(__ldg(allow + (v0 >> 5)), __ldg(allow + (v1 >> 5)), v0 & 31) << (v0 - v) & in;
    }
    if (!DENSE && n > 0 && in) bits &= ~(s_bits[e0 >> 5] >> (e0 & 31));
    cp_async_wait<kLgRing - 1>();
    const uint4 line = s_ring[k % kLgRing * THREADS + tid];
    fetch(k + kLgRing);
    T e[N];
    memcpy(e, &line, 16);
    if (EDGE && !whole)
#pragma unroll
      for (int i = 0; i < N; ++i) e[i] = in >> i & 1u ? xt[e0 + i] : (T)0;
    float f[N];
#pragma unroll
    for (int i = 0; i < N; ++i) f[i] = load(e[i]);
    if (DENSE && n > 0) {
      int c[N];
#pragma unroll
      for (int i = 0; i < N; i += 4) {
        const int4 q = *reinterpret_cast<const int4*>(s_cnt + e0 + i);
        c[i] = q.x;
        c[i + 1] = q.y;
        c[i + 2] = q.z;
        c[i + 3] = q.w;
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (c[i] > 0) f[i] = penalise(f[i], c[i]);
    }
    if (wide) {
      switch (bias_mis) {
        case 0: lg_add<N, 0>(b, f); break;
        case 1: lg_add<N, 1>(b, f); break;
        case 2: lg_add<N, 2>(b, f); break;
        default: lg_add<N, 3>(b, f); break;
      }
    } else if (EDGE && bias) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (in >> i & 1u) f[i] = __fadd_rn(f[i], bias[e0 + i]);
    }
    if (bits != (1u << N) - 1u) {
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (!(bits >> i & 1u)) f[i] = -INFINITY;
    }
    float top = f[0];
#pragma unroll
    for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
    if (__any_sync(0xffffffffu, top > wmax)) {
      if (top > wmax) {
        bv = top;
#pragma unroll
        for (int i = N - 1; i >= 0; --i)
          if (f[i] == top) bi = v + i;
      }
      wmax = warp_max(bv);
    }
    if (out) {
      if (whole && same) {
        uint4 w;
        if constexpr (N == 4)
          w = make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
        else
          w = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
        *reinterpret_cast<uint4*>(out + v) = w;
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i)
          if (!EDGE || (in >> i & 1u)) out[v + i] = store(f[i]);
      }
    }
  };
  // stretches [w_lo, w_hi) of the bit map's words with at most kLgList listed tokens
  for (int w_lo = 0, w_hi; w_lo < nw; w_lo = w_hi) {
    w_hi = nw;
    const int p0 = !DENSE && n > 0 ? s_pre[w_lo] : 0;
    if (!DENSE && n > 0) {
      int m = n - p0;
      if (m > kLgList) {  // as many of a warp's lines (N words) as fit
        int lo = w_lo / N + 1, hi = nw / N - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_pre[mid * N] - p0 <= kLgList) lo = mid;
          else hi = mid - 1;
        }
        w_hi = lo * N;
        m = s_pre[w_hi] - p0;
      }
      for (int i = tid; i < m; i += THREADS) s_cnt[i] = 0;
      __syncthreads();
      history([&](int e) {
        const int w = e >> 5;
        if (w < w_lo || w >= w_hi) return;
        const int i = s_pre[w] - p0 + __popc(s_bits[w] & ((1u << (e & 31)) - 1u));
        atomicAdd(&s_cnt[i], 1);
        s_tok[i] = e;
      });
      __syncthreads();
      for (int i0 = tid; i0 < m; i0 += 4 * THREADS) {
        T xl[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) xl[u] = i0 + u * THREADS < m ? xt[s_tok[i0 + u * THREADS]] : (T)0;
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int i = i0 + u * THREADS;
          if (i >= m) break;
          s_cnt[i] = __float_as_int(penalise(load(xl[u]), s_cnt[i]));
        }
      }
      __syncthreads();
    }
    // this warp's lines of the stretch, 32 at a time
    const int end = min(32 * w_hi, e_hi);
    for (int ew; (ew = (k * THREADS + 32 * warp) * N) < end; ++k) {
      const int vw = ew + j0 - phase;
      if (vw >= 4 && vw + 32 * N + 4 <= V && ew + 32 * N <= e_hi) step(k, std::false_type{});
      else step(k, std::true_type{});
    }
    __syncthreads();
    // the stretch's listed tokens
    if (!DENSE && n > 0) {
      const int m = (w_hi < nw ? s_pre[w_hi] : n) - p0;
      for (int i = tid; i < m; i += THREADS) {
        const int e = s_tok[i], v = e + j0 - phase;
        float f = __int_as_float(s_cnt[i]);
        if (bias) f = __fadd_rn(f, bias[e]);
        if (allow && !(__ldg(allow + (v >> 5)) >> (v & 31) & 1u)) f = -INFINITY;
        if (out) out[v] = store(f);
        if (lg_better(f, v, bv, bi)) {
          bv = f;
          bi = v;
        }
      }
      wmax = warp_max(bv);
    }
    __syncthreads();  // the list is free
  }
  if (((R.bias && brow >= R.n_bias) || (R.allow && arow >= R.n_allow)) && tid == 0)
    atomicCAS(a.err, 0, (int)MOE_ERR_INVALID_ARG);
  if (!a.tok && !a.best) return;
  auto warp_best = [&]() {
#pragma unroll
    for (int d = 16; d >= 1; d >>= 1) {
      const float ov = __shfl_xor_sync(0xffffffffu, bv, d);
      const int oi = __shfl_xor_sync(0xffffffffu, bi, d);
      if (oi >= 0 && (bi < 0 || lg_better(ov, oi, bv, bi))) {
        bv = ov;
        bi = oi;
      }
    }
  };
  warp_best();
  if (lane == 0) {
    s_bv[warp] = bv;
    s_bi[warp] = bi;
  }
  __syncthreads();
  if (warp != 0) return;
  bv = lane < THREADS / 32 ? s_bv[lane] : -INFINITY;
  bi = lane < THREADS / 32 ? s_bi[lane] : -1;
  warp_best();
  unsigned last = 0;
  if (a.ntile == 1) {
    if (lane == 0) {
      if (a.tok) a.tok[r] = bi;
      if (a.best) a.best[r] = bv;
    }
    return;
  }
  if (lane == 0) {
    a.part_v[(size_t)r * a.ntile + blockIdx.x] = bv;
    a.part_i[(size_t)r * a.ntile + blockIdx.x] = bi;
    __threadfence();
    last = atomicAdd(a.ticket + r, 1u) == (unsigned)a.ntile - 1;
  }
  if (!__shfl_sync(0xffffffffu, last, 0)) return;
  __threadfence();
  bv = -INFINITY;
  bi = -1;
  for (int i = lane; i < a.ntile; i += 32) {
    const float ov = __ldcg(a.part_v + (size_t)r * a.ntile + i);
    const int oi = __ldcg(a.part_i + (size_t)r * a.ntile + i);
    if (oi >= 0 && (bi < 0 || lg_better(ov, oi, bv, bi))) {
      bv = ov;
      bi = oi;
    }
  }
  warp_best();
  if (lane == 0) {
    if (a.tok) a.tok[r] = bi;
    if (a.best) a.best[r] = bv;
    a.ticket[r] = 0u;
  }
}

// Tokens of a CTA, a multiple of 1024: a row in n parts, the n with the least
// waves x (tile + what a CTA costs besides, about 4096 tokens' time).  (146
// rows of 157,142: parts of 79,872 and no second wave take 28 us, 131,072 and
// the rest 50.)
static int logit_tile(int R, int V) {
  const int slots = 2 * num_sms();
  const auto part = [&](int n) { return ((V + 7 + n - 1) / n + 1023) / 1024 * 1024; };
  const int least = (V + 7 + kLogitTile - 1) / kLogitTile, most = (V + 7) / 1024 + 1;
  int best = part(least);
  long long cost = -1;
  for (int w = 0; w <= 4; ++w) {  // the shortest parts of each number of waves
    int n = w * slots / R;
    n = n < least ? least : n > most ? most : n;
    const int t = part(n);
    const long long waves = ((long long)R * ((V + 7 + t - 1) / t) + slots - 1) / slots;
    const long long c = waves * ((t < V ? t : V) + 4096);
    if (cost < 0 || c < cost) {
      cost = c;
      best = t;
    }
  }
  return best;
}

cudaError_t launch_logits(const LogitArgs& a0, cudaStream_t s) {
  LogitArgs a = a0;
  a.tile = logit_tile(a.R, a.V);
  a.ntile = (a.V + 7 + a.tile - 1) / a.tile;  // the phase shifts a row by up to 7 elements
  const bool wide = a.tile > 4096;
  const auto ring = [](int threads) { return 16 * kLgRing * threads; };
  const auto list = [](int tile) { return tile > 4096 ? tile / 4 + 8 * kLgList : 4 * tile; };
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ntile, a.R);
  cfg.blockDim = dim3(wide ? 512 : 256);
  cfg.dynamicSmemBytes = ring(wide ? 512 : 256) + (a.rules.tokens ? list(a.tile) : 0);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern, cudaError_t e) { return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, a) : e; };
  const int most = ring(512) + list(kLogitTile);
  if (wide)
    return a.bf16 ? run(k_logits<uint16_t, 512>, prepare_kernel<k_logits<uint16_t, 512>>(most))
                  : run(k_logits<float, 512>, prepare_kernel<k_logits<float, 512>>(most));
  return a.bf16 ? run(k_logits<uint16_t, 256>, prepare_kernel<k_logits<uint16_t, 256>>(most))
                : run(k_logits<float, 256>, prepare_kernel<k_logits<float, 256>>(most));
}

}  // namespace moe
