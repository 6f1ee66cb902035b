// logits.cu -- the rules of a batch of rows on their logits (penalties for
// repeated tokens, biases, grammar masks) and each row's argmax, in one pass.
//
// CTA (tile, row) owns `tile` consecutive tokens of a row.  The history is
// turned into a short list of the tile's repeated tokens: a bit map of the
// tile, the number of bits before each of its words, and, by a second look at
// the history, the tokens' counts at their places in the list.  The penalties
// (a division among them) are then taken once per listed token, and the walk
// over all logits only picks them up: penalty, bias, mask, store, running
// maximum.  More than kLgList listed tokens are worked on a stretch of the
// tile at a time.  The row's last CTA (a ticket) takes the best of the tiles.
//
// What bounds it: the logits read and written once, and how much of a CTA's
// life its loads fill, so tiles are as long as leaves the SMs evenly filled
// (a table of counts per token instead of the bit map holds 8192 tokens where
// this one holds 65,536: 78 us against 67 for 256 rows of 128,003 tokens
// with histories of 4000, whose every tile then looks through the history
// again).  So that the arithmetic stays below that, a thread's 16-byte line
// of 4 or 8 tokens is one step: one look at the bit map, one shifted word of
// the mask, whole 16-byte loads of the bias, one maximum, and the index is
// searched only in a line that beats it.
//
// Rows start anywhere (an odd vocabulary): a row's elements are grouped by
// the 16-byte lines of its input, element j = v + phase with phase the row's
// offset from a line; whole lines inside the row take one 16-byte load.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ bool lg_better(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

// What a line of N tokens is worked with: its logits, the bias's 16-byte lines
// that hold its N values, the one or two words that hold its mask.
template <int N>
struct LgLine {
  uint4 x;
  float4 b[N / 4 + 1];
  uint32_t lo, hi;
};

// f[i] += the line's i-th bias, the first MIS floats behind the start of b.
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
constexpr int kLgDeep = 2;  // lines in flight a thread

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) k_logits(const __grid_constant__ LogitArgs a) {
  constexpr int N = 16 / sizeof(T);  // elements of a line
  extern __shared__ __align__(16) unsigned s_bits[];  // [tile / 32] bit map
  __shared__ float s_bv[THREADS / 32];
  __shared__ int s_bi[THREADS / 32];
  const moe_logit_rules& R = a.rules;
  const int r = blockIdx.y, V = a.V, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int nw = a.tile / 32;
  int* s_pre = reinterpret_cast<int*>(s_bits + nw);               // [nw] bits before the word
  int* s_cnt = s_pre + nw;                                        // [kLgList] counts, then values
  uint16_t* s_tok = reinterpret_cast<uint16_t*>(s_cnt + kLgList); // [kLgList] elements of the tile
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
  // the tile's lines come to L2 while the history is looked at
  if (R.tokens && tid == 0 && e_lo < e_hi) {
    const int p0 = (e_lo + N - 1) / N * N, p1 = e_hi / N * N;
    if (p0 < p1) l2_prefetch_span(xt + p0, (uint64_t)(p1 - p0) * sizeof(T));
  }
  auto load = [](T e) {
    if constexpr (sizeof(T) == 4) return (float)e;
    else return bf16_bits_to_float(e);
  };
  auto store = [](float f) {
    if constexpr (sizeof(T) == 4) return (T)f;
    else return (T)float_to_bf16_bits(f);
  };

  int h0 = 0, h1 = 0, n = 0;  // the history; listed tokens of the tile
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
    if (h0 < h1) {
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
  const int brow = R.bias ? R.bias_row[r] : -1, arow = R.allow ? R.allow_row[r] : -1;
  const float* bias = brow >= 0 && brow < R.n_bias ? R.bias + (size_t)brow * V + (j0 - phase) : nullptr;
  const uint32_t* allow = arow >= 0 && arow < R.n_allow ? R.allow + (size_t)arow * ((V + 31) / 32) : nullptr;
  if (((R.bias && brow >= R.n_bias) || (R.allow && arow >= R.n_allow)) && tid == 0)
    atomicCAS(a.err, 0, (int)MOE_ERR_INVALID_ARG);
  // where the tile's lines start in the bias: the same for all of them
  const int bias_mis = (int)((reinterpret_cast<uintptr_t>(bias) >> 2) & 3);

  float bv = -INFINITY;
  int bi = -1;
  // stretches [w_lo, w_hi) of the bit map's words with at most kLgList listed tokens
  for (int w_lo = 0, w_hi; w_lo < nw; w_lo = w_hi) {
    w_hi = nw;
    const int p0 = n > 0 ? s_pre[w_lo] : 0;
    if (n > 0) {
      int m = n - p0;
      if (m > kLgList) {  // the last word that still fits
        int lo = w_lo + 1, hi = nw - 1;
        while (lo < hi) {
          const int mid = (lo + hi + 1) >> 1;
          if (s_pre[mid] - p0 <= kLgList) lo = mid;
          else hi = mid - 1;
        }
        w_hi = lo;
        m = s_pre[w_hi] - p0;
      }
      for (int i = tid; i < m; i += THREADS) s_cnt[i] = 0;
      __syncthreads();
      history([&](int e) {
        const int w = e >> 5;
        if (w < w_lo || w >= w_hi) return;
        const int i = s_pre[w] - p0 + __popc(s_bits[w] & ((1u << (e & 31)) - 1u));
        atomicAdd(&s_cnt[i], 1);
        s_tok[i] = (uint16_t)e;
      });
      __syncthreads();
      const float rep = R.repetition ? R.repetition[r] : 1.f;
      const float pres = R.presence ? R.presence[r] : 0.f, freq = R.frequency ? R.frequency[r] : 0.f;
      for (int i = tid; i < m; i += THREADS) {
        float f = load(xt[s_tok[i]]);
        f = f > 0.f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
        s_cnt[i] = __float_as_int(__fsub_rn(f, __fadd_rn(pres, __fmul_rn((float)s_cnt[i], freq))));
      }
      __syncthreads();
    }
    const int end = min(32 * w_hi, e_hi);
    // everything that a line needs from memory, asked for at once
    auto ask = [&](int e, LgLine<N>& q) {
      if (e < e_lo || e + N > end) return;
      const int v = e + j0 - phase;
      q.x = *reinterpret_cast<const uint4*>(xt + e);
      if (bias && v >= 4 && v + N + 4 <= V) {  // whole lines, up to 3 floats more on each side
        const float4* p = reinterpret_cast<const float4*>(bias + e - bias_mis);
#pragma unroll
        for (int i = 0; i < N / 4 + 1; ++i) q.b[i] = __ldg(p + i);
      }
      if (allow) {
        q.lo = __ldg(allow + (v >> 5));
        q.hi = __ldg(allow + ((v + N - 1) >> 5));
      }
    };
    for (int e1 = 32 * w_lo + tid * N; e1 < end; e1 += kLgDeep * THREADS * N) {
      LgLine<N> lines[kLgDeep];
#pragma unroll
      for (int u = 0; u < kLgDeep; ++u) ask(e1 + u * THREADS * N, lines[u]);
#pragma unroll
      for (int u = 0; u < kLgDeep; ++u) {
        const int e0 = e1 + u * THREADS * N;
        if (e0 >= end) break;
        const LgLine<N>& q = lines[u];
        const int v = e0 + j0 - phase;
        unsigned hit = 0;
        if (n > 0) hit = (s_bits[e0 >> 5] >> (e0 & 31)) & ((1u << N) - 1u);
        auto listed = [&]() { return s_pre[e0 >> 5] - p0 + __popc(s_bits[e0 >> 5] & ((1u << (e0 & 31)) - 1u)); };
        if (e0 >= e_lo && e0 + N <= e_hi) {
          T e[N];
          memcpy(e, &q.x, 16);
          float f[N];
#pragma unroll
          for (int i = 0; i < N; ++i) f[i] = load(e[i]);
          if (hit) {
            int at = listed();
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (hit >> i & 1) f[i] = __int_as_float(s_cnt[at++]);
          }
          if (bias) {
            if (v >= 4 && v + N + 4 <= V) {
              switch (bias_mis) {
                case 0: lg_add<N, 0>(q.b, f); break;
                case 1: lg_add<N, 1>(q.b, f); break;
                case 2: lg_add<N, 2>(q.b, f); break;
                default: lg_add<N, 3>(q.b, f); break;
              }
            } else {
#pragma unroll
              for (int i = 0; i < N; ++i) f[i] = __fadd_rn(f[i], bias[e0 + i]);
            }
          }
          if (allow) {
            const uint32_t bits = __funnelshift_r(q.lo, q.hi, v & 31);
#pragma unroll
            for (int i = 0; i < N; ++i)
              if (!(bits >> i & 1u)) f[i] = -INFINITY;
          }
          float top = f[0];
#pragma unroll
          for (int i = 1; i < N; ++i) top = fmaxf(top, f[i]);
          if (top > bv) {
            bv = top;
#pragma unroll
            for (int i = N - 1; i >= 0; --i)
              if (f[i] == top) bi = v + i;
          }
          if (out) {
#pragma unroll
            for (int i = 0; i < N; ++i) e[i] = store(f[i]);
            if (same) {
              uint4 w;
              memcpy(&w, e, 16);
              *reinterpret_cast<uint4*>(out + v) = w;
            } else {
#pragma unroll
              for (int i = 0; i < N; ++i) out[v + i] = e[i];
            }
          }
        } else {  // a row's first or last line, in part
          int at = hit ? listed() : 0;
          for (int i = max(0, e_lo - e0); i < N && e0 + i < e_hi; ++i) {
            float f = load(xt[e0 + i]);
            if (hit >> i & 1) f = __int_as_float(s_cnt[at++]);
            if (bias) f = __fadd_rn(f, bias[e0 + i]);
            if (allow && !((allow[(v + i) >> 5] >> ((v + i) & 31)) & 1u)) f = -INFINITY;
            if (f > bv) {
              bv = f;
              bi = v + i;
            }
            if (out) out[v + i] = store(f);
          }
        }
      }
    }
    __syncthreads();  // the list is free
  }
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

// Tokens of a CTA: 1024 times a power of two up to kLogitTile, the one with
// the least waves x (tile + what a CTA costs besides, about 4096 tokens' time).
static int logit_tile(int R, int V) {
  int best = 1024;
  long long cost = -1;
  for (int t = 1024; t <= kLogitTile; t *= 2) {
    const long long ctas = (long long)R * ((V + t - 1) / t);
    const long long waves = (ctas + 2LL * num_sms() - 1) / (2LL * num_sms());
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
  const auto bytes = [](int tile) { return tile / 4 + 6 * kLgList; };
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ntile, a.R);
  cfg.blockDim = dim3(wide ? 512 : 256);
  cfg.dynamicSmemBytes = a.rules.tokens ? bytes(a.tile) : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern, cudaError_t e) { return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, a) : e; };
  const int most = bytes(kLogitTile);
  if (wide)
    return a.bf16 ? run(k_logits<uint16_t, 512>, prepare_kernel<k_logits<uint16_t, 512>>(most))
                  : run(k_logits<float, 512>, prepare_kernel<k_logits<float, 512>>(most));
  return a.bf16 ? run(k_logits<uint16_t, 256>, prepare_kernel<k_logits<uint16_t, 256>>(most))
                : run(k_logits<float, 256>, prepare_kernel<k_logits<float, 256>>(most));
}

}  // namespace moe
