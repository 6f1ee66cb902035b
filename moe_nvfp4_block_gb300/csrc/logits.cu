// logits.cu -- the rules of a batch of rows on their logits (penalties for
// repeated tokens, biases, grammar masks) and each row's argmax, in one pass.
//
// CTA (tile, row) owns `tile` consecutive tokens of a row.  It counts the
// row's history into a shared-memory table of its tokens (whole-number
// atomics: the order does not matter), so no count ever reaches memory, then
// walks its logits once: penalty, bias, mask, store, running maximum.  The
// row's last CTA (a ticket) takes the best of the tiles.
//
// What bounds it: the logits read and written once; the history is read by
// every tile of its row, which L2 serves (tiles are as large as the grid
// allows).  So that the arithmetic stays below that, a thread's 16-byte line
// of 4 or 8 tokens is one step: one look at the table's bit map (few tokens
// are repeats), one shifted word of the mask, whole 16-byte loads of the
// bias, one maximum, and the index is searched only in a line that beats it.
//
// Rows start anywhere (an odd vocabulary): a row's elements are grouped by
// the 16-byte lines of its input, element j = v + phase with phase the row's
// offset from a line; whole lines inside the row take one 16-byte load.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

__device__ __forceinline__ bool lg_better(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

// The N floats at p (4-byte aligned), by aligned 16-byte loads; reads up to
// 12 bytes before p and 16 after the last.
template <int N>
__device__ __forceinline__ void lg_floats(const float* p, float (&f)[N]) {
  const int mis = (int)((reinterpret_cast<uintptr_t>(p) >> 2) & 3);
  const float4* q = reinterpret_cast<const float4*>(p - mis);
  if (mis == 0) {
#pragma unroll
    for (int i = 0; i < N / 4; ++i) {
      const float4 v = __ldg(q + i);
      f[4 * i] = v.x;
      f[4 * i + 1] = v.y;
      f[4 * i + 2] = v.z;
      f[4 * i + 3] = v.w;
    }
    return;
  }
  float w[N + 4];
#pragma unroll
  for (int i = 0; i <= N / 4; ++i) {
    const float4 v = __ldg(q + i);
    w[4 * i] = v.x;
    w[4 * i + 1] = v.y;
    w[4 * i + 2] = v.z;
    w[4 * i + 3] = v.w;
  }
#pragma unroll
  for (int i = 0; i < N; ++i) f[i] = mis == 1 ? w[i + 1] : mis == 2 ? w[i + 2] : w[i + 3];
}

}  // namespace

template <typename T, int THREADS>
__global__ void __launch_bounds__(THREADS) k_logits(const __grid_constant__ LogitArgs a) {
  constexpr int N = 16 / sizeof(T);  // elements of a line
  extern __shared__ __align__(16) int s_cnt[];  // [tile] counts, then [tile / 32] words: which are not 0
  __shared__ float s_bv[THREADS / 32];
  __shared__ int s_bi[THREADS / 32];
  __shared__ int s_last;
  const moe_logit_rules& R = a.rules;
  const int r = blockIdx.y, V = a.V, tid = threadIdx.x;
  unsigned* s_hit = reinterpret_cast<unsigned*>(s_cnt + a.tile);
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(a.x) + r * a.xs;
  T* out = a.out ? static_cast<T*>(a.out) + r * a.os : nullptr;
  const int phase = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const bool same = out && (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(x) & 15);
  // this CTA's tokens [v0, v1); its lines start at element j0 = v0 + phase
  const int j0 = blockIdx.x * a.tile;
  const int v0 = max(0, j0 - phase), v1 = min(V, j0 + a.tile - phase);
  auto whole = [&](int v) { return v >= 0 && v + N <= V; };
  // the first line is on its way while the history is counted
  int j = j0 + tid * N;
  uint4 line = make_uint4(0u, 0u, 0u, 0u);
  if (j < j0 + a.tile && whole(j - phase)) line = *reinterpret_cast<const uint4*>(x + j - phase);

  bool counted = false;
  if (R.tokens) {
    const int h0 = max(0, R.begin[r]), h1 = min(R.n_tokens, R.end[r]);
    if (h0 < h1) {
      counted = true;
      uint4* z = reinterpret_cast<uint4*>(s_cnt);
      for (int i = tid; i < (a.tile + a.tile / 32) / 4; i += THREADS) z[i] = make_uint4(0u, 0u, 0u, 0u);
      __syncthreads();
      auto count = [&](int v) {
        if (v >= v0 && v < v1) {
          const int e = v + phase - j0;
          if (atomicAdd(&s_cnt[e], 1) == 0) atomicOr(&s_hit[e >> 5], 1u << (e & 31));
        }
      };
      // aligned groups of four, and the tokens before and after them
      const int mis = (int)((reinterpret_cast<uintptr_t>(R.tokens + h0) >> 2) & 3);
      const int g0 = min(h1, h0 + ((4 - mis) & 3)), g1 = g0 + ((h1 - g0) & ~3);
      if (tid < g0 - h0) count(R.tokens[h0 + tid]);
      if (tid < h1 - g1) count(R.tokens[g1 + tid]);
#pragma unroll 2
      for (int i = g0 + 4 * tid; i < g1; i += 4 * THREADS) {
        const int4 t = __ldg(reinterpret_cast<const int4*>(R.tokens + i));
        count(t.x);
        count(t.y);
        count(t.z);
        count(t.w);
      }
      __syncthreads();
    }
  }
  const float rep = R.repetition ? R.repetition[r] : 1.f;
  const float pres = R.presence ? R.presence[r] : 0.f, freq = R.frequency ? R.frequency[r] : 0.f;
  const float* bias = nullptr;
  const uint32_t* allow = nullptr;
  bool bad = false;
  if (R.bias) {
    const int b = R.bias_row[r];
    bad = b >= R.n_bias;
    if (b >= 0 && !bad) bias = R.bias + (size_t)b * V;
  }
  if (R.allow) {
    const int b = R.allow_row[r];
    if (b >= R.n_allow) bad = true;
    else if (b >= 0) allow = R.allow + (size_t)b * ((V + 31) / 32);
  }
  if (bad && tid == 0) atomicCAS(a.err, 0, (int)MOE_ERR_INVALID_ARG);

  auto penalty = [&](float f, int c) {
    f = f > 0.f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
    return __fsub_rn(f, __fadd_rn(pres, __fmul_rn((float)c, freq)));
  };
  auto load = [](T e) {
    if constexpr (sizeof(T) == 4) return (float)e;
    else return bf16_bits_to_float(e);
  };
  auto store = [](float f) {
    if constexpr (sizeof(T) == 4) return (T)f;
    else return (T)float_to_bf16_bits(f);
  };

  float bv = -INFINITY;
  int bi = -1;
  for (; j < j0 + a.tile; j += THREADS * N) {
    const int v = j - phase, e0 = j - j0;
    if (v >= V) break;
    // the next line is on its way
    uint4 next = make_uint4(0u, 0u, 0u, 0u);
    if (j + THREADS * N < j0 + a.tile && whole(v + THREADS * N)) next = *reinterpret_cast<const uint4*>(x + v + THREADS * N);
    if (whole(v)) {
      T e[N];
      memcpy(e, &line, 16);
      float f[N];
#pragma unroll
      for (int i = 0; i < N; ++i) f[i] = load(e[i]);
      if (counted) {
        const unsigned hit = (s_hit[e0 >> 5] >> (e0 & 31)) & ((1u << N) - 1u);
        if (hit) {
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (hit >> i & 1) f[i] = penalty(f[i], s_cnt[e0 + i]);
        }
      }
      if (bias) {
        float b[N];
        if (v >= 4 && v + N + 4 <= V) {
          lg_floats<N>(bias + v, b);
        } else {
#pragma unroll
          for (int i = 0; i < N; ++i) b[i] = bias[v + i];
        }
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __fadd_rn(f[i], b[i]);
      }
      if (allow) {
        const uint32_t lo = __ldg(allow + (v >> 5)), hi = __ldg(allow + ((v + N - 1) >> 5));
        const uint32_t bits = __funnelshift_r(lo, hi, v & 31);
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
      for (int i = max(0, -v); i < N && v + i < V; ++i) {
        float f = load(x[v + i]);
        if (counted && s_cnt[e0 + i]) f = penalty(f, s_cnt[e0 + i]);
        if (bias) f = __fadd_rn(f, bias[v + i]);
        if (allow && !((allow[(v + i) >> 5] >> ((v + i) & 31)) & 1u)) f = -INFINITY;
        if (f > bv) {
          bv = f;
          bi = v + i;
        }
        if (out) out[v + i] = store(f);
      }
    }
    line = next;
  }
  if (!a.tok && !a.best) return;
  const int lane = tid & 31, warp = tid >> 5;
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
  if (tid == 0) {
    for (int w = 1; w < THREADS / 32; ++w)
      if (s_bi[w] >= 0 && (bi < 0 || lg_better(s_bv[w], s_bi[w], bv, bi))) {
        bv = s_bv[w];
        bi = s_bi[w];
      }
    a.part_v[(size_t)r * a.ntile + blockIdx.x] = bv;
    a.part_i[(size_t)r * a.ntile + blockIdx.x] = bi;
    __threadfence();
    s_last = atomicAdd(a.ticket + r, 1u) == (unsigned)a.ntile - 1;
  }
  __syncthreads();
  if (!s_last || warp != 0) return;
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

// Tokens of a CTA: a multiple of 1024, as large as leaves about two CTAs an
// SM (fewer re-reads of the history), 1024 to kLogitTile.
static int logit_tile(int R, int V) {
  const int tiles = (2 * num_sms() + R - 1) / R;
  const int t = (V / tiles + 1023) / 1024 * 1024;
  return t < 1024 ? 1024 : t > kLogitTile ? kLogitTile : t;
}

cudaError_t launch_logits(const LogitArgs& a0, cudaStream_t s) {
  LogitArgs a = a0;
  a.tile = logit_tile(a.R, a.V);
  a.ntile = (a.V + 7 + a.tile - 1) / a.tile;  // the phase shifts a row by up to 7 elements
  const bool wide = a.tile >= 8192;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ntile, a.R);
  cfg.blockDim = dim3(wide ? 512 : 256);
  cfg.dynamicSmemBytes = a.rules.tokens ? sizeof(int) * (a.tile + a.tile / 32) : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                         (int)sizeof(int) * (kLogitTile + kLogitTile / 32));
    if (e == cudaSuccess) e = max_carveout(kern);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, a) : e;
  };
  if (wide) return a.bf16 ? run(k_logits<uint16_t, 512>) : run(k_logits<float, 512>);
  return a.bf16 ? run(k_logits<uint16_t, 256>) : run(k_logits<float, 256>);
}

}  // namespace moe
