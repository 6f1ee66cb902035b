// logits.cu -- the rules of a batch of rows on their logits (penalties for
// repeated tokens, biases, grammar masks) and each row's argmax, in one pass.
//
// CTA (tile, row) owns `tile` consecutive tokens of a row.  It counts the
// row's history into a shared-memory table of its tokens (whole-number
// atomics: the order does not matter), so no count ever reaches memory, then
// walks its logits once: penalty, bias, mask, store, running argmax.  The
// row's last CTA (a ticket) takes the best of the tiles.
//
// What bounds it: the logits read and written once; the history is read by
// every tile of its row, which L2 serves (tiles are as large as the grid
// allows).
//
// Rows start anywhere (an odd vocabulary): a row's elements are grouped by
// the 16-byte lines of its input, element j = v + phase with phase the row's
// offset from a line; whole lines inside the row take one 16-byte load.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kLgThreads = 256;

__device__ __forceinline__ bool lg_better(float a, int i, float b, int j) { return a > b || (a == b && i < j); }

}  // namespace

template <typename T>
__global__ void __launch_bounds__(kLgThreads) k_logits(const __grid_constant__ LogitArgs a) {
  constexpr int N = 16 / sizeof(T);  // elements of a line
  extern __shared__ int s_cnt[];     // [tile]
  __shared__ float s_bv[kLgThreads / 32];
  __shared__ int s_bi[kLgThreads / 32];
  __shared__ int s_last;
  const moe_logit_rules& R = a.rules;
  const int r = blockIdx.y, V = a.V, tid = threadIdx.x;
  pdl_wait();
  pdl_launch_dependents();
  const T* x = static_cast<const T*>(a.x) + r * a.xs;
  T* out = a.out ? static_cast<T*>(a.out) + r * a.os : nullptr;
  const int phase = (int)((reinterpret_cast<uintptr_t>(x) & 15) / sizeof(T));
  const bool same = out && (reinterpret_cast<uintptr_t>(out) & 15) == (reinterpret_cast<uintptr_t>(x) & 15);
  // this CTA's tokens [v0, v1); its lines start at element j0 = v0 + phase
  const int j0 = blockIdx.x * a.tile;
  const int v0 = max(0, j0 - phase), v1 = min(V, j0 + a.tile - phase);

  bool counted = false;
  if (R.tokens) {
    const int h0 = max(0, R.begin[r]), h1 = min(R.n_tokens, R.end[r]);
    if (h0 < h1) {
      counted = true;
      for (int i = tid; i < a.tile; i += kLgThreads) s_cnt[i] = 0;
      __syncthreads();
      for (int i = h0 + tid; i < h1; i += kLgThreads) {
        const int v = R.tokens[i];
        if (v >= v0 && v < v1) atomicAdd(&s_cnt[v + phase - j0], 1);
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

  auto rule = [&](float f, int v) {
    if (counted) {
      const int c = s_cnt[v + phase - j0];
      if (c) {
        f = f > 0.f ? __fdiv_rn(f, rep) : __fmul_rn(f, rep);
        f = __fsub_rn(f, __fadd_rn(pres, __fmul_rn((float)c, freq)));
      }
    }
    if (bias) f = __fadd_rn(f, bias[v]);
    if (allow && !((allow[v >> 5] >> (v & 31)) & 1u)) f = -INFINITY;
    return f;
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
  for (int j = j0 + tid * N; j < j0 + a.tile; j += kLgThreads * N) {
    const int v = j - phase;
    if (v >= V) break;
    if (v >= 0 && v + N <= V) {
      const uint4 line = *reinterpret_cast<const uint4*>(x + v);
      T e[N];
      memcpy(e, &line, 16);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const float f = rule(load(e[i]), v + i);
        if (f > bv) {
          bv = f;
          bi = v + i;
        }
        e[i] = store(f);
      }
      if (same) {
        uint4 w;
        memcpy(&w, e, 16);
        *reinterpret_cast<uint4*>(out + v) = w;
      } else if (out) {
#pragma unroll
        for (int i = 0; i < N; ++i) out[v + i] = e[i];
      }
    } else {
      for (int i = max(0, -v); i < N && v + i < V; ++i) {
        const float f = rule(load(x[v + i]), v + i);
        if (f > bv) {
          bv = f;
          bi = v + i;
        }
        if (out) out[v + i] = store(f);
      }
    }
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
    for (int w = 1; w < kLgThreads / 32; ++w)
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
int logit_tile(int R, int V) {
  const long long want = 2LL * num_sms();
  const int tiles = (int)((want + R - 1) / R);
  int t = (V / tiles + 1023) / 1024 * 1024;
  return t < 1024 ? 1024 : t > kLogitTile ? kLogitTile : t;
}

cudaError_t launch_logits(const LogitArgs& a0, cudaStream_t s) {
  LogitArgs a = a0;
  a.tile = logit_tile(a.R, a.V);
  a.ntile = (a.V + 7 + a.tile - 1) / a.tile;  // the phase shifts a row by up to 7 elements
  const size_t sm = sizeof(int) * a.tile;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ntile, a.R);
  cfg.blockDim = dim3(kLgThreads);
  cfg.dynamicSmemBytes = a.rules.tokens ? sm : 0;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    max_carveout(kern);
    return cudaLaunchKernelEx(&cfg, kern, a);
  };
  return a.bf16 ? run(k_logits<uint16_t>) : run(k_logits<float>);
}

}  // namespace moe
