// paged_attn.cuh -- what the two forms of the paged attention share: how a
// call's work is listed and cut, and the producer warp that walks it.
#pragma once

#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kPaChunk = 64;                     // positions of a chunk
constexpr int kPaHalf = kPaChunk * 256;          // a stage's keys (or values)
constexpr int kPaStageBytes = 2 * kPaHalf;
constexpr uint64_t kPaDrainNs = 2000000000ull;

template <int STAGES>
struct PaRing {
  uint64_t full[STAGES];
  uint64_t empty[STAGES];
  int abort;
};

// A sequence of the call: its rows, and the chunks that hold their visible
// positions: np of the kept prefix from cp, then those from cm on.
struct PaSeq {
  int q0, n, len, first, prefix;
  int cp, np, cm, nch;
};

__device__ __forceinline__ PaSeq pa_seq(const PagedAttnArgs& a, int b, int* err) {
  const PagedRows& P = a.p;
  PaSeq s{};
  s.q0 = P.start[b];
  const int q1 = P.start[b + 1];
  s.len = P.kv_len[b];
  s.first = a.first ? max(0, a.first[b]) : 0;
  s.prefix = a.prefix && a.window > 0 ? max(0, a.prefix[b]) : 0;
  if (q1 == s.q0) return s;
  int e = 0;
  if (s.q0 < 0 || q1 < s.q0 || q1 > P.T || q1 - s.q0 > a.max_rows || s.len < 0) e = MOE_ERR_INVALID_ARG;
  else if ((long long)s.len + (q1 - s.q0) > (long long)P.max_pages << P.lps) e = MOE_ERR_CAPACITY;
  if (e) {
    if (err) atomicCAS(err, 0, e);
    return s;
  }
  s.n = q1 - s.q0;
  const int hi = s.len + s.n;
  s.first = min(s.first, hi);
  s.prefix = min(s.prefix, hi);
  const int lo = a.window > 0 ? max(s.first, s.len - a.window + 1) : s.first;
  s.cm = lo / kPaChunk;
  s.nch = lo < hi ? (hi - 1) / kPaChunk + 1 - s.cm : 0;
  if (s.prefix > s.first && lo > s.first) {
    s.cp = s.first / kPaChunk;
    const int end = min((min(s.prefix, lo) - 1) / kPaChunk + 1, s.cm);
    s.np = max(0, end - s.cp);
    s.nch += s.np;
  }
  if (s.nch == 0) {  // rows that see nothing still have an output
    s.cm = 0;
    s.nch = 1;
  }
  return s;
}

// Whether some row sees a position of [p0, p1]; whether every row sees all.
__device__ __forceinline__ bool pa_any(int len, int n, int first, int prefix, int window, int p0, int p1) {
  const int hi = len + n, lo = window > 0 ? max(first, len - window + 1) : first;
  return (max(p0, lo) < hi && p1 >= lo) || (max(p0, first) < prefix && p1 >= first);  // (lo may be hi: nothing visible)
}
__device__ __forceinline__ bool pa_all(int len, int n, int first, int prefix, int window, int p0, int p1) {
  return p0 >= first && p1 <= len && (window == 0 || p0 > len + n - 1 - window || p1 < prefix);
}

// 2^x to 2 ulp, 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Two floats; two correctly rounded operations at a time.
__device__ __forceinline__ unsigned long long pa_pair(float x, float y) {
  unsigned long long p;
  asm("mov.b64 %0, {%1, %2};" : "=l"(p) : "f"(x), "f"(y));
  return p;
}
__device__ __forceinline__ void pa_unpair(unsigned long long p, float& x, float& y) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(x), "=f"(y) : "l"(p));
}
__device__ __forceinline__ unsigned long long pa_mul2(unsigned long long a, unsigned long long b) {
  unsigned long long d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ unsigned long long pa_fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}

// Two capped scores, cap tanh(x scale / cap), in the log2 domain; x, y: q . k.
// With w = 2 log2(e) z and z the tanh's argument, 1 - 2 / (2^w + 1) is off by
// FP32 roundings of 1 however small z is (an error of 1e-7 caps), so that below
// |z| = 1/8 the series z (1 - z^2/3 + 2 z^4/15) takes over, its first term the
// uncapped score: either way within 9e-7 of the score.
__device__ __forceinline__ void pa_capped(const PagedAttnArgs& a, float& x, float& y) {
  constexpr float h = 0.12011325348f;  // (ln 2 / 2)^2: z^2 = h w^2
  const unsigned long long xy = pa_pair(x, y), w = pa_mul2(xy, pa_pair(a.cap_in, a.cap_in)), t = pa_mul2(w, w);
  unsigned long long p = pa_fma2(pa_pair(2.f / 15.f * h * h, 2.f / 15.f * h * h), t, pa_pair(-h / 3.f, -h / 3.f));
  p = pa_mul2(pa_fma2(p, t, pa_pair(1.f, 1.f)), pa_mul2(xy, pa_pair(a.scale_log2, a.scale_log2)));
  float w0, w1, t0, t1, p0, p1;
  pa_unpair(w, w0, w1);
  pa_unpair(t, t0, t1);
  pa_unpair(p, p0, p1);
  const float l0 = __fmaf_rn(-2.f * a.cap_log2, rcp(ex2(w0) + 1.f), a.cap_log2);
  const float l1 = __fmaf_rn(-2.f * a.cap_log2, rcp(ex2(w1) + 1.f), a.cap_log2);
  x = t0 < 1.f / 64.f / h ? p0 : l0;
  y = t1 < 1.f / 64.f / h ? p1 : l1;
}

// Two weights, each times kPaUp, in two bf16 parts: hi + lo to 2^-16.  Both
// parts are positive where the weight is (hi is cut off, and kPaUp leaves more
// than nothing for lo): an infinite value times either is then that value again,
// where a lo that is negative or zero, as rounding leaves it, makes inf - inf or
// 0 * inf of it.  Sums are divided by kPaUp at the end (pa_inverse).  (hi cut
// from a little below the weight, without a factor at the end: two more
// instructions a pair, 143 us against 141 for 65,003 and 131,001 positions.)
constexpr float kPaUp = 1.f + 0x1p-16f;
__device__ __forceinline__ void pa_split(float x, float y, uint32_t& hi, uint32_t& lo) {
  hi = __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632);
  lo = pack_bf16(__fmaf_rn(x, kPaUp, -__uint_as_float(hi << 16)), __fmaf_rn(y, kPaUp, -__uint_as_float(hi & 0xFFFF0000u)));
}
// What makes a row's output of its sums; l: the weights' sum.
__device__ __forceinline__ float pa_inverse(float l) { return l == 0.f ? 0.f : 1.f / (l * kPaUp); }

// mbar_wait_bounded, with several tries before the first look at the clock.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort) {
  if (limit_ns == 0) return false;
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_bounded(bar, parity, limit_ns, abort);
}

// A CTA's segment of a (sequence, KV head) unit: chunks [j0, j1) of it.
struct PaSegment {
  PaSeq s;
  int kvh, j0, j1;
  int cf, np;  // np > 1: a cut unit, whose first CTA is cf and whose parts are np
  int slot;    // where this CTA's part goes (0 / 1)
  __device__ __forceinline__ int pos(int j) const { return (j < s.np ? s.cp + j : s.cm + j - s.np) * kPaChunk; }
};

// (Out of line: what runs before the first load should be short.)
__device__ __noinline__ long long pa_div(long long x, long long y) { return x / y; }

// The producer warp: the CTA's share of the call's slots (plan: every
// sequence; UNIT of them before each unit's chunks), chunk by chunk into the ring.
//   out.begin(segment, stage): a segment begins with this stage (false: gave up)
//   out.stage(segment, j, stage, bytes): one lane, before the loads of chunk j
//   out.put(slot, box, row, barrier): loads a box's keys and values, the
//     cache rows from `row` on
//   out.end(stage): the CTA's work is written down
// Returns the number of stages begun; *abort is set where a wait ran out.
template <int UNIT, int STAGES, class Out>
__device__ __forceinline__ int pa_produce(const PagedAttnParams& A, PaRing<STAGES>& T, const PaSeq* plan, int cta, int lane,
                                          Out out) {
  const PagedAttnArgs& a = A.a;
  const PagedRows& P = a.p;
  volatile int* abort = &T.abort;
  const int lbr = min(P.lps, 6), br = 1 << lbr;  // positions of a box
  // lane l sums the sequences [l k, (l + 1) k); the lane that holds the
  // CTA's first slot finds its sequence
  auto slots = [&](int nch) { return nch > 0 ? (long long)P.nkv * (nch + UNIT) : 0LL; };
  const int k = (P.n_seqs + 31) / 32;
  long long sum = 0;
  for (int i = 0; i < k; ++i)
    if (lane * k + i < P.n_seqs) sum += slots(plan[lane * k + i].nch);
  long long inc = sum;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, inc, d);
    if (lane >= d) inc += o;
  }
  const long long W = __shfl_sync(0xffffffffu, inc, 31);
  // no more CTAs than slots: every CTA inside a cut unit has a part of it
  const int G = (int)min((long long)gridDim.x, W);
  const bool small = W < 1 << 22;  // 32-bit divisions do
  auto div = [&](long long x, long long y) {
    return small ? (long long)((unsigned)x / (unsigned)y) : pa_div(x, y);
  };
  const long long w0 = cta < G ? div(cta * W, G) : W, w1 = cta < G ? div((cta + 1) * W, G) : W;
  long long base = inc - sum;
  int b = lane * k;
  const bool mine = base <= w0 && w0 < inc;
  if (mine)
    while (base + slots(plan[b].nch) <= w0) base += slots(plan[b++].nch);
  const unsigned who = __ballot_sync(0xffffffffu, mine);
  const int src = who ? __ffs(who) - 1 : 0;
  b = __shfl_sync(0xffffffffu, b, src);
  base = __shfl_sync(0xffffffffu, base, src);
  PaSeq s{};
  if (w0 < w1) s = plan[b];
  // the plan's memory becomes the ring's: its reads before the async writes
  __syncwarp();
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");

  const int lnb = 6 - lbr;  // log2 of a chunk's boxes
  int st = 0;
  // the next stage's place in the ring; false: given up
  auto begin = [&]() {
    bool ok = true;
    if (st >= STAGES)
      ok = !*abort && pa_wait(&T.empty[st % STAGES], (uint32_t)(st / STAGES - 1) & 1u, A.wait_ns, abort);
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) *abort = 1;
    return ok;
  };
  bool live = true;
  int kvh = s.nch > 0 ? (int)div(w0 - base, s.nch + UNIT) : 0;
  // page cache: lane l holds box l & (boxes - 1) of chunk cj + (l >> lnb) of sequence cb
  int cb = -1, cj = 0, crow = 0;
  bool cload = false;
  while (live) {
    const int span = s.nch + UNIT;
    const long long rs = base + (long long)kvh * span + UNIT, re = rs + s.nch;  // the unit's chunks
    if (rs >= w1 || w0 >= w1) break;
    PaSegment g{s, kvh, rs >= w0 ? 0 : (int)(w0 - rs), (int)(min(re, w1) - rs), 0, 1, rs >= w0};
    if (rs < w0 || re > w1) {
      g.cf = (int)div((rs + 1) * G - 1, W);
      g.np = (int)div(re * G - 1, W) - g.cf + 1;
    }
    live = out.begin(g, st);
    if (!live) break;
    for (int j = g.j0; j < g.j1; ++j) {
      if (b != cb || j < cj || j >= cj + (32 >> lnb)) {
        cb = b;
        cj = j;
        const int c = j + (lane >> lnb);
        const int p0 = g.pos(c) + ((lane & ((1 << lnb) - 1)) << lbr);
        cload = c < s.nch && pa_any(s.len, s.n, s.first, s.prefix, a.window, p0, p0 + br - 1);
        if (cload) {
          int page = P.table[(size_t)b * P.max_pages + (p0 >> P.lps)];
          if (page < 0 || page >= P.n_pages) {
            atomicCAS(P.err, 0, (int)MOE_ERR_INVALID_ARG);
            page = 0;
          }
          crow = (page * P.nkv << P.lps) + (p0 & ((1 << P.lps) - 1));
        }
      }
      live = begin();
      if (!live) break;
      const bool load = cload && (lane >> lnb) == j - cj;
      const unsigned boxes = __ballot_sync(0xffffffffu, load);
      out.stage(g, j, st, __popc(boxes) * (uint32_t)(br * 512));
      __syncwarp();
      if (load) out.put(st % STAGES, lane & ((1 << lnb) - 1), crow + (kvh << P.lps), &T.full[st % STAGES]);
      ++st;
    }
    if (!live || re >= w1) break;
    if (++kvh == P.nkv) {
      base += (long long)P.nkv * span;
      kvh = 0;
      do s = pa_seq(a, ++b, nullptr);
      while (s.nch == 0);
    }
  }
  if (live && begin() && out.end(st)) ++st;
  __syncwarp();
  return st;
}

// After a wait ran out: records it and waits for the ring's copies in flight
// (one thread, when every warp has left the ring).
template <int STAGES>
__device__ __forceinline__ void pa_drain(PaRing<STAGES>& T, int st, int* err) {
  atomicCAS(err, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
  for (int i = max(0, st - STAGES); i < st; ++i)
    mbar_wait_drain(&T.full[i % STAGES], (uint32_t)(i / STAGES) & 1u, kPaDrainNs);
}

}  // namespace

}  // namespace moe
