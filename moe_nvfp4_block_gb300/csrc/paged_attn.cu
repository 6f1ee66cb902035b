// paged_attn.cu -- attention of verify rows over a paged KV cache.
//
// For row t of sequence b (position pos = kv_len[b] + i) and query head h:
//   s_p = score(q . k_p),  o = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m)
// over the visible positions p, in one pass with a running maximum m (in the
// log2 domain) and, where a sequence is cut, a join of the parts' (m, l, o).
//
// What bounds it: each visible position's keys and values (512 bytes a KV
// head) are read once.  The work of a call is the list of all 64-position
// chunks of all (sequence, KV head) units, each unit preceded by kPaUnit
// slots for what its start and end cost; CTA c of G (two an SM) takes the
// slots [c W / G, (c + 1) W / G) of the W, whatever units they fall in, so
// that unequal lengths cost no balance.  A unit inside one CTA is written out
// there; the parts of a cut unit go to the workspace (at most two a CTA) and
// are joined, in CTA order, by a second kernel whose CTAs share the rows.
// (The join by the unit's last CTA to arrive, in the same kernel, reads all
// of its parts through one SM: 37 us against 21 for 4 rows at 16,384
// positions.  CTAs that wait for one another would need the whole GPU.)
//
// A producer warp walks the chunks: it looks up their pages (a chunk is one
// half or whole page, or several) and loads keys and values by TMA into a
// ring of three 32 KB stages, with a description of the chunk beside it.
// Eight warps compute.  The unit's rows (verify rows x heads of the KV head)
// are MT tiles of 16; the 8 / MT warps of a tile share a chunk twice: each
// takes 8 MT positions of S = Q K^T, they agree on the running maximum, leave
// P in shared memory, and each takes 16 MT dims of O += P V (mma.sync
// m16n8k16).  So a warp holds few sums (8 MT registers), 18 warps fit an SM,
// and a unit ends without adding up outputs: a warp alone is bound by the
// latency of its instructions, and with the positions split all the way (each
// warp its own maximum and all 128 dims, four warps of 168 registers) a chunk
// took 1.9 us and a unit's end 2.5 to 4.5.  P is split into two bf16 parts (P
// = hi + lo to 2^-17: one bf16 P would add as much error as the output's own
// rounding; the second product is free while the loads bound the kernel).
//
// Hidden positions: a score is replaced by -inf, and as 0 * v is not 0 for
// an infinite or NaN v, a slice with hidden positions is looked over for such
// values first and, with any, summed element by element over the visible
// positions alone.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr int kPaWarps = 8;                      // compute warps
constexpr int kPaThreads = (kPaWarps + 1) * 32;  // and the producer
constexpr int kPaChunk = 64;
constexpr int kPaStages = 3;
constexpr int kPaHalf = kPaChunk * 256;          // a stage's keys (or values)
constexpr int kPaStageBytes = 2 * kPaHalf;
constexpr int kPaUnit = 1;                       // slots before a unit's chunks
constexpr uint64_t kPaDrainNs = 2000000000ull;

// A chunk as its stage's readers see it.
struct PaDesc {
  int q0, n, len, kvh;       // the sequence's first row, rows, committed length; KV head
  int pos0, first, prefix;   // the chunk's first position; the sequence's limits
  int flags;                 // kPaLast: the segment's last chunk; kPaEnd; kPaAny, kPaAll
  int cf, np;                // np > 1: a cut unit, whose first CTA is cf and whose parts are np
  int slot, pad;             // where this CTA's part goes (0 / 1)
};
constexpr int kPaLast = 1, kPaEnd = 2;  // kPaEnd: no chunk, the CTA is done
constexpr int kPaAny = 4, kPaAll = 8;   // bit of the first of four 16-position slices: some row sees
                                        // some of it / every row sees all of it

struct PaTable {
  uint64_t full[kPaStages];
  uint64_t empty[kPaStages];
  uint64_t told[kPaStages];  // the description is written (the data may still be on its way)
  PaDesc desc[kPaStages];
  int abort;
  float m[kPaWarps * 16];  // [tile][row][part]: maxima of the parts' scores; at a segment's end their sums
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
  s.prefix = a.prefix && a.window > 0 ? a.prefix[b] : 0;
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
  return (p0 < hi && p1 >= lo) || (max(p0, first) < prefix && p1 >= first);
}
__device__ __forceinline__ bool pa_all(int len, int n, int first, int prefix, int window, int p0, int p1) {
  return p0 >= first && p1 <= len && (window == 0 || p0 > len + n - 1 - window || p1 < prefix);
}

__device__ __forceinline__ void pa_ldsm(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void pa_ldsm_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr));
}
__device__ __forceinline__ void pa_mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
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

// mbar_wait_bounded, with several tries before the first look at the clock.
__device__ __forceinline__ bool pa_wait(uint64_t* bar, uint32_t parity, uint64_t limit_ns, const volatile int* abort) {
  if (limit_ns == 0) return false;
#pragma unroll 1
  for (int i = 0; i < 16; ++i)
    if (mbar_try_wait(bar, parity)) return true;
  return mbar_wait_bounded(bar, parity, limit_ns, abort);
}

// Barrier of a tile's warps that also tells whether one has given up.  A warp
// that gives up (a wait ran out) takes part once more, with `fail`, and
// leaves; so does every warp at the end: each instance has all of them.
template <int THREADS>
__device__ __forceinline__ bool pa_sync(int tile, bool fail) {
  uint32_t any;
  asm volatile(
      "{\n .reg .pred p, q;\n setp.ne.u32 p, %1, 0;\n barrier.cta.red.or.pred q, %3, %2, p;\n selp.u32 %0, 1, 0, q;\n}"
      : "=r"(any)
      : "r"((uint32_t)fail), "n"(THREADS), "r"(tile + 1)
      : "memory");
  return any == 0;
}

}  // namespace

template <int MT>
__global__ void __launch_bounds__(kPaThreads, 2) k_paged_attn(const __grid_constant__ PagedAttnParams A) {
  constexpr int PARTS = kPaWarps / MT;  // warps of a tile
  const PagedAttnArgs& a = A.a;
  const PagedRows& P = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_p = smem + kPaStages * kPaStageBytes;  // P: [tile][hi, lo][16 rows][64 positions] bf16
  constexpr bool QS = MT == 2;  // the rows stay in shared memory ([tile][16 rows][128 dims]), not in registers
  PaTable& T = *reinterpret_cast<PaTable*>(s_p + MT * 4096 + (QS ? MT * 4096 : 0));
  PaSeq* plan = reinterpret_cast<PaSeq*>(smem);  // [n_seqs], in the ring before its first load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int lbr = min(P.lps, 6), br = 1 << lbr;  // positions of a box

  if (threadIdx.x == 0) {
    T.abort = 0;
    for (int i = 0; i < kPaStages; ++i) {
      mbar_init(&T.full[i], 1);
      mbar_init(&T.empty[i], kPaWarps);
      mbar_init(&T.told[i], 1);
    }
    fence_mbar_init();
    prefetch_tensormap(&A.km);
    prefetch_tensormap(&A.vm);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) A.rec[cta * 2].np = A.rec[cta * 2 + 1].np = 0;  // no parts yet
  for (int b = threadIdx.x; b < P.n_seqs; b += kPaThreads) plan[b] = pa_seq(a, b, cta == 0 ? P.err : nullptr);
  __syncthreads();

  volatile int* abort = &T.abort;
  if (warp == kPaWarps) {
    // ---------------------------------------------------------------- producer
    // lane l sums the sequences [l k, (l + 1) k); the lane that holds the
    // CTA's first slot finds its sequence
    auto slots = [&](int nch) { return nch > 0 ? (long long)P.nkv * (nch + kPaUnit) : 0LL; };
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
      return small ? (long long)((unsigned)x / (unsigned)y) : x / y;
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

    const uint64_t pol = policy_evict_first();
    const int lnb = 6 - lbr;  // log2 of a chunk's boxes
    int st = 0;
    // A stage: its description (written by lane 0) and its bytes; false: given up.
    auto begin = [&]() {
      const int sl = st % kPaStages;
      bool ok = true;
      if (st >= kPaStages)
        ok = !*abort && pa_wait(&T.empty[sl], (uint32_t)(st / kPaStages - 1) & 1u, A.wait_ns, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (!ok) *abort = 1;
      return ok;
    };
    bool live = true;
    int kvh = s.nch > 0 ? (int)div(w0 - base, s.nch + kPaUnit) : 0;
    // page cache: lane l holds box l & (boxes - 1) of chunk cj + (l >> lnb) of sequence cb
    int cb = -1, cj = 0, crow = 0;
    bool cload = false;
    while (live) {
      const int span = s.nch + kPaUnit;
      const long long rs = base + (long long)kvh * span + kPaUnit, re = rs + s.nch;  // the unit's chunks
      if (rs >= w1 || w0 >= w1) break;
      const int j0 = rs >= w0 ? 0 : (int)(w0 - rs), j1 = (int)(min(re, w1) - rs);
      int cf = 0, np = 1;
      if (rs < w0 || re > w1) {
        cf = (int)div((rs + 1) * G - 1, W);
        np = (int)div(re * G - 1, W) - cf + 1;
      }
      for (int j = j0; j < j1; ++j) {
        if (b != cb || j < cj || j >= cj + (32 >> lnb)) {
          cb = b;
          cj = j;
          const int c = j + (lane >> lnb);
          const int p0 = (c < s.np ? s.cp + c : s.cm + c - s.np) * kPaChunk + ((lane & ((1 << lnb) - 1)) << lbr);
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
        const int pos0 = (j < s.np ? s.cp + j : s.cm + j - s.np) * kPaChunk, sp = pos0 + 16 * (lane & 3);
        const unsigned any = __ballot_sync(0xffffffffu, pa_any(s.len, s.n, s.first, s.prefix, a.window, sp, sp + 15));
        const unsigned all = __ballot_sync(0xffffffffu, pa_all(s.len, s.n, s.first, s.prefix, a.window, sp, sp + 15));
        const int sl = st % kPaStages;
        if (lane == 0) {
          PaDesc& d = T.desc[sl];
          d.q0 = s.q0;
          d.n = s.n;
          d.len = s.len;
          d.kvh = kvh;
          d.pos0 = pos0;
          d.first = s.first;
          d.prefix = s.prefix;
          d.flags = (j == j1 - 1 ? kPaLast : 0) | (int)(any & 15u) << kPaAny | (int)(all & 15u) << kPaAll;
          d.cf = cf;
          d.np = np;
          d.slot = rs >= w0;
          mbar_arrive(&T.told[sl]);
          mbar_arrive_expect_tx(&T.full[sl], __popc(boxes) * (uint32_t)(br * 512));
        }
        __syncwarp();
        if (load) {
          unsigned char* dst = smem + (size_t)sl * kPaStageBytes + (lane & ((1 << lnb) - 1)) * (br * 256);
          const int row = crow + (kvh << P.lps);
          tma_load_3d(dst, &A.km, 0, row, 0, &T.full[sl], pol);
          tma_load_3d(dst + kPaHalf, &A.vm, 0, row, 0, &T.full[sl], pol);
        }
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
    if (live && (live = begin())) {
      if (lane == 0) {
        T.desc[st % kPaStages].flags = kPaEnd;
        mbar_arrive(&T.told[st % kPaStages]);
        mbar_arrive(&T.full[st % kPaStages]);
      }
      ++st;
    }
    __syncwarp();
    __syncthreads();  // every warp is done with the ring
    if (*abort && lane == 0) {
      atomicCAS(P.err, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
      for (int i = max(0, st - kPaStages); i < st; ++i)
        mbar_wait_drain(&T.full[i % kPaStages], (uint32_t)(i / kPaStages) & 1u, kPaDrainNs);
    }
    return;
  }

  // ------------------------------------------------------------------ compute
  const int g = lane >> 2, t = lane & 3;
  const int tile = warp % MT, part = warp / MT;
  const int lj = lane >> 3, lr = lane & 7;
  auto sync = [&](bool fail) { return pa_sync<PARTS * 32>(tile, fail); };
  float* t_m = T.m + tile * 16 * PARTS;
  const uint32_t p_hi = smem_addr(s_p + tile * 4096);  // lo 2048 bytes on
  const uint32_t hb = br * 128;                        // bytes of a box's dim half
  const uint32_t q_s = smem_addr(s_p + (MT + tile) * 4096);
  uint32_t qa[QS ? 1 : 8][4];
  float m[2], l[2], o[2 * MT][4], slope[2] = {0.f, 0.f};
  int rp[2] = {0, 0};  // positions of this thread's two rows
  bool fresh = true;  // a segment begins

  for (int st = 0;; ++st) {
    const int sl = st % kPaStages;
    const uint32_t par = (uint32_t)(st / kPaStages) & 1u;
    const PaDesc& D = T.desc[sl];
    bool ok = !*abort;
    if (fresh) {  // the rows are loaded while the keys are on their way
      ok = ok && pa_wait(&T.told[sl], par, A.wait_ns, abort);
      ok = __all_sync(0xffffffffu, ok);
      if (ok && !(D.flags & kPaEnd)) {
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          const int i = 16 * tile + g + 8 * hr;
          const uint32_t* q = nullptr;
          rp[hr] = D.len;
          if (i < D.n * a.group) {
            const int r = i / a.group, h = D.kvh * a.group + i - r * a.group;
            q = reinterpret_cast<const uint32_t*>(a.q + (D.q0 + r) * a.qs + h * 128);
            rp[hr] += r;
            if (a.slopes) slope[hr] = a.slopes[h] * 1.4426950408889634f;
          }
          if constexpr (!QS) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
              qa[ks][hr] = q ? q[8 * ks + t] : 0u;
              qa[ks][2 + hr] = q ? q[8 * ks + 4 + t] : 0u;
            }
          }
          m[hr] = -INFINITY;
          l[hr] = 0.f;
        }
#pragma unroll
        for (int nb = 0; nb < 2 * MT; ++nb)
#pragma unroll
          for (int c = 0; c < 4; ++c) o[nb][c] = 0.f;
        if constexpr (QS) {
          for (int u = part * 32 + lane; u < 256; u += PARTS * 32) {
            const int row = u >> 4, i = 16 * tile + row;
            uint4 v = make_uint4(0u, 0u, 0u, 0u);
            if (i < D.n * a.group) {
              const int r = i / a.group, h = D.kvh * a.group + i - r * a.group;
              v = *reinterpret_cast<const uint4*>(a.q + (D.q0 + r) * a.qs + h * 128 + 8 * (u & 15));
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(q_s + row * 256 + (((u & 15) ^ (row & 7)) << 4)),
                         "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w)
                         : "memory");
          }
          if (!sync(!ok)) break;
        }
      }
    }
    ok = ok && pa_wait(&T.full[sl], par, A.wait_ns, abort);
    if (!__all_sync(0xffffffffu, ok)) {
      *abort = 1;
      sync(true);
      break;
    }
    const int flags = D.flags, pos0 = D.pos0;
    fresh = (flags & kPaLast) != 0;
    if (flags & kPaEnd) {
      sync(false);
      break;
    }
    const int nrow = D.n * a.group;
    const bool live = 16 * tile < nrow;  // the tile has rows
    if (live) {
      const uint32_t stage = smem_addr(smem + (size_t)sl * kPaStageBytes);
      auto row_at = [&](int r) { return stage + ((r >> lbr) << (lbr + 8)) + (r & (br - 1)) * 128; };
      auto seen = [&](int hr, int p) {
        return p <= rp[hr] && p >= D.first && (a.window == 0 || p > rp[hr] - a.window || p < D.prefix);
      };
      // S: this warp's 8 MT positions (odd k-steps in a chain of their own)
      float sc[MT][4], sd[MT][4];
#pragma unroll
      for (int nb = 0; nb < MT; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[nb][c] = sd[nb][c] = 0.f;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        if constexpr (QS) {
          const uint32_t at = q_s + (lr + 8 * (lj & 1)) * 256;
          pa_ldsm(at + (((4 * q + (lj >> 1)) ^ lr) << 4), qa[0]);
        }
        uint32_t qb[4];
        if constexpr (QS) pa_ldsm(q_s + (lr + 8 * (lj & 1)) * 256 + (((4 * q + 2 + (lj >> 1)) ^ lr) << 4), qb);
#pragma unroll
        for (int nb = 0; nb < MT; ++nb) {
          uint32_t f[4];  // dims 32 q + 0-7, 8-15, 16-23, 24-31
          pa_ldsm(row_at(8 * (MT * part + nb)) + lr * 128 + (q >> 1) * hb + (((4 * (q & 1) + lj) ^ lr) << 4), f);
          if constexpr (QS) {
            pa_mma(sc[nb], qa[0], f[0], f[1]);
            pa_mma(sd[nb], qb, f[2], f[3]);
          } else {
            pa_mma(sc[nb], qa[2 * q], f[0], f[1]);
            pa_mma(sd[nb], qa[2 * q + 1], f[2], f[3]);
          }
        }
      }
#pragma unroll
      for (int nb = 0; nb < MT; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) sc[nb][c] += sd[nb][c];
      // scores in the log2 domain: (row g + 8 (c >> 1), position 8 nb + 2t + (c & 1))
#pragma unroll
      for (int nb = 0; nb < MT; ++nb) {
        const int w = 8 * (MT * part + nb), pb = pos0 + w;
        if (a.plain) {
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nb][c] *= a.scale_log2;
        } else {
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            // tanh(z) = 1 - 2 / (e^2z + 1): off by an FP32 rounding of 1, an
            // absolute error, which is what a score needs
            float x = sc[nb][c] * a.scale_log2;
            if (a.cap_log2 > 0.f) x = a.cap_log2 * (1.f - 2.f * rcp(ex2(sc[nb][c] * a.cap_in) + 1.f));
            sc[nb][c] = x + slope[c >> 1] * (float)(pb + 2 * t + (c & 1) - rp[c >> 1]);
          }
        }
        if (!(flags >> (kPaAll + (w >> 4)) & 1)) {
          const bool some = flags >> (kPaAny + (w >> 4)) & 1;  // else its page may not even be loaded
#pragma unroll
          for (int c = 0; c < 4; ++c)
            if (!some || !seen(c >> 1, pb + 2 * t + (c & 1))) sc[nb][c] = -INFINITY;
        }
      }
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        float v = -INFINITY;
#pragma unroll
        for (int nb = 0; nb < MT; ++nb) v = fmaxf(v, fmaxf(sc[nb][2 * hr], sc[nb][2 * hr + 1]));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
        v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
        if (t == 0) t_m[(g + 8 * hr) * PARTS + part] = v;
      }
      if (!sync(false)) break;
      float al[2];
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        float mx = m[hr];
#pragma unroll
        for (int w = 0; w < PARTS; ++w) mx = fmaxf(mx, t_m[(g + 8 * hr) * PARTS + w]);
        const float ref = mx == -INFINITY ? 0.f : mx;  // nothing visible yet
        al[hr] = ex2(m[hr] - ref);
        m[hr] = mx;
        l[hr] *= al[hr];
#pragma unroll
        for (int nb = 0; nb < MT; ++nb) {
          const float x = ex2(sc[nb][2 * hr] - ref), y = ex2(sc[nb][2 * hr + 1] - ref);
          l[hr] += x + y;
          const uint32_t hi = pa_pack(x, y);
          const uint32_t lo = pa_pack(x - __uint_as_float(hi << 16), y - __uint_as_float(hi & 0xFFFF0000u));
          const uint32_t at = p_hi + (g + 8 * hr) * 128 + (((MT * part + nb) ^ g) << 4) + 4 * t;
          asm volatile("st.shared.u32 [%0], %1;\n st.shared.u32 [%0 + 2048], %2;" ::"r"(at), "r"(hi), "r"(lo) : "memory");
        }
      }
      if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
        for (int nb = 0; nb < 2 * MT; ++nb) {
          o[nb][0] *= al[0];
          o[nb][1] *= al[0];
          o[nb][2] *= al[1];
          o[nb][3] *= al[1];
        }
      }
      if (!sync(false)) break;
      // O: this warp's 16 MT dims over the chunk's positions
      int odd_slices = 0;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        if (!(flags >> (kPaAny + ks) & 1)) continue;
        uint32_t ph[4], pl[4];
        const uint32_t at = p_hi + (lr + 8 * (lj & 1)) * 128 + (((2 * ks + (lj >> 1)) ^ lr) << 4);
        pa_ldsm(at, ph);
        pa_ldsm(at + 2048, pl);
        const uint32_t vrow = row_at(16 * ks) + kPaHalf;
        uint32_t vb[MT][4];  // (positions 0-7 | 8-15) x (dims 0-7 | 8-15) of each 16 dims
        bool odd = false;
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          const int c = 2 * (MT * part + n) + (lj >> 1);
          pa_ldsm_t(vrow + (c >> 3) * hb + (8 * (lj & 1) + lr) * 128 + (((c & 7) ^ lr) << 4), vb[n]);
        }
        if (!(flags >> (kPaAll + ks) & 1)) {
#pragma unroll
          for (int n = 0; n < MT; ++n)
#pragma unroll
            for (int u = 0; u < 4; ++u) odd |= __vcmpeq2(vb[n][u] & 0x7F807F80u, 0x7F807F80u) != 0u;
          odd = __any_sync(0xffffffffu, odd);
        }
        if (odd) {
          odd_slices |= 1 << ks;
          continue;
        }
#pragma unroll
        for (int n = 0; n < MT; ++n) {
          pa_mma(o[2 * n], ph, vb[n][0], vb[n][1]);
          pa_mma(o[2 * n + 1], ph, vb[n][2], vb[n][3]);
          pa_mma(o[2 * n], pl, vb[n][0], vb[n][1]);
          pa_mma(o[2 * n + 1], pl, vb[n][2], vb[n][3]);
        }
      }
      // slices with infinite or NaN values: element by element over the visible positions
#pragma unroll 1
      for (int pp = 0; odd_slices && pp < kPaChunk; ++pp) {
        if (!(odd_slices >> (pp >> 4) & 1)) continue;
        float p[2];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          uint16_t hi, lo;
          const uint32_t e = p_hi + (g + 8 * hr) * 128 + (((pp >> 3) ^ g) << 4) + 2 * (pp & 7);
          asm volatile("ld.shared.u16 %0, [%2];\n ld.shared.u16 %1, [%2 + 2048];" : "=h"(hi), "=h"(lo) : "r"(e));
          p[hr] = bf16_bits_to_float(hi) + bf16_bits_to_float(lo);
        }
        const bool see0 = seen(0, pos0 + pp), see1 = seen(1, pos0 + pp);
        const uint32_t vrow = row_at(pp) + kPaHalf + 4 * t;
#pragma unroll
        for (int nb = 0; nb < 2 * MT; ++nb) {
          const int c = 2 * MT * part + nb;
          uint32_t v;
          asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(vrow + (c >> 3) * hb + (((c & 7) ^ (pp & 7)) << 4)));
          const float v0 = __uint_as_float(v << 16), v1 = __uint_as_float(v & 0xFFFF0000u);
          if (see0) {
            o[nb][0] += p[0] * v0;
            o[nb][1] += p[0] * v1;
          }
          if (see1) {
            o[nb][2] += p[1] * v0;
            o[nb][3] += p[1] * v1;
          }
        }
      }
    }
    if (!(flags & kPaLast)) {
      __syncwarp();
      if (lane == 0) mbar_arrive(&T.empty[sl]);
      continue;
    }

    // the segment's end: the row's sum over its parts, then the output or this CTA's part of it
    if (live) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
        l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
        if (t == 0) t_m[(g + 8 * hr) * PARTS + part] = l[hr];
      }
      if (!sync(false)) break;
      float sum[2] = {0.f, 0.f};
#pragma unroll
      for (int hr = 0; hr < 2; ++hr)
#pragma unroll
        for (int w = 0; w < PARTS; ++w) sum[hr] += t_m[(g + 8 * hr) * PARTS + w];
      if (!sync(false)) break;  // the next chunk's maxima may come
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int i = 16 * tile + g + 8 * hr;
        if (i >= nrow) continue;
        const float L = sum[hr];
        if (D.np == 1) {
          const int r = i / a.group, h = D.kvh * a.group + i - r * a.group;
          const float inv = L == 0.f ? 0.f : 1.f / L;
          uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (D.q0 + r) * a.os + h * 128 + 16 * MT * part);
#pragma unroll
          for (int nb = 0; nb < 2 * MT; ++nb) out[4 * nb + t] = pa_pack(o[nb][2 * hr] * inv, o[nb][2 * hr + 1] * inv);
          if (a.lse && t == 0 && part == 0)
            a.lse[(size_t)(D.q0 + r) * a.nq + h] = L == 0.f ? -INFINITY : (m[hr] + log2f(L)) * 0.6931471805599453f;
        } else {
          const size_t row = (size_t)(cta * 2 + D.slot) * (16 * MT) + i;
          float2* po = reinterpret_cast<float2*>(A.part_o + row * 128 + 16 * MT * part);
#pragma unroll
          for (int nb = 0; nb < 2 * MT; ++nb) __stcg(po + 4 * nb + t, make_float2(o[nb][2 * hr], o[nb][2 * hr + 1]));
          if (t == 0 && part == 0) __stcg(reinterpret_cast<float2*>(A.part_ml + 2 * row), make_float2(m[hr], L));
        }
      }
    }
    if (D.np > 1 && threadIdx.x == 0) A.rec[cta * 2 + D.slot] = {D.cf, D.np, D.q0, D.n, D.kvh};
    __syncwarp();
    if (lane == 0) mbar_arrive(&T.empty[sl]);
  }
  __syncthreads();  // the ring is free
}

// The join of cut units: CTA c takes its share of the rows of the (at most
// two) units it had a part of, row i going to part i mod np.  Up to eight
// parts: a warp per row; more: the CTA's warps share a row's parts.  Either
// way a row's loads are all in flight at once (for up to 64 parts), and the
// parts are added in a fixed order.
constexpr int kPjWarps = 8;

__global__ void __launch_bounds__(kPjWarps * 32) k_paged_join(const __grid_constant__ PagedAttnParams A, int rows) {
  __shared__ float s_l[kPjWarps];
  __shared__ float4 s_v[kPjWarps][32];
  const PagedAttnArgs& a = A.a;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  PagedPart both[2] = {A.rec[c * 2], A.rec[c * 2 + 1]};
#pragma unroll
  for (int slot = 0; slot < 2; ++slot) {
    const PagedPart R = both[slot];
    if (R.np < 2) continue;
    const int nrow = R.n * a.group, p = c - R.cf;
    const bool wide = R.np > 8;
    auto part = [&](int u, int i) { return (size_t)((R.cf + u) * 2 + (u == 0)) * rows + i; };
    auto put = [&](int i, float M, float L, float4 v) {
      const int r = i / a.group, h = R.kvh * a.group + i - r * a.group;
      const float inv = L == 0.f ? 0.f : 1.f / L;
      *reinterpret_cast<uint2*>(a.o + (R.q0 + r) * a.os + h * 128 + 4 * lane) =
          make_uint2(pa_pack(v.x * inv, v.y * inv), pa_pack(v.z * inv, v.w * inv));
      if (a.lse && lane == 0)
        a.lse[(size_t)(R.q0 + r) * a.nq + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
    };
    for (int i = p + (wide ? 0 : R.np * warp); i < nrow; i += wide ? R.np : kPjWarps * R.np) {
      // this warp's parts of row i: u0, u0 + du, ...
      const int u0 = wide ? warp : 0, du = wide ? kPjWarps : 1;
      float M = -INFINITY, L = 0.f;
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      for (int b = u0; b < R.np || b == u0; b += 8 * du) {
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = b + k * du < R.np ? __ldcg(reinterpret_cast<const float4*>(A.part_o + part(b + k * du, i) * 128) + lane)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < 8 && b + lane * du < R.np)
          ml = __ldcg(reinterpret_cast<const float2*>(A.part_ml + 2 * part(b + lane * du, i)));
        if (b == u0) {  // the row's maximum, over all parts
          for (int u = lane; u < R.np; u += 32) M = fmaxf(M, __ldcg(A.part_ml + 2 * part(u, i)));
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
        }
        const float f = ml.x == -INFINITY ? 0.f : ex2(ml.x - M), fl = f * ml.y;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float w = __shfl_sync(0xffffffffu, f, k);
          L += __shfl_sync(0xffffffffu, fl, k);
          v.x += x[k].x * w;
          v.y += x[k].y * w;
          v.z += x[k].z * w;
          v.w += x[k].w * w;
        }
      }
      if (!wide) {
        put(i, M, L, v);
        continue;
      }
      s_v[warp][lane] = v;
      if (lane == 0) s_l[warp] = L;
      __syncthreads();
      if (warp == 0) {
        for (int w = 1; w < kPjWarps; ++w) {
          const float4 x = s_v[w][lane];
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
          L += s_l[w];
        }
        put(i, M, L, v);
      }
      __syncthreads();
    }
  }
}

cudaError_t launch_paged_attention(const PagedAttnParams& A, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int want = 2 * num_sms();
  cfg.gridDim = dim3(want < kPagedMaxCtas ? want : kPagedMaxCtas);
  cfg.blockDim = dim3(kPaThreads);
  const int rows = A.a.max_rows * A.a.group, MT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const size_t smem = kPaStages * kPaStageBytes + (MT == 1 ? 1 : 4) * 4096 + sizeof(PaTable);
  static_assert(2 * (kPaStages * kPaStageBytes + 4 * 4096 + sizeof(PaTable) + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(sizeof(PaSeq) * kPagedMaxSeqs <= kPaStages * kPaStageBytes, "the plan fits the ring");
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) e = max_carveout(kern);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, A) : e;
  };
  const cudaError_t e = MT == 1 ? run(k_paged_attn<1>) : MT == 2 ? run(k_paged_attn<2>) : run(k_paged_attn<4>);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(kPjWarps * 32);
  cfg.dynamicSmemBytes = 0;
  max_carveout(k_paged_join);
  return cudaLaunchKernelEx(&cfg, k_paged_join, A, 16 * MT);
}

}  // namespace moe
