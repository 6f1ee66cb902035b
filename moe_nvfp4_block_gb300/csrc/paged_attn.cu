// paged_attn.cu -- attention of verify rows over a paged KV cache.
//
// For row t of sequence b (position pos = kv_len[b] + i) and query head h:
//   s_p = score(q . k_p),  o = sum_p exp(s_p - m) v_p / sum_p exp(s_p - m)
// over the visible positions p, in one pass with a running maximum m (in the
// log2 domain) and, where a sequence is cut, a join of the parts' (m, l, o).
//
// What bounds it: each visible position's keys and values (512 bytes a KV
// head) are read once.  The work of a call is the list of all 64-position
// chunks of all (sequence, KV head) units; CTA c of G (two an SM) takes the
// chunks [c W / G, (c + 1) W / G) of the W, whatever units they fall in, so
// that unequal lengths cost no balance (with W < G the first W take one each).  A unit inside one CTA is written out
// there; the parts of a cut unit go to the workspace (at most two a CTA) and
// are joined, in CTA order, by a second kernel whose CTAs share the rows.
// (The join by the unit's last CTA to arrive, in the same kernel, reads all
// of its parts through one SM: 37 us against 21 for 4 rows at 16,384
// positions.  CTAs that wait for one another would need the whole GPU.)
//
// A producer warp walks the chunks: it looks up their pages (a chunk is one
// half or whole page, or several) and loads keys and values by TMA into a
// ring of three 32 KB stages, with a description of the chunk beside it.
// Four warps compute.  The unit's rows (verify rows x heads of the KV head)
// are MT tiles of 16; a warp has one tile and every (4 / MT)th 16-position
// slice of a chunk: S = Q K^T and O += P V by mma.sync m16n8k16, with P split
// into two bf16 parts (P = hi + lo to 2^-17: one bf16 P would add as much
// error as the output's own rounding; the second product is free while the
// loads bound the kernel).
//
// Hidden positions: a score is replaced by -inf, and as 0 * v is not 0 for
// an infinite or NaN v, a slice with hidden positions is looked over for such
// values first and, with any, summed element by element over the visible
// positions alone.
#include "internal.h"
#include "ptx.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr int kPaWarps = 4;                      // compute warps
constexpr int kPaThreads = (kPaWarps + 1) * 32;  // and the producer
constexpr int kPaChunk = 64;
constexpr int kPaStages = 3;
constexpr int kPaHalf = kPaChunk * 256;          // a stage's keys (or values)
constexpr int kPaStageBytes = 2 * kPaHalf;
constexpr int kPaPitch = 36;                     // floats a row of the merge buffer (32 dims)
constexpr uint64_t kPaDrainNs = 2000000000ull;

// A chunk as its stage's readers see it.
struct PaDesc {
  int q0, n, len, kvh;       // the sequence's first row, rows, committed length; KV head
  int pos0, first, prefix;   // the chunk's first position; the sequence's limits
  int flags;                 // kPaFirst, kPaLast: of the CTA's segment of the unit
  int cf, np;                // np > 1: a cut unit, whose first CTA is cf and whose parts are np
  int slot, pad;             // where this CTA's part goes (0 / 1)
};
constexpr int kPaFirst = 1, kPaLast = 2;

struct PaTable {
  uint64_t full[kPaStages];
  uint64_t empty[kPaStages];
  uint64_t seg;  // the compute warps' own barrier
  PaDesc desc[kPaStages];
  long long w_total;
  int nst;
  int abort;
  float m[kPaWarps][16];
  float l[kPaWarps][16];
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
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
      "{%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pa_pack(float lo, float hi) {
  uint32_t d;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(d) : "f"(hi), "f"(lo));
  return d;
}
__device__ __forceinline__ float ex2(float x) { return exp2f(x); }

}  // namespace

template <int MT>
__global__ void __launch_bounds__(kPaThreads, 2) k_paged_attn(const __grid_constant__ PagedAttnParams A) {
  constexpr int PG = kPaWarps / MT;  // warps (position groups) of a tile
  constexpr int NSL = kPaChunk / 16 / PG;  // slices of a chunk for a warp
  const PagedAttnArgs& a = A.a;
  const PagedRows& P = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  float* s_o = reinterpret_cast<float*>(smem + kPaStages * kPaStageBytes);  // [kPaWarps][16][kPaPitch]
  PaTable& T = *reinterpret_cast<PaTable*>(s_o + kPaWarps * 16 * kPaPitch);
  int* s_nch = reinterpret_cast<int*>(&T + 1);  // [n_seqs]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int cta = blockIdx.x;
  const int lbr = min(P.lps, 6), br = 1 << lbr;  // positions of a box

  if (threadIdx.x == 0) {
    T.abort = 0;
    for (int i = 0; i < kPaStages; ++i) {
      mbar_init(&T.full[i], 1);
      mbar_init(&T.empty[i], kPaWarps);
    }
    mbar_init(&T.seg, kPaWarps);
    fence_mbar_init();
    prefetch_tensormap(&A.km);
    prefetch_tensormap(&A.vm);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (threadIdx.x == 0) A.rec[cta * 2].np = A.rec[cta * 2 + 1].np = 0;  // no parts yet
  for (int b = threadIdx.x; b < P.n_seqs; b += kPaThreads) s_nch[b] = pa_seq(a, b, cta == 0 ? P.err : nullptr).nch;
  __syncthreads();

  volatile int* abort = &T.abort;
  if (warp == kPaWarps) {
    // ---------------------------------------------------------------- producer
    // lane l sums the sequences [l k, (l + 1) k); the lane that holds the
    // CTA's first chunk finds its sequence
    const int k = (P.n_seqs + 31) / 32;
    long long sum = 0;
    for (int i = 0; i < k; ++i)
      if (lane * k + i < P.n_seqs) sum += s_nch[lane * k + i];
    sum *= P.nkv;
    long long inc = sum;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, inc, d);
      if (lane >= d) inc += o;
    }
    const long long W = __shfl_sync(0xffffffffu, inc, 31);
    // no more CTAs than chunks: every one of a cut unit's CTAs has a part
    const int G = (int)min((long long)gridDim.x, W);
    const long long w0 = cta < G ? cta * W / G : W, w1 = cta < G ? (cta + 1) * W / G : W;
    long long base = inc - sum;
    int b = lane * k;
    const bool mine = base <= w0 && w0 < inc;
    if (mine)
      while (base + (long long)P.nkv * s_nch[b] <= w0) base += (long long)P.nkv * s_nch[b++];
    const unsigned who = __ballot_sync(0xffffffffu, mine);
    const int src = who ? __ffs(who) - 1 : 0;
    b = __shfl_sync(0xffffffffu, b, src);
    base = __shfl_sync(0xffffffffu, base, src);
    if (lane == 0) T.nst = (int)(w1 - w0);
    __syncthreads();

    const uint64_t pol = policy_evict_first();
    PaSeq s{};
    int nch = 0, kvh = 0, j = 0;  // of the current unit; j: the chunk
    bool fresh = true;
    int cf = 0, np = 1, slot = 0, st = 0;
    for (; st < (int)(w1 - w0); ++st) {
      const long long w = w0 + st;
      int flags = 0;
      if (st == 0 || j == nch) {  // a new unit
        flags = kPaFirst;
        if (st > 0) {
          j = 0;
          if (++kvh == P.nkv) {
            base += (long long)P.nkv * nch;
            do ++b;
            while (s_nch[b] == 0);
            kvh = 0;
            fresh = true;
          }
        }
        if (fresh) {
          s = pa_seq(a, b, nullptr);
          nch = s_nch[b];
          fresh = false;
          if (st == 0) {
            kvh = (int)((w - base) / nch);
            j = (int)((w - base) - (long long)kvh * nch);
          }
        }
        const long long us = base + (long long)kvh * nch, ue = us + nch;
        slot = us >= w0;
        np = 1;
        if (us < w0 || ue > w1) {
          cf = (int)(((us + 1) * G - 1) / W);
          np = (int)((ue * G - 1) / W) - cf + 1;
        }
      }
      if (j == nch - 1 || st == (int)(w1 - w0) - 1) flags |= kPaLast;
      const int pos0 = (j < s.np ? s.cp + j : s.cm + j - s.np) * kPaChunk;
      ++j;
      // this lane's box of the chunk
      const int p0 = pos0 + (lane << lbr);
      bool load = lane < (kPaChunk >> lbr) && pa_any(s.len, s.n, s.first, s.prefix, a.window, p0, p0 + br - 1);
      int row = 0;
      if (load) {
        int page = P.table[(size_t)b * P.max_pages + (p0 >> P.lps)];
        if (page < 0 || page >= P.n_pages) {
          atomicCAS(P.err, 0, (int)MOE_ERR_INVALID_ARG);
          page = 0;
        }
        row = ((page * P.nkv + kvh) << P.lps) + (p0 & ((1 << P.lps) - 1));
      }
      const unsigned boxes = __ballot_sync(0xffffffffu, load);
      const int sl = st % kPaStages;
      bool ok = true;
      if (st >= kPaStages)
        ok = !*abort && mbar_wait_bounded(&T.empty[sl], (uint32_t)(st / kPaStages - 1) & 1u, A.wait_ns, abort);
      if (!__all_sync(0xffffffffu, ok)) {
        *abort = 1;
        break;
      }
      if (lane == 0) {
        PaDesc& d = T.desc[sl];
        d.q0 = s.q0;
        d.n = s.n;
        d.len = s.len;
        d.kvh = kvh;
        d.pos0 = pos0;
        d.first = s.first;
        d.prefix = s.prefix;
        d.flags = flags;
        d.cf = cf;
        d.np = np;
        d.slot = slot;
        mbar_arrive_expect_tx(&T.full[sl], __popc(boxes) * (uint32_t)(br * 512));
      }
      __syncwarp();
      if (load) {
        unsigned char* dst = smem + (size_t)sl * kPaStageBytes + lane * (br * 256);
        tma_load_3d(dst, &A.km, 0, row, 0, &T.full[sl], pol);
        tma_load_3d(dst + kPaHalf, &A.vm, 0, row, 0, &T.full[sl], pol);
      }
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
  const int tile = warp % MT, pg = warp / MT;
  const int lj = lane >> 3, lr = lane & 7;
  const bool plain = a.softcap == 0.f && !a.slopes;
  const float scale_log2 = a.scale * kLog2e;
  const float cap_in = a.softcap > 0.f ? 2.f * kLog2e * a.scale / a.softcap : 0.f;
  const float cap_log2 = a.softcap * kLog2e;
  uint32_t qa[8][4];
  float m[2], l[2], o[16][4], slope[2] = {0.f, 0.f};
  int rp[2] = {0, 0};  // positions of this thread's two rows
  // Barrier of the compute warps.  Bounded, and left when a warp has given
  // up (a plain barrier would wait for that warp for ever): false then.
  uint32_t seg_parity = 0;
  auto pa_sync = [&]() {
    __syncwarp();
    if (lane == 0) mbar_arrive(&T.seg);
    const bool ok = __all_sync(0xffffffffu, mbar_wait_bounded(&T.seg, seg_parity, A.wait_ns, abort));
    seg_parity ^= 1u;
    if (!ok) *abort = 1;
    return ok;
  };
  __syncthreads();
  const int nst = T.nst;

  for (int st = 0; st < nst; ++st) {
    const int sl = st % kPaStages;
    bool ok = !*abort && mbar_wait_bounded(&T.full[sl], (uint32_t)(st / kPaStages) & 1u, A.wait_ns, abort);
    if (!__all_sync(0xffffffffu, ok)) {
      *abort = 1;
      break;
    }
    const PaDesc d = T.desc[sl];
    const int nrow = d.n * a.group;
    if (d.flags & kPaFirst) {
#pragma unroll
      for (int hr = 0; hr < 2; ++hr) {
        const int i = 16 * tile + g + 8 * hr;
        const uint32_t* q = nullptr;
        rp[hr] = d.len;
        if (i < nrow) {
          const int r = i / a.group, h = d.kvh * a.group + i - r * a.group;
          q = reinterpret_cast<const uint32_t*>(a.q + (d.q0 + r) * a.qs + h * 128);
          rp[hr] = d.len + r;
          if (a.slopes) slope[hr] = a.slopes[h] * kLog2e;
        }
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          qa[ks][hr] = q ? q[8 * ks + t] : 0u;
          qa[ks][2 + hr] = q ? q[8 * ks + 4 + t] : 0u;
        }
        m[hr] = -INFINITY;
        l[hr] = 0.f;
      }
#pragma unroll
      for (int nb = 0; nb < 16; ++nb)
#pragma unroll
        for (int c = 0; c < 4; ++c) o[nb][c] = 0.f;
    }
    const uint32_t stage = smem_addr(smem + (size_t)sl * kPaStageBytes);
    if (16 * tile < nrow) {
      for (int is = 0; is < NSL; ++is) {
        const int row0 = 16 * (pg + PG * is), pb = d.pos0 + row0;
        if (!pa_any(d.len, d.n, d.first, d.prefix, a.window, pb, pb + 15)) continue;
        const bool clear = pa_all(d.len, d.n, d.first, d.prefix, a.window, pb, pb + 15);
        const uint32_t kbase = stage + ((row0 >> lbr) << (lbr + 8)) + (row0 & (br - 1)) * 128;
        const uint32_t vbase = kbase + kPaHalf, hb = br * 128;  // hb: bytes of a box's dim half
        float sc[2][4];
#pragma unroll
        for (int nb = 0; nb < 2; ++nb)
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nb][c] = 0.f;
#pragma unroll
        for (int ks = 0; ks < 8; ++ks) {
          // matrices: (positions 0-7 | 8-15) x (dims lo | hi of the k-step)
          uint32_t kb[4];
          const int rr = 8 * (lj >> 1) + lr, c = (2 * ks + (lj & 1)) & 7;
          pa_ldsm(kbase + (ks >> 2) * hb + rr * 128 + ((c ^ lr) << 4), kb);
          pa_mma(sc[0], qa[ks], kb[0], kb[1]);
          pa_mma(sc[1], qa[ks], kb[2], kb[3]);
        }
        // scores in the log2 domain: (row g + 8 (c >> 1), position 8 nb + 2t + (c & 1))
        if (plain) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nb][c] *= scale_log2;
        } else {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              // tanh(z) = 1 - 2 / (e^2z + 1): off by an FP32 rounding of 1,
              // an absolute error, which is what a score needs
              float x = sc[nb][c] * scale_log2;
              if (a.softcap > 0.f) x = cap_log2 * (1.f - __fdividef(2.f, ex2(sc[nb][c] * cap_in) + 1.f));
              sc[nb][c] = x + slope[c >> 1] * (float)(pb + 8 * nb + 2 * t + (c & 1) - rp[c >> 1]);
            }
        }
        auto seen = [&](int hr, int p) {
          return p <= rp[hr] && p >= d.first && (a.window == 0 || p > rp[hr] - a.window || p < d.prefix);
        };
        if (!clear) {
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if (!seen(c >> 1, pb + 8 * nb + 2 * t + (c & 1))) sc[nb][c] = -INFINITY;
        }
        float al[2];
#pragma unroll
        for (int hr = 0; hr < 2; ++hr) {
          float v = fmaxf(fmaxf(sc[0][2 * hr], sc[0][2 * hr + 1]), fmaxf(sc[1][2 * hr], sc[1][2 * hr + 1]));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 1));
          v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, 2));
          const float mx = fmaxf(m[hr], v);
          const float ref = mx == -INFINITY ? 0.f : mx;  // nothing visible yet
          al[hr] = ex2(m[hr] - ref);
          m[hr] = mx;
          float add = 0.f;
#pragma unroll
          for (int nb = 0; nb < 2; ++nb)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
              sc[nb][2 * hr + c] = ex2(sc[nb][2 * hr + c] - ref);
              add += sc[nb][2 * hr + c];
            }
          l[hr] = l[hr] * al[hr] + add;
        }
        if (__any_sync(0xffffffffu, al[0] != 1.f || al[1] != 1.f)) {
#pragma unroll
          for (int nb = 0; nb < 16; ++nb) {
            o[nb][0] *= al[0];
            o[nb][1] *= al[0];
            o[nb][2] *= al[1];
            o[nb][3] *= al[1];
          }
        }
        // V by transposing ldmatrix: (positions 0-7 | 8-15) x (dims 16 np + 0-7 | 8-15)
        auto load_v = [&](int np, uint32_t(&vb)[4]) {
          const int rr = 8 * (lj & 1) + lr, c = (2 * np + (lj >> 1)) & 7;
          pa_ldsm_t(vbase + (np >> 2) * hb + rr * 128 + ((c ^ lr) << 4), vb);
        };
        bool odd = false;
        if (!clear) {
#pragma unroll
          for (int np = 0; np < 8; ++np) {
            uint32_t vb[4];
            load_v(np, vb);
#pragma unroll
            for (int u = 0; u < 4; ++u) odd |= __vcmpeq2(vb[u] & 0x7F807F80u, 0x7F807F80u) != 0u;
          }
          odd = __any_sync(0xffffffffu, odd);
        }
        if (!odd) {
          uint32_t ph[4], pl[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const float x = sc[u >> 1][2 * (u & 1)], y = sc[u >> 1][2 * (u & 1) + 1];
            ph[u] = pa_pack(x, y);
            pl[u] = pa_pack(x - __uint_as_float(ph[u] << 16), y - __uint_as_float(ph[u] & 0xFFFF0000u));
          }
#pragma unroll
          for (int np = 0; np < 8; ++np) {
            uint32_t vb[4];
            load_v(np, vb);
            pa_mma(o[2 * np], ph, vb[0], vb[1]);
            pa_mma(o[2 * np + 1], ph, vb[2], vb[3]);
            pa_mma(o[2 * np], pl, vb[0], vb[1]);
            pa_mma(o[2 * np + 1], pl, vb[2], vb[3]);
          }
        } else {
          // element by element over the visible positions
          for (int pp = 0; pp < 16; ++pp) {
            const int from = (lane & ~3) | ((pp & 7) >> 1);
            float p[2];
#pragma unroll
            for (int hr = 0; hr < 2; ++hr) {
              const float x0 = pp < 8 ? sc[0][2 * hr] : sc[1][2 * hr], x1 = pp < 8 ? sc[0][2 * hr + 1] : sc[1][2 * hr + 1];
              p[hr] = __shfl_sync(0xffffffffu, (pp & 1) ? x1 : x0, from);
            }
            const bool see0 = seen(0, pb + pp), see1 = seen(1, pb + pp);
#pragma unroll
            for (int nb = 0; nb < 16; ++nb) {
              uint32_t v;
              asm volatile("ld.shared.u32 %0, [%1];"
                           : "=r"(v)
                           : "r"(vbase + (nb >> 3) * hb + pp * 128 + (((nb & 7) ^ (pp & 7)) << 4) + 4 * t));
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
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&T.empty[sl]);
    if (!(d.flags & kPaLast)) continue;

    // ---------------------------------------------------------------- the segment's end
    // The position groups of a tile agree on a maximum; each scales its sums
    // to it, and they are added in group order, 32 dims at a time.
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 1);
      l[hr] += __shfl_xor_sync(0xffffffffu, l[hr], 2);
      if (t == 0) {
        T.m[warp][g + 8 * hr] = m[hr];
        T.l[warp][g + 8 * hr] = l[hr];
      }
    }
    if (!pa_sync()) break;
    float f[2];
#pragma unroll
    for (int hr = 0; hr < 2; ++hr) {
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < PG; ++w) M = fmaxf(M, T.m[tile + MT * w][g + 8 * hr]);
      f[hr] = m[hr] == -INFINITY ? 0.f : ex2(m[hr] - M);
    }
    const bool whole = d.np == 1;
    float* po = A.part_o + (size_t)(cta * 2 + d.slot) * (16 * MT * 128);
    float* pml = A.part_ml + (size_t)(cta * 2 + d.slot) * (16 * MT * 2);
    const int col = (threadIdx.x & 7) * 4, mr = threadIdx.x >> 3;  // this thread's 4 dims and row of a tile
    bool live = true;
#pragma unroll
    for (int dq = 0; dq < 4; ++dq) {
#pragma unroll
      for (int nb = 0; nb < 4; ++nb) {
        float* r0 = s_o + (warp * 16 + g) * kPaPitch + 8 * nb + 2 * t;
        *reinterpret_cast<float2*>(r0) = make_float2(o[4 * dq + nb][0] * f[0], o[4 * dq + nb][1] * f[0]);
        *reinterpret_cast<float2*>(r0 + 8 * kPaPitch) = make_float2(o[4 * dq + nb][2] * f[1], o[4 * dq + nb][3] * f[1]);
      }
      live = pa_sync();
      if (!live) break;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        const int i = 16 * u + mr;
        if (i < nrow) {
          float M = -INFINITY, L = 0.f;
#pragma unroll
          for (int w = 0; w < PG; ++w) M = fmaxf(M, T.m[u + MT * w][mr]);
          float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
          for (int w = 0; w < PG; ++w) {
            const float mw = T.m[u + MT * w][mr];
            L += mw == -INFINITY ? 0.f : T.l[u + MT * w][mr] * ex2(mw - M);
            const float4 x = *reinterpret_cast<const float4*>(s_o + ((u + MT * w) * 16 + mr) * kPaPitch + col);
            v.x += x.x;
            v.y += x.y;
            v.z += x.z;
            v.w += x.w;
          }
          if (whole) {
            const int r = i / a.group, h = d.kvh * a.group + i - r * a.group;
            const float inv = L == 0.f ? 0.f : 1.f / L;
            *reinterpret_cast<uint2*>(a.o + (d.q0 + r) * a.os + h * 128 + 32 * dq + col) =
                make_uint2(pa_pack(v.x * inv, v.y * inv), pa_pack(v.z * inv, v.w * inv));
            if (a.lse && dq == 0 && col == 0)
              a.lse[(size_t)(d.q0 + r) * a.nq + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
          } else {
            __stcg(reinterpret_cast<float4*>(po + i * 128 + 32 * dq + col), v);
            if (dq == 0 && col == 0) __stcg(reinterpret_cast<float2*>(pml + 2 * i), make_float2(M, L));
          }
        }
      }
      live = pa_sync();
      if (!live) break;
    }
    if (!live) break;
    if (whole) continue;

    if (threadIdx.x == 0) A.rec[cta * 2 + d.slot] = {d.cf, d.np, d.q0, d.n, d.kvh};
  }
  __syncthreads();  // the ring is free
}

// The join of cut units: CTA c takes its share of the rows of the (at most
// two) units it had a part of, row i going to part i mod np.  Up to eight
// parts: a warp per row, every load in flight at once; more: the CTA's warps
// share a row's parts.  Parts are added in a fixed order.
__global__ void __launch_bounds__(128) k_paged_join(const __grid_constant__ PagedAttnParams A, int rows) {
  __shared__ float s_l[4];
  __shared__ float4 s_v[4][32];
  const PagedAttnArgs& a = A.a;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  for (int slot = 0; slot < 2; ++slot) {
    const PagedPart R = A.rec[c * 2 + slot];
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
    for (int i = p + (wide ? 0 : R.np * warp); i < nrow; i += wide ? R.np : 4 * R.np) {
      // this warp's parts of row i: u0, u0 + du, ...
      const int u0 = wide ? warp : 0, du = wide ? 4 : 1;
      float M = -INFINITY;
      for (int u = lane; u < R.np; u += 32) M = fmaxf(M, __ldcg(A.part_ml + 2 * part(u, i)));
      float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
      float L = 0.f;
      bool first = true;
      for (int b = u0; b < R.np; b += 8 * du) {
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          x[k] = b + k * du < R.np ? __ldcg(reinterpret_cast<const float4*>(A.part_o + part(b + k * du, i) * 128) + lane)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (lane < 8 && b + lane * du < R.np)
          ml = __ldcg(reinterpret_cast<const float2*>(A.part_ml + 2 * part(b + lane * du, i)));
        if (first) {
#pragma unroll
          for (int d = 16; d >= 1; d >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, d));
          first = false;
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
        L = (s_l[0] + s_l[1]) + (s_l[2] + s_l[3]);
        for (int w = 1; w < 4; ++w) {
          const float4 x = s_v[w][lane];
          v.x += x.x;
          v.y += x.y;
          v.z += x.z;
          v.w += x.w;
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
  cfg.dynamicSmemBytes = kPaStages * kPaStageBytes + sizeof(float) * kPaWarps * 16 * kPaPitch + sizeof(PaTable) +
                         sizeof(int) * A.a.p.n_seqs;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern) {
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, 114 * 1024);
    if (e == cudaSuccess) e = max_carveout(kern);
    return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, A) : e;
  };
  const int rows = A.a.max_rows * A.a.group;
  const cudaError_t e = rows <= 16 ? run(k_paged_attn<1>) : rows <= 32 ? run(k_paged_attn<2>) : run(k_paged_attn<4>);
  if (e != cudaSuccess) return e;
  cfg.blockDim = dim3(128);
  cfg.dynamicSmemBytes = 0;
  max_carveout(k_paged_join);
  return cudaLaunchKernelEx(&cfg, k_paged_join, A, rows <= 16 ? 16 : rows <= 32 ? 32 : 64);
}

}  // namespace moe
