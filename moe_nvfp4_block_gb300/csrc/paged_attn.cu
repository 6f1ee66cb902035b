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
// of its parts through one SM: 37 us against 23 for 4 rows at 16,384
// positions.  CTAs that wait for one another would need the whole GPU.)
// 64 sequences of 500 to 16,000 positions (one row, 32 query and 8 KV heads)
// take 183 us: 6.5 TB/s, 96% of a copy's bandwidth.  One chunk a CTA takes 9.6
// us: 2.6 from the launch to the first load (the sequences, then the table, one
// after another), a first load of 1 to 4 (every CTA fills its ring), and the
// second kernel.  (The table or the queries brought to L2 beforehand gain
// nothing: the first loads of all CTAs fill the memory's time by themselves.)
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
// = hi + lo to 2^-16: one bf16 P would add as much error as the output's own
// rounding; the second product is free while the loads bound the kernel).
//
// Hidden positions: a score is replaced by -inf, and as 0 * v is not 0 for
// an infinite or NaN v, a slice with hidden positions is looked over for such
// values first and, with any, summed element by element over the visible
// positions alone.
#include "paged_attn.cuh"

namespace moe {

namespace {

constexpr int kPaWarps = 8;                      // compute warps
constexpr int kPaThreads = (kPaWarps + 1) * 32;  // and the producer
constexpr int kPaStages = 3;
// Slots before a unit's chunks (two: 29.7 us against 28.9 for 17 documents with a
// bias by distance, 32.1 against 30.8 for 32 sequences with a window of 512).
constexpr int kPaUnit = 1;

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
  PaRing<kPaStages> ring;
  uint64_t told[kPaStages];  // the description is written (the data may still be on its way)
  PaDesc desc[kPaStages];
  float m[kPaWarps * 16];  // [tile][row][part]: maxima of the parts' scores; at a segment's end their sums
};

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
    T.ring.abort = 0;
    for (int i = 0; i < kPaStages; ++i) {
      mbar_init(&T.ring.full[i], 1);
      mbar_init(&T.ring.empty[i], kPaWarps);
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

  volatile int* abort = &T.ring.abort;
  if (warp == kPaWarps) {
    struct Out {
      const PagedAttnParams& A;
      PaTable& T;
      unsigned char* ring;
      uint64_t pol;
      int lane, br, window;
      __device__ bool begin(const PaSegment&, int) { return true; }
      __device__ void stage(const PaSegment& g, int j, int st, uint32_t bytes) {
        const PaSeq& s = g.s;
        const int pos0 = g.pos(j), sp = pos0 + 16 * (lane & 3), sl = st % kPaStages;
        const unsigned any = __ballot_sync(0xffffffffu, pa_any(s.len, s.n, s.first, s.prefix, window, sp, sp + 15));
        const unsigned all = __ballot_sync(0xffffffffu, pa_all(s.len, s.n, s.first, s.prefix, window, sp, sp + 15));
        if (lane != 0) return;
        T.desc[sl] = {s.q0, s.n, s.len, g.kvh, pos0, s.first, s.prefix,
                      (j == g.j1 - 1 ? kPaLast : 0) | (int)(any & 15u) << kPaAny | (int)(all & 15u) << kPaAll,
                      g.cf, g.np, g.slot, 0};
        mbar_arrive(&T.told[sl]);
        mbar_arrive_expect_tx(&T.ring.full[sl], bytes);
      }
      __device__ void put(int sl, int box, int row, uint64_t* bar) {
        unsigned char* dst = ring + (size_t)sl * kPaStageBytes + box * (br * 256);
        tma_load_3d(dst, &A.km, 0, row, 0, bar, pol);
        tma_load_3d(dst + kPaHalf, &A.vm, 0, row, 0, bar, pol);
      }
      __device__ bool end(int st) {
        if (lane == 0) {
          T.desc[st % kPaStages].flags = kPaEnd;
          mbar_arrive(&T.told[st % kPaStages]);
          mbar_arrive(&T.ring.full[st % kPaStages]);
        }
        return true;
      }
    };
    const int st = pa_produce<kPaUnit>(A, T.ring, plan, cta, lane, Out{A, T, smem, policy_evict_first(), lane, br, a.window});
    __syncthreads();  // every warp is done with the ring
    if (*abort && lane == 0) pa_drain(T.ring, st, P.err);
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
    ok = ok && pa_wait(&T.ring.full[sl], par, A.wait_ns, abort);
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
          if (a.cap_log2 > 0.f) {
            pa_capped(a, sc[nb][0], sc[nb][1]);
            pa_capped(a, sc[nb][2], sc[nb][3]);
          } else {
#pragma unroll
            for (int c = 0; c < 4; ++c) sc[nb][c] *= a.scale_log2;
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) sc[nb][c] += slope[c >> 1] * (float)(pb + 2 * t + (c & 1) - rp[c >> 1]);
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
          uint32_t hi, lo;
          pa_split(x, y, hi, lo);
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
      if (lane == 0) mbar_arrive(&T.ring.empty[sl]);
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
          const float inv = pa_inverse(L);
          uint32_t* out = reinterpret_cast<uint32_t*>(a.o + (D.q0 + r) * a.os + h * 128 + 16 * MT * part);
#pragma unroll
          for (int nb = 0; nb < 2 * MT; ++nb) out[4 * nb + t] = pack_bf16(o[nb][2 * hr] * inv, o[nb][2 * hr + 1] * inv);
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
    if (lane == 0) mbar_arrive(&T.ring.empty[sl]);
  }
  __syncthreads();  // the ring is free
}

// The join of cut units: CTAs (c, slot, y) share the rows of the unit that CTA
// c of the attention left in `slot`, row i going to part i mod np.  Up to eight
// parts: a warp per row; more: the CTA's warps share a row's parts.  Either
// way a row's loads are all in flight at once (for up to 64 parts), a warp has
// about one row (several one after another, both slots in one CTA: 122 us
// against 110 for 64 sequences of 300 to 3000 positions and 64 query rows),
// and the parts are added in a fixed order.
constexpr int kPjWarps = 8;

__global__ void __launch_bounds__(kPjWarps * 32) k_paged_join(const __grid_constant__ PagedAttnParams A, int rows) {
  __shared__ float s_l[kPjWarps];
  __shared__ float4 s_v[kPjWarps][32];
  const PagedAttnArgs& a = A.a;
  const int c = blockIdx.x, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  pdl_wait();
  pdl_launch_dependents();
  const PagedPart R = A.rec[c * 2 + blockIdx.y];
  if (R.np < 2) return;
  const int y = blockIdx.z, ny = gridDim.z;
  const int nrow = R.n * a.group, p = c - R.cf;
  const bool wide = R.np > 8;
  auto part = [&](int u, int i) { return (size_t)((R.cf + u) * 2 + (u == 0)) * rows + i; };
  auto put = [&](int i, float M, float L, float4 v) {
    const int r = i / a.group, h = R.kvh * a.group + i - r * a.group;
    const float inv = pa_inverse(L);
    *reinterpret_cast<uint2*>(a.o + (R.q0 + r) * a.os + h * 128 + 4 * lane) =
        make_uint2(pack_bf16(v.x * inv, v.y * inv), pack_bf16(v.z * inv, v.w * inv));
    if (a.lse && lane == 0)
      a.lse[(size_t)(R.q0 + r) * a.nq + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
  };
  for (int i = p + R.np * (wide ? y : warp + kPjWarps * y); i < nrow; i += R.np * ny * (wide ? 1 : kPjWarps)) {
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

cudaError_t launch_paged_attention(const PagedAttnParams& A, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  const int want = paged_attention_tc(A.a) ? num_sms() : 2 * num_sms();
  cfg.gridDim = dim3(want < kPagedMaxCtas ? want : kPagedMaxCtas);
  cfg.blockDim = dim3(kPaThreads);
  const int rows = A.a.max_rows * A.a.group, MT = rows <= 16 ? 1 : rows <= 32 ? 2 : 4;
  const size_t smem = kPaStages * kPaStageBytes + (MT == 1 ? 1 : 4) * 4096 + sizeof(PaTable);  // P, and with MT 2 Q
  static_assert(2 * (kPaStages * kPaStageBytes + 4 * 4096 + sizeof(PaTable) + 1024) <= 228 * 1024, "two CTAs an SM");
  static_assert(sizeof(PaSeq) * kPagedMaxSeqs <= kPaStages * kPaStageBytes, "the plan fits the ring");
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  auto run = [&](auto kern, cudaError_t e) { return e == cudaSuccess ? cudaLaunchKernelEx(&cfg, kern, A) : e; };
  const cudaError_t e = paged_attention_tc(A.a) ? launch_paged_attention_tc(A, 16 * MT, s)
                        : MT == 1 ? run(k_paged_attn<1>, prepare_kernel<k_paged_attn<1>>((int)smem))
                                  : run(k_paged_attn<2>, prepare_kernel<k_paged_attn<2>>((int)smem));
  if (e != cudaSuccess) return e;
  cfg.gridDim.y = 2;
  cfg.gridDim.z = MT;
  cfg.blockDim = dim3(kPjWarps * 32);
  cfg.dynamicSmemBytes = 0;
  const cudaError_t ej = prepare_kernel<k_paged_join>(0);
  return ej == cudaSuccess ? cudaLaunchKernelEx(&cfg, k_paged_join, A, 16 * MT) : ej;
}

}  // namespace moe
