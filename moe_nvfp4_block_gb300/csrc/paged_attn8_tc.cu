// paged_attn8_tc.cu -- the attention over a paged cache of 8 bits on the
// 5th-generation tensor cores, for 33 to 64 query rows a KV head (and, in long
// tables, from 17 on).
//
// The work list, the two softmax groups and the segments' ends are those of
// paged_attn_tc.cu; the formula's scales those of paged_attn8.cu.  Per
// 128-position chunk (32 KB)
//   S [rows, 128]  = Q K^T   8 tcgen05.mma kind::f8f6f4 M128 N128 K32: K as it lies
//                            in the page, Q as two E4M3 parts (hi + lo) of its rows
//                            scaled to below 2^8: exact down to 2^-9 of the row's
//                            largest value, and to 2^-17 of that below.  Q is in
//                            tensor memory, each row twice: a row's two lanes
//                            (threads) take half of the positions each
//   O^T [128, rows] += V^T P^T   8 tcgen05.mma kind::f16 M128 N64 K16: P as in
//                            paged_attn8.cu, V unpacked to FP16 by four warps
// so that a weight keeps its 11 bits (two E4M3 parts of P would lose what many
// positions of 2^-20 of the largest weight add up to).  Shared memory gives 128
// bytes a clock, 180 KB in the time of a chunk at HBM's rate, and a chunk's trips
// through it are 176 KB: Q read from there with every product and O the other
// way round (rows twice there too), 224; K unpacked as well, 272.
//
// Measured: 65,003 and 131,001 positions, 8 KV heads of 64 query rows, 402 MB:
// 92 to 93 us (4.3 TB/s; the bf16 cache 132); 19 sequences of 4096 with 64 rows
// 46 us (58), with a softcap 78, with a bias by distance 73; 64 ragged sequences
// of 64 rows 137; 608 units of one chunk 35.  What paces a chunk is its one producer
// warp: it takes 1900 clocks of the chunk's 2150 (81 chunks a CTA), its scales' eight
// lanes of work with all 32 (by a 16th warp: 100 us).  Instructions come second: 15
// warps of five kinds share an SM's instruction cache (97% hits, an issue in 49% of
// the cycles), and a copy that knew whole chunks of plain scores only had 86, 7%
// less.  The tensor pipe is busy in 39% of the cycles.  Slower, too: 16 softmax warps (80 registers a thread: spills), chunks of
// 64 positions (half the work between the same waits), one pass over the scores with
// the last maximum, weights formed again where it grows (130: the next S waits for
// it), exponentials unrolled twice as far (101), rows of Q by the softmax warps (131).
#include "paged_attn8.cuh"
#include "paged_tc.cuh"

namespace moe {

namespace {

constexpr int kT8Chunk = 128;
constexpr int kT8Half = kT8Chunk * 128;   // a stage's keys (or values)
constexpr int kT8Keys = 3;                // stages of the ring of keys
constexpr int kT8Stages = 4;              // of the ring of values
constexpr int kT8Unit = 4;                // slots before a unit's chunks
constexpr int kT8P = 2 * 8192;            // a group's P: [half of the positions][64 rows][64] f16
constexpr int kT8V = 16384;               // unpacked values of half a chunk: [dim half][64 positions][64 dims]
constexpr int kT8Values = 4;              // of them
constexpr int kT8Cols = 512;              // tensor memory columns
constexpr int kT8S = 0, kT8O = 256, kT8Q = 384;  // S of group g at 128 g, O (transposed) at 256 + 64 g; Q of two segments: hi, lo, 32 columns each
constexpr float kT8Room = 8.f;            // growth of the maximum (log2) that the reference leaves room for
constexpr int kT8Conv = 4;                // warps that bring rows of Q into two parts and unpack values
// Warps: 0-3 and 4-7 softmax of the even and odd chunks, 8 producer, 9 and 10
// products (S; O), 11-14 rows of Q and values.
constexpr int kT8Producer = 8, kT8Mma = 9, kT8MmaO = 10, kT8Values0 = 11;
constexpr int kT8Warps = kT8Values0 + kT8Conv, kT8Threads = 32 * kT8Warps;
constexpr int kT8Segs = 4;                // segments described ahead
constexpr int kT8Readers = kT8Warps - 1;  // of a segment's description: every warp but the producer
// Chunks whose scales are kept: the producer is at most the keys' ring ahead of
// S, and S two chunks ahead of the softmax, which reads them to its chunk's end.
constexpr int kT8Scales = 8;
static_assert(kT8Keys + 2 < kT8Scales, "no scale is written over before it is read");

// A segment as the warps see it: chunks j0 .. j0 + count - 1 of its unit, in
// the ring's stages st0, st0 + 1, ...
struct T8Seg {
  int q0, n, len, kvh, first, prefix;
  int cp, np, cm;  // of PaSeq
  int j0, count, st0;
  int cf, parts, slot;
};

// Rows of a part in the workspace.
__host__ __device__ inline int t8_padded(const PagedAttnArgs& a) { return a.max_rows * a.group > 32 ? 64 : 32; }

struct T8Table {
  PaRing<kT8Stages> ring;                 // (full: keys and values; empty: values)
  uint64_t k_empty[kT8Keys];
  uint64_t told[kT8Segs], read[kT8Segs];  // the segment's description is written; is read by all
  uint64_t rows[kT8Segs];                 // what its rows count (qx) is written
  uint64_t scaled[kT8Scales];             // the scales of a chunk are written
  uint64_t v_full[kT8Values], v_empty[kT8Values];
  T8Seg seg[kT8Segs];
  uint64_t s_full[2], s_empty[2];  // S of group g is there; is read
  uint64_t x_full[2];   // group g's four warps have left what the others need
  uint64_t p_full[2];   // P of group g is there
  uint64_t o_done[2];   // the product with P of group g is done
  uint64_t q_full[2], q_empty[2];  // Q of segment i (mod 2) is there; its last product with it is done
  uint64_t ml_full;     // m and l of a segment of both groups are there
  uint64_t epi_done;    // its outputs are out of tensor memory (a group's first P of the next segment waits)
  uint64_t fin[2];
  uint64_t scale[kT8Scales][2];  // a byte for each 16 positions: keys, values
  int info[kT8Scales];           // p8_scales' of them
  uint32_t tmem;
  uint64_t wait_ns;
  int pv[2];            // slices to multiply (bits 0-7); bit 8: O holds sums already
  int qx[kT8Segs][64];  // row r's values are 2^qx those of the two parts; kP8Nan: it has infinite or NaN ones
  float top[2][2][2][64];  // maxima of the scores: [chunk mod 2][group][half][row]
  float m[2][64], l[2][2][64];  // a segment's end: the groups' references, and their halves' sums
  int odd[2][2][4];     // [chunk mod 2][group][warp] slices where it saw NaN values
  int has[2], vref[2];  // the group has sums; their reference scale
};

// What few chunks need is out of line: all warps' loops together have to stay
// in the instruction cache (in line, a fifth of the fetches missed it, and the
// next one was busy 84% of the time).

// Whether every lane sees phase `parity` of the barrier at shared address `bar` over.
__device__ __forceinline__ bool t8_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n vote.sync.all.pred p, p, 0xffffffff;\n"
      " selp.u32 %0, 1, 0, p;\n}"
      : "=r"(ok)
      : "r"(bar), "r"(parity)
      : "memory");
  return ok != 0;
}
// A wait whose first try has failed (one argument, the parity in bit 30: a wait
// is 60 instructions else).
__device__ __noinline__ bool t8_wait(uint32_t what, const T8Table& T) {
  volatile const int* abort = &T.ring.abort;
  uint64_t* bar = reinterpret_cast<uint64_t*>(__cvta_shared_to_generic(what & 0x3fffffffu));
  const bool r = !*abort && pa_wait(bar, what >> 30, T.wait_ns, abort);
  return (bool)__all_sync(0xffffffffu, r);
}

// A thread's 64 scores (in tensor memory at t) of positions d + c behind its
// row's: those that are no plain product times a float (!fold) brought into the
// log2 domain, with kw the slices' scales; those that `see` has no bit of, hidden.
// Returns the largest.
__device__ __noinline__ float t8_bend(const PagedAttnArgs& a, uint32_t t, bool fold, uint32_t kw, int qx, float slope, int d,
                                      unsigned long long see) {
  float top = -INFINITY;
#pragma unroll 1
  for (int c0 = 0; c0 < 64; c0 += 16) {
    uint32_t sr[16];
    float s[16];
    tc_ld16(t + c0, sr);
    tc_wait_ld();
#pragma unroll
    for (int c = 0; c < 16; ++c) s[c] = __uint_as_float(sr[c]);
    if (!fold) {
      float f0, f1;
      const int e = (int)(kw >> (c0 >> 1) & 255u);
      p8_pow2(qx == kP8Nan ? 0 : qx + e - 127, f0, f1);
      if (qx == kP8Nan || e == 255) f0 = __int_as_float(0x7fffffff);
#pragma unroll
      for (int c = 0; c < 16; ++c) s[c] = s[c] * f0 * f1;
      if (a.cap_log2 > 0.f) {
#pragma unroll
        for (int c = 0; c < 16; c += 2) pa_capped(a, s[c], s[c + 1]);
      } else {
#pragma unroll
        for (int c = 0; c < 16; ++c) s[c] *= a.scale_log2;
      }
      if (a.slopes) {
        const float from = (float)(d + c0);
#pragma unroll
        for (int c = 0; c < 16; ++c) s[c] = __fmaf_rn(slope, from + (float)c, s[c]);
      }
    }
    const uint32_t mine = (uint32_t)(see >> c0);
    if ((mine & 0xffffu) != 0xffffu) {
#pragma unroll
      for (int c = 0; c < 16; ++c)
        if (!(mine >> c & 1u)) s[c] = -INFINITY;
    }
#pragma unroll
    for (int c = 0; c < 16; ++c) {
      top = fmaxf(top, s[c]);
      sr[c] = __float_as_uint(s[c]);
    }
    __syncwarp();
    tc_st16(t + c0, sr);
  }
  tc_wait_st();
  return top;
}

// The slices of `some` that have NaN among their values (v0, v1: a chunk's
// halves, unpacked; vw: the slices' scales), of which this warp looks at quarter w.
__device__ __noinline__ int t8_nan(uint32_t v0, uint32_t v1, uint64_t vw, int some, int w, int lane) {
  int odd = 0;
#pragma unroll 1
  for (int ks = 0; ks < 8; ++ks) {
    if (!(some >> ks & 1)) continue;
    const uint32_t at = (ks < 4 ? v0 : v1) + (w >> 1) * 8192 + (ks & 3) * 2048 + (w & 1) * 1024 + lane * 16;
    bool bad = p8_byte(vw, ks) == 255u;
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      uint32_t x[4];
      asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(x[0]), "=r"(x[1]), "=r"(x[2]), "=r"(x[3])
                   : "r"(at + 512 * u));
#pragma unroll
      for (int i = 0; i < 4; ++i) bad |= __vcmpeq2(x[i] & 0x7C007C00u, 0x7C007C00u) != 0u;
    }
    odd |= __any_sync(0xffffffffu, bad) << ks;
  }
  return odd;
}

// Slices `odd` of half a chunk (values at v, their scales vw, weights at p)
// added element by element to a thread's dim of O's rows c .. c + 7 (at t;
// has: it holds sums), for the positions that `see` says its lane's row sees.
__device__ __noinline__ void t8_far(uint32_t t, bool has, uint32_t v, uint32_t vw, int vref, uint32_t p, int odd, int c, int dim,
                                    unsigned long long see) {
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i] = 0u;
  if (has) tc_ld8(t + c, o);
  tc_wait_ld();
  v += (dim >> 6) * 8192 + (dim & 7) * 2;
#pragma unroll 1
  for (int x = 0; x < 64; ++x) {
    if (!(odd >> (x >> 4) & 1)) continue;
    const uint32_t rows = __ballot_sync(0xffffffffu, see >> x & 1ull) >> (c & 31);
    const int e = (int)(vw >> (8 * (x >> 4)) & 255u);
    const float y = p8_half(lds16(v + x * 128 + ((((dim >> 3) & 7) ^ (x & 7)) << 4)), 0);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (!(rows >> i & 1u)) continue;
      const float w = p8_half(lds16(p + (c + i) * 128 + (((x >> 3) ^ i) << 4) + 2 * (x & 7)), 0) * y;
      o[i] = __float_as_uint(__uint_as_float(o[i]) + (p8_is_far(e, vref) ? p8_far(w, e, vref) : w));
    }
  }
  __syncwarp();
  tc_st8(t + c, o);
  tc_wait_st();
}

}  // namespace

__global__ void __launch_bounds__(kT8Threads, 1) k_paged_attn8_tc(const __grid_constant__ PagedAttn8Params A8) {
  const PagedAttnParams& A = A8.A;
  const PagedAttnArgs& a = A.a;
  const PagedRows& P = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_p = smem;
  unsigned char* s_v = s_p + 2 * kT8P;
  unsigned char* s_k = s_v + kT8Values * kT8V;  // rings: keys, values as they lie in the page
  unsigned char* s_raw = s_k + kT8Keys * kT8Half;
  T8Table& T = *reinterpret_cast<T8Table*>(s_raw + kT8Stages * kT8Half);
  PaSeq* plan = reinterpret_cast<PaSeq*>(s_raw);  // [n_seqs], in the ring before its first load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    T.ring.abort = 0;
    T.wait_ns = A.wait_ns;
    for (int i = 0; i < kT8Stages; ++i) {
      mbar_init(&T.ring.full[i], 1);
      mbar_init(&T.ring.empty[i], kT8Conv);
    }
    for (int i = 0; i < kT8Keys; ++i) mbar_init(&T.k_empty[i], 1);
    for (int i = 0; i < kT8Segs; ++i) {
      mbar_init(&T.told[i], 1);
      mbar_init(&T.read[i], kT8Readers);
      mbar_init(&T.rows[i], kT8Conv);
    }
    for (int i = 0; i < kT8Scales; ++i) mbar_init(&T.scaled[i], 1);
    for (int i = 0; i < kT8Values; ++i) {
      mbar_init(&T.v_full[i], kT8Conv);
      mbar_init(&T.v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T.s_full[i], 1);
      mbar_init(&T.s_empty[i], 4);
      mbar_init(&T.x_full[i], 4);
      mbar_init(&T.p_full[i], 4);
      mbar_init(&T.o_done[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T.q_full[i], kT8Conv);
      mbar_init(&T.q_empty[i], 1);
    }
    mbar_init(&T.ml_full, 8);
    mbar_init(&T.epi_done, 8);
    mbar_init(&T.fin[0], 1);
    mbar_init(&T.fin[1], 1);
    fence_mbar_init();
    prefetch_tensormap(&A.km);
    prefetch_tensormap(&A.vm);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (A.wait_ns == 0) {  // no wait may begin
    if (threadIdx.x == 0) {
      A.rec[cta * 2].np = A.rec[cta * 2 + 1].np = 0;
      atomicCAS(P.err, 0, (int)MOE_ERR_DEVICE_TIMEOUT);
    }
    return;
  }
  if (warp == kT8Mma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&T.tmem)), "n"(kT8Cols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) A.rec[cta * 2].np = A.rec[cta * 2 + 1].np = 0;  // no parts yet
  for (int b = threadIdx.x; b < P.n_seqs; b += kT8Threads) plan[b] = pa_seq<kT8Chunk>(a, b, cta == 0 ? P.err : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = T.tmem;
  volatile int* abort = &T.ring.abort;
  // the whole warp waits: true if every lane has seen the phase end
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    const uint32_t at = smem_addr(bar);
    return t8_try(at, parity) || t8_wait(at | parity << 30, T);
  };
  // segment i's description; done with it
  auto told = [&](int i) { return wait(&T.told[i % kT8Segs], (uint32_t)(i / kT8Segs) & 1u); };
  auto done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&T.read[i % kT8Segs]);
  };
  int issued = 0;  // stages of the producer

  if (warp == kT8Producer) {
    struct Out {
      const PagedAttn8Params& A8;
      T8Table& T;
      unsigned char *s_k, *s_raw;
      volatile int* abort;
      uint64_t pol;
      int lane, lbr, n;  // n: segments
      uint2 ks, vs;      // this lane's box's scales
      int st, any, all;  // the stage; which of its slices some row sees some of; kP8InfoAll: every row all of all
      int window, all_lo, all_hi;
      __device__ bool tell(const T8Seg& t) {
        bool ok = true;
        if (n >= kT8Segs)
          ok = !*abort && pa_wait(&T.read[n % kT8Segs], (uint32_t)(n / kT8Segs - 1) & 1u, A8.A.wait_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abort = 1;
        if (ok && lane == 0) {
          T.seg[n % kT8Segs] = t;
          mbar_arrive(&T.told[n % kT8Segs]);
        }
        ++n;
        return ok;
      }
      __device__ void look(int row, bool load) {
        if (!load) return;
        ks = p8_load_scales(A8.ks + (row >> 4), lbr);
        vs = p8_load_scales(A8.vs + (row >> 4), lbr);
      }
      __device__ bool begin(const PaSegment<kT8Chunk>& g, int st) {
        const PaSeq& s = g.s;
        all_lo = p8_all_lo(s, window);
        all_hi = p8_all_hi(s);
        return tell({s.q0, s.n, s.len, g.kvh, s.first, s.prefix, s.cp, s.np, s.cm, g.j0, g.j1 - g.j0, st, g.cf, g.np, g.slot});
      }
      __device__ bool stage(const PaSegment<kT8Chunk>& g, int j, int s, uint32_t bytes) {
        st = s;
        const int pos0 = g.pos(j), sp = pos0 + 16 * (lane & 7);
        any = 255, all = kP8InfoAll;
        if (pos0 < all_lo || pos0 > all_hi - kT8Chunk) {
          any = (int)__ballot_sync(0xffffffffu, pa_any(g.s.len, g.s.n, g.s.first, g.s.prefix, window, sp, sp + 15)) & 255;
          all = __all_sync(0xffffffffu, pa_all(g.s.len, g.s.n, g.s.first, g.s.prefix, window, sp, sp + 15)) ? kP8InfoAll : 0;
        }
        bool ok = true;
        if (s >= kT8Keys)
          ok = pa_next(&T.k_empty[s % kT8Keys], (uint32_t)(s / kT8Keys - 1) & 1u, A8.A.wait_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abort = 1;
        if (ok && lane == 0) mbar_arrive_expect_tx(&T.ring.full[s % kT8Stages], bytes);
        return ok;
      }
      __device__ void put(int sl, int box, int row, uint64_t* bar) {
        tma_load_2d(s_k + st % kT8Keys * kT8Half + (box << (lbr + 7)), &A8.A.km, 0, row, bar, pol);
        tma_load_2d(s_raw + sl * kT8Half + (box << (lbr + 7)), &A8.A.vm, 0, row, bar, pol);
      }
      __device__ void filled(int s, int box0) {
        p8_scales(T.scale[s % kT8Scales], &T.info[s % kT8Scales], ks, vs, box0, lbr, any, lane, all);
        if (lane == 0) mbar_arrive(&T.scaled[s % kT8Scales]);
      }
      __device__ bool end(int) {
        tell(T8Seg{});  // no chunks: the CTA is done
        return false;
      }
    };
    issued = pa_produce<kT8Unit, kT8Stages, kT8Chunk, 256>(
        A, T.ring, plan, cta, lane,
        Out{A8, T, s_k, s_raw, abort, policy_evict_first(), lane, P.lps, 0, make_uint2(0u, 0u), make_uint2(0u, 0u), 0, 0, 0, a.window, 0, 0});
  } else if (warp == kT8Mma || warp == kT8MmaO) {
    // ---------------------------------------------------------------- products
    const uint64_t p0 = tc_desc(smem_addr(s_p), 16, 1024);
    const uint64_t k0 = tc_desc(smem_addr(s_k), 16, 1024), v0 = tc_desc(smem_addr(s_v), 8192, 1024);
    constexpr uint32_t is = tc_idesc_e4m3(kT8Chunk), io = tc_idesc_f16(64, false) | kTcAMnMajor;
    bool ok = true;
    for (int seg = 0;; ++seg) {
      ok = told(seg);
      if (!ok) break;
      const int st0 = __shfl_sync(0xffffffffu, T.seg[seg % kT8Segs].st0, 0);
      const int st1 = st0 + __shfl_sync(0xffffffffu, T.seg[seg % kT8Segs].count, 0);
      if (st0 == st1) break;
      done(seg);
      if (warp == kT8Mma) {
        // S = Q K^T, up to two chunks ahead of what the softmax has read
        ok = wait(&T.q_full[seg & 1], (uint32_t)(seg >> 1) & 1u);
        for (int st = st0; ok && st < st1; ++st) {
          const int sl = st % kT8Stages;
          ok = wait(&T.ring.full[sl], (uint32_t)(st / kT8Stages) & 1u);
          if (ok && st > 1) ok = wait(&T.s_empty[st & 1], (uint32_t)((st >> 1) - 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t k = k0 + (unsigned)(st % kT8Keys * (kT8Half >> 4));
          if (tc_elect()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)  // 32 dims of hi, then of lo
              tc_mma_f8(tmem + kT8S + 128 * (st & 1), tmem + kT8Q + 64 * (seg & 1) + 8 * ks, k + (ks & 3) * 2, is, ks > 0);
            tc_commit(&T.s_full[st & 1]);
            tc_commit(&T.k_empty[st % kT8Keys]);
            if (st == st1 - 1) tc_commit(&T.q_empty[seg & 1]);
          }
          __syncwarp();
        }
      } else {
        // O^T += V^T P^T
        for (int st = st0; st < st1; ++st) {
          const int g = st & 1;
          ok = wait(&T.p_full[g], (uint32_t)(st >> 1) & 1u);
          if (!ok) break;
          const int pv = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&T.pv[g]), 0);
          tc_fence_after();
          const uint32_t d = tmem + kT8O + 64 * g;
          bool acc = pv & 256;
          for (int h = 0; h < 2; ++h) {
            const int sv = 2 * st + h, vl = sv % kT8Values;
            ok = wait(&T.v_full[vl], (uint32_t)(sv / kT8Values) & 1u);
            if (!ok) break;
            tc_fence_after();
            const uint64_t p = p0 + (unsigned)(g * (kT8P >> 4) + h * (8192 >> 4)), v = v0 + (unsigned)(vl * (kT8V >> 4));
            const int some = pv >> (4 * h) & 15;
            if (tc_elect()) {
              if (some == 15) {
#pragma unroll
                for (int ks = 0; ks < 4; ++ks) tc_mma(d, v + 128 * ks, p + 2 * ks, io, ks > 0 || acc);
              } else {
                bool more = acc;
#pragma unroll 1
                for (int ks = 0; ks < 4; ++ks) {
                  if (!(some >> ks & 1)) continue;
                  tc_mma(d, v + 128 * ks, p + 2 * ks, io, more);
                  more = true;
                }
              }
              tc_commit(&T.v_empty[vl]);
              if (h == 1) tc_commit(&T.o_done[g]);
            }
            __syncwarp();
            acc = acc || some != 0;
          }
          if (!ok) break;
        }
      }
      if (!ok) break;
    }
    if (!ok) *abort = 1;
    // every product has ended before the CTA frees its memory
    if (tc_elect()) {
      uint64_t* fin = &T.fin[warp - kT8Mma];
      tc_commit(fin);
      mbar_wait_drain(fin, 0, kPaDrainNs);
    }
    __syncwarp();
  } else if (warp >= kT8Values0) {
    // ---------------------------------------------------------------- rows of Q; values, unpacked
    // Unit u of half a chunk: 16 dims (chunk c of eight) of a position.  A
    // quarter of a warp takes four dim chunks of positions p and p ^ 5: eight
    // different 16-byte columns, read and written.
    const int u0 = (warp - kT8Values0) * 32 + lane;
    const int c = (lane & 3) + (lane >> 1 & 4), dp = (lane >> 2 & 1) * 5;
    int st0 = 0, st1 = 1;  // the stages of the segment at hand
    // Waits for segment seg's description; its stages; brings its rows of Q
    // into two parts.  False: given up.
    auto rows_of = [&](int seg) {
      if (!told(seg)) return false;
      const T8Seg& D = T.seg[seg % kT8Segs];
      st0 = D.st0;
      st1 = st0 + D.count;
      if (st0 == st1) return true;
      // A row a thread, each row in two lanes of tensor memory (for the halves
      // of the positions).  Read twice, for the largest value and for the parts:
      // kept in registers the parts are 20 KB of instructions.
      const int i = 32 * (warp & 1) + lane, r = i / a.group;
      const bool mine = i < D.n * a.group;
      const uint4* src = reinterpret_cast<const uint4*>(a.q + (D.q0 + r) * a.qs + (D.kvh * a.group + i - r * a.group) * 128);
      uint32_t most = 0;  // of both halves' magnitudes
#pragma unroll 1
      for (int u = 0; u < 16; u += 8) {
        uint4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] = mine ? src[u + k] : make_uint4(0u, 0u, 0u, 0u);
#pragma unroll
        for (int k = 0; k < 8; ++k)
          most = __vmaxu2(__vmaxu2(most, __vmaxu2(v[k].x & 0x7FFF7FFFu, v[k].y & 0x7FFF7FFFu)),
                          __vmaxu2(v[k].z & 0x7FFF7FFFu, v[k].w & 0x7FFF7FFFu));
      }
      float f;
      int x;
      p8_row_scale<7>(p8_most(most), f, x);
      if (mine && !(warp & 2)) T.qx[seg % kT8Segs][i] = x;
      done(seg);
      if (seg > 1 && !wait(&T.q_empty[seg & 1], (uint32_t)((seg >> 1) - 1) & 1u)) return false;
      tc_fence_after();
      const uint32_t to = tmem + ((uint32_t)(32 * (warp & 3)) << 16) + kT8Q + 64 * (seg & 1);
#pragma unroll 1
      for (int u = 0; u < 16; u += 4) {
        uint32_t hi[8], lo[8];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const uint4 v = mine ? src[u + k] : make_uint4(0u, 0u, 0u, 0u);
          p8_parts(make_uint2(v.x, v.y), f, hi[2 * k], lo[2 * k]);
          p8_parts(make_uint2(v.z, v.w), f, hi[2 * k + 1], lo[2 * k + 1]);
        }
        __syncwarp();
        tc_st8(to + 2 * u, hi);
        tc_st8(to + 32 + 2 * u, lo);
      }
      tc_wait_st();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(&T.rows[seg % kT8Segs]);
        mbar_arrive(&T.q_full[seg & 1]);
      }
      return true;
    };
    auto unpack = [&](int st) {
      const int sl = st % kT8Stages;
      bool ok = wait(&T.ring.full[sl], (uint32_t)(st / kT8Stages) & 1u);
      for (int h = 0; ok && h < 2; ++h) {
        const int sv = 2 * st + h, vl = sv % kT8Values;
        if (sv >= kT8Values) ok = wait(&T.v_empty[vl], (uint32_t)(sv / kT8Values - 1) & 1u);
        if (!ok) break;
        const uint32_t from = smem_addr(s_raw + sl * kT8Half) + h * 8192, to = smem_addr(s_v + vl * kT8V);
        uint32_t w[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = ((u0 >> 4) * 2 + j * 16) ^ dp;  // pairs (2i, 2i ^ 5) and, by the lanes' next bit, their neighbours
          asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(w[j][0]), "=r"(w[j][1]), "=r"(w[j][2]), "=r"(w[j][3])
                       : "r"(from + p * 128 + ((c ^ (p & 7)) << 4)));
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int p = ((u0 >> 4) * 2 + j * 16) ^ dp;
          uint32_t x[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) p8_unpack(w[j][i], x[2 * i], x[2 * i + 1]);
          const uint32_t at = to + (c >> 2) * 8192 + p * 128;
#pragma unroll
          for (int i = 0; i < 2; ++i)
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + (((2 * (c & 3) + i) ^ (p & 7)) << 4)),
                         "r"(x[4 * i]), "r"(x[4 * i + 1]), "r"(x[4 * i + 2]), "r"(x[4 * i + 3])
                         : "memory");
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&T.v_full[vl]);
          if (h == 1) mbar_arrive(&T.ring.empty[sl]);
        }
      }
      return ok;
    };
    bool ok = true;
    for (int seg = 0; ok; ++seg) {
      ok = rows_of(seg);
      if (st0 == st1) break;
      for (int st = st0; ok && st < st1; ++st) ok = unpack(st);
    }
    if (!ok) *abort = 1;
  } else {
    // ---------------------------------------------------------------- softmax
    // A thread has 64 positions of a row of S; of O, which has rows in columns, one dim of all rows, so it follows the
    // references of its row and of row ^ 32.
    const int g = warp >> 2, half = (warp >> 1) & 1, row = 32 * (warp & 1) + lane;  // 64 positions of a row
    const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + t_lane + kT8S + 128 * g + 64 * half, t_o = tmem + t_lane + kT8O + 64 * g;
    const uint32_t p_row = smem_addr(s_p) + g * kT8P + row * 128;  // (the second half's positions 8192 on)
    uint32_t xpar = 0;
    bool ok = true;
    int shared = 0, cleared = 0;  // segments of both groups so far, those whose end has been waited for
    // the group's four warps: what each wrote before is there for all after
    auto exchange = [&]() {
      __syncwarp();
      if (lane == 0) mbar_arrive(&T.x_full[g]);
      const bool r = wait(&T.x_full[g], xpar);
      xpar ^= 1u;
      return r;
    };
    for (int seg = 0;; ++seg) {
      ok = told(seg);
      if (!ok) break;
      const T8Seg& D = T.seg[seg % kT8Segs];
      const int st0 = D.st0, st1 = st0 + D.count;
      if (st0 == st1) break;
      const bool solo = st1 - st0 == 1;  // a segment of one chunk is its group's alone
      if (solo && (st0 & 1) != g) {
        done(seg);
        continue;
      }
      float m = -INFINITY, m2 = -INFINITY, l = 0.f, slope = 0.f;  // (m2: of row ^ 32)
      bool has = false;
      // the last shared segment's outputs are out
      auto cleaned = [&]() {
        if (cleared != shared) ok = wait(&T.epi_done, (uint32_t)(shared - 1) & 1u);
        cleared = shared;
        return ok;
      };
      const bool live = row < D.n * a.group;
      const int r = live ? row / a.group : 0, h = D.kvh * a.group + (live ? row - r * a.group : 0);
      const int rp = D.len + r, rp2 = D.len + ((row ^ 32) < D.n * a.group ? (row ^ 32) / a.group : 0);  // the rows' positions
      if (a.slopes) slope = a.slopes[h] * 1.4426950408889634f;
      ok = wait(&T.rows[seg % kT8Segs], (uint32_t)(seg / kT8Segs) & 1u);
      if (!ok) break;
      const int qx = live ? T.qx[seg % kT8Segs][row] : 0;
      int vref = 0;  // the group's sums' reference scale
      // (registers: the description's memory would be read again after every wait)
      const bool odd_q = __any_sync(0xffffffffu, qx < -40 || qx > 40);  // (kP8Nan among them)
      const float qf = odd_q ? 1.f : p8_exp(qx) * a.scale_log2;
      const bool folds = a.fold && !odd_q;
      const int np = st0 + D.np - D.j0;  // the stages before are of the kept prefix
      const int at_main = (D.cm - D.np + D.j0 - st0) * kT8Chunk;
      // what of positions from .. from + 63 the row at position rp sees
      auto sees = [&](int from, int rp) {
        const int lo = a.window > 0 ? max(D.first, rp - a.window + 1) : D.first;
        return tc_bits(lo - from, rp + 1 - from) | tc_bits(D.first - from, min(D.prefix, rp + 1) - from);
      };
      for (int st = st0 + ((st0 & 1) != g); st < st1; st += 2) {
        const int own = st >> 1, sc = st % kT8Scales;
        ok = wait(&T.scaled[sc], (uint32_t)(st / kT8Scales) & 1u);
        if (!ok) break;
        const int info = T.info[sc], r0 = vref;
        vref = p8_ref(vref, info & 255);
        // plain scores times f (of each slice) are in the log2 domain; else they are made so, and f is 1
        const bool fold = folds && (info & kP8InfoFold);
        int any = 255, clear = 255;  // which 16-position slices some row sees some of, every row all of
        int pos0 = 0;                // (not taken where all see all)
        if (!(info & kP8InfoAll)) {
          pos0 = st < np ? (D.cp + D.j0 + st - st0) * kT8Chunk : at_main + st * kT8Chunk;
          const int sp = pos0 + 16 * (lane & 7);
          any = __ballot_sync(0xffffffffu, pa_any(D.len, D.n, D.first, D.prefix, a.window, sp, sp + 15)) & 255;
          clear = __ballot_sync(0xffffffffu, pa_all(D.len, D.n, D.first, D.prefix, a.window, sp, sp + 15)) & 255;
        }
        const bool bent = !fold || !(info & kP8InfoAll);
        auto values = [&](int h) { return smem_addr(s_v) + (2 * st + h) % kT8Values * kT8V; };
        // Both halves of the chunk's values are there.  A wait on a parity tells a phase from the one before it, not from
        // the one before that, so the one before has to be known complete; v_full is waited for in few chunks only, but
        // its buffers' last values are what O's last product read: that product has ended, then those were there.
        auto unpacked = [&]() {
          return (own == 0 || wait(&T.o_done[g], (uint32_t)(own - 1) & 1u)) &&
                 wait(&T.v_full[2 * st % kT8Values], (uint32_t)(2 * st / kT8Values) & 1u) &&
                 wait(&T.v_full[(2 * st + 1) % kT8Values], (uint32_t)((2 * st + 1) / kT8Values) & 1u);
        };
        if (any & ~clear) {
          // slices with hidden positions: NaN values among them?
          ok = unpacked();
          if (!ok) break;
          const int odd = t8_nan(values(0), values(1), T.scale[sc][1], any & ~clear, warp & 3, lane);
          if (lane == 0) T.odd[own & 1][g][warp & 3] = odd;
        }
        ok = wait(&T.s_full[g], (uint32_t)own & 1u);
        if (!ok) break;
        tc_fence_after();
        // The scores are read twice, for their maximum and for the exponentials (kept meanwhile, 64 of them spill); those
        // that something hides or bends go back as they then are (bent twice, 19 sequences of 4096 with capped scores
        // took 113 us).
        const uint32_t kw = (uint32_t)(T.scale[sc][0] >> (32 * half));  // of this half's keys
        float f[4], mine_top = -INFINITY;
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = fold ? qf * __uint_as_float((kw >> (8 * k) & 255u) << 23) : 1.f;
        if (bent) {
          if (info & kP8InfoAll) pos0 = st < np ? (D.cp + D.j0 + st - st0) * kT8Chunk : at_main + st * kT8Chunk;
          const int pos1 = pos0 + 64 * half;
          mine_top = t8_bend(a, t_s, fold, kw, qx, slope, pos1 - rp, clear == 255 ? ~0ull : sees(pos1, rp));
        }
        if (fold) {
          mine_top = -INFINITY;
#pragma unroll 1
          for (int i = 0; i < 2; ++i) {
            uint32_t sr[32];
            tc_ld32(t_s + 32 * i, sr);
            tc_wait_ld();
            float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
            for (int c = 0; c < 32; ++c) mx[c >> 4] = fmaxf(mx[c >> 4], __uint_as_float(sr[c]));
            mine_top = fmaxf(mine_top, fmaxf(mx[0] * (i ? f[2] : f[0]), mx[1] * (i ? f[3] : f[1])));
          }
        }
        if (!cleaned()) break;
        float(&s_top)[2][64] = T.top[own & 1][g];
        s_top[half][row] = mine_top;
        if (!(ok = exchange())) break;
        // (else than by a maximum that grows from none: the row's sums are zeros)
        auto grow = [](float& m, float top) {
          if (!(top > m)) return 1.f;
          const float from = m;
          m = top + kT8Room;
          return from == -INFINITY ? 1.f : ex2(from - m);
        };
        float scale = grow(m, fmaxf(mine_top, s_top[half ^ 1][row])), scale2 = grow(m2, fmaxf(s_top[0][row ^ 32], s_top[1][row ^ 32]));
        l *= scale;
        if (r0 != vref) {
          scale *= p8_grown(r0, vref);
          scale2 *= p8_grown(r0, vref);
        }
        const float ref = m == -INFINITY ? 0.f : m;  // nothing visible yet
        // P's place (and O) is free when the product before has ended
        if (own > 0) ok = wait(&T.o_done[g], (uint32_t)(own - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        const uint32_t v_half = (uint32_t)(T.scale[sc][1] >> (32 * half));
        // A slice's 16 weights come out of the exponential times 2^u.
        auto weights = [&](const uint32_t* x, int slice, float fk) {
          const int u = p8_up_log2((int)(v_half >> (8 * slice) & 255u), vref);
          const float c0 = (float)u - ref;
          const unsigned long long f2 = pa_pair(fk, fk), c2 = pa_pair(c0, c0), one = pa_pair(1.f, 1.f);
          unsigned long long sum[2] = {0ull, 0ull};
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            uint32_t w[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
              float p0, p1;
              pa_unpair(pa_fma2(pa_pair(__uint_as_float(x[8 * c + 2 * q]), __uint_as_float(x[8 * c + 2 * q + 1])), f2, c2), p0, p1);
              p0 = ex2(p0);
              p1 = ex2(p1);
              sum[q & 1] = pa_fma2(pa_pair(p0, p1), one, sum[q & 1]);
              w[q] = pack_f16x2(p0, p1);
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(p_row + half * 8192 + (((2 * slice + c) ^ (row & 7)) << 4)),
                         "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3])
                         : "memory");
          }
          float s0, s1, s2, s3;
          pa_unpair(sum[0], s0, s1);
          pa_unpair(sum[1], s2, s3);
          l = __fmaf_rn((s0 + s1) + (s2 + s3), p8_exp(-u), l);
        };
#pragma unroll 1
        for (int i = 0; i < 2; ++i) {
          uint32_t sr[32];
          tc_ld32(t_s + 32 * i, sr);
          tc_wait_ld();
#pragma unroll
          for (int k = 0; k < 2; ++k) weights(sr + 16 * k, 2 * i + k, i ? f[2 + k] : f[k]);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.s_empty[g]);
        // rows whose reference has grown (this warp's 32, the other 32): their sums so far
        const uint32_t grown = __ballot_sync(0xffffffffu, scale != 1.f), grown2 = __ballot_sync(0xffffffffu, scale2 != 1.f);
        if (has && (grown | grown2)) {
#pragma unroll 1
          for (int c = 0; c < 64; c += 8) {
            const bool own_rows = (c & 32) == 32 * (warp & 1);
            if (!((own_rows ? grown : grown2) >> (c & 31) & 255u)) continue;
            const float by = own_rows ? scale : scale2;
            uint32_t o[8];
            tc_ld8(t_o + c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * __shfl_sync(0xffffffffu, by, (c & 31) + i));
            tc_st8(t_o + c, o);
          }
          tc_wait_st();
        }
        int pv = any;
        if ((any & ~clear) || p8_any_far(info, vref)) {
          // slices that are added element by element: NaN that some row does not see, a scale far above the reference
          const int(&s_odd)[4] = T.odd[own & 1][g];
          const uint64_t vw = T.scale[sc][1];
          int odd = (any & ~clear) ? s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3] : 0;
#pragma unroll 1
          for (int ks = 0; ks < 8; ++ks)
            if (p8_is_far((int)p8_byte(vw, ks), vref)) odd |= 1 << ks;
          odd &= any;
          if (odd) {
            pv &= ~odd;
            // (the same for all four warps) all rows' P, and the values
            if (!(ok = exchange() && unpacked())) break;
#pragma unroll 1
            for (int h = 0; h < 2; ++h) {
              if (!(odd >> (4 * h) & 15)) continue;
#pragma unroll 1
              for (int c = 0; c < 64; c += 8)
                t8_far(t_o, has, values(h), (uint32_t)(vw >> (32 * h)), vref, smem_addr(s_p) + g * kT8P + h * 8192, odd >> (4 * h) & 15, c,
                       32 * (warp & 3) + lane,
                       clear == 255 ? ~0ull : sees(pos0 + 64 * h, (c & 32) == 32 * (warp & 1) ? rp : rp2));
              has = true;
            }
          }
        }
        if ((warp & 3) == 0 && lane == 0) *reinterpret_cast<volatile int*>(&T.pv[g]) = pv | (has ? 256 : 0);
        has = has || pv != 0;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.p_full[g]);
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the segment's end
      const bool whole = D.parts == 1;
      const int nrow = D.n * a.group;
      const size_t part = (size_t)(cta * 2 + D.slot) * t8_padded(a);
      const int dim = 32 * (warp & 3) + lane;
      // this thread's dim of rows c .. c + 7: of their output, or of this CTA's part of it
      auto put = [&](int c, const float (&v)[8]) {
        int r = c / a.group, head = c - r * a.group;
        uint16_t* out = a.o + (D.q0 + r) * a.os + (D.kvh * a.group + head) * 128 + dim;
        float* po = A.part_o + (part + c) * 128 + dim;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          if (c + i >= nrow) break;
          if (whole) {
            *out = (uint16_t)pack_bf16(v[i], 0.f);
            out += 128;
            if (++head == a.group) {
              head = 0;
              out += a.os - a.group * 128;
            }
          } else {
            __stcg(po + i * 128, v[i]);
          }
        }
      };
      auto put_sums = [&](int row, float M, float L) {
        if (row >= nrow) return;
        const int r = row / a.group;
        if (whole && a.lse)
          a.lse[(size_t)(D.q0 + r) * a.nq + D.kvh * a.group + row - r * a.group] =
              L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        if (!whole) __stcg(reinterpret_cast<float2*>(A.part_ml + 2 * (part + row)), make_float2(M, L));
        if (!whole && row == 0) A.rec[cta * 2 + D.slot] = {D.cf, D.parts, D.q0, D.n, D.kvh};
      };
      // what makes the row's output, or its part, of its sums; the sums' unit
      auto inverse = [&](float L) { return !whole ? 1.f : L == 0.f ? 0.f : 1.f / L; };
      if (solo) {
        // One chunk: its group ends it while the other is at the next segment.
        T.l[g][half][row] = l;
        if (!(ok = exchange())) break;
        const float L = T.l[g][0][row] + T.l[g][1][row], L2 = T.l[g][0][row ^ 32] + T.l[g][1][row ^ 32];
        const float inv = inverse(L), inv2 = inverse(L2), unit = p8_unit(vref);
        if (has) ok = wait(&T.o_done[g], (uint32_t)(st0 >> 1) & 1u);
        if (!ok) break;
        tc_fence_after();
#pragma unroll 1
        for (int c = 0; c < nrow; c += 8) {
          const float by = (c & 32) == 32 * (warp & 1) ? inv : inv2;
          uint32_t o[8];
          float v[8];
          if (has) tc_ld8(t_o + c, o);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 8; ++i)
            v[i] = has ? __uint_as_float(o[i]) * unit * __shfl_sync(0xffffffffu, by, (c & 31) + i) : 0.f;
          put(c, v);
        }
        tc_fence_before();
        if (half == 0) put_sums(row, m, L);
        done(seg);
        continue;
      }
      // The groups' references and sums for all, then each group adds both's
      // products of 32 rows.
      const int n0 = (st1 + 1) >> 1, n1 = st1 >> 1;  // the groups' chunks so far
      if (!cleaned()) break;
      T.l[g][half][row] = l;
      if (half == 0) T.m[g][row] = m;
      if ((warp & 3) == 0 && lane == 0) {
        T.has[g] = has;
        T.vref[g] = vref;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&T.ml_full);
      ok = wait(&T.ml_full, (uint32_t)shared & 1u);
      const bool has0 = ok && T.has[0], has1 = ok && T.has[1];
      if (ok && has0) ok = wait(&T.o_done[0], (uint32_t)(n0 - 1) & 1u);
      if (ok && has1) ok = wait(&T.o_done[1], (uint32_t)(n1 - 1) & 1u);
      if (!ok) break;
      tc_fence_after();
      const int er = 32 * g + lane;
      const float m0 = has0 ? T.m[0][er] : -INFINITY, m1 = has1 ? T.m[1][er] : -INFINITY, M = fmaxf(m0, m1);
      const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), e1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
      const float L = (has0 ? T.l[0][0][er] + T.l[0][1][er] : 0.f) * e0 + (has1 ? T.l[1][0][er] + T.l[1][1][er] : 0.f) * e1;
      const float inv = inverse(L), f0 = e0 * p8_unit(T.vref[0]), f1 = e1 * p8_unit(T.vref[1]);
#pragma unroll 1
      for (int c = 0; c < 32; c += 8) {
        uint32_t o0[8], o1[8];
        float v[8];
        if (has0) tc_ld8(tmem + t_lane + kT8O + 32 * g + c, o0);
        if (has1) tc_ld8(tmem + t_lane + kT8O + 64 + 32 * g + c, o1);
        tc_wait_ld();
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v[i] = has0 ? __uint_as_float(o0[i]) * __shfl_sync(0xffffffffu, f0, c + i) : 0.f;
          if (has1) v[i] += __uint_as_float(o1[i]) * __shfl_sync(0xffffffffu, f1, c + i);
          v[i] *= __shfl_sync(0xffffffffu, inv, c + i);
        }
        put(32 * g + c, v);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&T.epi_done);
      if ((warp & 3) == 0) put_sums(er, M, L);
      ++shared;
      done(seg);
    }
    if (!ok) *abort = 1;
  }
  tc_fence_before();
  __syncthreads();  // every warp is done with the ring and the tensor memory
  tc_fence_after();
  if (warp == kT8Mma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kT8Cols));
  if (warp == kT8Producer && *abort && lane == 0) pa_drain(T.ring, issued, P.err);
}

cudaError_t launch_paged_attention8_tc(const PagedAttn8Params& A, cudaStream_t s) {
  constexpr int smem = 2 * kT8P + kT8Values * kT8V + (kT8Keys + kT8Stages) * kT8Half + (int)sizeof(T8Table);
  static_assert(smem <= 227 * 1024, "one CTA an SM");
  static_assert(sizeof(PaSeq) * kPagedMaxSeqs <= kT8Stages * kT8Half, "the plan fits the ring");
  const cudaError_t e = prepare_kernel<k_paged_attn8_tc>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() < kPagedMaxCtas ? num_sms() : kPagedMaxCtas);
  cfg.blockDim = dim3(kT8Threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const cudaError_t el = cudaLaunchKernelEx(&cfg, k_paged_attn8_tc, A);
  return el == cudaSuccess ? launch_paged_join(A.A, cfg.gridDim.x, t8_padded(A.A.a), 1.f, s) : el;
}

}  // namespace moe
