// paged_attn_tc.cu -- the paged attention for up to 64 query rows a KV head
// (verify rows x heads of the KV head) on the 5th-generation tensor cores
// (paged_attention_tc chooses).
//
// Same work list, ring and join as paged_attn.cu (one CTA an SM, five 32 KB
// stages).  With 64 rows the products are 256 multiply-adds a byte of keys
// and values: mma.sync's rate, and the fragments' trips through registers,
// bound the other form.  Here, per 64-position chunk:
//   S [rows, 64]    = Q K^T     8 tcgen05.mma M128 N64  K16, Q and K K-major
//   O [rows, 128]  += P V       8 tcgen05.mma M128 N128 K16 (P = hi + lo), V
//                               N-major as it lies in the page
// with S and O in tensor memory and Q, P, K and V in shared memory (128-byte
// swizzle).  M is 128 although 64 rows are real.  For S, rows 64-127 are the
// same queries again, so that the scores also lie in the tensor memory lanes
// that the other two of an SM's four warp slots reach: thread (row, half)
// owns 32 scores of a row, and maximum and sum need one exchange with one
// other thread.  For O, rows 64-127 read whatever follows P and end where
// nobody looks.  (Two sequences of 65,003 and 131,001 positions, 64 rows, 8 KV
// heads: 134 us, 6 TB/s, in short runs, 136 to 143 in long ones; by mma.sync 349.
// 152 units of 4096: 58 us, 64 with capped scores, 64 with a bias by distance,
// 77 with both, where the keys and values alone take 47 at a copy's bandwidth.)
//
// Two groups of four such warps take even and odd chunks, each with its own
// S, P and O (so one group's softmax runs beside the other's products) and
// its own running reference m; O is only rescaled when a score is above it, to
// 8 (in log2) above that score, so that growth by less than 2^8 costs nothing
// and no p is above 1 (with m at the maximum itself and p up to 256, p v passed
// FP32's range for values above 1e36).  At a segment's end the first warps of
// both groups add the two groups' sums; a segment of one chunk is its group's
// alone, and the other goes on with the next.  Such short segments take about 3
// us each, what one thread row does from its scores to its output, two at a
// time; outputs staged through shared memory to be stored in whole lines took
// no less.  All 168 registers a thread
// are in use: 32 columns of tensor memory at a time at a segment's end instead
// of 16 spill, and 133 us become 139.
//
// Hidden positions: as in paged_attn.cu a slice with hidden positions is
// looked over for infinite or NaN values, and such a slice is kept out of the
// product and added element by element.
#include "paged_attn.cuh"

namespace moe {

namespace {

constexpr int kTcStages = 5;
// Slots before a unit's chunks: what its ends cost in chunks (236 units of 1 to
// 5911 positions: 42 us, 48 with one slot, 43 with six).
constexpr int kTcUnit = 4;
constexpr int kTcThreads = 384;
constexpr int kTcP = 2 * 8192;   // a group's P: hi, lo [64 rows][64 positions] bf16
constexpr int kTcQ = 2 * 16384;  // Q: [dim half][64 rows twice][64 dims] bf16
constexpr int kTcCols = 512;     // tensor memory columns
constexpr int kTcS = 0, kTcO = 256;  // S of chunk c at 64 (c mod 4), O of group g at 256 + 128 g
constexpr float kTcRoom = 8.f;   // growth of the maximum (log2) that the reference leaves room for
// Warps: 0-3 and 4-7 softmax of the even and odd chunks (a warp reads the
// tensor memory lanes of its number mod 4), 8 producer, 9 and 10 products (S;
// O: one warp for both spent 870 of 2200 clocks a chunk between the two), 11
// rows of Q.
constexpr int kTcProducer = 8, kTcMma = 9, kTcMmaO = 10, kTcLoader = 11;
constexpr int kTcSegs = 4;       // segments described ahead
constexpr int kTcReaders = 11;   // of a segment's description: every warp but the producer

// A segment as the warps see it: chunks j0 .. j0 + count - 1 of its unit, in
// the ring's stages st0, st0 + 1, ...
struct TcSeg {
  int q0, n, len, kvh, first, prefix;
  int cp, np, cm;  // of PaSeq
  int j0, count, st0;
  int cf, parts, slot;
};

struct TcTable {
  PaRing<kTcStages> ring;
  uint64_t told[kTcSegs], read[kTcSegs];  // the segment's description is written; is read by all
  TcSeg seg[kTcSegs];
  uint64_t s_full[4], s_empty[4];  // S of chunk c (mod 4) is there; is read
  uint64_t x_full[2];   // group g's four warps have left what the others need
  uint64_t p_full[2];   // P of group g is there
  uint64_t o_done[2];   // the product with P of group g is done
  uint64_t q_full, q_empty;  // the segment's Q is there; its last product with it is done
  uint64_t ml_full;     // m and l of a segment of both groups are there
  uint64_t epi_done;    // its outputs are out of tensor memory (a group's first P of the next segment waits)
  uint64_t fin[2];
  uint32_t tmem;
  int pv[2];            // slices to multiply (bits 0-3); bit 4: O holds sums already
  // [group's chunk mod 2][group][half][row] maximum of a chunk's scores.  (A
  // warp may be a chunk ahead of the one that reads what it wrote, not two.)
  // At a segment's end the place of the group's next chunk takes its m and l
  // ([0][row], [1][row]) until the outputs are out (epi_done).
  float top[2][2][2][64];
  int odd[2][2][4];     // [chunk mod 2][group][warp] slices where it saw infinite or NaN values
  int has[2];           // the group has sums
};

__device__ __forceinline__ uint64_t tc_desc(uint32_t addr, uint32_t lbo, uint32_t sbo) {
  // shared-memory matrix descriptor: start, leading and stride byte offsets
  // (16-byte units), version 1, 128-byte swizzle
  return (uint64_t)((addr & 0x3FFFFu) >> 4) | (uint64_t)(lbo >> 4) << 16 | (uint64_t)(sbo >> 4) << 32 | 1ull << 46 |
         2ull << 61;
}
// Instruction descriptor of kind::f16: FP32 sums of bf16 products, M 128.
__host__ __device__ constexpr uint32_t tc_idesc(int n, bool b_mn_major) {
  return 1u << 4 | 1u << 7 | 1u << 10 | (b_mn_major ? 1u << 16 : 0u) | (uint32_t)(n >> 3) << 17 | (128u >> 4) << 24;
}
// One thread of the (whole) warp, the same one every time.
__device__ __forceinline__ bool tc_elect() {
  uint32_t p;
  asm volatile("{\n .reg .pred p;\n elect.sync _|p, 0xffffffff;\n selp.u32 %0, 1, 0, p;\n}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ void tc_mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n .reg .pred p;\n setp.ne.u32 p, %4, 0;\n tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n}" ::"r"(d),
      "l"(a), "l"(b), "r"(idesc), "r"((uint32_t)acc)
      : "memory");
}
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar))
               : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }

// 32 columns of this thread's lane.
__device__ __forceinline__ void tc_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, "
      "%17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
// 16 columns.
__device__ __forceinline__ void tc_ld16(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};" ::"r"(t),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Bits [lo, hi) of a 64-bit mask.
__device__ __forceinline__ unsigned long long tc_bits(int lo, int hi) {
  lo = max(lo, 0);
  hi = min(hi, 64);
  if (lo >= hi) return 0ull;
  const unsigned long long up = hi == 64 ? ~0ull : (1ull << hi) - 1ull;
  return up & ~((1ull << lo) - 1ull);
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

}  // namespace

__global__ void __launch_bounds__(kTcThreads, 1) k_paged_attn_tc(const __grid_constant__ PagedAttnParams A, int rows) {
  const PagedAttnArgs& a = A.a;
  const PagedRows& P = a.p;
  extern __shared__ __align__(1024) unsigned char smem[];
  unsigned char* s_p = smem;                   // [group][hi, lo]
  unsigned char* s_q = smem + 2 * kTcP;
  unsigned char* ring = s_q + kTcQ;
  TcTable& T = *reinterpret_cast<TcTable*>(ring + kTcStages * kPaStageBytes);
  PaSeq* plan = reinterpret_cast<PaSeq*>(ring);  // [n_seqs], in the ring before its first load
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, cta = blockIdx.x;

  if (threadIdx.x == 0) {
    T.ring.abort = 0;
    for (int i = 0; i < kTcStages; ++i) {
      mbar_init(&T.ring.full[i], 1);
      mbar_init(&T.ring.empty[i], 1);
    }
    for (int i = 0; i < kTcSegs; ++i) {
      mbar_init(&T.told[i], 1);
      mbar_init(&T.read[i], kTcReaders);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&T.s_full[i], 1);
      mbar_init(&T.s_empty[i], 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&T.x_full[i], 4);
      mbar_init(&T.p_full[i], 4);
      mbar_init(&T.o_done[i], 1);
    }
    mbar_init(&T.q_full, 1);
    mbar_init(&T.q_empty, 1);
    mbar_init(&T.ml_full, 4);
    mbar_init(&T.epi_done, 4);
    mbar_init(&T.fin[0], 1);
    mbar_init(&T.fin[1], 1);
    fence_mbar_init();
    prefetch_tensormap(&A.km);
    prefetch_tensormap(&A.vm);
  }
  pdl_wait();
  pdl_launch_dependents();
  if (warp == kTcMma) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&T.tmem)), "n"(kTcCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;");
  }
  if (threadIdx.x == 0) A.rec[cta * 2].np = A.rec[cta * 2 + 1].np = 0;  // no parts yet
  for (int b = threadIdx.x; b < P.n_seqs; b += kTcThreads) plan[b] = pa_seq(a, b, cta == 0 ? P.err : nullptr);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = T.tmem;
  volatile int* abort = &T.ring.abort;
  // the whole warp waits: true if every lane has seen the phase end
  auto wait = [&](uint64_t* bar, uint32_t parity) {
    bool r = A.wait_ns != 0 && mbar_try_wait(bar, parity);
    if (__all_sync(0xffffffffu, r)) return true;
    if (!r) r = !*abort && pa_wait(bar, parity, A.wait_ns, abort);
    return (bool)__all_sync(0xffffffffu, r);
  };
  // segment i's description; done with it
  auto told = [&](int i) { return wait(&T.told[i % kTcSegs], (uint32_t)(i / kTcSegs) & 1u); };
  auto done = [&](int i) {
    __syncwarp();
    if (lane == 0) mbar_arrive(&T.read[i % kTcSegs]);
  };
  int issued = 0;  // stages of the producer

  if (warp == kTcProducer) {
    struct Out {
      const PagedAttnParams& A;
      TcTable& T;
      unsigned char* ring;
      volatile int* abort;
      uint64_t pol;
      int lane, br, n;  // n: segments
      __device__ bool tell(const TcSeg& t) {
        bool ok = true;
        if (n >= kTcSegs)
          ok = !*abort && pa_wait(&T.read[n % kTcSegs], (uint32_t)(n / kTcSegs - 1) & 1u, A.wait_ns, abort);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) *abort = 1;
        if (ok && lane == 0) {
          T.seg[n % kTcSegs] = t;
          mbar_arrive(&T.told[n % kTcSegs]);
        }
        ++n;
        return ok;
      }
      __device__ bool begin(const PaSegment& g, int st) {
        const PaSeq& s = g.s;
        return tell({s.q0, s.n, s.len, g.kvh, s.first, s.prefix, s.cp, s.np, s.cm, g.j0, g.j1 - g.j0, st, g.cf, g.np, g.slot});
      }
      __device__ void stage(const PaSegment&, int, int st, uint32_t bytes) {
        if (lane == 0) mbar_arrive_expect_tx(&T.ring.full[st % kTcStages], bytes);
      }
      __device__ void put(int sl, int box, int row, uint64_t* bar) {
        unsigned char* dst = ring + (size_t)sl * kPaStageBytes + box * (br * 128);  // [dim half][64 positions][64 dims]
        tma_load_3d(dst, &A.km, 0, row, 0, bar, pol);
        tma_load_3d(dst + kPaHalf / 2, &A.km, 0, row, 1, bar, pol);
        tma_load_3d(dst + kPaHalf, &A.vm, 0, row, 0, bar, pol);
        tma_load_3d(dst + kPaHalf + kPaHalf / 2, &A.vm, 0, row, 1, bar, pol);
      }
      __device__ bool end(int) {
        tell(TcSeg{});  // no chunks: the CTA is done
        return false;
      }
    };
    issued = pa_produce<kTcUnit>(A, T.ring, plan, cta, lane,
                        Out{A, T, ring, abort, policy_evict_first(), lane, 1 << min(P.lps, 6), 0});
  } else if (warp == kTcMma || warp == kTcMmaO) {
    // ---------------------------------------------------------------- products
    // The warp walks as one and elects a thread for each batch of products:
    // their operands then stay in uniform registers (all by one thread of a
    // diverged warp: 252 us against 199).
    // (A descriptor's start address is its lowest bits, in 16-byte units: one
    // add moves it.)
    const uint64_t q0 = tc_desc(smem_addr(s_q), 16, 1024), p0 = tc_desc(smem_addr(s_p), 16, 1024);
    const uint64_t k0 = tc_desc(smem_addr(ring), 16, 1024), v0 = tc_desc(smem_addr(ring) + kPaHalf, 8192, 1024);
    constexpr uint32_t is = tc_idesc(64, false), io = tc_idesc(128, true);
    bool ok = true;
    for (int seg = 0;; ++seg) {
      ok = told(seg);
      if (!ok) break;
      const int st0 = __shfl_sync(0xffffffffu, T.seg[seg % kTcSegs].st0, 0);
      const int st1 = st0 + __shfl_sync(0xffffffffu, T.seg[seg % kTcSegs].count, 0);
      if (st0 == st1) break;
      done(seg);
      if (warp == kTcMma) {
        // S = Q K^T, up to four chunks ahead of what the softmax has read
        ok = wait(&T.q_full, (uint32_t)seg & 1u);
        for (int st = st0; ok && st < st1; ++st) {
          const int sl = st % kTcStages;
          ok = wait(&T.ring.full[sl], (uint32_t)(st / kTcStages) & 1u);
          if (ok && st > 3) ok = wait(&T.s_empty[st & 3], (uint32_t)((st >> 2) - 1) & 1u);
          if (!ok) break;
          tc_fence_after();
          const uint64_t k = k0 + (unsigned)(sl * (kPaStageBytes >> 4));
          if (tc_elect()) {
#pragma unroll
            for (int ks = 0; ks < 8; ++ks)
              tc_mma(tmem + kTcS + 64 * (st & 3), q0 + (ks >> 2) * 1024 + (ks & 3) * 2, k + (ks >> 2) * 512 + (ks & 3) * 2,
                     is, ks > 0);
            tc_commit(&T.s_full[st & 3]);
            if (st == st1 - 1) tc_commit(&T.q_empty);
          }
          __syncwarp();
        }
      } else {
        // O += P V
        for (int st = st0; st < st1; ++st) {
          const int sl = st % kTcStages, g = st & 1;
          ok = wait(&T.p_full[g], (uint32_t)(st >> 1) & 1u);
          if (!ok) break;
          const int pv = __shfl_sync(0xffffffffu, *reinterpret_cast<volatile int*>(&T.pv[g]), 0);
          tc_fence_after();
          const uint64_t p = p0 + (unsigned)(g * (kTcP >> 4)), v = v0 + (unsigned)(sl * (kPaStageBytes >> 4));
          const uint32_t d = tmem + kTcO + 128 * g;
          if (tc_elect()) {
            if ((pv & 15) == 15) {
#pragma unroll
              for (int ks = 0; ks < 4; ++ks) {
                tc_mma(d, p + 2 * ks, v + 128 * ks, io, ks > 0 || (pv & 16));
                tc_mma(d, p + 512 + 2 * ks, v + 128 * ks, io, true);
              }
            } else {
              bool acc = pv & 16;
#pragma unroll 1
              for (int ks = 0; ks < 4; ++ks) {
                if (!(pv >> ks & 1)) continue;
                tc_mma(d, p + 2 * ks, v + 128 * ks, io, acc);
                tc_mma(d, p + 512 + 2 * ks, v + 128 * ks, io, true);
                acc = true;
              }
            }
            tc_commit(&T.ring.empty[sl]);
            tc_commit(&T.o_done[g]);
          }
          __syncwarp();
        }
      }
      if (!ok) break;
    }
    if (!ok) *abort = 1;
    // every product has ended before the CTA frees its memory
    if (tc_elect()) {
      uint64_t* fin = &T.fin[warp - kTcMma];
      tc_commit(fin);
      mbar_wait_drain(fin, 0, kPaDrainNs);
    }
    __syncwarp();
  } else if (warp >= kTcLoader) {
    // ---------------------------------------------------------------- rows of Q
    const uint32_t q = smem_addr(s_q);
    bool ok = true;
    for (int seg = 0;; ++seg) {
      ok = told(seg);
      if (!ok) break;
      const TcSeg& D = T.seg[seg % kTcSegs];
      if (D.count == 0) break;
      // the segment's rows wait in registers until the last one's are done with
      const int nrow = D.n * a.group, c = lane & 15, i0 = lane >> 4;
      // (every second row: a head of the group, at least two, and the next
      // verify row after the last; with a division for each the one warp took
      // 4 us a segment)
      uint4 v[32];
      const int r0 = i0 / a.group;
      int head = i0 - r0 * a.group;
      const uint16_t* src = a.q + (D.q0 + r0) * a.qs + (D.kvh * a.group + head) * 128 + 8 * c;
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        v[u] = i0 + 2 * u < nrow ? *reinterpret_cast<const uint4*>(src) : make_uint4(0u, 0u, 0u, 0u);
        head += 2;
        src += 256;
        if (head >= a.group) {
          head -= a.group;
          src += a.qs - a.group * 128;
        }
      }
      done(seg);
      if (seg > 0) ok = wait(&T.q_empty, (uint32_t)(seg - 1) & 1u);
      if (!ok) break;
#pragma unroll
      for (int u = 0; u < 32; ++u) {
        const int i = i0 + 2 * u;
#pragma unroll
        for (int w = 0; w < 2; ++w)
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(q + (c >> 3) * 16384 + w * 8192 + i * 128 +
                                                                       (((c & 7) ^ (i & 7)) << 4)),
                       "r"(v[u].x), "r"(v[u].y), "r"(v[u].z), "r"(v[u].w)
                       : "memory");
      }
      asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
      __syncwarp();
      if (lane == 0) mbar_arrive(&T.q_full);
    }
    if (!ok) *abort = 1;
  } else {
    // ---------------------------------------------------------------- softmax
    const int g = warp >> 2, half = (warp >> 1) & 1, row = 32 * (warp & 1) + lane;  // 32 positions of a row
    const uint32_t t_lane = (uint32_t)(32 * (warp & 3)) << 16;
    const uint32_t t_s = tmem + t_lane + kTcS + 32 * half, t_o = tmem + t_lane + kTcO + 128 * g;
    const uint32_t p_row = smem_addr(s_p) + g * kTcP + row * 128;
    uint32_t xpar = 0;
    const float unit = a.plain ? a.scale_log2 : 1.f;
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
      const TcSeg& D = T.seg[seg % kTcSegs];
      const int st0 = D.st0, st1 = st0 + D.count;
      if (st0 == st1) break;
      const bool solo = st1 - st0 == 1;  // a segment of one chunk is its group's alone
      if (solo && (st0 & 1) != g) {
        done(seg);
        continue;
      }
      float m = -INFINITY, l = 0.f, slope = 0.f;
      bool has = false;
      // the last shared segment's outputs are out
      auto cleaned = [&]() {
        if (cleared != shared) ok = wait(&T.epi_done, (uint32_t)(shared - 1) & 1u);
        cleared = shared;
        return ok;
      };
      const bool live = row < D.n * a.group;
      const int r = live ? row / a.group : 0, h = D.kvh * a.group + (live ? row - r * a.group : 0);
      const int rp = D.len + r;  // the row's position
      if (a.slopes) slope = a.slopes[h] * 1.4426950408889634f;
      for (int st = st0 + ((st0 & 1) != g); st < st1; st += 2) {
        const int sl = st % kTcStages, own = st >> 1;
        const int j = D.j0 + st - st0, pos0 = (j < D.np ? D.cp + j : D.cm + j - D.np) * kPaChunk;
        // which 16-position slices some row sees some of, every row all of
        int any = 15, clear = 15;
        if (!pa_all(D.len, D.n, D.first, D.prefix, a.window, pos0, pos0 + 63)) {
          const int sp = pos0 + 16 * (lane & 3);
          any = __ballot_sync(0xffffffffu, pa_any(D.len, D.n, D.first, D.prefix, a.window, sp, sp + 15)) & 15;
          clear = __ballot_sync(0xffffffffu, pa_all(D.len, D.n, D.first, D.prefix, a.window, sp, sp + 15)) & 15;
        }
        // the scores of positions pos0 + 32 half + c
        ok = wait(&T.s_full[st & 3], (uint32_t)(st >> 2) & 1u);
        if (!ok) break;
        tc_fence_after();
        uint32_t sr[32];
        tc_ld32(t_s + 64 * (st & 3), sr);
        tc_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.s_empty[st & 3]);
        // in units of 1 / unit (log2 domain); plain scores are scaled with the exponential
        float s[32];
#pragma unroll
        for (int c = 0; c < 32; ++c) s[c] = __uint_as_float(sr[c]);
        if (!a.plain) {
          if (a.cap_log2 > 0.f) {
#pragma unroll
            for (int c = 0; c < 32; c += 2) pa_capped(a, s[c], s[c + 1]);
          } else {
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] *= a.scale_log2;
          }
          if (a.slopes) {
            const float d = (float)(pos0 + 32 * half - rp);
#pragma unroll
            for (int c = 0; c < 32; ++c) s[c] = __fmaf_rn(slope, d + (float)c, s[c]);
          }
        }
        unsigned long long see = ~0ull;
        if (clear != 15) {
          const int lo = a.window > 0 ? max(D.first, rp - a.window + 1) : D.first;
          see = tc_bits(lo - pos0, rp + 1 - pos0) | tc_bits(D.first - pos0, min(D.prefix, rp + 1) - pos0);
          const uint32_t mine = (uint32_t)(see >> (32 * half));
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (!(mine >> c & 1u)) s[c] = -INFINITY;
        }
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
        for (int c = 0; c < 32; ++c) mx[c & 3] = fmaxf(mx[c & 3], s[c]);
        if (!cleaned()) break;
        float(&s_top)[2][64] = T.top[own & 1][g];
        int(&s_odd)[4] = T.odd[own & 1][g];
        const float mine_top = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        s_top[half][row] = mine_top;
        const uint32_t v0 = smem_addr(ring + (size_t)sl * kPaStageBytes + kPaHalf);
        if (any & ~clear) {
          // slices with hidden positions: infinite or NaN values among them?
          // (each of the four warps a quarter of the slice's bytes)
          ok = wait(&T.ring.full[sl], (uint32_t)(st / kTcStages) & 1u);
          if (!ok) break;
          int odd = 0;
#pragma unroll
          for (int ks = 0; ks < 4; ++ks) {
            if (!((any & ~clear) >> ks & 1)) continue;
            const uint32_t at = v0 + ((warp >> 1) & 1) * 8192 + ks * 2048 + (warp & 1) * 1024 + lane * 16;
            bool bad = false;
#pragma unroll
            for (int u = 0; u < 2; ++u) {
              uint32_t w[4];
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                           : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                           : "r"(at + 512 * u));
#pragma unroll
              for (int i = 0; i < 4; ++i) bad |= __vcmpeq2(w[i] & 0x7F807F80u, 0x7F807F80u) != 0u;
            }
            odd |= __any_sync(0xffffffffu, bad) << ks;
          }
          if (lane == 0) s_odd[warp & 3] = odd;
        }
        if (!(ok = exchange())) break;
        const float top = unit * fmaxf(mine_top, s_top[half ^ 1][row]);
        float scale = 1.f;
        if (top > m) {
          const float up = top + kTcRoom;
          if (m != -INFINITY) scale = ex2(m - up);  // else the row's sums are zeros
          m = up;
          l *= scale;
        }
        const float ref = m == -INFINITY ? 0.f : m;  // nothing visible yet
        float add[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int c = 0; c < 32; ++c) {
          s[c] = ex2(__fmaf_rn(s[c], unit, -ref));
          add[c & 3] += s[c];
        }
        l += (add[0] + add[1]) + (add[2] + add[3]);
        // P's place (and O) is free when the product before has ended
        if (own > 0) ok = wait(&T.o_done[g], (uint32_t)(own - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        if (half == 0 && has && __any_sync(0xffffffffu, scale != 1.f)) {
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            tc_ld16(t_o + c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * scale);
            tc_st16(t_o + c, o);
          }
          tc_wait_st();
        }
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t hi[4], lo[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) pa_split(s[8 * c + 2 * u], s[8 * c + 2 * u + 1], hi[u], lo[u]);
          const uint32_t at = p_row + (((4 * half + c) ^ (row & 7)) << 4);
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(hi[0]), "r"(hi[1]), "r"(hi[2]), "r"(hi[3])
                       : "memory");
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(at + 8192), "r"(lo[0]), "r"(lo[1]), "r"(lo[2]), "r"(lo[3])
                       : "memory");
        }
        int pv = any;
        if (any & ~clear) {
          const int odd = s_odd[0] | s_odd[1] | s_odd[2] | s_odd[3];
          if (odd) {
            pv &= ~odd;
            // (the same for all four warps) the other half of the rows' P
            if (!(ok = exchange())) break;
#pragma unroll 1
            for (int c = 0; half == 0 && c < 128; c += 32) {
              uint32_t o[32];
              if (has) {
                tc_ld32(t_o + c, o);
                tc_wait_ld();
              } else {
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = 0u;
              }
#pragma unroll 1
              for (int p = 0; p < 64; ++p) {
                if (!(odd >> (p >> 4) & 1) || !(see >> p & 1ull)) continue;
                const uint32_t e = p_row + (((p >> 3) ^ (row & 7)) << 4) + 2 * (p & 7);
                uint16_t hi, lo;
                asm volatile("ld.shared.u16 %0, [%2];\n ld.shared.u16 %1, [%2 + 8192];" : "=h"(hi), "=h"(lo) : "r"(e));
                const float w = bf16_bits_to_float(hi) + bf16_bits_to_float(lo);
#pragma unroll
                for (int i = 0; i < 32; i += 2) {
                  const int dim = c + i;
                  const uint32_t v = lds32(v0 + (dim >> 6) * 8192 + p * 128 + ((((dim >> 3) & 7) ^ (p & 7)) << 4) + (dim & 7) * 2);
                  o[i] = __float_as_uint(__uint_as_float(o[i]) + w * __uint_as_float(v << 16));
                  o[i + 1] = __float_as_uint(__uint_as_float(o[i + 1]) + w * __uint_as_float(v & 0xFFFF0000u));
                }
              }
              __syncwarp();
              tc_st32(t_o + c, o);
            }
            tc_wait_st();
            has = true;
          }
        }
        if ((warp & 3) == 0 && lane == 0) *reinterpret_cast<volatile int*>(&T.pv[g]) = pv | (has ? 16 : 0);
        has = has || pv != 0;
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.p_full[g]);
      }
      if (!ok) break;
      // ---------------------------------------------------------------- the segment's end
      const bool whole = D.parts == 1;
      const size_t prow = (size_t)(cta * 2 + D.slot) * rows + row;
      // 16 dims of the row's output, or of this CTA's part of it
      auto put = [&](int c, const float (&v)[16]) {
        if (live && whole) {
          uint4* out = reinterpret_cast<uint4*>(a.o + (D.q0 + r) * a.os + h * 128 + c);
#pragma unroll
          for (int i = 0; i < 2; ++i)
            out[i] = make_uint4(pack_bf16(v[8 * i], v[8 * i + 1]), pack_bf16(v[8 * i + 2], v[8 * i + 3]),
                                pack_bf16(v[8 * i + 4], v[8 * i + 5]), pack_bf16(v[8 * i + 6], v[8 * i + 7]));
        } else if (live) {
          float4* out = reinterpret_cast<float4*>(A.part_o + prow * 128 + c);
#pragma unroll
          for (int i = 0; i < 4; ++i) __stcg(out + i, make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
        }
      };
      auto put_sums = [&](float M, float L) {
        if (live && whole && a.lse)
          a.lse[(size_t)(D.q0 + r) * a.nq + h] = L == 0.f ? -INFINITY : (M + log2f(L)) * 0.6931471805599453f;
        if (live && !whole) __stcg(reinterpret_cast<float2*>(A.part_ml + 2 * prow), make_float2(M, L));
        if (!whole && row == 0) A.rec[cta * 2 + D.slot] = {D.cf, D.parts, D.q0, D.n, D.kvh};
      };
      auto inverse = [&](float L) { return whole ? pa_inverse(L) : 1.f; };
      if (solo) {
        // One chunk: its group ends it while the other is at the next segment.
        // (The second half's l goes where the first half left its maximum, which
        // only the second half has read, and only the first writes again.)
        float& l1 = T.top[(st0 >> 1) & 1][g][0][row];
        if (half == 1) l1 = l;
        if (!(ok = exchange())) break;
        if (half == 0) {
          const float L = l + l1, f = inverse(L);
          if (has) ok = wait(&T.o_done[g], (uint32_t)(st0 >> 1) & 1u);
          if (!ok) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = 0; c < 128; c += 16) {
            uint32_t o[16];
            float v[16];
            if (has) tc_ld16(t_o + c, o);
            tc_wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) v[i] = has ? __uint_as_float(o[i]) * f : 0.f;
            put(c, v);
          }
          tc_fence_before();
          put_sums(m, L);
        }
        done(seg);
        continue;
      }
      // The second half's l joins the first's, and the groups hand theirs
      // over; then the two groups' first warps add both groups' sums, the
      // one's 64 dims and the other's.
      const int n0 = (st1 + 1) >> 1, n1 = st1 >> 1;  // the groups' chunks so far
      float(&s_ml)[2][64] = T.top[(g ? n1 : n0) & 1][g];
      if (!cleaned()) break;
      if (half == 1) s_ml[1][row] = l;
      if (!(ok = exchange())) break;
      if (half == 0) {
        s_ml[0][row] = m;
        s_ml[1][row] += l;
        if (row == 0) T.has[g] = has;
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.ml_full);
        ok = wait(&T.ml_full, (uint32_t)shared & 1u);
        const bool has0 = ok && T.has[0], has1 = ok && T.has[1];
        if (ok && has0) ok = wait(&T.o_done[0], (uint32_t)(n0 - 1) & 1u);
        if (ok && has1) ok = wait(&T.o_done[1], (uint32_t)(n1 - 1) & 1u);
        if (!ok) break;
        tc_fence_after();
        const float(&ml0)[2][64] = T.top[n0 & 1][0], (&ml1)[2][64] = T.top[n1 & 1][1];
        const float m0 = has0 ? ml0[0][row] : -INFINITY, m1 = has1 ? ml1[0][row] : -INFINITY, M = fmaxf(m0, m1);
        const float e0 = m0 == -INFINITY ? 0.f : ex2(m0 - M), e1 = m1 == -INFINITY ? 0.f : ex2(m1 - M);
        const float L = (has0 ? ml0[1][row] : 0.f) * e0 + (has1 ? ml1[1][row] : 0.f) * e1;
        const float f = inverse(L);
#pragma unroll 1
        for (int c = 64 * g; c < 64 * g + 64; c += 16) {
          uint32_t o0[16], o1[16];
          float v[16];
          if (has0) tc_ld16(tmem + t_lane + kTcO + c, o0);
          if (has1) tc_ld16(tmem + t_lane + kTcO + 128 + c, o1);
          tc_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            v[i] = has0 ? __uint_as_float(o0[i]) * e0 : 0.f;
            if (has1) v[i] += __uint_as_float(o1[i]) * e1;
            v[i] *= f;
          }
          put(c, v);
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&T.epi_done);
        if (g == 0) put_sums(M, L);
      }
      ++shared;
      done(seg);
    }
    if (!ok) *abort = 1;
  }
  tc_fence_before();
  __syncthreads();  // every warp is done with the ring and the tensor memory
  tc_fence_after();
  if (warp == kTcMma)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "n"(kTcCols));
  if (warp == kTcProducer && *abort && lane == 0) pa_drain(T.ring, issued, P.err);
}

cudaError_t launch_paged_attention_tc(const PagedAttnParams& A, int rows, cudaStream_t s) {
  constexpr int smem = 2 * kTcP + kTcQ + kTcStages * kPaStageBytes + (int)sizeof(TcTable);
  static_assert(smem <= 227 * 1024, "one CTA an SM");
  const cudaError_t e = prepare_kernel<k_paged_attn_tc>(smem);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(num_sms() < kPagedMaxCtas ? num_sms() : kPagedMaxCtas);
  cfg.blockDim = dim3(kTcThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, k_paged_attn_tc, A, rows);
}

}  // namespace moe
