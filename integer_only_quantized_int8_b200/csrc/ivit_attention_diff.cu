// ivit_attention_diff.cu -- differential attention on sm_100a (ivit_attention_diff):
// per head two query/key pairs of width 64, one value of width 128, and
//   ctx = sat_8((b_o sum_j (P1 - P2)_ij V_j) >> c_o),
// P1 and P2 the integer Shiftmax maps of the two pairs, P2's IntDiv numerator
// carrying the weight lambda_h 2^M.
//
// One CTA per SM walks work items (tile of query rows, head, image).  Both maps
// of an item are worked on at once, each by a softmax group of eight warps:
//   warp 0       TMA producer: Q and K of both pairs (one ring), V (another);
//   warps 1, 2   S issuer of map 0 / 1: S = Q K^T in chunks of keys into the
//                map's TMEM score buffer;
//   warp 3       P V issuer: O = P1 V, then O += (-P2) V onto the same
//                accumulator: P1 <= 128 is a u8 operand, -P2 >= -128 an s8 one,
//                so the difference needs no ninth bit and V is read as it is;
//   warps 4-19   two softmax groups;
//   warps 20-23  output readout of the previous item, one per TMEM lane quarter.
//
// Shiftmax needs a row's maximum before any exponential and its sum before any
// probability, so a row is passed over three times:
//   pass 1  reads each score once from TMEM, keeps the raw maximum (the logit
//           requant is monotone) and writes the saturated 8-bit logits back to
//           TMEM, four to a column -- a quarter of the score's space, which
//           frees the score buffer for the next chunk at once and makes 640
//           keys of two maps fit;
//   pass 2  looks e = ShiftExp(L - max L) up and sums it; where every e fits a byte
//           (I0 <= 255) it takes the logit's place, summed by dp4a;
//   pass 3  takes e (or looks it up again) and writes P in the logits' place, which is also
//           the layout in which the P V MMA takes its A operand from TMEM
//           (lane = row, four 8-bit values of K per column): P never passes
//           through shared memory.
// The table address of a score is one dp4a: byte * (-128) + (base + 128 max L),
// the table being replicated once per shared-memory bank (row stride 128 bytes,
// lane l reads copy l: no conflicts).  The four warps of a lane quarter's rows
// (w, w + 4 of each group) split a row's keys; partial maxima and sums meet in
// shared memory.
//
// What bounds it: 64 x 197 tokens in 6 head pairs are 19.2 M warp instructions, 15.9
// per 32 scores (rows and keys padded to 224), hence 16.5 us of issue slots and 17 of
// the ALU pipe, against 37.3 us measured from HBM (577 tokens, batch 16: 67.9; 197
// tokens, 3 pairs, one image: 9.8).  The rest is latency: the passes are dependent
// chains (TMEM load, table address, table load, byte pack) of four softmax warps per
// scheduler with one TMEM load in flight each, the slots are half used and waits for
// loads are the largest stall; no pipe is above 42 %.
//
// Keys past the last one are masked where they lie: out of the maximum and the
// sum, and to P = 0.  Whatever their logit bytes hold, their table addresses stay
// inside shared memory (|max L - L| <= 255 entries of 128 bytes, and the table
// lies above 64 KB of operands).
#include <climits>

#include "ivit_common.cuh"
#include "ivit_internal.h"

namespace ivit {
namespace {

constexpr int kHeadDim = 64;   // width of one query / key of a pair
constexpr int kValDim = 128;   // width of a value
constexpr int kQTile = 128;    // TMEM lanes; a tile holds up to this many query rows
constexpr int kSoftWarps = 8;  // per map
constexpr int kMaxChunk = 128;  // keys per score chunk
constexpr int kChunkUnits = kMaxChunk / 32;  // 16-key units of a chunk per half
constexpr int kSoftBase = 4, kReadBase = kSoftBase + 2 * kSoftWarps;
constexpr int kDiffThreads = 32 * (kReadBase + 4);

struct DiffLayout {
  int n64, n32, n16;
  int chunk, nchunks;          // keys per score chunk (a multiple of 16), chunks
  int lcols;                   // TMEM columns of one map's logits / P
  int sep;                     // O has columns of its own (else the score buffers')
  int o_col, s_col, s_stride;  // first columns of O and of map 0's score buffer
  int qk_bytes, v_bytes, depth;
  int v_off, tab_off, part_off, bar_off, total;
};

inline DiffLayout diff_layout(int N) {
  DiffLayout L;
  L.n64 = (N + 63) / 64 * 64;
  L.n32 = (N + 31) / 32 * 32;
  L.n16 = (N + 15) / 16 * 16;
  L.lcols = (L.n32 / 4 + 31) / 32 * 32;
  // 512 columns: both maps' logits, O, and the two score buffers of at least 96
  L.sep = 2 * L.lcols + kValDim + 2 * 96 <= 512;
  const int avail = (512 - 2 * L.lcols - (L.sep ? kValDim : 0)) / 2 / 32 * 32;
  const int widest = avail < kMaxChunk ? avail : kMaxChunk;
  L.nchunks = (L.n16 + widest - 1) / widest;
  L.chunk = ((L.n16 + L.nchunks - 1) / L.nchunks + 15) / 16 * 16;
  L.o_col = 2 * L.lcols;
  L.s_col = 2 * L.lcols + (L.sep ? kValDim : 0);
  L.s_stride = avail;
  L.qk_bytes = 2 * (kQTile + L.n64) * kHeadDim;
  L.v_bytes = L.n64 * kValDim;
  const int rest = 256 * 128 + 2 * 2 * 2 * kQTile * 4 + 256;
  L.depth = 2 * (L.qk_bytes + L.v_bytes) + rest + 1024 <= 227 * 1024 ? 2 : 1;
  L.v_off = L.depth * L.qk_bytes;
  L.tab_off = L.v_off + L.depth * L.v_bytes;
  L.part_off = L.tab_off + 256 * 128;
  L.bar_off = L.part_off + 2 * 2 * 2 * kQTile * 4;  // [map][max, sum][half][row]
  L.total = L.bar_off + 256;
  return L;
}

struct DiffArgs {
  int32_t B, N, H;
  int32_t logit_b, logit_c, bq;
  int32_t k_s, ks_lo, ks_hi;
  int32_t I0, M, k_out;
  const int32_t* lam;
  int32_t out_b, out_c, out_bq, out_fast, o_lo, o_hi;
  DiffLayout L;
  int8_t* ctx;
  int* status;
  int32_t withhold;  // diagnostic: CTA 0's producer stops before this local item (-1: never)
};

IVIT_DEV uint32_t pack_sat4_diff(int32_t y0, int32_t y1, int32_t y2, int32_t y3) {
  uint32_t t, d;
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(t) : "r"(y3), "r"(y2), "r"(0u));
  asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(d) : "r"(y1), "r"(y0), "r"(t));
  return d;
}

// floor(b S / 2^c) before the saturation: one mul.hi when bq = b 2^(32 - c) fits a positive int32
template <bool FASTQ>
IVIT_DEV int32_t logit_of(int32_t S, const DiffArgs& a) {
  if (FASTQ) return __mulhi(a.bq, S);
  const int64_t q = ((int64_t)a.logit_b * (int64_t)S) >> a.logit_c;
  return (int32_t)(q < (int64_t)INT_MIN ? (int64_t)INT_MIN : (q > (int64_t)INT_MAX ? (int64_t)INT_MAX : q));
}

// bounded wait that also gives up at once when another thread has
IVIT_DEV bool diff_wait(uint64_t* bar, uint32_t parity, int* status, volatile int* abort_flag) {
  if (*abort_flag) return false;
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (mbar_try_wait_sleep(bar, parity)) return true;
    if (*abort_flag) return false;
    if (globaltimer_ns() - t0 > kWaitBudgetNs) {
      report_timeout(status);
      *abort_flag = 1;
      return false;
    }
  }
}

// named barrier of the two warps that share a map's 32 rows (ids 1..8)
IVIT_DEV void pair_bar(int id) { asm volatile("bar.sync %0, 64;" ::"r"(1 + id) : "memory"); }

IVIT_DEV void tmem_st4(uint32_t taddr, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x4.b32 [%0], {%1, %2, %3, %4};" ::"r"(taddr), "r"(a), "r"(b), "r"(c),
               "r"(d)
               : "memory");
}
IVIT_DEV void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr)
               : "memory");
}
IVIT_DEV void tmem_st8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(taddr), "r"(r[0]),
               "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}
IVIT_DEV void tmem_ld8_wait(uint32_t (&r)[8]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7])
               :
               : "memory");
}

// D[tmem] (+)= A[tmem] * B[smem], kind::i8, int32 accumulate; single thread.
IVIT_DEV void umma_i8_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t b_desc, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::i8 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
      "r"(a_tmem), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}

IVIT_DEV int32_t lds32(uint32_t addr) {
  int32_t v;
  asm("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr));
  return v;
}

// Streams units 0..n-1 of eight TMEM columns through body(r, u).  One load at a
// time: the other warps cover its latency, and a second one in flight spills at
// the 80 registers that 24 warps leave a thread (101 us instead of 43.7 then).
template <typename F>
IVIT_DEV void stream_units(uint32_t t, int n, F&& body) {
  uint32_t r[8];
#pragma unroll 1
  for (int u = 0; u < n; ++u) {
    tmem_ld8(t + (uint32_t)(8 * u), r);
    tmem_ld8_wait(r);
    body(r, u);
  }
}

// exponentials of the four logits of w; base = table + 4 lane + 128 max L
IVIT_DEV void exp4(uint32_t w, int32_t base, uint32_t (&e)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) e[i] = (uint32_t)lds32((uint32_t)__dp4a((int)w, (int)(0x80u << (8 * i)), base));
}

// the low (TOP: top) bytes of four words
template <bool TOP>
IVIT_DEV uint32_t bytes4(uint32_t e0, uint32_t e1, uint32_t e2, uint32_t e3) {
  constexpr uint32_t sel = TOP ? 0x0073u : 0x0040u;
  return __byte_perm(__byte_perm(e0, e1, sel), __byte_perm(e2, e3, sel), 0x5410u);
}

// the first n bytes of a word (n <= 0: none, n >= 4: all)
IVIT_DEV uint32_t first_bytes(uint32_t w, int n) { return n >= 4 ? w : (n <= 0 ? 0u : w & ((1u << (8 * n)) - 1u)); }

// Pass 1 of one 16-key unit: the raw maximum, and the saturated logits as four words.
template <bool FASTQ, bool NARROW, bool RAGGED>
IVIT_DEV void logits16(const uint32_t (&r)[16], int lim, const DiffArgs& a, int32_t& mx, uint32_t (&lw)[4]) {
  int32_t m0 = mx, m1 = INT_MIN;
#pragma unroll
  for (int i = 0; i < 16; i += 4) {
    m0 = __vimax3_s32(m0, RAGGED && i >= lim ? INT_MIN : (int32_t)r[i], RAGGED && i + 1 >= lim ? INT_MIN : (int32_t)r[i + 1]);
    m1 = __vimax3_s32(m1, RAGGED && i + 2 >= lim ? INT_MIN : (int32_t)r[i + 2],
                      RAGGED && i + 3 >= lim ? INT_MIN : (int32_t)r[i + 3]);
  }
  mx = max(m0, m1);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    int32_t l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      l[i] = logit_of<FASTQ>((int32_t)r[4 * q + i], a);
      if (NARROW) l[i] = min(max(l[i], a.ks_lo), a.ks_hi);
    }
    lw[q] = pack_sat4_diff(l[0], l[1], l[2], l[3]);
  }
}

// Pass 2 of one 32-key unit: the exponentials' sum; E8 leaves them in r, a byte each.
template <bool E8, bool RAGGED>
IVIT_DEV void sum32(uint32_t (&r)[8], int lim, int32_t base, uint32_t& sum) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t e[4];
    exp4(r[q], base, e);
    if (E8) {
      uint32_t w = bytes4<false>(e[0], e[1], e[2], e[3]);
      if (RAGGED) w = first_bytes(w, lim - 4 * q);
      r[q] = w;
      sum = __dp4a(w, 0x01010101u, sum);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += RAGGED && 4 * q + i >= lim ? 0u : e[i];
    }
  }
}

// Pass 3 of one 32-key unit: r becomes P or -P bytes.  With X = dvs e, P = (Dv e) >>
// pshift is X's top byte (SHR: after a further shift by rsh), and -P that of
// -X + 2^24 - 1, so the sign costs nothing: mul = dvs, add = 0 or mul = -dvs, add =
// 2^24 - 1 (SHR: |mul| and, byte by byte, -p = (p + 127) ^ 127 for p <= 128).
template <bool E8, bool SHR, bool RAGGED>
IVIT_DEV void prob32(uint32_t (&r)[8], int lim, int32_t base, uint32_t mul, uint32_t add, int rsh, uint32_t neg) {
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    uint32_t e[4];
    if (E8) {
#pragma unroll
      for (int i = 0; i < 4; ++i) e[i] = __byte_perm(r[q], 0u, 0x4440u + i);
    } else {
      exp4(r[q], base, e);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) e[i] = SHR ? (e[i] * mul) >> rsh : e[i] * mul + add;
    uint32_t w = bytes4<true>(e[0], e[1], e[2], e[3]);
    if (SHR) w = (w + neg) ^ neg;
    if (RAGGED && !E8) w = first_bytes(w, lim - 4 * q);
    r[q] = w;
  }
}

// One row of O to 128 bytes of ctx: sat_8((b_o O) >> c_o).
template <bool FAST>
IVIT_DEV void read_out(uint32_t t_o, bool live, int8_t* dst, const DiffArgs& a) {
#pragma unroll 1
  for (int pr = 0; pr < 4; ++pr) {
    uint32_t ra[16], rb[16];
    tmem_ld16(t_o + (uint32_t)(32 * pr), ra);
    tmem_ld16(t_o + (uint32_t)(32 * pr + 16), rb);
    tmem_ld_wait_regs2(ra, rb);
    uint32_t packed[8];
#pragma unroll
    for (int wd = 0; wd < 8; ++wd) {
      int32_t y[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int32_t acc = (int32_t)(wd < 4 ? ra[wd * 4 + e] : rb[(wd - 4) * 4 + e]);
        if (FAST) {
          y[e] = __mulhi(a.out_bq, acc);  // floor(b_o acc / 2^c_o), exact
        } else {
          const int64_t v = (int64_t)a.out_b * min(max(acc, a.o_lo), a.o_hi);  // |v >> c| < 2^31 after the clamp
          y[e] = (int32_t)__funnelshift_r((uint32_t)v, (uint32_t)(v >> 32), (uint32_t)a.out_c);
        }
      }
      packed[wd] = pack_sat4_diff(y[0], y[1], y[2], y[3]);
    }
    if (live) {
      reinterpret_cast<int4*>(dst + 32 * pr)[0] = make_int4(packed[0], packed[1], packed[2], packed[3]);
      reinterpret_cast<int4*>(dst + 32 * pr)[1] = make_int4(packed[4], packed[5], packed[6], packed[7]);
    }
  }
}

// FASTQ: the logit requant is one mul.hi.  NARROW: k_s < 8, so the saturation is
// not the byte pack's.  E8: every exponential fits a byte (I0 <= 255).
template <bool FASTQ, bool NARROW, bool E8>
__global__ void __launch_bounds__(kDiffThreads, 1)
    attention_diff_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tmV,
                          const __grid_constant__ DiffArgs a) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int N = a.N;
  const DiffLayout& L = a.L;
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + L.bar_off);
  uint64_t* qk_full = bars + 0;    // [2] Q and K of both pairs landed
  uint64_t* qk_empty = bars + 2;   // [2] both maps' scores computed (one commit per S issuer)
  uint64_t* v_full = bars + 4;     // [2]
  uint64_t* v_empty = bars + 6;    // [2] P V of the item done
  uint64_t* s_full = bars + 8;     // [2] a score chunk of map g
  uint64_t* s_empty = bars + 10;   // [2] read by the group's warps
  uint64_t* p_full = bars + 12;    // [2] P of map g in TMEM
  uint64_t* p_empty = bars + 14;   // [2] consumed by P V
  uint64_t* o_full = bars + 16;
  uint64_t* o_empty = bars + 17;   // read out (one arrival per readout warp)
  uint64_t* drain = bars + 18;     // every MMA of the CTA done (one commit per issuer)
  uint32_t* tslot = reinterpret_cast<uint32_t*>(bars + 19);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(bars + 20);

  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int qtiles = (N + kQTile - 1) / kQTile;
  const int n_items = qtiles * a.H * a.B;
  const int n_local = n_items > (int)blockIdx.x ? (n_items - 1 - (int)blockIdx.x) / (int)gridDim.x + 1 : 0;
  const int D = a.H * kValDim;

  if (tid == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(&qk_full[i], 1);
      mbar_init(&qk_empty[i], 2);
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kSoftWarps);
      mbar_init(&p_full[i], kSoftWarps);
      mbar_init(&p_empty[i], 1);
    }
    mbar_init(o_full, 1);
    mbar_init(o_empty, 4);
    mbar_init(drain, 3);
    *abort_flag = 0;
    fence_barrier_init();
    prefetch_tensormap(&tm);
    prefetch_tensormap(&tmV);
  }
  if (warp == 3) {
    __syncwarp();
    tmem_alloc(tslot, 512);
    tmem_relinquish();
  }
  // tab[t * 32 + l] = ShiftExp(-t) for every lane l: one evaluation per entry,
  // staged in the partials' space
  int32_t* stage_t = reinterpret_cast<int32_t*>(smem + L.part_off);
  if (tid < 256) stage_t[tid] = tid < (1 << a.k_s) ? shift_exp(-tid, a.I0) : 0;
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  for (int i4 = tid; i4 < 256 * 8; i4 += kDiffThreads) {
    const int32_t e = stage_t[i4 >> 3];
    reinterpret_cast<int4*>(smem + L.tab_off)[i4] = make_int4(e, e, e, e);
  }
  __syncthreads();
  const uint32_t tmem = *tslot;
  pdl_wait();  // qkv comes from the previous kernel
  pdl_launch_dependents();

  if (warp == 0) {
    // ------------------------------------------------------------ TMA producer
    if (lane == 0) {
      for (int j = 0; j < n_local; ++j) {
        const int s = j % L.depth;
        const uint32_t ph = (uint32_t)((j / L.depth) & 1);
        const int item = (int)blockIdx.x + j * (int)gridDim.x;
        const int h = item % a.H, img = (item / a.H) % a.B, qt = item / (a.H * a.B);
        const int row0 = img * N;
        if (!diff_wait(&qk_empty[s], ph ^ 1, a.status, abort_flag)) break;
        if (j == a.withhold && blockIdx.x == 0) break;  // diagnostic (ivit_selftest_withhold)
        uint8_t* st = smem + s * L.qk_bytes;
        mbar_arrive_expect_tx(&qk_full[s], (uint32_t)L.qk_bytes);
        for (int m = 0; m < 2; ++m) {
          uint8_t* q = st + m * (kQTile + L.n64) * kHeadDim;
          const int col = h * kValDim + m * kHeadDim;
          for (int i = 0; i < 2; ++i)
            tma_load_2d(q + i * 64 * kHeadDim, &tm, col, row0 + qt * kQTile + 64 * i, &qk_full[s]);
          for (int i = 0; i < L.n64 / 64; ++i)
            tma_load_2d(q + (kQTile + 64 * i) * kHeadDim, &tm, D + col, row0 + 64 * i, &qk_full[s]);
        }
        if (!diff_wait(&v_empty[s], ph ^ 1, a.status, abort_flag)) break;
        uint8_t* v = smem + L.v_off + s * L.v_bytes;
        mbar_arrive_expect_tx(&v_full[s], (uint32_t)L.v_bytes);
        for (int i = 0; i < L.n64 / 64; ++i)
          tma_load_2d(v + 64 * i * kValDim, &tmV, 2 * D + h * kValDim, row0 + 64 * i, &v_full[s]);
      }
    }
  } else if (warp <= 2) {
    // ------------------------------------------------------------ S issuer of map g
    if (lane == 0) {
      const int g = warp - 1;
      const uint32_t d_s = tmem + (uint32_t)(L.s_col + g * L.s_stride);
      uint32_t n = 0;  // chunks issued
      bool ok = true;
      for (int j = 0; j < n_local && ok; ++j) {
        const int s = j % L.depth;
        if (!diff_wait(&qk_full[s], (uint32_t)((j / L.depth) & 1), a.status, abort_flag)) break;
        // O of the previous item lies in the score buffers
        if (!L.sep && j > 0 && !diff_wait(o_empty, (uint32_t)((j - 1) & 1), a.status, abort_flag)) break;
        const uint32_t qa = smem_u32(smem + s * L.qk_bytes + g * (kQTile + L.n64) * kHeadDim);
        const uint32_t ka = qa + kQTile * kHeadDim;
        for (int c = 0; c < L.nchunks; ++c, ++n) {
          if (!diff_wait(&s_empty[g], (n & 1) ^ 1, a.status, abort_flag)) {
            ok = false;
            break;
          }
          tc_fence_after();
          const int w = min(L.chunk, L.n16 - c * L.chunk);
          const uint32_t idesc = idesc_i8(kQTile, w, true, true, false);
          const uint32_t kc = ka + (uint32_t)(c * L.chunk * kHeadDim);
#pragma unroll
          for (int k = 0; k < kHeadDim / 32; ++k)
            umma_i8(d_s, smem_desc(qa + k * 32, 16, 512, kSwizzle64B), smem_desc(kc + k * 32, 16, 512, kSwizzle64B),
                    idesc, k != 0);
          umma_commit(&s_full[g]);
        }
        umma_commit(&qk_empty[s]);
      }
      umma_commit(drain);
    }
  } else if (warp == 3) {
    // ------------------------------------------------------------ P V issuer
    if (lane == 0) {
      const uint32_t d_o = tmem + (uint32_t)L.o_col;
      bool ok = true;
      for (int j = 0; j < n_local && ok; ++j) {
        const int s = j % L.depth;
        const uint32_t ph = (uint32_t)(j & 1);
        ok = diff_wait(&v_full[s], (uint32_t)((j / L.depth) & 1), a.status, abort_flag) &&
             diff_wait(&p_full[0], ph, a.status, abort_flag);
        // O's columns: read out (own region), or no longer holding either map's scores
        if (ok) ok = L.sep ? (j == 0 || diff_wait(o_empty, ph ^ 1, a.status, abort_flag))
                           : diff_wait(&p_full[1], ph, a.status, abort_flag);
        for (int g = 0; g < 2 && ok; ++g) {
          if (g == 1 && L.sep) ok = diff_wait(&p_full[1], ph, a.status, abort_flag);
          if (!ok) break;
          tc_fence_after();
          const uint32_t idesc = idesc_i8(kQTile, kValDim, g == 1, true, true);
          const uint32_t pa = tmem + (uint32_t)(g * L.lcols);
          const uint32_t va = smem_u32(smem + L.v_off + s * L.v_bytes);
          for (int k = 0; k < L.n32 / 32; ++k)
            umma_i8_ta(d_o, pa + (uint32_t)(8 * k),
                       smem_desc(va + (uint32_t)(32 * k * kValDim), 1024, 1024, kSwizzle128B), idesc, (uint32_t)(g | k));
          umma_commit(&p_empty[g]);
        }
        if (!ok) break;
        umma_commit(&v_empty[s]);
        umma_commit(o_full);
      }
      umma_commit(drain);
      mbar_wait(drain, 0, a.status);  // before TMEM is released
    }
  } else if (warp < kReadBase) {
    // ------------------------------------------------------------ softmax group of map g
    const int sw = warp - kSoftBase;
    const int g = sw / kSoftWarps;
    const int half = (sw >> 2) & 1;  // which half of the row's keys
    const int quarter = warp & 3;
    const int pair = 4 * g + quarter;
    const int row = quarter * 32 + lane;
    const uint32_t t_lane = tmem + ((uint32_t)(quarter * 32) << 16);
    const uint32_t t_s = t_lane + (uint32_t)(L.s_col + g * L.s_stride);
    const uint32_t t_l = t_lane + (uint32_t)(g * L.lcols);
    int32_t* part = reinterpret_cast<int32_t*>(smem + L.part_off) + g * (4 * kQTile);  // [max, sum][half][row]
    const uint32_t tab = smem_u32(smem + L.tab_off) + (uint32_t)(4 * lane);
    // passes 2 and 3: this half's 32-key units (8 logit columns each); the last unit of
    // all is ragged when it holds keys past N
    const int units = L.n32 / 32;
    const int u_lo = half ? (units + 1) / 2 : 0, u_n = (half ? units : (units + 1) / 2) - u_lo;
    const int u_ragged = (N & 31) != 0 && u_lo + u_n == units && u_n > 0 ? u_n - 1 : -1;
    const int lim_ragged = N - 32 * (units - 1);
    const uint32_t t_u = t_l + (uint32_t)(8 * u_lo);
    // P = (Dv e) >> pshift in the top byte of (Dv << lsh) e >> rsh: |.| <= 2^(23 + k_out) <= 2^31
    const int pshift = a.M - (a.k_out - 1);
    const int lsh = max(24 - pshift, 0), rsh = max(pshift - 24, 0);
    const uint32_t neg = g == 1 ? 0x7F7F7F7Fu : 0u;
    // item = h + H (img + B qt), advanced without divisions
    int h = (int)blockIdx.x % a.H, img = (int)blockIdx.x / a.H % a.B, qt = (int)blockIdx.x / (a.H * a.B);
    const int step_h = (int)gridDim.x % a.H, step_i = (int)gridDim.x / a.H;
    uint32_t n = 0;  // chunks seen
    bool ok = true;
    for (int j = 0; j < n_local; ++j) {
      // warps whose rows all lie past the tile or the image's last token skip the passes
      const bool rows = quarter * 32 < min(kQTile, N - qt * kQTile);
      uint32_t num = 1u << a.M;  // IntDiv's numerator
      if (g == 1) num = (uint32_t)min(max(__ldg(a.lam + h), 0), 1 << a.M);

      // ---- pass 1: maximum of the raw scores, 8-bit logits into TMEM
      // (written once the chunk is read and the previous item's P has been consumed)
      int32_t mx = INT_MIN;
      for (int c = 0; c < L.nchunks; ++c, ++n) {
        if (ok) ok = diff_wait(&s_full[g], n & 1, a.status, abort_flag);
        ok = __all_sync(0xffffffffu, ok);
        tc_fence_after();
        const int key0 = c * L.chunk + 16 * half;
        const int nu = (min(L.chunk, L.n16 - c * L.chunk) / 16 - half + 1) / 2;  // 16-key units, taken by the halves in turn
        uint32_t lw[kChunkUnits][4];
        if (ok && rows) {
#pragma unroll
          for (int u = 0; u < kChunkUnits; ++u)
            if (u < nu) {
              uint32_t r[16];
              tmem_ld16(t_s + (uint32_t)(16 * half + 32 * u), r);
              tmem_ld_wait_regs(r);
              const int lim = N - (key0 + 32 * u);
              if (lim >= 16)
                logits16<FASTQ, NARROW, false>(r, 16, a, mx, lw[u]);
              else
                logits16<FASTQ, NARROW, true>(r, lim, a, mx, lw[u]);
            }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&s_empty[g]);
        if (c == 0 && j > 0) {
          if (ok) ok = diff_wait(&p_empty[g], (uint32_t)((j - 1) & 1), a.status, abort_flag);
          ok = __all_sync(0xffffffffu, ok);
          tc_fence_after();
        }
        if (ok && rows) {
#pragma unroll
          for (int u = 0; u < kChunkUnits; ++u)
            if (u < nu) tmem_st4(t_l + (uint32_t)((key0 + 32 * u) / 4), lw[u][0], lw[u][1], lw[u][2], lw[u][3]);
        }
      }
      if (rows) {
        tmem_st_wait();
        part[half * kQTile + row] = mx;
        tc_fence_before();
        pair_bar(pair);
        tc_fence_after();
        const int32_t smax = max(part[row], part[kQTile + row]);
        const int32_t lmax = min(max(logit_of<FASTQ>(smax, a), a.ks_lo), a.ks_hi);
        const int32_t base = (int32_t)tab + 128 * lmax;

        // ---- pass 2: row sum of the exponentials
        uint32_t sum = 0;
        if (ok) {
          stream_units(t_u, u_n, [&](uint32_t(&r)[8], int u) {
            if (u != u_ragged)
              sum32<E8, false>(r, 32, base, sum);
            else
              sum32<E8, true>(r, lim_ragged, base, sum);
            if (E8) tmem_st8(t_u + (uint32_t)(8 * u), r);
          });
          if (E8) tmem_st_wait();
        }
        part[(2 + half) * kQTile + row] = (int32_t)sum;
        pair_bar(pair);
        sum = (uint32_t)part[2 * kQTile + row] + (uint32_t)part[3 * kQTile + row];
        const uint32_t dvs = (num / max(sum, 1u)) << lsh;
        const uint32_t mul = g == 0 || rsh != 0 ? dvs : 0u - dvs, add = g == 0 ? 0u : 0x00FFFFFFu;

        // ---- pass 3: P in the logits' place
        if (ok) {
          if (rsh == 0)
            stream_units(t_u, u_n, [&](uint32_t(&r)[8], int u) {
              if (E8 || u != u_ragged)
                prob32<E8, false, false>(r, 32, base, mul, add, 0, 0u);
              else
                prob32<E8, false, true>(r, lim_ragged, base, mul, add, 0, 0u);
              tmem_st8(t_u + (uint32_t)(8 * u), r);
            });
          else
            stream_units(t_u, u_n, [&](uint32_t(&r)[8], int u) {
              prob32<E8, true, true>(r, u != u_ragged ? 32 : lim_ragged, base, mul, 0u, rsh, neg);
              tmem_st8(t_u + (uint32_t)(8 * u), r);
            });
        }
        tmem_st_wait();
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&p_full[g]);
      h += step_h;
      img += step_i;
      if (h >= a.H) {
        h -= a.H;
        ++img;
      }
      while (img >= a.B) {
        img -= a.B;
        ++qt;
      }
    }
  } else {
    // ------------------------------------------------------------ readout warps
    const int quarter = warp & 3;
    const int row = quarter * 32 + lane;
    bool ok = true;
    for (int j = 0; j < n_local; ++j) {
      const int item = (int)blockIdx.x + j * (int)gridDim.x;
      const int h = item % a.H, img = (item / a.H) % a.B, qt = item / (a.H * a.B);
      if (ok) ok = diff_wait(o_full, (uint32_t)(j & 1), a.status, abort_flag);
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      const int nrow = min(kQTile, N - qt * kQTile);  // rows of the tile
      if (ok && quarter * 32 < nrow) {
        const uint32_t t_o = tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)L.o_col;
        int8_t* dst = a.ctx + (int64_t)(img * N + qt * kQTile + row) * D + h * kValDim;
        if (a.out_fast)
          read_out<true>(t_o, row < nrow, dst, a);
        else
          read_out<false>(t_o, row < nrow, dst, a);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(o_empty);
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 3) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

}  // namespace

ivit_status launch_attention_diff(const DeviceCtx& dc, const int8_t* qkv, int32_t B, int32_t N, int32_t H,
                                  ivit_dyadic logit, int32_t k_s, int32_t I0, int32_t M, int32_t k_out,
                                  const int32_t* lam, ivit_dyadic out, int8_t* ctx, cudaStream_t stream) {
  const int64_t T = (int64_t)B * N;
  const uint64_t width = (uint64_t)3 * kValDim * (uint64_t)H;
  CUtensorMap tm, tmV;  // boxes of 64 rows: 64 columns (Q, K) and 128 (V)
  ivit_status st = encode_tmap_2d_u8(&tm, qkv, width, (uint64_t)T, width, kHeadDim, 64, CU_TENSOR_MAP_SWIZZLE_64B);
  if (st != IVIT_OK) return st;
  st = encode_tmap_2d_u8(&tmV, qkv, width, (uint64_t)T, width, kValDim, 64, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != IVIT_OK) return st;
  DiffArgs a{};
  a.B = B;
  a.N = N;
  a.H = H;
  const bool fastq = logit.c >= 1 && (int64_t)logit.b < ((int64_t)1 << (logit.c - 1));
  a.logit_b = logit.b;
  a.logit_c = logit.c;
  a.bq = fastq ? (int32_t)((int64_t)logit.b << (32 - logit.c)) : 0;
  a.k_s = k_s;
  a.ks_lo = -(1 << (k_s - 1));
  a.ks_hi = (1 << (k_s - 1)) - 1;
  a.I0 = I0;
  a.M = M;
  a.k_out = k_out;
  a.lam = lam;
  a.out_b = out.b;
  a.out_c = out.c;
  a.out_fast = out.c >= 1 && (int64_t)out.b < ((int64_t)1 << (out.c - 1));
  a.out_bq = a.out_fast ? (int32_t)((int64_t)out.b << (32 - out.c)) : 0;
  // acc in [-u, u], u = 128 / 2^s with 2^s <= b / 2^c < 2^(s+1), keeps every unsaturated result,
  // saturates the rest the same way and keeps (b acc) >> c within int32
  a.o_lo = INT_MIN;
  a.o_hi = INT_MAX;
  if (out.b != 0) {
    int bl = 0;
    while (bl < 31 && (out.b >> bl) != 0) ++bl;
    const int sh = bl - 1 - out.c;
    const int64_t u = sh >= 7 ? 1 : (sh >= 0 ? (128 >> sh) : ((int64_t)128 << (-sh)));
    a.o_hi = (int32_t)(u > INT_MAX ? INT_MAX : u);
    a.o_lo = -a.o_hi;
  }
  a.ctx = ctx;
  a.status = dc.status;
  a.withhold = take_withhold(kWithholdAttention);
  const int64_t items = (int64_t)((N + kQTile - 1) / kQTile) * H * B;
  if (items > 0x7fffffff) return IVIT_ERR_UNSUPPORTED;
  a.L = diff_layout(N);
  const int smem = a.L.total + 1024;
  using Kernel = void (*)(CUtensorMap, CUtensorMap, DiffArgs);
  static const Kernel kernels[8] = {
      attention_diff_kernel<false, false, false>, attention_diff_kernel<false, false, true>,
      attention_diff_kernel<false, true, false>,  attention_diff_kernel<false, true, true>,
      attention_diff_kernel<true, false, false>,  attention_diff_kernel<true, false, true>,
      attention_diff_kernel<true, true, false>,   attention_diff_kernel<true, true, true>};
  const Kernel kern = kernels[(fastq ? 4 : 0) + (k_s < 8 ? 2 : 0) + (I0 <= 255 ? 1 : 0)];
  static bool attr_done[64];  // per device; benign race: the attribute value is the same
  if (!attr_done[dc.device]) {
    for (const Kernel k : kernels)
      if (cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, 227 * 1024) != cudaSuccess)
        return IVIT_ERR_CUDA;
    attr_done[dc.device] = true;
  }
  const unsigned grid = (unsigned)(items < dc.num_sms ? items : dc.num_sms);
  const cudaError_t e = launch_pdl(kern, dim3(grid), dim3(kDiffThreads), (size_t)smem, stream, tm, tmV, a);
  note_launch();
  return e == cudaSuccess ? IVIT_OK : IVIT_ERR_CUDA;
}

}  // namespace ivit
