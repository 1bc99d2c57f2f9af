// ivit_lora.cu -- the down projection of per-request low-rank adapters beside
// an int8 linear layer (ivit_linear_lora):
//   t_ir = sat_8((b_t[a, r] * sum_k X_ik A_a[r, k]) >> c_t[a, r]),  a = idx[i / rows]
// The up projection t B_a^T accumulates inside the GEMM (ivit_gemm.cu, LORA).
//
// One CTA per tile of up to 128 tokens of one request: tcgen05.mma kind::i8 with
// M = 128 tokens and N = R rank entries, X and A_a k-slices of 128 bytes brought
// by TMA into a ring.  X comes through a tensor map [request, row of request, K],
// so a tile never reads another request's rows.  A request without an adapter
// has no tile to do.
//
// Reading X bounds it in principle (25.8 MB for fc2 of ViT-L at batch 32: 4 us
// from HBM), latency in practice:
//   - one thread takes about 260 ns to wait for a k-slice, issue its four MMAs
//     and commit, so four threads take the slices in turn, each onto an
//     accumulator of its own (the epilogue adds them): 6 slices took 1.5 us of a
//     3.5 us kernel with one;
//   - tiles hold fewer than 128 tokens while there are SMs to take more of them.
//     Splitting K over a cluster instead, with the partial sums through
//     distributed shared memory, cost 4-6 us after the last MMA;
//   - the requant is one mul.hi when every multiplier of the adapter is below one
//     half, as in the GEMM.
// Back to back: 3.5 us for one row of K = 768, 3.7 for ViT-B QKV at batch 64 (R =
// 16), 4.1 for ViT-L fc1 at batch 32 (R = 32), 9.1 for its fc2 (R = 64).
#include <climits>

#include "ivit_common.cuh"
#include "ivit_internal.h"

namespace ivit {
namespace {

constexpr int kIssuers = 4;        // MMA-issuing warps, an accumulator each
constexpr int kDownEpiWarps = 8;   // two per TMEM lane quarter
constexpr int kDownThreads = 32 * (1 + kIssuers + kDownEpiWarps);
constexpr int kDownRows = 128;     // TMEM lanes of a tile; it may use the first few only
constexpr int kDownSlice = 128;    // bytes of K per stage
constexpr int kDownMaxStages = 16;
constexpr int kDownSmem = 200 * 1024;  // at most, the ring as deep as that allows

struct DownArgs {
  const int32_t* b;
  const int8_t* c;
  const int32_t* idx;
  int64_t rows;    // tokens per request
  uint32_t tiles;  // per request
  int32_t tile_rows;
  int32_t K, R, n, round;
  int32_t stages;  // ring depth, a multiple of kIssuers
  int8_t* T;
  int* status;
};

__host__ __device__ constexpr int down_stage_bytes(int R, int tile_rows) { return (tile_rows + R) * kDownSlice; }
// after the ring: what an MMA's 128 rows may reach past a shorter last X tile, barriers, b and c of the adapter
__host__ __device__ constexpr int down_fixed_bytes(int R) { return kDownRows * kDownSlice + 512 + 8 * R; }

// Sixteen rank entries of one row: sat_8((b t + half) >> c), |b t| < 2^31 2^28.
// FAST: b < 2^(c - 1) everywhere and b holds b 2^(32 - c).
template <bool FAST>
IVIT_DEV int4 requant16(const int32_t (&t)[16], const int32_t* b, const int32_t* c, bool round) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    int32_t y[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int32_t bb = b[4 * e + f], tt = t[4 * e + f];
      if (FAST) {
        y[f] = __mulhi(bb, tt);
        if (round) y[f] += (int32_t)(((uint32_t)bb * (uint32_t)tt) >> 31);
      } else {
        int64_t p = (int64_t)bb * tt;
        const int32_t cc = c[4 * e + f];
        if (round && cc > 0) p += (int64_t)1 << (cc - 1);
        p >>= cc;
        y[f] = (int32_t)(p < -128 ? -128 : (p > 127 ? 127 : p));
      }
    }
    uint32_t hi;
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(hi) : "r"(y[3]), "r"(y[2]), "r"(0u));
    asm("cvt.pack.sat.s8.s32.b32 %0, %1, %2, %3;" : "=r"(w[e]) : "r"(y[1]), "r"(y[0]), "r"(hi));
  }
  return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
}

__global__ void __launch_bounds__(kDownThreads)
    lora_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ DownArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int R = args.R, stages = args.stages;
  const int stage_bytes = down_stage_bytes(R, args.tile_rows);
  // a stage is A_a's R rows, then X's tile_rows; the X operand's 128 rows may run on into what follows
  uint8_t* after = smem + stages * stage_bytes + kDownRows * kDownSlice;
  uint64_t* full = reinterpret_cast<uint64_t*>(after);
  uint64_t* empty = full + kDownMaxStages;
  uint64_t* tfull = empty + kDownMaxStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tfull + 1);
  int32_t* s_b = reinterpret_cast<int32_t*>(after + 512);
  int32_t* s_c = s_b + R;
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_kb = (args.K + kDownSlice - 1) / kDownSlice;
  const int used = num_kb < kIssuers ? num_kb : kIssuers;  // issuers (and accumulators) with work
  const uint32_t acc_cols = (uint32_t)((R + 31) & ~31);
  const uint32_t tcols = acc_cols <= 32 ? 128u : (acc_cols <= 64 ? 256u : 512u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, (uint32_t)used);
    fence_barrier_init();
    prefetch_tensormap(&tmX);
    prefetch_tensormap(&tmA);
  }
  if (warp == 1) {
    __syncwarp();
    tmem_alloc(tslot, tcols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tslot;
  pdl_wait();  // X, idx and the buffer of T belong to earlier kernels
  pdl_launch_dependents();
  const int64_t q = blockIdx.x / args.tiles;
  const int32_t a = __ldg(args.idx + q);
  const int64_t i0 = (int64_t)(blockIdx.x % args.tiles) * args.tile_rows;  // first row of the tile within the request
  if (a >= 0 && a < args.n) {
    if (warp == 0) {
      if (lane == 0) {
        int s = 0;
        uint32_t ph = 0;
        for (int k = 0; k < num_kb; ++k) {
          if (!mbar_wait(&empty[s], ph ^ 1u, args.status)) break;
          uint8_t* st = smem + s * stage_bytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
          tma_load_3d(st, &tmA, k * kDownSlice, 0, a, &full[s]);
          tma_load_3d(st + R * kDownSlice, &tmX, k * kDownSlice, (int32_t)i0, (int32_t)q, &full[s]);
          if (++s == stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp <= kIssuers) {
      // issuer w takes slices w, w + 4, ...: with a ring of a multiple of four stages
      // those are stages of its own, so it never waits for a phase not its own
      const int w = warp - 1;
      if (lane == 0 && w < used) {
        const uint32_t idesc = idesc_i8(kDownRows, R, true, true, false);
        const uint64_t d0 = smem_desc(smem_u32(smem), 16, 1024, kSwizzle128B);
        const uint32_t lo0 = (uint32_t)d0, hi = (uint32_t)(d0 >> 32);
        const uint32_t acc = tmem + (uint32_t)w * acc_cols;
        int s = w;
        uint32_t ph = 0;
        for (int kb = w; kb < num_kb; kb += kIssuers) {
          if (!mbar_wait(&full[s], ph, args.status)) break;
          tc_fence_after();
          const uint32_t al = lo0 + (uint32_t)((s * stage_bytes) >> 4);
          const uint32_t xl = al + (uint32_t)((R * kDownSlice) >> 4);
          if (kb == w)
            umma_i8(acc, ((uint64_t)hi << 32) | xl, ((uint64_t)hi << 32) | al, idesc, 0u);
          else
            umma_i8_acc(acc, xl, hi, al, hi, idesc);
#pragma unroll
          for (int k = 1; k < kDownSlice / 32; ++k) umma_i8_acc(acc, xl + 2 * k, hi, al + 2 * k, hi, idesc);
          if (kb + stages < num_kb) umma_commit(&empty[s]);  // the stage is used again
          s += kIssuers;
          if (s >= stages) {
            s -= stages;
            ph ^= 1;
          }
        }
        umma_commit(tfull);
      }
    } else {
      const int e = (int)threadIdx.x - 32 * (1 + kIssuers);  // 0..255
      bool fast = true;
      if (e < R) {
        const int32_t b = __ldg(args.b + (int64_t)a * R + e), c = __ldg(args.c + (int64_t)a * R + e);
        fast = b == 0 || (c >= 1 && (int64_t)b < ((int64_t)1 << (c - 1)));
        s_b[e] = b;
        s_c[e] = c;
      }
      uint32_t all;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\tbar.red.and.pred p, 1, 256, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
          : "=r"(all)
          : "r"((uint32_t)fast)
          : "memory");
      if (all && e < R) s_b[e] = s_b[e] == 0 ? 0 : (int32_t)((uint32_t)s_b[e] << (32 - s_c[e]));
      asm volatile("bar.sync 1, 256;" ::: "memory");
      const int quarter = warp & 3;
      const int half = (warp - 1 - kIssuers) >> 2;  // the two warps of a quarter take 16 rank entries in turn
      const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull, 0, args.status));
      tc_fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
      const int row = quarter * 32 + lane;
      const int64_t i = i0 + row;
      int8_t* dst = args.T + (q * args.rows + i) * R;
      if (ok && quarter * 32 < args.tile_rows) {
        for (int r0 = 16 * half; r0 < R; r0 += 32) {
          int32_t t[16];
#pragma unroll
          for (int f = 0; f < 16; ++f) t[f] = 0;
          for (int w = 0; w < used; ++w) {
            uint32_t v[16];
            tmem_ld16(t_row + (uint32_t)w * acc_cols + (uint32_t)r0, v);
            tmem_ld_wait_regs(v);
#pragma unroll
            for (int f = 0; f < 16; ++f) t[f] += (int32_t)v[f];
          }
          const int4 y = all ? requant16<true>(t, s_b + r0, s_c + r0, args.round != 0)
                             : requant16<false>(t, s_b + r0, s_c + r0, args.round != 0);
          if (row < args.tile_rows && i < args.rows) *reinterpret_cast<int4*>(dst + r0) = y;
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, tcols);
  }
}

}  // namespace

ivit_status launch_lora_down(const DeviceCtx& dc, const int8_t* X, int64_t M, int32_t K, bool round,
                             const LoraGemm& lora, cudaStream_t stream) {
  const int64_t requests = M / lora.rows;
  // as many tiles of equal height (a multiple of the swizzle's eight rows) as still go round once
  int64_t per_request = requests < dc.num_sms ? dc.num_sms / requests : 1;
  if (per_request < (lora.rows + kDownRows - 1) / kDownRows) per_request = (lora.rows + kDownRows - 1) / kDownRows;
  const int tile_rows = (int)(((lora.rows + per_request - 1) / per_request + 7) / 8 * 8);
  const int64_t tiles = (lora.rows + tile_rows - 1) / tile_rows;  // tiles * requests <= M < 2^31
  CUtensorMap tmX, tmA;
  ivit_status st = encode_tmap_3d_u8(&tmX, X, (uint64_t)K, (uint64_t)lora.rows, (uint64_t)requests, kDownSlice,
                                     (uint32_t)tile_rows, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != IVIT_OK) return st;
  st = encode_tmap_3d_u8(&tmA, lora.A, (uint64_t)K, (uint64_t)lora.R, (uint64_t)lora.n, kDownSlice, (uint32_t)lora.R,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != IVIT_OK) return st;
  const int num_kb = (K + kDownSlice - 1) / kDownSlice;
  const int stage = down_stage_bytes(lora.R, tile_rows), fixed = down_fixed_bytes(lora.R) + 1024;
  int stages = (kDownSmem - fixed) / stage / kIssuers * kIssuers;  // at least four: stage <= 32 KB
  const int need = (num_kb + kIssuers - 1) / kIssuers * kIssuers;
  if (stages > need) stages = need;
  if (stages > kDownMaxStages) stages = kDownMaxStages;
  const DownArgs a{lora.b_t, lora.c_t, lora.idx, lora.rows, (uint32_t)tiles, tile_rows, K, lora.R, lora.n, round ? 1 : 0, stages, lora.T,
                   dc.status};
  static bool attr_done[64];  // per device; benign race: the attribute value is the same
  if (!attr_done[dc.device]) {
    if (cudaFuncSetAttribute(lora_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDownSmem) != cudaSuccess)
      return IVIT_ERR_CUDA;
    attr_done[dc.device] = true;
  }
  // Up to one tile per SM is kept to one CTA per SM (more than half its shared
  // memory): two on the SMs that the kernel before leaves first start the GEMM's
  // equal shares there late (ViT-L fc1 34.5 us instead of 31.9).
  int smem = stages * stage + fixed;
  if (tiles * requests <= dc.num_sms && smem < 116 * 1024) smem = 116 * 1024;
  const cudaError_t e = launch_pdl(lora_down_kernel, dim3((unsigned)(tiles * requests)), dim3(kDownThreads), (size_t)smem,
                                   stream, tmX, tmA, a);
  note_launch();
  return e == cudaSuccess ? IVIT_OK : IVIT_ERR_CUDA;
}

}  // namespace ivit
