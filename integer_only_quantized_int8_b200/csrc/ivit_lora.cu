// ivit_lora.cu -- the down projection of per-request low-rank adapters beside
// an int8 linear layer (ivit_linear_lora):
//   t_ir = sat_8((b_t[a, r] * sum_k X_ik A_a[r, k]) >> c_t[a, r]),  a = idx[i / rows]
// The up projection t B_a^T accumulates inside the GEMM (ivit_gemm.cu, LORA).
//
// One CTA per 128 tokens of one request: tcgen05.mma kind::i8 with M = 128
// tokens and N = R rank entries, X and A_a k-slices of 128 bytes brought by
// TMA into a ring.  X comes through a tensor map [request, row of request, K],
// so a tile never reads another request's rows.  A request without an adapter
// has no tile to do.
#include <climits>

#include "ivit_common.cuh"
#include "ivit_internal.h"

namespace ivit {
namespace {

constexpr int kDownThreads = 192;  // TMA warp, MMA warp, four epilogue warps (one per TMEM lane quarter)
constexpr int kDownTile = 128;     // tokens per tile
constexpr int kDownSlice = 128;    // bytes of K per stage
constexpr int kDownStages = 4;

struct DownArgs {
  const int32_t* b;
  const int8_t* c;
  const int32_t* idx;
  int64_t rows;  // tokens per request
  uint32_t tiles;  // per request
  int32_t K, R, n, round;
  int8_t* T;
  int* status;
};

__host__ __device__ constexpr int down_stage_bytes(int R) { return (kDownTile + R) * kDownSlice; }

__global__ void __launch_bounds__(kDownThreads)
    lora_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                     const DownArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int R = args.R;
  const int stage_bytes = down_stage_bytes(R);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kDownStages * stage_bytes);
  uint64_t* empty = full + kDownStages;
  uint64_t* tfull = empty + kDownStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tfull + 1);
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int num_kb = (args.K + kDownSlice - 1) / kDownSlice;
  const uint32_t tcols = R <= 32 ? 32u : (R <= 64 ? 64u : 128u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kDownStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    mbar_init(tfull, 1);
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
  const int64_t i0 = (int64_t)(blockIdx.x % args.tiles) * kDownTile;  // first row of the tile within the request
  if (a >= 0 && a < args.n) {
    if (warp == 0) {
      if (lane == 0) {
        for (int kb = 0; kb < num_kb; ++kb) {
          const int s = kb % kDownStages;
          if (!mbar_wait(&empty[s], (uint32_t)((kb / kDownStages) & 1) ^ 1u, args.status)) break;
          uint8_t* st = smem + s * stage_bytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
          tma_load_3d(st, &tmX, kb * kDownSlice, (int32_t)i0, (int32_t)q, &full[s]);
          tma_load_3d(st + kDownTile * kDownSlice, &tmA, kb * kDownSlice, 0, a, &full[s]);
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
        const uint32_t idesc = idesc_i8(kDownTile, R, true, true, false);
        for (int kb = 0; kb < num_kb; ++kb) {
          const int s = kb % kDownStages;
          if (!mbar_wait(&full[s], (uint32_t)((kb / kDownStages) & 1), args.status)) break;
          tc_fence_after();
          const uint32_t xa = smem_u32(smem + s * stage_bytes);
          const uint32_t aa = xa + kDownTile * kDownSlice;
#pragma unroll
          for (int k = 0; k < kDownSlice / 32; ++k)
            umma_i8(tmem, smem_desc(xa + k * 32, 16, 1024, kSwizzle128B), smem_desc(aa + k * 32, 16, 1024, kSwizzle128B),
                    idesc, (uint32_t)(kb | k));
          umma_commit(&empty[s]);
        }
        umma_commit(tfull);
      }
    } else {
      const int quarter = warp & 3;
      const int64_t i = i0 + quarter * 32 + lane;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull, 0, args.status));
      tc_fence_after();
      if (ok) {
        int8_t* dst = args.T + (q * args.rows + i) * R;
        for (int r0 = 0; r0 < R; r0 += 16) {
          uint32_t v[16];
          tmem_ld16(tmem + ((uint32_t)(quarter * 32) << 16) + (uint32_t)r0, v);
          tmem_ld_wait_regs(v);
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            uint32_t word = 0;
#pragma unroll
            for (int f = 0; f < 4; ++f) {
              const int64_t col = (int64_t)a * R + r0 + 4 * e + f;
              const int32_t b = __ldg(args.b + col), c = __ldg(args.c + col);
              int64_t p = (int64_t)b * (int32_t)v[4 * e + f];  // |p| < 2^31 2^28
              if (args.round && c > 0) p += (int64_t)1 << (c - 1);
              p >>= c;
              word |= ((uint32_t)(p < -128 ? -128 : (p > 127 ? 127 : p)) & 0xFFu) << (8 * f);
            }
            w[e] = word;
          }
          if (i < args.rows) *reinterpret_cast<int4*>(dst + r0) = make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
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

ivit_status launch_lora_down(const DeviceCtx& dc, const int8_t* X, int64_t M, int32_t K, const int8_t* A,
                             const int32_t* b_t, const int8_t* c_t, bool round, const LoraGemm& lora, int8_t* T,
                             cudaStream_t stream) {
  const int64_t requests = M / lora.rows;
  CUtensorMap tmX, tmA;
  ivit_status st = encode_tmap_3d_u8(&tmX, X, (uint64_t)K, (uint64_t)lora.rows, (uint64_t)requests, kDownSlice,
                                     kDownTile, CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != IVIT_OK) return st;
  st = encode_tmap_3d_u8(&tmA, A, (uint64_t)K, (uint64_t)lora.R, (uint64_t)lora.n, kDownSlice, (uint32_t)lora.R,
                         CU_TENSOR_MAP_SWIZZLE_128B);
  if (st != IVIT_OK) return st;
  const int64_t tiles = (lora.rows + kDownTile - 1) / kDownTile;  // tiles * requests <= M < 2^31
  const DownArgs a{b_t, c_t, lora.idx, lora.rows, (uint32_t)tiles, K, lora.R, lora.n, round ? 1 : 0, T, dc.status};
  const int smem = kDownStages * down_stage_bytes(lora.R) + (2 * kDownStages + 2) * 8 + 1024;
  static bool attr_done[64];  // per device; benign race: the attribute value is the same
  if (!attr_done[dc.device]) {
    if (cudaFuncSetAttribute(lora_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             kDownStages * down_stage_bytes(128) + 2048) != cudaSuccess)
      return IVIT_ERR_CUDA;
    attr_done[dc.device] = true;
  }
  const cudaError_t e = launch_pdl(lora_down_kernel, dim3((unsigned)(tiles * requests)), dim3(kDownThreads),
                                   (size_t)smem, stream, tmX, tmA, a);
  note_launch();
  return e == cudaSuccess ? IVIT_OK : IVIT_ERR_CUDA;
}

}  // namespace ivit
