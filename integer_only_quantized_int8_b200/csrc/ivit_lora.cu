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
//
// Reading X bounds it, and a tile's k-slices come one after another, so a long
// reduction with few tiles is split over a cluster of CTAs: each keeps the
// partial sums of its stretch of K and sends every CTA the rows that CTA
// finishes (st.shared::cluster); after a cluster barrier each adds what it got
// and requantises its 128 / split rows.  (fc2 of ViT-L at batch 32, K = 4096, 64
// tiles: 13 us with one CTA each.)
#include <climits>

#include "ivit_common.cuh"
#include "ivit_internal.h"

namespace ivit {
namespace {

constexpr int kDownThreads = 192;  // TMA warp, MMA warp, four epilogue warps (one per TMEM lane quarter)
constexpr int kDownTile = 128;     // tokens per tile
constexpr int kDownSlice = 128;    // bytes of K per stage
constexpr int kDownSmem = 200 * 1024;  // at most, the ring as deep as that allows

struct DownArgs {
  const int32_t* b;
  const int8_t* c;
  const int32_t* idx;
  int64_t rows;    // tokens per request
  uint32_t tiles;  // per request
  int32_t K, R, n, round;
  int32_t stages, split;  // ring depth; CTAs (the cluster) per tile: 1, 2 or 4
  int8_t* T;
  int* status;
};

__host__ __device__ constexpr int down_stage_bytes(int R) { return (kDownTile + R) * kDownSlice; }
__host__ __device__ constexpr int down_bars_bytes() { return 512; }  // barriers of up to 16 stages
__host__ __device__ constexpr int down_tab_bytes(int R) { return 8 * R; }  // b and c of the adapter
__host__ __device__ constexpr int down_part_bytes(int R, int split) { return split > 1 ? 4 * kDownTile * R : 0; }
constexpr int kDownMaxStages = 16;

// sixteen rank entries of one row: sat_8((b t + half) >> c), |b t| < 2^31 2^28
IVIT_DEV int4 requant16(const int32_t (&t)[16], const int32_t* b, const int32_t* c, bool round) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    uint32_t word = 0;
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      int64_t p = (int64_t)b[4 * e + f] * t[4 * e + f];
      const int32_t cc = c[4 * e + f];
      if (round && cc > 0) p += (int64_t)1 << (cc - 1);
      p >>= cc;
      word |= ((uint32_t)(p < -128 ? -128 : (p > 127 ? 127 : p)) & 0xFFu) << (8 * f);
    }
    w[e] = word;
  }
  return make_int4((int)w[0], (int)w[1], (int)w[2], (int)w[3]);
}

IVIT_DEV void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kDownThreads)
    lora_down_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmA,
                     const __grid_constant__ DownArgs args) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = align_smem_1024(smem_raw);
  const int R = args.R;
  const int stage_bytes = down_stage_bytes(R);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + args.stages * stage_bytes);
  uint64_t* empty = full + kDownMaxStages;
  uint64_t* tfull = empty + kDownMaxStages;
  uint32_t* tslot = reinterpret_cast<uint32_t*>(tfull + 1);
  int32_t* s_b = reinterpret_cast<int32_t*>(smem + args.stages * stage_bytes + down_bars_bytes());
  int32_t* s_c = s_b + R;
  int32_t* s_part = s_c + R;  // [split][R][128 / split], from every CTA of the cluster
  const int warp = threadIdx.x >> 5;
  const int lane = threadIdx.x & 31;
  const int split = args.split;
  const int rank = (int)blockIdx.x % split;
  const int num_kb = (args.K + kDownSlice - 1) / kDownSlice;
  const int kb0 = num_kb * rank / split, nkb = num_kb * (rank + 1) / split - kb0;  // this CTA's slices, at least one
  const uint32_t tcols = R <= 32 ? 32u : (R <= 64 ? 64u : 128u);

  if (threadIdx.x == 0) {
    for (int s = 0; s < args.stages; ++s) {
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
  if (split > 1) cluster_sync();  // every CTA of the cluster has started before its shared memory is written
  pdl_wait();  // X, idx and the buffer of T belong to earlier kernels
  pdl_launch_dependents();
  const uint32_t tile = blockIdx.x / (uint32_t)split;
  const int64_t q = tile / args.tiles;
  const int32_t a = __ldg(args.idx + q);
  const int64_t i0 = (int64_t)(tile % args.tiles) * kDownTile;  // first row of the tile within the request
  const bool has = a >= 0 && a < args.n;                        // the same in all of a cluster
  if (has) {
    if (warp == 0) {
      if (lane == 0) {
        int s = 0;
        uint32_t ph = 0;
        for (int k = 0; k < nkb; ++k) {
          if (!mbar_wait(&empty[s], ph ^ 1u, args.status)) break;
          uint8_t* st = smem + s * stage_bytes;
          mbar_arrive_expect_tx(&full[s], (uint32_t)stage_bytes);
          tma_load_3d(st, &tmX, (kb0 + k) * kDownSlice, (int32_t)i0, (int32_t)q, &full[s]);
          tma_load_3d(st + kDownTile * kDownSlice, &tmA, (kb0 + k) * kDownSlice, 0, a, &full[s]);
          if (++s == args.stages) {
            s = 0;
            ph ^= 1;
          }
        }
      }
    } else if (warp == 1) {
      if (lane == 0) {
        const uint32_t idesc = idesc_i8(kDownTile, R, true, true, false);
        int s = 0;
        uint32_t ph = 0;
        for (int kb = 0; kb < nkb; ++kb) {
          if (!mbar_wait(&full[s], ph, args.status)) break;
          tc_fence_after();
          const uint32_t xa = smem_u32(smem + s * stage_bytes);
          const uint32_t aa = xa + kDownTile * kDownSlice;
#pragma unroll
          for (int k = 0; k < kDownSlice / 32; ++k)
            umma_i8(tmem, smem_desc(xa + k * 32, 16, 1024, kSwizzle128B), smem_desc(aa + k * 32, 16, 1024, kSwizzle128B),
                    idesc, (uint32_t)(kb | k));
          umma_commit(&empty[s]);
          if (++s == args.stages) {
            s = 0;
            ph ^= 1;
          }
        }
        umma_commit(tfull);
      }
    } else {
      const int e = (int)threadIdx.x - 64;  // 0..127
      if (e < R) {
        s_b[e] = __ldg(args.b + (int64_t)a * R + e);
        s_c[e] = __ldg(args.c + (int64_t)a * R + e);
      }
      asm volatile("bar.sync 1, 128;" ::: "memory");
      const int quarter = warp & 3;
      const bool ok = __all_sync(0xffffffffu, mbar_wait(tfull, 0, args.status));
      tc_fence_after();
      const uint32_t t_row = tmem + ((uint32_t)(quarter * 32) << 16);
      if (split == 1) {
        const int64_t i = i0 + quarter * 32 + lane;
        int8_t* dst = args.T + (q * args.rows + i) * R;
        for (int r0 = 0; ok && r0 < R; r0 += 16) {
          uint32_t v[16];
          tmem_ld16(t_row + (uint32_t)r0, v);
          tmem_ld_wait_regs(v);
          int32_t t[16];
#pragma unroll
          for (int f = 0; f < 16; ++f) t[f] = (int32_t)v[f];
          const int4 w = requant16(t, s_b + r0, s_c + r0, args.round != 0);
          if (i < args.rows) *reinterpret_cast<int4*>(dst + r0) = w;
        }
      } else {
        const int per = kDownTile / split;                                   // rows each CTA finishes
        const int dest = (quarter * 32) / per, at = (quarter * 32) % per + lane;
        uint32_t base;
        asm("mapa.shared::cluster.u32 %0, %1, %2;"
            : "=r"(base)
            : "r"(smem_u32(s_part + rank * R * per + at)), "r"((uint32_t)dest));
        for (int r0 = 0; r0 < R; r0 += 16) {
          uint32_t v[16];
          tmem_ld16(t_row + (uint32_t)r0, v);
          tmem_ld_wait_regs(v);
#pragma unroll
          for (int f = 0; f < 16; ++f)
            asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(base + (uint32_t)(4 * per * (r0 + f))), "r"(v[f])
                         : "memory");
        }
      }
    }
  }
  if (split > 1) {
    __syncwarp();  // every warp whole again for the aligned barrier
    cluster_sync();
    if (has && warp >= 2) {
      const int per = kDownTile / split;
      const int e = (int)threadIdx.x - 64, at = e % per;
      const int64_t i = i0 + rank * per + at;
      int8_t* dst = args.T + (q * args.rows + i) * R;
      for (int r0 = 16 * (e / per); r0 < R && i < args.rows; r0 += 16 * split) {
        int32_t t[16];
#pragma unroll
        for (int f = 0; f < 16; ++f) {
          t[f] = 0;
          for (int src = 0; src < split; ++src) t[f] += s_part[(src * R + r0 + f) * per + at];
        }
        *reinterpret_cast<int4*>(dst + r0) = requant16(t, s_b + r0, s_c + r0, args.round != 0);
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
  // a reduction of at least eight slices is split while the SMs are not all busy
  const int num_kb = (K + kDownSlice - 1) / kDownSlice;
  int split = 1;
  while (split < 4 && num_kb >= 8 * split && tiles * requests * split * 2 <= dc.num_sms) split *= 2;
  const int fixed = down_bars_bytes() + down_tab_bytes(lora.R) + down_part_bytes(lora.R, split) + 1024;
  int stages = (kDownSmem - fixed) / down_stage_bytes(lora.R);
  const int per_cta = (num_kb + split - 1) / split;
  if (stages > per_cta) stages = per_cta;
  if (stages > kDownMaxStages) stages = kDownMaxStages;
  const DownArgs a{b_t, c_t, lora.idx, lora.rows, (uint32_t)tiles, K, lora.R, lora.n, round ? 1 : 0, stages, split, T,
                   dc.status};
  static bool attr_done[64];  // per device; benign race: the attribute value is the same
  if (!attr_done[dc.device]) {
    if (cudaFuncSetAttribute(lora_down_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDownSmem) != cudaSuccess)
      return IVIT_ERR_CUDA;
    attr_done[dc.device] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(tiles * requests * split));
  cfg.blockDim = dim3(kDownThreads);
  cfg.dynamicSmemBytes = (size_t)(stages * down_stage_bytes(lora.R) + fixed);
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)split;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = split > 1 ? 2 : 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, lora_down_kernel, tmX, tmA, a);
  note_launch();
  return e == cudaSuccess ? IVIT_OK : IVIT_ERR_CUDA;
}

}  // namespace ivit
