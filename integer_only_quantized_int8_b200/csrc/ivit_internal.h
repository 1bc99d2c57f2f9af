// ivit_internal.h -- launchers shared between the operator files and the C ABI.
#pragma once

#include <cstdint>
#include <cuda.h>
#include <cuda_runtime.h>

#include "../../include/ivit.h"

namespace ivit {

enum EpiMode : int { kEpiPlain = 0, kEpiResidual = 1, kEpiGelu = 2 };

struct GeluParams {
  int32_t I0, M, k_out;
  ivit_dyadic out;
};

// Per-device context: SM count, the status word's device address.
struct DeviceCtx {
  int device;
  int num_sms;
  int* status;
};
ivit_status device_ctx(DeviceCtx* out);

// Count a kernel launch (for ivit_launch_count).
void note_launch(int n = 1);

// Diagnostics (ivit_selftest_withhold): the index at which the next launch of
// the given kernel has its producer stop, or -1; taking it clears it.
enum WithholdKernel : int { kWithholdGemm = 1, kWithholdAttention = 2 };
int32_t take_withhold(int kernel);

// Launch with programmatic stream serialization: the kernel may start while
// the previous kernel of the stream finishes; it must call pdl_wait() before
// touching that kernel's outputs or writing global memory.
template <typename... KArgs, typename... Args>
cudaError_t launch_pdl(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t stream,
                       Args&&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, static_cast<Args&&>(args)...);
}

ivit_status encode_tmap_2d_u8(CUtensorMap* map, const void* base, uint64_t inner, uint64_t outer,
                              uint64_t row_stride_bytes, uint32_t box_inner, uint32_t box_outer,
                              CUtensorMapSwizzle swizzle);

// The same for a contiguous [d2 x d1 x d0] byte tensor with boxes of
// box0 x box1 x 1 (d0 a multiple of 16).
ivit_status encode_tmap_3d_u8(CUtensorMap* map, const void* base, uint64_t d0, uint64_t d1, uint64_t d2,
                              uint32_t box0, uint32_t box1, CUtensorMapSwizzle swizzle);

// The host-side checks of one encoder-block call other than those of its
// workspace (parameters, alignment, sizes, attention configuration).
ivit_status check_block_args(const ivit_block_params* p, const int8_t* x, const int8_t* y, int32_t B, int32_t N);

// Low-rank adapters beside a GEMM: request q = rows [q * rows, (q + 1) * rows)
// of X adds t B_a^T, t = sat_8((b_t (X A_a^T)) >> c_t), a = idx[q], to its
// accumulators.
struct LoraGemm {
  int8_t* T;           // [M x R], the workspace
  const int8_t* A;     // [n x R x K]
  const int32_t* b_t;  // [n x R]
  const int8_t* c_t;   // [n x R]
  const int8_t* B;     // [n x N x R]
  const int32_t* idx;  // [M / rows]; outside [0, n): no adapter
  int32_t n, R;
  int64_t rows;
};

// t of every request with an adapter into lora.T (the rows of the others are
// left as they were).
ivit_status launch_lora_down(const DeviceCtx& dc, const int8_t* X, int64_t M, int32_t K, bool round,
                             const LoraGemm& lora, cudaStream_t stream);

// The kernel that launch_gemm takes for a layer with adapters (only the sizes in lg are looked at).
struct LoraForm {
  enum Way : int { kOneKernel = 1, kMma = 2, kDp4a = 3, kDp4aLong = 4 };  // dp4a: ranks to 32, above
  Way way;
  int tokens;       // of a tile
  bool by_adapter;  // the reduction axis runs over the adapters, not the tile's requests
  bool own_tiles;   // the own-tile GEMM
};
LoraForm lora_form(const LoraGemm& lg, int64_t M, int32_t K, int32_t N, bool gelu, int num_sms);

// With lora, the down projection before the GEMM too (small calls: both in one kernel).
ivit_status launch_gemm(const DeviceCtx& dc, const int8_t* X, int64_t M, int32_t K, const int8_t* W, int32_t N,
                        const int32_t* bias, const int32_t* b, const int8_t* c, int32_t out_bits, bool round,
                        EpiMode mode, const int8_t* skip, ivit_residual res, const GeluParams* gelu, int8_t* Y,
                        cudaStream_t stream, const LoraGemm* lora = nullptr);

// Whether the attention kernels take (N, k_s, I0): up to 640 keys; logits
// wider than 8 bits (ShiftExp computed, not looked up) on up to 256 keys and
// with (largest -I_p) * I0 < 2^32.
bool attention_config_supported(int32_t N, int32_t k_s, int32_t I0);

// lis: Log-Int-Softmax instead of Shiftmax (logits of at most 8 bits, M >= 15;
// k_out is then unused)
ivit_status launch_attention(const DeviceCtx& dc, const int8_t* qkv, int32_t B, int32_t N, int32_t H,
                             ivit_dyadic logit, int32_t k_s, int32_t I0, int32_t M, int32_t k_out,
                             ivit_dyadic out, int8_t* ctx, cudaStream_t stream, bool lis = false);

ivit_status launch_shiftgelu(const DeviceCtx& dc, const int8_t* x, int64_t n, const GeluParams& g, int8_t* y,
                             cudaStream_t stream);

// ShiftGELU with the row's largest exponent as I_max, x [rows x cols]
// (cols a multiple of 16).
ivit_status launch_shiftgelu_rowmax(const DeviceCtx& dc, const int8_t* x, int64_t rows, int32_t cols,
                                    const GeluParams& g, int8_t* y, cudaStream_t stream);

// I-LayerNorm of x << alpha (alpha [cols], values 0 .. 3; cols a multiple of
// 16, at most 2048; M_ln <= 20).
ivit_status launch_layernorm_ptf(const DeviceCtx& dc, const int8_t* x, int64_t rows, int32_t cols,
                                 const uint8_t* alpha, const int8_t* gamma, const int32_t* beta, int32_t F,
                                 int32_t M_ln, ivit_dyadic out, int8_t* y, cudaStream_t stream);

// Patch rows z [B*Np x C*P*P] from img [B x C x Hi x Wi] (Hi, Wi multiples of P).
ivit_status launch_im2col(const DeviceCtx& dc, const int8_t* img, int32_t B, int32_t C, int32_t Hi, int32_t Wi,
                          int32_t P, int8_t* z, cudaStream_t stream);

// Tokens x [B*(Np+1) x D] from the class token, the patch embeddings e
// [B*Np x D] and the position embedding pos [(Np+1) x D] (D a multiple of 16).
ivit_status launch_tokens(const DeviceCtx& dc, const int8_t* e, const int8_t* cls, const int8_t* pos,
                          ivit_residual add, int32_t B, int32_t Np, int32_t D, int8_t* x, cudaStream_t stream);

// t [B x D] = the first of each image's Ntok rows of x (D a multiple of 16).
ivit_status launch_gather_rows(const DeviceCtx& dc, const int8_t* x, int32_t B, int32_t Ntok, int32_t D, int8_t* t,
                               cudaStream_t stream);

// A branch's end: y = skip and the branch (post-normed, gated, scaled) added,
// z = the next norm of y (post, gate and pre optional; cols as above).
ivit_status launch_residual_norm(const DeviceCtx& dc, const int8_t* skip, const int8_t* branch, int64_t rows,
                                 int32_t cols, const ivit_norm* post, const int8_t* gate, int64_t gate_rows,
                                 const int32_t* scale, int32_t b_skip, int32_t c, const ivit_norm* pre, int8_t* y,
                                 int8_t* z, cudaStream_t stream);

// Differential attention (H pairs of 64-wide maps; see ivit_attention_diff).
ivit_status launch_attention_diff(const DeviceCtx& dc, const int8_t* qkv, int32_t B, int32_t N, int32_t H,
                                  ivit_dyadic logit, int32_t k_s, int32_t I0, int32_t M, int32_t k_out,
                                  const int32_t* lam, ivit_dyadic out, int8_t* ctx, cudaStream_t stream);

// tables_ready: gamma and beta were written before a kernel that the same library
// call enqueued earlier on the stream.
ivit_status launch_layernorm(const DeviceCtx& dc, const int8_t* x, int64_t rows, int32_t cols,
                             const int8_t* gamma, const int32_t* beta, int32_t F, int32_t M_ln, ivit_dyadic out,
                             bool tables_ready, int8_t* y, cudaStream_t stream);

}  // namespace ivit
