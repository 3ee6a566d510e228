// Dense products with a fused epilogue:
//   out = act(x W^T + bias) + residual
//   out = act(x W_gate^T + bias_gate) * (x W_up^T + bias_up) + residual      (gated)
// "Chapter 30: Mixture of Experts" (LLM Transformer book), 30.2.1 and 30.2.4: the dense FFN
// whose place a sparse layer takes (SwiGLU: the gated form with SiLU, then the plain form).
#include <math.h>

#include "moe_internal.h"

namespace moe {

struct LinearArgs {
  const void* x;
  const void* W[2];        // gate, up (plain: W[0])
  const float* scale[2];   // 8-bit weights: per output row
  const float* bias[2];
  const void* residual;
  void* out;
  int64_t ldx, ldw, ldr, ldo;
  int M, N, K, act;
};

__device__ inline float act_f(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return fmaxf(z, 0.0f);
    case MOE_ACT_GELU: return 0.5f * z * (1.0f + erff(z * 0.70710678118654752f));
    case MOE_ACT_GELU_TANH:
      return z / (1.0f + expf(-1.5957691216057308f * (z + 0.044715f * z * z * z)));
    case MOE_ACT_SILU: return z / (1.0f + expf(-z));
    default: return z;
  }
}

__device__ inline float load_f(const float* p) { return *p; }
__device__ inline float load_f(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ inline float load_f(const uint8_t* p) {
  return __builtin_amdgcn_cvt_f32_fp8((int)*p, 0);
}
__device__ inline void store_f(float* p, float v) { *p = v; }
__device__ inline void store_f(bf16_t* p, float v) { *p = f32_to_bf16(v); }

// 64 x 64 output tile, 16-wide K steps through LDS, 4 x 4 sums per thread.
template <typename XT, typename WT, typename OT, bool GATED>
__global__ __launch_bounds__(256) void linear_tile_kernel(LinearArgs a) {
  constexpr int NW = GATED ? 2 : 1;
  __shared__ float xs[16][65];
  __shared__ float ws[NW][16][65];
  const int tiles_n = (a.N + 63) / 64;
  const int m0 = (int)(blockIdx.x / tiles_n) * 64, n0 = (int)(blockIdx.x % tiles_n) * 64;
  const int tx = threadIdx.x & 15, ty = threadIdx.x >> 4;
  const XT* x = (const XT*)a.x;
  float acc[NW][4][4] = {};
  for (int k0 = 0; k0 < a.K; k0 += 16) {
    for (int i = threadIdx.x; i < 64 * 16; i += 256) {
      const int r = i >> 4, k = k0 + (i & 15);
      xs[i & 15][r] = (m0 + r < a.M && k < a.K) ? load_f(x + (m0 + r) * a.ldx + k) : 0.0f;
#pragma unroll
      for (int q = 0; q < NW; ++q)
        ws[q][i & 15][r] = (n0 + r < a.N && k < a.K)
                               ? load_f((const WT*)a.W[q] + (n0 + r) * a.ldw + k) : 0.0f;
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 16; ++k)
#pragma unroll
      for (int q = 0; q < NW; ++q)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            acc[q][i][j] = fmaf(xs[k][ty + 16 * i], ws[q][k][tx + 16 * j], acc[q][i][j]);
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int m = m0 + ty + 16 * i, n = n0 + tx + 16 * j;
      if (m >= a.M || n >= a.N) continue;
      float z[NW];
#pragma unroll
      for (int q = 0; q < NW; ++q) {
        z[q] = acc[q][i][j];
        if (a.scale[q]) z[q] *= a.scale[q][n];
        if (a.bias[q]) z[q] += a.bias[q][n];
      }
      float v = act_f(z[0], a.act);
      if constexpr (GATED) v *= z[1];
      if (a.residual) v += load_f((const OT*)a.residual + m * a.ldr + n);
      store_f((OT*)a.out + m * a.ldo + n, v);
    }
}

template <typename XT, typename WT, typename OT>
static hipError_t launch_tiles(const LinearArgs& a, bool gated, hipStream_t s) {
  const int64_t grid = ceil_div(a.M, 64) * ceil_div(a.N, 64);
  if (gated)
    hipLaunchKernelGGL((linear_tile_kernel<XT, WT, OT, true>), dim3((unsigned)grid), dim3(256), 0,
                       s, a);
  else
    hipLaunchKernelGGL((linear_tile_kernel<XT, WT, OT, false>), dim3((unsigned)grid), dim3(256),
                       0, s, a);
  return hipGetLastError();
}

template <typename XT, typename WT>
static hipError_t launch_linear_o(const moe_linear_desc_t& d, const LinearArgs& a, bool gated,
                                  hipStream_t s) {
  return d.out_dtype == MOE_DTYPE_F32 ? launch_tiles<XT, WT, float>(a, gated, s)
                                      : launch_tiles<XT, WT, bf16_t>(a, gated, s);
}

static hipError_t launch_linear(const moe_linear_desc_t& d, const LinearArgs& a, bool gated,
                                bool fp8, hipStream_t s) {
  if (fp8) return launch_linear_o<bf16_t, uint8_t>(d, a, gated, s);
  return d.dtype == MOE_DTYPE_F32 ? launch_linear_o<float, float>(d, a, gated, s)
                                  : launch_linear_o<bf16_t, bf16_t>(d, a, gated, s);
}

// ------------------------------------------------------------------ host checks
constexpr int64_t kMaxStride = (int64_t)1 << 31;

static moe_status_t validate_linear(const moe_linear_desc_t* d, bool fp8) {
  if (!d) return MOE_E_NULL;
  if (d->M < 0 || d->N < 1 || d->K < 1) return MOE_E_SHAPE;
  if (d->ldx < 0 || d->ldw < 0 || d->ldr < 0 || d->ldo < 0) return MOE_E_SHAPE;
  if ((d->ldx && d->ldx < d->K) || (d->ldw && d->ldw < d->K) || (d->ldr && d->ldr < d->N) ||
      (d->ldo && d->ldo < d->N))
    return MOE_E_SHAPE;
  if (d->dtype != MOE_DTYPE_F32 && d->dtype != MOE_DTYPE_BF16) return MOE_E_UNSUPPORTED;
  if (d->out_dtype != MOE_DTYPE_F32 && d->out_dtype != MOE_DTYPE_BF16) return MOE_E_UNSUPPORTED;
  if (d->act < MOE_ACT_NONE || d->act > MOE_ACT_SILU) return MOE_E_UNSUPPORTED;
  if (fp8 && d->dtype != MOE_DTYPE_BF16) return MOE_E_UNSUPPORTED;
  if (d->M > (1 << 24) || d->N > (1 << 20) || d->K > (1 << 20) ||
      d->M * d->N > ((int64_t)1 << 40))
    return MOE_E_UNSUPPORTED;
  const int64_t xu = d->dtype == MOE_DTYPE_F32 ? 4 : 8;   // elements per 16 bytes
  const int64_t wu = fp8 ? 16 : xu;
  if (d->K % xu || d->K % wu || d->ldx % xu || d->ldw % wu) return MOE_E_UNSUPPORTED;
  if (d->ldx > kMaxStride || d->ldw > kMaxStride || d->ldr > kMaxStride || d->ldo > kMaxStride)
    return MOE_E_UNSUPPORTED;
  return MOE_OK;
}

static bool aligned_to(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

static moe_status_t linear_impl(const moe_linear_desc_t* desc, const void* x, const void* W0,
                                const void* W1, const float* s0, const float* s1,
                                const float* b0, const float* b1, const void* residual,
                                void* out, void* workspace, size_t workspace_bytes, void* stream,
                                bool gated, bool fp8) {
  moe_status_t st = validate_linear(desc, fp8);
  if (st != MOE_OK) return st;
  const moe_linear_desc_t& d = *desc;
  if (!W0 || (gated && !W1) || (fp8 && (!s0 || (gated && !s1))) || (d.M > 0 && (!x || !out)))
    return MOE_E_NULL;
  const uintptr_t ob = d.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(x, 16) || !aligned_to(W0, 16) || !aligned_to(W1, 16) || !aligned_to(s0, 4) ||
      !aligned_to(s1, 4) || !aligned_to(b0, 4) || !aligned_to(b1, 4) ||
      !aligned_to(residual, ob) || !aligned_to(out, ob))
    return MOE_E_UNSUPPORTED;
  (void)workspace;
  (void)workspace_bytes;
  if (d.M == 0) return MOE_OK;
  const LinearArgs a{x,
                     {W0, W1},
                     {s0, s1},
                     {b0, b1},
                     residual,
                     out,
                     d.ldx ? d.ldx : d.K,
                     d.ldw ? d.ldw : d.K,
                     d.ldr ? d.ldr : d.N,
                     d.ldo ? d.ldo : d.N,
                     (int)d.M,
                     (int)d.N,
                     (int)d.K,
                     d.act};
  return launch_linear(d, a, gated, fp8, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_linear_validate(const moe_linear_desc_t* desc, int fp8) {
  return validate_linear(desc, fp8 != 0);
}

size_t moe_linear_workspace_bytes(const moe_linear_desc_t* desc, int gated, int fp8) {
  (void)desc;
  (void)gated;
  (void)fp8;
  return 0;
}

moe_status_t moe_linear(const moe_linear_desc_t* desc, const void* x, const void* W,
                        const float* bias, const void* residual, void* out, void* workspace,
                        size_t workspace_bytes, void* stream) {
  return linear_impl(desc, x, W, nullptr, nullptr, nullptr, bias, nullptr, residual, out,
                     workspace, workspace_bytes, stream, false, false);
}

moe_status_t moe_linear_gated(const moe_linear_desc_t* desc, const void* x, const void* W_gate,
                              const void* W_up, const float* bias_gate, const float* bias_up,
                              const void* residual, void* out, void* workspace,
                              size_t workspace_bytes, void* stream) {
  return linear_impl(desc, x, W_gate, W_up, nullptr, nullptr, bias_gate, bias_up, residual, out,
                     workspace, workspace_bytes, stream, true, false);
}

moe_status_t moe_linear_fp8(const moe_linear_desc_t* desc, const void* x, const uint8_t* Wq,
                            const float* s, const float* bias, const void* residual, void* out,
                            void* workspace, size_t workspace_bytes, void* stream) {
  return linear_impl(desc, x, Wq, nullptr, s, nullptr, bias, nullptr, residual, out, workspace,
                     workspace_bytes, stream, false, true);
}

moe_status_t moe_linear_gated_fp8(const moe_linear_desc_t* desc, const void* x,
                                  const uint8_t* Wq_gate, const uint8_t* Wq_up,
                                  const float* s_gate, const float* s_up,
                                  const float* bias_gate, const float* bias_up,
                                  const void* residual, void* out, void* workspace,
                                  size_t workspace_bytes, void* stream) {
  return linear_impl(desc, x, Wq_gate, Wq_up, s_gate, s_up, bias_gate, bias_up, residual, out,
                     workspace, workspace_bytes, stream, true, true);
}

}  // extern "C"
