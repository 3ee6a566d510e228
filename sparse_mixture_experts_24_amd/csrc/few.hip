// The whole layer for at most 16 tokens.
//   logits = x W_r^T; p = softmax; top-k of p + b; renormalised weights; capacity; f and P
//   h = SiLU(x W_gate^T) * (x W_up^T);  y = sum_j w_j h_j W_down^T (+ shared) (+ residual)
// "Chapter 30: Mixture of Experts" (LLM Transformer book), 30.2.3, 30.2.4, 30.4.5, 30.6.1;
// "Mixture-of-experts in practice" (deepseekmodel.com), routing-math and capacity sections.
//
// A token chooses an expert at most once, so an expert's rows are a 16-bit set of tokens and
// the stable rank of an assignment is the number of lower tokens in the set.
#include <math.h>

#include "moe_internal.h"
#include "wave.h"

namespace moe {

constexpr int kFew = MOE_FEW_TOKENS;
constexpr int kFewThreads = 512, kFewWaves = kFewThreads / 64;

struct FewArgs {
  const void* x;
  const void* Wr;
  const float* bias;
  ExpertWeights w;
  const void* residual;
  void* out;
  float* f;
  float* p;
  float* logits;   // [T, E]
  float* H;        // [T*k + S*T, F], expert-contiguous rows
  int T, d, E, F, k, S, C;   // C: capacity, -1 none
};

// The routing of the call, held by every workgroup.
struct FewRoute {
  int nu;                              // experts with kept rows (the shared one last)
  int expert[kFew * kMaxTopK + 1];     // ascending
  int row0[kFew * kMaxTopK + 2];       // first H row of each
  uint16_t mask[kFew * kMaxTopK + 1];  // its kept tokens
  float w[kFew][kMaxTopK];             // renormalised weight of slot j
  int16_t row[kFew][kMaxTopK + 1];     // H row of slot j, -1 dropped; [k]: the shared row
};

__device__ inline float wide(const float* p) { return *p; }
__device__ inline float wide(const bf16_t* p) { return bf16_to_f32(*p); }
__device__ inline float wide(const uint8_t* p) { return __builtin_amdgcn_cvt_f32_fp8((int)*p, 0); }
__device__ inline void narrow(float* p, float v) { *p = v; }
__device__ inline void narrow(bf16_t* p, float v) { *p = f32_to_bf16(v); }

// Softmax, top-k, capacity and the touched experts from the logits, by one workgroup.
// Block 0 also writes f and P.  Ends with a barrier.
__device__ inline void few_route(const FewArgs& a, FewRoute& r) {
  __shared__ uint32_t chosen[kMaxExperts];    // token set of each expert
  __shared__ float psum[kFewWaves][kMaxExperts];
  __shared__ int16_t sel[kFew][kMaxTopK];
  constexpr int NV = kMaxExperts / 64;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int nv = (a.E + 63) / 64;
  for (int e = tid; e < kMaxExperts; e += kFewThreads) chosen[e] = 0;
  float ps[NV] = {};
  __syncthreads();
  for (int t = wv; t < a.T; t += kFewWaves) {
    float v[NV], s[NV], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      v[i] = e < a.E ? a.logits[t * a.E + e] : -INFINITY;
      m = fmaxf(m, v[i]);
    }
    m = wave_max(m);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      v[i] = lane + 64 * i < a.E ? expf(v[i] - m) : 0.0f;
      sum += v[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int e = lane + 64 * i;
      v[i] /= sum;   // p
      ps[i] += v[i];
      s[i] = e < a.E ? v[i] + (a.bias ? a.bias[e] : 0.0f) : -INFINITY;
    }
    unsigned taken = 0;
    float tot = 0.0f, mine = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      float bv = -INFINITY;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        if (i < nv && e < a.E && !((taken >> i) & 1u)) take_better(bv, be, s[i], e);
      }
      wave_argmax(bv, be);
      const bool ok = (unsigned)be < (unsigned)a.E;   // false only for non-finite scores
      float pp = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) pp = ok && i == (be >> 6) ? v[i] : pp;
      pp = __shfl(pp, be & 63, 64);
      if (ok && lane == (be & 63)) taken |= 1u << (be >> 6);
      tot += pp;
      mine = lane == j ? pp : mine;
      if (lane == 0) {
        sel[t][j] = ok ? (int16_t)be : (int16_t)-1;
        if (ok) atomicOr(&chosen[be], 1u << t);
      }
    }
    if (lane < a.k) r.w[t][lane] = mine / tot;
  }
#pragma unroll
  for (int i = 0; i < NV; ++i) psum[wv][lane + 64 * i] = ps[i];
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e < a.E; e += kFewThreads) {
      float v = 0.0f;
      for (int q = 0; q < kFewWaves; ++q) v += psum[q][e];
      if (a.f) a.f[e] = (float)((double)__popc(chosen[e]) / (double)(a.T * a.k));
      if (a.p) a.p[e] = v / (float)a.T;
    }
  }
  // The first C tokens of each expert are kept; experts with rows are listed in order, 64
  // experts at a time by wave 0.
  if (wv == 0) {
    int nu = 0, rows = 0;
    for (int i = 0; i < nv; ++i) {
      const int e = lane + 64 * i;
      uint32_t kept = chosen[e];   // zero past E
      int n = __popc(kept);
      while (a.C >= 0 && n > a.C) {
        kept &= ~(1u << (31 - __clz(kept)));
        --n;
      }
      const unsigned long long any = __ballot(n > 0);
      int incl = n;
      for (int o = 1; o < 64; o <<= 1) {
        const int u = __shfl_up(incl, o, 64);
        if (lane >= o) incl += u;
      }
      if (n > 0) {
        const int u = nu + __popcll(any & ((1ull << lane) - 1));
        r.expert[u] = e;
        r.mask[u] = (uint16_t)kept;
        r.row0[u] = rows + incl - n;
      }
      // chosen[e] becomes the expert's first row and kept set, for the slots below
      chosen[e] = kept | ((uint32_t)(rows + incl - n) << 16);
      nu += __popcll(any);
      rows += __shfl(incl, 63, 64);
    }
    if (lane == 0) {
      if (a.S) {
        r.expert[nu] = a.E;
        r.mask[nu] = (uint16_t)((1u << a.T) - 1);
        r.row0[nu++] = rows;
        rows += a.T;
      }
      r.row0[nu] = rows;
      r.nu = nu;
    }
  }
  __syncthreads();
  for (int i = tid; i < a.T * (a.k + 1); i += kFewThreads) {
    const int t = i / (a.k + 1), j = i % (a.k + 1);
    int row = -1;
    if (j < a.k) {
      const int e = sel[t][j];
      if (e >= 0) {
        const uint32_t c = chosen[e];
        if ((c >> t) & 1u) row = (int)(c >> 16) + __popc(c & ((1u << t) - 1));
      }
    } else if (a.S) {
      row = r.row0[r.nu - 1] + t;
    }
    r.row[t][j] = (int16_t)row;
  }
  __syncthreads();
}

template <typename XT>
__global__ __launch_bounds__(256) void few_logits_kernel(FewArgs a) {
  const int lane = threadIdx.x & 63, i = blockIdx.x * 4 + (threadIdx.x >> 6);
  if (i >= a.T * a.E) return;
  const XT* x = (const XT*)a.x + (int64_t)(i / a.E) * a.d;
  const XT* w = (const XT*)a.Wr + (int64_t)(i % a.E) * a.d;
  float s = 0.0f;
  for (int c = lane; c < a.d; c += 64) s = fmaf(wide(x + c), wide(w + c), s);
  s = wave_sum(s);
  if (lane == 0) a.logits[i] = s;
}

template <typename XT, typename WT>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs a) {
  __shared__ FewRoute r;
  few_route(a, r);
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)r.nu * a.F, step = (int64_t)gridDim.x * kFewWaves;
  for (int64_t i = blockIdx.x * kFewWaves + (threadIdx.x >> 6); i < n; i += step) {
    const int u = (int)(i / a.F);
    const int64_t wr = (int64_t)r.expert[u] * a.F + i % a.F;
    const WT* g = (const WT*)a.w.gate + wr * a.d;
    const WT* up = (const WT*)a.w.up + wr * a.d;
    int row = r.row0[u];
    for (uint32_t m = r.mask[u]; m; m &= m - 1, ++row) {
      const XT* x = (const XT*)a.x + (int64_t)(__ffs(m) - 1) * a.d;
      float sg = 0.0f, su = 0.0f;
      for (int c = lane; c < a.d; c += 64) {
        sg = fmaf(wide(x + c), wide(g + c), sg);
        su = fmaf(wide(x + c), wide(up + c), su);
      }
      sg = wave_sum(sg);
      su = wave_sum(su);
      if (a.w.fp8) {
        sg *= a.w.s_gate[wr];
        su *= a.w.s_up[wr];
      }
      if (lane == 0) a.H[(int64_t)row * a.F + i % a.F] = sg / (1.0f + expf(-sg)) * su;
    }
  }
}

template <typename WT, typename OT>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs a) {
  __shared__ FewRoute r;
  FewArgs b = a;
  b.f = b.p = nullptr;
  few_route(b, r);
  const int lane = threadIdx.x & 63;
  const int64_t n = (int64_t)a.T * a.d, step = (int64_t)gridDim.x * kFewWaves;
  for (int64_t i = blockIdx.x * kFewWaves + (threadIdx.x >> 6); i < n; i += step) {
    const int t = (int)(i / a.d), c0 = (int)(i % a.d);
    float y = 0.0f;
    for (int j = 0; j < a.k + a.S; ++j) {
      const int row = r.row[t][j];
      if (row < 0) continue;
      int u = 0;
      while (r.row0[u + 1] <= row) ++u;
      const int64_t wr = (int64_t)r.expert[u] * a.d + c0;
      const WT* w = (const WT*)a.w.down + wr * a.F;
      float s = 0.0f;
      for (int c = lane; c < a.F; c += 64) s = fmaf(a.H[(int64_t)row * a.F + c], wide(w + c), s);
      s = wave_sum(s);
      if (a.w.fp8) s *= a.w.s_down[wr];
      y += j < a.k ? r.w[t][j] * s : s;
    }
    if (lane == 0) {
      if (a.residual) y += wide((const OT*)a.residual + i);
      narrow((OT*)a.out + i, y);
    }
  }
}

// ------------------------------------------------------------------ host
struct FewWorkspace {
  float* logits;
  float* H;
  size_t bytes;
};

static FewWorkspace carve_few(const moe_desc_t& d, void* base) {
  size_t off = 0;
  auto take = [&](int64_t bytes) -> void* {
    void* r = base ? (char*)base + off : nullptr;
    off += (size_t)round_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  FewWorkspace w{};
  w.logits = (float*)take(d.T * d.n_experts * 4);
  w.H = (float*)take((d.T * d.top_k + d.n_shared * d.T) * d.d_ff * 4);
  w.bytes = off;
  return w;
}

static moe_status_t validate_few(const moe_desc_t* d) {
  const moe_status_t st = validate(d);
  if (st != MOE_OK) return st;
  return d->T > kFew ? MOE_E_UNSUPPORTED : MOE_OK;
}

template <typename XT, typename WT, typename OT>
static hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  const int grid = 4 * device_cu_count();
  hipLaunchKernelGGL(few_logits_kernel<XT>, dim3((unsigned)ceil_div(a.T * a.E, 4)), dim3(256), 0,
                     s, a);
  hipLaunchKernelGGL((few_gate_up_kernel<XT, WT>), dim3(grid), dim3(kFewThreads), 0, s, a);
  hipLaunchKernelGGL((few_down_kernel<WT, OT>), dim3(grid), dim3(kFewThreads), 0, s, a);
  return hipGetLastError();
}

static bool aligned_few(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }

static moe_status_t few_impl(const moe_desc_t* desc, const void* x, const void* W_router,
                             const float* bias, const ExpertWeights& ew, const void* residual,
                             void* out, float* f, float* p, void* workspace,
                             size_t workspace_bytes, void* stream) {
  const moe_status_t st = validate_few(desc);
  if (st != MOE_OK) return st;
  const moe_desc_t& d = *desc;
  if (!W_router || !ew.gate || !ew.up || !ew.down || (d.T > 0 && (!x || !out)))
    return MOE_E_NULL;
  if (ew.fp8) {
    if (d.dtype != MOE_DTYPE_BF16) return MOE_E_UNSUPPORTED;
    if (!ew.s_gate || !ew.s_up || !ew.s_down) return MOE_E_NULL;
  }
  const void* wide_ptrs[] = {x, W_router, ew.gate, ew.up, ew.down, residual, out};
  const void* f32_ptrs[] = {bias, ew.s_gate, ew.s_up, ew.s_down, f, p};
  for (const void* q : wide_ptrs)
    if (!aligned_few(q, 16)) return MOE_E_UNSUPPORTED;
  for (const void* q : f32_ptrs)
    if (!aligned_few(q, 4)) return MOE_E_UNSUPPORTED;
  const FewWorkspace w = carve_few(d, workspace);
  if (!workspace || workspace_bytes < w.bytes || !aligned_few(workspace, 256))
    return MOE_E_WORKSPACE;
  hipStream_t s = (hipStream_t)stream;
  if (d.T == 0) {   // no tokens: f and P are zero
    if (f && launch_zero_i32((int32_t*)f, (int)d.n_experts, s) != hipSuccess) return MOE_E_HIP;
    if (p && launch_zero_i32((int32_t*)p, (int)d.n_experts, s) != hipSuccess) return MOE_E_HIP;
    return MOE_OK;
  }
  const FewArgs a{x,
                  W_router,
                  bias,
                  ew,
                  residual,
                  out,
                  f,
                  p,
                  w.logits,
                  w.H,
                  (int)d.T,
                  (int)d.d_model,
                  (int)d.n_experts,
                  (int)d.d_ff,
                  (int)d.top_k,
                  (int)d.n_shared,
                  (int)capacity_of(d)};
  const bool of32 = d.out_dtype == MOE_DTYPE_F32;
  hipError_t e;
  if (ew.fp8)
    e = of32 ? launch_few<bf16_t, uint8_t, float>(a, s) : launch_few<bf16_t, uint8_t, bf16_t>(a, s);
  else if (d.dtype == MOE_DTYPE_F32)
    e = of32 ? launch_few<float, float, float>(a, s) : launch_few<float, float, bf16_t>(a, s);
  else
    e = of32 ? launch_few<bf16_t, bf16_t, float>(a, s) : launch_few<bf16_t, bf16_t, bf16_t>(a, s);
  return e == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_workspace_bytes_few(const moe_desc_t* desc) {
  return validate_few(desc) == MOE_OK ? carve_few(*desc, nullptr).bytes : 0;
}

moe_status_t moe_forward_few(const moe_desc_t* desc, const void* x, const void* W_router,
                             const float* router_bias, const void* W_gate, const void* W_up,
                             const void* W_down, const void* residual, void* out, float* f,
                             float* p, void* workspace, size_t workspace_bytes, void* stream) {
  const ExpertWeights ew{W_gate, W_up, W_down, nullptr, nullptr, nullptr, false};
  return few_impl(desc, x, W_router, router_bias, ew, residual, out, f, p, workspace,
                  workspace_bytes, stream);
}

moe_status_t moe_forward_few_fp8(const moe_desc_t* desc, const void* x, const void* W_router,
                                 const float* router_bias, const uint8_t* Wq_gate,
                                 const uint8_t* Wq_up, const uint8_t* Wq_down,
                                 const float* s_gate, const float* s_up, const float* s_down,
                                 const void* residual, void* out, float* f, float* p,
                                 void* workspace, size_t workspace_bytes, void* stream) {
  const ExpertWeights ew{Wq_gate, Wq_up, Wq_down, s_gate, s_up, s_down, true};
  return few_impl(desc, x, W_router, router_bias, ew, residual, out, f, p, workspace,
                  workspace_bytes, stream);
}

}  // extern "C"
