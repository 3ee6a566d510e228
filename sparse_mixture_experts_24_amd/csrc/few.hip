// The whole layer for at most 16 tokens.
//   logits = x W_r^T; p = softmax; top-k of p + b; renormalised weights; capacity; f and P
//   h = SiLU(x W_gate^T) * (x W_up^T);  y = sum_j w_j h_j W_down^T (+ shared) (+ residual)
// "Chapter 30: Mixture of Experts" (LLM Transformer book), 30.2.3, 30.2.4, 30.4.5, 30.6.1;
// "Mixture-of-experts in practice" (deepseekmodel.com), routing-math and capacity sections.
//
// A token chooses an expert at most once, so an expert's rows are a 16-bit set of tokens and
// the stable rank of an assignment is the number of lower tokens in the set: the routing
// needs no sort, and every workgroup of the first expert kernel forms it for itself.
//
// Launches: the logits (routers of more than 16 experts; smaller ones are computed by every
// workgroup of the next kernel), gate/up with the routing, down in parts of F, the final
// sums.  Bound by the bytes of the touched experts' weights (16 tokens of a d 4096, d_ff 14336,
// 8-expert layer: 2.8 GB in 436 us, 6.4 TB/s; gate/up alone 6.5), for one token of a
// small layer by the launches.  Tried and not kept: everything after the logits in one kernel
// whose workgroups hand their shares on through memory (one token of the Switch-shaped layer 60
// to 76 us against 32, the smallest layer 37 us against 16 on the GPU: a hand-over between 256
// workgroups past the XCDs' L2s costs more than a launch), and the final sums by whichever
// workgroup finishes a group of columns last (down kernel 149 -> 260 us for 16 tokens: the few
// that end last do nearly all of it).
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "moe_internal.h"
#include "stream.h"
#include "wave.h"

namespace moe {

constexpr int kFew = MOE_FEW_TOKENS;
// Experts of a router whose logits every workgroup of the gate/up kernel computes for itself (one
// MFMA block; reading the router again from each L2 costs less than a launch).
constexpr int kOwnLogits = 16;
constexpr int kFewThreads = kStreamThreads, kFewWaves = kStreamWaves;

struct FewRoute;

struct FewArgs {
  const void* x;
  const void* Wr;
  const float* bias;
  ExpertWeights w;
  const void* residual;
  void* out;
  float* f;
  float* p;
  float* logits;     // [ks, T, E] partial sums, or NULL (every workgroup's own)
  FewRoute* route;   // the routing, for the kernels after the first expert kernel
  void* H;           // [T*k + S*T, F] expert-contiguous rows: float, or bf16 values
  bf16_t* Hlo;       //   and (bf16 layers) the bf16 remainders
  float* part;       // [T*k + S*T, chunks, d] partial down products
  int T, d, E, F, k, S, C;   // C: capacity, -1 none
  int ks;            // parts that the logits are summed in
  int chunks;        // parts that the down products' F range is summed in
  bool out_f32;
};

// The routing of the call, held by every workgroup.
struct FewRoute {
  int nu;                              // experts with kept rows (the shared one last)
  int expert[kFew * kMaxTopK + 1];     // ascending
  int row0[kFew * kMaxTopK + 2];       // first H row of each
  uint16_t mask[kFew * kMaxTopK + 1];  // its kept tokens
  float w[kFew][kMaxTopK];             // renormalised weight of slot j
  int16_t row[kFew][kMaxTopK + 2];     // H row of slot j, -1 dropped; [k]: the shared row
};
static_assert(sizeof(FewRoute) % 4 == 0, "copied as int32");

// What the routing needs of LDS while it is formed.
struct RouteLds {
  uint32_t chosen[kMaxExperts];   // token set of each expert
  float psum[kFewWaves][kMaxExperts];
  int16_t sel[kFew][kMaxTopK];
};

// Softmax and top-k of the wave's tokens, at most NV experts per lane.
template <int NV>
__device__ __forceinline__ void route_tokens(const FewArgs& a, FewRoute& r, RouteLds& l,
                                             const float* logits) {
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
  float bias[NV], ps[NV] = {};
#pragma unroll
  for (int i = 0; i < NV; ++i)
    bias[i] = a.bias && lane + 64 * i < a.E ? a.bias[lane + 64 * i] : 0.0f;
  for (int t = wv; t < a.T; t += kFewWaves) {
    float v[NV], s[NV], m = -INFINITY, sum = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) v[i] = 0.0f;
    for (int q = 0; q < a.ks; ++q)   // the logits' partial sums, in order
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (lane + 64 * i < a.E) v[i] += logits[(q * a.T + t) * a.E + lane + 64 * i];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (lane + 64 * i >= a.E) v[i] = -INFINITY;
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
      v[i] /= sum;   // p
      ps[i] += v[i];
      s[i] = lane + 64 * i < a.E ? v[i] + bias[i] : -INFINITY;
    }
    unsigned taken = 0;
    float tot = 0.0f, mine = 0.0f;
    for (int j = 0; j < a.k; ++j) {
      float bv = -INFINITY;
      int be = 0x7fffffff;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int e = lane + 64 * i;
        const bool free = (e < a.E) & !((taken >> i) & 1u);
        take_better(bv, be, free ? s[i] : -INFINITY, free ? e : 0x7fffffff);
      }
      wave_argmax(bv, be);
      const bool ok = (unsigned)be < (unsigned)a.E;   // false only for non-finite scores
      float pp = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) pp = ok && i == (be >> 6) ? v[i] : pp;
      pp = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(pp), be & 63));
      if (ok && lane == (be & 63)) taken |= 1u << (be >> 6);
      tot += pp;
      mine = lane == j ? pp : mine;
      if (lane == 0) {
        l.sel[t][j] = ok ? (int16_t)be : (int16_t)-1;
        if (ok) atomicOr(&l.chosen[be], 1u << t);
      }
    }
    if (lane < a.k) r.w[t][lane] = mine / tot;
  }
  if (blockIdx.x == 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) l.psum[wv][lane + 64 * i] = ps[i];
  }
}

// Softmax, top-k, capacity and the touched experts from the logits, by one workgroup.
// Block 0 also writes f and P.  Ends with a barrier.
__device__ inline void few_route(const FewArgs& a, FewRoute& r, RouteLds& l, const float* logits) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  const int nv = (a.E + 63) / 64;
  uint32_t* chosen = l.chosen;
  for (int e = tid; e < 64 * nv; e += kFewThreads) chosen[e] = 0;
  __syncthreads();
  if (nv == 1)
    route_tokens<1>(a, r, l, logits);
  else if (nv <= 4)
    route_tokens<4>(a, r, l, logits);
  else
    route_tokens<8>(a, r, l, logits);
  __syncthreads();
  if (blockIdx.x == 0) {
    for (int e = tid; e < a.E; e += kFewThreads) {
      float v = 0.0f;
      for (int q = 0; q < kFewWaves; ++q) v += l.psum[q][e];
      if (a.f) a.f[e] = (float)((double)__popc(chosen[e]) / (double)(a.T * a.k));
      if (a.p) a.p[e] = v / (float)a.T;
    }
    __syncthreads();   // wave 0 reuses chosen below
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
      const int e = l.sel[t][j];
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

// Router logits of experts e0 .. e0 + 15 over steps st0 .. st1 - 1 of d, into out[T][ld].  Ends
// with the writes.
struct LogitsLds {
  __align__(16) char stage[kFewWaves][kStageBytes];
  float red[kFewWaves * kRedWave];
};
template <typename XT>
__device__ __forceinline__ void few_logits(const FewArgs& a, LogitsLds& l, int e0, int st0,
                                           int st1, float* out) {
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6, t = lane & 15;
  const XT* x = (const XT*)a.x + (int64_t)min(t, a.T - 1) * a.d;
  const char* row[2];
#pragma unroll
  for (int i = 0; i < 2; ++i)
    row[i] = (const char*)a.Wr +
             (int64_t)min(e0 + 8 * i + (lane >> 3), a.E - 1) * a.d * (int)sizeof(XT);
  floatx4 acc = {0.f, 0.f, 0.f, 0.f};
  stream_rows<XT, 4>(acc, l.stage[wv], st0, st1, [&](int i, int byte) { return row[i] + byte; },
                     [&](int k) { return t < a.T ? x + k : nullptr; });
  red_put(l.red + wv * kRedWave, acc);
  __syncthreads();
  const int m = tid >> 4, n = tid & 15;
  if (m < a.T && e0 + n < a.E) out[m * a.E + e0 + n] = red_get(l.red, kRedWave, m, n);
}

// 16 experts (blockIdx.x) over one part of d (blockIdx.y).
template <typename XT>
__global__ __launch_bounds__(kFewThreads) void few_logits_kernel(FewArgs a) {
  __shared__ LogitsLds l;
  const int nst = a.d / Stream<XT>::SK, y = blockIdx.y;
  few_logits<XT>(a, l, blockIdx.x * 16, nst * y / a.ks, nst * (y + 1) / a.ks,
                 a.logits + y * a.T * a.E);
}

// h = SiLU(x W_gate^T) * (x W_up^T).  A unit is 8 gate rows and the 8 matching up rows of a
// touched expert; all T tokens run through it (the matrix cores have the room), and the
// rows of the tokens that chose the expert are kept.
template <typename WT, int NS, int R, bool ENDS>
__global__ __launch_bounds__(kFewThreads) void few_gate_up_kernel(FewArgs a) {
  typedef Stream<WT> S;
  typedef typename S::X XT;
  __shared__ FewRoute r;
  __shared__ union {
    struct {
      LogitsLds logits;
      float sums[kFew * kOwnLogits];
      RouteLds route;
    };
    StreamLds<R> stream;
  } lds;
  if (a.logits) {
    few_route(a, r, lds.route, a.logits);
  } else {   // a small router: every workgroup computes the logits itself
    few_logits<XT>(a, lds.logits, 0, 0, a.d / Stream<XT>::SK, lds.sums);
    __syncthreads();
    few_route(a, r, lds.route, lds.sums);
  }
  const int tid = threadIdx.x, lane = tid & 63;
  if (blockIdx.x == 0)
    for (int i = tid; i < (int)(sizeof(FewRoute) / 4); i += kFewThreads)
      ((int*)a.route)[i] = ((const int*)&r)[i];
  const int upe = a.F / 8;   // units per expert
  int i0, i1;
  share_of((int64_t)r.nu * upe, blockIdx.x, gridDim.x, i0, i1);
  const int nst = (a.d + S::SK - 1) / S::SK, row_bytes = a.d * (int)sizeof(WT);
  const int nchunk = (nst + NS * kFewWaves - 1) / (NS * kFewWaves);
  stream_units<WT, NS, R, 1, true, ENDS>(
      i0, i1, nchunk, nst, row_bytes, lds.stream,
      [&](int i, UnitRows& rows) {
        const int u = i / upe;
        const int64_t f0 = (int64_t)r.expert[u] * a.F + i % upe * 8;
        rows.base[0] = uniform((const char*)a.w.gate + f0 * row_bytes);
        rows.base[1] = uniform((const char*)a.w.up + f0 * row_bytes);
        rows.off[0] = rows.off[1] = (uint32_t)(lane >> 3) * row_bytes;
        return 0;
      },
      [&](TokenRows& x) {
        x.base = (const char*)a.x;
        x.k = a.d;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x.off[h] = (uint32_t)min(8 * h + (lane >> 3), a.T - 1) * (uint32_t)(a.d * sizeof(XT));
      },
      [&](int i, int m, int n, float v) {
        const int u = i / upe, f = i % upe * 8;
        if constexpr (sizeof(WT) == 1) {
          const int64_t row = (int64_t)r.expert[u] * a.F + f;
          const float sg = pick<8>(a.w.s_gate, row, n & 7), su = pick<8>(a.w.s_up, row, n & 7);
          v *= n < 8 ? sg : su;
        }
        const float up = __shfl_xor(v, 8, 64);
        const uint32_t mask = r.mask[u];
        if (n < 8 && ((mask >> m) & 1u)) {
          const float h = v / (1.0f + expf(-v)) * up;
          const int64_t o = (int64_t)(r.row0[u] + __popc(mask & ((1u << m) - 1))) * a.F + f + n;
          if constexpr (sizeof(XT) == 4) {
            ((float*)a.H)[o] = h;
          } else {
            const bf16_t hi = f32_to_bf16(h);
            ((bf16_t*)a.H)[o] = hi;
            // infinite (or NaN) values have no remainder
            a.Hlo[o] = fabsf(h) < INFINITY && (hi & 0x7F80) != 0x7F80
                           ? f32_to_bf16(h - bf16_to_f32(hi))
                           : (bf16_t)0;
          }
        }
      });
}

// Partial down products: a unit is 16 rows of W_down of an expert over one chunk of F (NS steps
// per wave); the token operand (the expert's rows of h, in bf16 layers value and remainder)
// stays in registers over the units of an (expert, chunk).
template <typename WT, int NS, int R, bool ENDS>
__global__ __launch_bounds__(kFewThreads) void few_down_kernel(FewArgs a) {
  typedef Stream<WT> S;
  typedef typename S::X XT;
  constexpr int NH = sizeof(XT) == 4 ? 1 : 2;   // value, remainder
  __shared__ FewRoute r;
  __shared__ StreamLds<R> lds;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  for (int i = tid; i < (int)(sizeof(FewRoute) / 4); i += kFewThreads)
    ((int*)&r)[i] = ((const int*)a.route)[i];
  __syncthreads();
  const int upc = a.d / 16;   // units per (expert, chunk)
  int i0, i1, have = -1;
  share_of((int64_t)r.nu * a.chunks * upc, blockIdx.x, gridDim.x, i0, i1);
  const int nst = (a.F + S::SK - 1) / S::SK, row_bytes = a.F * (int)sizeof(WT);
  stream_units<WT, NS, R, NH, false, ENDS>(
      i0, i1, 1, nst, row_bytes, lds,
      [&](int i, UnitRows& rows) {
        const int uc = i / upc;
        const int64_t n0 = (int64_t)r.expert[uc / a.chunks] * a.d + i % upc * 16;
        rows.base[0] = uniform((const char*)a.w.down + n0 * row_bytes);
        rows.base[1] = rows.base[0] + 8 * (int64_t)row_bytes;
        rows.off[0] = rows.off[1] = (uint32_t)(lane >> 3) * row_bytes;
        return uc % a.chunks * NS * kFewWaves;
      },
      [&](int i, u32x4 (&xs)[NH][NS][S::XR]) {
        const int uc = i / upc, u = uc / a.chunks, c = uc % a.chunks, t = lane & 15;
        const int start = c * NS * kFewWaves;
        if (uc == have) return start;
        have = uc;
        const uint32_t mask = r.mask[u];
        const bool mine = (mask >> t) & 1u;
        const int64_t o = (int64_t)(r.row0[u] + __popc(mask & ((1u << t) - 1))) * a.F;
#pragma unroll
        for (int s = 0; s < NS; ++s)
#pragma unroll
          for (int q = 0; q < S::XR; ++q) {
            const int k = ((c * NS + s) * kFewWaves + wv) * S::SK + S::k_of(lane >> 4, q);
#pragma unroll
            for (int h = 0; h < NH; ++h) {
              xs[h][s][q] = u32x4{0, 0, 0, 0};
              if (mine && k < a.F)
                xs[h][s][q] = *reinterpret_cast<const u32x4*>(
                    (h == 0 ? (const XT*)a.H : (const XT*)a.Hlo) + o + k);
            }
          }
        landed();
        return start;
      },
      [&](int i, int m, int q, float v) {
        const int uc = i / upc, u = uc / a.chunks, n0 = i % upc * 16;
        const uint32_t mask = r.mask[u];
        if constexpr (sizeof(WT) == 1)
          v *= pick<16>(a.w.s_down, (int64_t)r.expert[u] * a.d + n0, q);
        if (!((mask >> m) & 1u)) return;
        const int64_t row = r.row0[u] + __popc(mask & ((1u << m) - 1));
        a.part[(row * a.chunks + uc % a.chunks) * a.d + n0 + q] = v;
      });
}

// y = sum over the slots of w (sum over chunks), the shared expert, the residual; a thread per
// output, eight partial sums loaded at a time (what bounds it is their latency).
constexpr int kJoinThreads = 256;
__global__ __launch_bounds__(kJoinThreads) void few_join_kernel(FewArgs a) {
  __shared__ FewRoute r;
  for (int i = threadIdx.x; i < (int)(sizeof(FewRoute) / 4); i += kJoinThreads)
    ((int*)&r)[i] = ((const int*)a.route)[i];
  __syncthreads();
  const int64_t i = (int64_t)blockIdx.x * kJoinThreads + threadIdx.x;
  if (i >= (int64_t)a.T * a.d) return;
  const int t = (int)(i / a.d), n = (int)(i % a.d);
  float s = 0.0f, res = 0.0f;
  float y = 0.0f * r.w[t][0];   // NaN where the token's scores were not finite (no experts)
  if (a.residual)
    res = a.out_f32 ? ((const float*)a.residual)[i] : bf16_to_f32(((const bf16_t*)a.residual)[i]);
  for (int j = 0, c = 0; j <= a.k;) {
    float v[8];
    int jj = j, cc = c;
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      const int row = jj <= a.k ? r.row[t][jj] : -1;
      v[q] = row >= 0 ? a.part[((int64_t)row * a.chunks + cc) * a.d + n] : 0.0f;
      if (++cc == a.chunks) {
        cc = 0;
        ++jj;
      }
    }
#pragma unroll
    for (int q = 0; q < 8; ++q) {
      if (j > a.k) break;
      s += v[q];
      if (++c == a.chunks) {
        if (r.row[t][j] >= 0) y += j < a.k ? r.w[t][j] * s : s;
        s = 0.0f;
        c = 0;
        ++j;
      }
    }
  }
  y += res;
  if (a.out_f32)
    ((float*)a.out)[i] = y;
  else
    ((bf16_t*)a.out)[i] = f32_to_bf16(y);
}

// ------------------------------------------------------------------ host
struct FewWorkspace {
  float* logits;
  FewRoute* route;
  void* H;
  bf16_t* Hlo;
  float* part;
  size_t bytes;
};

// Parts of d that the logits are summed in: one or two steps per wave each, as long as a
// workgroup's routing reads at most 1024 partial sums per token.
static int64_t logit_parts(const moe_desc_t& d) {
  if (d.n_experts <= kOwnLogits) return 1;
  const int64_t steps =
      d.d_model / (d.dtype == MOE_DTYPE_F32 ? Stream<float>::SK : Stream<bf16_t>::SK);
  return std::min(ceil_div(steps, 2 * kFewWaves), std::max<int64_t>(1, 1024 / d.n_experts));
}

// Steps per wave of a chunk of the down products, and the chunks of F: 4 steps (8 bits: 2, as
// each takes twice the operand's registers).
template <typename WT>
constexpr int down_steps() {
  return sizeof(WT) == 1 ? 2 : 4;
}
template <typename WT>
static int64_t chunks_of(int64_t F) {
  return ceil_div(F, (int64_t)Stream<WT>::SK * down_steps<WT>() * kFewWaves);
}
static int64_t down_chunks(const moe_desc_t& d, bool fp8) {
  if (fp8) return chunks_of<uint8_t>(d.d_ff);
  return d.dtype == MOE_DTYPE_F32 ? chunks_of<float>(d.d_ff) : chunks_of<bf16_t>(d.d_ff);
}

static FewWorkspace carve_few(const moe_desc_t& d, void* base) {
  size_t off = 0;
  auto take = [&](int64_t bytes) -> void* {
    void* r = base ? (char*)base + off : nullptr;
    off += (size_t)round_up(bytes > 0 ? bytes : 1, 256);
    return r;
  };
  FewWorkspace w{};
  const int64_t rows = d.T * d.top_k + d.n_shared * d.T;
  w.logits = (float*)take(logit_parts(d) * d.T * d.n_experts * 4);
  w.route = (FewRoute*)take(sizeof(FewRoute));
  w.H = take(rows * d.d_ff * (d.dtype == MOE_DTYPE_F32 ? 4 : 2));
  w.Hlo = (bf16_t*)take(d.dtype == MOE_DTYPE_F32 ? 0 : rows * d.d_ff * 2);
  // the 8-bit form has the same or fewer chunks
  w.part = (float*)take(rows * down_chunks(d, false) * d.d_model * 4);
  w.bytes = off;
  return w;
}

static moe_status_t validate_few(const moe_desc_t* d) {
  const moe_status_t st = validate(d);
  if (st != MOE_OK) return st;
  return d->T > kFew ? MOE_E_UNSUPPORTED : MOE_OK;
}

template <typename WT, int NS, int R, bool ENDS>
static void launch_gate_up_few(const FewArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((few_gate_up_kernel<WT, NS, R, ENDS>), dim3(device_cu_count()),
                     dim3(kFewThreads), 0, s, a);
}
template <typename WT, bool ENDS>
static void launch_down_few(const FewArgs& a, hipStream_t s) {
  hipLaunchKernelGGL((few_down_kernel<WT, down_steps<WT>(), 8, ENDS>), dim3(device_cu_count()),
                     dim3(kFewThreads), 0, s, a);
}

template <typename WT>
static hipError_t launch_few(const FewArgs& a, hipStream_t s) {
  typedef typename Stream<WT>::X XT;
  if (a.logits)
    hipLaunchKernelGGL(few_logits_kernel<XT>, dim3((unsigned)ceil_div(a.E, 16), a.ks),
                       dim3(kFewThreads), 0, s, a);
  launch_by_steps<WT>(a.d * (int64_t)sizeof(WT), [&](auto steps, auto ring, auto ends) {
    launch_gate_up_few<WT, steps.value, ring.value, ends.value>(a, s);
  });
  if constexpr (sizeof(WT) == 1) {
    launch_down_few<WT, false>(a, s);
  } else if (row_ends<WT>(a.F * (int64_t)sizeof(WT), down_steps<WT>())) {
    launch_down_few<WT, true>(a, s);
  } else {
    launch_down_few<WT, false>(a, s);
  }
  hipLaunchKernelGGL(few_join_kernel, dim3((unsigned)ceil_div((int64_t)a.T * a.d, kJoinThreads)),
                     dim3(kJoinThreads), 0, s, a);
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
                  d.n_experts > kOwnLogits ? w.logits : nullptr,
                  w.route,
                  w.H,
                  w.Hlo,
                  w.part,
                  (int)d.T,
                  (int)d.d_model,
                  (int)d.n_experts,
                  (int)d.d_ff,
                  (int)d.top_k,
                  (int)d.n_shared,
                  (int)capacity_of(d),
                  (int)logit_parts(d),
                  (int)down_chunks(d, ew.fp8),
                  d.out_dtype == MOE_DTYPE_F32};
  const hipError_t e = ew.fp8                         ? launch_few<uint8_t>(a, s)
                       : d.dtype == MOE_DTYPE_F32 ? launch_few<float>(a, s)
                                                  : launch_few<bf16_t>(a, s);
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
