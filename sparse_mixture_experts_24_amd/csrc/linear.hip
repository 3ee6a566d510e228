// Dense products with a fused epilogue:
//   out = act(x W^T + bias) + residual
//   out = act(x W_gate^T + bias_gate) * (x W_up^T + bias_up) + residual      (gated)
// "Chapter 30: Mixture of Experts" (LLM Transformer book), 30.2.1 and 30.2.4: the dense FFN
// whose place a sparse layer takes (SwiGLU: the gated form with SiLU, then the plain form).
#include <math.h>

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "moe_internal.h"
#include "stream.h"

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
  bool out_f32, wide_rows;
};

// The activations to some 3e-7 of |z| (exponential and reciprocal of the hardware).  GELU: the
// complementary error function of x = |z| / sqrt 2 as t (a1 + .. + a5 t^4) exp(-x^2) with
// t = 1 / (1 + p x) (Abramowitz and Stegun, 7.1.26, within 1.5e-7), a quarter of erff's
// instructions; the tails keep the sign and never cancel.
__device__ __forceinline__ float act_f(float z, int act) {
  switch (act) {
    case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;   // NaN stays
    case MOE_ACT_GELU: {
      const float y = __builtin_amdgcn_fmed3f(z, -16.0f, 16.0f);   // the tail of more is zero
      const float x = fabsf(y) * 0.70710678118654752f;
      const float t = __builtin_amdgcn_rcpf(fmaf(0.3275911f, x, 1.0f));
      float p = fmaf(1.061405429f, t, -1.453152027f);
      p = fmaf(p, t, 1.421413741f);
      p = fmaf(p, t, -0.284496736f);
      p = fmaf(p, t, 0.254829592f);
      const float tail = 0.5f * y * (p * t) * __expf(-x * x);   // z/2 erfc(x)
      return z < 0.0f ? tail : z - tail;                        // NaN stays
    }
    case MOE_ACT_GELU_TANH:
      return z * __builtin_amdgcn_rcpf(
                     1.0f + __expf(-1.5957691216057308f * fmaf(0.044715f * z * z, z, z)));
    case MOE_ACT_SILU: return z * __builtin_amdgcn_rcpf(1.0f + __expf(-z));
    default: return z;
  }
}

__device__ __forceinline__ void act8(float* z, int act) {
  switch (act) {
#define MOE_ACT8(A)                                           \
  case A:                                                     \
    _Pragma("unroll") for (int i = 0; i < 8; ++i) z[i] = act_f(z[i], A); \
    break;
    MOE_ACT8(MOE_ACT_RELU)
    MOE_ACT8(MOE_ACT_GELU)
    MOE_ACT8(MOE_ACT_GELU_TANH)
    MOE_ACT8(MOE_ACT_SILU)
#undef MOE_ACT8
    default: break;
  }
}

// p[n0 + q], 0 <= q < C, the last of n where that is past it.
template <int C>
__device__ __forceinline__ float column(const float* p, int n0, int n, int q) {
  float v = scalar_f(p, n0);
#pragma unroll
  for (int j = 1; j < C; ++j) v = q == j ? scalar_f(p, min(n0 + j, n - 1)) : v;
  return v;
}
__device__ inline float load_out(const LinearArgs& a, const void* base, int64_t i) {
  return a.out_f32 ? ((const float*)base)[i] : bf16_to_f32(((const bf16_t*)base)[i]);
}
__device__ inline void store_out(const LinearArgs& a, int64_t i, float v) {
  if (a.out_f32)
    ((float*)a.out)[i] = v;
  else
    ((bf16_t*)a.out)[i] = f32_to_bf16(v);
}

// What a lane needs of its 8 neighbouring columns n .. n + 7 (those past N: column N - 1).
struct Columns {
  float scale[8], bias[8];
  __device__ __forceinline__ void load(const LinearArgs& a, int mat, int n) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int c = min(n + i, a.N - 1);
      scale[i] = a.scale[mat] ? a.scale[mat][c] : 1.0f;
      bias[i] = a.bias[mat] ? a.bias[mat][c] : 0.0f;
    }
  }
};
// The residual's 8 values at element i, as they are stored (wide rows only).
struct Residual8 {
  u32x4 lo, hi;
  __device__ __forceinline__ void load(const LinearArgs& a, int64_t i) {
    if (a.out_f32) {
      lo = *reinterpret_cast<const u32x4*>((const float*)a.residual + i);
      hi = *reinterpret_cast<const u32x4*>((const float*)a.residual + i + 4);
    } else {
      lo = *reinterpret_cast<const u32x4*>((const bf16_t*)a.residual + i);
    }
  }
  __device__ __forceinline__ float get(const LinearArgs& a, int i) const {
    if (a.out_f32) return __uint_as_float(i < 4 ? lo[i & 3] : hi[i & 3]);
    return __uint_as_float(i & 1 ? lo[i >> 1] & 0xFFFF0000u : lo[i >> 1] << 16);
  }
};
// Stores 8 neighbouring values (wide rows).
__device__ __forceinline__ void store8(const LinearArgs& a, int64_t i, const float* v) {
  if (a.out_f32) {
    float* out = (float*)a.out + i;
    *reinterpret_cast<float4*>(out) = make_float4(v[0], v[1], v[2], v[3]);
    *reinterpret_cast<float4*>(out + 4) = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    u32x4 r;
#pragma unroll
    for (int q = 0; q < 4; ++q)
      r[q] = (uint32_t)f32_to_bf16(v[2 * q]) | (uint32_t)f32_to_bf16(v[2 * q + 1]) << 16;
    *reinterpret_cast<u32x4*>((bf16_t*)a.out + i) = r;
  }
}

// ------------------------------------------------------------------ blocks of 16 rows
// Bound by the weights' bytes, or for small ones by a launch and two trips to memory: one row
// of 2048 x 2048 3.9 us, 16 rows against 2 x 14336 x 4096 of 8 bits 24 us a call (4.8 TB/s).  A
// unit is 16 weight rows (gated: 8 gate rows and the 8 matching up rows); the workgroups of
// a row block take runs of units.
template <typename WT, int NS, int R, bool ENDS, bool GATED>
__global__ __launch_bounds__(kStreamThreads) void linear_rows_kernel(LinearArgs a) {
  typedef Stream<WT> S;
  typedef typename S::X XT;
  __shared__ StreamLds<R> lds;
  constexpr int COLS = GATED ? 8 : 16;   // output columns of a unit
  const int lane = threadIdx.x & 63;
  // The block's rows.  Neighbouring workgroups are of one block: the blocks' workgroups of the
  // same weight rows are then often on one XCD, whose L2 they share (float32 24 x 4096 x 4096
  // 19 us, 25 in the other order).
  const int m0 = blockIdx.y * 16;
  a.x = (const XT*)a.x + m0 * a.ldx;
  a.M = min(a.M - m0, 16);
  int i0, i1;
  share_of((a.N + COLS - 1) / COLS, blockIdx.x, gridDim.x, i0, i1);
  const int nst = (a.K + S::SK - 1) / S::SK;
  const int nchunk = (nst + NS * kStreamWaves - 1) / (NS * kStreamWaves);
  const uint32_t wrow = (uint32_t)(a.ldw * (int)sizeof(WT));
  stream_units<WT, NS, R, 1, true, ENDS>(
      i0, i1, nchunk, nst, a.K * (int)sizeof(WT), lds,
      [&](int i, UnitRows& rows) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int n0 = i * COLS, r = (GATED ? 0 : 8 * h) + (lane >> 3);
          rows.base[h] = uniform((const char*)a.W[GATED ? h : 0] + n0 * (int64_t)wrow);
          rows.off[h] = (uint32_t)min(r, a.N - 1 - n0) * wrow;
        }
        return 0;
      },
      [&](TokenRows& x) {
        x.base = (const char*)a.x;
        x.k = a.K;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x.off[h] = (uint32_t)min(8 * h + (lane >> 3), a.M - 1) *
                     (uint32_t)(a.ldx * (int)sizeof(XT));
      },
      [&](int i, int m, int q, float v) {
        const int n0 = i * COLS, n = n0 + (GATED ? q & 7 : q);
        // scale and bias by scalar loads, columns past N reading column N - 1
        float z[GATED ? 2 : 1];
#pragma unroll
        for (int t = 0; t < (GATED ? 2 : 1); ++t) {
          z[t] = v;
          if (a.scale[t]) z[t] *= column<COLS>(a.scale[t], n0, a.N, q & (COLS - 1));
          if (a.bias[t]) z[t] += column<COLS>(a.bias[t], n0, a.N, q & (COLS - 1));
        }
        if constexpr (GATED) {
          const float up = __shfl_xor(z[1], 8, 64);
          v = act_f(z[0], a.act) * up;
          if (q >= 8) return;
        } else {
          v = act_f(z[0], a.act);
        }
        if (m >= a.M || n >= a.N) return;
        if (a.residual) v += load_out(a, a.residual, (m0 + m) * a.ldr + n);
        store_out(a, (m0 + m) * a.ldo + n, v);
      });
}

// ------------------------------------------------------------------ MFMA tiles
// A tile per workgroup of WM x WN waves, a wave holding MB x NB blocks of 32 x 32 sums (each
// four MFMAs of 16 x 16: the 32 x 32 MFMA moves twice the sums through the registers per
// product, and large products run at the clock that the card's power allows: 1.44 GHz and
// 82% of it in MFMAs with the one, 1.62 GHz and 75% with the other).  K runs in steps of
// 128 bytes of an x row through ST LDS stages that global loads fill directly (no registers
// between).  A step is two slices of one k range per MFMA block; the
// operands of slice s + 1 are read from LDS while the MFMAs of slice s run.  The barrier that
// frees a stage stands before the last slice's MFMAs, whose operands are in registers by
// then, so the next stage's first reads and the loads ST steps ahead run under them.
//   Two stages whose x and weight parts are alike are five slots of one part, taken in the
// order x, w, x, w, ...: the fifth lets the x part of step t + 2 load during step t, so only
// its weight part waits for the barrier, and the loads spread over the whole step.
//   LDS rows are 128 bytes (8-bit weights: 64), the 16-byte chunk c of row r at position
// c ^ (r / 2 % 8) (8-bit: c ^ (r / 4 % 4)), applied to the addresses that the lanes load
// from: a direct load puts lane l's 16 bytes at 16 l.  The operand reads of 16 neighbouring
// rows then cover 256 bytes, all 64 banks.
//   Small products have less than a tile for every CU: there WK groups of waves with stages of
// their own take every WK-th step and their sums are added through LDS.
//   Gated: the weight blocks of a wave alternate gate and up rows of the same columns, so the
// two sums of an output meet in the epilogue's buffer.
//   Bound: MFMAs at the power limit for large products (gated 4096 x 14336 x 4096: 694 us, 1390
// TFLOP/s; the library's plain product of the same size 630-710 us; 2048 x 4096 x 14336 with
// the residual 216 us, 1110 TFLOP/s), the loads of a CU for small ones (64 x 7168 x 2048:
// 8.1 us with its inputs in the caches, 64 x 14336 x 4096 21 us against the library's 24).

// Barrier that LDS accesses do not cross.
__device__ __forceinline__ void stage_barrier() {
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// One MFMA block's product of a slice: 64 bytes of the x rows.  Lane (row, group g) holds the
// 16-byte chunk g of its x row's slice, and the weights of the same k.
template <typename WT>
struct Tile {   // bf16
  // k per step, bytes of a weight row in it, MFMAs of a block and slice
  static constexpr int BK = 64, WROW = 128, SUB = 1;
  typedef bf16_t X;
  typedef u32x4 WReg;
  __device__ static void mma(floatx4& acc, u32x4 x, u32x4 w, int) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x),
                                                  __builtin_bit_cast(bf16x8, w), acc, 0, 0, 0);
  }
  __device__ static u32x4 operand(u32x4 w) { return w; }
};
template <>
struct Tile<uint8_t> {
  static constexpr int BK = 64, WROW = 64, SUB = 1;
  typedef bf16_t X;
  typedef uint2 WReg;
  __device__ static void mma(floatx4& acc, u32x4 x, u32x4 w, int) {
    Tile<bf16_t>::mma(acc, x, w, 0);
  }
  __device__ static u32x4 operand(uint2 w) {
    return __builtin_bit_cast(u32x4, widen_e4m3(w.x, w.y));
  }
};
template <>
struct Tile<float> {
  static constexpr int BK = 32, WROW = 128, SUB = 4;
  typedef float X;
  typedef u32x4 WReg;
  __device__ static void mma(floatx4& acc, u32x4 x, u32x4 w, int j) {   // group g: k = 4 g + j
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[j]), __uint_as_float(w[j]), acc,
                                               0, 0, 0);
  }
  __device__ static u32x4 operand(u32x4 w) { return w; }
};

constexpr int kXRow = 128;   // bytes of an x row in a stage

// Rows of x, weight rows and outputs of a tile.
template <int MB, int WM>
constexpr int tile_m() { return 32 * MB * WM; }
template <int NB, int WN>
constexpr int tile_w() { return 32 * NB * WN; }
template <int NB, int WN, bool GATED>
constexpr int tile_n() { return tile_w<NB, WN>() / (GATED ? 2 : 1); }
template <typename WT, int MB, int NB, int WM, int WN>
constexpr int tile_stage_bytes() {
  return tile_m<MB, WM>() * kXRow + tile_w<NB, WN>() * Tile<WT>::WROW;
}
// The epilogue's transpose buffer: 32 rows of a wave's sums, padded by 4 floats.
template <int NB>
constexpr int tile_epilogue_ld() {
  return 32 * NB + 4;
}
// Two stages of equal x and weight parts share five slots of one part instead.
template <typename WT, int MB, int NB, int WM, int WN, int ST>
constexpr bool tile_slots() {
  return ST == 2 && 2 * tile_m<MB, WM>() * kXRow == tile_stage_bytes<WT, MB, NB, WM, WN>();
}
template <typename WT, int MB, int NB, int WM, int WN, int ST>
constexpr int tile_group_bytes() {
  const int stage = tile_stage_bytes<WT, MB, NB, WM, WN>();
  return tile_slots<WT, MB, NB, WM, WN, ST>() ? 5 * stage / 2 : ST * stage;
}
template <typename WT, int MB, int NB, int WM, int WN, int WK, int ST>
constexpr int tile_lds_bytes() {
  const int stages = WK * tile_group_bytes<WT, MB, NB, WM, WN, ST>();
  const int sums = (WK - 1) * tile_m<MB, WM>() * tile_w<NB, WN>() * 4;
  const int epi = sums + WM * WN * 32 * tile_epilogue_ld<NB>() * 4;
  return stages > epi ? stages : epi;
}

// Tile of a workgroup.  Workgroup i runs on XCD i % 8; every XCD takes a run of consecutive
// tiles, ordered in groups of 8 row tiles so that the tiles an XCD works on at a time share
// x rows and weight rows in its L2.
__device__ inline void tile_of(const LinearArgs& a, int tiles_m, int tiles_n, int& tm, int& tn) {
  const int total = tiles_m * tiles_n, xcd = blockIdx.x & 7, q = total >> 3, rest = total & 7;
  const int pos = xcd * q + min(xcd, rest) + (int)(blockIdx.x >> 3);
  const int per = 8 * tiles_n, grp = pos / per, rows = min(8, tiles_m - 8 * grp);
  tm = 8 * grp + pos % per % rows;
  tn = pos % per / rows;
}

template <typename WT, int MB, int NB, int WM, int WN, int WK, int ST, bool GATED>
__global__ __launch_bounds__(64 * WM * WN * WK) void linear_tile_kernel(LinearArgs a) {
  typedef Tile<WT> TT;
  typedef typename TT::X XT;
  static_assert(!GATED || NB % 2 == 0, "gate and up blocks come in pairs");
  constexpr int BM = tile_m<MB, WM>(), OUT_N = tile_n<NB, WN, GATED>();
  constexpr int STAGE = tile_stage_bytes<WT, MB, NB, WM, WN>(), XBYTES = BM * kXRow;
  constexpr bool W8 = sizeof(WT) == 1, SLOTS = tile_slots<WT, MB, NB, WM, WN, ST>();
  constexpr int WRPL = W8 ? 16 : 8;   // weight rows per load
  // loads per wave and step
  constexpr int NX = BM / 8 / (WM * WN), NW = tile_w<NB, WN>() / WRPL / (WM * WN);
  static_assert(NX % 2 == 0 && (NW % 2 == 0 || (W8 && NW * WRPL <= 32)), "loads per wave");
  static_assert(!GATED || NW * WRPL <= 64, "half of a wave's weight rows are of one matrix");
  extern __shared__ __align__(16) char smem[];
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wk = wave / (WM * WN);
  const int w = wave % (WM * WN), wm = w / WN, wn = w % WN;
  constexpr int GROUP = tile_group_bytes<WT, MB, NB, WM, WN, ST>();
  const int lds0 = wk * GROUP;   // the group's stages
  int tm, tn;
  tile_of(a, (a.M + BM - 1) / BM, (a.N + OUT_N - 1) / OUT_N, tm, tn);
  const int m0 = tm * BM, n0 = tn * OUT_N;

  // What this lane loads: rows of the tile (clamped into the matrices) at its chunk, as 32-bit
  // offsets from the tile's first rows (the host keeps tiles within 4 GB of them).  Load i of
  // x takes 8 rows, chunk lane % 8 ^ row / 2 % 8, whose third bit is the parity of i.
  const uint32_t xrow = (uint32_t)(a.ldx * (int)sizeof(XT));
  const uint32_t wrow = (uint32_t)(a.ldw * (int)sizeof(WT));
  const int xchunk = (lane & 7) ^ (lane >> 4);
  const int wchunk = W8 ? (lane & 3) ^ ((lane >> 4) & 3) : xchunk;
  uint32_t ox[NX], ow[NW];
#pragma unroll
  for (int i = 0; i < NX; ++i) {
    const int m = min(m0 + (w * NX + i) * 8 + (lane >> 3), a.M - 1) - m0;
    ox[i] = (uint32_t)m * xrow + 16 * (xchunk ^ (4 * (i & 1)));
  }
#pragma unroll
  for (int i = 0; i < NW; ++i) {
    const int j = (w * NW + i) * WRPL + (W8 ? lane >> 2 : lane >> 3);
    const int col = GATED ? (j / (32 * NB)) * (16 * NB) + ((j / 32) % NB >> 1) * 32 + (j & 31) : j;
    ow[i] = (uint32_t)(min(n0 + col, a.N - 1) - n0) * wrow + 16 * (wchunk ^ (W8 ? 0 : 4 * (i & 1)));
  }
  const char* bx = (const char*)a.x + (int64_t)m0 * xrow + wk * kXRow;
  const char* bw[2];   // of each half of the wave's weight rows
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int mat = GATED ? ((w * NW + h * (NW / 2)) * WRPL >> 5) & 1 : 0;
    bw[h] = (const char*)(mat ? a.W[1] : a.W[0]) + (int64_t)n0 * wrow + wk * TT::WROW;
  }
  // Step t of the group is step WK t + wk of K; steps are full below nfull in every group, and
  // every group takes nk steps (past K: zeros).
  const int nk = (a.K + WK * TT::BK - 1) / (WK * TT::BK), nfull = a.K / (WK * TT::BK);
  // Load i (x part, then weight part) of step t into the part at LDS byte `part`; a last step
  // that K does not fill (tail) has zeros past K.
  auto load = [&](auto tail, int i, int t, int part) {
    const bool isx = i < NX;
    const int q = isx ? i : i - NX;
    const uint32_t dst = (uint32_t)(lds0 + part + (w * (isx ? NX : NW) + q) * 1024);
    const char* base = isx ? bx : bw[q >= NW / 2 && NW > 1 ? 1 : 0];
    const uint32_t off = isx ? ox[isx ? q : 0] : ow[isx ? 0 : q];
    if constexpr (decltype(tail)::value) {
      const int chunk = isx ? xchunk ^ (4 * (q & 1)) : wchunk ^ (W8 ? 0 : 4 * (q & 1));
      const int k = (t * WK + wk) * TT::BK + chunk * (16 / (int)(isx ? sizeof(XT) : sizeof(WT)));
      if (k < a.K)
        load_to_lds(base, off, dst);
      else
        *reinterpret_cast<u32x4*>(smem + dst + 16 * lane) = u32x4{0, 0, 0, 0};
    } else {
      load_to_lds(base, off, dst);
    }
    if (i == NX - 1) bx += WK * kXRow;
    if (i == NX + NW - 1) {
      bw[0] += WK * TT::WROW;
      bw[1] += WK * TT::WROW;
    }
  };
  auto load_part = [&](int from, int to, int t, int part) {
    if (t < nfull) {
#pragma unroll
      for (int i = 0; i < NX + NW; ++i)
        if (i >= from && i < to) load(std::false_type{}, i, t, part);
    } else if (t < nk) {
#pragma unroll
      for (int i = 0; i < NX + NW; ++i)
        if (i >= from && i < to) load(std::true_type{}, i, t, part);
    }
  };

  // Operand reads: row lane % 16 of a 16-row block, chunk lane / 16 of the slice.
  constexpr int XB = 2 * MB, WB = 2 * NB;
  const int fr = lane & 15, fg = lane >> 4;
  const int xrd = lds0 + (wm * 32 * MB + fr) * kXRow, xsw = 16 * (fg ^ ((fr >> 1) & 7));
  const int wrd = lds0 + (wn * 32 * NB + fr) * TT::WROW;
  const int wsw = W8 ? 16 * ((fg >> 1) ^ ((fr >> 2) & 3)) : xsw;
  u32x4 xf[2][XB];
  typename TT::WReg wf[2][WB];
  auto read_x = [&](int buf, int i, int part, int s) {
    xf[buf][i] = *reinterpret_cast<const u32x4*>(smem + part + xrd + i * 16 * kXRow +
                                                 (xsw ^ (64 * s)));
  };
  auto read_w = [&](int buf, int i, int part, int s) {
    wf[buf][i] = *reinterpret_cast<const typename TT::WReg*>(
        smem + part + wrd + i * 16 * TT::WROW +
        (W8 ? (wsw ^ (32 * s)) + 8 * (fg & 1) : wsw ^ (64 * s)));
  };
  floatx4 acc[XB][WB];
#pragma unroll
  for (int i = 0; i < XB; ++i)
#pragma unroll
    for (int j = 0; j < WB; ++j) acc[i][j] = floatx4{0.f, 0.f, 0.f, 0.f};

  constexpr int L = NX + NW;
#pragma unroll
  for (int t = 0; t < ST; ++t) {
    load_part(0, NX, t, t * STAGE);
    load_part(NX, L, t, t * STAGE + XBYTES);
  }
  if (ST <= nfull)
    wait_loads<(ST - 1) * L>();
  else
    wait_loads();
  stage_barrier();
#pragma unroll
  for (int i = 0; i < XB; ++i) read_x(0, i, 0, 0);
#pragma unroll
  for (int i = 0; i < WB; ++i) read_w(0, i, XBYTES, 0);
  // Step t.  Body: step t + ST is a full one, whose loads go out between MFMAs, as early as
  // their part is free.  px, pw: where step t's parts are.
  int px = 0, pw = XBYTES;
  auto part_after = [&](int part, int by) {   // the part `by` slots on
    const int p = part + by * XBYTES;
    return p >= 5 * XBYTES ? p - 5 * XBYTES : p;
  };
  auto step = [&](auto body, int t) {
    int nx, nw;
    if constexpr (SLOTS) {
      nx = part_after(px, 2);
      nw = part_after(pw, 2);
    } else {
      nx = px == (ST - 1) * STAGE ? 0 : px + STAGE;
      nw = nx + XBYTES;
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int buf = s, sx = s == 0 ? px : nx, sw = s == 0 ? pw : nw, sn = s ^ 1;
      if (SLOTS && s == 0 && !decltype(body)::value) load_part(0, NX, t + 2, part_after(nx, 2));
      if (s == 1) {
        // step t's parts are read out by every wave, step t + 1 has landed
        if constexpr (decltype(body)::value)
          wait_loads<SLOTS ? NX : (ST - 2) * L>();
        else
          wait_loads();
        stage_barrier();
        if constexpr (!decltype(body)::value) {
          if (!SLOTS) load_part(0, NX, t + ST, px);
          load_part(NX, L, t + ST, SLOTS ? px : pw);
        }
      }
      u32x4 wo[WB];
#pragma unroll
      for (int i = 0; i < WB; ++i) wo[i] = TT::operand(wf[buf][i]);
      // Operand reads of the next slice (past the last step: stale, unused) go out one by one
      // between the MFMAs, in whose shadow they issue; so do the loads, of slots in the first
      // half of their slice (LF = 2: gated 4096-row product 760 -> 727 us; whole stages have
      // time to land and prefer an even spread, 213 against 216 us for 2048 x 4096 x 14336).
      // A block's SUB MFMAs are a round of all blocks apart: each needs the one before.
      constexpr int SUB = TT::SUB, B = XB * WB * SUB, RD = XB + WB, EVERY = B >= 2 * RD ? 2 : 1,
                    LF = SLOTS ? 2 : 1;
      static_assert(RD <= B, "a read per MFMA at most");
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < XB; ++i)
#pragma unroll
          for (int j = 0; j < WB; ++j) {
            const int q = (u * XB + i) * WB + j, rd = q / EVERY;
            TT::mma(acc[i][j], xf[buf][i], wo[j], u);
            if (q % EVERY == 0 && rd < RD) {
              if (rd < WB)
                read_w(buf ^ 1, rd < WB ? rd : 0, sw, sn);
              else
                read_x(buf ^ 1, rd >= WB ? rd - WB : 0, sx, sn);
            }
            if constexpr (decltype(body)::value) {
              if constexpr (SLOTS) {
                if (s == 0) {   // x part of step t + 2
#pragma unroll
                  for (int l = q * LF * NX / B; l < min((q + 1) * LF * NX / B, NX); ++l)
                    load(std::false_type{}, l, t + 2, part_after(nx, 2));
                } else {
#pragma unroll
                  for (int l = q * LF * NW / B; l < min((q + 1) * LF * NW / B, NW); ++l)
                    load(std::false_type{}, NX + l, t + 2, px);
                }
              } else if (s == 1) {
#pragma unroll
                for (int l = q * LF * L / B; l < min((q + 1) * LF * L / B, L); ++l)
                  load(std::false_type{}, l, t + ST, l < NX ? px : pw);
              }
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      __builtin_amdgcn_sched_barrier(0);
    }
    px = nx;
    pw = nw;
  };
  int t = 0;
  for (; t + ST < nfull; ++t) step(std::true_type{}, t);
  for (; t < nk; ++t) step(std::false_type{}, t);
  wait_loads();
  stage_barrier();   // the stages are free for what follows
  if constexpr (WK > 1) {
    // the groups' sums, added in order by the first group
    float* sums = (float*)smem + ((wk - 1) * WM * WN + w) * (64 * 4 * XB * WB) + lane * 4;
    if (wk > 0) {
#pragma unroll
      for (int i = 0; i < XB * WB; ++i)
        *reinterpret_cast<floatx4*>(sums + i * 256) = acc[i / WB][i % WB];
    }
    __syncthreads();
    if (wk > 0) return;
#pragma unroll
    for (int q = 1; q < WK; ++q) {
      sums = (float*)smem + ((q - 1) * WM * WN + w) * (64 * 4 * XB * WB) + lane * 4;
#pragma unroll
      for (int i = 0; i < XB * WB; ++i)
        acc[i / WB][i % WB] += *reinterpret_cast<const floatx4*>(sums + i * 256);
    }
  }

  // Epilogue, a wave by itself: the sums of 32 rows at a time through LDS, so that a lane
  // finishes 8 neighbouring columns of a row and rows leave in whole segments.  The lane's
  // columns are the same in every row; the sums and residual of its next row are read
  // while one is finished.  One copy of the code for all MB blocks (only the LDS writes
  // name the accumulators), as it holds every activation.
  constexpr int LD = tile_epilogue_ld<NB>(), WC = 32 * NB / (GATED ? 2 : 1), PER = WC / 8;
  constexpr int STEP = 64 / PER;   // rows a wave finishes at a time
  float* tr = (float*)smem + (WK - 1) * WM * WN * 64 * 4 * XB * WB + w * 32 * LD;
  const int c = lane % PER * 8, n = n0 + wn * WC + c, row0 = lane / PER;
  const float* z = tr + (GATED ? 64 * (c >> 5) + (c & 31) : c);   // gated: up sums 32 further
  Columns cg, cu;
  cg.load(a, 0, n);
  if constexpr (GATED) cu.load(a, 1, n);
  const bool wide = a.wide_rows && n + 8 <= a.N;
#pragma unroll 1
  for (int i = 0; i < MB; ++i) {
#pragma unroll
    for (int q = 0; q < MB; ++q)
      if (q == i) {
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int j = 0; j < WB; ++j)
#pragma unroll
            for (int r = 0; r < 4; ++r)
              tr[(16 * h + 4 * fg + r) * LD + 16 * j + fr] = acc[2 * q + h][j][r];
      }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    const int mw = m0 + (wm * MB + i) * 32 + row0;
    float zg[8], zu[8];
    Residual8 res;
    auto fetch = [&](int row) {   // row of the 32, from row0
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        zg[e] = z[(row0 + row) * LD + e];
        if constexpr (GATED) zu[e] = z[(row0 + row) * LD + 32 + e];
      }
      if (a.residual && wide && mw + row < a.M) res.load(a, (mw + row) * a.ldr + n);
    };
    fetch(0);
#pragma unroll 1
    for (int row = 0; row < 32; row += STEP) {
      float v[8], u[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = fmaf(zg[e], cg.scale[e], cg.bias[e]);
        if constexpr (GATED) u[e] = fmaf(zu[e], cu.scale[e], cu.bias[e]);
      }
      const Residual8 r = res;
      if (row + STEP < 32) fetch(row + STEP);
      act8(v, a.act);
      const int m = mw + row;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if constexpr (GATED) v[e] *= u[e];
        if (a.residual && wide) v[e] += r.get(a, e);
      }
      if (m >= a.M || n >= a.N) continue;
      if (wide) {
        store8(a, m * a.ldo + n, v);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (n + e < a.N)
            store_out(a, m * a.ldo + n + e,
                      a.residual ? v[e] + load_out(a, a.residual, m * a.ldr + n + e) : v[e]);
      }
    }
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  }
}

// The LDS of a tile kernel is above the default limit: raised once per device and kernel.
template <typename WT, int MB, int NB, int WM, int WN, int WK, int ST, bool GATED>
static hipError_t run_tiles(const LinearArgs& a, hipStream_t s) {
  static std::atomic<bool> done[kMaxDevices];
  constexpr int lds = tile_lds_bytes<WT, MB, NB, WM, WN, WK, ST>();
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  if (dev < 0 || dev >= kMaxDevices || !done[dev].load(std::memory_order_acquire)) {
    e = hipFuncSetAttribute((const void*)linear_tile_kernel<WT, MB, NB, WM, WN, WK, ST, GATED>,
                            hipFuncAttributeMaxDynamicSharedMemorySize, lds);
    if (e != hipSuccess) return e;
    if (dev >= 0 && dev < kMaxDevices) done[dev].store(true, std::memory_order_release);
  }
  const int64_t tiles = ceil_div(a.M, tile_m<MB, WM>()) * ceil_div(a.N, tile_n<NB, WN, GATED>());
  hipLaunchKernelGGL((linear_tile_kernel<WT, MB, NB, WM, WN, WK, ST, GATED>), dim3((unsigned)tiles),
                     dim3(64 * WM * WN * WK), lds, s, a);
  return hipGetLastError();
}

template <typename WT, int NS, int R, bool ENDS, bool GATED>
static hipError_t run_rows(const LinearArgs& a, hipStream_t s) {
  const int64_t units = ceil_div(a.N, GATED ? 8 : 16), blocks = ceil_div(a.M, 16);
  const int64_t per = std::max<int64_t>(1, device_cu_count() / blocks);
  hipLaunchKernelGGL((linear_rows_kernel<WT, NS, R, ENDS, GATED>),
                     dim3((unsigned)std::min(units, per), (unsigned)blocks),
                     dim3(kStreamThreads), 0, s, a);
  return hipGetLastError();
}

template <typename WT, bool GATED>
static hipError_t launch_rows(const LinearArgs& a, hipStream_t s) {
  hipError_t e = hipSuccess;
  launch_by_steps<WT>(a.K * (int64_t)sizeof(WT), [&](auto steps, auto ring, auto ends) {
    e = run_rows<WT, steps.value, ring.value, ends.value, GATED>(a, s);
  });
  return e;
}

constexpr int64_t kMaxGridY = 65535;

template <typename WT, bool GATED>
static hipError_t launch_linear_t(const LinearArgs& a, hipStream_t s) {
  if (a.M <= 16) return launch_rows<WT, GATED>(a, s);
  // The tile (x rows by weight rows) with the least estimated time: rounds of tiles over the
  // CUs times the clocks of a tile, its steps (the slower of the loads at 45 bytes a clock
  // and CU and of the MFMAs) and a prologue and epilogue that grow with it.  Against the
  // largest tile that fills the CUs: 64 x 7168 x 2048 takes 64 x 32 tiles, 224 of them (one
  // round, 8.1 us), not 448 of 32 x 32 (11.7 us); 256 x 14336 x 4096 takes 224 tiles of 128 x
  // 128 (35.7 us) instead of 896 of 64 x 64 (49 us), but 512 x 4096 x 4096 takes 512 tiles of
  // 64 x 64 (27 us), not 128 of 128 x 128 (32 us).
  constexpr int out = GATED ? 2 : 1;   // weight rows per output column
  typedef Tile<WT> TT;
  const int64_t cus = device_cu_count(), steps = ceil_div(a.K, TT::BK);
  const int64_t row =
      std::max(a.ldx * (int64_t)sizeof(typename TT::X), a.ldw * (int64_t)sizeof(WT));
  const bool near_rows = row * 256 < ((int64_t)1 << 32);   // for tiles taller than 64
  // per: products that a CU does in a clock on such a tile, as measured in bf16
  auto clocks = [&](int m, int w, double per) -> double {
    if (m > 64 && !near_rows) return 1e300;
    const double loads = (m * (double)kXRow + w * (double)TT::WROW) / 45.0;
    const double mma = m * (double)w / (sizeof(WT) == 4 ? 3.4 : per / 64);
    const double tile = steps * std::max(loads, mma) + 4000.0 + m * (double)w / 4.0;
    return (double)ceil_div(ceil_div(a.M, m) * ceil_div(a.N * (int64_t)out, w), cus) * tile;
  };
  // float MFMAs bound every tile alike, and the registers of 256 x 256 spill (4096 x 4096 x
  // 4096 in 940 us, 919 without it)
  constexpr bool LARGE = sizeof(WT) != 4;
  const double t[] = {LARGE ? clocks(256, 256, 1536) : 1e300, clocks(256, 128, 1280),
                      clocks(128, 128, 1024),                 clocks(64, 64 * out, 1024),
                      clocks(64, 32 * out, 1024),             clocks(32, 32 * out, 1024)};
  // Blocks of 16 rows as weight streams: the most workgroups for a product of few tiles and
  // the whole of a CU for each, a later start (gated float 83 x 70 x 5488 in 32 x 32 tiles 46
  // us, in 16-row blocks 19; bf16 15 and 8.5; but bf16 64 x 1000 x 2048 6.8 and 7.9).
  const int64_t blocks = ceil_div(a.M, 16), units = ceil_div(a.N * (int64_t)out, 16);
  const int64_t per = std::min(units, std::max<int64_t>(1, cus / blocks));
  const double step = 16 * (kXRow + TT::WROW) / 34.0;
  // long rows: the token rows again for every unit
  const bool again = units > per && rows_in_chunks<WT>(a.K * (int64_t)sizeof(WT));
  const double run = (double)(ceil_div(units, per) * steps) * step * (again ? 1.5 : 1.0);
  const double rows = (double)ceil_div(blocks * per, cus) * (run + 8000.0);
  const double* best = std::min_element(t, t + 6);
  if (blocks <= kMaxGridY && rows < *best) return launch_rows<WT, GATED>(a, s);
  // Stages of the smallest tiles: as many as gain (gated 64 x 4096 x 14336: 53 us with 3 and 2
  // stages in 64 x 32 and 32 x 32 tiles, 39 with 4 and 3; 24 x 4096 x 4096 18 and 14.4; 8-bit
  // 33 and 25, though 14.4 against 13.5 for 83 x 70 x 5488).  Plain 64 x 32 tiles lose with 6
  // (64 x 7168 x 2048 9.5 -> 9.9 us: a longer start).
  switch ((int)(best - t)) {
    case 0:
      if constexpr (LARGE) return run_tiles<WT, 4, 2, 2, 4, 1, 2, GATED>(a, s);
      [[fallthrough]];
    case 1: return run_tiles<WT, 2, 2, 4, 2, 1, 3, GATED>(a, s);
    case 2: return run_tiles<WT, 1, 2, 4, 2, 1, 4, GATED>(a, s);
    case 3: return run_tiles<WT, 1, out, 2, 2, 1, GATED ? 3 : 4, GATED>(a, s);
    case 4: return run_tiles<WT, 1, out, 2, 1, 2, 4, GATED>(a, s);
    default: return run_tiles<WT, 1, out, 1, 1, 4, GATED ? 3 : 4, GATED>(a, s);
  }
}

template <typename WT>
static hipError_t launch_linear_w(const LinearArgs& a, bool gated, hipStream_t s) {
  return gated ? launch_linear_t<WT, true>(a, s) : launch_linear_t<WT, false>(a, s);
}

static hipError_t launch_linear(const moe_linear_desc_t& d, const LinearArgs& a, bool gated,
                                bool fp8, hipStream_t s) {
  if (fp8) return launch_linear_w<uint8_t>(a, gated, s);
  return d.dtype == MOE_DTYPE_F32 ? launch_linear_w<float>(a, gated, s)
                                  : launch_linear_w<bf16_t>(a, gated, s);
}

// ------------------------------------------------------------------ host checks
constexpr int64_t kMaxStride = (int64_t)1 << 24;   // 64 float rows stay within 32-bit offsets

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
                                void* out, void* stream, bool gated, bool fp8) {
  moe_status_t st = validate_linear(desc, fp8);
  if (st != MOE_OK) return st;
  const moe_linear_desc_t& d = *desc;
  if (!W0 || (gated && !W1) || (fp8 && (!s0 || (gated && !s1))) || (d.M > 0 && (!x || !out)))
    return MOE_E_NULL;
  const int64_t ob = d.out_dtype == MOE_DTYPE_F32 ? 4 : 2;
  if (!aligned_to(x, 16) || !aligned_to(W0, 16) || !aligned_to(W1, 16) || !aligned_to(s0, 4) ||
      !aligned_to(s1, 4) || !aligned_to(b0, 4) || !aligned_to(b1, 4) ||
      !aligned_to(residual, ob) || !aligned_to(out, ob))
    return MOE_E_UNSUPPORTED;
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
                     d.act,
                     d.out_dtype == MOE_DTYPE_F32,
                     aligned_to(out, 16) && aligned_to(residual, 16) &&
                         (d.ldo ? d.ldo : d.N) * ob % 16 == 0 &&
                         (d.ldr ? d.ldr : d.N) * ob % 16 == 0};
  return launch_linear(d, a, gated, fp8, (hipStream_t)stream) == hipSuccess ? MOE_OK : MOE_E_HIP;
}

}  // namespace moe

using namespace moe;

extern "C" {

moe_status_t moe_linear_validate(const moe_linear_desc_t* desc, int fp8) {
  return validate_linear(desc, fp8 != 0);
}

moe_status_t moe_linear(const moe_linear_desc_t* desc, const void* x, const void* W,
                        const float* bias, const void* residual, void* out, void* stream) {
  return linear_impl(desc, x, W, nullptr, nullptr, nullptr, bias, nullptr, residual, out, stream,
                     false, false);
}

moe_status_t moe_linear_gated(const moe_linear_desc_t* desc, const void* x, const void* W_gate,
                              const void* W_up, const float* bias_gate, const float* bias_up,
                              const void* residual, void* out, void* stream) {
  return linear_impl(desc, x, W_gate, W_up, nullptr, nullptr, bias_gate, bias_up, residual, out,
                     stream, true, false);
}

moe_status_t moe_linear_fp8(const moe_linear_desc_t* desc, const void* x, const uint8_t* Wq,
                            const float* s, const float* bias, const void* residual, void* out,
                            void* stream) {
  return linear_impl(desc, x, Wq, nullptr, s, nullptr, bias, nullptr, residual, out, stream, false,
                     true);
}

moe_status_t moe_linear_gated_fp8(const moe_linear_desc_t* desc, const void* x,
                                  const uint8_t* Wq_gate, const uint8_t* Wq_up,
                                  const float* s_gate, const float* s_up,
                                  const float* bias_gate, const float* bias_up,
                                  const void* residual, void* out, void* stream) {
  return linear_impl(desc, x, Wq_gate, Wq_up, s_gate, s_up, bias_gate, bias_up, residual, out,
                     stream, true, true);
}

}  // extern "C"
