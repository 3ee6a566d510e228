// Weight rows streamed once through a workgroup against at most 16 token rows.
//
// With so few token rows a product reads far more weight bytes than it computes on (16 x 2
// operations for 2 bytes of bf16 at most, where the matrix cores do some 400 per byte of
// HBM), so everything here serves the stream: 16 weight rows at a time, the reduction
// dimension split over the 8 waves of a workgroup, each wave with several KB of loads in
// flight, and MFMA 16x16 tiles whose cost does not show.
//
// A step is 128 bytes of each of the 16 rows (SK elements); wave w takes steps w, w + 8, ...
// so the workgroup reads 1 KB runs of a row.  A step is loaded with 8 lanes per 128-byte
// segment (a lane per row, as the MFMA operand has it, would run the load path at a quarter
// of its rate) and put into operand order through a wave-private LDS buffer: 16-byte chunk
// c of row r at position c ^ ((r / 2) % 8), conflict-free both ways.  Lane (row r, group g)
// then holds chunks 2 g and 2 g + 1 of its row; token operands use the same k order.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <type_traits>

#include "moe_internal.h"

namespace moe {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef float floatx4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

constexpr int kStreamThreads = 512, kStreamWaves = kStreamThreads / 64;
constexpr int kStepBytes = 128;            // of each row
constexpr int kStageBytes = 16 * kStepBytes;   // a wave's LDS buffer

// 8 e4m3 codes (bytes of lo, then hi) -> 8 bf16 operands, exactly.
__device__ __forceinline__ bf16x8 widen_e4m3(uint32_t lo, uint32_t hi) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, false);
  const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)lo, 1.0f, true);
  const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, false);
  const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)hi, 1.0f, true);
  return bf16x8{a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
}

// One lane's token operand of a step, and the product with the staged weights.
//   XR  16-byte registers of the operand; register i holds the elements from
//       k_of(g, i) on (8 bf16 or 4 floats)
template <typename WT>
struct Stream;

template <>
struct Stream<bf16_t> {
  static constexpr int SK = 64, XR = 2, XE = 8;
  typedef bf16_t X;
  __device__ static int k_of(int g, int i) { return 16 * g + 8 * i; }
  __device__ static void mma(floatx4& acc, const u32x4* x, u32x4 w0, u32x4 w1) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[0]),
                                                  __builtin_bit_cast(bf16x8, w0), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[1]),
                                                  __builtin_bit_cast(bf16x8, w1), acc, 0, 0, 0);
  }
};

template <>
struct Stream<uint8_t> {
  static constexpr int SK = 128, XR = 4, XE = 8;
  typedef bf16_t X;
  __device__ static int k_of(int g, int i) { return 32 * g + 8 * i; }
  __device__ static void mma(floatx4& acc, const u32x4* x, u32x4 w0, u32x4 w1) {
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[0]),
                                                  widen_e4m3(w0[0], w0[1]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[1]),
                                                  widen_e4m3(w0[2], w0[3]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[2]),
                                                  widen_e4m3(w1[0], w1[1]), acc, 0, 0, 0);
    acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x[3]),
                                                  widen_e4m3(w1[2], w1[3]), acc, 0, 0, 0);
  }
};

template <>
struct Stream<float> {
  static constexpr int SK = 32, XR = 2, XE = 4;
  typedef float X;
  __device__ static int k_of(int g, int i) { return 8 * g + 4 * i; }
  __device__ static void mma(floatx4& acc, const u32x4* x, u32x4 w0, u32x4 w1) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[0][i]),
                                                 __uint_as_float(w0[i]), acc, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(x[1][i]),
                                                 __uint_as_float(w1[i]), acc, 0, 0, 0);
  }
};

// Puts a step's two loads (rows lane / 8 and 8 + lane / 8, chunk lane % 8) into operand
// order.  The buffer belongs to the wave and LDS operations of a wave run in order, so
// neither call needs a barrier.
__device__ __forceinline__ void stage_in(char* buf, int lane, u32x4 a, u32x4 b) {
  const int r = lane >> 3, c = lane & 7;
  *reinterpret_cast<u32x4*>(buf + r * kStepBytes + 16 * (c ^ (r >> 1))) = a;
  *reinterpret_cast<u32x4*>(buf + (r + 8) * kStepBytes + 16 * (c ^ ((r + 8) >> 1))) = b;
}
__device__ __forceinline__ void stage_out(const char* buf, int lane, u32x4& w0, u32x4& w1) {
  const int r = lane & 15, g = lane >> 4;
  w0 = *reinterpret_cast<const u32x4*>(buf + r * kStepBytes + 16 * ((2 * g) ^ (r >> 1)));
  w1 = *reinterpret_cast<const u32x4*>(buf + r * kStepBytes + 16 * ((2 * g + 1) ^ (r >> 1)));
}

// The wave's part of one product over steps st0 .. st1 - 1, all within the rows: w_at(i, byte)
// gives the address of load i (rows lane / 8, 8 + lane / 8) at a byte of the row, x_at(k) the
// lane's token operand at element k (or nullptr: zero).  R steps are loaded at a time.
template <typename WT, int R, typename WAt, typename XAt>
__device__ __forceinline__ void stream_rows(floatx4& acc, char* buf, int st0, int st1, WAt w_at,
                                            XAt x_at) {
  typedef Stream<WT> S;
  const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6, g = lane >> 4;
  for (int j = st0 + wv; j < st1; j += R * kStreamWaves) {
    u32x4 w[R][2], x[R][S::XR];
#pragma unroll
    for (int q = 0; q < R; ++q) {
      const int st = j + q * kStreamWaves;
      if (st >= st1) break;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        w[q][i] = *reinterpret_cast<const u32x4*>(w_at(i, st * kStepBytes + 16 * (lane & 7)));
#pragma unroll
      for (int i = 0; i < S::XR; ++i) {
        const auto* p = x_at(st * S::SK + S::k_of(g, i));
        x[q][i] = p ? *reinterpret_cast<const u32x4*>(p) : u32x4{0, 0, 0, 0};
      }
    }
#pragma unroll
    for (int q = 0; q < R; ++q) {
      if (j + q * kStreamWaves >= st1) break;
      u32x4 w0, w1;
      stage_in(buf, lane, w[q][0], w[q][1]);
      stage_out(buf, lane, w0, w1);
      S::mma(acc, x[q], w0, w1);
    }
  }
}

// The waves' 16 x 16 partial products, summed in wave order.  Row stride 20 floats: the four
// lane groups of a store hit different banks.
constexpr int kRedLd = 20, kRedWave = 16 * kRedLd;
__device__ __forceinline__ void red_put(float* red, const floatx4& acc) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) red[(4 * g + i) * kRedLd + n] = acc[i];
}
// Sum of element (m, n) over the waves; red_stride floats from wave to wave.
__device__ __forceinline__ float red_get(const float* red, int red_stride, int m, int n) {
  float v = red[m * kRedLd + n];
#pragma unroll
  for (int q = 1; q < kStreamWaves; ++q) v += red[q * red_stride + m * kRedLd + n];
  return v;
}

// Share s of `of`: a run of consecutive units of n, the shares as even as they go.
__device__ inline void share_of(int64_t n, int s, int of, int64_t& i0, int64_t& i1) {
  i0 = n * s / of;
  i1 = n * (s + 1) / of;
}

// LDS of stream_units.
template <int NG>
struct StreamLds {
  __align__(16) char stage[kStreamWaves][kStageBytes];
  float red[2][kStreamWaves * NG * kRedWave];
};

// Units i0 .. i1 - 1 of NG x 16 weight rows each, against a token operand that stays in
// registers while it can.  A unit is visited once per chunk of NS steps per wave (NS x 8
// steps of the row; one chunk where the row is no longer).  A ring of R steps (R divides
// NS) runs across the visits: as step s is used, step s + R goes out, of this visit or of
// the next, so a wave always has R NG 2 KB in flight.
//   point(i, base)       base[g][h]: the lane's row of load h of group g; returns the row's
//                        first step
//   load_x(i, c, xs)     the wave's token operand of chunk c, xs[0 .. NH - 1] multiplied by
//                        the same weights (only called where it may have changed)
//   done(i, g, m, n, v)  sum v of token m and row n of group g, called by 256 threads (whole
//                        waves) for each group; ends the unit
//   nst, row_bytes       steps and bytes of a weight row
// Steps past nst repeat its last one and bytes past the row its last chunk (cache hits); the
// token operand must be zero there.
template <typename WT, int NS, int R, int NG, int NH, typename Point, typename LoadX,
          typename Done>
__device__ __forceinline__ void stream_units(int64_t i0, int64_t i1, int nchunk, int nst,
                                             int row_bytes, StreamLds<NG>& lds, Point point,
                                             LoadX load_x, Done done) {
  typedef Stream<WT> S;
  static_assert(NS % R == 0, "ring slots keep their steps");
  if (i0 >= i1) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = tid >> 6;
  char* stage = lds.stage[wv];
  u32x4 xs[NH][NS][S::XR], ring[R][NG][2];
  const char* base[NG][2];
  auto load = [&](int s, int st0) {
    const int st = min(st0 + s * kStreamWaves + wv, nst - 1);
    const int byte = min(st * kStepBytes + 16 * (lane & 7), row_bytes - 16);
#pragma unroll
    for (int g = 0; g < NG; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        ring[s % R][g][h] = *reinterpret_cast<const u32x4*>(base[g][h] + byte);
  };
  floatx4 acc[NG];
  int first = point(i0, base);   // of the unit that base points to
  // Chunk c of a unit; in, cn: the next visit, if there is one.
  auto visit = [&](auto more, int c, int64_t in, int cn) {
    const int st0 = first + c * NS * kStreamWaves;
    int stn = 0;
#pragma unroll
    for (int s = 0; s < NS; ++s) {
#pragma unroll
      for (int g = 0; g < NG; ++g) {
        u32x4 w0, w1;
        stage_in(stage, lane, ring[s % R][g][0], ring[s % R][g][1]);
        stage_out(stage, lane, w0, w1);
#pragma unroll
        for (int h = 0; h < NH; ++h) S::mma(acc[g], xs[h][s], w0, w1);
      }
      if (s + R < NS) {
        load(s + R, st0);
      } else if constexpr (decltype(more)::value) {
        if (s + R == NS) {
          first = point(in, base);
          stn = first + cn * NS * kStreamWaves;
        }
        load(s + R - NS, stn);
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
#pragma unroll
  for (int s = 0; s < R; ++s) load(s, first);
  int par = 0;
  for (int64_t i = i0; i < i1; ++i) {
#pragma unroll
    for (int g = 0; g < NG; ++g) acc[g] = floatx4{0.f, 0.f, 0.f, 0.f};
    for (int c = 0; c < nchunk; ++c) {
      load_x(i, c, xs);
      const bool last = c + 1 == nchunk;
      if (last && i + 1 == i1)
        visit(std::false_type{}, c, 0, 0);
      else
        visit(std::true_type{}, c, last ? i + 1 : i, last ? 0 : c + 1);
    }
#pragma unroll
    for (int g = 0; g < NG; ++g) red_put(lds.red[par] + (wv * NG + g) * kRedWave, acc[g]);
    __syncthreads();
    // one half of the workgroup (NG 1: the halves take turns; NG 2: one group each) sums up;
    // the other buffer is free until it has passed the next barrier
    const int half = tid >> 8, g = NG == 1 ? 0 : half, m = (tid >> 4) & 15, n = tid & 15;
    if (NG == 2 || half == par)
      done(i, g, m, n, red_get(lds.red[par] + g * kRedWave, NG * kRedWave, m, n));
    par ^= 1;
  }
}

}  // namespace moe
