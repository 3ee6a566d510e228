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
// of its rate) and comes into operand order through wave-private LDS: 16-byte chunk c of row
// r at position c ^ ((r / 2) % 8), conflict-free both ways.  Lane (row r, group g) then holds
// chunks 2 g and 2 g + 1 of its row; token operands use the same k order.
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
__device__ inline void share_of(int64_t n, int s, int of, int& i0, int& i1) {
  i0 = (int)(n * s / of);
  i1 = (int)(n * (s + 1) / of);
}

// LDS of stream_units: the waves' rings of steps, the waves' sums of a unit (two, in turn).
template <int R>
struct StreamLds {
  __align__(16) char ring[kStreamWaves][R][kStageBytes];
  float red[2][kStreamWaves * kRedWave];
};

// 16 bytes per lane from base + off straight into LDS at lds + 16 lane (base and lds, a byte
// offset, are uniform).  The compiler does not count this load: wait with wait_loads().
// ONCE: data that is read once and not kept in the caches for another reader; weight streams
// larger than the 256 MB cache run at 6.5 TB/s so, at 5.7 without.
template <bool ONCE = false>
__device__ __forceinline__ void load_to_lds(const char* base, uint32_t off, uint32_t lds) {
  lds = __builtin_amdgcn_readfirstlane(lds);   // nothing else here uses m0
  if constexpr (ONCE)
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt"
                 :: "v"(off), "s"(base), "s"(lds));
  else
    asm volatile("s_mov_b32 m0, %2\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, %1"
                 :: "v"(off), "s"(base), "s"(lds));
}
// All but the youngest N of the wave's memory operations have landed, every LDS access of this
// wave is done, LDS contents are new to the compiler.
template <int N = 0>
__device__ __forceinline__ void wait_loads() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
}
// Every vector load of the wave has landed, said so that the compiler knows it: a load whose
// value lives across visits would otherwise be waited for, and the ring with it, at its
// first use in every visit.
__device__ __forceinline__ void landed() {
  __builtin_amdgcn_s_waitcnt(0x0F70);   // vmcnt(0), the other counters free
}
// LDS byte offset of p, for load_to_lds.
__device__ __forceinline__ uint32_t lds_offset(const void* p) {
  return __builtin_amdgcn_readfirstlane((uint32_t)(uintptr_t)(
      const __attribute__((address_space(3))) char*)p);
}
// A pointer that is the same in the whole wave, in scalar registers.
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t v = (uint64_t)p;
  return (const char*)((uint64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
                       (uint32_t)__builtin_amdgcn_readfirstlane((int)v));
}

// p[i] through the scalar cache, for values that no kernel writes and an index that is the
// same in the whole wave: a vector load's wait would also wait for the loads to LDS.
__device__ __forceinline__ float scalar_f(const float* p, int64_t i) {
  return *(const __attribute__((address_space(4))) float*)uniform((const char*)(p + i));
}

// p[i + q], 0 <= q < N: N scalar loads and a choice per lane.
template <int N>
__device__ __forceinline__ float pick(const float* p, int64_t i, int q) {
  const auto* s = (const __attribute__((address_space(4))) float*)uniform((const char*)(p + i));
  float v = s[0];
#pragma unroll
  for (int j = 1; j < N; ++j) v = q == j ? s[j] : v;
  return v;
}

// Where the rows of a unit are: load h takes row h * 8 + lane / 8 at base[h] + off[h].
struct UnitRows {
  const char* base[2];   // uniform
  uint32_t off[2];       // per lane
};

// Where the token rows are that do not change from unit to unit: row h * 8 + lane / 8 at
// base + off[h], k elements (rows past the last token: any row, their sums are not used).
struct TokenRows {
  const char* base;   // uniform
  uint32_t off[2];    // per lane
  int k;
};

// Units i0 .. i1 - 1 of 16 weight rows each, against a token operand that stays in registers
// while it can.  A unit is visited once per chunk of NS steps per wave (NS x 8 steps of the
// row; one chunk where the row is no longer).  The steps come through a ring of R in LDS,
// filled by direct loads: as a step is used, the one R further goes out, of this visit or a
// later one (R divides NS or NS divides R), so a wave always has R x 2 KB in flight and no
// registers wait for them.
//   point(i, rows)       where unit i is; returns the row's first step
//   load_x               FIXED tokens: load_x(rows) says where they are.  They come through
//                        the ring too, before the weights (loaded in operand order, a lane
//                        per row, 16 rows of 14336 elements take 13 us); with more than one
//                        chunk every visit starts over, tokens first.
//                        Else: load_x(i, xs) loads the wave's operand for unit i (or leaves
//                        it as it is), xs[0 .. NH - 1] multiplied by the same weights, zero
//                        past the rows' end, ends with landed() and returns the unit's
//                        first step; one chunk only
//   done(i, m, n, v)     sum v of token m and weight row n of the unit, called by 256 threads
//                        (whole waves); a vector load there empties the ring
//   nst, row_bytes       steps and bytes of a weight row
// Steps past nst repeat its last one and bytes past the row its last chunk (cache hits); the
// token operand is zero there, and with ENDS the weights, which may be infinite, as well.
template <typename WT, int NS, int R, int NH, bool FIXED, bool ENDS, typename Point,
          typename LoadX, typename Done>
__device__ __forceinline__ void stream_units(int i0, int i1, int nchunk, int nst, int row_bytes,
                                             StreamLds<R>& lds, Point point, LoadX load_x,
                                             Done done) {
  typedef Stream<WT> S;
  static_assert(NS % R == 0 || R % NS == 0, "the ring's phase is the same in every visit");
  constexpr int AHEAD = R >= NS ? R / NS : 1;   // visits from a step's use to the one loaded
  i0 = __builtin_amdgcn_readfirstlane(i0);   // the same in every lane, in scalar registers
  i1 = __builtin_amdgcn_readfirstlane(i1);
  if (i0 >= i1) return;
  const int tid = threadIdx.x, lane = tid & 63, wv = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int visits = (i1 - i0) * nchunk;
  const uint32_t ring = lds_offset(lds.ring[wv][0]);
  u32x4 xs[NH][NS][S::XR];
  UnitRows rows;
  int first = 0;   // first step of the visit that rows points to
  auto point_at = [&](int v) {
    first = point(i0 + v / nchunk, rows) + v % nchunk * NS * kStreamWaves;
  };
  // A load of 8 rows: chunk c of row r goes to position c ^ (r / 2 % 8).
  auto load = [&](int s, uint32_t slot) {
    const int st = min(first + s * kStreamWaves + wv, nst - 1);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int chunk = (lane & 7) ^ (4 * h | (lane >> 4));
      const int byte = min(st * kStepBytes + 16 * chunk, row_bytes - 16);
      load_to_lds<true>(rows.base[h], rows.off[h] + (uint32_t)byte,
                        ring + slot + h * (kStageBytes / 2));
    }
  };
  floatx4 acc;
  uint32_t slot = 0;   // of the step in use, bytes from ring
  // Visit v, whose first step is `start`; more: the steps R further exist for all its steps.
  auto visit = [&](auto more, int v, int start) {
    if (AHEAD > 1 || R == NS) {
      if constexpr (decltype(more)::value) point_at(v + AHEAD);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      // steps that may still be under way when this one is needed
      const int rest = decltype(more)::value || NS - s > R ? R - 1 : NS - 1 - s;
      switch (rest) {   // a constant once unrolled
#define MOE_WAIT(n) case n: wait_loads<2 * n>(); break;
        MOE_WAIT(0) MOE_WAIT(1) MOE_WAIT(2) MOE_WAIT(3) MOE_WAIT(4) MOE_WAIT(5) MOE_WAIT(6)
#undef MOE_WAIT
        default: wait_loads<14>(); break;
      }
      u32x4 w0, w1;
      stage_out(lds.ring[wv][0] + slot, lane, w0, w1);
      // the slot is read out before it is filled again
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if constexpr (ENDS) {
        const int left = row_bytes - (start + s * kStreamWaves + wv) * kStepBytes;
#pragma unroll
        for (int e = 0; e < 4; ++e) {   // no branch: it would spill the 24-step form in float
          w0[e] = 32 * (lane >> 4) < left ? w0[e] : 0u;
          w1[e] = 32 * (lane >> 4) + 16 < left ? w1[e] : 0u;
        }
      }
      if (s + R < NS) {
        load(s + R, slot);
      } else if constexpr (decltype(more)::value) {
        if (R < NS && s + R == NS) point_at(v + 1);
        load(R < NS ? s + R - NS : s, slot);
      }
#pragma unroll
      for (int h = 0; h < NH; ++h) S::mma(acc, xs[h][s], w0, w1);
      slot = slot == (R - 1) * kStageBytes ? 0 : slot + kStageBytes;
    }
  };
  static_assert(R <= 8, "waits");
  // The first steps of visits v ..: as many as the ring holds, n visits at most.
  auto fill = [&](int v, int n) {
    slot = 0;
#pragma unroll
    for (int q = 0; q < AHEAD; ++q)
      if (q < n) {
        point_at(v + q);
#pragma unroll
        for (int s = 0; s < (R < NS ? R : NS); ++s) load(s, (q * NS + s) * kStageBytes);
      }
  };
  // Chunk c of the fixed tokens, R ring slots (128 bytes of each row) at a time.
  TokenRows tokens;
  if constexpr (FIXED) load_x(tokens);
  auto stage_x = [&](int c) {
    constexpr int PARTS = S::SK * (int)sizeof(typename S::X) / kStepBytes;   // slots of a step
    static_assert(R % PARTS == 0 && S::XR == 2 * PARTS, "whole steps, two chunks a slot");
    const int g = lane >> 4, r = lane & 15;
    const int end = tokens.k * (int)sizeof(typename S::X) - 16;
#pragma unroll
    for (int s0 = 0; s0 < NS; s0 += R / PARTS) {
#pragma unroll
      for (int q = 0; q < R; ++q) {
        if (s0 + q / PARTS >= NS) break;
        const int st = (c * NS + s0 + q / PARTS) * kStreamWaves + wv;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int chunk = (lane & 7) ^ (4 * h | (lane >> 4));
          const int byte = min((st * PARTS + q % PARTS) * kStepBytes + 16 * chunk, end);
          load_to_lds(tokens.base, tokens.off[h] + (uint32_t)byte,
                      ring + q * kStageBytes + h * (kStageBytes / 2));
        }
      }
      wait_loads();
#pragma unroll
      for (int q = 0; q < R / PARTS; ++q) {
        if (s0 + q >= NS) break;
        const int st = (c * NS + s0 + q) * kStreamWaves + wv;
#pragma unroll
        for (int i = 0; i < S::XR; ++i) {
          const int at = S::XR * g + i;   // 16-byte chunk of the step
          const u32x4 v = *reinterpret_cast<const u32x4*>(
              lds.ring[wv][q * PARTS + (PARTS == 1 ? 0 : at >> 3)] + r * kStepBytes +
              16 * ((at & 7) ^ (r >> 1)));
          const bool in = st * S::SK + S::k_of(g, i) < tokens.k;
#pragma unroll
          for (int e = 0; e < 4; ++e) xs[0][s0 + q][i][e] = in ? v[e] : 0u;
        }
      }
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");   // read out before the next loads
    }
  };
  const bool restart = FIXED && nchunk > 1;
  if constexpr (FIXED) {
    if (!restart) stage_x(0);
  }
  if (!restart) fill(0, visits);
  int par = 0;
  for (int v = 0, i = i0; i < i1; ++i) {
    acc = floatx4{0.f, 0.f, 0.f, 0.f};
    if (restart) {
      if constexpr (FIXED) {
        for (int c = 0; c < nchunk; ++c, ++v) {
          stage_x(c);
          fill(v, 1);
          visit(std::false_type{}, v, c * NS * kStreamWaves);
        }
      }
    } else {
      int start = 0;
      if constexpr (!FIXED) start = __builtin_amdgcn_readfirstlane(load_x(i, xs));
      if (v + AHEAD < visits)
        visit(std::true_type{}, v, start);
      else
        visit(std::false_type{}, v, start);
      ++v;
    }
    red_put(lds.red[par] + wv * kRedWave, acc);
    __syncthreads();
    // the halves of the workgroup take turns to sum up; the other buffer is free until the
    // summing half has passed the next barrier
    if (tid >> 8 == par) {
      const int m = (tid >> 4) & 15, n = tid & 15;
      done(i, m, n, red_get(lds.red[par], kRedWave, m, n));
    }
    par ^= 1;
  }
}

// Whether rows of row_bytes end inside the NS x 8 steps of a visit.  A form of its own: masking
// costs 10% of float rows (14.8 -> 16.4 us for 16 x 4096 x 4096).  8-bit weights have no
// infinities and need none.
template <typename WT>
bool row_ends(int64_t row_bytes, int ns) {
  return sizeof(WT) > 1 && row_bytes % ((int64_t)ns * kStreamWaves * kStepBytes) != 0;
}

// Whether launch_by_steps runs rows of row_bytes in several chunks.
template <typename WT>
bool rows_in_chunks(int64_t row_bytes) {
  return row_bytes > (sizeof(WT) == 1 ? 8 : 24) * (int64_t)kStreamWaves * kStepBytes;
}

// Calls launch(steps, ring, ends) with the form of stream_units for rows of row_bytes: the least
// number of steps per wave that holds the rows, so that the token operand stays in registers;
// longer rows run in the chunks that pad them least.  An 8-bit step takes twice the
// operand's registers.
template <typename WT, typename Launch>
void launch_by_steps(int64_t row_bytes, Launch launch) {
  const int64_t per = ceil_div(row_bytes, (int64_t)kStreamWaves * kStepBytes);
  auto run = [&](auto steps, auto ring) {
    if constexpr (sizeof(WT) > 1) {
      if (row_ends<WT>(row_bytes, steps.value)) return launch(steps, ring, std::true_type{});
    }
    launch(steps, ring, std::false_type{});
  };
#define MOE_STEPS(n, r) run(std::integral_constant<int, n>{}, std::integral_constant<int, r>{})
  if (per <= 2) return MOE_STEPS(2, 8);
  if (per <= 4) return MOE_STEPS(4, 8);
  if constexpr (sizeof(WT) == 1) {
    return MOE_STEPS(8, 8);
  } else {
    if (per <= 8) return MOE_STEPS(8, 8);
    if (per <= 14) return MOE_STEPS(14, 7);
    if (per <= 16) return MOE_STEPS(16, 8);
    if (per <= 24) return MOE_STEPS(24, 8);
    return ceil_div(per, 14) * 14 < ceil_div(per, 16) * 16 ? MOE_STEPS(14, 7) : MOE_STEPS(16, 8);
  }
#undef MOE_STEPS
}

}  // namespace moe
