// Wave-wide reductions in registers (DPP and permlane swaps), shared by the routers.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Lane exchanges for wave-wide reductions.  Inside a 16-lane row: DPP quad swaps (1,0,3,2)
// and (2,3,0,1), then the half-row and row mirrors; across rows: v_permlane16_swap and
// v_permlane32_swap, which hand every lane the values of both rows (or halves) of its pair.
// After each step every lane of the group holds op(a, b) of the same two values, so with a
// commutative op all 64 lanes end with the same bits.
constexpr int DPP_QUAD_1032 = 0xB1, DPP_QUAD_2301 = 0x4E, DPP_HALF_MIRROR = 0x141,
              DPP_MIRROR = 0x140;

template <int CTRL>
__device__ inline int dpp_i(int v) {
  return __builtin_amdgcn_mov_dpp(v, CTRL, 0xf, 0xf, false);
}
template <int CTRL>
__device__ inline float dpp_f(float v) {
  return __int_as_float(dpp_i<CTRL>(__float_as_int(v)));
}

template <class Op>
__device__ inline float wave_reduce(float v, Op op) {
  v = op(v, dpp_f<DPP_QUAD_1032>(v));
  v = op(v, dpp_f<DPP_QUAD_2301>(v));
  v = op(v, dpp_f<DPP_HALF_MIRROR>(v));
  v = op(v, dpp_f<DPP_MIRROR>(v));
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v),
                                                  false, false);
  v = op(__uint_as_float(r[0]), __uint_as_float(r[1]));
  const auto q = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v),
                                                  false, false);
  return op(__uint_as_float(q[0]), __uint_as_float(q[1]));
}
__device__ inline float wave_max(float v) {
  return wave_reduce(v, [](float a, float b) { return fmaxf(a, b); });
}
__device__ inline float wave_sum(float v) {
  return wave_reduce(v, [](float a, float b) { return a + b; });
}

// (v, e) <- the better of (v, e) and (ov, oe): larger score, lower expert on equal scores.
// Written without short-circuit operators so that it compiles to compares and selects
// (a branch per compare, with its exec-mask bookkeeping, made each top-k round ~10x slower).
__device__ inline void take_better(float& v, int& e, float ov, int oe) {
  const bool better = (ov > v) | ((ov == v) & (oe < e));
  v = better ? ov : v;
  e = better ? oe : e;
}
template <int CTRL>
__device__ inline void argmax_step(float& v, int& e) {
  const float ov = dpp_f<CTRL>(v);
  const int oe = dpp_i<CTRL>(e);
  take_better(v, e, ov, oe);
}
// Wave-wide argmax of (score, expert); every lane ends with the winner.
__device__ inline void wave_argmax(float& v, int& e) {
  argmax_step<DPP_QUAD_1032>(v, e);
  argmax_step<DPP_QUAD_2301>(v, e);
  argmax_step<DPP_HALF_MIRROR>(v, e);
  argmax_step<DPP_MIRROR>(v, e);
  {
    const auto rv = __builtin_amdgcn_permlane16_swap(__float_as_uint(v), __float_as_uint(v),
                                                     false, false);
    const auto re = __builtin_amdgcn_permlane16_swap((unsigned)e, (unsigned)e, false, false);
    v = __uint_as_float(rv[0]);
    e = (int)re[0];
    take_better(v, e, __uint_as_float(rv[1]), (int)re[1]);
  }
  {
    const auto rv = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v),
                                                     false, false);
    const auto re = __builtin_amdgcn_permlane32_swap((unsigned)e, (unsigned)e, false, false);
    v = __uint_as_float(rv[0]);
    e = (int)re[0];
    take_better(v, e, __uint_as_float(rv[1]), (int)re[1]);
  }
}

}  // namespace moe
