// Host-side checks of the dense products' and the few-token layer's argument validation and
// workspace sizes, built with AddressSanitizer and UndefinedBehaviorSanitizer on the host code.
// Makes no GPU call: every entry point is driven only into paths that fail validation before
// anything is enqueued, or that enqueue nothing.  Exits nonzero on any violation.
#include <math.h>
#include <stdint.h>
#include <stdio.h>
#include <string.h>

#include "moe.h"

static int failures = 0;
#define CHECK(c)                                                       \
  do {                                                                 \
    if (!(c)) {                                                        \
      fprintf(stderr, "check failed at line %d: %s\n", __LINE__, #c); \
      ++failures;                                                      \
    }                                                                  \
  } while (0)

static uint64_t rng_state = 0x2545F4914F6CDD1Dull;
static uint64_t next_u64() {
  rng_state ^= rng_state >> 12;
  rng_state ^= rng_state << 25;
  rng_state ^= rng_state >> 27;
  return rng_state * 0x9E3779B97F4A7C15ull;
}
template <int N>
static int64_t pick(const int64_t (&v)[N]) {
  return v[next_u64() % N];
}

int main() {
  void* const fake = (void*)0x100000;   // never dereferenced
  const float* const ff = (const float*)fake;
  const uint8_t* const fq = (const uint8_t*)fake;

  const int64_t Ms[] = {-1, 0, 1, 16, 17, 4096, 1 << 24, (1 << 24) + 1, (int64_t)1 << 40, INT64_MAX,
                        INT64_MIN};
  const int64_t Ns[] = {-1, 0, 1, 1001, 14336, 1 << 20, (1 << 20) + 1, INT64_MAX, INT64_MIN};
  const int64_t Ks[] = {-8, 0, 1, 4, 8, 12, 16, 24, 4096, 1 << 20, (1 << 20) + 16, INT64_MAX - 15};
  const int64_t Ls[] = {-1, 0, 8, 16, 4096, 4104, 1 << 24, (1 << 24) + 16, INT64_MAX, INT64_MIN};
  int valid = 0, rejected = 0;
  for (int it = 0; it < 300000; ++it) {
    moe_linear_desc_t d;
    memset(&d, 0, sizeof d);
    d.M = pick(Ms);
    d.N = pick(Ns);
    d.K = pick(Ks);
    if (it & 1) {
      d.ldx = pick(Ls);
      d.ldw = pick(Ls);
      d.ldr = pick(Ls);
      d.ldo = pick(Ls);
    }
    d.dtype = (int32_t)(next_u64() % 4) - 1;
    d.out_dtype = (int32_t)(next_u64() % 4) - 1;
    d.act = (int32_t)(next_u64() % 7) - 1;
    for (int fp8 = 0; fp8 < 2; ++fp8) {
      const moe_status_t st = moe_linear_validate(&d, fp8);
      if (st == MOE_OK) {
        ++valid;
        CHECK(d.M >= 0 && d.M <= 1 << 24 && d.N >= 1 && d.N <= 1 << 20 && d.K >= 1);
        CHECK(d.K % (fp8 ? 16 : d.dtype == MOE_DTYPE_F32 ? 4 : 8) == 0);
        CHECK(!fp8 || d.dtype == MOE_DTYPE_BF16);
        // a NULL weight matrix is found before anything is enqueued
        CHECK((fp8 ? moe_linear_fp8(&d, fake, nullptr, ff, ff, fake, fake, nullptr)
                   : moe_linear(&d, fake, nullptr, ff, fake, fake, nullptr)) == MOE_E_NULL);
        CHECK((fp8 ? moe_linear_gated_fp8(&d, fake, fq, fq, ff, nullptr, ff, ff, fake, fake, nullptr)
                   : moe_linear_gated(&d, fake, fake, nullptr, ff, ff, fake, fake, nullptr)) ==
              MOE_E_NULL);
        if (d.M == 0)   // nothing is enqueued
          CHECK((fp8 ? moe_linear_fp8(&d, nullptr, fq, ff, nullptr, nullptr, nullptr, nullptr)
                     : moe_linear(&d, nullptr, fake, nullptr, nullptr, nullptr, nullptr)) == MOE_OK);
      } else {
        ++rejected;
        CHECK((fp8 ? moe_linear_fp8(&d, fake, fq, ff, ff, fake, fake, nullptr)
                   : moe_linear(&d, fake, fake, ff, fake, fake, nullptr)) == st);
      }
    }
  }
  CHECK(valid > 100 && rejected > 1000);
  CHECK(moe_linear_validate(nullptr, 0) == MOE_E_NULL);

  int few = 0;
  for (int it = 0; it < 200000; ++it) {
    moe_desc_t d;
    memset(&d, 0, sizeof d);
    d.T = (int64_t)(next_u64() % 20) - 1;
    d.d_model = 64 * (int64_t)(next_u64() % 1026);
    d.n_experts = (int64_t)(next_u64() % 515);
    d.d_ff = 64 * (int64_t)(next_u64() % 1026);
    d.top_k = (int64_t)(next_u64() % 18);
    d.n_shared = (int64_t)(next_u64() % 3);
    d.capacity_factor = it % 3 ? 0.0f : 1.25f;
    d.dtype = (int32_t)(next_u64() % 3);
    d.out_dtype = (int32_t)(next_u64() % 3);
    const bool ok = moe_validate(&d) == MOE_OK && d.T <= MOE_FEW_TOKENS;
    const size_t need = moe_workspace_bytes_few(&d);
    CHECK((need > 0) == ok);
    if (!ok) {
      CHECK(moe_forward_few(&d, fake, fake, ff, fake, fake, fake, fake, fake, nullptr, nullptr, fake,
                            SIZE_MAX, nullptr) != MOE_OK);
      continue;
    }
    ++few;
    CHECK(need % 256 == 0);
    // room for h and for at least one partial sum of every row
    const size_t rows = (size_t)(d.T * (d.top_k + d.n_shared));
    CHECK(need >= rows * (size_t)d.d_ff * 4 + rows * (size_t)d.d_model * 4);
    CHECK(moe_forward_few(&d, fake, fake, ff, fake, fake, fake, fake, fake, nullptr, nullptr, fake,
                          need - 1, nullptr) == MOE_E_WORKSPACE);
    CHECK(moe_forward_few(&d, fake, fake, ff, fake, nullptr, fake, fake, fake, nullptr, nullptr, fake,
                          need, nullptr) == MOE_E_NULL);
    CHECK(moe_forward_few_fp8(&d, fake, fake, ff, fq, fq, fq, ff, nullptr, ff, fake, fake, nullptr,
                              nullptr, fake, need, nullptr) ==
          (d.dtype == MOE_DTYPE_BF16 ? MOE_E_NULL : MOE_E_UNSUPPORTED));
  }
  CHECK(few > 1000);
  printf("%d valid products, %d rejected, %d valid layers, %d failures\n", valid, rejected, few,
         failures);
  return failures != 0;
}
