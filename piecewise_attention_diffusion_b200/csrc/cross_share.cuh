// How many CTAs k_cross_few gives to each head, for the kernel and for k_join.
#pragma once
#include "common.cuh"
#include "internal.h"

namespace bsa {
namespace cross {

// The real keys of a batch entry's heads, counted in rounds of a CTA.
struct Shares {
  const int32_t* key_len;
  int Bt, Hkv, Lk, round;
  int ctas;  // to be shared by rounds over at most ctas / 2 heads; 0: `runs` for every head
  int runs;
  __device__ __forceinline__ int len(int b) const {
    return key_len == nullptr ? Lk : min(max(__ldg(key_len + b), 0), Lk);
  }
  __device__ __forceinline__ int rounds(int b) const { return ceil_div(len(b), round); }
};

// Rounds per CTA so that `ctas` CTAs, none of which works for two heads, take all rounds: the
// least of 32 candidates, one per lane, from an even share to three times that (twice that is
// enough for ctas / 2 heads).
__device__ __forceinline__ int rounds_per_cta(const Shares& s) {
  const int lane = threadIdx.x % 32;
  int total = 0;
  for (int i = lane; i < s.Bt; i += 32) total += s.rounds(i);
  total = s.Hkv * __reduce_add_sync(0xffffffffu, total);
  const int even = max(1, ceil_div(total, s.ctas)), per = even + even * lane / 16;
  int need = 0;
#pragma unroll 4
  for (int i = 0; i < s.Bt; ++i) need += ceil_div(s.rounds(i), per);
  const uint32_t fits = __ballot_sync(0xffffffffu, s.Hkv * need <= s.ctas);
  return __shfl_sync(0xffffffffu, per, __ffs(fits) - 1);
}

}  // namespace cross
}  // namespace bsa
