// Device helpers of the short convolution and the selective scan.
#pragma once

#include "kda_device.h"
#include "kda_ssm_internal.h"

namespace kda {

// LDS operations are complete and all waves here; loads from memory stay in flight.
__device__ __forceinline__ void meet() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// a / b of numbers that are not negative, and mostly fit 32 bits.
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
  return a / b;
}

// The sequence that slot w belongs to where sequence n has the slots from cu[n] / len + n on:
// the last n with cu[n] / len + n <= w, 64 candidates at a time. w is uniform over the wave.
__device__ __forceinline__ int64_t find_sequence(const int64_t* cu, int64_t n, int64_t len,
                                                 int64_t w) {
  const int lane = threadIdx.x & 63;
  int64_t lo = 0, size = n;
  while (size > 1) {
    const int64_t step = (size + 63) / 64;
    const int64_t at = lo + lane * step;
    const bool ok = lane * step < size && divide(cu[at], len) + at <= w;
    const int c = __popcll(__ballot(ok));
    const int64_t skip = (c > 0 ? c - 1 : 0) * step;
    lo += skip;
    size = size - skip < step ? size - skip : step;
  }
  return lo;
}

__device__ __forceinline__ float load_state(const StateSlots& s, int64_t at) {
  return s.bf16 ? load1<true>(s.in, at) : load1<false>(s.in, at);
}

__device__ __forceinline__ void store_state(const StateSlots& s, int64_t at, float x) {
  if (s.bf16) static_cast<unsigned short*>(s.out)[at] = float_to_bf16_bits(x);
  else static_cast<float*>(s.out)[at] = x;
}

// Elements of a sequence's slot for reading or writing; negative where it has none.
__device__ __forceinline__ int64_t slot_in(const StateSlots& s, int64_t n) {
  const int64_t i = s.in_idx ? s.in_idx[n] : n;
  return s.in && i >= 0 && i < s.slots ? i * s.pitch : -1;
}
__device__ __forceinline__ int64_t slot_out(const StateSlots& s, int64_t n) {
  const int64_t i = s.out_idx ? s.out_idx[n] : n;
  return s.out && i >= 0 && i < s.slots ? i * s.pitch : -1;
}

// Four elements of a state that is read and written once in a call and then not until the
// next step, behind all other layers: past the caches. 128 states of 8192 x 16 FP32 between
// slots of a pool, buffers in turn: 29.1 us, 32.1 through the caches (28 and 22 where the same
// 134 MB are used again at once and stay in the last-level cache).
template <bool BF16>
__device__ __forceinline__ f32x4 load_once4(const void* base, int64_t at) {
  if constexpr (BF16) {
    const u32x2 w = __builtin_nontemporal_load(
        reinterpret_cast<const u32x2*>(static_cast<const unsigned short*>(base) + at));
    return f32x4{__uint_as_float(w[0] << 16), __uint_as_float(w[0] & 0xffff0000u),
                 __uint_as_float(w[1] << 16), __uint_as_float(w[1] & 0xffff0000u)};
  } else {
    return __builtin_nontemporal_load(reinterpret_cast<const f32x4*>(static_cast<const float*>(base) + at));
  }
}
template <bool BF16>
__device__ __forceinline__ void store_once4(void* base, int64_t at, f32x4 x) {
  if constexpr (BF16)
    __builtin_nontemporal_store(pack4(x), reinterpret_cast<i16x4*>(static_cast<unsigned short*>(base) + at));
  else
    __builtin_nontemporal_store(x, reinterpret_cast<f32x4*>(static_cast<float*>(base) + at));
}

// x / (1 + exp(-x))
__device__ __forceinline__ float siluf_(float x) { return x * sigmoidf_(x); }

constexpr float kLog2e = 1.44269504088896341f;

// log(1 + exp(x)) = max(x, 0) + log(w) + (e - (w - 1)), e = exp(-|x|), w = 1 + e rounded: the
// last term is what the rounding lost (its division by w is left out, 4e-8 of the result at
// most). Without it the small step sizes would lose all digits. Off by 5 units of 2^-24 for x
// from -2 on, 11 at -10, where the rounded exponent counts.
__device__ __forceinline__ float softplusf_(float x) {
  const float e = __builtin_amdgcn_exp2f(-kLog2e * fabsf(x));
  const float w = 1.f + e;
  return fmaxf(x, 0.f) + __builtin_fmaf(__builtin_amdgcn_logf(w), 0.693147180559945309f, e - (w - 1.f));
}

}  // namespace kda
