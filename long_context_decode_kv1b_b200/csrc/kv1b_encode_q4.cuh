// kv1b_encode_q4.cuh -- the encoders' form with 4 lanes per token (lane = 4 tau + j: token tau of an
// 8-token group, part j; lane j holds key channels j + 4 r, r = 0..31): rotation, fixed-order sums and
// row loads, shared by the contiguous and the paged prefill encoders.
#pragma once
#include "kv1b_device.cuh"

namespace kv1b {

// 32-bit mask of the rotation signs of lane j's key channels j + 4 r (bit r set: D = -1) for round rd:
// four coalesced loads, one ballot each (bit l of ballot i = channel 32 i + l), then the stride-4
// bits j, j + 4, .., j + 28 of each ballot packed into byte i.
__device__ __forceinline__ uint32_t sign_mask(const float* signs, int rd, int j) {
  const int lane = threadIdx.x & 31;
  uint32_t m = 0u;
  #pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t x = (__ballot_sync(kFull, __ldg(signs + rd * kD + 32 * i + lane) < 0.0f) >> j) & 0x11111111u;
    x = (x | (x >> 3)) & 0x03030303u;
    x = (x | (x >> 6)) & 0x000F000Fu;
    x = (x | (x >> 12)) & 0x000000FFu;
    m |= x << (8 * i);
  }
  return m;
}

// One round y <- H (D (.) y): stages h = 1, 2 across the token's 4 lanes, h = 4 .. 64 inside.
__device__ __forceinline__ void rotate_q4(float x[32], uint32_t smask, int j) {
  #pragma unroll
  for (int r = 0; r < 32; ++r)  // D: flip the sign bit where the mask has a 1
    x[r] = __int_as_float(__float_as_int(x[r]) ^ static_cast<int>((smask << (31 - r)) & 0x80000000u));
  #pragma unroll
  for (int h = 1; h <= 2; h <<= 1) {
    const float sgn = (j & h) ? -1.0f : 1.0f;  // the lane of the pair's upper element forms a - c
    #pragma unroll
    for (int r = 0; r < 32; ++r) x[r] = __fmaf_rn(sgn, x[r], __shfl_xor_sync(kFull, x[r], h));
  }
  #pragma unroll
  for (int hr = 1; hr <= 16; hr <<= 1) {
    #pragma unroll
    for (int r = 0; r < 32; ++r) {
      if (r & hr) continue;
      const float a = x[r], c = x[r + hr];
      x[r] = __fadd_rn(a, c);
      x[r + hr] = __fsub_rn(a, c);
    }
  }
}

// Fixed pairwise tree over the token's 128 channels (lane j: channels j + 4 r); h = 64 .. 4 inside
// the lane, 2 and 1 across lanes.  Returns the sum on each of the token's lanes.  a is overwritten.
__device__ __forceinline__ float tree_sum_q4(float a[32]) {
  #pragma unroll
  for (int hr = 16; hr >= 1; hr >>= 1)
    #pragma unroll
    for (int r = 0; r < hr; ++r) a[r] = __fadd_rn(a[r], a[r + hr]);
  float x = a[0];
  x = __fadd_rn(x, __shfl_xor_sync(kFull, x, 2));  // h = 2: lanes j < 2 add lane j + 2
  x = __fadd_rn(x, __shfl_xor_sync(kFull, x, 1));  // h = 1: lane 0 adds lane 1
  return __shfl_sync(kFull, x, (threadIdx.x & 31) & ~3);
}

// Element types of the K / V rows (the kernel is compiled once per type).
template <int DT> struct Elem;
template <> struct Elem<KV1B_DTYPE_F32> {
  typedef float T;
  static __device__ __forceinline__ float get(float x) { return x; }
};
template <> struct Elem<KV1B_DTYPE_BF16> {
  typedef unsigned short T;
  static __device__ __forceinline__ float get(unsigned short x) { return __uint_as_float(static_cast<uint32_t>(x) << 16); }
};
template <> struct Elem<KV1B_DTYPE_F16> {
  typedef unsigned short T;
  static __device__ __forceinline__ float get(unsigned short x) { return __half2float(__ushort_as_half(x)); }
};

// sum over i = 0..7 of (0x4B000000 << 4 i) modulo 2^32: the exponent bits of 2^23 + code, shifted
// into each nibble's place (only i = 0, 1 keep any bits)
constexpr uint32_t kMagicPacked = 0x4B000000u + (0x4B000000u << 4);

}  // namespace kv1b
