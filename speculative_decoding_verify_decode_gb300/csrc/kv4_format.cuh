// Layout and arithmetic of the 4-bit cache (include/sd_kv4.h), shared by its
// append, read and attention.  Internal to the library.
#pragma once

#include <cstdint>
#include <cuda_bf16.h>

#include "common.cuh"

namespace sdv {
namespace {

constexpr int kKv4Block = 32;                       // dims that share a scale
// Bytes of a K or V record of one (page, KV head), and of its codes (scales behind them).
__host__ __device__ constexpr int kv4_record(int dim) { return 9 * dim; }
__host__ __device__ constexpr int kv4_codes(int dim) { return 8 * dim; }
// A scale's bits that count, and the first magnitude that is none: 24 s (see kv4_pair) would not be finite.
constexpr uint32_t kKv4ScaleBits = 0xfff8u;
constexpr uint32_t kKv4BadScale = 0x7d30u;          // 1.375 * 2^123; the largest scale is 1.3125 * 2^123

// Bit of code e of a word of eight: the codes of neighbours lie in the two halves, so that one mask takes a pair.
__host__ __device__ constexpr int kv4_shift(int e) { return 16 * (e & 1) + 4 * (e >> 1); }

// Codes 2 i and 2 i + 1 of a word as bf16 values (c - 8) s.  A code set into the top mantissa bits of 16 is
// 16 + c; times s, less 24 s, is (c - 8) s in one exact fused step (24 s has 2 + 5 bits, the result 3 + 5).
__device__ __forceinline__ uint32_t kv4_pair(uint32_t word, int i, __nv_bfloat162 s, __nv_bfloat162 less) {
  const uint32_t at = i == 0 ? word << 3 : word >> (4 * i - 3);
  uint32_t x;   // (at & mask) | 16, as one instruction: the compiler makes two of it, a constant each
  asm("lop3.b32 %0, %1, %2, %3, 0xea;" : "=r"(x) : "r"(at), "r"(0x00780078u), "r"(0x41804180u));
  const __nv_bfloat162 y = __hfma2(*reinterpret_cast<const __nv_bfloat162*>(&x), s, less);
  return *reinterpret_cast<const uint32_t*>(&y);
}
__device__ __forceinline__ __nv_bfloat162 kv4_less(__nv_bfloat162 s) {
  const uint32_t m24 = 0xc1c0c1c0u;   // -24
  return __hmul2(s, *reinterpret_cast<const __nv_bfloat162*>(&m24));
}
__device__ __forceinline__ __nv_bfloat162 kv4_scale2(uint32_t bits) { return *reinterpret_cast<const __nv_bfloat162*>(&bits); }

// Two scales' bits with the uncounted ones cleared, and 0 in place of one that is none (`bad` then set).
__device__ __forceinline__ uint32_t kv4_sane(uint32_t two, bool& bad) {
  two &= kKv4ScaleBits | kKv4ScaleBits << 16;
  const uint32_t wrong = __vcmpgeu2(two & 0x7fff7fffu, kKv4BadScale | kKv4BadScale << 16);
  bad |= wrong != 0u;
  return two & ~wrong;
}

}  // namespace
}  // namespace sdv
