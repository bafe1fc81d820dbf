// cache.cuh -- what the paged-cache kernels share: the page lookup and the
// storage types (bf16, fp32, e4m3 with one power-of-two scale per row).
#pragma once

#include <cuda_fp8.h>

#include <atomic>

#include "common.cuh"
#include "internal.h"

namespace dropkv {

struct E4M3 {  // storage only
  uint8_t bits;
};

// n / d for 0 <= n < 2^31 and 1 <= d < 2^31, by a multiplication: with
// s = ceil(log2 d) and mul = floor(2^32 (2^s - d) / d) + 1, the quotient is
// (floor(mul n / 2^32) + n) >> s (the sum stays below 2^32).
struct FastDiv {
  uint32_t mul, shift;
  static FastDiv of(uint32_t d) {
    FastDiv f;
    f.shift = 0;
    while ((1ull << f.shift) < d) ++f.shift;
    f.mul = (uint32_t)(((1ull << 32) * ((1ull << f.shift) - d)) / d + 1);
    return f;
  }
  __device__ __forceinline__ uint32_t div(uint32_t n) const {
    return (__umulhi(n, mul) + n) >> shift;
  }
};

// The pages as the kernels see them (sizes were checked on the host).
struct CacheDev {
  int32_t B, Hkv, d, n_pages, page, max_pages;
  int32_t cap;  // max_pages * page: slots a sequence can have
  FastDiv fpage;
  void* k;
  void* v;
  uint8_t* ks;
  uint8_t* vs;
  const int32_t* table;
};

// Row index of slot `slot` (0 <= slot < cap) of (b, h) in the pools
// [n_pages, Hkv, page]; -1 where the table names no page of the pools.
__device__ __forceinline__ int64_t cache_row(const CacheDev& c, int b, int h, int slot) {
  const int pi = (int)c.fpage.div((uint32_t)slot);
  const int page = __ldg(c.table + (size_t)b * c.max_pages + pi);
  if ((uint32_t)page >= (uint32_t)c.n_pages) return -1;
  return ((int64_t)page * c.Hkv + h) * c.page + (slot - pi * c.page);
}

__device__ __forceinline__ void raise_arg(int32_t* status) {
  if (status) atomicMax(status, (int)DROPKV_ERR_ARG);
}

// 2^(byte - 127): the byte is the exponent field of an fp32, except at its two
// ends, 2^-127 (a subnormal) and NaN.
__device__ __forceinline__ float scale_of(uint32_t byte) {
  const uint32_t u = byte == 0 ? 0x00400000u : byte == 255 ? 0x7FC00000u : byte << 23;
  return __uint_as_float(u);
}

// The scale byte of a row whose largest |value| has the bits `amax` (the
// bits of non-negative floats order like the floats): the least e >= -127 with
// |value| <= 448 2^e = 1.75 2^(e + 8).  255 if the row holds an inf or a NaN.
__device__ __forceinline__ uint32_t scale_byte(uint32_t amax) {
  if (amax >= 0x7F800000u) return 255u;
  const int e = (int)(amax >> 23) - 8 + ((amax & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return (uint32_t)max(e, 0);
}
// 2^(127 - byte), the factor that takes the row into [-448, 448] (byte <= 247
// for finite rows, so this is a normal fp32); NaN for 255.
__device__ __forceinline__ float inv_scale_of(uint32_t byte) {
  return __uint_as_float(byte == 255 ? 0x7FC00000u : (254u - byte) << 23);
}

// Eight values <-> storage.  The product with a power of two is exact unless
// it falls below fp32's range, far under e4m3's smallest step, so the one
// rounding is e4m3's, to nearest even; satfinite never acts on |x| <= 448.
__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {
  return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}
__device__ __forceinline__ float2 unpack_e4m3(uint32_t two) {
  const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)two, __NV_E4M3);
  return __half22float2(__half2(h));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
  return *reinterpret_cast<const uint32_t*>(&v);
}


// Two e4m3 bytes of x to a bf16 pair, times 2^-120 f: the bytes, sign-extended to
// 16 bits each, four bits up, less the copies of the sign between sign and
// exponent; so the seven magnitude bits end at the bottom of bf16's exponent and
// the top of its mantissa (subnormals land on subnormals).  Two instructions of
// the ALU pipe and two of the FMA pipe (the shift is a product there).
constexpr uint32_t kBytes01 = 0x9180u, kBytes23 = 0xB3A2u, kBytes02 = 0xA280u, kBytes13 = 0xB391u;
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
template <uint32_t kSel>
__device__ __forceinline__ uint32_t widen_e4m3x2(uint32_t x, uint32_t f) {
  uint32_t z;
  asm("prmt.b32 %0, %1, %1, %2;" : "=r"(z) : "r"(x), "n"(kSel));
  return mul_bf16x2((z << 4) & 0x87F087F0u, f);
}

__device__ __forceinline__ bool non_finite(uint32_t two) {  // of a bf16 pair
  return (two & 0x7F80u) == 0x7F80u || (two & 0x7F800000u) == 0x7F800000u;
}
__device__ __forceinline__ uint32_t without_non_finite(uint32_t two) {
  if ((two & 0x7F80u) == 0x7F80u) two &= 0xFFFF0000u;
  if ((two & 0x7F800000u) == 0x7F800000u) two &= 0x0000FFFFu;
  return two;
}

CacheDev cache_dev(const dropkv_cache& c);

// Allows `kern` `bytes` of dynamic shared memory, once per device (the bit of a
// device is set after the call that does it, so calls at once do it twice).
template <auto kern>
cudaError_t allow_smem(int bytes) {
  static std::atomic<uint64_t> done{0};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? 1ull << dev : 0;
  if (done.load(std::memory_order_acquire) & bit) return cudaSuccess;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

}  // namespace dropkv
