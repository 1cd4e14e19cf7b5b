// dq_device.cuh -- device helpers shared by libdq's kernels (sm_100a).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cstdint>

#include "dq_internal.h"

namespace dqi {

constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ float load_elem(const void *base, int64_t idx, int dtype) {
  if (dtype == DQ_BF16) {
    const uint16_t b = __ldg(static_cast<const uint16_t *>(base) + idx);
    return __uint_as_float(static_cast<uint32_t>(b) << 16);
  }
  return __ldg(static_cast<const float *>(base) + idx);
}

__device__ __forceinline__ void store_elem(void *base, int64_t idx, float v, int dtype) {
  if (dtype == DQ_BF16)
    static_cast<__nv_bfloat16 *>(base)[idx] = __float2bfloat16_rn(v);
  else
    static_cast<float *>(base)[idx] = v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, o));
  return v;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}

// In-warp unnormalised Walsh-Hadamard transform of a 128-vector held as
// v[k] = z[lane + 32 k], stages h = 1, 2, ..., 64 in that order with the
// butterfly (a, b) -> (a + b, a - b). Each add/sub is one IEEE fp32 op, so the
// result is identical to the sequential definition.
__device__ __forceinline__ void wht128_warp(float (&v)[4], int lane) {
#pragma unroll
  for (int h = 1; h < 32; h <<= 1) {
    const bool upper = (lane & h) != 0;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = __shfl_xor_sync(kFull, v[k], h);
      v[k] = upper ? __fsub_rn(w, v[k]) : __fadd_rn(v[k], w);
    }
  }
  {  // h = 32: pairs (k=0,k=1), (k=2,k=3)
    const float a0 = v[0], a1 = v[1], a2 = v[2], a3 = v[3];
    v[0] = __fadd_rn(a0, a1);
    v[1] = __fsub_rn(a0, a1);
    v[2] = __fadd_rn(a2, a3);
    v[3] = __fsub_rn(a2, a3);
  }
  {  // h = 64: pairs (k=0,k=2), (k=1,k=3)
    const float a0 = v[0], a1 = v[1], a2 = v[2], a3 = v[3];
    v[0] = __fadd_rn(a0, a2);
    v[2] = __fsub_rn(a0, a2);
    v[1] = __fadd_rn(a1, a3);
    v[3] = __fsub_rn(a1, a3);
  }
}

// Raises kernel Kern's dynamic shared-memory limit to at least `bytes` on
// the current device. The attribute call is made only when a larger size is
// first needed on a device, so a launch sequence that repeats (a serving
// loop, one call per layer) pays the host-side attribute call once.
template <auto Kern>
cudaError_t ensure_max_dynamic_smem(int bytes) {
  constexpr int kDevs = 64;
  static std::atomic<int> set_to[kDevs];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kDevs;
  if (cached && set_to[dev].load(std::memory_order_acquire) >= bytes) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && cached) {
    int cur = set_to[dev].load(std::memory_order_relaxed);
    while (cur < bytes && !set_to[dev].compare_exchange_weak(cur, bytes, std::memory_order_release)) {
    }
  }
  return e;
}

// Lets kernel Kern be launched in clusters of more than 8 CTAs on the current
// device; the attribute call is made once per device, as above.
template <auto Kern>
cudaError_t allow_wide_cluster() {
  constexpr int kDevs = 64;
  static std::atomic<bool> set[kDevs];
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const bool cached = dev >= 0 && dev < kDevs;
  if (cached && set[dev].load(std::memory_order_acquire)) return cudaSuccess;
  e = cudaFuncSetAttribute(Kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e == cudaSuccess && cached) set[dev].store(true, std::memory_order_release);
  return e;
}

// What a sliding window leaves of a run of blocks: the blocks that hold the
// first tokens, then, `skip` blocks further, the blocks from the window's
// first token to the last one. Visible block j is block j (j < head) or
// j + skip; n of them.
struct WindowSpan {
  int64_t head, skip, n;
  __host__ __device__ __forceinline__ int64_t block(int64_t j) const { return j < head ? j : j + skip; }
};

// The visible blocks of `blk` tokens for tokens [0, sinks) and [lo, end), with
// 0 <= lo < end (or end = 0: none). Blocks that hold both are counted once.
__host__ __device__ __forceinline__ WindowSpan window_span(int64_t lo, int64_t end, int64_t sinks, int blk) {
  WindowSpan s;
  const int64_t first = (sinks + blk - 1) / blk, w0 = lo / blk;
  s.head = first < w0 ? first : w0;
  s.skip = w0 - s.head;
  s.n = (end + blk - 1) / blk - s.skip;
  return s;
}

// fp16 levels of four symbols by byte permutes instead of look-ups in shared
// memory, whose passes bound the decoders: byte s of the 8-byte pools lo and
// hi is the low and the high byte of level s; the four symbols (bits 11..13 of
// their table entries, bit 14 is 0) make one selector. (Decode attention of
// 128 x 8K tokens: 1980 us, 2076 us with look-ups.)
struct LevelPool {
  uint32_t lo0, lo1, hi0, hi1;
};
__device__ __forceinline__ uint32_t select_bits(uint32_t a, uint32_t b, uint32_t mask) { return (a & mask) | (b & ~mask); }
__device__ __forceinline__ uint32_t symbol_selector(uint32_t e0, uint32_t e1, uint32_t e2, uint32_t e3) {
  const uint32_t ab = select_bits(e0 >> 11, e1 >> 7, 0xFu), cd = select_bits(e2 >> 3, e3 << 1, 0xF00u);
  return select_bits(ab, cd, 0xFFu);
}
__device__ __forceinline__ uint2 pool_levels(const LevelPool &t, uint32_t sel) {
  const uint32_t lo = __byte_perm(t.lo0, t.lo1, sel), hi = __byte_perm(t.hi0, t.hi1, sel);
  return make_uint2(__byte_perm(lo, hi, 0x5140), __byte_perm(lo, hi, 0x7362));
}
// The pools of the levels in bits shift .. shift + 15 of v[0..7].
__device__ __forceinline__ LevelPool level_pool(const uint32_t *v, int shift) {
  LevelPool t{0u, 0u, 0u, 0u};
#pragma unroll
  for (int s = 0; s < 4; ++s) {
    t.lo0 |= ((v[s] >> shift) & 0xFFu) << (8 * s);
    t.lo1 |= ((v[s + 4] >> shift) & 0xFFu) << (8 * s);
    t.hi0 |= ((v[s] >> (shift + 8)) & 0xFFu) << (8 * s);
    t.hi1 |= ((v[s + 4] >> (shift + 8)) & 0xFFu) << (8 * s);
  }
  return t;
}

// Sign of coordinate lane + 32 k for a KV head: bit `lane` of sign word k.
__device__ __forceinline__ float apply_sign(float v, uint32_t word, int lane) {
  return ((word >> lane) & 1u) ? -v : v;
}

}  // namespace dqi
