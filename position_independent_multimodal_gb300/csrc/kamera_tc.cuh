// What the tcgen05 attention kernels share: the ring's places, operand descriptors, tensor maps.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace kamera {

constexpr int kChunk = 128 * 128;  // bytes of a 128 x 64 bf16 operand tile

template <int V>
struct Int {
  static constexpr int v = V;
};

// A place in the ring of N stages and the parity of its phase.
template <int N>
struct Place {
  uint32_t st = 0, ph = 0;
  __device__ __forceinline__ void advance(int n) {
    st += n;
    while (st >= (uint32_t)N) {
      st -= N;
      ph ^= 1;
    }
  }
};

// Halves of the matrix descriptors of 128-byte swizzled operands, whose eight rows of 128 bytes
// make a group of 1024 bytes (the stride offset): the start address and leading offset, to which the
// steps inside a tile are added, and the constant rest. MN-major, 64 elements along M or N make a
// row, and the leading offset is that of the next 64.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_k(uint32_t addr) { return (addr >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t desc_mn(uint32_t addr) {
  return (addr >> 4) | (uint32_t)(kChunk >> 4) << 16;
}
__device__ __forceinline__ uint64_t desc(uint32_t lo) {
  return (uint64_t)kDescHi << 32 | lo;
}

typedef CUresult (*EncodeFn)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                             const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                             const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                             CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

inline EncodeFn encode_fn() {
  static const EncodeFn fn = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult found;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault,
                                         &found) != cudaSuccess ||
        found != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<EncodeFn>(p);
  }();
  return fn;
}

// bf16 [n2][n1][n0] (row strides in elements), boxes of 64 x b1 x b2, 128-byte swizzle.
inline bool encode(CUtensorMap *m, const void *base, int rank, uint64_t n0, uint64_t n1,
                   uint64_t n2, uint64_t s1, uint64_t s2, uint32_t b1, uint32_t b2) {
  const cuuint64_t dims[3] = {n0, n1, n2}, strides[2] = {2 * s1, 2 * s2};
  const cuuint32_t box[3] = {64, b1, b2}, step[3] = {1, 1, 1};
  return encode_fn()(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void *>(base), dims,
                     strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
                     CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace kamera
