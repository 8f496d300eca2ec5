// Pieces shared by the kernels for low-rank adapters.
#pragma once
#include "act_quant.cuh"

namespace bl {

constexpr int kTile = 128;     // tokens of a tile (lora_tile.cu)
constexpr int kTileRuns = 8;   // a tile of at most so many runs of one adapter goes to the tensor cores

// The adapter of token m, -1 for none or out of range.
__device__ __forceinline__ int adapter_of(const int32_t* adapter, int64_t m, int64_t L) {
  const int a = adapter[m];
  return a >= 0 && a < L ? a : -1;
}

template <bool XB>
__device__ __forceinline__ float load1(const void* x, int64_t i) {
  if (XB) return bf16_bits_to_f32(reinterpret_cast<const uint16_t*>(x)[i]);
  return reinterpret_cast<const float*>(x)[i];
}
template <bool XB>
__device__ __forceinline__ void store1(void* x, int64_t i, float v) {
  if (XB)
    reinterpret_cast<uint16_t*>(x)[i] = f32_to_bf16_bits_rn(v);
  else
    reinterpret_cast<float*>(x)[i] = v;
}
// Eight elements at a 16-byte aligned address.
template <bool XB>
__device__ __forceinline__ void store8(void* at, const float (&v)[8]) {
  if (XB) {
    uint32_t w[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      w[j] = uint32_t(f32_to_bf16_bits_rn(v[2 * j])) | uint32_t(f32_to_bf16_bits_rn(v[2 * j + 1])) << 16;
    *reinterpret_cast<uint4*>(at) = make_uint4(w[0], w[1], w[2], w[3]);
  } else {
    reinterpret_cast<float4*>(at)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(at)[1] = make_float4(v[4], v[5], v[6], v[7]);
  }
}

// acc + the product of eight bf16 with eight floats.
__device__ __forceinline__ float dot8(uint4 q, const float (&v)[8], float acc) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    acc = fmaf(__uint_as_float(w[j] << 16), v[2 * j], acc);
    acc = fmaf(__uint_as_float(w[j] & 0xffff0000u), v[2 * j + 1], acc);
  }
  return acc;
}

}  // namespace bl
