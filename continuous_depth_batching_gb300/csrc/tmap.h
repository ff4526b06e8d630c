// Tensor-map (TMA descriptor) encoding for the kernels' 2D tiled copies.
#pragma once

#include <cuda.h>
#include <stdint.h>

namespace cdb {

// bf16 tensor [outer][inner] with a row stride of `stride` bytes, box
// box_inner x box_outer elements, swizzle of `swizzle` bytes (0, 32, 64 or
// 128).  Descriptors are encoded once per distinct argument set and cached for
// the process; nullptr when the driver entry point is missing or the encoder
// rejects the arguments.
const CUtensorMap* tmap_bf16_2d(const void* p, uint64_t inner, uint64_t outer, uint64_t stride, uint32_t box_inner,
                                uint32_t box_outer, int swizzle);

// The same for bytes, encoded into *out on every call (nothing is cached, so
// the map never outlives the memory it was made for); false as above.
bool tmap_u8_2d(CUtensorMap* out, const void* p, uint64_t inner, uint64_t outer, uint64_t stride, uint32_t box_inner,
                uint32_t box_outer, int swizzle);

// bf16 tensor [d2][d1][d0], strides of d1 and d2 in bytes, box b0 x b1 x b2,
// 128-byte swizzle; not cached.
bool tmap_bf16_3d(CUtensorMap* out, const void* p, uint64_t d0, uint64_t d1, uint64_t d2, uint64_t stride1, uint64_t stride2,
                  uint32_t b0, uint32_t b1, uint32_t b2);

// bf16 rows of hd elements (a multiple of 64) seen as [rows / 8][hd / 64][8][64], box 2 x hd/64 x 8 x 64
// (16 rows, their 64-element slices 8 rows at a time), 128-byte swizzle; not cached.
bool tmap_bf16_octets(CUtensorMap* out, const void* p, uint64_t hd, uint64_t rows);

}  // namespace cdb
