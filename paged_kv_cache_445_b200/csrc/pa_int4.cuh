// pa_int4.cuh -- the 4-bit KV cache: its layout and its rounding.
//
// A row's head_dim values are cut into chunks of 32.  A chunk has one fp16
// scale s = fp16(max|x| / 7) and 32 codes u = 8 + round(x / s) in 1 .. 15; the
// value is (u - 8) * s.  Both roundings are to nearest even, of exact
// quotients: a binary32 division of two values of at most 11 bits lands on the
// same side of every tie as the exact quotient does.
//
// One (block, head) is a record of block_size * head_dim * 9/16 bytes: the
// rows' codes (head_dim / 2 bytes each), then the rows' scales (head_dim / 32
// fp16 each).  The order of the codes is made for the tensor-core fragments:
//  - a chunk is 8 little-endian 16-bit units; unit u holds dims u, u + 8,
//    u + 16, u + 24 in its nibbles, lowest first.  Lane 4 g + t of an ldmatrix
//    then has, in nibble j of the two halves of its register, dims 8 j + 2 t
//    and 8 j + 2 t + 1 of row g (keys), or with .trans dim 8 j + g of rows 2 t
//    and 2 t + 1 (values): in both cases an f16x2 operand register of
//    m16n8k16 without any exchange between lanes;
//  - the 16-byte chunk c of row r stands at position c ^ ((r / (8/n)) % n) of
//    its row, n = head_dim / 32: eight rows of one chunk then lie in eight
//    different 16-byte bank groups of shared memory, and a record can be copied
//    there as one run of bytes.
#pragma once

#include <cuda_fp16.h>

#include "pa_device.cuh"

namespace pa {

__host__ __device__ constexpr int int4_record_bytes(int block_size, int head_dim) {
  return block_size * head_dim * 9 / 16;
}

// Byte of chunk c of row r in a record of rows of D dims, and of its scale.
template <int D>
__host__ __device__ __forceinline__ int int4_code_offset(int r, int c) {
  constexpr int n = D / 32;
  return r * (D / 2) + ((c ^ ((r / (8 / n)) % n)) << 4);
}
template <int D>
__host__ __device__ __forceinline__ int int4_scale_offset(int block_size, int r, int c) {
  return block_size * (D / 2) + (r * (D / 32) + c) * 2;
}

}  // namespace pa
