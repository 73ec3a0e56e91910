// Layout of packed 4-bit matrices [rows][cols] (rows % 32 == 0, cols % 64 == 0), shared by
// the kernels that write them and the products that read them.
//
// A block is 32 rows by 64 columns, 1024 bytes: entry 32 h + r (16 bytes) holds row r,
// columns 32 h .. 32 h + 31, two to a byte, the even column in the low half.  That is
// what lane 32 h + r of a wave feeds to four 32 x 32 x 16 matrix instructions, so that a
// wave's 16-byte load of a block is one contiguous kilobyte, needs no rearranging, and
// a lane's 32 values share one scale.  (Row-major, a wave would read 32 pieces of 32
// bytes.)  Blocks follow one another along the columns, then along the rows.
//
// Scales: one byte a group of 32 columns, the exponent s + 127 of 2^s (255: the group is
// NaN).  Four consecutive blocks' scales lie together, 256 bytes: byte 4 (32 h + r) + k % 4
// for block k, one dword a lane.  A row of blocks whose number is no multiple of four
// ends in unused bytes.
#pragma once

#include <stdint.h>

namespace moe {

constexpr int kFp4BlockRows = 32, kFp4BlockCols = 64, kFp4Group = 32;
constexpr int kFp4BlockBytes = 1024, kFp4ScaleBytes = 256;  // of a block; of four blocks' scales

constexpr int64_t fp4_scale_quads(int64_t cols) { return (cols + 255) / 256; }
constexpr int64_t fp4_scale_bytes(int64_t rows, int64_t cols) {
  return rows / kFp4BlockRows * fp4_scale_quads(cols) * kFp4ScaleBytes;
}

}  // namespace moe
