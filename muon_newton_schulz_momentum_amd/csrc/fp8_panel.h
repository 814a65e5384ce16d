// Where the loads of an 8-bit product's 256 x 256 tiles lie in an operand (no HIP: also built for the CPU).
#pragma once

#include <cstdint>

#if defined(__HIPCC__)
#define MUON_PANEL_FN __host__ __device__ __forceinline__
#else
#define MUON_PANEL_FN inline
#endif

namespace muon {

// A tile's rows of an operand (at most 256 of ld < 2^23 bytes, kp of them codes) are one buffer, whose end keeps loads
// inside: the hardware compares a load's offset with the buffer's size.  Whether the scalar part of the offset
// takes part in that, and how where it exceeds the size, is not relied on: the row is in the vector part, so that a row
// behind the last one is past the end by itself, and the scalar part stays inside a row's codes.
struct Panel {
    // vector part: 16-byte chunk c (< 8) of the lane's row r, and the rows that an instruction is further on
    static MUON_PANEL_FN int32_t lane(int32_t r, int32_t c, int32_t ld) { return r * ld + 16 * c; }
    static MUON_PANEL_FN int32_t rows(int32_t r, int32_t ld) { return r * ld; }
    // scalar part: block of 128 codes number kb
    static MUON_PANEL_FN int32_t block(int32_t kb) { return 128 * kb; }
    // size of the buffer of `rows` rows
    static MUON_PANEL_FN int32_t bytes(int32_t rows, int32_t ld, int32_t kp) { return (rows - 1) * ld + kp; }
};

}  // namespace muon
