// Ranges and offsets of the buffer loads of the MXFP4 products, free of HIP types so that host code can walk
// through them.
//
// A raw buffer load reads base + voff + soff.  Whether the scalar offset counts in the range check is not
// relied on: a load that may happen has voff + soff + 16 within the rows that there are, and one that must not
// has voff past every range (kPastRange, or a row past the part's last one) and a scalar offset that is no larger than
// the part, so that it is refused whether voff is compared with the range or with what the scalar offset leaves of it.
#pragma once

#include <stdint.h>

#ifdef __HIP__
#define MX_BOTH __host__ __device__ __forceinline__
#else
#define MX_BOTH inline
#endif

namespace nvfp4 {
namespace bounds {

constexpr uint32_t kPastRange = 0x80000000u;

// A range of bytes behind an operand's first row.
struct Part {
    int64_t base;
    uint32_t bytes;
};

// Rows row0 .. row0 + rows - 1 of a tile that has `have` rows, `row_bytes` apart, of which `row_len` bytes are read;
// empty when none of them is there.  rows * row_bytes is at most 2^29.
MX_BOTH Part rows_part(int row0, int rows, int have, int row_bytes, int row_len) {
    const int left = have - row0, n = left < rows ? left : rows;
    return n > 0 ? Part{(int64_t)row0 * row_bytes, (uint32_t)((n - 1) * row_bytes + row_len)} : Part{0, 0};
}

// Scalar offset of column byte `col`: never past the part.
MX_BOTH uint32_t part_soff(uint32_t col, uint32_t bytes) { return col < bytes ? col : bytes; }

// Lane offset of byte `at` of a step that starts at column byte `col` of rows of `row_len` bytes, its row starting at
// `row_off` in the part: past every range where the row ends before it.
MX_BOTH uint32_t lane_off(uint32_t row_off, int col, int at, int row_len) {
    return col + at < row_len ? row_off + (uint32_t)at : kPastRange;
}

// The two parts of lane_off where each lane's row is its own: the offset of byte `at` of row `row` (-1: none), and that
// offset at a step whose columns start at byte `col`: past every range where the row ends before it.
MX_BOTH uint32_t row_off(int row, int row_bytes, int at) {
    return row < 0 ? kPastRange : (uint32_t)row * (uint32_t)row_bytes + (uint32_t)at;
}
MX_BOTH uint32_t step_off(uint32_t off, int col, int at, int row_len) { return col + at < row_len ? off : kPastRange; }

}  // namespace bounds
}  // namespace nvfp4
