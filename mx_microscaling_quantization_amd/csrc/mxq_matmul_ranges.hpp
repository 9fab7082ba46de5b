// mxq_matmul_ranges.hpp -- lengths of the buffers through which the products
// read an operand from a column of its own on. Plain arithmetic, the same on
// the device and on the host.
#pragma once

#include <stdint.h>

namespace mxq {

// Bytes from container c0 of the first of `rows` operand rows (4 bytes a
// container, C containers a row) to the end of the last. A tile's last waves
// may start past the operand's last column: nothing is theirs to read, and an
// unsigned difference would be a range of 4 GiB.
constexpr uint32_t operand_range(uint32_t rows, uint32_t C, uint32_t c0)
{
    return c0 < C && rows > 0u ? rows * (4u * C) - 4u * c0 : 0u;
}

// The same for scale rows (one byte a container).
constexpr uint32_t scale_range(uint32_t rows, uint32_t C, uint32_t c0)
{
    return c0 < C && rows > 0u ? rows * C - c0 : 0u;
}

} // namespace mxq
