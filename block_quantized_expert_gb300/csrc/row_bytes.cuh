// row_bytes.cuh -- four bytes of a row of a matrix whose rows start and end at any address.
#pragma once

#include <cstdint>

namespace moe {

// How row_bytes4 reads; a test puts a record in its place.
struct PlainLoads {
    __host__ __device__ static uint32_t word(const int8_t* p) { return *reinterpret_cast<const uint32_t*>(p); }
    __host__ __device__ static uint32_t byte(const int8_t* p) { return (uint8_t)*p; }
};

// Bytes [c, c + 4) of the row [row, row + K), c < K, with zeros past its end: the one or two
// aligned words that hold them, shifted together.  Nothing outside the matrix, [lo, hi), is
// read: a word that reaches over either end of it comes in single bytes.  `inside`: none does.
template <typename Loads>
__host__ __device__ __forceinline__ uint32_t row_bytes4(const int8_t* row, int c, int K, bool inside, const int8_t* lo,
                                                        const int8_t* hi) {
    const int8_t* p = row + c;
    const int off = (int)((uintptr_t)p & 3), n = K - c;
    const bool two = off && n > 4 - off;
    if (inside || (p - off >= lo && p - off + (two ? 8 : 4) <= hi)) {
        const uint64_t low = Loads::word(p - off), high = two ? Loads::word(p - off + 4) : 0u;
        const uint32_t v = (uint32_t)((high << 32 | low) >> (8 * off));
        return n < 4 ? v & ((1u << (8 * n)) - 1u) : v;
    }
    uint32_t v = 0;
#pragma unroll 1
    for (int i = 0; i < 4 && i < n; ++i) v |= Loads::byte(p + i) << (8 * i);
    return v;
}

}  // namespace moe
