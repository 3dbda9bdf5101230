// row_bytes_probe.cu -- test-only host build of row_bytes.cuh whose loads record the
// addresses they touch (built and called by tests/test_row_bytes.py; needs no GPU).
#include "row_bytes.cuh"

static uint8_t* touched;       // one mark a byte of the buffer
static const int8_t* origin;

struct Recorded {
    __host__ __device__ static uint32_t word(const int8_t* p) {
#ifndef __CUDA_ARCH__
        for (int i = 0; i < 4; ++i) touched[p + i - origin] = 1;
#endif
        return moe::PlainLoads::word(p);
    }
    __host__ __device__ static uint32_t byte(const int8_t* p) {
#ifndef __CUDA_ARCH__
        touched[p - origin] = 1;
#endif
        return moe::PlainLoads::byte(p);
    }
};

extern "C" uint32_t probe_row_bytes(const int8_t* buffer, int row, int c, int K, int inside, int lo, int hi, uint8_t* marks) {
    origin = buffer;
    touched = marks;
    return moe::row_bytes4<Recorded>(buffer + row, c, K, inside != 0, buffer + lo, buffer + hi);
}
