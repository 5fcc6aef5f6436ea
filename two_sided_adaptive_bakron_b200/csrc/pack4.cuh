// pack4.cuh -- sizes of the 4-bit layout (described at bakron_pack4 in bakron.h).
#pragma once

#include "lowp.cuh"

namespace bakron {

struct Pack4Shape {
    int mt, kt, groups;   // row tiles of 16, column tiles of 64, grid steps per row
    __host__ __device__ Pack4Shape(int m, int n, int G)
        : mt((int)(((unsigned)m + 15) / 16)), kt((n + 63) / 64), groups(G) {}
    __host__ __device__ size_t tiles() const { return (size_t)mt * kt; }
    __host__ __device__ size_t code_bytes() const { return tiles() * 512; }
    __host__ __device__ size_t step_count() const { return (size_t)mt * groups * 16; }
    __host__ __device__ size_t bytes() const { return code_bytes() + step_count() * 4; }
};

inline bool pack4_ok(int m, int n, int group_size) {
    return m >= 1 && n >= 1 && n <= 65536 && (long long)m * n < (1LL << 31) &&
           group_ok(group_size, n);
}

}  // namespace bakron
