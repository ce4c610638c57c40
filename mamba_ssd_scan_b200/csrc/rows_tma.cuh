// rows_tma.cuh -- TMA copies of boxes of a [batch][rows][channels] array:
// box1 rows of 64 channels each, dense in shared memory (no swizzle).  Rows and
// channels past the array's ends read as zero and are not written.
#pragma once

#include "tma.cuh"

namespace ssd {

// The array's map: channels innermost (a multiple of 16 bytes), fp32 or bf16.
bool make_tmap_rows(CUtensorMap* map, const void* base, bool bf16, uint64_t channels, uint64_t rows,
                    uint64_t batch, uint32_t box1);

namespace tc {

__device__ __forceinline__ void tma_load_rows(uint32_t dst, const CUtensorMap* map, uint32_t mbar, int c, int row,
                                              int b) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];"
        :
        : "r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(mbar), "r"(c), "r"(row), "r"(b)
        : "memory");
}
// (bulk async group of the issuing thread)
__device__ __forceinline__ void tma_store_rows(const CUtensorMap* map, uint32_t src, int c, int row, int b) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :
                 : "l"(reinterpret_cast<uint64_t>(map)), "r"(src), "r"(c), "r"(row), "r"(b)
                 : "memory");
}

}  // namespace tc
}  // namespace ssd
