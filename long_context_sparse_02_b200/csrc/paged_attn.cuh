// What the two kernels of dsa_paged_attn share.
#pragma once

#include <cuda_fp16.h>

#include "paged_plan.cuh"

namespace dsa {

// Two fp32 values rounded to fp16 or bf16, lo in bits 0-15.
template <bool F16>
__device__ __forceinline__ uint32_t paged_pack2(float lo, float hi) {
    if (F16) {
        const __half2 v = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&v);
    }
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&v);
}

// Two e4m3 codes (bits 0-15) to fp16 (exact).
__device__ __forceinline__ uint32_t paged_widen(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.u16.u32 t, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, t;\n\t}" : "=r"(r) : "r"(v));
    return r;
}

__device__ __forceinline__ void tma_load_3d(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t x, int32_t y,
                                            int32_t z) {
    asm volatile(
        "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
        : "memory");
}
__device__ __forceinline__ void tma_load_4d(void *dst, const CUtensorMap *map, uint64_t *bar, int32_t x, int32_t y,
                                            int32_t z, int32_t w) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
        "l"(map), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
        : "memory");
}

// Maps of the cache's keys and values: a box is one page's 64 rows of one head, up to 128 bytes wide.
bool paged_kv_maps(const dsa_kv_cache &c, int num_pages, CUtensorMap *km, CUtensorMap *vm);

// The scale of a row of the tensor-core kernel stays above 0, where the first maximum would not count as grown and the
// reference not leave -inf.  Only 8-bit caches come near it (a division by their scale, and by the row's power of two),
// whose scores are below 2^33: less than 2^-80 in octaves, and 0 either way.
constexpr float PAGED_MIN_SCALE = 1e-37f;

// The tensor-core kernel for chunks (paged_attn_tc.cu): rows of its tiles, and its launch.
int paged_attn_tc_rows(int G);
dsa_status launch_paged_attn_tc(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st);

}  // namespace dsa
