// What the warp-level kernels of dsa_paged_attn share: the ring of units of
// keys and values that one warp fills by TMA, and the fragments that come
// out of it.
#pragma once

#include "paged_attn.cuh"

namespace dsa {

constexpr int UNIT_KEYS = 64;  // a unit: one page of one head, keys and values

// Softmax weights that are rounded to fp16 are taken as 2^(l - m + LIFT): at most 2^15 of fp16's 65504, so that fp16's
// whole steps reach 29 octaves below the largest and its last ones 39.  At most 1 they reached 14 and 24, and the many
// small weights of a long history under one large one were lost.  Their sum carries the same factor, which the quotient
// does not see and the log-sum-exp takes out.
constexpr float FP16_LIFT = 15.f;

template <int D, bool E4M3>
struct UnitRing {
    static constexpr int ELEM = E4M3 ? 1 : 2;
    static constexpr int ROW_BYTES = D * ELEM;                           // of one head
    static constexpr int BOX_BYTES = ROW_BYTES < 128 ? ROW_BYTES : 128;  // inner extent of a TMA box
    static constexpr int BOXES = ROW_BYTES / BOX_BYTES;
    static constexpr int TILE_BYTES = UNIT_KEYS * ROW_BYTES;                  // K or V of a unit
    static constexpr int STAGE = 2 * TILE_BYTES;
    // 128 KB of units, a power of two of them; of the largest ones the 160 KB that fit
    static constexpr int NST = STAGE == 32 * 1024 ? 5 : 128 * 1024 / STAGE;
};

// Byte offset of 16-byte chunk `chunk` of row `row` in a tile of one head:
// boxes of [64 rows][128 or 64 bytes], swizzled as the tensor map says.
template <int BOX_BYTES>
__device__ __forceinline__ uint32_t tile_off(int row, int chunk) {
    if (BOX_BYTES == 128)
        return (uint32_t)((chunk >> 3) * (UNIT_KEYS * 128) + row * 128 + (((chunk & 7) ^ (row & 7)) << 4));
    return (uint32_t)(row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4));
}

__device__ __forceinline__ void ldsm4(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t *r, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

template <bool F16>
__device__ __forceinline__ void mma16816(float *d, const uint32_t *a, uint32_t b0, uint32_t b1) {
    if (F16)
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
    else
        asm volatile(
            "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
            : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
            : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <bool F16>
__device__ __forceinline__ float2 unpack2(uint32_t v) {
    if (F16) return __half22float2(*reinterpret_cast<__half2 *>(&v));
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
}
// The loading warp: the CTA's segments' units into the ring, K and V of one head and page each.
template <class C>
__device__ __forceinline__ void load_units(const CUtensorMap &kmap, const CUtensorMap &vmap, const PagedAttnParams &p,
                                           Cursor cur, uint8_t *ring, uint64_t *full, uint64_t *empty, volatile int *abort) {
    const int lane = lane_id();
    Segment g;
    uint32_t it = 0;
    bool ok = true;
    while (ok && next_segment<UNIT_KEYS>(p, cur, g)) {
        const int hi_unit = (g.x.key_hi + UNIT_KEYS - 1) / UNIT_KEYS;
        for (int u = g.u_begin; ok && u < g.u_end; u += 32) {
            // page ids of the next 32 units, one a lane
            int page = p.pg.num_pages;  // outside the map: reads as zeros
            const int lp = g.x.u0 + u + lane;
            if (u + lane < g.u_end && lp < hi_unit) {
                const int id = lp < p.pg.max_blocks ? p.pg.block_table[(int64_t)g.b * p.pg.max_blocks + lp] : -1;
                if (id >= 0 && id < p.pg.num_pages)
                    page = id;
                else
                    record_error(p.err, DSA_DEVERR_PAGE);
            }
            const int cnt = min(32, g.u_end - u);
            for (int i = 0; i < cnt; ++i, ++it) {
                const int pg = __shfl_sync(0xffffffffu, page, i);
                const int s = it % C::NST;
                if (it >= C::NST) ok = mbar_wait(&empty[s], ((it / C::NST) - 1) & 1, p.err, abort);
                if (!__all_sync(0xffffffffu, ok)) {
                    ok = false;
                    break;
                }
                if (lane == 0) {
                    uint8_t *st = ring + s * C::STAGE;
                    mbar_expect_tx(&full[s], C::STAGE);
#pragma unroll
                    for (int x = 0; x < C::BOXES; ++x) {
                        const int col = x * (C::BOX_BYTES / C::ELEM);
                        tma_load_4d(st + x * UNIT_KEYS * C::BOX_BYTES, &kmap, &full[s], col, 0, g.h, pg);
                        tma_load_4d(st + C::TILE_BYTES + x * UNIT_KEYS * C::BOX_BYTES, &vmap, &full[s], col, 0, g.h, pg);
                    }
                }
                __syncwarp();
            }
        }
    }
    // copies in flight end before the block's shared memory does (after an abandoned run; otherwise the
    // consumers have waited for them all)
    if (!ok)
        for (uint32_t j = it > C::NST ? it - C::NST : 0; j < it; ++j)
            mbar_wait(&full[j % C::NST], (j / C::NST) & 1, p.err, nullptr);
}

// The kernel for up to eight packed rows over an 8-bit cache (paged_attn8.cu); p.TM == 8.
dsa_status launch_paged_attn8(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st);

}  // namespace dsa
