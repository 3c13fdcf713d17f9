// Attention of chunks of new tokens over the paged K/V cache: the same sums
// as paged_attn.cu on the fifth-generation tensor cores, for many packed rows
// a K/V head.  Tensor-bound: 4 D flops for each (query, head, key).
//
// One CTA per SM takes tiles of two row blocks ("streams") of up to 128
// packed rows (whole tokens: 128 / G of them) against units of 128 keys (two
// pages) that both streams share.  Per unit and stream: S = Q K^T into 128
// tensor-memory columns; a warpgroup turns S into the weights P (its thread r
// holds row r: no exchange between threads) and writes them over S; O += P V
// with P read from tensor memory and V, as it lies in the cache, as the
// N-major operand.  The streams run half a step apart, so that one's products
// fill the time of the other's exponentials:
//
//   tensor pipe:  ... PV0(i-1) S0(i) PV1(i-1) S1(i) PV0(i) S0(i+1) ...
//   warps 0-3:                      [softmax 0 (i)]
//   warps 4-7:        [softmax 1 (i-1)]            [softmax 1 (i)]
//
// Tensor memory is full: S0 S1 O0 O1 at 128 columns each.  The running
// maximum that the weights refer to is only moved when it has grown by more
// than 2^8 (weights stay below 2^8, their sum is fp32, and the quotient does
// not depend on the reference), so O is rarely rescaled.  fp16 weights, whose
// range is short, are lifted by 2^10 and follow the maximum within 2^5.  Rows of q come by
// tensor copies whose box is a row block; queries and scores never touch
// registers before the softmax.
//
// 4096 tokens over 32768 positions, 32 heads of 128 on 4, bf16: 1610-1690 us in
// short runs (1220-1280 TFLOP/s, 74-77% of the measured burst rate; 3650 clocks a unit
// of which the tensor pipe is busy 2048), 1920 under the power cap.  What it
// waits for is a row block's chain: scores 512 clocks, exponentials 1024 (16 a
// clock), product 512, and the reads and signals between.  An E4M3 cache: the
// wideners keep up at 2145-2190 us.
#include <cuda_fp16.h>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "paged_attn.cuh"

namespace dsa {
namespace {

constexpr int UNIT = 128;
constexpr int MMA_WARP = 8, LOAD_WARP = 10, CLEAR_WARP = 11;  // MMA_WARP + stream
constexpr int WIDEN_WARP = 12;  // 8-bit caches: a warpgroup of them

// E4M3: keys and values arrive as 8-bit codes in a ring of their own and are widened to fp16 (exactly) into the
// ring that the products read.
template <int D, bool E4M3>
struct Cfg {
    static constexpr int NH = D / 64;                 // 128-byte column blocks of a row
    static constexpr int BLOCK = 128 * 128;           // [128 rows][64 elements]
    static constexpr int TILE = NH * BLOCK;           // Q of a stream, K or V of a unit
    static constexpr int RAW = TILE / 2;              // the same in 8 bits
    static constexpr int NST = (E4M3 ? 96 : 160) * 1024 / TILE;  // ring slots (K and V alternate)
    static constexpr int NRAW = E4M3 ? 48 * 1024 / RAW : 0;
    static constexpr int SMEM = 2 * TILE + NST * TILE + NRAW * RAW + 1024;
    static constexpr uint32_t O_COL = 256;            // S0 at 0, S1 at 128, O0, O1
    static constexpr int THREADS = E4M3 ? 512 : 384;  // two softmax warpgroups, the single-warp roles, the wideners
    // registers: the roles' shares add up to what the block is launched with
    static constexpr int REG_LAUNCH = E4M3 ? 128 : 168, REG_SOFTMAX = E4M3 ? 184 : 208, REG_REST = E4M3 ? 72 : 88;
    static_assert(256 * REG_SOFTMAX + (THREADS - 256) * REG_REST == THREADS * REG_LAUNCH, "register shares");
};

__device__ __forceinline__ void mma_ts(uint32_t d_tmem, uint32_t a_tmem, uint64_t b, uint32_t id, uint32_t acc) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d_tmem),
        "r"(a_tmem), "l"(b), "r"(id), "r"(acc)
        : "memory");
}

// True in one thread of the (converged) warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

// Two fp32 values in one 64-bit register pair.
__device__ __forceinline__ uint64_t pk(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float2 upk(uint64_t v) {
    float2 r;
    asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
    return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}

// How far (in octaves) the maximum may outgrow the reference of the weights, and what the weights are lifted by: up to
// 2^15 together, so that fp16's whole steps reach 24 octaves below the largest weight and its last ones 34; unlifted
// they reached 14 and 24, and the many small weights of a long history under one large one were lost.  The lift costs
// 0.5% of a long fp16 chunk's time (4096 tokens over 32768: 1745 us, 1735 without), an octave more 2%.
template <bool F16>
constexpr float LAG = F16 ? 5.f : 8.f;
template <bool F16>
constexpr float LIFT = F16 ? 10.f : 0.f;

// A stream's rows of a tile, and the segment's units that they see ([lo, hi), of the tile's units).
struct Stream {
    int first, rows;  // of its row block: rows first .. rows - 1 are there
    int lo, hi;
    int tok0;         // the new token of its row 0 (below 0: not there)
    int p_first, p_last, key_lo, key_hi;
};
__device__ __forceinline__ Stream stream_info(const PagedAttnParams &p, const Segment &g, int st) {
    Stream s;
    const int rs = p.TM / 2, r0 = g.x.base + st * rs, past = g.s.L - g.s.n;
    const int begin = max(r0, 0), end = min(r0 + rs, g.s.n * p.G);  // packed rows (whole tokens)
    s.first = begin - r0, s.rows = end - r0;
    s.lo = s.hi = g.u_begin;
    s.tok0 = p.by_G.div(g.t * p.TM + st * rs) - p.by_G.div(g.s.shift);
    s.p_first = past + max(s.tok0, 0);
    s.p_last = past + s.tok0 + (s.rows > 0 ? p.by_G.div(s.rows) - 1 : -1);
    s.key_hi = max(s.p_last + 1, 0);
    s.key_lo = p.window ? max(s.p_first - p.window + 1, 0) : 0;
    if (s.rows > s.first && s.key_hi > s.key_lo) {
        s.lo = max(s.key_lo / UNIT - g.x.u0, g.u_begin);
        s.hi = max(min((s.key_hi + UNIT - 1) / UNIT - g.x.u0, g.u_end), s.lo);
    }
    return s;
}

// A softmax warp's place in the walk over the segments, and what it needs of the current one at its end.
struct Walk {
    Cursor cur;
    int64_t end;
    int h, whole, slot, row0, piece0, q0, tile_row0, tile_rows;
};

// 32 scores to weights 2^(c s - mc), mc being the scaled reference less the lift, rounded to the values' type and
// packed into out[0..15]; the sum of the unrounded ones.
template <bool F16>
__device__ __forceinline__ float weigh(const uint32_t *v, uint32_t *out, float c, float mc) {
    const uint64_t c2 = pk(c, c), n2 = pk(-mc, -mc);
    uint64_t sum[2] = {0, 0};
#pragma unroll
    for (int j = 0; j < 16; ++j) {
        float2 e = upk(fma2(pk(__uint_as_float(v[2 * j]), __uint_as_float(v[2 * j + 1])), c2, n2));
        e.x = ex2_approx(e.x), e.y = ex2_approx(e.y);
        sum[j & 1] = add2(sum[j & 1], pk(e.x, e.y));
        out[j] = paged_pack2<F16>(e.x, e.y);
    }
    const float2 s = upk(add2(sum[0], sum[1]));
    return s.x + s.y;
}
__device__ __forceinline__ float max32(const uint32_t *v) {
    float mx[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
        mx[q] = fmaxf(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
#pragma unroll
        for (int j = 8; j < 32; j += 8)
            mx[q] = fmaxf(fmaxf(mx[q], __uint_as_float(v[j + 2 * q])), __uint_as_float(v[j + 2 * q + 1]));
    }
    return fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
}

// 32 bytes to global memory: one store, so that no sector is written in two halves, where the address allows.
__device__ __forceinline__ void store32(void *dst, const uint32_t *w, bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(w[0]), "r"(w[1]), "r"(w[2]),
                     "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// What a warp's rows see of a unit: nothing of the chunks of 32 keys in `none`, all of those in neither mask,
// and of the others each row the keys in (lo, hi] of the unit.
struct Sight {
    uint32_t none, part;  // bit: chunk
    int hi, lo;
};
__device__ __forceinline__ Sight sight(int key0, int pos, int p_min, int p_max, int window) {
    Sight s;
    s.none = s.part = 0;
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        const int k = key0 + 32 * x;
        if (k > p_max || (window && k + 31 <= p_min - window))
            s.none |= 1u << x;
        else if (k + 31 > p_min || (window && k <= p_max - window))
            s.part |= 1u << x;
    }
    s.hi = pos - key0;
    s.lo = window ? s.hi - window : -1;
    return s;
}

// Moves the reference m to `top` if some row of the warp has outgrown it, and rescales what refers to it.
template <int D, bool F16>
__device__ __forceinline__ void move_reference(uint32_t to, float c, float top, bool first, float &m, float &l) {
    if (__any_sync(0xffffffffu, (top - m) * c > LAG<F16>)) {  // (false where both are -inf)
        const float f = ex2_approx((m - (top == -INFINITY ? 0.f : top)) * c);
        m = top;
        l *= f;
        if (!first) {
            // the scores are complete: so is the product before them, and O is still
#pragma unroll 1
            for (int j = 0; j < D; j += 16) {
                uint32_t o[16];
                tmem_ld16(to + j, o);
                tmem_wait_ld();
#pragma unroll
                for (int q = 0; q < 16; ++q) o[q] = __float_as_uint(__uint_as_float(o[q]) * f);
                tmem_st16(to + j, o);
            }
        }
    }
}

// One row's scores of a unit (tensor memory, 128 columns at ts) to weights (over them, packed) under the
// reference m, with their sum added to l.
template <int D, bool F16>
__device__ __forceinline__ void softmax_tile(uint32_t ts, uint32_t to, float c, bool first, float &m, float &l) {
    uint32_t v[128];
#pragma unroll
    for (int x = 0; x < 4; ++x) tmem_ld32(ts + 32 * x, v + 32 * x);
    tmem_wait_ld();
    const float top = fmaxf(fmaxf(max32(v), max32(v + 32)), fmaxf(max32(v + 64), max32(v + 96)));
    move_reference<D, F16>(to, c, fmaxf(top, m), first, m, l);
    const float mc = m == -INFINITY ? -LIFT<F16> : fmaf(m, c, -LIFT<F16>);
#pragma unroll
    for (int x = 0; x < 4; ++x) {
        l += weigh<F16>(v + 32 * x, v + 16 * x, c, mc);
        if (x & 1) tmem_st32(ts + 16 * (x - 1), v + 16 * (x - 1));
    }
    tmem_wait_st();
    tc_fence_before();
}

// The same where not all is seen: by chunks of 32 keys, of which those that no row of the warp sees cost
// nothing; the scores are read twice, for the maximum and for the weights.
template <int D, bool F16>
__device__ __forceinline__ void softmax_edge(uint32_t ts, uint32_t to, float c, const Sight &see, bool first, float &m,
                                             float &l) {
    uint32_t v[32];
    auto load = [&](int x) {
        tmem_ld32(ts + 32 * x, v);
        tmem_wait_ld();
        if (see.part >> x & 1) {
            // bit j: key j of the chunk is seen
            auto upto = [](int n) { return n < 0 ? 0u : n >= 31 ? ~0u : (2u << n) - 1; };
            const uint32_t seen = upto(see.hi - 32 * x) & ~upto(see.lo - 32 * x);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = seen & (1u << j) ? v[j] : 0xff800000u;
        }
    };
    float top = m;
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
        if (see.none >> x & 1) continue;
        load(x);
        top = fmaxf(top, max32(v));
    }
    move_reference<D, F16>(to, c, top, first, m, l);
    const float mc = m == -INFINITY ? -LIFT<F16> : fmaf(m, c, -LIFT<F16>);
#pragma unroll 1
    for (int x = 0; x < 4; ++x) {
        if (see.none >> x & 1) {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[j] = 0;
        } else {
            load(x);
            l += weigh<F16>(v, v, c, mc);
        }
        tmem_st16(ts + 16 * x, v);
    }
    tmem_wait_st();
    tc_fence_before();
}

// Whether a unit of the tile has positions that none of its rows sees.
__device__ __forceinline__ bool needs_clear(const Segment &g, int key0) {
    return key0 + UNIT > g.x.key_hi || key0 < g.x.key_lo;
}

// IO_F16: q and out are fp16 (else bf16); the products run in fp16 when IO_F16 or the cache is E4M3.
template <int D, bool IO_F16, bool E4M3>
__global__ void __launch_bounds__((Cfg<D, E4M3>::THREADS), 1)
    paged_attn_tc_kernel(const __grid_constant__ CUtensorMap qmap, const __grid_constant__ CUtensorMap kmap,
                         const __grid_constant__ CUtensorMap vmap, const PagedAttnParams p) {
    using C = Cfg<D, E4M3>;
    constexpr int NST = C::NST, NRAW = E4M3 ? C::NRAW : 1;
    constexpr bool F16 = IO_F16 || E4M3;         // type of the products
    constexpr bool FIT = E4M3 && !IO_F16;        // rows of q are fitted into fp16
    extern __shared__ uint8_t smem_raw[];
    uint8_t *Qs = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *ring = Qs + 2 * C::TILE, *raw = ring + NST * C::TILE;
    __shared__ uint64_t full[NST], empty[NST], q_full[2], q_empty[2], s_full[2], p_full[2], o_full[2], v_clear[NST], drain;
    __shared__ uint32_t tmem_slot;
    __shared__ uint64_t raw_full[NRAW], raw_empty[NRAW], q_fit[2];
    __shared__ float row_scale[FIT ? 2 : 1][2][FIT ? 128 : 1];  // by segment in turn, stream, row: what fitting took out
    __shared__ Walk walk[8];
    __shared__ int abort_flag;
    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        // (an E4M3 cache: filled by the four widening warps, which clear values too)
        for (int s = 0; s < NST; ++s)
            mbar_init(&full[s], E4M3 ? 4 : 1), mbar_init(&empty[s], E4M3 ? 2 : 3), mbar_init(&v_clear[s], 1);
        for (int s = 0; s < NRAW; ++s) mbar_init(&raw_full[s], 1), mbar_init(&raw_empty[s], 4);
        for (int s = 0; s < 2; ++s) {
            mbar_init(&q_full[s], 1), mbar_init(&q_empty[s], 1), mbar_init(&q_fit[s], 4);
            mbar_init(&s_full[s], 1), mbar_init(&p_full[s], 4), mbar_init(&o_full[s], 1);
        }
        mbar_init(&drain, 2);
        abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&qmap), tma_prefetch_desc(&kmap), tma_prefetch_desc(&vmap);
        p.rec[blockIdx.x].valid = 0;
    }
    if (warp == MMA_WARP) tmem_alloc(&tmem_slot, 512);
    pdl_trigger();
    PlanShared &plan = *reinterpret_cast<PlanShared *>(ring);  // before the ring's first use
    Cursor cur = plan_cta<UNIT>(p, blockIdx.x, gridDim.x, plan);
    fence_proxy_async_smem();  // the plan's stores before the copies into the same memory
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = __shfl_sync(0xffffffffu, tmem_slot, 0);
    Segment g;

    if (warp >= 8) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::REG_REST));
        if (warp == LOAD_WARP) {
            // ---- producer ----
            uint32_t it = 0, qn[2] = {0, 0};  // ring slots used, loads of each stream's Q
            bool ok = true;
            constexpr int N = E4M3 ? NRAW : NST;
            uint64_t *const filled = E4M3 ? raw_full : full, *const freed = E4M3 ? raw_empty : empty;
            auto load_tile = [&](const CUtensorMap *map, int h, int pg0, int pg1) {  // one K or V tile
                const uint32_t slot = it % N;
                if (ok && it >= N) ok = mbar_wait(&freed[slot], ((it / N) - 1) & 1, p.err, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) return;
                if (lane == 0) {
                    uint64_t *bar = &filled[slot];
                    if (E4M3) {
                        uint8_t *dst = raw + slot * C::RAW;
                        mbar_expect_tx(bar, C::RAW);
                        tma_load_4d(dst, map, bar, 0, 0, h, pg0);
                        tma_load_4d(dst + C::RAW / 2, map, bar, 0, 0, h, pg1);
                    } else {
                        uint8_t *dst = ring + slot * C::TILE;
                        mbar_expect_tx(bar, C::TILE);
#pragma unroll
                        for (int x = 0; x < C::NH; ++x) {
                            tma_load_4d(dst + x * C::BLOCK, map, bar, x * 64, 0, h, pg0);
                            tma_load_4d(dst + x * C::BLOCK + C::BLOCK / 2, map, bar, x * 64, 0, h, pg1);
                        }
                    }
                }
                __syncwarp();
                ++it;
            };
            while (ok && next_segment<UNIT>(p, cur, g)) {
                const int hi_page = (g.x.key_hi + 63) / 64;
                for (int u = g.u_begin; ok && u < g.u_end; u += 16) {
                    int page = p.pg.num_pages;  // outside the map: reads as zeros
                    const int lp = (g.x.u0 + u) * 2 + lane;
                    // (the first unit's first page may lie before the window: not looked at)
                    if (u + lane / 2 < g.u_end && lp < hi_page && lp >= g.x.key_lo / 64) {
                        const int id = lp < p.pg.max_blocks ? p.pg.block_table[(int64_t)g.b * p.pg.max_blocks + lp] : -1;
                        if (id >= 0 && id < p.pg.num_pages)
                            page = id;
                        else
                            record_error(p.err, DSA_DEVERR_PAGE);
                    }
                    const int cnt = min(16, g.u_end - u);
                    for (int i = 0; ok && i < cnt; ++i) {
                        const int pg0 = __shfl_sync(0xffffffffu, page, 2 * i);
                        const int pg1 = __shfl_sync(0xffffffffu, page, 2 * i + 1);
                        load_tile(&kmap, g.h, pg0, pg1);
                        if (ok && u + i == g.u_begin) {
                            // the streams' Q behind the first keys, which need not wait for the last segment's end
                            for (int st = 0; ok && st < 2; ++st) {
                                const Stream s = stream_info(p, g, st);
                                if (s.lo >= s.hi) continue;
                                if (qn[st]) ok = mbar_wait(&q_empty[st], (qn[st] - 1) & 1, p.err, &abort_flag);
                                ok = __all_sync(0xffffffffu, ok);
                                if (!ok) break;
                                if (lane == 0) {
                                    const int tok = g.s.q0 + s.tok0;  // (below 0: zeros)
                                    mbar_expect_tx(&q_full[st], (p.TM / 2) * 128 * C::NH);
#pragma unroll
                                    for (int x = 0; x < C::NH; ++x)
                                        tma_load_3d(Qs + st * C::TILE + x * C::BLOCK, &qmap, &q_full[st], x * 64, g.h * p.G,
                                                    tok);
                                }
                                __syncwarp();
                                ++qn[st];
                            }
                        }
                        if (ok) load_tile(&vmap, g.h, pg0, pg1);
                    }
                }
            }
            // an abandoned run: copies in flight end before the block's shared memory does
            if (!ok) {
                for (uint32_t j = it > N ? it - N : 0; j < it; ++j) mbar_wait(&filled[j % N], (j / N) & 1, p.err, nullptr);
                for (int st = 0; st < 2; ++st)
                    if (qn[st]) mbar_wait(&q_full[st], (qn[st] - 1) & 1, p.err, nullptr);
            }
        } else if (warp < MMA_WARP + 2) {
            // ---- matrix products: one thread.  What it does between two products is seen by the tensor pipe (its
            // queue is short), so it does little: descriptors differ in their start address alone (16-byte units
            // in the low bits), ring positions are counted along, and other warps clear values or widen codes. ----
            if (elect_one()) {
                constexpr uint32_t FMT = F16 ? 0 : 1;
                constexpr uint32_t ID_S = idesc(FMT, FMT, 0, 0, UNIT, 128);
                constexpr uint32_t ID_PV = idesc(FMT, FMT, 0, 1, D, 128);
                const uint64_t dq = sdesc(smem_u32(Qs), 16, 1024, SWZ_128B), dk = sdesc(smem_u32(ring), 16, 1024, SWZ_128B),
                               dv = sdesc(smem_u32(ring), C::BLOCK, 1024, SWZ_128B);
                const int st = warp - MMA_WARP;
                const uint32_t ta = tmem + st * 128, oa = tmem + C::O_COL + st * 128;
                const uint64_t dqs = dq + (st * C::TILE >> 4);
                int slot = 0, vslot = 0;  // ring positions of K(i) and V(i-1), and the parity of their use
                uint32_t par = 0, vpar = 0, qpar = 0, ppar = 0, cpar = 0;
                bool ok = true;
                auto wait = [&](uint64_t *bar, uint32_t parity) { return ok = mbar_wait(bar, parity, p.err, &abort_flag); };
                auto advance = [&] {
                    if (++slot == NST) slot = 0, par ^= 1;
                };
                while (ok && next_segment<UNIT>(p, cur, g)) {
                    const Stream s = stream_info(p, g, st);
                    const int key_u0 = g.x.u0 * UNIT;
                    for (int i = g.u_begin; i <= g.u_end; ++i) {
                        const bool has_s = i < g.u_end, has_pv = i > g.u_begin;
                        const int kslot = slot;
                        if (has_s) {
                            if (!wait(&full[kslot], par)) break;
                            advance();
                        }
                        if (has_pv) {
                            if (!wait(&full[vslot], vpar)) break;
                            const int key0 = key_u0 + (i - 1) * UNIT;
                            if (!E4M3 && needs_clear(g, key0)) {
                                // (a barrier a slot: the clearing warp may be two cleared units ahead)
                                if (!wait(&v_clear[vslot], (cpar >> vslot) & 1)) break;
                                cpar ^= 1u << vslot;
                            }
                            if (i - 1 >= s.lo && i - 1 < s.hi) {
                                const uint64_t vd = dv + vslot * (C::TILE >> 4);
                                if (!wait(&p_full[st], ppar)) break;
                                ppar ^= 1;
                                tc_fence_after();
                                mma_ts(oa, ta, vd, ID_PV, i - 1 > s.lo);
#pragma unroll
                                for (int k = 1; k < UNIT / 16; ++k) mma_ts(oa, ta + k * 8, vd + (2048 >> 4) * k, ID_PV, 1);
                                if (i == s.hi) mma_commit(&o_full[st]);
                            }
                        }
                        if (has_s && i >= s.lo && i < s.hi) {
                            const uint64_t kd = dk + kslot * (C::TILE >> 4);
                            if (i == s.lo) {
                                if (!wait(FIT ? &q_fit[st] : &q_full[st], qpar)) break;
                                qpar ^= 1;
                            }
#pragma unroll
                            for (int k = 0; k < D / 16; ++k) {
                                const uint32_t o = (k >> 2) * C::BLOCK + (k & 3) * 32;
                                mma_bf16(ta, dqs + (o >> 4), kd + (o >> 4), ID_S, k > 0);
                            }
                            mma_commit(&s_full[st]);
                            if (i + 1 == s.hi) mma_commit(&q_empty[st]);
                        }
                        if (has_pv) mma_commit(&empty[vslot]);
                        if (has_s) {
                            mma_commit(&empty[kslot]);
                            vslot = slot, vpar = par;  // V(i) follows K(i)
                            advance();
                        }
                    }
                }
                // products in flight end before tensor and shared memory are given back
                mma_commit(&drain);
                mbar_wait(&drain, 0, p.err, nullptr);
            }
            __syncwarp();
        } else if (E4M3 && warp >= WIDEN_WARP) {
            // ---- 8-bit tiles to fp16, and rows of q fitted into it ----
            const int x = threadIdx.x - WIDEN_WARP * 32;  // 0 .. 127
            uint32_t it = 0, qn[2] = {0, 0};              // tiles; loads of each stream's Q
            bool ok = true;
            auto wait = [&](uint64_t *bar, uint32_t parity) {
                ok = ok && mbar_wait(bar, parity, p.err, &abort_flag);
                return ok = __all_sync(0xffffffffu, ok);
            };
            auto widen_tile = [&](int key0, bool clear) {
                const uint32_t from = it % NRAW, to = it % NST;
                if (!wait(&raw_full[from], (it / NRAW) & 1)) return;
                if (it >= NST && !wait(&empty[to], ((it / NST) - 1) & 1)) return;
                const uint8_t *src = raw + from * C::RAW;
                uint8_t *dst = ring + to * C::TILE;
                constexpr int CH = D / 16;  // 16-byte chunks of a row's codes
#pragma unroll 4
                for (int i = x; i < 128 * CH; i += 128) {
                    const int row = i / CH, ch = i % CH;
                    const uint32_t at = CH == 8 ? row * 128 + ((ch ^ (row & 7)) << 4) : row * 64 + ((ch ^ ((row >> 1) & 3)) << 4);
                    uint4 v = *reinterpret_cast<const uint4 *>(src + at);
                    // (values at positions that no row of the tile sees may be anything: zeros instead)
                    if (clear && (key0 + row < g.x.key_lo || key0 + row >= g.x.key_hi)) v = make_uint4(0, 0, 0, 0);
                    uint8_t *out = dst + (ch >> 2) * C::BLOCK + row * 128;
                    const int c0 = (ch & 3) * 2, sw = row & 7;
                    *reinterpret_cast<uint4 *>(out + ((c0 ^ sw) << 4)) =
                        make_uint4(paged_widen(v.x), paged_widen(v.x >> 16), paged_widen(v.y), paged_widen(v.y >> 16));
                    *reinterpret_cast<uint4 *>(out + (((c0 + 1) ^ sw) << 4)) =
                        make_uint4(paged_widen(v.z), paged_widen(v.z >> 16), paged_widen(v.w), paged_widen(v.w >> 16));
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(&raw_empty[from]), mbar_arrive(&full[to]);
                ++it;
            };
            while (ok && next_segment<UNIT>(p, cur, g)) {
                if (FIT) {
                    for (int st = 0; ok && st < 2; ++st) {
                        const Stream s = stream_info(p, g, st);
                        if (s.lo >= s.hi) continue;
                        if (!wait(&q_full[st], qn[st] & 1)) break;
                        // this thread's row times 2^-e, 2^e <= max |q| < 2^(e+1): what fp16 loses lies 2^-24 below
                        // the row's largest element (rows past the stream's hold nothing of use)
                        uint8_t *row = Qs + st * C::TILE + x * 128;
                        float mx = 0.f;
#pragma unroll 2
                        for (int i = 0; i < D / 8; ++i) {
                            const uint4 v = *reinterpret_cast<const uint4 *>(row + (i >> 3) * C::BLOCK + (i & 7) * 16);
                            const uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                mx = fmaxf(mx, fmaxf(fabsf(__uint_as_float(q[j] << 16)), fabsf(__uint_as_float(q[j] & 0xFFFF0000u))));
                        }
                        int e = (int)(__float_as_uint(mx) >> 23) - 127;
                        e = mx > 0.f ? max(-126, min(e, 126)) : 0;
                        const float down = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 2
                        for (int i = 0; i < D / 8; ++i) {
                            uint4 *at = reinterpret_cast<uint4 *>(row + (i >> 3) * C::BLOCK + (i & 7) * 16);
                            const uint4 v = *at;
                            uint32_t q[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                            for (int j = 0; j < 4; ++j)
                                q[j] = paged_pack2<true>(__uint_as_float(q[j] << 16) * down,
                                                         __uint_as_float(q[j] & 0xFFFF0000u) * down);
                            *at = make_uint4(q[0], q[1], q[2], q[3]);
                        }
                        row_scale[FIT ? qn[st] & 1 : 0][st][FIT ? x : 0] = __uint_as_float((uint32_t)(127 + e) << 23);
                        ++qn[st];
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&q_fit[st]);
                    }
                }
                for (int i = g.u_begin; ok && i < g.u_end; ++i) {
                    const int key0 = (g.x.u0 + i) * UNIT;
                    widen_tile(key0, false);
                    if (ok) widen_tile(key0, needs_clear(g, key0));
                }
            }
        } else if (!E4M3 && warp == CLEAR_WARP) {
            // ---- values at positions that no row of the tile sees may be anything (unwritten rows, other
            // sequences'): weights of 0 do not silence a NaN, so they are set to zero before their product ----
            int slot = 0;
            uint32_t par = 0;
            bool ok = true;
            auto next = [&] {  // every position is waited for and released: its parity tells one use from the next
                ok = ok && mbar_wait(&full[slot], par, p.err, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                return ok;
            };
            auto release = [&] {
                __syncwarp();
                if (lane == 0) mbar_arrive(&empty[slot]);
                if (++slot == NST) slot = 0, par ^= 1;
            };
            while (ok && next_segment<UNIT>(p, cur, g)) {
                for (int i = g.u_begin; i < g.u_end; ++i) {
                    if (!next()) break;
                    release();  // keys
                    if (!next()) break;
                    const int key0 = (g.x.u0 + i) * UNIT;
                    if (needs_clear(g, key0)) {
                        uint8_t *v = ring + slot * C::TILE;
                        for (int x = lane; x < C::TILE / 16; x += 32) {
                            const int key = key0 + ((x >> 3) & 127);
                            if (key < g.x.key_lo || key >= g.x.key_hi)
                                *reinterpret_cast<uint4 *>(v + x * 16) = make_uint4(0, 0, 0, 0);
                        }
                        fence_proxy_async_smem();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&v_clear[slot]);
                    }
                    release();
                }
            }
        }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::REG_SOFTMAX));
        // ---- softmax and output of stream st: thread r holds row r ----
        const int st = warp >> 2, r = threadIdx.x & 127;
        const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's quarter: lane 32 x (warp % 4), bits 16 up
        const uint32_t ts = tmem + lanes + st * 128, to = tmem + lanes + C::O_COL + st * 128;
        float c = p.scale_log2;
        uint32_t sn = 0, on = 0;  // S tiles and outputs waited for
        bool ok = true;
        // A row of scores needs 128 registers: the walk's state waits in shared memory meanwhile.
        const int tok = p.by_G.div(r);
        Walk &wk = walk[warp];
        if (lane == 0) wk.cur = cur;
        __syncwarp();
        while (ok) {
            int i, hi, key0, pos, p_min, p_max;  // (p_min .. p_max: of the warp's rows)
            bool have;
            {
                Cursor cu = wk.cur;
                const bool more = next_segment<UNIT>(p, cu, g);
                __syncwarp();
                if (!more) break;
                const Stream s = stream_info(p, g, st);
                const int p0 = g.s.L - g.s.n + s.tok0;  // of row 0
                have = r >= s.first && r < s.rows;
                pos = have ? p0 + tok : -1;
                p_min = max(p0 + p.by_G.div(r & ~31), s.p_first), p_max = min(p0 + p.by_G.div(r | 31), s.p_last);
                i = s.lo, hi = s.hi, key0 = (g.x.u0 + s.lo) * UNIT;
                if (lane == 0) {
                    wk.cur = cu;
                    wk.end = cu.at - (g.u_end - g.u_begin) + g.x.nu;
                    wk.h = g.h, wk.q0 = g.s.q0, wk.tile_row0 = g.x.row0, wk.tile_rows = g.x.rows;
                    wk.whole = g.whole(), wk.slot = g.slot();
                    wk.row0 = g.s.q0 + s.tok0, wk.piece0 = g.x.base - g.x.row0 + st * (p.TM / 2);
                }
                __syncwarp();
            }
            const bool some = i < hi;
            // The reference that the weights refer to (raw scores), and their sum.  A row of the block that is not there
            // (nothing of the tile's, or what an earlier tile left in shared memory) has scores too; no score outgrows
            // its infinite reference, so it moves none, which a warp's rows do together, and the others' bits do not
            // depend on it.
            float m = have ? -INFINITY : INFINITY, l = 0.f;
            for (bool first = true; i < hi; ++i, key0 += UNIT, first = false) {
                ok = mbar_wait(&s_full[st], sn & 1, p.err, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++sn;
                tc_fence_after();
                // (the products that these scores come from waited for the row's fitting; `on` segments had any before)
                if (FIT && first) c = fmaxf(p.scale_log2 * row_scale[on & 1][st][FIT ? r : 0], PAGED_MIN_SCALE);
                if (key0 + UNIT - 1 <= p_min && (!p.window || key0 > p_max - p.window))
                    softmax_tile<D, F16>(ts, to, c, first, m, l);
                else
                    softmax_edge<D, F16>(ts, to, c, sight(key0, pos, p_min, p_max, p.window), first, m, l);
                __syncwarp();
                if (lane == 0) mbar_arrive(&p_full[st]);
            }
            if (!ok) break;
            if (some) {
                ok = mbar_wait(&o_full[st], on & 1, p.err, &abort_flag);
                ok = __all_sync(0xffffffffu, ok);
                if (!ok) break;
                ++on;
                tc_fence_after();
            }
            const bool whole = wk.whole;
            // (only a row that saw nothing has a sum of 0: a NaN goes on into the row's results)
            const float inv = l != 0.f ? p.v_inv / l : 0.f;
            const float ls = l != 0.f ? m * c + log2f(l) - LIFT<F16> : -INFINITY;
            const int64_t orow = (int64_t)(wk.row0 + tok) * p.H + wk.h * p.G + (r - tok * p.G);
            const int64_t piece = ((int64_t)blockIdx.x * 2 + wk.slot) * p.TM + wk.piece0 + r;
            if (have) {
                if (!whole)
                    p.part_l[piece] = ls;
                else if (p.lse)
                    p.lse[orow] = ls * 0.6931471805599453f;
            }
            uint16_t *orow_p = static_cast<uint16_t *>(p.out) + orow * D;
            const bool wide = (reinterpret_cast<uintptr_t>(p.out) & 31) == 0;
#pragma unroll 1
            for (int j = 0; j < D; j += 32) {
                uint32_t o[32];
                if (some) {
                    tmem_ld32(to + j, o);
                    tmem_wait_ld();
                }
#pragma unroll
                for (int q = 0; q < 32; ++q) o[q] = l != 0.f ? __float_as_uint(__uint_as_float(o[q]) * inv) : 0u;
                if (!have) continue;
                if (whole) {
#pragma unroll
                    for (int q = 0; q < 16; ++q)
                        o[q] = paged_pack2<IO_F16>(__uint_as_float(o[2 * q]), __uint_as_float(o[2 * q + 1]));
                    store32(orow_p + j, o, wide), store32(orow_p + j + 16, o + 8, wide);
                } else {
                    float *dst = p.part_o + piece * D + j;
#pragma unroll
                    for (int q = 0; q < 4; ++q) store32(dst + 8 * q, o + 8 * q, true);
                }
            }
            if (threadIdx.x == 0 && wk.slot == 1 && !whole)
                p.rec[blockIdx.x] = PieceRec{1, wk.q0, wk.h, wk.tile_row0, wk.tile_rows, wk.end, wk.cur.total};
            __syncwarp();  // the walk's state is read before the next segment's is written
            tc_fence_before();  // the reads of O before the next segment's first product, which waits for its weights
        }
    }
    tc_fence_before();
    __syncthreads();
    if (warp == MMA_WARP) {
        tc_fence_after();
        tmem_dealloc(tmem, 512);
    }
}

template <int D, bool IO_F16, bool E4M3>
dsa_status launch(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    using C = Cfg<D, E4M3>;
    auto fn = paged_attn_tc_kernel<D, IO_F16, E4M3>;
    // the roles' register shares draw on what the block was launched with
    static const bool regs_ok = [fn] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, fn) == cudaSuccess && fa.numRegs == C::REG_LAUNCH;
    }();
    if (!regs_ok || !ensure_smem(reinterpret_cast<const void *>(fn), C::SMEM)) return DSA_ERR_CUDA;
    CUtensorMap qm, km, vm;
    if (!paged_kv_maps(*a.cache, a.pg.num_pages, &km, &vm)) return DSA_ERR_CUDA;
    const uint64_t dims[3] = {(uint64_t)D, (uint64_t)p.H, (uint64_t)p.T};
    const uint32_t box[3] = {64, (uint32_t)p.G, (uint32_t)(p.TM / 2 / p.G)};
    const uint64_t hs = (uint64_t)(p.H > 1 ? p.q_head : D) * 2, ts = (uint64_t)(p.T > 1 ? p.q_token : D) * 2;
    if (!make_tmap_3d(&qm, p.q, IO_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, dims, hs, ts,
                      box, CU_TENSOR_MAP_SWIZZLE_128B))
        return DSA_ERR_CUDA;
    fn<<<nc, C::THREADS, C::SMEM, st>>>(qm, km, vm, p);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

template <int D>
dsa_status launch(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    const bool f16 = a.dtype == DSA_F16;
    if (a.cache->dtype == DSA_E4M3) return f16 ? launch<D, true, true>(a, p, nc, st) : launch<D, false, true>(a, p, nc, st);
    return f16 ? launch<D, true, false>(a, p, nc, st) : launch<D, false, false>(a, p, nc, st);
}

}  // namespace

int paged_attn_tc_rows(int G) { return 2 * (128 / G) * G; }

dsa_status launch_paged_attn_tc(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    return a.cache->Dk == 128 ? launch<128>(a, p, nc, st) : launch<64>(a, p, nc, st);
}

}  // namespace dsa
