// Attention of each sequence's newest tokens over its paged K/V cache, for
// few packed rows a K/V head (single tokens, drafts) and, as 128-row tiles,
// for any number: warp-level matrix instructions, one pass over the keys with
// the running maximum and sum of each row.
//
//   l_s = c q.k_s,  m = max l,  p_s = 2^(l_s - m),  out = sum p_s v_s / sum p_s
// with c = sm_scale log2(e), statistics and sums in fp32.
//
// With few rows the bound is HBM: a K/V head's keys and values are read once
// for all its query heads (rows are packed: see paged_plan.cuh).  One CTA per
// SM: a producer warp keeps a ring of units (64 positions = one page, K and V)
// full by TMA, 128 KB in flight per SM (160 KB of 2-byte caches of 128-wide heads); eight consumer warps take slices of 32
// or 16 keys in turn, each with the running statistics and the output of its
// 16 rows in registers, and join at the end of a tile in a fixed order.  Keys
// and values go from swizzled shared memory to the fragments by ldmatrix; an
// 8-bit cache is widened to fp16 (exact) in registers, one conversion for two
// values, and bf16 rows of q are scaled by a power of two into fp16, which loses
// what lies 2^-24 below a row's largest element.
//
// Measured: 64 sequences of 4096-65536 positions, one token each, 64 heads of
// 128 on 8, bf16: 1230 us in short runs, 1262 in long ones, for 8.95 GB (above
// the measured copy rate, which has writes in it); four drafts of 8 sequences of
// 131072 positions 610 and 750 us; one token over 4097 positions 15 us.
#include <cuda_fp16.h>

#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "paged_units.cuh"

namespace dsa {
namespace {

constexpr int UNIT = UNIT_KEYS;
constexpr int CW = 8;  // consumer warps
constexpr int THREADS = (CW + 4) * 32;  // and a warpgroup of which one warp loads
// registers: 384 x 168 at launch; the roles' shares add up to the same
constexpr int REG_LAUNCH = 168, REG_CONSUME = 216, REG_LOAD = 72;
static_assert(CW * 32 * REG_CONSUME + 128 * REG_LOAD == THREADS * REG_LAUNCH, "register shares");
constexpr int MERGE_LD = 4;  // floats of padding per merged row

template <int D, bool E4M3>
struct Cfg : UnitRing<D, E4M3> {
    static constexpr int MERGE_ROW = D + MERGE_LD;
    static constexpr int MERGE_BYTES = (CW / 2) * 16 * (MERGE_ROW + 2) * 4;
    static constexpr int SMEM = Cfg::NST * Cfg::STAGE + MERGE_BYTES + 1024;
};

template <bool B>
struct Bool {
    static constexpr bool value = B;
};

// MT = TM / 16 row groups of 16; the consumer warps are MT row groups x CW/MT
// key slots.  A unit has 64 / KW slices of KW keys; where a row group has more
// slots than that, they take turns unit by unit.
// IO_F16: q and out are fp16 (else bf16).  The matrix products run in fp16
// when IO_F16 or the cache is E4M3.
template <int D, bool IO_F16, bool E4M3, int KW>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const PagedAttnParams p, const int MT) {
    using C = Cfg<D, E4M3>;
    constexpr bool MM_F16 = IO_F16 || E4M3;
    constexpr float LIFT = MM_F16 ? FP16_LIFT : 0.f;
    constexpr int KS = D / 16;  // k-steps of q.k; also pairs of 8-wide output tiles
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(ring + C::NST * C::STAGE);
    __shared__ PlanShared plan;
    __shared__ uint64_t full[C::NST], empty[C::NST];
    __shared__ int abort_flag;
    const int warp = warp_id(), lane = lane_id();
    constexpr int SPU = UNIT / KW, NT = KW / 8;  // slices of a unit, 8-key tiles of a slice
    const int nslot = CW / MT;
    const int turns = nslot > SPU ? nslot / SPU : 1;  // units in turn (a power of two)
    // Where the ring holds a multiple of them, a stage always belongs to the same slots, and the others pass it by.
    // Else every warp waits for and releases every unit: one that skipped a stage's phase could not tell the one
    // after next by its parity.
    const bool own = C::NST % turns == 0;
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], own ? CW / turns : CW);
        }
        abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        p.rec[blockIdx.x].valid = 0;
    }
    pdl_trigger();
    Cursor cur = plan_cta<UNIT>(p, blockIdx.x, gridDim.x, plan);  // also orders the barrier setup before its use
    Segment g;

    if (warp >= CW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOAD));
        if (warp != CW) return;
        load_units<C>(kmap, vmap, p, cur, ring, full, empty, &abort_flag);
        return;
    }

    // ---- consumers ----
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_CONSUME));
    const int rg = warp % MT, slot = warp / MT;
    const int gid = lane >> 2, tig = lane & 3;
    uint32_t it = 0;
    while (next_segment<UNIT>(p, cur, g)) {
        const int rbase = g.x.row0 + rg * 16;
        const int last_row = g.x.row0 + g.x.rows;
        // this thread's two rows: gid and gid + 8 of the group
        int pos[2];
        float c[2];
        uint32_t qf[KS][4];
        bool have[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = rbase + gid + 8 * r;
            have[r] = row < last_row;
            const int tok = p.by_G.div(row), hg = row - tok * p.G;
            pos[r] = have[r] ? g.s.L - g.s.n + tok : -1;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (int64_t)(g.s.q0 + tok) * p.q_token +
                                  (int64_t)(g.h * p.G + hg) * p.q_head;
            c[r] = p.scale_log2;
            if (!E4M3) {
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    qf[k][r] = have[r] ? *reinterpret_cast<const uint32_t *>(src + k * 16 + tig * 2) : 0;
                    qf[k][2 + r] = have[r] ? *reinterpret_cast<const uint32_t *>(src + k * 16 + 8 + tig * 2) : 0;
                }
            } else {
                // an 8-bit key fragment holds four consecutive elements a thread: q takes the same order
                float mx = 0.f;
#pragma unroll
                for (int k = 0; k < KS; ++k) {
                    const uint2 v = have[r] ? *reinterpret_cast<const uint2 *>(src + k * 16 + tig * 4) : make_uint2(0, 0);
                    qf[k][r] = v.x, qf[k][2 + r] = v.y;
                    const float2 a = unpack2<IO_F16>(v.x), b = unpack2<IO_F16>(v.y);
                    mx = fmaxf(fmaxf(mx, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
                }
                if (!IO_F16) {
                    // bf16 to fp16: times 2^-e with 2^e <= max|q| < 2^(e+1), so that the row fits; what
                    // is lost lies 2^-24 below the row's largest element
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                    int e = (int)(__float_as_uint(mx) >> 23) - 127;
                    e = mx > 0.f ? max(-126, min(e, 126)) : 0;
                    const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                    c[r] *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                    for (int k = 0; k < KS; ++k) {
#pragma unroll
                        for (int x = 0; x < 2; ++x) {
                            const float2 a = unpack2<false>(qf[k][r + 2 * x]);
                            qf[k][r + 2 * x] = paged_pack2<true>(a.x * down, a.y * down);
                        }
                    }
                }
            }
        }
        float o[2 * KS][4];
#pragma unroll
        for (int i = 0; i < 2 * KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
        float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

        auto slice = [&](const uint8_t *st, int key0, int sl) {
            const uint32_t kb = smem_u32(st), vb = kb + C::TILE_BYTES;
            float s[NT][4];
#pragma unroll
            for (int i = 0; i < NT; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
            if (!E4M3) {
                const int row = sl * KW + ((lane >> 4) << 3) + (lane & 7), ch = (lane >> 3) & 1;
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int i = 0; i < NT; i += 2) {
                        uint32_t b[4];
                        ldsm4(b, kb + tile_off<C::BOX_BYTES>(row + i * 8, 2 * k + ch));
                        mma16816<MM_F16>(s[i], qf[k], b[0], b[1]);
                        mma16816<MM_F16>(s[i + 1], qf[k], b[2], b[3]);
                    }
            } else {
                const int row = sl * KW + (((lane >> 3) & 1) << 3) + (lane & 7), ch = lane >> 4;
#pragma unroll
                for (int k = 0; k < KS; k += 2)
#pragma unroll
                    for (int i = 0; i < NT; i += 2) {
                        uint32_t b[4];
                        ldsm4(b, kb + tile_off<C::BOX_BYTES>(row + i * 8, k + ch));
                        mma16816<true>(s[i], qf[k], paged_widen(b[0]), paged_widen(b[0] >> 16));
                        mma16816<true>(s[i + 1], qf[k], paged_widen(b[1]), paged_widen(b[1] >> 16));
                        mma16816<true>(s[i], qf[k + 1], paged_widen(b[2]), paged_widen(b[2] >> 16));
                        mma16816<true>(s[i + 1], qf[k + 1], paged_widen(b[3]), paged_widen(b[3] >> 16));
                    }
            }
            // scores in log2 units; masked where a row does not see the key
            const bool edge = key0 + KW - 1 > g.x.p_first || (p.window && key0 <= g.x.p_last - p.window);
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] *= c[e >> 1];
            if (edge) {
#pragma unroll
                for (int i = 0; i < NT; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + i * 8 + tig * 2 + (e & 1), r = e >> 1;
                        if (key > pos[r] || (p.window && key <= pos[r] - p.window)) s[i][e] = -INFINITY;
                    }
            }
            float f[2], mu[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = m[r];
#pragma unroll
                for (int i = 0; i < NT; ++i) x = fmaxf(x, fmaxf(s[i][2 * r], s[i][2 * r + 1]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 1));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 2));
                const float top = x == -INFINITY ? 0.f : x;
                f[r] = ex2_approx(m[r] - top);
                mu[r] = top - LIFT;
                m[r] = x;
            }
#pragma unroll
            for (int i = 0; i < NT; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = ex2_approx(s[i][e] - mu[e >> 1]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < NT; ++i) x += s[i][2 * r] + s[i][2 * r + 1];
                l[r] = l[r] * f[r] + x;
            }
            if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int i = 0; i < 2 * KS; ++i) o[i][0] *= f[0], o[i][1] *= f[0], o[i][2] *= f[1], o[i][3] *= f[1];
            }
            // values at positions that no row of the tile sees may be anything (unwritten rows): taken as 0
            const int row = sl * KW + (((lane >> 3) & 1) << 3) + (lane & 7), ch = lane >> 4;
            auto values = [&](auto clear) {
                constexpr bool CLEAR = decltype(clear)::value;
#pragma unroll
                for (int i = 0; i < NT; i += 2) {  // 16 keys
                    // weights rounded to the values' type for the second product (their sum l is of the unrounded ones)
                    const uint32_t a[4] = {paged_pack2<MM_F16>(s[i][0], s[i][1]), paged_pack2<MM_F16>(s[i][2], s[i][3]),
                                           paged_pack2<MM_F16>(s[i + 1][0], s[i + 1][1]),
                                           paged_pack2<MM_F16>(s[i + 1][2], s[i + 1][3])};
                    uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                    if (CLEAR) {
                        auto seen = [&](int k) { return k >= g.x.key_lo && k < g.x.key_hi; };
                        const int k = key0 + i * 8 + tig * 2;
                        keep0 = (seen(k) ? 0xffffu : 0u) | (seen(k + 1) ? 0xffff0000u : 0u);
                        keep1 = (seen(k + 8) ? 0xffffu : 0u) | (seen(k + 9) ? 0xffff0000u : 0u);
                    }
                    if (!E4M3) {
#pragma unroll
                        for (int j = 0; j < KS; ++j) {
                            uint32_t b[4];
                            ldsm4_t(b, vb + tile_off<C::BOX_BYTES>(row + i * 8, 2 * j + ch));
                            mma16816<MM_F16>(o[2 * j], a, b[0] & keep0, b[1] & keep1);
                            mma16816<MM_F16>(o[2 * j + 1], a, b[2] & keep0, b[3] & keep1);
                        }
                    } else {
                        // a transposed 16-bit element is two neighbouring elements of one row: o[2j] takes the
                        // even ones of 16, o[2j + 1] the odd ones
#pragma unroll
                        for (int j = 0; j < KS; j += 2) {
                            uint32_t b[4];
                            ldsm4_t(b, vb + tile_off<C::BOX_BYTES>(row + i * 8, j + ch));
#pragma unroll
                            for (int x = 0; x < 2; ++x) {
                                const uint32_t b0 = b[2 * x], b1 = b[2 * x + 1];
                                mma16816<true>(o[2 * (j + x)], a, paged_widen(__byte_perm(b0, 0, 0x4420)) & keep0,
                                               paged_widen(__byte_perm(b1, 0, 0x4420)) & keep1);
                                mma16816<true>(o[2 * (j + x) + 1], a, paged_widen(__byte_perm(b0, 0, 0x4431)) & keep0,
                                               paged_widen(__byte_perm(b1, 0, 0x4431)) & keep1);
                            }
                        }
                    }
                }
            };
            if (key0 + KW > g.x.key_hi || key0 < g.x.key_lo)
                values(Bool<true>{});
            else
                values(Bool<false>{});
        };

        bool ok = true;
        for (int u = g.u_begin; ok && u < g.u_end; ++u, ++it) {
            const bool mine = (slot / SPU & (turns - 1)) == (int)(it & (turns - 1));
            if (own && !mine) continue;
            const int s = it % C::NST;
            ok = mbar_wait(&full[s], (it / C::NST) & 1, p.err, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint8_t *st = ring + s * C::STAGE;
            const int key0 = (g.x.u0 + u) * UNIT;
            if (mine)
                for (int sl = slot % SPU; sl < SPU; sl += nslot) slice(st, key0 + sl * KW, sl);
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[s]);
        }
        // every consumer warp leaves together when a wait ran out in one of them
        if (named_bar_or(1, CW * 32, !ok)) return;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 1);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 2);
        }
        // ---- join the key slots, the upper half into the lower one, in a fixed order ----
        const bool two = rbase + 8 < last_row;  // (the group's upper eight rows are there)
        for (int half = nslot >> 1; half > 0; half >>= 1) {
            const int cell = (slot >= half ? slot - half : slot) * MT + rg;
            float *mo = merge + cell * 16 * (C::MERGE_ROW + 2);
            float *ml = mo + 16 * C::MERGE_ROW;
            if (slot >= half && slot < 2 * half) {
#pragma unroll
                for (int i = 0; i < 2 * KS; ++i) {
                    *reinterpret_cast<float2 *>(mo + gid * C::MERGE_ROW + i * 8 + tig * 2) = make_float2(o[i][0], o[i][1]);
                    if (two)
                        *reinterpret_cast<float2 *>(mo + (gid + 8) * C::MERGE_ROW + i * 8 + tig * 2) =
                            make_float2(o[i][2], o[i][3]);
                }
                if (tig == 0)
#pragma unroll
                    for (int r = 0; r < 2; ++r) ml[(gid + 8 * r) * 2] = m[r], ml[(gid + 8 * r) * 2 + 1] = l[r];
            }
            named_bar_sync(1, CW * 32);
            if (slot < half) {
                float fa[2], fb[2];
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    const float om = ml[(gid + 8 * r) * 2], ol = ml[(gid + 8 * r) * 2 + 1];
                    const float nm = fmaxf(m[r], om), mu = nm == -INFINITY ? 0.f : nm;
                    fa[r] = ex2_approx(m[r] - mu), fb[r] = ex2_approx(om - mu);
                    l[r] = l[r] * fa[r] + ol * fb[r];
                    m[r] = nm;
                }
#pragma unroll
                for (int i = 0; i < 2 * KS; ++i) {
                    const float2 x = *reinterpret_cast<const float2 *>(mo + gid * C::MERGE_ROW + i * 8 + tig * 2);
                    o[i][0] = o[i][0] * fa[0] + x.x * fb[0], o[i][1] = o[i][1] * fa[0] + x.y * fb[0];
                    if (two) {
                        const float2 y = *reinterpret_cast<const float2 *>(mo + (gid + 8) * C::MERGE_ROW + i * 8 + tig * 2);
                        o[i][2] = o[i][2] * fa[1] + y.x * fb[1], o[i][3] = o[i][3] * fa[1] + y.y * fb[1];
                    }
                }
            }
            named_bar_sync(1, CW * 32);
        }
        if (slot == 0) {
            const bool whole = g.whole();
            const int64_t piece = (int64_t)blockIdx.x * 2 + g.slot();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                if (!have[r]) continue;
                const int row = rbase + gid + 8 * r, tok = p.by_G.div(row), hg = row - tok * p.G;
                // (only a row that saw nothing has a sum of 0: a NaN goes on into the row's results)
                const float inv = l[r] != 0.f ? p.v_inv / l[r] : 0.f;
                const float ls = l[r] != 0.f ? m[r] + log2f(l[r]) - LIFT : -INFINITY;
                const int64_t orow = (int64_t)(g.s.q0 + tok) * p.H + g.h * p.G + hg;
                const int trow = row - g.x.row0;
                if (tig == 0) {
                    if (!whole)
                        p.part_l[piece * p.TM + trow] = ls;
                    else if (p.lse)
                        p.lse[orow] = ls * 0.6931471805599453f;
                }
                uint16_t *dst = static_cast<uint16_t *>(p.out) + orow * D;
                float *prt = p.part_o + (piece * p.TM + trow) * D;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const float a0 = o[2 * j][2 * r] * inv, a1 = o[2 * j][2 * r + 1] * inv;
                    const float b0 = o[2 * j + 1][2 * r] * inv, b1 = o[2 * j + 1][2 * r + 1] * inv;
                    if (E4M3) {  // four consecutive elements
                        const int d = 16 * j + tig * 4;
                        if (whole)
                            *reinterpret_cast<uint2 *>(dst + d) = make_uint2(paged_pack2<IO_F16>(a0, b0), paged_pack2<IO_F16>(a1, b1));
                        else
                            *reinterpret_cast<float4 *>(prt + d) = make_float4(a0, b0, a1, b1);
                    } else {
                        const int d = 16 * j + tig * 2;
                        if (whole) {
                            *reinterpret_cast<uint32_t *>(dst + d) = paged_pack2<IO_F16>(a0, a1);
                            *reinterpret_cast<uint32_t *>(dst + d + 8) = paged_pack2<IO_F16>(b0, b1);
                        } else {
                            *reinterpret_cast<float2 *>(prt + d) = make_float2(a0, a1);
                            *reinterpret_cast<float2 *>(prt + d + 8) = make_float2(b0, b1);
                        }
                    }
                }
            }
            if (g.slot() == 1 && !whole && rg == 0 && lane == 0)
                p.rec[blockIdx.x] = PieceRec{
                    1, g.s.q0, g.h, g.x.row0, g.x.rows, cur.at - (g.u_end - g.u_begin) + g.x.nu, cur.total};
        }
    }
}

// Joins the pieces of the tile that began in CTA blockIdx.x and went on: row
// by row, out = sum_i w_i o_i / sum_i w_i with w_i = 2^(lse_i - max lse), over
// the pieces in the order of the line.  One warp a row.
constexpr int JOIN_WARPS = 8;
template <int D, bool IO_F16>
__global__ void __launch_bounds__(JOIN_WARPS * 32) paged_attn_join_kernel(const PagedAttnParams p, int nc) {
    pdl_wait();  // the pieces come from the previous kernel
    const int c = blockIdx.x, lane = lane_id();
    const PieceRec rec = p.rec[c];
    if (!rec.valid) return;
    const int r = blockIdx.y * JOIN_WARPS + warp_id();
    if (r >= rec.rows) return;
    const int parts = line_parts(p, nc), part = line_part(p, c);
    const Line line(rec.total, parts);
    const int last = min(line.next(rec.end), parts);  // pieces: slot 1 of this part, slot 0 of the next ones before `last`
    const int stride = p.locked ? p.Hkv : 1;          // from a part's CTA to the next one's
    auto at = [&](int i) { return ((int64_t)(c + (i - part) * stride) * 2 + (i == part ? 1 : 0)) * p.TM + r; };
    constexpr int V = D / 32;
    float acc[V], sum = 0.f, mx = -INFINITY;
#pragma unroll
    for (int j = 0; j < V; ++j) acc[j] = 0.f;
    for (int base = part; base < last; base += 32) {  // 32 pieces at a time, a lane each for their weights
        const int mine = base + lane, cnt = min(32, last - base);
        float o[8][V];
        auto load = [&](int i0) {  // eight rows in flight, the first before their weights are known
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const bool some = i0 + i < cnt;
                const float *src = p.part_o + at(base + i0 + i) * D + lane * V;
                if (V == 4) {
                    const float4 t = some ? *reinterpret_cast<const float4 *>(src) : make_float4(0.f, 0.f, 0.f, 0.f);
                    o[i][0] = t.x, o[i][1] = t.y, o[i][V - 2] = t.z, o[i][V - 1] = t.w;
                } else {
                    const float2 t = some ? *reinterpret_cast<const float2 *>(src) : make_float2(0.f, 0.f);
                    o[i][0] = t.x, o[i][1] = t.y;
                }
            }
        };
        load(0);
        const float ls = mine < last && (mine == part || line.start(mine) < line.start(mine + 1)) ? p.part_l[at(mine)] : -INFINITY;
        float top = ls;
#pragma unroll
        for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
        top = fmaxf(top, mx);
        const bool nan = __any_sync(0xffffffffu, isnan(ls));  // (which the maximum leaves out, and the weights do not)
        if (top == -INFINITY) {
            if (!nan) continue;
            top = 0.f;
        }
        const float f = ex2_approx(mx - top), w = ex2_approx(ls - top);
        mx = top;
        sum *= f;
#pragma unroll
        for (int j = 0; j < V; ++j) acc[j] *= f;
        for (int i0 = 0;;) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float wi = __shfl_sync(0xffffffffu, w, (i0 + i) & 31);
                if (i0 + i < cnt && wi != 0.f) {  // (a piece without weight may be unwritten)
                    sum += wi;
#pragma unroll
                    for (int j = 0; j < V; ++j) acc[j] = fmaf(wi, o[i][j], acc[j]);
                }
            }
            if ((i0 += 8) >= cnt) break;
            load(i0);
        }
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    const int row = rec.row0 + r, tok = p.by_G.div(row);
    const int64_t orow = (int64_t)(rec.q0 + tok) * p.H + rec.h * p.G + (row - tok * p.G);
    uint32_t *dst = reinterpret_cast<uint32_t *>(static_cast<uint16_t *>(p.out) + orow * D + lane * V);
#pragma unroll
    for (int j = 0; j < V; j += 2) dst[j / 2] = paged_pack2<IO_F16>(acc[j] * inv, acc[j + 1] * inv);
    if (p.lse && lane == 0) p.lse[orow] = sum != 0.f ? (mx + log2f(sum)) * 0.6931471805599453f : -INFINITY;
}

// Rows of a tile: enough 16-row groups for one sequence's packed rows, up to
// 128; up to eight rows over an 8-bit cache have a kernel of their own, in which
// they are columns (33 sequences of 1000-40000 positions, one token of 8 heads a
// K/V head, in short runs: 252 us against 257 as half of a 16-row tile; the gap was wider in long ones).
int tile_rows(int64_t max_rows, bool e4m3) {
    if (e4m3 && max_rows <= 8) return 8;
    int mt = 1;
    while (mt < CW && mt * 16 < max_rows) mt *= 2;
    return 16 * mt;
}

struct Plan {
    int TM, nc;
    size_t o_off, l_off, rec_off, total;
};
// `unit` keys a unit, tiles of TM rows.
Plan make_plan(int TM, int unit, int num_seqs, int G, int Hkv, int D, int max_q, int max_len, int window, int sms) {
    Plan pl{};
    pl.TM = TM;
    const int64_t tiles = ((int64_t)max_q * G + TM - 1) / TM;
    int64_t units = ((int64_t)max_len + unit - 1) / unit;
    if (window) {
        const int64_t w = ((int64_t)window + TM) / unit + 2;
        units = w < units ? w : units;
    }
    int64_t most = units;  // no more CTAs than units in the largest call of these bounds
    for (const int64_t x : {tiles, (int64_t)Hkv, (int64_t)num_seqs}) most = most > sms ? most : most * x;
    pl.nc = (int)(most < sms ? most : sms);
    size_t off = 0;
    pl.o_off = off, off += align_up((size_t)pl.nc * 2 * TM * D * 4, 256);
    pl.l_off = off, off += align_up((size_t)pl.nc * 2 * TM * 4, 256);
    pl.rec_off = off, off += align_up((size_t)pl.nc * sizeof(PieceRec), 256);
    pl.total = off;
    return pl;
}

// Few packed rows a K/V head go to the warp-level kernel, more to the tensor
// cores.  8 sequences of 32768 positions, 8 K/V heads of 128, us (warp-level /
// tensor cores): 2-byte cache 32 rows 171 / 204, 64 rows 264 / 208, 128 rows
// 464 / 212; E4M3 32 rows 171 / 264, 64 rows 309 / 266 (8 x 1024: 25 / 31),
// 96 rows 543 / 268.
bool tc_shape(int G, int max_q, bool e4m3) { return G <= 128 && (int64_t)max_q * G > (e4m3 ? 64 : 32); }
// What else the tensor-core kernel needs of a call: a positive scale that stays
// one in fp32 (the maximum is taken before scaling) and q reachable by a tensor map.
bool tc_call(const PagedAttnArgs &a) {
    auto ok = [](int64_t stride, int64_t n) { return n <= 1 || (stride > 0 && stride < ((int64_t)1 << 39)); };
    return a.sm_scale > 1e-30f && ok(a.q.token_stride, a.T) && ok(a.q.head_stride, a.q.heads);
}

bool kv_map(CUtensorMap *m, const void *base, int dtype, int D, int heads, int pages, int64_t page, int64_t row,
            int64_t head) {
    const int e = dtype == DSA_E4M3 ? 1 : 2;
    const int inner = D * e < 128 ? D : 128 / e;
    const uint64_t dims[4] = {(uint64_t)D, 64, (uint64_t)heads, (uint64_t)pages};
    // the stride of a dimension of one entry only has to be a valid one
    const uint64_t strides[3] = {(uint64_t)(row * e), (uint64_t)((heads > 1 ? head : row) * e),
                                 (uint64_t)((pages > 1 ? page : row) * e)};
    const uint32_t box[4] = {(uint32_t)inner, 64, 1, 1};
    const CUtensorMapDataType dt = dtype == DSA_BF16  ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16
                                   : dtype == DSA_F16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16
                                                      : CU_TENSOR_MAP_DATA_TYPE_UINT8;
    return make_tmap_4d(m, base, dt, dims, strides, box,
                        inner * e == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B, D * e);
}

template <int D, bool IO_F16, bool E4M3, int KW>
dsa_status launch_kw(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    auto fn = paged_attn_kernel<D, IO_F16, E4M3, KW>;
    constexpr int SMEM = Cfg<D, E4M3>::SMEM;
    // the roles' register shares draw on what the block was launched with
    static const bool regs_ok = [fn] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, fn) == cudaSuccess && fa.numRegs == REG_LAUNCH;
    }();
    if (!regs_ok || !ensure_smem(reinterpret_cast<const void *>(fn), SMEM)) return DSA_ERR_CUDA;
    CUtensorMap km, vm;
    if (!paged_kv_maps(*a.cache, a.pg.num_pages, &km, &vm)) return DSA_ERR_CUDA;
    fn<<<nc, THREADS, SMEM, st>>>(km, vm, p, p.TM / 16);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}
// Slices of 32 keys, twice as many independent products and half as many exchanges a key as of 16; but where one
// row group's eight slots would then hold four units of a five-unit ring (16 rows, 2-byte cache, D = 128), 16.
template <int D, bool IO_F16, bool E4M3>
dsa_status launch(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    if constexpr (E4M3)
        if (p.TM == 8) return launch_paged_attn8(a, p, nc, st);
    if constexpr (Cfg<D, E4M3>::NST < 8)
        if (p.TM == 16) return launch_kw<D, IO_F16, E4M3, 16>(a, p, nc, st);
    return launch_kw<D, IO_F16, E4M3, 32>(a, p, nc, st);
}

template <int D>
dsa_status launch(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    const bool f16 = a.dtype == DSA_F16;
    if (a.cache->dtype == DSA_E4M3) return f16 ? launch<D, true, true>(a, p, nc, st) : launch<D, false, true>(a, p, nc, st);
    return f16 ? launch<D, true, false>(a, p, nc, st) : launch<D, false, false>(a, p, nc, st);
}

template <int D, bool IO_F16>
dsa_status launch_join(const PagedAttnParams &p, int nc, cudaStream_t st) {
    if (nc == 1) return DSA_OK;  // one CTA holds every tile whole
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(nc, (p.TM + JOIN_WARPS - 1) / JOIN_WARPS);
    cfg.blockDim = dim3(JOIN_WARPS * 32);
    cfg.stream = st;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = at, cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, paged_attn_join_kernel<D, IO_F16>, p, nc) == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

bool paged_kv_maps(const dsa_kv_cache &c, int num_pages, CUtensorMap *km, CUtensorMap *vm) {
    return kv_map(km, c.k, c.dtype, c.Dk, c.heads, num_pages, c.k_page_stride, c.k_row_stride, c.k_head_stride) &&
           kv_map(vm, c.v, c.dtype, c.Dk, c.heads, num_pages, c.v_page_stride, c.v_row_stride, c.v_head_stride);
}

// Enough for every call of these bounds: fewer tokens, shorter sequences or windows and fewer sequences never take more,
// but smaller groups of heads can (a chunk's tile has 2 (128 / G) G rows), so each size of them is looked at.
size_t paged_attn_workspace_bytes(int32_t num_seqs, int32_t H, int32_t Hkv, int32_t D, bool e4m3, int32_t max_q,
                                  int32_t max_len, int32_t window, int sm_count) {
    size_t need = 0;
    for (int G = H / Hkv; G > 0; --G) {
        const size_t few = make_plan(tile_rows((int64_t)max_q * G, e4m3), UNIT, num_seqs, G, Hkv, D, max_q, max_len,
                                     window, sm_count).total;
        need = few > need ? few : need;
        if (tc_shape(G, max_q, e4m3)) {  // (the call's scale and strides decide between the two)
            const size_t tc =
                make_plan(paged_attn_tc_rows(G), 128, num_seqs, G, Hkv, D, max_q, max_len, window, sm_count).total;
            need = tc > need ? tc : need;
        }
    }
    return need;
}

dsa_status launch_paged_attn(const PagedAttnArgs &a, cudaStream_t st) {
    const DeviceInfo *dev = current_device();
    if (!dev) return DSA_ERR_CUDA;
    const dsa_kv_cache &c = *a.cache;
    const int H = a.q.heads, D = c.Dk, G = H / c.heads;
    const bool tc = tc_shape(G, a.max_q, c.dtype == DSA_E4M3) && tc_call(a);
    const Plan pl = make_plan(tc ? paged_attn_tc_rows(G) : tile_rows((int64_t)a.max_q * G, c.dtype == DSA_E4M3), tc ? 128 : UNIT,
                              a.pg.num_seqs, G, c.heads, D, a.max_q, a.max_len, a.window, dev->sm_count);
    if (!a.ws || a.ws_bytes < pl.total || (reinterpret_cast<uintptr_t>(a.ws) & 255u)) return DSA_ERR_WORKSPACE;
    const bool e4m3 = c.dtype == DSA_E4M3;
    uint8_t *ws = static_cast<uint8_t *>(a.ws);
    PagedAttnParams p{};
    p.q = a.q.data, p.q_token = a.q.token_stride, p.q_head = a.q.head_stride;
    p.q_start = a.q_start, p.pg = a.pg;
    p.T = a.T, p.H = H, p.Hkv = c.heads, p.G = G, p.TM = pl.TM;
    p.by_G = FastDiv::of(G), p.by_TM = FastDiv::of(pl.TM);
    p.max_q = a.max_q, p.max_len = a.max_len, p.window = a.window;
    // Windowed chunks of heads with keys of their own: row blocks of 128 tokens that begin at multiples of 128 see two
    // key units within a window of 128 instead of three (eight chunks of 257-2048 tokens, 64 heads: 208 us against
    // 238, window 1000: 503 against 519).  Shorter blocks, of groups, see as few anyway (two heads a group: 202 us
    // against 192).
    p.align = tc && a.window && p.G == 1 ? 128 : 0;
    // Heads in step, where that idles no more than one CTA in twenty: 64 sequences' decode 1230 us against 1280,
    // an 8-bit cache 252 against 284, drafts 605 against 630, in short runs.  Chunks, whose keys come from L2, were slower (1658
    // against 1634).
    const int even = pl.nc / c.heads * c.heads;
    p.locked = !tc && c.heads > 1 && even * 20 >= pl.nc * 19;
    const int nc = p.locked ? even : pl.nc;
    p.scale_log2 = (float)(a.sm_scale * 1.4426950408889634 / (e4m3 ? c.k_scale : 1.f));
    if (tc) p.scale_log2 = fmaxf(p.scale_log2, PAGED_MIN_SCALE);
    p.v_inv = e4m3 ? 1.f / c.v_scale : 1.f;
    p.out = a.out, p.lse = a.lse;
    p.part_o = reinterpret_cast<float *>(ws + pl.o_off);
    p.part_l = reinterpret_cast<float *>(ws + pl.l_off);
    p.rec = reinterpret_cast<PieceRec *>(ws + pl.rec_off);
    p.err = dev->err;
    const bool f16 = a.dtype == DSA_F16;
    dsa_status s;
    if (tc)
        s = launch_paged_attn_tc(a, p, nc, st);
    else
        s = D == 128 ? launch<128>(a, p, nc, st) : launch<64>(a, p, nc, st);
    if (s != DSA_OK) return s;
    if (D == 128) return f16 ? launch_join<128, true>(p, nc, st) : launch_join<128, false>(p, nc, st);
    return f16 ? launch_join<64, true>(p, nc, st) : launch_join<64, false>(p, nc, st);
}

}  // namespace dsa
