// Attention of single tokens over an 8-bit paged K/V cache, for up to eight
// packed rows a K/V head (one token of up to eight query heads): the sums of
// paged_attn.cu with keys as the 16-row operand of the matrix instruction and
// the queries as its 8-column one,
//   S^T = K Q^T,  P^T = 2^(c S^T - m),  O^T += V^T P^T,
// where 16-row tiles of queries would be half empty.  Products, registers and
// exponentials halve, so that sixteen warps a CTA fit, and the widening of the
// codes (two conversions a pair of elements, most of the instructions) hides
// behind the loads.  HBM-bound by intent: 33 sequences of 1000-40000
// positions, 64 heads of 128 on 8: 256 us in short runs, 276 in long ones, for
// 1.43 GB (85% and 79% of the measured copy rate; a page's rows lie 128 bytes a
// head apart, and heads read in step find them together: 284 us out of step).
#include "dsa_device.cuh"
#include "dsa_internal.h"
#include "paged_units.cuh"

namespace dsa {
namespace {

constexpr int UNIT = UNIT_KEYS;
constexpr int CW = 16;     // consumer warps, a key slot each
constexpr int KW = 32;     // keys of a slice
constexpr int SPU = UNIT / KW, TURNS = CW / SPU;  // slices of a unit; units in turn
constexpr int THREADS = (CW + 4) * 32;
// registers: 640 x 96 at launch; the roles' shares add up to the same
constexpr int REG_LAUNCH = 96, REG_CONSUME = 104, REG_LOAD = 64;
static_assert(CW * 32 * REG_CONSUME + 128 * REG_LOAD == THREADS * REG_LAUNCH, "register shares");

template <int D>
struct Cfg : UnitRing<D, true> {
    static_assert(Cfg::NST % TURNS == 0, "a stage belongs to the same warps");
    static constexpr int MERGE_ROW = D + 4;
    static constexpr int MERGE_CELL = 8 * MERGE_ROW + 16;  // floats: eight rows, their maxima and sums
    static constexpr int SMEM = Cfg::NST * Cfg::STAGE + (CW / 2) * MERGE_CELL * 4 + 1024;
};

// An 8x8 matrix of 16-bit elements, spread over the warp by rows, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
    return r;
}

// Thread (gid, tig) = (lane / 4, lane % 4) holds scores of queries 2 tig, 2 tig + 1.
template <int D, bool IO_F16>
__global__ void __launch_bounds__(THREADS, 1)
    paged_attn8_kernel(const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                       const PagedAttnParams p) {
    using C = Cfg<D>;
    constexpr int KS = D / 16;  // k-steps of q.k; also 16-row tiles of the output
    extern __shared__ uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    float *merge = reinterpret_cast<float *>(ring + C::NST * C::STAGE);
    __shared__ PlanShared plan;
    __shared__ uint64_t full[C::NST], empty[C::NST];
    __shared__ int abort_flag;
    const int warp = warp_id(), lane = lane_id();
    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NST; ++s) mbar_init(&full[s], 1), mbar_init(&empty[s], SPU);
        abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&kmap);
        tma_prefetch_desc(&vmap);
        p.rec[blockIdx.x].valid = 0;
    }
    pdl_trigger();
    Cursor cur = plan_cta<UNIT>(p, blockIdx.x, gridDim.x, plan);  // also orders the barrier setup before its use
    if (warp >= CW) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(REG_LOAD));
        if (warp == CW) load_units<C>(kmap, vmap, p, cur, ring, full, empty, &abort_flag);
        return;
    }
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(REG_CONSUME));
    const int gid = lane >> 2, tig = lane & 3;
    const int turn = warp / SPU, sl = warp % SPU;
    Segment g;
    uint32_t it = 0;
    while (next_segment<UNIT>(p, cur, g)) {
        // this thread loads query row gid, and has scores of rows 2 tig and 2 tig + 1 (one tile: row0 = 0)
        const int rows = g.x.rows;
        uint32_t qf[KS][2];
        float scale;
        {
            const bool have = gid < rows;
            const int tok = p.by_G.div(gid), hg = gid - tok * p.G;
            const uint16_t *src = static_cast<const uint16_t *>(p.q) + (int64_t)(g.s.q0 + tok) * p.q_token +
                                  (int64_t)(g.h * p.G + hg) * p.q_head;
            // an 8-bit key fragment holds four consecutive elements a thread: q takes the same order
            float mx = 0.f;
#pragma unroll
            for (int k = 0; k < KS; ++k) {
                const uint2 v = have ? *reinterpret_cast<const uint2 *>(src + k * 16 + tig * 4) : make_uint2(0, 0);
                qf[k][0] = v.x, qf[k][1] = v.y;
                const float2 a = unpack2<IO_F16>(v.x), b = unpack2<IO_F16>(v.y);
                mx = fmaxf(fmaxf(mx, fmaxf(fabsf(a.x), fabsf(a.y))), fmaxf(fabsf(b.x), fabsf(b.y)));
            }
            scale = p.scale_log2;
            if (!IO_F16) {
                // bf16 to fp16: times 2^-e with 2^e <= max|q| < 2^(e+1), so that the row fits; what is lost lies
                // 2^-24 below the row's largest element
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
                int e = (int)(__float_as_uint(mx) >> 23) - 127;
                e = mx > 0.f ? max(-126, min(e, 126)) : 0;
                const float down = __uint_as_float((uint32_t)(127 - e) << 23);
                scale *= __uint_as_float((uint32_t)(127 + e) << 23);
#pragma unroll
                for (int k = 0; k < KS; ++k)
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const float2 a = unpack2<false>(qf[k][x]);
                        qf[k][x] = paged_pack2<true>(a.x * down, a.y * down);
                    }
            }
        }
        float c[2], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
        int pos[2];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            const int row = 2 * tig + r;
            c[r] = __shfl_sync(0xffffffffu, scale, row * 4);
            pos[r] = row < rows ? g.s.L - g.s.n + p.by_G.div(row) : -1;
        }
        float o[KS][4];
#pragma unroll
        for (int i = 0; i < KS; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;

        bool ok = true;
        for (int u = g.u_begin; ok && u < g.u_end; ++u, ++it) {
            if ((int)(it & (TURNS - 1)) != turn) continue;  // other warps' stage
            const int stage = it % C::NST;
            ok = mbar_wait(&full[stage], (it / C::NST) & 1, p.err, &abort_flag);
            ok = __all_sync(0xffffffffu, ok);
            if (!ok) break;
            const uint32_t kb = smem_u32(ring + stage * C::STAGE), vb = kb + C::TILE_BYTES;
            const int key0 = (g.x.u0 + u) * UNIT + sl * KW;
            const int row = sl * KW + (((lane >> 3) & 1) << 3) + (lane & 7), ch = lane >> 4;
            float s[KW / 16][4];  // keys 16 i + gid (+ 8), queries 2 tig (+ 1)
#pragma unroll
            for (int i = 0; i < KW / 16; ++i) s[i][0] = s[i][1] = s[i][2] = s[i][3] = 0.f;
#pragma unroll
            for (int k = 0; k < KS; k += 2)
#pragma unroll
                for (int i = 0; i < KW / 16; ++i) {
                    uint32_t b[4];
                    ldsm4(b, kb + tile_off<C::BOX_BYTES>(row + i * 16, k + ch));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t a[4] = {paged_widen(b[2 * x]), paged_widen(b[2 * x + 1]), paged_widen(b[2 * x] >> 16),
                                               paged_widen(b[2 * x + 1] >> 16)};
                        mma16816<true>(s[i], a, qf[k + x][0], qf[k + x][1]);
                    }
                }
            // scores in log2 units; masked where a row does not see the key
#pragma unroll
            for (int i = 0; i < KW / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] *= c[e & 1];
            if (key0 + KW - 1 > g.x.p_first || (p.window && key0 <= g.x.p_last - p.window)) {
#pragma unroll
                for (int i = 0; i < KW / 16; ++i)
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const int key = key0 + i * 16 + gid + (e >> 1) * 8, r = e & 1;
                        if (key > pos[r] || (p.window && key <= pos[r] - p.window)) s[i][e] = -INFINITY;
                    }
            }
            float f[2], mu[2];
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = m[r];
#pragma unroll
                for (int i = 0; i < KW / 16; ++i) x = fmaxf(x, fmaxf(s[i][r], s[i][2 + r]));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
                x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
                const float top = x == -INFINITY ? 0.f : x;
                f[r] = ex2_approx(m[r] - top);
                mu[r] = top - FP16_LIFT;
                m[r] = x;
            }
#pragma unroll
            for (int i = 0; i < KW / 16; ++i)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[i][e] = ex2_approx(s[i][e] - mu[e & 1]);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                float x = 0.f;
#pragma unroll
                for (int i = 0; i < KW / 16; ++i) x += s[i][r] + s[i][2 + r];
                l[r] = l[r] * f[r] + x;
            }
            if (__any_sync(0xffffffffu, f[0] != 1.f || f[1] != 1.f)) {
#pragma unroll
                for (int i = 0; i < KS; ++i) o[i][0] *= f[0], o[i][1] *= f[1], o[i][2] *= f[0], o[i][3] *= f[1];
            }
            // values at positions that no row of the tile sees may be anything (unwritten rows): taken as 0
            const bool clear = key0 + KW > g.x.key_hi || key0 < g.x.key_lo;
#pragma unroll
            for (int i = 0; i < KW / 16; ++i) {  // 16 keys
                // weights rounded to fp16 for the second product (their sum l is of the unrounded ones), keys along the warp
                const uint32_t w0 = transpose8(paged_pack2<true>(s[i][0], s[i][1]));
                const uint32_t w1 = transpose8(paged_pack2<true>(s[i][2], s[i][3]));
                uint32_t keep0 = 0xffffffffu, keep1 = 0xffffffffu;
                if (clear) {
                    auto seen = [&](int k) { return k >= g.x.key_lo && k < g.x.key_hi; };
                    const int k = key0 + i * 16 + tig * 2;
                    keep0 = (seen(k) ? 0xffffu : 0u) | (seen(k + 1) ? 0xffff0000u : 0u);
                    keep1 = (seen(k + 8) ? 0xffffu : 0u) | (seen(k + 9) ? 0xffff0000u : 0u);
                }
                // a transposed 16-bit element is two neighbouring elements of one row: the tile's rows gid are the
                // even ones of 16, its rows gid + 8 the odd ones
#pragma unroll
                for (int j = 0; j < KS; j += 2) {
                    uint32_t b[4];
                    ldsm4_t(b, vb + tile_off<C::BOX_BYTES>(row + i * 16, j + ch));
#pragma unroll
                    for (int x = 0; x < 2; ++x) {
                        const uint32_t b0 = b[2 * x], b1 = b[2 * x + 1];
                        const uint32_t a[4] = {
                            paged_widen(__byte_perm(b0, 0, 0x4420)) & keep0, paged_widen(__byte_perm(b0, 0, 0x4431)) & keep0,
                            paged_widen(__byte_perm(b1, 0, 0x4420)) & keep1, paged_widen(__byte_perm(b1, 0, 0x4431)) & keep1};
                        mma16816<true>(o[j + x], a, w0, w1);
                    }
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[stage]);
        }
        // every consumer warp leaves together when a wait ran out in one of them
        if (named_bar_or(1, CW * 32, !ok)) return;
#pragma unroll
        for (int r = 0; r < 2; ++r) {
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 4);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 8);
            l[r] += __shfl_xor_sync(0xffffffffu, l[r], 16);
        }
        // ---- join the warps, the upper half into the lower one, in a fixed order ----
        // element (row 2 tig + r, d) of the output: d = 16 j + 2 gid in o[j][r], the next one in o[j][2 + r]
        for (int half = CW / 2; half > 0; half >>= 1) {
            float *mo = merge + (warp >= half ? warp - half : warp) * C::MERGE_CELL, *ml = mo + 8 * C::MERGE_ROW;
            if (warp >= half && warp < 2 * half) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (2 * tig + r < rows) {
#pragma unroll
                        for (int j = 0; j < KS; ++j)
                            *reinterpret_cast<float2 *>(mo + (2 * tig + r) * C::MERGE_ROW + 16 * j + 2 * gid) =
                                make_float2(o[j][r], o[j][2 + r]);
                    }
                    if (gid == 0) ml[(2 * tig + r) * 2] = m[r], ml[(2 * tig + r) * 2 + 1] = l[r];
                }
            }
            named_bar_sync(1, CW * 32);
            if (warp < half) {
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                    if (2 * tig + r >= rows) continue;
                    const float om = ml[(2 * tig + r) * 2], ol = ml[(2 * tig + r) * 2 + 1];
                    const float nm = fmaxf(m[r], om), mu = nm == -INFINITY ? 0.f : nm;
                    const float fa = ex2_approx(m[r] - mu), fb = ex2_approx(om - mu);
                    l[r] = l[r] * fa + ol * fb;
                    m[r] = nm;
#pragma unroll
                    for (int j = 0; j < KS; ++j) {
                        const float2 x =
                            *reinterpret_cast<const float2 *>(mo + (2 * tig + r) * C::MERGE_ROW + 16 * j + 2 * gid);
                        o[j][r] = o[j][r] * fa + x.x * fb, o[j][2 + r] = o[j][2 + r] * fa + x.y * fb;
                    }
                }
            }
            named_bar_sync(1, CW * 32);
        }
        if (warp == 0) {
            const bool whole = g.whole();
            const int64_t piece = (int64_t)blockIdx.x * 2 + g.slot();
#pragma unroll
            for (int r = 0; r < 2; ++r) {
                const int row = 2 * tig + r;
                if (row >= rows) continue;
                const int tok = p.by_G.div(row), hg = row - tok * p.G;
                // (only a row that saw nothing has a sum of 0: a NaN goes on into the row's results)
                const float inv = l[r] != 0.f ? p.v_inv / l[r] : 0.f;
                const float ls = l[r] != 0.f ? m[r] + log2f(l[r]) - FP16_LIFT : -INFINITY;
                const int64_t orow = (int64_t)(g.s.q0 + tok) * p.H + g.h * p.G + hg;
                if (gid == 0) {
                    if (!whole)
                        p.part_l[piece * p.TM + row] = ls;
                    else if (p.lse)
                        p.lse[orow] = ls * 0.6931471805599453f;
                }
                uint16_t *dst = static_cast<uint16_t *>(p.out) + orow * D;
                float *prt = p.part_o + (piece * p.TM + row) * D;
#pragma unroll
                for (int j = 0; j < KS; ++j) {
                    const float a = o[j][r] * inv, b = o[j][2 + r] * inv;
                    const int d = 16 * j + 2 * gid;
                    if (whole)
                        *reinterpret_cast<uint32_t *>(dst + d) = paged_pack2<IO_F16>(a, b);
                    else
                        *reinterpret_cast<float2 *>(prt + d) = make_float2(a, b);
                }
            }
            if (g.slot() == 1 && !whole && lane == 0)
                p.rec[blockIdx.x] = PieceRec{
                    1, g.s.q0, g.h, g.x.row0, g.x.rows, cur.at - (g.u_end - g.u_begin) + g.x.nu, cur.total};
        }
    }
}

template <int D, bool IO_F16>
dsa_status launch(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    auto fn = paged_attn8_kernel<D, IO_F16>;
    // the roles' register shares draw on what the block was launched with
    static const bool regs_ok = [fn] {
        cudaFuncAttributes fa;
        return cudaFuncGetAttributes(&fa, fn) == cudaSuccess && fa.numRegs == REG_LAUNCH;
    }();
    if (!regs_ok || !ensure_smem(reinterpret_cast<const void *>(fn), Cfg<D>::SMEM)) return DSA_ERR_CUDA;
    CUtensorMap km, vm;
    if (!paged_kv_maps(*a.cache, a.pg.num_pages, &km, &vm)) return DSA_ERR_CUDA;
    fn<<<nc, THREADS, Cfg<D>::SMEM, st>>>(km, vm, p);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

}  // namespace

dsa_status launch_paged_attn8(const PagedAttnArgs &a, const PagedAttnParams &p, int nc, cudaStream_t st) {
    const bool f16 = a.dtype == DSA_F16;
    if (a.cache->Dk == 128) return f16 ? launch<128, true>(a, p, nc, st) : launch<128, false>(a, p, nc, st);
    return f16 ? launch<64, true>(a, p, nc, st) : launch<64, false>(a, p, nc, st);
}

}  // namespace dsa
