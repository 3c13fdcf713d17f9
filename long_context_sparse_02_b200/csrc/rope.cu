// Rotary positions, alone (dsa_rope) and on the way into a paged cache
// (dsa_append_rope): one kernel, which moves the heads of a call's tokens to
// where they go and turns the pairs of their rotated part by
//   theta_i = pos * inv_freq[i]:  (a, b) -> factor (a cos - b sin, b cos + a sin).
//
// The angle is formed in fp64 and reduced to a fraction of a turn in
// [-1/2, 1/2] before fp32 takes over: at position 2^20 an fp32 angle would be
// off by up to 0.06 radians.  A block is a few tokens (or a part of one token's
// heads, when there are few tokens): its threads take the sines and cosines
// into shared memory (shared by all heads of a token) and look up where the
// tokens go.  A thread keeps its place within a head (a unit: two 16-byte
// vectors) and goes from head to head, two at a time in flight, so that a
// unit costs its loads, products and stores and little else.  The first
// loads are issued before the sines, the page lookup and the barrier, whose
// latency they hide.
// HBM-bound: each element is read and written once.
#include <cuda_fp16.h>
#include <math.h>

#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int ROPE_THREADS = 128;
constexpr int MAX_SEG = 3;

// One array of heads: where its tokens' heads come from, where they go.
struct Seg {
    const void *in;
    void *out;
    int64_t in_token, in_head, out_token, out_head;  // elements
    int64_t out_page, out_row;                       // paged destinations (paged != 0)
    int32_t heads, D;
    int32_t units;  // per head: rotated ones first, then copied ones
    int32_t rot;    // rotated units per head (0: copied whole)
    int32_t wide;   // a copied unit is two vectors
    FastDiv by_units, by_heads;  // (by_units: of the first ROPE_THREADS)
    int32_t paged, e4m3;
    float scale;
};

struct MoveParams {
    Seg seg[MAX_SEG];
    int32_t nseg, tokens;
    int32_t per_block;    // tokens per block
    int32_t heads, part;  // heads of a token, all segments; those that a block moves
    const int32_t *pos, *tok_seq;  // tok_seq NULL: nothing is paged
    PagedDev pg;
    const double *inv_freq;
    int32_t dim, offset;
    float factor, sin_sign;
    uint32_t *err;
};

template <typename T>
struct Conv;
template <>
struct Conv<__nv_bfloat16> {
    static __device__ __forceinline__ float2 up(uint32_t v) {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
    }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __nv_bfloat162 r = __floats2bfloat162_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ float up1(__nv_bfloat16 v) { return __bfloat162float(v); }
    static __device__ __forceinline__ __nv_bfloat16 down1(float v) { return __float2bfloat16_rn(v); }
};
template <>
struct Conv<__half> {
    static __device__ __forceinline__ float2 up(uint32_t v) { return __half22float2(*reinterpret_cast<__half2 *>(&v)); }
    static __device__ __forceinline__ uint32_t down(float a, float b) {
        const __half2 r = __floats2half2_rn(a, b);
        return *reinterpret_cast<const uint32_t *>(&r);
    }
    static __device__ __forceinline__ float up1(__half v) { return __half2float(v); }
    static __device__ __forceinline__ __half down1(float v) { return __float2half_rn(v); }
};

// Two fp32 values to two e4m3 codes (nearest, ties to even, saturating): lo in bits 0-7.
__device__ __forceinline__ uint32_t to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n\t.reg .b16 t;\n\tcvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n\tcvt.u32.u16 %0, t;\n\t}"
        : "=r"(r)
        : "f"(hi), "f"(lo));
    return r;
}

// VEC elements as fp32 from / to memory.  8: one 16-byte vector; 1: one element.
template <typename T, int VEC>
struct Vec;
template <typename T>
struct Vec<T, 8> {
    uint4 v;
    __device__ __forceinline__ void load(const T *p) { v = *reinterpret_cast<const uint4 *>(p); }
    __device__ __forceinline__ void floats(float *f) const {
        const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 t = Conv<T>::up(w[i]);
            f[2 * i] = t.x, f[2 * i + 1] = t.y;
        }
    }
    static __device__ __forceinline__ void store(T *p, const float *f) {
        *reinterpret_cast<uint4 *>(p) = make_uint4(Conv<T>::down(f[0], f[1]), Conv<T>::down(f[2], f[3]),
                                                   Conv<T>::down(f[4], f[5]), Conv<T>::down(f[6], f[7]));
    }
    __device__ __forceinline__ void copy(T *p) const { *reinterpret_cast<uint4 *>(p) = v; }
    static __device__ __forceinline__ void store8(uint8_t *p, const float *f, float s) {
        const uint32_t a = to_e4m3x2(f[0] * s, f[1] * s), b = to_e4m3x2(f[2] * s, f[3] * s);
        const uint32_t c = to_e4m3x2(f[4] * s, f[5] * s), d = to_e4m3x2(f[6] * s, f[7] * s);
        *reinterpret_cast<uint2 *>(p) = make_uint2(a | (b << 16), c | (d << 16));
    }
};
template <typename T>
struct Vec<T, 1> {
    T v;
    __device__ __forceinline__ void load(const T *p) { v = *p; }
    __device__ __forceinline__ void floats(float *f) const { f[0] = Conv<T>::up1(v); }
    static __device__ __forceinline__ void store(T *p, const float *f) { *p = Conv<T>::down1(f[0]); }
    __device__ __forceinline__ void copy(T *p) const { *p = v; }
    static __device__ __forceinline__ void store8(uint8_t *p, const float *f, float s) {
        *p = static_cast<uint8_t>(to_e4m3x2(f[0] * s, 0.f));
    }
};

// Where a unit lies in its head.  A rotated one is two vectors: elements e0..
// and e1.. (the pair partners in the half layout, neighbours in the
// interleaved one); a copied one is two neighbours too, or one where their
// number is odd or the rotated part begins between two (then e1 = e0).
struct Unit {
    int e0, e1;
};

template <int VEC, bool INTER>
__device__ __forceinline__ Unit unit_of(const MoveParams &p, const Seg &g, int x) {
    if (x < g.rot) {
        const int e = p.offset + (INTER ? 2 * x * VEC : x * VEC);
        return Unit{e, INTER ? e + VEC : e + p.dim / 2};
    }
    int e = (x - g.rot) * (g.wide ? 2 * VEC : VEC);
    if (g.rot && e >= p.offset) e += p.dim;  // past the rotated part
    return Unit{e, g.wide ? e + VEC : e};
}

constexpr int MAX_TOKENS = 32;  // per block
struct Dest {
    int64_t page;  // -1: nothing is written for the token
    int row;
};

// The sines and cosines of a unit's VEC pairs, and where they lie in shared memory (of `rot` units a token):
// pairs 2j, 2j + 1 of neighbouring units next to each other, so that neighbouring threads read neighbouring
// 16 bytes.
template <int VEC>
__device__ __forceinline__ int cs_at(int pair, int rot) {
    if (VEC == 1) return pair;
    return ((pair % VEC >> 1) * rot + pair / VEC) * 2 + (pair & 1);
}
template <int VEC>
__device__ __forceinline__ void load_cs(float2 *w, const float2 *cs, int x, int rot) {
    if (VEC == 1) {
        w[0] = cs[x];
    } else {
#pragma unroll
        for (int j = 0; j + 1 < VEC; j += 2) {
            const float4 v = *reinterpret_cast<const float4 *>(cs + ((j >> 1) * rot + x) * 2);
            w[j] = make_float2(v.x, v.y), w[j + 1] = make_float2(v.z, v.w);
        }
    }
}
__device__ __forceinline__ void turn1(float &a, float &b, float2 w) {
    const float a0 = a, b0 = b;
    a = a0 * w.x - b0 * w.y;
    b = b0 * w.x + a0 * w.y;
}
template <int VEC, bool INTER>
__device__ __forceinline__ void turn(float *x, float *y, const float2 *w) {
    if (INTER && VEC > 1) {  // pairs lie next to each other: x holds VEC / 2 of them, y the next VEC / 2
#pragma unroll
        for (int i = 0; i + 1 < VEC; i += 2) turn1(x[i], x[i + 1], w[i / 2]), turn1(y[i], y[i + 1], w[VEC / 2 + i / 2]);
    } else {
#pragma unroll
        for (int i = 0; i < VEC; ++i) turn1(x[i], y[i], w[i]);
    }
}

constexpr int BATCH = 2;  // heads of a thread in flight
constexpr int WORK = 16;  // units of a thread in a block, where there are enough

// cos and sin of the block's tokens, [tokens][dim/2], in dynamic shared memory.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) move_heads_kernel(const __grid_constant__ MoveParams p) {
    extern __shared__ __align__(16) float2 cs[];
    __shared__ Dest dest[MAX_TOKENS];
    const int t0 = blockIdx.x * p.per_block, nt = min(p.per_block, p.tokens - t0), half = p.dim / 2;
    const int h_begin = blockIdx.y * p.part, h_end = min(h_begin + p.part, p.heads);  // (all heads, or one token's)
    // this thread's walk: segment s, units x0 .. of its heads; items m (head of a token) from m0, step apart, below n
    int s = 0, x0 = 0, before = 0, m0 = 0, n = 0, step = 1, lo = 0;
    int x = 0;  // the unit
    Unit un{};
    auto enter = [&] {
        const Seg &g = p.seg[s];
        lo = max(h_begin - before, 0);
        const int nh = min(h_end - before, g.heads) - lo;
        const int ux = min(g.units - x0, ROPE_THREADS);
        const int hl = ux == ROPE_THREADS ? 0 : x0 ? threadIdx.x / ux : g.by_units.div(threadIdx.x);
        step = ux == ROPE_THREADS ? 1 : x0 ? ROPE_THREADS / ux : g.by_units.div(ROPE_THREADS);
        x = x0 + threadIdx.x - hl * ux;
        un = unit_of<VEC, INTER>(p, g, x);
        m0 = hl;
        n = nh > 0 && hl < step ? nt * nh : 0;
    };
    Vec<T, VEC> a[BATCH], b[BATCH];
    auto token_of = [&](const Seg &g, int m) { return nt == 1 ? 0 : g.by_heads.div(m); };
    auto fetch = [&] {
        const Seg &g = p.seg[s];
        const T *in = static_cast<const T *>(g.in) + t0 * g.in_token;
        const bool two = un.e1 != un.e0;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int m = m0 + k * step;
            if (m >= n) break;
            const int t = token_of(g, m);
            const T *src = in + t * g.in_token + (m - t * g.heads + lo) * g.in_head;
            a[k].load(src + un.e0);
            if (two) b[k].load(src + un.e1);
        }
    };
    auto put = [&] {
        const Seg &g = p.seg[s];
        const bool two = un.e1 != un.e0;
#pragma unroll
        for (int k = 0; k < BATCH; ++k) {
            const int m = m0 + k * step;
            if (m >= n) break;
            const int t = token_of(g, m);
            int64_t at = (m - t * g.heads + lo) * g.out_head;
            if (p.tok_seq) {
                const Dest d = dest[t];
                if (d.page < 0) continue;
                if (g.paged) at += d.page * g.out_page + d.row * g.out_row;
            }
            if (!g.paged) at += (int64_t)(t0 + t) * g.out_token;
            if (x >= g.rot && !g.e4m3) {
                T *o = static_cast<T *>(g.out) + at;
                a[k].copy(o + un.e0);
                if (two) b[k].copy(o + un.e1);
                continue;
            }
            float f[VEC], h[VEC];
            a[k].floats(f);
            b[k].floats(h);
            if (x < g.rot) {
                float2 w[VEC];
                load_cs<VEC>(w, cs + t * half, x, g.rot);
                turn<VEC, INTER>(f, h, w);
            }
            if (g.e4m3) {
                uint8_t *o = static_cast<uint8_t *>(g.out) + at;
                Vec<T, VEC>::store8(o + un.e0, f, g.scale);
                if (two) Vec<T, VEC>::store8(o + un.e1, h, g.scale);
            } else {
                T *o = static_cast<T *>(g.out) + at;
                Vec<T, VEC>::store(o + un.e0, f);
                Vec<T, VEC>::store(o + un.e1, h);
            }
        }
    };
    // to the next segment (or run of units of this one) that has something for this thread
    auto next = [&] {
        while (s < p.nseg) {
            enter();
            if (n > m0) return true;
            x0 += ROPE_THREADS;
            if (x0 >= p.seg[s].units) before += p.seg[s].heads, ++s, x0 = 0;
        }
        return false;
    };
    bool more = next();
    if (more) fetch();
    if (p.tok_seq && threadIdx.x < nt) {
        const int t = t0 + threadIdx.x, sq = p.tok_seq[t], pos = p.pos[t];
        Dest d{-1, 0};
        if (sq != -1) {  // (-1: padding)
            uint32_t bad = 0;
            if (sq < 0 || sq >= p.pg.num_seqs || pos < 0 || pos >= p.pg.seq_lens[sq]) {
                bad = DSA_DEVERR_POSITION;
            } else {
                const int lp = pos >> 6;
                d.page = lp < p.pg.max_blocks ? p.pg.block_table[(int64_t)sq * p.pg.max_blocks + lp] : -1;
                d.row = pos & 63;
                if (d.page < 0 || d.page >= p.pg.num_pages) bad = DSA_DEVERR_PAGE;
            }
            if (bad) {
                d.page = -1;
                if (blockIdx.y == 0) record_error(p.err, bad);
            }
        }
        dest[threadIdx.x] = d;
    }
    for (int i = threadIdx.x; i < nt * half; i += ROPE_THREADS) {
        const int t = nt == 1 ? 0 : i / half;
        const double turns = (double)p.pos[t0 + t] * p.inv_freq[i - t * half] * 0.15915494309189535;  // 1 / 2 pi
        float sn, c;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
        const int pair = i - t * half;
        cs[t * half + cs_at<VEC>(pair, half / VEC)] = make_float2(c * p.factor, sn * p.factor * p.sin_sign);
    }
    __syncthreads();
    while (more) {
        put();
        m0 += BATCH * step;
        if (m0 >= n) {
            x0 += ROPE_THREADS;
            if (x0 >= p.seg[s].units) before += p.seg[s].heads, ++s, x0 = 0;
            more = next();
        }
        if (more) fetch();
    }
}

template <typename T, int VEC, bool INTER>
dsa_status launch_move(MoveParams &p, int T_tokens, int sm_count, cudaStream_t st) {
    int64_t total = 0, heads = 0;
    for (int s = 0; s < p.nseg; ++s) {
        Seg &g = p.seg[s];
        g.rot = g.rot ? p.dim / (2 * VEC) : 0;
        // heads rotated in place leave their other elements where they are
        const bool still = g.in == g.out && !g.paged && g.rot;
        const int copied = still ? 0 : (g.D - (g.rot ? p.dim : 0)) / VEC;
        g.wide = copied % 2 == 0 && (!g.rot || p.offset % (2 * VEC) == 0);
        g.units = g.rot + (g.wide ? copied / 2 : copied);
        g.by_units = FastDiv::of(g.units < ROPE_THREADS ? g.units : ROPE_THREADS);
        g.by_heads = FastDiv::of(g.heads);
        total += (int64_t)g.heads * g.units;
        heads += g.heads;
    }
    if (total == 0 || T_tokens == 0) return DSA_OK;
    if (total > (1 << 26)) return DSA_ERR_UNSUPPORTED;
    p.heads = (int32_t)heads;
    p.tokens = T_tokens;
    // A block moves about WORK units a thread, which pays for its start, sines and barrier: that many tokens,
    // as far as their sines fit (16 KB) and two blocks an SM remain.  Fewer tokens than that are split over
    // their heads, down to one unit a thread.  Measured: 16384 tokens of 128 heads of 128 at 16, 8 and 4 units
    // a thread 168, 175 and 192 us; 32768 latent rows 21 us, at a block a token 97 us.
    int64_t per = WORK * ROPE_THREADS / total;
    const int64_t fit = p.dim ? 4096 / p.dim : MAX_TOKENS, spread = T_tokens / (2 * (int64_t)sm_count);
    for (const int64_t x : {fit, spread, (int64_t)MAX_TOKENS}) per = x < per ? x : per;
    p.per_block = per > 1 ? (int32_t)per : 1;
    int64_t split = 1;
    if (p.per_block == 1) {
        const int64_t most = (total + ROPE_THREADS - 1) / ROPE_THREADS;
        split = (2 * (int64_t)sm_count + T_tokens - 1) / T_tokens;
        const int64_t full = total / (WORK * ROPE_THREADS);  // long tokens: WORK units a thread here too
        split = split > full ? split : full;
        split = split < most ? split : most;
        split = split < heads ? split : heads;
        split = split < 1 ? 1 : split > 65535 ? 65535 : split;
    }
    p.part = (int32_t)((heads + split - 1) / split);
    split = (heads + p.part - 1) / p.part;
    const unsigned blocks = (unsigned)((T_tokens + p.per_block - 1) / p.per_block);
    const size_t smem = (size_t)p.per_block * (p.dim / 2) * sizeof(float2);
    auto fn = move_heads_kernel<T, VEC, INTER>;
    // (without asking, a kernel has 48 KB, its static shared memory among them)
    if (smem + sizeof(Dest) * MAX_TOKENS > 48 * 1024 && !ensure_smem(reinterpret_cast<const void *>(fn), (int)smem))
        return DSA_ERR_UNSUPPORTED;
    fn<<<dim3(blocks, (unsigned)split), ROPE_THREADS, smem, st>>>(p);
    return cudaGetLastError() == cudaSuccess ? DSA_OK : DSA_ERR_CUDA;
}

bool vec_ok(const Seg &g) {
    const uintptr_t in = reinterpret_cast<uintptr_t>(g.in), out = reinterpret_cast<uintptr_t>(g.out);
    return !(in & 15) && !(out & (g.e4m3 ? 7 : 15)) && !(g.D & 7) && !((g.in_token | g.in_head) & 7) &&
           !((g.out_token | g.out_head | g.out_page | g.out_row) & 7);
}

dsa_status launch_any(MoveParams &p, const dsa_rope_spec *rope, int T, int dtype, cudaStream_t st) {
    const DeviceInfo *dev = current_device();
    if (!dev) return DSA_ERR_CUDA;
    p.err = dev->err;
    const bool inter = rope && rope->layout == DSA_ROPE_INTERLEAVED;
    p.inv_freq = rope ? rope->inv_freq : nullptr;
    p.dim = rope ? rope->dim : 0;
    p.offset = rope ? rope->offset : 0;
    p.factor = rope ? rope->factor : 1.f;
    p.sin_sign = rope && rope->inverse ? -1.f : 1.f;
    bool vec = !(p.dim & 15) && !(p.offset & 7);
    for (int s = 0; s < p.nseg; ++s) vec = vec && vec_ok(p.seg[s]);
    const int sms = dev->sm_count;
#define DSA_MOVE(TYPE)                                                                            \
    return vec ? (inter ? launch_move<TYPE, 8, true>(p, T, sms, st) : launch_move<TYPE, 8, false>(p, T, sms, st)) \
               : (inter ? launch_move<TYPE, 1, true>(p, T, sms, st) : launch_move<TYPE, 1, false>(p, T, sms, st))
    if (dtype == DSA_BF16) DSA_MOVE(__nv_bfloat16);
    DSA_MOVE(__half);
#undef DSA_MOVE
}

Seg heads_seg(const HeadsIn &in, const HeadsOut &out, int D) {
    Seg g{};
    g.in = in.data, g.out = out.data;
    g.in_token = in.token_stride, g.in_head = in.heads > 1 ? in.head_stride : 0;
    g.out_token = out.token_stride, g.out_head = in.heads > 1 ? out.head_stride : 0;
    g.heads = in.heads, g.D = D, g.rot = 1, g.scale = 1.f;
    return g;
}

}  // namespace

dsa_status launch_rope(const RopeArgs &a, cudaStream_t st) {
    MoveParams p{};
    if (a.q.heads) p.seg[p.nseg++] = heads_seg(a.q, a.q_out, a.D);
    if (a.k.heads) p.seg[p.nseg++] = heads_seg(a.k, a.k_out, a.D);
    p.pos = a.pos;
    return launch_any(p, a.rope, a.T, a.dtype, st);
}

dsa_status launch_append_rope(const AppendRopeArgs &a, cudaStream_t st) {
    MoveParams p{};
    const dsa_kv_cache &c = *a.cache;
    const bool e4m3 = c.dtype == DSA_E4M3;
    Seg k = heads_seg(a.k, HeadsOut{c.k, 0, c.k_head_stride}, c.Dk);
    k.out_page = a.pg.num_pages > 1 ? c.k_page_stride : 0, k.out_row = c.k_row_stride, k.paged = 1, k.e4m3 = e4m3;
    k.scale = c.k_scale, k.rot = a.rope != nullptr;
    p.seg[p.nseg++] = k;
    if (a.v.heads) {
        Seg v = heads_seg(a.v, HeadsOut{c.v, 0, c.v_head_stride}, c.Dv);
        v.out_page = a.pg.num_pages > 1 ? c.v_page_stride : 0, v.out_row = c.v_row_stride, v.paged = 1, v.e4m3 = e4m3;
        v.scale = c.v_scale, v.rot = 0;
        p.seg[p.nseg++] = v;
    }
    if (a.q.heads) p.seg[p.nseg++] = heads_seg(a.q, a.q_out, c.Dk);
    p.pos = a.tok_pos, p.tok_seq = a.tok_seq, p.pg = a.pg;
    return launch_any(p, a.rope, a.n, a.dtype, st);
}

}  // namespace dsa
