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
// tokens go, then move 16-byte vectors, a pair of vectors for a rotated unit,
// two units of each thread in flight.  The first units' loads are issued
// before the sines, the page lookup and the barrier, whose latency they hide.
// HBM-bound: each element is read and written once.
#include <cuda_fp16.h>
#include <math.h>

#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {
namespace {

constexpr int ROPE_THREADS = 256;
constexpr int MAX_SEG = 3;

// One array of heads: where its tokens' heads come from, where they go.
struct Seg {
    const void *in;
    void *out;
    int64_t in_token, in_head, out_token, out_head;  // elements
    int64_t out_page, out_row;                       // paged destinations (paged != 0)
    int32_t heads, D;
    FastDiv by_units;
    int32_t units;   // per head: rotated ones first, then copied ones
    int32_t rot;     // rotated units per head (0: copied whole)
    int32_t paged, e4m3;
    float scale;
};

struct MoveParams {
    Seg seg[MAX_SEG];
    int32_t nseg, tokens;
    int32_t per_block;  // tokens per block
    int32_t part;       // units of each of them that a block moves
    int32_t total;      // units per token, all segments
    FastDiv by_part;
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

// Where a unit lies: its segment, head and elements.  A rotated unit is two
// vectors: elements e0.. and e1.. (the pair partners in the half layout,
// neighbours in the interleaved one); a copied one is the vector at e0.
struct Unit {
    int seg, head, e0, e1, pair;  // pair < 0: copied; else the first pair's index
};

template <int VEC, bool INTER>
__device__ __forceinline__ Unit unit_of(const MoveParams &p, int u) {
    Unit r;
    r.seg = 0;
#pragma unroll
    for (int s = 0; s < MAX_SEG - 1; ++s) {
        const int n = p.seg[s].heads * p.seg[s].units;
        if (r.seg == s && s + 1 < p.nseg && u >= n) u -= n, r.seg = s + 1;
    }
    const Seg &g = p.seg[r.seg];
    r.head = g.by_units.div(u);
    const int x = u - r.head * g.units;
    if (x < g.rot) {
        r.pair = x * VEC;
        r.e0 = p.offset + (INTER ? 2 * x * VEC : x * VEC);
        r.e1 = INTER ? r.e0 + VEC : r.e0 + p.dim / 2;
    } else {
        int e = (x - g.rot) * VEC;
        if (g.rot && e >= p.offset) e += p.dim;  // past the rotated part
        r.pair = -1, r.e0 = e, r.e1 = e;
    }
    return r;
}

constexpr int MAX_TOKENS = 32;  // per block
struct Dest {
    int64_t page;  // -1: nothing is written for the token
    int row;
};

// One unit on its way: read by fetch(), turned and written by put().
template <typename T, int VEC, bool INTER>
struct Moving {
    Unit un;
    int token;  // of the block
    Vec<T, VEC> a, b;

    __device__ __forceinline__ void fetch(const MoveParams &p, int t0, int u) {
        token = p.by_part.div(u);
        un = unit_of<VEC, INTER>(p, blockIdx.y * p.part + u - token * p.part);
        const Seg &g = p.seg[un.seg];
        const T *src = static_cast<const T *>(g.in) + (t0 + token) * g.in_token + un.head * g.in_head;
        a.load(src + un.e0);
        b.load(src + un.e1);
    }
    __device__ __forceinline__ void put(const MoveParams &p, int t0, const float2 *cs_all, const Dest *dest) {
        const Seg &g = p.seg[un.seg];
        int64_t at = (int64_t)un.head * g.out_head;
        if (p.tok_seq) {
            const Dest d = dest[token];
            if (d.page < 0) return;
            if (g.paged) at += d.page * g.out_page + d.row * g.out_row;
        }
        if (!g.paged) at += (t0 + token) * g.out_token;
        if (un.pair < 0 && !g.e4m3) {
            a.copy(static_cast<T *>(g.out) + at + un.e0);
            return;
        }
        const float2 *cs = cs_all + token * (p.dim / 2) + un.pair;
        float x[VEC], y[VEC];
        a.floats(x);
        b.floats(y);
        if (un.pair >= 0) {
            if (INTER && VEC == 1) {
                const float2 w = cs[0];
                const float x0 = x[0], y0 = y[0];
                x[0] = x0 * w.x - y0 * w.y;
                y[0] = y0 * w.x + x0 * w.y;
            } else if (INTER) {
                // pairs lie next to each other: x holds VEC / 2 of them, y the next VEC / 2
#pragma unroll
                for (int i = 0; i + 1 < VEC; i += 2) {
                    const float2 w = cs[i / 2], z = cs[VEC / 2 + i / 2];
                    const float x0 = x[i], x1 = x[i + 1], y0 = y[i], y1 = y[i + 1];
                    x[i] = x0 * w.x - x1 * w.y;
                    x[i + 1] = x1 * w.x + x0 * w.y;
                    y[i] = y0 * z.x - y1 * z.y;
                    y[i + 1] = y1 * z.x + y0 * z.y;
                }
            } else {
#pragma unroll
                for (int i = 0; i < VEC; ++i) {
                    const float2 w = cs[i];
                    const float x0 = x[i], y0 = y[i];
                    x[i] = x0 * w.x - y0 * w.y;
                    y[i] = y0 * w.x + x0 * w.y;
                }
            }
        }
        if (g.e4m3) {
            uint8_t *o = static_cast<uint8_t *>(g.out) + at;
            Vec<T, VEC>::store8(o + un.e0, x, g.scale);
            if (un.pair >= 0) Vec<T, VEC>::store8(o + un.e1, y, g.scale);
        } else {
            T *o = static_cast<T *>(g.out) + at;
            Vec<T, VEC>::store(o + un.e0, x);
            Vec<T, VEC>::store(o + un.e1, y);
        }
    }
};

// cos and sin of the block's tokens, [tokens][dim/2], in dynamic shared memory.
template <typename T, int VEC, bool INTER>
__global__ void __launch_bounds__(ROPE_THREADS) move_heads_kernel(const __grid_constant__ MoveParams p) {
    extern __shared__ float2 cs[];
    __shared__ Dest dest[MAX_TOKENS];
    const int t0 = blockIdx.x * p.per_block, nt = min(p.per_block, p.tokens - t0);
    const int units = nt * min(p.part, p.total - (int)blockIdx.y * p.part);  // (parts are whole, or one token's last)
    int u = threadIdx.x;
    Moving<T, VEC, INTER> a, b;
    if (u < units) a.fetch(p, t0, u);
    if (u + ROPE_THREADS < units) b.fetch(p, t0, u + ROPE_THREADS);
    if (p.tok_seq && threadIdx.x < nt) {
        const int t = t0 + threadIdx.x, s = p.tok_seq[t], pos = p.pos[t];
        Dest d{-1, 0};
        if (s != -1) {  // (-1: padding)
            uint32_t bad = 0;
            if (s < 0 || s >= p.pg.num_seqs || pos < 0 || pos >= p.pg.seq_lens[s]) {
                bad = DSA_DEVERR_POSITION;
            } else {
                const int lp = pos >> 6;
                d.page = lp < p.pg.max_blocks ? p.pg.block_table[(int64_t)s * p.pg.max_blocks + lp] : -1;
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
    const int half = p.dim / 2;
    for (int i = threadIdx.x; i < nt * half; i += ROPE_THREADS) {
        const int t = i / half;
        const double turns = (double)p.pos[t0 + t] * p.inv_freq[i - t * half] * 0.15915494309189535;  // 1 / 2 pi
        float sn, c;
        sincospif(2.f * (float)(turns - rint(turns)), &sn, &c);
        cs[i] = make_float2(c * p.factor, sn * p.factor * p.sin_sign);
    }
    __syncthreads();
    while (u < units) {
        a.put(p, t0, cs, dest);
        if (u + ROPE_THREADS < units) b.put(p, t0, cs, dest);
        u += 2 * ROPE_THREADS;
        if (u < units) a.fetch(p, t0, u);
        if (u + ROPE_THREADS < units) b.fetch(p, t0, u + ROPE_THREADS);
    }
}

template <typename T, int VEC, bool INTER>
dsa_status launch_move(MoveParams &p, int T_tokens, int sm_count, cudaStream_t st) {
    int64_t total = 0;
    for (int s = 0; s < p.nseg; ++s) {
        Seg &g = p.seg[s];
        g.rot = g.rot ? p.dim / (2 * VEC) : 0;
        // heads rotated in place leave their other elements where they are
        const bool still = g.in == g.out && !g.paged && g.rot;
        g.units = g.rot + (still ? 0 : (g.D - (g.rot ? p.dim : 0)) / VEC);
        g.by_units = FastDiv::of(g.units > 0 ? g.units : 1);
        total += (int64_t)g.heads * g.units;
    }
    if (total == 0 || T_tokens == 0) return DSA_OK;
    if (total > (1 << 26)) return DSA_ERR_UNSUPPORTED;
    p.total = (int32_t)total;
    p.tokens = T_tokens;
    // A block moves about four units a thread: that many tokens, as far as their sines fit (16 KB) and two
    // blocks an SM remain.  Fewer tokens than that are split over their heads, down to one unit a thread.
    // (32768 latent rows, 68 units each: 97 us with a block a token.)
    int64_t per = 4 * ROPE_THREADS / total;
    const int64_t fit = p.dim ? 4096 / p.dim : MAX_TOKENS, spread = T_tokens / (2 * (int64_t)sm_count);
    for (const int64_t x : {fit, spread, (int64_t)MAX_TOKENS}) per = x < per ? x : per;
    p.per_block = per > 1 ? (int32_t)per : 1;
    int64_t split = 1;
    if (p.per_block == 1) {
        const int64_t most = (total + ROPE_THREADS - 1) / ROPE_THREADS;
        split = (2 * (int64_t)sm_count + T_tokens - 1) / T_tokens;
        const int64_t full = total / (4 * ROPE_THREADS);  // long tokens: four units a thread here too
        split = split > full ? split : full;
        split = split < most ? split : most;
        split = split < 1 ? 1 : split > 65535 ? 65535 : split;
    }
    p.part = (int32_t)((total + split - 1) / split);
    p.by_part = FastDiv::of(p.part);
    split = (total + p.part - 1) / p.part;
    const unsigned blocks = (unsigned)((T_tokens + p.per_block - 1) / p.per_block);
    const size_t smem = (size_t)p.per_block * (p.dim / 2) * sizeof(float2);
    auto fn = move_heads_kernel<T, VEC, INTER>;
    if (smem > 48 * 1024 && !ensure_smem(reinterpret_cast<const void *>(fn), (int)smem)) return DSA_ERR_UNSUPPORTED;
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
