// Sharing the work of dsa_paged_attn out over CTAs.
//
// A tile is TM packed rows of one sequence and one K/V head: row r is query
// head (r % G) of the group and the sequence's new token r / G, so all query
// heads that share a K/V head share its loads.  (Within a window, chunks' tiles
// may begin at multiples of `align` positions, a sequence's first tile having
// fewer rows: a row block then touches one key unit less, more often than not.)  Its work is the run of units
// (UNIT consecutive key positions, aligned) that its rows see.  All tiles'
// units, in the order sequence, head, tile, unit, form one line, which is cut
// into equal parts, one per CTA: whatever the mix of lengths, every CTA gets
// the same number of units, and a long sequence of few heads is split over as
// many CTAs as it takes.  A CTA that holds a tile whole writes its rows;
// pieces of a tile go to the workspace (at most two per CTA: one that began
// in an earlier CTA, one that goes on in the next) and are joined by a second
// kernel in the order of the line.  Where the heads divide the CTAs (`locked`),
// every head has a line of its own and the CTAs of one part of all of them read
// the same pages at the same time, so that the rows of a page, which lie
// interleaved by heads, come from memory together.  Lengths are read on the device: every CTA
// sums the units of all sequences itself, tile by tile where a sequence has several, and again to find its place where
// there are more than 1024 sequences; a cost that grows with both, spread over the block's warps.  The result depends
// on nothing but the lengths.
#pragma once

#include "dsa_device.cuh"
#include "dsa_internal.h"

namespace dsa {

struct PagedAttnParams {
    const void *q;
    int64_t q_token, q_head;
    const int32_t *q_start;
    PagedDev pg;
    int32_t T, H, Hkv, G, TM;  // T H < 2^31 - 512
    int32_t align;             // tokens; 0: a tile begins wherever the last one ended
    int32_t locked;            // a line a head: CTA c is part c / Hkv of head c % Hkv
    FastDiv by_G, by_TM;
    int32_t max_q, max_len, window;
    float scale_log2;  // sm_scale * log2(e) (and 1 / k_scale)
    float v_inv;       // 1 / v_scale
    void *out;
    float *lse;
    float *part_o;   // [CTAs][2][TM][D]: normalised partial outputs
    float *part_l;   // [CTAs][2][TM]: log2 of the sum of exponentials
    struct PieceRec *rec;  // [CTAs]
    uint32_t *err;
};

// A tile that began in this CTA and goes on in the next ones.
struct PieceRec {
    int32_t valid, q0, h, row0, rows;  // the sequence's first row of q; the K/V head; packed rows
    int64_t end, total;                // where the tile's units end on the line; the line's length
};

struct SeqInfo {
    int n, L, q0;  // new tokens, length, first row of q
    int shift;     // packed rows that the first tile goes without
};
__device__ __forceinline__ SeqInfo seq_info(const PagedAttnParams &p, int b, bool report = false) {
    SeqInfo s;
    s.L = max(p.pg.seq_lens[b], 0);
    uint32_t bad = 0;
    if (p.q_start) {
        s.q0 = p.q_start[b];
        const int64_t n = (int64_t)p.q_start[b + 1] - s.q0;
        if (s.q0 < 0 || n < 0 || s.q0 + n > p.T || n > p.max_q) bad = DSA_DEVERR_SHAPE;
        s.n = (int)n;
    } else {
        s.q0 = b;
        s.n = 1;
    }
    if (s.L > p.max_len) bad = DSA_DEVERR_SHAPE;
    if (bad) {
        if (report) record_error(p.err, bad);
        s.n = 0;
    }
    s.shift = p.align && s.L > s.n ? (s.L - s.n) % p.align * p.G : 0;
    return s;
}

struct Tile {
    int row0, rows;        // packed rows
    int base;              // where they would begin without a shift's limit (at most row0)
    int p_first, p_last;   // positions of its first and last token (below 0: no such position)
    int key_lo, key_hi;    // positions that some row sees
    int u0, nu;            // units
};
template <int UNIT>
__device__ __forceinline__ Tile tile_info(const PagedAttnParams &p, const SeqInfo &s, int t) {
    Tile x;
    const int total = s.n * p.G;
    x.base = t * p.TM - s.shift;
    x.row0 = max(x.base, 0);
    x.rows = min(x.base + p.TM, total) - x.row0;
    x.p_first = s.L - s.n + p.by_G.div(x.row0);
    x.p_last = s.L - s.n + p.by_G.div(x.row0 + x.rows - 1);
    x.key_hi = max(x.p_last + 1, 0);
    x.key_lo = p.window ? max(x.p_first - p.window + 1, 0) : 0;
    x.u0 = x.key_lo / UNIT;
    x.nu = max((x.key_hi + UNIT - 1) / UNIT - x.u0, 1);  // a tile that sees nothing has one unit, for its zeros
    return x;
}
__device__ __forceinline__ int seq_tiles(const PagedAttnParams &p, const SeqInfo &s) {
    return s.n ? p.by_TM.div(s.n * p.G + s.shift - 1) + 1 : 0;
}

__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {  // a >= 0, b > 0; short where both are
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}
// A line's parts: the first `more` have per + 1 units, the others per.
struct Line {
    int64_t per;
    int more;
    __device__ __forceinline__ Line(int64_t total, int nc) {
        per = div64(total, nc);
        more = (int)(total - per * nc);
    }
    __device__ __forceinline__ int64_t start(int c) const { return per * c + min(c, more); }
    // the first part that begins at or behind `at`
    __device__ __forceinline__ int next(int64_t at) const {
        const int64_t big = (per + 1) * more;
        if (at <= big) return (int)div64(at + per, per + 1);
        return more + (int)(per > 0 ? div64(at - big + per - 1, per) : 0);
    }
};

// How many parts a line has, and which one CTA c of nc holds.
__device__ __forceinline__ int line_parts(const PagedAttnParams &p, int nc) { return p.locked ? nc / p.Hkv : nc; }
__device__ __forceinline__ int line_part(const PagedAttnParams &p, int c) { return p.locked ? c / p.Hkv : c; }

struct Cursor {
    int b, h, t, u;   // sequence, K/V head, tile, unit of the tile
    int64_t at, end;  // this place on the line, and the CTA's end
    int64_t total;
};

constexpr int PLAN_SEQS = 1024;
struct PlanShared {
    int64_t units[PLAN_SEQS];  // per sequence, one head
    int64_t total;
    Cursor cur;
    int found;
};

// Where CTA c begins.  All threads of the block; a barrier of the block is among it.
template <int UNIT>
__device__ Cursor plan_cta(const PagedAttnParams &p, int c, int nc, PlanShared &sh) {
    const int lane = lane_id(), warp = warp_id(), nw = blockDim.x >> 5;
    const int B = p.pg.num_seqs;
    const bool single = ((int64_t)p.max_q + p.align) * p.G <= p.TM;  // one tile a sequence at most
    const int lines = p.locked ? 1 : p.Hkv;              // heads on this CTA's line
    const int head = p.locked ? c % p.Hkv : 0, parts = line_parts(p, nc), part = line_part(p, c);
    if (single && B <= 32) {
        // small batches of single tokens, where the plan's latency counts: every warp by itself, a lane a sequence
        int64_t per_head = 0;
        if (lane < B) {
            const SeqInfo s = seq_info(p, lane, c == 0 && warp == 0);
            if (s.n) per_head = tile_info<UNIT>(p, s, 0).nu;
        }
        const int64_t w = per_head * lines;
        int64_t inc = w;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
            if (lane >= o) inc += v;
        }
        const int64_t total = __shfl_sync(0xffffffffu, inc, 31);
        const Line line(total, parts);
        Cursor cur{0, head, 0, 0, line.start(part), line.start(part + 1), total};
        const uint32_t past = __ballot_sync(0xffffffffu, inc > cur.at);
        if (cur.at < cur.end && past) {
            cur.b = __ffs(past) - 1;
            const int64_t off = cur.at - __shfl_sync(0xffffffffu, inc - w, cur.b);
            const int64_t ph = __shfl_sync(0xffffffffu, per_head, cur.b);
            const int h = (int)div64(off, ph);
            cur.h += h;
            cur.u = (int)(off - h * ph);
        }
        __syncthreads();
        return cur;
    }
    auto fill = [&](int base, bool report) {
        const int cnt = min(PLAN_SEQS, B - base);
        if (single) {
            for (int i = threadIdx.x; i < cnt; i += blockDim.x) {
                const SeqInfo s = seq_info(p, base + i, report);
                sh.units[i] = s.n ? tile_info<UNIT>(p, s, 0).nu : 0;
            }
        } else {
            for (int i = warp; i < cnt; i += nw) {
                const SeqInfo s = seq_info(p, base + i, report && lane == 0);
                const int nt = seq_tiles(p, s);
                int64_t sum = 0;
                for (int t = lane; t < nt; t += 32) sum += tile_info<UNIT>(p, s, t).nu;
#pragma unroll
                for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                if (lane == 0) sh.units[i] = sum;
            }
        }
        __syncthreads();
        return cnt;
    };
    if (threadIdx.x == 0) sh.total = 0, sh.found = 0;
    for (int base = 0; base < B; base += PLAN_SEQS) {
        const int cnt = fill(base, c == 0);
        if (warp == 0) {
            int64_t sum = 0;
            for (int i = lane; i < cnt; i += 32) sum += sh.units[i];
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
            if (lane == 0) sh.total += sum * lines;
        }
        __syncthreads();
    }
    const int64_t total = sh.total;
    const Line line(total, parts);
    const int64_t begin = line.start(part), end = line.start(part + 1);
    if (threadIdx.x == 0) sh.cur = Cursor{0, head, 0, 0, begin, end, total};
    __syncthreads();
    if (begin >= end) return sh.cur;
    int64_t before = 0;  // warp 0: units before the group of 32 sequences looked at
    for (int base = 0; base < B; base += PLAN_SEQS) {
        const int cnt = B > PLAN_SEQS ? fill(base, false) : B;
        if (warp == 0) {
            for (int g = 0; g < cnt; g += 32) {
                const int64_t w = g + lane < cnt ? sh.units[g + lane] * lines : 0;
                int64_t inc = w;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int64_t v = __shfl_up_sync(0xffffffffu, inc, o);
                    if (lane >= o) inc += v;
                }
                const uint32_t past = __ballot_sync(0xffffffffu, before + inc > begin);
                if (past) {
                    const int l = __ffs(past) - 1;
                    const int b = base + g + l;
                    const int64_t per_head = sh.units[g + l];
                    int64_t off = begin - before - __shfl_sync(0xffffffffu, inc - w, l);
                    const int h = (int)div64(off, per_head);
                    off -= h * per_head;
                    const SeqInfo s = seq_info(p, b);
                    const int nt = seq_tiles(p, s);
                    int64_t sum = 0;
                    for (int t0 = 0; t0 < nt; t0 += 32) {
                        const int64_t nu = t0 + lane < nt ? tile_info<UNIT>(p, s, t0 + lane).nu : 0;
                        int64_t ti = nu;
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const int64_t v = __shfl_up_sync(0xffffffffu, ti, o);
                            if (lane >= o) ti += v;
                        }
                        const uint32_t tp = __ballot_sync(0xffffffffu, sum + ti > off);
                        if (tp) {
                            const int tl = __ffs(tp) - 1;
                            if (lane == tl) {
                                sh.cur.b = b, sh.cur.h = head + h, sh.cur.t = t0 + tl;
                                sh.cur.u = (int)(off - sum - (ti - nu));
                                sh.found = 1;
                            }
                            break;
                        }
                        sum += __shfl_sync(0xffffffffu, ti, 31);
                    }
                    break;
                }
                before += __shfl_sync(0xffffffffu, inc, 31);
            }
        }
        __syncthreads();
        if (sh.found) break;
    }
    __syncthreads();
    return sh.cur;
}

// A run of units of one tile that a CTA works on.
struct Segment {
    SeqInfo s;
    Tile x;
    int b, h, t;
    int u_begin, u_end;  // of the tile's units
    __device__ __forceinline__ bool whole() const { return u_begin == 0 && u_end == x.nu; }
    __device__ __forceinline__ int slot() const { return u_begin == 0 ? 1 : 0; }  // of the CTA's two pieces
};
// The next segment, or false at the CTA's end.  Every role of a CTA walks the
// same segments with its own copy of the cursor.
template <int UNIT>
__device__ __forceinline__ bool next_segment(const PagedAttnParams &p, Cursor &c, Segment &g) {
    if (c.at >= c.end) return false;
    g.s = seq_info(p, c.b);
    int nt = seq_tiles(p, g.s);
    while (c.t >= nt) {  // the cursor stands behind a head's last tile, or at a sequence without rows
        c.t = 0;
        if (nt == 0 || p.locked || ++c.h == p.Hkv) {
            if (!p.locked) c.h = 0;
            if (++c.b >= p.pg.num_seqs) return false;  // the lengths changed under the call
            g.s = seq_info(p, c.b);
            nt = seq_tiles(p, g.s);
        }
    }
    g.x = tile_info<UNIT>(p, g.s, c.t);
    g.b = c.b, g.h = c.h, g.t = c.t;
    g.u_begin = c.u;
    const int64_t left = c.end - c.at;
    g.u_end = left < g.x.nu - c.u ? c.u + (int)left : g.x.nu;
    c.at += g.u_end - g.u_begin;
    c.u = 0;
    ++c.t;
    return true;
}

}  // namespace dsa
