"""Attention of new tokens over a paged K/V cache against its 64-bit form, on the GPU."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_rope import BF16, F16, L, gen, no_error, paged_case, randn  # noqa: F401

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn
KS, VS = 24.0, 40.0


class Case:
    """Sequences of lens with new tokens each; K/V rows past every length (and unused pages) hold NaN."""

    def __init__(self, L, lens, new, H, Hkv, D, dtype=BF16, cdt=None, order="rows", seed=0, spare=0):
        g = gen(seed + sum(lens) + H)
        self.L, self.lens, self.new, self.H, self.D, self.dtype = L, lens, new, H, D, dtype
        self.cdt = cdt or dtype
        self.seq_lens, self.table, self.pages = paged_case(g, lens)
        self.T = sum(new) + spare
        self.q = randn(g, self.T, H, D, dtype=dtype)
        self.q_start = torch.tensor([sum(new[:b]) for b in range(len(new) + 1)], device="cuda", dtype=torch.int32)

        def make(scale):
            shape = (self.pages, 64, Hkv, D) if order == "rows" else (self.pages, Hkv, 64, D)
            x = torch.randn(shape, generator=g, device="cuda") * (scale if self.cdt == E4M3 else 1.0)
            x = x.to(self.cdt)
            x = x if order == "rows" else x.transpose(1, 2)
            bits = x.view(torch.uint8) if self.cdt == E4M3 else x
            live = torch.zeros(self.pages, 64, device="cuda", dtype=torch.bool)
            for b, n in enumerate(lens):
                p = torch.arange(n, device="cuda")
                live[self.table[b, p // 64].long(), p % 64] = True
            bits[~live] = 0x7F if self.cdt == E4M3 else math.nan
            return x

        self.k, self.v = make(KS), make(VS)
        self.cache = L.kv_cache(self.k, self.v, KS, VS)
        self.pg = L.paged(self.seq_lens, self.table, self.pages)

    def run(self, window=0, sm_scale=None, q=None, **kw):
        kw.setdefault("max_len", max(max(self.lens), 1))
        kw.setdefault("max_q", max(max(self.new), 1))
        return self.L.paged_attn(self.q if q is None else q, self.cache, self.pg, self.q_start, window=window,
                                 sm_scale=sm_scale, want_lse=True, **kw)

    def ref(self, b, window=0, sm_scale=None, rows=None):
        n, m, at = self.lens[b], self.new[b], int(self.q_start[b])
        pos = torch.arange(n - m, n, device="cuda")
        q = self.q[at:at + m]
        if rows is not None:
            pos, q = pos[rows], q[rows]
        return ref.attend(q, ref.gather(self.k, self.table[b], n, KS), ref.gather(self.v, self.table[b], n, VS), pos, window,
                          self.D ** -0.5 if sm_scale is None else sm_scale)

    def check(self, out, lse, window=0, sm_scale=None):
        no_error(self.L)
        for b, m in enumerate(self.new):
            at = int(self.q_start[b])
            if m:
                ref.assert_attended(out[at:at + m], self.ref(b, window, sm_scale), lse[at:at + m],
                                    F16 if self.cdt == E4M3 else None)


SHAPES = [
    # lens, new, H, Hkv, D
    ([1], [1], 1, 1, 64),
    ([4097], [1], 64, 8, 128),
    ([1, 63, 64, 65, 128, 129, 4999], [1] * 7, 8, 1, 128),
    ([300, 20, 77], [4, 1, 3], 40, 8, 64),
    ([300, 1000], [9, 5], 5, 5, 128),
    ([200, 90, 700], [130, 90, 17], 6, 2, 128),   # 390 packed rows, a group of 3
    ([515], [515], 8, 1, 64),
    ([1000, 64, 2000], [257, 64, 1], 4, 4, 128),
    ([150], [150], 96, 1, 64),                     # 96 query heads on one K/V head
    ([260], [40], 160, 1, 128),                    # more heads than a tile has rows
]


@pytest.mark.parametrize("lens,new,H,Hkv,D", SHAPES)
@pytest.mark.parametrize("dtype,cdt", [(BF16, None), (F16, None), (BF16, E4M3), (F16, E4M3)])
def test_attention(L, lens, new, H, Hkv, D, dtype, cdt):  # noqa: F811
    c = Case(L, lens, new, H, Hkv, D, dtype, cdt)
    c.check(*c.run())


@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 129, 1000, 2 ** 31 - 1])
@pytest.mark.parametrize("lens,new,H,Hkv,D,cdt", [([700, 64, 1], [1, 1, 1], 8, 2, 128, None),
                                                  ([700, 64, 90], [300, 64, 3], 6, 2, 128, None),
                                                  ([515, 140], [200, 1], 4, 4, 64, E4M3),
                                                  ([700, 64, 1], [2, 1, 1], 8, 2, 128, E4M3)])
def test_window(L, lens, new, H, Hkv, D, cdt, window):  # noqa: F811
    c = Case(L, lens, new, H, Hkv, D, BF16, cdt)
    c.check(*c.run(window), window)


@pytest.mark.parametrize("n,m", [(255, 128), (256, 128), (257, 257), (700, 573), (700, 572), (1000, 1), (300, 299), (130, 131)])
def test_window_of_aligned_tiles(L, n, m):  # noqa: F811
    """Chunks that begin on, before and behind a multiple of 128, from the sequence's start and from before it."""
    c = Case(L, [n, 200], [m, 150], 3, 3, 128)
    c.check(*c.run(128), 128)


def test_no_tokens(L):  # noqa: F811
    """Calls of no tokens return empty results and launch nothing."""
    c = Case(L, [64], [1], 4, 2, 64)
    freq = L.rope_frequencies(64)[0].cuda()
    none = torch.empty(0, device="cuda", dtype=torch.int32)
    q, kv = torch.empty(0, 4, 64, device="cuda", dtype=BF16), torch.empty(0, 2, 64, device="cuda", dtype=BF16)
    assert L.rope(q, none, L.rope_spec(freq), k=kv)[1].shape == (0, 2, 64)
    assert L.append_rope(kv, kv, none, none, c.pg, c.cache, L.rope_spec(freq), q=q).shape == (0, 4, 64)
    c.q_start.zero_()
    out, lse = L.paged_attn(q, c.cache, c.pg, c.q_start, 1, 64, want_lse=True)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    no_error(L)


def test_two_graphs_share_a_workspace(L):  # noqa: F811
    """Two captured calls of different shapes on one workspace, replayed in turn."""
    a, b = Case(L, [3000, 40], [1, 1], 16, 2, 128), Case(L, [500, 900], [200, 3], 16, 2, 128, seed=3)
    ws = L.paged_attn_workspace(203, 16, b.cache, b.pg, 200, 3000)
    outs, graphs = [], []
    for c in (a, b):
        c.run(ws=ws)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run(ws=ws))
        graphs.append(g)
    for _ in range(3):
        for g in graphs:
            g.replay()
    torch.cuda.synchronize()
    for c, (out, lse) in zip((a, b), outs):
        c.check(out, lse)


@pytest.mark.parametrize("cdt", [None, E4M3])
def test_cache_strides(L, cdt):  # noqa: F811
    """Heads before rows; keys and values as halves of one array; q a slice of a fused projection."""
    c = Case(L, [200, 90], [70, 1], 8, 2, 128, BF16, cdt, order="heads")
    c.check(*c.run())
    both = torch.stack((c.k, c.v), 1)  # [pages, 2, 64, heads, D]
    c.cache = L.kv_cache(both[:, 0], both[:, 1], KS, VS)
    fused = torch.randn(c.T, 12 * 128 + 8, device="cuda").to(BF16)
    fused[:, 128:9 * 128] = c.q.flatten(1)
    got = c.run(q=fused[:, 128:9 * 128].unflatten(1, (8, 128)))
    c.check(*got)
    by_head = c.q.transpose(0, 1).contiguous().transpose(0, 1)
    again = c.run(q=by_head)
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("D", [64, 128])
def test_empty_and_untouched(L, D):  # noqa: F811
    """Sequences without tokens or without history, more queries than history, rows behind the last sequence."""
    lens, new = [0, 100, 3, 0, 70], [2, 0, 5, 1, 70]
    c = Case(L, lens, new, 4, 2, D, spare=3)
    out = torch.full((c.T, 4, D), 5.0, device="cuda", dtype=BF16)
    lse = torch.full((c.T, 4), 5.0, device="cuda")
    c.run(out=out, lse=lse)
    c.check(out, lse)
    none = [0, 1, 2, 3, 7]  # the first sequence, two rows before the third's beginning, the fourth
    assert (out[none] == 0).all() and (lse[none] == -math.inf).all()
    assert (out[78:] == 5.0).all() and (lse[78:] == 5.0).all()
    # a call whose every sequence is empty
    c.q_start.zero_()
    out.fill_(5.0)
    c.run(out=out, lse=lse)
    no_error(L)
    assert (out == 5.0).all()


@pytest.mark.parametrize("new", [1, 90])
def test_one_query_for_all_and_an_odd_output(L, new):  # noqa: F811
    """A query given to every token by a stride of 0, and outputs that begin 16 bytes off a 32-byte boundary."""
    c = Case(L, [300, 90], [new, new], 4, 2, 128)
    one = c.q[:1].expand(c.T, 4, 128)
    c.q = one.contiguous()
    want, lse = c.run()
    c.check(want, lse)
    got, _ = c.run(q=one)
    for b in range(2):
        rows = slice(b * new, (b + 1) * new)
        ref.assert_attended(got[rows], c.ref(b))
    room = torch.zeros(want.numel() + 8, device="cuda", dtype=BF16)
    odd = room[8:].view(want.shape)
    c.run(out=odd)
    no_error(L)
    assert torch.equal(odd, want) and (room[:8] == 0).all()


def test_decode_without_q_start(L):  # noqa: F811
    c = Case(L, [900, 64, 0, 1], [1] * 4, 16, 4, 128)
    want = c.run()
    c.q_start = None
    got = c.run()
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])


def test_freed_pages_before_the_window(L):  # noqa: F811
    """A ring of pages: table entries of pages before the first needed one are not read."""
    c = Case(L, [1000, 700], [40, 1], 4, 2, 128)
    want = c.run(128)
    c.check(*want, 128)
    for b, (n, m) in enumerate(zip(c.lens, c.new)):
        c.table[b, : max(n - m - 128 + 1, 0) // 64] = -7
    got = c.run(128)
    no_error(L)
    assert torch.equal(want[0], got[0])
    c.run(0)
    no_error(L, L.DEVERR_PAGE)


def test_bounds_are_checked_on_the_device(L):  # noqa: F811
    """Sequences over a host bound, or with q_start out of order, are skipped; the others are not."""
    c = Case(L, [300, 500, 200], [3, 2, 4], 8, 2, 64)
    full, _ = c.run()
    for kw, skipped in (({"max_len": 300}, [1]), ({"max_q": 3}, [2])):
        out = torch.full_like(full, 5.0)
        c.run(out=out, **kw)
        no_error(L, L.DEVERR_SHAPE)
        for b in range(3):
            rows = slice(int(c.q_start[b]), int(c.q_start[b + 1]))
            if b in skipped:
                assert (out[rows] == 5.0).all()
            else:
                ref.assert_attended(out[rows], c.ref(b))
    starts = c.q_start.clone()
    for bad in ([0, 3, 2, 9], [-1, 3, 5, 9], [0, 3, 5, 10], [0, 3, 5, -(1 << 31)]):
        c.q_start.copy_(torch.tensor(bad, device="cuda", dtype=torch.int32))
        c.run()
        no_error(L, L.DEVERR_SHAPE)
    c.q_start.copy_(starts)
    c.check(*c.run())


@pytest.mark.parametrize("new,cdt", [(1, None), (1, E4M3), (150, None)])
def test_bad_pages_read_as_zeros(L, new, cdt):  # noqa: F811
    c = Case(L, [200], [new], 2, 1, 64, BF16, cdt)
    c.table[0, 1] = c.pages
    out, lse = c.run()
    no_error(L, L.DEVERR_PAGE)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    c.table[0, 1] = -1
    again, _ = c.run()
    no_error(L, L.DEVERR_PAGE)
    assert torch.equal(out, again)
    c.pg.max_blocks_per_seq = 1  # a table narrower than the sequence
    c.run()
    no_error(L, L.DEVERR_PAGE)


@pytest.mark.parametrize("sm_scale", [0.0, -0.3, 30.0])
def test_scales(L, sm_scale):  # noqa: F811
    c = Case(L, [333], [20], 4, 1, 64)
    c.check(*c.run(sm_scale=sm_scale), 0, sm_scale)


@pytest.mark.parametrize("cdt", [None, E4M3])
def test_large_and_small_queries(L, cdt):  # noqa: F811
    """Rows of q at the ends of bf16's range (an 8-bit cache multiplies in fp16 all the same)."""
    c = Case(L, [150], [6], 2, 1, 64, BF16, cdt)
    c.q[0] *= 1e30
    c.q[1] *= 1e-30
    c.q[2] = 0
    c.q[3] *= 2.0 ** -20
    c.q[3, :, 0] = 1000.0
    out, lse = c.run(sm_scale=0.125)
    no_error(L)
    r = c.ref(0, 0, 0.125)
    # the first row's softmax is one-hot wherever two scores are this far apart
    ref.assert_attended(out[1:6], tuple(x[1:6] for x in r), lse[1:6], F16 if cdt else None)
    ref.assert_attended(out[:1], tuple(x[:1] for x in r[:4]) + (torch.zeros_like(r[4][:1]),), None, F16 if cdt else None)


def test_split_is_deterministic_and_timing_free(L):  # noqa: F811
    """A single long sequence is split over every SM; the result does not change from run to run or with the workspace."""
    c = Case(L, [70000], [1], 8, 1, 128)
    out, lse = c.run()
    c.check(out, lse)
    ws = L.paged_attn_workspace(1, 8, c.cache, c.pg, 1, 70000).fill_(0xFF)
    for _ in range(3):
        o2, l2 = c.run(ws=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2)


def test_many_sequences(L):  # noqa: F811
    """More sequences than one pass of the planner holds, most of them tiny, some empty."""
    g = torch.Generator().manual_seed(5)
    lens = [int(x) for x in torch.randint(0, 90, (2500,), generator=g)]
    new = [int(x) for x in torch.randint(0, 3, (2500,), generator=g)]
    c = Case(L, lens, new, 2, 1, 64)
    out, lse = c.run()
    no_error(L)
    for b in list(range(0, 2500, 97)) + [1023, 1024, 1025, 2047, 2048, 2499]:
        at, m = int(c.q_start[b]), new[b]
        if m:
            ref.assert_attended(out[at:at + m], c.ref(b), lse[at:at + m])


@pytest.mark.parametrize("D,cdt,new,H", [(128, BF16, 1, 16), (128, E4M3, 1, 16), (64, E4M3, 1, 40), (64, BF16, 4, 16),
                                         (128, BF16, 20, 16), (128, E4M3, 4, 24), (128, E4M3, 1, 64)])
def test_long_streams(L, D, cdt, new, H):  # noqa: F811
    """Hundreds of units through each CTA's ring, over gigabytes of cache."""
    lens = [8192 + 1777 * (b % 7) for b in range(48)]
    c = Case(L, lens, [new] * 48, H, 8, D, BF16, cdt)
    out, lse = c.run()
    no_error(L)
    for b in (0, 1, 13, 29, 46, 47):
        rows = slice(b * new, (b + 1) * new)
        ref.assert_attended(out[rows], c.ref(b), lse[rows], F16 if cdt == E4M3 else None)


@pytest.mark.parametrize("Hkv,window,dtype,cdt", [(16, 128, BF16, None), (16, 100, F16, None), (4, 300, BF16, None),
                                                  (2, 0, BF16, None), (16, 128, BF16, E4M3), (2, 0, F16, E4M3),
                                                  (4, 500, BF16, E4M3)])
def test_long_chunks(L, Hkv, window, dtype, cdt):  # noqa: F811
    """Many short segments a CTA, each with keys to leave out at both ends."""
    lens, new = [2048, 3000, 2500, 1300, 4000, 700], [1999, 2000, 1024, 1300, 257, 129]
    c = Case(L, lens, new, 16, Hkv, 128, dtype, cdt)
    out, lse = c.run(window)
    no_error(L)
    for b in range(6):
        at = int(c.q_start[b])
        rows = torch.cat((torch.arange(0, 60), torch.arange(new[b] // 2, new[b] // 2 + 60), torch.arange(new[b] - 9, new[b]))).cuda()
        ref.assert_attended(out[at + rows], c.ref(b, window, rows=rows), lse[at + rows], F16 if cdt else None)


def test_long_offsets(L):  # noqa: F811
    """A cache whose far pages lie past 2^32 bytes and 2^31 elements."""
    pages, Hkv, D = 280000, 1, 128
    k = torch.empty(pages, 64, Hkv, D, device="cuda", dtype=BF16)
    v = torch.empty(pages, 64, Hkv, D, device="cuda", dtype=BF16)
    g = gen(8)
    ids = torch.tensor([[pages - 1, 5, pages - 2, 262143, 262144]], device="cuda", dtype=torch.int32)
    k[ids[0].long()], v[ids[0].long()] = randn(g, 5, 64, Hkv, D), randn(g, 5, 64, Hkv, D)
    cache = L.kv_cache(k, v)
    seq_lens = torch.tensor([310], device="cuda", dtype=torch.int32)
    pg = L.paged(seq_lens, ids, pages)
    freq = L.rope_frequencies(128)[0].cuda()
    kn, vn, q = randn(g, 2, 1, D), randn(g, 2, 1, D), randn(g, 2, 4, D)
    pos = torch.tensor([308, 309], device="cuda", dtype=torch.int32)
    qo = L.append_rope(kn, vn, torch.zeros(2, device="cuda", dtype=torch.int32), pos, pg, cache, L.rope_spec(freq), q=q)
    out, lse = L.paged_attn(qo, cache, pg, torch.tensor([0, 2], device="cuda", dtype=torch.int32), 2, 310, want_lse=True)
    no_error(L)
    kk, vv = ref.gather(k, ids[0], 310), ref.gather(v, ids[0], 310)
    ref.assert_rotated(kk[308:].to(BF16), ref.rotate(kn, pos, freq), kn)
    assert torch.equal(vv[308:], vn.double())
    ref.assert_attended(out, ref.attend(qo, kk, vv, pos, 0, D ** -0.5), lse)


@pytest.mark.parametrize("cdt,window", [(BF16, 128), (torch.uint8, 0)])
def test_a_layer_step_by_step(L, cdt, window):  # noqa: F811
    """The three together as a layer runs them: prompts in chunks, then single tokens, the last ones replayed from a captured
    graph; every output against the 64-bit layer over the whole history."""
    g = gen(21)
    H, Hkv, D, B = 8, 2, 128, 3
    total = [200, 131, 70]
    steps = [[100, 64, 1], [97, 64, 66], [1, 1, 1], [1, 1, 1], [1, 1, 1]]  # tokens of each sequence in each call
    blocks = [-(-n // 64) for n in total]
    pages = sum(blocks)
    table = torch.zeros(B, max(blocks), device="cuda", dtype=torch.int32)
    order, at = torch.randperm(pages, generator=g, device="cuda").int(), 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    kc = torch.empty(pages, 64, Hkv, D, device="cuda", dtype=cdt).fill_(0x7F if cdt == torch.uint8 else math.nan)
    vc = kc.clone()
    cache = L.kv_cache(kc, vc, KS, VS)
    seq_lens = torch.zeros(B, device="cuda", dtype=torch.int32)
    pg = L.paged(seq_lens, table, pages)
    freq, factor = L.rope_frequencies(64, scheme="yarn", scale=8, orig_len=64)
    freq = freq.cuda()
    spec = L.rope_spec(freq, 0, True, factor=factor)
    qkv = [randn(g, n, H + 2 * Hkv, D) for n in total]
    done = [0] * B
    history = [[] for _ in range(B)]

    def call(x, tok_seq, tok_pos, q_start, max_q, ws):
        q = L.append_rope(x[:, H:H + Hkv], x[:, H + Hkv:], tok_seq, tok_pos, pg, cache, spec, q=x[:, :H])
        return L.paged_attn(q, cache, pg, q_start, max_q, 256, window, ws=ws)

    static = None
    for i, new in enumerate(steps):
        x = torch.cat([qkv[b][done[b]:done[b] + m] for b, m in enumerate(new)])
        ints = [torch.tensor(a, device="cuda", dtype=torch.int32) for a in (
            [b for b, m in enumerate(new) for _ in range(m)], [done[b] + j for b, m in enumerate(new) for j in range(m)],
            [sum(new[:b]) for b in range(B + 1)])]
        done = [a + m for a, m in zip(done, new)]
        seq_lens.copy_(torch.tensor(done, device="cuda", dtype=torch.int32))
        if i < 3:
            ws = L.paged_attn_workspace(x.shape[0], H, cache, pg, max(new), 256, window)
            out = call(x, *ints, max(new), ws)
        else:  # the fourth call is captured (which runs nothing) and replayed, the fifth only replayed
            if static is None:
                static = [x.clone(), *[t.clone() for t in ints]]
                ws = L.paged_attn_workspace(B, H, cache, pg, 1, 256, window)
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    out = call(*static, 1, ws)
            for s, t in zip(static, (x, *ints)):
                s.copy_(t)
            graph.replay()
        no_error(L)
        at = 0
        for b, m in enumerate(new):
            history[b].append(out[at:at + m].clone())
            at += m
    for b in range(B):
        n = done[b]
        pos = torch.arange(n, device="cuda")
        k, v = ref.gather(kc, table[b], n, KS), ref.gather(vc, table[b], n, VS)
        if cdt == BF16:  # what the cache holds is the rotated history
            ref.assert_rotated(k.to(BF16), ref.rotate(qkv[b][:n, H:H + Hkv], pos, freq, 0, True, False, factor),
                               qkv[b][:n, H:H + Hkv], factor)
        q = L.rope(qkv[b][:n, :H], pos.int(), spec)[0]  # as the append rotated it
        ref.assert_attended(torch.cat(history[b]), ref.attend(q, k, v, pos, window, D ** -0.5), None,
                            F16 if cdt == torch.uint8 else None)


def test_two_streams(L):  # noqa: F811
    """Two calls at once, each with its own workspace."""
    a, b = Case(L, [5000, 300], [1, 1], 16, 2, 128), Case(L, [400, 900], [200, 150], 4, 2, 64, seed=7)
    torch.cuda.synchronize()
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = []
    for _ in range(4):
        for s, c in zip(streams, (a, b)):
            with torch.cuda.stream(s):
                got.append((c, c.run()))
    torch.cuda.synchronize()
    for c, (out, lse) in got:
        c.check(out, lse)
