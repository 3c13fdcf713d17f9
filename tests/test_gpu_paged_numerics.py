"""Paged attention where its numbers are hardest, on the GPU, through each of its kernels."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attn import E4M3, VS, Case
from tests.test_gpu_rope import BF16, F16, L, gen, no_error  # noqa: F401

pytestmark = pytest.mark.gpu


# query heads on one K/V head and new tokens that reach each kernel: up to 8 rows over an 8-bit cache, row groups of 16,
# the tensor cores
KERNELS = [(BF16, E4M3, 8, 1), (F16, E4M3, 8, 1), (F16, None, 8, 1), (F16, None, 4, 8), (BF16, E4M3, 8, 6), (F16, None, 8, 16),
           (BF16, E4M3, 8, 16), (F16, E4M3, 5, 40), (BF16, None, 8, 1), (BF16, None, 8, 16)]


@pytest.mark.parametrize("cdt", [None, E4M3])
@pytest.mark.parametrize("G", [3, 5, 8])
def test_rows_that_are_not_there(L, G, cdt):  # noqa: F811
    """Groups that do not divide 128 leave rows of a row block without a query, and a last tile's rows lie past the
    sequence: neither what an earlier call left in shared memory nor what q holds behind the last sequence reaches the
    results, which are the same bits each time."""
    c = Case(L, [8000], [1003], 2 * G, 2, 128, BF16, cdt, spare=40)
    before = Case(L, [8000], [1000], 16, 2, 128, BF16, cdt)
    want = None
    for scale in (0.0, 1000.0, 0.01, -30.0):
        c.q[1003:] = c.q[:40] * scale
        before.run(q=before.q * scale)
        out, lse = c.run()
        no_error(L)
        want = want or (out[:1003], lse[:1003])
        assert torch.equal(out[:1003], want[0]) and torch.equal(lse[:1003], want[1])


@pytest.mark.parametrize("depth", [13.7, 23.6, 25.5])
@pytest.mark.parametrize("dtype,cdt,G,new", KERNELS)
def test_concentrated_weights(L, dtype, cdt, G, new, depth):  # noqa: F811
    """One key in 32 holds nearly all of the weight and has a value of 0; the others, `depth` octaves below, make the
    output.  A weight is rounded once to the products' type; of fp16's, what lies 35 octaves below the largest is lost."""
    D, n = 128, 4096
    c = Case(L, [n], [new], G, 1, D, dtype, cdt)
    pages = c.table[0].long()
    g = gen(int(depth) + new)
    k = torch.randn(n, D, generator=g, device="cuda") * 0.05 * 8
    k[::32] = 8.0  # the sinks; every query is all ones
    v = torch.rand(n, D, generator=g, device="cuda") * 500 + 250
    v[::32] = 0
    ks, vs = (24.0, 0.25) if cdt else (1.0, 1.0)
    for x, y, s in ((c.k, k, ks), (c.v, v, vs)):
        x.view(torch.uint8 if cdt else x.dtype)[pages] = (y * s).to(c.cdt).reshape(-1, 64, 1, D).view(
            torch.uint8 if cdt else x.dtype)
    c.cache = L.kv_cache(c.k, c.v, ks, vs)
    c.q.fill_(1.0)
    sm = depth * math.log(2) / (8 * D)
    out, lse = c.run(sm_scale=sm)
    no_error(L)
    kd, vd = ref.gather(c.k, c.table[0], n, ks)[:, 0], ref.gather(c.v, c.table[0], n, vs)[:, 0]
    s = kd.sum(-1) * sm
    for t in range(new):
        m = n - new + t + 1
        w = torch.exp(s[:m] - s[:m].max())
        want = (w @ vd[:m]) / w.sum()
        half = ref.HALF_STEP[F16 if cdt else dtype]
        # weights: one rounding, and 2^-35 of the largest (half of fp16's smallest step, 2^-25, of weights that are lifted
        # by 2^10 at least); scores: an fp32 product of D terms, as in assert_attended; the output's rounding, also among
        # fp16's smallest numbers
        ds = (D + 4) * 2.0 ** -24 * float((kd[:m].abs().sum(-1) * sm).max())
        tol = (half + 2 * ds + 2.0 ** -18 + ref.HALF_STEP[dtype]) * 1.01 * want + 2.0 ** -35 * vd[:m].sum(0) / w.sum() + 2.0 ** -25
        err = (out[t].double() - want).abs()
        assert (err <= tol).all(), f"{float((err / want).max())} of the output"
        e = (lse[t].double() - torch.logsumexp(s[:m], 0)).abs()
        assert (e <= 2 * ds + 2.0 ** -21 * depth + 2.0 ** -17).all()


@pytest.mark.parametrize("n", [300, 40000])
@pytest.mark.parametrize("dtype,cdt,G,new", KERNELS)
@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_queries_that_are_not_finite(L, dtype, cdt, G, new, n, bad):  # noqa: F811
    """A query of NaN or infinity gives no number, whether its keys were split or not; the other rows are as ever."""
    c = Case(L, [n], [new], G, 1, 128, dtype, cdt)
    c.q[0, 1, 5] = bad
    out, lse = c.run()
    no_error(L)
    assert not torch.isfinite(out[0, 1]).any() and not torch.isfinite(lse[0, 1])
    if bad != bad:
        assert torch.isnan(out[0, 1]).all() and torch.isnan(lse[0, 1])
    c.q[0, 1] = 0
    r = [x.clone() for x in c.ref(0)]
    out[0, 1], lse[0, 1] = r[0][0, 1].to(dtype), r[1][0, 1].float()
    ref.assert_attended(out, tuple(r), lse, F16 if cdt else None)


@pytest.mark.parametrize("new", [1, 2, 16])
def test_tiny_queries_and_scales(L, new):  # noqa: F811
    """Scores that vanish in fp32 weigh all keys alike; rows of every magnitude share a tile."""
    c = Case(L, [500], [new], 8, 1, 128, BF16, E4M3)
    c.q[:, ::2] *= 2.0 ** -125
    c.q[:, 1] *= 2.0 ** 40
    sm = 1e-9
    out, lse = c.run(sm_scale=sm)
    no_error(L)
    r = c.ref(0, 0, sm)
    keep = [0, 2, 3, 4, 5, 6, 7]
    ref.assert_attended(out[:, keep], tuple(x[:, keep] for x in r), lse[:, keep], F16)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()


@pytest.mark.parametrize("dtype,cdt,G,new", [(BF16, E4M3, 1, 3), (BF16, E4M3, 2, 6), (BF16, E4M3, 2, 45), (BF16, E4M3, 3, 300),
                                             (BF16, None, 2, 3), (BF16, None, 2, 300)])
def test_rows_of_every_magnitude(L, dtype, cdt, G, new):  # noqa: F811
    """Rows of q at the ends of bf16's range, tile after tile: each is fitted by a power of two of its own."""
    c = Case(L, [700, 900], [new, new], G, 1, 128, dtype, cdt)
    step = torch.arange(c.T, device="cuda")
    c.q *= (2.0 ** -((step * 37) % 90).double()).to(dtype)[:, None, None]
    c.q[1] = 0
    c.q[2] *= 2.0 ** -30
    out, lse = c.run(sm_scale=0.125)
    c.check(out, lse, 0, 0.125)


@pytest.mark.parametrize("dtype,cdt,H,Hkv,new,n", [(BF16, E4M3, 8, 1, 1, 70000), (F16, None, 8, 1, 4, 70000),
                                                   (BF16, None, 8, 2, 300, 20000), (BF16, E4M3, 6, 2, 300, 20000),
                                                   (F16, E4M3, 5, 1, 300, 20000)])
def test_same_bits_each_time(L, dtype, cdt, H, Hkv, new, n):  # noqa: F811
    """Tiles split over many CTAs, in each kernel: the workspace's contents and what ran before leave no trace."""
    c = Case(L, [n], [new], H, Hkv, 128, dtype, cdt)
    out, lse = c.run()
    ws = L.paged_attn_workspace(new, H, c.cache, c.pg, new, n).fill_(0xFF)
    other = Case(L, [900], [400], 8, 1, 128, dtype, cdt, seed=1)
    for _ in range(3):
        other.run(q=other.q * 100)
        o2, l2 = c.run(ws=ws)
        assert torch.equal(out, o2) and torch.equal(lse, l2)
    no_error(L)


@pytest.mark.parametrize("octaves", [3.0, 0.7, 40.0])
@pytest.mark.parametrize("dtype,cdt,G,new", KERNELS)
def test_scores_that_grow(L, dtype, cdt, G, new, octaves):  # noqa: F811
    """Scores that rise by `octaves` every 128 keys: the weights' reference follows, at once or after a while, and no
    weight leaves the range of the products' type."""
    D, n = 128, 2048
    c = Case(L, [n], [new], G, 1, D, dtype, cdt)
    pages = c.table[0].long()
    ks = 24.0 if cdt else 1.0  # codes up to 24 x 17 = 408 of 448
    k = ((torch.arange(n, device="cuda") / 128 + 1)[:, None] * torch.ones(D, device="cuda") * ks).to(c.cdt)
    bits = torch.uint8 if cdt else c.cdt
    c.k.view(bits)[pages] = k.reshape(-1, 64, 1, D).view(bits)
    c.cache = L.kv_cache(c.k, c.v, ks, VS)
    c.q.fill_(1.0)
    sm = octaves * math.log(2) / D
    out, lse = c.run(sm_scale=sm)
    no_error(L)
    kd, vd = ref.gather(c.k, c.table[0], n, ks), ref.gather(c.v, c.table[0], n, VS)
    want = ref.attend(c.q[:new], kd, vd, torch.arange(n - new, n, device="cuda"), 0, sm)
    ref.assert_attended(out, want, lse, F16 if cdt else None)


@pytest.mark.parametrize("H,Hkv,window,cdt", [(4, 1, 0, None), (4, 1, 0, E4M3), (2, 2, 100, None)])
def test_many_chunks(L, H, Hkv, window, cdt):  # noqa: F811
    """More sequences than one pass of the planner holds, in the chunk kernel."""
    g = torch.Generator().manual_seed(6)
    lens = [int(x) for x in torch.randint(0, 300, (2100,), generator=g)]
    new = [min(int(x), n + 1) for x, n in zip(torch.randint(0, 41, (2100,), generator=g), lens)]
    c = Case(L, lens, new, H, Hkv, 64, BF16, cdt)
    out, lse = c.run(window)
    no_error(L)
    for b in list(range(0, 2100, 97)) + [1023, 1024, 1025, 2047, 2048, 2099]:
        at, m = int(c.q_start[b]), new[b]
        if m:
            ref.assert_attended(out[at:at + m], c.ref(b, window), lse[at:at + m], F16 if cdt else None)
