"""Paged attention where its numbers are hardest, on the GPU, through each of its kernels."""
import math

import pytest
import torch

from tests import paged_ref as ref
from tests.test_gpu_paged_attn import E4M3, Case
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
    output.  A weight is rounded once to the products' type; of fp16's, what lies 36 octaves below the largest is lost."""
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
        # weights: one rounding, and 2^-37 of the largest (half a step of fp16's smallest, lifted); scores: an fp32 product
        # of D terms, as in assert_attended; the output's rounding, also among fp16's smallest numbers
        ds = (D + 4) * 2.0 ** -24 * float((kd[:m].abs().sum(-1) * sm).max())
        tol = (half + 2 * ds + 2.0 ** -18 + ref.HALF_STEP[dtype]) * 1.01 * want + 2.0 ** -36 * vd[:m].sum(0) / w.sum() + 2.0 ** -25
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
