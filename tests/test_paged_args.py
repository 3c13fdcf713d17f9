"""Rotary frequencies, and the calls that the rotating append and paged attention refuse before any CUDA call (no GPU needed)."""
import ctypes
import math
import random

import pytest
import torch

P = ctypes.c_void_p
NAN = float("nan")


@pytest.fixture(scope="module")
def L():
    from long_context_sparse_02_b200 import build
    build.build()
    from long_context_sparse_02_b200 import _lib
    return _lib


def test_frequencies(L):
    f, s = L.rope_frequencies(64, 10000.0)
    assert f.dtype == torch.float64 and f.shape == (32,) and s == 1.0
    assert torch.allclose(f, 10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32), rtol=1e-14, atol=0)
    lin, s = L.rope_frequencies(64, 10000.0, "linear", 8.0)
    assert torch.allclose(lin, f / 8, rtol=1e-14, atol=0) and s == 1.0
    ntk, s = L.rope_frequencies(64, 10000.0, "ntk", 8.0)
    assert s == 1.0 and ntk[0] == 1.0 and torch.allclose(ntk[-1], f[-1] / 8, rtol=1e-12, atol=0)
    assert (ntk <= f).all() and (ntk >= f / 8 * (1 - 1e-12)).all()
    yarn, s = L.rope_frequencies(64, 10000.0, "yarn", 16.0, 4096)
    assert s == pytest.approx(0.1 * math.log(16) + 1, rel=1e-6)
    turns = f * 4096 / (2 * math.pi)
    assert torch.equal(yarn[:10], f[:10]) and turns[9] > 32     # fast pairs stay
    assert torch.allclose(yarn[-6:], f[-6:] / 16, rtol=1e-13, atol=0) and turns[-6] < 1  # slow ones are interpolated
    assert ((yarn <= f) & (yarn >= f / 16 * (1 - 1e-12))).all() and (yarn[1:] < yarn[:-1]).all()
    one, s = L.rope_frequencies(2, 500.0)
    assert one.tolist() == [1.0]


@pytest.mark.parametrize("args", [(63,), (0,), (64, 1.0), (64, NAN), (64, 1e4, "linear", 0.5), (64, 1e4, "yarn", 4.0, 0),
                                  (2, 1e4, "ntk", 4.0), (64, 1e4, "linear", NAN), (64, math.inf)])
def test_frequencies_refused(L, args):
    with pytest.raises(L.DsaError):
        L.rope_frequencies(*args)


def test_frequencies_scheme(L):
    with pytest.raises(ValueError):
        L.rope_frequencies(64, scheme="other")


def spec(L, **kw):
    a = dict(inv_freq=P(256), dim=64, offset=0, layout=0, inverse=0, factor=1.0) | kw
    return ctypes.byref(L.RopeSpec(*a.values()))


def cache(L, **kw):
    a = dict(k=P(256), v=P(512), kps=64 * 256, krs=256, khs=128, vps=64 * 256, vrs=256, vhs=128, heads=2, Dk=128, Dv=128,
             dtype=0, ks=1.0, vs=1.0) | kw
    return ctypes.byref(L.KvCache(*a.values()))


def pages(L, **kw):
    a = dict(lens=P(256), table=P(512), seqs=2, blocks=4, size=64, pages=8) | kw
    return ctypes.byref(L.Paged(*a.values()))


def call_rope(L, **kw):
    a = dict(q=P(256), qt=256, qh=128, Hq=2, qo=P(512), qot=256, qoh=128, k=None, kt=0, kh=0, Hk=0, ko=None, kot=0, koh=0,
             pos=P(256), T=3, D=128, dtype=0, rope=spec(L), stream=None) | kw
    return L.lib.dsa_rope(*a.values())


def call_append(L, **kw):
    a = dict(k=P(256), kt=256, kh=128, v=P(256), vt=256, vh=128, q=None, qt=0, qh=0, H=0, qo=None, qot=0, qoh=0, seq=P(256),
             pos=P(256), pg=pages(L), n=3, dtype=0, rope=spec(L), cache=cache(L), stream=None) | kw
    return L.lib.dsa_append_rope(*a.values())


def call_attn(L, **kw):
    a = dict(q=P(256), qt=1024, qh=128, H=8, cache=cache(L), pg=pages(L), start=P(256), T=5, max_q=4, max_len=100, window=0,
             scale=0.1, dtype=0, out=P(256), lse=None, ws=P(256), wsb=1 << 40, stream=None) | kw
    return L.lib.dsa_paged_attn(*a.values())


BAD_SPECS = [dict(inv_freq=None), dict(dim=0), dict(dim=63), dict(offset=-1), dict(offset=65), dict(dim=130), dict(layout=2),
             dict(inverse=2), dict(factor=NAN), dict(factor=math.inf)]
BAD_CACHES = [dict(k=None), dict(k=P(264)), dict(v=P(520)), dict(krs=4), dict(kps=0), dict(khs=-128), dict(vhs=100),
              dict(vps=1 << 40), dict(heads=0), dict(Dk=0), dict(Dv=0), dict(v=None), dict(dtype=3), dict(dtype=-1),
              dict(dtype=2, ks=0.0), dict(dtype=2, ks=NAN), dict(dtype=2, vs=-1.0), dict(dtype=2, vs=math.inf)]


def test_rope_refused(L):
    assert call_rope(L, rope=None) == 1
    for s in BAD_SPECS:
        assert call_rope(L, rope=spec(L, **s)) == 1, s
    for kw in (dict(T=-1), dict(Hq=-1), dict(Hk=-1), dict(D=1), dict(dtype=2), dict(dtype=-1), dict(q=None), dict(qo=None),
               dict(pos=None), dict(Hk=2), dict(Hk=2, k=P(256)), dict(qo=P(256), qot=512), dict(qo=P(256), qoh=64),
               dict(Hk=2, k=P(64), ko=P(64), kt=256, kh=128, kot=128, koh=128)):
        assert call_rope(L, **kw) == 1, kw
    assert call_rope(L, T=0) == 0 and call_rope(L, Hq=0, q=None, qo=None) == 0


def test_one_place_for_several_heads_refused(L):
    """One head given to all (a stride of 0) is an input; rotated into one place, in place or not, it is refused."""
    for kw in (dict(qot=0), dict(qoh=0), dict(qo=P(256), qt=0, qot=0), dict(qo=P(256), qh=0, qoh=0),
               dict(Hk=2, k=P(64), ko=P(64), kt=0, kh=128, kot=0, koh=128), dict(Hk=2, k=P(64), ko=P(512), kt=256, kh=128, kot=256)):
        assert call_rope(L, **kw) == 1, kw
    for kw in (dict(qot=0), dict(qoh=0), dict(qo=P(256), qt=0, qot=0)):
        assert call_append(L, **dict(q=P(256), H=4, qo=P(512), qt=512, qh=128, qot=512, qoh=128) | kw) == 1, kw


def test_append_refused(L):
    for s in BAD_SPECS:
        assert call_append(L, rope=spec(L, **s)) == 1, s
    for c in BAD_CACHES:
        assert call_append(L, cache=cache(L, **c)) == 1, c
    assert call_append(L, cache=cache(L, Dk=72)) == 2
    for kw in (dict(n=-1), dict(pg=None), dict(pg=pages(L, size=32)), dict(pg=pages(L, lens=None)), dict(dtype=2), dict(dtype=1),
               dict(cache=None), dict(k=None), dict(v=None), dict(seq=None), dict(pos=None), dict(q=P(256)), dict(H=4),
               dict(q=P(256), H=4), dict(q=P(256), H=4, qo=P(512), rope=None), dict(cache=cache(L, v=None, Dv=0)),
               dict(q=P(256), H=4, qo=P(256), qt=512, qh=128, qot=1024, qoh=128)):
        assert call_append(L, **kw) == 1, kw
    assert call_append(L, n=0) == 0 and call_append(L, n=0, rope=None) == 0
    # one page, one head: their strides are not looked at
    assert call_append(L, n=0, pg=pages(L, pages=1), cache=cache(L, heads=1, kps=3, vps=-1, khs=0, vhs=5)) == 0


def test_attention_refused(L):
    for c in BAD_CACHES:
        assert call_attn(L, cache=cache(L, **c)) == 1, c
    for kw in (dict(T=-1), dict(H=0), dict(max_q=0), dict(max_len=0), dict(window=-1), dict(scale=NAN), dict(scale=math.inf),
               dict(dtype=2), dict(dtype=1), dict(pg=None), dict(pg=pages(L, pages=0)), dict(cache=None), dict(q=None), dict(out=None),
               dict(q=P(264)), dict(out=P(264)), dict(qt=1025), dict(qh=100), dict(start=None)):
        assert call_attn(L, **kw) == 1, kw
    for kw in (dict(H=7), dict(cache=cache(L, v=None, Dv=0)), dict(cache=cache(L, Dv=64)), dict(cache=cache(L, Dk=96, Dv=96)),
               dict(cache=cache(L, Dk=576, Dv=576))):
        assert call_attn(L, **kw) == 2, kw
    for kw in (dict(max_len=(1 << 30) + 1), dict(max_q=(1 << 30) + 1), dict(T=(1 << 30) + 1), dict(T=1 << 30)):
        assert call_attn(L, **kw) == 2, kw
    assert call_attn(L, T=0) == 0


def test_workspace_size(L):
    f = L.lib.dsa_paged_attn_workspace_bytes
    assert f(8, 8, 64, cache(L), 1, 1000, 0) > 0
    for bad in ((0, 8, 64, cache(L), 1, 1000, 0), (8, 0, 64, cache(L), 1, 1000, 0), (8, 8, 63, cache(L), 1, 1000, 0),
                (8, 8, 64, cache(L), 0, 1000, 0), (8, 8, 64, cache(L), 1, 0, 0), (8, 8, 64, cache(L), 1, 1000, -1),
                (8, 8, 64, None, 1, 1000, 0)):
        assert f(*bad) == 0
    assert f(8, 8, 64, cache(L), 1, 1000, 1000) == f(8, 8, 64, cache(L), 1, 1000, 0) == f(8, 8, 64, cache(L), 1, 1000, 2 ** 31 - 1)
    # a bound, whatever the lengths: no more for a million positions than for a few thousand
    assert f(8, 8, 64, cache(L), 1, 1 << 20, 0) == f(8, 8, 64, cache(L), 1, 1 << 16, 0)


def test_workspace_of_larger_calls_serves_smaller_ones(L):
    """A workspace made for some sizes is enough for every call of at most these."""
    r = random.Random(4)

    def need(B, G, max_q, max_len, window, Hkv, D, dtype):
        return L.lib.dsa_paged_attn_workspace_bytes(9, B, G * Hkv, cache(L, heads=Hkv, Dk=D, Dv=D, dtype=dtype), max_q, max_len, window)

    for _ in range(3000):
        top = (r.randint(1, 40), r.randint(1, 160), int(2 ** r.uniform(0, 11)), int(2 ** r.uniform(0, 16)), int(2 ** r.uniform(0, 17)))
        kind = (r.choice([1, 2, 8]), r.choice([64, 128]), r.choice([0, 2]))
        less = tuple(r.randint(1, x) if r.random() < 0.5 else x for x in top)
        assert need(*less, *kind) <= need(*top, *kind), (less, top, kind)
        assert need(*top, *kind) <= need(*top[:4], 0, *kind)  # (no window: all of the length)


def test_python_checks(L):
    t = torch.zeros(2, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA"):
        L.rope(t, torch.zeros(2, dtype=torch.int32), L.RopeSpec())
    with pytest.raises(ValueError, match="CUDA"):
        L.kv_cache(torch.zeros(2, 64, 1, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="CUDA"):
        L.rope_spec(torch.zeros(4, dtype=torch.float64))


def test_page_tables_have_a_row_a_sequence(L):
    """The kernels read a row of the block table for each sequence: a table of fewer is refused before they do."""
    lens = torch.ones(3, dtype=torch.int32)
    for table in (torch.zeros(2, 4, dtype=torch.int32), torch.zeros(12, dtype=torch.int32)):
        with pytest.raises(ValueError, match="row for each"):
            L.paged(lens, table, 8)
