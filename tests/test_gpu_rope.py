"""Rotary positions and the rotating append against their 64-bit forms, on the GPU."""
import pytest
import torch

from tests import paged_ref as ref

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def L():
    from long_context_sparse_02_b200 import build
    build.build()
    from long_context_sparse_02_b200 import _lib
    _lib.device_error(reset=True)
    return _lib


def randn(g, *shape, dtype=BF16):
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def no_error(L, want=0):
    torch.cuda.synchronize()
    assert L.device_error(reset=True) == want


ROPE = [
    # T, H, Hk, D, dim, offset, interleaved, inverse, scheme, dtype, top position
    (1, 1, 0, 64, 64, 0, False, False, "plain", BF16, 10),
    (8, 128, 0, 576, 64, 512, True, False, "plain", BF16, 131072),
    (257, 5, 1, 128, 128, 0, False, False, "plain", BF16, 4096),
    (33, 7, 3, 128, 64, 64, True, True, "yarn", F16, 1 << 20),
    (19, 3, 2, 96, 24, 8, False, False, "ntk", BF16, 1 << 20),      # half of 12: one element at a time
    (19, 3, 2, 100, 34, 3, True, True, "linear", F16, 2000000000),  # nothing aligned, far positions
    (2, 4, 4, 2, 2, 0, True, False, "plain", BF16, 7),
    (3000, 2, 0, 256, 128, 128, False, False, "plain", F16, 1 << 20),
]


@pytest.mark.parametrize("T,H,Hk,D,dim,offset,inter,inverse,scheme,dtype,top", ROPE)
def test_rope(L, T, H, Hk, D, dim, offset, inter, inverse, scheme, dtype, top):
    g = gen(T + D)
    freq, factor = L.rope_frequencies(dim, 10000.0, scheme, 16.0, 4096)
    freq = freq.cuda()
    pos = torch.randint(0, top, (T,), generator=g, device="cuda", dtype=torch.int32)
    pos[0] = top - 1
    if T > 2:
        pos[1], pos[2] = 0, -5
    spec = L.rope_spec(freq, offset, inter, inverse, factor)
    q = randn(g, T, H, D, dtype=dtype)
    k = randn(g, T, Hk, D, dtype=dtype) if Hk else None
    got_q, got_k = L.rope(q, pos, spec, k=k)
    no_error(L)
    ref.assert_rotated(got_q, ref.rotate(q, pos, freq, offset, inter, inverse, factor), q, factor)
    outside = [i for i in range(D) if not offset <= i < offset + dim]
    assert torch.equal(got_q[..., outside], q[..., outside])
    if Hk:
        ref.assert_rotated(got_k, ref.rotate(k, pos, freq, offset, inter, inverse, factor), k, factor)
    else:
        assert got_k is None
    # in place, the same values
    mine = q.clone()
    same, _ = L.rope(mine, pos, spec, q_out=mine)
    assert same is mine and torch.equal(mine, got_q)


@pytest.mark.parametrize("slack", [8, 1])
def test_rope_strided_and_untouched(L, slack):
    """q and k as slices of one fused projection, outputs as slices of wider buffers: nothing else is written."""
    g = gen(3)
    T, H, Hk, D = 37, 6, 2, 64
    freq, _ = L.rope_frequencies(D)
    freq = freq.cuda()
    spec = L.rope_spec(freq)
    pos = torch.arange(T, device="cuda", dtype=torch.int32)
    fused = randn(g, T, (H + 2 * Hk) * D + slack)  # slack 1: rows start off 16-byte boundaries
    q, k = fused[:, :H * D].unflatten(1, (H, D)), fused[:, H * D:(H + Hk) * D].unflatten(1, (Hk, D))
    buf = torch.full((T, H + Hk + 3, D + slack), 7.0, device="cuda", dtype=BF16)
    qo, ko = buf[:, 1:1 + H, :D], buf[:, 2 + H:2 + H + Hk, :D]
    L.rope(q, pos, spec, k=k, q_out=qo, k_out=ko)
    no_error(L)
    ref.assert_rotated(qo, ref.rotate(q, pos, freq), q)
    ref.assert_rotated(ko, ref.rotate(k, pos, freq), k)
    qo.fill_(7.0), ko.fill_(7.0)
    assert (buf == 7.0).all()
    # heads and tokens in the other order, and one k row given to all tokens (a stride of 0)
    qt = randn(g, H, T, D).transpose(0, 1)
    one = randn(g, 1, Hk, D).expand(T, Hk, D)
    a, b = L.rope(qt, pos, spec, k=one)
    ref.assert_rotated(a, ref.rotate(qt, pos, freq), qt)
    ref.assert_rotated(b, ref.rotate(one, pos, freq), one)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_inverse_is_the_gradient(L, inter):
    """The inverse is the transpose: <g, R x> = <R^T g, x>, and it agrees with differences of the 64-bit form."""
    g = gen(4)
    T, H, D, dim = 5, 3, 64, 32
    freq, _ = L.rope_frequencies(dim)
    freq = freq.cuda()
    pos = torch.tensor([0, 3, 100, 70000, 1048575], device="cuda", dtype=torch.int32)
    x, dy = randn(g, T, H, D, dtype=F16), randn(g, T, H, D, dtype=F16)
    dx, _ = L.rope(dy, pos, L.rope_spec(freq, 16, inter, inverse=True))
    no_error(L)
    xd = x.double().requires_grad_()
    ref.rotate(xd, pos, freq, 16, inter).backward(dy.double())
    ref.assert_rotated(dx, xd.grad, dy)
    for e in (17, 40):
        step = torch.zeros(T, H, D, device="cuda", dtype=torch.float64)
        step[..., e] = 1e-3
        diff = ((ref.rotate(x.double() + step, pos, freq, 16, inter) - ref.rotate(x.double() - step, pos, freq, 16, inter))
                * dy.double()).sum(-1) / 2e-3
        # differences of a linear map: exact but for fp64 rounding; dx is one fp16 rounding off
        tol = ref.HALF_STEP[F16] * diff.abs() + 2 ** -17 * dy.double().abs().amax(-1)
        assert ((dx[..., e].double() - diff).abs() <= tol).all()


def paged_case(g, lens, extra=3):
    blocks = [-(-n // 64) for n in lens]
    pages = sum(blocks) + extra
    order = torch.randperm(pages, generator=g, device="cuda").int()
    table = torch.full((len(lens), max(max(blocks), 1)), 1 << 30, device="cuda", dtype=torch.int32)  # unused: out of range
    at = 0
    for b, n in enumerate(blocks):
        table[b, :n] = order[at:at + n]
        at += n
    return torch.tensor(lens, device="cuda", dtype=torch.int32), table, pages


APPEND = [
    # lens, new tokens, H, Hkv, Dk, Dv, dim, offset, interleaved, dtype, cache
    ([1], [1], 0, 1, 64, 64, 64, 0, False, BF16, BF16),
    ([130, 64, 65], [3, 1, 65], 16, 8, 128, 128, 128, 0, False, BF16, BF16),
    ([700, 5], [511, 5], 0, 1, 576, 0, 64, 512, True, BF16, BF16),
    ([200, 1000], [77, 300], 10, 2, 128, 64, 64, 64, True, F16, F16),
    ([65, 129], [64, 2], 4, 2, 128, 128, 64, 0, False, BF16, torch.uint8),
    ([300], [299], 0, 3, 64, 64, 32, 0, True, F16, torch.float8_e4m3fn),
    ([100], [50], 0, 2, 64, 64, 0, 0, False, BF16, BF16),  # no rotation
]


@pytest.mark.parametrize("lens,new,H,Hkv,Dk,Dv,dim,offset,inter,dtype,cdt", APPEND)
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_append(L, lens, new, H, Hkv, Dk, Dv, dim, offset, inter, dtype, cdt, order):
    g = gen(sum(lens))
    seq_lens, table, pages = paged_case(g, lens)
    eight = cdt in (torch.uint8, torch.float8_e4m3fn)

    def make(width):
        shape = (pages, 64, Hkv, width) if order == "rows" else (pages, Hkv, 64, width)
        c = torch.randint(0, 100, shape, generator=g, device="cuda", dtype=torch.uint8)
        c = c.view(cdt) if eight else c.to(cdt)
        return c if order == "rows" else c.transpose(1, 2)

    kc, vc = make(Dk), make(Dv) if Dv else None
    bits = lambda c: c.view(torch.uint8) if eight else c  # noqa: E731
    k_was, v_was = bits(kc).clone(), bits(vc).clone() if Dv else None
    ks, vs = 24.0, 400.0  # v saturates here and there
    cache, pg = L.kv_cache(kc, vc, ks, vs), L.paged(seq_lens, table, pages)
    n = sum(new)
    tok_seq = torch.tensor([b for b, m in enumerate(new) for _ in range(m)], device="cuda", dtype=torch.int32)
    tok_pos = torch.tensor([x - m + i for x, m in zip(lens, new) for i in range(m)], device="cuda", dtype=torch.int32)
    mix = torch.randperm(n, generator=g, device="cuda")
    tok_seq, tok_pos = tok_seq[mix].contiguous(), tok_pos[mix].contiguous()
    k = randn(g, n, Hkv, Dk, dtype=dtype)
    v = randn(g, n, Hkv, Dv, dtype=dtype) if Dv else None
    q = randn(g, n, H, Dk, dtype=dtype) if H else None
    freq = L.rope_frequencies(dim)[0].cuda() if dim else None
    spec = L.rope_spec(freq, offset, inter, factor=1.25) if dim else None
    qo = L.append_rope(k, v, tok_seq, tok_pos, pg, cache, spec, q=q)
    no_error(L)
    turn = lambda x: ref.rotate(x, tok_pos, freq, offset, inter, False, 1.25) if dim else x.double()  # noqa: E731
    if H:
        ref.assert_rotated(qo, turn(q), q, 1.25)
    else:
        assert qo is None
    page, row = table[tok_seq.long(), (tok_pos // 64).long()].long(), (tok_pos % 64).long()
    for c, was, want, src, scale in ((kc, k_was, turn(k), k, ks), (vc, v_was, v.double() if Dv else None, v, vs)):
        if c is None:
            continue
        got = bits(c)[page, row]
        if eight:
            x = (want * scale).clamp(-448, 448)
            val = got.contiguous().view(torch.float8_e4m3fn).double()
            # half a step of 3 mantissa bits (2^-4; 2^-10 among subnormals), and fp32 arithmetic before it
            top = src.double().abs().amax(-1, keepdim=True) * 1.25 * scale
            assert ((val - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -10 + 2.0 ** -17 * top).all()
        elif dim and c is kc:
            ref.assert_rotated(got, want, src, 1.25)
        else:
            assert torch.equal(got, src)
        bits(c)[page, row] = was[page, row]  # all else is as it was
        assert torch.equal(bits(c), was)


@pytest.mark.parametrize("cdt", [BF16, torch.uint8])
def test_append_from_odd_places(L, cdt):
    """New rows as slices that begin off 16-byte boundaries, many heads of one token, and a cache of one page."""
    g = gen(12)
    kc = torch.zeros(1, 64, 40, 64, device="cuda", dtype=cdt)
    vc = torch.zeros_like(kc)
    seq_lens = torch.tensor([64], device="cuda", dtype=torch.int32)
    pg = L.paged(seq_lens, torch.zeros(1, 1, device="cuda", dtype=torch.int32), 1)
    cache = L.kv_cache(kc, vc, 16.0, 16.0)
    freq = L.rope_frequencies(32)[0].cuda()
    spec = L.rope_spec(freq, 16, False)
    fused = randn(g, 3, 120 * 64 + 1)[:, 1:].unflatten(1, (120, 64))
    k, v, q = fused[:, :40], fused[:, 40:80], fused[:, 80:]
    pos = torch.tensor([63, 0, 31], device="cuda", dtype=torch.int32)
    seq = torch.zeros(3, device="cuda", dtype=torch.int32)
    qo = L.append_rope(k, v, seq, pos, pg, cache, spec, q=q)
    no_error(L)
    ref.assert_rotated(qo, ref.rotate(q, pos, freq, 16), q)
    want = ref.rotate(k, pos, freq, 16)
    if cdt == BF16:
        ref.assert_rotated(kc[0, pos.long()], want, k)
        assert torch.equal(vc[0, pos.long()], v)
    else:
        for c, x in ((kc, want), (vc, v.double())):
            got = c[0, pos.long()].view(torch.float8_e4m3fn).double()
            assert ((got - 16 * x).abs() <= 2.0 ** -4 * (16 * x).abs() + 2.0 ** -10 + 2.0 ** -17 * 64).all()
    # q rotated in place: the elements around the rotated part stay
    mine = q.clone()
    kc.zero_(), vc.zero_()
    assert L.append_rope(k, v, seq, pos, pg, cache, spec, q=mine, q_out=mine) is mine
    no_error(L)
    assert torch.equal(mine, qo)


def test_append_skips(L):
    """Padding, sequences and positions out of range, bad pages: those tokens write nothing, the others as ever."""
    g = gen(9)
    seq_lens, table, pages = paged_case(g, [200, 70])
    kc = torch.zeros(pages, 64, 2, 64, device="cuda", dtype=BF16)
    vc = torch.zeros_like(kc)
    cache, pg = L.kv_cache(kc, vc), L.paged(seq_lens, table, pages)
    freq = L.rope_frequencies(64)[0].cuda()
    spec = L.rope_spec(freq)

    def run(seqs, poss):
        kc.zero_(), vc.zero_()
        n = len(seqs)
        k, v, q = (randn(g, n, h, 64) for h in (2, 2, 4))
        qo = torch.full_like(q, 9.0)
        L.append_rope(k, v, torch.tensor(seqs, device="cuda", dtype=torch.int32),
                      torch.tensor(poss, device="cuda", dtype=torch.int32), pg, cache, spec, q=q, q_out=qo)
        return k, v, q, qo

    k, v, q, qo = run([-1, 0, -1], [5, 199, 0])
    no_error(L)
    assert (qo[[0, 2]] == 9.0).all()
    pos = torch.tensor([5, 199, 0], device="cuda", dtype=torch.int32)
    ref.assert_rotated(qo[1:2], ref.rotate(q, pos, freq)[1:2], q[1:2])
    assert torch.equal(vc[int(table[0, 3]), 7], v[1])
    assert int((vc != 0).any(-1).sum()) == 2  # one row of two heads
    _, v, _, qo = run([0, 2, -2, 1, 1, 0], [200, 0, 0, -1, 69, 0])
    no_error(L, L.DEVERR_POSITION)
    assert (qo[:4] == 9.0).all() and torch.equal(vc[int(table[1, 1]), 5], v[4]) and int((vc != 0).any(-1).sum()) == 4
    seq_lens[1] = 200  # its third page is not in the table's range
    run([1], [130])
    no_error(L, L.DEVERR_PAGE)
    assert not vc.any()
    seq_lens[1] = 1000  # past the table
    run([1], [999])
    no_error(L, L.DEVERR_PAGE)
    assert not vc.any()


@pytest.mark.parametrize("dim", [12160, 12176, 12288, 12304, 50000])
def test_wide_rotations(L, dim):
    """Sines and cosines around the shared memory that a kernel has without asking."""
    g = gen(dim)
    q = randn(g, 3, 2, dim)
    freq = L.rope_frequencies(dim)[0].cuda()
    pos = torch.tensor([0, 7, 100000], device="cuda", dtype=torch.int32)
    got, _ = L.rope(q, pos, L.rope_spec(freq))
    no_error(L)
    ref.assert_rotated(got, ref.rotate(q, pos, freq), q)


def test_latent_rows_for_the_sparse_layer(L):
    """The layer's latent cache as a cache of one head: rows appended rotated are the rows rotated and then appended, and
    the sparse attention over them is the same."""
    g = gen(31)
    seq_lens, table, pages = paged_case(g, [300, 70])
    pg = L.paged(seq_lens, table, pages)
    n, H, K = 40, 16, 64
    tok_seq = torch.tensor([0] * 30 + [1] * 10, device="cuda", dtype=torch.int32)
    tok_pos = torch.tensor([*range(270, 300), *range(60, 70)], device="cuda", dtype=torch.int32)
    freq = L.rope_frequencies(64)[0].cuda()
    spec = L.rope_spec(freq, offset=512, interleaved=True)
    latent = randn(g, n, 1, 576)
    a = randn(g, pages, 64, 576)
    b = a.clone()
    L.append_rope(latent, None, tok_seq, tok_pos, pg, L.kv_cache(a.unsqueeze(2)), spec)
    turned, _ = L.rope(latent, tok_pos, spec)
    codes = torch.zeros(pages, 64, 64, device="cuda", dtype=torch.uint8)
    L.append_kv(randn(g, n, 64), 1.0, turned[:, 0].contiguous(), tok_seq, tok_pos, pg, codes, b)
    no_error(L)
    assert torch.equal(a, b)
    idx = torch.arange(K, device="cuda", dtype=torch.int32).repeat(2, 1)
    q, _ = L.rope(randn(g, 2, H, 576), seq_lens - 1, spec)
    gate = randn(g, 2, H)
    out = [L.sparse_attn(q, x, pg, None, idx, gate, 576 ** -0.5, 512) for x in (a, b)]
    no_error(L)
    assert torch.equal(*out) and torch.isfinite(out[0].float()).all()
