"""Paged attention where its numbers are hardest, on the GPU, through each of its kernels."""
import pytest
import torch

from tests.test_gpu_paged_attn import E4M3, Case
from tests.test_gpu_rope import BF16, L, no_error  # noqa: F401

pytestmark = pytest.mark.gpu


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
