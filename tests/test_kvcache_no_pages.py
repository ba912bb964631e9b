"""A cache without pages: reading it and attending over it still launch (they write zeros, and -inf
for lse), and the kernels take the head scales, so those are checked (host only, no GPU needed)."""
import pytest

from scale_search_weights_amd import kvcache
from test_abi import EALIGN, ENULL, FAKE, OK, P
from test_kvcache_host import C, attention

S_BAD = [(dict(S=None), ENULL), (dict(S_k=None), ENULL), (dict(S_v=None), ENULL), (dict(S_k=FAKE + 2), EALIGN),
         (dict(S_v=FAKE + 1), EALIGN)]


@pytest.fixture(scope="module")
def L():
    return kvcache.lib()


@pytest.mark.parametrize("bad,rc", S_BAD, ids=[str(b[0]) for b in S_BAD])
def test_head_scales_are_checked_without_pages(L, bad, rc):
    def c():
        return C(pages=0, codes=None, scales=None, **bad)
    assert L.nvfp4_kv_read(c(), P(FAKE), 4, P(FAKE), P(FAKE), 1, None) == rc
    assert L.nvfp4_kv_read(c(), P(FAKE), 4, None, P(FAKE), 0, None) == rc
    assert attention(L, c()) == rc
    assert attention(L, c(), max_kv=0, table=None, lens=None, prefix=40, pp=FAKE) == rc
    # nothing to do: nothing is read
    assert L.nvfp4_kv_read(c(), None, 0, None, None, 1, None) == OK
    assert L.nvfp4_kv_write(c(), P(FAKE), P(FAKE), 1, 4, 128, 64, 128, 64, P(FAKE), None) == OK
    assert attention(L, c(), tokens=0, max_q=0) == OK
