"""Counts of heads at which a token's runs of rows would end behind 2^31 - 1: refused on the host."""
import pytest

from sparse_top_landmark_gb300 import build as B
from sparse_top_landmark_gb300 import mita
from test_decode_abi import APPEND, BACKWARD, ROPE, call, msg

MOST = 1 << 30


@pytest.fixture(scope="module")
def lib():
    B.build()
    return mita.load()


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("heads", [dict(Hq=MOST + 1, Hkv=0), dict(Hq=MOST - 1, Hkv=2),
                                   dict(Hq=2 ** 31 - 2, Hkv=1), dict(Hq=1, Hkv=MOST)])
def test_norm_rope(lib, suffix, heads):
    one = dict(B=1, N=1)
    for name, layout, base in (("mita_qk_norm_rope", mita._NORM_ROPE, ROPE),
                               ("mita_qk_norm_rope_backward", mita._NORM_ROPE_BACKWARD, BACKWARD)):
        assert call(lib, name + suffix, layout, base, {**one, **heads}) == 2, msg(lib)
        assert "2^30" in msg(lib)
        # up to there the next check is the one that fails
        fits = {**one, "Hq": MOST - 4, "Hkv": 4, "rot": 12}
        assert call(lib, name + suffix, layout, base, fits) == 1 and "rot" in msg(lib)


@pytest.mark.parametrize("suffix", ["", "_f32"])
@pytest.mark.parametrize("heads", [dict(Hq=MOST, Hkv=1), dict(Hq=0, Hkv=MOST // 2 + 1),
                                   dict(Hq=2 ** 31 - 3, Hkv=1)])
def test_append(lib, suffix, heads):
    name = "mita_cache_append" + suffix
    assert call(lib, name, mita._CACHE_APPEND, APPEND, dict(T=1, **heads)) == 2, msg(lib)
    assert "2^30" in msg(lib)
    fits = dict(T=1, Hq=MOST - 8, Hkv=4, kc=0)
    assert call(lib, name, mita._CACHE_APPEND, APPEND, fits) == 1 and "k_cache" in msg(lib)
