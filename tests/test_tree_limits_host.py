"""Limits of the trees' entry points that the sizes of any GPU's memory are below:
checked before anything is launched, so on the CPU with addresses that are never
read.  No GPU needed."""
import ctypes

import pytest

import test_tree_host as host
from tile_level_overlap_gb300 import build, mk

at = host.at


@pytest.fixture(scope="module")
def lib():
    build.build()
    return mk.lib()


@pytest.mark.parametrize("mixed", [False, True])
def test_extents_of_probabilities(lib, mixed):
    def call(rows, **kw):
        ok = dict(parents=at(1 << 20), tokens=at(2 << 20), p=at(3), ps=100, q=None, qs=0, vocab=100, u=at(4 << 20), ul=at(5), path=at(6 << 20), emitted=at(7 << 20),
                  kept=at(9), lens=at(10), status=None)
        b = ctypes.byref(host.batch(max_tokens=rows))
        args = [*{**ok, **kw}.values(), None]
        return lib.mk_tree_verify_mixed(b, 1, *args) if mixed else lib.mk_tree_verify(b, *args)

    most = (1 << 31) - 1
    # rows x stride x 4 bytes past 2^62 are refused as such, whatever the product's low bits
    for stride in (1 << 30, 1 << 31, 1 << 32, 1 << 33, (1 << 37) + 5, (1 << 38) - 1):
        assert call(most, ps=stride) == 5, stride
        assert call(most, q=at(8), qs=stride) == 5, stride
        assert call(most, ps=stride, q=at(8), qs=stride) == 5, stride
    # below, what lies inside them is still found (so nothing of these is launched)
    far = at(3) + (1 << 58)
    for kw in (dict(ps=1 << 29), dict(q=at(3), qs=1 << 29), dict(q=at(3), qs=(1 << 29) - 1)):
        assert call(most, path=far, **kw) == 1, kw
    assert call(2, ps=(1 << 38) - 1, path=at(3) + 4 * ((1 << 38) - 1) + 396) == 1
    assert call(3, ps=(1 << 38) - 1, path=at(3) + 8 * ((1 << 38) - 1) + 396) == 1
