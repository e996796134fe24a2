"""Host checks of the 8-bit verify's merge settings."""
import pytest

from mla_tree_verify_gb300 import binding, build


@pytest.mark.parametrize("mode,limit", [(-1, 0), (3, 0), (0, -1), (2, 10 ** 9 + 1), (1, 1 << 62)])
def test_merge_settings_that_are_refused(mode, limit):
    build.build()
    a = dict(q=16, kv=16, sc=16, kvi=16, kvp=16, ocl=16, mask=16, mip=16, qop=16, scale=0.1, out=16, lse=16, ws=256,
             wsb=1 << 40, bs=1, mq=4, heads=64, slots=10, total_q=4, nkvi=3, mlen=28, block=1)
    assert binding.load().mla_tree_verify_q8_debug_merge(*a.values(), mode, limit, None) == -3


def test_other_arguments_are_checked_as_ever():
    build.build()
    a = dict(q=16, kv=0, sc=16, kvi=16, kvp=16, ocl=16, mask=16, mip=16, qop=16, scale=0.1, out=16, lse=16, ws=256,
             wsb=1 << 40, bs=1, mq=4, heads=64, slots=10, total_q=4, nkvi=3, mlen=28, block=1)
    assert binding.load().mla_tree_verify_q8_debug_merge(*a.values(), 1, 100, None) == -1
