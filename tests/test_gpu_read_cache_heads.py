"""kvq_read_cache at head counts that leave the blocks of a wave unevenly shared, with every SM at work (bounds:
test_gpu_read_cache)."""
import pytest

from test_gpu_read_cache import Cache

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("kinds", [("dense", "dense"), ("signed_hadamard", "signed_hadamard"), ("identity", "identity"),
                                   ("dense", "identity")])
@pytest.mark.parametrize("hkv,tokens", [(13, 2500), (32, 1900), (40, 1100), (80, 700), (200, 300)])
def test_heads_that_share_a_wave_unevenly(hkv, tokens, kinds, dtype):
    """Two roles of 32 heads take 256 places of 304, of 80 heads 160, of 200 heads 400: several waves."""
    ranges = [(11, tokens), (0, 130)]
    c = Cache(31, [tokens + 20, 140], hkv, 16, kinds)
    c.check(c.run(ranges, dtype), ranges, dtype)


@pytest.mark.parametrize("which", ["k", "v"])
@pytest.mark.parametrize("hkv", [32, 80, 170])
def test_one_role_of_many_heads(hkv, which):
    ranges = [(0, 1000)]
    c = Cache(32, [1000], hkv, 8, ("dense", "dense"))
    c.check(c.run(ranges, "f32", which=which), ranges, "f32")
