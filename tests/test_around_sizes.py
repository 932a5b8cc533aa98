"""The size queries of the calls around the block attention (CPU): any sizes are answered, with 0 where
the call refuses them."""
import random

import pytest

from piecewise_attention_diffusion_b200 import bsattn as b
from tests.test_around_abi import _cross, _linear

# rows past 2^30, their product past 2^31 and 2^32 (to a 32-bit 0, a negative and a small count);
# columns and sums near 2^31; tiles past 2^31
LINEAR = [(65536, 65536, 64, 64), (32768, 131072, 64, 64), (32768, 65536, 64, 64), (65537, 65536, 64, 64),
          (1, 2 ** 31 - 1, 64, 64), (2 ** 31 - 1, 1, 64, 64), (2 ** 31 - 1, 2 ** 31 - 1, 8, 8),
          (1, 8, 2 ** 31 - 8, 64), (1, 8, 64, 2 ** 31 - 1), (1, 8, 2 ** 30, 64), (1, 8, 64, 2 ** 30),
          (2 ** 14, 2 ** 15, 128, 2 ** 20), (1, 2 ** 30 - 1, 8, 2 ** 20)]


@pytest.mark.parametrize("Bt,L,K,N", LINEAR)
def test_linear_sizes_that_are_refused(Bt, L, K, N):
    assert b.bsa_linear_workspace_bytes(Bt, L, K, N) == 0
    assert _linear(Bt=Bt, L=L, K=K, N=N) == b.ERR_UNSUPPORTED


def test_linear_sizes_that_are_not_positive():
    for sizes in ((0, 8, 64, 64), (1, -8, 64, 64), (1, 8, 0, 64), (1, 8, 64, -(2 ** 31))):
        assert b.bsa_linear_workspace_bytes(*sizes) == 0


def test_linear_sizes_at_the_limits():
    for sizes in ((1, 2 ** 30 - 1, 8, 64), (2 ** 30 - 1, 1, 8, 64), (2 ** 15, 2 ** 15 - 1, 64, 64),
                  (1, 1, 2 ** 30 - 8, 64), (1, 1, 8, 2 ** 30 - 1), (1, 1, 8, 1), (1, 16, 2 ** 30 - 8, 2 ** 30 - 1)):
        need = b.bsa_linear_workspace_bytes(*sizes)
        # two slots of at most 256 x 256 sums for each of a few hundred groups
        assert 0 <= need <= 2 * 1024 * 256 * 256 * 4


def test_any_sizes_are_answered():
    """Where a query asks for a workspace, the call without one is refused before it launches."""
    rng = random.Random(3)
    size = lambda: rng.choice((1, -1)) * int(2 ** rng.uniform(0, 31)) if rng.random() < 0.05 \
        else int(2 ** rng.uniform(0, 31))
    for _ in range(20000):
        sizes = [size() for _ in range(4)]
        if b.bsa_linear_workspace_bytes(*sizes):
            assert _linear(**dict(zip(("Bt", "L", "K", "N"), sizes)), ws=None) in (
                b.ERR_WORKSPACE, b.ERR_UNSUPPORTED)
    for _ in range(4000):
        sizes = [size() for _ in range(5)] + [rng.choice((64, 128, 96))]
        if b.bsa_cross_workspace_bytes(*sizes):
            assert _cross(**dict(zip(("Bt", "H", "Hkv", "Lq", "Lk", "d"), sizes)), ws=None) in (
                b.ERR_WORKSPACE, b.ERR_UNSUPPORTED, b.ERR_INVALID_ARG)
