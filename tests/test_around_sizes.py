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


class _Devices:
    """A current device and a library whose plans count its SMs, without a GPU."""
    sms = (148, 74)

    def __init__(self):
        self.now = 0

    def device(self, index):
        outer = self

        class Context:
            def __enter__(self):
                self.before, outer.now = outer.now, index

            def __exit__(self, *_):
                outer.now = self.before
        return Context()

    def bsa_linear_workspace_bytes(self, *sizes):
        return self.sms[self.now] * sum(sizes)

    bsa_cross_workspace_bytes = bsa_linear_workspace_bytes


@pytest.mark.parametrize("query", ["bsa_linear_workspace_bytes", "bsa_cross_workspace_bytes"])
def test_helpers_ask_for_the_tensors_device(monkeypatch, query):
    dev = _Devices()
    monkeypatch.setattr(b, "_lib", dev)
    monkeypatch.setattr(b.torch._C, "_cuda_getDevice", lambda: dev.now, raising=False)
    monkeypatch.setattr(b.torch.cuda, "device", dev.device)
    asked = []
    monkeypatch.setattr(b, "_scratch", lambda like, n, stream: asked.append(n))
    # a helper is run up to its launch with stand-ins of tensors on device 1
    monkeypatch.setattr(b, "_view", lambda *a, **k: None)
    monkeypatch.setattr(b, "_empty", lambda *a, **k: None)
    for name in ("_linear", "_cross"):
        monkeypatch.setattr(b, name, lambda *a, **k: None)
    monkeypatch.setattr(b, "_workspace_of", lambda ws, index: (None, 0))
    meta = lambda *shape: _OnDevice1(b.torch.empty(*shape, device="meta"))
    if query == "bsa_linear_workspace_bytes":
        b.linear(meta(1, 4, 64), b.torch.empty(32, 64, device="meta"))
        want = 74 * (1 + 4 + 64 + 32)
    else:
        b.cross_forward(meta(1, 2, 3, 64), b.torch.empty(1, 2, 9, 64, device="meta"), None)
        want = 74 * (1 + 2 + 2 + 3 + 9 + 64)
    assert asked == [want] and dev.now == 0


class _OnDevice1:
    def __init__(self, t):
        self.shape, self.dim = t.shape, t.dim

    def get_device(self):
        return 1
