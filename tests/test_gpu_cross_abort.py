"""The abort path of bsa_cross_forward's tensor-core kernel where a wait always runs out, with and
without a key mask. One CTA per SM takes two row tiles of 128 tiles of keys each. Three tiles of 256
rows to a head, the third of 44 rows, so that for a third of the CTAs the first has no rows for the
second stream: its softmax waits for the whole of that tile (more than 100 us), whatever the time for
which a test of a barrier itself waits."""
import ctypes

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b
from tests.test_gpu_cross import DEV, _check, _randn

P = ctypes.c_void_p(1 << 20)          # 16-byte aligned; never dereferenced


def test_mask_timeout_selftest_refuses():
    call = b.lib().bsa_selftest_cross_mask_timeout
    for wait in (0, -1, 10 ** 10 + 1):
        assert call(P, P, P, P, 0, 2, 8, 64, 64, None, P, P, 1 << 40, wait, P, None) == b.ERR_INVALID_ARG
    assert call(P, P, P, P, 0, 2, 8, 64, 64, None, P, P, 1 << 40, 100, None, None) == b.ERR_INVALID_ARG
    assert call(P, P, P, P, 0, 2, 8, 64, 96, None, P, P, 1 << 40, 100, P, None) == b.ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("wait_ns", [1, 500])
def test_a_wait_that_always_runs_out(cuda_ok, d, masked, wait_ns):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    H, Lq, Lk = 2 * sms // 3, 556, 16384
    assert sms % 3 != 0 and b.bsa_cross_workspace_bytes(1, H, H, Lq, Lk, d) == 0
    q, k, v = _randn(1, H, Lq, d), _randn(1, H, Lk, d, seed=1), _randn(1, H, Lk, d, seed=2)
    n = torch.tensor([Lk - 5], dtype=torch.int32, device=DEV)
    mask = (torch.arange(Lk, device=DEV) % 5 != 0).to(torch.uint8)
    o = torch.zeros_like(q[0])
    ws = torch.empty(16, dtype=torch.uint8, device=DEV)

    def call(wait):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        if masked:
            b.bsa_selftest_cross_mask_timeout(q[0], k[0], v[0], o, mask, ws, wait, st, key_len=n)
        else:
            b.bsa_selftest_cross_timeout(q[0], k[0], v[0], o, ws, wait, st, key_len=n)
        torch.cuda.synchronize()
        return st.item()

    assert call(wait_ns) == b.ERR_TIMEOUT
    assert call(2_000_000_000) == 0
    want, _ = b.cross_forward(q, k, v, key_len=n, key_mask=mask[None] if masked else None)
    assert torch.equal(o, want[0])
    for h in (0, H - 1):
        s = slice(h, h + 1)
        _check(o[None, s], None, q[:, s], k[:, s], v[:, s], key_len=n,
               key_mask=mask[None] if masked else None)
