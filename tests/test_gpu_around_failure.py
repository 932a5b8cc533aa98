"""The abort paths of the kernels of bsa_linear and bsa_cross_forward, run without a fault: with
waits limited to a few nanoseconds a wait runs out while copies and products are in flight, the
kernel drains and reports BSA_ERR_TIMEOUT, and the next call is right again. (A test of a
barrier itself waits for some microseconds before the limit is looked at, so a short call may
end in time all the same: then its result is right. The long ones always run out.)"""
import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b
from tests import test_gpu_cross as tc
from tests import test_gpu_linear as tl

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _st():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# short ones, then long sums, which keep the epilogue waiting for tens of microseconds: few rows,
# whole tiles and shared ones; tiles of CTA pairs, whole and shared
SHORT = [(4, 512, 4096), (4, 8192, 512), (3000, 1024, 2048), (300, 8192, 512)]
LONG = [(4, 16384, 18944), (4, 16384, 8192), (3000, 16384, 2048), (300, 32768, 1024)]


@pytest.mark.parametrize("L,K,N", SHORT + LONG)
@pytest.mark.parametrize("wait_ns", [1, 500])
def test_linear_aborts_and_recovers(L, K, N, wait_ns):
    x, w = tl._randn(1, L, K), tl._randn(N, K, seed=1, scale=K ** -0.5)
    y = torch.zeros(L, N, dtype=torch.bfloat16, device=DEV)
    ws = torch.empty(max(16, b.bsa_linear_workspace_bytes(1, L, K, N)), dtype=torch.uint8, device=DEV)
    st = _st()
    b.bsa_selftest_linear_timeout(x[0], w, y, ws, wait_ns, st)
    torch.cuda.synchronize()
    assert st.item() == b.ERR_TIMEOUT or ((L, K, N) in SHORT and st.item() == 0)
    if st.item() == 0:
        tl._check(y[None], x, w)
    st = _st()
    b.bsa_selftest_linear_timeout(x[0], w, y, ws, 2_000_000_000, st)
    torch.cuda.synchronize()
    assert st.item() == 0
    tl._check(y[None], x, w)


@pytest.mark.parametrize("Lq,Lk,d", [(700, 900, 128), (2000, 77, 64), (20, 6000, 64)])
@pytest.mark.parametrize("masked", [False, True])
@pytest.mark.parametrize("wait_ns", [1, 500])
def test_cross_aborts_and_recovers(Lq, Lk, d, masked, wait_ns):
    H = 6
    q, k, v = tc._randn(1, H, Lq, d), tc._randn(1, H, Lk, d, seed=1), tc._randn(1, H, Lk, d, seed=2)
    n = torch.tensor([Lk - 5], dtype=torch.int32, device=DEV) if masked else None
    o = torch.zeros_like(q[0])
    ws = torch.empty(max(16, b.bsa_cross_workspace_bytes(1, H, H, Lq, Lk, d)), dtype=torch.uint8,
                     device=DEV)
    st = _st()
    b.bsa_selftest_cross_timeout(q[0], k[0], v[0], o, ws, wait_ns, st, key_len=n)
    torch.cuda.synchronize()
    assert st.item() in (b.ERR_TIMEOUT, 0)
    if st.item() == 0:
        tc._check(o[None], None, q, k, v, key_len=n)
    st = _st()
    b.bsa_selftest_cross_timeout(q[0], k[0], v[0], o, ws, 2_000_000_000, st, key_len=n)
    torch.cuda.synchronize()
    assert st.item() == 0
    tc._check(o[None], None, q, k, v, key_len=n)
