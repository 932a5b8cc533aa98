"""bsa_cross_forward over long key sequences of which a mask leaves few keys: the log-sum-exp and the
output against 64 bits, with the tolerance of test_gpu_cross.py, whose bound on the log-sum-exp does
not grow with the number of keys. Enough row tiles to fill the SMs, so that one CTA passes over all
keys of a row (with fewer the keys are split, and each run is short)."""
import math

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b
from tests.test_gpu_cross import DEV, _check, _randn

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _whole(d, Lk):
    """Heads of 1000 queries whose row tiles are one per SM, so that the keys are not split."""
    H = torch.cuda.get_device_properties(0).multi_processor_count // 4
    assert b.bsa_cross_workspace_bytes(1, H, H, 1000, Lk, d) == 0
    return H


def _check_heads(o, lse, q, k, v, mask):
    """A few heads (the host's 64-bit form is slow); every head has inputs of its own."""
    for h in (0, q.shape[1] // 2, q.shape[1] - 1):
        s = slice(h, h + 1)
        _check(o[:, s], lse[:, s], q[:, s], k[:, s], v[:, s], key_mask=mask)


# A mask used as padding: the first keys are real, behind them 256 tiles without a real key. The
# row's reference is high (scores of several units), so that what a masked key would add is small.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("real,scale", [(8, 2.0), (64, 2.0), (1, 3.0), (200, 1.0)])
def test_few_real_keys_in_front_of_a_long_masked_rest(dtype, d, real, scale):
    Lk, H = 32768, _whole(d, 32768)
    q = _randn(1, H, 1000, d, dtype=dtype, scale=scale)
    k, v = (_randn(1, H, real, d, dtype=dtype, seed=s) for s in (1, 2))
    kk, vv = (torch.full((1, H, Lk, d), float("nan"), dtype=dtype, device=DEV) for _ in range(2))
    kk[:, :, :real], vv[:, :, :real] = k, v
    mask = torch.zeros(1, Lk, dtype=torch.uint8, device=DEV)
    mask[:, :real] = 1
    o, lse = b.cross_forward(q, kk, vv, key_mask=mask, want_lse=True)
    _check_heads(o, lse, q, k, v, mask[:, :real])


# Every other key masked, one key that holds most of the weight, and many that hold little each:
# 2^-23.5 of it, 1.4e-3 together, which is far above the tolerance of 5e-5.
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
def test_small_weights_beside_masked_keys(dtype, d):
    Lk, H = 32768, _whole(d, 32768)
    unit = math.log(2) / math.sqrt(d)   # of a key's components, per unit of a score in base 2
    q = torch.ones(1, H, 1000, d, dtype=dtype, device=DEV)
    k = (-20 * unit * (1 + _randn(1, H, Lk, d).float() / 64)).to(dtype)
    k[:, :, 0] = 3.5 * unit
    v = _randn(1, H, Lk, d, dtype=dtype, seed=2)
    mask = (torch.arange(Lk, device=DEV) % 2 == 0).to(torch.uint8)[None]
    o, lse = b.cross_forward(q, k, v, key_mask=mask, want_lse=True)
    one = slice(0, 40)   # every row has the same query
    _check_heads(o[:, :, one], lse[:, :, one], q[:, :, one], k, v, mask)


@pytest.mark.parametrize("d", [64, 128])
def test_queries_that_are_not_finite_over_no_real_key(d):
    """A row without a real key is zeros and -inf whatever its query holds, as is one whose real
    keys all have the score -inf; beside any other real key it is NaN."""
    q, k, v = _randn(3, 2, 300, d), _randn(3, 2, 700, d, seed=1), _randn(3, 2, 700, d, seed=2)
    q[:, :, 5, 0], q[:, :, 140, 1], q[:, :, 299] = float("nan"), float("inf"), float("-inf")
    mask = torch.zeros(3, 700, dtype=torch.uint8, device=DEV)
    mask[1, 300:] = 1
    mask[2, 699] = 1
    k[mask[:, None, :, None].expand_as(k) == 0] = float("nan")
    o, lse = b.cross_forward(q, k, v, key_mask=mask, want_lse=True)
    assert not o[0].any() and (lse[0] == float("-inf")).all()
    bad = [5, 140, 299]
    for i, h, t in ((i, h, t) for i in (1, 2) for h in (0, 1) for t in bad):
        if (k[i, h, mask[i] != 0].double() @ q[i, h, t].double() == float("-inf")).all():
            assert not o[i, h, t].any() and lse[i, h, t] == float("-inf")
        else:
            assert torch.isnan(o[i, h, t]).all() and torch.isnan(lse[i, h, t])
    keep = [i for i in range(300) if i not in bad]
    z = torch.zeros((), dtype=k.dtype, device=DEV)
    _check(o[:, :, keep], lse[:, :, keep], q[:, :, keep], torch.where(torch.isfinite(k), k, z), v,
           key_mask=mask)


@pytest.mark.parametrize("Lq", [2, 150])
def test_a_mask_of_truth_values(Lq):
    q, k, v = _randn(2, 2, Lq, 64), _randn(2, 2, 500, 64, seed=1), _randn(2, 2, 500, 64, seed=2)
    mask = torch.arange(1000, device=DEV).view(2, 500) % 3 != 0
    o, lse = b.cross_forward(q, k, v, key_mask=mask, want_lse=True)
    _check(o, lse, q, k, v, key_mask=mask)
    want, _ = b.cross_forward(q, k, v, key_mask=mask.to(torch.uint8))
    assert torch.equal(o, want)
    with pytest.raises(ValueError, match="key_mask"):
        b.cross_forward(q, k, v, key_mask=mask.int())
    with pytest.raises(ValueError, match="key_mask"):
        b.cross_forward(q, k, v, key_mask=mask.t().contiguous().t())
