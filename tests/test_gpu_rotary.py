"""bsa_rotary against the rotation written as complex numbers in 64 bits.

Tolerance, from the arithmetic: the angle is reduced in 64 bits and rounded to fp32 as a
fraction of a half turn in [-1, 1] (an error of at most pi 2^-25 in the angle), sine and
cosine are then within 2 ulp, so each is off by less than 2^-22; a product and its sum add
at most 2^-23 of |x_lo| + |x_hi|. Together e = 2^-21 (|x_lo| + |x_hi|) bounds the fp32
result with room to spare, and rounding to the type adds half a step of the result:
eps/2 |y|, or half the smallest subnormal step below the normal range.
"""
import numpy as np
import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _turned(x, pos, axes, halves, inverse, base=10000.0):
    """(y, |x_lo| + |x_hi| of every component, 0 where it is copied), in 64 bits."""
    x = x.detach().cpu().double().numpy()
    pos = pos.cpu().double().numpy()
    if pos.ndim == 2:
        pos = np.broadcast_to(pos, (x.shape[0],) + pos.shape)
    y, size, at = x.copy(), np.zeros_like(x), 0
    for a, n in enumerate(axes):
        sec = x[..., at:at + n]
        lo, hi = (sec[..., :n // 2], sec[..., n // 2:]) if halves else (sec[..., ::2], sec[..., 1::2])
        phi = pos[:, None, :, a, None] * base ** (-2.0 * np.arange(n // 2) / n)
        z = (lo + 1j * hi) * np.exp(-1j * phi if inverse else 1j * phi)
        m = np.abs(lo) + np.abs(hi)
        if halves:
            y[..., at:at + n] = np.concatenate((z.real, z.imag), -1)
            size[..., at:at + n] = np.concatenate((m, m), -1)
        else:
            y[..., at:at + n:2], y[..., at + 1:at + n:2] = z.real, z.imag
            size[..., at:at + n:2] = size[..., at + 1:at + n:2] = m
        at += n
    return y, size


def _check(got, x, pos, axes, halves=False, inverse=False, base=10000.0):
    want, size = _turned(x, pos, axes, halves, inverse, base)
    fi = torch.finfo(got.dtype)
    e = 2.0 ** -21 * size
    tol = fi.eps / 2 * (np.abs(want) + e) + e + fi.smallest_normal * fi.eps / 2
    tol[size == 0] = 0.0
    err = np.abs(got.cpu().double().numpy() - want)
    assert (err <= tol).all(), f"worst {np.max(err - tol):.3e}"


def _x(shape, dtype, rows=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    if rows:
        Bt, H, L, d = shape
        return torch.randn(Bt, L, H, d, generator=g).to(dtype).to(DEV).transpose(1, 2)
    return torch.randn(*shape, generator=g).to(dtype).to(DEV)


def _pos(L, n, Bt=None, seed=1, top=64):
    g = torch.Generator().manual_seed(seed)
    shape = (L, n) if Bt is None else (Bt, L, n)
    p = torch.rand(*shape, generator=g) * top
    return torch.where(torch.rand(shape, generator=g) < 0.5, p.floor(), p).to(DEV)


# (shape, axes): the last sections leave a tail of d, have odd halves (21: one pair per
# thread), or halves of 2, 4 and 8 modulo 16
SHAPES = [((1, 1, 1, 64), (16, 24, 24)), ((2, 5, 33, 128), (44, 42, 42)),
          ((1, 3, 130, 128), (16, 56, 56)), ((3, 2, 7, 120), (40, 40, 36)),
          ((1, 9, 17, 8), (2,)), ((2, 1, 64, 256), (64, 64, 64, 64)),
          ((1, 2, 257, 96), (8, 32, 32, 16)), ((1, 13, 40, 40), (2, 2, 2)),
          ((1, 4, 5, 64), (64,))]


@pytest.mark.parametrize("shape,axes", SHAPES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("halves", [False, True])
def test_matches_complex_rotation(shape, axes, dtype, halves):
    x = _x(shape, dtype, rows=halves)
    for inverse, batched in ((False, False), (True, True)):
        pos = _pos(shape[2], len(axes), shape[0] if batched else None)
        y = b.rotary(x, pos, axes, pairing=b.PAIR_HALVES if halves else b.PAIR_ADJACENT,
                     inverse=inverse)
        assert y.is_contiguous() and y.shape == x.shape
        _check(y, x, pos, axes, halves, inverse)


def test_far_fractional_and_negative_positions():
    x = _x((1, 2, 6, 128), torch.float32)
    pos = torch.tensor([[0.0, 0.5, -3.25], [16384.0, 1e6, 16777215.0], [-1e6, 123456.5, 7.0],
                        [1e9, -1e9, 4e9], [1.0, 0.0, 0.0], [32767.0, 4095.5, 0.0]]).to(DEV)
    _check(b.rotary(x, pos, (44, 42, 42), base=256.0), x, pos, (44, 42, 42), base=256.0)


def test_zero_position_and_tail_are_copied_bit_for_bit():
    x = _x((1, 3, 9, 72), torch.bfloat16)
    x[0, 0, 0, 70] = float("inf")
    x[0, 1, 2, 71] = float("nan")
    for pairing in (b.PAIR_ADJACENT, b.PAIR_HALVES):
        y = b.rotary(x, torch.zeros(9, 2, device=DEV), (32, 32), pairing=pairing)
        assert torch.equal(y.view(torch.int16), x.contiguous().view(torch.int16))
        y = b.rotary(x, torch.full((9, 2), 3.0, device=DEV), (32, 32), pairing=pairing)
        assert torch.equal(y[..., 64:].view(torch.int16), x[..., 64:].view(torch.int16))


def test_a_position_that_is_not_finite_spoils_its_token_alone():
    x = _x((1, 2, 4, 64), torch.float32)
    pos = _pos(4, 1)
    pos[2, 0] = float("inf")
    y = b.rotary(x, pos, (32,))
    assert torch.isnan(y[:, :, 2, :32]).all() and torch.equal(y[:, :, 2, 32:], x[:, :, 2, 32:])
    keep = [0, 1, 3]
    _check(y[:, :, keep], x[:, :, keep], pos[keep], (32,))


@pytest.mark.parametrize("pairing", [b.PAIR_ADJACENT, b.PAIR_HALVES])
def test_in_place_and_into_strided_outputs(pairing):
    shape, axes = (2, 6, 21, 128), (44, 42, 42)
    x = _x(shape, torch.bfloat16, rows=True)
    pos = _pos(21, 3, 2)
    want = b.rotary(x, pos, axes, pairing=pairing)
    # a slot of a wider buffer, whose other rows stay as they were
    wide = torch.full((2, 21, 10, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    b.rotary(x, pos, axes, pairing=pairing, out=wide[:, :, 2:8].transpose(1, 2))
    assert torch.equal(wide[:, :, 2:8].transpose(1, 2), want)
    assert (wide[:, :, :2] == 7).all() and (wide[:, :, 8:] == 7).all()
    # every batch entry from one broadcast tensor
    one = x[:1].expand(2, -1, -1, -1)
    assert torch.equal(b.rotary(one, pos, axes, pairing=pairing)[0], want[0])
    # in place
    b.rotary(x, pos, axes, pairing=pairing, out=x)
    assert torch.equal(x, want)


@pytest.mark.parametrize("pairing", [b.PAIR_ADJACENT, b.PAIR_HALVES])
def test_inverse_is_the_gradient(pairing):
    """<g, R x> = <R^T g, x>, and central differences of <g, R x> along a direction give
    <R^T g, direction>: R is linear, so the difference has no truncation error, and what
    remains is fp32 rounding, at most 2^-20 of the sum of |g| (|x_lo| + |x_hi|) + |x| (|g_lo|
    + |g_hi|) <= 4 |g| |x| over the components, divided by the step for the difference."""
    shape, axes = (1, 4, 50, 96), (24, 40, 28)
    x, g, v = (_x(shape, torch.float32, seed=s) for s in (3, 4, 5))
    pos = _pos(50, 3)
    rot = lambda t, inv=False: b.rotary(t, pos, axes, pairing=pairing, inverse=inv).double()
    back = rot(g, True)
    bound = lambda p, q: 2.0 ** -20 * 4 * float(p.double().norm() * q.double().norm())
    assert abs(float((g.double() * rot(x)).sum() - (back * x).sum())) <= bound(g, x)
    h = 0.25
    f = lambda t: float((g.double() * rot(t)).sum())
    diff = (f(x + h * v) - f(x - h * v)) / (2 * h)
    slack = (bound(g, x + h * v) + bound(g, x - h * v)) / (2 * h) + bound(g, v)
    assert abs(diff - float((back * v).sum())) <= slack
    # and there and back
    _check(rot(rot(x).float(), True).float(), rot(x).float(), pos, axes,
           pairing == b.PAIR_HALVES, True)


def test_another_stream_and_a_replayed_graph():
    x, pos, axes = _x((1, 8, 300, 64), torch.float16), _pos(300, 3), (16, 24, 24)
    want = b.rotary(x, pos, axes)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(want)
    b.rotary(x, pos, axes, out=out, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.rotary(x, pos, axes, out=out)
    x.copy_(_x(x.shape, torch.float16, seed=9))
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, b.rotary(x, pos, axes))


def test_more_than_2_31_elements():
    """Offsets past 32 bits: the last token of a tensor of 2^31 + elements."""
    L = (1 << 31) // (128 * 128) + 5
    x = torch.zeros(1, 128, L, 128, dtype=torch.bfloat16, device=DEV)
    x[0, 127, -3:] = _x((1, 1, 3, 128), torch.bfloat16)[0, 0]
    pos = torch.full((L, 1), 5.0, device=DEV)
    want = b.rotary(x[:, 127:, -3:].clone(), pos[-3:].clone(), (128,))
    b.rotary(x, pos, (128,), out=x)
    assert torch.equal(x[:, 127:, -3:], want)
    assert not x[0, 126, -1].any()


# CTAs that go on to further tokens: few heads, sections with odd halves, entries that end inside
# a CTA's tokens; threads per token that divide the CTA's, and that do not
@pytest.mark.parametrize("H,d,axes", [(3, 40, (2, 36)), (1, 64, (18, 46)), (13, 40, (38,))])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_few_heads_of_many_tokens(H, d, axes, dtype):
    Bt, L = 3, 13001
    x = _x((Bt, H, L, d), dtype, rows=True)
    pos = _pos(L, len(axes), Bt)
    y = b.rotary(x, pos, axes, pairing=b.PAIR_HALVES, inverse=True)
    _check(y, x, pos, axes, True, True)
    one = _pos(L, len(axes), seed=2)
    _check(b.rotary(x, one, axes, pairing=b.PAIR_HALVES), x, one, axes, True)
