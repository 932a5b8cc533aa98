"""bsa_linear against the formula in 64 bits.

Tolerance, from the arithmetic: a product of two 16-bit operands is exact in fp32; the
tensor core adds 16 of them at a time to the fp32 sum, so a sum over K takes K / 16 + 1
additions, each off by at most 2^-22 of the sum of magnitudes so far (an additional bit for
truncation instead of rounding), and split sums a few more: e = (K / 16 + 8) 2^-22 sum_k
|x_k w_k|. The bias adds 2^-24 of the result; the activations' slopes are at most 1.13 and
their own evaluation (one exponential, one division) is off by at most 2^-19 of |z|; the
gate scales this and the residual adds 2^-23 of the sum. Rounding to the type is half a step
of the result: eps/2 |y| (below the normal range, half of its smallest step).
"""
import math

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b

pytestmark = pytest.mark.gpu
DEV = "cuda"
ACTS = {b.ACT_NONE: lambda z: z,
        b.ACT_GELU_TANH: lambda z: z * torch.sigmoid(2 * math.sqrt(2 / math.pi)
                                                     * (z + 0.044715 * z ** 3)),
        b.ACT_GELU_ERF: lambda z: z * torch.special.ndtr(z),
        b.ACT_SILU: lambda z: z * torch.sigmoid(z)}


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _randn(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 31 * len(shape) + shape[-1])
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def _columns(x):
    """[Bt, H, L, d] -> [Bt, L, H d] in 64 bits on the host."""
    x = x.detach().cpu().double()
    return x.transpose(1, 2).flatten(2) if x.dim() == 4 else x


def _check(got, x, w, bias=None, act=b.ACT_NONE, gate=None, residual=None):
    xd, wd = _columns(x), w.detach().cpu().double()
    K = wd.shape[1]
    z = xd @ wd.t()
    e = (K / 16 + 8) * 2.0 ** -22 * (xd.abs() @ wd.abs().t())
    if bias is not None:
        z = z + bias.cpu().double()
        e = e + 2.0 ** -24 * z.abs()
    e = 1.13 * e + 2.0 ** -19 * z.abs() if act != b.ACT_NONE else e
    y = ACTS[act](z)
    if gate is not None:
        g = gate.cpu().double()[:, None]
        y, e = y * g, e * g.abs() + 2.0 ** -23 * (y * g).abs()
    if residual is not None:
        y = y + _columns(residual)
        e = e + 2.0 ** -23 * y.abs()
    fi = torch.finfo(got.dtype)
    tol = e + fi.eps / 2 * (y.abs() + e) + fi.smallest_normal * fi.eps / 2
    err = (_columns(got) - y).abs()
    assert bool((err <= tol).all()), f"worst {float((err - tol).max()):.3e} at {int((err - tol).argmax())}"


def _st():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# (Bt, L, K, N): one of everything; odd widths and a last row tile of one row; few rows over
# long sums; column tiles that end inside; entries merged into one run; many tiles per SM
SIZES = [(1, 1, 8, 1), (1, 1, 72, 9), (2, 77, 1000, 1003), (1, 300, 64, 64), (3, 129, 192, 320),
         (1, 257, 72, 257), (4, 1, 5120, 640), (2, 3, 4096, 1000), (1, 17, 2048, 384),
         (1, 64, 1024, 1024), (1, 65, 1024, 1032), (5, 31, 640, 512), (2, 513, 640, 512),
         (1, 40, 16384, 128), (1, 2304, 128, 2048), (3, 1000, 64, 5000)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matches_formula(size, dtype):
    Bt, L, K, N = size
    x, w = _randn(Bt, L, K, dtype=dtype), _randn(N, K, dtype=dtype, seed=1, scale=K ** -0.5)
    st = _st()
    y = b.linear(x, w, status=st)
    assert y.shape == (Bt, L, N) and y.is_contiguous()
    _check(y, x, w)
    bias, gate = _randn(N, dtype=dtype, seed=2), _randn(Bt, N, dtype=dtype, seed=3)
    res = _randn(Bt, L, N, dtype=dtype, seed=4)
    for act in ACTS:
        _check(b.linear(x, w, bias, act, gate, res, status=st), x, w, bias, act, gate, res)
    _check(b.linear(x, w, bias, b.ACT_SILU, None, res, status=st), x, w, bias, b.ACT_SILU, None, res)
    _check(b.linear(x, w, None, b.ACT_GELU_TANH, gate, status=st), x, w, None, b.ACT_GELU_TANH, gate)
    assert st.item() == 0


@pytest.mark.parametrize("hin,hout", [(1, 3), (2, 1), (5, 4), (12, 0), (0, 12)])
@pytest.mark.parametrize("Bt,L,d", [(1, 1, 64), (2, 130, 128), (3, 1, 128), (2, 7, 64)])
def test_heads_in_and_out(hin, hout, Bt, L, d):
    K, N = max(hin, 2) * d, max(hout, 3) * d
    x = _randn(Bt, hin, L, d) if hin > 1 else _randn(Bt, L, K)
    w, bias = _randn(N, K, seed=1, scale=K ** -0.5), _randn(N, seed=2)
    gate = _randn(Bt, N, seed=3)
    shape = (Bt, hout, L, d) if hout > 1 else (Bt, L, N)
    res = _randn(*shape, seed=5)
    heads = hout if hout > 1 else 0
    y = b.linear(x, w, bias, b.ACT_NONE, gate, res, heads=heads)
    assert y.shape == shape
    _check(y, x, w, bias, b.ACT_NONE, gate, res)


@pytest.mark.parametrize("Bt,L", [(2, 300), (2, 5)])
def test_strided_views_and_what_lies_beside_them(Bt, L):
    K, N = 192, 200
    wide = _randn(Bt, L, 3 * K)
    x = wide[:, :, K:2 * K]
    wall = _randn(N, K + 64, seed=1, scale=K ** -0.5)
    w = wall[:, 8:8 + K]
    res = _randn(1, L, N, seed=4).expand(Bt, L, N)
    for pad in (8, 3):   # row strides of whole 16 bytes, and not
        buf = torch.full((Bt, L + 2, N + pad), 9.0, dtype=torch.bfloat16, device=DEV)
        out = buf[:, 1:L + 1, :N]
        y = b.linear(x, w, residual=res, out=out)
        assert y.data_ptr() == out.data_ptr()
        _check(out, x, w, residual=res)
        assert (buf[:, 0] == 9).all() and (buf[:, L + 1] == 9).all() and (buf[:, :, N:] == 9).all()
    one = x[:1].expand(Bt, L, K)   # one tensor for every entry
    gate = _randn(Bt, N, seed=6)
    _check(b.linear(one, w, gate=gate), one, w, gate=gate)


@pytest.mark.parametrize("L,K,N", [(1, 1, 1), (5, 3, 130), (300, 17, 40)])
def test_sums_shorter_than_their_rows(L, K, N):
    """K of any size where the rows lie 16 bytes apart: what lies behind K is not read into it."""
    x = _randn(1, L, 24)
    w = _randn(N, 32, seed=1)
    x[..., K:], w[:, K:] = float("nan"), float("inf")
    _check(b.linear(x[..., :K], w[:, :K]), x[..., :K], w[:, :K])


@pytest.mark.parametrize("L,N", [(400, 256), (3, 256), (90, 77)])
def test_residual_in_place(L, N):
    x, w, r = _randn(2, L, 128), _randn(N, 128, seed=1, scale=0.1), _randn(2, L, N, seed=2)
    keep = r.clone()
    b.linear(x, w, residual=r, out=r)
    _check(r, x, w, residual=keep)


@pytest.mark.parametrize("L", [200, 6])
def test_a_row_that_is_not_finite_stays_alone(L):
    x, w = _randn(1, L, 256), _randn(300, 256, seed=1, scale=0.06)
    x[0, 3, 7], x[0, 4, 9], x[0, L - 1, 0] = float("nan"), float("inf"), float("-inf")
    y = b.linear(x, w)
    bad = [3, 4, L - 1]
    assert not torch.isfinite(y[0, bad]).any()
    keep = [i for i in range(L) if i not in bad]
    _check(y[:, keep], x[:, keep], w)


def test_activations_at_their_ends():
    """Sums that pass every finite exponent, and infinities, through each activation."""
    z = torch.tensor([0.0, -0.0, 1e-4, -1e-4, 5.0, -5.0, -12.0, 30.0, -30.0, 300.0, -300.0, 1e4, -1e4,
                      3e38, -3e38, float("inf")])
    x = torch.zeros(1, len(z), 8, dtype=torch.bfloat16)
    x[0, :, 0] = z.to(torch.bfloat16)
    w = torch.zeros(8, 8, dtype=torch.bfloat16)
    w[:, 0] = 1
    x, w = x.to(DEV), w.to(DEV)
    zd = x[0, :, 0].cpu().double()
    for act in ACTS:
        y = b.linear(x, w, act=act)[0, :, 0].cpu().double()
        want = torch.where(zd > 1e30, zd, torch.where(zd < -1e30, zd if act == b.ACT_NONE else 0.0, ACTS[act](zd)))
        tol = 2.0 ** -9 * 1.01 * want.abs() + 2.0 ** -18 * (want.abs() if act == b.ACT_NONE else zd.abs().clamp(max=40))
        fin = torch.isfinite(want)
        assert bool(((y - want).abs()[fin] <= tol[fin]).all()), (act, y, want)
        assert torch.equal(y[~fin], want[~fin])


def test_same_bits_every_time_other_streams_and_a_replayed_graph():
    for L, K, N in ((3, 4096, 1100), (700, 256, 512)):
        x, w, bias = _randn(2, L, K), _randn(N, K, seed=1, scale=K ** -0.5), _randn(N, seed=2)
        want = b.linear(x, w, bias)
        s = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.zeros_like(want) for _ in s]
        torch.cuda.synchronize()
        for o, q in zip(outs, s):   # at once, each with a workspace of its own
            with torch.cuda.stream(q):
                for _ in range(5):
                    b.linear(x, w, bias, out=o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        graph = torch.cuda.CUDAGraph()
        out = torch.zeros_like(want)
        with torch.cuda.graph(graph):
            b.linear(x, w, bias, out=out)
        x.copy_(_randn(2, L, K, seed=8))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.linear(x, w, bias))


@pytest.mark.parametrize("L,K,N", [(2, 8192, 256), (300, 16384, 128)])
def test_workspace_at_any_16_byte_boundary(L, K, N):
    x, w = _randn(1, L, K), _randn(N, K, seed=1, scale=K ** -0.5)
    need = b.bsa_linear_workspace_bytes(1, L, K, N)
    assert need > 0
    want = b.linear(x, w)
    _check(want, x, w)
    for off in (16, 32, 48):
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
        assert torch.equal(b.linear(x, w, ws=ws[off:off + need]), want)
        assert (ws[:off] == 255).all() and (ws[off + need:] == 255).all()


def test_more_than_2_31_outputs():
    """Offsets past 32 bits: rows at the end of an output of 2^31 + elements."""
    N = 4096
    L = (1 << 31) // N + 260
    x = torch.zeros(1, L, 8, dtype=torch.bfloat16, device=DEV)
    x[0, -300:] = _randn(1, 300, 8)[0]
    w = _randn(N, 8, seed=1)
    y = b.linear(x, w)
    assert not y[0, :L - 300].any()
    _check(y[:, -300:], x[:, -300:], w)


# the residual's rows, heads or entries one copy; its base and rows off 16 bytes while the
# output's are on them, and the other way round
@pytest.mark.parametrize("L", [300, 4])
@pytest.mark.parametrize("kind", ["rows", "heads", "entries", "base", "stride", "out"])
def test_residuals_and_outputs_of_any_stride(L, kind):
    Bt, K, H, d = 2, 328, 4, 64
    N = H * d
    x, w = _randn(Bt, L, K), _randn(N, K, seed=1, scale=K ** -0.5)
    gate, out = _randn(Bt, N, seed=3), None
    if kind == "rows":
        res = _randn(Bt, H, 1, d, seed=4).expand(Bt, H, L, d)
    elif kind == "heads":
        res = _randn(Bt, 1, L, d, seed=4).expand(Bt, H, L, d)
    elif kind == "entries":
        res = _randn(1, H, L, d, seed=4).expand(Bt, H, L, d)
    elif kind == "base":
        res = _randn(Bt * H * L * d + 3, 1, seed=4)[3:].view(Bt, H, L, d)
    elif kind == "stride":
        res = _randn(Bt, H, L, d + 5, seed=4)[..., :d]
    else:
        res = _randn(Bt, H, L, d, seed=4)
        out = torch.full((Bt, H, L, d + 2), 9.0, dtype=torch.bfloat16, device=DEV)[..., :d]
    y = b.linear(x, w, None, b.ACT_SILU, gate, res, heads=H, out=out)
    _check(y, x, w, None, b.ACT_SILU, gate, res)
    if out is not None:
        assert y.data_ptr() == out.data_ptr()


@pytest.mark.parametrize("L", [300, 4])
@pytest.mark.parametrize("step", [8, 16, 3])
def test_a_residual_whose_rows_overlap(L, step):
    """A window that moves by fewer elements than it is wide: rows are only read."""
    N, K = 192, 136
    x, w = _randn(1, L, K), _randn(N, K, seed=1, scale=K ** -0.5)
    res = _randn(L * step + N, 1, seed=4).as_strided((1, L, N), (0, step, 1))
    _check(b.linear(x, w, residual=res), x, w, residual=res)
    xs = _randn(L * 8 + K, 1, seed=5).as_strided((1, L, K), (0, 8, 1))
    _check(b.linear(xs, w), xs, w)
