"""A transformer block as it would be run: projections into heads, rotary positions, the
block attention, the gated output projection, cross attention to text, the feed-forward layer.
Every step is checked, by the tolerance of its own test, against the formula on what the step
before it left on the GPU; then the whole is captured, replayed and compared bit for bit.
"""
import numpy as np
import pytest
import torch

import oracle as orc
from piecewise_attention_diffusion_b200 import bsattn as b
from tests import test_gpu_cross as tc
from tests import test_gpu_linear as tl
from tests import test_gpu_rotary as tr
from tests._util import assert_close_out, f64

pytestmark = pytest.mark.gpu
DEV = "cuda"
BT, H, L, D, BLOCK, KTOP, TEXT, WIDE = 2, 2, 512, 64, 64, 3, 77, 96
C = H * D
AXES = (16, 24, 24)


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _inputs(seed):
    g = torch.Generator().manual_seed(seed)

    def rnd(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g) * scale).to(torch.bfloat16).to(DEV)

    p = {n: rnd(C, C, scale=C ** -0.5) for n in ("q", "k", "v", "o", "cq", "co")}
    p |= {n: rnd(C, WIDE, scale=WIDE ** -0.5) for n in ("ck", "cv")}
    p |= {"up": rnd(4 * C, C, scale=C ** -0.5), "down": rnd(C, 4 * C, scale=(4 * C) ** -0.5),
          "mod": rnd(2 * C, C, scale=C ** -0.5), "bias": rnd(C), "bias_up": rnd(4 * C),
          "bias_mod": rnd(2 * C)}
    i = torch.arange(L)
    pos = torch.stack((i // 64, i // 8 % 8, i % 8), 1).float().to(DEV)
    return p, rnd(BT, L, C), rnd(BT, TEXT, WIDE), rnd(BT, 1, C), pos, \
        torch.tensor([TEXT, 31], dtype=torch.int32, device=DEV)


def _block(p, x, text, step, pos, n_text, status):
    """The block's output and everything on the way."""
    r = {}
    mod = r["mod"] = b.linear(step, p["mod"], p["bias_mod"], b.ACT_SILU, status=status)
    g1, g2 = (t.contiguous() for t in mod[:, 0].chunk(2, 1))
    r["g1"], r["g2"] = g1, g2
    q, k, v = (b.linear(x, p[n], p["bias"], heads=H, status=status) for n in "qkv")
    r["q0"], r["k0"], r["v"] = q, k, v
    q, k = r["q"], r["k"] = b.rotary(q, pos, AXES), b.rotary(k, pos, AXES)
    stats = r["stats"] = b.precompute(k, v, BLOCK, status=status)
    r["lists"] = b.route(q, stats["kbar"], stats["Mnorm"], BLOCK, KTOP, status=status)
    o, _ = b.forward(q, k, v, BLOCK, r["lists"][0], r["lists"][1], 1, b.MODE_PISA, stats=stats,
                     status=status)
    r["o"] = o
    y = r["y"] = b.linear(o, p["o"], p["bias"], gate=g1, residual=x, status=status)
    cq = r["cq"] = b.linear(y, p["cq"], heads=H, status=status)
    ck, cv = (b.linear(text, p[n], heads=H, status=status) for n in ("ck", "cv"))
    r["ck"], r["cv"] = ck, cv
    c, _ = b.cross_forward(cq, ck, cv, key_len=n_text, status=status)
    r["c"] = c
    z = r["z"] = b.linear(c, p["co"], p["bias"], residual=y, status=status)
    up = r["up"] = b.linear(z, p["up"], p["bias_up"], b.ACT_GELU_TANH, status=status)
    r["out"] = b.linear(up, p["down"], p["bias"], gate=g2, residual=z, status=status)
    return r


def test_block_step_by_step():
    p, x, text, step, pos, n_text = _inputs(1)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = _block(p, x, text, step, pos, n_text, st)
    assert st.item() == 0, b.status_string(st.item())
    tl._check(r["mod"], step, p["mod"], p["bias_mod"], b.ACT_SILU)
    for n, got in (("q", "q0"), ("k", "k0"), ("v", "v")):
        tl._check(r[got], x, p[n], p["bias"])
    tr._check(r["q"], r["q0"], pos, AXES)
    tr._check(r["k"], r["k0"], pos, AXES)
    # the block attention with the lists that the GPU chose
    M, scale = L // BLOCK, D ** -0.5
    rp, ci = (t.cpu().numpy() for t in r["lists"][:2])
    for h in range(BT * H):
        qh, kh, vh = (f64(r[n].reshape(BT * H, L, D)[h]) for n in "qkv")
        kbar, vsum, _, Hbar, _ = orc.precompute_head(kh, vh, BLOCK)
        grp, gci = orc.head_csr(rp, ci, h, M, True)
        want, _ = orc.pisa_head(qh, kh, vh, np.asarray(grp), np.asarray(gci), BLOCK, scale, kbar,
                                vsum, Hbar)
        assert_close_out(r["o"].reshape(BT * H, L, D)[h], want, f"head {h}")
    tl._check(r["y"], r["o"], p["o"], p["bias"], gate=r["g1"], residual=x)
    tl._check(r["cq"], r["y"], p["cq"])
    tl._check(r["ck"], text, p["ck"])
    tc._check(r["c"], None, r["cq"], r["ck"], r["cv"], key_len=n_text)
    tl._check(r["z"], r["c"], p["co"], p["bias"], residual=r["y"])
    tl._check(r["up"], r["z"], p["up"], p["bias_up"], b.ACT_GELU_TANH)
    tl._check(r["out"], r["up"], p["down"], p["bias"], gate=r["g2"], residual=r["z"])


def test_block_captured_and_replayed():
    p, x, text, step, pos, n_text = _inputs(2)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    _block(p, x, text, step, pos, n_text, st)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = _block(p, x, text, step, pos, n_text, st)["out"]
    _, x2, text2, step2, _, _ = _inputs(3)
    for dst, src in ((x, x2), (text, text2), (step, step2)):
        dst.copy_(src)
    graph.replay()
    torch.cuda.synchronize()
    want = _block(p, x, text, step, pos, n_text, st)["out"]
    assert torch.isfinite(want).all() and torch.equal(got, want) and st.item() == 0


def test_helpers_on_a_given_stream_keep_their_workspaces():
    """A helper's workspace belongs to the stream it was asked for: what the current stream
    allocates and writes right after the call does not reach it."""
    s = torch.cuda.Stream()
    x, w = tl._randn(1, 4, 8192), tl._randn(256, 8192, seed=1, scale=8192 ** -0.5)
    q, k, v = tc._randn(1, 2, 1, 64), tc._randn(1, 2, 30000, 64, seed=1), tc._randn(1, 2, 30000, 64, seed=2)
    assert b.bsa_linear_workspace_bytes(1, 4, 8192, 256) > 0
    want_y, want_o = b.linear(x, w), b.cross_forward(q, k, v)[0]
    torch.cuda.synchronize()
    for _ in range(20):
        ys = [b.linear(x, w, stream=s) for _ in range(4)]
        os_ = [b.cross_forward(q, k, v, stream=s)[0] for _ in range(4)]
        junk = [torch.full((1 << 18,), float("nan"), device=DEV) for _ in range(8)]
        s.synchronize()
        assert all(torch.equal(y, want_y) for y in ys) and all(torch.equal(o, want_o) for o in os_)
        del junk
