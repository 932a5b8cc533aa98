"""bsa_cross_forward against softmax attention over the real keys in 64 bits.

Tolerance, from the arithmetic. A score is a sum of d exact products, added 16 at a time in
fp32: off by at most es = (d / 16 + 2) 2^-22 s sum |q k|, with the exponent's own rounding
(|x| 2^-23 for an exponent x up to 2^7 that still counts) and the exponential's (2^-18 with a
polynomial on part of them) p is off by ep = 2 es + 2^-16 / 2 relative. Rounding p to the type
adds eps/2; in fp16, whose p is held 2^7 times larger, a p below the normal range is off by
2^-32 of the largest instead. The products with v add (Lk / 16 + 8) 2^-22. All of this scales
the weighted mean of |v|; the output's rounding adds eps/2 |o|. The denominator has the same
ep; lse is off by ep and its own rounding.
"""
import math

import pytest
import torch

from piecewise_attention_diffusion_b200 import bsattn as b

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.fixture(autouse=True)
def _need_gpu(cuda_ok):
    yield


def _randn(*shape, dtype=torch.bfloat16, seed=0, scale=1.0):
    g = torch.Generator().manual_seed(seed + 7 * shape[-2] + shape[1])
    return (torch.randn(*shape, generator=g) * scale).to(dtype).to(DEV)


def _exact(q, k, v, key_len=None, key_mask=None, scale=0.0):
    """(o, lse, tolerance of o, of lse) in 64 bits on the host."""
    q, k, v = (t.detach().cpu().double() for t in (q, k, v))
    Bt, H, Lq, d = q.shape
    Hkv, Lk = k.shape[1:3]
    s = scale or d ** -0.5
    eps = torch.finfo(b_type[0]).eps
    o, lse = torch.zeros(Bt, H, Lq, d).double(), torch.full((Bt, H, Lq), -math.inf).double()
    to, tl = torch.zeros_like(o), torch.zeros_like(lse)
    for i in range(Bt):
        real = torch.ones(Lk, dtype=torch.bool)
        if key_len is not None:
            real[max(0, int(key_len[i])):] = False
        if key_mask is not None:
            real &= key_mask[i].cpu() != 0
        if not real.any():
            continue
        for h in range(H):
            kk, vv = k[i, h * Hkv // H, real], v[i, h * Hkv // H, real]
            z = s * q[i, h] @ kk.t()
            size = s * q[i, h].abs() @ kk.abs().t()
            ep = 2 * (d / 16 + 2) * 2.0 ** -22 * size.amax(1) + 2.0 ** -17
            lse[i, h] = torch.logsumexp(z, 1)
            w = torch.exp(z - lse[i, h][:, None])
            o[i, h] = w @ vv
            rel = 2 * ep + eps / 2 + (Lk / 16 + 8) * 2.0 ** -22
            to[i, h] = rel[:, None] * (w @ vv.abs())
            if b_type[0] == torch.float16:
                to[i, h] += 2.0 ** -32 * w.amax(1, keepdim=True) * vv.abs().sum(0)
            tl[i, h] = ep + 2.0 ** -22 * lse[i, h].abs()
    fi = torch.finfo(b_type[0])
    to = to + fi.eps / 2 * (o.abs() + to) + fi.smallest_normal * fi.eps / 2
    return o, lse, to, tl


b_type = [torch.bfloat16]   # the type of the case at hand


def _check(o, lse, q, k, v, **kw):
    b_type[0] = q.dtype
    want, wl, to, tl = _exact(q, k, v, **kw)
    err = (o.cpu().double() - want).abs()
    assert bool((err <= to).all()), f"worst {float((err - to).max()):.3e}, error {float(err.max()):.3e}"
    if lse is not None:
        got = lse.cpu().double()
        none = wl == -math.inf
        assert torch.equal(got[none], wl[none])
        err = (got - wl)[~none].abs()
        assert bool((err <= tl[~none]).all()), f"lse: {float((err - tl[~none]).max()):.3e}"


def _st():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# (Bt, H, Hkv, Lq, Lk, d): one and no key; tiles that end inside, on the border and past it, in
# queries and keys; key heads shared; few queries over many keys (split), with and without sharing
SIZES = [(1, 1, 1, 1, 1, 64), (2, 2, 1, 3, 0, 64), (1, 2, 2, 128, 128, 128), (2, 3, 3, 129, 77, 64),
         (1, 4, 2, 255, 127, 128), (2, 2, 2, 257, 129, 128), (1, 5, 1, 300, 300, 64),
         (3, 2, 2, 513, 640, 128), (1, 40, 40, 640, 512, 128), (2, 16, 4, 1000, 77, 64),
         (1, 2, 2, 1, 2000, 64), (2, 4, 2, 1, 5000, 128), (1, 1, 1, 7, 20000, 64),
         (2, 8, 1, 2, 1537, 128), (1, 4, 4, 100, 1025, 64), (1, 2, 1, 130, 4096, 128)]


@pytest.mark.parametrize("size", SIZES)
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_matches_softmax(size, dtype):
    Bt, H, Hkv, Lq, Lk, d = size
    q = _randn(Bt, H, Lq, d, dtype=dtype)
    k, v = (_randn(Bt, Hkv, Lk, d, dtype=dtype, seed=s) for s in (1, 2))
    st = _st()
    o, lse = b.cross_forward(q, k, v, want_lse=True, status=st)
    assert o.is_contiguous() and st.item() == 0
    _check(o, lse, q, k, v)
    o2, none = b.cross_forward(q, k, v, scale=0.3)
    assert none is None
    _check(o2, None, q, k, v, scale=0.3)


def _spoil(k, v, key_len, key_mask):
    """NaN and infinities where no key is real."""
    Lk = k.shape[2]
    for i in range(k.shape[0]):
        out = torch.zeros(Lk, dtype=torch.bool, device=DEV)
        if key_len is not None:
            out[max(0, int(key_len[i])):] = True
        if key_mask is not None:
            out |= key_mask[i] == 0
        at = out.nonzero()[:, 0]
        for j, bad in enumerate((float("nan"), float("inf"), float("-inf"), 3e4)):
            k[i, :, at[j::4]] = bad
            v[i, :, at[j::4]] = bad


@pytest.mark.parametrize("size", [(4, 2, 2, 130, 300, 64), (5, 2, 1, 257, 129, 128),
                                  (4, 2, 1, 1, 3000, 64), (3, 4, 4, 5, 2050, 128),
                                  (4, 16, 16, 64, 77, 64)])
@pytest.mark.parametrize("kind", ["count", "mask", "both"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_keys_that_are_not_real(size, kind, dtype):
    Bt, H, Hkv, Lq, Lk, d = size
    q = _randn(Bt, H, Lq, d, dtype=dtype)
    k, v = (_randn(Bt, Hkv, Lk, d, dtype=dtype, seed=s) for s in (1, 2))
    key_len = key_mask = None
    if kind != "mask":   # none, one, some and all; the tile's border
        key_len = torch.tensor([0, Lk, 1, min(128, Lk), Lk - 1][:Bt], dtype=torch.int32, device=DEV)
    if kind != "count":
        g = torch.Generator().manual_seed(5)
        key_mask = (torch.rand(Bt, Lk, generator=g) < 0.6).to(torch.uint8).to(DEV) * 3
        key_mask[1] = 0                       # nothing left
        key_mask[Bt - 1, :min(Lk - 1, 200)] = 0   # nothing in the first tiles
        key_mask[Bt - 1, Lk - 1] = 255
    _spoil(k, v, key_len, key_mask)
    st = _st()
    o, lse = b.cross_forward(q, k, v, key_len, key_mask, want_lse=True, status=st)
    assert st.item() == 0
    z = torch.zeros((), dtype=dtype, device=DEV)
    _check(o, lse, q, torch.where(torch.isfinite(k), k, z), torch.where(torch.isfinite(v), v, z),
           key_len=key_len, key_mask=key_mask)
    empty = [i for i in range(Bt) if (key_len is not None and int(key_len[i]) == 0)
             or (key_mask is not None and i == 1)]
    assert not o[empty].any() and (lse[empty] == float("-inf")).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("scale,sign", [(1e-3, 0), (0.3, 0), (1.0, 1), (1.0, -1), (6.0, -1), (25.0, 0)])
@pytest.mark.parametrize("kept", [0.03, 0.5, 0.97])
def test_masked_scores_against_any_reference(dtype, d, scale, sign, kept):
    """Scores near 0, all positive, all (far) negative and large ones, with few and many keys
    masked: whatever the masked keys hold must not reach the rows' references nor their sums."""
    Lq, Lk = 131, 650
    q, k, v = (_randn(1, 2, n, d, dtype=dtype, seed=s) for n, s in ((Lq, 0), (Lk, 1), (Lk, 2)))
    if sign:   # |q| and +-|k|: every score has this sign
        q, k = q.abs(), k.abs() * sign
    q = (q.float() * scale).to(dtype)
    g = torch.Generator().manual_seed(int(kept * 100) + d)
    mask = (torch.rand(1, Lk, generator=g) < kept).to(torch.uint8).to(DEV)
    mask[0, 130:256] = 0          # a tile with two real keys at most, then one with none
    mask[0, 256:384] = 0
    k[:, :, 384:][:, :, mask[0, 384:] == 0] = float("nan")
    k[:, :, :130][:, :, mask[0, :130] == 0] *= -50.0
    o, lse = b.cross_forward(q, k, v, key_mask=mask, want_lse=True)
    z = torch.zeros((), dtype=dtype, device=DEV)
    _check(o, lse, q, torch.where(torch.isfinite(k), k, z), v, key_mask=mask)


@pytest.mark.parametrize("Lq", [140, 2])
def test_counts_out_of_range_are_reported_and_clamped(Lq):
    q, k, v = _randn(3, 2, Lq, 64), _randn(3, 2, 1100, 64, seed=1), _randn(3, 2, 1100, 64, seed=2)
    st = _st()
    o, _ = b.cross_forward(q, k, v, torch.tensor([-5, 70, 1 << 30], dtype=torch.int32, device=DEV),
                           status=st)
    assert st.item() == b.ERR_BAD_PADDING
    _check(o, None, q, k, v, key_len=torch.tensor([0, 70, 1100]))


@pytest.mark.parametrize("Lq,Lk", [(200, 333), (2, 1500)])
def test_strided_views_and_what_lies_beside_them(Lq, Lk):
    Bt, H, d = 2, 3, 64
    qkv = _randn(Bt, Lq, 2 * H, d)
    q = qkv[:, :, H:].transpose(1, 2)
    kv = _randn(Bt, Lk, 4 * H, d, seed=1)
    k, v = kv[:, :, :H].transpose(1, 2), kv[:, :, 2 * H:3 * H].transpose(1, 2)
    buf = torch.full((Bt, Lq + 3, H, d), 5.0, dtype=torch.bfloat16, device=DEV)
    out = buf[:, 1:Lq + 1].transpose(1, 2)
    o, lse = b.cross_forward(q, k, v, out=out, want_lse=True)
    assert o.data_ptr() == out.data_ptr()
    _check(o, lse, q, k, v)
    assert (buf[:, 0] == 5).all() and (buf[:, Lq + 1:] == 5).all()
    # one encoder for every entry, one key head for every query head
    k1, v1 = (t[:1, :1].expand(Bt, H, Lk, d) for t in (k, v))
    o, lse = b.cross_forward(q, k1, v1, want_lse=True)
    _check(o, lse, q, k1, v1)


@pytest.mark.parametrize("d,Lk", [(64, 2000), (128, 3001)])
def test_workspace_at_any_16_byte_boundary_and_outputs_too(d, Lk):
    q, k, v = _randn(1, 3, 1, d), _randn(1, 3, Lk, d, seed=1), _randn(1, 3, Lk, d, seed=2)
    need = b.bsa_cross_workspace_bytes(1, 3, 3, 1, Lk, d)
    assert need > 0
    for off in (0, 16, 32, 48):
        ws = torch.full((need + 64,), 255, dtype=torch.uint8, device=DEV)
        buf = torch.full((3 * d + 64,), 6.0, dtype=torch.bfloat16, device=DEV)
        out = buf[off // 2:off // 2 + 3 * d].view(1, 3, 1, d)
        o, lse = b.cross_forward(q, k, v, ws=ws[off:off + need], out=out, want_lse=True)
        _check(o, lse, q, k, v)
        assert (ws[:off] == 255).all() and (ws[off + need:] == 255).all()
        assert (buf[:off // 2] == 6).all() and (buf[off // 2 + 3 * d:] == 6).all()


@pytest.mark.parametrize("Lq,Lk", [(150, 260), (3, 1300)])
def test_scores_at_their_ends(Lq, Lk):
    """Scores in the thousands of either sign, rows that grow from tile to tile, and rows that
    are not finite, which stay alone."""
    q, k, v = _randn(1, 2, Lq, 64, scale=30.0), _randn(1, 2, Lk, 64, seed=1, scale=10.0), _randn(
        1, 2, Lk, 64, seed=2)
    k = (k.float() * torch.linspace(0.1, 3.0, Lk, device=DEV)[:, None]).to(torch.bfloat16)
    o, lse = b.cross_forward(q, k, v, want_lse=True)
    assert torch.isfinite(o).all()
    _check(o, lse, q, k, v)
    q[0, 0, 1, 3], q[0, 1, Lq - 1, 0], q[0, 1, 0, 0] = float("nan"), float("nan"), float("inf")
    got, glse = b.cross_forward(q, k, v, want_lse=True)
    for h, t in ((0, 1), (1, Lq - 1), (1, 0)):
        assert torch.isnan(got[0, h, t]).all() and torch.isnan(glse[0, h, t])
        got[0, h, t], glse[0, h, t] = o[0, h, t], lse[0, h, t]
    assert torch.equal(got, o) and torch.equal(glse, lse)


def test_v_that_is_not_finite_spoils_its_column_alone():
    q, k, v = _randn(1, 1, 130, 64), _randn(1, 1, 200, 64, seed=1), _randn(1, 1, 200, 64, seed=2)
    want, _ = b.cross_forward(q, k, v)
    v[0, 0, 150, 5] = float("nan")
    got, _ = b.cross_forward(q, k, v)
    assert torch.isnan(got[..., 5]).all()
    keep = [c for c in range(64) if c != 5]
    assert torch.equal(got[..., keep], want[..., keep])


def test_same_bits_every_time_other_streams_and_a_replayed_graph():
    for Lq, Lk in ((600, 500), (2, 6000)):
        q, k, v = _randn(2, 4, Lq, 64), _randn(2, 2, Lk, 64, seed=1), _randn(2, 2, Lk, 64, seed=2)
        n = torch.tensor([Lk - 3, Lk // 2], dtype=torch.int32, device=DEV)
        want, lse = b.cross_forward(q, k, v, n, want_lse=True)
        streams = [torch.cuda.Stream() for _ in range(2)]
        outs = [torch.zeros_like(want) for _ in streams]
        torch.cuda.synchronize()
        for o, s in zip(outs, streams):
            with torch.cuda.stream(s):
                for _ in range(5):
                    b.cross_forward(q, k, v, n, out=o)
        torch.cuda.synchronize()
        assert all(torch.equal(o, want) for o in outs)
        out = torch.zeros_like(want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            b.cross_forward(q, k, v, n, out=out)
        q.copy_(_randn(2, 4, Lq, 64, seed=8))
        n.copy_(torch.tensor([Lk // 3, 0], dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, b.cross_forward(q, k, v, n)[0])


def test_more_than_2_31_elements_of_keys():
    """Offsets past 32 bits: the last keys of K and V of 2^31 + elements, for one query."""
    Lk = (1 << 31) // 128 + 300
    k = torch.zeros(1, 1, Lk, 128, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    mask = torch.zeros(1, Lk, dtype=torch.uint8, device=DEV)
    mask[0, -200:] = 1
    k[0, 0, -200:], v[0, 0, -200:] = _randn(1, 1, 200, 128)[0, 0], _randn(1, 1, 200, 128, seed=1)[0, 0]
    q = _randn(1, 1, 2, 128, seed=3)
    o, lse = b.cross_forward(q, k, v, key_mask=mask, want_lse=True)
    _check(o, lse, q, k[:, :, -200:], v[:, :, -200:])


# key counts that share the CTAs of few query rows: alike, apart, all but one empty, none; more
# heads than a wave of CTAs; more entries than a warp's lanes; few keys in all
@pytest.mark.parametrize("size,lens", [
    ((2, 16, 16, 1, 9000, 64), (9000, 9000)), ((3, 4, 4, 1, 9000, 128), (9000, 1, 0)),
    ((8, 2, 2, 1, 5000, 64), (0, 0, 0, 4999, 0, 0, 0, 0)), ((3, 2, 1, 2, 4000, 64), (0, 0, 0)),
    ((40, 1, 1, 3, 1500, 64), tuple(1500 * (i % 3 == 0) + i for i in range(39)) + (7,)),
    ((100, 1, 1, 1, 700, 128), tuple(7 * i for i in range(100))),
    ((10, 40, 40, 1, 600, 64), (600, 599, 0, 1, 257, 300, 0, 128, 64, 600)),
    ((2, 4, 1, 1, 31, 64), (31, 2)), ((149, 1, 1, 1, 300, 64), (300,) * 149)])
def test_key_counts_share_the_work(size, lens):
    Bt, H, Hkv, Lq, Lk, d = size
    q = _randn(Bt, H, Lq, d)
    k, v = (_randn(Bt, Hkv, Lk, d, seed=s) for s in (1, 2))
    n = torch.tensor([min(x, Lk) for x in lens], dtype=torch.int32, device=DEV)
    _spoil(k, v, n, None)
    st = _st()
    o, lse = b.cross_forward(q, k, v, key_len=n, want_lse=True, status=st)
    assert st.item() == 0
    _check(o, lse, q, k, v, key_len=n)
    again, _ = b.cross_forward(q, k, v, key_len=n)
    assert torch.equal(o, again)


# query heads that share a key head: one after the other in memory (taken as one head), in rows
# side by side, with gaps between heads or rows, all heads one copy
@pytest.mark.parametrize("Lq", [1, 2, 5, 40, 300])
@pytest.mark.parametrize("layout", ["heads", "rows", "head gaps", "row gaps", "one copy"])
def test_query_heads_of_one_key_head(Lq, layout):
    Bt, H, Hkv, Lk, d = 2, 12, 2, 1300, 64
    q = _randn(Bt, H, Lq, d)
    if layout == "rows":
        q = q.transpose(1, 2).contiguous().transpose(1, 2)
    elif layout == "head gaps":
        q = _randn(Bt, H, Lq + 3, d)[:, :, :Lq]
    elif layout == "row gaps":
        q = _randn(Bt, H, Lq, 2 * d)[..., :d]
    elif layout == "one copy":
        q = q[:, :1].expand(Bt, H, Lq, d)
    k, v = (_randn(Bt, Hkv, Lk, d, seed=s) for s in (1, 2))
    n = torch.tensor([Lk, 700], dtype=torch.int32, device=DEV)
    for out in ("heads", "rows"):
        room = torch.full((Bt, H, Lq, d) if out == "heads" else (Bt, Lq, H, d), 7.0, dtype=q.dtype,
                          device=DEV)
        o = room if out == "heads" else room.transpose(1, 2)
        o, lse = b.cross_forward(q, k, v, key_len=n, want_lse=True, out=o)
        _check(o, lse, q, k, v, key_len=n)


# heads and masks together where heads are folded, and long runs of keys joined from many parts
@pytest.mark.parametrize("size", [(2, 8, 2, 1, 3001, 128), (1, 8, 1, 33, 2500, 64),
                                  (3, 6, 2, 1, 900, 64), (1, 1, 1, 1, 70000, 64),
                                  (2, 40, 8, 1, 2049, 128)])
def test_folded_heads_under_masks_and_counts(size):
    Bt, H, Hkv, Lq, Lk, d = size
    q = _randn(Bt, H, Lq, d, dtype=torch.float16)
    k, v = (_randn(Bt, Hkv, Lk, d, dtype=torch.float16, seed=s) for s in (1, 2))
    g = torch.Generator().manual_seed(3)
    mask = (torch.rand(Bt, Lk, generator=g) < 0.7).to(torch.uint8).to(DEV)
    n = torch.tensor([Lk - 3, Lk // 3, 0][:Bt], dtype=torch.int32, device=DEV)
    _spoil(k, v, n, mask)
    o, lse = b.cross_forward(q, k, v, key_len=n, key_mask=mask, want_lse=True)
    _check(o, lse, q, k, v, key_len=n, key_mask=mask)
