"""The operators around the block attention of a diffusion transformer: what is measured, and their plain forms.

Three operators, in the order in which a transformer block calls them around the library's attention:

  linear   Y = R + g * act(X W^T + b): the Q/K/V projections (written head by head, the layout that the
           attention reads), the output projection (read head by head), the feed-forward layers, and the
           modulation and embedding layers that see few rows;
  rotary   rotary positions with several axes (time, height, width) on the projected queries and keys,
           and the transposed map for gradients;
  cross    attention of the image or video tokens over an encoder's states of another length, with
           real-key counts or masks, shared key heads, and few queries over many keys.

Sizes are those of the library's own workloads (40 heads x 16384 tokens x 128, 16 heads x 1152 tokens x 64,
77 text tokens) or generic.
"""
import math

import torch

own = False

TYPES = {"bfloat16": torch.bfloat16, "float16": torch.float16, "float32": torch.float32}


# ------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the video workload's queries as the projection leaves them, [batch, token, head, d]: 16 x 32 x 32 tokens,
        # time / height / width axes, written head by head for the attention
        dict(name="rotary_video", op="rotary", bt=1, h=40, l=16384, d=128, axes="44,42,42", pairing="adjacent",
             inverse=False, layout="rows", batched=False, type="bfloat16"),
        # the multimodal workload: every batch entry with positions of its own (crops), halves paired
        dict(name="rotary_multimodal", op="rotary", bt=8, h=16, l=1152, d=64, axes="16,24,24", pairing="halves",
             inverse=False, layout="rows", batched=True, type="float16"),
        # a gradient in 32 bits taken back through the rotation: odd token count, a tail of d left unrotated
        dict(name="rotary_gradient", op="rotary", bt=2, h=12, l=4099, d=120, axes="40,40,36", pairing="adjacent",
             inverse=True, layout="heads", batched=False, type="float32"),
        # one token per batch entry (a timestep or pooled token): latency
        dict(name="rotary_token", op="rotary", bt=2, h=16, l=1, d=64, axes="16,24,24", pairing="adjacent",
             inverse=False, layout="rows", batched=True, type="bfloat16"),
        # video tokens over 512 encoder states, all real
        dict(name="cross_video", op="cross", bt=1, h=40, hkv=40, lq=16384, lk=512, d=128, keys="all", lse=False,
             layout="heads", type="bfloat16"),
        # a batch of images over up to 77 text tokens, some prompts empty (the unconditional half of a batch)
        dict(name="cross_multimodal", op="cross", bt=8, h=16, hkv=16, lq=1024, lk=77, d=64, keys="count", lse=False,
             layout="rows", type="float16"),
        # a ragged image over a long reference sequence, key heads shared by four query heads, masked holes
        dict(name="cross_reference", op="cross", bt=2, h=16, hkv=4, lq=4101, lk=4352, d=128, keys="mask", lse=True,
             layout="rows", type="bfloat16"),
        # one query token per entry over a long encoder sequence: work split over the keys
        dict(name="cross_token", op="cross", bt=2, h=16, hkv=16, lq=1, lk=32768, d=64, keys="count", lse=True,
             layout="heads", type="bfloat16"),
        # the video workload's output projection: the attention's O read head by head, gate and residual
        dict(name="linear_video_out", op="linear", bt=1, l=16384, k=5120, n=5120, hin=40, hout=0, act="none",
             bias=True, gate=True, residual=True, type="bfloat16"),
        # the multimodal workload's feed-forward layer with its activation
        dict(name="linear_multimodal_ffn", op="linear", bt=8, l=1152, k=1024, n=4096, hin=0, hout=0, act="gelu_tanh",
             bias=True, gate=False, residual=False, type="float16"),
        # six modulation vectors from one embedding per batch entry: the weight is read once for four rows
        dict(name="linear_modulation", op="linear", bt=4, l=1, k=5120, n=30720, hin=0, hout=0, act="none",
             bias=True, gate=False, residual=False, type="bfloat16"),
        # an embedding of 77 text tokens with odd widths: the smallest matrix product
        dict(name="linear_text_odd", op="linear", bt=2, l=77, k=1000, n=1003, hin=0, hout=0, act="gelu_erf",
             bias=True, gate=False, residual=True, type="bfloat16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("rotary", "cross", "linear"))
    if op == "rotary":
        d = rng.choice((64, 128, 128, 40, 96, 120, 256))
        n = rng.randint(1, 4)
        rest, axes = d - rng.choice((0, 0, 2, 8)), []
        for a in range(n):
            x = rest if a == n - 1 else 2 * rng.randint(1, max(1, rest // 2 // (n - a)))
            axes.append(x)
            rest -= x
        bt, h = rng.randint(1, 8), rng.randint(1, 40)
        most = 16384 * 5120 // (bt * h * d)
        kind = rng.choice(("bfloat16", "bfloat16", "float16", "float32"))
        most = most // 2 if kind == "float32" else most
        return dict(op=op, bt=bt, h=h, l=_log(rng, 1, min(32768, most)), d=d, axes=",".join(map(str, axes)),
                    pairing=rng.choice(("adjacent", "halves")), inverse=rng.random() < 0.4,
                    layout=rng.choice(("rows", "heads")), batched=rng.random() < 0.5, type=kind)
    if op == "cross":
        d = rng.choice((64, 128))
        hkv = rng.choice((1, 2, 4, 8, 16, 40))
        h = hkv * rng.choice([r for r in (1, 1, 2, 4, 8) if hkv * r <= 40])
        bt = rng.randint(1, 8)
        lk = _log(rng, 1, min(16384, 16384 * 5120 // (bt * h * d)))
        most = min(int(2.9e11 / (4 * bt * h * lk * d)), 16384 * 5120 // (bt * h * d))
        return dict(op=op, bt=bt, h=h, hkv=hkv, lq=_log(rng, 1, max(1, min(16384, most))), lk=lk, d=d,
                    keys=rng.choice(("all", "count", "mask")), lse=rng.random() < 0.5,
                    layout=rng.choice(("rows", "heads")), type=rng.choice(("bfloat16", "float16")))
    bt = rng.randint(1, 8)
    hin = rng.choice((0, 0, 2, 12, 16, 40))
    hout = rng.choice((0, 0, 2, 12, 16, 40))
    k = hin * rng.choice((64, 128)) if hin else 8 * _log(rng, 2, 1280)
    n = hout * rng.choice((64, 128)) if hout else _log(rng, 9, 20480)
    k, n = (x + 8 if x == 24 * 128 else x for x in (k, n))
    most = min(int(8.5e11 / (2 * bt * k * n)), 16384 * 10240 // (bt * (k + n)))
    return dict(op=op, bt=bt, l=_log(rng, 1, max(1, min(16384, most))), k=k, n=n, hin=hin, hout=hout,
                act=rng.choice(("none", "gelu_tanh", "gelu_erf", "silu")), bias=rng.random() < 0.7,
                gate=rng.random() < 0.4, residual=rng.random() < 0.5, type=rng.choice(("bfloat16", "float16")))


# ------------------------------------------------------------------------------------- inputs
def _axes(case):
    return tuple(int(a) for a in case["axes"].split(","))


def _heads(gen, case, bt, h, l, d, kind):
    """[bt, h, l, d]: contiguous, or a view of a projection's [bt, l, h, d]."""
    if case["layout"] == "rows":
        return torch.randn(bt, l, h, d, generator=gen, device="cuda").to(kind).transpose(1, 2)
    return torch.randn(bt, h, l, d, generator=gen, device="cuda").to(kind)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    kind = TYPES[case["type"]]
    s = {"case": case, "op": case["op"]}
    if case["op"] == "rotary":
        axes = _axes(case)
        s["axes"] = axes
        s["x"] = _heads(gen, case, case["bt"], case["h"], case["l"], case["d"], kind)
        # raster order over frames of 32 x 32; with positions per entry, each has an offset and a step of its own
        i = torch.arange(case["l"], device="cuda")
        columns = {1: (i,), 2: (i // 32, i % 32), 3: (i // 1024, i // 32 % 32, i % 32),
                   4: (i, i // 1024, i // 32 % 32, i % 32)}[len(axes)]
        grid = torch.stack(columns, 1).float()
        if case["batched"]:
            step = 0.5 + torch.rand(case["bt"], 1, len(axes), generator=gen, device="cuda")
            start = torch.randint(0, 64, (case["bt"], 1, len(axes)), generator=gen, device="cuda").float()
            grid = start + step * grid
        s["pos"] = grid.contiguous()
    elif case["op"] == "cross":
        bt, lk = case["bt"], case["lk"]
        s["q"] = _heads(gen, case, bt, case["h"], case["lq"], case["d"], kind)
        s["k"] = _heads(gen, case, bt, case["hkv"], lk, case["d"], kind)
        s["v"] = _heads(gen, case, bt, case["hkv"], lk, case["d"], kind)
        s["key_len"] = s["key_mask"] = None
        if case["keys"] == "count":  # from none to all
            n = torch.randint(0, lk + 1, (bt,), generator=gen, device="cuda")
            n[0] = lk
            if bt > 2:
                n[bt // 2] = 0
            s["key_len"] = n.to(torch.int32)
        elif case["keys"] == "mask":  # a fifth of the keys dropped
            s["key_mask"] = (torch.rand(bt, lk, generator=gen, device="cuda") < 0.8).to(torch.uint8)
    else:
        bt, l, k, n = case["bt"], case["l"], case["k"], case["n"]
        if case["hin"]:
            s["x"] = torch.randn(bt, case["hin"], l, k // case["hin"], generator=gen, device="cuda").to(kind)
        else:
            s["x"] = torch.randn(bt, l, k, generator=gen, device="cuda").to(kind)
        s["w"] = (torch.randn(n, k, generator=gen, device="cuda") / math.sqrt(k)).to(kind)
        s["bias"] = torch.randn(n, generator=gen, device="cuda").to(kind) if case["bias"] else None
        s["gate"] = torch.randn(bt, n, generator=gen, device="cuda").to(kind) if case["gate"] else None
        shape = (bt, case["hout"], l, n // case["hout"]) if case["hout"] else (bt, l, n)
        s["residual"] = torch.randn(*shape, generator=gen, device="cuda").to(kind) if case["residual"] else None
    return s


def work(case):
    size = 4 if case["type"] == "float32" else 2
    if case["op"] == "rotary":
        n = case["bt"] * case["h"] * case["l"] * case["d"]
        pos = (case["bt"] if case["batched"] else 1) * case["l"] * len(_axes(case)) * 4
        return {"bytes": 2 * n * size + pos, "flops": 3 * n}
    if case["op"] == "cross":
        bt, lk, d = case["bt"], case["lk"], case["d"]
        real = bt * lk * 0.8 if case["keys"] == "mask" else bt * lk
        if case["keys"] == "count":  # one entry whole, from three on one empty, the others half on average
            real = lk + max(0, bt - (2 if bt > 2 else 1)) * lk / 2
        rows = bt * case["h"] * case["lq"]
        extra = {"all": 0, "count": 4 * bt, "mask": bt * lk}[case["keys"]]
        return {"bytes": 2 * rows * d * size + 2 * real * case["hkv"] * d * size + extra
                + (4 * rows if case["lse"] else 0), "flops": 4 * case["h"] * case["lq"] * real * d}
    m, k, n = case["bt"] * case["l"], case["k"], case["n"]
    extra = n * case["bias"] + case["bt"] * n * case["gate"] + m * n * case["residual"]
    return {"bytes": size * (m * k + n * k + m * n + extra), "flops": 2 * m * k * n}


# ------------------------------------------------------------------------------------- plain forms
def _pairs(axes, pairing, device):
    """Of every rotated pair: its first and second component, its axis, and its exponent 2 i / d_axis."""
    half = torch.tensor([a // 2 for a in axes], device=device)
    axis = torch.repeat_interleave(torch.arange(len(axes), device=device), half)
    begin = (torch.cumsum(half, 0) - half)[axis]
    i = torch.arange(axis.numel(), device=device) - begin
    if pairing == "adjacent":
        lo = 2 * begin + 2 * i
        hi = lo + 1
    else:
        lo = 2 * begin + i
        hi = lo + half[axis]
    return lo, hi, axis, i.double() / half[axis]


def plain_rotary(x, pos, axes, pairing, inverse, base=10000.0):
    lo, hi, axis, exponent = _pairs(axes, pairing, x.device)
    angle = pos.double()[..., axis] * torch.pow(base, -exponent)
    if pos.dim() == 3:
        angle = angle[:, None]
    c, s = torch.cos(angle).float(), torch.sin(angle).float()
    s = -s if inverse else s
    a, b = x[..., lo].float(), x[..., hi].float()
    y = x.float().contiguous()
    y = y.clone() if y.data_ptr() == x.data_ptr() else y
    y[..., lo] = a * c - b * s
    y[..., hi] = a * s + b * c
    return y.to(x.dtype)


def plain_cross(q, k, v, key_len, key_mask, want_lse):
    lk = k.shape[2]
    real = torch.ones(k.shape[0], lk, dtype=torch.bool, device=k.device)
    if key_len is not None:
        real = torch.arange(lk, device=k.device) < key_len[:, None]
    if key_mask is not None:
        real = key_mask != 0
    share = q.shape[1] // k.shape[1]
    real = real[:, None, :, None]
    kf = torch.where(real, k.float(), 0.0).repeat_interleave(share, 1)
    vf = torch.where(real, v.float(), 0.0).repeat_interleave(share, 1)
    scores = q.float() @ kf.transpose(2, 3) / math.sqrt(q.shape[3])
    scores = scores.masked_fill(~real.transpose(2, 3), -math.inf)
    top = scores.amax(3, keepdim=True)
    p = torch.exp(scores - torch.where(top == -math.inf, 0.0, top))
    total = p.sum(3, keepdim=True)
    o = (p @ vf / torch.where(total > 0, total, 1.0)).to(q.dtype)
    return (o, (top + torch.log(total))[..., 0]) if want_lse else o


def _act(z, act):
    if act == "gelu_tanh":
        return 0.5 * z * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z * z * z)))
    if act == "gelu_erf":
        return 0.5 * z * (1 + torch.erf(z / math.sqrt(2)))
    return z / (1 + torch.exp(-z)) if act == "silu" else z


def plain_linear(x, w, bias, act, gate, residual, heads):
    if x.dim() == 4:
        x = x.transpose(1, 2).flatten(2)
    y = x.float() @ w.float().t()
    y = _act(y + bias.float() if bias is not None else y, act)
    if gate is not None:
        y = y * gate.float()[:, None]
    if heads:
        y = y.unflatten(2, (heads, -1)).transpose(1, 2)
    if residual is not None:
        y = y + residual.float()
    return y.to(x.dtype).contiguous()


def run(s):
    case = s["case"]
    if own:
        from piecewise_attention_diffusion_b200 import bsattn as b
        if s["op"] == "rotary":
            pairing = b.PAIR_ADJACENT if case["pairing"] == "adjacent" else b.PAIR_HALVES
            return b.rotary(s["x"], s["pos"], s["axes"], pairing=pairing, inverse=case["inverse"])
        if s["op"] == "cross":
            o, lse = b.cross_forward(s["q"], s["k"], s["v"], key_len=s["key_len"], key_mask=s["key_mask"],
                                     want_lse=case["lse"])
            return (o, lse) if case["lse"] else o
        act = {"none": b.ACT_NONE, "gelu_tanh": b.ACT_GELU_TANH, "gelu_erf": b.ACT_GELU_ERF,
               "silu": b.ACT_SILU}[case["act"]]
        return b.linear(s["x"], s["w"], bias=s["bias"], act=act, gate=s["gate"], residual=s["residual"],
                        heads=case["hout"])
    if s["op"] == "rotary":
        return plain_rotary(s["x"], s["pos"], s["axes"], case["pairing"], case["inverse"])
    if s["op"] == "cross":
        return plain_cross(s["q"], s["k"], s["v"], s["key_len"], s["key_mask"], case["lse"])
    return plain_linear(s["x"], s["w"], s["bias"], case["act"], s["gate"], s["residual"], case["hout"])


# ------------------------------------------------------------------------------------- in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "rotary":
        # every axis turns its own section of d, as complex numbers
        x = s["x"].double().contiguous()
        y, begin = x.clone(), 0
        for a, da in enumerate(s["axes"]):
            part = x[..., begin:begin + da]
            p = s["pos"][..., a].double()
            rate = torch.tensor([10000.0 ** (-2 * i / da) for i in range(da // 2)], dtype=torch.float64, device="cuda")
            turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), p[..., None] * rate)
            turn = turn[:, None] if p.dim() == 2 else turn
            turn = turn.conj() if case["inverse"] else turn
            if case["pairing"] == "adjacent":
                z = torch.complex(part[..., 0::2], part[..., 1::2]) * turn
                y[..., begin:begin + da:2], y[..., begin + 1:begin + da:2] = z.real, z.imag
            else:
                z = torch.complex(part[..., :da // 2], part[..., da // 2:]) * turn
                y[..., begin:begin + da] = torch.cat((z.real, z.imag), -1)
            begin += da
        return y
    if case["op"] == "cross":
        q, k, v = s["q"], s["k"], s["v"]
        bt, h, lq, d = q.shape
        o = torch.zeros(bt, h, lq, d, dtype=torch.float64, device="cuda")
        lse = torch.full((bt, h, lq), -math.inf, dtype=torch.float64, device="cuda")
        for i in range(bt):
            keep = torch.arange(k.shape[2], device="cuda")
            if s["key_len"] is not None:
                keep = keep[:int(s["key_len"][i])]
            if s["key_mask"] is not None:
                keep = keep[s["key_mask"][i].bool()]
            if not keep.numel():
                continue
            for j in range(h):
                g = j * k.shape[1] // h
                z = torch.einsum("qd,kd->qk", q[i, j].double(), k[i, g, keep].double()) * d ** -0.5
                lse[i, j] = torch.logsumexp(z, 1)
                o[i, j] = torch.einsum("qk,kd->qd", torch.exp(z - lse[i, j, :, None]), v[i, g, keep].double())
        return (o, lse) if case["lse"] else o
    rows = []
    for i in range(case["bt"]):
        x = s["x"][i].double()
        x = torch.cat(list(x), -1) if x.dim() == 3 else x
        z = torch.einsum("lk,nk->ln", x, s["w"].double())
        if s["bias"] is not None:
            z += s["bias"].double()
        if case["act"] == "gelu_tanh":
            z = z * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))
        elif case["act"] == "gelu_erf":
            z = z * torch.special.ndtr(z)
        elif case["act"] == "silu":
            z = z * torch.sigmoid(z)
        if s["gate"] is not None:
            z = z * s["gate"][i].double()
        if case["hout"]:
            z = torch.stack(z.chunk(case["hout"], -1))
        if s["residual"] is not None:
            z = z + s["residual"][i].double()
        rows.append(z)
    return torch.stack(rows)
