"""Measured cases of the operators around the attention: rotary positions on several axes, the root-mean-square norm
with the residual's addition, 8-bit activation checkpoints and the attention's backward from them.

``own = False`` computes the plain forms with elementary torch operations; ``own = True`` makes the calls of
``block_sparse_attention_fwd_gb300``.
"""
import math

import torch

own = False

EPS = 1e-6
QMAX = {"int8": 127.0, "e4m3": 448.0}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # one new token of each of 32 sequences of a decoder, at far positions: latency
        dict(name="rope_token", op="rope", B=32, n=1, H=32, Hk=8, d=128, sections="64", layout="half",
             inverse=False, dtype="bf16", start=131071, Y=0, X=0),
        # q and k of a video block: 21 x 30 x 52 latent grid, 44 + 42 + 42 dimensions in pairs (2p, 2p + 1)
        dict(name="rope_video", op="rope", B=1, n=32760, H=40, Hk=40, d=128, sections="22,21,21",
             layout="interleaved", inverse=False, dtype="bf16", start=0, Y=30, X=52),
        # gradients of a decoder's q and k, grouped heads, half of the head dim rotated
        dict(name="rope_grads", op="rope", B=1, n=16384, H=32, Hk=8, d=128, sections="32", layout="half",
             inverse=True, dtype="bf16", start=4095, Y=0, X=0),
        # the block's entry norm for a handful of tokens: latency
        dict(name="norm_token", op="norm", rows=8, cols=4096, residual=True, out="same", group=0, dtype="bf16",
             wtype="bf16"),
        # the video block's entry norm, whose output feeds an 8-bit product
        dict(name="norm_video_e4m3", op="norm", rows=32760, cols=5120, residual=True, out="e4m3", group=128,
             dtype="bf16", wtype="fp32"),
        # q/k norm over single heads
        dict(name="norm_heads", op="norm", rows=8192 * 32, cols=128, residual=False, out="same", group=0,
             dtype="bf16", wtype="fp32"),
        # backward of a decoder's entry norm, the stream's own gradient added
        dict(name="norm_grads", op="norm_grads", rows=16384, cols=4096, saved="same", group=0, g_h=True,
             dtype="bf16", wtype="bf16"),
        # backward of the video block's entry norm from its 8-bit checkpoint
        dict(name="norm_grads_video_int8", op="norm_grads", rows=32760, cols=5120, saved="int8", group=128,
             g_h=True, dtype="bf16", wtype="fp32"),
        # checkpoint of the video block's q: one scale a token and head, saved and loaded
        dict(name="act_video", op="act", rows=32760 * 40, cols=128, fmt="int8", group=0, dtype="bf16"),
        # an activation of odd width, whose rows start anywhere
        dict(name="act_odd", op="act", rows=8190, cols=1001, fmt="e4m3", group=32, dtype="fp16"),
        # attention backward from 8-bit q, k, v and o at a small training shape
        dict(name="attn_grads_int8", op="attn_grads", B=2, n=4096, H=12, Hk=12, d=64, causal=False, fmt="int8",
             o8=True),
        # short causal sequence with grouped heads; o kept in bf16
        dict(name="attn_grads_causal", op="attn_grads", B=1, n=1000, H=8, Hk=2, d=128, causal=True, fmt="e4m3",
             o8=False),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["rope", "norm", "norm_grads", "act", "attn_grads"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op == "rope":
        Hk = rng.randint(1, 8)
        H = Hk * rng.randint(1, 5)
        d = rng.choice([64, 128, 80, 96])
        n = _log(rng, 1, min(40000, 150000000 // ((H + Hk) * d)))
        B = rng.randint(1, max(1, min(64, 40000 // n, 150000000 // (n * (H + Hk) * d))))
        layout = rng.choice(["half", "interleaved"])
        Y = X = 0
        if rng.random() < 0.5:
            a, b = rng.randint(1, d // 6), rng.randint(1, d // 6)
            sections = "%d,%d,%d" % (d // 2 - a - b, a, b)
            Y, X = rng.randint(2, 40), rng.randint(2, 60)
        else:
            sections = str(rng.choice([d // 2, d // 4]))
        return dict(op=op, B=B, n=n, H=H, Hk=Hk, d=d, sections=sections, layout=layout,
                    inverse=rng.random() < 0.5, dtype=dtype, start=_log(rng, 1, 1000000), Y=Y, X=X)
    if op == "attn_grads":
        Hk = rng.randint(1, 4)
        return dict(op=op, B=rng.randint(1, 2), n=_log(rng, 1, 3000), H=Hk * rng.randint(1, 3), Hk=Hk,
                    d=rng.choice([64, 128]), causal=rng.random() < 0.5, fmt=rng.choice(["int8", "e4m3"]),
                    o8=rng.random() < 0.5)
    cols = _log(rng, 16, 8192)
    if rng.random() < 0.7:
        cols = -(-cols // 8) * 8
    rows = _log(rng, 1, max(1, min(200000, 100000000 // cols)))
    group = rng.choice([0, 32, 64, 128])
    fmt = rng.choice(["int8", "e4m3"])
    if op == "act":
        return dict(op=op, rows=rows, cols=cols, fmt=fmt, group=group, dtype=rng.choice(["bf16", "fp16"]))
    if op == "norm":
        out = rng.choice(["same", "8"])
        if out == "8":
            out, dtype = fmt, rng.choice(["bf16", "fp16"])
        return dict(op=op, rows=rows, cols=cols, residual=rng.random() < 0.7, out=out, group=group, dtype=dtype,
                    wtype=rng.choice([dtype, "fp32"]))
    return dict(op=op, rows=rows, cols=cols, saved=rng.choice(["same", fmt]), group=group, g_h=rng.random() < 0.7,
                dtype=dtype, wtype=rng.choice([dtype, "fp32"]))


# --- inputs ------------------------------------------------------------------

def _freqs(case):
    """Frequencies of the pairs: section s of m pairs has 10000^(-j / m), j = 0 .. m - 1."""
    out = []
    for m in (int(x) for x in case["sections"].split(",")):
        out += [10000.0 ** (-j / m) for j in range(m)]
    return out


def _positions(case):
    """int32 [B, n, axes]: a grid's (t, y, x) for three sections, else each sequence's own run of positions."""
    B, n = case["B"], case["n"]
    i = torch.arange(n, device="cuda")
    if case["Y"]:
        Y, X = case["Y"], case["X"]
        p = torch.stack([i // (Y * X), i // X % Y, i % X], -1)[None].expand(B, n, 3)
    else:
        p = (i[None, :] + case["start"] - 37 * torch.arange(B, device="cuda")[:, None])[..., None]
    return p.to(torch.int32).contiguous()


def _quantise(x, fmt, group):
    """fp32 [rows, cols] -> (codes as fp32 [rows, groups, size], scales [rows, groups])."""
    rows, cols = x.shape
    size = group or cols
    groups = -(-cols // size)
    x = torch.nn.functional.pad(x, (0, groups * size - cols)).view(rows, groups, size)
    scales = torch.clamp(x.abs().amax(-1) / QMAX[fmt], min=2.0 ** -126)
    c = x * (1.0 / scales)[..., None]
    c = c.round().clamp(-127, 127) if fmt == "int8" else c.to(torch.float8_e4m3fn).float()
    return c, scales


def _codes(c, fmt, cols):
    c = c.flatten(1)[:, :cols]
    return c.to(torch.int8 if fmt == "int8" else torch.float8_e4m3fn).contiguous()


def _expand(codes, scales, group):
    """8-bit codes [rows, cols] and their scales -> fp32 values."""
    cols = codes.shape[1]
    return codes.float() * scales.repeat_interleave(group or cols, 1)[:, :cols]


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    s = dict(case=case, op=op)
    if op == "rope":
        t = TYPES[case["dtype"]]
        B, n, d = case["B"], case["n"], case["d"]
        s["q"] = normal(B, n, case["H"], d, dtype=t)
        s["k"] = normal(B, n, case["Hk"], d, dtype=t)
        s["positions"] = _positions(case)
        s["freqs"] = torch.tensor(_freqs(case), dtype=torch.float64, device="cuda")
        sections = [int(x) for x in case["sections"].split(",")]
        s["axis"] = torch.repeat_interleave(torch.arange(len(sections)), torch.tensor(sections)).cuda()
        if own:
            import block_sparse_attention_fwd_gb300 as bl
            s["plan"] = bl.RopePlan(d, sections, theta=10000.0, layout=case["layout"], device="cuda")
        return s
    if op == "attn_grads":
        B, n, H, Hk, d = (case[x] for x in ("B", "n", "H", "Hk", "d"))
        q, k, v = (normal(B, n, h, d, dtype=torch.bfloat16) for h in (H, Hk, Hk))
        s["g_o"] = normal(B, n, H, d, dtype=torch.bfloat16)
        x = (q.float().transpose(1, 2) @ _heads(k, H).transpose(2, 3)) * d ** -0.5
        if case["causal"]:
            x.masked_fill_(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), -math.inf)
        s["lse"] = torch.logsumexp(x, -1)
        o = (torch.exp(x.sub_(s["lse"][..., None])) @ _heads(v, H)).transpose(1, 2).to(torch.bfloat16).contiguous()
        s["o"] = o
        for name, t in (("q", q), ("k", k), ("v", v)) + ((("o", o),) if case["o8"] else ()):
            c, sc = _quantise(t.float().reshape(-1, d), case["fmt"], 0)
            s[name + "8"] = _codes(c, case["fmt"], d).view(t.shape)
            s[name + "s"] = sc.view(t.shape[:-1])
        return s
    rows, cols = case["rows"], case["cols"]
    t = TYPES[case["dtype"]]
    # the residual stream's columns differ in size: a few carry most of it
    size = torch.exp(0.7 * normal(cols))
    s["x"] = (normal(rows, cols) * size).to(t)
    if op == "act":
        return s
    s["w"] = (1 + 0.2 * normal(cols)).to(TYPES[case["wtype"]])
    if op == "norm":
        s["r"] = (3 * normal(rows, cols) * size).to(t) if case["residual"] else None
        return s
    h = s["x"]
    s["rstd"] = 1 / torch.sqrt((h.float() * h.float()).mean(-1) + EPS)
    s["g_y"] = normal(rows, cols, dtype=t)
    s["g_h"] = normal(rows, cols, dtype=t) if case["g_h"] else None
    if case["saved"] != "same":
        c, s["scales"] = _quantise(h.float(), case["saved"], case["group"])
        s["codes"] = _codes(c, case["saved"], cols)
        del s["x"]
    return s


def _heads(k, H):
    """[B, n, Hk, d] -> fp32 [B, H, n, d], each head repeated for its group."""
    return k.float().transpose(1, 2).repeat_interleave(H // k.shape[2], 1)


# --- one pass ----------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import block_sparse_attention_fwd_gb300 as bl
    case, op = s["case"], s["op"]
    if op == "rope":
        return bl.rope(s["q"], s["k"], s["positions"], s["plan"], inverse=case["inverse"])
    if op == "norm":
        if case["out"] == "same":
            y, h, rstd = bl.rms_norm_fwd(s["x"], s["w"], EPS, residual=s["r"])
            return (y, h, rstd) if case["residual"] else (y, rstd)
        y8, h, rstd = bl.rms_norm_fwd_8bit(s["x"], s["w"], EPS, residual=s["r"], fmt=case["out"],
                                           group=case["group"])
        y = bl.act_load(y8)
        return (y, y8.scales, h, rstd) if case["residual"] else (y, y8.scales, rstd)
    if op == "norm_grads":
        h = s["x"] if case["saved"] == "same" else bl.Act8(s["codes"], s["scales"], case["group"],
                                                           TYPES[case["dtype"]])
        return bl.rms_norm_bwd(s["g_y"], h, s["rstd"], s["w"], g_h=s["g_h"])
    if op == "act":
        a = bl.act_save(s["x"], fmt=case["fmt"], group=case["group"])
        return bl.act_load(a), a.scales
    B, n, H, Hk, d = (case[x] for x in ("B", "n", "H", "Hk", "d"))
    shape = bl.make_shape(B, n, H, Hk, d, 128, 128, int(case["causal"]))
    q, k, v = (bl.Act8(s[x + "8"], s[x + "s"], 0, torch.bfloat16) for x in "qkv")
    o = bl.Act8(s["o8"], s["os"], 0, torch.bfloat16) if case["o8"] else s["o"]
    return bl.attn_bwd_act8(shape, q, k, v, o, s["g_o"], s["lse"], d ** -0.5)


def _plain(s):
    case, op = s["case"], s["op"]
    if op == "rope":
        angle = s["positions"].double()[..., s["axis"]] * s["freqs"]
        c, sn = torch.cos(angle).float()[:, :, None], torch.sin(angle).float()[:, :, None]
        if case["inverse"]:
            sn = -sn
        return _rotate(s["q"], c, sn, case["layout"]), _rotate(s["k"], c, sn, case["layout"])
    if op == "norm":
        t = TYPES[case["dtype"]]
        h = s["x"].float()
        if case["residual"]:
            h = h + s["r"].float()
        rstd = 1 / torch.sqrt((h * h).mean(-1) + EPS)
        y = h * rstd[:, None] * s["w"].float()
        if case["out"] == "same":
            y = y.to(t)
            return (y, h.to(t), rstd) if case["residual"] else (y, rstd)
        c, scales = _quantise(y, case["out"], case["group"])
        y = (c * scales[..., None]).flatten(1)[:, :case["cols"]].to(t)
        return (y, scales, h.to(t), rstd) if case["residual"] else (y, scales, rstd)
    if op == "norm_grads":
        h = s["x"].float() if case["saved"] == "same" else _expand(s["codes"], s["scales"], case["group"])
        unit = h * s["rstd"][:, None]
        g_y = s["g_y"].float()
        wg = g_y * s["w"].float()
        g_x = s["rstd"][:, None] * (wg - unit * (wg * unit).mean(-1, keepdim=True))
        if case["g_h"]:
            g_x = g_x + s["g_h"].float()
        return g_x.to(s["g_y"].dtype), (g_y * unit).sum(0).to(s["w"].dtype)
    if op == "act":
        c, scales = _quantise(s["x"].float(), case["fmt"], case["group"])
        return (c * scales[..., None]).flatten(1)[:, :case["cols"]].to(s["x"].dtype), scales
    n, H, Hk, d = (case[x] for x in ("n", "H", "Hk", "d"))
    # a checkpoint stands for values of the type that was saved
    q, k, v = ((s[x + "8"].float() * s[x + "s"][..., None]).to(torch.bfloat16) for x in "qkv")
    o = s["o8"].float() * s["os"][..., None] if case["o8"] else s["o"].float()
    g_o = s["g_o"].float()
    q, g_o, o = (x.float().transpose(1, 2) for x in (q, g_o, o))
    k, v = _heads(k, H), _heads(v, H)
    p = torch.exp((q @ k.transpose(2, 3)) * d ** -0.5 - s["lse"][..., None])
    if case["causal"]:
        p = p * torch.ones(n, n, device="cuda").tril()
    D = (g_o * o).sum(-1, keepdim=True)
    g_s = p * (g_o @ v.transpose(2, 3) - D) * d ** -0.5
    g_q, g_k, g_v = g_s @ k, g_s.transpose(2, 3) @ q, p.transpose(2, 3) @ g_o
    group = (lambda x: x.unflatten(1, (Hk, H // Hk)).sum(2))
    return tuple(x.transpose(1, 2).to(torch.bfloat16).contiguous() for x in (g_q, group(g_k), group(g_v)))


def _rotate(x, c, s, layout):
    P = c.shape[-1]
    out = x.float()
    a, b = (out[..., 0:2 * P:2], out[..., 1:2 * P:2]) if layout == "interleaved" else (out[..., :P], out[..., P:2 * P])
    u, v = a * c - b * s, a * s + b * c
    turned = torch.stack((u, v), -1).flatten(-2) if layout == "interleaved" else torch.cat((u, v), -1)
    return torch.cat((turned, out[..., 2 * P:]), -1).to(x.dtype)


# --- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    if op == "rope":
        x = case["B"] * case["n"] * (case["H"] + case["Hk"]) * case["d"]
        turned = 2 * sum(int(m) for m in case["sections"].split(",")) / case["d"]
        return dict(bytes=2 * x * size[case["dtype"]] + case["B"] * case["n"] * 12, flops=3 * x * turned)
    if op == "attn_grads":
        B, n, H, Hk, d = (case[x] for x in ("B", "n", "H", "Hk", "d"))
        pairs = n * (n + 1) // 2 if case["causal"] else n * n
        heads = B * n * (H + 2 * Hk)
        o = B * n * H * (d + 4 if case["o8"] else 2 * d)
        return dict(bytes=heads * (d + 4) + o + 2 * B * n * H * d + 4 * B * n * H + 2 * heads * d,
                    flops=10.0 * B * H * pairs * d)
    rows, cols = case["rows"], case["cols"]
    t, x = size[case["dtype"]], rows * cols
    groups = rows * (-(-cols // case["group"]) if case["group"] else 1)
    if op == "act":  # read, codes written and read, written; scales written and read
        return dict(bytes=x * (2 * t + 2) + 8 * groups, flops=4 * x)
    w = cols * size[case["wtype"]]
    if op == "norm":
        moved = (4 if case["residual"] else 2) * t
        if case["out"] == "same":
            return dict(bytes=x * moved + w + 4 * rows, flops=5 * x)
        return dict(bytes=x * (moved + 2) + 8 * groups + w + 4 * rows, flops=9 * x)
    moved = 2 * t + (t if case["g_h"] else 0) + (t if case["saved"] == "same" else 1)
    return dict(bytes=x * moved + (0 if case["saved"] == "same" else 4 * groups) + 2 * w + 4 * rows, flops=10 * x)


# --- in 64 bits --------------------------------------------------------------

def _round8(y, fmt):
    """To the nearest code, ties to even, of values within the format's range."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.frexp(y)[1].clamp(min=-5) - 4     # 3 bits behind the leading one; subnormals below 2^-6
    step = torch.ldexp(torch.ones_like(y), e)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _through8(x, fmt, group):
    """What remains of fp64 [rows, cols] after 8 bits, and the scales; a block of rows at a time."""
    size = group or x.shape[1]
    values, scales = torch.empty_like(x), []
    for j in range(0, x.shape[1], size):
        part = x[:, j:j + size]
        sc = (part.abs().max(1, keepdim=True).values / QMAX[fmt]).clamp(min=2.0 ** -126)
        values[:, j:j + size] = _round8(part / sc, fmt) * sc
        scales.append(sc)
    return values, torch.cat(scales, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "rope":
        P = s["freqs"].numel()
        angle = torch.stack([s["positions"][..., int(a)].double() * f for a, f in zip(s["axis"].tolist(), s["freqs"])], -1)
        turn = torch.polar(torch.ones_like(angle), -angle if case["inverse"] else angle)[:, :, None, :]
        out = []
        for x in (s["q"].double(), s["k"].double()):
            if case["layout"] == "interleaved":
                z = torch.complex(x[..., 0:2 * P:2], x[..., 1:2 * P:2]) * turn
                x[..., 0:2 * P:2], x[..., 1:2 * P:2] = z.real, z.imag
            else:
                z = torch.complex(x[..., :P], x[..., P:2 * P]) * turn
                x[..., :P], x[..., P:2 * P] = z.real, z.imag
            out.append(x)
        return tuple(out)
    if op == "act":
        return _through8(s["x"].double(), case["fmt"], case["group"])
    if op == "norm":
        h = s["x"].double() + (s["r"].double() if case["residual"] else 0)
        norm = torch.sqrt(torch.einsum("rc,rc->r", h, h) / case["cols"] + EPS)
        y = h / norm[:, None] * s["w"].double()
        got = (y,) if case["out"] == "same" else _through8(y, case["out"], case["group"])
        return (*got, h, 1 / norm) if case["residual"] else (*got, 1 / norm)
    if op == "norm_grads":
        if case["saved"] == "same":
            h = s["x"].double()
        else:
            h = s["codes"].to(torch.float64)
            size = case["group"] or case["cols"]
            for j in range(s["scales"].shape[1]):
                h[:, j * size:(j + 1) * size] *= s["scales"][:, j:j + 1].double()
        rstd, w, g_y = s["rstd"].double(), s["w"].double(), s["g_y"].double()
        # y_c = w_c h_c rstd, and rstd's own derivative: d rstd / d h_c = -rstd^3 h_c / cols
        along = torch.einsum("rc,rc,c->r", g_y, h, w) * rstd ** 3 / case["cols"]
        g_x = torch.addcmul(g_y * w * rstd[:, None], h, along[:, None], value=-1)
        if case["g_h"]:
            g_x += s["g_h"].double()
        return g_x, torch.einsum("rc,rc,r->c", g_y, h, rstd)
    B, H, Hk, d, n = (case[x] for x in ("B", "H", "Hk", "d", "n"))
    scale = 1 / math.sqrt(d)
    q, k, v = ((s[x + "8"].float() * s[x + "s"][..., None]).to(torch.bfloat16).double() for x in "qkv")
    o = s["o8"].double() * s["os"].double()[..., None] if case["o8"] else s["o"].double()
    g_o, lse = s["g_o"].double(), s["lse"].double()
    g_q, g_k, g_v = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    later = torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1) if case["causal"] else None
    for b in range(B):
        for h in range(H):
            j = h // (H // Hk)
            p = torch.exp(torch.einsum("id,jd->ij", q[b, :, h], k[b, :, j]) * scale - lse[b, h][:, None])
            if case["causal"]:
                p[later] = 0
            g_v[b, :, j] += torch.einsum("ij,id->jd", p, g_o[b, :, h])
            p *= torch.einsum("id,jd->ij", g_o[b, :, h], v[b, :, j]) - torch.einsum("id,id->i", g_o[b, :, h], o[b, :, h])[:, None]
            g_q[b, :, h] = scale * torch.einsum("ij,jd->id", p, k[b, :, j])
            g_k[b, :, j] += scale * torch.einsum("ij,id->jd", p, q[b, :, h])
    return g_q, g_k, g_v
