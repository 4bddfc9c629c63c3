"""Measured cases of the linear layers around the attention: products of 8-bit codes with a scale for each block of 128
and the gradients of such a layer, the layer norm and its backward, and dropout whose mask is never stored.

``own = False`` computes the plain forms with elementary torch operations; ``own = True`` makes the calls of
``block_sparse_attention_fwd_gb300``.
"""
import math

import torch

own = False

EPS = 1e-5
# the format: scale = amax * fl32(1 / largest code), code = x * fl32(1 / scale) to the nearest
STEP = {"int8": 1 / 127.0, "e4m3": 1 / 448.0}
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --- cases -------------------------------------------------------------------

def listed():
    return [
        # the output projection for one new token of each of 8 sequences: the weight's bytes
        dict(name="product_token", op="product", form="y", M=8, N=5120, K=5120, dtype="bf16"),
        # q, k and v of a video block in one product: 32760 tokens, 3 x 40 heads of 128
        dict(name="product_video", op="product", form="y", M=32760, N=15360, K=5120, dtype="bf16"),
        # gradient of a decoder's input: 32 + 2 x 8 heads of 128
        dict(name="product_g_x", op="product", form="g_x", M=16384, N=6144, K=4096, dtype="bf16"),
        # gradient of a weight of odd sizes from an odd number of tokens
        dict(name="product_g_w_odd", op="product", form="g_w", M=4095, N=2050, K=1001, dtype="fp32"),
        # a whole step of a decoder's linear layer from bf16: the product and both gradients
        dict(name="linear_step", op="linear", M=16384, N=4096, K=4096, dtype="bf16"),
        # the block's entry norm for a handful of tokens: latency
        dict(name="ln_token", op="norm", rows=8, cols=4096, residual=True, out="same", group=0, dtype="bf16",
             wtype="bf16"),
        # the video block's entry norm, whose output feeds an 8-bit product
        dict(name="ln_video_e4m3", op="norm", rows=32760, cols=5120, residual=True, out="e4m3", group=128,
             dtype="bf16", wtype="fp32"),
        # its backward, the stream's own gradient added
        dict(name="ln_grads_video", op="norm_grads", rows=32760, cols=5120, g_h=True, dtype="bf16", wtype="fp32"),
        # rows of odd width
        dict(name="ln_grads_odd", op="norm_grads", rows=8190, cols=1001, g_h=False, dtype="fp16", wtype="fp16"),
        # dropout of the attention's output in front of the residual's addition, video block
        dict(name="drop_video", op="dropout", rows=32760, cols=5120, residual=True, p=0.1, dtype="bf16"),
        # its gradient in a decoder
        dict(name="drop_grads", op="dropout", rows=16384, cols=4096, residual=False, p=0.05, dtype="bf16"),
        # a short sequence of odd width: latency
        dict(name="drop_short", op="dropout", rows=13, cols=1001, residual=True, p=0.25, dtype="fp16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, round(math.exp(rng.uniform(math.log(lo), math.log(hi))))))


def draw(rng):
    op = rng.choice(["product", "product", "linear", "norm", "norm_grads", "dropout"])
    dtype = rng.choice(["bf16", "bf16", "fp16", "fp32"])
    if op in ("product", "linear"):
        N, K = _log(rng, 16, 16384), _log(rng, 16, 16384)
        if rng.random() < 0.7:
            N, K = -(-N // 16) * 16, -(-K // 16) * 16
        most = 2.0e12 if op == "product" else 2.5e11
        M = _log(rng, 1, max(1, min(40000, int(most / (N * K)), 400000000 // max(N, K))))
        case = dict(op=op, M=M, N=N, K=K, dtype=dtype)
        if op == "product":
            case["form"] = rng.choice(["y", "y", "g_x", "g_w"])
        return case
    cols = _log(rng, 16, 16384)
    if rng.random() < 0.7:
        cols = -(-cols // 8) * 8
    rows = _log(rng, 1, max(1, min(200000, 100000000 // cols)))
    if op == "dropout":
        return dict(op=op, rows=rows, cols=cols, residual=rng.random() < 0.5, p=rng.choice([0.05, 0.1, 0.25, 0.5]),
                    dtype=dtype)
    if op == "norm":
        out, group = rng.choice(["same", "e4m3", "int8"]), rng.choice([0, 32, 64, 128])
        if out != "same":
            dtype = rng.choice(["bf16", "fp16"])
        return dict(op=op, rows=rows, cols=cols, residual=rng.random() < 0.7, out=out, group=group, dtype=dtype,
                    wtype=rng.choice([dtype, "fp32"]))
    return dict(op=op, rows=rows, cols=cols, g_h=rng.random() < 0.7, dtype=dtype, wtype=rng.choice([dtype, "fp32"]))


# --- inputs ------------------------------------------------------------------

def _groups8(x, group, fmt="e4m3"):
    """fp32 [rows, cols] -> codes [rows, cols] in 8 bits and scales [rows, groups], one for every `group` elements."""
    rows, cols = x.shape
    size = group or cols
    groups = -(-cols // size)
    x = torch.nn.functional.pad(x, (0, groups * size - cols)).view(rows, groups, size)
    scales = torch.clamp(x.abs().amax(-1) * STEP[fmt], min=2.0 ** -126)
    c = (x * (1.0 / scales)[..., None]).flatten(1)[:, :cols]
    c = c.round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else c.to(torch.float8_e4m3fn)
    return c.contiguous(), scales


def _cols8(x):
    """The same in groups of 128 elements of a column: codes [rows, cols], scales [groups, cols]."""
    c, scales = _groups8(x.t(), 128)
    return c.t().contiguous(), scales.t().contiguous()


def _blocks8(w):
    """The same with one scale for every 128 x 128 elements."""
    rows, cols = w.shape
    R, C = -(-rows // 128), -(-cols // 128)
    x = torch.nn.functional.pad(w, (0, C * 128 - cols, 0, R * 128 - rows)).view(R, 128, C, 128)
    scales = torch.clamp(x.abs().amax((1, 3)) * STEP["e4m3"], min=2.0 ** -126)
    c = (x * (1.0 / scales)[:, None, :, None]).reshape(R * 128, C * 128)[:rows, :cols]
    return c.to(torch.float8_e4m3fn).contiguous(), scales


def prepare(case, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    op = case["op"]

    def normal(*shape, dtype=torch.float32):
        return torch.randn(shape, generator=g, device="cuda").to(dtype)

    t = TYPES[case["dtype"]]
    s = dict(case=case, op=op)
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        # an activation's columns differ in size: a few carry most of it
        x = normal(M, K) * torch.exp(0.7 * normal(K))
        w = normal(N, K) * K ** -0.5
        g_y = 0.01 * normal(M, N) * torch.exp(normal(M, 1))
        if op == "linear":
            s["x"], s["w"], s["g_y"] = x.to(t), w.to(t), g_y.to(t)
            return s
        form = case["form"]
        if form == "g_w":
            a, b = _cols8(g_y), _cols8(x)
        else:
            a, b = _groups8(x if form == "y" else g_y, 128), _blocks8(w)
        s["a"], s["b"] = a, b
        if own:
            import block_sparse_attention_fwd_gb300 as bl
            s["a8"] = bl.Cols8(*a, t) if form == "g_w" else bl.Act8(*a, 128, t)
            s["b8"] = bl.Cols8(*b, t) if form == "g_w" else bl.Weight8(*b, t)
        return s
    rows, cols = case["rows"], case["cols"]
    if op == "dropout":
        s["x"] = normal(rows, cols, dtype=t)
        s["r"] = 3 * normal(rows, cols, dtype=t) if case["residual"] else None
        s["state"] = torch.tensor([0x5DEECE66D1234567 ^ seed % 2 ** 48, (seed % 2 ** 30 << 32) + 41], dtype=torch.int64,
                                  device="cuda")
        return s
    size = torch.exp(0.7 * normal(cols))
    s["x"] = (0.3 + normal(rows, cols) * size).to(t)
    s["w"] = (1 + 0.2 * normal(cols)).to(TYPES[case["wtype"]])
    if op == "norm":
        s["bias"] = (0.1 * normal(cols)).to(TYPES[case["wtype"]])
        s["r"] = (3 * normal(rows, cols) * size).to(t) if case["residual"] else None
        return s
    h = s["x"].float()
    s["mean"] = h.mean(-1)
    h = h - s["mean"][:, None]
    s["rstd"] = 1 / torch.sqrt((h * h).mean(-1) + EPS)
    s["g_y"] = normal(rows, cols, dtype=t)
    s["g_h"] = normal(rows, cols, dtype=t) if case["g_h"] else None
    return s


# --- one pass ----------------------------------------------------------------

def run(s):
    return _own(s) if own else _plain(s)


def _own(s):
    import block_sparse_attention_fwd_gb300 as bl
    case, op = s["case"], s["op"]
    if op == "product":
        return {"y": bl.matmul8, "g_x": bl.matmul8_gx, "g_w": bl.matmul8_gw}[case["form"]](s["a8"], s["b8"])
    if op == "linear":
        w8 = bl.weight_save(s["w"])
        x8, x8_cols = bl.act_save_both(s["x"])
        y = bl.matmul8(x8, w8)
        g8, g8_cols = bl.act_save_both(s["g_y"])
        return y, bl.matmul8_gx(g8, w8), bl.matmul8_gw(g8_cols, x8_cols)
    if op == "norm":
        if case["out"] == "same":
            y, h, mean, rstd = bl.layer_norm_fwd(s["x"], s["w"], s["bias"], EPS, residual=s["r"])
            return (y, h, mean, rstd) if case["residual"] else (y, mean, rstd)
        y8, h, mean, rstd = bl.layer_norm_fwd_8bit(s["x"], s["w"], s["bias"], EPS, residual=s["r"], fmt=case["out"],
                                                   group=case["group"])
        y = bl.act_load(y8)
        return (y, y8.scales, h, mean, rstd) if case["residual"] else (y, y8.scales, mean, rstd)
    if op == "norm_grads":
        return bl.layer_norm_bwd(s["g_y"], s["x"], s["mean"], s["rstd"], s["w"], g_h=s["g_h"])
    return bl.dropout(s["x"], case["p"], s["state"], residual=s["r"])


def _plain(s):
    case, op = s["case"], s["op"]
    t = TYPES[case["dtype"]]
    if op == "product":
        if case["form"] == "g_w":
            return (_from_cols(*s["a"]).t() @ _from_cols(*s["b"])).to(t)
        a, w = _from_groups(*s["a"], 128), _from_blocks(*s["b"])
        return (a @ (w.t() if case["form"] == "y" else w)).to(t)
    if op == "linear":
        x, w, g = s["x"].float(), s["w"].float(), s["g_y"].float()
        w = _from_blocks(*_blocks8(w))
        y = _from_groups(*_groups8(x, 128), 128) @ w.t()
        g_x = _from_groups(*_groups8(g, 128), 128) @ w
        g_w = _from_cols(*_cols8(g)).t() @ _from_cols(*_cols8(x))
        return y.to(t), g_x.to(t), g_w.to(t)
    if op == "norm":
        h = s["x"].float()
        if case["residual"]:
            h = h + s["r"].float()
        mean = h.mean(-1)
        centred = h - mean[:, None]
        rstd = 1 / torch.sqrt((centred * centred).mean(-1) + EPS)
        y = centred * rstd[:, None] * s["w"].float() + s["bias"].float()
        if case["out"] == "same":
            y = y.to(t)
            return (y, h.to(t), mean, rstd) if case["residual"] else (y, mean, rstd)
        c, scales = _groups8(y, case["group"], case["out"])
        y = _from_groups(c, scales, case["group"]).to(t)
        return (y, scales, h.to(t), mean, rstd) if case["residual"] else (y, scales, mean, rstd)
    if op == "norm_grads":
        unit = (s["x"].float() - s["mean"][:, None]) * s["rstd"][:, None]
        g_y = s["g_y"].float()
        wg = g_y * s["w"].float()
        g_x = s["rstd"][:, None] * (wg - wg.mean(-1, keepdim=True) - unit * (wg * unit).mean(-1, keepdim=True))
        if case["g_h"]:
            g_x = g_x + s["g_h"].float()
        return g_x.to(t), (g_y * unit).sum(0).to(s["w"].dtype), g_y.sum(0).to(s["w"].dtype)
    x = s["x"].float()
    kept = _words(s["state"], x.numel()) >= round(case["p"] * 2 ** 32)
    y = torch.where(kept.view(x.shape), x * (1 / (1 - case["p"])), 0.0)
    if case["residual"]:
        y = y + s["r"].float()
    return y.to(t)


def _from_groups(c, scales, group):
    cols = c.shape[1]
    return c.float() * scales.repeat_interleave(group or cols, 1)[:, :cols]


def _from_cols(c, scales):
    return c.float() * scales.repeat_interleave(128, 0)[:c.shape[0]]


def _from_blocks(c, scales):
    return c.float() * scales.repeat_interleave(128, 0)[:c.shape[0]].repeat_interleave(128, 1)[:, :c.shape[1]]


def _words(state, n):
    """The first n words of Philox4x32-10 (Salmon, Moraes, Dror and Shaw, SC 2011), as int64: words 4 j .. 4 j + 3 from
    the counter (j, offset) of 2 x 64 bits and the key `seed`; state is (seed, offset)."""
    low = 0xFFFFFFFF
    j = torch.arange(-(-n // 4), device=state.device)
    seed, offset = state[0], state[1]
    k0, k1 = seed & low, (seed >> 32) & low
    c = [j & low, j >> 32, (offset & low).expand_as(j), ((offset >> 32) & low).expand_as(j)]

    def high(m, x):                        # the upper 32 of the 64 bits of a product of 32-bit words
        return ((m >> 16) * x + ((m & 0xFFFF) * x >> 16)) >> 16

    for _ in range(10):
        a, b = c[0], c[2]
        c = [high(0xCD9E8D57, b) ^ c[1] ^ k0, (0xCD9E8D57 * b) & low,
             high(0xD2511F53, a) ^ c[3] ^ k1, (0xD2511F53 * a) & low]
        k0, k1 = (k0 + 0x9E3779B9) & low, (k1 + 0xBB67AE85) & low
    return torch.stack(c, -1).flatten()[:n]


# --- what a pass cannot do without -------------------------------------------

def work(case):
    op = case["op"]
    size = {"bf16": 2, "fp16": 2, "fp32": 4}
    t = size[case["dtype"]]
    if op in ("product", "linear"):
        M, N, K = case["M"], case["N"], case["K"]
        if op == "linear":                 # x, w and g_y in; y, g_x and g_w out
            return dict(bytes=2 * t * (M * K + N * K + M * N), flops=6.0 * M * N * K)
        if case["form"] == "g_w":
            moved = M * N + M * K + 4 * -(-M // 128) * (N + K) + t * N * K
        else:
            inner, outer = (K, N) if case["form"] == "y" else (N, K)
            moved = M * inner + N * K + 4 * -(-inner // 128) * (M + -(-outer // 128)) + t * M * outer
        return dict(bytes=moved, flops=2.0 * M * N * K)
    rows, cols = case["rows"], case["cols"]
    x = rows * cols
    if op == "dropout":
        return dict(bytes=x * t * (3 if case["residual"] else 2), flops=3 * x)
    w = 2 * cols * size[case["wtype"]]
    if op == "norm":
        moved = (4 if case["residual"] else 2) * t
        if case["out"] == "same":
            return dict(bytes=x * moved + w + 8 * rows, flops=8 * x)
        groups = rows * (-(-cols // case["group"]) if case["group"] else 1)
        return dict(bytes=x * (moved + 2) + 8 * groups + w + 8 * rows, flops=12 * x)
    return dict(bytes=x * (4 if case["g_h"] else 3) * t + 3 * w // 2 + 8 * rows, flops=14 * x)


# --- in 64 bits --------------------------------------------------------------

def _round8(y, fmt):
    """To the nearest code, ties to even, of values within the format's range."""
    if fmt == "int8":
        return torch.round(y).clamp(-127, 127)
    e = torch.frexp(y)[1].clamp(min=-5) - 4     # 3 bits behind the leading one; subnormals below 2^-6
    step = torch.ldexp(torch.ones_like(y), e)
    return (torch.round(y / step) * step).clamp(-448, 448)


def _through8(x, down, along, fmt="e4m3"):
    """What remains of [rows, cols] after 8 bits with one scale for every `down` x `along` elements, and the scales; a
    strip of them at a time.  Of fp32 values the codes are those that the format's two fp32 products define (values of
    a 16-bit type lie on borders between codes often); of fp64 values those of their quotients."""
    values, strips = torch.empty(x.shape, dtype=torch.float64, device=x.device), []
    top = 127.0 if fmt == "int8" else 448.0
    single = x.dtype == torch.float32

    def through(strip, largest):
        sc = (largest * (1 / torch.full_like(largest, top)) if single else largest / top).clamp(min=2.0 ** -126)
        ratio = (strip * (1 / sc)).double() if single else strip / sc
        return _round8(ratio, fmt) * sc.double(), sc

    if down > 1:
        for i in range(0, x.shape[0], down):
            strip = x[i:i + down]
            largest = strip.abs().max(0).values
            if along > 1:
                largest = torch.cat([p.max().expand(p.numel()) for p in largest.split(along)])
            values[i:i + down], sc = through(strip, largest)
            strips.append(sc[::along])
        return values, torch.stack(strips)
    for j in range(0, x.shape[1], along):
        strip = x[:, j:j + along]
        values[:, j:j + along], sc = through(strip, strip.abs().max(1, keepdim=True).values)
        strips.append(sc)
    return values, torch.cat(strips, 1)


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "product":
        M, N, K = case["M"], case["N"], case["K"]
        if 2.0 * M * N * K > 1.2e13:       # 64-bit products at about 1 TFLOP/s
            return None
        out = torch.zeros((N, K) if case["form"] == "g_w" else (M, N if case["form"] == "y" else K),
                          dtype=torch.float64, device="cuda")
        (ac, asc), (bc, bsc) = s["a"], s["b"]
        # block by block of the summed dim, the scales outside the block's own product
        inner = M if case["form"] == "g_w" else K if case["form"] == "y" else N
        for i, lo in enumerate(range(0, inner, 128)):
            k = slice(lo, min(lo + 128, inner))
            if case["form"] == "g_w":
                a, b = ac[k].double() * asc[i].double(), bc[k].double() * bsc[i].double()
                out += torch.einsum("mn,mk->nk", a, b)
                continue
            a = ac[:, k].double() * asc[:, i:i + 1].double()
            if case["form"] == "y":
                b = bc[:, k].double() * bsc[:, i].double().repeat_interleave(128)[:N, None]
                out += torch.einsum("mk,nk->mn", a, b)
            else:
                b = bc[k].double() * bsc[i].double().repeat_interleave(128)[:K]
                out += torch.einsum("mn,nk->mk", a, b)
        return out
    if op == "linear":
        x, w, g = s["x"].float(), s["w"].float(), s["g_y"].float()
        if 6.0 * case["M"] * case["N"] * case["K"] > 1.2e13:
            return None
        w = _through8(w, 128, 128)[0]
        y = torch.einsum("mk,nk->mn", _through8(x, 1, 128)[0], w)
        g_x = torch.einsum("mn,nk->mk", _through8(g, 1, 128)[0], w)
        return y, g_x, torch.einsum("mn,mk->nk", _through8(g, 128, 1)[0], _through8(x, 128, 1)[0])
    if op == "norm":
        h = s["x"].double() + (s["r"].double() if case["residual"] else 0)
        mean = torch.einsum("rc->r", h) / case["cols"]
        var = torch.einsum("rc,rc->r", h - mean[:, None], h - mean[:, None]) / case["cols"]
        norm = torch.sqrt(var + EPS)
        y = torch.addcmul(s["bias"].double(), (h - mean[:, None]) / norm[:, None], s["w"].double())
        got = (y,) if case["out"] == "same" else _through8(y, 1, case["group"] or case["cols"], case["out"])
        return (*got, h, mean, 1 / norm) if case["residual"] else (*got, mean, 1 / norm)
    if op == "norm_grads":
        h, mean, rstd, w, g_y = (s[k].double() for k in ("x", "mean", "rstd", "w", "g_y"))
        h = h - mean[:, None]
        # y_c = w_c (h_c - mean) rstd + b_c; d rstd / d h_c = -rstd^3 (h_c - mean) / cols, d mean / d h_c = 1 / cols
        flat = torch.einsum("rc,c->r", g_y, w) * rstd / case["cols"]
        along = torch.einsum("rc,rc,c->r", g_y, h, w) * rstd ** 3 / case["cols"]
        g_x = torch.addcmul(g_y * w * rstd[:, None] - flat[:, None], h, along[:, None], value=-1)
        if case["g_h"]:
            g_x += s["g_h"].double()
        return g_x, torch.einsum("rc,rc,r->c", g_y, h, rstd), torch.einsum("rc->c", g_y)
    x = s["x"].double()
    draws = _generator(s["state"].tolist(), x.numel())
    out = torch.zeros_like(x)
    kept = (draws >= round(case["p"] * 2.0 ** 32)).view(x.shape)
    out[kept] = x[kept] / (1 - case["p"])
    return out + s["r"].double() if case["residual"] else out


def _generator(state, n):
    """The n words of dropout's generator, with 16-bit limbs in products that stay below 2^53."""
    seed, offset = (v & (2 ** 64 - 1) for v in state)
    out = torch.empty(-(-n // 4), 4, dtype=torch.int64, device="cuda")
    step = 1 << 24
    for lo in range(0, out.shape[0], step):
        j = torch.arange(lo, min(lo + step, out.shape[0]), device="cuda")
        x0, x1 = j % 2 ** 32, j // 2 ** 32
        x2, x3 = torch.full_like(j, offset % 2 ** 32), torch.full_like(j, offset // 2 ** 32)
        for r in range(10):
            key0, key1 = (seed % 2 ** 32 + r * 0x9E3779B9) % 2 ** 32, (seed // 2 ** 32 + r * 0xBB67AE85) % 2 ** 32
            p_hi, p_lo = _wide(x0, 0xD2511F53)
            q_hi, q_lo = _wide(x2, 0xCD9E8D57)
            x0, x1, x2, x3 = q_hi ^ x1 ^ key0, q_lo, p_hi ^ x3 ^ key1, p_lo
        out[lo:lo + j.numel()] = torch.stack((x0, x1, x2, x3), -1)
    return out.flatten()[:n]


def _wide(x, m):
    """(upper, lower) 32 bits of x * m, both below 2^32."""
    x1, x0, m1, m0 = x // 65536, x % 65536, m // 65536, m % 65536
    mid = x1 * m0 + x0 * m0 // 65536
    mid2 = x0 * m1 + mid % 65536
    return x1 * m1 + mid // 65536 + mid2 // 65536, (mid2 % 65536) * 65536 + (x0 * m0) % 65536
