"""The autograd modules of the linear layers around the attention on the GPU: gradients
against fp64 autograd and differences, a whole block, streams and captured graphs."""
import numpy as np
import pytest
import torch

from oracle import linear as OL

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    import __graft_entry__ as g
    g.build()


@pytest.fixture(scope="module")
def bl():
    import block_sparse_attention_fwd_gb300 as bl
    return bl


def _randn(*shape, dtype=torch.float32, seed=0):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def _rel(a, b):
    a, b = a.detach().double(), b.detach().double()
    return float((a - b).norm() / b.norm())


def _norm64(x, w, b, eps):
    c = x - x.mean(-1, keepdim=True)
    y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + eps)
    return y if w is None else y * w + (0 if b is None else b)


# --- layer norm --------------------------------------------------------------------

@pytest.mark.parametrize("cols", [96, 1024])
@pytest.mark.parametrize("residual", [False, True])
def test_layer_norm_gradients(bl, residual, cols):
    """fp32: against fp64 autograd (some 64 roundings of 2^-24 are 4e-6) and against central
    differences of the module itself along a direction."""
    norm = bl.BLLayerNorm(cols, eps=1e-5, device="cuda")
    with torch.no_grad():
        norm.weight.copy_(1 + 0.3 * _randn(cols, seed=1))
        norm.bias.copy_(0.3 * _randn(cols, seed=2))
    x, r = (_randn(2, 5, cols, seed=s).requires_grad_() for s in (3, 4))
    gy, gh = _randn(2, 5, cols, seed=5), _randn(2, 5, cols, seed=6)

    def loss(x, r):
        if not residual:
            return (norm(x).double() * gy).sum()
        y, h = norm(x, r)
        return (y.double() * gy).sum() + (h.double() * gh).sum()

    leaves = [x, norm.weight, norm.bias] + ([r] if residual else [])
    got = torch.autograd.grad(loss(x, r), leaves)
    a, w, b, c = (t.detach().double().requires_grad_() for t in (x, norm.weight, norm.bias, r))
    h = a + c if residual else a
    ref_loss = (_norm64(h, w, b, 1e-5) * gy).sum() + ((h * gh).sum() if residual else 0)
    ref = torch.autograd.grad(ref_loss, [a, w, b] + ([c] if residual else []))
    for g, f in zip(got, ref):
        assert _rel(g, f) <= 4e-6
    d, e = _randn(2, 5, cols, seed=7), 1e-2
    with torch.no_grad():
        slope = float(loss(x + e * d, r) - loss(x - e * d, r)) / (2 * e)
    assert abs(slope - float((got[0].double() * d).sum())) <= 1e-3 * float(got[0].norm() * d.norm())


def test_layer_norm_unused_outputs_and_parts(bl):
    norm = bl.BLLayerNorm(64, device="cuda", dtype=torch.bfloat16)
    x = _randn(3, 64, dtype=torch.bfloat16, seed=8).requires_grad_()
    r = _randn(3, 64, dtype=torch.bfloat16, seed=9).requires_grad_()
    _, h = norm(x, r)
    gx, gr, gw, gb = torch.autograd.grad(h.float().sum(), [x, r, norm.weight, norm.bias], allow_unused=True)
    assert (gx == 1).all() and (gr == 1).all() and (gw == 0).all() and (gb == 0).all()
    y, _ = norm(x, r)
    gx, gr, gb = torch.autograd.grad(y.sum(), [x, r, norm.bias])      # a gradient that is one number expanded
    assert torch.equal(gx, gr) and (gb == 3).all()
    y, h = norm(x, x)
    g, = torch.autograd.grad(h.sum(), x)
    assert (g == 2).all()
    plain = bl.BLLayerNorm(64, affine=False)
    g, = torch.autograd.grad(plain(x), x, _randn(3, 64, dtype=torch.bfloat16, seed=10))
    a = x.detach().double().requires_grad_()
    ref, = torch.autograd.grad(_norm64(a, None, None, 1e-5), a, _randn(3, 64, dtype=torch.bfloat16, seed=10).double())
    assert _rel(g, ref) <= 2 ** -8
    frozen = bl.BLLayerNorm(64, bias=False, device="cuda").requires_grad_(False)
    frozen(x).float().sum().backward()
    assert x.grad is not None and frozen.weight.grad is None
    assert bl.BLLayerNorm(64, device="cuda")(x.detach()).requires_grad


@pytest.mark.parametrize("fmt,tol", [("int8", 0.02), ("e4m3", 0.06)])
def test_layer_norm_with_a_checkpoint(bl, fmt, tol):
    """h in 8 bits: half a step is amax / 254 (int8: about 1% of an element of normal size) or
    2^-4 (e4m3: 3.6% root mean square at most) of u, which enters g_w once and g_x's smaller
    terms; g_b does not read h."""
    x = _randn(200, 640, dtype=torch.bfloat16, seed=11).requires_grad_()
    gy = _randn(200, 640, dtype=torch.bfloat16, seed=12)
    got = {}
    for c in (None, fmt):
        norm = bl.BLLayerNorm(640, checkpoint=c, device="cuda")
        y = norm(x)
        got[c] = (y, *torch.autograd.grad(y, [x, norm.weight, norm.bias], gy))
    assert torch.equal(got[None][0], got[fmt][0]) and torch.equal(got[None][3], got[fmt][3])
    assert _rel(got[fmt][1], got[None][1]) <= tol and _rel(got[fmt][2], got[None][2]) <= tol


# --- linear --------------------------------------------------------------------------

@pytest.mark.parametrize("M,N,K", [(300, 200, 328), (1, 64, 128), (37, 1001, 77)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_linear_is_the_product_of_what_it_saved(bl, M, N, K, dtype):
    """y, g_x and g_w against fp64 products of the codes' values: half a step of the type and
    some 300 roundings of 2^-24 (norms); and within 8 bits' noise, 2^-4 / sqrt(3) an element of
    each factor, 0.06 together, of the products of x, w and g themselves."""
    lin = bl.BLLinear8(K, N, device="cuda", dtype=dtype)
    x = _randn(M, K, dtype=dtype, seed=1).requires_grad_()
    g = _randn(M, N, dtype=dtype, seed=2)
    y = lin(x)
    gx, gw = torch.autograd.grad(y, [x, lin.weight], g)
    xr, xc = (bl.act_load(t).double() for t in _as_fp32(bl, x.detach()))
    gr, gc = (bl.act_load(t).double() for t in _as_fp32(bl, g))
    w = bl.act_load(bl.weight_save(lin.weight.detach().float())).double()
    tol = torch.finfo(dtype).eps / 2 + 300 * 2.0 ** -24
    for got, ref, plain in ((y, xr @ w.T, x.double() @ lin.weight.double().T),
                            (gx, gr @ w, g.double() @ lin.weight.double()),
                            (gw, gc.T @ xc, g.double().T @ x.double())):
        assert got.dtype == dtype and _rel(got, ref) <= tol
        assert _rel(got, plain) <= 0.06
    assert torch.equal(lin(x.view(1, M, K))[0], y)
    assert torch.equal(lin(x, w8=bl.weight_save(lin.weight.detach())), y)


def _as_fp32(bl, t):
    """The Act8 and Cols8 of t, to be loaded without a rounding."""
    a, c = bl.act_save_both(t)
    return bl.Act8(a.codes, a.scales, 128, torch.float32), bl.Cols8(c.codes, c.scales, torch.float32)


def test_linear_of_a_norms_codes_and_what_it_keeps(bl):
    x = _randn(50, 256, dtype=torch.bfloat16, seed=3)
    lin = bl.BLLinear8(256, 384, device="cuda", dtype=torch.bfloat16)
    y8 = bl.layer_norm_fwd_8bit(x, None, None)[0]
    with pytest.raises(ValueError):
        lin(y8)                                          # the weight wants a gradient
    with torch.no_grad():
        w8 = bl.weight_save(lin.weight)
        assert torch.equal(lin(y8), bl.matmul8(y8, w8)) and torch.equal(lin(y8, w8), bl.matmul8(y8, w8))
    held = []
    hooks = torch.autograd.graph.saved_tensors_hooks(lambda t: held.append(t) or t, lambda t: t)
    with hooks:
        lin(x)                                           # no gradient of x: nothing of the weight
    assert sum(t.numel() * t.element_size() for t in held) == 50 * 256 + 4 * 256
    held.clear()
    with hooks:
        lin(x.clone().requires_grad_())
    assert sum(t.numel() * t.element_size() for t in held) == 50 * 256 + 4 * 256 + 384 * 256 + 4 * 6
    held.clear()
    with hooks, torch.no_grad():
        lin(x)
    assert not held
    lin.requires_grad_(False)
    leaf = x.clone().requires_grad_()
    lin(leaf).float().sum().backward()                   # an expanded gradient, of x alone
    assert leaf.grad is not None and lin.weight.grad is None


# --- dropout -------------------------------------------------------------------------

def test_dropout_gradients_and_state(bl):
    drop = bl.BLDropout(0.3, seed=21, device="cuda")
    x, r = (_randn(40, 33, seed=s).requires_grad_() for s in (1, 2))
    for call in range(3):
        y = drop(x, r)
        keep = torch.from_numpy(OL.kept(40 * 33, 0.3, 21, call)).view(40, 33).cuda()
        assert torch.equal(y != r, keep) and drop.state.tolist() == [21, call + 1]
        g = _randn(40, 33, seed=5 + call)
        gx, gr = torch.autograd.grad(y, [x, r], g)
        assert torch.equal(gr, g) and torch.equal(gx, torch.where(keep, g * np.float32(1 / 0.7).item(), 0.0))
    # two calls before their backward passes, and a saved state
    state = drop.state_dict()
    a, b = drop(x), drop(x)
    ga, = torch.autograd.grad(a.sum(), x, retain_graph=True)
    gb, = torch.autograd.grad(b.sum(), x)
    assert torch.equal(ga != 0, a != 0) and torch.equal(gb != 0, b != 0) and not torch.equal(ga, gb)
    again = bl.BLDropout(0.3, device="cuda")
    again.load_state_dict({k: v.clone() for k, v in state.items()})
    again.state[1] -= 2
    assert torch.equal(again(x), a)
    same, = torch.autograd.grad(drop(x, x).sum(), x)
    assert ((same - 1).abs() < 1e-6).logical_or((same - 1 - 1 / 0.7).abs() < 1e-6).all()
    assert torch.equal(drop.eval()(x, r), x + r) and drop(x) is x
    drop.train()
    leaf = _randn(6, 8, seed=9).t().requires_grad_()     # any strides
    drop(leaf).sum().backward()
    assert leaf.grad is not None


# --- together ------------------------------------------------------------------------

class _Block(torch.nn.Module):
    """Entry norm, q, k and v in one product, q/k norm, attention, output product, dropout and
    the stream's addition, exit norm."""

    def __init__(self, bl, H, Hk, d, p, causal):
        super().__init__()
        t = dict(device="cuda", dtype=torch.bfloat16)
        self.H, self.Hk, self.d = H, Hk, d
        self.entry = bl.BLLayerNorm(H * d, **t)
        self.qkv = bl.BLLinear8(H * d, (H + 2 * Hk) * d, **t)
        self.attn = bl.BLAttention(0.0, causal=causal, q_norm=bl.BLLayerNorm(d, **t),
                                   k_norm=bl.BLLayerNorm(d, **t))
        self.out = bl.BLLinear8(H * d, H * d, **t)
        self.drop = bl.BLDropout(p, seed=5, device="cuda")
        self.exit = bl.BLLayerNorm(H * d, checkpoint="int8", **t)

    def forward(self, x):
        B, n, _ = x.shape
        q, k, v = self.qkv(self.entry(x)).view(B, n, -1, self.d).split([self.H, self.Hk, self.Hk], 2)
        o = self.attn(q, k, v)
        h = self.drop(self.out(o.flatten(2)), x)
        return self.exit(h)

    def reference(self, x, keep, p):
        """The same in fp64 on given weights, without 8 bits."""
        B, n, c = x.shape
        P = {k: v.detach().double().requires_grad_() for k, v in self.named_parameters()}
        norm = lambda t, m: _norm64(t, P[m + ".weight"], P[m + ".bias"], 1e-5)      # noqa: E731
        qkv = norm(x, "entry") @ P["qkv.weight"].T
        q, k, v = qkv.view(B, n, -1, self.d).split([self.H, self.Hk, self.Hk], 2)
        q, k = norm(q, "attn.q_norm").transpose(1, 2), norm(k, "attn.k_norm").transpose(1, 2)
        k, v = (t.repeat_interleave(self.H // self.Hk, 1) for t in (k, v.transpose(1, 2)))
        s = q @ k.transpose(2, 3) * self.d ** -0.5
        if self.attn.causal:
            s = s.masked_fill(torch.ones(n, n, dtype=torch.bool, device="cuda").triu(1), float("-inf"))
        o = (s.softmax(-1) @ v).transpose(1, 2).flatten(2) @ P["out.weight"].T
        h = x + torch.where(keep, o / (1 - p), 0.0)
        return norm(h, "exit"), P


@pytest.mark.parametrize("B,n,H,Hk,d,causal", [(2, 200, 4, 2, 64, True), (1, 333, 2, 2, 128, False)])
def test_block_together(bl, B, n, H, Hk, d, causal):
    """Output and gradients of all weights and of x against fp64 without 8 bits.  Each product
    has up to 0.05 of 8 bits' noise (two factors, 2^-4 / sqrt(3) of an element each at most);
    two follow one another forward and two more backward, and the softmax passes theirs on:
    0.25 of the norm for gradients, 0.1 for the output."""
    p = 0.2
    block = _Block(bl, H, Hk, d, p, causal)
    x = _randn(B, n, H * d, dtype=torch.bfloat16, seed=1).requires_grad_()
    g = _randn(B, n, H * d, dtype=torch.bfloat16, seed=2)
    y = block(x)
    got = torch.autograd.grad(y, [x, *block.parameters()], g)
    keep = torch.from_numpy(OL.kept(x.numel(), p, 5, 0)).view(x.shape).cuda()
    x64 = x.detach().double().requires_grad_()
    ref, P = block.reference(x64, keep, p)
    want = torch.autograd.grad(ref, [x64, *P.values()], g.double())
    assert _rel(y, ref) <= 0.1
    names = ["x", *P]
    for name, a, b in zip(names, got, want):
        # the softmax takes no notice of a shift of the keys' scores: g of k's bias is noise
        if name == "attn.k_norm.bias":
            continue
        assert torch.isfinite(a).all() and _rel(a, b) <= 0.25, (name, _rel(a, b))


def test_block_without_gradients(bl):
    """The same block for a few tokens, from codes to codes: what a user serves it with."""
    block = _Block(bl, 4, 2, 64, 0.2, True).eval()
    x = _randn(3, 1, 256, dtype=torch.bfloat16, seed=4)
    with torch.no_grad():
        want = block(x)
        qkv8, out8 = bl.weight_save(block.qkv.weight), bl.weight_save(block.out.weight)
        y8, _, _, _ = bl.layer_norm_fwd_8bit(x, block.entry.weight, block.entry.bias)
        q, k, v = block.qkv(y8, qkv8).view(3, 1, 8, 64).split([4, 2, 2], 2)
        o = block.attn(q, k, v)
        y, h, _, _ = bl.layer_norm_fwd(block.out(bl.act_save(o.flatten(2), "e4m3", 128), out8),
                                       block.exit.weight, block.exit.bias, residual=x)
    # the entry norm's y in 8 bits comes from before its rounding to bf16, and the stream is
    # added before a rounding: a code's step in few of 256 elements, 2^-4 / 16 of a row's norm
    assert _rel(y, want) <= 2 ** -4


# --- streams, graphs -------------------------------------------------------------------

def _operators(bl):
    """name -> (call, outputs)."""
    t = torch.bfloat16
    x, r, g = (_randn(700, 1032, dtype=t, seed=s) for s in (1, 2, 3))
    w, b = _randn(1032, seed=4), _randn(1032, seed=5)
    weight = _randn(520, 1032, dtype=t, seed=6)
    w8, (x8, xc) = bl.weight_save(weight), bl.act_save_both(x)
    g8, gc = bl.act_save_both(_randn(700, 520, dtype=t, seed=7))
    odd = bl.act_save(x[:, :1001].contiguous(), "e4m3", 128)
    odd_w = bl.weight_save(weight[:, :1001])
    few = bl.act_save(x[:5], "e4m3", 128)
    _, _, mean, rstd = bl.layer_norm_fwd(x, w, b)
    st = torch.tensor([3, 4], device="cuda")
    codes = lambda a: [a.codes.view(torch.uint8), a.scales]      # noqa: E731
    return {
        "weight_save": lambda: codes(bl.weight_save(weight)),
        "act_save_both": lambda: [c for a in bl.act_save_both(x) for c in codes(a)],
        "y": lambda: [bl.matmul8(x8, w8)], "y few": lambda: [bl.matmul8(few, w8)],
        "y odd": lambda: [bl.matmul8(odd, odd_w)],
        "g_x": lambda: [bl.matmul8_gx(g8, w8)], "g_w": lambda: [bl.matmul8_gw(gc, xc)],
        "norm": lambda: [*bl.layer_norm_fwd(x, w, b, residual=r)],
        "norm 8": lambda: codes(bl.layer_norm_fwd_8bit(x, w, b, residual=r)[0]),
        "norm bwd": lambda: [*bl.layer_norm_bwd(g, x, mean, rstd, w, g_h=r)],
        "dropout": lambda: [bl.dropout(x, 0.2, st, r)],
    }


def test_another_stream(bl):
    ops = _operators(bl)
    want = {k: f() for k, f in ops.items()}
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = {k: f() for k, f in ops.items()}
    side.synchronize()
    for k in ops:
        assert all(torch.equal(a, b) for a, b in zip(got[k], want[k])), k


def test_two_streams_at_once(bl):
    """The same calls on two streams beside each other: nothing is shared between calls."""
    ops = _operators(bl)
    want = {k: f() for k, f in ops.items()}
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(3):
        for k, f in ops.items():
            for i, side in enumerate(sides):
                with torch.cuda.stream(side):
                    got[i].append((k, f()))
    torch.cuda.synchronize()
    for outs in got:
        for k, o in outs:
            assert all(torch.equal(a, b) for a, b in zip(o, want[k])), k


def test_operators_replay_from_a_graph(bl):
    ops = _operators(bl)
    want = {k: f() for k, f in ops.items()}
    torch.cuda.synchronize()
    graphs = {}
    for k, f in ops.items():
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = f()
        graphs[k] = (graph, out)
    for _ in range(2):
        for graph, out in graphs.values():
            for o in out:
                if o.dtype != torch.bfloat16 or o.numel() != 700 * 1032:
                    o.zero_()
            graph.replay()
    torch.cuda.synchronize()
    for k, (_, out) in graphs.items():
        assert all(torch.equal(a, b) for a, b in zip(out, want[k])), k


def test_a_training_step_replays_from_a_graph(bl):
    """Forward, backward and update, captured: every replay draws another mask and goes on
    from the last one's weights, as the same steps run one by one do."""
    def setup():
        torch.manual_seed(0)
        lin = bl.BLLinear8(256, 256, device="cuda", dtype=torch.float32)
        norm = bl.BLLayerNorm(256, device="cuda")
        drop = bl.BLDropout(0.3, seed=1, device="cuda")
        return lin, norm, drop, [*lin.parameters(), *norm.parameters()]

    x, g = _randn(64, 256, seed=1), _randn(64, 256, seed=2)

    def step(lin, norm, drop, params):
        y = norm(drop(lin(x), x))
        grads = torch.autograd.grad(y, params, g)
        with torch.no_grad():
            for p, d in zip(params, grads):
                p.sub_(d, alpha=1e-3)
        return y

    lin, norm, drop, params = setup()
    masks = []
    for _ in range(4):
        step(lin, norm, drop, params)
        masks.append(drop.state.tolist())
    lin2, norm2, drop2, params2 = setup()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(lin2, norm2, drop2, params2)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(lin2, norm2, drop2, params2)
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert masks[-1] == drop2.state.tolist() == [1, 4]
    for a, b in zip(params, params2):
        assert torch.equal(a, b)
