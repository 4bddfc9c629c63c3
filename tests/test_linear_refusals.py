"""Refusals of the linear layers around the attention: the C ABI's checks on the host,
before any launch, and the checks of the torch calls (CPU only)."""
import ctypes
import os
import re
import shutil

import pytest
import torch

from block_sparse_attention_fwd_gb300 import _lib, api, linear

OK, ODD = 0x10000, 0x10001
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_fwd_gb300 import build
    if not os.path.exists(_lib.LIB_PATH) or not build.up_to_date():
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc not available to build libbl_attn.so")
        build.build()
    return _lib.load()


TILE = dict(rows=4, cols=64, xs=64, rs=64, cs=64, bs=64, x=OK, rc=OK, rsc=OK, cc=OK, csc=OK, bc=0,
            bsc=0, dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=3), 1), (dict(x=0), 1), (dict(x=ODD), 1),
    (dict(xs=63), 1), (dict(rs=63), 1), (dict(cs=10), 1), (dict(rsc=0), 1), (dict(csc=ODD), 1),
    (dict(rc=0, cc=0), 1), (dict(bc=OK, bsc=OK), 1), (dict(cc=0, bc=OK), 1),
    (dict(rows=0, x=0), 0),
    (dict(rows=2 ** 38, cols=2 ** 20, xs=2 ** 20, rs=2 ** 20, cs=2 ** 20), 2)])
def test_tile_save_refuses(lib, kw, code):
    a = dict(TILE)
    a.update(kw)
    assert lib.bl_tile8_save(linear._TILE8_ARGS.pack(*a.values()), None) == code


@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=0), dict(dtype=4), dict(codes=None), dict(scales=None), dict(scales=ODD),
    dict(stride=63), dict(blocks=2), dict(x=None), dict(x=ODD)])
def test_tile_load_refuses(lib, kw):
    a = dict(rows=4, cols=64, dtype=0, codes=OK, stride=64, scales=OK, blocks=1, x=OK)
    a.update(kw)
    assert lib.bl_tile8_load(*a.values(), None) == 1
    assert lib.bl_tile8_load(0, 64, 0, None, 64, None, 0, None, None) == 0


MATMUL = dict(m=64, n=128, k=256, a=OK, asc=OK, ast=256, b=OK, bsc=OK, bst=256, out=OK, ws=0, wsb=0,
              form=0, dtype=0)


@pytest.mark.parametrize("kw,code", [
    (dict(m=-1), 1), (dict(n=0), 1), (dict(k=0), 1), (dict(m=2 ** 31), 1), (dict(a=0), 1),
    (dict(asc=0), 1), (dict(asc=ODD), 1), (dict(ast=255), 1), (dict(bst=100), 1), (dict(b=0), 1),
    (dict(bsc=0), 1), (dict(out=0), 1), (dict(out=ODD), 1), (dict(dtype=3), 1), (dict(form=3), 1),
    (dict(form=-1), 1), (dict(m=0), 0),
    (dict(form=1, ast=127), 1), (dict(form=2, ast=127, bst=256), 1),
    (dict(a=ODD), 4), (dict(ast=257), 4), (dict(ast=257, ws=OK, wsb=64 * 256 - 1), 4),
    (dict(bst=260, ws=ODD, wsb=1 << 20), 4),
    (dict(m=2 ** 23, n=2 ** 22, k=16, ast=16, bst=16), 2)])
def test_product_refuses(lib, kw, code):
    a = dict(MATMUL)
    a.update(kw)
    assert lib.bl_matmul8(linear._MATMUL8_ARGS.pack(*a.values()), None) == code
    assert lib.bl_matmul8(None, None) == 1


def test_product_workspace(lib):
    def need(**kw):
        return lib.bl_matmul8_workspace_bytes(linear._MATMUL8_ARGS.pack(*dict(MATMUL, **kw).values()))
    assert need() == 0 and need(n=0) == 0
    assert need(k=250, ast=250) == 64 * 256                       # rows of 256 bytes
    assert need(k=1, ast=1, bst=16) == 1024
    assert need(k=1, ast=1, bst=1) == 1024 + 2048
    assert need(form=1, ast=129) == 64 * 128
    assert need(form=2, ast=128, bst=257) == 64 * 256


NORM = dict(rows=4, cols=64, xs=64, rs=64, x=OK, r=0, w=OK, b=OK, y=OK, h=0, mean=OK, rstd=OK, y8=0,
            eps=1e-5, dtype=0, wt=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=7), 1), (dict(x=0), 1), (dict(xs=63), 1),
    (dict(x=ODD), 1), (dict(r=OK, rs=10), 1), (dict(r=ODD), 1), (dict(wt=1), 1), (dict(w=0, wt=1), 1),
    (dict(w=ODD), 1), (dict(b=ODD), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(y=0), 1), (dict(h=OK), 1), (dict(rstd=ODD), 1), (dict(mean=ODD), 1),
    (dict(cols=16385, xs=16385), 2), (dict(rows=0, x=0, y=0), 0)])
def test_layer_norm_forward_refuses(lib, kw, code):
    a = dict(NORM)
    a.update(kw)
    assert lib.bl_layer_norm_fwd(linear._LAYER_NORM_ARGS.pack(*a.values()), None) == code
    y8 = _lib.Act8Struct(OK, OK, 2, 48)
    assert lib.bl_layer_norm_fwd(linear._LAYER_NORM_ARGS.pack(
        *dict(NORM, y8=ctypes.addressof(y8)).values()), None) == 1


BWD = dict(rows=4, cols=64, gy=OK, h=OK, h8=0, mean=OK, rstd=OK, w=OK, gh=0, gx=OK, gw=0, gb=0, ws=0,
           wsb=0, dtype=0, wt=0)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(dtype=5), 1), (dict(gy=0), 1), (dict(h=0), 1), (dict(mean=0), 1),
    (dict(rstd=0), 1), (dict(gx=0), 1), (dict(gh=ODD), 1), (dict(wt=1), 1), (dict(mean=ODD), 1),
    (dict(w=0, gb=OK, wt=1), 1), (dict(gb=ODD), 1), (dict(gw=OK), 4), (dict(gb=OK, ws=OK, wsb=16), 4),
    (dict(cols=16385), 2)])
def test_layer_norm_backward_refuses(lib, kw, code):
    a = dict(BWD)
    a.update(kw)
    assert lib.bl_layer_norm_bwd(linear._LAYER_NORM_BWD_ARGS.pack(*a.values()), None) == code
    h8 = _lib.Act8Struct(OK, OK, 1, 0)
    assert lib.bl_layer_norm_bwd(linear._LAYER_NORM_BWD_ARGS.pack(
        *dict(BWD, h8=ctypes.addressof(h8)).values()), None) == 1      # h and h8
    assert lib.bl_layer_norm_bwd_workspace_bytes(5, 64) > 0
    assert lib.bl_layer_norm_bwd_workspace_bytes(5, 20000) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=3), 1), (dict(x=None), 1), (dict(x=ODD), 1),
    (dict(xs=63), 1), (dict(r=OK, rs=3), 1), (dict(r=ODD), 1), (dict(p=-0.1), 1), (dict(p=1.1), 1),
    (dict(p=float("nan")), 1), (dict(state=None), 1), (dict(state=OK + 4), 1), (dict(y=None), 1),
    (dict(rows=2 ** 30, cols=2 ** 13, xs=2 ** 13), 2), (dict(rows=0, x=None, y=None), 0)])
def test_dropout_refuses(lib, kw, code):
    a = dict(rows=4, cols=64, dtype=0, x=OK, xs=64, r=None, rs=64, p=0.5, state=OK, y=OK)
    a.update(kw)
    assert lib.bl_dropout(*a.values(), None) == code
    assert lib.bl_dropout_next(None, OK, None) == 1 and lib.bl_dropout_next(OK, OK, None) == 1
    assert lib.bl_dropout_next(OK + 4, OK, None) == 1


def test_arguments_are_laid_out_as_the_structs():
    """The packed bytes against the header's members, one by one."""
    text = open(os.path.join(ROOT, "include", "bl_attn.h")).read()
    text = re.sub(r"/\*.*?\*/", "", text, flags=re.S)
    sizes = {"int64_t": "q", "int": "i", "float": "f", "size_t": "Q"}
    for name, packer in (("bl_tile8_args", linear._TILE8_ARGS), ("bl_matmul8_args", linear._MATMUL8_ARGS),
                         ("bl_layer_norm_args", linear._LAYER_NORM_ARGS),
                         ("bl_layer_norm_bwd_args", linear._LAYER_NORM_BWD_ARGS)):
        body = re.search(r"typedef struct \{([^{}]*)\} " + name + ";", text).group(1)
        want = ""
        for line in filter(None, (s.strip() for s in body.split(";"))):
            if "*" in line:
                want += "Q"
            else:
                kind, names = line.split(None, 1)
                want += sizes[kind] * len(names.split(","))
        have = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), packer.format.lstrip("<"))
        assert have.rstrip("x") == want and packer.size % 8 == 0, name


def test_cpu_tensors_and_types_are_refused():
    x, st = torch.zeros(2, 8), torch.zeros(2, dtype=torch.int64)
    codes = torch.zeros(2, 8, dtype=torch.float8_e4m3fn)
    for call in (lambda: linear.weight_save(x), lambda: linear.act_save_both(x),
                 lambda: linear.layer_norm_fwd(x, None, None), lambda: linear.dropout(x, 0.1, st),
                 lambda: linear.layer_norm_bwd(x, x, x, x, None), lambda: linear.dropout_next(st),
                 lambda: linear.Weight8(codes, x, torch.bfloat16),
                 lambda: linear.Cols8(codes, x, torch.bfloat16),
                 lambda: linear.matmul8(x, x), lambda: linear.matmul8_gx(x, x),
                 lambda: linear.matmul8_gw(x, x)):
        with pytest.raises(TypeError):
            call()


def test_modules_refuse():
    for call in (lambda: api.BLLayerNorm(0), lambda: api.BLLayerNorm(20000),
                 lambda: api.BLLayerNorm(8, checkpoint="fp8"), lambda: api.BLLayerNorm(8, group=7),
                 lambda: api.BLDropout(1.5), lambda: api.BLDropout(-0.1), lambda: api.BLLinear8(0, 4),
                 lambda: api.BLLinear8(4, 8)(torch.zeros(2, 5)),
                 lambda: api.BLLinear8(4, 8)(torch.zeros(2, 4), w8=torch.zeros(8, 4)),
                 lambda: api.BLLayerNorm(8)(torch.zeros(2, 9))):
        with pytest.raises(ValueError):
            call()
    norm = api.BLLayerNorm(8, affine=False)
    assert norm.weight is None and norm.bias is None
    assert api.BLLayerNorm(8, bias=False).bias is None
    drop = api.BLDropout(0.3, seed=11, device="cpu")
    assert drop.state.tolist() == [11, 0]
    x = torch.ones(3)
    assert drop.eval()(x) is x and torch.equal(drop(x, x), 2 * x)
    assert "state" in drop.state_dict()
