"""Refusals of the operators around the attention: the C ABI's checks on the
host, before any launch, and the checks of the torch calls (CPU only)."""
import ctypes
import os
import shutil

import pytest
import torch

from block_sparse_attention_fwd_gb300 import _lib, api, ops

OK = 0x10000
ODD = 0x10001
OKP = ctypes.c_void_p(OK)


@pytest.fixture(scope="module")
def lib():
    from block_sparse_attention_fwd_gb300 import build
    if not os.path.exists(_lib.LIB_PATH) or not build.up_to_date():
        if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
            pytest.skip("nvcc not available to build libbl_attn.so")
        build.build()
    return _lib.load()


def _act8(codes=OK, scales=OK, fmt=1, group=0):
    return _lib.Act8Struct(codes, scales, fmt, group)


# --- C ABI ----------------------------------------------------------------------

@pytest.mark.parametrize("kw", [
    dict(rows=-1), dict(cols=0), dict(dtype=3), dict(dtype=-1), dict(x=None), dict(x=ODD),
    dict(stride=63), dict(a=dict(fmt=0)), dict(a=dict(fmt=3)), dict(a=dict(group=16)),
    dict(a=dict(group=-32)), dict(a=dict(codes=None)), dict(a=dict(scales=None)),
    dict(a=dict(scales=ODD)), dict(a=None)])
def test_act_save_and_load_refuse(lib, kw):
    a = dict(rows=4, cols=64, dtype=0, x=OK, stride=64, a={})
    a.update(kw)
    s = None if a["a"] is None else ctypes.byref(_act8(**a["a"]))
    assert lib.bl_act_save(a["rows"], a["cols"], a["dtype"], a["x"], a["stride"], s, None) == 1
    if "stride" not in kw:
        assert lib.bl_act_load(a["rows"], a["cols"], a["dtype"], s, a["x"], None) == 1


def test_no_rows_launch_nothing(lib):
    empty = ctypes.byref(_act8(codes=None, scales=None))
    assert lib.bl_act_save(0, 64, 0, None, 64, empty, None) == 0
    assert lib.bl_act_load(0, 64, 0, empty, None, None) == 0
    assert lib.bl_rms_norm_fwd(0, 64, 0, None, 64, None, 64, None, 0, 1e-6, None, None, None, None,
                               None) == 0
    assert lib.bl_rms_norm_bwd(0, 64, 0, None, None, None, None, None, 0, None, None, None, None, 0,
                               None) == 0
    assert lib.bl_rms_norm_bwd_workspace_bytes(0, 64) == 0


NORM = dict(rows=4, cols=64, dtype=0, x=OK, xs=64, r=None, rs=64, w=OK, wt=0, eps=1e-6, y=OK, h=None,
            rstd=OK, y8=None)


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(cols=0), 1), (dict(dtype=7), 1), (dict(x=None), 1), (dict(xs=63), 1),
    (dict(x=ODD), 1), (dict(r=OK, rs=10), 1), (dict(r=ODD), 1), (dict(wt=1), 1),
    (dict(dtype=2, wt=0), 1), (dict(w=ODD), 1), (dict(eps=-1.0), 1), (dict(eps=float("nan")), 1),
    (dict(eps=float("inf")), 1), (dict(y=None), 1), (dict(h=OK), 1), (dict(rstd=ODD), 1),
    (dict(y8=dict(group=48)), 1), (dict(y8=dict(fmt=9)), 1),
    (dict(cols=16385, xs=16385), 2)])
def test_norm_forward_refuses(lib, kw, code):
    a = dict(NORM)
    a.update(kw)
    y8 = None if a["y8"] is None else ctypes.byref(_act8(**a["y8"]))
    assert lib.bl_rms_norm_fwd(a["rows"], a["cols"], a["dtype"], a["x"], a["xs"], a["r"], a["rs"],
                               a["w"], a["wt"], a["eps"], a["y"], a["h"], a["rstd"], y8,
                               None) == code


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), 1), (dict(dtype=5), 1), (dict(gy=None), 1), (dict(h=None), 1),
    (dict(h8={}), 1), (dict(rstd=None), 1), (dict(gx=None), 1), (dict(gh=ODD), 1), (dict(wt=1), 1),
    (dict(h=None, h8=dict(group=5)), 1), (dict(ws=None), 4), (dict(ws=0x10004), 4), (dict(short=1), 4),
    (dict(cols=16392), 2)])
def test_norm_backward_refuses(lib, kw, code):
    a = dict(rows=4, cols=64, dtype=0, gy=OK, h=OK, h8=None, rstd=OK, w=OK, wt=0, gh=None, gx=OK,
             gw=OK, ws=OK, short=0)
    a.update(kw)
    h8 = None if a["h8"] is None else ctypes.byref(_act8(**a["h8"]))
    need = lib.bl_rms_norm_bwd_workspace_bytes(4, 64)
    assert need >= 64 * 4 and lib.bl_rms_norm_bwd_workspace_bytes(4, 16392) == 0
    assert lib.bl_rms_norm_bwd(a["rows"], a["cols"], a["dtype"], a["gy"], a["h"], h8, a["rstd"],
                               a["w"], a["wt"], a["gh"], a["gx"], a["gw"], a["ws"],
                               need - a["short"], None) == code


def _rope_args(**kw):
    a = _lib.RopeArgs()
    v = dict(B=2, n=5, H=4, Hk=2, d=64, pairs=32, axes=1, sections=(32,), interleaved=0, inverse=0,
             dtype=0, q=OK, k=OK, q_out=2 * OK, k_out=3 * OK, q_strides=(1280, 256, 64),
             k_strides=(640, 128, 64), q_out_strides=(1280, 256, 64), k_out_strides=(640, 128, 64),
             positions=OK, positions_batch_stride=5, freqs=OK)
    v.update(kw)
    for name, x in v.items():
        if isinstance(x, tuple):
            getattr(a, name)[:len(x)] = x
        else:
            setattr(a, name, x)
    return a


@pytest.mark.parametrize("kw", [
    dict(B=-1), dict(n=-1), dict(H=0), dict(Hk=-1), dict(d=1), dict(pairs=0), dict(pairs=33),
    dict(axes=0), dict(axes=5), dict(sections=(31,)), dict(sections=(33,)),
    dict(axes=2, sections=(32, 0)), dict(axes=2, sections=(30, 3)), dict(dtype=3),
    dict(interleaved=2), dict(inverse=-1), dict(q=None), dict(k=None), dict(q_out=None),
    dict(k_out=None), dict(positions=None), dict(freqs=None), dict(q=ODD), dict(freqs=OK + 4),
    dict(positions=OK + 2), dict(q_strides=(-1280, 256, 64)), dict(q_out_strides=(1280, 256, 32)),
    dict(k_out_strides=(640, 32, 64)), dict(q_out_strides=(0, 256, 64)),
    dict(q_out=OK, q_strides=(2560, 512, 64)), dict(positions_batch_stride=4)])
def test_rope_refuses(lib, kw):
    assert lib.bl_rope(ctypes.byref(_rope_args(**kw)), None) == 1


# one tensor [2, 5, 6 heads, 64] behind both, token stride 384, batch stride 1920
_ONE = (1920, 384, 64)


@pytest.mark.parametrize("at", [0, 64, 3 * 64, -64, 32, 384, -384 + 64, 1920, 1920 - 384 + 128])
def test_rope_refuses_outputs_that_share_elements(lib, at):
    """k begins `at` elements behind q: some head of k is (part of) one of q's."""
    k = OK + 2 * at
    args = _rope_args(q=OK, q_out=OK, k=k, k_out=k, q_strides=_ONE, q_out_strides=_ONE,
                      k_strides=_ONE, k_out_strides=_ONE)
    assert lib.bl_rope(ctypes.byref(args), None) == 1


@pytest.mark.parametrize("strides", [(64, 384, 64), (0, 384, 64), (10 ** 9, 384, 64),
                                     (7, 64, 320)])
def test_rope_refuses_shared_elements_of_one_batch(lib, strides):
    """One batch, whose stride says nothing; the last: heads before tokens."""
    args = _rope_args(B=1, q=OK, q_out=OK, k=OK + 2 * strides[2], k_out=OK + 2 * strides[2],
                      q_strides=strides, q_out_strides=strides, k_strides=strides,
                      k_out_strides=strides)
    assert lib.bl_rope(ctypes.byref(args), None) == 1


@pytest.mark.parametrize("kw", [
    dict(H=1, strides=(64, 64, 64)),                     # the same elements as batch and token
    dict(H=1, strides=(128, 64, 64)),                    # batches that begin within one another
    dict(H=4, strides=(1216, 256, 64)),                  # by one head
    dict(H=4, strides=(1280, 64, 64)),                   # tokens and heads
    dict(H=4, strides=(1280, 192, 64)),
    dict(H=4, strides=(256, 512, 64), B=3),              # batches within tokens: three of 256 in 512
    dict(H=4, strides=(64, 512, 128), B=3),
    dict(H=4, strides=(2 ** 62, 256, 64))])              # past any memory
@pytest.mark.parametrize("which", ["q", "k"])
def test_rope_refuses_an_output_that_meets_itself(lib, which, kw):
    kw = dict(kw)
    H, st = kw.pop("H"), kw.pop("strides")
    at = {"q": dict(H=H, q=OK, q_out=OK, q_strides=st, q_out_strides=st),
          "k": dict(Hk=H, k=OK, k_out=OK, k_strides=st, k_out_strides=st)}[which]
    assert lib.bl_rope(ctypes.byref(_rope_args(**at, **kw)), None) == 1


@pytest.mark.parametrize("H,Hk,step_q,step_k,at", [
    (3, 2, 2, 1, 1),        # heads 0, 2, 4 and 1, 2
    (6, 2, 1, 3, 2),        # all and 2, 5
    (2, 3, 3, 2, 1),        # 0, 3 and 1, 3, 5
    (1, 6, 5, 1, 0), (3, 1, 2, 9, 4)])
def test_rope_refuses_heads_of_other_steps_that_meet(lib, H, Hk, step_q, step_k, at):
    """q takes every step_q-th of a tensor's six heads, k every step_k-th from `at`."""
    q, k = (1920, 384, 64 * step_q), (1920, 384, 64 * step_k)
    k_at = OK + 128 * at if at else OK + 2               # or one element behind q
    args = _rope_args(H=H, Hk=Hk, q=OK, q_out=OK, k=k_at, k_out=k_at, q_strides=q,
                      q_out_strides=q, k_strides=k, k_out_strides=k)
    assert lib.bl_rope(ctypes.byref(args), None) == 1


def test_rope_refuses_one_tensor_in_two_forms(lib):
    assert lib.bl_rope(ctypes.byref(_rope_args(q_out=2 * OK, k_out=2 * OK)), None) == 1


@pytest.mark.parametrize("kw", [dict(H=65535, Hk=0, d=65536), dict(H=30000, Hk=2768, d=65536)])
def test_rope_refuses_tokens_past_32_bits(lib, kw):
    H, Hk, d = kw["H"], kw["Hk"], kw["d"]
    q, k = (H * d, H * d, d), (max(Hk, 1) * d, max(Hk, 1) * d, d)
    args = _rope_args(B=1, n=1, q_strides=q, q_out_strides=q, k_strides=k, k_out_strides=k, **kw)
    assert lib.bl_rope(ctypes.byref(args), None) == 1


def test_rope_arguments_are_laid_out_as_the_struct():
    """The call packs bl_rope_args itself: the same bytes as the structure's."""
    v = (2, 5, 4, 2, 64, 32, 2, 30, 2, 0, 0, 1, 0, 1, 11, 12, 13, 14, *range(20, 32), 41, 10, 43)
    a = _rope_args(B=2, n=5, H=4, Hk=2, d=64, pairs=32, axes=2, sections=(30, 2, 0, 0), interleaved=1,
                   inverse=0, dtype=1, q=11, k=12, q_out=13, k_out=14, q_strides=(20, 21, 22),
                   k_strides=(23, 24, 25), q_out_strides=(26, 27, 28), k_out_strides=(29, 30, 31),
                   positions=41, positions_batch_stride=10, freqs=43)
    assert ops._ROPE_ARGS.pack(*v) == bytes(a)


def test_rope_takes_empty_batches(lib):
    assert lib.bl_rope(None, None) == 1
    assert lib.bl_rope(ctypes.byref(_rope_args(B=0)), None) == 0
    assert lib.bl_rope(ctypes.byref(_rope_args(n=0, q=None)), None) == 0


def test_attention_backward_from_8_bits_refuses(lib):
    s = _lib.make_shape(1, 256, 2, 1, 64, 128, 128)
    need = lib.bl_attn_bwd_act8_workspace_bytes(ctypes.byref(s))
    base = _lib.bwd_workspace_bytes(s)
    assert need >= base + 2 * 256 * 64 * (2 + 1 + 1)
    assert lib.bl_attn_bwd_act8_workspace_bytes(ctypes.byref(_lib.make_shape(
        1, 256, 2, 1, 96, 128, 128))) == 0

    def call(shape=s, q=None, k=None, v=None, o=OK, o8=None, g=OK, scale=0.125, ws=OK, size=need):
        q, k, v = (x if x is not None else _act8() for x in (q, k, v))
        return lib.bl_attn_bwd_act8(ctypes.byref(shape), ctypes.byref(q), ctypes.byref(k),
                                    ctypes.byref(v), o, None if o8 is None else ctypes.byref(o8), g,
                                    OK, scale, None, OK, OK, OK, ws, size, None)

    assert call(o=None) == 1                                  # no output at all
    assert call(o8=_act8()) == 1                              # both of them
    assert call(q=_act8(group=32)) == 1
    assert call(k=_act8(fmt=2)) == 1                          # another format than q's
    assert call(o=None, o8=_act8(fmt=2)) == 1
    assert call(v=_act8(codes=OK + 8)) == 1
    assert call(g=None) == 1 and call(g=OK + 4) == 1
    assert call(scale=0.0) == 1 and call(scale=float("nan")) == 1
    assert call(ws=None) == 4 and call(size=need - 1) == 4
    t = _lib.Shape.from_buffer_copy(s)
    t.q_strides[:] = (256 * 256, 256, 64, 1)
    assert call(shape=t) == 2                                 # strided
    assert lib.bl_attn_bwd_act8_workspace_bytes(ctypes.byref(t)) == 0


# --- torch calls ------------------------------------------------------------------

def test_cpu_tensors_and_types_are_refused():
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    for call in (lambda: ops.act_save(x), lambda: ops.rms_norm_fwd(x, None),
                 lambda: ops.rms_norm_fwd_8bit(x, None), lambda: ops.rms_norm_bwd(x, x, x, None),
                 lambda: ops.rope(x[None, None], None, x, ops.RopePlan(64, (8,), device="cpu"))):
        with pytest.raises(TypeError):
            call()


@pytest.mark.parametrize("kw", [
    dict(sections=()), dict(sections=(4, 0)), dict(sections=(1, 1, 1, 1, 1)), dict(sections=(40,)),
    dict(layout="pairs"), dict(theta=0.0), dict(theta=float("inf")), dict(freqs=[1.0]),
    dict(freqs=[float("nan")] * 8), dict(head_dim=1)])
def test_rope_plan_refuses(kw):
    a = dict(head_dim=64, sections=(8,), device="cpu")
    a.update(kw)
    with pytest.raises(ValueError):
        ops.RopePlan(**a)


def test_act8_checks_its_parts():
    codes = torch.zeros(2, 64, dtype=torch.int8)
    for bad in (lambda: ops.Act8(codes.to(torch.uint8), codes, 0, torch.bfloat16),
                lambda: ops.Act8(codes, codes, 16, torch.bfloat16),
                lambda: ops.Act8(codes, codes, 0, torch.int8),
                lambda: ops.Act8(codes, codes, 0, torch.bfloat16)):    # not on a GPU
        with pytest.raises((TypeError, ValueError)):
            bad()


def test_modules_refuse():
    with pytest.raises(ValueError):
        api.BLRMSNorm(0)
    with pytest.raises(ValueError):
        api.BLRMSNorm(16385)
    with pytest.raises(ValueError):
        api.BLRMSNorm(64, checkpoint="int4")
    with pytest.raises(ValueError):
        api.BLRMSNorm(64, checkpoint="int8", group=48)
    with pytest.raises(ValueError):
        api.BLAttention(checkpoint="bf16")
    with pytest.raises(ValueError):
        api.BLAttention(checkpoint_out=True)
    with pytest.raises(ValueError):
        api.BLAttention(checkpoint_in_forward=True)
    t = torch.zeros(1, 4, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):                       # positions without a rotary module
        api.BLAttention()(t, t, t, positions=torch.zeros(4, 1, dtype=torch.int32))
    with pytest.raises(ValueError):                       # and the other way round
        api.BLAttention(rotary=api.Rotary(64, (32,), device="cpu"))(t, t, t)
    with pytest.raises(ValueError):                       # neither a head nor all heads
        api.BLAttention(q_norm=api.BLRMSNorm(96))(t, t, t)
    with pytest.raises(ValueError):
        api.BLRMSNorm(32)(t)


# --- host arithmetic ----------------------------------------------------------------

def test_frequencies_in_fixed_point_are_exact():
    """round(f / (2 pi) 2^64) against 40-digit decimal arithmetic, and the angle it
    gives at far positions against fp64's."""
    from decimal import Decimal, getcontext
    getcontext().prec = 60
    pi = Decimal("3.14159265358979323846264338327950288419716939937510582")
    freqs = tuple(10000.0 ** (-j / 22) for j in range(22)) + (-0.5, 7.5, 0.0)
    for f, F in zip(freqs, ops._fixed_point_freqs(freqs)):
        want = int((Decimal(f) / (2 * pi) * 2 ** 64).to_integral_value()) % 2 ** 64
        assert F % 2 ** 64 == want
        for pos in (1, 131071, -1000003, 2 ** 31 - 1):
            turns = (pos * F) % 2 ** 64 / 2 ** 64
            exact = float((Decimal(pos) * Decimal(f) / (2 * pi)) % 1) % 1.0
            off = abs(turns - exact)
            assert min(off, 1 - off) < 2.0 ** -33


def test_row_strides():
    x = torch.zeros(4, 6, 32)
    assert ops.row_stride(x) == 32
    assert ops.row_stride(x[:, :, :16]) == 32
    assert ops.row_stride(x[:, :3]) is None            # two distances between rows
    assert ops.row_stride(x[:, 0]) == 6 * 32
    assert ops.row_stride(x.transpose(0, 1)) is None
    assert ops.row_stride(x.transpose(1, 2)) is None
    assert ops.row_stride(x[:1, :1].expand(4, 6, 32)) is None
    assert ops.row_stride(x[:, :, :1]) == 32
    assert ops.row_stride(x[2:2]) == 32


# --- replicas ------------------------------------------------------------------------

def test_rotary_replicas_keep_their_own_frequencies(monkeypatch):
    """Replicas of a module share its plan; each call, and the backward behind it, reads the
    frequencies of its own replica's buffer, whichever replica was called last."""
    read = []

    def turn(q, k, positions, plan, fixed, inverse=False):
        read.append((fixed, inverse))
        return q * 1, k * 1

    monkeypatch.setattr(ops, "rope_with", turn, raising=False)
    rot = api.Rotary(64, (32,), device="cpu")
    replicas = []
    for _ in range(2):
        r = rot._replicate_for_data_parallel()
        r._buffers["fixed"] = rot.fixed.clone()          # as a copy on a device of its own
        replicas.append(r)
    assert replicas[0].plan is replicas[1].plan
    own = rot.plan.fixed
    pos = torch.zeros(4, 1, dtype=torch.int32)
    outs = []
    for r in replicas:
        q = torch.zeros(1, 4, 2, 64, requires_grad=True)
        outs.append(r(q, q, pos)[0])
    for o in outs:
        o.sum().backward()
    assert rot.plan.fixed is own
    assert [i for _, i in read] == [False, False, True, True]
    for j, r in enumerate(replicas):
        assert read[j][0].data_ptr() == r.fixed.data_ptr() == read[2 + j][0].data_ptr()
