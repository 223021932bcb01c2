"""CPU checks of the experts' products: argument validation through the C ABI (every call here
fails validation or has nothing to work on), the binding's and ExpertPath's refusals, and the
64-bit plain forms that the GPU tests compare with (their gradients against autograd and
against differences, their bounds against planted mistakes)."""
import ctypes
import os

import pytest
import torch

import combine_ep_get_03_amd as ep
import plain_experts as X
import plain_ops as PL
from combine_ep_get_03_amd import _binding, pipeline

P = ctypes.c_void_p
A16 = P(0x10000)  # an aligned, non-NULL stand-in (never dereferenced)
A8 = P(0x10008)
MIS = P(0x10002)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(_binding.LIB_PATH):
        import __graft_entry__

        __graft_entry__.build()
    return ep.load()


def call(lib, name, sizes, args):
    """sizes: E, rows, H, I; args: pointers by name, in the order of the C call."""
    E, n, H, I = (sizes[s] for s in ("E", "n", "H", "I"))
    a = args
    return {
        "gate_up": lambda: lib.ep_expert_gate_up(a["x"], a["w"], a["off"], E, n, H, I, a["act"],
                                                 a["gu"], a["c"], a["s"], a["err"], None),
        "gate_up_fp8": lambda: lib.ep_expert_gate_up_fp8(a["x"], a["xs"], a["w"], a["ws"], a["off"],
                                                         E, n, H, I, a["c"], a["s"], a["err"], None),
        "down": lambda: lib.ep_expert_down(a["x"], a["w"], a["off"], E, n, H, I, a["out"], a["err"],
                                           None),
        "down_fp8": lambda: lib.ep_expert_down_fp8(a["x"], a["xs"], a["w"], a["ws"], a["off"], E, n,
                                                   H, I, a["out"], a["err"], None),
        "down_grad": lambda: lib.ep_expert_down_grad(a["x"], a["w"], a["off"], E, n, H, I, a["gu"],
                                                     a["c"], a["s"], a["out"], a["act"], a["err"],
                                                     None),
        "gate_up_grad": lambda: lib.ep_expert_gate_up_grad(a["x"], a["w"], a["off"], E, n, H, I,
                                                           a["out"], a["err"], None),
        "weight_grad": lambda: lib.ep_expert_weight_grad(a["x"], a["w"], a["off"], E, n, H, I,
                                                         a["out"], 0, 0, a["err"], None),
    }[name]()


# required pointers, nullable ones, pointers to 16 bytes, to 4 bytes, multiple of the widths
CALLS = {
    "gate_up": (("x", "w", "off", "act"), ("gu", "err"), ("x", "w", "act", "gu", "c"),
                ("off", "s", "err"), 8),
    "gate_up_fp8": (("x", "xs", "w", "ws", "off", "c", "s"), ("err",), ("x", "w", "c"),
                    ("xs", "ws", "off", "s", "err"), 128),
    "down": (("x", "w", "off", "out"), ("err",), ("x", "w", "out"), ("off", "err"), 8),
    "down_fp8": (("x", "xs", "w", "ws", "off", "out"), ("err",), ("x", "w", "out"),
                 ("xs", "ws", "off", "err"), 128),
    "down_grad": (("x", "w", "off", "out"), ("act", "err"), ("x", "w", "c", "out", "act"),
                  ("off", "s", "err"), 8),
    "gate_up_grad": (("x", "w", "off", "out"), ("err",), ("x", "w", "out"), ("off", "err"), 8),
    "weight_grad": (("x", "w", "off", "out"), ("err",), ("x", "w", "out"), ("off", "err"), 8),
}
NAMES = ("x", "xs", "w", "ws", "off", "act", "gu", "c", "s", "out", "err")


def good(name):
    args = {n: A16 for n in NAMES}
    if name == "down_grad":
        args["gu"] = None  # kept in e4m3
    return dict(E=4, n=64, H=256, I=128), args


@pytest.mark.parametrize("name", CALLS)
def test_refusals(lib, name):
    required, _, rows, words, unit = CALLS[name]
    sizes, args = good(name)
    for bad in (dict(E=0), dict(E=-1), dict(E=8193), dict(n=-1), dict(n=2**31), dict(H=0),
                dict(I=0), dict(H=-8), dict(H=2**22), dict(I=2**22),
                dict(n=2**31 - 1, H=2**20, I=2**19)):  # more tiles than 32 bits number
        assert call(lib, name, {**sizes, **bad}, args) == ep.EP_ERR_ARG, bad
    for bad in (dict(H=256 + unit // 2), dict(I=128 + unit // 2)):
        assert call(lib, name, {**sizes, **bad}, args) == ep.EP_ERR_ALIGN, bad
    for n in required:
        assert call(lib, name, sizes, {**args, n: None}) == ep.EP_ERR_ARG, n
    for n in rows:
        assert call(lib, name, sizes, {**args, n: A8}) == ep.EP_ERR_ALIGN, n
    for n in words:
        assert call(lib, name, sizes, {**args, n: MIS}) == ep.EP_ERR_ALIGN, n
    if name != "weight_grad":  # which writes its zeros
        assert call(lib, name, {**sizes, "n": 0}, args) == ep.EP_OK


def test_kept_forms_are_refused_in_part_or_together(lib):
    sizes, args = good("gate_up")
    assert call(lib, "gate_up", sizes, {**args, "c": None}) == ep.EP_ERR_ARG
    assert call(lib, "gate_up", sizes, {**args, "s": None}) == ep.EP_ERR_ARG
    assert call(lib, "gate_up", {**sizes, "I": 136}, args) == ep.EP_ERR_ALIGN  # e4m3: of 128
    sizes, args = good("down_grad")
    assert call(lib, "down_grad", sizes, {**args, "gu": A16}) == ep.EP_ERR_ARG  # both forms
    assert call(lib, "down_grad", sizes, {**args, "c": None, "s": None}) == ep.EP_ERR_ARG
    assert call(lib, "down_grad", sizes, {**args, "c": None}) == ep.EP_ERR_ARG
    assert call(lib, "down_grad", {**sizes, "I": 136}, args) == ep.EP_ERR_ALIGN


@pytest.mark.skipif(torch.cuda.is_available() or os.path.exists("/dev/kfd"),
                    reason="the stand-in pointers are only safe where no kernel can start")
@pytest.mark.parametrize("name", CALLS)
def test_a_launch_that_fails_is_reported(lib, name):
    """Without a GPU every launch fails: each call that gets past its checks says so, whatever
    the tile that its sizes take."""
    sizes, args = good(name)
    for kw in (dict(), dict(n=64, H=128, I=128), dict(E=1, n=1), dict(n=4 * 64, H=16384, I=8192),
               dict(n=4 * 2000, H=16384, I=8192), dict(E=8192, n=10)):
        assert call(lib, name, {**sizes, **kw}, args) == ep.EP_ERR_HIP, kw
    for n in CALLS[name][1]:
        assert call(lib, name, sizes, {**args, n: None}) == ep.EP_ERR_HIP, n


def b16(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def f32(*shape):
    return torch.zeros(shape, dtype=torch.float32)


def u8(*shape):
    return torch.zeros(shape, dtype=torch.uint8)


OFF = torch.zeros(3, dtype=torch.int32)
BINDING = {  # every call with tensors of the right shapes, on the host
    "ep_expert_gate_up": lambda **k: ep.ep_expert_gate_up(
        **{**dict(x=b16(4, 256), w_gate_up=b16(2, 256, 256), expert_offset=OFF, act=b16(4, 128)), **k}),
    "ep_expert_gate_up_fp8": lambda **k: ep.ep_expert_gate_up_fp8(
        **{**dict(x_fp8=u8(4, 256), x_scales=f32(4, 2), w_fp8=u8(2, 256, 256), w_scales=f32(2, 2, 2),
                  expert_offset=OFF, act_fp8=u8(4, 128), act_scales=f32(4, 1)), **k}),
    "ep_expert_down": lambda **k: ep.ep_expert_down(
        **{**dict(act=b16(4, 128), w_down=b16(2, 256, 128), expert_offset=OFF,
                  expert_out=b16(4, 256)), **k}),
    "ep_expert_down_fp8": lambda **k: ep.ep_expert_down_fp8(
        **{**dict(act_fp8=u8(4, 128), act_scales=f32(4, 1), w_fp8=u8(2, 256, 128),
                  w_scales=f32(2, 2, 1), expert_offset=OFF, expert_out=b16(4, 256)), **k}),
    "ep_expert_down_grad": lambda **k: ep.ep_expert_down_grad(
        **{**dict(grad_expert_out=b16(4, 256), w_down=b16(2, 256, 128), expert_offset=OFF,
                  grad_gate_up=b16(4, 256), gate_up=b16(4, 256)), **k}),
    "ep_expert_gate_up_grad": lambda **k: ep.ep_expert_gate_up_grad(
        **{**dict(grad_gate_up=b16(4, 256), w_gate_up=b16(2, 256, 256), expert_offset=OFF,
                  grad_x=b16(4, 256)), **k}),
    "ep_expert_weight_grad": lambda **k: ep.ep_expert_weight_grad(
        **{**dict(grad=b16(4, 256), input=b16(4, 128), expert_offset=OFF,
                  grad_weight=f32(2, 256, 128)), **k}),
}
FIRST = {"ep_expert_gate_up": "x", "ep_expert_gate_up_fp8": "x_fp8", "ep_expert_down": "act",
         "ep_expert_down_fp8": "act_fp8", "ep_expert_down_grad": "grad_expert_out",
         "ep_expert_gate_up_grad": "grad_gate_up", "ep_expert_weight_grad": "grad"}


@pytest.mark.parametrize("name", BINDING)
def test_binding_refuses_host_tensors_shapes_and_types(name):
    first = FIRST[name]
    with pytest.raises(ValueError, match="device tensor"):
        BINDING[name]()
    for bad in (None, 3.0, "x"):
        with pytest.raises((ValueError, TypeError), match=first):
            BINDING[name](**{first: bad})
    with pytest.raises(ValueError, match=f"{first}: expected 2 dimensions"):
        BINDING[name](**{first: b16(4)})
    third = {"ep_expert_gate_up": "w_gate_up", "ep_expert_gate_up_fp8": "w_fp8",
             "ep_expert_down": "w_down", "ep_expert_down_fp8": "w_fp8",
             "ep_expert_down_grad": "w_down", "ep_expert_gate_up_grad": "w_gate_up",
             "ep_expert_weight_grad": "grad_weight"}[name]
    with pytest.raises(ValueError, match=f"{third}: expected 3 dimensions"):
        BINDING[name](**{third: b16(4, 4)})
    with pytest.raises((ValueError, TypeError), match=third):
        BINDING[name](**{third: None})


def test_binding_refuses_odd_and_missing_forms():
    with pytest.raises(ValueError, match="gate's and up's"):
        BINDING["ep_expert_gate_up"](w_gate_up=b16(2, 255, 256))
    with pytest.raises(ValueError, match="gate's and up's"):
        BINDING["ep_expert_gate_up_grad"](grad_gate_up=b16(4, 255))
    with pytest.raises(ValueError, match="one of gate_up and gate_up_fp8"):
        BINDING["ep_expert_down_grad"](gate_up=None)
    with pytest.raises(ValueError, match="one of gate_up and gate_up_fp8"):
        BINDING["ep_expert_down_grad"](gate_up_fp8=u8(4, 256))


def test_expert_path_refuses_what_it_was_not_built_for(monkeypatch):
    seen = []
    for n in ("ep_expert_gate_up", "ep_expert_down", "ep_expert_down_grad", "ep_expert_gate_up_grad",
              "ep_expert_weight_grad", "ep_combine_unpermute_grad", "ep_expert_gate_up_fp8",
              "ep_expert_down_fp8"):
        monkeypatch.setattr(pipeline.B, n, lambda *a, _n=n, **k: seen.append(_n))
    make = pipeline.ExpertPath
    w = b16(2, 256, 128), b16(2, 128, 128)
    with pytest.raises(ValueError, match="built with inter"):
        make(4, 128, 2, 1, device="cpu").experts(*w)
    with pytest.raises(ValueError, match="built with inter"):
        make(4, 128, 2, 1, device="cpu", training=True).experts_grad(*w)
    with pytest.raises(ValueError, match="training=True"):
        make(4, 128, 2, 1, device="cpu", inter=128).experts_grad(*w)
    with pytest.raises(ValueError, match="bf16 rows"):
        make(4, 128, 2, 1, device="cpu", inter=128, training=True, fp8=True)
    with pytest.raises(ValueError, match="checkpoint"):
        make(4, 128, 2, 1, device="cpu", inter=128, checkpoint="int8")
    for kw in (dict(fp8=True), dict(training=True, checkpoint="fp8")):
        with pytest.raises(ValueError, match="multiple of 128"):
            make(4, 128, 2, 1, device="cpu", inter=136, **kw)
    p = make(4, 128, 2, 1, device="cpu", inter=136, training=True)
    with pytest.raises(ValueError, match="experts\\(\\) first"):
        p.experts_grad(*w)
    assert not seen
    p.experts(*w)
    p.experts_grad(*w)
    assert seen == ["ep_expert_gate_up", "ep_expert_down", "ep_expert_down_grad",
                    "ep_expert_gate_up_grad"]


# ------------------------------------------------------------------------ the plain forms

def case(seed=0):
    g = torch.Generator().manual_seed(seed)

    def r(*s):
        return torch.randn(s, generator=g, dtype=torch.float64)

    off = [0, 3, 3, 8]
    return off, r(8, 6), r(3, 8, 6), r(3, 6, 4), r(8, 6)  # H 6, I 4: x, w_gate_up, w_down, dout


def block(x, w, wd, off):
    _, _, act, _ = X.gate_up(x, w, off)
    return X.nt(act, wd, off)[0]


def test_plain_gradients_against_autograd_and_differences():
    off, x, w, wd, dout = case()
    for t in (x, w, wd):
        t.requires_grad_(True)
    out = torch.cat([(torch.nn.functional.silu(x[r] @ w[e, :4].T) * (x[r] @ w[e, 4:].T)) @ wd[e].T
                     for e, r in X.experts(off)])
    (out * dout).sum().backward()
    with torch.no_grad():
        gu, _, act, _ = X.gate_up(x, w, off)
        torch.testing.assert_close(block(x, w, wd, off), out, rtol=1e-12, atol=1e-12)
        dgu, _, again, _ = X.down_grad(dout, wd, gu, off)
        torch.testing.assert_close(again, act, rtol=1e-12, atol=1e-12)
        dx, _ = X.nn(dgu, w, off)
        dw, _ = X.weight_grad(dgu, x, off)
        dwd, _ = X.weight_grad(dout, act, off)
        for got, want in ((dx, x.grad), (dw, w.grad), (dwd, wd.grad)):
            torch.testing.assert_close(got, want, rtol=1e-11, atol=1e-11)
        assert bool((dw[1] == 0).all()) and bool((dwd[1] == 0).all())  # no rows
        step = 1e-5
        for t, grad in ((x, dx), (w, dw), (wd, dwd)):
            flat, g = t.view(-1), grad.reshape(-1)
            for i in range(0, flat.numel(), max(1, flat.numel() // 12)):
                keep = flat[i].item()
                flat[i] = keep + step
                up = (block(x, w, wd, off) * dout).sum()
                flat[i] = keep - step
                down = (block(x, w, wd, off) * dout).sum()
                flat[i] = keep
                diff = ((up - down) / (2 * step)).item()
                assert abs(diff - g[i].item()) <= 1e-6 * (1 + abs(diff))


def test_bounds_reject_a_planted_mistake():
    """Values off by a little more than a rounding fall outside, the rounded ones inside."""
    g = torch.Generator().manual_seed(3)
    off, H, I = [0, 40], 256, 128
    x = torch.randn((40, H), generator=g).to(torch.bfloat16).double()
    w = (torch.randn((1, 2 * I, H), generator=g) * H**-0.5).to(torch.bfloat16).double()
    gu, err, act, act_err = X.gate_up(x, w, off)
    X.assert_within(act.to(torch.bfloat16), act, X.rounded(act, act_err), "act")
    with pytest.raises(AssertionError):
        X.assert_within((act * 1.02).to(torch.bfloat16), act, X.rounded(act, act_err), "act")
    swapped = torch.cat([gu[:, I:], gu[:, :I]], dim=1).to(torch.bfloat16)
    with pytest.raises(AssertionError):
        X.assert_within(swapped, gu, X.rounded(gu, err), "gate_up")
    scale = PL.fp8_scales(gu)
    code = (gu / scale.repeat_interleave(128, dim=1)).float().to(torch.float8_e4m3fn)
    value = X.fp8_rows(code, scale)
    X.assert_within(value, gu, X.codes_bound(gu, err, scale), "codes")
    with pytest.raises(AssertionError):
        X.assert_within(value * 1.08, gu, X.codes_bound(gu, err, scale), "codes")


def split(lib, E=1, n=4096, M=256, N=128, out=A16, ws=A16, ws_bytes=None):
    need = ep.ep_expert_weight_grad_workspace_bytes(E, n, M, N)
    return lib.ep_expert_weight_grad_split(A16, A16, A16, E, n, M, N, out, 1, 0, None, ws,
                                           need if ws_bytes is None else ws_bytes, None)


def test_workspace_of_a_weight_gradient_in_pieces(lib):
    size = ep.ep_expert_weight_grad_workspace_bytes
    assert size(1, 4096, 256, 128) > 0
    # many tiles, few rows, no rows, sizes that are refused
    for E, n, M, N in ((32, 32768, 4096, 7168), (1, 511, 256, 128), (1, 0, 8, 8), (0, 4096, 8, 8),
                       (1, 4096, 12, 8), (1, -1, 8, 8), (1, 2**31, 8, 8), (1, 4096, 2**22, 8)):
        assert size(E, n, M, N) == 0, (E, n, M, N)
    for E in (1, 3, 64, 128):
        for n in (600, 4097, 10**6, 2**31 - 1):
            for M, N in ((8, 8), (136, 264), (1032, 1000), (2048, 2048)):
                one = M * N * 4  # whole pieces, one per expert at least
                assert size(E, n, M, N) % one == 0 and size(E, n, M, N) <= 64 << 20
                assert size(E, n, M, N) == 0 or size(E, n, M, N) >= E * one
    assert split(lib, ws=None) == ep.EP_ERR_CAPACITY
    assert split(lib, ws_bytes=size(1, 4096, 256, 128) - 1) == ep.EP_ERR_CAPACITY
    assert split(lib, ws=A8) == ep.EP_ERR_ALIGN
    assert split(lib, out=None) == ep.EP_ERR_ARG
    assert split(lib, n=-1) == ep.EP_ERR_ARG
