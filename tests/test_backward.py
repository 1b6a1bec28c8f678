"""Backward pass on the CPU: the oracle's formula against differences and
autograd in 64 bits, and every refusal of the entry point (no kernel runs)."""
import ctypes

import pytest
import torch

import scaled_dot_product_13_b200 as sdpa
from tests import bwd_oracle as O

CASES = [dict(), dict(causal=True), dict(causal=True, window=3), dict(causal=True, offset=1, sinks=True),
         dict(sinks=True, dlse=True), dict(causal=True, dlse=True)]


def _exact(m, **kw):
    """The oracle's gradients with the unrounded out and lse."""
    out, lse = O.forward(m["q"], m["k"], m["v"], m["scale"], m["causal"], m["window"], m["offset"], m["sinks"])
    return O.gradients(**{**m, "out": out, "lse": lse})[0]


@pytest.mark.parametrize("kw", CASES)
def test_oracle_equals_autograd(kw):
    m = O.make(2, 4, 2, 6, 9, 16, 8, torch.float16, **kw)
    leaves = {n: m[n].double().requires_grad_() for n in ("q", "k", "v")}
    sinks = None if m["sinks"] is None else m["sinks"].double().requires_grad_()
    out, lse = O.forward(leaves["q"], leaves["k"], leaves["v"], m["scale"], m["causal"], m["window"], m["offset"], sinks)
    loss = (out * m["dout"].double()).sum()
    if m["dlse"] is not None:
        loss = loss + (lse * m["dlse"].double()).sum()
    loss.backward()
    got = _exact(m)
    for n in ("q", "k", "v"):
        assert (got["d" + n] - leaves[n].grad).abs().max() < 1e-12
    if sinks is not None:
        assert (got["dsinks"] - sinks.grad).abs().max() < 1e-12


@pytest.mark.parametrize("kw", CASES)
def test_oracle_against_differences(kw):
    """Central differences along random directions: third-order error h^2 |f'''|
    / 6 (f''' of order 10^2 here), plus 2^-52 |f| / h of rounding."""
    m = O.make(1, 4, 2, 5, 8, 8, 8, torch.float16, seed=3, **kw)
    got = _exact(m)
    gen = torch.Generator("cpu").manual_seed(9)
    h = 1e-4
    for name in ("q", "k", "v") + (("sinks",) if m["sinks"] is not None else ()):
        way = torch.randn(m[name].shape, generator=gen, dtype=torch.float64)

        def f(step):
            x = {n: m[n] if m[n] is None else m[n].double() for n in ("q", "k", "v", "sinks")}
            x[name] = x[name] + step * way
            out, lse = O.forward(x["q"], x["k"], x["v"], m["scale"], m["causal"], m["window"], m["offset"], x["sinks"])
            return (out * m["dout"].double()).sum() + (0 if m["dlse"] is None else (lse * m["dlse"].double()).sum())

        want = (f(h) - f(-h)) / (2 * h)
        assert abs(want - (got["d" + name] * way).sum()) < 1e-5


A = dict(q=0x100000, k=0x200000, v=0x300000, out=0x400000, lse=0x500000, dout=0x600000, dq=0x700000, dk=0x800000,
         dv=0x900000, B=1, Hq=4, Hkv=2, L=8, S=16, Dqk=64, Dv=64, scale=0.125, causal=0, window=0, dtype=0, opt=None,
         ws=None, wsb=0, stream=None)


def _call(**kw):
    lib = sdpa.load_library()
    a = {**A, **{k: v for k, v in kw.items() if k in A}}
    o = sdpa.BackwardOptions()
    for n, x in kw.items():
        if n not in A:
            setattr(o, n, x)
    a["opt"] = ctypes.byref(o)
    st = lib.sdpa_backward(*a.values())
    return st, lib.sdpa_last_error_message().decode()


@pytest.mark.parametrize("name", ["q", "k", "v", "out", "lse", "dout", "dq", "dk", "dv"])
def test_null_and_misaligned_pointers(name):
    st, msg = _call(**{name: None})
    assert st == 1 and "non-NULL" in msg
    st, msg = _call(**{name: A[name] + (2 if name == "lse" else 8)})
    assert st == 1 and "aligned" in msg


@pytest.mark.parametrize("kw,status,words", [
    (dict(B=0), 1, ">= 1"), (dict(L=0), 1, ">= 1"), (dict(S=0), 1, ">= 1"), (dict(Hq=3), 1, "multiple of Hkv"),
    (dict(Dqk=68), 2, "multiples of 8"), (dict(Dv=520), 2, "[8, 512]"), (dict(dtype=2), 2, "dtype"),
    (dict(causal=2), 1, "causal"), (dict(causal=1, L=17), 1, "L <= S"), (dict(window=4), 2, "causal"),
    (dict(causal=1, window=-1), 1, "window_size"), (dict(scale=float("nan")), 1, "scale"),
    (dict(causal=1, has_q_offset=1, q_offset=-1), 1, "q_offset"),
    (dict(causal=1, window=2, has_q_offset=1, q_offset=20), 1, "sees no key"),
    (dict(sinks=0x10002), 1, "4-byte"), (dict(dlse=0x10001), 1, "4-byte"), (dict(dsinks=0x10000), 1, "needs sinks"),
    (dict(dsinks=0x10002, sinks=0x20000), 1, "4-byte"),
    (dict(dq=A["q"]), 1, "overlap an input"), (dict(dk=A["k"] + 1024), 1, "overlap an input"),
    (dict(dv=A["dout"]), 1, "overlap an input"), (dict(dv=A["lse"] - 16), 1, "overlap an input"),
    (dict(dk=A["dv"]), 1, "overlap each other"), (dict(dsinks=A["dq"], sinks=0x20000), 1, "overlap each other"),
    (dict(dsinks=0x20000, sinks=0x20000), 1, "overlap an input"),
    (dict(ws=0x10004, wsb=1 << 20), 1, "workspace"),
])
def test_refusals_before_any_cuda_call(kw, status, words):
    st, msg = _call(**kw)
    assert st == status and words in msg, (st, msg)


def test_python_checks_name_the_tensor():
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(sdpa.SdpaError, match="CUDA tensor"):
        sdpa.backward(x, x, x, x, torch.zeros(1, 2, 8), x)
