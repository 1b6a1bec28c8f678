"""Rotary positions: the plan's frequencies against the formulas in exact
arithmetic, and every refusal (CPU; no kernel is launched)."""
import ctypes
import math
from fractions import Fraction

import pytest

import scaled_dot_product_13_b200 as sdpa

TWO_PI = 6.283185307179586476925286766559


def _turns(plan):
    return [plan.turns[i] for i in range(plan.rotary_dim // 2)]


def _expected(R, base=10000.0, scaling="none", factor=1.0, orig=0, fast=None, slow=1.0):
    """Frequencies in turns per position, in double precision."""
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    got = []
    for i in range(R // 2):
        w = base ** (-2.0 * i / R)
        keep = 1.0
        if scaling == "linear":
            keep = 0.0
        elif scaling == "yarn":
            lo = max(math.floor(R * math.log(orig / ((fast or 32.0) * TWO_PI)) / (2 * math.log(base))), 0)
            hi = min(math.ceil(R * math.log(orig / (slow * TWO_PI)) / (2 * math.log(base))), R - 1)
            keep = 1 - min(max((i - lo) / max(hi - lo, 0.001), 0.0), 1.0)
        elif scaling == "banded":
            keep = min(max((orig * w / TWO_PI - slow) / ((fast or 4.0) - slow), 0.0), 1.0)
        got.append((w * keep + w / factor * (1 - keep)) / TWO_PI)
    return got


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=4.0),
    dict(scaling="ntk", factor=8.0), dict(scaling="yarn", factor=4.0, original_length=2048),
    dict(scaling="banded", factor=8.0, original_length=8192),
    dict(scaling="yarn", factor=2.0, original_length=4096, beta_fast=16.0, beta_slow=2.0),
])
@pytest.mark.parametrize("R", [4, 64, 72, 128, 512])
def test_plan_frequencies(R, kw):
    plan = sdpa.rotary_plan(512, rotary_dim=R, **kw)
    want = _expected(R, kw.get("base", 10000.0), kw.get("scaling", "none"), kw.get("factor", 1.0),
                     kw.get("original_length", 0), kw.get("beta_fast"), kw.get("beta_slow", 1.0))
    for t, w in zip(_turns(plan), want):
        # the oracle is in doubles: a few roundings of 2^-53, log and pow; the
        # plan holds the nearest multiple of 2^-64, at most 2^-65 away
        assert abs(t / 2.0 ** 64 - w) <= 64 * 2.0 ** -53 * w + 2.0 ** -65


def test_first_pair_is_exact_to_the_last_bit():
    # one radian per position, in turns: 1 / (2 pi), from 40 digits of pi
    pi = Fraction(3141592653589793238462643383279502884197, 10 ** 39)
    want = 1 / (2 * pi) * 2 ** 64
    assert abs(_turns(sdpa.rotary_plan(64))[0] - want) <= 2  # the long double's own 2^-64


def test_magnitude():
    assert sdpa.rotary_plan(64).magnitude == 1.0
    m = sdpa.rotary_plan(64, scaling="yarn", factor=4.0, original_length=2048).magnitude
    assert abs(m - (0.1 * math.log(4.0) + 1)) < 1e-7
    assert sdpa.rotary_plan(64, scaling="yarn", factor=4.0, original_length=2048, magnitude=1.0).magnitude == 1.0


@pytest.mark.parametrize("kw,words", [
    (dict(head_dim=0), "head_dim"), (dict(head_dim=514), "head_dim"),
    (dict(head_dim=64, rotary_dim=33), "rotary_dim"), (dict(head_dim=64, rotary_dim=66), "rotary_dim"),
    (dict(head_dim=64, rotary_dim=-2), "rotary_dim"), (dict(head_dim=64, rotary_dim=0), "rotary_dim"),
    (dict(head_dim=65), "rotary_dim"),
    (dict(head_dim=64, base=1.0), "base"), (dict(head_dim=64, base=float("nan")), "base"),
    (dict(head_dim=64, scaling="other"), "scaling"),
    (dict(head_dim=64, scaling="linear", factor=0.0), "factor"),
    (dict(head_dim=64, scaling="linear", factor=float("inf")), "factor"),
    (dict(head_dim=64, scaling="yarn", factor=2.0), "original_length"),
    (dict(head_dim=64, scaling="banded", factor=2.0, original_length=2048, beta_fast=1.0), "beta_fast"),
    (dict(head_dim=64, scaling="ntk", factor=2.0, rotary_dim=2), "ntk"),
    (dict(head_dim=64, magnitude=-1.0), "magnitude"),
])
def test_plan_refusals(kw, words):
    with pytest.raises(sdpa.SdpaError) as ei:
        sdpa.rotary_plan(**kw)
    assert ei.value.status == 1 and words in ei.value.message


def _call(plan=None, x=0x10000, out=0x900000, heads=2, xs=(512, 256, 64), os_=(512, 256, 64), count=1, B=2, L=4,
          pos=None, bits=0, pstride=0, inverse=0, dtype=0):
    lib = sdpa.load_library()
    plan = plan or sdpa.rotary_plan(64)
    t = (sdpa.RotaryTensor * 2)()
    t[0] = sdpa.RotaryTensor(x, out, heads, sdpa.Strides(*xs), sdpa.Strides(*os_))
    st = lib.sdpa_rotary(ctypes.byref(plan), t, count, B, L, pos, bits, pstride, 0, inverse, dtype, None)
    return st, lib.sdpa_last_error_message().decode()


@pytest.mark.parametrize("kw,status,words", [
    (dict(plan=sdpa.RotaryPlan()), 1, "not filled"),
    (dict(count=0), 1, "count"), (dict(count=3), 1, "count"), (dict(count=2), 1, "non-NULL"),
    (dict(x=None), 1, "non-NULL"), (dict(out=None), 1, "non-NULL"), (dict(x=0x10001), 1, "2-byte"),
    (dict(heads=0), 1, "heads"), (dict(B=0), 1, ">= 1"), (dict(L=0), 1, ">= 1"),
    (dict(inverse=2), 1, "inverse"), (dict(dtype=7), 2, "dtype"),
    (dict(pos=0x5000, bits=16), 1, "position_bits"), (dict(pos=None, bits=32), 1, "position_bits"),
    (dict(pos=0x5004, bits=64), 1, "aligned"), (dict(pos=0x5000, bits=64, pstride=-1), 1, "stride"),
    (dict(xs=(-512, 256, 64)), 1, "strides"),
    (dict(os_=(512, 256, 0)), 1, "apart"), (dict(os_=(256, 256, 64)), 1, "apart"), (dict(os_=(512, 256, 63)), 1, "apart"),
    (dict(out=0x10000 + 128), 1, "overlap"), (dict(out=0x10000, xs=(512, 64, 128)), 1, "overlap"),
    (dict(B=1 << 16, L=1 << 16), 2, "2^31"),
])
def test_call_refusals_before_any_cuda_call(kw, status, words):
    st, msg = _call(**kw)
    assert st == status and words in msg, (st, msg)


def test_python_checks():
    torch = pytest.importorskip("torch")
    plan = sdpa.rotary_plan(64)
    with pytest.raises(sdpa.SdpaError, match="CUDA tensor"):
        sdpa.rotary(plan, torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(sdpa.SdpaError, match="must be"):
        sdpa.rotary(plan, torch.zeros(2, 3, 64, dtype=torch.bfloat16))
    with pytest.raises(sdpa.SdpaError, match="rotary_plan"):
        sdpa.rotary(None, torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16))


# Two tensors of one call: (x, out, heads, x strides, out strides) each, in elements of 2
# bytes; B = 2, L = 4, D = 64.  FUSED: rows of 6 heads, [B][L][6][64]; HEADS: [B][6][L][64].
FUSED, HEADS, DENSE = (1536, 64, 384), (1536, 256, 64), (512, 256, 64)
X, Y, FAR, OUT = 0x100000, 0x200000, 0x300000, 0x400000


@pytest.mark.parametrize("first,second,refused", [
    ((X, OUT, 2, DENSE, DENSE), (Y, OUT, 2, DENSE, DENSE), True),                # the same output
    ((X, OUT, 2, DENSE, DENSE), (Y, OUT + 2048 - 16, 2, DENSE, DENSE), True),     # outputs meet by 8 elements
    ((X, OUT, 2, DENSE, DENSE), (Y, OUT + 2048, 2, DENSE, DENSE), False),         # one behind the other
    ((X, Y, 2, DENSE, DENSE), (Y, OUT, 2, DENSE, DENSE), True),                   # writes the other's input
    ((X, OUT, 2, DENSE, DENSE), (Y, X, 2, DENSE, DENSE), True),
    ((X, OUT, 2, DENSE, DENSE), (X, FAR, 2, DENSE, DENSE), False),                # one input twice
    ((X, X, 4, FUSED, FUSED), (X + 512, X + 512, 2, FUSED, FUSED), False),        # slices in place: heads 0-3, 4-5
    ((X, X, 4, FUSED, FUSED), (X + 384, X + 384, 2, FUSED, FUSED), True),         # heads 0-3, 3-4
    ((X, X, 4, FUSED, FUSED), (X + 640, X + 640, 2, FUSED, FUSED), True),         # heads 5-6: the next token's head 0
    ((X, X, 4, HEADS, HEADS), (X + 2048, X + 2048, 2, HEADS, HEADS), False),
    ((X, X, 4, HEADS, HEADS), (X + 1536, X + 1536, 2, HEADS, HEADS), True),
    ((X, OUT, 2, DENSE, FUSED), (Y, OUT + 256, 4, (1024, 256, 64), FUSED), False),
    ((X, OUT, 2, DENSE, FUSED), (Y, OUT + 256, 4, (1024, 256, 64), HEADS), True),  # layouts that cross
])
def test_tensors_of_a_call_kept_apart(first, second, refused):
    torch = pytest.importorskip("torch")
    if torch.cuda.is_available():
        pytest.skip("the addresses are made up: an accepted call must find no device")
    lib = sdpa.load_library()
    plan = sdpa.rotary_plan(64)
    t = (sdpa.RotaryTensor * 2)()
    for i, (x, out, heads, xs, os_) in enumerate((first, second)):
        t[i] = sdpa.RotaryTensor(x, out, heads, sdpa.Strides(*xs), sdpa.Strides(*os_))
    st = lib.sdpa_rotary(ctypes.byref(plan), t, 2, 2, 4, None, 0, 0, 0, 0, 0, None)
    msg = lib.sdpa_last_error_message().decode()
    if refused:
        assert st == 1 and "another tensor" in msg, (st, msg)
    else:  # past the checks, stopped by the missing device
        assert st not in (0, 1), (st, msg)


def _pair(first, second, B, L, D):
    """(status, message) of a call with two tensors, each x, out, heads, x's and out's strides."""
    lib = sdpa.load_library()
    plan = sdpa.rotary_plan(D)
    t = (sdpa.RotaryTensor * 2)()
    for i, (x, out, heads, xs, os_) in enumerate((first, second)):
        t[i] = sdpa.RotaryTensor(x, out, heads, sdpa.Strides(*xs), sdpa.Strides(*os_))
    st = lib.sdpa_rotary(ctypes.byref(plan), t, 2, B, L, None, 0, 0, 0, 0, 0, None)
    return st, lib.sdpa_last_error_message().decode()


def _no_device():
    if pytest.importorskip("torch").cuda.is_available():
        pytest.skip("the addresses are made up: an accepted call must find no device")


# batch, head and token strides of one head's element in an array of H heads
LAYOUTS = {"BLH": lambda B, L, H, D: (L * H * D, D, H * D), "BHL": lambda B, L, H, D: (H * L * D, L * D, D),
           "BLH3": lambda B, L, H, D: (L * H * 3 * D, 3 * D, H * 3 * D), "BL3H": lambda B, L, H, D: (L * 3 * H * D, D, 3 * H * D),
           "LBH": lambda B, L, H, D: (H * D, D, B * H * D), "LBH3": lambda B, L, H, D: (H * 3 * D, 3 * D, B * H * 3 * D),
           "HBL": lambda B, L, H, D: (L * D, B * L * D, D), "LHB": lambda B, L, H, D: (D, B * D, H * B * D)}
STEP = {"BLH": lambda B, L, H, D: 2 * D, "BHL": lambda B, L, H, D: 2 * L * D, "BLH3": lambda B, L, H, D: D,
        "BL3H": lambda B, L, H, D: H * D, "LBH": lambda B, L, H, D: 2 * D, "LBH3": lambda B, L, H, D: D,
        "HBL": lambda B, L, H, D: 2 * B * L * D, "LHB": lambda B, L, H, D: 2 * B * D}  # from q to k


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("B,L", [(2, 4), (1, 7), (3, 1), (1, 1), (8, 4096)])
def test_slices_of_one_projection_in_place(layout, B, L):
    """q and k of one array, rotated in place in one call, in every order of its
    dimensions: accepted; one element nearer to each other: refused."""
    _no_device()
    H, D = 2, 64
    whole = 4 if layout in ("BLH", "BHL", "LBH", "HBL", "LHB") else H  # q's and k's heads next to each other
    s = LAYOUTS[layout](B, L, whole, D)
    k = X + 2 * STEP[layout](B, L, H, D)
    st, msg = _pair((X, X, H, s, s), (k, k, H, s, s), B, L, D)
    assert st not in (0, 1), (st, msg)
    st, msg = _pair((X, X, H, s, s), (k - 2, k - 2, H, s, s), B, L, D)
    assert st == 1 and "another tensor" in msg, (st, msg)
    # the gradient into it, from dense tensors elsewhere
    dense = LAYOUTS["BHL"](B, L, H, D)
    st, msg = _pair((X + (1 << 40), X, H, dense, s), (X + (1 << 41), k, H, dense, s), B, L, D)
    assert st not in (0, 1), (st, msg)


def test_views_against_their_elements():
    """Random views of small arrays: refused exactly when an element is shared."""
    import random

    _no_device()
    rng, seen = random.Random(1), {True: 0, False: 0}
    B, L, D = 2, 3, 4

    def elements(p, h, s):
        return {p // 2 + b * s[0] + i * s[1] + l * s[2] + d for b in range(B) for i in range(h) for l in range(L) for d in range(D)}

    def view(h):
        # nested in any order, with gaps, so that the elements of an output are apart
        s, span = [0, 0, 0], D
        for i in rng.sample(range(3), 3):
            s[i] = span + rng.choice([0, 0, 1, D, 2 * D, 5 * D])
            span = s[i] * ((B, h, L)[i] - 1) + span
        return tuple(s)

    for _ in range(4000):
        h0, h1 = rng.randint(1, 3), rng.randint(1, 3)
        s0 = view(h0)
        s1 = s0 if rng.random() < 0.5 and h0 == h1 else view(h1)
        at = X + 2 * rng.randint(-60, 60)
        far0, far1 = X + (1 << 30), X + (1 << 31)
        kind = rng.randint(0, 3)
        if kind == 0:    # both in place
            one, two = (X, X, h0, s0, s0), (at, at, h1, s1, s1)
        elif kind == 1:  # outputs near each other
            one, two = (far0, X, h0, s0, s0), (far1, at, h1, s1, s1)
        elif kind == 2:  # one writes near what the other reads
            one, two = (far0, X, h0, s0, s0), (at, far1, h1, s1, s1)
        else:            # only read near each other: always fine
            one, two = (X, far0, h0, s0, s0), (at, far1, h1, s1, s1)
        shared = kind != 3 and bool(elements(X, h0, s0) & elements(at, h1, s1))
        st, msg = _pair(one, two, B, L, D)
        assert (st == 1) == shared and st != 0, (kind, at - X, h0, s0, h1, s1, st, msg)
        seen[shared] += 1
        # a tensor's own output near its input
        if kind == 0 and (at != X or s0 != s1) and h0 == h1:
            st, msg = _pair((X, at, h0, s0, s1), (far0, far1, h1, s1, s1), B, L, D)
            assert (st == 1) == shared and st != 0, (at - X, h0, s0, s1, st, msg)
    assert min(seen.values()) > 300, seen


def test_strides_past_the_address_space():
    st, msg = _call(xs=(1 << 40, 256, 64), B=1 << 20, L=4)
    assert st == 1 and "2^48" in msg, (st, msg)
    st, msg = _call(os_=(1 << 20, 64, 1 << 40), B=2, L=1 << 29)
    assert st == 1 and "2^48" in msg, (st, msg)


def test_current_stream_without_torchs_private_function(monkeypatch):
    torch = pytest.importorskip("torch")
    device = torch.device("cuda", 1)
    monkeypatch.delattr(torch._C, "_cuda_getCurrentRawStream", raising=False)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d: type("S", (), {"cuda_stream": 77 if d == device else 0}))
    assert sdpa._call_stream(None, device) == 77
    assert sdpa._call_stream(5, device) == 5
