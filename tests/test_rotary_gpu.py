"""Rotary positions on the GPU against the rotation in 64 bits.

Tolerance: the kernel's angle is exact to 2^-32 of a turn plus the fp32
rounding of the half-turns (2^-24 of at most pi), cos and sin are fp32, and the
two products and their sum round at 2^-24 each: below 2^-21 of |a| + |b|, far
under the one rounding of the result, half a step: 2^-8 (bf16) or 2^-11 (fp16)
of the value, plus half of fp16's subnormal step 2^-24."""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

HALF = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}


def oracle(x, pos, R, interleaved, inverse, base=10000.0, magnitude=1.0, freq=None):
    """x [B, H, L, D] in 64 bits on the CPU, pos [B, L] of integers."""
    x = x.detach().double().cpu()
    i = torch.arange(R // 2, dtype=torch.float64)
    w = base ** (-2 * i / R) if freq is None else freq
    t = pos.cpu().double()[:, None, :, None] * w
    z = torch.polar(torch.tensor(float(magnitude), dtype=torch.float64), -t if inverse else t)
    y = x.clone()
    at = (slice(0, R, 2), slice(1, R, 2)) if interleaved else (slice(0, R // 2), slice(R // 2, R))
    r = torch.complex(x[..., at[0]], x[..., at[1]]) * z
    y[..., at[0]], y[..., at[1]] = r.real, r.imag
    return y


def check(got, x, pos, R, interleaved, inverse, **kw):
    want = oracle(x, pos, R, interleaved, inverse, **kw)
    xa = x.detach().double().cpu().abs()
    rows = (xa.pow(2).sum(-1, keepdim=True)).sqrt()  # bounds |a| + |b| up to sqrt(2)
    # float64 angles of the oracle itself: position * 2^-53 * a few
    tol = HALF[x.dtype] * want.abs() + 2.0 ** -21 * rows + 2.0 ** -25
    err = (got.double().cpu() - want).abs()
    assert (err <= tol).all(), float((err - tol).max())


def made(shape, dtype, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(dtype)


# every access width (8, 4, 2 and 1 elements), both pairings, parts of the head
DIMS = [(128, 128), (72, 72), (72, 36), (192, 64), (64, 2), (80, 80), (512, 512), (6, 6), (7, 4), (20, 12)]


@pytest.mark.parametrize("D,R", DIMS)
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_head_dims(cuda_lib, D, R, interleaved, dtype):
    plan = cuda_lib.rotary_plan(D, rotary_dim=R, interleaved=interleaved)
    q, k = made((2, 5, 37, D), dtype, 1), made((2, 2, 37, D), dtype, 2)
    pos = torch.arange(37).expand(2, 37) + 11
    for inverse in (False, True):
        oq, ok = cuda_lib.rotary(plan, q, k, offset=11, inverse=inverse)
        check(oq, q, pos, R, interleaved, inverse)
        check(ok, k, pos, R, interleaved, inverse)


@pytest.mark.parametrize("B,H,L", [(1, 1, 1), (32, 40, 1), (3, 7, 2), (1, 1, 1025), (1, 129, 3), (2, 64, 700)])
def test_sizes(cuda_lib, B, H, L):
    plan = cuda_lib.rotary_plan(128)
    x = made((B, H, L, 128), torch.bfloat16, 3)
    check(cuda_lib.rotary(plan, x), x, torch.arange(L).expand(B, L), 128, False, False)


@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("shape", ["L", "1L", "BL", "expanded", "rows apart"])
def test_positions(cuda_lib, dtype, shape):
    B, L = 3, 17
    plan = cuda_lib.rotary_plan(64)
    x = made((B, 4, L, 64), torch.float16, 4)
    pos = torch.randint(0, 1 << 30, (B, L), dtype=dtype, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    if shape in ("L", "1L", "expanded"):
        pos = pos[0] if shape == "L" else pos[:1]
        full = pos.reshape(1, L).expand(B, L)
        if shape == "expanded":
            pos = pos.expand(B, L)
    elif shape == "rows apart":
        wide = torch.zeros(B, 2 * L, dtype=dtype, device="cuda")
        wide[:, :L] = pos
        pos, full = wide[:, :L], pos
    else:
        full = pos
    # positions near 2^30: the oracle's doubles hold the angle to 2^30 * 2^-52
    # (radians, |w| <= 1 rounded twice) = 2^-22 of the row
    got = cuda_lib.rotary(plan, x, positions=pos)
    want = oracle(x, full, 64, False, False)
    rows = x.double().cpu().pow(2).sum(-1, keepdim=True).sqrt()
    tol = 2.0 ** -11 * want.abs() + (2.0 ** -21 + 2.0 ** -21) * rows + 2.0 ** -25
    assert ((got.double().cpu() - want).abs() <= tol).all()


def test_angles_wrap_exactly(cuda_lib):
    """Positions of both signs, at the far ends of 64 bits: angle of p + 2^40
    is the product's own modulus, checked with whole numbers."""
    plan = cuda_lib.rotary_plan(16)
    ps = [0, -1, 5, (1 << 40) + 3, -(1 << 40), (1 << 62), -(1 << 62) + 7]
    x = torch.zeros(1, 1, len(ps), 16, dtype=torch.float16, device="cuda")
    x[..., :8] = 1  # pairs (1, 0): the result is (cos, sin)
    got = cuda_lib.rotary(plan, x, positions=torch.tensor(ps, device="cuda"))
    for l, p in enumerate(ps):
        for i in range(8):
            t = (p * plan.turns[i]) % (1 << 64) / 2.0 ** 64 * 2 * math.pi
            for j, want in ((i, math.cos(t)), (8 + i, math.sin(t))):
                assert abs(float(got[0, 0, l, j]) - want) <= 2.0 ** -11 * abs(want) + 2.0 ** -21, (p, i)


@pytest.mark.parametrize("interleaved", [False, True])
def test_layouts(cuda_lib, interleaved):
    """Slices of a fused projection in, dense heads out, and the gradient the
    other way, into slices of a fused gradient; then in place on the slices."""
    B, L, Hq, Hkv, D = 2, 33, 6, 2, 72
    plan = cuda_lib.rotary_plan(D, rotary_dim=48, interleaved=interleaved)
    x = made((B, L, Hq + 2 * Hkv, D), torch.bfloat16, 6)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
    pos = torch.arange(L).expand(B, L)
    oq, ok = cuda_lib.rotary(plan, q, k)
    assert oq.is_contiguous() and ok.is_contiguous()
    check(oq, q, pos, 48, interleaved, False)
    check(ok, k, pos, 48, interleaved, False)
    dx = torch.full_like(x, 7.0)
    dq, dk = dx[:, :, :Hq].transpose(1, 2), dx[:, :, Hq:Hq + Hkv].transpose(1, 2)
    cuda_lib.rotary(plan, oq, ok, inverse=True, out_q=dq, out_k=dk)
    check(dq, oq, pos, 48, interleaved, True)
    check(dk, ok, pos, 48, interleaved, True)
    assert (dx[:, :, Hq + Hkv:] == 7.0).all()  # v's slice is not touched
    y = x.clone()
    yq, yk = y[:, :, :Hq].transpose(1, 2), y[:, :, Hq:Hq + Hkv].transpose(1, 2)
    cuda_lib.rotary(plan, yq, yk, out_q=yq, out_k=yk)
    assert torch.equal(yq, oq) and torch.equal(yk, ok)
    assert torch.equal(y[:, :, Hq + Hkv:], x[:, :, Hq + Hkv:])


def test_unaligned_views(cuda_lib):
    """Bases and pitches at odd elements take the narrow accesses."""
    plan = cuda_lib.rotary_plan(64)
    buf = made((2 * 3 * 9 * 68 + 4,), torch.float16, 7)
    for first, pitch in ((1, 67), (0, 67), (2, 66), (4, 68)):
        x = buf[first:first + 2 * 3 * 9 * pitch].view(2, 3, 9, pitch)[..., :64]
        check(cuda_lib.rotary(plan, x), x, torch.arange(9).expand(2, 9), 64, False, False)


@pytest.mark.parametrize("kw", [dict(scaling="yarn", factor=4.0, original_length=2048),
                                dict(scaling="linear", factor=2.0), dict(scaling="ntk", factor=4.0),
                                dict(scaling="banded", factor=8.0, original_length=2048)])
def test_scaled(cuda_lib, kw):
    plan = cuda_lib.rotary_plan(128, **kw)
    freq = torch.tensor([plan.turns[i] / 2.0 ** 64 * 2 * math.pi for i in range(64)], dtype=torch.float64)
    x = made((1, 2, 50, 128), torch.bfloat16, 8)
    check(cuda_lib.rotary(plan, x, offset=20000), x, (torch.arange(50) + 20000).expand(1, 50), 128, False, False,
          freq=freq, magnitude=plan.magnitude)


def test_nan_and_inf_stay_in_their_pair(cuda_lib):
    plan = cuda_lib.rotary_plan(64, rotary_dim=32)
    x = made((1, 1, 4, 64), torch.bfloat16, 9)
    y = cuda_lib.rotary(plan, x, offset=3)
    x2 = x.clone()
    x2[0, 0, 1, 5] = float("nan")
    x2[0, 0, 2, 40] = float("inf")  # a copied element
    y2 = cuda_lib.rotary(plan, x2, offset=3)
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[0, 0, 1, 5] = bad[0, 0, 1, 21] = bad[0, 0, 2, 40] = True
    assert torch.equal(y[~bad], y2[~bad])
    assert y2[0, 0, 1, 5].isnan() and y2[0, 0, 1, 21].isnan() and y2[0, 0, 2, 40].isinf()


def test_inverse_is_the_gradient(cuda_lib):
    """<R x, y> = <x, R' y>: both sides in 64 bits of the rounded outputs, so
    each differs from the exact product by its outputs' roundings, at most
    2^-11 of the sum of |values|."""
    plan = cuda_lib.rotary_plan(96, rotary_dim=64, scaling="yarn", factor=4.0, original_length=2048)
    x, y = made((2, 3, 21, 96), torch.float16, 10), made((2, 3, 21, 96), torch.float16, 11)
    a, b = cuda_lib.rotary(plan, x, offset=7), cuda_lib.rotary(plan, y, offset=7, inverse=True)
    lhs, rhs = (a.double() * y.double()), (x.double() * b.double())
    tol = 2.0 ** -11 * 1.01 * (lhs.abs().sum() + rhs.abs().sum()) + 1e-6
    assert (lhs.sum() - rhs.sum()).abs() <= tol


def test_streams_and_graphs(cuda_lib):
    plan = cuda_lib.rotary_plan(128)
    x = made((1, 8, 64, 128), torch.bfloat16, 12)
    pos = torch.arange(64, device="cuda")
    want = cuda_lib.rotary(plan, x, positions=pos)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out = torch.zeros_like(x)
    cuda_lib.rotary(plan, x, positions=pos, out_q=out, stream=side)
    side.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    out2 = torch.zeros_like(x)
    with torch.cuda.graph(g):
        cuda_lib.rotary(plan, x, positions=pos, out_q=out2)
    g.replay()
    assert torch.equal(out2, want)
    # a replay reads the positions and inputs as they are then
    pos += 5
    x.mul_(0.5)
    g.replay()
    assert torch.equal(out2, cuda_lib.rotary(plan, x, positions=pos))


def test_python_refusals_on_device(cuda_lib):
    plan = cuda_lib.rotary_plan(64)
    x = torch.zeros(2, 3, 8, 64, dtype=torch.bfloat16, device="cuda")
    bad = [dict(k=x[:1]), dict(k=x.half()), dict(positions=torch.zeros(8)), dict(positions=torch.zeros(8, device="cuda")),
           dict(positions=torch.zeros(7, dtype=torch.int64, device="cuda")), dict(out_q=x.float()), dict(out_k=x),
           dict(positions=torch.zeros(16, dtype=torch.int64, device="cuda")[::2]), dict(out_q=x[:1].expand(2, 3, 8, 64))]
    for kw in bad:
        with pytest.raises(cuda_lib.SdpaError) as ei:
            cuda_lib.rotary(plan, x, **kw)
        assert ei.value.status == 1, kw
    with pytest.raises(cuda_lib.SdpaError) as ei:
        cuda_lib.rotary(plan, x.float())
    assert ei.value.status == 2
    with pytest.raises(cuda_lib.SdpaError):
        cuda_lib.rotary(plan, torch.zeros(1, 1, 8, 128, dtype=torch.bfloat16, device="cuda")[..., ::2])


@pytest.mark.parametrize("order", ["BLH", "BHL", "BLH3", "BL3H", "LBH", "LBH3", "HBL", "LHB"])
@pytest.mark.parametrize("interleaved", [False, True])
def test_two_slices_of_one_array_in_every_layout(cuda_lib, order, interleaved):
    """q and k as slices of one projection in any order of its dimensions, in place in
    one call, and their gradient written into it: the same bits as from dense tensors,
    and nothing else is touched."""
    sizes = {"B": 3, "L": 29, "H": 5, "3": 3}
    D, R = 72, 40
    plan = cuda_lib.rotary_plan(D, rotary_dim=R, interleaved=interleaved)
    x = made(tuple(sizes[c] for c in order) + (D,), torch.bfloat16, 13)

    def parts(t):
        """q (and k, v): three of the five heads each, or q, k, v of every head."""
        if "3" in order:
            three = [t.select(order.index("3"), i) for i in range(3)]
            rest = order.replace("3", "")
        else:
            three = [t.narrow(order.index("H"), 0, 3), t.narrow(order.index("H"), 3, 1), t.narrow(order.index("H"), 4, 1)]
            rest = order
        return [p.permute(rest.index("B"), rest.index("H"), rest.index("L"), 3) for p in three]

    q, k, v = parts(x)
    want_q, want_k = cuda_lib.rotary(plan, q, k, offset=9)
    check(want_q, q, (torch.arange(29) + 9).expand(3, 29), R, interleaved, False)
    y = x.clone()
    yq, yk, yv = parts(y)
    cuda_lib.rotary(plan, yq, yk, offset=9, out_q=yq, out_k=yk)
    assert torch.equal(yq, want_q) and torch.equal(yk, want_k) and torch.equal(yv, v)
    z = torch.full_like(x, 7.0)
    zq, zk, zv = parts(z)
    cuda_lib.rotary(plan, want_q, want_k, offset=9, inverse=True, out_q=zq, out_k=zk)
    back_q, back_k = cuda_lib.rotary(plan, want_q, want_k, offset=9, inverse=True)
    assert torch.equal(zq, back_q) and torch.equal(zk, back_k) and (zv == 7.0).all()
