"""Backward pass on the GPU against the 64-bit formula, element by element
within the bounds that tests/bwd_oracle.py derives from the roundings."""
import pytest
import torch

from tests import bwd_oracle as O

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "f16": torch.float16}
TERMS = [1, 2]  # 16-bit terms of P and dS; 0, the choice by size, is 2 up to 2^20 pairs


def run(sdpa, m, terms=0, **kw):
    c = {n: (m[n].cuda() if m[n] is not None else None) for n in ("q", "k", "v", "out", "lse", "dout", "sinks", "dlse")}
    dsinks = torch.full_like(c["sinks"], float("nan")) if c["sinks"] is not None else None
    args = dict(scale=m["scale"], causal=m["causal"], window_size=m["window"], q_offset=m["offset"], sinks=c["sinks"],
                dlse=c["dlse"], dsinks=dsinks, weight_terms=terms)
    args.update(kw)
    dq, dk, dv = sdpa.backward(c["q"], c["k"], c["v"], c["out"], c["lse"], c["dout"], **args)
    got = {"dq": dq, "dk": dk, "dv": dv}
    if dsinks is not None:
        got["dsinks"] = dsinks
    return got


def check(sdpa, m, terms=0, **kw):
    got = run(sdpa, m, terms, **kw)
    sdpa.device_status(clear=True)
    pairs = m["q"].shape[0] * m["q"].shape[1] * m["q"].shape[2] * m["k"].shape[2]
    want, tol = O.gradients(**m, terms=terms or (2 if pairs <= 1 << 20 else 1))
    for n in want:
        err = (got[n].double().cpu() - want[n]).abs()
        assert torch.isfinite(got[n].float()).all(), n
        over = err - tol[n]
        assert (over <= 0).all(), f"{n}: {float(err.max()):.3e}, {float(over.max()):.3e} over its bound at {int(over.argmax())}"
        # a mistake in few elements hides under no large bound: in the 2-norm the
        # roundings, independent and at most u each, add up to less than 2 u
        if n != "dsinks" and want[n].norm() > 0 and m["q"].dtype == torch.bfloat16:
            assert err.norm() <= 2 * O.U[m["q"].dtype] * want[n].norm(), n
    return got


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("Dqk,Dv", [(64, 64), (72, 72), (128, 128), (192, 128), (256, 256), (8, 8), (16, 256), (512, 512), (320, 40), (104, 96), (192, 192), (128, 64)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_head_dims(cuda_lib, terms, Dqk, Dv, dtype):
    check(cuda_lib, O.make(2, 4, 2, 150, 150, Dqk, Dv, DT[dtype], seed=1, causal=True), terms)
    check(cuda_lib, O.make(1, 3, 1, 77, 201, Dqk, Dv, DT[dtype], seed=2), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("L,S", [(1, 1), (1, 2), (1, 64), (1, 1000), (2, 129), (31, 33), (64, 64), (65, 63), (127, 128), (128, 127),
                                 (129, 257), (300, 20), (383, 385), (600, 1)])
@pytest.mark.parametrize("g", [1, 5, 8])
def test_lengths(cuda_lib, terms, L, S, g):
    check(cuda_lib, O.make(2, 2 * g, 2, L, S, 64, 64, torch.bfloat16, seed=L + S), terms)
    if L <= S:
        check(cuda_lib, O.make(1, 2 * g, 2, L, S, 128, 128, torch.float16, seed=L + S, causal=True), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("window", [1, 2, 63, 64, 65, 128, 200, 1000])
@pytest.mark.parametrize("L,S,g", [(300, 300, 2), (33, 400, 4), (257, 700, 1)])
def test_windows(cuda_lib, terms, window, L, S, g):
    check(cuda_lib, O.make(1, 2 * g, 2, L, S, 64, 64, torch.bfloat16, seed=4, causal=True, window=window), terms)
    check(cuda_lib, O.make(1, 2 * g, 2, L, S, 192, 128, torch.float16, seed=5, causal=True, window=window), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("offset", [0, 1, 40, 200, 500])
@pytest.mark.parametrize("D", [64, 256, 512])
def test_query_offset(cuda_lib, terms, offset, D):
    m = O.make(1, 4, 2, 100, 300, D, D, torch.bfloat16, seed=6, causal=True, offset=offset)
    got = check(cuda_lib, m, terms)
    unseen = offset + 100
    if unseen < 300:  # keys behind the last row: exactly no gradient
        assert (got["dk"][:, :, unseen:] == 0).all() and (got["dv"][:, :, unseen:] == 0).all()
    check(cuda_lib, O.make(1, 4, 2, 100, 300, D, D, torch.float16, seed=7, causal=True, offset=min(offset, 250), window=60), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_sinks_and_lse_gradient(cuda_lib, terms, dtype):
    check(cuda_lib, O.make(2, 6, 2, 130, 190, 64, 64, DT[dtype], seed=8, causal=True, sinks=True), terms)
    check(cuda_lib, O.make(2, 6, 2, 130, 190, 128, 64, DT[dtype], seed=9, dlse=True), terms)
    check(cuda_lib, O.make(3, 6, 3, 1, 50, 64, 64, DT[dtype], seed=10, sinks=True, dlse=True), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("scale", [0.0, -0.2, 0.01, 1.0])
def test_scales(cuda_lib, terms, scale):
    check(cuda_lib, O.make(1, 4, 2, 90, 140, 64, 64, torch.bfloat16, seed=11, scale=scale, causal=True), terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("dout_scale,v_scale", [(2.0 ** -12, 1.0), (2.0 ** 6, 1.0), (1.0, 200.0), (2.0 ** -12, 200.0)])
def test_fp16_ranges(cuda_lib, terms, dout_scale, v_scale):
    """fp16's dS neither overflows nor drowns, whatever the gradient's scale
    (the results themselves must stay in fp16's range)."""
    check(cuda_lib, O.make(1, 4, 2, 96, 500, 64, 64, torch.float16, seed=12, dout_scale=dout_scale, v_scale=v_scale), terms)


@pytest.mark.parametrize("terms", TERMS)
def test_many_equal_keys_in_fp16(cuda_lib, terms):
    """Weights of 1/6000, below fp16's normal range without their scale."""
    m = O.make(1, 1, 1, 40, 6000, 64, 64, torch.float16, seed=13)
    m["q"] = m["q"] * 0
    out, lse = O.forward(m["q"], m["k"], m["v"], m["scale"])
    m["out"], m["lse"] = out.half(), lse.float()
    check(cuda_lib, m, terms)


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_rows_without_keys(cuda_lib, terms, D):
    """lse = -inf: the row takes no part, whatever its out and dout hold."""
    m = O.make(1, 4, 2, 140, 140, D, D, torch.bfloat16, seed=14, causal=True, sinks=True, dlse=True)
    m["lse"][0, 1, 5:40] = -torch.inf
    m["lse"][0, 3, 139] = -torch.inf
    got = check(cuda_lib, m, terms)
    assert (got["dq"][0, 1, 5:40] == 0).all() and (got["dq"][0, 3, 139] == 0).all()


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("Dqk,Dv", [(64, 64), (72, 72), (128, 128), (192, 128), (192, 192), (256, 256), (320, 512), (16, 256)])
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("fill", [float("nan"), float("inf"), None])
def test_nothing_of_a_row_without_keys_reaches_a_gradient(cuda_lib, terms, Dqk, Dv, dtype, fill):
    """Rows with lse = -inf (a padded batch): the largest finite numbers in their q and
    dout, and anything in their out and dlse, give the same bits as zeros there, in all
    gradients (the scores and dP overflow in bf16; fp16's scaling must not see them)."""
    most = torch.finfo(DT[dtype]).max
    for kw in (dict(causal=True, sinks=True, dlse=True), dict(dlse=True), dict(causal=True, window=50)):
        m = O.make(2, 4, 2, 141, 170, Dqk, Dv, DT[dtype], seed=24, **kw)
        dead = torch.zeros(2, 4, 141, dtype=torch.bool)
        dead[0, 1, 5:40] = dead[0, 3, 140] = dead[0, 2, 0] = True
        dead[1, :, 100:] = True  # the second sequence is shorter
        m["lse"][dead] = -torch.inf
        names = [n for n in ("q", "out", "dout", "dlse") if m[n] is not None]
        for n in names:
            m[n][dead] = 0
        clean = check(cuda_lib, m, terms)
        for n in names:
            m[n][dead] = most if n in ("q", "dout") or fill is None else fill
        m["q"][..., ::2] = torch.where(dead[..., None], -m["q"][..., ::2], m["q"][..., ::2])  # sums of both signs: inf - inf
        got = run(cuda_lib, m, terms)
        cuda_lib.device_status(clear=True)
        for n in clean:
            assert torch.equal(got[n], clean[n]), (n, kw)
        assert (got["dq"][dead.cuda()] == 0).all()


@pytest.mark.parametrize("D", [64, 128, 256, 512])
def test_a_slab_of_rows_without_keys(cuda_lib, D):
    """Every row of some query heads left out, and block lists cut into parts."""
    for shape in ((1, 4, 2, 140, 140, D, D), (1, 4, 1, 40, 5000, D, D)):
        m = O.make(*shape, torch.float16, seed=25)
        m["lse"][:, :2] = -torch.inf
        for n in ("q", "out", "dout"):
            m[n][:, :2] = 0
        clean = check(cuda_lib, m)
        for n, x in (("q", 65504.0), ("out", float("nan")), ("dout", -65504.0)):
            m[n][:, :2] = x
        got = run(cuda_lib, m)
        assert all(torch.equal(got[n], clean[n]) for n in clean)
        assert (got["dq"][:, :2] == 0).all()


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_a_log_sum_exp_of_infinity(cuda_lib, terms, dtype):
    """exp(s - inf) = 0 for every finite score: those rows' dq is 0, and the other
    gradients those of the other rows."""
    m = O.make(1, 4, 2, 100, 130, 64, 64, DT[dtype], seed=26)
    m["lse"][0, 1, 3:70] = torch.inf
    got = check(cuda_lib, m, terms)
    assert (got["dq"][0, 1, 3:70] == 0).all()


@pytest.mark.parametrize("terms", TERMS)
def test_not_a_number_stays_in_its_slab(cuda_lib, terms):
    m = O.make(2, 4, 2, 100, 130, 64, 64, torch.float16, seed=15)
    clean = run(cuda_lib, m, terms)
    m["dout"][0, 1, 50, 3] = float("nan")  # head 1 reads KV head 0
    m["v"][1, 1, 129, 0] = float("inf")
    got = run(cuda_lib, m, terms)
    for n, heads in (("dq", [(0, 2), (0, 3), (1, 0), (1, 1)]), ("dk", [(0, 1), (1, 0)]), ("dv", [(0, 1), (1, 0)])):
        for b, h in heads:
            assert torch.equal(got[n][b, h], clean[n][b, h]), n
    assert got["dq"][0, 1, 50].isnan().all()


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
@pytest.mark.parametrize("name,x", [("dout", float("nan")), ("dout", float("inf")), ("out", float("inf")), ("dlse", float("nan")), ("q", float("inf"))])
def test_a_row_that_is_not_finite_keeps_to_its_own_dq(cuda_lib, terms, dtype, name, x):
    """Its KV head's dk and dv are lost, but the other rows' dq are what they are without
    it: fp16's scaling, taken from the sizes of all rows, must not go with it (values at
    which an unscaled dS overflows)."""
    m = O.make(1, 4, 2, 150, 200, 64, 64, DT[dtype], seed=27, causal=True, dlse=True, dout_scale=64.0)
    if name == "dlse":
        m[name][0, 1, 77] = x
    else:
        m[name][0, 1, 77, 5] = x
    got = run(cuda_lib, m, terms)
    cuda_lib.device_status(clear=True)
    m[name][0, 1, 77] = 0
    want, tol = O.gradients(**m, terms=terms)
    keep = torch.ones(1, 4, 150, dtype=torch.bool)
    keep[0, 1, 77] = False
    err = (got["dq"].double().cpu() - want["dq"]).abs()[keep]
    assert (err <= tol["dq"][keep]).all(), float((err - tol["dq"][keep]).max())
    for n in ("dk", "dv"):  # the other KV head's
        assert ((got[n][:, 1].double().cpu() - want[n][:, 1]).abs() <= tol[n][:, 1]).all()


@pytest.mark.parametrize("terms", TERMS)
def test_future_values_that_are_not_numbers(cuda_lib, terms):
    """Keys that the causal mask hides from every row of a whole block do not
    reach it: their blocks are skipped."""
    m = O.make(1, 2, 2, 100, 400, 64, 64, torch.bfloat16, seed=16, causal=True, offset=0)
    clean = run(cuda_lib, m, terms)
    m["k"][:, :, 256:] = float("nan")
    m["v"][:, :, 256:] = float("inf")
    got = run(cuda_lib, m, terms)
    assert torch.equal(got["dq"], clean["dq"])
    assert torch.equal(got["dk"][:, :, :256], clean["dk"][:, :, :256]) and torch.equal(got["dv"][:, :, :256], clean["dv"][:, :, :256])


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("shape", [(2, 6, 2, 70, 90, 72, 72), (1, 8, 8, 64, 2000, 128, 128), (1, 2, 1, 300, 300, 256, 256), (1, 2, 1, 300, 300, 512, 512),
                                   (1, 2, 1, 20, 3000, 512, 320)])
def test_nothing_else_is_written(cuda_lib, terms, shape):
    """Guard bands around every output and the workspace; the workspace's old
    contents do not matter; a second call gives the same bits."""
    m = O.make(*shape, torch.float16, seed=17, sinks=True)
    pad, bufs, outs = 4096, {}, {}
    for n, like in (("dq", m["q"]), ("dk", m["k"]), ("dv", m["v"])):
        bufs[n] = torch.full((like.numel() + 2 * pad,), 1234.0, dtype=like.dtype, device="cuda")
        outs[n] = bufs[n][pad:pad + like.numel()].view(like.shape)
    B, Hq, Hkv, L, S, Dqk, Dv = shape
    need = cuda_lib.backward_workspace_bytes(B, Hq, Hkv, L, S, Dqk, Dv, dtype="f16", weight_terms=terms)
    ws = torch.full((need + 2 * pad,), 255, dtype=torch.uint8, device="cuda")
    first = {n: t.clone() for n, t in run(cuda_lib, m, terms, workspace=ws[pad:pad + need], **outs).items()}
    for n, b in bufs.items():
        assert (b[:pad] == 1234.0).all() and (b[-pad:] == 1234.0).all(), n
        assert torch.isfinite(outs[n].float()).all()
    assert (ws[:pad] == 255).all() and (ws[-pad:] == 255).all()
    ws.fill_(127)
    for t in outs.values():
        t.fill_(7)
    again = run(cuda_lib, m, terms, workspace=ws[pad:pad + need], **outs)
    for n in first:
        assert torch.equal(first[n], again[n]), n
    with pytest.raises(cuda_lib.SdpaError) as ei:
        run(cuda_lib, m, terms, workspace=ws[pad:pad + need - 16], **outs)
    assert ei.value.status == 3
    big = torch.zeros(need + 2 * m["q"].numel(), dtype=torch.uint8, device="cuda")
    over = big[:2 * m["q"].numel()].view(m["q"].dtype).view(m["q"].shape)
    with pytest.raises(cuda_lib.SdpaError) as ei:  # over an output
        run(cuda_lib, m, terms, workspace=big[:need], **dict(outs, dq=over))
    assert ei.value.status == 1 and "workspace" in ei.value.message


@pytest.mark.parametrize("terms", TERMS)
def test_streams_and_graphs(cuda_lib, terms):
    m = O.make(1, 8, 2, 200, 200, 128, 128, torch.bfloat16, seed=18, causal=True)
    want = run(cuda_lib, m, terms)
    c = {n: m[n].cuda() for n in ("q", "k", "v", "out", "lse", "dout")}
    args = [c[n] for n in ("q", "k", "v", "out", "lse", "dout")]
    kw = dict(scale=m["scale"], causal=True, weight_terms=terms)

    def empty():
        return {n: torch.zeros_like(t) for n, t in want.items()}

    torch.cuda.synchronize()
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    one, two = empty(), empty()
    torch.cuda.synchronize()
    cuda_lib.backward(*args, stream=side, **one, **kw)  # two calls at once
    cuda_lib.backward(*args, stream=other, **two, **kw)
    torch.cuda.synchronize()
    for got in (one, two):
        assert all(torch.equal(got[n], want[n]) for n in want)
    graphs = []
    for _ in range(2):  # two graphs, each with its own workspace
        g, got = torch.cuda.CUDAGraph(), empty()
        with torch.cuda.graph(g):
            cuda_lib.backward(*args, **got, **kw)
        graphs.append((g, got))
    for g, got in graphs + graphs:
        for t in got.values():
            t.zero_()
        g.replay()
        assert all(torch.equal(got[n], want[n]) for n in want)
    c["dout"].mul_(0.5)  # a replay reads the inputs as they are then
    graphs[0][0].replay()
    assert torch.equal(graphs[0][1]["dv"], want["dv"] * 0.5)


def test_terms_by_size(cuda_lib):
    """The choice by size: two terms up to 2^20 pairs, one above, and what each gives."""
    for L, chosen in ((512, 2), (513, 1)):  # 4 heads
        m = O.make(1, 4, 2, L, L, 64, 64, torch.bfloat16, seed=19, causal=True)
        auto, one, two = (run(cuda_lib, m, t) for t in (0, 1, 2))
        for n in auto:
            assert torch.equal(auto[n], (one, two)[chosen - 1][n])
            assert not torch.equal(one[n], two[n])


def test_two_terms_leave_one_rounding(cuda_lib):
    """With two terms each result is the nearest 16-bit value, but where the fp32
    sums before it are within their own error of a tie: 2^-10 of them here (sums
    of 300 terms, 2^-24 each, against a half step of 2^-9)."""
    m = O.make(1, 4, 2, 300, 300, 64, 64, torch.bfloat16, seed=21)
    got, want = run(cuda_lib, m, 2), O.gradients(**m)[0]
    for n in got:
        off = (got[n].cpu() != want[n].to(torch.bfloat16)).float().mean()
        assert off < 0.02, (n, float(off))


@pytest.mark.parametrize("shape", [(1, 8, 1, 600, 2000, 64, 64), (1, 4, 1, 40, 9000, 128, 128), (1, 16, 1, 700, 700, 192, 128),
                                   (1, 2, 1, 16, 6000, 256, 256), (1, 3, 1, 30, 5000, 512, 512), (1, 6, 1, 900, 130, 72, 72)])
@pytest.mark.parametrize("kind", ["full", "causal", "window"])
def test_split_block_lists(cuda_lib, shape, kind):
    """Few tiles with long block lists, which are cut into parts and joined; lists
    of very different lengths (causal, window), so that some tiles have one part."""
    if kind != "full" and shape[3] > shape[4]:
        pytest.skip("causal needs L <= S")
    kw = dict(full={}, causal=dict(causal=True), window=dict(causal=True, window=300))[kind]
    for dtype in (torch.bfloat16, torch.float16):
        check(cuda_lib, O.make(*shape, dtype, seed=22, **kw))


@pytest.mark.parametrize("terms", TERMS)
@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_keys_in_chunks(cuda_lib, terms, dtype):
    """The gradients of a chunk of the keys, from the out and lse over all of them:
    chunks whose values differ by a factor of 1000, in fp16 near its range."""
    m = O.make(1, 4, 2, 120, 400, 64, 64, DT[dtype], seed=23)
    m["v"][:, :, :150] *= 2.0 ** -10
    m["v"][:, :, 150:] *= 2.0 ** 5
    out, lse = O.forward(m["q"], m["k"], m["v"], m["scale"])
    m["out"], m["lse"] = out.to(DT[dtype]), lse.float()
    for lo, hi in ((0, 150), (150, 400)):
        c = dict(m, k=m["k"][:, :, lo:hi].contiguous(), v=m["v"][:, :, lo:hi].contiguous())
        got = run(cuda_lib, c, terms)
        want, tol = O.gradients(**c, terms=terms)
        for n in want:
            assert ((got[n].double().cpu() - want[n]).abs() <= tol[n]).all(), (n, lo)


def test_unknown_terms_are_refused(cuda_lib):
    m = O.make(1, 2, 2, 8, 8, 64, 64, torch.bfloat16)
    for t in (-1, 3):
        with pytest.raises(cuda_lib.SdpaError) as ei:
            run(cuda_lib, m, t)
        assert ei.value.status == 1


def test_python_refusals_on_device(cuda_lib):
    m = O.make(1, 4, 2, 16, 16, 64, 64, torch.bfloat16)
    c = {n: m[n].cuda() for n in ("q", "k", "v", "out", "lse", "dout")}
    bad = [dict(out=c["out"][:, :2]), dict(dout=c["dout"].half()), dict(lse=c["lse"].double()), dict(lse=None),
           dict(dout=c["dout"].transpose(1, 2).contiguous().transpose(1, 2)), dict(dq=c["k"].clone()), dict(dsinks=torch.zeros(4)),
           dict(dlse=torch.zeros(1, 4, 16)), dict(dq=c["q"]), dict(dsinks=torch.zeros(4, device="cuda"))]
    for kw in bad:
        with pytest.raises(cuda_lib.SdpaError) as ei:
            cuda_lib.backward(**{**c, **kw})
        assert ei.value.status == 1, kw


@pytest.mark.parametrize("dtype", ["bf16", "f16"])
def test_training_step_through_projection_rotation_and_attention(cuda_lib, dtype):
    """The operators together, as a step uses them: a fused projection, rotated
    into dense heads, attention with its log-sum-exp, and the way back into the
    projection's layout; each stage within its bounds given the stage before,
    and the whole against autograd in 64 bits."""
    dt = DT[dtype]
    B, L, Hq, Hkv, D = 2, 150, 4, 2, 64
    gen = torch.Generator("cpu").manual_seed(20)
    x = torch.randn(B, L, Hq + 2 * Hkv, D, generator=gen).to(dt)
    dout = torch.randn(B, Hq, L, D, generator=gen).to(dt)
    plan = cuda_lib.rotary_plan(D)
    xc = x.cuda()
    q, k = cuda_lib.rotary(plan, xc[:, :, :Hq].transpose(1, 2), xc[:, :, Hq:Hq + Hkv].transpose(1, 2), offset=100)
    v = xc[:, :, Hq + Hkv:].transpose(1, 2).contiguous()
    lse = torch.empty(B, Hq, L, device="cuda")
    out = cuda_lib.forward_ex(q, k, v, causal=True, lse=lse)
    dq, dk, dv = cuda_lib.backward(q, k, v, out, lse, dout.cuda(), causal=True)
    dx = torch.empty_like(xc)
    cuda_lib.rotary(plan, dq, dk, offset=100, inverse=True, out_q=dx[:, :, :Hq].transpose(1, 2),
                    out_k=dx[:, :, Hq:Hq + Hkv].transpose(1, 2))
    dx[:, :, Hq + Hkv:] = dv.transpose(1, 2)
    cuda_lib.device_status(clear=True)
    m = dict(q=q, k=k, v=v, out=out, lse=lse, dout=dout)
    want, tol = O.gradients(**{n: t.cpu() for n, t in m.items()}, scale=D ** -0.5, causal=True)
    for n, t in (("dq", dq), ("dk", dk), ("dv", dv)):
        assert ((t.double().cpu() - want[n]).abs() <= tol[n] * 1.0 + 2.0 ** -20).all(), n
    leaf = x.double().requires_grad_()
    i = torch.arange(D // 2, dtype=torch.float64)
    angle = (torch.arange(L) + 100).double()[:, None] * 10000.0 ** (-2 * i / D)

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    h = leaf.transpose(1, 2)
    o, _ = O.forward(turn(h[:, :Hq]), turn(h[:, Hq:Hq + Hkv]), h[:, Hq + Hkv:], D ** -0.5, causal=True)
    (o * dout.double()).sum().backward()
    # in the 2-norm: q, k, v, out, P, dS, the gradients and the result round
    # once each, independently: below 8 u all together
    err = (dx.double().cpu() - leaf.grad).norm() / leaf.grad.norm()
    assert err <= 8 * O.U[dt]
