"""Backward pass at the sizes of real layers, on the GPU: rows of dq and keys of dk and
dv picked from all over the problem, each against the 64-bit formula within the bounds
of tests/bwd_oracle.py; and shapes with very long block lists, compared in full.

A row of dq is the formula's for that row alone (its position as the query offset),
a key's dk and dv those of that key alone (the offset moved by the key), given the
out and lse of the whole."""
import pytest
import torch

from tests import bwd_oracle as O
from tests.test_backward_gpu import check

pytestmark = pytest.mark.gpu


# 32/8 heads at two sequences, 64/8 at head dims 192/128, head dim 256 full and windowed,
# the encoders' 64 and 72, head dim 512, a short answer behind a long context, a chunk
# in the middle of the keys
CASES = [(2, 32, 8, 4096, 4096, 128, 128, dict(causal=True)), (1, 64, 8, 2048, 2048, 192, 128, dict(causal=True)),
         (1, 16, 8, 8192, 8192, 256, 256, dict(causal=True, window=1024)), (1, 16, 8, 8192, 8192, 256, 256, dict(causal=True)),
         (1, 20, 20, 1500, 1500, 64, 64, {}), (1, 16, 16, 4096, 4096, 72, 72, {}), (1, 8, 8, 3000, 3000, 512, 512, dict(causal=True)),
         (1, 32, 8, 64, 16384, 128, 128, {}), (3, 24, 4, 777, 1201, 128, 128, dict(causal=True, offset=300)),
         (1, 8, 1, 65536, 128, 64, 64, {}), (1, 16, 4, 1, 60000, 128, 128, {})]


@pytest.mark.parametrize("B,Hq,Hkv,L,S,Dqk,Dv,mask", CASES)
def test_rows_and_keys_of_large_problems(cuda_lib, B, Hq, Hkv, L, S, Dqk, Dv, mask):
    gen = torch.Generator("cuda").manual_seed(30)
    g, scale = Hq // Hkv, Dqk ** -0.5
    causal, window = mask.get("causal", False), mask.get("window", 0)
    offset = mask.get("offset", S - L)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").bfloat16()

    q, k, v, dout = normal(B, Hq, L, Dqk), normal(B, Hkv, S, Dqk), normal(B, Hkv, S, Dv), normal(B, Hq, L, Dv)
    lse = torch.empty(B, Hq, L, device="cuda")
    kw = dict(scale=scale, causal=causal, window_size=window, q_offset=mask.get("offset"))
    out = cuda_lib.forward_ex(q, k, v, lse=lse, **kw)
    got = dict(zip(("dq", "dk", "dv"), cuda_lib.backward(q, k, v, out, lse, dout, **kw)))
    cuda_lib.device_status(clear=True)
    assert all(torch.isfinite(t).all() for t in got.values())
    pick = torch.Generator("cpu").manual_seed(31)

    def some(n, ends):
        return sorted(set(torch.randint(0, n, (6,), generator=pick).tolist() + [e for e in ends if 0 <= e < n]))

    def near(name, b, h, at, want, tol):
        err = (got[name][b, h, at].double().cpu() - want).abs()
        assert (err <= tol).all(), (name, b, h, at, float(err.max()), float((err - tol).max()))

    terms = 2 if B * Hq * L * S <= 1 << 20 else 1
    fixed = dict(scale=scale, causal=causal, window=window, terms=terms)
    slabs = {(0, 0), (B - 1, Hkv - 1), (B // 2, Hkv // 2)}
    for b, hk in slabs:
        heads = slice(hk * g, (hk + 1) * g)
        one = [t[b:b + 1, heads].cpu() for t in (q, out, lse, dout)]
        kk, vv = k[b:b + 1, hk:hk + 1].cpu(), v[b:b + 1, hk:hk + 1].cpu()
        for i in some(L, (0, 127, 128, L - 1)):
            row = [t[:, :, i:i + 1] for t in one]
            want, tol = O.gradients(row[0], kk, vv, row[1], row[2], row[3], offset=offset + i, **fixed)
            for h in range(g):
                near("dq", b, hk * g + h, i, want["dq"][0, h, 0], tol["dq"][0, h, 0])
        for j in some(S, (0, 127, 128, S - 1)):
            want, tol = O.gradients(one[0], kk[:, :, j:j + 1], vv[:, :, j:j + 1], *one[1:], offset=offset - j, **fixed)
            for n in ("dk", "dv"):
                near(n, b, hk, j, want[n][0, 0, 0], tol[n][0, 0, 0])


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("shape,kw", [
    ((1, 16, 4, 1, 20000, 128, 128), {}), ((8, 32, 8, 1, 3000, 128, 128), dict(sinks=True)), ((2, 8, 8, 1, 5000, 64, 64), dict(dlse=True)),
    ((1, 6, 2, 1, 9000, 256, 256), dict(causal=True)), ((1, 4, 2, 1, 4000, 512, 512), {}), ((1, 32, 8, 4, 4000, 128, 128), dict(causal=True)),
    ((1, 8, 1, 8192, 128, 64, 64), {}), ((1, 4, 1, 6000, 100, 192, 128), dict(sinks=True)),
    ((1, 8, 1, 2000, 2000, 64, 64), dict(causal=True, window=100)), ((1, 128, 1, 2, 4000, 64, 64), dict(causal=True, window=1500)),
    ((1, 96, 1, 33, 900, 80, 80), dict(causal=True))])
def test_long_block_lists_in_full(cuda_lib, dtype, shape, kw):
    """Single tokens and a few rows over many keys, many rows over few keys, and lists
    whose parts begin inside a head or behind many short ones."""
    check(cuda_lib, O.make(*shape, dtype, seed=32, **kw))
