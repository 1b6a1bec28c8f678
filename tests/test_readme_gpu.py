"""The README's Python runs as it is written, and its training step gives the
gradients of the whole step."""
import re
from pathlib import Path

import pytest
import torch

pytestmark = pytest.mark.gpu

README = Path(__file__).resolve().parents[1] / "README.md"


def test_the_code_of_the_readme(cuda_lib):
    code = re.search(r"Use from Python:\n\n((?:    .*\n|\n)+)", README.read_text()).group(1)
    code = "\n".join(line[4:] for line in code.splitlines())
    B, L, Hq, Hkv, D = 2, 120, 4, 2, 64
    gen = torch.Generator("cpu").manual_seed(40)
    x = torch.randn(B, L, Hq + 2 * Hkv, D, generator=gen).half()
    dout = torch.randn(B, Hq, L, D, generator=gen).half()
    names = dict(torch=torch, B=B, L=L, Hq=Hq, Hkv=Hkv, D=D, x=x.cuda(), dout=dout.cuda())
    names["q"], names["k"], names["v"] = (torch.randn(B, h, L, D, generator=gen).half().cuda() for h in (Hq, Hkv, Hkv))
    exec(code, names)
    cuda_lib.device_status()
    leaf = x.double().requires_grad_()
    angle = torch.arange(L).double()[:, None] * 10000.0 ** (-2 * torch.arange(D // 2, dtype=torch.float64) / D)

    def turn(t):
        a, b = t[..., :D // 2], t[..., D // 2:]
        return torch.cat((a * angle.cos() - b * angle.sin(), a * angle.sin() + b * angle.cos()), -1)

    h = leaf.transpose(1, 2)
    q, k, v = turn(h[:, :Hq]), turn(h[:, Hq:Hq + Hkv]), h[:, Hq + Hkv:]
    s = q @ k.repeat_interleave(2, 1).transpose(2, 3) * D ** -0.5
    s = s.masked_fill(~torch.ones(L, L, dtype=torch.bool).tril(), -torch.inf)
    ((s.softmax(-1) @ v.repeat_interleave(2, 1)) * dout.double()).sum().backward()
    # in the 2-norm: q, k, v, out, P, dS, the gradients and the result round once each,
    # independently, at most 2^-11 each: below 8 of those all together
    err = (names["dx"].double().cpu() - leaf.grad).norm() / leaf.grad.norm()
    assert err <= 8 * 2.0 ** -11
