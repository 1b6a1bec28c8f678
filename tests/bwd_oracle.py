"""Attention's gradient in 64 bits, and how far a kernel that rounds P, dS and
the results to 16 bits may be from it (test infrastructure).

``gradients`` is the formula, materialised.  ``bounds`` carries the roundings
through it, element by element, with u = half a step of the 16-bit type, e =
2^-24, and v = u where P and dS enter their products as one 16-bit value, u^2
where as two (the second holds what the first's rounding left, to u of it):

  scores   s = scale q.k: a sum of Dqk products in fp32, off by at most
           (Dqk + 4) e sum |q k| scale; lse is an fp32 input, its product with
           log2(e) and the exponential add 2^-22 (1 + |lse| + |s|): together
           dP/P <= es
  P        v, and (fp16) half a subnormal step of the scaled value, 2^-39
  dV       sum over rows of (v + es) P |dO| + 2^-39 |dO|, fp32 sums n e, one
           rounding u |dV| of the result (fp16: 2^-25 below its normal range)
  dP-delta two sums of Dv products: (Dv + 4) e (sum |dO V| + sum |dO O| + |dlse|)
  dS       P ((v + es) |dP - delta| + that), and (fp16) 2^-39 of the bound that
           its scale is taken from
  dQ, dK   those through the last product, its fp32 sums, one rounding
"""
import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
E = 2.0 ** -24


def visible(L, S, causal, window, offset):
    """[L, S]: which keys a row sees."""
    at = torch.arange(L)[:, None] + (S - L if offset is None else offset)
    key = torch.arange(S)[None, :]
    seen = torch.ones(L, S, dtype=torch.bool)
    if causal:
        seen &= key <= at
    if window:
        seen &= at - key < window
    return seen


def forward(q, k, v, scale, causal=False, window=0, offset=None, sinks=None):
    """(out, lse) in 64 bits."""
    q, k, v = (t.double() for t in (q, k, v))
    g = q.shape[1] // k.shape[1]
    s = scale * q @ k.repeat_interleave(g, 1).transpose(2, 3)
    s = s.masked_fill(~visible(q.shape[2], k.shape[2], causal, window, offset), -torch.inf)
    lse = torch.logsumexp(s, -1)
    if sinks is not None:
        lse = torch.logaddexp(lse, sinks.double()[None, :, None])
    return torch.exp(s - lse[..., None]) @ v.repeat_interleave(g, 1), lse


def gradients(q, k, v, out, lse, dout, scale, causal=False, window=0, offset=None, sinks=None, dlse=None, terms=1):
    """{"dq", "dk", "dv", "dsinks"} in 64 bits, and their bounds, given the
    forward pass's (rounded) out and lse."""
    dt = q.dtype
    u = U[dt]
    half = dt == torch.float16
    uv = u ** terms
    B, Hq, L, Dqk = q.shape
    Hkv, S, Dv = k.shape[1], k.shape[2], v.shape[3]
    g = Hq // Hkv
    q, k, v, out, lse, do = (t.double() for t in (q, k, v, out, lse, dout))
    dl = torch.zeros(B, Hq, L, dtype=torch.float64) if dlse is None else dlse.double()
    kk, vv = k.repeat_interleave(g, 1), v.repeat_interleave(g, 1)
    kT, vT = kk.transpose(2, 3), vv.transpose(2, 3)
    seen = visible(L, S, causal, window, offset) & (lse != -torch.inf)[..., None]
    s = scale * q @ kT
    p = torch.where(seen, torch.exp(s - lse[..., None]), 0.0)
    delta = (do * out).sum(-1) - dl
    t = do @ vT - delta[..., None]
    ds = torch.where(seen, p * t, 0.0)

    def shared(x):  # sum over the query heads of a KV head
        return x.view(B, Hkv, g, *x.shape[2:]).sum(2)

    got = {"dq": scale * ds @ kk, "dk": scale * shared(ds.transpose(2, 3) @ q), "dv": shared(p.transpose(2, 3) @ do)}
    if sinks is not None:
        w = torch.where(lse == -torch.inf, 0.0, torch.exp(sinks.double()[None, :, None] - lse))
        got["dsinks"] = -(w * delta).sum((0, 2))

    fl = torch.where(torch.isinf(lse), 0.0, lse.abs())[..., None]
    es = (Dqk + 4) * E * abs(scale) * (q.abs() @ kT.abs()) + 2.0 ** -22 * (1 + fl + s.abs())
    ep = torch.where(seen, p * (uv + es) + (2.0 ** -39 if half else 0.0), 0.0)
    et = (Dv + 4) * E * (do.abs() @ vT.abs() + (do * out).abs().sum(-1, keepdim=True) + dl.abs()[..., None])
    low = 2.0 ** -39 * (do.norm(dim=-1).amax() * (v.norm(dim=-1).amax() + out.norm(dim=-1).amax()) + dl.abs().amax()) if half else 0.0
    eds = torch.where(seen, p * ((uv + es) * t.abs() + et) * (1 + 2 * u) + low, 0.0)
    sub = 2.0 ** -25 if half else 0.0

    def final(name, err, size, n):  # through the last product
        return err + n * E * size + u * got[name].abs() + u * err + sub

    a = abs(scale)
    tol = {"dq": final("dq", a * eds @ kk.abs(), a * ds.abs() @ kk.abs(), S + 4),
           "dk": final("dk", a * shared(eds.transpose(2, 3) @ q.abs()), a * shared(ds.abs().transpose(2, 3) @ q.abs()), g * L + 4),
           "dv": final("dv", shared(ep.transpose(2, 3) @ do.abs()), shared(p.transpose(2, 3) @ do.abs()), g * L + 4)}
    if sinks is not None:
        # delta in fp32, its factor to 2^-21 (1 + |exponent|), summed in 64 bits
        ed = (Dv + 4) * E * ((do * out).abs().sum(-1) + dl.abs())
        ex = torch.where(lse == -torch.inf, 0.0, (sinks.double()[None, :, None] - lse).abs())
        tol["dsinks"] = (w * (ed + 2.0 ** -21 * (1 + ex) * delta.abs())).sum((0, 2)) + E * got["dsinks"].abs()
    return got, tol


def make(B, Hq, Hkv, L, S, Dqk, Dv, dtype, seed=0, causal=False, window=0, offset=None, sinks=False, dlse=False,
         scale=None, dout_scale=1.0, v_scale=1.0):
    """Inputs of one backward call on the CPU, from the seed alone."""
    gen = torch.Generator("cpu").manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float32)

    scale = Dqk ** -0.5 if scale is None else scale
    q, k, v = normal(B, Hq, L, Dqk).to(dtype), normal(B, Hkv, S, Dqk).to(dtype), (v_scale * normal(B, Hkv, S, Dv)).to(dtype)
    dout = (dout_scale * normal(B, Hq, L, Dv)).to(dtype)
    sk = normal(Hq) if sinks else None
    dl = dout_scale * normal(B, Hq, L) if dlse else None
    out, lse = forward(q, k, v, scale, causal, window, offset, sk)
    return dict(q=q, k=k, v=v, out=out.to(dtype), lse=lse.float(), dout=dout, scale=scale, causal=causal,
                window=window, offset=offset, sinks=sk, dlse=dl)
