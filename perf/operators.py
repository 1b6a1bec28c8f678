"""The operators next to the attention forward pass, as they are measured: attention's backward pass and
rotary positions.

A case is a dict of plain values.  ``prepare`` makes what a training or serving step has in hand before the
call, ``run`` is one call: in elementary torch operations in 32 bits (``own = False``), or through this
package's public entry points (``own = True``).  ``exact`` is the same operator in 64 bits, from its
definition.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16}


# --------------------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------------------
def _backward(name, B, Hq, Hkv, L, S, Dqk, Dv, dtype, causal, window=0, offset=-1, sinks=False, dlse=False):
    c = dict(name=name) if name else {}
    c.update(op="backward", B=B, Hq=Hq, Hkv=Hkv, L=L, S=S, Dqk=Dqk, Dv=Dv, dtype=dtype, causal=causal,
             window=window, offset=offset, sinks=sinks, dlse=dlse)
    return c


def _rotary(name, B, Hq, Hkv, L, D, R, dtype, interleaved, scaling, base, factor, original, first, gradient):
    c = dict(name=name) if name else {}
    c.update(op="rotary", B=B, Hq=Hq, Hkv=Hkv, L=L, D=D, R=R, dtype=dtype, interleaved=interleaved,
             scaling=scaling, base=base, factor=factor, original=original, first=first, gradient=gradient)
    return c


def listed():
    return [
        # the smallest training step: the tiny causal GQA problem, where launches and latency are all there is
        _backward("bwd_tiny_d64", 1, 4, 2, 128, 128, 64, 64, "bf16", True),
        # fine-tuning an audio encoder's layer: 1500 tokens (not a multiple of any tile), head dim 64, no mask
        _backward("bwd_encoder_d64", 1, 20, 20, 1500, 1500, 64, 64, "bf16", False),
        # fine-tuning a vision encoder's layer with head dim 72 on a large image
        _backward("bwd_encoder_d72", 1, 16, 16, 4096, 4096, 72, 72, "bf16", False),
        # the ordinary step of a decoder layer: GQA 32/8, causal, two sequences
        _backward("bwd_causal_d128", 2, 32, 8, 4096, 4096, 128, 128, "bf16", True),
        # head dims 192/128, eight query heads on each key head, causal
        _backward("bwd_causal_d192_128", 1, 64, 8, 2048, 2048, 192, 128, "bf16", True),
        # a sliding-window layer, head dim 256
        _backward("bwd_window_d256", 1, 16, 8, 8192, 8192, 256, 256, "bf16", True, window=1024),
        # the full-attention layer next to it, at the same length
        _backward("bwd_causal_d256", 1, 16, 8, 8192, 8192, 256, 256, "bf16", True),
        # a short answer trained on behind a long, frozen context: 64 query rows over 16384 keys, fp16
        _backward("bwd_short_over_long", 1, 32, 8, 64, 16384, 128, 128, "f16", False),
        # a ragged chunk with sinks, its log-sum-exp merged with another chunk's (so that it has a gradient)
        _backward("bwd_ragged_sinks", 3, 24, 4, 777, 1201, 128, 128, "f16", True, offset=300, sinks=True, dlse=True),
        # one decoded token of 8 sequences, far into their contexts: q and k in one call
        _rotary("rope_decode", 8, 32, 8, 1, 128, 128, "f16", False, "none", 500000.0, 1.0, 0, 90000, False),
        # a prompt whose context was extended past the trained length; q and k are slices of one projection
        _rotary("rope_prompt", 1, 16, 8, 8192, 256, 256, "bf16", False, "yarn", 10000.0, 4.0, 2048, 0, False),
        # the gradient through the rotation of 64 of 192 dims in pairs of neighbours, ragged length
        _rotary("rope_grad_partial", 1, 64, 8, 4095, 192, 64, "bf16", True, "linear", 10000.0, 2.0, 0, 0, True),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.6:
        Dqk, Dv = rng.choice([(64, 64), (64, 64), (72, 72), (96, 96), (128, 128), (128, 128), (192, 128), (256, 256), (512, 512)])
        Hkv = rng.choice([1, 2, 4, 8, 20])
        g = rng.choice([1, 1, 2, 4, 8])
        B = rng.choice([1, 1, 2, 3])
        L = _spread(rng, 1, 8192)
        # 16 keys at least: a row that sees one key alone has no gradient but rounding
        S = max(L, 16) if rng.random() < 0.6 else _spread(rng, 16, 16384)
        causal = rng.random() < 0.6
        if causal and S < L:
            L, S = S, L
        # no dearer than the largest listed case, and scores that a plain form can hold
        most = min(1.0e8 if Dqk > 256 else 1.3e12 / (6 * Dqk + 4 * Dv), 1.0e9)
        while B * Hkv * g * L * S > most:
            if B > 1:
                B -= 1
            elif g > 1:
                g //= 2
            elif Hkv > 1:
                Hkv = (Hkv + 1) // 2
            else:
                L, S = (L + 1) // 2, max(16, S // 2)
        window = min(S, _spread(rng, 16, 2048)) if causal and rng.random() < 0.4 else 0
        offset = rng.randint(15, S - L) if causal and not window and S - L >= 15 and rng.random() < 0.5 else -1
        return _backward(None, B, Hkv * g, Hkv, L, S, Dqk, Dv, rng.choice(["bf16", "f16"]), causal, window, offset,
                         rng.random() < 0.3, rng.random() < 0.3)
    D = rng.choice([64, 72, 80, 96, 128, 192, 256])
    R = rng.choice([D, D, D // 2, D // 4 * 2])
    Hkv = rng.choice([1, 2, 4, 8, 20])
    Hq = Hkv * rng.choice([1, 2, 4, 8])
    B = rng.choice([1, 1, 2, 5, 8, 32])
    L = _spread(rng, 1, 8192)
    while B * L * (Hq + Hkv) * D > 5.5e7:
        B, L = (B // 2, L) if B > 1 else (B, L // 2)
    scaling = rng.choice(["none", "none", "linear", "ntk", "yarn", "banded"])
    return _rotary(None, B, Hq, Hkv, L, D, R, rng.choice(["bf16", "f16"]), rng.random() < 0.5, scaling,
                   rng.choice([10000.0, 500000.0, 1000000.0]), 1.0 if scaling == "none" else rng.choice([2.0, 4.0, 8.0]),
                   0 if scaling == "none" else rng.choice([2048, 8192]), _spread(rng, 1, 120000) - 1, rng.random() < 0.4)


# --------------------------------------------------------------------------------------------------------
# what a step has in hand
# --------------------------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(DEVICE).manual_seed(seed)
    dt = TYPES[case["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=g, device=DEVICE, dtype=torch.float32)

    if case["op"] == "rotary":
        B, Hq, Hkv, L, D = (case[n] for n in ("B", "Hq", "Hkv", "L", "D"))
        # each sequence at its own place
        start = torch.randint(0, 1000, (B, 1), generator=g, device=DEVICE) + case["first"]
        pos = start + torch.arange(L, device=DEVICE)
        if case["gradient"]:
            # what attention's backward pass writes; the result goes back to the projection's layout
            q, k = normal(B, Hq, L, D).to(dt), normal(B, Hkv, L, D).to(dt)
        else:
            # slices of one fused projection [B, L, (Hq + 2 Hkv) D], seen as [B, H, L, D]
            x = normal(B, L, Hq + 2 * Hkv, D).to(dt)
            q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        st = dict(case=case, q=q, k=k, pos=pos, plan=None)
        if own:
            import scaled_dot_product_13_b200 as sdpa

            st["plan"] = sdpa.rotary_plan(D, rotary_dim=case["R"], base=case["base"], interleaved=case["interleaved"],
                                          scaling=case["scaling"], factor=case["factor"],
                                          original_length=case["original"])
        return st
    B, Hq, Hkv, L, S, Dqk, Dv = (case[n] for n in ("B", "Hq", "Hkv", "L", "S", "Dqk", "Dv"))
    q, k, v = normal(B, Hq, L, Dqk).to(dt), normal(B, Hkv, S, Dqk).to(dt), normal(B, Hkv, S, Dv).to(dt)
    dout = (0.05 * normal(B, Hq, L, Dv)).to(dt)
    sinks = normal(Hq) if case["sinks"] else None
    dlse = 0.05 * normal(B, Hq, L) if case["dlse"] else None
    # the forward pass's output and log-sum-exp
    s = _scores(case, q, k)
    lse = torch.logsumexp(s, -1).view(B, Hq, L)
    if sinks is not None:
        lse = torch.logaddexp(lse, sinks.view(1, Hq, 1))
    s.sub_(lse.view(B, Hkv, -1, 1)).exp_()
    out = (s @ v.float()).view(B, Hq, L, Dv).to(dt)
    return dict(case=case, q=q, k=k, v=v, out=out, lse=lse.contiguous(), dout=dout, sinks=sinks, dlse=dlse)


def _visible(case):
    """[L, S] truth values: which keys a query row sees."""
    L, S = case["L"], case["S"]
    if not case["causal"]:
        return None
    at = torch.arange(L, device=DEVICE)[:, None] + (S - L if case["offset"] < 0 else case["offset"])
    key = torch.arange(S, device=DEVICE)[None, :]
    seen = key <= at
    return seen & (at - key < case["window"]) if case["window"] else seen


def _scores(case, q, k):
    """Scaled and masked scores [B, Hkv, g L, S], the rows of a KV head's query heads one after another."""
    B, Hq, Hkv, L, S = (case[n] for n in ("B", "Hq", "Hkv", "L", "S"))
    s = q.float().view(B, Hkv, -1, case["Dqk"]) @ k.float().transpose(2, 3)
    s.mul_(case["Dqk"] ** -0.5)
    seen = _visible(case)
    if seen is not None:
        s.view(B, Hkv, Hq // Hkv, L, S).masked_fill_(~seen, -math.inf)
    return s


# --------------------------------------------------------------------------------------------------------
# one pass
# --------------------------------------------------------------------------------------------------------
def run(state):
    return (_run_rotary if state["case"]["op"] == "rotary" else _run_backward)(state)


def _run_backward(st):
    case, q, k, v, out, lse, dout, sinks, dlse = (st[n] for n in ("case", "q", "k", "v", "out", "lse", "dout", "sinks", "dlse"))
    if own:
        import scaled_dot_product_13_b200 as sdpa

        dsinks = torch.empty_like(sinks) if sinks is not None else None
        dq, dk, dv = sdpa.backward(q, k, v, out, lse, dout, scale=case["Dqk"] ** -0.5, causal=case["causal"],
                                   window_size=case["window"], q_offset=None if case["offset"] < 0 else case["offset"],
                                   sinks=sinks, dlse=dlse, dsinks=dsinks)
        return {"dq": dq, "dk": dk, "dv": dv} if dsinks is None else {"dq": dq, "dk": dk, "dv": dv, "dsinks": dsinks}
    B, Hq, Hkv, L, Dqk, Dv = (case[n] for n in ("B", "Hq", "Hkv", "L", "Dqk", "Dv"))
    scale = Dqk ** -0.5
    do = dout.float()
    delta = (do * out.float()).sum(-1)  # [B, Hq, L]: sum over j of p dp
    if dlse is not None:
        delta -= dlse
    p = _scores(case, q, k).sub_(lse.view(B, Hkv, -1, 1)).exp_()
    do = do.view(B, Hkv, -1, Dv)
    dv = p.transpose(2, 3) @ do
    ds = (do @ v.float().transpose(2, 3)).sub_(delta.view(B, Hkv, -1, 1)).mul_(p)
    dq = (ds @ k.float()).mul_(scale).view(B, Hq, L, Dqk)
    dk = (ds.transpose(2, 3) @ q.float().view(B, Hkv, -1, Dqk)).mul_(scale)
    r = {"dq": dq.to(q.dtype), "dk": dk.to(q.dtype), "dv": dv.to(q.dtype)}
    if sinks is not None:
        # in 64 bits: a sum over all rows, of terms of both signs
        r["dsinks"] = -(torch.exp(sinks.view(1, Hq, 1).double() - lse) * delta).sum((0, 2)).float()
    return r


def _frequencies(case):
    """Radians per position of each rotated pair, [R / 2] in 64 bits, and the factor on cos and sin."""
    R, base, scaling, factor, original = (case[n] for n in ("R", "base", "scaling", "factor", "original"))
    i = torch.arange(R // 2, device=DEVICE, dtype=torch.float64)
    if scaling == "ntk":
        base = base * factor ** (R / (R - 2))
    f = base ** (-2 * i / R)
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        lo, hi = (R * math.log(original / (turns * 2 * math.pi)) / (2 * math.log(base)) for turns in (32.0, 1.0))
        lo, hi = max(math.floor(lo), 0), min(math.ceil(hi), R - 1)
        ramp = ((i - lo) / max(hi - lo, 1e-3)).clamp(0, 1)
        return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1
    if scaling == "banded":
        keep = ((original * f / (2 * math.pi) - 1) / 3).clamp(0, 1)  # all from 4 turns of the trained length on, none below one
        return f / factor * (1 - keep) + f * keep, 1.0
    return f, 1.0


def _run_rotary(st):
    case, q, k, pos = (st[n] for n in ("case", "q", "k", "pos"))
    inverse = case["gradient"]
    if own:
        import scaled_dot_product_13_b200 as sdpa

        if not inverse:
            return sdpa.rotary(st["plan"], q, k, positions=pos)
        # the gradient goes to the projection's layout [B, L, H, D]
        oq, ok = (torch.empty(x.shape[0], x.shape[2], x.shape[1], x.shape[3], dtype=x.dtype, device=DEVICE).transpose(1, 2) for x in (q, k))
        return sdpa.rotary(st["plan"], q, k, positions=pos, inverse=True, out_q=oq, out_k=ok)
    R = case["R"]
    f, m = _frequencies(case)
    angle = pos[:, None, :, None].double() * f  # 64 bits: far positions times fast pairs
    cos, sin = (torch.cos(angle) * m).float(), (torch.sin(angle) * m).float()
    if inverse:
        sin = -sin

    def turned(x):
        y = x.float()
        a, b = (y[..., 0:R:2], y[..., 1:R:2]) if case["interleaved"] else (y[..., :R // 2], y[..., R // 2:R])
        u, w = a * cos - b * sin, a * sin + b * cos
        head = torch.stack((u, w), -1).flatten(-2) if case["interleaved"] else torch.cat((u, w), -1)
        y = torch.cat((head, y[..., R:]), -1).to(x.dtype)
        return y.transpose(1, 2).contiguous().transpose(1, 2) if inverse else y.contiguous()

    return turned(q), turned(k)


# --------------------------------------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------------------------------------
def work(case):
    if case["op"] == "rotary":
        B, H, L, D, R = case["B"], case["Hq"] + case["Hkv"], case["L"], case["D"], case["R"]
        return {"bytes": 2 * 2 * B * H * L * D + 8 * B * L, "flops": 3 * B * H * L * R}
    B, Hq, Hkv, L, S, Dqk, Dv = (case[n] for n in ("B", "Hq", "Hkv", "L", "S", "Dqk", "Dv"))
    pairs = L * S
    if case["causal"]:
        first = S - L if case["offset"] < 0 else case["offset"]
        pairs = sum(min(first + i + 1, S) - (max(0, first + i + 1 - case["window"]) if case["window"] else 0) for i in range(L))
    rows, keys = B * Hq * L, B * Hkv * S
    # q, dq, out, dout; k, dk, v, dv; lse (and its gradient)
    nbytes = 2 * rows * (2 * Dqk + 2 * Dv) + 2 * keys * (2 * Dqk + 2 * Dv) + 4 * rows * (2 if case["dlse"] else 1)
    # the products q k', do v', p' do, ds' q and ds k, over the pairs that the mask leaves
    return {"bytes": nbytes, "flops": 2 * B * Hq * pairs * (3 * Dqk + 2 * Dv)}


# --------------------------------------------------------------------------------------------------------
# 64 bits
# --------------------------------------------------------------------------------------------------------
def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(st)
    # from the definition, one query head at a time: the weights A = softmax(Z) anew, and with the output
    # that the forward pass gave, dZ = A (dA - dO O'), the sum of A dA over a row being dO O'
    B, Hq, Hkv, L, S, Dqk, Dv = (case[n] for n in ("B", "Hq", "Hkv", "L", "S", "Dqk", "Dv"))
    q, k, v, dout = (st[n].double() for n in ("q", "k", "v", "dout"))
    scale = 1 / math.sqrt(Dqk)
    dq, dk, dv = torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v)
    dsinks = torch.zeros(Hq, dtype=torch.float64, device=DEVICE) if case["sinks"] else None
    hidden = None
    if case["causal"]:
        shift = case["offset"] if case["offset"] >= 0 else S - L
        ahead = torch.arange(S, device=DEVICE) - torch.arange(L, device=DEVICE).unsqueeze(1) - shift  # key's position less the query's
        hidden = ahead > 0
        if case["window"]:
            hidden |= ahead <= -case["window"]
    for b in range(B):
        for h in range(Hq):
            kv = h * Hkv // Hq
            z = torch.einsum("id,jd->ij", q[b, h], k[b, kv]) * scale
            if hidden is not None:
                z[hidden] = -math.inf
            top = z.max(1, keepdim=True).values
            if case["sinks"]:
                top = torch.maximum(top, st["sinks"][h].double())
            z = (z - top).exp_()
            total = z.sum(1, keepdim=True)
            if case["sinks"]:
                rest = (st["sinks"][h].double() - top).exp()
                total = total + rest
            a = z.div_(total)
            da = torch.einsum("id,jd->ij", dout[b, h], v[b, kv])
            mean = (dout[b, h] * st["out"][b, h].double()).sum(1, keepdim=True)
            # d lse / d score is the weight itself
            if case["dlse"]:
                mean = mean - st["dlse"][b, h].double().unsqueeze(1)
            dv[b, kv] += torch.einsum("ij,id->jd", a, dout[b, h])
            dz = da.sub_(mean).mul_(a)
            dq[b, h] = torch.einsum("ij,jd->id", dz, k[b, kv]) * scale
            dk[b, kv] += torch.einsum("ij,id->jd", dz, q[b, h]) * scale
            if case["sinks"]:
                dsinks[h] -= (rest / total * mean).sum()
    return {"dq": dq, "dk": dk, "dv": dv} if dsinks is None else {"dq": dq, "dk": dk, "dv": dv, "dsinks": dsinks}


def _exact_rotary(st):
    case, pos = st["case"], st["pos"].double()
    R, n = case["R"], case["R"] // 2
    s, factor, original = case["scaling"], case["factor"], case["original"]
    gain, angles = 1.0, []
    if s == "yarn":
        def index(turns):  # of the pair that makes so many turns over the trained length
            return R / 2 * math.log(original / (2 * math.pi * turns)) / math.log(case["base"])

        left, right = max(math.floor(index(32)), 0), min(math.ceil(index(1)), R - 1)
        gain = 1 + math.log(factor) / 10
    for i in range(n):
        w = case["base"] ** (-i / n)
        if s == "linear":
            w /= factor
        elif s == "ntk":
            w = (case["base"] * factor ** (n / (n - 1))) ** (-i / n)
        elif s == "yarn":
            slow = min(max((i - left) / max(right - left, 0.001), 0.0), 1.0)
            w *= 1 - slow + slow / factor
        elif s == "banded":
            turns = original * w / (2 * math.pi)
            fast = min(max((turns - 1.0) / (4.0 - 1.0), 0.0), 1.0)
            w *= fast + (1 - fast) / factor
        angles.append(pos * w)
    turn = torch.polar(torch.full((1,), gain, dtype=torch.float64, device=DEVICE), torch.stack(angles, -1)[:, None])
    if case["gradient"]:
        turn = turn.conj()
    got = []
    for x in (st["q"].double(), st["k"].double()):
        y = x.clone()
        at = (slice(0, R, 2), slice(1, R, 2)) if case["interleaved"] else (slice(0, n), slice(n, R))
        z = torch.complex(x[..., at[0]], x[..., at[1]]) * turn
        y[..., at[0]], y[..., at[1]] = z.real, z.imag
        got.append(y)
    return tuple(got)
