"""What the rotary, linear-attention and single-token operators are measured on.

Cases are plain dicts; `prepare` makes a case's inputs on the GPU from a seed, `run` is one
pass (plain torch operations, or this repository's kernels when `own` is set), `exact` is the
same result from the definition in 64 bits and `work` the bytes and operations that a pass
cannot do without.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"bf16": 2, "f32": 4}


def listed():
    return [
        # q and k of the 256 x 256-pixel workload (6 heads of 64 channels) before attention
        dict(name="rotary-65536", op="rotary", B=1, H=6, N=65536, D=64, dtype="bf16", rot=64, first=0,
             interleaved=False, far=False, yarn=False, strided=False, train=False),
        # training step of a 128-channel model whose projections leave [B, N, H, D]: part of the
        # head rotated, interleaved pairs, forward and gradients
        dict(name="rotary-train-16384-d128", op="rotary", B=2, H=6, N=16384, D=128, dtype="bf16", rot=64, first=0,
             interleaved=True, far=False, yarn=False, strided=True, train=True),
        # one token for each of 64 requests, far into long contexts, scaled frequencies
        dict(name="rotary-decode-64", op="rotary", B=64, H=6, N=1, D=64, dtype="bf16", rot=64, first=0,
             interleaved=False, far=True, yarn=True, strided=True, train=False),
        # fp32, an odd length and an odd number of pairs
        dict(name="rotary-f32-odd", op="rotary", B=2, H=5, N=4099, D=64, dtype="f32", rot=46, first=8,
             interleaved=False, far=True, yarn=False, strided=False, train=False),
        # one layer's inference at 65536 tokens
        dict(name="linear-65536", op="linear", B=1, H=6, N=65536, D=64, dtype="bf16", ragged=False, carry=False,
             strided=False, train=False),
        # the same layer's training step
        dict(name="linear-train-65536", op="linear", B=1, H=6, N=65536, D=64, dtype="bf16", ragged=False, carry=False,
             strided=False, train=True),
        # the training step with 128-channel heads
        dict(name="linear-train-65536-d128", op="linear", B=1, H=6, N=65536, D=128, dtype="bf16", ragged=False,
             carry=False, strided=False, train=True),
        # a serving batch of prompts of unequal lengths, states carried in and out, [B, N, H, D] projections
        dict(name="linear-prompts-ragged", op="linear", B=8, H=16, N=1999, D=128, dtype="bf16", ragged=True,
             carry=True, strided=True, train=False),
        # one short prompt, where latency counts
        dict(name="linear-prompt-100", op="linear", B=1, H=6, N=100, D=64, dtype="bf16", ragged=False, carry=False,
             strided=False, train=False),
        # the small fp32 workload's training step, gradients through the carried state too
        dict(name="linear-train-f32-1024", op="linear", B=1, H=2, N=1024, D=64, dtype="f32", ragged=False, carry=True,
             strided=False, train=True),
        # one request's next token
        dict(name="step-1", op="step", B=1, H=6, D=64, dtype="bf16"),
        # a full decode batch over a pool of states
        dict(name="step-256-d128", op="step", B=256, H=16, D=128, dtype="bf16"),
    ]


def _log_uniform(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["rotary", "linear", "linear", "step"])
    D = rng.choice([64, 128])
    if op == "step":
        B, H = _log_uniform(rng, 1, 256), rng.randint(1, 16)
        return dict(op="step", B=B, H=H, D=D, dtype=rng.choice(["bf16", "bf16", "f32"]))
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    train = rng.random() < 0.5
    most = 65536 * 6 * 64 // (2 if train else 1) // (4 if op == "linear" and dtype == "f32" else 1)
    N = _log_uniform(rng, 1, 65536)
    H = rng.randint(1, max(1, min(24, most // (N * D))))
    B = min(64, _log_uniform(rng, 1, max(1, most // (N * H * D))))
    strided = rng.random() < 0.5
    if op == "rotary":
        rot = rng.choice([D, D // 2, 2 * rng.randint(1, D // 2)])
        first = rng.choice([0, D - rot, 2 * rng.randint(0, (D - rot) // 2)])
        return dict(op="rotary", B=B, H=H, N=N, D=D, dtype=dtype, rot=rot, first=first,
                    interleaved=rng.random() < 0.5, far=rng.random() < 0.5, yarn=rng.random() < 0.5, strided=strided,
                    train=train)
    return dict(op="linear", B=B, H=H, N=N, D=D, dtype=dtype, ragged=rng.random() < 0.5, carry=rng.random() < 0.5,
                strided=strided, train=train)


# ---------------------------------------------------------------------------- inputs


def _frequencies(case):
    """Radians per position of each pair (64 bits), and the factor of the rotated channels."""
    n = case["rot"] // 2
    f = 10000.0 ** (-torch.arange(n, dtype=torch.float64) / n)
    if not case["yarn"]:
        return f, 1.0
    # frequencies that turn less than once in the original context are divided by the factor,
    # those that turn more than 32 times are kept, the ones between are blended
    factor, original = 8.0, 8192
    turns = original * f / (2 * math.pi)
    keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0.0, 1.0)
    return f / factor * (1.0 - keep) + f * keep, 0.1 * math.log(factor) + 1.0


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev).manual_seed(int(seed) * 7919 + 11)
    B, H, D, dt = case["B"], case["H"], case["D"], DTYPES[case["dtype"]]

    def normal(*shape, dtype=dt):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    def tokens():
        if case.get("strided"):
            return normal(B, case["N"], H, D).transpose(1, 2)
        return normal(B, H, case["N"], D)

    st = dict(case=dict(case))
    if case["op"] == "rotary":
        st["q"], st["k"] = tokens(), tokens()
        f, st["scale"] = _frequencies(case)
        st["freq"] = f.to(dev)
        N = case["N"]
        if case["far"]:  # every request at its own place in a context of up to 2^20 tokens
            start = torch.randint(0, (1 << 20) - N, (B, 1), generator=g, device=dev)
            st["pos"] = start + torch.arange(N, device=dev)
        else:
            st["pos"] = torch.arange(N, device=dev)
        if case["train"]:
            st["q"].requires_grad_(), st["k"].requires_grad_()
            st["dq"], st["dk"] = normal(B, H, N, D), normal(B, H, N, D)
        return st
    # decays 1 - 2^-x, x between 2 and 10: memories of 4 to 1024 tokens
    x = 2.0 + 8.0 * torch.rand(H, generator=g, device=dev, dtype=torch.float64)
    st["log_decay"] = torch.log1p(-torch.exp2(-x)).float()
    if case["op"] == "step":
        st["q"], st["k"], st["v"] = normal(B, H, D), normal(B, H, D), normal(B, H, D)
        # a pool with room for two generations: each request's state is read from one slot and
        # written to another (the old one stays for a rejected token)
        st["pool"] = 4.0 * normal(2 * B, H, D, D, dtype=torch.float32)
        order = torch.randperm(2 * B, generator=g, device=dev).to(torch.int32)
        st["slots"], st["out_slots"] = order[:B].contiguous(), order[B:].contiguous()
        return st
    st["q"], st["k"], st["v"] = tokens(), tokens(), tokens()
    N = case["N"]
    st["lengths"] = None
    if case["ragged"]:
        st["lengths"] = torch.randint(0, N + 1, (B,), generator=g, device=dev).to(torch.int32)
    st["initial"] = 4.0 * normal(B, H, D, D, dtype=torch.float32) if case["carry"] else None
    if case["train"]:
        for n in ("q", "k", "v"):
            st[n].requires_grad_()
        st["do"] = normal(B, H, N, D)
        if case["carry"]:
            st["initial"].requires_grad_()
            st["dstate"] = normal(B, H, D, D, dtype=torch.float32)
    return st


# ---------------------------------------------------------------------------- plain forms


def _plain_rotary(x, pos, freq, case, scale):
    n, first = case["rot"] // 2, case["first"]
    angle = pos.double()[..., None] * freq
    if angle.dim() == 3:
        angle = angle[:, None]
    cos, sin = (angle.cos() * scale).float(), (angle.sin() * scale).float()
    xf = x.float()
    part = xf[..., first:first + 2 * n]
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :n], part[..., n:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((xf[..., :first], part, xf[..., first + 2 * n:]), -1).to(x.dtype)


def _plain_linear(q, k, v, log_decay, initial, lengths):
    B, H, N, D = q.shape
    C = 128
    M = -(-N // C)
    dev, scale, a = q.device, D ** -0.5, log_decay.double()
    pos = torch.arange(N, device=dev)
    length = torch.full((B,), N, device=dev) if lengths is None else lengths.long()
    live = (pos < length[:, None])[:, None, :, None]
    q, k, v = (torch.where(live, x.float(), 0.0) for x in (q, k, v))
    qc, kc, vc = (torch.nn.functional.pad(x, (0, 0, 0, M * C - N)).view(B, H, M, C, D) for x in (q, k, v))
    n, m = torch.arange(C, device=dev), torch.arange(M, device=dev)

    def decay(steps):  # e^(a steps) for each head, 0 where steps are negative
        return torch.where(steps >= 0, torch.exp(a.view(H, *[1] * steps.dim()) * steps.clamp(min=0)), 0.0).float()

    inside = (qc @ kc.transpose(-1, -2) * decay(n[:, None] - n)[:, None]) @ vc
    local = (kc * decay(C - 1 - n)[:, None, :, None]).transpose(-1, -2) @ vc
    start = (decay(C * (m[:, None] - 1 - m)) @ local.flatten(3)).view(B, H, M, D, D)
    if initial is not None:
        start = start + decay(C * m)[:, :, None, None] * initial[:, :, None]
    o = scale * (inside + (qc * decay(n + 1)[:, None, :, None]) @ start).view(B, H, M * C, D)[:, :, :N]
    left = length[:, None] - 1 - pos  # [B, N]
    final = (k * decay(left).transpose(0, 1)[..., None]).transpose(-1, -2) @ v
    if initial is not None:
        final = final + decay(length).t()[..., None, None] * initial
    return torch.where(live, o, 0.0), final


def _run_rotary(st):
    case, q, k = st["case"], st["q"], st["k"]
    if own:
        from log_linear_hierarchical_b200 import llsa_rotary
        q2, k2 = llsa_rotary(q, k, st["pos"], st["freq"], interleaved=case["interleaved"], first=case["first"],
                             scale=st["scale"])
    else:
        q2, k2 = (_plain_rotary(x, st["pos"], st["freq"], case, st["scale"]) for x in (q, k))
    if not case["train"]:
        return [q2, k2]
    return [q2.detach(), k2.detach(), *torch.autograd.grad([q2, k2], [q, k], [st["dq"], st["dk"]])]


def _run_linear(st):
    case, q, k, v, initial = st["case"], st["q"], st["k"], st["v"], st["initial"]
    if own:
        from log_linear_hierarchical_b200 import llsa_linear_attention
        o = llsa_linear_attention(q, k, v, st["log_decay"], initial_state=initial, lengths=st["lengths"],
                                  return_state=case["carry"])
        o, final = o if case["carry"] else (o, None)
    else:
        o, final = _plain_linear(q, k, v, st["log_decay"], initial, st["lengths"])
        o = o.to(q.dtype)
    if not case["train"]:
        return [o, final] if case["carry"] else [o]
    if not case["carry"]:
        return [o.detach(), *torch.autograd.grad([o], [q, k, v], [st["do"]])]
    return [o.detach(), final.detach(),
            *torch.autograd.grad([o, final], [q, k, v, initial], [st["do"], st["dstate"]])]


def _run_step(st):
    q, k, v, pool = st["q"], st["k"], st["v"], st["pool"]
    if own:
        from log_linear_hierarchical_b200 import llsa_linear_step
        o = llsa_linear_step(q, k, v, st["log_decay"], pool, slots=st["slots"], out_slots=st["out_slots"])
        return [o, pool]
    D = q.shape[-1]
    s = pool[st["slots"].long()] * torch.exp(st["log_decay"])[:, None, None]
    s = s + k.float()[..., :, None] * v.float()[..., None, :]
    pool[st["out_slots"].long()] = s
    o = (q.float()[..., :, None] * s).sum(-2) * D ** -0.5
    return [o.to(q.dtype), pool]


def run(state):
    op = state["case"]["op"]
    if op == "rotary":
        return _run_rotary(state)
    if op == "step":
        return _run_step(state)
    return _run_linear(state)


# ---------------------------------------------------------------------------- 64 bits


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rotary":
        return _exact_rotary(case, st)
    if case["op"] == "step":
        pool = st["pool"].double()
        o = torch.zeros(st["q"].shape, dtype=torch.float64, device=pool.device)
        lam = torch.exp(st["log_decay"].double())
        old = pool.clone()
        for b, (i, j) in enumerate(zip(st["slots"].tolist(), st["out_slots"].tolist())):
            new = lam[:, None, None] * old[i] + torch.einsum("hd,he->hde", st["k"][b].double(), st["v"][b].double())
            pool[j] = new
            o[b] = torch.einsum("hd,hde->he", st["q"][b].double(), new) / math.sqrt(case["D"])
        return [o, pool]
    if case["B"] * case["H"] * case["N"] ** 2 > 6e10:
        return None
    return _exact_linear(case, st)


def _exact_rotary(case, st):
    n, first = case["rot"] // 2, case["first"]
    lo = torch.arange(n, device=st["freq"].device)
    ia, ib = (first + 2 * lo, first + 2 * lo + 1) if case["interleaved"] else (first + lo, first + n + lo)
    turn = torch.polar(torch.full_like(st["freq"], st["scale"]).expand(*st["pos"].shape, n),
                       st["pos"].double().unsqueeze(-1) * st["freq"])
    turn = turn.unsqueeze(1) if turn.dim() == 3 else turn

    def rotate(x, w):
        y = x.detach().double().clone()
        z = torch.complex(y[..., ia], y[..., ib]) * w
        y[..., ia], y[..., ib] = z.real, z.imag
        return y

    got = [rotate(st["q"], turn), rotate(st["k"], turn)]
    if case["train"]:
        got += [rotate(st["dq"], turn.conj()), rotate(st["dk"], turn.conj())]
    return got


def _exact_linear(case, st):
    """Every pair of positions, one row block after the other."""
    B, H, N, D = st["q"].shape
    dev, scale = st["q"].device, 1.0 / math.sqrt(D)
    zeros = lambda *s: torch.zeros(*s, dtype=torch.float64, device=dev)  # noqa: E731
    o, dq, dk, dv = (zeros(B, H, N, D) for _ in range(4))
    final, dinitial = zeros(B, H, D, D), zeros(B, H, D, D)
    for b in range(B):
        L = N if st["lengths"] is None else int(st["lengths"][b])
        t = torch.arange(L, device=dev, dtype=torch.float64)
        for h in range(H):
            a = st["log_decay"][h].double()
            q, k, v = (st[x][b, h, :L].detach().double() for x in ("q", "k", "v"))
            s0 = st["initial"][b, h].detach().double() if case["carry"] else zeros(D, D)
            lead, tail = torch.exp(a * (t + 1))[:, None], torch.exp(a * (L - 1 - t))[:, None]
            final[b, h] = torch.exp(a * L) * s0 + (tail * k).t() @ v
            do = st["do"][b, h, :L].double() if case["train"] else None
            for r in range(0, L, 2048):
                e = min(L, r + 2048)
                w = torch.exp(a * (t[r:e, None] - t[None, :e]).clamp(min=0)).tril_(r) * scale
                p = (q[r:e] @ k[:e].t()) * w
                o[b, h, r:e] = p @ v[:e] + scale * (lead[r:e] * q[r:e]) @ s0
                if case["train"]:
                    dp = (do[r:e] @ v[:e].t()) * w
                    dq[b, h, r:e] = dp @ k[:e] + scale * lead[r:e] * (do[r:e] @ s0.t())
                    dk[b, h, :e] += dp.t() @ q[r:e]
                    dv[b, h, :e] += p.t() @ do[r:e]
            if case["train"] and case["carry"]:
                ds = st["dstate"][b, h].double()
                dk[b, h, :L] += tail * (v @ ds.t())
                dv[b, h, :L] += tail * (k @ ds)
                dinitial[b, h] = torch.exp(a * L) * ds + scale * (lead * q).t() @ do
    got = [o, final] if case["carry"] else [o]
    if case["train"]:
        got += [dq, dk, dv] + ([dinitial] if case["carry"] else [])
    return got


def work(case):
    B, H, D, e = case["B"], case["H"], case["D"], BYTES[case["dtype"]]
    if case["op"] == "step":
        return {"bytes": B * H * (8 * D * D + 4 * D * e), "flops": 5 * B * H * D * D}
    n = B * H * case["N"]
    if case["op"] == "rotary":
        passes = 2 if case["train"] else 1
        return {"bytes": passes * 2 * 2 * n * D * e, "flops": passes * 2 * 6 * n * (case["rot"] // 2)}
    # a token's share: the state's update and its read (forward), five such products behind
    state = 2 * 4 * B * H * D * D if case["carry"] else 0
    if case["train"]:
        return {"bytes": 11 * n * D * e + 2 * state, "flops": (4 + 10) * n * D * D}
    return {"bytes": 4 * n * D * e + state, "flops": 4 * n * D * D}
