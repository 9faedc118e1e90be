"""What the decay scan and the group norm cost: the cases, their inputs, their plain forms and their work.

The decay scan is linear attention with one decay a_h in [0, 1] per head: S_t = a_h S_{t-1} + v_t k_t^T,
o_t = S_t q_t, over prompts (forward, backward) and for single tokens.  The group norm is
y = act(n w + b), or (n w + b) act(gate), with n normalised over each sample's positions and one
group of channels, channels last.  ``run`` computes the plain form with elementary torch operations, or
(``own``) calls the library; ``exact`` computes the same from the definitions in 64 bits.
"""
import math

import torch

own = False

WIDTHS = (32, 64, 128)
CHUNK = 128  # of the plain chunked form


def listed():
    bf, f32 = "bf16", "f32"
    return [
        # one long context on few heads (the long-context workload's sizes), with an entry state
        dict(name="scan long", op="scan", B=1, H=16, Hkv=16, T=65536, dk=128, dv=128, io=bf, ragged=False, S0=True),
        # a padded batch of behaviour sequences (the recommendation workload's sizes)
        dict(name="scan padded batch", op="scan", B=32, H=4, Hkv=4, T=8192, dk=64, dv=64, io=bf, ragged=True, S0=False),
        # a short prompt of odd length, keys and values shared by four heads: latency counts
        dict(name="scan short shared", op="scan", B=2, H=8, Hkv=2, T=777, dk=64, dv=128, io=bf, ragged=True, S0=True),
        # 32-bit inputs, unequal widths
        dict(name="scan f32", op="scan", B=4, H=8, Hkv=8, T=1000, dk=128, dv=64, io=f32, ragged=False, S0=False),
        # the language-model training shape
        dict(name="scan grad train", op="scan_grad", B=4, H=8, Hkv=8, T=4096, dk=128, dv=128, io=bf, ragged=False, S0=False),
        # gradients of shared keys and values, odd length, small widths
        dict(name="scan grad shared", op="scan_grad", B=3, H=6, Hkv=2, T=1021, dk=32, dv=64, io=bf, ragged=True, S0=True),
        # one token for each of many sequences (the decode workload's sizes)
        dict(name="step many", op="step", B=256, H=32, Hkv=32, T=1, dk=128, dv=128, io=bf, ragged=False, S0=True),
        # one token of one sequence: the latency of a single user's decode
        dict(name="step one", op="step", B=1, H=16, Hkv=16, T=1, dk=128, dv=128, io=bf, ragged=False, S0=True),
        # the norm behind a scan: every token on its own, one group per head, gated
        dict(name="norm heads gated", op="norm", N=65536, S=1, C=2048, G=16, io=bf, act="silu", gate=True, affine=True),
        # image-like positions, statistics over them
        dict(name="norm positions", op="norm", N=8, S=4096, C=320, G=32, io=bf, act="silu", gate=False, affine=True),
        # training of the gated norm behind the scan at the training shape
        dict(name="norm grad heads gated", op="norm_grad", N=16384, S=1, C=1024, G=8, io=bf, act="silu", gate=True, affine=True),
        # odd positions in 32 bits
        dict(name="norm grad odd f32", op="norm_grad", N=3, S=391, C=96, G=8, io=f32, act="gelu", gate=False, affine=True),
    ]


def _spread(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["scan", "scan", "scan", "scan_grad", "scan_grad", "step", "norm", "norm", "norm_grad"])
    io = "f32" if rng.random() < 0.25 else "bf16"
    if op in ("norm", "norm_grad"):
        if rng.random() < 0.5:  # per token: a group is one head
            S, G, D = 1, rng.randint(1, 32), rng.choice([32, 64, 128])
            N = _spread(rng, 1, 32768)
        else:  # over positions: any even or odd channel count
            S, G, D = _spread(rng, 16, 4096), rng.randint(1, 32), rng.randint(1, 40)
            N = rng.randint(1, 16)
        while N * S * G * D > 1 << 26:
            N = max(1, N // 2)
            S = max(1, S // 2) if N == 1 else S
        return dict(op=op, N=N, S=S, C=G * D, G=G, io=io, act=rng.choice(["none", "silu", "gelu"]),
                    gate=rng.random() < 0.5, affine=rng.random() < 0.8)
    dk, dv = rng.choice(WIDTHS), rng.choice(WIDTHS)
    group = rng.choice([1, 1, 2, 4])
    H = group * rng.randint(1, 8)
    if op == "step":
        B, T = _spread(rng, 1, 256), 1
    else:
        B, T = rng.randint(1, 8), _spread(rng, 1, 16384 if io == "bf16" else 4096)
        while B * T * H > (1 << 19 if op == "scan" else 1 << 18):
            B = max(1, B // 2)
            T = max(1, T // 2) if B == 1 else T
    return dict(op=op, B=B, H=H, Hkv=H // group, T=T, dk=dk, dv=dv, io=io,
                ragged=op != "step" and rng.random() < 0.4, S0=op == "step" or rng.random() < 0.5)


# ---- inputs ------------------------------------------------------------------------------------


def prepare(case, seed):
    dev = torch.device("cuda")
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    io = torch.float32 if case["io"] == "f32" else torch.bfloat16

    def normal(*shape, dtype=io, std=1.0, mean=0.0):
        return (torch.randn(shape, generator=g, device=dev) * std + mean).to(dtype)

    c, st = case, {"case": case}
    if c["op"] in ("norm", "norm_grad"):
        shape = (c["N"], c["S"], c["C"])
        st["x"] = normal(*shape, mean=0.5)
        st["gate"] = normal(*shape) if c["gate"] else None
        st["weight"] = normal(c["C"], dtype=torch.float32, std=0.2, mean=1.0) if c["affine"] else None
        st["bias"] = normal(c["C"], dtype=torch.float32, std=0.2) if c["affine"] else None
        st["eps"] = 1e-5
        if c["op"] == "norm_grad":  # what the forward call of a training step left
            st["dy"] = normal(*shape)
            x = st["x"].double().view(c["N"], c["S"], c["G"], -1)
            var, mean = torch.var_mean(x, dim=(1, 3), unbiased=False)
            st["mean"], st["rstd"] = mean.float(), (var + st["eps"]).rsqrt().float()
        return st
    B, H, Hkv, T, dk, dv = (c[n] for n in ("B", "H", "Hkv", "T", "dk", "dv"))
    st["q"] = normal(B, T, H, dk)
    st["k"] = torch.nn.functional.normalize(normal(B, T, Hkv, dk, dtype=torch.float32), dim=-1).to(io)
    st["v"] = normal(B, T, Hkv, dv)
    # heads of short to long memory: 1 - a from 2^-2 to 2^-12
    st["decay"] = (1 - 2.0 ** -torch.linspace(2, 12, H, dtype=torch.float64)).float().to(dev)
    st["S0"] = normal(B, H, dv, dk, dtype=torch.float32, std=0.1) if c["S0"] else None
    st["lengths"] = None
    if c["ragged"]:  # a padded batch: the longest sequence fills it
        n = torch.randint(1, T + 1, (B,), generator=g, device=dev, dtype=torch.int32)
        n[0] = T
        st["lengths"] = n
    if c["op"] == "scan_grad":
        st["dO"] = normal(B, T, H, dv)
        st["dS"] = normal(B, H, dv, dk, dtype=torch.float32, std=0.1) if c["S0"] else None
    return st


def work(case):
    c = case
    e = 4 if c["io"] == "f32" else 2
    if c["op"] in ("norm", "norm_grad"):
        n = c["N"] * c["S"] * c["C"]
        small = (8 * c["C"] if c["affine"] else 0) + 8 * c["N"] * c["G"]
        if c["op"] == "norm":
            return {"bytes": n * e * (3 if c["gate"] else 2) + small, "flops": 12.0 * n}
        return {"bytes": n * e * (5 if c["gate"] else 3) + 2 * small, "flops": 25.0 * n}
    B, H, Hkv, T, dk, dv = (c[n] for n in ("B", "H", "Hkv", "T", "dk", "dv"))
    rows = B * T * (H * (dk + dv) + Hkv * (dk + dv)) * e  # q, o, k, v
    state = B * H * dk * dv
    if c["op"] == "step":
        return {"bytes": rows + 8 * state, "flops": 5.0 * state}
    if c["op"] == "scan":
        return {"bytes": rows + 4 * state * (2 if c["S0"] else 1), "flops": 4.0 * T * state}
    grads = B * T * (H * dk + Hkv * (dk + dv)) * e
    return {"bytes": rows + grads + 4 * state * (3 if c["S0"] else 1), "flops": 10.0 * T * state}


# ---- the plain forms ----------------------------------------------------------------------------


def _pow(decay, n):
    """decay[h] ^ n for whole exponents n >= 0 ([...] -> [H, ...]), rounded once to 32 bits."""
    d = decay.double().view(-1, *[1] * n.dim())
    return torch.pow(d, n.double().unsqueeze(0)).float()


def _heads(x, H):
    """[B, T, Hkv, d] -> fp32 [B, H, T, d]."""
    return x.float().repeat_interleave(H // x.shape[2], dim=2).transpose(1, 2)


def _chunks(x, n, pad):
    return torch.nn.functional.pad(x, (0, 0, 0, pad)).unflatten(2, (n, CHUNK))


def _setup(st):
    c = st["case"]
    B, H, T = c["B"], c["H"], c["T"]
    dev = st["q"].device
    t = torch.arange(T, device=dev)
    ends = torch.full((B,), T, device=dev) if st["lengths"] is None else st["lengths"].long()
    live = (t < ends[:, None])[:, None, :, None]  # [B, 1, T, 1]
    n = -(-T // CHUNK)
    i = torch.arange(CHUNK, device=dev)
    diff = i[:, None] - i
    inner = _pow(st["decay"], diff.clamp(min=0)) * (diff >= 0)  # [H, C, C]
    m = torch.arange(n, device=dev)
    gap = m[:, None] - 1 - m
    outer = _pow(st["decay"], (gap * CHUNK).clamp(min=0)) * (gap >= 0)  # [H, n, n]: chunk m's writes at chunk n's entry
    return dict(B=B, H=H, T=T, n=n, pad=n * CHUNK - T, t=t, i=i, ends=ends, live=live, inner=inner[:, None], outer=outer, m=m)


def _plain_pass(p, x, y, z, inner, rows, entry):
    """o = (x y^T o inner) z + rows x entry, per chunk."""
    o = ((x @ y.transpose(-1, -2)) * inner) @ z + (x @ entry) * rows
    return o.flatten(2, 3)[:, :, : p["T"]]


def _masked(x, live):
    return torch.where(live, x, torch.zeros((), device=x.device))


def _forward_entries(st, p, k, v):
    """Entry state of every chunk, transposed: [B, H, n, dk, dv]."""
    w = _pow(st["decay"], CHUNK - 1 - p["i"])[:, None, :, None]
    F = (k * w).transpose(-1, -2) @ v
    E = (p["outer"] @ F.flatten(3)).unflatten(3, F.shape[3:])
    if st["S0"] is not None:
        E = E + _pow(st["decay"], p["m"] * CHUNK)[:, :, None, None] * st["S0"].transpose(-1, -2)[:, :, None]
    return E


def _state_weights(st, p):
    """a^(len - 1 - t) for live tokens, [B, H, T, 1], and a^len, [B, H, 1, 1]."""
    left = p["ends"][:, None] - 1 - p["t"]
    w = _pow(st["decay"], left.clamp(min=0)).transpose(0, 1).unsqueeze(-1) * p["live"]
    return w, _pow(st["decay"], p["ends"]).t()[:, :, None, None]


def _plain_scan(st):
    p, H = _setup(st), st["case"]["H"]
    io = st["q"].dtype
    q, k, v = (_masked(_heads(st[n], H), p["live"]) for n in "qkv")
    w, whole = _state_weights(st, p)
    S = v.transpose(-1, -2) @ (k * w)
    if st["S0"] is not None:
        S = S + whole * st["S0"]
    q, k, v = (_chunks(x, p["n"], p["pad"]) for x in (q, k, v))
    rows = _pow(st["decay"], p["i"] + 1)[:, None, :, None]
    o = _plain_pass(p, q, k, v, p["inner"], rows, _forward_entries(st, p, k, v))
    return {"o": _masked(o, p["live"]).transpose(1, 2).to(io).contiguous(), "S": S}


def _plain_scan_grad(st):
    p, c = _setup(st), st["case"]
    H, Hkv, io, a = c["H"], c["Hkv"], st["q"].dtype, st["decay"]
    q, k, v, dO = (_masked(_heads(st[n], H), p["live"]) for n in ("q", "k", "v", "dO"))
    w, whole = _state_weights(st, p)
    first = _pow(a, p["t"] + 1)[:, :, None]
    dS0 = dO.transpose(-1, -2) @ (q * first)
    # what dS_final adds to dk and dv: its weight at token t is a^(len - 1 - t)
    dk_end = dv_end = 0.0
    if st["dS"] is not None:
        dS0 = dS0 + whole * st["dS"]
        dk_end = w * (v @ st["dS"])
        dv_end = w * (k @ st["dS"].transpose(-1, -2))
    q, k, v, dO = (_chunks(x, p["n"], p["pad"]) for x in (q, k, v, dO))
    E = _forward_entries(st, p, k, v)
    dq = _plain_pass(p, dO, v, k, p["inner"], _pow(a, p["i"] + 1)[:, None, :, None], E.transpose(-1, -2))
    # the gradient of the state at each chunk's end, [B, H, n, dv, dk]
    F = (dO * _pow(a, p["i"] + 1)[:, None, :, None]).transpose(-1, -2) @ q
    G = (p["outer"].transpose(-1, -2) @ F.flatten(3)).unflatten(3, F.shape[3:])
    rows = _pow(a, CHUNK - 1 - p["i"])[:, None, :, None]
    back = p["inner"].transpose(-1, -2)
    dk = _plain_pass(p, v, dO, q, back, rows, G) + dk_end
    dv = _plain_pass(p, k, q, dO, back, rows, G.transpose(-1, -2)) + dv_end

    def out(x, heads):
        x = _masked(x, p["live"]).unflatten(1, (heads, H // heads)).sum(2)
        return x.transpose(1, 2).to(io).contiguous()

    return {"dq": out(dq, H), "dk": out(dk, Hkv), "dv": out(dv, Hkv), "dS0": dS0}


def _plain_step(st):
    H, S = st["case"]["H"], st["S0"]
    q, k, v = (_heads(st[n], H)[:, :, 0] for n in "qkv")  # [B, H, d]
    S.mul_(st["decay"][:, None, None]).add_(v[..., :, None] * k[..., None, :])
    o = (S * q[..., None, :]).sum(-1)
    return {"o": o[:, None].to(st["q"].dtype), "S": S}


def _act(name, x):
    if name == "silu":
        return x / (1 + torch.exp(-x))
    if name == "gelu":
        return x * 0.5 * (1 + torch.erf(x * math.sqrt(0.5)))
    return x


def _act_slope(name, x):
    if name == "silu":
        s = 1 / (1 + torch.exp(-x))
        return s * (1 + x * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) / math.sqrt(2 * math.pi)
    return torch.ones_like(x)


def _plain_norm(st):
    c = st["case"]
    x = st["x"].float().view(c["N"], c["S"], c["G"], -1)
    mean = x.mean(dim=(1, 3), keepdim=True)
    d = x - mean
    rstd = 1 / torch.sqrt((d * d).mean(dim=(1, 3), keepdim=True) + st["eps"])
    z = (d * rstd).view(c["N"], c["S"], c["C"])
    if st["weight"] is not None:
        z = z * st["weight"] + st["bias"]
    y = _act(c["act"], z) if st["gate"] is None else z * _act(c["act"], st["gate"].float())
    return {"y": y.to(st["x"].dtype), "mean": mean.view(c["N"], c["G"]), "rstd": rstd.view(c["N"], c["G"])}


def _plain_norm_grad(st):
    c = st["case"]
    N, S, C, G = c["N"], c["S"], c["C"], c["G"]
    x, dy = st["x"].float().view(N, S, G, -1), st["dy"].float()
    n = ((x - st["mean"].view(N, 1, G, 1)) * st["rstd"].view(N, 1, G, 1)).view(N, S, C)
    z = n if st["weight"] is None else n * st["weight"] + st["bias"]
    out = {}
    if st["gate"] is None:
        dz = dy * _act_slope(c["act"], z)
    else:
        gate = st["gate"].float()
        dz = dy * _act(c["act"], gate)
        out["dgate"] = (dy * z * _act_slope(c["act"], gate)).to(st["x"].dtype)
    dn = dz
    if st["weight"] is not None:
        dn = dz * st["weight"]
        out["dweight"] = (dz * n).sum(dim=(0, 1))
        out["dbias"] = dz.sum(dim=(0, 1))
    dn, n = dn.view(N, S, G, -1), n.view(N, S, G, -1)
    dx = (dn - dn.mean(dim=(1, 3), keepdim=True) - n * (dn * n).mean(dim=(1, 3), keepdim=True)) * st["rstd"].view(N, 1, G, 1)
    out["dx"] = dx.view(N, S, C).to(st["x"].dtype)
    return out


# ---- the library's calls ------------------------------------------------------------------------


def _own(st):
    from delta_rule_sequence_b200 import prism

    c = st["case"]
    if c["op"] == "scan":
        o, S = prism.prism_decay_scan_fwd(st["q"], st["k"], st["v"], st["decay"], st["S0"], st["lengths"])
        return {"o": o, "S": S}
    if c["op"] == "scan_grad":
        return prism.prism_decay_scan_bwd(st["q"], st["k"], st["v"], st["decay"], st["S0"], st["lengths"],
                                          dO=st["dO"], dS_final=st["dS"])
    if c["op"] == "step":
        return {"o": prism.prism_decay_step(st["q"], st["k"], st["v"], st["decay"], st["S0"]), "S": st["S0"]}
    if c["op"] == "norm":
        y, mean, rstd = prism.prism_group_norm_fwd(st["x"], c["G"], st["weight"], st["bias"], st["gate"],
                                                   eps=st["eps"], activation=c["act"])
        return {"y": y, "mean": mean, "rstd": rstd}
    return prism.prism_group_norm_bwd(st["x"], c["G"], st["mean"], st["rstd"], st["weight"], st["bias"], st["gate"],
                                      dy=st["dy"], activation=c["act"])


PLAIN = {"scan": _plain_scan, "scan_grad": _plain_scan_grad, "step": _plain_step, "norm": _plain_norm,
         "norm_grad": _plain_norm_grad}


def run(state):
    return _own(state) if own else PLAIN[state["case"]["op"]](state)


# ---- the definitions in 64 bits -----------------------------------------------------------------


def _exact_scan(st, grad):
    """The quadratic form, one (batch, head) and one block of rows at a time."""
    c = st["case"]
    B, H, Hkv, T, dk, dv = (c[n] for n in ("B", "H", "Hkv", "T", "dk", "dv"))
    dev, f8 = st["q"].device, torch.float64
    out = {"o": torch.zeros(B, T, H, dv, device=dev, dtype=f8), "S": torch.zeros(B, H, dv, dk, device=dev, dtype=f8)}
    if grad:
        out = {"dq": torch.zeros(B, T, H, dk, device=dev, dtype=f8), "dk": torch.zeros(B, T, Hkv, dk, device=dev, dtype=f8),
               "dv": torch.zeros(B, T, Hkv, dv, device=dev, dtype=f8), "dS0": torch.zeros(B, H, dv, dk, device=dev, dtype=f8)}
    ends = [T] * B if st["lengths"] is None else st["lengths"].tolist()
    for b in range(B):
        n = ends[b]
        t = torch.arange(n, device=dev, dtype=f8)
        for h in range(H):
            kv = h * Hkv // H
            a = st["decay"][h].double()
            q, k, v = st["q"][b, :n, h].double(), st["k"][b, :n, kv].double(), st["v"][b, :n, kv].double()
            S0 = torch.zeros(dv, dk, device=dev, dtype=f8) if st["S0"] is None else st["S0"][b, h].double()
            if grad:
                dO = st["dO"][b, :n, h].double()
                dS = torch.zeros_like(S0) if st["dS"] is None else st["dS"][b, h].double()
                out["dS0"][b, h] = a ** n * dS + torch.einsum("t,tv,tk->vk", a ** (t + 1), dO, q)
                out["dk"][b, :n, kv] += (a ** (n - 1 - t))[:, None] * (v @ dS)
                out["dv"][b, :n, kv] += (a ** (n - 1 - t))[:, None] * (k @ dS.T)
            else:
                out["S"][b, h] = a ** n * S0 + torch.einsum("t,tv,tk->vk", a ** (n - 1 - t), v, k)
            for r in range(0, n, 2048):
                e = min(n, r + 2048)
                gap = t[r:e, None] - t[:e]
                M = torch.where(gap >= 0, a ** gap.clamp(min=0), torch.zeros((), device=dev, dtype=f8))
                first = (a ** (t[r:e] + 1))[:, None]
                if not grad:
                    out["o"][b, r:e, h] = (M * (q[r:e] @ k[:e].T)) @ v[:e] + first * (q[r:e] @ S0.T)
                    continue
                dP = M * (dO[r:e] @ v[:e].T)
                out["dq"][b, r:e, h] = dP @ k[:e] + first * (dO[r:e] @ S0)
                out["dk"][b, :e, kv] += dP.T @ q[r:e]
                out["dv"][b, :e, kv] += (M * (q[r:e] @ k[:e].T)).T @ dO[r:e]
    return out


def _exact_norm(st, grad):
    """Through float64 group_norm and its autograd, positions and channels in their usual order."""
    c = st["case"]
    x = st["x"].double().transpose(1, 2)
    names = [n for n in ("weight", "bias", "gate") if st[n] is not None]
    leaf = {n: st[n].double().requires_grad_(grad) for n in names}
    x.requires_grad_(grad)
    z = torch.nn.functional.group_norm(x, c["G"], leaf.get("weight"), leaf.get("bias"), st["eps"]).transpose(1, 2)
    act = {"none": lambda u: u, "silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu}[c["act"]]
    y = act(z) if st["gate"] is None else z * act(leaf["gate"])
    if not grad:
        var, mean = torch.var_mean(x.unflatten(1, (c["G"], -1)), dim=(2, 3), unbiased=False)
        return {"y": y, "mean": mean, "rstd": (var + st["eps"]).rsqrt()}
    y.backward(st["dy"].double())
    return {"dx": x.grad.transpose(1, 2).contiguous(), **{"d" + n: leaf[n].grad for n in names}}


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] in ("norm", "norm_grad"):
        return _exact_norm(st, case["op"] == "norm_grad")
    if case["op"] in ("scan", "scan_grad"):
        return _exact_scan(st, case["op"] == "scan_grad")
    heads = {n: st[n].double().repeat_interleave(case["H"] // st[n].shape[2], dim=2)[:, 0] for n in "qkv"}
    S = st["decay"].double()[:, None, None] * st["S0"].double() + torch.einsum("bhv,bhk->bhvk", heads["v"], heads["k"])
    return {"o": torch.einsum("bhvk,bhk->bhv", S, heads["q"])[:, None], "S": S}
