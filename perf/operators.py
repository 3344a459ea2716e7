"""Timed cases of the attention operators: per-head norms of queries and keys
with their position rotation (``qk_norm_rope``), and softmax attention forward
and backward (``attn``).

Each case is one call as a program makes it: a serving step, a prefill, or a
training step (forward and backward through autograd).  With ``own`` false
``run`` evaluates the operators' definitions with elementary torch operations
in float32; with ``own`` true it calls the library.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


# ------------------------------------------------------------------- cases

def _norm(name, dtype, train, B, Hq, Hk, N, D, R, interleaved, pos0):
    return {"name": name, "op": "norm_rope", "dtype": dtype, "train": train, "B": B, "Hq": Hq,
            "Hk": Hk, "N": N, "D": D, "R": R, "interleaved": interleaved, "pos0": pos0}


def _attn(name, dtype, train, B, Hq, Hk, Nq, Nk, D, causal, ragged):
    return {"name": name, "op": "attn", "dtype": dtype, "train": train, "B": B, "Hq": Hq,
            "Hk": Hk, "Nq": Nq, "Nk": Nk, "D": D, "causal": causal, "ragged": ragged}


def listed():
    return [
        # one new token of 32 requests, far into their sequences: latency counts
        _norm("norm_rope_step", "bf16", False, 32, 32, 8, 1, 128, 128, False, 100000),
        # a prefill batch, projections in [B, N, H, D] layout, shared key heads
        _norm("norm_rope_prefill", "bf16", False, 4, 32, 8, 4096, 128, 128, False, 0),
        # a training step at the forward + backward workload's sizes
        # (batch 8, 8 heads of 32, 16,384 tokens)
        _norm("norm_rope_train", "bf16", True, 8, 8, 8, 16384, 32, 32, False, 0),
        # float32, an odd token count, part of each head rotated, adjacent pairs
        _norm("norm_rope_train_fp32", "fp32", True, 3, 6, 6, 1111, 80, 48, True, 17),
        # the smallest serving step: one request, one token, a short cache
        _attn("attn_step_small", "bf16", False, 1, 8, 2, 1, 777, 64, False, False),
        # one token of 16 requests over caches filled to different lengths
        _attn("attn_step", "bf16", False, 16, 32, 8, 1, 16384, 128, False, True),
        # a piece of a prompt over what the cache already holds, odd sizes
        _attn("attn_chunk", "bf16", False, 2, 16, 4, 333, 5001, 64, True, True),
        # causal prefill with shared key heads
        _attn("attn_prefill", "bf16", False, 2, 32, 8, 4096, 4096, 128, True, False),
        # causal training step with shared key heads
        _attn("attn_train_causal", "bf16", True, 2, 16, 4, 4096, 4096, 128, True, False),
        # training step over all pairs of tokens (a mesh), padded batch
        _attn("attn_train_full", "bf16", True, 2, 8, 8, 6000, 6000, 64, False, True),
        # latents attending to a long sequence (an encode with heads of 64)
        _attn("attn_train_latent", "bf16", True, 2, 8, 8, 256, 65536, 64, False, False),
        # float32 training step
        _attn("attn_train_fp32", "fp32", True, 2, 8, 4, 1000, 1000, 64, True, False),
    ]


def _logint(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.randrange(10)
    if kind < 4:                       # norms and rotation
        train = kind >= 2
        dtype = rng.choice(["bf16", "bf16", "fp32"])
        D = rng.choice([32, 48, 64, 80, 96, 128])
        Hk = rng.choice([1, 2, 3, 4, 8])
        Hq = Hk * rng.choice([1, 2, 4])
        B = rng.randint(1, 32)
        N = _logint(rng, 1, max(1, (4 * 40 * 4096 * 128) // (B * (Hq + Hk) * D)))
        N = min(N, 32768)
        R = rng.choice([D, D, 16 * (D // 32)])
        return _norm("", dtype, train, B, Hq, Hk, N, D, R, rng.random() < 0.3,
                     _logint(rng, 1, 200000))
    D = rng.choice([32, 64, 64, 80, 128, 128])
    Hk = rng.choice([1, 2, 4, 8])
    Hq = Hk * rng.choice([1, 2, 4])
    B = rng.randint(1, 4)
    ragged = rng.random() < 0.5
    if kind < 6:                       # serving: one or a few tokens over a cache
        B = rng.randint(1, 16)
        Nq = rng.choice([1, 1, 1, 2, 5])
        Nk = _logint(rng, max(Nq, 64), 16384)
        return _attn("", "bf16", False, B, Hq, Hk, Nq, Nk, D, True, ragged)
    train = kind >= 7
    if kind == 9 and rng.random() < 0.4:
        Nq = _logint(rng, 16, 900)
        Nk = _logint(rng, 16, 900)
        return _attn("", "fp32", True, B, Hq, Hk, Nq, Nk, D, rng.random() < 0.5, ragged)
    if rng.random() < 0.3:             # few queries, many keys
        Nq = _logint(rng, 16, 512)
        Nk = _logint(rng, 1024, 65536)
        causal = False
    else:
        Nq = _logint(rng, 64, 4096)
        causal = rng.random() < 0.5
        Nk = Nq if rng.random() < 0.6 else _logint(rng, 64, 4096)
    most = 2 * 16 * 4096 * 4096
    B = max(1, min(B, most // (Hq * Nq * Nk)))
    if B * Hq * Nq * Nk > most:
        Hq = Hk
    if B * Hq * Nq * Nk > most:
        Nk = max(64, most // (B * Hq * Nq))
    return _attn("", "bf16", train, B, Hq, Hk, Nq, Nk, D, causal, ragged)


def _lens(case, n, parts):
    """Valid lengths of a ragged batch: from n down to about n (1 - 1/parts)."""
    B = case["B"]
    return [max(1, n - (b * n) // (parts * B)) for b in range(B)]


def _k_lens(case):
    return _lens(case, case["Nk"], 2) if case["ragged"] else [case["Nk"]] * case["B"]


def _q_lens(case):
    """Queries are padded in training only (a serving call has them all)."""
    return _lens(case, case["Nq"], 2) if case["ragged"] and case["train"] \
        else [case["Nq"]] * case["B"]


# ------------------------------------------------------------------ inputs

def _randn(shape, dtype, gen):
    return torch.randn(shape, dtype=torch.float32, device="cuda", generator=gen).to(dtype)


def _tokens(B, H, N, D, dtype, gen):
    """A [B,H,N,D] view of a projection's [B,N,H,D] output."""
    return _randn((B, N, H, D), dtype, gen).transpose(1, 2)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = DTYPES[case["dtype"]]
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    st = {"case": case}
    if case["op"] == "norm_rope":
        N, R = case["N"], case["R"]
        st["q"] = _tokens(B, Hq, N, D, dt, gen)
        st["k"] = _tokens(B, Hk, N, D, dt, gen)
        st["wq"] = (1.0 + 0.1 * _randn((D,), torch.float32, gen)).to(dt)
        st["wk"] = (1.0 + 0.1 * _randn((D,), torch.float32, gen)).to(dt)
        pos = case["pos0"] + torch.arange(N, dtype=torch.float64, device="cuda")
        freq = 10000.0 ** (-torch.arange(0, R, 2, dtype=torch.float64, device="cuda") / R)
        ang = pos[:, None] * freq[None, :]
        st["cos"], st["sin"] = ang.cos().float(), ang.sin().float()
        if case["train"]:
            st["dqo"] = _tokens(B, Hq, N, D, dt, gen)
            st["dko"] = _tokens(B, Hk, N, D, dt, gen)
        return st
    Nq, Nk = case["Nq"], case["Nk"]
    # queries are sharper than unit scale, as trained ones are
    st["q"] = _randn((B, Nq, Hq, D), dt, gen).mul_(1.5).transpose(1, 2)
    if case["train"] or Nq == Nk:
        st["k"] = _tokens(B, Hk, Nk, D, dt, gen)
        st["v"] = _tokens(B, Hk, Nk, D, dt, gen)
    else:                              # a cache: [B,H,N,D]
        st["k"] = _randn((B, Hk, Nk, D), dt, gen)
        st["v"] = _randn((B, Hk, Nk, D), dt, gen)
    st["k_lens"] = st["q_lens"] = None
    if case["ragged"]:
        st["k_lens"] = torch.tensor(_k_lens(case), dtype=torch.int32, device="cuda")
        if case["train"]:
            st["q_lens"] = torch.tensor(_q_lens(case), dtype=torch.int32, device="cuda")
    if case["train"]:
        st["dy"] = _tokens(B, Hq, Nq, D, dt, gen)
    return st


# ---------------------------------------------------------- the operators

def _library():
    import rank_latent_attention_flare_b200 as fl
    return fl


def run(state):
    case = state["case"]
    if case["op"] == "norm_rope":
        return _run_norm_own(state) if own else _run_norm_plain(state)
    return _run_attn_own(state) if own else _run_attn_plain(state)


def _run_norm_own(st):
    fl, case = _library(), st["case"]
    args = (st["cos"], st["sin"])
    if not case["train"]:
        return fl.qk_norm_rope_fwd(st["q"], st["k"], st["wq"], st["wk"], *args, eps=1e-6,
                                   interleaved=case["interleaved"])
    leaves = [st[n].detach().requires_grad_() for n in ("q", "k", "wq", "wk")]
    qo, ko = fl.qk_norm_rope(*leaves, *args, eps=1e-6, interleaved=case["interleaved"])
    return (qo, ko, *torch.autograd.grad((qo, ko), leaves, (st["dqo"], st["dko"])))


def _run_attn_own(st):
    fl, case = _library(), st["case"]
    kw = dict(causal=case["causal"], q_lens=st["q_lens"], k_lens=st["k_lens"])
    if not case["train"]:
        return fl.attn_fwd(st["q"], st["k"], st["v"], **kw)
    leaves = [st[n].detach().requires_grad_() for n in ("q", "k", "v")]
    y = fl.attn(*leaves, **kw)
    return (y, *torch.autograd.grad(y, leaves, st["dy"]))


def _rotate(x, cos, sin, interleaved):
    R = 2 * cos.shape[-1]
    a, b = (x[..., 0:R:2], x[..., 1:R:2]) if interleaved else (x[..., :R // 2], x[..., R // 2:R])
    u, v = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((u, v), -1).flatten(-2) if interleaved else torch.cat((u, v), -1)
    return torch.cat((turned, x[..., R:]), -1)


def _norm_plain(x, w, st):
    x = x.float()
    xh = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    return _rotate(xh * w.float(), st["cos"], st["sin"], st["case"]["interleaved"])


def _norm_grad_plain(x, w, dy, st):
    x, w = x.float(), w.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
    xh = x * r
    g = _rotate(dy.float(), st["cos"], -st["sin"], st["case"]["interleaved"])
    gw = g * w
    dx = r * (gw - xh * (gw * xh).mean(-1, keepdim=True))
    return dx, (g * xh).sum((0, 1, 2))


def _run_norm_plain(st):
    dt = st["q"].dtype
    qo = _norm_plain(st["q"], st["wq"], st).to(dt)
    ko = _norm_plain(st["k"], st["wk"], st).to(dt)
    if not st["case"]["train"]:
        return qo, ko
    dq, dwq = _norm_grad_plain(st["q"], st["wq"], st["dqo"], st)
    dk, dwk = _norm_grad_plain(st["k"], st["wk"], st["dko"], st)
    return qo, ko, dq.to(dt), dk.to(dt), dwq.to(dt), dwk.to(dt)


def _visible(st):
    """[B, 1, Nq, Nk] truth values: which keys a query sees."""
    case, dev = st["case"], st["q"].device
    B, Nq, Nk = case["B"], case["Nq"], case["Nk"]
    ql = st["q_lens"] if st["q_lens"] is not None else torch.full((B,), Nq, device=dev)
    kl = st["k_lens"] if st["k_lens"] is not None else torch.full((B,), Nk, device=dev)
    i = torch.arange(Nq, device=dev).view(1, 1, Nq, 1)
    j = torch.arange(Nk, device=dev).view(1, 1, 1, Nk)
    ql, kl = ql.view(B, 1, 1, 1), kl.view(B, 1, 1, 1)
    seen = (j < kl) & (i < ql)
    return seen & (j <= i + (kl - ql)) if case["causal"] else seen


def _run_attn_plain(st):
    case, dt = st["case"], st["q"].dtype
    B, Hq, Hk, Nq, Nk, D = (case[n] for n in ("B", "Hq", "Hk", "Nq", "Nk", "D"))
    G, s = Hq // Hk, 1.0 / math.sqrt(D)
    # one matrix product per key head: its G query heads stacked
    q = st["q"].float().reshape(B, Hk, G * Nq, D)
    k, v = st["k"].float(), st["v"].float()
    a = torch.matmul(q, k.transpose(-1, -2)).view(B, Hk, G, Nq, Nk)
    if case["causal"] or case["ragged"]:
        a = a.masked_fill(~_visible(st).unsqueeze(2), -math.inf)
    top = a.amax(-1, keepdim=True)
    p = torch.exp((a - torch.where(torch.isinf(top), 0.0, top)) * s)
    del a
    total = p.sum(-1, keepdim=True)
    p = p / torch.where(total == 0, 1.0, total)
    y = torch.matmul(p.view(B, Hk, G * Nq, Nk), v).view(B, Hq, Nq, D)
    if not case["train"]:
        return y.to(dt)
    dy = st["dy"].float()
    if st["q_lens"] is not None:
        dy = dy * (torch.arange(Nq, device=dy.device) < st["q_lens"].view(B, 1)).view(B, 1, Nq, 1)
    dy = dy.reshape(B, Hk, G * Nq, D)
    pm = p.view(B, Hk, G * Nq, Nk)
    dv = torch.matmul(pm.transpose(-1, -2), dy)
    delta = (dy * y.reshape(B, Hk, G * Nq, D)).sum(-1, keepdim=True)
    ds = pm * (torch.matmul(dy, v.transpose(-1, -2)) - delta) * s
    dq = torch.matmul(ds, k).view(B, Hq, Nq, D)
    dk = torch.matmul(ds.transpose(-1, -2), q)
    return y.to(dt), dq.to(dt), dk.to(dt), dv.to(dt)


# ------------------------------------------------------------------- floors

def _pairs(case):
    """Query-key pairs that see each other, per query head, over the batch."""
    total = 0
    for ql, kl in zip(_q_lens(case), _k_lens(case)):
        if not case["causal"]:
            total += ql * kl
            continue
        off = kl - ql                  # query i sees min(kl, i + off + 1) keys, at least none
        first = max(0, -off)
        n = ql - first
        total += n * (first + off + 1) + n * (n - 1) // 2 if n > 0 else 0
    return total


def work(case):
    esz = 2 if case["dtype"] == "bf16" else 4
    B, Hq, Hk, D = case["B"], case["Hq"], case["Hk"], case["D"]
    if case["op"] == "norm_rope":
        N, R = case["N"], case["R"]
        rows = B * N * (Hq + Hk)
        tables = N * R * 4 + 2 * D * esz
        if not case["train"]:
            return {"bytes": 2 * rows * D * esz + tables, "flops": rows * (4 * D + 3 * R)}
        # x and the upstream gradient in; outputs and input gradients out
        return {"bytes": 4 * rows * D * esz + tables + 2 * D * esz,
                "flops": rows * (15 * D + 6 * R)}
    nq, nk, pairs = sum(_q_lens(case)), sum(_k_lens(case)), _pairs(case)
    q_bytes, kv_bytes = nq * Hq * D * esz, nk * Hk * D * esz
    if not case["train"]:
        return {"bytes": 2 * q_bytes + 2 * kv_bytes, "flops": 4 * Hq * pairs * D}
    # forward: two products; backward: five (the logits again, dP, dV, dK, dQ)
    return {"bytes": 4 * q_bytes + 4 * kv_bytes, "flops": 14 * Hq * pairs * D}


# ------------------------------------------------------- 64-bit definition

def _exact_norm(st, name):
    """Row by row definition: y = T (w x / rms(x)) with T the rotation."""
    case = st["case"]
    x, w = st[name].double(), st["w" + name].double()
    D, R = case["D"], case["R"]
    idx = torch.arange(R // 2, device=x.device)
    first = 2 * idx if case["interleaved"] else idx
    second = first + (1 if case["interleaved"] else R // 2)
    c, s = st["cos"].double(), st["sin"].double()
    rms = ((x ** 2).sum(-1, keepdim=True) / D + 1e-6).sqrt()
    u = w * x / rms
    y = u.clone()
    y[..., first] = c * u[..., first] - s * u[..., second]
    y[..., second] = s * u[..., first] + c * u[..., second]
    if not case["train"]:
        return y, None, None
    dy = st["d" + name + "o"].double()
    du = dy.clone()
    du[..., first] = c * dy[..., first] + s * dy[..., second]
    du[..., second] = c * dy[..., second] - s * dy[..., first]
    dw = (du * x / rms).sum((0, 1, 2))
    dn = du * w
    dx = dn / rms - x * (dn * x).sum(-1, keepdim=True) / (D * rms ** 3)
    return y, dx, dw


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "norm_rope":
        q, k = _exact_norm(st, "q"), _exact_norm(st, "k")
        return (q[0], k[0], q[1], k[1], q[2], k[2]) if case["train"] else (q[0], k[0])
    B, Hq, Hk, Nq, Nk, D = (case[n] for n in ("B", "Hq", "Hk", "Nq", "Nk", "D"))
    G, s = Hq // Hk, D ** -0.5
    dev = st["q"].device
    y = torch.zeros((B, Hq, Nq, D), dtype=torch.float64, device=dev)
    dq = torch.zeros_like(y)
    dk = torch.zeros((B, Hk, Nk, D), dtype=torch.float64, device=dev)
    dv = torch.zeros_like(dk)
    for b, (ql, kl) in enumerate(zip(_q_lens(case), _k_lens(case))):
        hidden = None
        if case["causal"]:
            hidden = torch.arange(kl, device=dev)[None, :] \
                > torch.arange(ql, device=dev)[:, None] + (kl - ql)
            none = hidden.all(-1)
        for h in range(Hq):
            q = st["q"][b, h, :ql].double()
            k = st["k"][b, h // G, :kl].double()
            v = st["v"][b, h // G, :kl].double()
            a = (q @ k.T) * s
            if hidden is not None:
                a.masked_fill_(hidden, -math.inf)
                a[none] = 0.0
            p = torch.softmax(a, -1)
            if hidden is not None:
                p[none] = 0.0
            y[b, h, :ql] = p @ v
            if case["train"]:
                g = st["dy"][b, h, :ql].double()
                dv[b, h // G, :kl] += p.T @ g
                dp = g @ v.T
                da = p * (dp - (p * dp).sum(-1, keepdim=True)) * s
                dq[b, h, :ql] = da @ k
                dk[b, h // G, :kl] += da.T @ q
    return (y, dq, dk, dv) if case["train"] else y
