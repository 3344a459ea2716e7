"""Per-head norms with position rotation (qk_norm_rope) against the 64-bit
definition, and a layer of them with attention and FLARE."""
import math

import pytest
import torch

import rank_latent_attention_flare_b200 as fl
from attn_ref import Attn, NormRope, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def make(dt, B, Hq, Hk, N, D, R, seed=0, layout="bnhd", per_batch=False, pos0=0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def one(H):
        shape = (B, N, H, D) if layout == "bnhd" else (B, H, N, D)
        t = torch.randn(shape, device=DEV, generator=g).to(dt)
        return t.transpose(1, 2) if layout == "bnhd" else t
    w = [(1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(dt) for _ in range(2)]
    cos = sin = None
    if R:
        pos = torch.arange(N, device=DEV, dtype=torch.float64) + pos0
        if per_batch:
            pos = pos + 100 * torch.arange(B, device=DEV).view(B, 1)
        ang = pos.unsqueeze(-1) * 10000.0 ** (
            -torch.arange(0, R, 2, device=DEV, dtype=torch.float64) / R)
        cos, sin = ang.cos().float(), ang.sin().float()
    return one(Hq), one(Hk), *w, cos, sin, one(Hq), one(Hk)


# B, Hq, Hk, N, D, R, interleaved, layout, per_batch
CASES = {
    "step": (32, 32, 8, 1, 128, 128, False, "bnhd", False),
    "step_own_positions": (5, 8, 2, 1, 64, 64, False, "bnhd", True),
    "one": (1, 1, 1, 1, 8, 0, False, "bhnd", False),
    "d16": (2, 3, 1, 33, 16, 16, False, "bhnd", False),
    "d32": (2, 8, 8, 257, 32, 32, False, "bnhd", False),
    "d40_part": (2, 5, 1, 100, 40, 32, True, "bnhd", True),
    "d48": (1, 2, 2, 70, 48, 48, False, "bhnd", False),
    "d64_heads_first": (3, 7, 2, 300, 64, 32, False, "bhnd", False),
    "d80_part": (2, 6, 6, 111, 80, 48, True, "bnhd", False),
    "d96": (1, 4, 2, 200, 96, 96, False, "bnhd", True),
    "d120_norm_only": (2, 3, 1, 90, 120, 0, False, "bnhd", False),
    "d128": (2, 12, 4, 700, 128, 128, False, "bnhd", False),
    "d128_pairs": (1, 2, 1, 129, 128, 64, True, "bhnd", False),
}


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_against_definition(name, dt):
    B, Hq, Hk, N, D, R, il, layout, per_batch = CASES[name]
    q, k, wq, wk, cos, sin, dqo, dko = make(dt, B, Hq, Hk, N, D, R, len(name), layout, per_batch)
    kw = dict(eps=1e-5, interleaved=il)
    qo, ko = fl.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, **kw)
    got = fl.qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dqo, dko, **kw)
    for i, (x, w, y, dy, t) in enumerate(((q, wq, qo, dqo, "q"), (k, wk, ko, dko, "k"))):
        ref = NormRope(x, w, cos, sin, 1e-5, il)
        within(y, ref.y, ref.y_bound, t + "o")
        assert y.stride() == x.stride()
        (dx, dw), (bx, bw) = ref.grads(dy)
        within(got[i], dx, bx, "d" + t)
        within(got[2 + i], dw, bw, "dw" + t)


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_without_weights_in_place_and_slices(dt):
    """No weights; outputs over the inputs, inside an interleaved buffer whose
    values keep their bits."""
    B, N, H, D = 2, 50, 4, 64
    *_, cos, sin, _, _ = make(dt, B, H, H, N, D, D, seed=1)
    qkv = torch.randn(B, N, 3, H, D, device=DEV).to(dt)
    was = qkv.clone()
    q, k = qkv[:, :, 0].transpose(1, 2), qkv[:, :, 1].transpose(1, 2)
    refs = [NormRope(t.clone(), None, cos, sin, 1e-6, False) for t in (q, k)]
    fl.qk_norm_rope_fwd(q, k, None, None, cos, sin, out=(q, k))
    for t, ref in zip((q, k), refs):
        within(t, ref.y, ref.y_bound, "out")
    assert torch.equal(qkv[:, :, 2], was[:, :, 2])


def test_zero_rows_and_large_values():
    q, k, wq, wk, cos, sin, dqo, dko = make(F32, 1, 2, 2, 20, 64, 64, seed=2)
    q[:, :, 3] = 0.0
    k *= 1e12
    refq, refk = NormRope(q, wq, cos, sin, 1e-6, False), NormRope(k, wk, cos, sin, 1e-6, False)
    qo, ko = fl.qk_norm_rope_fwd(q, k, wq, wk, cos, sin)
    within(qo, refq.y, refq.y_bound, "q")
    within(ko, refk.y, refk.y_bound, "k")
    got = fl.qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dqo, dko)
    (dx, _), (bx, _) = refq.grads(dqo)
    within(got[0], dx, bx, "dq")


def test_autograd_and_differences():
    """Against the formula and central differences of the 64-bit definition
    (step 1e-5, as for attention)."""
    q, k, wq, wk, cos, sin, dqo, dko = make(F32, 2, 3, 1, 17, 48, 32, seed=3)
    leaves = [t.clone().requires_grad_() for t in (q, k, wq, wk)]
    out = fl.qk_norm_rope(*leaves, cos, sin, eps=1e-6)
    got = torch.autograd.grad(out, leaves, (dqo, dko))

    def loss(x):
        a = NormRope(x[0], x[2], cos, sin, 1e-6, False).y
        b = NormRope(x[1], x[3], cos, sin, 1e-6, False).y
        return ((a * dqo.double()).sum() + (b * dko.double()).sum()).item()
    U64 = [t.double() for t in (q, k, wq, wk)]
    import attn_ref
    attn_ref.U[torch.float64] = 0.0
    gen = torch.Generator(device=DEV)
    gen.manual_seed(4)
    for i in range(4):
        d = torch.randn(U64[i].shape, dtype=torch.float64, device=DEV, generator=gen)
        ends = [loss([t + s * d if j == i else t for j, t in enumerate(U64)])
                for s in (1e-5, -1e-5)]
        num = (ends[0] - ends[1]) / 2e-5
        val = (got[i].double() * d).sum().item()
        # a float32 gradient's roundings, relative to the terms' magnitudes
        slack = 1e-5 * (got[i].double().abs() * d.abs()).sum().item()
        assert abs(val - num) <= slack + 1e-6, (i, val, num)


def test_repeatable_captured_other_stream():
    q, k, wq, wk, cos, sin, dqo, dko = make(BF, 2, 8, 2, 3000, 64, 64, seed=5)

    def step(**kw):
        return (*fl.qk_norm_rope_fwd(q, k, wq, wk, cos, sin, **kw),
                *fl.qk_norm_rope_bwd(q, k, wq, wk, cos, sin, dqo, dko, **kw))
    want = step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = step()
    g.replay()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other = step(stream=side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) and torch.equal(a, c) for a, b, c in zip(want, out, other))
    none = fl.qk_norm_rope_bwd(q, k, wq, None, cos, sin, dqo, dko, need_dw=False)
    assert none[2] is None and none[3] is None and torch.equal(none[0], want[2])


def test_layer_of_them_together():
    """A mixing layer: norms and rotation of a fused projection, then softmax
    attention and FLARE of the same heads, forward and backward."""
    B, N, H, D, M = 2, 300, 4, 32, 128
    gen = torch.Generator(device=DEV)
    gen.manual_seed(6)
    *_, wq, wk, cos, sin, _, _ = make(BF, B, H, H, N, D, D, seed=7)
    qkv = torch.randn(B, N, 3, H, D, device=DEV, generator=gen).to(BF).requires_grad_()
    lat = torch.randn(H, M, D, device=DEV, generator=gen).to(BF).requires_grad_()
    dy = torch.randn(B, H, N, D, device=DEV, generator=gen).to(BF)
    lens = torch.tensor([300, 171], dtype=torch.int32, device=DEV)
    ws = [w.requires_grad_() for w in (wq, wk)]

    def layer():
        q, k, v = (qkv[:, :, i].transpose(1, 2) for i in range(3))
        qo, ko = fl.qk_norm_rope(q, k, *ws, cos, sin)
        full = fl.attn(qo, ko, v, q_lens=lens, k_lens=lens)
        low = fl.flare(lat, ko, v, seq_lens=lens)
        return qo, ko, full, low
    qo, ko, full, low = layer()
    q, k, v = (qkv.detach()[:, :, i].transpose(1, 2) for i in range(3))
    for x, w, y in ((q, wq, qo), (k, wk, ko)):
        ref = NormRope(x, w.detach(), cos, sin, 1e-6, False)
        within(y.detach(), ref.y, ref.y_bound, "norm")
    ref = Attn(qo.detach(), ko.detach(), v, q_lens=[300, 171], k_lens=[300, 171])
    within(full.detach(), ref.y, ref.y_bound, "attn")
    assert torch.equal(low.detach(), fl.flare_fwd(lat.detach(), ko.detach(), v, seq_lens=lens))
    leaves = [qkv, lat, *ws]
    grads = torch.autograd.grad(((full + low) * dy).float().sum(), leaves)
    # by hand, with the library's own calls
    y, lse, low = fl.attn_fwd(qo.detach(), ko.detach(), v, q_lens=lens, k_lens=lens,
                              save_low=True)
    dqo, dko, dv = fl.attn_bwd(qo.detach(), ko.detach(), v, y, dy, lse, q_lens=lens, k_lens=lens,
                               y_low=low)
    _, Z, l2 = fl.flare_fwd(lat.detach(), ko.detach(), v, save=True, seq_lens=lens)
    dl, dk2, dv2 = fl.flare_bwd(lat.detach(), ko.detach(), v, dy, Z, l2, seq_lens=lens)
    dq, dk, dwq, dwk = fl.qk_norm_rope_bwd(q, k, wq.detach(), wk.detach(), cos, sin, dqo,
                                           dko + dk2)
    assert torch.equal(grads[1], dl)
    assert torch.equal(grads[2], dwq) and torch.equal(grads[3], dwk)
    assert torch.equal(grads[0][:, :, 0], dq.transpose(1, 2))
    assert torch.equal(grads[0][:, :, 1], dk.transpose(1, 2))
    assert torch.equal(grads[0][:, :, 2], (dv + dv2).transpose(1, 2))
    assert all(torch.isfinite(t).all() for t in grads)
    assert math.isfinite(full.float().sum().item())
