"""Softmax attention with NaN and infinities at keys that queries see: the rows
that the definition makes NaN are NaN, whatever the key's column in its tile,
and no others."""
import math

import pytest
import torch

import rank_latent_attention_flare_b200 as fl
from attn_ref import Attn, within
from test_gpu_attn import BF, F32, tensors

pytestmark = pytest.mark.gpu

# B, Hq, Hk, Nq, Nk: one query tile a CTA; keys split over CTAs; the heads'
# queries in one tile; two query tiles a CTA (many pieces)
SIZES = {"one_tile": (1, 4, 4, 128, 384), "split": (1, 2, 1, 33, 5000),
         "packed": (2, 8, 2, 3, 640), "two_tiles": (2, 160, 80, 256, 384)}
COLUMNS = range(12)   # every place in the pattern of the exponentials' pairs


def step(q, k, v, dy):
    y, lse = fl.attn_fwd(q, k, v, save=True)
    return (y, lse, *fl.attn_bwd(q, k, v, y, dy, lse))


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("name", SIZES)
def test_nan_key(name, D, dt):
    """A NaN key of batch 0, key head 0: everything of its heads is NaN, the
    other heads keep their bits."""
    B, Hq, Hk, Nq, Nk = SIZES[name]
    if dt == F32 and name == "two_tiles":
        B, Hq, Hk = 1, 2, 1
    q, k, v, dy = tensors(dt, B, Hq, Hk, Nq, Nk, D, seed=30)
    G = Hq // Hk
    clean = step(q, k, v, dy)
    for col in COLUMNS:
        bad = k.clone()
        bad[0, 0, 128 + col, 3] = math.nan
        got = step(q, bad, v, dy)
        for what, g, c, heads in zip(("y", "lse", "dq", "dk", "dv"), got, clean, (G, G, G, 1, 1)):
            assert torch.isnan(g[0, :heads]).all(), (what, col)
            assert torch.equal(g[0, heads:], c[0, heads:]), (what, col)
            assert torch.equal(g[1:], c[1:]), (what, col)


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("D", [32, 64, 128])
@pytest.mark.parametrize("name", SIZES)
def test_infinite_key(name, D, dt):
    """Logits of +inf make their rows NaN; rows where they are -inf are those of
    the other keys."""
    B, Hq, Hk, Nq, Nk = SIZES[name]
    if dt == F32 and name == "two_tiles":
        B, Hq, Hk = 1, 2, 1
    q, k, v, _ = tensors(dt, B, Hq, Hk, Nq, Nk, D, seed=31)
    q[..., 3] = torch.where(q[..., 3] >= 0, 1.0, -1.0).to(dt)   # no 0 x inf
    up = q[..., 3] > 0
    for col in COLUMNS:
        at = 128 + col
        bad = k.clone()
        bad[:, :, at, 3] = math.inf
        y, lse = fl.attn_fwd(q, bad, v, save=True)
        assert torch.equal(torch.isnan(y).all(-1), up) and torch.equal(torch.isnan(y).any(-1), up)
        assert torch.equal(torch.isnan(lse), up)
        rest = [j for j in range(Nk) if j != at]
        ref = Attn(q, k[:, :, rest], v[:, :, rest])
        down = ~up.unsqueeze(-1)
        within(torch.where(down, y, 0.0), torch.where(down, ref.y, 0.0), ref.y_bound, "y")
        err = (lse.double() - ref.lse).abs()
        assert (err <= ref.lse_bound)[~up].all()


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_nan_query(dt):
    """A NaN query spoils its own row, and the gradients of the keys it sees."""
    q, k, v, dy = tensors(dt, 1, 2, 2, 200, 384, 64, seed=32)
    ref = Attn(q, k, v)
    (want, _, _), (bound, _, _) = ref.grads(dy)
    q[0, 0, 37, 5] = math.nan
    y, lse, dq, dk, dv = step(q, k, v, dy)
    row = torch.zeros(1, 2, 200, dtype=torch.bool, device=q.device)
    row[0, 0, 37] = True
    for t in (y, dq):
        assert torch.equal(torch.isnan(t).all(-1), row) and torch.equal(torch.isnan(t).any(-1), row)
    assert torch.equal(torch.isnan(lse), row)
    keep = ~row.unsqueeze(-1)
    within(torch.where(keep, y, 0.0), torch.where(keep, ref.y, 0.0), ref.y_bound, "y")
    within(torch.where(keep, dq, 0.0), torch.where(keep, want, 0.0), bound, "dq")
    assert torch.isnan(dk[0, 0]).all() and torch.isnan(dv[0, 0]).all()
    assert torch.isfinite(dk[0, 1]).all() and torch.isfinite(dv[0, 1]).all()


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("Nk", [300, 384])
def test_row_without_weight(Nk, dt):
    """Every logit -inf: as a query that sees no key, 0 and no gradient."""
    q, k, v, dy = tensors(dt, 1, 2, 2, 200, Nk, 64, seed=33)
    q[..., 3] = -1.0
    for low, what in ((2.0 ** 30, "the lowest weight"), (math.inf, "none")):
        k[..., 3] = low
        y, lse = fl.attn_fwd(q, k, v, save=True)
        if low == math.inf:
            assert not y.any() and (lse == -math.inf).all(), what
        else:
            assert torch.isfinite(y).all() and torch.isfinite(lse).all(), what
            continue
        k[..., 3] = 0.0   # what multiplies a weight of 0 is finite
        dq, dk, dv = fl.attn_bwd(q, k, v, y, dy, lse)
        assert not dq.any() and not dk.any() and not dv.any()
