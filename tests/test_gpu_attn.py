"""Softmax attention (attn) against the 64-bit definition: sizes, masks,
lengths, layouts, shared heads, graphs, streams."""
import math

import pytest
import torch

import rank_latent_attention_flare_b200 as fl
from attn_ref import Attn, within

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF, F32 = torch.bfloat16, torch.float32


def tensors(dt, B, Hq, Hk, Nq, Nk, D, seed=0, layout="bhnd", sharp=1.5):
    """q, k, v, dy; layout bnhd: views of [B,N,H,D] projections."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def one(H, N, f=1.0):
        shape = (B, N, H, D) if layout == "bnhd" else (B, H, N, D)
        t = (f * torch.randn(shape, device=DEV, generator=g)).to(dt)
        return t.transpose(1, 2) if layout == "bnhd" else t
    return one(Hq, Nq, sharp), one(Hk, Nk), one(Hk, Nk), one(Hq, Nq)


def dev_lens(lens):
    return None if lens is None else torch.tensor(lens, dtype=torch.int32, device=DEV)


def poison(t, lens):
    """NaN in the rows past the lengths: they must not matter."""
    if lens is not None:
        for b, n in enumerate(lens):
            t[b, :, n:] = math.nan


def check(q, k, v, dy, causal=False, q_lens=None, k_lens=None, scale=None, backward=True):
    for t, lens in ((q, q_lens), (dy, q_lens), (k, k_lens), (v, k_lens)):
        poison(t, lens)
    kw = dict(causal=causal, q_lens=dev_lens(q_lens), k_lens=dev_lens(k_lens))
    ref = Attn(q, k, v, scale, causal, q_lens, k_lens)
    B, Hq, Nq, D = q.shape
    Hk, Nk = k.shape[1], k.shape[2]
    ws = torch.empty(fl.attn_workspace_size(False, B, Hq, Hk, Nq, Nk, D, q.dtype),
                     dtype=torch.uint8, device=DEV)
    y, lse, low = fl.attn_fwd(q, k, v, scale, save_low=True, workspace=ws, **kw)
    assert fl.device_status(ws) == 0
    within(y, ref.y, ref.y_bound, "y")
    if low is None:
        assert q.dtype == F32
    else:   # y and its remainder together are as good as before the rounding
        within(y.double() + low.double(), ref.y, ref.y_pure + 2.0 ** -16 * ref.y.abs(), "y + low")
        poison(low, q_lens)
    empty = torch.isinf(ref.lse)
    assert torch.equal(torch.isinf(lse) & (lse < 0), empty)
    assert not y[empty].any()
    err = (torch.where(empty, 0.0, lse.double()) - torch.where(empty, 0.0, ref.lse)).abs()
    assert (err <= ref.lse_bound).all()
    if not backward:
        return
    poison(y, q_lens)   # y and dy are not read past the lengths
    ws = torch.empty(fl.attn_workspace_size(True, B, Hq, Hk, Nq, Nk, D, q.dtype),
                     dtype=torch.uint8, device=DEV)
    for rest in (None, low):
        got = fl.attn_bwd(q, k, v, y, dy, lse, scale, workspace=ws, y_low=rest, **kw)
        assert fl.device_status(ws) == 0
        want, bounds = ref.grads(dy, low=rest is not None)
        for name, a, b, e in zip(("dq", "dk", "dv"), got, want, bounds):
            within(a, b, e, name)


# B, Hq, Hk, Nq, Nk, D, causal, q_lens, k_lens
CASES = {
    "one_token": (3, 8, 2, 1, 777, 64, True, None, None),
    "one_key": (2, 2, 2, 5, 1, 32, False, None, None),
    "one_by_one": (1, 1, 1, 1, 1, 8, True, None, None),
    "few_tokens": (2, 8, 2, 5, 700, 128, True, None, [700, 333]),
    "tile_edges": (1, 2, 1, 128, 256, 64, True, None, None),
    "past_the_edge": (1, 2, 1, 129, 257, 64, True, None, None),
    "before_the_edge": (1, 2, 1, 127, 255, 64, False, None, None),
    "d24": (2, 3, 1, 200, 190, 24, True, None, None),
    "d40": (1, 2, 2, 65, 300, 40, False, None, None),
    "d72": (1, 2, 2, 140, 140, 72, True, None, None),
    "d80": (2, 4, 2, 333, 301, 80, False, None, [301, 12]),
    "d96": (1, 2, 1, 77, 513, 96, True, None, None),
    "d128": (2, 4, 2, 300, 300, 128, True, None, None),
    "more_queries_than_keys": (2, 2, 1, 400, 150, 64, True, None, None),
    "empty_batch": (3, 2, 2, 130, 130, 64, True, [130, 0, 7], [130, 5, 0]),
    "no_keys_at_all": (2, 2, 1, 40, 60, 32, False, None, [0, 0]),
    "ragged": (4, 4, 4, 500, 500, 32, False, [500, 1, 129, 384], [1, 500, 128, 383]),
    "ragged_causal": (4, 4, 1, 300, 600, 64, True, [300, 1, 129, 256], [600, 2, 60, 257]),
    "five_shared": (1, 10, 2, 150, 150, 48, True, None, None),
    "split_keys": (1, 2, 1, 33, 9000, 64, False, None, None),
    "split_queries": (1, 4, 1, 3000, 40, 128, False, None, None),
    # more key tiles than SMs, one or a few query tiles each
    "latents": (2, 4, 4, 100, 9000, 64, False, None, [9000, 4097]),
    "latents_shared": (3, 8, 2, 130, 7000, 32, False, [130, 0, 128], [1, 7000, 6500]),
    "window_of_keys": (2, 4, 2, 200, 9000, 64, True, [200, 77], [8999, 150]),
}


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
@pytest.mark.parametrize("name", CASES)
def test_against_definition(name, dt):
    B, Hq, Hk, Nq, Nk, D, causal, q_lens, k_lens = CASES[name]
    layout = "bnhd" if len(name) % 2 else "bhnd"
    check(*tensors(dt, B, Hq, Hk, Nq, Nk, D, seed=len(name), layout=layout), causal, q_lens,
          k_lens)


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_scale_and_large_logits(dt):
    # rows whose maximum grows from tile to tile, far apart in size
    q, k, v, dy = tensors(dt, 1, 2, 2, 150, 1000, 64, seed=3, sharp=4.0)
    k *= torch.linspace(0.1, 3.0, 1000, device=DEV).view(1, 1, -1, 1).to(dt)
    check(q, k, v, dy, scale=0.5)
    check(q, -k, v, dy, causal=True, scale=0.5)


@pytest.mark.parametrize("D", [64, 128])
def test_many_heads(D):
    """More batch elements times heads than a grid has rows, one token each."""
    q, k, v, dy = tensors(BF, 1100, 64, 8, 1, 20, D, seed=20)
    check(q, k, v, dy, causal=True, k_lens=[1 + i % 20 for i in range(1100)])


def test_second_derivative_is_refused():
    q, k, v, dy = (t.requires_grad_() for t in tensors(F32, 1, 1, 1, 8, 8, 32, seed=21))
    (dq,) = torch.autograd.grad(fl.attn(q, k, v), q, dy, create_graph=True)
    with pytest.raises(RuntimeError):
        torch.autograd.grad(dq.sum(), k)


def test_key_gradients_alone():
    """A frozen query, a frozen cache: only what needs a gradient gets one."""
    q, k, v, dy = tensors(BF, 2, 4, 2, 70, 200, 64, seed=22)
    ref = Attn(q, k, v)
    want, bounds = ref.grads(dy, low=True)
    for which in ((0,), (1,), (2,), (1, 2)):
        leaves = [t.detach().requires_grad_(i in which) for i, t in enumerate((q, k, v))]
        got = torch.autograd.grad(fl.attn(*leaves), [leaves[i] for i in which], dy)
        for g, i in zip(got, which):
            within(g, want[i], bounds[i], "qkv"[i])


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_shared_inputs(dt):
    """Latents shared by the batch, one key head expanded over all."""
    q, k, v, dy = tensors(dt, 3, 4, 4, 100, 300, 64, seed=5)
    check(q[:1].expand(3, 4, 100, 64), k[:, :1].expand(3, 4, 300, 64), v[:1].expand(3, 4, 300, 64),
          dy)
    check(q[:1, :1].expand(3, 4, 100, 64), k, v, dy[:, :1].expand(3, 4, 100, 64), causal=True)
    one = q[:, :, :1]
    check(one[:, :1].expand(3, 4, 1, 64), k[:, :2], v[:, :2], dy[:, :, :1])


def test_long_strides():
    """A batch stride past 32 bits of elements; a sliced interleaved buffer."""
    step = (1 << 32) + 64
    buf = torch.empty(step + 2 * 300 * 64, dtype=BF, device=DEV)
    q, k, v, dy = tensors(BF, 2, 4, 2, 200, 300, 64, seed=6)
    far = torch.as_strided(buf, (2, 2, 300, 64), (step, 300 * 64, 64, 1))
    far.copy_(k)
    qkv = torch.empty(2, 300, 3, 2, 64, dtype=BF, device=DEV)
    qkv[:, :, 2] = v.transpose(1, 2)
    check(q, far, qkv[:, :, 2].transpose(1, 2), dy, causal=True)


def test_rows_behind_an_output_stay():
    """Only the output's own rows are written."""
    q, k, v, _ = tensors(BF, 2, 2, 1, 130, 200, 64, seed=7)
    buf = torch.full((2, 2, 160, 64), 7.0, dtype=BF, device=DEV)
    fl.attn_fwd(q, k, v, out=buf[:, :, 16:146])
    ref = Attn(q, k, v)
    within(buf[:, :, 16:146], ref.y, ref.y_bound, "y")
    assert (buf[:, :, :16] == 7.0).all() and (buf[:, :, 146:] == 7.0).all()


def test_bad_length_is_clamped_and_reported():
    q, k, v, _ = tensors(BF, 2, 2, 2, 40, 100, 32, seed=8)
    ws = torch.empty(fl.attn_workspace_size(False, 2, 2, 2, 40, 100, 32, BF), dtype=torch.uint8,
                     device=DEV)
    y = fl.attn_fwd(q, k, v, k_lens=dev_lens([101, -3]), workspace=ws)
    with pytest.raises(fl.FlareError):
        fl.device_status(ws)
    assert not y[1].any()
    assert torch.equal(y, fl.attn_fwd(q, k, v, k_lens=dev_lens([100, 0])))


@pytest.mark.parametrize("dt", [F32, BF], ids=["fp32", "bf16"])
def test_repeatable_and_parts(dt):
    """The same bits every time; dq alone, dk and dv alone."""
    q, k, v, dy = tensors(dt, 2, 4, 2, 300, 900, 64, seed=9)
    y, lse = fl.attn_fwd(q, k, v, causal=True, save=True)
    a = fl.attn_bwd(q, k, v, y, dy, lse, causal=True)
    b = fl.attn_bwd(q, k, v, y, dy, lse, causal=True)
    assert torch.equal(y, fl.attn_fwd(q, k, v, causal=True))
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    dq, none, none2 = fl.attn_bwd(q, k, v, y, dy, lse, causal=True, need_dkv=False)
    assert none is None and none2 is None and torch.equal(dq, a[0])
    none, dk, dv = fl.attn_bwd(q, k, v, y, dy, lse, causal=True, need_dq=False)
    assert none is None and torch.equal(dk, a[1]) and torch.equal(dv, a[2])


def test_autograd_and_differences():
    """Through autograd, against the formula and central differences of the
    64-bit definition (step 1e-5: truncation about 1e-10 of the third
    derivative, rounding 1e-11)."""
    q, k, v, dy = tensors(F32, 2, 4, 2, 60, 70, 32, seed=10)
    lens = [70, 33]
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    y = fl.attn(*leaves, causal=True, k_lens=dev_lens(lens))
    grads = torch.autograd.grad(y, leaves, dy)
    ref = Attn(q, k, v, causal=True, k_lens=lens)
    want, bounds = ref.grads(dy)
    for a, b, e, name in zip(grads, want, bounds, "qkv"):
        within(a, b, e, "d" + name)
    gen = torch.Generator(device=DEV)
    gen.manual_seed(11)
    for which in range(3):
        d = torch.randn(leaves[which].shape, device=DEV, generator=gen, dtype=torch.float64)
        h = 1e-5

        def loss(step):
            x = [q.double(), k.double(), v.double()]
            x[which] = x[which] + step * d
            return (Attn.__new__(Attn).plain(x, lens) * dy.double()).sum().item()
        num = (loss(h) - loss(-h)) / (2 * h)
        got = (grads[which].double() * d).sum().item()
        slack = (bounds[which] * d.abs()).sum().item()
        assert abs(got - num) <= slack + 1e-6 * abs(num) + 1e-6


def _plain(self, x, lens):
    from attn_ref import visible
    q, k, v = x
    G = q.shape[1] // k.shape[1]
    k, v = k.repeat_interleave(G, 1), v.repeat_interleave(G, 1)
    see = visible(q.shape[0], q.shape[2], k.shape[2], True, None, lens, q.device)
    a = (q @ k.transpose(-1, -2) / math.sqrt(q.shape[-1])).masked_fill(~see, -math.inf)
    p = torch.softmax(a, -1).nan_to_num(0.0)   # rows without keys
    return p @ v


Attn.plain = _plain


def test_no_gradient_and_expanded_leaves():
    q, k, v, dy = tensors(BF, 2, 4, 1, 100, 120, 64, seed=12)
    with torch.no_grad():
        y0 = fl.attn(q, k, v)
    lat = q[:1].clone().requires_grad_()
    y = fl.attn(lat.expand(2, 4, 100, 64), k, v)
    y.sum().backward()   # a gradient with zero strides
    assert torch.equal(y[0], y0[0])
    ref = Attn(lat.detach().expand(2, 4, 100, 64), k, v)
    (dq, _, _), (bq, _, _) = ref.grads(torch.ones_like(y))
    # the two batch elements' gradients are rounded, added and rounded again
    within(lat.grad, dq.sum(0, keepdim=True),
           bq.sum(0, keepdim=True) + 2.0 ** -8 * (dq.abs() + bq).sum(0, keepdim=True), "dlat")


def test_captured_and_replayed():
    """Two graphs of the whole step, replayed on new inputs in turn."""
    q, k, v, dy = tensors(BF, 1, 4, 2, 200, 700, 64, seed=13)
    fl.attn_fwd(q, k, v)

    def step():
        y, lse = fl.attn_fwd(q, k, v, causal=True, save=True)
        return (y, *fl.attn_bwd(q, k, v, y, dy, lse, causal=True))
    graphs, outs = [], []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(step())
        graphs.append(g)
    for seed in (14, 15):
        for t, n in zip((q, k, v, dy), tensors(BF, 1, 4, 2, 200, 700, 64, seed=seed)):
            t.copy_(n)
        for g in graphs:
            g.replay()
        want = step()
        torch.cuda.synchronize()
        for out in outs:
            assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_backward_captured_through_autograd():
    q, k, v, dy = tensors(BF, 1, 2, 2, 150, 150, 32, seed=16)
    leaves = [t.requires_grad_() for t in (q, k, v)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        torch.autograd.grad(fl.attn(*leaves), leaves, dy)
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = torch.autograd.grad(fl.attn(*leaves), leaves, dy)
    g.replay()
    want = torch.autograd.grad(fl.attn(*leaves), leaves, dy)
    assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_two_streams_at_once():
    sets = [tensors(BF, 1, 4, 2, 64, 4000, 64, seed=s) for s in (17, 18)]
    want = [fl.attn_fwd(*s[:3]) for s in sets]
    streams = [torch.cuda.Stream() for _ in sets]
    torch.cuda.synchronize()
    got = [[fl.attn_fwd(*s[:3], stream=st) for _ in range(5)] for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        assert all(torch.equal(w, x) for x in g)
