"""What the binding of the attention calls tells autograd, and what it refuses
because autograd would not learn of it."""
import pytest
import torch

import rank_latent_attention_flare_b200 as fl


def heads(device="cpu", dtype=torch.float32, B=1, H=2, N=20, D=32, seed=0):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return [torch.randn(B, H, N, D, device=device, generator=g).to(dtype) for _ in range(3)]


def test_angles_that_need_a_gradient_are_refused():
    q, k, _ = heads()
    cos, sin = torch.ones(20, 16), torch.zeros(20, 16)
    for c, s in ((cos.clone().requires_grad_(), sin), (cos, sin.clone().requires_grad_())):
        with pytest.raises(ValueError, match="no gradient"):
            fl.qk_norm_rope(q, k, None, None, c, s)


@pytest.mark.gpu
def test_angles_without_a_graph():
    """Where nothing is differentiated, learned angles are as good as others."""
    q, k, _ = heads("cuda")
    ang = torch.rand(20, 16, device="cuda")
    cos, sin = ang.cos().requires_grad_(), ang.sin().requires_grad_()
    want = fl.qk_norm_rope(q, k, None, None, cos.detach(), sin.detach())
    with torch.no_grad():
        got = fl.qk_norm_rope(q, k, None, None, cos, sin)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_a_scale_that_needs_a_gradient_is_refused():
    with pytest.raises(ValueError, match="no gradient"):
        fl.attn(*heads(), torch.tensor(0.5, requires_grad=True))


@pytest.mark.gpu
def test_outputs_written_in_place_are_counted():
    """A tensor that autograd saved and a call then overwrites: the backward
    reports it."""
    q, k, v = heads("cuda")
    w = torch.ones(32, device="cuda", requires_grad=True)
    for write in (lambda: fl.qk_norm_rope_fwd(q, k, out=(q, k)),
                  lambda: fl.attn_fwd(q, k, v, out=q)):
        loss = (w * q).sum()   # saves q
        was = q._version
        write()
        assert q._version > was
        with pytest.raises(RuntimeError, match="inplace"):
            loss.backward()
    assert k._version > 0


@pytest.mark.gpu
def test_outputs_of_a_graph_are_refused():
    """An output that autograd holds a history of would keep the old one."""
    q, k, v = heads("cuda")
    x = (2.0 * q).requires_grad_()
    for call in (lambda o: fl.attn_fwd(q, k, v, out=o),
                 lambda o: fl.qk_norm_rope_fwd(q, k, out=(o, torch.empty_like(k))),
                 lambda o: fl.qk_norm_rope_fwd(q, k, out=(torch.empty_like(k), o))):
        with pytest.raises(ValueError, match="gradient"):
            call(x)
    with torch.no_grad():
        assert fl.attn_fwd(q, k, v, out=x) is x
    with torch.inference_mode():
        y = torch.empty_like(q)
        fl.attn_fwd(q, k, v, out=y)
    assert torch.equal(x.detach(), y)


def test_a_misaligned_gradient_is_copied():
    """A gradient that begins inside a 16-byte group, contiguous or not."""
    from rank_latent_attention_flare_b200.attention import _grad_view
    buf = torch.arange(2 * 3 * 8 * 16 + 8, dtype=torch.bfloat16)
    assert buf.data_ptr() % 16 == 0
    for off in range(8):
        t = buf[off:off + 2 * 3 * 8 * 16].view(2, 3, 8, 16)
        for x in (t, t.transpose(1, 2)):
            got = _grad_view(x)
            assert got.data_ptr() % 16 == 0 and torch.equal(got, x)
            assert (got.data_ptr() == x.data_ptr()) == (off == 0)


@pytest.mark.gpu
def test_a_misaligned_gradient_through_autograd():
    q, k, v = (t.requires_grad_() for t in heads("cuda"))
    flat = torch.randn(q.numel() + 1, device="cuda")
    dy = flat[1:].view(q.shape)
    y = fl.attn(q, k, v)
    got = torch.autograd.grad(y, (q, k, v), dy, retain_graph=True)
    want = torch.autograd.grad(y, (q, k, v), dy.clone())
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    out = fl.qk_norm_rope(q, k)
    got = torch.autograd.grad(out, (q, k), (dy, dy), retain_graph=True)
    want = torch.autograd.grad(out, (q, k), (dy.clone(), dy.clone()))
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_without_a_graph_nothing_is_saved(monkeypatch):
    """Parameters need gradients, the call is made under no_grad: y alone."""
    import importlib
    att = importlib.import_module("rank_latent_attention_flare_b200.attention")
    asked = []

    def fake(q, k, v, scale=None, **kw):
        saving = kw.get("save") or kw.get("save_low")
        asked.append(bool(saving))
        return (q.clone(), q[..., 0].clone(), None) if saving else q.clone()
    monkeypatch.setattr(att, "attn_fwd", fake)
    q, k, v = (t.requires_grad_() for t in heads())
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            assert not fl.attn(q, k, v).requires_grad
    assert fl.attn(q, k, v).requires_grad
    assert asked == [False, False, True]
