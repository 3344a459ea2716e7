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
