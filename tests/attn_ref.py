"""The attention operators in 64 bits, with bounds on what a kernel's roundings
may add: the plain implementation of the operators' tests.

Bounds.  A rounding to type t is off by at most u_t = eps_t / 2 of the value
(bf16 2^-8, fp32 2^-24); a float32 sum of n terms by (n + 1) 2^-23 of the sum
of their magnitudes (any order; 2^-23 also covers a truncating adder).  With
  a      the largest sum of magnitudes behind one logit,
  e_p =  relative error of a probability: exp of a logit that is off by
         (D + 2) 2^-23 a, the log-sum-exp the same again, its sum of Nk terms,
         and the exponential itself (2^-21; bf16: the polynomial's 1e-4),
  r   =  u_bf16 for bf16 operands (P and dS are rounded for their products), 0
         for float32,
the elementwise bounds are those of ``forward`` and ``backward`` below.
"""
import math

import torch

U = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}
S = 2.0 ** -23


def visible(B, Nq, Nk, causal, q_lens, k_lens, device="cpu"):
    """[B,1,Nq,Nk]: the keys each query sees."""
    ql = torch.tensor(q_lens if q_lens is not None else [Nq] * B, device=device).view(B, 1, 1, 1)
    kl = torch.tensor(k_lens if k_lens is not None else [Nk] * B, device=device).view(B, 1, 1, 1)
    i = torch.arange(Nq, device=device).view(1, 1, Nq, 1)
    j = torch.arange(Nk, device=device).view(1, 1, 1, Nk)
    see = (i < ql) & (j < kl)
    return see & (j <= i + kl - ql) if causal else see


class Attn:
    """Reference values and bounds; inputs of any float type, padding rows may
    hold anything (they are cleared first)."""

    def __init__(self, q, k, v, scale=None, causal=False, q_lens=None, k_lens=None):
        self.dt = q.dtype
        B, Hq, Nq, D = q.shape
        Hk, Nk = k.shape[1], k.shape[2]
        self.G = Hq // Hk
        self.s = 1.0 / math.sqrt(D) if scale is None else scale
        self.see = visible(B, Nq, Nk, causal, q_lens, k_lens, q.device)
        row = lambda n, lens: None if lens is None else (  # noqa: E731
            torch.arange(n, device=q.device) < torch.tensor(lens, device=q.device).view(B, 1)
        ).view(B, 1, n, 1)
        self.mq, self.mk = row(Nq, q_lens), row(Nk, k_lens)
        self.q = self.clean(q, self.mq)
        self.k = self.clean(k, self.mk).repeat_interleave(self.G, 1)
        self.v = self.clean(v, self.mk).repeat_interleave(self.G, 1)
        a = self.s * self.q @ self.k.transpose(-1, -2)
        a = a.masked_fill(~self.see, -math.inf)
        self.lse = torch.logsumexp(a, -1)
        top = torch.where(torch.isinf(self.lse), 0.0, self.lse).unsqueeze(-1)
        self.p = torch.exp(a - top)
        self.y = self.p @ self.v
        mag = (self.s * self.q.abs() @ self.k.abs().transpose(-1, -2)).max().item()
        self.n = Nk
        self.nq = Nq
        self.e_p = 2 * (D + 2) * S * mag + (Nk + 1) * S + \
            (2.0 ** -21 if self.dt == torch.float32 else 2e-4)
        self.r = 0.0 if self.dt == torch.float32 else U[self.dt]
        self.D = D
        self.yabs = self.p @ self.v.abs()
        # before the output's rounding, and with it
        self.y_pure = (self.r + 2 * self.e_p + (Nk + 1) * S) * self.yabs + 1e-30
        self.y_bound = self.y_pure + U[self.dt] * self.y.abs()
        self.lse_bound = self.e_p + 2.0 ** -22 * torch.where(torch.isinf(self.lse), 0.0,
                                                             self.lse.abs()) + 1e-6

    @staticmethod
    def clean(t, mask):
        t = t.double()
        return t if mask is None else torch.where(mask, t, 0.0)

    def _heads(self, t):
        """Sum over the query heads of a key head."""
        B, H, N, D = t.shape
        return t.view(B, H // self.G, self.G, N, D).sum(2)

    def grads(self, dy, low=False):
        """(dq, dk, dv), their bounds; ``low``: delta comes from y and the
        remainder of its rounding, which is off by 2^-16 of y."""
        dy = self.clean(dy, self.mq)
        p, s, r, u = self.p, self.s, self.r, U[self.dt]
        dp = dy @ self.v.transpose(-1, -2)
        delta = (dy * self.y).sum(-1, keepdim=True)
        ds = p * (dp - delta)
        dv = self._heads(p.transpose(-1, -2) @ dy)
        dq = s * ds @ self.k
        dk = self._heads(s * ds.transpose(-1, -2) @ self.q)
        # dP and delta are float32 sums of D terms; delta sees the rounded y
        e_y = self.y_pure + U[self.dt] ** 2 * self.y.abs() if low else self.y_bound
        e_dp = (self.D + 1) * S * (dy.abs() @ self.v.abs().transpose(-1, -2))
        e_delta = (dy.abs() * (e_y + (self.D + 1) * S * self.y.abs())).sum(-1, keepdim=True)
        e_ds = (r + self.e_p + 4 * S) * ds.abs() + 2 * p * (e_dp + e_delta)
        nq, nk = (self.nq * self.G + 1) * S, (self.n + 1) * S
        t = ds.abs() + e_ds
        b_dv = self._heads((r + self.e_p + nq) * p.transpose(-1, -2) @ dy.abs()) + u * dv.abs()
        b_dq = s * (e_ds + nk * t) @ self.k.abs() + u * dq.abs()
        b_dk = self._heads(s * (e_ds + nq * t).transpose(-1, -2) @ self.q.abs()) + u * dk.abs()
        return (dq, dk, dv), tuple(b + 1e-30 for b in (b_dq, b_dk, b_dv))


def rotate(u, cos, sin, interleaved, sign=1.0):
    """Rotation of the first R = 2 cos.shape[-1] elements; cos, sin [..., N, R/2]."""
    half = cos.shape[-1]
    a, b = (u[..., 0:2 * half:2], u[..., 1:2 * half:2]) if interleaved else \
        (u[..., :half], u[..., half:2 * half])
    x, y = a * cos - sign * b * sin, b * cos + sign * a * sin
    turned = torch.stack((x, y), -1).flatten(-2) if interleaved else torch.cat((x, y), -1)
    return torch.cat((turned, u[..., 2 * half:]), -1)


class NormRope:
    """One of q, k through the norm and rotation: values, gradients, bounds.

    r = rsqrt(mean + eps) is off by (D + 3) 2^-23 (the sum, the mean, the
    reciprocal root's 2 ulp); a product or a rotation adds a few 2^-23 of the
    magnitudes that enter; the result is rounded once."""

    def __init__(self, x, w, cos, sin, eps, interleaved):
        self.dt, self.il = x.dtype, interleaved
        B, H, N, D = x.shape
        self.x = x.double()
        self.w = torch.ones(D, dtype=torch.float64, device=x.device) if w is None else w.double()
        self.c = self.sn = None
        if cos is not None:
            lift = lambda t: t.double().unsqueeze(1) if t.dim() == 3 else t.double()  # noqa: E731
            self.c, self.sn = lift(cos), lift(sin)
        self.rs = 1.0 / torch.sqrt((self.x ** 2).mean(-1, keepdim=True) + eps)
        self.e_r = (D + 6) * S
        u = self.w * self.x * self.rs
        self.y = self.turn(u)
        mag = u.abs() if self.c is None else rotate(u.abs(), self.c.abs(), -self.sn.abs(), self.il) \
            .abs().maximum(rotate(u.abs(), self.c.abs(), self.sn.abs(), self.il).abs())
        self.y_bound = self.e_r * mag + U[self.dt] * self.y.abs() + 1e-30

    def turn(self, u, sign=1.0):
        return u if self.c is None else rotate(u, self.c, self.sn, self.il, sign)

    def grads(self, dy):
        """(dx, dw), their bounds."""
        D, dy = self.x.shape[-1], dy.double()
        du = self.turn(dy, -1.0)
        mag = dy.abs() if self.c is None else \
            rotate(dy.abs(), self.c.abs(), self.sn.abs(), self.il).abs().maximum(
                rotate(dy.abs(), self.c.abs(), -self.sn.abs(), self.il).abs())
        g = du * self.w
        gm = mag * self.w.abs()
        m = (g * self.x).mean(-1, keepdim=True)
        dx = self.rs * (g - self.x * self.rs ** 2 * m)
        dw = (du * self.x * self.rs).sum((0, 1, 2))
        rows = self.x.shape[0] * self.x.shape[1] * self.x.shape[2]
        mm = (gm * self.x.abs()).mean(-1, keepdim=True)
        b_dx = (4 * self.e_r) * self.rs * (gm + self.x.abs() * self.rs ** 2 * mm) + \
            U[self.dt] * dx.abs() + 1e-30
        # sums of at most `rows` terms, in parts
        b_dw = (self.e_r + 4 * S + (rows + 1) * S) * (mag * self.x.abs() * self.rs).sum((0, 1, 2)) + \
            U[self.dt] * dw.abs() + 1e-30
        return (dx, dw), (b_dx, b_dw)


def within(got, ref, bound, what):
    """Every element of ``got`` within its bound of the reference."""
    got = got.double()
    assert torch.isfinite(got).all(), f"{what}: not finite"
    over = ((got - ref).abs() / bound).max().item()
    assert over <= 1.0, f"{what}: {over:.3f} of its bound"
