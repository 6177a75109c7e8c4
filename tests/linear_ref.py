"""Plain 64-bit implementation of the fused linear operators and the inputs of
their tests (CPU, torch float64; independent of the library's code)."""
from __future__ import annotations

import math
from dataclasses import dataclass

import torch

F16, BF16 = 0, 1
TD = {F16: torch.float16, BF16: torch.bfloat16}
#: largest relative error of one rounding to the type (half a unit in the last place)
ULP = {F16: 2.0 ** -11, BF16: 2.0 ** -8}
NONE, RELU, SILU, GELU, GELU_TANH = range(5)
ACTS = (NONE, RELU, SILU, GELU, GELU_TANH)


def act(v, a):
    """act(v) and act'(v) from their definitions."""
    if a == NONE:
        return v.clone(), torch.ones_like(v)
    if a == RELU:
        return v.clamp(min=0), torch.where(torch.isnan(v), v, (v > 0).to(v.dtype))      # NaN stays NaN
    if a == SILU:
        s = 1 / (1 + torch.exp(-v))
        return v * s, s * (1 + v * (1 - s))
    if a == GELU:
        c = 0.5 * (1 + torch.erf(v / math.sqrt(2)))
        return v * c, c + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
    k = math.sqrt(2 / math.pi)
    t = torch.tanh(k * (v + 0.044715 * v ** 3))
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)


@dataclass
class Layer:
    K: int
    N: int
    group: int
    dt: int
    q: torch.Tensor          # [K][N] stored nibble values: 0..15 with zero, -8..7 without
    scale: torch.Tensor      # [K/group][N], dtype
    zero: torch.Tensor | None
    bias: torch.Tensor | None

    def weights(self):
        q = self.q.double()
        if self.zero is not None:
            q = q - self.zero.double().repeat_interleave(self.group, 0)
        return q * self.scale.double().repeat_interleave(self.group, 0)

    def packed_plain(self):
        """[K][N/2] bytes: low nibble = even column."""
        u = (self.q & 15).to(torch.uint8)
        return u[:, 0::2] | (u[:, 1::2] << 4)

    def zero_packed(self):
        if self.zero is None:
            return None
        z = self.zero.to(torch.uint8)
        return z[:, 0::2] | (z[:, 1::2] << 4)


def layer(K, N, group=128, dt=BF16, zero=False, bias=True, seed=0):
    g = torch.Generator().manual_seed(seed)
    G = K // group
    if zero:
        q = torch.randint(0, 16, (K, N), generator=g)
        z = torch.randint(6, 10, (G, N), generator=g)
    else:
        q, z = torch.randint(-8, 8, (K, N), generator=g), None
    s = (torch.rand((G, N), generator=g) * 0.008 + 0.002).to(TD[dt])
    b = (torch.randn(N, generator=g) * 0.5).to(TD[dt]) if bias else None
    return Layer(K, N, group, dt, q, s, z, b)


def normal(rows, cols, std, dt, seed):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn((rows, cols), generator=g) * std).to(TD[dt])


def pre(x, L):
    p = x.double() @ L.weights()
    return p if L.bias is None else p + L.bias.double()


def ep(x, L, a, residual=None):
    p = pre(x, L)
    y = act(p, a)[0]
    return (y if residual is None else y + residual.double()), p


def glu(x, L, a):
    h = pre(x, L)
    g, u = h.chunk(2, 1)
    return act(g, a)[0] * u, h


def ep_backward(dy, p, L, a, addend=None):
    """dx, dpre, dbias."""
    d = dy.double() if a == NONE else dy.double() * act(p.double(), a)[1]
    dx = d @ L.weights().t()
    return (dx if addend is None else dx + addend.double()), d, d.sum(0)


def glu_backward(da, h, L, a, addend=None):
    g, u = h.double().chunk(2, 1)
    f, df = act(g, a)
    d = torch.cat((da.double() * u * df, da.double() * f), 1)
    dx = d @ L.weights().t()
    return (dx if addend is None else dx + addend.double()), d, d.sum(0)


# ---- tolerances -------------------------------------------------------------------
# One rounding to the type: ULP |ref|.  The fp32 sums: in code units a chain over
# one 128-row group holds values up to about 143 sum |x| (the decode kernel
# multiplies codes biased by 128) and rounds each of its 128 additions by at
# most 2^-24 of that, against a result of 4.6 sqrt(128) |x|; as independent
# errors that is 143 * 0.8 * 128 * 2^-24 * sqrt(128) / sqrt(12) / (4.6 sqrt(128)) = 6e-5
# of the result's size: 2^-12 (four of those) times its rms is allowed.  The
# activations' slopes are below 1.13, the gated product multiplies by the other
# half, whose own error enters the same way.
SUM = 2.0 ** -12


def tol_sum(p):
    return SUM * p.square().mean().sqrt() * torch.ones_like(p)


def tol_ep(y, p, dt):
    return ULP[dt] * 1.01 * y.abs() + 1.13 * tol_sum(p)


def tol_glu(y, h, dt):
    g, u = h.chunk(2, 1)
    e = tol_sum(h)
    eg, eu = e.chunk(2, 1)
    return ULP[dt] * 1.01 * y.abs() + 1.13 * eg * u.abs() + eu * g.abs() + eg * eu


def tol_dx(dx, d, L, dt):
    """d and W each rounded to the type: independent relative errors of
    standard deviation at most ULP / sqrt 3, so the sum's is
    ULP sqrt(2/3) sqrt(sum d^2 w^2); six of those, and the result's own
    rounding."""
    q = (d.square() @ L.weights().square().t()).sqrt()
    return ULP[dt] * 1.01 * dx.abs() + 6 * math.sqrt(2 / 3) * ULP[dt] * q + 2.0 ** -24


def tol_d(d, dt):
    """One rounding of a value computed in fp32 (a few 2^-23 relative to the
    size of its factors, which reach 1.13 |dy| (1 + |v|))."""
    tiny = 2.0 ** -24 if dt == F16 else 0.0       # subnormal fp16 spacing
    return ULP[dt] * 1.01 * d.abs() + 2.0 ** -18 * d.abs().amax() + tiny


def close(got, ref, tol, what):
    got = got.double().cpu()
    bad = (got - ref).abs() > tol
    worst = ((got - ref).abs() / tol.clamp_min(1e-300)).max().item() if ref.numel() else 0.0
    print(f"[linear] {what}: worst error / tolerance {worst:.3f}", flush=True)
    assert torch.isfinite(got).all(), what
    assert not bad.any(), (what, worst, bad.nonzero()[:4].tolist())
