"""64-bit references of the W8A8 products and the MoE router, and the bounds
of their results' errors.  CPU tensors in, CPU tensors out."""
import torch

F16, BF16, F32 = 0, 1, 2
TORCH = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}
U32 = 2.0 ** -24                       # half a step of fp32, relative


def half_step(td):
    return torch.finfo(td).eps / 2


def pack8(w):
    """The 8-bit weight layout from codes w [E][K][N] (int8): 2048-byte tiles
    (expert, 16-column block, 128-row group), slot 16 c + j holds rows
    32 c .. 32 c + 31 of column j, stored as q + 128."""
    E, K, N = w.shape
    t = w.contiguous().view(torch.uint8).view(E, K // 128, 4, 32, N // 16, 16)
    return (t.permute(0, 4, 1, 2, 5, 3) ^ 128).contiguous()


def quantize(x):
    """Codes (float64) and fp32 scales of the rows of x."""
    top = x.float().abs().amax(1)
    bad = ~torch.isfinite(x.float()).all(1)
    s = top / torch.tensor(127.0)                           # fp32 division
    div = torch.where((s == 0) | bad, torch.ones_like(s), s).double()
    q = torch.round(torch.nan_to_num(x.double(), 0, 0, 0) / div[:, None]).clamp(-127, 127)
    q[(s == 0) | bad] = 0
    return q, torch.where(bad, torch.full_like(s, float("nan")), s)


def gemm(q, s, w, sw, bias=None):
    """(y, sum part) in float64."""
    part = (q.double() @ w.double()) * s.double()[:, None] * sw.double()
    return (part if bias is None else part + bias.double()), part


def gemm_bound(y, part, td):
    """|result - y|: the sum to fp32, the scales' product, their product and the
    bias addition are off by half a step of fp32 each, then comes one rounding (below the
    type's normal numbers half of its smallest step, and a step of fp32's)."""
    tiny = torch.finfo(td)
    v = 4 * U32 * part.abs() + U32 * y.abs()
    return v * (1 + half_step(td)) + half_step(td) * y.abs() + tiny.smallest_normal * tiny.eps / 2 + 2.0 ** -149


def softmax_parts(z):
    z = z.double()
    top = z.amax(1, keepdim=True)
    e = torch.exp(z - top)
    return e / e.sum(1, keepdim=True)


def kinds(z, mask):
    """Per token: 0 a distribution, 1 nothing (padding or every logit -inf), 2 NaN."""
    z = z.float()
    k = torch.zeros(z.shape[0], dtype=torch.int64)
    k[(z == float("-inf")).all(1)] = 1
    k[torch.isnan(z).any(1) | (z == float("inf")).any(1)] = 2
    if mask is not None:
        k[mask == 0] = 1
    return k


def route(z, topk, renorm, mask=None):
    """ids, weights, counts [E + 1], loss, all from the definitions."""
    T, E = z.shape
    kind = kinds(z, mask)
    ok = kind == 0
    zz = torch.where(ok[:, None], z.double(), torch.zeros((), dtype=torch.float64))
    p = softmax_parts(zz)
    order = torch.sort(zz, dim=1, descending=True, stable=True)[1][:, :topk]
    got = zz.gather(1, order)
    ids = torch.where(ok[:, None] & (got > float("-inf")), order, torch.full_like(order, -1))
    w = torch.where(ids >= 0, p.gather(1, order), torch.zeros((), dtype=torch.float64))
    if renorm:
        w = w / torch.where(w.sum(1, keepdim=True) > 0, w.sum(1, keepdim=True), torch.ones((), dtype=torch.float64))
    w[kind == 2] = float("nan")
    cnt = torch.bincount(ids[ids >= 0].reshape(-1), minlength=E)
    tokens = int((kind != 1).sum())
    if bool((kind == 2).any()):
        loss = float("nan")
    elif int(cnt.sum()) == 0:
        loss = 0.0
    else:
        loss = float(E * (cnt.double() / cnt.sum() * p[ok].sum(0) / tokens).sum())
    return ids.to(torch.int32), w, torch.cat((cnt, torch.tensor([tokens]))).to(torch.int32), loss


def spread(z):
    """Distance of every logit from its row's maximum; 0 where there is none or where the
    exponential is below fp32's smallest step (104 > 149 ln 2)."""
    z = z.double()
    f = torch.where(torch.isfinite(z), z, torch.full_like(z, float("-inf")))
    d = f.amax(1, keepdim=True) - f
    return torch.where(d < 104, d, torch.zeros_like(d))


def prob_bound(z):
    """Relative error of a softmax weight, in half steps of fp32.  The difference d = max - z and
    its product with log2(e) round once each, and log2(e) = 1.44269504 in fp32 is off by 1.93e-8, less than
    a quarter of a half step: |d| (1 + 1 + 1/4) in the exponent; exp2 is within one step (2).
    The sum over the row carries the mean of these errors by weight: the mean of d under the
    softmax is at most its entropy, ln 1024 < 7.  That sum goes through at most 16 + 6 additions,
    then a reciprocal, a product and, renormalized, a sum of the chosen ones and a division."""
    far = spread(z).amax()
    return U32 * (2.25 * (far + min(float(far), 7.0)) + 2 + 2 + 22 + 3 + 12)


def route_backward(z, ids, w, counts, dw, dloss, renorm, mask=None):
    """dlogits and the sum of the magnitudes that enter each (for its error bound)."""
    T, E = z.shape
    kind = kinds(z, mask)
    ok = kind == 0
    zz = torch.where(ok[:, None], z.double(), torch.zeros((), dtype=torch.float64))
    p = softmax_parts(zz)
    h = torch.zeros((T, E), dtype=torch.float64)
    if dloss is not None:
        c, tv = counts[:E].double(), int(counts[E])
        if float(c.sum()) > 0 and tv > 0:
            h += dloss * (E * c - c.sum()) / (c.sum() * tv)
    sel = torch.zeros((T, E), dtype=torch.float64)
    if dw is not None:
        held = ids >= 0
        at = ids.long().clamp(min=0)
        wd, g = w.double(), dw.double()
        v = wd * (g - torch.where(held, wd * g, torch.zeros_like(g)).sum(1, keepdim=True)) if renorm else g
        sel.scatter_add_(1, at, torch.where(held, v, torch.zeros_like(v)))
    hh = h if renorm else h + sel
    dz = p * (hh - (p * hh).sum(1, keepdim=True))
    size = p * (hh.abs() + (p * hh.abs()).sum(1, keepdim=True))
    if renorm:
        dz = dz + sel
        if dw is not None:
            a = torch.where(held, wd.abs() * (g.abs() + (wd * g).abs().sum(1, keepdim=True)), torch.zeros_like(g))
            size = size + torch.zeros_like(size).scatter_add_(1, at, a)
    dz[kind == 1] = 0
    size[kind == 1] = 0
    dz[kind == 2] = float("nan")
    return dz, size
