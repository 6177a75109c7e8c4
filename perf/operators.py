"""Workloads of the fused W4A16 linear operators: what is timed and compared.

Four operators around one int4 weight matrix W [K][N] (one 16-bit scale and
optionally one uint4 zero point per `group` rows and column):

  ep       y = act(x . W + bias) + residual, pre = x . W + bias kept for a
           backward pass when `save` is set
  ep_bwd   dpre = dy * act'(pre) (dy itself without an activation),
           dbias = column sums of dpre, dx = dpre . W^T + addend
  glu      W holds gate columns then up columns (N = 2 I):
           h = x . W + bias, a = act(h_gate) * h_up, h kept when `save` is set
  glu_bwd  dh = (da * h_up * act'(h_gate), da * act(h_gate)),
           dbias = column sums of dh, dx = dh . W^T + addend

With `own` False every operator runs in plain torch operations in 32 bits,
rounded once at the end; with `own` True it is one call of this library.
"""
import math

import torch

own = False

F16, BF16 = 0, 1
NONE, RELU, SILU, GELU, GELU_TANH = range(5)
_TORCH = {F16: torch.float16, BF16: torch.bfloat16}


def _case(name, op, M, K, N, act, dt=BF16, group=128, zero=False, bias=True, residual=False, save=False, pad=0):
    """N counts the columns of W (twice the width for glu); pad: extra elements
    in every row of x and dy (a slice of a wider buffer)."""
    return {"name": name, "op": op, "M": M, "K": K, "N": N, "act": act, "dt": dt, "group": group, "zero": zero,
            "bias": bias, "residual": residual, "save": save, "pad": pad}


def listed():
    return [
        # a tiny projection: launch latency is all there is
        _case("ep tiny", "ep", 4, 256, 256, GELU, dt=F16),
        # down projection of one decoded token, added to the residual stream
        _case("ep decode 1", "ep", 1, 14336, 4096, NONE, zero=True, bias=False, residual=True),
        # the same weights for a ragged short prompt: the long K is split
        _case("ep prompt 77", "ep", 77, 14336, 4096, NONE, zero=True, bias=False, residual=True),
        # training forward of a square projection with its pre-activation kept
        _case("ep train 4096", "ep", 4096, 4096, 4096, GELU_TANH, save=True),
        # gate/up projection of one decoded token and of a batch of 16
        _case("glu decode 1", "glu", 1, 4096, 28672, SILU, zero=True, bias=False),
        _case("glu decode 16", "glu", 16, 4096, 28672, SILU, zero=True, bias=False),
        # an expert-sized gate/up projection over an odd number of tokens
        _case("glu 333", "glu", 333, 2048, 2816, GELU, dt=F16, pad=64),
        # training forward of the gate/up projection, h kept
        _case("glu train 4096", "glu", 4096, 4096, 28672, SILU, save=True, bias=False),
        # backward of a small biased layer, an odd number of rows
        _case("ep_bwd 61", "ep_bwd", 61, 1024, 2048, RELU, dt=F16, group=256, zero=True),
        # backward of the down projection
        _case("ep_bwd 2048", "ep_bwd", 2048, 14336, 4096, NONE, bias=False),
        # backward of the expert-sized gate/up projection with biases
        _case("glu_bwd 519", "glu_bwd", 519, 2048, 2816, GELU_TANH, zero=True, residual=True),
        # backward of the gate/up projection, the residual's gradient added
        _case("glu_bwd 4096", "glu_bwd", 4096, 4096, 28672, SILU, bias=False, residual=True),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    """Any operator, type, activation and option; rows 1..4096, K 128..14336,
    widths 64..14336 (N up to 28672 for glu), within the largest listed cost."""
    op = rng.choice(["ep", "ep_bwd", "glu", "glu_bwd"])
    while True:
        M = max(1, min(4096, round(_log(rng, 1, 4097))))
        K = 128 * max(1, round(_log(rng, 128, 14336) / 128))
        W = 64 * max(1, round(_log(rng, 64, 14336) / 64))
        N = 2 * W if op.startswith("glu") else W
        if K * N >= 1 << 16 and M * K * N <= 4096 * 4096 * 28672 // 2 and K * N <= 4096 * 28672:
            break
    group = rng.choice([g for g in (128, 256, 512, K) if K % g == 0])
    c = _case("", op, M, K, N, rng.choice([NONE, RELU, SILU, GELU, GELU_TANH]), rng.choice([F16, BF16]), group,
              rng.random() < 0.5, rng.random() < 0.5, rng.random() < 0.5 and op != "glu", rng.random() < 0.5,
              rng.choice([0, 0, 8, 192]))
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------

def _pack(w, K, N):
    """The library's documented weight layout from codes w [K][N] (uint8,
    0..15): 1024-byte tiles (16-column block, 128-row group), slot 16 c + j
    holds column j, rows 32 c .. 32 c + 31, word t rows 8 t + i at bit
    4 (i / 2) + 16 (i % 2)."""
    t = w.view(K // 128, 4, 4, 4, 2, N // 16, 16)          # g, c, t, i / 2, i % 2, nb, j
    t = t.permute(5, 0, 1, 6, 2, 4, 3).contiguous()        # nb, g, c, j, t, i % 2, i / 2
    t = t.view(-1, 2)
    return (t[:, 0] | (t[:, 1] << 4)).contiguous()


def prepare(case, seed):
    c, dev = case, "cuda"
    M, K, N, td = c["M"], c["K"], c["N"], _TORCH[c["dt"]]
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 13)

    def normal(rows, cols, std, pad=0):
        return (torch.randn((rows, cols + pad), device=dev, generator=gen) * std).to(td)[:, :cols]

    codes = torch.randint(0, 16, (K, N), device=dev, dtype=torch.uint8, generator=gen)
    packed = _pack(codes, K, N)
    zero = None
    if c["zero"]:                                          # unsigned codes with zero points 6..9
        z = torch.randint(6, 10, (K // c["group"], N), device=dev, dtype=torch.uint8, generator=gen)
        zero = z[:, 0::2] | (z[:, 1::2] << 4)
    else:                                                  # the same codes as signed nibbles (u - 8)
        codes = codes ^ 8
    s = {
        "case": dict(c), "packed": packed, "zero": zero,
        "w": codes[:, 0::2] | (codes[:, 1::2] << 4),       # plain layout: [K][N/2], low nibble = even column
        "scale": (torch.rand((K // c["group"], N), device=dev, generator=gen) * 0.008 + 0.002).to(td),
        "bias": normal(1, N, 0.5)[0] if c["bias"] else None,
    }
    width = N // 2 if c["op"].startswith("glu") else N
    if c["op"] in ("ep", "glu"):
        s["x"] = normal(M, K, 1.0, c["pad"])
        s["residual"] = normal(M, N, 1.0) if c["residual"] else None
        s["y"] = torch.empty((M, width), device=dev, dtype=td)
        s["keep"] = torch.empty((M, N), device=dev, dtype=td) if c["save"] else None
    else:
        s["dy"] = normal(M, width, 0.02, c["pad"])
        if c["act"] != NONE or c["op"] == "glu_bwd":       # the saved pre-activation (else dpre is dy itself)
            s["keep"] = normal(M, N, 1.5)
            s["dkeep"] = torch.empty((M, N), device=dev, dtype=td)
        s["residual"] = normal(M, K, 0.02) if c["residual"] else None
        s["dx"] = torch.empty((M, K), device=dev, dtype=td)
        s["dbias"] = torch.empty(N, device=dev, dtype=torch.float32) if c["bias"] else None
    return s


# ---- plain form -------------------------------------------------------------------

def _weights(s):
    c = s["case"]
    w, K, N = s["w"], c["K"], c["N"]
    q = torch.stack((w & 15, w >> 4), -1).view(K, N)
    if s["zero"] is None:
        q = (q ^ 8).float() - 8.0
    else:
        z = torch.stack((s["zero"] & 15, s["zero"] >> 4), -1).view(-1, N).float()
        q = q.float() - z.repeat_interleave(c["group"], 0)
    return q * s["scale"].float().repeat_interleave(c["group"], 0)


def _act(v, act):
    if act == RELU:
        return torch.where(v > 0, v, torch.zeros_like(v))
    if act == SILU:
        return v / (1 + torch.exp(-v))
    if act == GELU:
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == GELU_TANH:
        return 0.5 * v * (1 + torch.tanh(math.sqrt(2 / math.pi) * (v + 0.044715 * v * v * v)))
    return v


def _dact(v, act):
    if act == RELU:
        return (v > 0).to(v.dtype)
    if act == SILU:
        e = 1 / (1 + torch.exp(-v))
        return e * (1 + v * (1 - e))
    if act == GELU:
        return 0.5 * (1 + torch.erf(v * math.sqrt(0.5))) + v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if act == GELU_TANH:
        k = math.sqrt(2 / math.pi)
        t = torch.tanh(k * (v + 0.044715 * v * v * v))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * k * (1 + 3 * 0.044715 * v * v)
    return torch.ones_like(v)


def _plain(s):
    c, td = s["case"], _TORCH[s["case"]["dt"]]
    act, W = c["act"], _weights(s)
    if c["op"] in ("ep", "glu"):
        h = s["x"].float() @ W
        if s["bias"] is not None:
            h = h + s["bias"].float()
        if c["op"] == "ep":
            y = _act(h, act)
            if s["residual"] is not None:
                y = y + s["residual"].float()
        else:
            g, u = h.chunk(2, 1)
            y = _act(g, act) * u
        return [y.to(td)] + ([h.to(td)] if c["save"] else [])
    dy = s["dy"].float()
    if c["op"] == "ep_bwd":
        d = dy if act == NONE else dy * _dact(s["keep"].float(), act)
    else:
        g, u = s["keep"].float().chunk(2, 1)
        d = torch.cat((dy * u * _dact(g, act), dy * _act(g, act)), 1)
    dx = d @ W.t()
    if s["residual"] is not None:
        dx = dx + s["residual"].float()
    return [dx.to(td)] + ([d.to(td)] if "keep" in s else []) + ([d.sum(0)] if c["bias"] else [])


# ---- the library's calls ------------------------------------------------------------

def _handle(s):
    """The weight description and workspace that a program keeps with its weights."""
    import weight_only_quantized_amd as w4
    c = s["case"]
    lin = w4.linear(c["K"], c["N"], s["packed"], s["scale"], s["zero"], s["bias"], c["group"])
    query = {"ep": w4.w4a16_gemm_ep_workspace_bytes, "ep_bwd": w4.w4a16_gemm_ep_backward_workspace_bytes,
             "glu": w4.w4a16_glu_gemm_workspace_bytes, "glu_bwd": w4.w4a16_glu_gemm_backward_workspace_bytes}[c["op"]]
    nbytes = query(lin, c["M"])
    ws = torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None
    s["handle"] = (w4, lin, ws, nbytes)
    return s["handle"]


def _own(s):
    c = s["case"]
    w4, lin, ws, nbytes = s.get("handle") or _handle(s)
    if c["op"] == "ep":
        w4.w4a16_gemm_ep(s["x"], lin, s["y"], c["M"], c["act"], s["residual"], s["keep"], c["dt"],
                         ldx=c["K"] + c["pad"], workspace=ws, workspace_bytes=nbytes)
    elif c["op"] == "glu":
        w4.w4a16_glu_gemm(s["x"], lin, s["y"], c["M"], c["act"], s["keep"], c["dt"], ldx=c["K"] + c["pad"],
                          workspace=ws, workspace_bytes=nbytes)
    elif c["op"] == "ep_bwd":
        w4.w4a16_gemm_ep_backward(s["dy"], s.get("keep"), lin, s["dx"], c["M"], c["act"], s.get("dkeep"), s["dbias"],
                                  s["residual"], c["dt"], lddy=c["N"] + c["pad"], workspace=ws,
                                  workspace_bytes=nbytes)
    else:
        w4.w4a16_glu_gemm_backward(s["dy"], s["keep"], lin, s["dx"], c["M"], c["act"], s["dkeep"], s["dbias"],
                                   s["residual"], c["dt"], ldda=c["N"] // 2 + c["pad"], workspace=ws,
                                   workspace_bytes=nbytes)
    if c["op"] in ("ep", "glu"):
        return [s["y"]] + ([s["keep"]] if c["save"] else [])
    return [s["dx"]] + ([s["dkeep"]] if "dkeep" in s else []) + ([s["dbias"]] if c["bias"] else [])


def run(state):
    return _own(state) if own else _plain(state)


# ---- cost and reference ---------------------------------------------------------------

def work(case):
    c = case
    M, K, N = c["M"], c["K"], c["N"]
    width = N // 2 if c["op"].startswith("glu") else N
    G = K // c["group"]
    b = K * N // 2 + 2 * G * N + (G * N // 2 if c["zero"] else 0)
    if c["op"] in ("ep", "glu"):
        b += 2 * M * K + 2 * M * width + (2 * N if c["bias"] else 0)
        b += 2 * M * N * (c["residual"] + c["save"])
    else:
        b += 2 * M * width + 2 * M * K + 2 * M * K * c["residual"]
        b += 4 * M * N if c["act"] != NONE or c["op"] == "glu_bwd" else 0
        b += 4 * N if c["bias"] else 0
    return {"bytes": b, "flops": 2 * M * K * N}


def exact(case, seed):
    """The definitions in 64 bits, group by group of W's rows."""
    s, c = prepare(case, seed), case
    K, N, gs, act = c["K"], c["N"], c["group"], c["act"]
    d64 = torch.float64

    def rows(g):
        """dequant(W) rows of scale group g"""
        b = s["w"][g * gs:(g + 1) * gs].to(torch.int16)
        q = torch.empty((gs, N), dtype=d64, device=b.device)
        q[:, 0::2], q[:, 1::2] = (b % 16).to(d64), (b // 16).to(d64)
        if s["zero"] is None:
            q = torch.where(q >= 8, q - 16, q)
        else:
            zb = s["zero"][g].to(torch.int16)
            q[:, 0::2] -= (zb % 16).to(d64)
            q[:, 1::2] -= (zb // 16).to(d64)
        return q * s["scale"][g].to(d64)

    def phi(v):                                            # activation and derivative, from their definitions
        if act == NONE:
            return v, torch.ones_like(v)
        if act == RELU:
            return v.clamp(min=0), torch.heaviside(v, torch.zeros_like(v))
        if act == SILU:
            e = torch.sigmoid(v)
            return v * e, e + v * e * (1 - e)
        if act == GELU:
            cdf = torch.special.ndtr(v)
            return v * cdf, cdf + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)
        r = math.sqrt(8 / math.pi)                         # (1 + tanh(y)) / 2 = sigmoid(2 y)
        e = torch.sigmoid(r * (v + 0.044715 * v ** 3))
        return v * e, e + v * e * (1 - e) * r * (1 + 0.134145 * v ** 2)

    if c["op"] in ("ep", "glu"):
        x = s["x"].to(d64)
        h = torch.zeros((c["M"], N), dtype=d64, device=x.device)
        for g in range(K // gs):
            h += x[:, g * gs:(g + 1) * gs] @ rows(g)
        if c["bias"]:
            h += s["bias"].to(d64)
        if c["op"] == "ep":
            y = phi(h)[0]
            if c["residual"]:
                y = y + s["residual"].to(d64)
        else:
            y = phi(h[:, :N // 2])[0] * h[:, N // 2:]
        return [y] + ([h] if c["save"] else [])
    dy = s["dy"].to(d64)
    if c["op"] == "ep_bwd":
        d = dy * phi(s["keep"].to(d64))[1] if "keep" in s else dy
    else:
        h = s["keep"].to(d64)
        f, df = phi(h[:, :N // 2])
        d = torch.cat((dy * h[:, N // 2:] * df, dy * f), 1)
    dx = torch.cat([d @ rows(g).t() for g in range(K // gs)], 1)
    if c["residual"]:
        dx = dx + s["residual"].to(d64)
    return [dx] + ([d] if "keep" in s else []) + ([d.sum(0)] if c["bias"] else [])
