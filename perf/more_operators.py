"""Workloads of the W8A8 products and the MoE router: what is timed and compared.

Four operators of a layer with int8 weights and experts:

  gemm       y = s_m sw_n sum_k q_mk W_kn + bias_n: x (16-bit) is quantized per
             token, s_m = fl32(max |x_m| / 127), q = x / s_m rounded to nearest
             even; W int8 with one fp32 scale sw per column
  grouped    the same for every expert's rows (expert_offsets), row r reading
             the token sorted_ids[r] / topk of x, or x row r itself
  route      top-k experts of every token's logits (ties to the lowest index),
             their softmax weights, per-expert counts and the balance loss
             E sum_e (c_e / C) mean_t p_te
  route_bwd  gradient of the weights and of the loss through the logits

With `own` False every operator runs in plain torch operations; with `own` True
it is one call of this library.
"""
import math

import torch

own = False

F16, BF16, F32 = 0, 1, 2
_TORCH = {F16: torch.float16, BF16: torch.bfloat16, F32: torch.float32}


def _gemm(name, M, K, N, dt=BF16, bias=False, pad=0):
    """pad: extra elements in every row of x (a slice of a wider buffer)."""
    return {"name": name, "op": "gemm", "M": M, "K": K, "N": N, "dt": dt, "bias": bias, "pad": pad}


def _grouped(name, T, topk, E, K, N, dt=BF16, gather=True, drop=0.0):
    """T tokens with topk experts each; gather: x holds the tokens, else the
    routed rows; drop: share of the routing entries that go to no expert."""
    return {"name": name, "op": "grouped", "T": T, "topk": topk, "E": E, "K": K, "N": N, "dt": dt, "gather": gather,
            "drop": drop}


def _route(name, op, T, E, topk, dt=F32, renorm=True, mask=0.0):
    """mask: share of the tokens that are padding."""
    return {"name": name, "op": op, "T": T, "E": E, "topk": topk, "dt": dt, "renorm": renorm, "mask": mask}


def listed():
    return [
        # a tiny projection: launch latency is all there is
        _gemm("gemm tiny", 4, 256, 256, F16),
        # gate/up projection of one decoded token and of a batch of 16
        _gemm("gemm decode 1", 1, 4096, 14336),
        _gemm("gemm decode 16", 16, 4096, 14336),
        # a short ragged prompt in fp16 with a bias, x a slice of a wider buffer
        _gemm("gemm prompt 77", 77, 8192, 8192, F16, bias=True, pad=64),
        # a long prompt
        _gemm("gemm prefill 4096", 4096, 4096, 14336),
        # experts' down projection while 4 tokens are decoded
        _grouped("grouped decode 4", 4, 8, 64, 1408, 2048, gather=False),
        # experts' gate/up projection of a prompt's tokens, read by token
        _grouped("grouped prompt 512", 512, 8, 64, 2048, 2816),
        # router of a few decoded tokens
        _route("route 16", "route", 16, 64, 8),
        # router of a training batch, the weights not renormalized
        _route("route 16384", "route", 16384, 256, 8, BF16, renorm=False),
        # its backward passes: an odd batch with padding, and the training batch
        _route("route_bwd 519", "route_bwd", 519, 64, 8, mask=0.1),
        _route("route_bwd 16384", "route_bwd", 16384, 256, 8, BF16),
    ]


def _log(rng, lo, hi):
    return math.exp(rng.uniform(math.log(lo), math.log(hi)))


def draw(rng):
    """Any operator, type and option; rows 1..4096, K 128..14336, N 64..14336,
    4..64 experts of the products, routers of 1..16384 tokens and 4..512
    experts, within the largest listed cost."""
    op = rng.choice(["gemm", "gemm", "grouped", "route", "route_bwd"])
    if op in ("route", "route_bwd"):
        T, E = max(1, min(16384, round(_log(rng, 1, 16385)))), max(4, min(512, round(_log(rng, 4, 513))))
        c = _route("", op, T, E, rng.randint(1, min(E, 10)), rng.choice([F16, BF16, F32, F32]), rng.random() < 0.5,
                   rng.choice([0.0, 0.0, 0.25]))
    else:
        while True:
            M = max(1, min(4096, round(_log(rng, 1, 4097))))
            K = 128 * max(1, round(_log(rng, 128, 14336) / 128))
            N = 64 * max(1, round(_log(rng, 64, 14336) / 64))
            E, topk = rng.randint(4, 64), rng.randint(1, 8)
            if op == "gemm" and K * N >= 1 << 16 and M * K * N <= 4096 * 4096 * 14336:
                break
            if op == "grouped" and M <= 1024 and 1 << 20 <= E * K * N <= 64 * 2048 * 2816:
                break
        dt = rng.choice([F16, BF16])
        if op == "gemm":
            c = _gemm("", M, K, N, dt, rng.random() < 0.5, rng.choice([0, 0, 8, 192]))
        else:
            c = _grouped("", M, min(topk, E), E, K, N, dt, rng.random() < 0.5, rng.choice([0.0, 0.0, 0.1]))
    del c["name"]
    return c


# ---- inputs ---------------------------------------------------------------------

def _pack(w):
    """The library's documented 8-bit layout from codes w [E][K][N] (int8):
    2048-byte tiles (expert, 16-column block, 128-row group), slot 16 c + j
    holds rows 32 c .. 32 c + 31 of column j, stored as q + 128."""
    E, K, N = w.shape
    t = w.view(torch.uint8).view(E, K // 128, 4, 32, N // 16, 16)      # e, g, c, r, nb, j
    return (t.permute(0, 4, 1, 2, 5, 3) ^ 128).contiguous()             # e, nb, g, c, j, r


def prepare(case, seed):
    c, dev = case, "cuda"
    gen = torch.Generator(device=dev).manual_seed(seed * 7919 + 17)

    def randn(*shape):
        return torch.randn(shape, device=dev, generator=gen)

    def rand(*shape):
        return torch.rand(shape, device=dev, generator=gen)

    s, td = {"case": dict(c)}, _TORCH[c["dt"]]
    if c["op"] in ("gemm", "grouped"):
        K, N, E = c["K"], c["N"], c.get("E", 1)
        s["w"] = (randn(E, K, N) * 36).round().clamp(-127, 127).to(torch.int8)
        s["packed"] = _pack(s["w"])
        s["sw"] = (rand(E, N) + 0.5) * 1e-3
        channels = 1 + 19 * (rand(K) < 0.01).float()                    # a few channels hold outliers
    if c["op"] == "gemm":
        M = c["M"]
        full = (randn(M, K + c["pad"]) * torch.cat((channels, torch.ones(c["pad"], device=dev)))).to(td)
        s["x"] = full[:, :K]
        s["bias"] = randn(N).to(td) if c["bias"] else None
        s["y"] = torch.empty((M, N), device=dev, dtype=td)
    elif c["op"] == "grouped":
        T, topk = c["T"], c["topk"]
        R = T * topk
        pop = torch.arange(1, E + 1, device=dev).float().pow(-1.1)      # a skewed popularity of the experts
        ids = (torch.log(pop) - torch.log(-torch.log(rand(T, E)))).topk(topk, 1)[1]
        ids = torch.where(rand(T, topk) < c["drop"], torch.full_like(ids, E), ids).reshape(-1)
        order = torch.sort(ids, stable=True)[1]
        cnt = torch.bincount(ids, minlength=E + 1)[:E]
        s["offsets"] = torch.cat((cnt.new_zeros(1), cnt.cumsum(0))).to(torch.int32)
        s["sorted"] = order.to(torch.int32) if c["gather"] else None
        s["most"] = int(cnt.max())                                       # rows of the largest expert (plain form)
        s["x"] = (randn(T if c["gather"] else R, K) * channels).to(td)
        s["y"] = torch.zeros((R, N), device=dev, dtype=td)
    else:
        T, E, topk = c["T"], c["E"], c["topk"]
        s["logits"] = (randn(T, E) * 1.5 + randn(E) * 0.5).to(td)
        s["mask"] = (rand(T) >= c["mask"]).to(torch.uint8) if c["mask"] else None
        if c["op"] == "route":
            s["ids"] = torch.empty((T, topk), device=dev, dtype=torch.int32)
            s["w"] = torch.empty((T, topk), device=dev)
            s["counts"] = torch.empty(E + 1, device=dev, dtype=torch.int32)
            s["loss"] = torch.empty((), device=dev)
        else:                                                            # what the forward pass left
            s["ids"], s["w"], s["counts"] = _route_plain(s)[:3]
            s["dw"] = randn(T, topk) * 0.02
            s["dloss"] = torch.full((), 0.01, device=dev)
            s["dlogits"] = torch.empty((T, E), device=dev, dtype=td)
    return s


# ---- plain form -------------------------------------------------------------------

def _quantize(x):
    """Codes and scales of the rows of x; the quotients in 64 bits, since values
    next to a rounding border decide whole codes."""
    scale = x.float().abs().amax(1) / 127
    q = torch.round(x.double() / torch.where(scale == 0, torch.ones_like(scale), scale).double()[:, None])
    return torch.clamp(q, -127, 127).float(), scale


def _gemm_plain(s):
    q, scale = _quantize(s["x"])
    y = (q @ s["w"][0].float()) * scale[:, None] * s["sw"]
    if s["bias"] is not None:
        y = y + s["bias"].float()
    return y.to(s["x"].dtype)


def _grouped_plain(s):
    """Every expert's rows padded to the largest expert's, then one product."""
    c = s["case"]
    q, scale = _quantize(s["x"])
    R = c["T"] * c["topk"]
    off = s["offsets"].long()
    row = off[:-1, None] + torch.arange(s["most"], device=off.device)
    held = row < off[1:, None]
    row = torch.where(held, row, torch.zeros_like(row))
    src = s["sorted"].long()[row] // c["topk"] if c["gather"] else row
    h = torch.bmm(q[src], s["w"].float()) * scale[src][..., None] * s["sw"][:, None, :]
    y = torch.zeros((R, c["N"]), device=q.device, dtype=s["x"].dtype)
    y[row[held]] = h[held].to(y.dtype)
    return y


def _softmax(z):
    e = torch.exp(z - z.amax(1, keepdim=True))
    return e / e.sum(1, keepdim=True)


def _route_plain(s):
    c, z = s["case"], s["logits"].float()
    E, topk = c["E"], c["topk"]
    p = _softmax(z)
    ids = torch.sort(z, dim=1, descending=True, stable=True)[1][:, :topk]
    w = p.gather(1, ids)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    if s["mask"] is not None:
        real = s["mask"].bool()[:, None]
        ids = torch.where(real, ids, torch.full_like(ids, -1))
        w, p = torch.where(real, w, torch.zeros_like(w)), torch.where(real, p, torch.zeros_like(p))
        tokens = real.sum()
    else:
        tokens = torch.full((), c["T"], device=z.device)
    cnt = torch.zeros(E + 1, device=z.device, dtype=torch.int64)
    cnt = cnt.scatter_add(0, torch.where(ids < 0, torch.full_like(ids, E), ids).reshape(-1), torch.ones_like(ids).reshape(-1))
    cnt = cnt[:E]
    loss = E * (cnt.float() / cnt.sum().clamp(min=1) * (p.sum(0) / tokens.clamp(min=1))).sum()
    return [ids.to(torch.int32), w, torch.cat((cnt, tokens[None])).to(torch.int32), loss]


def _route_bwd_plain(s):
    c, z = s["case"], s["logits"].float()
    E = c["E"]
    p = _softmax(z)
    ids, w, dw = s["ids"].long(), s["w"], s["dw"]
    held = ids >= 0
    at = torch.where(held, ids, torch.zeros_like(ids))
    cnt, tokens = s["counts"][:E].float(), s["counts"][E].float().clamp(min=1)
    h = (s["dloss"] * E / tokens) * (cnt / cnt.sum().clamp(min=1) - 1 / E).expand(z.shape)
    if c["renorm"]:
        own_part = torch.where(held, w * (dw - (w * dw).sum(1, keepdim=True)), torch.zeros_like(w))
    else:
        h = h.scatter_add(1, at, torch.where(held, dw, torch.zeros_like(dw)))
    dz = p * (h - (p * h).sum(1, keepdim=True))
    if c["renorm"]:
        dz = dz.scatter_add(1, at, own_part)
    if s["mask"] is not None:
        dz = torch.where(s["mask"].bool()[:, None], dz, torch.zeros_like(dz))
    return dz.to(s["logits"].dtype)


# ---- the library's calls ------------------------------------------------------------

def _handle(s):
    """The workspace that a program keeps."""
    import weight_only_quantized_amd as w4
    c = s["case"]
    if c["op"] == "gemm":
        nbytes = w4.w8a8_workspace_bytes(c["M"], c["K"])
    elif c["op"] == "grouped":
        nbytes = w4.w8a8_grouped_workspace_bytes(c["T"] * c["topk"], c["K"])
    elif c["op"] == "route":
        nbytes = w4.w4a16_moe_route_workspace_bytes(c["T"], c["E"])
    else:
        nbytes = 0
    s["handle"] = (w4, torch.empty(nbytes, dtype=torch.uint8, device="cuda") if nbytes else None, nbytes)
    return s["handle"]


def _own(s):
    c = s["case"]
    w4, ws, nbytes = s.get("handle") or _handle(s)
    if c["op"] == "gemm":
        w4.w8a8_gemm(s["x"], s["packed"], s["sw"], s["y"], c["M"], c["K"], c["N"], bias=s["bias"], dt=c["dt"],
                     ldx=c["K"] + c["pad"], workspace=ws, workspace_bytes=nbytes)
        return s["y"]
    if c["op"] == "grouped":
        w4.w8a8_grouped_gemm(s["x"], s["offsets"], s["packed"], s["sw"], s["y"], c["E"], c["T"] * c["topk"], c["K"],
                             c["N"], sorted_ids=s["sorted"], topk=c["topk"], dt=c["dt"], workspace=ws,
                             workspace_bytes=nbytes)
        return s["y"]
    if c["op"] == "route":
        w4.w4a16_moe_route(s["logits"], c["T"], c["E"], c["topk"], s["ids"], s["w"], counts=s["counts"],
                           loss=s["loss"], token_mask=s["mask"], renormalize=c["renorm"], dt=c["dt"], workspace=ws,
                           workspace_bytes=nbytes)
        return [s["ids"], s["w"], s["counts"], s["loss"]]
    w4.w4a16_moe_route_backward(s["logits"], s["ids"], s["w"], s["dlogits"], c["T"], c["E"], c["topk"],
                                counts=s["counts"], dtopk_w=s["dw"], dloss=s["dloss"], token_mask=s["mask"],
                                renormalize=c["renorm"], dt=c["dt"])
    return s["dlogits"]


_PLAIN = {"gemm": _gemm_plain, "grouped": _grouped_plain, "route": _route_plain, "route_bwd": _route_bwd_plain}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


# ---- cost and reference ---------------------------------------------------------------

def work(case):
    c = case
    if c["op"] == "gemm":
        M, K, N = c["M"], c["K"], c["N"]
        return {"bytes": 2 * M * K + K * N + 4 * N + (2 * N if c["bias"] else 0) + 2 * M * N, "flops": 2 * M * K * N}
    if c["op"] == "grouped":
        T, R, K, N = c["T"], c["T"] * c["topk"], c["K"], c["N"]
        used = min(c["E"], R)                                 # weights of at most so many experts are touched
        return {"bytes": 2 * (T if c["gather"] else R) * K + used * N * (K + 4) + 2 * R * N + 4 * (c["E"] + 1)
                + (4 * R if c["gather"] else 0), "flops": 2 * R * K * N}
    T, E, topk = c["T"], c["E"], c["topk"]
    size = 4 if c["dt"] == F32 else 2
    mask = T if c["mask"] else 0
    if c["op"] == "route":
        return {"bytes": size * T * E + 8 * T * topk + 4 * (E + 2) + mask, "flops": 4 * T * E}
    return {"bytes": 2 * size * T * E + 12 * T * topk + 4 * (E + 2) + mask, "flops": 8 * T * E}


def exact(case, seed):
    """The definitions in 64 bits; experts one by one, gradients by differentiating."""
    s, c = prepare(case, seed), case
    d64 = torch.float64
    if c["op"] in ("gemm", "grouped"):
        x = s["x"].to(d64)
        top = x.abs().max(1)[0]
        scale = (top.to(torch.float32) / torch.tensor(127.0, device=x.device)).to(d64)
        q = (x / scale.clamp(min=1e-300)[:, None]).round().clamp(-127, 127)
        if c["op"] == "gemm":
            y = (q @ s["w"][0].to(d64)) * s["sw"].to(d64) * scale[:, None]
            return y + s["bias"].to(d64) if c["bias"] else y
        y = torch.zeros((c["T"] * c["topk"], c["N"]), dtype=d64, device=x.device)
        off = s["offsets"].tolist()
        for e in range(c["E"]):
            rows = torch.arange(off[e], off[e + 1], device=x.device)
            if len(rows):
                src = s["sorted"][rows].long().div(c["topk"], rounding_mode="floor") if c["gather"] else rows
                y[rows] = (q[src] @ s["w"][e].to(d64)) * s["sw"][e].to(d64) * scale[src][:, None]
        return y
    T, E, topk = c["T"], c["E"], c["topk"]
    z = s["logits"].to(d64).requires_grad_(True)
    live = s["mask"].bool() if s["mask"] is not None else torch.ones(T, dtype=torch.bool, device=z.device)
    p = torch.softmax(z, 1)
    index = torch.arange(E, device=z.device)
    if c["op"] == "route":
        with torch.no_grad():
            left, picks = z.detach().clone(), []
            for _ in range(topk):                             # the largest that is left, the first of equals
                best = left.max(1, keepdim=True)[0]
                i = torch.where(left == best, index, E).min(1, keepdim=True)[0]
                picks.append(i)
                left.scatter_(1, i, -math.inf)
            ids = torch.cat(picks, 1)
            w = p.gather(1, ids)
            w = w / w.sum(1, keepdim=True) if c["renorm"] else w
            ids, w = ids.masked_fill(~live[:, None], -1), w.masked_fill(~live[:, None], 0)
            cnt = torch.stack([(ids == e).sum() for e in range(E)])
            loss = E * (cnt.to(d64) / cnt.sum().clamp(min=1) * p[live].sum(0) / live.sum().clamp(min=1)).sum()
            return [ids.to(torch.int32), w, torch.cat((cnt, live.sum()[None])).to(torch.int32), loss]
    ids = s["ids"].long()
    w = p.gather(1, ids.clamp(min=0))
    w = w / w.sum(1, keepdim=True) if c["renorm"] else w
    cnt = s["counts"][:E].to(d64)
    loss = E * (cnt / cnt.sum().clamp(min=1) * p[live].sum(0) / live.sum().clamp(min=1)).sum()
    total = (w * s["dw"].to(d64))[live].sum() + s["dloss"].to(d64) * loss
    return torch.autograd.grad(total, z)[0]
