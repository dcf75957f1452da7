"""The block-scaled FP8 and mixture-of-experts operators in plain torch, and the cases that they are measured on.

Four operators, as a serving program calls them (``group_quantized_w4a4_b200`` where ``own`` is true):

* ``linear``: y = x . W^T with E4M3 operands.  x [M, K] is quantized online in groups of 1 x 128 (scale = fp32(absmax / 448),
  codes = E4M3 rounding, half to even, of the exact quotient); W [N, K] was quantized offline in blocks of 128 x 128 by the same
  rule.  Each 128-wide K-group's products are summed and scaled by both scales; y has x's type.
* ``route``: scores of E experts for every token, the top k of them, their weights, and the tokens grouped by expert.
* ``moe``: the experts' products for tokens grouped by expert: h = silu(x . Wg^T) * (x . Wu^T), quantized again in groups of 128,
  y = sum over a token's experts of weight * (h . Wd^T).
* ``norm``: the norm behind a block, its gate, the residual scale, the residual, the norm before the next block, and that block's
  quantized input.

Plain values are computed in 32 bits and rounded once; quotients next to a rounding border, and scores that are compared with a
bias or summed over a group, are computed in 64.
"""
import math

import numpy as np
import torch

own = False

F16, BF16 = torch.float16, torch.bfloat16
TYPES = {"fp16": F16, "bf16": BF16}
DEV = "cuda"


def listed():
    return [
        # one token through a dense 8192 x 8192 projection: a single user's decode step
        {"name": "linear_m1", "op": "linear", "M": 1, "N": 8192, "K": 8192, "dtype": "bf16"},
        # a decode batch of 16 on the same matrix, the benchmark's decode shape
        {"name": "linear_m16", "op": "linear", "M": 16, "N": 8192, "K": 8192, "dtype": "fp16"},
        # a short prompt through odd sizes: a ragged last K-group, weight block and token tile
        {"name": "linear_ragged", "op": "linear", "M": 333, "N": 5000, "K": 2064, "dtype": "bf16"},
        # prefill, the benchmark's prefill shape
        {"name": "linear_m4096", "op": "linear", "M": 4096, "N": 8192, "K": 8192, "dtype": "fp16"},
        # one token's experts: latency alone
        {"name": "route_t1", "op": "route", "T": 1, "E": 64, "k": 8, "G": 1, "TG": 1, "score": "softmax", "bias": False, "renorm": True, "scale": 1.0, "masked": 0.0, "dtype": "bf16"},
        # a padded batch over an expert count that is no power of two, group-limited
        {"name": "route_t777", "op": "route", "T": 777, "E": 160, "k": 6, "G": 8, "TG": 3, "score": "softmax", "bias": False, "renorm": False, "scale": 2.0, "masked": 0.2, "dtype": "fp32"},
        # prefill over many experts with a balance bias
        {"name": "route_t16384", "op": "route", "T": 16384, "E": 256, "k": 8, "G": 8, "TG": 4, "score": "sigmoid", "bias": True, "renorm": True, "scale": 2.5, "masked": 0.0, "dtype": "fp32"},
        # a decode batch of 16: about two tokens for each expert, the weights' stream bounds it
        {"name": "moe_t16", "op": "moe", "T": 16, "E": 64, "k": 8, "H": 2048, "I": 1024, "masked": 0.0, "dtype": "bf16"},
        # a padded batch, ragged widths, few experts
        {"name": "moe_t333", "op": "moe", "T": 333, "E": 20, "k": 3, "H": 1040, "I": 720, "masked": 0.1, "dtype": "fp16"},
        # prefill: about 512 tokens for each expert, the tensor cores bound it
        {"name": "moe_t4096", "op": "moe", "T": 4096, "E": 64, "k": 8, "H": 2048, "I": 1024, "masked": 0.0, "dtype": "bf16"},
        # the norms between two blocks for one token
        {"name": "norm_t1", "op": "norm", "T": 1, "H": 8192, "gates": 1, "post": True, "alpha": 0.5, "offset": 0.0, "dtype": "bf16"},
        # and for a prefill, with a gate for each of four sequences
        {"name": "norm_t4096", "op": "norm", "T": 4096, "H": 8192, "gates": 4, "post": True, "alpha": 0.25, "offset": 1.0, "dtype": "fp16"},
    ]


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["linear", "route", "moe", "norm"])
    dtype = rng.choice(["fp16", "bf16"])
    if op == "linear":
        return {"op": op, "M": _log(rng, 1, 4096), "N": _log(rng, 200, 8192), "K": 16 * _log(rng, 8, 512), "dtype": dtype}
    if op == "route":
        G = rng.choice([1, 1, 2, 4, 8])
        E = G * rng.randint(2 if G > 1 else 4, 256 // G)
        TG = rng.randint(1, G)
        return {"op": op, "T": _log(rng, 1, 16384), "E": E, "k": rng.randint(1, min(8, TG * (E // G))), "G": G, "TG": TG,
                "score": rng.choice(["softmax", "sigmoid"]), "bias": rng.random() < 0.5, "renorm": rng.random() < 0.5,
                "scale": rng.choice([1.0, 2.5]), "masked": rng.choice([0.0, 0.0, 0.3]), "dtype": rng.choice(["fp16", "bf16", "fp32"])}
    if op == "moe":
        E = _log(rng, 2, 64)
        return {"op": op, "T": _log(rng, 1, 4096), "E": E, "k": rng.randint(1, min(8, E)), "H": 16 * _log(rng, 8, 128), "I": 16 * _log(rng, 8, 64),
                "masked": rng.choice([0.0, 0.0, 0.2]), "dtype": dtype}
    T = _log(rng, 1, 4096)
    return {"op": op, "T": T, "H": 16 * _log(rng, 8, 512), "gates": rng.choice([0, 1, T]), "post": rng.random() < 0.7,
            "alpha": rng.choice([1.0, 0.5]), "offset": rng.choice([0.0, 1.0]), "dtype": dtype}


# ------------------------------------------------------------------ the plain forms


def _e4m3(q):
    """64-bit values rounded to E4M3, half to even, saturating at 448 (three mantissa bits, exponents from -6)."""
    q = q.clamp(-448.0, 448.0)
    step = torch.ldexp(torch.ones_like(q), (torch.frexp(q)[1] - 1).clamp(min=-6) - 3)
    return torch.round(q / step) * step


def _scale(amax):
    """fp32(absmax / 448); the 64-bit quotient of a 24-bit value by 448 = 7 * 64 never sits at an fp32 border."""
    return (amax.double() / 448.0).float()


def _div(x, s):
    """x / s in 64 bits, 0 where s is 0."""
    return torch.where(s == 0, 0.0, x.double() / torch.where(s == 0, 1.0, s.double()))


def _quantize_rows(x):
    """x [R, K] -> (E4M3 values [R, K] fp32, scales [R, ceil(K / 128)] fp32)."""
    R, K = x.shape
    g = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(R, -1, 128)
    s = _scale(g.abs().amax(-1))
    return _e4m3(_div(g, s[..., None])).float().view(R, -1)[:, :K], s


def _quantize_blocks(w):
    """w [..., N, K] -> (E4M3 codes [..., N, K] uint8, scales [..., ceil(N / 128), ceil(K / 128)] fp32)."""
    N, K = w.shape[-2:]
    p = torch.nn.functional.pad(w.float(), (0, -K % 128, 0, -N % 128))
    b = p.view(*w.shape[:-2], p.shape[-2] // 128, 128, p.shape[-1] // 128, 128)
    s = _scale(b.abs().amax((-3, -1)))
    q = _e4m3(_div(b, s[..., :, None, :, None])).to(torch.float8_e4m3fn)
    return q.view(torch.uint8).view(p.shape)[..., :N, :K].contiguous(), s


def _rows(q, s):
    return q.float() * s.repeat_interleave(128, -1)[..., : q.shape[-1]]


def _blocks(codes, s):
    N, K = codes.shape[-2:]
    full = s.repeat_interleave(128, -2).repeat_interleave(128, -1)[..., :N, :K]
    return codes.view(torch.float8_e4m3fn).float() * full


def _plain_linear(s):
    return (_rows(*_quantize_rows(s["x"])) @ _blocks(s["w"], s["ws"]).T).to(s["x"].dtype)


def _plain_route(s):
    c, z = s["case"], s["logits"].double()
    T, E, k, G = c["T"], c["E"], c["k"], c["G"]
    p = torch.exp(z - z.amax(-1, keepdim=True)) if c["score"] == "softmax" else 1.0 / (1.0 + torch.exp(-z))
    if c["score"] == "softmax":
        p = p / p.sum(-1, keepdim=True)
    v = p + s["bias"].double() if c["bias"] else p
    if G > 1:
        top = torch.sort(v.view(T, G, E // G), dim=-1, descending=True)[0][..., :2].sum(-1)
        kept = torch.sort(top, dim=-1, descending=True, stable=True)[1][:, : c["TG"]]
        open_ = torch.zeros(T, G, dtype=torch.bool, device=z.device).scatter_(1, kept, True)
        v = torch.where(open_.repeat_interleave(E // G, 1), v, -math.inf)
    ids = torch.sort(v, dim=-1, descending=True, stable=True)[1][:, :k]
    w = p.gather(1, ids)
    w = w / w.sum(-1, keepdim=True) if c["renorm"] else w
    w = (w * c["scale"]).float()
    if s["mask"] is not None:
        ids, w = torch.where(s["mask"][:, None], ids, -1), torch.where(s["mask"][:, None], w, 0.0)
    ids = ids.int()
    offsets, order = _plan(ids, E)
    return w, ids, offsets, order


def _plan(ids, E):
    flat = ids.reshape(-1).long()
    key = torch.where(flat < 0, E, flat)
    counts = torch.zeros(E + 1, dtype=torch.long, device=ids.device).scatter_add_(0, key, torch.ones_like(key))
    offsets = torch.nn.functional.pad(counts[:E].cumsum(0), (1, 0)).int()
    order = torch.sort(key, stable=True)[1]
    here = torch.arange(flat.numel(), device=ids.device) < offsets[E]
    return offsets, torch.where(here, order, -1).int()


def _plain_moe(s):
    c = s["case"]
    T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
    # every expert's rows side by side, padded to the longest: slot -> (expert, place), place -> token
    at = torch.arange(s["most"], device=DEV)
    slot = s["offsets"][:E, None].long() + at
    live = at < (s["offsets"][1:] - s["offsets"][:-1])[:, None]
    flat = torch.where(live, s["order"].long()[slot.clamp(max=T * k - 1)], 0)
    x = _rows(*_quantize_rows(s["x"]))[flat // k] * live[..., None]
    gu = torch.bmm(x, _blocks(s["w13"], s["w13s"]).view(E, 2 * I, H).transpose(1, 2))
    g, u = gu[..., :I], gu[..., I:]
    h = _rows(*_quantize_rows((g / (1.0 + torch.exp(-g)) * u).view(-1, I))).view(E, -1, I)
    y = torch.bmm(h, _blocks(s["w2"], s["w2s"]).transpose(1, 2))
    # back to (token, choice): where each flat index went
    back = torch.full((T * k + 1,), E * s["most"], dtype=torch.long, device=DEV)
    back[torch.where(live, flat, T * k).view(-1)] = torch.arange(E * s["most"], device=DEV)
    y = torch.nn.functional.pad(y.view(-1, H), (0, 0, 0, 1))[back[: T * k]].view(T, k, H)
    return (y * torch.where(s["ids"] < 0, 0.0, s["weights"])[..., None]).sum(1).to(s["x"].dtype)


def _plain_norm(s):
    c, z = s["case"], s["x"].float()
    if c["post"]:
        z = z * torch.rsqrt(z.square().mean(-1, keepdim=True) + 1e-6) * (c["offset"] + s["post"].float())
    if c["gates"]:
        z = z * s["gate"].float().repeat_interleave(c["T"] // c["gates"], 0)
    h = s["residual"].float() + c["alpha"] * z
    y = h * torch.rsqrt(h.square().mean(-1, keepdim=True) + 1e-6) * (c["offset"] + s["pre"].float())
    q, qs = _quantize_rows(y)
    return h.to(s["x"].dtype), y.to(s["x"].dtype), q.to(torch.float8_e4m3fn), qs


# ------------------------------------------------------------------ inputs


def _normal(gen, shape, dtype, std=1.0):
    return (torch.randn(shape, generator=gen, device=DEV) * std).to(dtype)


def _activations(gen, rows, width, dtype):
    """N(0, 1) with one channel in a hundred twenty times as large, the same channels for every token."""
    loud = torch.where(torch.rand(width, generator=gen, device=DEV) < 0.01, 20.0, 1.0)
    return (torch.randn((rows, width), generator=gen, device=DEV) * loud).to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device=DEV)
    gen.manual_seed(int(seed))
    c, op = dict(case), case["op"]
    if op == "linear":
        w, ws = _quantize_blocks(_normal(gen, (c["N"], c["K"]), torch.float32, 0.02))
        return {"case": c, "x": _activations(gen, c["M"], c["K"], TYPES[c["dtype"]]), "w": w, "ws": ws}
    if op == "norm":
        t = TYPES[c["dtype"]]
        centre = 1.0 - c["offset"]
        return {"case": c, "x": _activations(gen, c["T"], c["H"], t), "residual": _normal(gen, (c["T"], c["H"]), t, 2.0),
                "post": (centre + 0.1 * torch.randn(c["H"], generator=gen, device=DEV)).to(t) if c["post"] else None,
                "pre": (centre + 0.1 * torch.randn(c["H"], generator=gen, device=DEV)).to(t),
                "gate": _normal(gen, (c["gates"], c["H"]), t) if c["gates"] else None}
    # some experts are chosen more often than others, as in a trained router
    liked = torch.randn(c["E"], generator=gen, device=DEV) * 0.5
    logits = torch.randn((c["T"], c["E"]), generator=gen, device=DEV) + liked
    mask = torch.rand(c["T"], generator=gen, device=DEV) >= c["masked"] if c["masked"] else None
    if op == "route":
        t = {**TYPES, "fp32": torch.float32}[c["dtype"]]
        bias = torch.randn(c["E"], generator=gen, device=DEV) * 0.05 if c["bias"] else None
        return {"case": c, "logits": logits.to(t), "bias": bias, "mask": mask}
    k, E, H, I = c["k"], c["E"], c["H"], c["I"]
    top = torch.sort(logits, dim=-1, descending=True, stable=True)
    ids, weights = top[1][:, :k], torch.softmax(top[0][:, :k], -1)
    if mask is not None:
        ids, weights = torch.where(mask[:, None], ids, -1), torch.where(mask[:, None], weights, 0.0)
    ids, weights = ids.int().contiguous(), weights.contiguous()
    offsets, order = _plan(ids, E)
    w13, w13s = _quantize_blocks(_normal(gen, (E, 2, I, H), torch.float32, 0.02))
    w2, w2s = _quantize_blocks(_normal(gen, (E, H, I), torch.float32, 0.02))
    return {"case": c, "x": _activations(gen, c["T"], H, TYPES[c["dtype"]]), "ids": ids, "weights": weights, "offsets": offsets, "order": order,
            "most": max(1, int((offsets[1:] - offsets[:-1]).max())), "w13": w13, "w13s": w13s, "w2": w2, "w2s": w2s}


def run(state):
    if own:
        return _own(state)
    return {"linear": _plain_linear, "route": _plain_route, "moe": _plain_moe, "norm": _plain_norm}[state["case"]["op"]](state)


def _own(s):
    import group_quantized_w4a4_b200 as apex

    c = s["case"]
    if c["op"] == "linear":
        return apex.linear_fp8_block(s["x"], s["w"], s["ws"])
    if c["op"] == "route":
        return apex.route_experts(s["logits"], c["k"], bias=s["bias"], score=c["score"], groups=c["G"], topk_groups=c["TG"],
                                  renormalize=c["renorm"], scale=c["scale"], mask=s["mask"], plan=True)
    if c["op"] == "moe":
        return apex.moe_mlp_fp8_block(s["x"], s["weights"], s["ids"], s["offsets"], s["order"], s["w13"], s["w13s"], s["w2"], s["w2s"])
    h, y, codes, scales = apex.block_norm(s["x"], s["pre"], residual=s["residual"], post_weight=s["post"], gate=s["gate"], alpha=c["alpha"],
                                          eps=1e-6, weight_offset=c["offset"], out="both")
    return h, y, codes.view(torch.float8_e4m3fn), scales


# ------------------------------------------------------------------ what a pass cannot do without


def _codes_bytes(rows, width):
    return rows * width + 4 * rows * -(-width // 128)


def _weight_bytes(n, rows, width):
    return n * (rows * width + 4 * -(-rows // 128) * -(-width // 128))


def work(case):
    c, op = case, case["op"]
    if op == "linear":
        M, N, K = c["M"], c["N"], c["K"]
        return {"bytes": 2 * M * K + _weight_bytes(1, N, K) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "route":
        T, E, k = c["T"], c["E"], c["k"]
        size = 4 if c["dtype"] == "fp32" else 2
        return {"bytes": size * T * E + (4 * E if c["bias"] else 0) + (T if c["masked"] else 0) + 12 * T * k + 4 * (E + 1), "flops": 10 * T * E}
    if op == "moe":
        T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
        slots = T * k * (1 - c["masked"])
        active = E * (1 - (1 - 1 / E) ** slots)
        return {"bytes": int(4 * T * H + 16 * T * k + 4 * E + active * (_weight_bytes(2, I, H) + _weight_bytes(1, H, I))), "flops": int(6 * slots * H * I)}
    T, H = c["T"], c["H"]
    return {"bytes": 2 * T * H * 4 + _codes_bytes(T, H) + 2 * H * (c["gates"] + 2), "flops": 20 * T * H}


# ------------------------------------------------------------------ the definitions in 64 bits


def _table():
    """The 127 finite E4M3 magnitudes in the order of their codes."""
    v = [m * 2.0**-9 for m in range(8)] + [(8 + m) * 2.0 ** (e - 10) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:127], dtype=torch.float64, device=DEV)


def _to_e4m3(q):
    """Nearest table entry; half-way goes to the even code."""
    v = _table()
    mids, a = (v[1:] + v[:-1]) / 2, q.abs().contiguous()
    low = torch.bucketize(a, mids)
    return torch.copysign(v[torch.where(low % 2 == 0, low, torch.bucketize(a, mids, right=True))], q)


def _groups64(x):
    """Every row's groups of 128, quantized and multiplied out again."""
    parts, values, scales = torch.split(x, 128, dim=1), [], []
    for p in parts:
        s = (p.abs().amax(1, keepdim=True) / 448.0).float().double()
        q = _to_e4m3(p / torch.where(s > 0, s, 1.0))
        values.append(torch.where(s > 0, q, 0.0))
        scales.append(s)
    return torch.cat(values, 1), torch.cat(scales, 1)


def _multiplied(values, scales):
    return torch.cat([p * scales[:, i : i + 1] for i, p in enumerate(torch.split(values, 128, dim=1))], 1)


def _weights64(codes, s):
    v = torch.cat([_table(), torch.full((1,), math.nan, device=DEV, dtype=torch.float64)])
    w = torch.cat([v, -v])[codes.long()]
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            w[128 * i : 128 * i + 128, 128 * j : 128 * j + 128] *= s[i, j].double()
    return w


def exact(case, seed):
    st, c = prepare(case, seed), case
    if c["op"] == "linear":
        return _multiplied(*_groups64(st["x"].double())) @ _weights64(st["w"], st["ws"]).T
    if c["op"] == "route":
        return _exact_route(c, st)
    if c["op"] == "moe":
        T, E, k, H, I = (c[n] for n in ("T", "E", "k", "H", "I"))
        x, out = _multiplied(*_groups64(st["x"].double())), torch.zeros(T, H, dtype=torch.float64, device=DEV)
        for e in range(E):
            t, j = torch.nonzero(st["ids"] == e, as_tuple=True)
            if t.numel():
                g, u = (x[t] @ _weights64(st["w13"][e, n], st["w13s"][e, n]).T for n in (0, 1))
                h = _multiplied(*_groups64(g * torch.sigmoid(g) * u))
                out[t] += st["weights"][t, j].double()[:, None] * (h @ _weights64(st["w2"][e], st["w2s"][e]).T)
        return out
    z = st["x"].double()
    if c["post"]:
        z = z / (z.pow(2).sum(1, keepdim=True) / c["H"] + 1e-6).sqrt() * (st["post"].double() + c["offset"])
    if c["gates"]:
        z = (z.view(c["gates"], -1, c["H"]) * st["gate"].double()[:, None]).view(c["T"], c["H"])
    h = st["residual"].double() + z * c["alpha"]
    y = h / (h.pow(2).sum(1, keepdim=True) / c["H"] + 1e-6).sqrt() * (st["pre"].double() + c["offset"])
    q, qs = _groups64(y)
    return h, y, q, qs


def _exact_route(c, st):
    z = st["logits"].double().cpu().numpy()
    T, E, k, G, TG = (c[n] for n in ("T", "E", "k", "G", "TG"))
    if c["score"] == "softmax":
        p = np.exp(z - z.max(1, keepdims=True))
        p /= p.sum(1, keepdims=True)
    else:
        p = 1 / (1 + np.exp(-z))
    v = p + (st["bias"].double().cpu().numpy() if c["bias"] else 0.0)
    if G > 1:
        parts = np.sort(v.reshape(T, G, -1), axis=2)
        best = np.argsort(-parts[:, :, -2:].sum(2), axis=1, kind="stable")[:, TG:]
        for t, g in zip(np.repeat(np.arange(T), G - TG), best.ravel()):
            v[t, g * (E // G) : (g + 1) * (E // G)] = -np.inf
    ids = np.argsort(-v, axis=1, kind="stable")[:, :k]
    w = np.take_along_axis(p, ids, 1)
    if c["renorm"]:
        w = w / w.sum(1, keepdims=True)
    w = w * c["scale"]
    if st["mask"] is not None:
        off = ~st["mask"].cpu().numpy()
        ids[off], w[off] = -1, 0.0
    flat = ids.ravel()
    order = np.concatenate([np.flatnonzero(flat == e) for e in range(E)] + [np.full(int((flat < 0).sum()), -1)])
    offsets = np.concatenate([[0], np.cumsum([(flat == e).sum() for e in range(E)])])
    return w, ids.astype(np.int32), offsets.astype(np.int32), order.astype(np.int32)
