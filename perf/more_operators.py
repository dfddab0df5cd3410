"""The router with a bias and groups, and the experts' products over 4-bit weights, as cases to measure.

Four families of cases, told apart by ``op``:

route     logits and a bias for each expert -> the best groups of experts, the
          K experts among them and their weights; with ``grad`` also the
          gradient of the logits (a training step).
weights   weights -> 4 bits with a scale for each group of inputs -> the bf16
          weights that those stand for.
product   expert-major rows in bf16 times 4-bit weights.  ``gate_up``: the gate
          and up products with SwiGLU.  ``down``: the down product.  ``dense``:
          one matrix.
few       the whole expert layer for T <= 64 tokens over 4-bit weights.

4-bit weights: w[n, k] = q[n, k] * scale[k // group, n], q in [-8, 7] as four
bits of two's complement.  Eight consecutive inputs make four bytes, the lower
four bits named first: (0, 2), (4, 6), (1, 3), (5, 7).  The scales are bf16
values of five significant bits (a group's largest magnitude / 7, rounded), so
that q * scale is a bf16 value too.
"""

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the next token of one conversation: nothing but latency
        dict(name="route_one_token", op="route", T=1, E=256, K=8, G=8, G_top=4, each=2, bias=True, dtype="f32",
             scoring="sigmoid", renormalize=True, scale=2.5, pad=0, grad=False),
        # a ragged batch, softmax weights, a group's best expert decides, bf16 logits with many
        # equal ones, two experts of 160 that only fill up the table
        dict(name="route_ragged_bf16", op="route", T=1237, E=160, K=6, G=8, G_top=3, each=1, bias=False,
             dtype="bf16", scoring="softmax", renormalize=False, scale=1.0, pad=2, grad=True),
        # a training step's tokens: bias for balance, the sum of a group's two best decides
        dict(name="route_train", op="route", T=16384, E=256, K=8, G=8, G_top=4, each=2, bias=True, dtype="f32",
             scoring="sigmoid", renormalize=True, scale=2.5, pad=0, grad=True),
        # one expert's weights in fp32, small groups
        dict(name="weights_one_expert", op="weights", E=1, rows=512, cols=2048, group=32, dtype="f32"),
        # all gate weights of the layer at H=2048 E=128 I=768
        dict(name="weights_layer", op="weights", E=128, rows=768, cols=2048, group=128, dtype="bf16"),
        # a short prompt: few rows for each expert, odd counts
        dict(name="gate_up_short", op="product", form="gate_up", T=203, H=2048, E=64, K=8, I=512, group=128,
             skew=0.0, out="bf16"),
        # a full prompt batch, up (some experts chosen much more often than others) and down
        dict(name="gate_up_prompt", op="product", form="gate_up", T=4096, H=2048, E=128, K=8, I=768, group=128,
             skew=0.5, out="bf16"),
        dict(name="down_prompt", op="product", form="down", T=4096, H=2048, E=128, K=8, I=768, group=64,
             skew=0.0, out="bf16"),
        # one dense layer for a handful of rows, fp32 out
        dict(name="dense_few_rows", op="product", form="dense", T=19, H=4096, E=1, K=1, I=4096, group=32, skew=0.0,
             out="f32"),
        # one token through 8 of 128 experts: latency
        dict(name="few_one_token", op="few", T=1, H=2048, E=128, K=8, I=768, group=128, shared=False),
        # a decoding batch of a large layer, with a shared expert
        dict(name="few_16_large", op="few", T=16, H=7168, E=256, K=8, I=512, group=128, shared=True),
        # an odd batch that reaches most experts, small groups
        dict(name="few_45", op="few", T=45, H=2048, E=128, K=8, I=768, group=32, shared=False),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["route", "weights", "product", "few"])
    if op == "route":
        while True:
            E, G = rng.choice([32, 64, 96, 128, 160, 256, 512]), rng.choice([1, 2, 4, 8, 16])
            c = dict(op=op, T=_log(rng, 1, 16384), E=E, K=rng.randint(1, 8), G=G, G_top=rng.randint(1, G),
                     each=rng.randint(1, 2), bias=rng.random() < 0.7, dtype=rng.choice(["f32", "bf16"]),
                     scoring=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.5,
                     scale=rng.choice([1.0, 2.5]), pad=rng.choice([0, 0, 1, 5]), grad=rng.random() < 0.7)
            if c["T"] * E <= 16384 * 256 and c["G_top"] * (E // G) >= c["K"] + c["pad"]:
                return c
    if op == "weights":
        dtype = rng.choice(["f32", "bf16"])
        rows, cols, group = 64 * _log(rng, 1, 48), 128 * _log(rng, 2, 32), rng.choice([32, 64, 128])
        top = max(1, (128 * 768 * 2048 // (2 if dtype == "f32" else 1)) // (rows * cols))
        return dict(op=op, E=min(128, _log(rng, 1, top)), rows=rows, cols=cols, group=group, dtype=dtype)
    if op == "product":
        form, group = rng.choice(["gate_up", "down", "dense"]), rng.choice([32, 64, 128])
        step = max(group, 64)
        H = step * _log(rng, 512 // step, 2048 // step)
        out = "bf16" if form == "gate_up" else rng.choice(["bf16", "f32"])
        if form == "dense":
            return dict(op=op, form=form, T=_log(rng, 1, 4096), H=H, E=1, K=1, I=64 * _log(rng, 4, 64), group=group,
                        skew=0.0, out=out)
        return dict(op=op, form=form, T=_log(rng, 8, 4096), H=H, E=rng.choice([8, 24, 64, 100, 128]),
                    K=rng.randint(1, 8), I=step * _log(rng, 256 // step, 768 // step), group=group,
                    skew=rng.choice([0.0, 0.5]), out=out)
    group = rng.choice([32, 64, 128])
    step = max(group, 64)
    T, H = _log(rng, 1, 64), step * _log(rng, 512 // step, 7168 // step)
    E, K = rng.choice([8, 24, 64, 100, 128, 256]), rng.randint(1, 8)
    # as many columns as keep the weights that are read under those of the largest listed case
    hit = E * (1.0 - (1.0 - K / E) ** T)
    top = max(1, min(1536 // step, int(5.4e8 / (hit * 1.5 * H * step)), int(1.4e9 / (E * 1.5 * H * step))))
    return dict(op=op, T=T, H=H, E=E, K=K, I=step * rng.randint(max(1, top // 6), top), group=group,
                shared=rng.random() < 0.5)


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _pack(q):
    """Whole numbers [..., k] in [-8, 7] as bytes [..., k / 2]."""
    v = (q.to(torch.int16) & 15).unflatten(-1, (-1, 2, 2, 2))  # element = 4 a + 2 b + c of eight
    low, high = v[..., 0, :], v[..., 1, :]                     # b = 0, 1: [..., a, c]
    return (low | high << 4).transpose(-1, -2).flatten(-3).to(torch.uint8)  # bytes in the order (c, a)


def _unpack(p):
    """The whole numbers, as floats."""
    v = p.to(torch.int16).unflatten(-1, (-1, 2, 2))            # [..., c, a]
    v = torch.stack((v & 15, v >> 4), dim=-1)                  # [..., c, a, b]
    v = torch.movedim(v, -3, -1).flatten(-4)
    return ((v ^ 8) - 8).float()


def _round4(w, group):
    """Weights [..., n, k] as whole numbers (floats) and scales [..., k / group, n]."""
    w = w.float().unflatten(-1, (-1, group))
    bits = (w.abs().amax(dim=-1) * (1.0 / 7.0)).view(torch.int32)
    bits = (bits + 0x3ffff + (bits >> 19 & 1)) & ~0x7ffff      # the 5 leading bits, ties to even
    scale = bits.view(torch.float32)
    s = scale.unsqueeze(-1)
    q = torch.where(s > 0, torch.round(w / s), 0.0).clamp(-8, 7)
    return q.flatten(-2), scale.to(torch.bfloat16).transpose(-1, -2).contiguous()


def _spread(scale, group):
    """Scales [..., k / group, n] for each weight [..., n, k]."""
    return scale.float().transpose(-1, -2).repeat_interleave(group, dim=-1)


def _four_bit(g, E, n, k, group):
    """Weights N(0, 0.02) in 4 bits; made for some experts at a time."""
    packed = torch.empty((E, n, k // 2), dtype=torch.uint8, device=DEV)
    scales = torch.empty((E, k // group, n), dtype=torch.bfloat16, device=DEV)
    some = max(1, 2 ** 27 // (n * k))
    for e in range(0, E, some):
        q, s = _round4(_normal(g, (min(some, E - e), n, k), 0.02, torch.float32), group)
        packed[e:e + some], scales[e:e + some] = _pack(q), s
    return packed, scales


def _ids(g, T, K, E, skew=0.0):
    """K distinct experts for each token, expert r drawn with a weight of (r + 1)^-skew."""
    weight = torch.arange(1, E + 1, device=DEV, dtype=torch.float32) ** -skew
    at = torch.rand((T, E), generator=g, device=DEV).clamp_min(1e-20).log() / weight
    return at.topk(K, dim=1).indices.to(torch.int32)


def _offsets(ids, E):
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return offsets, int(counts.max())


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "route":
        T, E, K, pad = case["T"], case["E"], case["K"], case["pad"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = _normal(g, (T, E), 1.5, dt)
        if pad:
            s["logits"][:, E - pad:] = float("-inf")
        s["bias"] = _normal(g, (E,), 0.1, torch.float32) if case["bias"] else None
        s["grad_probs"] = _normal(g, (T, K), 1.0, torch.float32)
        return s
    if case["op"] == "weights":
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["w"] = _normal(g, (case["E"], case["rows"], case["cols"]), 0.02, dt)
        return s
    T, H, E, K, I, group = (case[n] for n in ("T", "H", "E", "K", "I", "group"))
    if case["op"] == "product":
        if case["form"] == "dense":
            s["x"] = _normal(g, (T, H))
            s["offsets"], s["rows"] = None, T
            s["w"], s["ws"] = _four_bit(g, 1, I, H, group)
            return s
        s["offsets"], s["rows"] = _offsets(_ids(g, T, K, E, case["skew"]), E)
        if case["form"] == "gate_up":
            s["x"] = _normal(g, (T * K, H))
            s["wg"], s["gs"] = _four_bit(g, E, I, H, group)
            s["wu"], s["us"] = _four_bit(g, E, I, H, group)
        else:
            # what SwiGLU leaves: silu of one normal value times another
            a, b = _normal(g, (T * K, I), 1.0, torch.float32), _normal(g, (T * K, I), 1.0, torch.float32)
            s["x"] = (a * torch.sigmoid(a) * b).to(torch.bfloat16)
            s["w"], s["ws"] = _four_bit(g, E, H, I, group)
        return s
    s["x"] = _normal(g, (T, H))
    s["ids"] = _ids(g, T, K, E)
    s["probs"] = torch.softmax(_normal(g, (T, K), 1.0, torch.float32), dim=1)
    s["shared"] = _normal(g, (T, H)) if case["shared"] else None
    s["wg"], s["gs"] = _four_bit(g, E, I, H, group)
    s["wu"], s["us"] = _four_bit(g, E, I, H, group)
    s["wd"], s["ds"] = _four_bit(g, E, H, I, group)
    return s


# ---- the framework's calls -----------------------------------------------------

def _run_own(s):
    from unpermute_moe_permute_gb300 import binding as lib
    c = s["case"]
    if c["op"] == "route":
        how = dict(scoring=c["scoring"], renormalize=c["renormalize"], scale=c["scale"])
        ids, probs = lib.moe_router_topk_grouped(s["logits"], c["K"], bias=s["bias"], num_groups=c["G"],
                                                 top_groups=c["G_top"], group_top=c["each"], **how)
        if not c["grad"]:
            return [ids, probs]
        return [ids, probs, lib.moe_router_topk_grad(s["grad_probs"], s["logits"], ids, **how)]
    if c["op"] == "weights":
        q, scale = lib.moe_quantize_weights_int4(s["w"], c["group"])
        return [lib.moe_dequantize_weights_int4(q, scale), scale]
    if c["op"] == "few":
        return [lib.moe_layer_few_tokens_int4(s["x"], s["ids"], s["probs"], s["wg"], s["gs"], s["wu"], s["us"],
                                              s["wd"], s["ds"], shared_x=s["shared"])]
    if c["form"] == "gate_up":
        return [lib.moe_gate_up_swiglu_int4(s["x"], s["offsets"], s["wg"], s["gs"], s["wu"], s["us"])]
    return [lib.moe_down_proj_int4(s["x"], s["offsets"], s["w"], s["ws"],
                                   out_dtype=torch.bfloat16 if c["out"] == "bf16" else torch.float32)]


# ---- the plain forms -----------------------------------------------------------

def _plain_route(s):
    """Scores in 64 bits: in 32, two that lie next to each other may change places."""
    c = s["case"]
    l = s["logits"].double()
    T, E, K, G, scale = (c[n] for n in ("T", "E", "K", "G", "scale"))
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    by = p if s["bias"] is None else p + s["bias"].double()
    live = l > float("-inf")
    # a group's value; groups with fewer experts to choose from come last
    best = torch.where(live, by, -1e6).view(T, G, E // G).sort(dim=2, descending=True).values
    value = best[:, :, :c["each"]].sum(dim=2)
    keep = value.sort(dim=1, descending=True, stable=True).indices[:, :c["G_top"]]
    kept = torch.zeros_like(value).scatter(1, keep, 1.0).repeat_interleave(E // G, dim=1) > 0
    order = torch.where(kept, torch.where(live, by, -1e6), -1e9)
    ids = order.sort(dim=1, descending=True, stable=True).indices[:, :K]
    sel = p.gather(1, ids)
    total = sel.sum(dim=1, keepdim=True)
    q = sel / total if c["renormalize"] else sel
    out = [ids.to(torch.int32), (q * scale).float()]
    if not c["grad"]:
        return out
    g = s["grad_probs"].double() * scale
    if c["scoring"] == "softmax":
        if c["renormalize"]:
            d = torch.zeros_like(l).scatter(1, ids, q * (g - (g * q).sum(dim=1, keepdim=True)))
        else:
            d = p * (torch.zeros_like(l).scatter(1, ids, g) - (g * q).sum(dim=1, keepdim=True))
    else:
        d = (g - (g * q).sum(dim=1, keepdim=True)) / total if c["renormalize"] else g
        d = torch.zeros_like(l).scatter(1, ids, d * sel * (1.0 - sel))
    return out + [d.to(s["logits"].dtype)]


def _plain_weights(s):
    c = s["case"]
    q, scale = _round4(s["w"], c["group"])
    return [(q * _spread(scale, c["group"])).to(torch.bfloat16), scale]


def _by_expert(rows, offsets, cap):
    """[N, Kd] expert-major rows as [E, cap, Kd] (rows past an expert's end repeat row 0),
    and for each of the N rows its place there."""
    n = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(offsets[1:].long(), n, right=True)
    place = e * cap + n - offsets.long()[e]
    at = torch.zeros((offsets.numel() - 1) * cap, dtype=torch.long, device=rows.device)
    at[place] = n
    return rows[at].view(offsets.numel() - 1, cap, -1), place


def _weights32(q, scale, group):
    return _unpack(q) * _spread(scale, group)


def _plain_product(s):
    c = s["case"]
    x = s["x"].float()
    to = torch.bfloat16 if c["out"] == "bf16" else torch.float32
    if c["form"] == "dense":
        return [(x @ _weights32(s["w"][0], s["ws"][0], c["group"]).t()).to(to)]
    x, place = _by_expert(x, s["offsets"], s["rows"])
    if c["form"] == "down":
        y = torch.bmm(x, _weights32(s["w"], s["ws"], c["group"]).transpose(1, 2))
    else:
        gate = torch.bmm(x, _weights32(s["wg"], s["gs"], c["group"]).transpose(1, 2))
        up = torch.bmm(x, _weights32(s["wu"], s["us"], c["group"]).transpose(1, 2))
        y = gate / (1.0 + torch.exp(-gate)) * up
    return [y.reshape(-1, y.shape[-1])[place].to(to)]


def _plain_few(s):
    """Every token through every expert that any token chose; the weights of the sum are
    zero where a token did not choose it."""
    group = s["case"]["group"]
    active, where = torch.unique(s["ids"].long(), return_inverse=True)
    T, A = s["x"].shape[0], active.numel()
    p = torch.zeros((A, T), device=s["x"].device)
    p[where, torch.arange(T, device=p.device)[:, None]] = s["probs"]
    wg = _weights32(s["wg"][active], s["gs"][active], group)
    wu = _weights32(s["wu"][active], s["us"][active], group)
    wd = _weights32(s["wd"][active], s["ds"][active], group)
    x = s["x"].float().expand(A, -1, -1)
    gate, up = torch.bmm(x, wg.transpose(1, 2)), torch.bmm(x, wu.transpose(1, 2))
    act = gate / (1.0 + torch.exp(-gate)) * up * p[..., None]
    out = torch.bmm(act, wd.transpose(1, 2)).sum(dim=0)
    if s["shared"] is not None:
        out = out + s["shared"].float()
    return [out.to(torch.bfloat16)]


def run(state):
    if own:
        return _run_own(state)
    return {"route": _plain_route, "weights": _plain_weights, "product": _plain_product,
            "few": _plain_few}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "route":
        T, E, K = case["T"], case["E"], case["K"]
        b = 4 if case["dtype"] == "f32" else 2
        # logits, ids and weights; backward: the weights' gradient and the logits' gradient
        bytes_ = T * E * b + 8 * T * K + 4 * E * case["bias"] + (T * E * b + 4 * T * K if case["grad"] else 0)
        return dict(bytes=bytes_, flops=(12 if case["grad"] else 8) * T * E)
    if case["op"] == "weights":
        n = case["E"] * case["rows"] * case["cols"]
        # the weights, the bytes that are kept, the bf16 weights, the scales
        return dict(bytes=n * (4 if case["dtype"] == "f32" else 2) + n // 2 + 2 * n + 2 * n // case["group"], flops=4 * n)
    T, H, E, K, I = (case[n] for n in "THEKI")
    weight = 0.5 + 2.0 / case["group"]  # bytes of a weight with its share of a scale
    if case["op"] == "product":
        N = T * K
        to = 2 if case["out"] == "bf16" else 4
        if case["form"] == "dense":
            return dict(bytes=2 * T * H + weight * I * H + to * T * I, flops=2 * T * H * I)
        hit = E * (1.0 - (1.0 - K / E) ** T)  # experts with rows, on average
        if case["form"] == "gate_up":
            return dict(bytes=2 * N * H + 4 * (E + 1) + hit * 2 * weight * I * H + to * N * I, flops=4 * N * H * I)
        return dict(bytes=2 * N * I + 4 * (E + 1) + hit * weight * I * H + to * N * H, flops=2 * N * H * I)
    hit = E * (1.0 - (1.0 - K / E) ** T)
    return dict(bytes=hit * 3 * weight * I * H + (6 if case["shared"] else 4) * T * H + 8 * T * K,
                flops=6 * T * K * H * I)


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_route(s):
    c = s["case"]
    l = s["logits"].double()
    T, E, K, G = (c[n] for n in "TEKG")
    p = torch.softmax(l, dim=1) if c["scoring"] == "softmax" else torch.sigmoid(l)
    low = -1e9
    by = (p + s["bias"].double() if s["bias"] is not None else p).masked_fill(l == float("-inf"), low)
    groups = by.reshape(T, G, E // G).topk(c["each"], dim=2).values.sum(dim=2)
    # (of equal values the first: argsort of the negative, stable)
    chosen = torch.argsort(-groups, dim=1, stable=True)[:, :c["G_top"]]
    out_of = torch.ones_like(groups).scatter_(1, chosen, 0.0).bool()
    by = by.masked_fill(out_of.repeat_interleave(E // G, dim=1), 2 * low)
    order = torch.argsort(-by, dim=1, stable=True)[:, :K]
    picked = torch.zeros_like(l).scatter_(1, order, 1.0)
    m = p * picked
    S = m.sum(dim=1, keepdim=True) if c["renormalize"] else torch.ones_like(l[:, :1])
    out = [order.to(torch.int32), (c["scale"] * m / S).gather(1, order)]
    if c["grad"]:
        g = torch.zeros_like(l).scatter_(1, order, s["grad_probs"].double())
        # d(scale m / S), then through the scores
        dm = c["scale"] * (g / S - ((g * m).sum(dim=1, keepdim=True) / S ** 2 if c["renormalize"] else 0.0)) * picked
        if c["scoring"] == "softmax":
            d = p * (dm - (dm * p).sum(dim=1, keepdim=True))
        else:
            d = dm * p * torch.sigmoid(-l)
        out.append(d)
    return out


def _exact_weights(s):
    c = s["case"]
    w = s["w"].double().reshape(c["E"], c["rows"], -1, c["group"])
    # (the largest magnitude times 1 / 7 in 32 bits, then five significant bits of it)
    part, power = torch.frexp(w.abs().max(dim=3, keepdim=True).values.float() * (1.0 / 7.0))
    step = (power.long() + 1018 << 52).view(torch.float64)  # 2^(power - 5); torch.ldexp is off by a bit at times
    scale = torch.round(part.double() * 32.0) * step
    q = torch.clamp(torch.round(w / scale.clamp_min(1e-300)), min=-8, max=7)
    return [(q * scale).reshape(s["w"].shape), scale.squeeze(3).transpose(1, 2)]


def _exact_matrix(p, scale, group):
    """[n, k] in 64 bits from one expert's bytes and scales."""
    low, high = (p & 15).double(), (p >> 4).double()
    w = torch.empty((p.shape[0], 2 * p.shape[1]), dtype=torch.float64, device=p.device)
    for byte, (a, b) in enumerate(((0, 2), (4, 6), (1, 3), (5, 7))):
        w[:, a::8], w[:, b::8] = low[:, byte::4], high[:, byte::4]
    w = torch.where(w > 7.5, w - 16.0, w)
    return (w.view(p.shape[0], -1, group) * scale.double().t().unsqueeze(2)).view(p.shape[0], -1)


def _exact_product(s):
    c = s["case"]
    group = c["group"]
    if c["form"] == "dense":
        return [s["x"].double() @ _exact_matrix(s["w"][0], s["ws"][0], group).t()]
    cut = s["offsets"].tolist()
    got = []
    for e in range(len(cut) - 1):
        x = s["x"][cut[e]:cut[e + 1]].double()
        if c["form"] == "down":
            got.append(x @ _exact_matrix(s["w"][e], s["ws"][e], group).t())
        else:
            gate = x @ _exact_matrix(s["wg"][e], s["gs"][e], group).t()
            got.append(gate * torch.sigmoid(gate) * (x @ _exact_matrix(s["wu"][e], s["us"][e], group).t()))
    return [torch.cat(got)]


def _exact_few(s):
    ids, probs, group = s["ids"].tolist(), s["probs"].double(), s["case"]["group"]
    out = s["shared"].double() if s["shared"] is not None else torch.zeros(s["x"].shape, device=DEV).double()
    tokens = {}
    for t, row in enumerate(ids):
        for k, e in enumerate(row):
            tokens.setdefault(e, []).append((t, k))
    for e, slots in tokens.items():
        t = torch.tensor([a for a, _ in slots], device=DEV)
        p = torch.stack([probs[a, b] for a, b in slots])[:, None]
        x = s["x"][t].double()
        gate = x @ _exact_matrix(s["wg"][e], s["gs"][e], group).t()
        up = x @ _exact_matrix(s["wu"][e], s["us"][e], group).t()
        out.index_add_(0, t, p * ((gate * torch.sigmoid(gate) * up) @ _exact_matrix(s["wd"][e], s["ds"][e], group).t()))
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"route": _exact_route, "weights": _exact_weights, "product": _exact_product,
            "few": _exact_few}[case["op"]](s)
