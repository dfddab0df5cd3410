"""The router, the 8-bit expert products and the layer for a few tokens, as cases to measure.

Three families of cases, told apart by ``op``:

router    logits -> the K experts of each token and their weights; with
          ``grad`` also the gradient of the logits (a training step).
int8      rows of bf16 -> 8-bit rows with a scale each -> the product with
          8-bit weights that have a scale for each channel.  ``gate_up``: the
          experts' gate and up products with SwiGLU, on the tokens of each
          expert (their copy into expert-major order included).  ``down``: the experts'
          down product on expert-major rows.  ``dense``: one matrix.
few       the whole expert layer for T <= 64 tokens, weights in bf16 or in 8
          bits.
"""

import torch

own = False

DEV = "cuda"


def listed():
    return [
        # the next token of one conversation: nothing but latency
        dict(name="router_one_token", op="router", T=1, E=128, K=8, dtype="f32", scoring="softmax",
             renormalize=True, scale=1.0, grad=False),
        # a ragged batch in bf16 (many equal logits), sigmoid weights, forward and backward
        dict(name="router_ragged_bf16", op="router", T=1237, E=200, K=6, dtype="bf16", scoring="sigmoid",
             renormalize=True, scale=2.5, grad=True),
        # a training step's tokens through a router of 256 experts
        dict(name="router_train", op="router", T=16384, E=256, K=8, dtype="f32", scoring="softmax",
             renormalize=False, scale=1.0, grad=True),
        # a short prompt: few rows for each expert, odd counts
        dict(name="int8_gate_up_short", op="int8", form="gate_up", T=203, H=2048, E=64, K=8, I=512),
        # a full prompt batch of the layer at H=2048 E=128 I=768, up and down
        dict(name="int8_gate_up_prompt", op="int8", form="gate_up", T=4096, H=2048, E=128, K=8, I=768),
        dict(name="int8_down_prompt", op="int8", form="down", T=4096, H=2048, E=128, K=8, I=768),
        # one dense matrix (a shared expert's or a projection's) over many tokens: compute bound
        dict(name="int8_dense", op="int8", form="dense", T=8192, H=4096, E=1, K=1, I=4096),
        # decoding: one token, a small batch, the largest batch that counts as few
        dict(name="few_one_token", op="few", T=1, H=2048, E=128, K=8, I=768, weights="bf16", shared=False),
        dict(name="few_wide_bf16", op="few", T=16, H=7168, E=256, K=8, I=512, weights="bf16", shared=True),
        dict(name="few_largest_bf16", op="few", T=64, H=2048, E=128, K=8, I=768, weights="bf16", shared=False),
        dict(name="few_int8_small", op="few", T=5, H=4096, E=64, K=8, I=1536, weights="int8", shared=False),
        dict(name="few_int8_batch", op="few", T=48, H=2048, E=256, K=8, I=512, weights="int8", shared=True),
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["router", "int8", "few"])
    if op == "router":
        E = rng.choice([8, 60, 64, 100, 128, 160, 256])
        return dict(op=op, T=_log(rng, 1, 16384), E=E, K=rng.randint(1, 8), dtype=rng.choice(["f32", "bf16"]),
                    scoring=rng.choice(["softmax", "sigmoid"]), renormalize=rng.random() < 0.5,
                    scale=rng.choice([1.0, 2.5]), grad=rng.random() < 0.7)
    if op == "int8":
        form = rng.choice(["gate_up", "down", "dense"])
        H = 16 * _log(rng, 32, 128)
        if form == "dense":
            return dict(op=op, form=form, T=_log(rng, 1, 8192), H=H, E=1, K=1, I=16 * _log(rng, 16, 256))
        return dict(op=op, form=form, T=_log(rng, 8, 4096), H=H, E=rng.choice([8, 24, 64, 100, 128]),
                    K=rng.randint(1, 8), I=16 * _log(rng, 16, 48))
    T, H, E, K = _log(rng, 1, 64), 64 * _log(rng, 8, 112), rng.choice([8, 24, 64, 100, 128, 256]), rng.randint(1, 8)
    # as many columns as keep the weights that are read under those of the largest listed case
    hit = E * (1.0 - (1.0 - K / E) ** T)
    top = max(1, min(24, int(2.2e9 / (hit * 6 * H * 64)), int(5.6e9 / (E * 6 * H * 64))))
    return dict(op=op, T=T, H=H, E=E, K=K, I=64 * rng.randint(max(1, top // 6), top),
                weights=rng.choice(["bf16", "int8"]), shared=rng.random() < 0.5)


def _generator(seed):
    return torch.Generator(device=DEV).manual_seed(seed)


def _normal(g, shape, std=1.0, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float32) * std).to(dtype)


def _eight_bit(g, shape):
    """Weights N(0, 0.02) held in 8 bits with a scale for each channel (row)."""
    w = _normal(g, shape, 0.02, torch.float32)
    top = w.abs().amax(dim=-1, keepdim=True)
    q = torch.round(w / top * 127.0).to(torch.int8)
    return q, (top / 127.0).squeeze(-1).contiguous()


def _ids(g, T, K, E):
    """K distinct experts for each token."""
    return torch.rand((T, E), generator=g, device=DEV).topk(K, dim=1).indices.to(torch.int32)


def _routing(ids, E):
    """The slots in expert-major order, each slot's row there, and the experts' row offsets."""
    flat = ids.reshape(-1).long()
    order = torch.sort(flat, stable=True).indices
    row_map = torch.empty_like(order)
    row_map[order] = torch.arange(order.numel(), device=DEV)
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0).to(torch.int32)
    return order.to(torch.int32), row_map.to(torch.int32), offsets, int(counts.max())


def prepare(case, seed):
    g = _generator(seed)
    s = dict(case=case)
    if case["op"] == "router":
        T, E, K = case["T"], case["E"], case["K"]
        dt = torch.float32 if case["dtype"] == "f32" else torch.bfloat16
        s["logits"] = _normal(g, (T, E), 1.5, dt)
        s["grad_probs"] = _normal(g, (T, K), 1.0, torch.float32)
        return s
    T, H, E, K, I = (case[n] for n in "THEKI")
    if case["op"] == "int8":
        form = case["form"]
        if form == "dense":
            s["x"] = _normal(g, (T, H))
            s["offsets"], s["rows"] = None, T
            s["w"], s["cs"] = _eight_bit(g, (1, I, H))
            return s
        s["order"], s["row_map"], s["offsets"], s["rows"] = _routing(_ids(g, T, K, E), E)
        if form == "gate_up":
            s["x"] = _normal(g, (T, H))
            s["wg"], s["gs"] = _eight_bit(g, (E, I, H))
            s["wu"], s["us"] = _eight_bit(g, (E, I, H))
        else:
            # what SwiGLU leaves: silu of one normal value times another
            a, b = _normal(g, (T * K, I), 1.0, torch.float32), _normal(g, (T * K, I), 1.0, torch.float32)
            s["x"] = (a * torch.sigmoid(a) * b).to(torch.bfloat16)
            s["w"], s["cs"] = _eight_bit(g, (E, H, I))
        return s
    s["x"] = _normal(g, (T, H))
    s["ids"] = _ids(g, T, K, E)
    s["probs"] = torch.softmax(_normal(g, (T, K), 1.0, torch.float32), dim=1)
    s["shared"] = _normal(g, (T, H)) if case["shared"] else None
    if case["weights"] == "bf16":
        s["wg"], s["wu"] = _normal(g, (E, I, H), 0.02), _normal(g, (E, I, H), 0.02)
        s["wd"] = _normal(g, (E, H, I), 0.02)
        s["scales"] = None
    else:
        s["wg"], gs = _eight_bit(g, (E, I, H))
        s["wu"], us = _eight_bit(g, (E, I, H))
        s["wd"], ds = _eight_bit(g, (E, H, I))
        s["scales"] = (gs, us, ds)
    return s


# ---- the framework's calls -----------------------------------------------------

def _run_own(s):
    from unpermute_moe_permute_gb300 import binding as lib
    c = s["case"]
    if c["op"] == "router":
        how = dict(scoring=c["scoring"], renormalize=c["renormalize"], scale=c["scale"])
        ids, probs = lib.moe_router_topk(s["logits"], c["K"], **how)
        if not c["grad"]:
            return [ids, probs]
        return [ids, probs, lib.moe_router_topk_grad(s["grad_probs"], s["logits"], ids, **how)]
    if c["op"] == "few":
        return [lib.moe_layer_few_tokens(s["x"], s["ids"], s["probs"], s["wg"], s["wu"], s["wd"],
                                         scales=s["scales"], shared_x=s["shared"])]
    if c["form"] == "gate_up":
        q, rs = lib.moe_quantize_rows(s["x"], row_map=s["row_map"], K=c["K"])
        return [lib.moe_gate_up_swiglu_int8(q, rs, s["offsets"], s["wg"], s["gs"], s["wu"], s["us"])]
    q, rs = lib.moe_quantize_rows(s["x"])
    return [lib.moe_down_proj_int8(q, rs, s["offsets"], s["w"], s["cs"])]


# ---- the plain forms -----------------------------------------------------------

def _plain_router(s):
    c = s["case"]
    l = s["logits"].float()
    K, scale = c["K"], c["scale"]
    ids = torch.sort(l, dim=1, descending=True, stable=True).indices[:, :K]
    top = l.gather(1, ids)
    if c["scoring"] == "softmax":
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
    else:
        p = 1.0 / (1.0 + torch.exp(-l))
    sel = p.gather(1, ids)
    total = sel.sum(dim=1, keepdim=True)
    q = sel / total if c["renormalize"] else sel
    out = [ids.to(torch.int32), q * scale]
    if not c["grad"]:
        return out
    g = s["grad_probs"] * scale
    if c["scoring"] == "softmax":
        if c["renormalize"]:
            d = torch.zeros_like(l).scatter(1, ids, q * (g - (g * q).sum(dim=1, keepdim=True)))
        else:
            d = p * (torch.zeros_like(l).scatter(1, ids, g) - (g * q).sum(dim=1, keepdim=True))
    else:
        dsel = (g - (g * q).sum(dim=1, keepdim=True)) / total if c["renormalize"] else g
        d = torch.zeros_like(l).scatter(1, ids, dsel / (1.0 + torch.exp(-top)) / (1.0 + torch.exp(top)))
    return out + [d.to(s["logits"].dtype)]


def _plain_quantize(x):
    """Whole numbers (as floats) and the rows' scales: x is about q * scale."""
    x = x.float()
    top = x.abs().amax(dim=1, keepdim=True)
    return torch.round(x * 127.0 / top), top / 127.0


def _by_expert(rows, offsets, cap):
    """[N, Kd] expert-major rows as [E, cap, Kd] (rows past an expert's end repeat row 0),
    and for each of the N rows its place there."""
    n = torch.arange(rows.shape[0], device=rows.device)
    e = torch.searchsorted(offsets[1:].long(), n, right=True)
    place = e * cap + n - offsets.long()[e]
    at = torch.zeros((offsets.numel() - 1) * cap, dtype=torch.long, device=rows.device)
    at[place] = n
    return rows[at].view(offsets.numel() - 1, cap, -1), place


def _plain_int8(s):
    c = s["case"]
    if c["form"] == "dense":
        q, rs = _plain_quantize(s["x"])
        y = q @ s["w"][0].float().t()
        return [(y * rs * s["cs"]).to(torch.bfloat16)]
    x = s["x"][(s["order"] // c["K"]).long()] if c["form"] == "gate_up" else s["x"]
    q, rs = _plain_quantize(x)
    q, place = _by_expert(q, s["offsets"], s["rows"])
    rs, _ = _by_expert(rs, s["offsets"], s["rows"])
    if c["form"] == "down":
        y = torch.bmm(q, s["w"].float().transpose(1, 2)) * rs * s["cs"][:, None]
    else:
        gate = torch.bmm(q, s["wg"].float().transpose(1, 2)) * rs * s["gs"][:, None]
        up = torch.bmm(q, s["wu"].float().transpose(1, 2)) * rs * s["us"][:, None]
        y = gate / (1.0 + torch.exp(-gate)) * up
    return [y.reshape(-1, y.shape[-1])[place].to(torch.bfloat16)]


def _plain_few(s):
    """Every token through every expert that any token chose; the weights of the sum are
    zero where a token did not choose it."""
    active, where = torch.unique(s["ids"].long(), return_inverse=True)
    T, A = s["x"].shape[0], active.numel()
    p = torch.zeros((A, T), device=s["x"].device)
    p[where, torch.arange(T, device=p.device)[:, None]] = s["probs"]
    wg, wu, wd = s["wg"][active].float(), s["wu"][active].float(), s["wd"][active].float()
    if s["scales"] is not None:
        gs, us, ds = s["scales"]
        wg, wu, wd = wg * gs[active][..., None], wu * us[active][..., None], wd * ds[active][..., None]
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
    return {"router": _plain_router, "int8": _plain_int8, "few": _plain_few}[state["case"]["op"]](state)


# ---- what a pass cannot do without ------------------------------------------------

def work(case):
    if case["op"] == "router":
        T, E, K = case["T"], case["E"], case["K"]
        b = 4 if case["dtype"] == "f32" else 2
        # logits, ids and weights; backward: the weights' gradient and the logits' gradient
        bytes_ = T * E * b + 8 * T * K + (T * E * b + 4 * T * K if case["grad"] else 0)
        return dict(bytes=bytes_, flops=(8 if case["grad"] else 4) * T * E)
    T, H, E, K, I = (case[n] for n in "THEKI")
    if case["op"] == "int8":
        if case["form"] == "dense":
            return dict(bytes=2 * T * H + I * H + 4 * I + 2 * T * I, flops=2 * T * H * I)
        N = T * K
        hit = E * (1.0 - (1.0 - K / E) ** T)  # experts with rows, on average
        if case["form"] == "gate_up":
            return dict(bytes=2 * T * H + 4 * N + 4 * (E + 1) + hit * 2 * (I * H + 4 * I) + 2 * N * I,
                        flops=4 * N * H * I)
        return dict(bytes=2 * N * I + 4 * (E + 1) + hit * (I * H + 4 * H) + 2 * N * H, flops=2 * N * H * I)
    hit = E * (1.0 - (1.0 - K / E) ** T)
    each = 3 * I * H * 2 if case["weights"] == "bf16" else 3 * I * H + 4 * (2 * I + H)
    return dict(bytes=hit * each + (6 if case["shared"] else 4) * T * H + 8 * T * K, flops=6 * T * K * H * I)


# ---- the definitions in 64 bits -----------------------------------------------------

def _exact_router(s):
    c = s["case"]
    l = s["logits"].double()
    order = torch.argsort(-l, dim=1, stable=True)[:, :c["K"]]
    chosen = torch.zeros_like(l).scatter_(1, order, 1.0)
    if c["scoring"] == "softmax":
        p = torch.softmax(l, dim=1)
    else:
        p = torch.sigmoid(l)
    m = p * chosen
    S = m.sum(dim=1, keepdim=True) if c["renormalize"] else torch.ones_like(l[:, :1])
    w = c["scale"] * m / S
    out = [order.to(torch.int32), w.gather(1, order)]
    if c["grad"]:
        g = torch.zeros_like(l).scatter_(1, order, s["grad_probs"].double())
        # d(scale m / S), then through the scores
        dm = c["scale"] * (g / S - ((g * m).sum(dim=1, keepdim=True) / S ** 2 if c["renormalize"] else 0.0)) * chosen
        if c["scoring"] == "softmax":
            d = p * (dm - (dm * p).sum(dim=1, keepdim=True))
        else:
            d = dm * p * torch.sigmoid(-l)
        out.append(d)
    return out


def _exact_rows(x):
    x = x.double()
    top = x.abs().max(dim=1, keepdim=True).values
    return torch.round(127.0 * x / top), top / 127.0


def _exact_int8(s):
    c = s["case"]
    if c["form"] == "dense":
        q, rs = _exact_rows(s["x"])
        return [rs * (q @ s["w"][0].double().t()) * s["cs"].double()]
    x = s["x"][torch.div(s["order"].long(), c["K"], rounding_mode="floor")] if c["form"] == "gate_up" else s["x"]
    q, rs = _exact_rows(x)
    cut = s["offsets"].tolist()
    got = []
    for e in range(len(cut) - 1):
        a, r = q[cut[e]:cut[e + 1]], rs[cut[e]:cut[e + 1]]
        if c["form"] == "down":
            got.append(r * (a @ s["w"][e].double().t()) * s["cs"][e].double())
        else:
            gate = r * (a @ s["wg"][e].double().t()) * s["gs"][e].double()
            up = r * (a @ s["wu"][e].double().t()) * s["us"][e].double()
            got.append(gate * torch.sigmoid(gate) * up)
    return [torch.cat(got)]


def _exact_few(s):
    ids, probs = s["ids"].tolist(), s["probs"].double()
    out = s["shared"].double() if s["shared"] is not None else torch.zeros(s["x"].shape, device=DEV).double()
    tokens = {}
    for t, row in enumerate(ids):
        for k, e in enumerate(row):
            tokens.setdefault(e, []).append((t, k))
    for e, slots in tokens.items():
        t = torch.tensor([a for a, _ in slots], device=DEV)
        p = torch.stack([probs[a, b] for a, b in slots])[:, None]
        wg, wu, wd = s["wg"][e].double(), s["wu"][e].double(), s["wd"][e].double()
        if s["scales"] is not None:
            gs, us, ds = (v[e].double()[:, None] for v in s["scales"])
            wg, wu, wd = wg * gs, wu * us, wd * ds
        x = s["x"][t].double()
        gate, up = x @ wg.t(), x @ wu.t()
        out.index_add_(0, t, p * ((gate * torch.sigmoid(gate) * up) @ wd.t()))
    return [out]


def exact(case, seed):
    s = prepare(case, seed)
    return {"router": _exact_router, "int8": _exact_int8, "few": _exact_few}[case["op"]](s)
