"""Cases, plain forms and exact values for timing the operators around a transformer block's
quantized linears: routing to experts, low-rank adapters and the fused residual and norm.

A case is one call as a serving or inference program makes it:

* ``route`` -- router logits to chosen experts and their weights: softmax or sigmoid scores, a
  bias that balances the experts, groups of experts, top-k, renormalised weights;
* ``lora``  -- the low-rank adapters of many requests added to a shared projection's output: every
  row has its own adapter, or none;
* ``norm``  -- a branch's output through its own norm and gate onto the residual stream, and the
  norm ahead of the next branch, modulated by sequence; its result as bf16, or quantized to
  MXFP4 and multiplied with the next projection.

``run`` computes a case in elementary torch operations, or with ``own`` set through this
repository's package.
"""
import math
import random

import torch

own = False

_E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0)


def listed():
    return [
        # one decoded token, fine-grained experts in groups, balanced by a bias: launch latency
        {"name": "route-1-token", "op": "route", "T": 1, "E": 256, "top_k": 8, "scores": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True, "scale": 2.5},
        # a short prompt, a number of experts that is no multiple of a wave, shares of the whole softmax
        {"name": "route-ragged", "op": "route", "T": 333, "E": 60, "top_k": 4, "scores": "softmax", "bias": False,
         "groups": 1, "top_groups": 1, "group_best": 1, "renormalize": False, "scale": 1.0},
        # a prompt, groups ranked by their best expert
        {"name": "route-prompt", "op": "route", "T": 4096, "E": 160, "top_k": 6, "scores": "softmax", "bias": False,
         "groups": 8, "top_groups": 3, "group_best": 1, "renormalize": False, "scale": 16.0},
        # many prompts together, groups ranked by their two best
        {"name": "route-prompts", "op": "route", "T": 32768, "E": 256, "top_k": 8, "scores": "sigmoid", "bias": True,
         "groups": 8, "top_groups": 4, "group_best": 2, "renormalize": True, "scale": 2.5},
        # one decoded token and its adapter
        {"name": "lora-1-token", "op": "lora", "T": 1, "requests": 1, "L": 8, "R": 16, "K": 4096, "N": 4096},
        # a decode batch whose sequences use many adapters, a width that is no multiple of any tile
        {"name": "lora-batch-48", "op": "lora", "T": 48, "requests": 48, "L": 32, "R": 32, "K": 2560, "N": 1001},
        # prompts of different lengths in one batch, into an MLP's up-projection
        {"name": "lora-mixed", "op": "lora", "T": 1999, "requests": 24, "L": 16, "R": 64, "K": 4096, "N": 14336},
        # many long prompts, small adapters: memory bandwidth
        {"name": "lora-prompts", "op": "lora", "T": 16384, "requests": 12, "L": 8, "R": 16, "K": 4096, "N": 4096},
        # one decoded token: the residual and the norm ahead of the next branch
        {"name": "norm-1-token", "op": "norm", "M": 1, "H": 4096, "kind": "rms", "post": False, "bias": False, "gate": False,
         "modulate": False, "groups": 1, "quantize": False, "N": 0},
        # three images of a diffusion batch: layer norm, gate, scale and shift of each, an odd width
        {"name": "norm-modulated", "op": "norm", "M": 999, "H": 1160, "kind": "layer", "post": False, "bias": False, "gate": True,
         "modulate": True, "groups": 3, "quantize": False, "N": 0},
        # a decode batch through norms on both sides, quantized for the next projection and multiplied
        {"name": "norm-quantized-64", "op": "norm", "M": 64, "H": 4096, "kind": "rms", "post": True, "bias": False, "gate": False,
         "modulate": False, "groups": 1, "quantize": True, "N": 4096},
        # many prompts through norms on both sides, with learned gates: memory bandwidth
        {"name": "norm-prompts", "op": "norm", "M": 16384, "H": 8192, "kind": "rms", "post": True, "bias": False, "gate": True,
         "modulate": False, "groups": 1, "quantize": False, "N": 0},
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A row length: most are whole multiples of 128, some only of 32."""
    step = rng.choice((128, 128, 32))
    return step * _log_int(rng, lo // step, hi // step)


def draw(rng):
    op = rng.choice(("route", "lora", "norm"))
    if op == "route":
        groups, size = rng.choice(((1, 8), (1, 16), (1, 60), (1, 64), (1, 128), (1, 200), (4, 16), (4, 32), (8, 8), (8, 20), (8, 32)))
        top_groups = rng.randint((groups + 1) // 2, groups)
        return {"op": op, "T": _log_int(rng, 1, 32768), "E": groups * size, "top_k": rng.randint(1, 8),
                "scores": rng.choice(("softmax", "sigmoid")), "bias": rng.random() < 0.5, "groups": groups,
                "top_groups": top_groups, "group_best": rng.choice((1, 2)), "renormalize": rng.random() < 0.5,
                "scale": rng.choice((1.0, 2.5))}
    if op == "lora":
        T = _log_int(rng, 1, 8192)
        return {"op": op, "T": T, "requests": _log_int(rng, 1, min(T, 64)), "L": rng.choice((1, 4, 8, 16, 32)),
                "R": rng.choice((8, 16, 16, 24, 32, 64)), "K": _width(rng, 512, 4096), "N": _log_int(rng, 256, 4096)}
    quantize = rng.random() < 0.3
    modulate = rng.random() < 0.4
    groups = _log_int(rng, 1, 8) if modulate else 1
    return {"op": op, "M": groups * _log_int(rng, 1, 2048 if quantize else 8192 // groups),
            "H": _width(rng, 512, 8192) if quantize else 8 * _log_int(rng, 64, 1024), "kind": rng.choice(("rms", "layer")),
            "post": rng.random() < 0.4, "bias": rng.random() < 0.3, "gate": modulate or rng.random() < 0.3,
            "modulate": modulate, "groups": groups, "quantize": quantize, "N": _log_int(rng, 256, 4096) if quantize else 0}


# ---- MXFP4, in plain torch ---------------------------------------------------------------


def _pow2(byte):
    """2^(byte - 127) as float32, for E8M0 bytes 0..254."""
    b = byte.to(torch.int32)
    return torch.where(b == 0, torch.full_like(b, 0x00400000), b << 23).view(torch.float32)


def _decode(packed, scales):
    """float32 values of packed codes [..., K/2] and scale bytes [..., K/32]."""
    table = torch.tensor(_E2M1, dtype=torch.float32, device=packed.device)
    codes = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2)
    v = table[codes.to(torch.int32)].unflatten(-1, (-1, 32))
    return (v * _pow2(scales)[..., None]).flatten(-2)


def _encode(x):
    """Packed codes and scale bytes of a tensor [..., K]: the block's exponent is that of its largest magnitude less 2."""
    f = x.float().unflatten(-1, (-1, 32))
    field = f.abs().amax(-1).view(torch.int32) >> 23
    byte = torch.where(field == 0, torch.zeros_like(field), (field - 2).clamp(min=0))
    y = f.abs() * _pow2(254 - byte)[..., None]
    code = ((y > 0.25).to(torch.uint8) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0)).to(torch.uint8)
    code = (code | (torch.signbit(f).to(torch.uint8) << 3)).flatten(-2).unflatten(-1, (-1, 2))
    return code[..., 0] | (code[..., 1] << 4), byte.to(torch.uint8)


# ---- inputs ------------------------------------------------------------------------------


def _normal(g, *shape):
    return torch.randn(shape, device="cuda", generator=g)


def _activations(g, rows, K):
    """Normal values with a magnitude of their own for each row and a few channels of large ones."""
    x = _normal(g, rows, K) * torch.exp(0.3 * _normal(g, rows, 1))
    large = torch.rand((1, K), device="cuda", generator=g) < 0.003
    return torch.where(large, 12.0 * x, x).to(torch.bfloat16)


def _route_inputs(g, case):
    T, E = case["T"], case["E"]
    # logits of a trained router: some experts liked by most tokens, some tokens far from all
    logits = 1.2 * _normal(g, T, E) + 0.6 * _normal(g, 1, E) - (1.0 if case["scores"] == "sigmoid" else 0.0)
    if T > 1:  # a batch is padded to its length: rows that route nowhere
        padding = torch.rand((T, 1), device="cuda", generator=g) < 0.02
        logits = logits.masked_fill(padding, -math.inf)
    bias = 0.1 * _normal(g, E) if case["bias"] else None
    return {"logits": logits, "bias": bias}


def _lora_inputs(g, case, seed):
    T, L, R, K, N, requests = (case[k] for k in ("T", "L", "R", "K", "N", "requests"))
    rng = random.Random(seed)
    ends = sorted(rng.sample(range(1, T), requests - 1)) + [T]  # sequences of different lengths
    rows = []
    for start, end in zip([0] + ends, ends):
        # one request in eight has no adapter, where there are several
        which = -1 if requests > 1 and rng.random() < 0.125 else rng.randrange(L)
        rows += [which] * (end - start)
    return {
        "x": _activations(g, T, K),
        "y": _normal(g, T, N).to(torch.bfloat16),
        "a": (_normal(g, L, R, K) / math.sqrt(K)).to(torch.bfloat16),
        "b": (_normal(g, L, N, R) / math.sqrt(R)).to(torch.bfloat16),
        "scales": 0.25 + torch.rand((L,), device="cuda", generator=g),
        "adapters": torch.tensor(rows, dtype=torch.int32, device="cuda"),
    }


def _norm_inputs(g, case):
    M, H, G = case["M"], case["H"], case["groups"]

    def weight(shift):
        return (shift + 0.2 * _normal(g, H)).to(torch.bfloat16)

    def per_group(sd):
        return (sd * _normal(g, G, H)).to(torch.bfloat16)

    s = {"x": _activations(g, M, H), "y": _activations(g, M, H)}
    # a modulated norm's own weight is in its scale
    s["weight"] = None if case["modulate"] else weight(1.0)
    s["bias"] = weight(0.0) if case["bias"] else None
    s["post_weight"] = weight(0.5) if case["post"] else None
    s["gate"] = per_group(0.5) if case["gate"] else None
    s["scale"] = per_group(0.2) if case["modulate"] else None
    s["shift"] = per_group(0.2) if case["modulate"] else None
    s["w"] = _encode((_normal(g, case["N"], H) / math.sqrt(H)).to(torch.bfloat16)) if case["quantize"] else None
    return s


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "route":
        inputs = _route_inputs(g, case)
    elif case["op"] == "lora":
        inputs = _lora_inputs(g, case, seed)
    else:
        inputs = _norm_inputs(g, case)
    return {**case, **inputs}  # tensors, or None, in the place of truth values


# ---- one pass ----------------------------------------------------------------------------


def _run_own(s):
    import nvfp4_block_scaled_02_amd as nv

    if s["op"] == "route":
        return nv.moe_route(s["logits"], s["top_k"], bias=s["bias"], scores=s["scores"], groups=s["groups"],
                            top_groups=s["top_groups"], group_best=s["group_best"], renormalize=s["renormalize"], scale=s["scale"])
    if s["op"] == "lora":
        return nv.lora(s["y"], s["x"], s["a"], s["b"], s["adapters"], scales=s["scales"])
    h, n = nv.add_norm(s["x"], s["y"], weight=s["weight"], bias=s["bias"], post_weight=s["post_weight"], gate=s["gate"],
                       scale=s["scale"], shift=s["shift"], kind=s["kind"], eps=1e-6, residual_scale=1.0,
                       quantize="mxfp4" if s["quantize"] else None)
    return (h, nv.mxfp4_gemm(*n, *s["w"])) if s["quantize"] else (h, n)


def _plain_route(s):
    # in 64 bits: two experts, or two groups, next to each other in rank
    logits, k, G = s["logits"].double(), s["top_k"], s["groups"]
    T, E = logits.shape
    top = logits.amax(1, keepdim=True)
    if s["scores"] == "softmax":
        score = torch.exp(logits - torch.where(top == -math.inf, torch.zeros_like(top), top))
        share = score / score.sum(1, keepdim=True)
    else:
        share = 1.0 / (1.0 + torch.exp(-logits))
    key = share if s["bias"] is None else share + s["bias"].double()
    key = torch.where(logits == -math.inf, torch.full_like(key, -math.inf), key)
    best = torch.sort(key.view(T, G, E // G), dim=2, descending=True).values[:, :, : s["group_best"]]
    group = torch.where(best == -math.inf, torch.zeros_like(best), best).sum(2)
    group = torch.where(best[:, :, 0] == -math.inf, best[:, :, 0], group)
    kept = torch.sort(group, dim=1, descending=True, stable=True).indices[:, : s["top_groups"]]
    open_ = torch.zeros((T, G), dtype=torch.bool, device=key.device).scatter(1, kept, True)
    # without a bias the order is that of the logits
    order = torch.where(key == -math.inf, key, logits if s["bias"] is None else key)
    order = torch.where(open_.repeat_interleave(E // G, dim=1), order, torch.full_like(order, -math.inf))
    ranked = torch.sort(order, dim=1, descending=True, stable=True)
    ids, found = ranked.indices[:, :k], ranked.values[:, :k] != -math.inf
    w = torch.where(found, share.gather(1, ids), torch.zeros((), dtype=torch.float64, device=key.device))
    if s["renormalize"]:
        total = w.sum(1, keepdim=True)
        w = w / torch.where(total == 0, torch.ones_like(total), total)
    return torch.where(found, ids, torch.full_like(ids, -1)).to(torch.int32), (w * s["scale"]).float()


def _plain_lora(s):
    x, a, b, adapters = s["x"].float(), s["a"].float(), s["b"].float(), s["adapters"]
    L, R, _ = a.shape
    # the products with all adapters, those of a row's own kept
    v = torch.matmul(x, a.flatten(0, 1).T)
    mine = adapters[:, None] == torch.arange(L, device=x.device, dtype=torch.int32).repeat_interleave(R)
    v = torch.where(mine, v * s["scales"].repeat_interleave(R), torch.zeros_like(v))
    return (s["y"].float() + torch.matmul(v, b.permute(0, 2, 1).flatten(0, 1))).to(torch.bfloat16)


def _plain_normed(v, kind):
    if kind == "layer":
        v = v - v.mean(1, keepdim=True)
    return v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-6)


def _plain_norm(s):
    x, z = s["x"].float(), s["y"].float()
    each = x.shape[0] // s["groups"]
    if s["post_weight"] is not None:
        z = _plain_normed(z, s["kind"]) * s["post_weight"].float()
    if s["gate"] is not None:
        z = z * s["gate"].float().repeat_interleave(x.shape[0] // s["gate"].shape[0], dim=0)
    h = (x + z).to(torch.bfloat16)
    n = _plain_normed(h.float(), s["kind"])
    if s["weight"] is not None:
        n = n * s["weight"].float()
    if s["bias"] is not None:
        n = n + s["bias"].float()
    if s["scale"] is not None:
        n = n * (1.0 + s["scale"].float().repeat_interleave(each, dim=0)) + s["shift"].float().repeat_interleave(each, dim=0)
    n = n.to(torch.bfloat16)
    if s["quantize"]:
        n = torch.matmul(_decode(*_encode(n)), _decode(*s["w"]).T).to(torch.bfloat16)
    return h, n


def run(state):
    if own:
        return _run_own(state)
    if state["op"] == "route":
        return _plain_route(state)
    return _plain_lora(state) if state["op"] == "lora" else _plain_norm(state)


def work(case):
    if case["op"] == "route":
        T, E, k = case["T"], case["E"], case["top_k"]
        # a score and a comparison for each expert, a comparison for each of the chosen
        return {"bytes": 4 * T * E + 8 * T * k + (4 * E if case["bias"] else 0), "flops": 2 * T * E}
    if case["op"] == "lora":
        T, L, R, K, N = (case[k] for k in ("T", "L", "R", "K", "N"))
        met = L * (1.0 - (1.0 - 1.0 / L) ** case["requests"])  # adapters that so many requests use, on average
        return {"bytes": 2 * T * K + 4 * T * N + 2 * met * R * (K + N) + 4 * T, "flops": 2 * T * R * (K + N)}
    M, H, N = case["M"], case["H"], case["N"]
    vectors = (not case["modulate"]) + case["bias"] + case["post"] + case["groups"] * (case["gate"] + 2 * case["modulate"])
    # x and y in, h out; the norm's result out, or its product with MXFP4 weights
    out = 2 * M * N + N * H * 17 / 32 if case["quantize"] else 2 * M * H
    return {"bytes": 6 * M * H + 2 * H * vectors + out, "flops": 8 * M * H + 2 * M * H * N}


# ---- exact values ------------------------------------------------------------------------


def _exact_route(s):
    """A chunk of rows at a time, ranks by counting what comes before."""
    logits, k, G = s["logits"].double(), s["top_k"], s["groups"]
    E = logits.shape[1]
    size = E // G
    place = torch.arange(E, device=logits.device)

    def ahead(v, index):
        """How many others come before each: larger ones, and equal ones of lower index."""
        a, b = v[:, :, None], v[:, None, :]
        return ((b > a) | ((b == a) & (index[None, None, :] < index[None, :, None]))).sum(2)

    all_ids, all_weights = [], []
    for l in logits.split(1024):
        there = torch.isfinite(l)
        if s["scores"] == "softmax":
            share = torch.softmax(torch.where(there, l, -1e300), dim=1)
        else:
            share = torch.sigmoid(l)
        key = (share + s["bias"].double()) if s["bias"] is not None else share
        key = key.masked_fill(~there, -math.inf)
        in_groups = key.unflatten(1, (G, size))
        best = in_groups.topk(min(s["group_best"], size), dim=2).values
        score = best.masked_fill(torch.isinf(best), 0.0).sum(2).masked_fill(torch.isinf(best).all(2), -math.inf)
        open_ = ahead(score, place[:G]) < s["top_groups"]
        order = (key if s["bias"] is not None else l).masked_fill(~(there & open_.repeat_interleave(size, dim=1)), -math.inf)
        rank = ahead(order, place)
        ids = torch.full((l.shape[0], k), -1, dtype=torch.int32, device=l.device)
        weights = torch.zeros((l.shape[0], k), dtype=torch.float64, device=l.device)
        t, e = ((rank < k) & torch.isfinite(order)).nonzero(as_tuple=True)
        ids[t, rank[t, e]] = e.to(torch.int32)
        weights[t, rank[t, e]] = share[t, e]
        if s["renormalize"]:
            weights = weights / weights.sum(1, keepdim=True).clamp(min=1e-300)
        all_ids.append(ids)
        all_weights.append(s["scale"] * weights)
    return torch.cat(all_ids), torch.cat(all_weights)


def _exact_lora(s):
    out = s["y"].double()
    for i in range(s["a"].shape[0]):
        rows = (s["adapters"] == i).nonzero().flatten()
        if rows.numel():
            down = s["x"][rows].double() @ s["a"][i].double().T
            out[rows] += s["scales"][i].double() * (down @ s["b"][i].double().T)
    return out


def _exact_values(packed, scales):
    """float64 values: sign, two exponent bits and one mantissa bit of each code, times 2^(byte - 127)."""
    codes = torch.stack((packed & 15, packed >> 4), dim=-1).flatten(-2).double()
    sign = 1.0 - 2.0 * (codes >= 8)
    m = codes % 8
    power = torch.floor(m / 2)
    v = torch.where(m < 2, 0.5 * m, (2.0 + m % 2) * torch.exp2(power - 2.0))
    return sign * v * torch.exp2(scales.double() - 127.0).repeat_interleave(32, dim=-1)


def _exact_rounded(x):
    """float64 values that the blocks of x take: steps of 0.5, 1 and 2 of the block's scale below 2, 4 and 6, ties to even."""
    b = x.double().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = torch.where(top > 0, torch.frexp(top).exponent - 3, torch.full_like(top, -127, dtype=torch.int32)).clamp(min=-127)
    scale = torch.exp2(e.double())
    y = b.abs() / scale
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    return (torch.sign(b) * (torch.round(y / step) * step).clamp(max=6.0) * scale).flatten(-2)


def _exact_norm(s):
    """The residual stream is held in bf16: what the second norm takes is its rounded value."""
    M, G = s["x"].shape[0], s["groups"]
    group = torch.arange(M, device=s["x"].device) // (M // G)

    def normed(v):
        if s["kind"] == "layer":
            v = v - v.sum(1, keepdim=True) / v.shape[1]
        return v * torch.rsqrt(v.square().sum(1, keepdim=True) / v.shape[1] + 1e-6)

    hs, ns = [], []
    for rows in torch.arange(M, device=s["x"].device).split(2048):
        z = s["y"][rows].double()
        if s["post_weight"] is not None:
            z = normed(z) * s["post_weight"].double()
        if s["gate"] is not None:
            z = z * s["gate"].double()[group[rows]]
        h = s["x"][rows].double() + z
        n = normed(h.to(torch.bfloat16).double())
        if s["weight"] is not None:
            n = n * s["weight"].double()
        if s["bias"] is not None:
            n = n + s["bias"].double()
        if s["scale"] is not None:
            n = n * (1.0 + s["scale"].double()[group[rows]]) + s["shift"].double()[group[rows]]
        if s["quantize"]:
            n = _exact_rounded(n.to(torch.bfloat16)) @ _exact_values(*s["w"]).T
        hs.append(h)
        ns.append(n)
    return torch.cat(hs), torch.cat(ns)


def exact(case, seed):
    s = prepare(case, seed)
    if s["op"] == "route":
        return _exact_route(s)
    return _exact_lora(s) if s["op"] == "lora" else _exact_norm(s)
