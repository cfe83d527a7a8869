"""What is timed of the routing by scores, groups and a balancing bias, and of
the experts in microscaled 4-bit floating point: the cases, their inputs, the
plain forms and the library's calls.

Two operators:

* ``route``, ``route_backward``: a token's scores s are the softmax or the
  sigmoid of its logits.  Experts rank by c = s + bias.  With groups of
  consecutive experts a group's score is the sum of its ``group_top`` largest
  c, and only the ``top_groups`` best groups take part.  The k best experts
  are taken (ties go to the lower index); their weights are
  scale * s / (sum of the chosen s, or 1 without ``renorm``).  The backward
  pass takes the weights' gradients to the logits.
* ``mx_rows``, ``mx_weights``, ``mx_ffn``, ``mx_down``: numbers in 4 bits
  (sign, two exponent bits, one mantissa bit: 0, 0.5, 1, 1.5, 2, 3, 4, 6) that
  share an 8-bit scale in blocks of the reduction axis.  Blocks of 32 have a
  power of two, 2^(floor(log2 of the largest magnitude) - 2).  Blocks of 16
  have a number of 4 exponent and 3 mantissa bits, the largest magnitude over
  6, of values that are multiplied by the reciprocal of the tensor's float32
  scale beforehand.  ``mx_ffn`` is the SwiGLU FFN of the routed rows, rows and
  activations quantised on the way, over experts held in this form;
  ``mx_down`` one product of it.

``own`` chooses what ``run`` does: the plain form (elementary torch, 32 bits,
in 64 where experts are ranked, rounded once at each stored value) or the
library.
"""
import math

import torch

own = False

# the costliest cases that draw() may give: the listed ones
MAX_LOGITS = 65536 * 256
MAX_ELEMENTS = 8192 * 7168
MAX_WEIGHTS = 256 * 3 * 7168 * 2048
MAX_PRODUCTS = 32768 * 3 * 7168 * 2048


def _route(name, op, T, E, k, score, groups, top_groups, group_top, bias,
           renorm, scale):
    return {"name": name, "op": op, "T": T, "E": E, "k": k, "score": score,
            "groups": groups, "top_groups": top_groups,
            "group_top": group_top, "bias": bias, "renorm": renorm,
            "scale": scale}


def _mx(name, op, block, dtype, T, H, F=0, E=1, k=1, skew=0.0):
    return {"name": name, "op": op, "block": block, "dtype": dtype, "T": T,
            "H": H, "F": F, "E": E, "k": k, "skew": skew}


def listed():
    v3 = ("sigmoid", 8, 4, 2, True, True, 2.5)
    return [
        # one token of one sequence through the DeepSeek-V3-shaped router
        _route("route token", "route", 1, 256, 8, *v3),
        # a training step's tokens through the same router
        _route("route batch", "route", 65536, 256, 8, *v3),
        # an ungrouped softmax router without a bias, odd sizes
        _route("route softmax", "route", 8191, 60, 4, "softmax", 1, 1, 1,
               False, False, 1.0),
        # their gradients; the grouped one renormalises softmax scores
        _route("route backward", "route_backward", 65536, 256, 8, *v3),
        _route("route backward softmax", "route_backward", 8191, 128, 6,
               "softmax", 4, 2, 1, False, True, 1.0),
        # activations of a prompt, as the products take them
        _mx("mx rows", "mx_rows", 32, "bf16", 8192, 7168),
        # expert matrices quantised and laid out when a model is loaded
        _mx("mx weights", "mx_weights", 16, "bf16", 0, 7168, 2048, 8),
        # one token, DeepSeek-V3-shaped experts: 8 of 256 are read
        _mx("mx token", "mx_ffn", 16, "bf16", 1, 7168, 2048, 256, 8),
        # a decode batch with a popular few experts (Zipf)
        _mx("mx batch", "mx_ffn", 32, "bf16", 64, 7168, 2048, 256, 8, 1.0),
        # the Llama4-Maverick-shaped experts, one expert a token
        _mx("mx wide", "mx_ffn", 32, "bf16", 16, 5120, 8192, 128, 1),
        # a prompt: about 1000 rows for each expert of a shard
        _mx("mx prompt", "mx_ffn", 16, "bf16", 4096, 7168, 2048, 32, 8),
        # float32 rows through one product; nothing is a multiple of a tile
        _mx("mx down f32", "mx_down", 32, "f32", 33, 1440, 992, 7, 3),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    if rng.random() < 0.45:
        groups = rng.choice((1, 1, 2, 4, 8))
        E = groups * max(1, _log_int(rng, 2, 512) // groups)
        top_groups = rng.randint(max(1, groups // 2), groups)
        kept = top_groups * (E // groups)
        k = rng.randint(1, min(16, kept))
        T = max(1, min(_log_int(rng, 1, 65536), MAX_LOGITS // E))
        # the one weight of k = 1 is constant if it is renormalised
        case = _route("", rng.choice(("route", "route", "route_backward")),
                      T, E, k, rng.choice(("softmax", "sigmoid")), groups,
                      top_groups, rng.randint(1, min(2, E // groups)),
                      rng.random() < 0.6, k > 1 and rng.random() < 0.6,
                      rng.choice((1.0, 2.5)))
        del case["name"]
        return case
    op = rng.choice(("mx_rows", "mx_weights", "mx_ffn", "mx_ffn", "mx_ffn",
                     "mx_down"))
    dtype = "bf16" if op == "mx_ffn" else rng.choice(("bf16", "f32"))
    block = rng.choice((16, 32))
    H = 32 * _log_int(rng, 1, 7168 // 32)
    F = 32 * _log_int(rng, 2, 8192 // 32)
    E, k, T, skew = 1, 1, _log_int(rng, 1, 8192), 0.0
    if op == "mx_rows":
        F = 0
        T = max(1, min(T, MAX_ELEMENTS // H // (2 if dtype == "f32" else 1)))
    else:
        E = _log_int(rng, 1, 256)
    if op == "mx_weights":
        T = 0
        E = max(1, min(E, 8 * 7168 * 2048 // (H * F)
                       // (2 if dtype == "f32" else 1)))
        F = min(F, 8 * 7168 * 2048 // H)
    elif op != "mx_rows":
        k, skew = rng.randint(1, min(8, E)), rng.choice((0.0, 1.0))
        while 3 * E * H * F > MAX_WEIGHTS:
            E = max(1, E // 2)
            k = min(k, E)
        while 3 * T * k * H * F > MAX_PRODUCTS:
            T = max(1, T // 2)
    case = _mx("", op, block, dtype, T, H, F, E, k, skew)
    del case["name"]
    return case


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _draws(case, seed):
    """The case's inputs from the seed alone, and nothing of the library."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=g, device="cuda")

    s, T = {}, case["T"]
    if case["op"].startswith("route"):
        E, k = case["E"], case["k"]
        s["logits"] = normal(T, E) * 1.5
        s["bias"] = normal(E) * 0.02 if case["bias"] else None
        if case["op"] == "route_backward":
            s["dw"] = normal(T, k)
            # what the forward pass chose: distinct experts of each token
            s["idx"] = (torch.rand((T, E), generator=g, device="cuda")
                        + s["logits"].sigmoid()).topk(k).indices.int()
        return s
    E, H, F, dt = case["E"], case["H"], case["F"], _dtype(case)
    small = case["block"] == 16
    # values per unit of a tensor's block scales (blocks of 16 alone)
    s["x_scale"], s["h_scale"] = (0.011, 0.013) if small else (1.0, 1.0)
    if case["op"] == "mx_rows":
        # channels of unlike size, some of them far out
        s["x"] = (normal(T, H) * (normal(H) * 0.7).exp()).to(dt)
        return s
    if case["op"] == "mx_weights":
        s["w"] = torch.stack([(normal(H, F) * 0.02).to(dt)
                              for _ in range(E)])
        s["scale"] = (s["w"].reshape(E, -1).abs().amax(1).float()
                      / (448 * 6)) if small else None
        return s
    k = case["k"]
    # the k largest of Gumbel noise plus the popularity of the experts
    u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
    pop = torch.arange(1, E + 1, device="cuda").log() * -case["skew"]
    chosen = (pop - (-u.log()).log()).topk(k, dim=1).indices
    counts = torch.bincount(chosen.reshape(-1), minlength=E)
    s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
    shapes = (("gate", H, F), ("up", H, F), ("down", F, H))
    if case["op"] == "mx_down":
        s["h"] = normal(T * k, F).to(dt)
        shapes = shapes[2:]
    else:
        s["x"] = (normal(T * k, H) * (normal(H) * 0.5).exp()).to(dt)
    for name, K, N in shapes:
        G = -(-K // case["block"] // 4) * 4
        q = {"codes": torch.randint(0, 256, (E, N, K // 2), generator=g,
                                    device="cuda", dtype=torch.uint8),
             # magnitudes of about 0.02 either way
             "scales": torch.randint(*((0x60, 0x7f) if small else (118, 121)),
                                     (E, N, G), generator=g, device="cuda",
                                     dtype=torch.uint8),
             "scale": 2e-5 + 4e-5 * torch.rand(E, generator=g, device="cuda")
             if small else None}
        s[name] = q
    return s


def _active(offsets):
    """Groups with rows, and for each the sorted rows it holds, padded to the
    longest group with a row number past the end."""
    counts = (offsets[1:] - offsets[:-1]).long()
    groups = counts.nonzero().reshape(-1)
    at = offsets[:-1].long()[groups, None] + torch.arange(
        int(counts.max()), device=offsets.device)
    inside = at < offsets[1:].long()[groups, None]
    return groups, torch.where(inside, at, int(offsets[-1])), inside


def prepare(case, seed):
    s = _draws(case, seed)
    s["case"] = case
    if case["op"] in ("mx_ffn", "mx_down"):
        # how the routed rows lie: a serving program knows it from routing
        s["groups"], s["rows"], s["inside"] = _active(s["offsets"])
    if own:
        _prepare_own(s)
    return s


def _prepare_own(s):
    import mixture_experts_token_gb300 as moe
    case = s["case"]
    s["moe"], op, T, E, k = moe, case["op"], case["T"], case["E"], case["k"]

    def empty(shape, dtype):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if op.startswith("route"):
        s["cfg"] = moe.make_config(T, 8, E, k, 0, 1)
        s["opt"] = moe.make_route_scores(
            moe.MOE_SCORE_SIGMOID if case["score"] == "sigmoid" else
            moe.MOE_SCORE_SOFTMAX, case["groups"], case["top_groups"],
            case["group_top"], case["renorm"], case["scale"])
        if op == "route":
            s["idx"] = empty((T, k), torch.int32)
            s["w"] = empty((T, k), torch.float32)
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        else:
            s["dlogits"] = empty((T, E), torch.float32)
        return
    H, F, dt = case["H"], case["F"], _dtype(case)
    s["mx"] = moe.make_mx(case["block"], s["x_scale"], s["h_scale"])
    if op == "mx_rows":
        s["q"] = moe.alloc_mx_rows(s["mx"], T, H)
        s["values"] = empty((T, H), dt)
    elif op == "mx_weights":
        s["q"] = moe.alloc_mx_rows(s["mx"], E * F, H)
        s["packed"] = moe.alloc_mx(s["mx"], E, H, F)
        s["values"] = empty((E, H, F), dt)
    else:
        s["cfg"] = moe.make_config(T, H, E, k, F, 1, dtype=case["dtype"])
        # the weights laid out once, as a program does when it loads them
        for name, K, N in (("gate", H, F), ("up", H, F), ("down", F, H)):
            if name in s:
                q = s[name]
                q["packed"] = moe.alloc_mx(s["mx"], E, K, N)
                moe.moe_mx_pack(s["mx"], E, K, N, q.pop("codes"),
                                q.pop("scales"), q["packed"])
        s["y"] = empty((T * k, H), dt)
        s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        if op == "mx_down":
            s["q"] = moe.alloc_mx_rows(s["mx"], T * k, F)
        else:
            s["ws"] = moe.mx_workspace(s["cfg"], s["mx"])


# ------------------------------------------------------- the plain forms --
def _ranked(v):
    """Values and indexes from the largest down, equal ones by index."""
    return torch.sort(v, dim=-1, descending=True, stable=True)


def _plain_route(s):
    case, T, E = s["case"], s["case"]["T"], s["case"]["E"]
    x = s["logits"].double()
    p = torch.sigmoid(x)
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    c = p if s["bias"] is None else p + s["bias"].double()
    if case["groups"] > 1:
        by_group = c.view(T, case["groups"], -1)
        best = _ranked(by_group)[0][..., :case["group_top"]].sum(2)
        kept = _ranked(best)[1][:, :case["top_groups"]]
        keep = torch.zeros_like(best, dtype=torch.bool).scatter_(1, kept, True)
        c = torch.where(keep[..., None], by_group, -math.inf).view(T, E)
    idx = _ranked(c)[1][:, :case["k"]]
    w = p.gather(1, idx)
    if case["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return {"idx": idx.int(), "w": (w * case["scale"]).float()}


def _plain_route_backward(s):
    case, x = s["case"], s["logits"]
    idx, dw = s["idx"].long(), s["dw"] * case["scale"]
    p = torch.sigmoid(x)
    if case["score"] == "softmax":
        p = torch.exp(x - x.amax(1, keepdim=True))
        p = p / p.sum(1, keepdim=True)
    chosen = p.gather(1, idx)
    if case["renorm"]:
        z = chosen.sum(1, keepdim=True)
        dw = (dw - (dw * chosen).sum(1, keepdim=True) / z) / z
    dp = torch.zeros_like(x).scatter_(1, idx, dw)
    if case["score"] == "sigmoid":
        return {"dlogits": dp * p * (1 - p)}
    return {"dlogits": p * (dp - (dp * p).sum(1, keepdim=True))}


def _two_to(e):
    """2^e in float32, exactly, for whole numbers e of -126 to 127."""
    return ((e + 127).int() << 23).view(torch.float32)


def _quantised(v, block, scale):
    """What the rows of float32 v [..., K] are worth once quantised."""
    b = v.reshape(*v.shape[:-1], -1, block)
    if block == 16:
        b = b * (1 / torch.tensor(scale, device=v.device))
    most = b.abs().amax(-1, keepdim=True)
    if block == 32:
        # the exponent e of most = m 2^e, 1/2 <= m < 1, less one and two
        s = _two_to(torch.frexp(most)[1].clamp(min=-123) - 3)
    else:
        s = (most / 6).clamp(max=448).to(torch.float8_e4m3fn).float()
    q = torch.where(s > 0, b.abs() / s, 0.0)
    # steps of 0.5 up to 2, of 1 up to 4 and of 2 up to 6, ties to even
    q = torch.where(q < 2, (q * 2).round() / 2,
                    torch.where(q < 4, q.round(), (q / 2).round() * 2))
    q = torch.copysign(q.clamp(max=6.0), b) * s
    return (q if block == 32 else q * scale).reshape(v.shape)


def _expanded(q, groups, block):
    """float32 weights [active, N, K] of the groups that have rows."""
    c, at = q["codes"][groups], q["scales"][groups]
    c = torch.stack([c & 15, c >> 4], 3).flatten(2)
    values = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=c.device)
    w = torch.cat([values, -values])[c.int()].unflatten(2, (-1, block))
    if block == 32:
        at = _two_to(at.int() - 127)
    else:
        at = (at.view(torch.float8_e4m3fn).float()
              * q["scale"][groups][:, None, None])
    return (w * at[:, :, :w.shape[2], None]).flatten(2)


def _product(x, q, s):
    """Rows x [active, most, K] of the groups times their weights."""
    return torch.bmm(x, _expanded(q, s["groups"],
                                  s["case"]["block"]).transpose(1, 2))


def _plain_mx(s):
    case, block, dt = s["case"], s["case"]["block"], _dtype(s["case"])
    if case["op"] == "mx_rows":
        return {"x": _quantised(s["x"].float(), block, s["x_scale"]).to(dt)}
    if case["op"] == "mx_weights":
        w = s["w"].float().transpose(1, 2)
        if block == 16:
            w = w * (1 / s["scale"])[:, None, None]
        w = _quantised(w, block, 1.0)
        if block == 16:
            w = w * s["scale"][:, None, None]
        return {"w": w.transpose(1, 2).contiguous().to(dt)}
    name = "h" if case["op"] == "mx_down" else "x"
    rows = _quantised(s[name].float(), block, s[name + "_scale"])
    h = torch.cat([rows, rows.new_zeros((1, rows.shape[1]))])[s["rows"]]
    if case["op"] == "mx_ffn":
        g, u = _product(h, s["gate"], s), _product(h, s["up"], s)
        h = _quantised(g * torch.sigmoid(g) * u, block, s["h_scale"])
    return {"y": _product(h, s["down"], s)[s["inside"]].to(dt)}


def _plain(s):
    op = s["case"]["op"]
    if op == "route":
        return _plain_route(s)
    if op == "route_backward":
        return _plain_route_backward(s)
    return _plain_mx(s)


def run(s):
    if not own:
        return _plain(s)
    moe, case = s["moe"], s["case"]
    op, H, F, E, T = case["op"], case.get("H"), case.get("F"), case["E"], \
        case["T"]
    if op == "route":
        moe.moe_route_scores(s["cfg"], s["opt"], s["logits"], s["bias"],
                             s["idx"], s["w"], s["status"])
        return {"idx": s["idx"], "w": s["w"]}
    if op == "route_backward":
        moe.moe_route_scores_backward(s["cfg"], s["opt"], s["logits"],
                                      s["idx"], s["dw"], s["dlogits"])
        return {"dlogits": s["dlogits"]}
    if op == "mx_rows":
        codes, scales = s["q"]
        moe.moe_mx_quantize_rows(s["mx"], T, H, s["x"], s["x_scale"], codes,
                                 scales)
        moe.moe_mx_dequantize_rows(s["mx"], T, H, codes, scales, s["x_scale"],
                                   s["values"])
        return {"x": s["values"]}
    if op == "mx_weights":
        codes, scales = s["q"]
        moe.moe_mx_quantize(s["mx"], E, H, F, s["w"], s["scale"], codes,
                            scales)
        moe.moe_mx_pack(s["mx"], E, H, F, codes, scales, s["packed"])
        moe.moe_mx_dequantize(s["mx"], E, H, F, s["packed"], s["scale"],
                              s["values"])
        return {"w": s["values"]}
    if op == "mx_down":
        codes, scales = s["q"]
        moe.moe_mx_quantize_rows(s["mx"], T * case["k"], F, s["h"],
                                 s["h_scale"], codes, scales)
        moe.moe_gmm_down_mx(s["cfg"], s["mx"], codes, scales, s["offsets"],
                            s["down"]["packed"], s["down"]["scale"], s["y"],
                            s["status"])
        return {"y": s["y"]}
    moe.moe_gmm_swiglu_mx(
        s["cfg"], s["mx"], s["x"], s["offsets"], s["gate"]["packed"],
        s["up"]["packed"], s["down"]["packed"], s["gate"]["scale"],
        s["up"]["scale"], s["down"]["scale"], s["y"], s["status"], s["ws"])
    return {"y": s["y"]}


def work(case):
    """Inputs read once, outputs written once; for the products the weights
    of the experts that expect a row."""
    T, E, k = case["T"], case["E"], case["k"]
    if case["op"] == "route":
        return {"bytes": 4 * T * E + 8 * T * k, "flops": 10 * T * E}
    if case["op"] == "route_backward":
        # the sigmoid's gradient needs the chosen logits alone
        read = k if case["score"] == "sigmoid" else E
        return {"bytes": 4 * T * (read + E + 2 * k), "flops": 8 * T * E}
    b = 4 if case["dtype"] == "f32" else 2
    H, F, R = case["H"], case["F"], T * k
    if case["op"] == "mx_rows":
        return {"bytes": 2 * b * T * H, "flops": 6 * T * H}
    if case["op"] == "mx_weights":
        return {"bytes": 2 * b * E * H * F, "flops": 6 * E * H * F}
    each = H * F * (0.5 + 1 / case["block"])
    active = sum(_expected(case))
    if case["op"] == "mx_down":
        return {"bytes": int(active * each + b * R * (H + F)) + 4 * (E + 1),
                "flops": 2 * R * H * F}
    return {"bytes": int(3 * active * each + 2 * b * R * H) + 4 * (E + 1),
            "flops": 6 * R * H * F}


def _expected(case):
    """The chance of each expert to have a row: T tokens draw k experts with
    probabilities proportional to rank**-skew (without replacement, which
    k draws with replacement stand for except where k = E)."""
    E, k, T = case["E"], case["k"], case["T"]
    if k == E:
        return [1.0] * E
    if case["skew"] == 0.0:
        return [1 - (1 - k / E) ** T] * E
    p = [(e + 1.0) ** -case["skew"] for e in range(E)]
    z = sum(p)
    return [1 - (1 - min(1.0, q / z)) ** (k * T) for q in p]


# ------------------------------------------- the definitions in 64 bits --
def exact(case, seed):
    s = _draws(case, seed)
    if case["op"] == "route":
        return _exact_route(case, s)
    if case["op"] == "route_backward":
        return _exact_route_backward(case, s)
    block, scale = case["block"], s["x_scale"]
    if case["op"] == "mx_rows":
        return {"x": torch.cat([_grid(r.double(), block, scale)
                                for r in s["x"].split(1024)])}
    if case["op"] == "mx_weights":
        return {"w": torch.stack([
            _grid(w.double().T, block,
                  None if s["scale"] is None else s["scale"][e]).T
            for e, w in enumerate(s["w"])])}
    off, rows = s["offsets"].tolist(), []
    for e in range(case["E"]):
        if off[e] == off[e + 1]:
            continue
        if case["op"] == "mx_down":
            h = s["h"][off[e]:off[e + 1]].double()
        else:
            x = _grid(s["x"][off[e]:off[e + 1]].double(), block, scale)
            g = x @ _value(s["gate"], e, block)
            h = g / (1 + torch.exp(-g)) * (x @ _value(s["up"], e, block))
        h = _grid(h, block, s["h_scale"])
        rows.append(h @ _value(s["down"], e, block))
    return {"y": torch.cat(rows)}


def _exact_route(case, s):
    """Ranks are counts of what stands before: a larger score, or the same at
    a lower index."""
    T, E, G = case["T"], case["E"], case["groups"]

    def rank(v):
        n = torch.arange(v.shape[-1], device="cuda")
        before = (v[..., None, :] > v[..., :, None]) | (
            (v[..., None, :] == v[..., :, None]) & (n[None, :] < n[:, None]))
        return before.sum(-1)

    idx, weights = [], []
    for x in s["logits"].split(max(1, (1 << 27) // (E * E))):
        x = x.double()
        p = 1 / (1 + torch.exp(-x)) if case["score"] == "sigmoid" else \
            torch.exp(x - torch.logsumexp(x, 1)[:, None])
        c = p + (0 if s["bias"] is None else s["bias"].double())
        if G > 1:
            c = c.reshape(len(x), G, -1)
            front = rank(c) < case["group_top"]
            kept = rank((c * front).sum(2)) < case["top_groups"]
            c = c.masked_fill(~kept[:, :, None], -1e300).reshape(len(x), E)
        # the expert of rank j, for each j < k
        i = rank(c).argsort(1)[:, :case["k"]]
        w = torch.take_along_dim(p, i, 1)
        z = w.sum(1)[:, None] if case["renorm"] else 1.0
        idx.append(i.int())
        weights.append(case["scale"] * w / z)
    return {"idx": torch.cat(idx), "w": torch.cat(weights)}


def _exact_route_backward(case, s):
    """The Jacobian's rows, one chosen expert after another."""
    x, idx, k = s["logits"].double(), s["idx"].long(), case["k"]
    lp = torch.nn.functional.logsigmoid(x) if case["score"] == "sigmoid" \
        else x - torch.logsumexp(x, 1)[:, None]
    p = torch.exp(lp)
    w = torch.take_along_dim(p, idx, 1)
    if case["renorm"]:
        w = w / w.sum(1)[:, None]
    # d log w_j / d log p_i is [i = j] - w_i with renorm, else [i = j]
    a = case["scale"] * s["dw"].double() * w
    if case["renorm"]:
        a = a - w * a.sum(1)[:, None]
    # d log p_i / d x_e is [i = e](1 - p_i), or [i = e] - p_e
    out = torch.zeros_like(x)
    for j in range(k):
        out.scatter_add_(1, idx[:, j:j + 1], a[:, j:j + 1])
    if case["score"] == "sigmoid":
        return {"dlogits": out * (1 - p)}
    return {"dlogits": out - p * a.sum(1)[:, None]}


def _leading_bit(v):
    """The largest power of two that is not above v > 0, from v's bits."""
    return (v.view(torch.int64) >> 52 << 52).view(torch.float64)


def _grid(v, block, scale):
    """v [R, K] in float64 on the grid of its blocks: the nearest of the eight
    magnitudes, at a midpoint the one whose code is even."""
    if scale is not None and not torch.is_tensor(scale):
        scale = torch.tensor(scale, device="cuda")
    b = v.reshape(len(v), -1, block)
    if block == 16:
        # the product with the reciprocal is rounded to float32 by definition
        one = torch.ones((), device="cuda") if scale is None else scale
        b = (b.float() * one.reciprocal()).double()
    top = b.abs().max(2).values
    if block == 32:
        step = _leading_bit(top.clamp(min=2.0 ** -125)) / 4
    else:
        fine = _leading_bit((top / 6).clamp(min=2.0 ** -6)) / 8
        step = ((top / 6 / fine).round() * fine).clamp(max=448.0)
    unit = b.abs() / step.masked_fill(step == 0, 1.0)[..., None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0],
                       dtype=torch.float64, device="cuda")
    # a midpoint between codes c and c + 1 counts where c + 1 is even
    low = torch.bucketize(unit, mid, right=False)
    high = torch.bucketize(unit, mid, right=True)
    code = torch.where(high % 2 == 0, high, low)
    size = torch.where(code < 2, code * 0.5,
                       (1 + code % 2 * 0.5) * (1 << code // 2) / 2)
    out = b.sign() * size * step[..., None]
    if block == 16 and scale is not None:
        out = out * scale.double()
    return out.reshape(v.shape)


def _value(q, e, block):
    """Expert e's weights [K, N] in float64."""
    c = q["codes"][e].int()
    c = torch.stack([c % 16, c // 16], 2).reshape(len(c), -1)
    m = c % 8
    w = torch.where(m < 2, m * 0.5,
                    (1 + m % 2 * 0.5) * (1 << m // 2) / 2).double()
    w = w * (1 - 2 * (c // 8))
    at = q["scales"][e].int().repeat_interleave(block, 1)[:, :w.shape[1]]
    if block == 32:
        return (w * torch.exp2(at.double() - 127)).T
    # 4 exponent bits over 7, 3 mantissa bits; exponent 0 has no leading one
    ex, fr = at // 8, (at % 8) / 8.0
    s = torch.where(ex == 0, fr * 2.0 ** -6,
                    (1 + fr) * torch.exp2(ex.double() - 7))
    return (w * s * q["scale"][e].double()).T
