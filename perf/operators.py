"""What is timed of the block norms and of the experts' products with 4-bit
weights: the cases, their inputs, the plain forms and the library's calls.

Two operators:

* ``norm``, ``norm_backward``, ``out``, ``combine_out``, ``out_backward``:
  the norms before and after the MoE layer, with the gate and the residual
  scale of the branch.  N(v; w) = v * rstd * w, rstd = 1/sqrt(mean v^2 + eps);
  out = res_scale * x + gate * N(y; w_post), h = N(out; w_next).  ``out`` and
  the combined ``y`` are stored in the layer's type, and the norm that follows
  reads what was stored.
* ``w4``: the SwiGLU FFN of the routed rows with every expert's weights held
  as 4-bit codes with a scale (and optionally a zero point) for each group of
  the reduction axis: w = (code - zero) * scale.

``own`` chooses what ``run`` does: the plain form (elementary torch, 32 bits,
rounded once at each stored value) or the library.
"""
import math

import torch

own = False

EPS = 1e-6
GATES = ("none", "token", "channel", "full")
NORM_OPS = ("norm", "norm_backward", "out", "combine_out", "out_backward")
# the costliest cases that draw() may give: the listed ones
MAX_NORM_ELEMENTS = 8192 * 7168
MAX_WEIGHTS = 256 * 3 * 7168 * 2048
MAX_PRODUCTS = 1024 * 8 * 3 * 7168 * 2048


def _norm(name, op, T, H, dtype, gate="channel", k=1):
    return {"name": name, "op": op, "T": T, "H": H, "dtype": dtype,
            "gate": gate, "k": k}


def _w4(name, T, H, F, E, k, dtype, group, zeros, skew):
    return {"name": name, "op": "w4", "T": T, "H": H, "F": F, "E": E, "k": k,
            "dtype": dtype, "group": group, "zeros": zeros, "skew": skew}


def listed():
    return [
        # one token of one sequence leaves the DeepSeek-V3-shaped layer
        _norm("out token", "out", 1, 7168, "bf16"),
        # a training batch or a long prompt through the same layer
        _norm("out prompt", "out", 8192, 7168, "bf16"),
        # a decode batch: eight expert rows a token gathered on the way
        _norm("combine out batch", "combine_out", 128, 7168, "bf16", k=8),
        # the Llama4-Maverick-shaped layer (one expert a token), the gate a
        # number for each token
        _norm("combine out prompt", "combine_out", 8192, 5120, "bf16",
              "token"),
        # the training step's backward at the DeepSeek-V3-shaped layer
        _norm("out backward", "out_backward", 8192, 7168, "bf16"),
        # float32 training with a gate computed for every element, T odd
        _norm("out backward f32", "out_backward", 2047, 5120, "f32", "full"),
        # the norm before the small layer, backward
        _norm("norm backward small", "norm_backward", 4096, 1024, "bf16"),
        # one token, DeepSeek-V3-shaped experts: 8 of 256 are read
        _w4("w4 token", 1, 7168, 2048, 256, 8, "bf16", 128, False, 0.0),
        # a decode batch with a popular few experts (Zipf)
        _w4("w4 batch", 64, 7168, 2048, 256, 8, "bf16", 128, False, 1.0),
        # the Llama4-Maverick-shaped experts, small groups with zero points
        _w4("w4 wide", 16, 5120, 8192, 128, 1, "bf16", 32, True, 0.0),
        # odd sizes in float32: nothing is a multiple of a tile
        _w4("w4 odd f32", 33, 1412, 1004, 7, 3, "f32", 64, True, 0.0),
        # a short prompt: about 32 rows for each expert
        _w4("w4 prompt", 1024, 7168, 2048, 256, 8, "bf16", 128, False, 0.0),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dtype = rng.choice(("bf16", "bf16", "bf16", "f32"))
    step = 8 if dtype == "bf16" else 4
    if rng.random() < 0.55:
        op = rng.choice(NORM_OPS)
        H = max(1, _log_int(rng, 64, 7168) // step) * step
        T = _log_int(rng, 1, 8192)
        k = rng.choice((1, 2, 3, 4, 8)) if op == "combine_out" else 1
        scale = (2 if dtype == "f32" else 1) * (k + 4) / 5
        T = max(1, min(T, int(MAX_NORM_ELEMENTS / H / scale)))
        case = _norm("", op, T, H, dtype, rng.choice(GATES), k)
    else:
        H = max(1, _log_int(rng, 64, 7168) // step) * step
        F = max(1, _log_int(rng, 64, 8192) // step) * step
        E = _log_int(rng, 1, 256)
        k = rng.randint(1, min(8, E))
        T = _log_int(rng, 1, 1024)
        while 3 * E * H * F > MAX_WEIGHTS:
            E = max(1, E // 2)
            k = min(k, E)
        while 3 * T * k * H * F > MAX_PRODUCTS / (8 if dtype == "f32" else 1):
            T = max(1, T // 2)
        case = _w4("", T, H, F, E, k, dtype, rng.choice((32, 64, 128)),
                   rng.random() < 0.5, rng.choice((0.0, 1.0)))
    del case["name"]
    return case


def _dtype(case):
    return torch.float32 if case["dtype"] == "f32" else torch.bfloat16


def _draws(case, seed):
    """The case's inputs from the seed alone, and nothing of the library."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    dt, T, H = _dtype(case), case["T"], case["H"]

    def normal(shape, std=1.0, dtype=dt, mean=0.0):
        v = torch.randn(shape, generator=g, device="cuda")
        return v.mul_(std).add_(mean).to(dtype)

    def permutation(n):
        return torch.rand(n, generator=g, device="cuda").argsort()

    s = {}
    if case["op"] == "w4":
        E, k, F, group = case["E"], case["k"], case["F"], case["group"]
        # the k largest of Gumbel noise plus the popularity of the experts
        u = torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)
        pop = torch.arange(1, E + 1, device="cuda").log() * -case["skew"]
        idx = (pop - (-u.log()).log()).topk(k, dim=1).indices
        counts = torch.bincount(idx.reshape(-1), minlength=E)
        s["x"] = normal((T * k, H))
        s["offsets"] = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).int()
        for name, K, N in (("gate", H, F), ("up", H, F), ("down", F, H)):
            G = -(-K // group)
            s[name] = {
                "codes": torch.randint(0, 256, (E, K // 2, N), generator=g,
                                       device="cuda", dtype=torch.uint8),
                # 16 steps that span about two standard deviations of 0.02
                "scales": (0.005 * (0.5 + torch.rand(
                    (E, G, N), generator=g, device="cuda"))).bfloat16(),
                "zeros": torch.randint(6, 11, (E, G, N), generator=g,
                                       device="cuda", dtype=torch.uint8)
                if case["zeros"] else None}
        return s
    s["w_post"] = normal(H, 0.1, torch.float32, 1.0)
    s["w_next"] = normal(H, 0.1, torch.float32, 1.0)
    s["gate"] = {"none": lambda: None,
                 "token": lambda: normal(T, 0.3, torch.float32, 0.5),
                 "channel": lambda: normal(H, 0.3, torch.float32, 0.5),
                 "full": lambda: normal((T, H), 0.3, dt, 0.5)}[case["gate"]]()
    s["x"] = normal((T, H), 2.0)
    if case["op"] == "combine_out":
        k = case["k"]
        s["y_sorted"] = normal((T * k, H))
        s["row_of"] = permutation(T * k).int().reshape(T, k)
        # rows that a full shard dropped
        s["row_of"][torch.rand((T, k), generator=g, device="cuda") < 0.02] = -1
        s["topk_w"] = torch.rand((T, k), generator=g, device="cuda").softmax(1)
    else:
        s["y"] = normal((T, H))
    if case["op"].endswith("backward"):
        s["dout"] = normal((T, H))
        s["dh"] = normal((T, H))
        # what the forward pass kept: its float32 statistics
        for name, v in (("rstd_y", s["y"]), ("rstd_x", s["x"])):
            s[name] = (v.float().square().mean(1) + EPS).rsqrt()
    return s


def _active(offsets, E):
    """Groups with rows, and for each the sorted rows it holds, padded to the
    longest group with a row number past the end."""
    counts = (offsets[1:] - offsets[:-1]).long()
    groups = counts.nonzero().reshape(-1)
    most = int(counts.max())
    at = offsets[:-1].long()[groups, None] + torch.arange(
        most, device=offsets.device)
    inside = at < offsets[1:].long()[groups, None]
    return groups, torch.where(inside, at, int(offsets[-1])), inside


def prepare(case, seed):
    s = _draws(case, seed)
    s["case"] = case
    dt, T, H = _dtype(case), case["T"], case["H"]

    def empty(shape, dtype=dt):
        return torch.empty(shape, dtype=dtype, device="cuda")

    if case["op"] == "w4":
        E, F, R = case["E"], case["F"], case["T"] * case["k"]
        # how the routed rows lie: a serving program knows it from routing
        s["groups"], s["rows"], s["inside"] = _active(s["offsets"], E)
        if own:
            import mixture_experts_token_gb300 as moe
            s["moe"] = moe
            s["cfg"] = moe.make_config(case["T"], H, E, case["k"], F, 1,
                                       dtype=case["dtype"])
            s["w4"] = moe.make_w4(case["group"], case["zeros"])
            # the weights laid out once, as a program does when it loads them
            for name, K, N in (("gate", H, F), ("up", H, F), ("down", F, H)):
                q = s[name]
                s[name] = moe.alloc_w4(s["w4"], E, K, N)
                moe.moe_w4_pack(s["w4"], E, K, N, q["codes"], q["scales"],
                                q["zeros"], s[name])
            s["h"], s["y"] = empty((R, F)), empty((R, H))
            s["status"] = torch.zeros(1, dtype=torch.int32, device="cuda")
        return s
    if own:
        import mixture_experts_token_gb300 as moe
        s["moe"] = moe
        k = case["k"]
        s["cfg"] = moe.make_config(T, H, k, k, 0, 1, dtype=case["dtype"])
        s["opt"] = moe.make_block_norm(
            eps=EPS, res_scale=0.9, gate=GATES.index(case["gate"]))
        for name in ("out", "h", "y_out", "dx", "dy"):
            s[name] = empty((T, H))
        s["rstd"] = [empty(T, torch.float32) for _ in range(2)]
        s["dw"] = [empty(H, torch.float32) for _ in range(2)]
        s["dgate"] = None if s["gate"] is None else torch.empty_like(s["gate"])
        s["ws"] = moe.layer_workspace(s["cfg"], moe.MOE_WS_BLOCK_BACKWARD)
    return s


def _rows_norm(v, w):
    r = (v.square().mean(1) + EPS).rsqrt()
    return v * r[:, None] * w, r




def _gate(case, gate):
    if gate is None:
        return 1.0
    return gate.float()[:, None] if case["gate"] == "token" else gate.float()


def _dequantised(q, groups, case, K):
    """float32 weights [active, K, N] of the groups that have rows."""
    c = q["codes"][groups]
    w = torch.stack([c & 15, c >> 4], 2).reshape(len(groups), K, -1).float()
    g = torch.arange(K, device=c.device) // case["group"]
    w -= q["zeros"][groups].float()[:, g] if case["zeros"] else 8.0
    w *= q["scales"][groups].float()[:, g]
    return w


def _plain_w4(s):
    case, H, F = s["case"], s["case"]["H"], s["case"]["F"]
    groups, rows, inside = s["groups"], s["rows"], s["inside"]
    x = torch.cat([s["x"].float(), s["x"].new_zeros((1, H)).float()])[rows]
    g = torch.bmm(x, _dequantised(s["gate"], groups, case, H))
    u = torch.bmm(x, _dequantised(s["up"], groups, case, H))
    h = g * torch.sigmoid(g) * u
    y = torch.bmm(h, _dequantised(s["down"], groups, case, F))
    dt = s["x"].dtype
    return {"h": h[inside].to(dt), "y": y[inside].to(dt)}


def _norm_backward(v, r, w, dh):
    """Gradients of N(v; w) for the upstream gradient dh."""
    vh = v * r[:, None]
    dv = dh * w
    dv = r[:, None] * (dv - vh * (dv * vh).mean(1)[:, None])
    return dv, (dh * vh).sum(0)


def _plain(s):
    case, op, dt = s["case"], s["case"]["op"], s["x"].dtype
    if op == "w4":
        return _plain_w4(s)
    x, gate = s["x"].float(), _gate(case, s["gate"])
    if op == "norm":
        h, r = _rows_norm(x, s["w_next"])
        return {"h": h.to(dt), "rstd": r}
    if op == "norm_backward":
        dx, dw = _norm_backward(x, s["rstd_x"], s["w_next"], s["dh"].float())
        return {"dx": (dx + s["dout"].float()).to(dt), "dw": dw}
    if op == "out_backward":
        # s["x"] stands for the stored output of the forward pass
        do, dw_next = _norm_backward(x, s["rstd_x"], s["w_next"],
                                     s["dh"].float())
        do = do + s["dout"].float()
        y, r = s["y"].float(), s["rstd_y"]
        dn = do * gate
        dy, dw_post = _norm_backward(y, r, s["w_post"], dn)
        got = {"dx": (0.9 * do).to(dt), "dy": dy.to(dt), "dw_post": dw_post,
               "dw_next": dw_next}
        if s["gate"] is not None:
            dg = do * (y * r[:, None] * s["w_post"])
            dg = dg.sum(1) if case["gate"] == "token" else dg
            dg = dg.sum(0) if case["gate"] == "channel" else dg
            got["dgate"] = dg.to(s["gate"].dtype)
        return got
    got = {}
    if op == "combine_out":
        rows = s["row_of"].long()
        w = torch.where(rows >= 0, s["topk_w"], 0.0)
        y = (s["y_sorted"][rows.clamp(min=0)].float() * w[..., None]).sum(1)
        got["y"] = y.to(dt)
        y = got["y"].float()
    else:
        y = s["y"].float()
    n, got["rstd_y"] = _rows_norm(y, s["w_post"])
    got["out"] = (0.9 * x + gate * n).to(dt)
    h, got["rstd_out"] = _rows_norm(got["out"].float(), s["w_next"])
    got["h"] = h.to(dt)
    return got


def run(s):
    if not own:
        return _plain(s)
    moe, op = s["moe"], s["case"]["op"]
    if op == "w4":
        moe.moe_gmm_swiglu_w4(s["cfg"], s["w4"], s["x"], s["offsets"],
                              s["gate"], s["up"], s["down"], s["h"], s["y"],
                              s["status"])
        return {"h": s["h"], "y": s["y"]}
    if op == "norm":
        moe.moe_norm(s["cfg"], s["opt"], s["x"], s["w_next"], s["h"],
                     s["rstd"][0])
        return {"h": s["h"], "rstd": s["rstd"][0]}
    if op == "norm_backward":
        moe.moe_norm_backward(s["cfg"], s["opt"], s["x"], s["w_next"],
                              s["rstd_x"], s["dh"], s["dout"], s["dx"],
                              s["dw"][0], False, s["ws"])
        return {"dx": s["dx"], "dw": s["dw"][0]}
    if op == "out_backward":
        moe.moe_block_out_backward(
            s["cfg"], s["opt"], s["y"], s["w_post"], s["gate"], s["rstd_y"],
            s["x"], s["w_next"], s["rstd_x"], s["dout"], s["dh"], s["dx"],
            s["dy"], s["dw"][0], s["dgate"], s["dw"][1], False, s["ws"])
        got = {"dx": s["dx"], "dy": s["dy"], "dw_post": s["dw"][0],
               "dw_next": s["dw"][1]}
        if s["dgate"] is not None:
            got["dgate"] = s["dgate"]
        return got
    got = {"rstd_y": s["rstd"][0], "out": s["out"], "rstd_out": s["rstd"][1],
           "h": s["h"]}
    if op == "combine_out":
        moe.moe_combine_block_out(
            s["cfg"], s["opt"], s["y_sorted"], s["row_of"], s["topk_w"],
            s["x"], s["w_post"], s["gate"], s["w_next"], s["y_out"], s["out"],
            s["h"], s["rstd"][0], s["rstd"][1])
        got["y"] = s["y_out"]
    else:
        moe.moe_block_out(s["cfg"], s["opt"], s["x"], s["y"], s["w_post"],
                          s["gate"], s["w_next"], s["out"], s["h"],
                          s["rstd"][0], s["rstd"][1])
    return got


def work(case):
    """Inputs read once, outputs written once; for w4 the weights of the
    experts that expect a row (with all experts equally likely)."""
    b = 4 if case["dtype"] == "f32" else 2
    T, H = case["T"], case["H"]
    if case["op"] == "w4":
        E, k, F, R = case["E"], case["k"], case["F"], case["T"] * case["k"]
        active = sum(_expected(case))
        groups = 2 * -(-H // case["group"]) * F + -(-F // case["group"]) * H
        per_expert = 3 * H * F // 2 + groups * (3 if case["zeros"] else 2)
        return {"bytes": active * per_expert + R * (2 * H + F) * b + 4 * (E + 1),
                "flops": 2 * 3 * R * H * F}
    gate = {"none": 0, "token": 4 * T, "channel": 4 * H, "full": b * T * H}
    row, full = b * T * H, gate[case["gate"]]
    if case["op"] == "norm":
        return {"bytes": 2 * row + 4 * (T + H), "flops": 4 * T * H}
    if case["op"] == "norm_backward":
        return {"bytes": 4 * row + 4 * (T + 2 * H), "flops": 9 * T * H}
    if case["op"] == "out":
        return {"bytes": 4 * row + full + 8 * (T + H), "flops": 10 * T * H}
    if case["op"] == "combine_out":
        k = case["k"]
        return {"bytes": (k + 4) * row + 8 * T * k + full + 8 * (T + H),
                "flops": (10 + 2 * k) * T * H}
    return {"bytes": 6 * row + 2 * full + 8 * T + 16 * H,
            "flops": 24 * T * H}


def _expected(case):
    """The chance of each expert to have a row: T tokens draw k experts with
    probabilities proportional to rank**-skew (without replacement, which
    k draws with replacement stand for except where k = E)."""
    E, k, T = case["E"], case["k"], case["T"]
    if k == E:
        return [1.0] * E
    p = [(e + 1.0) ** -case["skew"] for e in range(E)]
    z = sum(p)
    if case["skew"] == 0.0:
        return [1 - (1 - k / E) ** T] * E
    return [1 - (1 - min(1.0, q / z)) ** (k * T) for q in p]


def exact(case, seed):
    """The definitions in 64 bits, one expert or one block of rows at a time.
    Stored values (out, y) are rounded to the layer's type, as the definition
    says, before the norm that reads them."""
    s = _draws(case, seed)
    d, dt, op = torch.float64, _dtype(case), case["op"]
    if op == "w4":
        return _exact_w4(case, s)
    T, H = case["T"], case["H"]
    keys = {}
    sums = {}
    for a in range(0, T, 2048):
        z = min(T, a + 2048)
        got, add = _exact_rows(case, s, a, z, d, dt, op)
        for name, v in got.items():
            keys.setdefault(name, []).append(v)
        for name, v in add.items():
            sums[name] = sums.get(name, 0) + v
    out = {name: torch.cat(v) for name, v in keys.items()}
    out.update(sums)
    return out


def _exact_rows(case, s, a, z, d, dt, op):
    """Rows a..z: (values by row, column sums over these rows)."""
    H = case["H"]
    wp, wn = s["w_post"].to(d), s["w_next"].to(d)
    x = s["x"][a:z].to(d)
    g = torch.ones((z - a, H), dtype=d, device="cuda")
    if case["gate"] == "channel":
        g = g * s["gate"].to(d)
    elif case["gate"] == "token":
        g = g * s["gate"][a:z].to(d).unsqueeze(1)
    elif case["gate"] == "full":
        g = s["gate"][a:z].to(d)

    def inverse_rms(v):
        return 1 / torch.sqrt(torch.einsum("tc,tc->t", v, v) / H + EPS)

    def transposed(v, r, w, up):
        # d/dv of v r(v) w along `up`: r*up*w - r^3 v <up*w, v>/H
        dot = torch.einsum("tc,tc,c->t", up, v, w) / H
        return (torch.einsum("t,tc,c->tc", r, up, w)
                - torch.einsum("t,tc->tc", r ** 3 * dot, v))

    if op == "norm":
        r = inverse_rms(x)
        return {"h": torch.einsum("tc,t,c->tc", x, r, wn), "rstd": r}, {}
    if op.endswith("backward"):
        up, res = s["dh"][a:z].to(d), s["dout"][a:z].to(d)
        rx = s["rstd_x"][a:z].to(d)
        do = transposed(x, rx, wn, up) + res
        dwn = torch.einsum("tc,tc,t->c", up, x, rx)
        if op == "norm_backward":
            return {"dx": do}, {"dw": dwn}
        y, ry = s["y"][a:z].to(d), s["rstd_y"][a:z].to(d)
        got = {"dx": 0.9 * do, "dy": transposed(y, ry, wp, do * g)}
        add = {"dw_next": dwn,
               "dw_post": torch.einsum("tc,tc,tc,t->c", do, g, y, ry)}
        if case["gate"] == "channel":
            add["dgate"] = torch.einsum("tc,tc,t,c->c", do, y, ry, wp)
        elif case["gate"] == "token":
            got["dgate"] = torch.einsum("tc,tc,t,c->t", do, y, ry, wp)
        elif case["gate"] == "full":
            got["dgate"] = torch.einsum("tc,tc,t,c->tc", do, y, ry, wp)
        return got, add
    got = {}
    if op == "combine_out":
        y = torch.zeros((z - a, H), dtype=d, device="cuda")
        for j in range(case["k"]):
            row = s["row_of"][a:z, j].long()
            kept = row >= 0
            y[kept] += (s["y_sorted"][row[kept]].to(d)
                        * s["topk_w"][a:z, j].to(d)[kept].unsqueeze(1))
        got["y"] = y
        y = y.to(dt).to(d)
    else:
        y = s["y"][a:z].to(d)
    ry = inverse_rms(y)
    got["rstd_y"] = ry
    got["out"] = 0.9 * x + g * torch.einsum("tc,t,c->tc", y, ry, wp)
    o = got["out"].to(dt).to(d)
    ro = inverse_rms(o)
    got["rstd_out"] = ro
    got["h"] = torch.einsum("tc,t,c->tc", o, ro, wn)
    return got, {}


def _exact_w4(case, s):
    d, H, F, g = torch.float64, case["H"], case["F"], case["group"]
    off = s["offsets"].tolist()
    h = torch.empty((off[-1], F), dtype=d, device="cuda")
    y = torch.empty((off[-1], H), dtype=d, device="cuda")

    def weights(q, e, K):
        out = torch.empty((K, q["codes"].shape[2]), dtype=d, device="cuda")
        out[0::2] = (q["codes"][e] % 16).to(d)
        out[1::2] = (q["codes"][e] // 16).to(d)
        for i in range(q["scales"].shape[1]):
            rows = out[i * g:(i + 1) * g]
            rows -= q["zeros"][e, i].to(d) if case["zeros"] else 8.0
            rows *= q["scales"][e, i].to(d)
        return out

    for e in range(case["E"]):
        a, z = off[e], off[e + 1]
        if a == z:
            continue
        x = s["x"][a:z].to(d)
        p = x @ weights(s["gate"], e, H)
        h[a:z] = p / (1 + torch.exp(-p)) * (x @ weights(s["up"], e, H))
        y[a:z] = h[a:z] @ weights(s["down"], e, F)
    return {"h": h, "y": y}
