"""The block norms on the GPU against the float64 oracle.

Tolerances.  A float32 evaluation of these formulas rounds each term a few
times (at most 12) and adds at most H of them in a tree whose serial part is
under 64 long, so its error is below (12 + 64 + 10) * 2^-24 < 6e-6 of the sum
of absolute terms (the oracle returns it).  A column sum over T rows adds at
most T/304 + 64 serial steps: 1e-5 covers T <= 10000.  What is stored in bf16
is rounded once more, and rounding keeps order: the stored value lies between
the two ends of that interval, rounded.
"""
import numpy as np
import pytest
import torch

import mixture_experts_token_gb300 as moe
from oracle import block_ref as ref
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

GATES = ("none", "token", "channel", "full")
REL = 1e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(got, want, mag, what=""):
    """|got - want| within REL of the terms' magnitude, before the
    rounding to the stored type."""
    tol = REL * mag + 1e-30
    lo, hi = (f64(torch.from_numpy(np.asarray(v)).float().to(got.dtype))
              for v in (want - tol, want + tol))
    v = f64(got)
    bad = ~((lo <= v) & (v <= hi))
    worst = float(np.nanmax(np.abs(v - want) / tol))
    assert not bad.any(), (what, int(bad.sum()), worst)


def tensors(T, H, dtype, kind, seed=0):
    g = torch.Generator().manual_seed(seed)

    def normal(*shape, std=1.0, mean=0.0, dt=DT[dtype]):
        return (torch.randn(*shape, generator=g) * std + mean).to(dt).cuda()
    f = torch.float32
    gate = {"none": lambda: None, "token": lambda: normal(T, dt=f),
            "channel": lambda: normal(H, dt=f),
            "full": lambda: normal(T, H)}[kind]()
    return dict(x=normal(T, H, std=2.0), y=normal(T, H),
                w_post=normal(H, std=0.2, mean=1.0, dt=f),
                w_next=normal(H, std=0.2, mean=1.0, dt=f), gate=gate,
                dout=normal(T, H), dh=normal(T, H))


def config(T, H, dtype, k=1):
    return moe.make_config(T, H, k, k, 0, 1, dtype=dtype)


def n64(t):
    return None if t is None else f64(t)


def forward(c, o, s, kind, post=True, nxt=True, combine=None):
    T, H, dt = s["x"].shape[0], s["x"].shape[1], s["x"].dtype
    e = lambda *shape, d=dt: torch.full(shape, 7, dtype=d, device="cuda")  # noqa: E731
    out = dict(out=e(T, H), h=e(T, H) if nxt else None,
               rstd_y=e(T, d=torch.float32), rstd_out=e(T, d=torch.float32))
    tail = (s["w_post"] if post else None, s["gate"],
            s["w_next"] if nxt else None)
    if combine is None:
        moe.moe_block_out(c, o, s["x"], s["y"], *tail, *out.values())
    else:
        out["y"] = e(T, H)
        moe.moe_combine_block_out(
            c, o, *combine, s["x"], *tail, out["y"], out["out"], out["h"],
            out["rstd_y"], out["rstd_out"])
    torch.cuda.synchronize()
    return out


def check_forward(got, s, y, kind, o, post=True, nxt=True):
    want, mag = ref.block_out(f64(s["x"]), y, n64(s["w_post"]) if post
                              else None, n64(s["gate"]), kind, o.eps,
                              o.w_offset, o.res_scale)
    close(got["out"], want, mag, "out")
    if post:
        r = ref.rstd(y, o.eps)
        close(got["rstd_y"], r, r, "rstd_y")
    if nxt:  # the next norm reads what was stored
        stored = f64(got["out"])
        h = ref.norm(stored, n64(s["w_next"]), o.eps, o.w_offset)
        close(got["h"], h, np.abs(stored) * ref.rstd(stored, o.eps)[:, None]
              * (abs(o.w_offset) + np.abs(n64(s["w_next"]))), "h")
        r = ref.rstd(stored, o.eps)
        close(got["rstd_out"], r, r, "rstd_out")


# a warp per row with 1, 2 and 4 words a lane, a CTA per row with 1, 2 and 4
# words a thread, and the widest row; T below, at and past a CTA's rows
SIZES = [(1, 8, "bf16"), (5, 64, "f32"), (9, 264, "bf16"), (3, 512, "bf16"),
         (130, 1000, "bf16"), (4, 1024, "bf16"), (7, 1032, "bf16"),
         (2, 4096, "bf16"), (6, 4104, "bf16"), (33, 7168, "bf16"),
         (3, 8200, "bf16"), (2, 16392, "bf16"), (2, 32768, "bf16"),
         (1, 4, "f32"), (11, 516, "f32"), (5, 1412, "f32"), (3, 5120, "f32"),
         (2, 16384, "f32")]


@pytest.mark.parametrize("T,H,dtype", SIZES)
@pytest.mark.parametrize("kind", GATES)
def test_block_out(T, H, dtype, kind):
    s = tensors(T, H, dtype, kind)
    o = moe.make_block_norm(1e-5, 0.0, 0.9, GATES.index(kind))
    got = forward(config(T, H, dtype), o, s, kind)
    check_forward(got, s, f64(s["y"]), kind, o)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("post,nxt", [(False, False), (False, True),
                                      (True, False)])
def test_block_out_without_a_norm(dtype, post, nxt):
    s = tensors(19, 264, dtype, "channel")
    o = moe.make_block_norm(1e-6, 1.0, -1.5, moe.MOE_GATE_CHANNEL)
    got = forward(config(19, 264, dtype), o, s, "channel", post, nxt)
    check_forward(got, s, f64(s["y"]), "channel", o, post, nxt)


@pytest.mark.parametrize("T,H,dtype", SIZES)
def test_norm(T, H, dtype):
    s = tensors(T, H, dtype, "none", seed=2)
    o = moe.make_block_norm(1e-6, 1.0)
    h = torch.empty_like(s["x"])
    r = torch.empty(T, device="cuda")
    moe.moe_norm(config(T, H, dtype), o, s["x"], s["w_next"], h, r)
    x = f64(s["x"])
    want = ref.norm(x, f64(s["w_next"]), o.eps, 1.0)
    close(h, want, np.abs(x) * ref.rstd(x, o.eps)[:, None]
          * (1 + np.abs(f64(s["w_next"]))), "h")
    close(r, ref.rstd(x, o.eps), ref.rstd(x, o.eps), "rstd")
    # in place, and without the statistic
    moe.moe_norm(config(T, H, dtype), o, s["x"], s["w_next"], s["x"])
    assert torch.equal(s["x"], h)


@pytest.mark.parametrize("T,H,k,dtype", [
    (1, 64, 1, "bf16"), (5, 1000, 2, "bf16"), (17, 1032, 8, "bf16"),
    (130, 512, 3, "bf16"), (4, 7168, 8, "bf16"), (6, 64, 32, "f32"),
    (3, 5120, 5, "f32"), (2, 16392, 4, "bf16")])
def test_combine_block_out(T, H, k, dtype):
    s = tensors(T, H, dtype, "full", seed=5)
    g = torch.Generator().manual_seed(9)
    ys = torch.randn(T * k, H, generator=g).to(DT[dtype]).cuda()
    row_of = torch.randperm(T * k, generator=g).int().reshape(T, k)
    row_of[torch.rand(T, k, generator=g) < 0.3] = -1
    row_of[T - 1] = -1                      # a token that lost every row
    w = torch.rand(T, k, generator=g)
    if T > 2:                               # a row that is not read may hold
        lost = sorted(set(range(T * k)) - set(row_of.reshape(-1).tolist()))
        ys[lost] = float("nan")             # anything
    c, o = config(T, H, dtype, k), moe.make_block_norm(
        1e-5, 0.0, 1.0, moe.MOE_GATE_FULL)
    row_of, w = row_of.cuda(), w.cuda()
    got = forward(c, o, s, "full", combine=(ys, row_of, w))
    y = torch.empty_like(s["y"])
    moe.moe_combine(c, ys, row_of, w, y)
    assert torch.equal(got["y"], y)         # the bits of the separate call
    check_forward(got, s, f64(y), "full", o)
    # and the same outputs without keeping y
    again = {n: torch.empty_like(v) for n, v in got.items()}
    moe.moe_combine_block_out(c, o, ys, row_of, w, s["x"], s["w_post"],
                              s["gate"], s["w_next"], None, again["out"],
                              again["h"])
    assert torch.equal(again["out"], got["out"])
    assert torch.equal(again["h"], got["h"])


def backward(c, o, s, out, kind, post=True, nxt=True, dout=True,
             accumulate=False, sums=None):
    T, H, dt = s["x"].shape[0], s["x"].shape[1], s["x"].dtype
    e = lambda *shape, d=dt: torch.full(shape, 7, dtype=d, device="cuda")  # noqa: E731
    f = torch.float32
    got = dict(dx=e(T, H), dy=e(T, H), dw_post=e(H, d=f) if post else None,
               dgate=None if s["gate"] is None else e(*s["gate"].shape,
                                                      d=s["gate"].dtype),
               dw_next=e(H, d=f) if nxt else None)
    got.update(sums or {})
    ry = ref.rstd(f64(s["y"]), o.eps)
    ro = ref.rstd(f64(out), o.eps)
    dev = lambda a: torch.from_numpy(a).float().cuda()  # noqa: E731
    ws = moe.layer_workspace(c, moe.MOE_WS_BLOCK_BACKWARD)
    ws.fill_(0xAB)
    moe.moe_block_out_backward(
        c, o, s["y"], s["w_post"] if post else None, s["gate"],
        dev(ry) if post else None, out, s["w_next"] if nxt else None,
        dev(ro) if nxt else None, s["dout"] if dout else None,
        s["dh"] if nxt else None, got["dx"], got["dy"], got["dw_post"],
        got["dgate"], got["dw_next"], accumulate, ws)
    torch.cuda.synchronize()
    return got


def check_backward(got, s, out, kind, o, post=True, nxt=True, dout=True):
    want = ref.block_out_backward(
        f64(s["y"]), n64(s["w_post"]) if post else None, n64(s["gate"]), kind,
        f64(out), n64(s["w_next"]) if nxt else None,
        f64(s["dout"]) if dout else None, f64(s["dh"]) if nxt else None,
        o.eps, o.w_offset, o.res_scale)
    for name, (v, mag) in want.items():
        close(got[name], v, mag, name)


@pytest.mark.parametrize("T,H,dtype", SIZES + [
    (2000, 64, "bf16"), (1217, 1024, "bf16"), (305, 1032, "bf16"),
    (609, 4104, "bf16"), (700, 516, "f32")])
@pytest.mark.parametrize("kind", GATES)
def test_block_out_backward(T, H, dtype, kind):
    s = tensors(T, H, dtype, kind, seed=1)
    o = moe.make_block_norm(1e-5, 1.0, 0.9, GATES.index(kind))
    out = s["x"]      # stands for the stored output of the forward pass
    got = backward(config(T, H, dtype), o, s, out, kind)
    check_backward(got, s, out, kind, o)


@pytest.mark.parametrize("kind", GATES)
@pytest.mark.parametrize("post,nxt,dout", [
    (False, False, True), (False, True, False), (True, False, True),
    (True, True, False)])
def test_block_out_backward_without_parts(kind, post, nxt, dout):
    s = tensors(37, 1032, "bf16", kind, seed=4)
    o = moe.make_block_norm(1e-6, 0.0, -0.5, GATES.index(kind))
    got = backward(config(37, 1032, "bf16"), o, s, s["x"], kind, post, nxt,
                   dout)
    check_backward(got, s, s["x"], kind, o, post, nxt, dout)


@pytest.mark.parametrize("T,H,dtype", SIZES + [(4096, 1024, "bf16"),
                                               (700, 4104, "bf16")])
@pytest.mark.parametrize("res", [False, True])
def test_norm_backward(T, H, dtype, res):
    s = tensors(T, H, dtype, "none", seed=6)
    c, o = config(T, H, dtype), moe.make_block_norm(1e-6, 1.0, 3.0)
    r = torch.from_numpy(ref.rstd(f64(s["x"]), o.eps)).float().cuda()
    dx, dw = torch.empty_like(s["x"]), torch.full((H,), 3.0, device="cuda")
    ws = moe.layer_workspace(c, moe.MOE_WS_BLOCK_BACKWARD)
    for accumulate in (False, True):
        moe.moe_norm_backward(c, o, s["x"], s["w_next"], r, s["dh"],
                              s["dout"] if res else None, dx, dw, accumulate,
                              ws)
    want, dwant, mag, dmag = ref.norm_backward(f64(s["x"]), f64(s["w_next"]),
                                               f64(s["dh"]), o.eps, 1.0)
    if res:
        want, mag = want + f64(s["dout"]), mag + np.abs(f64(s["dout"]))
    close(dx, want, mag, "dx")
    close(dw, 2 * dwant, 2 * dmag, "dw")    # overwritten, then added to


def test_backward_accumulates_and_repeats():
    s = tensors(401, 1000, "bf16", "channel", seed=8)
    c = config(401, 1000, "bf16")
    o = moe.make_block_norm(1e-6, 0.0, 1.0, moe.MOE_GATE_CHANNEL)
    one = backward(c, o, s, s["x"], "channel")
    two = backward(c, o, s, s["x"], "channel")
    for n in one:                           # no order that changes
        assert torch.equal(one[n], two[n]), n
    names = ("dw_post", "dgate", "dw_next")
    sums = {n: one[n].clone() for n in names}
    backward(c, o, s, s["x"], "channel", accumulate=True, sums=sums)
    for n in names:
        assert torch.equal(sums[n], one[n] + one[n]), n


def test_in_place():
    s = tensors(40, 1032, "bf16", "token", seed=10)
    c, o = config(40, 1032, "bf16"), moe.make_block_norm(
        gate=moe.MOE_GATE_TOKEN)
    want = forward(c, o, s, "token")
    x, y = s["x"].clone(), s["y"].clone()
    moe.moe_block_out(c, o, x, y, s["w_post"], s["gate"], s["w_next"], x, y)
    assert torch.equal(x, want["out"]) and torch.equal(y, want["h"])
    grads = backward(c, o, s, s["x"], "token")
    ws = moe.layer_workspace(c, moe.MOE_WS_BLOCK_BACKWARD)
    r = [torch.from_numpy(ref.rstd(f64(s[n]), o.eps)).float().cuda()
         for n in ("y", "x")]
    d, y = s["dout"].clone(), s["y"].clone()
    dw = [torch.empty(1032, device="cuda") for _ in range(2)]
    dg = torch.empty(40, device="cuda")
    moe.moe_block_out_backward(c, o, y, s["w_post"], s["gate"], r[0], s["x"],
                               s["w_next"], r[1], d, s["dh"], d, y, dw[0],
                               dg, dw[1], False, ws)
    assert torch.equal(d, grads["dx"]) and torch.equal(y, grads["dy"])


def test_zero_rows_and_no_rows():
    s = tensors(6, 264, "bf16", "channel", seed=11)
    s["y"][2] = 0
    s["x"][2] = 0
    c, o = config(6, 264, "bf16"), moe.make_block_norm(
        1e-6, gate=moe.MOE_GATE_CHANNEL)
    got = forward(c, o, s, "channel")
    check_forward(got, s, f64(s["y"]), "channel", o)
    assert (got["out"][2] == 0).all() and (got["h"][2] == 0).all()
    assert abs(got["rstd_y"][2].item() - 1e3) < 1e-2
    grads = backward(c, o, s, s["x"], "channel")
    check_backward(grads, s, s["x"], "channel", o)
    # no tokens: nothing but the column gradients, which are zero
    c0 = config(0, 264, "bf16")
    e = torch.empty((0, 264), dtype=torch.bfloat16, device="cuda")
    moe.moe_block_out(c0, o, e, e, s["w_post"], s["gate"], s["w_next"], e, e)
    sums = [torch.full((264,), 5.0, device="cuda") for _ in range(3)]
    ws = moe.layer_workspace(c0, moe.MOE_WS_BLOCK_BACKWARD)
    moe.moe_block_out_backward(c0, o, e, s["w_post"], s["gate"], None, e,
                               s["w_next"], None, None, None, e, e, sums[0],
                               sums[1], sums[2], False, ws)
    assert all((v == 0).all() for v in sums)


def test_nonfinite_rows_stay_in_their_row():
    s = tensors(7, 1032, "bf16", "none", seed=12)
    c, o = config(7, 1032, "bf16"), moe.make_block_norm()
    clean = forward(c, o, s, "none")
    s["y"][3, 5] = float("nan")
    s["x"][5, 9] = float("inf")
    got = forward(c, o, s, "none")
    for t in (0, 1, 2, 4, 6):
        assert torch.equal(got["out"][t], clean["out"][t])
        assert torch.equal(got["h"][t], clean["h"][t])
    assert got["out"][3].isnan().all()
    assert got["out"][5, 9].isinf() and got["h"][5].isfinite().sum() >= 1031


def test_columns_off_16_bytes_and_other_stream():
    """Column weights need only their natural alignment; a call runs on the
    stream it is given."""
    s = tensors(21, 1032, "bf16", "channel", seed=13)
    c, o = config(21, 1032, "bf16"), moe.make_block_norm(
        gate=moe.MOE_GATE_CHANNEL)
    want, back = forward(c, o, s, "channel"), None
    back = backward(c, o, s, s["x"], "channel")
    for n in ("w_post", "w_next", "gate"):
        s[n] = torch.cat([s[n].new_zeros(1), s[n]])[1:]
        assert s[n].data_ptr() % 16
    got = forward(c, o, s, "channel")
    again = backward(c, o, s, s["x"], "channel")
    for n in want:
        assert torch.equal(got[n], want[n]), n
    for n in back:
        assert torch.equal(again[n], back[n]), n
    side = torch.cuda.Stream()
    out, h = torch.zeros_like(s["x"]), torch.zeros_like(s["x"])
    side.wait_stream(torch.cuda.current_stream())
    moe.moe_block_out(c, o, s["x"], s["y"], s["w_post"], s["gate"],
                      s["w_next"], out, h, stream=side)
    side.synchronize()
    assert torch.equal(out, want["out"]) and torch.equal(h, want["h"])


@pytest.mark.parametrize("H,dtype", [(8, "bf16"), (264, "bf16"),
                                     (2048, "bf16"), (4104, "bf16"),
                                     (16392, "bf16"), (1024, "f32")])
@pytest.mark.parametrize("accumulate", [False, True])
def test_norm_backward_without_rows(H, dtype, accumulate):
    """No tokens: the row tensors are empty (their address is null) and the
    column gradient is zero, or stays as it was."""
    c, o = config(0, H, dtype), moe.make_block_norm()
    e = torch.empty((0, H), dtype=DT[dtype], device="cuda")
    r = torch.empty(0, device="cuda")
    dw = torch.arange(H, dtype=torch.float32, device="cuda")
    want = dw.clone() if accumulate else torch.zeros_like(dw)
    ws = moe.layer_workspace(c, moe.MOE_WS_BLOCK_BACKWARD)
    ws.fill_(0xAB)
    w = torch.ones(H, device="cuda")
    moe.moe_norm_backward(c, o, e, w, r, e, None, e, dw, accumulate, ws)
    assert torch.equal(dw, want)
    moe.moe_norm_backward(c, o, e, w, r, e, e, e, dw, accumulate, ws)
    assert torch.equal(dw, want)


# Rows too wide for the streamed kernels, and enough of them that every CTA
# (at most 304) has two or three: float32 rows of 7168, bf16 rows of 16392 columns.
WIDE = [(700, 7168, "f32"), (610, 16392, "bf16")]


@pytest.mark.parametrize("T,H,dtype", WIDE)
@pytest.mark.parametrize("res", [False, True])
def test_norm_backward_wide_rows(T, H, dtype, res):
    """One row sum a row: each follows the last without another between."""
    test_norm_backward(T, H, dtype, res)


@pytest.mark.parametrize("T,H,dtype", WIDE)
@pytest.mark.parametrize("kind,post,nxt", [
    ("none", True, True), ("channel", False, True), ("full", True, False),
    ("token", False, False), ("token", True, True)])
def test_block_out_backward_wide_rows(T, H, dtype, kind, post, nxt):
    s = tensors(T, H, dtype, kind, seed=14)
    o = moe.make_block_norm(1e-5, 1.0, 0.9, GATES.index(kind))
    got = backward(config(T, H, dtype), o, s, s["x"], kind, post, nxt)
    check_backward(got, s, s["x"], kind, o, post, nxt)
    again = backward(config(T, H, dtype), o, s, s["x"], kind, post, nxt)
    for n in got:
        assert got[n] is None or torch.equal(got[n], again[n]), n


# Rows enough that each CTA of the persistent kernels takes several: its queue
# then runs across rows, the row sums' buffers alternate, a token's gate is
# loaded a row ahead, and the combine's ring of rows (13 rows, or 4 of 32
# experts) comes round.
@pytest.mark.parametrize("T,H,dtype,kind,post,nxt", [
    (2500, 4104, "bf16", "none", True, True),
    (2500, 4104, "bf16", "token", True, True),
    (2500, 4104, "bf16", "full", True, True),
    (2500, 7168, "bf16", "channel", True, True),
    (6000, 1032, "bf16", "token", True, True),
    (6001, 1032, "bf16", "full", False, True),
    (2500, 4104, "bf16", "token", False, True),
    (2500, 4104, "bf16", "channel", True, False),
    (2500, 4104, "bf16", "full", False, False),
    (2500, 5120, "f32", "token", True, True)])
def test_block_out_many_rows(T, H, dtype, kind, post, nxt):
    s = tensors(T, H, dtype, kind, seed=15)
    o = moe.make_block_norm(1e-5, 1.0, 0.9, GATES.index(kind))
    got = forward(config(T, H, dtype), o, s, kind, post, nxt)
    check_forward(got, s, f64(s["y"]), kind, o, post, nxt)


@pytest.mark.parametrize("T,H,dtype", [(6000, 1032, "bf16"),
                                       (2500, 7168, "bf16"),
                                       (2500, 5120, "f32")])
def test_norm_many_rows(T, H, dtype):
    test_norm(T, H, dtype)


@pytest.mark.parametrize("T,H,k,dtype,kind,post,nxt", [
    (6000, 1032, 1, "bf16", "token", True, True),
    (2500, 4104, 2, "bf16", "full", True, True),
    (2500, 7168, 8, "bf16", "channel", True, True),
    (2500, 4104, 32, "bf16", "full", True, True),
    (2500, 4104, 32, "bf16", "token", False, True),
    (2500, 7168, 1, "bf16", "none", True, False),
    (2500, 7168, 1, "bf16", "token", False, False),
    (2500, 4104, 2, "bf16", "full", False, False),
    (2500, 5120, 3, "f32", "channel", True, True)])
def test_combine_block_out_many_rows(T, H, k, dtype, kind, post, nxt):
    s = tensors(T, H, dtype, kind, seed=16)
    g = torch.Generator(device="cuda").manual_seed(17)
    on = dict(generator=g, device="cuda")
    ys = torch.randn(T * k, H, **on).to(DT[dtype])
    row_of = torch.randperm(T * k, **on).int().reshape(T, k)
    lost = torch.rand(T, k, **on) < 0.2
    lost[T // 3] = lost[T - 1] = True       # tokens that lost every row
    ys[row_of[lost].long()] = float("nan")  # and rows that are not read
    row_of[lost] = -1
    w = torch.rand(T, k, **on)
    c = config(T, H, dtype, k)
    o = moe.make_block_norm(1e-5, 1.0, 0.9, GATES.index(kind))
    got = forward(c, o, s, kind, post, nxt, combine=(ys, row_of, w))
    y = torch.empty_like(s["y"])
    moe.moe_combine(c, ys, row_of, w, y)
    assert torch.equal(got["y"], y)
    check_forward(got, s, f64(y), kind, o, post, nxt)
