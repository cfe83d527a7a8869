"""4-bit expert weights on the GPU against the float64 oracle.

Tolerances.  Packing and expanding move whole numbers: expanded values equal
(code - zero) * scale rounded once, bit for bit.  A product's float32 sum over
K terms is within (K/256 + 64) serial roundings of 2^-24 (256-row steps, then
a short tree and the warps), doubled for the matrix instruction's truncation:
REL = 2e-5 of the sum of absolute terms covers K <= 8192.  silu is within a
few roundings of its argument's error times 1.1 (its largest slope).  y is
checked from the h that the kernel stored.  A value stored in bf16 lies
between the two rounded ends of its float32 interval.
"""
import numpy as np
import pytest
import torch

import mixture_experts_token_gb300 as moe
from oracle import w4_ref as ref
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

REL = 2e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def close(got, want, tol, what):
    lo, hi = (f64(torch.from_numpy(v).float().to(got.dtype))
              for v in (want - tol, want + tol))
    v = f64(got)
    bad = ~((lo <= v) & (v <= hi))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4],
                           float(np.nanmax(np.abs(v - want) / tol)))


def matrix(n, K, N, group, zeros, seed, scale=0.02):
    """Codes, scales and zeros on the device, and the packed buffer."""
    g = torch.Generator().manual_seed(seed)
    G = -(-K // group)
    codes = torch.randint(0, 256, (n, K // 2, N), generator=g,
                          dtype=torch.uint8).cuda()
    scales = ((torch.rand(n, G, N, generator=g) + 0.5) * scale).bfloat16()
    zp = torch.randint(0, 16, (n, G, N), generator=g,
                       dtype=torch.uint8).cuda() if zeros else None
    w4 = moe.make_w4(group, zeros)
    packed = moe.alloc_w4(w4, n, K, N)
    packed.fill_(0xCD)
    moe.moe_w4_pack(w4, n, K, N, codes, scales.cuda(), zp, packed)
    w = ref.dequantize(codes.cpu().numpy(), f64(scales),
                       None if zp is None else zp.cpu().numpy(), group)
    return packed, w


@pytest.mark.parametrize("n,K,N", [(1, 2, 1), (2, 64, 16), (3, 66, 17),
                                   (2, 256, 48), (1, 330, 40), (2, 1024, 31),
                                   (1, 8, 300)])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_pack_and_expand(n, K, N, group, zeros):
    packed, w = matrix(n, K, N, group, zeros, seed=K + N)
    w4 = moe.make_w4(group, zeros)
    for dt in (torch.float32, torch.bfloat16):
        out = torch.empty((n, K, N), dtype=dt, device="cuda")
        moe.moe_w4_dequantize(w4, n, K, N, packed, out)
        assert torch.equal(out.cpu(), torch.from_numpy(w).float().to(dt))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128])
@pytest.mark.parametrize("zeros", [False, True])
def test_quantize(dtype, group, zeros):
    n, K, N = 3, 330, 37
    g = torch.Generator().manual_seed(group)
    w = (torch.randn(n, K, N, generator=g) * 0.02).to(DT[dtype])
    w[0, :, 3] = 0                        # groups of zeros
    w[1, :, 5] = w[1, :, 5].abs()         # one-sided
    w[2, 0:32, 7] = 0.25                  # constant
    G = -(-K // group)
    w4 = moe.make_w4(group, zeros)
    codes = torch.empty((n, K // 2, N), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, G, N), dtype=torch.bfloat16, device="cuda")
    zp = torch.empty((n, G, N), dtype=torch.uint8,
                     device="cuda") if zeros else None
    moe.moe_w4_quantize(w4, n, K, N, w.cuda(), codes, scales, zp)
    q = ref.unpack(codes.cpu().numpy())
    s, w64 = f64(scales), w.double().numpy()
    z = None if zp is None else zp.cpu().numpy()
    for i in range(G):
        rows = slice(i * group, (i + 1) * group)
        v = w64[:, rows]
        lo, hi = np.minimum(v.min(1), 0), np.maximum(v.max(1), 0)
        span = (hi - lo) / 15 if zeros else np.maximum(-lo, hi) / 7
        # rounded to bf16: within half a step of its 8 bits
        assert np.all(np.abs(s[:, i] - span) <= 2.0 ** -8 * span * 1.0001)
        zero = z[:, i:i + 1] if zeros else 8.0
        step = s[:, i:i + 1]
        back = (q[:, rows] - zero) * step
        # nearest under the rounded scale, except where the range's rounded
        # ends clip: a scale 2^-8 too small leaves 15 * 2^-8 of a step more,
        # and with zero points the zero's own rounding another half
        extra = (0.5 if zeros else 0.0) + 15 * 2.0 ** -8
        assert np.all(np.abs(back - v) <= step * (0.5 + extra) + 1e-12)
        inner = (q[:, rows] > 0) & (q[:, rows] < 15)
        assert np.all((np.abs(back - v) <= step * 0.5001 + 1e-12)[inner])
    assert (s[0, :, 3] == 0).all()
    expect = 8 if not zeros else 0
    assert (q[0, :, 3] == expect).all()


def run_swiglu(cfg, w4, x, off, packs, groups=None, status=None):
    R = cfg.T * cfg.k
    h = torch.full((R, cfg.F), 7.0, device="cuda").to(x.dtype)
    y = torch.full((R, cfg.H), 7.0, device="cuda").to(x.dtype)
    if groups is None:
        moe.moe_gmm_swiglu_w4(cfg, w4, x, off, *packs, h, y, status)
    else:
        kw = dict(n_groups=len(groups),
                  group_expert=torch.tensor(groups, dtype=torch.int32).cuda())
        moe.moe_gmm_gate_up_w4(cfg, w4, x, off, packs[0], packs[1], h, status,
                               **kw)
        moe.moe_gmm_down_w4(cfg, w4, h, off, packs[2], y, status, **kw)
    torch.cuda.synchronize()
    return h, y


def check_swiglu(x, offsets, experts, ws, h, y):
    x64, h64 = f64(x), f64(h)
    wg, wu, wd = ws
    for i, e in enumerate(experts):
        a, z = offsets[i], offsets[i + 1]
        if a == z:
            continue
        r = x64[a:z]
        g, u = r @ wg[e], r @ wu[e]
        eg, eu = (REL * (np.abs(r) @ np.abs(w[e])) for w in (wg, wu))
        s = ref.silu(g)
        tol = (1.1 * eg + 4 * 2.0 ** -23 * np.abs(s)) * (np.abs(u) + eu) \
            + np.abs(s) * eu + 1e-30
        close(h[a:z], s * u, tol, ("h", i))
        m = np.abs(h64[a:z]) @ np.abs(wd[e])
        close(y[a:z], h64[a:z] @ wd[e], REL * m + 1e-30, ("y", i))


def case(counts, H, F, E, dtype, group, zeros, seed=0, k=1, scale=0.02):
    """Rows sorted into groups of the given counts."""
    off = np.concatenate([[0], np.cumsum(counts)]).tolist()
    T = max(1, -(-off[-1] // k))
    cfg = moe.make_config(T, H, E, k, F, 1, dtype=dtype)
    g = torch.Generator().manual_seed(seed + 100)
    x = torch.randn(T * k, H, generator=g).to(DT[dtype]).cuda()
    mats = [matrix(E, K, N, group, zeros, seed + i, scale)
            for i, (K, N) in enumerate(((H, F), (H, F), (F, H)))]
    return (cfg, moe.make_w4(group, zeros), x, off,
            torch.tensor(off, dtype=torch.int32).cuda(),
            [p for p, _ in mats], [w for _, w in mats])


# rows of a group around the kernels' row blocks; sizes that end inside a
# tile of 64 or 256 rows, inside 16 and 128 columns, and inside a group
@pytest.mark.parametrize("counts,H,F,dtype", [
    ([1], 64, 64, "bf16"), ([1], 8, 8, "bf16"), ([1], 4, 4, "f32"),
    ([0, 3, 0, 8, 9], 72, 40, "bf16"), ([7, 0, 16, 17], 264, 136, "bf16"),
    ([1, 1, 0, 1, 0], 1000, 328, "bf16"), ([33, 5], 520, 264, "bf16"),
    ([64, 65], 256, 512, "bf16"), ([130, 1], 128, 200, "bf16"),
    ([2, 0, 0, 1], 2048, 1024, "bf16"), ([3], 4104, 72, "bf16"),
    ([12, 31, 0, 2], 136, 1416, "bf16"), ([300], 320, 64, "bf16"),
    ([5, 0, 9], 68, 36, "f32"), ([17, 2], 516, 260, "f32"),
    ([40, 0, 1], 1412, 132, "f32"), ([1], 2048, 516, "f32"),
    ([100], 64, 100, "f32")])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False),
                                         (128, True), (128, False)])
def test_swiglu(counts, H, F, dtype, group, zeros):
    cfg, w4, x, off, doff, packs, ws = case(counts, H, F, len(counts), dtype,
                                            group, zeros)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, y = run_swiglu(cfg, w4, x, doff, packs, status=status)
    assert status.item() == 0
    check_swiglu(x, off, range(len(counts)), ws, h, y)


# groups of many rows: one pass of 48 rows, parts of one, and several; one
# tile of k, odd numbers of tiles, ends inside a tile; columns that end inside
# a record, a quarter and a tile
@pytest.mark.parametrize("counts,H,F", [
    ([16], 8, 8), ([17, 0, 15], 72, 40), ([48], 64, 136), ([49, 97], 200, 328),
    ([33, 5], 1000, 264), ([60, 0, 60, 13], 264, 1416), ([250], 2056, 520),
    ([13, 14, 40, 7, 31], 520, 2056), ([1] * 8 + [300], 264, 136),
    # enough items for the tensor cores' form: columns and row passes
    ([1000, 0, 21], 8, 5000), ([48 * 40], 72, 2312), ([30] * 40, 328, 1032),
    ([25] * 60 + [0, 96], 200, 520), ([700, 701], 1000, 1504)])
@pytest.mark.parametrize("group,zeros", [(32, False), (32, True), (64, True),
                                         (64, False), (128, True),
                                         (128, False)])
def test_swiglu_many_rows(counts, H, F, group, zeros):
    cfg, w4, x, off, doff, packs, ws = case(counts, H, F, len(counts), "bf16",
                                            group, zeros, seed=11)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    h, y = run_swiglu(cfg, w4, x, doff, packs, status=status)
    assert status.item() == 0
    check_swiglu(x, off, range(len(counts)), ws, h, y)


def test_many_rows_next_to_nonfinite_rows():
    """A pass may read rows of the next group; they stay apart."""
    cfg, w4, x, off, doff, packs, ws = case([620, 700], 264, 1416, 2, "bf16",
                                            64, True, seed=12)
    h0, y0 = run_swiglu(cfg, w4, x, doff, packs)
    x = x.clone()
    x[620:] = float("nan")
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    assert torch.equal(h[:620], h0[:620]) and torch.equal(y[:620], y0[:620])
    assert h[620:].isnan().all() and y[620:].isnan().all()


def test_stalled_rows_time_out_and_context_survives():
    """The bounded waits of the many-row products: with the copies of x
    stopped, the kernel reports MOE_DEV_TIMEOUT and returns, and the next
    call is right."""
    cfg, w4, x, off, doff, packs, ws = case([600, 700], 520, 1416, 2, "bf16",
                                            64, False, seed=13)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    try:
        moe.moe_test_stall_gemm_producer(3)
        run_swiglu(cfg, w4, x, doff, packs, status=status)
    finally:
        moe.moe_test_stall_gemm_producer(-1)
    assert status.item() & moe.MOE_DEV_TIMEOUT
    status.zero_()
    h, y = run_swiglu(cfg, w4, x, doff, packs, status=status)
    assert status.item() == 0
    check_swiglu(x, off, range(2), ws, h, y)


def test_many_experts_one_token():
    """One token of a layer with many experts: few of the groups have a row,
    wherever they lie."""
    E, k, H, F = 200, 6, 136, 72
    counts = np.zeros(E, dtype=int)
    counts[[0, 63, 64, 127, 198, 199]] = 1
    cfg, w4, x, off, doff, packs, ws = case(counts, H, F, E, "bf16", 64, False,
                                            k=k)
    assert cfg.T == 1
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    check_swiglu(x, off, range(E), ws, h, y)


def test_rows_past_the_end_and_empty_call():
    """Rows past group_offsets[E] (a capped pass) are left alone; no rows at
    all write nothing."""
    cfg, w4, x, off, doff, packs, ws = case([3, 0, 4], 264, 136, 3, "bf16", 64,
                                            True)
    cfg = cfg.with_(T=20)
    x = torch.cat([x, torch.full((13, 264), float("nan")).bfloat16().cuda()])
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    check_swiglu(x, off, range(3), ws, h, y)
    assert (h[7:] == 7).all() and (y[7:] == 7).all()
    h, y = run_swiglu(cfg, w4, x, torch.zeros_like(doff), packs)
    assert (h == 7).all() and (y == 7).all()
    c0 = cfg.with_(T=0)
    moe.moe_gmm_swiglu_w4(c0, w4, x[:0], doff, *packs, x[:0], x[:0])


def test_duplicate_groups_and_bad_index():
    cfg, w4, x, off, doff, packs, ws = case([3, 0, 4, 9], 136, 264, 2, "bf16",
                                            128, False)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    # two groups share expert 1; an unused slot has no rows
    h, y = run_swiglu(cfg, w4, x, doff, packs, [1, -1, 0, 1], status)
    assert status.item() == 0
    check_swiglu(x, off, [1, 0, 0, 1], ws, h, y)
    h, y = run_swiglu(cfg, w4, x, doff, packs, [1, 0, 2, 0], status)
    assert status.item() == moe.MOE_DEV_BAD_INDEX
    assert (h[3:7] == 7).all() and (y[3:7] == 7).all()
    check_swiglu(x, [0, 3, 3, 3], [1, 0, 0], ws, h[:3], y[:3])


def test_nonfinite_rows_stay_in_their_row():
    args = case([9, 20], 264, 136, 2, "bf16", 64, True, seed=3)
    cfg, w4, x, off, doff, packs, ws = args
    h0, y0 = run_swiglu(cfg, w4, x, doff, packs)
    x = x.clone()
    x[4, 17] = float("nan")
    x[15, 200] = float("inf")
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    keep = [r for r in range(29) if r not in (4, 15)]
    assert torch.equal(h[keep], h0[keep]) and torch.equal(y[keep], y0[keep])
    assert h[4].isnan().all() and y[4].isnan().all()
    assert not y[15].isfinite().any()


def test_silu_at_large_arguments():
    """Products far outside exp's range: silu goes to 0 or to its argument."""
    args = case([5, 3], 72, 40, 2, "bf16", 64, False, seed=5, scale=8.0)
    cfg, w4, x, off, doff, packs, ws = args
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    check_swiglu(x, off, range(2), ws, h, y)


def test_repeats_bit_for_bit():
    """Nothing depends on timing."""
    args = case([70], 520, 264, 1, "bf16", 64, True, seed=7)
    cfg, w4, x, off, doff, packs, ws = args
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    h2, y2 = run_swiglu(cfg, w4, x, doff, packs)
    assert torch.equal(h, h2) and torch.equal(y, y2)


def test_other_stream():
    args = case([4, 9], 136, 72, 2, "bf16", 32, True, seed=8)
    cfg, w4, x, off, doff, packs, ws = args
    want = run_swiglu(cfg, w4, x, doff, packs)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    h, y = (torch.zeros_like(t) for t in want)
    moe.moe_gmm_swiglu_w4(cfg, w4, x, doff, *packs, h, y, stream=side)
    side.synchronize()
    assert torch.equal(h, want[0]) and torch.equal(y, want[1])


def test_offsets_past_32_bits():
    """The last expert's weights lie past 2^32 bytes of the packed buffer."""
    E, H, F, w4 = 600, 4096, 4096, moe.make_w4(128)
    per = moe.moe_w4_bytes(w4, 1, H, F)
    assert (E - 1) * per > 1 << 32
    packs = [torch.zeros(E * per, dtype=torch.uint8, device="cuda")
             for _ in range(3)]
    one = [matrix(1, H, F, 128, False, 20 + i) for i in range(3)]
    for p, (q, _) in zip(packs, one):
        p[(E - 1) * per:] = q
    cfg = moe.make_config(2, H, E, 1, F, 1)
    off = [0] * E + [2]
    x = torch.randn(2, H, generator=torch.Generator().manual_seed(1))
    x = x.bfloat16().cuda()
    h, y = run_swiglu(cfg, w4, x, torch.tensor(off, dtype=torch.int32).cuda(),
                      packs)
    check_swiglu(x, [0, 2], [0], [w for _, w in one], h, y)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_codes_scales_and_zeros_at_any_element(dtype):
    """One matrix of several, and views whose addresses end in an odd byte
    (codes, zeros) or half a word (scales): the bits of aligned copies."""
    n, K, N, group = 1, 66, 17, 64
    w = torch.randn(n, K, N, generator=torch.Generator().manual_seed(3))
    w, w4, G = w.to(DT[dtype]).cuda(), moe.make_w4(group, True), 2

    def run(skip):
        def view(rows, dt):
            t = torch.zeros(n * rows * N + skip, dtype=dt, device="cuda")
            return t[skip:]
        codes, zp = view(K // 2, torch.uint8), view(G, torch.uint8)
        scales = view(G, torch.bfloat16)
        assert codes.data_ptr() % 4 == skip
        assert scales.data_ptr() % 4 == 2 * skip
        moe.moe_w4_quantize(w4, n, K, N, w, codes, scales, zp)
        packed = moe.alloc_w4(w4, n, K, N)
        moe.moe_w4_pack(w4, n, K, N, codes, scales, zp, packed)
        return codes, scales, zp, packed
    for a, b in zip(run(0), run(1)):
        assert torch.equal(a, b)


# each form of the kernel: k over four warps; 8 and 16 rows a pass
@pytest.mark.parametrize("counts,H,F", [([30, 3, 16], 520, 260),
                                        ([4] * 40, 512, 2056),
                                        ([64] * 8, 520, 2056)])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False),
                                         (128, True)])
def test_float32_products_lean_neither_way(counts, H, F, group, zeros):
    """Rounding to nearest errs to both sides alike; a sum that is truncated
    once errs by half a unit in its last place towards zero on average, that
    is 2^-24 of it.  The mean of the signed errors of the 10^4 and more outputs
    has to be below that (their own scatter leaves about 1e-9 of it)."""
    cfg, w4, x, off, doff, packs, ws = case(counts, H, F, len(counts), "f32",
                                            group, zeros, seed=21)
    h, y = run_swiglu(cfg, w4, x, doff, packs)
    x64, h64 = f64(x), f64(h)
    wh, wy = np.empty_like(h64), np.empty((off[-1], H))
    for e in range(len(counts)):
        r = slice(off[e], off[e + 1])
        wh[r] = ref.silu(x64[r] @ ws[0][e]) * (x64[r] @ ws[1][e])
        wy[r] = h64[r] @ ws[2][e]
    for got, want, what in ((h64, wh, "h"), (f64(y), wy, "y")):
        lean = ((got - want) * np.sign(want)).mean() / np.abs(want).mean()
        assert abs(lean) < 2.0 ** -24, (what, lean)
