"""Microscaled 4-bit experts on the GPU against the float64 oracle.

Tolerances.  Codes, scales, layouts and their values are exact: bit for bit.
A product of two codes and two scales is exact in float32; the sum over K adds
K/64 of the instructions' sums one after another, each addition truncated to 24
bits at worst, 2^-23 of it: (K/64 + 32) 2^-23 <= 2e-5 = REL of the sum of
absolute terms for K <= 8192.  silu is within a few roundings and 2^-22 of its
exponential of its argument's error times 1.1 (its largest slope).  h is
quantised from its float32 value, so what was stored lies within half a step of
codes of that; its scale is the oracle's for a largest magnitude within the
same error.  y is checked from the h that the kernel stored.  A value stored in
bf16 lies between the two rounded ends of its float32 interval.
"""
import numpy as np
import pytest
import torch

import mixture_experts_token_gb300 as moe
from oracle import mx_ref as ref
from tests.gpu_util import f64

pytestmark = pytest.mark.gpu

REL = 2e-5
DT = {"f32": torch.float32, "bf16": torch.bfloat16}


def np8(t):
    return t.cpu().numpy()


def make(block, x_scale=0.011, h_scale=0.013):
    return moe.make_mx(block, *((x_scale, h_scale) if block == 16 else
                                (1.0, 1.0)))


def by_row(scales):
    """Scales [steps, R, 256/block] of rows as [R, ..] in their order."""
    s = np8(scales).transpose(1, 0, 2)
    return s.reshape(s.shape[0], -1)


def hard_rows(R, K, dtype, seed, unit=1.0):
    """Rows of unlike sizes, with ties (multiples of a quarter of a power of
    two), zeros, extremes and blocks of one value."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(R, K, generator=g) * (torch.randn(R, K, generator=g)
                                          * 1.5).exp()
    x[::3] = torch.randint(-24, 25, (len(x[::3]), K), generator=g) / 4
    x[1::5, ::2] = 0.0
    x[2::7, :K // 2] = 0.0
    x[2::7, 0] = -0.0
    x = x * unit
    if R > 8:
        x[4] = torch.finfo(torch.float32).tiny * torch.randn(K, generator=g)
        x[5] = 1e-41 * torch.randn(K, generator=g)
        x[6] = 3e38 * (torch.rand(K, generator=g) - 0.5)
        x[7, 3] = float("nan")
        x[8, K - 1] = float("-inf")
    return x.to(dtype)


@pytest.mark.parametrize("R,K", [(1, 32), (3, 64), (9, 96), (40, 160),
                                 (33, 544), (12, 7168)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.011])
def test_rows_bit_for_bit(R, K, block, dtype, scale):
    scale = scale if block == 16 else 1.0
    mx = make(block)
    x = hard_rows(R, K, DT[dtype], R + K, scale)
    codes, scales = moe.alloc_mx_rows(mx, R, K)
    assert scales.numel() == moe.moe_mx_row_scale_bytes(mx, R, K)
    scales.fill_(0xAB)
    moe.moe_mx_quantize_rows(mx, R, K, x.cuda(), scale, codes, scales)
    want, ws = ref.quantize_rows(x.float().numpy(), block, scale)
    got = by_row(scales)
    assert np.array_equal(got[:, :K // block], ws[:, :K // block])
    assert not got[:, K // block:].any()
    nan = 255 if block == 32 else 127
    fine = np.repeat(ws[:, :K // block] != nan, block // 2, 1)
    assert np.array_equal(np8(codes)[fine], want[fine])
    for out in (torch.float32, torch.bfloat16):
        v = torch.empty((R, K), dtype=out, device="cuda")
        moe.moe_mx_dequantize_rows(mx, R, K, codes, scales, scale, v)
        # the last product is rounded to float32
        w = torch.from_numpy(ref.dequantize_rows(want, ws, block, scale)
                             .astype(np.float32)).to(out)
        got = v.cpu()
        assert torch.equal(got.isnan(), w.isnan())
        assert torch.equal(got.nan_to_num(), w.nan_to_num())


def matrices(n, K, N, block, dtype="f32", seed=0, std=0.02):
    """Quantised weights: (packed, tensor scales, float64 values)."""
    g = torch.Generator().manual_seed(seed)
    mx = make(block)
    w = (torch.randn(n, K, N, generator=g) * std).to(DT[dtype])
    scale = None
    if block == 16:
        scale = (w.float().abs().amax((1, 2)) / (448 * 6)).cuda()
    codes, scales = moe.alloc_mx_codes(mx, n, K, N)
    scales.fill_(0xAB)
    moe.moe_mx_quantize(mx, n, K, N, w.cuda(), scale, codes, scales)
    packed = moe.alloc_mx(mx, n, K, N)
    packed.fill_(0xCD)
    moe.moe_mx_pack(mx, n, K, N, codes, scales, packed)
    values = np.empty((n, K, N))
    for e in range(n):
        t = 1.0 if scale is None else float(scale[e])
        values[e] = ref.dequantize_rows(np8(codes[e]), np8(scales[e]), block,
                                        t).T
    return packed, scale, values, (w, codes, scales)


@pytest.mark.parametrize("n,K,N", [(1, 32, 1), (2, 64, 128), (3, 288, 37),
                                   (1, 256, 129), (2, 544, 200)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_weights_bit_for_bit(n, K, N, block, dtype):
    mx = make(block)
    packed, scale, values, (w, codes, scales) = matrices(n, K, N, block,
                                                         dtype, K + N)
    for e in range(n):
        rows = w[e].float().T.contiguous().numpy()
        want, ws = ref.quantize_rows(
            rows, block, 1.0 if scale is None else float(scale[e]))
        assert np.array_equal(np8(scales[e]), ws)
        assert np.array_equal(np8(codes[e]), want)
    for out in (torch.float32, torch.bfloat16):
        v = torch.empty((n, K, N), dtype=out, device="cuda")
        moe.moe_mx_dequantize(mx, n, K, N, packed, scale, v)
        assert torch.equal(v.cpu(), torch.from_numpy(
            values.astype(np.float32)).to(out))


@pytest.mark.parametrize("K,N", [(32, 10), (288, 9), (544, 72), (256, 16)])
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("scale", [1.0, 0.011])
def test_hard_weights_bit_for_bit(K, N, block, dtype, scale):
    """Ties, zeros, extremes, NaN and infinities as columns of a matrix, with
    odd and even numbers of them; a matrix of zeros beside them."""
    scale = scale if block == 16 else 1.0
    mx = make(block)
    rows = hard_rows(N, K, DT[dtype], K + N, scale)
    w = torch.stack([rows.T, torch.zeros(K, N).to(rows.dtype)]).contiguous()
    t = torch.tensor([scale, 1.0]).cuda() if block == 16 else None
    codes, scales = moe.alloc_mx_codes(mx, 2, K, N)
    scales.fill_(0xAB)
    moe.moe_mx_quantize(mx, 2, K, N, w.cuda(), t, codes, scales)
    want, ws = ref.quantize_rows(rows.float().numpy(), block, scale)
    assert np.array_equal(np8(scales[0]), ws)
    nan = 255 if block == 32 else 127
    fine = np.repeat(ws[:, :K // block] != nan, block // 2, 1)
    assert np.array_equal(np8(codes[0])[fine], want[fine])
    zero, zs = ref.quantize_rows(np.zeros((N, K), np.float32), block, 1.0)
    assert np.array_equal(np8(codes[1]), zero)
    assert np.array_equal(np8(scales[1]), zs)
    packed = moe.alloc_mx(mx, 2, K, N)
    moe.moe_mx_pack(mx, 2, K, N, codes, scales, packed)
    for out in (torch.float32, torch.bfloat16):
        v = torch.empty((2, K, N), dtype=out, device="cuda")
        moe.moe_mx_dequantize(mx, 2, K, N, packed, t, v)
        # the last product is rounded to float32
        values = torch.from_numpy(ref.dequantize_rows(want, ws, block, scale)
                                  .astype(np.float32)).to(out).T
        got = v.cpu()
        assert torch.equal(got[0].isnan(), values.isnan())
        assert torch.equal(got[0].nan_to_num(), values.nan_to_num())
        assert (got[1] == 0).all()


@pytest.mark.parametrize("block", [16, 32])
def test_more_matrices_than_a_grid_has(block):
    """5000 small ones: a CTA takes a second matrix."""
    n, K, N = 5000, 32, 2
    g = torch.Generator().manual_seed(32)
    w = torch.randn(n, K, N, generator=g) * 0.02
    mx = make(block)
    codes, scales = moe.alloc_mx_codes(mx, n, K, N)
    moe.moe_mx_quantize(mx, n, K, N, w.cuda(), None, codes, scales)
    want, ws = ref.quantize_rows(w.transpose(1, 2).reshape(n * N, K).numpy(),
                                 block, 1.0)
    assert np.array_equal(np8(codes).reshape(n * N, -1), want)
    assert np.array_equal(np8(scales).reshape(n * N, -1), ws)
    packed = moe.alloc_mx(mx, n, K, N)
    moe.moe_mx_pack(mx, n, K, N, codes, scales, packed)
    v = torch.empty((n, K, N), device="cuda")
    moe.moe_mx_dequantize(mx, n, K, N, packed, None, v)
    values = ref.dequantize_rows(want, ws, block, 1.0).reshape(n, N, K)
    assert torch.equal(v.cpu(), torch.from_numpy(
        values.transpose(0, 2, 1).astype(np.float32)))


def test_weights_of_a_checkpoint():
    """Scales whose padding is not zero are packed as if it were."""
    mx, n, K, N = make(32), 1, 160, 8
    packed, _, values, (w, codes, scales) = matrices(n, K, N, 32)
    again = moe.alloc_mx(mx, n, K, N)
    scales[:, :, 5:] = 255
    moe.moe_mx_pack(mx, n, K, N, codes, scales, again)
    assert torch.equal(again, packed)


# -------------------------------------------------------- the products ---
def close(got, want, tol, what):
    lo, hi = (f64(torch.from_numpy(v).float().to(got.dtype))
              for v in (want - tol, want + tol))
    v = f64(got)
    bad = ~((lo <= v) & (v <= hi))
    assert not bad.any(), (what, int(bad.sum()), np.argwhere(bad)[:4],
                           float(np.nanmax(np.abs(v - want) / tol)))


class Case:
    """Rows sorted into groups of the given counts, and quantised experts."""

    def __init__(self, counts, H, F, dtype, block, E=None, k=1, seed=0,
                 std=0.05):
        self.off = np.concatenate([[0], np.cumsum(counts)]).tolist()
        E = len(counts) if E is None else E
        T = max(1, -(-self.off[-1] // k))
        self.cfg = moe.make_config(T, H, E, k, F, 1, dtype=dtype)
        self.mx, self.block, self.dtype = make(block), block, dtype
        g = torch.Generator().manual_seed(seed + 100)
        self.x = torch.randn(T * k, H, generator=g).to(DT[dtype]).cuda()
        mats = [matrices(E, K, N, block, "f32", seed + i, std)
                for i, (K, N) in enumerate(((H, F), (H, F), (F, H)))]
        self.packs = [m[0] for m in mats]
        self.scales = [m[1] for m in mats]
        self.w = [m[2] for m in mats]
        self.offsets = torch.tensor(self.off, dtype=torch.int32).cuda()
        self.status = torch.zeros(1, dtype=torch.int32, device="cuda")

    def steps(self, groups=None):
        """The calls one by one: (x, h) codes and scales, and y."""
        c, mx, R = self.cfg, self.mx, self.cfg.T * self.cfg.k
        kw = {} if groups is None else dict(
            n_groups=len(groups),
            group_expert=torch.tensor(groups, dtype=torch.int32).cuda())
        xq = moe.alloc_mx_rows(mx, R, c.H)
        hq = moe.alloc_mx_rows(mx, R, c.F)
        for t in hq:
            t.fill_(0x77)
        y = torch.full((R, c.H), 7.0, device="cuda").to(self.x.dtype)
        moe.moe_mx_quantize_rows(mx, R, c.H, self.x, mx.x_scale, *xq)
        moe.moe_gmm_gate_up_mx(c, mx, *xq, self.offsets, *self.packs[:2],
                               *self.scales[:2], *hq, self.status, **kw)
        moe.moe_gmm_down_mx(c, mx, *hq, self.offsets, self.packs[2],
                            self.scales[2], y, self.status, **kw)
        torch.cuda.synchronize()
        return xq, hq, y

    def whole(self, **kw):
        y = torch.full((self.x.shape[0], self.cfg.H), 7.0,
                       device="cuda").to(self.x.dtype)
        ws = moe.mx_workspace(self.cfg, self.mx)
        ws.fill_(0xEE)
        moe.moe_gmm_swiglu_mx(self.cfg, self.mx, self.x, self.offsets,
                              *self.packs, *self.scales, y, self.status, ws,
                              **kw)
        torch.cuda.synchronize()
        return y

    def check(self, xq, hq, y, experts=None, off=None):
        mx, off = self.mx, off or self.off
        hs = by_row(hq[1])
        x = ref.dequantize_rows(np8(xq[0]), by_row(xq[1]), self.block,
                                mx.x_scale)
        h = ref.dequantize_rows(np8(hq[0]), hs, self.block, mx.h_scale)
        wg, wu, wd = self.w
        for i, e in enumerate(experts or range(len(off) - 1)):
            a, z = off[i], off[i + 1]
            if a == z:
                continue
            r = x[a:z]
            g, u = r @ wg[e], r @ wu[e]
            eg, eu = (REL * (np.abs(r) @ np.abs(w[e])) for w in (wg, wu))
            s = ref.silu(g)
            tol = (1.1 * eg + 8 * 2.0 ** -23 * np.abs(s)) \
                * (np.abs(u) + eu) + np.abs(s) * eu + 1e-30
            self.check_h(h[a:z], hs[a:z], s * u, tol)
            m = np.abs(h[a:z]) @ np.abs(wd[e])
            close(y[a:z], h[a:z] @ wd[e], REL * m + 1e-30, ("y", i))

    def check_h(self, got, byte, want, tol):
        b, F = self.block, self.cfg.F
        r = 1.0 if b == 32 else float(np.float32(1) / np.float32(
            self.mx.h_scale))
        # a rounding of the product with the reciprocal
        v = (want * r).reshape(len(want), -1, b)
        t = (tol * r + 2.0 ** -23 * np.abs(want * r)).reshape(v.shape)
        top = np.abs(v).max(-1)
        err = t.max(-1)
        lo, _ = ref.block_scales(np.maximum(top - err, 0)[..., None], b)
        hi, _ = ref.block_scales((top + err)[..., None], b)
        at = byte[:, :F // b].astype(int)
        assert np.all((lo <= at) & (at <= hi)), "scale"
        s = ref.scale_values(byte[:, :F // b], b)[..., None]
        q = np.abs(got.reshape(v.shape)) * (1 if b == 32 else
                                            1 / float(np.float32(
                                                self.mx.h_scale)))
        q = q / np.where(s > 0, s, 1)
        # half the step above and below the value, which magnitudes over 6
        # are cut to first; a scale of 0 leaves what is below half of the
        # smallest one times 6
        half = np.where(q < 1.9, 0.25, np.where(q < 3.9, 0.5, 1.0)) * s
        half = np.where(s == 0, 6 * 2.0 ** -10, half)
        v = np.where(s > 0, np.clip(v, -6 * s, 6 * s), v)
        off = np.abs(got.reshape(v.shape) * (1.0 if b == 32 else 1 / float(
            np.float32(self.mx.h_scale))) - v)
        assert np.all(off <= half + t + 1e-6 * np.abs(v)), \
            (off - half - t).max()


# Rows around the kernels' row blocks (16, 64 and their large ones) and sizes
# that end inside 256 of k, inside 64 of it and inside a tile of 128 columns.
COUNTS = [([1], 32, 32), ([1], 256, 128), ([2], 288, 160),
          ([0, 3, 0, 16, 17], 96, 64), ([7, 0, 15, 1], 544, 288),
          ([1, 1, 0, 1, 0], 1024, 352), ([9, 9], 2080, 64),
          ([33, 5, 64], 320, 256), ([65, 0, 12], 256, 544),
          ([96, 97], 160, 384), ([192, 193, 31], 224, 128),
          ([300], 512, 96), ([16, 32, 48, 80, 112, 127, 128, 129], 64, 288),
          ([1] * 8 + [200], 384, 160), ([1000, 0, 21], 96, 1056)]


@pytest.mark.parametrize("counts,H,F", COUNTS)
@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_products(counts, H, F, block, dtype):
    c = Case(counts, H, F, dtype, block)
    xq, hq, y = c.steps()
    assert c.status.item() == 0
    c.check(xq, hq, y)
    # the three in one call: the same bits
    assert torch.equal(c.whole(), y)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("counts,H,F", [([1] * 40, 512, 1056),
                                        ([20] * 40 + [0, 70], 256, 640),
                                        ([200] * 30, 288, 800),
                                        ([4, 0, 9], 8192, 64)])
def test_products_of_more_items_than_sms(counts, H, F, block):
    c = Case(counts, H, F, "bf16", block, seed=3)
    xq, hq, y = c.steps()
    assert c.status.item() == 0
    c.check(xq, hq, y)
    assert torch.equal(c.whole(), y)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("counts", [
    # chunks of two passes of 64 rows, and of two of a pair's 192
    [30] * 1000 + [5000], [60000, 0, 41000]])
def test_more_rows_than_work_items(block, counts):
    c = Case(counts, 32, 64, "bf16", block, seed=17)
    xq, hq, y = c.steps()
    assert c.status.item() == 0
    c.check(xq, hq, y)
    assert torch.equal(c.whole(), y)


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("counts,H,F", [
    ([384, 385], 512, 128), ([191, 0, 200, 97], 288, 416), ([208], 32, 32),
    ([1000], 4128, 160), ([130] * 40, 256, 1312)])
def test_products_on_pairs(counts, H, F, block):
    """Many rows a group: odd numbers of column tiles, halves of rows that end
    inside a copy, one stage and many."""
    c = Case(counts, H, F, "bf16", block, seed=18)
    xq, hq, y = c.steps()
    assert c.status.item() == 0
    c.check(xq, hq, y)
    assert torch.equal(c.whole(), y)


@pytest.mark.parametrize("block", [16, 32])
def test_many_experts_one_token(block):
    E, k, H, F = 200, 6, 160, 96
    counts = np.zeros(E, dtype=int)
    counts[[0, 63, 64, 127, 198, 199]] = 1
    c = Case(counts, H, F, "bf16", block, k=k)
    assert c.cfg.T == 1
    c.check(*c.steps())


@pytest.mark.parametrize("block", [16, 32])
def test_rows_past_the_end_and_empty_call(block):
    """Rows behind the last group are left alone (a capped pass), whatever
    they hold; no rows at all write nothing."""
    c = Case([3, 0, 4], 288, 160, "bf16", block)
    c.cfg = c.cfg.with_(T=20)
    c.x = torch.cat([c.x, torch.full((13, 288), float("nan")).bfloat16()
                     .cuda()])
    xq, hq, y = c.steps()
    c.check(xq, hq, y)
    assert (y[7:] == 7).all()
    assert (hq[0][7:] == 0x77).all() and (hq[1][:, 7:] == 0x77).all()
    assert torch.equal(c.whole(), y)
    c.offsets = torch.zeros_like(c.offsets)
    assert (c.whole() == 7).all()
    c0 = c.cfg.with_(T=0)
    moe.moe_gmm_swiglu_mx(c0, c.mx, None, None, None, None, None, None, None,
                          None, None, None, None)


@pytest.mark.parametrize("block", [16, 32])
def test_duplicate_groups_and_bad_index(block):
    c = Case([3, 0, 4, 9], 160, 288, "bf16", block, E=2)
    out = c.steps([1, -1, 0, 1])
    assert c.status.item() == 0
    c.check(*out, experts=[1, 0, 0, 1])
    xq, hq, y = c.steps([1, 0, 2, 0])
    assert c.status.item() == moe.MOE_DEV_BAD_INDEX
    assert (hq[0][3:7] == 0x77).all() and (y[3:7] == 7).all()
    c.check(xq, hq, y, experts=[1, 0, 0], off=[0, 3, 3, 3])


@pytest.mark.parametrize("block", [16, 32])
@pytest.mark.parametrize("counts", [[9, 20], [120, 230]])
def test_nonfinite_rows_stay_in_their_row(block, counts):
    c = Case(counts, 288, 160, "bf16", block, seed=4)
    y0 = c.whole()
    c.x = c.x.clone()
    c.x[4, 17] = float("nan")
    c.x[15, 280] = float("inf")
    c.x[-1, 3] = float("nan")
    y = c.whole()
    R = len(y)
    keep = [r for r in range(R) if r not in (4, 15, R - 1)]
    assert torch.equal(y[keep], y0[keep])
    assert y[[4, 15, R - 1]].isnan().all()


@pytest.mark.parametrize("block", [16, 32])
def test_large_and_zero_products(block):
    """silu far outside exp's range, and rows of zeros."""
    c = Case([5, 3], 96, 64, "f32", block, seed=5, std=20.0)
    c.x[1] = 0
    xq, hq, y = c.steps()
    c.check(xq, hq, y)
    assert (y[1] == 0).all()


# powers of two on the scales of x, the gate, up and down matrices and h, with
# values to match: the product of two scales that float32 rounds coarsely or
# not at all, with rows and up's sums that make up for it; that is infinite;
# that is large; h far over its scale's range
@pytest.mark.parametrize("powers", [
    (-70, -50, 100, -20, -90), (50, -50, 50, 60, 100), (60, -60, -60, 110, 0),
    (0, 0, 0, 0, -110), (-100, 100, 100, -30, 0), (100, -100, -100, -40, -100)])
@pytest.mark.parametrize("counts", [[9, 0, 5], [5, 0, 200]])
def test_tensor_scales_near_the_ends_of_float32(counts, powers):
    c = Case(counts, 288, 160, "f32", 16, seed=31)
    two = [2.0 ** p for p in powers]
    c.mx = moe.make_mx(16, 0.011 * two[0], 0.013 * two[4])
    c.x = c.x * two[0]
    c.x[1] = 0
    for i in range(3):
        c.scales[i], c.w[i] = c.scales[i] * two[1 + i], c.w[i] * two[1 + i]
        assert c.scales[i].min() >= 2.0 ** -126
        assert c.scales[i].isfinite().all()
    xq, hq, y = c.steps()
    hs = by_row(hq[1])
    x = ref.dequantize_rows(np8(xq[0]), by_row(xq[1]), 16, c.mx.x_scale)
    h = ref.dequantize_rows(np8(hq[0]), hs, 16, c.mx.h_scale)
    for e in range(len(counts)):
        r = slice(c.off[e], c.off[e + 1])
        if counts[e] == 0:
            continue
        g, u = x[r] @ c.w[0][e], x[r] @ c.w[1][e]
        eg, eu = (REL * (np.abs(x[r]) @ np.abs(w[e])) for w in c.w[:2])
        s = ref.silu(g)
        tol = (1.1 * eg + 8 * 2.0 ** -23 * np.abs(s)) * (np.abs(u) + eu) \
            + np.abs(s) * eu
        c.check_h(h[r], hs[r], s * u, tol)
        close(y[r], h[r] @ c.w[2][e],
              REL * (np.abs(h[r]) @ np.abs(c.w[2][e])), ("y", e))
    assert c.status.item() == 0 and (y[1] == 0).all()
    assert torch.equal(c.whole(), y)


def test_h_beyond_float32_is_nan():
    """A row whose h overflows float32 is NaN, the others are not."""
    c = Case([4], 64, 64, "f32", 32, seed=6, std=1.0)
    c.x[2] *= 1e25
    y = c.whole()
    assert y[2].isnan().all() and y[[0, 1, 3]].isfinite().all()


@pytest.mark.parametrize("block", [16, 32])
def test_repeats_bit_for_bit_on_another_stream_and_in_a_graph(block):
    c = Case([70, 3, 200], 544, 288, "bf16", block, seed=7)
    y = c.whole()
    assert torch.equal(c.whole(), y)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    assert torch.equal(c.whole(stream=side), y)
    ws, out = moe.mx_workspace(c.cfg, c.mx), torch.zeros_like(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.moe_gmm_swiglu_mx(c.cfg, c.mx, c.x, c.offsets, *c.packs,
                              *c.scales, out, c.status, ws)
    x0 = c.x.clone()
    for x in (x0, -x0, x0):
        c.x.copy_(x)
        graph.replay()
        torch.cuda.synchronize()
        got = out.clone()
        assert torch.equal(got, c.whole())
    assert torch.equal(got, y)


def test_calls_that_share_a_workspace_in_order():
    """One workspace, many calls of different sizes without waiting."""
    cases = [Case(n, 256, 128, "bf16", 16, seed=8 + i)
             for i, n in enumerate(([3, 90], [1], [200, 7], [16, 16, 16]))]
    want = [c.whole() for c in cases]
    ws = max((moe.mx_workspace(c.cfg, c.mx) for c in cases),
             key=lambda t: t.numel())
    outs = [torch.zeros_like(y) for y in want]
    for _ in range(20):
        for c, y in zip(cases, outs):
            moe.moe_gmm_swiglu_mx(c.cfg, c.mx, c.x, c.offsets, *c.packs,
                                  *c.scales, y, c.status, ws)
    torch.cuda.synchronize()
    for a, b in zip(outs, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("block", [16, 32])
def test_calls_at_once_on_three_streams(block):
    """Each with a workspace of its own: a few rows, singles, pairs."""
    cases = [Case(n, 512, 256, "bf16", block, seed=20 + i) for i, n in
             enumerate(([1], [30, 0, 50], [300, 290]))]
    want = [c.whole() for c in cases]
    room = [moe.mx_workspace(c.cfg, c.mx) for c in cases]
    outs = [torch.zeros_like(y) for y in want]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for c, ws, y, s in zip(cases, room, outs, streams):
            moe.moe_gmm_swiglu_mx(c.cfg, c.mx, c.x, c.offsets, *c.packs,
                                  *c.scales, y, c.status, ws, stream=s)
    torch.cuda.synchronize()
    for c, a, b in zip(cases, outs, want):
        assert torch.equal(a, b) and c.status.item() == 0


def test_inputs_written_by_the_kernel_before():
    """Rows and offsets that torch writes on the stream just before a call."""
    c = Case([40, 25, 7], 512, 256, "bf16", 16, seed=30)
    offsets = [torch.tensor(o, dtype=torch.int32).cuda()
               for o in ([0, 40, 65, 72], [0, 0, 1, 72], [0, 72, 72, 72])]
    rows = [c.x.clone(), -c.x, c.x.flip(0).contiguous()]
    ws = moe.mx_workspace(c.cfg, c.mx)

    def call(x, o):
        y = torch.zeros_like(x)
        moe.moe_gmm_swiglu_mx(c.cfg, c.mx, x, o, *c.packs, *c.scales, y,
                              c.status, ws)
        return y
    want = []
    for x, o in zip(rows, offsets):
        torch.cuda.synchronize()
        want.append(call(x, o))
    x, o = torch.zeros_like(c.x), torch.zeros_like(offsets[0])
    for _ in range(10):
        for i in range(3):
            x.copy_(rows[i])
            o.copy_(offsets[i])
            assert torch.equal(call(x, o), want[i])


@pytest.mark.parametrize("counts", [[60, 70], [300, 290]])
def test_stalled_copies_time_out_and_context_survives(counts):
    """Single CTAs and pairs, in which one's waits end the other's."""
    c = Case(counts, 1056, 416, "bf16", 16, seed=13)
    try:
        moe.moe_test_stall_gemm_producer(3)
        c.whole()
    finally:
        moe.moe_test_stall_gemm_producer(-1)
    assert c.status.item() & moe.MOE_DEV_TIMEOUT
    c.status.zero_()
    xq, hq, y = c.steps()
    assert c.status.item() == 0
    c.check(xq, hq, y)


def test_offsets_past_32_bits():
    """The last expert's weights lie past 2^32 bytes of the packed buffer."""
    E, H, F, mx = 520, 4096, 4096, make(32)
    per = moe.moe_mx_bytes(mx, 1, H, F)
    assert (E - 1) * per > 1 << 32
    c = Case([2], H, F, "bf16", 32, seed=20, std=0.02)
    big = [torch.zeros(E * per, dtype=torch.uint8, device="cuda")
           for _ in range(3)]
    for b, p in zip(big, c.packs):
        b[(E - 1) * per:] = p
    want = c.whole()
    c.packs, c.cfg = big, c.cfg.with_(E=E)
    c.offsets = torch.tensor([0] * E + [2], dtype=torch.int32).cuda()
    assert torch.equal(c.whole(), want)
