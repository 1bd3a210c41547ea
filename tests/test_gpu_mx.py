"""Microscaled 4-bit floating point on the GPU against the oracle: packed
bytes bit for bit, products within a bound derived here.

Product bound.  Every product of two elements and their scales is exact in
fp32 (4-bit significands).  The tensor core adds 64 products to the
accumulator at a time; taking each of those 65 additions to lose at most one
unit of 2^-23 of the sum of magnitudes A = sum |x w| (truncation of an aligned
24-bit sum), K / 64 steps lose at most K * 65 / 64 * 2^-23 * A.  nvfp4's row
scales are two fp32 multiplications (powers of two unless packed by the
caller): 2^-23 |y|.  A split over at most 8 blocks adds 8 * 2^-24 * A.  The
output's rounding is half a step of its type.
"""
import numpy as np
import pytest
import torch

import workloads
from oracle import mx_oracle as O

pytestmark = pytest.mark.gpu

FMTS = ["mxfp4", "nvfp4"]


@pytest.fixture(scope="module")
def lq():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import dequant_gemv_group_b200 as m
    return m


def _f64(t):
    return t.double().cpu().numpy()


def _x(m, k, seed, std=1.0):
    x = workloads.normal_weights(m, k, std, seed=seed, outlier_frac=1e-2)
    if m > 2:
        x[2] = 0.0                       # a row of zeros
    if m > 4:
        x[4, :32] = 0.0                  # a block of zeros
        x[4, 1] = -0.0
    if m > 5:
        x[5] *= 2.0 ** -100              # far exponents
    if m > 6:
        x[6] *= 2.0 ** 100
    if m > 7:
        x[7, 0] = 2.0 ** -126            # beside ordinary values: underflows to 0
    return x


def _same_packed(got, codes, scales, rows, fmt):
    want, known = O.pack(codes, scales, rows, fmt)
    got = got.cpu().numpy()
    assert got.shape == want.shape
    np.testing.assert_array_equal(got[known], want[known])


def _bound(y, mag, k, dtype):
    eps = torch.finfo(dtype).eps / 2
    return (k * 65 / 64 * 2.0 ** -23 + 2.0 ** -21) * mag + (2.0 ** -23 + eps * 1.01) * np.abs(y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("n,k", [(1, 32), (9, 96), (128, 256), (130, 288), (33, 4096),
                                 (1301, 352), (1290, 8192), (1250, 8256)])
def test_quantize_bit_exact(lq, fmt, n, k):
    x = _x(n, k, seed=n + k)
    st = lq.new_status()
    got = lq.lutq_mx_quantize(x.cuda(), fmt, status=st)
    codes, scales, rows = O.quantize(_f64(x), fmt)
    _same_packed(got, codes, scales, rows, fmt)
    assert int(st.item()) == 0
    vals = O.values(codes, scales, rows, fmt)
    back = lq.lutq_mx_dequantize(got, n, k, fmt, dtype=torch.float32)
    # below 2^-126 the fp32 values stay exact (subnormals); the levels have 6 bits at most
    np.testing.assert_array_equal(_f64(back), vals)
    small = np.abs(vals) < 2.0 ** 15
    half = lq.lutq_mx_dequantize(got, n, k, fmt, dtype=torch.float16)
    np.testing.assert_array_equal(half.cpu().numpy()[small], vals[small].astype(np.float16))
    bf = lq.lutq_mx_dequantize(got, n, k, fmt)
    normal = (np.abs(vals) >= 2.0 ** -126) | (vals == 0)
    np.testing.assert_array_equal(_f64(bf)[normal], vals[normal])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_quantize_types(lq, fmt, dtype):
    x = (torch.randn(40, 320, generator=torch.Generator().manual_seed(1)) * 3)
    x = x.to(torch.bfloat16 if dtype == torch.float32 else dtype).to(dtype)
    got = lq.lutq_mx_quantize(x.cuda(), fmt)
    _same_packed(got, *O.quantize(_f64(x), fmt), fmt)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("beside", [1.0, 0.0])
def test_quantize_every_bf16(lq, fmt, beside):
    """All finite bf16 values, alone in their blocks and beside 1.0, in rows with and without it;
    then the same rows through the product that quantizes inside the kernel."""
    bits = torch.arange(0, 65536, dtype=torch.int32).to(torch.int16)
    v = bits.view(torch.bfloat16)
    v = v[torch.isfinite(v)]
    x = torch.zeros(v.numel(), 64, dtype=torch.bfloat16)
    x[:, 0] = v
    x[:, 32] = v
    x[:, 33] = beside
    x[:, 34] = -v                        # another value of the block on its levels
    got = lq.lutq_mx_quantize(x.cuda(), fmt)
    _same_packed(got, *O.quantize(_f64(x), fmt), fmt)
    w = lq.lutq_mx_quantize(torch.eye(64, dtype=torch.bfloat16, device="cuda") * 2.0 ** -20, fmt)
    xs = torch.cat([x[:16], x[5:21], x[200:216], x[-16:]]).cuda()
    for i in range(0, 64, 16):
        part = xs[i:i + 16].contiguous()
        y = lq.lutq_mx_gemm(lq.lutq_mx_quantize(part, fmt), 16, w, 64, 64, fmt)
        assert torch.equal(lq.lutq_mx_gemv(part, w, 64, 64, fmt), y)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_batched_and_packed(lq, fmt):
    """Several matrices at once, and the same bytes from codes and scales."""
    b, n, k = 3, 37, 224
    x = torch.stack([_x(n, k, seed=i) for i in range(b)])
    got = lq.lutq_mx_quantize(x.cuda(), fmt)
    assert got.shape == (b, lq.lutq_mx_packed_bytes(n, k, fmt))
    parts = [O.quantize(_f64(x[i]), fmt) for i in range(b)]
    for i in range(b):
        _same_packed(got[i], *parts[i], fmt)
    codes = np.stack([p[0] for p in parts])
    scales = torch.from_numpy(np.stack([p[1] for p in parts])).cuda()
    rows = torch.from_numpy(np.stack([p[2] for p in parts])).cuda()
    pair = torch.from_numpy(codes[..., 0::2] | (codes[..., 1::2] << 4)).cuda()
    again = lq.lutq_mx_pack(pair, scales, fmt, rows if fmt == "nvfp4" else None)
    for i in range(b):
        _same_packed(again[i], *parts[i], fmt)
    deq = lq.lutq_mx_dequantize(got, n, k, fmt, dtype=torch.float32)
    assert deq.shape == (b, n, k)
    for i in range(b):
        np.testing.assert_array_equal(_f64(deq[i]), O.values(*parts[i], fmt))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_reported(lq, fmt, bad):
    x = _x(20, 512, seed=5)
    x[11, 300] = bad
    st = lq.new_status()
    got = lq.lutq_mx_quantize(x.cuda(), fmt, status=st)
    _same_packed(got, *O.quantize(_f64(x), fmt), fmt)
    assert int(st.item()) == 5
    # every output of that row is NaN, the others are not
    w = lq.lutq_mx_quantize(workloads.normal_weights(64, 512, 0.02, seed=1).cuda(), fmt)
    y = lq.lutq_mx_gemm(got, 20, w, 64, 512, fmt)
    assert torch.isnan(y[11]).all() and torch.isfinite(y[:11]).all() and torch.isfinite(y[12:]).all()
    st = lq.new_status()
    y = lq.lutq_mx_gemv(x[8:16].contiguous().cuda(), w, 64, 512, fmt, status=st)
    assert int(st.item()) == 5
    assert torch.isnan(y[3]).all() and torch.isfinite(y[:3]).all() and torch.isfinite(y[4:]).all()


def _case(lq, m, n, k, fmt, seed=0):
    x = _x(m, k, seed=seed + m)
    if m > 5:
        x[5] *= 2.0 ** 100               # back in range of the products
    if m > 6:
        x[6] *= 2.0 ** -100
    w = workloads.normal_weights(n, k, 0.02, seed=seed + n, outlier_frac=1e-3)
    wp = lq.lutq_mx_quantize(w.cuda(), fmt)
    xv = O.values(*O.quantize(_f64(x), fmt), fmt)
    wv = O.values(*O.quantize(_f64(w), fmt), fmt)
    return x, wp, *O.product(xv, wv)


SHAPES = [(1, 1, 32), (1, 128, 256), (2, 7, 96), (3, 256, 512), (8, 1000, 2048), (15, 130, 4128),
          (16, 64, 14336), (17, 33, 288), (31, 513, 1024), (33, 128, 4096), (64, 640, 800),
          (65, 96, 2080), (127, 257, 544), (128, 384, 4096), (129, 1024, 256), (200, 200, 3232),
          (300, 2049, 96), (513, 300, 1056),
          (1, 20000, 512), (4, 1024, 28672), (13, 64, 8224),
          (40, 300, 14336), (250, 700, 14336), (290, 520, 8192), (70, 1030, 4128),
          # more tiles than pairs of blocks: 1 and 2 token tiles, row pitches that no 16-byte copy
          # can write, tokens beyond one pass over the weights
          (77, 9601, 288), (160, 9480, 64), (300, 8200, 96), (600, 4096, 544), (1000, 2564, 1312),
          (4099, 640, 160),
          # tiles of 512 weight rows: one round and several, rows behind the last
          (17, 19456, 288), (133, 19333, 544), (192, 37890, 96), (90, 76200, 64), (161, 57600, 1056)]


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", SHAPES)
def test_products(lq, fmt, m, n, k):
    x, wp, ref, mag = _case(lq, m, n, k, fmt)
    st = lq.new_status()
    xp = lq.lutq_mx_quantize(x.cuda(), fmt)
    y = lq.lutq_mx_gemm(xp, m, wp, n, k, fmt, status=st)
    assert int(st.item()) == 0
    err = np.abs(_f64(y) - ref)
    assert (err <= _bound(ref, mag, k, torch.float32)).all(), (err / np.maximum(mag, 1e-300)).max()
    yb = lq.lutq_mx_gemm(xp, m, wp, n, k, fmt, dtype=torch.bfloat16)
    assert torch.equal(yb, y.to(torch.bfloat16))
    yh = lq.lutq_mx_gemm(xp, m, wp, n, k, fmt, dtype=torch.float16)
    assert torch.equal(yh, y.to(torch.float16))
    if m <= 16:
        z = lq.lutq_mx_gemv(x.cuda(), wp, n, k, fmt, status=st)
        assert (np.abs(_f64(z) - ref) <= _bound(ref, mag, k, torch.float32)).all()
        assert int(st.item()) == 0


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [torch.float16, torch.float32])
def test_gemv_types(lq, fmt, dtype):
    m, n, k = 5, 200, 1120
    x = torch.randn(m, k, generator=torch.Generator().manual_seed(2)).to(torch.bfloat16).to(dtype)
    w = lq.lutq_mx_quantize(workloads.normal_weights(n, k, 0.02, seed=3).cuda(), fmt)
    y = lq.lutq_mx_gemv(x.cuda(), w, n, k, fmt)
    assert torch.equal(lq.lutq_mx_gemv(x.bfloat16().cuda(), w, n, k, fmt), y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [
    (16, 12288, 7168), (6, 12288, 7168), (16, 8192, 8192), (5, 28672, 2080), (16, 28672, 8192),
    (16, 14336, 4096), (2, 38000, 1056), (16, 2304, 28704), (9, 9600, 14336), (16, 40000, 2080),
    (1, 9472, 2048), (7, 4736, 4096), (3, 4097, 4128)])
def test_few_tokens_of_large_matrices(lq, fmt, m, n, k):
    """One tile a block and several, split or not, tokens kept in shared memory or not: against
    fp64 products of the values."""
    g = torch.Generator("cuda").manual_seed(n + m)
    w = lq.lutq_mx_quantize(torch.randn(n, k, device="cuda", generator=g).bfloat16(), fmt)
    x = torch.randn(m, k, device="cuda", generator=g).bfloat16()
    x[m // 2] *= 8
    xv, wv = (lq.lutq_mx_dequantize(p, r, k, fmt, dtype=torch.float32).double()
              for p, r in ((lq.lutq_mx_quantize(x, fmt), m), (w, n)))
    ref, mag = _f64(xv @ wv.t()), _f64(xv.abs() @ wv.abs().t())
    y = lq.lutq_mx_gemv(x, w, n, k, fmt)
    assert (np.abs(_f64(y) - ref) <= _bound(ref, mag, k, torch.float32)).all()
    assert torch.equal(lq.lutq_mx_gemv(x, w, n, k, fmt), y)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m", [1, 16, 40, 150, 700])
def test_exact_sums(lq, fmt, m):
    """Small integers in scales of 1: every partial sum is exact, so y is too, in every tile."""
    n, k = 391, 1312
    g = torch.Generator().manual_seed(m)
    lv = torch.tensor([0.0, 1.0, 2.0, 3.0, 4.0, 6.0])
    pick = lambda *s: lv[torch.randint(0, 6, s, generator=g)] * (  # noqa: E731
        torch.randint(0, 2, s, generator=g) * 2 - 1)
    x, w = pick(m, k), pick(n, k)
    x[:, 0::32], w[:, 0::32] = 6.0, 6.0
    x[:, 16::32], w[:, 16::32] = 6.0, 6.0
    y = lq.lutq_mx_gemm(lq.lutq_mx_quantize(x.bfloat16().cuda(), fmt), m,
                        lq.lutq_mx_quantize(w.bfloat16().cuda(), fmt), n, k, fmt)
    if fmt == "nvfp4":  # s = 6 / 6 / g = 256 = 1 / g
        assert float(O.quantize(_f64(x), fmt)[2].max()) == 2.0 ** -8
    assert torch.equal(y.cpu(), (x.double() @ w.double().t()).float())


@pytest.mark.parametrize("fmt", FMTS)
def test_one_hot(lq, fmt):
    """A token that is 1 at one position reads a column of the weights, scales and all."""
    n, k = 160, 1056
    w = workloads.normal_weights(n, k, 0.02, seed=8, outlier_frac=1e-2)
    wp = lq.lutq_mx_quantize(w.cuda(), fmt)
    wv = O.values(*O.quantize(_f64(w), fmt), fmt)
    pos = list(range(0, k, 5)) + [k - 1]
    x = torch.zeros(len(pos), k)
    x[torch.arange(len(pos)), pos] = 1.0
    y = lq.lutq_mx_gemm(lq.lutq_mx_quantize(x.bfloat16().cuda(), fmt), len(pos), wp, n, k, fmt)
    # nvfp4: 1 = 6 * (170.67 -> 176) / 1024 * ... is not a level: the oracle's value of x scales it
    xv = O.values(*O.quantize(_f64(x), fmt), fmt)
    np.testing.assert_allclose(_f64(y), xv @ wv.T, rtol=2.0 ** -22, atol=0)


def test_nvfp4_row_scales_from_a_checkpoint(lq):
    """Row scales that are no powers of two, and none."""
    n, k, m = 70, 256, 20
    g = torch.Generator().manual_seed(9)
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)
    scales = torch.randint(0, 0x60, (n, k // 16), generator=g).to(torch.uint8)
    rows = torch.rand(n, generator=g) + 0.1
    x = _x(m, k, seed=1)
    x[5], x[6] = x[0], x[1]
    xp = lq.lutq_mx_quantize(x.cuda(), "nvfp4")
    xv = O.values(*O.quantize(_f64(x), "nvfp4"), "nvfp4")
    c = codes.numpy()
    c = np.stack([c & 15, c >> 4], -1).reshape(n, k)
    for r in (rows, None):
        wp = lq.lutq_mx_pack(codes.cuda(), scales.cuda(), "nvfp4", None if r is None else r.cuda())
        wv = O.values(c, scales.numpy(), np.ones(n) if r is None else r.numpy(), "nvfp4")
        ref, mag = O.product(xv, wv)
        y = lq.lutq_mx_gemm(xp, m, wp, n, k, "nvfp4")
        assert (np.abs(_f64(y) - ref) <= _bound(ref, mag, k, torch.float32)).all()


def test_pack_drops_the_sign_of_e4m3(lq):
    n, k = 5, 64
    g = torch.Generator().manual_seed(3)
    codes = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8).cuda()
    scales = torch.randint(0, 0x7f, (n, k // 16), generator=g).to(torch.uint8).cuda()
    wp = lq.lutq_mx_pack(codes, scales, "nvfp4")
    assert torch.equal(lq.lutq_mx_dequantize(lq.lutq_mx_pack(codes, scales | 0x80, "nvfp4"), n, k,
                                             "nvfp4"),
                       lq.lutq_mx_dequantize(wp, n, k, "nvfp4"))


@pytest.mark.parametrize("fmt", FMTS)
def test_one_very_long_row(lq, fmt):
    """More chunks than a grid has blocks in its second dimension."""
    k, part = (1 << 28) + 64, 4096
    w = torch.zeros(1, k, dtype=torch.bfloat16, device="cuda")
    ends = workloads.normal_weights(1, 2 * part, 1.0, seed=8)
    w[:, :part], w[:, k - part:] = ends[:, :part].cuda(), ends[:, part:].cuda()
    back = lq.lutq_mx_dequantize(lq.lutq_mx_quantize(w, fmt), 1, k, fmt)
    assert (back[:, part:k - part] == 0).all()
    got = torch.cat([back[:, :part], back[:, k - part:]], 1)
    want = O.values(*O.quantize(_f64(ends), fmt), fmt)
    assert np.array_equal(_f64(got), want)


@pytest.mark.parametrize("fmt", FMTS)
def test_offsets_beyond_32_bits(lq, fmt):
    """The last rows of a matrix of 2.3 GB and the last outputs of 5.6 GB are what they are in
    small ones."""
    n, k, last = (1 << 20) + 100, 4096, 356
    w = torch.randn(n, k, dtype=torch.bfloat16, device="cuda",
                    generator=torch.Generator("cuda").manual_seed(1))
    x = torch.randn(20, k, device="cuda").bfloat16()
    wp = lq.lutq_mx_quantize(w, fmt)
    tail = lq.lutq_mx_quantize(w[n - last:].contiguous(), fmt)
    back = lq.lutq_mx_dequantize(wp, n, k, fmt)
    assert torch.equal(back[n - last:], lq.lutq_mx_dequantize(tail, last, k, fmt))
    del w, back
    xp = lq.lutq_mx_quantize(x, fmt)
    tv = _f64(lq.lutq_mx_dequantize(tail, last, k, fmt, dtype=torch.float32))
    xv = _f64(lq.lutq_mx_dequantize(xp, 20, k, fmt, dtype=torch.float32))
    ref, mag = O.product(xv, tv)
    y = _f64(lq.lutq_mx_gemm(xp, 20, wp, n, k, fmt)[:, n - last:])
    assert (np.abs(y - ref) <= _bound(ref, mag, k, torch.float32)).all()
    y = _f64(lq.lutq_mx_gemv(x[:3].contiguous(), wp, n, k, fmt)[:, n - last:])
    assert (np.abs(y - ref[:3]) <= _bound(ref[:3], mag[:3], k, torch.float32)).all()
    del wp
    m, n, k = 70000, 40008, 64
    x = torch.randn(m, k, device="cuda").bfloat16()
    w = torch.randn(n, k, device="cuda").bfloat16()
    y = lq.lutq_mx_gemm(lq.lutq_mx_quantize(x, fmt), m, lq.lutq_mx_quantize(w, fmt), n, k, fmt,
                        dtype=torch.bfloat16)
    # (one order of the sum whatever the tile: K is a single chunk)
    z = lq.lutq_mx_gemm(lq.lutq_mx_quantize(x[m - 300:].contiguous(), fmt), 300,
                        lq.lutq_mx_quantize(w[n - 500:].contiguous(), fmt), 500, k, fmt,
                        dtype=torch.bfloat16)
    assert torch.equal(y[m - 300:, n - 500:], z)


@pytest.mark.parametrize("fmt", FMTS)
def test_deterministic_and_in_bounds(lq, fmt):
    """Twice the same bits; nothing behind y is written; garbage in the codes' padding and in the
    rows behind the last one does not matter."""
    for m, n, k in [(1, 1000, 4096), (16, 333, 2048), (50, 130, 1024), (140, 257, 512)]:
        x, wp, _, _ = _case(lq, m, n, k, fmt, seed=4)
        xp = lq.lutq_mx_quantize(x.cuda(), fmt)
        buf = torch.full((m * n + 512,), 7.0, device="cuda")
        y = buf[:m * n].view(m, n)
        lq.lutq_mx_gemm(xp, m, wp, n, k, fmt, y=y)
        assert (buf[m * n:] == 7.0).all()
        for _ in range(3):
            assert torch.equal(lq.lutq_mx_gemm(xp, m, wp, n, k, fmt), y)
        if m <= 16:
            z = lq.lutq_mx_gemv(x.cuda(), wp, n, k, fmt)
            for _ in range(3):
                assert torch.equal(lq.lutq_mx_gemv(x.cuda(), wp, n, k, fmt), z)


def test_refusals(lq):
    """What the binding refuses on a GPU: strides, shapes, sizes, alignment."""
    x = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda")
    w = lq.lutq_mx_quantize(torch.ones(8, 128, dtype=torch.bfloat16, device="cuda"), "nvfp4")
    with pytest.raises(ValueError):
        lq.lutq_mx_quantize(x.t(), "mxfp4")
    with pytest.raises(ValueError):
        lq.lutq_mx_quantize(x.double(), "mxfp4")
    with pytest.raises(ValueError):
        lq.lutq_mx_gemv(x[:, ::2], w, 8, 64, "nvfp4")
    for bad in (lambda: lq.lutq_mx_quantize(x[:, :48].contiguous(), "mxfp4"),
                lambda: lq.lutq_mx_quantize(x[0], "mxfp4"),
                lambda: lq.lutq_mx_gemv(x, w, 8, 96, "nvfp4"),
                lambda: lq.lutq_mx_gemv(x, w, 9, 128, "nvfp4"),
                lambda: lq.lutq_mx_gemv(x, w, 8, 128, "mxfp4"),
                lambda: lq.lutq_mx_gemv(x.repeat(5, 1), w, 8, 128, "nvfp4"),
                lambda: lq.lutq_mx_gemm(w, 9, w, 8, 128, "nvfp4"),
                lambda: lq.lutq_mx_gemm(w, 8, w, 8, 128, "nvfp4", y=torch.empty(8, 9, device="cuda")),
                lambda: lq.lutq_mx_dequantize(w, 8, 96, "nvfp4"),
                lambda: lq.lutq_mx_gemv(torch.ones(513, dtype=torch.bfloat16, device="cuda")[1:]
                                        .view(4, 128), w, 8, 128, "nvfp4")):
        with pytest.raises(lq.LutqError):
            bad()
    with pytest.raises(ValueError):
        lq.lutq_mx_gemm(w, 8, w, 8, 128, "nvfp4", dtype=torch.float64)


def test_empty(lq):
    w = lq.lutq_mx_quantize(torch.ones(8, 64, dtype=torch.bfloat16, device="cuda"), "mxfp4")
    none = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    assert lq.lutq_mx_gemv(none, w, 8, 64, "mxfp4").shape == (0, 8)
    xp = lq.lutq_mx_quantize(none, "mxfp4")
    assert xp.numel() == 0
    assert lq.lutq_mx_gemm(xp, 0, w, 8, 64, "mxfp4").shape == (0, 8)


@pytest.mark.parametrize("fmt", FMTS)
def test_streams_and_graphs(lq, fmt):
    """Two streams at once, and a captured chain replayed on new inputs."""
    m, n, k = 12, 1024, 4096
    x, wp, _, _ = _case(lq, m, n, k, fmt, seed=6)
    x = x.cuda()
    want = lq.lutq_mx_gemv(x, wp, n, k, fmt)
    both = lq.lutq_mx_gemm(lq.lutq_mx_quantize(x, fmt), m, wp, n, k, fmt)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        for s in (s1, s2):
            with torch.cuda.stream(s):
                got.append(lq.lutq_mx_gemv(x, wp, n, k, fmt))
                got.append(lq.lutq_mx_gemm(lq.lutq_mx_quantize(x, fmt), m, wp, n, k, fmt))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got[0::2])
    assert all(torch.equal(g, both) for g in got[1::2])
    xin = torch.zeros_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = lq.lutq_mx_gemv(xin, wp, n, k, fmt)
        b = lq.lutq_mx_gemm(lq.lutq_mx_quantize(xin, fmt), m, wp, n, k, fmt)
    for scale in (1.0, -2.0):
        xin.copy_(x * scale)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(a, want * scale) and torch.equal(b, both * scale)
