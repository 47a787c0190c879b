"""GPU tests of the microscaled 4-bit operators against the plain form in 64 bits."""
import numpy as np
import pytest
import torch

import mx4_ref as ref
import w8a8_int8_dynamic_b200 as w8
from gpu_util import require_gpu

pytestmark = pytest.mark.gpu

HALF = torch.finfo(torch.bfloat16).eps / 2  # a rounding to bf16, relative to the value


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    assert w8.poll_status() == 0


def bf(a):
    return torch.from_numpy(np.asarray(a)).to(torch.bfloat16).cuda()


def f64(t):
    return t.double().cpu().numpy()


def sample(rng, rows, K, kind="outliers"):
    x = rng.standard_normal((rows, K))
    if kind == "outliers":
        x[:, rng.permutation(K)[: max(1, K // 50)]] *= 20
    elif kind == "wide":  # block maxima over the whole range of bf16
        x *= np.exp2(rng.integers(-140, 120, (rows, K)).astype(np.float64))
    elif kind == "ties":  # eighths: every tie of the grid occurs under a scale of 1
        x = rng.integers(-63, 64, (rows, K)) / 8.0
    return bf(x)


SHAPES = [(1, 16), (1, 5120), (2, 32), (3, 48), (127, 272), (128, 256), (129, 240), (200, 1808), (300, 528)]


@pytest.mark.parametrize("rows,K", SHAPES)
@pytest.mark.parametrize("kind", ["outliers", "wide", "ties"])
def test_quant_codes_and_scales(rows, K, kind):
    x = sample(np.random.default_rng(rows * 7 + K), rows, K, kind)
    x[rows // 2, : min(K, 32)] = 0
    x[0, 0] = -0.0
    codes, scales = w8.mx4_quant(x).unpack()
    want_c, want_s = ref.encode(f64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert np.array_equal(ref.unpack_codes(codes.cpu().numpy()), want_c)
    assert np.array_equal(f64(w8.mx4_quant(x).dequant()), f64(bf(ref.values(want_c, want_s))))


def test_quant_subnormals_infinities_and_nan():
    x = torch.zeros((6, 64), dtype=torch.bfloat16, device="cuda")
    x[0, 3] = 2.0 ** -133          # the smallest subnormal: the smallest scale, code 0
    x[1, 3], x[1, 4] = 2.0 ** -127, -1.5 * 2.0 ** -127
    x[2, 5] = float("inf")
    x[3, 40] = float("nan")
    x[4, 0] = torch.finfo(torch.bfloat16).max
    x[5, 1] = -float("inf")
    codes, scales = w8.mx4_quant(x).unpack()
    want_c, want_s = ref.encode(f64(x))
    assert np.array_equal(scales.cpu().numpy(), want_s)
    assert want_s[2].tolist() == [255, 0] and want_s[3].tolist() == [0, 255] and want_s[4, 0] == 252
    assert np.array_equal(ref.unpack_codes(codes.cpu().numpy()), want_c)
    back = w8.mx4_quant(x).dequant()
    assert back[2, :32].isnan().all() and not back[2, 32:].any() and back[3, 32:].isnan().all()


@pytest.mark.parametrize("rows,K", [(1, 16), (130, 272), (5, 1040)])
def test_pack_and_unpack_every_code(rows, K):
    rng = np.random.default_rng(3)
    codes = torch.from_numpy(rng.integers(0, 256, (rows, K // 2), dtype=np.uint8)).cuda()
    scales = torch.from_numpy(rng.integers(0, 256, (rows, -(-K // 32)), dtype=np.uint8)).cuda()
    t = w8.mx4_pack(codes, scales)
    c, s = t.unpack()
    assert torch.equal(c, codes) and torch.equal(s, scales)
    v = ref.values(ref.unpack_codes(codes.cpu().numpy()), scales.cpu().numpy())
    assert np.array_equal(f64(t.dequant()), f64(bf(v)), equal_nan=True)


def test_quant_strides_leading_sizes_and_rows_behind():
    rng = np.random.default_rng(5)
    wide = sample(rng, 60, 400)
    want = w8.mx4_quant(wide[:, 16:288].contiguous()).unpack()
    for x in (wide[:, 16:288], wide[:, 16:288].reshape(5, 12, 272), wide.t().contiguous().t()[:, 16:288]):
        t = w8.mx4_quant(x)
        got = t.unpack()
        assert all(torch.equal(g, w) for g, w in zip(got, want))
        assert t.dequant().shape == x.shape
    # rows past the last one of the image keep what they held
    image = torch.full((w8.mx4_bytes(60, 272),), 0xA5, dtype=torch.uint8, device="cuda")
    w8.mx4_quant(wide[:, 16:288], image=image)
    rest = w8.MX4Tensor(image, (128,), 272).unpack()
    assert (rest[0][60:] == 0xA5).all() and (rest[1][60:] == 0xA5).all()


def operands(seed, M, N, K, bias=True):
    rng = np.random.default_rng(seed)
    x = sample(rng, M, K)
    w = w8.mx4_quant(bf(rng.standard_normal((N, K)) * K ** -0.5))
    b = bf(rng.standard_normal(N) * 0.1) if bias else None
    return x, w, b


def plain(t):
    c, s = t.unpack()
    return ref.values(ref.unpack_codes(c.cpu().numpy()), s.cpu().numpy())


def check_product(y, a, w, b, act):
    """y against the 64-bit product of the images' values: the fp32 sum's error, the bias's addition, and one
    rounding to bf16; with GELU, of the rounded value, whose rounding may go either way within that error."""
    va, vw = plain(a), plain(w)
    K = a.K
    t = va @ vw.T + (f64(b) if b is not None else 0.0)
    err = ref.sum_error(va, vw, K) + 2.0 ** -23 * np.abs(t)
    got = f64(y).reshape(t.shape)
    if act == w8.ACT_NONE:
        assert (np.abs(got - t) <= err + HALF * (np.abs(t) + err)).all()
        return
    # 2^-14: the activation's own accuracy (act.cuh); subnormal outputs: one step
    sides = np.stack([ref.gelu(f64(bf(t + d * err))) for d in (-1, 0, 1)])
    # GELU falls and rises: a range of one rounding step may hold its minimum, which changes it by less than the step
    lo, hi = sides.min(0), sides.max(0)
    slack = (HALF + 2.0 ** -14) * np.maximum(np.abs(lo), np.abs(hi)) + 2.0 ** -133
    assert ((got >= lo - slack) & (got <= hi + slack)).all()


PRODUCTS = [(1, 8, 16), (1, 128, 256), (2, 24, 48), (7, 136, 528), (16, 264, 1040), (17, 256, 512), (33, 520, 272),
            (65, 128, 2064), (128, 128, 256), (129, 392, 784), (200, 1000, 496), (300, 640, 1808), (520, 776, 560)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
@pytest.mark.parametrize("bias,act", [(False, w8.ACT_NONE), (True, w8.ACT_NONE), (True, w8.ACT_GELU_TANH)])
def test_product(M, N, K, bias, act):
    x, w, b = operands(M + N + K, M, N, K, bias)
    a = w8.mx4_quant(x)
    y = w8.mx4_scaled_mm(a, w, b, act=act)
    check_product(y, a, w, b, act)
    assert torch.equal(w8.mx4_linear(x, w, b, act=act), y)


@pytest.mark.parametrize("M,N,K", [(m, n // 16 * 16, k) for m, n, k in PRODUCTS if n >= 16])
@pytest.mark.parametrize("act", [w8.ACT_NONE, w8.ACT_GELU_TANH])
def test_product_with_codes_of_its_output(M, N, K, act):
    x, w, b = operands(M + N + K, M, N, K)
    image = torch.full((w8.mx4_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")  # NaN scales where unwritten
    t = w8.mx4_linear_quant(x, w, b, image=image, act=act)
    want = w8.mx4_quant(w8.mx4_linear(x, w, b, act=act))
    assert all(torch.equal(g, v) for g, v in zip(t.unpack(), want.unpack()))
    # the padding up to the image's last column is zeros with a finite scale: the next product may read it
    padded = -(-N // 256) * 256
    c, s = w8.MX4Tensor(t.image, (M,), padded).unpack()
    assert not c[:, N // 2:].any() and not (s[:, -(-N // 32):] == 255).any()


@pytest.mark.parametrize("path", [w8.PATH_LARGE, w8.PATH_SMALL])
@pytest.mark.parametrize("M,N,K", [(1, 1000, 5120), (4, 520, 13824), (16, 4096, 1040), (16, 136, 8208), (13, 5120, 784),
                                   (17, 4096, 528), (30, 136, 13824), (64, 2056, 4112), (50, 8, 16384),
                                   (33, 27648, 272), (65, 1000, 5136), (100, 4096, 528), (128, 136, 13824),
                                   (77, 27648, 272)])
def test_product_of_few_rows_on_either_path(M, N, K, path):
    """One and several slabs a cluster, K whole and split in up to eight: both kernels, y and its codes."""
    x, w, b = operands(M + N + K, M, N, K)
    a = w8.mx4_quant(x)
    w8.set_path(path)
    try:
        y = w8.mx4_scaled_mm(a, w, b)
        check_product(y, a, w, b, w8.ACT_NONE)
        for _ in range(5):
            assert torch.equal(w8.mx4_scaled_mm(a, w, b), y)
        if path == w8.PATH_SMALL or M > 16:
            assert torch.equal(w8.mx4_linear(x, w, b), y)
        if N % 16 == 0:
            image = torch.full((w8.mx4_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")
            t = w8.mx4_scaled_mm_quant(a, w, b, image=image)
            want, padded = w8.mx4_quant(y), -(-N // 256) * 256
            for g, v in zip(w8.MX4Tensor(t.image, (128,), padded).unpack(), w8.MX4Tensor(want.image, (M,), padded).unpack()):
                assert torch.equal(g[:M], v)
                assert (g[M:] == 0xFF).all()  # the rows behind are left alone
    finally:
        w8.set_path(w8.PATH_AUTO)


@pytest.mark.parametrize("path", [w8.PATH_LARGE, w8.PATH_LARGE_PAIR])
@pytest.mark.parametrize("M,N,K,act", [(1, 8, 16, 0), (128, 256, 256, 0), (129, 264, 272, 1), (256, 256, 4096, 0),
                                       (300, 640, 1808, 1), (384, 1168, 528, 0), (1000, 1040, 784, 1),
                                       (2600, 2064, 1040, 0), (700, 5136, 272, 0), (300, 512, 12304, 0)])
def test_product_of_many_rows_on_either_path(M, N, K, act, path):
    """Ragged tiles, several tiles a CTA, K from one step to more than the ring: both kernels, y and its codes."""
    x, w, b = operands(M + N + K, M, N, K)
    a = w8.mx4_quant(x)
    w8.set_path(path)
    try:
        y = w8.mx4_linear(x, w, b, act=act)
        check_product(y, a, w, b, act)
        assert torch.equal(w8.mx4_scaled_mm(a, w, b, act=act), y)
        if N % 16 == 0:
            image = torch.full((w8.mx4_bytes(M, N),), 0xFF, dtype=torch.uint8, device="cuda")
            t = w8.mx4_scaled_mm_quant(a, w, b, image=image, act=act)
            padded = -(-N // 256) * 256
            want = w8.mx4_quant(y)
            for g, v in zip(w8.MX4Tensor(t.image, (M,), padded).unpack(),
                            w8.MX4Tensor(want.image, (M,), padded).unpack()):
                assert torch.equal(g, v)
            if M % 128:  # rows behind the last one are left as they were
                c, s = w8.MX4Tensor(t.image, (-(-M // 128) * 128,), padded).unpack()
                assert (c[M:] == 255).all() and (s[M:] == 255).all()
    finally:
        w8.set_path(w8.PATH_AUTO)


@pytest.mark.parametrize("M,N,K", [(13, 5120, 2064), (30, 5120, 2064), (60, 5120, 4112), (3, 12288, 4112),
                                   (8, 20864, 7440), (20, 20864, 7440), (60, 20864, 7440), (1, 27648, 5120),
                                   (65, 5120, 7440), (97, 1040, 13824), (128, 6152, 12304), (128, 5120, 5136)])
def test_product_of_few_rows_over_every_split(M, N, K):
    """Clusters of one to four CTAs, one slab each or several in turn, against the 64-bit product of the values."""
    g = torch.Generator(device="cuda").manual_seed(N + K)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    w = w8.mx4_quant(torch.randn(N, K, device="cuda", generator=g).mul_(K ** -0.5).bfloat16())
    b = torch.randn(N, device="cuda", generator=g).bfloat16()
    a = w8.mx4_quant(x)
    va, vw = a.dequant().double(), w.dequant().double()
    t = va @ vw.t() + b.double()
    err = (K / 64 + 8) * 2.0 ** -22 * (va.abs() @ vw.abs().t()) + 2.0 ** -23 * t.abs()
    y = w8.mx4_scaled_mm(a, w, b)
    assert ((y.double() - t).abs() <= err + HALF * (t.abs() + err)).all()
    for _ in range(4):
        assert torch.equal(w8.mx4_linear(x, w, b), y)
    if N % 16 == 0:  # an output image's condition
        assert all(torch.equal(p, q) for p, q in zip(w8.mx4_linear_quant(x, w, b).unpack(), w8.mx4_quant(y).unpack()))
