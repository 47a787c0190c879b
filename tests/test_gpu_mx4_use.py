"""GPU tests of the 4-bit layers and the block norm as a serving program runs them: together, on other streams, in
CUDA graphs, back to back, in place, with rows or values left out, and on tensors longer than 32-bit offsets reach."""
import threading

import numpy as np
import pytest
import torch

import mx4_ref as ref
import w8a8_int8_dynamic_b200 as w8
from gpu_util import require_gpu
from test_gpu_mx4 import bf, check_product, f64, operands, plain, sample

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    assert w8.poll_status() == 0


def layers(seed, D, F):
    rng = np.random.default_rng(seed)
    up = w8.MX4Linear.from_float(bf(rng.standard_normal((F, D)) * D ** -0.5), bf(rng.standard_normal(F) * 0.1),
                                 act=w8.ACT_GELU_TANH)
    down = w8.MX4Linear.from_float(bf(rng.standard_normal((D, F)) * F ** -0.5), bf(rng.standard_normal(D) * 0.1))
    n = w8.Norm("layer", bf(1 + 0.1 * rng.standard_normal(D)), bf(0.1 * rng.standard_normal(D)))
    mod = bf(rng.standard_normal((2, 3 * D)) * 0.3).split(D, 1)
    return up, down, n, mod


def block(x, stream, up, down, n, mod, per):
    """A transformer block's second half: norm after attention into the stream, MLP, its norm into the stream."""
    a = w8.block_norm(x, stream, gate=mod[0], pre=n, scale=mod[1], shift=mod[2], rows_per_group=per, codes="mx4")
    h = up.quantised(a.mx4)
    return w8.block_norm(down(h), a.residual, post=n, gate=mod[0], residual_scale=0.9, pre=n, rows_per_group=per)


def block_in_steps(x, stream, up, down, n, mod, per):
    """The same by unfused calls: each is tested against its formula elsewhere."""
    a = w8.block_norm(x, stream, gate=mod[0], pre=n, scale=mod[1], shift=mod[2], rows_per_group=per)
    y = w8.mx4_scaled_mm(w8.mx4_quant(a.y), up.w, up.bias, act=w8.ACT_GELU_TANH)
    z = w8.mx4_scaled_mm(w8.mx4_quant(y), down.w, down.bias)
    return w8.block_norm(z, a.residual, post=n, gate=mod[0], residual_scale=0.9, pre=n, rows_per_group=per)


@pytest.mark.parametrize("M", [1, 5, 16, 17, 64, 65, 300, 1100])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_a_block_fused_equals_its_steps(M, dtype):
    D, F = 1040, 2064
    up, down, n, mod = layers(3, D, F)
    x = sample(np.random.default_rng(M), M, D)
    stream = torch.randn(M, D, device="cuda").to(dtype)
    per = -(-M // 2)
    got, want = block(x, stream, up, down, n, mod, per), block_in_steps(x, stream, up, down, n, mod, per)
    assert torch.equal(got.residual, want.residual) and torch.equal(got.y, want.y)
    # the products in the middle, against 64 bits
    a = w8.block_norm(x, stream, gate=mod[0], pre=n, scale=mod[1], shift=mod[2], rows_per_group=per, codes="mx4").mx4
    check_product(up(a), a, up.w, up.bias, w8.ACT_GELU_TANH)
    h = up.quantised(a)
    check_product(down(h), h, down.w, down.bias, w8.ACT_NONE)


@pytest.mark.parametrize("M", [1, 16, 17, 500])
def test_int8_layer_on_the_norms_codes(M):
    D, N = 528, 1032
    rng = np.random.default_rng(M)
    layer = w8.W8A8Linear(torch.from_numpy(rng.integers(-127, 128, (N, D), dtype=np.int8)).cuda(),
                          torch.rand(N, device="cuda") * 1e-2, bf(rng.standard_normal(N)))
    x, n = sample(rng, M, D), w8.Norm("rms", bf(1 + 0.1 * rng.standard_normal(D)))
    out = w8.block_norm(x.view(1, M, D), pre=n, codes="int8", y=True)
    y = layer.apply_codes(out.q, out.a_scale)
    assert y.shape == (1, M, N) and torch.equal(y, layer(out.y))


@pytest.mark.parametrize("M", [1, 40, 700])
def test_graphs_replayed_on_new_inputs_beside_each_other(M):
    """Two captures of the same layers, replayed by turns on new inputs, with eager calls between them."""
    D, F = 784, 1552
    up, down, n, mod = layers(5, D, F)
    rng = np.random.default_rng(M)
    per = -(-M // 2)
    held = []
    for _ in range(2):
        x, stream = sample(rng, M, D), torch.randn(M, D, device="cuda")
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            block(x, stream, up, down, n, mod, per)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            out = block(x, stream, up, down, n, mod, per)
        held.append((g, x, stream, out))
    for i in range(6):
        g, x, stream, out = held[i % 2]
        x.copy_(sample(rng, M, D))
        stream.copy_(torch.randn(M, D, device="cuda"))
        g.replay()
        want = block(x, stream, up, down, n, mod, per)
        torch.cuda.synchronize()
        assert torch.equal(out.residual, want.residual) and torch.equal(out.y, want.y)
    for g, *_ in held:
        g.reset()


@pytest.mark.parametrize("M", [3, 17, 300])
def test_other_streams(M):
    """Calls given a stream, from a thread whose current stream is another; one layer on two streams at once."""
    D, F = 784, 1552
    up, down, n, mod = layers(7, D, F)
    x = sample(np.random.default_rng(M), M, D)
    want = down(up.quantised(x))
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for s in (s1, s2):
        s.wait_stream(torch.cuda.current_stream())
    got = []
    for i in range(20):
        for s in (s1, s2):
            h = up.quantised(x, stream=s)
            got.append(down(h, stream=s))
            q = w8.mx4_quant(x, stream=s)
            r = w8.block_norm(q.dequant(stream=s), pre=n, codes="mx4", stream=s)
            got.append(w8.mx4_scaled_mm(r.mx4, up.w, stream=s))
    torch.cuda.synchronize()
    second = w8.mx4_scaled_mm(w8.block_norm(w8.mx4_quant(x).dequant(), pre=n, codes="mx4").mx4, up.w)
    for i, y in enumerate(got):
        assert torch.equal(y, second if i % 2 else want)


def test_many_calls_back_to_back():
    """Chains whose kernels start before the ones ahead have ended: every shape's kernel before and after every
    other's, on memory that the allocator hands from one call to the next, weights made just before their use."""
    rng = np.random.default_rng(11)
    D = 784
    cases = []
    for M in (1, 16, 17, 33, 65, 130, 600):
        for N in (136, 1040):
            x, w, b = operands(M + N, M, N, D)
            codes, scales = w.unpack()
            cases.append((x, codes, scales, b, w8.mx4_linear(x, w, b)))
    n = w8.Norm("rms")
    torch.cuda.synchronize()
    for _ in range(6):
        order = rng.permutation(len(cases))
        got = []
        for i in order:
            x, codes, scales, b, _ = cases[i]
            w = w8.mx4_pack(codes, scales)
            y = w8.mx4_linear(x, w, b)
            w8.block_norm(x, pre=n, codes="mx4")
            got.append((i, y))
        torch.cuda.synchronize()
        for i, y in got:
            assert torch.equal(y, cases[i][4])


def test_weights_that_the_kernel_ahead_has_just_written():
    """The right operand may come from any kernel: a quantisation, a product's epilogue, a norm."""
    x, w, _ = operands(13, 24, 528, 272, bias=False)
    v = sample(np.random.default_rng(1), 272, 528)
    n = w8.Norm("rms")
    for _ in range(30):
        for make in (lambda: w8.mx4_quant(v), lambda: w8.mx4_scaled_mm_quant(w8.mx4_quant(v), w8.mx4_quant(v[:, :528])),
                     lambda: w8.block_norm(v, pre=n, codes="mx4").mx4):
            t = make()
            a = sample(np.random.default_rng(2), 5, t.K)
            got = w8.mx4_linear(a, t)
            torch.cuda.synchronize()
            assert torch.equal(got, w8.mx4_linear(a, t))


def test_nan_and_infinity_stay_in_their_rows():
    for M in (5, 20, 200):
        x, w, b = operands(M, M, 264, 528)
        y = w8.mx4_linear(x, w, b)
        x[1, 100], x[3, 527] = float("nan"), float("-inf")
        got = w8.mx4_linear(x, w, b)
        rest = [m for m in range(M) if m not in (1, 3)]
        assert got[1].isnan().all() and got[3].isnan().all() and torch.equal(got[rest], y[rest])
        # a row of zeros gives the bias
        x[:] = 0
        assert torch.equal(w8.mx4_linear(x, w, b), b.expand(M, -1))


def test_no_rows_no_launch():
    x, w, b = operands(1, 4, 264, 272)
    before = w8.launch_count()
    for lead in ((0,), (2, 0)):
        e = x[:0].view(*lead, 272)
        assert w8.mx4_linear(e, w, b).shape == (*lead, 264)
        t = w8.mx4_quant(e)
        assert t.dequant().shape == e.shape and w8.mx4_scaled_mm(t, w, b).shape == (*lead, 264)
        assert w8.mx4_scaled_mm_quant(t, w, b[:264]).lead == lead if w.rows % 16 == 0 else True
        assert w8.block_norm(e, e.float(), pre=w8.Norm("rms"), codes="int8").q.shape == e.shape
    assert w8.launch_count() == before


def test_one_launch_a_few_row_layer_and_two_a_larger_one():
    x, w, b = operands(1, 17, 264, 272)
    for M, launches in ((1, 1), (16, 1), (17, 2)):
        before = w8.launch_count()
        w8.mx4_linear(x[:M], w, b)
        assert w8.launch_count() - before == launches


def test_outputs_given_and_refused():
    x, w, b = operands(2, 20, 272, 272)
    want = w8.mx4_linear(x, w, b)
    out = torch.empty(20 * 272, dtype=torch.bfloat16, device="cuda")
    assert torch.equal(w8.mx4_linear(x, w, b, out=out), want) and torch.equal(out.view(20, 272), want)
    ws = torch.empty(w8.mx4_linear_workspace_bytes(20, 272, 272), dtype=torch.uint8, device="cuda")
    assert torch.equal(w8.mx4_linear(x, w, b, workspace=ws), want)
    t = w8.mx4_quant(x)
    for f in (lambda: w8.mx4_linear(x, w, b, out=out.float()), lambda: w8.mx4_linear(x, w, b[:8]),
              lambda: w8.mx4_linear(x.float(), w, b), lambda: w8.mx4_linear(x[:, :256], w, b),
              lambda: w8.mx4_scaled_mm(t, w, b, out=torch.empty(272, 20, dtype=torch.bfloat16, device="cuda").t()),
              lambda: w8.mx4_scaled_mm(w8.MX4Tensor(t.image[:100], (20,), 272), w, b),
              lambda: w8.mx4_pack(*w.unpack()[:1], torch.zeros(272, 8, dtype=torch.uint8, device="cuda")),
              lambda: w8.block_norm(x, x[:4], pre=w8.Norm("rms")), lambda: w8.block_norm(x),
              lambda: w8.block_norm(x, pre=w8.Norm("batch")), lambda: w8.block_norm(x, pre=w8.Norm("rms"), codes="fp8"),
              lambda: w8.block_norm(x, pre=w8.Norm("rms"), gate=b), lambda: w8.block_norm(x, x.double(), pre=w8.Norm("rms")),
              lambda: w8.block_norm(x, pre=w8.Norm("rms"), y=False), lambda: w8.block_norm(x, x, scale=b),
              lambda: w8.block_norm(x, x, gate=b.view(1, -1).expand(2, -1), pre=w8.Norm("rms"),
                                    scale=b.view(1, -1).expand(3, -1))):
        with pytest.raises(ValueError):
            f()
    for f in (lambda: w8.mx4_linear(x, w, b, workspace=ws[:16]), lambda: w8.mx4_quant(x, image=t.image[:16]),
              lambda: w8.mx4_quant(x[:, :40]), lambda: w8.block_norm(x, x, gate=b.expand(2, -1), rows_per_group=3)):
        with pytest.raises(w8.W8A8Error):
            f()


def test_offsets_past_32_bits():
    """Images, streams and codes of more than 2^32 bytes: their last rows equal those of a call on these alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    rows, K = 66000, 131072
    x = torch.randn(rows, K, device="cuda", generator=g, dtype=torch.bfloat16)
    assert w8.mx4_bytes(rows, K) > 1 << 32
    t = w8.mx4_quant(x)
    tail = slice(rows - 200, rows)
    want = w8.mx4_quant(x[tail])
    back = t.dequant()
    assert torch.equal(back[tail], want.dequant()) and torch.equal(back[:100], w8.mx4_quant(x[:100]).dequant())
    del back
    w = w8.mx4_quant(torch.randn(16, K, device="cuda", generator=g).mul_(K ** -0.5).bfloat16())
    y = w8.mx4_scaled_mm(t, w)
    check_product(y[tail], want, w, None, w8.ACT_NONE)
    # as the right operand: many output columns
    a = w8.mx4_quant(x[:3])
    z = w8.mx4_scaled_mm(a, t)
    check_product(z[:, tail], a, want, None, w8.ACT_NONE)
    del x, t, y, z
    M, D = 300000, 8192
    x = torch.randn(M, D, device="cuda", generator=g, dtype=torch.bfloat16)
    n = w8.Norm("layer", bf(1 + 0.1 * np.random.default_rng(0).standard_normal(D)))
    tail = slice(M - 300, M)
    small = w8.block_norm(x[tail], x[tail].float(), pre=n, post=n, codes="int8", y=True)
    big = w8.block_norm(x, x.float(), pre=n, post=n, codes="int8", y=True)
    for name in ("residual", "y", "q", "a_scale"):
        assert torch.equal(getattr(big, name)[tail], getattr(small, name))


@pytest.mark.parametrize("M", [1, 20, 200])
def test_ends_of_the_range(M):
    """Sums past bf16 become infinities of their sign, products down to fp32's subnormals keep their value, a weight
    block with the NaN scale gives NaN in its column alone."""
    top = 6 * 2.0 ** 125  # 3e38 saturates: its block's scale is 2^125
    for xs, ws, want in ((3e38, 100.0, float("inf")), (3e38, -100.0, -float("inf")), (3e38, 1.0, top),
                         (2.0 ** -120, 1.0, 2.0 ** -120), (2.0 ** -100, 2.0 ** -30, 2.0 ** -130), (2.0 ** -133, 2.0 ** 100, 0.0)):
        x, w = (torch.zeros(n, 64, dtype=torch.bfloat16, device="cuda") for n in (M, 16))
        x[:, 5], w[:, 5] = xs, ws
        y = w8.mx4_linear(x, w8.mx4_quant(w))
        assert (y.double() == want).all()
    x, w, b = operands(M, M, 272, 528)
    codes, scales = w.unpack()
    y = w8.mx4_linear(x, w, b)
    scales[7, 3] = 255
    got = w8.mx4_linear(x, w8.mx4_pack(codes, scales), b)
    rest = [n for n in range(272) if n != 7]
    assert got[:, 7].isnan().all() and torch.equal(got[:, rest], y[:, rest])


def test_one_row_without_leading_sizes():
    x, w, b = operands(3, 1, 272, 528)
    v = x[0]
    assert torch.equal(w8.mx4_linear(v, w, b), w8.mx4_linear(x, w, b)[0])
    assert torch.equal(w8.mx4_quant(v).dequant(), w8.mx4_quant(x).dequant()[0])
    n = w8.Norm("layer")
    out, want = w8.block_norm(v, v.float(), pre=n, codes="int8"), w8.block_norm(x, x.float(), pre=n, codes="int8")
    assert torch.equal(out.residual, want.residual[0]) and torch.equal(out.q, want.q[0])
    assert torch.equal(out.a_scale, want.a_scale)


def test_pack_of_other_than_a_matrix_refused():
    codes, scales = (torch.zeros(2, 16, n, dtype=torch.uint8, device="cuda") for n in (8, 1))
    for c, s in ((codes, scales), (codes, scales[:, 0]), (codes[0, 0], scales[0, 0])):
        with pytest.raises(ValueError):
            w8.mx4_pack(c, s)


@pytest.mark.parametrize("width", [400, 404])
@pytest.mark.parametrize("M", [1, 5, 40])
def test_slices_at_any_element(M, width):
    """A start that is no 16-byte boundary, in a parent whose rows are on them and in one whose are not."""
    wide = sample(np.random.default_rng(M), M, width)
    x, w, b = wide[:, 4:276], *operands(1, 1, 272, 272)[1:]
    c = x.contiguous()
    offset = torch.empty(M * 272 + 4, dtype=torch.bfloat16, device="cuda")[4:].view(M, 272).copy_(c)
    n, mod = w8.Norm("layer"), wide[:1, 100:372].contiguous()
    want, stream = w8.block_norm(c, c.float(), gate=mod, pre=n, shift=mod, codes="int8"), w8.block_norm(c, c, gate=mod).residual
    codes, scales = w.unpack()
    for v in (x, offset):
        assert all(torch.equal(p, q) for p, q in zip(w8.mx4_quant(v).unpack(), w8.mx4_quant(c).unpack()))
        assert torch.equal(w8.mx4_linear(v, w, b), w8.mx4_linear(c, w, b))
        assert all(torch.equal(p, q) for p, q in zip(w8.mx4_linear_quant(v, w).unpack(), w8.mx4_linear_quant(c, w).unpack()))
        got = w8.block_norm(v, v.float(), gate=wide[0, 100:372], pre=n, shift=wide[:1, 100:372], codes="int8")
        assert torch.equal(got.residual, want.residual) and torch.equal(got.q, want.q) and torch.equal(got.a_scale, want.a_scale)
        assert torch.equal(w8.block_norm(v, v, gate=wide[:1, 100:372]).residual, stream)
    # a weight's rows cut out of a taller one
    lone = torch.empty(codes.numel() + 8, dtype=torch.uint8, device="cuda")[8:].view(codes.shape).copy_(codes)
    assert all(torch.equal(p, q) for p, q in zip(w8.mx4_pack(lone, scales).unpack(), (codes, scales)))


@pytest.mark.parametrize("M", [2, 40, 300])
def test_vectors_and_biases_that_the_kernel_ahead_writes_in_place(M):
    """Modulation, bias and rows in buffers that every step writes anew just before they are read, by kernels that start
    while the one ahead, and the reader of the old values before it, still run."""
    D, steps = 1040, 40
    rng = np.random.default_rng(M)
    cond = [sample(rng, 2, D) for _ in range(steps)]
    make = w8.MX4Linear.from_float(bf(rng.standard_normal((3 * D, D)) * D ** -0.5))
    layer = w8.mx4_quant(bf(rng.standard_normal((D, D)) * D ** -0.5))
    x, n = sample(rng, M, D), w8.Norm("layer")
    per = M // 2

    def step(c, mod, rows):
        make(c, out=mod)
        gate, scale, shift = mod.split(D, 1)
        a = w8.block_norm(x, x, gate=gate, pre=n, scale=scale, shift=shift, rows_per_group=per, codes="mx4")
        w8.mx4_dequant(a.mx4, out=rows)
        y = w8.mx4_linear(rows, layer, mod[1, D:2 * D])  # a bias from the same buffer
        return y, w8.mx4_quant(rows).dequant()

    mod = torch.empty(2, 3 * D, dtype=torch.bfloat16, device="cuda")
    rows = torch.empty(M, D, dtype=torch.bfloat16, device="cuda")
    got = [step(c, mod, rows) for c in cond]
    torch.cuda.synchronize()
    for c, pair in zip(cond, got):
        want = step(c, torch.empty_like(mod), torch.empty_like(rows))
        torch.cuda.synchronize()
        assert all(torch.equal(g, v) for g, v in zip(pair, want))


@pytest.mark.parametrize("M", [1, 4, 16, 17, 200])
def test_a_layer_in_place(M):
    """y over x, whole or shifted, however few the rows: the layer is that of quantisation and product."""
    K = 2048
    x, w, b = operands(M, M, K, K)
    want = w8.mx4_scaled_mm(w8.mx4_quant(x), w, b)
    for _ in range(20):
        v = x.clone()
        assert w8.mx4_linear(v, w, b, out=v).data_ptr() == v.data_ptr() and torch.equal(v, want)
        both = torch.zeros(2 * M + 40, K, dtype=torch.bfloat16, device="cuda")
        both[1:M + 1] = x
        w8.mx4_linear(both[1:M + 1], w, b, out=both[:M])
        assert torch.equal(both[:M], want) and not both[M + 1:].any()
        both[:M] = x
        image = both.view(torch.uint8).view(-1)[:w8.mx4_bytes(M, K)]
        t = w8.mx4_linear_quant(both[:M], w, b, image=image)
        assert all(torch.equal(p, q) for p, q in zip(t.unpack(), w8.mx4_quant(want).unpack()))
    layer = w8.MX4Linear(*w.unpack(), b)
    v = x.clone()
    assert torch.equal(layer(v, out=v), want)
    t = w8.mx4_quant(x)
    with pytest.raises(w8.W8A8Error, match="INVALID_ARG"):
        w8.mx4_scaled_mm_quant(t, w, b, image=t.image)


@pytest.mark.parametrize("M", [1, 16, 17])
def test_a_wide_layer_over_its_input(M):
    """More weight slabs than SMs: x is still read when the first outputs are stored."""
    N, K = 40960, 5120
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn(M, K, device="cuda", generator=g).bfloat16()
    w = w8.mx4_quant(torch.randn(N, K, device="cuda", generator=g).mul_(K ** -0.5).bfloat16())
    b = torch.randn(N, device="cuda", generator=g).bfloat16()
    want = w8.mx4_scaled_mm(w8.mx4_quant(x), w, b)
    for _ in range(5):
        buffer = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
        v = buffer.view(-1)[:M * K].view(M, K).copy_(x)
        assert torch.equal(w8.mx4_linear(v, w, b, out=buffer), want)


def test_calls_from_several_host_threads():
    """Four threads, each on a stream of its own, with layers, norms and codes that they share: every result is that of
    one thread, the first calls of each shape among them."""
    D, F = 656, 1296
    up, down, n, mod = layers(13, D, F)
    eight = w8.W8A8Linear.from_float(up.w.dequant())
    xs = [sample(np.random.default_rng(M), M, D) for M in (1, 9, 16, 18, 33, 70, 129, 400)]
    torch.cuda.synchronize()

    def work(x):
        out = block(x, x.float(), up, down, n, mod, -(-x.shape[0] // 2))
        q = w8.block_norm(x, pre=n, codes="int8")
        return out.residual, out.y, eight.apply_codes(q.q, q.a_scale), w8.mx4_quant(x).dequant()

    got, failed = {}, []

    def run(i):
        try:
            s = torch.cuda.Stream()
            with torch.cuda.stream(s):
                for r in range(12):
                    k = (i * 3 + r) % len(xs)
                    got[i, r] = (k, work(xs[k]))
            s.synchronize()
        except BaseException as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    want = [work(x) for x in xs]
    torch.cuda.synchronize()
    for k, outs in got.values():
        assert all(torch.equal(g, v) for g, v in zip(outs, want[k]))
