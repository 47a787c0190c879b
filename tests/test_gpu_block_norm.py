"""GPU tests of the fused norms around a block against the plain form in 64 bits."""
import numpy as np
import pytest
import torch

import w8a8_int8_dynamic_b200 as w8
from gpu_util import require_gpu
from w8a8_int8_dynamic_b200.binding import _raw_stream, lib
from w8a8_int8_dynamic_b200.norms import _ARGS

pytestmark = pytest.mark.gpu

U = 2.0 ** -24                                   # a rounding in fp32, relative
HALF = torch.finfo(torch.bfloat16).eps / 2
#: roundings on the longest way through the kernel's sum over a row: 64 elements of a lane one after
#: another, 5 shuffles, 16 warps, the factor 1/K and its own rounding
DEPTH = 64 + 5 + 16 + 2


@pytest.fixture(autouse=True)
def _gpu():
    require_gpu()
    yield
    assert w8.poll_status() == 0


def f64(t):
    return None if t is None else t.double().cpu().numpy()


def norm64(t, n):
    """(norm of t, bound on the fp32 kernel's error): the sums' roundings, those of the differences and
    products, and two ulps (2^-22) of the reciprocal root."""
    layer = n.kind == "layer"
    mean = t.mean(1, keepdims=True) if layer else np.zeros((len(t), 1))
    d = t - mean
    e_d = U * (DEPTH * np.abs(t).mean(1, keepdims=True) + np.abs(mean) + np.abs(d)) if layer else np.zeros_like(t)
    var = (d * d).mean(1, keepdims=True) + n.eps
    rel = (DEPTH + 2) * U / 2 + (np.abs(d) * e_d).mean(1, keepdims=True) / var + 2.0 ** -22
    z = d / np.sqrt(var)
    e_z = e_d / np.sqrt(var) + np.abs(z) * (rel + U)
    w = 1.0 if n.weight is None else f64(n.weight)
    b = 0.0 if n.bias is None else f64(n.bias)
    return z * w + b, np.abs(w) * e_z + 2 * U * (np.abs(z * w) + np.abs(b))


def rows(v, index, M):
    return 0.0 if v is None else f64(v).reshape(-1, v.shape[-1])[index]


def check(out, x, residual, kw, index):
    """The stream against the formula, then the output against the formula of the stream as it was stored."""
    t, err = f64(x), 0.0
    stream = t
    if residual is not None:
        if kw.get("post"):
            t, err = norm64(t, kw["post"])
        gate = 1.0 if kw.get("gate") is None else rows(kw["gate"], index, len(t))
        r = kw.get("residual_scale", 1.0) * f64(residual)
        want = r + gate * t
        err = np.abs(gate) * err + 2 * U * (np.abs(r) + np.abs(gate * t))
        got = f64(out.residual)
        half = HALF if residual.dtype == torch.bfloat16 else U
        assert (np.abs(got - want) <= err + half * (np.abs(want) + err)).all()
        stream = got
    if not kw.get("pre"):
        return
    h, err = norm64(stream, kw["pre"])
    s, sh = 1 + rows(kw.get("scale"), index, len(h)), rows(kw.get("shift"), index, len(h))
    want = h * s + sh
    err = np.abs(s) * err + 2 * U * (np.abs(h * s) + np.abs(sh))
    assert (np.abs(f64(out.y) - want) <= err + HALF * (np.abs(want) + err)).all()


def tensors(seed, M, K, groups=0, dtype=torch.bfloat16, mean=0.0):
    g = torch.Generator(device="cuda").manual_seed(seed)

    def n(*shape, std=1.0, m=0.0):
        return (torch.randn(*shape, device="cuda", generator=g) * std + m).bfloat16()

    x, r = n(M, K, m=mean), n(M, K, std=2.0).to(dtype)
    x[:, :: max(1, K // 7)] *= 10
    if M > 1:
        x[M // 2] = 0  # a row of zeros
    mod = n(groups, 3 * K, std=0.5).split(K, 1) if groups else (None,) * 3
    return x, r, (n(K, std=0.2, m=1.0), n(K, std=0.2)), (n(K, std=0.2, m=1.0), n(K, std=0.2)), mod


SHAPES = [(1, 8), (1, 5120), (3, 24), (5, 264), (7, 1000), (130, 2048), (33, 4104), (4, 12288), (2, 14336), (5, 10008)]


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_norm_before(M, K, kind):
    x, _, (w, b), _, (_, scale, shift) = tensors(M + K, M, K, groups=1, mean=3.0)
    for kw in ({}, {"scale": scale, "shift": shift}, {"shift": shift[0]}):
        kw["pre"] = w8.Norm(kind, w, b if kw else None, 1e-5)
        check(w8.block_norm(x, **kw), x, None, kw, np.zeros(M, int))


@pytest.mark.parametrize("M,K", SHAPES)
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_norms_around_the_residual(M, K, kind, dtype):
    groups = min(M, 3)
    x, r, (pw, pb), (w, b), (gate, scale, shift) = tensors(M * 3 + K, M, K, groups, dtype)
    per = -(-M // groups)
    kw = dict(post=w8.Norm(kind, pw, pb, 1e-6), gate=gate, residual_scale=0.7, pre=w8.Norm(kind, w, b, 1e-6),
              scale=scale, shift=shift, rows_per_group=per)
    check(w8.block_norm(x, r, **kw), x, r, kw, np.arange(M) // per)
    # each part alone
    for kw in ({}, {"gate": gate, "rows_per_group": per}, {"post": w8.Norm(kind, pw)}, {"pre": w8.Norm(kind)}):
        out = w8.block_norm(x, r, **kw)
        check(out, x, r, kw, np.arange(M) // per)
        assert (out.y is None) == ("pre" not in kw)


@pytest.mark.parametrize("M,K", [(1, 16), (1, 5120), (5, 272), (129, 1040), (300, 2048), (3, 12288), (2, 14336), (1200, 64)])
@pytest.mark.parametrize("codes", ["int8", "mx4"])
def test_codes_are_those_of_the_output(M, K, codes):
    x, r, (pw, _), (w, b), (gate, scale, shift) = tensors(M + 5 * K, M, K, 1)
    kw = dict(post=w8.Norm("rms", pw), gate=gate, pre=w8.Norm("layer", w, b), scale=scale, shift=shift, codes=codes)
    out = w8.block_norm(x, r, y=True, **kw)
    assert torch.equal(out.y, w8.block_norm(x, r, **{**kw, "codes": None}).y)
    alone = w8.block_norm(x, r, **kw)
    assert alone.y is None
    if codes == "int8":
        q, s = w8.quant_act(out.y)
        for o in (out, alone):
            assert torch.equal(o.q, q) and torch.equal(o.a_scale, s)
    else:
        want = w8.mx4_quant(out.y)
        for o in (out, alone):
            # to the end of the last tile: its padding is zeros
            padded = -(-K // 256) * 256
            for g, v in zip(w8.MX4Tensor(o.mx4.image, (M,), padded).unpack(),
                            w8.MX4Tensor(want.image, (M,), padded).unpack()):
                assert torch.equal(g, v)


def test_rows_of_zeros_infinities_and_nan():
    x, r, _, (w, b), _ = tensors(9, 6, 512)
    x[1], x[2, 5], x[3, 6] = 0, float("inf"), float("nan")
    clean = [0, 1, 4, 5]
    for kind in ("rms", "layer"):
        n = w8.Norm(kind, w, b)
        out = w8.block_norm(x, pre=n, y=True, codes="mx4")
        ok = w8.block_norm(x[clean], pre=n)
        assert torch.equal(out.y[clean], ok.y)
        assert out.y[3].isnan().all() and out.y[2].isnan().any()
        assert torch.isfinite(out.y[1]).all()
        assert out.mx4.dequant()[3].isnan().all()


def test_group_index_and_padding_rows():
    M, K, groups = 37, 1040, 4
    x, r, (pw, _), (w, _), (gate, scale, shift) = tensors(11, M, K, groups)
    index = torch.randint(0, groups, (M,), dtype=torch.int32, device="cuda")
    skip = [0, 17, 36]
    index[skip[0]], index[skip[1]], index[skip[2]] = -1, groups, 2 ** 31 - 1
    keep = [m for m in range(M) if m not in skip]
    kw = dict(post=w8.Norm("rms", pw), gate=gate, pre=w8.Norm("layer", w), scale=scale, shift=shift)
    stream = r.clone()
    out = w8.block_norm(x, stream, residual_out=stream, group_index=index, codes="mx4", y=True, **kw)
    assert out.residual.data_ptr() == stream.data_ptr()
    assert torch.equal(stream[skip], r[skip])
    for g in range(groups):
        at = [m for m in keep if index[m] == g]
        if not at:
            continue
        one = w8.block_norm(x[at], r[at], **{**kw, "gate": gate[g], "scale": scale[g], "shift": shift[g]})
        assert torch.equal(stream[at], one.residual) and torch.equal(out.y[at], one.y)
    # an image given rows to leave alone: the other rows' codes are those of y
    c, s = out.mx4.unpack()
    cw, sw = w8.mx4_quant(out.y).unpack()
    assert torch.equal(c[keep], cw[keep]) and torch.equal(s[keep], sw[keep])


@pytest.mark.parametrize("M,K", [(1500, 264), (700, 1040), (400, 4104), (350, 10248), (350, 12304)])
def test_many_rows_with_a_group_and_padding_each(M, K):
    """Several rows a CTA, groups that change and recur, padding rows between them, one norm or both."""
    groups = 7
    x, r, (pw, pb), (w, b), (gate, scale, shift) = tensors(M, M, K, groups)
    index = torch.randint(-1, groups + 1, (M,), dtype=torch.int32, device="cuda")
    index[100:200] = 3
    index[-40:] = -1
    keep = ((index >= 0) & (index < groups)).nonzero().flatten()
    for kw in (dict(post=w8.Norm("layer", pw, pb), gate=gate, pre=w8.Norm("rms", w), scale=scale, shift=shift),
               dict(pre=w8.Norm("layer", w, b), scale=scale), dict(gate=gate), dict(post=w8.Norm("rms"), gate=gate)):
        stream = torch.full_like(r, 7.0)
        out = w8.block_norm(x, r, residual_out=stream, group_index=index, **kw)
        some = type(out)(*(t[keep] if torch.is_tensor(t) else t for t in out))
        check(some, x[keep], r[keep], kw, index[keep].cpu().numpy())
        skipped = torch.ones(M, dtype=torch.bool, device="cuda")
        skipped[keep] = False
        assert (stream[skipped] == 7.0).all()


def test_strides_and_leading_sizes():
    x, r, _, (w, _), _ = tensors(13, 24, 528)
    n = w8.Norm("rms", w)
    want = w8.block_norm(x, r, pre=n)
    wide_x, wide_r = torch.zeros(24, 1000, dtype=torch.bfloat16, device="cuda"), torch.zeros(24, 800, device="cuda")
    wide_x[:, 8:536], wide_r[:, 4:532] = x, r.float()
    got = w8.block_norm(wide_x[:, 8:536], wide_r[:, 4:532], residual_out=wide_r[:, 4:532], pre=n)
    assert torch.equal(wide_r[:, 4:532].bfloat16(), want.residual)
    assert not wide_r[:, :4].any() and not wide_r[:, 532:].any()
    shaped = w8.block_norm(x.view(2, 3, 4, 528), r.view(2, 3, 4, 528), pre=n, codes="int8", y=True)
    assert shaped.residual.shape == shaped.y.shape == shaped.q.shape == (2, 3, 4, 528)
    assert torch.equal(shaped.y.view(24, 528), want.y) and got.y.shape == (24, 528)
    assert w8.block_norm(x[:0], r[:0], pre=n, codes="mx4").residual.shape == (0, 528)


def test_group_index_without_vectors_leaves_only_negative_rows():
    M, K = 23, 272
    x, r, (pw, _), (w, _), _ = tensors(17, M, K)
    index = torch.arange(M, dtype=torch.int32, device="cuda") * 1000
    index[4] = index[22] = -3
    keep = [m for m in range(M) if m not in (4, 22)]
    kw = dict(post=w8.Norm("rms", pw), pre=w8.Norm("rms", w))
    want, stream = w8.block_norm(x, r, **kw), r.clone()
    out = w8.block_norm(x, stream, residual_out=stream, group_index=index, **kw)
    assert torch.equal(stream[keep], want.residual[keep]) and torch.equal(out.y[keep], want.y[keep])
    assert torch.equal(stream[[4, 22]], r[[4, 22]])


def test_no_groups_refused():
    x, r, _, _, (gate, scale, shift) = tensors(19, 5, 272, 3)
    index = torch.zeros(5, dtype=torch.int32, device="cuda")
    n = w8.Norm("rms")
    for kw in (dict(gate=gate[:0]), dict(gate=gate[:0], pre=n, scale=scale), dict(pre=n, shift=shift[:0])):
        for i in (None, index):
            with pytest.raises(ValueError, match="groups"):
                w8.block_norm(x, r, group_index=i, **kw)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("M,K", [(3700, 4096), (3700, 3600), (2500, 5120), (1300, 6160), (700, 8208), (20, 4112)])
def test_y_alone_and_codes_alone_agree(M, K, dtype):
    """However many rows: the codes of one call are those of another call's y."""
    x, r, (pw, pb), (w, b), (gate, scale, shift) = tensors(M + K, M, K, 2, dtype)
    kw = dict(post=w8.Norm("rms", pw, pb), gate=gate, pre=w8.Norm("layer", w, b), scale=scale, shift=shift,
              rows_per_group=M // 2 + 1)
    y = w8.block_norm(x, r, **kw)
    four, eight = w8.block_norm(x, r, codes="mx4", **kw), w8.block_norm(x, r, codes="int8", **kw)
    assert torch.equal(four.residual, y.residual) and torch.equal(eight.residual, y.residual)
    assert all(torch.equal(p, q) for p, q in zip(four.mx4.unpack(), w8.mx4_quant(y.y).unpack()))
    q, s = w8.quant_act(y.y)
    assert torch.equal(eight.q, q) and torch.equal(eight.a_scale, s)


def test_vectors_of_no_norm_are_not_looked_at():
    """The C call with kind NONE and a weight, bias and eps beside it: u is x, whatever they hold."""
    M, K = 5, 272
    x, r, (w, b), _, (gate, _, _) = tensors(23, M, K, 1)
    want = w8.block_norm(x, r, gate=gate)
    out = torch.empty_like(r)
    for weight, bias in ((w.data_ptr(), 0), (0, b.data_ptr()), (w.data_ptr(), b.data_ptr()), (2, 2)):
        norm = (0, float("nan"), weight, bias)
        args = _ARGS.pack(M, K, x.data_ptr(), K, r.data_ptr(), out.data_ptr(), K, K, 0, 1.0, *norm, *norm,
                          gate.data_ptr(), 0, 0, K, 0, 0, 1, M, 0, 0, 0, 0, 0, 0, 0)
        assert lib().w8a8_block_norm(args, _raw_stream(0)) == 0
        assert torch.equal(out, want.residual)


@pytest.mark.parametrize("K", [264, 1000, 5120, 14336])
def test_layer_norm_of_rows_far_from_zero(K):
    """A mean whose square is no float: the squares that the norm takes are of the differences."""
    g = torch.Generator(device="cuda").manual_seed(K)
    x = ((1 + torch.randint(0, 2, (5, K), device="cuda", generator=g) / 128) * 2.0 ** 65).bfloat16()
    x[1] *= -1
    kw = dict(pre=w8.Norm("layer", eps=1e-6))
    check(w8.block_norm(x, **kw), x, None, kw, np.zeros(5, int))


@pytest.mark.parametrize("K", [8, 24, 1000, 4104, 5120, 8200, 12304, 14336])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_layer_norm_of_constant_rows_is_the_bias(K, dtype):
    """The sum of a row of equal bf16 values is exact in fp32 (8 bits and 14 of the count), so is its mean: nothing is
    left for 1 / sqrt(eps) to enlarge, before the block or after it."""
    values = torch.tensor([1000.0, -3.140625, 0.01, 57344.0, 1 / 3, 1e4, 0.0, -2.0 ** 100], device="cuda").bfloat16()
    rows = values.view(-1, 1).repeat(1, K)
    _, r, (w, b), _, _ = tensors(K, len(values), K)
    n = w8.Norm("layer", w, b, 1e-6)
    for out in (w8.block_norm(rows, pre=n), w8.block_norm(torch.zeros_like(rows), rows.to(dtype), pre=n)):
        assert torch.equal(out.y, b.expand_as(rows))
    r = r.to(dtype)
    assert torch.equal(w8.block_norm(rows, r, post=w8.Norm("layer", w, eps=1e-6)).residual, r)


@pytest.mark.parametrize("codes", [None, "int8", "mx4"])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_outputs_of_strided_inputs(codes, dtype):
    """Rows of a wider tensor, a transposed one and a row repeated: every output is dense and that of contiguous copies."""
    M, K = 24, 528
    x, r, _, (w, _), (gate, _, _) = tensors(29, M, K, 1, dtype)
    n = w8.Norm("layer", w)
    wide_x = torch.zeros(M, 1000, dtype=torch.bfloat16, device="cuda")
    wide_r = torch.zeros(M, 800, dtype=dtype, device="cuda")
    wide_x[:, 8:536], wide_r[:, 16:544] = x, r
    for xs, rs in ((wide_x[:, 8:536], wide_r[:, 16:544]), (x, wide_r[:, 16:544]), (wide_x[:, 8:536], r),
                   (x.t().contiguous().t(), r.t().contiguous().t()), (x[:1].expand(M, K), r[:1].expand(M, K)),
                   (wide_x.view(4, 6, 1000)[..., 8:536], wide_r.view(4, 6, 800)[..., 16:544])):
        kw = dict(gate=gate, pre=n, codes=codes, y=True)
        got, want = w8.block_norm(xs, rs, **kw), w8.block_norm(xs.contiguous(), rs.contiguous(), **kw)
        for name in ("residual", "y", "q", "a_scale"):
            g, v = getattr(got, name), getattr(want, name)
            assert (g is None) == (v is None) and (v is None or g.is_contiguous() and torch.equal(g, v)), name
        if codes == "mx4":
            assert all(torch.equal(g, v) for g, v in zip(got.mx4.unpack(), want.mx4.unpack()))
        assert torch.equal(w8.block_norm(xs, pre=n).y, w8.block_norm(xs.contiguous(), pre=n).y)


@pytest.mark.parametrize("M,K", [(3, 16384), (2, 15008), (300, 16384), (170, 14352), (160, 12304)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_longest_rows(M, K, dtype):
    """To K = 16384 with three of a group's vectors, one row a CTA and several, and the codes of such rows."""
    x, r, (pw, pb), (w, b), (gate, scale, shift) = tensors(M + K, M, K, 2, dtype)
    per = -(-M // 2)
    for kw in (dict(post=w8.Norm("rms", pw), gate=gate, pre=w8.Norm("layer", w, b), scale=scale, shift=shift, rows_per_group=per),
               dict(post=w8.Norm("layer", pw, pb), gate=gate, pre=w8.Norm("rms", w), rows_per_group=per)):
        out = w8.block_norm(x, r, **kw)
        check(out, x, r, kw, np.arange(M) // per)
        eight, four = w8.block_norm(x, r, codes="int8", **kw), w8.block_norm(x, r, codes="mx4", **kw)
        q, s = w8.quant_act(out.y)
        assert torch.equal(eight.q, q) and torch.equal(eight.a_scale, s)
        assert all(torch.equal(g, v) for g, v in zip(four.mx4.unpack(), w8.mx4_quant(out.y).unpack()))
    if K > 14336:  # a fourth vector does not fit beside them
        with pytest.raises(w8.W8A8Error, match="UNSUPPORTED_SHAPE"):
            w8.block_norm(x, r, post=w8.Norm("rms", pw, pb), pre=w8.Norm("rms", w, b))


@pytest.mark.parametrize("M", [1, 5, 2500])
def test_the_stream_over_its_inputs(M):
    """residual_out as residual, as x, and as columns or rows beside them; other overlaps are refused."""
    K, wide = 272, 800
    x, r, (pw, _), (w, _), (gate, _, _) = tensors(31, M, K, 1)
    kw = dict(post=w8.Norm("layer", pw), gate=gate, residual_scale=0.7, pre=w8.Norm("rms", w))
    want = w8.block_norm(x, r, **kw)
    buffer = torch.zeros(M, wide, dtype=torch.bfloat16, device="cuda")
    for a, b in ((0, 0), (0, 272), (0, 528), (528, 0), (272, 0)):
        buffer.zero_()
        buffer[:, a:a + K] = r
        out = w8.block_norm(x, buffer[:, a:a + K], residual_out=buffer[:, b:b + K], **kw)
        assert torch.equal(buffer[:, b:b + K], want.residual) and torch.equal(out.y, want.y)
        assert a == b or torch.equal(buffer[:, a:a + K], r)
    over = x.clone()
    out = w8.block_norm(over, r, residual_out=over, **kw)
    assert torch.equal(over, want.residual) and torch.equal(out.y, want.y)
    line = torch.zeros(3 * M, K, dtype=torch.bfloat16, device="cuda")
    line[M:2 * M] = r
    for at in (0, 2 * M):  # rows ahead and behind
        w8.block_norm(x, line[M:2 * M], residual_out=line[at:at + M], **kw)
        assert torch.equal(line[at:at + M], want.residual) and torch.equal(line[M:2 * M], r)
    refused = [(buffer[:, :K], buffer[:, 8:8 + K]), (buffer[:, 8:8 + K], buffer[:, :K])]
    if M > 1:
        refused += [(line[1:M + 1], line[:M]), (line[:M], line[1:M + 1]), (buffer[:, :K], buffer.view(-1)[:M * K].view(M, K))]
    for a, b in refused:
        with pytest.raises(w8.W8A8Error, match="INVALID_ARG"):
            w8.block_norm(x, a, residual_out=b, **kw)


def test_int8_codes_of_rows_at_the_ends_of_the_range():
    """Codes and scales of the output as quant_act forms them, bit for bit: NaN and infinite rows, zeros, scales below 1e-30."""
    x, _, _, (w, b), _ = tensors(37, 8, 1040)
    x[1, 3], x[2, 5], x[3] = float("nan"), float("inf"), 0
    x[4] *= 2.0 ** -40
    x[5] *= 2.0 ** -100
    for kw in (dict(pre=w8.Norm("rms", w, eps=1e-2)), dict(pre=w8.Norm("layer", w, b)),
               dict(pre=w8.Norm("rms", (w.double() * 2.0 ** -110).bfloat16())), dict(pre=w8.Norm("rms", w * 1e30))):
        out = w8.block_norm(x, y=True, codes="int8", **kw)
        q, s = w8.quant_act(out.y)
        assert torch.equal(out.q, q) and torch.equal(out.a_scale.view(torch.int32), s.view(torch.int32))


@pytest.mark.parametrize("codes", ["int8", "mx4"])
def test_outputs_of_one_row_of_a_wider_tensor(codes):
    """A lone row's stride may be any, and its tensor still counts as contiguous: the outputs' strides are those of dense
    rows, which the next call takes."""
    K = 272
    x, r, _, (w, _), _ = tensors(41, 1, K)
    want = w8.block_norm(x, r, pre=w8.Norm("rms", w), codes=codes, y=True)
    for width in (276, 299, 400):
        wx, wr = (torch.zeros(1, width, dtype=t.dtype, device="cuda")[:, :K].copy_(t) for t in (x, r))
        assert wx.stride() == (width, 1)
        got = w8.block_norm(wx, wr, pre=w8.Norm("rms", w), codes=codes, y=True)
        for g, v in zip((got.residual, got.y, got.q), (want.residual, want.y, want.q)):
            assert v is None or g.stride() == (K, 1) and torch.equal(g, v)
        q, s = w8.quant_act(got.y)
        if codes == "int8":
            assert torch.equal(q, got.q) and torch.equal(s, got.a_scale)
