"""The 4-bit layers and the block norm on the host, without a GPU: what the C entry points refuse before any
CUDA call, their sizes, what the binding refuses, and the test suite's own 64-bit reference pinned to the format."""
import ctypes
import struct

import numpy as np
import pytest
import torch

import mx4_ref as ref

FAKE = ctypes.c_void_p(1 << 20)        # never dereferenced: checks fail first
FAKE_MIS = ctypes.c_void_p((1 << 20) + 4)
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    from w8a8_int8_dynamic_b200 import build
    build.build()
    from w8a8_int8_dynamic_b200 import binding
    return binding.lib()


def calls(f, ok):
    """f with every argument of `ok` but those given by position (a3=...)."""
    def call(**kw):
        a = list(ok)
        for i, v in kw.items():
            a[int(i[1:])] = v
        return f(*a)
    return call


def test_image_bytes(L):
    out = ctypes.c_size_t()
    for rows, K, tiles in [(1, 16, 1), (128, 256, 1), (129, 256, 2), (128, 272, 2), (27648, 5120, 216 * 20)]:
        assert L.w8a8_mx4_bytes(rows, K, ctypes.byref(out)) == 0 and out.value == tiles * 17408
    assert L.w8a8_mx4_bytes(1, 24, ctypes.byref(out)) == 3
    assert L.w8a8_mx4_bytes(1, 131072 + 16, ctypes.byref(out)) == 3
    assert L.w8a8_mx4_bytes(0, 16, ctypes.byref(out)) == 1
    assert L.w8a8_mx4_bytes(1 << 31, 16, ctypes.byref(out)) == 1
    assert L.w8a8_mx4_bytes(1, 16, None) == 1


def test_quant_pack_unpack_dequant_refuse(L):
    q = calls(L.w8a8_mx4_quant, (FAKE, 4, 32, 32, FAKE, BIG, None))
    assert q(a0=None) == q(a4=None) == q(a1=0) == q(a1=-1) == q(a3=16) == q(a1=1 << 31) == 1
    assert q(a2=24, a3=24) == q(a2=1 << 18, a3=1 << 18) == 3
    assert q(a0=FAKE_MIS) == q(a4=FAKE_MIS) == q(a3=36) == 2
    assert q(a5=17407) == 6
    p = calls(L.w8a8_mx4_pack, (FAKE, FAKE, 4, 32, FAKE, BIG, None))
    assert p(a0=None) == p(a1=None) == p(a4=None) == p(a2=0) == 1
    assert p(a3=40) == 3 and p(a0=FAKE_MIS) == p(a4=FAKE_MIS) == 2 and p(a5=100) == 6
    u = calls(L.w8a8_mx4_unpack, (FAKE, 4, 32, FAKE, FAKE, None))
    assert u(a0=None) == u(a3=None) == u(a4=None) == u(a1=0) == 1 and u(a2=8) == 3 and u(a0=FAKE_MIS) == 2
    d = calls(L.w8a8_mx4_dequant, (FAKE, 4, 32, FAKE, None))
    assert d(a0=None) == d(a3=None) == d(a1=0) == 1 and d(a2=8) == 3 and d(a3=FAKE_MIS) == 2


def test_products_refuse(L):
    y = calls(L.w8a8_mx4_scaled_mm, (FAKE, FAKE, None, FAKE, 4, 8, 32, 0, None))
    assert y(a0=None) == y(a1=None) == y(a3=None) == y(a4=0) == y(a5=0) == y(a6=0) == y(a7=2) == y(a7=-1) == 1
    assert y(a5=12) == y(a6=40) == y(a6=1 << 18) == 3
    assert y(a0=FAKE_MIS) == y(a1=FAKE_MIS) == y(a2=FAKE_MIS) == y(a3=FAKE_MIS) == 2
    i = calls(L.w8a8_mx4_scaled_mm_quant, (FAKE, FAKE, None, FAKE, BIG, 4, 16, 32, 0, None))
    assert i(a3=None) == i(a5=0) == 1
    assert i(a6=24) == i(a6=131072 + 16) == 3   # the next product's K
    assert i(a3=FAKE_MIS) == 2 and i(a4=17407) == 6
    n = calls(L.w8a8_mx4_linear, (FAKE, 32, FAKE, None, FAKE, 20, 8, 32, 0, FAKE, BIG, None))
    assert n(a0=None) == n(a1=16) == n(a2=None) == n(a4=None) == n(a8=3) == 1
    assert n(a6=4) == n(a7=24) == 3
    assert n(a0=FAKE_MIS) == n(a1=36) == n(a9=FAKE_MIS) == 2
    assert n(a9=None) == n(a10=17407) == 6
    m = calls(L.w8a8_mx4_linear_quant, (FAKE, 32, FAKE, None, FAKE, BIG, 20, 16, 32, 0, FAKE, BIG, None))
    assert m(a4=None) == 1 and m(a7=8) == 3 and m(a5=1) == m(a11=1) == 6
    out = ctypes.c_size_t()
    for M, want in [(1, 0), (16, 0), (17, 2 * 17408), (200, 4 * 17408)]:
        assert L.w8a8_mx4_linear_workspace_bytes(M, 64, 512, ctypes.byref(out)) == 0 and out.value == want
    assert L.w8a8_mx4_linear_workspace_bytes(1, 4, 32, ctypes.byref(out)) == 3
    assert L.w8a8_mx4_linear_workspace_bytes(1, 8, 32, None) == 1


def test_block_norm_refuses(L):
    from w8a8_int8_dynamic_b200.norms import _ARGS
    fields = ("M K x ldx residual residual_out ldr ldro dtype rscale post post_eps post_w post_b pre pre_eps pre_w pre_b "
              "gate scale shift ld_gate ld_scale ld_shift groups rows index y ldy q a_scale image image_bytes").split()
    A, MIS = 1 << 20, (1 << 20) + 4
    ok = dict.fromkeys(fields, 0) | dict(M=4, K=64, x=A, ldx=64, residual=A, residual_out=A, ldr=64, ldro=64, rscale=1.0,
                                         post=1, post_eps=1e-6, pre=2, pre_eps=1e-6, gate=A, scale=A, shift=A, ld_gate=64,
                                         ld_scale=64, ld_shift=64, groups=2, rows=2, y=A, ldy=64)
    assert _ARGS.size == struct.calcsize("@" + "q" * 30)

    def call(**kw):
        return L.w8a8_block_norm(_ARGS.pack(*(ok | kw).values()), None)

    assert L.w8a8_block_norm(None, None) == 1
    assert call(x=0) == call(M=0) == call(K=0) == call(ldx=63) == call(post=3) == call(pre=-1) == 1
    assert call(pre_eps=0.0) == call(pre_eps=float("nan")) == call(post_eps=float("inf")) == call(post_eps=-1.0) == 1
    assert call(residual_out=0) == call(residual=0, residual_out=0) == call(dtype=2) == call(ldr=32) == call(ldro=32) == 1
    assert call(y=0) == call(pre=0) == call(y=0, pre=0) == call(ldy=32) == call(q=A) == call(a_scale=A) == 1
    assert call(groups=0) == call(rows=0) == call(rows=1) == call(groups=1) == 1     # 2 groups of 2 rows are 4
    assert call(index=A, groups=0) == 1
    assert call(ld_gate=32) == call(ld_scale=-64) == 1
    assert call(K=16392, ldx=16392, ldr=16392, ldro=16392, ldy=16392, ld_gate=16392, ld_scale=16392, ld_shift=16392) == 3
    assert call(K=60) == call(K=56, image=A, image_bytes=BIG) == call(K=56, q=A, a_scale=A) == 3
    wide = dict(K=14400, **dict.fromkeys("ldx ldr ldro ldy ld_gate ld_scale ld_shift".split(), 14400))
    assert call(**wide, post_b=A) == 3                                               # four vectors of a group
    for name in "x residual residual_out y gate scale shift post_w post_b pre_w pre_b".split():
        assert call(**{name: MIS}) == 2, name
    assert call(q=MIS, a_scale=A) == call(q=A, a_scale=MIS) == call(image=MIS) == call(index=A + 2) == 2
    assert call(ldx=68) == call(ldr=68) == call(ldro=68) == call(ldy=68) == call(ld_gate=68) == 2
    assert call(dtype=1, ldr=66) == 2
    assert call(image=A, image_bytes=17407) == 6


def test_binding_refuses_host_tensors_and_wrong_shapes():
    import w8a8_int8_dynamic_b200 as w8
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    n = w8.Norm("rms")
    for f in (lambda: w8.mx4_quant(x), lambda: w8.block_norm(x, pre=n), lambda: w8.MX4Linear.from_float(x),
              lambda: w8.mx4_pack(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8)),
              lambda: w8.mx4_dequant(w8.MX4Tensor(torch.zeros(17408, dtype=torch.uint8), (4,), 64)),
              lambda: w8.MX4Tensor(torch.zeros(100, dtype=torch.uint8), (4,), 64).unpack(),   # too small
              lambda: w8.mx4_linear(x, w8.MX4Tensor(torch.zeros(17408, dtype=torch.uint8), (8,), 64))):
        with pytest.raises(ValueError):
            f()


def test_reference_pins():
    """The format's worked values: the grid, ties to the even code, saturation, block scales, signs of zeros."""
    x = np.zeros((1, 64))
    x[0, :16] = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.0, -0.25, -0.75, -5.0, 0.26, 0.74, 4.9, 5.1, -0.0]
    codes, scales = ref.encode(x)
    assert scales.tolist() == [[127, 0]]                       # amax 7: floor(log2 7) - 2 = 0; a block of zeros
    assert codes[0, :16].tolist() == [0, 2, 2, 4, 4, 6, 6, 7, 8, 10, 14, 1, 1, 6, 7, 8]
    assert ref.values(codes, scales)[0, :8].tolist() == [0, 1, 1, 2, 2, 4, 4, 6]
    for amax, scale in [(1.0, 125), (1.99, 125), (2.0, 126), (2.0 ** -133, 0), (2.0 ** -125, 0), (2.0 ** -124, 1),
                        (2.0 ** 127, 252)]:
        x = np.zeros((1, 32))
        x[0, 7] = -amax
        assert ref.encode(x)[1].tolist() == [[scale]]
    x = np.zeros((1, 96))
    x[0, 3], x[0, 40] = np.inf, np.nan
    codes, scales = ref.encode(x)
    assert scales.tolist() == [[255, 255, 0]] and not codes.any()
    assert np.isnan(ref.values(codes, scales)[0, :64]).all()
    r = np.random.default_rng(0).integers(0, 256, (3, 8)).astype(np.uint8)
    assert np.array_equal(ref.pack_codes(ref.unpack_codes(r)), r)
    # a value between neighbours goes to the nearer one, for every pair of neighbours
    for lo, hi in zip(ref.GRID[:-1], ref.GRID[1:]):
        x = np.zeros((1, 32))
        x[0, 0], x[0, 1], x[0, 2] = 4.0, lo + 0.49 * (hi - lo), lo + 0.51 * (hi - lo)
        assert ref.values(*ref.encode(x))[0, 1:3].tolist() == [lo, hi]


def test_vectors_of_several_groups_need_a_grouping():
    import w8a8_int8_dynamic_b200 as w8
    x, v = torch.zeros(6, 64, dtype=torch.bfloat16), torch.zeros(2, 64, dtype=torch.bfloat16)
    n = w8.Norm("rms")
    for kw in (dict(gate=v), dict(pre=n, scale=v), dict(pre=n, shift=v), dict(gate=v[:1], pre=n, scale=v)):
        with pytest.raises(ValueError, match="rows_per_group or group_index"):
            w8.block_norm(x, x, **kw)
    # what has a grouping, or needs none, goes on to the next check
    for kw in (dict(gate=v, rows_per_group=3), dict(gate=v, group_index=torch.zeros(6, dtype=torch.int32)), dict(gate=v[:1]),
               dict(gate=v[0])):
        with pytest.raises(ValueError, match="CUDA tensor"):
            w8.block_norm(x, x, **kw)


def test_rows_are_on_16_byte_boundaries_whatever_the_slice():
    """What the calls hand to the library: the tensor itself where that is possible, else a copy."""
    from w8a8_int8_dynamic_b200.binding import _rows_of
    base = torch.randn(13 * 48 * 8).bfloat16()
    assert base.data_ptr() % 16 == 0
    for width in (40, 44, 48):
        wide = base[:6 * 2 * width].view(6, 2, width)
        for x, same in ((wide[..., :40], None), (wide[:, 0, :40], None), (wide[:, 0, 4:36], False), (wide[:, 1, 8:40], None),
                        (wide[2:3, 1, 4:36], None), (base[4:132].view(4, 32), False), (base[8:136].view(4, 32), True),
                        (wide[..., 0:32:2], False), (wide[:, :, 4:36], False), (base[:32].expand(3, 32), False)):
            x2, rows, ld = _rows_of(x)
            assert x2.data_ptr() % 16 == 0 and (rows == 1 or ld % 8 == 0) and x2.stride(-1) == 1
            K = x.shape[-1]
            assert rows == x.numel() // K and ld >= K
            got = torch.as_strided(x2, (rows, K), (ld, 1), x2.storage_offset())
            assert torch.equal(got, x.reshape(rows, K))
            if same is not None:
                assert (x2.data_ptr() == x.data_ptr()) == same


def test_kernels_that_start_early_read_through_the_coherent_path():
    """A kernel with a wait for the one ahead runs while that one still writes what it will read: __ldg, ld.global.nc and
    const __restrict__ parameters promise memory that nothing writes while the kernel runs."""
    import os
    import re
    from w8a8_int8_dynamic_b200 import build
    seen = 0
    for name in ("block_norm.cu", "mx4_common.cuh", "mx4_gemm.cu", "mx4_pair.cu", "mx4_quant.cu", "mx4_stream.cu"):
        text = re.sub(r"//[^\n]*", "", open(os.path.join(build.CSRC, name)).read())
        assert not re.search(r"\b__ldg\s*\(|global\.nc|ld_stream_u4", text), name
        for kernel in re.split(r"(?=__global__)", text)[1:]:
            head, body = kernel.split("{", 1)
            if "griddep_wait" in body:
                seen += 1
                assert "__restrict__" not in head, (name, head)
            else:
                assert "griddep_launch_dependents" not in body, (name, head)
    assert seen == 6


def test_products_refuse_outputs_over_their_inputs(L):
    """Host checks alone: none of these addresses is one of memory, and every call is refused."""
    A, W, B, Y, WS = (ctypes.c_void_p(n << 24) for n in range(1, 6))
    M, N, K = 20, 256, 512
    image = 2 * 17408                                            # of x
    inputs = [(A, image), (W, 4 * 17408), (B, 512)]
    y = calls(L.w8a8_mx4_scaled_mm, (A, W, B, Y, M, N, K, 0, None))
    i = calls(L.w8a8_mx4_scaled_mm_quant, (A, W, B, Y, BIG, M, N, K, 0, None))
    for at, size in inputs:
        for end in (at.value, at.value + size - 16):
            assert y(a3=ctypes.c_void_p(end)) == i(a3=ctypes.c_void_p(end)) == 1
        assert y(a3=ctypes.c_void_p(at.value - M * N * 2 + 16)) == i(a3=ctypes.c_void_p(at.value - 17408 + 16)) == 1
    n = calls(L.w8a8_mx4_linear, (A, K, W, B, Y, M, N, K, 0, WS, BIG, None))
    m = calls(L.w8a8_mx4_linear_quant, (A, K, W, B, Y, BIG, M, N, K, 0, WS, BIG, None))
    for at in (W, B):
        assert n(a4=at) == m(a4=at) == n(a4=at, a5=4) == m(a4=at, a6=4) == 1
    for at in (A, Y):
        assert n(a9=at) == m(a10=at) == 1
    # few rows in place need the image of x
    assert n(a4=A, a5=4, a9=None) == m(a4=A, a6=4, a10=None) == n(a4=A, a5=4, a10=image - 1) == m(a4=A, a6=4, a11=100) == 1


def test_block_norm_refuses_outputs_that_overlap_its_inputs(L):
    """Host checks alone: no address is one of memory, and every call is refused."""
    from w8a8_int8_dynamic_b200.norms import _ARGS
    M, K, ld = 4, 64, 256
    X, R, O, Y = (n << 24 for n in range(1, 5))

    def call(x=X, r=R, o=O, y=Y, ldro=K, ldr=K, ldy=K, ldx=K, dtype=1, M=M):
        return L.w8a8_block_norm(_ARGS.pack(M, K, x, ldx, r, o, ldr, ldro, dtype, 1.0, 0, 0.0, 0, 0, 1, 1e-6, 0, 0, 0, 0, 0,
                                            0, 0, 0, 0, 0, 0, y, ldy, 0, 0, 0, 0), None)

    rows = M * K * 4                                               # bytes of the fp32 stream
    for o in (R + 16, R - 16, R + rows - 16, R - rows + 16, X, X + rows // 2 - 16, Y, Y + 16):
        assert call(o=o) == 1, hex(o)
    for y in (R, R + rows - 16, X + 16, X - 16, X + rows // 2 - 16, O):
        assert call(y=y) == 1, hex(y)
    assert call(o=R, ldro=ld) == call(o=R + K * 4, ldro=ld) == 1    # other strides in one range
    # columns of one wide tensor: side by side or not
    for d in (16, K * 4 - 16, -16, ld * 4 - 16, 2 * ld * 4 + 16, -K * 4 + 16):
        assert call(o=R + d, ldro=ld, ldr=ld) == 1, d
    assert call(o=R + 16, M=1) == call(o=R - 16, M=1) == 1
