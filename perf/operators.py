"""What is measured of the 4-bit microscaled layers and of the fused norms around a block.

A case is one call, or one short run of calls, as a serving program makes them: the quantisation of a tensor, a linear
layer, an MLP, the norm step between two layers, and that step together with the layer behind it. ``run`` has each in a
plain form (elementary torch operations) and, where ``own`` is true, as calls of this repository's package.

The 4-bit format is the MX one: blocks of 32 consecutive values of a row share a scale 2^e, the values are e2m1
(0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives), e = floor(log2(largest magnitude)) - 2, at least -127.
"""
import math

import torch
import torch.nn.functional as F  # F.pad alone

own = False


# ---- the cases ------------------------------------------------------------------
def listed():
    return [
        # quantisation, there and back: one token's hidden state; an MLP's hidden activations of an image's tokens
        {"name": "quant_1x5120", "op": "quant", "M": 1, "K": 5120},
        {"name": "quant_4096x12288", "op": "quant", "M": 4096, "K": 12288},
        # a linear layer: one decoded token against an LLM's up-projection (weight streaming)
        {"name": "linear_1x27648x5120", "op": "linear", "M": 1, "N": 27648, "K": 5120, "bias": False, "act": False},
        # a small decode batch against a down-projection
        {"name": "linear_13x5120x13824", "op": "linear", "M": 13, "N": 5120, "K": 13824, "bias": True, "act": False},
        # a square projection of a short prompt
        {"name": "linear_512x4096x4096", "op": "linear", "M": 512, "N": 4096, "K": 4096, "bias": True, "act": False},
        # odd sizes in every direction: a ragged batch, K that ends inside a block
        {"name": "linear_1337x2056x1808", "op": "linear", "M": 1337, "N": 2056, "K": 1808, "bias": True, "act": True},
        # a transformer's MLP: a decode batch, and an image's tokens
        {"name": "mlp_4x5120x13824", "op": "mlp", "M": 4, "K": 5120, "N": 13824},
        {"name": "mlp_4096x4096x12288", "op": "mlp", "M": 4096, "K": 4096, "N": 12288},
        # the norm step between two layers: one token (RMS, no modulation, residual kept in fp32) ...
        {"name": "norm_1x5120_rms", "op": "norm", "M": 1, "K": 5120, "kind": "rms", "post": False, "groups": 0,
         "residual": "float32"},
        # ... and an image batch: norm after the block, gate, residual, modulated norm before the next
        {"name": "norm_8192x4096_layer", "op": "norm", "M": 8192, "K": 4096, "kind": "layer", "post": True, "groups": 2,
         "residual": "bfloat16"},
        # that step and the layer behind it, whose codes the step forms: int8 and 4-bit
        {"name": "block_int8_1000x4096x4096", "op": "block", "M": 1000, "K": 4096, "N": 4096, "kind": "layer",
         "post": False, "groups": 3, "residual": "bfloat16", "codes": "int8"},
        {"name": "block_mx4_2048x4096x12288", "op": "block", "M": 2048, "K": 4096, "N": 12288, "kind": "rms", "post": True,
         "groups": 1, "residual": "float32", "codes": "mx4"},
    ]


def draw(rng):
    def size(lo, hi, step):
        return max(lo, step * round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step))

    op = rng.choice(("quant", "linear", "linear", "mlp", "norm", "block"))
    M, K, N = size(1, 4096, 1), size(64, 13824, 16), size(64, 27648, 16)
    if op in ("linear", "mlp", "block"):  # no dearer than the largest listed case
        while M * N * K > 4096 * 4096 * 12288:
            M, N = max(1, M // 2), max(64, N // 32 * 16)
    norm = {"kind": rng.choice(("rms", "layer")), "post": rng.random() < 0.5, "groups": min(M, rng.choice((0, 1, 2, 5))),
            "residual": rng.choice(("bfloat16", "float32"))}
    if op == "quant":
        return {"op": op, "M": M, "K": K}
    if op == "linear":
        return {"op": op, "M": M, "N": N, "K": K, "bias": rng.random() < 0.5, "act": rng.random() < 0.3}
    if op == "mlp":
        return {"op": op, "M": M, "K": K, "N": N}
    if op == "norm":
        return {"op": op, "M": size(1, 8192, 1), "K": min(K, 8192), **norm}
    return {"op": op, "M": M, "K": K, "N": N, **norm, "codes": rng.choice(("int8", "mx4"))}


# ---- inputs -----------------------------------------------------------------------
def _inputs(case, seed):
    """The case's tensors, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))

    def normal(*shape, std=1.0, mean=0.0):
        return torch.randn(*shape, device="cuda", generator=g).mul_(std).add_(mean)

    def activations(M, K):  # a few outlier channels, as transformers have them
        x = normal(M, K)
        x[:, torch.randperm(K, device="cuda", generator=g)[: max(1, K // 100)]] *= 10.0
        return x.bfloat16()

    def bias(n):
        return normal(n, std=0.02).bfloat16()

    op, M, K, N = case["op"], case["M"], case["K"], case.get("N")
    s = {"x": activations(M, K)}
    if op == "linear":
        s["w"] = _encode(normal(N, K, std=K ** -0.5))
        s["bias"] = bias(N) if case["bias"] else None
    if op == "mlp":
        s["w"], s["bias"] = _encode(normal(N, K, std=K ** -0.5)), bias(N)
        s["w2"], s["bias2"] = _encode(normal(K, N, std=N ** -0.5)), bias(K)
    if op in ("norm", "block"):
        s["residual"] = normal(M, K, std=2.0).to(getattr(torch, case["residual"]))
        s["weight"] = normal(K, std=0.1, mean=1.0).bfloat16()
        s["post_weight"] = normal(K, std=0.1, mean=1.0).bfloat16() if case["post"] else None
        if case["groups"]:  # one modulation vector for each image: gate, scale and shift in one tensor's columns
            s["mod"] = normal(case["groups"], 3 * K, std=0.3).bfloat16()
    if op == "block":
        s["bias"] = bias(N)
        if case["codes"] == "mx4":
            s["w"] = _encode(normal(N, K, std=K ** -0.5))
        else:
            s["w"] = torch.randint(-127, 128, (N, K), device="cuda", generator=g, dtype=torch.int8)
            s["w_scale"] = torch.rand(N, device="cuda", generator=g).mul_(4.5e-3).add_(5e-4)
    return s


def _power(e):
    """2^e in 64 bits, exactly (exp2 of a whole number may be an ulp off)."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _encode(w):
    """A weight as a 4-bit checkpoint holds it: (codes, two to a byte with the lower k in the lower half, scale bytes)."""
    rows, K = w.shape
    blocks = F.pad(w, (0, -K % 32)).view(rows, -1, 32)
    _, e = torch.frexp(blocks.abs().amax(-1))
    e = (e - 3).clamp_(min=-127)
    v = blocks * _power(-e).float()[..., None]
    a = v.abs().clamp_(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    a = torch.round(a / step) * step
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = (code | ((v < 0).to(torch.uint8) << 3)).view(rows, -1)
    return (code[:, 0::2] | (code[:, 1::2] << 4))[:, : K // 2].contiguous(), (e + 127).to(torch.uint8)


def _decode(w, K, dtype):
    """The values of a checkpoint's weight."""
    codes, scales = w
    table = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6, -0.0, -0.5, -1, -1.5, -2, -3, -4, -6], dtype=dtype, device="cuda")
    q = torch.stack((table[(codes & 15).int()], table[(codes >> 4).int()]), -1).view(codes.shape[0], K)
    return q * _power(scales.int() - 127).to(dtype).repeat_interleave(32, 1)[:, :K]


def prepare(case, seed):
    """The inputs, and the weights as a program keeps them: laid out for the kernels, or as plain values."""
    s = _inputs(case, seed)
    s["case"] = case
    if case["op"] in ("norm", "block"):
        K, M, groups = case["K"], case["M"], case["groups"]
        s["rows"] = -(-M // groups) if groups else M
        s["gate"], s["scale"], s["shift"] = s.pop("mod").split(K, 1) if groups else (None, None, None)
    if own:
        import w8a8_int8_dynamic_b200 as w8
        s["w8"] = w8
        if case["op"] in ("linear", "mlp"):
            s["layer"] = w8.MX4Linear(*s.pop("w"), s.pop("bias"),
                                      act=w8.ACT_GELU_TANH if case.get("act", True) else w8.ACT_NONE)
        if case["op"] == "mlp":
            s["layer2"] = w8.MX4Linear(*s.pop("w2"), s.pop("bias2"))
        if case["op"] == "block":
            s["layer"] = (w8.MX4Linear(*s.pop("w"), s.pop("bias")) if case["codes"] == "mx4" else
                          w8.W8A8Linear(s.pop("w"), s.pop("w_scale"), s.pop("bias")))
        if case["op"] in ("norm", "block"):
            s["pre"] = w8.Norm(case["kind"], s["weight"], eps=1e-6)
            s["post"] = w8.Norm(case["kind"], s["post_weight"], eps=1e-6) if case["post"] else None
    else:
        for name, K in (("w", case["K"]), ("w2", case.get("N"))):
            if name in s:
                s[name] = _decode(s[name], K, torch.float32) if isinstance(s[name], tuple) else s[name].float()
    return s


# ---- one pass -----------------------------------------------------------------------
def run(s):
    return _run_own(s) if own else _run_plain(s)


def _run_own(s):
    w8, op = s["w8"], s["case"]["op"]
    if op == "quant":
        return w8.mx4_quant(s["x"]).dequant()
    if op == "linear":
        return s["layer"](s["x"])
    if op == "mlp":
        return s["layer2"](s["layer"].quantised(s["x"]))
    out = w8.block_norm(s["x"], s["residual"], post=s["post"], gate=s["gate"], residual_scale=0.75, pre=s["pre"],
                        scale=s["scale"], shift=s["shift"], rows_per_group=s["rows"],
                        codes=s["case"].get("codes"))
    if op == "norm":
        return out.residual, out.y
    if s["case"]["codes"] == "mx4":
        return out.residual, s["layer"](out.mx4)
    return out.residual, s["layer"].apply_codes(out.q, out.a_scale)


def _values(x):
    """What the 4-bit codes of x stand for."""
    rows, K = x.shape
    blocks = F.pad(x, (0, -K % 32)).view(rows, -1, 32)
    _, e = torch.frexp(blocks.abs().amax(-1, keepdim=True))
    unit = _power((e - 3).clamp_(min=-127)).float()
    a = (blocks / unit).abs().clamp_(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return (torch.copysign(torch.round(a / step) * step, blocks) * unit).view(rows, -1)[:, :K]


def _gelu(y):
    y = y.bfloat16().float()
    return y * torch.sigmoid(2 * math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3))


def _norm(t, kind, weight):
    if kind == "layer":
        t = t - t.mean(-1, keepdim=True)
    return t * torch.rsqrt(t.square().mean(-1, keepdim=True) + 1e-6) * weight.float()


def _run_plain(s):
    case = s["case"]
    x = s["x"].float()
    if case["op"] == "quant":
        return _values(x).bfloat16()
    if case["op"] in ("linear", "mlp"):
        y = _values(x) @ s["w"].t()
        if s["bias"] is not None:
            y = y + s["bias"].float()
        if case.get("act", True):
            y = _gelu(y)
        if case["op"] == "mlp":
            y = _values(y.bfloat16().float()) @ s["w2"].t() + s["bias2"].float()
        return y.bfloat16()
    group = torch.arange(case["M"], device="cuda") // s["rows"]
    u = _norm(x, case["kind"], s["post_weight"]) if case["post"] else x
    if s["gate"] is not None:
        u = u * s["gate"].float()[group]
    residual = (0.75 * s["residual"].float() + u).to(s["residual"].dtype)
    h = _norm(residual.float(), case["kind"], s["weight"])
    if s["scale"] is not None:
        h = h * (1 + s["scale"].float()[group]) + s["shift"].float()[group]
    h = h.bfloat16()
    if case["op"] == "norm":
        return residual, h
    h = h.float()
    if case["codes"] == "mx4":
        y = _values(h) @ s["w"].t()
    else:
        unit = h.abs().amax(-1, keepdim=True) / 127
        y = torch.round(h / unit.clamp(min=1e-38)) @ s["w"].t() * unit * s["w_scale"]
    return residual, (y + s["bias"].float()).bfloat16()


# ---- the same from the definition, in 64 bits ------------------------------------------
def exact(case, seed):
    s = _inputs(case, seed)
    op, M, K = case["op"], case["M"], case["K"]

    def rounded(t, dtype=torch.bfloat16):  # a rounding that the definition has between two steps
        return t.to(dtype).double()

    grid = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64, device="cuda")

    def four_bit(t):
        """Nearest grid value under the block's scale; a tie goes to the value with the even code."""
        k = t.shape[1]
        t = F.pad(t, (0, -k % 32)).unflatten(1, (-1, 32))
        most = t.abs().amax(-1, keepdim=True)
        unit = _power(((most.view(torch.int64) >> 52) - 1025).clamp(min=-127))  # a zero: the smallest
        size = t.abs() / unit
        mids = (grid[1:] + grid[:-1]) / 2
        up = torch.bucketize(size, mids, right=True)     # a tie: the upper neighbour
        down = torch.bucketize(size, mids, right=False)  # a tie: the lower one
        return (torch.sign(t) * grid[torch.where(up % 2 == 0, up, down)] * unit).flatten(1)[:, :k]

    def gelu(t):
        return 0.5 * t * (1 + torch.tanh(math.sqrt(2 / math.pi) * (t + 0.044715 * t * t * t)))

    x = s["x"].double()
    if op == "quant":
        return four_bit(x)
    if op in ("linear", "mlp"):
        y = four_bit(x).matmul(_decode(s["w"], K, torch.float64).t())
        if s["bias"] is not None:
            y += s["bias"].double()
        if op == "linear":
            return gelu(rounded(y)) if case["act"] else y
        hidden = rounded(gelu(rounded(y)))
        return four_bit(hidden).matmul(_decode(s["w2"], case["N"], torch.float64).t()) + s["bias2"].double()

    def norm(t, weight):
        centre = t.mean(1, keepdim=True) if case["kind"] == "layer" else 0.0
        return (t - centre) / torch.sqrt(((t - centre) ** 2).mean(1, keepdim=True) + 1e-6) * weight.double()

    per_row = [None, None, None]
    if case["groups"]:
        which = torch.arange(M, device="cuda").div(-(-M // case["groups"]), rounding_mode="floor")
        per_row = [s["mod"][:, i * K:(i + 1) * K].double().index_select(0, which) for i in range(3)]
    gate, scale, shift = per_row
    branch = norm(x, s["post_weight"]) if case["post"] else x
    total = s["residual"].double() * 0.75 + (branch if gate is None else gate * branch)
    h = norm(rounded(total, s["residual"].dtype), s["weight"])
    if scale is not None:
        h = h + h * scale + shift
    if op == "norm":
        return total, h
    h = rounded(h)
    if case["codes"] == "mx4":
        y = four_bit(h).matmul(_decode(s["w"], K, torch.float64).t())
    else:
        unit = h.abs().amax(1, keepdim=True) / 127
        y = torch.where(unit > 0, h / unit, 0.0).round().matmul(s["w"].double().t()) * unit * s["w_scale"].double()
    return total, y + s["bias"].double()


# ---- what a pass cannot do without --------------------------------------------------------
def work(case):
    op, M, K, N = case["op"], case["M"], case["K"], case.get("N", 0)
    four = 17 / 32  # bytes of a 4-bit value with its share of the scale
    if op == "quant":  # x in, the values out
        return {"bytes": M * K * (2 + 2), "flops": 2 * M * K}
    if op == "linear":
        return {"bytes": 2 * M * K + four * N * K + (2 * N if case["bias"] else 0) + 2 * M * N, "flops": 2 * M * N * K}
    if op == "mlp":
        return {"bytes": 2 * M * K + 2 * four * N * K + 2 * (N + K) + 2 * M * K, "flops": 4 * M * N * K}
    held = 4 if case["residual"] == "float32" else 2
    step = M * K * (2 + 2 * held) + 2 * K * (1 + case["post"] + 3 * case["groups"])
    flops = M * K * (8 + 4 * case["post"])
    if op == "norm":
        return {"bytes": step + 2 * M * K, "flops": flops}
    weight = (four if case["codes"] == "mx4" else 1) * N * K + (0 if case["codes"] == "mx4" else 4 * N)
    return {"bytes": step + weight + 2 * N + 2 * M * N, "flops": flops + 2 * M * N * K}
