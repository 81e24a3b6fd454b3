"""Cases and plain forms of the library's language-model operators.

Three operators that work together in a residual block run in 4 bits:

quantize  microscaled 4-bit floating point: every block of consecutive elements of a row shares
          one scale, each element is E2M1 (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
          "mx": blocks of 32, scale 2^e (E8M0), e = floor(log2(max |x|)) - 2, at least -127;
          "nv": blocks of 16, scale s * g with a tensor scale g and s = E4M3(max |x| / (6 g)).
          Measured with the way back: the values that the codes stand for.
linear    y = act(Q(x) W4^T + bias + residual): the activations are quantised on the way in, the
          weights are held in 4 bits.
norm      x' = x + rs * g(gate) * norm_post(z);  h = norm_pre(x'): the norm behind a block with its
          gate and residual scale, and the norm in front of the next one.
block     the path: x' = x + rs * gate * norm_post(W2 gelu(W1 Q(norm_pre(x)) + b1) + b2), with the
          hidden layer quantised again, and h = norm_final(x').

``run`` computes them from elementary operations in 32 bits, or calls the library where ``own``.
"""
import math

import torch

own = False  # True: run() calls the library's operators

EPS = 1e-6
BLOCK = {"mx": 32, "nv": 16}
DTYPE = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---- cases -------------------------------------------------------------------


def listed():
    return [
        # one row of a network's activations and back: only latency
        quantize_case("mx", 1, 4096, "bf16", name="quantize_row_mx"),
        # a large activation matrix: memory rate, and 64-bit element offsets near by
        quantize_case("nv", 16384, 8192, "bf16", name="quantize_large_nv"),
        # one token through a square projection: the weights' bytes and the launches
        linear_case("mx", 1, 4096, 4096, "bf16", "bf16", "none", True, False, name="linear_token_mx"),
        # the 1000-way classifier over 2048 pooled channels at batch 64
        linear_case("nv", 64, 2048, 1000, "bf16", "f32", "none", True, False, name="linear_classifier_nv"),
        # ragged in every direction, with a residual: tails of tiles, blocks and rows
        linear_case("mx", 777, 1456, 1111, "f32", "bf16", "relu", True, True, name="linear_ragged_mx"),
        # the expanding 1x1 convolution 256 -> 1024 over 14 x 14 pixels of 64 images
        linear_case("mx", 12544, 256, 1024, "bf16", "bf16", "relu", True, True, name="linear_pixels_mx"),
        # a prompt's expanding projection with its activation
        linear_case("nv", 4096, 4096, 16384, "bf16", "bf16", "gelu", True, False, name="linear_prompt_nv"),
        # one token between two blocks, both norms and a gate of its own
        norm_case("rms", "rms", 1, 4096, "bf16", "sigmoid", 1, name="norm_token"),
        # layer norms over an odd number of channels of 14 x 14 pixel maps, one gate per image
        norm_case("layer", "layer", 12544, 1001, "f32", "linear", 196, name="norm_images_odd"),
        # a long prompt's residual stream
        norm_case("rms", "rms", 32768, 8192, "bf16", "none", 1, name="norm_large"),
        # the path for one token
        block_case("mx", 1, 2048, 8192, 1, name="block_token_mx"),
        # the path for a long prompt
        block_case("nv", 8192, 4096, 16384, 1024, name="block_prompt_nv"),
    ]


def quantize_case(fmt, m, k, x, **more):
    return {"op": "quantize", "fmt": fmt, "m": m, "k": k, "x": x, **more}


def linear_case(fmt, m, k, n, x, y, act, bias, residual, **more):
    return {"op": "linear", "fmt": fmt, "m": m, "k": k, "n": n, "x": x, "y": y, "act": act,
            "bias": bias, "residual": residual, **more}


def norm_case(post, pre, m, c, x, gate, gate_rows, **more):
    return {"op": "norm", "post": post, "pre": pre, "m": m, "c": c, "x": x, "gate": gate,
            "gate_rows": gate_rows, **more}


def block_case(fmt, m, c, hidden, gate_rows, **more):
    return {"op": "block", "fmt": fmt, "m": m, "c": c, "hidden": hidden, "gate_rows": gate_rows,
            **more}


def _between(rng, lo, hi):
    """A whole number in [lo, hi], spread over its logarithm; two of three are multiples of 32."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v >= 64 and rng.random() < 0.67:
        v = v // 32 * 32
    return min(max(v, lo), hi)


def draw(rng):
    op = rng.choice(["quantize", "linear", "linear", "norm", "block"])
    fmt = rng.choice(["mx", "nv"])
    x = rng.choice(["bf16", "bf16", "f32"])
    if op == "quantize":
        k = _between(rng, 16, 16384)
        return quantize_case(fmt, _between(rng, 1, min(32768, (1 << 27) // k)), k, x)
    if op == "linear":
        k, n = _between(rng, 64, 16384), _between(rng, 32, 16384)
        m = _between(rng, 1, min(65536, (1 << 38) // (k * n), (1 << 27) // max(k, n)))
        return linear_case(fmt, m, k, n, x, rng.choice(["bf16", "bf16", "f32"]),
                           rng.choice(["none", "relu", "relu6", "gelu", "silu"]),
                           rng.random() < 0.7, rng.random() < 0.4)
    if op == "norm":
        c = _between(rng, 32, 16384)
        m = _between(rng, 1, min(65536, (1 << 27) // c))
        kinds = ["rms", "layer"]
        return norm_case(rng.choice(kinds + ["none"]), rng.choice(kinds), m, c, x,
                         rng.choice(["none", "linear", "sigmoid"]), rng.choice([1, 1, 49, 196, m]))
    c = _between(rng, 64, 4096)
    hidden = _between(rng, 128, 16384)
    m = _between(rng, 1, min(32768, (1 << 39) // (c * hidden), (1 << 27) // max(c, hidden)))
    return block_case(fmt, m, c, hidden, rng.choice([1, 49, 196, m]))


def work(case):
    op = case["op"]
    size = {"bf16": 2, "f32": 4}
    if op == "block":
        m, c, h = case["m"], case["c"], case["hidden"]
        weights = 2 * c * h * _bits(case["fmt"]) / 8
        # x in, x' and h out, the gates; the hidden layer need not leave the chip
        moved = 3 * 2 * m * c + 2 * c * -(-m // case["gate_rows"]) + 4 * (4 * c + h)
        return {"bytes": weights + moved, "flops": 4.0 * m * c * h + 20.0 * m * c}
    if op == "norm":
        m, c, b = case["m"], case["c"], size[case["x"]]
        gate = 0 if case["gate"] == "none" else b * c * -(-m // case["gate_rows"])
        return {"bytes": 4 * b * m * c + gate + 16 * c, "flops": 12.0 * m * c}
    m, k = case["m"], case["k"]
    if op == "quantize":  # in, codes and scales out and in again, values out
        return {"bytes": m * k * (2 * size[case["x"]] + 2 * _bits(case["fmt"]) / 8),
                "flops": 6.0 * m * k}
    n = case["n"]
    moved = size[case["x"]] * m * k + n * k * _bits(case["fmt"]) / 8 + size[case["y"]] * m * n
    moved += 4 * n * case["bias"] + size[case["y"]] * m * n * case["residual"]
    return {"bytes": moved, "flops": 2.0 * m * n * k}


def _bits(fmt):
    return 4 + 8 / BLOCK[fmt]


# ---- plain forms ---------------------------------------------------------------


def _round_e2m1(v):
    """Nearest E2M1 value, ties to the even one, the largest magnitude 6."""
    a = v.abs().clamp(max=6.0)
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.copysign(torch.round(a / step) * step, v)


def _quantize(x, fmt, g):
    """The E2M1 values [m, blocks, block] and scales of x's blocks, in 32 bits: for mx the
    scales 2^e, for nv the E4M3 scales s (a value is E2M1 * s * g)."""
    b = BLOCK[fmt]
    m, k = x.shape
    v = torch.nn.functional.pad(x.float(), (0, -k % b)).view(m, -1, b)
    top = v.abs().amax(dim=2, keepdim=True)
    if fmt == "mx":
        e = (torch.frexp(top)[1] - 3).clamp(min=-127)
        e = torch.where(top > 0, e, torch.full_like(e, -127))
        s = torch.exp2(e.float())
        return _round_e2m1(v / s), s
    s = (top / (6.0 * g)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
    t = s * g
    return torch.where(t > 0, _round_e2m1(v / t), torch.zeros_like(v)), s


def _values(q, s, g, k):
    """The values that E2M1 values and scales stand for, [m, k] in 32 bits."""
    return (q * (s * g)).view(q.shape[0], -1)[:, :k]


def _through(x, fmt, g):
    q, s = _quantize(x, fmt, g)
    return _values(q, s, g, x.shape[1])


_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _held(w, fmt, g):
    """Weights as a checkpoint holds them: codes [n, 16 * ceil(k / 32)], two to a byte with the
    even element in the low half, and one scale byte for each block, row by row."""
    q, s = _quantize(w, fmt, g)
    n, k = w.shape
    index = (q.abs() * 2).to(torch.uint8)  # 0 1 2 3 4 6 8 12
    code = index - (index > 4).to(torch.uint8) - 2 * (index > 6).to(torch.uint8) - (
        index > 8).to(torch.uint8) * 2
    code = (code + 8 * (q < 0).to(torch.uint8)).view(n, -1)
    code = torch.nn.functional.pad(code, (0, -code.shape[1] % 32))
    packed = code[:, 0::2] + 16 * code[:, 1::2]
    if fmt == "mx":
        scales = (torch.frexp(s)[1] - 1 + 127).to(torch.uint8)
    else:
        scales = s.to(torch.float8_e4m3fn).view(torch.uint8)
    return packed.contiguous(), scales.view(n, -1).contiguous()


def _held_values(packed, scales, fmt, g, k):
    """What such weights stand for, [n, k] in 32 bits."""
    levels = torch.tensor(_LEVELS + [-v for v in _LEVELS], device=packed.device)
    q = torch.stack([levels[(packed & 15).long()], levels[(packed >> 4).long()]], dim=2)
    b = BLOCK[fmt]
    q = q.view(packed.shape[0], -1)[:, : scales.shape[1] * b].reshape(packed.shape[0], -1, b)
    if fmt == "mx":
        s = torch.exp2(scales.float() - 127)
    else:
        s = scales.view(torch.float8_e4m3fn).float()
    return _values(q, s.unsqueeze(2), g, k)


def _act(v, act):
    if act == "relu":
        return v.clamp(min=0)
    if act == "relu6":
        return v.clamp(min=0, max=6)
    if act == "gelu":
        return 0.5 * v * (1 + torch.erf(v * math.sqrt(0.5)))
    if act == "silu":
        return v / (1 + torch.exp(-v))
    return v


def _norm(v, kind, w, b):
    if kind == "none":
        return v
    if kind == "layer":
        v = v - v.mean(dim=1, keepdim=True)
    v = v / torch.sqrt((v * v).mean(dim=1, keepdim=True) + EPS) * w
    return v + b if b is not None else v


def _gated(x, u, gate, kind, rows, rs):
    """x + rs * g(gate) * u, one row of gates for `rows` rows."""
    if kind == "none":
        return x + rs * u
    at = torch.arange(x.shape[0], device=x.device) // rows
    g = gate.to(u.dtype)
    g = 1 / (1 + torch.exp(-g)) if kind == "sigmoid" else g
    return x + rs * g[at] * u


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_plain(s):
    c = s["case"]
    op, fmt = c["op"], c.get("fmt")
    if op == "quantize":
        return _through(s["x"], fmt, s["gx"]).to(s["x"].dtype)
    if op == "linear":
        w = _held_values(s["w"], s["ws"], fmt, s["gw"], c["k"])
        y = _through(s["x"], fmt, s["gx"]) @ w.t()
        y = y if s["bias"] is None else y + s["bias"]
        y = y if s["residual"] is None else y + s["residual"].float()
        return _act(y, c["act"]).to(DTYPE[c["y"]])
    x = s["x"].float()
    if op == "norm":
        u = _norm(s["z"].float(), c["post"], s["w_post"], s["b_post"])
        x = _gated(x, u, s["gate"], c["gate"], c["gate_rows"], s["rs"])
        h = _norm(x, c["pre"], s["w_pre"], s["b_pre"])
        return [x.to(s["x"].dtype), h.to(s["x"].dtype)]
    w1 = _held_values(s["w1"], s["ws1"], fmt, s["gw1"], c["c"])
    w2 = _held_values(s["w2"], s["ws2"], fmt, s["gw2"], c["hidden"])
    h = _norm(x, "rms", s["w_pre"], None)
    t = _act(_through(h, fmt, s["gh"]) @ w1.t() + s["b1"], "gelu")
    z = _through(t, fmt, s["gt"]) @ w2.t() + s["b2"]
    u = _norm(z, "rms", s["w_post"], None)
    x = _gated(x, u, s["gate"], "linear", c["gate_rows"], s["rs"])
    h = _norm(x, "rms", s["w_final"], None)
    return [x.to(s["x"].dtype), h.to(s["x"].dtype)]


# ---- the library's operators ------------------------------------------------------


def _run_own(s):
    op = s["case"]["op"]
    if op == "quantize":
        from cnn_convolution_gemm_gb300 import fp4
        fp4.quantize(s["x"], s["fmt"], s["gx"], out=s["held"])
        return fp4.dequantize(s["held"], out=s["y"])
    if op == "linear":
        return s["layer"](s["x"], bias=s["bias"], residual=s["residual"], out=s["y"])
    if op == "norm":
        return list(s["layer"](s["x"], s["z"], gate=s["gate"], x_out=s["x_out"], h_out=s["h_out"]))
    return list(s["block"](s["x"], gate=s["gate"], x_out=s["x_out"], h_out=s["h_out"]))


def _own_handles(s):
    """The layers and output buffers that a program of the library keeps."""
    from cnn_convolution_gemm_gb300 import binding as B
    from cnn_convolution_gemm_gb300 import fp4
    c = s["case"]
    x = s["x"]
    fmts = {"mx": B.CONV_FP4_MX, "nv": B.CONV_FP4_NV}
    acts = {"none": B.CONV_ACT_NONE, "relu": B.CONV_ACT_RELU, "relu6": B.CONV_ACT_RELU6,
            "gelu": B.CONV_ACT_GELU, "silu": B.CONV_ACT_SILU}
    norms = {"none": B.CONV_NORM_NONE, "rms": B.CONV_NORM_RMS, "layer": B.CONV_NORM_LAYER}
    gates = {"none": B.CONV_GATE_NONE, "linear": B.CONV_GATE_LINEAR, "sigmoid": B.CONV_GATE_SIGMOID}
    if c["op"] == "quantize":
        s["fmt"] = fmts[c["fmt"]]
        s["held"] = fp4.empty(c["m"], c["k"], s["fmt"], x.device)
        s["y"] = torch.empty_like(x)
    elif c["op"] == "linear":
        s["layer"] = fp4.Fp4Linear(c["k"], c["n"], fmts[c["fmt"]], x_dtype=x.dtype,
                                   y_dtype=DTYPE[c["y"]], act=acts[c["act"]],
                                   has_residual=c["residual"], x_scale=s["gx"])
        s["layer"].load(s["w"], s["ws"], s["gw"])
        s["y"] = torch.empty(c["m"], c["n"], dtype=DTYPE[c["y"]], device=x.device)
    elif c["op"] == "norm":
        from cnn_convolution_gemm_gb300.norm import ResidualNorm
        s["layer"] = ResidualNorm(c["c"], x.dtype, eps=EPS, residual_scale=s["rs"],
                                  post=norms[c["post"]], w_post=s["w_post"], b_post=s["b_post"],
                                  pre=norms[c["pre"]], w_pre=s["w_pre"], b_pre=s["b_pre"],
                                  gate=gates[c["gate"]], gate_rows=c["gate_rows"])
        s["x_out"], s["h_out"] = torch.empty_like(x), torch.empty_like(x)
    else:
        from cnn_convolution_gemm_gb300.residual_block import Fp4ResidualBlock
        s["block"] = Fp4ResidualBlock(
            c["c"], c["hidden"], fmts[c["fmt"]], eps=EPS, residual_scale=s["rs"],
            gate=B.CONV_GATE_LINEAR, gate_rows=c["gate_rows"], w_pre=s["w_pre"],
            w_post=s["w_post"], w_next=s["w_final"], b1=s["b1"], b2=s["b2"],
            h_scale=s["gh"], t_scale=s["gt"])
        s["block"].load(s["w1"], s["ws1"], s["gw1"], s["w2"], s["ws2"], s["gw2"])
        s["x_out"], s["h_out"] = torch.empty_like(x), torch.empty_like(x)


# ---- inputs --------------------------------------------------------------------


def _inputs(case, seed):
    """What the operators read, from the seed alone: normal activations whose channels differ in
    size, with a few large ones; weights of a usual initialisation, held in 4 bits."""
    dev = "cuda"
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device=dev)

    def activations(m, k, dtype):
        return (normal(m, k) * torch.exp(0.5 * normal(k))).to(dtype)

    def weights(n, k, fmt):
        w = normal(n, k).mul_(1 / math.sqrt(k))
        # a checkpoint's tensor scale: the largest weight becomes 6 * 448
        g = 1.0 if fmt == "mx" else float(torch.tensor(6.0 / math.sqrt(k) / (6 * 448)))
        return (*_held(w.to(torch.bfloat16), fmt, g), g)

    # calibrated tensor scales of the activations: a high quantile, 23.4837 (the hidden layer:
    # 7.8142), becomes 6 * 448; numbers that 32 bits hold
    g_act = 1.0 if case.get("fmt") == "mx" else float(torch.tensor(23.4837 / (6 * 448)))
    op = case["op"]
    s = {"case": dict(case)}
    if op == "quantize":
        s |= {"x": activations(case["m"], case["k"], DTYPE[case["x"]]), "gx": g_act}
    elif op == "linear":
        s |= {"x": activations(case["m"], case["k"], DTYPE[case["x"]]), "gx": g_act}
        s["w"], s["ws"], s["gw"] = weights(case["n"], case["k"], case["fmt"])
        s["bias"] = 0.1 * normal(case["n"]) if case["bias"] else None
        s["residual"] = normal(case["m"], case["n"]).to(DTYPE[case["y"]]) if case["residual"] else None
    elif op == "norm":
        m, c, dt = case["m"], case["c"], DTYPE[case["x"]]
        s |= {"x": 4 * activations(m, c, dt), "z": activations(m, c, dt), "rs": 0.5}
        for side in ("post", "pre"):
            kind = case[side]
            s["w_" + side] = 1 + 0.1 * normal(c) if kind != "none" else None
            s["b_" + side] = 0.1 * normal(c) if kind == "layer" else None
        rows = -(-m // case["gate_rows"])
        s["gate"] = normal(rows, c).to(dt) if case["gate"] != "none" else None
    else:
        m, c, h, fmt = case["m"], case["c"], case["hidden"], case["fmt"]
        dt = torch.bfloat16
        s |= {"x": 4 * activations(m, c, dt), "rs": 0.5}
        s["w1"], s["ws1"], s["gw1"] = weights(h, c, fmt)
        s["w2"], s["ws2"], s["gw2"] = weights(c, h, fmt)
        s["b1"], s["b2"] = 0.1 * normal(h), 0.1 * normal(c)
        for side in ("w_pre", "w_post", "w_final"):
            s[side] = 1 + 0.1 * normal(c)
        s["gate"] = normal(-(-m // case["gate_rows"]), c).to(dt)
        s["gh"] = g_act
        s["gt"] = 1.0 if fmt == "mx" else float(torch.tensor(7.8142 / (6 * 448)))
    return s


def prepare(case, seed):
    s = _inputs(case, seed)
    if own:
        _own_handles(s)
    return s


# ---- the definitions in 64 bits ---------------------------------------------------


def _exact_through(x, fmt, g):
    """Q(x) in 64 bits: the nearest level by counting the midpoints that lie below."""
    x = x.double()
    m, k = x.shape
    b = BLOCK[fmt]
    full = torch.zeros(m, -(-k // b) * b, dtype=torch.float64, device=x.device)
    full[:, :k] = x
    full = full.reshape(m, -1, b)
    top = full.abs().max(dim=2, keepdim=True).values
    if fmt == "mx":
        e = torch.floor(torch.log2(torch.where(top > 0, top, torch.ones_like(top))))
        e = e + (torch.pow(2.0, e + 1) <= top).double() - (torch.pow(2.0, e) > top).double()
        scale = torch.pow(2.0, torch.where(top > 0, (e - 2).clamp(min=-127), e * 0 - 127))
    else:
        want = (top / (6 * g)).clamp(max=448)
        p = torch.floor(torch.log2(want.clamp(min=2.0 ** -6)))
        unit = torch.pow(2.0, p - 3)  # spacing of E4M3 at this size
        n = torch.floor(want / unit)
        rest = want / unit - n
        n = n + ((rest > 0.5) | ((rest == 0.5) & (torch.remainder(n, 2) == 1))).double()
        scale = n * unit * g
    size = torch.where(scale > 0, full.abs() / scale, torch.zeros_like(full))
    level = torch.zeros_like(full)
    for i in range(7):
        middle = (_LEVELS[i] + _LEVELS[i + 1]) / 2
        passed = size > middle if i % 2 == 0 else size >= middle  # a tie goes to the even code
        level = level + passed.double() * (_LEVELS[i + 1] - _LEVELS[i])
    return (torch.sign(full) * level * scale).reshape(m, -1)[:, :k]


def _exact_weights(packed, scales, fmt, g, k):
    code = torch.stack([packed % 16, packed // 16], dim=2).reshape(packed.shape[0], -1)[:, :k]
    code = code.long()
    e, f = (code % 8) // 2, code % 2
    size = torch.where(e > 0, torch.pow(2.0, (e - 1).double()) * (1 + 0.5 * f), 0.5 * f.double())
    raw = scales.long()
    if fmt == "mx":
        scale = torch.pow(2.0, raw.double() - 127)
    else:
        e4, f3 = raw // 8, (raw % 8).double()
        scale = torch.where(e4 > 0, torch.pow(2.0, e4.double() - 7) * (1 + f3 / 8),
                            f3 * 2.0 ** -9) * g
    return size * (1 - 2.0 * (code // 8)) * scale.repeat_interleave(BLOCK[fmt], dim=1)[:, :k]


def _exact_norm(v, kind, w, b):
    if kind == "none":
        return v
    mean = v.sum(1, keepdim=True) / v.shape[1] if kind == "layer" else 0.0
    var = ((v - mean) ** 2).sum(1, keepdim=True) / v.shape[1]
    out = (v - mean) * (var + EPS) ** -0.5 * w.double()
    return out if b is None else out + b.double()


def _exact_act(v, act):
    if act == "gelu":
        return v * torch.special.ndtr(v)
    if act == "silu":
        return v * torch.sigmoid(v)
    if act in ("relu", "relu6"):
        v = torch.maximum(v, torch.zeros_like(v))
        return torch.minimum(v, torch.full_like(v, 6.0)) if act == "relu6" else v
    return v


def exact(case, seed):
    s = _inputs(case, seed)
    op, fmt = case["op"], case.get("fmt")
    if op == "quantize":
        return _exact_through(s["x"], fmt, s["gx"])
    if op == "linear":
        w = _exact_weights(s["w"], s["ws"], fmt, s["gw"], case["k"])
        y = torch.matmul(_exact_through(s["x"], fmt, s["gx"]), w.t())
        for more in (s["bias"], s["residual"]):
            y = y if more is None else y + more.double()
        return _exact_act(y, case["act"])
    x = s["x"].double()
    rows = torch.div(torch.arange(x.shape[0], device=x.device), case["gate_rows"],
                     rounding_mode="floor")
    gate = 1.0 if s["gate"] is None else s["gate"].double()[rows]
    if op == "norm":
        gate = torch.sigmoid(gate) if case["gate"] == "sigmoid" else gate
        x = x + s["rs"] * gate * _exact_norm(s["z"].double(), case["post"], s["w_post"], s["b_post"])
        return [x, _exact_norm(x, case["pre"], s["w_pre"], s["b_pre"])]
    h = _exact_through(_exact_norm(x, "rms", s["w_pre"], None), fmt, s["gh"])
    t = torch.matmul(h, _exact_weights(s["w1"], s["ws1"], fmt, s["gw1"], case["c"]).t())
    t = _exact_through(_exact_act(t + s["b1"].double(), "gelu"), fmt, s["gt"])
    z = torch.matmul(t, _exact_weights(s["w2"], s["ws2"], fmt, s["gw2"], case["hidden"]).t())
    x = x + s["rs"] * gate * _exact_norm(z + s["b2"].double(), "rms", s["w_post"], None)
    return [x, _exact_norm(x, "rms", s["w_final"], None)]
