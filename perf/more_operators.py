"""The workloads by which the microscaled 4-bit operators and the per-head norms are measured.

Four paths of a transformer block whose projections hold microscaled 4-bit
floating point (MXFP4: blocks of 32 values, each value one of 0, 0.5, 1, 1.5,
2, 3, 4, 6 with a sign, times the block's power of two):

  quant   values -> codes and scales -> the values they stand for, by which a
          quantizer's error is measured
  linear  out[t][k] = sum_j x_tj w_kj + b_k, both operands MXFP4
  down    the down projection: x = bf16(SiLU(gate) up) or x itself, rotated by
          a Hadamard matrix and flipped by the calibrated signs, quantized,
          times the folded weights
             y = (x H / sqrt n) * d,  d = sigma H[c],  out = MXFP4(y) w^T
  qk      the norm of each head of the queries and keys, then their rotation
          by the token's position

`run` computes them in elementary torch operations in binary32 where `own` is
false, and through the package's entry points where it is true.
"""

import math

import torch

own = False

EPS = 1e-6
# hidden and intermediate widths of the package's own workloads
HIDDEN = (4096, 5120, 8192)
INNER = (11008, 13824, 14336, 28672)
# widths of the down projection, with the order of the outer Hadamard factor (1: powers of two)
ROTATED = {4096: 1, 8192: 1, 14336: 28, 28672: 28, 13824: 108, 5120: 20}


def listed():
    return [
        # the error of one token's activations
        {"name": "quant_t1_n4096", "op": "quant", "tokens": 1, "n": 4096, "in": "bf16", "rule": "floor"},
        # odd sizes: the last block is short, and no row begins on a vector
        {"name": "quant_t613_n1111_f32", "op": "quant", "tokens": 613, "n": 1111, "in": "f32", "rule": "noclip"},
        # a prompt batch at the down projection's input
        {"name": "quant_t8192_n14336", "op": "quant", "tokens": 8192, "n": 14336, "in": "bf16", "rule": "floor"},
        # decode: one token through an up projection
        {"name": "linear_t1_n4096_r14336", "op": "linear", "tokens": 1, "n": 4096, "rows": 14336, "out": "bf16",
         "bias": False},
        # odd sizes in every direction: no tile or step ends where the data does
        {"name": "linear_t613_n1120_r777", "op": "linear", "tokens": 613, "n": 1120, "rows": 777, "out": "f32",
         "bias": True},
        # a prompt batch through an up projection
        {"name": "linear_t8192_n4096_r14336", "op": "linear", "tokens": 8192, "n": 4096, "rows": 14336,
         "out": "bf16", "bias": False},
        # a decode batch at the widest down projection, the SwiGLU producer fused in
        {"name": "down_t16_n28672_r8192", "op": "down", "tokens": 16, "n": 28672, "rows": 8192, "swiglu": True},
        # a short prompt at a width with another outer order
        {"name": "down_t200_n13824_r5120", "op": "down", "tokens": 200, "n": 13824, "rows": 5120, "swiglu": False},
        # a prompt batch
        {"name": "down_t8192_n14336_r4096", "op": "down", "tokens": 8192, "n": 14336, "rows": 4096, "swiglu": True},
        # decode: one token of grouped-query attention
        {"name": "qk_t1_h32_8_d128", "op": "qk", "tokens": 1, "q_heads": 32, "k_heads": 8, "head": 128, "rotary": 128,
         "norm": "rms", "interleaved": False, "in": "bf16"},
        # heads of an odd number of vectors, LayerNorm with biases, half of each head rotated, adjacent pairs
        {"name": "qk_t777_h12_12_d80_f32", "op": "qk", "tokens": 777, "q_heads": 12, "k_heads": 12, "head": 80,
         "rotary": 40, "norm": "layer", "interleaved": True, "in": "f32"},
        # a prompt batch at the widest attention
        {"name": "qk_t8192_h64_8_d128", "op": "qk", "tokens": 8192, "q_heads": 64, "k_heads": 8, "head": 128,
         "rotary": 128, "norm": "rms", "interleaved": False, "in": "bf16"},
    ]


_MOST = 8000 * 14336 * 4096  # products of one drawn pass


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("quant", "linear", "down", "qk"))
    tokens = _log(rng, 1, 8192)
    if rng.random() < 0.3:
        tokens = rng.choice((1, 2, 4, 16, 64))
    if op == "quant":
        n = rng.choice(HIDDEN + INNER) if rng.random() < 0.5 else _log(rng, 8, 14336)
        return {"op": op, "tokens": max(1, min(tokens, 8192 * 14336 // n)), "n": n, "in": rng.choice(("bf16", "f32")),
                "rule": rng.choice(("floor", "noclip"))}
    if op == "linear":
        if rng.random() < 0.6:
            n, rows = rng.choice(HIDDEN), rng.choice(INNER)
            if rng.random() < 0.3:
                n, rows = rows, n
        else:
            n, rows = 32 * _log(rng, 2, 512), _log(rng, 64, 16384)
        return {"op": op, "tokens": max(1, min(tokens, _MOST // (n * rows))), "n": n, "rows": rows,
                "out": rng.choice(("bf16", "f32")), "bias": rng.random() < 0.5}
    if op == "down":
        n, rows = rng.choice(tuple(ROTATED)), rng.choice(HIDDEN)
        return {"op": op, "tokens": max(1, min(tokens, _MOST // (n * rows))), "n": n, "rows": rows,
                "swiglu": ROTATED[n] in (1, 28) and rng.random() < 0.5}
    head = rng.choice((64, 128, 128, 256)) if rng.random() < 0.6 else 8 * rng.randint(2, 32)
    k_heads = rng.choice((1, 2, 4, 8, 12, 16))
    return {"op": op, "tokens": tokens, "q_heads": k_heads * rng.choice((1, 2, 4)), "k_heads": k_heads, "head": head,
            "rotary": head if rng.random() < 0.6 else 2 * rng.randint(1, head // 2),
            "norm": rng.choice(("rms", "rms", "layer", "none")), "interleaved": rng.random() < 0.4,
            "in": rng.choice(("bf16", "bf16", "f32"))}


# ---- inputs ----------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _pow2(e):
    """2^e in binary32 for whole e in [-127, 127], from its bits."""
    e = e.to(torch.int32)
    return torch.where(e < -126, 1 << 22, (e + 127) << 23).view(torch.float32)


def _blocks(x):
    """[T, n] -> [T, blocks, 32], the last block filled with zeros."""
    t, n = x.shape
    return torch.nn.functional.pad(x, (0, -n % 32)).reshape(t, -1, 32)


def _quantize(x, rule):
    """binary32 rows -> (values in units of the scale [T, blocks, 32], exponents [T, blocks])."""
    b = _blocks(x)
    m, e = torch.frexp(b.abs().amax(dim=2))  # amax = m 2^e, m in [0.5, 1)
    e = e - 3
    if rule == "noclip":
        e = e + (m > 0.75).int()  # above 6 2^e
    e = torch.where(m > 0, e, -127).clamp(-127, 127)
    v = b / _pow2(e)[:, :, None]
    a = v.abs()
    step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
    return torch.sign(v) * (torch.round(a / step) * step).clamp(max=6.0), e


def _pack(v, e):
    """Units [T, blocks, 32] and exponents -> (codes u8 [T, 16 blocks], scales u8 [T, blocks])."""
    a = v.abs()
    code = torch.where(a < 2, 2 * a, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code + 8 * (v < 0).to(torch.uint8)
    codes = code[:, :, 0::2] | (code[:, :, 1::2] << 4)
    return codes.reshape(v.shape[0], -1).contiguous(), (e + 127).to(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t = case["tokens"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    def weights(rows, n):
        """A trained projection's weights, quantized offline."""
        w = normal(rows, n)
        w *= (torch.rand((rows, 1), generator=gen, device="cuda") + 0.5) / math.sqrt(n)
        return _pack(*_quantize(w, "floor"))

    s = {"case": dict(case)}
    if case["op"] == "quant":
        x = normal(t, case["n"]) * (0.2 + torch.rand((t, 1), generator=gen, device="cuda"))
        x[:, case["n"] // 2] *= 30.0  # a massive channel
        s["x"] = x.to(_TYPES[case["in"]])
    elif case["op"] == "linear":
        x = normal(t, case["n"]) * (0.2 + torch.rand((t, 1), generator=gen, device="cuda"))
        s["codes"], s["scale"] = _pack(*_quantize(x, "floor"))
        s["w"], s["w_scale"] = weights(case["rows"], case["n"])
        s["bias"] = normal(case["rows"]) * 0.1 if case["bias"] else None
    elif case["op"] == "down":
        n = case["n"]
        s["channel"], s["sigma"] = int(seed * 7919 % n), 1 if seed % 2 else -1
        heavy = torch.rand(t, generator=gen, device="cuda") < 0.2
        peak = 800.0 + 1700.0 * torch.rand(t, generator=gen, device="cuda")
        if case["swiglu"]:
            gate, up = normal(t, n) * 1.5, normal(t, n) * 0.6
            gate[heavy, s["channel"]] = 8.0
            up[heavy, s["channel"]] = s["sigma"] * peak[heavy] / 8.0
            s["gate"], s["up"] = gate.to(torch.bfloat16), up.to(torch.bfloat16)
        else:
            x = normal(t, n) * 0.7
            x[heavy, s["channel"]] = s["sigma"] * peak[heavy]
            s["x"] = x.to(torch.bfloat16)
        s["w"], s["w_scale"] = weights(case["rows"], n)
    else:
        hq, hk, d, r = case["q_heads"], case["k_heads"], case["head"], case["rotary"]
        both = normal(t, (hq + 2 * hk) * d) * 1.5  # queries, keys and values as the projection leaves them
        both[:, :: max(d // 2, 1)] *= 8.0
        both = both.to(_TYPES[case["in"]])
        s["q"] = both[:, :hq * d].view(t, hq, d)
        s["k"] = both[:, hq * d:(hq + hk) * d].view(t, hk, d)
        layer = case["norm"] == "layer"
        for name in ("q", "k"):
            s[name + "_weight"] = (1.0 + 0.1 * normal(d)).to(torch.bfloat16) if case["norm"] != "none" else None
            s[name + "_bias"] = (0.1 * normal(d)).to(torch.bfloat16) if layer else None
        # packed sequences of different lengths: positions count from each one's start, a few far into a context
        places = 32768
        cuts = torch.randint(0, t, (5,), generator=gen, device="cuda")
        where = torch.arange(t, device="cuda")
        start = torch.where(cuts[None, :] <= where[:, None], cuts[None, :], 0).amax(dim=1)
        first = torch.randint(0, places - t, (1,), generator=gen, device="cuda")
        s["positions"] = torch.where(start == 0, first + where, where - start).to(torch.int32)
        inverse = 500000.0 ** (-torch.arange(0, r, 2, device="cuda", dtype=torch.float64) / r)
        angle = torch.arange(places, device="cuda", dtype=torch.float64)[:, None] * inverse[None, :]
        s["cos"], s["sin"] = angle.cos().float(), angle.sin().float()
    return s


# ---- one pass --------------------------------------------------------------


def _values(codes, scale):
    """MXFP4 codes and scales -> [T, n] in binary32."""
    t = codes.shape[0]
    c = torch.stack((codes & 15, codes >> 4), dim=2).reshape(t, -1, 32)
    m = (c & 7).float()
    a = torch.where(m < 4, m / 2, torch.where(m < 6, m - 2, 2 * m - 8))
    a = torch.where(c > 7, -a, a) * _pow2(scale.int() - 127)[:, :, None]
    return a.reshape(t, -1)


def _parity(x):
    x = x ^ (x >> 8)
    x = x ^ (x >> 4)
    x = x ^ (x >> 2)
    return (x ^ (x >> 1)) & 1


def _sylvester(order):
    i = torch.arange(order, device="cuda")
    return 1.0 - 2.0 * _parity(i[:, None] & i[None, :]).float()


def _outer(m):
    """The outer Hadamard factor of order m: 1, or Paley's first construction over GF(m - 1)."""
    if m == 1:
        return torch.ones((1, 1), device="cuda")
    q = m - 1
    e = torch.arange(q, device="cuda")
    if q == 27:  # GF(3)[t] / (t^3 + 2t + 1): t^3 = t + 2, t^4 = t^2 + 2t
        c0, c1, c2 = e % 3, e // 3 % 3, e // 9
        squares = ((c0 * c0 + 4 * c1 * c2) % 3 + 3 * ((2 * c0 * c1 + 2 * c1 * c2 + 2 * c2 * c2) % 3)
                   + 9 * ((c1 * c1 + 2 * c0 * c2 + c2 * c2) % 3))
        digit = torch.stack((c0, c1, c2))
        less = (digit[:, :, None] - digit[:, None, :]) % 3
        diff = less[0] + 3 * less[1] + 9 * less[2]
    else:
        squares = e * e % q
        diff = (e[:, None] - e[None, :]) % q
    is_square = torch.zeros(q, device="cuda").index_fill(0, squares, 1.0)
    chi = 2.0 * is_square[diff] - 1.0
    h = torch.ones((m, m), device="cuda")
    h[1:, 0] = -1.0
    h[1:, 1:] = torch.where(diff == 0, 1.0, chi)
    return h


def _rotated(x, m, channel, sigma):
    """(x H / sqrt n) * sigma H[channel] in binary32, H the outer factor times a Sylvester matrix."""
    t, n = x.shape
    inner = n // m
    a, b = _outer(m), _sylvester(inner)
    y = (x.reshape(t * m, inner) @ b).reshape(t, m, inner)
    y = torch.matmul(a.T.contiguous(), y)
    d = sigma * (a[channel // inner][:, None] * b[channel % inner][None, :])
    return (y * d).reshape(t, n) * (1.0 / math.sqrt(n))


def _headed(x, weight, bias, case, cos, sin):
    """The norm of each head and the rotation of its first channels, in binary32."""
    x = x.float()
    if case["norm"] == "layer":
        x = x - x.mean(dim=2, keepdim=True)
    if case["norm"] != "none":
        x = x * torch.rsqrt((x * x).mean(dim=2, keepdim=True) + EPS) * weight.float()
        x = x if bias is None else x + bias.float()
    r = case["rotary"]
    if case["interleaved"]:
        a, b = x[:, :, 0:r:2], x[:, :, 1:r:2]
    else:
        a, b = x[:, :, :r // 2], x[:, :, r // 2:r]
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack((a, b), dim=3).flatten(2) if case["interleaved"] else torch.cat((a, b), dim=2)
    return torch.cat((turned, x[:, :, r:]), dim=2).to(_TYPES[case["in"]])


def _plain(s):
    case = s["case"]
    if case["op"] == "quant":
        v, e = _quantize(s["x"].float(), case["rule"])
        y = (v * _pow2(e)[:, :, None]).reshape(case["tokens"], -1)[:, :case["n"]]
        return y.to(torch.bfloat16), (e + 127).to(torch.uint8)
    if case["op"] == "linear":
        out = _values(s["codes"], s["scale"]) @ _values(s["w"], s["w_scale"]).T
        out = out if s["bias"] is None else out + s["bias"]
        return out.to(_TYPES[case["out"]])
    if case["op"] == "down":
        if case["swiglu"]:
            gate = s["gate"].float()
            x = (gate / (1.0 + torch.exp(-gate)) * s["up"].float()).to(torch.bfloat16)
        else:
            x = s["x"]
        v, e = _quantize(_rotated(x.float(), ROTATED[case["n"]], s["channel"], s["sigma"]), "floor")
        y = (v * _pow2(e)[:, :, None]).reshape(case["tokens"], case["n"])
        return (y @ _values(s["w"], s["w_scale"]).T).to(torch.bfloat16)
    at = s["positions"].long()
    cos, sin = s["cos"][at][:, None, :], s["sin"][at][:, None, :]
    return (_headed(s["q"], s["q_weight"], s["q_bias"], case, cos, sin),
            _headed(s["k"], s["k_weight"], s["k_bias"], case, cos, sin))


def _own(s):
    import rotation_activation_quantization_amd as R

    case = s["case"]
    if case["op"] == "quant":
        codes, scale = R.quant_mxfp4(s["x"], rule=case["rule"])
        return R.dequant_mxfp4(codes, scale, n=case["n"], dtype=torch.bfloat16), scale
    if case["op"] == "linear":
        return R.mxfp4_linear(s["codes"], s["scale"], s["w"], s["w_scale"], bias=s["bias"], dtype=_TYPES[case["out"]])
    if case["op"] == "down":
        if case["swiglu"]:
            codes, scale = R.swiglu_rotate_quant_mxfp4(s["gate"], s["up"], s["channel"], s["sigma"])
        else:
            codes, scale = R.rotate_quant_mxfp4(s["x"], s["channel"], s["sigma"])
        return R.mxfp4_linear(codes, scale, s["w"], s["w_scale"])
    return R.qk_norm_rope(s["q"], s["k"], s["cos"], s["sin"], s["positions"], norm=case["norm"], eps=EPS,
                          q_weight=s["q_weight"], k_weight=s["k_weight"], q_bias=s["q_bias"], k_bias=s["k_bias"],
                          interleaved=case["interleaved"])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what one pass cannot do without ----------------------------------------


def work(case):
    t = case["tokens"]
    if case["op"] == "quant":
        n, blocks = case["n"], (case["n"] + 31) // 32
        size = 2 if case["in"] == "bf16" else 4
        return {"bytes": t * n * size + 2 * t * n + t * blocks, "flops": 4 * t * n}
    if case["op"] == "qk":
        heads, d, r = case["q_heads"] + case["k_heads"], case["head"], case["rotary"]
        size = 2 if case["in"] == "bf16" else 4
        params = 2 * {"none": 0, "rms": 2, "layer": 4}[case["norm"]] * d
        return {"bytes": 2 * t * heads * d * size + 4 * t * r + 4 * t + params, "flops": 8 * t * heads * d}
    n, rows = case["n"], case["rows"]
    packed = n // 2 + n // 32  # bytes of a row
    if case["op"] == "linear":
        size = 2 if case["out"] == "bf16" else 4
        return {"bytes": (t + rows) * packed + size * t * rows + (4 * rows if case["bias"] else 0),
                "flops": 2 * t * n * rows}
    wide = 4 if case["swiglu"] else 2
    return {"bytes": t * n * wide + rows * packed + 2 * t * rows,
            "flops": 2 * t * n * rows + t * n * (ROTATED[n] + int(math.log2(n // ROTATED[n])))}


# ---- the definition in 64 bits -----------------------------------------------

_LEVELS = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def exact(case, seed):
    s = prepare(case, seed)
    t = case["tokens"]
    levels = torch.tensor(_LEVELS, dtype=torch.float64, device="cuda")

    def power(e):
        """2^e, exactly (a library's power of two may be off by a rounding)."""
        return ((e.long() + 1023) << 52).view(torch.float64)

    def nearest(y, rule):
        """The MXFP4 values of y [T, n], and the exponents: nearest level of each value, the even code at a tie."""
        n = y.shape[1]
        b = torch.zeros((t, (n + 31) // 32 * 32), dtype=torch.float64, device="cuda")
        b[:, :n] = y
        b = b.view(t, -1, 32)
        top = b.abs().max(dim=2).values
        e = (top.view(torch.int64) >> 52) - 1023 - 2  # top >= 0: the exponent's bits alone
        if rule == "noclip":
            e += (top > 6.0 * power(e.clamp(min=-200))).long()
        e = e.clamp(min=-127)
        unit = power(e)
        u = b.abs() / unit[:, :, None]
        best = torch.zeros_like(u)
        for i in range(1, 8):
            half = (_LEVELS[i - 1] + _LEVELS[i]) / 2  # to level i above it, and at it where i is even
            best = torch.where((u > half) | ((u == half) if i % 2 == 0 else torch.zeros_like(u, dtype=torch.bool)),
                               levels[i], best)
        return (torch.copysign(best, b) * unit[:, :, None]).reshape(t, -1)[:, :n], e

    def dense(codes, scale):
        c = torch.empty((codes.shape[0], 2 * codes.shape[1]), dtype=torch.int64, device="cuda")
        c[:, 0::2] = (codes % 16).long()
        c[:, 1::2] = (codes // 16).long()
        signed = torch.cat((levels, -levels))[c]
        return signed * torch.repeat_interleave(power(scale.long() - 127), 32, dim=1)

    def hadamard(m):
        """The outer factor, entry by entry from the quadratic character."""
        if m == 1:
            return torch.ones((1, 1), dtype=torch.float64, device="cuda")
        q = m - 1
        p = 3 if q == 27 else q

        def digits(a):
            return [a % p, a // p % p, a // (p * p) % p] if q == 27 else [a]

        def times(a, b):
            if q != 27:
                return a * b % q
            out = [0] * 5
            for i, u in enumerate(digits(a)):
                for j, v in enumerate(digits(b)):
                    out[i + j] += u * v
            for k in (4, 3):  # t^k = t^(k - 3) (t + 2)
                out[k - 2] += out[k]
                out[k - 3] += 2 * out[k]
            return sum(p ** k * (out[k] % p) for k in range(3))

        def minus(a, b):
            return sum(p ** k * ((u - v) % p) for k, (u, v) in enumerate(zip(digits(a), digits(b))))

        squares = {times(a, a) for a in range(1, q)}
        rows = [[1.0] * m]
        for a in range(q):
            rows.append([-1.0] + [1.0 if a == b or minus(a, b) in squares else -1.0 for b in range(q)])
        return torch.tensor(rows, dtype=torch.float64, device="cuda")

    if case["op"] == "quant":
        y, _ = nearest(s["x"].double(), case["rule"])
        return y, None
    if case["op"] == "linear":
        out = torch.matmul(dense(s["codes"], s["scale"]), dense(s["w"], s["w_scale"]).T.contiguous())
        return out if s["bias"] is None else out + s["bias"].double()
    if case["op"] == "down":
        n, m = case["n"], ROTATED[case["n"]]
        if case["swiglu"]:
            gate = s["gate"].double()
            x = (gate * torch.sigmoid(gate) * s["up"].double()).to(torch.bfloat16).double()
        else:
            x = s["x"].double()
        unit = torch.zeros((1, n), dtype=torch.float64, device="cuda")
        unit[0, s["channel"]] = s["sigma"]  # its transform is sigma H[channel]
        y = torch.cat((x, unit)).view(-1, m, n // m)
        half = n // m // 2
        while half:  # the transform over the powers of two, one bit at a time
            z = y.view(-1, m, n // m // (2 * half), 2, half)
            y = torch.stack((z[:, :, :, 0] + z[:, :, :, 1], z[:, :, :, 0] - z[:, :, :, 1]), dim=3).view(-1, m, n // m)
            half //= 2
        y = torch.matmul(hadamard(m).T.contiguous(), y).view(-1, n)
        y, _ = nearest(y[:-1] * y[-1:] / math.sqrt(n), "floor")
        return torch.matmul(y, dense(s["w"], s["w_scale"]).T.contiguous())

    def turned(x, weight, bias):
        x = x.double()
        if case["norm"] != "none":
            if case["norm"] == "layer":
                x = x - x.sum(dim=2, keepdim=True) / case["head"]
            x = weight.double() * (x / (x.pow(2).sum(dim=2, keepdim=True) / case["head"] + EPS).sqrt())
            if bias is not None:
                x = x + bias.double()
        out, r = x.clone(), case["rotary"]
        for i in range(r // 2):
            a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + r // 2)
            c, z = (s[name].double()[s["positions"].long(), i][:, None] for name in ("cos", "sin"))
            out[:, :, a] = x[:, :, a] * c - x[:, :, b] * z
            out[:, :, b] = x[:, :, a] * z + x[:, :, b] * c
        return out

    return turned(s["q"], s["q_weight"], s["q_bias"]), turned(s["k"], s["k_weight"], s["k_bias"])
