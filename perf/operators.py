"""The workloads by which the INT8 operators and the residual norms are measured.

Three paths of a quantized transformer block:

  norm   the norm after a block, its gate and scale, the residual sum and the
         norm before the next block, in one pass
             h' = beta h + alpha g * Norm_post(y)
             u  = Norm_pre(h') * (1 + m_scale) + m_shift
         With "quant", u leaves as per-token INT8 codes that go straight into
         the next product.
  w8a8   per-token INT8 activations times per-channel INT8 weights
             out[t][k] = s_t v_k sum_j q_tj w_kj + b_k
         from bf16 activations: the quantizer and the product.
  w8a4   the rotated INT4 activations (codes, scale, zero-point) times
         per-channel INT8 weights
             out[t][k] = s_t v_k sum_j (q_tj - z_t) w_kj + b_k

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


def listed():
    return [
        # decode: the norms around one token's attention block
        {"name": "norm_t1_n4096", "op": "norm", "tokens": 1, "n": 4096, "norm": "rms", "stream": "bf16",
         "mods": "none", "rows": 0},
        # packed sequences of different lengths, LayerNorm with biases, each sequence with its own gate, scale and
        # shift, the residual stream held in binary32
        {"name": "norm_t1237_n5120", "op": "norm", "tokens": 1237, "n": 5120, "norm": "layer", "stream": "f32",
         "mods": "sequence", "rows": 0},
        # a prompt batch at the widest hidden size, RMS norms, a per-channel gate
        {"name": "norm_t8192_n8192", "op": "norm", "tokens": 8192, "n": 8192, "norm": "rms", "stream": "bf16",
         "mods": "channel", "rows": 0},
        # a small decode batch: norms with INT8 output, then the gate projection
        {"name": "normq_t4_n8192_r28672", "op": "norm", "tokens": 4, "n": 8192, "norm": "rms", "stream": "bf16",
         "mods": "none", "rows": 28672},
        # the same on a prompt
        {"name": "normq_t2048_n4096_r14336", "op": "norm", "tokens": 2048, "n": 4096, "norm": "rms",
         "stream": "bf16", "mods": "channel", "rows": 14336},
        # one token through a quantized up projection
        {"name": "w8a8_t1_n4096_r14336", "op": "w8a8", "tokens": 1, "n": 4096, "rows": 14336, "out": "bf16",
         "bias": False},
        # odd sizes in every direction: no tile, vector or row ends where the data does
        {"name": "w8a8_t613_n1111_r777", "op": "w8a8", "tokens": 613, "n": 1111, "rows": 777, "out": "f32",
         "bias": True},
        # a prompt batch through an up projection
        {"name": "w8a8_t8192_n4096_r14336", "op": "w8a8", "tokens": 8192, "n": 4096, "rows": 14336, "out": "bf16",
         "bias": False},
        # the down projection on the rotated codes: one token
        {"name": "w8a4_t1_n14336_r4096", "op": "w8a4", "tokens": 1, "n": 14336, "rows": 4096, "out": "bf16",
         "bias": False},
        # a decode batch at the widest down projection
        {"name": "w8a4_t16_n28672_r8192", "op": "w8a4", "tokens": 16, "n": 28672, "rows": 8192, "out": "bf16",
         "bias": False},
        # a short prompt whose length fills no tile
        {"name": "w8a4_t200_n11008_r4096", "op": "w8a4", "tokens": 200, "n": 11008, "rows": 4096, "out": "f32",
         "bias": True},
        # a prompt batch
        {"name": "w8a4_t8192_n14336_r4096", "op": "w8a4", "tokens": 8192, "n": 14336, "rows": 4096, "out": "bf16",
         "bias": False},
    ]


_MOST = 8000 * 14336 * 4096  # products of one drawn pass


def _log(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(("norm", "w8a8", "w8a4"))
    tokens = _log(rng, 1, 8192)
    if rng.random() < 0.3:
        tokens = rng.choice((1, 2, 4, 16, 64))
    if op == "norm":
        n = rng.choice(HIDDEN) if rng.random() < 0.5 else _log(rng, 64, 8192)
        rows = 0 if rng.random() < 0.6 else rng.choice(INNER)
        tokens = max(1, min(tokens, _MOST // (n * max(rows, 1))))
        return {"op": op, "tokens": tokens, "n": n,
                "norm": rng.choice(("rms", "layer")), "stream": rng.choice(("bf16", "f32")),
                "mods": rng.choice(("none", "channel", "sequence")), "rows": rows}
    if rng.random() < 0.6:
        n, rows = rng.choice(HIDDEN), rng.choice(INNER)
        if op == "w8a4":
            n, rows = rows, n
    else:
        n, rows = _log(rng, 64, 16384), _log(rng, 64, 16384)
    if op == "w8a4":
        n += n % 2  # two codes to a byte
    tokens = max(1, min(tokens, _MOST // (n * rows)))
    return {"op": op, "tokens": tokens, "n": n, "rows": rows, "out": rng.choice(("bf16", "f32")),
            "bias": rng.random() < 0.5}


# ---- inputs ----------------------------------------------------------------


def _weights(gen, rows, n):
    """INT8 weights of a trained projection, quantized offline for each output channel."""
    w = torch.randn((rows, n), generator=gen, device="cuda")
    w *= (torch.rand((rows, 1), generator=gen, device="cuda") + 0.5) / math.sqrt(n)
    top = w.abs().amax(dim=1, keepdim=True)
    q = torch.round(w * 127.0 / top).to(torch.int8)
    return q, (top / 127.0).reshape(rows)


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    t, n, rows = case["tokens"], case["n"], case["rows"]

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    s = {"case": dict(case)}
    if case["op"] == "norm":
        layer = case["norm"] == "layer"
        h = normal(t, n) * 2.0
        h[:, n // 3] *= 40.0  # the residual stream's massive channel
        s["h"] = h if case["stream"] == "f32" else h.to(torch.bfloat16)
        s["y"] = (normal(t, n) * 0.5).to(torch.bfloat16)
        for name in ("post", "pre"):
            s[name + "_weight"] = (1.0 + 0.1 * normal(n)).to(torch.bfloat16)
            s[name + "_bias"] = (0.1 * normal(n)).to(torch.bfloat16) if layer else None
        s["alpha"], s["beta"] = (0.7, 1.0) if case["mods"] != "none" else (1.0, 1.0)
        s["gate"] = s["mod_scale"] = s["mod_shift"] = s["index"] = None
        if case["mods"] == "channel":
            s["gate"] = (0.5 + 0.2 * normal(n)).to(torch.bfloat16)
        elif case["mods"] == "sequence":
            seqs = min(t, 7)
            cuts = torch.randint(0, t, (seqs - 1,), generator=gen, device="cuda") if seqs > 1 else None
            where = torch.arange(t, device="cuda")
            s["index"] = torch.zeros(t, dtype=torch.int32, device="cuda")
            if cuts is not None:
                s["index"] = (where[:, None] >= cuts[None, :]).sum(dim=1).to(torch.int32)
            for name in ("gate", "mod_scale", "mod_shift"):
                s[name] = (0.3 * normal(seqs, n)).to(torch.bfloat16)
    elif case["op"] == "w8a8":
        x = normal(t, n) * (0.2 + torch.rand((t, 1), generator=gen, device="cuda"))
        x[:, n // 2] *= 20.0
        s["x"] = x.to(torch.bfloat16)
    else:
        # what the rotation's quantizer gives: bell-shaped codes, zero-points near the middle and, on the tokens
        # with a massive outlier, far outside of the codes' range
        q = torch.round(normal(t, n) * 2.2 + 7.5).clamp_(0, 15).to(torch.uint8)
        s["codes"] = (q[:, 0::2] | (q[:, 1::2] << 4)).contiguous()
        s["scale"] = torch.rand(t, generator=gen, device="cuda") * 0.3 + 0.1
        heavy = (torch.rand(t, generator=gen, device="cuda") < 0.2).float()
        s["zero"] = 7.5 + normal(t) * 0.5 - heavy * 60.0
    if rows:
        s["w"], s["w_scale"] = _weights(gen, rows, n)
        if case["op"] == "w8a4":
            s["w_sum"] = s["w"].sum(dim=1, dtype=torch.int32)
        s["bias"] = normal(rows) * 0.1 if case.get("bias") else None
    return s


# ---- one pass --------------------------------------------------------------

_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _norm(x, kind, weight, bias):
    if kind == "layer":
        x = x - x.mean(dim=1, keepdim=True)
    x = x * torch.rsqrt((x * x).mean(dim=1, keepdim=True) + EPS) * weight.float()
    return x if bias is None else x + bias.float()


def _per_token(mod, index):
    return mod.float() if index is None else mod.float()[index.long()]


def _quantize(u):
    """INT8 codes and scales of binary32 rows."""
    top = u.abs().amax(dim=1, keepdim=True)
    scale = torch.where(top > 0, top / 127.0, torch.ones_like(top))
    q = torch.round(u * 127.0 / torch.where(top > 0, top, torch.ones_like(top)))
    return q, scale


def _plain(s):
    case = s["case"]
    if case["op"] == "norm":
        branch = _norm(s["y"].float(), case["norm"], s["post_weight"], s["post_bias"])
        if s["gate"] is not None:
            branch = branch * _per_token(s["gate"], s["index"])
        h = s["beta"] * s["h"].float() + s["alpha"] * branch
        u = _norm(h, case["norm"], s["pre_weight"], s["pre_bias"])
        if s["mod_scale"] is not None:
            u = u * (1.0 + _per_token(s["mod_scale"], s["index"])) + _per_token(s["mod_shift"], s["index"])
        h = h.to(s["h"].dtype)
        if not case["rows"]:
            return h, u.to(torch.bfloat16)
        q, scale = _quantize(u)
        out = (q @ s["w"].float().T) * scale * s["w_scale"]
        return h, out.to(torch.bfloat16)
    if case["op"] == "w8a8":
        q, scale = _quantize(s["x"].float())
        out = (q @ s["w"].float().T) * scale * s["w_scale"]
    else:
        q = torch.stack((s["codes"] & 15, s["codes"] >> 4), dim=2).reshape(case["tokens"], case["n"]).float()
        y = s["scale"][:, None] * (q - s["zero"][:, None])
        out = (y @ s["w"].float().T) * s["w_scale"]
    if s["bias"] is not None:
        out = out + s["bias"]
    return out.to(_TYPES[case["out"]])


def _own(s):
    import rotation_activation_quantization_amd as R

    case = s["case"]
    if case["op"] == "norm":
        named = {"norm": case["norm"], "eps": EPS, "post_weight": s["post_weight"], "post_bias": s["post_bias"],
                 "gate": s["gate"], "alpha": s["alpha"], "beta": s["beta"], "weight": s["pre_weight"],
                 "bias": s["pre_bias"], "mod_scale": s["mod_scale"], "mod_shift": s["mod_shift"],
                 "mod_index": s["index"]}
        if not case["rows"]:
            return R.residual_norm(s["h"], s["y"], **named)
        h, codes, scale = R.residual_norm_quant_int8(s["h"], s["y"], **named)
        return h, R.int8_linear(codes, scale, s["w"], s["w_scale"])
    if case["op"] == "w8a8":
        codes, scale = R.quant_int8(s["x"])
        return R.int8_linear(codes, scale, s["w"], s["w_scale"], bias=s["bias"], dtype=_TYPES[case["out"]])
    return R.int4_w8_linear(s["codes"], s["scale"], s["zero"], s["w"], s["w_scale"], s["w_sum"], bias=s["bias"],
                            dtype=_TYPES[case["out"]])


def run(state):
    return _own(state) if own else _plain(state)


# ---- what one pass cannot do without ----------------------------------------


def work(case):
    t, n, rows = case["tokens"], case["n"], case["rows"]
    if case["op"] == "norm":
        stream = 2 if case["stream"] == "bf16" else 4
        params = (4 if case["norm"] == "layer" else 2) * 2 * n
        params += {"none": 0, "channel": 2 * n, "sequence": 3 * min(t, 7) * 2 * n + 4 * t}[case["mods"]]
        total = t * n * (2 * stream + 2) + params  # h in and out, y
        ops = 16 * t * n
        if not rows:
            return {"bytes": total + 2 * t * n, "flops": ops}
        return {"bytes": total + rows * n + 4 * rows + 2 * t * rows, "flops": ops + 2 * t * n * rows}
    size = 2 if case["out"] == "bf16" else 4
    total = rows * n + 4 * rows + size * t * rows + (4 * rows if case["bias"] else 0)
    if case["op"] == "w8a8":
        return {"bytes": total + 2 * t * n, "flops": 2 * t * n * rows + 4 * t * n}
    return {"bytes": total + t * n // 2 + 8 * t + 4 * rows, "flops": 2 * t * n * rows}


# ---- the definition in 64 bits -----------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    t, n = case["tokens"], case["n"]

    def rows_of(name):
        m = s[name]
        if m is None:
            return None
        m = m.double()
        return m[s["index"].long()] if m.dim() == 2 else m[None, :]

    def normed(x, which):
        centre = x.sum(dim=1, keepdim=True) / n if case["norm"] == "layer" else 0.0
        x = x - centre
        var = x.pow(2).sum(dim=1, keepdim=True) / n
        x = s[which + "_weight"].double() * (x / (var + EPS).sqrt())
        return x if s[which + "_bias"] is None else x + s[which + "_bias"].double()

    def product(q, scale):
        """scale * v * (q . w): whole numbers in 64 bits, so the sum is exact."""
        return scale[:, None] * (s["w_scale"].double() * torch.matmul(q, s["w"].double().T.contiguous()))

    def codes_of(u):
        top = u.abs().max(dim=1).values
        some = top > 0
        step = torch.where(some, top, torch.full_like(top, 127.0)) / 127.0
        return (u * 127.0 / torch.where(some, top, torch.ones_like(top))[:, None]).round(), step

    if case["op"] == "norm":
        branch, gate = normed(s["y"].double(), "post"), rows_of("gate")
        h = s["beta"] * s["h"].double() + s["alpha"] * (branch if gate is None else gate * branch)
        u, m_scale = normed(h, "pre"), rows_of("mod_scale")
        if m_scale is not None:
            u = u + u * m_scale + rows_of("mod_shift")
        if not case["rows"]:
            return h, u
        q, step = codes_of(u)
        return h, product(q, step)
    if case["op"] == "w8a8":
        q, step = codes_of(s["x"].double())
        out = product(q, step)
    else:
        q = torch.empty((t, n), dtype=torch.float64, device="cuda")
        q[:, 0::2] = (s["codes"] % 16).double()
        q[:, 1::2] = (s["codes"] // 16).double()
        whole = s["w"].double().sum(dim=1)
        out = product(q, s["scale"].double())
        out -= (s["scale"].double() * s["zero"].double())[:, None] * (s["w_scale"].double() * whole)
    return out if s["bias"] is None else out + s["bias"].double()
