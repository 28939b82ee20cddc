"""signrot_residual_norm against the float64 definition.

Tolerance, from u = 2^-24 and the depth of a sum (a thread adds at most n / 64
values, the threads' sums meet in at most 16 steps: L = n / 64 + 16 roundings
on the longest path), to first order with 1.1 for the rest:

  statistics of x with input errors dx (absolute, per element):
    dmean = mean |dx| + L u mean |x|  (layer)
    dinv / inv = (sum |x - mean| (|dx| + dmean) / n) inv^2 + (L / 2 + 4) u
  a norm's value v = (x - mean) inv w + b:
    dv = |w| inv (|dx| + dmean + 2u |x - mean|) + |v - b| (dinv / inv + 2u) + u |v|
  h' = beta h + alpha g v:  dh = |alpha g| dv + 4u (|beta h| + |alpha g v|)
  u: the norm's dv with x = h', dx = dh, then |1 + m| dv + 4u (|v (1 + m)| + |c|)

and half a unit in the last place of the output's type (2^-8 relative for bf16, 8 significant bits,
2^-24 for float32).  A code may differ from rint(127 u / a) only by what moves
127 u / a over a rounding boundary: |code - 127 u / a| <= 1/2 + 127 (du + da) / a
+ 4u 127, da = max du.
"""

import numpy as np
import pytest

torch = pytest.importorskip("torch")

import rotation_activation_quantization_amd as R  # noqa: E402
from oracle import block_oracle as B  # noqa: E402

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: 2.0 ** -24}


def norm_error(x, dx, kind, eps, w, b):
    n = x.shape[1]
    if kind == "none":
        return x, dx
    depth = n / 64 + 16
    mean, inv = B.norm_parts(x, kind, eps)
    dmean = 0.0
    if kind == "layer":
        dmean = dx.mean(axis=1, keepdims=True) + depth * U * np.abs(x).mean(axis=1, keepdims=True)
    c = np.abs(x - mean)
    rel = (c * (dx + dmean)).mean(axis=1, keepdims=True) * inv ** 2 + (depth / 2 + 4) * U
    v = B.normed(x, kind, eps, w, b)
    part = v if b is None else v - b
    aw = 1.0 if w is None else np.abs(w)
    return v, aw * inv * (dx + dmean + 2 * U * c) + np.abs(part) * (rel + 2 * U) + U * np.abs(v)


def reference(a):
    """(h', dh, u, du) of the arguments dict (float64 arrays, modulations spread to rows)."""
    h = a["h"]
    hp, dh = a["beta"] * h, U * np.abs(a["beta"] * h)
    if a["y"] is not None:
        v, dv = norm_error(a["y"], np.zeros_like(a["y"]), a["post_norm"], a["post_eps"], a["post_weight"], a["post_bias"])
        g = a["alpha"] * (1.0 if a["gate"] is None else a["gate"])
        hp = hp + g * v
        dh = np.abs(g) * dv + 4 * U * (np.abs(a["beta"] * h) + np.abs(g * v))
    v, dv = norm_error(hp, dh, a["norm"], a["eps"], a["weight"], a["bias"])
    m = 1.0 if a["mod_scale"] is None else 1.0 + a["mod_scale"]
    c = 0.0 if a["mod_shift"] is None else a["mod_shift"]
    u = v * m + c
    du = np.abs(m) * dv + 4 * U * (np.abs(v * m) + np.abs(c))
    return hp, 1.1 * dh, u, 1.1 * du


ORACLE_KEYS = ("norm", "post_norm", "eps", "post_eps", "post_weight", "post_bias", "gate", "alpha", "beta", "weight",
               "bias", "mod_scale", "mod_shift")


def case(t, n, seed=0, norm="rms", post_norm=None, stream=torch.bfloat16, param=torch.bfloat16, bias=False, mods=None,
         branch=True, alpha=0.75, beta=1.25, eps=1e-5, post_eps=1e-6, weight=True):
    """(tensors for the call, float64 arguments for the reference)."""
    g = np.random.default_rng([13, t, n, seed])

    def draw(shape, loc=0.0, size=1.0, dtype=param):
        return torch.from_numpy(loc + size * g.standard_normal(shape)).to(dtype)

    call = {"h": draw((t, n), 0.3, 2.0, stream), "y": draw((t, n), -0.2, 0.7, torch.bfloat16) if branch else None,
            "post_weight": draw(n, 1.0, 0.2) if weight else None, "weight": draw(n, 1.0, 0.2) if weight else None,
            "post_bias": draw(n, 0, 0.3) if bias else None, "bias": draw(n, 0, 0.3) if bias else None,
            "gate": None, "mod_scale": None, "mod_shift": None, "mod_index": None}
    call["h"][:, n // 2] *= 50
    index = None
    if mods == "channel":
        call["gate"], call["mod_shift"] = draw(n, 0.5, 0.3), draw(n, 0, 0.3)
    elif mods in ("token", "index"):
        m = t if mods == "token" else 3
        for k in ("gate", "mod_scale", "mod_shift"):
            call[k] = draw((m, n), 0, 0.4)
        if mods == "index":
            index = g.integers(0, m, t).astype(np.int32)
            call["mod_index"] = torch.from_numpy(index)
    opts = {"norm": norm, "post_norm": norm if post_norm is None else post_norm, "eps": eps, "post_eps": post_eps,
            "alpha": alpha, "beta": beta}
    ref = {k: None if v is None else v.double().numpy() for k, v in call.items() if k != "mod_index"}
    for k in ("gate", "mod_scale", "mod_shift"):
        if ref[k] is not None:
            ref[k] = ref[k][None, :] if ref[k].ndim == 1 else (ref[k] if index is None else ref[k][index])
    return {k: None if v is None else v.cuda() for k, v in call.items()}, opts, {**ref, **opts}


def within(got, ref, tol, dtype, label):
    tol = tol + HALF[dtype] * 1.01 * (np.abs(ref) + tol) + 1e-37
    over = np.abs(got.double().cpu().numpy() - ref) / tol
    print(f"[gpu] {label}: worst {over.max():.3f} of the tolerance", flush=True)
    assert over.max() <= 1.0, label


def check(t, n, **kw):
    call, opts, a = case(t, n, **kw)
    hp, dh, u, du = reference(a)
    defined, same = B.residual_norm(a["h"], a["y"], **{k: a[k] for k in ORACLE_KEYS})
    assert np.allclose(defined, hp) and np.allclose(same, u)
    label = f"residual_norm {t} x {n} {kw}"
    h_out, got = R.residual_norm(**call, **opts)
    assert h_out.dtype == call["h"].dtype and got.dtype == torch.bfloat16
    within(h_out, hp, dh, h_out.dtype, label + " h")
    within(got, u, du, torch.bfloat16, label + " u")
    h2, codes, scale = R.residual_norm_quant_int8(**call, **opts)
    assert torch.equal(h2, h_out)
    top, dtop = np.abs(u).max(axis=1, keepdims=True), du.max(axis=1, keepdims=True)
    within(scale[:, None], np.where(top > 0, top / 127, 1.0), dtop / 127 + 2 * U * top, torch.float32, label + " scale")
    q = codes.cpu().numpy().astype(np.float64)
    safe = np.where(top > 0, top, 1.0)
    band = 0.5 + 127 * (du + dtop) / safe + 4 * U * 127
    assert (np.abs(q - 127 * u / safe) <= band).all(), label
    # nearly every code is the definition's own
    assert (q != np.rint(127 * u / safe)).mean() <= 2e-3 + 2.0 / q.size, label


WIDTHS = [1, 2, 7, 8, 63, 64, 72, 127, 256, 504, 512, 1000, 1024, 1111, 2048, 2056, 4096, 5120, 8192, 8200, 11008, 14336,
          16384, 28672, 32768, 32776, 40000]


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("n", WIDTHS)
def test_widths(n, norm):
    check(3, n, norm=norm, bias=norm == "layer", mods="channel")


def test_widest_row():
    check(1, 131071, norm="layer", stream=torch.float32)


@pytest.mark.parametrize("t", [1, 2, 5, 64, 129, 1023, 2500])
@pytest.mark.parametrize("n", [128, 1000, 4096])
def test_token_counts(t, n):
    check(t, n, mods="index")


@pytest.mark.parametrize("norm,post", [("rms", "none"), ("none", "rms"), ("layer", "rms"), ("rms", "layer"),
                                       ("none", "none")])
@pytest.mark.parametrize("n", [96, 1111, 4096])
def test_norm_kinds(norm, post, n):
    check(4, n, norm=norm, post_norm=post, bias=True)


@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("param", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("mods", [None, "channel", "token", "index"])
@pytest.mark.parametrize("n", [640, 1003, 5120])
def test_types_and_modulations(stream, param, mods, n):
    check(6, n, stream=stream, param=param, mods=mods, bias=True, norm="layer")


@pytest.mark.parametrize("n", [64, 1111, 4096, 8192])
def test_without_branch_or_weights(n):
    check(5, n, branch=False)
    check(5, n, branch=False, weight=False, beta=1.0, norm="layer")
    check(5, n, weight=False)


@pytest.mark.parametrize("n", [512, 1000, 8192])
def test_in_place_stream(n):
    call, opts, _ = case(9, n, mods="index")
    h_out, u = R.residual_norm(**call, **opts)
    h = call["h"].clone()
    h2, u2 = R.residual_norm(**{**call, "h": h}, **opts, h_out=h)
    assert h2 is h and torch.equal(h, h_out) and torch.equal(u, u2)


@pytest.mark.parametrize("n,ldh,offh,ldy,offy,ldo,offo", [(1024, 1032, 8, 1040, 16, 1024, 0), (1024, 1025, 1, 1024, 0, 1030, 3),
                                                          (100, 101, 0, 104, 4, 100, 1), (4096, 4100, 2, 4097, 5, 4104, 8)])
@pytest.mark.parametrize("stream", [torch.bfloat16, torch.float32])
def test_strides_offsets_and_guards(n, ldh, offh, ldy, offy, ldo, offo, stream):
    t = 5
    call, opts, _ = case(t, n, stream=stream, mods="token", bias=True)

    def place(v, ld, off, fill=9.0):
        buf = torch.full((off + t * ld,), fill, dtype=v.dtype, device="cuda")
        view = buf[off:].view(t, ld)[:, :n]
        view.copy_(v)
        return buf, view

    want_h, want_u = R.residual_norm(**call, **opts)
    _, want_q, want_s = R.residual_norm_quant_int8(**call, **opts)
    _, h = place(call["h"], ldh, offh)
    _, y = place(call["y"], ldy, offy)
    bh, ho = place(torch.zeros_like(call["h"]), ldo, offo)
    bu, uo = place(torch.zeros_like(want_u), ldo, offo)
    bq, qo = place(torch.zeros_like(want_q), ldo, offo, 9)
    mods = {k: place(call[k], ldy, offy)[1] for k in ("mod_scale", "mod_shift")}
    mods["gate"] = place(call["gate"], ldh, offh)[1]
    args = {**call, **opts, "h": h, "y": y, **mods}
    R.residual_norm(**args, h_out=ho, out=uo)
    scale = torch.empty(t, device="cuda")
    R.residual_norm_quant_int8(**args, h_out=ho, out=(qo, scale))
    # the sums of another layout may be added in another order: a rounding step apart at most
    step = 2.0 ** -7 if stream == torch.bfloat16 else 2.0 ** -20
    assert torch.allclose(ho.float(), want_h.float(), rtol=step, atol=1e-5)
    assert torch.allclose(uo.float(), want_u.float(), rtol=2.0 ** -7, atol=1e-5)
    assert (qo.int() - want_q.int()).abs().max() <= 1 and torch.allclose(scale, want_s, rtol=1e-5)
    for buf, view in ((bh, ho), (bu, uo), (bq, qo)):
        keep = torch.ones_like(buf, dtype=torch.bool)
        keep[offo:].view(t, ldo)[:, :n] = False
        assert (buf[keep] == 9).all()


def test_index_outside_is_clamped():
    call, opts, _ = case(4, 256, mods="index")
    call["mod_index"] = torch.tensor([-5, 0, 2, 1000000], dtype=torch.int32, device="cuda")
    got = R.residual_norm(**call, **opts)
    call["mod_index"] = torch.tensor([0, 0, 2, 2], dtype=torch.int32, device="cuda")
    want = R.residual_norm(**call, **opts)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_zero_and_non_finite_rows():
    for n in (320, 1111, 4096):
        call, opts, _ = case(5, n, weight=False)
        want = R.residual_norm_quant_int8(**call, **opts)
        call["h"][1] = 0.0
        call["y"][1] = 0.0
        call["h"][2, 5] = float("inf")
        call["y"][3, n - 1] = float("nan")
        h_out, codes, scale = R.residual_norm_quant_int8(**call, **opts)
        assert (h_out[1] == 0).all() and (codes[1] == 0).all() and scale[1] == 1.0
        assert not torch.isfinite(scale[2]) and not torch.isfinite(scale[3])
        for r in (0, 4):
            for a, b in zip((h_out, codes, scale), want):
                assert torch.equal(a[r], b[r])


def test_large_offset_layer_norm_keeps_the_variance():
    """A row far from zero: the centred sum of squares does not cancel."""
    n = 4096
    g = np.random.default_rng(21)
    h = torch.from_numpy((3000.0 + g.standard_normal((3, n))).astype(np.float32)).cuda()
    _, u = R.residual_norm(h, norm="layer")
    v = h.double()
    v = v - v.mean(dim=1, keepdim=True)
    ref = v / (v.pow(2).mean(dim=1, keepdim=True) + 1e-6).sqrt()
    # mean: L u |x| / sd = (64 + 16) 2^-24 3000 = 0.0143; half a bf16 unit of values below 8: 2^-6
    assert (u.double() - ref).abs().max() <= 0.0143 + 2.0 ** -6


def test_rows_beyond_two_gib():
    t, n = 300000, 8192
    h = torch.zeros((t, n), dtype=torch.bfloat16, device="cuda")
    rows = torch.tensor([0, 131071, 131072, 262144, t - 1], device="cuda")
    h[rows] = torch.randn((5, n), device="cuda").to(torch.bfloat16)
    h_out, u = R.residual_norm(h, h, alpha=0.5)
    want_h, want_u = R.residual_norm(h[rows].contiguous(), h[rows].contiguous(), alpha=0.5)
    assert torch.equal(h_out[rows], want_h) and torch.equal(u[rows], want_u)
    assert u[1].abs().max() == 0 and u[262143].abs().max() == 0


def test_empty_and_refusals():
    call, opts, _ = case(3, 64, mods="token")
    e = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda")
    h_out, u = R.residual_norm(e, e)
    assert h_out.shape == u.shape == (0, 64)
    bad = [{"h": call["h"].cpu()}, {"h": call["h"].half()}, {"y": call["y"][:2]}, {"y": call["y"].float()},
           {"weight": call["weight"][:32]}, {"weight": call["weight"].float()}, {"gate": call["gate"][:2]},
           {"norm": "batch"}, {"mod_index": torch.zeros(3, dtype=torch.int64, device="cuda")},
           {"h_out": torch.empty((3, 64), device="cuda")}, {"out": torch.empty((3, 64), device="cuda")},
           {"gate": call["gate"].t().contiguous().t()}]
    for i, kw in enumerate(bad):
        with pytest.raises(ValueError):
            R.residual_norm(**{**call, **opts, **kw})
            print("accepted", i)
    with pytest.raises(R.SignRotError):
        R.residual_norm(**{**call, **opts, "eps": -1.0})


def test_side_stream_and_graph():
    call, opts, _ = case(40, 1024, mods="index")
    want = R.residual_norm_quant_int8(**call, **opts)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = R.residual_norm_quant_int8(**call, **opts)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = R.residual_norm_quant_int8(**call, **opts)
    for i in range(4):
        call["h"].copy_(torch.randn(call["h"].shape, device="cuda") * (i + 1))
        want = R.residual_norm_quant_int8(**call, **opts)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(held, want)), i


@pytest.mark.parametrize("norm", ["rms", "layer"])
@pytest.mark.parametrize("t,n", [(1024, 8192), (1025, 8192), (769, 8192), (768, 8192), (1280, 5120), (1025, 5120),
                                 (2048, 4096), (2049, 4096), (1537, 4096), (6000, 1024)])
def test_row_counts_around_a_full_device(t, n, norm):
    """Row counts on both sides of what the device holds at once, where the number
    of chunks a thread takes changes."""
    check(t, n, norm=norm, bias=norm == "layer", mods="index")
