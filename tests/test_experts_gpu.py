"""GPU tests of the routed layer's operators (routing, grouping, MXFP4
quantisation and product, combine) against the fp64 oracle.

Tolerances.  u = 2^-24 (fp32), h = half a step of the output type.
  whole numbers, codes, scales and dequantised values: equal.
  routing weights: an expf (2 u) of a difference of two numbers up to `range`
    (range * u), a sum of at most E terms in fp32, each within the former
    ((E / 32 + 5) u for the adding order), a division and a product: relative
    error at most (2 range + E / 32 + 16) u.
  product: the tensor cores add in fp32, 64 products a step: K / 64 steps, each
    dropping at most 2 ulps (2^-22) of the sum of the products' magnitudes so
    far, then one rounding: (K / 64 + 4) 2^-22 * sum |x w| + h |y|.
  combine: top_k + 1 fused steps: (top_k + 2) u * sum |w y| + h |out|.
"""
import numpy as np
import pytest

from adapter_lora_serving_b200 import lora as L
from oracle import experts_oracle as O

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = ["bf16", "f16", "f32"]


def _torch():
    import torch
    return torch


def _dtype(name):
    t = _torch()
    return {"bf16": t.bfloat16, "f16": t.float16, "f32": t.float32}[name]


def _half(name):
    return _torch().finfo(_dtype(name)).eps / 2


def _dev(a, dtype):
    t = _torch()
    return t.from_numpy(np.ascontiguousarray(a)).cuda().to(dtype)


def _i32(a):
    t = _torch()
    return t.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _host(x):
    return x.double().cpu().numpy()


def _rounded(x, name):
    """fp64 values rounded once to the type (torch goes through fp32)."""
    eps, tiny = _torch().finfo(_dtype(name)).eps, _torch().finfo(_dtype(name)).smallest_normal
    step = 2.0 ** np.floor(np.log2(np.maximum(np.abs(x), tiny))) * eps
    return _host(_torch().from_numpy(np.round(x / step) * step).to(_dtype(name)))


def _held(ref, name):
    """fp64 values as the type's range holds them: infinite from half a step past
    its largest number on."""
    fin = _torch().finfo(_dtype(name))
    return np.where(np.abs(ref) >= fin.max * (1 + fin.eps / 4), np.copysign(np.inf, ref), ref)


def _flags():
    t = _torch()
    return t.zeros(1, dtype=t.int32, device="cuda")


def _close(got, ref, tol, what):
    with np.errstate(invalid="ignore"):
        off = ~((np.abs(got - ref) <= tol) | (got == ref))
    assert not off.any(), (f"{what}: {off.sum()} of {off.size} out of tolerance, first at "
                           f"{np.argwhere(off)[0]}: {got[off][0]!r} for {ref[off][0]!r}")


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

def _quantize(x, name, rows, F, index=None, count=None, act=L.LORA_ACT_NONE, keep=False, fill=0x5a):
    t = _torch()
    codes = t.full((rows, F // 2), fill, dtype=t.uint8, device="cuda")
    scales = t.full((rows, F // 32), fill, dtype=t.uint8, device="cuda")
    out = t.full((rows, F), 3.0, dtype=_dtype(name), device="cuda") if keep else None
    flags = _flags()
    L.lora_mx_quantize(x, codes, scales, rows, F, row_index=index, row_count=count, rows_out=out,
                       activation=act, err_flags=flags)
    return codes, scales, out, int(flags.item())


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("rows,F", [(1, 32), (3, 64), (37, 2048), (129, 96), (1, 14336)])
def test_quantize(name, rows, F):
    rng = np.random.default_rng(rows + F)
    x = _dev(rng.standard_normal((rows, F)) * np.exp(rng.uniform(-6, 6, (rows, 1))), _dtype(name))
    codes, scales, _, flags = _quantize(x, name, rows, F)
    c, s = O.mx_quantize(_host(x))
    assert (O.unpack(codes.cpu().numpy()) == c).all() and (scales.cpu().numpy() == s).all()
    assert flags == 0


def test_quantize_every_code_border():
    """Values next to and on every border, signs, zeros, subnormals, the largest
    finite ones, in fp32."""
    mids = (O.E2M1[1:] + O.E2M1[:-1]) / 2
    near = np.concatenate([O.E2M1, mids, np.nextafter(mids.astype(np.float32), 9).astype(np.float64),
                           np.nextafter(mids.astype(np.float32), 0).astype(np.float64), [7.0, 7.99]])
    rows = []
    for e in (0, 5, -30, 120, -120, -126, -128, -140):
        block = np.zeros(32)
        block[0] = 4.0                       # holds the scale
        block[1:31] = np.where(np.arange(30) % 2, 1, -1) * np.resize(near, 30)
        rows.append(np.concatenate([block, np.resize(near[::-1], 32) * -1]) * 2.0 ** e)
    rows.append(np.zeros(64))
    rows.append(np.full(64, -0.0))
    rows.append(np.full(64, float(np.finfo(np.float32).max)))
    rows.append(np.full(64, 1.4e-45))
    x = np.array(rows).astype(np.float32)
    codes, scales, _, flags = _quantize(_dev(x, _dtype("f32")), "f32", len(x), 64)
    c, s = O.mx_quantize(x.astype(np.float64))
    assert (scales.cpu().numpy() == s).all()
    assert (O.unpack(codes.cpu().numpy()) == c).all() and flags == 0


def test_quantize_nonfinite_blocks():
    x = np.ones((2, 96), dtype=np.float32)
    x[0, 40] = np.nan
    x[1, 5] = -np.inf
    codes, scales, _, flags = _quantize(_dev(x, _dtype("f32")), "f32", 2, 96)
    c, s = O.mx_quantize(x.astype(np.float64))
    assert (scales.cpu().numpy() == s).all() and s[0].tolist() == [125, 255, 125]
    assert (O.unpack(codes.cpu().numpy()) == c).all() and flags == L.LORA_FLAG_NONFINITE


@pytest.mark.parametrize("name", TYPES)
def test_quantize_gather_and_count(name):
    """Rows taken by index (repeated ones too), a device row count, an index out
    of range: rows past the count and bad rows stay as they were."""
    rng = np.random.default_rng(5)
    x = _dev(rng.standard_normal((9, 160)), _dtype(name))
    index = rng.integers(0, 9, 50)
    index[7], index[11] = 9, -1
    codes, scales, out, flags = _quantize(x, name, 50, 160, _i32(index), _i32([41])[0:], keep=True)
    rows = np.arange(50)
    live = (rows < 41) & (index >= 0) & (index < 9)
    v = _host(x)[np.where(live, index, 0)]
    c, s = O.mx_quantize(v)
    got = O.unpack(codes.cpu().numpy())
    assert (got[live] == c[live]).all() and (scales.cpu().numpy()[live] == s[live]).all()
    assert (_host(out)[live] == v[live]).all()
    assert (codes.cpu().numpy()[~live] == 0x5a).all() and (scales.cpu().numpy()[~live] == 0x5a).all()
    assert (_host(out)[~live] == 3.0).all() and flags == L.LORA_FLAG_BAD_ROW


@pytest.mark.parametrize("name", TYPES)
def test_quantize_silu_mul(name):
    """SwiGLU rounded once to the type (equal to the fp64 value rounded), then
    quantised; gate values far out, where the exponential over- or underflows."""
    rng = np.random.default_rng(6)
    x = rng.standard_normal((257, 2 * 192)) * 3
    x[0, :24] = np.linspace(-120, 120, 24)
    x[1, :8] = [-87, -88.5, -90, -100, 60000, 88.8, 0.0, -0.0]
    x = _dev(x, _dtype(name))
    codes, scales, out, flags = _quantize(x, name, 257, 192, act=L.LORA_ACT_SILU_MUL, keep=True)
    ref = _rounded(O.silu_mul(_host(x)), name)
    if name == "f32":   # two fp64 formulas, each rounded to fp32
        _close(_host(out), ref, 2 * U * np.abs(ref), "silu_mul")
    else:
        assert (_host(out) == ref).all()
    c, s = O.mx_quantize(_host(out))
    assert (O.unpack(codes.cpu().numpy()) == c).all() and (scales.cpu().numpy() == s).all()
    assert flags == 0


@pytest.mark.parametrize("name", TYPES)
def test_dequantize_every_code_and_scale(name):
    t = _torch()
    codes = np.tile(np.arange(32) % 16, (256, 1))
    scales = np.arange(256)[:, None]
    out = t.empty(256, 32, dtype=_dtype(name), device="cuda")
    L.lora_mx_dequantize(_dev(O.pack(codes), t.uint8), _dev(scales, t.uint8), out, 256, 32)
    with np.errstate(over="ignore"):
        ref = _host(t.from_numpy(O.mx_values(codes, scales)).float().to(_dtype(name)))
    assert np.array_equal(_host(out), ref, equal_nan=True)


# ---------------------------------------------------------------------------
# routing
# ---------------------------------------------------------------------------

def _route(x, bias, k, score="softmax", G=1, g=1, pair=False, renorm=True, scale=1.0):
    t = _torch()
    T, E = x.shape
    ids = t.full((T, k), 77, dtype=t.int32, device="cuda")
    w = t.full((T, k), -5.0, device="cuda")
    flags = _flags()
    L.lora_route_experts(x, bias, ids, w, T, E, k, score=L.LORA_SCORE_SIGMOID if score == "sigmoid"
                         else L.LORA_SCORE_SOFTMAX, num_groups=G, top_groups=g,
                         group_score=L.LORA_GROUP_TOP_PAIR if pair else L.LORA_GROUP_MAX,
                         renormalize=renorm, scale=scale, err_flags=flags)
    return ids, w, int(flags.item())


def _check_route(x, bias, k, repeat=1, **kw):
    """repeat: the rows that many times over (the oracle sees them once)."""
    ids, w, flags = _route(x.repeat(repeat, 1), bias, k, **kw)
    xh = _host(x)
    ref_ids, ref_w, ref_flags = O.route(
        xh, None if bias is None else _host(bias), k, kw.get("score", "softmax"), kw.get("G", 1),
        kw.get("g", 1), kw.get("pair", False), kw.get("renorm", True), kw.get("scale", 1.0))
    ref_ids, ref_w = np.tile(ref_ids, (repeat, 1)), np.tile(ref_w, (repeat, 1))
    assert (ids.cpu().numpy() == ref_ids).all(), np.argwhere(ids.cpu().numpy() != ref_ids)[:4]
    fin = np.where(np.isfinite(xh), np.abs(xh), 0)
    tol = (4 * fin.max() + x.shape[1] / 32 + 16) * U * np.abs(ref_w) + 2.0 ** -126
    _close(_host(w), ref_w, tol, "weights")
    assert flags == ref_flags


@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,k", [(1, 8, 1), (3, 60, 4), (33, 64, 8), (17, 128, 8), (9, 256, 8),
                                   (5, 160, 6), (4, 512, 10), (3, 1000, 32), (2, 33, 32), (2, 5, 5)])
def test_route(name, score, T, E, k):
    rng = np.random.default_rng(E + k)
    x = _dev(rng.standard_normal((T, E)) * 2, _dtype(name))
    bias = _dev(rng.standard_normal(E) * 0.1, _dtype("f32"))
    for renorm, scale in ((True, 1.0), (False, 2.5)):
        _check_route(x, None, k, score=score, renorm=renorm, scale=scale)
        _check_route(x, bias, k, score=score, renorm=renorm, scale=scale)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("pair", [False, True])
@pytest.mark.parametrize("E,G,g,k", [(256, 8, 4, 8), (64, 8, 3, 6), (60, 4, 2, 5), (96, 3, 1, 4),
                                     (32, 32, 5, 5), (160, 8, 3, 6), (16, 2, 2, 4), (512, 32, 7, 8)])
def test_route_groups(score, pair, E, G, g, k):
    rng = np.random.default_rng(E * G + k)
    x = _dev(rng.standard_normal((21, E)) * 2, _dtype("bf16"))
    bias = _dev(rng.standard_normal(E) * 0.2, _dtype("f32"))
    _check_route(x, None, k, score=score, G=G, g=g, pair=pair)
    _check_route(x, bias, k, score=score, G=G, g=g, pair=pair, renorm=False)


@pytest.mark.parametrize("name,score,E,k,kw", [
    ("bf16", "sigmoid", 256, 8, dict(G=8, g=4, pair=True)), ("bf16", "softmax", 128, 6, dict()),
    ("f32", "sigmoid", 160, 15, dict(renorm=False)), ("f16", "softmax", 72, 3, dict(scale=2.5)),
    ("bf16", "softmax", 200, 4, dict(renorm=False)), ("f32", "softmax", 128, 8, dict(G=16, g=5)),
    ("bf16", "sigmoid", 128, 8, dict(G=4, g=2, pair=True, renorm=False)),
    ("bf16", "softmax", 8, 2, dict()), ("f32", "sigmoid", 8, 3, dict(renorm=False)),
    ("f16", "softmax", 16, 12, dict(renorm=False)), ("bf16", "sigmoid", 27, 4, dict(scale=2.5)),
    ("f32", "softmax", 32, 6, dict())])
def test_route_many_tokens(name, score, E, k, kw):
    """Several tokens a warp: masked and padded tokens, ties and close calls among
    the rest."""
    t = _torch()
    rng = np.random.default_rng(E + k)
    x = rng.standard_normal((4203, E)) * 2
    x[7, :] = -np.inf
    x[8, 3:] = -np.inf
    x[100:200] = np.round(x[100:200])               # ties
    x[4202] = 0
    bias = rng.standard_normal(E) * 0.1
    x = _dev(x, _dtype(name))
    for r in range(300, 900, 50):                   # keys of one token within 2^-25 of .5 ...
        row = _host(x)[r]
        s = 1 / (1 + np.exp(-row)) if score == "sigmoid" else np.exp(row - row.max()) / np.exp(row - row.max()).sum()
        close = bias.copy()
        close[::2] = (0.5 - s)[::2]                 # (every other expert's)
    _check_route(x, _dev(bias, t.float32), k, score=score, repeat=4 if E <= 32 else 1, **kw)
    _check_route(x, _dev(close, t.float32), k, score=score, repeat=4 if E <= 32 else 1, **kw)
    _check_route(x, None, k, score=score, repeat=4 if E <= 32 else 1, **kw)
    x[11, 5], x[4000, 0] = float("nan"), float("inf")
    _check_route(x, _dev(bias, t.float32), k, score=score, repeat=4 if E <= 32 else 1, **kw)


def test_route_ties_go_to_the_lowest_index():
    t = _torch()
    for bias in (None, t.zeros(64, device="cuda")):
        for G, g in ((1, 1), (8, 3)):
            for pair in (False, True):
                _check_route(t.zeros(3, 64, device="cuda"), bias, 6, G=G, g=g, pair=pair)
                x = t.tensor([1.0, 2.0, 1.0, 2.0] * 16, device="cuda").repeat(2, 1).bfloat16()
                _check_route(x, bias, 6, score="sigmoid", G=G, g=g, pair=pair)
    x = t.tensor([[0.0, -0.0, 0.0, -0.0]], device="cuda")
    _check_route(x, None, 3)


def test_route_close_scores_as_in_64_bits():
    """Scores whose fp32 values are equal or swapped: logits one step apart where
    the sigmoid is flat, biases that undo the difference to a few 2^-40."""
    t = _torch()
    x = 15.0 + np.arange(64) * 2.0 ** -20          # 1 - sigmoid ~ 3e-7
    x = np.stack([x, x[::-1], np.roll(x, 5)])
    zero = np.zeros(64)
    _check_route(_dev(x, t.float32), _dev(zero, t.float32), 8, score="sigmoid")
    rng = np.random.default_rng(3)
    x = rng.standard_normal((200, 64)).astype(np.float32).astype(np.float64)
    s = np.exp(x - x.max(1, keepdims=True))
    s /= s.sum(1, keepdims=True)
    for r in range(0, 200, 40):
        bias = (0.5 - s[r]).astype(np.float32)     # row r: all keys within 2^-25 of .5
        _check_route(_dev(x, t.float32), _dev(bias, t.float32), 8)
        _check_route(_dev(x, t.float32), _dev(bias, t.float32), 4, G=8, g=2, pair=True)


def test_route_keys_a_few_steps_apart():
    """Equal small scores and biases 18 (and 9) fp32 steps apart, in an order that
    has nothing to do with the experts': every neighbour counts."""
    t = _torch()
    rng = np.random.default_rng(8)
    for E in (256, 128, 64):
        x = np.zeros((16, E))
        for step in (18, 9, 25):
            for score, kw in (("softmax", {}), ("sigmoid", {}), ("softmax", dict(G=8, g=3, pair=True))):
                bias = 1.0 + step * rng.permutation(E) * 2.0 ** -23
                _check_route(_dev(x, t.float32), _dev(bias, t.float32), 8, score=score, **kw)


def test_route_masked_and_nonfinite():
    t = _torch()
    inf, nan = np.inf, np.nan
    x = np.array([[-inf] * 8, [1, -inf, -inf, 2, -inf, -inf, -inf, -inf],
                  [1, nan, 3, inf, 0, -1, -inf, 2], [5, 5, 5, 5, 5, 5, 5, 5.0]])
    for name in ("bf16", "f32"):
        for kw in (dict(), dict(renorm=False), dict(score="sigmoid"),
                   dict(score="sigmoid", renorm=False), dict(G=4, g=2), dict(G=4, g=2, pair=True)):
            for rows in (x[:2], x):
                _check_route(_dev(rows, _dtype(name)), None, 4, **kw)
                b = np.array([0, 0, -inf, 0.25, 0, 0, 0, 0])
                _check_route(_dev(rows, _dtype(name)), _dev(b, t.float32), 4, **kw)
    b = np.array([0, nan, 0, inf, 0, 0, 0, 0])
    _check_route(_dev(x[3:], t.float32), _dev(b, t.float32), 8)


def test_route_far_logits():
    """Scores that underflow (softmax) or saturate (sigmoid) in fp32."""
    t = _torch()
    x = np.array([[-200.0, -150, -300, -180] * 4, [300.0, 0, -80, -90] * 4,
                  [90.0, 95, 100, 120] * 4])
    x = x + np.arange(16) / 8
    for score in ("softmax", "sigmoid"):
        _check_route(_dev(x, t.float32), None, 5, score=score)
    # without renormalisation a score below the smallest fp32 number is 0
    _check_route(_dev(x, t.float32), None, 5, renorm=False)


# ---------------------------------------------------------------------------
# grouping
# ---------------------------------------------------------------------------

def _group(ids, slot, E):
    t = _torch()
    T, k = ids.shape
    n = T * k
    off = t.full((E + 1,), -9, dtype=t.int32, device="cuda")
    tok, pair, rslot = (t.full((n,), -9, dtype=t.int32, device="cuda") for _ in range(3))
    flags = _flags()
    L.lora_group_experts(_i32(ids), None if slot is None else _i32(slot), off, tok, pair,
                         None if slot is None else rslot, T, k, E, err_flags=flags)
    return (off.cpu().numpy(), tok.cpu().numpy(), pair.cpu().numpy().reshape(T, k),
            rslot.cpu().numpy(), int(flags.item()))


@pytest.mark.parametrize("T,k,E", [(1, 1, 1), (1, 8, 128), (37, 8, 128), (700, 3, 60), (2048, 8, 64),
                                   (513, 8, 1024), (5000, 2, 8), (9000, 4, 256), (20011, 4, 1024)])
def test_group(T, k, E):
    rng = np.random.default_rng(T + k + E)
    ids = np.stack([rng.permutation(E)[:k] for _ in range(T)])
    if T > 30:
        ids[T - T // 10:] = -1                       # a padded batch
        ids[3, 0], ids[5, k - 1] = E, -2             # out of range
    slot = rng.integers(-1, 9, T)
    off, tok, pair, rslot, flags = _group(ids, slot, E)
    r_off, r_tok, r_pair, r_slot, r_flags = _sorted(ids, slot, E)
    n = r_off[-1]
    assert (off == r_off).all() and (tok[:n] == r_tok).all() and (pair == r_pair).all()
    assert (rslot[:n] == r_slot).all() and flags == r_flags
    assert (tok[n:] == -9).all() and (rslot[n:] == -9).all()


def _sorted(ids, slot, E):
    """The oracle's grouping by numpy's stable sort (the oracle itself for small
    sizes)."""
    T, k = ids.shape
    if T * k * E < 200000:
        return O.group(ids, slot, E)
    flat = ids.reshape(-1)
    ok = (flat >= 0) & (flat < E)
    order = np.nonzero(ok)[0][np.argsort(flat[ok], kind="stable")]
    off = np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))])
    pair = np.full(T * k, -1)
    pair[order] = np.arange(len(order))
    bad = ((flat < -1) | (flat >= E)).any()
    return off, order // k, pair.reshape(T, k), slot[order // k], O.FLAG_BAD_EXPERT if bad else 0


def test_group_edges():
    """No token, no live choice, the same expert twice, no slots."""
    off, _, _, _, flags = _group(np.zeros((0, 4), dtype=int), np.zeros(0), 12)
    assert (off == 0).all() and flags == 0
    off, tok, pair, rslot, flags = _group(np.full((40, 2), -1), np.zeros(40), 12)
    assert (off == 0).all() and (pair == -1).all() and (tok == -9).all() and (rslot == -9).all()
    off, tok, pair, _, _ = _group(np.array([[3, 3], [3, 0]]), None, 4)
    assert off.tolist() == [0, 1, 1, 1, 4] and tok.tolist() == [1, 0, 0, 1]
    assert pair.tolist() == [[1, 2], [3, 0]]


# ---------------------------------------------------------------------------
# combine
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("name", TYPES)
@pytest.mark.parametrize("T,k,F", [(1, 1, 8), (37, 8, 2048), (5, 9, 24), (200, 4, 168), (3, 32, 64)])
@pytest.mark.parametrize("residual", [False, True])
def test_combine(name, T, k, F, residual):
    rng = np.random.default_rng(T + F)
    cap = T * k + 3
    y = _dev(rng.standard_normal((cap, F)), _dtype(name))
    pair = rng.permutation(cap)[:T * k].reshape(T, k)
    pair[rng.random((T, k)) < 0.2] = -1
    if T > 2:
        pair[1] = -1                                   # a token without rows
        pair[2, 0] = cap
    w = _dev(rng.standard_normal((T, k)), _dtype("f32"))
    res = _dev(rng.standard_normal((T, F)), _dtype(name)) if residual else None
    t = _torch()
    out = t.empty(T, F, dtype=_dtype(name), device="cuda")
    flags = _flags()
    L.lora_combine_experts(y, _i32(pair), w, res, out, T, k, cap, F, err_flags=flags)
    ref, mag, ref_flags = O.combine(_host(y), pair, _host(w), None if res is None else _host(res))
    _close(_host(out), ref, (k + 2) * U * mag + _half(name) * np.abs(ref) + 2.0 ** -133, "combine")
    assert int(flags.item()) == ref_flags
    if residual:                                       # in place
        L.lora_combine_experts(y, _i32(pair), w, res, res, T, k, cap, F)
        assert t.equal(res, out)


# ---------------------------------------------------------------------------
# products
# ---------------------------------------------------------------------------

def _operand(rng, *shape, spread=2.0):
    """Random MXFP4 codes (every code) and scales, packed, on the device; and
    their values."""
    t = _torch()
    codes = rng.integers(0, 16, shape)
    scales = np.round(127 + spread * rng.standard_normal((*shape[:-1], shape[-1] // 32))).astype(int)
    return (_dev(O.pack(codes), t.uint8), _dev(scales.astype(np.uint8), t.uint8),
            O.mx_values(codes, scales))


def _tol(name, K, mag, ref):
    return (K / 64 + 4) * 2.0 ** -22 * mag + _half(name) * np.abs(ref)


def _check_linear(name, rows, K, N, seed=0, **kw):
    t = _torch()
    rng = np.random.default_rng(seed + rows + K + N)
    xc, xs, x = _operand(rng, rows, K, **kw)
    wc, ws, w = _operand(rng, N, K, **kw)
    y = t.full((rows + 1, N), 7.0, dtype=_dtype(name), device="cuda")
    flags = _flags()
    L.lora_mx_linear(xc, xs, wc, ws, y, rows, K, N, err_flags=flags)
    ref, mag = O.mx_linear(x, w)
    got = _host(y)
    assert (got[rows:] == 7.0).all()
    _close(got[:rows], _held(ref, name), _tol(name, K, mag, ref), f"linear {rows} {K} {N}")
    assert int(flags.item()) == 0


def test_linear_one_tile_unit_scales():
    _check_linear("f32", 16, 256, 128, spread=0.0)


def test_linear_one_tile():
    _check_linear("f32", 16, 256, 128)


@pytest.mark.parametrize("rows", [1, 7, 16, 17, 33, 64, 65, 128, 129, 300])
@pytest.mark.parametrize("K,N", [(256, 128), (32, 8), (96, 136), (1056, 264), (2048, 512), (640, 392),
                                 (768, 2048), (4608, 1000)])
def test_linear(rows, K, N):
    _check_linear("bf16", rows, K, N)


@pytest.mark.parametrize("name", ["f16", "f32"])
@pytest.mark.parametrize("rows,K,N", [(1, 4096, 128), (40, 544, 200), (200, 1024, 384)])
def test_linear_types(name, rows, K, N):
    _check_linear(name, rows, K, N, spread=0.5)


def test_linear_many_tiles():
    """Every CTA runs several tiles (rings and accumulators go round)."""
    _check_linear("bf16", 520, 1280, 8192)
    _check_linear("bf16", 5, 512, 60000)


@pytest.mark.parametrize("name,rows,K,N", [("f32", 2304, 512, 2304), ("bf16", 2300, 1024, 2440),
                                           ("bf16", 4096, 512, 8192), ("f16", 300, 1536, 9736)])
def test_linear_many_rows(name, rows, K, N):
    """The tiles that two CTAs share; partial ones at both ends."""
    _check_linear(name, rows, K, N, spread=0.5)


def test_expert_linear_many_rows():
    for name in ("bf16", "f32"):
        _check_expert(name, [400, 0, 300, 1, 900], 512, 4000, tail=3)


def test_linear_rerun_bit_exact():
    t = _torch()
    rng = np.random.default_rng(9)
    xc, xs, _ = _operand(rng, 70, 2048)
    wc, ws, _ = _operand(rng, 640, 2048)
    ys = [t.empty(70, 640, dtype=t.float32, device="cuda") for _ in range(3)]
    for y in ys:
        L.lora_mx_linear(xc, xs, wc, ws, y, 70, 2048, 640)
    assert t.equal(ys[0], ys[1]) and t.equal(ys[0], ys[2])


def _check_expert(name, counts, K, N, seed=0, offsets=None, tail=0, start=0):
    t = _torch()
    rng = np.random.default_rng(seed + K + N + len(counts))
    E = len(counts)
    if offsets is None:
        offsets = start + np.concatenate([[0], np.cumsum(counts)])
    rows = start + int(np.sum(counts)) + tail
    xc, xs, x = _operand(rng, rows, K)
    wc, ws, w = _operand(rng, E, N, K)
    y = t.full((rows, N), 7.0, dtype=_dtype(name), device="cuda")
    flags = _flags()
    L.lora_mx_expert_linear(xc, xs, wc, ws, _i32(offsets), y, rows, K, N, E, err_flags=flags)
    ref, mag, touched, ref_flags = O.mx_expert_linear(x, w, offsets)
    got = _host(y)
    assert (got[~touched] == 7.0).all()
    # rows that two experts claim have no specified result
    owners = np.zeros(rows, dtype=int)
    for lo, hi in zip(offsets[:-1], offsets[1:]):
        if 0 <= lo <= hi <= rows:
            owners[lo:hi] += 1
    touched &= owners == 1
    _close(got[touched], _held(ref, name)[touched], _tol(name, K, mag, ref)[touched],
           f"experts {counts}")
    assert int(flags.item()) == ref_flags


@pytest.mark.parametrize("counts", [[1], [0, 0, 5, 0], [3, 1, 0, 17, 2, 2], [40, 0, 64, 1],
                                    [130, 257, 0, 12, 128], [1] * 40, [0, 0, 0]])
@pytest.mark.parametrize("K,N", [(256, 128), (96, 72), (800, 328), (768, 512), (2048, 136), (384, 3000)])
def test_expert_linear(counts, K, N):
    _check_expert("bf16", counts, K, N)


def test_expert_linear_padding_and_types():
    """Rows before the first and behind the last expert's stay as they were."""
    for name in TYPES:
        _check_expert(name, [5, 0, 33, 2], 160, 136, tail=9, start=4)
    _check_expert("bf16", list(range(0, 130)), 64, 64)


def test_expert_linear_bad_offsets_skip_the_expert():
    _check_expert("bf16", [10, 20, 30], 128, 64, offsets=np.array([-3, 10, 30, 70]))
    _check_expert("bf16", [10, 20, 30], 128, 64, offsets=np.array([0, 30, 10, 60]))


def test_expert_linear_offsets_that_go_back_and_forth():
    """Offsets 0, rows, 0, rows, ...: every other expert claims all rows.  Flagged;
    the rows' values are unspecified, but only rows of y are written."""
    t = _torch()
    rng = np.random.default_rng(4)
    E, rows, K, N = 64, 100, 512, 256
    xc, xs, _ = _operand(rng, rows, K)
    wc, ws, _ = _operand(rng, E, N, K)
    y = t.full((rows + 40, N), 7.0, device="cuda")
    flags = _flags()
    L.lora_mx_expert_linear(xc, xs, wc, ws, _i32(np.arange(E + 1) % 2 * rows), y, rows, K, N, E,
                            err_flags=flags)
    assert (y[rows:] == 7.0).all() and int(flags.item()) == L.LORA_FLAG_BAD_OFFSETS


@pytest.mark.parametrize("rows,K,N", [(40, 512, 136), (5, 2048, 128), (700, 1056, 4096), (2304, 512, 2304)])
def test_linear_nan_scale_stays_in_its_row(rows, K, N):
    """A block without a scale (byte 255) makes its row (of x) or feature (of w) NaN
    and nothing else."""
    t = _torch()
    rng = np.random.default_rng(rows)
    xc, xs, x = _operand(rng, rows, K, spread=0.5)
    wc, ws, w = _operand(rng, N, K, spread=0.5)
    xs[3, K // 32 - 1] = 255
    ws[N - 2, 1] = 255
    y = t.empty(rows, N, device="cuda")
    L.lora_mx_linear(xc, xs, wc, ws, y, rows, K, N)
    got = _host(y)
    assert np.isnan(got[3]).all() and np.isnan(got[:, N - 2]).all()
    keep = np.ones((rows, N), dtype=bool)
    keep[3], keep[:, N - 2] = False, False
    ref, mag = O.mx_linear(x, w)
    _close(got[keep], ref[keep], _tol("f32", K, mag, ref)[keep], "beside NaN")


def test_products_of_two_streams_at_once():
    """Pair tiles, split tiles and experts' tiles in flight together on two streams
    give the bits of each alone."""
    t = _torch()
    rng = np.random.default_rng(12)
    calls = []
    for rows, K, N, E in ((2304, 512, 2304, 0), (3, 4096, 256, 0), (160, 1056, 264, 0), (500, 768, 520, 9)):
        xc, xs, _ = _operand(rng, rows, K)
        wc, ws, _ = _operand(rng, max(E, 1) * N, K)
        off = _i32(np.linspace(0, rows, E + 1).astype(int)) if E else None

        def call(y, rows=rows, K=K, N=N, E=E, a=(xc, xs, wc, ws), off=off, flags=None):
            if E:
                L.lora_mx_expert_linear(*a, off, y, rows, K, N, E, err_flags=flags)
            else:
                L.lora_mx_linear(*a, y, rows, K, N, err_flags=flags)
        want = t.empty(rows, N, dtype=t.bfloat16, device="cuda")
        call(want)
        calls.append((call, want))
    flags = _flags()
    streams = [t.cuda.Stream(), t.cuda.Stream()]
    outs = [[t.empty_like(w) for _ in range(10)] for _, w in calls]
    t.cuda.synchronize()
    for j in range(10):
        for i, (call, _) in enumerate(calls):
            with t.cuda.stream(streams[(i + j) % 2]):
                call(outs[i][j], flags=flags)
    t.cuda.synchronize()
    for out, (_, w) in zip(outs, calls):
        assert all(t.equal(o, w) for o in out)
    assert int(flags.item()) == 0


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("E,G", [(64, 8), (256, 8), (96, 3), (512, 32)])
def test_route_pair_sums_past_fp32(score, E, G):
    """Biases whose pairwise sums leave fp32's range, up or down: the groups are still
    ranked by those sums, and a group whose sum is below the range can be chosen."""
    t = _torch()
    rng = np.random.default_rng(E + G)
    x = _dev(rng.standard_normal((9, E)), t.float32)
    far = 2.0e38 + 1e35 * rng.permutation(E)
    mixed = np.where(np.arange(E) % 3 == 0, 1.0, -1.0) * far
    for bias in (far, -far, mixed, np.where(np.arange(E) < E // G, far, 0.01 * np.arange(E))):
        for g in (1, 2):
            _check_route(x, _dev(bias, t.float32), 4, score=score, G=G, g=g, pair=True)


def _ids(x, bias, k, repeat=1, **kw):
    t = _torch()
    b = None if bias is None else _dev(np.asarray(bias, dtype=np.float64), t.float32)
    ids, _, flags = _route(_dev(np.asarray(x, dtype=np.float64), t.float32).repeat(repeat, 1), b, k, **kw)
    assert flags == 0
    return ids.cpu().numpy()


@pytest.mark.parametrize("repeat", [1, 8192])      # a warp a token, a thread a token
def test_route_saturated_scores_by_hand(repeat):
    """Scores that are equal in 64 bits: sigmoids of 38, 50 and 60 are 1, softmax
    scores of -800 and -760 beside 0 are 0.  With one bias for all the larger logit
    has the larger key all the same; with several, equal keys go by the index."""
    x = [[38.0, 50.0, -1.0, 50.0, 60.0, 0.0, 37.9, 45.0]] * 2
    want = [[4, 1, 3, 7, 0]] * (2 * repeat)
    for bias in (None, [0.0] * 8, [0.25] * 8, [1e9] * 8, [-3.0] * 8):
        assert _ids(x, bias, 5, repeat, score="sigmoid").tolist() == want
    x = [[-800.0, 0.0, -760.0, -900.0, -760.0, -1.0, -790.0, -2000.0]] * 2
    want = [[1, 5, 2, 4, 6, 0, 3, 7]] * (2 * repeat)
    for bias in (None, [0.0] * 8, [0.5] * 8):
        assert _ids(x, bias, 8, repeat).tolist() == want
    # keys 1, 1.5, 1.5 - 8e-7 and 1
    x = [[39.0, 38.0, 14.0, 60.0]] * 2
    assert _ids(x, [0.0, 0.5, 0.5, 0.0], 4, repeat, score="sigmoid").tolist() == [[1, 2, 0, 3]] * (2 * repeat)


@pytest.mark.parametrize("E", [8, 27, 64, 128, 256, 384, 512, 1000])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_one_bias_leaves_the_order_of_the_logits(E, score):
    """Logits over a range where most scores are equal in 64 bits: with one bias for
    all experts, small or large, the choice is that without any."""
    rng = np.random.default_rng(E)
    t = _torch()
    x = np.round(rng.uniform(-900, 900, (40, E))) * (1.0 if score == "softmax" else 0.25)
    x = np.concatenate([x, np.abs(x) + 40.0])
    for kw in [dict()] + ([dict(G=8, g=3)] if E % 8 == 0 and E > 8 else []):
        k = min(8, E)
        want = _ids(x, None, k, score=score, **kw)
        for bias in (0.0, 0.375, -7.0, 1e12):
            assert (_ids(x, np.full(E, bias), k, score=score, **kw) == want).all()
        _check_route(_dev(x, t.float32), _dev(np.full(E, 0.375), t.float32), k, score=score, **kw)


@pytest.mark.parametrize("E", [8, 32, 64, 128, 256, 384, 512, 1024])
def test_route_close_keys_where_the_sum_is_least_exact(E):
    """One expert at 0 and the others where the mean error of the softmax's terms is
    largest (z e^z weighted by their number), and biases that leave the keys an odd
    fraction of an fp32 step to a few steps apart, in an order of their own; with a
    few of them far below."""
    t = _torch()
    rng = np.random.default_rng(E)
    w = np.linspace(1.0, 8.0, 2000)
    r = (E - 1) * np.exp(-w)
    w = w[np.argmax(w * r / (1 + r))]
    x = np.full((6, E), -w) + rng.uniform(-0.2, 0.2, (6, E))
    x[:, 0] = 0.0
    x[3:, E // 2 :] -= 20.0
    x = x.astype(np.float32).astype(np.float64)
    s = np.exp(x - x.max(1, keepdims=True))
    s /= s.sum(1, keepdims=True)
    k = min(8, E)
    for row in (0, 1, 3, 5):
        for step in (0.3, 2.7, 40.0):
            bias = 0.25 + step * 2.0 ** -25 * rng.permutation(E) - s[row]
            for repeat in ([1, 2731] if E <= 32 else [1]):
                _check_route(_dev(x, t.float32), _dev(bias, t.float32), k, repeat=repeat)
            if E >= 64:
                _check_route(_dev(x, t.float32), _dev(bias, t.float32), k, G=8, g=3, pair=True)
                _check_route(_dev(x, t.float32), _dev(bias, t.float32), k, G=8, g=3)


@pytest.mark.parametrize("name,score,E,k,kw", [
    ("bf16", "sigmoid", 256, 8, dict(G=8, g=4, pair=True)), ("bf16", "softmax", 128, 6, dict()),
    ("bf16", "softmax", 8, 2, dict()), ("f32", "sigmoid", 8, 3, dict(renorm=False)),
    ("f16", "softmax", 16, 12, dict(renorm=False)), ("bf16", "sigmoid", 27, 4, dict(scale=2.5)),
    ("f32", "softmax", 32, 6, dict())])
def test_route_many_tokens_close_and_masked_biases(name, score, E, k, kw):
    """Many tokens, and for each of several a bias that brings the keys of every other
    expert within 2^-25 of one half for it; then biases that mask experts (-inf) and
    that are NaN or infinite."""
    t = _torch()
    rng = np.random.default_rng(E * k)
    T = 4203 if E <= 32 else 900
    x = rng.standard_normal((T, E)) * 2
    x[7, :] = -np.inf
    x[8, 3:] = -np.inf
    x[100:200] = np.round(x[100:200])
    x = _dev(x, _dtype(name))
    bias = rng.standard_normal(E) * 0.1
    repeat = 4 if E <= 32 else 1
    for r in range(300, 900, 100):
        row = _host(x)[r]
        e = np.exp(row - row.max())
        s = 1 / (1 + np.exp(-row)) if score == "sigmoid" else e / e.sum()
        close = np.where(np.arange(E) % 2 == 0, 0.5 - s, bias)
        _check_route(x, _dev(close, t.float32), k, score=score, repeat=repeat, **kw)
    masked = bias.copy()
    masked[1:E:3] = -np.inf
    _check_route(x, _dev(masked, t.float32), k, score=score, repeat=repeat, **kw)
    masked[0], masked[E - 2] = np.nan, np.inf
    _check_route(x, _dev(masked, t.float32), k, score=score, repeat=repeat, **kw)
    _check_route(x, _dev(np.full(E, -np.inf), t.float32), k, score=score, repeat=repeat, **kw)


@pytest.mark.parametrize("name,score,E,k,rows,kw", [
    ("bf16", "sigmoid", 32, 1, 8, dict()), ("f32", "softmax", 27, 2, 12, dict(renorm=False)),
    ("f16", "sigmoid", 17, 4, 20, dict(scale=2.5)), ("f32", "softmax", 32, 8, 36, dict()),
    ("bf16", "softmax", 16, 12, 13, dict(renorm=False)), ("bf16", "sigmoid", 9, 4, 5, dict()),
    ("bf16", "softmax", 32, 9, 40, dict()), ("f32", "sigmoid", 8, 8, 4, dict())])
def test_route_on_both_sides_of_a_thread_a_token(name, score, E, k, rows, kw):
    """The number of tokens from which a thread takes a token grows with the row and
    the choices: the same tokens few and `rows` times over, with close and masked
    biases."""
    t = _torch()
    rng = np.random.default_rng(E * k + rows)
    x = rng.standard_normal((4203, E)) * 2
    x[7, :], x[8, 1:], x[9, 0] = -np.inf, -np.inf, np.nan
    x[100:200] = np.round(x[100:200])
    x = _dev(x, _dtype(name))
    row = _host(x)[500]
    e = np.exp(row - row.max())
    s = 1 / (1 + np.exp(-row)) if score == "sigmoid" else e / e.sum()
    close = 0.5 - s
    masked = np.where(np.arange(E) % 5 == 2, -np.inf, 0.1 * rng.standard_normal(E))
    for bias in (None, close, masked):
        for repeat in (1, rows):
            _check_route(x, None if bias is None else _dev(bias, t.float32), k, score=score,
                         repeat=repeat, **kw)


@pytest.mark.parametrize("E", [64, 96, 512])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_route_with_every_group_kept(E, score):
    """The choice is that without groups, also among scores equal in 64 bits."""
    rng = np.random.default_rng(E)
    x = np.round(rng.uniform(-900, 900, (20, E))) * (1.0 if score == "softmax" else 0.25)
    for bias in (None, np.full(E, 0.5), 0.1 * rng.standard_normal(E)):
        want = _ids(x, bias, 8, score=score)
        for pair in (False, True):
            assert (_ids(x, bias, 8, score=score, G=8, g=8, pair=pair) == want).all()
    _check_route(_dev(x, _dtype("f32")), None, 8, score=score, G=8, g=8, pair=True)
