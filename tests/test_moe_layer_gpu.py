"""The routed layer as a whole (adapter_lora_serving_b200.moe): every step's output
against the fp64 oracle of that step on the buffers that the step read, and the
call eager, captured, on another stream and with fewer tokens than the buffers hold.
Tolerances: those of the operators' own tests, and the expert folds' of theirs."""
import numpy as np
import pytest

from adapter_lora_serving_b200 import lora as L
from adapter_lora_serving_b200 import workloads as W
from oracle import experts_oracle as O
from oracle import lora_oracle as LO

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def _torch():
    import torch
    return torch


def _host(t):
    return t.double().cpu().numpy()


def _close(got, ref, tol, what):
    off = ~(np.abs(got - ref) <= tol)
    assert not off.any(), f"{what}: {off.sum()} of {off.size}, first {got[off][0]!r} for {ref[off][0]!r}"


class Case:
    def __init__(self, T, hidden=256, inter=96, E=16, k=3, slots=3, R=16, seed=0, adapters=True,
                 router=True, max_tokens=None, residual=True, **routing):
        from adapter_lora_serving_b200 import moe
        t = _torch()
        g = t.Generator(device="cuda").manual_seed(seed)

        def randn(*s, std=1.0):
            return t.randn(*s, generator=g, device="cuda") * std

        def weight(n, kk):
            codes = t.empty(E, n, kk // 2, dtype=t.uint8, device="cuda")
            scales = t.empty(E, n, kk // 32, dtype=t.uint8, device="cuda")
            w = randn(E * n, kk, std=kk ** -0.5).bfloat16()
            L.lora_mx_quantize(w, codes, scales, E * n, kk)
            return codes, scales

        self.T, self.hidden, self.inter, self.E, self.k = T, hidden, inter, E, k
        self.slots, self.R = slots, R
        self.ranks = t.tensor([R, R // 2, 0, R][:slots] * (1 + slots // 4), dtype=t.int32,
                              device="cuda")[:slots].contiguous()
        self.scalings = t.linspace(0.5, 2.0, slots, device="cuda")
        self.gu_ad = self.dn_ad = self.rt_ad = None
        if adapters:
            pairs = slots * E // 2
            index = t.full((slots * E,), -1, dtype=t.int32, device="cuda")
            at = t.randperm(slots * E, generator=g, device="cuda")[:pairs]
            index[at] = t.arange(pairs, dtype=t.int32, device="cuda")

            def pool(n_in, n_out, s):
                return moe.ExpertAdapters(randn(pairs, s * R, n_in, std=n_in ** -0.5).bfloat16(),
                                          randn(pairs, n_out, R, std=0.2).bfloat16(), index,
                                          self.ranks, self.scalings)
            self.gu_ad, self.dn_ad = pool(hidden, 2 * inter, 2), pool(inter, hidden, 1)
        if router:
            self.rt_ad = moe.RouterAdapters(randn(slots, R, hidden, std=hidden ** -0.5).bfloat16(),
                                            randn(slots, E, R, std=0.2).bfloat16(), self.ranks,
                                            self.scalings)
        self.layer = moe.MoeLayer(max_tokens or T, hidden, inter, E, k, weight(2 * inter, hidden),
                                  weight(hidden, inter), self.gu_ad, self.dn_ad, self.rt_ad,
                                  **routing)
        self.routing = routing
        self.x = randn(T, hidden).bfloat16()
        self.logits = randn(T, E, std=1.5).bfloat16()
        self.residual = randn(T, hidden).bfloat16() if residual else None
        slot = np.random.default_rng(seed).integers(-1, slots, T)
        order, indptr = W.csr_by_slot(slot, slots)
        self.slot_np, self.order_np, self.indptr_np = slot, order, indptr
        self.slot, self.order, self.indptr = (
            t.from_numpy(np.ascontiguousarray(v, dtype=np.int32)).cuda() for v in (slot, order, indptr))
        self.flags = t.zeros(1, dtype=t.int32, device="cuda")

    def run(self, logits, out, stream=None):
        return self.layer.forward(self.x, logits, out, self.slot, self.order, self.indptr,
                                  self.residual, self.flags, stream)

    def fresh(self):
        t = _torch()
        return self.logits.clone(), t.full((self.T, self.hidden), 7.0, dtype=t.bfloat16, device="cuda")


def _values(codes, scales):
    return O.mx_values(O.unpack(codes.cpu().numpy()), scales.cpu().numpy())


def _check_steps(c):
    ly = c.layer
    logits, out = c.fresh()
    c.run(logits, out)
    T, k, E, rows = c.T, c.k, c.E, c.T * c.k
    lg = _host(logits)
    if c.rt_ad is not None:
        ref, _, _ = LO.apply_router(_host(c.x), _host(c.logits), _host(c.rt_ad.a), _host(c.rt_ad.b),
                                    c.order_np, c.indptr_np, _host(c.ranks).astype(int),
                                    _host(c.scalings), c.R)
        assert LO.within_tolerance(lg, ref).all()
    pair = c.routing.get("group_score", 0) == L.LORA_GROUP_TOP_PAIR
    ids, w, _ = O.route(lg, None if ly.bias is None else _host(ly.bias), k,
                        "sigmoid" if c.routing.get("score") == L.LORA_SCORE_SIGMOID else "softmax",
                        c.routing.get("num_groups", 1), c.routing.get("top_groups", 1), pair,
                        c.routing.get("renormalize", True), c.routing.get("scale", 1.0))
    got_ids = ly.topk_ids.cpu().numpy()[:rows].reshape(T, k)
    got_w = _host(ly.topk_weights)[:rows].reshape(T, k)
    assert (got_ids == ids).all()
    fin = np.abs(lg[np.isfinite(lg)]).max(initial=0)
    _close(got_w, w, (4 * fin + E / 32 + 16) * U * np.abs(w), "weights")
    off, tok, pair_row, row_slot, _ = O.group(ids, c.slot_np, E)
    n = int(off[-1])
    assert (ly.expert_offsets.cpu().numpy() == off).all()
    assert (ly.row_token.cpu().numpy()[:n] == tok).all()
    assert (ly.pair_row.cpu().numpy()[:rows].reshape(T, k) == pair_row).all()
    assert (ly.row_slot.cpu().numpy()[:n] == row_slot).all()
    xs = _host(ly.x_sorted)[:n]
    assert (xs == _host(c.x)[tok]).all()
    xq = _values(ly.x_codes[:n], ly.x_scales[:n])
    assert (xq == O.mx_values(*O.mx_quantize(xs))).all()

    def product_and_fold(x, xq, weight, y, ad, slices, what):
        ref, mag, _, _ = O.mx_expert_linear(xq, _values(*weight), off)
        K = xq.shape[1]
        tol = (K / 64 + 4) * 2.0 ** -22 * mag + 2.0 ** -8 * np.abs(ref)
        if ad is not None:
            # the fold adds to the product rounded to bf16 (which may be the
            # neighbour of the oracle's): its own tolerance on top
            ref, _, _ = LO.expert_apply(x, ref, _host(ad.a), _host(ad.b),
                                        ad.pair_index.cpu().numpy(), _host(c.ranks).astype(int),
                                        _host(c.scalings), row_slot, off, c.R, slices, c.slots, E,
                                        ad.num_pairs)
            tol = tol + 1e-2 + 1.6e-2 * np.abs(ref)
        _close(_host(y)[:n], ref, tol, what)

    product_and_fold(xs, xq, ly.gate_up, ly.gate_up_out, c.gu_ad, (c.inter, c.inter), "gate/up")
    gu = _host(ly.gate_up_out)[:n]
    act = _host(ly.act)[:n]
    ref = O.silu_mul(gu)
    _close(act, ref, 2.0 ** -8 * np.abs(ref), "silu_mul")
    aq = _values(ly.act_codes[:n], ly.act_scales[:n])
    assert (aq == O.mx_values(*O.mx_quantize(act))).all()
    product_and_fold(act, aq, ly.down, ly.down_out, c.dn_ad, (c.hidden,), "down")
    ref, mag, _ = O.combine(_host(ly.down_out)[:rows], pair_row, got_w,
                            None if c.residual is None else _host(c.residual))
    _close(_host(out), ref, (k + 2) * U * mag + 2.0 ** -8 * np.abs(ref), "out")
    assert int(c.flags.item()) == 0
    return out


@pytest.mark.parametrize("kw", [
    dict(T=1), dict(T=37), dict(T=200, k=2, E=8), dict(T=33, adapters=False, router=False, residual=False),
    dict(T=64, hidden=512, inter=160, E=32, k=6, score=L.LORA_SCORE_SIGMOID, num_groups=4,
         top_groups=2, group_score=L.LORA_GROUP_TOP_PAIR, scale=2.5),
    dict(T=5, max_tokens=300), dict(T=600, hidden=64, inter=64, E=40, k=8)])
def test_layer_steps(kw):
    _check_steps(Case(**kw))


def test_layer_masked_tokens():
    """Padded tokens (all logits -inf) go to no expert: their output is the
    residual."""
    t = _torch()
    c = Case(T=50, router=False)
    c.logits[40:] = float("-inf")
    c.logits[:, 3] = float("-inf")          # an expert that is off
    out = _check_steps(c)
    assert t.equal(out[40:], c.residual[40:])
    assert (c.layer.topk_ids[:50 * c.k].view(50, c.k)[40:] == -1).all()


def test_layer_captured_and_on_another_stream():
    """The captured layer replayed (also on new inputs), and the layer on a side
    stream, give the bits of the eager call."""
    t = _torch()
    c = Case(T=48)
    logits, eager = c.fresh()
    c.run(logits, eager)
    side = t.cuda.Stream()
    logits, other = c.fresh()
    side.wait_stream(t.cuda.current_stream())
    c.run(logits, other, stream=side)
    t.cuda.current_stream().wait_stream(side)
    assert t.equal(other, eager)
    static, captured = c.fresh()
    t.cuda.synchronize()
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        c.run(static, captured)
    for _ in range(2):
        static.copy_(c.logits)
        captured.zero_()
        graph.replay()
        assert t.equal(captured, eager)
    c.x.copy_(c.x.flip(0))
    static.copy_(c.logits)
    graph.replay()
    logits, again = c.fresh()
    c.run(logits, again)
    assert t.equal(captured, again) and not t.equal(captured, eager)


def test_layers_of_two_streams():
    """Two layers (each with its own buffers) at once on two streams."""
    t = _torch()
    cases = [Case(T=90, seed=1), Case(T=70, seed=2)]
    want = []
    for c in cases:
        logits, out = c.fresh()
        c.run(logits, out)
        want.append(out)
    streams = [t.cuda.Stream() for _ in cases]
    inputs = [[c.fresh() for _ in range(5)] for c in cases]
    t.cuda.synchronize()
    for j in range(5):
        for c, s, inp in zip(cases, streams, inputs):
            c.run(*inp[j], stream=s)
    t.cuda.synchronize()
    for w, inp in zip(want, inputs):
        for _, out in inp:
            assert t.equal(out, w)


def test_layer_refusals():
    t = _torch()
    c = Case(T=8)
    logits, out = c.fresh()
    with pytest.raises(ValueError, match="room"):
        c.layer.forward(c.x.repeat(2, 1), logits.repeat(2, 1), out.repeat(2, 1), c.slot, c.order, c.indptr)
    with pytest.raises(ValueError, match="token_slot"):
        c.layer.forward(c.x, logits, out)
    with pytest.raises(L.LoraError, match="contiguous"):
        Case(T=8, router=False, adapters=False).layer.forward(
            c.x, t.zeros(16, 8, dtype=t.bfloat16, device="cuda").t(), out)
    with pytest.raises(L.LoraError, match="element"):
        L.lora_mx_dequantize(c.layer.x_codes, c.layer.x_scales, out, c.T + 1, c.hidden)


def test_layer_with_router_refuses_before_the_fold():
    """With router adapters nothing is written when an input is not as the fold, which
    takes addresses, reads it."""
    t = _torch()
    c = Case(T=8)
    logits, out = c.fresh()
    kept = logits.clone()
    wide = t.zeros(8, 2 * c.hidden, dtype=t.bfloat16, device="cuda")

    def call(match, x=c.x, lg=logits, o=out, order=c.order, residual=c.residual):
        with pytest.raises(L.LoraError, match=match):
            c.layer.forward(x, lg, o, c.slot, order, c.indptr, residual, c.flags)
        assert t.equal(logits, kept) and (out == 7.0).all()

    call("element type", lg=logits.float())
    call("element type", x=c.x.half())
    call("contiguous", lg=t.zeros(c.E, 8, dtype=t.bfloat16, device="cuda").t())
    call("contiguous", x=wide[:, :c.hidden])
    call("contiguous", x=c.x[:1].expand(8, c.hidden))
    call("features", x=wide)
    call("features", x=c.x[:, :32].contiguous())
    call("rows of", lg=t.zeros(8, 2 * c.E, dtype=t.bfloat16, device="cuda"))
    call("contiguous", o=wide[:, :c.hidden])
    call("fewer", residual=c.residual[:4])
    call("element type", order=c.order.long())
    call("not on a CUDA device", order=c.order.cpu())
    c.run(logits, out)
    assert not (out == 7.0).all() and int(c.flags.item()) == 0


@pytest.mark.parametrize("name", ["float32", "float16"])
def test_layer_takes_other_logits_without_a_router_fold(name):
    c = Case(T=20, router=False)
    c.logits = c.logits.to(getattr(_torch(), name))
    _check_steps(c)
