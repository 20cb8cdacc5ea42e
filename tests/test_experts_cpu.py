"""The routed layer's entry points on a host without a GPU: refusals before any
launch (C ABI and binding), and hand-derived pins of their fp64 oracle."""
import os
import re

import numpy as np
import pytest

from adapter_lora_serving_b200 import lora as L
from oracle import experts_oracle as O

FAKE = 1 << 20          # a 16-byte aligned, never dereferenced address


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(L.LIB_PATH):
        from adapter_lora_serving_b200 import build
        build.build()
    return L.load()


def _route(lib, **kw):
    a = dict(logits=FAKE, type=0, bias=None, ids=FAKE, weights=FAKE, T=4, E=64, k=8, score=0, G=1,
             g=1, gs=0, renorm=1, scale=1.0, flags=None)
    a.update(kw)
    return lib.lora_route_experts(*a.values(), None)


def _group(lib, **kw):
    a = dict(ids=FAKE, slot=FAKE, off=FAKE, tok=FAKE, pair=FAKE, rslot=FAKE, T=4, k=2, E=8,
             flags=None)
    a.update(kw)
    return lib.lora_group_experts(*a.values(), None)


def _quant(lib, **kw):
    a = dict(x=FAKE, type=0, index=None, count=None, out=None, codes=FAKE, scales=FAKE, x_rows=4,
             rows=4, F=64, act=0, flags=None)
    a.update(kw)
    return lib.lora_mx_quantize(*a.values(), None)


def _dequant(lib, **kw):
    a = dict(codes=FAKE, scales=FAKE, out=FAKE, type=0, rows=4, F=64)
    a.update(kw)
    return lib.lora_mx_dequantize(*a.values(), None)


def _linear(lib, **kw):
    a = dict(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, y=FAKE, type=0, rows=4, K=64, N=64, flags=None)
    a.update(kw)
    return lib.lora_mx_linear(*a.values(), None)


def _expert(lib, **kw):
    a = dict(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, off=FAKE, y=FAKE, type=0, rows=4, K=64, N=64, E=8,
             flags=None)
    a.update(kw)
    return lib.lora_mx_expert_linear(*a.values(), None)


def _combine(lib, **kw):
    a = dict(y=FAKE, type=0, pair=FAKE, w=FAKE, res=None, out=FAKE, T=4, k=2, cap=8, F=64,
             flags=None)
    a.update(kw)
    return lib.lora_combine_experts(*a.values(), None)


INVALID = [
    (_route, kw) for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(type=3), dict(type=-1),
                            dict(score=2), dict(gs=2), dict(G=0), dict(G=7), dict(G=8, g=9),
                            dict(G=8, g=0), dict(G=16, g=1, k=5), dict(k=65), dict(logits=None),
                            dict(logits=FAKE + 8), dict(ids=FAKE + 2), dict(weights=None),
                            dict(bias=FAKE + 1), dict(flags=FAKE + 2))
] + [
    (_group, kw) for kw in (dict(T=-1), dict(E=0), dict(k=0), dict(ids=None), dict(off=None),
                            dict(slot=None), dict(rslot=None), dict(tok=FAKE + 1),
                            dict(pair=None), dict(T=0, off=None))
] + [
    (_quant, kw) for kw in (dict(F=0), dict(F=48), dict(rows=-1), dict(x_rows=-1), dict(type=4),
                            dict(act=2), dict(x_rows=3), dict(x=None), dict(x=FAKE + 4),
                            dict(codes=FAKE + 8), dict(scales=None), dict(out=FAKE + 8),
                            dict(index=FAKE + 2), dict(count=FAKE + 2))
] + [
    (_dequant, kw) for kw in (dict(F=16), dict(rows=-2), dict(type=9), dict(out=None),
                              dict(codes=FAKE + 1))
] + [
    (_linear, kw) for kw in (dict(K=48), dict(K=0), dict(N=12), dict(N=0), dict(rows=-1),
                             dict(type=3), dict(xc=None), dict(xs=FAKE + 4), dict(wc=FAKE + 8),
                             dict(ws=None), dict(y=FAKE + 2), dict(flags=FAKE + 1))
] + [
    (_expert, kw) for kw in (dict(K=33), dict(N=4), dict(E=0), dict(rows=-1), dict(off=None),
                             dict(off=FAKE + 2), dict(y=None))
] + [
    (_combine, kw) for kw in (dict(T=-1), dict(k=0), dict(cap=-1), dict(F=12), dict(type=7),
                              dict(y=None), dict(pair=FAKE + 2), dict(w=None), dict(res=FAKE + 8),
                              dict(out=None))
]


@pytest.mark.parametrize("call,kw", INVALID)
def test_refused_before_launch(lib, call, kw):
    assert call(lib, **kw) == L.LORA_ERR_INVALID
    assert lib.lora_last_error().decode().startswith("lora_")


@pytest.mark.parametrize("call,kw", [
    (_route, dict(E=1032)), (_route, dict(E=64, k=33)), (_route, dict(E=128, G=64, g=64)),
    (_group, dict(E=1025)), (_group, dict(T=1 << 28, k=8)), (_expert, dict(E=2048)),
    (_linear, dict(N=1 << 30, rows=1 << 20)), (_quant, dict(F=1 << 25))])
def test_beyond_the_limits(lib, call, kw):
    assert call(lib, **kw) == L.LORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("call,kw", [
    (_route, dict(T=0, logits=None)), (_quant, dict(rows=0, x=None)),
    (_dequant, dict(rows=0, out=None)), (_linear, dict(rows=0, xc=None)),
    (_expert, dict(rows=0, off=None)), (_combine, dict(T=0, y=None))])
def test_empty_calls_launch_nothing(lib, call, kw):
    assert call(lib, **kw) == L.LORA_OK


def test_binding_refuses_tensors():
    import torch
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    ids, w = torch.zeros(4, 8, dtype=torch.int32), torch.zeros(4, 8)
    for bad in (dict(topk_ids=ids.long()), dict(topk_weights=w.half()), dict()):
        args = dict(logits=x, bias=None, topk_ids=ids, topk_weights=w, T=4, num_experts=64, top_k=8)
        with pytest.raises(L.LoraError):      # the last: host tensors
            L.lora_route_experts(**{**args, **bad})
    with pytest.raises(L.LoraError, match="element type"):
        L.lora_route_experts(x.long(), None, ids, w, 4, 64, 8)
    with pytest.raises(L.LoraError, match="type"):
        L.lora_route_experts(FAKE, None, FAKE, FAKE, 4, 64, 8)


# ---------------------------------------------------------------------------
# oracle pins
# ---------------------------------------------------------------------------

def test_oracle_route_by_hand():
    """Logits ln 1, ln 2, ln 3, ln 4: softmax .1 .2 .3 .4.  Top-2: experts 3 and
    2; renormalised 4/7 and 3/7.  A bias of .35 on expert 0 makes its key .45:
    it is chosen first, with its own score .1."""
    x = np.log([[1.0, 2.0, 3.0, 4.0]])
    ids, w, flags = O.route(x, None, 2, renormalize=False)
    assert ids.tolist() == [[3, 2]] and flags == 0
    assert np.allclose(w, [[0.4, 0.3]], rtol=1e-14)
    ids, w, _ = O.route(x, None, 2)
    assert np.allclose(w, [[4 / 7, 3 / 7]], rtol=1e-14)
    ids, w, _ = O.route(x, [0.35, 0, 0, 0], 2, renormalize=False, scale=2.0)
    assert ids.tolist() == [[0, 3]] and np.allclose(w, [[0.2, 0.8]], rtol=1e-14)


def test_oracle_route_groups_by_hand():
    """Keys 5 1 | 3 4: the best group by its largest is the first (5 > 4), by the
    sum of two the second (7 > 6).  Sigmoid leaves the order, so logits serve."""
    x = np.array([[0.5, -3.0, 0.3, 0.4]])
    assert O.route(x, None, 1, "sigmoid", 2, 1, False)[0].tolist() == [[0]]
    assert O.route(x, None, 1, "sigmoid", 2, 1, True)[0].tolist() == [[3]]
    # ties to the lowest group and expert; masked experts are never chosen
    assert O.route(np.zeros((1, 4)), None, 2, "sigmoid", 2, 1)[0].tolist() == [[0, 1]]
    ids, w, flags = O.route([[-np.inf, 1.0, np.nan, -np.inf]], None, 2)
    assert ids.tolist() == [[1, -1]] and w.tolist() == [[1.0, 0.0]] and flags == O.FLAG_NONFINITE


def test_oracle_group_by_hand():
    """Tokens 0..2 choose (1, 0), (1, -1), (0, 1): expert 0 gets tokens 0, 2 and
    expert 1 tokens 0, 1, 2."""
    ids = np.array([[1, 0], [1, -1], [0, 1]])
    off, tok, pair, slot, flags = O.group(ids, [7, -1, 5], 2)
    assert off.tolist() == [0, 2, 5] and tok.tolist() == [0, 2, 0, 1, 2]
    assert pair.tolist() == [[2, 0], [3, -1], [1, 4]]
    assert slot.tolist() == [7, 5, 7, -1, 5] and flags == 0


def test_oracle_quantize_by_hand():
    """max |v| = 10: e = floor(log2 10) - 2 = 1, so v / 2.  10 -> 5 (a tie of 4
    and 6: code 6 is the even one, 4), 0.5 -> .25 (tie of 0 and .5: 0), 1.5 -> .75
    (tie of .5 and 1: code 2, 1), -7 -> -3.5 (tie of 3 and 4: code 6, 4)."""
    v = np.zeros((1, 32))
    v[0, :4] = [10.0, 0.5, 1.5, -7.0]
    codes, scales = O.mx_quantize(v)
    assert scales.tolist() == [[128]] and codes[0, :4].tolist() == [6, 0, 2, 14]
    assert O.mx_values(codes, scales)[0, :4].tolist() == [8.0, 0.0, 2.0, -8.0]
    assert (O.unpack(O.pack(codes)) == codes).all()
    # every value of the format is a fixed point
    w = np.concatenate([O.E2M1, -O.E2M1, O.E2M1, -O.E2M1])[None] * 2.0 ** -5
    c, s = O.mx_quantize(w)
    assert (O.mx_values(c, s) == w).all()
    # beyond 6 times the scale: 7.9 has e = 0 and becomes 6
    v[:] = 0
    v[0, 0] = 7.9
    assert O.mx_values(*O.mx_quantize(v))[0, 0] == 6.0
    v[0, 1] = np.inf
    assert O.mx_quantize(v)[1].tolist() == [[255]]


def test_oracle_combine_by_hand():
    y = np.array([[1.0, 2.0], [10.0, 20.0]])
    out, _, flags = O.combine(y, np.array([[1, 0], [-1, 1], [0, 5]]),
                              np.array([[0.5, 2.0], [9.0, 0.1], [1.0, 1.0]]), np.ones((3, 2)))
    assert np.allclose(out, [[8.0, 15.0], [2.0, 3.0], [2.0, 3.0]]) and flags == O.FLAG_BAD_ROW


# ---------------------------------------------------------------------------
# ordering between the CTAs of a cluster
# ---------------------------------------------------------------------------

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "adapter_lora_serving_b200", "csrc")


def _csrc():
    for name in sorted(os.listdir(CSRC)):
        yield name, open(os.path.join(CSRC, name)).read()


def test_arrivals_at_another_cta_have_cluster_scope():
    """An arrival without a scope orders the arriving CTA's accesses for that CTA
    alone, whatever the waiting side acquires."""
    found = 0
    for name, text in _csrc():
        for op in re.findall(r'"(mbarrier\.arrive[a-z_.:]*shared::cluster[a-z0-9_.:]*)', text):
            found += 1
            assert re.search(r"\.(release|relaxed)\.cluster\.", op), f"{name}: {op}"
    assert found


def test_scales_of_the_second_cta_are_released():
    """The reordered scales are plain stores to shared memory, which the tensor core
    reads on the other CTA's request: the arrival that announces them releases them
    at cluster scope, and every wait of that kernel acquires there."""
    text = dict(_csrc())["mx_linear.cu"]
    release = 'if (RELEASE) asm volatile("fence.release.sync_restrict::shared::cta.cluster;"'
    assert release in text and "if (PAIR) arrive_at_first<true>(&ready[b.s]);" in text
    assert "fence.acquire.sync_restrict::shared::cluster.cluster;" in text
    pair = text[text.index("mx_linear_pair_kernel(const __grid_constant__"):]
    assert "wait_or_stop<true>(" in pair and "wait_or_stop(" not in pair


def test_warps_give_up_together():
    """A bounded wait ahead of warp-wide instructions ends alike in all lanes: those
    of the warps that reorder scales and that drain the accumulator."""
    text = dict(_csrc())["mx_linear.cu"]
    waits = re.findall(r"(\w+)(?:<true>)?\((&raw\[b\.s\]|&accfull\[acc\.s\]), ", text)
    assert len(waits) == 4 and {w for w, _ in waits} == {"warp_wait"}
    assert "__all_sync(0xffffffffu, wait_or_stop" in text


def test_oracle_route_saturated_by_hand():
    """Sigmoids of 50 and 60 are 1 in 64 bits: with one bias for all experts the
    logits decide, with several the lowest index."""
    x = [[50.0, 60.0, 0.0, 50.0]]
    for bias in (None, [0.0] * 4, [2.5] * 4):
        assert O.route(x, bias, 3, "sigmoid")[0].tolist() == [[1, 0, 3]]
        assert O.route(x, bias, 3, "sigmoid", 2, 1)[0][0, :2].tolist() == [1, 0]
    assert O.route(x, [0.0, 0.0, 0.25, 0.0], 3, "sigmoid")[0].tolist() == [[0, 1, 3]]


def test_combine_at_its_widest(lib):
    """65535 blocks of 1024 columns are the grid's second dimension at its end."""
    assert _combine(lib, T=0, F=65535 * 1024) == L.LORA_OK
    for F in (65535 * 1024 + 8, 1 << 26):
        assert _combine(lib, T=0, F=F) == L.LORA_ERR_UNSUPPORTED


@pytest.mark.parametrize("by", [0, 4, -4, 4092, -4092])
def test_group_in_place_is_refused(lib, by):
    """Many pairs keep their counts in pair_row while the ids are still read."""
    assert _group(lib, ids=FAKE, pair=FAKE + by, T=512, k=2) == L.LORA_ERR_INVALID
    assert "overlaps" in lib.lora_last_error().decode()


def test_oracle_route_with_every_group_kept_by_hand():
    """Sums of two scores decide nothing when no group is left out."""
    x = [[50.0, 60.0, 0.0, 50.0]]
    for bias in (None, [1.0] * 4):
        assert O.route(x, bias, 3, "sigmoid", 2, 2, True)[0].tolist() == [[1, 0, 3]]
