"""The routed layer's own refusals (adapter_lora_serving_b200.moe) on a host without
a GPU: what a call or the adapters hold wrong is refused before the first kernel."""
import os

import pytest

from adapter_lora_serving_b200 import lora as L

T, HIDDEN, INTER, E, K, SLOTS, R = 6, 64, 32, 8, 2, 3, 8


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(L.LIB_PATH):
        from adapter_lora_serving_b200 import build
        build.build()
    return L.load()


def _adapters(**bad):
    import torch
    from adapter_lora_serving_b200 import moe
    bf16, pairs = torch.bfloat16, 4
    ranks, scalings = torch.full((SLOTS,), R, dtype=torch.int32), torch.ones(SLOTS)
    index = torch.zeros(SLOTS * E, dtype=torch.int32)

    def pick(name, value):
        return bad.get(name, value)

    gate_up = moe.ExpertAdapters(pick("gu_a", torch.zeros(pairs, 2 * R, HIDDEN, dtype=bf16)),
                                 torch.zeros(pairs, 2 * INTER, R, dtype=bf16),
                                 pick("index", index), ranks, pick("scalings", scalings))
    down = moe.ExpertAdapters(torch.zeros(pairs, R, INTER, dtype=bf16),
                              pick("dn_b", torch.zeros(pairs, HIDDEN, R, dtype=bf16)), index,
                              pick("ranks", ranks), scalings)
    router = moe.RouterAdapters(pick("rt_a", torch.zeros(SLOTS, R, HIDDEN, dtype=bf16)),
                                pick("rt_b", torch.zeros(SLOTS, E, R, dtype=bf16)), ranks, scalings)
    return gate_up, down, router


def _layer(router=True, **bad):
    import torch
    from adapter_lora_serving_b200 import moe
    u8 = torch.uint8
    gate_up = (torch.zeros(E, 2 * INTER, HIDDEN // 2, dtype=u8), torch.zeros(E, 2 * INTER, HIDDEN // 32, dtype=u8))
    down = (torch.zeros(E, HIDDEN, INTER // 2, dtype=u8), torch.zeros(E, HIDDEN, INTER // 32, dtype=u8))
    gu, dn, rt = _adapters(**bad)
    return moe.MoeLayer(T, HIDDEN, INTER, E, K, gate_up, down, gu, dn, rt if router else None)


def _call(layer, monkeypatch, **bad):
    """forward on host tensors: the first kernel's entry point fails the test."""
    import torch

    def ran(*a, **kw):
        raise AssertionError("a kernel's entry point was called")

    for name in ("lora_apply_router", "lora_route_experts"):
        monkeypatch.setattr(L, name, ran)
    i32, bf16 = torch.int32, torch.bfloat16
    a = dict(x=torch.zeros(T, HIDDEN, dtype=bf16), gate_logits=torch.zeros(T, E, dtype=bf16),
             out=torch.zeros(T, HIDDEN, dtype=bf16), token_slot=torch.zeros(T, dtype=i32),
             token_order=torch.zeros(T, dtype=i32), slot_indptr=torch.zeros(SLOTS + 1, dtype=i32))
    a.update(bad)
    layer.forward(**a)


def _refusals():
    import torch
    bf16, i32 = torch.bfloat16, torch.int32
    return [
        (dict(gate_logits=torch.zeros(T, E)), "gate_logits has element type"),
        (dict(gate_logits=torch.zeros(T, E, dtype=torch.float16)), "gate_logits has element type"),
        (dict(gate_logits=torch.zeros(T, 2 * E, dtype=bf16)), "gate_logits has rows of 16"),
        (dict(x=torch.zeros(T, HIDDEN)), "x has element type"),
        (dict(x=torch.zeros(T, HIDDEN // 2, dtype=bf16)), "x has 32 features"),
        (dict(x=torch.zeros(T, 2 * HIDDEN, dtype=bf16)), "x has 128 features"),
        (dict(out=torch.zeros(T, HIDDEN)), "out has element type"),
        (dict(out=torch.zeros(T, HIDDEN // 2, dtype=bf16)), "out has rows of 32"),
        (dict(residual=torch.zeros(T, HIDDEN, dtype=torch.float16)), "residual has element type"),
        (dict(residual=torch.zeros(T, 2 * HIDDEN, dtype=bf16)), "residual has rows of 128"),
        (dict(token_slot=torch.zeros(T, dtype=torch.int64)), "token_slot has element type"),
        (dict(token_order=torch.zeros(T, dtype=torch.int64)), "token_order has element type"),
        (dict(slot_indptr=torch.zeros(SLOTS + 1)), "slot_indptr has element type"),
        (dict(err_flags=torch.zeros(1)), "err_flags has element type"),
        (dict(), "x is not on a CUDA device"),
    ]


@pytest.mark.parametrize("i", range(15))
def test_forward_refuses_before_any_kernel(i, monkeypatch):
    bad, why = _refusals()[i]
    # a tensor that is wrong in itself is named first; otherwise host tensors are
    if why.endswith("element type") and not why.startswith("x "):
        monkeypatch.setattr(L, "_pointers", _types_only)
    with pytest.raises(L.LoraError, match=why):
        _call(_layer(), monkeypatch, **bad)


def _types_only(op, tensors, kinds, least, names):
    """L._pointers for host tensors: every check but the device's."""
    if L._dtypes is None:
        L._import_torch()
    for t, kind, n, name in zip(tensors, kinds, least, names):
        if t is not None and (t.dtype is not L._dtypes[kind] or not t.is_contiguous() or t.numel() < n):
            what = "element type" if t.dtype is not L._dtypes[kind] else "too few or not contiguous"
            L._refuse(op, f"{name} has {what}")


@pytest.mark.parametrize("layout", ["transposed", "expanded", "few"])
@pytest.mark.parametrize("name", ["x", "gate_logits", "out"])
def test_forward_refuses_layouts(name, layout, monkeypatch):
    import torch
    n = E if name == "gate_logits" else HIDDEN
    t = {"transposed": torch.zeros(n, T, dtype=torch.bfloat16).t(),
         "expanded": torch.zeros(1, n, dtype=torch.bfloat16).expand(T, n),
         "few": torch.zeros(T - 1, n, dtype=torch.bfloat16)}[layout]
    if name == "x" and layout == "few":
        t = torch.zeros(T, n - 32, dtype=torch.bfloat16)
    monkeypatch.setattr(L, "_pointers", _types_only)
    with pytest.raises(L.LoraError, match=f"{name} has"):
        _call(_layer(), monkeypatch, **{name: t})


def test_logits_of_other_types_without_a_router_fold(monkeypatch):
    """They reach the routing, whose entry point takes them."""
    import torch
    monkeypatch.setattr(L, "_pointers", _types_only)
    for dtype in (torch.float32, torch.float16, torch.bfloat16):
        with pytest.raises(Exception) as e:     # of torch (no such device), or _call's own
            _call(_layer(router=False), monkeypatch, gate_logits=torch.zeros(T, E, dtype=dtype))
        assert not isinstance(e.value, L.LoraError)
    with pytest.raises(L.LoraError, match="gate_logits"):
        _call(_layer(router=False), monkeypatch, gate_logits=torch.zeros(T, E, dtype=torch.int32))


def test_adapters_are_checked_once():
    import torch
    bf16 = torch.bfloat16
    for bad in (dict(rt_a=torch.zeros(SLOTS, R, HIDDEN)),
                dict(rt_a=torch.zeros(SLOTS, R, HIDDEN // 2, dtype=bf16)),
                dict(rt_b=torch.zeros(SLOTS, R, E, dtype=bf16).transpose(1, 2)),
                dict(gu_a=torch.zeros(4, R, HIDDEN, dtype=bf16)),
                dict(dn_b=torch.zeros(4, HIDDEN, R, dtype=torch.float16)),
                dict(index=torch.zeros(SLOTS * E, dtype=torch.int64)),
                dict(index=torch.zeros(E, dtype=torch.int32)),
                dict(ranks=torch.full((SLOTS,), R)),
                dict(scalings=torch.ones(SLOTS, dtype=torch.float64))):
        with pytest.raises(ValueError, match="adapters"):
            _layer(**bad)
    _layer()


@pytest.mark.parametrize("router", [False, True])
def test_other_shapes_of_the_same_rows_pass(router, monkeypatch):
    """Logits by expert group, flat buffers, buffers with room for more tokens."""
    import torch
    bf16 = torch.bfloat16
    monkeypatch.setattr(L, "_pointers", _types_only)
    for kw in (dict(gate_logits=torch.zeros(T, 2, E // 2, dtype=bf16)),
               dict(gate_logits=torch.zeros(T * E, dtype=bf16)),
               dict(gate_logits=torch.zeros(T + 3, E, dtype=bf16)),
               dict(out=torch.zeros(T + 1, HIDDEN, dtype=bf16)),
               dict(x=torch.zeros(T, 4, HIDDEN // 4, dtype=bf16)),
               dict(residual=torch.zeros(T, HIDDEN, dtype=bf16))):
        with pytest.raises(Exception) as e:
            _call(_layer(router=router), monkeypatch, **kw)
        assert not isinstance(e.value, L.LoraError)
