"""The language-model selections without a GPU: argument checks of the C-ABI
(made before any device work) and the float64 definitions the GPU tests use."""
import ctypes as C

import numpy as np
import pytest

from oracle import selections as ref


def test_sample_tokens_checks_arguments(pk):
    from streaming_selection_primitive_gb300 import _abi
    lib, p, odd = pk.lib(), C.c_void_p(256), C.c_void_p(257)
    how = _abi.Sampling(all_temperature=1.0, all_top_p=1.0)

    def call(logits=p, kind=_abi.F32, rows=2, n=10, ld=10, noise=p, noise_ld=10, mask=None, mask_ld=0, how=how, tok=p, lp=p):
        return lib.profk_sample_tokens(logits, kind, rows, n, ld, noise, noise_ld, mask, mask_ld, how, tok, lp, None)

    assert call(rows=0) == 0  # nothing to do
    for bad in ({"kind": 3}, {"rows": -1}, {"n": 0}, {"ld": 9}, {"noise_ld": 9}, {"logits": None}, {"noise": None},
                {"tok": None}, {"lp": None}, {"how": None}, {"mask": p, "mask_ld": -1}, {"n": 33, "ld": 33, "noise_ld": 33, "mask": p, "mask_ld": 1}):
        assert call(**bad) == _abi.PROFK_ERR_INVALID, bad
    for bad in ({"logits": odd}, {"noise": odd}, {"tok": C.c_void_p(260)}, {"lp": odd}, {"mask": odd, "mask_ld": 1},
                {"n": 1 << 31, "ld": 1 << 31, "noise_ld": 1 << 31}, {"rows": 1 << 31}):
        assert call(**bad) == _abi.PROFK_ERR_UNSUPPORTED, bad
    nan = float("nan")
    for bad in ({"all_temperature": -1.0}, {"all_temperature": nan}, {"all_temperature": 1.0, "all_top_p": nan},
                {"all_temperature": 1.0, "all_min_p": nan}):
        assert call(how=_abi.Sampling(**bad)) == _abi.PROFK_ERR_INVALID, bad


def test_route_checks_arguments(pk):
    from streaming_selection_primitive_gb300 import _abi
    lib, p, odd = pk.lib(), C.c_void_p(256), C.c_void_p(257)
    how = _abi.Routing(0, 1)

    def call(logits=p, kind=_abi.BF16, tokens=4, E=16, ld=16, k=2, how=how, gates=p, experts=p, counts=p, loss=None):
        return lib.profk_route(logits, kind, tokens, E, ld, k, how, gates, experts, counts, loss, None)

    for bad in ({"kind": -1}, {"tokens": -1}, {"E": 0}, {"ld": 15}, {"k": 0}, {"k": 17}, {"how": None},
                {"how": _abi.Routing(2, 1)}, {"logits": None}, {"gates": None}, {"experts": None}, {"counts": None}):
        assert call(**bad) == _abi.PROFK_ERR_INVALID, bad
    for bad in ({"E": 1025, "ld": 1025}, {"E": 64, "ld": 64, "k": 33}, {"tokens": 1 << 32}, {"logits": odd}, {"gates": odd},
                {"experts": C.c_void_p(260)}, {"counts": C.c_void_p(260)}, {"loss": odd}, {"how": _abi.Routing(0, 1, odd)}):
        assert call(**bad) == _abi.PROFK_ERR_UNSUPPORTED, bad

    def back(logits=p, tokens=4, E=16, ld=16, k=2, how=how, chosen=p, counts=p, dg=p, dl=p, out=p, out_ld=16):
        return lib.profk_route_backward(logits, _abi.BF16, tokens, E, ld, k, how, chosen, counts, dg, dl, out, out_ld, None)

    assert back(tokens=0) == 0
    for bad in ({"out_ld": 15}, {"counts": None}, {"chosen": None}, {"out": None}, {"logits": None}, {"k": 17}):
        assert back(**bad) == _abi.PROFK_ERR_INVALID, bad
    for bad in ({"chosen": C.c_void_p(260)}, {"dg": odd}, {"dl": odd}, {"out": odd}, {"E": 1025, "ld": 1025, "out_ld": 1025}):
        assert back(**bad) == _abi.PROFK_ERR_UNSUPPORTED, bad


def test_token_definition():
    l = np.log(np.array([1.0, 4.0, 2.0, 4.0, 1.0]))
    all_ = np.ones(5, bool)
    even = np.ones(5)
    # Order 1, 3, 2, 0, 4 with masses 4 4 2 1 1 of 12.
    assert ref.order_of(l).tolist() == [1, 3, 2, 0, 4]
    q = np.array([1.0, 1.0, 1e-3, 1.0, 1e-4])
    assert ref.token(l, q, all_, 1.0, 0, 1.0, 0.0)[0] == 4
    assert ref.token(l, q, all_, 1.0, 3, 1.0, 0.0)[0] == 2      # 0 and 4 cut
    assert ref.token(l, q, all_, 1.0, 0, 0.6, 0.0)[0] == 1      # mass before 2 is 2/3
    assert ref.token(l, q, all_, 1.0, 0, 0.7, 0.0)[0] == 2
    assert ref.token(l, q, all_, 1.0, 3, 0.7, 0.0)[0] == 1      # of the first three: 4/5 before 2
    assert ref.token(l, q, all_, 1.0, 0, 1.0, 0.4)[0] == 2      # w = 1, 1, 1/2, 1/4, 1/4
    assert ref.token(l, q, all_, 1.0, 0, 1.0, 0.6)[0] == 1
    assert ref.token(l, q, all_, 0.0, 0, 1.0, 0.0)[:2] == (1, 0.0)
    assert ref.token(l, even, all_, 1.0, 0, 0.0, 0.0)[:2] == (1, 0.0)
    assert np.isclose(ref.token(l, even, all_, 1.0, 0, 1.0, 0.0)[1], np.log(4 / 12))
    assert ref.token(l, even, ~all_, 1.0, 0, 1.0, 0.0)[:2] == (-1, -np.inf)
    l[2] = np.nan
    assert ref.token(l, even, all_, 1.0, 0, 1.0, 0.0)[0] == -1


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("normalize", [True, False])
def test_routing_gradient_definition(score, normalize):
    # The written-out gradient against central differences of the definition, in float64.
    rng = np.random.default_rng(3)
    z = rng.normal(size=(5, 9)).astype(np.float32)
    dg, dl, k, h = rng.normal(size=(5, 3)), 4.0, 3, 2.0 ** -10
    _, experts, counts, _ = ref.routing(z, k, score, normalize)
    grad = ref.routing_gradient(z, experts, counts, score, normalize, dg, dl)

    def f(zz):
        g, e, _, loss = ref.routing(zz, k, score, normalize)
        assert np.array_equal(e, experts)
        return (g * dg).sum() + dl * loss

    for t in range(5):
        for e in range(9):
            a, b = z.copy(), z.copy()
            a[t, e] += np.float32(h)
            b[t, e] -= np.float32(h)
            slope = (f(a) - f(b)) / (float(a[t, e]) - float(b[t, e]))
            assert abs(slope - grad[t, e]) < 1e-5 * (1 + np.abs(dg).sum())
