"""Group-limited routing and the orthogonalisation without a GPU: the oracle's
definitions on cases worked out by hand and against differences, and the
refusals of the C entry points."""
import ctypes

import numpy as np
import pytest

from mixture_experts_ffn_bias_b200 import binding as B
from mixture_experts_ffn_bias_b200 import build as build_mod
from oracle import moe_oracle as O


@pytest.fixture(scope="module")
def lib():
    build_mod.build()
    return B.lib()


class _Addr:
    """An address with a shape; never dereferenced (every call is refused)."""

    def __init__(self, shape=(), addr=1 << 20, stride=None, nbytes=0):
        self.shape, self._a, self._n = shape, addr, nbytes
        st, out = 1, []
        for n in reversed(shape):
            out.append(st)
            st *= n
        self._st = tuple(stride) if stride else tuple(reversed(out))

    def data_ptr(self):
        return self._a

    def stride(self, i=None):
        return self._st if i is None else self._st[i]

    def numel(self):
        return self._n

    def element_size(self):
        return 1


# ------------------------------------------------------------------- oracle
def test_groups_limit_the_choice():
    # group 0 holds the best expert, group 1 the best pair
    l = np.log(np.array([[0.9, 0.1, 0.7, 0.6]]) / (1 - np.array([[0.9, 0.1, 0.7, 0.6]])))
    idx, w, _ = O.route_groups(l, 2, O.GATE_SIGMOID, False, n_group=2, topk_group=1)
    assert idx.tolist() == [[2, 3]] and np.allclose(w, [[0.7, 0.6]])
    idx, _, _ = O.route_groups(l, 2, O.GATE_SIGMOID, False, n_group=2, topk_group=1,
                               group_score=1)
    assert idx.tolist() == [[0, 1]]
    idx, w, _ = O.route_groups(l, 2, O.GATE_SIGMOID, True, n_group=2, topk_group=2, scale=2.0)
    assert idx.tolist() == [[0, 2]] and np.allclose(w, [[1.125, 0.875]])


def test_one_group_is_the_plain_router():
    rng = np.random.default_rng(0)
    x, wr = rng.standard_normal((50, 8)), rng.standard_normal((12, 8))
    b = rng.uniform(-0.5, 0.5, 12)
    for gate in (O.GATE_SOFTMAX, O.GATE_SIGMOID):
        for space in (0, 1):
            r = O.router(x, wr, 3, gate, True, b, bias_space=space)
            idx, w, _ = O.route_groups(r.logits, 3, gate, True, b, bias_space=space)
            assert np.array_equal(idx, r.topk_idx)
            np.testing.assert_allclose(w, r.topk_w, rtol=1e-14)


def test_masked_experts_and_tokens():
    ninf = -np.inf
    l = np.array([[ninf, ninf, ninf, ninf], [0.0, ninf, np.nan, 1.0], [1.0, 2.0, 3.0, 4.0],
                  [0.0, 1.0, 2.0, 3.0]])
    idx, w, _ = O.route_groups(l, 3, O.GATE_SIGMOID, True, token_mask=[1, 1, 0, 1],
                               sel_bias=[0, 0, 0, ninf])
    assert idx.tolist() == [[-1, -1, -1], [0, -1, -1], [-1, -1, -1], [2, 1, 0]]
    assert np.all(w[0] == 0) and np.all(w[2] == 0) and w[1, 0] > 0.99
    idx, _, _ = O.route_groups(l, 3, O.GATE_SOFTMAX, True)
    assert idx[1].tolist() == [-1, -1, -1]      # a NaN leaves a softmax row without scores


@pytest.mark.parametrize("gate", [O.GATE_SOFTMAX, O.GATE_SIGMOID])
@pytest.mark.parametrize("norm", [True, False])
def test_routing_gradient_against_differences(gate, norm):
    rng = np.random.default_rng(4)
    l = rng.standard_normal((6, 12))
    dw = rng.standard_normal((6, 3))
    f = lambda z: O.route_groups(z, 3, gate, norm, n_group=3, topk_group=2, scale=1.5)
    idx, w, _ = f(l)
    g = O.route_groups_backward(l, idx, dw, gate, norm, 1.5)
    h = 1e-6
    for t in range(6):
        for e in range(12):
            z = l.copy()
            z[t, e] += h
            i1, w1, _ = f(z)
            z[t, e] -= 2 * h
            i0, w0, _ = f(z)
            assert np.array_equal(i1, idx) and np.array_equal(i0, idx)
            # central differences: h^2 and 1e-16 / h, both below 1e-9
            assert abs(np.sum(dw * (w1 - w0)) / (2 * h) - g[t, e]) < 1e-8


def test_orthogonalize_is_the_polynomial_of_the_singular_values():
    rng = np.random.default_rng(5)
    for shape in ((1, 7, 11), (2, 9, 4), (1, 1, 5), (1, 6, 6)):
        g = rng.standard_normal(shape)
        out = O.orthogonalize(g, eps=1e-7, scale=0.5)
        a, b, c = (float(np.float32(v)) for v in (3.4445, -4.7750, 2.0315))
        for m, o in zip(g, out):
            u, s, vt = np.linalg.svd(m, full_matrices=False)
            s = s / (np.linalg.norm(m) + float(np.float32(1e-7)))
            for _ in range(5):
                s = a * s + b * s ** 3 + c * s ** 5
            np.testing.assert_allclose(o, 0.5 * (u * s) @ vt, atol=1e-12)


# ---------------------------------------------------------------- refusals
def test_struct_sizes():
    assert ctypes.sizeof(B.MoEGroupOpts) == 32
    assert ctypes.sizeof(B.MoEOrthoConfig) == 80
    assert B.MoEOrthoConfig.g_row_stride.offset == 48


CFG = dict(T=16, d_model=128, n_experts=16, d_ff=128, top_k=4)


@pytest.mark.parametrize("field,value,expect", [
    ("n_group", 0, B.MOE_ERR_INVALID), ("n_group", 5, B.MOE_ERR_INVALID),
    ("topk_group", 0, B.MOE_ERR_INVALID), ("topk_group", 5, B.MOE_ERR_INVALID),
    ("group_score", 0, B.MOE_ERR_INVALID), ("group_score", 3, B.MOE_ERR_INVALID),
    ("bias_space", 2, B.MOE_ERR_INVALID), ("logits_dtype", 2, B.MOE_ERR_INVALID),
    ("scale", float("inf"), B.MOE_ERR_INVALID), ("scale", float("nan"), B.MOE_ERR_INVALID),
])
def test_route_options_refused(lib, field, value, expect):
    cfg = B.make_config(**CFG)
    o = B.make_group_opts(4, 2)
    setattr(o, field, value)
    l = _Addr((16, 16))
    assert B.moe_route_groups(cfg, o, l, None, None, l, l, stream=0, check=False) == expect
    assert B.moe_route_groups_backward(cfg, o, l, l, l, l, stream=0, check=False) == expect
    w = {k: l for k in ("w1", "w3", "w2")}
    ws = _Addr(nbytes=B.moe_workspace_size(cfg))
    assert B.moe_forward_grouped(cfg, o, l, l, None, None, None, w, l, l, l, l, ws, stream=0,
                                 check=False) == expect
    assert B.moe_backward_grouped(cfg, o, l, l, None, w, l, l, l, l, l, w, ws, ws, stream=0,
                                  check=False) == expect


def test_route_arguments_refused(lib):
    cfg = B.make_config(**CFG)
    o = B.make_group_opts(4, 2)
    l, odd = _Addr((16, 16)), _Addr((16, 16), addr=(1 << 20) + 2)
    run = lambda *a: B.moe_route_groups(cfg, o, *a, stream=0, check=False)
    assert run(odd, None, None, l, l) == B.MOE_ERR_INVALID
    assert run(l, odd, None, l, l) == B.MOE_ERR_INVALID
    assert run(l, None, None, odd, l) == B.MOE_ERR_INVALID
    assert run(l, None, None, l, None) == B.MOE_ERR_INVALID
    assert run(_Addr((16, 16), stride=(15, 1)), None, None, l, l) == B.MOE_ERR_INVALID
    bwd = lambda *a: B.moe_route_groups_backward(cfg, o, *a, stream=0, check=False)
    assert bwd(l, l, None, l) == B.MOE_ERR_INVALID
    assert bwd(l, l, l, odd) == B.MOE_ERR_INVALID
    assert bwd(l, None, l, l) == B.MOE_ERR_INVALID
    assert bwd(l, l, l, _Addr((16, 16), stride=(8, 1))) == B.MOE_ERR_INVALID
    # shapes and strides the binding itself refuses
    for bad in (_Addr((16, 15)), _Addr((15, 16)), _Addr((16, 16), stride=(1, 16))):
        with pytest.raises(B.MoEError):
            run(bad, None, None, l, l)
        with pytest.raises(B.MoEError):
            bwd(l, l, l, bad)
    big = B.make_config(**{**CFG, "n_experts": 66})
    assert B.moe_route_groups(big, B.make_group_opts(33, 2), _Addr((16, 66)), None, None, l, l,
                              stream=0, check=False) == B.MOE_ERR_UNSUPPORTED
    # the layer calls take fp32 logits options only, and their options
    w = {k: l for k in ("w1", "w3", "w2")}
    ws = _Addr(nbytes=B.moe_workspace_size(cfg))
    o16 = B.make_group_opts(4, 2, logits_dtype=B.DTYPE_BF16)
    assert B.moe_forward_grouped(cfg, o16, l, l, None, None, None, w, l, l, l, l, ws, stream=0,
                                 check=False) == B.MOE_ERR_INVALID
    assert lib.moe_forward_grouped(ctypes.byref(cfg), None, *[None] * 11, 0, None) == \
        B.MOE_ERR_INVALID
    assert lib.moe_backward_grouped(ctypes.byref(cfg), None, *[None] * 11, 0, None, 0, None) == \
        B.MOE_ERR_INVALID
    # no tokens: nothing to do, nothing dereferenced
    none = B.make_config(**{**CFG, "T": 0})
    e = _Addr((0, 16))
    assert B.moe_route_groups(none, o, e, None, None, None, None, stream=0) == B.MOE_OK
    assert B.moe_route_groups_backward(none, o, e, None, None, e, stream=0) == B.MOE_OK


@pytest.mark.parametrize("kw,expect", [
    (dict(batch=-1), B.MOE_ERR_INVALID), (dict(rows=0), B.MOE_ERR_INVALID),
    (dict(cols=0), B.MOE_ERR_INVALID), (dict(steps=0), B.MOE_ERR_INVALID),
    (dict(in_dtype=2), B.MOE_ERR_INVALID), (dict(out_dtype=-1), B.MOE_ERR_INVALID),
    (dict(eps=0.0), B.MOE_ERR_INVALID), (dict(eps=float("nan")), B.MOE_ERR_INVALID),
    (dict(scale=float("inf")), B.MOE_ERR_INVALID),
    (dict(coeffs=(float("nan"), 0.0, 0.0)), B.MOE_ERR_INVALID),
    (dict(steps=33), B.MOE_ERR_UNSUPPORTED), (dict(rows=65537), B.MOE_ERR_UNSUPPORTED),
    (dict(batch=65536), B.MOE_ERR_UNSUPPORTED),
    # polynomials whose iterates leave the fp16 planes' range
    (dict(coeffs=(3.4445, 0.0, 0.0)), B.MOE_ERR_UNSUPPORTED),
    (dict(coeffs=(1.5, -9.0, 0.0)), B.MOE_ERR_UNSUPPORTED),
    (dict(coeffs=(2.0, 1.0, 1.0), steps=3), B.MOE_ERR_UNSUPPORTED),
])
def test_orthogonalize_configuration_refused(lib, kw, expect):
    full = dict(batch=2, rows=32, cols=48)
    full.update(kw)
    cfg = B.make_ortho_config(**full)
    assert B.moe_orthogonalize_workspace_size(cfg) == 0
    st = lib.moe_orthogonalize(ctypes.byref(cfg), 1 << 20, 1 << 20, 1 << 20, 1 << 40, None)
    assert st == expect


def test_orthogonalize_arguments_refused(lib):
    cfg = B.make_ortho_config(2, 32, 48, B.DTYPE_F32, B.DTYPE_BF16)
    n = B.moe_orthogonalize_workspace_size(cfg)
    assert n > 0
    for coeffs in ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (3.0, -3.2, 1.2)):   # usual ones
        assert B.moe_orthogonalize_workspace_size(
            B.make_ortho_config(2, 32, 48, coeffs=coeffs, steps=20)) > 0
    g, ws = _Addr((2, 32, 48)), _Addr(nbytes=n)
    run = lambda *a: B.moe_orthogonalize(cfg, *a, stream=0, check=False)
    assert run(_Addr((2, 32, 48), addr=(1 << 20) + 2), g, ws) == B.MOE_ERR_INVALID
    assert run(g, _Addr((2, 32, 48), addr=(1 << 20) + 1), ws) == B.MOE_ERR_INVALID
    assert run(g, g, _Addr(addr=(1 << 20) + 16, nbytes=n)) == B.MOE_ERR_INVALID
    assert run(g, g, _Addr(nbytes=n - 1)) == B.MOE_ERR_WORKSPACE
    # a row stride below the columns, a batch stride below the matrix
    assert run(_Addr((2, 32, 48), stride=(2000, 40, 1)), g, ws) == B.MOE_ERR_INVALID
    assert run(g, _Addr((2, 32, 48), stride=(1535, 48, 1)), ws) == B.MOE_ERR_INVALID
    for bad in (_Addr((2, 32, 47)), _Addr((32, 48)), _Addr((2, 32, 48), stride=(1536, 1, 32))):
        with pytest.raises(B.MoEError):
            run(bad, g, ws)
    empty = B.make_ortho_config(0, 32, 48)
    assert lib.moe_orthogonalize(ctypes.byref(empty), None, None, None, 0, None) == B.MOE_OK


def test_orthogonalize_terms_by_the_growth_of_errors(lib):
    """bf16 results of products of one term only where the errors those leave
    stay bounded: the planes a workspace has room for tell which are taken."""
    size = lambda **kw: B.moe_orthogonalize_workspace_size(
        B.make_ortho_config(3, 333, 517, **kw))
    pairs = lambda **kw: size(**kw) == size(**{**kw, "out_dtype": B.DTYPE_F32})
    assert not any(pairs(steps=n) for n in range(1, 6))
    assert all(pairs(steps=n) for n in range(6, 33))
    for coeffs in ((2.0, -1.5, 0.5), (1.5, -0.5, 0.0), (3.0, -3.2, 1.2), (1.875, -1.25, 0.375)):
        assert not any(pairs(steps=n, coeffs=coeffs) for n in (1, 5, 8, 32)), coeffs
    # steeper than the usual polynomial
    assert pairs(steps=4, coeffs=(3.7418, -5.5913, 2.3037))
    assert pairs(steps=2, coeffs=(4.0848, -6.8946, 2.9270))
    # a value that becomes zero on the way: its direction has no relative error
    assert pairs(steps=2, coeffs=(1.0, -1.0, 0.0))


@pytest.mark.parametrize("rows,cols", [(333, 517), (130, 130), (100, 5000), (5000, 100), (1, 1),
                                       (100, 200), (65536, 65536)])
@pytest.mark.parametrize("out_dtype", [B.DTYPE_F32, B.DTYPE_BF16])
def test_orthogonalize_of_no_matrices(lib, rows, cols, out_dtype):
    """An empty batch has a workspace size like any other, and is a no-op."""
    cfg = B.make_ortho_config(0, rows, cols, out_dtype=out_dtype)
    n = B.moe_orthogonalize_workspace_size(cfg)
    assert n == 256
    g = _Addr((0, rows, cols))
    assert B.moe_orthogonalize(cfg, g, g, _Addr(nbytes=n), stream=0) == B.MOE_OK
    assert B.moe_orthogonalize(cfg, g, g, None, stream=0) == B.MOE_OK


def test_orthogonalize_refuses_expanded_tensors(lib):
    """Rows or matrices of stride 0: the C call takes 0 for dense, and would read
    or write memory the tensor does not have."""
    cfg = B.make_ortho_config(2, 32, 48, B.DTYPE_F32, B.DTYPE_F32)
    ws = _Addr(nbytes=B.moe_orthogonalize_workspace_size(cfg), addr=(1 << 20) + 16)   # refused
    g = _Addr((2, 32, 48))
    for st in ((0, 48, 1), (1536, 0, 1), (0, 0, 1)):
        bad = _Addr((2, 32, 48), stride=st)
        for args in ((bad, g), (g, bad)):
            with pytest.raises(B.MoEError):
                B.moe_orthogonalize(cfg, *args, ws, stream=0, check=False)
    # one row, or one matrix: its stride says nothing
    one = B.make_ortho_config(1, 1, 48, B.DTYPE_F32, B.DTYPE_F32)
    g = _Addr((1, 1, 48), stride=(0, 0, 1))
    assert B.moe_orthogonalize(one, g, g, _Addr(nbytes=0), stream=0, check=False) == \
        B.MOE_ERR_WORKSPACE


def test_routing_looks_at_its_own_fields_alone(lib):
    """The sizes and type of a layer do not matter to calls on given logits: any
    values pass, and a bad one of routing's own fields is refused beside them."""
    o, l = B.make_group_opts(4, 2), _Addr((16, 16))
    for other in (dict(d_model=100, d_ff=1), dict(d_model=0, d_ff=0), dict(d_model=-1, d_ff=7)):
        cfg = B.make_config(**{**CFG, **other, "T": 0})
        e = _Addr((0, 16))
        assert B.moe_route_groups(cfg, o, e, None, None, None, None, stream=0) == B.MOE_OK
        assert B.moe_route_groups_backward(cfg, o, e, None, None, e, stream=0) == B.MOE_OK
        assert B.moe_check_config(cfg) != B.MOE_OK
        for field, value, expect in (("top_k", 17, B.MOE_ERR_INVALID),
                                     ("top_k", 0, B.MOE_ERR_INVALID),
                                     ("gate", 2, B.MOE_ERR_INVALID),
                                     ("norm_topk_prob", 2, B.MOE_ERR_INVALID),
                                     ("T", -1, B.MOE_ERR_INVALID)):
            bad = B.make_config(**{**CFG, **other})
            setattr(bad, field, value)
            g = _Addr((max(bad.T, -1), 16))
            assert B.moe_route_groups(bad, o, g, None, None, l, l, stream=0,
                                      check=False) == expect
        # the layer calls look at all of them
        cfg = B.make_config(**{**CFG, **other})
        w = {k: l for k in ("w1", "w3", "w2")}
        assert B.moe_forward_grouped(cfg, o, l, l, None, None, None, w, l, l, l, l,
                                     _Addr(nbytes=1 << 30), stream=0, check=False) != B.MOE_OK
