"""Group-limited routing, its gradient and the orthogonalisation on the GPU,
through the binding, against the oracle's 64-bit definitions on the same
inputs; then all of them together as one training step of a layer."""
import numpy as np
import pytest
import torch

import _parity as P
from mixture_experts_ffn_bias_b200 import binding as B
from mixture_experts_ffn_bias_b200 import build as build_mod
from mixture_experts_ffn_bias_b200 import inputs as I
from mixture_experts_ffn_bias_b200.layer import MoELayer, to_device
from oracle import moe_oracle as O

pytestmark = pytest.mark.gpu

INF = float("inf")
SOFT, SIG = B.GATE_SOFTMAX, B.GATE_SIGMOID
# Weights: the softmax's sum is of terms within (2 + 1.16 |x|) 2^-23 of e^x
# (x = l - max), at most ln E + 2 of |x| in their weighted mean, so 1.1e-6; the
# score's own exponential 2 ulp and |x| 2^-24 for the rounding of x (|x| < 30
# here: 1.8e-6); sum, quotients and scale 6 roundings.  Sigmoid weights have
# only the last two parts.
W_RTOL = 4e-6


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")
    build_mod.build()
    B.lib()


def _logits(T, E, seed, dtype=torch.float32, pad=0, spread=1.2):
    rng = np.random.default_rng(seed)
    a = (spread * rng.standard_normal((T, E + pad)) + 0.6 * rng.standard_normal(E + pad))
    return torch.from_numpy(a.astype(np.float32)).to(dtype).cuda()[:, :E]


def _route(l, k, gate=SIG, norm=True, bias=None, mask=None, groups=1, topk_group=1, score=2,
           space=1, scale=1.0, stream=None):
    T, E = l.shape
    cfg = B.make_config(T, 128, E, 128, k, gate=gate, norm_topk_prob=int(norm))
    o = B.make_group_opts(groups, topk_group, score, space, scale,
                          B.DTYPE_BF16 if l.dtype == torch.bfloat16 else B.DTYPE_F32)
    idx = torch.full((T, k), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T, k), -7.0, device="cuda")
    B.moe_route_groups(cfg, o, l, bias, mask, idx, w, stream=stream)
    return cfg, o, idx, w


def _check(l, k, **kw):
    cfg, o, idx, w = _route(l, k, **kw)
    bias, mask = kw.get("bias"), kw.get("mask")
    ri, rw, s = O.route_groups(l.double().cpu().numpy(), k, kw.get("gate", SIG),
                               kw.get("norm", True),
                               None if bias is None else bias.cpu().numpy(),
                               kw.get("groups", 1), kw.get("topk_group", 1), kw.get("score", 2),
                               kw.get("space", 1), kw.get("scale", 1.0),
                               None if mask is None else mask.cpu().numpy())
    np.testing.assert_array_equal(idx.cpu().numpy(), ri)
    got = w.double().cpu().numpy()
    assert np.all(np.abs(got - rw) <= W_RTOL * np.abs(rw) + 1e-30)
    return cfg, o, idx, w


CASES = [
    # T, E, k, groups, topk_group, score, gate, space, norm
    (1, 64, 6, 8, 3, 2, SIG, 1, True),
    (1, 1, 1, 1, 1, 1, SOFT, 1, True),
    (3, 2, 2, 2, 1, 2, SIG, 1, True),
    (5, 33, 4, 1, 1, 2, SOFT, 1, False),
    (67, 96, 6, 6, 2, 2, SIG, 0, True),
    (67, 96, 6, 6, 2, 1, SOFT, 1, True),
    (130, 160, 6, 8, 3, 1, SOFT, 1, False),
    (200, 256, 8, 8, 4, 2, SIG, 1, True),
    (129, 255, 32, 3, 2, 2, SOFT, 1, True),
    (64, 224, 16, 32, 5, 2, SIG, 1, True),
    (64, 250, 9, 25, 7, 1, SIG, 1, False),
    (33, 128, 32, 16, 4, 2, SOFT, 0, True),
    (9, 256, 1, 2, 1, 2, SIG, 1, True),
]


@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_routing_matches_the_oracle(case, biased, dtype):
    T, E, k, groups, tg, score, gate, space, norm = case
    l = _logits(T, E, T + E, dtype, pad=5)
    rng = np.random.default_rng(E)
    bias = None
    if biased:
        bias = torch.from_numpy((0.2 * rng.uniform(-1, 1, E)).astype(np.float32)).cuda()
    mask = torch.from_numpy(rng.uniform(size=T) > 0.15).cuda() if T > 3 else None
    _check(l, k, gate=gate, norm=norm, bias=bias, mask=mask, groups=groups, topk_group=tg,
           score=score, space=space, scale=2.5)


@pytest.mark.parametrize("gate", [SIG, SOFT])
@pytest.mark.parametrize("space", [0, 1])
def test_routing_ties_and_near_ties(gate, space):
    """Equal keys go to the lower id; keys a few fp32 roundings apart are
    ordered as in fp64."""
    T, E, k = 96, 128, 8
    rng = np.random.default_rng(8)
    # few distinct logits, so that most choices are ties
    l = torch.from_numpy(rng.integers(-3, 4, (T, E)).astype(np.float32) * 0.5).cuda()
    zero = torch.zeros(E, device="cuda")
    few = torch.from_numpy(rng.integers(0, 3, E).astype(np.float32) * 0.25).cuda()
    for bias in (None, zero, few):
        for score in (1, 2):
            _check(l, k, gate=gate, space=space, bias=bias, groups=8, topk_group=4, score=score)
    # logits one or two ulp apart around a common value, and biases that
    # nearly undo the differences of the scores
    base = np.full((T, E), 0.7, np.float32)
    steps = rng.integers(0, 3, (T, E))
    near = base
    for _ in range(2):
        near = np.where(steps > 0, np.nextafter(near, np.float32(2)), near)
        steps = steps - 1
    l2 = torch.from_numpy(near).cuda()
    tiny = torch.from_numpy((rng.integers(0, 4, E) * 3e-8).astype(np.float32)).cuda()
    for bias in (None, tiny):
        for score in (1, 2):
            _check(l2, k, gate=gate, space=space, bias=bias, groups=16, topk_group=5,
                   score=score)
        _check(l2, 32, gate=gate, space=space, bias=bias)
    # scores that fp64 cannot tell apart: sigmoids of 40, softmax terms e^-800
    wide = torch.from_numpy(rng.choice([-800.0, -799.0, 40.0, 41.0, 0.0],
                                       (T, E)).astype(np.float32)).cuda()
    for bias in (None, zero):
        _check(wide, 32, gate=gate, space=space, bias=bias, groups=4, topk_group=3, score=1,
               norm=False)


@pytest.mark.parametrize("gate", [SIG, SOFT])
def test_routing_many_ties_at_the_border(gate):
    """Exact ties of the last chosen expert hide others whose keys differ by less
    than fp32 shows; logits so near zero that their fp64 scores are equal;
    and tokens whose logits are all equal."""
    T, E, k = 64, 128, 8
    rng = np.random.default_rng(12)
    l = np.full((T, E), 0.7, np.float32)
    up = rng.uniform(size=(T, E)) < 0.2
    l[up] = np.nextafter(np.float32(0.7), np.float32(1))
    l[:, ::7] = -1.0
    tiny = (rng.integers(0, 3, E) * 2e-8).astype(np.float32)
    small = (rng.integers(-2, 3, (T, E)) * 1e-18).astype(np.float32)
    flat = np.zeros((T, E), np.float32)
    for a in (l, small, flat):
        for b in (None, np.zeros(E, np.float32), tiny):
            for space in (0, 1):
                for groups, tg in ((1, 1), (8, 3)):
                    for score in (1, 2):
                        _check(torch.from_numpy(a).cuda(), k, gate=gate, space=space,
                               bias=None if b is None else torch.from_numpy(b).cuda(),
                               groups=groups, topk_group=tg, score=score)


def test_routing_signed_zeros():
    """-0 and 0 are equal: each expert once, in the order of their ids."""
    l = torch.zeros(8, 64, device="cuda")
    l[:, ::3] = -0.0
    l[:, 40:] = -1.0
    for bias in (None, torch.zeros(64, device="cuda")):
        for space in (0, 1):
            _check(l, 20, space=space, bias=bias, groups=4, topk_group=3, score=1)
            _check(l, 32, space=space, bias=bias)


@pytest.mark.parametrize("gate", [SIG, SOFT])
@pytest.mark.parametrize("space", [0, 1])
@pytest.mark.parametrize("score", [1, 2])
def test_routing_masked_values(gate, space, score):
    """-inf, the lowest finite value, NaN and +inf among logits and biases;
    tokens and groups with nothing eligible."""
    T, E, k = 40, 64, 6
    rng = np.random.default_rng(21)
    a = rng.standard_normal((T, E)).astype(np.float32)
    lowest = np.finfo(np.float32).min
    a[rng.uniform(size=(T, E)) < 0.2] = -np.inf
    a[5] = -np.inf                       # nothing eligible
    a[6, 3:] = -np.inf                   # fewer than k
    a[7, 8:] = lowest                    # all but a group at the lowest value
    a[8, 4] = np.nan
    a[9, 4] = np.inf
    a[10] = np.nan
    a[11, :32] = -np.inf                 # half of the groups empty
    a[12] = lowest
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for b in (None, "plain", "off", "low", "nan"):
        bb = bias.copy()
        if b == "off":
            bb[::3] = -np.inf
        if b == "low":
            bb[8:40] = lowest
        if b == "nan":
            bb[2] = np.nan
        l = torch.from_numpy(a).cuda()
        bt = None if b is None else torch.from_numpy(bb).cuda()
        for tg in (2, 8):
            _, _, idx, w = _check_nan(l, k, gate, space, bt, tg, score)
    lb = torch.from_numpy(a).cuda().to(torch.bfloat16)   # the lowest rounds to -inf
    _check_nan(lb, k, gate, space, None, 3, score)


def _check_nan(l, k, gate, space, bias, tg, score):
    out = _route(l, k, gate=gate, space=space, bias=bias, groups=8, topk_group=tg, score=score)
    with np.errstate(all="ignore"):
        ri, rw, _ = O.route_groups(l.double().cpu().numpy(), k, gate, True,
                                   None if bias is None else bias.cpu().numpy(), 8, tg, score,
                                   space)
    np.testing.assert_array_equal(out[2].cpu().numpy(), ri)
    got = out[3].double().cpu().numpy()
    # scores below fp32's normal numbers (1.2e-38) are rounded on its grid
    np.testing.assert_allclose(got, rw, rtol=W_RTOL, atol=1e-28)
    assert np.all(got[ri < 0] == 0)
    return out


def test_routing_rows_behind_are_left_and_runs_repeat():
    l = _logits(1000, 128, 3)
    idx = torch.full((1100, 8), -9, dtype=torch.int32, device="cuda")
    w = torch.full((1100, 8), -9.0, device="cuda")
    cfg = B.make_config(1000, 128, 128, 128, 8, gate=SIG)
    o = B.make_group_opts(8, 4)
    B.moe_route_groups(cfg, o, l, None, None, idx, w)
    assert torch.all(idx[1000:] == -9) and torch.all(w[1000:] == -9.0)
    i0, w0 = idx.clone(), w.clone()
    B.moe_route_groups(cfg, o, l, None, None, idx, w)
    assert torch.equal(i0, idx) and torch.equal(w0, w)


def test_routing_many_tokens_match_the_fp64_selection():
    """Enough tokens that some land inside every fp32 margin: against fp64 keys
    and a stable sort."""
    for gate, biased, dtype in ((SIG, True, torch.float32), (SOFT, False, torch.float32),
                                (SIG, False, torch.bfloat16), (SOFT, True, torch.bfloat16)):
        T, E, k, G, tg = 60000, 256, 8, 8, 4
        g = torch.Generator(device="cuda").manual_seed(5)
        l = torch.randn(T, E, generator=g, device="cuda").to(dtype)
        bias = torch.rand(E, generator=g, device="cuda") * 0.1 if biased else None
        _, _, idx, w = _route(l, k, gate=gate, bias=bias, groups=G, topk_group=tg)
        s = torch.sigmoid(l.double()) if gate == SIG else torch.softmax(l.double(), 1)
        key = s if bias is None else s + bias.double()
        gs = key.view(T, G, E // G).sort(2, descending=True).values[:, :, :2].sum(2)
        keep = torch.zeros(T, G, dtype=torch.bool, device="cuda")
        keep.scatter_(1, torch.sort(gs, dim=1, descending=True, stable=True).indices[:, :tg], True)
        key = key.masked_fill(~keep.repeat_interleave(E // G, 1), -INF)
        ref = torch.sort(key, dim=1, descending=True, stable=True).indices[:, :k]
        assert torch.equal(idx.long(), ref)
        rw = s.gather(1, ref)
        rw = rw / (rw.sum(1, keepdim=True) + 1e-9)
        assert torch.all((w.double() - rw).abs() <= W_RTOL * rw)


@pytest.mark.parametrize("E,k,groups,topk_group,pad", [(96, 6, 6, 2, 0), (63, 5, 1, 1, 1),
                                                       (128, 8, 8, 4, 0), (250, 9, 25, 7, 3)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_routing_a_long_batch_as_its_pieces(E, k, groups, topk_group, pad, dtype):
    """Large calls use larger blocks: tokens choose what they choose in small
    calls (which are checked against the oracle)."""
    T = 50003
    l = _logits(T, E, E + T, dtype, pad)
    mask = (torch.rand(T, device="cuda") > 0.1).to(torch.uint8)
    bias = torch.linspace(-0.05, 0.05, E, device="cuda")
    kw = dict(bias=bias, groups=groups, topk_group=topk_group, scale=1.5)
    _, _, idx, w = _route(l, k, mask=mask, **kw)
    for i in range(0, T, 2000):
        _, _, pi, pw = _route(l[i:i + 2000], k, mask=mask[i:i + 2000].clone(), **kw)
        assert torch.equal(idx[i:i + 2000], pi)
        assert torch.all((w[i:i + 2000] - pw).abs() <= 2 * W_RTOL * pw)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_routing_layouts_streams_and_graphs(dtype):
    """Rows at odd offsets and strides give what dense ones give; captured and
    replayed on new logits; two calls at once on two streams."""
    T, E, k = 333, 64, 6
    base = _logits(T, E + 9, 31, dtype)
    views = [base[:, 1:E + 1], base[:, 4:E + 4], base[:, 8:E + 8]]
    kw = dict(groups=8, topk_group=3, bias=0.1 * torch.rand(E, device="cuda"))
    for v in views:
        cfg, o, i0, w0 = _route(v, k, **kw)
        _, _, i1, w1 = _route(v.contiguous(), k, **kw)
        assert torch.equal(i0, i1) and torch.equal(w0, w1)
        dw = torch.randn(T, k, device="cuda")
        a = torch.zeros(T, E + 3, dtype=dtype, device="cuda")
        b = torch.empty(T, E, dtype=dtype, device="cuda")
        B.moe_route_groups_backward(cfg, o, v, i0, dw, a[:, 1:E + 1])
        B.moe_route_groups_backward(cfg, o, v.contiguous(), i0, dw, b)
        assert torch.equal(a[:, 1:E + 1], b) and torch.all(a[:, 0] == 0)
    l, idx, w = views[1].contiguous(), torch.empty_like(i0), torch.empty_like(w0)
    dl = torch.empty_like(l)
    B.moe_route_groups(cfg, o, l, kw["bias"], None, idx, w)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_route_groups(cfg, o, l, kw["bias"], None, idx, w)
        B.moe_route_groups_backward(cfg, o, l, idx, w, dl)
    for v in (views[0], views[2]):
        l.copy_(v)
        graph.replay()
        torch.cuda.synchronize()
        _, _, i1, w1 = _route(v, k, **kw)
        d1 = torch.empty_like(dl)
        B.moe_route_groups_backward(cfg, o, v, i1, w1, d1)
        assert torch.equal(idx, i1) and torch.equal(w, w1) and torch.equal(dl, d1)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    r1 = [_route(views[0], k, stream=s1, **kw) for _ in range(3)]
    r2 = [_route(views[2], k, stream=s2, **kw) for _ in range(3)]
    torch.cuda.synchronize()
    for r, v in ((r1, views[0]), (r2, views[2])):
        _, _, i1, w1 = _route(v, k, **kw)
        assert all(torch.equal(x[2], i1) and torch.equal(x[3], w1) for x in r)


# ----------------------------------------------------------------- gradient
@pytest.mark.parametrize("case", CASES, ids=str)
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_routing_gradient_matches_the_oracle(case, dtype):
    T, E, k, groups, tg, score, gate, space, norm = case
    l = _logits(T, E, 7 * T + E, dtype, pad=3)
    mask = torch.arange(T, device="cuda") % 5 != 4
    cfg, o, idx, w = _route(l, k, gate=gate, norm=norm, mask=mask, groups=groups, topk_group=tg,
                            score=score, space=space, scale=2.5)
    rng = np.random.default_rng(k)
    dw = rng.standard_normal((T, k)).astype(np.float32)
    dwt = torch.from_numpy(dw).cuda()
    dwt[idx < 0] = float("nan")           # not there: not read
    full = torch.full((T, E + 4), 7.0, dtype=dtype, device="cuda")
    B.moe_route_groups_backward(cfg, o, l, idx, dwt, full[:, :E])
    assert torch.all(full[:, E:] == 7.0)
    got = full[:, :E].double().cpu().numpy()
    ri = idx.cpu().numpy()
    l64 = l.double().cpu().numpy()
    ref = O.route_groups_backward(l64, ri, dw, gate, norm, 2.5)
    # per token: scores carry W_RTOL, and every term of the formula is at most
    # S = scale max|dw| / D times the largest chosen score (D = their sum when
    # renormalised, else 1); three such terms.  bf16 results: half a step.
    s = O.sigmoid(l64) if gate == SIG else O.softmax_rows(l64)
    sj = np.where(ri >= 0, np.take_along_axis(s, np.maximum(ri, 0), 1), 0.0)
    D = sj.sum(1) + 1e-9 if norm else np.ones(T)
    S = 2.5 * np.abs(dw).max(1) / D * sj.max(1)
    tol = 3 * W_RTOL * S[:, None] + (2.0 ** -8 * np.abs(ref) if dtype == torch.bfloat16 else 0)
    assert np.all(np.abs(got - ref) <= tol + 1e-30)
    assert np.all(got[ri[:, 0] < 0] == 0)


@pytest.mark.parametrize("gate", [SIG, SOFT])
def test_routing_gradient_of_one_renormalised_expert(gate):
    """top_k 1: w = s / (s + 1e-9), whose gradient is 1e-9 of its terms."""
    l = _logits(50, 40, 2)
    cfg, o, idx, _ = _route(l, 1, gate=gate)
    dw = torch.ones(50, 1, device="cuda")
    dl = torch.empty(50, 40, device="cuda")
    B.moe_route_groups_backward(cfg, o, l, idx, dw, dl)
    ref = O.route_groups_backward(l.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy(), gate,
                                  True)
    at = idx.long().cpu().numpy()
    got = np.take_along_axis(dl.double().cpu().numpy(), at, 1)
    # softmax: dl = p (ds - ds p), the difference rounded once against ds
    s = np.take_along_axis(O.softmax_rows(l.double().cpu().numpy()), at, 1)
    amp = 1.0 / (1.0 - s) if gate == SOFT else 1.0
    want = np.take_along_axis(ref, at, 1)
    assert np.all(np.abs(got - want) <= 4 * W_RTOL * amp * np.abs(want))


def test_routing_gradient_of_foreign_pairs():
    """Ids outside [0, E) are no pairs; an id listed twice counts twice."""
    l = _logits(4, 20, 9)
    idx = torch.tensor([[3, 3, 5], [-1, 20, 7], [-1, -1, -1], [2 ** 30, -2 ** 31, 0]],
                       dtype=torch.int32, device="cuda")
    dw = torch.tensor([[1.0, 2.0, -1.0], [INF, INF, 1.0], [1.0, 1.0, 1.0], [1.0, 1.0, 0.5]],
                      device="cuda")
    for gate in (SIG, SOFT):
        for norm in (True, False):
            cfg = B.make_config(4, 128, 20, 128, 3, gate=gate, norm_topk_prob=int(norm))
            dl = torch.empty(4, 20, device="cuda")
            B.moe_route_groups_backward(cfg, B.make_group_opts(), l, idx, dw, dl)
            ref = O.route_groups_backward(l.cpu().numpy(), idx.cpu().numpy(), dw.cpu().numpy(),
                                          gate, norm)
            assert np.all(np.abs(dl.double().cpu().numpy() - ref) <= 3 * W_RTOL * 4)
            assert torch.all(dl[2] == 0)


# --------------------------------------------------------- orthogonalisation
# fp32 results: operands carry 2^-22, sums are rounded at 2^-24 over chunks;
# each step adds about 1e-6 of X and multiplies what is there by at most
# |p'| on the small directions (where the relative error stays) and below 1.5 on
# the others: 1e-5 over up to six steps.  bf16 results: operands at 2^-12, 3e-4
# of X a step (X, A, B once each) and the same growth, 3e-3; and the rounding,
# 2^-9 of the largest elements, 1.7e-3 rms.
O_TOL = {torch.float32: 1e-5, torch.bfloat16: 5e-3}
DT = {torch.float32: B.DTYPE_F32, torch.bfloat16: B.DTYPE_BF16}


def _ortho(g, out_dtype, out=None, steps=5, coeffs=B.MUON_COEFFS, eps=1e-7, scale=1.0,
           stream=None):
    b, r, c = g.shape
    cfg = B.make_ortho_config(b, r, c, DT[g.dtype], DT[out_dtype], steps, coeffs, eps, scale)
    ws = torch.empty(max(256, B.moe_orthogonalize_workspace_size(cfg)), dtype=torch.uint8,
                     device="cuda")
    out = torch.empty((b, r, c), dtype=out_dtype, device="cuda") if out is None else out
    B.moe_orthogonalize(cfg, g, out, ws, stream=stream)
    return out, ws


def _ortho_err(out, g, **kw):
    ref = O.orthogonalize(g.double().cpu().numpy(), **kw)
    got = out.double().cpu().numpy()
    return max(np.linalg.norm(a - b) / max(np.linalg.norm(b), 1e-300) for a, b in zip(got, ref))


SHAPES = [(1, 1, 1), (2, 1, 7), (2, 7, 1), (1, 16, 64), (3, 63, 65), (2, 64, 64), (1, 128, 128),
          (2, 129, 127), (1, 128, 1000), (2, 130, 258), (1, 256, 256), (3, 333, 517),
          (2, 517, 333), (1, 1000, 24), (5, 96, 96), (1, 520, 777), (70, 40, 56)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("din", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
def test_orthogonalize_matches_the_oracle(shape, din, dout):
    rng = np.random.default_rng(sum(shape))
    g = torch.from_numpy((1e-3 * rng.standard_normal(shape)).astype(np.float32)).cuda().to(din)
    out, ws = _ortho(g, dout)
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)
    assert _ortho_err(out, g) <= O_TOL[dout]


def _ref64(g, steps=5, coeffs=B.MUON_COEFFS, eps=1e-7):
    """The oracle's iteration in torch on the GPU, 64 bits, for larger batches."""
    a, b, c = (float(np.float32(v)) for v in coeffs)
    x = g.double()
    tall = x.shape[1] > x.shape[2]
    x = x.transpose(1, 2) if tall else x
    x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + float(np.float32(eps)))
    for _ in range(steps):
        A = x @ x.transpose(1, 2)
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.transpose(1, 2) if tall else x


# every tile shape of every product, with and without mirrored tiles, ragged at
# their edges; rows below 64 that do not fit one launch; widths from one to
# sixteen CTAs of the one-launch kernel, four boxes a CTA, and both orders;
# products split over two and four CTAs
BATCHES = [(20, 400, 400), (9, 510, 510), (64, 250, 287), (64, 250, 250), (3, 900, 900),
           (40, 400, 805), (20, 700, 700), (9, 330, 331), (40, 130, 130), (6, 805, 400),
           (2, 40, 2500), (2, 2500, 40), (1, 128, 2048), (1, 1100, 100), (3, 100, 1500),
           (150, 100, 250), (40, 70, 600), (5, 128, 129), (2, 129, 128), (1, 3, 2048),
           (1, 512, 2048), (2, 256, 1024), (1, 130, 3000), (2, 3000, 140), (1, 513, 515),
           (40, 70, 500), (33, 260, 90), (4, 66, 400), (13, 1000, 90), (12, 90, 1000),
           (13, 1025, 65), (70, 64, 256), (3, 100, 2000), (1, 120, 4096), (2, 4000, 66),
           (3, 40, 2500), (1, 128, 4100)]


@pytest.mark.parametrize("shape", BATCHES, ids=str)
@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
def test_orthogonalize_batches(shape, dout):
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    g = torch.randn(*shape, generator=gen, device="cuda")
    out, ws = _ortho(g, dout)
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)
    ref = _ref64(g)
    err = torch.linalg.vector_norm(out.double() - ref, dim=(1, 2)) / \
        torch.linalg.vector_norm(ref, dim=(1, 2))
    assert err.max().item() <= O_TOL[dout]
    again, _ = _ortho(g, dout)
    assert torch.equal(out, again)
    # a matrix alone gives what it gives in the batch, to the same bound
    if shape[0] > 1:
        one, _ = _ortho(g[-1:], dout)
        assert _ortho_err(one, g[-1:]) <= O_TOL[dout]


@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("steps,coeffs,scale", [(1, B.MUON_COEFFS, 0.2), (2, B.MUON_COEFFS, 1.0),
                                                (6, B.MUON_COEFFS, -3.0),
                                                (8, (2.0, -1.5, 0.5), 1.0),
                                                (3, (1.5, -0.5, 0.0), 1.0)])
def test_orthogonalize_steps_and_coefficients(dout, steps, coeffs, scale):
    rng = np.random.default_rng(steps)
    g = torch.from_numpy(rng.standard_normal((2, 140, 200)).astype(np.float32)).cuda()
    out, _ = _ortho(g, dout, steps=steps, coeffs=coeffs, scale=scale)
    assert _ortho_err(out, g, steps=steps, coeffs=coeffs, scale=scale) <= O_TOL[dout]


@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("rows,cols", [(200, 300), (100, 180), (600, 66)])
def test_orthogonalize_low_rank(dout, rows, cols):
    """Few strong directions over noise 1e-4 of them, which grows by 3.44 a
    step: bf16 results keep the iterate to 22 bits for this."""
    rng = np.random.default_rng(3)
    a = rng.standard_normal((2, rows, 12)) @ rng.standard_normal((2, 12, cols))
    g = torch.from_numpy((a + 1e-4 * rng.standard_normal(a.shape)).astype(np.float32)).cuda()
    out, _ = _ortho(g, dout)
    # fp32: the noise directions are 1e-4 of the operands' 2^-22, so 1e-3 of
    # themselves would be 2.4e-7 / 1e-4; they are a part of the result only
    assert _ortho_err(out, g) <= (1e-4 if dout == torch.float32 else 5e-3)


@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", [(6, 48, 80), (6, 300, 280)], ids=str)
def test_orthogonalize_special_matrices(dout, shape):
    """Zeros give zeros; very large and very small gradients are normalised;
    a NaN or an infinity stays in its matrix."""
    rng = np.random.default_rng(11)
    g = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda()
    g[0] = 0
    g[1] *= 1e30
    g[2] *= 1e-30
    g[3, 5, 7] = float("nan")
    g[4, 5, 7] = INF
    out, ws = _ortho(g, dout, eps=1e-30)
    assert torch.all(out[0] == 0)
    for i in (1, 2, 5):
        # 1e-30 times N(0, 1): the norm is far above eps = 1e-30, which is
        # still 1e-2 of it and part of the definition
        assert _ortho_err(out[i:i + 1], g[i:i + 1], eps=1e-30) <= O_TOL[dout]
    for i in (3, 4):
        assert torch.isnan(out[i]).any() and not torch.isfinite(out[i]).all()
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)


@pytest.mark.parametrize("shape", [(3, 50, 70), (3, 290, 100), (2, 100, 290)], ids=str)
def test_orthogonalize_strides_and_in_place(shape):
    b, r, c = shape
    rng = np.random.default_rng(17)
    big = torch.from_numpy(rng.standard_normal((b, r + 3, c + 5)).astype(np.float32)).cuda()
    g = big[:, 1:r + 1, 2:c + 2]                       # odd offset, strided rows
    for dout in (torch.float32, torch.bfloat16):
        dst = torch.full((b + 1, r + 2, c + 1), 9.0, dtype=dout, device="cuda")
        out, _ = _ortho(g, dout, out=dst[:b, 1:r + 1, 1:])
        assert _ortho_err(out, g) <= O_TOL[dout]
        assert torch.all(dst[b] == 9) and torch.all(dst[:, 0] == 9) and \
            torch.all(dst[:, :, 0] == 9) and torch.all(dst[:, r + 1] == 9)
        dense, _ = _ortho(g.contiguous(), dout)
        assert torch.equal(dense, out)                 # and the layout changes nothing
    keep = g.clone()
    _ortho(g, torch.float32, out=g)
    assert _ortho_err(g, keep) <= O_TOL[torch.float32]


def test_orthogonalize_graph_streams_and_repeats():
    """Captured and replayed on new data; two calls at once on two streams with
    their own workspaces; bit for bit the same each time."""
    rng = np.random.default_rng(29)
    a = torch.from_numpy(rng.standard_normal((4, 200, 330)).astype(np.float32)).cuda()
    b = torch.from_numpy(rng.standard_normal((1, 700, 256)).astype(np.float32)).cuda()
    ra, _ = _ortho(a, torch.float32)
    rb, _ = _ortho(b, torch.bfloat16)
    cfg = B.make_ortho_config(4, 200, 330, B.DTYPE_F32, B.DTYPE_F32)
    ws = torch.empty(B.moe_orthogonalize_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    x, out = torch.zeros_like(a), torch.empty_like(a)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        B.moe_orthogonalize(cfg, x, out, ws)
    for src in (a, -a, a):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, ra if src is a else -ra)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = []
    for _ in range(5):
        oa, ob = torch.empty_like(ra), torch.empty_like(rb)
        torch.cuda.synchronize()
        w1 = _ortho(a, torch.float32, out=oa, stream=s1)
        w2 = _ortho(b, torch.bfloat16, out=ob, stream=s2)
        outs.append((oa, ob, w1, w2))
        torch.cuda.synchronize()
    for oa, ob, _, _ in outs:
        assert torch.equal(oa, ra) and torch.equal(ob, rb)


# -------------------------------------------------------------- the layer
LAYERS = {
    "sigmoid_shared": (I.WORKLOADS["skew"].replace(T=500, d_model=256, d_ff=256,
                                                   d_ff_shared=128), 8, 3, 2, 1, 2.5),
    "softmax": (I.WORKLOADS["qwen3_30b"].replace(T=300, d_model=256, d_ff=128), 16, 4, 1, 1, 1.0),
    "logit_space": (I.WORKLOADS["page2"].replace(T=130, d_model=128, d_ff=128, d_ff_shared=128),
                    4, 2, 2, 0, 1.0),
}


def _layer(name):
    shape, g, tg, score, space, scale = LAYERS[name]
    host = I.make_inputs(shape)
    rng = np.random.default_rng(shape.T)
    host["sel_bias"] = (0.1 * rng.uniform(-1, 1, shape.n_experts)).astype(np.float32)
    layer = MoELayer(shape, host, groups=B.make_group_opts(g, tg, score, space, scale))
    return shape, host, layer, (g, tg, score, space, scale)


@pytest.mark.parametrize("name", list(LAYERS))
@pytest.mark.parametrize("padded", [False, True])
def test_layer_step_with_groups(name, padded):
    """Forward, backward and the update directions of one layer, as a training
    step uses them, against the oracle."""
    shape, host, layer, (g, tg, score, space, scale) = _layer(name)
    T, E, k = shape.T, shape.n_experts, shape.top_k
    mask = None
    if padded:
        mask = torch.arange(T, device="cuda") % 7 < 5
        mask[-40:] = False
    layer.ws.fill_(0xff)                 # NaN wherever nothing is written
    layer.forward(token_mask=mask)
    assert layer.device_status() == (B.MOE_OK, 0)
    logits = torch.empty(T, E, device="cuda")
    ws2 = torch.empty_like(layer.ws)
    B.moe_router_logits(layer.cfg, layer.x, layer.w_router, layer.logit_offset, logits, ws2)
    ri, rw, s = O.route_groups(logits.cpu().numpy(), k, shape.gate, bool(shape.norm_topk_prob),
                               host["sel_bias"], g, tg, score, space, scale,
                               None if mask is None else mask.cpu().numpy())
    idx = layer.topk_idx.cpu().numpy()
    np.testing.assert_array_equal(idx, ri)
    np.testing.assert_allclose(layer.topk_w.cpu().numpy(), rw, rtol=W_RTOL)
    np.testing.assert_array_equal(layer.counts.cpu().numpy(),
                                  np.bincount(ri[ri >= 0], minlength=E))
    r = O.Routing(logits.double().cpu().numpy(), s, s, ri, rw, None, None)
    ref, _ = O.moe_forward(host, k, shape.gate, True, routing=r)
    out = layer.out.float().cpu().numpy()
    assert P.rel_err(out, ref) <= P.OUT_TOL_BF16
    if padded and not shape.n_shared:
        assert np.all(out[~mask.cpu().numpy()] == 0)
    # backward, twice: rows behind the routed ones hold what the first left
    dout_h = I.round_to_bf16(np.random.default_rng(5).standard_normal(
        (T, shape.d_model)).astype(np.float32))
    dout = to_device(dout_h, torch.bfloat16, "cuda")
    grads = layer.backward(dout)
    assert B.moe_device_status(layer.bws) == (B.MOE_OK, 0)
    gr = O.moe_backward(host, k, shape.gate, bool(shape.norm_topk_prob), dout_h, routing=r)
    dl = O.route_groups_backward(logits.double().cpu().numpy(), ri, gr["dtopk_w"], shape.gate,
                                 bool(shape.norm_topk_prob), scale)
    wr = host["w_router"].astype(np.float64)
    gr["dx"] = gr["dx"] - gr["dlogits"] @ wr + dl @ wr
    gr["dw_router"] = dl.T @ host["x"].astype(np.float64)
    keys = ["dx", "dw_router", "dw1", "dw3", "dw2"]
    keys += ["dws1", "dws3", "dws2"] if shape.n_shared else []
    for key in keys:
        err = P.rel_err(grads[key].float().cpu().numpy(), gr[key])
        assert err <= 3e-2, f"{key}: relative error {err:.3e}"    # the layer's gradient bar
    again = layer.backward(dout)
    for key in keys:
        assert torch.equal(grads[key], again[key]), key
    # update directions of the very gradients, experts without tokens included
    upd = layer.orthogonalize(grads)
    assert set(upd) == {key for key in keys if key != "dx"}
    for key, u in upd.items():
        gg = grads[key] if grads[key].dim() == 3 else grads[key][None]
        uu = u if u.dim() == 3 else u[None]
        assert u.dtype == grads[key].dtype
        pick = range(min(4, gg.shape[0]))
        for i in pick:
            n = torch.linalg.vector_norm(gg[i].double()).item()
            if n == 0:
                assert torch.all(uu[i] == 0)
            else:
                assert _ortho_err(uu[i:i + 1], gg[i:i + 1]) <= 2 * O_TOL[u.dtype]


def test_layer_update_keeps_what_a_graph_uses():
    """A captured update goes on with its workspace after a larger one."""
    layer = _layer("softmax")[2]
    gen = torch.Generator(device="cuda").manual_seed(1)
    small = {"dw_router": torch.randn(140, 200, generator=gen, device="cuda")}
    large = {"dw1": torch.randn(20, 300, 320, generator=gen, device="cuda")}
    want = layer.orthogonalize(small)["dw_router"].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.orthogonalize(small)["dw_router"]
    n = layer.ows[-1].numel()
    layer.orthogonalize(large)
    assert layer.ows[-1].numel() > n
    fill = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
    got.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(bool((f == 255).all()) for f in fill)


def test_layer_with_groups_fp32():
    shape = I.WORKLOADS["tiny"]
    host = I.make_inputs(shape)
    layer = MoELayer(shape, host, groups=B.make_group_opts(2, 1, 2, 1, 1.5))
    mask = torch.ones(shape.T, dtype=torch.uint8, device="cuda")
    mask[::9] = 0
    layer.forward(token_mask=mask)
    r = P.oracle_routing(shape, host)
    ri, rw, s = O.route_groups(r.logits, shape.top_k, shape.gate, True, None, 2, 1, 2, 1, 1.5,
                               mask.cpu().numpy())
    np.testing.assert_array_equal(layer.topk_idx.cpu().numpy(), ri)
    ref, _ = O.moe_forward(host, shape.top_k, shape.gate, True,
                           routing=O.Routing(r.logits, s, s, ri, rw, None, None))
    assert P.rel_err(layer.out.cpu().numpy(), ref) <= P.OUT_TOL_F32
    assert layer.device_status() == (B.MOE_OK, 0)


def test_layer_with_one_group_selects_as_the_router():
    """groups of all experts and scale 1: the experts moe_forward picks, but
    where two keys are as close as the logits' fp32 error."""
    shape = I.WORKLOADS["skew"].replace(T=700, d_model=256, d_ff=128, d_ff_shared=128)
    host = I.make_inputs(shape)
    a = MoELayer(shape, host)
    b = MoELayer(shape, host, groups=B.make_group_opts(1, 1, 1, 0, 1.0))
    a.forward()
    b.forward()
    r = P.oracle_routing(shape, host)
    clear = r.min_gap > 1e-4
    assert clear.mean() > 0.9
    np.testing.assert_array_equal(a.topk_idx.cpu().numpy()[clear],
                                  b.topk_idx.cpu().numpy()[clear])
    with pytest.raises(B.MoEError):
        b.forward(gather_rows=True)
    with pytest.raises(B.MoEError):
        a.forward(token_mask=torch.ones(shape.T, dtype=torch.uint8, device="cuda"))


def test_dispatch_reports_missing_experts_outside_the_layer_call():
    """moe_permute on its own still reports id -1, as any id outside [0, E)."""
    cfg = B.make_config(4, 128, 8, 128, 2)
    idx = torch.tensor([[0, 1], [-1, 2], [3, 4], [5, 6]], dtype=torch.int32, device="cuda")
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = torch.empty(B.moe_workspace_size(cfg), dtype=torch.uint8, device="cuda")
    B.moe_permute(cfg, idx, x, torch.empty(8, **i32), torch.empty(9, **i32),
                  torch.empty(4, 2, **i32), torch.empty(8, **i32),
                  torch.empty(8, 128, dtype=torch.bfloat16, device="cuda"), ws)
    assert B.moe_device_status(ws)[0] == B.MOE_ERR_DATA


def test_binding_refuses_tensors_it_cannot_pass_on():
    """Other types, too small, not dense, or on the host: refused before a launch."""
    l = _logits(8, 16, 1)
    cfg, o = B.make_config(8, 128, 16, 128, 2), B.make_group_opts(4, 2)
    idx = torch.full((8, 2), -7, dtype=torch.int32, device="cuda")
    w = torch.full((8, 2), -7.0, device="cuda")
    dl = torch.full((8, 16), -7.0, device="cuda")
    bias, mask = torch.zeros(16, device="cuda"), torch.ones(8, device="cuda")
    bad = [(l.double(), None, None, idx, w), (l.cpu(), None, None, idx, w),
           (l, None, None, idx.long(), w), (l, None, None, idx.cpu(), w),
           (l, None, None, idx[:4], w), (l, None, None, idx, w.t()),
           (l, bias[:8], None, idx, w), (l, bias.double(), None, idx, w), (l, None, mask, idx, w)]
    for args in bad:
        with pytest.raises(B.MoEError):
            B.moe_route_groups(cfg, o, *args)
    for args in [(l, idx.long(), w, dl), (l, idx, w.cpu(), dl), (l, idx, w, dl.half()),
                 (l, idx, w[:1], dl), (l.cpu(), idx, w, dl)]:
        with pytest.raises(B.MoEError):
            B.moe_route_groups_backward(cfg, o, *args)
    oc = B.make_ortho_config(1, 8, 16, B.DTYPE_F32, B.DTYPE_F32)
    ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
    for g, out in [(l.half(), dl), (l, dl.half()), (l.cpu(), dl), (l, dl.cpu())]:
        with pytest.raises(B.MoEError):
            B.moe_orthogonalize(oc, g, out, ws)
    torch.cuda.synchronize()
    assert torch.all(idx == -7) and torch.all(w == -7.0) and torch.all(dl == -7.0)


def test_orthogonalize_refuses_a_workspace_on_the_host():
    g = torch.randn(1, 200, 200, device="cuda")
    out = torch.full_like(g, -7.0)
    oc = B.make_ortho_config(1, 200, 200, B.DTYPE_F32, B.DTYPE_F32)
    ws = torch.empty(B.moe_orthogonalize_workspace_size(oc) + 256, dtype=torch.uint8)
    with pytest.raises(B.MoEError):
        B.moe_orthogonalize(oc, g, out, ws[(-ws.data_ptr()) % 256:])
    torch.cuda.synchronize()
    assert torch.all(out == -7.0)


def _equal_values(rank, rows, cols, seed):
    """A matrix of `rank` equal singular values with random singular vectors."""
    g = torch.Generator().manual_seed(seed)
    u = torch.linalg.qr(torch.randn(rows, rank, generator=g, dtype=torch.float64))[0]
    v = torch.linalg.qr(torch.randn(cols, rank, generator=g, dtype=torch.float64))[0]
    return (u @ v.T)[None].float().cuda()


@pytest.mark.parametrize("rows,cols", [(333, 517), (517, 333), (700, 900), (100, 300), (96, 96),
                                       (128, 2500)])
@pytest.mark.parametrize("steps,coeffs,grow", [
    (6, B.MUON_COEFFS, 150), (9, B.MUON_COEFFS, 520), (5, (3.7418, -5.5913, 2.3037), 480)])
def test_orthogonalize_bf16_of_many_steps(rows, cols, steps, coeffs, grow):
    """More steps than products of one term bear ([333, 517] so: 4.6e-3 and 1.3e-2
    at 6 and 9 steps).  grow: the relative error's largest growth over the steps
    (1 x 1 matrices, simulated); 22-bit operands and fp32 sums leave about 1e-6 of
    the iterate a step, and the result is rounded by at most 2^-8."""
    g = _equal_values(min(rows, cols), rows, cols, rows + cols)
    out, ws = _ortho(g, torch.bfloat16, steps=steps, coeffs=coeffs)
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)
    assert _ortho_err(out, g, steps=steps, coeffs=coeffs) <= 2.0 ** -8 + 1e-6 * grow


@pytest.mark.parametrize("rows,cols", [(64, 96), (333, 517)])
def test_orthogonalize_roundings_that_coincide(rows, cols):
    """A scaled identity of rank 43, whose elements all round alike: products of
    one term stay within the bound that admits them, 100 2^-12, and 22 bits
    within as many of theirs."""
    g = torch.zeros(1, rows, cols, device="cuda")
    i = torch.arange(43, device="cuda")
    g[0, i, i] = 0.37
    out, _ = _ortho(g, torch.bfloat16)
    assert _ortho_err(out, g) <= 100 * 2.0 ** -12 + 2.0 ** -8
    out, _ = _ortho(g, torch.float32)
    assert _ortho_err(out, g) <= 100 * 2.0 ** -22 + 5 * 1e-6


@pytest.mark.parametrize("gate", [SIG, SOFT])
@pytest.mark.parametrize("space", [0, 1])
@pytest.mark.parametrize("score", [1, 2])
@pytest.mark.parametrize("per", [8, 5])
def test_routing_biases_beyond_fp32_sums(gate, space, score, per):
    """Experts forced on by +inf or by 3e38, switched off by -3e38 or the lowest
    value: keys, and sums of two, that leave fp32's range on either side."""
    G, T, k = 8, 17, 6
    E = G * per
    rng = np.random.default_rng(10 * per + score)
    low, high = np.finfo(np.float32).min, np.finfo(np.float32).max
    a = rng.standard_normal((T, E)).astype(np.float32)
    a[3, ::2] = low
    a[4, :per] = -np.inf
    a[5] = low
    a[6] = -np.inf
    a[7, 1::2] = -np.inf
    plain = (0.1 * rng.standard_normal(E)).astype(np.float32)
    biases = []
    for value in (np.inf, high, 3e38, 2e38, -2e38, -3e38, low):
        for which in ([1], [1, 2], [0, per + 1, 2 * per], range(3, E, per), range(0, E, 2),
                      range(per, 3 * per), range(E - 3, E), range(E)):
            b = plain.copy()
            b[list(which)] = value
            biases.append(b)
    b = plain.copy()                       # both sides in one group
    b[0], b[1], b[per], b[per + 1] = 3e38, low, -1e38, 0.0
    biases.append(b)
    b = plain.copy()
    b[::3], b[1::3] = np.inf, -np.inf
    biases.append(b)
    b = np.full(E, low)                    # groups of the lowest beside empty ones
    b[:per], b[2 * per:3 * per] = -np.inf, -np.inf
    biases.append(b)
    l = torch.from_numpy(a).cuda()
    for b in biases:
        for tg in (1, 3):
            _check_nan(l, k, gate, space, torch.from_numpy(b).cuda(), tg, score)


def test_routing_forced_expert_beside_a_close_call():
    """An expert forced on by +inf keeps its group where two others are close."""
    T, per, G = 64, 8, 4
    rng = np.random.default_rng(3)
    a = (0.01 * rng.standard_normal((T, per * G)) - 1.0).astype(np.float32)
    a[:, 2 * per] = 0.5
    a[:, 3 * per] = np.nextafter(np.float32(0.5), np.float32(1))
    b = np.zeros(per * G, np.float32)
    b[1] = np.inf
    b[2 * per] = 3e-8
    for gate in (SIG, SOFT):
        for score in (1, 2):
            for space in (0, 1):
                out = _route(torch.from_numpy(a).cuda(), 4, gate=gate, space=space, groups=G,
                             topk_group=2, score=score, bias=torch.from_numpy(b).cuda())
                ri, rw, _ = O.route_groups(a, 4, gate, True, b, G, 2, score, space)
                assert np.all(ri[:, 0] == 1)
                np.testing.assert_array_equal(out[2].cpu().numpy(), ri)
                assert np.all(np.abs(out[3].double().cpu().numpy() - rw) <= W_RTOL * rw)


@pytest.mark.parametrize("E", [61, 62, 63, 64])
def test_routing_ties_at_inf_at_the_end_of_a_row(E):
    """The k-th and further keys +inf, rows and bias that end with the last
    expert of a buffer: ties go to the lower ids."""
    T, k = 5, 4
    l = torch.zeros(T * E, device="cuda").view(T, E)
    bias = torch.full((E,), INF, device="cuda")
    for gate in (SIG, SOFT):
        for space in (0, 1):
            _, _, idx, w = _route(l, k, gate=gate, space=space, bias=bias)
            assert torch.equal(idx.cpu(), torch.arange(k, dtype=torch.int32).expand(T, k))
            assert torch.all((w - 0.25).abs() <= W_RTOL * 0.25)


def test_routing_groups_of_subnormal_scores():
    """Unbiased softmax scores that are fp32 subnormals, or zero there: their groups
    rank as the fp64 sums do."""
    per, G, T = 4, 6, 400
    rng = np.random.default_rng(44)
    a = (-100.0 + 6.0 * rng.uniform(-1, 1, (T, per * G)) * rng.uniform(0.01, 1, (T, 1)))
    a[:, 0] = 0.0                        # the first group holds all the weight
    a[:, 1:4] = -300.0
    a[0] = [0, -300, -300, -300] + [-101.56, -101.76, -300, -300] + \
        [-101.64, -101.64, -300, -300] + [-300] * 12
    a[1] = [0, -300, -300, -300] + [-101.64, -101.64, -300, -300] + \
        [-101.56, -101.76, -300, -300] + [-300] * 12
    l = torch.from_numpy(a.astype(np.float32)).cuda()
    for tg in (2, 4):
        out = _route(l, 6, gate=SOFT, groups=G, topk_group=tg, score=2)
        ri, _, _ = O.route_groups(l.double().cpu().numpy(), 6, SOFT, True, None, G, tg, 2, 1)
        np.testing.assert_array_equal(out[2].cpu().numpy(), ri)


# clusters of 4, 8, 16, 16, 8 and 8 CTAs, 1, 3, 7, 7, 3 and 1 of them without a column
IDLE_CTAS = [(1, 100, 320), (2, 90, 576), (1, 128, 1088), (2, 1100, 128), (12, 580, 100),
             (3, 100, 800)]


@pytest.mark.parametrize("shape", IDLE_CTAS, ids=str)
@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
def test_orthogonalize_clusters_with_idle_ctas(shape, dout):
    """CTAs without columns reach the exchange of the norm long before, or after,
    the others: the sums are whole, call after call."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    g = torch.randn(*shape, generator=gen, device="cuda")
    ref = _ref64(g)
    first = None
    for _ in range(30):
        out, ws = _ortho(g, dout)
        assert B.moe_device_status(ws) == (B.MOE_OK, 0)
        first = out if first is None else first
        assert torch.equal(out, first)
    err = torch.linalg.vector_norm(first.double() - ref, dim=(1, 2)) / \
        torch.linalg.vector_norm(ref, dim=(1, 2))
    assert err.max().item() <= O_TOL[dout]


@pytest.mark.parametrize("shape", [(6, 48, 80), (6, 300, 280), (6, 100, 600), (6, 70, 90),
                                   (6, 1200, 100), (6, 1, 40), (6, 200, 1200)], ids=str)
@pytest.mark.parametrize("din", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dout", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("steps", [1, 5])
def test_orthogonalize_spreads_what_is_not_finite(shape, din, dout, steps):
    """A matrix with a NaN or an infinity gives NaN everywhere, also where its parts
    lie on several CTAs; the others, and zeros, are what they are alone."""
    rng = np.random.default_rng(sum(shape))
    g = torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).cuda().to(din)
    r, c = shape[1] - 1, shape[2] // 3
    clean = g.clone()
    g[0, r, c], g[1, 0, -1], g[2, r, c] = float("nan"), INF, -INF
    g[3] = 0
    out, ws = _ortho(g, dout, steps=steps)
    want, _ = _ortho(clean, dout, steps=steps)
    assert torch.isnan(out[:3]).all()
    assert torch.all(out[3] == 0)
    assert torch.equal(out[4:], want[4:])
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)


def test_layer_update_on_another_stream():
    """Results and workspace are not in memory that the current stream's queued
    work still uses; streams by object and by address."""
    layer = _layer("softmax")[2]
    gen = torch.Generator(device="cuda").manual_seed(2)
    grads = {"dw1": torch.randn(20, 300, 320, generator=gen, device="cuda"),
             "dw_router": torch.randn(140, 200, generator=gen, device="cuda")}
    want = {k: u.clone() for k, u in layer.orthogonalize(grads).items()}
    n = layer.ows[-1].numel()
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, None):
        layer.ows.clear()
        torch.cuda.synchronize()
        gone = [torch.empty_like(g) for g in grads.values()]
        gone.append(torch.empty(n, dtype=torch.uint8, device="cuda"))
        torch.cuda._sleep(20_000_000)           # 10 ms of the current stream's time
        for t in gone:
            t.fill_(7)
        del t, gone                             # freed on the host, written later
        got = layer.orthogonalize(grads, stream=stream)
        torch.cuda.synchronize()
        for k in grads:
            assert torch.equal(got[k], want[k]), k


@pytest.mark.parametrize("name", list(LAYERS))
@pytest.mark.parametrize("T,on", [(1, 1), (1, 0), (70, 0), (70, 1)])
def test_layer_step_of_few_or_no_routed_tokens(name, T, on):
    """`on` of T tokens are no padding: experts, and all of them, without rows."""
    shape, g, tg, score, space, scale = LAYERS[name]
    shape = shape.replace(T=T)
    host = I.make_inputs(shape)
    layer = MoELayer(shape, host, groups=B.make_group_opts(g, tg, score, space, scale))
    mask = torch.zeros(T, dtype=torch.uint8, device="cuda")
    mask[T - on:] = 1
    layer.ws.fill_(0xff)
    layer.forward(token_mask=mask)
    assert layer.device_status() == (B.MOE_OK, 0)
    idx, w = layer.topk_idx.cpu().numpy(), layer.topk_w.double().cpu().numpy()
    assert np.all(idx[:T - on] == -1) and np.all(w[:T - on] == 0) and np.all(idx[T - on:] >= 0)
    assert layer.counts.sum().item() == on * shape.top_k
    logits = host["x"].astype(np.float64) @ host["w_router"].astype(np.float64).T
    if host.get("logit_offset") is not None:
        logits = logits + host["logit_offset"]
    s = O.sigmoid(logits) if shape.gate == O.GATE_SIGMOID else O.softmax_rows(logits)
    r = O.Routing(logits, s, s, idx.astype(np.int64), w, None, None)
    ref, _ = O.moe_forward(host, shape.top_k, shape.gate, True, routing=r)
    out = layer.out.double().cpu().numpy()
    assert np.all(np.isfinite(out))
    if on or shape.n_shared:
        assert P.rel_err(out, ref) <= P.OUT_TOL_BF16
    else:
        assert np.all(out == 0)
    dout_h = I.round_to_bf16(np.random.default_rng(6).standard_normal(
        (T, shape.d_model)).astype(np.float32))
    grads = layer.backward(to_device(dout_h, torch.bfloat16, "cuda"))
    assert B.moe_device_status(layer.bws) == (B.MOE_OK, 0)
    assert all(torch.isfinite(v).all() for v in grads.values())
    used = torch.from_numpy(np.isin(np.arange(shape.n_experts), idx)).cuda()
    for key in ("dw1", "dw3", "dw2"):
        assert torch.all(grads[key][~used] == 0)
    if not on:
        assert torch.all(grads["dw_router"] == 0)
    if on:
        gr = O.moe_backward(host, shape.top_k, shape.gate, bool(shape.norm_topk_prob), dout_h,
                            routing=r)
        for key in ("dw1", "dw3", "dw2"):
            assert P.rel_err(grads[key].float().cpu().numpy(), gr[key]) <= 3e-2, key
    upd = layer.orthogonalize(grads)
    assert all(torch.isfinite(u).all() for u in upd.values())


def test_layer_update_of_no_experts():
    """An empty stack of gradients among others."""
    layer = _layer("softmax")[2]
    g = {"dw1": torch.empty(0, 300, 320, device="cuda"), "dw_router": torch.eye(40, device="cuda")}
    out = layer.orthogonalize(g)
    assert out["dw1"].shape == (0, 300, 320)
    assert _ortho_err(out["dw_router"][None], g["dw_router"][None]) <= 100 * 2.0 ** -22 + 5e-6


@pytest.mark.parametrize("shape", [(20, 700, 700), (40, 400, 805), (6, 805, 400), (64, 250, 287),
                                   (24, 768, 2048), (1, 512, 2048), (2, 3000, 140),
                                   (150, 100, 250), (12, 90, 1000), (1, 120, 4096)], ids=str)
def test_orthogonalize_bf16_of_six_steps_in_batches(shape):
    """bf16 results of three-term products on every tile shape and cluster width:
    the fp32 results' error (1e-4 at six steps) and the rounding, 2^-8 at most."""
    gen = torch.Generator(device="cuda").manual_seed(sum(shape))
    g = torch.randn(*shape, generator=gen, device="cuda").to(torch.bfloat16)
    out, ws = _ortho(g, torch.bfloat16, steps=6)
    assert B.moe_device_status(ws) == (B.MOE_OK, 0)
    ref = _ref64(g, steps=6)
    err = torch.linalg.vector_norm(out.double() - ref, dim=(1, 2)) / \
        torch.linalg.vector_norm(ref, dim=(1, 2))
    assert err.max().item() <= 2.0 ** -8 + 1e-4
    # and they are the fp32 results, rounded
    full, _ = _ortho(g, torch.float32, steps=6)
    assert torch.equal(out, full.to(torch.bfloat16))
