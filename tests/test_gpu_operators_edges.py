"""The handle-free operators where fp32 alone would decide wrongly: accuracy of the
gated unit and its gradient, experts and groups whose keys saturate, cancel or
nearly tie, blocks of tiny values.

U = 2^-24 is half a step of fp32 relative to the value; an approximate power of 2 is
within 4 U, an approximate reciprocal within 2 U, tanhf within 2 ulp (4 U), a sum,
division or product within U.
"""
from decimal import Decimal, localcontext

import numpy as np
import pytest

import operators_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def torch():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    return torch


@pytest.fixture(scope="module")
def moe():
    import deterministic_expert_b200
    return deterministic_expert_b200


# ------------------------------------------------------------- gated unit
def _one_a_block(torch, values, width):
    """bf16 rows [values, width], each block of 128 zero but for its first element."""
    x = torch.zeros(len(values), width, dtype=torch.bfloat16)
    x[:, ::128] = torch.tensor(values, dtype=torch.float32).to(torch.bfloat16)[:, None]
    return x.cuda()


def _values(scales):
    """The magnitude of a block's only element: its scale is that / 448, rounded once."""
    return scales.cpu().numpy().astype(np.float64) * 448.0


def _bf16(torch, v):
    return torch.tensor(v, dtype=torch.float32).to(torch.bfloat16).double().numpy()


GATES = [float(v) for v in np.concatenate([np.linspace(-80, 80, 641), np.linspace(-3, 3, 97)])]


@pytest.mark.parametrize("kw", [dict(), dict(gate_clamp_max=90.0, up_clamp=2.0)], ids=str)
def test_glu_is_accurate(torch, moe, kw):
    """h = g sigmoid(g) to 10 U: the exponential 5 U, its sum with 1 U, the reciprocal
    2 U, the product and the scale U each; the product with 1 is exact."""
    g = _bf16(torch, GATES)
    gu = torch.cat([_one_a_block(torch, GATES, 256), _one_a_block(torch, [1.0] * len(GATES), 256)], dim=1)
    _, s = moe.glu_quantize_fp8(gu, **kw)
    want = np.abs(g * R.sigmoid(g))
    live = want > 0
    for got in _values(s):
        assert np.all(np.abs(got - want)[live] <= 10 * U * want[live])


def test_glu_situ_is_accurate(torch, moe):
    """h = bg tanh(g / bg) sigmoid(g) bu tanh(u / bu): two tanh of rounded arguments
    10 U, the sigmoid 8 U, five products and the scale."""
    g = _bf16(torch, GATES)
    gu = torch.cat([_one_a_block(torch, GATES, 128), _one_a_block(torch, [1.0] * len(GATES), 128)], dim=1)
    _, s = moe.glu_quantize_fp8(gu, activation=1, situ_beta_gate=1.5, situ_beta_up=2.0)
    want = np.abs(1.5 * np.tanh(g / 1.5) * R.sigmoid(g) * 2 * np.tanh(0.5))
    live = want > 0
    assert np.all(np.abs(_values(s)[0] - want)[live] <= 24 * U * want[live])


@pytest.mark.parametrize("kw", [dict(), dict(gate_clamp_max=90.0, up_clamp=2.0)], ids=str)
def test_glu_gradient_is_accurate(torch, moe, kw):
    """da = s (1 + g (1 - s)) to 12 U of its terms s (1 + |g| (1 - s)): s 8 U, less the
    more of it lies in 1 - s, which is as accurate; its product, the fused sum, the
    product and the scale U each."""
    g = _bf16(torch, GATES)
    one = _one_a_block(torch, [1.0] * len(GATES), 128)
    gu = torch.cat([_one_a_block(torch, GATES, 128), one], dim=1)
    _, s = moe.glu_backward_quantize_fp8(gu, one, **kw)
    sg, c = R.sigmoid(g), R.sigmoid(-g)
    got, (up,) = _values(s[:1])[0], _values(s[1:])
    live = np.abs(sg * (1 + g * c)) > 0
    assert np.all(np.abs(got - np.abs(sg * (1 + g * c)))[live] <= 12 * U * (sg * (1 + np.abs(g) * c))[live])
    h = np.abs(g * sg)
    assert np.all(np.abs(up - h)[h > 0] <= 10 * U * h[h > 0])


def test_glu_situ_gradient_is_accurate(torch, moe):
    """The slope of a tanh is 1 - t^2, to 24 U of 1: t 5 U twice, its square and the
    difference; the other factors as above."""
    beta = 1.5
    x = [v for v in GATES if abs(v) <= 30]
    g = _bf16(torch, x)
    one = _one_a_block(torch, [1.0] * len(x), 128)
    edge = _one_a_block(torch, x, 128)
    slope = 1 / np.cosh(g / beta) ** 2
    # Of the up half: du = d a(g = 1) slope.
    _, s = moe.glu_backward_quantize_fp8(torch.cat([one, edge], dim=1), one, activation=1, situ_beta_gate=beta, situ_beta_up=beta)
    a1 = beta * np.tanh(1 / beta) * R.sigmoid(np.float64(1.0))
    got = _values(s)[1]
    got[got == 448] = 0      # a block of zeros has scale 1
    assert np.all(np.abs(got - a1 * slope) <= 32 * U * a1)
    # Of the gate half: dg = d b(u = 1) (slope sigmoid + a (1 - sigmoid)).
    _, s = moe.glu_backward_quantize_fp8(torch.cat([edge, one], dim=1), one, activation=1, situ_beta_gate=beta, situ_beta_up=beta)
    b = beta * np.tanh(1 / beta)
    t2 = beta * np.tanh(g / beta) * R.sigmoid(g) * R.sigmoid(-g)
    got = _values(s)[0]
    got[got == 448] = 0
    assert np.all(np.abs(got - np.abs(slope * R.sigmoid(g) + t2) * b) <= 40 * U * (R.sigmoid(g) + np.abs(t2)) * b)


@pytest.mark.parametrize("kw", [dict(), dict(up_clamp=2.0), dict(gate_clamp_max=3.3e38), dict(activation=1)], ids=str)
def test_glu_of_the_largest_gates(torch, moe, kw):
    """Gates whose product with log2 e is past fp32: the sigmoid is 1 or 0, the unit and
    its gradient are finite; infinities and NaN give the block's scale NaN."""
    big = [2.3e38, 2.4e38, 3.3e38, -2.3e38, -2.4e38, -3.3e38]
    gu = torch.cat([_one_a_block(torch, big, 128), _one_a_block(torch, [0.5] * 6, 128)], dim=1)
    one = _one_a_block(torch, [1.0] * 6, 128)
    ref = dict(act="situ") if kw.get("activation") else dict(cg=kw.get("gate_clamp_max", np.inf), cu=kw.get("up_clamp", np.inf))
    for (q, s), want in ((moe.glu_quantize_fp8(gu, **kw), R.glu(gu.double().cpu().numpy(), **ref)),
                         (moe.glu_backward_quantize_fp8(gu, one, **kw),
                          R.glu_backward(gu.double().cpu().numpy(), one.double().cpu().numpy(), **ref))):
        for b in range(s.shape[0]):
            w = np.abs(want[:, b * 128])
            got = np.where(w == 0, 0.0, _values(s)[b])
            assert np.all(np.abs(got - w) <= 40 * U * np.maximum(w, 1e-30)), (b, got, w)
            assert np.all((q.cpu().numpy()[:, b * 128] & 0x7F) == np.where(w == 0, 0, 0x7E))
    for v in (float("inf"), float("nan")):
        bad = gu.clone()
        bad[0, 0] = v
        _, s = moe.glu_quantize_fp8(bad, **kw)
        clamped = v > 0 and (kw.get("gate_clamp_max") or kw.get("activation"))
        assert torch.isnan(s[0, 0]).item() == (not clamped) and not torch.isnan(s[0, 1:]).any()


# ----------------------------------------------------------------- routing
def _exact_route(l, k, scores, n_groups, keep):
    """Experts of one row without a bias, groups scored by their two best, in decimals
    long enough that nothing saturates."""
    E = len(l)
    n = E // n_groups
    with localcontext() as ctx:
        ctx.prec = 1200
        ctx.Emin, ctx.Emax = -10 ** 9, 10 ** 9
        d = [Decimal(float(v)) for v in l]
        m = max(d)
        f = (lambda v: 1 / (1 + (-v).exp())) if scores == "sigmoid" else (lambda v: (v - m).exp())
        known = {}

        def score(v):
            if v not in known:
                known[v] = f(v)
            return known[v]

        best = [sum(score(v) for v in sorted(d[g * n:(g + 1) * n], reverse=True)[:2]) for g in range(n_groups)]
        # Within the context: a decimal's sign change rounds to it.
        kept = sorted(range(n_groups), key=lambda g: (-best[g], g))[:keep]
        inside = [e for e in range(E) if e // n in kept]
        return sorted(inside, key=lambda e: (-d[e], e))[:k]


def _saturated_rows(E, seed):
    """Rows whose scores are 1 (or 0) to 64 bits, with distinct logits."""
    rng = np.random.default_rng(seed)
    f32 = np.float32
    rows = [40 + np.arange(E) % 16, rng.uniform(38, 60, E), rng.uniform(28, 60, E), rng.uniform(28, 29, E),
            50 + rng.permutation(E) * 3.8e-6, -60 - rng.uniform(0, 30, E), -800 - 3 * rng.permutation(E) % 400,
            rng.uniform(-60, 60, E), np.where(np.arange(E) % 3 == 0, rng.uniform(40, 60, E), -rng.uniform(40, 60, E)),
            rng.integers(28, 34, E)]
    rows[1] = np.where(np.arange(E) == 5, 0.0, rows[1])          # softmax: the rest below exp(-745) of it
    rows.append(np.where(np.arange(E) == 3, 1000.0, rng.integers(0, 40, E)))
    rows.append(np.where(np.arange(E) % (E // 4) == 1, 900.0, rng.uniform(0, 60, E)))   # equal bests, the second decides
    return np.array(rows, f32)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("E,groups,keep,k", [(16, 4, 2, 2), (64, 8, 3, 6), (512, 4, 2, 8), (1024, 8, 4, 8)])
def test_route_saturated_scores(torch, moe, scores, E, groups, keep, k):
    l = _saturated_rows(E, E)
    idx, _ = moe.route(torch.from_numpy(l).cuda(), k, scores=scores, n_groups=groups, topk_groups=keep, group_top=2,
                       renormalize=True)
    got = idx.cpu().numpy()
    for t in range(len(l)):
        assert got[t].tolist() == _exact_route(l[t], k, scores, groups, keep), (t, l[t][:16])


def test_route_saturated_worked_examples(torch, moe):
    kw = dict(scores="sigmoid", group_top=2)
    idx, _ = moe.route(torch.arange(40.0, 56.0).cuda()[None], 2, n_groups=4, topk_groups=2, **kw)
    assert idx.tolist() == [[15, 14]]
    idx, _ = moe.route(torch.tensor([[40.0, 41, 39, 42, 40, 40, 38, 38]]).cuda(), 2, n_groups=2, topk_groups=1, **kw)
    assert idx.tolist() == [[3, 1]]


@pytest.mark.parametrize("E", [64, 256, 512, 1024])
def test_route_near_ties_beside_many_small_scores(torch, moe, E):
    """One score of nearly 1 among many that an fp32 sum may drop one by one; a bias
    lifts another key to within a few 1e-7 of the first."""
    for base in (-16.645, -16.3, -16.9, -15.95, -17.4):
        l = np.full((1, E), base, np.float32)
        l[0, 0] = 0.0
        s = R.scores_of(l[0].astype(np.float64), "softmax")[0]
        for gap in (2e-7, 3e-7, 6e-7, 1e-6, -2e-7, -3e-7, -6e-7, -1e-6):
            b = np.zeros(E, np.float32)
            b[E // 2 + 3] = np.float32(s[0] - s[1] + gap)
            idx, _ = moe.route(torch.from_numpy(l).cuda(), 1, bias=torch.from_numpy(b).cuda())
            want, _ = R.route(l, 1, bias=b.astype(np.float64))
            assert idx.cpu().numpy().tolist() == want.tolist(), (base, gap)


@pytest.mark.parametrize("scores", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [100.0, 1000.0])
def test_route_groups_whose_keys_cancel(torch, moe, scores, size):
    """Biases that force one expert of a group on and another off: each key rounds at
    its own size, their sum is small."""
    rng = np.random.default_rng(int(size))
    l = np.repeat(rng.uniform(-2, 2, (400, 1, 2)), 4, axis=1)
    l = (l + rng.uniform(-2e-5, 2e-5, (400, 4, 2))).astype(np.float32).reshape(400, 8)
    b = np.array([size, -size] * 4, np.float32)
    kw = dict(scores=scores, n_groups=4, topk_groups=2, group_top=2, renormalize=True)
    idx, _ = moe.route(torch.from_numpy(l).cuda(), 3, bias=torch.from_numpy(b).cuda(), **kw)
    want, _ = R.route(l, 3, bias=b.astype(np.float64), **kw)
    assert np.array_equal(idx.cpu().numpy(), want)


def test_route_group_sums_past_fp32(torch, moe):
    l = np.zeros((1, 8), np.float32)
    b = np.array([3.0e38, 3.0e38, 3.2e38, 3.1e38, 3.3e38, 2.0e38, -3.3e38, -3.3e38], np.float32)
    kw = dict(scores="sigmoid", n_groups=4, topk_groups=1, group_top=2)
    idx, _ = moe.route(torch.from_numpy(l).cuda(), 2, bias=torch.from_numpy(b).cuda(), **kw)
    want, _ = R.route(l, 2, bias=b.astype(np.float64), **kw)
    assert want.tolist() == [[2, 3]] and idx.cpu().numpy().tolist() == want.tolist()


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_backward_of_masked_logits(torch, moe, scores, renorm):
    """An index given for a masked logit has no gradient, whatever its dw is."""
    g = torch.Generator().manual_seed(4)
    l, dw = torch.randn(6, 24, generator=g), torch.randn(6, 3, generator=g)
    idx = torch.tensor([[0, 5, 9]] * 6, dtype=torch.int32)
    l[0, 5], l[1, 5], l[2, 0] = float("-inf"), float("nan"), float("-inf")
    dw[0, 1], dw[1, 1], dw[2, 0] = float("inf"), 1.0, float("nan")
    idx[3, 1], dw[3, 1] = -1, float("nan")
    idx[4, 2], dw[4, 2] = 24, float("inf")
    got = moe.route_backward(l.cuda(), idx.cuda(), dw.cuda(), scores=scores, renormalize=renorm).cpu()
    clean = dw.clone()
    for t, j in ((0, 1), (1, 1), (2, 0), (3, 1), (4, 2)):
        clean[t, j] = 0.0
    want = R.route_backward(l.double().numpy(), idx.numpy(), clean.double().numpy(), scores, renorm)
    assert np.all(np.abs(got.double().numpy() - want) <= 1e-6)      # |dw| sums to less than 6; 64 U each


# ------------------------------------------------------------ quantisation
def _tiny_blocks(exact_in):
    """Blocks whose scale is exact (or raised to 2^-126), filled with exact middles of
    codes and their neighbours, the maxima from 2^-133 to 2^-105."""
    mids = (R.GRID[1:] + R.GRID[:-1]) / 2
    rows = []
    for k in range(-143, -112):
        for c in range(16, 32):
            s = max(c * 2.0 ** k, 2.0 ** -126)
            amax = 448.0 * c * 2.0 ** k
            x = np.concatenate([mids, R.GRID[:-1]]) * s
            x = x[(x <= amax) & exact_in(x)]
            if not exact_in(np.array([amax]))[0]:
                continue
            x = np.resize(np.concatenate([[amax], x]), 128) * np.resize([1.0, -1.0, 1.0], 128)
            x[0] = amax
            rows.append(x)
    return np.array(rows)


def test_quantize_tiny_blocks_fp32(torch, moe):
    x = _tiny_blocks(lambda v: v.astype(np.float32).astype(np.float64) == v)
    q, s = moe.quantize_rows_fp8(torch.from_numpy(x.astype(np.float32)).cuda())
    rq, rs = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def _bf16_exact(v):
    f = v.astype(np.float32)
    return (f.astype(np.float64) == v) & ((f.view(np.uint32) & 0xFFFF) == 0)


def test_quantize_tiny_blocks_bf16(torch, moe):
    x = _tiny_blocks(_bf16_exact)
    bits = (x.astype(np.float32).view(np.uint32) >> 16).astype(np.uint16)
    xt = torch.from_numpy(bits.view(np.int16)).cuda().view(torch.bfloat16)
    q, s = moe.quantize_rows_fp8(xt)
    rq, rs = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)
    # The weights' quantiser: the same blocks, one above the other.
    for r in range(0, len(x), 37):
        w, ws = moe.quantize_weights_fp8(xt[r:r + 1])
        assert np.array_equal(w.cpu().numpy(), rq[r:r + 1]) and float(ws[0, 0]) == float(rs[0, r])


def test_quantize_every_bf16_significand(torch, moe):
    """Every pair of significands of an element and its block's maximum, over the
    binades that codes reach."""
    rows = []
    for b in range(128, 256):
        x = np.array([a * 2.0 ** e for e in range(-18, 1) for a in range(128, 256)])
        x = x[x <= b]
        for i in range(0, len(x), 127):
            rows.append(np.concatenate([[b], np.resize(x[i:i + 127], 127)]))
    x = np.array(rows) * np.resize([1.0, -1.0], len(rows))[:, None]
    q, s = moe.quantize_rows_fp8(torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16).cuda())
    rq, rs = R.quantize_rows(x)
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


# ---------------------------------------------------------------- time-outs
@pytest.mark.parametrize("M,N,K,loaded", [(8, 128, 4096, 0), (8, 128, 4096, 3), (20, 300, 8192, 1), (100, 512, 2048, 6),
                                          (600, 512, 8192, 0), (2560, 2048, 2048, 0), (2560, 2048, 2048, 9),
                                          (2560, 2048, 8192, 20)])
def test_matmul_waits_run_out(torch, moe, M, N, K, loaded):
    """Loads that stop early (clusters that divide a contraction, small tiles, full
    ones): the error word says so once, the next products are right."""
    from deterministic_expert_b200 import selftest_matmul_timeout
    g = torch.Generator().manual_seed(M)
    a, sa = moe.quantize_rows_fp8(torch.randn(700, 1024, generator=g).cuda())
    w, sw = moe.quantize_weights_fp8(torch.randn(384, 1024, generator=g).to(torch.bfloat16).cuda())
    parts = [slice(0, 8), slice(8, 90), slice(0, 700)]
    want = [moe.matmul_fp8(a[p], sa[:, p], w, sw) for p in parts]
    assert moe.operator_error() == moe.MOE_OK
    assert selftest_matmul_timeout(M, N, K, loaded) == moe.MOE_ETIMEOUT
    assert moe.operator_error() == moe.MOE_OK
    for _ in range(3):
        for p, x in zip(parts, want):
            assert torch.equal(moe.matmul_fp8(a[p], sa[:, p], w, sw), x)
    assert moe.operator_error() == moe.MOE_OK


@pytest.mark.parametrize("M,N,K", [(8, 128, 1024), (300, 512, 1024), (2560, 2048, 1024)])
def test_matmul_waits_do_not_run_out_otherwise(torch, moe, M, N, K):
    from deterministic_expert_b200 import selftest_matmul_timeout
    assert selftest_matmul_timeout(M, N, K, K // 128) == moe.MOE_OK
    assert selftest_matmul_timeout(M, N, K, 1000) == moe.MOE_OK


def test_matmul_errors_are_read_once_and_not_lost(torch, moe):
    """Failing products on one stream while another thread reads the error word on its
    own: each failure is seen by one of the two, and no more reads see one than waits
    that could raise it."""
    import threading
    import time
    from deterministic_expert_b200 import selftest_matmul_timeout
    runs, seen, stop = 12, [0, 0], threading.Event()
    streams = [torch.cuda.Stream() for _ in range(2)]
    assert moe.operator_error() == moe.MOE_OK

    def read():
        while not stop.is_set():
            status = moe.operator_error(stream=streams[1])
            assert status in (moe.MOE_OK, moe.MOE_ETIMEOUT)
            seen[1] += status == moe.MOE_ETIMEOUT

    t = threading.Thread(target=read)
    t.start()
    try:
        for _ in range(runs):
            before = seen[1]
            mine = selftest_matmul_timeout(100, 512, 2048, 3, stream=streams[0]) == moe.MOE_ETIMEOUT
            seen[0] += mine
            # What the self-test did not find, the other had taken: before it returned.
            for _ in range(1000):
                if mine or seen[1] > before:
                    break
                time.sleep(0.001)
            assert mine or seen[1] > before
    finally:
        stop.set()
        t.join()
    assert sum(seen) >= runs
    assert moe.operator_error() == moe.MOE_OK


# ------------------------------------------------------------ given streams
def _calls(torch, moe):
    """Every operator with tensors of its own: (call of (tensors, stream), tensors)."""
    g = torch.Generator().manual_seed(3)

    def rn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g).to(dtype).cuda()

    bf = torch.bfloat16
    x, logits, bias = rn(64, 512, dtype=bf), rn(64, 16), rn(16)
    idx, w = moe.route(logits, 4)
    off, tok, slot = moe.group_rows(idx, 16)
    q, s = moe.quantize_rows_fp8(x, token_of_row=tok)
    wq, ws = moe.quantize_weights_fp8(rn(16, 256, 512, dtype=bf))
    y, gu, dh, n = rn(256, 512, dtype=bf), rn(256, 512, dtype=bf), rn(256, 256, dtype=bf), off[16:].clone()
    return {
        "route": (lambda t, st: moe.route(t[0], 4, bias=t[1], stream=st), (logits, bias)),
        "route_backward": (lambda t, st: moe.route_backward(t[0], t[1], t[2], stream=st), (logits, idx, w)),
        "group_rows": (lambda t, st: moe.group_rows(t[0], 16, stream=st), (idx,)),
        "quantize_rows_fp8": (lambda t, st: moe.quantize_rows_fp8(t[0], token_of_row=t[1], n_rows=t[2], stream=st), (x, tok, n)),
        "quantize_weights_fp8": (lambda t, st: moe.quantize_weights_fp8(t[0], stream=st), (y,)),
        "glu_quantize_fp8": (lambda t, st: moe.glu_quantize_fp8(t[0], stream=st), (gu,)),
        "glu_backward_quantize_fp8": (lambda t, st: moe.glu_backward_quantize_fp8(t[0], t[1], stream=st), (gu, dh)),
        "matmul_fp8": (lambda t, st: moe.matmul_fp8(*t[:4], offsets=t[4], stream=st), (q, s, wq, ws, off)),
        "combine_rows": (lambda t, st: moe.combine_rows(t[0], t[1], t[2], addend=t[3], stream=st), (y, slot, w, x)),
        "combine_rows_backward": (lambda t, st: moe.combine_rows_backward(t[3], t[0], t[1], t[2], stream=st), (y, slot, w, x)),
    }


@pytest.mark.parametrize("raw", [False, True])
def test_tensors_dropped_after_a_call_on_another_stream(torch, moe, raw):
    """A busy stream reads its tensors long after the caller let go of them: their
    memory is not handed out meanwhile."""
    side = torch.cuda.Stream()
    for name, (call, tensors) in _calls(torch, moe).items():
        want = call(tensors, None)
        torch.cuda.synchronize()
        mine = [t.clone() for t in tensors]
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)       # about 10 ms
        got = call(mine, side.cuda_stream if raw else side)
        del mine
        # The same sizes again, which the allocator would take from what was dropped.
        other = [torch.zeros_like(t) for t in tensors for _ in range(2)]
        torch.cuda.synchronize()
        for a, b in zip(got if isinstance(got, tuple) else (got,), want if isinstance(want, tuple) else (want,)):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), name
        del other


def test_captured_on_a_given_stream(torch, moe):
    """A graph of calls on a given stream whose temporaries are dropped meanwhile."""
    g = torch.Generator().manual_seed(8)
    x = torch.randn(64, 512, generator=g).to(torch.bfloat16).cuda()
    w, sw = moe.quantize_weights_fp8(torch.randn(256, 512, generator=g).to(torch.bfloat16).cuda())
    want = moe.matmul_fp8(*moe.quantize_rows_fp8(x), w, sw)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for _ in range(3):
            q, s = moe.quantize_rows_fp8(x, stream=side)
            out = moe.matmul_fp8(q, s, w, sw, stream=side.cuda_stream)
            del q, s
    out.zero_()
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_tensors_that_require_a_gradient(torch, moe):
    """Refused where a gradient would be lost, each tensor of each call; taken without
    one, and inside an autograd function."""
    for name, (call, tensors) in _calls(torch, moe).items():
        for i, t in enumerate(tensors):
            if not t.is_floating_point():
                continue
            mine = list(tensors)
            mine[i] = t.clone().requires_grad_()
            with pytest.raises(ValueError, match="gradient"):
                call(mine, None)
            with torch.no_grad():
                call(mine, None)

    class Weights(torch.autograd.Function):
        @staticmethod
        def forward(ctx, logits):
            idx, w = moe.route(logits, 4, renormalize=True)
            ctx.save_for_backward(logits, idx)
            ctx.mark_non_differentiable(idx)
            return idx, w

        @staticmethod
        def backward(ctx, _, dw):
            logits, idx = ctx.saved_tensors
            return moe.route_backward(logits, idx, dw.contiguous(), renormalize=True)

    l = torch.randn(8, 16, generator=torch.Generator().manual_seed(1)).cuda().requires_grad_()
    dw = torch.randn(8, 4, generator=torch.Generator().manual_seed(2)).cuda()
    idx, w = Weights.apply(l)
    w.backward(dw)
    assert torch.equal(l.grad, moe.route_backward(l.detach(), idx, dw, renormalize=True))
