"""GPU parity of the handle-free expert-layer operators against their fp64
statements (tests/operators_ref.py).

Tolerances, fixed before the first run:
  integers (experts, grouping, E4M3 codes of given values, fp32 scales of given
      values)                                      equal
  routing weights, fp32   64 * 2^-24 relative (expf 2 ulp, its rounded argument up
      to |l| <= 16, a sum of at most 1024 terms in a tree, two divisions)
  gated units, fp32       16 * 2^-24 relative before the code's rounding
  products                (128 + blocks) * 2^-23 of the terms' magnitudes (every
      addition of a block and of the blocks rounds, or truncates, once), and half a
      step of the output type: 2^-8 relative for bf16, 2^-24 for fp32
  combine                 (k + 1) * 2^-24 of the terms' magnitudes and half a step
"""
import numpy as np
import pytest

import operators_ref as R

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
HALF = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}


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


def _dt(torch, name):
    return {"bf16": torch.bfloat16, "f32": torch.float32}[name]


def _randn(torch, seed, *shape, dtype="f32", scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(_dt(torch, dtype)).cuda()


def n64(t):
    import torch
    if t.dtype == torch.float8_e4m3fn:
        t = t.float()
    return (t.double() if t.is_floating_point() else t).cpu().numpy()


# ----------------------------------------------------------------- routing
ROUTES = [
    # T, E, k, scores, bias, groups, keep, top, renorm, dtype
    (1, 256, 8, "sigmoid", True, 8, 4, 2, True, "f32"),
    (33, 256, 8, "sigmoid", True, 8, 4, 2, True, "bf16"),
    (17, 64, 6, "softmax", False, 1, 1, 1, True, "f32"),
    (9, 64, 6, "softmax", True, 1, 1, 1, False, "bf16"),
    (5, 160, 6, "softmax", False, 8, 3, 1, False, "f32"),
    (5, 160, 6, "softmax", False, 8, 3, 2, True, "f32"),
    (7, 7, 7, "sigmoid", False, 1, 1, 1, False, "f32"),
    (4, 1, 1, "softmax", True, 1, 1, 2, False, "f32"),
    (6, 60, 4, "sigmoid", True, 5, 2, 2, False, "bf16"),
    (3, 1024, 32, "softmax", True, 1, 1, 1, True, "f32"),
    (3, 896, 16, "sigmoid", True, 1, 1, 1, True, "f32"),
    (5, 384, 8, "sigmoid", True, 32, 4, 2, True, "f32"),
    (5, 100, 3, "softmax", True, 2, 1, 2, True, "bf16"),
    (130, 128, 8, "sigmoid", False, 16, 8, 2, True, "bf16"),
]


def _route_args(c):
    T, E, k, scores, bias, groups, keep, top, renorm, dtype = c
    return dict(scores=scores, n_groups=groups, topk_groups=keep, group_top=top, renormalize=renorm, routed_scale=2.5)


def _check_route(torch, moe, logits, k, bias, kw, alone=True):
    idx, w = moe.route(logits, k, bias=bias, **kw)
    torch.cuda.synchronize()
    ref_idx, ref_w = R.route(n64(logits), k, bias=None if bias is None else n64(bias), **kw)
    assert np.array_equal(idx.cpu().numpy(), ref_idx)
    got = n64(w)
    assert np.all(np.abs(got - ref_w) <= 64 * U * np.abs(ref_w) + 1e-37)
    if alone:   # a row does not depend on the others
        for t in (0, logits.shape[0] - 1):
            i1, w1 = moe.route(logits[t:t + 1], k, bias=bias, **kw)
            assert torch.equal(i1[0], idx[t]) and torch.equal(w1[0].view(torch.int32), w[t].view(torch.int32))
    return idx, w


@pytest.mark.parametrize("c", ROUTES, ids=lambda c: "-".join(str(v) for v in c))
def test_route(torch, moe, c):
    T, E, k, scores, bias, groups, keep, top, renorm, dtype = c
    logits = _randn(torch, T + E, T, E, dtype=dtype, scale=2.0)
    b = _randn(torch, 5, E, scale=0.1) if bias else None
    _check_route(torch, moe, logits, k, b, _route_args(c))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_route_strides_and_alignment(torch, moe, dtype):
    base = _randn(torch, 1, 12, 300, dtype=dtype)
    for off, E in ((0, 256), (1, 256), (8, 128), (3, 61)):
        v = base[:, off:off + E]
        kw = dict(scores="sigmoid", n_groups=1, renormalize=True)
        _check_route(torch, moe, v, 5, None, kw)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("groups,keep,top", [(1, 1, 1), (4, 2, 1), (4, 2, 2)])
def test_route_ties_and_masks(torch, moe, scores, bias, groups, keep, top):
    """Equal keys, neighbours one fp32 step apart, masked experts, rows with fewer
    than k experts left, rows with none."""
    E, k = 32, 6
    l = _randn(torch, 7, 24, E).cpu()
    l[0] = 0.0                                   # all equal
    l[1] = torch.tensor([1.0, 2.0, 2.0, 1.0] * 8)
    l[2, 1::2] = l[2, 0::2]                      # pairs of equals
    one = torch.nextafter(torch.tensor(0.5), torch.tensor(1.0))
    l[3] = torch.where(torch.arange(E) % 3 == 1, one, torch.tensor(0.5))   # one step apart
    l[4] = 0.5 + torch.arange(E) * 6e-8
    l[5] = float("-inf")                         # nothing left
    l[6] = float("nan")
    l[7, 4:] = float("-inf")                     # four left
    l[8, ::2] = float("nan")
    l[9, :16] = float("-inf")                    # whole groups masked
    l[10] = torch.finfo(torch.float32).min       # the type's lowest value is a number
    l[11] = torch.finfo(torch.float32).min
    l[11, 5] = 3.0
    l[12, 31] = float("-inf")
    l[13, 1:] = float("-inf")
    l[14] = -0.0
    l[14, ::2] = 0.0                             # equal as numbers
    b = None
    if bias:
        b = torch.zeros(E)
        b[8:] = _randn(torch, 9, E - 8).cpu() * 0.05
        b[3] = float("-inf")                     # an expert taken out by its bias
        b = b.cuda()
    kw = dict(scores=scores, n_groups=groups, topk_groups=keep, group_top=top, renormalize=True, routed_scale=1.0)
    idx, w = _check_route(torch, moe, l.cuda(), k, b, kw, alone=False)
    assert (idx[5] == -1).all() and (w[5] == 0).all() and (idx[6] == -1).all()


def test_route_far_below_zero(torch, moe):
    """Sigmoids that underflow in fp32 still have weights that add to one."""
    l = _randn(torch, 3, 4, 16).cpu() - torch.tensor([[70.0], [100.0], [300.0], [30000.0]])
    kw = dict(scores="sigmoid", renormalize=True)
    _, w = _check_route(torch, moe, l.cuda(), 4, None, kw)
    assert torch.allclose(w.sum(1), torch.ones(4, device="cuda"), atol=1e-6)


def test_route_near_ties_in_bulk(torch, moe):
    """Logits on a coarse grid with a bias of fine steps: many keys closer than
    fp32 can order, all in the order of 64 bits."""
    g = torch.Generator().manual_seed(2)
    l = torch.randint(-8, 8, (64, 64), generator=g).float() / 4
    b = torch.randint(0, 4, (64,), generator=g).double() * 2.0 ** -26
    for scores in ("sigmoid", "softmax"):
        kw = dict(scores=scores, n_groups=8, topk_groups=3, group_top=2, renormalize=False)
        _check_route(torch, moe, l.cuda(), 8, b.float().cuda(), kw, alone=False)


@pytest.mark.parametrize("c", ROUTES, ids=lambda c: "-".join(str(v) for v in c))
def test_route_backward(torch, moe, c):
    T, E, k, scores, bias, groups, keep, top, renorm, dtype = c
    logits = _randn(torch, T + E, T, E, dtype=dtype, scale=2.0)
    kw = _route_args(c)
    idx, _ = moe.route(logits, k, **kw)
    dw = _randn(torch, 11, T, k)
    got = n64(moe.route_backward(logits, idx, dw, **kw))
    ref = R.route_backward(n64(logits), idx.cpu().numpy(), n64(dw), scores, renorm, 2.5)
    # Differences of fp32 values of the size of scale * dw * s.
    s = np.stack([R.scores_of(r, scores)[0] for r in n64(logits)])
    if renorm:
        s = np.minimum(1.0, s / np.maximum(np.take_along_axis(s, idx.cpu().numpy(), 1).sum(1, keepdims=True), 1e-300))
    big = 2.5 * np.abs(n64(dw)).sum(axis=1, keepdims=True) * s
    assert np.all(np.abs(got - ref) <= 64 * U * big + HALF[dtype] * np.abs(ref) + 1e-37)


def test_route_backward_indexes(torch, moe):
    """Unfilled slots have no gradient, an expert named twice gets both, masked
    logits get none; wide and narrow rows of a wider buffer."""
    l = _randn(torch, 1, 6, 40)
    l[1, 3] = float("-inf")
    l[2] = float("-inf")
    idx = torch.tensor([[0, 5, 39], [3, 3, 4], [1, 2, 3], [-1, 7, 99], [-1, -1, -1], [8, 8, 8]], dtype=torch.int32)
    dw = _randn(torch, 2, 6, 3)
    for scores in ("softmax", "sigmoid"):
        for renorm in (False, True):
            out = torch.full((6, 48), 7.0, device="cuda")
            moe.route_backward(l, idx.cuda(), dw, scores=scores, renormalize=renorm, out=out[:, 3:43])
            ref = R.route_backward(n64(l), idx.numpy(), n64(dw), scores, renorm)
            assert np.all(np.abs(n64(out[:, 3:43]) - ref) <= 1e-6)   # |dw| sums to less than 6; 64 u each
            assert (out[:, :3] == 7).all() and (out[:, 43:] == 7).all()


# ---------------------------------------------------------------- grouping
@pytest.mark.parametrize("T,k,E", [(0, 2, 8), (1, 1, 1), (1, 8, 256), (16, 8, 256), (100, 3, 7), (1000, 6, 64),
                                   (8192, 8, 256), (513, 2, 1024), (40000, 2, 60)])
def test_group_rows(torch, moe, T, k, E):
    g = torch.Generator().manual_seed(T + E)
    idx = torch.randint(-1 if T % 2 else 0, E, (T, k), generator=g, dtype=torch.int32)   # repeats and -1 among them
    if T > 10:
        idx[3] = E + 5
        idx[4, :] = 0
    off, tok, slot = moe.group_rows(idx.cuda(), E)
    torch.cuda.synchronize()
    flat = idx.reshape(-1).numpy()
    ok = (flat >= 0) & (flat < E)
    order = np.nonzero(ok)[0][np.argsort(flat[ok], kind="stable")]
    want_tok = np.full(T * k, -1, np.int32)
    want_tok[:len(order)] = order // k
    want_slot = np.full(T * k, -1, np.int32)
    want_slot[order] = np.arange(len(order))
    assert np.array_equal(off.cpu().numpy(), np.concatenate([[0], np.cumsum(np.bincount(flat[ok], minlength=E))]))
    assert np.array_equal(tok.cpu().numpy(), want_tok)
    assert np.array_equal(slot.cpu().numpy().reshape(-1), want_slot)
    if T <= 1000:
        o, t, s = R.group_rows(idx.numpy(), E)
        assert np.array_equal(o, off.cpu().numpy()) and np.array_equal(t, want_tok) and np.array_equal(s.reshape(-1), want_slot)


# ------------------------------------------------------------ quantisation
def _edge_rows(torch, dtype, R_, K):
    x = _randn(torch, K, R_, K, dtype=dtype).cpu()
    x[0] = 0.0
    if R_ > 4:
        x[1, :] = -0.0
        x[1, 0] = 448.0                                     # scale 1: exact middles of codes below
        x[1, 1:min(K, 16)] = torch.tensor([1.0625, 1.1875, -1.3125, 2.0 ** -10, 3 * 2.0 ** -10, -5 * 2.0 ** -10, 232.0,
                                           240.0, 0.0009, 17.0, 19.0, 432.0, 416.0, 2.0 ** -7, 0.0146])[:min(K, 16) - 1].to(x.dtype)
        x[2] = torch.arange(K).to(x.dtype) * 2.0 ** -100    # tiny
        x[3] *= 1e30
        x[4, K // 2] = 1e4                                  # one large among small
    return x.cuda()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("rows,K", [(1, 16), (2, 128), (7, 144), (33, 272), (5, 2048), (129, 1408)])
def test_quantize_rows(torch, moe, dtype, rows, K):
    x = _edge_rows(torch, dtype, rows, K)
    q, s = moe.quantize_rows_fp8(x)
    torch.cuda.synchronize()
    rq, rs = R.quantize_rows(n64(x))
    assert np.array_equal(s.cpu().numpy(), rs)
    assert np.array_equal(q.cpu().numpy(), rq)


def test_quantize_middles_of_codes(torch, moe):
    """fp32 values chosen within a few steps of the middle of two codes under scales
    that are not powers of two."""
    rng = np.random.default_rng(5)
    mids = (R.GRID[1:] + R.GRID[:-1]) / 2
    rows = []
    for _ in range(64):
        amax = np.float32(rng.uniform(0.5, 2.0))
        s = np.float64(R.scale_of(amax))
        m = np.float32(rng.choice(mids, 127) * s)
        m = (m.view(np.int32) + rng.integers(-3, 4, 127).astype(np.int32)).view(np.float32)
        rows.append(np.concatenate([[amax], np.minimum(m, amax) * rng.choice([-1, 1], 127)]))
    x = np.array(rows, np.float32)
    q, s = moe.quantize_rows_fp8(torch.from_numpy(x).cuda())
    rq, rs = R.quantize_rows(x.astype(np.float64))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def test_quantize_gather_strides_and_untouched_rows(torch, moe):
    base = _randn(torch, 3, 10, 512, dtype="bf16")
    x = base[:, 64:64 + 272]
    tok = torch.tensor([3, 9, -1, 0, 0, 10, 5], dtype=torch.int32, device="cuda")
    q = torch.full((7, 272), 0x55, dtype=torch.uint8, device="cuda")
    sb = torch.full((3, 11), -3.0, device="cuda")
    n = torch.tensor([6], dtype=torch.int32, device="cuda")
    moe.quantize_rows_fp8(x, token_of_row=tok, n_rows=n, out_codes=q, out_scales=sb[:, 2:9])
    torch.cuda.synchronize()
    rq, rs = R.quantize_rows(n64(x))
    for r, t in enumerate([3, 9, -1, 0, 0, -1, -1]):    # 10 is no row of x; row 6 lies behind n_rows
        if t < 0:
            assert (q[r] == 0x55).all() and (sb[:, 2 + r] == -3).all()
        else:
            assert np.array_equal(q[r].cpu().numpy(), rq[t]) and np.array_equal(sb[:, 2 + r].cpu().numpy(), rs[:, t])
    assert (sb[:, :2] == -3).all() and (sb[:, 9:] == -3).all()


def test_quantize_non_finite(torch, moe):
    x = _randn(torch, 1, 4, 256)
    x[0, 5] = float("nan")
    x[1, 200] = float("inf")
    x[2, 0] = -float("inf")
    q, s = moe.quantize_rows_fp8(x)
    rq, rs = R.quantize_rows(n64(x))
    assert np.array_equal(s.cpu().numpy(), rs, equal_nan=True) and np.array_equal(q.cpu().numpy(), rq)
    assert torch.isnan(s).sum() == 3


@pytest.mark.parametrize("G,N,K", [(1, 128, 128), (2, 200, 272), (3, 1, 16), (1, 257, 640)])
def test_quantize_weights(torch, moe, G, N, K):
    w = _randn(torch, N, G, N, K, dtype="bf16", scale=0.02)
    w[0, :, :16] = 0
    q, s = moe.quantize_weights_fp8(w)
    rq, rs = R.quantize_weights(n64(w))
    assert np.array_equal(s.cpu().numpy(), rs) and np.array_equal(q.cpu().numpy(), rq)


def _check_quantised(q, s, ref, K):
    """Codes and scales of values known to 16 u relative."""
    scale = R.scale_of(np.stack([np.abs(ref[:, b:b + 128]).max(axis=1) for b in range(0, K, 128)]))
    assert np.all(np.abs(s - scale) <= 17 * U * scale)
    wide = np.repeat(s.T.astype(np.float64), 128, axis=1)[:, :K]
    err = np.abs(R.code_values(q) * wide - ref)
    # Half a step of the code (2^-4 relative, or half the smallest step), the value's own error.
    assert np.all(err <= np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide) * (1 + 2.0 ** -15) + 40 * U * np.abs(ref))


GLUS = [dict(), dict(gate_clamp_max=1.0, up_clamp=0.75), dict(activation=1), dict(activation=1, situ_beta_gate=1.5, situ_beta_up=2.0)]


def _ref_kw(kw):
    if kw.get("activation"):
        return dict(act="situ", bg=kw.get("situ_beta_gate", 4.0), bu=kw.get("situ_beta_up", 25.0))
    return dict(cg=kw.get("gate_clamp_max", np.inf), cu=kw.get("up_clamp", np.inf))


@pytest.mark.parametrize("kw", GLUS, ids=str)
@pytest.mark.parametrize("rows,I", [(1, 16), (17, 144), (33, 1408)])
def test_glu_quantize(torch, moe, kw, rows, I):
    gu = _randn(torch, I, rows, 2 * I, dtype="bf16", scale=2.0)
    gu[0, 0], gu[0, I] = 30.0, 5.0
    gu[0, 1] = -200.0
    q, s = moe.glu_quantize_fp8(gu, **kw)
    _check_quantised(q.cpu().numpy(), s.cpu().numpy(), R.glu(n64(gu), **_ref_kw(kw)), I)


@pytest.mark.parametrize("kw", GLUS, ids=str)
@pytest.mark.parametrize("rows,I", [(1, 128), (19, 256), (6, 1408)])
def test_glu_backward_quantize(torch, moe, kw, rows, I):
    gu = _randn(torch, I, rows, 2 * I, dtype="bf16", scale=2.0)
    gu[0, 0], gu[0, 1], gu[0, I] = 1.0, 40.0, 0.75      # at the clamps: the gradient passes
    dh = _randn(torch, 8, rows, I, dtype="bf16")
    q, s = moe.glu_backward_quantize_fp8(gu, dh, **kw)
    ref = R.glu_backward(n64(gu), n64(dh), **_ref_kw(kw))
    got = R.wide_rows(q.cpu().numpy(), s.cpu().numpy())
    # da has a difference of terms of size 1: an absolute error of the terms' size.
    terms = np.tile(np.abs(n64(dh)), 2) * (1 + np.tile(np.abs(n64(gu)[:, :I]), 2)) * (1 + np.tile(np.abs(n64(gu)[:, I:]), 2))
    wide = np.repeat(s.cpu().numpy().T.astype(np.float64), 128, axis=1)
    tol = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * wide) * (1 + 2.0 ** -15) + 64 * U * terms * (1 + 1 / min(kw.get("situ_beta_gate", 4.0), 1))
    assert np.all(np.abs(got - ref) <= tol)


def test_glu_rows_left_alone(torch, moe):
    gu = _randn(torch, 1, 5, 256, dtype="bf16")
    dh = _randn(torch, 2, 5, 128, dtype="bf16")
    n = torch.tensor([2], dtype=torch.int32, device="cuda")
    for call, width in ((lambda **o: moe.glu_quantize_fp8(gu, **o), 128),
                        (lambda **o: moe.glu_backward_quantize_fp8(gu, dh, **o), 256)):
        q = torch.full((5, width), 9, dtype=torch.uint8, device="cuda")
        s = torch.full((width // 128, 5), 9.0, device="cuda")
        call(n_rows=n, out_codes=q, out_scales=s)
        full, fs = call()
        assert torch.equal(q[:2], full[:2]) and torch.equal(s[:, :2], fs[:, :2])
        assert (q[2:] == 9).all() and (s[:, 2:] == 9).all()


# ---------------------------------------------------------------- products
def _operands(torch, moe, seed, M, N, K, G=1, transposed=False):
    con = N if transposed else K
    a, sa = moe.quantize_rows_fp8(_randn(torch, seed, M, con) * torch.exp(_randn(torch, seed + 1, M, 1)))
    w, sw = moe.quantize_weights_fp8(_randn(torch, seed + 2, G, N, K, dtype="bf16", scale=0.05))
    return a, sa, w, sw


def _check_matmul(torch, moe, a, sa, w, sw, offsets=None, transposed=False, dtype="bf16", out=None):
    kw = dict(transposed=transposed)
    if offsets is not None:
        kw["offsets"] = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    M = a.shape[0]
    width = w.shape[-1] if transposed else w.shape[-2]
    if out is None:
        out = torch.full((M, width), 77.0, dtype=_dt(torch, dtype), device="cuda")
    moe.matmul_fp8(a, sa, w, sw, out=out, **kw)
    torch.cuda.synchronize()
    assert moe.operator_error() == moe.MOE_OK
    ref, mag = R.matmul(a.cpu().numpy(), sa.cpu().numpy(), w.cpu().numpy(), sw.cpu().numpy(), offsets, transposed)
    got = n64(out)
    outside = np.isnan(ref)
    assert np.all(got[outside] == 77.0)
    nb = -(-a.shape[1] // 128)
    tol = (128 + nb) * 2.0 ** -23 * mag + HALF[dtype] * np.abs(ref)
    bad = ~outside & ~(np.abs(got - np.where(outside, 0, ref)) <= tol)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], ref[bad][:5])
    return out


SIZES = [(1, 256, 128), (1, 1, 16), (2, 100, 48), (8, 512, 512), (15, 264, 144), (16, 128, 400), (17, 40, 1024),
         (100, 300, 272), (129, 256, 256), (255, 256, 384), (256, 256, 128), (257, 264, 272), (300, 130, 640),
         (512, 512, 256), (700, 1000, 528)]


@pytest.mark.parametrize("M,N,K", SIZES)
def test_matmul_dense(torch, moe, M, N, K):
    a, sa, w, sw = _operands(torch, moe, M + N + K, M, N, K)
    _check_matmul(torch, moe, a, sa, w, sw)


@pytest.mark.parametrize("M,N,K", [(1, 16, 16), (3, 128, 256), (17, 272, 48), (129, 400, 144), (256, 256, 256),
                                   (300, 512, 272), (600, 144, 784)])
def test_matmul_transposed(torch, moe, M, N, K):
    a, sa, w, sw = _operands(torch, moe, M + N + K, M, N, K, transposed=True)
    _check_matmul(torch, moe, a, sa, w, sw, transposed=True, dtype="f32")


OFFSETS = [[0, 0, 5, 5, 40], [3, 10, 10, 11, 30], [0, 300, 301, 301, 900], [0, 256, 512, 600, 640], [7, 7, 7, 7, 7],
           [0, 0, 0, 0, 1], [0, 17, 273, 530, 1000]]


@pytest.mark.parametrize("transposed", [False, True])
@pytest.mark.parametrize("off", OFFSETS, ids=str)
def test_matmul_grouped(torch, moe, off, transposed):
    M, N, K = max(off[-1], 1) + (5 if off[0] else 0), 272, 400
    a, sa, w, sw = _operands(torch, moe, M, M, N, K, G=4, transposed=transposed)
    _check_matmul(torch, moe, a, sa, w, sw, off, transposed, "f32" if transposed else "bf16")


def test_matmul_many_groups(torch, moe):
    G = 200
    sizes = np.random.default_rng(1).integers(0, 9, G)
    off = [0] + [int(v) for v in np.cumsum(sizes)]
    a, sa, w, sw = _operands(torch, moe, 5, off[-1], 40, 144, G=G)
    _check_matmul(torch, moe, a, sa, w, sw, off)


@pytest.mark.parametrize("dtype,ld,shift", [("bf16", 301, 0), ("bf16", 304, 1), ("f32", 303, 0), ("f32", 304, 2), ("bf16", 320, 8)])
@pytest.mark.parametrize("M", [9, 270])
def test_matmul_output_strides(torch, moe, M, dtype, ld, shift):
    """Any pitch and alignment of the output; what lies between the rows stays."""
    a, sa, w, sw = _operands(torch, moe, M, M, 290, 272)
    buf = torch.full((M * ld + shift,), 5.0, dtype=_dt(torch, dtype), device="cuda")
    out = buf[shift:].view(M, ld)[:, :290]
    out.fill_(77.0)
    _check_matmul(torch, moe, a, sa, w, sw, dtype=dtype, out=out)
    assert (buf[shift:].view(M, ld)[:, 290:] == 5).all() and (buf[:shift] == 5).all()


@pytest.mark.parametrize("N", [1, 2, 63, 64, 65, 127, 129, 191, 193, 255, 321])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_matmul_rows_that_start_anywhere(torch, moe, N, dtype):
    """Full and small tiles of groups whose output rows start on odd elements and end
    inside every part of a segment."""
    off = [2, 2, 160, 420, 423]
    a, sa, w, sw = _operands(torch, moe, N, 430, N, 160, G=4)
    for ld, shift in ((N, 0), (N + 1, 1), (N + 3, 0)):
        buf = torch.full((430 * ld + shift,), 5.0, dtype=_dt(torch, dtype), device="cuda")
        out = buf[shift:].view(430, ld)[:, :N]
        out.fill_(77.0)
        _check_matmul(torch, moe, a, sa, w, sw, off, dtype=dtype, out=out)
        assert (buf[shift:].view(430, ld)[:, N:] == 5).all() and (buf[:shift] == 5).all()


def test_matmul_scale_pitch_and_empty(torch, moe):
    a, sa, w, sw = _operands(torch, moe, 3, 20, 64, 272)
    wide = torch.full((3, 37), float("nan"), device="cuda")
    wide[:, 5:25] = sa
    _check_matmul(torch, moe, a, wide[:, 5:25], w, sw)
    assert moe.matmul_fp8(a[:0], sa[:, :0], w, sw).shape == (0, 64)


@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_rows_do_not_depend_on_the_batch(torch, moe, transposed):
    """Each row's bits: in a batch of 1000, in small batches, in groups that share
    the same weights, and through every tile shape."""
    N, K = 384, 528
    a, sa, w, sw = _operands(torch, moe, 9, 1000, N, K, transposed=transposed)
    kw = dict(transposed=transposed, out_dtype=torch.float32)
    whole = moe.matmul_fp8(a, sa, w, sw, **kw)
    for lo, hi in ((0, 1), (999, 1000), (5, 21), (100, 133), (200, 330), (300, 556), (300, 900)):
        part = moe.matmul_fp8(a[lo:hi].contiguous(), sa[:, lo:hi].contiguous(), w, sw, **kw)
        assert torch.equal(part.view(torch.int32), whole[lo:hi].view(torch.int32)), (lo, hi)
    g = w.expand(5, N, K).contiguous()
    gs = sw.expand(5, *sw.shape[1:]).contiguous()
    off = torch.tensor([0, 3, 260, 700, 701, 1000], dtype=torch.int32, device="cuda")
    grouped = moe.matmul_fp8(a, sa, g, gs, offsets=off, **kw)
    assert torch.equal(grouped.view(torch.int32), whole.view(torch.int32))
    for _ in range(3):
        again = moe.matmul_fp8(a, sa, w, sw, **kw)
        assert torch.equal(again.view(torch.int32), whole.view(torch.int32))


def test_matmul_non_finite_rows_stay_apart(torch, moe):
    a, sa, w, sw = _operands(torch, moe, 2, 40, 64, 256)
    clean = moe.matmul_fp8(a, sa, w, sw)
    sa[1, 7] = float("nan")
    a[9, 3] = 0x7F                               # E4M3 NaN
    got = moe.matmul_fp8(a, sa, w, sw)
    keep = [r for r in range(40) if r not in (7, 9)]
    assert torch.isnan(got[7]).all() and torch.isnan(got[9]).all()
    assert torch.equal(got[keep], clean[keep])


def test_matmul_offsets_are_bounded(torch, moe):
    """Offsets outside the rows are taken as the nearest row there is."""
    a, sa, w, sw = _operands(torch, moe, 4, 30, 64, 128, G=2)
    off = torch.tensor([-5, 10, 1000], dtype=torch.int32, device="cuda")
    got = moe.matmul_fp8(a, sa, w, sw, offsets=off)
    want = moe.matmul_fp8(a, sa, w, sw, offsets=torch.tensor([0, 10, 30], dtype=torch.int32, device="cuda"))
    assert torch.equal(got, want)


# ----------------------------------------------------------------- combine
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,D", [(1, 1, 8), (5, 3, 264), (33, 8, 2048), (4, 32, 72), (7, 9, 4104)])
@pytest.mark.parametrize("weighted,added", [(True, False), (False, True)])
def test_combine(torch, moe, dtype, T, k, D, weighted, added):
    y = _randn(torch, D, T * k + 3, D, dtype=dtype)
    slots = torch.randperm(T * k + 3, generator=torch.Generator().manual_seed(1))[:T * k].reshape(T, k).to(torch.int32)
    slots[0, 0] = -1
    if k > 2:
        slots[T - 1, 2] = T * k + 3               # no row of y
    slots = slots.cuda()
    w = _randn(torch, 2, T, k) if weighted else None
    add = _randn(torch, 3, T, D, dtype="bf16") if added else None
    s, w64 = slots.cpu().numpy(), None if w is None else n64(w)
    ref = R.combine(n64(y), s, w64, None if add is None else n64(add))
    mag = R.combine(np.abs(n64(y)), s, None if w is None else np.abs(w64), None if add is None else np.abs(n64(add)))
    for odt in ("bf16", "f32"):
        got = n64(moe.combine_rows(y, slots, w, addend=add, out_dtype=_dt(torch, odt)))
        assert np.all(np.abs(got - ref) <= (k + 1) * U * mag + HALF[odt] * np.abs(ref))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,k,D", [(1, 1, 8), (5, 3, 264), (9, 8, 2048), (3, 32, 4104)])
def test_combine_backward(torch, moe, dtype, T, k, D):
    rows = T * k + 2
    y = _randn(torch, D, rows, D + 16, dtype=dtype)[:, 8:8 + D]
    slots = torch.randperm(rows, generator=torch.Generator().manual_seed(1))[:T * k].reshape(T, k).to(torch.int32)
    slots[0, k - 1] = -1
    w, dout = _randn(torch, 2, T, k), _randn(torch, 3, T, D, dtype="bf16")
    dy = torch.full((rows, D + 16), 7.0, dtype=y.dtype, device="cuda")[:, 8:8 + D]
    _, dw = moe.combine_rows_backward(dout, y, slots.cuda(), w, out_dy=dy)
    Y, Dd, W, s = n64(y), n64(dout), n64(w), slots.numpy()
    named = set()
    for t in range(T):
        for j in range(k):
            r = s[t, j]
            if r < 0:
                assert dw[t, j] == 0
                continue
            named.add(int(r))
            want = W[t, j] * Dd[t]
            assert np.all(np.abs(n64(dy[r]) - want) <= HALF[dtype] * np.abs(want) + 1e-37)
            # A dot product of D terms, in a tree.
            assert abs(float(dw[t, j]) - Dd[t] @ Y[r]) <= (D / 256 + 24) * U * (np.abs(Dd[t]) @ np.abs(Y[r]))
    for r in set(range(rows)) - named:
        assert (dy[r] == 7).all()
    dy2, none = moe.combine_rows_backward(dout, y, slots.cuda(), w, need_dw=False)
    assert none is None and all(torch.equal(dy2[r], dy[r]) for r in named)


# ------------------------------------------------- the operators together
def _layer(torch, moe, x, logits, bias, Wgu, Wd, kw, E, k, addend=None):
    """A layer of E frozen E4M3 experts, forward, as a user composes it."""
    (wgu, sgu), (wd, sd) = Wgu, Wd
    idx, w = moe.route(logits, k, bias=bias, **kw)
    off, tok, slot = moe.group_rows(idx, E)
    n = off[E:]
    xq, xs = moe.quantize_rows_fp8(x, token_of_row=tok)
    gu = moe.matmul_fp8(xq, xs, wgu, sgu, offsets=off)
    hq, hs = moe.glu_quantize_fp8(gu, n_rows=n)
    y = moe.matmul_fp8(hq, hs, wd, sd, offsets=off)
    out = moe.combine_rows(y, slot, w, addend=addend)
    return dict(idx=idx, w=w, off=off, tok=tok, slot=slot, n=n, xq=xq, xs=xs, gu=gu, hq=hq, hs=hs, y=y, out=out)


def _layer_backward(torch, moe, f, dout, logits, Wgu, Wd, kw):
    """Gradients of the tokens and of the logits."""
    (wgu, sgu), (wd, sd) = Wgu, Wd
    dy, dw = moe.combine_rows_backward(dout, f["y"], f["slot"], f["w"])
    dyq, dys = moe.quantize_rows_fp8(dy, n_rows=f["n"])
    dh = moe.matmul_fp8(dyq, dys, wd, sd, offsets=f["off"], transposed=True)
    dgq, dgs = moe.glu_backward_quantize_fp8(f["gu"], dh, n_rows=f["n"])
    dxr = moe.matmul_fp8(dgq, dgs, wgu, sgu, offsets=f["off"], transposed=True, out_dtype=torch.float32)
    dx = moe.combine_rows(dxr, f["slot"])
    return dict(dx=dx, dw=dw, dlogits=moe.route_backward(logits, f["idx"], dw, **kw))


def _layer_inputs(torch, moe, T, D, I, E, seed=0):
    x = _randn(torch, seed + 1, T, D, dtype="bf16")
    logits = _randn(torch, seed + 2, T, E)
    Wgu = moe.quantize_weights_fp8(_randn(torch, seed + 3, E, 2 * I, D, dtype="bf16", scale=D ** -0.5))
    Wd = moe.quantize_weights_fp8(_randn(torch, seed + 4, E, D, I, dtype="bf16", scale=I ** -0.5))
    return x, logits, _randn(torch, seed + 5, E, scale=0.05), Wgu, Wd


KW = dict(scores="sigmoid", n_groups=4, topk_groups=2, group_top=2, renormalize=True, routed_scale=2.5)


def test_layer_and_its_gradients(torch, moe):
    """The whole chain against fp64 with the same E4M3 weights and no quantised
    activations.  A row's codes are off by at most 2^-4 relative, so a stage's
    result moves by at most 2^-4 of its norm for random terms; the forward pass has
    two such stages, the gradients two more."""
    T, D, I, E, k = 96, 256, 128, 16, 4
    x, logits, bias, Wgu, Wd = _layer_inputs(torch, moe, T, D, I, E)
    logits[5] = float("-inf")                    # a padding row
    f = _layer(torch, moe, x, logits, bias, Wgu, Wd, KW, E, k)
    dout = _randn(torch, 9, T, D, dtype="bf16")
    b = _layer_backward(torch, moe, f, dout, logits, Wgu, Wd, KW)
    torch.cuda.synchronize()
    ref_idx, _ = R.route(n64(logits), k, bias=n64(bias), **KW)
    assert np.array_equal(f["idx"].cpu().numpy(), ref_idx)
    assert (f["out"][5] == 0).all() and (b["dx"][5] == 0).all() and (b["dlogits"][5] == 0).all()
    # fp64 with autograd over the same choice.
    xd = x.double().cpu().requires_grad_(True)
    ld = torch.where(torch.isinf(logits), 0.0, logits).double().cpu().requires_grad_(True)
    wgu = torch.from_numpy(R.wide_weights(Wgu[0].cpu().numpy(), Wgu[1].cpu().numpy()))
    wd = torch.from_numpy(R.wide_weights(Wd[0].cpu().numpy(), Wd[1].cpu().numpy()))
    outs = []
    for t in range(T):
        o = torch.zeros(D, dtype=torch.float64)
        if t != 5:
            s = torch.sigmoid(ld[t])[ref_idx[t]]
            w = s / s.sum() * 2.5
            for j, e in enumerate(ref_idx[t]):
                gu = wgu[e] @ xd[t]
                o = o + w[j] * (wd[e] @ (torch.nn.functional.silu(gu[:I]) * gu[I:]))
        outs.append(o)
    ref = torch.stack(outs)
    (ref * dout.double().cpu()).sum().backward()

    def rel(got, want):
        got, want = n64(got), want.detach().numpy()
        return np.linalg.norm(got - want) / np.linalg.norm(want)

    assert rel(f["out"], ref) <= 2 * 2.0 ** -4
    assert rel(b["dx"], xd.grad) <= 4 * 2.0 ** -4
    assert rel(b["dlogits"], ld.grad) <= 4 * 2.0 ** -4


def test_layer_stages_follow_each_other(torch, moe):
    """Every stage against fp64 on the previous stage's own outputs."""
    T, D, I, E, k = 70, 272, 256, 8, 3
    kw = dict(scores="softmax", renormalize=False, routed_scale=1.5)
    x, logits, bias, Wgu, Wd = _layer_inputs(torch, moe, T, D, I, E, seed=40)
    add = _randn(torch, 50, T, D, dtype="bf16")
    f = _layer(torch, moe, x, logits, bias, Wgu, Wd, kw, E, k, addend=add)
    torch.cuda.synchronize()
    assert moe.operator_error() == moe.MOE_OK
    c = {n: v.cpu().numpy() for n, v in f.items() if v.dtype != torch.bfloat16}
    off, tok, slot = R.group_rows(c["idx"], E)
    assert np.array_equal(off, c["off"]) and np.array_equal(tok, c["tok"]) and np.array_equal(slot, c["slot"])
    rq, rs = R.quantize_rows(n64(x)[tok])
    assert np.array_equal(rq, c["xq"]) and np.array_equal(rs, c["xs"])
    wgu, sgu, wd, sd = (v.cpu().numpy() for v in Wgu + Wd)
    ref, mag = R.matmul(c["xq"], c["xs"], wgu, sgu, off)
    assert np.all(np.abs(n64(f["gu"]) - ref) <= 140 * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(ref))
    _check_quantised(c["hq"], c["hs"], R.glu(n64(f["gu"])), I)
    ref, mag = R.matmul(c["hq"], c["hs"], wd, sd, off)
    assert np.all(np.abs(n64(f["y"]) - ref) <= 140 * 2.0 ** -23 * mag + 2.0 ** -8 * np.abs(ref))
    ref = R.combine(n64(f["y"]), slot, c["w"], n64(add))
    mag = R.combine(np.abs(n64(f["y"])), slot, np.abs(c["w"]), np.abs(n64(add)))
    assert np.all(np.abs(n64(f["out"]) - ref) <= 5 * U * mag + 2.0 ** -8 * np.abs(ref))


def test_layer_rows_do_not_depend_on_the_batch(torch, moe):
    T, D, I, E, k = 300, 256, 128, 16, 4
    x, logits, bias, Wgu, Wd = _layer_inputs(torch, moe, T, D, I, E, seed=20)
    dout = _randn(torch, 9, T, D, dtype="bf16")
    f = _layer(torch, moe, x, logits, bias, Wgu, Wd, KW, E, k)
    b = _layer_backward(torch, moe, f, dout, logits, Wgu, Wd, KW)
    for rows in (slice(0, 1), slice(7, 40), slice(250, 300)):
        f2 = _layer(torch, moe, x[rows], logits[rows], bias, Wgu, Wd, KW, E, k)
        b2 = _layer_backward(torch, moe, f2, dout[rows], logits[rows], Wgu, Wd, KW)
        assert torch.equal(f2["out"], f["out"][rows])
        assert torch.equal(b2["dx"], b["dx"][rows]) and torch.equal(b2["dlogits"], b["dlogits"][rows])


def test_layer_captured_replayed_and_on_other_streams(torch, moe):
    """Two captured graphs of the layer with its gradients, replayed in turn with new
    inputs, and two streams at once, give the eager bits."""
    T, D, I, E, k = 64, 256, 128, 16, 4
    sets = []
    for n in range(2):
        x, logits, bias, Wgu, Wd = _layer_inputs(torch, moe, T, D, I, E, seed=60 + 10 * n)
        sets.append((x, logits, bias, Wgu, Wd, _randn(torch, 90 + n, T, D, dtype="bf16")))

    def both(s):
        x, logits, bias, Wgu, Wd, dout = s
        f = _layer(torch, moe, x, logits, bias, Wgu, Wd, KW, E, k)
        b = _layer_backward(torch, moe, f, dout, logits, Wgu, Wd, KW)
        return f["out"], b["dx"], b["dlogits"]

    eager = [both(s) for s in sets]
    torch.cuda.synchronize()
    graphs = []
    for s in sets:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = both(s)
        graphs.append((g, outs))
    for rep in range(2):
        for (g, outs), want in zip(graphs, eager):
            g.replay()
        torch.cuda.synchronize()
        for (g, outs), want in zip(graphs, eager):
            assert all(torch.equal(a, b) for a, b in zip(outs, want))
    # New inputs in the same buffers.
    new = _randn(torch, 777, T, D, dtype="bf16")
    sets[0][0].copy_(new)
    graphs[0][0].replay()
    want = both(sets[0])
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(graphs[0][1], want))
    # Two streams at once.
    streams = [torch.cuda.Stream() for _ in sets]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    results = []
    for _ in range(3):
        for st, s in zip(streams, sets):
            with torch.cuda.stream(st):
                results.append(both(s))
    torch.cuda.synchronize()
    want = [want, eager[1]]
    for i, r in enumerate(results):
        assert all(torch.equal(a, b) for a, b in zip(r, want[i % 2]))


def test_stream_argument(torch, moe):
    st = torch.cuda.Stream()
    x = _randn(torch, 1, 33, 256, dtype="bf16")
    torch.cuda.synchronize()
    q, s = moe.quantize_rows_fp8(x, stream=st)
    q2, s2 = moe.quantize_rows_fp8(x, stream=st.cuda_stream)
    st.synchronize()
    q0, s0 = moe.quantize_rows_fp8(x)
    assert torch.equal(q, q0) and torch.equal(s, s0) and torch.equal(q2, q0) and torch.equal(s2, s0)


def test_binding_refuses(torch, moe):
    x = _randn(torch, 1, 8, 256, dtype="bf16")
    q, s = moe.quantize_rows_fp8(x)
    w, sw = moe.quantize_weights_fp8(_randn(torch, 2, 2, 128, 256, dtype="bf16"))
    i = torch.zeros(8, 2, dtype=torch.int32, device="cuda")
    refused = [
        lambda: moe.matmul_fp8(q, s, w, sw),                              # groups without offsets
        lambda: moe.matmul_fp8(q, s, w[0], sw),                           # scales of another shape
        lambda: moe.matmul_fp8(q, s.t().contiguous(), w[0], sw[0]),
        lambda: moe.matmul_fp8(q[:, :128].contiguous(), s[:1], w[0], sw[0]),
        lambda: moe.matmul_fp8(q, s, w[0], sw[0], transposed=True),
        lambda: moe.matmul_fp8(x, s, w[0], sw[0]),
        lambda: moe.matmul_fp8(q[:, ::2], s, w[0], sw[0]),
        lambda: moe.matmul_fp8(q, s, w[0], sw[0], out_dtype=torch.float16),
        lambda: moe.route(x, 2, scores="relu"),
        lambda: moe.route(x, 2, bias=torch.zeros(4, device="cuda")),
        lambda: moe.route(x.half(), 2),
        lambda: moe.route_backward(x, i.long(), torch.zeros(8, 2, device="cuda")),
        lambda: moe.group_rows(i.long(), 4),
        lambda: moe.quantize_rows_fp8(x.t()),
        lambda: moe.quantize_rows_fp8(x, token_of_row=i),
        lambda: moe.quantize_rows_fp8(x, n_rows=i),
        lambda: moe.glu_quantize_fp8(x.float()),
        lambda: moe.glu_backward_quantize_fp8(x, x),
        lambda: moe.combine_rows(x, i, torch.zeros(8, 3, device="cuda")),
        lambda: moe.combine_rows(x, i, addend=x.float()),
        lambda: moe.combine_rows_backward(x.float(), x, i),
    ]
    for n, call in enumerate(refused):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {n} was not refused")
    for call, status in ((lambda: moe.quantize_rows_fp8(x[:, :250]), moe.MOE_EUNSUPPORTED),
                         (lambda: moe.quantize_rows_fp8(_randn(torch, 1, 8, 260, dtype="bf16")[:, 4:]), moe.MOE_EINVAL),
                         (lambda: moe.route(x, 33), moe.MOE_EUNSUPPORTED),
                         (lambda: moe.combine_rows(x, i, out=torch.empty(8 * 256 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(8, 256)),
                          moe.MOE_EINVAL)):
        with pytest.raises(moe.MoEError) as err:
            call()
        assert err.value.status == status


# Shapes with too few tiles for the device, whose contraction is divided over the
# CTAs of a cluster: both splits (2, 4), runs of unequal length, rows to the last of a
# tile, and shapes just outside.
@pytest.mark.parametrize("M,N,K", [(1, 128, 16), (8, 256, 384), (16, 1000, 1040), (17, 4096, 1152), (33, 130, 2064),
                                   (32, 512, 4096), (30, 384, 1152), (8, 4096, 2048), (5, 8000, 640), (8, 1024, 7168),
                                   (32, 256, 8192), (32, 256, 9216)])
@pytest.mark.parametrize("transposed", [False, True])
def test_matmul_of_few_tiles(torch, moe, M, N, K, transposed):
    N = -(-N // 16) * 16 if transposed else N
    a, sa, w, sw = _operands(torch, moe, M + N + K, M, N, K, transposed=transposed)
    _check_matmul(torch, moe, a, sa, w, sw, transposed=transposed, dtype="f32" if M % 2 else "bf16")


@pytest.mark.parametrize("off", [[0, 3, 3, 20], [2, 2, 18, 30], [0, 0, 0, 0], [0, 30, 30, 30], [0, 64, 129, 130]], ids=str)
def test_matmul_of_few_tiles_grouped(torch, moe, off):
    M = max(off[-1], 1) + 2
    a, sa, w, sw = _operands(torch, moe, M, M, 200, 1168, G=3)
    _check_matmul(torch, moe, a, sa, w, sw, off)


@pytest.mark.parametrize("K", [384, 2064, 7168])
def test_matmul_of_few_tiles_has_the_same_bits(torch, moe, K):
    """Rows alone, in batches whose contraction is divided, and in one that is not."""
    a, sa, w, sw = _operands(torch, moe, 9, 3000, 1024, K)
    whole = moe.matmul_fp8(a, sa, w, sw, out_dtype=torch.float32)
    for lo, hi in ((0, 1), (7, 23), (100, 133), (500, 564), (1000, 1128), (2000, 2300)):
        part = moe.matmul_fp8(a[lo:hi].contiguous(), sa[:, lo:hi].contiguous(), w, sw, out_dtype=torch.float32)
        assert torch.equal(part.view(torch.int32), whole[lo:hi].view(torch.int32)), (lo, hi)
    assert moe.operator_error() == moe.MOE_OK


# ------------------------------------------------ offsets past 32 bits
def _large(torch, rows, cols):
    x = torch.empty(rows, cols, dtype=torch.bfloat16, device="cuda")
    x.normal_(generator=torch.Generator(device="cuda").manual_seed(rows))
    return x


def test_offsets_past_32_bits_in_rows(torch, moe):
    """Rows behind the 2^31st element: the bits of the same rows in a small call."""
    R_, K = 270_000, 8192
    tail = slice(R_ - 200, R_)
    x = _large(torch, R_, K)
    q, s = moe.quantize_rows_fp8(x)
    q2, s2 = moe.quantize_rows_fp8(x[tail])
    assert torch.equal(q[tail], q2) and torch.equal(s[:, tail], s2)
    w, sw = moe.quantize_weights_fp8(_randn(torch, 3, K, K, dtype="bf16"))
    w2, sw2 = w[:, :K // 64].contiguous(), sw[:, :1].contiguous()          # 128 columns: a short contraction
    out = moe.matmul_fp8(q[:, :128].contiguous(), s[:1].contiguous(), w2, sw2, out_dtype=torch.float32)
    want = moe.matmul_fp8(q2[:, :128].contiguous(), s2[:1].contiguous(), w2, sw2, out_dtype=torch.float32)
    assert torch.equal(out[tail], want)
    del out
    out = moe.matmul_fp8(q, s, w[:256].contiguous(), sw[:2].contiguous())
    assert torch.equal(out[tail], moe.matmul_fp8(q2, s2.contiguous(), w[:256].contiguous(), sw[:2].contiguous()))
    del out
    h, hs = moe.glu_quantize_fp8(x)
    h2, hs2 = moe.glu_quantize_fp8(x[tail])
    assert torch.equal(h[tail], h2) and torch.equal(hs[:, tail], hs2)
    del h
    d = _large(torch, 200, K // 2)
    dh = torch.zeros(R_, K // 2, dtype=torch.bfloat16, device="cuda")
    dh[tail] = d
    g, gs = moe.glu_backward_quantize_fp8(x, dh, out_codes=q, out_scales=s)
    g2, gs2 = moe.glu_backward_quantize_fp8(x[tail], d)
    assert torch.equal(g[tail], g2) and torch.equal(gs[:, tail], gs2)
    del dh
    slots = torch.arange(R_ - 200, R_, dtype=torch.int32, device="cuda").view(100, 2)
    wt = torch.rand(100, 2, device="cuda")
    assert torch.equal(moe.combine_rows(x, slots, wt), moe.combine_rows(x[tail], slots - (R_ - 200), wt))
    dout = _large(torch, 100, K)
    dy, dw = moe.combine_rows_backward(dout, x, slots, wt)
    dy2, dw2 = moe.combine_rows_backward(dout, x[tail], slots - (R_ - 200), wt)
    assert torch.equal(dy[tail], dy2) and torch.equal(dw, dw2)
    assert moe.operator_error("cuda") == moe.MOE_OK


def test_offsets_past_32_bits_in_weights_and_logits(torch, moe):
    G, N, K = 9, 16384, 16384
    w = torch.empty(G, N, K, dtype=torch.bfloat16, device="cuda")
    w.normal_(generator=torch.Generator(device="cuda").manual_seed(5))
    q, s = moe.quantize_weights_fp8(w)
    last, slast = moe.quantize_weights_fp8(w[-1])
    assert torch.equal(q[-1], last) and torch.equal(s[-1], slast)
    del w
    a, sa = moe.quantize_rows_fp8(_randn(torch, 1, 20, K, dtype="bf16"))
    off = torch.tensor([0] * G + [20], dtype=torch.int32, device="cuda")
    for transposed in (False, True):
        assert torch.equal(moe.matmul_fp8(a, sa, q, s, offsets=off, transposed=transposed),
                           moe.matmul_fp8(a, sa, last, slast, transposed=transposed))
    del q
    T, E, k = 2_200_000, 1024, 4
    logits = _large(torch, T, E)
    tail = slice(T - 100, T)
    idx, wt = moe.route(logits, k, renormalize=True)
    idx2, wt2 = moe.route(logits[tail], k, renormalize=True)
    assert torch.equal(idx[tail], idx2) and torch.equal(wt[tail], wt2)
    dl = moe.route_backward(logits, idx, wt)
    assert torch.equal(dl[tail], moe.route_backward(logits[tail], idx2, wt2))


def test_products_on_two_streams_at_once(torch, moe):
    """Products that divide a contraction over clusters beside ones of whole tiles."""
    few = _operands(torch, moe, 1, 8, 2048, 4096)
    many = _operands(torch, moe, 2, 700, 2048, 1024)
    want = [moe.matmul_fp8(*few), moe.matmul_fp8(*many)]
    streams = [torch.cuda.Stream() for _ in range(3)]
    torch.cuda.synchronize()
    got = []
    for i in range(60):
        with torch.cuda.stream(streams[i % 3]):
            got.append(moe.matmul_fp8(*(few if i % 2 == 0 else many)))
    torch.cuda.synchronize()
    assert moe.operator_error() == moe.MOE_OK
    assert all(torch.equal(g, want[i % 2]) for i, g in enumerate(got))
