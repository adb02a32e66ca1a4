"""The handle-free operators without a GPU: what the entry points and the binding
refuse, the binding against the header, and the fp64 statements the GPU tests
compare with against worked values, differences and each other."""
import ctypes
import re

import numpy as np
import pytest
import torch

import deterministic_expert_b200 as moe
import operators_ref as R
from deterministic_expert_b200 import operators as ops

FAKE = 1 << 20   # an aligned address; never read: every call here is refused first


def _cfg(**kw):
    c = dict(E=64, k=6, scores=0, n_groups=1, topk_groups=1, group_top=1, renormalize=1, routed_scale=1.0,
             logits_dtype=1)
    c.update(kw)
    return ops.moe_route_config(*c.values())


def _route(cfg, T=4, logits=FAKE, ld=64, bias=None, idx=FAKE, w=FAKE):
    return ops._fn("moe_route")(ctypes.byref(cfg) if cfg is not None else None, T, logits, ld, bias, idx, w, None)


@pytest.mark.parametrize("kw,status", [
    (dict(E=0), moe.MOE_EINVAL), (dict(E=1025), moe.MOE_EUNSUPPORTED), (dict(k=0), moe.MOE_EINVAL),
    (dict(k=33), moe.MOE_EUNSUPPORTED), (dict(E=4, k=5), moe.MOE_EUNSUPPORTED), (dict(scores=2), moe.MOE_EINVAL),
    (dict(n_groups=0), moe.MOE_EINVAL), (dict(n_groups=3, topk_groups=1), moe.MOE_EUNSUPPORTED),
    (dict(n_groups=64, topk_groups=8), moe.MOE_EUNSUPPORTED), (dict(n_groups=8, topk_groups=9), moe.MOE_EINVAL),
    (dict(topk_groups=0), moe.MOE_EINVAL), (dict(group_top=3), moe.MOE_EINVAL), (dict(logits_dtype=2), moe.MOE_EINVAL),
    (dict(routed_scale=float("nan")), moe.MOE_EINVAL),
    # 5 groups of 200 have 4 lanes each: 50 experts a lane
    (dict(E=1000, n_groups=5, topk_groups=2), moe.MOE_EUNSUPPORTED),
])
def test_route_refuses_bad_configs(kw, status):
    assert _route(_cfg(**kw), ld=2048) == status


def test_route_refuses_bad_arguments():
    ok = _cfg()
    assert _route(None) == moe.MOE_EINVAL
    assert _route(ok, T=-1) == moe.MOE_EINVAL
    for kw in (dict(logits=None), dict(idx=None), dict(w=None), dict(ld=63), dict(logits=FAKE + 2), dict(idx=FAKE + 1)):
        assert _route(ok, **kw) == moe.MOE_EINVAL, kw
    assert _route(ok, T=0, logits=None, idx=None, w=None) == moe.MOE_OK
    back = ops._fn("moe_route_backward")
    assert back(ctypes.byref(ok), 4, FAKE, 64, None, FAKE, FAKE, 64, None) == moe.MOE_EINVAL
    assert back(ctypes.byref(ok), 4, FAKE, 64, FAKE, FAKE, FAKE, 63, None) == moe.MOE_EINVAL
    assert back(ctypes.byref(ok), 0, None, 64, None, None, None, 64, None) == moe.MOE_OK


def test_group_rows_refuses():
    f = ops._fn("moe_group_rows")
    assert f(-1, 2, 8, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(4, 0, 8, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(4, 2, 0, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(4, 2, 1025, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_EUNSUPPORTED
    assert f(1 << 30, 2, 8, FAKE, FAKE, FAKE, FAKE, None) == moe.MOE_EUNSUPPORTED
    assert f(4, 2, 8, None, FAKE, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert f(4, 2, 8, FAKE, None, FAKE, FAKE, None) == moe.MOE_EINVAL


def test_quantisers_refuse():
    f = ops._fn("moe_quantize_rows_fp8")

    def rows(n=4, K=256, x=FAKE, dt=0, ld=256, src=4, codes=FAKE, scales=FAKE, ld_s=4):
        return f(n, K, x, dt, ld, src, None, None, codes, scales, ld_s, None)

    for kw in (dict(n=-1), dict(K=0), dict(x=None), dict(dt=2), dict(ld=255), dict(ld=260), dict(x=FAKE + 8),
               dict(codes=None), dict(codes=FAKE + 8), dict(scales=None), dict(ld_s=3)):
        assert rows(**kw) == moe.MOE_EINVAL, kw
    assert rows(K=120, ld=256) == moe.MOE_EUNSUPPORTED
    assert rows(n=0, x=None) == moe.MOE_OK
    g = ops._fn("moe_quantize_weights_fp8")
    assert g(1, 0, 128, FAKE, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert g(1, 128, 120, FAKE, FAKE, FAKE, None) == moe.MOE_EUNSUPPORTED
    assert g(70000, 128, 128, FAKE, FAKE, FAKE, None) == moe.MOE_EUNSUPPORTED
    assert g(1, 128, 128, None, FAKE, FAKE, None) == moe.MOE_EINVAL
    u, b = ops._fn("moe_glu_quantize_fp8"), ops._fn("moe_glu_backward_quantize_fp8")
    inf = float("inf")
    good = ops.moe_glu_config(0, inf, inf, 4.0, 25.0)
    for cfg in (ops.moe_glu_config(2, inf, inf, 4, 25), ops.moe_glu_config(0, float("nan"), inf, 4, 25),
                ops.moe_glu_config(0, inf, -1.0, 4, 25), ops.moe_glu_config(1, inf, inf, 0.0, 25),
                ops.moe_glu_config(1, inf, inf, 4, inf)):
        assert u(ctypes.byref(cfg), 4, 128, FAKE, 256, None, FAKE, FAKE, 4, None) == moe.MOE_EINVAL
    assert u(None, 4, 128, FAKE, 256, None, FAKE, FAKE, 4, None) == moe.MOE_EINVAL
    assert u(ctypes.byref(good), 4, 128, FAKE, 255, None, FAKE, FAKE, 4, None) == moe.MOE_EINVAL
    assert u(ctypes.byref(good), 4, 100, FAKE, 256, None, FAKE, FAKE, 4, None) == moe.MOE_EUNSUPPORTED
    assert b(ctypes.byref(good), 4, 64, FAKE, 256, FAKE, 64, None, FAKE, FAKE, 4, None) == moe.MOE_EUNSUPPORTED
    assert b(ctypes.byref(good), 4, 128, FAKE, 256, None, 128, None, FAKE, FAKE, 4, None) == moe.MOE_EINVAL
    assert b(ctypes.byref(good), 4, 128, FAKE, 256, FAKE, 127, None, FAKE, FAKE, 4, None) == moe.MOE_EINVAL


def test_matmul_refuses():
    f = ops._fn("moe_matmul_fp8")

    def mm(t=0, G=1, off=None, M=4, N=64, K=128, a=FAKE, sa=FAKE, ld_as=4, w=FAKE, sw=FAKE, out=FAKE, dt=0, ldo=128):
        return f(t, G, off, M, N, K, a, sa, ld_as, w, sw, out, dt, ldo, None)

    for kw in (dict(t=2), dict(G=0), dict(G=2), dict(M=-1), dict(N=0), dict(K=0), dict(dt=3), dict(a=None),
               dict(sa=None), dict(w=None), dict(sw=None), dict(out=None), dict(ld_as=3), dict(ldo=63),
               dict(a=FAKE + 8), dict(w=FAKE + 8), dict(out=FAKE + 1), dict(t=1, ldo=127)):
        assert mm(**kw) == moe.MOE_EINVAL, kw
    for kw in (dict(K=120), dict(t=1, N=72), dict(G=1025, off=FAKE), dict(M=(1 << 31) - 2)):
        assert mm(**kw) == moe.MOE_EUNSUPPORTED, kw
    assert mm(M=0, a=None) == moe.MOE_OK


def test_sizes_that_pass_32_bits_are_refused():
    most, no = (1 << 31) - 257, moe.MOE_EUNSUPPORTED
    cfg = _cfg(k=1)
    assert _route(cfg, T=most + 1) == no and _route(_cfg(k=2), T=most) == no
    assert ops._fn("moe_route_backward")(ctypes.byref(cfg), most + 1, FAKE, 64, FAKE, FAKE, FAKE, 64, None) == no
    assert ops._fn("moe_group_rows")(most + 1, 1, 8, FAKE, FAKE, FAKE, FAKE, None) == no
    q = ops._fn("moe_quantize_rows_fp8")
    assert q(most + 1, 128, FAKE, 0, 128, 4, None, None, FAKE, FAKE, most + 1, None) == no
    assert q(4, (1 << 20) + 16, FAKE, 0, 1 << 21, 4, None, None, FAKE, FAKE, 4, None) == no
    w = ops._fn("moe_quantize_weights_fp8")
    assert w(1, (1 << 31) - 1, 128, FAKE, FAKE, FAKE, None) == no
    assert w(1, 128, (1 << 31) - 16, FAKE, FAKE, FAKE, None) == no
    inf = float("inf")
    glu = ops.moe_glu_config(0, inf, inf, 4.0, 25.0)
    assert ops._fn("moe_glu_quantize_fp8")(ctypes.byref(glu), most + 1, 128, FAKE, 256, None, FAKE, FAKE, most + 1,
                                           None) == no
    glu.gate_clamp_max = -inf          # would clamp every gate away
    assert ops._fn("moe_glu_quantize_fp8")(ctypes.byref(glu), 4, 128, FAKE, 256, None, FAKE, FAKE, 4,
                                           None) == moe.MOE_EINVAL
    mm = ops._fn("moe_matmul_fp8")
    for M, N, K, G in ((1 << 28, 1 << 28, 16, 1), (1 << 24, 1 << 20, 128, 1024), (most, most, 16, 1), (4, most + 1, 16, 1)):
        assert mm(0, G, FAKE, M, N, K, FAKE, FAKE, M, FAKE, FAKE, FAKE, 0, N, None) == no, (M, N, K, G)
    assert ops._fn("moe_combine_rows")(most + 1, 1, 64, 8, FAKE, 0, 64, FAKE, None, None, FAKE, 0, None) == no
    assert ops._fn("moe_combine_rows")(4, 1, 64, most + 1, FAKE, 0, 64, FAKE, None, None, FAKE, 0, None) == no
    assert ops._fn("moe_combine_rows_backward")(most + 1, 1, 64, 8, FAKE, FAKE, 0, 64, FAKE, None, FAKE, FAKE,
                                                None) == no


def test_configurations_are_kept_by_value():
    scale, bound = torch.tensor(1.5), torch.tensor(7.0)
    first = ops._route_config(8, 2, torch.float32, "sigmoid", 1, 1, 2, False, scale).routed_scale
    clamp = ops._glu_config(0, bound, bound, 4.0, 25.0).up_clamp
    scale.fill_(2.5)
    bound.fill_(3.0)
    assert first == 1.5 and clamp == 7.0
    assert ops._route_config(8, 2, torch.float32, "sigmoid", 1, 1, 2, False, scale).routed_scale == 2.5
    assert ops._glu_config(0, bound, bound, 4.0, 25.0).up_clamp == 3.0


def test_combine_refuses():
    f, b = ops._fn("moe_combine_rows"), ops._fn("moe_combine_rows_backward")

    def fwd(T=4, k=2, D=64, rows=8, y=FAKE, dt=0, ld=64, slots=FAKE, out=FAKE, odt=0):
        return f(T, k, D, rows, y, dt, ld, slots, None, None, out, odt, None)

    for kw in (dict(T=-1), dict(k=0), dict(D=0), dict(rows=-1), dict(y=None), dict(dt=2), dict(odt=2), dict(ld=56),
               dict(ld=68), dict(slots=None), dict(out=None), dict(y=FAKE + 8), dict(out=FAKE + 8)):
        assert fwd(**kw) == moe.MOE_EINVAL, kw
    assert fwd(D=60) == moe.MOE_EUNSUPPORTED and fwd(k=33) == moe.MOE_EUNSUPPORTED
    assert fwd(T=0, y=None) == moe.MOE_OK
    assert b(4, 2, 64, 8, None, FAKE, 0, 64, FAKE, None, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert b(4, 2, 64, 8, FAKE, None, 0, 64, FAKE, None, FAKE, FAKE, None) == moe.MOE_EINVAL
    assert b(4, 2, 64, 8, FAKE, FAKE, 0, 64, FAKE, None, None, FAKE, None) == moe.MOE_EINVAL


def test_matmul_self_test_refuses():
    f = ops._fn("moe_selftest_matmul_timeout")
    for args in ((0, 128, 128, 1), (9000, 128, 128, 1), (8, 0, 128, 1), (8, 128, 0, 1), (8, 128, 9000, 1), (8, 128, 128, -1)):
        assert f(*args, None) == moe.MOE_EINVAL, args
    assert f(8, 128, 120, 1, None) == moe.MOE_EUNSUPPORTED


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    c = torch.zeros(4, 128, dtype=torch.uint8)
    s = torch.zeros(1, 4)
    for call in (lambda: moe.route(x, 2), lambda: moe.route_backward(x, i, s), lambda: moe.group_rows(i, 4),
                 lambda: moe.quantize_rows_fp8(x), lambda: moe.quantize_weights_fp8(x),
                 lambda: moe.glu_quantize_fp8(x), lambda: moe.glu_backward_quantize_fp8(x, x),
                 lambda: moe.matmul_fp8(c, s, c, s), lambda: moe.combine_rows(x, i),
                 lambda: moe.combine_rows_backward(x, x, i)):
        with pytest.raises(ValueError):
            call()


def test_binding_refuses_tensors_whose_gradient_it_would_drop():
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    i = torch.zeros(4, 2, dtype=torch.int32)
    c = torch.zeros(4, 128, dtype=torch.uint8)
    s, g = torch.zeros(1, 4), torch.zeros(4, 2)
    xg, sg, gg = (t.clone().requires_grad_() for t in (x, s, g))
    calls = (lambda x, s, g: moe.route(x, 2), lambda x, s, g: moe.route_backward(x, i, g),
             lambda x, s, g: moe.quantize_rows_fp8(x), lambda x, s, g: moe.quantize_weights_fp8(x),
             lambda x, s, g: moe.glu_quantize_fp8(x), lambda x, s, g: moe.glu_backward_quantize_fp8(x, x),
             lambda x, s, g: moe.combine_rows(x, i, g), lambda x, s, g: moe.combine_rows_backward(x, x, i, g))
    for n, call in enumerate(calls):
        with pytest.raises(ValueError, match="gradient"):
            call(xg, sg, gg)
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):      # refused as host tensors only
            call(xg, sg, gg)
        with pytest.raises(ValueError, match="CUDA"):
            call(xg.detach(), sg.detach(), gg.detach())


def test_operators_are_reached_through_the_package():
    for n in moe.OPERATORS:
        assert callable(getattr(moe, n))
    with pytest.raises(AttributeError):
        moe.no_such_operator


def test_binding_matches_the_header():
    with open(moe.HEADER_PATH) as f:
        hdr = re.sub(r"/\*.*?\*/", "", f.read(), flags=re.S)
    for name, args in ops.ARGTYPES.items():
        m = re.search(r"int\s+" + name + r"\s*\(([^;]*?)\)\s*;", hdr, flags=re.S)
        decl = [p.strip() for p in m.group(1).split(",")]
        assert len(decl) == len(args), name
        for d, t in zip(decl, args):
            want = (ctypes.c_longlong if d.startswith("long long") else
                    ctypes.c_int if re.match(r"int \w+$", d) else None)
            assert want is None or t is want, (name, d)


def test_config_structs_match_the_c_layout(tmp_path):
    import os
    import shutil
    import subprocess
    if shutil.which("gcc") is None:
        pytest.skip("no C compiler")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "moe.h"', "int main(void) {"]
    structs = {"moe_route_config": ops.moe_route_config, "moe_glu_config": ops.moe_glu_config}
    for n, ct in structs.items():
        lines.append(f'  printf("%zu", sizeof({n}));')
        lines += [f'  printf(" %zu", offsetof({n}, {f}));' for f, _ in ct._fields_]
        lines.append('  printf("\\n");')
    src = tmp_path / "l.c"
    src.write_text("\n".join(lines + ["  return 0;", "}"]))
    exe = tmp_path / "l"
    subprocess.check_call(["gcc", "-std=c99", "-Wall", "-Werror", "-I", os.path.dirname(moe.HEADER_PATH), str(src),
                           "-o", str(exe)])
    out = subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.strip().split("\n")
    for line, ct in zip(out, structs.values()):
        got = [int(v) for v in line.split()]
        assert got == [ctypes.sizeof(ct)] + [getattr(ct, f).offset for f, _ in ct._fields_]


# ------------------------------------------------- the fp64 statements
def test_e4m3_grid_and_rounding():
    assert len(R.GRID) == 127 and R.GRID[-1] == 448 and R.GRID[8] == 2.0 ** -6 and R.GRID[1] == 2.0 ** -9
    v = torch.arange(256, dtype=torch.uint8)
    want = v.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(R.code_values(v.numpy()), want, equal_nan=True)
    # Middles go to the even code; values past 448 saturate.
    assert list(R.round_e4m3([1.0625, 1.1875, 2.0 ** -10, 3 * 2.0 ** -10, 500.0, -0.0])) == \
        [0x38, 0x3A, 0x00, 0x02, 0x7E, 0x80]


def test_quantisation_error_is_half_a_step():
    """|code * s - x| <= 2^-4 |x| (half of E4M3's 2^-3 steps), or half of the
    smallest step times s."""
    x = np.random.default_rng(1).standard_normal((5, 300))
    c, s = R.quantize_rows(x)
    err = np.abs(R.wide_rows(c, s) - x)
    small = np.repeat(s.T.astype(np.float64), 128, axis=1)[:, :300] * 2.0 ** -10
    assert (err <= np.maximum(2.0 ** -4 * np.abs(x), small) * (1 + 1e-6)).all()
    assert s[0, 0] == np.float32(np.abs(x[0, :128]).max() / 448)


def test_route_worked_example():
    # Two groups of two: key sums 0.9 + 0.1 and 0.6 + 0.5, so the second group stays.
    l = np.log(np.array([[0.9, 0.1, 0.6, 0.5]]) / (1 - np.array([[0.9, 0.1, 0.6, 0.5]])))
    idx, w = R.route(l, 2, "sigmoid", n_groups=2, topk_groups=1, group_top=2, renormalize=True, routed_scale=2.0)
    assert idx.tolist() == [[2, 3]] and np.allclose(w, [[2 * 0.6 / 1.1, 2 * 0.5 / 1.1]])
    idx, _ = R.route(l, 2, "sigmoid", n_groups=2, topk_groups=1, group_top=1)
    assert idx.tolist() == [[0, 1]]
    # The bias selects and does not weigh.
    idx, w = R.route(l, 1, "sigmoid", bias=np.array([0, 1.0, 0, 0]))
    assert idx.tolist() == [[1]] and np.allclose(w, 0.1)


@pytest.mark.parametrize("scores", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_route_gradient_against_differences(scores, renorm):
    rng = np.random.default_rng(3)
    l, dw = rng.standard_normal((3, 9)), rng.standard_normal((3, 4))
    idx, _ = R.route(l, 4, scores)
    got = R.route_backward(l, idx, dw, scores, renorm, 1.7)
    h = 1e-6
    for t in range(3):
        for e in range(9):
            up, dn = l[t].copy(), l[t].copy()
            up[e] += h
            dn[e] -= h
            d = (R.weights_of(up, idx[t], scores, renorm, 1.7) - R.weights_of(dn, idx[t], scores, renorm, 1.7)) @ dw[t]
            assert abs(d / (2 * h) - got[t, e]) < 1e-8


@pytest.mark.parametrize("act,cg,cu", [("swiglu", np.inf, np.inf), ("swiglu", 0.7, 0.9), ("situ", 0, 0)])
def test_glu_gradient_against_differences(act, cg, cu):
    rng = np.random.default_rng(4)
    gu, dh = rng.standard_normal((2, 16)), rng.standard_normal((2, 8))
    got = R.glu_backward(gu, dh, act, cg, cu)
    h = 1e-6
    for t in range(2):
        for c in range(16):
            up, dn = gu.copy(), gu.copy()
            up[t, c] += h
            dn[t, c] -= h
            d = ((R.glu(up, act, cg, cu) - R.glu(dn, act, cg, cu)) * dh).sum() / (2 * h)
            assert abs(d - got[t, c]) < 1e-8


def test_group_rows_worked_example():
    off, tok, slot = R.group_rows(np.array([[2, 0], [0, -1], [2, 1]], np.int32), 3)
    assert off.tolist() == [0, 2, 3, 5]
    assert tok.tolist() == [0, 1, 2, 0, 2, -1]
    assert slot.tolist() == [[3, 0], [1, -1], [4, 2]]
