"""Norms and joins whose workgroups stride over several blocks of rows, on the GPU against the float64
oracle: the loads ahead of the next row, the LDS that a row's sums share with the rows around it, weight
gradients of many rows per lane and of many workgroups. And rows whose last elements, which two vectors
hold, are the ones that count."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.block_oracle import gated_norm_ref, join_ref
from test_ridge_regression_amd import block, gka

from gka_testutil import log

pytestmark = pytest.mark.gpu

EPS = 1e-5
TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gka.load()


def num(t):
    return t.detach().double().cpu().numpy()


def rand(seed, shape, dtype, mean=0.0, sd=1.0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn(*shape, device="cuda", generator=g) * sd + mean).to(TORCH[dtype])


def check(got, ref, what):
    for name, t in got.items():
        if t is None:
            continue
        value, bound = ref[name]
        g, tol = num(t), HALF_ULP[t.dtype] * (np.abs(value) + bound) + bound + 1e-37
        assert g.shape == value.shape and np.isfinite(g).all(), (what, name)
        off = np.abs(g - value) / tol
        assert off.max() <= 1.0, (what, name, np.unravel_index(np.argmax(off), off.shape), off.max())


def blocks_of(kind, rows, H, D, dtype):
    """(workgroups, blocks of rows that the busiest of them takes) by the plan's rule."""
    elem = 2 if dtype == "bf16" else 4
    bwd = kind.endswith("bwd")
    vec = 4 if kind == "join_bwd" else 16 // elem
    vec = 1 if D < vec else vec
    n = -(-D // vec)
    nv = 2 if n > (1024 if bwd else 64) else 1
    team, nt = 1, 256
    if n <= 64 * nv:
        while team * nv < n:
            team *= 2
    else:
        team, nt = 0, -(-n // (64 * nv)) * 64
    teams = nt // team if team else 1
    nhb = -(-H // teams)
    hp = -(-H // nhb)
    tt = teams // hp
    if bwd:
        top = 256 * max(1, (20 if kind == "join_bwd" and team else 16) * 64 // nt)
    else:
        top = 4096 if kind == "norm" and elem == 2 and nv == 1 else 16384
    ntb = max(1, min(-(-rows // tt), max(1, top // nhb)))
    return ntb * nhb, -(-rows // (ntb * tt)), ntb


def assert_loops(kind, rows, H, D, dtype, per_head=False):
    workgroups, loops, ntb = blocks_of(kind, rows, H, D, dtype)
    assert loops >= 2, (kind, rows, H, D, "one block of rows per workgroup")
    code = {"bf16": 0, "fp32": 1}[dtype]
    if kind == "norm_bwd":  # the partial rows in the workspace are the plan's workgroups
        p = gka.GkaGatedNormParams(rows, H, D, int(per_head), 0, code, EPS, H * D, H * D)
        parts = ntb * H * D if per_head else workgroups * D
        need = gka.load().gka_gated_norm_bwd_workspace_bytes(ctypes.byref(p))
    elif kind == "join_bwd":
        p = gka.GkaJoinParams(rows, D, 0, code, code, EPS, 1.0, D, D, D)
        parts = ntb * 3 * D
        need = gka.load().gka_join_bwd_workspace_bytes(ctypes.byref(p))
    else:
        return workgroups
    assert need == -(-parts * 4 // 256) * 256, "the plan has another rule"
    return workgroups


# a team of 16, 32 or 64 lanes per row; a workgroup per row, one and two vectors per lane; ragged ends
JOIN_BWD = [(45007, 64), (23003, 100), (12001, 250), (2100, 333), (1500, 1001), (700, 2049), (600, 4096),
            (400, 5120), (400, 8191)]


@pytest.mark.parametrize("dtype,res_dtype", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("rows,C", JOIN_BWD)
def test_join_backward_over_blocks_of_rows(rows, C, dtype, res_dtype):
    log(f"join backward rows {rows}x{C} {dtype}/{res_dtype}")
    assert assert_loops("join_bwd", rows, 1, C, dtype) >= 256
    run_join_bwd(rows, C, dtype, res_dtype, "gpsn")


@pytest.mark.parametrize("present", ["gsn", "gps", "psn", "p", "n", "s", "g"])
@pytest.mark.parametrize("rows,C,dtype,res_dtype", [(700, 2049, "bf16", "fp32"), (700, 1537, "fp32", "fp32"),
                                                    (300, 8191, "bf16", "bf16"), (12001, 250, "bf16", "fp32")])
def test_join_backward_parts_over_blocks_of_rows(rows, C, dtype, res_dtype, present):
    log(f"join backward parts {rows}x{C} {dtype}/{res_dtype} {present}")
    assert_loops("join_bwd", rows, 1, C, dtype)
    run_join_bwd(rows, C, dtype, res_dtype, present)


def run_join_bwd(rows, C, dtype, res_dtype, present):
    res, y, g = rand(1, (rows, C), res_dtype, sd=2.0), rand(2, (rows, C), dtype), rand(3, (rows, C), dtype)
    w = {n: rand(4 + i, (C,), "fp32", 1.0, 0.3) if k in present else None
         for i, (k, n) in enumerate((("p", "w_post"), ("s", "scale"), ("n", "w_pre")))}
    dres, dn = rand(8, (rows, C), res_dtype), rand(9, (rows, C), dtype) if "n" in present else None
    gate = g if "g" in present else None
    got = block.join_bwd(res, y, dres, dn, gate=gate, **w, alpha=0.7, eps=EPS)._asdict()
    opt = lambda t: None if t is None else num(t)
    ref = join_ref(num(res), num(y), opt(gate), *(opt(w[k]) for k in ("w_post", "scale", "w_pre")), 0.7,
                   EPS, "silu", num(dres), opt(dn))
    check(got, ref, f"{rows}x{C} {dtype}/{res_dtype} {present}")


NORM_BWD = [(2500, 8, 128), (3401, 5, 77), (11003, 3, 64), (1501, 17, 128), (90001, 1, 24), (2100, 1, 1000),
            (2100, 1, 513), (600, 1, 4096), (200, 2, 8192), (400, 1, 8191)]


@pytest.mark.parametrize("per_head", [False, True])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("rows,H,D", NORM_BWD)
def test_gated_norm_backward_over_blocks_of_rows(rows, H, D, dtype, per_head):
    log(f"norm backward rows {rows}x{H}x{D} {dtype} {per_head}")
    assert_loops("norm_bwd", rows, H, D, dtype, per_head)
    x, gate, dy = (rand(k, (rows, H, D), dtype) for k in (11, 12, 13))
    w = rand(14, (H, D) if per_head else (D,), "fp32", 1.0, 0.3)
    dx, dg, dw = block.gated_norm_bwd(x, gate, w, dy, EPS, "silu")
    ref = gated_norm_ref(num(x), num(gate), num(w), EPS, "silu", num(dy))
    check({"dx": dx, "dgate": dg, "dweight": dw}, ref, f"{rows}x{H}x{D} {dtype}")


def some_rows(rows):
    """First and last rows, and some of every part: rows do not see each other in the forward."""
    rng = np.random.default_rng(rows)
    return np.unique(np.concatenate([np.arange(20), np.arange(rows - 20, rows), rng.integers(0, rows, 160)]))


@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("rows,C,dtype,res_dtype", [
    (33001, 1033, "bf16", "bf16"), (20003, 2049, "bf16", "fp32"), (17001, 1040, "fp32", "fp32"),
    (66001, 520, "bf16", "fp32"), (140003, 130, "fp32", "fp32")])
def test_join_over_blocks_of_rows(rows, C, dtype, res_dtype, post, pre):
    log(f"join rows {rows}x{C} {dtype}/{res_dtype} {post} {pre}")
    assert_loops("join", rows, 1, C, dtype)
    res, y, g = rand(21, (rows, C), res_dtype, sd=2.0), rand(22, (rows, C), dtype), rand(23, (rows, C), dtype)
    wp, sc, wn = (rand(k, (C,), "fp32", 1.0, 0.3) for k in (24, 25, 26))
    wp, wn = wp if post else None, wn if pre else None
    out, n = block.join(res, y, g, wp, sc, wn, 0.7, EPS)
    k = some_rows(rows)
    at = torch.from_numpy(k).cuda()
    opt = lambda t: None if t is None else num(t)
    ref = join_ref(num(res[at]), num(y[at]), num(g[at]), opt(wp), num(sc), opt(wn), 0.7, EPS, "silu")
    check({"res_out": out[at], "n": None if n is None else n[at]}, ref, f"{rows}x{C}")
    # every row: the same call on the rows in another order
    flip = lambda t: t.flip(0).contiguous()
    out2, n2 = block.join(flip(res), flip(y), flip(g), wp, sc, wn, 0.7, EPS)
    assert torch.equal(flip(out2), out) and (n is None or torch.equal(flip(n2), n))


@pytest.mark.parametrize("rows,H,D,dtype", [
    (40001, 1, 512, "bf16"), (40001, 4, 128, "bf16"), (33001, 1, 1033, "bf16"), (17001, 1, 520, "fp32"),
    (70001, 1, 200, "fp32"), (5001, 4, 1040, "bf16")])
def test_gated_norm_over_blocks_of_rows(rows, H, D, dtype):
    log(f"norm rows {rows}x{H}x{D} {dtype}")
    assert_loops("norm", rows, H, D, dtype)
    x, g, w = rand(31, (rows, H, D), dtype), rand(32, (rows, H, D), dtype), rand(33, (D,), "fp32", 1.0, 0.3)
    y = block.gated_norm(x, g, w, EPS)
    at = torch.from_numpy(some_rows(rows)).cuda()
    check({"y": y[at]}, gated_norm_ref(num(x[at]), num(g[at]), num(w), EPS, "silu"), f"{rows}x{H}x{D}")
    y2 = block.gated_norm(x.flip(0).contiguous(), g.flip(0).contiguous(), w, EPS)
    assert torch.equal(y2.flip(0), y)


def heavy_tail(t):
    """The last elements 30 times the others: those that the last vector shares with the one before."""
    t = t.clone()
    t[..., -8:] *= 30.0
    return t


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("D", [9, 13, 31, 77, 127, 250, 513, 1001, 2049, 4001, 8189, 8190, 8191])
def test_shared_elements_count_once(D, dtype):
    log(f"heavy tail {D} {dtype}")
    x, dy, r = (heavy_tail(rand(k, (6, 1, D), dtype)) for k in (41, 42, 43))
    w = rand(44, (D,), "fp32", 1.0, 0.3)
    ref = gated_norm_ref(num(x), None, num(w), EPS, "silu", num(dy))
    dx, _, dw = block.gated_norm_bwd(x, None, w, dy, EPS)
    check({"y": block.gated_norm(x, None, w, EPS), "dx": dx, "dweight": dw}, ref, f"norm {D}")
    x, dy, r = x[:, 0].contiguous(), dy[:, 0].contiguous(), r[:, 0].contiguous()
    ref = join_ref(num(r), num(x), None, num(w), num(w), num(w), 0.7, EPS, "silu", num(dy), num(x))
    out, n = block.join(r, x, None, w, w, w, 0.7, EPS)
    grads = block.join_bwd(r, x, dy, x, w_post=w, scale=w, w_pre=w, alpha=0.7, eps=EPS)._asdict()
    check({"res_out": out, "n": n, **grads}, ref, f"join {D}")
