"""The block operators' C ABI without a GPU: every refusal happens on the host before anything is
enqueued (the addresses below are never dereferenced), sizes of workspaces and carries, and the same
checks under AddressSanitizer and UndefinedBehaviorSanitizer."""
import ctypes
import os
import subprocess
import sys

import pytest

from test_ridge_regression_amd import build, gka

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CLANG = "/opt/rocm/llvm/bin/clang"
ADDR = [0x7F0000000000 + i * (1 << 40) for i in range(20)]
V = [ctypes.c_void_p(a) for a in ADDR]


def at(i, off):
    return ctypes.c_void_p(ADDR[i] + off)


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gka.LIB_PATH):
        build.build_library()
    return gka.load()


def norm(**kw):
    d = dict(rows=4, H=2, D=64, per_head=0, act=0, dtype=0, eps=1e-6, x_stride=128,
             gate_stride=128)
    d.update(kw)
    return ctypes.byref(gka.GkaGatedNormParams(*d.values()))


def join(**kw):
    d = dict(rows=4, C=64, act=0, dtype=0, res_dtype=0, eps=1e-6, alpha=1.0, res_stride=64,
             y_stride=64, gate_stride=64)
    d.update(kw)
    return ctypes.byref(gka.GkaJoinParams(*d.values()))


def recur(**kw):
    d = dict(B=2, T=300, C=64, complement=1, dtype=0, xb=300 * 64, xt=64, fb=300 * 64, ft=64)
    d.update(kw)
    return ctypes.byref(gka.GkaRecurParams(*d.values()))


BIG = 1 << 41
BAD_NORM = [(dict(dtype=2), 4), (dict(rows=-1), 2), (dict(H=0), 2), (dict(D=0), 2),
            (dict(D=8193, x_stride=BIG, gate_stride=BIG), 2), (dict(per_head=2), 2),
            (dict(H=1 << 10, D=8192, x_stride=1 << 23, gate_stride=1 << 23), 2),
            (dict(rows=1 << 40), 2), (dict(x_stride=127), 2), (dict(gate_stride=0), 2),
            (dict(x_stride=-128), 2), (dict(x_stride=BIG), 2), (dict(rows=1 << 30, x_stride=1 << 32), 2),
            (dict(eps=0.0), 3), (dict(eps=-1.0), 3), (dict(eps=float("inf")), 3),
            (dict(eps=float("nan")), 3), (dict(eps=1e-42), 3), (dict(act=2), 3), (dict(act=-1), 3)]


@pytest.mark.parametrize("kw,code", BAD_NORM)
def test_gated_norm_refuses_bad_params(lib, kw, code):
    p = norm(**kw)
    assert lib.gka_gated_norm(p, V[0], V[1], V[2], V[3], None) == code
    assert lib.gka_gated_norm_bwd(p, V[0], V[1], V[2], V[3], V[4], V[5], V[6], V[7], 1 << 30,
                                  None) == code
    if "gate_stride" not in kw or "x_stride" in kw:
        assert lib.gka_gated_norm_bwd_workspace_bytes(p) == 0


def test_gated_norm_refuses_bad_pointers(lib):
    fwd = lambda x=V[0], g=V[1], w=V[2], y=V[3], **kw: lib.gka_gated_norm(norm(**kw), x, g, w, y, None)
    assert lib.gka_gated_norm(None, V[0], V[1], V[2], V[3], None) == 1
    assert fwd(x=None) == 1 and fwd(y=None) == 1
    assert fwd(x=at(0, 1)) == 2 and fwd(g=at(1, 1)) == 2 and fwd(w=at(2, 2)) == 2
    assert fwd(y=at(3, 2), dtype=1) == 2
    assert fwd(y=V[0]) == 7 and fwd(y=at(1, 4 * 128 * 2 - 2)) == 7 and fwd(y=at(2, 252)) == 7
    # a strided input reaches past its dense size
    assert fwd(y=at(0, 3 * 1000 * 2 + 254), x_stride=1000) == 7
    assert fwd(rows=0, x=None, y=None) == 0
    need = lib.gka_gated_norm_bwd_workspace_bytes(norm())
    assert need > 0 and need % 256 == 0

    def bwd(x=V[0], g=V[1], w=V[2], dy=V[3], dx=V[4], dg=V[5], dw=V[6], ws=V[7], n=need, **kw):
        return lib.gka_gated_norm_bwd(norm(**kw), x, g, w, dy, dx, dg, dw, ws, n, None)
    assert bwd(x=None) == 1 and bwd(dy=None) == 1 and bwd(dx=None) == 1 and bwd(dg=None) == 1
    assert bwd(ws=None) == 5 and bwd(n=need - 1) == 5 and bwd(ws=at(7, 8)) == 5
    assert bwd(dx=V[0]) == 7 and bwd(dg=V[3]) == 7 and bwd(dx=V[5]) == 7 and bwd(dw=at(7, 4)) == 7
    assert bwd(dw=at(6, 1)) == 2 and bwd(dy=at(3, 1)) == 2
    assert bwd(rows=0, x=None, dy=None, dx=None, dg=None, dw=None, ws=None, n=0) == 0


BAD_JOIN = [(dict(dtype=3), 4), (dict(res_dtype=3), 4), (dict(dtype=1, res_dtype=0), 4),
            (dict(rows=-1), 2), (dict(C=0), 2),
            (dict(C=8193, res_stride=9000, y_stride=9000, gate_stride=9000), 2),
            (dict(rows=1 << 40), 2), (dict(res_stride=63), 2), (dict(y_stride=0), 2),
            (dict(y_stride=BIG), 2), (dict(eps=0.0), 3), (dict(alpha=float("nan")), 3),
            (dict(alpha=float("inf")), 3), (dict(act=5), 3)]


def bwd_join(lib, p, **kw):
    a = dict(res=V[0], y=V[1], gate=V[2], wp=V[3], s=V[4], wn=V[5], dro=V[6], dn=V[7], dr=V[8],
             dy=V[9], dg=V[10], dwp=V[11], ds=V[12], dwn=V[13], ws=V[14], n=1 << 30)
    a.update(kw)
    return lib.gka_join_bwd(p, *a.values(), None)


@pytest.mark.parametrize("kw,code", BAD_JOIN)
def test_join_refuses_bad_params(lib, kw, code):
    assert lib.gka_join(join(**kw), V[0], V[1], V[2], V[3], V[4], V[5], V[6], V[7], None) == code
    assert bwd_join(lib, join(**kw)) == code
    assert lib.gka_join_bwd_workspace_bytes(join(**kw)) == 0


def test_join_refuses_bad_pointers(lib):
    def fwd(p=None, **kw):
        a = dict(res=V[0], y=V[1], gate=V[2], wp=V[3], s=V[4], wn=V[5], ro=V[6], n=V[7])
        a.update(kw)
        return lib.gka_join(p or join(), *a.values(), None)
    assert lib.gka_join(None, V[0], V[1], V[2], V[3], V[4], V[5], V[6], V[7], None) == 1
    assert fwd(res=None) == 1 and fwd(y=None) == 1 and fwd(ro=None) == 1
    assert fwd(n=None) == 1 and fwd(wn=None) == 1  # n exactly when w_pre
    assert fwd(y=at(1, 1)) == 2 and fwd(s=at(4, 2)) == 2 and fwd(res=at(0, 2), p=join(res_dtype=1)) == 2
    assert fwd(n=V[0]) == 7 and fwd(n=V[6]) == 7 and fwd(ro=V[1]) == 7 and fwd(ro=at(0, 2)) == 7
    assert fwd(ro=V[0], p=join(res_stride=80)) == 7  # in place needs the dense stride
    assert fwd(p=join(rows=0), res=None, y=None, ro=None, n=None) == 0
    need = lib.gka_join_bwd_workspace_bytes(join())
    assert need >= 3 * 64 * 4
    bwd = lambda p=None, **kw: bwd_join(lib, p or join(), **kw)
    for k in ("res", "y", "dro", "dn", "dr", "dy", "dg", "dwp", "ds", "dwn", "wp", "s", "wn"):
        assert bwd(**{k: None}) == 1, k
    assert bwd(ws=None) == 5 and bwd(n=need - 1) == 5 and bwd(ws=at(14, 4)) == 5
    assert bwd(dr=V[0]) == 7 and bwd(dy=V[7]) == 7 and bwd(dg=V[9]) == 7 and bwd(dwn=V[5]) == 7
    assert bwd(dwp=at(11, 2)) == 2 and bwd(dy=at(9, 1)) == 2
    assert bwd(join(rows=0), res=None, y=None, gate=None, wp=None, s=None, wn=None, dwp=None,
               ds=None, dwn=None, ws=None, n=0, dn=None) == 0


BAD_RECUR = [(dict(dtype=2), 4), (dict(B=0), 2), (dict(T=-1), 2), (dict(C=0), 2),
             (dict(complement=2), 3), (dict(xt=63), 2), (dict(ft=-64), 2), (dict(xb=300 * 64 - 1), 2),
             (dict(fb=0), 2), (dict(xt=1 << 41, xb=1 << 50), 2),
             (dict(B=1 << 16, C=1 << 15, xt=1 << 15, ft=1 << 15, xb=300 << 15, fb=300 << 15), 2),
             (dict(B=1 << 20, T=1 << 14, C=1, xt=1, ft=1, xb=1 << 14, fb=1 << 14), 2)]


@pytest.mark.parametrize("kw,code", BAD_RECUR)
def test_recur_refuses_bad_params(lib, kw, code):
    p = recur(**kw)
    assert lib.gka_recur(p, V[0], V[1], V[2], V[3], V[4], V[5], 1 << 39, None) == code
    assert lib.gka_recur_bwd(p, V[0], V[1], V[2], V[3], V[4], V[5], V[6], V[7], V[8], 1 << 39,
                             None) == code
    assert lib.gka_recur_workspace_bytes(p) == lib.gka_recur_carry_bytes(p) == 0


def test_recur_refuses_bad_pointers(lib):
    need = lib.gka_recur_workspace_bytes(recur())

    def fwd(x=V[0], f=V[1], h=V[2], st=V[3], ca=V[4], ws=V[5], n=need, **kw):
        return lib.gka_recur(recur(**kw), x, f, h, st, ca, ws, n, None)
    assert lib.gka_recur(None, V[0], V[1], V[2], None, None, V[5], need, None) == 1
    assert fwd(x=None) == 1 and fwd(f=None) == 1 and fwd(h=None) == 1
    assert fwd(x=at(0, 1)) == 2 and fwd(st=at(3, 2)) == 2
    assert fwd(ca=at(4, 4)) == 5
    assert fwd(h=V[0]) == 7 and fwd(h=at(1, 256)) == 7 and fwd(st=V[2]) == 7 and fwd(ca=V[2]) == 7
    if need:
        assert fwd(ws=None) == 5 and fwd(n=need - 1) == 5 and fwd(ws=V[0]) == 7
    assert fwd(T=0, x=None, f=None, h=None) == 0
    step = lambda x=V[0], f=V[1], h=V[2], st=V[3], **kw: lib.gka_recur_step(
        recur(**{"xb": 64, "fb": 64, **kw}), x, f, h, st, None)
    assert step(x=None) == 1 and step(st=None) == 1 and step(xb=63) == 2
    assert step(h=V[1]) == 7 and step(st=V[0]) == 7 and step(st=at(3, 1)) == 2
    needb = lib.gka_recur_bwd_workspace_bytes(recur())

    def bwd(x=V[0], f=V[1], dh=V[2], ca=V[3], d1=V[4], dx=V[5], df=V[6], d0=V[7], ws=V[8], n=needb,
            **kw):
        return lib.gka_recur_bwd(recur(**kw), x, f, dh, ca, d1, dx, df, d0, ws, n, None)
    for k in ("x", "f", "dh", "ca", "dx", "df"):
        assert bwd(**{k: None}) == 1, k
    assert bwd(dx=V[0]) == 7 and bwd(df=V[5]) == 7 and bwd(d0=V[4]) == 7 and bwd(dx=V[3]) == 7
    assert bwd(d0=at(7, 2)) == 2 and bwd(d1=at(4, 1)) == 2 and bwd(ca=at(3, 8)) == 5
    if needb:
        assert bwd(ws=None) == 5 and bwd(n=needb - 1) == 5
    assert bwd(T=0, x=None, f=None, dh=None, ca=None, dx=None, df=None, d0=None) == 0
    assert bwd(T=0, d0=V[4]) == 7


def test_carry_covers_every_segment(lib):
    # one float32 state per segment, batch row and channel; at least one segment, none without tokens
    assert lib.gka_recur_carry_bytes(recur(T=0)) == 0
    sizes = [lib.gka_recur_carry_bytes(recur(T=t, xb=t * 64, fb=t * 64)) for t in (1, 1000, 100000)]
    assert sizes[0] >= 2 * 64 * 4 and sizes == sorted(sizes)
    # it does not depend on strides
    assert lib.gka_recur_carry_bytes(recur(xt=1000, xb=300 * 1000)) == lib.gka_recur_carry_bytes(recur())


def _asan_runtime():
    if not os.path.exists(CLANG):
        return None
    r = subprocess.run([CLANG, "-print-file-name=libclang_rt.asan-x86_64.so"], capture_output=True,
                       text=True)
    path = r.stdout.strip()
    return path if r.returncode == 0 and os.path.isabs(path) and os.path.exists(path) else None


@pytest.mark.timeout(600)
@pytest.mark.skipif("GKA_LIBRARY" in os.environ, reason="already the sanitized library")
def test_host_code_under_asan_and_ubsan(tmp_path):
    rt = _asan_runtime()
    if rt is None:
        pytest.skip("the ASan runtime is not available")
    src = "gka_block_api.cpp"
    others = [os.path.join(build.BUILD, s + ".o") for s in build.SOURCES if s != src]
    if not all(os.path.exists(o) for o in others):
        build.build_library()
    san = ["-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined"]
    obj, out = str(tmp_path / "block_api_san.o"), str(tmp_path / "libgka_san.so")
    cc = [build.HIPCC, "-x", "hip", "--offload-arch=gfx950", "-O1", "-g", "-std=c++17", "-fPIC",
          "-I" + os.path.join(ROOT, "include"), *san, "-Xarch_host",
          "-fno-sanitize-recover=undefined", "-c", os.path.join(build.CSRC, src), "-o", obj]
    r = subprocess.run(cc, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    ld = [build.HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", obj, *others, *san,
          "-shared-libasan", "-o", out]
    r = subprocess.run(ld, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    env = dict(os.environ, LD_PRELOAD=rt, GKA_LIBRARY=out,
               ASAN_OPTIONS="detect_leaks=0:abort_on_error=1",
               UBSAN_OPTIONS="halt_on_error=1:print_stacktrace=1")
    r = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider",
                        os.path.abspath(__file__)], cwd=ROOT, env=env, capture_output=True,
                       text=True)
    assert r.returncode == 0, r.stdout[-3000:] + r.stderr[-3000:]
    assert "passed" in r.stdout and "failed" not in r.stdout


@pytest.mark.parametrize("dtype", [0, 1])
@pytest.mark.parametrize("T", [(1 << 31) - 1, (1 << 31) - 100, (1 << 31) - 255, (1 << 31) - 256, 1 << 30])
def test_recur_refuses_more_segments_than_a_grid(lib, T, dtype):
    """Sequences near the largest 32-bit length: the count of segments rounds up past 32 bits."""
    p = recur(B=1, T=T, C=1, dtype=dtype, xb=T, xt=1, fb=T, ft=1)
    assert lib.gka_recur(p, V[0], V[1], V[2], V[3], None, V[5], 1 << 39, None) == 2
    assert lib.gka_recur_bwd(p, V[0], V[1], V[2], V[3], None, V[5], V[6], V[7], V[8], 1 << 39, None) == 2
    assert lib.gka_recur_workspace_bytes(p) == lib.gka_recur_bwd_workspace_bytes(p) == 0
    assert lib.gka_recur_carry_bytes(p) == 0
