"""The block operators at the edges of their inputs, on the GPU: infinities."""
import numpy as np
import pytest
import torch

from oracle.block_oracle import recur_ref
from test_ridge_regression_amd import block, gka

from gka_testutil import log

pytestmark = pytest.mark.gpu

TORCH = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF_ULP = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float32)}


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gka.load()


def num(t):
    return t.detach().double().cpu().numpy()


def on_gpu(a, dtype):
    return torch.from_numpy(np.asarray(a, np.float32)).cuda().to(TORCH[dtype])


def ref(x, f, state, complement, dh=None, dstate=None):
    with np.errstate(invalid="ignore"):
        return recur_ref(x, f, state, complement, dh, dstate)


def same(got, want):
    """Infinities and NaN in the same places; finite values to the rounding of their type and the
    oracle's bound, which is finite where the value is."""
    for name, (w, bound) in want.items():
        t = got[name]
        g, fin = num(t), np.isfinite(w)
        assert np.array_equal(np.isnan(g), np.isnan(w)), (name, "NaN")
        assert np.array_equal(g[np.isinf(g)], w[np.isinf(g)]) and not np.isinf(w[np.isfinite(g)]).any(), \
            (name, "inf")
        w, b, g = w[fin], bound[fin], g[fin]
        off = np.abs(g - w) / (HALF_ULP[t.dtype] * (np.abs(w) + b) + b + 1e-37)
        assert off.max(initial=0.0) <= 1.0, (name, off.max())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("complement", [True, False])
@pytest.mark.parametrize("B,T,C", [(2, 1, 64), (2, 5, 66), (3, 700, 33), (1, 1500, 130), (1, 5001, 16),
                                   (2, 260, 3)])
def test_recur_infinities(B, T, C, complement, dtype):
    """Infinite inputs, states and gradients under gates of either sign, finite ones that open or
    close the channel for long (its gates' product underflows) and infinite ones."""
    log(f"recur infinities {B}x{T}x{C} {dtype} {complement}")
    rng = np.random.default_rng(T + C)
    inf = float("inf")
    draw = lambda *s: num(on_gpu(rng.standard_normal(s), dtype))
    x, f, dh = draw(B, T, C), draw(B, T, C), draw(B, T, C)
    state, ds = rng.standard_normal((B, C)), rng.standard_normal((B, C))
    state, ds = state.astype(np.float32).astype(float), ds.astype(np.float32).astype(float)
    kind = np.arange(C) % 11
    f[..., kind == 1] += 4.0
    f[..., kind == 2] -= 4.0
    f = num(on_gpu(f, dtype))
    at = lambda k: rng.integers(0, T)
    x[:, at(0), kind == 0] = inf
    x[:, at(0), kind == 1] = -inf
    x[:, at(0), kind == 2] = inf
    x[:, at(0), kind == 2] = -inf
    state[:, kind == 3] = inf
    state[:, kind == 4] = -inf
    f[:, at(0), kind == 4] = inf
    dh[:, at(0), kind == 5] = inf
    dh[:, at(0), kind == 5] = -inf
    ds[:, kind == 6] = -inf
    state[:, kind == 7] = inf
    f[:, at(0), kind == 7] = -inf  # 0 times an infinity
    x[:, T - 1, kind == 8] = inf
    dh[:, 0, kind == 8] = -inf
    f[:, at(0), kind == 9] = -inf
    x[:, at(0), kind == 9] = inf
    ds[:, kind == 10] = inf
    f[:, at(0), kind == 10] = inf
    want = ref(x, f, state, complement, dh, ds)
    xt, ft, dt = (on_gpu(v, dtype) for v in (x, f, dh))
    st = on_gpu(state, "fp32")
    h, carry = block.recur(xt, ft, state=st, complement=complement, return_carry=True)
    dx, df, d0 = block.recur_bwd(xt, ft, dt, carry, dstate=on_gpu(ds, "fp32"), complement=complement)
    same({"h": h, "state": st, "dx": dx, "df": df, "dstate": d0}, want)
    # token by token
    st = on_gpu(state, "fp32")
    steps = [block.recur_step(xt[:, t], ft[:, t], st, complement=complement) for t in range(min(T, 60))]
    same({"h": torch.stack(steps, 1)}, {"h": tuple(v[:, :60] for v in want["h"])})


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_recur_infinities_leave_other_channels(dtype):
    """Bit for bit, and in the vector that holds the infinite channel too."""
    rng = np.random.default_rng(7)
    B, T, C = 2, 700, 70
    x, f, dh = (on_gpu(rng.standard_normal((B, T, C)), dtype) for _ in range(3))

    def run():
        h, carry = block.recur(x, f, return_carry=True)
        return (h, *block.recur_bwd(x, f, dh, carry))
    want = run()
    odd = [5, 33, 69]
    x[:, 300, 5], x[:, 400, 33], dh[:, 500, 69] = float("inf"), -float("inf"), float("inf")
    keep = [c for c in range(C) if c not in odd]
    for a, b in zip(run(), want):
        assert torch.equal(a[..., keep], b[..., keep]) and not torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T", [1, 7, 300, 1500])
def test_recur_of_the_largest_values(T, dtype):
    """h stays between its inputs, whose difference is beyond float32."""
    rng = np.random.default_rng(T)
    x = num(on_gpu(3e38 * rng.choice([-1.0, 1.0], (2, T, 40)), dtype))
    f = num(on_gpu(rng.standard_normal((2, T, 40)), dtype))
    state = num(on_gpu(np.full((2, 40), -3e38), "fp32"))
    want = ref(x, f, state, True)
    st = on_gpu(state, "fp32")
    same({"h": block.recur(on_gpu(x, dtype), on_gpu(f, dtype), state=st), "state": st}, want)
    st = on_gpu(state, "fp32")
    h = block.recur_step(on_gpu(x[:, 0], dtype), on_gpu(f[:, 0], dtype), st)
    same({"h": h[:, None]}, {"h": tuple(v[:, :1] for v in want["h"])})


@pytest.mark.parametrize("device", ["cpu", "cuda"])
@pytest.mark.parametrize("side", [False, True])
def test_a_scalar_tensor_is_read_by_every_call(device, side):
    """A residual scale that is learnt: the same tensor with another value gives the other result."""
    rng = np.random.default_rng(11)
    res, y, g = (on_gpu(rng.standard_normal((5, 64)), "fp32") for _ in range(3))
    torch.cuda.synchronize()
    kw = {"stream": torch.cuda.Stream()} if side else {}
    alpha = torch.tensor(0.5, device=device)
    for value in (0.5, 0.125):
        alpha.fill_(value)
        torch.cuda.synchronize()
        out, dy = block.join(res, y, alpha=alpha, **kw)[0], block.join_bwd(res, y, g, alpha=alpha, **kw).dy
        torch.cuda.synchronize()
        assert torch.equal(out, torch.add(res, y, alpha=value)) and torch.equal(dy, value * g)


def test_keywords_in_any_order():
    rng = np.random.default_rng(12)
    x, g = (on_gpu(rng.standard_normal((5, 2, 32)), "bf16") for _ in range(2))
    assert torch.equal(block.gated_norm(eps=1e-5, gate=g, x=x), block.gated_norm(x, g, eps=1e-5))
    assert torch.equal(block.gated_norm(gate=None, x=x), block.gated_norm(x))
    assert torch.equal(block.join(alpha=0.5, y=g, res=x)[0], block.join(x, g, alpha=0.5)[0])
    assert torch.equal(block.recur(complement=False, f=g, x=x), block.recur(x, g, complement=False))


def test_precision_of_the_smaller_sigmoid():
    """A step from state 1 with x = 0 under f < 0 leaves sigmoid(f) itself: exp2 and the reciprocal to 1 ulp
    (2 units of 2^-24 each), a sum and a product, and the argument of exp2 rounded twice (1.25 |f| units)."""
    f = -torch.linspace(0.0, 80.0, 1 << 16, device="cuda")[None]
    state = torch.ones_like(f)
    block.recur_step(torch.zeros_like(f), f, state)
    f, got = num(f), num(state)
    want = np.exp(f) / (1.0 + np.exp(f))
    units = np.abs(got / want - 1.0) / 2.0 ** -24
    assert (units <= 6 + 1.25 * np.abs(f)).all(), units.max()


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("B,T,C", [(1, 100000, 16), (2, 50001, 70)])
def test_hundreds_of_segments_repeat_bit_for_bit(B, T, C, dtype):
    """Whichever words a segment's look-back finds, the chain of operations is the same."""
    log(f"recur long chains {B}x{T}x{C} {dtype}")
    rng = np.random.default_rng(T)
    x, f, dh = (on_gpu(rng.standard_normal((B, T, C)) + m, dtype) for m in (0.0, 3.0, 0.0))
    s0, ds = (on_gpu(rng.standard_normal((B, C)), "fp32") for _ in range(2))

    def run():
        st = s0.clone()
        h, carry = block.recur(x, f, state=st, return_carry=True)
        return (h, st, *block.recur_bwd(x, f, dh, carry, dstate=ds))
    first = run()
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(run(), first))
