"""The oracle's bounds are small enough to show the mistakes that the kernels' sums could make: an element
of a row's last vector counted twice or not at all, a row left out of a weight gradient. The mistakes are
planted here, in float64 forms of the operators beside the oracle's."""
import numpy as np
import pytest

from oracle.block_oracle import gated_norm_ref, join_ref

EPS = 1e-5
HALF_ULP = 2.0 ** -24  # float32


def beyond(got, ref):
    """The largest of |got - ref| over what the GPU tests allow."""
    value, bound = ref
    return (np.abs(got - value) / (HALF_ULP * (np.abs(value) + bound) + bound)).max()


def norm(x, counts, eps=EPS):
    """x / rms(x) with every element counted ``counts`` times in the mean."""
    return x / np.sqrt((counts * x * x).sum(-1, keepdims=True) / x.shape[-1] + eps)


@pytest.mark.parametrize("D", [33, 77, 1001, 4001, 8191])
@pytest.mark.parametrize("times", [0.0, 2.0])
def test_a_tail_element_counted_wrongly_shows(D, times):
    rng = np.random.default_rng(D)
    x = rng.standard_normal((6, 1, D))
    counts = np.ones(D)
    counts[D - 4] = times  # the first element of the last whole vector of four
    ref = gated_norm_ref(x, None, None, EPS, "silu")["y"]
    assert beyond(norm(x, np.ones(D)), ref) <= 1.0
    assert beyond(norm(x, counts), ref) > 1.0
    rows = x[:, 0]
    ref = join_ref(np.zeros_like(rows), rows, None, np.ones(D), None, None, 1.0, EPS, "silu")["res_out"]
    assert beyond(norm(rows, counts), ref) > 1.0
    ref = join_ref(rows, np.zeros_like(rows), None, None, None, np.ones(D), 1.0, EPS, "silu")["n"]
    assert beyond(norm(rows, counts), ref) > 1.0


@pytest.mark.parametrize("rows,H,D", [(2500, 8, 128), (1237, 5, 77), (600, 1, 2048)])
@pytest.mark.parametrize("per_head", [False, True])
def test_a_row_left_out_of_a_weight_gradient_shows(rows, H, D, per_head):
    rng = np.random.default_rng(rows)
    x, dy = rng.standard_normal((2, rows, H, D))
    ref = gated_norm_ref(x, None, np.ones((H, D) if per_head else (D,)), EPS, "silu", dy)["dweight"]
    t = dy * norm(x, np.ones(D))
    axes = (0,) if per_head else (0, 1)
    assert beyond(t.sum(axes), ref) <= 1.0
    t[rows // 2] = 0.0
    assert beyond(t.sum(axes), ref) > 1.0


@pytest.mark.parametrize("rows,C", [(12000, 250), (700, 2049)])
def test_a_row_left_out_of_a_join_gradient_shows(rows, C):
    rng = np.random.default_rng(rows)
    res, y, dres, dn = rng.standard_normal((4, rows, C))
    one = np.ones(C)
    ref = join_ref(res, y, None, one, one, one, 0.7, EPS, "silu", dres, dn)
    keep = np.arange(rows) != rows // 3
    part = join_ref(res[keep], y[keep], None, one, one, one, 0.7, EPS, "silu", dres[keep], dn[keep])
    for name in ("dw_post", "dscale", "dw_pre"):
        assert beyond(part[name][0], ref[name]) > 1.0, name
