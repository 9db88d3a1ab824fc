"""The binding of the block operators without a GPU: what its calls hand to the library, recorded by a
stand-in for it."""
import pytest
import torch

from test_ridge_regression_amd import block, gka


class Library:
    """Records the parameter block of every call; sizes are 0."""

    def __init__(self):
        self.last = None

    def __getattr__(self, name):
        def call(p, *args):
            if not name.endswith("_bytes"):
                self.last = p._obj
            return 0
        return call


@pytest.fixture
def lib(monkeypatch):
    lib = Library()
    monkeypatch.setattr(gka, "load", lambda: lib)
    monkeypatch.setattr(block, "_stream", lambda x: 0)
    return lib


def on_cpu(fn):
    """The call without the wrapper that refuses host tensors."""
    return fn.__wrapped__


X = torch.zeros(4, 2, 16)
W = torch.ones(16)
F = torch.zeros(2, 5, 8)
SCALAR_CALLS = {
    "gated_norm eps": (lambda v: on_cpu(block.gated_norm)(X, eps=v), "eps"),
    "gated_norm_bwd eps": (lambda v: on_cpu(block.gated_norm_bwd)(X, None, None, X, eps=v), "eps"),
    "join eps": (lambda v: on_cpu(block.join)(X, X, eps=v), "eps"),
    "join alpha": (lambda v: on_cpu(block.join)(X, X, alpha=v), "alpha"),
    "join_bwd alpha": (lambda v: on_cpu(block.join_bwd)(X, X, X, alpha=v), "alpha"),
    "recur complement": (lambda v: on_cpu(block.recur)(F, F, complement=v), "complement"),
    "recur_step complement": (lambda v: on_cpu(block.recur_step)(F[:, 0], F[:, 0], torch.zeros(2, 8),
                                                                 complement=v), "complement"),
}


@pytest.mark.parametrize("name", SCALAR_CALLS)
def test_a_scalar_tensor_is_read_by_every_call(lib, name):
    """A learnt residual scale, say: the same tensor holds another value at the next call."""
    call, field = SCALAR_CALLS[name]
    value = torch.tensor(1.0)
    call(value)
    assert getattr(lib.last, field) == 1
    value.fill_(0.0 if field == "complement" else 0.25)
    call(value)
    assert getattr(lib.last, field) == value.item()


@pytest.mark.parametrize("shape", [((1 << 32) + 3, 1, 1), (1, (1 << 32) + 5, 1), (1, 1, (1 << 32) + 8)])
def test_recur_refuses_sizes_beyond_32_bits(lib, shape):
    """A dimension that the parameter block would hold modulo 2^32: the call would cover a part of it."""
    x = torch.empty(shape, device="meta")
    with pytest.raises(ValueError):
        on_cpu(block.recur)(x, x)
    carry = torch.empty(0, device="meta", dtype=torch.float32)
    with pytest.raises(ValueError):
        on_cpu(block.recur_bwd)(x, x, x, carry)
    if shape[1] == 1:
        row, state = x[:, 0], torch.empty(shape[0], shape[2], device="meta")
        with pytest.raises(ValueError):
            on_cpu(block.recur_step)(row, row, state)


def test_norm_and_join_hand_wide_rows_over_whole(lib):
    """Their rows may be as wide as the C side checks: a width beyond 32 bits shows in the stride."""
    x = torch.empty((1, 1, (1 << 32) + 64), device="meta")
    on_cpu(block.gated_norm)(x)
    assert lib.last.x_stride == (1 << 32) + 64
    on_cpu(block.join)(x, x)
    assert lib.last.res_stride == lib.last.y_stride == (1 << 32) + 64


def _first_tensor(monkeypatch, fn, **kw):
    """What the wrapper of ``fn`` takes for the tensor that names the device, called with keywords."""
    seen = []

    class Device(torch.Tensor):
        def get_device(self):
            seen.append(self.tag)
            return -1
    tensors = {}
    for k, v in kw.items():
        if isinstance(v, torch.Tensor):
            v = v.as_subclass(Device)
            v.tag = k
        tensors[k] = v
    with pytest.raises(ValueError):
        fn(**tensors)
    return seen[0] if seen else None


@pytest.mark.parametrize("fn,first,kw", [
    (block.gated_norm, "x", {"eps": 1e-5, "x": X}), (block.gated_norm, "x", {"gate": None, "x": X}),
    (block.gated_norm, "x", {"act": "silu", "gate": X.clone(), "x": X}),
    (block.gated_norm_bwd, "x", {"dy": X.clone(), "weight": None, "gate": None, "x": X}),
    (block.join, "res", {"alpha": 0.5, "y": X.clone(), "res": X}),
    (block.join_bwd, "res", {"dn": None, "dres_out": X.clone(), "y": X.clone(), "res": X}),
    (block.recur, "x", {"complement": False, "f": F.clone(), "x": F}),
    (block.recur_step, "x", {"state": torch.zeros(2, 8), "f": F[:, 0], "x": F[:, 0]}),
    (block.recur_bwd, "x", {"dstate": None, "carry": W, "dh": F, "f": F, "x": F})])
def test_keywords_in_any_order(monkeypatch, fn, first, kw):
    assert _first_tensor(monkeypatch, fn, **kw) == first


def test_a_missing_tensor_is_named():
    with pytest.raises(TypeError, match="'x'"):
        block.gated_norm(gate=X)
    with pytest.raises(TypeError, match="'res'"):
        block.join(y=X)
