"""Host-side checks of the expert block's calls that need no GPU: a null group
or handle is refused before any CUDA call, and the binding checks types and
shapes before it calls the library."""
import ctypes
import shutil

import pytest
import torch

INVALID = 1


@pytest.fixture(scope="module")
def ep():
    import os
    if shutil.which("nvcc") is None and not os.path.exists("/usr/local/cuda/bin/nvcc"):
        pytest.skip("no CUDA toolkit")
    from combine_layout_gb300 import build
    build.build()
    import combine_layout_gb300.moe_ep as ep
    return ep


def test_null_handles_are_refused(ep):
    lib = ep._lib
    assert lib.moe_ep_ffn_gate_up(None, None, None, 64, 0, None, None, 0, None) == INVALID
    assert lib.moe_ep_ffn_down(None, None, None, 64, None, 0, None) == INVALID
    assert lib.moe_ep_ffn_down_backward(None, None, None, None, 64, 0, None, None, 0, None) == INVALID
    assert lib.moe_ep_ffn_gate_up_backward(None, None, None, 64, None, 0, None) == INVALID
    assert lib.moe_ep_ffn_weight_grad(None, None, 64, None, 64, None, 0, 0, 0, None) == INVALID
    assert lib.moe_ep_combine_backward(None, None, None, None, None, None, 0, None) == INVALID
    assert lib.moe_ep_norm_residual(None, None, None, None, None, 0, None, 1.0, 1e-6, 0, None, None, None) == INVALID
    assert lib.moe_ep_norm_residual_backward(None, *[None] * 4, 0, None, 1.0, 1e-6, 0, *[None] * 9) == INVALID
    n = ctypes.c_int64()
    assert lib.moe_ep_norm_work_floats(None, ctypes.byref(n)) == INVALID


def test_binding_checks_types_and_shapes(ep, monkeypatch):
    E, H, F, n = 4, 64, 32, 10
    monkeypatch.setitem(ep._sizes, 1, (E, H, 0))
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, hid, w, wd = z(n, H), z(n, F), z(E, 2 * F, H), z(E, H, F)
    bad = [
        lambda: ep.moe_ep_ffn_gate_up(1, x.float(), w, hid),
        lambda: ep.moe_ep_ffn_gate_up(1, z(n, H + 8), w, hid),
        lambda: ep.moe_ep_ffn_gate_up(1, x, z(E - 1, 2 * F, H), hid),
        lambda: ep.moe_ep_ffn_gate_up(1, x, w, hid, z(n, F)),
        lambda: ep.moe_ep_ffn_down(1, hid, z(E, F, H), x),
        lambda: ep.moe_ep_ffn_down_backward(1, x, wd, z(n, F), z(n, 2 * F)),
        lambda: ep.moe_ep_ffn_gate_up_backward(1, z(n, 2 * F), w, z(n, F)),
        lambda: ep.moe_ep_ffn_weight_grad(1, hid, x, z(E, F, H, dtype=torch.float16)),
        lambda: ep.moe_ep_ffn_weight_grad(1, hid, x, z(E, H, F)),
        lambda: ep.moe_ep_combine_backward(1, x, x, z(n, 2), z(n, H), z(n, 2)),
        lambda: ep.moe_ep_norm_residual(1, x, z(n - 1, H), None, None, None, x, None),
        lambda: ep.moe_ep_norm_residual(1, x, x, z(H), None, None, x, None),
        lambda: ep.moe_ep_norm_residual(1, x, x, None, z(n - 1, dtype=torch.float32), None, x, None, gate_per_token=True),
    ]
    for f in bad:
        with pytest.raises(ValueError):
            f()


def test_numbers_that_do_not_fit_are_refused(ep, monkeypatch):
    H, n = 64, 10
    monkeypatch.setitem(ep._sizes, 1, (4, H, 0))
    z = lambda *s, dtype=torch.bfloat16: torch.zeros(s, dtype=dtype)  # noqa: E731
    x, far = z(n, H), -2**32 + 5                     # 5 in 32 bits
    for f in (lambda: ep.moe_ep_norm_residual(1, x, None, None, None, None, x, None, num_tokens=far),
              lambda: ep.moe_ep_norm_residual_backward(1, x, None, None, None, None, x, None, x, None, None, None,
                                                       None, z(1, dtype=torch.float32)[:0], num_tokens=far),
              lambda: ep.moe_ep_ffn_gate_up(1, x, z(4, 64, H), z(n, 32), act=2**32),
              lambda: ep.moe_ep_ffn_down_backward(1, x, z(4, H, 32), z(n, 64), z(n, 64), act=2**32)):
        with pytest.raises(ValueError, match="out of range"):
            f()


def test_routed_sizes_of_a_null_handle(ep):
    a, b = ctypes.c_int(), ctypes.c_int()
    assert ep._lib.moe_ep_get_routed(None, ctypes.byref(a), ctypes.byref(b)) == INVALID
