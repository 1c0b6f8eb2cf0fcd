"""Distances between rows of queries behind a shared prefix: refused before anything is launched where the
prefix kernel's 32-bit steps would not reach."""

import ctypes

import pytest

X = 256  # a device address that is never read


@pytest.mark.parametrize("name", ["kitty_tree_attention", "kitty_f16kv_tree_attention"])
def test_rows_too_far_apart(name):
    from mixed_precision_bit_gb300 import kitty
    cfg = kitty.Config(num_kv_heads=2, num_q_heads=8).c()
    f16 = "f16" in name
    nodes, B, n_prefix, max_pages = 16, 40, 128, 3
    size = kitty.f16kv_tree_workspace_bytes if f16 else kitty.tree_workspace_bytes
    # partials of a prefix that is attended by the prefix kernel
    assert (size(kitty.Config(num_kv_heads=2, num_q_heads=8), B, B * nodes, nodes, max_pages, n_prefix)
            > size(kitty.Config(num_kv_heads=2, num_q_heads=8), B, B * nodes, nodes, max_pages, 0))
    lens = [X] if f16 else [X, X, X, X]
    for stride, code in (((1 << 29) + 8, -2), (1 << 29, -4)):  # the second has no workspace
        rc = getattr(kitty.load(), name)(ctypes.byref(cfg), X, stride, X, 256, X, 256, B * nodes, X, None, nodes, X, 500, X,
                                         n_prefix, None, X, max_pages, *lens, 0.1, X, 2, None, 0, B, None, None)
        assert rc == code, stride
