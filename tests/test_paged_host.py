"""The paged cache's binding and limits, on the host (no GPU needed)."""
import ctypes

import pytest

import sparse_kv_prefetch_gb300 as dd


def _shape(**kw):
    base = dict(batch=2, n_q_heads=8, n_kv_heads=2, head_dim=128, page_size=16, n_pages=10,
                max_pages=4, dtype=dd.DD_BF16, format=dd.DD_PAGES_PLAIN)
    base.update(kw)
    return dd.PagedShape(**base)


def test_a_shape_hands_out_structures_of_its_own():
    """Writing to the structure of one shape changes no other call of an equal shape."""
    want = dd.paged_pool_bytes(_shape())
    c = _shape().c()
    c.n_pages = 1000
    assert _shape().c().n_pages == 10 and dd.paged_pool_bytes(_shape()) == want


def test_pointer_checks_ask_for_a_device_only_when_a_pointer_needs_one():
    """Absent pointers are no host pointers, with a device or without."""
    f = getattr(dd.lib(), "_ZN2dd10all_deviceESt16initializer_listIPKvE")
    f.argtypes, f.restype = [ctypes.c_void_p, ctypes.c_size_t], ctypes.c_bool
    two = (ctypes.c_void_p * 2)()
    assert f(two, 2) and f(two, 0)
    two[1] = ctypes.addressof(two)
    assert not f(two, 2)


def test_calls_beyond_the_largest_grid_are_unsupported():
    """Refused by their sizes, before anything is launched."""
    L, most = dd.lib(), 1 << 30
    s = _shape(n_q_heads=64, n_kv_heads=64, head_dim=64, batch=64)
    seqs = dd.dd_paged_seqs(16, 16, 16, 16, 16)

    def append(n, q):
        return L.dd_paged_append(ctypes.byref(s.c()), ctypes.byref(seqs), n, q, 16, 16, 64 * 64,
                                 64 * 64, 64 * 64, q and 32, None, 0, 0, 0, None)

    def read(count):
        return L.dd_paged_read(ctypes.byref(s.c()), ctypes.byref(seqs), 0, count, 16, 16, None)

    def attn(n):  # split: merged by a grid of a CTA for every row
        return L.dd_paged_attn(ctypes.byref(s.c()), ctypes.byref(seqs), n, 16, 64 * 64, 1, most, 0,
                               0, 16, None, 16, 1 << 62, None)

    # within the grid the addresses are what is refused
    assert append(most, 16) == dd.DD_ERR_UNSUPPORTED and append(1000, 16) == dd.DD_ERR_INVALID_ARG
    assert read(most) == dd.DD_ERR_UNSUPPORTED and read(1000) == dd.DD_ERR_INVALID_ARG
    assert attn(most) == dd.DD_ERR_UNSUPPORTED and attn(1000) == dd.DD_ERR_INVALID_ARG
