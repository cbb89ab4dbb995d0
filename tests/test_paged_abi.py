"""Refusals of the growing cache's entry points that need no GPU: everything below is rejected on the
host, before any launch or device allocation."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def J():
    from tensor_decomposition_b200 import build
    build.build()
    from tensor_decomposition_b200 import jolt
    return jolt


@pytest.fixture()
def untouched(J):
    before = J.jolt_launch_count(), J.jolt_alloc_count()
    yield
    assert (J.jolt_launch_count(), J.jolt_alloc_count()) == before


def _buf():
    b = ctypes.create_string_buffer(4096 + 16)
    at = (ctypes.addressof(b) + 15) // 16 * 16
    return b, at


@pytest.mark.parametrize("shape,status", [
    ((0, 8, 16, 128, 0), 1), ((4, 0, 16, 128, 0), 1), ((4, 8, 0, 128, 0), 1), ((4, 8, 16, 64, 0), 1),
    ((4, 8, 16, 128, 1), 9), ((4, 8, 16, 128, 5), 9), ((4, 8, 24, 128, 0), 9), ((4, 8, 1 << 25, 128, 2), 9),
    ((4, 1 << 20, 1 << 20, 128, 2), 9),
])
def test_pages_create_refuses(J, untouched, shape, status):
    keep, p = _buf()
    h = ctypes.c_void_p()
    sh = J.PageShape(*shape)
    assert J._lib.jolt_pages_create(ctypes.byref(sh), p, p, None, ctypes.byref(h)) == status
    assert not h.value and J._lib.jolt_last_error().decode().startswith("jolt_pages_create")


def test_pages_create_refuses_null_and_unaligned_pages(J, untouched):
    keep, p = _buf()
    h = ctypes.c_void_p()
    sh = J.PageShape(4, 8, 16, 128, 0)
    for k, v in ((None, p), (p, None), (p + 8, p), (p, p + 2)):
        assert J._lib.jolt_pages_create(ctypes.byref(sh), k, v, None, ctypes.byref(h)) == 1
    assert J._lib.jolt_pages_create(None, p, p, None, ctypes.byref(h)) == 1
    assert J._lib.jolt_pages_create(ctypes.byref(sh), p, p, None, None) == 1


def test_null_handles(J, untouched):
    keep, p = _buf()
    L = J._lib
    d = J.BatchDesc(1, 1, 1, 1, p, p, p)
    calls = {
        "jolt_pages_status": lambda: L.jolt_pages_status(None, None),
        "jolt_paged_append": lambda: L.jolt_paged_append(None, ctypes.addressof(d), p, 128, 128, p, 128, 128, None, 1e-6,
                                                         None, None, 0, 0, None),
        "jolt_paged_attention": lambda: L.jolt_paged_attention(None, ctypes.addressof(d), p, 128, 128, 8, 1.0, 1, None,
                                                               None, p, None, None),
    }
    for name, call in calls.items():
        assert call() == 1, name
        msg = L.jolt_last_error().decode()
        assert msg.startswith(name) and "null" in msg
    L.jolt_pages_destroy(None)


def test_norm_rope_refuses(J, untouched):
    keep, p = _buf()

    def call(dtype=0, tokens=1, q=p, qs=128, hq=1, qo=p, k=None, hk=0, ko=None, w=None, pos=p, fr=p, rd=128):
        return J._lib.jolt_qk_norm_rope(dtype, tokens, q, 128, qs, hq, w, qo, 128, 128, k, 128, 128, hk, None, ko, 128, 128,
                                        1e-6, pos, fr, rd, 0, None)

    assert call(dtype=1) == 9                       # float32 rows
    assert call(tokens=-1) == 1
    assert call(q=None) == 1 and call(qo=None) == 1 and call(hq=0) == 1
    assert call(qs=100) == 1 and call(q=p + 8) == 1 and call(w=p + 4) == 1
    assert call(hk=2, k=p) == 1 and call(hk=2, ko=p) == 1 and call(hk=-1) == 1
    assert call(pos=None) == 1
    for rd in (0, 8, 24, 144, -16):
        assert call(rd=rd) == 1
    assert call(tokens=0, q=None, qo=None) == 0     # nothing to do
