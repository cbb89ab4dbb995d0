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
        "jolt_attention_lse": lambda: L.jolt_attention_lse(None, 0, p, 8, 1, 1.0, p, p, None),
        "jolt_qk_norm_rope": lambda: L.jolt_qk_norm_rope(None, None),
        "jolt_paged_append": lambda: L.jolt_paged_append(None, ctypes.addressof(d), bytes(J._NEW_ROWS.size), None),
        "jolt_paged_attention": lambda: L.jolt_paged_attention(None, ctypes.addressof(d), bytes(J._QUERIES.size), None),
    }
    for name, call in calls.items():
        assert call() == 1, name
        msg = L.jolt_last_error().decode()
        assert msg.startswith(name) and "null" in msg
    L.jolt_pages_destroy(None)


def test_norm_rope_refuses(J, untouched):
    keep, p = _buf()

    def call(dtype=0, tokens=1, q=p, qs=128, hq=1, qo=p, k=None, hk=0, ko=None, w=None, pos=p, fr=p, rd=128):
        z = [x or 0 for x in (q, w, qo, k, ko, pos, fr)]
        return J._lib.jolt_qk_norm_rope(J._NORM_ROPE.pack(z[0], 128, qs, z[1], z[2], 128, 128, z[3], 128, 128, 0, z[4], 128,
                                                          128, z[5], z[6], dtype, tokens, hq, hk, rd, 0, 1e-6), None)

    assert call(dtype=1) == 9                       # float32 rows
    assert call(tokens=-1) == 1
    assert call(q=None) == 1 and call(qo=None) == 1 and call(hq=0) == 1
    assert call(qs=1 << 32) == 9                    # strides beyond 32 bits
    assert call(hq=1 << 20, tokens=1 << 12) == 9    # rows beyond 32 bits
    assert call(qs=100) == 1 and call(q=p + 8) == 1 and call(w=p + 4) == 1
    assert call(hk=2, k=p) == 1 and call(hk=2, ko=p) == 1 and call(hk=-1) == 1
    assert call(pos=None) == 1
    for rd in (0, 8, 24, 144, -16):
        assert call(rd=rd) == 1
    assert call(tokens=0, q=None, qo=None) == 0     # nothing to do


def test_packed_structs_match_the_header(J):
    """The binding's packed layouts against the structs of the header, compiled by the host compiler."""
    import os
    import subprocess
    import tempfile
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    with tempfile.TemporaryDirectory() as d:
        src = os.path.join(d, "s.c")
        with open(src, "w") as f:
            f.write('#include <stddef.h>\n#include <stdio.h>\n#include "jolt.h"\nint main(void) { printf("%zu %zu %zu %zu %zu",'
                    'offsetof(jolt_norm_rope, eps), offsetof(jolt_new_rows, eps), offsetof(jolt_queries, scale),'
                    'sizeof(jolt_batch), sizeof(jolt_page_shape)); return 0; }')
        exe = os.path.join(d, "s")
        subprocess.run(["gcc", "-I", os.path.join(root, "include"), src, "-o", exe], check=True)
        got = [int(x) for x in subprocess.run([exe], capture_output=True, text=True, check=True).stdout.split()]
    assert got == [J._NORM_ROPE.size - 4, J._NEW_ROWS.size - 4, J._QUERIES.size - 4, ctypes.sizeof(J.BatchDesc),
                   ctypes.sizeof(J.PageShape)]


def test_the_codec_has_no_f16(J, untouched):
    """The type of pages that the codec's caches do not have is refused there."""
    with pytest.raises(J.JoltError) as e:
        J.jolt_plan(2, 8, 64, 128, True, J.JOLT_F16, 10 ** 6, 1)
    assert e.value.status == 1
    keep, p = _buf()
    d = ctypes.c_double()
    assert J._lib.jolt_rel_frob_error(p, p, 16, J.JOLT_F16, None, ctypes.byref(d)) == 1


def test_pages_whose_head_stride_is_beyond_32_bits(J, untouched):
    keep, p = _buf()
    h = ctypes.c_void_p()
    sh = J.PageShape(1, 1, 1 << 24, 128, 0)
    assert J._lib.jolt_pages_create(ctypes.byref(sh), p, p, None, ctypes.byref(h)) == 9 and not h.value


def test_output_rows_that_overlap_are_refused(J, untouched):
    """Rows written over one another (an expanded output, a token stride shorter than a token) leave results that
    depend on their order. Layouts that look odd but keep their rows apart are none of them: those get as far as the
    next check, of the weights' alignment."""
    keep, p = _buf()

    def call(tokens, hq, qts, qhs, hk=0, kts=0, khs=0):
        return J._lib.jolt_qk_norm_rope(J._NORM_ROPE.pack(p, 128, 128, p + 2, p, qts, qhs, p if hk else 0, 128, 128, 0,
                                                          p if hk else 0, kts, khs, 0, 0, 0, tokens, hq, hk, 0, 0, 1e-6), None)

    def said():
        return J._lib.jolt_last_error().decode()

    for a in ((2, 1, 0, 128), (1, 2, 256, 0), (2, 2, 128, 128), (3, 4, 504, 128), (2, 2, 256, 120), (9, 5, 128, 1024),
              (4, 3, 256, 384), (2, 1, -64, 128), (7, 2, 128, -640)):
        assert call(*a) == 1 and "overlap" in said(), a
        assert call(a[0], 1, 128, 0, a[1], a[2], a[3]) == 1 and "overlap" in said(), a
    for a in ((1, 1, 0, 0), (2, 2, 256, 128), (5, 3, 128, 640), (3, 2, 256, 384), (3, 2, -256, 128), (2, 3, 384, 256),
              (5, 40, 40 * 128 + 8, 128)):
        assert call(*a) == 1 and "weights" in said(), (a, said())
