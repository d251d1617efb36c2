"""Caches whose k and v lie in one buffer: refused where a row of v shares elements
with a row of k, accepted where they only lie between one another.  Nothing is
launched (no moves, no tokens)."""
import ctypes
import itertools
import random

import pytest

from packed_varlen_non_gb300 import h3attn as H

K = 1 << 40


def status(lib, n, strides, delta):
    """Of a cache with n = (pages, tokens, heads) and v `delta` elements behind k."""
    c = H.h3attn_cache(K, K + 2 * delta, *n, *strides)
    of = {lib.load().h3attn_cache_move(ctypes.byref(c), None, None, 0, 1, None),
          lib.load().h3attn_rotary_store(ctypes.byref(H.h3attn_rope_init()), None, 0, None, 0, None, 0, 0, None, None, 0, ctypes.byref(c),
                                         None, None)}
    assert len(of) == 1
    return of.pop()


def meet(n, strides, delta):
    rows = [sum(i * s for i, s in zip(at, strides)) for at in itertools.product(*(range(x) for x in n))]
    return any(abs(a + delta - b) < 128 for a in rows for b in rows)


# pages, tokens, heads and strides: tokens' heads together, heads' tokens together, room between, single ones
LAYOUTS = [((4, 8, 2), (2048, 256, 128)), ((4, 8, 2), (4096, 256, 128)), ((3, 4, 2), (4096, 512, 128)), ((3, 4, 2), (4096, 512, 256)),
           ((3, 4, 3), (4096, 128, 1024)), ((1, 4, 2), (8, 512, 128)), ((2, 1, 3), (1024, 8, 256)), ((5, 3, 1), (1024, 136, 64)),
           ((1, 1, 1), (0, 0, 0)), ((2, 3, 2), (136, 4096, 512))]


@pytest.mark.parametrize("n,strides", LAYOUTS)
def test_shared_elements_are_refused(lib, n, strides):
    span = 128 + sum((x - 1) * s for x, s in zip(n, strides))
    near = {0, 8, 120, 128, 136, 256, span - 8, span, span + 8, *strides, *(s // 2 for s in strides), *(s - 128 for s in strides)}
    rng = random.Random(5)
    near |= {8 * rng.randrange(0, span // 8 + 2) for _ in range(60)}
    for delta in sorted(x // 8 * 8 for x in near):
        for sign in (1, -1):
            want = H.H3ATTN_EINVAL if meet(n, strides, sign * delta) else H.H3ATTN_OK
            assert status(lib, n, strides, sign * delta) == want, (delta, sign)


def test_usual_buffers_are_accepted(lib):
    page, heads = 16, 8
    for strides, delta in (((2 * page * heads * 128, heads * 128, 128), page * heads * 128),       # [pages, 2, page, heads, 128]
                           ((2 * page * heads * 128, 2 * heads * 128, 128), heads * 128),          # [pages, page, 2, heads, 128]
                           ((2 * page * heads * 128, 2 * heads * 128, 256), 128),                  # [pages, page, heads, 2, 128]
                           ((page * heads * 128, heads * 128, 128), 1000 * page * heads * 128),    # [2, pages, page, heads, 128]
                           ((6 * page * heads * 128, 128, page * 128), 3 * page * heads * 128)):   # head-major, layers between
        assert status(lib, (1000, page, heads), strides, delta) == H.H3ATTN_OK
        assert status(lib, (1000, page, heads), strides, -delta) == H.H3ATTN_OK


def test_what_was_taken_for_two_tensors(lib):
    # v one head, one token or a few elements into k's rows
    for delta in (128, 256, 8, 64, -128, 2048, 2048 * 3):
        assert status(lib, (4, 8, 2), (2048, 256, 128), delta) == H.H3ATTN_EINVAL
    # far apart, with strides as large as they may be (half a stride away, and three of them)
    for delta in (1 << 45, -(1 << 37)):
        assert status(lib, (4, 8, 2), (1 << 38, 256, 128), delta) == H.H3ATTN_OK
    assert status(lib, (4, 8, 2), (1 << 38, 256, 128), 3 << 38) == H.H3ATTN_EINVAL
