"""Refusals of the rotary and cache calls that need no GPU: nothing is launched,
so plain numbers stand for the pointers."""
import ctypes
import math

import pytest
import torch

from packed_varlen_non_gb300 import h3attn as H

E, U = H.H3ATTN_EINVAL, H.H3ATTN_EUNSUPPORTED
Q, K, Q2, K2, POS, LIST = (1 << 40, 2 << 40, 3 << 40, 4 << 40, 5 << 40, 6 << 40)
KC, VC = 7 << 40, 8 << 40


def status(fn):
    with pytest.raises(H.H3AttnError) as e:
        fn()
    return e.value.status


@pytest.mark.parametrize("kw,want", [
    (dict(rope_dims=0), U), (dict(rope_dims=24), U), (dict(rope_dims=144), U), (dict(rope_dims=-16), U),
    (dict(base=1.0), E), (dict(base=math.nan), E), (dict(base=math.inf), E), (dict(scaling="linear", factor=0.5), E),
    (dict(scaling="ntk", factor=math.nan), E), (dict(scaling="ntk", factor=1e300, rope_dims=16), E),
    (dict(scaling="parts", factor=2.0), E), (dict(scaling="parts", factor=2.0, original_len=math.inf), E),
    (dict(scaling="parts", factor=2.0, original_len=100, beta_fast=1.0), E),
    (dict(scaling="parts", factor=2.0, original_len=100, beta_slow=-1.0), E),
    (dict(scaling="parts", factor=2.0, original_len=100, beta_slow=math.nan), E),
    (dict(amplitude=-1.0), E), (dict(amplitude=math.nan), E), (dict(amplitude=math.inf), E),
    (dict(n_axes=4), E), (dict(n_axes=-1), E), (dict(axes=[2] * 64, n_axes=2), E)])
def test_rope_init(lib, kw, want):
    assert status(lambda: H.h3attn_rope_init(**kw)) == want


def test_rope_init_values(lib):
    for bad in (dict(scaling="other"), dict(axes=[0] * 63), dict(axes=[3] * 64), dict(axes=[-1] * 64)):
        with pytest.raises(ValueError):
            H.h3attn_rope_init(**bad)
    assert lib.load().h3attn_rope_init(None, ctypes.byref(H.h3attn_rope())) == E
    assert lib.load().h3attn_rope_init(ctypes.byref(H.h3attn_rope_opts()), None) == E


def rotary(lib, **kw):
    a = dict(rope=H.h3attn_rope_init(), pos=POS, n=10, q=Q, qs=512, q2=Q2, q2s=512, h=4, k=K, ks=256, k2=K2, k2s=256, hk=2)
    a.update(kw)
    r = ctypes.byref(a["rope"]) if a["rope"] is not None else None
    return lib.load().h3attn_rotary(r, a["pos"], a["n"], a["q"], a["qs"], a["q2"], a["q2s"], a["h"], a["k"], a["ks"], a["k2"],
                                    a["k2s"], a["hk"], 0, None)


def unfilled(**kw):
    r = H.h3attn_rope_init()
    for name, x in kw.items():
        setattr(r, name, x)
    return r


def test_rotary(lib):
    bad_axis = H.h3attn_rope_init()
    bad_axis.axis[40] = 1
    for kw in (dict(rope=None), dict(pos=None), dict(pos=POS + 2), dict(n=-1), dict(n=1 << 31), dict(q=None), dict(q2=None),
               dict(k=None), dict(k2=None), dict(q=None, q2=None, k=None, k2=None), dict(q=Q + 8), dict(k2=K2 + 2), dict(qs=511),
               dict(qs=504), dict(q2s=516), dict(ks=248), dict(h=0), dict(h=-4), dict(hk=0), dict(h=1 << 21, qs=1 << 30, q2s=1 << 30),
               dict(qs=1 << 62), dict(rope=H.h3attn_rope()), dict(rope=unfilled(rope_dims=24)), dict(rope=unfilled(n_axes=0)),
               dict(rope=unfilled(interleaved=2)), dict(rope=bad_axis),
               # overlaps: shifted rows, other strides, each other, positions
               dict(q2=Q + 1024), dict(q2=Q + 256), dict(q2=Q, q2s=1024), dict(k2=Q), dict(k2=Q2), dict(k2=Q2 + 512),
               dict(q2=K), dict(k=K, k2=K, k2s=512), dict(q2=POS - 16)):
        assert rotary(lib, **kw) == E, kw
    # windows of one buffer that do not touch are no overlap (refused for another reason: the last argument)
    assert rotary(lib, n=0, pos=None, q=None, q2=None, k=None, k2=None) == H.H3ATTN_OK


def cache(**kw):
    a = dict(k=KC, v=VC, n_pages=4, page_size=8, num_kv_heads=2, page_stride=2048, token_stride=256, head_stride=128)
    a.update(kw)
    return H.h3attn_cache(*a.values())


BAD_CACHES = [dict(k=None), dict(v=None), dict(k=KC + 8), dict(v=VC + 2), dict(n_pages=0), dict(page_size=0), dict(num_kv_heads=0),
              dict(n_pages=1 << 28), dict(page_stride=2047), dict(page_stride=2040), dict(token_stride=128), dict(head_stride=120),
              dict(head_stride=0), dict(token_stride=0), dict(page_stride=0), dict(page_stride=-2048), dict(head_stride=2048),
              dict(page_stride=1 << 39), dict(v=KC)]


def store(lib, **kw):
    a = dict(rope=H.h3attn_rope_init(), pos=POS, n=10, q=Q, qs=512, q2=Q2, q2s=512, h=4, k=K, v=K2, ks=256, cache=cache(), slots=LIST)
    a.update(kw)
    c = ctypes.byref(a["cache"]) if a["cache"] is not None else None
    return lib.load().h3attn_rotary_store(ctypes.byref(a["rope"]), a["pos"], a["n"], a["q"], a["qs"], a["q2"], a["q2s"], a["h"],
                                          a["k"], a["v"], a["ks"], c, a["slots"], None)


def test_store(lib):
    for kw in (dict(pos=None), dict(slots=None), dict(slots=LIST + 1), dict(cache=None), dict(q=None), dict(q2=None), dict(k=None),
               dict(v=None), dict(ks=248), dict(ks=260), dict(qs=504), dict(h=0), dict(q2=Q + 16), dict(q2=K), dict(q2=K2 + 256),
               dict(k=KC), dict(v=VC + 64), dict(q2=KC), dict(q=VC), dict(slots=KC), dict(pos=VC), dict(q2=LIST - 256)):
        assert store(lib, **kw) == E, kw
    for kw in BAD_CACHES:
        assert store(lib, cache=cache(**kw)) == E, kw
    assert store(lib, n=0, pos=None, slots=None, k=None, v=None) == H.H3ATTN_OK


def test_move(lib):
    def move(c=cache(), src=LIST, dst=POS, n=3, width=4):
        return lib.load().h3attn_cache_move(ctypes.byref(c) if c is not None else None, src, dst, n, width, None)
    for kw in (dict(c=None), dict(src=None), dict(dst=None), dict(src=LIST + 2), dict(dst=POS + 1), dict(n=-1), dict(n=1 << 31),
               dict(src=KC + 128), dict(dst=VC)):
        assert move(**kw) == E, kw
    for kw in BAD_CACHES:
        assert move(c=cache(**kw)) == E, kw
    for kw in (dict(width=0), dict(width=257), dict(c=cache(num_kv_heads=32768, token_stride=1 << 22, page_stride=1 << 25))):
        assert move(**kw) == U, kw
    assert move(n=0, src=None, dst=None) == H.H3ATTN_OK


def test_the_tree_calls_refuse_a_null_plan(lib):
    assert status(lambda: H.h3attn_plan_set_tree(None, 1, stream=0)) == E
    assert lib.load().h3attn_forward_tree(None, Q, 512, ctypes.byref(cache()), POS, 4, LIST, None, Q2, 512, 0.1, None, None) == E


def test_a_cache_whose_size_passes_64_bits(lib):
    # (its span would wrap around to a small one)
    for kw in (dict(n_pages=1 << 27, page_stride=1 << 38), dict(n_pages=1 << 24, page_stride=1 << 37),
               dict(page_size=1 << 28, n_pages=1, token_stride=1 << 36)):
        assert store(lib, cache=cache(**kw)) == E, kw
        assert lib.load().h3attn_cache_move(ctypes.byref(cache(**kw)), LIST, POS, 3, 4, None) == E, kw


def test_the_binding_refuses_host_tensors(lib):
    # all of them: each agrees with the others on its device
    rope, n = H.h3attn_rope_init(), 4
    q = [torch.zeros(n, 2, 128, dtype=torch.bfloat16) for _ in range(4)]
    pos = torch.zeros(n, dtype=torch.int32)
    for args in ((q[0], q[1]), (q[0], q[1], q[2], q[3]), (None, None, q[2], q[3])):
        with pytest.raises(ValueError, match="GPU"):
            H.h3attn_rotary(rope, pos, *args)
    with pytest.raises(ValueError, match="GPU"):
        H.Cache(torch.zeros(2, 8, 2, 128, dtype=torch.bfloat16), torch.zeros(2, 8, 2, 128, dtype=torch.bfloat16))
