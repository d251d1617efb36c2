"""Rotary positions and the cache's row moves on the GPU, against the fp64
oracle: layouts, dims, scalings, axes, far positions, strides, slots, and the
ways a program calls them."""
import numpy as np
import pytest
import torch

from oracle import serving
from packed_varlen_non_gb300 import h3attn as H
from tests import walk_cases as W

pytestmark = pytest.mark.gpu


def check(got, x, want, amplitude=1.0):
    """One rounding to bf16 (2^-8 of the value), and fp32 arithmetic on two terms:
    the angle's conversion (2^-25 of a half turn: 2^-23 radians), sine and cosine (two steps, 2^-22), the
    products and their sum (2^-23) add up to less than 2^-20 (|a| + |b|)."""
    x = W.f64(x)
    pair = np.abs(x).max(axis=-1, keepdims=True) * 2 * amplitude
    bad = ~(np.abs(W.f64(got) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -20 * pair)
    assert not bad.any(), f"{int(bad.sum())} out of tolerance, first at {np.argwhere(bad)[0]}"


def positions(n, axes, seed, far=5000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (axes, n), generator=g).to(torch.int32)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("dims", [16, 32, 48, 96, 112, 128])
@pytest.mark.parametrize("n,heads,kv", [(1, 1, 1), (3, 7, 1), (33, 28, 4), (700, 5, 5)])
def test_rotary_matches_the_oracle(lib, n, heads, kv, dims, interleaved):
    q, k, pos = W.rows(n, heads, 1), W.rows(n, kv, 2), positions(n, 1, 3)
    rope = H.h3attn_rope_init(dims, 1e4, interleaved=interleaved)
    f, _ = serving.frequencies(dims, 1e4)
    q2, k2 = torch.full_like(q, float("nan")), torch.full_like(k, float("nan"))
    H.h3attn_rotary(rope, pos.cuda(), q, q2, k, k2)
    check(q2, q, serving.rotate(W.f64(q), pos.numpy(), f, interleaved=interleaved))
    check(k2, k, serving.rotate(W.f64(k), pos.numpy(), f, interleaved=interleaved))
    assert torch.equal(q2[..., dims:], q[..., dims:])
    # each alone, and in place, give the same bits
    q3, k3 = q.clone(), torch.empty_like(k)
    H.h3attn_rotary(rope, pos[0].cuda(), q3, q3)
    H.h3attn_rotary(rope, pos.cuda(), None, None, k, k3)
    assert torch.equal(q3, q2) and torch.equal(k3, k2)


@pytest.mark.parametrize("scaling,factor", [("linear", 8.0), ("ntk", 4.0), ("parts", 4.0), ("none", 1.0)])
@pytest.mark.parametrize("axes", [1, 2, 3])
def test_scalings_axes_and_the_inverse(lib, scaling, factor, axes):
    n, dims = 77, 128
    line = [j % axes for j in range(dims // 2)] if axes != 2 else [0] * 20 + [1] * 44
    rope = H.h3attn_rope_init(dims, 1e6, scaling=scaling, factor=factor, original_len=4096, axes=line)
    f, a = serving.frequencies(dims, 1e6, scaling, factor, 4096)
    q, pos = W.rows(n, 3, 4), positions(n, axes, 5)
    q2, q3 = torch.empty_like(q), torch.empty_like(q)
    H.h3attn_rotary(rope, pos.cuda(), q, q2)
    check(q2, q, serving.rotate(W.f64(q), pos.numpy(), f, a, line), a)
    H.h3attn_rotary(rope, pos.cuda(), q, q3, inverse=True)
    check(q3, q, serving.rotate(W.f64(q), pos.numpy(), f, a, line, inverse=True), a)


def test_the_inverse_is_the_gradient(lib):
    # <g, R x> = <R^T g, x>: exact up to the two roundings to bf16
    n, rope, pos = 40, H.h3attn_rope_init(96, 1e4, interleaved=True, amplitude=1.25), positions(40, 1, 6).cuda()
    x, g = W.rows(n, 2, 7), W.rows(n, 2, 8)
    y, back = torch.empty_like(x), torch.empty_like(x)
    H.h3attn_rotary(rope, pos, x, y)
    H.h3attn_rotary(rope, pos, g, back, inverse=True)
    a, b = g.double() * y.double(), back.double() * x.double()
    tol = 2.0 ** -8 * (a.abs().sum(-1) + b.abs().sum(-1)) + 1e-5 * 1.25 * (g.double().norm(dim=-1) * x.double().norm(dim=-1))
    assert ((a.sum(-1) - b.sum(-1)).abs() <= tol).all()
    # and against differences of the rotation itself (a linear map: one step is exact up to the roundings)
    for lane in (0, 1, 40, 95, 100):
        e = torch.zeros_like(x)
        e[..., lane] = 1.0
        H.h3attn_rotary(rope, pos, e, y)
        want = (g.double() * y.double()).sum(-1)
        tol = 2.0 ** -8 * ((g.double() * y.double()).abs().sum(-1) + want.abs()) + 1e-5 * g.double().norm(dim=-1)
        assert ((back[..., lane].double() - want).abs() <= tol).all()


def test_far_and_negative_positions(lib):
    # (the oracle's angle: position times frequency modulo a turn in exact arithmetic)
    far = [0, 1, -1, 2 ** 31 - 1, -2 ** 31, 10 ** 6, 123456789, -987654321]
    pos = torch.tensor([far], dtype=torch.int32)
    q = W.rows(len(far), 2, 9)
    rope = H.h3attn_rope_init(128, 1e6)
    q2 = torch.empty_like(q)
    H.h3attn_rotary(rope, pos.cuda(), q, q2)
    turns = np.array([[(p * int(rope.turns[j])) % 2 ** 64 / 2.0 ** 64 for j in range(64)] for p in far])
    c, s = np.cos(2 * np.pi * turns)[:, None], np.sin(2 * np.pi * turns)[:, None]
    x = W.f64(q)
    a, b = x[..., :64], x[..., 64:]
    check(q2, q, np.concatenate([a * c - b * s, b * c + a * s], -1))
    # at a million the fp64 product is good to 2^-30
    f, _ = serving.frequencies(128, 1e6)
    check(q2[5:6], q[5:6], serving.rotate(x[5:6], [[10 ** 6]], f))


def test_a_fused_buffer_in_place_and_guards(lib):
    n, heads, kv = 50, 6, 2
    w = (heads + 2 * kv) * 128
    buf = torch.randn(n + 1, w + 8, device="cuda").to(torch.bfloat16)
    q, k = buf[:n, :heads * 128].view(n, heads, 128), buf[:n, heads * 128:(heads + kv) * 128].view(n, kv, 128)
    before, rope, pos = buf.clone(), H.h3attn_rope_init(64, 1e4), positions(n, 1, 10).cuda()
    q2, k2 = torch.empty(n, heads, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(n, kv, 128, dtype=torch.bfloat16, device="cuda")
    H.h3attn_rotary(rope, pos, q, q2, k, k2)
    assert torch.equal(buf, before)
    H.h3attn_rotary(rope, pos, q, q, k, k)
    assert torch.equal(q, q2) and torch.equal(k, k2)
    assert torch.equal(buf[:, (heads + kv) * 128:], before[:, (heads + kv) * 128:]) and torch.equal(buf[n], before[n])


def caches(pages, page, kv, head_major, seed=0):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for _ in range(2):
        shape = (pages, kv, page, 128) if head_major else (pages, page, kv, 128)
        x = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        out.append(x.transpose(1, 2) if head_major else x)
    return out


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("n,heads,kv,page", [(1, 4, 1, 8), (37, 8, 2, 16), (300, 3, 3, 5), (5, 2, 2, 1)])
def test_store_puts_rows_into_their_slots(lib, n, heads, kv, page, head_major):
    pages = -(-n // page) + 2
    kc, vc = caches(pages, page, kv, head_major)
    cache, total = H.Cache(kc, vc), pages * page
    q, k, v, pos = W.rows(n, heads, 11), W.rows(n, kv, 12), W.rows(n, kv, 13), positions(n, 1, 14).cuda()
    slots = torch.randperm(total, generator=torch.Generator().manual_seed(15))[:n].to(torch.int32)
    if n > 4:  # padding and slots that are no rows of the cache
        slots[0], slots[1], slots[2], slots[3] = -1, total, 2 ** 31 - 1, -2 ** 31
    rope = H.h3attn_rope_init(128, 1e5, interleaved=True)
    q2, k2, q3 = torch.empty_like(q), torch.empty_like(k), torch.empty_like(q)
    H.h3attn_rotary(rope, pos, q, q2, k, k2)
    want = [kc.clone().reshape(total, kv, 128), vc.clone().reshape(total, kv, 128)]
    there = (slots >= 0) & (slots < total)
    at = slots[there].long().cuda()
    want[0][at], want[1][at] = k2[there.cuda()], v[there.cuda()]
    H.h3attn_rotary_store(rope, pos, q, q3, k, v, cache, slots.cuda())
    assert torch.equal(q3, q2)
    assert torch.equal(kc.reshape(total, kv, 128), want[0]) and torch.equal(vc.reshape(total, kv, 128), want[1])
    # without q, the same rows again
    H.h3attn_rotary_store(rope, pos, None, None, k, v, cache, slots.cuda())
    assert torch.equal(kc.reshape(total, kv, 128), want[0]) and torch.equal(vc.reshape(total, kv, 128), want[1])


@pytest.mark.parametrize("head_major", [False, True])
@pytest.mark.parametrize("groups,width,page,kv", [(1, 1, 8, 1), (5, 16, 16, 2), (3, 17, 8, 3), (7, 64, 64, 1), (2, 65, 16, 2),
                                                  (2, 256, 7, 1)])
def test_moves_match_the_oracle(lib, groups, width, page, kv, head_major):
    pages = -(-2 * groups * width // page) + 1
    kc, vc = caches(pages, page, kv, head_major)
    total, g = pages * page, np.random.default_rng(16)
    own = g.permutation(total)[:2 * groups * width].reshape(groups, 2 * width)  # slots of one group only
    src = np.stack([g.choice(x, width) for x in own]).astype(np.int32)           # any of them, some twice
    dst = np.stack([g.permutation(x)[:width] for x in own]).astype(np.int32)     # sources among them
    if width > 3:
        src[0, 0], dst[0, 1], src[0, 2], dst[0, 3] = -1, -1, total, 2 ** 31 - 1
    want = [serving.moved(W.f64(c.float()).reshape(total, kv, 128), src, dst) for c in (kc, vc)]
    H.h3attn_cache_move(H.Cache(kc, vc), torch.from_numpy(src).cuda(), torch.from_numpy(dst).cuda())
    for c, w in zip((kc, vc), want):
        assert np.array_equal(W.f64(c.float()).reshape(total, kv, 128), w)


def test_nothing_to_do(lib):
    kc, vc = caches(2, 8, 2, False)
    before, none = kc.clone(), torch.empty(0, dtype=torch.int32, device="cuda")
    e = torch.empty(0, 2, 128, dtype=torch.bfloat16, device="cuda")
    rope = H.h3attn_rope_init()
    H.h3attn_rotary(rope, none, e, e, e, e)
    H.h3attn_rotary_store(rope, none, e, e, e, e, H.Cache(kc, vc), none)
    H.h3attn_cache_move(H.Cache(kc, vc), none.view(0, 4), none.view(0, 4))
    torch.cuda.synchronize()
    assert torch.equal(kc, before)


def test_offsets_past_32_bits(lib):
    # tokens and pages a megabyte of elements apart: the last ones lie past 2^32 bytes
    n, stride = 2200, 1 << 20
    big = torch.empty(n, stride, dtype=torch.bfloat16, device="cuda")
    q, k, v, pos = W.rows(n, 1, 17), W.rows(n, 1, 18), W.rows(n, 1, 19), positions(n, 1, 20).cuda()
    rope = H.h3attn_rope_init(128, 1e4)
    ref, kref = torch.empty_like(q), torch.empty_like(k)
    H.h3attn_rotary(rope, pos, q, ref, k, kref)
    far = [big[:, 256 * i:256 * i + 128].unflatten(1, (1, 128)) for i in range(4)]
    for x, y in zip(far, (q, k, v)):
        x.copy_(y)
    pool = torch.empty(n, stride, dtype=torch.bfloat16, device="cuda")  # (no byte range shared with the rows)
    kc, vc = (pool[:, 256 * i:256 * i + 128].view(n, 1, 1, 128) for i in range(2))
    slots = torch.arange(n - 1, -1, -1, dtype=torch.int32, device="cuda")
    H.h3attn_rotary_store(rope, pos, far[0], far[3], far[1], far[2], H.Cache(kc, vc), slots)
    assert torch.equal(far[3], ref) and torch.equal(kc[:, 0].flip(0), kref) and torch.equal(vc[:, 0].flip(0), v)
    src = torch.tensor([[n - 1, 0]], dtype=torch.int32, device="cuda")
    H.h3attn_cache_move(H.Cache(kc, vc), src, src.flip(1).contiguous())
    assert torch.equal(kc[0, 0], kref[0]) and torch.equal(kc[n - 1, 0], kref[n - 1]) and torch.equal(vc[n - 1, 0], v[n - 1])


def test_streams_and_capture(lib):
    n, heads, kv, page = 20, 4, 2, 8
    kc, vc = caches(6, page, kv, False)
    cache, rope = H.Cache(kc, vc), H.h3attn_rope_init(96, 1e4)
    q, k, v, pos = W.rows(n, heads, 21), W.rows(n, kv, 22), W.rows(n, kv, 23), positions(n, 1, 24).cuda()
    slots = torch.arange(10, 10 + n, dtype=torch.int32, device="cuda")
    src = torch.tensor([[10, 11, 29]], dtype=torch.int32, device="cuda")
    dst = torch.tensor([[0, 1, 2]], dtype=torch.int32, device="cuda")
    q2 = torch.empty_like(q)

    def step(stream=None):
        H.h3attn_rotary_store(rope, pos, q, q2, k, v, cache, slots, stream=stream)
        H.h3attn_cache_move(cache, src, dst, stream=stream)

    side = torch.cuda.Stream()
    step(side)
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        step()
    for seed in (30, 40):
        for x, s in ((q, 0), (k, 1), (v, 2)):
            x.copy_(W.rows(n, x.shape[1], seed + s))
        pos.copy_(positions(n, 1, seed + 3))
        for x in (q2, kc, vc):
            x.zero_()
        graph.replay()
        got = [x.clone() for x in (q2, kc, vc)]
        for x in (q2, kc, vc):
            x.zero_()
        step()
        assert all(torch.equal(x, y) for x, y in zip(got, (q2, kc, vc)))
        assert torch.equal(kc.view(-1, kv, 128)[[0, 1, 2]], kc.view(-1, kv, 128)[[10, 11, 29]])


def test_the_binding_refuses_other_tensors(lib):
    n, heads, kv = 10, 4, 2
    kc, vc = caches(4, 8, kv, False)
    q, k, v, pos = W.rows(n, heads, 31), W.rows(n, kv, 32), W.rows(n, kv, 33), positions(n, 1, 34).cuda()
    rope, cache, slots = H.h3attn_rope_init(), H.Cache(kc, vc), torch.arange(n, dtype=torch.int32, device="cuda")
    rot = dict(rope=rope, positions=pos, q_in=q, q_out=torch.empty_like(q), k_in=k, k_out=torch.empty_like(k))
    store = dict(rope=rope, positions=pos, q_in=q, q_out=torch.empty_like(q), k_in=k, v_in=v, cache=cache, slots=slots)
    move = dict(cache=cache, src=slots.view(2, 5), dst=(slots + 16).view(2, 5))
    for fn, kw, names in ((H.h3attn_rotary, rot, "positions q_in q_out k_in k_out"),
                          (H.h3attn_rotary_store, store, "positions q_in q_out k_in v_in slots"),
                          (H.h3attn_cache_move, move, "src dst")):
        fn(**kw)
        for name in names.split():
            t = kw[name]
            bads = [t.cpu(), t[:-1] if t.dim() != 2 or name in ("src", "dst") else t[:, :-1], t.double()]
            if t.dtype is torch.int32:
                bads += [t.long(), torch.stack([t, t], -1)[..., 0]]
            else:
                bads += [t.half(), t.reshape(n, -1), t.transpose(0, 1), t[:, :, :64], t[:, :1].expand(-1, 2, -1)]
            for bad in bads:
                if name == "src" and bad.shape != t.shape:
                    continue  # (its shape is what dst is held to)
                with pytest.raises(ValueError):
                    fn(**{**kw, name: bad})
    with pytest.raises(ValueError):
        H.h3attn_rotary(rope, pos, q, None)
    with pytest.raises(ValueError):
        H.h3attn_rotary(rope, pos, q, k.clone(), k, torch.empty_like(k))
    for a, b in ((kc, vc.float()), (kc, vc[:3]), (kc.cpu(), vc.cpu()), (kc[..., :64], vc[..., :64]),
                 (kc.transpose(2, 3), vc.transpose(2, 3)), (kc, vc.transpose(0, 1).contiguous().transpose(0, 1))):
        with pytest.raises(ValueError):
            H.Cache(a, b)
    # the library's own refusals reach the caller
    wide = torch.empty(2 * n, heads, 128, dtype=torch.bfloat16, device="cuda")
    with pytest.raises(H.H3AttnError):
        H.h3attn_rotary(rope, pos, wide[:n], wide[1:n + 1])
    with pytest.raises(H.H3AttnError):
        H.h3attn_rotary_store(**{**store, "v_in": vc.view(-1, kv, 128)[:n]})
    with pytest.raises(H.H3AttnError):
        H.h3attn_cache_move(H.Cache(kc, kc), slots.view(2, 5), slots.view(2, 5))
    torch.cuda.synchronize()
