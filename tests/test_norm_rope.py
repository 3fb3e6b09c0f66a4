"""Norm and rotation of query and key heads, and the norm-and-rotate write into the latent
cache, against the formulas in 64 bits.

Tolerance: the kernels compute in fp32 and round once to bf16.  The sum of squares, the
reciprocal root and the products are off by at most 2^-18 of an element, the rotation adds
two roundings, so before the last rounding a result is off by at most 2^-17 (|a| + |b|)
<= 2^-16 of the row's largest normed element; the rounding to bf16 adds half a step, 2^-8
of the value."""
import ctypes

import numpy as np
import pytest
import torch

EPS = 1e-6


# ------------------------------------------------------------------ the formulas, 64 bits
def table_of(rows, rot, device="cuda"):
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    ang = torch.arange(rows, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def ref_norm(x, w):
    x = x.double()
    if w is None:
        return x
    return x / (x.square().mean(-1, keepdim=True) + EPS).sqrt() * w.double()


def ref_rotate(x, pos, table, inter):
    rot = x.shape[-1]
    row = table.double()[pos.long()].view(x.shape[0], *([1] * (x.dim() - 2)), rot)
    c, s = row[..., : rot // 2], row[..., rot // 2:]
    out = torch.empty_like(x)
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else (x[..., : rot // 2], x[..., rot // 2:])
    first, second = a * c - b * s, a * s + b * c
    if inter:
        out[..., 0::2], out[..., 1::2] = first, second
    else:
        out[..., : rot // 2], out[..., rot // 2:] = first, second
    return out


def ref_heads(x, w, pos, table, off, inter):
    y = ref_norm(x, w)
    rot = table.shape[1]
    z = y.clone()
    z[..., off:off + rot] = ref_rotate(y[..., off:off + rot], pos, table, inter)
    return y, z


def within(got, ref, normed):
    tol = 2.0 ** -8 * ref.abs() + 2.0 ** -16 * normed.abs().amax(-1, keepdim=True)
    d = (got.double() - ref).abs()
    assert torch.isfinite(got.double()).all()
    assert bool((d <= tol).all()), float((d / tol.clamp_min(1e-300)).max())


def normal(*shape, seed=0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return torch.randn(*shape, generator=g, device="cuda").to(torch.bfloat16)


# ------------------------------------------------------------------ refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_kd_b200 import build
    build.build()
    from tree_speculative_decoding_kd_b200 import kd
    return kd.lib


def test_host_validation(lib):
    V = ctypes.c_void_p
    qk = [V(16), 512, 128, V(16), 512, 128, V(16), V(16), 1e-6, V(16), 100, V(16), 4, 4, 4, 128, 128, 0, 0,
          V(16), 512, 128, V(16), 512, 128, None, None]
    for i, v in ((0, None), (0, V(8)), (1, 12), (2, -8), (3, None), (8, -1.0), (8, float("nan")), (9, None), (9, V(4)),
                 (10, 0), (11, None), (12, -1), (13, 0), (14, -1), (15, 12), (15, 264), (16, 8), (16, 144), (17, 4),
                 (17, 16), (19, None), (22, V(24)), (20, 4), (6, V(8))):
        bad = list(qk)
        bad[i] = v
        assert lib.kd_qk_norm_rope(*bad) == -1, i
    bad = list(qk)
    bad[12], bad[13] = 1 << 30, 4                      # T (H + Hk) beyond 32 bits
    assert lib.kd_qk_norm_rope(*bad) == -1
    none = list(qk)
    none[12] = 0                                        # no tokens: nothing to do
    assert lib.kd_qk_norm_rope(*none) == 0
    wr = [V(16), V(16), 512, 64, 100, V(16), V(16), 576, V(16), 1e-6, V(16), 100, V(16), 1, V(16), 2, 8, V(16), 768,
          192, 4, V(16), None, None]
    for i, v in ((0, None), (2, 500), (3, 60), (4, 0), (5, None), (6, None), (6, V(2)), (7, 568), (7, 580), (9, -1.0),
                 (10, None), (11, 0), (15, 0), (16, -1), (16, (1 << 27) + 1), (17, None), (17, V(4)), (18, 4),
                 (20, 129), (21, None), (8, V(18))):
        bad = list(wr)
        bad[i] = v
        assert lib.kd_kv_norm_rope_write(*bad) == -1, i
    odd = list(wr)
    odd[14], odd[16] = None, 9                          # 9 tokens do not divide among 2 requests
    assert lib.kd_kv_norm_rope_write(*odd) == -1
    pg = wr[:4] + [16, V(16), 10, 100] + wr[5:]
    for i, v in ((4, 0), (5, None), (6, 0), (7, 0), (7, 1 << 30)):
        bad = list(pg)
        bad[i] = v
        assert lib.kd_kv_norm_rope_write_paged(*bad) == -1, i


def test_binding_refuses_cpu_tensors_and_shapes(lib):
    from tree_speculative_decoding_kd_b200 import kd
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    pos, table = torch.zeros(2, dtype=torch.int32), torch.zeros(8, 64)
    with pytest.raises(ValueError):
        kd.kd_qk_norm_rope(q, None, pos, table)
    with pytest.raises(ValueError):
        kd.kd_kv_norm_rope_write(torch.zeros(1, 4, 512, dtype=torch.bfloat16), torch.zeros(1, 4, 64, dtype=torch.bfloat16),
                                 pos[:1], torch.zeros(2, 576, dtype=torch.bfloat16), pos, table)


def test_formulas():
    """The reference itself: a rotation keeps a pair's length, position 0 changes nothing, and
    the two pairings are the same rotation of permuted elements."""
    g = torch.Generator().manual_seed(0)
    x = torch.randn(5, 3, 64, generator=g, dtype=torch.float64)
    table = table_of(40, 64, "cpu")
    pos = torch.tensor([0, 1, 7, 39, 2])
    for inter in (False, True):
        y = ref_rotate(x, pos, table, inter)
        assert torch.equal(y[0], x[0])
        assert torch.allclose(y.square().sum(-1), x.square().sum(-1), rtol=1e-6)
    perm = torch.cat([torch.arange(0, 64, 2), torch.arange(1, 64, 2)])
    assert torch.allclose(ref_rotate(x, pos, table, True)[..., perm], ref_rotate(x[..., perm], pos, table, False))
    ang = 7 * 10000.0 ** (-2 * 5 / 64)
    want = x[2, 0, 10] * np.cos(ang) - x[2, 0, 11] * np.sin(ang)
    assert abs(float(ref_rotate(x, pos, table, True)[2, 0, 10] - want)) < 1e-6


# ------------------------------------------------------------------ query and key heads
@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hk,D,rot,off,inter,norm", [
    (1, 1, 0, 128, 128, 0, False, True), (1, 32, 8, 128, 128, 0, False, True), (3, 5, 1, 64, 64, 0, True, True),
    (37, 7, 7, 128, 64, 64, False, True), (19, 4, 2, 192, 64, 128, True, False), (9, 3, 2, 256, 256, 0, False, True),
    (11, 6, 3, 72, 16, 8, False, True), (5, 2, 1, 16, 16, 0, True, True), (1025, 64, 8, 128, 96, 32, False, True),
    (8, 128, 128, 64, 48, 16, False, False), (17, 2, 2, 136, 112, 24, False, True)])
def test_heads(kd, T, H, Hk, D, rot, off, inter, norm):
    qkv = normal(T, H + 2 * Hk, D, seed=T)
    q, k = qkv[:, :H], qkv[:, H:H + Hk] if Hk else None
    table = table_of(5000, rot)
    pos = torch.randint(0, 5000, (T,), device="cuda", dtype=torch.int32)
    pos[0] = 4999
    qw, kw = (normal(D, seed=1), normal(D, seed=2)) if norm else (None, None)
    err = kd.new_error_word()
    qo, ko = kd.kd_qk_norm_rope(q, k, pos, table, q_weight=qw, k_weight=kw, eps=EPS, rot_offset=off, interleaved=inter,
                                dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    for x, w, got in ((q, qw, qo), (k, kw, ko)):
        if x is not None:
            y, ref = ref_heads(x, w, pos, table, off, inter)
            within(got, ref, y)


@pytest.mark.gpu
def test_heads_in_place_and_norm_of_one_side(kd):
    """In place over strided views; the values beside them stay; only the keys are normed."""
    T, H, Hk, D = 21, 6, 2, 128
    qkv = normal(T, H + 2 * Hk, D, seed=3)
    was = qkv.clone()
    table, pos = table_of(100, D), torch.arange(T, device="cuda", dtype=torch.int32)
    q, k, kw = qkv[:, :H], qkv[:, H:H + Hk], normal(D, seed=4)
    kd.kd_qk_norm_rope(q, k, pos, table, k_weight=kw, eps=EPS, q_out=q, k_out=k)
    for x, w, got in ((was[:, :H], None, q), (was[:, H:H + Hk], kw, k)):
        y, ref = ref_heads(x, w, pos, table, 0, False)
        within(got, ref, y)
    assert torch.equal(qkv[:, H + Hk:], was[:, H + Hk:])


@pytest.mark.gpu
def test_heads_bad_position_zero_rows_and_large_values(kd):
    T, H, D = 6, 4, 128
    q = normal(T, H, D, seed=5)
    q[1] = 0                                            # a head of zeros: eps keeps it finite
    q[2] = q[2] * 1e18                                  # squares near fp32's top
    table, w = table_of(50, D), normal(D, seed=6)
    pos = torch.tensor([0, 1, 2, 50, -1, 49], dtype=torch.int32, device="cuda")
    out, err = torch.full_like(q, 7.0), kd.new_error_word()
    kd.kd_qk_norm_rope(q, None, pos, table, q_weight=w, eps=EPS, q_out=out, dev_error=err)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_POSITION"]
    assert bool((out[3:5] == 7.0).all())
    ok = [0, 1, 2, 5]
    y, ref = ref_heads(q[ok], w, pos[ok], table, 0, False)
    within(out[ok], ref, y)
    assert bool((out[1] == 0).all())
    e, _ = kd.kd_qk_norm_rope(q[:0], None, pos[:0], table)
    assert e.shape == (0, H, D)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H,Hk,D,rot,off,inter", [
    (40003, 1, 1, 192, 32, 160, True), (30001, 3, 0, 64, 64, 0, False), (9001, 7, 2, 128, 48, 16, False),
    (5003, 20, 3, 72, 16, 8, True), (2501, 9, 5, 256, 240, 0, False), (20011, 1, 3, 16, 16, 0, True)])
def test_heads_of_many_tokens_in_a_row(kd, T, H, Hk, D, rot, off, inter):
    """Head counts that leave a run of heads to several tokens: the tokens' own angles, a token of
    a bad position between good ones left as it was, and the same values in place."""
    qkv = normal(T, H + 2 * Hk + 1, D, seed=T)
    q, k = qkv[:, :H], qkv[:, H:H + Hk] if Hk else None
    table, qw, kw = table_of(700, rot), normal(D, seed=1), normal(D, seed=2)
    pos = torch.randint(0, 700, (T,), device="cuda", dtype=torch.int32)
    bad = torch.zeros(T, dtype=torch.bool, device="cuda")
    bad[5::97] = True
    bad[T - 1] = bad[1000:1020] = True
    pos[bad] = torch.where(torch.arange(int(bad.sum()), device="cuda") % 2 == 0, -1, 700).int()
    outs = [torch.full_like(q, 7.0), None if k is None else torch.full_like(k, 7.0)]
    err = kd.new_error_word()
    args = dict(q_weight=qw, k_weight=kw if Hk else None, eps=EPS, rot_offset=off, interleaved=inter)
    kd.kd_qk_norm_rope(q, k, pos, table, q_out=outs[0], k_out=outs[1], dev_error=err, **args)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_POSITION"]
    was = qkv.clone()
    kd.kd_qk_norm_rope(q, k, pos, table, q_out=q, k_out=k, **args)
    for x, y, w, got in ((was[:, :H], q, qw, outs[0]), (was[:, H:H + Hk], k, kw, outs[1])):
        if got is None:
            continue
        normed, ref = ref_heads(x[~bad], w, pos[~bad], table, off, inter)
        within(got[~bad], ref, normed)
        assert bool((got[bad] == 7.0).all())
        assert torch.equal(y[~bad], got[~bad]) and torch.equal(y[bad], x[bad])
    assert torch.equal(qkv[:, H + Hk:], was[:, H + Hk:])


# ------------------------------------------------------------------ into the cache
def cache(kd, B, cap, page, wide, seed):
    """c, r, page table, rows of every slot [B][cap]; `wide`: one 576-wide interleaved buffer."""
    g = torch.Generator().manual_seed(seed)
    M = -(-cap // page) if page else 0
    rows = (B * M + 2) * page if page else B * cap
    if wide:
        buf = torch.full((rows, 576), 5.0, dtype=torch.bfloat16, device="cuda")
        c, r = buf[:, :512], buf[:, 512:]
    else:
        c = torch.full((rows, 512), 5.0, dtype=torch.bfloat16, device="cuda")
        r = torch.full((rows, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    if not page:
        return c.view(B, cap, 512) if not wide else buf.view(B, cap, 576)[..., :512], \
            r.view(B, cap, 64) if not wide else buf.view(B, cap, 576)[..., 512:], None, \
            torch.arange(B * cap).view(B, cap)
    pt = torch.randperm(B * M + 2, generator=g)[: B * M].view(B, M)
    slots = torch.arange(cap)
    return c, r, pt.int().cuda(), pt[:, slots // page] * page + slots % page


@pytest.mark.gpu
@pytest.mark.parametrize("lens,ragged,H,page,wide,inter,norm,with_pos", [
    ([1], False, 64, 0, False, True, True, True), ([17] * 5, False, 64, 0, False, True, True, True),
    ([3] * 4, False, 5, 16, False, False, True, False), ([0, 1, 130, 2, 0, 64], True, 16, 64, False, True, True, True),
    ([200, 1], True, 128, 0, True, True, True, False), ([7, 9, 1], True, 0, 1, False, False, False, True),
    ([33] * 3, False, 17, 0, True, False, True, True), ([1] * 70, True, 1, 128, False, True, True, False)])
def test_write(kd, lens, ragged, H, page, wide, inter, norm, with_pos):
    B, T = len(lens), sum(lens)
    extra = 3 if ragged else 0                          # rows behind the last sequence
    past = [(11 * b) % 40 for b in range(B)]
    cap = 40 + max(lens) + 3
    c, r, pt, rows = cache(kd, B, cap, page, wide, seed=B)
    kv = normal(T + extra, 640, seed=T)[:, :576]
    qr = normal(T + extra, H, 192, seed=T + 1)[:, :, 128:] if H else None
    w = normal(512, seed=8) if norm else None
    table = table_of(cap + 50, 64)
    at = [p + i for p, n in zip(past, lens) for i in range(n)]
    pos = torch.tensor([x + 5 for x in at] + [0] * extra, dtype=torch.int32, device="cuda") if with_pos else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda") if ragged else None
    L = torch.tensor(past, dtype=torch.int32, device="cuda")
    qo = torch.full((T + extra, H, 64), 9.0, dtype=torch.bfloat16, device="cuda") if H else None
    err = kd.new_error_word()
    more = dict(cu_seqlens=cu, kv_weight=w, eps=EPS, interleaved=inter, q_rope_in=qr, q_rope_out=qo, dev_error=err)
    if page:
        kd.kd_kv_norm_rope_write_paged(c, r, pt, page, L, kv, pos, table, **more)
    else:
        kd.kd_kv_norm_rope_write(c, r, L, kv, pos, table, **more)
    assert kd.kd_read_device_error(err) == 0
    where = torch.tensor([int(rows[b, past[b] + i]) for b, n in enumerate(lens) for i in range(n)], device="cuda")
    p = pos[:T] if with_pos else torch.tensor(at, device="cuda")
    cf, rf = (c.reshape(-1, 512), r.reshape(-1, 64))
    y = ref_norm(kv[:T, :512], w)
    within(cf[where], y, y)
    x = kv[:T, 512:].double()
    within(rf[where], ref_rotate(x, p, table, inter), x)
    other = torch.ones(cf.shape[0], dtype=torch.bool, device="cuda")
    other[where] = False
    assert bool((cf[other] == 5.0).all()) and bool((rf[other] == 5.0).all())
    if H:
        x = qr[:T].double()
        within(qo[:T], ref_rotate(x, p, table, inter), x)
        assert bool((qo[T:] == 9.0).all())
    assert torch.equal(L.cpu(), torch.tensor(past, dtype=torch.int32))


@pytest.mark.gpu
def test_write_device_errors(kd):
    """A full request, a bad page, a bad position and bad cumulative lengths: each sets its bit
    and leaves its rows; the others are written."""
    B, n, cap, page = 3, 4, 32, 16
    table, kv, w = table_of(100, 64), normal(B * n, 576, seed=1), normal(512, seed=2)
    L = torch.tensor([2, 29, 0], dtype=torch.int32, device="cuda")           # 29 + 4 > 32
    c, r, _, _ = cache(kd, B, cap, 0, False, 0)
    err = kd.new_error_word()
    pos = torch.arange(B * n, dtype=torch.int32, device="cuda")
    pos[1] = 100
    kd.kd_kv_norm_rope_write(c, r, L, kv, pos, table, kv_weight=w, eps=EPS, dev_error=err)
    assert set(kd.decode_device_error(kd.kd_read_device_error(err))) == {"CACHE_FULL", "BAD_POSITION"}
    assert bool((c[1] == 5.0).all()) and bool((c[0, 3] == 5.0).all()) and bool((c[2, n:] == 5.0).all())
    y = ref_norm(kv[:, :512], w)
    within(c[2, :n], y[8:], y[8:])
    within(c[0, [2, 4, 5]], y[[0, 2, 3]], y[[0, 2, 3]])

    c, r, pt, rows = cache(kd, B, cap, page, False, 1)
    pt[0, 0] = 10 ** 6
    pt[1, 1] = -1
    L = torch.tensor([14, 14, 0], dtype=torch.int32, device="cuda")          # slots 14..17 cross a page
    kd.kd_kv_norm_rope_write_paged(c, r, pt, page, L, kv, None, table, kv_weight=w, eps=EPS, dev_error=err)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_PAGE"]
    want = [(0, 16, 2), (0, 17, 3), (1, 14, 4), (1, 15, 5)] + [(2, i, 8 + i) for i in range(n)]
    at = torch.tensor([int(rows[b, s]) for b, s, _ in want], device="cuda")
    t = torch.tensor([x for _, _, x in want], device="cuda")
    within(c[at], y[t], y[t])
    other = torch.ones(c.shape[0], dtype=torch.bool, device="cuda")
    other[at] = False
    assert bool((c[other] == 5.0).all())

    c, r, _, _ = cache(kd, 2, cap, 0, False, 0)
    L = torch.zeros(2, dtype=torch.int32, device="cuda")
    for cu in ([1, 4, 8], [0, 4, 99], [-3, 4, 8], [0, 9, 8]):
        kd.kd_kv_norm_rope_write(c, r, L, kv[:8].contiguous(), None, table, kv_weight=w, eps=EPS, dev_error=err,
                                 cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
        assert "BAD_SEQLENS" in kd.decode_device_error(kd.kd_read_device_error(err)), cu


@pytest.mark.gpu
def test_write_refuses_no_requests_and_uneven_tokens(kd):
    table, lens = table_of(10, 64), torch.zeros(2, dtype=torch.int32, device="cuda")
    for B, T in ((0, 0), (0, 3), (2, 3)):
        with pytest.raises(ValueError):
            kd.kd_kv_norm_rope_write(normal(B, 8, 512), normal(B, 8, 64), lens[:B], normal(T, 576), None, table)


@pytest.mark.gpu
def test_write_agrees_with_the_node_write(kd):
    """Without a norm and at position 0 the call is kd_kv_write_nodes, bit for bit."""
    B, n, cap = 3, 17, 40
    kv = normal(B * n, 576, seed=3)
    L = torch.tensor([0, 5, 23], dtype=torch.int32, device="cuda")
    c, r, _, _ = cache(kd, B, cap, 0, False, 0)
    c2, r2 = c.clone(), r.clone()
    pos = torch.zeros(B * n, dtype=torch.int32, device="cuda")
    kd.kd_kv_norm_rope_write(c, r, L, kv, pos, table_of(4, 64))
    kd.kd_kv_write_nodes(c2, r2, L, kv[:, :512].reshape(B, n, 512).contiguous(), kv[:, 512:].reshape(B, n, 64).contiguous())
    assert torch.equal(c.view(torch.int16), c2.view(torch.int16)) and torch.equal(r.view(torch.int16), r2.view(torch.int16))


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
@pytest.mark.parametrize("cu", [[0, 8, 4], [0, 5, 3, 8], [0, 4, 8, 6, 8], [0, 5, 12], [0, 8, 9], [0, -1, 8], [1, 4, 8],
                                [0] * 200 + [8, 7] + [8] * 150, [0] * 300 + [8] * 50 + [9]])
def test_write_with_bad_cumulative_lengths_leaves_everything(kd, cu, page):
    """One bad entry anywhere, also of a request without tokens: its bit is set and neither the
    cache nor the queries are touched."""
    B, T, H = len(cu) - 1, 8, 3
    c, r, pt, _ = cache(kd, B, 32, page, False, 0)
    kv, q = normal(T, 576, seed=1), normal(T, H, 64, seed=2)
    qo, err = torch.full((T, H, 64), 9.0, dtype=torch.bfloat16, device="cuda"), kd.new_error_word()
    L = torch.zeros(B, dtype=torch.int32, device="cuda")
    more = dict(cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"), q_rope_in=q, q_rope_out=qo, dev_error=err)
    if page:
        kd.kd_kv_norm_rope_write_paged(c, r, pt, page, L, kv, None, table_of(64, 64), **more)
    else:
        kd.kd_kv_norm_rope_write(c, r, L, kv, None, table_of(64, 64), **more)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_SEQLENS"]
    assert bool((c == 5.0).all()) and bool((r == 5.0).all()) and bool((qo == 9.0).all())


@pytest.mark.gpu
def test_write_of_many_ragged_requests(kd):
    """More requests than a block has threads, many of them without tokens, rows behind the last one."""
    lens = [(b * b) % 4 if b % 3 else 0 for b in range(700)]
    B, T, cap = len(lens), sum(lens), 8
    c, r, _, _ = cache(kd, B, cap, 0, False, 0)
    kv, w, table, err = normal(T + 5, 576, seed=1), normal(512, seed=2), table_of(16, 64), kd.new_error_word()
    past = [b % 5 for b in range(B)]
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    kd.kd_kv_norm_rope_write(c, r, torch.tensor(past, dtype=torch.int32, device="cuda"), kv, None, table, cu_seqlens=cu,
                             kv_weight=w, eps=EPS, dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    at = [past[b] + i for b, n in enumerate(lens) for i in range(n)]
    where = torch.tensor([b * cap + past[b] + i for b, n in enumerate(lens) for i in range(n)], device="cuda")
    y, x = ref_norm(kv[:T, :512], w), kv[:T, 512:].double()
    within(c.view(-1, 512)[where], y, y)
    within(r.view(-1, 64)[where], ref_rotate(x, torch.tensor(at, device="cuda"), table, True), x)
    other = torch.ones(B * cap, dtype=torch.bool, device="cuda")
    other[where] = False
    assert bool((c.view(-1, 512)[other] == 5.0).all()) and bool((r.view(-1, 64)[other] == 5.0).all())


@pytest.mark.gpu
def test_write_reports_a_bad_length_beside_bad_positions(kd):
    """A length below 0 or past the capacity is reported whatever the tokens' positions are; nothing
    of that request is cached, and the queries are written where the position is valid."""
    B, n, H, cap, table, w = 2, 4, 2, 32, table_of(40, 64), normal(512, seed=3)
    kv, q = normal(B * n, 576, seed=1), normal(B * n, H, 64, seed=2)
    x = q.double()
    for first, pos, bits, live in (
            (-5, None, {"CACHE_FULL", "BAD_POSITION"}, []), (-2, None, {"CACHE_FULL", "BAD_POSITION"}, [2, 3]),
            (-5, [3, 4, 5, 6], {"CACHE_FULL"}, [0, 1, 2, 3]), (30, [-1, -1, 40, 99], {"CACHE_FULL", "BAD_POSITION"}, []),
            (30, [0, 1, 40, 2], {"CACHE_FULL", "BAD_POSITION"}, [0, 1, 3])):
        c, r, _, _ = cache(kd, B, cap, 0, False, 0)
        qo, err = torch.full((B * n, H, 64), 9.0, dtype=torch.bfloat16, device="cuda"), kd.new_error_word()
        p = None if pos is None else torch.tensor(pos + [7, 8, 9, 10], dtype=torch.int32, device="cuda")
        kd.kd_kv_norm_rope_write(c, r, torch.tensor([first, 7], dtype=torch.int32, device="cuda"), kv, p, table,
                                 kv_weight=w, eps=EPS, q_rope_in=q, q_rope_out=qo, dev_error=err)
        assert set(kd.decode_device_error(kd.kd_read_device_error(err))) == bits
        assert bool((c[0] == 5.0).all()) and bool((r[0] == 5.0).all())
        y = ref_norm(kv[n:, :512], w)
        within(c[1, 7:7 + n], y, y)
        at = torch.tensor(pos or [first + i for i in range(n)], device="cuda")
        within(qo[live], ref_rotate(x[live], at[live], table, True), x[live])
        dead = [i for i in range(n) if i not in live]
        assert bool((qo[dead] == 9.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("B,H,page", [(4099, 20, 0), (9000, 3, 16), (6000, 0, 0)])
def test_write_of_thousands_of_requests(kd, B, H, page):
    """So many that a block takes several tokens: every row and query as with one, errors of single
    requests among them; a decrease at the far end ends the call."""
    lens = [1 + (b % 7 == 3) - (b % 11 == 5) for b in range(B)]
    T, cap, n_bad = sum(lens), 8, [17, B - 2]
    past = [b % 5 for b in range(B)]
    for b in n_bad:
        past[b] = -(-cap // page) * page if page else cap    # no room
    c, r, pt, rows = cache(kd, B, cap, page, False, 0)
    kv, w, table, err = normal(T + 3, 576, seed=1), normal(512, seed=2), table_of(32, 64), kd.new_error_word()
    q = normal(T + 3, H, 64, seed=3) if H else None
    qo = torch.full((T + 3, H, 64), 9.0, dtype=torch.bfloat16, device="cuda") if H else None
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")
    L = torch.tensor(past, dtype=torch.int32, device="cuda")

    def write(cu):
        more = dict(cu_seqlens=cu, kv_weight=w, eps=EPS, q_rope_in=q, q_rope_out=qo, dev_error=err)
        if page:
            kd.kd_kv_norm_rope_write_paged(c, r, pt, page, L, kv, None, table, **more)
        else:
            kd.kd_kv_norm_rope_write(c, r, L, kv, None, table, **more)
        return kd.decode_device_error(kd.kd_read_device_error(err))

    wrong = cu.clone()
    wrong[B - 1] = T + 1
    assert write(wrong) == ["BAD_SEQLENS"]
    cf, rf = c.reshape(-1, 512), r.reshape(-1, 64)
    assert bool((cf == 5.0).all()) and bool((rf == 5.0).all()) and (not H or bool((qo == 9.0).all()))
    assert write(cu) == ["CACHE_FULL"]
    tok = [(b, i) for b, n in enumerate(lens) for i in range(n)]
    ok = [t for t, (b, _) in enumerate(tok) if b not in n_bad]
    where = torch.tensor([int(rows[tok[t][0], past[tok[t][0]] + tok[t][1]]) for t in ok], device="cuda")
    at = torch.tensor([past[b] + i for b, i in tok], device="cuda")
    y, x = ref_norm(kv[ok, :512], w), kv[ok, 512:].double()
    within(cf[where], y, y)
    within(rf[where], ref_rotate(x, at[ok], table, True), x)
    other = torch.ones(cf.shape[0], dtype=torch.bool, device="cuda")
    other[where] = False
    assert bool((cf[other] == 5.0).all()) and bool((rf[other] == 5.0).all())
    if H:
        within(qo[:T], ref_rotate(q[:T].double(), at, table, True), q[:T].double())
        assert bool((qo[T:] == 9.0).all())


def any_stride(x, axes):
    """x with a stride of 3 along its axes of length 1: never used, as after a transpose of one column."""
    assert all(x.shape[a] == 1 for a in axes)
    return x.as_strided(x.shape, [3 if a in axes else s for a, s in enumerate(x.stride())])


@pytest.mark.gpu
def test_strides_of_single_tokens_and_heads_do_not_matter(kd):
    """One token, one head: torch gives an axis of length 1 any stride (a column transposed has 1)."""
    table, table128, w = table_of(20, 64), table_of(20, 128), normal(512, seed=1)
    one, lens = torch.tensor([5], dtype=torch.int32, device="cuda"), torch.tensor([3], dtype=torch.int32, device="cuda")
    q, k, kv, qr = normal(1, 4, 128, seed=2), normal(1, 1, 128, seed=3), normal(576, 1, seed=4).t(), normal(1, 4, 64, seed=5)
    assert kv.is_contiguous() and kv.stride(0) == 1
    qo, ko = any_stride(torch.zeros_like(q), [0]), any_stride(torch.zeros_like(k), [0, 1])
    kd.kd_qk_norm_rope(any_stride(q, [0]), any_stride(k, [0, 1]), one, table128, q_out=qo, k_out=ko)
    want = kd.kd_qk_norm_rope(q, k, one, table128)
    assert torch.equal(qo, want[0]) and torch.equal(ko, want[1])

    got = []
    for a, b in ((kv, any_stride(qr, [0])), (kv.clone(memory_format=torch.contiguous_format).view(-1).view(1, 576), qr)):
        c, r = torch.zeros(1, 9, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(1, 9, 64, dtype=torch.bfloat16, device="cuda")
        cp, rp, pt = torch.zeros_like(c[0, :8]), torch.zeros_like(r[0, :8]), torch.tensor([[1, 0]], dtype=torch.int32, device="cuda")
        x = kd.kd_kv_norm_rope_write(c, r, lens, a, None, table, kv_weight=w, q_rope_in=b)
        y = kd.kd_kv_norm_rope_write_paged(cp, rp, pt, 4, lens, a, None, table, kv_weight=w, q_rope_in=b)
        got.append((c, r, cp, rp, x, y))
    for a, b in zip(*got):
        assert torch.equal(a, b) and bool((a != 0).any())


@pytest.mark.gpu
def test_prompt_strides_of_single_tokens_and_heads_do_not_matter(kd):
    cu = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
    q, k, v = normal(1, 1, 128, seed=1), normal(1, 1, 128, seed=2), normal(1, 1, 128, seed=3)
    qr, kr = normal(1, 1, 64, seed=4), normal(1, 64, seed=5)
    want = kd.kd_prompt_attn(q, k, v, cu, q_rope=qr, k_rope=kr)
    odd = [any_stride(x, [0, 1]) for x in (q, k, v, qr)]
    for rope in (any_stride(kr, [0]), any_stride(kr.view(1, 1, 64), [0, 1])):
        got = kd.kd_prompt_attn(odd[0], odd[1], odd[2], cu, q_rope=odd[3], k_rope=rope)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
