"""Accumulated attention weights, eviction by them, and a run of the operators together.

Tolerance of the weights: a score's bf16 products are exact in fp32; they are added in at most
36 steps (16 products each) whose sums round to 2^-23 of at most A = scale sum |q k|, so a
score is off by at most 2 x 36 x 2^-23 A; the exponential's argument and value add
2^-20 (1 + |s - lse|); adding R rows rounds to at most R 2^-24 of the sum:
  |col - ref| <= col (72 x 2^-23 max A + 2^-20 (1 + max |s - lse|) + R 2^-24)
and the sum with what was there rounds once more (2^-24 of the value).  Eviction moves bits:
exact."""
import ctypes
import math

import numpy as np
import pytest
import torch

SCALE = 1.0 / math.sqrt(192.0)


def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------ the definitions
def ref_keep(w, L, keep, sink, recent):
    """Kept slots of one request: python's sort, equal weights by slot, NaN last."""
    if L <= keep:
        return list(range(L))
    mid = list(range(sink, L - recent))
    val = {j: (-math.inf if math.isnan(w[j]) else float(w[j]) + 0.0) for j in mid}
    nan = {j: math.isnan(w[j]) for j in mid}
    best = sorted(mid, key=lambda j: (nan[j], -val[j], j))[: keep - sink - recent]
    return sorted(list(range(sink)) + best + list(range(L - recent, L)))


def tree(n, seed):
    """Random parents, vis words and a root path with its length."""
    r = np.random.RandomState(seed)
    par = [-1] + [int(r.randint(i)) for i in range(1, n)]
    vis = np.zeros((n, (n + 31) // 32), np.uint32)
    for i in range(n):
        if i:
            vis[i] = vis[par[i]]
        vis[i, i // 32] |= np.uint32(1 << (i % 32))
    path, at = [], int(r.randint(n))
    while at >= 0:
        path.append(at)
        at = par[at]
    path = path[::-1]
    return par, vis, path


def ref_weights(qa, qr, c, r, L, vis, lse, path, w_in):
    """One request, float64: c, r [L + n][..] in slot order.  (values, tolerance factor)."""
    n = qa.shape[0]
    q = torch.cat([qa, qr], -1).double()
    k = torch.cat([c, r], -1).double()
    col, a_max, d_max, rows = torch.zeros(L + n, dtype=torch.float64, device=k.device), 0.0, 0.0, 0
    for i in path:
        s = SCALE * (q[i] @ k.T) - lse[i].double()[:, None]
        a_max = max(a_max, float(SCALE * (q[i].abs() @ k.abs().T).amax()))
        see = torch.ones(L + n, dtype=torch.bool, device=k.device)
        see[L:] = torch.tensor([bool(int(vis[i, j // 32]) >> (j % 32) & 1) for j in range(n)])
        use = (~lse[i].isneginf())[:, None] & see
        d_max = max(d_max, float(s[use].abs().amax()) if bool(use.any()) else 0.0)
        col += torch.where(use, s, -math.inf).exp().sum(0)
        rows += q.shape[1]
    got = torch.cat([col[:L], col[L + torch.tensor(path, device=k.device)]])
    tol = got * (72 * 2.0 ** -23 * a_max + 2.0 ** -20 * (1 + d_max) + rows * 2.0 ** -24)
    if w_in is not None:
        got[:L] += w_in[:L].double()
    return got, tol + 2.0 ** -24 * got.abs()


# ------------------------------------------------------------------ refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_kd_b200 import build
    build.build()
    from tree_speculative_decoding_kd_b200 import kd
    return kd.lib


def test_host_validation(lib):
    V = ctypes.c_void_p
    aw = [V(16), V(16), V(16), V(16), 512, 64, 100, V(16), V(16), V(16), V(16), V(16), 2, 17, 64, 0.1, V(16), 100, V(32),
          100, None, None]
    for i, v in ((0, None), (0, V(8)), (1, None), (2, V(4)), (4, 500), (5, 60), (6, 0), (7, None), (8, None), (9, None),
                 (10, None), (11, None), (12, 0), (12, 65536), (13, 0), (13, 129), (14, 0), (14, 129), (15, 0.0),
                 (15, float("inf")), (17, 99), (18, None), (19, 99)):
        bad = list(aw)
        bad[i] = v
        assert lib.kd_kv_attn_weights(*bad) == -1, i
    same = list(aw)
    same[18], same[19] = V(16), 101                     # in place with another stride
    assert lib.kd_kv_attn_weights(*same) == -1
    pg = aw[:6] + [64, V(16), 4, 100] + aw[7:]
    pg[20], pg[22] = 256, 256
    for i, v in ((6, 32), (6, 0), (7, None), (8, 0), (9, 0), (20, 255), (22, 255)):
        bad = list(pg)
        bad[i] = v
        assert lib.kd_kv_attn_weights_paged(*bad) == -1, i
    M = 1 << 30                                         # separate buffers
    ev = [V(16), V(M), 512, 64, 100, V(16), V(16), 100, 10, 2, 3, 2, V(2 * M), V(3 * M), 512, 64, 50, V(32), 50, V(16),
          V(16), None, None]
    for i, v in ((0, None), (1, V(M + 2)), (2, 508), (4, 0), (5, None), (6, None), (7, 99), (8, 0), (8, 4), (9, -1), (10, -1),
                 (10, 9), (11, 0), (11, 65536), (12, None), (13, V(3 * M + 8)), (14, 400), (16, 0), (17, None), (18, 9),
                 (19, None), (20, None), (12, V(16)), (13, V(M)), (12, V(16 + 1024))):
        bad = list(ev)
        bad[i] = v
        assert lib.kd_kv_evict(*bad) == -1, i
    inp = list(ev)
    inp[12], inp[13], inp[16] = inp[0], inp[1], 100     # in place: the same capacity and strides
    for i, v in ((16, 99), (14, 520), (15, 72)):
        bad = list(inp)
        bad[i] = v
        assert lib.kd_kv_evict(*bad) == -1, i
    pe = ev[:4] + [16, V(16), 10, 100] + ev[5:16] + [V(16), 10, 100] + ev[17:]
    pe[10] = 160
    for i, v in ((4, 0), (5, None), (6, 0), (7, 0), (19, None), (20, 0), (21, 0), (10, 159)):
        bad = list(pe)
        bad[i] = v
        assert lib.kd_kv_evict_paged(*bad) == -1, i


def test_evict_refuses_more_slots_than_it_numbers(lib):
    """keep and the capacities up to 2^30: beyond, a 32-bit number of a step's last slot would wrap."""
    V, M = ctypes.c_void_p, 1 << 44
    ok = [V(16), V(M), 512, 64, 1 << 30, V(16), V(16), 1 << 31, 50, 1, 1, 1, V(2 * M), V(3 * M), 512, 64, 1 << 30, V(16),
          1 << 31, V(16), V(16), None, None]
    if not torch.cuda.is_available():                   # refused for want of a device, not for the arguments
        assert lib.kd_kv_evict(*ok) not in (-1, 0)
    for i, v in ((4, (1 << 30) + 1), (8, (1 << 30) + 1), (8, (1 << 31) - 1), (16, (1 << 30) + 1), (16, (1 << 31) - 1)):
        bad = list(ok)
        bad[i] = v
        assert lib.kd_kv_evict(*bad) == -1, i


def test_reference_selection():
    assert ref_keep([5, 1, 3, 3, 9, 3], 6, 4, 1, 1) == [0, 2, 4, 5]
    assert ref_keep([0, math.nan, -math.inf, -0.0, 0.0, 0], 6, 4, 1, 1) == [0, 3, 4, 5]
    assert ref_keep([1, 2], 2, 4, 1, 1) == [0, 1]
    assert ref_keep([1.0] * 9, 9, 5, 2, 2) == [0, 1, 2, 7, 8]


# ------------------------------------------------------------------ weights
def pages_for(B, cap, P, seed):
    g = torch.Generator().manual_seed(seed)
    M = -(-cap // P)
    pt = torch.randperm(B * M + 2, generator=g)[: B * M].view(B, M)
    return pt, (B * M + 2) * P


@pytest.mark.gpu
@pytest.mark.parametrize("Ls,n,H,page,accept,with_in", [
    ([0], 1, 1, 0, False, False), ([0, 1, 5], 3, 2, 0, True, True), ([127, 128, 129], 1, 64, 0, False, True),
    ([255, 256, 257, 3], 17, 5, 0, True, True), ([1000], 17, 16, 64, True, True), ([63, 64, 400], 33, 3, 128, False, True),
    ([700, 20], 128, 2, 256, True, False), ([90], 128, 128, 0, False, True), ([511, 130], 7, 128, 64, True, True),
    ([300] * 9, 2, 64, 0, True, True), ([2000], 65, 64, 0, True, True), ([40] * 200, 4, 7, 0, True, True)])
def test_weights(kd, Ls, n, H, page, accept, with_in):
    B, cap = len(Ls), max(Ls) + n + 2
    trees = [tree(n, 7 * b + n) for b in range(B)]
    vis = torch.from_numpy(np.stack([t[1] for t in trees]).view(np.int32)).cuda()
    qa, qr = normal(B, n, H, 512, seed=1), normal(B, n, H, 64, seed=2)
    if page:
        pt, pool = pages_for(B, cap, page, n)
        cap = pt.shape[1] * page
        c, r = normal(pool, 512, seed=3), normal(pool, 64, seed=4)
        slots = torch.arange(cap)
        rows = (pt[:, slots // page] * page + slots % page).cuda()
    else:
        buf = normal(B, cap, 576, seed=3)               # interleaved rows
        c, r = buf[..., :512], buf[..., 512:]
        rows = torch.arange(B * cap, device="cuda").view(B, cap)
    lens = i32(Ls)
    lse = (lens.float() + 1).log()[:, None, None] + 0.5 * SCALE ** 2 * (
        qa.float().square().sum(-1) + qr.float().square().sum(-1))
    if H > 1:
        lse[0, 0, 1] = -math.inf                        # a row that saw nothing adds nothing
    paths = [t[2] for t in trees] if accept else [list(range(n))] * B
    path = i32([p + [-1] * (n - len(p)) for p in paths]) if accept else None
    alen = i32([len(p) for p in paths]) if accept else None
    w_in = torch.rand(B, cap + 3, device="cuda") * 9 if with_in else None
    if with_in:
        for b in range(B):
            w_in[b, Ls[b]:] = math.nan                  # what lies behind the length is not read
    w_out = torch.full((B, cap + 1), 7.0, device="cuda")
    err = kd.new_error_word()
    more = dict(path=path, length=alen, weights_in=w_in, weights_out=w_out, dev_error=err)
    if page:
        # slots behind the last node hold NaN
        for b in range(B):
            c[rows[b, Ls[b] + n:]] = math.nan
            r[rows[b, Ls[b] + n:]] = math.nan
        call = lambda: kd.kd_kv_attn_weights_paged(qa, qr, c, r, pt.int().cuda(), page, lens, vis, lse, **more)  # noqa: E731
    else:
        for b in range(B):
            buf[b, Ls[b] + n:] = math.nan
        call = lambda: kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, **more)  # noqa: E731
    call()
    assert kd.kd_read_device_error(err) == 0
    for b in range(B):
        L, at = Ls[b], rows[b, : Ls[b] + n]
        cb, rb = (c[at], r[at]) if page else (c[b, : L + n], r[b, : L + n])
        ref, tol = ref_weights(qa[b], qr[b], cb, rb, L, trees[b][1], lse[b], paths[b], w_in[b] if with_in else None)
        m = L + len(paths[b])
        d = (w_out[b, :m].double() - ref).abs()
        assert bool((d <= tol).all()), (b, float((d / tol.clamp_min(1e-300)).max()))
        assert bool((w_out[b, m:] == 7.0).all())
    first = w_out.clone()
    call()
    assert torch.equal(first, w_out)                    # the same bits again


@pytest.mark.gpu
def test_weights_of_true_lse_sum_to_one(kd):
    """With the attention's own lse, a counted row's weights add up to 1: the whole call's
    sum is the number of rows.  (Chain, every node counted: each row sees only counted keys.)"""
    B, n, H, L, cap = 2, 33, 8, 500, 600
    qa, qr = normal(B, n, H, 512, seed=1), normal(B, n, H, 64, seed=2)
    c, r = normal(B, cap, 512, seed=3), normal(B, cap, 64, seed=4)
    vis, _ = kd.kd_tree_build_mask(i32([[i - 1 for i in range(n)]] * B))
    lens = i32([L, L - 77])
    _, lse = kd.kd_tree_verify_attn(qa, qr, c, r, lens, vis)
    w = kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse)
    # each row's sum is off by at most the scores' error against lse's: 1e-3, the attention's own bound
    assert torch.allclose(w.double().sum(1), torch.full((B,), float(n * H), dtype=torch.float64, device="cuda"), rtol=1e-3)
    acc = kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, weights_in=w.clone())
    twice = kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, weights_in=w, weights_out=w)
    assert torch.equal(acc[0, :L], twice[0, :L])        # accumulating in place is the same


@pytest.mark.gpu
@pytest.mark.parametrize("B,hi,n,H", [(64, 3000, 17, 64), (150, 700, 3, 16), (16, 4000, 1, 64), (40, 900, 40, 5)])
def test_weights_launch_after_launch(kd, B, hi, n, H):
    """Many units per CTA with one to many query tiles in turn, a hundred launches behind each
    other: no wait gives up and the bits stay the same."""
    rng = np.random.RandomState(B)
    trees = [tree(n, 3 * b + 1) for b in range(B)]
    vis = torch.from_numpy(np.stack([t[1] for t in trees]).view(np.int32)).cuda()
    paths = [t[2] if b % 3 else [0] for b, t in enumerate(trees)]
    path, alen = i32([p + [-1] * (n - len(p)) for p in paths]), i32([len(p) for p in paths])
    lens = i32(rng.randint(1, hi, B).tolist())
    cap = hi + n
    qa, qr = normal(B, n, H, 512, seed=1, scale=0.5), normal(B, n, H, 64, seed=2, scale=0.5)
    c, r = normal(B, cap, 512, seed=3), normal(B, cap, 64, seed=4)
    lse, err = torch.full((B, n, H), 8.0, device="cuda"), kd.new_error_word()
    w = [torch.zeros(B, cap, device="cuda") for _ in range(2)]
    for i in range(100):
        kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, path=path, length=alen, weights_out=w[i > 0], dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    assert torch.equal(*w)


@pytest.mark.gpu
def test_weights_device_errors(kd):
    B, n, H, cap = 6, 4, 2, 64
    qa, qr = normal(B, n, H, 512, seed=1), normal(B, n, H, 64, seed=2)
    c, r = normal(B, cap, 512, seed=3), normal(B, cap, 64, seed=4)
    lens, lse = i32([10, 61, -1, 10, 10, 10]), torch.full((B, n, H), 5.0, device="cuda")
    t = tree(n, 1)
    vis = torch.from_numpy(np.stack([t[1]] * B).view(np.int32)).cuda()
    path = i32([[0, 1, -1, -1]] * 3 + [[0, 4, -1, -1], [0, -1, -1, -1], [0, 1, -1, -1]])
    alen = i32([2, 2, 2, 2, 5, 0])
    w, err = torch.full((B, cap), 7.0, device="cuda"), kd.new_error_word()
    kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, path=path, length=alen, weights_out=w, dev_error=err)
    assert set(kd.decode_device_error(kd.kd_read_device_error(err))) == {"CACHE_FULL", "BAD_PATH"}
    assert bool((w[1:] == 7.0).all())
    ref, tol = ref_weights(qa[0], qr[0], c[0, :14], r[0, :14], 10, t[1], lse[0], [0, 1], None)
    assert bool(((w[0, :12].double() - ref).abs() <= tol).all())

    pool = normal(6 * 64, 512, seed=5), normal(6 * 64, 64, seed=6)
    pt = i32([[0, 9], [2, -1], [4, 5]])
    w.fill_(7.0)
    wp = torch.full((3, 128), 7.0, device="cuda")
    kd.kd_kv_attn_weights_paged(qa[:3], qr[:3], *pool, pt, 64, i32([62, 20, 70]), vis[:3], lse[:3], weights_out=wp,
                                dev_error=err)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_PAGE"]
    assert bool((wp[0] == 7.0).all())                   # 62 + 4 slots reach its bad page
    for b, L, pages in ((1, 20, [2]), (2, 70, [4, 5])):  # the bad page of request 1 is never reached
        at = torch.cat([torch.arange(p * 64, p * 64 + 64) for p in pages])[: L + n].cuda()
        ref, tol = ref_weights(qa[b], qr[b], pool[0][at], pool[1][at], L, t[1], lse[b], [0, 1, 2, 3], None)
        assert bool(((wp[b, : L + n].double() - ref).abs() <= tol).all())


# ------------------------------------------------------------------ eviction
def check_evict(kept, w_out, lens_out, Ls, w, keep, sink, recent, get, put, before):
    """get(b, slots) / put(b, slots): source and destination rows as int16."""
    for b, L in enumerate(Ls):
        ids = ref_keep(w[b].tolist(), L, keep, sink, recent)
        assert kept[b].tolist() == ids + [-1] * (keep - len(ids)), b
        assert int(lens_out[b]) == len(ids)
        for x, y in zip(get(b, ids), put(b, list(range(len(ids))))):
            assert torch.equal(x, y), b
        want = w[b][ids]
        got = w_out[b][: len(ids)]
        assert torch.equal(want.view(torch.int32), got.cpu().view(torch.int32)), b


WEIGHTS = {
    "random": lambda r, n: r.standard_normal(n).astype(np.float32),
    "ties": lambda r, n: r.randint(0, 3, n).astype(np.float32) if hasattr(r, "randint") else r.integers(0, 3, n).astype(np.float32),
    "equal": lambda r, n: np.full(n, 2.5, np.float32),
    "odd": lambda r, n: r.choice(np.array([0.0, -0.0, np.nan, np.inf, -np.inf, 1e-45, -1e-45, 3e38, 1.0], np.float32), n),
    "close": lambda r, n: (np.float32(1.0) + np.float32(2.0 ** -23) * r.integers(0, 50, n)).astype(np.float32),
    "tiny": lambda r, n: np.exp(-20 * r.random(n)).astype(np.float32),
}


@pytest.mark.gpu
@pytest.mark.parametrize("kind", sorted(WEIGHTS))
@pytest.mark.parametrize("Ls,keep,sink,recent,page,inplace", [
    ([1], 1, 0, 0, 0, False), ([7, 0, 12], 5, 1, 2, 0, True), ([300, 5, 1025, 64], 64, 4, 16, 0, False),
    ([1025, 3000, 100], 1500, 0, 0, 0, True), ([5000, 4097], 4096, 16, 4080, 0, True), ([200, 77], 50, 25, 25, 16, True),
    ([1000, 900, 3], 333, 1, 0, 64, False), ([9000], 8999, 3, 100, 0, True), ([640, 100], 100, 0, 100, 1, True)])
def test_evict(kd, kind, Ls, keep, sink, recent, page, inplace):
    B, cap = len(Ls), max(Ls) + 3
    rng = np.random.default_rng(keep)
    if page:
        pt, pool = pages_for(B, cap, page, 1)
        cap = pt.shape[1] * page
        c, r = normal(pool, 512, seed=3), normal(pool, 64, seed=4)
        slots = torch.arange(cap)
        rows = pt[:, slots // page] * page + slots % page
    else:
        c, r = normal(B, cap, 512, seed=3), normal(B, cap, 64, seed=4)
        rows = torch.arange(B * cap).view(B, cap)
    w = torch.from_numpy(np.stack([WEIGHTS[kind](rng, cap) for _ in range(B)]))
    src = c.reshape(-1, 512).view(torch.int16).cpu().clone(), r.reshape(-1, 64).view(torch.int16).cpu().clone()
    lens, win, err = i32(Ls), w.cuda(), kd.new_error_word()
    if inplace:
        if page:
            kept, wo, lo = kd.kd_kv_evict_paged(c, r, pt.int().cuda(), page, lens, win, keep, sink, recent, dev_error=err)
        else:
            kept, wo, lo = kd.kd_kv_evict(c, r, lens, win, keep, sink, recent, dev_error=err)
        assert wo is win and lo is lens
        dst, drows = (c, r), rows
    else:
        dcap = keep + 5
        if page:
            dpt, dpool = pages_for(B, dcap, page, 2)
            dst = torch.full((dpool, 512), 5.0, dtype=torch.bfloat16, device="cuda"), \
                torch.full((dpool, 64), 5.0, dtype=torch.bfloat16, device="cuda")
            dcap = dpt.shape[1] * page
            slots = torch.arange(dcap)
            drows = dpt[:, slots // page] * page + slots % page
            kept, wo, lo = kd.kd_kv_evict_paged(c, r, pt.int().cuda(), page, lens, win, keep, sink, recent, c_dst=dst[0],
                                                r_dst=dst[1], dst_page_table=dpt.int().cuda(), dev_error=err)
        else:
            buf = torch.full((B, dcap, 576), 5.0, dtype=torch.bfloat16, device="cuda")
            dst, drows = (buf[..., :512], buf[..., 512:]), torch.arange(B * dcap).view(B, dcap)
            kept, wo, lo = kd.kd_kv_evict(c, r, lens, win, keep, sink, recent, c_dst=dst[0], r_dst=dst[1], dev_error=err)
        assert torch.equal(lens, i32(Ls))
    assert kd.kd_read_device_error(err) == 0
    now = dst[0].reshape(-1, 512).view(torch.int16).cpu(), dst[1].reshape(-1, 64).view(torch.int16).cpu()
    check_evict(kept.cpu(), wo, lo.cpu(), Ls, w, keep, sink, recent, lambda b, s: [x[rows[b, s]] for x in src],
                lambda b, s: [x[drows[b, s]] for x in now], None)
    # rows that are no destination stay as they were
    moved = torch.cat([drows[b, : min(L, keep)] for b, L in enumerate(Ls)])
    rest = torch.ones(now[0].shape[0], dtype=torch.bool)
    rest[moved] = False
    five = torch.tensor(5.0, dtype=torch.bfloat16).view(torch.int16)
    for x, y in zip(now, src):
        assert bool((x[rest] == (y[rest] if inplace else five)).all())


@pytest.mark.gpu
def test_evict_many_requests_and_long(kd):
    for Ls, keep, sink, recent in (([40] * 300 + [7] * 20, 16, 2, 4), ([70001], 40000, 8, 512)):
        B, cap = len(Ls), max(Ls)
        c, r = normal(B, cap, 512, seed=1), normal(B, cap, 64, seed=2)
        w = torch.rand(B, cap, device="cuda").square()
        src = c.view(torch.int16).clone(), r.view(torch.int16).clone()
        wc = w.cpu().clone()
        kept, wo, lo = kd.kd_kv_evict(c, r, i32(Ls), w, keep, sink, recent)
        now = c.view(torch.int16), r.view(torch.int16)
        check_evict(kept.cpu(), wo, lo.cpu(), Ls, wc, keep, sink, recent, lambda b, s: [x[b, s] for x in src],
                    lambda b, s: [x[b, s] for x in now], None)


@pytest.mark.gpu
@pytest.mark.parametrize("B,L,keep,page", [(40, 1500, 1100, 0), (40, 1500, 300, 64), (3, 6000, 4500, 0), (2, 4000, 3999, 16)])
def test_evict_in_place_in_many_steps(kd, B, L, keep, page):
    """Rows that move a little and rows that move far, over many steps of a CTA; few and many requests."""
    Ls = [L - 7 * b for b in range(B)]
    cap = L + 2
    if page:
        pt, pool = pages_for(B, cap, page, 1)
        cap = pt.shape[1] * page
        slots = torch.arange(cap)
        rows = pt[:, slots // page] * page + slots % page
    else:
        pool, rows = B * cap, torch.arange(B * cap).view(B, cap)
    c, r = normal(pool, 512, seed=1), normal(pool, 64, seed=2)
    src = [x.view(torch.int16).cpu().clone() for x in (c, r)]
    w = torch.from_numpy(np.random.default_rng(B).random((B, cap)).astype(np.float32))
    w[:, : L // 2] += 0.5 * (torch.arange(B) % 2)[:, None]
    lens, win = i32(Ls), w.cuda()
    if page:
        kept, wo, lo = kd.kd_kv_evict_paged(c, r, pt.int().cuda(), page, lens, win, keep, 4, 50)
    else:
        kept, wo, lo = kd.kd_kv_evict(c.view(B, cap, 512), r.view(B, cap, 64), lens, win, keep, 4, 50)
    now = [x.view(torch.int16).cpu() for x in (c, r)]
    check_evict(kept.cpu(), wo, lo.cpu(), Ls, w, keep, 4, 50, lambda b, s: [x[rows[b, s]] for x in src],
                lambda b, s: [x[rows[b, s]] for x in now], None)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["equal", "random", "ties"])
def test_evict_longer_than_a_cluster_reads_at_once(kd, kind):
    """Caches numbered in several steps (a cluster holds 32768 slots), with equal weights on both
    sides of a step, into another cache; unaligned rows of weights."""
    Ls, keep, sink, recent = [70001, 33000, 32769], 21000, 3, 700
    B, cap = len(Ls), max(Ls)
    c, r = normal(B, cap, 512, seed=1), normal(B, cap, 64, seed=2)
    rng = np.random.default_rng(5)
    w = torch.from_numpy(np.stack([WEIGHTS[kind](rng, cap) for _ in range(B)]))
    win = torch.empty(B, cap + 3, device="cuda")[:, :cap]
    win.copy_(w)
    dst = torch.zeros(B, keep, 512, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(B, keep, 64, dtype=torch.bfloat16, device="cuda")
    lens = i32(Ls)
    kept, wo, lo = kd.kd_kv_evict(c, r, lens, win, keep, sink, recent, c_dst=dst[0], r_dst=dst[1])
    src, now = [x.view(torch.int16) for x in (c, r)], [x.view(torch.int16) for x in dst]
    check_evict(kept.cpu(), wo, lo.cpu(), Ls, w, keep, sink, recent, lambda b, s: [x[b, s] for x in src],
                lambda b, s: [x[b, s] for x in now], None)


@pytest.mark.gpu
def test_results_belong_to_the_stream_of_the_call(kd):
    """A call on another stream than the current one, which is busy: what the call allocates (zeros
    behind the stored weights) is not filled by the current stream after the kernels ran."""
    B, cap, n, H, keep = 2, 300, 3, 16, 100
    c, r = normal(B, cap, 512, seed=1), normal(B, cap, 64, seed=2)
    qa, qr = normal(B, n, H, 512, seed=3), normal(B, n, H, 64, seed=4)
    vis, _ = kd.kd_tree_build_mask(i32([[-1, 0, 1]] * B))
    lens, lse = i32([250, 297]), torch.zeros(B, n, H, device="cuda")
    dst = torch.empty(B, keep, 512, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(B, keep, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.rand(B, cap, device="cuda")

    def both(stream):
        ww = kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, scale=0.01, stream=stream)
        kept, wo, lo = kd.kd_kv_evict(c, r, lens, w, keep, 2, 10, c_dst=dst[0], r_dst=dst[1], stream=stream)
        return ww, kept, wo, lo

    want = both(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    torch.cuda._sleep(200_000_000)                      # the current stream is busy for about 0.1 s
    got = both(side)
    side.synchronize()
    torch.cuda.synchronize()
    for x, y in zip(got, want):
        assert torch.equal(x, y) and bool((x != 0).any())


@pytest.mark.gpu
def test_weights_of_a_repeated_path_entry(kd):
    """A path that names a node twice counts its rows twice and writes its slot's weight at both places."""
    n, H, L, cap = 5, 16, 200, 230
    qa, qr = normal(1, n, H, 512, seed=1), normal(1, n, H, 64, seed=2)
    c, r = normal(1, cap, 512, seed=3), normal(1, cap, 64, seed=4)
    t = tree(n, 3)
    vis, lse = torch.from_numpy(t[1][None].view(np.int32)).cuda(), torch.full((1, n, H), 8.0, device="cuda")
    path = [0, 2, 2, 4]
    w = kd.kd_kv_attn_weights(qa, qr, c, r, i32([L]), vis, lse, path=i32([path + [-1]]), length=i32([4]))
    ref, tol = ref_weights(qa[0], qr[0], c[0, :L + n], r[0, :L + n], L, t[1], lse[0], path, None)
    assert bool(((w[0, :L + 4].double() - ref).abs() <= tol).all())


@pytest.mark.gpu
def test_evict_keep_beyond_the_cache(kd):
    c, r, w = normal(2, 50, 512, seed=1), normal(2, 50, 64, seed=2), torch.rand(2, 50, device="cuda")
    was, lens = c.clone(), i32([50, 20])
    kept, _, _ = kd.kd_kv_evict(c, r, lens, w, 70, 5, 5)
    assert lens.tolist() == [50, 20] and torch.equal(c, was)
    assert kept[0].tolist() == list(range(50)) + [-1] * 20 and kept[1].tolist() == list(range(20)) + [-1] * 50


@pytest.mark.gpu
def test_evict_device_errors(kd):
    Ls, cap, keep = [50, -1, 65, 40, 60], 64, 30
    c, r = normal(5, cap, 512, seed=1), normal(5, cap, 64, seed=2)
    w, lens, err = torch.rand(5, cap, device="cuda"), i32(Ls), kd.new_error_word()
    d = torch.full((5, 20, 512), 5.0, dtype=torch.bfloat16, device="cuda"), \
        torch.full((5, 20, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    wo, lo = torch.full((5, 20), 3.0, device="cuda"), i32([9] * 5)
    # the destination holds 20 slots and 30 are kept: nothing moves
    kept, _, _ = kd.kd_kv_evict(c, r, lens, w, keep, 1, 2, c_dst=d[0], r_dst=d[1], weights_out=wo, lens_out=lo, dev_error=err)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["CACHE_FULL"]
    assert bool((kept == -1).all()) and bool((d[0] == 5.0).all()) and bool((wo == 3.0).all()) and lo.tolist() == [9] * 5
    was, ww = c.clone(), w.clone()
    kept, _, _ = kd.kd_kv_evict(c, r, lens, w, keep, 1, 2, dev_error=err)       # in place: bad lengths stay
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["CACHE_FULL"]
    assert lens.tolist() == [30, -1, 65, 30, 30]
    assert torch.equal(c[1:3], was[1:3]) and torch.equal(w[1:3], ww[1:3]) and bool((kept[1:3] == -1).all())
    ids = ref_keep(ww[0].tolist(), 50, keep, 1, 2)
    assert torch.equal(c[0, :keep].view(torch.int16), was[0, ids].view(torch.int16))

    pool = normal(8 * 16, 512, seed=3), normal(8 * 16, 64, seed=4)
    pt = i32([[0, 1, 99], [2, 3, -1], [4, -7, 5]])
    was, lens, w = pool[0].clone(), i32([40, 30, 32]), torch.rand(3, 48, device="cuda")
    ww = w.clone()
    kept, _, _ = kd.kd_kv_evict_paged(*pool, pt, 16, lens, w, 10, 0, 0, dev_error=err)
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_PAGE"]
    assert lens.tolist() == [40, 10, 32] and bool((kept[0] == -1).all()) and bool((kept[2] == -1).all())
    at = torch.arange(32, 64, device="cuda")
    ids = torch.tensor(ref_keep(ww[1].tolist(), 30, 10, 0, 0), device="cuda")
    assert torch.equal(pool[0][32:42], was[at[ids]])
    rest = [*range(32), *range(42, 128)]
    assert torch.equal(pool[0][rest], was[rest])


@pytest.mark.gpu
def test_evict_within_one_pool(kd):
    """Into fresh pages of the same pool: the source's rows stay."""
    P, pool = 16, (normal(10 * 16, 512, seed=3), normal(10 * 16, 64, seed=4))
    was = pool[0].clone()
    w = torch.rand(2, 48, device="cuda")
    kept, wo, lo = kd.kd_kv_evict_paged(*pool, i32([[0, 1, 2], [9, 8, 7]]), P, i32([48, 33]), w, 20, 2, 2,
                                        dst_page_table=i32([[3, 4], [6, 5]]))
    for b, (L, src, dst) in enumerate(((48, [0, 1, 2], [3, 4]), (33, [9, 8, 7], [6, 5]))):
        ids = ref_keep(w[b].tolist(), L, 20, 2, 2)
        assert kept[b].tolist() == ids
        rows = torch.cat([torch.arange(p * P, p * P + P) for p in src])[ids].cuda()
        to = torch.cat([torch.arange(p * P, p * P + P) for p in dst])[:20].cuda()
        assert torch.equal(pool[0][to], was[rows])
    still = [*range(48), *range(7 * 16, 160)]
    assert torch.equal(pool[0][still], was[still])


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 16])
def test_evict_lengths_of_failed_requests_are_zero(kd, page):
    """Into another cache, lens_out made by the binding: a request that fails holds nothing there."""
    B, cap, keep = 4, 64, 30
    c, r, w = normal(B, cap, 512, seed=1), normal(B, cap, 64, seed=2), torch.rand(B, cap, device="cuda")
    d, e = torch.zeros(B, 32, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, 32, 64, dtype=torch.bfloat16, device="cuda")
    lens = i32([50, -1, 65, 20])
    dirty = [torch.full((B,), 7, dtype=torch.int32, device="cuda") for _ in range(64)]      # what the allocator hands out next
    torch.cuda.synchronize()
    del dirty
    if page:
        pt = i32([[4 * b + i for i in range(4)] for b in range(B)])
        dpt = i32([[2 * b + i for i in range(2)] for b in range(B)])
        kept, _, lo = kd.kd_kv_evict_paged(c.view(-1, 512), r.view(-1, 64), pt, 16, lens, w, keep, 1, 2, c_dst=d.view(-1, 512),
                                           r_dst=e.view(-1, 64), dst_page_table=dpt)
    else:
        kept, _, lo = kd.kd_kv_evict(c, r, lens, w, keep, 1, 2, c_dst=d, r_dst=e)
    assert lo.tolist() == [30, 0, 0, 20] and lens.tolist() == [50, -1, 65, 20]
    assert bool((kept[1:3] == -1).all()) and bool((d[1:3] == 0).all())


# ------------------------------------------------------------------ together
def test_names_in_the_header():
    import os
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "kd_verify.h")).read()
    for name in ("kd_qk_norm_rope", "kd_kv_norm_rope_write", "kd_prompt_attn", "kd_kv_attn_weights", "kd_kv_evict"):
        assert name + "(" in src


@pytest.mark.gpu
@pytest.mark.parametrize("page", [0, 64])
def test_prompt_to_evicted_decode(kd, page):
    """A model's layer from the prompt to a decode step over an evicted cache.  Ragged prompts go
    through the norm-and-rotate write and the prompt attention; the last tokens are verified
    again as a tree step in absorb form, accepted, weighed, compacted and evicted; the next
    single-token step reads what is left.  Where the absorb form and the per-head form meet
    (values = latents through W, keys = W^T applied to the query) they have to agree."""
    torch.manual_seed(0)
    H, lens = 4, [150, 97, 260]
    B, T, cap, keep = 3, sum(lens), 512, 128
    W_uk, W_uv = torch.randn(H, 128, 512, device="cuda") / 22, torch.randn(H, 512, 128, device="cuda") / 22
    kv, w = normal(T, 576, seed=1), (1 + 0.1 * torch.randn(512, device="cuda")).to(torch.bfloat16)
    q = normal(T, H, 192, seed=2)
    inv = 10000.0 ** (-torch.arange(0, 64, 2, dtype=torch.float64, device="cuda") / 64)
    ang = torch.arange(1024, dtype=torch.float64, device="cuda")[:, None] * inv
    table = torch.cat([ang.cos(), ang.sin()], 1).float()
    cu = i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
    err, L = kd.new_error_word(), i32([0] * B)
    if page:
        pt, pool = pages_for(B, cap, page, 3)
        pt = pt.int().cuda()
        c, r = torch.zeros(pool, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(pool, 64, dtype=torch.bfloat16, device="cuda")
        slots = torch.arange(cap, device="cuda")
        rows = pt.long()[:, slots // page] * page + slots % page
        view = lambda: (c[rows], r[rows])  # noqa: E731
        write = lambda *a, **k: kd.kd_kv_norm_rope_write_paged(c, r, pt, page, *a, **k)  # noqa: E731
    else:
        c, r = torch.zeros(B, cap, 512, dtype=torch.bfloat16, device="cuda"), torch.zeros(B, cap, 64, dtype=torch.bfloat16, device="cuda")
        view = lambda: (c, r)  # noqa: E731
        write = lambda *a, **k: kd.kd_kv_norm_rope_write(c, r, *a, **k)  # noqa: E731
    q_rope = write(L, kv, None, table, cu_seqlens=cu, kv_weight=w, q_rope_in=q[..., 128:], dev_error=err)
    cv, rv = view()
    lat = torch.cat([cv[b, :n] for b, n in enumerate(lens)]).float()
    kr = torch.cat([rv[b, :n] for b, n in enumerate(lens)]).contiguous()
    k_nope = torch.einsum("td,hkd->thk", lat, W_uk).to(torch.bfloat16)
    v = torch.einsum("td,hdk->thk", lat, W_uv).to(torch.bfloat16)
    out, lse = kd.kd_prompt_attn(q[..., :128], k_nope, v, cu, q_rope=q_rope, k_rope=kr, dev_error=err)

    # the last n tokens of every prompt once more, as a chain over the committed rest
    n = 17
    L = i32([x - n for x in lens])
    last = torch.cat([torch.arange(int(cu[b + 1]) - n, int(cu[b + 1])) for b in range(B)]).cuda()
    q_abs = torch.einsum("thk,hkd->thd", q[last][..., :128].float(), W_uk).to(torch.bfloat16).view(B, n, H, 512).contiguous()
    qr = q_rope[last].view(B, n, H, 64).contiguous()
    parents = i32([[i - 1 for i in range(n)]] * B)
    vis, _ = kd.kd_tree_build_mask(parents, dev_error=err)
    if page:
        o2, z2 = kd.kd_tree_verify_attn_paged(q_abs, qr, c, r, pt, page, L, vis)
    else:
        o2, z2 = kd.kd_tree_verify_attn(q_abs, qr, c, r, L, vis)
    # two roundings to bf16 of 128- and 512-long sums apart (k_nope, q_abs): scores of size ~ 10 x 2^-8
    assert torch.allclose(z2.view(B * n, H), lse[last], atol=0.05)
    got = torch.einsum("bnhd,hdk->bnhk", o2.float(), W_uv).reshape(B * n, H, 128)
    ref = out[last].float()
    assert float((got - ref).norm() / ref.norm()) < 0.05

    # accept everything but the last four nodes, weigh, compact, evict
    tokens = i32([list(range(n))] * B)
    argmax = i32([[i + 1 if i < n - 5 else 999 for i in range(n)]] * B)
    path, length, _ = kd.kd_tree_accept(tokens, parents, argmax, dev_error=err)
    assert length.tolist() == [n - 4] * B
    cv, rv = (x.clone() for x in view())
    if page:
        weights = kd.kd_kv_attn_weights_paged(q_abs, qr, c, r, pt, page, L, vis, z2, path=path, length=length, dev_error=err)
        kd.kd_kv_compact_paged(c, r, pt, page, path, length, L, err)
        kept, weights, L = kd.kd_kv_evict_paged(c, r, pt, page, L, weights, keep, 4, 32, dev_error=err)
    else:
        weights = kd.kd_kv_attn_weights(q_abs, qr, c, r, L, vis, z2, path=path, length=length, dev_error=err)
        kd.kd_kv_compact(c, r, path, length, L, err)
        kept, weights, L = kd.kd_kv_evict(c, r, L, weights, keep, 4, 32, dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    assert L.tolist() == [min(x - 4, keep) for x in lens]
    for b, x in enumerate(lens):
        ids = kept[b][: int(L[b])].long()
        assert ids.tolist() == sorted(ids.tolist()) and set(range(4)) <= set(ids.tolist())
        now = view()
        assert torch.equal(now[0][b, : int(L[b])], cv[b, ids]) and torch.equal(now[1][b, : int(L[b])], rv[b, ids])

    # one more token for each: its row written behind what is left, at its true position
    tok, qt = normal(B, 576, seed=7), normal(B, H, 192, seed=8)
    pos = i32([x - 4 for x in lens])
    q1 = write(L, tok, pos, table, kv_weight=w, q_rope_in=qt[..., 128:], dev_error=err).view(B, 1, H, 64)
    qa1 = torch.einsum("thk,hkd->thd", qt[..., :128].float(), W_uk).to(torch.bfloat16).view(B, 1, H, 512).contiguous()
    one = torch.ones(B, 1, 1, dtype=torch.int32, device="cuda")
    o3, z3 = kd.kd_tree_verify_attn_paged(qa1, q1, c, r, pt, page, L, one) if page else \
        kd.kd_tree_verify_attn(qa1, q1, c, r, L, one)
    assert kd.kd_read_device_error(err) == 0
    cv, rv = view()
    for b in range(B):
        m = int(L[b]) + 1
        s = SCALE * (qa1[b, 0].double() @ cv[b, :m].double().T + q1[b, 0].double() @ rv[b, :m].double().T)
        assert torch.allclose(torch.logsumexp(s, -1), z3[b, 0].double(), atol=1e-3)
        ref = torch.softmax(s, -1) @ cv[b, :m].double()
        assert float((o3[b, 0].double() - ref).norm() / ref.norm()) < 5e-3


@pytest.mark.gpu
def test_graph_of_a_whole_step(kd):
    """Write, verify, accept, weigh, compact and evict captured once and replayed: the same as run eagerly."""
    B, n, H, cap, keep = 4, 9, 8, 300, 100
    kv, q = normal(B * n, 576, seed=1), normal(B * n, H, 192, seed=2)
    w, table = normal(512, seed=3), torch.rand(400, 64, device="cuda")
    qa = normal(B, n, H, 512, seed=4)
    parents = i32([tree(n, b)[0] for b in range(B)])
    tokens, argmax = i32([list(range(n))] * B), i32([[1, 2, 3, 4, 5, 6, 7, 8, 9]] * B)
    c0, r0 = normal(B, cap, 512, seed=5), normal(B, cap, 64, seed=6)
    c, r, L, wt = c0.clone(), r0.clone(), i32([200, 101, 90, 250]), torch.rand(B, cap, device="cuda")
    L0, w0 = L.clone(), wt.clone()
    out, lse = torch.empty(B, n, H, 512, dtype=torch.bfloat16, device="cuda"), torch.empty(B, n, H, device="cuda")
    vis, depth = torch.empty(B, n, 1, dtype=torch.int32, device="cuda"), torch.empty(B, n, dtype=torch.int32, device="cuda")
    path, ln, bonus = torch.empty(B, n, dtype=torch.int32, device="cuda"), i32([0] * B), i32([0] * B)
    q1, kept, err = torch.empty(B * n, H, 64, dtype=torch.bfloat16, device="cuda"), i32([[0] * keep] * B), kd.new_error_word()
    ws = kd.new_workspace(B, n, H, cap)

    def step():
        kd.kd_kv_norm_rope_write(c, r, L, kv, None, table, kv_weight=w, q_rope_in=q[..., 128:], q_rope_out=q1, dev_error=err)
        kd.kd_tree_build_mask(parents, vis, depth, err)
        kd.kd_tree_verify_attn(qa, q1.view(B, n, H, 64), c, r, L, vis, out=out, lse=lse, workspace=ws)
        kd.kd_tree_accept(tokens, parents, argmax, path, ln, bonus, err)
        kd.kd_kv_attn_weights(qa, q1.view(B, n, H, 64), c, r, L, vis, lse, path=path, length=ln, weights_in=wt,
                              weights_out=wt, dev_error=err)
        kd.kd_kv_compact(c, r, path, ln, L, err)
        kd.kd_kv_evict(c, r, L, wt, keep, 4, 20, kept=kept, dev_error=err)

    def reset():
        c.copy_(c0), r.copy_(r0), L.copy_(L0), wt.copy_(w0)

    step()
    torch.cuda.synchronize()
    want = [x.clone() for x in (c, r, L, wt, kept, out)]
    assert kd.kd_read_device_error(err) == 0 and L.tolist()[0] == keep
    reset()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for _ in range(2):
        reset()
        g.replay()
        torch.cuda.synchronize()
        for x, y in zip(want, (c, r, L, wt, kept, out)):
            assert torch.equal(x, y)
