"""The calls next to the verify step where element offsets pass 32 bits, and calls that overlap
on two streams.  Tolerances are those derived in the calls' own test files."""
import math

import numpy as np
import pytest
import torch

from tests.test_evict import i32, normal, ref_keep, ref_weights, tree
from tests.test_norm_rope import EPS, ref_heads, ref_norm, ref_rotate, table_of, within
from tests.test_prompt_attn import check, cu_of, inputs

pytestmark = pytest.mark.gpu
FAR = 4300000                                           # rows of 512 elements: 2^31 elements are 4194304


def far_cache(B, cap):
    return torch.empty(B, cap, 512, dtype=torch.bfloat16, device="cuda"), \
        torch.empty(B, cap, 64, dtype=torch.bfloat16, device="cuda")


def test_write_weigh_and_evict_in_the_last_request_of_a_large_cache(kd):
    B, cap, n, H, L = 2, FAR // 2 + 10, 9, 16, 700
    c, r = far_cache(B, cap)                            # 4.9 GB; only the rows used are set
    c[1, :L], r[1, :L] = normal(L, 512, seed=1), normal(L, 64, seed=2)
    c[0, :n], r[0, :n] = 0, 0
    lens, table, w = i32([0, L]), table_of(L + n, 64), normal(512, seed=3)
    kv, q = normal(B * n, 576, seed=4), normal(B * n, H, 64, seed=5)
    err = kd.new_error_word()
    qo = kd.kd_kv_norm_rope_write(c, r, lens, kv, None, table, kv_weight=w, eps=EPS, q_rope_in=q, dev_error=err)
    y = ref_norm(kv[n:, :512], w)
    within(c[1, L:L + n], y, y)
    pos = torch.arange(L, L + n, device="cuda")
    within(r[1, L:L + n], ref_rotate(kv[n:, 512:].double(), pos, table, True), kv[n:, 512:].double())

    qa, qr = normal(B, n, H, 512, seed=6), qo.view(B, n, H, 64)
    t = tree(n, 2)
    vis = torch.from_numpy(np.stack([t[1]] * B).view(np.int32)).cuda()
    lse = torch.full((B, n, H), 8.0, device="cuda")
    weights = torch.zeros(B, cap, device="cuda")
    path = i32([t[2] + [-1] * (n - len(t[2]))] * B)
    kd.kd_kv_attn_weights(qa, qr, c, r, lens, vis, lse, path=path, length=i32([len(t[2])] * B), weights_out=weights,
                          dev_error=err)
    ref, tol = ref_weights(qa[1], qr[1], c[1, :L + n], r[1, :L + n], L, t[1], lse[1], t[2], None)
    m = L + len(t[2])
    assert bool(((weights[1, :m].double() - ref).abs() <= tol).all())

    was, ww = c[1, :L].clone(), weights[1, :L].cpu()
    kept, _, _ = kd.kd_kv_evict(c, r, lens, weights, 300, 4, 50, dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    ids = ref_keep(ww.tolist(), L, 300, 4, 50)
    assert kept[1].tolist() == ids
    assert torch.equal(c[1, :300].view(torch.int16), was[ids].view(torch.int16))


def test_far_pages(kd):
    """Pages at the end of a pool of more than 2^31 elements."""
    P, pages, n, H, L = 64, FAR // 64 + 1, 3, 16, 130
    c = torch.empty(pages * P, 512, dtype=torch.bfloat16, device="cuda")
    r = torch.empty(pages * P, 64, dtype=torch.bfloat16, device="cuda")
    pt = i32([[pages - 2, pages - 1, pages - 3, 0]])
    rows = (pt[0].long()[:, None] * P + torch.arange(P, device="cuda")).flatten()
    c[rows], r[rows] = normal(4 * P, 512, seed=1), normal(4 * P, 64, seed=2)
    kv, w, table, err, lens = normal(n, 576, seed=3), normal(512, seed=4), table_of(300, 64), kd.new_error_word(), i32([L])
    kd.kd_kv_norm_rope_write_paged(c, r, pt, P, lens, kv, None, table, kv_weight=w, eps=EPS, dev_error=err)
    y = ref_norm(kv[:, :512], w)
    within(c[rows[L:L + n]], y, y)
    qa, qr = normal(1, n, H, 512, seed=5), normal(1, n, H, 64, seed=6)
    t = tree(n, 1)
    vis, lse = torch.from_numpy(t[1][None].view(np.int32)).cuda(), torch.full((1, n, H), 7.0, device="cuda")
    weights = kd.kd_kv_attn_weights_paged(qa, qr, c, r, pt, P, lens, vis, lse, dev_error=err)
    ref, tol = ref_weights(qa[0], qr[0], c[rows[:L + n]], r[rows[:L + n]], L, t[1], lse[0], list(range(n)), None)
    assert bool(((weights[0, :L + n].double() - ref).abs() <= tol).all())
    was, ww = c[rows[:L]].clone(), weights[0, :L].cpu()
    kept, _, _ = kd.kd_kv_evict_paged(c, r, pt, P, lens, weights, 70, 1, 20, dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    ids = ref_keep(ww.tolist(), L, 70, 1, 20)
    assert kept[0].tolist() == ids and torch.equal(c[rows[:70]].view(torch.int16), was[ids].view(torch.int16))


def test_heads_and_prompt_behind_wide_tokens(kd):
    """Token strides of 600 K elements: the last tokens start beyond 2^31."""
    T, wide, H = 3700, 600064, 2
    buf = torch.empty(T, wide, dtype=torch.bfloat16, device="cuda")                   # 4.4 GB
    parts = buf[:, : 4 * H * 128].unflatten(1, (4 * H, 128))
    parts.copy_(normal(T, 4 * H, 128, seed=1))
    q, k, v = parts[:, :H], parts[:, H:2 * H], parts[:, 2 * H:3 * H]
    table, pos, w = table_of(T, 128), torch.arange(T, device="cuda", dtype=torch.int32), normal(128, seed=2)
    qo = parts[:, 3 * H:]
    kd.kd_qk_norm_rope(q, None, pos, table, q_weight=w, eps=EPS, q_out=qo)
    y, ref = ref_heads(q[-50:], w, pos[-50:], table, 0, False)
    within(qo[-50:], ref, y)
    out, lse = kd.kd_prompt_attn(q, k, v, cu_of([T]))
    check(out, lse, q, k, v, [T], [T], 1.0 / math.sqrt(128.0), heads=(1,))


def test_overlapping_calls_on_two_streams(kd):
    """The same calls side by side on two streams give what they give one after the other."""
    lens = [700, 33, 1500]
    sets = []
    for seed in (1, 20):
        q, k, v, kr, _ = inputs(lens, lens, 4, 4, True, seed=seed)
        B, n, H, cap = 3, 17, 16, 2000
        t = [tree(n, seed + b) for b in range(B)]
        sets.append(dict(
            q=q, k=k, v=v, kr=kr, cu=cu_of(lens), qa=normal(B, n, H, 512, seed=seed), qr=normal(B, n, H, 64, seed=seed + 1),
            c=normal(B, cap, 512, seed=seed + 2), r=normal(B, cap, 64, seed=seed + 3), lens=i32([1900, 900, 40]),
            vis=torch.from_numpy(np.stack([x[1] for x in t]).view(np.int32)).cuda(),
            lse=torch.full((B, n, H), 9.0, device="cuda"), w0=torch.rand(B, cap, device="cuda")))

    def run(s, stream):
        out, lse = torch.empty(sum(lens), 4, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(sum(lens), 4, device="cuda")
        w, d = torch.empty(3, 2000, device="cuda"), (torch.empty(3, 400, 512, dtype=torch.bfloat16, device="cuda"),
                                                     torch.empty(3, 400, 64, dtype=torch.bfloat16, device="cuda"))
        kept, wo, lo = torch.empty(3, 300, dtype=torch.int32, device="cuda"), torch.zeros(3, 400, device="cuda"), i32([0] * 3)
        torch.cuda.synchronize()
        for _ in range(20):
            kd.kd_prompt_attn(s["q"][..., :128], s["k"], s["v"], s["cu"], q_rope=s["q"][..., 128:], k_rope=s["kr"], out=out,
                              lse=lse, stream=stream)
            kd.kd_kv_attn_weights(s["qa"], s["qr"], s["c"], s["r"], s["lens"], s["vis"], s["lse"], weights_in=s["w0"],
                                  weights_out=w, stream=stream)
            kd.kd_kv_evict(s["c"], s["r"], s["lens"], w, 300, 4, 32, c_dst=d[0], r_dst=d[1], weights_out=wo, lens_out=lo,
                           kept=kept, stream=stream)
        return out, lse, w, kept, wo, lo

    want = []
    for s in sets:
        want.append([x.clone() for x in run(s, torch.cuda.current_stream())])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in sets]
    got = [run(s, st) for s, st in zip(sets, streams)]
    torch.cuda.synchronize()
    for a, b in zip(want, got):
        for i, (x, y) in enumerate(zip(a, b)):
            if i == 2:                                  # behind a request's last slot nothing is written
                for j, L in enumerate((1900, 900, 40)):
                    assert torch.equal(x[j, :L + 17], y[j, :L + 17])
            else:
                assert torch.equal(x, y), i


def test_calls_in_flight_at_once_on_two_streams(kd):
    """Every call enqueued on two streams in turn, with nothing waited for until both are full: the
    same bits as one after the other, and the streams did run at the same time."""
    lens, B, n, H, cap, keep = [700, 33, 1500], 3, 17, 16, 2000, 300
    T, Ls = sum(lens), (1900, 900, 40)

    def made(seed):
        q, k, v, kr, _ = inputs(lens, lens, 4, 4, True, seed=seed)
        t = [tree(n, seed + b) for b in range(B)]
        s = dict(q=q, k=k, v=v, kr=kr, cu=cu_of(lens), qa=normal(B, n, H, 512, seed=seed), qr=normal(B, n, H, 64, seed=seed + 1),
                 c=normal(B, cap, 512, seed=seed + 2), r=normal(B, cap, 64, seed=seed + 3), lens=i32(Ls),
                 vis=torch.from_numpy(np.stack([x[1] for x in t]).view(np.int32)).cuda(),
                 lse=torch.full((B, n, H), 9.0, device="cuda"), w0=torch.rand(B, cap, device="cuda"),
                 kv=normal(T, 576, seed=seed + 4), w=normal(512, seed=seed + 5), zero=i32([0] * B),
                 table=table_of(cap, 64), table2=table_of(cap, 128), pos=torch.arange(T, device="cuda", dtype=torch.int32) % cap)
        return s

    def outputs():
        def bf(*a):
            return torch.zeros(*a, dtype=torch.bfloat16, device="cuda")
        return dict(out=bf(T, 4, 128), lse=torch.zeros(T, 4, device="cuda"), w=torch.zeros(B, cap, device="cuda"),
                    c=bf(B, 400, 512), r=bf(B, 400, 64), wo=torch.zeros(B, 400, device="cuda"), lo=i32([0] * B),
                    kept=i32([[0] * keep] * B), c2=bf(B, 1600, 512), r2=bf(B, 1600, 64), q2=bf(T, 4, 64), heads=bf(T, 4, 128),
                    keys=bf(T, 4, 128), err=kd.new_error_word())

    def step(s, o, st):
        kd.kd_qk_norm_rope(s["q"][..., :128], s["k"], s["pos"], s["table2"], q_out=o["heads"], k_out=o["keys"], dev_error=o["err"],
                           stream=st)
        kd.kd_kv_norm_rope_write(o["c2"], o["r2"], s["zero"], s["kv"], None, s["table"], cu_seqlens=s["cu"], kv_weight=s["w"],
                                 q_rope_in=s["q"][..., 128:], q_rope_out=o["q2"], dev_error=o["err"], stream=st)
        kd.kd_prompt_attn(o["heads"], o["keys"], s["v"], s["cu"], q_rope=o["q2"], k_rope=s["kr"], out=o["out"], lse=o["lse"],
                          dev_error=o["err"], stream=st)
        kd.kd_kv_attn_weights(s["qa"], s["qr"], s["c"], s["r"], s["lens"], s["vis"], s["lse"], weights_in=s["w0"],
                              weights_out=o["w"], dev_error=o["err"], stream=st)
        kd.kd_kv_evict(s["c"], s["r"], s["lens"], o["w"], keep, 4, 32, c_dst=o["c"], r_dst=o["r"], weights_out=o["wo"],
                       lens_out=o["lo"], kept=o["kept"], dev_error=o["err"], stream=st)

    sets = [made(1), made(20)]
    want = [outputs() for _ in sets]
    for s, o in zip(sets, want):                        # one after the other
        for _ in range(2):
            step(s, o, torch.cuda.current_stream())
        torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in sets], [outputs() for _ in sets]
    begin, end = ([torch.cuda.Event(enable_timing=True) for _ in sets] for _ in range(2))
    torch.cuda.synchronize()
    for st, e in zip(streams, begin):
        with torch.cuda.stream(st):
            torch.cuda._sleep(40_000_000)               # about 20 ms: both queues fill meanwhile
        e.record(st)
    for _ in range(30):
        for s, o, st in zip(sets, got, streams):
            step(s, o, st)
    for st, e in zip(streams, end):
        e.record(st)
    torch.cuda.synchronize()
    assert begin[0].elapsed_time(end[1]) > 0 and begin[1].elapsed_time(end[0]) > 0       # neither ended before the other began
    for a, b in zip(want, got):
        assert kd.kd_read_device_error(a["err"]) == 0 and kd.kd_read_device_error(b["err"]) == 0
        for name in a:
            assert torch.equal(a[name], b[name]), name
