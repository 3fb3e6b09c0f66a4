"""Causal attention of packed prompts against the formula in 64 bits.

Tolerances.  Scores: bf16 products are exact in fp32 and at most 192 of them are added, in
steps of 16 or fewer whose sums round to 2^-23 of at most A = scale sum |q k|: 2 x 12 x 2^-23 A.
exp2 and its argument are off by at most 2^-20 (1 + |s - max|).  P is rounded to bf16 before
the second product (half a step, 2^-8 of each weight) and the output once more (2^-8 of the
value):
  |out - ref| <= (2^-8 + 2^-11 + D) sum_j p_j |v_j| + 2^-8 |ref|,  D = 2 x 24 x 2^-23 A
  |lse - ref| <= 2 x 24 x 2^-23 A + 2^-20 (1 + spread) + n 2^-24
(2^-11: the fp32 sums of up to 4096 terms; spread: largest minus smallest score seen, whose
weight in the sum is small, so it enters with 1 + min(spread, 30).)"""
import ctypes
import math

import numpy as np
import pytest
import torch


def normal(*shape, seed=0, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(torch.bfloat16)


def cu_of(lens):
    return torch.tensor(np.concatenate([[0], np.cumsum(lens)]), dtype=torch.int32, device="cuda")


def reference(q, k, v, scale, ahead):
    """One sequence and head, float64: out, lse, sum p |v|, A."""
    s = (q @ k.T) * scale
    a = scale * (q.abs() @ k.abs().T)
    nq, nk = s.shape
    seen = torch.arange(nk, device=s.device) <= torch.arange(nq, device=s.device)[:, None] + ahead
    s = s.masked_fill(~seen, -math.inf)
    lse = torch.logsumexp(s, -1) if nk else torch.full((nq,), -math.inf, dtype=s.dtype, device=s.device)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isinf(), 0.0, lse)[:, None]), 0.0)
    big = torch.where(seen, a, 0.0).amax(-1) if nk else torch.zeros_like(lse)
    return p @ v, lse, p @ v.abs(), big


def check(out, lse, q, k, v, lens, klens, scale, heads=None, rows=None):
    H, g = q.shape[1], q.shape[1] // k.shape[1]
    t = u = 0
    for n, m in zip(lens, klens):
        for h in heads if heads is not None else range(H):
            o, z, pv, A = reference(q[t:t + n, h].double(), k[u:u + m, h // g].double(), v[u:u + m, h // g].double(),
                                    scale, m - n)
            D = 48 * 2.0 ** -23 * A[:, None]
            tol = (2.0 ** -8 + 2.0 ** -11 + D) * pv + 2.0 ** -8 * o.abs()
            d = (out[t:t + n, h].double() - o).abs()
            assert bool((d <= tol + 1e-30).all()), (n, m, h, float((d - tol).max()))
            fin = z.isfinite()
            got = lse[t:t + n, h].double()
            assert torch.equal(got[~fin], z[~fin])
            tl = 48 * 2.0 ** -23 * A + 2.0 ** -20 * 31 + m * 2.0 ** -24
            assert bool(((got - z).abs()[fin] <= tl[fin]).all()), (n, m, h, float((got - z).abs()[fin].max()))
        t, u = t + n, u + m


def inputs(lens, klens, H, Hk, rope, seed=0, scale=1.0):
    T, Tk = sum(lens), sum(klens)
    q = normal(T, H, 192 if rope else 128, seed=seed, scale=scale)
    kv = normal(Tk, Hk, 256, seed=seed + 1)
    kr = normal(Tk, 64, seed=seed + 2) if rope else None
    k = kv[:, :, :128]
    full = torch.cat([k, kr[:, None].expand(-1, Hk, -1)], -1) if rope else k
    return q, k, kv[:, :, 128:], kr, full


# ------------------------------------------------------------------ refusals (no GPU)
@pytest.fixture(scope="module")
def lib():
    from tree_speculative_decoding_kd_b200 import build
    build.build()
    from tree_speculative_decoding_kd_b200 import kd
    return kd.lib


def test_host_validation(lib):
    V = ctypes.c_void_p
    ok = [V(16), 512, 128, V(16), 256, 64, V(16), 512, 128, V(16), 64, 0, V(16), 512, 128, V(16), None, 2, 10, 10, 4, 2,
          0.1, V(32), V(16), None, None]
    for i, v in ((0, None), (0, V(8)), (1, 9), (2, -8), (3, None), (4, 4), (6, None), (9, None), (12, V(20)), (13, 1),
                 (15, None), (17, 0), (17, 65536), (18, -1), (19, -1), (20, 0), (20, 129), (20, 3), (21, 0), (21, 8),
                 (22, 0.0), (22, float("nan")), (22, float("inf")), (23, None), (23, V(48)), (24, None)):
        bad = list(ok)
        bad[i] = v
        assert lib.kd_prompt_attn(*bad) == -1, i
    bad = list(ok)
    bad[18], bad[20] = 1 << 30, 4
    assert lib.kd_prompt_attn(*bad) == -1
    none = list(ok)
    none[18] = 0
    assert lib.kd_prompt_attn(*none) == 0


def test_binding_refuses(lib):
    from tree_speculative_decoding_kd_b200 import kd
    x = torch.zeros(4, 2, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kd.kd_prompt_attn(x, x, x, torch.tensor([0, 4], dtype=torch.int32))


# ------------------------------------------------------------------ GPU
@pytest.mark.gpu
@pytest.mark.parametrize("lens,H,Hk,rope", [
    ([1], 1, 1, False), ([1, 1, 1], 4, 2, True), ([2, 0, 5], 3, 3, True), ([16], 8, 1, False), ([127, 128, 129], 2, 1, True),
    ([255, 1, 257], 4, 4, True), ([64, 200, 31, 0, 513], 6, 2, False), ([1000], 2, 2, True), ([385, 640], 5, 1, False),
    ([1] * 300, 2, 2, True), ([2049], 1, 1, False)])
def test_prompt(kd, lens, H, Hk, rope):
    q, k, v, kr, full = inputs(lens, lens, H, Hk, rope, seed=sum(lens))
    err = kd.new_error_word()
    out, lse = kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:] if rope else None, k_rope=kr,
                                 dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    check(out, lse, q, full, v, lens, lens, 1.0 / math.sqrt(192.0 if rope else 128.0))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,klens,H,Hk,rope", [
    ([1, 1], [300, 1], 8, 2, False), ([5, 130, 3], [5, 700, 131], 2, 2, True), ([100, 7], [40, 0], 2, 1, False),
    ([300], [130], 1, 1, True), ([1], [4097], 4, 1, True), ([257, 0, 1], [513, 20, 129], 2, 2, True)])
def test_suffix_queries_and_rows_without_keys(kd, lens, klens, H, Hk, rope):
    """The queries are a sequence's last positions; where there are fewer keys than queries the
    first rows see none: out 0, lse -inf."""
    q, k, v, kr, full = inputs(lens, klens, H, Hk, rope, seed=sum(klens))
    out, lse = kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:] if rope else None, k_rope=kr,
                                 cu_seqlens_k=cu_of(klens), scale=0.05)
    check(out, lse, q, full, v, lens, klens, 0.05)


@pytest.mark.gpu
def test_no_keys_at_all(kd):
    q = normal(5, 2, 192, seed=1)
    none = torch.empty(0, 1, 128, dtype=torch.bfloat16, device="cuda")
    out, lse = kd.kd_prompt_attn(q[..., :128], none, none, cu_of([2, 3]), q_rope=q[..., 128:],
                                 k_rope=torch.empty(0, 64, dtype=torch.bfloat16, device="cuda"), cu_seqlens_k=cu_of([0, 0]))
    assert bool((out == 0).all()) and bool(lse.isneginf().all())
    out, lse = kd.kd_prompt_attn(q[:0, :, :128], none, none, cu_of([0]))
    assert out.shape == (0, 2, 128)


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk", [(28, 4), (7, 1), (128, 128), (128, 1)])
def test_groups_and_expanded_heads(kd, H, Hk):
    """Groups that are no power of two, and keys whose heads are one head expanded (stride 0)."""
    lens = [37, 150]
    q, k, v, _, _ = inputs(lens, lens, H, Hk, False, seed=H)
    out, lse = kd.kd_prompt_attn(q, k, v, cu_of(lens))
    check(out, lse, q, k, v, lens, lens, 1.0 / math.sqrt(128.0), heads=(0, H // 2, H - 1))
    k1, v1 = k[:, :1].expand(-1, H, -1), v[:, :1].expand(-1, H, -1)
    out, lse = kd.kd_prompt_attn(q, k1, v1, cu_of(lens))
    check(out, lse, q, k[:, :1], v[:, :1], lens, lens, 1.0 / math.sqrt(128.0), heads=(0, H - 1))


@pytest.mark.gpu
@pytest.mark.parametrize("lens,klens,H,Hk,rope,heads", [
    ([65, 3, 0, 200], None, 32, 2, True, (0, 15, 16, 31)), ([1, 9, 16, 17], None, 16, 2, False, None),
    ([33, 1, 130], [40, 500, 131], 32, 4, True, (0, 7, 8, 31)), ([300, 2], None, 64, 1, False, (0, 33, 63)),
    ([1] * 70, [77] * 70, 8, 2, False, (0, 3, 4)), ([5, 70, 4], [3, 0, 9], 8, 1, False, None),
    ([37, 0, 18, 19, 300], None, 14, 2, True, (0, 6, 7, 13)), ([130, 1], [7, 200], 15, 3, False, (0, 4, 5)),
    ([25, 26, 60], None, 57, 3, False, (0, 18, 19, 56)), ([70, 3], None, 43, 1, False, (0, 42)),
    ([129], [300], 66, 2, True, (0, 32, 33)), ([2300, 2100], None, 8, 1, False, (0, 7)), ([2049], [2100], 4, 2, True, (1, 2)), ([2050], None, 6, 2, False, (0, 4))])
def test_heads_that_share_keys(kd, lens, klens, H, Hk, rope, heads):
    """Groups of 2 to 64 heads that share a tile (short prompts, with rows to spare or not) and groups
    that do not (long ones, those that would leave much of it empty); what lies behind the last
    sequence stays."""
    klens = klens or lens
    T = sum(lens)
    q, k, v, kr, full = inputs(lens + [3], klens, H, Hk, rope, seed=T)
    out = torch.full((T + 3, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 3, H), 4.0, device="cuda")
    kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:] if rope else None, k_rope=kr,
                      cu_seqlens_k=cu_of(klens), scale=0.07, out=out, lse=lse)
    check(out, lse, q, full, v, lens, klens, 0.07, heads=heads)
    assert bool((out[T:] == 3.0).all()) and bool((lse[T:] == 4.0).all())


@pytest.mark.gpu
@pytest.mark.parametrize("big", [8.0, 40.0])
def test_peaked_scores(kd, big):
    """Scores that climb along the keys: the running maximum moves in every tile."""
    lens = [700, 130]
    q, k, v, kr, full = inputs(lens, lens, 2, 2, False, seed=5)
    ramp = torch.linspace(0.1, 1.0, sum(lens), device="cuda")[:, None, None]
    k = (k.float() * ramp * big).to(torch.bfloat16)
    out, lse = kd.kd_prompt_attn(q, k, v, cu_of(lens))
    check(out, lse, q, k, v, lens, lens, 1.0 / math.sqrt(128.0))


@pytest.mark.gpu
def test_other_sequences_never_enter(kd):
    """NaN and infinite keys and values of a neighbour, and of rows behind the last sequence,
    reach no other row; rows behind the last sequence keep what they held."""
    lens, H = [130, 77, 50], 2
    T = sum(lens)
    q, k, v, kr, full = inputs(lens + [40], lens + [40], H, 1, True, seed=9)
    k, v, kr = k.clone(), v.clone(), kr.clone()
    k[130:207], v[130:207], kr[130:207] = math.nan, math.inf, -math.inf
    k[T:], v[T:], kr[T:], q[T:] = math.nan, math.nan, math.inf, math.nan
    out = torch.full((T + 40, H, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((T + 40, H), 4.0, device="cuda")
    kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:], k_rope=kr, out=out, lse=lse)
    full = torch.cat([k, kr[:, None]], -1)
    for t, n in ((0, 130), (207, 50)):
        check(out[t:t + n], lse[t:t + n], q[t:t + n], full[t:t + n], v[t:t + n], [n], [n], 1.0 / math.sqrt(192.0))
    assert bool((out[T:] == 3.0).all()) and bool((lse[T:] == 4.0).all())


@pytest.mark.gpu
def test_masked_keys_never_enter_inside_a_sequence(kd):
    """Infinite and NaN keys at later positions reach no earlier row."""
    n, H = 200, 1
    q, k, v, _, _ = inputs([n], [n], H, 1, False, seed=2)
    k = k.clone()
    k[150:175], k[175:] = math.nan, math.inf
    out, lse = kd.kd_prompt_attn(q, k, v, cu_of([n]))
    check(out[:150], lse[:150], q[:150], k[:150], v[:150], [150], [150], 1.0 / math.sqrt(128.0))


@pytest.mark.gpu
def test_bad_cumulative_lengths_write_nothing(kd):
    q, k, v, _, _ = inputs([64], [64], 2, 1, False, seed=3)
    out = torch.full((64, 2, 128), 3.0, dtype=torch.bfloat16, device="cuda")
    lse, err = torch.full((64, 2), 4.0, device="cuda"), kd.new_error_word()
    good = [0, 20, 30, 64]
    for cu, ck in (([0, 20, 30, 65], None), ([0, 40, 30, 64], None), ([-5, 10, 30, 64], None), ([1, 20, 30, 64], None),
                   ([0, 2, 3, 2 ** 31 - 1], None), (good, [0, 10, 20, 65]), (good, [0, 20, 10, 64]), (good, [3, 10, 20, 64])):
        kd.kd_prompt_attn(q, k, v, torch.tensor(cu, dtype=torch.int32, device="cuda"), out=out, lse=lse, dev_error=err,
                          cu_seqlens_k=None if ck is None else torch.tensor(ck, dtype=torch.int32, device="cuda"))
        assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_SEQLENS"], cu
        assert bool((out == 3.0).all()) and bool((lse == 4.0).all())
    kd.kd_prompt_attn(q, k[:50], v[:50], torch.tensor([0, 64], dtype=torch.int32, device="cuda"), out=out, lse=lse,
                      dev_error=err)                    # fewer keys than the queries' lengths say
    assert kd.decode_device_error(kd.kd_read_device_error(err)) == ["BAD_SEQLENS"]
    kd.kd_prompt_attn(q, k, v, cu_of([64]), out=out, lse=lse, dev_error=err)
    assert kd.kd_read_device_error(err) == 0
    check(out, lse, q, k, v, [64], [64], 1.0 / math.sqrt(128.0))


@pytest.mark.gpu
def test_strides_repeat_streams_and_graph(kd):
    """Views with odd strides, the same bits again, another stream, and a captured call replayed
    on new inputs."""
    lens, H, Hk = [90, 300], 4, 2
    T = sum(lens)
    buf = normal(T, 3 * H + 1, 136, seed=4)
    q, k, v = buf[:, :H, :128], buf[:, H:H + Hk, 8:136], buf[:, 2 * H:2 * H + Hk, :128]
    cu = cu_of(lens)
    out, lse = kd.kd_prompt_attn(q, k, v, cu)
    check(out, lse, q, k, v, lens, lens, 1.0 / math.sqrt(128.0))
    again, lse2 = kd.kd_prompt_attn(q, k, v, cu)
    assert torch.equal(out, again) and torch.equal(lse, lse2)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o3, z3 = torch.empty_like(out), torch.empty_like(lse)
    torch.cuda.synchronize()
    kd.kd_prompt_attn(q, k, v, cu, out=o3, lse=z3, stream=side)
    side.synchronize()
    assert torch.equal(out, o3)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        kd.kd_prompt_attn(q, k, v, cu, out=o3, lse=z3)
    buf.copy_(normal(T, 3 * H + 1, 136, seed=6))
    g.replay()
    torch.cuda.synchronize()
    check(o3, z3, q, k, v, lens, lens, 1.0 / math.sqrt(128.0))


@pytest.mark.gpu
@pytest.mark.parametrize("H,Hk", [(8, 2), (7, 1), (3, 3)])
def test_heads_before_tokens(kd, H, Hk):
    """Inputs laid out [heads][tokens][elements], each head's tokens in a row, and keys of which
    only every second token is used."""
    lens = [19, 1, 140]
    T = sum(lens)
    q = normal(H, T, 192, seed=1).transpose(0, 1)
    k = normal(Hk, 2 * T, 128, seed=2).transpose(0, 1)[::2]
    kr = normal(1, T, 64, seed=3).transpose(0, 1)[:, 0]
    v = normal(Hk, T, 136, seed=4).transpose(0, 1)[..., 8:]
    out, lse = kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:], k_rope=kr, scale=0.06)
    check(out, lse, q, torch.cat([k, kr[:, None].expand(-1, Hk, -1)], -1), v, lens, lens, 0.06)


@pytest.mark.gpu
def test_long_prompt_sampled_heads(kd):
    lens = [5000]
    q, k, v, kr, full = inputs(lens, lens, 16, 2, True, seed=7)
    out, lse = kd.kd_prompt_attn(q[..., :128], k, v, cu_of(lens), q_rope=q[..., 128:], k_rope=kr)
    check(out, lse, q, full, v, lens, lens, 1.0 / math.sqrt(192.0), heads=(0, 7, 15))
