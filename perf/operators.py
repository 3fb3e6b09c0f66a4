"""Operators around the latent cache, measured: their cases, their plain forms and their calls.

  qk_norm_rope   RMS norm of every query and key head and the position rotation, one pass
  kv_write       latents normed, rope keys rotated and both stored in the cache's next slots,
                 the queries' rope part rotated beside them (contiguous and paged caches)
  prompt_attn    causal attention of packed sequences with grouped heads
  attn_weights   attention weight that each cached slot receives from the accepted nodes,
                 added to what it had received before
  evict          the cache cut down to its sinks, its most recent slots and the slots of the
                 largest accumulated weight

``run`` computes an operator with elementary torch operations when ``own`` is false and calls
the library when it is true.
"""
import math
import random

import numpy as np
import torch

own = False
_KD = []

DC, DR = 512, 64                      # latent and rope widths of the cache
SCALE = 1.0 / math.sqrt(192.0)
EPS = 1e-6


def _kd():
    if not _KD:
        from tree_speculative_decoding_kd_b200 import kd
        _KD.append(kd)
    return _KD[0]


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token for each of 64 requests of a drafter with grouped heads: latency
        dict(name="qk_decode", op="qk_norm_rope", T=64, H=32, Hk=8, D=128, rot=128, off=0, inter=False, norm=True),
        # a batch of prompts of the same drafter: memory bound
        dict(name="qk_prompt", op="qk_norm_rope", T=16385, H=32, Hk=8, D=128, rot=128, off=0, inter=False, norm=True),
        # the node write of the verify step loop (64 requests, 17 nodes)
        dict(name="write_verify", op="kv_write", B=64, lo=17, hi=17, ragged=False, H=64, page=0, past=1900, mix=4),
        # ragged prompts into a paged cache
        dict(name="write_prompt", op="kv_write", B=24, lo=1, hi=1600, ragged=True, H=64, page=64, past=300, mix=7),
        # many short prompts, one token among their lengths: launch and tile-edge costs
        dict(name="prompt_short", op="prompt_attn", B=32, lo=1, hi=300, prefix=0, H=64, Hk=64, rope=True, mix=11),
        # a few prompts of a 64-head latent-attention model, keys and values up-projected
        dict(name="prompt_mla", op="prompt_attn", B=4, lo=900, hi=3100, prefix=0, H=64, Hk=64, rope=True, mix=12),
        # one long prompt of a model with grouped heads
        dict(name="prompt_long", op="prompt_attn", B=1, lo=16384, hi=16384, prefix=0, H=16, Hk=2, rope=False, mix=0),
        # the single-request verify step, every node counted
        dict(name="weights_single", op="attn_weights", B=1, lo=4096, hi=4096, n=17, H=64, accept=False, page=0, mix=1),
        # the verify step loop: the accepted path of each request
        dict(name="weights_loop", op="attn_weights", B=64, lo=2048, hi=16384, n=17, H=64, accept=True, page=0, mix=4),
        # the last 128 tokens of long prompts as the observation window
        dict(name="weights_window", op="attn_weights", B=4, lo=16384, hi=16384, n=128, H=64, accept=False, page=128, mix=5),
        # the loop's caches cut to 2048 slots each
        dict(name="evict_loop", op="evict", B=64, lo=2048, hi=16384, keep=2048, sink=4, recent=256, page=0, mix=4),
        # long contexts cut in half
        dict(name="evict_long", op="evict", B=8, lo=32768, hi=32768, keep=16384, sink=16, recent=1024, page=0, mix=6),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["qk_norm_rope", "kv_write", "prompt_attn", "attn_weights", "evict"])
    mix = rng.randrange(1 << 20)
    if op == "qk_norm_rope":
        D = rng.choice([64, 128, 192, 256])
        Hk = rng.choice([1, 2, 4, 8])
        H = Hk * rng.choice([1, 2, 3, 4, 7, 8])
        most = 16385 * 40 * 128 // ((H + Hk) * D)
        rot = 16 * rng.randint(1, D // 16)
        return dict(op=op, T=_log(rng, 1, most), H=H, Hk=Hk, D=D, rot=rot, off=rng.choice([0, D - rot]),
                    inter=rng.random() < 0.5, norm=rng.random() < 0.8)
    if op == "kv_write":
        page = rng.choice([0, 0, 16, 64, 128])
        H = rng.choice([5, 16, 32, 64, 128])
        if rng.random() < 0.5:
            n = _log(rng, 1, 128)
            return dict(op=op, B=_log(rng, 1, 96), lo=n, hi=n, ragged=False, H=H, page=page,
                        past=rng.randint(0, 900), mix=mix)
        B = _log(rng, 1, 32)
        return dict(op=op, B=B, lo=1, hi=_log(rng, 2, 16000 // B), ragged=True, H=H, page=page,
                    past=rng.randint(0, 900), mix=mix)
    if op == "prompt_attn":
        rope = rng.random() < 0.6
        Hk = rng.choice([1, 2, 4, 8]) if not rope else rng.choice([8, 16, 32, 64])
        H = Hk * rng.choice([1, 2, 4, 7]) if not rope else Hk
        B = _log(rng, 1, 32)
        hi = max(1, int(min(_log(rng, 1, 8192), math.sqrt(3.0e8 / (H * B)))))
        return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi,
                    prefix=rng.choice([0, 0, rng.randint(1, 700)]), H=H, Hk=Hk, rope=rope, mix=mix)
    if op == "attn_weights":
        H, n = rng.choice([5, 16, 64, 128]), _log(rng, 1, 128)
        B = _log(rng, 1, 64)
        hi = min(_log(rng, 1, 32768), int(6.0e8 / (B * n * H)))
        return dict(op=op, B=B, lo=max(0, hi // rng.choice([1, 2, 8])), hi=max(1, hi), n=n, H=H,
                    accept=rng.random() < 0.5, page=rng.choice([0, 0, 64, 128, 256]), mix=mix)
    B = _log(rng, 1, 64)
    hi = min(_log(rng, 8, 32768), 600000 // B)
    keep = rng.randint(1, max(1, min(hi, 250000 // B)))
    recent = rng.randint(0, keep // 2)
    return dict(op=op, B=B, lo=max(1, hi // rng.choice([1, 2, 8])), hi=hi, keep=keep,
                sink=rng.randint(0, min(16, keep - recent)), recent=recent, page=rng.choice([0, 0, 64]), mix=mix)


def _lens(case):
    """Lengths of the case's requests (tokens written, prompt lengths or committed lengths)."""
    r = random.Random(case["mix"])
    return [r.randint(case["lo"], case["hi"]) for _ in range(case["B"])]


def _accepted(case):
    """Accepted nodes of each request: 1 + the count of successes before the first failure (p = 0.7)."""
    r, out = random.Random(case["mix"] + 1), []
    for _ in range(case["B"]):
        k = 1
        while k < case["n"] and r.random() < 0.7:
            k += 1
        out.append(k if case["accept"] else case["n"])
    return out


def work(case):
    op = case["op"]
    if op == "qk_norm_rope":
        e = case["T"] * (case["H"] + case["Hk"]) * case["D"]
        b = 4 * e + case["T"] * (4 + 4 * case["rot"])
        return dict(bytes=b + (4 * case["D"] if case["norm"] else 0), flops=7 * e)
    if op == "kv_write":
        t = sum(_lens(case))
        return dict(bytes=t * (4 * (DC + DR) + 4 * case["H"] * DR + 4 * DR + 4), flops=t * (4 * DC + 3 * DR * (1 + case["H"])))
    if op == "prompt_attn":
        dk, H, Hk, p = 128 + (64 if case["rope"] else 0), case["H"], case["Hk"], case["prefix"]
        flops = sum((n * (n + 1) // 2 + n * p) * 2 * (dk + 128) * H for n in _lens(case))
        q, k = sum(_lens(case)), sum(_lens(case)) + p * case["B"]
        return dict(bytes=2 * q * H * (dk + 128) + 2 * k * (Hk * 256 + (64 if case["rope"] else 0)) + 4 * q * H, flops=flops)
    if op == "attn_weights":
        b = f = 0
        for L, a in zip(_lens(case), _accepted(case)):
            rows = a * case["H"]
            b += (L + a) * (2 * (DC + DR) + 4) + L * 4 + rows * (2 * (DC + DR) + 4)
            f += rows * (L + a) * (2 * (DC + DR) + 2)
        return dict(bytes=b, flops=f)
    b = 0
    for L in _lens(case):
        k = min(L, case["keep"])
        b += L * 4 + k * (4 * (DC + DR) + 4 + 4) + 8
    return dict(bytes=b, flops=sum(_lens(case)))


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)


def _i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


def _table(rows, rot):
    """cos | sin of position * 10000^(-2i / rot): angles in 64 bits, rounded once."""
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = torch.arange(rows, dtype=torch.float64, device="cuda")[:, None] * inv
    return torch.cat([ang.cos(), ang.sin()], 1).to(torch.float32).contiguous()


def _pages(g, B, cap, page):
    """Shuffled page table [B][ceil(cap / page)] with a few pages that no request has."""
    M = -(-cap // page)
    perm = torch.randperm(B * M + 3, generator=g, device="cuda")
    return perm[: B * M].view(B, M).to(torch.int32).contiguous(), B * M + 3


def prepare(case, seed):
    g, op = _gen(seed), case["op"]
    s = dict(case=case, op=op, err=torch.zeros(1, dtype=torch.int32, device="cuda"))
    if op == "qk_norm_rope":
        T, H, Hk, D = case["T"], case["H"], case["Hk"], case["D"]
        qkv = _normal(g, T, H + 2 * Hk, D)                       # the fused projection's output
        s["q"], s["k"] = qkv[:, :H], qkv[:, H:H + Hk]
        s["pos"] = torch.randint(0, 40960, (T,), generator=g, device="cuda", dtype=torch.int32)
        s["table"] = _table(40960, case["rot"])
        s["qw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["kw"] = (1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(torch.bfloat16) if case["norm"] else None
        s["q_out"] = torch.zeros(T, H, D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.zeros(T, Hk, D, dtype=torch.bfloat16, device="cuda")
    elif op == "kv_write":
        lens, B, H, page = _lens(case), case["B"], case["H"], case["page"]
        T, r = sum(lens), random.Random(seed)
        past = [r.randint(0, case["past"]) for _ in range(B)]
        cap = case["past"] + max(lens) + case["mix"] % 10
        s["kv"] = _normal(g, T, DC + DR)                          # the down-projection's output
        s["q_rope"] = _normal(g, T, H, 192)[:, :, 128:]           # the rope part of the query heads
        s["lens"], s["n"] = _i32(past), lens[0]
        s["cu"] = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist()) if case["ragged"] else None
        s["pos"] = _i32([p + i for p, n in zip(past, lens) for i in range(n)])
        s["w"] = (1 + 0.2 * torch.randn(DC, generator=g, device="cuda")).to(torch.bfloat16)
        s["table"] = _table(cap + 128, DR)
        s["pt"], pool = _pages(g, B, cap, page) if page else (None, 0)
        rows = (pool * page,) if page else (B, cap)
        s["c_kv"] = torch.zeros(*rows, DC, dtype=torch.bfloat16, device="cuda")
        s["k_rope"] = torch.zeros(*rows, DR, dtype=torch.bfloat16, device="cuda")
        s["q_out"] = torch.zeros(T, H, DR, dtype=torch.bfloat16, device="cuda")
    elif op == "prompt_attn":
        lens, H, Hk, p = _lens(case), case["H"], case["Hk"], case["prefix"]
        T, Tk = sum(lens), sum(lens) + p * case["B"]
        q = _normal(g, T, H, 192 if case["rope"] else 128)
        kv = _normal(g, Tk, Hk, 256)                              # keys and values of one up-projection
        s["q"], s["k"], s["v"] = q[:, :, :128], kv[:, :, :128], kv[:, :, 128:]
        s["q_rope"] = q[:, :, 128:] if case["rope"] else None
        s["k_rope"] = _normal(g, Tk, DR) if case["rope"] else None   # one rope key for all heads
        s["cu"] = _i32(np.concatenate([[0], np.cumsum(lens)]).tolist())
        s["cu_k"] = _i32(np.concatenate([[0], np.cumsum([n + p for n in lens])]).tolist()) if p else None
        s["scale"] = 1.0 / math.sqrt(192.0 if case["rope"] else 128.0)
        s["out"] = torch.zeros(T, H, 128, dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros(T, H, dtype=torch.float32, device="cuda")
    elif op == "attn_weights":
        B, n, H, page = case["B"], case["n"], case["H"], case["page"]
        lens, acc, r = _lens(case), _accepted(case), random.Random(seed)
        cap = max(lens) + n + case["mix"] % 6
        paths, vis = [], np.zeros((B, n, (n + 31) // 32), np.uint32)
        for b in range(B):
            path = [0] + sorted(r.sample(range(1, n), acc[b] - 1))
            par = [-1] + [r.randrange(i) for i in range(1, n)]
            for u, v in zip(path, path[1:]):
                par[v] = u
            for i in range(n):
                if par[i] >= 0:
                    vis[b, i] = vis[b, par[i]]
                vis[b, i, i // 32] |= np.uint32(1 << (i % 32))
            paths.append(path + [-1] * (n - len(path)))
        s["q"], s["q_rope"] = _normal(g, B, n, H, DC), _normal(g, B, n, H, DR)
        s["pt"], pool = _pages(g, B, cap, page) if page else (None, 0)
        rows = (pool * page,) if page else (B, cap)
        s["c_kv"], s["k_rope"] = _normal(g, *rows, DC), _normal(g, *rows, DR)
        s["lens"] = _i32(lens)
        s["vis"] = torch.from_numpy(vis.view(np.int32)).cuda()
        s["path"], s["alen"] = (_i32(paths), _i32(acc)) if case["accept"] else (None, None)
        # lse of normal scores: ln(keys) + variance / 2
        q2 = s["q"].float().square().sum(-1) + s["q_rope"].float().square().sum(-1)
        s["lse"] = (s["lens"].float() + 1).log()[:, None, None] + 0.5 * SCALE * SCALE * q2
        cap = s["pt"].shape[1] * page if page else cap
        s["w_in"] = -torch.rand(B, cap, generator=g, device="cuda").clamp_min(1e-9).log()
        s["w_out"] = torch.zeros(B, cap, dtype=torch.float32, device="cuda")
    else:
        B, page, lens = case["B"], case["page"], _lens(case)
        cap, dcap = max(lens) + case["mix"] % 8, case["keep"] + 64
        s["pt"], pool = _pages(g, B, cap, page) if page else (None, 0)
        s["dpt"], dpool = _pages(g, B, dcap, page) if page else (None, 0)
        rows, drows = ((pool * page,), (dpool * page,)) if page else ((B, cap), (B, dcap))
        s["c_kv"], s["k_rope"] = _normal(g, *rows, DC), _normal(g, *rows, DR)
        s["c_dst"] = torch.zeros(*drows, DC, dtype=torch.bfloat16, device="cuda")
        s["r_dst"] = torch.zeros(*drows, DR, dtype=torch.bfloat16, device="cuda")
        cap = s["pt"].shape[1] * page if page else cap
        dcap = s["dpt"].shape[1] * page if page else dcap
        w = -torch.rand(B, cap, generator=g, device="cuda").clamp_min(1e-9).log()
        s["w_in"] = (w * 64).floor() / 64                        # equal weights occur
        s["w_out"] = torch.zeros(B, dcap, dtype=torch.float32, device="cuda")
        s["lens"] = _i32(lens)
        s["lens_out"] = torch.zeros(B, dtype=torch.int32, device="cuda")
        s["kept"] = torch.zeros(B, case["keep"], dtype=torch.int32, device="cuda")
    return s


# ------------------------------------------------------------------ plain forms
def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, cs, inter):
    """Rotates the last axis of x (fp32); cs: cos | sin rows that broadcast against x."""
    h = x.shape[-1] // 2
    c, s = cs[..., :h], cs[..., h:]
    if inter:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * c - b * s, a * s + b * c], -1).flatten(-2)
    a, b = x[..., :h], x[..., h:]
    return torch.cat([a * c - b * s, a * s + b * c], -1)


def _rows(pt, page, cap, B):
    """Row of every logical slot [B][slots] in a flat cache."""
    if pt is None:
        return torch.arange(B * cap, device="cuda").view(B, cap)
    inside = torch.arange(page, device="cuda")
    return (pt.long()[:, :, None] * page + inside).flatten(1)


def _plain_qk(s):
    c = s["case"]
    lo, hi, cs = c["off"], c["off"] + c["rot"], s["table"][s["pos"].long()][:, None]
    outs = []
    for x, w, out in ((s["q"], s["qw"], s["q_out"]), (s["k"], s["kw"], s["k_out"])):
        y = _norm(x.float(), w)
        out.copy_(torch.cat([y[..., :lo], _rotate(y[..., lo:hi], cs, c["inter"]), y[..., hi:]], -1))
        outs.append(out)
    return outs


def _token_slots(s):
    """Request and cache slot of every token."""
    c, T = s["case"], s["kv"].shape[0]
    cu = s["cu"] if s["cu"] is not None else torch.arange(c["B"] + 1, device="cuda", dtype=torch.int32) * s["n"]
    t = torch.arange(T, device="cuda", dtype=torch.int32)
    b = torch.searchsorted(cu, t, right=True) - 1
    return b, s["lens"][b].long() + (t - cu[b]).long()


def _plain_write(s):
    c = s["case"]
    cs = s["table"][s["pos"].long()]
    lat = _norm(s["kv"][:, :DC].float(), s["w"])
    rope = _rotate(s["kv"][:, DC:].float(), cs, True)
    s["q_out"].copy_(_rotate(s["q_rope"].float(), cs[:, None], True))
    b, slot = _token_slots(s)
    cap = s["c_kv"].shape[1] if s["pt"] is None else 0
    row = _rows(s["pt"], c["page"], cap, c["B"])[b, slot]
    s["c_kv"].view(-1, DC)[row] = lat.to(torch.bfloat16)
    s["k_rope"].view(-1, DR)[row] = rope.to(torch.bfloat16)
    return [s["c_kv"], s["k_rope"], s["q_out"]]


def _prompt_mask(s):
    """[T][Tk]: same sequence, and not after the query (the queries are the sequence's last tokens)."""
    cu, ck = s["cu"].long(), (s["cu_k"] if s["cu_k"] is not None else s["cu"]).long()
    t, u = torch.arange(s["q"].shape[0], device="cuda"), torch.arange(s["k"].shape[0], device="cuda")
    bt, bu = torch.searchsorted(cu, t, right=True) - 1, torch.searchsorted(ck, u, right=True) - 1
    end = ck[bt + 1] - (cu[bt + 1] - t) + 1
    return (bt[:, None] == bu) & (u < end[:, None])


def _plain_prompt(s):
    g = s["case"]["H"] // s["case"]["Hk"]
    q, k = s["q"].float(), s["k"].float()
    if s["k_rope"] is not None:
        q = torch.cat([q, s["q_rope"].float()], -1)
        k = torch.cat([k, s["k_rope"].float()[:, None].expand(-1, k.shape[1], -1)], -1)
    k, v = k.repeat_interleave(g, 1), s["v"].float().repeat_interleave(g, 1)
    p = torch.matmul(q.transpose(0, 1), k.permute(1, 2, 0)).mul_(s["scale"])         # [H][T][Tk]
    p.masked_fill_(~_prompt_mask(s), -math.inf)
    m = p.amax(-1, keepdim=True)
    m = torch.where(m.isinf(), 0.0, m)                      # a row without keys
    p.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.transpose(0, 1)) / torch.where(z > 0, z, 1.0)
    s["out"].copy_(o.transpose(0, 1))
    s["lse"].copy_((z.log() + m)[..., 0].t())
    return [s["out"], s["lse"]]


def _plain_weights(s):
    c, n = s["case"], s["case"]["n"]
    B, cap = s["w_in"].shape
    flat = _rows(s["pt"], c["page"], cap, B)
    k = torch.cat([s["c_kv"].view(-1, DC)[flat], s["k_rope"].view(-1, DR)[flat]], -1).float()
    q = torch.cat([s["q"], s["q_rope"]], -1).float()                                   # [B][n][H][576]
    node = torch.arange(n, device="cuda").expand(B, n) if s["path"] is None else s["path"].long()
    count = torch.full((B,), n, device="cuda") if s["path"] is None else s["alen"].long()
    here = torch.arange(n, device="cuda") < count[:, None]                              # [B][n] counted
    node = torch.where(here, node, 0)
    q = q.gather(1, node[:, :, None, None].expand(-1, -1, *q.shape[2:]))
    lse = s["lse"].gather(1, node[:, :, None].expand(-1, -1, c["H"]))
    bits = (s["vis"][..., None] >> torch.arange(32, device="cuda", dtype=torch.int32)).bitwise_and(1).flatten(2)[..., :n].bool()
    bits = bits.gather(1, node[:, :, None].expand(-1, -1, n)) & here[:, :, None]       # [B][n][n]
    j = torch.arange(cap, device="cuda")
    L = s["lens"].long()[:, None]
    tree = (j - L).clamp(0, n - 1)                                                      # [B][cap]
    see = torch.where((j < L)[:, None], here[:, :, None], bits.gather(2, tree[:, None].expand(-1, n, -1)))
    see &= (j < L + n)[:, None]
    p = torch.matmul(q.flatten(1, 2), k.transpose(1, 2)).view(B, n, c["H"], cap)
    p.mul_(SCALE).sub_(lse[..., None]).exp_().masked_fill_(~see[:, :, None], 0.0)
    col = p.sum((1, 2))
    src = torch.where(j < L, j, L + node.gather(1, tree)).clamp_max(cap - 1)            # compacted order
    got = col.gather(1, src) + torch.where(j < L, s["w_in"], 0.0)
    s["w_out"].copy_(torch.where(j < L + count[:, None], got, s["w_out"]))
    return [s["w_out"]]


def _plain_evict(s):
    c, keep = s["case"], s["case"]["keep"]
    B, cap = s["w_in"].shape
    L, j = s["lens"].long()[:, None], torch.arange(cap, device="cuda")
    w = s["w_in"].double()
    w = torch.where((j < c["sink"]) | (j >= L - c["recent"]), math.inf, w)
    w = torch.where(j < L, w, -math.inf)
    best = torch.sort(w, dim=1, descending=True, stable=True).indices[:, :keep]          # ties: the lowest slot
    new = L.clamp_max(keep)[:, 0]
    slot = torch.arange(best.shape[1], device="cuda")
    live = slot < new[:, None]
    kept = torch.where(live, best, cap).sort(1).values
    s["kept"].fill_(-1)
    s["kept"][:, : best.shape[1]] = torch.where(live, kept, -1).int()
    s["lens_out"].copy_(new)
    src = _rows(s["pt"], c["page"], cap, B).gather(1, kept.clamp_max(cap - 1))[live]
    dst = _rows(s["dpt"], c["page"], s["w_out"].shape[1], B)[:, : best.shape[1]][live]
    s["c_dst"].view(-1, DC)[dst] = s["c_kv"].view(-1, DC)[src]
    s["r_dst"].view(-1, DR)[dst] = s["k_rope"].view(-1, DR)[src]
    moved = s["w_in"].gather(1, kept.clamp_max(cap - 1))
    s["w_out"][:, : best.shape[1]] = torch.where(live, moved, s["w_out"][:, : best.shape[1]])
    return [s["c_dst"], s["r_dst"], s["w_out"], s["kept"], s["lens_out"]]


# ------------------------------------------------------------------ the library's calls
def _own_qk(s):
    c = s["case"]
    return list(_kd().kd_qk_norm_rope(s["q"], s["k"], s["pos"], s["table"], q_weight=s["qw"], k_weight=s["kw"],
                                      eps=EPS, rot_offset=c["off"], interleaved=c["inter"], q_out=s["q_out"],
                                      k_out=s["k_out"], dev_error=s["err"]))


def _own_write(s):
    kd, page = _kd(), s["case"]["page"]
    more = dict(cu_seqlens=s["cu"], B=s["case"]["B"], kv_weight=s["w"], eps=EPS, interleaved=True,
                q_rope_in=s["q_rope"], q_rope_out=s["q_out"], dev_error=s["err"])
    if page:
        kd.kd_kv_norm_rope_write_paged(s["c_kv"], s["k_rope"], s["pt"], page, s["lens"], s["kv"], s["pos"],
                                       s["table"], **more)
    else:
        kd.kd_kv_norm_rope_write(s["c_kv"], s["k_rope"], s["lens"], s["kv"], s["pos"], s["table"], **more)
    return [s["c_kv"], s["k_rope"], s["q_out"]]


def _own_prompt(s):
    return list(_kd().kd_prompt_attn(s["q"], s["k"], s["v"], s["cu"], q_rope=s["q_rope"], k_rope=s["k_rope"],
                                     cu_seqlens_k=s["cu_k"], scale=s["scale"], out=s["out"], lse=s["lse"],
                                     dev_error=s["err"]))


def _own_weights(s):
    kd, page = _kd(), s["case"]["page"]
    more = dict(path=s["path"], length=s["alen"], scale=SCALE, weights_in=s["w_in"], weights_out=s["w_out"],
                dev_error=s["err"])
    if page:
        return [kd.kd_kv_attn_weights_paged(s["q"], s["q_rope"], s["c_kv"], s["k_rope"], s["pt"], page, s["lens"],
                                            s["vis"], s["lse"], **more)]
    return [kd.kd_kv_attn_weights(s["q"], s["q_rope"], s["c_kv"], s["k_rope"], s["lens"], s["vis"], s["lse"], **more)]


def _own_evict(s):
    kd, c = _kd(), s["case"]
    more = dict(keep=c["keep"], sink=c["sink"], recent=c["recent"], weights_out=s["w_out"], lens_out=s["lens_out"],
                kept=s["kept"], dev_error=s["err"])
    if c["page"]:
        kd.kd_kv_evict_paged(s["c_kv"], s["k_rope"], s["pt"], c["page"], s["lens"], s["w_in"], c_dst=s["c_dst"],
                             r_dst=s["r_dst"], dst_page_table=s["dpt"], **more)
    else:
        kd.kd_kv_evict(s["c_kv"], s["k_rope"], s["lens"], s["w_in"], c_dst=s["c_dst"], r_dst=s["r_dst"], **more)
    return [s["c_dst"], s["r_dst"], s["w_out"], s["kept"], s["lens_out"]]


def run(state):
    if own:
        return {"qk_norm_rope": _own_qk, "kv_write": _own_write, "prompt_attn": _own_prompt,
                "attn_weights": _own_weights, "evict": _own_evict}[state["op"]](state)
    return {"qk_norm_rope": _plain_qk, "kv_write": _plain_write, "prompt_attn": _plain_prompt,
            "attn_weights": _plain_weights, "evict": _plain_evict}[state["op"]](state)


# ------------------------------------------------------------------ the definitions in 64 bits
def _turned(x, pos, inter):
    """x (float64) [T][...][rot] as complex numbers, pair i multiplied by the table's cos + i sin at pos."""
    rot = x.shape[-1]
    inv = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
    ang = (pos.double()[:, None] * inv).view(pos.shape[0], *([1] * (x.dim() - 2)), rot // 2)
    # the rotation's cosines and sines are inputs, held in 32 bits
    e = torch.complex(ang.cos().float().double(), ang.sin().float().double())
    pair = x.unflatten(-1, (rot // 2, 2)) if inter else torch.stack(x.split(rot // 2, -1), -1)
    z = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * e)
    return z.flatten(-2) if inter else torch.cat([z[..., 0], z[..., 1]], -1)


def _scaled(x, w):
    if w is None:
        return x
    n = x.shape[-1]
    return x * w.double() / ((x * x).sum(-1, keepdim=True) / n + EPS).sqrt()


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "qk_norm_rope":
        got = []
        for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
            y = _scaled(x.double(), w)
            part = slice(case["off"], case["off"] + case["rot"])
            y[..., part] = _turned(y[..., part], s["pos"], case["inter"])
            got.append(y)
        return got
    if op == "kv_write":
        lens, past, page = _lens(case), s["lens"].tolist(), case["page"]
        rows, t = [], 0
        for b, n in enumerate(lens):
            slots = torch.arange(past[b], past[b] + n, device="cuda")
            rows.append(s["pt"][b].long()[slots // page] * page + slots % page if page
                        else b * s["c_kv"].shape[1] + slots)
        rows = torch.cat(rows)
        c, r = s["c_kv"].double(), s["k_rope"].double()
        c.view(-1, DC)[rows] = _scaled(s["kv"][:, :DC].double(), s["w"])
        r.view(-1, DR)[rows] = _turned(s["kv"][:, DC:].double(), s["pos"], True)
        return [c, r, _turned(s["q_rope"].double(), s["pos"], True)]
    if op == "prompt_attn":
        H, g, p = case["H"], case["H"] // case["Hk"], case["prefix"]
        out = torch.zeros(s["q"].shape[0], H, 128, dtype=torch.float64, device="cuda")
        lse = torch.zeros(s["q"].shape[0], H, dtype=torch.float64, device="cuda")
        t = u = 0
        for n in _lens(case):
            ahead = torch.ones(n, n + p, dtype=torch.bool, device="cuda").triu(p + 1)
            for h in range(H):
                x = s["q"][t:t + n, h].double() @ s["k"][u:u + n + p, h // g].double().T
                if s["k_rope"] is not None:
                    x += s["q_rope"][t:t + n, h].double() @ s["k_rope"][u:u + n + p].double().T
                x = (x * s["scale"]).masked_fill(ahead, -math.inf)
                lse[t:t + n, h] = torch.logsumexp(x, -1)
                out[t:t + n, h] = torch.softmax(x, -1) @ s["v"][u:u + n + p, h // g].double()
            t, u = t + n, u + n + p
        return [out, lse]
    if op == "attn_weights":
        w = s["w_out"].double()
        vis = s["vis"].cpu().numpy().view(np.uint32)
        for b, (L, a) in enumerate(zip(_lens(case), _accepted(case))):
            path = s["path"][b, :a].tolist() if s["path"] is not None else list(range(case["n"]))
            slots = torch.arange(L + case["n"], device="cuda")
            if case["page"]:
                at = s["pt"][b].long()[slots // case["page"]] * case["page"] + slots % case["page"]
                c, r = s["c_kv"][at].double(), s["k_rope"][at].double()
            else:
                c, r = s["c_kv"][b, : L + case["n"]].double(), s["k_rope"][b, : L + case["n"]].double()
            total = torch.zeros(L + case["n"], dtype=torch.float64, device="cuda")
            for i in path:
                x = SCALE * (s["q"][b, i].double() @ c.T + s["q_rope"][b, i].double() @ r.T)
                x = torch.exp(x - s["lse"][b, i].double()[:, None]).sum(0)
                seen = [bool(vis[b, i, k // 32] >> np.uint32(k % 32) & 1) for k in range(case["n"])]
                x[L:] = torch.where(torch.tensor(seen, device="cuda"), x[L:], 0.0)
                total += x
            w[b, :L] = s["w_in"][b, :L].double() + total[:L]
            w[b, L:L + a] = total[L + torch.tensor(path, device="cuda")]
        return [w]
    c, r, w = s["c_dst"].double(), s["r_dst"].double(), s["w_out"].double()
    kept = np.full((case["B"], case["keep"]), -1, np.int32)
    new, weights, page = [], s["w_in"].cpu().numpy(), case["page"]
    for b, L in enumerate(_lens(case)):
        first = min(case["sink"], L)
        last = max(first, L - case["recent"])
        ids = list(range(L))
        if L > case["keep"]:
            order = np.lexsort((np.arange(first, last), -weights[b, first:last])) + first
            room = case["keep"] - first - (L - last)
            ids = sorted([*range(first), *order[:room].tolist(), *range(last, L)])
        kept[b, : len(ids)] = ids
        new.append(len(ids))
        at, to = torch.tensor(ids, device="cuda"), torch.arange(len(ids), device="cuda")
        w[b, to] = s["w_in"][b, at].double()
        if page:
            at = s["pt"][b].long()[at // page] * page + at % page
            to = s["dpt"][b].long()[to // page] * page + to % page
            c[to], r[to] = s["c_kv"][at].double(), s["k_rope"][at].double()
        else:
            c[b, to], r[b, to] = s["c_kv"][b, at].double(), s["k_rope"][b, at].double()
    return [c, r, w, torch.from_numpy(kept), torch.tensor(new, dtype=torch.int32)]
