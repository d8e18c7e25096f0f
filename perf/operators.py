"""The serving operators next to the KV codec, as they are timed: one pass of each through the
framework (own = True) or in elementary torch operations (own = False).

  append     new tokens' keys and values rotated and written into a paged cache, the queries
             rotated beside them (sz_kv_append_paged)
  norm_rope  RMS norm of every query and key head and the position rotation (sz_qk_norm_rope)
  attn       attention of new tokens over the paged cache (sz_attn_paged)

Head layouts are those of the KV configurations in kvgen (Llama-3-8B and Qwen3-32B: 8 KV heads of
128; Qwen3-30B-A3B: 4 of 128, E5M2; Phi-2: 32 of 80), with 4 or 8 query heads to a KV head where
queries are grouped.
"""
import math
import random

import torch

own = False

EPS = 1e-6
BASE = 10000.0


# ------------------------------------------------------------------------------------ the cases

def _append(name, seqs, new, kv, heads, kv_heads, dim, rot, page, e5m2=False, norm=False, interleaved=False):
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "kv": kv, "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "rot": rot, "page": page, "e5m2": e5m2, "norm": norm,
            "interleaved": interleaved}


def _norm_rope(name, tokens, heads, kv_heads, dim, rot, interleaved=False):
    return {"name": name, "op": "norm_rope", "tokens": tokens, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "rot": rot, "interleaved": interleaved}


def _attn(name, seqs, new, kv, heads, kv_heads, dim, page, e5m2=False, window=0, ragged=True, lse=False):
    return {"name": name, "op": "attn", "seqs": seqs, "new": new, "kv": kv, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "page": page, "e5m2": e5m2, "window": window, "ragged": ragged, "lse": lse}


def listed():
    return [
        # one stream's next token: latency is everything
        _append("append 1 token", 1, 1, 777, 32, 8, 128, 128, 16),
        # a full decode batch of a model that normalises its queries and keys
        _append("append 256 decoding", 256, 1, 2048, 64, 8, 128, 128, 16, norm=True),
        # chunks of several prompts into an 8-bit cache
        _append("append chunks e5m2", 6, 1500, 4096, 32, 4, 128, 128, 64, e5m2=True),
        # a prompt of the partly rotated, ungrouped 80-wide heads, odd length and page
        _append("append prompt 80 wide", 1, 1023, 1023, 32, 32, 80, 32, 13),
        # a decode batch whose cache is kept contiguous
        _norm_rope("norm+rope 48 tokens", 48, 64, 8, 128, 128),
        # a long prompt's chunk
        _norm_rope("norm+rope 16384 tokens", 16384, 32, 8, 128, 128),
        # one stream's next token over a short context
        _attn("attn 1 token", 1, 1, 777, 32, 8, 128, 16),
        # a ragged decode batch over long contexts
        _attn("attn 64 decoding", 64, 1, 8192, 32, 8, 128, 16),
        # one stream over a very long context in 8 bits
        _attn("attn long e5m2", 1, 1, 131072, 32, 4, 128, 64, e5m2=True, ragged=False),
        # a chunk of a prompt over what came before it
        _attn("attn chunk", 1, 2048, 8192, 32, 8, 128, 16, ragged=False, lse=True),
        # chunks of several prompts, ragged, with a window, 8 bits, pages that no tile ends on
        _attn("attn ragged window e5m2", 5, 700, 5000, 32, 4, 128, 13, e5m2=True, window=1024),
        # a whole prompt of the ungrouped 80-wide heads
        _attn("attn prompt 80 wide", 2, 1024, 1024, 32, 32, 80, 16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kv_heads, group, dim = rng.choice([(8, 4, 128), (8, 8, 128), (4, 8, 128), (32, 1, 80), (8, 1, 64), (2, 7, 128)])
    heads = kv_heads * group
    page = rng.choice([8, 13, 16, 32, 64, 100])
    rot = rng.choice([dim, dim, dim // 2 // 8 * 8])
    op = rng.choice(["append", "norm_rope", "attn", "attn"])
    e5m2 = rng.random() < 0.4
    if op == "norm_rope":
        return {k: v for k, v in _norm_rope("", _log(rng, 1, 8000), heads, kv_heads, dim, rot,
                                            rng.random() < 0.3).items() if k != "name"}
    if rng.random() < 0.5:  # decoding: a token or a few of many sequences
        seqs, new = _log(rng, 1, 200), rng.choice([1, 1, 1, 2, 5])
        kv = max(new, _log(rng, 64, min(100000, 400000 // seqs)))
    else:                   # prompts: chunks of a few sequences
        seqs, new = rng.randint(1, 6), _log(rng, 16, 1600)
        kv = new + rng.choice([0, _log(rng, 16, 5000)])
        new = max(1, min(new, 12000000 // (seqs * kv)))
    if op == "append":
        c = _append("", seqs, new, kv, heads, kv_heads, dim, rot, page, e5m2, rng.random() < 0.4,
                    rng.random() < 0.3)
    else:
        c = _attn("", seqs, new, kv, heads, kv_heads, dim, page, e5m2, rng.choice([0, 0, 0, _log(rng, 16, 2000)]),
                  rng.random() < 0.7, rng.random() < 0.5)
    del c["name"]
    return c


def _lengths(case):
    """New tokens and context length (the new tokens included) of every sequence."""
    n, new, kv = case["seqs"], case["new"], case["kv"]
    if not case.get("ragged", True) or n == 1:
        return [new] * n, [kv] * n
    r = random.Random(n * 1000003 + new * 1009 + kv)
    q = [new if new == 1 else r.randint(max(1, new // 4), new) for _ in range(n)]
    q[0] = new
    total = [max(a, r.randint(kv // 4, kv)) for a in q]
    total[0] = kv
    return q, total


# ------------------------------------------------------------------------------------ the inputs

def _rope_table(positions, rot, device):
    """[positions, rot] float32: the cosines of a position's rot/2 angles, then their sines."""
    inv = BASE ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=device) / rot)
    a = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _heads(g, shape, device):
    """Activations of attention heads: normal, with a scale for each channel."""
    s = torch.exp(0.5 * torch.randn(shape[-2:], generator=g, device=device))
    return (torch.randn(shape, generator=g, device=device) * s).bfloat16()


def prepare(case, seed):
    dev = torch.device("cuda", torch.cuda.current_device())
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    s = {"case": dict(case)}
    if case["op"] == "norm_rope":
        t = case["tokens"]
        qkv = _heads(g, (t, h + 2 * hk, d), dev)  # the projection's output: queries and keys are views of it
        s.update(q=qkv[:, :h], k=qkv[:, h:h + hk], q_out=torch.empty(t, h, d, dtype=torch.bfloat16, device=dev),
                 k_out=torch.empty(t, hk, d, dtype=torch.bfloat16, device=dev), rope=_rope_table(2 * t + 64, case["rot"], dev),
                 positions=torch.randint(0, 2 * t + 64, (t,), generator=g, device=dev, dtype=torch.int32))
    else:
        q_len, kv_len = _lengths(case)
        t, p = sum(q_len), case["page"]
        counts = [-(-n // p) for n in kv_len]
        pages = sum(counts) + 3
        perm = torch.randperm(pages, generator=g, device=dev).int()
        table = torch.zeros(case["seqs"], max(counts), dtype=torch.int32, device=dev)
        first = torch.tensor([sum(counts[:b]) for b in range(len(counts))], device=dev)
        j = torch.arange(max(counts), device=dev)
        used = j[None] < torch.tensor(counts, device=dev)[:, None]
        table[used] = perm[(first[:, None] + j[None])[used]]
        kind = torch.float8_e5m2 if case["e5m2"] else torch.bfloat16
        pools = [_heads(g, (pages, p, hk, d), dev).to(kind) for _ in range(2)]
        ends = torch.cumsum(torch.tensor([0] + q_len, device=dev), 0)
        s.update(k_pool=pools[0], v_pool=pools[1], table=table, cu_q=ends.int(),
                 kv_len=torch.tensor(kv_len, device=dev, dtype=torch.int32), max_q=max(q_len), max_kv=max(kv_len))
        if case["op"] == "append":
            qkv = _heads(g, (t, h + 2 * hk, d), dev)
            s.update(q=qkv[:, :h], k=qkv[:, h:h + hk], v=qkv[:, h + hk:],
                     q_out=torch.empty(t, h, d, dtype=torch.bfloat16, device=dev),
                     rope=_rope_table(max(kv_len), case["rot"], dev))
        else:
            s.update(q=_heads(g, (t, h, d), dev), out=torch.empty(t, h, d, dtype=torch.bfloat16, device=dev),
                     lse=torch.empty(t, h, dtype=torch.float32, device=dev) if case["lse"] else None)
    if case["op"] == "norm_rope" or case.get("norm"):
        s.update(q_norm=(1 + 0.2 * torch.randn(d, generator=g, device=dev)).bfloat16(),
                 k_norm=(1 + 0.2 * torch.randn(d, generator=g, device=dev)).bfloat16())
    if own:  # the cache's handle and the workspace that a serving program keeps
        import fp8_kv_cache_exp_b200 as sz
        s["sz"] = sz
        if case["op"] == "norm_rope":
            s["ws"] = sz.new_ops_workspace(device=dev)
        else:
            s["cache"] = sz.KVCache(s["k_pool"], s["v_pool"], s["table"])
            s["ws"] = sz.new_ops_workspace(s["cache"], device=dev)
    return s


# ------------------------------------------------------------------------------------ one pass

def run(state):
    case = state["case"]
    if own:
        return _own[case["op"]](state, case)
    return _plain[case["op"]](state, case)


def _own_append(s, c):
    s["sz"].sz_kv_append_paged(s["cache"], s["k"], s["v"], s["cu_q"], s["kv_len"], s["ws"], q=s["q"], q_out=s["q_out"],
                               q_norm=s.get("q_norm"), k_norm=s.get("k_norm"), eps=EPS, rope=s["rope"],
                               interleaved=c["interleaved"])
    return s["q_out"], s["k_pool"], s["v_pool"]


def _own_norm_rope(s, c):
    s["sz"].sz_qk_norm_rope(s["q"], s["k"], s["q_out"], s["k_out"], s["ws"], q_norm=s["q_norm"], k_norm=s["k_norm"],
                            eps=EPS, rope=s["rope"], positions=s["positions"], interleaved=c["interleaved"])
    return s["q_out"], s["k_out"]


def _own_attn(s, c):
    s["sz"].sz_attn_paged(s["cache"], s["q"], s["cu_q"], s["kv_len"], s["out"], s["ws"], causal=True,
                          window=c["window"], lse=s["lse"])
    return s["out"], s["lse"]


_own = {"append": _own_append, "norm_rope": _own_norm_rope, "attn": _own_attn}


# ------------------------------------------------------------------------------------ plain forms

def _norm(x, w):
    return x if w is None else x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * w.float()


def _rotate(x, rows, interleaved):
    """x [t, h, d] float32, rows [t, rot]: cosines, then sines."""
    r = rows.shape[1]
    cos, sin = rows[:, None, : r // 2], rows[:, None, r // 2:]
    a, b = (x[..., 0:r:2], x[..., 1:r:2]) if interleaved else (x[..., : r // 2], x[..., r // 2: r])
    a, b = a * cos - b * sin, b * cos + a * sin
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., r:]], -1)


def _places(s):
    """Sequence and position of every new token."""
    t = torch.arange(s["q"].shape[0], device=s["q"].device)
    seq = torch.searchsorted(s["cu_q"], t, right=True) - 1
    return seq, (t - s["cu_q"][seq + 1] + s["kv_len"][seq]).long()


def _plain_append(s, c):
    seq, pos = _places(s)
    rows = s["rope"][pos]
    s["q_out"].copy_(_rotate(_norm(s["q"].float(), s.get("q_norm")), rows, c["interleaved"]))
    page, at = s["table"][seq, pos // c["page"]].long(), pos % c["page"]
    kind = s["k_pool"].dtype
    s["k_pool"][page, at] = _rotate(_norm(s["k"].float(), s.get("k_norm")), rows, c["interleaved"]).to(kind)
    s["v_pool"][page, at] = s["v"].float().to(kind)
    return s["q_out"], s["k_pool"], s["v_pool"]


def _plain_norm_rope(s, c):
    rows = s["rope"][s["positions"].long()]
    s["q_out"].copy_(_rotate(_norm(s["q"].float(), s["q_norm"]), rows, c["interleaved"]))
    s["k_out"].copy_(_rotate(_norm(s["k"].float(), s["k_norm"]), rows, c["interleaved"]))
    return s["q_out"], s["k_out"]


def _plain_attn(s, c):
    h, hk, d, p = c["heads"], c["kv_heads"], c["dim"], c["page"]
    dev, n, nq, nk = s["q"].device, c["seqs"], s["max_q"], s["max_kv"]
    j = torch.arange(nk, device=dev)
    page = s["table"][:, j // p].long()                                          # [n, nk]
    k = s["k_pool"][page, j % p].float().permute(0, 2, 3, 1)                     # [n, hk, d, nk]
    v = s["v_pool"][page, j % p].float().permute(0, 2, 1, 3)                     # [n, hk, nk, d]
    seq, pos = _places(s)
    row = torch.arange(s["q"].shape[0], device=dev) - s["cu_q"][seq]
    q = torch.zeros(n, nq, h, d, device=dev)
    q[seq, row] = s["q"].float()
    q = q.view(n, nq, hk, h // hk, d).permute(0, 2, 3, 1, 4).reshape(n, hk, h // hk * nq, d)
    x = (q @ k).view(n, hk, h // hk, nq, nk) * d ** -0.5
    at = (s["kv_len"] - s["cu_q"].diff())[:, None] + torch.arange(nq, device=dev)  # a row's position
    seen = (j <= at[..., None]) & (j < s["kv_len"][:, None, None])
    if c["window"]:
        seen &= j > at[..., None] - c["window"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    x = torch.exp(x - torch.where(top == -math.inf, 0.0, top))
    total = x.sum(-1, keepdim=True)
    o = x.view(n, hk, h // hk * nq, nk) @ v
    o = (o / total.view(n, hk, -1, 1).clamp_min(1e-37)).view(n, h, nq, d).permute(0, 2, 1, 3)
    s["out"].copy_(o[seq, row])
    if s["lse"] is not None:
        s["lse"].copy_((top + total.log()).view(n, h, nq).permute(0, 2, 1)[seq, row])
    return s["out"], s["lse"]


_plain = {"append": _plain_append, "norm_rope": _plain_norm_rope, "attn": _plain_attn}


# ------------------------------------------------------------------------------------ work and exact values

def work(case):
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    if case["op"] == "norm_rope":
        t = case["tokens"]
        return {"bytes": t * (4 * (h + hk) * d + 4 + 4 * case["rot"]) + 4 * d,
                "flops": t * (h + hk) * (4 * d + 3 * case["rot"])}
    eb = 1 if case["e5m2"] else 2
    q_len, kv_len = _lengths(case)
    t = sum(q_len)
    if case["op"] == "append":
        return {"bytes": t * (4 * h * d + 2 * hk * d * (2 + eb) + 4 * case["rot"]),
                "flops": t * (h + hk) * (3 * case["rot"] + (4 * d if case["norm"] else 0))}
    w = case["window"] or 1 << 60
    read = sum(min(n, m + w - 1) for m, n in zip(q_len, kv_len))
    pairs = sum(min(n - m + i + 1, w) for m, n in zip(q_len, kv_len) for i in range(m))
    return {"bytes": 2 * read * hk * d * eb + t * h * (4 * d + (4 if case["lse"] else 0)), "flops": 4 * pairs * h * d}


def _turn64(x, w, rows, interleaved):
    """The norm and the rotation as a product of complex numbers, in 64 bits."""
    x = x.double()
    if w is not None:
        x = x * w.double() / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + EPS).sqrt()
    r = rows.shape[-1]
    unit = torch.complex(*rows.double().chunk(2, -1)).unsqueeze(1)
    out = x.clone()
    if interleaved:
        z = torch.view_as_complex(x[..., :r].reshape(*x.shape[:-1], r // 2, 2)) * unit
        out[..., :r] = torch.view_as_real(z).reshape(*x.shape[:-1], r)
    else:
        z = torch.complex(x[..., : r // 2].contiguous(), x[..., r // 2: r].contiguous()) * unit
        out[..., : r // 2], out[..., r // 2: r] = z.real, z.imag
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm_rope":
        rows = s["rope"][s["positions"].long()]
        return (_turn64(s["q"], s["q_norm"], rows, case["interleaved"]),
                _turn64(s["k"], s["k_norm"], rows, case["interleaved"]))
    q_len, kv_len = _lengths(case)
    p, starts = case["page"], [sum(q_len[:b]) for b in range(len(q_len))]
    if case["op"] == "append":
        pos = torch.cat([torch.arange(n - m, n, device=s["q"].device) for m, n in zip(q_len, kv_len)])
        rows = s["rope"][pos]
        q = _turn64(s["q"], s.get("q_norm"), rows, case["interleaved"])
        k = _turn64(s["k"], s.get("k_norm"), rows, case["interleaved"])
        kp, vp = s["k_pool"].double(), s["v_pool"].double()
        e5m2 = lambda x: x.float().to(torch.float8_e5m2).double() if case["e5m2"] else x  # noqa: E731
        for b, (m, n) in enumerate(zip(q_len, kv_len)):
            at = torch.arange(n - m, n, device=kp.device)
            page = s["table"][b].long()[at // p]
            kp[page, at % p] = e5m2(k[starts[b]: starts[b] + m])
            vp[page, at % p] = e5m2(s["v"][starts[b]: starts[b] + m].double())
        # behind a norm the last bits of a 32-bit sum decide on which side of an 8-bit value's border a key falls
        return q, None if case["e5m2"] and case["norm"] else kp, vp
    h, hk, d = case["heads"], case["kv_heads"], case["dim"]
    outs, lses = [], []
    for b, (m, n) in enumerate(zip(q_len, kv_len)):
        page = s["table"][b, : -(-n // p)].long()
        k, v = (x[page].flatten(0, 1)[:n].double().transpose(0, 1) for x in (s["k_pool"], s["v_pool"]))
        q = s["q"][starts[b]: starts[b] + m].double().transpose(0, 1)
        far = torch.arange(n - m, n, device=q.device)[:, None] - torch.arange(n, device=q.device)[None]
        bad = (far < 0) | (far >= (case["window"] or 1 << 60))
        o = torch.empty(m, h, d, dtype=torch.float64, device=q.device)
        lse = torch.empty(m, h, dtype=torch.float64, device=q.device)
        for i in range(h):
            x = (q[i] @ k[i // (h // hk)].T / math.sqrt(d)).masked_fill_(bad, -math.inf)
            lse[:, i] = torch.logsumexp(x, -1)
            o[:, i] = torch.exp(x - lse[:, i, None]) @ v[i // (h // hk)]
        outs.append(o)
        lses.append(lse)
    return torch.cat(outs), torch.cat(lses) if case["lse"] else None
