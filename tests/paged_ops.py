"""Plain forms, in 64 bits, of the operators on a paged cache, and the caches that their tests use.

The bounds that come with them count roundings: half a step of a type is 2^-8 of
the value for bf16, 2^-11 for fp16, 2^-3 for E5M2 (2^-17 below its normal range);
a sum of up to a few hundred products in 32 bits, the rotation's and the norm's
few steps, and the approximate exp2 (2^-22 of the value) stay within 2^-18 of the
sum of magnitudes that they run over.
"""
import math
from dataclasses import dataclass

import torch

POISON = float("nan")


@dataclass
class Paged:
    k_pool: torch.Tensor
    v_pool: torch.Tensor
    table: torch.Tensor
    k: list       # per sequence [kv_len, kv_heads, dim], as the pools hold them
    v: list


def build_cache(gen, dtype, kv_lens, page, kv_heads, dim, gap=0, spare=2, room=0, device="cuda", scale=1.0):
    """Sequences scattered over a pool in random page order; every place that holds no token is NaN.
    gap: elements between pages; room: places kept free behind each sequence."""
    counts = [max(1, -(-(n + room) // page)) for n in kv_lens]
    pages = sum(counts) + spare
    order = torch.randperm(pages, generator=gen)
    width = max(counts)
    table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
    run = page * kv_heads * dim
    pools, data = [], []
    for _ in range(2):
        flat = torch.full((pages, run + gap), POISON, dtype=torch.float32).to(dtype)
        pools.append(flat)
        data.append([])
    at = 0
    for b, n in enumerate(kv_lens):
        ids = order[at: at + counts[b]]
        at += counts[b]
        table[b, : counts[b]] = ids.int()
        for pool, out in zip(pools, data):
            x = (torch.randn(n, kv_heads, dim, generator=gen) * scale).to(dtype)
            out.append(x)
            raw = x.view(torch.uint8).reshape(-1) if n else torch.empty(0, dtype=torch.uint8)
            es = x.element_size()
            for j in range(counts[b]):
                piece = raw[j * run * es: (j + 1) * run * es]
                pool[ids[j]].view(torch.uint8)[: piece.numel()] = piece
    views = [p.to(device)[:, :run].unflatten(1, (page, kv_heads, dim)) for p in pools]
    return Paged(views[0], views[1], table.to(device), data[0], data[1])


def lengths(q_lens, kv_lens, device="cuda"):
    cu = torch.tensor([0] + list(q_lens), dtype=torch.int32).cumsum(0).int()
    return cu.to(device), torch.tensor(kv_lens, dtype=torch.int32).to(device)


def attention(q, k, v, causal=True, window=0, scale=None):
    """One sequence: q [m, heads, dim], k, v [n, kv_heads, dim] -> (out, lse, magnitude, reach), 64 bits.
    magnitude: what each output's terms sum to in absolute value; reach: the largest sum of absolute
    products in a row's scores."""
    q, k, v = q.double(), k.double(), v.double()
    m, heads, dim = q.shape
    n, kv_heads = k.shape[0], k.shape[1]
    scale = dim ** -0.5 if scale is None else scale
    if n == 0:
        z = torch.zeros(m, heads, dim, dtype=torch.float64)
        return z, torch.full((m, heads), -math.inf, dtype=torch.float64), z, torch.zeros(m, heads, dtype=torch.float64)
    k = k.repeat_interleave(heads // kv_heads, 1)
    v = v.repeat_interleave(heads // kv_heads, 1)
    x = torch.einsum("mhd,nhd->mhn", q, k) * scale
    reach = torch.einsum("mhd,nhd->mhn", q.abs(), k.abs()) * scale
    place = torch.arange(n - m, n)[:, None]
    j = torch.arange(n)[None]
    seen = (j <= place) if causal else torch.ones(m, n, dtype=torch.bool)
    if window:
        seen = seen & (j > place - window)
    seen = seen[:, None].expand(m, heads, n)
    x = torch.where(seen, x, -math.inf)
    reach = torch.where(seen, reach, 0.0).nan_to_num(0).amax(-1)
    lse = torch.logsumexp(x, -1)
    p = torch.where(seen, torch.exp(x - torch.where(torch.isfinite(lse), lse, 0.0)[..., None]), 0.0)
    vv = torch.where(torch.isfinite(v), v, 0.0)
    out = torch.einsum("mhn,nhd->mhd", p, vv)
    mag = torch.einsum("mhn,nhd->mhd", p, vv.abs())
    bad = ~torch.isfinite(v)
    if bad.any():  # an unseen place has no say, whatever it holds
        hit = torch.einsum("mhn,nhd->mhd", seen.double(), bad.double()) > 0
        out = torch.where(hit, math.nan, out)
    return out, lse, mag, reach


def attention_bound(out, mag, reach, e5m2):
    """How far a bf16 output may be off: its own rounding; the weights', each off by half a step of the
    type that they are multiplied in; and the 32-bit sums, in the scores (then in the exponent) and in
    the output."""
    weights = 2.0 ** -11 if e5m2 else 2.0 ** -8
    return 2.0 ** -8 * out.abs() + (weights + 2.0 ** -16 + 2.0 ** -18 * reach[..., None]) * mag + 1e-30


def norm(x, w, eps):
    x = x.double()
    return x if w is None else x * w.double() / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def rotate(x, table, pos, interleaved):
    """x [t, heads, dim] (64 bits), table [positions, rot], pos [t]."""
    if table is None:
        return x
    rot = table.shape[1]
    rows = table.double()[pos]
    cos, sin = rows[:, None, : rot // 2], rows[:, None, rot // 2:]
    out = x.clone()
    if interleaved:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        out[..., 0:rot:2], out[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., : rot // 2], x[..., rot // 2: rot]
        out[..., : rot // 2], out[..., rot // 2: rot] = a * cos - b * sin, b * cos + a * sin
    return out


def rope_bound(ref, x, dtype):
    """Half a step of the output's type, and the 32-bit steps over the head's largest magnitude."""
    step = {torch.bfloat16: 2.0 ** -8, torch.float8_e5m2: 2.0 ** -3}[dtype]
    tiny = {torch.bfloat16: 2.0 ** -134, torch.float8_e5m2: 2.0 ** -17}[dtype]
    return step * ref.abs() + 2.0 ** -18 * x.abs().amax(-1, keepdim=True) + tiny
