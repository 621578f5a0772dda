"""Batches for the full attention tests that give its thread blocks work of
every kind, what the schedule makes of them, and the definition in 64 bits on
the GPU (test_gpu_full_attn.py has it on the host, for small problems)."""
import math
import os
import re

import torch

from tests.test_gpu_full_attn import make

SMS = 152
_SOURCE = os.path.join(os.path.dirname(__file__), "..", "top_sparse_attention_chunked_gb300", "csrc", "full_attn.cu")


def constants():
    """The schedule's constants, from the source."""
    with open(_SOURCE) as f:
        text = f.read()
    names = ("kTileKeys", "kSlotRows", "kMaxCtas", "kCostRows", "kCostKeys", "kCostItem", "kCostEmpty")
    return {n: int(re.search(rf"\b{n} = (\d+)", text).group(1)) for n in names}


def items(q_len, total_len, hq, hkv, first_key=None, window=0):
    """(rows, key tiles) of every item, in order."""
    k, out, grp = constants(), [], hq // hkv
    for b, (n, t) in enumerate(zip(q_len, total_len)):
        for _ in range(hkv):
            for row0 in range(0, n * grp, 2 * k["kSlotRows"]):
                rows = min(2 * k["kSlotRows"], n * grp - row0)
                hi = t - n + (row0 + rows - 1) // grp + 1
                lo = first_key[b] if first_key else 0
                if window:
                    lo = max(lo, t - n + row0 // grp - window + 1)
                lo = min(lo, hi)
                out.append((rows, -(-hi // k["kTileKeys"]) - lo // k["kTileKeys"] if lo < hi else 0))
    return out


def segments(*args, **kw):
    """What each thread block works on: lists of (rows, tiles, whole item)."""
    k, its = constants(), items(*args, **kw)
    unit = lambda rows: k["kCostRows"] if rows > k["kSlotRows"] else k["kCostKeys"]
    base = lambda n: k["kCostItem"] if n else k["kCostEmpty"]
    cost = sum(base(n) + n * unit(rows) for rows, n in its)
    units = sum(max(n, 1) for _, n in its)
    want = min(SMS, k["kMaxCtas"], units)
    runs = []
    if units <= want:
        runs = [(i, t) for i, (_, n) in enumerate(its) for t in range(max(n, 1))]
    else:
        at, c = 0, 0
        for i, (rows, n) in enumerate(its):
            end = at + base(n) + n * unit(rows)
            while c < want and cost * c < end * want:
                t = max(0, cost * c // want - at - base(n)) // unit(rows)
                c += 1
                if not runs or runs[-1] < (i, t):
                    runs.append((i, t))
            at = end
    out = []
    for (i, t), (end_i, end_t) in zip(runs, runs[1:] + [(len(its), 0)]):
        block = []
        while (i, t) < (end_i, end_t):
            stop = end_t if i == end_i else its[i][1]
            block.append((its[i][0], stop - t, t == 0 and stop == its[i][1]))
            i, t = i + 1, 0
        out.append(block)
    return out


def changes(blocks):
    """How often a block goes from a segment of up to kSlotRows rows ("keys") to a wider one ("rows"), by
    the first one's number of tiles, and the other way."""
    slot = constants()["kSlotRows"]
    to_rows, to_keys = [], []
    for block in blocks:
        for (r0, n0, _), (r1, n1, _) in zip(block, block[1:]):
            if n0 and n1 and r0 <= slot < r1:
                to_rows.append(n0)
            if n0 and n1 and r1 <= slot < r0:
                to_keys.append(n0)
    return to_rows, to_keys


# single tokens beside a chunk, and chunks whose last item of a head is a narrow one
MIXED = {
    "eight_tokens_and_1000": dict(q_len=[1] * 8 + [1000], total_len=[4000] * 8 + [1000], hq=24, hkv=2),
    "twelve_tokens_and_2048": dict(q_len=[1] * 12 + [2048], total_len=[3000] * 12 + [2048], hq=24, hkv=2),
    "two_chunks": dict(q_len=[700, 650], total_len=[2000, 1500], hq=16, hkv=4),
}

# left-padded prompts: runs of items without a key in one block, before and between items that see some
NO_KEY = {
    "prompt_of_4096": dict(q_len=[4096], total_len=[4096], hq=24, hkv=2, first_key=[4000]),
    "prompt_of_2048_then_chunks": dict(q_len=[2048, 300, 1], total_len=[2048, 700, 500], hq=8, hkv=2, first_key=[1900, 0, 0]),
    # slot 1 has eight rows of 136
    "17_tokens_of_8_heads": dict(q_len=[17] * 30 + [17], total_len=[17] * 30 + [400], hq=16, hkv=2, first_key=[17] * 30 + [0]),
    "5_tokens_then_chunk": dict(q_len=[5] * 40 + [200], total_len=[9] * 40 + [200], hq=16, hkv=2, first_key=[9] * 40 + [0]),
    "64_prompts_of_300": dict(q_len=[300] * 64, total_len=[300] * 64, hq=16, hkv=4, first_key=[299] * 20 + [300] * 40 + [0] * 4),
    # more tiles than blocks: the items are laid out by cost
    "padded_batch": dict(q_len=[1500] * 4, total_len=[1500] * 4, hq=16, hkv=4, first_key=[1200, 0, 1499, 700]),
}

# several tiles a segment and several segments a block, items of up to 128 rows, wider ones, and both in turn
LOOPS = {
    "single_tokens": dict(q_len=[1] * 6, total_len=[9000, 12001, 7777, 128, 10240, 9985], hq=8, hkv=4),
    "eight_tokens": dict(q_len=[8, 7, 8], total_len=[13000, 12800, 12929], hq=24, hkv=2),
    "chunk_of_300": dict(q_len=[300], total_len=[6000], hq=24, hkv=2),
    "unequal_chunks": dict(q_len=[129, 1, 64, 300, 2, 0, 520], total_len=[3000, 8000, 1000, 2500, 5001, 9, 2049], hq=12, hkv=4),
    "chunk_of_2000": dict(q_len=[2000], total_len=[2000], hq=16, hkv=2),
    "many_short": dict(q_len=[(1, 30, 50, 5, 64)[i % 5] for i in range(48)], total_len=[300 + 31 * i for i in range(48)], hq=16,
                       hkv=4),
}

# narrow items of one tile, which only one slot works on, before wider ones
ONE_TILE = {
    "token_then_300": dict(q_len=[1, 300] * 20, total_len=[100, 900] * 20, hq=24, hkv=2),
    "small_and_wide": dict(q_len=[3, 200, 1, 130] * 16, total_len=[90, 700, 128, 400] * 16, hq=8, hkv=4),
}

TYPES = [("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"), ("fp16", "int8")]


def grow(c, top):
    """Keys whose logits grow along the cache, to about `top`: the running maximum is raised all along."""
    ramp = torch.linspace(0, 1, c["cap"])[None, :, None]
    seen = torch.stack([(torch.arange(c["cap"]) < t) for t in c["total_len"]])[..., None]
    per_unit = 128 * 1.2 / math.sqrt(128)        # a logit, of keys of 1 and queries of mean 1.2
    if c["k_scale"] is not None:
        c["k"] = torch.where(c["k"] == 127, c["k"], c["k"].abs().clamp(1, 90))
        scale = (1e-4 + ramp * top / per_unit / 45).expand(c["k_scale"].shape)
        c["k_scale"] = torch.where(seen, scale, c["k_scale"]).contiguous()
    else:
        k = torch.sign(c["k"].float()) * 0.02 + (ramp * top / per_unit)[..., None]
        c["k"] = torch.where(seen[..., None], k, c["k"].float()).to(c["k"].dtype)
    c["q"] = c["q"].abs()
    return c


def batch(name_or_case, q, kv, **kw):
    case = dict(MIXED[name_or_case] if isinstance(name_or_case, str) else name_or_case)
    case.update(kw)
    return make(case.pop("q_len"), case.pop("total_len"), case.pop("hq"), case.pop("hkv"), q, kv, **case)


def reference(c, window=0, softcap=0.0, slopes=None, scale=None):
    """(out, lse, magnitude, logits' error) in 64 bits as test_gpu_full_attn.check takes them."""
    scale = scale or 1 / math.sqrt(128)
    grp, dev = c["hq"] // c["hkv"], "cuda"
    n_all = sum(c["q_len"])
    f64 = dict(dtype=torch.float64, device=dev)
    out, mag = torch.zeros(n_all, c["hq"], 128, **f64), torch.zeros(n_all, c["hq"], 128, **f64)
    lse, dz = torch.full((n_all, c["hq"]), -math.inf, **f64), torch.zeros(n_all, c["hq"], **f64)
    # (an FP16 weight below its normal numbers: see the host's reference)
    tiny = 2.0 ** -21 if c["kvdt"] == "fp16" else 0.0
    n0 = 0
    for b, (n, t) in enumerate(zip(c["q_len"], c["total_len"])):
        f = c["first_key"][b]
        for g in range(c["hkv"] if n and f < t else 0):
            k, v = (c[x][b, f:t, g].to(dev).double() for x in ("k", "v"))
            if c["k_scale"] is not None:
                k = k * c["k_scale"][b, f:t, g].to(dev).double()[:, None]
                v = v * c["v_scale"][b, f:t, g].to(dev).double()[:, None]
            key = torch.arange(f, t, device=dev)
            for i0 in range(0, n, 512):
                i1 = min(n, i0 + 512)
                heads = slice(g * grp, (g + 1) * grp)
                q = c["q"][n0 + i0:n0 + i1, heads].to(dev).double()
                pos = torch.arange(t - n + i0, t - n + i1, device=dev)[:, None, None]
                z = q @ k.T * scale                                              # [tokens, G, keys]
                err = (q.abs() @ k.abs().T) * (scale * 130 * 2.0 ** -24) + z.abs() * 2.0 ** -21
                if softcap:
                    z = softcap * torch.tanh(z / softcap)
                    err += z.abs() * 2.0 ** -20      # relative: a cap much wider than the logits costs nothing
                if slopes is not None:
                    d = slopes.to(dev).double()[heads][None, :, None] * (key - pos)
                    z = z + d
                    err += d.abs() * 2.0 ** -22
                seen = key <= pos
                if window:
                    seen &= key > pos - window
                m = z.masked_fill(~seen, -math.inf).amax(-1, keepdim=True)
                some = m > -math.inf
                m = torch.where(some, m, torch.zeros_like(m))
                zmax = z.abs().masked_fill(~seen, 0).amax(-1, keepdim=True)
                err += (zmax + (z - m).abs()) * 2.0 ** -22
                p = torch.where(seen, torch.exp(z - m), torch.zeros_like(z))
                total = p.sum(-1, keepdim=True)
                p = p / torch.where(some, total, torch.ones_like(total))
                rows = slice(n0 + i0, n0 + i1)
                out[rows, heads] = p @ v
                mag[rows, heads] = (p + tiny * seen) @ v.abs()
                lse[rows, heads] = (m + torch.log(total))[..., 0]
                dz[rows, heads] = (p * err).sum(-1) + err.masked_fill(p <= 1e-9, 0).amax(-1)
        n0 += n
    return tuple(x.cpu().numpy() for x in (out, lse, mag, dz))
