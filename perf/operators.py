"""Serving operators around a paged cache: what they compute, on which sizes.

Three operators, each in a plain form (elementary torch operations) and as the
library's call:

* ``attn``  full GQA attention of every sequence's new tokens (one or many)
  over a paged K/V cache, causal, optionally with a sliding window, scores
  capped by a tanh and a bias that is linear in the distance;
* ``update`` / ``compact``  the pages themselves: fork, reorder, free and grow
  sequences of a block table (a shared page that is about to be written is
  copied first), and move the live pages to the front of the pool;
* ``beam``  beam search's selection over beams x vocabulary.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass, ``exact`` gives the same result from the
definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1}
D = 128          # attention head dim
DI = 64          # index-key dim of a cached token


def _lib():
    from top_sparse_attention_chunked_gb300 import dsa
    return dsa


# --------------------------------------------------------------------- cases
def _attn(name, batch, q_len, dq, total, dt, hq, hkv, q, kv, block=256, window=0, softcap=0.0, slopes=False):
    """Sequence b has max(0, q_len - b * dq) new tokens and max(new, total - b * dt) tokens in all."""
    return dict(name=name, op="attn", batch=batch, q_len=q_len, dq=dq, total=total, dt=dt, hq=hq, hkv=hkv, q=q,
                kv=kv, block=block, window=window, softcap=softcap, slopes=slopes)


def _pages(name, op, groups, beams, length, dlen, grow, layers, hkv, block=256, spare=0.5, mode="beam"):
    """`groups` requests of `beams` sequences; request i has max(1, length - i * dlen) tokens, `grow` are added.
    mode: beam (every request's sequences follow random ones of it), fork (all follow the request's first),
    serve (an eighth of the sequences ends, the others grow)."""
    return dict(name=name, op=op, groups=groups, beams=beams, length=length, dlen=dlen, grow=grow, layers=layers,
                hkv=hkv, block=block, spare=spare, mode=mode)


def _beam(name, batch, beams, vocab, select, dtype, finished=False):
    return dict(name=name, op="beam", batch=batch, beams=beams, vocab=vocab, select=select, dtype=dtype,
                finished=finished)


def listed():
    return [
        # one token of one short conversation: latency alone
        _attn("decode_4k", 1, 1, 0, 4096, 0, 8, 2, "bf16", "bf16"),
        # a serving batch at one token each, lengths from a few keys to 32K
        _attn("decode_16_ragged_32k", 16, 1, 0, 32768, 2184, 24, 2, "bf16", "fp16"),
        # eight speculated tokens each, four sequences of 32K
        _attn("grouped_decode_32k", 4, 8, 0, 32768, 0, 24, 2, "bf16", "fp16"),
        # eight tokens on a 256K INT8 cache
        _attn("decode_256k_int8", 1, 8, 0, 262144, 0, 24, 2, "bf16", "int8"),
        # chunked prefill of unequal chunks beside decoding sequences, with a window and capped scores
        _attn("chunks_window_softcap", 4, 2048, 509, 16500, 3001, 16, 4, "fp16", "fp16", 128, 4096, 30.0),
        # the largest: 8,192 new tokens after 32,768
        _attn("prefill_8k_on_32k", 1, 8192, 0, 40960, 0, 24, 2, "bf16", "bf16"),
        # one step of beam search: eight requests of four beams, about 2,000 tokens each
        _pages("beam_step", "update", 8, 4, 2047, 97, 1, 2, 2),
        # a serving step on 256 sequences of up to 32K: some end, the others grow by a block boundary here and there
        _pages("serve_256_rows", "update", 64, 4, 32700, 509, 8, 1, 1, 256, 0.2, "serve"),
        # defragment the pool of a 256K-token request mix (1,037 blocks and more) after half of it was freed
        _pages("compact_pool", "compact", 32, 2, 16000, 401, 0, 2, 2, 256, 0.6),
        # a single request with four beams
        _beam("beam_4_of_32000", 1, 4, 32000, 8, "fp32"),
        # odd sizes, some beams finished
        _beam("beam_5_of_50001", 8, 5, 50001, 10, "fp16", True),
        # a full batch on a large vocabulary
        _beam("beam_64x8_of_131072", 64, 8, 131072, 16, "bf16"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.choice(["decode", "decode", "chunk", "chunk", "update", "compact", "beam", "beam"])
    if what in ("decode", "chunk"):
        hq, hkv = rng.choice([(8, 2), (24, 2), (16, 4), (8, 8), (32, 8), (12, 1), (40, 2)])
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"), ("fp16", "int8")])
        softcap = rng.choice([0.0, 0.0, 0.0, 30.0, 50.0])
        slopes = rng.random() < 0.2
        block = rng.choice([128, 256, 256, 512])
        if what == "decode":
            batch = _log(rng, 1, 32)
            total = _log(rng, 1, min(262144, 524288 // (batch * hkv)))
            q_len = min(total, rng.choice([1, 1, 1, 2, 4, 8, 16]))
            dt = rng.randint(0, max(0, (total - q_len) // batch))
            window = rng.choice([0, 0, 0, max(1, total // 3)])
            return _attn("", batch, q_len, 0, total, dt, hq, hkv, q, kv, block, window, softcap, slopes)
        batch = rng.choice([1, 1, 2, 3, 4])
        q_len = _log(rng, 17, 8192 // batch)
        total = q_len + rng.choice([0, _log(rng, 1, 32768 // batch)])
        dq = rng.randint(0, q_len // batch)
        dt = rng.randint(0, total // batch)
        window = rng.choice([0, 0, 0, max(1, total // 3)])
        return _attn("", batch, q_len, dq, total, dt, hq, hkv, q, kv, block, window, softcap, slopes)
    if what in ("update", "compact"):
        groups, beams = _log(rng, 1, 64), rng.choice([1, 2, 4, 5])
        length = _log(rng, 1, 65536 // max(4, groups))
        return _pages("", what, groups, beams, length, rng.randint(0, length // groups), rng.choice([0, 1, 1, 8, 300]),
                      rng.choice([1, 2, 3]), rng.choice([1, 2, 4]), rng.choice([128, 256]), rng.uniform(0.1, 1.0),
                      rng.choice(["beam", "fork", "serve"]))
    batch, beams = _log(rng, 1, 32), rng.choice([1, 2, 3, 4, 8, 16])
    vocab = _log(rng, 1000, min(262144, 67108864 // (batch * beams)))
    return _beam("", batch, beams, vocab, rng.choice([beams, 2 * beams]), rng.choice(["bf16", "fp16", "fp32"]),
                 rng.random() < 0.3)


# ----------------------------------------------------------------- attention
def _lens(c):
    q = [max(0, c["q_len"] - b * c["dq"]) for b in range(c["batch"])]
    t = [max(q[b], 1, c["total"] - b * c["dt"]) for b in range(c["batch"])]
    return q, t


def _prepare_attn(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    q_lens, t_lens = _lens(c)
    bs = c["block"]
    used = [-(-t // bs) for t in t_lens]
    per_seq, blocks = max(used), sum(used) + 3
    order = list(range(blocks))
    r.shuffle(order)
    rows, k = [], 0
    for n in used:
        rows.append(order[k:k + n] + [-1] * (per_seq - n))
        k += n
    n_tok = blocks * bs
    s = dict(case=c, q_lens=q_lens, t_lens=t_lens, table=torch.tensor(rows, dtype=torch.int32, device="cuda"),
             blocks=blocks)
    s["q"] = (torch.randn(sum(q_lens), c["hq"], D, device="cuda", generator=g) * 1.5).to(_DT[c["q"]])
    for name in ("k", "v"):
        x = torch.randn(n_tok, c["hkv"], D, device="cuda", generator=g)
        if c["kv"] == "int8":
            scale = x.abs().amax(-1) / 127
            s[name], s[name + "_scale"] = torch.round(x / scale[..., None]).to(torch.int8), scale.contiguous()
        else:
            s[name], s[name + "_scale"] = x.to(_DT[c["kv"]]), None
    s["slopes"] = None
    if c["slopes"]:  # a geometric series over the heads
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda")
    s["T"] = torch.tensor(t_lens, device="cuda")
    s["S"] = torch.tensor(q_lens, device="cuda")
    if own:
        lib = _lib()
        p = lib.make_full_attn_problem(q_lens, t_lens, c["hq"], c["hkv"], cache_capacity=per_seq * bs,
                                       window=c["window"], softcap=c["softcap"], q_dtype=c["q"], kv_dtype=c["kv"])
        s["p"], s["pages"] = p, lib.make_pages(s["table"], bs, blocks)
        s["ws"] = lib.alloc_full_attn_workspace(p)
        s["out"] = torch.empty_like(s["q"])
        s["lse"] = torch.empty(s["q"].shape[:2], dtype=torch.float32, device="cuda")
    return s


def _attn_plain(s):
    c = s["case"]
    bs, hkv, grp, nb = c["block"], c["hkv"], c["hq"] // c["hkv"], c["batch"]
    smax, tmax = max(s["q_lens"]), max(s["t_lens"])
    t = torch.arange(tmax, device="cuda")
    here = t[None] < s["T"][:, None]                                            # [B, T]
    row = s["table"].long()[:, t // bs] * bs + t % bs
    row = torch.where(here, row, torch.zeros_like(row))
    k, v = s["k"][row].float(), s["v"][row].float()                             # [B, T, Hkv, D]
    if s["k_scale"] is not None:
        k, v = k * s["k_scale"][row][..., None], v * s["v_scale"][row][..., None]
    i = torch.arange(smax, device="cuda")
    real = i[None] < s["S"][:, None]                                            # [B, S]
    first = torch.cumsum(s["S"], 0) - s["S"]
    src = torch.where(real, first[:, None] + i, torch.zeros_like(first)[:, None])
    pos = (s["T"] - s["S"])[:, None] + i                                        # [B, S]
    q = s["q"][src].float().view(nb, smax, hkv, grp, D).permute(0, 2, 1, 3, 4).reshape(nb, hkv, smax * grp, D)
    x = torch.matmul(q, k.permute(0, 2, 3, 1)).mul_(1 / math.sqrt(D))           # [B, Hkv, S * G, T]
    if c["softcap"]:
        x = x.div_(c["softcap"]).tanh_().mul_(c["softcap"])
    x = x.view(nb, hkv, smax, grp, tmax)
    dist = t[None, None] - pos[..., None]                                       # [B, S, T]
    if s["slopes"] is not None:
        x += s["slopes"].view(1, hkv, 1, grp, 1) * dist[:, None, :, None]
    seen = (dist <= 0) & here[:, None]
    if c["window"]:
        seen &= dist > -c["window"]
    x.masked_fill_(~seen[:, None, :, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    x = x.sub_(m.masked_fill(m == -math.inf, 0.0)).exp_()
    total = x.sum(-1, keepdim=True)
    o = torch.matmul(x.view(nb, hkv, smax * grp, tmax), v.permute(0, 2, 1, 3)).view(nb, hkv, smax, grp, D)
    o = torch.where(total > 0, o / total, torch.zeros_like(o)).permute(0, 2, 1, 3, 4).reshape(nb, smax, c["hq"], D)
    lse = (m + total.log()).squeeze(-1).permute(0, 2, 1, 3).reshape(nb, smax, c["hq"])
    return [o[real].to(s["q"].dtype), lse[real]]


def _attn_own(s):
    _lib().dsa_full_attn(s["p"], s["q"], s["k"], s["v"], s["k_scale"], s["v_scale"], s["out"], s["ws"],
                         slopes=s["slopes"], lse=s["lse"], pages=s["pages"])
    return [s["out"], s["lse"]]


def _attn_exact(c, seed):
    if _work_attn(c)["flops"] > 8e12:
        return None
    s = _prepare_attn(c, seed)
    grp, bs, n0 = c["hq"] // c["hkv"], c["block"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, t) in enumerate(zip(s["q_lens"], s["t_lens"])):
        blk = s["table"][b, :-(-t // bs)].long()
        kb, vb = (s[x].view(s["blocks"], bs, c["hkv"], D)[blk].view(-1, c["hkv"], D)[:t].double() for x in ("k", "v"))
        if s["k_scale"] is not None:
            kb, vb = (y * s[x].view(s["blocks"], bs, c["hkv"])[blk].view(-1, c["hkv"])[:t].double()[..., None]
                      for x, y in (("k_scale", kb), ("v_scale", vb)))
        for a in range(0, n, 1024):
            e = min(n, a + 1024)
            p = torch.arange(t - n + a, t - n + e, device="cuda")
            lo = max(0, t - n + a - c["window"] + 1) if c["window"] else 0
            hi = t - n + e
            key = torch.arange(lo, hi, device="cuda")
            off = key[None].double() - p[:, None].double()
            ok = off <= 0
            if c["window"]:
                ok &= off > -c["window"]
            for h in range(c["hq"]):
                z = s["q"][n0 + a:n0 + e, h].double() @ kb[lo:hi, h // grp].T / math.sqrt(D)
                if c["softcap"]:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                if s["slopes"] is not None:
                    z = z + s["slopes"][h].double() * off
                z = z.masked_fill(~ok, -math.inf)
                lse[n0 + a:n0 + e, h] = torch.logsumexp(z, 1)
                out[n0 + a:n0 + e, h] = torch.softmax(z, 1) @ vb[lo:hi, h // grp]
        n0 += n
    return [out, lse]


def _work_attn(c):
    q_lens, t_lens = _lens(c)
    pairs = keys = 0
    for n, t in zip(q_lens, t_lens):
        if not n:
            continue
        w = c["window"] or t
        first, last = t - n + 1, t                      # visible keys of the first and the last query, unwindowed
        full = max(0, min(last, w) - first + 1) if first <= w else 0
        pairs += sum((first, first + full - 1)) * full // 2 + (n - full) * min(w, t)
        keys += min(t, n + w - 1)
    n = sum(q_lens)
    per_key = 2 * c["hkv"] * (D * _BYTES[c["kv"]] + (4 if c["kv"] == "int8" else 0))
    return {"bytes": keys * per_key + n * c["hq"] * (2 * D * _BYTES[c["q"]] + 4), "flops": 4 * D * c["hq"] * pairs}


# --------------------------------------------------------------------- pages
def _plan(c, seed):
    """The block table, what its rows shall follow, and how many blocks the pool has."""
    r = random.Random(seed)
    bs, beams = c["block"], c["beams"]
    n_rows = c["groups"] * beams
    lens = [max(1, c["length"] - (i // beams) * c["dlen"]) for i in range(n_rows)]
    rows, nxt = [], 0
    for i, n in enumerate(lens):
        nb, shared = -(-n // bs), (n - 1) // bs     # the request's sequences share all but the block being written
        if i % beams == 0:
            head, nxt = list(range(nxt, nxt + shared)), nxt + shared
        rows.append(head + list(range(nxt, nxt + nb - shared)))
        nxt += nb - shared
    parent = list(range(n_rows))
    if c["mode"] == "beam":
        parent = [i - i % beams + r.randrange(beams) for i in range(n_rows)]
    elif c["mode"] == "fork":
        parent = [i - i % beams for i in range(n_rows)]
    else:
        parent = [-1 if r.random() < 0.125 else i for i in range(n_rows)]
    keep = [lens[p] if p >= 0 else 0 for p in parent]
    new = [k + c["grow"] if p >= 0 else 0 for k, p in zip(keep, parent)]
    need = sum(-(-(n + c["grow"]) // bs) - n // bs for n in lens)      # whoever ends: the pool's size is the case's alone
    blocks = nxt + need + max(1, int(c["spare"] * nxt))
    order = list(range(blocks))
    r.shuffle(order)
    per_seq = -(-(max(lens) + c["grow"]) // bs) + 1
    table = [[order[x] for x in row] + [-1] * (per_seq - len(row)) for row in rows]
    return table, parent, keep, new, blocks


def _prepare_pages(c, seed):
    table, parent, keep, new, blocks = _plan(c, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    bs = c["block"]
    s = dict(case=c, blocks=blocks, table=torch.tensor(table, dtype=torch.int32, device="cuda"))
    flat = s["table"].view(-1).long()
    s["refs"] = torch.bincount(flat[flat >= 0], minlength=blocks).to(torch.int32)
    for name, v in (("parent", parent), ("keep", keep), ("new", new)):
        s[name] = torch.tensor(v, dtype=torch.int32, device="cuda")
    shape = (c["layers"], blocks, bs)
    s["kI"] = torch.randn(*shape, DI, device="cuda", generator=g, dtype=torch.bfloat16)
    s["k"] = torch.randn(*shape, c["hkv"], D, device="cuda", generator=g, dtype=torch.bfloat16)
    s["v"] = torch.randn(*shape, c["hkv"], D, device="cuda", generator=g, dtype=torch.bfloat16)
    if own:
        lib = _lib()
        s["table_out"], s["refs_out"] = torch.empty_like(s["table"]), torch.empty_like(s["refs"])
        s["remap"] = torch.empty_like(s["refs"])
        s["st"] = lib.make_page_state(s["table"], s["refs"], bs)
        s["pools"] = lib.make_page_pools([s[n][i] for i in range(c["layers"]) for n in ("kI", "k", "v")], blocks)
        s["ws"] = lib.alloc_pages_workspace(s["st"])
    return s


def _update_plain(s):
    bs, table, blocks = s["case"]["block"], s["table"].long(), s["blocks"]
    n_rows, per_seq = table.shape
    parent, keep, new = s["parent"].long(), s["keep"].long(), s["new"].long()
    j = torch.arange(per_seq, device="cuda")
    kept_n, new_n = (keep + bs - 1) // bs, (new + bs - 1) // bs
    kept = torch.where(j[None] < kept_n[:, None], table[parent.clamp(min=0)], torch.full_like(table, -1))
    one = torch.ones_like(table)

    def count(t):
        # -1 counts into a bin of its own, behind the others
        idx = torch.where(t >= 0, t, torch.full_like(t, blocks))
        return torch.zeros(blocks + 1, dtype=torch.long, device="cuda").index_add_(0, idx.view(-1), one.view(-1))[:blocks]

    refs = s["refs"].long() - count(table) + count(kept)
    # rows that write into a block they keep, and who else holds it
    r = torch.arange(n_rows, device="cuda")
    tail = kept[r, (kept_n - 1).clamp(min=0)]
    writes = (keep % bs != 0) & (new > keep)
    at = torch.where(writes, tail, torch.full_like(tail, blocks))
    writers = count(torch.where(writes, tail, torch.full_like(tail, -1))[:, None].expand(n_rows, per_seq)) // per_seq
    lowest = torch.full((blocks + 1,), n_rows, device="cuda").scatter_reduce_(0, at, r, "amin")
    safe = tail.clamp(min=0)
    copy = writes & ~((refs[safe] == writers[safe]) & (lowest[safe] == r))
    refs = refs - count(torch.where(copy, tail, torch.full_like(tail, -1))[:, None].expand(n_rows, per_seq)) // per_seq
    # fresh blocks: the free ones in ascending order, to the rows in order
    fresh_from = kept_n - copy.long()
    wants = (j[None] >= fresh_from[:, None]) & (j[None] < new_n[:, None])
    free = (s["refs"].long() - count(table) + count(kept)) == 0
    free_ids = free.nonzero().view(-1)
    rank = torch.cumsum(wants.view(-1).long(), 0).view_as(wants) - 1
    out = torch.where(wants, free_ids[rank.clamp(0, max(0, free_ids.numel() - 1))], kept)
    out = torch.where(j[None] < new_n[:, None], out, torch.full_like(out, -1))
    refs = refs + count(torch.where(wants, out, torch.full_like(out, -1)))
    rows = copy.nonzero().view(-1)
    src, dst = tail[rows], out[rows, fresh_from[rows]]
    for n in ("kI", "k", "v"):
        s[n][:, dst] = s[n][:, src]
    return [out.to(torch.int32), refs.to(torch.int32), s["kI"], s["k"], s["v"]]


def _compact_plain(s):
    live = s["refs"] > 0
    n = live.sum()
    ids = torch.arange(s["blocks"], device="cuda")
    holes, movers = (~live & (ids < n)).nonzero().view(-1), (live & (ids >= n)).nonzero().view(-1)
    remap = torch.where(live, ids, torch.full_like(ids, -1))
    remap[movers] = holes
    table = s["table"].long()
    out = torch.where(table >= 0, remap[table.clamp(min=0)], table)
    refs = torch.zeros_like(s["refs"]).scatter_(0, remap[live], s["refs"][live])
    for x in ("kI", "k", "v"):
        s[x][:, holes] = s[x][:, movers]
    return [out.to(torch.int32), refs, remap.to(torch.int32), s["kI"], s["k"], s["v"]]


def _update_own(s):
    _lib().dsa_pages_update(s["st"], s["parent"], s["keep"], s["new"], s["pools"], s["ws"], table_out=s["table_out"],
                            refs_out=s["refs_out"])
    return [s["table_out"], s["refs_out"], s["kI"], s["k"], s["v"]]


def _compact_own(s):
    _lib().dsa_pages_compact(s["st"], s["pools"], s["ws"], table_out=s["table_out"], refs_out=s["refs_out"],
                             remap=s["remap"])
    return [s["table_out"], s["refs_out"], s["remap"], s["kI"], s["k"], s["v"]]


def _work_pages(c):
    table, parent, keep, new, blocks = _plan(c, 0)
    bs = c["block"]
    block_bytes = c["layers"] * bs * (DI * 2 + 2 * c["hkv"] * D * 2)
    refs = {}
    for row in table:
        for x in row:
            refs[x] = refs.get(x, 0) + (x >= 0)
    if c["op"] == "compact":
        live = sorted(x for x in refs if x >= 0)
        moved, extra = sum(x >= len(live) for x in live), 4 * blocks
    else:
        after, tails = {}, {}
        for p, k, m in zip(parent, keep, new):
            for x in (table[p][:-(-k // bs)] if p >= 0 else []):
                after[x] = after.get(x, 0) + 1
            if k % bs and m > k:
                t = table[p][(k - 1) // bs]
                tails[t] = tails.get(t, 0) + 1
        moved, extra = sum(n - (after[t] == n) for t, n in tails.items()), 12 * len(table)
    return {"bytes": 8 * len(table) * len(table[0]) + 8 * blocks + extra + 2 * moved * block_bytes, "flops": 0}


# ---------------------------------------------------------------------- beam
_EOS = 2         # what a finished beam goes on with


def _prepare_beam(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n = c["batch"] * c["beams"]
    s = dict(case=c, logits=(torch.randn(n, c["vocab"], device="cuda", generator=g) * 2.5).to(_DT[c["dtype"]]))
    s["scores"] = -4.0 * torch.rand(n, device="cuda", generator=g)
    s["finished"] = None
    if c["finished"]:
        s["finished"] = (torch.rand(n, device="cuda", generator=g) < 0.25).to(torch.uint8)
    if own:
        lib = _lib()
        s["p"] = lib.make_beam_problem(c["batch"], c["beams"], c["vocab"], c["select"], c["dtype"], pad_token=_EOS)
        s["ws"] = lib.alloc_beam_workspace(s["p"])
        shape = (c["batch"], c["select"])
        s["out"] = (torch.empty(shape, device="cuda"), torch.empty(shape, dtype=torch.int32, device="cuda"),
                    torch.empty(shape, dtype=torch.int32, device="cuda"))
    return s


def _beam_plain(s):
    c = s["case"]
    x = s["logits"].double()                 # in 64 bits: totals of different beams may lie close together
    m = x.amax(1, keepdim=True)
    lse = (x - m).exp_().sum(1, keepdim=True).log_() + m
    x = x + (s["scores"].double()[:, None] - lse)
    if s["finished"] is not None:
        done = s["finished"].bool()[:, None]
        stay = torch.full_like(x, -math.inf)
        stay[:, _EOS] = s["scores"].double()
        x = torch.where(done, stay, x)
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x).view(c["batch"], -1)
    val, at = torch.sort(x, dim=1, descending=True, stable=True)
    val, at = val[:, :c["select"]], at[:, :c["select"]]
    none = val == -math.inf
    row = at // c["vocab"] + torch.arange(c["batch"], device="cuda")[:, None] * c["beams"]
    return [val.float(), torch.where(none, -1, at % c["vocab"]).to(torch.int32), torch.where(none, -1, row).to(torch.int32)]


def _beam_own(s):
    _lib().dsa_beam_select(s["p"], s["logits"], s["scores"], *s["out"], s["ws"], finished=s["finished"])
    return list(s["out"])


def _beam_exact(c, seed):
    s = _prepare_beam(c, seed)
    lp = torch.log_softmax(s["logits"].double(), 1) + s["scores"].double()[:, None]
    if s["finished"] is not None:
        for i in s["finished"].nonzero().view(-1).tolist():
            lp[i] = -math.inf
            lp[i, _EOS] = s["scores"][i].double()
    return [lp.view(c["batch"], -1).topk(c["select"], 1).values, None, None]


def _work_beam(c):
    n = c["batch"] * c["beams"] * c["vocab"]
    return {"bytes": n * _BYTES[c["dtype"]] + c["batch"] * (5 * c["beams"] + 12 * c["select"]), "flops": 3 * n}


# ----------------------------------------------------------------- interface
def prepare(case, seed):
    make = {"attn": _prepare_attn, "update": _prepare_pages, "compact": _prepare_pages, "beam": _prepare_beam}
    return make[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _attn_own, "update": _update_own, "compact": _compact_own, "beam": _beam_own}[op](state)
    return {"attn": _attn_plain, "update": _update_plain, "compact": _compact_plain, "beam": _beam_plain}[op](state)


def exact(case, seed):
    if case["op"] == "attn":
        return _attn_exact(case, seed)
    if case["op"] == "beam":
        return _beam_exact(case, seed)
    return None      # whole numbers and copied blocks


def work(case):
    return {"attn": _work_attn, "update": _work_pages, "compact": _work_pages, "beam": _work_beam}[case["op"]](case)
