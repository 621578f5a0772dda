"""Operators of a serving step on packed, ragged batches with rolling caches:
what they compute, on which sizes.

Five operators, each in a plain form (elementary torch operations) and as the
library's call:

* ``attn``    full GQA attention over a paged K/V cache with a sliding window
  beside which every sequence's first tokens stay visible;
* ``norm``    a residual's addition, RMS norm, and an output in 16 bits or in
  e4m3 with a scale per row or per 128 values;
* ``rope``    RMS norm and rotary positions with several axes (time, height,
  width) for packed queries and keys, and keys and values into the cache rows
  that a slot map names;
* ``slots``   that slot map, from request lengths and a block table;
* ``sample``  temperature, top-k, top-p, min-p and a draw from one given
  random number per row.

A case is a dict of plain values; ``prepare`` makes its inputs on the GPU from
a seed, ``run`` makes one pass, ``exact`` gives the same result from the
definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "int8": torch.int8,
       "e4m3": torch.float8_e4m3fn}
_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "int8": 1, "e4m3": 1}
D = 128          # attention head dim


def _lib():
    from top_sparse_attention_chunked_gb300 import dsa
    return dsa


# --------------------------------------------------------------------- cases
def _attn(name, batch, q_len, dq, total, dt, hq, hkv, q, kv, block, window, sinks, softcap=0.0, slopes=False, pad=0):
    """Sequence b has max(0, q_len - b * dq) new tokens, max(new, total - b * dt) tokens in all, and begins at key b * pad."""
    return dict(name=name, op="attn", batch=batch, q_len=q_len, dq=dq, total=total, dt=dt, hq=hq, hkv=hkv, q=q, kv=kv,
                block=block, window=window, sinks=sinks, softcap=softcap, slopes=slopes, pad=pad)


def _norm(name, rows, hidden, x, out, group=0, add=True):
    """group: values of a row that share a scale (0: all of them)."""
    return dict(name=name, op="norm", rows=rows, hidden=hidden, x=x, out=out, group=group, add=add)


def _rope(name, tokens, hq, hkv, rot, sections, mode, q, kv, norm=True, padded=0):
    """sections: rotary pairs of each axis, "16,24,24"; mode: whole (an axis's pairs lie together) or turns (dealt out in turn)."""
    return dict(name=name, op="rope", tokens=tokens, hq=hq, hkv=hkv, rot=rot, sections=sections, mode=mode, q=q, kv=kv,
                norm=norm, padded=padded)


def _slots(name, rows, q_len, total, block, spare):
    """rows requests with up to q_len new tokens on up to `total`; `spare` entries of the packed step stay unused."""
    return dict(name=name, op="slots", rows=rows, q_len=q_len, total=total, block=block, spare=spare)


def _sample(name, rows, vocab, dtype, mode):
    """mode: what the rows ask for: heat (a temperature), topk, topp, minp, or mixed (each row its own)."""
    return dict(name=name, op="sample", rows=rows, vocab=vocab, dtype=dtype, mode=mode)


def listed():
    return [
        # a serving batch at one token each, long conversations behind a window of 4,096 and four first tokens
        _attn("sinks_decode_16_ragged", 16, 1, 0, 32768, 2000, 24, 2, "bf16", "fp16", 256, 4096, 4),
        # two prompts in chunks, the first block stays
        _attn("sinks_chunks", 2, 4096, 701, 20480, 3001, 16, 4, "fp16", "fp16", 128, 2048, 64),
        # eight tokens on a 256K INT8 cache that see a system prompt of 1,000 tokens and the last 32K
        _attn("sinks_256k_int8", 1, 8, 0, 262144, 0, 24, 2, "bf16", "int8", 256, 32768, 1000),
        # between two layers of a decoding batch: latency alone
        _norm("norm_8x5120", 8, 5120, "bf16", "bf16"),
        # between two layers of a prefill chunk, for a product in 8 bits
        _norm("norm_8192x8192_e4m3", 8192, 8192, "bf16", "e4m3", 128),
        # a decoding batch of 16 text tokens
        _rope("rope_16_tokens", 16, 24, 2, 128, "16,24,24", "whole", "bf16", "fp16"),
        # a prompt of images: 8,192 tokens, 160 of them padding
        _rope("rope_8192_tokens", 8192, 32, 8, 128, "24,20,20", "turns", "bf16", "bf16", True, 160),
        # 64 decoding requests
        _slots("slots_64_rows", 64, 1, 32768, 256, 0),
        # a packed step of 500 requests, prompts beside decodes
        _slots("slots_500_rows", 500, 2048, 30000, 128, 1000),
        # one conversation
        _sample("sample_1_of_32000", 1, 32000, "fp32", "topk"),
        # odd sizes, nucleus sampling
        _sample("sample_37_of_50257", 37, 50257, "fp16", "topp"),
        # a full batch on a large vocabulary, every request with its own settings
        _sample("sample_64_of_131072", 64, 131072, "bf16", "mixed"),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    what = rng.choice(["attn", "attn", "norm", "norm", "rope", "rope", "slots", "sample", "sample"])
    if what == "attn":
        hq, hkv = rng.choice([(8, 2), (24, 2), (16, 4), (8, 8), (32, 8), (12, 1), (40, 2)])
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8"), ("fp16", "int8")])
        block = rng.choice([128, 256, 256, 512])
        sinks = rng.choice([1, 4, 4, 16, 100, 128, 500])
        softcap, slopes = rng.choice([0.0, 0.0, 0.0, 30.0]), rng.random() < 0.15
        if rng.random() < 0.5:
            batch = _log(rng, 1, 32)
            total = _log(rng, 1, min(262144, 524288 // (batch * hkv)))
            q_len = min(total, rng.choice([1, 1, 1, 2, 4, 8, 16]))
            dt, dq = rng.randint(0, max(0, (total - q_len) // batch)), 0
        else:
            batch = rng.choice([1, 1, 2, 3, 4])
            q_len = _log(rng, 17, 4096 // batch)
            total = q_len + rng.choice([0, _log(rng, 1, 16384 // batch)])
            dq, dt = rng.randint(0, q_len // batch), rng.randint(0, total // batch)
        window = _log(rng, 1, max(1, total))
        return _attn("", batch, q_len, dq, total, dt, hq, hkv, q, kv, block, window, sinks, softcap, slopes,
                     rng.choice([0, 0, rng.randint(0, max(0, total // batch))]))
    if what == "norm":
        rows, hidden = _log(rng, 1, 8192), _log(rng, 64, 8192)
        hidden = rng.choice([hidden, (hidden + 7) // 8 * 8, (hidden + 127) // 128 * 128])
        return _norm("", rows, min(hidden, 8192), rng.choice(["bf16", "fp16", "bf16", "fp32"]),
                     rng.choice(["bf16", "fp16", "e4m3", "e4m3"]), rng.choice([0, 128]), rng.random() < 0.8)
    if what == "rope":
        hq, hkv = rng.choice([(8, 2), (24, 2), (16, 4), (8, 8), (32, 8), (12, 1)])
        q, kv = rng.choice([("bf16", "bf16"), ("bf16", "fp16"), ("fp16", "fp16"), ("bf16", "int8")])
        rot, sections = rng.choice([(128, "16,24,24"), (128, "24,20,20"), (128, "32,32"), (128, "64"), (64, "8,12,12"),
                                    (96, "16,16,16"), (128, "16,16,16,16")])
        tokens = _log(rng, 1, 8192)
        return _rope("", tokens, hq, hkv, rot, sections, rng.choice(["whole", "turns"]), q, kv, rng.random() < 0.7,
                     rng.choice([0, rng.randint(0, tokens)]))
    if what == "slots":
        return _slots("", _log(rng, 1, 500), _log(rng, 1, 2048), _log(rng, 2048, 30000), rng.choice([128, 256]),
                      rng.choice([0, 0, rng.randint(1, 1000)]))
    rows = _log(rng, 1, 64)
    return _sample("", rows, _log(rng, 1000, min(262144, 8388608 // rows)), rng.choice(["bf16", "fp16", "fp32"]),
                   rng.choice(["heat", "topk", "topp", "minp", "mixed"]))


# ----------------------------------------------------------------- attention
def _lens(c):
    q = [max(0, c["q_len"] - b * c["dq"]) for b in range(c["batch"])]
    t = [max(q[b], 1, c["total"] - b * c["dt"]) for b in range(c["batch"])]
    return q, t, [min(t[b], b * c["pad"]) for b in range(c["batch"])]


def _prepare_attn(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    q_lens, t_lens, first = _lens(c)
    bs = c["block"]
    used = [-(-t // bs) for t in t_lens]
    per_seq, blocks = max(used), sum(used) + 3
    order = list(range(blocks))
    r.shuffle(order)
    rows, k = [], 0
    for n in used:
        rows.append(order[k:k + n] + [-1] * (per_seq - n))
        k += n
    s = dict(case=c, q_lens=q_lens, t_lens=t_lens, firsts=first, blocks=blocks,
             table=torch.tensor(rows, dtype=torch.int32, device="cuda"))
    s["q"] = (torch.randn(sum(q_lens), c["hq"], D, device="cuda", generator=g) * 1.5).to(_DT[c["q"]])
    for name in ("k", "v"):
        x = torch.randn(blocks * bs, c["hkv"], D, device="cuda", generator=g)
        if c["kv"] == "int8":
            scale = x.abs().amax(-1) / 127
            s[name], s[name + "_scale"] = torch.round(x / scale[..., None]).to(torch.int8), scale.contiguous()
        else:
            s[name], s[name + "_scale"] = x.to(_DT[c["kv"]]), None
    s["slopes"] = None
    if c["slopes"]:  # a geometric series over the heads
        s["slopes"] = torch.tensor([2.0 ** (-8.0 * (h + 1) / c["hq"]) for h in range(c["hq"])], device="cuda")
    for name, v in (("T", t_lens), ("S", q_lens), ("F", first)):
        s[name] = torch.tensor(v, device="cuda")
    if own:
        lib = _lib()
        p = lib.make_full_attn_problem(q_lens, t_lens, c["hq"], c["hkv"], cache_capacity=per_seq * bs,
                                       window=c["window"], softcap=c["softcap"], first_key=first, q_dtype=c["q"],
                                       kv_dtype=c["kv"])
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
    stays = (t[None] < s["F"][:, None] + c["sinks"])[:, None]                   # the first tokens
    seen = (dist <= 0) & here[:, None] & (t[None] >= s["F"][:, None])[:, None] & (stays | (dist > -c["window"]))
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
                         slopes=s["slopes"], lse=s["lse"], pages=s["pages"], sinks=s["case"]["sinks"])
    return [s["out"], s["lse"]]


def _attn_exact(c, seed):
    if _work_attn(c)["flops"] > 4e12:
        return None
    s = _prepare_attn(c, seed)
    grp, bs, n0 = c["hq"] // c["hkv"], c["block"], 0
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    for b, (n, t, f) in enumerate(zip(s["q_lens"], s["t_lens"], s["firsts"])):
        blk = s["table"][b, :-(-t // bs)].long()
        kb, vb = (s[x].view(s["blocks"], bs, c["hkv"], D)[blk].view(-1, c["hkv"], D)[:t] for x in ("k", "v"))
        scale = [s[x] if s[x] is None else s[x].view(s["blocks"], bs, c["hkv"])[blk].view(-1, c["hkv"])[:t].double()
                 for x in ("k_scale", "v_scale")]
        for a in range(0, n, 512):
            e = min(n, a + 512)
            p = torch.arange(t - n + a, t - n + e, device="cuda")
            lo, hi = max(f, t - n + a - c["window"] + 1), t - n + e
            sink_end = min(lo, f + c["sinks"], hi)
            key = torch.cat([torch.arange(f, max(f, sink_end), device="cuda"),
                             torch.arange(min(lo, hi), hi, device="cuda")])
            if not key.numel():
                continue
            off = key[None].double() - p[:, None].double()
            ok = (off <= 0) & ((off > -c["window"]) | (key[None] < f + c["sinks"]))
            for h in range(c["hq"]):
                kk, vv = kb[key, h // grp].double(), vb[key, h // grp].double()
                if scale[0] is not None:
                    kk, vv = kk * scale[0][key, h // grp, None], vv * scale[1][key, h // grp, None]
                z = s["q"][n0 + a:n0 + e, h].double() @ kk.T / math.sqrt(D)
                if c["softcap"]:
                    z = c["softcap"] * torch.tanh(z / c["softcap"])
                if s["slopes"] is not None:
                    z = z + s["slopes"][h].double() * off
                z = z.masked_fill(~ok, -math.inf)
                lse[n0 + a:n0 + e, h] = torch.logsumexp(z, 1)
                w = torch.softmax(z, 1).nan_to_num(0.0)
                out[n0 + a:n0 + e, h] = w @ vv
        n0 += n
    return [out, lse]


def _work_attn(c):
    pairs = keys = 0
    for n, t, f in zip(*_lens(c)):
        w, s = c["window"], c["sinks"]
        lo = max(f, t - n - w + 1)                     # what some query sees: [f, f + s) and [lo, t)
        keys += (max(0, t - lo) + max(0, min(lo, f + s) - f)) if n else 0
        for p in range(t - n, t):
            a = max(f, p - w + 1)
            pairs += max(0, p + 1 - a) + max(0, min(a, f + s, p + 1) - f)
    n = sum(_lens(c)[0])
    per_key = 2 * c["hkv"] * (D * _BYTES[c["kv"]] + (4 if c["kv"] == "int8" else 0))
    return {"bytes": keys * per_key + n * c["hq"] * (2 * D * _BYTES[c["q"]] + 4), "flops": 4 * D * c["hq"] * pairs}


# ---------------------------------------------------------------------- norm
_EPS = 1e-6


def _prepare_norm(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, h = c["rows"], c["hidden"]
    s = dict(case=c)
    s["x"] = torch.randn(n, h, device="cuda", generator=g).to(_DT[c["x"]])
    s["r"] = None
    if c["add"]:
        # a residual stream: some channels are much larger than the rest
        big = 1 + 30 * (torch.rand(h, device="cuda", generator=g) < 0.005)
        s["r"] = (torch.randn(n, h, device="cuda", generator=g) * 3 * big).to(_DT[c["x"]])
    s["gamma"] = 1 + 0.2 * torch.randn(h, device="cuda", generator=g)
    s["groups"] = -(-h // c["group"]) if c["group"] else 1
    if own:
        lib = _lib()
        s["p"] = lib.make_norm_problem(n, h, c["x"], c["out"], eps=_EPS, scale_group=c["group"] if c["out"] == "e4m3" else 0)
        s["y"] = torch.empty(n, h, device="cuda", dtype=_DT[c["out"]])
        s["h"] = torch.empty_like(s["x"]) if c["add"] else None
        s["scale"] = torch.empty(n, s["groups"], device="cuda") if c["out"] == "e4m3" else None
    return s


def _norm_plain(s):
    c = s["case"]
    h = s["x"].float()
    res = []
    if c["add"]:
        h16 = (h + s["r"].float()).to(s["x"].dtype)
        res, h = [h16], h16.float()
    y = h * (s["gamma"] / torch.sqrt((h * h).mean(1, keepdim=True) + _EPS))
    if c["out"] != "e4m3":
        return res + [y.to(_DT[c["out"]])]
    n, g = c["rows"], s["groups"]
    width = -(-c["hidden"] // g) if not c["group"] else c["group"]
    z = torch.zeros(n, g * width, device="cuda")
    z[:, :c["hidden"]] = y
    z = z.view(n, g, width)
    scale = z.abs().amax(2) / 448
    q = (z / scale.masked_fill(scale == 0, 1.0)[..., None]).clamp(-448, 448)
    return res + [q.view(n, -1)[:, :c["hidden"]].to(torch.float8_e4m3fn).contiguous(), scale]


def _norm_own(s):
    _lib().dsa_add_rmsnorm(s["p"], s["x"], s["r"], s["gamma"], s["h"], s["y"], s["scale"])
    return [t for t in (s["h"], s["y"], s["scale"]) if t is not None]


def _norm_exact(c, seed):
    s = _prepare_norm(c, seed)
    h, res = s["x"].double(), []
    if s["r"] is not None:
        res = [h + s["r"].double()]
        h = res[0].to(s["x"].dtype).double()           # what is stored is what is normed
    y = s["gamma"].double() * h * torch.rsqrt(h.square().mean(1, keepdim=True) + _EPS)
    if c["out"] != "e4m3":
        return res + [y]
    step = c["group"] or c["hidden"]
    parts = [y[:, a:a + step] for a in range(0, c["hidden"], step)]
    scale = torch.stack([p.abs().amax(1) for p in parts], 1) / 448
    return res + [torch.cat([p / scale[:, i:i + 1] for i, p in enumerate(parts)], 1), scale]


def _work_norm(c):
    n, h = c["rows"], c["hidden"]
    b = _BYTES[c["x"]]
    groups = (-(-h // c["group"]) if c["group"] else 1) if c["out"] == "e4m3" else 0
    return {"bytes": n * h * (b * (3 if c["add"] else 1) + _BYTES[c["out"]]) + 4 * h + 4 * n * groups, "flops": 6 * n * h}


# ---------------------------------------------------------------------- rope
_POSITIONS = 32768


def _axis_of(c):
    """The axis whose position turns each rotary pair."""
    sec = [int(x) for x in c["sections"].split(",")]
    if c["mode"] == "whole":
        return [a for a, n in enumerate(sec) for _ in range(n)]
    left, out = list(sec), []
    while sum(left):
        for a in range(len(sec)):
            if left[a]:
                left[a] -= 1
                out.append(a)
    return out


def _prepare_rope(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, hq, hkv, r = c["tokens"], c["hq"], c["hkv"], random.Random(seed)
    axes = len(c["sections"].split(","))
    s = dict(case=c, axes=axes)
    # a projection's rows, of which the queries, keys and values are columns
    s["qkv"] = torch.randn(n, (hq + 2 * hkv) * D, device="cuda", generator=g).to(_DT[c["q"]])
    s["q"], s["k"], s["v"] = s["qkv"].split([hq * D, hkv * D, hkv * D], 1)
    # text, then an image's rows and columns, then text again
    at, pos = r.randrange(_POSITIONS // 2), []
    text, wide = n // 3, r.randint(8, 64)
    for i in range(n):
        if i < text or i >= 2 * text:
            pos.append([at + i % 4096] * axes)
        else:
            j = i - text
            pos.append(([at + text, at + text + j // wide % 4096, at + text + j % wide, at + text + j % 7])[:axes])
    s["pos"] = torch.tensor(pos, device="cuda").view(n, axes).clamp(max=_POSITIONS - 1).to(torch.int32).T.contiguous()
    ang = torch.arange(_POSITIONS, device="cuda").double()[:, None] * \
        1e6 ** (-torch.arange(c["rot"] // 2, device="cuda").double() * 2 / c["rot"])
    s["cos"], s["sin"] = ang.cos().float(), ang.sin().float()
    s["gq"] = 1 + 0.2 * torch.randn(D, device="cuda", generator=g) if c["norm"] else None
    s["gk"] = 1 + 0.2 * torch.randn(D, device="cuda", generator=g) if c["norm"] else None
    rows = (n + 255) // 128 * 128
    slots = torch.randperm(rows, device="cuda", generator=g)[:n]
    slots[n - c["padded"]:] = -1
    s["slots"], s["rows"] = slots.to(torch.int32), rows
    for name in ("K", "V"):     # (one row more, for what the plain form leaves out)
        s[name] = torch.zeros(rows + 1, hkv, D, device="cuda").to(_DT[c["kv"]])
        s[name + "_scale"] = torch.zeros(rows + 1, hkv, device="cuda") if c["kv"] == "int8" else None
    s["out"] = torch.empty(n, hq, D, device="cuda", dtype=_DT[c["q"]])
    if own:
        lib = _lib()
        s["p"] = lib.make_rope_axes_problem(n, hq, hkv, rows, [int(x) for x in c["sections"].split(",")], _POSITIONS,
                                            in_turn=c["mode"] == "turns", eps=_EPS, q_dtype=c["q"], kv_dtype=c["kv"])
    return s


def _rope_caches(s):
    """The caches as the values that they hold."""
    n = s["rows"]
    if s["K_scale"] is None:
        return [s["K"][:n], s["V"][:n]]
    return [(s[x][:n].float() * s[x + "_scale"][:n, :, None]).to(s["q"].dtype) for x in ("K", "V")]


def _rope_plain(s):
    c = s["case"]
    h, n, dt = c["rot"] // 2, c["tokens"], s["q"].dtype
    axis = torch.tensor(_axis_of(c), device="cuda")
    p = s["pos"].long()[axis].T                                                  # [N, r / 2]
    pair = torch.arange(h, device="cuda")
    cos, sin = s["cos"][p, pair][:, None], s["sin"][p, pair][:, None]

    def turn(x, gamma):
        x = x.float().view(n, -1, D)
        if gamma is not None:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS) * gamma
        a, b = x[..., :h], x[..., h:2 * h]
        return torch.cat([a * cos - b * sin, b * cos + a * sin, x[..., 2 * h:]], -1).to(dt)

    s["out"].copy_(turn(s["q"], s["gq"]))
    to = torch.where(s["slots"] >= 0, s["slots"], torch.full_like(s["slots"], s["rows"])).long()
    for name, x in (("K", turn(s["k"], s["gk"])), ("V", s["v"].view(n, -1, D))):
        if c["kv"] == "int8":
            scale = x.float().abs().amax(-1) / 127
            s[name][to] = torch.round(x.float() / scale[..., None]).clamp(-127, 127).to(torch.int8)
            s[name + "_scale"][to] = scale
        else:
            s[name][to] = x.to(s[name].dtype)
    return [s["out"]] + _rope_caches(s)


def _rope_own(s):
    n = s["rows"]
    ks, vs = (None, None) if s["K_scale"] is None else (s["K_scale"][:n], s["V_scale"][:n])
    _lib().dsa_rope_axes_append(s["p"], s["q"], s["k"], s["v"], s["gq"], s["gk"], s["cos"], s["sin"], s["pos"],
                                s["slots"], s["out"], s["K"][:n], s["V"][:n], ks, vs)
    return [s["out"]] + _rope_caches(s)


def _rope_exact(c, seed):
    s = _prepare_rope(c, seed)
    n, h = c["tokens"], c["rot"] // 2
    res = []
    cos, sin = (torch.stack([s[x][s["pos"][a].long(), i] for i, a in enumerate(_axis_of(c))], 1).double()
                for x in ("cos", "sin"))
    turn = torch.complex(cos, sin)[:, None]
    for x, gamma in ((s["q"], s["gq"]), (s["k"], s["gk"])):
        x = x.reshape(n, -1, D).double()
        if gamma is not None:
            x = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + _EPS) * gamma.double()
        z = torch.complex(x[..., :h].contiguous(), x[..., h:2 * h].contiguous()) * turn
        res.append(torch.cat([z.real, z.imag, x[..., 2 * h:]], -1))
    live = n - c["padded"]
    at = s["slots"][:live].long()
    for x in (res[1], s["v"].reshape(n, -1, D).double()):
        cache = torch.zeros(s["rows"], c["hkv"], D, dtype=torch.float64, device="cuda")
        if c["kv"] == "int8":      # what is quantised is the 16-bit value
            x = x.to(s["q"].dtype).double()
            step = x.abs().amax(-1, keepdim=True) / 127
            x = torch.round(x / step) * step
        cache[at] = x[:live]
        res.append(cache)
    return [res[0], res[2], res[3]]


def _work_rope(c):
    n, b = c["tokens"], _BYTES[c["q"]]
    live = n - c["padded"]
    kv = D * _BYTES[c["kv"]] + (4 if c["kv"] == "int8" else 0)
    axes = len(c["sections"].split(","))
    return {"bytes": n * c["hq"] * D * 2 * b + live * 2 * c["hkv"] * (D * b + kv) + n * (4 * c["rot"] + 4 * axes + 4),
            "flops": 8 * D * n * (c["hq"] + c["hkv"])}


# --------------------------------------------------------------------- slots
def _prepare_slots(c, seed):
    r = random.Random(seed)
    bs, n = c["block"], c["rows"]
    q = [1 if r.random() < 0.6 else r.randint(0, c["q_len"]) for _ in range(n)]
    q[0] = c["q_len"]
    t = [x + r.randint(0, c["total"] - x) for x in q]
    t[-1] = c["total"]
    used = [-(-x // bs) for x in t]
    per_seq, blocks = -(-c["total"] // bs), sum(used) + 5
    order, rows, k = list(range(blocks)), [], 0
    r.shuffle(order)
    for x in used:
        rows.append(order[k:k + x] + [-1] * (per_seq - x))
        k += x
    # the packed step's length is the case's, whatever the seed: the last tokens of a longer one wait for the next
    size = max(c["q_len"], n, int(n * (0.6 + 0.2 * c["q_len"])))
    total = 0
    for i in range(n):
        q[i] = min(q[i], size - total)
        total += q[i]
    s = dict(case=c, size=size + c["spare"], blocks=blocks)
    for name, v in (("S", q), ("T", t), ("table", rows)):
        s[name] = torch.tensor(v, dtype=torch.int32, device="cuda")
    if own:
        s["pages"] = _lib().make_pages(s["table"], bs, blocks)
        s["outs"] = [torch.empty(s["size"], dtype=torch.int32, device="cuda") for _ in range(3)]
        s["outs"].append(torch.empty(n + 1, dtype=torch.int32, device="cuda"))
    return s


def _slots_plain(s):
    bs = s["case"]["block"]
    end = torch.cumsum(s["S"].long(), 0)
    i = torch.arange(s["size"], device="cuda")
    row = torch.searchsorted(end, i, right=True)
    real = row < end.numel()
    row = torch.where(real, row, torch.zeros_like(row))
    pos = torch.where(real, s["T"].long()[row] - end[row] + i, torch.zeros_like(i))
    slot = s["table"].long()[row, pos // bs] * bs + pos % bs
    res = [torch.where(real, slot, -1), pos, torch.where(real, row, -1),
           torch.cat([torch.zeros(1, dtype=torch.long, device="cuda"), end])]
    return [x.to(torch.int32) for x in res]


def _slots_own(s):
    slots, pos, row, first = s["outs"]
    _lib().dsa_slot_map(s["S"], s["T"], slots, pages=s["pages"], positions=pos, rows=row, first=first)
    return list(s["outs"])


def _slots_size(c):
    return max(c["q_len"], c["rows"], int(c["rows"] * (0.6 + 0.2 * c["q_len"]))) + c["spare"]


def _work_slots(c):
    n = _slots_size(c)
    return {"bytes": 12 * n + 12 * c["rows"] + 4 * (n // c["block"] + c["rows"]), "flops": 0}


# -------------------------------------------------------------------- sample
def _prepare_sample(c, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = random.Random(seed)
    n, v = c["rows"], c["vocab"]
    x = torch.randn(n, v, device="cuda", generator=g) * 2
    # a few words that fit, in every row another number of them
    for i in range(n):
        k = r.choice([1, 3, 10, 40, 200])
        at = torch.randperm(v, device="cuda", generator=g)[:k]
        x[i, at] += 3 + 7 * torch.rand(k, device="cuda", generator=g)
    s = dict(case=c, logits=x.to(_DT[c["dtype"]]), u=torch.rand(n, device="cuda", generator=g))
    heat, k, p, low = [], [], [], []
    for i in range(n):
        what = c["mode"] if c["mode"] != "mixed" else r.choice(["heat", "topk", "topp", "minp", "greedy", "all"])
        heat.append(0.0 if what == "greedy" else r.choice([0.6, 0.7, 0.8, 1.0, 1.0, 1.3]))
        k.append(r.choice([5, 20, 40, 50, 100, 500]) if what in ("topk", "all") else 0)
        p.append(r.choice([0.5, 0.8, 0.9, 0.95, 0.99]) if what in ("topp", "all") else 1.0)
        low.append(r.choice([0.02, 0.05, 0.1]) if what in ("minp", "all") else 0.0)
    s["heat"] = torch.tensor(heat, device="cuda")
    s["k"] = torch.tensor(k, dtype=torch.int32, device="cuda") if max(k) else None
    s["p"] = torch.tensor(p, device="cuda") if min(p) < 1 else None
    s["low"] = torch.tensor(low, device="cuda") if max(low) else None
    if own:
        s["plan"] = _lib().make_sample_problem(n, v, c["dtype"])
        s["token"] = torch.empty(n, dtype=torch.int32, device="cuda")
        s["logprob"] = torch.empty(n, device="cuda")
    return s


def _sample_plain(s):
    # in 64 bits: where a draw falls between two of 100,000 tokens is next to a border nearly always
    c = s["case"]
    x = s["logits"].double()
    n, v = x.shape
    x = torch.where(x.isnan(), torch.full_like(x, -math.inf), x)
    greedy = (s["heat"] <= 0)[:, None]
    heat = torch.where(greedy, 1.0, s["heat"].double()[:, None])
    w = ((x - x.amax(1, keepdim=True)) / heat).exp_()
    val, at = torch.sort(x, dim=1, descending=True, stable=True)
    w = w.gather(1, at)
    keep = torch.arange(v, device="cuda")[None].expand(n, v)
    keep = (keep == 0) | ~greedy
    if s["k"] is not None:
        k = torch.where(s["k"] > 0, s["k"], torch.full_like(s["k"], v))[:, None]
        keep = keep & (torch.arange(v, device="cuda")[None] < k)
    if s["low"] is not None:
        low = w >= s["low"].double()[:, None]
    if s["p"] is not None:
        before = torch.cumsum(w * keep, 1)
        p = s["p"].double()[:, None]
        keep = keep & ((before - w < p * before[:, -1:]) | (p >= 1))
    if s["low"] is not None:
        keep = keep & low
    kept = torch.zeros_like(w).scatter_(1, at, w * keep)
    mass = torch.cumsum(kept, 1)
    total = mass[:, -1:]
    token = (mass <= s["u"].double()[:, None] * total).sum(1, keepdim=True).clamp(max=v - 1)
    return [token.view(-1).to(torch.int32), (kept.gather(1, token) / total).log().view(-1).float()]


def _sample_own(s):
    _lib().dsa_sample(s["plan"], s["logits"], s["u"], s["token"], temperature=s["heat"], top_k=s["k"], top_p=s["p"],
                      min_p=s["low"], logprobs=s["logprob"])
    return [s["token"], s["logprob"]]


def _sample_exact(c, seed):
    s = _prepare_sample(c, seed)
    res = []
    heat = s["heat"].tolist()
    for i in range(c["rows"]):
        if heat[i] <= 0:
            res.append(torch.zeros((), dtype=torch.float64, device="cuda"))
            continue
        z = s["logits"][i].double() / s["heat"][i].double()
        k = int(s["k"][i]) if s["k"] is not None else 0
        z, ids = torch.sort(z, descending=True, stable=True)
        z, ids = (z[:k], ids[:k]) if k else (z, ids)
        lp = torch.log_softmax(z, 0)
        n = z.numel()
        if s["p"] is not None and float(s["p"][i]) < 1:
            n = min(n, int((lp.exp().cumsum(0) < float(s["p"][i])).sum()) + 1)
        if s["low"] is not None and float(s["low"][i]) > 0:
            n = min(n, int((lp >= lp[0] + math.log(float(s["low"][i]))).sum()))
        lp = torch.log_softmax(z[:n], 0)
        ids, back = torch.sort(ids[:n])
        at = int((lp[back].exp().cumsum(0) <= float(s["u"][i])).sum())
        res.append(lp[back][min(at, n - 1)])
    return [None, torch.stack(res)]


def _work_sample(c):
    n = c["rows"] * c["vocab"]
    return {"bytes": n * _BYTES[c["dtype"]] + 28 * c["rows"], "flops": 4 * n}


# ----------------------------------------------------------------- interface
def prepare(case, seed):
    return {"attn": _prepare_attn, "norm": _prepare_norm, "rope": _prepare_rope, "slots": _prepare_slots,
            "sample": _prepare_sample}[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"attn": _attn_own, "norm": _norm_own, "rope": _rope_own, "slots": _slots_own, "sample": _sample_own}[op](state)
    return {"attn": _attn_plain, "norm": _norm_plain, "rope": _rope_plain, "slots": _slots_plain,
            "sample": _sample_plain}[op](state)


def exact(case, seed):
    if case["op"] == "slots":
        return None      # whole numbers
    return {"attn": _attn_exact, "norm": _norm_exact, "rope": _rope_exact, "sample": _sample_exact}[case["op"]](case, seed)


def work(case):
    return {"attn": _work_attn, "norm": _work_norm, "rope": _work_rope, "slots": _work_slots,
            "sample": _work_sample}[case["op"]](case)
