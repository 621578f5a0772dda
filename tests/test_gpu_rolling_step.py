"""A decoder layer on rolling paged caches, the calls together as a server makes
them: residual + norm, projection, the blocks' growth, the slot map, rotary
positions of several axes with the append, attention with a window and first
tokens, residual + norm, logits and sampling. Requests of unequal prompts run in
one packed, padded step; every stage is held against 64 bits on what the GPU's
stage before it gave."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_add_rmsnorm import check as check_norm
from tests.test_gpu_full_attn import D, check as check_attn  # noqa: F401 (D is a fixture)
from tests.test_gpu_full_attn_sinks import reference as attn_reference
from tests.test_gpu_rope_axes import reference as rope_reference
from tests.test_gpu_sample import NEAR, reference as sample_reference

pytestmark = pytest.mark.gpu

HQ, HKV, HIDDEN, VOCAB, BLOCK, EPS = 8, 2, 640, 1003, 128, 1e-6
WINDOW, SINKS, SECTIONS, STEPS, PAD = 150, 5, (24, 20, 20), 40, 3
PROMPTS = (301, 1, 140)


@pytest.mark.parametrize("kv", ["bf16", "fp16", "int8"])
def test_packed_steps(D, kv):  # noqa: F811
    dev, bf, B = "cuda", torch.bfloat16, len(PROMPTS)
    g = torch.Generator(device=dev).manual_seed(11)
    r = lambda *s, std=1.0: torch.randn(*s, device=dev, generator=g) * std  # noqa: E731
    width = (HQ + 2 * HKV) * 128
    embed, wqkv, wo = r(VOCAB, HIDDEN).to(bf), r(HIDDEN, width, std=HIDDEN ** -0.5).to(bf), r(HQ * 128, HIDDEN, std=0.05).to(bf)
    wl = r(HIDDEN, VOCAB, std=3 * HIDDEN ** -0.5).to(bf)
    g1, g2, gq, gk = 1 + r(HIDDEN, std=0.2), 1 + r(HIDDEN, std=0.2), 1 + r(128, std=0.2), 1 + r(128, std=0.2)
    max_pos, half = 512, sum(SECTIONS)
    ang = torch.arange(max_pos, device=dev).double()[:, None] * 1e4 ** (-torch.arange(half, device=dev).double() / half)
    cos, sin = ang.cos().float(), ang.sin().float()

    per_seq, nb = 3, 12
    cap = per_seq * BLOCK
    i32 = dict(dtype=torch.int32, device=dev)
    kdt = {"bf16": bf, "fp16": torch.float16, "int8": torch.int8}[kv]
    K, V = (torch.zeros(nb * BLOCK, HKV, 128, device=dev).to(kdt) for _ in range(2))
    ks, vs = (torch.zeros(nb * BLOCK, HKV, device=dev) if kv == "int8" else None for _ in range(2))
    table, refs = torch.full((B, per_seq), -1, **i32), torch.zeros(nb, **i32)
    state, pages = D.make_page_state(table, refs, BLOCK), D.make_pages(table, BLOCK, nb)
    pools = D.make_page_pools([t for t in (K, V, ks, vs) if t is not None], nb)
    pws = D.alloc_pages_workspace(state)
    own = torch.arange(B, **i32)

    heat, top_k = torch.tensor([0.7, 1.0, 0.0], device=dev), torch.tensor([40, 0, 0], **i32)
    top_p, min_p = torch.tensor([0.95, 0.9, 1.0], device=dev), torch.tensor([0.0, 0.01, 0.0], device=dev)
    gen = torch.Generator().manual_seed(12)
    tokens = [torch.randint(0, VOCAB, (n,), generator=gen).tolist() for n in PROMPTS]
    total, fresh, checked = [0] * B, [list(t) for t in tokens], 0
    for step in range(STEPS):
        q_len = [len(f) for f in fresh]
        total = [t + n for t, n in zip(total, q_len)]
        n = sum(q_len)
        N = n + PAD                                           # the step is padded
        ids = torch.tensor(sum(fresh, []) + [0] * PAD, device=dev)
        res = embed[ids]

        # residual + norm (nothing to add in front of the first layer), projection
        x = torch.empty_like(res)
        D.dsa_add_rmsnorm(D.make_norm_problem(N, HIDDEN, eps=EPS), res, None, g1, None, x)
        check_norm(res.cpu(), g1.cpu(), x, None, "bf16", 0, EPS)
        qkv = x @ wqkv
        q, k, v = qkv.split([HQ * 128, HKV * 128, HKV * 128], 1)

        # blocks, slots, positions, append
        dt, dq = torch.tensor(total, **i32), torch.tensor(q_len, **i32)
        D.dsa_pages_update(state, own, dt - dq, dt, pools, pws)
        assert D.dsa_read_device_status(pws) == 0
        slots, pos, first = torch.empty(N, **i32), torch.empty(N, **i32), torch.empty(B + 1, **i32)
        D.dsa_slot_map(dq, dt, slots, pages=pages, positions=pos, first=first)
        assert first.tolist() == [sum(q_len[:b]) for b in range(B + 1)]
        axes = torch.stack([pos, pos // 2, (pos * 7) % 100]).contiguous()   # (as an image's rows and columns might go)
        old = [t.clone() for t in (K, V)]
        p = D.make_rope_axes_problem(N, HQ, HKV, nb * BLOCK, SECTIONS, max_pos, in_turn=True, eps=EPS, kv_dtype=kv)
        qr = torch.empty(N, HQ, 128, device=dev, dtype=bf)
        D.dsa_rope_axes_append(p, q, k, v, gq, gk, cos, sin, axes, slots, qr, K, V, ks, vs)
        rope = dict(tokens=N, hq=HQ, hkv=HKV, sections=list(SECTIONS), half=half, qdt="bf16", max_pos=max_pos, qkv=qkv.cpu(),
                    split=[HQ * 128, HKV * 128, HKV * 128], pos=axes.cpu(), cos=cos.cpu(), sin=sin.cpu(), gq=gq.cpu(), gk=gk.cpu())
        (rq, eq), (rk, ek) = rope_reference(rope, True, EPS)
        assert (np.abs(qr.double().cpu().numpy() - rq) <= 2.0 ** -8 * (np.abs(rq) + eq) + eq).all()
        at = slots[:n].long().cpu()
        where = table.long().cpu()
        want = torch.cat([where[b, torch.arange(total[b] - q_len[b], total[b]) // BLOCK] * BLOCK +
                          torch.arange(total[b] - q_len[b], total[b]) % BLOCK for b in range(B)])
        assert torch.equal(at, want) and (slots[n:] == -1).all()
        scale = (lambda s: s.double().cpu()[..., None]) if kv == "int8" else (lambda s: 1.0)
        kd, vd = K.double().cpu() * scale(ks), V.double().cpu() * scale(vs)
        # BF16's rounding, then half a step of the cache's (INT8: of its scale)
        lost = 0.501 * ks.double().cpu().numpy()[at][..., None] if kv == "int8" else 0.0
        assert (np.abs(kd[at].numpy() - rk[:n]) <= 2.0 ** -8 * (np.abs(rk[:n]) + ek[:n]) + ek[:n] + lost + 2.0 ** -25).all()
        rest = torch.ones(nb * BLOCK, dtype=torch.bool)
        rest[at] = False
        assert torch.equal(K.cpu()[rest], old[0].cpu()[rest]) and torch.equal(V.cpu()[rest], old[1].cpu()[rest])

        # attention over the window and the first tokens
        ap = D.make_full_attn_problem(q_len, total, HQ, HKV, cap, window=WINDOW, kv_dtype=kv)
        ws = D.alloc_full_attn_workspace(ap)
        att, lse = torch.zeros(N, HQ, 128, device=dev, dtype=bf), torch.zeros(N, HQ, device=dev)
        D.dsa_full_attn(ap, qr, K, V, ks, vs, att, ws, lse=lse, pages=pages, sinks=SINKS)
        assert D.dsa_read_device_status(ws) == 0 and (att[n:] == 0).all()
        c = dict(q_len=q_len, total_len=total, first_key=[0] * B, hq=HQ, hkv=HKV, qdt="bf16", kvdt=kv, q=qr.cpu())
        rows = (where.clamp(min=0)[:, :, None] * BLOCK + torch.arange(BLOCK)).view(B, cap)
        c["k"], c["v"] = K.cpu()[rows], V.cpu()[rows]
        c["k_scale"], c["v_scale"] = (None, None) if ks is None else (ks.cpu()[rows], vs.cpu()[rows])
        check_attn(c, att, lse, attn_reference(c, WINDOW, SINKS), "bf16")

        # the layer's end, logits of the requests' last tokens, and what comes next
        h, y = torch.empty_like(res), torch.empty_like(res)
        back = att.view(N, HQ * 128) @ wo
        D.dsa_add_rmsnorm(D.make_norm_problem(N, HIDDEN, eps=EPS), back, res, g2, h, y)
        assert torch.equal(h, (back.float() + res.float()).to(bf))
        check_norm(h.cpu(), g2.cpu(), y, None, "bf16", 0, EPS)
        logits = y[first[1:].long() - 1] @ wl
        u, tok, lp = torch.rand(B, generator=gen), torch.empty(B, **i32), torch.empty(B, device=dev)
        D.dsa_sample(D.make_sample_problem(B, VOCAB), logits, u.to(dev), tok, temperature=heat, top_k=top_k, top_p=top_p, min_p=min_p,
                     logprobs=lp)
        for b in range(B):
            t, wlp, near = sample_reference(logits[b].double().cpu().numpy(), float(u[b]), float(heat[b]), int(top_k[b]),
                                            float(top_p[b]), float(min_p[b]))
            if near >= NEAR:
                checked += 1
                assert int(tok[b]) == t and math.isclose(float(lp[b]), wlp, rel_tol=2.0 ** -20, abs_tol=2.0 ** -28)
        fresh = [[int(t)] for t in tok]
    assert checked >= 0.95 * STEPS * B
