"""dsa_full_attn on batches whose thread blocks work on several items of
different kinds, against the definition in 64 bits."""
import pytest
import torch

from tests._full_attn_batches import LOOPS, MIXED, NO_KEY, ONE_TILE, TYPES, batch, grow, reference
from tests.test_gpu_full_attn import D, call, check  # noqa: F401 (D is a fixture)

pytestmark = pytest.mark.gpu


def run(D, c, repeats=1, **kw):  # noqa: F811
    """One checked call; `repeats` more must give the same bits."""
    out, lse, st = call(D, c, **kw)
    check(c, out, lse, reference(c, **{k: v for k, v in kw.items() if k in ("window", "softcap", "slopes", "scale")}),
          kw.get("out_dtype") or c["qdt"])
    ws, n = D.alloc_full_attn_workspace(st["p"]), sum(c["q_len"])
    slopes = kw.get("slopes")
    slopes = None if slopes is None else slopes.cuda()
    for _ in range(repeats):
        o, s = torch.empty_like(out), torch.empty_like(lse)
        D.dsa_full_attn(st["p"], st["q"], st["dev"]["k"], st["dev"]["v"], st["dev"]["k_scale"], st["dev"]["v_scale"],
                        o, ws, slopes=slopes, lse=s, pages=st["pages"])
        assert torch.equal(o[:n], out[:n]) and torch.equal(s[:n], lse[:n])


@pytest.mark.parametrize("kv", ["fp16", "int8"])
@pytest.mark.parametrize("name", list(MIXED))
def test_scaled_queries_of_narrow_and_wide_items(D, name, kv):  # noqa: F811
    """BF16 queries that are scaled for products in FP16, where a block goes from an item of up to 128 rows
    to a wider one: the second one's units must not touch the first one's statistics."""
    run(D, batch(name, "bf16", kv, block=256, seed=21), repeats=40)


@pytest.mark.parametrize("q,kv", [("bf16", "bf16"), ("bf16", "fp16"), ("bf16", "int8"), ("fp16", "int8")])
@pytest.mark.parametrize("name", list(NO_KEY))
def test_runs_of_items_without_a_key(D, name, q, kv):  # noqa: F811
    """Many items of more than 128 rows that see nothing, in a row in one block: zeros, -infinity, and what
    follows is right. (A hand-over with the tensor core that such items take part in has no bound on how far
    one half of the rows runs ahead of the other.)"""
    run(D, batch(NO_KEY[name], q, kv, block=128, seed=22), repeats=5, out_dtype="fp32" if q == "fp16" else None)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("name", list(LOOPS))
def test_several_tiles_and_segments_a_block(D, name, q, kv):  # noqa: F811
    """The main loop in earnest: the rings go round, slots are joined, blocks change items."""
    run(D, batch(LOOPS[name], q, kv, block=128, seed=23), repeats=3)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("name", list(LOOPS))
def test_window_cap_and_bias_over_several_tiles(D, name, q, kv):  # noqa: F811
    c = batch(LOOPS[name], q, kv, seed=24, first_key=[min(100, t) for t in LOOPS[name]["total_len"]])
    slopes = torch.tensor([2.0 ** (-4 - 0.25 * h) for h in range(c["hq"])])
    run(D, c, window=2500, softcap=20.0, slopes=slopes)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("name", list(LOOPS))
@pytest.mark.parametrize("top", [30.0, 400.0])
def test_logits_that_grow_over_several_tiles(D, name, q, kv, top):  # noqa: F811
    """O is rescaled within segments, at every tile or every few."""
    run(D, grow(batch(LOOPS[name], q, kv, seed=25), top), out_dtype="fp32")


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("name", list(ONE_TILE))
def test_narrow_items_of_one_tile_before_wide_ones(D, name, q, kv):  # noqa: F811
    """The slot without a tile of such an item must not run ahead of the product thread."""
    run(D, batch(ONE_TILE[name], q, kv, block=128, seed=30), repeats=20)


CAPPED = ([1, 0, 2], [40], [150, 3])


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("kw", [dict(softcap=1e3), dict(softcap=1e4), dict(softcap=1e6), dict(softcap=3e38),
                                dict(softcap=1e4, scale=8.0), dict(softcap=300.0, scale=2.0), dict(softcap=30.0)])
def test_wide_caps_keep_the_logits_precision(D, q, kv, kw):  # noqa: F811
    """A cap far above the logits leaves them as they are, to a few roundings of the logit (not of the cap)."""
    for q_len in CAPPED:
        c = batch(dict(q_len=q_len, total_len=[700 + 100 * n for n in q_len], hq=12, hkv=2), q, kv, block=128, seed=26)
        run(D, c, out_dtype="fp32", **kw)


@pytest.mark.parametrize("q,kv", TYPES)
def test_wide_caps_beside_masked_and_large_keys(D, q, kv):  # noqa: F811
    """What masked keys hold, or another row's large logits, do not cost a row's precision."""
    c = batch(dict(q_len=[40, 3, 200], total_len=[450, 300, 400], hq=12, hkv=2, first_key=[70, 5, 3]), q, kv, seed=27)
    if kv != "int8":
        for b, f in enumerate(c["first_key"]):
            c["k"][b, :f] = 3e4
    c["q"][::3] *= 300
    run(D, c, out_dtype="fp32", softcap=1e4)
    run(D, c, out_dtype="fp32", softcap=1e6)


@pytest.mark.parametrize("q,kv", TYPES)
@pytest.mark.parametrize("softcap,q_mul", [(1e-4, 2.0 ** -13), (1e-4, 1.0), (1e-5, 2.0 ** -21), (1e-5, 2.0 ** -20), (1e-5, 2.0 ** -18),
                                           (1e-9, 2.0 ** -34), (1e-9, 2.0 ** -33), (1e-30, 1.0), (1e-42, 1.0)])
def test_narrow_caps(D, q, kv, softcap, q_mul):  # noqa: F811
    """Caps far below the unit of the logits, arguments in each range: no overflow on the way."""
    for q_len in CAPPED:
        c = batch(dict(q_len=q_len, total_len=[700 + 100 * n for n in q_len], hq=12, hkv=2), q, kv, seed=28)
        c["q"] = (c["q"].float() * q_mul).to(c["q"].dtype)
        c["q"][:, 1] = 0
        run(D, c, out_dtype="fp32", softcap=softcap)


@pytest.mark.parametrize("kv", ["fp16", "int8"])
def test_a_narrow_cap_on_large_queries(D, kv):  # noqa: F811
    """Units of a scaled row over a cap that leave fp32, beside keys of zeros."""
    c = batch(dict(q_len=[2, 40, 150], total_len=[300, 300, 300], hq=12, hkv=2), "bf16", kv, seed=29)
    c["q"] = (c["q"].float() * 2.0 ** 100).to(torch.bfloat16)
    c["k"][:, ::3] = 0
    run(D, c, out_dtype="fp32", softcap=1e-30)


def test_a_short_block_table_is_refused(D):  # noqa: F811
    c = batch(dict(q_len=[1, 2], total_len=[300, 200], hq=8, hkv=2), "bf16", "bf16", block=128)
    p = D.make_full_attn_problem(c["q_len"], c["total_len"], 8, 2, cache_capacity=c["cap"])
    q, k, v = c["q"].cuda(), c["pools"]["k"].cuda(), c["pools"]["v"].cuda()
    with pytest.raises(ValueError, match="rows for 2 sequences"):
        D.dsa_full_attn(p, q, k, v, None, None, torch.empty_like(q), D.alloc_full_attn_workspace(p),
                        pages=D.make_pages(c["table"][:1].contiguous().cuda(), 128, c["nb"]))
    # (rows behind the call's sequences are another call's)
    more = torch.cat([c["table"], torch.full_like(c["table"], 1 << 30)])
    D.dsa_full_attn(p, q, k, v, None, None, torch.empty_like(q), ws := D.alloc_full_attn_workspace(p),
                    pages=D.make_pages(more.cuda(), 128, c["nb"]))
    assert D.dsa_read_device_status(ws) == 0
