"""Host-side checks of the full attention, page and beam calls: bad arguments
are refused before CUDA is touched, and workspaces are sized."""
import ctypes

import pytest


@pytest.fixture(scope="module")
def D():
    from top_sparse_attention_chunked_gb300 import build_lib, dsa
    build_lib.build()
    dsa.load_library()
    return dsa


def full(D, **kw):
    a = dict(q_len=[1, 5], total_len=[100, 300], num_q_heads=24, num_kv_heads=2, cache_capacity=512)
    a.update(kw)
    return D.make_full_attn_problem(**a)


@pytest.mark.parametrize("kw,frag", [
    (dict(q_len=[], total_len=[], cache_capacity=1), "batch"), (dict(num_q_heads=25), "multiple"), (dict(num_kv_heads=0), "multiple"),
    (dict(head_dim=64), "head_dim"), (dict(q_len=[1, 301]), "total_len"), (dict(q_len=[-1, 1]), "q_len"),
    (dict(total_len=[100, 513]), "total_len"), (dict(first_key=[0, 301]), "first_key"), (dict(first_key=[-1, 0]), "first_key"),
    (dict(window=-1), "window"), (dict(softcap=-1.0), "softcap"), (dict(softcap=float("inf")), "softcap"),
    (dict(softcap=float("nan")), "softcap"), (dict(softmax_scale=float("nan")), "softmax_scale"),
    (dict(q_dtype="int8", out_dtype="bf16"), "q_dtype"), (dict(q_dtype="fp32", out_dtype="bf16"), "q_dtype"),
    (dict(kv_dtype="fp32"), "kv_dtype"), (dict(q_dtype="fp16", kv_dtype="bf16"), "FP16 query"), (dict(out_dtype="int8"), "out_dtype"),
    (dict(q_len=[1, 1], total_len=[100, (1 << 20) + 1], cache_capacity=1 << 21), "above"),
])
def test_full_attention_refusals(D, kw, frag):
    p = full(D, **kw)
    lib = D.load_library()
    assert lib.dsa_full_attn_workspace_size(ctypes.byref(p)) == 0
    assert frag in lib.dsa_last_error_string().decode()


def call_full(D, p, pages=None, ws=0x10000, ws_bytes=1 << 40, **ptr):
    lib = D.load_library()
    v = dict(q=0x1000, k=0x2000, v=0x3000, ks=None, vs=None, slopes=None, out=0x4000, lse=None)
    v.update(ptr)
    args = [v[n] for n in ("q", "k", "v", "ks", "vs", "slopes", "out", "lse")] + [ws, ws_bytes, None]
    if pages is None:
        return lib.dsa_full_attn(ctypes.byref(p), *args)
    return lib.dsa_full_attn_paged(ctypes.byref(p), ctypes.byref(pages), *args)


def test_full_attention_pointer_checks(D):
    p = full(D)
    need = D.dsa_full_attn_workspace_size(p)
    assert call_full(D, p, q=0) == D.DSA_ERR_INVALID_ARG
    assert call_full(D, p, k=0x2008) == D.DSA_ERR_MISALIGNED
    assert call_full(D, p, out=0x4004) == D.DSA_ERR_MISALIGNED
    assert call_full(D, p, lse=0x4002) == D.DSA_ERR_MISALIGNED
    assert call_full(D, p, ks=0x5000, vs=0x5000) == D.DSA_ERR_INVALID_ARG
    assert call_full(D, full(D, kv_dtype="int8")) == D.DSA_ERR_INVALID_ARG
    assert call_full(D, p, ws_bytes=need - 1) == D.DSA_ERR_WORKSPACE
    assert call_full(D, p, ws=0x10010) == D.DSA_ERR_WORKSPACE
    assert call_full(D, p, ws=None) == D.DSA_ERR_WORKSPACE
    pages = D.DsaKvPages(128, 10, 4, 0x7000)
    assert call_full(D, p, D.DsaKvPages(64, 10, 8, 0x7000)) == D.DSA_ERR_UNSUPPORTED
    assert call_full(D, p, D.DsaKvPages(128, 10, 5, 0x7000)) == D.DSA_ERR_INVALID_ARG
    assert call_full(D, p, D.DsaKvPages(128, 10, 4, None)) == D.DSA_ERR_INVALID_ARG
    import torch
    if not torch.cuda.is_available():
        assert call_full(D, p) == D.DSA_ERR_NO_DEVICE
        assert call_full(D, p, pages) == D.DSA_ERR_NO_DEVICE


def test_full_attention_workspace_holds_every_block_s_parts(D):
    """At most one block per tile of 128 keys, 192 at the most, two parts each:
    a device with fewer SMs may use more blocks than one with more."""
    import random
    for seed in list(range(40)) + [63, 1330, 1979]:
        r = random.Random(seed)
        n = r.randint(1, 64)
        q = [r.choice([1, 1, 1, 2, r.randint(0, 40)]) for _ in range(n)]
        if sum(q) == 0:
            continue
        total = [x + r.choice([0, r.randint(0, 600), r.randint(0, 60)]) for x in q]
        grp, hkv = r.choice([1, 4, 12, 20, 130]), r.choice([1, 2, 4, 8])
        tiles = rows = 0
        for s, t in zip(q, total):
            rows = max(rows, min(256, s * grp))
            for row0 in range(0, s * grp, 256):
                tiles += hkv * -(-(t - s + (min(row0 + 256, s * grp) - 1) // grp + 1) // 128)
        p = D.make_full_attn_problem(q, total, grp * hkv, hkv)
        assert D.dsa_full_attn_workspace_size(p) >= 2 * min(tiles, 192) * rows * 130 * 4


def state(D, **kw):
    a = dict(block_size=128, num_blocks=16, rows=4, blocks_per_seq=8, block_table=0x10000, refs=0x20000)
    a.update(kw)
    return D.DsaPageState(*[a[n] for n, _ in D.DsaPageState._fields_])


@pytest.mark.parametrize("kw,frag", [(dict(block_size=100), "block_size"), (dict(block_size=64), "block_size"),
                                     (dict(num_blocks=0), "num_blocks"), (dict(num_blocks=(1 << 24) + 1), "num_blocks"),
                                     (dict(rows=0), "rows"), (dict(rows=4097), "rows"), (dict(blocks_per_seq=0), "blocks_per_seq"),
                                     (dict(blocks_per_seq=1 << 25), "blocks_per_seq")])
def test_page_state_refusals(D, kw, frag):
    lib = D.load_library()
    st = state(D, **kw)
    assert lib.dsa_pages_workspace_size(ctypes.byref(st)) == 0
    assert frag in lib.dsa_last_error_string().decode()


def call_update(D, st, pools=(), ws=0x900000, ws_bytes=1 << 40, **ptr):
    lib = D.load_library()
    v = dict(parent=0x30000, keep=0x31000, new=0x32000, first=None, table=0x10000, refs=0x20000, counts=None)
    v.update(ptr)
    arr = (D.DsaPagePool * max(1, len(pools)))(*[D.DsaPagePool(*x) for x in pools])
    return lib.dsa_pages_update(ctypes.byref(st), v["parent"], v["keep"], v["new"], v["first"], len(pools), arr,
                                v["table"], v["refs"], v["counts"], ws, ws_bytes, None)


def test_page_call_checks(D):
    st = state(D)
    assert call_update(D, st, parent=None) == D.DSA_ERR_INVALID_ARG
    assert call_update(D, st, keep=0x31002) == D.DSA_ERR_MISALIGNED
    assert call_update(D, st, table=None) == D.DSA_ERR_INVALID_ARG
    assert call_update(D, st, table=0x10004) == D.DSA_ERR_INVALID_ARG          # overlaps the old table
    assert call_update(D, st, refs=0x10010) == D.DSA_ERR_INVALID_ARG           # lies in the table
    assert call_update(D, st, parent=0x10010) == D.DSA_ERR_INVALID_ARG
    assert call_update(D, st, [(0, 256)]) == D.DSA_ERR_INVALID_ARG
    assert call_update(D, st, [(0x100008, 256)]) == D.DSA_ERR_MISALIGNED
    assert call_update(D, st, [(0x100000, 40)]) == D.DSA_ERR_MISALIGNED
    assert call_update(D, st, [(0x100000, 0)]) == D.DSA_ERR_INVALID_ARG
    assert call_update(D, st, [(0x100000, 256), (0x100100, 256)]) == D.DSA_ERR_INVALID_ARG   # overlap
    assert call_update(D, st, [(0xff00, 256)]) == D.DSA_ERR_INVALID_ARG        # over the table
    assert call_update(D, st, ws=0x900010) == D.DSA_ERR_WORKSPACE
    assert call_update(D, st, ws_bytes=D.dsa_pages_workspace_size(st) - 1) == D.DSA_ERR_WORKSPACE
    import torch
    if not torch.cuda.is_available():
        assert call_update(D, st, [(0x100000, 256), (0x200000, 512)]) == D.DSA_ERR_NO_DEVICE


@pytest.mark.parametrize("kw,frag", [(dict(batch=0), "batch"), (dict(beams=65), "beams"), (dict(vocab=0), "vocab"),
                                     (dict(vocab=(1 << 24) + 1), "vocab"), (dict(select=0), "select"), (dict(select=65), "select"),
                                     (dict(logits_dtype="int8"), "logits"), (dict(pad_token=100), "pad_token"),
                                     (dict(pad_token=-1), "pad_token"), (dict(row_stride=99), "row_stride"),
                                     (dict(batch=60000, beams=2), "65535")])
def test_beam_refusals(D, kw, frag):
    a = dict(batch=2, beams=4, vocab=100, select=8)
    a.update(kw)
    p = D.make_beam_problem(**a)
    lib = D.load_library()
    assert lib.dsa_beam_workspace_size(ctypes.byref(p)) == 0
    assert frag in lib.dsa_last_error_string().decode()


def test_beam_call_checks(D):
    lib = D.load_library()
    p = D.make_beam_problem(2, 4, 100, 8, "fp32")
    need = D.dsa_beam_workspace_size(p)

    def call(logits=0x1000, scores=0x2000, o=0x3000, ws=0x10000, n=need, tokens=0x4000, done=None, p=p):
        return lib.dsa_beam_select(ctypes.byref(p), logits, scores, done, o, tokens, 0x5000, ws, n, None)

    assert call(logits=None) == D.DSA_ERR_INVALID_ARG
    assert call(o=0x2000) == D.DSA_ERR_INVALID_ARG           # select != beams
    assert call(o=0x1ffc) == D.DSA_ERR_INVALID_ARG
    assert call(tokens=0x3010) == D.DSA_ERR_INVALID_ARG
    assert call(o=0x1000 + 8 * 400 - 4) == D.DSA_ERR_INVALID_ARG
    assert call(done=0x4020) == D.DSA_ERR_INVALID_ARG
    same = D.make_beam_problem(2, 8, 100, 8, "fp32")
    assert call(tokens=0x2000, p=same) == D.DSA_ERR_INVALID_ARG
    import torch
    if not torch.cuda.is_available():
        assert call(o=0x2000, p=same, logits=0x8000, ws=0x100000, n=1 << 40) == D.DSA_ERR_NO_DEVICE
        assert call() == D.DSA_ERR_NO_DEVICE
    assert call(logits=0x1002) == D.DSA_ERR_MISALIGNED
    assert call(o=0x3001) == D.DSA_ERR_MISALIGNED
    assert call(n=need - 1) == D.DSA_ERR_WORKSPACE
    assert call(ws=0x10020) == D.DSA_ERR_WORKSPACE


def test_struct_layouts_match_the_header(D):
    assert ctypes.sizeof(D.DsaFullProblem) == 4 * (6 + 3 * 64 + 2 + 3)
    assert ctypes.sizeof(D.DsaPageState) == 32 and D.DsaPageState.block_table.offset == 16
    assert ctypes.sizeof(D.DsaPagePool) == 16
    assert ctypes.sizeof(D.DsaBeamProblem) == 32 and D.DsaBeamProblem.row_stride.offset == 24
