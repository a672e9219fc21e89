"""Attention over 4-bit KV pages (CSA_MIXED_MXFP4_BF16) and the writers of such pages, against
float64 forms on the same bytes (tests/fp4_util.py)."""
import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
import tests.fp4_util as F

pytestmark = [pytest.mark.gpu]


@pytest.fixture(autouse=True)
def no_device_error():
    csa.device_error()
    yield
    assert csa.device_error() == 0


SPARSE = dict(m=4, page_rows=32)


@pytest.mark.parametrize("kw", [
    dict(B=1, pages=1, page_rows=1, pos=[0]),                       # the query's own token only
    dict(B=2, pages=1, page_rows=1, pos=[127, 128]),                # no entry, one entry
    dict(B=3, pages=64, page_rows=1, pos=[128 * 63 + 5, 128 * 64, 128 * 65 + 1]),
    dict(B=3, pages=13, page_rows=5, pos=[130, 128 * 33, 10 ** 6], H=128),  # ends inside a page
    dict(B=2, pages=40, page_rows=8, pos=[128 * 319, 128 * 100 + 3], sink=False),
    dict(B=2, pages=40, page_rows=8, weight=True, H=192),
    dict(B=1, pages=129, page_rows=32),                             # many chunks a CTA
    dict(B=40, pages=9, page_rows=16, H=256),                       # one split a stream
    dict(B=2, pages=5, page_rows=8, n_win=0, sink=False),           # entries only
    dict(B=2, pages=5, page_rows=8, n_win=0, pos=[5, 700], sink=False),  # nothing at all
    dict(B=2, T=3, pages=30, page_rows=8, pos=[1000, 128 * 200]),   # several queries, linear window
    dict(B=2, pages=30, page_rows=8, n_win=37),
    dict(B=1, pages=4, page_rows=8, base=500.0, scale=0.2),
], ids=str)
def test_dense(kw):
    P = F.Problem(seed=1, **kw)
    F.check_attention(P.attention(), P.out64(), str(kw), P.scale)


@pytest.mark.parametrize("kw", [
    dict(B=1, k=1, pages=1, pos=[4]),
    dict(B=2, k=7, pages=2, pos=[3, 200]),                          # no entry, more entries than k
    dict(B=3, k=64, pages=20, pos=[40, 256, 2560]),                 # fewer, as many, more than k
    dict(B=3, k=512, pages=40, pos=[2051, 5119, 5120], H=64, weight=True),
    dict(B=2, k=1024, pages=80, H=128, sink=False),
    dict(B=2, k=2048, pages=100, H=64),
    dict(B=5, T=33, k=100, pages=30, pos=[900, 4, 2000, 3000, 100]),
    dict(B=1, T=200, k=257, pages=30, pos=[700]),
], ids=str)
def test_sparse(kw):
    P = F.Problem(seed=2, **SPARSE, **kw)
    F.check_attention(P.attention(), P.out64(), str(kw), P.scale)


def test_list_with_holes_duplicates_and_out_of_range_entries():
    P = F.Problem(B=2, k=200, pages=20, seed=3, **SPARSE)
    idx = P.idx.cpu().numpy()
    idx[0, 0, ::3] = -1
    idx[0, 0, 1] = P.N + 5
    idx[0, 0, 4] = idx[0, 0, 5]  # a row listed twice counts twice
    idx[1, 0, :] = -1            # window and sink only
    P.idx = torch.from_numpy(idx).cuda()
    F.check_attention(P.attention(), P.out64(), "holes")


def test_pages_evicted_or_missing():
    P = F.Problem(B=2, pages=40, page_rows=4, seed=4)
    P.table[0, 3:9] = -2
    P.table[1, :] = -2   # every page evicted: the window alone
    P.refresh()
    F.check_attention(P.attention(), P.out64(), "evicted")
    torch.cuda.synchronize()
    assert csa.device_error() == 0
    P.table[0, 1], P.table[0, 2] = -1, P.n_pages
    P.refresh()
    F.check_attention(P.attention(), P.out64(), "missing")
    torch.cuda.synchronize()
    assert csa.device_error() == 216


def test_evicted_pages_of_bf16_rows_are_masked_quietly():
    P = F.Problem(B=2, pages=40, page_rows=4, seed=5, fmt="bf16")
    P.table[0, 3:9] = -2
    P.refresh()
    got = P.attention().double().cpu().numpy()
    ref = P.out64()
    assert np.sqrt(((got - ref) ** 2).sum() / (ref ** 2).sum()) <= 5e-3  # the bf16 path's own bound


def _poison(P):
    """NaN in every byte that the queries may not read: rows of the pool that no visible entry
    has, and window rows outside the last n_win positions."""
    keep = np.zeros((P.n_pages, P.page_rows), bool)
    for b in range(P.B):
        vis = min(int(P.pos[b].max()) // P.m, P.N)
        e = np.arange(vis) if not P.k else np.unique(P.idx[b].cpu().numpy())
        e = e[e >= 0]
        keep[P.table[b, e // P.page_rows], e % P.page_rows] = True
        rows = np.unique([t for q in P.pos[b] for t in range(max(0, q - P.n_win + 1), q + 1)])
        at = rows % P.L if P.win_pos0 is None else rows - int(P.win_pos0[b])
        gone = np.setdiff1d(np.arange(P.L), at)
        P.win[b, torch.from_numpy(gone).cuda()] = float("nan")
    P.pool.view(torch.uint8)[torch.from_numpy(~keep).cuda()] = 255


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(B=2, pages=40, page_rows=8, pos=[128 * 100 + 5, 128 * 3]),
    dict(B=2, pages=6, page_rows=8, pos=[60, 128 * 21], ring=False),
    dict(B=2, T=3, k=70, pages=20, page_rows=32, m=4, pos=[41, 2000]),
], ids=str)
def test_not_a_number_where_nothing_is_read(kw, fmt):
    P = F.Problem(seed=9, fmt=fmt, **kw)
    _poison(P)
    if fmt == "fp4":
        F.check_attention(P.attention(), P.out64(), str(kw))
    got = P.mass(torch.zeros((P.B, P.N), device="cuda")).double().cpu().numpy()
    ref = P.mass64(torch.zeros((P.B, P.N)), 1.0)
    # an entry's weight is a sum of T * H weights, each off by a few 1e-6 of itself at most
    assert np.abs(got - ref).max() <= 1e-5 * P.T * P.H


@pytest.mark.parametrize("k", [0, 300])
def test_far_offsets_and_large_logits(k):
    """Pages whose byte offset passes 2^32, and logits so large that one row takes all weight
    and the running maximum is raised again and again."""
    n_pages = (1 << 32) // (32 * 368) + 500
    P = F.Problem(B=1, k=k, pages=24, page_rows=32, m=4 if k else 128, seed=6, scale=1.5)
    pool = torch.zeros((n_pages, 32, 368), dtype=torch.uint8, device="cuda")
    far = n_pages - 1 - np.arange(P.n_pages)
    pool[torch.from_numpy(far).cuda()] = P.pool
    P.table64 = P.table
    P.pool, P.table = pool, far[P.table].astype(np.int32)
    P.n_pages, rows64 = n_pages, P.rows64
    P.refresh()
    got = P.attention()
    torch.cuda.synchronize()
    P.n_pages, P.table, P.rows64 = len(far), P.table64, rows64
    F.check_attention(got, P.out64(), "far", scale=1.5)


@pytest.mark.parametrize("kw", [
    dict(B=80, H=128, pages=20, page_rows=16),               # a stream a CTA, seven chunks
    dict(B=3, T=60, k=500, pages=30, page_rows=32, m=4),     # several streams a CTA
    dict(B=16, pages=400, page_rows=8),                      # nine splits of several chunks
    dict(B=16, pages=400, page_rows=8, sink=False, n_win=0),
], ids=str)
def test_maxima_raised_in_later_chunks(kw):
    """Logits with a standard deviation of 34: most chunks raise some head's running maximum by
    more than any threshold would let pass."""
    P = F.Problem(seed=8, scale=1.5, **kw)
    F.check_attention(P.attention(), P.out64(), str(kw), scale=1.5)


def test_graph_replay_other_stream_and_repeatability():
    P = F.Problem(B=2, pages=70, page_rows=8, seed=7, H=128)
    ref = P.attention()
    ws = torch.empty((csa.workspace_size(P.p, csa.CSA_WS_HCA_MQA, P.kv_fmt, P.B, P.T, P.N),),
                     dtype=torch.uint8, device="cuda")
    out = torch.zeros_like(ref)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        P.attention(out=out, ws=ws)
    s.synchronize()
    assert torch.equal(out, ref)  # no atomics: the same bits
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        P.attention(out=out, ws=ws)
    P.q.copy_(torch.roll(P.q, 1, 2))
    for _ in range(3):
        out.zero_()
        g.replay()
    torch.cuda.synchronize()
    F.check_attention(out, P.out64(), "replayed")


# ------------------------------- the writers -------------------------------

def _rows(n, c, r, seed=0):
    g = np.random.default_rng(seed)
    x = g.standard_normal((n, c)).astype(np.float32)
    x[0] = 0
    x[1, ::2] = 0
    x[2] *= 1e6    # saturates
    x[3] *= 1e-7   # below the smallest exponent
    x[4] = np.tile([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, -0.25, -0.75, -5.0, -6.0, 0.5, -3.5,
                    4.0, 1.0], c // 16)  # midpoints
    x[5, :32] = [65504.0] + [1.0] * 31
    return x


@pytest.mark.parametrize("c,r", [(512, 64), (512, 32), (256, 128), (128, 64)])
@pytest.mark.parametrize("io", ["f32", "bf16"])
def test_encode_paged_bytes(c, r, io):
    n, B, page_rows, first = 21, 2, 4, 3
    x = np.stack([_rows(n, c, r, s) for s in range(B)])
    t = torch.from_numpy(x)
    t = t if io == "f32" else t.to(torch.bfloat16)
    pages = -(-(first + n) // page_rows)
    table = np.random.default_rng(1).permutation(B * pages).reshape(B, pages).astype(np.int32)
    pool = torch.full((B * pages, page_rows, F.row_bytes(c, r)), 0xAB, dtype=torch.uint8, device="cuda")
    td = torch.from_numpy(table).cuda()
    kv = csa.paged_kv(csa.CSA_MIXED_MXFP4_BF16, pool, None, td, B * pages, page_rows, pages)
    p = csa.make_params(c=c, rope_dims=r)
    rows = t.cuda()
    csa.csa_encode_paged(p, csa.CSA_F32 if io == "f32" else csa.CSA_BF16, B, n, first, rows, kv)
    got = pool.cpu().numpy()
    for b in range(B):
        want = F.encode_rows(t[b].float().numpy(), r)
        for i in range(n):
            e = first + i
            assert (got[table[b, e // page_rows], e % page_rows] == want[i]).all(), (b, i)
        for e in list(range(first)) + list(range(first + n, pages * page_rows)):
            assert (got[table[b, e // page_rows], e % page_rows] == 0xAB).all()  # untouched


@pytest.mark.parametrize("overlap,m", [(1, 4), (0, 8)])
def test_state_append_writes_the_encoded_entry(overlap, m):
    """The appended entry equals the encoding of the same entry appended in fp32."""
    B, c, n_tok, page_rows = 3, 512, 5 * m, 2
    g = np.random.default_rng(9)
    p = csa.make_params(m=m, overlap=overlap, c=c)
    S, Rr = (2 * m, 4) if overlap else (m, 2)
    bias = torch.from_numpy(g.standard_normal(((2 if overlap else 1) * m, c)).astype(np.float32)).cuda()
    pages = -(-5 // page_rows)
    table = torch.arange(B * pages, dtype=torch.int32, device="cuda").view(B, pages)
    out = {}
    for fmt in (csa.CSA_F32, csa.CSA_MIXED_MXFP4_BF16):
        gg = np.random.default_rng(10)
        state = torch.zeros((B, S, Rr, c), device="cuda")
        width = c * 4 if fmt == csa.CSA_F32 else 368
        pool = torch.zeros((B * pages, page_rows, width), dtype=torch.uint8, device="cuda")
        for t in range(n_tok):
            x = [torch.from_numpy(gg.standard_normal((B, c)).astype(np.float32)).cuda()
                 for _ in range(4)]
            pos = torch.full((B,), t, dtype=torch.int64, device="cuda")
            csa.csa_state_append(p, csa.CSA_F32, B, pos, x[0], x[1] if overlap else None, x[2],
                                 x[3] if overlap else None, None, bias, None, 1, state, None, fmt,
                                 pool, None, B * pages, page_rows, table, pages)
        out[fmt] = pool.cpu().numpy()
    f32 = out[csa.CSA_F32].view(np.float32).reshape(-1, c)[:]
    got = out[csa.CSA_MIXED_MXFP4_BF16].reshape(-1, 368)
    live = [b * pages * page_rows + i for b in range(B) for i in range(5)]
    assert (got[live] == F.encode_rows(f32[live])).all()
