"""The attention weight per cache entry (csa_attn_mass_paged) against float64 forms, the page
eviction by it (csa_evict_pages) against a plain form, and the three together: attention, weight,
eviction, attention over what is left."""
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


def _acc(P, seed=0):
    g = np.random.default_rng(seed)
    return torch.from_numpy(g.random((P.B, P.N)).astype(np.float32)).cuda()


def check_mass(got, ref, before, decay, what=""):
    """A logit is off by the rest of q_hat that its two parts leave (2^-16 of a value for bf16,
    2^-22 for f16; at most 8.8e-6 rms of a logit at the default scale), by fp32 sums of 512
    products and of an exponent's argument of up to about 30 (30 * 2^-24 = 1.8e-6): a weight by
    about 1e-5 rms. Six of that bound one entry; the sum over 64 heads and more, whose errors are
    independent, is held to a fifth of it in the 2-norm. 2^-40 steps and fp32 rounding of acc are
    far below."""
    got = got.double().cpu().numpy()
    d = got - ref
    added = ref - decay * before
    assert (np.abs(d) <= 6e-5 * np.abs(added) + 2.0 ** -22 * np.abs(ref) + 1e-9).all(), what
    assert np.sqrt((d * d).sum()) <= 1.2e-5 * np.sqrt((added ** 2).sum()) + \
        2.0 ** -23 * np.sqrt((ref ** 2).sum()) + 1e-9, what


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(B=1, pages=1, page_rows=1, pos=[5]),                        # nothing visible: decay only
    dict(B=2, pages=1, page_rows=1, pos=[127, 128]),
    dict(B=3, pages=13, page_rows=5, pos=[130, 128 * 33, 10 ** 6], H=128, weight=True),
    dict(B=2, pages=40, page_rows=8, pos=[128 * 319, 128 * 100 + 3], sink=False),
    dict(B=1, pages=129, page_rows=32),
    dict(B=40, pages=9, page_rows=16, H=192),                        # one split a stream
    dict(B=2, T=5, pages=30, page_rows=8, pos=[1000, 128 * 200]),
    dict(B=2, pages=5, page_rows=8, n_win=0, sink=False),
], ids=str)
def test_dense(kw, fmt):
    P = F.Problem(seed=11, fmt=fmt, **kw)
    acc = _acc(P)
    before = acc.double().cpu().numpy()
    check_mass(P.mass(acc.clone(), 0.9), P.mass64(acc, 0.9), before, 0.9, str(kw))


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("kw", [
    dict(B=1, k=1, pages=1, pos=[4]),
    dict(B=2, k=7, pages=2, pos=[3, 200]),
    dict(B=3, k=512, pages=40, pos=[2051, 5119, 5120], weight=True, H=128),
    dict(B=2, T=6, k=300, pages=30, pos=[900, 30]),
    dict(B=1, k=2048, pages=100, sink=False),
], ids=str)
def test_sparse(kw, fmt):
    P = F.Problem(seed=12, fmt=fmt, m=4, page_rows=32, **kw)
    acc = _acc(P)
    before = acc.double().cpu().numpy()
    check_mass(P.mass(acc.clone(), 1.0), P.mass64(acc, 1.0), before, 1.0, str(kw))


def test_list_with_duplicates_and_holes_repeats_bit_for_bit():
    P = F.Problem(B=2, T=3, k=200, pages=20, page_rows=32, m=4, seed=13)
    idx = P.idx.cpu().numpy()
    idx[0, :, 1::4] = idx[0, :, ::4]
    idx[1, 0, ::3] = -1
    idx[1, 1, 5] = P.N
    P.idx = torch.from_numpy(idx).cuda()
    acc = _acc(P)
    before = acc.double().cpu().numpy()
    got = [P.mass(acc.clone(), 0.5) for _ in range(3)]
    check_mass(got[0], P.mass64(acc, 0.5), before, 0.5)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_evicted_and_missing_pages_and_not_a_number():
    P = F.Problem(B=2, pages=40, page_rows=4, seed=14)
    P.table[0, 3:9] = -2
    P.refresh()
    acc = _acc(P)
    check_mass(P.mass(acc.clone()), P.mass64(acc, 1.0), acc.double().cpu().numpy(), 1.0)
    P.table[0, 1] = -1
    P.refresh()
    P.mass(acc.clone())
    torch.cuda.synchronize()
    assert csa.device_error() == 226
    P = F.Problem(B=1, k=40, pages=4, page_rows=32, m=4, seed=15)
    P.q[0, 0, 3, 7] = float("nan")  # the queries of one head: every listed entry's sum
    got = P.mass(torch.zeros((1, P.N), device="cuda")).cpu().numpy()[0]
    listed = P.idx.cpu().numpy().ravel()
    assert np.isnan(got[listed]).all()
    assert (np.delete(got, listed) == 0).all()


def test_mass_captured_on_another_stream():
    P = F.Problem(B=2, k=100, pages=10, page_rows=32, m=4, seed=16)
    need = csa.attn_mass_workspace_size(P.p, P.B, P.T, P.N, 1)
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    acc0 = _acc(P)
    acc = acc0.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        P.mass(acc, 0.9, ws=ws)
    acc.copy_(acc0)
    g.replay()
    g.replay()
    want = P.mass64(torch.from_numpy(P.mass64(acc0, 0.9)), 0.9)
    torch.cuda.synchronize()
    check_mass(acc, want, acc0.double().cpu().numpy(), 0.81)


# ------------------------------- eviction -------------------------------

def plain_evict(m, page_rows, pos, acc, table, budget, first, last):
    B, P = table.shape
    out = dict(table=table.copy(), kept=np.full((B, budget), -1), evicted=np.full((B, P), -1),
               entries=np.full((B, budget * page_rows), -1), counts=np.zeros((B, 3), int))
    for b in range(B):
        n = min(max(pos[b] + 1, 0) // m, P * page_rows)
        used = -(-n // page_rows)
        live = [k for k in range(used) if table[b, k] >= 0]
        always = {k for k in live if k < first or k >= used - last}

        def score(k):
            w = acc[b, k * page_rows:min((k + 1) * page_rows, n)].astype(np.float64)
            w = w[~np.isnan(w)]
            return w.max() if len(w) else -np.inf

        def rank(k):
            nan = np.isnan(acc[b, k * page_rows:min((k + 1) * page_rows, n)]).all()
            return (nan, -score(k), k)

        rest = sorted((k for k in live if k not in always), key=rank)
        keep = sorted(list(always) + rest[:max(0, budget - len(always))])
        stay = set(keep)
        gone = [k for k in live if k not in stay]
        ent = [e for k in keep for e in range(k * page_rows, min((k + 1) * page_rows, n))]
        out["table"][b, gone] = -2
        out["kept"][b, :len(keep)] = keep
        out["evicted"][b, :len(gone)] = gone
        out["entries"][b, :len(ent)] = ent
        out["counts"][b] = len(keep), len(ent), len(gone)
    return out


def run_evict(m, page_rows, pos, acc, table, budget, first, last, in_place=False, entries=True):
    B, P = table.shape
    p = csa.make_params(m=m)
    i32 = dict(dtype=torch.int32, device="cuda")
    td = torch.from_numpy(table).cuda()
    o = dict(table=td if in_place else torch.full((B, P), 77, **i32),
             kept=torch.full((B, budget), 77, **i32), evicted=torch.full((B, P), 77, **i32),
             entries=torch.full((B, budget * page_rows), 77, **i32) if entries else None,
             counts=torch.full((B, 3), 77, **i32))
    need = csa.evict_pages_workspace_size(B, P)
    ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
    csa.csa_evict_pages(p, B, page_rows, P, torch.from_numpy(np.asarray(pos, np.int64)).cuda(),
                        torch.from_numpy(acc).cuda(), td, budget, first, last, o["table"], o["kept"],
                        o["entries"], o["evicted"], o["counts"], ws, need)
    return {k: v.cpu().numpy() for k, v in o.items() if v is not None}


@pytest.mark.parametrize("pages,page_rows,budget,first,last,m", [
    (1, 1, 1, 0, 0, 4), (5, 3, 2, 1, 1, 4), (37, 32, 11, 2, 3, 4), (600, 1, 512, 4, 16, 128),
    (1500, 2, 700, 0, 1, 8), (5000, 5, 1, 0, 0, 4), (9000, 1, 4096, 0, 0, 128), (70, 33, 70, 3, 3, 4),
    (2049, 64, 1024, 10, 10, 4), (20001, 4, 9000, 1, 1, 4), (3, 12, 2, 1, 0, 4)])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict(pages, page_rows, budget, first, last, m, kind):
    g = np.random.default_rng(pages + page_rows)
    B, N = 4, pages * page_rows
    acc = (g.exponential(size=(B, N)) ** 3).astype(np.float32)
    if kind == "ties":
        acc = np.round(acc * 2) / 2
        acc[1] = 0.25
    if kind == "odd":
        acc[g.random((B, N)) < 0.3] = np.nan
        acc[g.random((B, N)) < 0.1] = np.inf
        acc[g.random((B, N)) < 0.2] = -0.0
        acc[2] *= -1
    table = g.permutation(B * pages).reshape(B, pages).astype(np.int32)
    table[2, g.random(pages) < 0.4] = -2
    table[3, pages // 2:] = -1
    pos = [N * m - 1, N * m - 1 - m * (page_rows // 2 + 1), int(0.7 * N * m), N * m + 1000]
    if kind == "odd":
        pos[1] = -1
    want = plain_evict(m, page_rows, pos, acc, table, budget, first, last)
    for in_place in (False, True):
        got = run_evict(m, page_rows, pos, acc, table, budget, first, last, in_place)
        for k in want:
            assert (got[k] == want[k]).all(), (k, in_place)
    assert set(run_evict(m, page_rows, pos, acc, table, budget, first, last, entries=False)) == \
        {"table", "kept", "evicted", "counts"}


def test_evict_more_pages_than_shared_memory_holds():
    """Keys in the workspace (more than 40960 pages a request), and several digits to decide."""
    g = np.random.default_rng(5)
    pages, B = 90003, 2
    acc = g.integers(0, 1 << 24, size=(B, pages)).astype(np.float32)
    table = np.arange(B * pages, dtype=np.int32).reshape(B, pages)
    table[1, ::7] = -2
    pos = [pages - 1, pages - 5]
    for budget, rows in ((1, 1), (50000, 1), (90000, 1), (30000, 3)):
        w = np.repeat(acc, rows, 1)
        p = [rows * x for x in pos]
        want = plain_evict(1, rows, p, w, table, budget, 0, 1)
        got = run_evict(1, rows, p, w, table, budget, 0, 1)
        for k in want:
            assert (got[k] == want[k]).all(), (k, budget)


# ------------------------------- together -------------------------------

def test_a_cache_under_a_budget():
    """Decode steps of an HCA layer over 4-bit pages of one entry: the weight is accumulated,
    the eviction keeps the most attended entries, the allocator takes their pages back, and the
    attention over the list of kept entries equals the dense attention over the evicted table,
    both equal to the float64 form over what is left."""
    P = F.Problem(B=2, pages=300, page_rows=1, m=128, pos=[128 * 300, 128 * 211 + 5], seed=17)
    alloc = csa.PageAlloc(P.n_pages, P.B, P.pages)
    used = [300, 211]
    for b in range(P.B):
        alloc.reserve(b, used[b])
    rows64, pool = P.rows64.copy(), P.pool.clone()
    for b in range(P.B):  # the problem's rows where the allocator put their pages
        for e in range(used[b]):
            rows64[alloc.table[b, e]] = P.rows64[P.table[b, e]]
            pool[alloc.table[b, e]] = P.pool[P.table[b, e]]
    P.rows64, P.pool, P.table = rows64, pool, np.array(alloc.table)
    P.refresh()
    acc = torch.zeros((P.B, P.N), device="cuda")
    want = acc
    for step in range(3):
        P.q.copy_(torch.roll(P.q, 1, 3))
        want = torch.from_numpy(P.mass64(want, 0.9))
        P.mass(acc, 0.9)
    check_mass(acc, want.numpy(), np.zeros((P.B, P.N)), 1.0)
    budget = 100
    pos = P.pos[:, 0] - 1
    got = run_evict(128, 1, pos, acc.cpu().numpy(), P.table, budget, 4, 16)
    ref = plain_evict(128, 1, pos, acc.cpu().numpy(), P.table, budget, 4, 16)
    for k in ref:
        assert (got[k] == ref[k]).all(), k
    free = alloc.free_pages
    for b in range(P.B):
        alloc.evict(b, got["evicted"][b][:got["counts"][b, 2]])
    assert alloc.free_pages == free + int(got["counts"][:, 2].sum())
    P.table = np.array(alloc.table)
    assert (P.table == got["table"]).all()
    P.refresh()
    dense = P.attention()
    ref = P.out64()
    F.check_attention(dense, ref, "dense over the evicted table")
    P.k, P.p.topk = budget, budget
    P.idx = torch.from_numpy(got["entries"].reshape(P.B, 1, budget).astype(np.int32)).cuda()
    F.check_attention(P.attention(), ref, "list of kept entries")
    alloc.reserve(0, 300)  # evicted pages are not mapped again
    assert (np.array(alloc.table) == P.table).all()
