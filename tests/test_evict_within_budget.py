"""Page eviction where some or all requests of a batch lie within their budget, so that nothing is
to be chosen for them: below it, at it and one above it, over one and several rounds of 8192 pages,
called again and again on one stream and captured, with equal results."""
import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
from tests.test_attn_mass import plain_evict, run_evict

pytestmark = [pytest.mark.gpu]


@pytest.mark.parametrize("pages,page_rows,budget", [
    (31, 1, 31), (600, 1, 640), (8192, 1, 8192), (9000, 1, 9000), (8192, 4, 8192), (9000, 3, 9500),
    (20000, 1, 19999), (45000, 2, 45000)])
def test_batches_around_the_budget(pages, page_rows, budget):
    g = np.random.default_rng(pages + budget)
    B, N, m = 8, pages * page_rows, 4
    acc = g.exponential(size=(B, N)).astype(np.float32)
    acc[5] = 0.5
    table = g.permutation(B * pages).reshape(B, pages).astype(np.int32)
    table[6, ::3] = -2
    # used pages: none, one, half, one below, at and one above the budget (as far as the table goes)
    used = [0, 1, pages // 2, budget - 1, budget, budget + 1, pages, pages]
    pos = [min(u, pages) * page_rows * m - 1 for u in used]
    want = plain_evict(m, page_rows, pos, acc, table, budget, 1, 2)
    for _ in range(5):
        got = run_evict(m, page_rows, pos, acc, table, budget, 1, 2)
        for k in want:
            assert (got[k] == want[k]).all(), k


def test_many_requests_within_their_budget_repeat():
    """148 requests at once, each within its budget, replayed from a graph: every replay writes the
    table as it was, all pages as kept and none as evicted."""
    B, pages, page_rows, m = 148, 8192, 1, 128
    p = csa.make_params(m=m)
    i32 = dict(dtype=torch.int32, device="cuda")
    acc = torch.rand((B, pages), device="cuda")
    table = torch.randperm(B * pages, device="cuda").to(torch.int32).view(B, pages)
    used = (torch.arange(B, device="cuda") * 55 + 9).clamp_max(pages)
    pos = used * m - 1
    new, gone = torch.empty((B, pages), **i32), torch.empty((B, pages), **i32)
    kept, counts = torch.empty((B, pages), **i32), torch.empty((B, 3), **i32)
    need = csa.evict_pages_workspace_size(B, pages)
    ws = torch.empty((max(need, 16),), dtype=torch.uint8, device="cuda")

    def call():
        csa.csa_evict_pages(p, B, page_rows, pages, pos, acc, table, pages, 1, 1, new, kept, None, gone,
                            counts, ws, need)

    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        call()
    e = torch.arange(pages, device="cuda")
    want_kept = torch.where(e < used[:, None], e, -1).to(torch.int32)
    want_counts = torch.stack((used, used, torch.zeros_like(used)), 1).to(torch.int32)
    bad = torch.zeros((), dtype=torch.int64, device="cuda")
    for _ in range(200):
        for t in (new, gone, kept, counts):
            t.fill_(77)
        g.replay()
        bad += (new != table).sum() + (gone != -1).sum() + (kept != want_kept).sum() + \
            (counts != want_counts).sum()
    assert int(bad) == 0
