"""The CSA layer over 4-bit KV pages (csa_forward_paged), and the calls over one cache side by
side: graphs that share a workspace, two streams at once, the eviction in place."""
import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
from long_context_sparse_08_b200 import runner as R
from long_context_sparse_08_b200 import workloads as W
import tests.fp4_util as F
import tests.parity_util as U
from tests.test_kv_layout_attention import _dev, _paged, _paged_forward

pytestmark = [pytest.mark.gpu]


@pytest.fixture(autouse=True)
def no_device_error():
    csa.device_error()
    yield
    assert csa.device_error() == 0


@pytest.mark.parametrize("name,bf16_scores", [
    ("edge_decode_fp8_tc", 0), ("edge_decode_bf16_tc", 1), ("edge_decode_mxfp4", 0),
    ("mid_prefill_bf16_tc", 0)])
def test_forward_is_the_selection_and_the_attention(name, bf16_scores):
    """The selection does not depend on the KV format, and the attention gets the same list
    whether one call or two are made, so both parts agree bit for bit."""
    s, inp = U.inputs(name)
    dev = R.upload(inp, s)
    kv = W.bf16_bits_to_f32(inp["kv_cache"])
    rows = F.encode_rows(kv.reshape(-1, s.c)).reshape(s.B, s.n_cap, -1)
    out, idx, sc = _paged_forward(s, inp, dev, csa.CSA_MIXED_MXFP4_BF16, rows, None, bf16_scores)
    _, idx16, sc16 = _paged_forward(s, inp, dev, csa.CSA_BF16, inp["kv_cache"], None, bf16_scores)
    assert torch.equal(idx, idx16)
    for b in range(s.B):
        for t in range(s.T):
            n = int(max(0, min(inp["q_pos"][b, t] // s.m, s.n_cap)))
            assert torch.equal(sc[b, t, :n], sc16[b, t, :n])
    p = R.params_for(s)
    pool, table = _paged(rows, 32, 7)
    pages = csa.paged_kv(csa.CSA_MIXED_MXFP4_BF16, _dev(pool), None, _dev(table), pool.shape[0], 32,
                         table.shape[1])
    need = csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, csa.CSA_MIXED_MXFP4_BF16, s.B, s.T, s.n_cap)
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    alone = torch.empty_like(out)
    csa.csa_sparse_mqa_paged(p, s.B, s.T, dev["q"], dev["q_pos"], pages, idx, dev["win_kv"],
                             dev["win_kv"].shape[1], dev["win_pos0"], dev["sink"], None, alone, ws,
                             need)
    assert torch.equal(out, alone)
    assert torch.isfinite(out.float()).all()


def test_graphs_that_share_a_workspace():
    """The attention and the weight captured on the same workspace and replayed in turn."""
    P = F.Problem(B=2, pages=70, page_rows=8, seed=21)
    acc0 = torch.rand((P.B, P.N), device="cuda")
    want_out, want_acc = P.attention(), P.mass(acc0.clone(), 0.5)
    need = max(csa.workspace_size(P.p, csa.CSA_WS_HCA_MQA, P.kv_fmt, P.B, P.T, P.N),
               csa.attn_mass_workspace_size(P.p, P.B, P.T, P.N, 0))
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    out, acc = torch.zeros_like(want_out), acc0.clone()
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    with torch.cuda.graph(graphs[0]):
        P.attention(out=out, ws=ws)
    with torch.cuda.graph(graphs[1]):
        P.mass(acc, 0.5, ws=ws)
    for _ in range(3):
        out.zero_()
        acc.copy_(acc0)
        graphs[0].replay()
        graphs[1].replay()
        graphs[0].replay()
        assert torch.equal(out, want_out)
        assert torch.equal(acc, want_acc)


def test_two_streams_at_once():
    """The three operators on two streams, each with its own workspace and results."""
    P = F.Problem(B=2, k=300, pages=40, page_rows=32, m=4, seed=22)
    acc0 = torch.rand((P.B, P.N), device="cuda")
    want_out, want_acc = P.attention(), P.mass(acc0.clone(), 0.25)
    need_a = csa.workspace_size(P.p, csa.CSA_WS_SPARSE_MQA, P.kv_fmt, P.B, P.T, P.N)
    need_m = csa.attn_mass_workspace_size(P.p, P.B, P.T, P.N, 1)
    need_e = csa.evict_pages_workspace_size(P.B, P.pages)
    budget = 17
    pos = torch.from_numpy(P.pos[:, 0] - 1).cuda()
    runs = []
    for _ in range(2):
        runs.append(dict(
            stream=torch.cuda.Stream(), acc=acc0.clone(), out=torch.zeros_like(want_out),
            wa=torch.empty((need_a,), dtype=torch.uint8, device="cuda"),
            wm=torch.empty((need_m,), dtype=torch.uint8, device="cuda"),
            we=torch.empty((need_e,), dtype=torch.uint8, device="cuda"),
            table=P.table_d.clone(),
            kept=torch.empty((P.B, budget), dtype=torch.int32, device="cuda"),
            gone=torch.empty((P.B, P.pages), dtype=torch.int32, device="cuda"),
            counts=torch.empty((P.B, 3), dtype=torch.int32, device="cuda")))
    torch.cuda.synchronize()
    for _ in range(4):
        for r in runs:
            with torch.cuda.stream(r["stream"]):
                r["acc"].copy_(acc0)
                r["table"].copy_(P.table_d)
                P.attention(out=r["out"], ws=r["wa"])
                P.mass(r["acc"], 0.25, ws=r["wm"])
                csa.csa_evict_pages(P.p, P.B, P.page_rows, P.pages, pos, r["acc"], r["table"],
                                    budget, 1, 2, r["table"], r["kept"], None, r["gone"],
                                    r["counts"], r["we"], need_e)
    torch.cuda.synchronize()
    score = want_acc.view(P.B, P.pages, P.page_rows).amax(-1).cpu().numpy()
    for r in runs:
        assert torch.equal(r["out"], want_out)
        assert torch.equal(r["acc"], want_acc)
        for b in range(P.B):
            rest = sorted(range(1, P.pages - 2), key=lambda k: (-score[b, k], k))
            keep = sorted([0, P.pages - 2, P.pages - 1] + rest[:budget - 3])
            assert r["kept"][b].tolist() == keep
            gone = np.setdiff1d(np.arange(P.pages), keep)
            table = P.table[b].copy()
            table[gone] = -2
            assert r["table"][b].tolist() == table.tolist()  # written over its own input


@pytest.mark.parametrize("captured", [False, True])
def test_calls_one_after_another_on_one_workspace(captured):
    """Attention of few and of many queries, weight and eviction in turn, each with inputs that a
    copy just before it wrote, all on one workspace and with nothing waited for in between."""
    few = F.Problem(B=2, pages=70, page_rows=8, seed=31)
    many = F.Problem(B=3, T=70, k=40, pages=20, page_rows=32, m=4, pos=[2000, 900, 41], seed=32)
    need = max([csa.workspace_size(few.p, csa.CSA_WS_HCA_MQA, few.kv_fmt, 2, 1, few.N),
                csa.workspace_size(many.p, csa.CSA_WS_SPARSE_MQA, many.kv_fmt, 3, 70, many.N),
                csa.attn_mass_workspace_size(few.p, 2, 1, few.N, 0),
                csa.evict_pages_workspace_size(2, few.pages)])
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    n = 6
    q_few = [torch.roll(few.q, i, 3).contiguous() for i in range(n)]
    q_many = [torch.roll(many.q, i, 3).contiguous() for i in range(n)]
    pos = torch.from_numpy(few.pos[:, 0] - 1).cuda()
    budget = 20

    def buffers():
        return dict(few=[torch.zeros_like(few.q) for _ in range(n)],
                    many=[torch.zeros_like(many.q) for _ in range(n)],
                    acc=[torch.zeros((2, few.N), device="cuda") for _ in range(n)],
                    kept=[torch.zeros((2, budget), dtype=torch.int32, device="cuda") for _ in range(n)])

    table = torch.empty_like(few.table_d)
    gone = torch.empty_like(few.table_d)
    counts = torch.empty((2, 3), dtype=torch.int32, device="cuda")

    def steps(b, wait):
        for i in range(n):
            few.q.copy_(q_few[i])
            wait()
            few.attention(out=b["few"][i], ws=ws)
            wait()
            few.mass(b["acc"][i], 0.5, ws=ws)
            wait()
            csa.csa_evict_pages(few.p, 2, few.page_rows, few.pages, pos, b["acc"][i], few.table_d,
                                budget, 1, 1, table, b["kept"][i], None, gone, counts, ws, need)
            wait()
            many.q.copy_(q_many[i])
            many.attention(out=b["many"][i], ws=ws)
            wait()
            few.attention(out=b["few"][i], ws=ws)
            wait()

    want, got = buffers(), buffers()
    steps(want, torch.cuda.synchronize)
    if captured:
        s = torch.cuda.Stream()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            steps(got, lambda: None)
        for _ in range(3):
            for acc in got["acc"]:
                acc.zero_()
            g.replay()
    else:
        steps(got, lambda: None)
    torch.cuda.synchronize()
    for key in want:
        for i in range(n):
            assert torch.equal(want[key][i], got[key][i]), (key, i)
