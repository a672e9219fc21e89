"""The query operand of the attention over 4-bit rows and of the attention weight: many queries (from
65536 heads on a warp prepares eight, and the launch is an ordinary one), and queries that the launch
right before has written."""
import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
import tests.fp4_util as F
from tests.test_attn_mass import check_mass

pytestmark = [pytest.mark.gpu]


@pytest.fixture(autouse=True)
def no_device_error():
    csa.device_error()
    yield
    assert csa.device_error() == 0


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
def test_queries_written_by_the_launch_before(fmt):
    """A step writes q and its positions and calls at once, on one stream and in a graph; each time
    the results are those of a call that found q there."""
    P = F.Problem(B=3, k=70, pages=20, page_rows=32, m=4, seed=62, fmt=fmt)
    qs = [torch.roll(P.q, i, 2).contiguous() for i in range(4)]
    acc0 = torch.rand((P.B, P.N), device="cuda")
    pos0 = P.q_pos.clone()
    need_a = csa.workspace_size(P.p, csa.CSA_WS_SPARSE_MQA, P.kv_fmt, P.B, P.T, P.N)
    need_m = csa.attn_mass_workspace_size(P.p, P.B, P.T, P.N, 1)
    ws = torch.empty((max(need_a, need_m),), dtype=torch.uint8, device="cuda")
    out = torch.empty((P.B, P.T, P.H, 512), dtype=torch.bfloat16, device="cuda")
    accs = [acc0.clone() for _ in qs]
    outs = [torch.empty_like(out) for _ in qs]

    def step(i):
        P.q_pos.copy_(pos0 - 128 * i)
        P.q.copy_(qs[i])
        if fmt == "fp4":
            P.attention(out=outs[i], ws=ws)
        P.q.copy_(qs[i - 1])
        P.q.copy_(qs[i])
        P.mass(accs[i], 0.5, ws=ws)

    want = []
    for i in range(len(qs)):
        step(i)
        torch.cuda.synchronize()
        P.q.copy_(qs[i])
        torch.cuda.synchronize()
        alone = P.mass(acc0.clone(), 0.5)
        torch.cuda.synchronize()
        assert torch.equal(alone, accs[i])
        want.append((outs[i].clone(), alone))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        for i in range(len(qs)):
            step(i)
    for turn in range(30):
        for a in accs:
            a.copy_(acc0)
        if turn % 2:
            g.replay()
        else:
            for i in range(len(qs)):
                step(i)
        for i in range(len(qs)):
            assert torch.equal(accs[i], want[i][1])
            if fmt == "fp4":
                assert torch.equal(outs[i], want[i][0])


MANY = [dict(B=1, T=1024, k=16),                      # the first size at which a warp takes eight heads
        dict(B=3, T=114, k=9, H=192, weight=True),    # 65664 heads, three groups each
        dict(B=16, T=65, k=33, n_win=37)]


@pytest.mark.parametrize("kw", MANY, ids=str)
def test_attention_of_many_queries(kw):
    P = F.Problem(pages=30, page_rows=32, m=4, seed=60, pos=[500 + 90 * b for b in range(kw["B"])], **kw)
    assert P.B * P.T * P.H >= 65536
    F.check_attention(P.attention(), P.out64(), str(kw))


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("kw", MANY + [dict(B=2, T=512, k=0, pages=3, m=128, pos=[60, 20000])], ids=str)
def test_weight_of_many_queries(kw, fmt):
    """The end of a prompt, lists and dense."""
    d = dict(pages=30, page_rows=32, m=4, seed=61, pos=[500 + 90 * b for b in range(kw["B"])])
    d.update(kw)
    P = F.Problem(fmt=fmt, **d)
    assert P.B * P.T * P.H >= 65536
    acc = torch.from_numpy(np.random.default_rng(0).random((P.B, P.N)).astype(np.float32)).cuda()
    before = acc.double().cpu().numpy()
    check_mass(P.mass(acc.clone(), 0.9), P.mass64(acc, 0.9), before, 0.9, str(kw))
