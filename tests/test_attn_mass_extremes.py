"""The attention weight per entry at the ends of its range: rows that are not numbers, weights far
below the largest, sums as large as they can be,
no rows at all."""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
import tests.fp4_util as F
from tests.fp4_values import C, encode_rows

pytestmark = [pytest.mark.gpu]


@pytest.fixture(autouse=True)
def no_device_error():
    csa.device_error()
    yield
    assert csa.device_error() == 0


# ------------------------------- not a number -------------------------------

def _spoil(P, b, entries):
    """NaN in the last RoPE value (bf16 in either format) of entries of request b."""
    for e in entries:
        row = P.pool[int(P.table[b, e // P.page_rows]), e % P.page_rows].view(torch.uint8)
        row[-2:] = torch.tensor([0xc0, 0x7f], dtype=torch.uint8, device="cuda")


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("kw,entries", [
    (dict(pages=1, page_rows=1), [0]),                      # the only entry
    (dict(pages=65, page_rows=1), [64]),                    # the only row of its chunk
    (dict(pages=65, page_rows=1, n_win=0, sink=False), [64]),
    (dict(pages=385, page_rows=2, H=128), [768, 769]),      # the two rows of its chunk
    (dict(pages=40, page_rows=8, n_win=65), [3]),           # among others
    (dict(pages=600, page_rows=1, k=65, m=4), None),        # last of a list
    (dict(pages=600, page_rows=1, k=1, m=4), None),
], ids=str)
def test_an_entry_that_is_not_a_number(kw, entries, fmt):
    """A weight is a share of a sum over all rows of its query: where one of them is NaN, all are.
    The other request keeps its values."""
    P = F.Problem(B=2, seed=31, fmt=fmt, **kw)
    if entries is None:
        entries = [int(P.idx[0, 0, -1])]
    _spoil(P, 0, entries)
    acc0 = torch.rand((P.B, P.N), device="cuda")
    got = P.mass(acc0.clone(), 0.5)
    listed = P.idx[0].flatten().long() if P.k else torch.arange(P.N, device="cuda")
    assert torch.isnan(got[0, listed]).all()
    rest = torch.ones(P.N, dtype=torch.bool, device="cuda")
    rest[listed] = False
    assert torch.equal(got[0, rest], acc0[0, rest] * 0.5)
    assert torch.isfinite(got[1]).all()
    if fmt == "fp4":
        out = P.attention()
        assert torch.isnan(out[0]).all() and torch.isfinite(out[1]).all()


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
def test_a_window_row_that_is_not_a_number(fmt):
    """The window's 65th row is the only one of its chunk."""
    P = F.Problem(B=2, pages=10, page_rows=8, n_win=65, seed=32, fmt=fmt)
    P.win[0, int(P.pos[0, 0]) % 65, 100] = float("nan")
    got = P.mass(torch.zeros((P.B, P.N), device="cuda"))
    assert torch.isnan(got[0]).all() and torch.isfinite(got[1]).all()


def test_sink_beside_rows_that_are_not_numbers():
    """All rows NaN, the sink finite."""
    P = F.Problem(B=1, pages=3, page_rows=1, n_win=0, seed=33)
    _spoil(P, 0, [0, 1, 2])
    assert torch.isnan(P.mass(torch.zeros((1, 3), device="cuda"))).all()


# ------------------------------- small weights, large sums -------------------------------

def _two_kinds(fmt, n, strong, B, T, H, k, log2_ratio, n_win=0):
    """Entries that hold 1 in dims 128-447 (weak) or 0-127 (strong) under a query that is 2 in dims
    0-127 after its normalisation: a weak row's weight is 2^-log2_ratio of a strong one's, and only
    fp32 roundings lie between."""
    rows = np.zeros((n, C), np.float32)
    rows[:, 128:448] = 1
    rows[strong, :128], rows[strong, 128:448] = 1, 0
    scale = log2_ratio * math.log(2) / 256
    P = F.Problem(B=B, T=T, H=H, k=k, pages=n, page_rows=1, m=1, n_win=n_win, sink=False, fmt=fmt,
                  scale=scale, seed=41, pos=[n] * B)
    order = torch.from_numpy(P.table[0].astype(np.int64)).cuda()
    data = torch.from_numpy(encode_rows(rows)).cuda() if fmt == "fp4" else \
        torch.from_numpy(rows).to(torch.bfloat16).cuda()
    P.pool[order, 0] = data
    P.q.zero_()
    P.q[..., :128] = 0.75
    z = 256 / math.sqrt(1 + 1e-6 / (0.75 ** 2 / 4)) * scale
    return P, math.exp(-z)


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("sparse", [False, True])
@pytest.mark.parametrize("T,H", [(1, 64), (3, 192)])
@pytest.mark.parametrize("log2_ratio", [35.0, 41.0, 50.0])
def test_small_weights_are_kept(fmt, sparse, T, H, log2_ratio):
    """One strong row and 32 weak ones. An entry's sum over the heads is rounded to steps of
    2^-(62 - log2(T H)) in a list (at most 2^-52 here, half of it T times: 3 * 2^-53 against
    3 * 192 * 2^-50, 2^-10.6 of the sum; H = 64 less), a logit of -50 to 2^-19 and its fp32
    exponential to 2^-21."""
    P, w = _two_kinds(fmt, 33, [7], 1, T, H, 33 if sparse else 0, log2_ratio)
    if T > 1:
        P.q_pos.fill_(33)
        P.pos[:] = 33
    if sparse:
        P.idx = torch.arange(33, dtype=torch.int32, device="cuda").flip(0).expand(1, T, -1).contiguous()
    got = P.mass(torch.zeros((1, 33), device="cuda")).double().cpu()[0]
    den = 1 + 32 * w
    weak = np.delete(got.numpy(), 7)
    assert np.abs(weak / (T * H * w / den) - 1).max() <= 2.0 ** -10
    assert abs(float(got[7]) / (T * H / den) - 1) <= 2.0 ** -18


@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("T,H,copies", [(128, 1024, 1), (683, 192, 1), (3, 64, 4)])
def test_sums_of_whole_weights(fmt, T, H, copies):
    """Every query lists one and the same entry: all its weight, T * H in all, the most that the
    sums of a list have to hold, and exact (a weight of 2^0). Listed four times, each has a weight of
    2^-2, whose exponent is off by half a step of 3 (2^-23) and its exponential by 2^-22."""
    P, _ = _two_kinds(fmt, 5, [2], 1, T, H, copies, 1.0)
    P.q_pos.fill_(5)
    P.idx = torch.full((1, T, copies), 2, dtype=torch.int32, device="cuda")
    acc = torch.ones((1, 5), device="cuda")
    got = P.mass(acc, 0.5).cpu()[0]
    want = torch.tensor([0.5, 0.5, T * H + 0.5, 0.5, 0.5])
    assert ((got - want).abs() <= want * (0 if copies == 1 else 2.0 ** -21)).all()


# ------------------------------- no rows -------------------------------

@pytest.mark.parametrize("fmt", ["fp4", "bf16"])
@pytest.mark.parametrize("k", [0, 3])
def test_queries_without_any_row_then_with(k, fmt):
    """No entry visible, no window, no sink (padding of a batch, position -1): the sums only decay.
    Then, on the same workspace at once, queries that have rows, again and again."""
    empty = F.Problem(B=70, H=128, k=k, pages=3, page_rows=4, m=4, n_win=0, sink=False, seed=51, fmt=fmt,
                      pos=[-1] * 70)
    full = F.Problem(B=70, H=128, k=k, pages=3, page_rows=4, m=4, n_win=0, sink=False, seed=52, fmt=fmt)
    need = csa.attn_mass_workspace_size(full.p, 70, 1, full.N, 1 if k else 0)
    ws = torch.full((need,), 255, dtype=torch.uint8, device="cuda")
    acc0 = torch.rand((70, full.N), device="cuda")
    want = full.mass(acc0.clone(), 0.5)
    for _ in range(20):
        a, b = acc0.clone(), acc0.clone()
        empty.mass(a, 0.25, ws=ws)
        full.mass(b, 0.5, ws=ws)
        assert torch.equal(a, acc0 * 0.25)
        assert torch.equal(b, want)
