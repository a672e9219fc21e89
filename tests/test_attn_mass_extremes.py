"""The attention weight per entry at the ends of its range: rows that are not numbers."""
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
