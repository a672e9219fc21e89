"""How streams are cut over CTAs: lists around the switch from one chunk a CTA to two, tables much
longer than what is visible (most CTAs have no rows), and pages that an eviction took."""
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


@pytest.mark.parametrize("B,H,chunks", [(1, 64, 32), (3, 64, 28), (3, 64, 30), (4, 64, 21), (4, 64, 22),
                                        (2, 128, 22), (5, 64, 16), (5, 64, 17), (6, 64, 17), (8, 64, 18)])
def test_lists_of_one_and_two_chunks_a_cta(B, H, chunks):
    """`chunks` of 64 rows: the list's, its last one row short, and two of the window."""
    P = F.Problem(B=B, H=H, k=64 * (chunks - 2) - 1, pages=70, page_rows=32, m=4, seed=70)
    F.check_attention(P.attention(), P.out64(), f"{B} x {chunks}")


@pytest.mark.parametrize("kw", [dict(B=1, pos=[0]), dict(B=1, pos=[130]), dict(B=2, pos=[128 * 70, 5]),
                                dict(B=5, H=128, pos=[128, 128 * 3, 128 * 9000, 128 * 64, 40])], ids=str)
def test_short_requests_in_long_tables(kw):
    P = F.Problem(pages=300, page_rows=32, m=128, seed=71, **kw)
    F.check_attention(P.attention(), P.out64(), str(kw))
    acc = torch.rand((P.B, P.N), device="cuda")
    check_mass(P.mass(acc.clone(), 0.9), P.mass64(acc, 0.9), acc.double().cpu().numpy(), 0.9, str(kw))


@pytest.mark.parametrize("fmt", ["fp4", "bf16", "fp8"])
def test_evicted_pages_and_entries_left_out_of_a_list(fmt):
    """Entries of evicted pages are masked like entries that the list leaves out: the same bits."""
    P = F.Problem(B=2, k=300, pages=30, page_rows=32, m=4, seed=72, fmt="bf16" if fmt == "fp8" else fmt)
    scales = None
    if fmt == "fp8":  # any bytes serve as e4m3 codes but the NaN ones
        g = np.random.default_rng(0)
        code = g.integers(0, 0x7f, size=(P.n_pages, 32, 448 + 128)).astype(np.uint8)
        code[..., 448:] = torch.randn((P.n_pages, 32, 64)).to(torch.bfloat16).view(torch.uint8).numpy()
        pool = torch.from_numpy(code).cuda()
        scales = torch.full((P.n_pages, 32), 2.0 ** -7, device="cuda")

    def attend():
        if fmt == "fp8":
            P.kv_fmt = csa.CSA_MIXED_FP8_BF16
            P.kv = csa.paged_kv(P.kv_fmt, pool, scales, P.table_d, P.n_pages, 32, P.pages)
        return P.attention()

    whole = P.idx.clone()
    gone = [0, 3, 4, 11, 29]
    e = P.idx.clone()
    e[torch.isin(P.idx // 32, torch.tensor(gone, device="cuda", dtype=torch.int32))] = -1
    assert (e != whole).any()
    P.idx = e
    want = attend()
    P.idx = whole
    P.table[:, gone] = -2
    P.refresh()
    got = attend()
    assert torch.isfinite(got.float()).all() and torch.equal(got, want)
    torch.cuda.synchronize()
    assert csa.device_error() == 0
