"""Attention over 4-bit rows where most of the rows have weights far below the largest."""
import math

import numpy as np
import pytest
import torch

import long_context_sparse_08_b200 as csa
from tests.fp4_values import C, encode_rows

pytestmark = [pytest.mark.gpu]


@pytest.mark.parametrize("B,strong", [
    (148, [0]),                                    # a CTA a request, its first row the strong one
    (148, [262143]),                               # the maximum raised by the last row
    (1, list(range(0, 262144, 4096))),             # 32 splits, strong rows in each
], ids=["first", "last", "splits"])
def test_many_rows_of_small_weight(B, strong):
    """262144 entries: weak rows hold 1 in dims 128-447, strong rows 1 in dims 0-127, and the query
    (the same in all heads) is 2 in dims 0-127 after its normalisation. So a weak row's weight is
    2^-26.5 of a strong one's, and dims 128-447 of the output are the weak rows' share: 2^-8.5 in all
    for one strong row.

    Tolerance, relative: the output's rounding to bf16 2^-8; P in f16, where a strong row's is at
    least 2^8.5 and a weak row's 2^-18 (half a step there: 2^-25, 2^-7 of it, but 2^-18 is itself a
    step's multiple and P is 1e-5 beside it): 2^-8 at most; a strong row's P 2^-11; fp32 sums of 4096
    chunks, each addition cut off at 2^-23: 2^-12 on average; and q_hat = 2 (1 - 5e-7) is 2 in f16
    (5e-7 * 18.4 of a weight)."""
    n, page_rows = 262144, 4096
    pages = n // page_rows
    weak, strong_row = np.zeros((1, C), np.float32), np.zeros((1, C), np.float32)
    weak[0, 128:448] = 1
    strong_row[0, :128] = 1
    pool = torch.from_numpy(encode_rows(weak)).cuda().expand(n, -1).contiguous()
    pool[torch.tensor(strong, device="cuda")] = torch.from_numpy(encode_rows(strong_row)).cuda()
    log2_ratio = 26.5
    p = csa.make_params(m=4, overlap=0, n_heads=64, n_win=0,
                        sm_scale=log2_ratio * math.log(2) / 256)
    table = torch.arange(pages, dtype=torch.int32, device="cuda").expand(B, -1).contiguous()
    kv = csa.paged_kv(csa.CSA_MIXED_MXFP4_BF16, pool.view(pages, page_rows, -1), None, table, pages,
                      page_rows, pages)
    q = torch.zeros((B, 1, 64, C), dtype=torch.bfloat16, device="cuda")
    q[..., :128] = 0.75
    q_pos = torch.full((B, 1), 4 * n, dtype=torch.int64, device="cuda")
    need = csa.workspace_size(p, csa.CSA_WS_HCA_MQA, csa.CSA_MIXED_MXFP4_BF16, B, 1, n)
    ws = torch.empty((need,), dtype=torch.uint8, device="cuda")
    out = torch.empty((B, 1, 64, C), dtype=torch.bfloat16, device="cuda")
    csa.hca_dense_mqa_paged(p, B, 1, q, q_pos, kv, None, 0, None, None, None, out, ws, need)
    # 64 bits: weights relative to a strong row's
    z = 256 / math.sqrt(1 + 1e-6 / (0.75 ** 2 / 4)) * p.sm_scale
    w = math.exp(-z) * (n - len(strong))
    got = out.double().cpu()
    share = w / (w + len(strong))
    tol = 2.0 ** -8 + 2.0 ** -8 + 2.0 ** -10
    assert (got[..., 128:448] / share - 1).abs().max() <= tol
    assert (got[..., :128] / (1 - share) - 1).abs().max() <= 2.0 ** -8 + 2.0 ** -10
    assert (got[..., 448:] == 0).all()
    assert csa.device_error() == 0
