"""The workspace that csa_forward and csa_forward_paged demand: what their own attention takes, not
what an attention over another format of KV rows would."""
import ctypes
import re

import pytest

import long_context_sparse_08_b200 as csa
from long_context_sparse_08_b200 import build as B

FAKE = 0x10000  # aligned, never dereferenced: a call without a workspace launches nothing


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def _asked(call):
    assert call() == csa.CSA_ERR_WORKSPACE
    return int(re.search(r"needs (\d+) workspace bytes", csa.last_error()).group(1))


def _selection(p, b, t, n):
    return csa.workspace_size(p, csa.CSA_WS_INDEX_TOPK, csa.CSA_BF16, b, t, n)


def _bf16_attention(p, b, t, n):
    """The attention over bf16 rows and its q_hat, 2 bytes a value."""
    return csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, csa.CSA_BF16, b, t, n) + \
        b * t * p.n_heads * p.c * 2


SIZES = [(1, 1, 8192, 128, 1024), (4, 1, 262144, 128, 1024), (8, 1, 32768, 64, 512), (1, 1, 512, 64, 64),
         (2, 3, 4096, 64, 2048), (1, 2048, 16384, 64, 512), (3, 1, 640, 192, 7)]


@pytest.mark.parametrize("b,t,n,heads,k", SIZES)
def test_forward(b, t, n, heads, k):
    p = csa.make_params(n_heads=heads, topk=k)
    a = csa.forward_args(idx_dtype=csa.CSA_BF16, qI=FAKE, w=FAKE, KI=FAKE, q=FAKE, q_pos=FAKE,
                         kv_cache=FAKE, N_cap=n, win_kv=FAKE, L_raw=128 + t, win_pos0=FAKE, out_idx=FAKE,
                         out=FAKE)
    asked = _asked(lambda: csa.lib().csa_forward(ctypes.byref(p), csa.CSA_BF16, b, t, ctypes.byref(a),
                                                 None, 0, None))
    assert asked == _selection(p, b, t, n) + _bf16_attention(p, b, t, n)
    assert asked <= csa.workspace_size(p, csa.CSA_WS_FORWARD, csa.CSA_BF16, b, t, n)


@pytest.mark.parametrize("fmt", [csa.CSA_BF16, csa.CSA_MIXED_FP8_BF16, csa.CSA_MIXED_MXFP4_BF16])
@pytest.mark.parametrize("b,t,n,heads,k", SIZES)
def test_forward_paged(b, t, n, heads, k, fmt):
    p = csa.make_params(n_heads=heads, topk=k)
    kv = csa.CsaPagedKv(fmt, FAKE, FAKE, FAKE, 9, 32, n // 32)
    keys = csa.CsaPagedKv(csa.CSA_BF16, FAKE, None, FAKE, 9, 128, n // 128)
    asked = _asked(lambda: csa.lib().csa_forward_paged(
        ctypes.byref(p), b, t, ctypes.byref(kv), ctypes.byref(keys), 0, FAKE, None, FAKE, FAKE, None, FAKE,
        FAKE, 128 + t, FAKE, None, FAKE, None, FAKE, None, 0, None))
    own = csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, fmt, b, t, n) \
        if fmt == csa.CSA_MIXED_MXFP4_BF16 else _bf16_attention(p, b, t, n)
    assert asked == _selection(p, b, t, n) + own
    assert asked <= csa.workspace_size(p, csa.CSA_WS_FORWARD, csa.CSA_BF16, b, t, n)


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["edge_decode_bf16_tc", "mid_decode_mxfp4_sel", "mid_prefill_bf16_tc"])
def test_forward_in_its_own_workspace(name):
    """With exactly the bytes demanded and guard bytes behind them: the same results."""
    import torch

    from long_context_sparse_08_b200 import runner as R
    import tests.parity_util as U

    s, inp = U.inputs(name)
    dev = R.upload(inp, s)
    full, own = R.Step(s, dev), R.Step(s, dev)
    p = own.p
    own.ws_bytes = _selection(p, s.B, s.T, s.n_cap) + _bf16_attention(p, s.B, s.T, s.n_cap)
    assert own.ws_bytes <= full.ws_bytes
    own.ws = torch.full((own.ws_bytes + 4096,), 0x5A, dtype=torch.uint8, device="cuda")
    full()
    own()
    torch.cuda.synchronize()
    assert torch.equal(full.out, own.out) and torch.equal(full.out_idx, own.out_idx)
    assert (own.ws[own.ws_bytes:] == 0x5A).all()
    assert csa.device_error() == 0
