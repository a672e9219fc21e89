"""Refusals of the calls over 4-bit pages, the attention weight and the page eviction, and the
allocator's eviction: host checks only, no GPU (nothing is launched on any of these paths)."""
import ctypes
import os
import subprocess
import tempfile

import numpy as np
import pytest

import long_context_sparse_08_b200 as csa
from long_context_sparse_08_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # aligned, never dereferenced
INVALID, UNSUPPORTED, WORKSPACE = (csa.CSA_ERR_INVALID_ARG, csa.CSA_ERR_UNSUPPORTED,
                                   csa.CSA_ERR_WORKSPACE)


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def fp4(**kw):
    d = dict(fmt=csa.CSA_MIXED_MXFP4_BF16, pages=FAKE, scales=None, table=FAKE, n=64, rows=32, max=16)
    d.update(kw)
    return csa.CsaPagedKv(d["fmt"], d["pages"], d["scales"], d["table"], d["n"], d["rows"], d["max"])


def test_attention_over_4_bit_pages():
    L = csa.lib()
    call = lambda kv, p, ws=FAKE, n=1 << 40, B_=1: L.csa_sparse_mqa_paged(  # noqa: E731
        ctypes.byref(p), B_, 1, FAKE, FAKE, ctypes.byref(kv), FAKE, FAKE, 128, FAKE, None, None, FAKE,
        ws, n, None)
    p = csa.make_params(topk=512)
    need = csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, csa.CSA_MIXED_MXFP4_BF16, 1, 1, 512)
    assert need > 0
    assert call(fp4(), p, n=need - 1) == WORKSPACE
    assert call(fp4(), p, ws=None) == WORKSPACE
    assert call(fp4(), p, ws=FAKE + 8) == WORKSPACE
    assert call(fp4(pages=None), p) == INVALID
    assert call(fp4(pages=FAKE + 8), p) == INVALID
    assert call(fp4(table=None), p) == INVALID
    assert call(fp4(rows=0), p) == INVALID
    assert call(fp4(rows=1 << 20, max=1 << 12), p) == INVALID  # N_cap past 2^31
    for bad in (dict(rope_dims=32), dict(rope_dims=128), dict(n_heads=16), dict(c=256)):
        assert call(fp4(), csa.make_params(**bad)) == UNSUPPORTED, bad
    assert call(fp4(), p, B_=0) == csa.CSA_OK
    assert L.hca_dense_mqa_paged(ctypes.byref(csa.make_params(m=128, overlap=0)), 1, 1, FAKE, FAKE,
                                 ctypes.byref(fp4()), FAKE, 128, FAKE, None, None, FAKE, None, 0,
                                 None) == WORKSPACE
    # other formats keep their sizes
    assert csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, 0, 1, 1, 512) == \
        csa.workspace_size(p, csa.CSA_WS_SPARSE_MQA, csa.CSA_MIXED_FP8_BF16, 1, 1, 512)


@pytest.mark.parametrize("B,T,N", [(1, 1, 512), (8, 1, 32768), (1, 8192, 16384)])
def test_forward_workspace_has_room_for_either_attention(B, T, N):
    """The selection's bytes, then either the bf16 attention with its q_hat (1 KB a head) or the
    attention over 4-bit rows, which brings its own: their maximum, not their sum."""
    p = csa.make_params(topk=512)
    size = lambda entry, kdt: csa.workspace_size(p, entry, kdt, B, T, N)  # noqa: E731
    either = max(size(csa.CSA_WS_SPARSE_MQA, csa.CSA_BF16) + B * T * p.n_heads * p.c * 2,
                 size(csa.CSA_WS_SPARSE_MQA, csa.CSA_MIXED_MXFP4_BF16))
    assert size(csa.CSA_WS_FORWARD, csa.CSA_BF16) == size(csa.CSA_WS_INDEX_TOPK, csa.CSA_BF16) + either


def test_writers_of_4_bit_pages():
    L = csa.lib()
    enc = lambda p, kv: L.csa_encode_paged(  # noqa: E731
        ctypes.byref(p), csa.CSA_BF16, 0, 4, 0, FAKE, ctypes.byref(kv), None)
    assert enc(csa.make_params(), fp4()) == csa.CSA_OK  # B = 0, and no scales are asked for
    for r in (0, 16, 48, 512):
        assert enc(csa.make_params(rope_dims=r), fp4()) == INVALID, r
    app = lambda p: L.csa_state_append(  # noqa: E731
        ctypes.byref(p), 1, 0, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 1, FAKE, FAKE,
        csa.CSA_MIXED_MXFP4_BF16, FAKE, None, 8, 32, FAKE, 4, None)
    assert app(csa.make_params()) == csa.CSA_OK
    assert app(csa.make_params(rope_dims=16)) == INVALID
    comp = csa.CsaPagedKv(csa.CSA_MIXED_MXFP4_BF16, FAKE, None, FAKE, 8, 32, 4)
    assert L.csa_compress_paged(ctypes.byref(csa.make_params()), csa.CSA_BF16, 1, 16, 0, FAKE, FAKE,
                                FAKE, FAKE, FAKE, None, None, None, 1, ctypes.byref(comp),
                                None) == INVALID  # compress, then encode


def test_attention_weight():
    L = csa.lib()
    p = csa.make_params(m=128, overlap=0, topk=512)
    need = csa.attn_mass_workspace_size(p, 2, 1, 512, 0)
    assert need >= 2 * 64 * 512 * 4

    def call(kv=None, params=p, B_=2, T=1, q=FAKE, idx=None, win=FAKE, L_raw=128, pos0=None, decay=1.0,
             acc=FAKE, ws=FAKE, n=1 << 40):
        return L.csa_attn_mass_paged(ctypes.byref(params), B_, T, q, FAKE,
                                     ctypes.byref(kv or fp4()), idx, win, L_raw, pos0, None, None, decay,
                                     acc, ws, n, None)

    assert call(B_=0) == csa.CSA_OK
    assert call(T=0) == csa.CSA_OK
    assert call(n=need - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    for decay in (-0.1, 1.5, float("nan"), float("inf")):
        assert call(decay=decay) == INVALID, decay
    assert call(acc=None) == INVALID
    assert call(acc=FAKE + 4) == INVALID
    assert call(q=None) == INVALID
    assert call(idx=FAKE + 4) == INVALID
    assert call(T=2) == INVALID             # the ring serves one query per request
    assert call(L_raw=64) == INVALID        # the ring holds n_win rows
    assert call(win=None) == INVALID
    assert call(B_=65535, T=2, pos0=FAKE) == INVALID
    wide = csa.make_params(m=128, overlap=0, n_heads=128)
    assert call(params=wide, T=32769, B_=1, pos0=FAKE) == INVALID  # T * n_heads > 2^22
    assert call(params=csa.make_params(m=128, overlap=0, n_heads=8256)) == INVALID
    assert call(kv=fp4(fmt=csa.CSA_MIXED_FP8_BF16, scales=FAKE)) == UNSUPPORTED
    assert call(kv=fp4(fmt=csa.CSA_MXFP4)) == INVALID
    for bad in (dict(rope_dims=32), dict(n_heads=16), dict(c=256)):
        assert call(params=csa.make_params(**bad)) == UNSUPPORTED, bad
    assert call(params=csa.make_params(topk=4096), idx=FAKE) == INVALID
    assert csa.attn_mass_workspace_size(csa.make_params(n_heads=16), 2, 1, 512, 0) == 0
    assert csa.last_error()


def test_page_eviction():
    L = csa.lib()
    p = csa.make_params()
    need = csa.evict_pages_workspace_size(3, 100)
    assert need >= 3 * 100 * 4

    def call(B_=3, rows=32, pages=100, budget=50, first=1, last=1, ws=FAKE, n=1 << 30, **ptr):
        a = {k: ptr.get(k, FAKE) for k in ("pos", "acc", "table", "new", "kept", "entries", "evicted",
                                            "counts")}
        return L.csa_evict_pages(ctypes.byref(p), B_, rows, pages, a["pos"], a["acc"], a["table"], budget,
                                 first, last, a["new"], a["kept"], a["entries"], a["evicted"],
                                 a["counts"], ws, n, None)

    assert call(B_=0) == csa.CSA_OK
    assert call(B_=-1) == INVALID
    assert call(rows=0) == INVALID
    assert call(pages=0) == INVALID
    assert call(rows=1 << 16, pages=1 << 16) == INVALID
    assert call(budget=0, first=0, last=0) == INVALID
    assert call(first=-1) == INVALID
    assert call(first=30, last=21) == INVALID  # more than the budget
    assert call(budget=(1 << 31) - 1) == INVALID
    for name in ("pos", "acc", "table", "new", "kept", "evicted", "counts"):
        assert call(**{name: None}) == INVALID, name
    assert call(entries=FAKE + 4) == INVALID
    assert call(n=need - 1) == WORKSPACE
    assert call(ws=None) == WORKSPACE
    assert call(ws=FAKE + 8) == WORKSPACE
    assert csa.evict_pages_workspace_size(1, 0) == 0


def test_allocator_evicts_single_pages():
    a = csa.PageAlloc(12, 2, 8)
    a.reserve(0, 6)
    a.reserve(1, 4)
    assert a.free_pages == 2
    before = np.array(a.table)
    for bad in ([5, 4], [3, 3], [6], [-1], [0, 7]):  # not ascending, twice, not mapped
        with pytest.raises(csa.CsaError):
            a.evict(0, bad)
        assert (a.table == before).all() and a.free_pages == 2  # all or nothing
    with pytest.raises(csa.CsaError):
        a.evict(2, [0])
    a.evict(0, [1, 4])
    assert a.free_pages == 4 and list(a.table[0, :6]) == [0, -2, 2, 3, -2, 5]
    with pytest.raises(csa.CsaError):
        a.evict(0, [1])  # already gone
    a.evict(0, [])
    assert a.mapped(0) == 6
    a.reserve(0, 8)  # the evicted pages are not mapped again
    assert list(a.table[0]) == [0, -2, 2, 3, -2, 5, 10, 11]
    a.reserve(1, 6)  # they serve another request
    assert list(a.table[1, :6]) == [6, 7, 8, 9, 1, 4] and a.free_pages == 0
    a.release(0)
    assert a.free_pages == 6 and (a.table[0] == -1).all()
    assert csa.lib().csa_page_alloc_evict(None, 0, None, 0) == INVALID


HOST = r'''
#include <cstdio>
#include <cmath>
#include "state_append.cuh"
int main() {
  float v;
  while (std::scanf("%f", &v) == 1) {
    const int E = csa::state::kv_mx_exponent(std::fabs(v));
    std::printf("%d %u\n", E, csa::state::e2m1_code(v / csa::state::pow2f(E)));
  }
  std::printf("%zu %zu %zu\n", csa::state::fp4_row_bytes(512, 64), csa::state::fp4_rope_offset(512, 64),
              csa::state::fp4_row_bytes(256, 128));
}
'''


def test_encoding_arithmetic_on_the_host():
    """Exponent and code of single values (each its own block's largest), from zero to infinity."""
    from tests import fp4_values as V

    vals = [0.0, 1.0, -1.0, 3.9, 4.0, 6.0, 7.0, 1e-9, 2.0 ** -14, 2.0 ** -16, 49152.0, 49153.0, 65504.0,
            65536.0, 1e30, float("inf"), -5.0, 0.1, 6.0 * 2 ** -16, 2.0 ** -126]
    with tempfile.TemporaryDirectory() as d:
        src, exe = os.path.join(d, "t.cu"), os.path.join(d, "t")
        open(src, "w").write(HOST)
        subprocess.check_call([B.nvcc(), "-std=c++17", "-I", B.CSRC, "-I", os.path.join(ROOT, "include"),
                               src, "-o", exe])
        out = subprocess.run([exe], input="\n".join(map(repr, vals)), capture_output=True, text=True,
                             check=True).stdout.split("\n")
    for v, line in zip(vals, out):
        E, code = map(int, line.split())
        assert -14 <= E <= 13
        assert (E, code) == V.exponent_and_code(v), v
    assert out[len(vals)].split() == ["368", "240", "336"]
