"""Plain float64 forms and input makers for the 4-bit KV rows (CSA_MIXED_MXFP4_BF16), the
attention over them, the attention weight per cache entry and the page eviction. Written from
the formats' and operators' definitions; shares no code with the library's kernels."""
import math

import numpy as np
import torch

import long_context_sparse_08_b200 as csa
from long_context_sparse_08_b200 import workloads as W

from tests.fp4_values import C, NOPE, R, WIN, decode_rows, encode_rows, row_bytes  # noqa: F401


class Problem:
    """A batch of queries over paged caches: device tensors, and float64 results on request."""

    def __init__(self, *, B, T=1, H=64, k=0, pages=8, page_rows=8, m=128, pos=None, fmt="fp4",
                 sink=True, weight=False, n_win=WIN, ring=None, seed=0, base=10000.0, scale=0.0):
        g = np.random.default_rng(seed)
        self.B, self.T, self.H, self.k, self.m, self.fmt = B, T, H, k, m, fmt
        self.pages, self.page_rows, self.N, self.n_win = pages, page_rows, pages * page_rows, n_win
        self.base = base
        self.p = csa.make_params(m=m, overlap=1 if k else 0, n_heads=H, topk=max(k, 1),
                                 n_win=n_win, rope_base=base, sm_scale=scale)
        self.scale = scale if scale > 0 else 1 / math.sqrt(C)
        pos = np.asarray(pos if pos is not None else [m * self.N] * B, np.int64)
        self.pos = pos[:, None] + np.arange(T) if pos.ndim == 1 else pos
        ring = (T == 1) if ring is None else ring
        self.n_pages = B * pages + 3
        self.table = g.permutation(self.n_pages)[:B * pages].reshape(B, pages).astype(np.int32)
        x = g.standard_normal((self.n_pages * page_rows, C)).astype(np.float32)
        x += (g.random((len(x), 1)) ** 4 * g.standard_normal(C)).astype(np.float32)
        x /= np.sqrt((x * x).mean(-1, keepdims=True))
        if fmt == "fp4":
            pool = encode_rows(x)
            self.rows64 = decode_rows(pool)
            self.pool = torch.from_numpy(pool.reshape(self.n_pages, page_rows, -1)).cuda()
        else:
            bits = W.f32_to_bf16_bits(x)
            self.rows64 = W.bf16_bits_to_f32(bits).astype(np.float64)
            self.pool = torch.from_numpy(x).to(torch.bfloat16).view(self.n_pages, page_rows, C).cuda()
        self.q = torch.from_numpy(g.standard_normal((B, T, H, C)).astype(np.float32) * 2).to(
            torch.bfloat16).cuda()
        self.sink = torch.from_numpy(g.standard_normal(H).astype(np.float32)).cuda() if sink else None
        self.w = torch.from_numpy((1 + .2 * g.standard_normal(C)).astype(np.float32)).to(
            torch.bfloat16).cuda() if weight else None
        self.L = n_win if ring else n_win - 1 + T + 3
        self.win = self.win_pos0 = None
        if n_win:
            wv = g.standard_normal((B, self.L, C)).astype(np.float32)
            self.win = torch.from_numpy(wv).to(torch.bfloat16).cuda()
            if not ring:
                self.win_pos0 = torch.from_numpy(
                    np.maximum(self.pos[:, 0] - (n_win - 1) - 2, 0)).cuda()
        else:
            self.L = 0
        self.idx = None
        if k:
            idx = np.full((B, T, k), -1, np.int32)
            for b in range(B):
                for t in range(T):
                    vis = min(max(self.pos[b, t], 0) // m, self.N)
                    n = min(k, vis)
                    idx[b, t, :n] = g.permutation(vis)[:n]
            self.idx = torch.from_numpy(idx).cuda()
        self.q_pos = torch.from_numpy(np.ascontiguousarray(self.pos)).cuda()
        self.refresh()

    def refresh(self):
        """Page table to the device (after a test changed it)."""
        self.table_d = torch.from_numpy(self.table).cuda()
        fmt = csa.CSA_MIXED_MXFP4_BF16 if self.fmt == "fp4" else csa.CSA_BF16
        self.kv_fmt = fmt
        self.kv = csa.paged_kv(fmt, self.pool, None, self.table_d, self.n_pages, self.page_rows,
                               self.pages)

    def attention(self, out=None, ws=None, stream=None):
        entry = csa.CSA_WS_SPARSE_MQA if self.k else csa.CSA_WS_HCA_MQA
        need = csa.workspace_size(self.p, entry, self.kv_fmt, self.B, self.T, self.N)
        if out is None:
            out = torch.full((self.B, self.T, self.H, C), float("nan"), dtype=torch.bfloat16,
                             device="cuda")
        if ws is None:
            ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
        if self.k:
            csa.csa_sparse_mqa_paged(self.p, self.B, self.T, self.q, self.q_pos, self.kv, self.idx,
                                     self.win, self.L, self.win_pos0, self.sink, self.w, out, ws,
                                     need, stream)
        else:
            csa.hca_dense_mqa_paged(self.p, self.B, self.T, self.q, self.q_pos, self.kv, self.win,
                                    self.L, self.win_pos0, self.sink, self.w, out, ws, need, stream)
        return out

    def mass(self, acc, decay=1.0, ws=None, stream=None):
        need = csa.attn_mass_workspace_size(self.p, self.B, self.T, self.N, 1 if self.k else 0)
        if ws is None:
            ws = torch.full((max(need, 16),), 255, dtype=torch.uint8, device="cuda")
        csa.csa_attn_mass_paged(self.p, self.B, self.T, self.q, self.q_pos, self.kv, self.idx,
                                self.win, self.L, self.win_pos0, self.sink, self.w, decay, acc, ws,
                                need, stream)
        return acc

    # ---- float64 ----
    def _rope(self, x, pos, sign):
        f = self.base ** (-np.arange(0, R, 2) / R)
        c, s = np.cos(pos * f), sign * np.sin(pos * f)
        y = x.copy()
        a, b = x[..., NOPE::2], x[..., NOPE + 1::2]
        y[..., NOPE::2], y[..., NOPE + 1::2] = a * c - b * s, a * s + b * c
        return y

    def query64(self, b, t):
        """(entries, weights [H, entries], out [H, 512]) of query (b, t)."""
        pos = int(self.pos[b, t])
        q = self.q[b, t].double().cpu().numpy()
        q = q / np.sqrt((q * q).mean(-1, keepdims=True) + 1e-6)
        if self.w is not None:
            q = q * self.w.double().cpu().numpy()
        q = self._rope(q, pos, 1.0)
        if self.k:
            e = self.idx[b, t].cpu().numpy().astype(np.int64)
            e = e[(e >= 0) & (e < self.N)]
        else:
            e = np.arange(min(max(pos, 0) // self.m, self.N))
        pg = self.table[b, e // self.page_rows]
        e, pg = e[(pg >= 0) & (pg < self.n_pages)], pg[(pg >= 0) & (pg < self.n_pages)]
        rows = self.rows64[pg.astype(np.int64) * self.page_rows + e % self.page_rows]
        tok = np.arange(max(0, pos - self.n_win + 1), pos + 1) if self.n_win else np.arange(0)
        if len(tok):
            at = tok % self.L if self.win_pos0 is None else tok - int(self.win_pos0[b])
            at = at[(at >= 0) & (at < self.L)]
            rows = np.concatenate((rows, self.win[b].double().cpu().numpy()[at]))
        z = q @ rows.T * self.scale
        sink = self.sink.double().cpu().numpy() if self.sink is not None else np.full(self.H, -np.inf)
        top = np.maximum(z.max(-1, initial=-np.inf), sink)
        top = np.where(np.isfinite(top), top, 0.0)
        ex = np.exp(z - top[:, None])
        den = ex.sum(-1) + np.exp(sink - top)
        p = ex / np.where(den > 0, den, 1.0)[:, None]
        return e, p[:, :len(e)], self._rope(p @ rows, pos, -1.0)

    def out64(self):
        return np.stack([[self.query64(b, t)[2] for t in range(self.T)] for b in range(self.B)])

    def mass64(self, acc, decay):
        acc = acc.double().cpu().numpy() * decay
        for b in range(self.B):
            for t in range(self.T):
                e, p, _ = self.query64(b, t)
                np.add.at(acc[b], e, p.sum(0))
        return acc


def check_attention(got, ref, what="", scale=1 / math.sqrt(C)):
    """The output is rounded to bf16 once: half a step is 2^-8 of the value, at most
    2^-8 / sqrt(3) = 2.26e-3 rms. q_hat and P are f16, half a step 2^-11, at most 2.8e-4 rms.
    Rounding q_hat moves a logit by s = 2.8e-4 * scale * sqrt(sum q_hat_i^2 k_i^2) rms, and
    with q_hat and k of unit rms the root is sqrt(512): 2.8e-4 at the default scale
    1/sqrt(512), more at a larger one. A weight is then off by the factor e^(s x), x normal, in
    the numerator and in the sum. So the relative rms is at most 2.26e-3, 2.8e-4 and 2 s in
    quadrature (a tenth is added). One value is off by 2^-8 of itself, 1e-2 of its head's rms, and
    what the logits do: between two rows a and b of weights p and 1 - p the difference of the
    logits is off by sqrt(2) s x, and dim d of the output by p (1 - p) sqrt(2) s x (k_a - k_b)_d =
    p (1 - p) 2 s x y with x and y normal, while the head's rms is sqrt(p^2 + (1 - p)^2): at most
    0.71 s |x y| of it, at p = 1/2. |x y| passes t with a probability below e^-t, so among 10^7
    values it stays below 16: 11.4 s."""
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all(), what
    s = 2.8e-4 * scale * math.sqrt(C)
    d = got - ref
    n = np.sqrt((ref * ref).sum())
    rel = np.sqrt((d * d).sum()) / n if n else np.abs(d).max(initial=0.0)
    assert rel <= 1.1 * math.sqrt(2.26e-3 ** 2 + 2.8e-4 ** 2 + 4 * s * s), \
        f"{what}: relative rms {rel:.2e}"
    rms = np.sqrt((ref * ref).mean(-1, keepdims=True))
    bad = np.abs(d) > 2.0 ** -8 * np.abs(ref) + (1e-2 + 11.4 * s) * rms
    assert not bad.any(), f"{what}: {bad.sum()} values off, worst {np.abs(d).max():.2e}"
