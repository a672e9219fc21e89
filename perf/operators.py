"""Cases of the operators that serve a long context on a small cache: attention over KV entries
held in about four bits, the attention weight that each cache entry has received, and the
choice of the cache pages to evict by that weight.

`run` computes a case in elementary torch operations, or, with `own` set, by the library's
calls. Formulas (one request; a query at position t, head h, c = 512 values, r = 64 RoPE dims):

  q_hat = RoPE_t(RMSNorm(q) * w)          rows = the listed or visible entries, then the window
  z_j   = q_hat . row_j / sqrt(c)         p_j = e^{z_j} / (sum_j e^{z_j} + e^{sink_h})
  out   = RoPE_{-t}(sum_j p_j row_j)
  acc_e = decay * acc_e + sum over queries and heads of p_e
  evict: page score = largest acc of its entries; the first and last pages stay, the best
         scored others fill the budget (equal scores: the lower page stays).

A cache row of the 4-bit format is 368 bytes: 448 e2m1 codes (element 2j in the low nibble),
14 e8m0 exponents (one per 32 values; 2 bytes of padding) and the 64 RoPE values as bf16.
"""
import math

import torch

own = False

C, R, NOPE, WIN = 512, 64, 448, 128
ROW_BYTES = 368
GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
SCALE = 1.0 / math.sqrt(C)


# --------------------------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------------------------

def listed():
    def attn(name, B, T, H, k, N, ctx, page_rows, **kw):
        d = dict(name=name, op="attn", fmt="fp4", B=B, T=T, H=H, k=k, N=N, ctx=ctx,
                 page_rows=page_rows, sink=True, weight=False)
        d.update(kw)
        return d

    def mass(name, B, T, H, k, N, ctx, page_rows, fmt, decay, **kw):
        return attn(name, B, T, H, k, N, ctx, page_rows, op="mass", fmt=fmt, decay=decay, **kw)

    def evict(name, B, N, ctx, page_rows, budget, first, last):
        return dict(name=name, op="evict", B=B, N=N, ctx=ctx, page_rows=page_rows,
                    budget=budget, first=first, last=last)

    return [
        # one request just past its prompt: a short dense list, where latency is all
        attn("dense_small", 1, 1, 64, 0, 64, 5200, 1),
        # dense HCA decode at 1M tokens, one-entry pages, the batch of the library's benchmark
        attn("dense_1m", 16, 1, 64, 0, 8192, 1048576, 1),
        # dense decode of ragged requests, 128 heads, the list ends inside a page
        attn("dense_ragged", 7, 1, 128, 0, 4104, 525389, 8, weight=True),
        # sparse CSA decode at 131k tokens, 64 heads
        attn("sparse_131k", 8, 1, 64, 512, 32768, 131072, 32),
        # sparse CSA decode at 1M tokens, 128 heads
        attn("sparse_1m", 4, 1, 128, 1024, 262144, 1048576, 32),
        # a prefill chunk: every query its own selected entries
        attn("sparse_prefill", 1, 2048, 64, 512, 16384, 57344, 32),
        # weight per entry of the dense decode at 1M tokens (what eviction is decided from)
        mass("mass_dense_1m", 16, 1, 64, 0, 8192, 1048576, 1, "fp4", 0.99),
        # the same over bf16 pages, few short requests
        mass("mass_dense_bf16", 3, 1, 64, 0, 600, 76900, 8, "bf16", 1.0, weight=True),
        # weight of the selected entries of a sparse decode, several tokens verified at once
        mass("mass_sparse", 4, 4, 128, 1024, 65536, 262144, 32, "fp4", 0.95),
        # half of the one-entry pages of sixteen 1M-token requests go
        evict("evict_1m", 16, 8192, 1048576, 1, 4096, 4, 64),
        # pages of 32 entries at 1M tokens
        evict("evict_pages", 4, 262144, 1048573, 32, 2000, 1, 33),
        # the smallest eviction: one request a little over its budget
        evict("evict_small", 1, 600, 76900, 1, 512, 4, 16),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("sparse", "sparse", "dense", "dense", "mass", "mass", "evict"))
    if op == "evict":
        page_rows = rng.choice((1, 2, 8, 32))
        N = page_rows * _log_int(rng, 16, min(8192, 262144 // page_rows))
        B = _log_int(rng, 1, 16)
        pages = N // page_rows
        m = 128 if page_rows < 32 else 4
        first = rng.randint(0, min(8, pages // 8))
        last = rng.randint(1, max(1, pages // 8))
        budget = rng.randint(first + last, pages)
        return dict(op="evict", B=B, N=N, ctx=max(1, int(N * m * rng.uniform(0.5, 1.05))),
                    page_rows=page_rows, budget=budget, first=first, last=last)
    is_mass = op == "mass"
    H = rng.choice((64, 128))
    sparse = op == "sparse" or (is_mass and rng.random() < 0.5)
    page_rows = 32 if sparse else rng.choice((1, 2, 8, 32))
    if sparse:
        k = _log_int(rng, 1, 2048)
        N = 32 * _log_int(rng, 2, 4096)
        B = _log_int(rng, 1, 16)
        T = rng.choice((1, 1, 1, _log_int(rng, 2, 16), _log_int(rng, 32, 1024)))
        T = min(T, 16) if is_mass else T
        while B * T * (k + WIN) * H > 2048 * 640 * 64 * (0.2 if is_mass else 1):
            B, T = max(1, B // 2), max(1, T // 2)
        ctx = max(1, int(4 * N * rng.uniform(0.05, 1.05)))
    else:
        k = 0
        N = page_rows * _log_int(rng, 1, 8192 // page_rows)
        B = _log_int(rng, 1, 16)
        T = rng.choice((1, 1, 1, rng.randint(2, 5)))
        while B * T * (N + WIN) * H > 16 * 8320 * 64:
            B, T = max(1, B // 2), max(1, T - 1)
        ctx = max(1, int(128 * N * rng.uniform(0.05, 1.05)))
    d = dict(op="mass" if is_mass else "attn", fmt=rng.choice(("fp4", "bf16")) if is_mass else "fp4",
             B=B, T=T, H=H, k=k, N=N, ctx=ctx, page_rows=page_rows,
             sink=rng.random() < 0.7, weight=rng.random() < 0.5)
    if is_mass:
        d["decay"] = rng.choice((1.0, 0.99, 0.9))
    return d


def _m(case):
    if case["op"] == "evict":
        return 4 if case["page_rows"] == 32 else 128
    return 4 if case["k"] else 128


def _positions(case):
    """Position of each request's first query: ragged, the first request the longest."""
    B = case["B"]
    return [max(0, case["ctx"] - case.get("T", 1) - (b * 37 * case["ctx"]) // (100 * max(B, 8)))
            for b in range(B)]


def work(case):
    if case["op"] == "evict":
        pages = case["N"] // case["page_rows"]
        B = case["B"]
        ints = 3 * pages + case["budget"] * (1 + case["page_rows"]) + 2
        return {"bytes": 4.0 * B * (case["N"] + ints), "flops": 0.0}
    B, T, H, k, N, m = case["B"], case["T"], case["H"], case["k"], case["N"], _m(case)
    row_bytes = ROW_BYTES if case["fmt"] == "fp4" else 2 * C
    rows = entries = wins = 0
    for p0 in _positions(case):
        vis = [min((p0 + i) // m, N) for i in range(T)]
        per = [min(v, k) if k else v for v in vis]
        rows += sum(per) + sum(min(p0 + i + 1, WIN) for i in range(T))
        entries += min(sum(per), max(vis)) if k else max(vis)
        wins += min(p0 + T, WIN + T - 1)
    b = B * T * H * C * 2 + entries * row_bytes + wins * C * 2 + (4 * B * T * k)
    b += 4 * math.ceil(entries / case["page_rows"])
    if case["op"] == "attn":
        return {"bytes": float(b + B * T * H * C * 2), "flops": 4.0 * H * C * rows}
    return {"bytes": float(b + 8 * B * N), "flops": 2.0 * H * C * rows}


# --------------------------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------------------------

def _encode(x):
    """Rows [n, 512] fp32 -> [n, 368] bytes of the 4-bit format."""
    blk = x[:, :NOPE].reshape(-1, 14, 32)
    amax = blk.abs().amax(-1)
    e = torch.frexp(amax.clamp_min(1e-30))[1] - 3
    e = e.clamp(-14, 13)
    v = (blk / torch.exp2(e.float()).unsqueeze(-1)).reshape(-1, NOPE)
    mids = torch.tensor((0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0), device=x.device)
    code = torch.bucketize(v.abs().clamp_max(6.0), mids)
    code = torch.where((v < 0) & (code > 0), code + 8, code).to(torch.uint8)
    out = torch.zeros((x.shape[0], ROW_BYTES), dtype=torch.uint8, device=x.device)
    out[:, :NOPE // 2] = code[:, 0::2] | (code[:, 1::2] << 4)
    out[:, 224:238] = (e + 127).to(torch.uint8)
    out[:, 240:] = x[:, NOPE:].to(torch.bfloat16).contiguous().view(torch.uint8)
    return out


def _decode(b):
    """[..., 368] bytes -> [..., 512] fp32 (exact)."""
    grid = torch.tensor(GRID + tuple(-g for g in GRID), device=b.device)
    codes = torch.stack((b[..., :224] & 15, b[..., :224] >> 4), -1).flatten(-2).long()
    v = grid[codes].unflatten(-1, (14, 32))
    v = v * torch.exp2(b[..., 224:238].float() - 127.0).unsqueeze(-1)
    rope = b[..., 240:].contiguous().view(torch.bfloat16).float()
    return torch.cat((v.flatten(-2), rope), -1)


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed) * 7919 + 13)
    return g


def prepare(case, seed):
    g = _generator(seed)
    dev = "cuda"
    B, N, pr = case["B"], case["N"], case["page_rows"]
    m, pages = _m(case), N // pr
    st = dict(case=case)
    if case["op"] == "evict":
        u = torch.rand((B, N), generator=g, device=dev)
        st["acc"] = (-torch.log1p(-u)) ** 4  # few entries hold most of the weight
        n_pages = B * pages + 3
        st["table"] = torch.randperm(n_pages, generator=g, device=dev)[:B * pages].to(
            torch.int32).view(B, pages).contiguous()
        st["pos"] = torch.tensor([p for p in _positions(case)], dtype=torch.int64, device=dev)
        return st

    T, H, k = case["T"], case["H"], case["k"]
    st["pos_host"] = _positions(case)
    pos0 = torch.tensor(st["pos_host"], dtype=torch.int64, device=dev)
    st["q_pos"] = (pos0[:, None] + torch.arange(T, device=dev)).contiguous()
    topic = torch.randn((B, 1, C), generator=g, device=dev)  # what a request is about

    # entries: normalised rows, some of them strongly on the request's topic
    n_pages = B * pages + 3
    perm = torch.randperm(n_pages, generator=g, device=dev)[:B * pages].to(torch.int32)
    st["table"] = perm.view(B, pages).contiguous()
    width = ROW_BYTES if case["fmt"] == "fp4" else 2 * C
    pool = torch.zeros((n_pages, pr, width), dtype=torch.uint8, device=dev)
    for b in range(B):
        on = torch.rand((N, 1), generator=g, device=dev) ** 6
        x = torch.randn((N, C), generator=g, device=dev) + on * topic[b]
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True))
        rows = _encode(x) if case["fmt"] == "fp4" else \
            x.to(torch.bfloat16).view(torch.uint8)
        pool[st["table"][b].long()] = rows.view(pages, pr, width)
    st["pool"] = pool if case["fmt"] == "fp4" else pool.view(torch.bfloat16)

    q = torch.randn((B, T, H, C), generator=g, device=dev)
    q = q + torch.rand((B, T, H, 1), generator=g, device=dev) * topic[:, None]
    st["q"] = q.to(torch.bfloat16)
    st["sink"] = torch.randn((H,), generator=g, device=dev) if case["sink"] else None
    st["q_rms_w"] = (1 + 0.1 * torch.randn((C,), generator=g, device=dev)).to(torch.bfloat16) \
        if case["weight"] else None
    # window rows, normalised: the decode ring (position p in row p mod 128), or a linear
    # buffer that starts 127 tokens before the first query
    L = WIN if T == 1 else WIN - 1 + T
    w = torch.randn((B, L, C), generator=g, device=dev) + 0.3 * topic
    st["win"] = (w * torch.rsqrt(w.square().mean(-1, keepdim=True))).to(torch.bfloat16)
    st["win_pos0"] = None if T == 1 else (pos0 - (WIN - 1)).clamp_min(0)
    if k:
        # distinct visible entries per query in no particular order, -1 where there are fewer:
        # e -> (e * mult + shift) mod n over the n visible ones, mult prime to every n
        vis = (st["q_pos"] // m).clamp_max(N)
        j = torch.arange(k, device=dev, dtype=torch.int64)
        shift = torch.randint(0, 1 << 30, (B, T, 1), generator=g, device=dev)
        n = vis[..., None].clamp_min(1)
        e = (j * 1000003 + shift) % n
        st["idx"] = torch.where(j < vis[..., None], e, -1).to(torch.int32).contiguous()
    if case["op"] == "mass":
        u = torch.rand((B, N), generator=g, device=dev)
        st["acc"] = 0.05 * (-torch.log1p(-u)) ** 2
    return st


# --------------------------------------------------------------------------------------------
# the plain form
# --------------------------------------------------------------------------------------------

def _rotate(x, pos, sign):
    """Adjacent pairs of the last 64 values turned by sign * pos * 10000^(-2p/64); the angles
    of far positions need 64 bits. x [B, T, H, 512] fp32, pos [B, T]."""
    p = torch.arange(R // 2, device=x.device, dtype=torch.float64)
    ang = pos.double()[..., None] * 10000.0 ** (-2.0 * p / R)
    cs, sn = torch.cos(ang).float()[:, :, None], sign * torch.sin(ang).float()[:, :, None]
    a, b = x[..., NOPE::2], x[..., NOPE + 1::2]
    y = torch.stack((a * cs - b * sn, a * sn + b * cs), -1).flatten(-2)
    return torch.cat((x[..., :NOPE], y), -1)


def _logits(st):
    """Logits of the entry rows and of the window rows, their rows, and the masks."""
    case = st["case"]
    B, T, N, k, pr = case["B"], case["T"], case["N"], case["k"], case["page_rows"]
    q = st["q"].float()
    q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + 1e-6)
    if st["q_rms_w"] is not None:
        q = q * st["q_rms_w"].float()
    q = _rotate(q, st["q_pos"], 1.0)
    vis = (st["q_pos"] // _m(case)).clamp_max(N)
    table = st["table"].long()
    if k:
        e = st["idx"].long()
        live = e >= 0
        e = e.clamp_min(0)
        bi = torch.arange(B, device=e.device)[:, None, None]
        rows = st["pool"][table[bi, e // pr], e % pr]
        rows = _decode(rows) if case["fmt"] == "fp4" else rows.float()
        z = torch.einsum("bthc,btkc->bthk", q, rows)
    else:
        n = min(N, max(st["pos_host"]) + T)
        rows = st["pool"][table].flatten(1, 2)[:, :n]
        rows = _decode(rows) if case["fmt"] == "fp4" else rows.float()
        live = torch.arange(n, device=q.device) < vis[..., None]
        z = torch.einsum("bthc,bkc->bthk", q, rows)
    # window tokens t - 127 .. t
    p = st["q_pos"][..., None] - (WIN - 1) + torch.arange(WIN, device=q.device)
    at = p % WIN if st["win_pos0"] is None else p - st["win_pos0"][:, None, None]
    wlive = p >= 0
    bi = torch.arange(B, device=q.device)[:, None, None]
    wrows = st["win"][bi, at.clamp_min(0)].float()
    zw = torch.einsum("bthc,btkc->bthk", q, wrows)
    z = torch.where(live[:, :, None], z * SCALE, float("-inf"))
    zw = torch.where(wlive[:, :, None], zw * SCALE, float("-inf"))
    return z, zw, rows, wrows


def _weights(st):
    z, zw, rows, wrows = _logits(st)
    top = torch.maximum(z.amax(-1), zw.amax(-1)) if z.shape[-1] else zw.amax(-1)
    if st["sink"] is not None:
        top = torch.maximum(top, st["sink"][None, None])
    e, ew = torch.exp(z - top[..., None]), torch.exp(zw - top[..., None])
    den = e.sum(-1) + ew.sum(-1)
    if st["sink"] is not None:
        den = den + torch.exp(st["sink"][None, None] - top)
    return e / den[..., None], ew / den[..., None], rows, wrows


def _run_attn(st):
    p, pw, rows, wrows = _weights(st)
    o = torch.einsum("bthk,btkc->bthc" if st["case"]["k"] else "bthk,bkc->bthc", p, rows)
    o = o + torch.einsum("bthk,btkc->bthc", pw, wrows)
    return _rotate(o, st["q_pos"], -1.0).to(torch.bfloat16)


def _run_mass(st):
    p = _weights(st)[0].sum(2)  # over the heads: [B, T, rows]
    acc = st["acc"]
    acc.mul_(st["case"]["decay"])
    if st["case"]["k"]:
        e = st["idx"].long()
        acc.scatter_add_(1, e.clamp_min(0).flatten(1), torch.where(e >= 0, p, 0.0).flatten(1))
    else:
        acc[:, :p.shape[-1]] += p.sum(1)
    return acc


def _run_evict(st):
    case = st["case"]
    B, N, pr, K = case["B"], case["N"], case["page_rows"], case["budget"]
    pages = N // pr
    dev = st["acc"].device
    entries = ((st["pos"] + 1) // _m(case)).clamp_max(N)
    used = ((entries + pr - 1) // pr)[:, None]  # pages with an entry
    page = torch.arange(pages, device=dev)[None]
    e = torch.arange(N, device=dev)[None]
    score = torch.where(e < entries[:, None], st["acc"], float("-inf")).view(B, pages, pr).amax(-1)
    present = page < used
    kept_always = present & ((page < case["first"]) | (page >= used - case["last"]))
    score = torch.where(kept_always, float("inf"), score)
    order = torch.sort(torch.where(present, score, float("-inf")), dim=1, descending=True,
                       stable=True).indices
    rank = torch.empty_like(order).scatter_(1, order, page.expand(B, -1).contiguous())
    keep = present & (rank < K)
    gone = present & ~keep

    def compact(mask, values, width):
        slot = torch.cumsum(mask, 1) - 1
        out = torch.full((B, width + 1), -1, dtype=torch.int32, device=dev)
        out.scatter_(1, torch.where(mask, slot, width), values.to(torch.int32).expand(B, -1))
        out[:, width] = -1
        return out[:, :width].contiguous()

    keep_e = keep.repeat_interleave(pr, 1) & (e < entries[:, None])
    return {"table": torch.where(gone, -2, st["table"]),
            "kept": compact(keep, page, K),
            "entries": compact(keep_e, e, K * pr),
            "evicted": compact(gone, page, pages),
            "counts": torch.stack((keep.sum(1), keep_e.sum(1), gone.sum(1)), 1).to(torch.int32)}


# --------------------------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------------------------

def _own_setup(st):
    """What a serving program keeps between its calls: parameters, the page descriptor, the
    workspace and the output."""
    import long_context_sparse_08_b200 as csa

    case = st["case"]
    B, N, pr = case["B"], case["N"], case["page_rows"]
    pages = N // pr
    dev = "cuda"
    if case["op"] == "evict":
        K = case["budget"]
        st["p"] = csa.make_params(m=_m(case))
        i32 = dict(dtype=torch.int32, device=dev)
        st["out"] = {"table": torch.empty((B, pages), **i32), "kept": torch.empty((B, K), **i32),
                     "entries": torch.empty((B, K * pr), **i32),
                     "evicted": torch.empty((B, pages), **i32),
                     "counts": torch.empty((B, 3), **i32)}
        need = csa.evict_pages_workspace_size(B, pages)
        st["ws"], st["need"] = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev), need
        return csa
    T, H, k = case["T"], case["H"], case["k"]
    st["p"] = csa.make_params(m=_m(case), overlap=1 if k else 0, n_heads=H, topk=max(k, 1))
    fmt = csa.CSA_MIXED_MXFP4_BF16 if case["fmt"] == "fp4" else csa.CSA_BF16
    st["kv"] = csa.paged_kv(fmt, st["pool"], None, st["table"], st["pool"].shape[0], pr, pages)
    if case["op"] == "attn":
        entry = csa.CSA_WS_SPARSE_MQA if k else csa.CSA_WS_HCA_MQA
        need = csa.workspace_size(st["p"], entry, fmt, B, T, N)
        st["out"] = torch.empty((B, T, H, C), dtype=torch.bfloat16, device=dev)
    else:
        need = csa.attn_mass_workspace_size(st["p"], B, T, N, 1 if k else 0)
    st["ws"], st["need"] = torch.empty((max(need, 1),), dtype=torch.uint8, device=dev), need
    return csa


def _run_own(st):
    if "csa" not in st:
        st["csa"] = _own_setup(st)
    csa, case = st["csa"], st["case"]
    B, p, ws, need = case["B"], st["p"], st["ws"], st["need"]
    if case["op"] == "evict":
        o = st["out"]
        csa.csa_evict_pages(p, B, case["page_rows"], case["N"] // case["page_rows"], st["pos"],
                            st["acc"], st["table"], case["budget"], case["first"], case["last"],
                            o["table"], o["kept"], o["entries"], o["evicted"], o["counts"], ws,
                            need)
        return o
    T, win = case["T"], st["win"]
    if case["op"] == "mass":
        csa.csa_attn_mass_paged(p, B, T, st["q"], st["q_pos"], st["kv"], st.get("idx"), win,
                                win.shape[1], st["win_pos0"], st["sink"], st["q_rms_w"],
                                case["decay"], st["acc"], ws, need)
        return st["acc"]
    if case["k"]:
        csa.csa_sparse_mqa_paged(p, B, T, st["q"], st["q_pos"], st["kv"], st["idx"], win,
                                 win.shape[1], st["win_pos0"], st["sink"], st["q_rms_w"],
                                 st["out"], ws, need)
    else:
        csa.hca_dense_mqa_paged(p, B, T, st["q"], st["q_pos"], st["kv"], win, win.shape[1],
                                st["win_pos0"], st["sink"], st["q_rms_w"], st["out"], ws, need)
    return st["out"]


def run(state):
    if own:
        return _run_own(state)
    return {"attn": _run_attn, "mass": _run_mass, "evict": _run_evict}[state["case"]["op"]](state)


# --------------------------------------------------------------------------------------------
# 64 bits, from the definition
# --------------------------------------------------------------------------------------------

def _value64(pool, fmt):
    if fmt == "bf16":
        return pool.double()
    lo, hi = pool[:, :224] % 16, torch.div(pool[:, :224], 16, rounding_mode="floor")
    code = torch.zeros((pool.shape[0], NOPE), dtype=torch.int64, device=pool.device)
    code[:, 0::2], code[:, 1::2] = lo.long(), hi.long()
    mag = code % 8
    # e2m1: exponent bits e, mantissa bit f: f / 2 at e = 0, else (1 + f / 2) 2^(e - 1)
    e, f = torch.div(mag, 2, rounding_mode="floor"), (mag % 2).double()
    v = torch.where(e == 0, f / 2, (1 + f / 2) * torch.pow(2.0, e.double() - 1))
    v = torch.where(code >= 8, -v, v)
    ex = pool[:, 224:238].double() - 127
    v = v * torch.pow(2.0, ex).repeat_interleave(32, 1)
    return torch.cat((v, pool[:, 240:].contiguous().view(torch.bfloat16).double()), 1)


def exact(case, seed):
    if case["op"] == "evict":
        return None  # whole numbers only
    st = prepare(case, seed)
    B, T, H, k, N, pr, m = case["B"], case["T"], case["H"], case["k"], case["N"], \
        case["page_rows"], _m(case)
    dev = st["q"].device
    out = torch.empty((B, T, H, C), dtype=torch.float64, device=dev)
    acc = st["acc"].double() * case["decay"] if case["op"] == "mass" else None
    freq = torch.exp(-math.log(10000.0) * torch.arange(0, R, 2, device=dev).double() / R)
    for b in range(B):
        full = None
        if not k:
            full = _value64(st["pool"][st["table"][b].long()].flatten(0, 1), case["fmt"])
        for t in range(T):
            pos = st["pos_host"][b] + t
            vis = min(pos // m, N)
            q = st["q"][b, t].double()
            q = q / torch.sqrt((q * q).sum(-1, keepdim=True) / C + 1e-6)
            if st["q_rms_w"] is not None:
                q = q * st["q_rms_w"].double()
            turn = torch.polar(torch.ones_like(freq), freq * pos)
            tail = torch.view_as_complex(q[:, NOPE:].reshape(H, R // 2, 2).contiguous()) * turn
            q = torch.cat((q[:, :NOPE], torch.view_as_real(tail).reshape(H, R)), 1)
            if k:
                ids = st["idx"][b, t, :min(k, vis)].long()
                body = _value64(st["pool"][st["table"][b, ids // pr].long(), ids % pr], case["fmt"])
            else:
                ids, body = None, full[:vis]
            tok = torch.arange(max(0, pos - WIN + 1), pos + 1, device=dev)
            row = tok % WIN if st["win_pos0"] is None else tok - st["win_pos0"][b]
            keys = torch.cat((body, st["win"][b, row].double()))
            z = q @ keys.T / math.sqrt(C)
            if st["sink"] is not None:
                z = torch.cat((z, st["sink"].double()[:, None]), 1)
            w = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))[:, :keys.shape[0]]
            if acc is not None:
                part = w[:, :body.shape[0]].sum(0)
                if k:
                    acc[b].index_add_(0, ids, part)
                else:
                    acc[b, :vis] += part
                continue
            o = w @ keys
            tail = torch.view_as_complex(o[:, NOPE:].reshape(H, R // 2, 2).contiguous())
            out[b, t, :, :NOPE] = o[:, :NOPE]
            out[b, t, :, NOPE:] = torch.view_as_real(tail * turn.conj()).reshape(H, R)
    return acc if acc is not None else out
