"""What the operators of the 8-bit latent cache and of drafted trees are measured on.

Four operators that a serving program calls around the sparse attention:

* ``write``  -- new tokens' latent rows (and indexer keys) quantised to E4M3 as they enter the cache
* ``read``   -- cache rows read back as bf16
* ``sparse`` -- the sparse MLA attention over rows of the 8-bit cache
* ``tree``   -- the attention of a tree of drafted tokens: each node over its selected cache rows
  (8-bit or bf16) and its ancestors among the drafted rows

A case is a dict of plain values; ``prepare`` makes its inputs, ``run`` makes one pass: the
plain form in elementary torch operations, or with ``own`` the library's calls.
"""
import math

import torch

own = False

GROUP = 128            # latent dims that share one scale
E4M3_MAX = 448.0
PROD = {"heads": 128, "d_latent": 512, "d_rope": 64, "idx_dim": 128}
TINY = {"heads": 8, "d_latent": 64, "d_rope": 16, "idx_dim": 32}
ODD = {"heads": 37, "d_latent": 320, "d_rope": 24, "idx_dim": 80}
DIMS = {"prod": PROD, "tiny": TINY, "odd": ODD}


# ----------------------------------------------------------------------------- cases
def listed():
    return [
        # a decode step's new tokens, one row per sequence: all latency
        {"name": "write decode 64", "op": "write", "dims": "prod", "batch": 64, "n": 1, "max_len": 2048, "n_src": 0},
        # a prompt enters the cache
        {"name": "write prompt 32k", "op": "write", "dims": "prod", "batch": 1, "n": 32768, "max_len": 32768,
         "n_src": 0},
        # the accepted paths of drafted trees are committed: at most 7 of each sequence's 33 drafted rows
        {"name": "commit paths", "op": "write", "dims": "prod", "batch": 37, "n": 7, "max_len": 4096, "n_src": 33},
        # a cached prefix back as bf16 for the masked dense mode, four ragged sequences
        {"name": "read prefix 4x8000", "op": "read", "dims": "prod", "batch": 4, "n": 8000, "max_len": 8192,
         "listed": False},
        # the selected rows of a decode step gathered as bf16
        {"name": "read listed 8x2048", "op": "read", "dims": "prod", "batch": 8, "n": 2048, "max_len": 32768,
         "listed": True},
        # one sequence's decode step at a 128K context: few rows, latency
        {"name": "sparse decode 1", "op": "sparse", "dims": "prod", "batch": 1, "n": 1, "max_len": 131072,
         "topk": 2048},
        # a batched decode step, lengths from 1 up, so some rows of the selection are mostly padding
        {"name": "sparse decode 64", "op": "sparse", "dims": "prod", "batch": 64, "n": 1, "max_len": 16384,
         "topk": 2048},
        # a chunk of a long prompt
        {"name": "sparse chunk 1024", "op": "sparse", "dims": "prod", "batch": 1, "n": 1024, "max_len": 65536,
         "topk": 2048},
        # small dims, short context, odd selection width
        {"name": "sparse tiny", "op": "sparse", "dims": "tiny", "batch": 2, "n": 100, "max_len": 501, "topk": 77},
        # a tree of 16 drafted tokens after one long context
        {"name": "tree 1x16", "op": "tree", "dims": "prod", "batch": 1, "n": 16, "max_len": 131072, "topk": 2048,
         "qcache": True},
        # drafted trees of a batch, the largest that fill one 64-row block and one row more
        {"name": "tree 4x65", "op": "tree", "dims": "prod", "batch": 4, "n": 65, "max_len": 16384, "topk": 1500,
         "qcache": True},
        # drafted trees over the bf16 cache
        {"name": "tree bf16 16x8", "op": "tree", "dims": "prod", "batch": 16, "n": 8, "max_len": 8192, "topk": 2048,
         "qcache": False},
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["write", "read", "sparse", "tree"])
    dims = rng.choice(["prod", "prod", "prod", "odd", "tiny"])
    if op == "write":
        batch = _log_int(rng, 1, 128)
        n = _log_int(rng, 1, max(1, 32768 // batch))
        n_src = rng.choice([0, 0, n + rng.randint(0, 40)])
        return {"op": op, "dims": dims, "batch": batch, "n": n, "max_len": n + rng.randint(0, 300), "n_src": n_src}
    if op == "read":
        batch = _log_int(rng, 1, 64)
        n = _log_int(rng, 1, max(1, 32000 // batch))
        listed_rows = rng.random() < 0.5
        return {"op": op, "dims": dims, "batch": batch, "n": n, "max_len": n + rng.randint(0, 4000),
                "listed": listed_rows}
    if op == "sparse":
        topk = _log_int(rng, 1, 2048)
        queries = _log_int(rng, 1, 1000)
        batch = _log_int(rng, 1, min(queries, 96))
        n = max(1, queries // batch)
        return {"op": op, "dims": dims, "batch": batch, "n": n, "max_len": n + _log_int(rng, 1, 16000), "topk": topk}
    topk = _log_int(rng, 1, 2048)
    n = _log_int(rng, 1, 200)
    batch = _log_int(rng, 1, max(1, 600 // n))
    return {"op": op, "dims": dims, "batch": batch, "n": n, "max_len": n + _log_int(rng, 1, 16000), "topk": topk,
            "qcache": rng.random() < 0.6}


# ----------------------------------------------------------------------------- inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _latents(g, *shape):
    """Normalised latents with a spread of magnitudes from row to row."""
    x = torch.randn(shape, generator=g, device="cuda", dtype=torch.float32)
    s = torch.rand(shape[:-1], generator=g, device="cuda", dtype=torch.float32)
    return (x * (0.5 + s[..., None])).to(torch.bfloat16)


def _lengths(g, batch, lo, hi):
    """int32 [batch] in [lo, hi], the first of them hi."""
    x = torch.randint(lo, hi + 1, (batch,), generator=g, device="cuda", dtype=torch.int32)
    x[0] = hi
    return x


def _selection(g, lengths, n, topk, max_len):
    """int32 [B, n, topk] distinct-looking positions below each sequence's length, -1 behind the last."""
    batch = lengths.numel()
    u = torch.rand((batch, n, topk), generator=g, device="cuda")
    j = torch.arange(topk, device="cuda")
    ln = lengths.view(batch, 1, 1).to(torch.float64)
    # entry j lies in the j-th of topk equal slices of the sequence where it is longer than topk,
    # and is position j where it is not
    spread = ((j + u) * (ln / topk)).floor().clamp(max=max_len - 1)
    pos = torch.where(ln > topk, torch.minimum(spread, ln - 1), j.to(torch.float64).expand(batch, n, topk))
    return torch.where(pos < ln, pos, torch.full_like(pos, -1.0)).to(torch.int32)


def _qcache(g, d, batch, max_len):
    codes = (torch.randn((batch, max_len, d["d_latent"]), generator=g, device="cuda") * 100.0).clamp(-448, 448)
    groups = -(-d["d_latent"] // GROUP)
    e = torch.randint(-8, -5, (batch, max_len, groups), generator=g, device="cuda")
    return {"codes": codes.to(torch.float8_e4m3fn).view(torch.uint8), "scales": torch.exp2(e.float()),
            "rope": _latents(g, batch, max_len, d["d_rope"])}


def prepare(case, seed):
    d = DIMS[case["dims"]]
    g = _gen(seed)
    b, n, max_len = case["batch"], case["n"], case["max_len"]
    width = d["d_latent"] + d["d_rope"]
    st = {"case": case, "d": d}
    groups = -(-d["d_latent"] // GROUP)
    if case["op"] == "write":
        rows = case["n_src"] or n
        st["latent"] = _latents(g, b, rows, width)
        st["keys"] = _latents(g, b, rows, d["idx_dim"])
        st["start"] = torch.randint(0, max_len - n + 1, (b,), generator=g, device="cuda", dtype=torch.int32)
        count = _lengths(g, b, 1, n)
        st["lengths"] = st["start"] + count
        st["src"] = None
        if case["n_src"]:
            # an accepted path: rising node numbers, -1 behind its last
            order = torch.rand((b, rows), generator=g, device="cuda").argsort(dim=1)[:, :n].sort(dim=1).values
            keep = torch.arange(n, device="cuda")[None, :] < count[:, None]
            st["src"] = torch.where(keep, order, torch.full_like(order, -1)).to(torch.int32)
        st["cache"] = {"codes": torch.zeros((b, max_len, d["d_latent"]), dtype=torch.uint8, device="cuda"),
                       "scales": torch.zeros((b, max_len, groups), device="cuda"),
                       "rope": torch.zeros((b, max_len, d["d_rope"]), dtype=torch.bfloat16, device="cuda")}
        st["k_idx"] = torch.zeros((b, max_len, d["idx_dim"]), dtype=torch.uint8, device="cuda")
        st["k_scale"] = torch.zeros((b, max_len), device="cuda")
    elif case["op"] == "read":
        st["cache"] = _qcache(g, d, b, max_len)
        st["lengths"] = _lengths(g, b, 1, max_len)
        st["start"] = torch.zeros((b,), dtype=torch.int32, device="cuda")
        st["rows"] = None
        if case["listed"]:
            st["rows"] = _selection(g, st["lengths"], 1, n, max_len).view(b, n)
    else:
        if case.get("qcache", True):
            st["cache"] = _qcache(g, d, b, max_len)
        else:
            st["kv"] = _latents(g, b, max_len, width)
        lengths = _lengths(g, b, 1, max_len)
        st["q"] = torch.randn((b, n, d["heads"], width), generator=g, device="cuda").to(torch.bfloat16)
        st["idx"] = _selection(g, lengths, n, case["topk"], max_len)
        st["scale"] = float(torch.tensor(width ** -0.5, dtype=torch.float32))
        if case["op"] == "tree":
            st["draft"] = _latents(g, b, n, width)
            # node i hangs below the last committed token (-1) or below an earlier node
            u = torch.rand((b, n), generator=g, device="cuda")
            i = torch.arange(n, device="cuda")
            parents = (u * (i + 1)).floor().to(torch.int32) - 1
            # a padded batch: the nodes behind a sequence's last are absent (-2)
            nodes = _lengths(g, b, max(1, n // 2), n)
            st["parents"] = torch.where(i[None, :] < nodes[:, None], parents, torch.full_like(parents, -2))
    if own:
        _prepare_own(st)
    return st


def _prepare_own(st):
    """The handles that a program keeps beside its buffers: dims, workspace, cache."""
    import sparse_attention_long_indexer_b200 as dsa
    case, d = st["case"], st["d"]
    st["dsa"] = dsa
    st["dims"] = dsa.make_dims(case["batch"], case["n"], case["max_len"], idx_dim=d["idx_dim"], n_heads=d["heads"],
                               d_latent=d["d_latent"], d_rope=d["d_rope"], softmax_scale=st.get("scale"))
    st["ws"] = dsa.Workspace.create_qcache(st["dims"], case.get("topk", 1))
    if "cache" in st:
        c = st["cache"]
        st["handle"] = dsa.QCache(c["codes"], c["scales"], c["rope"], st.get("k_idx"), st.get("k_scale"))


# ----------------------------------------------------------------------------- plain forms
def _quantise(x):
    """fp32 [..., k]: E4M3 codes and the power-of-two scale of each row: the smallest 2^e with
    amax <= 448 * 2^e, e in [-100, 100]; 1 for a row of zeros. amax is over the finite values;
    infinities become the largest code, NaN E4M3's NaN."""
    mag = x.abs()
    amax = torch.where(torch.isfinite(x), mag, torch.zeros_like(mag)).amax(dim=-1)
    m, e = torch.frexp(amax)
    e = torch.where(m <= 0.875, e - 9, e - 8).clamp(-100, 100)
    e = torch.where(amax > 0, e, torch.zeros_like(e))
    y = (x * torch.exp2(-e.float())[..., None]).clamp(-E4M3_MAX, E4M3_MAX)
    return y.to(torch.float8_e4m3fn).view(torch.uint8), torch.exp2(e.float())


def _run_write(st):
    d, case = st["d"], st["case"]
    b, n, max_len, dl = case["batch"], case["n"], case["max_len"], d["d_latent"]
    j = torch.arange(n, device="cuda")
    src = st["src"].long() if st["src"] is not None else j.expand(b, n)
    pos = st["start"].long()[:, None] + j
    ok = (src >= 0) & (pos >= 0) & (pos < st["lengths"].long()[:, None]) & (pos < max_len)
    seq = torch.arange(b, device="cuda")[:, None].expand(b, n)[ok]
    at, of = pos[ok], src[ok]
    x = st["latent"][seq, of].float()
    groups = -(-dl // GROUP)
    lat = torch.nn.functional.pad(x[:, :dl], (0, groups * GROUP - dl)).view(-1, groups, GROUP)
    codes, scales = _quantise(lat)
    scales = scales.masked_fill(lat.isnan().any(dim=-1), math.nan)      # a group that holds a NaN reads as NaN
    c = st["cache"]
    c["codes"][seq, at] = codes.reshape(-1, groups * GROUP)[:, :dl]
    c["scales"][seq, at] = scales
    c["rope"][seq, at] = x[:, dl:].to(torch.bfloat16)
    kc, ks = _quantise(st["keys"][seq, of].float())
    st["k_idx"][seq, at] = kc
    st["k_scale"][seq, at] = ks


def _written(st):
    c = st["cache"]
    return {"codes": c["codes"].view(torch.float8_e4m3fn), "scales": c["scales"], "rope": c["rope"],
            "k_idx": st["k_idx"].view(torch.float8_e4m3fn), "k_scale": st["k_scale"]}


def _rows8(cache, seq, pos):
    """fp32 rows of the 8-bit cache at (seq, pos), index tensors of one shape."""
    codes = cache["codes"].view(torch.float8_e4m3fn)[seq, pos].float()
    dl = codes.shape[-1]
    s = cache["scales"][seq, pos].repeat_interleave(GROUP, dim=-1)[..., :dl]
    return torch.cat([codes * s, cache["rope"][seq, pos].float()], dim=-1)


def _read_positions(st):
    case = st["case"]
    b, n = case["batch"], case["n"]
    if st["rows"] is not None:
        pos = st["rows"].long()
        return pos, pos >= 0
    pos = st["start"].long()[:, None] + torch.arange(n, device="cuda")
    return pos, (pos >= 0) & (pos < st["lengths"].long()[:, None])


def _run_read(st):
    b = st["case"]["batch"]
    pos, ok = _read_positions(st)
    seq = torch.arange(b, device="cuda")[:, None].expand_as(pos)
    x = _rows8(st["cache"], seq, torch.where(ok, pos, torch.zeros_like(pos)))
    return torch.where(ok[..., None], x, torch.zeros_like(x)).to(torch.bfloat16)


def _ancestors(parents, dtype):
    """bool [B, n, n]: node s is node i itself or an ancestor of it; no node for an absent i."""
    n = parents.shape[1]
    eye = torch.eye(n, device=parents.device, dtype=dtype)
    step = (parents.long()[..., None] == torch.arange(n, device=parents.device)).to(dtype)
    reach = torch.linalg.matrix_power(eye + step, n) > 0
    return reach & (parents >= -1)[..., None]


def _attend(st, dtype):
    case, d = st["case"], st["d"]
    b, n, h, dl = case["batch"], case["n"], d["heads"], d["d_latent"]
    idx = st["idx"].long()
    ok = idx >= 0
    seq = torch.arange(b, device="cuda")[:, None, None].expand_as(idx)
    at = torch.where(ok, idx, torch.zeros_like(idx))
    rows = _rows8(st["cache"], seq, at) if "cache" in st else st["kv"][seq, at].to(dtype)
    rows = rows.to(dtype).view(b * n, -1, rows.shape[-1])
    q = st["q"].to(dtype).view(b * n, h, -1)
    z = torch.bmm(q, rows.transpose(1, 2)) * st["scale"]
    if case["op"] == "tree":
        draft = st["draft"].to(dtype)
        anc = _ancestors(st["parents"], torch.float64)
        zt = torch.bmm(q.reshape(b, n * h, -1), draft.transpose(1, 2)).view(b * n, h, n) * st["scale"]
        ok = torch.cat([(ok & (st["parents"] >= -1)[..., None]).view(b * n, 1, -1), anc.view(b * n, 1, n)], dim=2)
        z = torch.cat([z, zt], dim=2)
    else:
        ok = ok.view(b * n, 1, -1)
    z = z.masked_fill(~ok, -math.inf)
    m = z.amax(dim=2, keepdim=True)
    m = torch.where(torch.isfinite(m), m, torch.zeros_like(m))
    p = torch.exp(z - m)
    total = p.sum(dim=2, keepdim=True)
    p = p / torch.where(total > 0, total, torch.ones_like(total))
    k = rows.shape[1]
    out = torch.bmm(p[:, :, :k], rows[:, :, :dl])
    if case["op"] == "tree":
        out = out + torch.bmm(p[:, :, k:].reshape(b, n * h, n), draft[..., :dl]).view(b * n, h, dl)
    lse = (torch.log(total) + m).squeeze(2)
    return out.view(b, n, h, dl), lse.view(b, n, h)


def run(st):
    op = st["case"]["op"]
    if own:
        return _run_own(st, op)
    if op == "write":
        _run_write(st)
        return _written(st)
    if op == "read":
        return _run_read(st)
    out, lse = _attend(st, torch.float32)
    return out.to(torch.bfloat16), lse


def _run_own(st, op):
    dsa = st["dsa"]
    if op == "write":
        dsa.qcache_write(st["dims"], st["handle"], st["latent"], st["keys"], st["ws"], start=st["start"],
                         lengths=st["lengths"], src_rows=st["src"])
        return _written(st)
    if op == "read":
        if st["rows"] is not None:
            return dsa.qcache_read(st["dims"], st["handle"], st["ws"], rows=st["rows"])
        return dsa.qcache_read(st["dims"], st["handle"], st["ws"], start=st["start"], lengths=st["lengths"])
    topk = st["case"]["topk"]
    if op == "sparse":
        return dsa.sparse_mla_attn_qcache(st["dims"], st["q"], st["handle"], st["idx"], topk, st["ws"])
    return dsa.tree_mla_attn(st["dims"], st["q"], st["handle"] if "cache" in st else st["kv"], st["idx"], topk,
                             st["draft"], st["parents"], st["ws"])


# ----------------------------------------------------------------------------- the definition in 64 bits
def _exact_codes(x):
    """float64 [..., k]: values of the nearest E4M3 codes after scaling (ties to even), and the scales."""
    amax = x.abs().amax(dim=-1)
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, E4M3_MAX)) / E4M3_MAX)).clamp(-100, 100)
    e = torch.where(amax > E4M3_MAX * torch.exp2(e), e + 1, e)          # log2 beside a power of two
    e = torch.where((amax > 0) & (amax <= E4M3_MAX * torch.exp2(e - 1)), e - 1, e).clamp(-100, 100)
    scale = torch.exp2(e)
    y = x / scale[..., None]
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)   # spacing of the codes there
    return torch.round(y / step) * step, scale


def exact(case, seed):
    st = prepare(case, seed)
    d, b, n = st["d"], case["batch"], case["n"]
    dl = d["d_latent"]
    if case["op"] == "write":
        groups = -(-dl // GROUP)
        width = case["max_len"]
        j = torch.arange(width, device="cuda")[None, :] - st["start"].long()[:, None]     # row of each position
        ok = (j >= 0) & (j < n) & (j < (st["lengths"] - st["start"]).long()[:, None])
        j = j.clamp(0, n - 1)
        row = j if st["src"] is None else torch.gather(st["src"].long(), 1, j)
        ok = ok & (row >= 0)
        row = row.clamp(min=0)[..., None]
        x = torch.gather(st["latent"], 1, row.expand(b, width, dl + d["d_rope"])).double()
        lat = torch.nn.functional.pad(x[..., :dl], (0, groups * GROUP - dl)).view(b, width, groups, GROUP)
        codes, scales = _exact_codes(lat)
        kc, ks = _exact_codes(torch.gather(st["keys"], 1, row.expand(b, width, d["idx_dim"])).double())
        o = ok[..., None]
        return {"codes": codes.reshape(b, width, -1)[..., :dl] * o, "scales": scales * o, "rope": x[..., dl:] * o,
                "k_idx": kc * o, "k_scale": ks * ok}
    if case["op"] == "read":
        pos, ok = _read_positions(st)
        at = torch.where(ok, pos, torch.zeros_like(pos))[..., None]
        c = st["cache"]
        groups = c["scales"].shape[-1]
        code = torch.gather(c["codes"], 1, at.expand(b, n, dl)).view(torch.float8_e4m3fn).double()
        scale = torch.gather(c["scales"], 1, at.expand(b, n, groups)).double()
        rope = torch.gather(c["rope"], 1, at.expand(b, n, d["d_rope"])).double()
        of = torch.arange(dl, device="cuda") // GROUP
        return torch.cat([code * scale[..., of], rope], dim=-1) * ok[..., None]
    return _exact_attention(st)


def _exact_attention(st):
    """Every query's softmax over its own rows in float64: the weights exp(z - lse) with the lse of all rows."""
    case, d = st["case"], st["d"]
    b, n, h, dl = case["batch"], case["n"], d["heads"], d["d_latent"]
    dev = "cuda"
    outs, lses = [], []
    if case["op"] == "tree":
        par = st["parents"].cpu().tolist()
        own_path = torch.zeros((b, n, n), dtype=torch.bool)
        for s in range(b):
            for i in range(n):
                if par[s][i] >= -1:
                    own_path[s, i, i] = True
                    if par[s][i] >= 0:
                        own_path[s, i] |= own_path[s, par[s][i]]
        own_path = own_path.to(dev)
    of = torch.arange(dl, device=dev) // GROUP
    for s in range(b):
        if "cache" in st:
            c = st["cache"]
            table = torch.cat([c["codes"][s].view(torch.float8_e4m3fn).double() * c["scales"][s].double()[:, of],
                               c["rope"][s].double()], dim=1)
        else:
            table = st["kv"][s].double()
        step = max(1, 200_000 // case["topk"])
        for a in range(0, n, step):
            e = min(n, a + step)
            ix = st["idx"][s, a:e].long()
            valid = ix >= 0
            rows = table[ix.clamp(min=0).reshape(-1)].view(e - a, -1, table.shape[1])
            if case["op"] == "tree":
                tail = st["draft"][s].double().expand(e - a, n, table.shape[1])
                rows = torch.cat([rows, tail], dim=1)
                valid = torch.cat([valid & (st["parents"][s, a:e] >= -1)[:, None], own_path[s, a:e]], dim=1)
            z = torch.einsum("thd,tkd->thk", st["q"][s, a:e].double(), rows) * st["scale"]
            z = torch.where(valid[:, None, :], z, torch.full_like(z, -math.inf))
            lse = torch.logsumexp(z, dim=2)
            w = torch.where(valid[:, None, :], torch.exp(z - lse[..., None]), torch.zeros_like(z))
            outs.append(torch.einsum("thk,tkd->thd", w, rows[..., :dl]))
            lses.append(lse)
    return torch.cat(outs).view(b, n, h, dl), torch.cat(lses).view(b, n, h)


# ----------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    d = DIMS[case["dims"]]
    b, n = case["batch"], case["n"]
    width = d["d_latent"] + d["d_rope"]
    row8 = d["d_latent"] + 2 * d["d_rope"] + 4 * -(-d["d_latent"] // GROUP)
    if case["op"] == "write":
        # on average half of the rows are inside a sequence's count; the first sequence is full
        rows = n * (1 + 0.5 * (b - 1))
        return {"bytes": rows * (2 * width + 2 * d["idx_dim"] + row8 + d["idx_dim"] + 4), "flops": 0}
    if case["op"] == "read":
        return {"bytes": b * n * (row8 * 0.75 + 2 * width), "flops": 0}
    topk, h = case["topk"], d["heads"]
    rows = min(b * n * topk, b * case["max_len"])
    bytes_ = rows * (row8 if case.get("qcache", True) else 2 * width)
    bytes_ += b * n * (2 * h * width + 2 * h * d["d_latent"] + 4 * h + 4 * topk)
    pairs = b * n * topk
    if case["op"] == "tree":
        bytes_ += b * n * 2 * width
        pairs += b * n * math.log2(n + 1)
    return {"bytes": bytes_, "flops": 2 * pairs * h * (width + d["d_latent"])}
