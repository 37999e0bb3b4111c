"""The operators of a serving loop around the decode step, as they are measured.

Prompt prologue and prompt attention (packed prompts, and chunks over a paged cache), verification
of drafted tokens, and the upkeep of a paged cache (fork, resize, compact, with the page copies).

``own = False`` computes each operator in plain torch operations; ``own = True`` makes the calls a
user of ``load_balanced_split_step_b200`` makes. Both take what ``prepare`` gives.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------ cases
def listed():
    return [
        # one short prompt on a small model: time to first token is launch latency
        dict(name="prompt_short", op="attention", lens="128", heads=8, kv_heads=2, head_dim=64, lse=False),
        # a serving batch of packed prompts of very different lengths, odd ones among them
        dict(name="prompt_mixed", op="attention", lens="1,17,4096,513,2050,64,1023,200", heads=64, kv_heads=8,
             head_dim=128, lse=False),
        # one long prompt: the compute-bound end
        dict(name="prompt_long", op="attention", lens="16384", heads=64, kv_heads=8, head_dim=128, lse=True),
        # chunked prefill: new tokens of each request attend to the cached pages before them too
        dict(name="prompt_chunks", op="paged", lens="512,2048,100,1", ctx="8192,14003,30000,4095", heads=64,
             kv_heads=8, head_dim=128, page=64, layout="HND", lse=True),
        # the prologue of one short prompt into a bf16 cache
        dict(name="prologue_short", op="prologue", lens="100", ctx="0", heads=8, kv_heads=2, head_dim=64, page=16,
             kv="bf16", layout="HND"),
        # packed prompts into an E4M3 cache, one of them the continuation of a cached prefix
        dict(name="prologue_mixed", op="prologue", lens="4096,777,2048,1,1270", ctx="0,0,2001,511,64",
             heads=64, kv_heads=8, head_dim=128, page=64, kv="e4m3", layout="NHD"),
        # one user, three drafted tokens: latency
        dict(name="verify_one", op="verify", batch=1, drafts=3, vocab=32000, dtype="fp32", onehot=False, ragged=False),
        # a batch of users with ragged drafts over a large vocabulary
        dict(name="verify_batch", op="verify", batch=64, drafts=3, vocab=131071, dtype="fp32", onehot=False,
             ragged=True),
        # a few beams reordered after a step: some go on twice, some are dropped
        dict(name="fork_beams", op="fork", batch=4, max_len=1000, max_pages=64, page=16, num_pages=512, kv_heads=2,
             head_dim=64, layers=1, reorder=True),
        # several samples drawn from each prompt of a large batch: every copy of a part-filled page
        dict(name="fork_samples", op="fork", batch=256, max_len=4096, max_pages=80, page=64, num_pages=4096,
             kv_heads=8, head_dim=128, layers=1, reorder=False),
        # the reservation before and the roll-back after speculation, requests of many lengths
        dict(name="resize_batch", op="resize", batch=256, max_len=4000, max_pages=256, page=16, num_pages=40000,
             kv_heads=2, head_dim=64, layers=1),
        # a fragmented pool closed up
        dict(name="compact_pool", op="compact", batch=64, max_len=4096, max_pages=72, page=64, num_pages=4096,
             kv_heads=8, head_dim=128, layers=1),
    ]


def _text(ints):
    return ",".join(str(i) for i in ints)


def _lengths(case):
    """(new tokens, cached tokens before them) of each request."""
    lens = [int(x) for x in case["lens"].split(",")]
    return lens, [int(x) for x in case["ctx"].split(",")] if "ctx" in case else [0] * len(lens)


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "paged", "prologue", "verify", "fork", "resize", "compact"])
    if op in ("attention", "paged", "prologue"):
        kv_heads = rng.choice([1, 2, 4, 8])
        heads = kv_heads * rng.choice([1, 2, 4, 8])
        D = rng.choice([64, 128])
        n = _log(rng, 1, 24)
        if op == "prologue":
            lens = [_log(rng, 1, 8192 // n) for _ in range(n)]
            ctx = [rng.choice([0, _log(rng, 1, 30000 // n)]) for _ in lens]
            return dict(op=op, lens=_text(lens), ctx=_text(ctx), heads=heads, kv_heads=kv_heads, head_dim=128 if (kv := rng.choice(["bf16", "e4m3"])) == "e4m3" else D,
                        page=rng.choice([16, 32, 64, 128]), kv=kv, layout=rng.choice(["HND", "NHD"]))
        lens = [_log(rng, 1, 8192 if n < 4 else 8192 // n) for _ in range(n)]
        c = dict(op=op, lens=_text(lens), heads=heads, kv_heads=kv_heads, head_dim=D, lse=rng.random() < 0.5)
        if op == "paged":
            c.update(ctx=_text([rng.choice([0, _log(rng, 1, 16000)]) for _ in lens]), page=rng.choice([16, 32, 64, 128]),
                     layout=rng.choice(["HND", "NHD"]))
        return c
    if op == "verify":
        return dict(op=op, batch=_log(rng, 1, 64), drafts=rng.randint(1, 7), vocab=_log(rng, 1000, 130000),
                    dtype=rng.choice(["fp32", "bf16"]), onehot=rng.random() < 0.3, ragged=rng.random() < 0.5)
    page = rng.choice([16, 32, 64])
    batch, max_len = _log(rng, 1, 256), _log(rng, 20, 4096)
    max_pages = max_len // page + 4
    return dict(op=op, batch=batch, max_len=max_len, max_pages=max_pages, page=page,
                num_pages=max(64, int(batch * max_pages * rng.uniform(1.2, 2.0))) if page < 64 else
                min(max(64, int(batch * max_pages * 1.5)), 4096 if batch * max_pages < 2700 else 26000),
                kv_heads=rng.choice([1, 2]), head_dim=64, layers=rng.randint(1, 2), reorder=rng.random() < 0.5)


# ------------------------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.float32)


def _cu(lens):
    return torch.tensor([0] + list(np.cumsum(lens)), dtype=torch.int32, device=DEV)


def _table(rng, need, num_pages, width):
    """A block table over a random permutation of the pool, -1 past each request's pages."""
    perm = rng.permutation(num_pages)
    t = np.full((len(need), width), -1, dtype=np.int32)
    o = 0
    for r, n in enumerate(need):
        t[r, :n] = perm[o:o + n]
        o += n
    return t


def _cache(g, num_pages, kv_heads, page, D, layout, fill=True):
    shape = (num_pages, kv_heads, page, D) if layout == "HND" else (num_pages, page, kv_heads, D)
    if not fill:
        return torch.zeros(shape, dtype=torch.bfloat16, device=DEV)
    return torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)


def prepare(case, seed):
    g = _gen(seed)
    rng = np.random.default_rng(seed)
    op = case["op"]
    s = dict(case=case)
    if op in ("attention", "paged", "prologue"):
        (lens, ctx), Hq, Hkv, D = _lengths(case), case["heads"], case["kv_heads"], case["head_dim"]
        n = sum(lens)
        s["cu"] = _cu(lens)
        # the projection's output: q, k and v heads of every token side by side
        qkv = _randn(g, n, Hq + 2 * Hkv, D).to(torch.bfloat16)
        s["qkv"] = qkv
        if op == "attention":
            s["q"] = qkv[:, :Hq].contiguous()
            s["k"], s["v"] = qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]  # views, as a program slices them
            return s
        total = [a + b for a, b in zip(ctx, lens)]
        P = case["page"]
        need = [-(-t // P) for t in total]
        num_pages = sum(need) + 3
        s["seq_lens"] = torch.tensor(total, dtype=torch.int32, device=DEV)
        s["table"] = torch.from_numpy(_table(rng, need, num_pages, max(need) + 1)).to(DEV)
        if op == "paged":
            s["q"] = qkv[:, :Hq].contiguous()
            s["k_pages"] = _cache(g, num_pages, Hkv, P, D, case["layout"])
            s["v_pages"] = _cache(g, num_pages, Hkv, P, D, case["layout"])
            return s
        s["k_pages"] = _cache(g, num_pages, Hkv, P, D, case["layout"], fill=False)
        s["v_pages"] = torch.zeros_like(s["k_pages"])
        if case["kv"] == "e4m3":
            s["k_pages"] = s["k_pages"].to(torch.float8_e4m3fn)
            s["v_pages"] = s["v_pages"].to(torch.float8_e4m3fn)
            s["k_scale"] = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
            s["v_scale"] = 0.01 + 0.01 * torch.rand(Hkv, generator=g, device=DEV)
        s["q_norm_w"] = 1.0 + 0.1 * _randn(g, D)
        s["k_norm_w"] = 1.0 + 0.1 * _randn(g, D)
        return s
    if op == "verify":
        Bn, T, V = case["batch"], case["drafts"], case["vocab"]
        dt = torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
        logits = 3.0 * _randn(g, Bn, T + 1, V)
        s["p"] = torch.softmax(logits, -1).to(dt)
        dl = logits[:, :T] + 0.7 * _randn(g, Bn, T, V)  # a draft model that mostly agrees
        q = torch.softmax(dl, -1)
        s["x"] = torch.multinomial(q.reshape(Bn * T, V), 1, generator=g).reshape(Bn, T).to(torch.int32)
        s["q"] = None if case["onehot"] else q.to(dt)
        s["u"] = torch.rand((Bn, T + 1), generator=g, device=DEV)
        lens = rng.integers(0, T + 1, Bn) if case["ragged"] else np.full(Bn, T)
        s["draft_lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
        s["seq_lens"] = torch.from_numpy(rng.integers(T + 1, 5000, Bn).astype(np.int32)).to(DEV)
        return s
    # page upkeep: lengths, a table over a scattered pool, reference counts
    Bn, P, M, N = case["batch"], case["page"], case["max_pages"], case["num_pages"]
    lens = rng.integers(1, case["max_len"] + 1, Bn)
    if op == "fork" and not case["reorder"]:  # one live request in four; the others are still empty rows
        lens[np.arange(Bn) % 4 != 0] = 0
    need = -(-lens // P)
    while need.sum() > N * 3 // 4:  # leave room
        lens = lens // 2
        need = -(-lens // P)
    table = _table(rng, need, N, M)
    if op in ("resize", "compact") and Bn > 1:  # requests that share a prefix of pages
        for r in range(1, Bn, 2):
            k = int(min(need[r - 1], need[r]) // 2)
            table[r, :k] = table[r - 1, :k]
    ref = np.bincount(table[table >= 0], minlength=N).astype(np.int32)
    s["table"] = torch.from_numpy(table).to(DEV)
    s["lens"] = torch.from_numpy(lens.astype(np.int32)).to(DEV)
    s["ref"] = torch.from_numpy(ref).to(DEV)
    if op == "fork":
        parents = rng.integers(0, Bn, Bn) if case["reorder"] else np.arange(Bn) // 4 * 4
        s["parents"] = torch.from_numpy(parents.astype(np.int32)).to(DEV)
    if op == "resize":
        # most grow by a few tokens, some are rolled back, some end
        d = rng.integers(1, 6, Bn)
        d = np.where(rng.random(Bn) < 0.3, -rng.integers(0, 4 * P, Bn), d)
        new = np.clip(lens + d, 0, M * P)
        new[rng.random(Bn) < 0.1] = 0
        s["new_lens"] = torch.from_numpy(new.astype(np.int32)).to(DEV)
    s["table_out"], s["ref_out"] = torch.empty_like(s["table"]), torch.empty_like(s["ref"])
    s["lens_out"] = torch.empty_like(s["lens"])
    s["caches"] = [_cache(g, N, case["kv_heads"], P, case["head_dim"], "HND") for _ in range(2 * case["layers"])]
    return s


# ------------------------------------------------------------------------------------ one pass
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s, op)
    return {"attention": _plain_attention, "paged": _plain_paged, "prologue": _plain_prologue,
            "verify": _plain_verify, "fork": _plain_fork, "resize": _plain_resize, "compact": _plain_compact}[op](s)


def _own(s, op):
    from load_balanced_split_step_b200 import binding as B
    c = s["case"]
    if op == "attention":
        out, lse, _ = B.prompt_attention(s["q"], s["k"], s["v"], s["cu"], return_lse=c["lse"])
        return (out, lse) if c["lse"] else out
    if op == "paged":
        out, lse, _ = B.prompt_attention_paged(s["q"], s["k_pages"], s["v_pages"], s["table"], s["seq_lens"], s["cu"],
                                               kv_layout=c["layout"], return_lse=c["lse"])
        return (out, lse) if c["lse"] else out
    if op == "prologue":
        q, k, _ = B.prompt_prologue(s["qkv"], s["cu"], s["q_norm_w"], s["k_norm_w"], s["k_pages"], s["v_pages"],
                                    s["table"], s["seq_lens"], c["heads"], c["kv_heads"], kv_dtype=c["kv"],
                                    kv_layout=c["layout"], k_scale=s.get("k_scale"), v_scale=s.get("v_scale"))
        return q, k, _values(s, "k"), _values(s, "v")
    if op == "verify":
        tokens, accepted, lens, _ = B.verify_drafts(s["x"], s["p"], s["q"], s["u"], draft_lens=s["draft_lens"],
                                                    seq_lens=s["seq_lens"])
        return tokens, accepted, lens
    kw = dict(block_table_out=s["table_out"], ref_count_out=s["ref_out"])
    if op == "fork":
        up = B.fork_pages(s["table"], s["lens"], s["ref"], s["parents"], c["page"], seq_lens_out=s["lens_out"], **kw)
    elif op == "resize":
        up = B.resize_pages(s["table"], s["lens"], s["new_lens"], s["ref"], c["page"], **kw)
    else:
        up = B.compact_pages(s["table"], s["ref"], **kw)
    B.copy_pages(s["caches"], up.moves, up.n_moves, status=up.status)
    if op == "fork":
        return up.block_table, up.seq_lens, up.ref_count, s["caches"]
    if op == "resize":
        return up.block_table, up.ref_count, s["caches"]
    return up.block_table, up.ref_count, up.page_map, s["caches"]


def _values(s, which):
    """The cache as a caller reads it: E4M3 codes as the numbers they stand for (exact in bf16)."""
    t = s[which + "_pages"]
    return t.to(torch.bfloat16) if t.dtype == torch.float8_e4m3fn else t


# ------------------------------------------------------------------------------------ plain forms
def _attend(q, k, v, off, scale, out, lse):
    """q [n, Hq, D], k / v [m, Hkv, D]: row i sees keys 0 .. i + off. fp32, rounded at the end."""
    n, Hq, D = q.shape
    m, Hkv, _ = k.shape
    G = Hq // Hkv
    step = max(1, (1 << 27) // max(1, m * G))
    for h in range(Hkv):
        kh, vh = k[:, h].float(), v[:, h].float()
        for a in range(0, n, step):
            b = min(n, a + step)
            qh = q[a:b, h * G:(h + 1) * G].float().reshape((b - a) * G, D)
            x = (qh @ kh.t()) * scale
            lim = torch.arange(a, b, device=q.device).repeat_interleave(G) + off
            x.masked_fill_(torch.arange(m, device=q.device)[None, :] > lim[:, None], float("-inf"))
            top = x.amax(-1, keepdim=True)
            x = torch.exp(x - top)
            z = x.sum(-1, keepdim=True)
            out[a:b, h * G:(h + 1) * G] = ((x @ vh) / z).reshape(b - a, G, D).to(out.dtype)
            if lse is not None:
                lse[a:b, h * G:(h + 1) * G] = (top + torch.log(z)).reshape(b - a, G)


def _outputs(s):
    q = s["q"]
    return torch.zeros_like(q), (torch.zeros(q.shape[:2], device=q.device) if s["case"]["lse"] else None)


def _plain_attention(s):
    c = s["case"]
    out, lse = _outputs(s)
    o = 0
    for n in _lengths(c)[0]:
        e = o + n
        _attend(s["q"][o:e], s["k"][o:e], s["v"][o:e], 0, c["head_dim"] ** -0.5, out[o:e],
                None if lse is None else lse[o:e])
        o = e
    return out if lse is None else (out, lse)


def _gather(pages, row, total, layout):
    t = pages[row]
    if layout == "HND":
        t = t.transpose(1, 2)
    return t.reshape(-1, t.shape[2], t.shape[3])[:total]


def _plain_paged(s):
    c = s["case"]
    out, lse = _outputs(s)
    o = 0
    for r, (n, before) in enumerate(zip(*_lengths(c))):
        e, total = o + n, before + n
        row = s["table"][r, :-(-total // c["page"])].long()
        _attend(s["q"][o:e], _gather(s["k_pages"], row, total, c["layout"]),
                _gather(s["v_pages"], row, total, c["layout"]), before, c["head_dim"] ** -0.5, out[o:e],
                None if lse is None else lse[o:e])
        o = e
    return out if lse is None else (out, lse)


def _positions(s):
    """The request and the position of every packed token."""
    cu, lens = s["cu"].long(), s["seq_lens"].long()
    n = s["qkv"].shape[0]
    tok = torch.arange(n, device=DEV)
    req = torch.searchsorted(cu[1:], tok, right=True)
    return req, lens[req] - (cu[req + 1] - tok)


def _plain_prologue(s, eps=1e-6, theta=1e6):
    c = s["case"]
    Hq, Hkv, D, P = c["heads"], c["kv_heads"], c["head_dim"], c["page"]
    req, pos = _positions(s)
    freq = theta ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    ang = pos.double()[:, None] * freq
    cs, sn = torch.cos(ang).float()[:, None], torch.sin(ang).float()[:, None]

    def rotate(x, w):
        x = x.float()
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w
        a, b = x[..., :D // 2], x[..., D // 2:]
        return torch.cat([a * cs - b * sn, b * cs + a * sn], -1)

    q = rotate(s["qkv"][:, :Hq], s["q_norm_w"]).to(torch.bfloat16)
    k = rotate(s["qkv"][:, Hq:Hq + Hkv], s["k_norm_w"])
    v = s["qkv"][:, Hq + Hkv:]
    page, slot = s["table"][req, pos // P].long(), pos % P
    for which, x in (("k", k), ("v", v)):
        dst = s[which + "_pages"]
        if c["kv"] == "e4m3":
            x = (x.float() / s[which + "_scale"][:, None]).clamp(-E4M3_MAX, E4M3_MAX)
        x = x.to(dst.dtype)
        if dst.dtype == torch.float8_e4m3fn:
            dst, x = dst.view(torch.uint8), x.view(torch.uint8)
        if c["layout"] == "HND":
            dst[page, :, slot] = x
        else:
            dst[page, slot] = x
    return q, k.to(torch.bfloat16), _values(s, "k"), _values(s, "v")


def _plain_verify(s):
    x, u, n = s["x"].long(), s["u"].double(), s["draft_lens"].long()
    Bn, T = x.shape
    rows = torch.arange(Bn, device=DEV)
    px = s["p"][:, :T].gather(2, x[..., None])[..., 0].double()
    qx = torch.ones_like(px) if s["q"] is None else s["q"].gather(2, x[..., None])[..., 0].double()
    ok = (u[:, :T] * qx < px) & (torch.arange(T, device=DEV) < n[:, None])
    a = ok.long().cumprod(1).sum(1)
    w = s["p"][rows, a].double()
    cut = a < n
    at = a.clamp(max=T - 1)
    if s["q"] is None:
        own_x = torch.arange(w.shape[1], device=DEV)[None, :] == x[rows, at][:, None]
        w = torch.where(cut[:, None] & own_x, torch.zeros_like(w), w)
    else:
        r = (w - s["q"][rows, at].double()).clamp(min=0)
        w = torch.where((cut & (r.sum(1) > 0))[:, None], r, w)
    cum = w.cumsum(1)
    new = (cum > u[:, T:] * cum[:, -1:]).long().argmax(1)
    idx = torch.arange(T + 1, device=DEV)[None, :]
    drafts = torch.cat([x, x[:, :1]], 1)
    tokens = torch.where(idx < a[:, None], drafts, torch.where(idx == a[:, None], new[:, None], -1))
    return tokens.to(torch.int32), a.to(torch.int32), (s["seq_lens"].long() - n + a).to(torch.int32)


def _copy(s, src, dst):
    for t in s["caches"]:
        t[dst] = t[src]


def _free(ref, count):
    """The lowest ``count`` free pages."""
    return torch.nonzero(ref == 0)[:count, 0]


def _plain_fork(s):
    c = s["case"]
    P, M, N = c["page"], c["max_pages"], c["num_pages"]
    par, table, lens = s["parents"].long(), s["table"], s["lens"].long()
    new_lens, new = lens[par], table[par].clone()
    rows = torch.arange(len(par), device=DEV)
    first = torch.full_like(lens, len(par)).scatter_reduce(0, par, rows, "amin")
    col = new_lens // P
    part = (new_lens % P != 0) & (rows != first[par])
    keep = torch.arange(M, device=DEV)[None, :] < ((new_lens + P - 1) // P)[:, None]
    new = torch.where(keep, new, -1)
    r = torch.nonzero(part)[:, 0]
    src = new[r, col[r]].long()
    new[r, col[r]] = -1
    ref = s["ref"].long()
    old = table[torch.arange(M, device=DEV)[None, :] < ((lens + P - 1) // P)[:, None]].long()
    ref = ref - torch.bincount(old, minlength=N) + torch.bincount(new[new >= 0].long(), minlength=N)
    dst = _free(ref, len(r))
    new[r, col[r]] = dst.to(new.dtype)
    ref[dst] = 1
    _copy(s, src, dst)
    return new, new_lens.to(torch.int32), ref.to(torch.int32), s["caches"]


def _plain_resize(s):
    c = s["case"]
    P, M, N = c["page"], c["max_pages"], c["num_pages"]
    old, want = s["lens"].long(), s["new_lens"].long()
    a, b = (old + P - 1) // P, (want + P - 1) // P
    cols = torch.arange(M, device=DEV)[None, :]
    new = s["table"].clone()
    gone = (cols >= b[:, None]) & (cols < a[:, None])
    ref = s["ref"].long() - torch.bincount(new[gone].long(), minlength=N)
    new[cols.expand_as(new) >= torch.minimum(a, b)[:, None]] = -1
    rows = torch.arange(len(old), device=DEV)
    at = (old // P).clamp(max=M - 1)
    last = new[rows, at].long()
    cow = (want > old) & (old % P != 0)
    cow = cow & (ref[last.clamp(min=0)] > 1)
    fresh = (cols >= a[:, None]) & (cols < b[:, None])
    fresh = fresh | (cow[:, None] & (cols == at[:, None]))
    where = torch.nonzero(fresh)  # request order, then column
    dst = _free(ref, len(where))
    src = last[cow]
    ref = ref - torch.bincount(src, minlength=N)
    new[where[:, 0], where[:, 1]] = dst.to(new.dtype)
    ref[dst] = 1
    _copy(s, src, new[rows[cow], at[cow]].long())
    return new, ref.to(torch.int32), s["caches"]


def _plain_compact(s):
    N = s["case"]["num_pages"]
    live = s["ref"] > 0
    n = int(live.sum())
    ids = torch.arange(N, device=DEV)
    src, dst = ids[live & (ids >= n)], ids[~live & (ids < n)]
    page_map = torch.where(live, ids, -1)
    page_map[src] = dst
    ref = s["ref"].clone()
    ref[dst] = s["ref"][src]
    ref[src] = 0
    t = s["table"]
    new = torch.where(t >= 0, page_map[t.clamp(min=0).long()], -1).to(torch.int32)
    _copy(s, src, dst)
    return new, ref, page_map.to(torch.int32), s["caches"]


# ------------------------------------------------------------------------------------ bytes and flops
def work(case):
    op = case["op"]
    if op in ("attention", "paged", "prologue"):
        (lens, ctx), Hq, Hkv, D = _lengths(case), case["heads"], case["kv_heads"], case["head_dim"]
        n = sum(lens)
        if op == "prologue":
            e = 1 if case["kv"] == "e4m3" else 2
            return {"bytes": n * D * (2 * (Hq + 2 * Hkv) + 2 * Hq + 2 * Hkv + 2 * e * Hkv),
                    "flops": n * D * (Hq + Hkv) * 8}
        pairs = sum(m * x + x * (x + 1) // 2 for x, m in zip(lens, ctx))
        kv = sum(x + m for x, m in zip(lens, ctx))
        return {"bytes": 2 * D * (2 * n * Hq + 2 * kv * Hkv) + (4 * n * Hq if case["lse"] else 0),
                "flops": 4 * D * Hq * pairs}
    if op == "verify":
        e = 4 if case["dtype"] == "fp32" else 2
        rows = 1 if case["onehot"] else 2
        return {"bytes": case["batch"] * case["vocab"] * e * rows, "flops": case["batch"] * case["vocab"] * 3}
    # expected values; the tables and counts are read and written once
    Bn, M, N, P = case["batch"], case["max_pages"], case["num_pages"], case["page"]
    page = 2 * P * case["kv_heads"] * case["head_dim"] * 2 * case["layers"]
    small = 8 * (Bn * M + N)
    pages = min(Bn * (case["max_len"] // (2 * P) + 1), N * 3 // 4)
    moves = {"fork": Bn * 3 // 4, "resize": Bn // 20, "compact": pages * (N - pages) // N}[op]
    return {"bytes": small + 2 * page * moves, "flops": Bn * M + N}


# ------------------------------------------------------------------------------------ exact
def exact(case, seed):
    """What ``run`` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op = case["op"]
    if op in ("attention", "paged"):
        return _exact_attention(case, s)
    if op == "prologue":
        return _exact_prologue(case, s)
    if op == "verify":
        return _exact_verify(case, s)
    return _exact_pages(case, s)


def _exact_attention(case, s):
    (lens, ctx), Hq, Hkv, D = _lengths(case), case["heads"], case["kv_heads"], case["head_dim"]
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["q"].shape[:2], dtype=torch.float64, device=DEV)
    o = 0
    for r, n in enumerate(lens):
        m = n + ctx[r]
        if case["op"] == "paged":
            ids = s["table"][r].tolist()
            P = case["page"]
            where = [(ids[t // P], t % P) for t in range(0, m, P)]
            hnd = case["layout"] == "HND"
            k = torch.cat([(s["k_pages"][p] if hnd else s["k_pages"][p].transpose(0, 1)) for p, _ in where], 1)[:, :m]
            v = torch.cat([(s["v_pages"][p] if hnd else s["v_pages"][p].transpose(0, 1)) for p, _ in where], 1)[:, :m]
        else:
            k, v = s["k"][o:o + n].transpose(0, 1), s["v"][o:o + n].transpose(0, 1)
        step = max(1, (1 << 28) // m)
        for h in range(Hq):
            kk, vv = k[h * Hkv // Hq].double(), v[h * Hkv // Hq].double()
            for a in range(0, n, step):
                b = min(n, a + step)
                z = s["q"][o + a:o + b, h].double() @ kk.mT / math.sqrt(D)
                z = z.masked_fill(torch.ones_like(z, dtype=torch.bool).triu(a + ctx[r] + 1), -math.inf)
                ls = torch.logsumexp(z, 1)
                out[o + a:o + b, h] = torch.exp(z - ls[:, None]) @ vv
                lse[o + a:o + b, h] = ls
        o += n
    return (out, lse) if case["lse"] else out


def _e4m3(y):
    """The E4M3 value nearest to y, ties to even, saturating: 3 mantissa bits, exponents from -6."""
    step = torch.exp2(torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX)


def _exact_prologue(case, s):
    Hq, Hkv, D, P = case["heads"], case["kv_heads"], case["head_dim"], case["page"]
    x = s["qkv"].double()
    where, pos = [], []
    table = s["table"].tolist()
    for r, (n, before) in enumerate(zip(*_lengths(case))):
        for t in range(before, before + n):
            pos.append(t)
            where.append((table[r][t // P], t % P))
    pos = torch.tensor(pos, dtype=torch.float64, device=DEV)
    x[:, :Hq] *= s["q_norm_w"].double()
    x[:, Hq:Hq + Hkv] *= s["k_norm_w"].double()
    ms = s["qkv"].double().square().mean(-1, keepdim=True)
    x[:, :Hq + Hkv] /= torch.sqrt(ms[:, :Hq + Hkv] + 1e-6)
    i = torch.arange(D // 2, device=DEV, dtype=torch.float64)
    turn = torch.polar(torch.ones((len(pos), D // 2), dtype=torch.float64, device=DEV),
                       pos[:, None] * torch.exp(-2.0 * i / D * math.log(1e6)))[:, None]
    z = torch.complex(x[:, :Hq + Hkv, :D // 2].contiguous(), x[:, :Hq + Hkv, D // 2:].contiguous()) * turn
    x[:, :Hq + Hkv] = torch.cat([z.real, z.imag], -1)
    page = torch.tensor([a for a, _ in where], device=DEV)
    slot = torch.tensor([b for _, b in where], device=DEV)
    caches = []
    for which, lo in (("k", Hq), ("v", Hq + Hkv)):
        y = x[:, lo:lo + Hkv]
        full = torch.zeros(s[which + "_pages"].shape, dtype=torch.float64, device=DEV)
        if case["kv"] == "e4m3":
            y = _e4m3(y / s[which + "_scale"].double()[:, None])
        if case["layout"] == "HND":
            full[page, :, slot] = y
        else:
            full[page, slot] = y
        caches.append(full)
    return x[:, :Hq].clone(), x[:, Hq:Hq + Hkv].clone(), caches[0], caches[1]


def _exact_verify(case, s):
    Bn, T = case["batch"], case["drafts"]
    x, u, n = s["x"].tolist(), s["u"].tolist(), s["draft_lens"].tolist()
    tokens = np.full((Bn, T + 1), -1, dtype=np.int32)
    acc = np.zeros(Bn, dtype=np.int32)
    for r in range(Bn):
        p = s["p"][r].double().cpu().numpy()
        q = None if s["q"] is None else s["q"][r].double().cpu().numpy()
        t = 0
        while t < n[r]:
            d = x[r][t]
            if not u[r][t] * (1.0 if q is None else q[t][d]) < p[t][d]:
                break
            tokens[r, t] = d
            t += 1
        w = p[t].copy()
        if t < n[r]:
            if q is None:
                w[x[r][t]] = 0.0
            else:
                rest = np.maximum(p[t] - q[t], 0.0)
                w = rest if rest.sum() > 0 else w
        cum = np.cumsum(w)
        tokens[r, t] = int(np.searchsorted(cum, u[r][T] * cum[-1], side="right"))
        acc[r] = t
    new = s["seq_lens"].cpu().numpy() - np.array(n) + acc
    return (torch.from_numpy(tokens).to(DEV), torch.from_numpy(acc).to(DEV),
            torch.from_numpy(new.astype(np.int32)).to(DEV))


def _exact_pages(case, s):
    """Request by request on the host."""
    op, P, N = case["op"], case["page"], case["num_pages"]
    table, lens, ref = s["table"].tolist(), s["lens"].tolist(), s["ref"].tolist()
    caches, moves = s["caches"], []
    i32 = dict(dtype=torch.int32, device=DEV)

    def held(n):
        return -(-n // P)

    def lowest(count):
        return [p for p in range(N) if ref[p] == 0][:count]

    if op == "fork":
        par = s["parents"].tolist()
        rows, out_lens, seen, want = [], [], set(), []
        for r, n in enumerate(lens):
            for j in range(held(n)):
                ref[table[r][j]] -= 1
        for r, f in enumerate(par):
            n = lens[f]
            row = [table[f][j] if j < held(n) else -1 for j in range(len(table[f]))]
            if n % P and f in seen:
                want.append((r, n // P, row[n // P]))
                row[n // P] = -1
            seen.add(f)
            for p in row:
                if p >= 0:
                    ref[p] += 1
            rows.append(row)
            out_lens.append(n)
        for (r, j, src), dst in zip(want, lowest(len(want))):
            rows[r][j] = dst
            ref[dst] = 1
            moves.append((src, dst))
        result = [torch.tensor(rows, **i32), torch.tensor(out_lens, **i32), torch.tensor(ref, **i32)]
    elif op == "resize":
        new, want = s["new_lens"].tolist(), []
        for r, n in enumerate(lens):
            for j in range(held(new[r]), held(n)):
                ref[table[r][j]] -= 1
                table[r][j] = -1
        for r, n in enumerate(lens):
            if new[r] > n and n % P and ref[table[r][n // P]] > 1:
                want.append((r, n // P, table[r][n // P]))
            want += [(r, j, -1) for j in range(held(n), held(new[r]))]
        take = lowest(len(want))
        for (r, j, src), dst in zip(want, take):
            if src >= 0:
                ref[src] -= 1
                moves.append((src, dst))
            table[r][j] = dst
            ref[dst] = 1
        result = [torch.tensor(table, **i32), torch.tensor(ref, **i32)]
    else:
        live = [p for p in range(N) if ref[p] > 0]
        n = len(live)
        to = {p: p for p in live}
        moves = list(zip([p for p in live if p >= n], [p for p in range(n) if ref[p] == 0]))
        for a, b in moves:
            to[a] = b
            ref[b], ref[a] = ref[a], 0
        result = [torch.tensor([[to.get(p, -1) for p in row] for row in table], **i32), torch.tensor(ref, **i32),
                  torch.tensor([to.get(p, -1) for p in range(N)], **i32)]
    if moves:
        a, b = (torch.tensor(t, device=DEV) for t in zip(*moves))
        for t in caches:
            t[b] = t[a]
    return (*result, caches)
