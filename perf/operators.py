"""Cases for the softmax operators that stand beside the recurrent scans: windowed attention (forward, and forward
with its backward pass), one decode step over a paged key-value cache, and the cache's own upkeep (append, fork,
compact).  ``run`` computes the plain form in elementary torch operations, or, where ``own`` is true, makes the
library's calls.

Shapes: q [B, H, L, d], k and v [B, Hkv, L, d] (head h reads k/v head h // (H / Hkv)); a page holds ``page`` tokens
of every k/v head, [num_pages, Hkv, page, d].  Token t sees token j when j <= t and (j > t - window or j < sinks).
"""

import math
import random

import torch

own = False

DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # a short prompt in front of an interactive session: latency
        dict(name="attn-short", kind="attn", dtype="bf16", B=1, H=4, Hkv=4, L=96, d=64, window=32, sinks=4, ragged=False),
        # prefill of a local-attention layer with shared k/v heads
        dict(name="attn-prefill", kind="attn", dtype="bf16", B=4, H=16, Hkv=4, L=4096, d=128, window=1024, sinks=4,
             ragged=False),
        # a padded batch in single precision (evaluation against a reference)
        dict(name="attn-ragged-f32", kind="attn", dtype="f32", B=3, H=8, Hkv=8, L=1531, d=64, window=257, sinks=16,
             ragged=True),
        # a training step of one layer
        dict(name="train-layer", kind="train", dtype="bf16", B=2, H=16, Hkv=4, L=4096, d=128, window=1024, sinks=4,
             ragged=False),
        # a training step on a padded batch, narrow heads
        dict(name="train-ragged", kind="train", dtype="bf16", B=4, H=8, Hkv=2, L=2047, d=64, window=512, sinks=8,
             ragged=True),
        # a small single-precision step, as in a gradient check or a toy run
        dict(name="train-small-f32", kind="train", dtype="f32", B=2, H=4, Hkv=4, L=515, d=32, window=128, sinks=1,
             ragged=False),
        # one user, a short cache: latency
        dict(name="step-one", kind="step", dtype="bf16", B=1, H=8, Hkv=2, d=128, page=16, most=200, window=0, sinks=0),
        # a serving batch with caches of all lengths
        dict(name="step-batch", kind="step", dtype="bf16", B=64, H=32, Hkv=8, d=128, page=64, most=8192, window=0,
             sinks=0),
        # one sequence with a very long cache: only splitting the length fills the GPU
        dict(name="step-long", kind="step", dtype="bf16", B=1, H=16, Hkv=2, d=128, page=16, most=131071, window=0,
             sinks=0),
        # every serving step: one new token per sequence goes into the pages
        dict(name="append-step", kind="append", dtype="bf16", rows=128, tokens=1, Hkv=8, d=128, page=64, most=2048),
        # a beam step: every kept hypothesis continues from a shared prefix
        dict(name="fork-beams", kind="fork", dtype="bf16", rows=96, forks=64, Hkv=8, d=128, page=64, most=2048),
        # defragmentation after many sequences have ended
        dict(name="compact-pool", kind="compact", dtype="bf16", rows=96, Hkv=8, d=128, page=16, pages=8192, most=768),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(["attn", "attn", "train", "train", "step", "step", "append", "fork", "compact"])
    if kind in ("attn", "train"):
        dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
        Hkv, group = rng.choice([1, 2, 4]), rng.choice([1, 2, 3, 4])
        L = _log(rng, 1, 4096 if dtype == "bf16" else 1600)
        return dict(kind=kind, dtype=dtype, B=rng.randint(1, 3 if dtype == "bf16" else 2), H=Hkv * group, Hkv=Hkv, L=L,
                    d=rng.choice([64, 128]) if dtype == "bf16" else rng.choice([32, 64, 128]), window=_log(rng, 1, 2048),
                    sinks=rng.choice([0, 1, 4, 17, 64]), ragged=rng.random() < 0.5)
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind == "step":
        B, Hkv = _log(rng, 1, 64), rng.choice([1, 2, 4, 8])
        most = _log(rng, 1, min(131072, (1 << 21) // (B * Hkv)))
        return dict(kind=kind, dtype=dtype, B=B, H=Hkv * rng.choice([1, 2, 4, 5, 8]), Hkv=Hkv, d=rng.choice([64, 128]),
                    page=rng.choice([16, 32, 64, 128]), most=most, window=rng.choice([0, 0, _log(rng, 1, most)]),
                    sinks=rng.choice([0, 4, 33]))
    case = dict(kind=kind, dtype=dtype, rows=_log(rng, 2, 128), Hkv=rng.choice([1, 2, 4, 8]), d=rng.choice([64, 128]),
                page=rng.choice([16, 32, 64]), most=_log(rng, 1, 1500))
    if kind == "append":
        case["tokens"] = rng.choice([1, 1, _log(rng, 2, 200)])
    elif kind == "fork":
        case["forks"] = rng.randint(1, case["rows"] - 1)
    else:
        used = case["rows"] * -(-case["most"] // case["page"])
        case["pages"] = used + _log(rng, 1, 2 * used + 2)
    return case


def _lens(case):
    """Tokens per sequence, fixed by the case: of all lengths up to the largest, which occurs."""
    if case["kind"] in ("attn", "train"):
        n, most = case["B"], case["L"]
        if not case["ragged"]:
            return [most] * n
    else:
        n, most = case.get("rows", case.get("B")), case["most"]
    rng = random.Random("lengths %d %d" % (n, most))
    return [most] + [rng.randint(0 if case["kind"] in ("step", "attn", "train") else 1, most) for _ in range(n - 1)]


def _seen(n, window, sinks):
    """Number of (query, key) pairs a sequence of n tokens has."""
    w = min(window, n)
    pairs = w * (w + 1) // 2 + (n - w) * w
    # query t >= window also sees the sinks that have left its window: min(sinks, t - window + 1) of them
    far = max(0, n - window)
    s = min(sinks, far)
    return pairs + s * (s + 1) // 2 + (far - s) * s


def _size(case):
    return 2 if case["dtype"] == "bf16" else 4


def work(case):
    e, d, Hkv, lens = _size(case), case["d"], case["Hkv"], _lens(case)
    if case["kind"] in ("attn", "train"):
        H, n = case["H"], sum(lens)
        pairs = H * sum(_seen(x, case["window"], case["sinks"]) for x in lens)
        fwd = e * d * n * (2 * H + 2 * Hkv) + 4 * n * H
        if case["kind"] == "attn":
            return {"bytes": fwd, "flops": 4 * d * pairs}
        return {"bytes": fwd + e * d * n * (2 * H + 2 * Hkv), "flops": 14 * d * pairs}
    if case["kind"] == "step":
        w, s = case["window"], case["sinks"]
        seen = sum(x if not w else min(w, x) + min(s, max(0, x - w)) for x in lens)
        return {"bytes": 2 * e * d * Hkv * seen + case["B"] * case["H"] * (2 * e * d + 4), "flops": 4 * d * case["H"] * seen}
    token = 2 * e * Hkv * d  # bytes of one token's keys and values
    meta = 4 * (case["rows"] * 2 + _pool(case)[0])
    if case["kind"] == "append":
        return {"bytes": 2 * token * case["rows"] * case["tokens"] + meta, "flops": 0}
    if case["kind"] == "fork":
        moved = sum(x % case["page"] != 0 for x in (lens[i] for i in _forks(case)[0]))
        return {"bytes": 2 * token * case["page"] * moved + meta, "flops": 0}
    used = sum(-(-x // case["page"]) for x in lens)
    # pages in use are spread evenly over the pool: the share behind the first `used` has to move
    moved = used * (case["pages"] - used) // case["pages"]
    return {"bytes": 2 * token * case["page"] * moved + meta, "flops": 0}


# ------------------------------------------------------------------------------------------------ inputs

def _forks(case):
    """Source and destination rows of a fork: the sources are taken with repetition, as beams share a parent."""
    rng = random.Random("forks %d %d" % (case["rows"], case["forks"]))
    held = case["rows"] - case["forks"]
    return [rng.randrange(held) for _ in range(case["forks"])], list(range(held, case["rows"]))


def _pool(case):
    """(pages of the pool, entries of a table row)."""
    page, lens = case["page"], _lens(case)
    used = sum(-(-x // page) for x in lens)
    if case["kind"] == "append":
        most = -(-(case["most"] + case["tokens"]) // page)
        return case["rows"] * most, most
    most = -(-case["most"] // page)
    if case["kind"] == "fork":
        return used + case["forks"], most
    if case["kind"] == "compact":
        return case["pages"], most
    return used + 3, max(1, most)


def _normal(g, dtype, *shape):
    x = torch.empty(*shape, device=DEV, dtype=dtype)
    return x.normal_(generator=g)


def prepare(case, seed):
    g = torch.Generator(device=DEV).manual_seed(seed)
    dtype, d, Hkv, lens = DTYPES[case["dtype"]], case["d"], case["Hkv"], _lens(case)
    st = {"case": case}
    if case["kind"] in ("attn", "train"):
        B, H, L = case["B"], case["H"], case["L"]
        st["q"], st["k"], st["v"] = (_normal(g, dtype, B, h, L, d) for h in (H, Hkv, Hkv))
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV) if case["ragged"] else None
        if case["kind"] == "train":
            st["dO"] = _normal(g, dtype, B, H, L, d)
        return st
    page = case["page"]
    num, most = _pool(case)
    rows = len(lens)
    if case["kind"] == "fork":  # the destination rows hold nothing yet
        lens = [n if i < rows - case["forks"] else 0 for i, n in enumerate(lens)]
    st["k_pages"], st["v_pages"] = _normal(g, dtype, num, Hkv, page, d), _normal(g, dtype, num, Hkv, page, d)
    # the rows' pages are scattered over the pool, as after a while of serving
    scatter = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).tolist()
    table, refs, at = [[-1] * most for _ in range(rows)], [0] * num, 0
    for r, n in enumerate(lens):
        for i in range(-(-n // page)):
            table[r][i], refs[scatter[at]], at = scatter[at], 1, at + 1
    st["table"] = torch.tensor(table, dtype=torch.int32, device=DEV)
    st["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
    st["refs"] = torch.tensor(refs, dtype=torch.int32, device=DEV)
    if case["kind"] == "step":
        st["q"] = _normal(g, dtype, case["B"], case["H"], d)
    elif case["kind"] == "append":
        st["rows"] = torch.arange(rows, dtype=torch.int32, device=DEV)
        st["k"], st["v"] = (_normal(g, dtype, rows, Hkv, case["tokens"], d) for _ in range(2))
    elif case["kind"] == "fork":
        src, dst = _forks(case)
        st["src"], st["dst"] = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in (src, dst))
    return st


# ------------------------------------------------------------------------------------------------ the library's calls

def _run_own(st):
    from delta_rule_recurrent_scan_b200 import kdn

    case = st["case"]
    if case["kind"] == "attn":
        o, lse = kdn.window_attn(st["q"], st["k"], st["v"], case["window"], n_sink=case["sinks"], lens=st["lens"])
        return {"o": o, "lse": lse}
    if case["kind"] == "train":
        o, lse = kdn.window_attn(st["q"], st["k"], st["v"], case["window"], n_sink=case["sinks"], lens=st["lens"])
        g = kdn.window_attn_backward(st["q"], st["k"], st["v"], o, lse, st["dO"], case["window"], n_sink=case["sinks"],
                                     lens=st["lens"])
        return {"o": o, "lse": lse, "dq": g["dq"], "dk": g["dk"], "dv": g["dv"]}
    if case["kind"] == "step":
        o, lse = kdn.paged_attn_step(st["q"], st["k_pages"], st["v_pages"], st["table"], st["lens"],
                                     window=case["window"], n_sink=case["sinks"])
        return {"o": o, "lse": lse}
    # a pass starts from the same books each time; the pages are the state's own
    pages = kdn.Pages(st["table"].clone(), st["lens"].clone(), st["refs"].clone(), case["page"])
    if case["kind"] == "append":
        kdn.pages_reserve(pages, st["rows"], case["tokens"])
        kdn.pages_write(pages, st["rows"], st["k"], st["v"], st["k_pages"], st["v_pages"])
    elif case["kind"] == "fork":
        moves = kdn.pages_fork(pages, st["src"], st["dst"])
        kdn.pages_copy(moves, st["k_pages"], st["v_pages"])
    else:
        moves = kdn.pages_compact(pages)
        kdn.pages_copy(moves, st["k_pages"], st["v_pages"])
    return {"table": pages.table, "lens": pages.lens, "refs": pages.refs, "k_pages": st["k_pages"],
            "v_pages": st["v_pages"]}


# ------------------------------------------------------------------------------------------------ the plain forms

def _attend(st):
    """(heads grouped by k/v head: q, k, v in 32 bits; P [B, Hkv, G, L, L]; o; lse; which rows exist)."""
    case = st["case"]
    B, H, Hkv, L, d = (case[x] for x in ("B", "H", "Hkv", "L", "d"))
    q = st["q"].float().view(B, Hkv, H // Hkv, L, d)
    k, v = st["k"].float().unsqueeze(2), st["v"].float().unsqueeze(2)
    t = torch.arange(L, device=DEV)
    j = t[None, :]
    seen = (j <= t[:, None]) & ((j > t[:, None] - case["window"]) | (j < case["sinks"]))
    s = torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    p = p.div_(total)
    lse = (top + total.log()).squeeze(-1)
    o = torch.matmul(p, v)
    live = t[None, :] < st["lens"][:, None] if st["lens"] is not None else None
    if live is not None:
        live = live[:, None, None, :]
        lse = torch.where(live, lse, 0.0)
        o = torch.where(live[..., None], o, 0.0)
    return q, k, v, p, o, lse, live


def _free_first(refs):
    """Page numbers with the free ones first, in rising order."""
    return torch.sort((refs != 0).int(), stable=True).indices


def _run_plain(st):
    case = st["case"]
    if case["kind"] in ("attn", "train"):
        q, k, v, p, o, lse, live = _attend(st)
        dtype = st["q"].dtype
        out = {"o": o.flatten(1, 2).to(dtype), "lse": lse.flatten(1, 2)}
        if case["kind"] == "attn":
            return out
        dO = st["dO"].float().view(o.shape)
        if live is not None:
            dO = torch.where(live[..., None], dO, 0.0)
        dv = torch.matmul(p.transpose(-1, -2), dO).sum(2)
        ds = torch.matmul(dO, v.transpose(-1, -2)).sub_((dO * o).sum(-1, keepdim=True)).mul_(p)
        dq = torch.matmul(ds, k) * case["d"] ** -0.5
        dk = torch.matmul(ds.transpose(-1, -2), q).sum(2) * case["d"] ** -0.5
        return {**out, "dq": dq.flatten(1, 2).to(dtype), "dk": dk.to(dtype), "dv": dv.to(dtype)}
    page = case["page"]
    if case["kind"] == "step":
        B, H, Hkv, d = (case[x] for x in ("B", "H", "Hkv", "d"))
        table, n = st["table"].long().clamp(min=0), st["lens"].long()[:, None]
        # [B, entries, Hkv, page, d] -> [B, Hkv, tokens, d]
        k, v = (x[table].transpose(1, 2).flatten(2, 3).float() for x in (st["k_pages"], st["v_pages"]))
        j = torch.arange(k.shape[2], device=DEV)[None, :]
        seen = j < n
        if case["window"]:
            seen = seen & ((j > n - 1 - case["window"]) | (j < case["sinks"]))
        seen = seen[:, None, None, :]
        q = st["q"].float().view(B, Hkv, H // Hkv, d)
        s = (torch.matmul(q, k.transpose(-1, -2)) * d ** -0.5).masked_fill_(~seen, -math.inf)
        top = s.amax(-1, keepdim=True)
        top = torch.where(top == -math.inf, 0.0, top)
        p = (s - top).exp()
        total = p.sum(-1, keepdim=True)
        o = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
        lse = (top + total.log()).squeeze(-1)
        return {"o": o.flatten(1, 2).to(st["q"].dtype), "lse": lse.flatten(1, 2)}
    table, lens, refs = (st[x].long() for x in ("table", "lens", "refs"))
    if case["kind"] == "append":
        rows, T = st["rows"].long(), case["tokens"]
        had, has = (lens[rows] + page - 1) // page, (lens[rows] + T + page - 1) // page
        need = has - had
        before = need.cumsum(0) - need
        order = _free_first(refs)
        e = torch.arange(table.shape[1], device=DEV)[None, :]
        fresh = (e >= had[:, None]) & (e < has[:, None])
        pick = order[(before[:, None] + e - had[:, None]).clamp(0, refs.numel() - 1)]
        table = table.index_put((rows,), torch.where(fresh, pick, table[rows]))
        refs = refs.scatter_add(0, order, (torch.arange(refs.numel(), device=DEV) < need.sum()).long())
        at = lens[rows][:, None] + torch.arange(T, device=DEV)[None, :]
        where = torch.gather(table[rows], 1, at // page)
        st["k_pages"][where, :, at % page] = st["k"].transpose(1, 2)
        st["v_pages"][where, :, at % page] = st["v"].transpose(1, 2)
        lens = lens.index_put((rows,), lens[rows] + T)
    elif case["kind"] == "fork":
        src, dst = st["src"].long(), st["dst"].long()
        n = lens[src]
        part = n % page != 0
        last = torch.gather(table[src], 1, (n // page).clamp(max=table.shape[1] - 1)[:, None])[:, 0]
        new = _free_first(refs)[(part.long().cumsum(0) - 1).clamp(min=0)]
        entries = table[src]
        e = torch.arange(table.shape[1], device=DEV)[None, :]
        entries = torch.where(part[:, None] & (e == (n // page)[:, None]), new[:, None], entries)
        refs = refs.index_add(0, entries.clamp(min=0).flatten(), (entries >= 0).long().flatten())
        table, lens = table.index_put((dst,), entries), lens.index_put((dst,), n)
        # a row without a part-filled page copies its first page onto itself
        a = torch.where(part, last, table[src][:, 0])
        b = torch.where(part, new, table[src][:, 0])
        st["k_pages"][b] = st["k_pages"][a]
        st["v_pages"][b] = st["v_pages"][a]
    else:
        num = refs.numel()
        at = torch.arange(num, device=DEV)
        used = refs > 0
        count = used.sum()
        hole, mover = ~used & (at < count), used & (at >= count)
        holes, movers = (torch.sort(x.int(), stable=True, descending=True).indices for x in (hole, mover))
        # at most half the pages move, the i-th mover into the i-th hole; the rest of the list stays in place
        dst = holes[:num // 2]
        moves = at[:num // 2] < mover.sum()
        src = torch.where(moves, movers[:num // 2], dst)
        to = torch.arange(num + 1, device=DEV).scatter(0, torch.where(moves, movers[:num // 2], num), dst)
        refs = torch.where(at < count, refs.scatter(0, dst, refs[src]), 0)
        table = torch.where(table >= 0, to[table.clamp(min=0)], table)
        st["k_pages"][dst] = st["k_pages"][src]
        st["v_pages"][dst] = st["v_pages"][src]
    return {"table": table.int(), "lens": lens.int(), "refs": refs.int(), "k_pages": st["k_pages"],
            "v_pages": st["v_pages"]}


def run(state):
    if own:
        return _run_own(state)
    else:
        return _run_plain(state)


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    """From the definitions: softmax over each row's visible keys in 64 bits, its gradients by differentiation; the
    cache's books by walking the rows in order."""
    st = prepare(case, seed)
    if case["kind"] in ("attn", "train"):
        B, H, Hkv, L, d = (case[x] for x in ("B", "H", "Hkv", "L", "d"))
        train = case["kind"] == "train"
        zeros = lambda h, *more: torch.zeros(B, h, L, *more, dtype=torch.float64, device=DEV)  # noqa: E731
        out = {"o": zeros(H, d), "lse": zeros(H)}
        if train:
            out.update(dq=zeros(H, d), dk=zeros(Hkv, d), dv=zeros(Hkv, d))
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            back = torch.arange(n, device=DEV)[:, None] - torch.arange(n, device=DEV)  # how far key j lies behind
            hidden = (back < 0) | ((back >= case["window"]) & (torch.arange(n, device=DEV) >= case["sinks"]))
            for h in range(H):
                kv = h * Hkv // H
                q, k, v = (x[b, i, :n].double().requires_grad_(train)
                           for x, i in ((st["q"], h), (st["k"], kv), (st["v"], kv)))
                logits = torch.where(hidden, -math.inf, q @ k.T / math.sqrt(d))
                o = torch.softmax(logits, -1) @ v
                out["o"][b, h, :n], out["lse"][b, h, :n] = o.detach(), torch.logsumexp(logits, -1).detach()
                if train:
                    dq, dk, dv = torch.autograd.grad(o, (q, k, v), st["dO"][b, h, :n].double())
                    out["dq"][b, h, :n] = dq
                    out["dk"][b, kv, :n] += dk
                    out["dv"][b, kv, :n] += dv
        return out
    page = case["page"]
    if case["kind"] == "step":
        B, H, Hkv, d = (case[x] for x in ("B", "H", "Hkv", "d"))
        o = torch.zeros(B, H, d, dtype=torch.float64, device=DEV)
        lse = torch.full((B, H), -math.inf, dtype=torch.float64, device=DEV)
        for b, n in enumerate(_lens(case)):
            if n == 0:
                continue
            seen = [j for j in range(n) if not case["window"] or n - 1 - j < case["window"] or j < case["sinks"]]
            seen = torch.tensor(seen, device=DEV)
            where = st["table"][b].long()[seen // page]
            for h in range(H):
                kv = h * Hkv // H
                k, v = (x[where, kv, seen % page].double() for x in (st["k_pages"], st["v_pages"]))
                logits = k @ st["q"][b, h].double() / math.sqrt(d)
                o[b, h], lse[b, h] = torch.softmax(logits, 0) @ v, torch.logsumexp(logits, 0)
        return {"o": o, "lse": lse}
    table, lens, refs = (st[x].tolist() for x in ("table", "lens", "refs"))
    free = [i for i, n in enumerate(refs) if n == 0]
    kp, vp = st["k_pages"].double(), st["v_pages"].double()
    if case["kind"] == "append":
        for r in st["rows"].tolist():
            for t in range(case["tokens"]):
                if lens[r] % page == 0:
                    table[r][lens[r] // page] = free.pop(0)
                    refs[table[r][lens[r] // page]] = 1
                kp[table[r][lens[r] // page], :, lens[r] % page] = st["k"][r, :, t].double()
                vp[table[r][lens[r] // page], :, lens[r] % page] = st["v"][r, :, t].double()
                lens[r] += 1
    elif case["kind"] == "fork":
        for a, b in zip(st["src"].tolist(), st["dst"].tolist()):
            lens[b] = lens[a]
            for i in range(-(-lens[a] // page)):
                p = table[a][i]
                if (i + 1) * page > lens[a]:
                    p = free.pop(0)
                    kp[p], vp[p] = kp[table[a][i]], vp[table[a][i]]
                table[b][i] = p
                refs[p] += 1
    else:
        used = sum(n > 0 for n in refs)
        to = {p: h for p, h in zip([i for i, n in enumerate(refs) if n and i >= used], free)}
        for p, h in to.items():
            kp[h], vp[h], refs[h], refs[p] = kp[p], vp[p], refs[p], 0
        table = [[to.get(p, p) for p in row] for row in table]
    whole = lambda x: torch.tensor(x, dtype=torch.int32, device=DEV)  # noqa: E731
    return {"table": whole(table), "lens": whole(lens), "refs": whole(refs), "k_pages": kp, "v_pages": vp}
