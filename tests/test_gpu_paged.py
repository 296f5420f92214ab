"""The paged key-value cache and the decode step that reads it, on the GPU, against the float64 and plain-Python oracle."""

import random

import pytest
import torch

import oracle.attn as oa
from attn_ref import HALF, U
from delta_rule_recurrent_scan_b200 import kdn
from delta_rule_recurrent_scan_b200.workloads import WORKLOADS, make_scan_inputs

pytestmark = pytest.mark.gpu
DEV = "cuda"
STATUS = {"ok": kdn.KDN_OK, "invalid": kdn.KDN_ERR_INVALID_ARG, "capacity": kdn.KDN_ERR_CAPACITY}


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


# ------------------------------------------------------------------------------------------ decode step

def _cache(lens, Hkv, dk, dv, page, dtype, seed=0, spare=2, most=None):
    g = torch.Generator(device=DEV).manual_seed(seed)
    held = [-(-n // page) for n in lens]
    num = sum(held) + spare
    most = max([1, *held]) if most is None else most
    order = torch.randperm(num, generator=torch.Generator().manual_seed(seed)).tolist()
    table = [[-1] * most for _ in lens]
    for r, n in enumerate(held):
        for e in range(n):
            table[r][e] = order.pop()
    k = torch.randn(num, Hkv, page, dk, generator=g, device=DEV).to(dtype)
    v = torch.randn(num, Hkv, page, dv, generator=g, device=DEV).to(dtype)
    return k, v, _i32(table), _i32(lens), g


def _dense_step(q, k, v, table, lens, window, n_sink, scale, w, out):
    """Float64 result and the bound of attn_ref for one row (no heads shared between rows of the loop)."""
    n, H, dk = q.shape
    _, Hkv, page, dv = v.shape
    scale = dk ** -0.5 if scale is None else scale
    o, eo = torch.zeros(n, H, dv, dtype=torch.float64, device=DEV), torch.zeros(n, H, dv, dtype=torch.float64, device=DEV)
    lse, el = torch.full((n, H), -torch.inf, dtype=torch.float64, device=DEV), torch.zeros(n, H, dtype=torch.float64, device=DEV)
    for i in range(n):
        m = int(lens[i])
        if m == 0:
            continue
        j = torch.arange(m, device=DEV)
        if window:
            j = j[(j > m - 1 - window) | (j < n_sink)]
        at = table[i].long()[j // page]
        kk, vv = (x[at, :, j % page].double().transpose(0, 1).repeat_interleave(H // Hkv, 0) for x in (k, v))
        qq = q[i].double()[:, None]
        s = scale * (qq * kk).sum(-1)
        sabs = scale * (qq * kk).abs().sum(-1).amax(-1)
        lse[i] = torch.logsumexp(s, -1)
        p = torch.exp(s - lse[i][:, None])
        e_s, A = (dk + 4) * U * sabs, 2 * sabs
        e_p = 2 * e_s + (2 * A + len(j) + 16) * U
        o[i] = (p[:, None] @ vv)[:, 0]
        eo[i] = (e_p + w)[:, None] * (p[:, None] @ vv.abs())[:, 0] + out * o[i].abs()
        el[i] = e_s + (A + len(j) + 16) * U + 2 * U * lse[i].abs()
    return o, eo, lse, el


def _check_step(q, k, v, table, lens, window=0, n_sink=0, scale=None, rows=None, out_dtype=None):
    tc = q.dtype == torch.bfloat16 and q.shape[-1] == v.shape[-1] and q.shape[-1] in (64, 128)
    o, lse = kdn.paged_attn_step(q, k, v, table, lens, rows=rows, window=window, n_sink=n_sink, scale=scale, out_dtype=out_dtype)
    torch.cuda.synchronize()
    if rows is not None:
        table, lens = table[rows.long()], lens[rows.long()]
    # hi + lo pairs of bf16 keep a weight to 2^-16
    ro, eo, rl, el = _dense_step(q, k, v, table, lens, window, n_sink, scale, 2.0 ** -16 if tc else 0.0, HALF[o.dtype])
    empty = lens == 0
    assert bool((o[empty] == 0).all()) and bool((lse[empty] == -torch.inf).all())
    live = ~empty
    assert bool(((o.double() - ro).abs() <= eo)[live].all()), float(((o.double() - ro).abs() / (eo + 1e-300))[live].max())
    assert bool(((lse.double() - rl).abs() <= el)[live].all())
    return o, lse


CASES = [(torch.float32, 32), (torch.float32, 128), (torch.bfloat16, 64), (torch.bfloat16, 128)]


@pytest.mark.parametrize("dtype,d", CASES)
@pytest.mark.parametrize("page", [1, 8, 16, 64, 256])
def test_lengths_and_pages(dtype, d, page):
    lens = [1, 2, 15, 16, 17, 31, 33, 0, 63, 64, 65, 127, 129, 300, 1027]
    k, v, table, ln, g = _cache(lens, 2, d, d, page, dtype, seed=page)
    q = torch.randn(len(lens), 4, d, generator=g, device=DEV).to(dtype)
    _check_step(q, k, v, table, ln)


@pytest.mark.parametrize("dtype,d", CASES)
@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 1), (16, 4), (64, 33), (100, 130), (2000, 5), (2**31 - 1, 0)])
def test_windows(dtype, d, window, n_sink):
    lens = [1, 17, 64, 65, 100, 101, 333, 0, 1500]
    k, v, table, ln, g = _cache(lens, 1, d, d, 16, dtype, seed=1)
    q = torch.randn(len(lens), 3, d, generator=g, device=DEV).to(dtype)
    _check_step(q, k, v, table, ln, window=window, n_sink=n_sink)


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_sizes(dk, dv, dtype):
    k, v, table, ln, g = _cache([70, 1, 200], 2, dk, dv, 32, dtype, seed=2)
    q = torch.randn(3, 6, dk, generator=g, device=DEV).to(dtype)
    _check_step(q, k, v, table, ln)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (5, 1), (8, 1), (9, 1), (16, 1), (17, 1), (40, 2), (64, 1), (8, 8)])
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_shared_heads(H, Hkv, dtype, d):
    k, v, table, ln, g = _cache([513, 90], Hkv, d, d, 16, dtype, seed=3)
    q = torch.randn(2, H, d, generator=g, device=DEV).to(dtype)
    _check_step(q, k, v, table, ln)


@pytest.mark.parametrize("dtype,d", CASES)
def test_long_caches_are_split_and_joined(dtype, d):
    """One long sequence next to short ones and empty ones: parts without a token join too."""
    lens = [20001, 5, 0, 777]
    k, v, table, ln, g = _cache(lens, 1, d, d, 64, dtype, seed=4)
    q = torch.randn(4, 8, d, generator=g, device=DEV).to(dtype)
    a = _check_step(q, k, v, table, ln)
    b = _check_step(q, k, v, table, ln)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])  # a fixed order
    _check_step(q, k, v, table, ln, window=9000, n_sink=100)
    _check_step((q.float() * 30).to(dtype), k, v, table, ln)
    _check_step(q, k, v, table, ln, scale=2.0, out_dtype=torch.float32 if dtype == torch.bfloat16 else torch.bfloat16)


@pytest.mark.parametrize("dtype,d", CASES)
def test_what_lies_behind_a_length_takes_no_part(dtype, d):
    lens = [33, 1, 64, 130, 5000]
    k, v, table, ln, g = _cache(lens, 2, d, d, 16, dtype, seed=5, most=400)
    q = torch.randn(5, 4, d, generator=g, device=DEV).to(dtype)
    a = _check_step(q, k, v, table, ln)
    used = torch.zeros(k.shape[0], 16, dtype=torch.bool, device=DEV)
    for r, n in enumerate(lens):
        j = torch.arange(n, device=DEV)
        used[table[r].long()[j // 16], j % 16] = True
    for x in (k, v):
        x.masked_fill_(~used[:, None, :, None], float("nan"))
    b = _check_step(q, k, v, table, ln)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,d", CASES)
def test_chosen_rows_and_broken_entries(dtype, d):
    lens = [50, 0, 300, 20]
    k, v, table, ln, g = _cache(lens, 1, d, d, 16, dtype, seed=6)
    q = torch.randn(5, 4, d, generator=g, device=DEV).to(dtype)
    _check_step(q, k, v, table, ln, rows=_i32([2, 0, 0, 1, 3]))
    good = kdn.paged_attn_step(q[:4], k, v, table, ln)
    for broken in (-1, k.shape[0], -(2**31), 2**31 - 1):
        t = table.clone()
        t[2, 3] = broken
        o, lse = kdn.paged_attn_step(q[:4], k, v, t, ln)
        assert bool(o[2].isnan().all()) and bool(lse[2].isnan().all())
        keep = [0, 1, 3]
        assert torch.equal(o[keep], good[0][keep]) and torch.equal(lse[keep], good[1][keep])
        # an entry the window does not reach is not read
        o, lse = kdn.paged_attn_step(q[:4], k, v, t, ln, window=40)
        assert torch.isfinite(o).all()
    o, lse = kdn.paged_attn_step(q, k, v, table, ln, rows=_i32([2, 4, -1, 1, 2**31 - 1]))
    assert bool(o[[1, 2, 4]].isnan().all()) and bool(lse[[1, 2, 4]].isnan().all()) and torch.isfinite(o[[0, 3]]).all()
    # lengths beyond the table are held to it
    o, _ = kdn.paged_attn_step(q[:1], k, v, table[2:3].contiguous(), _i32([9999]))
    assert torch.equal(o, kdn.paged_attn_step(q[:1], k, v, table[2:3].contiguous(), _i32([304]))[0])


@pytest.mark.parametrize("dtype,d", CASES)
@pytest.mark.parametrize("page", [1, 4, 16])
def test_broken_entries_of_hidden_tokens_do_not_matter(dtype, d, page):
    """Entries right before the window's first token and right behind the sinks, inside the same tiles."""
    k, v, table, ln, g = _cache([300], 1, d, d, page, dtype, seed=8)
    q = torch.randn(1, 4, d, generator=g, device=DEV).to(dtype)
    good = kdn.paged_attn_step(q, k, v, table, ln, window=41, n_sink=3)
    table[0, -(-3 // page):259 // page] = -7
    o, lse = kdn.paged_attn_step(q, k, v, table, ln, window=41, n_sink=3)
    assert torch.equal(o, good[0]) and torch.equal(lse, good[1])
    table[0, 259 // page] = -7
    assert bool(kdn.paged_attn_step(q, k, v, table, ln, window=41, n_sink=3)[0].isnan().all())


def test_step_in_a_graph_follows_the_lengths():
    k, v, table, ln, g = _cache([900, 40], 2, 128, 128, 16, torch.bfloat16, seed=7)
    q = torch.randn(2, 8, 128, generator=g, device=DEV).to(torch.bfloat16)
    kdn.paged_attn_step(q, k, v, table, ln)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, lse = kdn.paged_attn_step(q, k, v, table, ln)
    for lens in ([900, 40], [1, 0], [555, 3]):
        ln.copy_(_i32(lens))
        graph.replay()
        a, b = _check_step(q, k, v, table, ln)
        assert torch.equal(o, a) and torch.equal(lse, b)


def test_step_refusals():
    k, v, table, ln, g = _cache([50, 3], 2, 64, 64, 16, torch.bfloat16)
    q = torch.randn(2, 4, 64, device=DEV).to(torch.bfloat16)
    with pytest.raises(kdn.KdnError, match="kv_heads"):
        kdn.paged_attn_step(q[:, :3].contiguous(), k, v, table, ln)
    with pytest.raises(kdn.KdnError, match="window"):
        kdn.paged_attn_step(q, k, v, table, ln, window=-1)
    with pytest.raises(kdn.KdnError, match="rows"):
        kdn.paged_attn_step(q.repeat(2, 1, 1), k, v, table, ln)
    with pytest.raises(ValueError, match="contiguous"):
        kdn.paged_attn_step(q, k.transpose(1, 2).contiguous().transpose(1, 2), v, table, ln)
    with pytest.raises(ValueError, match="lens"):
        kdn.paged_attn_step(q, k, v, table, ln[:1])
    o, lse = kdn.paged_attn_step(q[:0], k, v, table, ln)
    assert o.shape == (0, 4, 64)


# ------------------------------------------------------------------------------------------ books and pages

def _same(pages, books):
    assert pages.table.tolist() == books.table and pages.lens.tolist() == books.lens and pages.refs.tolist() == books.refs


@pytest.mark.parametrize("seed", range(4))
@pytest.mark.parametrize("num,page,rows,most", [(40, 4, 7, 9), (9000, 1, 50, 400), (3, 16, 3, 2)])
def test_random_runs_of_the_books(num, page, rows, most, seed):
    """Every call in any order, refused ones among them, against the entry-by-entry oracle."""
    rng = random.Random(seed)
    pages, books = kdn.make_pages(num, page, rows, most), oa.Books(num, page, rows, most)
    seen = set()
    for _ in range(60):
        op = rng.choice(["reserve", "reserve", "fork", "free", "compact", "bad"])
        moves = None
        if op == "reserve":
            r = rng.sample(range(rows), rng.randint(0, rows))
            c = [rng.randint(0, max(1, most * page // 2)) for _ in r]
            if rng.random() < 0.4:
                c = [rng.randint(0, 3)] * len(r)
                kdn.pages_reserve(pages, _i32(r), c[0] if c else 0)
            else:
                kdn.pages_reserve(pages, _i32(r), _i32(c))
            want = books.reserve(r, c)
        elif op == "fork":
            empty = [r for r in range(rows) if books.lens[r] == 0]
            dst = rng.sample(empty, rng.randint(0, len(empty)))
            rest = [r for r in range(rows) if r not in dst]
            src = [rng.choice(rest) for _ in dst] if rest else []
            moves = kdn.pages_fork(pages, _i32(src), _i32(dst[:len(src)]))
            want, expect = books.fork(src, dst[:len(src)])
        elif op == "free":
            r = [rng.randrange(rows) for _ in range(rng.randint(0, rows))]
            kdn.pages_free(pages, _i32(r))
            want = books.free(r)
        elif op == "compact":
            moves = kdn.pages_compact(pages)
            expect, want = books.compact(), "ok"
        else:
            bad = rng.choice([[rows], [-1], [0, rng.randrange(rows), 0], [2**31 - 1]])
            which = rng.choice(["reserve", "fork", "free"])
            if which == "reserve":
                kdn.pages_reserve(pages, _i32(bad), 1)
                want = books.reserve(bad, [1] * len(bad))
            elif which == "fork":
                moves = kdn.pages_fork(pages, _i32([rng.randrange(rows) for _ in bad]), _i32(bad))
                want, expect = "invalid", [(-1, -1)] * len(bad)
            else:
                kdn.pages_free(pages, _i32(bad))
                want = books.free(bad)
        assert kdn.read_device_status(pages.workspace) == STATUS[want], op
        if moves is not None:
            assert [tuple(x) for x in moves.tolist()] == [tuple(x) for x in expect]
        _same(pages, books)
        seen.add((op, want))
    assert len(seen) >= 5


def test_negative_count_is_refused_whole():
    pages = kdn.make_pages(8, 4, 3, 2)
    kdn.pages_reserve(pages, _i32([0, 1]), _i32([4, -1]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_INVALID_ARG
    assert pages.lens.tolist() == [0, 0, 0] and pages.refs.sum() == 0


def test_more_pages_than_32_bits_can_count_are_refused():
    """4096 rows asking for 2^30 tokens each: the sum of the needs passes 2^32 pages."""
    pages = kdn.Pages(torch.zeros(1, 1, dtype=torch.int32, device=DEV).expand(1, 1).contiguous(), _i32([0]), _i32([0] * 8), 1)
    pages.table = torch.full((4096, 1 << 10), -1, dtype=torch.int32, device=DEV)
    pages.lens = torch.zeros(4096, dtype=torch.int32, device=DEV)
    kdn.pages_reserve(pages, torch.arange(4096, dtype=torch.int32, device=DEV), 1 << 10)
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_CAPACITY
    assert int(pages.lens.sum()) == 0 and int(pages.refs.sum()) == 0


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv,Hkv,page", [(16, 16, 1, 1), (128, 64, 3, 16), (64, 128, 2, 64)])
def test_copy_moves_whole_pages_and_skips_the_rest(dtype, dk, dv, Hkv, page):
    g = torch.Generator(device=DEV).manual_seed(0)
    k = torch.randn(50, Hkv, page, dk, generator=g, device=DEV).to(dtype)
    v = torch.randn(50, Hkv, page, dv, generator=g, device=DEV).to(dtype)
    moves = [(3, 40), (-1, -1), (3, 41), (49, 0), (50, 5), (7, -1), (6, 50), (9, 9), (2**31 - 1, 8)]
    ek, ev = k.clone(), v.clone()
    for a, b in moves:
        if 0 <= a < 50 and 0 <= b < 50:
            ek[b], ev[b] = k[a], v[a]
    kdn.pages_copy(_i32(moves), k, v)
    assert torch.equal(k, ek) and torch.equal(v, ev)
    kdn.pages_copy(_i32(moves)[:0], k, v)
    assert torch.equal(k, ek)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("dk,dv,Hkv,page,T", [(16, 32, 1, 1, 3), (128, 128, 2, 16, 1), (64, 64, 3, 32, 70)])
def test_write_puts_the_newest_tokens(dtype, dk, dv, Hkv, page, T):
    pages = kdn.make_pages(200, page, 6, 200 // 6)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.zeros(200, Hkv, page, d, device=DEV, dtype=dtype) for d in (dk, dv))
    ek, ev = k.clone(), v.clone()
    for rows, counts in (([0, 3, 5], None), ([5, 1, 0], [min(2, T), T, 0])):
        n = len(rows)
        kn, vn = (torch.randn(n, Hkv, T, d, generator=g, device=DEV).to(dtype) for d in (dk, dv))
        c = counts or [T] * n
        kdn.pages_reserve(pages, _i32(rows), _i32(counts) if counts else T)
        kdn.pages_write(pages, _i32(rows), kn, vn, k, v, counts=_i32(counts) if counts else None)
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
        table, lens = pages.table.tolist(), pages.lens.tolist()
        for i, r in enumerate(rows):
            for t in range(c[i]):
                pos = lens[r] - c[i] + t
                ek[table[r][pos // page], :, pos % page] = kn[i, :, t]
                ev[table[r][pos // page], :, pos % page] = vn[i, :, t]
        assert torch.equal(k, ek) and torch.equal(v, ev)
    # rows, counts and pages out of range are skipped
    kn, vn = (torch.randn(3, Hkv, T, d, generator=g, device=DEV).to(dtype) for d in (dk, dv))
    kdn.pages_write(pages, _i32([6, -1, 2]), kn, vn, k, v)  # row 2 is empty: no page
    kdn.pages_write(pages, _i32([0, 1, 3]), kn, vn, k, v, counts=_i32([-1, T + 1, 0]))
    assert torch.equal(k, ek) and torch.equal(v, ev)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 128)])
def test_serving_run_next_to_the_recurrent_state(dtype, d):
    """A layer that mixes the recurrent state with windowed attention: prefill with the scan and window_attn, tokens
    appended to pages, decode with decode_step and paged_attn_step, a fork into two beams, a freed row and a
    compaction between steps.  Every step equals the last row of the whole sequence run at once."""
    B, H, Hkv, L0, steps, page, window, sink = 2, 4, 2, 75, 6, 16, 33, 3
    wl = WORKLOADS["gdn_d128"].with_(dk=d, dv=d, dtype="f32" if dtype == torch.float32 else "bf16")
    L = L0 + steps
    x = make_scan_inputs(wl, seed=3, device=DEV, B=B, H=H, L=L)
    g = torch.Generator(device=DEV).manual_seed(4)
    qa = torch.randn(B, H, L, d, generator=g, device=DEV).to(dtype)
    ka, va = (torch.randn(B, Hkv, L, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    o_all, lse_all = kdn.window_attn(qa, ka, va, window, n_sink=sink)
    s_all = kdn.scan_delta(x["q"], x["k"], x["v"], x["beta"], a=x["a"])[0]
    cut = lambda t, a, b: t[:, :, a:b].contiguous()  # noqa: E731
    # prefill
    o0, _ = kdn.window_attn(cut(qa, 0, L0), cut(ka, 0, L0), cut(va, 0, L0), window, n_sink=sink)
    assert torch.equal(o0, o_all[:, :, :L0])
    _, _, S = kdn.scan_delta(cut(x["q"], 0, L0), cut(x["k"], 0, L0), cut(x["v"], 0, L0), cut(x["beta"], 0, L0),
                             a=cut(x["a"], 0, L0))
    pages = kdn.make_pages(64, page, 8, 8)
    kp, vp = (torch.full((64, Hkv, page, d), float("nan"), device=DEV, dtype=dtype) for _ in range(2))
    kdn.pages_reserve(pages, _i32([7]), 40)  # another user's row, freed later: leaves holes
    rows = _i32([1, 4])
    kdn.pages_reserve(pages, rows, L0)
    kdn.pages_write(pages, rows, cut(ka, 0, L0), cut(va, 0, L0), kp, vp)
    # each sequence continues as two beams with the same tokens
    both = torch.cat([rows, _i32([5, 6])])
    kdn.pages_copy(kdn.pages_fork(pages, rows, _i32([5, 6])), kp, vp)
    S2 = torch.cat([S, S])
    twice = lambda t: torch.cat([t, t]).contiguous()  # noqa: E731
    for t in range(L0, L):
        if t == L0 + 2:
            kdn.pages_free(pages, _i32([7]))
            kdn.pages_copy(kdn.pages_compact(pages), kp, vp)
            used = int((pages.refs > 0).sum())
            assert bool((pages.refs[:used] > 0).all())
        if t == L0 + 4:  # the beams of sequence 1 are dropped
            kdn.pages_free(pages, _i32([6]))
            both, S2 = both[:3].contiguous(), S2[:3].contiguous()
        m = both.numel()
        kdn.pages_reserve(pages, both, 1)
        kdn.pages_write(pages, both, twice(cut(ka, t, t + 1))[:m], twice(cut(va, t, t + 1))[:m], kp, vp)
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
        o, lse = kdn.paged_attn_step(twice(qa[:, :, t])[:m], kp, vp, pages.table, pages.lens, rows=both, window=window,
                                     n_sink=sink)
        # two runs of the same read: each within its weights' rounding (2^-8 at most, bf16) of the exact one
        tol = 1e-4 if dtype == torch.float32 else 4 * 2.0 ** -8
        ref = twice(o_all[:, :, t])[:m]
        assert float((o.float() - ref.float()).abs().max()) <= tol * float(va.float().abs().max())
        assert float((lse - twice(lse_all[:, :, t])[:m]).abs().max()) <= 1e-4
        one = lambda n: twice(x[n][:, :, t])[:m]  # noqa: E731
        so, _ = kdn.decode_step("delta", one("q"), one("k"), one("v"), S2, beta=one("beta"), a=one("a"))
        ref = twice(s_all[:, :, t])[:m]
        assert float((so - ref).abs().max() / ref.abs().max()) <= 3e-3
    assert int(pages.refs.sum()) == sum(-(-n // page) for n in pages.lens.tolist())
    kdn.pages_free(pages, torch.arange(8, dtype=torch.int32, device=DEV))
    assert int(pages.refs.abs().sum()) == 0 and bool((pages.table == -1).all())


def test_calls_at_once_on_several_streams():
    """Prefill, backward, decode and page calls of different layers in flight together, each with workspaces of its
    own, give what they give alone."""
    jobs, alone = [], []
    for i in range(3):
        g = torch.Generator(device=DEV).manual_seed(30 + i)
        d = (64, 128, 32)[i]
        dt = torch.bfloat16 if i < 2 else torch.float32
        q, k, v, dO = (torch.randn(1, h, 700, d, generator=g, device=DEV).to(dt) for h in (4, 2, 2, 4))
        kp, vp, table, ln, _ = _cache([900, 3000, 5], 2, d, d, 16, dt, seed=i)
        qs = torch.randn(3, 4, d, generator=g, device=DEV).to(dt)
        free = sorted(set(range(kp.shape[0])) - set(table.flatten().tolist()))  # pages that no row reads
        moves = _i32([[int(table[0, 0]), free[0]], [int(table[1, 0]), free[1]]])
        jobs.append((q, k, v, dO, kp, vp, table, ln, qs, moves))

    def run(job, stream):
        q, k, v, dO, kp, vp, table, ln, qs, moves = job
        o, lse = kdn.window_attn(q, k, v, 100, n_sink=3, stream=stream)
        grads = kdn.window_attn_backward(q, k, v, o, lse, dO, 100, n_sink=3, stream=stream)
        step = kdn.paged_attn_step(qs, kp, vp, table, ln, stream=stream)
        kdn.pages_copy(moves, kp, vp, stream=stream)
        return [o, lse, *grads.values(), *step]

    for job in jobs:
        alone.append([x.clone() for x in run(job, None)])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in jobs]
    for _ in range(5):
        together = [run(job, s) for job, s in zip(jobs, streams)]
        torch.cuda.synchronize()
        for a, b in zip(alone, together):
            assert all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,num", [(torch.bfloat16, 17000), (torch.float32, 17000)])
def test_a_pool_whose_offsets_pass_32_bits(dtype, num):
    """Pages at the end of a pool of more than 2^31 elements: written, copied and read as in a small one."""
    Hkv, page, d, held = 8, 128, 128, 9
    kp, vp = (torch.empty(num, Hkv, page, d, device=DEV, dtype=dtype) for _ in range(2))
    assert kp.numel() > 1 << 31
    used = [num - 1 - 3 * i for i in range(held)]
    n = held * page - 5
    books = kdn.Pages(_i32([used]), _i32([n]), _i32([0] * num), page)
    g = torch.Generator(device=DEV).manual_seed(1)
    k, v = (torch.randn(1, Hkv, n, d, generator=g, device=DEV).to(dtype) for _ in range(2))
    q = torch.randn(1, 16, d, generator=g, device=DEV).to(dtype)
    kdn.pages_write(books, _i32([0]), k, v, kp, vp)
    kdn.pages_copy(_i32([[used[0], num - 2], [used[1], 0]]), kp, vp)
    for x, new in ((kp, k), (vp, v)):
        seq = x[used].transpose(0, 1).reshape(Hkv, held * page, d)
        assert torch.equal(seq[:, :n], new[0])
        assert torch.equal(x[num - 2], x[used[0]]) and torch.equal(x[0], x[used[1]])
    table = _i32([[num - 2, 0] + used[2:]])
    o, lse = kdn.paged_attn_step(q, kp, vp, table, books.lens)
    o1, lse1 = kdn.paged_attn_step(q, kp[used].contiguous(), vp[used].contiguous(), _i32([list(range(held))]), books.lens)
    assert torch.equal(o, o1) and torch.equal(lse, lse1)


# ------------------------------------------------------------------------------------------ refused calls

def _full_pool(page=4, Hkv=2, d=64, dtype=torch.bfloat16):
    """Rows 0 and 1 share two full pages, row 2 holds the rest of the pool: no page is left."""
    g = torch.Generator(device=DEV).manual_seed(40)
    pages = kdn.make_pages(6, page, 4, 6)
    k, v = (torch.zeros(6, Hkv, page, d, device=DEV, dtype=dtype) for _ in range(2))
    new = lambda n, t: [torch.randn(n, Hkv, t, d, generator=g, device=DEV).to(dtype) for _ in range(2)]  # noqa: E731
    kdn.pages_reserve(pages, _i32([0]), 2 * page)
    kdn.pages_write(pages, _i32([0]), *new(1, 2 * page), k, v)
    kdn.pages_copy(kdn.pages_fork(pages, _i32([0]), _i32([1])), k, v)
    kdn.pages_reserve(pages, _i32([2]), 4 * page)
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK and bool((pages.refs > 0).all())
    return pages, k, v, new


def _rows_hold(pages, k, v, row, kn, vn):
    """The newest tokens of a row are kn, vn [Hkv, T, d]."""
    page, T = pages.page_size, kn.shape[1]
    j = torch.arange(T, device=DEV) + int(pages.lens[row]) - T
    at = pages.table[row].long()[j // page], j % page
    return torch.equal(k[at[0], :, at[1]].transpose(0, 1), kn) and torch.equal(v[at[0], :, at[1]].transpose(0, 1), vn)


@pytest.mark.parametrize("counts", [1, [1, 1]])
def test_a_write_behind_a_refused_reservation_changes_nothing(counts):
    """No page is left: the write that follows (every layer's) must not land on the rows' older tokens, which other
    rows may share."""
    pages, k, v, new = _full_pool()
    k0, v0 = k.clone(), v.clone()
    both = _i32([0, 1])
    kn, vn = new(2, 1)
    kdn.pages_reserve(pages, both, counts if isinstance(counts, int) else _i32(counts))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_CAPACITY
    for _ in range(2):
        kdn.pages_write(pages, both, kn, vn, k, v, counts=None if isinstance(counts, int) else _i32(counts))
        assert torch.equal(k, k0) and torch.equal(v, v0)
    # row 2 was not in the refused call: its own tokens may still be written
    kn2, vn2 = new(1, 16)
    kdn.pages_write(pages, _i32([2]), kn2, vn2, k, v)
    assert _rows_hold(pages, k, v, 2, kn2[0], vn2[0])
    # other books' calls between the refusal and the write do not lift it
    kdn.pages_compact(pages)
    kdn.pages_free(pages, _i32([3]))
    k0, v0 = k.clone(), v.clone()
    kdn.pages_write(pages, both, kn, vn, k, v)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    # a page is there again: the reservation and its write go through
    kdn.pages_free(pages, _i32([2]))
    kdn.pages_reserve(pages, both, 1)
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
    kdn.pages_write(pages, both, kn, vn, k, v)
    assert _rows_hold(pages, k, v, 0, kn[0], vn[0]) and _rows_hold(pages, k, v, 1, kn[1], vn[1])


@pytest.mark.parametrize("rows,counts", [([0, 1, 0], [1, 1, 1]), ([0, 1, 9], [1, 1, 1]), ([1, 0, -1], [1, 1, 1]),
                                         ([0, 1, 3], [1, 1, 25]), ([0, 1, 3], [1, -1, 1])])
def test_every_kind_of_refusal_holds_the_write_back(rows, counts):
    """Rows listed twice or out of range, a row too long for the table, a negative count."""
    pages, k, v, new = _full_pool()
    kdn.pages_free(pages, _i32([2]))
    k0, v0 = k.clone(), v.clone()
    kdn.pages_reserve(pages, _i32(rows), _i32(counts))
    assert kdn.read_device_status(pages.workspace) != kdn.KDN_OK
    kdn.pages_write(pages, _i32(rows), *new(3, 1), k, v)
    assert torch.equal(k, k0) and torch.equal(v, v0)
    kn, vn = new(1, 3)  # adding no token is a reservation too: the newest tokens may be written again
    kdn.pages_reserve(pages, _i32([1]), 0)
    kdn.pages_write(pages, _i32([1]), kn, vn, k, v)
    assert _rows_hold(pages, k, v, 1, kn[0], vn[0])


def test_a_row_that_is_emptied_or_forked_anew_forgets_its_refusal():
    pages, k, v, new = _full_pool()
    kdn.pages_reserve(pages, _i32([0, 1]), 1)  # refused
    kdn.pages_free(pages, _i32([1]))
    kdn.pages_copy(kdn.pages_fork(pages, _i32([0]), _i32([1])), k, v)
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
    kn, vn = new(2, 1)
    before = k.clone()
    kdn.pages_write(pages, _i32([0]), kn[:1], vn[:1], k, v)  # row 0 itself: still held back
    assert torch.equal(k, before)
    kdn.pages_write(pages, _i32([1]), kn[1:], vn[1:], k, v)  # asks for the newest token of the copy
    assert _rows_hold(pages, k, v, 1, kn[1], vn[1])


def test_a_captured_reservation_and_write_follow_the_pool():
    """One graph of a reservation and its write, replayed while no page is left and again when there is one."""
    pages, k, v, new = _full_pool()
    both = _i32([0, 1])
    kn, vn = new(2, 1)
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        kdn.pages_reserve(pages, both, 1)
        kdn.pages_write(pages, both, kn, vn, k, v)
    k0 = k.clone()
    graph.replay()
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_CAPACITY and torch.equal(k, k0)
    kdn.pages_free(pages, _i32([2]))
    for n in (9, 10, 11):
        for x in (kn, vn):
            x.add_(1)
        graph.replay()
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK and pages.lens.tolist()[:2] == [n, n]
        assert _rows_hold(pages, k, v, 0, kn[0], vn[0]) and _rows_hold(pages, k, v, 1, kn[1], vn[1])


def test_books_that_no_call_has_touched_report_no_error():
    """The status word of new books, whatever the memory they got held before."""
    for _ in range(20):
        torch.full((1 << 14,), -1, dtype=torch.int32, device=DEV)  # freed at once: the next small arrays may lie here
        pages = kdn.make_pages(64, 16, 8, 4)
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
        torch.full((1 << 8,), -1, dtype=torch.int32, device=DEV)
        assert kdn.read_device_status(kdn.Pages(pages.table, pages.lens, pages.refs, 16).workspace) == kdn.KDN_OK
        del pages


def _books(pages):
    return [pages.table.clone(), pages.lens.clone(), pages.refs.clone()]


@pytest.mark.parametrize("entry", [-1, 40, 2**31 - 1, -(2**31), "free"])
@pytest.mark.parametrize("at", [0, 2, 3])
def test_calls_that_meet_a_broken_entry_change_nothing(entry, at):
    """Row 2 (3 full pages and a part of one) has an entry that names no page, or one that is free: fork and free refuse
    the whole call, other rows' parts of it too."""
    pages = kdn.make_pages(40, 4, 8, 6)
    kdn.pages_reserve(pages, _i32([0, 2, 4]), _i32([9, 14, 8]))
    pages.table[2, at] = entry if entry != "free" else 39
    before = _books(pages)
    moves = kdn.pages_fork(pages, _i32([0, 2, 4]), _i32([1, 3, 5]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_INVALID_ARG
    assert bool((moves == -1).all()) and all(torch.equal(a, b) for a, b in zip(before, _books(pages)))
    kdn.pages_free(pages, _i32([0, 2, 2, 4]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, _books(pages)))
    # without that row both go through
    kdn.pages_fork(pages, _i32([0, 4]), _i32([1, 5]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
    kdn.pages_free(pages, _i32([0, 4, 0, 1, 5]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
    assert pages.lens.tolist() == [0, 0, 14, 0, 0, 0, 0, 0]
    held = [p for p in pages.table[2].tolist() if 0 <= p < 40 and p != 39]
    assert int(pages.refs.sum()) == 4 and all(int(pages.refs[p]) == 1 for p in held)


def test_free_refuses_counts_and_lengths_that_do_not_agree():
    """Two rows that name a page counted once, and a row longer than the table: nothing changes."""
    pages = kdn.make_pages(40, 4, 8, 6)
    kdn.pages_reserve(pages, _i32([0, 1, 2]), _i32([9, 14, 8]))
    pages.table[1, 1] = pages.table[0, 2]
    before = _books(pages)
    kdn.pages_free(pages, _i32([2, 0, 1]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_INVALID_ARG
    assert all(torch.equal(a, b) for a, b in zip(before, _books(pages)))
    kdn.pages_free(pages, _i32([0, 2]))
    assert kdn.read_device_status(pages.workspace) == kdn.KDN_OK
    pages.lens[4] = 25
    before = _books(pages)
    for call in (lambda: kdn.pages_free(pages, _i32([4])), lambda: kdn.pages_fork(pages, _i32([4]), _i32([5])),
                 lambda: kdn.pages_reserve(pages, _i32([4]), 0)):
        call()
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_INVALID_ARG
        assert all(torch.equal(a, b) for a, b in zip(before, _books(pages)))


def test_a_first_call_on_another_stream_follows_the_making_of_the_books():
    """The workspace is set to zero on the stream that is current when the books are made; a call on another stream, and
    what it leaves in the workspace, must not be overtaken by that."""
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    table, lens, refs, rows = _i32([[-1] * 4] * 3), _i32([0] * 3), _i32([0] * 2), _i32([0, 1, 2])
    kdn.pages_reserve(kdn.Pages(table, lens, refs, 4), rows, 0)  # a kernel's first launch may wait for the device
    torch.cuda.synchronize()
    for given in (False, True):
        ws = torch.full((1 << 12,), -1, dtype=torch.int8, device=DEV).view(torch.uint8) if given else None
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(20_000_000)  # about 10 ms: the zeros come behind it
            pages = kdn.Pages(table, lens, refs, 4, ws)
        kdn.pages_reserve(pages, rows, 4, stream=other)  # three pages of two
        torch.cuda.synchronize()
        assert kdn.read_device_status(pages.workspace) == kdn.KDN_ERR_CAPACITY
        k, v = (torch.zeros(2, 1, 4, 64, device=DEV) for _ in range(2))
        kdn.pages_reserve(pages, rows[:2], 4, stream=other)
        kdn.pages_reserve(pages, rows, 4, stream=other)  # refused
        new = torch.ones(2, 1, 4, 64, device=DEV)
        torch.cuda.synchronize()
        kdn.pages_write(pages, rows[:2], new, new, k, v, stream=other)
        torch.cuda.synchronize()
        assert not k.any() and not v.any()
        kdn.pages_free(pages, rows, stream=other)
        torch.cuda.synchronize()


def test_books_that_are_dropped_keep_their_memory_until_their_calls_have_ended():
    """The workspace of books that die right after a call on another stream is not handed out again while the call waits."""
    side = torch.cuda.Stream()
    tables = [[_i32([[-1] * 4] * 3), _i32([0] * 3), _i32([0] * 2)] for _ in range(8)]
    rows = _i32([0, 1, 2])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)  # about 20 ms
    for t in tables:
        kdn.pages_reserve(kdn.Pages(*t, 4), rows, 4, stream=side)  # refused: writes its status and marks
    size = kdn.Pages(*tables[0], 4).workspace.numel()
    mine = [torch.full((size,), 7, dtype=torch.uint8, device=DEV) for _ in range(16)]
    torch.cuda.synchronize()
    assert all(bool((x == 7).all()) for x in mine)


@pytest.mark.parametrize("seed", range(6))
@pytest.mark.parametrize("num,page,rows,most", [(12, 4, 6, 5), (9, 1, 5, 6), (30, 16, 8, 4)])
def test_random_runs_keep_every_rows_tokens(num, page, rows, most, seed):
    """Reservations, each followed by its write whether it was refused or not, forks and compactions with their copies,
    freed rows: after every step each row reads back the tokens of a plain list."""
    rng = random.Random(100 + seed)
    pages = kdn.make_pages(num, page, rows, most)
    k, v = (torch.zeros(num, 1, page, 16, device=DEV) for _ in range(2))
    model, serial, refused = [[] for _ in range(rows)], 0, 0
    for step in range(80):
        op = rng.choice(["grow", "grow", "grow", "fork", "free", "compact"])
        if op == "grow":
            r = rng.sample(range(rows), rng.randint(1, rows))
            c = [rng.randint(0, 2 * page) for _ in r]
            T = max(1, *c)
            new = torch.arange(serial, serial + len(r) * T, device=DEV, dtype=torch.float32).view(len(r), 1, T, 1)
            new = new.expand(-1, -1, -1, 16).contiguous()
            kdn.pages_reserve(pages, _i32(r), _i32(c))
            kdn.pages_write(pages, _i32(r), new, -new, k, v, counts=_i32(c))
            if kdn.read_device_status(pages.workspace) == kdn.KDN_OK:
                for i, x in enumerate(r):
                    model[x] += [serial + i * T + t for t in range(c[i])]
            else:
                refused += 1
            serial += len(r) * T
        elif op == "fork":
            dst = [x for x in range(rows) if not model[x]][:2]
            src = [rng.choice([x for x in range(rows) if x not in dst]) for _ in dst] if len(dst) < rows else []
            kdn.pages_copy(kdn.pages_fork(pages, _i32(src), _i32(dst[:len(src)])), k, v)
            if kdn.read_device_status(pages.workspace) == kdn.KDN_OK:
                for a, b in zip(src, dst):
                    model[b] = list(model[a])
        elif op == "free":
            r = rng.sample(range(rows), rng.randint(0, 2))
            kdn.pages_free(pages, _i32(r))
            for x in r:
                model[x] = []
        else:
            kdn.pages_copy(kdn.pages_compact(pages), k, v)
        assert pages.lens.tolist() == [len(x) for x in model]
        table, kk, vv = pages.table.tolist(), k[:, 0, :, 0].tolist(), v[:, 0, :, 15].tolist()
        for r, tokens in enumerate(model):
            for j, x in enumerate(tokens):
                assert kk[table[r][j // page]][j % page] == x and vv[table[r][j // page]][j % page] == -x, (step, op, r, j)
    assert refused > 3


def test_a_workspace_that_is_not_on_the_device_is_refused():
    pages = kdn.make_pages(4, 16, 2, 2)
    books = kdn.Pages(pages.table, pages.lens, pages.refs, 16, torch.zeros(1 << 12, dtype=torch.uint8))
    with pytest.raises(kdn.KdnError, match="workspace"):
        kdn.pages_free(books, _i32([0]))
    short = kdn.Pages(pages.table, pages.lens, pages.refs, 16, torch.zeros(256, dtype=torch.uint8, device=DEV))
    with pytest.raises(kdn.KdnError, match="workspace_bytes"):
        kdn.pages_free(short, _i32([0]))
