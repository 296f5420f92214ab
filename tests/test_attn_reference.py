"""The references of the windowed attention against each other, against differences, and the library's host-side
refusals (no GPU)."""

import ctypes
import os
import shutil
import subprocess

import numpy as np
import pytest
import torch

import oracle.attn as oa
from attn_ref import dense
from delta_rule_recurrent_scan_b200 import build, kdn


def _draw(B, H, Hkv, L, dk, dv, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(B, h, L, d, generator=g, dtype=torch.float64) for h, d in ((H, dk), (Hkv, dk), (Hkv, dv), (H, dv))]


@pytest.mark.parametrize("window,n_sink", [(1, 0), (4, 0), (4, 2), (3, 9), (100, 3)])
def test_dense_reference_is_the_row_by_row_oracle(window, n_sink):
    q, k, v, dO = _draw(2, 4, 2, 13, 8, 6)
    lens = torch.tensor([13, 5], dtype=torch.int32)
    d = dense(q, k, v, window, n_sink, lens, dO=dO, out=0.0)
    o, lse = oa.window_attn(q, k, v, window, n_sink, lens)
    g = oa.window_attn_backward(q, k, v, dO, window, n_sink, lens)
    for name, x in (("o", o), ("lse", lse), ("dq", g["dq"]), ("dk", g["dk"]), ("dv", g["dv"])):
        np.testing.assert_allclose(d[name][0].numpy(), x, rtol=1e-10, atol=1e-12)


def test_gradients_against_differences():
    q, k, v, dO = (x.numpy() for x in _draw(1, 2, 1, 7, 4, 3, seed=1))
    g = oa.window_attn_backward(q, k, v, dO, 3, 1)
    loss = lambda: float((oa.window_attn(q, k, v, 3, 1)[0] * dO).sum())  # noqa: E731
    for x, name in ((q, "dq"), (k, "dk"), (v, "dv")):
        for at in np.ndindex(*x.shape):
            keep = x[at]
            x[at] = keep + 1e-5
            hi = loss()
            x[at] = keep - 1e-5
            lo = loss()
            x[at] = keep
            assert abs((hi - lo) / 2e-5 - g[name][at]) < 1e-7


def test_paged_step_oracle_is_the_last_row_of_the_window():
    q, k, v, _ = _draw(1, 4, 2, 21, 8, 8, seed=2)
    o, lse = oa.window_attn(q, k, v, 6, 3)
    kp, vp = (torch.zeros(6, 2, 4, 8, dtype=torch.float64) for _ in range(2))
    table = [[3, 1, 5, 0, 2, 4]]
    for t in range(21):
        kp[table[0][t // 4], :, t % 4], vp[table[0][t // 4], :, t % 4] = k[0, :, t], v[0, :, t]
    o1, lse1 = oa.paged_attn_step(q[:, :, -1], kp, vp, table, [21], window=6, n_sink=3)
    np.testing.assert_allclose(o1, o[:, :, -1], rtol=1e-12)
    np.testing.assert_allclose(lse1, lse[:, :, -1], rtol=1e-12)


# ------------------------------------------------------------------------------------------ refusals

@pytest.fixture(scope="module")
def L():
    build.build()
    return kdn.lib()


def _attn(L, d, kv=1, window=4, n_sink=0, scale=1.0):
    return L.kdn_window_attn(ctypes.byref(d), kv, None, None, None, None, 0, window, n_sink, scale, None, None, None, 0, None)


def test_window_attention_refusals(L):
    d = kdn.Dims(1, 4, 8, 64, 64, 0, 1, 1, 0)
    assert _attn(L, d, kv=3) == kdn.KDN_ERR_INVALID_ARG and b"kv_heads" in L.kdn_last_error()
    assert _attn(L, d, kv=0) == kdn.KDN_ERR_INVALID_ARG
    assert _attn(L, d, window=0) == kdn.KDN_ERR_INVALID_ARG and b"window" in L.kdn_last_error()
    assert _attn(L, d, n_sink=-1) == kdn.KDN_ERR_INVALID_ARG
    for bad in (0.0, -1.0, float("inf"), float("nan")):
        assert _attn(L, d, scale=bad) == kdn.KDN_ERR_INVALID_ARG and b"scale" in L.kdn_last_error()
    assert _attn(L, kdn.Dims(1, 4, 8, 48, 64, 0, 1, 1, 0)) == kdn.KDN_ERR_UNSUPPORTED
    assert _attn(L, kdn.Dims(1 << 14, 1 << 10, 1 << 14, 64, 64, 0, 1, 1, 0)) == kdn.KDN_ERR_UNSUPPORTED
    assert _attn(L, d) == kdn.KDN_ERR_INVALID_ARG and b"q is NULL" in L.kdn_last_error()
    args = [None] * 3 + [None, 0, 4, 0, 1.0] + [None] * 7 + [0, None]
    assert L.kdn_window_attn_backward(ctypes.byref(d), 1, *args) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_window_workspace_bytes(ctypes.byref(d), 3, 4, 0, 1) == 0
    assert L.kdn_window_workspace_bytes(ctypes.byref(d), 2, 4, 0, 0) >= 256
    assert L.kdn_window_workspace_bytes(ctypes.byref(d), 2, 4, 0, 1) >= 256 + 4 * 8 * 4


def test_paged_cache_refusals(L):
    ok = dict(num_pages=8, page_size=16, rows=4, max_pages=2)
    assert L.kdn_pages_workspace_bytes(ctypes.byref(kdn.PagesC(**ok))) >= 256 + 4 * 16
    for bad, status in ((dict(num_pages=0), 1), (dict(rows=0), 1), (dict(max_pages=0), 1), (dict(page_size=0), 2),
                        (dict(page_size=24), 2), (dict(page_size=2048), 2), (dict(rows=1 << 20), 2),
                        (dict(max_pages=1 << 30), 2)):
        c = kdn.PagesC(**{**ok, **bad})
        assert L.kdn_pages_workspace_bytes(ctypes.byref(c)) == 0
        assert L.kdn_pages_free(ctypes.byref(c), 0, None, None, 0, None) == status
        assert L.kdn_paged_step_workspace_bytes(ctypes.byref(c), 1, 4, 2, 64, 64, 1, 0, 0) == 0
    c = kdn.PagesC(**ok)
    assert L.kdn_pages_free(None, 0, None, None, 0, None) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_pages_free(ctypes.byref(c), -1, None, None, 0, None) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_pages_reserve(ctypes.byref(c), 1, None, None, -1, None, 0, None) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_pages_free(ctypes.byref(c), 0, None, None, 0, None) == kdn.KDN_ERR_INVALID_ARG
    assert b"table" in L.kdn_last_error()
    step = lambda n=1, H=4, kv=2, dk=64, dv=64, it=1, ot=1, window=0, sink=0, scale=1.0: L.kdn_paged_attn_step(  # noqa: E731
        ctypes.byref(c), n, None, H, kv, dk, dv, it, ot, None, None, None, window, sink, scale, None, None, None, 0, None)
    assert step(kv=3) == kdn.KDN_ERR_INVALID_ARG
    assert step(dk=48) == kdn.KDN_ERR_UNSUPPORTED
    assert step(it=7) == kdn.KDN_ERR_INVALID_ARG and step(ot=7) == kdn.KDN_ERR_INVALID_ARG
    assert step(window=-1) == kdn.KDN_ERR_INVALID_ARG and step(sink=-1) == kdn.KDN_ERR_INVALID_ARG
    assert step(scale=0.0) == kdn.KDN_ERR_INVALID_ARG
    assert step(n=5) == kdn.KDN_ERR_INVALID_ARG and b"rows" in L.kdn_last_error()
    assert step(n=-1) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_pages_copy(1, None, 8, 16, 2, 64, 64, 1, None, None, None) == kdn.KDN_ERR_INVALID_ARG
    assert L.kdn_pages_copy(1, None, 8, 24, 2, 64, 64, 1, None, None, None) == kdn.KDN_ERR_UNSUPPORTED
    assert L.kdn_status_string(6).decode() == "KDN_ERR_CAPACITY"


def test_outputs_may_not_overlap(L):
    """Refused from the addresses alone, before anything reads them."""
    d = kdn.Dims(1, 4, 8, 64, 64, 0, 1, 1, 0)  # bf16: q, o 4096 bytes, k, v (2 heads) 2048, lse 128
    at = dict(q=0x10000, k=0x20000, v=0x30000, o=0x40000, lse=0x50000, dO=0x60000, dq=0x70000, dk=0x80000, dv=0x90000,
              ws=0xa0000)

    def forward(**new):
        a = {**at, **new}
        st = L.kdn_window_attn(ctypes.byref(d), 2, a["q"], a["k"], a["v"], None, 0, 4, 0, 1.0, a["o"], a["lse"], a["ws"], 256, None)
        return st, L.kdn_last_error()

    def backward(**new):
        a = {**at, **new}
        st = L.kdn_window_attn_backward(ctypes.byref(d), 2, a["q"], a["k"], a["v"], None, 0, 4, 0, 1.0, a["o"], a["lse"],
                                        a["dO"], a["dq"], a["dk"], a["dv"], a["ws"], 256, None)
        return st, L.kdn_last_error()

    c = kdn.PagesC(num_pages=8, page_size=16, rows=4, max_pages=2)

    def step(**new):
        a = {**at, **new}  # q, o [2, 4, 64], pages [8, 2, 16, 64]: 32,768 bytes
        st = L.kdn_paged_attn_step(ctypes.byref(c), 2, None, 4, 2, 64, 64, 1, 1, a["q"], a["k"], a["v"], 0, 0, 1.0, a["o"],
                                   a["lse"], a["ws"], 256, None)
        return st, L.kdn_last_error()

    for call, new, says in (
            (forward, dict(o=at["q"]), b"o overlaps q"), (forward, dict(o=at["k"] + 2032), b"o overlaps k"),
            (forward, dict(o=at["v"] - 4080), b"o overlaps v"), (forward, dict(lse=at["o"] + 4080), b"o overlaps lse"),
            (forward, dict(lse=at["q"] - 112), b"lse overlaps q"), (forward, dict(ws=at["v"]), b"workspace overlaps v"),
            (backward, dict(dq=at["dO"]), b"dq overlaps dO"), (backward, dict(dk=at["k"]), b"dk overlaps k"),
            (backward, dict(dv=at["dk"] + 2032), b"dk overlaps dv"), (backward, dict(dq=at["lse"]), b"dq overlaps lse"),
            (backward, dict(dv=at["o"] + 4080), b"dv overlaps o"),
            (step, dict(o=at["q"] + 1008), b"o overlaps q"), (step, dict(lse=at["k"] + 32752), b"lse overlaps k_pages"),
            (step, dict(ws=at["v"] + 256), b"workspace overlaps v_pages")):
        st, said = call(**new)
        assert st == kdn.KDN_ERR_INVALID_ARG and said.endswith(says), (says, said)
    for call, new in ((forward, dict(o=at["q"] + 4096)), (backward, dict(dq=at["dO"] + 4096)),
                      (backward, dict(dv=at["dk"] + 2048)), (step, dict(o=at["q"] + 1024))):
        assert b"overlaps" not in call(**new)[1]  # neighbours are not overlaps (what follows refuses the made-up addresses)


def test_more_new_tokens_than_the_write_counts_are_refused(L):
    c = kdn.PagesC(num_pages=8, page_size=16, rows=4, max_pages=2)
    st = L.kdn_pages_write(ctypes.byref(c), 1, None, None, (1 << 24) + 1, 2, 64, 64, 1, None, None, None, None, None)
    assert st == kdn.KDN_ERR_UNSUPPORTED and b"2^24" in L.kdn_last_error()


def test_binding_refuses_cpu_tensors_and_bad_shapes():
    x = torch.zeros(1, 2, 4, 16)
    with pytest.raises(ValueError, match="CUDA"):
        kdn.window_attn(x, x, x, 4)
    with pytest.raises(ValueError, match="q must be"):
        kdn.window_attn(x[0], x, x, 4)
    with pytest.raises(ValueError, match="unsupported"):
        kdn.window_attn(x.half(), x, x, 4)
    pages = kdn.make_pages(4, 16, 2, 2, device="cpu")
    with pytest.raises(ValueError, match="CUDA"):
        kdn.pages_free(pages, torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA"):
        kdn.paged_attn_step(x[0], x, x, pages.table, pages.lens)


def test_books_oracle_keeps_its_counts():
    """refs always equals the number of table entries naming a page, through a run of every call."""
    b = oa.Books(12, 4, 5, 4)

    def count():
        n = [0] * 12
        for r, row in enumerate(b.table):
            held = [p for p in row if p >= 0]
            assert len(held) == -(-b.lens[r] // 4)
            for p in held:
                n[p] += 1
        assert n == b.refs

    assert b.reserve([0, 2], [9, 4]) == "ok"
    count()
    assert b.table[0][:3] == [0, 1, 2] and b.table[2][0] == 3
    assert b.fork([0, 0, 2], [1, 3, 4]) == ("ok", [(2, 4), (2, 5), (-1, -1)])
    count()
    assert b.refs[0] == 3 and b.fork([0], [1])[0] == "invalid"
    assert b.free([0, 0]) == "ok"
    count()
    assert b.reserve([1], [8]) == "capacity" and b.reserve([1, 1], [1, 1]) == "invalid"
    assert b.reserve([2], [40]) == "capacity"
    assert b.compact()[0] == (5, 2)
    count()


def test_binding_refuses_numbers_beyond_32_bits():
    x = torch.zeros(1, 2, 4, 16)
    for bad in (dict(window=2**31), dict(window=4, n_sink=2**32 + 1)):
        with pytest.raises(ValueError, match="32 bits"):
            kdn.window_attn(x, x, x, **bad)


def test_page_calls_refuse_arrays_that_overlap(L):
    """kdn_pages_write, _write_reserved and _copy, the books' calls, and the integer arrays of the attention calls; from
    the addresses alone."""
    c = kdn.PagesC(num_pages=8, page_size=16, rows=4, max_pages=2, table=0x100000, lens=0x110000, refs=0x120000)
    at = dict(k=0x200000, v=0x300000, kn=0x400000, vn=0x500000, rows=0x600000, counts=0x610000, moves=0x620000, ws=0x630000,
              dst=0x640000)
    ws = L.kdn_pages_workspace_bytes(ctypes.byref(c))

    def call(name, *args):
        st = getattr(L, name)(*args)
        return st, L.kdn_last_error()

    def write(**n):  # pages [8, 2, 16, 64] bf16: 32,768 bytes; new tokens [3, 2, 5, 64]: 3,840 bytes
        a = {**at, **n}
        return call("kdn_pages_write", ctypes.byref(c), 3, a["rows"], a["counts"], 5, 2, 64, 64, 1, a["kn"], a["vn"], a["k"],
                    a["v"], None)

    def reserved(**n):
        a = {**at, **n}
        return call("kdn_pages_write_reserved", ctypes.byref(c), 3, a["rows"], a["counts"], 5, 2, 64, 64, 1, a["kn"], a["vn"],
                    a["k"], a["v"], a["ws"], ws, None)

    def copy(**n):
        a = {**at, **n}
        return call("kdn_pages_copy", 3, a["moves"], 8, 16, 2, 64, 64, 1, a["k"], a["v"], None)

    def reserve(**n):
        a = {**at, **n}
        return call("kdn_pages_reserve", ctypes.byref(c), 3, a["rows"], a["counts"], 0, a["ws"], ws, None)

    def fork(**n):
        a = {**at, **n}
        return call("kdn_pages_fork", ctypes.byref(c), 3, a["rows"], a["dst"], a["moves"], a["ws"], ws, None)

    def free(**n):
        a = {**at, **n}
        return call("kdn_pages_free", ctypes.byref(c), 3, a["rows"], a["ws"], ws, None)

    def compact(**n):
        a = {**at, **n}
        return call("kdn_pages_compact", ctypes.byref(c), a["moves"], a["ws"], ws, None)

    d = kdn.Dims(2, 4, 8, 64, 64, 0, 1, 1, 0)

    def forward(lens):
        return call("kdn_window_attn", ctypes.byref(d), 2, 0x10000, 0x20000, 0x30000, lens, 0, 4, 0, 1.0, 0x40000, 0x50000,
                    None, 0, None)

    def backward(lens):
        return call("kdn_window_attn_backward", ctypes.byref(d), 2, 0x10000, 0x20000, 0x30000, lens, 0, 4, 0, 1.0, 0x40000,
                    0x50000, 0x60000, 0x70000, 0x80000, 0x90000, 0xa0000, 256, None)

    def step(o, rows=None):
        return call("kdn_paged_attn_step", ctypes.byref(c), 2, rows, 4, 2, 64, 64, 1, 1, 0x10000, at["k"], at["v"], 0, 0, 1.0,
                    o, None, None, 0, None)

    for (st, said), says in (
            (write(kn=at["k"] + 32752), b"k_pages overlaps k_new"), (write(vn=at["k"] + 16), b"k_pages overlaps v_new"),
            (write(vn=at["v"] - 3824), b"v_pages overlaps v_new"), (write(k=at["v"] + 32752), b"k_pages overlaps v_pages"),
            (write(rows=at["v"] + 64), b"v_pages overlaps rows"), (write(counts=at["k"]), b"k_pages overlaps counts"),
            (write(k=0x110000), b"k_pages overlaps lens"), (write(v=0x100000 - 32752), b"v_pages overlaps table"),
            (reserved(kn=at["k"] + 32752), b"k_pages overlaps k_new"), (reserved(ws=at["v"]), b"v_pages overlaps workspace"),
            (copy(v=at["k"] + 32752), b"k_pages overlaps v_pages"), (copy(moves=at["v"] + 32760), b"v_pages overlaps moves"),
            (reserve(rows=0x110004), b"lens overlaps rows"), (reserve(counts=0x100000), b"table overlaps counts"),
            (reserve(ws=0x120000 - 256), b"refs overlaps workspace"), (reserve(rows=at["ws"] + 256), b"workspace overlaps rows"),
            (fork(moves=0x11fff8), b"refs overlaps moves"), (fork(dst=at["moves"] + 16), b"moves overlaps dst_rows"),
            (fork(rows=0x120000), b"refs overlaps src_rows"), (free(rows=0x100010), b"table overlaps rows"),
            (compact(moves=0x110008), b"lens overlaps moves"),
            (forward(0x40008), b"o overlaps lens"), (backward(0x70ffc - 0xffc), b"dq overlaps lens"),
            (step(0x110000), b"o overlaps lens"), (step(0x100010), b"o overlaps table"), (step(0x10000 + 1024, 0x10000 + 1024), b"o overlaps rows")):
        assert st == kdn.KDN_ERR_INVALID_ARG and said.endswith(says), (says, said)
    for st, said in (write(kn=at["k"] + 32768), write(v=at["k"] + 32768), copy(v=at["k"] + 32768), copy(moves=at["v"] + 32768),
                     reserve(rows=0x110010), fork(dst=at["moves"] + 24), fork(dst=at["rows"]), free(rows=0x100020),
                     reserve(counts=at["rows"])):
        assert b"overlaps" not in said, said  # neighbours, and lists that are only read


def test_first_sweeps_are_short(tmp_path):
    """Which query tiles of the backward walk their keys twice (for delta from the weights): those whose rows see few keys,
    sinks among them, and none whose walk is long.  The kernel's own code, compiled for the host."""
    if shutil.which(build._nvcc()) is None:
        pytest.skip("nvcc not available")
    exe, here = tmp_path / "sweeps", os.path.dirname(os.path.abspath(__file__))
    subprocess.run([build._nvcc(), "-gencode", "arch=compute_100a,code=sm_100a", "-std=c++17", "-O2",
                    "--expt-relaxed-constexpr", "-I", build.CSRC, "-I", build.INCLUDE,
                    os.path.join(here, "native", "window_sweeps_check.cu"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout[-2000:] + r.stderr


def test_needs_that_pass_32_bits_are_larger_than_any_pool(tmp_path):
    """The sums behind kdn_pages_reserve, compiled for the host: no call on a GPU could show a sum that is too short
    without handing out pages that are not there."""
    if shutil.which("g++") is None:
        pytest.skip("g++ not available")
    exe, here = tmp_path / "need", os.path.dirname(os.path.abspath(__file__))
    subprocess.run(["g++", "-std=c++17", "-O1", "-Wall", "-Werror", "-I", build.CSRC,
                    os.path.join(here, "native", "pages_need_check.cpp"), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stdout + r.stderr
    kernel = open(os.path.join(build.CSRC, "pages.cu")).read()
    assert "PageSum need;" in kernel and "PageSum need = 0;" in kernel and "pool_too_small(s.need" in kernel


def test_a_reserved_write_wants_the_books_workspace(L):
    c = kdn.PagesC(num_pages=8, page_size=16, rows=4, max_pages=2)
    args = [ctypes.byref(c), 1, None, None, 1, 2, 64, 64, 1, None, None, None, None]
    assert L.kdn_pages_write_reserved(*args, None, 0, None) == kdn.KDN_ERR_INVALID_ARG
    assert b"workspace" in L.kdn_last_error()
    # a word per row beside the scratch of the searches
    one = L.kdn_pages_workspace_bytes(ctypes.byref(c))
    c.rows = 1 << 18
    assert L.kdn_pages_workspace_bytes(ctypes.byref(c)) >= one - 256 + 4 * (1 << 18)
