"""Windowed attention and its backward pass on the GPU against the dense float64 reference, every error held to the
bound that attn_ref derives from the arithmetic."""

import pytest
import torch

from attn_ref import HALF, dense, worst
from delta_rule_recurrent_scan_b200 import kdn

pytestmark = pytest.mark.gpu
DEV = "cuda"


def _tc(dtype, dk, dv):
    return dtype == torch.bfloat16 and dk == dv and dk in (64, 128)


def _weight(dtype, dk, dv):
    """Half step of the softmax weights' type in their product."""
    return 2.0 ** -8 if _tc(dtype, dk, dv) else 0.0


def _inputs(B, H, Hkv, L, dk, dv, dtype, seed=0, scale=1.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    return [(torch.randn(B, h, L, d, generator=g, device=DEV) * s).to(dtype)
            for h, d, s in ((H, dk, scale), (Hkv, dk, 1.0), (Hkv, dv, 1.0), (H, dv, 1.0))]


def _check(q, k, v, dO, window, n_sink, lens=None, scale=None, out_dtype=None):
    dk, dv = q.shape[-1], v.shape[-1]
    w = _weight(q.dtype, dk, dv)
    od = out_dtype or q.dtype
    dO = dO.to(od)
    o, lse = kdn.window_attn(q, k, v, window, n_sink=n_sink, lens=lens, scale=scale, out_dtype=od)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, window, n_sink=n_sink, lens=lens, scale=scale)
    torch.cuda.synchronize()
    ref = dense(q, k, v, window, n_sink, lens, scale, w=w, out=HALF[od])
    assert o.dtype == od and lse.dtype == torch.float32
    for name, x in (("o", o), ("lse", lse)):
        assert worst(x, ref[name]) <= 1, name
    # on the tensor cores dO enters its products as bf16: an fp32 dO is rounded first, which the bound has to hold
    ref = dense(q, k, v, window, n_sink, lens, scale, dO=dO, w=w + (2.0 ** -8 if w and od == torch.float32 else 0.0),
                out=HALF[q.dtype], o_half=HALF[od])
    for name in ("dq", "dk", "dv"):
        assert g[name].dtype == q.dtype
        if w and od == torch.float32:  # dP and delta see the rounding too
            extra = 2.0 ** -8 * _abs_terms(q, k, v, dO, window, n_sink, lens, scale)[name]
            ref[name] = ref[name][0], ref[name][1] + extra
        assert worst(g[name], ref[name]) <= 1, name
    return o, lse, g


def _abs_terms(q, k, v, dO, window, n_sink, lens, scale):
    """What a relative change of every dO element by one unit can move: the gradients with dP and delta's terms taken
    absolutely."""
    from attn_ref import mask

    B, H, L, dk = q.shape
    Hkv = k.shape[1]
    G = H // Hkv
    scale = dk ** -0.5 if scale is None else scale
    live = torch.ones(B, L, dtype=torch.bool, device=q.device)
    if lens is not None:
        live = torch.arange(L, device=q.device)[None] < lens[:, None].clamp(0, L)
    zap = lambda x: torch.where(live[:, None, :, None], x.double(), 0.0)  # noqa: E731
    qd, kd, vd = zap(q).view(B, Hkv, G, L, dk), zap(k)[:, :, None], zap(v)[:, :, None]
    g = zap(dO).view(B, Hkv, G, L, -1).abs()
    s = (scale * qd @ kd.transpose(-1, -2)).masked_fill(~mask(L, window, n_sink, q.device) | ~live[:, None, None, None], -torch.inf)
    p = torch.softmax(s, -1).nan_to_num()
    a = p * (g @ vd.abs().transpose(-1, -2) + (p @ (g @ vd.abs().transpose(-1, -2)).transpose(-1, -2)).diagonal(dim1=-2, dim2=-1)[..., None])
    return {"dq": (scale * a @ kd.abs()).flatten(1, 2), "dk": (scale * a.transpose(-1, -2) @ qd.abs()).sum(2),
            "dv": (p.transpose(-1, -2) @ g).sum(2)}


@pytest.mark.parametrize("L", [1, 2, 63, 64, 65, 127, 128, 129, 257, 515])
@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_lengths(L, dtype, d):
    _check(*_inputs(1, 2, 1, L, d, d, dtype, seed=L), 100, 5)


@pytest.mark.parametrize("window,n_sink", [(1, 0), (1, 3), (2, 128), (63, 1), (64, 64), (65, 65), (128, 129), (200, 300),
                                           (700, 0), (2**31 - 1, 2**31 - 1)])
@pytest.mark.parametrize("dtype,d", [(torch.float32, 64), (torch.bfloat16, 64), (torch.bfloat16, 128)])
def test_windows_and_sinks(window, n_sink, dtype, d):
    _check(*_inputs(1, 2, 2, 650, d, d, dtype, seed=3), window, n_sink)


@pytest.mark.parametrize("dk", [16, 32, 64, 128])
@pytest.mark.parametrize("dv", [16, 32, 64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_head_sizes(dk, dv, dtype):
    _check(*_inputs(1, 2, 1, 150, dk, dv, dtype, seed=4), 70, 3)


@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (6, 2), (8, 8)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_shared_heads(H, Hkv, dtype):
    _check(*_inputs(2, H, Hkv, 300, 64, 64, dtype, seed=5), 90, 9)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("n_sink", [1, 128, 200, 300])
@pytest.mark.parametrize("H,Hkv", [(1, 1), (3, 1), (4, 2)])
def test_sinks_of_a_long_sequence(dtype, d, n_sink, H, Hkv):
    """One or two sink tiles whose walk over the later queries is cut into parts (and three, where it is not), in a
    batch whose shorter sequences leave some parts empty."""
    lens = torch.tensor([1700, 1700, 130, 0], dtype=torch.int32, device=DEV)
    _check(*_inputs(4, H, Hkv, 1700, d, d, dtype, seed=16), 60, n_sink, lens)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("H,Hkv,window,n_sink", [(4, 1, 1500, 0), (8, 1, 100, 5), (4, 2, 300, 150), (8, 1, 200, 700), (3, 1, 1, 0)])
@pytest.mark.parametrize("lens", [[1500], [1500, 70, 0]])
def test_few_key_tiles_whose_walks_are_cut(dtype, d, H, Hkv, window, n_sink, lens):
    """Fewer key tiles than half of the SMs: every walk is cut, the sinks' into more parts than the others; without a
    window the last tiles have fewer query tiles than parts, and short sequences leave parts empty."""
    _check(*_inputs(len(lens), H, Hkv, 1500, d, d, dtype, seed=18), window, n_sink, torch.tensor(lens, dtype=torch.int32, device=DEV))


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.float32, 16), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("B,H,Hkv", [(5, 12, 4), (7, 7, 7)])
def test_more_work_than_multiprocessors(dtype, d, B, H, Hkv):
    """Every CTA takes several works in turn, of sequences of all lengths."""
    lens = torch.tensor([900, 0, 513, 1, 256, 899, 128][:B], dtype=torch.int32, device=DEV)
    _check(*_inputs(B, H, Hkv, 900, d, d, dtype, seed=17), 200, 20, lens)


@pytest.mark.parametrize("dtype,d", [(torch.float32, 32), (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("window,n_sink", [(50, 4), (1000, 0), (130, 140)])
def test_padded_batch_with_nan_behind_the_sequences(dtype, d, window, n_sink):
    """Whatever lies behind a sequence's end takes no part, and its rows of every output stay as they were."""
    lens = torch.tensor([300, 0, 1, 129, 128, 77, 9999, -5], dtype=torch.int32, device=DEV)
    L = 300
    q, k, v, dO = _inputs(8, 2, 1, L, d, d, dtype, seed=6)
    clean = [x.clone() for x in (q, k, v, dO)]
    for b, n in enumerate(lens.clamp(0, L).tolist()):
        for x in (q, k, v, dO):
            x[b, :, n:] = float("nan")
    o, lse, g = _check(q, k, v, dO, window, n_sink, lens)
    o0, lse0, g0 = _check(*clean, window, n_sink, lens)
    assert torch.equal(o, o0) and torch.equal(lse, lse0) and all(torch.equal(g[x], g0[x]) for x in g)
    for x in (o, lse, *g.values()):  # rows of arrays that the call made itself are zero
        for b, n in enumerate(lens.clamp(0, L).tolist()):
            assert bool((x[b, :, n:] == 0).all())
    half, _ = kdn.window_attn(q, k, v, window, n_sink=n_sink, lens=lens, lse=torch.full_like(lse, 7.0))
    assert torch.equal(half, o)
    o = torch.full_like(o, 7.0)
    lse = torch.full_like(lse, 7.0)
    kdn.window_attn(q, k, v, window, n_sink=n_sink, lens=lens, o=o, lse=lse)
    given = {"dq": torch.full_like(q, 7.0), "dk": torch.full_like(k, 7.0), "dv": torch.full_like(v, 7.0)}
    kdn.window_attn_backward(q, k, v, o, lse, dO, window, n_sink=n_sink, lens=lens, **given)
    for b, n in enumerate(lens.clamp(0, L).tolist()):
        for x, y in ((o, o0), (lse, lse0), *((given[a], g0[a]) for a in given)):
            assert bool((x[b, :, n:] == 7.0).all()) and torch.equal(x[b, :, :n], y[b, :, :n])


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128])
def test_large_scores_and_other_scales(dtype, d):
    """Scores of several hundred: the running maximum moves often, and most weights underflow."""
    q, k, v, dO = _inputs(1, 2, 1, 400, d, d, dtype, seed=7, scale=30.0)
    _check(q, k, v, dO, 150, 4)
    _check(q, k, v, dO, 150, 4, scale=1e-3)


@pytest.mark.parametrize("d", [64, 128])
def test_rising_scores(d):
    """Every key tile holds larger scores than all before it, and the first ones are very low."""
    q, k, v, dO = _inputs(1, 1, 1, 700, d, d, torch.bfloat16, seed=8)
    q[...] = 1.0
    k[...] = torch.linspace(-40, 40, 700, device=DEV).to(torch.bfloat16)[None, None, :, None] / d ** 0.5
    _check(q, k, v, dO, 700, 0)
    _check(q, k.flip(2).contiguous(), v, dO, 300, 2)


@pytest.mark.parametrize("dtype,out_dtype", [(torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16)])
def test_output_types(dtype, out_dtype):
    for d in (32, 64, 128):
        _check(*_inputs(2, 2, 1, 200, d, d, dtype, seed=9), 64, 2, out_dtype=out_dtype)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("L,window,n_sink", [(40, 1000, 0), (500, 3, 0), (500, 12, 4), (700, 200, 0), (900, 900, 0)])
def test_gradient_error_where_rows_see_few_keys(L, window, n_sink, d):
    """The error of dq and dk over the whole array, where delta from a rounded o would show.  The result's rounding and
    that of dS are independent, each uniform over a half step: together sqrt(2) of what rounding the exact gradient
    costs.  On the fp32 path (d = 32) only the first is there.  0.1 is left for the scatter of these sample sizes and
    the share of the rows beyond the first ones (1 / sqrt(n - 1) of a rounding for n keys)."""
    q, k, v, dO = _inputs(2, 4, 2, L, d, d, torch.bfloat16, seed=20)
    o, lse = kdn.window_attn(q, k, v, window, n_sink=n_sink)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, window, n_sink=n_sink)
    ref = dense(q, k, v, window, n_sink, dO=dO)
    for name in ("dq", "dk"):
        exact = ref[name][0]
        off = float((g[name].double() - exact).norm())
        rounded = float((exact.bfloat16().double() - exact).norm())
        assert off <= ((2.0 if d >= 64 else 1.0) ** 0.5 + 0.1) * rounded, name


@pytest.mark.parametrize("dtype,d", [(torch.float32, 16), (torch.float32, 32), (torch.float32, 128), (torch.bfloat16, 32),
                                     (torch.bfloat16, 64), (torch.bfloat16, 128)])
@pytest.mark.parametrize("L,window", [(1, 5), (300, 1)])
def test_a_softmax_over_one_key_has_no_gradient(L, window, dtype, d):
    """dq and dk are exactly zero, dv is dO summed over the heads that share it (its weights are within 2 u |s| of 1)."""
    q, k, v, dO = _inputs(2, 4, 2, L, d, d, dtype, seed=21)
    for out_dtype in (torch.float32, torch.bfloat16):
        o, lse, g = _check(q, k, v, dO, window, 0, out_dtype=out_dtype)
        assert bool((g["dq"] == 0).all()) and bool((g["dk"] == 0).all())
    # the first row of a longer sequence, next to rows that do have a gradient
    q, k, v, dO = _inputs(1, 2, 1, 80, d, d, dtype, seed=22)
    assert bool((_check(q, k, v, dO, 60, 3)[2]["dq"][:, :, 0] == 0).all())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_runs_are_equal_bit_for_bit(dtype):
    q, k, v, dO = _inputs(2, 6, 2, 900, 64, 64, dtype, seed=10)
    a = _check(q, k, v, dO, 200, 40)
    b = _check(q, k, v, dO, 200, 40)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and all(torch.equal(a[2][x], b[2][x]) for x in a[2])


def test_gradients_against_differences_on_the_gpu():
    """The directional derivative of sum(o dO) along random directions, fp32 (central differences of the float64
    reference's loss would test the reference; here the library's own o is differenced)."""
    q, k, v, dO = _inputs(1, 2, 1, 90, 32, 32, torch.float32, seed=11)
    o, lse = kdn.window_attn(q, k, v, 30, n_sink=3)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, 30, n_sink=3)
    gen = torch.Generator(device=DEV).manual_seed(12)
    h = 2.0 ** -7
    for i, name in enumerate(("dq", "dk", "dv")):
        x = [q, k, v]
        u = torch.randn(x[i].shape, generator=gen, device=DEV)
        u /= u.norm()
        loss = []
        for sign in (1, -1):
            y = list(x)
            y[i] = x[i] + sign * h * u
            loss.append((kdn.window_attn(*y, 30, n_sink=3)[0].double() * dO.double()).sum())
        diff = float(loss[0] - loss[1]) / (2 * h)
        want = float((g[name].double() * u.double()).sum())
        # o's fp32 error, up to about 1e-5 of sum|dO||v| over 5760 elements with random signs, is divided by 2 h = 2^-6;
        # the third derivative along a unit direction times h^2 / 6 is below 1e-4 of the gradient's norm
        assert abs(diff - want) <= 2e-2 * float(g[name].double().norm()) / 10 + 64 * 1e-6 * float(dO.norm())


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_empty_sequence_batch_of_none(dtype):
    q, k, v, dO = _inputs(1, 2, 1, 0, 64, 64, dtype)
    o, lse = kdn.window_attn(q, k, v, 4)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, 4)
    assert o.numel() == lse.numel() == g["dq"].numel() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_arrays_on_16_byte_boundaries(d, dtype):
    """The interface asks for 16-byte alignment, no more: every array here starts 16 bytes behind a larger boundary."""
    def moved(x):
        y = torch.empty(x.numel() + 64, dtype=x.dtype, device=DEV)[16 // x.element_size():][:x.numel()].view(x.shape)
        y.copy_(x)
        assert y.data_ptr() % 32 == 16
        return y

    q, k, v, dO = _inputs(1, 2, 1, 200, d, d, dtype, seed=18)
    o, lse = kdn.window_attn(q, k, v, 70, n_sink=2)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, 70, n_sink=2)
    q, k, v, dO = map(moved, (q, k, v, dO))
    o1, lse1 = kdn.window_attn(q, k, v, 70, n_sink=2, o=moved(torch.zeros_like(o)))
    assert torch.equal(o, o1) and torch.equal(lse, lse1)
    given = {"dq": moved(torch.zeros_like(q)), "dk": moved(torch.zeros_like(k)), "dv": moved(torch.zeros_like(v))}
    kdn.window_attn_backward(q, k, v, moved(o), lse1, dO, 70, n_sink=2, **given)
    assert all(torch.equal(given[x], g[x]) for x in g)


def test_own_stream_and_captured_graph():
    """Forward and backward on a side stream, then captured and replayed on new inputs, next to the eager results."""
    q, k, v, dO = _inputs(1, 4, 2, 513, 128, 128, torch.bfloat16, seed=13)
    o0, lse0 = kdn.window_attn(q, k, v, 200, n_sink=4)
    g0 = kdn.window_attn_backward(q, k, v, o0, lse0, dO, 200, n_sink=4)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    o1, lse1 = kdn.window_attn(q, k, v, 200, n_sink=4, stream=side)
    g1 = kdn.window_attn_backward(q, k, v, o1, lse1, dO, 200, n_sink=4, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(o0, o1) and torch.equal(lse0, lse1) and all(torch.equal(g0[x], g1[x]) for x in g0)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, lse2 = kdn.window_attn(q, k, v, 200, n_sink=4)
        g2 = kdn.window_attn_backward(q, k, v, o2, lse2, dO, 200, n_sink=4)
    for seed in (14, 15):
        for x, y in zip((q, k, v, dO), _inputs(1, 4, 2, 513, 128, 128, torch.bfloat16, seed=seed)):
            x.copy_(y)
        graph.replay()
        o, lse = kdn.window_attn(q, k, v, 200, n_sink=4)
        g = kdn.window_attn_backward(q, k, v, o, lse, dO, 200, n_sink=4)
        torch.cuda.synchronize()
        assert torch.equal(o, o2) and torch.equal(lse, lse2) and all(torch.equal(g[x], g2[x]) for x in g)


def test_refusals():
    q, k, v, dO = _inputs(1, 4, 2, 16, 64, 64, torch.bfloat16)
    for bad in (dict(window=0), dict(n_sink=-1), dict(scale=0.0)):
        with pytest.raises(kdn.KdnError):
            kdn.window_attn(q, k, v, **{"window": 4, **bad})
    with pytest.raises(kdn.KdnError, match="kv_heads"):
        kdn.window_attn(q[:, :3].contiguous(), k, v, 4)
    with pytest.raises(ValueError, match="contiguous"):
        kdn.window_attn(q.transpose(1, 2).contiguous().transpose(1, 2), k, v, 4)
    with pytest.raises(ValueError, match="lens"):
        kdn.window_attn(q, k, v, 4, lens=torch.ones(2, dtype=torch.int32, device=DEV))
    with pytest.raises(ValueError, match="dtype"):
        kdn.window_attn(q, k.float(), v, 4)
    o, lse = kdn.window_attn(q, k, v, 4)
    with pytest.raises(ValueError, match="dO"):
        kdn.window_attn_backward(q, k, v, o, lse, dO.float(), 4)
    with pytest.raises(kdn.KdnError, match="workspace_bytes"):
        kdn.window_attn_backward(q, k, v, o, lse, dO, 4, workspace=torch.empty(256, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dtype,d,backward", [(torch.bfloat16, 128, True), (torch.float32, 64, False)])
def test_offsets_beyond_32_bits(dtype, d, backward):
    """Arrays of more than 2^31 elements: the last head gives what it gives alone, bit for bit (the same tiles in the same
    order; the other heads' queries and dO are zero and add nothing to dk and dv)."""
    L = (1 << 17) + 77
    H = (1 << 31) // (L * d) + 2
    q = torch.zeros(1, H, L, d, device=DEV, dtype=dtype)
    assert q.numel() > 1 << 31
    q1, k, v, dO1 = _inputs(1, 1, 1, L, d, d, dtype, seed=3)
    q[:, -1:] = q1
    o, lse = kdn.window_attn(q, k, v, 70)
    o1, lse1 = kdn.window_attn(q1, k, v, 70)
    assert torch.equal(o[:, -1:], o1) and torch.equal(lse[:, -1:], lse1)
    if backward:
        dO = torch.zeros_like(q)
        dO[:, -1:] = dO1
        g = kdn.window_attn_backward(q, k, v, o, lse, dO, 70)
        g1 = kdn.window_attn_backward(q1, k, v, o1, lse1, dO1, 70)
        assert torch.equal(g["dq"][:, -1:], g1["dq"]) and torch.equal(g["dk"], g1["dk"]) and torch.equal(g["dv"], g1["dv"])


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("L,window,n_sink", [(40, 1000, 0), (500, 2, 0), (500, 3, 0), (500, 12, 4), (700, 200, 0), (900, 900, 0)])
def test_gradient_error_with_fp32_outputs(L, window, n_sink, d):
    """As test_gradient_error_where_rows_see_few_keys, for bf16 q, k, v with o and dO in fp32.  On the tensor cores dO is
    rounded to bf16 for its products: a third rounding next to those of dS and of the result, as large and independent of
    them: sqrt(3) in all.  That holds for a delta made from the same rounded dO (and, where rows see few keys, from the
    unrounded weights); the fp32 path (d = 32) has the result's rounding only."""
    q, k, v, dO = _inputs(2, 4, 2, L, d, d, torch.bfloat16, seed=23)
    dO = torch.randn(dO.shape, generator=torch.Generator(device=DEV).manual_seed(24), device=DEV)
    o, lse = kdn.window_attn(q, k, v, window, n_sink=n_sink, out_dtype=torch.float32)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, window, n_sink=n_sink)
    ref = dense(q, k, v, window, n_sink, dO=dO)
    for name in ("dq", "dk"):
        exact = ref[name][0]
        off = float((g[name].double() - exact).norm())
        rounded = float((exact.bfloat16().double() - exact).norm())
        assert off <= ((3.0 if d >= 64 else 1.0) ** 0.5 + 0.1) * rounded, (name, off / rounded)


@pytest.mark.parametrize("d", [32, 64, 128])
@pytest.mark.parametrize("out_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("L,window,n_sink", [(1200, 64, 800), (1000, 3, 40), (900, 20, 130)])
def test_gradient_error_of_small_windows_with_many_sinks(L, window, n_sink, out_dtype, d):
    """The same bounds where the sinks, not the window, decide how many keys a row sees."""
    q, k, v, dO = _inputs(2, 4, 2, L, d, d, torch.bfloat16, seed=25)
    dO = dO.to(out_dtype)
    o, lse = kdn.window_attn(q, k, v, window, n_sink=n_sink, out_dtype=out_dtype)
    g = kdn.window_attn_backward(q, k, v, o, lse, dO, window, n_sink=n_sink)
    ref = dense(q, k, v, window, n_sink, dO=dO)
    for name in ("dq", "dk"):
        exact = ref[name][0]
        off = float((g[name].double() - exact).norm())
        rounded = float((exact.bfloat16().double() - exact).norm())
        assert off <= ((2.0 if d >= 64 else 1.0) ** 0.5 + 0.1) * rounded, (name, off / rounded)
