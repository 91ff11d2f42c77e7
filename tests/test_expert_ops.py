"""The expert operators beside the layer call: grouped products, 8-bit activation checkpoints
and 4-bit expert products, against plain 64-bit implementations.

Tolerances, derived (a step of a type is torch.finfo(t).eps, a rounding is off by half a step):
  * a sum of K products in fp32: every addition is off by at most one step, 2^-23, of a partial
    sum that is at most S = sum |a_i b_i|; with the few operations around it (K + 8) 2^-23 S;
  * one rounding to bf16: 2^-8 of the value (fp32: 2^-24);
  * Phi (the normal distribution function): absolute error 2^-21; the sigmoid: relative error
    2^-20 + |v| 2^-23 (the exponent v log2 e is rounded to 2^-24 of itself), and below 2^-126, where
    exp(-v) leaves the range of fp32, an absolute error of 2^-126 (it may come out as 0).
Checkpoint bytes, scales, and the values read back are exact.
"""
import itertools
import math

import pytest
import torch

import sparse_mixture_experts_10_b200 as moe

BF, F32, F64 = torch.bfloat16, torch.float32, torch.float64
BAD = (moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED)


def half_step(dt):
    return torch.finfo(dt).eps / 2


def close(got, ref, tol):
    """got within tol of ref plus got's own rounding; NaN and infinities in the same places."""
    ref, got64 = ref.to(F64), got.to(F64)
    assert got.shape == ref.shape
    fine = torch.isfinite(ref)
    assert torch.equal(torch.isnan(ref), torch.isnan(got64))
    assert torch.equal(ref[~fine & ~torch.isnan(ref)], got64[~fine & ~torch.isnan(ref)])
    bound = tol + half_step(got.dtype) * (ref.abs() + tol) + 1e-37
    over = ((got64 - ref).abs() - bound)[fine]
    assert over.numel() == 0 or float(over.max()) <= 0, f"{float(over.max()):.3e} over the bound"


def randn(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * std).to(dtype)


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def status_clear():
    torch.cuda.synchronize()
    return moe.moe_get_device_status()


# ===================================================================== grouped products
def offsets(lengths, start=0):
    return [start] + [start + s for s in itertools.accumulate(lengths)]


def gmm_reference(kind, a, b, off, c_shape):
    """(result, S) in 64 bits; rows outside every segment are NaN in the result (not compared)."""
    ref = torch.full(c_shape, float("nan"), dtype=F64, device="cuda")
    S = torch.zeros(c_shape, dtype=F64, device="cuda")
    for g in range(len(off) - 1):
        lo, hi = off[g], off[g + 1]
        x = a[lo:hi].to(F64)
        if kind == moe.MOE_GMM_TN:
            y = b[lo:hi].to(F64)
            ref[g], S[g] = x.t() @ y, x.t().abs() @ y.abs()
        else:
            w = b[g].to(F64)
            w = w.t() if kind == moe.MOE_GMM_NT else w
            ref[lo:hi], S[lo:hi] = x @ w, x.abs() @ w.abs()
    return ref, S


def gmm_case(kind, lengths, n, k, dt, out, seed=0, start=0, extra=0, pads=(0, 0, 0), accumulate=False, run=None):
    """One product with `start` rows before the first segment, `extra` behind the last, and rows of a,
    b, c that are pads elements longer than they need to be (those, and rows outside the segments, keep
    what they hold)."""
    g = gen(seed)
    off = offsets(lengths, start)
    rows, G = off[-1] + extra, len(lengths)
    tn = kind == moe.MOE_GMM_TN
    aw, bw, cw = (k if kind == moe.MOE_GMM_NT else n), k, (n if kind == moe.MOE_GMM_NT else k)
    af = randn(g, rows, aw + pads[0], dtype=dt)
    bf = randn(g, *((rows,) if tn else (G, n)), bw + pads[1], dtype=dt)
    cf = randn(g, *((G, n) if tn else (rows,)), cw + pads[2], dtype=out)
    # what lies outside the operands must not reach a result
    af[..., aw:] = float("nan")
    bf[..., bw:] = float("inf")
    for t in (af, bf) if tn else (af,):
        t[:start] = float("nan")
        t[off[-1]:] = float("inf")
    before = cf.clone()
    a, b, c = af[..., :aw], bf[..., :bw], cf[..., :cw]
    d = moe.make_gmm(kind, G, n, k, moe.dtype_code(dt), moe.dtype_code(out), accumulate, aw + pads[0], bw + pads[1],
                     cw + pads[2])
    o = torch.tensor(off, dtype=torch.int32, device="cuda")
    (run or (lambda f: f()))(lambda: moe.check(moe.moe_grouped_mm(d, af, bf, cf, o, rows), "grouped_mm"))
    assert status_clear() == 0
    ref, S = gmm_reference(kind, a, b, off, c.shape)
    terms = max(lengths) if tn else (k if kind == moe.MOE_GMM_NT else n)
    if accumulate:
        ref, S = ref + before[..., :cw].to(F64), S + before[..., :cw].to(F64).abs()
    tol = (terms + 8) * 2.0 ** -23 * S
    if tn:
        close(c, ref, tol)
    else:
        close(c[start:off[-1]], ref[start:off[-1]], tol[start:off[-1]])
        assert torch.equal(cf[:start], before[:start]) and torch.equal(cf[off[-1]:], before[off[-1]:])
    assert torch.equal(cf[..., cw:], before[..., cw:])
    return cf


KINDS = [moe.MOE_GMM_NT, moe.MOE_GMM_NN, moe.MOE_GMM_TN]
TYPES = [(BF, BF), (BF, F32), (F32, F32)]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,out", TYPES)
@pytest.mark.parametrize("lengths,n,k", [
    ([1], 8, 8), ([0, 1, 0], 64, 64), ([5, 0, 130, 64, 1], 72, 200), ([129, 127, 256, 1, 0, 63], 264, 136),
    ([300, 17], 520, 72), ([2, 3, 65], 8, 1032), ([513], 256, 256), ([0, 0, 0], 32, 16), ([700, 0, 33, 257], 384, 512),
    ([300, 0, 1, 777, 129], 4104, 1000), ([130, 600, 2, 0, 511], 1000, 4104)])
def test_grouped_mm(kind, dt, out, lengths, n, k):
    if sum(lengths) == 0 and kind != moe.MOE_GMM_TN:
        gmm_case(kind, lengths, n, k, dt, out, extra=5)
        return
    gmm_case(kind, lengths, n, k, dt, out, seed=n + k)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,out", TYPES)
def test_grouped_mm_strides_and_rows_outside_the_segments(kind, dt, out):
    gmm_case(kind, [70, 0, 5, 200], 136, 200, dt, out, seed=1, start=3, extra=77, pads=(8, 16, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt,out", TYPES)
@pytest.mark.parametrize("lengths", [[64, 16, 48, 15, 17, 31, 33], [1040, 1024, 1008], [2000]])
def test_grouped_mm_widths_of_whole_chunks(kind, dt, out, lengths):
    """Widths that are multiples of 64 (with row strides that are not), lengths around multiples of 16 and 64."""
    gmm_case(kind, lengths, 320, 192, dt, out, seed=len(lengths), start=5, extra=3, pads=(24, 8, 16))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_long_sums_in_fp32(kind):
    """fp32 results of bf16 operands over 16384 terms: runs of at most 768 terms, 16 a step, each step off by
    at most 2^-23 of a partial sum, then at most 22 roundings of the runs' sum."""
    terms, other = 16384, 264
    g = gen(41)
    tn = kind == moe.MOE_GMM_TN
    n, k = (other, 136) if tn else (other, terms) if kind == moe.MOE_GMM_NT else (terms, other)
    rows = terms if tn else 130
    a = randn(g, rows, k if kind == moe.MOE_GMM_NT else n)
    b = randn(g, rows, k) if tn else randn(g, 1, n, k)
    c = torch.empty(*((1, n) if tn else (rows,)), n if kind == moe.MOE_GMM_NT else k, device="cuda")
    d = moe.make_gmm(kind, 1, n, k, moe.MOE_BF16, moe.MOE_F32)
    moe.check(moe.moe_grouped_mm(d, a, b, c, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), rows))
    ref, S = gmm_reference(kind, a, b, [0, rows], c.shape)
    close(c, ref, (768 / 16 + 22) * 2.0 ** -23 * S)
    # and in all no more than 1e-6 of the result: the losses towards zero do not add up over the whole length
    assert relative(c, ref) <= 1e-6


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("terms,other", [(1 << 23, 8), (40008, 72)])
def test_grouped_mm_long_sums_in_bf16(kind, terms, other):
    """bf16 results of sums without cancellation: runs of at most 16384 terms, 16 a step; a step drops less than 2^-25 of
    the partial sum for each term and 2^-23 at its end, 5 * 2^-23 in all; then 2^-24 for every run's addition."""
    g = gen(44)
    tn = kind == moe.MOE_GMM_TN
    n, k = (other, other) if tn else (other, terms) if kind == moe.MOE_GMM_NT else (terms, other)
    rows = terms if tn else other + 1
    a = randn(g, rows, k if kind == moe.MOE_GMM_NT else n).abs()
    b = (randn(g, rows, k) if tn else randn(g, 1, n, k)).abs()
    c = torch.empty(*((1, n) if tn else (rows,)), n if kind == moe.MOE_GMM_NT else k, dtype=BF, device="cuda")
    d = moe.make_gmm(kind, 1, n, k, moe.MOE_BF16, moe.MOE_BF16)
    moe.check(moe.moe_grouped_mm(d, a, b, c, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), rows))
    assert status_clear() == 0
    ref, S = gmm_reference(kind, a, b, [0, rows], c.shape)
    close(c, ref, (16384 / 16 * 5 + terms / 16384 / 2 + 8) * 2.0 ** -23 * S)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_long_sums_in_bf16_beside_short_ones(kind):
    """Several runs and a single one, in CTA pairs; row strides; a weight gradient that is added to."""
    if kind == moe.MOE_GMM_TN:
        for accumulate in (False, True):
            gmm_case(kind, [20000, 0, 33, 1500], 1288, 1280, BF, BF, seed=45, start=2, extra=9, pads=(8, 16, 24),
                     accumulate=accumulate)
    else:
        n, k = (2048, 16648) if kind == moe.MOE_GMM_NT else (16648, 2048)
        gmm_case(kind, [300, 0, 2300, 33], n, k, BF, BF, seed=46, start=2, extra=9, pads=(8, 16, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_graph_follows_new_offsets(kind):
    """A captured call reads its offsets when it is replayed: any other segments of as many rows."""
    n, k, rows = 136, 200, 400
    g = gen(42)
    tn = kind == moe.MOE_GMM_TN
    a = randn(g, rows, k if kind == moe.MOE_GMM_NT else n)
    b = randn(g, rows, k) if tn else randn(g, 4, n, k)
    c = torch.empty(*((4, n) if tn else (rows,)), n if kind == moe.MOE_GMM_NT else k, device="cuda")
    o = torch.tensor([0, 100, 200, 300, 400], dtype=torch.int32, device="cuda")
    d = moe.make_gmm(kind, 4, n, k, moe.MOE_BF16, moe.MOE_F32)
    moe.check(moe.moe_grouped_mm(d, a, b, c, o, rows))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.check(moe.moe_grouped_mm(d, a, b, c, o, rows))
    for off in ([0, 0, 0, 0, 400], [0, 1, 399, 399, 400], [0, 257, 258, 300, 400]):
        o.copy_(torch.tensor(off, dtype=torch.int32))
        c.fill_(7.0)
        graph.replay()
        assert status_clear() == 0
        ref, S = gmm_reference(kind, a, b, off, c.shape)
        close(c, ref, (400 + 8) * 2.0 ** -23 * S)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_grouped_mm_many_groups(kind, dt):
    g = torch.Generator().manual_seed(3)
    lengths = torch.randint(0, 9, (1024,), generator=g).tolist()
    lengths[500] = 300
    gmm_case(kind, lengths, 16, 40, dt, F32, seed=4)


@pytest.mark.gpu
@pytest.mark.parametrize("dt,out", TYPES)
def test_grouped_mm_adds_to_weight_gradients(dt, out):
    gmm_case(moe.MOE_GMM_TN, [100, 0, 31], 136, 72, dt, out, seed=5, accumulate=True, pads=(0, 0, 8))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_infinities_stay_in_their_segment(kind):
    """A NaN row or expert reaches its own results only, at segment borders inside a tile."""
    lengths, n, k = [40, 9, 90], 72, 136
    off = offsets(lengths)
    g = gen(6)
    tn = kind == moe.MOE_GMM_TN
    a = randn(g, off[-1], k if kind == moe.MOE_GMM_NT else n)
    b = randn(g, off[-1], k) if tn else randn(g, 3, n, k)
    c = torch.empty(*((3, n) if tn else (off[-1],)), n if kind == moe.MOE_GMM_NT else k, dtype=F32, device="cuda")
    (b[off[1]:off[2]] if tn else b[1]).fill_(float("nan"))
    a[off[1]:off[2]] = float("inf")
    d = moe.make_gmm(kind, 3, n, k, moe.MOE_BF16, moe.MOE_F32)
    moe.check(moe.moe_grouped_mm(d, a, b, c, torch.tensor(off, dtype=torch.int32, device="cuda"), off[-1]))
    parts = [c[0], c[1], c[2]] if tn else [c[off[i]:off[i + 1]] for i in range(3)]
    assert torch.isfinite(parts[0]).all() and torch.isfinite(parts[2]).all() and torch.isnan(parts[1]).all()


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_is_reproducible_and_captures(kind):
    """Bitwise the same eagerly, on a side stream, replayed from a graph, and beside a second call."""
    a = gmm_case(kind, [200, 0, 77, 300], 264, 328, BF, F32, seed=7)

    def on_side(f):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        torch.cuda.current_stream().wait_stream(s)

    def in_graph(f):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        for _ in range(3):
            graph.replay()

    def twice_at_once(f):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        f()
        torch.cuda.current_stream().wait_stream(s)

    for how in (on_side, in_graph, twice_at_once):
        assert torch.equal(a, gmm_case(kind, [200, 0, 77, 300], 264, 328, BF, F32, seed=7, run=how))


# Segments that take tiles of two accumulators (more than 256 rows a tile) and of one, with rows enough for tiles of
# 512 rows; each CTA pair works on several of them.
MIXED = [1500, 0, 700, 17, 900, 260, 200]


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [moe.MOE_GMM_NT, moe.MOE_GMM_NN])
@pytest.mark.parametrize("width,terms", [(4104, 1000), (4096, 640), (5120, 328), (4224, 2056)])
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_mm_tiles_of_512_rows(kind, width, terms, out):
    """bf16 results (fp32 ones have tiles of 256 rows) over many slices, in whole chunks of 64 and not, with row
    strides and NaN outside the operands."""
    n, k = (width, terms) if kind == moe.MOE_GMM_NT else (terms, width)
    gmm_case(kind, MIXED, n, k, BF, out, seed=width, start=3, extra=5, pads=(8, 16, 24))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", [moe.MOE_GMM_NT, moe.MOE_GMM_NN])
def test_grouped_mm_tiles_of_512_rows_in_many_groups(kind):
    """More groups than are put in order: long and short tiles alternate."""
    n, k = (2304, 136) if kind == moe.MOE_GMM_NT else (136, 2304)
    gmm_case(kind, [600, 40] * 66, n, k, BF, BF, seed=9)


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("n,k", [(1288, 1352), (1536, 1280)])
def test_grouped_mm_weight_gradients_of_cta_pairs(out, accumulate, n, k):
    gmm_case(moe.MOE_GMM_TN, [100, 0, 31, 330, 64, 1, 720], n, k, BF, out, seed=n, start=7, extra=9, pads=(8, 16, 24),
             accumulate=accumulate)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_mm_infinities_stay_in_their_segment_of_cta_pairs(kind, out):
    """Segments of NaN rows and experts between others, at borders inside a tile and a slice."""
    lengths, bad = [300, 9, 700, 64, 433, 50, 600], (1, 3, 5)
    off = offsets(lengths)
    n, k = (1288, 1352) if kind == moe.MOE_GMM_TN else (4104, 200) if kind == moe.MOE_GMM_NT else (200, 4104)
    g = gen(13)
    tn = kind == moe.MOE_GMM_TN
    a = randn(g, off[-1], k if kind == moe.MOE_GMM_NT else n)
    b = randn(g, off[-1], k) if tn else randn(g, len(lengths), n, k)
    c = torch.empty(*((len(lengths), n) if tn else (off[-1],)), n if kind == moe.MOE_GMM_NT else k, dtype=out, device="cuda")
    ref, S = gmm_reference(kind, a, b, off, c.shape)
    for i in bad:
        a[off[i]:off[i + 1]] = float("inf")
        (b[off[i]:off[i + 1]] if tn else b[i]).fill_(float("nan"))
    d = moe.make_gmm(kind, len(lengths), n, k, moe.MOE_BF16, moe.dtype_code(out))
    moe.check(moe.moe_grouped_mm(d, a, b, c, torch.tensor(off, dtype=torch.int32, device="cuda"), off[-1]))
    assert status_clear() == 0
    for i in range(len(lengths)):
        at = i if tn else slice(off[i], off[i + 1])
        if i in bad:
            assert torch.isnan(c[at]).all()
        else:
            close(c[at], ref[at], (max(lengths + [n if kind == moe.MOE_GMM_NN else k]) + 8) * 2.0 ** -23 * S[at])


def on_side(f):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    torch.cuda.current_stream().wait_stream(s)


def in_graph(f):
    f()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f()
    for _ in range(3):
        graph.replay()


def twice_at_once(f):
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        f()
    f()
    torch.cuda.current_stream().wait_stream(s)


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("out", [BF, F32])
def test_grouped_mm_of_cta_pairs_is_reproducible_and_captures(kind, out):
    n, k = (1288, 1352) if kind == moe.MOE_GMM_TN else (4104, 328) if kind == moe.MOE_GMM_NT else (328, 4104)
    first = gmm_case(kind, MIXED, n, k, BF, out, seed=14)
    for how in (on_side, in_graph, twice_at_once):
        assert torch.equal(first, gmm_case(kind, MIXED, n, k, BF, out, seed=14, run=how))


@pytest.mark.gpu
@pytest.mark.parametrize("kind", KINDS)
def test_grouped_mm_of_cta_pairs_follows_new_offsets_in_a_graph(kind):
    """Replays with other segments of as many rows, other numbers of tiles and of slices to clear."""
    n, k = (1288, 1352) if kind == moe.MOE_GMM_TN else (4104, 328) if kind == moe.MOE_GMM_NT else (328, 4104)
    g, rows, tn = gen(15), 3600, kind == moe.MOE_GMM_TN
    a = randn(g, rows, k if kind == moe.MOE_GMM_NT else n)
    b = randn(g, rows, k) if tn else randn(g, 7, n, k)
    c = torch.empty(*((7, n) if tn else (rows,)), n if kind == moe.MOE_GMM_NT else k, dtype=BF, device="cuda")
    o = torch.tensor(offsets([500] * 6 + [600]), dtype=torch.int32, device="cuda")
    d = moe.make_gmm(kind, 7, n, k)
    call = lambda: moe.check(moe.moe_grouped_mm(d, a, b, c, o, rows))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for lengths in ([0] * 6 + [3600], [3600] + [0] * 6, [1, 1799, 3, 1, 1000, 255, 541], [257, 513, 16, 0, 15, 1, 2798]):
        off = offsets(lengths)
        o.copy_(torch.tensor(off, dtype=torch.int32))
        c.fill_(float("nan"))
        graph.replay()
        assert status_clear() == 0
        ref, S = gmm_reference(kind, a, b, off, c.shape)
        close(c, ref, (rows + 8) * 2.0 ** -23 * S)


@pytest.mark.gpu
def test_grouped_mm_clamps_offsets_that_break_the_rule():
    d = moe.make_gmm(moe.MOE_GMM_NT, 3, 16, 16, moe.MOE_BF16, moe.MOE_F32)
    a, b = randn(gen(8), 20, 16), randn(gen(9), 3, 16, 16)
    for off, use in (([-5, 10, 4, 100], [0, 10, 10, 20]), ([0, 25, 30, 20], [0, 20, 20, 20])):
        c = torch.zeros(20, 16, device="cuda")
        moe.check(moe.moe_grouped_mm(d, a, b, c, torch.tensor(off, dtype=torch.int32, device="cuda"), 20))
        assert status_clear() == moe.MOE_STATUS_BOUNDS
        ref, S = gmm_reference(moe.MOE_GMM_NT, a, b, use, c.shape)
        close(c, ref, 24 * 2.0 ** -23 * S)


@pytest.mark.gpu
def test_grouped_mm_places_past_32_bits():
    """Results whose element index passes 2^32, and a weight gradient over as many rows."""
    rows, n, k = 270000, 16384, 64
    a, b = randn(gen(10), rows, k), randn(gen(11), 2, n, k)
    c = torch.zeros(rows, n, dtype=BF, device="cuda")
    off = torch.tensor([0, 1000, rows], dtype=torch.int32, device="cuda")
    d = moe.make_gmm(moe.MOE_GMM_NT, 2, n, k, moe.MOE_BF16, moe.MOE_BF16)
    moe.check(moe.moe_grouped_mm(d, a, b, c, off, rows))
    assert status_clear() == 0
    for lo, hi, e in ((0, 200, 0), (rows // 2, rows // 2 + 200, 1), (rows - 200, rows, 1)):
        x, w = a[lo:hi].double(), b[e].double()
        close(c[lo:hi], x @ w.t(), (k + 8) * 2.0 ** -23 * (x.abs() @ w.abs().t()))
    d = moe.make_gmm(moe.MOE_GMM_TN, 2, n, k, moe.MOE_BF16, moe.MOE_F32)
    dw = torch.empty(2, n, k, device="cuda")
    moe.check(moe.moe_grouped_mm(d, c, a, dw, off, rows))
    assert status_clear() == 0
    cols = slice(n - 128, n)
    x = c[1000:, cols].double()
    close(dw[1, cols], x.t() @ a[1000:].double(), (rows + 8) * 2.0 ** -23 * (x.abs().t() @ a[1000:].double().abs()))


@pytest.mark.gpu
@pytest.mark.parametrize("dt,width", [(BF, 8), (F32, 4)])
def test_grouped_mm_most_rows(dt, width):
    """The largest number of rows, most of them in one segment.  Entries are -1, 0 and 1, so the results are exact."""
    rows, part = 2 ** 31 - 1025, 1 << 26
    a = torch.empty(rows, width, dtype=dt, device="cuda")
    for lo in range(0, rows, part):
        a[lo:lo + part].random_(0, 3, generator=gen(lo)).sub_(1)
    off = torch.tensor([0, 3, 17, rows], dtype=torch.int32, device="cuda")
    b = torch.empty(3, width, width, dtype=dt, device="cuda").random_(0, 3, generator=gen(16)).sub_(1)
    c = torch.full((rows, width), float("nan"), dtype=dt, device="cuda")
    code = moe.dtype_code(dt)
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_NT, 3, width, width, code, code), a, b, c, off, rows))
    assert status_clear() == 0
    for g, (lo, hi) in enumerate(((0, 3), (3, 17))):
        assert torch.equal(c[lo:hi].double(), a[lo:hi].double() @ b[g].double().t())
    for lo in range(17, rows, part):
        x = a[lo:min(lo + part, rows)].float()
        want = sum(x[:, i:i + 1] * b[2, :, i].float() for i in range(width))
        assert torch.equal(c[lo:lo + part].float(), want)
    del c
    # weight gradients of 1024 segments
    off = torch.linspace(0, rows, 1025, dtype=F64).round().to(torch.int32).cuda()
    dw = torch.empty(1024, width, width, device="cuda")
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_TN, 1024, width, width, code, moe.MOE_F32), a, a, dw, off, rows))
    assert status_clear() == 0
    o = off.tolist()
    for g in (0, 1, 512, 1022, 1023):
        x = a[o[g]:o[g + 1]].double()
        assert torch.equal(dw[g].double(), x.t() @ x)


@pytest.mark.gpu
def test_grouped_mm_ragged_segment_behind_long_ones():
    """A segment whose length is no multiple of 16 behind one whose tiles take more than a second in all: the wait for
    its last slice begins with the call and is longer than any bound on one tile's work (2.2e15 operations, 1.6 s
    at the sustained rate, against 1.008 s).  Entries are -1, 0 and 1, so the sums are exact."""
    rows, tail, n = 262144, 17, 65536
    x = torch.empty(rows + tail, n, dtype=BF, device="cuda").random_(0, 3, generator=gen(12)).sub_(1)
    c = torch.full((2, n, n), float("nan"), dtype=BF, device="cuda")
    d = moe.make_gmm(moe.MOE_GMM_TN, 2, n, n, moe.MOE_BF16, moe.MOE_BF16)
    off = torch.tensor([0, rows, rows + tail], dtype=torch.int32, device="cuda")
    moe.check(moe.moe_grouped_mm(d, x, x, c, off, rows + tail))
    assert status_clear() == 0
    last = x[rows:].float()
    for i in range(0, n, 8192):
        assert torch.equal(c[1, i:i + 8192].float(), last[:, i:i + 8192].t() @ last)
    for i, j in ((0, 0), (0, n - 128), (n - 128, 4096), (n - 128, n - 128), (32768, 32640)):
        ref = x[:rows, i:i + 128].double().t() @ x[:rows, j:j + 128].double()
        assert torch.equal(c[0, i:i + 128, j:j + 128], ref.to(BF))


def test_grouped_mm_refusals():
    ok = dict(kind=0, groups=4, n=64, k=64)

    def rc(rows=16, a=256, b=256, c=256, off=256, **kw):
        return moe.moe_grouped_mm(moe.make_gmm(**{**ok, **kw}), a, b, c, off, rows, 0)

    for kw in (dict(kind=3), dict(kind=-1), dict(groups=0), dict(groups=1025), dict(n=0), dict(k=-8), dict(n=60),
               dict(k=12), dict(dtype=2), dict(out_dtype=5), dict(dtype=moe.MOE_F32, out_dtype=moe.MOE_BF16),
               dict(accumulate=True), dict(lda=56), dict(ldb=65), dict(ldc=60), dict(lda=-64), dict(rows=-1),
               dict(rows=2 ** 31), dict(a=None), dict(b=None), dict(c=None), dict(off=None), dict(a=264), dict(b=258),
               dict(c=264), dict(off=258)):
        assert rc(**kw) in BAD, kw
    d = moe.make_gmm(**ok)
    d.accumulate = 2
    assert moe.moe_grouped_mm(d, 256, 256, 256, 256, 16, 0) in BAD
    d = moe.make_gmm(**ok)
    d.reserved = 1
    assert moe.moe_grouped_mm(d, 256, 256, 256, 256, 16, 0) in BAD
    assert moe.load_library().moe_grouped_mm(None, 256, 256, 256, 256, 16, None) in BAD
    for kind in (moe.MOE_GMM_NT, moe.MOE_GMM_NN):   # no rows: nothing to do
        assert rc(rows=0, kind=kind, a=None, b=None, c=None, off=None) == moe.MOE_OK
    assert rc(rows=0, kind=moe.MOE_GMM_TN, c=None) in BAD


def test_grouped_mm_refuses_weights_beyond_64_bits():
    """n rows of ldb (ldc) elements whose bytes pass 2^63 and come out small or negative when multiplied."""
    for kind, ld in ((moe.MOE_GMM_NT, "ldb"), (moe.MOE_GMM_NN, "ldb"), (moe.MOE_GMM_TN, "ldc")):
        for n, s in ((2 ** 31 - 8, 2 ** 32), (2 ** 31 - 8, 2 ** 32 - 8), (2 ** 30, 2 ** 32)):
            d = moe.make_gmm(kind, 4, n, 64, accumulate=kind == moe.MOE_GMM_TN, **{ld: s})
            assert moe.moe_grouped_mm(d, None, None, None, None, 0, 0) == moe.MOE_ERR_UNSUPPORTED, (kind, n, s)


def test_grouped_mm_refuses_lengths_at_the_end_of_32_bits():
    """A contraction (or width) whose place after the last slice would pass 2^31."""
    for kind in KINDS:
        for dt, step in ((moe.MOE_BF16, 8), (moe.MOE_F32, 4)):
            for n, k in ((2 ** 31 - step, 8), (8, 2 ** 31 - step), (8, 2 ** 31 - 1024)):
                d = moe.make_gmm(kind, 1, n, k, dt, moe.MOE_F32, accumulate=kind == moe.MOE_GMM_TN)
                assert moe.moe_grouped_mm(d, None, None, None, None, 0, 0) in BAD, (kind, dt, n, k)


def test_grouped_mm_limits_weights_only():
    """The limit of 2^40 bytes is one on a group's weights: n rows of the other operands are not a thing."""
    for kind, n, k, kw in ((moe.MOE_GMM_NT, 2 ** 20, 64, {}), (moe.MOE_GMM_NN, 2 ** 20, 64, dict(ldc=2 ** 19)),
                           (moe.MOE_GMM_TN, 2 ** 20, 64, dict(ldb=2 ** 19, accumulate=True))):
        d = moe.make_gmm(kind, 4, n, k, **kw)
        assert moe.moe_grouped_mm(d, None, None, None, None, 0, 0) == moe.MOE_OK, kind


@pytest.mark.gpu
def test_grouped_mm_wide_results():
    """Rows of 2^20 results of a short contraction."""
    rows, n, k = 40, 2 ** 20, 64
    a, b = randn(gen(47), rows, k), randn(gen(48), 1, n, k)
    off = torch.tensor([0, rows], dtype=torch.int32, device="cuda")
    for dt in (BF, F32):
        c = torch.full((rows, n), float("nan"), dtype=dt, device="cuda")
        x, w = a.to(dt), b.to(dt)
        d = moe.make_gmm(moe.MOE_GMM_NT, 1, n, k, moe.dtype_code(dt), moe.dtype_code(dt))
        moe.check(moe.moe_grouped_mm(d, x, w, c, off, rows))
        assert status_clear() == 0
        ref, S = gmm_reference(moe.MOE_GMM_NT, a, b, [0, rows], c.shape)
        close(c, ref, (k + 8) * 2.0 ** -23 * S)


@pytest.mark.gpu
def test_grouped_mm_without_rows_clears_weight_gradients():
    c = torch.ones(3, 16, 24, device="cuda")
    d = moe.make_gmm(moe.MOE_GMM_TN, 3, 16, 16, moe.MOE_BF16, moe.MOE_F32, ldc=24)
    moe.check(moe.moe_grouped_mm(d, None, None, c, None, 0))
    torch.cuda.synchronize()
    assert int(c[..., :16].abs().sum()) == 0 and torch.equal(c[..., 16:], torch.ones_like(c[..., 16:]))
    d = moe.make_gmm(moe.MOE_GMM_TN, 3, 16, 16, moe.MOE_BF16, moe.MOE_F32, accumulate=True, ldc=24)
    c.fill_(2)
    moe.check(moe.moe_grouped_mm(d, None, None, c, None, 0))
    torch.cuda.synchronize()
    assert torch.equal(c, torch.full_like(c, 2))


# ===================================================================== 8-bit checkpoints
def saved_reference(u, group, fmt):
    """(q, scale bytes, values) of one half [rows, width], in 64 bits; q as int8 or e4m3 values."""
    rows, width = u.shape
    sg = -(-width // group)
    x = torch.zeros(rows, sg * group, dtype=F64)
    x[:, :width] = u.cpu().to(F64)
    x = x.view(rows, sg, group)
    L = 127.0 if fmt == moe.MOE_CKPT_INT8 else 448.0
    bad = ~torch.isfinite(x).all(2, keepdim=True)
    amax = torch.where(torch.isfinite(x), x, torch.zeros_like(x)).abs().amax(2, keepdim=True)
    e = torch.full(amax.shape, -126, dtype=torch.int32)
    for i in range(-126, 121 if L == 127 else 119):   # the smallest integer with amax <= L 2^e, up to the last
        e = torch.where((amax > L * 2.0 ** i) & (e == i), i + 1, e)
    y = (x / torch.tensor(2.0, dtype=F64) ** e).clamp(-L, L)
    if fmt == moe.MOE_CKPT_INT8:
        q = torch.round(y)
    else:
        lead = torch.floor(torch.log2(y.abs().clamp(min=2.0 ** -40)))
        step = torch.tensor(2.0, dtype=F64) ** (lead.clamp(min=-6) - 3)
        q = torch.round(y / step) * step
    q = torch.where(bad, torch.zeros_like(q), q)
    v = torch.where(bad, torch.full_like(q, float("nan")), q * torch.tensor(2.0, dtype=F64) ** e)
    s = torch.where(bad, 255, e + 127).to(torch.uint8).view(rows, sg)
    return q.view(rows, -1)[:, :width], s, v.view(rows, -1)[:, :width]


def held(q, fmt):
    return (q.view(torch.int8) if fmt == moe.MOE_CKPT_INT8 else q.view(torch.float8_e4m3fn)).cpu().to(F64)


def ckpt_inputs(rows, cols, dt, seed):
    g = gen(seed)
    u = torch.randn(rows, cols, generator=g, device="cuda") * torch.rand(rows, 1, generator=g, device="cuda") * 4
    return (u * (1 + 9 * (torch.rand(cols, generator=g, device="cuda") < 0.02))).to(dt)


def run_forward(d, u, rows, width, fmt, group, halves, h_pad=0):
    q = torch.full((rows, halves * width), 77, dtype=torch.uint8, device="cuda")
    s = torch.full((rows, halves * -(-width // group)), 78, dtype=torch.uint8, device="cuda")
    h = torch.full((rows, width + h_pad), 5.0, dtype=u.dtype, device="cuda")
    moe.check(moe.moe_ckpt_forward(d, u, rows, h, q, s), "ckpt_forward")
    return h, q, s


def silu_ref(v):
    return v * torch.sigmoid(v)


def sig_err(v):
    """Absolute error of the computed sigmoid."""
    return torch.sigmoid(v) * (2.0 ** -20 + v.abs() * 2.0 ** -23) + 2.0 ** -126


ACTS = {"gelu": moe.MOE_ACT_GELU, "swiglu": moe.MOE_ACT_SWIGLU}
FORMATS = [moe.MOE_CKPT_INT8, moe.MOE_CKPT_E4M3]


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("rows,width,group", [(1, 8, 32), (3, 72, 32), (5, 264, 64), (2, 2200, 128), (9, 256, 128),
                                              (7, 4104, 64), (130, 520, 32), (5200, 328, 64),
                                              (2400, 2056, 128)])
def test_ckpt_forward_and_backward(act, dt, fmt, rows, width, group):
    halves = 2 if act == "swiglu" else 1
    u = ckpt_inputs(rows, halves * width, dt, rows + width)
    d = moe.make_ckpt(width, ACTS[act], moe.dtype_code(dt), fmt, group)
    h, q, s = run_forward(d, u, rows, width, fmt, group, halves)
    back = torch.empty(rows, halves * width, dtype=F32, device="cuda")
    moe.check(moe.moe_ckpt_load(moe.make_ckpt(width, ACTS[act], moe.MOE_F32, fmt, group), q, s, rows, back))
    parts = [saved_reference(u[:, i * width:(i + 1) * width], group, fmt) for i in range(halves)]
    assert torch.equal(held(q, fmt), torch.cat([p[0] for p in parts], 1))
    assert torch.equal(s.cpu(), torch.cat([p[1] for p in parts], 1))
    values = torch.cat([p[2] for p in parts], 1)
    assert torch.equal(back.cpu().to(F64), values)
    # forward: the activation of u itself
    x = u.to(F64)
    if act == "gelu":
        close(h, x * torch.special.ndtr(x), x.abs() * 2.0 ** -21)
    else:
        x, y = x[:, :width], x[:, width:]
        close(h, silu_ref(x) * y, (x * y).abs() * (sig_err(x) + 2.0 ** -22 * torch.sigmoid(x)))
    # backward: from the checkpoint's values
    g = gen(rows)
    dh = randn(g, rows, width, dtype=dt, std=0.1)
    for w in (torch.rand(rows, generator=g, device="cuda"), None):
        du = torch.empty(rows, halves * width, dtype=dt, device="cuda")
        hw = torch.empty(rows, width, dtype=dt, device="cuda")
        dw = torch.empty(rows, device="cuda")
        moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, du, hw, dw), "ckpt_backward")
        assert status_clear() == 0
        v = values.cuda().requires_grad_()
        wt = torch.ones(rows, 1, dtype=F64, device="cuda") if w is None else w.to(F64)[:, None]
        d64 = dh.to(F64)
        if act == "gelu":
            hv = v * torch.special.ndtr(v)
        else:
            a, b = v[:, :width], v[:, width:]
            hv = silu_ref(a) * b
        ref_du, = torch.autograd.grad(hv, v, wt * d64)
        hv, v = hv.detach(), v.detach()
        gd = (wt * d64).abs()
        if act == "gelu":
            hv_tol, du_tol = v.abs() * 2.0 ** -21, gd * 2.0 ** -19
        else:
            a, b = v[:, :width], v[:, width:]
            sg, e = torch.sigmoid(a), sig_err(a)
            # |d/ds of s (1 + a (1 - s))| <= 1 + |a|; each further operation is off by 2^-24 of a term
            hv_tol = (a * b).abs() * (e + 2.0 ** -22 * sg)
            du_tol = torch.cat([gd * b.abs() * (1 + a.abs()) * (2 * e + 2.0 ** -21 * sg),
                                gd * a.abs() * (e + 2.0 ** -22 * sg)], 1)
        close(du, ref_du, du_tol + 2.0 ** -22 * ref_du.abs())
        close(hw, wt * hv, wt * (hv_tol + 2.0 ** -22 * hv.abs()))
        close(dw, (d64 * hv).sum(1),
              ((d64 * hv).abs() * (width + 16) * 2.0 ** -24).sum(1) + (d64.abs() * hv_tol).sum(1))
        # the optional outputs left out
        du2 = torch.empty_like(du)
        moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, du2, None, None))
        assert torch.equal(du, du2)


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["gelu", "swiglu"])
def test_ckpt_backward_matches_differences(act):
    """du and dw against central differences of the plain activation around the checkpoint's values."""
    rows, width = 4, 40
    halves = 2 if act == "swiglu" else 1
    u = ckpt_inputs(rows, halves * width, F32, 3)
    d = moe.make_ckpt(width, ACTS[act], moe.MOE_F32, moe.MOE_CKPT_INT8, 32)
    _, q, s = run_forward(d, u, rows, width, moe.MOE_CKPT_INT8, 32, halves)
    v = torch.empty(rows, halves * width, device="cuda")
    moe.check(moe.moe_ckpt_load(d, q, s, rows, v))
    dh, w = randn(gen(4), rows, width, dtype=F32), torch.rand(rows, device="cuda")
    du, dw = torch.empty_like(v), torch.empty(rows, device="cuda")
    moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, du, None, dw))

    def loss(v, w):
        hv = v * torch.special.ndtr(v) if act == "gelu" else silu_ref(v[:, :width]) * v[:, width:]
        return (w.to(F64)[:, None] * dh.to(F64) * hv).sum()

    v64, w64, step = v.to(F64), w.to(F64), 1e-4
    # the truncation error is step^2 / 6 times a third derivative, below 4 (1 + |up|) |w dh| here
    for r, c in itertools.product(range(rows), range(0, halves * width, 7)):
        p, m = v64.clone(), v64.clone()
        p[r, c] += step
        m[r, c] -= step
        num = (loss(p, w) - loss(m, w)) / (2 * step)
        scale = float((w64[r] * dh[r, c % width].to(F64)).abs()) * (1 + float(v64[r].abs().max())) ** 2
        assert abs(float(du[r, c]) - float(num)) <= 1e-5 * scale + 1e-7
    for r in range(rows):
        p, m = w64.clone(), w64.clone()
        p[r] += step
        m[r] -= step
        num = float((loss(v64, p) - loss(v64, m)) / (2 * step))
        assert abs(float(dw[r]) - num) <= 1e-5 * (1 + abs(num))


def cdf_err(v, dt):
    """Relative error of the computed Phi for v < 0, where a small value is no difference of large ones.
    fp32: the exponent v^2 / 2 is rounded three times (v^2, the constant, the product), 0.75 v^2 of 2^-23; 2^x is off by
    2 of them, t by 1.5 and the polynomial by up to twice as much for it, by 2 for its sum and fit, the product by 0.5:
    0.75 v^2 + 7.5, below v^2 + 1.5 |v| + 6 from 1 on.  bf16: the fit's 2^-12.3, the exponent's 2^-23 v^2 / 2
    (v^2 of an 8-bit value is exact) and 2^-18 of the special-function unit and the sum: below 1.1 2^-12 down to
    v = -13.2."""
    return 2.0 ** -23 * (v * v + 1.5 * v.abs() + 6) if dt == F32 else torch.full_like(v, 1.1 * 2.0 ** -12)


def cdf(v):
    """Phi in 64 bits; torch.special.ndtr is 0 on the device from -8.3 down, where Phi is 5e-17."""
    return 0.5 * torch.special.erfc(v * -math.sqrt(0.5))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
def test_ckpt_gelu_of_negative_values_keeps_its_relative_error(dt):
    """h, w h and its derivative from -1 to -13 (each group of the checkpoint has values of one size)."""
    width, rows = 1536, 3
    u = -torch.linspace(1, 13, rows * width, device="cuda").view(rows, width).to(dt)
    d = moe.make_ckpt(width, moe.MOE_ACT_GELU, moe.dtype_code(dt), moe.MOE_CKPT_INT8, 32)
    h, q, s = run_forward(d, u, rows, width, moe.MOE_CKPT_INT8, 32, 1)
    x = u.to(F64)
    ref = x * cdf(x)
    close(h, ref, ref.abs() * cdf_err(x, dt))
    v = torch.empty(rows, width, device="cuda")
    moe.check(moe.moe_ckpt_load(moe.make_ckpt(width, moe.MOE_ACT_GELU, moe.MOE_F32, moe.MOE_CKPT_INT8, 32), q, s, rows, v))
    v = v.to(F64)
    dh, w = torch.ones(rows, width, dtype=dt, device="cuda"), torch.tensor([1.0, 0.5, 2.0], device="cuda")
    du, hw = torch.empty_like(u), torch.empty_like(u)
    moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, du, hw, None))
    assert status_clear() == 0
    wt, below = w.to(F64)[:, None], cdf(v)
    close(hw, wt * v * below, wt * (v * below).abs() * (cdf_err(v, dt) + 2.0 ** -23))
    slope = v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)   # v times the density, off by 2^-23 (0.75 v^2 + 8)
    close(du, wt * (below + slope), wt * (below * cdf_err(v, dt) + slope.abs() * 2.0 ** -23 * (0.75 * v * v + 8) +
                                        (below + slope).abs() * 2.0 ** -23))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_ckpt_of_plain_rows(dt, fmt):
    """MOE_ACT_NONE: rows saved and read back in their own type, with row strides."""
    rows, width, group = 33, 328, 64
    full = ckpt_inputs(rows, width + 8, dt, 11)
    d = moe.make_ckpt(width, moe.MOE_ACT_NONE, moe.dtype_code(dt), fmt, group, ldu=width + 8)
    q = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, -(-width // group), dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_ckpt_forward(d, full, rows, None, q, s))
    out = torch.full_like(full, 3.0)
    moe.check(moe.moe_ckpt_load(d, q, s, rows, out))
    rq, rs, rv = saved_reference(full[:, :width], group, fmt)
    assert torch.equal(held(q, fmt), rq) and torch.equal(s.cpu(), rs)
    assert torch.equal(out[:, :width].cpu().to(F64), rv)
    assert torch.equal(out[:, width:], torch.full_like(out[:, width:], 3.0))


@pytest.mark.gpu
@pytest.mark.parametrize("dt", [BF, F32])
@pytest.mark.parametrize("fmt", FORMATS)
def test_ckpt_extremes(dt, fmt):
    """Zeros, the smallest and largest values, values at the scale's borders, infinities and NaN."""
    group, width = 32, 32
    L = 127.0 if fmt == moe.MOE_CKPT_INT8 else 448.0
    rowsv = [torch.zeros(32), -torch.zeros(32), torch.full((32,), 2.0 ** -126), torch.full((32,), torch.finfo(dt).max),
             torch.full((32,), L), torch.full((32,), L) * (1 + torch.finfo(dt).eps), torch.arange(32) * 0.5,
             torch.tensor([L] + [i + 0.5 for i in range(31)]), torch.tensor([-L] + [2.0 ** -i for i in range(31)]),
             torch.tensor([1.0] * 31 + [float("inf")]), torch.tensor([float("nan")] + [1.0] * 31),
             torch.tensor([1.0] * 31 + [-float("inf")]), torch.full((32,), 2.0 ** -133)]
    u = torch.stack(rowsv).to(dt).cuda()
    rows = u.shape[0]
    d = moe.make_ckpt(width, moe.MOE_ACT_NONE, moe.dtype_code(dt), fmt, group)
    q = torch.empty(rows, width, dtype=torch.uint8, device="cuda")
    s = torch.empty(rows, 1, dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_ckpt_forward(d, u, rows, None, q, s))
    v = torch.empty(rows, width, device="cuda")
    moe.check(moe.moe_ckpt_load(moe.make_ckpt(width, moe.MOE_ACT_NONE, moe.MOE_F32, fmt, group), q, s, rows, v))
    rq, rs, rv = saved_reference(u, group, fmt)
    assert torch.equal(s.cpu(), rs)
    assert torch.equal(held(q, fmt), rq)
    assert torch.equal(torch.nan_to_num(v.cpu().to(F64), nan=-1e300), torch.nan_to_num(rv, nan=-1e300))
    # a NaN group's gradients are NaN, its neighbours' are not
    d = moe.make_ckpt(width, moe.MOE_ACT_GELU, moe.dtype_code(dt), fmt, group)
    du = torch.empty(rows, width, dtype=dt, device="cuda")
    dw = torch.empty(rows, device="cuda")
    moe.check(moe.moe_ckpt_backward(d, q, s, rows, torch.ones_like(u), None, du, None, dw))
    nan = torch.isnan(rv).any(1)
    assert torch.equal(torch.isnan(du).all(1).cpu(), nan) and torch.equal(torch.isnan(dw).cpu(), nan)


@pytest.mark.gpu
def test_ckpt_strides_graph_and_reproducibility():
    rows, width, group = 50, 264, 64
    full = ckpt_inputs(rows, 2 * width + 16, BF, 21)
    d = moe.make_ckpt(width, moe.MOE_ACT_SWIGLU, moe.MOE_BF16, moe.MOE_CKPT_INT8, group, ldu=2 * width + 16,
                      ldh=width + 8)
    tight = moe.make_ckpt(width, moe.MOE_ACT_SWIGLU, moe.MOE_BF16, moe.MOE_CKPT_INT8, group)
    h, q, s = run_forward(d, full, rows, width, moe.MOE_CKPT_INT8, group, 2, h_pad=8)
    h2, q2, s2 = run_forward(tight, full[:, :2 * width].contiguous(), rows, width, moe.MOE_CKPT_INT8, group, 2)
    assert torch.equal(h[:, :width], h2) and torch.equal(q, q2) and torch.equal(s, s2)
    assert torch.equal(h[:, width:], torch.full_like(h[:, width:], 5.0))
    dh = randn(gen(22), rows, width + 8)
    w = torch.rand(rows, device="cuda")
    outs = [torch.full((rows, 2 * width + 16), 9.0, dtype=BF, device="cuda"),
            torch.full((rows, width + 8), 9.0, dtype=BF, device="cuda"), torch.empty(rows, device="cuda")]
    moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, *outs))
    assert torch.equal(outs[0][:, 2 * width:], torch.full_like(outs[0][:, 2 * width:], 9.0))
    assert torch.equal(outs[1][:, width:], torch.full_like(outs[1][:, width:], 9.0))
    first = [o.clone() for o in outs]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        moe.check(moe.moe_ckpt_forward(d, full, rows, h, q, s))
        moe.check(moe.moe_ckpt_backward(d, q, s, rows, dh, w, *outs))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, outs))


@pytest.mark.gpu
def test_ckpt_places_past_32_bits():
    rows, width = 300000, 8192   # 4.9e9 values of u
    u = torch.zeros(rows, 2 * width, dtype=BF, device="cuda")
    u[-3:] = ckpt_inputs(3, 2 * width, BF, 31)
    d = moe.make_ckpt(width, moe.MOE_ACT_SWIGLU, moe.MOE_BF16, moe.MOE_CKPT_E4M3, 128)
    h, q, s = run_forward(d, u, rows, width, moe.MOE_CKPT_E4M3, 128, 2)
    last = u[-3:].clone()
    h2, q2, s2 = run_forward(d, last, 3, width, moe.MOE_CKPT_E4M3, 128, 2)
    assert torch.equal(h[-3:], h2) and torch.equal(q[-3:], q2) and torch.equal(s[-3:], s2)
    moe.check(moe.moe_ckpt_backward(d, q, s, rows, h, None, u, None, None))   # du in u's place
    du2 = torch.empty_like(last)
    moe.check(moe.moe_ckpt_backward(d, q2, s2, 3, h2, None, du2, None, None))
    assert torch.equal(u[-3:], du2)


def test_ckpt_refusals():
    def d(**kw):
        return moe.make_ckpt(**{**dict(width=64), **kw})

    def fwd(c, u=256, rows=4, h=256, q=256, s=256):
        return moe.moe_ckpt_forward(c, u, rows, h, q, s, 0)

    def bwd(c, q=256, s=256, rows=4, dh=256, w=256, du=256, hw=256, dw=256):
        return moe.moe_ckpt_backward(c, q, s, rows, dh, w, du, hw, dw, 0)

    bad = [d(width=0), d(width=-8), d(width=60), d(width=2, dtype=moe.MOE_F32), d(act=3), d(act=-1), d(dtype=4),
           d(format=2), d(group=16), d(group=96), d(group=256), d(ldu=120), d(ldu=129), d(ldh=63), d(ldh=68)]
    r = d()
    r.reserved = 1
    for c in bad + [r]:
        assert fwd(c) in BAD and bwd(c) in BAD
        assert moe.moe_ckpt_load(c, 256, 256, 4, 256, 0) in BAD
    for kw in (dict(u=None), dict(h=None), dict(q=None), dict(s=None), dict(rows=-1), dict(rows=2 ** 31), dict(u=264),
               dict(h=260), dict(q=257)):
        assert fwd(d(), **kw) in BAD, kw
    for kw in (dict(q=None), dict(s=None), dict(dh=None), dict(du=None), dict(rows=-1), dict(dh=258), dict(du=264),
               dict(hw=264), dict(q=264), dict(w=258), dict(dw=257)):
        assert bwd(d(), **kw) in BAD, kw
    assert bwd(d(act=moe.MOE_ACT_NONE)) in BAD
    assert moe.moe_ckpt_load(d(), 256, 256, 4, None, 0) in BAD
    assert fwd(d(), u=None, rows=0) == moe.MOE_OK and bwd(d(), dh=None, rows=0) == moe.MOE_OK
    assert moe.load_library().moe_ckpt_forward(None, 256, 4, 256, 256, 256, None) in BAD


# ===================================================================== 4-bit weights
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def q4_values(codes, scales, k, group, fmt):
    """Weights in 64 bits."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()
    if fmt == moe.MOE_Q4_INT4:
        v, sc = (q - 8).to(F64), scales.to(F64)
    else:
        v = torch.tensor(E2M1 + [-x for x in E2M1], dtype=F64, device=codes.device)[q]
        sc = torch.where(scales == 255, float("nan"), 2.0 ** (scales.to(F64) - 127))
    return v * sc.repeat_interleave(group, -1)[..., :k]


def q4_weights(g, N, n, k, group, fmt):
    codes = torch.randint(0, 256, (N, n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    sg = -(-k // group)
    if fmt == moe.MOE_Q4_INT4:
        return codes, (torch.rand(N, n, sg, generator=g, device="cuda") * 0.02).to(BF)
    return codes, torch.randint(110, 124, (N, n, sg), generator=g, device="cuda", dtype=torch.uint8)


def q4_case(N, n, k, group, fmt, act, pairs, x_div, out, gate, seed=0, experts=None, run=None):
    g = gen(seed)
    codes, scales = q4_weights(g, N, n, k, group, fmt)
    x = randn(g, -(-pairs // x_div), k)
    if experts is None:
        experts = torch.randint(0, N, (pairs,), generator=g, device="cuda").tolist()
    e = torch.tensor(experts, dtype=torch.int32, device="cuda")
    w = torch.rand(pairs, generator=g, device="cuda") if gate else None
    cols = n // 2 if act == moe.MOE_ACT_SWIGLU else n
    y = torch.full((pairs + 2, cols), 7.0, dtype=out, device="cuda")
    d = moe.make_q4(N, n, k, group, fmt, act)
    (run or (lambda f: f()))(lambda: moe.check(
        moe.moe_q4_matvec(d, x, pairs, x_div, e, codes, scales, w, y, moe.dtype_code(out)), "q4_matvec"))
    status = status_clear()
    assert torch.equal(y[pairs:], torch.full_like(y[pairs:], 7.0))
    W = q4_values(codes, scales, k, group, fmt)
    ref = torch.zeros(pairs, cols, dtype=F64, device="cuda")
    tol = torch.zeros_like(ref)
    for p, ex in enumerate(experts):
        if not 0 <= ex < N:
            continue
        v = x[p // x_div].to(F64)
        a, err = W[ex] @ v, (k + 8) * 2.0 ** -23 * (W[ex].abs() @ v.abs())
        if act == moe.MOE_ACT_GELU:      # |gelu'| < 1.13
            a, err = a * torch.special.ndtr(a), 1.13 * err + a.abs() * 2.0 ** -21
        elif act == moe.MOE_ACT_SWIGLU:  # |silu'| < 1.1
            ga, up, eg, eu = a[:cols], a[cols:], err[:cols], err[cols:]
            a = silu_ref(ga) * up
            err = 1.1 * eg * (up.abs() + eu) + silu_ref(ga).abs() * eu + (ga * up).abs() * sig_err(ga) + a.abs() * 2.0 ** -22
        gw = 1.0 if w is None else float(w[p])
        ref[p], tol[p] = gw * a, gw * (err + 2.0 ** -23 * a.abs())
    close(y[:pairs], ref, tol)
    return y, status


FMT_GROUPS = [(moe.MOE_Q4_INT4, 32), (moe.MOE_Q4_INT4, 64), (moe.MOE_Q4_INT4, 128), (moe.MOE_Q4_E2M1, 32)]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", FMT_GROUPS)
@pytest.mark.parametrize("act", [moe.MOE_ACT_NONE, moe.MOE_ACT_GELU, moe.MOE_ACT_SWIGLU])
@pytest.mark.parametrize("N,n,k,pairs,x_div", [(1, 16, 32, 1, 1), (4, 48, 96, 5, 1), (8, 144, 288, 12, 4),
                                               (3, 272, 1056, 40, 2), (16, 32, 2880, 64, 4), (2, 2064, 160, 70, 1)])
def test_q4_matvec(fmt, group, act, N, n, k, pairs, x_div):
    _, status = q4_case(N, n, k, group, fmt, act, pairs, x_div, BF, gate=False, seed=n + k)
    assert status == 0
    _, status = q4_case(N, n, k, group, fmt, act, pairs, x_div, F32, gate=True, seed=n + k + 1)
    assert status == 0


@pytest.mark.gpu
def test_q4_matvec_eight_rows_of_n():
    """n a multiple of 8 but not of 16, and every pair on one expert, more pairs than any batch."""
    for n in (8, 24, 136):
        q4_case(3, n, 64, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, 9, 1, F32, True, seed=n)
    q4_case(3, 40, 96, 32, moe.MOE_Q4_E2M1, moe.MOE_ACT_NONE, 300, 3, F32, True, seed=1, experts=[2] * 300)


@pytest.mark.gpu
def test_q4_matvec_dropped_and_bad_experts():
    """-1 is a dropped assignment: zeros.  Another index out of range: zeros and the status bit."""
    y, status = q4_case(4, 32, 64, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_SWIGLU, 6, 2, F32, True,
                        experts=[0, -1, 3, 3, -1, 1])
    assert status == 0 and int((y[1] != 0).sum()) == 0 and int((y[4] != 0).sum()) == 0
    y, status = q4_case(4, 32, 64, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, 5, 1, BF, False,
                        experts=[4, 0, -2, 1 << 30, 2])
    assert status == moe.MOE_STATUS_BOUNDS
    q4_case(4, 32, 64, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, 3, 1, BF, False, experts=[-1, -1, -1])


@pytest.mark.gpu
def test_q4_matvec_most_pairs_and_experts():
    g = torch.Generator().manual_seed(2)
    experts = torch.randint(0, 1024, (4096,), generator=g).tolist()
    q4_case(1024, 16, 32, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, 4096, 8, F32, False, experts=experts)


@pytest.mark.gpu
def test_q4_matvec_streams_and_graphs():
    args = (8, 96, 416, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_SWIGLU, 24, 4, BF, True)
    first, _ = q4_case(*args, seed=5)

    def in_graph(f):
        f()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            f()
        for _ in range(3):
            graph.replay()

    def on_two_streams(f):
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            f()
        f()
        torch.cuda.current_stream().wait_stream(s)

    for how in (in_graph, on_two_streams):
        again, _ = q4_case(*args, seed=5, run=how)
        assert torch.equal(first, again)


@pytest.mark.gpu
def test_q4_matvec_graph_follows_new_experts():
    """A captured call reads its experts when it is replayed."""
    N, n, k, pairs = 8, 96, 416, 24
    g = gen(43)
    codes, scales = q4_weights(g, N, n, k, 32, moe.MOE_Q4_INT4)
    x = randn(g, pairs, k)
    e = torch.zeros(pairs, dtype=torch.int32, device="cuda")
    y = torch.empty(pairs, n, device="cuda")
    d = moe.make_q4(N, n, k, 32)
    call = lambda: moe.check(moe.moe_q4_matvec(d, x, pairs, 1, e, codes, scales, None, y, moe.MOE_F32))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    W = q4_values(codes, scales, k, 32, moe.MOE_Q4_INT4)
    for new in ([3] * pairs, list(range(8)) * 3, [-1] * 20 + [7, 0, 7, 1]):
        e.copy_(torch.tensor(new, dtype=torch.int32))
        y.fill_(9.0)
        graph.replay()
        assert status_clear() == 0
        for p, ex in enumerate(new):
            ref, S = (W[ex] @ x[p].to(F64), W[ex].abs() @ x[p].to(F64).abs()) if ex >= 0 else (torch.zeros(n, dtype=F64, device="cuda"),) * 2
            close(y[p], ref, (k + 8) * 2.0 ** -23 * S)


@pytest.mark.gpu
def test_q4_matvec_wide_rows():
    """Rows of x of which shared memory holds only a few at a time, and one at the limit; longer ones are refused."""
    q4_case(2, 32, 14336, 128, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, 9, 1, F32, False, seed=1)
    q4_case(2, 16, 40960, 32, moe.MOE_Q4_E2M1, moe.MOE_ACT_SWIGLU, 3, 1, F32, False, seed=2)
    d = moe.make_q4(1, 16, 1 << 20, 128)
    t = torch.empty(1 << 20, dtype=BF, device="cuda")
    e = torch.zeros(1, dtype=torch.int32, device="cuda")
    assert moe.moe_q4_matvec(d, t, 1, 1, e, t, t, None, t, moe.MOE_F32) == moe.MOE_ERR_UNSUPPORTED


@pytest.mark.gpu
@pytest.mark.parametrize("k,pairs", [(41728, 4096), (49920, 64)])
def test_q4_matvec_widest_rows(k, pairs):
    """The largest k for the most pairs, and the most pairs for the largest k."""
    q4_case(2, 16, k, 128, moe.MOE_Q4_INT4, moe.MOE_ACT_NONE, pairs, 8, F32, True, seed=3)


def test_q4_matvec_refuses_rows_beyond_shared_memory():
    """Before anything is asked of a device: one chunk of 256 above the documented limits."""
    for k, pairs in ((41760, 4096), (49952, 1), (1 << 20, 1)):
        for fmt in (moe.MOE_Q4_INT4, moe.MOE_Q4_E2M1):
            d = moe.make_q4(4, 32, k, 32, fmt)
            rc = moe.moe_q4_matvec(d, 256, pairs, 1, 256, 256, 256, None, 256, moe.MOE_F32, 0)
            assert rc == moe.MOE_ERR_UNSUPPORTED, (k, pairs, rc)
    # no pairs: nothing to do, whatever the rows
    assert moe.moe_q4_matvec(moe.make_q4(4, 32, 1 << 20, 32), None, 0, 1, None, None, None, None, None, 0, 0) == moe.MOE_OK


@pytest.mark.gpu
def test_q4_matvec_special_scales_and_inputs():
    """A NaN scale or an infinite input reaches the results that use it, and no others; e2m1's extreme
    exponents and subnormal int4 scales count."""
    N, n, k = 2, 32, 128
    for fmt in (moe.MOE_Q4_INT4, moe.MOE_Q4_E2M1):
        codes, scales = q4_weights(gen(1), N, n, k, 32, fmt)
        codes[codes == 0x88] = 0x99
        x = randn(gen(2), 2, k)
        scales[0, 5, 1] = 255 if fmt == moe.MOE_Q4_E2M1 else float("nan")
        if fmt == moe.MOE_Q4_E2M1:
            scales[0, 6], scales[0, 7] = 0, 230
        else:
            scales[0, 6], scales[0, 7] = 2.0 ** -130, 2.0 ** 100
        y = torch.empty(2, n, device="cuda")
        d = moe.make_q4(N, n, k, 32, fmt)
        e = torch.tensor([0, 1], dtype=torch.int32, device="cuda")
        moe.check(moe.moe_q4_matvec(d, x, 2, 1, e, codes, scales, None, y, moe.MOE_F32))
        W = q4_values(codes, scales, k, 32, fmt)
        ref = torch.stack([W[p] @ x[p].to(F64) for p in range(2)])
        S = torch.stack([W[p].abs() @ x[p].to(F64).abs() for p in range(2)])
        assert torch.isnan(ref[0, 5]) and int(torch.isnan(ref).sum()) == 1
        close(y, ref, torch.nan_to_num((k + 8) * 2.0 ** -23 * S))
        x[1, 40] = float("inf")
        moe.check(moe.moe_q4_matvec(d, x, 2, 1, e, codes, scales, None, y, moe.MOE_F32))
        assert not torch.isfinite(y[1]).any() and torch.isfinite(y[0]).sum() == n - 1


@pytest.mark.gpu
@pytest.mark.parametrize("out", [BF, F32])
def test_q4_matvec_gelu_of_negative_products_keeps_its_relative_error(out):
    """A matrix of ones and zeros passes x[0] on exactly: GELU of each bf16 value from -1 to -13."""
    n, k = 16, 32
    v = -torch.linspace(1, 13, 400, device="cuda").to(BF).unique()
    pairs = v.numel()
    x = torch.zeros(pairs, k, dtype=BF, device="cuda")
    x[:, 0] = v
    codes = torch.full((1, n, k // 2), 0x88, dtype=torch.uint8, device="cuda")
    codes[..., 0] = 0x89   # 1, then zeros
    scales = torch.ones(1, n, 1, dtype=BF, device="cuda")
    y = torch.empty(pairs, n, dtype=out, device="cuda")
    d = moe.make_q4(1, n, k, 32, moe.MOE_Q4_INT4, moe.MOE_ACT_GELU)
    e = torch.zeros(pairs, dtype=torch.int32, device="cuda")
    moe.check(moe.moe_q4_matvec(d, x, pairs, 1, e, codes, scales, None, y, moe.dtype_code(out)))
    assert status_clear() == 0
    a = v.to(F64)[:, None].expand(pairs, n)
    ref = a * cdf(a)
    close(y, ref, ref.abs() * cdf_err(a, F32))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", FMT_GROUPS)
@pytest.mark.parametrize("dt", [BF, F32])
def test_q4_quantize_and_dequantize(fmt, group, dt):
    N, n, k = 3, 24, 416
    W = randn(gen(7), N, n, k, dtype=dt)
    W[0, 0], W[0, 1, :5] = 0.0, float("inf")
    W[0, 2, 3], W[0, 3] = float("nan"), torch.finfo(dt).tiny
    W[1, 0, :8] = torch.tensor([6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0])
    W[1, 0, 8:group] = 0
    sg = -(-k // group)
    codes = torch.empty(N, n, k // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(N, n, sg, dtype=BF if fmt == moe.MOE_Q4_INT4 else torch.uint8, device="cuda")
    d = moe.make_q4(N, n, k, group, fmt)
    moe.check(moe.moe_q4_quantize(d, W, moe.dtype_code(dt), codes, scales), "quantize")
    w = torch.zeros(N, n, sg * group, dtype=F64, device="cuda")
    w[..., :k] = W.to(F64)
    w = w.view(N, n, sg, group)
    bad = ~torch.isfinite(w).all(-1)
    amax = torch.where(bad[..., None], 0.0, w).abs().amax(-1)
    values = q4_values(codes, scales, k, group, fmt)
    assert torch.equal(torch.isnan(values), bad.repeat_interleave(group, -1)[..., :k])
    if fmt == moe.MOE_Q4_INT4:
        # max|w| / 7 in fp32, rounded to bf16
        assert torch.equal(scales[~bad], (amax.to(F32) / 7.0).to(BF)[~bad])
        s = scales.to(F64)
    else:
        s = torch.where(bad, float("nan"), 2.0 ** (scales.to(F64) - 127))
        small = scales == 1
        assert (amax <= 6 * s)[~bad].all() and (amax > 3 * s)[~bad & ~small].all()
    # every value is at the nearest code: half a step of the grid around it off, and the division's rounding
    diff = (values - W.to(F64)).abs()
    se = s.repeat_interleave(group, -1)[..., :k]
    y = W.to(F64).abs() / torch.where(se == 0, 1.0, se)
    grid = 0.5 if fmt == moe.MOE_Q4_INT4 else torch.where(y < 2, 0.25, torch.where(y < 4, 0.5, 1.0))
    fine = ~torch.isnan(values)
    over = torch.where(se == 0, W.to(F64).abs(), se * (grid + 7 * 2.0 ** -8 * (fmt == moe.MOE_Q4_INT4) * (y > 7) + 2.0 ** -20))
    assert (diff <= over)[fine].all()
    if fmt == moe.MOE_Q4_E2M1:   # ties take the even code
        assert values[1, 0, :8].tolist() == [6.0, 0.0, 1.0, 1.0, 2.0, 2.0, 4.0, 4.0]
    for t in (F32, BF):
        out = torch.empty(N, n, k, dtype=t, device="cuda")
        moe.check(moe.moe_q4_dequantize(d, codes, scales, out, moe.dtype_code(t)))
        close(out, values, torch.zeros_like(torch.nan_to_num(values)))


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", [moe.MOE_Q4_INT4, moe.MOE_Q4_E2M1])
def test_q4_places_past_32_bits(fmt):
    """The last expert of a tensor whose codes (and weights) pass 2^32: as if it stood alone."""
    N, n, k = 66, 16384, 8192
    W = torch.zeros(N, n, k, dtype=BF, device="cuda")
    W[-1] = randn(gen(51), n, k, std=0.05)
    codes = torch.full((N, n, k // 2), 0x5A, dtype=torch.uint8, device="cuda")
    scales = torch.zeros(N, n, k // 32, dtype=BF if fmt == moe.MOE_Q4_INT4 else torch.uint8, device="cuda")
    alone = [torch.empty_like(t[:1]) for t in (codes, scales, W)]
    big, one = moe.make_q4(N, n, k, 32, fmt), moe.make_q4(1, n, k, 32, fmt)
    moe.check(moe.moe_q4_quantize(big, W, moe.MOE_BF16, codes, scales))
    moe.check(moe.moe_q4_quantize(one, W[-1:].contiguous(), moe.MOE_BF16, alone[0], alone[1]))
    assert torch.equal(codes[-1:], alone[0]) and torch.equal(scales[-1:], alone[1])
    W.fill_(1.0)
    moe.check(moe.moe_q4_dequantize(big, codes, scales, W, moe.MOE_BF16))
    moe.check(moe.moe_q4_dequantize(one, alone[0], alone[1], alone[2], moe.MOE_BF16))
    assert torch.equal(W[-1:], alone[2]) and int((W[:-1] != 0).sum()) == 0
    x = randn(gen(52), 1, k)
    y, y1 = torch.empty(1, n, device="cuda"), torch.empty(1, n, device="cuda")
    for d, c, s, e, out in ((big, codes, scales, N - 1, y), (one, alone[0], alone[1], 0, y1)):
        ex = torch.tensor([e], dtype=torch.int32, device="cuda")
        moe.check(moe.moe_q4_matvec(d, x, 1, 1, ex, c, s, None, out, moe.MOE_F32))
    assert status_clear() == 0
    assert torch.equal(y, y1)
    w = q4_values(alone[0][0, -64:], alone[1][0, -64:], k, 32, fmt)
    close(y[0, -64:], w @ x[0].to(F64), (k + 8) * 2.0 ** -23 * (w.abs() @ x[0].to(F64).abs()))


def test_q4_refusals():
    ok = dict(experts=4, n=32, k=64, group=32)

    def rc(c=None, x=256, pairs=4, x_div=1, e=256, codes=256, s=256, gate=256, y=256, yd=0, **kw):
        return moe.moe_q4_matvec(c or moe.make_q4(**{**ok, **kw}), x, pairs, x_div, e, codes, s, gate, y, yd, 0)

    for kw in (dict(experts=0), dict(experts=1025), dict(n=0), dict(n=12), dict(n=24, act=moe.MOE_ACT_SWIGLU),
               dict(k=0), dict(k=48), dict(group=16), dict(group=256), dict(format=2),
               dict(format=moe.MOE_Q4_E2M1, group=64), dict(act=3)):
        assert rc(**kw) in BAD, kw
        c = moe.make_q4(**{**ok, **kw})
        assert moe.moe_q4_quantize(c, 256, 0, 256, 256, 0) in BAD
        assert moe.moe_q4_dequantize(c, 256, 256, 256, 0, 0) in BAD
    for kw in (dict(x=None), dict(e=None), dict(codes=None), dict(s=None), dict(y=None), dict(pairs=-1),
               dict(pairs=4097), dict(x_div=0), dict(yd=3), dict(x=264), dict(codes=260), dict(s=258), dict(y=264),
               dict(e=257), dict(gate=258)):
        assert rc(**kw) in BAD, kw
    assert rc(pairs=0, x=None, e=None, codes=None, s=None, y=None) == moe.MOE_OK
    for kw in (dict(W=None), dict(codes=None), dict(scales=None), dict(w_dtype=7), dict(W=264)):
        a = {**dict(W=256, w_dtype=0, codes=256, scales=256), **kw}
        assert moe.moe_q4_quantize(moe.make_q4(**ok), a["W"], a["w_dtype"], a["codes"], a["scales"], 0) in BAD
        assert moe.moe_q4_dequantize(moe.make_q4(**ok), a["codes"], a["scales"], a["W"], a["w_dtype"], 0) in BAD
    assert moe.load_library().moe_q4_matvec(None, 256, 4, 1, 256, 256, 256, 256, 256, 0, None) in BAD


def test_layer_rejects_the_operators_activation():
    """MOE_ACT_NONE is no expert FFN kind."""
    assert moe.moe_workspace_size(moe.make_config(64, 64, 4, 2, moe.MOE_ACT_NONE, moe.MOE_BF16), 16) == 0


# ===================================================================== used together
def relative(got, ref):
    return float((got.to(F64) - ref.to(F64)).norm() / ref.to(F64).norm().clamp(min=1e-300))


@pytest.mark.gpu
@pytest.mark.parametrize("act", ["swiglu", "gelu"])
def test_training_step_of_the_experts(act):
    """Route, group the rows by expert, the expert FFN with 8-bit checkpoints of its pre-activations and
    inputs, and its whole backward pass, against 64-bit autograd on the same checkpoint values.

    A chain of at most four bf16 roundings (each at most 2^-8 of an element) sets the bound 2^-6 on the
    relative 2-norm."""
    T, D, H, N, K = 300, 256, 328, 8, 2
    halves = 2 if act == "swiglu" else 1
    g = gen(1)
    x, W_g = randn(g, T, D), randn(g, D, N, std=0.1)
    W1, W2 = randn(g, N, halves * H, D, std=0.06), randn(g, N, D, H, std=0.05)
    cfg = moe.make_config(D, H, N, K, ACTS[act], moe.MOE_BF16)
    Wt = moe.make_weights(W_g, W1, W2)
    M = T * K
    # every expert as a rank of its own: the rows come grouped by expert, in token order
    xs = torch.empty(M, D, dtype=BF, device="cuda")
    e, w = torch.empty(M, dtype=torch.int32, device="cuda"), torch.empty(M, device="cuda")
    counts, pos = torch.empty(N, dtype=torch.int32, device="cuda"), torch.empty(M, dtype=torch.int32, device="cuda")
    ws = torch.empty(moe.moe_ep_workspace_size(cfg, N, T), dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_ep_dispatch(cfg, N, x, T, Wt, xs, e, w, counts, pos, None, ws, ws.numel()))
    off = torch.cat([counts.new_zeros(1), counts.cumsum(0).to(torch.int32)])
    # forward
    up = moe.make_gmm(moe.MOE_GMM_NT, N, halves * H, D)
    u = torch.empty(M, halves * H, dtype=BF, device="cuda")
    moe.check(moe.moe_grouped_mm(up, xs, W1, u, off, M))
    ck = moe.make_ckpt(H, ACTS[act], moe.MOE_BF16, moe.MOE_CKPT_INT8, 64)
    h, q, s = run_forward(ck, u, M, H, moe.MOE_CKPT_INT8, 64, halves)
    cx = moe.make_ckpt(D, moe.MOE_ACT_NONE, moe.MOE_BF16, moe.MOE_CKPT_INT8, 64)
    qx = torch.empty(M, D, dtype=torch.uint8, device="cuda")
    sx = torch.empty(M, D // 64, dtype=torch.uint8, device="cuda")
    moe.check(moe.moe_ckpt_forward(cx, xs, M, None, qx, sx))
    z = torch.empty(M, D, device="cuda")
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_NT, N, D, H, moe.MOE_BF16, moe.MOE_F32), h, W2, z, off, M))
    y = torch.empty(T, D, device="cuda")
    moe.check(moe.moe_ep_combine(cfg, z * w[:, None], T, pos, y, moe.MOE_F32))
    # the layer call computes the same
    wsl = moe.alloc_workspace(cfg, T)
    y_layer = torch.empty(T, D, device="cuda")
    moe.check(moe.moe_forward(cfg, x, T, Wt, y_layer, moe.MOE_F32, None, wsl, wsl.numel()))
    assert status_clear() == 0
    assert relative(y, y_layer) <= 2.0 ** -6
    # backward of sum(y * dy); dy of every (token, slot) row, in the rows' order
    dy = randn(g, T, D)
    token = torch.empty(M, dtype=torch.long, device="cuda")
    token[pos.long()] = torch.arange(M, device="cuda") // K
    dyr = dy[token].contiguous()
    del u, h
    dh = torch.empty(M, H, dtype=BF, device="cuda")
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_NN, N, D, H), dyr, W2, dh, off, M))
    du = torch.empty(M, halves * H, dtype=BF, device="cuda")
    hw, dw = torch.empty(M, H, dtype=BF, device="cuda"), torch.empty(M, device="cuda")
    moe.check(moe.moe_ckpt_backward(ck, q, s, M, dh, w, du, hw, dw))
    dW2, dW1 = torch.empty(N, D, H, device="cuda"), torch.empty(N, halves * H, D, device="cuda")
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_TN, N, D, H, moe.MOE_BF16, moe.MOE_F32), dyr, hw, dW2, off, M))
    xb = torch.empty_like(xs)
    moe.check(moe.moe_ckpt_load(cx, qx, sx, M, xb))
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_TN, N, halves * H, D, moe.MOE_BF16, moe.MOE_F32), du, xb,
                                 dW1, off, M))
    dxs = torch.empty(M, D, device="cuda")
    moe.check(moe.moe_grouped_mm(moe.make_gmm(moe.MOE_GMM_NN, N, halves * H, D, moe.MOE_BF16, moe.MOE_F32), du, W1,
                                 dxs, off, M))
    assert status_clear() == 0
    # 64-bit autograd around the same checkpoint values
    uv = torch.empty(M, halves * H, device="cuda")
    moe.check(moe.moe_ckpt_load(moe.make_ckpt(H, ACTS[act], moe.MOE_F32, moe.MOE_CKPT_INT8, 64), q, s, M, uv))
    o = off.tolist()
    for ex in range(N):
        sl = slice(o[ex], o[ex + 1])
        if o[ex] == o[ex + 1]:
            assert int(dW1[ex].abs().sum()) == 0 and int(dW2[ex].abs().sum()) == 0
            continue
        xv, w1 = xb[sl].to(F64).requires_grad_(), W1[ex].to(F64).requires_grad_()
        w2, wr = W2[ex].to(F64).requires_grad_(), w[sl].to(F64).requires_grad_()
        pre = xv @ w1.t()
        pre = pre + (uv[sl].to(F64) - pre).detach()   # the checkpoint's value, the linear's gradient
        hv = pre * torch.special.ndtr(pre) if act == "gelu" else silu_ref(pre[:, :H]) * pre[:, H:]
        loss = (wr[:, None] * (hv @ w2.t()) * dyr[sl].to(F64)).sum()
        gx, g1, g2, gw = torch.autograd.grad(loss, (xv, w1, w2, wr))
        for got, ref in ((dxs[sl], gx), (dW1[ex], g1), (dW2[ex], g2), (dw[sl], gw)):
            assert relative(got, ref) <= 2.0 ** -6


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,group", FMT_GROUPS)
def test_decode_step_with_4_bit_experts(fmt, group):
    """Route, up projection with SwiGLU, down projection with the gate weights, combine: against the layer
    call on the same weights in bf16.

    Both round h to bf16 and the layer's weights were rounded to bf16 as well (int4): three roundings
    of at most 2^-8 each on either side, below 2^-6 of the relative 2-norm."""
    T, D, H, N, K = 5, 288, 352, 8, 4
    g = gen(2)
    x, W_g = randn(g, T, D), randn(g, D, N, std=0.1)
    up, down = moe.make_q4(N, 2 * H, D, group, fmt, moe.MOE_ACT_SWIGLU), moe.make_q4(N, D, H, group, fmt)
    packed = []
    for d, shape in ((up, (N, 2 * H, D)), (down, (N, D, H))):
        W = randn(g, *shape, std=0.06)
        codes = torch.empty(*shape[:2], shape[2] // 2, dtype=torch.uint8, device="cuda")
        scales = torch.empty(*shape[:2], -(-shape[2] // group), device="cuda",
                             dtype=BF if fmt == moe.MOE_Q4_INT4 else torch.uint8)
        moe.check(moe.moe_q4_quantize(d, W, moe.MOE_BF16, codes, scales))
        plain = torch.empty(*shape, dtype=BF, device="cuda")
        moe.check(moe.moe_q4_dequantize(d, codes, scales, plain, moe.MOE_BF16))
        packed.append((codes, scales, plain))
    cfg = moe.make_config(D, H, N, K, moe.MOE_ACT_SWIGLU, moe.MOE_BF16)
    W = moe.make_weights(W_g, packed[0][2], packed[1][2])
    ws = moe.alloc_workspace(cfg, T)
    idx = torch.empty(T, K, dtype=torch.int32, device="cuda")
    tw = torch.empty(T, K, device="cuda")
    moe.check(moe.moe_route(cfg, x, T, W, None, idx, tw, None, ws, ws.numel()))
    h = torch.empty(T * K, H, dtype=BF, device="cuda")
    moe.check(moe.moe_q4_matvec(up, x, T * K, K, idx, packed[0][0], packed[0][1], None, h, moe.MOE_BF16))
    z = torch.empty(T * K, D, device="cuda")
    moe.check(moe.moe_q4_matvec(down, h, T * K, 1, idx, packed[1][0], packed[1][1], tw, z, moe.MOE_F32))
    pos = torch.arange(T * K, dtype=torch.int32, device="cuda")
    y, y_layer = torch.empty(T, D, device="cuda"), torch.empty(T, D, device="cuda")
    moe.check(moe.moe_ep_combine(cfg, z, T, pos, y, moe.MOE_F32))
    moe.check(moe.moe_forward(cfg, x, T, W, y_layer, moe.MOE_F32, None, ws, ws.numel()))
    assert status_clear() == 0
    assert relative(y, y_layer) <= 2.0 ** -6
