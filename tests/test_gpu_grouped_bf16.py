"""The bf16 expert products (grouped_gemm_bf16_fwd / _dgrad / _wgrad) against 64-bit products.

Tolerances, derived before any run: a sum of n fp32-accumulated products is off by at most
n 2^-23 S, S the sum of the products' magnitudes (each of at most n additions rounds, or
truncates, by at most 2^-23 of a partial sum no larger than S); a bf16 output adds half a unit
in its last place, at most 2^-8 of its magnitude (8 significant bits), and 2^-133 where it is subnormal.  The fp32 weight
gradient is also held to 1e-5 in the relative 2-norm: fp32 rounding, not bf16's."""
import numpy as np
import pytest
import torch

from mxfp8_block_scaled_rowwise_gb300 import binding as mx
from mxfp8_block_scaled_rowwise_gb300 import synth
from gpu_util import check_dev_err, dev, offsets  # noqa: F401

pytestmark = pytest.mark.gpu

# (rows per expert, N, K): one row, one token's experts, rows around every tile edge, empty
# experts first, last and between, widths from one 16-byte piece to several tiles and a ragged rest
CASES = [
    ([1], 8, 8),
    ([0, 1, 0], 72, 40),
    ([1, 1, 1, 0, 1, 1, 1, 1, 1], 520, 264),
    ([5, 0, 17, 64, 63, 65], 136, 1112),
    ([127, 128, 129, 0, 255, 256, 257, 2], 256, 192),
    ([300, 0, 0, 700], 264, 72),
    ([0, 0, 600], 1000, 520),
    ([33, 31, 32, 16, 15, 48, 8, 7], 392, 2056),
    ([1500], 512, 128),
    ([2, 0, 900, 1, 0, 40], 712, 1288),
]


def _make(counts, N, K, dev, seed, extra=0):
    """A [R, K], dY [R, N], W [E, N, K] in bf16; `extra` rows past the last expert's."""
    g = synth.generator(seed)
    R, E = sum(counts) + extra, len(counts)
    a = synth.randn_bf16((R, K), g)
    dy = synth.randn_bf16((R, N), g)
    w = synth.randn_bf16((E, N, K), g)
    off = torch.from_numpy(offsets(counts)[0])
    return a.to(dev), dy.to(dev), w.to(dev), off.to(dev), R, E


def _bf16_bound(ref, mag, n):
    return 2.0 ** -8 * ref.abs() + n * 2.0 ** -23 * mag + 2.0 ** -133


def _check_rows(got, x, w, counts, transposed):
    """got [R, *] against x [R, k] and w [E, ...] per expert; transposed: w[e] is [out, k]."""
    off = offsets(counts)[0]
    for e, c in enumerate(counts):
        if c == 0:
            continue
        xe = x[off[e]:off[e + 1]].double()
        we = w[e].double().t() if transposed else w[e].double()
        ref, mag = xe @ we, xe.abs() @ we.abs()
        err = (got[off[e]:off[e + 1]].double() - ref).abs()
        assert bool((err <= _bf16_bound(ref, mag, x.shape[1])).all()), "expert %d: %g" % (e, float(err.max()))


def _check_wgrad(got, dy, x, counts):
    off = offsets(counts)[0]
    for e, c in enumerate(counts):
        d, xe = dy[off[e]:off[e + 1]].double(), x[off[e]:off[e + 1]].double()
        ref, mag = d.t() @ xe, d.t().abs() @ xe.abs()
        if c == 0:
            assert not got[e].any()
            continue
        err = (got[e].double() - ref).abs()
        assert bool((err <= c * 2.0 ** -23 * mag).all()), "expert %d: %g" % (e, float((err / mag).max()))
        assert float(err.norm() / ref.norm()) <= 1e-5


def _run_all(a, dy, w, off, R, E, N, K, dev, fill=0.0):
    err = mx.new_dev_err(dev)
    C = torch.full((R, N), fill, dtype=torch.bfloat16, device=dev)
    dX = torch.full((R, K), fill, dtype=torch.bfloat16, device=dev)
    dW = torch.full((E, N, K), 7.0, dtype=torch.float32, device=dev)
    mx.grouped_gemm_bf16_fwd(a, w, off, E, R, N, K, C, err)
    mx.grouped_gemm_bf16_dgrad(dy, w, off, E, R, K, N, dX, err)
    mx.grouped_gemm_bf16_wgrad(dy, a, off, E, R, N, K, dW, err)
    check_dev_err(err)
    return C, dX, dW


@pytest.mark.parametrize("counts,N,K", CASES)
def test_products_match_64_bit(dev, counts, N, K):
    a, dy, w, off, R, E = _make(counts, N, K, dev, 11 + N + K)
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev)
    _check_rows(C, a, w, counts, True)
    _check_rows(dX, dy, w, counts, False)
    _check_wgrad(dW, dy, a, counts)


@pytest.mark.parametrize("E,skew", [(4, False), (130, True), (1024, True)])
def test_many_experts_routed(dev, E, skew):
    g = synth.generator(5 + E)
    ids = synth.zipf_ids(900, E, 2, g, n_zero=E // 8) if skew else synth.uniform_ids(900, E, 2, g)
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).tolist()
    N, K = 104, 88
    a, dy, w, off, R, E = _make(counts, N, K, dev, 21)
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev)
    _check_rows(C, a, w, counts, True)
    _check_rows(dX, dy, w, counts, False)
    _check_wgrad(dW, dy, a, counts)


@pytest.mark.parametrize("T,k,E,N,K", [(1, 8, 32, 1024, 1792), (3, 2, 8, 1160, 3000), (16, 4, 16, 640, 4096),
                                       (64, 8, 32, 384, 2048), (200, 6, 60, 776, 904)])
def test_serving_batches(dev, T, k, E, N, K):
    """Few tokens over many experts, long contractions: the calls a decoding step makes."""
    ids = synth.uniform_ids(T, E, k, synth.generator(T + E))
    counts = torch.bincount(ids.reshape(-1).long(), minlength=E).tolist()
    a, dy, w, off, R, E = _make(counts, N, K, dev, 31)
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev)
    _check_rows(C, a, w, counts, True)
    _check_rows(dX, dy, w, counts, False)
    _check_wgrad(dW, dy, a, counts)


@pytest.mark.parametrize("counts,N,K", [([60, 10, 70, 0, 133], 200, 328), ([3, 1, 2, 0, 9], 200, 328)])
def test_other_experts_and_dropped_rows_stay_out(dev, counts, N, K):
    """NaN and Inf in every other expert's rows and weights and in the rows past off[E] leave an
    expert's outputs as they are, bit for bit; rows past off[E] of the outputs are not written."""
    a, dy, w, off, R, E = _make(counts, N, K, dev, 41, extra=50)
    used = sum(counts)
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev, fill=-3.0)
    assert bool((C[used:] == -3.0).all()) and bool((dX[used:] == -3.0).all())
    o = offsets(counts)[0]
    for e, c in enumerate(counts):
        if c == 0:
            continue
        a2, dy2, w2 = a.clone(), dy.clone(), w.clone()
        for t in (a2, dy2):
            t[:o[e]] = float("nan")
            t[o[e + 1]:] = float("inf")
        w2[:e] = float("-inf")
        w2[e + 1:] = float("nan")
        C2, dX2, dW2 = _run_all(a2, dy2, w2, off, R, E, N, K, dev)
        s = slice(int(o[e]), int(o[e + 1]))
        assert torch.equal(C2[s], C[s]) and torch.equal(dX2[s], dX[s]) and torch.equal(dW2[e], dW[e])


@pytest.mark.parametrize("counts,N,K", [([1029, 271, 0, 1300, 15], 264, 392), ([512, 528, 513, 527, 16], 136, 264),
                                        ([577, 1, 31, 1041], 520, 128)])
def test_last_rows_of_long_groups(dev, counts, N, K):
    """Groups long enough for pairs of CTAs, ending 0, 1, 15 and other numbers of rows after a
    multiple of 16, right at and right after the 512 rows of a partial sum: each expert's gradient
    against 64 bits, and unchanged bit for bit by NaN and Inf in its neighbours' rows."""
    a, dy, w, off, R, E = _make(counts, N, K, dev, 47, extra=20)
    err = mx.new_dev_err(dev)
    dW, dW2 = (torch.full((E, N, K), 7.0, dtype=torch.float32, device=dev) for _ in range(2))
    mx.grouped_gemm_bf16_wgrad(dy, a, off, E, R, N, K, dW, err)
    check_dev_err(err)
    _check_wgrad(dW, dy, a, counts)
    o = offsets(counts)[0]
    for e, c in enumerate(counts):
        a2, dy2 = a.clone(), dy.clone()
        for t in (a2, dy2):
            t[:o[e]] = float("nan")
            t[o[e + 1]:] = float("inf")
        mx.grouped_gemm_bf16_wgrad(dy2, a2, off, E, R, N, K, dW2, err)
        check_dev_err(err)
        assert torch.equal(dW2[e], dW[e])


def test_gradients_are_differences_of_the_forward(dev):
    """On small integers every sum is exact, so the change of L = sum C dY under a unit step of one
    input element is that element's gradient, exactly."""
    counts, N, K = [3, 0, 130, 17], 24, 40
    g = synth.generator(51)
    R, E = sum(counts), len(counts)

    def ints(*shape):
        return torch.randint(-1, 2, shape, generator=g).to(torch.bfloat16).to(dev)
    a, dy, w = ints(R, K), ints(R, N), ints(E, N, K)
    off = torch.from_numpy(offsets(counts)[0]).to(dev)
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev)
    loss = (C.double() * dy.double()).sum()
    for r, k in [(0, 0), (2, 39), (3, 7), (70, 20), (132, 39), (149, 1)]:
        a2 = a.clone()
        a2[r, k] += 1
        d = (_run_all(a2, dy, w, off, R, E, N, K, dev)[0].double() * dy.double()).sum() - loss
        assert float(d) == float(dX[r, k])
    for e, n, k in [(0, 0, 0), (1, 3, 3), (2, 23, 39), (3, 11, 0)]:
        w2 = w.clone()
        w2[e, n, k] += 1
        d = (_run_all(a, dy, w2, off, R, E, N, K, dev)[0].double() * dy.double()).sum() - loss
        assert float(d) == float(dW[e, n, k])


@pytest.mark.parametrize("n_rows", [1, 2000])
def test_infinities_follow_the_formula(dev, n_rows):
    """Inf and NaN of an expert's own rows and weights reach exactly the outputs they feed."""
    N, K = 72, 200
    a, dy, w, off, R, E = _make([n_rows], N, K, dev, 61)
    a[0, 3] = float("inf")
    w[0, 5, 7] = float("nan")
    C, dX, dW = _run_all(a, dy, w, off, R, E, N, K, dev)
    finite = torch.isfinite(C)
    assert not finite[0].any() and not finite[:, 5].any()
    rest = torch.cat([finite[1:, :5], finite[1:, 6:]], 1)
    assert bool(rest.all())
    fx = torch.isfinite(dX)
    assert not fx[:, 7].any() and bool(torch.cat([fx[:, :7], fx[:, 8:]], 1).all())
    fw = torch.isfinite(dW[0])
    assert not fw[:, 3].any() and bool(torch.cat([fw[:, :3], fw[:, 4:]], 1).all())


def test_no_rows(dev):
    err = mx.new_dev_err(dev)
    off = torch.zeros(4, dtype=torch.int32, device=dev)
    w = torch.randn(3, 16, 24, device=dev).bfloat16()
    e = torch.empty(0, 24, dtype=torch.bfloat16, device=dev)
    e2 = torch.empty(0, 16, dtype=torch.bfloat16, device=dev)
    dW = torch.full((3, 16, 24), 5.0, device=dev)
    mx.grouped_gemm_bf16_fwd(e, w, off, 3, 0, 16, 24, e2, err)
    mx.grouped_gemm_bf16_dgrad(e2, w, off, 3, 0, 24, 16, e, err)
    mx.grouped_gemm_bf16_wgrad(e2, e, off, 3, 0, 16, 24, dW, err)
    check_dev_err(err)
    assert not dW.any()
    # rows, but none of them in an expert (every routing id was dropped)
    a, dy = torch.full((9, 24), float("nan"), dtype=torch.bfloat16, device=dev), torch.full((9, 16), float("nan"), dtype=torch.bfloat16, device=dev)
    C, dX = torch.full((9, 16), 2.0, dtype=torch.bfloat16, device=dev), torch.full((9, 24), 2.0, dtype=torch.bfloat16, device=dev)
    dW.fill_(5.0)
    mx.grouped_gemm_bf16_fwd(a, w, off, 3, 9, 16, 24, C, err)
    mx.grouped_gemm_bf16_dgrad(dy, w, off, 3, 9, 24, 16, dX, err)
    mx.grouped_gemm_bf16_wgrad(dy, a, off, 3, 9, 16, 24, dW, err)
    check_dev_err(err)
    assert not dW.any() and bool((C == 2.0).all()) and bool((dX == 2.0).all())


@pytest.mark.parametrize("bad", [[0, 5, 3, 20], [1, 5, 9, 20], [0, 5, 9, 21], [0, -1, 9, 20]])
@pytest.mark.parametrize("N,K", [(16, 24), (264, 512)])
def test_bad_offsets_are_reported_and_nothing_is_written(dev, bad, N, K):
    off = torch.tensor(bad, dtype=torch.int32, device=dev)
    a, dy = torch.ones(20, K, dtype=torch.bfloat16, device=dev), torch.ones(20, N, dtype=torch.bfloat16, device=dev)
    w = torch.ones(3, N, K, dtype=torch.bfloat16, device=dev)
    outs = [torch.full((20, N), 2.0, dtype=torch.bfloat16, device=dev), torch.full((20, K), 2.0, dtype=torch.bfloat16, device=dev),
            torch.full((3, N, K), 2.0, device=dev)]
    for call, args, out in ((mx.grouped_gemm_bf16_fwd, (a, w, off, 3, 20, N, K), outs[0]),
                            (mx.grouped_gemm_bf16_dgrad, (dy, w, off, 3, 20, K, N), outs[1]),
                            (mx.grouped_gemm_bf16_wgrad, (dy, a, off, 3, 20, N, K), outs[2])):
        err = mx.new_dev_err(dev)
        call(*args, out, err)
        torch.cuda.synchronize()
        assert int(err.item()) == mx.MX_DEVERR_BAD_SEGMENTS
        assert bool((out == 2.0).all())


def test_same_bytes_again_on_other_streams_in_a_graph_and_from_unaligned_buffers(dev):
    counts, N, K = [7, 0, 300, 64, 129], 328, 456
    a, dy, w, off, R, E = _make(counts, N, K, dev, 71)
    ref = _run_all(a, dy, w, off, R, E, N, K, dev)
    again = _run_all(a, dy, w, off, R, E, N, K, dev)
    assert all(torch.equal(x, y) for x, y in zip(ref, again))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        other = _run_all(a, dy, w, off, R, E, N, K, dev)
    assert all(torch.equal(x, y) for x, y in zip(ref, other))

    def shifted(t):   # the same values from a buffer that is 16-byte, not 32-byte aligned
        pad = 16 // t.element_size()
        b = torch.zeros(t.numel() + pad, dtype=t.dtype, device=dev)
        b[pad:] = t.reshape(-1)
        return b[pad:].view(t.shape)
    outs = [shifted(torch.zeros_like(x)) for x in ref]
    err = mx.new_dev_err(dev)
    a2, dy2, w2 = shifted(a), shifted(dy), shifted(w)

    def calls():
        mx.grouped_gemm_bf16_fwd(a2, w2, off, E, R, N, K, outs[0], err)
        mx.grouped_gemm_bf16_dgrad(dy2, w2, off, E, R, K, N, outs[1], err)
        mx.grouped_gemm_bf16_wgrad(dy2, a2, off, E, R, N, K, outs[2], err)
    calls()
    check_dev_err(err)
    assert all(torch.equal(x, y) for x, y in zip(ref, outs))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        calls()
    for o in outs:
        o.zero_()
    graph.replay()
    check_dev_err(err)
    assert all(torch.equal(x, y) for x, y in zip(ref, outs))


def test_offsets_past_32_bits(dev):
    """Rows whose element offsets pass 2^31 and byte offsets pass 2^32, in every operand."""
    K = N = 7168
    counts = [5, 299990, 0, 21]
    R, E = sum(counts), len(counts)
    off = torch.from_numpy(offsets(counts)[0]).to(dev)
    a = torch.zeros(R, K, dtype=torch.bfloat16, device=dev)
    g = synth.generator(81, dev)
    last = slice(R - 40, R)
    a[last] = synth.randn_bf16((40, K), g, device=dev)
    w = synth.randn_bf16((E, 16, K), g, device=dev)
    err = mx.new_dev_err(dev)
    C = torch.empty(R, 16, dtype=torch.bfloat16, device=dev)
    mx.grouped_gemm_bf16_fwd(a, w, off, E, R, 16, K, C, err)
    check_dev_err(err)
    assert not C[:-40].any()
    for s, e in ((slice(R - 40, R - 21), 1), (slice(R - 21, R), 3)):
        x, we = a[s].double(), w[e].double().t()
        ref, mag = x @ we, x.abs() @ we.abs()
        assert bool(((C[s].double() - ref).abs() <= _bf16_bound(ref, mag, K)).all())
    # dX rows past 2^31 elements, and the weight gradient that reads the same rows
    dy = torch.zeros(R, 16, dtype=torch.bfloat16, device=dev)
    dy[last] = synth.randn_bf16((40, 16), g, device=dev)
    a0 = a[last].clone()
    dW = torch.empty(E, 16, K, device=dev)
    mx.grouped_gemm_bf16_wgrad(dy, a, off, E, R, 16, K, dW, err)
    mx.grouped_gemm_bf16_dgrad(dy, w, off, E, R, K, 16, a, err)
    check_dev_err(err)
    d, x = dy[R - 21:].double(), a0[19:].double()
    assert bool(((dW[3].double() - d.t() @ x).abs() <= 21 * 2.0 ** -23 * (d.t().abs() @ x.abs())).all())
    assert not dW[2].any() and not dW[0].any()
    assert not a[:-40].any()
    ref, mag = d @ w[3].double(), d.abs() @ w[3].double().abs()
    assert bool(((a[R - 21:].double() - ref).abs() <= _bf16_bound(ref, mag, 16)).all())
