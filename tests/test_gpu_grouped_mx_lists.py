"""The forward product's kernel that walks lists of 256 x 256 tiles and stores a tile's results under the next tile's products:
both of its forms, rounds that end with whole tiles, halves and quarters, and what it must leave alone."""
import pytest
import torch

import mxfp8_mixed_precision_amd as mx
from gpu_util import require_gpu
from test_gpu_grouped_mx import check_fwd, offsets, operand, values

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def plan(counts, M, N, K):
    """(stages with stores, an XCD's tiles past whole rounds) of the list kernel for this call, by its rule; None: another kernel."""
    ncu = torch.cuda.get_device_properties(0).multi_processor_count
    ct, met = -(-N // 256), min(len(counts), M)
    tiles = (2 * (M // 256) + met) * ct // 2
    if N % 8 or not ((K > 896 and tiles >= 4 * ncu) or (K >= 4096 and 2 * tiles >= ncu)):
        return None
    real = sum(-(-c // 256) for c in counts) * ct
    per = ncu // 8
    return 16 if K > 1920 else 8, (real // 8 + (1 if real % 8 else 0)) % per, real // 8 // per


def kernel_names(fn):
    from torch.profiler import ProfilerActivity, profile
    with profile(activities=[ProfilerActivity.CUDA]) as p:
        fn()
        torch.cuda.synchronize()
    return " ".join(e.key for e in p.key_averages())


SEVEN = [5000, 0, 3333, 1, 9000, 4097, 257]
# rows per expert, rows past the last, N, K, (stores' stages, tiles of an XCD's last round, whole rounds before it)
LISTS = [(SEVEN, 3, 3016, 2048, (16, 7, 4)), (SEVEN, 3, 3016, 1000, (8, 7, 4)), ([5000, 0, 3333, 1, 9000, 2049], 0, 3496, 2300, (16, 12, 4)),
         ([5000, 0, 3333, 1, 9000, 2049], 5, 3496, 1920, (8, 12, 4)), ([300] * 66 + [7000], 1, 2304, 2050, (16, 20, 5)),
         ([2000, 100], 0, 4096, 4096, (16, 18, 0)), ([1500, 200], 400, 4096, 4096, (16, 14, 0)), ([700, 100], 1300, 4096, 4100, (16, 8, 0)),
         ([1], 2100, 4096, 4096, (16, 2, 0)), ([0, 0], 2100, 4096, 4096, (16, 0, 0))]


@pytest.mark.parametrize("counts,tail,N,K,want", LISTS)
def test_lists_of_tiles(counts, tail, N, K, want):
    require_gpu()
    assert plan(counts, sum(counts) + tail, N, K) == want
    check_fwd(counts, N, K, False, BF, seed=N, tail=tail)


def test_the_rule_above_is_the_library_s():
    require_gpu()
    at, offs = offsets([1500, 200])
    x, w = operand(2100, 4096, 1), operand(4096, 4096, 2, lead=(2,))
    assert "grouped_mx_stream_kernel<16" in kernel_names(lambda: mx.grouped_gemm_mxfp4_fwd(x, w, offs))
    at, offs = offsets(SEVEN)
    x, w = operand(at[-1], 1000, 1), operand(3016, 1000, 2, lead=(7,))
    assert "grouped_mx_stream_kernel<8" in kernel_names(lambda: mx.grouped_gemm_mxfp4_fwd(x, w, offs))


@pytest.mark.parametrize("counts,tail,N,K,ld", [(SEVEN, 700, 3016, 2300, 3024), (SEVEN, 700, 3016, 1000, 3080), ([1500, 257], 400, 4096, 4096, 4104),
                                                ([700, 1], 1400, 4088, 4096, 4096), ([1500, 257], 400, 4096, 4096, (1 << 20) + 8)])
def test_rows_and_columns_outside_are_left(counts, tail, N, K, ld):
    """Rows past offs[E], the gaps between y's rows and what follows y keep their values; a tile's rows past its expert's end are the
    next expert's."""
    require_gpu()
    at, offs = offsets(counts)
    M = at[-1] + tail
    assert plan(counts, M, N, K) is not None
    x, w = operand(M, K, 1), operand(N, K, 2, lead=(len(counts),))
    want = mx.grouped_gemm_mxfp4_fwd(x, w, offs)[:at[-1]]
    y = torch.full((M + 256, ld), 7.0, dtype=BF, device="cuda")
    mx.mxf_grouped_gemm_mxfp4_fwd(mx.GroupedDesc(len(counts), 0, M, N, K, 0, ld), offs, *x, *w, y)
    assert torch.equal(y[:at[-1], :N], want)
    assert (y[at[-1]:] == 7).all() and (y[:, N:] == 7).all()


@pytest.mark.parametrize("bad", [[0, 1500, 1400], [0, 1500, 2101], [-256, 0, 2100], [1, 1500, 2100]])
def test_offsets_that_break_the_contract(bad):
    require_gpu()
    x, w = operand(2100, 4096, 1), operand(4096, 4096, 2, lead=(2,))
    assert plan([1500, 600], 2100, 4096, 4096) is not None
    st = torch.full((1,), -1, dtype=torch.int32, device="cuda")
    y = torch.full((2100, 4096), 7.0, dtype=BF, device="cuda")
    mx.mxf_grouped_gemm_mxfp4_fwd(mx.GroupedDesc(2, 0, 2100, 4096, 4096, 0, 4096), torch.tensor(bad, dtype=torch.int32, device="cuda"),
                                  *x, *w, y, st)
    assert int(st) == 1 and (y == 7).all()


@pytest.mark.parametrize("counts,N,K", [(SEVEN, 3016, 2300), ([1500, 200], 4096, 4096)])
def test_scales_that_are_nan_stay_in_their_rows_and_columns(counts, N, K):
    require_gpu()
    at, offs = offsets(counts)
    M = at[-1] + 400
    assert plan(counts, M, N, K) is not None
    x, w = operand(M, K, 3), operand(N, K, 4, lead=(len(counts),))
    clean = mx.grouped_gemm_mxfp4_fwd(x, w, offs)[:at[-1]]
    e = max(range(len(counts)), key=lambda i: counts[i])
    row, other = at[e] + counts[e] - 1, 3
    for r in (row, other):
        x[1][1, r, 2] = 255
    w[1][e, 2, 700, 0] = 255
    y = mx.grouped_gemm_mxfp4_fwd(x, w, offs)[:at[-1]]
    bad = torch.zeros_like(y, dtype=torch.bool)
    bad[row] = bad[other] = True
    bad[at[e]:at[e + 1], 700] = True
    assert torch.equal(y.isnan(), bad) and torch.equal(y[~bad], clean[~bad])


def test_streams_and_graphs():
    require_gpu()
    at, offs = offsets(SEVEN)
    x, w = operand(at[-1], 2300, 1), operand(3016, 2300, 2, lead=(7,))
    _, o2 = offsets([1500, 200])
    x2, w2 = operand(2100, 4096, 3), operand(4096, 4096, 4, lead=(2,))
    assert plan(SEVEN, at[-1], 3016, 2300) is not None and plan([1500, 200], 2100, 4096, 4096) is not None
    step = lambda: (mx.grouped_gemm_mxfp4_fwd(x, w, offs), mx.grouped_gemm_mxfp4_fwd(x2, w2, o2)[:1700])  # noqa: E731
    want = step()
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], []
    for _ in range(3):
        for st in streams:
            with torch.cuda.stream(st):
                got.append(step())
    torch.cuda.synchronize()
    for a in got:
        assert all(torch.equal(u, v) for u, v in zip(a, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for seed in range(3):
        x[0].copy_(operand(at[-1], 2300, 20 + seed)[0])
        x2[1].copy_(operand(2100, 4096, 30 + seed)[1])
        want = step()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(u, v) for u, v in zip(out, want))


def test_small_results_against_float64():
    """A long contraction of few tiles, whole: every element."""
    require_gpu()
    at, offs = offsets([2048])
    x, w = operand(2048, 8192, 5), operand(4096, 8192, 6, lead=(1,))
    assert plan([2048], 2048, 4096, 8192) == (16, 16, 0)
    y = mx.grouped_gemm_mxfp4_fwd(x, w, offs)
    X, W = values(*x), values(*w)[0]
    tol = 1024 * 2.0 ** -23 * (X.abs() @ W.abs().t()) + (X @ W.t()).abs() * 2.0 ** -8
    assert ((y.double() - X @ W.t()).abs() <= tol).all()
