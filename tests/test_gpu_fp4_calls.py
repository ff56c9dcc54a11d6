"""The 4-bit calls as a program makes them: in place, captured and replayed with
new contents, two replayed graphs at once, rows far apart."""
import pytest
import torch

import post_quantization_kronq_b200 as kq

pytestmark = pytest.mark.gpu
DEV = "cuda"
MX, NV = kq.MXFP4, kq.NVFP4


def quantized(x, fmt, deq=None):
    c = torch.empty(x.shape[0], kq.kronq_fp4_code_row_bytes(x.shape[1]), dtype=torch.uint8, device=DEV)
    s = torch.empty(x.shape[0], kq.kronq_fp4_scale_row_bytes(fmt, x.shape[1]), dtype=torch.uint8, device=DEV)
    g = torch.empty(1, device=DEV) if fmt == NV else None
    kq.kronq_fp4_quantize(x, fmt, c, s, gscale=g, deq=deq)
    return c, s, g


def same(p, q):
    return all(a is None or torch.equal(a, b) for a, b in zip(p, q))


@pytest.mark.parametrize("fmt", [MX, NV])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("rows,n,ld,first", [(700, 413, 420, 3), (33, 4099, 4099, 0), (1000, 64, 67, 1), (5, 1, 3, 1)])
def test_quantize_in_place_of_unaligned_rows(fmt, dt, rows, n, ld, first):
    base = torch.randn(rows, ld, device=DEV).to(dt)
    x, after = base[:, first:first + n], base.clone()
    want = torch.empty(rows, n, dtype=dt, device=DEV)
    alone = quantized(x.contiguous(), fmt, want)
    after[:, first:first + n] = want
    assert same(quantized(x, fmt, x), alone) and torch.equal(base, after)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_captured_groups_follow_their_offsets(fmt):
    E, T, m, n = 6, 300, 260, 544
    w, x = quantized(torch.randn(E * m, n, device=DEV), fmt), quantized(torch.randn(T, n, device=DEV), fmt)
    wc, ws = w[0].view(E, m, -1), w[1].view(E, m, -1)
    wg = None if fmt == MX else w[2].expand(E).contiguous()
    off = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    y, want = torch.empty(2, T, m, device=DEV)

    def call(out):
        kq.kronq_fp4_grouped_matmul(x[0], x[1], off, wc, ws, fmt, n, out, xg=x[2], wg=wg)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call(y)
    for cuts in ([0] * 7, [0, 0, 0, 300, 300, 300, 300], [0, 1, 2, 3, 4, 5, 6], [0, 50, 120, 130, 130, 299, 300]):
        off.copy_(torch.tensor(cuts, dtype=torch.int32))
        y.fill_(7.0), want.fill_(7.0)
        graph.replay()
        call(want)
        assert torch.equal(y, want)
        assert bool((y[cuts[-1]:] == 7.0).all()) and not bool((y[:cuts[-1]] == 7.0).all(1).any())


def test_two_replayed_graphs_at_once():
    T, m, n = 16, 1100, 4096
    jobs = []
    for fmt in (MX, NV):
        w, x = quantized(0.02 * torch.randn(m, n, device=DEV), fmt), torch.randn(T, n, device=DEV)
        x[3, ::100] = 1e-33                          # a token that takes the other path
        want, y = torch.empty(2, T, m, device=DEV)
        kq.kronq_fp4_matvec(x, w[0], w[1], fmt, want, wg=w[2])
        ws = kq.workspace(kq.kronq_fp4_matvec_workspace_bytes(T, m, n, fmt), DEV)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            kq.kronq_fp4_matvec(x, w[0], w[1], fmt, y, wg=w[2], ws=ws)
        jobs.append((graph, torch.cuda.Stream(), y, want, (w, x, ws)))
    for _ in range(20):
        for _, _, y, _, _ in jobs:
            y.zero_()
        torch.cuda.synchronize()
        for graph, stream, _, _, _ in jobs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, want) for _, _, y, want, _ in jobs)


@pytest.mark.parametrize("fmt", [MX, NV])
def test_rows_far_apart(fmt):
    """Rows more than 2^31 elements apart."""
    big = torch.empty(2 ** 31 + 1024, dtype=torch.bfloat16, device=DEV)
    w, x = quantized(torch.randn(300, 512, device=DEV), fmt), torch.randn(2, 512, device=DEV).to(torch.bfloat16)
    far = big.as_strided((2, 512), (2 ** 31 + 8, 1))
    far.copy_(x)
    q = quantized(x, fmt)
    assert same(quantized(far, fmt), q)
    y, z = torch.empty(2, 2, 300, dtype=torch.bfloat16, device=DEV)
    kq.kronq_fp4_matvec(x, w[0], w[1], fmt, y, wg=w[2])
    kq.kronq_fp4_matvec(far, w[0], w[1], fmt, z, wg=w[2])
    assert torch.equal(y, z)
    kq.kronq_fp4_matmul(q[0], q[1], w[0], w[1], fmt, 512, y, xg=q[2], wg=w[2])
    out = big.as_strided((2, 300), (2 ** 31 + 8, 1))
    kq.kronq_fp4_matmul(q[0], q[1], w[0], w[1], fmt, 512, out, xg=q[2], wg=w[2])
    assert torch.equal(out, y)
    kq.kronq_fp4_dequantize(q[0], q[1], fmt, far, gscale=q[2])
    kq.kronq_fp4_dequantize(q[0], q[1], fmt, x, gscale=q[2])
    assert torch.equal(far, x)
