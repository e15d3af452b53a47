"""GPU product of e4m3 operands: every kernel that sizes reach, among them those
whose sums of parts of k meet in a workspace, on streams and in graphs.  Whole
codes and steps that are powers of two: every kernel's sums are exact."""
import sys

import pytest
import torch

from gpu_util import canaries_intact, guarded

pytestmark = pytest.mark.gpu
E4 = torch.float8_e4m3fn

# with the sizes of the other file they reach every kernel, which a CPU test checks
PATHS = [(801, 4096, 13696), (617, 7168, 11008), (298, 1024, 9984), (54, 7168, 10496)]
# parts of k in both types: a second launch and a workspace
JOINED = [(300, 4096, 11008), (801, 4096, 13696), (298, 1024, 9984)]


def note(msg):
    print("[case] " + msg, flush=True)
    sys.stdout.flush()


@pytest.fixture(scope="module")
def qg():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    import quantized_gemv_amd as q
    q.lib()
    return q


def operands(qg, m, n, k, seed):
    """(W, x, s_x, y in fp64): terms of up to 16, times steps of 1/4 .. 4, so sums stay below 2^24
    in units of 1/4."""
    assert 64 * 4 * k < 2 ** 24 * 4
    torch.manual_seed(seed)
    x = torch.randint(-4, 5, (m, k), device="cuda").float().to(E4)
    w = torch.randint(-4, 5, (n, k), device="cuda").float().to(E4)
    s_x = 2.0 ** torch.randint(-1, 2, (k // 128, m), device="cuda").float()
    s_w = 2.0 ** torch.randint(-1, 2, (-(-n // 128), k // 128), device="cuda").float()
    xs = x.double().view(m, k // 128, 128) * s_x.t().double()[:, :, None]
    ws = w.double().view(n, k // 128, 128) * s_w.double().repeat_interleave(128, 0)[:n, :, None]
    return qg.QWeight(qg.QG_WFMT_FP8, n, k, w, s_w), x, s_x, torch.matmul(xs.view(m, k), ws.view(n, k).t().contiguous())


@pytest.mark.parametrize("m,n,k", PATHS)
def test_every_kernel_exact(qg, m, n, k):
    W, x, s_x, ref = operands(qg, m, n, k, m + n + k)
    for tiled in (False, True):
        L = qg.tiled16(W) if tiled else W
        for dtype in (torch.float32, torch.bfloat16):
            note("paths m=%d n=%d k=%d tiled=%s %s" % (m, n, k, tiled, dtype))
            full, y = guarded(m * n, dtype)
            need = qg.lib().qg_qgemm_fp8_workspace_bytes(m, n, k, 0 if dtype == torch.float32 else 1)
            wfull, ws = guarded(need, torch.uint8)
            qg.qgemm_fp8(L, x, s_x, y=y.view(m, n), ws=ws)
            assert torch.equal(y.view(m, n), ref.float().to(dtype))
            assert canaries_intact(full, m * n) and canaries_intact(wfull, need)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_joined_products_on_streams_and_in_a_graph(qg, dtype):
    """Each launch with a workspace of its own: at once on streams, and captured,
    replayed among eager work on the same memory."""
    note("joined products %s" % dtype)
    launches, want = [], []
    for i, (m, n, k) in enumerate(JOINED):
        W, x, s_x, ref = operands(qg, m, n, k, i)
        assert qg.lib().qg_qgemm_fp8_workspace_bytes(m, n, k, 0 if dtype == torch.float32 else 1) > 0
        launches.append(qg.QgemmFp8Launch(qg.tiled16(W) if i == 1 else W, x, s_x, y_dtype=dtype))
        want.append(ref.float().to(dtype))
    streams = [torch.cuda.Stream() for _ in launches]
    torch.cuda.synchronize()
    for _ in range(3):
        for a in launches:
            a.y.fill_(float("nan"))
        torch.cuda.synchronize()
        for a, st in zip(launches, streams):
            with torch.cuda.stream(st):
                a.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a.y, w) for a, w in zip(launches, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for a in launches:
            a.launch()
    for _ in range(3):
        for a in launches:
            a.y.fill_(float("nan"))
            a._ws.fill_(255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a.y, w) for a, w in zip(launches, want))
        for a in launches:
            a.launch()
        torch.cuda.synchronize()
        assert all(torch.equal(a.y, w) for a, w in zip(launches, want))


def test_functions_captured_with_their_workspaces(qg):
    """qgemm_fp8 makes its output and workspace inside the capture: two graphs
    of the same size, replayed at once on two streams."""
    note("captured functions")
    m, n, k = JOINED[0]
    made = [operands(qg, m, n, k, 7 + i) for i in range(2)]
    graphs, ys = [torch.cuda.CUDAGraph() for _ in made], []
    for graph, (W, x, s_x, _) in zip(graphs, made):
        with torch.cuda.graph(graph):
            ys.append(qg.qgemm_fp8(W, x, s_x))
    streams = [torch.cuda.Stream() for _ in made]
    for _ in range(3):
        for y in ys:
            y.fill_(float("nan"))
        torch.cuda.synchronize()
        for graph, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, ref.float().bfloat16()) for y, (_, _, _, ref) in zip(ys, made))
