"""The kernels of the 8-bit output and of the backward are chosen when a handle first needs them, not when it is made: that
first time inside a capture, and in two threads at once."""
import threading

import pytest
import torch

from operator_checks import DEV, gen, randn, rank_sum

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def car():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import __graft_entry__

    __graft_entry__.build()
    import rank_sum_reduce_gb300 as car

    return car


# the row kernels (whole rows, split rows) and the pipelines, each shape and type run by no other test
SHAPES = [(2, 5, 648, "fp16"), (8, 3, 8208, "fp16"), (4, 911, 4112, "fp16"), (1, 900, 4120, "fp32")]


class Call:
    def __init__(self, car, W, M, N, dtype):
        g = gen(W + M + N)
        self.xs, self.res = [randn(g, (M, N), dtype) for _ in range(W)], randn(g, (M, N), dtype)
        self.w = (torch.rand(N, generator=g, device=DEV) + 0.5).to(self.res.dtype)
        self.make = lambda: car.Car(W, M, N, dtype)
        self.shape = (M, N)

    def outputs(self):
        M, N = self.shape
        return (torch.empty_like(self.res), torch.empty(M, N, dtype=torch.float8_e4m3fn, device=DEV),
                torch.empty(M, 1, device=DEV), torch.empty_like(self.res), torch.empty(N, device=DEV))

    def run(self, c, out, stream=None, workspace=None):
        ro, q, s, dx, dw = out
        c.reduce_residual_rmsnorm_quant(self.xs, self.res, self.w, 1e-6, "row", ro, q, s, stream=stream)
        c.reduce_residual_rmsnorm_backward(self.xs, ro, self.w, 1e-6, None, dx, dw, workspace=workspace, stream=stream)

    def same(self, a, b):
        assert torch.equal(a[0], (rank_sum(self.xs) + self.res.float()).to(self.res.dtype))
        assert all(torch.equal(x.view(torch.uint8), y.view(torch.uint8)) for x, y in zip(a, b))


@pytest.mark.parametrize("shape", SHAPES)
def test_first_use_in_a_capture(car, shape):
    k = Call(car, *shape)
    captured, eager = k.outputs(), k.outputs()
    with k.make() as c, k.make() as other:
        graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=side):
            k.run(c, captured)
        graph.replay()
        c.sync()
        k.run(other, eager)
        other.sync()
        k.same(captured, eager)
        del graph


@pytest.mark.parametrize("shape", SHAPES)
def test_first_use_in_two_threads(car, shape):
    k = Call(car, *shape)
    outs, want, failed = [k.outputs() for _ in range(2)], k.outputs(), []
    with k.make() as c, k.make() as other:
        k.run(other, want)
        ws = [torch.empty(other.backward_workspace_bytes, dtype=torch.uint8, device=DEV) for _ in range(2)]
        streams = [torch.cuda.Stream() for _ in range(2)]
        torch.cuda.synchronize()
        gate = threading.Barrier(2)

        def go(i):
            try:
                gate.wait(10)
                k.run(c, outs[i], stream=streams[i], workspace=ws[i])
            except Exception as e:  # noqa: BLE001
                failed.append(e)

        ts = [threading.Thread(target=go, args=(i,)) for i in range(2)]
        for t in ts:
            t.start()
        for t in ts:
            t.join()
        torch.cuda.synchronize()
        c.sync()
        assert not failed
        for o in outs:
            k.same(o, want)
