"""Two captured graphs of the block's operators, replayed in turn and at once on two
streams, with eager calls between them.  Needs a GPU."""
import pytest
import torch

from moe_grouped_gemm_block_amd import dg
from test_gpu_norm import B, DEV

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a GPU"
    dg.lib()


class Calls:
    """Every operator that has a workspace, on inputs of its own."""

    def __init__(self, seed):
        self.g = torch.Generator(device=DEV).manual_seed(seed)
        self.x = torch.empty(6000, 256, device=DEV)
        self.R, self.Y, self.d = (torch.empty(700, 1000, dtype=B, device=DEV) for _ in range(3))
        self.w = torch.ones(1000, device=DEV)
        self.grads = [torch.empty(n, device=DEV) for n in (300000, 17, 90001)]
        self.out = [torch.empty_like(t) for t in self.grads]
        self.fill()

    def fill(self):
        for t in (self.x, self.R, self.Y, self.d, *self.grads):
            t.normal_(generator=self.g)

    def run(self):
        r = dg.moe_route(self.x, 8, score="sigmoid")
        n = dg.residual_norm(self.R, self.Y, w_post=self.w, w_pre=self.w)
        b = dg.residual_norm_bwd(self.d, self.d, n.R, self.Y, w_post=self.w, w_pre=self.w)
        norm = dg.grad_norm(self.grads)
        dg.clip_grads(self.grads, norm, 1.0, out=self.out)
        return [t for t in (*r, *n, *b, norm) if t is not None] + [t.clone() for t in self.out]


def test_two_graphs():
    calls = [Calls(1), Calls(2)]
    graphs, outs = [], []
    for c in calls:
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(c.run())
        graphs.append(g)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for turn in range(4):
        for c in calls:
            c.fill()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s if turn % 2 else torch.cuda.current_stream()):
                g.replay()
        torch.cuda.synchronize()
        got = [[t.clone() for t in o] for o in outs]
        for c, o in zip(calls, got):
            for a, b in zip(o, c.run()):
                assert torch.equal(a, b)
