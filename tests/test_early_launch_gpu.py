"""Calls whose kernels may be launched before their predecessor ends, where that predecessor
is not one kernel: first in a graph, behind copies and fills, behind two joined streams, on
the legacy default stream beside others, and right behind one another over the same buffers."""
import pytest
import torch

from exact_io_aware_64_b200 import binding

pytestmark = pytest.mark.gpu


class Step:
    """One of the calls with buffers of its own; ``run`` writes self.outs."""

    def __init__(self, name):
        g = torch.Generator().manual_seed(len(name))

        def rand(*shape):
            return torch.randn(*shape, generator=g).bfloat16().cuda()

        i32 = {"dtype": torch.int32, "device": "cuda"}
        if name == "mod":
            self.ins = [rand(1, 4, 600, 64), rand(1, 2, 600, 64), rand(1, 2, 600, 64), rand(1, 4, 600, 64)]
            q, k, v, do = self.ins
            ids = (torch.arange(600, device="cuda") // 170).int()[None].contiguous()
            self.ins.append(ids)
            rng = [torch.empty_like(ids), torch.empty_like(ids)]
            O, L = torch.empty_like(q), torch.empty(1, 4, 600, device="cuda")
            grads = [torch.empty_like(t) for t in (q, k, v)]
            ws = torch.empty(binding.workspace_bytes(1, 4, 600, 64), dtype=torch.uint8, device="cuda")
            self.outs = [O, L, *grads]

            def run(stream=None):
                docs = binding.doc_ranges(ids, *rng, stream=stream)
                kw = {"causal": True, "softcap": 20.0, "docs": docs, "stream": stream}
                binding.fwd_mod(q, k, v, O=O, LSE=L, **kw)
                binding.bwd_mod(q, k, v, O, do, L, dQ=grads[0], dK=grads[1], dV=grads[2],
                                workspace=ws, **kw)
        elif name == "rotary":
            self.ins = [rand(2, 4, 90, 64), rand(2, 2, 90, 64),
                        torch.arange(180, **i32).view(2, 90).contiguous()]
            q, k, pos = self.ins
            f, _ = binding.rotary_frequencies(64)
            self.outs = [torch.empty_like(q), torch.empty_like(k)]

            def run(stream=None):
                binding.rotary(q, k, f, positions=pos, Q_out=self.outs[0], K_out=self.outs[1],
                               stream=stream)
        else:
            self.ins = [rand(3, 8, 4, 128), rand(30, 2, 16, 128), rand(30, 2, 16, 128),
                        torch.randperm(30, generator=g).int().view(3, 10).cuda(),
                        torch.tensor([150, 99, 4], **i32)]
            q, k, v, table, lens = self.ins
            self.outs = [torch.empty_like(q), torch.empty(3, 8, 4, device="cuda")]
            ws = torch.empty(binding.tree_workspace_bytes(3, 8, 2, 4, 128), dtype=torch.uint8,
                             device="cuda")

            def run(stream=None):
                binding.fwd_tree(q, k, v, table, lens, O=self.outs[0], LSE=self.outs[1],
                                 workspace=ws, stream=stream)
        self.run = run
        self.good = [t.clone() for t in self.ins]
        run()
        torch.cuda.synchronize()
        binding.check_device_error()
        self.want = [t.clone() for t in self.outs]

    def spoil(self):
        """In-range values that give other results (lengths, ids and tables stay valid)."""
        for t in self.ins:
            t.zero_()
        for t in self.outs:
            t.fill_(5)

    def restore(self):
        for t, g in zip(self.ins, self.good):
            t.copy_(g)

    def check(self):
        torch.cuda.synchronize()
        binding.check_device_error()
        assert all(torch.equal(a, b) for a, b in zip(self.outs, self.want))


@pytest.fixture(params=["mod", "rotary", "tree"])
def step(request):
    return Step(request.param)


def replayed(g, step, times=5):
    for _ in range(times):
        step.spoil()
        step.restore()
        g.replay()
        step.check()


def capture(body):
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, capture_error_mode="relaxed"):
        body()
    return g


def test_first_in_a_graph(step):
    g = capture(step.run)
    replayed(g, step)
    del g


def test_behind_copies_and_fills_of_a_graph(step):
    def body():
        step.spoil()
        step.restore()
        step.run()
        step.restore()

    g = capture(body)
    for _ in range(5):
        step.spoil()
        g.replay()
        step.check()
    del g


def test_behind_two_joined_streams(step):
    """The call's predecessors are a kernel of its own stream and one of another."""
    side = torch.cuda.Stream()
    half = len(step.ins) // 2
    work = torch.randn(4 << 20, device="cuda")

    def restore(which):
        for _ in range(10):
            torch.sort(work[:1 << 16])
        for t, g in list(zip(step.ins, step.good))[which]:
            t.copy_(g)
            t.add_(0)  # a kernel, not a copy, is last

    def body():
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            restore(slice(half, None))
        restore(slice(0, half))
        here.wait_stream(side)
        step.run()

    for _ in range(10):
        step.spoil()
        body()
        step.check()
    g = capture(body)
    for _ in range(5):
        step.spoil()
        g.replay()
        step.check()
    del g


def test_right_behind_one_another(step):
    """The same call again over the same outputs and workspace, then on another stream."""
    side = torch.cuda.Stream()
    for _ in range(30):
        step.run()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(30):
        step.run(side)
    torch.cuda.current_stream().wait_stream(side)
    step.check()
    step.spoil()
    step.restore()
    step.run()
    step.check()


def test_read_and_overwritten_by_what_follows(step):
    """What follows the call may overwrite its inputs, and reads all its outputs."""
    for _ in range(20):
        step.restore()
        step.run()
        got = [t.clone() for t in step.outs]
        step.spoil()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, step.want))
