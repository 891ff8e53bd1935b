"""Workspaces on another stream than the one that made them: the calls there come after the making (the
header's zeroing, and earlier work that the memory served), and the memory is not handed out again
before they are done."""
import pytest
import torch

from mla_latent_kv_17_gb300 import inputs, ops

pytestmark = pytest.mark.gpu
BUSY = 100_000_000  # cycles: some 50 ms


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from mla_latent_kv_17_gb300 import build
    build.build()
    ops.lib()


class Decode:
    def __init__(self):
        self.c = inputs.make_case(3, 128, [300, 9000, 65], seed=62).to("cuda")
        self.out, self.lse = torch.empty(3, 128, 512, device="cuda"), torch.empty(3, 128, device="cuda")

    def workspace(self):
        return ops.Workspace(3, 128)

    def plan(self, ws, stream=None):
        ops.plan(ws, self.c.seq_lens, stream=stream)

    def call(self, ws, stream=None):
        c = self.c
        ops.decode(ws, c.q_nope, c.q_rope, c.cache, c.block_table, c.seq_lens, c.scale, out=self.out, lse=self.lse, stream=stream)


class Tree:
    def __init__(self):
        c = self.c = inputs.make_case(2, 64, [700, 9000], seed=63).to("cuda")
        g = torch.Generator().manual_seed(1)
        rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        self.q = rand(2, 4, 64, 512), rand(2, 4, 64, 64)
        self.mask = torch.tensor([[1, 3, 7, 15]] * 2, dtype=torch.int64, device="cuda")
        self.out, self.lse = torch.empty(2, 4, 64, 512, device="cuda"), torch.empty(2, 4, 64, device="cuda")

    def workspace(self):
        return ops.TreeWorkspace(2, 4, 64)

    def plan(self, ws, stream=None):
        ops.plan_tree(ws, self.c.seq_lens, stream=stream)

    def call(self, ws, stream=None):
        c = self.c
        ops.decode_tree(ws, *self.q, c.cache, c.block_table, c.seq_lens, None, self.mask, c.scale, out=self.out, lse=self.lse,
                        stream=stream)


class Cross:
    def __init__(self):
        g = torch.Generator().manual_seed(2)
        rand = lambda *s: torch.randn(*s, generator=g).to(torch.bfloat16).cuda()
        self.ins = rand(205, 4, 128), rand(205, 4, 64), rand(9300, 576), rand(4, 9300, 128), rand(4, 9300, 128)
        self.cu = [torch.tensor(v, dtype=torch.int32, device="cuda") for v in ([0, 5, 205], [0, 9000, 9300])]
        self.out, self.lse = torch.empty(205, 4, 128, device="cuda"), torch.empty(205, 4, device="cuda")

    def workspace(self):
        return ops.CrossWorkspace(2, 4, 205)

    def plan(self, ws, stream=None):
        ops.plan_cross(ws, *self.cu, 9300, causal=True, stream=stream)

    def call(self, ws, stream=None):
        ops.cross_attention(ws, *self.ins, 0.07, out=self.out, lse=self.lse, stream=stream)


@pytest.fixture(params=[Decode, Tree, Cross])
def kind(request):
    """The case, and what it computes."""
    k = request.param()
    ws = k.workspace()
    k.plan(ws)
    k.call(ws)
    assert ops.status(ws) == 0
    return k, (k.out.clone(), k.lse.clone()), ws.nbytes


def same(k, want):
    ok = torch.equal(k.out, want[0]) and torch.equal(k.lse, want[1])
    k.out.fill_(7)
    k.lse.fill_(7)
    torch.cuda.synchronize()
    return ok


@pytest.mark.parametrize("given", [True, False])
def test_first_calls_on_another_stream(kind, given):
    # given: the stream is an argument; else it is the current one
    k, want, nbytes = kind
    side = torch.cuda.Stream()
    same(k, want)
    torch.cuda._sleep(BUSY)
    earlier = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    earlier.fill_(0xFF)  # still to come, in memory that the workspace may get
    del earlier
    ws = k.workspace()
    if given:
        k.plan(ws, side)
        k.call(ws, side)
    else:
        with torch.cuda.stream(side):
            k.plan(ws)
            k.call(ws)
    torch.cuda.synchronize()
    assert same(k, want)
    k.call(ws)  # the plan is still there
    torch.cuda.synchronize()
    assert same(k, want) and ops.status(ws) == 0


def test_memory_stays_until_another_stream_is_done(kind):
    k, want, nbytes = kind
    side = torch.cuda.Stream()
    same(k, want)
    ws = k.workspace()
    with torch.cuda.stream(side):
        torch.cuda._sleep(BUSY)
    k.plan(ws, side)
    k.call(ws, side)
    del ws
    later = torch.full((nbytes,), 0xFF, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    assert same(k, want) and bool((later == 0xFF).all())


def test_captured_on_another_stream(kind):
    # made eagerly, called in a graph first; and made in the graph
    k, want, _ = kind
    for inside in (False, True):
        same(k, want)
        ws = None if inside else k.workspace()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            if inside:
                ws = k.workspace()
            k.plan(ws)
            k.call(ws)
        for _ in range(2):
            graph.replay()
            torch.cuda.synchronize()
            assert same(k, want)
        assert ops.status(ws) == 0
