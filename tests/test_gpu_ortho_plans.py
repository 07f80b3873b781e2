"""Orthogonalisation plans over several binds, captured executions and
workspaces on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu

capi = pytest.importorskip("sharded_shard_amd.capi")
from sharded_shard_amd.group import Orthogonalizer  # noqa: E402

DEV = "cuda"


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    yield
    torch.cuda.synchronize()


def matrices(shapes, seed, dtype=torch.bfloat16):
    g = torch.Generator().manual_seed(seed)
    return [(1e-3 * torch.randn(s, generator=g)).to(dtype).to(DEV) for s in shapes]


def empty(shapes):
    return [torch.full(s, 7.0, dtype=torch.bfloat16, device=DEV) for s in shapes]


def alone(mats):
    """Outputs of a plan of its own."""
    outs = empty([m.shape for m in mats])
    with Orthogonalizer([m.shape for m in mats]) as o:
        o.bind(mats, outs)
        o.execute()
        torch.cuda.synchronize()
    return outs


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "f32"])
def test_replays_follow_the_binding_and_its_dtype_stays(dtype):
    """A captured execution works on what is bound when it is replayed; inputs of
    another dtype are refused, and the binding stays as it was."""
    shapes = [(150, 260), (20, 30), (260, 150), (64, 2048)]
    other = torch.float32 if dtype == torch.bfloat16 else torch.bfloat16
    first, second = matrices(shapes, 1, dtype), matrices(shapes, 2, dtype)
    outs = [empty(shapes) for _ in range(2)]
    want = [alone(first), alone(second)]
    o = Orthogonalizer(shapes)
    o.bind(first, outs[0])
    o.allocate()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        o.execute(stream=side)
    for _ in range(2):
        for ins, out, right in ((first, outs[0], want[0]), (second, outs[1], want[1])):
            o.bind(ins, out)
            with pytest.raises(capi.FsdpError) as ei:
                o.bind(matrices(shapes, 3, other), empty(shapes))
            assert ei.value.status == capi.FSDP_E_STATE
            for x in out:
                x.fill_(7.0)
            graph.replay()
            torch.cuda.synchronize()
            for x, y in zip(out, right):
                assert torch.equal(x, y)
    o.execute()
    torch.cuda.synchronize()
    for x, y in zip(outs[1], want[1]):
        assert torch.equal(x, y)
    del graph
    o.close()


def test_a_workspace_is_replaced_after_the_executions_in_it():
    """Memory let go of while another stream still works in it would be handed out
    again."""
    u, = matrices([(300, 500)], 4)
    out, = empty([u.shape])
    want, = alone([u])
    side = torch.cuda.Stream()
    with Orthogonalizer([u.shape]) as o:
        o.bind([u], [out])
        o.allocate()
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            torch.cuda._sleep(200_000_000)
        o.execute(stream=side)
        assert not side.query()
        o.allocate(torch.empty(o.workspace_bytes, dtype=torch.uint8, device=DEV))
        assert side.query()
        assert torch.equal(out, want)
        out.fill_(7.0)
        o.execute()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
