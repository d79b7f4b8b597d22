"""The backward of calls without queries, whose kernel follows a fill and no kernel: eagerly,
captured and replayed, batch and packed."""
import pytest

from test_gpu_attention import BF, HF, inputs, pkg  # noqa: F401

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")


@pytest.mark.parametrize("dtype", [BF, HF], ids=str)
@pytest.mark.parametrize("packed", [False, True])
def test_in_a_graph(pkg, packed, dtype):  # noqa: F811
    q, k, v = inputs(1, None if packed else 3, 0, 5000, 8, 4, 64, dtype)
    kw = {}
    if packed:
        kw = {"offsets": torch.zeros(4, dtype=torch.int32, device="cuda"),
              "kv_offsets": torch.tensor([0, 1000, 1001, 4990], dtype=torch.int32, device="cuda")}
    out, lse = pkg.attention_fwd(q, k, v, want_stats=True, **kw)

    def step():
        return pkg.attention_bwd(out, q, k, v, out, lse, **kw)[1:]

    assert all((t == 0).all() for t in step())
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        held = step()
    for _ in range(5):
        for t in held:
            t.fill_(float("nan"))
        graph.replay()
        assert all((t == 0).all() for t in held)
