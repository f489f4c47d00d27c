"""spec_logprobs leaves its workspace alone: calls that overlap may share one."""
import pytest
import torch

from test_logprobs_gpu import BF, F32, built, lp, zipf  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,V,top", [(9, 256000, 5), (200, 30001, 64), (700, 20000, 0)])
def test_calls_on_two_streams_share_a_workspace(lp, R, V, top):
    g = torch.Generator().manual_seed(R)
    x = [zipf(9, V, g, d)[torch.arange(R) % 9].cuda() for d in (BF, F32)]
    t = torch.randint(0, V, (R, 3), generator=g).to(torch.int32).cuda()
    n = lp.spec_logprobs_workspace_size(R, V, 1, 3, top)
    ws = torch.full((n,), 137, dtype=torch.uint8, device="cuda")

    def outputs():
        f = lambda *s: torch.zeros(*s, device="cuda")
        return dict(logprobs=f(R, 3), entropy=f(R), normalizer=f(R, 2),
                    top_tokens=torch.zeros(R, top, dtype=torch.int32, device="cuda") if top else None,
                    top_logprobs=f(R, top) if top else None)

    def call(k, o):
        lp.spec_logprobs(x[k], t, o["logprobs"], ws, T=0.9, entropy=o["entropy"],
                         normalizer=o["normalizer"], top_tokens=o["top_tokens"],
                         top_logprobs=o["top_logprobs"])

    alone, shared = [outputs(), outputs()], [outputs(), outputs()]
    for k in range(2):
        call(k, alone[k])
        torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for k in range(2):
        with torch.cuda.graph(graphs[k], stream=streams[k]):
            for _ in range(20):
                call(k, shared[k])
    for _ in range(5):
        for k in range(2):
            with torch.cuda.stream(streams[k]):
                graphs[k].replay()
    torch.cuda.synchronize()
    for k in range(2):
        for name, v in alone[k].items():
            assert v is None or torch.equal(v, shared[k][name]), name
    assert bool((ws == 137).all())
