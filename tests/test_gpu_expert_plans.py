"""A captured decode of named experts, replayed after others were named."""
import pytest
import torch

import synth
import lossless_entropy_coded_ecf8_amd as E

pytestmark = pytest.mark.gpu
D = torch.device("cuda", 0)


def test_a_captured_decode_of_named_experts_outlives_the_naming_of_others():
    n, inner, K = 6, 64, 96
    stacks = [[torch.from_numpy(synth.small_stable(r * c, 1.8, 100 * m + e)).view(r, c) for e in range(n)]
              for m, (r, c) in enumerate(((inner, K), (inner, K), (K, inner)))]
    layer = E.ECF8Experts(*stacks, torch.ones(3, n), device=D)
    layer.decode([0, 3])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer.decode([3, 0])
    for other in ([1], [2, 4], [0, 5]):
        layer.decode(other)
        filler = [torch.full((1 << 16,), 255, dtype=torch.uint8, device=D) for _ in range(8)]     # what a freed plan's memory would be
        torch.cuda.synchronize()
        layer._pool.zero_()
        graph.replay()
        torch.cuda.synchronize()
        for w, stack in zip(out, stacks):
            assert all(torch.equal(w[e].cpu(), stack[e]) for e in (0, 3)) and not any(bool(w[e].any()) for e in (1, 2, 4, 5))
        del filler
