"""GPU: masks of several layers over several steps from one captured graph."""

import pytest
import torch

from bit_quantized_finetuning_nf4_amd import ops
from oracle import dropout as OD
from tests.helpers import torch_to_f64

pytestmark = pytest.mark.gpu

N, LAYERS, STEPS = 4096, 3, 4


def masks(offsets):
    """(layer, step) -> the mask that a replay of the captured layers drew."""
    x = torch.ones(N, dtype=torch.bfloat16, device="cuda")
    step = torch.zeros(1, dtype=torch.int64, device="cuda")
    drops = [ops.Dropout(0.5, 9, o, step) for o in offsets]
    outs = [torch.empty_like(x) for _ in offsets]
    run = lambda: [ops.dropout(x, d, out=o) for d, o in zip(drops, outs)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=stream):
        run()
    got = {}
    for t in range(STEPS):
        step.fill_(t)
        g.replay()
        torch.cuda.synchronize()
        for l, o in enumerate(outs):
            got[l, t] = torch_to_f64(o) != 0
            assert (got[l, t] == OD.keep_mask(N, 0.5, 9, offsets[l] + t)).all()
    return got


def test_layers_spaced_by_2_32_share_no_mask():
    got = list(masks([l << 32 for l in range(LAYERS)]).values())
    for i, a in enumerate(got):
        for b in got[:i]:
            assert 0.4 < (a == b).mean() < 0.6   # independent: half agree, N = 4096 within 13 standard deviations


def test_offsets_next_to_each_other_are_the_next_steps():
    """What the documentation warns of."""
    got = masks(list(range(LAYERS)))
    for l in range(1, LAYERS):
        for t in range(STEPS - 1):
            assert (got[l, t] == got[l - 1, t + 1]).all()
