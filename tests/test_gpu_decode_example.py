"""The decode-step example: the operators run together as a serving loop, and agree with
themselves between the prompt's form and the single-token form."""
import os
import sys

import pytest
import torch

from qmm_testlib import require_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
pytestmark = pytest.mark.gpu


def _model(dtype=torch.bfloat16, **kw):
    from decode_step import Config, Decoder
    return Decoder(Config(dtype=dtype, **kw), device=require_gpu())


def test_generation_repeats_and_returns_its_pages():
    m = _model()
    dev = m.device
    prompt = torch.randint(0, m.cfg.vocab, (3, 21), generator=torch.Generator().manual_seed(1), dtype=torch.int32).to(dev)
    u = torch.rand(6, 3, generator=torch.Generator().manual_seed(2)).to(dev)
    kw = dict(temperature=0.9, top_k=40, top_p=0.9)
    first = m.generate(prompt, 6, u, **kw)
    again = m.generate(prompt, 6, u, **kw)
    torch.cuda.synchronize()
    assert first.shape == (3, 6) and ((first >= 0) & (first < m.cfg.vocab)).all()
    assert torch.equal(first, again) and sorted(m.free) == list(range(m.cfg.pages))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_prompt_at_once_and_token_by_token_agree(dtype):
    """The last logits of a prompt fed at once (the matrix kernels, the prompt attention) and
    token by token (the decode kernels, single-token attention).  Both feed the same values
    through one layer; what differs is the order of sums, so a rounding to the type may go the
    other way by one unit (2^-7 or 2^-10 of the value, at worst) at each of the eight roundings
    on the way to the logits, and a key or value code by one step of a fifteenth of its group's
    range, for few of them.  Eight whole units bound the norm of the difference."""
    m = _model(dtype, layers=1)
    dev, n = m.device, 40
    tokens = torch.randint(0, m.cfg.vocab, (2, n), generator=torch.Generator().manual_seed(3), dtype=torch.int32).to(dev)
    blocks = -(-n // m.cfg.page)
    table = torch.arange(2 * blocks, dtype=torch.int32).view(2, blocks).to(dev)
    slot = (table[:, :, None] * m.cfg.page + torch.arange(m.cfg.page, dtype=torch.int32, device=dev)).flatten(1)
    full = torch.full((2,), n, dtype=torch.int32, device=dev)
    whole = m.logits(tokens, slot[:, :n].contiguous(), table, full, n)
    for i in range(n):
        step = m.logits(tokens[:, i:i + 1].contiguous(), slot[:, i:i + 1].contiguous(), table, full - (n - 1 - i), i + 1)
    torch.cuda.synchronize()
    a, b = whole.float(), step.float()
    assert torch.isfinite(a).all() and torch.isfinite(b).all()
    assert ((a - b).norm() / a.norm()).item() < 8 * (2 ** -7 if dtype == torch.bfloat16 else 2 ** -10)


def test_step_replays_from_a_graph():
    """One step (both layers, then sampling) captured once: lengths, slots and
    tokens are read from the device, so replays go on as the sequence grows."""
    m = _model()
    dev, batch, n, steps = m.device, 2, 9, 5
    cfg = m.cfg
    blocks = -(-(n + steps) // cfg.page)
    table = torch.arange(batch * blocks, dtype=torch.int32).view(batch, blocks).to(dev)
    slot = (table[:, :, None] * cfg.page + torch.arange(cfg.page, dtype=torch.int32, device=dev)).flatten(1)
    prompt = torch.randint(0, cfg.vocab, (batch, n), generator=torch.Generator().manual_seed(5), dtype=torch.int32).to(dev)
    u = torch.rand(steps, batch, generator=torch.Generator().manual_seed(6)).to(dev)
    longest = n + steps                                          # a bound that holds for every step
    lengths = torch.full((batch,), n, dtype=torch.int32, device=dev)
    tokens, place, draw = prompt[:, -1:].contiguous(), slot[:, :1].contiguous(), u[0].clone()

    def step():
        return q_sample(m.logits(tokens, place, table, lengths, longest), draw, top_k=20)[0]

    from bit_affine_quantized_qmv_amd import sample as q_sample

    def feed(i, token):
        tokens.copy_(token[:, None]), place.copy_(slot[:, n + i:n + i + 1]), draw.copy_(u[i]), lengths.fill_(n + i + 1)

    def run(call):
        m.logits(prompt, slot[:, :n].contiguous(), table, torch.full_like(lengths, n), longest)
        token, out = prompt[:, -1], []
        for i in range(steps):
            feed(i, token)
            token = call().clone()
            torch.cuda.synchronize()
            out.append(token)
        return torch.stack(out, 1)

    eager = run(step)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        held = step()

    def replay():
        graph.replay()
        return held

    for _ in range(3):
        assert torch.equal(run(replay), eager)
