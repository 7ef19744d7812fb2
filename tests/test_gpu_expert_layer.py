"""The layer of examples/expert_layer.py, forward, backward and decoding, against plain torch.

Bounds: every tensor between operators is rounded to bf16 once (half a step is 2^-9 of the value's
binade, 2^-8 at most relative to it), and rounding errors of independent elements add in squares:
four roundings on the way forward (rows exact; h1 and h3, the gate, y, out) leave at most sqrt(5) *
2^-8 = 0.9% in the 2-norm, twice as many on the way back at most sqrt(10) * 2^-8 = 1.3%; the
derivative of the gate can double an error of its argument.
"""
import os
import sys

import pytest
import torch

from tests.gpu_util import need_gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import expert_layer as ex  # noqa: E402

pytestmark = pytest.mark.gpu


@pytest.fixture(autouse=True)
def _gpu():
    need_gpu()


@pytest.mark.parametrize("tokens,top_k,experts,cols,hidden", [(600, 2, 8, 256, 512), (77, 3, 5, 136, 200), (1, 1, 4, 64, 64)])
def test_training_step(tokens, top_k, experts, cols, hidden):
    x, router, w1, w3, w2, d_out = ex.make(tokens, experts, cols, hidden)
    routing = ex.Routing(tokens, top_k, experts)
    out, d_x, d_w, g1, g3, g2 = ex.train_step(routing, x, router, w1, w3, w2, d_out, top_k)
    # the same layer, differentiated by torch in fp32 (routing fixed, so that d_x is the experts' part)
    ids, weights = ex.route(x, router, top_k)
    leaves = [t.float().requires_grad_() for t in (x, w1, w3, w2, weights)]
    xf, a1, a3, a2, wf = leaves
    want = torch.zeros(tokens, cols, device="cuda")
    for e in range(experts):
        t, j = (ids == e).nonzero(as_tuple=True)
        h = xf[t]
        y = (torch.nn.functional.silu(h @ a1[e]) * (h @ a3[e])) @ a2[e]
        want = want.index_add(0, t, y * wf[t, j][:, None])
    want.backward(d_out.float())
    assert ex.far(out, want.detach()) < 0.02
    for got, leaf in ((d_x, xf), (g1, a1), (g3, a3), (g2, a2), (d_w, wf)):
        assert ex.far(got, leaf.grad) < 0.03


@pytest.mark.parametrize("tokens", [1, 16, 50])
def test_decoding_step(tokens):
    x, router, w1, w3, w2, _ = ex.make(tokens, 8, 256, 384, seed=1)
    q = [ex.Q4Weights(w) for w in (w1, w3, w2)]
    got = ex.decode_step(ex.Routing(tokens, 2, 8), x, router, *q, 2)
    want = ex.plain(x, router, *[w.dense() for w in q], 2)
    assert ex.far(got, want) < 0.02
