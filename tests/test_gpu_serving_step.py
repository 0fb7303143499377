"""The serving step of examples/serving_step.py: every step's output against
the oracle on that step's own inputs (a chain of references would differ by
the quantiser's rounding of inputs that differ in their last bit)."""
import os
import sys

import numpy as np
import pytest
import torch

import oracle
from oracle import step

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


def _np(t):
    return t.detach().cpu().numpy()


def _unpack(codes):
    c = _np(codes)
    return np.stack([(c >> (2 * s)) & 3 for s in range(4)], axis=-1).reshape(c.shape[0], -1).astype(
        np.int8) - 1


@pytest.mark.parametrize("requests,drafts", [(1, 0), (3, 2), (6, 5), (40, 3)])
def test_every_step_against_the_oracle(requests, drafts):
    import serving_step as ex
    from gemm_pq2_ternary_gb300 import binding as pq2
    hidden, inner, vocab, adapters, rank = 256, 384, 1003, 2, 8
    rows = requests * (drafts + 1)
    b = ex.Block(rows, hidden, inner, vocab, adapters, rank, requests, seed=requests)
    a = ex.random_step(b, drafts, adapters, seed=drafts)
    # drafts that have a chance: the argmax of a first pass
    b.step(**a)
    a["drafts"] = b.logits.argmax(-1).to(torch.int32)
    accepted, tokens = b.step(**a)
    torch.cuda.synchronize()
    assert pq2.pq2_last_device_error() == pq2.PQ2_OK

    x = _np(b.x)
    want = step.rmsnorm(_np(a["r"]).astype(np.float64), _np(b.w1), ex.EPS)
    assert np.all(np.abs(x - want) <= 2 ** -11 * np.abs(want) * 1.02 + 1e-6)

    def matmul(xin, w):
        qp, S, _ = oracle.quantize_act(xin)
        return oracle.matmul(qp, S, oracle.pack(_unpack(w[0])), _np(w[1]))

    # gate/up with the adapter added in place: the projection's tolerance, and
    # the adapter's (fp32 products and sums over 256 columns and 8 ranks, v to
    # 2^-22 of its largest: well below 1e-5 of the sums of magnitudes)
    base, A = matmul(x, b.gate_up)
    gu, (bv, bs, bm) = step.lora(x, _np(b.A), _np(b.B), _np(a["ids"]), None, _np(b.scales), base)
    tol = oracle.fp32_tolerance(base, A, hidden // 128) + 1e-5 * (bv + bm) + 2.0 ** -22 * bs
    assert np.all(np.abs(_np(b.gu) - gu) <= tol)

    qp, S, _ = oracle.quantize_act(oracle.swiglu(_np(b.gu)))
    y, A = oracle.matmul(qp, S, oracle.pack(_unpack(b.down[0])), _np(b.down[1]))
    assert np.all(np.abs(_np(b.y) - y) <= oracle.fp32_tolerance(y, A, inner // 128))

    r2, x2, _ = step.norm_residual(_np(b.y), _np(a["r"]), _np(b.w2), None, None, _np(b.w3), ex.EPS,
                                   ex.ALPHA, True)
    assert np.all(np.abs(_np(b.r_out) - r2) <= 1e-5 * (np.abs(r2) + 1))
    assert np.all(np.abs(_np(b.x_out) - x2) <= 2 ** -11 * np.abs(x2) * 1.02 + 2e-5)

    logits, A = matmul(_np(b.x_out), b.lm_head)
    assert np.all(np.abs(_np(b.logits) - logits) <= oracle.fp32_tolerance(logits, A, hidden // 128))

    acc, tok, margin = step.verify(_np(b.logits), _np(a["row_start"]), _np(a["drafts"]), None,
                                   _np(a["u"]), _np(a["e"]), _np(a["temperature"]))
    if margin > 1e-5:      # else fp32 may decide either way
        assert np.array_equal(_np(accepted), acc) and np.array_equal(_np(tokens), tok)
