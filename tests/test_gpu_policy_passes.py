"""The policy step's head in passes over the rows, at vocabularies whose rows take more than a warp: the same bytes
as in one pass, and the oracle's loss and gradients."""
import numpy as np
import pytest

import layer_streamed_qlora_streaming_b200 as lst
import synthetic as syn
from oracle import model as M
from helpers import GRAD_COS, GRAD_MAXREL, LOSS_RTOL, build_inputs, compare_grads, make_context
from test_gpu_policy_step import _bytes, _rollout, _run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _step(wl, inp, roll, **cfg):
    ctx = make_context(wl, inp, streamed=True, **cfg)
    out, grads = _run(ctx, wl, *roll, kl_beta=0.1, norm=lst.POLICY_TOKEN_MEAN)
    logp = np.zeros(wl.tokens, dtype=np.float32)
    ctx.logp(logp)
    return ctx, out, grads, logp


@pytest.mark.parametrize("V", [1000, 5000, 20000, 32000])
def test_policy_passes_give_the_same_bytes(V):
    # 640 rows in one pass, in passes of 96 with a short last one, and in passes of a few rows
    wl = syn.WORKLOADS["tiny"].with_(n_layers=1, vocab=V, batch=8, seq=80)
    inp = build_inputs(wl)
    roll = _rollout(wl)
    runs = []
    for chunk in (0, 96, 24):
        ctx, out, grads, logp = _step(wl, inp, roll, head_chunk=chunk)
        runs.append((*_bytes(out, grads), logp.tobytes()))
        ctx.close()
    assert runs[0] == runs[1] == runs[2]


def test_policy_passes_match_oracle():
    wl = syn.WORKLOADS["tiny"].with_(n_layers=1, vocab=5000, batch=4, seq=80)
    inp = build_inputs(wl)
    roll = _rollout(wl)
    ctx, out, grads, logp = _step(wl, inp, roll, head_chunk=96)
    toks, tgts, mask, adv, old = roll
    ref = M.policy_step(wl, inp["raw"], inp["head"], toks, tgts, adv, old=old.astype(np.float64), mask=mask, norm="token",
                        beta=0.1, bf16_acts=True)
    size = np.abs(ref["out"]).max()
    assert abs(out["loss"] - ref["out"][0]) <= LOSS_RTOL * size and abs(out["ratio"] - ref["out"][3]) <= LOSS_RTOL * size
    assert np.max(np.abs(logp - ref["logp"])) <= LOSS_RTOL * np.abs(ref["logp"]).max()
    for l, p, w, cs, mr in compare_grads(ctx, grads, ref["grads"]):
        assert cs >= GRAD_COS and mr <= GRAD_MAXREL, (l, p, w, cs, mr)
    ctx.close()
