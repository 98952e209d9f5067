"""Windowed attention inside whole steps on the GPU: what the engine's form of it adds to the kernels' (a probability
in two bf16 parts, D from the unrounded output, the rotary embedding undone in the gradients), and every kind
of step under a window against the oracle."""
import numpy as np
import pytest

import layer_streamed_qlora_streaming_b200 as lst
import synthetic as syn
from oracle import model as M
from helpers import GRAD_COS, GRAD_MAXREL, LOSS_RTOL, build_inputs, compare_grads, make_context, run_step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, F = 2.0 ** -8, 2.0 ** -24  # half a step of bf16 and of fp32, relative to a value


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


LAYER = syn.WORKLOADS["tiny"].with_(n_layers=1, vocab=0, base_format="bf16", n_kv_heads=2)
WIDE = LAYER.with_(head_dim=128)


def _check_grads(ctx, grads, ref):
    for l, p, w, cs, mr in compare_grads(ctx, grads, ref):
        assert cs >= GRAD_COS and mr <= GRAD_MAXREL, (l, p, w, cs, mr)


def _hidden_step(wl, inp, window, sinks):
    """One step without a head against the oracle with bf16 activations."""
    ctx = make_context(wl, inp, streamed=True)
    ctx.set_attention_window(window, sinks)
    loss, grads, _ = run_step(ctx, wl, inp)
    ref = M.step(wl, raw_layers=inp["raw"], x_in=inp["x"], G=inp["G"], bf16_acts=True, window=window, sinks=sinks)
    _check_grads(ctx, grads, ref["grads"])
    ctx.close()
    # the loss is a sum of terms of either sign: held to their size
    assert abs(loss - ref["loss"]) <= LOSS_RTOL * max(abs(ref["loss"]), np.linalg.norm(inp["G"]))


@pytest.mark.parametrize("wl,window,sinks", [
    (LAYER.with_(batch=2, seq=40), 2, 0),     # two keys a row
    (WIDE.with_(batch=2, seq=150), 3, 2),     # sinks in a block of their own
    (WIDE.with_(batch=1, seq=65), 12, 0),     # a last block one key wide
    (LAYER.with_(batch=1, seq=300), 6, 70)])  # sinks that cross a block
def test_probabilities_keep_sixteen_bits(wl, window, sinks):
    # The step's own q, k, v and o. P in two bf16 parts is off by at most u (u P): o is held to its own rounding,
    # u |o|, and (u^2 + 2 e) sum P |v|, e the error of scores, exponentials and sums over at most window + sinks keys as
    # in test_gpu_window.py. Values that cancel leave |o| far below sum P |v|; one bf16 part would add u sum P |v|.
    inp = build_inputs(wl)
    ctx = make_context(wl, inp, streamed=True)
    ctx.set_attention_window(window, sinks)
    run_step(ctx, wl, inp)
    qkv = torch.empty(wl.tokens, wl.dq + 2 * wl.dkv, dtype=torch.bfloat16, device="cuda")
    got = torch.empty(wl.tokens, wl.dq, dtype=torch.bfloat16, device="cuda")
    ctx.activation("qkv", 0, qkv)
    ctx.activation("o", 0, got)
    ctx.close()
    hd, grp = wl.head_dim, wl.n_heads // wl.n_kv_heads
    heads = lambda x: x.double().reshape(wl.batch, wl.seq, -1, hd).transpose(1, 2)  # noqa: E731
    q, k, v = (heads(x) for x in qkv.split([wl.dq, wl.dkv, wl.dkv], 1))
    k, v = (x.repeat_interleave(grp, 1) for x in (k, v))
    vis = torch.from_numpy(M.visible(wl.seq, window, sinks)).cuda()
    P = torch.softmax((q @ k.transpose(-1, -2) * hd ** -0.5).masked_fill(~vis, -np.inf), -1)
    e = ((hd + 4) * F * hd ** -0.5 * (q.abs() @ k.abs().transpose(-1, -2)).masked_fill(~vis, 0).amax(-1, keepdim=True)
         + (3 * min(wl.seq, window + sinks) + 16) * F + 2.0 ** -21)
    o = P @ v
    tol = U * o.abs() + (U * U + 2 * e) * (P @ v.abs())
    assert ((heads(got) - o).abs() / tol).max().item() <= 1.0


@pytest.mark.parametrize("window,sinks", [(0, 0), (100, 0), (40, 4)])
@pytest.mark.parametrize("wl", [LAYER.with_(batch=2, seq=100, qkv_bias=True), WIDE.with_(batch=1, seq=200, qkv_bias=True)],
                         ids=["hd64", "hd128"])
def test_gradients_with_keys_and_values_far_from_zero(wl, window, sinks):
    # D has to match P's normalisation: from the rounded o it is off by do . (o - bf16 o), and dq by that times the mean
    # key. Offsets of 4 in k and v (a q/k/v bias) make that 0.19 of the q gradients' largest value.
    inp = build_inputs(wl)
    r = np.random.default_rng(1)
    bias = inp["raw"][0]["bias"]
    for p in ("k", "v"):
        bias[p] = (bias[p] + 4 * np.sign(r.normal(size=bias[p].shape))).astype(np.float32)
    _hidden_step(wl, inp, window, sinks)
