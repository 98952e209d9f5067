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


def _parts(wl, window, sinks):
    """fp32 values that the dK / dV kernel leaves for the kernel that joins the parts of cut key tiles."""
    n = lst.attention_window_scratch(wl.tokens, wl.seq, wl.n_heads, wl.n_kv_heads, wl.head_dim, window, sinks)
    return n - 2 * wl.batch * wl.n_heads * -(-wl.seq // 128) * 128  # without (lse, D) of every query


@pytest.mark.parametrize("wl,window,sinks,cut", [
    (WIDE.with_(batch=1, seq=1500), 256, 4, True),      # key tiles cut into shares, joined
    (LAYER.with_(batch=1, seq=1100), 300, 130, True),   # sinks that cross a tile
    (WIDE.with_(batch=2, seq=300), 200, 4, False)])     # whole key tiles
def test_rotary_embedding_undone_in_every_tile(wl, window, sinks, cut):
    # only a step undoes the embedding in dq and dk; far positions and the joined tiles have their own code for it
    assert (_parts(wl, window, sinks) > 0) == cut
    _hidden_step(wl, build_inputs(wl), window, sinks)


@pytest.mark.parametrize("window,sinks", [(17, 4), (5, 0)])
def test_dpo_step_under_a_window(window, sinks):
    wl = syn.WORKLOADS["tiny"].with_(batch=4, n_kv_heads=2)
    inp = build_inputs(wl)
    toks, tgts, mask = syn.preference_pairs(wl)
    ctx = make_context(wl, inp, streamed=True)
    ctx.set_attention_window(window, sinks)
    grads = np.zeros(ctx.lora_numel(), dtype=np.float32)
    loss = ctx.step_dpo(toks, tgts, mask, wl.batch // 2, wl.seq, 0.5, grads)
    ref = M.dpo_step(wl, inp["raw"], inp["head"], toks, tgts, wl.batch // 2, 0.5, mask=mask, bf16_acts=True, window=window,
                     sinks=sinks)
    assert abs(loss - ref["loss"]) <= LOSS_RTOL * abs(ref["loss"])
    _check_grads(ctx, grads, ref["grads"])
    ctx.close()


def test_window_and_lengths_that_change_between_steps():
    # the backward's scratch grows with the steps; a step's bytes do not depend on the ones before it
    wl = WIDE.with_(batch=2, seq=700)
    inp = build_inputs(wl)
    ctx = make_context(wl, inp, streamed=True)
    grads = {}

    def step(batch, seq, window, sinks):
        g = np.zeros(ctx.lora_numel(), dtype=np.float32)
        ctx.set_attention_window(window, sinks)
        n = batch * seq
        ctx.step_hidden(syn.to_bf16_bits(inp["x"][:n]), syn.to_bf16_bits(inp["G"][:n]), batch, seq, g)
        return g.tobytes()

    runs = [(1, 9, 3, 0), (2, 700, 100, 4), (1, 700, 700, 0), (2, 700, 30, 200), (2, 64, 5, 5)]
    for i in (0, 1, 2, 3, 4, 2, 0, 3, 1):
        assert grads.setdefault(i, step(*runs[i])) == step(*runs[i])
    ctx.close()


@pytest.mark.slow
def test_32b_shaped_layers_under_a_window():
    # the layers whose top q / k gradients are the most sensitive to rounding: the bound of the causal path
    wl = syn.WORKLOADS["qwen32b"].with_(n_layers=2, batch=1, seq=256)
    inp = build_inputs(wl)
    ctx = make_context(wl, inp, streamed=True)
    window, sinks = 100, 4
    ctx.set_attention_window(window, sinks)
    loss, grads, _ = run_step(ctx, wl, inp, want_logits=False)
    ctx.close()
    ref = M.step(wl, raw_layers=inp["raw"], head=inp["head"], tokens=inp["tokens"], targets=inp["targets"], bf16_acts=True,
                 window=window, sinks=sinks)
    assert abs(loss - ref["loss"]) <= LOSS_RTOL * abs(ref["loss"])
    _check_grads(ctx, grads, ref["grads"])
