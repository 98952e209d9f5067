"""Policy-gradient steps and windowed attention in the engine, on the GPU: against the oracle's step, the
schedules' invariants, and a run of both together as a user trains on sampled answers."""
import numpy as np
import pytest

import synthetic as syn
from oracle import model as M
from helpers import GRAD_COS, GRAD_MAXREL, LOSS_RTOL, build_inputs, compare_grads, make_context, oracle_step, run_step

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
lst = pytest.importorskip("layer_streamed_qlora_streaming_b200")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


WORKLOADS = {
    "tiny": syn.WORKLOADS["tiny"].with_(batch=3),
    # GQA, q/k/v bias, bf16 base, ragged sequence
    "tiny_gqa_bias_bf16": syn.WORKLOADS["tiny"].with_(n_kv_heads=2, qkv_bias=True, base_format="bf16", batch=2, seq=100),
}


def _rollout(wl, seed=0):
    """Targets, mask (an answer behind a prompt, some padding), advantages and log-probabilities of an older policy
    near the untrained model's."""
    r = np.random.default_rng(seed)
    toks, tgts = syn.tokens(wl, seed)
    pos = np.arange(wl.seq)[None, :]
    start = r.integers(1, wl.seq // 2, (wl.batch, 1))
    mask = ((pos >= start) & (pos < wl.seq - r.integers(0, 5, (wl.batch, 1)))).astype(np.int32).reshape(-1)
    adv = r.normal(size=wl.batch).astype(np.float32)
    old = (-np.log(wl.vocab) + r.normal(size=wl.tokens) * 0.1).astype(np.float32)
    return toks, tgts, mask, adv, old


def _run(ctx, wl, toks, tgts, mask, adv, old, **kw):
    grads = np.zeros(ctx.lora_numel(), dtype=np.float32)
    out = ctx.step_policy(toks, tgts, adv, wl.batch, wl.seq, old_logp=old, mask=mask, grads=grads, **kw)
    return out, grads


def _bytes(out, g):
    return np.array([out[k] for k in ("loss", "kl", "clipped", "ratio")], np.float32).tobytes(), g.tobytes()


@pytest.mark.parametrize("window,sinks", [(0, 0), (17, 4)])
@pytest.mark.parametrize("beta,norm", [(0.0, "token"), (0.2, "seq"), (0.2, "fixed")])
@pytest.mark.parametrize("name", list(WORKLOADS))
def test_policy_step_matches_oracle(name, beta, norm, window, sinks):
    wl = WORKLOADS[name]
    inp = build_inputs(wl)
    toks, tgts, mask, adv, old = _rollout(wl)
    tgts_masked = np.where(mask != 0, tgts, -100).astype(np.int32)  # not read where the mask is 0
    ctx = make_context(wl, inp, streamed=True)
    ctx.set_attention_window(window, sinks)
    code = {"token": lst.POLICY_TOKEN_MEAN, "seq": lst.POLICY_SEQ_MEAN, "fixed": lst.POLICY_FIXED}[norm]
    out, grads = _run(ctx, wl, toks, tgts_masked, mask, adv, old, kl_beta=beta, norm=code, clip_lo=0.2, clip_hi=0.28)
    logp = np.zeros(wl.tokens, dtype=np.float32)
    ctx.logp(logp)
    assert ctx.stats()["layer_reads_last_step"] == (3 if beta > 0 else 2) * wl.n_layers
    ref = M.policy_step(wl, inp["raw"], inp["head"], toks, tgts, adv, old=old.astype(np.float64), mask=mask, norm=norm,
                        lo=0.2, hi=0.28, beta=beta, bf16_acts=True, window=window, sinks=sinks)
    # the surrogate's terms have either sign: the loss is held to the size of its terms
    size = np.abs(ref["out"]).max()
    assert abs(out["loss"] - ref["out"][0]) <= LOSS_RTOL * size and abs(out["ratio"] - ref["out"][3]) <= LOSS_RTOL * size
    assert abs(out["kl"] - ref["out"][1]) <= LOSS_RTOL * max(ref["out"][1], 1e-3)
    assert np.max(np.abs(logp - ref["logp"])) <= LOSS_RTOL * np.abs(ref["logp"]).max()
    for l, p, w, cs, mr in compare_grads(ctx, grads, ref["grads"]):
        assert cs >= GRAD_COS and mr <= GRAD_MAXREL, (l, p, w, cs, mr)
    ctx.close()


def test_windowed_sft_step_matches_oracle():
    wl = syn.WORKLOADS["tiny"].with_(batch=2, n_kv_heads=2)
    inp = build_inputs(wl)
    ctx = make_context(wl, inp, streamed=True)
    plain = run_step(ctx, wl, inp)
    ctx.set_attention_window(11, 3)
    loss, grads, logits = run_step(ctx, wl, inp)
    ref = M.step(wl, raw_layers=inp["raw"], head=inp["head"], tokens=inp["tokens"], targets=inp["targets"], bf16_acts=True,
                 window=11, sinks=3)
    assert abs(loss - ref["loss"]) <= LOSS_RTOL * abs(ref["loss"])
    assert np.max(np.abs(logits - ref["logits"])) <= 1e-2 * np.abs(ref["logits"]).max()
    for l, p, w, cs, mr in compare_grads(ctx, grads, ref["grads"]):
        assert cs >= GRAD_COS and mr <= GRAD_MAXREL, (l, p, w, cs, mr)
    # a window of the whole sequence is causal attention; off again, the step gives its first bytes
    ctx.set_attention_window(wl.seq, 0)
    full = oracle_step(wl, inp)
    for l, p, w, cs, mr in compare_grads(ctx, run_step(ctx, wl, inp)[1], full["grads"]):
        assert cs >= GRAD_COS and mr <= GRAD_MAXREL, (l, p, w, cs, mr)
    ctx.set_attention_window(0)
    again = run_step(ctx, wl, inp)
    assert again[0] == plain[0] and again[1].tobytes() == plain[1].tobytes()
    ctx.close()


def test_policy_schedules_give_the_same_bytes():
    wl = WORKLOADS["tiny"].with_(n_layers=3)
    inp = build_inputs(wl)
    roll = _rollout(wl)
    runs = {}
    for key, kw in {"streamed": dict(streamed=True), "resident": dict(streamed=False),
                    "reuse": dict(streamed=True, reuse=True), "head_passes": dict(streamed=True, head_chunk=96)}.items():
        ctx = make_context(wl, inp, **kw)
        ctx.set_attention_window(30, 2)
        runs[key] = [_bytes(*_run(ctx, wl, *roll, kl_beta=0.1)) for _ in range(2)]
        ctx.close()
    assert runs["streamed"][0] == runs["streamed"][1]
    for key in ("resident", "reuse", "head_passes"):
        assert runs[key] == runs["streamed"], key


def test_updates_on_the_same_samples():
    # the loop of a user: the first update is on-policy (no old_logp), the next ones take its log-probabilities
    wl = WORKLOADS["tiny"]
    inp = build_inputs(wl)
    toks, tgts, mask, adv, _ = _rollout(wl, 3)
    ctx = make_context(wl, inp, streamed=True)
    ctx.set_attention_window(24, 4)
    ctx.set_optimizer(lr=1e-3)
    out, g0 = _run(ctx, wl, toks, tgts, mask, adv, None, kl_beta=0.05)
    old = torch.empty(wl.tokens, device="cuda")
    ctx.logp(old)
    assert out["ratio"] == pytest.approx(1.0, abs=1e-5) and out["clipped"] == 0 and np.any(g0 != 0)
    assert np.all(old.cpu().numpy()[mask == 0] == 0) and np.all(old.cpu().numpy()[mask != 0] < 0)
    second, g1 = _run(ctx, wl, toks, tgts, mask, adv, old, kl_beta=0.05)
    # the same samples again: the ratio has moved off 1, and the surrogate has improved on the first step's
    assert second["ratio"] != 1.0 and np.any(g1 != g0)
    # the ratio at unchanged weights is 1 whatever the schedule: old_logp are this policy's own
    ctx.set_optimizer(off=True)
    ctx.step_policy(toks, tgts, adv, wl.batch, wl.seq, mask=mask)
    ctx.logp(old)
    third = ctx.step_policy(toks, tgts, adv, wl.batch, wl.seq, old_logp=old, mask=mask)
    assert third["ratio"] == pytest.approx(1.0, abs=1e-6) and third["clipped"] == 0
    ctx.close()


def test_policy_step_per_token_advantages_and_empty_mask():
    wl = WORKLOADS["tiny"]
    inp = build_inputs(wl)
    toks, tgts, mask, adv, old = _rollout(wl)
    ctx = make_context(wl, inp, streamed=True)
    a = _run(ctx, wl, toks, tgts, mask, adv, old)
    b = _run(ctx, wl, toks, tgts, mask, np.repeat(adv, wl.seq), old, adv_per_seq=False)
    assert _bytes(*a) == _bytes(*b)
    none, g = _run(ctx, wl, toks, tgts, np.zeros_like(mask), adv, old, kl_beta=0.1)
    assert all(v == 0 for v in none.values()) and np.all(g == 0)
    ctx.close()


def test_policy_step_refusals_and_state():
    wl = WORKLOADS["tiny"]
    inp = build_inputs(wl)
    toks, tgts, mask, adv, old = _rollout(wl)
    ctx = make_context(wl, inp, streamed=True)
    buf = np.zeros(wl.tokens, dtype=np.float32)

    def refused(status, f):
        with pytest.raises(lst.LstError) as e:
            f()
        assert e.value.status == status

    refused(2, lambda: ctx.logp(buf))
    for kw in (dict(clip_lo=-0.1), dict(clip_lo=2.0), dict(clip_hi=float("nan")), dict(kl_beta=-1.0), dict(norm=5)):
        refused(1, lambda: _run(ctx, wl, toks, tgts, mask, adv, old, **kw))
    refused(1, lambda: ctx.step_policy(toks, tgts, None, wl.batch, wl.seq))
    refused(1, lambda: ctx.step_policy(toks, tgts, adv, wl.batch + 1, wl.seq))
    refused(1, lambda: ctx.set_attention_window(-1))
    refused(1, lambda: ctx.set_attention_window(4, -1))
    _run(ctx, wl, toks, tgts, mask, adv, old)
    ctx.logp(buf)
    run_step(ctx, wl, inp, want_logits=False)
    refused(2, lambda: ctx.logp(buf))
    # a counted target out of range is a device error, and the next step is clean
    bad = tgts.copy()
    bad[np.nonzero(mask)[0][0]] = wl.vocab
    refused(6, lambda: _run(ctx, wl, toks, bad, mask, adv, old))
    good = _run(ctx, wl, toks, tgts, mask, adv, old)
    fresh = make_context(wl, inp, streamed=True)
    assert _bytes(*good) == _bytes(*_run(fresh, wl, toks, tgts, mask, adv, old))
    ctx.close()
    fresh.close()
