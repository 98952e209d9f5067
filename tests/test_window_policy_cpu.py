"""CPU checks of windowed attention and the policy loss: the oracle's formulas against torch autograd
and central differences, and the library's refusals (no argument that is refused reaches the GPU)."""
import ctypes as C

import numpy as np
import pytest

import layer_streamed_qlora_streaming_b200 as lst
import synthetic as syn
from oracle import model as M

torch = pytest.importorskip("torch")


# ------------------------------------------------------------------------------------ oracle
@pytest.mark.parametrize("seq,window,sinks", [(1, 1, 0), (7, 1, 0), (9, 3, 2), (12, 5, 9), (6, 40, 3)])
def test_visible_is_the_rule_pair_by_pair(seq, window, sinks):
    vis = M.visible(seq, window, sinks)
    for i in range(seq):
        for j in range(seq):
            assert vis[i, j] == (j <= i and (i - j < window or j < sinks))
    assert np.array_equal(M.visible(seq), M.visible(seq, seq, 0))


@pytest.mark.parametrize("window,sinks", [(1, 0), (3, 2), (50, 0), (4, 11)])
def test_windowed_attention_matches_autograd(window, sinks):
    B, S, hq, hkv, hd = 2, 11, 4, 2, 8
    g = torch.Generator().manual_seed(3)
    q, k, v, do = (torch.randn(B * S, h, hd, generator=g, dtype=torch.float64) for h in (hq, hkv, hkv, hq))
    leaves = [t.clone().requires_grad_() for t in (q, k, v)]
    qq, kk, vv = (t.reshape(B, S, -1, hd).transpose(1, 2) for t in leaves)
    kk, vv = (t.repeat_interleave(hq // hkv, 1) for t in (kk, vv))
    o = torch.nn.functional.scaled_dot_product_attention(qq, kk, vv, attn_mask=torch.from_numpy(M.visible(S, window, sinks)))
    o = o.transpose(1, 2).reshape(B * S, hq, hd)
    o.backward(do)
    on, P = M.attention(q.numpy(), k.numpy(), v.numpy(), B, S, window, sinks)
    grads = M.attention_bwd(do.numpy(), q.numpy(), k.numpy(), v.numpy(), P, B, S)
    np.testing.assert_allclose(on, o.detach().numpy(), atol=1e-12)
    for a, t in zip(grads, leaves):
        np.testing.assert_allclose(a, t.grad.numpy(), atol=1e-12)


def _policy_case(nseq, S, V, seed=0):
    r = np.random.default_rng(seed)
    T = nseq * S
    x = r.normal(size=(T, V)) * 2
    y = r.integers(0, V, T)
    mask = (r.uniform(size=T) < 0.7).astype(np.int32)
    mask[:S] = 0  # a sequence without a counted token
    logp = x[np.arange(T), y] - np.log(np.exp(x).sum(1))
    return x, y, mask, logp + r.normal(size=T) * 0.2, logp + r.normal(size=T) * 0.3, r.normal(size=T), r


@pytest.mark.parametrize("norm", ["token", "seq", "fixed"])
@pytest.mark.parametrize("beta", [0.0, 0.3])
def test_policy_gradient_matches_autograd_and_differences(norm, beta):
    nseq, S, V, lo, hi = 4, 5, 13, 0.2, 0.28
    x, y, mask, old, ref, adv, r = _policy_case(nseq, S, V)
    out, g, logp = M.policy_dlogits(x, y, old, ref, adv, mask, nseq, S, norm, lo, hi, beta)
    t = torch.from_numpy(x).requires_grad_()
    lp = torch.log_softmax(t, -1).gather(1, torch.from_numpy(y)[:, None])[:, 0]
    ratio, A = torch.exp(lp - torch.from_numpy(old)), torch.from_numpy(adv)
    d = torch.from_numpy(ref) - lp
    token = -torch.minimum(ratio * A, ratio.clamp(1 - lo, 1 + hi) * A) + beta * (torch.exp(d) - d - 1)
    m = torch.from_numpy(mask).double().reshape(nseq, S)
    w = {"token": m / m.sum(), "seq": m / m.sum(1, keepdim=True).clamp(min=1) / nseq, "fixed": m / m.numel()}[norm]
    loss = (w.reshape(-1) * token).sum()
    loss.backward()
    assert out[0] == pytest.approx(loss.item(), rel=1e-12)
    np.testing.assert_allclose(g, t.grad.numpy(), atol=1e-13)
    assert 0 < out[2] < 1 and np.all(g[mask == 0] == 0) and np.all(logp[mask == 0] == 0)
    # central differences of the loss in a few logits (none of the ratios lies within 1e-4 of the clip's borders)
    ratios = np.exp(logp - old)[mask != 0]
    assert np.min(np.abs(ratios[:, None] - [1 - lo, 1 + hi])) > 1e-4
    for _ in range(20):
        i, j, h = r.integers(nseq * S), r.integers(V), 1e-6
        up, down = x.copy(), x.copy()
        up[i, j] += h
        down[i, j] -= h
        f = [M.policy_dlogits(z, y, old, ref, adv, mask, nseq, S, norm, lo, hi, beta)[0][0] for z in (up, down)]
        assert (f[0] - f[1]) / (2 * h) == pytest.approx(g[i, j], abs=1e-8)


def test_policy_on_policy_gradient_is_the_advantage():
    # ratio 1 everywhere: the gradient in logp is -w A, the loss -sum w A
    x, y, mask, _, _, adv, _ = _policy_case(3, 4, 9, 2)
    out, g, _ = M.policy_dlogits(x, y, None, None, adv, mask, 3, 4, "token", 0.2, 0.2, 0.0)
    w = M.policy_weights(mask, 3, 4, "token")
    assert out[0] == pytest.approx(-(w * adv).sum()) and out[2] == 0 and out[3] == pytest.approx(1)
    on = mask != 0
    p = np.exp(x) / np.exp(x).sum(1, keepdims=True)
    np.testing.assert_allclose(g[on, y[on]], (-(w * adv))[on] * (1 - p[on, y[on]]), atol=1e-14)


def test_policy_step_equals_the_sft_gradient_direction_on_policy():
    # on-policy, advantage 1, no KL: dL/dlogp = -1/T per token, the gradient of the mean cross-entropy
    wl = syn.WORKLOADS["tiny"].with_(n_layers=1, batch=2, seq=12)
    raw = [syn.layer_weights(wl, 0)]
    head = (syn.embedding(wl), syn.norm_gain(wl), syn.lm_head(wl))
    toks, tgts = syn.tokens(wl, 0)
    pol = M.policy_step(wl, raw, head, toks, tgts, np.ones(wl.batch), norm="fixed", window=5, sinks=2)
    sft = M.step(wl, raw, head=head, tokens=toks, targets=tgts, window=5, sinks=2)
    for p in syn.PROJ:
        for a, b in zip(pol["grads"][0][p], sft["grads"][0][p]):
            np.testing.assert_allclose(a, b, atol=1e-15 + 1e-12 * np.abs(b).max())


# ------------------------------------------------------------------------------------ refusals
OK_W = dict(q=4096, ldq=64, k=4096, ldk=64, v=4096, ldv=64, o=4096, ldo=64, lse=4096, T=8, S=4, hq=1, hkv=1, hd=64,
            window=2, sinks=1)


@pytest.mark.parametrize("bad", [
    dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(T=0), dict(T=7), dict(S=0), dict(S=-4),
    dict(hq=3, hkv=2), dict(hq=0), dict(hkv=0), dict(hd=96), dict(hd=0), dict(window=0), dict(window=-1), dict(sinks=-1),
    dict(ldq=68), dict(ldk=60), dict(ldv=56), dict(ldo=63), dict(q=4098), dict(k=4104), dict(v=4097), dict(o=4104),
    dict(T=1 << 40, S=1 << 20), dict(T=1 << 30, S=1 << 20, hq=4, hkv=1, ldq=256, ldo=256)])
def test_window_forward_refuses(bad):
    n = lst.launch_count()
    with pytest.raises(lst.LstError) as e:
        lst.k_attention_window_fwd(**{**OK_W, **bad})
    assert e.value.status == 1 and lst.launch_count() == n


@pytest.mark.parametrize("bad", [
    dict(dout=None), dict(scratch=None), dict(dq=None), dict(dk=None), dict(dv=None), dict(scratch=4100), dict(lddo=68),
    dict(lddq=4), dict(lddk=60), dict(lddv=0), dict(dq=4098), dict(dk=4104), dict(dv=4097), dict(window=0), dict(hd=80),
    dict(T=6)])
def test_window_backward_refuses(bad):
    ok = {**OK_W, "dout": 4096, "lddo": 64, "scratch": 4096, "dq": 4096, "lddq": 64, "dk": 4096, "lddk": 64, "dv": 4096,
          "lddv": 64}
    n = lst.launch_count()
    with pytest.raises(lst.LstError) as e:
        lst.k_attention_window_bwd(**{**ok, **bad})
    assert e.value.status == 1 and lst.launch_count() == n


def test_window_scratch_sizes():
    assert lst.attention_window_scratch(8, 4, 2, 1, 64, 2, 1) >= 16
    for bad in ((7, 4, 2, 1, 64, 2, 1), (8, 4, 3, 2, 64, 2, 1), (8, 4, 2, 1, 72, 2, 1), (8, 4, 2, 1, 64, 0, 1),
                (8, 4, 2, 1, 64, 2, -1)):
        with pytest.raises(lst.LstError):
            lst.attention_window_scratch(*bad)


OK_P = dict(logits=4096, T=6, V=10, targets=4096, S=3, adv=4096, logp=4096, out=4096, scratch=4096, dlogits=4096,
            old_logp=4096, ref_logp=4096, mask=4096, clip_lo=0.2, clip_hi=0.2, kl_beta=0.1, norm=0)


@pytest.mark.parametrize("bad", [
    dict(logits=None), dict(targets=None), dict(adv=None), dict(logp=None), dict(out=None), dict(scratch=None),
    dict(scratch=4104), dict(T=0), dict(T=7), dict(S=0), dict(V=0), dict(V=(1 << 20) + 1), dict(clip_lo=-0.1),
    dict(clip_lo=1.5), dict(clip_hi=-0.1), dict(clip_lo=float("nan")), dict(clip_hi=float("nan")), dict(kl_beta=-1.0),
    dict(kl_beta=float("nan")), dict(kl_beta=float("inf")), dict(ref_logp=None), dict(norm=3), dict(norm=-1),
    dict(T=1 << 40, S=1)])
def test_policy_loss_refuses(bad):
    n = lst.launch_count()
    with pytest.raises(lst.LstError) as e:
        lst.k_policy_loss(**{**OK_P, **bad})
    assert e.value.status == 1 and lst.launch_count() == n


def test_policy_scratch_sizes():
    assert lst.policy_scratch(6, 3) >= 4 * 6 + 2
    for bad in ((0, 1), (7, 3), (6, 0), (-6, 3)):
        with pytest.raises(lst.LstError):
            lst.policy_scratch(*bad)
    assert C.sizeof(lst.Policy) == 20


def test_pointer_of_a_one_element_tensor_with_any_stride():
    # a dimension of one element has no stride to speak of; two strided ones are refused
    x = torch.arange(8.0)
    assert lst._ptr(x[::4][:1]) == x.data_ptr()
    assert lst._ptr(x.view(4, 2)[:, :1].t()[:, :1]) == x.data_ptr()
    with pytest.raises(ValueError):
        lst._ptr(x[::4])


def test_null_context_is_refused():
    L = lst.lib()
    assert L.lst_set_attention_window(None, 4, 0) == 1
    assert L.lst_get_logp(None, None) == 1
    assert L.lst_step_policy(None, None, None, None, None, None, 1, 1, None, None, None) == 1


def test_policy_factors_of_zero_take_out_what_overflows():
    # an advantage of 0 the ratio, a weight of 0 the KL term; one that counts stays infinite
    logp, old, ref = np.array([-1.0, -1.0, -np.inf]), np.array([-1000.0, -1.2, -1.0]), np.array([-1.0, 1000.0, -1.0])
    w, adv = np.full(3, 1 / 3), np.array([0.0, 2.0, -1.0])
    out, g = M.policy_loss(logp, old, ref, adv, w, 0.2, 0.2, 0.0)
    assert np.all(np.isfinite(out[[0, 2]])) and np.all(np.isinf(out[[1, 3]])) and np.all(np.isfinite(g))
    assert g[0] == 0 and out[0] == pytest.approx((-1.2 * 2 + 0.8) / 3)
    out, g = M.policy_loss(logp, old, ref, adv, w, 0.2, 0.2, 0.1)
    assert np.isposinf(out[0]) and g[0] == 0 and np.isneginf(g[1])


def test_pointer_of_a_strided_column_is_refused():
    # [4, 1] with an innermost stride of its own: no leading dimension tells an entry point about its rows
    x = torch.arange(8.0)
    for y in (x.as_strided((4, 1), (2, 3)), x.view(4, 2)[:, :1].t().as_strided((4, 1), (2, 2)), x.view(1, 8).t()):
        with pytest.raises(ValueError):
            lst._ptr(y)
    assert lst._ptr(x.view(8, 1)) == x.data_ptr()  # contiguous
    assert lst._ptr(x[:1].as_strided((1, 1), (5, 7))) == x.data_ptr()  # one element
