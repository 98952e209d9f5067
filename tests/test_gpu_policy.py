"""Clipped policy loss on the GPU against the oracle's formula in 64 bits.

Tolerances: f = 2^-24 is fp32's half step relative to a value, u = 2^-8 bf16's. logp = (x_y - m) - log s:
the sum of V exponentials in fp32 (threads' chains of at most V / 256 terms, then trees) with an
exponential within 2 ulp of its value gives log s an error of at most (V / 256 + 64) f + 2^-21, and the
differences round to f of |x_y| + |m| + |logp|: el. The ratio, the KL slope and the weight then carry
el + 2^-20 relative, so dlogits is off by at most u |dlogits| + c (el + 2^-20) (p + onehot), where c
bounds w |slope| with each of its two terms taken absolutely (+ beta w for the cancellation of
1 - exp(d)). out: f-level sums of terms whose logp is off by el: (el + 2^-20) sum w (|r A| + beta (|kl| +
|1 - exp d|) ...) and so on; the counts of clipped tokens are exact because no ratio lies within 1e-4 of
a border."""
import numpy as np
import pytest

from oracle import model as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
lst = pytest.importorskip("layer_streamed_qlora_streaming_b200")

U, F = 2.0 ** -8, 2.0 ** -24
NORMS = {"token": lst.POLICY_TOKEN_MEAN, "seq": lst.POLICY_SEQ_MEAN, "fixed": lst.POLICY_FIXED}


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Case:
    def __init__(self, nseq, S, V, norm="token", beta=0.1, per_seq=True, keep=0.7, seed=0, offset=0, lo=0.2, hi=0.28):
        r = np.random.default_rng(seed + 7 * V + S)
        T = nseq * S
        self.nseq, self.S, self.V, self.T, self.norm, self.beta, self.per_seq, self.lo, self.hi = nseq, S, V, T, norm, beta, per_seq, lo, hi
        self.x = (r.normal(size=(T, V)) * 2.5).astype(np.float32)
        self.y = r.integers(0, V, T).astype(np.int32)
        self.mask = (r.uniform(size=T) < keep).astype(np.int32) * r.integers(1, 9, T).astype(np.int32)  # any nonzero counts
        m = self.x.max(1).astype(np.float64)
        logp = self.x[np.arange(T), self.y] - m - np.log(np.exp(self.x.astype(np.float64) - m[:, None]).sum(1))
        self.old = (logp + r.normal(size=T) * 0.2).astype(np.float32)
        for _ in range(20):  # away from the clip's borders
            near = np.min(np.abs(np.exp(logp - self.old)[:, None] - [1 - lo, 1 + hi]), 1) < 1e-4
            self.old[near] += 0.001
        self.ref = (logp + r.normal(size=T) * 0.3).astype(np.float32)
        self.ref[::5] = logp[::5]  # tokens where the policy is at the reference
        self.adv = r.normal(size=nseq if per_seq else T).astype(np.float32)
        dev = lambda a: torch.from_numpy(a).cuda()  # noqa: E731
        # logits that start `offset` floats behind a 16-byte boundary
        flat = torch.empty(T * V + offset, device="cuda")
        self.tx = flat[offset:].view(T, V)
        self.tx.copy_(dev(self.x))
        self.ty, self.tmask, self.told, self.tref, self.tadv = (dev(a) for a in (self.y, self.mask, self.old, self.ref, self.adv))
        self.logp = torch.full((T + 1,), 7.0, device="cuda")
        self.out = torch.full((5,), 7.0, device="cuda")
        self.dlog = torch.full((T * V + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.n = lst.policy_scratch(T, S)
        self.scratch = torch.full((self.n + 4,), 7.0, device="cuda")

    def run(self, stream=None, **kw):
        a = dict(dlogits=self.dlog, old_logp=self.told, ref_logp=self.tref if self.beta > 0 else None, mask=self.tmask,
                 clip_lo=self.lo, clip_hi=self.hi, kl_beta=self.beta, norm=NORMS[self.norm], adv_per_seq=self.per_seq)
        lst.k_policy_loss(self.tx, self.T, self.V, self.ty, self.S, self.tadv, self.logp, self.out, self.scratch,
                          stream=stream, **{**a, **kw})

    def check(self, old="own", mask="own", ref="own", grads=True):
        T, V = self.T, self.V
        old = self.old.astype(np.float64) if isinstance(old, str) else old
        mask = self.mask if isinstance(mask, str) else np.ones(T)
        ref = (self.ref.astype(np.float64) if self.beta > 0 else None) if isinstance(ref, str) else ref
        x, adv = self.x.astype(np.float64), self.adv.astype(np.float64)
        out, g, logp = M.policy_dlogits(x, self.y, old, ref, adv, mask, self.nseq, self.S, self.norm, self.lo, self.hi, self.beta)
        on = np.asarray(mask) != 0
        w = M.policy_weights(mask, self.nseq, self.S, self.norm)
        mx = np.abs(np.where(np.isfinite(x), x, 0)).max(1)
        el = np.where(on, (V / 256 + 64) * F + 2.0 ** -21 + 4 * F * (2 * mx + np.abs(np.where(on, logp, 0))), 0)
        e = el + 2.0 ** -20
        got = self.logp[:T].double().cpu().numpy()
        assert np.all(np.abs(got - logp) <= el), np.max(np.abs(got - logp) / np.maximum(el, 1e-30))
        A = np.repeat(adv, self.S) if self.per_seq else adv
        r = np.exp(logp - old) if old is not None else np.ones(T)
        d = ref - logp if ref is not None else np.zeros(T)
        size = np.stack([np.abs(r * A) + self.beta * (np.abs(np.expm1(d)) + np.expm1(d) - d), np.abs(np.expm1(d)) + np.expm1(d) - d,
                         np.zeros(T), r])
        # (the clipped surrogate is below (1 + hi) |A| or |r A| in magnitude; the sum of T terms rounds once to fp32)
        size[0] += (1 + (self.hi if np.isfinite(self.hi) else 0)) * np.abs(A)
        tol = np.where(on, w * e, 0) @ np.where(on, size, 0).T + 8 * F * np.abs(out) + 1e-12
        assert np.all(np.abs(self.out[:4].double().cpu().numpy() - out) <= tol), (self.out[:4], out, tol)
        if grads:
            p = np.exp(x - x.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            p[np.arange(T)[on], self.y[on]] += 1
            c = np.where(on, w * (np.abs(r * A) + self.beta * (np.abs(np.expm1(d)) + 1)), 0)
            bound = U * np.abs(g) + (c * e)[:, None] * p + 1e-37
            dl = self.dlog[:T * V].double().cpu().numpy().reshape(T, V)
            assert np.all(np.abs(dl - g) <= bound), np.max(np.abs(dl - g) / bound)
        assert torch.all(self.dlog[T * V:] == 7) and torch.all(self.logp[T:] == 7) and torch.all(self.out[4:] == 7)
        assert torch.all(self.scratch[self.n:] == 7)
        assert lst.device_error() == 0


@pytest.mark.parametrize("norm", list(NORMS))
@pytest.mark.parametrize("nseq,S,V,per_seq,beta,offset", [
    (1, 1, 1, True, 0.1, 0),          # one token, one word
    (1500, 1, 33, True, 0.1, 0),      # more sequences than are counted at once: of one token,
    (1030, 33, 12, True, 0.1, 0),     # of more than a warp's width
    (1025, 5, 40, False, 0.1, 0),     # and of fewer
    (2, 1500, 20, True, 0.1, 0),      # sequences of several hundred tokens, over a short vocabulary
    (2, 3, 2, False, 0.1, 1),
    (4, 32, 512, True, 0.1, 0),
    (3, 17, 1001, False, 0.0, 3),     # odd vocabulary, odd base
    (2, 9, 509, True, 0.1, 2),        # the longest rows of a warp's variants and the next ones
    (2, 9, 2044, False, 0.1, 0),
    (3, 7, 2047, True, 0.1, 1),
    (2, 9, 4092, True, 0.1, 0),
    (2, 9, 4094, False, 0.1, 3),
    (2, 9, 16384, True, 0.1, 2),
    (1, 40, 32003, False, 0.1, 0),
    (5, 1, 4099, False, 0.5, 1),      # sequences of one token
    (1, 6, 151936, True, 0.1, 0),
    (1, 5, 262145, True, 0.1, 1)])
def test_policy_loss(norm, nseq, S, V, per_seq, beta, offset):
    c = Case(nseq, S, V, norm, beta, per_seq, offset=offset)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_policy_loss_largest_vocabulary():
    c = Case(1, 3, 1 << 20, "seq", 0.1, True, keep=1.1)
    c.run()
    torch.cuda.synchronize()
    c.check()


def test_policy_variants():
    c = Case(3, 20, 777, "seq", 0.0)
    c.run(old_logp=None)
    torch.cuda.synchronize()
    c.check(old=None)
    c.run(mask=None)
    torch.cuda.synchronize()
    c.check(mask=None)
    # a reference without a KL weight: the KL is reported, the loss and gradient do not have it
    c.run(ref_logp=c.tref)
    torch.cuda.synchronize()
    c.check(ref=c.ref.astype(np.float64))
    # no upper clip; loss only
    before = c.dlog.clone()
    c.hi = float("inf")
    c.run(dlogits=None)
    torch.cuda.synchronize()
    c.check(grads=False)
    assert torch.equal(before, c.dlog)


@pytest.mark.parametrize("V", [4096, 4099, 40000])
def test_policy_dlogits_at_any_element(V):
    # logits aligned, dlogits not: the same gradient, nothing around it touched
    c = Case(2, 9, V)
    c.run()
    c.check()
    n = c.T * V
    for off in (1, 2, 3, 4, 5):
        flat = torch.full((n + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        c.run(dlogits=flat[off:off + n])
        diff = (flat[off:off + n].float() - c.dlog[:n].float()).abs()
        assert torch.all(diff <= 2 * U * c.dlog[:n].float().abs())  # (a row's ends are formed apart)
        assert torch.all(flat[:off] == 7) and torch.all(flat[off + n:] == 7)


@pytest.mark.parametrize("V", [300, 5001])
def test_policy_masked_tokens_are_not_read(V):
    c = Case(4, 8, V, "seq", 0.1, False)
    c.mask[8:16] = 0  # a sequence without a counted token
    c.tmask.copy_(torch.from_numpy(c.mask))
    off = torch.from_numpy(c.mask == 0).cuda()
    c.tx[off] = float("nan")
    c.ty[off] = -100
    c.told[off] = float("nan")
    c.tref[off] = float("inf")
    c.tadv[off] = float("nan")
    c.run()
    torch.cuda.synchronize()
    c.y = np.where(c.mask != 0, c.y, 0)
    c.check()
    # nothing counts at all: zeros, not 0 / 0
    c.tmask.zero_()
    for n in NORMS.values():
        c.run(norm=n)
        torch.cuda.synchronize()
        assert torch.all(c.out[:4] == 0) and torch.all(c.dlog[:c.T * c.V] == 0) and torch.all(c.logp[:c.T] == 0)


@pytest.mark.parametrize("V", [1000, 5000])
def test_policy_words_that_are_ruled_out(V):
    # -inf logits (words a sampler was not allowed to draw) take no probability and no gradient
    c = Case(2, 10, V, "token", 0.1)
    ban = np.random.default_rng(1).uniform(size=c.x.shape) < 0.9
    ban[np.arange(c.T), c.y] = False
    c.x[ban] = -np.inf
    m = c.x.max(1).astype(np.float64)
    logp = c.x[np.arange(c.T), c.y] - m - np.log(np.exp(c.x - m[:, None]).sum(1))
    c.old = (logp + 0.05).astype(np.float32)
    c.ref = (logp - 0.1).astype(np.float32)
    c.tx.copy_(torch.from_numpy(c.x))
    c.told.copy_(torch.from_numpy(c.old))
    c.tref.copy_(torch.from_numpy(c.ref))
    c.run()
    torch.cuda.synchronize()
    c.check()
    assert torch.all(c.dlog[:c.T * c.V].view(c.T, c.V)[torch.from_numpy(ban).cuda()] == 0)


@pytest.mark.parametrize("V", [100, 6000])
def test_policy_bad_target_is_reported_and_adds_nothing(V):
    c = Case(2, 6, V, "fixed", 0.1, keep=1.1)
    c.run()
    torch.cuda.synchronize()
    c.ty[3] = V
    c.ty[7] = -1
    c.run()
    torch.cuda.synchronize()
    assert lst.device_error() == 2
    c.mask[3] = c.mask[7] = 0  # the fixed normalisation does not depend on the count
    c.check()


@pytest.mark.parametrize("V", [900, 9000])
def test_policy_two_streams_and_a_graph(V):
    cs = [Case(3, 16, V, "seq", 0.1, seed=s) for s in range(2)]
    for c in cs:
        c.run()
    torch.cuda.synchronize()
    want = [(c.out.clone(), c.logp.clone(), c.dlog.clone()) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    for _ in range(3):
        for c, s in zip(cs, streams):
            c.run(stream=s)
    torch.cuda.synchronize()
    for c, w in zip(cs, want):
        assert all(torch.equal(a, b) for a, b in zip((c.out, c.logp, c.dlog), w))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        cs[0].run(stream=torch.cuda.current_stream())
    for name in ("tx", "ty", "tmask", "told", "tref", "tadv"):
        getattr(cs[0], name).copy_(getattr(cs[1], name))
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip((cs[0].out, cs[0].logp, cs[0].dlog), want[1]))
