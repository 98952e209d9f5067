"""The policy loss where it can go wrong by value or by the number of rows, on the GPU; formula, cases and tolerances
of test_gpu_policy.py."""
import numpy as np
import pytest

from test_gpu_policy import Case

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
lst = pytest.importorskip("layer_streamed_qlora_streaming_b200")


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


def _result(c):
    torch.cuda.synchronize()
    assert lst.device_error() == 0
    return c.out[:4].cpu().numpy().copy(), c.logp[:c.T].cpu().numpy().copy(), c.dlog[:c.T * c.V].clone()


VOCABULARIES = [300, 5001, 40000, 310001]  # a warp, clusters, rows read twice


@pytest.mark.parametrize("V", VOCABULARIES)
def test_policy_zero_advantage_with_a_ratio_that_overflows(V):
    # u = 0 A = 0 whatever the ratio: all but the reported ratio is what any finite one gives
    c = Case(2, 4, V, "seq", 0.1, False, keep=1.1)
    c.adv[::3] = 0
    c.tadv.copy_(torch.from_numpy(c.adv))
    c.run()
    torch.cuda.synchronize()
    c.check()
    want = _result(c)
    c.told[::3] -= 200.0
    c.run()
    out, logp, dlog = _result(c)
    assert np.array_equal(out[:3], want[0][:3]) and np.isposinf(out[3])
    assert np.array_equal(logp, want[1]) and torch.equal(dlog, want[2])


@pytest.mark.parametrize("V", VOCABULARIES)
def test_policy_reference_without_a_weight_that_overflows(V):
    # kl_beta 0: the KL estimate is reported and nothing else depends on it
    c = Case(2, 4, V, "token", 0.0, True, keep=1.1)
    c.x[1, c.y[1]] = -np.inf  # a target that was ruled out: log-probability minus infinity
    c.tx.copy_(torch.from_numpy(c.x))
    c.run()
    want = _result(c)
    assert np.isneginf(want[1][1]) and np.all(np.isfinite(want[0])) and torch.all(torch.isfinite(want[2]))
    c.tref[5] += 500.0
    c.run(ref_logp=c.tref)
    out, logp, dlog = _result(c)
    assert np.array_equal(out[[0, 2, 3]], want[0][[0, 2, 3]]) and np.isposinf(out[1])
    assert np.array_equal(logp, want[1]) and torch.equal(dlog, want[2])


class Many:
    """Many rows, made and checked on the GPU in 64 bits; the tolerances of Case."""

    def __init__(self, T, V, S, offset=0, seed=0, beta=0.1, lo=0.2, hi=0.28):
        g = torch.Generator(device="cuda").manual_seed(seed * 1009 + V + T)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.T, self.V, self.S, self.beta, self.lo, self.hi = T, V, S, beta, lo, hi
        self.x = torch.empty(T * V + offset, device="cuda")[offset:].view(T, V)
        self.x.copy_(rnd(T, V).mul_(2.5))
        self.y = torch.randint(0, V, (T,), generator=g, device="cuda", dtype=torch.int32)
        self.mask = (torch.rand(T, generator=g, device="cuda") < 0.6).int()
        self.mask[100:150] = 0  # a run without a counted row
        self.mask[7::33] = 0    # rows that one cluster of 33, as many of eight CTAs as fit two an SM, would take
        logp = torch.cat([self._logp(r) for r in self._chunks()])
        self.old = (logp + 0.2 * rnd(T)).float()
        self.old[((logp - self.old).exp()[:, None] - torch.tensor([1 - lo, 1 + hi], device="cuda")).abs().amin(1) < 1e-3] += 0.01
        self.ref = (logp + 0.3 * rnd(T)).float()
        self.adv = rnd(T)
        self.logp = torch.full((T + 1,), 7.0, device="cuda")
        self.out = torch.full((5,), 7.0, device="cuda")
        self.dlog = torch.full((T * V + 8,), 7.0, dtype=torch.bfloat16, device="cuda")
        self.scratch = torch.empty(lst.policy_scratch(T, S), device="cuda")

    def _chunks(self):
        n = max(1, (1 << 25) // self.V)
        return [slice(i, min(self.T, i + n)) for i in range(0, self.T, n)]

    def _logp(self, rows):
        x = self.x[rows].double()
        return x.gather(1, self.y[rows, None].long())[:, 0] - torch.logsumexp(x, 1)

    def run(self):
        lst.k_policy_loss(self.x, self.T, self.V, self.y, self.S, self.adv, self.logp, self.out, self.scratch, dlogits=self.dlog,
                          old_logp=self.old, ref_logp=self.ref, mask=self.mask, clip_lo=self.lo, clip_hi=self.hi,
                          kl_beta=self.beta, norm=lst.POLICY_SEQ_MEAN)

    def check(self):
        from test_gpu_policy import F, U
        on = self.mask != 0
        m = on.double().view(-1, self.S)
        w = (m / m.sum(1, keepdim=True).clamp(min=1) / m.shape[0]).view(-1)
        logp = torch.where(on, torch.cat([self._logp(r) for r in self._chunks()]), 0.0)
        r, A, d = (logp - self.old.double()).exp(), self.adv.double(), self.ref.double() - logp
        cut = r * A > r.clamp(1 - self.lo, 1 + self.hi) * A
        u = torch.where(cut, r.clamp(1 - self.lo, 1 + self.hi) * A, r * A)
        kl = torch.expm1(d) - d
        el = (self.V / 256 + 64) * F + 2.0 ** -21 + 4 * F * (2 * self.x.abs().amax(1).double() + logp.abs())
        e = el + 2.0 ** -20
        assert torch.all(torch.where(on, (self.logp[:self.T] - logp).abs() <= el, self.logp[:self.T] == 0))
        want = torch.stack([w @ torch.where(on, t, 0.0) for t in (self.beta * kl - u, kl, cut.double(), r)])
        size = torch.stack([(r * A).abs() + (1 + self.hi) * A.abs() + self.beta * (torch.expm1(d).abs() + kl), torch.expm1(d).abs() + kl,
                            torch.zeros_like(r), r])
        tol = torch.where(on, size * e, 0.0) @ w + 8 * F * want.abs() + 1e-12
        assert torch.all((self.out[:4].double() - want).abs() <= tol), (self.out, want, tol)
        coef = torch.where(on, w * (torch.where(cut, 0.0, -r * A) - self.beta * torch.expm1(d)), 0.0)[:, None]
        c = torch.where(on, w * ((r * A).abs() + self.beta * (torch.expm1(d).abs() + 1)) * e, 0.0)[:, None]
        for rows in self._chunks():
            p = torch.softmax(self.x[rows].double(), 1)
            y = self.y[rows, None].long()
            g = -coef[rows] * p
            g.scatter_add_(1, y, coef[rows])
            p.scatter_add_(1, y, torch.ones_like(coef[rows]))
            got = self.dlog[:self.T * self.V].view(self.T, self.V)[rows].double()
            assert torch.all((got - g).abs() <= U * g.abs() + c[rows] * p + 1e-37)
        assert torch.all(self.dlog[self.T * self.V:] == 7) and torch.all(self.logp[self.T:] == 7) and torch.all(self.out[4:] == 7)
        assert lst.device_error() == 0


@pytest.mark.parametrize("T,V,S,offset", [
    (1500, 4100, 100, 0), (1500, 4099, 100, 1),     # several short rows a CTA
    (1500, 5000, 100, 0), (1500, 5003, 100, 1),     # either side of the bound of short slices
    (1500, 16384, 50, 0), (1500, 16383, 50, 2),     # several long ones
    (400, 32000, 100, 0), (400, 32003, 100, 0),     # clusters of two, whose rows start anywhere in 16 bytes
    (200, 128256, 40, 0),                           # of eight
    (1320, 80000, 110, 0), (1320, 80001, 110, 3),   # more rows a cluster than its producer reads the scalars of at once
    (160, 200001, 20, 0)])                          # one CTA an SM
def test_policy_many_rows_a_cluster(T, V, S, offset):
    # the ring of half rows, the pairs' parities and the rows' scalars used over and over, counted rows and others in turn
    c = Many(T, V, S, offset)
    c.run()
    torch.cuda.synchronize()
    c.check()
    first = c.out.clone(), c.logp.clone(), c.dlog.clone()
    c.run()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(first, (c.out, c.logp, c.dlog)))
