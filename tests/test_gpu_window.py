"""Attention under a sliding window with sinks on the GPU, against the formula in 64 bits.

Tolerances, elementwise, counted from the roundings that the operator documents. Inputs are exact in
bf16; u = 2^-8 is bf16's half step relative to a value (torch.finfo(torch.bfloat16).eps / 2), f = 2^-24
that of fp32.
  scores: fp32 sums of hd products: |ds| <= es = (hd + 4) f max_j (scale sum_c |q_c k_c|); the
    exponentials are within 2 ulp and the running sums of at most S terms add S f.
    With e = es + (S + 16) f + 2^-21:
  o: P rounded to bf16 before the product (u sum P|v|) and o rounded once (u |o|), on top of e:
    u |o| + (u (1 + u) + 2 e) sum P |v|;      lse: e + 2 f |lse|.
  backward, with the forward's own o and lse (the reference takes D = do . o from them too):
    dP and D are fp32 sums of hd products: ed = (2 hd + 8) f max(sum |do||v|, sum |do||o|);
    dS = P (dP - D) has error P ed + e |dS| and is rounded to bf16 (u |dS|), P to bf16 in dv:
    dq: u |dq| + scale sum_j [(u (1 + u) + 2 e) |dS| + P ed] |k|, dk the same with q over (h, i);
    dv: u |dv| + (u (1 + u) + 2 e) sum P |do|.
The fp32 sums of the products over keys (at most 2 S terms of the magnitudes summed above) are below
2 S f of them: counted in e."""
import numpy as np
import pytest

from oracle import model as M

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
lst = pytest.importorskip("layer_streamed_qlora_streaming_b200")

U, F = 2.0 ** -8, 2.0 ** -24


@pytest.fixture(autouse=True, scope="module")
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA device")


class Case:
    """Inputs as column ranges of a fused q/k/v matrix with a padded row stride, outputs the same way,
    everything behind the outputs filled with a pattern that has to stay."""

    def __init__(self, B, S, hq, hkv, hd, window, sinks, seed=0, pad=8, scale=1.0):
        self.B, self.S, self.hq, self.hkv, self.hd, self.window, self.sinks = B, S, hq, hkv, hd, window, sinks
        self.T, self.cq, self.ck = B * S, hq * hd, hkv * hd
        self.ld, self.ldo = self.cq + 2 * self.ck + pad, self.cq + pad
        g = torch.Generator(device="cuda").manual_seed(seed * 1000003 + S * 131 + hq * 17 + window)
        rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
        self.qkv = (rnd(self.T, self.ld) * scale).bfloat16()
        self.dout = rnd(self.T, self.ldo).bfloat16()
        self.q, self.k, self.v = self.cols(self.qkv)
        self.o = torch.full((self.T, self.ldo), 7.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((self.T + 1, hq), 7.0, device="cuda")
        self.dqkv = torch.full((self.T, self.ld), 7.0, dtype=torch.bfloat16, device="cuda")
        self.dq, self.dk, self.dv = self.cols(self.dqkv)
        n = lst.attention_window_scratch(self.T, S, hq, hkv, hd, window, sinks)
        self.scratch = torch.full((n + 4,), 7.0, device="cuda")
        self.n = n

    def cols(self, x):
        return x[:, :self.cq], x[:, self.cq:self.cq + self.ck], x[:, self.cq + self.ck:self.cq + 2 * self.ck]

    def forward(self, stream=None):
        lst.k_attention_window_fwd(self.q, self.ld, self.k, self.ld, self.v, self.ld, self.o, self.ldo, self.lse, self.T,
                                   self.S, self.hq, self.hkv, self.hd, self.window, self.sinks, stream=stream)

    def backward(self, stream=None):
        lst.k_attention_window_bwd(self.q, self.ld, self.k, self.ld, self.v, self.ld, self.o, self.ldo, self.dout, self.ldo,
                                   self.lse, self.scratch, self.dq, self.ld, self.dk, self.ld, self.dv, self.ld, self.T,
                                   self.S, self.hq, self.hkv, self.hd, self.window, self.sinks, stream=stream)

    def untouched(self):
        assert torch.all(self.o[:, self.cq:] == 7) and torch.all(self.dqkv[:, self.cq + 2 * self.ck:] == 7)
        assert torch.all(self.lse[self.T:] == 7) and torch.all(self.scratch[self.n:] == 7)

    def heads(self, x, n):
        return x.double().reshape(self.B, self.S, n, self.hd).transpose(1, 2)

    def check(self, backward=True):
        f64, S, hd, grp = torch.float64, self.S, self.hd, self.hq // self.hkv
        vis = torch.from_numpy(M.visible(S, self.window, self.sinks)).cuda()
        q = self.heads(self.q, self.hq)
        k, v = (self.heads(x, self.hkv).repeat_interleave(grp, 1) for x in (self.k, self.v))
        scale = hd ** -0.5
        s = (q @ k.transpose(-1, -2) * scale).masked_fill(~vis, -np.inf)
        lse = torch.logsumexp(s, -1)
        P = torch.softmax(s, -1)
        e = ((hd + 4) * F * scale * (q.abs() @ k.abs().transpose(-1, -2)).masked_fill(~vis, 0).amax(-1, keepdim=True)
             + (3 * S + 16) * F + 2.0 ** -21)
        got_o = self.heads(self.o[:, :self.cq], self.hq)
        got_l = self.lse[:self.T].double().reshape(self.B, S, self.hq).transpose(1, 2)

        def within(name, got, ref, tol):
            off = ((got - ref).abs() / tol.clamp(min=1e-300)).max().item()
            assert off <= 1.0, (name, off)

        o = P @ v
        within("o", got_o, o, U * o.abs() + (U * (1 + U) + 2 * e) * (P @ v.abs()))
        within("lse", got_l, lse, e[..., 0] + 2 * F * lse.abs())
        if not backward:
            return
        do = self.heads(self.dout[:, :self.cq], self.hq)
        P = torch.exp(s - got_l[..., None])
        D = (do * got_o).sum(-1, keepdim=True)
        dP = do @ v.transpose(-1, -2)
        dS = P * (dP - D)
        abs_d = (do.abs() * got_o.abs()).sum(-1, keepdim=True)
        ed = (2 * hd + 8) * F * torch.maximum((do.abs() @ v.abs().transpose(-1, -2)).masked_fill(~vis, 0).amax(-1, keepdim=True), abs_d)
        off_dS = (U * (1 + U) + 2 * e) * dS.abs() + P * ed
        shared = lambda x: x.reshape(self.B, self.hkv, grp, S, hd).sum(2)  # noqa: E731
        dq = scale * dS @ k
        within("dq", self.heads(self.dq, self.hq), dq, U * dq.abs() + scale * off_dS @ k.abs() + 1e-30)
        dk = shared(scale * dS.transpose(-1, -2) @ q)
        within("dk", self.heads(self.dk, self.hkv), dk, U * dk.abs() + shared(scale * off_dS.transpose(-1, -2) @ q.abs()) + 1e-30)
        dv = shared(P.transpose(-1, -2) @ do)
        within("dv", self.heads(self.dv, self.hkv), dv,
               U * dv.abs() + shared(((U * (1 + U) + 2 * e) * P).transpose(-1, -2) @ do.abs()) + 1e-30)
        assert lst.device_error() == 0


SHAPES = [
    # B, S, hq, hkv, hd, window, sinks
    (1, 1, 1, 1, 64, 1, 0),            # one token
    (3, 1, 4, 1, 128, 5, 3),           # sequences of one token
    (2, 7, 4, 2, 128, 3, 2),
    (1, 64, 3, 3, 64, 1, 0),           # every row sees itself alone
    (2, 128, 4, 4, 64, 48, 4),         # the smallest step
    (2, 129, 8, 2, 128, 64, 1),        # one row behind a tile
    (1, 127, 2, 2, 128, 127, 0),       # causal, one row short of a tile
    (1, 300, 5, 1, 128, 300, 0),       # causal through window = S, five heads a group
    (2, 257, 2, 2, 128, 1 << 30, 1 << 30),  # a window and sinks far past S
    (2, 391, 7, 1, 64, 100, 130),      # sinks that cross a tile, seven heads a group
    (1, 640, 4, 1, 128, 17, 300),      # more sinks than window
    (1, 512, 16, 2, 128, 128, 0),      # window of one tile, no sinks
    (1, 513, 16, 1, 64, 129, 1),       # sixteen heads a group
    (1, 1025, 3, 3, 64, 129, 64),
    (1, 700, 12, 4, 128, 200, 699),    # every key a sink
    (1, 700, 2, 1, 128, 5, 128),       # sinks of one tile
    (1, 1500, 2, 1, 128, 256, 4),
    (1, 2048, 2, 2, 64, 31, 33),
    (4, 96, 32, 8, 128, 40, 16),
    (37, 33, 2, 1, 64, 9, 5),          # many short sequences
    # more key tiles than CTAs: whole ones in rounds, the rest cut into shares, some of them empty
    (22, 1, 16, 8, 128, 1, 0),
    (19, 1, 24, 8, 64, 128, 0),
    (39, 1, 16, 8, 64, 128, 0),
    (11, 129, 7, 7, 64, 128, 0),
    (16, 300, 16, 8, 128, 200, 130),
]


@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s)))
def test_window_attention(shape):
    c = Case(*shape)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check()
    c.untouched()


def test_window_attention_peaked_scores():
    # scores of +-200: the running maximum moves far between blocks, most probabilities vanish
    c = Case(1, 700, 4, 2, 128, 200, 4, scale=5.0)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    c.check()


def test_window_of_s_equals_causal_attention():
    c = Case(2, 333, 8, 2, 128, 333, 0, pad=0)
    c.forward()
    o = torch.empty_like(c.o)
    lse = torch.empty_like(c.lse[:c.T])
    lst.k_attention_fwd(c.q, c.ld, c.k, c.ld, c.v, c.ld, o, c.ldo, lse, c.T, c.S, c.hq, c.hkv, c.hd)
    torch.cuda.synchronize()
    # each within u (|o| + sum P|v|) of the formula; sum P|v| is below max |v|
    assert (o.float() - c.o.float()).abs().max() <= 2 * 2 * U * c.v.float().abs().max()
    assert (lse - c.lse[:c.T]).abs().max() <= 1e-4


def test_window_gradients_match_differences():
    # L = sum(o * dout): central differences of the operator's own forward in fp32-visible steps of one
    # input element are dominated by o's bf16 rounding, so the differences are taken of the formula in
    # 64 bits at the operator's inputs, and the operator's gradients are held to them
    c = Case(1, 40, 2, 1, 64, 9, 3, seed=5)
    c.forward()
    c.backward()
    torch.cuda.synchronize()
    vis = torch.from_numpy(M.visible(c.S, c.window, c.sinks)).cuda()
    q, k, v = (c.heads(x, n) for x, n in ((c.q, 2), (c.k, 1), (c.v, 1)))
    do = c.heads(c.dout[:, :c.cq], 2)

    def loss(q, k, v):
        s = (q @ k.expand(-1, 2, -1, -1).transpose(-1, -2) / 8).masked_fill(~vis, -np.inf)
        return (torch.softmax(s, -1) @ v.expand(-1, 2, -1, -1) * do).sum().item()

    h = 1e-4
    for which, (x, grad) in enumerate(((q, c.heads(c.dq, 2)), (k, c.heads(c.dk, 1)), (v, c.heads(c.dv, 1)))):
        for at in ((0, 0, 0, 5), (0, x.shape[1] - 1, 17, 63), (0, 0, 39, 0)):
            f = []
            for sign in (1, -1):
                y = x.clone()
                y[at] += sign * h
                f.append(loss(*[y if n == which else z for n, z in enumerate((q, k, v))]))
            # gradients of order one: bf16 roundings of dS / P over at most 40 x 2 terms
            assert grad[at].item() == pytest.approx((f[0] - f[1]) / (2 * h), abs=80 * U)


def test_window_neighbouring_sequences_do_not_mix():
    # NaN in the other sequence's rows (and behind the last one) must not reach this one
    c = Case(3, 150, 2, 1, 128, 60, 4)
    clean = Case(3, 150, 2, 1, 128, 60, 4)
    c.qkv[150:300] = float("nan")
    c.dout[150:300] = float("nan")
    for x in (clean, c):
        x.forward()
        x.backward()
    torch.cuda.synchronize()
    for a, b in ((c.o, clean.o), (c.dqkv, clean.dqkv)):
        for rows in (slice(0, 150), slice(300, 450)):
            assert torch.equal(a[rows], b[rows])


def test_window_deterministic_streams_and_graphs():
    cs = [Case(1, 900, 8, 2, 128, 200, 4, seed=s) for s in range(2)]
    want = []
    for c in cs:
        c.forward()
        c.backward()
    torch.cuda.synchronize()
    want = [(c.o.clone(), c.lse.clone(), c.dqkv.clone()) for c in cs]
    # two calls at once on two streams, each with its own scratch
    streams = [torch.cuda.Stream() for _ in cs]
    for c, s in zip(cs, streams):
        c.o.zero_(), c.lse.zero_(), c.dqkv.zero_()
        s.wait_stream(torch.cuda.current_stream())
    for c, s in zip(cs, streams):
        c.forward(s)
        c.backward(s)
    torch.cuda.synchronize()
    for c, (o, lse, g) in zip(cs, want):
        assert torch.equal(c.o[:, :c.cq], o[:, :c.cq]) and torch.equal(c.lse[:c.T], lse[:c.T])
        assert torch.equal(c.dqkv[:, :c.cq + 2 * c.ck], g[:, :c.cq + 2 * c.ck])
    # captured, replayed on changed inputs
    c = cs[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.forward(torch.cuda.current_stream())
        c.backward(torch.cuda.current_stream())
    c.qkv.copy_(cs[1].qkv)
    c.dout.copy_(cs[1].dout)
    graph.replay()
    torch.cuda.synchronize()
    o, lse, g = want[1]
    assert torch.equal(c.o[:, :c.cq], o[:, :c.cq]) and torch.equal(c.dqkv[:, :c.cq + 2 * c.ck], g[:, :c.cq + 2 * c.ck])
    assert lst.device_error() == 0
