"""The operators of reinforcement fine-tuning on long sampled answers, as cases to be measured: attention
with a sliding window and sinks (forward, backward) and the clipped policy loss with a KL term (loss,
log-probabilities and the gradient with respect to the logits in one call).

Window attention: key j is visible to query i of the same sequence when j <= i and (i - j < window or
j < sinks). Policy loss: per counted token -min(r A, clip(r) A) + beta k3, r = exp(logp - old_logp),
k3 = exp(ref - logp) - (ref - logp) - 1, weighted by one of three normalisations.
"""
import math

import torch

own = False

TOKEN_MEAN, SEQ_MEAN, FIXED = 0, 1, 2


def _attn(name, op, B, S, hq, hkv, hd, window, sinks):
    return {"name": name, "op": op, "B": B, "S": S, "hq": hq, "hkv": hkv, "hd": hd, "window": window, "sinks": sinks}


def _policy(name, B, S, V, prompt, pad, norm, kl, per_seq):
    return {"name": name, "op": "policy", "B": B, "S": S, "V": V, "prompt": prompt, "pad": pad, "norm": norm, "kl": kl,
            "per_seq": per_seq}


def listed():
    return [
        # the smallest step of the tests: two short sequences, head size 64; the launch counts
        _attn("fwd_small", "fwd", 2, 128, 4, 4, 64, 48, 4),
        # the batch that the benchmark trains on, with a window of half a sequence
        _attn("fwd_batch", "fwd", 4, 512, 32, 8, 128, 256, 4),
        # ragged: five heads a group, a length and a window that end inside a tile, seventeen sinks
        _attn("fwd_ragged", "fwd", 3, 777, 40, 8, 128, 300, 17),
        # one long sampled answer under a window of 1024
        _attn("fwd_long", "fwd", 1, 16384, 32, 8, 128, 1024, 4),
        # the backward of the smallest step
        _attn("bwd_small", "bwd", 2, 128, 4, 4, 64, 48, 4),
        # the backward of the benchmark's batch
        _attn("bwd_batch", "bwd", 4, 512, 32, 8, 128, 256, 4),
        # eight heads a group, odd length, sinks that cross a tile
        _attn("bwd_ragged", "bwd", 2, 1531, 16, 2, 128, 513, 130),
        # the backward of a long answer
        _attn("bwd_long", "bwd", 1, 8192, 32, 8, 128, 1024, 4),
        # the tests' vocabulary: a few short answers, on-policy normalisation over tokens
        _policy("policy_small", 4, 32, 512, 8, 3, TOKEN_MEAN, True, True),
        # an odd vocabulary (rows start unaligned), one sequence without a counted token, per-token advantages
        _policy("policy_odd", 3, 333, 32003, 100, 250, SEQ_MEAN, True, False),
        # the benchmark's batch and vocabulary: prompt half masked
        _policy("policy_batch", 4, 512, 128256, 256, 0, SEQ_MEAN, True, True),
        # eight answers of 512 tokens over the largest vocabulary of the workloads, no reference model
        _policy("policy_long", 8, 512, 151936, 64, 40, TOKEN_MEAN, False, True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))


def draw(rng):
    op = rng.choice(["fwd", "bwd", "policy"])
    if op == "policy":
        B, S = rng.randint(1, 8), _log(rng, 1, 1024)
        V = min(_log(rng, 100, 151936), 8 * 512 * 151936 // (B * S))
        prompt = rng.randint(0, S // 2)
        return {"op": op, "B": B, "S": S, "V": V, "prompt": prompt, "pad": rng.randint(0, max(0, S // 8)),
                "norm": rng.choice([TOKEN_MEAN, SEQ_MEAN, FIXED]), "kl": rng.random() < 0.6, "per_seq": rng.random() < 0.5}
    hq, hkv = rng.choice([(4, 4), (16, 2), (32, 8), (40, 8), (8, 1), (14, 2), (6, 3)])
    hd = rng.choice([64, 128])
    B, S, window = rng.randint(1, 4), _log(rng, 1, 16384), _log(rng, 1, 4096)
    sinks = rng.choice([0, 1, 4, rng.randint(2, 64), rng.randint(65, 200)])
    most = (16384 if op == "fwd" else 8192) * 1028 * 32 * 128
    S = max(1, min(S, most // (B * hq * hd * min(S, window + sinks))))
    return {"op": op, "B": B, "S": S, "hq": hq, "hkv": hkv, "hd": hd, "window": window, "sinks": sinks}


def _counted(c):
    """int32 [B * S]: the positions that count. Sequence b has its prompt in front and b * pad tokens of padding behind."""
    pos = torch.arange(c["S"]).expand(c["B"], -1)
    end = c["S"] - torch.arange(c["B"])[:, None] * c["pad"]
    return ((pos >= c["prompt"]) & (pos < end)).to(torch.int32).reshape(-1)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *shape: torch.randn(*shape, generator=g, device="cuda")  # noqa: E731
    st = {"case": dict(case), "scratch": None}
    if case["op"] == "policy":
        T, V = case["B"] * case["S"], case["V"]
        x = randn(T, V).mul_(2.5)
        # targets as a sampler draws them: one draw of softmax(x) for each row (the exponential race)
        race = torch.empty(T, V, device="cuda").exponential_(generator=g).log_()
        y = torch.sub(x, race, out=race).argmax(-1)
        del race
        logp = x.gather(-1, y[:, None])[:, 0] - torch.logsumexp(x, -1)
        st.update(
            logits=x, targets=y.to(torch.int32), mask=_counted(case).cuda(),
            adv=randn(case["B"] if case["per_seq"] else T), old=logp + 0.15 * randn(T),
            ref=logp + 0.3 * randn(T) if case["kl"] else None, beta=0.04 if case["kl"] else 0.0, lo=0.2, hi=0.28,
            logp=torch.empty(T, device="cuda"), out=torch.empty(4, device="cuda"),
            dlogits=torch.empty(T, V, dtype=torch.bfloat16, device="cuda"))
        return st
    T, hq, hkv, hd = case["B"] * case["S"], case["hq"], case["hkv"], case["hd"]
    dq, dk = hq * hd, hkv * hd
    qkv = randn(T, dq + 2 * dk)
    qkv[:, :dq] *= 1.5
    qkv = qkv.to(torch.bfloat16)  # q, k, v of a fused projection: three column ranges of one matrix
    st.update(qkv=qkv, q=qkv[:, :dq], k=qkv[:, dq:dq + dk], v=qkv[:, dq + dk:],
              o=torch.empty(T, dq, dtype=torch.bfloat16, device="cuda"), lse=torch.empty(T, hq, device="cuda"))
    if case["op"] == "bwd":
        o, lse = _forward(st)
        dqkv = torch.empty(T, dq + 2 * dk, dtype=torch.bfloat16, device="cuda")
        st.update(o=o, lse=lse, dout=randn(T, dq).to(torch.bfloat16), dqkv=dqkv, dq=dqkv[:, :dq],
                  dk=dqkv[:, dq:dq + dk], dv=dqkv[:, dq + dk:])
    return st


def _band(case):
    """Blocks of queries and, for each, the keys that any of them sees: (block rows C, positions [n, K], clamped
    positions, visible [n, C, K])."""
    S, W, s = case["S"], min(case["window"], case["S"]), min(case["sinks"], case["S"])
    C = min(S, 256)
    n = -(-S // C)
    at = lambda a: torch.arange(a, device="cuda")  # noqa: E731
    first = at(n)[:, None] * C - (W - 1)
    pos = torch.cat([at(s).expand(n, s), first + at(C + W - 1)], 1)
    i = (at(n)[:, None] * C + at(C))[:, :, None]
    p = pos[:, None, :]
    early = (at(s + C + W - 1) < s)[None, None, :]
    vis = (p >= 0) & (p <= i) & (i < S) & torch.where(early, p < first[:, :, None], (i - p < W) | (p < s))
    return C, pos.clamp(0, S - 1), vis


def _blocks(x, case, heads, C):
    """[T, heads * hd] as fp32 blocks [B, n, hkv, group * C, hd], rows behind the sequence zero."""
    B, S, hkv, hd = case["B"], case["S"], case["hkv"], case["hd"]
    n, grp = -(-S // C), heads // hkv
    x = torch.nn.functional.pad(x.float().reshape(B, S, heads * hd), (0, 0, 0, n * C - S))
    return x.reshape(B, n, C, hkv, grp, hd).permute(0, 1, 3, 4, 2, 5).reshape(B, n, hkv, grp * C, hd)


def _rows(x, case, C):
    """The inverse of _blocks: [B, n, hkv, group * C, e] to [T, heads * e]."""
    B, S, hkv = case["B"], case["S"], case["hkv"]
    n, grp, e = x.shape[1], x.shape[3] // C, x.shape[4]
    x = x.reshape(B, n, hkv, grp, C, e).permute(0, 1, 4, 2, 3, 5).reshape(B, n * C, hkv * grp * e)
    return x[:, :S].reshape(B * S, hkv * grp * e)


def _keys(x, case, pos):
    """[T, hkv * hd] gathered to fp32 [B, n, hkv, K, hd]."""
    return x.float().reshape(case["B"], case["S"], case["hkv"], case["hd"])[:, pos].transpose(2, 3)


def _scores(st, C, pos, vis):
    c = st["case"]
    s = _blocks(st["q"], c, c["hq"], C) @ _keys(st["k"], c, pos).transpose(-1, -2) * c["hd"] ** -0.5
    return s.masked_fill_(~vis.repeat(1, c["hq"] // c["hkv"], 1)[None, :, None], -math.inf)


def _forward(st):
    c = st["case"]
    C, pos, vis = _band(c)
    s = _scores(st, C, pos, vis)
    m = s.amax(-1, keepdim=True)
    m = torch.where(m > -math.inf, m, 0.0)
    p = torch.exp(s.sub_(m))
    total = p.sum(-1, keepdim=True)
    o = p @ _keys(st["v"], c, pos) / total
    return _rows(o, c, C).to(torch.bfloat16), _rows(m + torch.log(total), c, C)


def _backward(st):
    c = st["case"]
    B, S, hq, hkv, hd = c["B"], c["S"], c["hq"], c["hkv"], c["hd"]
    C, pos, vis = _band(c)
    s = _scores(st, C, pos, vis)
    lse = _blocks(st["lse"], dict(c, hd=1), hq, C)
    p = torch.exp(s.sub_(lse))
    do = _blocks(st["dout"], c, hq, C)
    delta = (do * _blocks(st["o"], c, hq, C)).sum(-1, keepdim=True)
    dv = p.transpose(-1, -2) @ do
    ds = p.mul_(do @ _keys(st["v"], c, pos).transpose(-1, -2) - delta)
    dq = ds @ _keys(st["k"], c, pos) * hd ** -0.5
    dk = ds.transpose(-1, -2) @ _blocks(st["q"], c, hq, C) * hd ** -0.5
    back = lambda d: torch.zeros(B, S, hkv * hd, device="cuda").index_add_(  # noqa: E731
        1, pos.reshape(-1), d.transpose(2, 3).reshape(B, -1, hkv * hd)).reshape(B * S, hkv * hd).to(torch.bfloat16)
    return _rows(dq, c, C).to(torch.bfloat16), back(dk), back(dv)


def _weights(c, mask, dtype):
    m = mask.reshape(c["B"], c["S"]).to(dtype)
    if c["norm"] == SEQ_MEAN:
        return (m / m.sum(1, keepdim=True).clamp(min=1) / c["B"]).reshape(-1)
    return (m / (m.sum().clamp(min=1) if c["norm"] == TOKEN_MEAN else m.numel())).reshape(-1)


def _loss(st):
    c, x, y = st["case"], st["logits"], st["targets"].long()
    on = st["mask"] != 0
    m = x.amax(-1, keepdim=True)
    lse = m[:, 0].double() + torch.exp(x - m).sum(-1, dtype=torch.float64).log()
    logp = torch.where(on, x.gather(-1, y[:, None])[:, 0].double() - lse, 0.0)
    # the token's terms in 64 bits: they are few, and the clip has borders
    w = _weights(c, st["mask"], torch.float64)
    adv = (st["adv"].repeat_interleave(c["S"]) if c["per_seq"] else st["adv"]).double()
    ratio = torch.exp(logp - st["old"].double())
    inner, outer = ratio * adv, ratio.clamp(1 - st["lo"], 1 + st["hi"]) * adv
    slope = torch.where(inner <= outer, -inner, 0.0)
    d = st["ref"].double() - logp if c["kl"] else torch.zeros_like(logp)
    kl = torch.expm1(d) - d
    slope = slope - st["beta"] * torch.expm1(d)
    token = st["beta"] * kl - torch.minimum(inner, outer)
    sums = torch.stack([token, kl, (inner > outer).double(), ratio], 1)
    out = (torch.where(on, w, 0.0)[:, None] * torch.where(on[:, None], sums, 0.0)).sum(0).float()
    coef = torch.where(on, -w * slope, 0.0).float()[:, None]
    grad = torch.exp(x - lse.float()[:, None]).mul_(coef)
    grad.scatter_add_(1, y[:, None], -coef)
    return out, logp.float(), grad.to(torch.bfloat16)


def run(state):
    c = state["case"]
    if own:
        import layer_streamed_qlora_streaming_b200 as lst

        s = torch.cuda.current_stream()
        if c["op"] == "policy":
            T, V = state["logits"].shape
            if state["scratch"] is None:
                state["scratch"] = torch.empty(lst.policy_scratch(T, c["S"]), device="cuda")
            lst.k_policy_loss(state["logits"], T, V, state["targets"], c["S"], state["adv"], state["logp"], state["out"],
                              state["scratch"], dlogits=state["dlogits"], old_logp=state["old"], ref_logp=state["ref"],
                              mask=state["mask"], clip_lo=state["lo"], clip_hi=state["hi"], kl_beta=state["beta"],
                              norm=c["norm"], adv_per_seq=c["per_seq"], stream=s)
            return state["out"], state["logp"], state["dlogits"]
        T, ld = state["q"].shape[0], state["qkv"].shape[1]
        hq, hkv, hd = c["hq"], c["hkv"], c["hd"]
        if c["op"] == "fwd":
            lst.k_attention_window_fwd(state["q"], ld, state["k"], ld, state["v"], ld, state["o"], hq * hd, state["lse"],
                                       T, c["S"], hq, hkv, hd, c["window"], c["sinks"], stream=s)
            return state["o"], state["lse"]
        if state["scratch"] is None:
            state["scratch"] = torch.empty(lst.attention_window_scratch(T, c["S"], hq, hkv, hd, c["window"], c["sinks"]),
                                           device="cuda")
        lst.k_attention_window_bwd(state["q"], ld, state["k"], ld, state["v"], ld, state["o"], hq * hd, state["dout"],
                                   hq * hd, state["lse"].contiguous(), state["scratch"], state["dq"], ld, state["dk"], ld, state["dv"],
                                   ld, T, c["S"], hq, hkv, hd, c["window"], c["sinks"], stream=s)
        return state["dq"], state["dk"], state["dv"]
    return {"fwd": _forward, "bwd": _backward, "policy": _loss}[c["op"]](state)


def work(case):
    if case["op"] == "policy":
        T, V = case["B"] * case["S"], case["V"]
        live = int(_counted(case).sum())
        return {"bytes": live * V * 4 + T * V * 2 + T * 24, "flops": live * V * 6}
    B, S, hq, hkv, hd = case["B"], case["S"], case["hq"], case["hkv"], case["hd"]
    W, s = min(case["window"], S), case["sinks"]
    pairs = W * (W + 1) // 2 + (S - W) * W  # keys of the window
    far = max(0, S - W)  # queries with keys in front of their window: 1, 2, ..., at most s of them are sinks
    pairs += s * (s + 1) // 2 + (far - s) * s if far >= s else far * (far + 1) // 2
    rows = B * S * hd * 2
    if case["op"] == "fwd":
        return {"bytes": rows * (2 * hq + 2 * hkv) + B * S * hq * 4, "flops": 4 * pairs * hd * hq * B}
    return {"bytes": rows * (4 * hq + 4 * hkv) + B * S * hq * 4, "flops": 10 * pairs * hd * hq * B}


def exact(case, seed):
    st = prepare(case, seed)
    f64 = torch.float64
    if case["op"] == "policy":
        outs, logps, grads = torch.zeros(4, dtype=f64, device="cuda"), [], []
        B, S, mask = case["B"], case["S"], st["mask"].tolist()
        total, each = sum(mask), [sum(mask[b * S:(b + 1) * S]) for b in range(B)]
        adv, old = st["adv"].tolist(), st["old"].tolist()
        ref = st["ref"].tolist() if case["kl"] else None
        for t0 in range(0, B * S, 256):
            x = st["logits"][t0:t0 + 256].double()
            lsm = torch.log_softmax(x, -1)
            got = lsm.gather(1, st["targets"][t0:t0 + 256].long()[:, None])[:, 0].tolist()
            coefs = []
            for r, lp in enumerate(got):
                t = t0 + r
                if not mask[t]:
                    got[r] = 0.0
                    coefs.append(0.0)
                    continue
                w = 1.0 / {TOKEN_MEAN: total, SEQ_MEAN: B * each[t // S], FIXED: B * S}[case["norm"]]
                a, rho = adv[t // S if case["per_seq"] else t], math.exp(lp - old[t])
                # the clip takes effect where it lowers the surrogate
                cut = rho > 1 + st["hi"] if a > 0 else rho < 1 - st["lo"] if a < 0 else False
                value = (1 + st["hi"] if a > 0 else 1 - st["lo"]) * a if cut else rho * a
                delta = ref[t] - lp if ref else 0.0
                k3 = math.expm1(delta) - delta
                outs += w * torch.tensor([st["beta"] * k3 - value, k3, float(cut), rho], dtype=f64, device="cuda")
                coefs.append(w * ((0.0 if cut else -rho * a) - st["beta"] * math.expm1(delta)))
            coef = torch.tensor(coefs, dtype=f64, device="cuda")[:, None]
            grad = -coef * lsm.exp_()
            grad[torch.arange(len(x), device="cuda"), st["targets"][t0:t0 + 256].long()] += coef[:, 0]
            logps.append(torch.tensor(got, dtype=f64, device="cuda"))
            grads.append(grad.float())  # the gradient is held to 8 bits: 24 are enough here, and half the memory
        return outs, torch.cat(logps), torch.cat(grads)
    B, S, hq, hkv, hd = case["B"], case["S"], case["hq"], case["hkv"], case["hd"]
    grp = hq // hkv
    # one sequence and head at a time, dense over its keys
    q, k, v = (st[n].reshape(B, S, -1, hd) for n in "qkv")
    j = torch.arange(S, device="cuda")
    o = torch.empty(B, S, hq, hd, dtype=f64, device="cuda")
    lse = torch.empty(B, S, hq, dtype=f64, device="cuda")
    dq, dk, dv = (torch.zeros(B, S, h, hd, dtype=f64, device="cuda") for h in (hq, hkv, hkv))
    for b in range(B):
        for h in range(hq):
            kk, vv = k[b, :, h // grp].double(), v[b, :, h // grp].double()
            for i0 in range(0, S, 4096):
                i = j[i0:i0 + 4096, None]
                n = int(i[-1]) + 1  # keys behind the block's last query are not seen
                hidden = (j[:n] > i) | ((i - j[:n] >= case["window"]) & (j[:n] >= case["sinks"]))
                qq = q[b, i0:i0 + 4096, h].double()
                z = (qq @ kk[:n].T / math.sqrt(hd)).masked_fill_(hidden, -math.inf)
                lse[b, i0:i0 + 4096, h] = torch.logsumexp(z, -1)
                prob = torch.softmax(z, -1)
                oo = prob @ vv[:n]
                o[b, i0:i0 + 4096, h] = oo
                if case["op"] == "bwd":
                    dd = st["dout"].reshape(B, S, hq, hd)[b, i0:i0 + 4096, h].double()
                    dz = prob * (dd @ vv[:n].T - (dd * oo).sum(-1, keepdim=True)) / math.sqrt(hd)
                    dq[b, i0:i0 + 4096, h] = dz @ kk[:n]
                    dk[b, :n, h // grp] += dz.T @ qq
                    dv[b, :n, h // grp] += prob.T @ dd
    if case["op"] == "fwd":
        return o.reshape(B * S, -1), lse.reshape(B * S, -1)
    return dq.reshape(B * S, -1), dk.reshape(B * S, -1), dv.reshape(B * S, -1)
