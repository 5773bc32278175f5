"""Linear attention over pooled states, and the sampling that ends a speculative step, as measured cases.

A hybrid model runs linear-attention layers with a fixed decay for each head over the same kind of state pool as its Gated
DeltaNet layers.  A speculative step verifies drafts on those states, turns the head's logits into probabilities, accepts
drafts and samples one token, and commits the accepted prefix:

* ``decode``   S = g S + v k^T, o = scale S q for a token of each lane, the new state into the lane's slot;
* ``verify``   several draft tokens from read-only states, with or without the state after every token;
* ``commit``   the accepted tokens again, without outputs, the new state into the lane's slot;
* ``prefill``  packed prompts of any lengths from a cached state or from zero;
* ``probs``    softmax of logits with a temperature for each lane (0: the first of the largest);
* ``accept``   drafts against the target's probabilities with given random numbers, and the token after them.

States are read from one slot and written to another (a cached prefix stays), so a pass can be repeated.  ``run`` computes
the plain form in elementary torch operations, or calls the framework where ``own``.
"""
import math

import torch

own = False

STATE_OPS = ("decode", "verify", "commit", "prefill")
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def listed():
    return [
        # the smallest call: one lane, one token, its latency
        dict(name="decode B1 D128", op="decode", B=1, T=1, HK=16, HV=32, DK=128, DV=128, io="bf16", state="bf16", padded=False),
        # an ordinary decode batch on fp32 states
        dict(name="decode B64 f32", op="decode", B=64, T=1, HK=16, HV=32, DK=128, DV=128, io="bf16", state="f32", padded=False),
        # a verify step of 4 tokens with the state after every token kept for the commit
        dict(name="verify B128 T4 states", op="verify", B=128, T=4, HK=16, HV=32, DK=128, DV=128, io="bf16", state="bf16",
             padded=False, kept=True),
        # a verify step of 8 tokens, a tenth of the lanes padded, nothing kept
        dict(name="verify B256 T8 padded", op="verify", B=256, T=8, HK=16, HV=32, DK=128, DV=128, io="bf16", state="bf16",
             padded=True, kept=False),
        # the commit of such a step: the accepted tokens run again
        dict(name="commit B256 T8 padded", op="commit", B=256, T=8, HK=16, HV=32, DK=128, DV=128, io="bf16", state="bf16",
             padded=True),
        # 8 prompts of 8192 tokens
        dict(name="prefill B8 L8192", op="prefill", B=8, lo=8192, hi=8192, HK=16, HV=32, DK=128, DV=128, io="bf16",
             state="bf16", padded=False),
        # one long prompt: few heads to spread over the GPU
        dict(name="prefill B1 L16384", op="prefill", B=1, lo=16384, hi=16384, HK=16, HV=16, DK=128, DV=128, io="bf16",
             state="f32", padded=False),
        # a packed batch of prompts of odd lengths, narrow heads
        dict(name="prefill B32 ragged D64", op="prefill", B=32, lo=17, hi=2048, HK=8, HV=32, DK=64, DV=64, io="bf16",
             state="f32", padded=True),
        # the logits of a verify step of 4 tokens over a large vocabulary
        dict(name="probs B128 T4 V131072", op="probs", B=128, T=4, V=131072, io="bf16", masked=0.0, pad=0),
        # one token's logits in fp32, an odd vocabulary in rows with room behind, half of it forbidden
        dict(name="probs B1 V50001 f32", op="probs", B=1, T=1, V=50001, io="f32", masked=0.5, pad=31),
        # the drafts of 256 lanes against the target, a tenth of the lanes padded
        dict(name="accept B256 T8 V131072", op="accept", B=256, T=8, V=131072, padded=True, probs=True),
        # one lane, drafts taken greedily (no draft probabilities), an odd vocabulary
        dict(name="accept B1 T4 V50001", op="accept", B=1, T=4, V=50001, padded=False, probs=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("decode", "verify", "commit", "prefill", "prefill", "probs", "accept"))
    if op == "probs":
        V = _log(rng, 1000, 200000)
        T = rng.randint(1, 8)
        return dict(op=op, B=_log(rng, 1, max(1, min(512, (1 << 26) // (V * T)))), T=T, V=V, io=rng.choice(("f32", "bf16")),
                    masked=rng.choice((0.0, 0.0, 0.5, 0.99)), pad=rng.choice((0, 0, 1, 64)))
    if op == "accept":
        V = _log(rng, 1000, 200000)
        T = rng.randint(1, 16)
        return dict(op=op, B=_log(rng, 1, max(1, min(512, (1 << 27) // (V * T)))), T=T, V=V, padded=rng.random() < 0.3,
                    probs=T > 1 and rng.random() < 0.7)
    HK = rng.choice((1, 2, 3, 4, 8, 16))
    HV = HK * rng.choice((1, 2, 3, 4))
    rare = rng.random() < 0.25
    DK = rng.choice((16, 32, 256)) if rare else rng.choice((64, 128))
    DV = rng.choice((DK, DK, 64, 128, 96, 40, 33))
    c = dict(op=op, HK=HK, HV=HV, DK=DK, DV=DV, io="f32" if rng.random() < 0.2 else "bf16", state=rng.choice(("f32", "bf16")),
             padded=rng.random() < 0.3)
    if op == "prefill":
        plain = DK in (64, 128) and c["io"] == "bf16"
        hi = _log(rng, 1, 8192 if plain else 1024)
        most = max(1, min(64, (1 << 21 if plain else 1 << 18) // (hi * HV)))
        return dict(c, B=_log(rng, 1, most), lo=rng.choice((hi, max(1, hi // 16))), hi=hi)
    most = max(1, min(256, (1 << 27) // (HV * DK * DV)))
    c.update(B=_log(rng, 1, most), T=1 if op == "decode" and rng.random() < 0.7 else rng.randint(1, 16))
    if op == "verify":
        c["kept"] = rng.random() < 0.4
        if c["kept"]:
            c["B"] = max(1, c["B"] // c["T"])
    return c


# ---- inputs ----------------------------------------------------------------------------------------------
def _lengths(case, gen):
    """Tokens of each prompt, the same ones for every seed in an order that the seed gives."""
    mine = torch.Generator().manual_seed(case["B"] * 1000003 + case["hi"] * 101 + case["HV"])
    n = torch.randint(case["lo"], case["hi"] + 1, (case["B"],), generator=mine)
    if case["B"] > 4:
        n[1] = 0  # a prompt without tokens
    return n[torch.randperm(case["B"], generator=gen)]


def _softmax(x):
    x = torch.exp(x - x.amax(-1, keepdim=True))
    return x / x.sum(-1, keepdim=True)


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape):
        return torch.randn(shape, generator=gen, device="cuda")

    st = dict(case)
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    B = case["B"]
    if case["op"] in ("probs", "accept"):
        T, V = case["T"], case["V"]
        x = normal(B, T, V).mul_(2.5)
        if case["op"] == "probs":
            if case["masked"] > 0:
                x.masked_fill_(torch.rand((B, T, V), generator=gen, device="cuda") < case["masked"], -math.inf)
            wide = torch.zeros((B, T, V + case["pad"]), dtype=TYPES[case["io"]], device="cuda")
            wide[..., :V] = x
            temp = 0.3 + torch.rand(B, generator=host)
            temp[::5] = 0.0 if B > 1 else 0.7  # lanes that decode greedily sit among the others
            st.update(logits=wide[..., :V], temperature=temp.cuda(),
                      out=torch.zeros((B, T, V), dtype=torch.float32, device="cuda"))
            return st
        # the draft model's logits are the target's and an error
        y = x[:, : T - 1] + 0.7 * normal(B, T - 1, V)
        if case["probs"]:
            race = torch.empty_like(y).exponential_(generator=gen)
            st["draft_probs"] = _softmax(y)
            st["drafts"] = (st["draft_probs"] / race).argmax(-1).to(torch.int32)
            del race
        else:
            st["draft_probs"], st["drafts"] = None, y.argmax(-1).to(torch.int32)
        del y
        st["probs_in"] = _softmax(x)
        index = torch.arange(B, dtype=torch.int32)
        if case["padded"]:
            index[torch.randperm(B, generator=host)[: B // 10]] = -1
        st.update(index=index.cuda(), u=torch.rand((B, T), generator=gen, device="cuda"),
                  accept_len=torch.zeros(B, **i32), tokens=torch.zeros((B, T), **i32))
        return st
    HK, HV, DK, DV, io, state = (case[n] for n in ("HK", "HV", "DK", "DV", "io", "state"))
    slots = 2 * B + 3
    order = torch.randperm(slots, generator=host)[: 2 * B].to(torch.int32)
    read, write = order[:B].clone(), order[B:].clone()
    if case["padded"]:
        off = torch.randperm(B, generator=host)[: B // 10]
        read[off], write[off] = -1, -1
    st["pool"] = (0.5 * normal(slots, HV, DV, DK)).to(TYPES[state])
    # slopes in powers of two over the heads, as fixed decays are chosen, and some spread
    slope = torch.exp2(-8.0 * (torch.arange(HV) + 1) / HV)
    st["log_decay"] = (-slope * (0.75 + 0.5 * torch.rand(HV, generator=host))).cuda()
    st.update(read=read.cuda(), write=write.cuda(), scale=DK ** -0.5)
    if case["op"] == "prefill":
        n = _lengths(case, host)
        cu = torch.zeros(B + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(n, 0)
        N = int(cu[-1]) + 5  # a buffer with room behind the last prompt
        has = torch.randint(0, 2, (B,), generator=host)
        st.update(N=N, L=int(n.max()), cu=cu.to(**i32), has=has.to(**i32))
        lead = (N,)
    else:
        lead = (B, case["T"])
        st["accept_len"] = torch.randint(1, case["T"] + 1, (B,), generator=host).to(**i32)
    st["q"] = normal(*lead, HK, DK).to(TYPES[io])
    st["k"] = normal(*lead, HK, DK).to(TYPES[io])
    st["v"] = normal(*lead, HV, DV).to(TYPES[io])
    st["o"] = torch.zeros((*lead, HV, DV), dtype=TYPES[io], device="cuda")
    st["states"] = None
    if case.get("kept"):
        st["states"] = torch.zeros((B, case["T"], HV, DV, DK), dtype=TYPES[state], device="cuda")
    return st


# ---- the plain forms ---------------------------------------------------------------------------------------
def _power(log_decay, e):
    """g^e for every head and exponent (e >= 0) from 64-bit angles; g^0 is 1."""
    x = log_decay.double().view(-1, *[1] * e.dim()) * e.double()
    return torch.where(e == 0, torch.ones_like(x), torch.exp(x)).float()


def _plain_linear(st, S, q, k, v, n, outputs, chunk=64):
    """The recurrence of lanes [B, L, ...] with n tokens each from states S [B, HV, DV, DK], a chunk of tokens at a time."""
    B, L, HK, DK = k.shape
    HV, DV = v.shape[2:]
    G = HV // HK
    out = []
    for c in range(0, L, chunk):
        C = min(chunk, L - c)
        t = torch.arange(C, device=k.device)
        here = (n - c).clamp(0, C)  # tokens of each lane in this chunk
        kc = k[:, c:c + C].float().transpose(1, 2).repeat_interleave(G, 1)  # [B, HV, C, DK]
        vc = v[:, c:c + C].float().transpose(1, 2)
        if outputs:
            qc = q[:, c:c + C].float().transpose(1, 2).repeat_interleave(G, 1)
            far = t[:, None] - t[None, :]
            w = _power(st["log_decay"], far.clamp(min=0)) * (far >= 0)
            a = torch.matmul(qc, kc.transpose(-1, -2)) * w
            first = _power(st["log_decay"], t + 1)[None, :, :, None]
            o = torch.matmul(a, vc) + first * torch.matmul(qc, S.transpose(-1, -2))
            out.append((o * st["scale"]).transpose(1, 2))
        left = here[:, None] - 1 - t  # steps between a token and its lane's last one here
        w = _power(st["log_decay"], left.clamp(min=0)).transpose(0, 1) * (left >= 0)[:, None]
        last = _power(st["log_decay"], here).transpose(0, 1)[..., None, None]
        S = last * S + torch.matmul((vc * w.unsqueeze(-1)).transpose(-1, -2), kc)
    return (torch.cat(out, 1) if outputs else None), S


def _plain_states(st):
    read, write, pool, op = st["read"].long(), st["write"].long(), st["pool"], st["op"]
    act = torch.nonzero(read >= 0).squeeze(-1)
    S = pool[read[act]].float()
    if op == "prefill":
        cu = st["cu"].long()
        n = (cu[1:] - cu[:-1])[act]
        t = torch.arange(st["L"], device=cu.device)
        at = (cu[:-1][act, None] + t).clamp(max=st["N"] - 1)
        here = t < n[:, None]
        S = S * (st["has"][act] != 0)[:, None, None, None]
        o, S = _plain_linear(st, S, st["q"][at], st["k"][at], st["v"][at], n, True)
        res = torch.zeros_like(st["o"])
        res[at[here]] = o[here].to(res.dtype)
        pool[write[act]] = S.to(pool.dtype)
        return [res, pool]
    k, v = st["k"][act], st["v"][act]
    if op == "commit":
        S = _plain_linear(st, S, None, k, v, st["accept_len"].long()[act], False)[1]
        pool[write[act]] = S.to(pool.dtype)
        return [pool]
    q = st["q"][act]
    n = torch.full_like(act, st["T"])
    o, last = _plain_linear(st, S, q, k, v, n, True)
    res = torch.zeros_like(st["o"])
    res[act] = o.to(res.dtype)
    if op == "decode":
        pool[write[act]] = last.to(pool.dtype)
        return [res, pool]
    if st["states"] is None:
        return [res]
    states = torch.zeros_like(st["states"])
    for t in range(st["T"]):
        S = _plain_linear(st, S, None, k[:, t:t + 1], v[:, t:t + 1], torch.ones_like(n), False)[1]
        states[act, t] = S.to(states.dtype)
    return [res, states]


def _first(hit):
    """The lowest index with a truth value along the last axis (its length where there is none)."""
    V = hit.shape[-1]
    i = torch.arange(V, device=hit.device)
    return torch.where(hit, i, torch.full_like(i, V)).amin(-1)


def _plain_probs(st):
    x = st["logits"].float()
    temp = st["temperature"].float()[:, None, None]
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), torch.zeros_like(top), top)  # a row without any entry
    p = torch.exp((x - top) / torch.where(temp > 0, temp, torch.ones_like(temp)))
    s = p.sum(-1, keepdim=True)
    p = p / torch.where(s > 0, s, torch.ones_like(s))
    i = torch.arange(x.shape[-1], device=x.device)
    greedy = (i == _first((x == top) & torch.isfinite(x)).unsqueeze(-1)).float()
    return [torch.where(temp > 0, p, greedy)]


def _plain_accept(st):
    B, T, V = st["B"], st["T"], st["V"]
    p, drafts, u, q = st["probs_in"], st["drafts"].long(), st["u"].double(), st["draft_probs"]
    lane = torch.arange(B, device=p.device)
    px = p[:, : T - 1].gather(-1, drafts.unsqueeze(-1)).squeeze(-1).double()
    qx = torch.ones_like(px) if q is None else q.gather(-1, drafts.unsqueeze(-1)).squeeze(-1).double()
    good = u[:, : T - 1] * qx < px
    n = torch.cumprod(good.long(), 1).sum(1)
    row = p[lane, n].double()
    refused = n < T - 1
    if T > 1:
        at = n.clamp(max=T - 2)
        if q is None:
            other = (torch.arange(V, device=p.device) == drafts[lane, at][:, None]).double()
        else:
            other = q[lane, at].double()
        r = (row - other * refused[:, None]).clamp(min=0)
    else:
        r = row
    r = torch.where(r.sum(-1, keepdim=True) > 0, r, row)
    upto = torch.cumsum(r, -1)
    token = _first((upto > u[:, -1:] * upto[:, -1:]) & (r > 0))
    tokens = torch.full((B, T), -1, dtype=torch.long, device=p.device)
    t = torch.arange(T, device=p.device)
    if T > 1:
        tokens[:, : T - 1] = torch.where(t[: T - 1] < n[:, None], drafts, tokens[:, : T - 1])
    tokens[lane, n] = token
    act = (st["index"] >= 0)
    return [torch.where(act, n + 1, torch.zeros_like(n)).to(torch.int32),
            torch.where(act[:, None], tokens, torch.zeros_like(tokens)).to(torch.int32)]


def run(st):
    op = st["op"]
    if not own:
        return _plain_states(st) if op in STATE_OPS else _plain_probs(st) if op == "probs" else _plain_accept(st)
    import gated_deltanet_linear_mtp_gb300 as gdn
    if op == "probs":
        gdn.gdn_token_probs(st["logits"], st["temperature"], st["out"], err_word=st["err"])
        return [st["out"]]
    if op == "accept":
        gdn.gdn_draft_accept(st["probs_in"], st["drafts"], st["u"], st["index"], st["accept_len"], st["tokens"],
                             draft_probs=st["draft_probs"], err_word=st["err"])
        return [st["accept_len"], st["tokens"]]
    if op == "prefill":
        if "workspace" not in st:
            st["workspace"] = gdn.linear_prefill_workspace(st["N"], st["B"], st["HV"], st["DK"], st["DV"])
        gdn.gdn_linear_prefill(st["q"], st["k"], st["v"], st["log_decay"], st["pool"], st["read"], st["cu"], st["o"],
                               st["workspace"], has_initial_state=st["has"], out_indices=st["write"], err_word=st["err"],
                               scale=st["scale"])
        return [st["o"], st["pool"]]
    if op == "commit":
        gdn.gdn_linear_commit(st["k"], st["v"], st["log_decay"], st["pool"], st["read"], st["accept_len"],
                              out_indices=st["write"], err_word=st["err"])
        return [st["pool"]]
    if op == "decode":
        gdn.gdn_linear_decode(st["q"], st["k"], st["v"], st["log_decay"], st["pool"], st["read"], st["o"],
                              out_indices=st["write"], err_word=st["err"], scale=st["scale"])
        return [st["o"], st["pool"]]
    gdn.gdn_linear_verify(st["q"], st["k"], st["v"], st["log_decay"], st["pool"], st["read"], st["o"],
                          intermediate_states=st["states"], err_word=st["err"], scale=st["scale"])
    return [st["o"]] if st["states"] is None else [st["o"], st["states"]]


def work(case):
    op, B = case["op"], case["B"]
    size = {"f32": 4, "bf16": 2}
    if op == "probs":
        n = B * case["T"] * case["V"]
        return {"bytes": n * (size[case["io"]] + 4), "flops": 4 * n}
    lanes = B - (B // 10 if case["padded"] else 0)
    if op == "accept":  # the row that the token comes from, and the draft's
        rows = 2 if case["probs"] else 1
        return {"bytes": lanes * (case["V"] * 4 * rows + case["T"] * 24), "flops": 3 * lanes * case["V"]}
    HK, HV, DK, DV = (case[n] for n in ("HK", "HV", "DK", "DV"))
    io, state = size[case["io"]], HV * DV * DK * size[case["state"]]
    kv = HK * DK + HV * DV
    if op == "commit":
        T = (1 + case["T"]) / 2
        return {"bytes": lanes * (2 * state + T * kv * io), "flops": 2 * lanes * T * HV * DV * DK}
    if op == "prefill":
        n = (case["lo"] + case["hi"]) / 2 * lanes
        return {"bytes": n * 2 * kv * io + 1.5 * lanes * state, "flops": 4 * n * HV * DV * DK}
    T = case["T"]
    times = 2 if op == "decode" else 1 + (T if case["kept"] else 0)
    return {"bytes": lanes * (times * state + T * 2 * kv * io), "flops": 4 * lanes * T * HV * DV * DK}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------
def exact(case, seed):
    op = case["op"]
    if op == "accept":
        return None  # whole numbers
    if op == "prefill":
        cost = 2.0 * case["B"] * case["hi"] ** 2 * case["HV"] * (case["DK"] + case["DV"])
        if cost > 1.2e13:
            return None
    st = prepare(case, seed)
    if op == "probs":
        x = st["logits"].double()
        out = torch.zeros_like(x)
        for b, T in enumerate(st["temperature"].double().tolist()):
            for t in range(case["T"]):
                row = x[b, t]
                if not bool(torch.isfinite(row).any()):
                    continue
                if T == 0:
                    out[b, t, int(torch.nonzero(row == row.max())[0])] = 1
                else:
                    y = row / T
                    out[b, t] = torch.exp(y - torch.logsumexp(y, 0))
        return [out]
    G, scale = case["HV"] // case["HK"], st["scale"]
    ld = st["log_decay"].double()
    pool = st["pool"].double()
    o = torch.zeros(st["o"].shape, dtype=torch.float64, device="cuda")
    q, k, v = (st[n].double() for n in ("q", "k", "v"))
    states = None if st["states"] is None else torch.zeros(st["states"].shape, dtype=torch.float64, device="cuda")
    read, write = st["read"].tolist(), st["write"].tolist()
    if op != "prefill":
        last = st["accept_len"].tolist() if op == "commit" else [case["T"]] * case["B"]
        for b in range(case["B"]):
            if read[b] < 0:
                continue
            S = pool[read[b]].clone()
            for t in range(last[b]):
                kt, qt = k[b, t].repeat_interleave(G, 0), q[b, t].repeat_interleave(G, 0)
                S = torch.exp(ld)[:, None, None] * S + v[b, t][:, :, None] * kt[:, None, :]
                o[b, t] = scale * (S * qt[:, None, :]).sum(-1)
                if states is not None:
                    states[b, t] = S
            if op != "verify":
                pool[write[b]] = S
        return {"decode": [o, pool], "commit": [pool], "verify": [o] if states is None else [o, states]}[op]
    cu, has = st["cu"].tolist(), st["has"].tolist()
    for b in range(case["B"]):
        if read[b] < 0:
            continue
        lo, n = cu[b], cu[b + 1] - cu[b]
        S0 = pool[read[b]] if has[b] else torch.zeros_like(pool[0])
        age = torch.arange(n + 1, dtype=torch.float64, device="cuda")
        for h in range(case["HV"]):
            g = torch.exp(ld[h] * age)  # g^0 .. g^n
            kh, vh, qh = k[lo:lo + n, h // G], v[lo:lo + n, h], q[lo:lo + n, h // G]
            for a in range(0, n, 2048):
                e = min(n, a + 2048)
                i = torch.arange(a, e, device="cuda")[:, None] - torch.arange(e, device="cuda")[None]
                s = (qh[a:e] @ kh[:e].T) * torch.where(i >= 0, g[i.clamp(min=0)], torch.zeros((), dtype=torch.float64, device="cuda"))
                o[lo + a:lo + e, h] = scale * (s @ vh[:e] + g[a + 1:e + 1, None] * (qh[a:e] @ S0[h].T))
            pool[write[b], h] = g[n] * S0[h] + (vh * g[:n].flip(0)[:, None]).T @ kh
    return [o, pool]
