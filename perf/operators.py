"""The operators of a softmax-attention layer over a paged 4-bit key/value cache, as measured cases.

A hybrid model runs such layers between its Gated DeltaNet layers.  A serving step uses these operators together:

* ``plan``       block tables, slot map, positions and offsets of a step's tokens, built on the GPU from request lengths;
* ``norm_rope``  RMS norm of every query and key head with the position rotation, in one pass;
* ``store``      the same pass, with the keys and values quantised into the cache's 4-bit pages, and those rows read back;
* ``attend``     causal attention of each request's queries over its cached pages (one token, a few drafts, a prompt).

The cache holds, per page, keys and values of ``page`` tokens: codes ``[pages, 2, HK, page, D/2]`` (two e2m1 numbers a
byte, the lower half first) and e4m3 scales ``[pages, 2, HK, page, D/16]``, one for each 16 dimensions; a value is
code * scale.  ``run`` computes the plain form in elementary torch operations, or calls the framework where ``own``.
"""
import math

import torch

own = False

EPS = 1e-6
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
BORDERS = (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)  # midpoints of the magnitudes; a tie goes to the even code


def listed():
    return [
        # one speculative step's bookkeeping: 256 lanes with 8 drafts each, a tenth of the lanes padded
        dict(name="plan verify B256 T8", op="plan", B=256, lo=8, hi=8, ctx=32768, page=64, padded=True),
        # a packed prefill batch: 64 prompts of 256 to 4096 tokens, small pages
        dict(name="plan prompts B64", op="plan", B=64, lo=256, hi=4096, ctx=1024, page=16, padded=False),
        # a prompt chunk's queries and keys on their way to attention, full rotation in halves, fused qkv rows
        dict(name="norm_rope N8192 D128", op="norm_rope", N=8192, HQ=32, HK=8, D=128, R=128, pairs=False, far=32768),
        # the smallest call: one token, wide heads, a quarter of the dimensions rotated, a far position
        dict(name="norm_rope N1 D256", op="norm_rope", N=1, HQ=16, HK=2, D=256, R=64, pairs=False, far=1000000),
        # the verify rows of 128 lanes, 4 drafts each, written to the cache
        dict(name="store N512 D256", op="store", N=512, HQ=16, HK=2, D=256, R=64, pairs=False, far=262144, page=64),
        # a long ragged prompt chunk written to the cache, rotation of neighbouring pairs
        dict(name="store N16381 D128", op="store", N=16381, HQ=32, HK=8, D=128, R=128, pairs=True, far=131072, page=16),
        # one request far into its context: the latency of a single token over a long cache
        dict(name="attend B1 T1 L131071", op="attend", B=1, lo=1, hi=1, ctx=131070, even=True, HQ=32, HK=4, D=128,
             page=64, padded=False),
        # an ordinary decode batch, ragged contexts, wide heads
        dict(name="attend B64 T1 D256", op="attend", B=64, lo=1, hi=1, ctx=8192, even=False, HQ=16, HK=2, D=256,
             page=64, padded=False),
        # a verify step of 4 drafts over 128 ragged contexts
        dict(name="attend B128 T4 D128", op="attend", B=128, lo=4, hi=4, ctx=16384, even=False, HQ=32, HK=4, D=128,
             page=64, padded=False),
        # a verify step of 8 drafts, a tenth of the lanes padded, narrow heads, small pages
        dict(name="attend B256 T8 D64", op="attend", B=256, lo=8, hi=8, ctx=4096, even=False, HQ=32, HK=4, D=64,
             page=16, padded=True),
        # two prompt chunks of 2048 tokens behind 8192 cached ones
        dict(name="attend prompts B2 T2048", op="attend", B=2, lo=2048, hi=2048, ctx=8192, even=True, HQ=32, HK=4,
             D=128, page=64, padded=False),
        # a packed batch of new prompts of odd lengths
        dict(name="attend prompts B16 ragged", op="attend", B=16, lo=64, hi=2048, ctx=0, even=False, HQ=16, HK=2,
             D=128, page=32, padded=False),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("plan", "norm_rope", "store", "attend", "attend", "attend"))
    if op == "plan":
        few = rng.random() < 0.5
        hi = rng.randint(1, 16) if few else _log(rng, 17, 4096)
        B = _log(rng, 1, 512 if few else 64)
        return dict(op=op, B=B, lo=hi if few else max(1, hi // 16), hi=hi, ctx=_log(rng, 16, 32768),
                    page=rng.choice((16, 32, 64, 128, 256)), padded=rng.random() < 0.3)
    D = rng.choice((64, 128, 256))
    HK = rng.choice((1, 2, 4, 8)) if D < 256 else rng.choice((1, 2, 4))
    HQ = HK * rng.choice((1, 2, 3, 4, 6, 8))
    if op in ("norm_rope", "store"):
        c = dict(op=op, N=_log(rng, 1, 8192), HQ=HQ, HK=HK, D=D, R=rng.choice((0, 32, D // 2, D)),
                 pairs=rng.random() < 0.4, far=_log(rng, 64, 1000000))
        return dict(c, page=rng.choice((16, 32, 64, 128, 256))) if op == "store" else c
    page = rng.choice((16, 32, 64, 128, 256))
    shape = rng.choice(("one", "drafts", "prompts"))
    if shape == "prompts":
        hi = _log(rng, 17, 1500)
        return dict(op=op, B=rng.randint(1, 4), lo=max(1, hi // 8), hi=hi, ctx=_log(rng, 1, 4096),
                    even=rng.random() < 0.5, HQ=HQ, HK=HK, D=D, page=page, padded=rng.random() < 0.3)
    T = 1 if shape == "one" else rng.randint(2, 16)
    ctx = _log(rng, 1, 65536)
    B = min(_log(rng, 1, 128), max(1, (1 << 22) // (ctx * HK * D // 64)))
    return dict(op=op, B=B, lo=T, hi=T, ctx=ctx, even=rng.random() < 0.3, HQ=HQ, HK=HK, D=D, page=page,
                padded=rng.random() < 0.3)


# ---- inputs ----------------------------------------------------------------------------------------------
def _lengths(case, gen):
    """Cached and new tokens of each lane (on the host); padded lanes have neither.  A case always has the same
    lengths, in an order of lanes that the seed gives, so that its outputs keep their shapes."""
    B, ctx = case["B"], case["ctx"]
    mine = torch.Generator().manual_seed(B * 1000003 + ctx * 101 + case["hi"])
    new = torch.randint(case["lo"], case["hi"] + 1, (B,), generator=mine)
    if case.get("even"):
        old = torch.full((B,), ctx)
    else:
        old = torch.randint(ctx // 32, ctx + 1, (B,), generator=mine)
    if case["padded"]:
        old[: B // 10], new[: B // 10] = 0, 0
    order = torch.randperm(B, generator=gen)
    return old[order], new[order]


def _pages_of(lens, page):
    return (lens + page - 1) // page


def _quantise(x):
    """e2m1 codes and e4m3 scales (as bytes) of each 16 values along the last axis, and the values they stand for."""
    g = x.reshape(*x.shape[:-1], -1, 16)
    top = g.abs().amax(-1)
    s = (top / torch.full_like(top, 6)).clamp(max=448.0)
    # rounded to e4m3 before the cast, which would go through 32 bits: multiples of 2^(e - 3), 2^-9 at least
    units = torch.tensor([2.0 ** e for e in range(-9, 6)], dtype=s.dtype, device=s.device)
    unit = units[(torch.frexp(s).exponent + 5).clamp(0, 14)]
    s = (torch.round(s / unit) * unit).to(torch.float8_e4m3fn)
    f = s.to(x.dtype).unsqueeze(-1)
    y = torch.where(f > 0, g.abs() / f, torch.zeros_like(g))
    b = torch.tensor(BORDERS, dtype=x.dtype, device=x.device)
    up = torch.tensor([i % 2 == 1 for i in range(7)], device=x.device)
    mag = ((y.unsqueeze(-1) > b) | ((y.unsqueeze(-1) == b) & up)).sum(-1)
    val = torch.tensor(E2M1, dtype=x.dtype, device=x.device)[mag] * f
    val = torch.where(g < 0, -val, val).reshape(x.shape)
    code = (mag + 8 * (g < 0)).to(torch.uint8).reshape(*x.shape[:-1], -1, 2)
    return code[..., 0] | (code[..., 1] << 4), s.view(torch.uint8), val


def prepare(case, seed):
    host = torch.Generator().manual_seed(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)

    def normal(*shape, std=1.0):
        return torch.randn(shape, generator=gen, device="cuda") * std

    st = dict(case)
    st["err"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if case["op"] in ("plan", "attend"):
        page, B = case["page"], case["B"]
        old, new = _lengths(case, host)
        total = old + new
        held, need = _pages_of(old, page), _pages_of(total, page)
        width = int(need.max()) + 1
        num_pages = int(need.sum()) + B + 1
        order = torch.randperm(num_pages, generator=host, dtype=torch.int32)
        # the pages of the tokens that are cached already come first in the order of taking
        col = torch.arange(width).expand(B, width)
        first = torch.cumsum(held, 0) - held
        table = torch.where(col < held[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)],
                            torch.full((B, width), -1, dtype=torch.int32))
        i32 = dict(dtype=torch.int32, device="cuda")
        st.update(width=width, num_pages=num_pages)
        if case["op"] == "plan":
            N = int(new.sum()) + case["hi"]  # a step's buffers have room for more tokens than it brings
            st.update(N=N, old=old.to(**i32), new=new.to(**i32), table=table.to(**i32), held=held.to(**i32),
                      free=order.to(**i32), taken=held.sum().reshape(1).to(**i32),
                      cu=torch.zeros(B + 1, **i32), pos=torch.zeros(N, **i32), slots=torch.zeros(N, **i32),
                      total=torch.zeros(B, **i32), held_out=torch.zeros(B, **i32),
                      taken_out=torch.zeros(1, **i32), ticket=torch.zeros(1, **i32))
            return st
        first = torch.cumsum(need, 0) - need
        table = torch.where(col < need[:, None], order[(first[:, None] + col).clamp(max=num_pages - 1)],
                            torch.full((B, width), -1, dtype=torch.int32))
        HQ, HK, D = case["HQ"], case["HK"], case["D"]
        cu = torch.zeros(B + 1, dtype=torch.int64)
        cu[1:] = torch.cumsum(new, 0)
        N = int(cu[-1])
        codes = torch.empty((num_pages, 2, HK, page, D // 2), dtype=torch.uint8, device="cuda")
        scales = torch.empty((num_pages, 2, HK, page, D // 16), dtype=torch.uint8, device="cuda")
        step = max(1, (1 << 25) // (2 * HK * page * D))
        for p in range(0, num_pages, step):
            n = min(step, num_pages - p)
            # normed keys are of order one with a few strong dimensions; the last token of a page is hardly larger
            x = normal(n, 2, HK, page, D) * (1 + 2 * (torch.arange(D, device="cuda") % 61 == 7))
            codes[p:p + n], scales[p:p + n], _ = _quantise(x)
        st.update(N=N, q=normal(N, HQ, D, std=1.2).bfloat16(), codes=codes, scales=scales, table=table.to(**i32),
                  total=total.to(**i32), cu=cu.to(**i32), even_q=case["lo"] == case["hi"] and not case["padded"],
                  max_q=max(1, int(new.max())),
                  o=torch.zeros((N, HQ, D), dtype=torch.bfloat16, device="cuda"),
                  lse=torch.zeros((N, HQ), dtype=torch.float32, device="cuda"))
        if st["max_q"] <= 16 and st["even_q"]:
            st["cu_arg"] = None  # the same number of tokens for each lane
        else:
            st["cu_arg"] = st["cu"]
        return st
    N, HQ, HK, D, R = (case[n] for n in ("N", "HQ", "HK", "D", "R"))
    # one row of the fused projection for each token: queries, keys and values side by side
    qkv = (normal(N, HQ + 2 * HK, D) * (0.5 + torch.rand((N, HQ + 2 * HK, 1), generator=gen, device="cuda"))).bfloat16()
    st["q"], st["k"], st["v"] = qkv.split((HQ, HK, HK), dim=1)
    st["qw"], st["kw"] = 1 + normal(D, std=0.1), 1 + normal(D, std=0.1)
    start = torch.randint(0, max(1, case["far"] - N) + 1, (1,), generator=host)
    st["pos"] = (start + torch.arange(N)).to(torch.int32).cuda()
    i = torch.arange(0, R, 2, dtype=torch.float64)
    st["freq"] = (1e6 ** (-i / max(R, 1))).float().cuda()
    st["q_out"] = torch.zeros((N, HQ, D), dtype=torch.bfloat16, device="cuda")
    st["k_out"] = torch.zeros((N, HK, D), dtype=torch.bfloat16, device="cuda")
    if case["op"] == "store":
        page = case["page"]
        num_pages = (N + page - 1) // page + 3
        order = torch.randperm(num_pages, generator=host)
        t = torch.arange(N)
        st["slots"] = (order[t // page] * page + t % page).to(torch.int32).cuda()
        st["codes"] = torch.zeros((num_pages, 2, HK, page, D // 2), dtype=torch.uint8, device="cuda")
        st["scales"] = torch.zeros((num_pages, 2, HK, page, D // 16), dtype=torch.uint8, device="cuda")
        st["v_out"] = torch.zeros((N, HK, D), dtype=torch.bfloat16, device="cuda")
    return st


# ---- the plain forms ---------------------------------------------------------------------------------------
def _plain_plan(st):
    B, N, page = st["B"], st["N"], st["page"]
    old, new, held = st["old"].long(), st["new"].long(), st["held"].long()
    left = st["free"].numel() - st["taken"].long()
    need = (_pages_of(old + new, page) - held).clamp(min=0)
    upto = torch.cumsum(need, 0)
    ok = (need == 0) | (upto <= left)
    total = torch.where(ok, old + new, old)
    cu = torch.cat((torch.zeros_like(new[:1]), torch.cumsum(new, 0)))
    col = torch.arange(st["width"], device=old.device)
    at = st["taken"].long() + (upto - need)[:, None] + col - held[:, None]
    fresh = ok[:, None] & (col >= held[:, None]) & (col < (held + need)[:, None])
    table = torch.where(fresh, st["free"][at.clamp(0, st["free"].numel() - 1)], st["table"])
    t = torch.arange(N, device=old.device)
    lane = torch.searchsorted(cu[1:], t, right=True).clamp(max=B - 1)
    real = t < cu[-1]
    pos = old[lane] + t - cu[lane]
    slot = table[lane, (pos // page).clamp(max=st["width"] - 1)].long() * page + pos % page
    slot = torch.where(real & ok[lane], slot, torch.full_like(slot, -1))
    pos = torch.where(real, pos, torch.zeros_like(pos))
    taken = st["taken"].long() + torch.where(ok, upto, torch.zeros_like(upto)).max()
    return [x.to(torch.int32) for x in (table, cu, pos, slot, total, torch.where(ok, held + need, held), taken)]


def _plain_norm_rope(x, w, st, dtype):
    """Norm and rotation in `dtype`; angles in 64 bits, where far positions need them."""
    x = x.to(dtype)
    y = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * w.to(dtype)
    R = st["R"]
    if R == 0:
        return y
    angle = st["pos"].double()[:, None, None] * st["freq"].double()
    c, s = torch.cos(angle).to(dtype), torch.sin(angle).to(dtype)
    r, rest = y[..., :R], y[..., R:]
    a, b = (r[..., 0::2], r[..., 1::2]) if st["pairs"] else (r[..., : R // 2], r[..., R // 2:])
    a, b = a * c - b * s, b * c + a * s
    r = torch.stack((a, b), -1).flatten(-2) if st["pairs"] else torch.cat((a, b), -1)
    return torch.cat((r, rest), -1)


def _dense(st, which, lanes_pages):
    """Keys (0) or values (1) of every lane's pages as numbers: [B, HK, L, D] in 32 bits."""
    c = st["codes"][lanes_pages, which]
    num = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=c.device)
    pairs = torch.stack((num.repeat(16), num.repeat_interleave(16)), -1)
    x = pairs[c.int()].flatten(-2)
    s = st["scales"][lanes_pages, which].view(torch.float8_e4m3fn).float()
    x = (x.unflatten(-1, (-1, 16)) * s.unsqueeze(-1)).flatten(-2)
    B, n, HK, page, D = x.shape
    return x.transpose(1, 2).reshape(B, HK, n * page, D)


def _plain_attend(st):
    B, HQ, HK, D, N, T = (st[n] for n in ("B", "HQ", "HK", "D", "N", "max_q"))
    G = HQ // HK
    pages = st["table"].long().clamp(min=0)
    cu, total = st["cu"].long(), st["total"].long()
    t = torch.arange(T, device=cu.device)
    mine = cu[:-1, None] + t
    here = mine < cu[1:, None]
    q = st["q"][mine.clamp(max=N - 1)].float().view(B, T, HK, G, D).permute(0, 2, 3, 1, 4).reshape(B, HK, G * T, D)
    k = _dense(st, 0, pages)
    s = torch.matmul(q, k.transpose(-1, -2)).view(B, HK, G, T, -1).mul_(1 / math.sqrt(D))
    del k
    limit = total[:, None] - (cu[1:] - cu[:-1])[:, None] + t  # the last key that query t of a lane sees
    sees = torch.arange(s.shape[-1], device=cu.device) <= limit[:, :, None]
    s.masked_fill_(~sees[:, None, None], -math.inf)
    m = s.amax(-1, keepdim=True)
    m = torch.where(torch.isinf(m), torch.zeros_like(m), m)
    p = s.sub_(m).exp_()
    l = p.sum(-1, keepdim=True)
    seen = sees[:, None, None, :, :].any(2).transpose(-1, -2).any(-1)  # keys that some query sees
    v = _dense(st, 1, pages) * seen[:, :, :, None]
    o = torch.matmul(p.view(B, HK, G * T, -1), v).view(B, HK, G, T, D) / torch.where(l > 0, l, torch.ones_like(l))
    lse = (m + torch.log(l)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, T, HQ, D)[here]
    lse = lse.permute(0, 3, 1, 2).reshape(B, T, HQ)[here]
    return [o.bfloat16(), lse]


def run(st):
    op = st["op"]
    if own:
        import gated_deltanet_linear_mtp_gb300 as gdn
        if op == "plan":
            plan = st.setdefault("plan", gdn.PagePlan(st["cu"], st["pos"], st["slots"], st["total"], st["held_out"],
                                                      st["taken_out"]))
            gdn.gdn_page_plan(st["old"], st["new"], st["page"], st["table"], st["held"], st["free"], st["taken"],
                              plan, st["ticket"], st["err"])
            return [st["table"], st["cu"], st["pos"], st["slots"], st["total"], st["held_out"], st["taken_out"]]
        if op == "attend":
            if "cache" not in st:
                st["cache"] = gdn.Kv4Cache(st["codes"], st["scales"])
                st["workspace"] = gdn.kv4_attention_workspace(st["B"], st["max_q"], st["HQ"], st["HK"], st["D"])
            gdn.gdn_kv4_attention(st["q"], st["cache"], st["table"], st["total"], st["o"], st["workspace"],
                                  cu_seqlens=st["cu_arg"], max_q=st["max_q"], lse=st["lse"],
                                  scale=1 / math.sqrt(st["D"]), err_word=st["err"])
            return [st["o"], st["lse"]]
        if op == "norm_rope":
            gdn.gdn_qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["pos"], st["freq"], st["q_out"],
                                 st["k_out"], eps=EPS, interleaved=st["pairs"], err_word=st["err"])
            return [st["q_out"], st["k_out"]]
        if "cache" not in st:
            st["cache"] = gdn.Kv4Cache(st["codes"], st["scales"])
        gdn.gdn_qk_norm_rope(st["q"], st["k"], st["qw"], st["kw"], st["pos"], st["freq"], st["q_out"], None, eps=EPS,
                             interleaved=st["pairs"], v=st["v"], cache=st["cache"], slot_map=st["slots"],
                             err_word=st["err"])
        gdn.gdn_kv4_read(st["cache"], st["slots"], st["k_out"], st["v_out"], err_word=st["err"])
        return [st["q_out"], st["k_out"], st["v_out"]]
    if op == "plan":
        return _plain_plan(st)
    if op == "attend":
        return _plain_attend(st)
    q = _plain_norm_rope(st["q"], st["qw"], st, torch.float32).bfloat16()
    if op == "norm_rope":
        return [q, _plain_norm_rope(st["k"], st["kw"], st, torch.float32).bfloat16()]
    # in 64 bits: a key next to a border of the 4-bit codes goes to its own side
    k = _quantise(_plain_norm_rope(st["k"], st["kw"], st, torch.float64))[2]
    return [q, k.bfloat16(), _quantise(st["v"].double())[2].bfloat16()]


def work(case):
    op = case["op"]
    if op == "plan":
        mean_new = (case["lo"] + case["hi"]) / 2
        lanes = case["B"] * (0.9 if case["padded"] else 1)
        tokens = lanes * mean_new + case["hi"]
        fresh = lanes * (mean_new + case["page"] / 2) / case["page"]
        return {"bytes": 4 * (case["B"] * 6 + 2 * tokens + 2 * fresh), "flops": 4 * tokens}
    D, HK, HQ = case["D"], case["HK"], case["HQ"]
    if op == "attend":
        lanes = case["B"] - (case["B"] // 10 if case["padded"] else 0)
        new = (case["lo"] + case["hi"]) / 2
        old = case["ctx"] if case["even"] else case["ctx"] * 33 / 64
        cached = 2 * HK * (D // 2 + D // 16)
        reads = lanes * (old + new) * cached + lanes * new * HQ * D * 2
        return {"bytes": reads + lanes * new * HQ * (D * 2 + 4),
                "flops": 4 * lanes * new * HQ * D * (old + (new + 1) / 2)}
    N = case["N"]
    row = 2 * D * 2 * (HQ + HK)
    if op == "store":  # written at 4 bits, read back, written as numbers
        row = 2 * D * 2 * HQ + 2 * HK * (D * 2 + 2 * (D // 2 + D // 16) + D * 2)
    return {"bytes": N * (row + 4 + (4 if op == "store" else 0)) + 8 * D + 2 * case["R"],
            "flops": N * D * 8 * (HQ + HK * (1 if op == "norm_rope" else 4))}


# ---- the definitions in 64 bits ------------------------------------------------------------------------------
def _exact_code(x):
    """Nearest e2m1 value (ties to the even code) times the group's e4m3 scale, by distance to every candidate."""
    grid = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    e4m3 = [e * 2.0 ** -9 if e < 8 else (8 + e % 8) * 2.0 ** (e // 8 - 10) for e in range(127)]
    e4m3 = torch.tensor(e4m3, dtype=torch.float64, device=x.device)

    def nearest(v, table):
        hi = torch.searchsorted(table, v.contiguous()).clamp(1, table.numel() - 1)
        lo = hi - 1
        dl, dh = v - table[lo], table[hi] - v
        up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
        return torch.where(up, table[hi], table[lo])

    g = x.unflatten(-1, (-1, 16))
    top = g.abs().max(-1).values
    scale = nearest(top / torch.full_like(top, 6), e4m3).unsqueeze(-1)  # a quotient, not a product with 1/6
    unit = torch.where(scale > 0, g.abs() / scale.clamp(min=1e-30), torch.zeros_like(g))
    return (torch.sign(g) * nearest(unit, grid) * scale).flatten(-2)


def exact(case, seed):
    if case["op"] == "plan":
        return None
    st = prepare(case, seed)
    D = case["D"]
    if case["op"] != "attend":
        R = case["R"]
        phase = st["pos"].double()[:, None] * st["freq"].double()[None]
        rot = torch.polar(torch.ones_like(phase), phase)[:, None]

        def rotated(x, w):
            x = x.double()
            y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / D + EPS) * w.double()
            if R:
                i = torch.arange(R // 2, device=x.device)
                a, b = (2 * i, 2 * i + 1) if case["pairs"] else (i, i + R // 2)
                z = torch.complex(y[..., a], y[..., b]) * rot
                y = y.clone()
                y[..., a], y[..., b] = z.real, z.imag
            return y

        q, k = rotated(st["q"], st["qw"]), rotated(st["k"], st["kw"])
        return [q, k] if case["op"] == "norm_rope" else [q, _exact_code(k), _exact_code(st["v"].double())]
    page, HQ, HK = case["page"], case["HQ"], case["HK"]
    G = HQ // HK
    o = torch.zeros((st["N"], HQ, D), dtype=torch.float64, device="cuda")
    lse = torch.full((st["N"], HQ), -math.inf, dtype=torch.float64, device="cuda")
    cu, total, table = st["cu"].tolist(), st["total"].tolist(), st["table"].long()
    grid = torch.tensor(E2M1 + tuple(-v for v in E2M1), dtype=torch.float64, device="cuda")
    for b in range(case["B"]):
        n, L = cu[b + 1] - cu[b], total[b]
        if n == 0:
            continue
        j = torch.arange(L, device="cuda")
        where = table[b, j // page]
        seen = j[None, :] <= (L - n + torch.arange(n, device="cuda"))[:, None]
        for h in range(HK):
            kv = []
            for which in (0, 1):
                byte = st["codes"][where, which, h, j % page].long()
                num = torch.stack((grid[byte % 16], grid[byte // 16]), -1).reshape(L, D)
                s = st["scales"][where, which, h, j % page].view(torch.float8_e4m3fn).double()
                kv.append(num * s.repeat_interleave(16, -1))
            q = st["q"][cu[b]:cu[b + 1], h * G:(h + 1) * G].double()
            for g in range(G):
                s = torch.where(seen, q[:, g] @ kv[0].T / math.sqrt(D), torch.full((), -math.inf, dtype=torch.float64, device="cuda"))
                z = torch.logsumexp(s, -1)
                lse[cu[b]:cu[b + 1], h * G + g] = z
                o[cu[b]:cu[b + 1], h * G + g] = torch.exp(s - z[:, None]) @ kv[1]
    return [o, lse]
