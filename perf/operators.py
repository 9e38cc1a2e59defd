"""The operators that surround the routed experts in a decoder layer, as workloads to time.

Four operators: the scored route plan (softmax or sigmoid scores, a balance bias, expert groups,
renormalised weights), the per-head norm with position rotation of queries and keys, the 4-bit
(MXFP4) key/value cache as it is written and read back, and attention over that cache.

`run` computes them from elementary torch operations, or, with `own` set, through the library's
entry points. Head counts: 56 x 128 and 32 x 128 are the layer widths 7168 and 4096 of the
repository's workloads; 896 and 256 experts are their routers; the other sizes are generic.
"""
import math

import torch

own = False
DEV = "cuda"


def listed():
    """The cases: for each operator the latency of a decode step, and a prefill or a long context."""
    return [
        # one token of the 896-expert layer: a decode step's routing, bound by latency
        dict(name="route_one", op="route", T=1, E=896, k=16, score="softmax", groups=1, keep=1,
             top=1, renorm=True, scale=1.0),
        # a prefill batch of a 256-expert layer with expert groups, an odd token count
        dict(name="route_groups", op="route", T=4099, E=256, k=8, score="sigmoid", groups=8,
             keep=4, top=2, renorm=True, scale=2.5),
        # the 16384-token batch of the 896-expert layer
        dict(name="route_wide", op="route", T=16384, E=896, k=16, score="sigmoid", groups=1,
             keep=1, top=1, renorm=True, scale=1.0),
        # queries and keys of a five-sequence decode step, cut out of one fused projection
        dict(name="rope_step", op="rope", T=5, H=56, KV=8, d=128, rot=128, pairs="halves",
             n_pos=32768),
        # a long prefill batch, half of each head rotated in interleaved pairs
        dict(name="rope_prefill", op="rope", T=8191, H=64, KV=8, d=128, rot=64,
             pairs="interleaved", n_pos=16384),
        # one new token in each of 16 sequences
        dict(name="cache_step", op="cache", T=16, KV=8, d=128, page=16, pages=1024),
        # a prefill batch's keys and values
        dict(name="cache_prefill", op="cache", T=16384, KV=8, d=128, page=64, pages=600),
        # one short sequence, small pages: latency
        dict(name="attn_one", op="attn", B=1, q=1, kv=777, ragged=False, H=56, KV=8, d=128,
             page=16, window=0),
        # an ordinary decode batch: sequences of very different lengths
        dict(name="attn_batch", op="attn", B=64, q=1, kv=8192, ragged=True, H=32, KV=4, d=128,
             page=64, window=0),
        # two sequences with a long context: the cache read is everything
        dict(name="attn_long", op="attn", B=2, q=1, kv=262143, ragged=False, H=64, KV=8, d=128,
             page=64, window=0),
        # several draft tokens a sequence, a sliding window, one key head for each query head
        dict(name="attn_draft", op="attn", B=24, q=5, kv=3000, ragged=True, H=16, KV=16, d=64,
             page=32, window=1024),
        # prompts taken in behind a cached prefix, some longer than what is cached
        dict(name="attn_prefill", op="attn", B=3, q=2000, kv=8000, ragged=True, H=32, KV=4, d=128,
             page=128, window=0),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of the listed ones' ranges."""
    op = rng.choice(["route", "rope", "cache", "attn", "attn", "attn"])
    if op == "route":
        E, k = rng.choice([(64, 6), (128, 8), (160, 6), (256, 8), (384, 8), (896, 16), (1000, 12)])
        groups = rng.choice([g for g in (1, 1, 4, 8) if E % g == 0])
        keep = groups if groups == 1 else rng.choice([g for g in range(1, groups) if g * E // groups >= k])
        return dict(op=op, T=_log(rng, 1, 16384), E=E, k=k, score=rng.choice(["softmax", "sigmoid"]),
                    groups=groups, keep=keep, top=1 if groups == 1 else rng.choice([1, 2]),
                    renorm=rng.random() < 0.75, scale=rng.choice([1.0, 2.5]))
    H, KV = rng.choice([(56, 8), (32, 4), (64, 8), (16, 16), (40, 8), (24, 2), (12, 1)])
    d = rng.choice([64, 128, 128])
    if op == "rope":
        return dict(op=op, T=_log(rng, 1, 8192), H=H, KV=KV, d=d, rot=rng.choice([d, d, d // 2, 48]),
                    pairs=rng.choice(["halves", "interleaved"]), n_pos=rng.choice([4096, 16384]))
    page = rng.choice([16, 32, 64, 128])
    if op == "cache":
        T = _log(rng, 1, 16384)
        return dict(op=op, T=T, KV=min(KV, 8), d=d, page=page, pages=-(-(T + 4096) // page))
    kind = rng.choice(["step", "step", "long", "draft", "prefill"])
    window = rng.choice([0, 0, 0, 512])
    if kind == "step":
        B = _log(rng, 1, 64)
        kv = _log(rng, 1, 8192)
        return dict(op=op, B=B, q=1, kv=kv, ragged=rng.random() < 0.5, H=H, KV=min(KV, 8) if H % 8 == 0 else KV,
                    d=d, page=page, window=window)
    if kind == "long":
        return dict(op=op, B=rng.choice([1, 2]), q=1, kv=_log(rng, 20000, 200000), ragged=False, H=H,
                    KV=min(KV, 8), d=d, page=page, window=0)
    if kind == "draft":
        return dict(op=op, B=_log(rng, 1, 32), q=rng.randrange(2, 12), kv=_log(rng, 30, 4000),
                    ragged=rng.random() < 0.5, H=H, KV=KV, d=d, page=page, window=window)
    return dict(op=op, B=rng.choice([1, 2, 3]), q=_log(rng, 60, 1500), kv=_log(rng, 100, 6000), ragged=True,
                H=32, KV=rng.choice([4, 8]), d=d, page=page, window=window)


def _lens(c):
    """(queries, cached tokens) of every sequence; the cached ones end with the queries' own, and a
    ragged batch has empty sequences and ones with fewer cached tokens than queries."""
    if not c["ragged"]:
        return [c["q"]] * c["B"], [max(c["kv"], 1)] * c["B"]
    part = [1.0] + [(0.618034 * i) % 1.0 for i in range(1, c["B"])]
    q = [max(1, int(c["q"] * (1 - p / 2))) if c["q"] > 16 else c["q"] for p in part]
    kv = [0 if i % 11 == 7 else int(c["kv"] * p) for i, p in enumerate(part)]
    return q, kv


def _visible(nq, nkv, window):
    """Pairs of a query and a key that it sees, and the keys that any of them sees."""
    first, pairs = nkv, 0
    for i in range(nq):
        p = nkv - nq + i
        n = p + 1 if window <= 0 else min(p + 1, window)
        if n > 0:
            pairs += n
            first = min(first, p + 1 - n)
    return pairs, nkv - first


def work(case):
    c = case
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        return {"bytes": 4 * T * E + 4 * E + 16 * T * k + 12 * E, "flops": 6 * T * E}
    if c["op"] == "rope":
        n = c["T"] * (c["H"] + c["KV"])
        return {"bytes": 4 * n * c["d"] + 4 * c["T"] * (c["rot"] + 1) + 4 * c["d"],
                "flops": n * (4 * c["d"] + 3 * c["rot"])}
    if c["op"] == "cache":
        n = c["T"] * c["KV"] * 2
        return {"bytes": n * (4 * c["d"] + 2 * (c["d"] // 2 + c["d"] // 32)) + 8 * c["T"],
                "flops": 4 * n * c["d"]}
    per = 2 * (c["d"] // 2 + c["d"] // 32)
    nbytes = flops = 0
    for nq, nkv in zip(*_lens(c)):
        pairs, keys = _visible(nq, nkv, c["window"])
        nbytes += keys * c["KV"] * per + nq * c["H"] * (4 * c["d"] + 4)
        flops += 4 * c["d"] * c["H"] * pairs
    return {"bytes": nbytes, "flops": flops}


def _levels(a):
    """The nearest of the eight magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6, as its number; ties to the even one."""
    n = (a > 0.25).to(torch.uint8)
    for edge, tie in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        n += (a >= edge) if tie else (a > edge)
    return n


def _codes(x):
    """Codes (a byte each) and biased scale exponents of x [..., d] in blocks of 32."""
    b = x.float().unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    e = (torch.frexp(top)[1] - 3).clamp(-127, 127)
    e = torch.where(top == 0, torch.full_like(e, -127), e)
    y = torch.ldexp(b, -e)
    code = _levels(y.abs()) | (torch.signbit(b).to(torch.uint8) << 3)
    return code.flatten(-2), (e.squeeze(-1) + 127).to(torch.uint8)


def _cache(c, pages, seed, k_std, v_std):
    """A cache's four arrays with quantised normal keys and values, in the library's layout."""
    KV, d, page = c["KV"], c["d"], c["page"]
    g = torch.Generator(device=DEV).manual_seed(seed)
    out = []
    for std in (k_std, v_std):
        q = torch.empty((pages, KV, page // 8, d // 32, 8, 16), dtype=torch.uint8, device=DEV)
        # scale bytes: a token's together for the keys, two tokens' side by side for the values
        s = torch.empty((pages, KV, page, d // 32) if not out else (pages, KV, page // 2, d // 32, 2),
                        dtype=torch.uint8, device=DEV)
        channel = std * torch.exp(0.4 * torch.randn(KV, 1, d, device=DEV, generator=g))
        step = max(1, (1 << 26) // (KV * page * d))
        for p in range(0, pages, step):
            n = min(step, pages - p)
            x = (torch.randn(n, KV, page, d, device=DEV, generator=g) * channel).bfloat16()
            code, exp = _codes(x)
            code = code[..., 0::2] | (code[..., 1::2] << 4)
            q[p:p + n] = code.view(n, KV, page // 8, 8, d // 32, 16).transpose(3, 4)
            s[p:p + n] = exp if not out else exp.view(n, KV, page // 2, 2, d // 32).transpose(3, 4)
        out += [q, s]
    return out


def _fused(T, widths, g):
    """Slices of one fused projection's output [T][sum of widths]: strided rows, as a layer has them."""
    x = torch.randn(T, sum(widths), device=DEV, generator=g).bfloat16()
    return x.split(widths, dim=1)


def _angles(n_pos, rot):
    """cos then sin of position x frequency, made in 64 bits: fp32 [n_pos][rot]."""
    f = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device=DEV) / rot)
    a = torch.arange(n_pos, dtype=torch.float64, device=DEV)[:, None] * f
    return torch.cat([a.cos(), a.sin()], 1).float()


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV).manual_seed(seed)
    s = {"case": c}
    if c["op"] == "route":
        T, E, k = c["T"], c["E"], c["k"]
        s["logits"] = torch.randn(T, E, device=DEV, generator=g)
        s["bias"] = torch.randn(E, device=DEV, generator=g) * (0.05 if c["score"] == "sigmoid" else 0.3 / E)
        if own:  # the layer and the plan buffers that a program keeps
            from mxfp4_routed_expert_03_gb300 import MOE_SCORE_SIGMOID, MOE_SCORE_SOFTMAX, moe_route_desc
            from mxfp4_routed_expert_03_gb300.layer import Layer, Plan, alloc_weights
            s["layer"] = Layer(256, 128, E, k, alloc_weights(E, 256, 128))
            s["plan"] = Plan(T, E, k)
            s["plan"].active.zero_()
            s["route"] = moe_route_desc(MOE_SCORE_SIGMOID if c["score"] == "sigmoid" else MOE_SCORE_SOFTMAX,
                                        c["groups"], c["keep"], c["top"], int(c["renorm"]), c["scale"])
        return s
    KV, d = c["KV"], c["d"]
    if c["op"] == "rope":
        T, H = c["T"], c["H"]
        s["q"], s["k"], _ = _fused(T, [H * d, KV * d, KV * d], g)
        s["wq"], s["wk"] = ((1 + 0.2 * torch.randn(d, device=DEV, generator=g)).bfloat16() for _ in range(2))
        s["pos"] = torch.randint(c["n_pos"], (T,), device=DEV, generator=g, dtype=torch.int32)
        s["table"] = _angles(c["n_pos"], c["rot"])
        if own:
            from mxfp4_routed_expert_03_gb300.attention import Attention, Rope, alloc_kv_cache
            s["attn"] = Attention(H, KV, d, 16, 1, alloc_kv_cache(KV, d, 16, 1))
            s["rope"] = Rope(s["table"], c["rot"], interleaved=c["pairs"] == "interleaved", eps=1e-6,
                             q_weight=s["wq"], k_weight=s["wk"])
            s["q_out"] = torch.empty(T, H * d, dtype=torch.bfloat16, device=DEV)
            s["k_out"] = torch.empty(T, KV * d, dtype=torch.bfloat16, device=DEV)
        return s
    if c["op"] == "cache":
        T, page, pages = c["T"], c["page"], c["pages"]
        _, s["k"], s["v"] = _fused(T, [KV * d, KV * d, KV * d], g)
        # whole pages in any order, filled from their start, as an allocator hands them out
        order = torch.randperm(pages, device=DEV, generator=g)
        if T <= 64:  # one token in each of T sequences
            s["slots"] = (order[:T] * page + torch.randint(page, (T,), device=DEV, generator=g)).int()
        else:
            at = torch.arange(T, device=DEV)
            s["slots"] = (order[at // page] * page + at % page).int()
        if own:
            from mxfp4_routed_expert_03_gb300.attention import Attention, alloc_kv_cache
            s["attn"] = Attention(KV, KV, d, page, pages, alloc_kv_cache(KV, d, page, pages))
            s["k_out"] = torch.empty(T, KV * d, dtype=torch.bfloat16, device=DEV)
            s["v_out"] = torch.empty(T, KV * d, dtype=torch.bfloat16, device=DEV)
        return s
    nq, nkv = _lens(c)
    B, H, page, T = c["B"], c["H"], c["page"], sum(nq)
    need = [-(-n // page) for n in nkv]
    pages = sum(need) + 3
    s["cache"] = _cache(c, pages, seed + 1, 1.0, 1.0)
    order = torch.randperm(pages, device=DEV, generator=g).int()
    table = torch.zeros(B, max(max(need), 1), dtype=torch.int32, device=DEV)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    s["table"] = table
    s["q"] = (2 * torch.randn(T, H * d, device=DEV, generator=g)).bfloat16()
    s["nq"] = torch.tensor(nq, dtype=torch.int32, device=DEV)
    s["cu"] = torch.nn.functional.pad(s["nq"].cumsum(0), (1, 0)).int()
    s["kv"] = torch.tensor(nkv, dtype=torch.int32, device=DEV)
    s["max_q"], s["max_kv"] = max(nq), max(nkv)
    s["scale"] = d ** -0.5
    if own:
        from mxfp4_routed_expert_03_gb300.attention import Attention, Batch
        names = ("k_q", "k_s", "v_q", "v_s")
        s["attn"] = Attention(H, KV, d, page, pages, dict(zip(names, s["cache"])))
        s["batch"] = Batch(B, T, s["max_q"], max(s["max_kv"], 1), s["cu"], s["kv"], table, s["scale"],
                           c["window"])
        s["out"] = torch.empty(T, H * d, dtype=torch.bfloat16, device=DEV)
        s["lse"] = torch.empty(T, H, dtype=torch.float32, device=DEV)
    return s


def _plan_of(idx, E):
    """counts, offsets, perm, inv and active of the chosen experts [T][k]."""
    flat = idx.flatten()
    counts = torch.bincount(flat, minlength=E)
    offsets = torch.nn.functional.pad(counts.cumsum(0), (1, 0))
    perm = torch.sort(flat, stable=True)[1]
    inv = torch.empty_like(perm)
    inv[perm] = torch.arange(perm.numel(), device=perm.device)
    used = counts > 0
    active = torch.zeros(E + 1, dtype=torch.int64, device=idx.device)
    active[0] = used.sum()
    place = torch.where(used, used.cumsum(0), torch.zeros_like(counts))
    active.scatter_add_(0, place, torch.arange(E, device=idx.device) * used)
    return [t.int() for t in (counts, offsets, perm, inv, active)]


def _plain_route(s):
    c, x = s["case"], s["logits"]
    if c["score"] == "sigmoid":
        p = 1.0 / (1.0 + torch.exp(-x))
    else:
        e = torch.exp(x - x.amax(1, keepdim=True))
        # the sum rounded once, so that which expert is chosen does not hang on its order
        p = e / e.double().sum(1, keepdim=True).float()
    biased = p + s["bias"]
    if c["groups"] > 1:
        by = biased.unflatten(1, (c["groups"], -1))
        score = by.sort(dim=2, descending=True)[0][:, :, :c["top"]].sum(2)
        kept = score.sort(dim=1, descending=True, stable=True)[1][:, :c["keep"]]
        open_ = torch.zeros_like(score, dtype=torch.bool).scatter_(1, kept, True)
        biased = torch.where(open_[:, :, None], by, torch.full_like(by, -math.inf)).flatten(1)
    idx = biased.sort(dim=1, descending=True, stable=True)[1][:, :c["k"]]
    w = p.gather(1, idx)
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [idx.int(), w * c["scale"]] + _plan_of(idx, c["E"])


def _plain_rope(s):
    c, d, rot = s["case"], s["case"]["d"], s["case"]["rot"]
    cos, sin = s["table"][s["pos"].long()][:, None].chunk(2, -1)
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.float().unflatten(1, (-1, d))
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-6) * w.float()
        r = y[..., :rot]
        if c["pairs"] == "halves":
            a, b = r.chunk(2, -1)
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        else:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        out.append(torch.cat([r, y[..., rot:]], -1).flatten(1).bfloat16())
    return out


_VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def _plain_cache(s):
    c = s["case"]
    KV, d, page, pages = c["KV"], c["d"], c["page"], c["pages"]
    slots = s["slots"].long()
    value = torch.tensor(_VALUES + [-v for v in _VALUES], device=DEV)
    out = []
    for x in (s["k"], s["v"]):
        code, exp = _codes(x.unflatten(1, (KV, d)))
        q = torch.empty((pages * page, KV, d // 2), dtype=torch.uint8, device=DEV)
        e = torch.empty((pages * page, KV, d // 32), dtype=torch.uint8, device=DEV)
        q[slots] = code[..., 0::2] | (code[..., 1::2] << 4)
        e[slots] = exp
        back = q[slots]
        y = value[torch.stack([back & 15, back >> 4], -1).flatten(-2).long()]
        y = torch.ldexp(y.unflatten(-1, (-1, 32)), e[slots].int()[..., None] - 127)
        out.append(y.flatten(1).bfloat16())
    return out


def _plain_attn(s):
    c = s["case"]
    H, KV, d, page = c["H"], c["KV"], c["d"], c["page"]
    B, S, Q = c["B"], s["table"].shape[1] * page, s["max_q"]
    value = torch.tensor(_VALUES + [-v for v in _VALUES], device=DEV)
    kv = []
    for q, e in (s["cache"][:2], s["cache"][2:]):
        q, e = q[s["table"].long()], e[s["table"].long()]
        # [B][pages][KV][page/8][d/32][8][16] -> [B][KV][S][d]
        q = q.permute(0, 2, 1, 3, 5, 4, 6).reshape(B, KV, S, d // 2)
        if e.dim() == 6:  # the values' scales: [B][pages][KV][page/2][d/32][2]
            e = e.transpose(4, 5).reshape(B, -1, KV, page, d // 32)
        e = e.transpose(1, 2).reshape(B, KV, S, d // 32)
        y = value[torch.stack([q & 15, q >> 4], -1).flatten(-2).int()]
        kv.append((y.unflatten(-1, (-1, 32)) * torch.exp2(e.float() - 127)[..., None]).flatten(-2))
    k, v = kv
    row = torch.arange(Q, device=DEV)
    real = row < s["nq"][:, None]
    q = torch.zeros(B, Q, H, d, device=DEV)
    q[real] = s["q"].float().view(-1, H, d)
    q = q.view(B, Q, KV, H // KV, d).permute(0, 2, 3, 1, 4).reshape(B, KV, -1, d)
    x = (q @ k.transpose(2, 3)).unflatten(2, (H // KV, Q)) * s["scale"]
    pos = (s["kv"] - s["nq"])[:, None] + row
    key = torch.arange(S, device=DEV)
    seen = key <= pos[..., None]
    if c["window"] > 0:
        seen &= key > pos[..., None] - c["window"]
    x = x.masked_fill(~seen[:, None, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top.clamp(min=-3e38))
    total = p.sum(-1, keepdim=True)
    o = (p.flatten(2, 3) @ v).unflatten(2, (H // KV, Q)) / total.clamp(min=1e-37)
    lse = (top + torch.log(total)).squeeze(-1)
    o = o.permute(0, 3, 1, 2, 4).reshape(B, Q, H * d)
    lse = lse.permute(0, 3, 1, 2).reshape(B, Q, H)
    return [o[real].bfloat16(), lse[real]]


def run(state):
    s, c = state, state["case"]
    if not own:
        return {"route": _plain_route, "rope": _plain_rope, "cache": _plain_cache, "attn": _plain_attn}[c["op"]](s)
    from mxfp4_routed_expert_03_gb300 import check
    st = torch.cuda.current_stream()
    if c["op"] == "route":
        p = s["plan"]
        check(s["layer"].plan_scored(c["T"], s["logits"], None, p, s["route"], s["bias"], st), "moe_plan_scored")
        return [p.topk_idx, p.topk_w, p.counts, p.offsets, p.perm, p.inv, p.active]
    a = s["attn"]
    if c["op"] == "rope":
        check(a.norm_rope(c["T"], s["q"], s["k"], s["pos"], s["rope"], s["q_out"], s["k_out"], st), "moe_qk_norm_rope")
        return [s["q_out"], s["k_out"]]
    if c["op"] == "cache":
        check(a.append(c["T"], s["k"], s["v"], s["slots"], st), "moe_kv_append")
        check(a.read(c["T"], s["slots"], s["k_out"], s["v_out"], st), "moe_kv_read")
        return [s["k_out"], s["v_out"]]
    check(a.forward(s["batch"], s["q"], s["out"], s["lse"], st), "moe_attn_forward")
    return [s["out"], s["lse"]]


def _exact_route(s):
    c, x = s["case"], s["logits"].double()
    p = torch.sigmoid(x) if c["score"] == "sigmoid" else torch.softmax(x, 1)
    sel = p + s["bias"].double()
    if c["groups"] > 1:
        size = c["E"] // c["groups"]
        score = sel.view(-1, c["groups"], size).topk(c["top"], 2)[0].sum(2)
        shut = torch.ones_like(score, dtype=torch.bool).scatter_(1, score.topk(c["keep"], 1)[1], False)
        sel = sel.masked_fill(shut.repeat_interleave(size, 1), -math.inf)
    w = torch.gather(p, 1, sel.topk(c["k"], 1)[1])
    if c["renorm"]:
        w = w / w.sum(1, keepdim=True)
    return [None, w * c["scale"], None, None, None, None, None]


def _exact_rope(s):
    c, d, rot = s["case"], s["case"]["d"], s["case"]["rot"]
    angle = s["table"].double()[s["pos"].long()]
    turn = torch.complex(angle[:, :rot // 2], angle[:, rot // 2:])[:, None]
    out = []
    for x, w in ((s["q"], s["wq"]), (s["k"], s["wk"])):
        x = x.double().reshape(c["T"], -1, d)
        y = x * torch.rsqrt(x.pow(2).sum(-1, keepdim=True) / d + 1e-6) * w.double()
        if c["pairs"] == "halves":
            z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * turn
            y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
        else:
            z = torch.complex(y[..., 0:rot:2], y[..., 1:rot:2]) * turn
            y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
        out.append(y.reshape(c["T"], -1))
    return out


def _exact_cache(s):
    c = s["case"]
    levels = torch.tensor(_VALUES, dtype=torch.float64, device=DEV)
    out = []
    for x in (s["k"], s["v"]):
        b = x.double().reshape(-1, 32)
        top = b.abs().max(1, keepdim=True)[0]
        unit = torch.exp2((torch.floor(torch.log2(top.clamp(min=1e-300))) - 2).clamp(min=-127))
        y = (b / unit).abs()
        # distance to each level; an odd level loses a tie
        far = (y[..., None] - levels).abs() + torch.arange(8, device=DEV) % 2 * 1e-12
        out.append((torch.copysign(levels[far.argmin(-1)], b) * unit).reshape(c["T"], -1))
    return out


def _exact_attn(s):
    c = s["case"]
    H, KV, d, page = c["H"], c["KV"], c["d"], c["page"]
    levels = torch.tensor(_VALUES + [-v for v in _VALUES], dtype=torch.float64, device=DEV)
    dim = torch.arange(d, device=DEV)
    out, lse = [], []
    for b, (nq, nkv) in enumerate(zip(*_lens(c))):
        at = int(s["cu"][b])
        q = s["q"][at:at + nq].double().view(nq, H, d)
        o = torch.zeros(nq, H, d, dtype=torch.float64, device=DEV)
        l_ = torch.full((nq, H), -math.inf, dtype=torch.float64, device=DEV)
        tok = torch.arange(nkv, device=DEV)
        where = s["table"][b].long()[tok // page] if nkv else tok
        pos = nkv - nq + torch.arange(nq, device=DEV)[:, None]
        seen = tok <= pos
        if c["window"] > 0:
            seen = seen & (tok > pos - c["window"])
        live = seen.any(1)
        for h in range(KV if nkv else 0):
            kv = []
            for codes, exps in (s["cache"][:2], s["cache"][2:]):
                off = tok % page
                byte = codes.view(-1)[(((where * KV + h) * (page // 8) + off // 8)[:, None] * (d // 32) + dim // 32) * 128
                                      + (off % 8 * 16)[:, None] + dim % 32 // 2]
                nb = d // 32
                if kv:  # the second pair of arrays: the values
                    at_e = ((((where * KV + h) * (page // 2) + off // 2)[:, None] * nb + dim // 32) * 2 + (off % 2)[:, None])
                else:
                    at_e = ((where * KV + h) * page + off)[:, None] * nb + dim // 32
                e = exps.view(-1)[at_e]
                kv.append(levels[((byte >> (dim % 2 * 4)) & 15).int()] * torch.exp2(e.double() - 127))
            for j in range(h * (H // KV), (h + 1) * (H // KV)):
                x = (q[:, j] @ kv[0].T * s["scale"]).masked_fill(~seen, -math.inf)
                l_[live, j] = torch.logsumexp(x[live], 1)
                o[live, j] = torch.softmax(x[live], 1) @ kv[1]
        out.append(o.reshape(nq, -1))
        lse.append(l_)
    return [torch.cat(out), torch.cat(lse)]


def exact(case, seed):
    c = dict(case)
    if c["op"] == "attn":
        nq, nkv = _lens(c)
        if sum(a * b for a, b in zip(nq, nkv)) * c["H"] * c["d"] > 1.5e12:
            return None
    s = prepare(c, seed)
    return {"route": _exact_route, "rope": _exact_rope, "cache": _exact_cache, "attn": _exact_attn}[c["op"]](s)
