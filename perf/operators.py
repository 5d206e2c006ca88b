"""Cases of the operators around a compressed K/V cache that several readers share and that is kept
within a budget:

* ``attention``: softmax attention of a batch of sequences over one compressed prefix that all of them
  share, joined with each sequence's own uncompressed tail;
* ``weights``: the attention weight that every token of the compressed prefix receives from such a
  batch, added to what it received before;
* ``evict``: the tokens with the most accumulated weight (and the first and the latest ones) are kept,
  and the packed streams of keys and values close up over the others.

A cache is made of the packed streams themselves (2-bit codes, E4M3 scales and zero points, uint8
centroid indices, bf16 centroid tables), as a program has them in hand that quantised its chunks before.
"""
import math

import torch

own = False

D = 128
DEV = "cuda"


def _attention(name, **kw):
    return dict(op="attention", name=name, **kw)


def _weights(name, **kw):
    return dict(op="weights", name=name, **kw)


def _evict(name, **kw):
    return dict(op="evict", name=name, **kw)


def listed():
    """H K/V heads, `group` query heads to each, B sequences of Nq queries, Nk cached tokens, tails of up to
    `tail` tokens; T stages of K centroids, groups of G channels, one scale (sym) or scale and zero point."""
    return [
        # the smallest call: two samples drawn from one short prompt, a token each, a short ragged tail
        _attention("attention_two_samples", H=4, group=1, B=2, Nq=1, Nk=512, K=16, T=1, G=16, sym=False, tail=16, causal=True,
                   evicted=False),
        # eight requests behind one long prompt, a token each, grouped heads, tails of unlike lengths
        _attention("attention_requests", H=8, group=4, B=8, Nq=1, Nk=38000, K=256, T=2, G=64, sym=False, tail=512, causal=True,
                   evicted=False),
        # one sequence, one token, over a cache that evictions have thinned (positions with gaps)
        _attention("attention_one_token", H=32, group=1, B=1, Nq=1, Nk=28011, K=256, T=1, G=64, sym=True, tail=33, causal=True,
                   evicted=True),
        # a frame with and without its condition: both read the same past, each its own frame
        _attention("attention_guided_frame", H=12, group=1, B=2, Nq=1560, Nk=14040, K=256, T=2, G=64, sym=False, tail=1560,
                   causal=False, evicted=False),
        # the largest: four variations of a piece of the next frame of a wide model behind 25 frames
        _attention("attention_four_variations", H=32, group=1, B=4, Nq=380, Nk=38000, K=256, T=2, G=64, sym=False, tail=380,
                   causal=False, evicted=True),
        # one token's weights, the smallest call
        _weights("weights_one_token", H=4, group=1, B=1, Nq=1, Nk=700, K=16, T=1, G=16, sym=False, tail=5, causal=True,
                 evicted=False),
        # a decoding step of four requests, grouped heads, over a thinned cache
        _weights("weights_requests", H=8, group=4, B=4, Nq=1, Nk=37999, K=256, T=2, G=64, sym=False, tail=256, causal=True,
                 evicted=True),
        # the weights that one frame gives to five chunks of the past
        _weights("weights_frame", H=12, group=1, B=1, Nq=1560, Nk=23400, K=256, T=2, G=64, sym=False, tail=1560, causal=False,
                 evicted=False),
        # a piece of a prompt, causal within its own tail, the four-stage setting
        _weights("weights_prompt", H=8, group=2, B=2, Nq=300, Nk=9001, K=256, T=4, G=16, sym=True, tail=300, causal=True,
                 evicted=False),
        # a short cache of a few heads loses a quarter
        _evict("evict_short", H=2, Nk=501, K=16, T=1, G=16, sym=False, keep=376, first=4, recent=32),
        # one chunk's worth leaves a cache of five chunks
        _evict("evict_chunk", H=12, Nk=23400, K=256, T=2, G=64, sym=False, keep=18720, first=1560, recent=4680),
        # half of a long cache leaves, the four-stage setting with an odd budget
        _evict("evict_half", H=32, Nk=38000, K=256, T=4, G=16, sym=True, keep=18999, first=1520, recent=4560),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    T, G, sym = rng.choice([(1, 64, True), (2, 64, False), (4, 16, True), (1, 16, False), (3, 32, False), (0, 32, False), (2, 128, True)])
    c = dict(K=rng.choice([16, 64, 200, 256]), T=T, G=G, sym=sym)
    op = rng.choice(["attention", "attention", "weights", "weights", "evict"])
    H = rng.choice([1, 2, 3, 4, 8, 12, 16, 32])
    Nk = _log(rng, 1, 38000)
    if op == "evict":
        keep = max(1, int(Nk * rng.uniform(0.2, 1.0)))
        first = rng.randint(0, keep // 4)
        return dict(op=op, H=H, Nk=Nk, keep=keep, first=first, recent=rng.randint(0, (keep - first) // 2), **c)
    if rng.random() < 0.5:      # single tokens, or a few drafted ones
        B, group, Nq, causal = rng.choice([1, 2, 3, 5, 8, 16]), rng.choice([1, 2, 4, 8]), rng.choice([1, 1, 1, 2, 4]), True
        tail = rng.choice([0, 1, _log(rng, 2, 600)])
    else:                       # blocks of queries
        B, group, Nq, causal = rng.choice([1, 2, 3, 4]), rng.choice([1, 1, 2]), _log(rng, 30, 1600), rng.random() < 0.5
        tail = rng.choice([0, Nq, Nq + rng.randint(1, 200)])
    while H * B * group * Nq * (Nk + tail) > 32 * 1520 * 23000 or B * H * tail * D > 3e7:
        H, Nq, tail = max(1, H // 2), max(1, Nq * 2 // 3), tail * 2 // 3
    return dict(op=op, H=H, group=group, B=B, Nq=Nq, Nk=Nk, tail=tail, causal=causal, evicted=rng.random() < 0.5, **c)


# ------------------------------------------------------------------ inputs

def _streams(g, c):
    """Packed streams of H blocks of Nk tokens: the residuals are a fraction of the centroids, as after k-means."""
    H, N, K, T, G = c["H"], c["Nk"], c["K"], c["T"], c["G"]
    scale = (torch.rand((H, N, D // G), generator=g, device=DEV) * 0.25 + 0.05) * 0.5 ** T
    zero = (scale * (torch.rand(scale.shape, generator=g, device=DEV) - 2.0)).to(torch.float8_e4m3fn).view(torch.uint8)
    size = 0.35 ** torch.arange(T, device=DEV).view(T, 1, 1, 1)
    tables = torch.randn((T, H, K, D), generator=g, device=DEV) * size
    # some clusters hold many tokens, most hold few
    assign = (torch.rand((T, H, N), generator=g, device=DEV) ** 2 * K).clamp_(0, K - 1).to(torch.uint8)
    return dict(codes=torch.randint(0, 256, (H, N, D // 4), generator=g, device=DEV, dtype=torch.uint8),
                scale=scale.to(torch.float8_e4m3fn).view(torch.uint8),
                zero=torch.empty((0,), dtype=torch.uint8, device=DEV) if c["sym"] else zero,
                assign=assign, centroids=tables.to(torch.bfloat16))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(seed * 7919 + 11)
    H, Nk = c["H"], c["Nk"]
    s = dict(case=c, k=_streams(g, c))
    if c["op"] == "evict":
        s["v"] = _streams(g, c)
        w = torch.randn((H, Nk), generator=g, device=DEV).mul_(1.5).exp_()
        w[:, Nk - Nk // 10:] = 0.0                     # the newest tokens have not been looked at yet
        s["weights"] = w
        # the cache has been thinned before: positions ascend, with gaps
        s["k_pos"] = torch.cumsum(torch.randint(1, 3, (H, Nk), generator=g, device=DEV), 1) - 1
        return s
    B, group, Nq, tail = c["B"], c["group"], c["Nq"], c["tail"]
    if c["op"] == "attention":
        s["v"] = _streams(g, c)
    s["Q"] = (torch.randn((B, H * group, Nq, D), generator=g, device=DEV) * 1.5).to(torch.bfloat16)
    s["k_pos"], past = None, Nk
    if c["evicted"]:
        s["k_pos"] = torch.cumsum(torch.randint(1, 3, (H, Nk), generator=g, device=DEV), 1) - 1
        past = 2 * Nk
    s["tail_k"] = s["tail_v"] = s["tail_pos"] = s["tail_len"] = None
    length = torch.full((B,), tail, dtype=torch.int32, device=DEV)
    if tail:
        s["tail_k"] = (torch.randn((B, H, tail, D), generator=g, device=DEV) * 1.1).to(torch.bfloat16)
        s["tail_v"] = torch.randn((B, H, tail, D), generator=g, device=DEV).to(torch.bfloat16)
        s["tail_pos"] = (past + torch.arange(tail, device=DEV)).repeat(B, 1)
        if c["causal"]:         # sequences of unlike lengths
            length[1:] = torch.randint(0, tail + 1, (B - 1,), generator=g, device=DEV, dtype=torch.int32)
        s["tail_len"] = length
    n = torch.arange(Nq, device=DEV)
    if c["causal"]:             # the queries are the last tokens of each sequence; rows before its tail are padding
        at = length[:, None].long() - Nq + n
        s["q_pos"] = torch.where(at < 0, -1, past + at) if tail else past + n.repeat(B, 1)
    else:
        s["q_pos"] = past + n.repeat(B, 1)
    # rotary tables: a 256-byte header of zeros, then fp32 (cos, sin) of p * 10000^(-2i/d), formed in fp64
    rows = past + max(tail, Nq) + 1
    angle = torch.arange(rows, device=DEV, dtype=torch.float64)[:, None] * \
        10000.0 ** (-2.0 * torch.arange(D // 2, device=DEV, dtype=torch.float64) / D)
    turns = torch.stack([angle.cos(), angle.sin()], -1).float()
    s["tables"] = torch.cat([torch.zeros(256, dtype=torch.uint8, device=DEV), turns.view(torch.uint8).reshape(-1)])
    if c["op"] == "weights":    # what the tokens received before
        s["received"] = torch.empty((H, Nk), device=DEV).exponential_(1.0, generator=g) * (4.0 * B * group * Nq / Nk)
    return s


# ------------------------------------------------------------------ the plain form

def _values(p, c):
    """The reconstruction: s*q + m (or s*(u - 2)), plus the centroids from the last stage to the first, to bf16."""
    q = (p["codes"][..., None] >> torch.tensor([0, 2, 4, 6], device=DEV, dtype=torch.uint8)) & 3
    q = q.reshape(*p["codes"].shape[:2], D).float()
    e4m3 = lambda x: x.view(torch.float8_e4m3fn).float().repeat_interleave(c["G"], -1)  # noqa: E731
    y = e4m3(p["scale"]) * (q - 2.0) if c["sym"] else e4m3(p["scale"]) * q + e4m3(p["zero"])
    head = torch.arange(c["H"], device=DEV)[:, None]
    for t in reversed(range(c["T"])):
        y = y + p["centroids"][t][head, p["assign"][t].long()].float()
    return y.to(torch.bfloat16).float()


def _rotate(x, cs):
    a, b = x[..., 0::2], x[..., 1::2]
    return torch.stack([a * cs[..., 0] - b * cs[..., 1], a * cs[..., 1] + b * cs[..., 0]], -1).flatten(-2)


def _logits(s, c):
    """Rotated q.k / sqrt(d) of every row (b, head of K/V: group x Nq) with the prefix and the row's own tail, and
    which of them the row sees."""
    B, H, Nq, Nk, tail = c["B"], c["H"], c["Nq"], c["Nk"], c["tail"]
    turns = s["tables"][256:].view(torch.float32).view(-1, D // 2, 2)
    q_pos = s["q_pos"]
    q = _rotate(s["Q"].float(), turns[q_pos.clamp(min=0)][:, None]).view(B, H, -1, D)
    k_pos = torch.arange(Nk, device=DEV).repeat(H, 1) if s["k_pos"] is None else s["k_pos"]
    k = _rotate(_values(s["k"], c), turns[k_pos])
    x = torch.matmul(q, k.transpose(1, 2)) / math.sqrt(D)
    rows = q_pos.repeat(1, c["group"])[:, None, :, None]                     # [B][1][group x Nq][1]
    sees = rows >= 0
    if c["causal"]:
        sees = sees & (k_pos[:, None, :] <= rows)
    sees = sees.expand(x.shape)
    if tail:
        kt = _rotate(s["tail_k"].float(), turns[s["tail_pos"]][:, None])
        xt = torch.matmul(q, kt.transpose(2, 3)) / math.sqrt(D)
        there = (torch.arange(tail, device=DEV) < s["tail_len"][:, None])[:, None, None, :] & (rows >= 0)
        if c["causal"]:
            there = there & (s["tail_pos"][:, None, None, :] <= rows)
        x, sees = torch.cat([x, xt], -1), torch.cat([sees, there.expand(xt.shape)], -1)
    return x, sees


def _softmax(x, sees):
    x = x.masked_fill(~sees, -math.inf)
    m = x.amax(-1, keepdim=True)
    e = (x - m.masked_fill(m == -math.inf, 0.0)).exp()
    z = e.sum(-1, keepdim=True)
    return e / z.masked_fill(z == 0.0, 1.0)


def _plain_attention(s, c):
    p = _softmax(*_logits(s, c))
    o = torch.matmul(p[..., :c["Nk"]], _values(s["v"], c))
    if c["tail"]:
        v = s["tail_v"].float()
        there = (torch.arange(c["tail"], device=DEV) < s["tail_len"][:, None])[:, None, :, None]
        o = o + torch.matmul(p[..., c["Nk"]:], v.masked_fill(~there, 0.0))
    return o.view(s["Q"].shape).to(torch.bfloat16)


def _plain_weights(s, c):
    return s["received"] + _softmax(*_logits(s, c))[..., :c["Nk"]].sum((0, 2))


def _plain_evict(s, c):
    H, Nk = c["H"], c["Nk"]
    at = torch.arange(Nk, device=DEV)
    rank = s["weights"].masked_fill((at < c["first"]) | (at >= Nk - c["recent"]), math.inf)
    kept = rank.sort(dim=1, descending=True, stable=True).indices[:, :c["keep"]].sort(dim=1).values
    head = torch.arange(H, device=DEV)[:, None]

    def closed(p):
        return [p["codes"][head, kept], p["scale"][head, kept]] + ([] if c["sym"] else [p["zero"][head, kept]]) + \
            [p["assign"][:, head, kept]]
    return [kept.int(), s["k_pos"][head, kept], s["weights"][head, kept], *closed(s["k"]), *closed(s["v"])]


# ------------------------------------------------------------------ one pass

def run(state):
    s, c = state, state["case"]
    if not own:
        return {"attention": _plain_attention, "weights": _plain_weights, "evict": _plain_evict}[c["op"]](s, c)
    from bit_kv_cache_qvg_b200 import qvg
    cfg = qvg.config(K=c["K"], T=c["T"], group_size=c["G"], scale_mode=qvg.SYM if c["sym"] else qvg.ASYM)
    packed = lambda p: qvg.Packed(cfg=cfg, N=c["Nk"], H=c["H"], d=D, dtype=qvg.BF16, **p)  # noqa: E731
    if c["op"] == "evict":
        e = qvg.evict(packed(s["k"]), packed(s["v"]), s["weights"], c["keep"], first=c["first"], recent=c["recent"],
                      k_pos=s["k_pos"])
        closed = lambda p: [p.codes, p.scale] + ([] if c["sym"] else [p.zero]) + [p.assign]  # noqa: E731
        return [e.kept, e.pos, e.weights, *closed(e.k), *closed(e.v)]
    tail = qvg.Tail(k=s["tail_k"], v=s["tail_v"], pos=s["tail_pos"], length=s["tail_len"]) if c["tail"] else None
    if c["op"] == "attention":
        return qvg.attention_batch(packed(s["k"]), packed(s["v"]), s["Q"], s["q_pos"], s["tables"], tail=tail, k_pos=s["k_pos"],
                                   causal=c["causal"])
    return qvg.attention_weights(packed(s["k"]), s["Q"], s["q_pos"], s["tables"], received=s["received"], tail=tail,
                                 k_pos=s["k_pos"], causal=c["causal"])


def work(case):
    c = case
    H, Nk, T, G = c["H"], c["Nk"], c["T"], c["G"]
    token = D // 4 + (1 if c["sym"] else 2) * (D // G) + T
    tables = T * c["K"] * D * 2
    if c["op"] == "evict":
        # every weight, what is kept of both caches read and written once, with positions, weights and indices
        return {"bytes": H * (4 * Nk + c["keep"] * (2 * 2 * token + 2 * 8 + 4 + 4)), "flops": H * Nk}
    B, rows, tail = c["B"], c["B"] * c["group"] * c["Nq"], c["tail"]
    caches = 2 if c["op"] == "attention" else 1
    bytes_ = caches * H * (Nk * token + tables + B * tail * D * 2) + H * rows * D * 2 + B * c["Nq"] * 8
    bytes_ += H * Nk * 8 if c["evicted"] else 0
    bytes_ += H * rows * D * 2 if c["op"] == "attention" else 2 * H * Nk * 4
    return {"bytes": bytes_, "flops": caches * 2 * D * H * rows * (Nk + tail)}


# ------------------------------------------------------------------ the definition in 64 bits

def _exact_token_values(p, c, h):
    """Head h's reconstruction; its two roundings (each sum in fp32, the result to bf16) are part of its definition."""
    shifts = 2 * (torch.arange(D, device=DEV) % 4)
    q = (p["codes"][h].long()[:, torch.arange(D, device=DEV) // 4] >> shifts) & 3
    of = torch.arange(D, device=DEV) // c["G"]
    scale = p["scale"][h].view(torch.float8_e4m3fn).double()[:, of]
    y = scale * (q - 2) if c["sym"] else scale * q + p["zero"][h].view(torch.float8_e4m3fn).double()[:, of]
    y = y.float()
    for t in range(c["T"] - 1, -1, -1):
        y = (y.double() + torch.index_select(p["centroids"][t, h].double(), 0, p["assign"][t, h].int())).float()
    return y.bfloat16().double()


def _exact_turn(x, pos):
    """Channel pairs as complex numbers, turned by pos * 10000^(-2i/d)."""
    theta = torch.exp(torch.arange(D // 2, device=DEV, dtype=torch.float64) * (-2.0 * math.log(10000.0) / D))
    z = torch.view_as_complex(x.double().reshape(*x.shape[:-1], D // 2, 2).contiguous())
    z = z * torch.polar(torch.ones((), dtype=torch.float64, device=DEV), pos.double()[..., None] * theta)
    return torch.view_as_real(z).reshape(x.shape)


def exact(case, seed):
    s, c = prepare(case, seed), case
    H, Nk, tail = c["H"], c["Nk"], c["tail"] if "tail" in c else 0
    if c["op"] == "evict":
        return None             # its outputs are whole numbers and copies
    B, group, Nq = c["B"], c["group"], c["Nq"]
    out = torch.zeros((B, H * group, Nq, D), dtype=torch.float64, device=DEV)
    got = s["received"].double() if c["op"] == "weights" else None
    for h in range(H):
        kp = torch.arange(Nk, device=DEV) if s["k_pos"] is None else s["k_pos"][h]
        k = _exact_turn(_exact_token_values(s["k"], c, h), kp)
        v = _exact_token_values(s["v"], c, h) if c["op"] == "attention" else None
        for b in range(B):
            n = int(s["tail_len"][b]) if tail else 0
            keys, at = k, kp
            if n:
                keys = torch.cat([k, _exact_turn(s["tail_k"][b, h, :n], s["tail_pos"][b, :n])])
                at = torch.cat([kp, s["tail_pos"][b, :n]])
            pos = s["q_pos"][b]
            live = (pos >= 0).nonzero()[:, 0]
            if not len(live):
                continue
            sees = (at[None, :] <= pos[live, None]) if c["causal"] else torch.ones((1, 1), dtype=torch.bool, device=DEV)
            for j in range(h * group, (h + 1) * group):
                q = _exact_turn(s["Q"][b, j, live], pos[live])
                x = (q @ keys.T / D ** 0.5).where(sees, -math.inf)
                m = x.max(1, keepdim=True).values.nan_to_num(neginf=0.0)
                p = torch.exp(x - m)
                p = p / p.sum(1, keepdim=True).clamp(min=1e-300)
                if c["op"] == "weights":
                    got[h] += p[:, :Nk].sum(0)
                else:
                    out[b, j, live] = p @ (torch.cat([v, s["tail_v"][b, h, :n].double()]) if n else v)
    return got if c["op"] == "weights" else out
