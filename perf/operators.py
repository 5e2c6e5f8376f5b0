"""What is measured of the serving operators behind the multi-LoRA delta: the paged key/value cache
(quantised as it is written, and read back), the attention of a step's new tokens over it, and the
check of drafted tokens against the target's probabilities.

``run`` computes each in its plain form (elementary torch operations, 32 bits or more, rounded once
at the end), or, where ``own`` is true, makes the calls of the package. ``exact`` is the operator's
definition in 64 bits.

Cache layout, per page and key/value head, in groups of 16 tokens (element (t, d) of a group, with
c = 16 bytes of elements):
  k  [D / c][16][c]   16-byte pieces of d, tokens inside
  v  [D][16]          tokens innermost, in the order 0-3, 8-11, 4-7, 12-15
and one fp32 scale per (page, head, token) for the 8-bit formats. A value is code * scale.
"""
import math

import torch

own = False

DEVICE = "cuda"
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
         "i8": torch.int8}
TOP = {"e4m3": 448.0, "i8": 127.0}
BYTES = {"f32": 4, "bf16": 2, "e4m3": 1, "i8": 1}
ORDER = [0, 1, 2, 3, 8, 9, 10, 11, 4, 5, 6, 7, 12, 13, 14, 15]  # its own inverse


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def attention(name, dtype, cache, B, q, past, heads, kv_heads, dim, page, window=0, ones=0):
    return {"name": name, "kind": "attention", "dtype": dtype, "cache": cache, "B": B,
            "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1], "ones": ones,
            "heads": heads, "kv_heads": kv_heads, "dim": dim, "page": page, "window": window}


def cached(name, dtype, cache, B, q, past, kv_heads, dim, page, back):
    return {"name": name, "kind": "cache", "dtype": dtype, "cache": cache, "B": B,
            "q_lo": q[0], "q_hi": q[1], "past_lo": past[0], "past_hi": past[1], "ones": 0,
            "kv_heads": kv_heads, "dim": dim, "page": page, "back": back}


def verify(name, dtype, B, drafts, vocab, point):
    return {"name": name, "kind": "verify", "dtype": dtype, "B": B, "n_lo": drafts[0],
            "n_hi": drafts[1], "vocab": vocab, "point": point}


def listed():
    return [
        # one user's reply being generated: the latency of a single token
        attention("decode one bf16", "bf16", "bf16", 1, (1, 1), (1000, 1000), 32, 8, 128, 16),
        # a full decode batch, one token of each of 256 sequences, heads of an 8192-wide model
        attention("decode 256 bf16", "bf16", "bf16", 256, (1, 1), (128, 4096), 64, 8, 128, 64),
        # long documents being answered from a quantised cache
        attention("decode long e4m3", "bf16", "e4m3", 16, (1, 1), (8001, 64003), 64, 8, 128, 128),
        # drafted tokens scored in one step: a few new tokens each, int8 cache
        attention("drafts i8", "bf16", "i8", 64, (2, 6), (500, 8000), 32, 8, 128, 32),
        # a step that mixes prompt chunks with decoding sequences
        attention("mixed step bf16", "bf16", "bf16", 4, (300, 700), (0, 2048), 32, 8, 128, 64,
                  ones=28),
        # the chunks of eight prompts, heads of an 8192-wide model
        attention("prompt chunks bf16", "bf16", "bf16", 8, (64, 1024), (0, 4096), 64, 8, 128, 16),
        # a late chunk of one long prompt over its quantised cache
        attention("late chunk e4m3", "bf16", "e4m3", 1, (2048, 2048), (14001, 14001), 32, 8, 128,
                  128),
        # a small fp32 model with uneven heads and a sliding window
        attention("small f32 window", "f32", "f32", 4, (1, 40), (0, 600), 14, 2, 80, 16, 256),
        # a decode step's 256 new tokens quantised into the cache, and read back
        cached("append e4m3", "bf16", "e4m3", 256, (1, 1), (0, 512), 8, 128, 64, "new"),
        # prompt chunks quantised into the cache, and whole sequences read back (to move them)
        cached("store and fetch i8", "bf16", "i8", 16, (64, 1024), (0, 4096), 8, 128, 32, "all"),
        # one user's drafts checked
        verify("verify one f32", "f32", 1, (4, 4), 32000, False),
        # a full batch's drafts checked, large vocabulary
        verify("verify 256 f32", "f32", 256, (1, 5), 131072, False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "attention", "cache", "verify"])
    if kind == "verify":
        B, vocab, lo = _log(rng, 1, 256), _log(rng, 1000, 131072), rng.randint(0, 3)
        c = verify("", rng.choice(["f32", "bf16"]), B, (lo, lo + rng.randint(1, 5 - lo)), vocab,
                   rng.random() < 0.3)
        del c["name"]
        return c
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    cache = rng.choice([dtype, dtype, "e4m3", "i8"])
    dim, page = rng.choice([64, 80, 96, 128, 128, 128, 192, 256]), rng.choice([16, 32, 64, 128, 256])
    kv_heads = rng.choice([1, 2, 4, 8])
    if kind == "cache":
        B = _log(rng, 1, 256)
        new = _log(rng, 1, max(1, 8192 // B))
        past = _log(rng, 1, max(1, 32768 // B))
        c = cached("", dtype, cache, B, (max(1, new // 4), new), (past // 4, past), kv_heads, dim,
                   page, rng.choice(["new", "all"]))
        del c["name"]
        return c
    group = rng.choice([1, 2, 4, 5, 7, 8])
    most = 2_000_000_000 // (2 * kv_heads * dim * BYTES[cache])  # cached tokens in all
    form = rng.choice(["decode", "drafts", "chunks", "mixed"])
    window, ones = rng.choice([0, 0, 0, rng.randint(1, 2000)]), 0
    if form in ("decode", "drafts"):
        B = _log(rng, 1, 256)
        past = _log(rng, 16, min(65536, most // B))
        q = (1, 1) if form == "decode" else (1, rng.randint(2, 9))
        past = (past // 4, past)
    else:
        B = _log(rng, 1, 8 if dim <= 128 else 4)
        most = _log(rng, 17, (1024 if dtype == "bf16" else 256) // (2 if form == "mixed" else 1))
        past = rng.randint(0, 4096 if B <= 4 else 2048)
        q, past = (max(1, most // 3), most), (past // 3, past)
        ones = _log(rng, 1, 24) if form == "mixed" else 0
    c = attention("", dtype, cache, B, q, past, kv_heads * group, kv_heads, dim, page, window, ones)
    del c["name"]
    return c


def _spread(lo, hi, n, phase):
    """n whole numbers over [lo, hi], ragged, the same ones for the same case."""
    return [lo + int((hi - lo + 1) * ((0.5 + phase + 0.6180339887498949 * i) % 1.0))
            for i in range(n)]


def _lengths(case):
    """New tokens and past tokens of each sequence; the single-token sequences come last."""
    n = case["B"] + case["ones"]
    q = _spread(case["q_lo"], case["q_hi"], case["B"], 0.0) + [1] * case["ones"]
    return q, _spread(case["past_lo"], case["past_hi"], n, 0.3)


def _drafts(case):
    return _spread(case["n_lo"], case["n_hi"], case["B"], 0.0)


def _pairs(q, past, window):
    """(token, visible token) pairs of one sequence, and the tokens visible to any of them."""
    seen = q * past + q * (q + 1) // 2
    most = past + q
    if window:
        seen = sum(min(window, past + i + 1) for i in range(q))
        most = min(past + q, window + q - 1)
    return seen, most


def work(case):
    if case["kind"] == "verify":
        n, e = _drafts(case), BYTES[case["dtype"]]
        # a sequence's last row of the target is read whole, and the draft's where one of its
        # drafts was rejected: with about four of five accepted, 1 - 0.8^n of the sequences
        rows = sum(1.0 + (0.0 if case["point"] else 1.0 - 0.8 ** k) for k in n)
        return {"bytes": rows * case["vocab"] * e + 16.0 * sum(n) + 8.0 * case["B"],
                "flops": 3.0 * rows * case["vocab"]}
    q, past = _lengths(case)
    e, c = BYTES[case["dtype"]], BYTES[case["cache"]]
    H, D = case["kv_heads"], case["dim"]
    token = 2.0 * H * (D * c + (4 if case["cache"] in TOP else 0))  # K and V of one token, cached
    if case["kind"] == "cache":
        new = sum(q)
        back = new if case["back"] == "new" else new + sum(past)
        old = 0 if case["back"] == "new" else sum(past)
        return {"bytes": new * (2.0 * H * D * e + token) + old * token + back * 2.0 * H * D * e,
                "flops": 4.0 * (new + back) * H * D}
    got = [_pairs(a, b, case["window"]) for a, b in zip(q, past)]
    return {"bytes": sum(m for _, m in got) * token + sum(q) * case["heads"] * (2.0 * D * e + 4),
            "flops": 4.0 * D * case["heads"] * sum(s for s, _ in got)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def _stored(g, case, pages):
    """A cache in use: K and V of `pages` pages as earlier steps left them."""
    H, D, ps, form = case["kv_heads"], case["dim"], case["page"], case["cache"]
    c = 16 // BYTES[form]
    out = {}
    for part, shape in (("k", (pages, H, ps // 16, D // c, 16, c)), ("v", (pages, H, ps // 16, D, 16))):
        x = torch.randn(shape, generator=g, device=DEVICE, dtype=torch.bfloat16)
        if form in TOP:  # the largest of a row's D normal values is about 2.7 deviations
            x = (x.mul_(TOP[form] / 2.8)).clamp_(-TOP[form], TOP[form])
            x = x.round_().to(torch.int8) if form == "i8" else x.to(TYPES[form])
            amax = torch.rand((pages, H, ps), generator=g, device=DEVICE) + 2.3
            out[part + "_scale"] = amax / TOP[form]
        out[part] = x.to(TYPES[form])
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed) + 1)
    dtype = TYPES[case["dtype"]]
    if case["kind"] == "verify":
        return _prepare_verify(case, g, dtype)
    q_len, past = _lengths(case)
    n, ps, H, D = len(q_len), case["page"], case["kv_heads"], case["dim"]
    kv_len = [a + b for a, b in zip(q_len, past)]
    need = [-(-v // ps) for v in kv_len]
    pages = sum(need) + 3
    ids = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    first = [sum(need[:b]) for b in range(n)]
    held = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    where = (torch.tensor(first)[:, None] + torch.arange(max(need))[None, :])[held]
    table = table.to(DEVICE)
    table[held.to(DEVICE)] = ids[where.to(DEVICE)]
    start = [sum(q_len[:b]) for b in range(n + 1)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEVICE)  # noqa: E731
    st = {"case": case, "q_start": i32(start), "kv_len": i32(kv_len), "table": table,
          "tokens": start[-1], "max_q": max(q_len), "max_kv": max(kv_len),
          **_stored(g, case, pages)}
    st["seq"] = torch.repeat_interleave(torch.arange(n, device=DEVICE), i32(q_len).long())
    if case["kind"] == "attention":
        st["q"] = torch.randn((start[-1], case["heads"], D), generator=g, device=DEVICE).to(dtype)
        return st
    # a few channels of real keys are much larger than the rest
    channel = 1 + 5 * (torch.rand((H, D), generator=g, device=DEVICE) < 0.04)
    st["k_new"] = (torch.randn((start[-1], H, D), generator=g, device=DEVICE) * channel).to(dtype)
    st["v_new"] = torch.randn((start[-1], H, D), generator=g, device=DEVICE).to(dtype)
    back = q_len if case["back"] == "new" else kv_len
    out = [sum(back[:b]) for b in range(n + 1)]
    st["out_start"], st["rows"] = i32(out), out[-1]
    st["row_seq"] = torch.repeat_interleave(torch.arange(n, device=DEVICE), i32(back).long())
    return st


def _prepare_verify(case, g, dtype):
    n, V, B = _drafts(case), case["vocab"], case["B"]
    total = sum(n)
    start = [sum(n[:b]) for b in range(B + 1)]
    seq = torch.repeat_interleave(torch.arange(B, device=DEVICE),
                                  torch.tensor(n, device=DEVICE, dtype=torch.long))
    logits = 2.5 * torch.randn((total + B, V), generator=g, device=DEVICE)
    st = {"case": case, "seq": seq, "max_drafts": max(n),
          "draft_start": torch.tensor(start, dtype=torch.int32, device=DEVICE)}
    row = torch.arange(total, device=DEVICE) + seq
    guess = logits[row] + 0.4 * torch.randn((total, V), generator=g, device=DEVICE)
    guess = torch.softmax(guess, 1)
    st["target"] = torch.softmax(logits, 1).to(dtype)
    ids = torch.multinomial(guess, 1, generator=g)[:, 0] if total else seq
    st["ids"] = ids.to(torch.int32)
    st["draft"] = None if case["point"] else guess.to(dtype)
    st["accept_u"] = torch.rand(total, generator=g, device=DEVICE)
    st["sample_u"] = torch.rand(B, generator=g, device=DEVICE)
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    if kind == "attention":
        return _plain_attention(state)
    return _plain_cache(state) if kind == "cache" else _plain_verify(state)


def _own(st, kind):
    import segmented_gather_gemv_amd as sg
    if kind == "verify":
        tokens, accepted = sg.sgmv_verify_drafts(st["target"], st["draft"], st["ids"],
                                                 st["draft_start"], st["accept_u"],
                                                 st["sample_u"], st["max_drafts"])
        return {"tokens": tokens, "accepted": accepted}
    if "plan" not in st:  # the handles a serving loop keeps beside its cache and its batch
        st["plan"] = (sg.sgmv_kv_wrap(st["k"], st["v"], st.get("k_scale"), st.get("v_scale")),
                      sg.sgmv_kv_batch(st["q_start"], st["kv_len"], st["table"], st["tokens"],
                                       st["max_q"], st["max_kv"]))
    cache, batch = st["plan"]
    if kind == "attention":
        out, lse = sg.sgmv_kv_attention(st["q"], batch, cache, window=st["case"]["window"])
        return {"out": out, "lse": lse}
    sg.sgmv_kv_write(st["k_new"], st["v_new"], batch, cache)
    k, v = sg.sgmv_kv_read(batch, cache, st["out_start"], st["rows"], st["k_new"].dtype)
    return {"k": k, "v": v}


def _rows(code, scale):
    """Values, in 32 bits."""
    return code.float() if scale is None else code.float() * scale[..., None]


def _plain_attention(st):
    case, table = st["case"], st["table"].long()
    H, D, ps, Hq = case["kv_heads"], case["dim"], case["page"], case["heads"]
    n, L, G = table.shape[0], table.shape[1] * ps, Hq // H
    page = table.clamp(min=0)
    order = torch.tensor(ORDER, device=DEVICE)
    # [n, pages, H, ps / 16, ...] -> [n, H, L, D]
    raw = torch.int8 if case["cache"] in TOP else st["k"].dtype
    k = st["k"].view(raw)[page].permute(0, 2, 1, 3, 5, 4, 6).reshape(n, H, L, D)
    v = st["v"].view(raw)[page][..., order].permute(0, 2, 1, 3, 5, 4).reshape(n, H, L, D)
    k, v = k.view(st["k"].dtype), v.view(st["v"].dtype)
    scales = [None, None]
    if case["cache"] in TOP:
        scales = [st[w][page].permute(0, 2, 1, 3).reshape(n, H, L) for w in ("k_scale", "v_scale")]
    k, v = _rows(k, scales[0]), _rows(v, scales[1])
    q_len = (st["q_start"][1:] - st["q_start"][:-1]).long()
    i = torch.arange(st["max_q"], device=DEVICE)
    row = st["q_start"][:-1].long()[:, None] + torch.minimum(i[None, :], q_len[:, None] - 1)
    q = st["q"][row].float().reshape(n, -1, H, G, D).permute(0, 2, 1, 3, 4).reshape(n, H, -1, D)
    s = torch.matmul(q, k.transpose(2, 3)) * (1.0 / math.sqrt(D))
    pos = (st["kv_len"].long() - q_len)[:, None] + i[None, :]  # [n, max_q]
    t = torch.arange(L, device=DEVICE)
    seen = (t <= pos[..., None]) & (t < st["kv_len"][:, None, None])
    seen &= (table >= 0).repeat_interleave(ps, 1)[:, None, :]
    if case["window"]:
        seen &= t > pos[..., None] - case["window"]
    seen = seen.repeat_interleave(G, 1)[:, None]
    s = s.masked_fill_(~seen, -math.inf)
    top = s.amax(-1, keepdim=True)
    p = s.sub_(torch.where(top == -math.inf, 0.0, top)).exp_()
    total = p.sum(-1, keepdim=True)
    out = torch.matmul(p, v) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log())[..., 0].reshape(n, H, -1, G).permute(0, 2, 1, 3).reshape(n, -1, Hq)
    out = out.reshape(n, H, -1, G, D).permute(0, 2, 1, 3, 4).reshape(n, -1, Hq, D)
    at = torch.arange(st["tokens"], device=DEVICE) - st["q_start"][st["seq"]].long()
    return {"out": out[st["seq"], at].to(st["q"].dtype), "lse": lse[st["seq"], at]}


def _quantise(x, form):
    """Codes of rows, and their scales. In 64 bits: what is next to a border has to fall right."""
    amax = x.double().abs().amax(-1, keepdim=True)
    y = x.double() * TOP[form] / torch.where(amax == 0, 1.0, amax)
    if form == "i8":
        code = y.round().to(torch.int8)
    else:  # 3 bits after the leading one, 2^-9 the smallest step
        step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp(min=-5) - 4)
        code = ((y / step).round() * step).to(TYPES[form])
    return code, (amax[..., 0].float() / TOP[form])


def _plain_cache(st):
    case, ps, table = st["case"], st["case"]["page"], st["table"].long()
    H, D, form = case["kv_heads"], case["dim"], case["cache"]
    c = 16 // BYTES[form]
    raw = torch.uint8 if BYTES[form] == 1 else TYPES[form]
    order = torch.tensor(ORDER, device=DEVICE)
    q_start, kv_len = st["q_start"].long(), st["kv_len"].long()
    pos = kv_len[st["seq"]] + torch.arange(st["tokens"], device=DEVICE) - q_start[st["seq"] + 1]
    page, off = table[st["seq"], pos // ps], pos % ps
    kc, vc = st["k"].view(raw), st["v"].view(raw)
    k, v = st["k_new"], st["v_new"]
    if form in TOP:
        (k, st["k_scale"][page, :, off]), (v, st["v_scale"][page, :, off]) = (
            _quantise(k, form), _quantise(v, form))
    kc[page, :, off // 16, :, off % 16, :] = k.view(raw).reshape(-1, H, D // c, c)
    vc[page, :, off // 16, :, order[off % 16]] = v.view(raw)
    # read back
    out_start, seq = st["out_start"].long(), st["row_seq"]
    pos = kv_len[seq] + torch.arange(st["rows"], device=DEVICE) - out_start[seq + 1]
    page, off = table[seq, pos // ps], pos % ps
    k = kc[page, :, off // 16, :, off % 16, :].reshape(-1, H, D).view(TYPES[form])
    v = vc[page, :, off // 16, :, order[off % 16]].view(TYPES[form])
    scales = [st[w][page, :, off] if form in TOP else None for w in ("k_scale", "v_scale")]
    dtype = st["k_new"].dtype
    return {"k": _rows(k, scales[0]).to(dtype), "v": _rows(v, scales[1]).to(dtype)}


def _plain_verify(st):
    target, draft, ids, seq = st["target"], st["draft"], st["ids"].long(), st["seq"]
    start = st["draft_start"].long()
    B, most = start.numel() - 1, st["max_drafts"]
    n = start[1:] - start[:-1]
    each = torch.arange(ids.numel(), device=DEVICE)
    p = target[each + seq, ids].double()
    q = 1.0 if draft is None else draft[each, ids].double()
    taken = torch.zeros((B, most), dtype=torch.long, device=DEVICE)
    taken[seq, each - start[seq]] = (st["accept_u"].double() * q < p).long()
    accepted = taken.cumprod(1).sum(1)
    b = torch.arange(B, device=DEVICE)
    p = target[start[:-1] + b + accepted].double()
    rest = p
    if ids.numel():
        at = (start[:-1] + accepted).clamp(max=ids.numel() - 1)
        out = (accepted < n)[:, None]
        if draft is None:
            rest = p.masked_fill(out & (torch.arange(p.shape[1], device=DEVICE) == ids[at][:, None]), 0)
        else:
            rest = torch.where(out, (p - draft[at].double()).clamp(min=0), p)
    rest = torch.where(rest.sum(1, keepdim=True) > 0, rest, p)
    upto = rest.cumsum(1)
    token = (upto <= upto[:, -1:] * st["sample_u"].double()[:, None]).sum(1)
    token = torch.where(upto[:, -1] > 0, token, -1)
    tokens = torch.full((B, most + 1), -1, dtype=torch.long, device=DEVICE)
    tokens[seq, each - start[seq]] = ids
    i = torch.arange(most + 1, device=DEVICE)
    tokens = torch.where(i < accepted[:, None], tokens, -1)
    tokens = torch.where(i == accepted[:, None], token[:, None], tokens)
    return {"tokens": tokens.to(torch.int32), "accepted": accepted.to(torch.int32)}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
def _token_rows(st, part, b, t):
    """K or V of tokens t of sequence b: [len(t), H, D] in 64 bits, looked up element by element."""
    case = st["case"]
    ps, H, D = case["page"], case["kv_heads"], case["dim"]
    x, c = st[part], 16 // BYTES[case["cache"]]
    page = st["table"][b].long()[t // ps][:, None, None]
    group, r = ((t % ps) // 16)[:, None, None], (t % 16)[:, None, None]
    h, d = torch.arange(H, device=DEVICE)[None, :, None], torch.arange(D, device=DEVICE)[None, None, :]
    bits = x.view(torch.uint8) if case["cache"] == "e4m3" else x
    if part == "k":
        y = bits[page, h, group, d // c, r, d % c]
    else:  # the middle two quads of a group change places
        y = bits[page, h, group, d, r + 4 * ((r // 4) == 1) - 4 * ((r // 4) == 2)]
    y = y.view(x.dtype).double()
    if case["cache"] in TOP:
        y = y * st[part + "_scale"][page[:, 0], h[:, :, 0], (t % ps)[:, None]].double()[..., None]
    return y


def _nearest(y):
    """The e4m3 value next to each y in 64 bits, ties to the even code."""
    codes = torch.arange(127, dtype=torch.uint8, device=DEVICE)
    values = codes.view(torch.float8_e4m3fn).double()
    edge = (values[1:] + values[:-1]) / 2
    a = y.abs()
    low, high = torch.searchsorted(edge, a), torch.searchsorted(edge, a, right=True)
    at = torch.where(low == high, low, torch.where(low % 2 == 0, low, high))
    return values[at] * torch.sign(y)


def exact(case, seed):
    if case["kind"] == "verify":
        return None  # whole numbers
    st = prepare(case, seed)
    q_len, past = _lengths(case)
    H, D = case["kv_heads"], case["dim"]
    first = 0
    parts = []
    for b, (n, m) in enumerate(zip(q_len, past)):
        if case["kind"] == "attention":
            G = case["heads"] // H
            t = torch.arange(m + n, device=DEVICE)
            lo = max(0, m + 1 - case["window"]) if case["window"] else 0
            t = t[lo:]
            k, v = _token_rows(st, "k", b, t), _token_rows(st, "v", b, t)
            q = st["q"][first:first + n].double()
            pos = torch.arange(m, m + n, device=DEVICE)[:, None]
            hide = t[None, :] > pos
            if case["window"]:
                hide = hide | (t[None, :] + case["window"] <= pos)
            out = torch.empty((n, case["heads"], D), dtype=torch.float64, device=DEVICE)
            lse = torch.empty((n, case["heads"]), dtype=torch.float64, device=DEVICE)
            for h in range(case["heads"]):
                s = (q[:, h] @ k[:, h // G].T) / math.sqrt(D)
                s = s.masked_fill(hide, -math.inf)
                lse[:, h] = torch.logsumexp(s, 1)
                out[:, h] = torch.exp(s - lse[:, h, None]) @ v[:, h // G]
            parts.append((out, lse))
        else:
            back = n if case["back"] == "new" else m + n
            t = torch.arange(m + n - back, m, device=DEVICE)
            got = []
            for part in ("k", "v"):
                x = st[part + "_new"][first:first + n].double()
                if case["cache"] in TOP:
                    top = TOP[case["cache"]]
                    amax = x.abs().amax(-1, keepdim=True)
                    x = x * top / amax  # a row of normal values is never all zero
                    x = (torch.round(x) if top == 127.0 else _nearest(x)) * (amax / top)
                got.append(torch.cat([_token_rows(st, part, b, t), x]) if len(t) else x)
            parts.append(tuple(got))
        first += n
    names = ("out", "lse") if case["kind"] == "attention" else ("k", "v")
    return {name: torch.cat([p[i] for p in parts]) for i, name in enumerate(names)}
