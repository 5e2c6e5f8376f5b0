"""What is measured of the operators around the multi-LoRA delta and the cache of a serving step: the
root-mean-square norm of a layer's input (with the residual's addition and an 8-bit output beside the one
that the adapters take), the product with a base weight held in 4 bits, which the delta is added to, and the
step's keys and values appended to the paged cache, rotated by their positions on the way, with its queries.

``run`` computes each in its plain form (elementary torch operations, 32 bits or more, rounded once
at the end), or, where ``own`` is true, makes the calls of the package. ``exact`` is the operator's
definition in 64 bits.

Cache layout, per page and key/value head, in groups of 16 tokens (element (t, d) of a group, with
c = 16 bytes of elements):
  k  [D / c][16][c]   16-byte pieces of d, tokens inside
  v  [D][16]          tokens innermost, in the order 0-3, 8-11, 4-7, 12-15
and one fp32 scale per (page, head, token) for the 8-bit formats. A value is code * scale.

A 4-bit weight is [N][ceil(K / 2)] bytes, the even k in the low bits, with a scale (and a zero point) for every
`group` values of k of a row; its values are scale * (code - zero) or, of e2m1 codes (32 values of k to a scale
that is a power of two, one byte), 2^(scale - 127) * e2m1(code).
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
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]
EPS = 1e-5


# ---------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------
def norm(name, dtype, rows, heads, width, residual, quantise):
    return {"name": name, "kind": "norm", "dtype": dtype, "rows": rows, "heads": heads,
            "width": width, "residual": residual, "quantise": quantise}


def append(name, dtype, cache, B, q, past, heads, kv_heads, dim, page, rotary, interleaved=False):
    return {"name": name, "kind": "append", "dtype": dtype, "cache": cache, "B": B, "q_lo": q[0],
            "q_hi": q[1], "past_lo": past[0], "past_hi": past[1], "heads": heads,
            "kv_heads": kv_heads, "dim": dim, "page": page, "rotary": rotary,
            "interleaved": interleaved}


def product(name, dtype, form, T, N, K, group, zero=False):
    return {"name": name, "kind": "product", "dtype": dtype, "form": form, "T": T, "N": N, "K": K,
            "group": group, "zero": zero}


def listed():
    return [
        # the input of a layer for one user's next token, of an 8192-wide model
        norm("norm one bf16", "bf16", 1, 1, 8192, True, ""),
        # the decode batch, its rows also quantised for a base weight of 8 bits
        norm("norm 256 e4m3", "bf16", 256, 1, 4096, True, "e4m3"),
        # a step of prompt chunks of an 8192-wide model, rows and codes
        norm("norm chunks i8", "bf16", 8192, 1, 8192, True, "i8"),
        # keys of a step normed head by head, odd numbers of rows, fp32
        norm("norm heads f32", "f32", 1003, 7, 80, False, ""),
        # one user's next token: queries rotated, its key and value appended
        append("append one bf16", "bf16", "bf16", 1, (1, 1), (1000, 1000), 32, 8, 128, 16, 128),
        # the decode batch's, quantised
        append("append 256 e4m3", "bf16", "e4m3", 256, (1, 1), (0, 512), 64, 8, 128, 64, 128),
        # prompt chunks, quantised
        append("append chunks i8", "bf16", "i8", 16, (64, 1024), (0, 1024), 32, 8, 128, 32, 128),
        # a small fp32 model with uneven heads, a part of each rotated in neighbouring pairs
        append("append part f32", "f32", "f32", 4, (1, 40), (0, 600), 14, 2, 80, 16, 32, True),
        # one user's next token through an 8192-wide base weight of 4 bits
        product("product one i4", "bf16", "i4", 1, 8192, 8192, 128),
        # a few users' (or drafted) tokens through a wide one of small floats
        product("product 16 e2m1", "bf16", "e2m1", 16, 28672, 8192, 32),
        # a small fp32 model with odd sizes, zero points, short groups
        product("product odd f32", "f32", "i4", 5, 1003, 2750, 64, True),
        # a prompt's chunk through the output projection of the mixed batch, zero points
        product("product chunk i4", "bf16", "i4", 2048, 11008, 4096, 128, True),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.99)))))))


def draw(rng):
    kind = rng.choice(["norm", "append", "product"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    if kind == "norm":
        heads = rng.choice([1, 1, 1, 2, 7, 8, 32])
        width = rng.choice([64, 80, 96, 128, 192, 256]) if heads > 1 else _log(rng, 64, 16384)
        rows = _log(rng, 1, min(8192, (32_000_000 if dtype == "bf16" else 16_000_000) // (heads * width)))
        c = norm("", dtype, rows, heads, width, rng.random() < 0.7, rng.choice(["", "e4m3", "i8"]))
    elif kind == "append":
        cache = rng.choice([dtype, dtype, "e4m3", "i8"])
        dim, page = rng.choice([64, 80, 96, 128, 128, 128, 192, 256]), rng.choice([16, 32, 64, 128])
        kv_heads, B = rng.choice([1, 2, 4, 8]), _log(rng, 1, 256)
        new = rng.choice([1, _log(rng, 1, max(1, 8192 // B))])
        past = _log(rng, 1, max(1, 16384 // B))
        rotary = rng.choice([dim, dim, dim - 16, 16 * ((dim // 2 + 15) // 16)])
        c = append("", dtype, cache, B, (max(1, new // 4), new), (past // 4, past),
                   kv_heads * rng.choice([1, 2, 4, 5, 7, 8]), kv_heads, dim, page, rotary, rng.random() < 0.3)
    else:
        form, group = rng.choice([("i4", 32), ("i4", 64), ("i4", 128), ("i4", 128), ("i4", 256), ("e2m1", 32)])
        N, K = _log(rng, 100, 28672), _log(rng, 100, 16384)
        N, K = (N, K) if rng.random() < 0.3 else (-(-N // 64) * 64, -(-K // 64) * 64)
        T = rng.choice([1, _log(rng, 1, 64), _log(rng, 1, 2048)])
        T = min(T, max(1, (90_000_000_000 if dtype == "bf16" else 30_000_000_000) // (N * K)))
        c = product("", dtype, form, T, N, K, group, form == "i4" and rng.random() < 0.5)
    del c["name"]
    return c


def _spread(lo, hi, n, phase):
    """n whole numbers over [lo, hi], ragged, the same ones for the same case."""
    return [lo + int((hi - lo + 1) * ((0.5 + phase + 0.6180339887498949 * i) % 1.0))
            for i in range(n)]


def _lengths(case):
    """New tokens and past tokens of each sequence."""
    return (_spread(case["q_lo"], case["q_hi"], case["B"], 0.0),
            _spread(case["past_lo"], case["past_hi"], case["B"], 0.3))


def _groups(case):
    return -(-case["K"] // case["group"])


def work(case):
    e = BYTES[case["dtype"]]
    if case["kind"] == "norm":
        rows, W = case["rows"] * case["heads"], case["width"]
        each = 2 * e + (2 * e if case["residual"] else 0) + (1 if case["quantise"] else 0)
        return {"bytes": rows * (W * each + (4.0 if case["quantise"] else 0.0)) + W * e, "flops": 5.0 * rows * W}
    if case["kind"] == "product":
        T, N, K, g = case["T"], case["N"], case["K"], _groups(case)
        scale = 1 if case["form"] == "e2m1" else e + (1 if case["zero"] else 0)
        return {"bytes": N * ((K + 1) // 2) + float(N) * g * scale + float(e) * T * (K + N),
                "flops": 2.0 * T * N * K}
    q, _ = _lengths(case)
    T, H, D, c = sum(q), case["kv_heads"], case["dim"], BYTES[case["cache"]]
    # (queries that are not rotated are rows of the output all the same)
    return {"bytes": T * (2.0 * case["heads"] * D * e + 2.0 * H * (D * (e + c) + (4 if case["cache"] in TOP else 0))
                          + 4.0 * case["rotary"]),
            "flops": 3.0 * T * case["rotary"] * (case["heads"] + H)}


# ---------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------
def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(int(seed) + 1)
    return {"norm": _prepare_norm, "append": _prepare_append, "product": _prepare_product}[case["kind"]](
        case, g, TYPES[case["dtype"]])


def _prepare_norm(case, g, dtype):
    shape = (case["rows"], case["heads"], case["width"])
    W = case["width"]
    # a few channels of a residual stream are much larger than the rest
    channel = 1 + 30 * (torch.rand(W, generator=g, device=DEVICE) < 0.005)
    st = {"case": case, "x": torch.randn(shape, generator=g, device=DEVICE).to(dtype),
          "weight": (1 + 0.2 * torch.randn(W, generator=g, device=DEVICE)).to(dtype), "residual": None}
    if case["residual"]:
        st["residual"] = (3 * torch.randn(shape, generator=g, device=DEVICE) * channel).to(dtype)
    return st


def _prepare_append(case, g, dtype):
    q_len, past = _lengths(case)
    n, ps, H, D = len(q_len), case["page"], case["kv_heads"], case["dim"]
    kv_len = [a + b for a, b in zip(q_len, past)]
    need = [-(-v // ps) for v in kv_len]
    pages, form = sum(need) + 3, case["cache"]
    ids = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    table = torch.full((n, max(need)), -1, dtype=torch.int32)
    first = [sum(need[:b]) for b in range(n)]
    held = torch.arange(max(need))[None, :] < torch.tensor(need)[:, None]
    where = (torch.tensor(first)[:, None] + torch.arange(max(need))[None, :])[held]
    table = table.to(DEVICE)
    table[held.to(DEVICE)] = ids[where.to(DEVICE)]
    start = [sum(q_len[:b]) for b in range(n + 1)]
    T, rot = start[-1], case["rotary"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device=DEVICE)  # noqa: E731
    st = {"case": case, "q_start": i32(start), "kv_len": i32(kv_len), "table": table, "tokens": T,
          "max_q": max(q_len), "max_kv": max(kv_len)}
    st["seq"] = torch.repeat_interleave(torch.arange(n, device=DEVICE), i32(q_len).long())
    # a cache in use: K and V as earlier steps left them
    c = 16 // BYTES[form]
    for part, shape in (("k", (pages, H, ps // 16, D // c, 16, c)), ("v", (pages, H, ps // 16, D, 16))):
        x = torch.randn(shape, generator=g, device=DEVICE)
        if form in TOP:
            x = x.mul_(TOP[form] / 2.8).clamp_(-TOP[form], TOP[form])
            x = x.round_() if form == "i8" else x
            amax = torch.rand((pages, H, ps), generator=g, device=DEVICE) + 2.3
            st[part + "_scale"] = amax / TOP[form]
        st[part] = x.to(TYPES[form])
    # the projection of the step's tokens, keys with a few large channels
    width = (case["heads"] + 2 * H) * D
    qkv = torch.randn((T, width), generator=g, device=DEVICE)
    channel = 1 + 5 * (torch.rand(H * D, generator=g, device=DEVICE) < 0.04)
    qkv[:, case["heads"] * D:(case["heads"] + H) * D] *= channel
    q, k, v = qkv.to(dtype).split([case["heads"] * D, H * D, H * D], 1)
    st["q"], st["k_new"], st["v_new"] = q.unflatten(1, (-1, D)), k.unflatten(1, (-1, D)), v.unflatten(1, (-1, D))
    # cosines and sines of every position, from angles in 64 bits
    angle = torch.arange(max(kv_len), device=DEVICE).double()[:, None] * (
        10000.0 ** (-torch.arange(0, rot, 2, device=DEVICE).double() / rot))
    st["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    return st


def _prepare_product(case, g, dtype):
    T, N, K, G = case["T"], case["N"], case["K"], _groups(case)
    codes = torch.randint(0, 256, (N, (K + 1) // 2), generator=g, device=DEVICE, dtype=torch.uint8)
    scale = (0.5 + torch.rand((N, G), generator=g, device=DEVICE)) * (0.2 * K ** -0.5)
    scale = (127 + torch.log2(scale).round()).to(torch.uint8) if case["form"] == "e2m1" else scale.to(dtype)
    st = {"case": case, "codes": codes, "scale": scale, "zero": None,
          "x": torch.randn((T, K), generator=g, device=DEVICE).to(dtype)}
    if case["zero"]:
        st["zero"] = torch.randint(6, 11, (N, G), generator=g, device=DEVICE, dtype=torch.uint8)
    return st


# ---------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------
def run(state):
    kind = state["case"]["kind"]
    if own:
        return _own(state, kind)
    return {"norm": _plain_norm, "append": _plain_append, "product": _plain_product}[kind](state)


def _own(st, kind):
    import segmented_gather_gemv_amd as sg
    case = st["case"]
    if kind == "norm":
        got = sg.sgmv_rms_norm(st["x"], st["weight"], EPS, residual=st["residual"],
                               quantise=TYPES[case["quantise"]] if case["quantise"] else None)
        return {"out": got.out, "residual": got.residual, "codes": got.codes, "scale": got.scale}
    if kind == "product":
        if "plan" not in st:  # the weight as a serving program keeps it
            st["plan"] = sg.sgmv_base_pack(st["codes"], st["scale"], st["zero"], K=case["K"], group=case["group"],
                                           format=sg.BASE_I4 if case["form"] == "i4" else sg.BASE_E2M1,
                                           dtype=st["x"].dtype)
        return {"y": sg.sgmv_base_product(st["x"], st["plan"])}
    if "plan" not in st:  # the handles a serving loop keeps beside its cache and its batch
        st["plan"] = (sg.sgmv_kv_wrap(st["k"], st["v"], st.get("k_scale"), st.get("v_scale")),
                      sg.sgmv_kv_batch(st["q_start"], st["kv_len"], st["table"], st["tokens"],
                                       st["max_q"], st["max_kv"]))
    cache, batch = st["plan"]
    q = sg.sgmv_kv_append(st["q"], st["k_new"], st["v_new"], batch, cache, st["cos_sin"],
                          interleaved=case["interleaved"])
    return {"q": q, "k": st["k"], "v": st["v"], "k_scale": st.get("k_scale"), "v_scale": st.get("v_scale")}


def _codes(x, form):
    """Codes of rows, and their maxima. In 64 bits: what is next to a border has to fall right."""
    amax = x.double().abs().amax(-1, keepdim=True)
    y = x.double() * TOP[form] / torch.where(amax == 0, 1.0, amax)
    if form == "i8":
        code = y.round().to(torch.int8)
    else:  # 3 bits after the leading one, 2^-9 the smallest step
        step = torch.ldexp(torch.ones_like(y), torch.frexp(y)[1].clamp(min=-5) - 4)
        code = ((y / step).round() * step).to(TYPES[form])
    return code, amax[..., 0].float()


def _plain_norm(st):
    case, dtype = st["case"], st["x"].dtype
    h = st["x"].float()
    if case["residual"]:
        h = h + st["residual"].float()
    y = h * st["weight"].float()
    r = 1.0 / torch.sqrt(h.square().mean(-1, keepdim=True) + EPS)
    out = {"out": (y * r).to(dtype), "residual": h.to(dtype) if case["residual"] else None, "codes": None,
           "scale": None}
    if case["quantise"]:
        out["codes"], amax = _codes(y, case["quantise"])
        out["scale"] = amax * r[..., 0] / TOP[case["quantise"]]
    return out


def _weight(st, dtype):
    """The weight's values [N, K]."""
    case = st["case"]
    code = torch.stack([st["codes"] & 15, st["codes"] >> 4], 2).flatten(1)[:, :case["K"]]
    at = torch.arange(case["K"], device=DEVICE) // case["group"]
    if case["form"] == "e2m1":
        return torch.tensor(E2M1, dtype=dtype, device=DEVICE)[code.long()] * torch.exp2(st["scale"].to(dtype) - 127)[:, at]
    return (code.to(dtype) - (8 if st["zero"] is None else st["zero"].to(dtype)[:, at])) * st["scale"].to(dtype)[:, at]


def _plain_product(st):
    return {"y": (st["x"].float() @ _weight(st, torch.float32).T).to(st["x"].dtype)}


def _rotated(x, c, s, interleaved):
    """Rows x [T, H, D], each pair of the first values turned by its angle."""
    rot = 2 * c.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2], x[..., rot // 2:rot])
    y = [a * c - b * s, b * c + a * s]
    y = torch.stack(y, -1).flatten(-2) if interleaved else torch.cat(y, -1)
    return torch.cat([y, x[..., rot:]], -1)


def _positions(st):
    """Of each row of the step."""
    return st["kv_len"].long()[st["seq"]] + torch.arange(st["tokens"], device=DEVICE) - st["q_start"].long()[st["seq"] + 1]


def _place(st, part, x, pos, stored):
    """Puts rows x [T, H, D] into a part of the cache."""
    case, ps = st["case"], st["case"]["page"]
    H, D, c = case["kv_heads"], case["dim"], 16 // BYTES[case["cache"]]
    page, off = st["table"].long()[st["seq"], pos // ps], pos % ps
    if part == "k":
        stored[page, :, off // 16, :, off % 16, :] = x.reshape(-1, H, D // c, c)
    else:
        stored[page, :, off // 16, :, torch.tensor(ORDER, device=DEVICE)[off % 16]] = x
    return page, off


def _plain_append(st):
    case, form, dtype = st["case"], st["case"]["cache"], st["q"].dtype
    pos = _positions(st)
    c, s = st["cos_sin"][pos][:, None, :].chunk(2, -1)
    raw = torch.uint8 if BYTES[form] == 1 else TYPES[form]
    rows = {"k": _rotated(st["k_new"].float(), c, s, case["interleaved"]), "v": st["v_new"].float()}
    for part, x in rows.items():
        amax = None
        if form in TOP:
            x, amax = _codes(x, form)
        page, off = _place(st, part, x.to(TYPES[form]).view(raw), pos, st[part].view(raw))
        if form in TOP:
            st[part + "_scale"][page, :, off] = amax / TOP[form]
    return {"q": _rotated(st["q"].float(), c, s, case["interleaved"]).to(dtype), "k": st["k"], "v": st["v"],
            "k_scale": st.get("k_scale"), "v_scale": st.get("v_scale")}


# ---------------------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------------------
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
    st = prepare(case, seed)
    if case["kind"] == "norm":
        h = st["x"].double()
        if case["residual"]:
            h = h + st["residual"].double()
        y = h * st["weight"].double() / (h.square().sum(-1, keepdim=True) / case["width"] + EPS).sqrt()
        out = {"out": y, "residual": h if case["residual"] else None, "codes": None, "scale": None}
        if case["quantise"]:
            top, amax = TOP[case["quantise"]], y.abs().amax(-1, keepdim=True)
            out["codes"] = _nearest(y * top / amax) if case["quantise"] == "e4m3" else None  # int8: whole numbers
            out["scale"] = amax[..., 0] / top
        return out
    if case["kind"] == "product":
        y = torch.empty((case["T"], case["N"]), dtype=torch.float64, device=DEVICE)
        x, g, half = st["x"].double(), case["group"], torch.tensor(E2M1, dtype=torch.float64, device=DEVICE)
        for n in range(0, case["N"], 4096):
            code = torch.empty((len(st["codes"][n:n + 4096]), case["K"]), dtype=torch.float64, device=DEVICE)
            for odd in (0, 1):
                part = (st["codes"][n:n + 4096] // 16 if odd else st["codes"][n:n + 4096] % 16)[:, :(case["K"] + 1 - odd) // 2]
                code[:, odd::2] = half[part.long()] if case["form"] == "e2m1" else part.double()
            total = 0
            for i in range(_groups(case)):
                at = slice(g * i, min(g * i + g, case["K"]))
                w = code[:, at]
                if case["form"] == "i4":
                    w = w - (8.0 if st["zero"] is None else st["zero"][n:n + 4096, i, None].double())
                scale = st["scale"][n:n + 4096, i].double()
                total = total + (x[:, at] @ w.T) * (torch.exp2(scale - 127) if case["form"] == "e2m1" else scale)
            y[:, n:n + 4096] = total
        return {"y": y}
    # turned as complex numbers, one angle for each pair
    pos, rot = _positions(st), case["rotary"]
    turn = torch.complex(*st["cos_sin"][pos].double().chunk(2, 1))[:, None, :]
    i = torch.arange(rot // 2, device=DEVICE)
    a, b = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
    got = {}
    for name in ("q", "k_new"):
        x = st[name].double()
        z = torch.complex(x[..., a], x[..., b]) * turn
        x[..., a], x[..., b] = z.real, z.imag
        got[name] = x
    out = {"q": got["q"], "k_scale": None, "v_scale": None}
    form = case["cache"]
    for part, x in (("k", got["k_new"]), ("v", st["v_new"].double())):
        stored = st[part].double()
        if form in TOP:
            amax = x.abs().amax(-1, keepdim=True)
            x = _nearest(x * TOP[form] / amax) if form == "e4m3" else x
            scale = st[part + "_scale"].double()
        page, off = _place(st, part, x, pos, stored)
        out[part] = None if form == "i8" else stored  # whole numbers
        if form in TOP:
            scale[page, :, off] = amax[..., 0] / TOP[form]
            out[part + "_scale"] = scale
    return out
