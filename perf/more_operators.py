"""More operators beside the swap-in path, as cases to measure.

Four operators around the rows that the swap-in path moves (a token's row: 512
latent channels and 64 rotary channels, which every attention head shares):

  write    a token's row from its projection: the latent norm, the rotation of the
           rotary channels and the row's form (16 bits, or 8 with a scale a row) in
           one pass, into rows for an append or into each request's context
  read     rows of either form back as values: those of a slot list, or the last
           ones of ragged contexts
  rotate   the norm of each head's queries and keys with the position's rotation
  shared   absorbed latent attention of a batch over a prefix that all requests
           share and over rows of their own

``run`` computes a case in plain torch operations, or with ``own`` through the
library's calls; both get the same state from ``prepare``.
"""
import math

import torch

own = False

LATENT, ROPE, ROW = 512, 64, 576
ROW8_BYTES = 592  # 576 e4m3 values, one fp32 scale, 12 bytes of padding
E4M3_MAX = 448.0
SCALE = (128 + ROPE) ** -0.5
EPS = 1e-6
THETA = 10000.0
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases ---------------------------------------------------------------------------

def _write(name, dtype, cache, new, before=0, staged=False, pairs=True, norm=True):
    """new: tokens of each request; before: rows that each context has already (at random up to this)."""
    return {"name": name, "op": "write", "dtype": dtype, "cache": cache, "new": new, "before": before,
            "staged": staged, "pairs": pairs, "norm": norm}


def _read(name, dtype, cache, out, batch=0, rows=0, entries=0, holes=0.0, lengths=""):
    return {"name": name, "op": "read", "dtype": dtype, "cache": cache, "out": out, "batch": batch,
            "rows": rows, "entries": entries, "holes": holes, "lengths": lengths}


def _rotate(name, dtype, tokens, heads, keys, dim, rope, norm, pairs):
    return {"name": name, "op": "rotate", "dtype": dtype, "tokens": tokens, "heads": heads, "keys": keys,
            "dim": dim, "rope": rope, "norm": norm, "pairs": pairs}


def _shared(name, dtype, cache, batch, positions, heads, prefix, rows, entries=0, ragged=False, partial=False):
    """entries 0: own rows are the first ones of ragged (or full) contexts; partial: requests share
    prefixes of different lengths, one of them none."""
    return {"name": name, "op": "shared", "dtype": dtype, "cache": cache, "batch": batch,
            "positions": positions, "heads": heads, "prefix": prefix, "rows": rows, "entries": entries,
            "ragged": ragged, "partial": partial}


def listed():
    return [
        # a decode step of 64 requests: their tokens' 8-bit rows, for the append to the device tail
        _write("write8_append_b64", "bf16", "e4m3", ",".join(["1"] * 64), before=65536, staged=True),
        # a few prompts, one of them a next chunk, into 16-bit contexts on the device
        _write("write16_ragged", "fp16", "16", "1,37,2000,5,777", before=4096, pairs=False),
        # prompts of 65,536 tokens in all into 8-bit contexts
        _write("write8_prompts_64k", "bf16", "e4m3", ",".join(["8192"] * 8)),
        # what a step of the 64-request workload resolved, as values for another kernel
        _read("read8_slots_b64_k2048", "bf16", "e4m3", "bf16", 64, 4608, 2048),
        # cached contexts as the rows of a prompt's next chunk
        _read("read16_contexts", "bf16", "16", "bf16", 4, 16384, lengths="15872,1,333,4097"),
        # one step's indices with padding, in fp32
        _read("read8_slots_b3_k77", "fp16", "e4m3", "fp32", 3, 512, 77, holes=0.1),
        # a decode step of 64 requests, all heads on one GPU: the queries' rotary channels
        _rotate("rotate_b64_h128", "bf16", 64, 128, 0, 192, 64, False, True),
        # a prompt's queries and keys with their norms
        _rotate("rotate_norm_8192", "bf16", 8192, 32, 8, 128, 128, True, False),
        # a single token, heads split over eight GPUs
        _rotate("rotate_norm_1", "fp16", 1, 16, 1, 192, 64, True, True),
        # 64 requests behind one long system prompt, heads split over eight GPUs
        _shared("shared_b64_h16_16k", "bf16", "16", 64, 1, 16, 16384, 512, ragged=True),
        # the same batch with all heads, over 32K shared tokens
        _shared("shared_b64_h128_32k", "bf16", "16", 64, 1, 128, 32768, 256),
        # draft positions of few requests that share parts of an 8-bit prefix and list their own rows
        _shared("shared8_b5_p3_h20", "bf16", "e4m3", 5, 3, 20, 3001, 700, 333, partial=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def _unnamed(case):
    return {k: v for k, v in case.items() if k != "name"}


def draw(rng):
    op = rng.choice(("write", "read", "rotate", "shared", "shared"))
    dtype, cache = rng.choice(("bf16", "bf16", "fp16")), rng.choice(("16", "e4m3"))
    if op == "write":
        batch = _log(rng, 1, 256)
        new = [_log(rng, 1, 65536 // batch) for _ in range(batch)]
        if rng.random() < 0.3:
            new = [1] * batch
        return _unnamed(_write("", dtype, cache, ",".join(map(str, new)), rng.choice((0, 100, 1000)),
                               rng.random() < 0.4, rng.random() < 0.5, rng.random() < 0.8))
    if op == "read":
        out = rng.choice((dtype, "fp32"))
        if rng.random() < 0.5:
            entries = _log(rng, 1, 2048)
            batch = _log(rng, 1, max(1, min(256, 64 * 2048 // (2 * entries))))
            return _unnamed(_read("", dtype, cache, out, batch, entries + _log(rng, 1, 2048), entries,
                                  holes=rng.choice((0.0, 0.1, 0.5)) if batch > 1 else 0.0))
        batch = _log(rng, 1, 16)
        lengths = [_log(rng, 1, 32768 // batch) for _ in range(batch)]
        return _unnamed(_read("", dtype, cache, out, batch, max(lengths) + rng.choice((0, 3, 100)),
                              lengths=",".join(map(str, lengths))))
    if op == "rotate":
        kind = rng.choice(("bf16", "fp16", "fp32"))
        dim = rng.choice((64, 80, 96, 128, 192, 256, 576))
        heads, keys = rng.choice((1, 8, 16, 20, 32, 64, 128)), rng.choice((0, 1, 4, 8))
        rope = rng.choice([r for r in (32, 64, 128, dim) if r <= dim])
        tokens = _log(rng, 1, max(1, 8192 * 40 * 128 // ((heads + keys) * dim * BYTES[kind] // 2)))
        return _unnamed(_rotate("", kind, tokens, heads, keys, dim, rope, rng.random() < 0.6,
                                rng.random() < 0.5))
    heads, positions = rng.choice((1, 8, 16, 20, 32, 64, 100, 128)), rng.choice((1, 1, 1, 2, 3))
    batch = _log(rng, 1, 256)
    prefix = _log(rng, 1, max(1, min(65536, 64 * 128 * 32768 // (4 * batch * positions * heads))))
    rows = _log(rng, positions, 2048)
    entries = rng.choice((0, 0, _log(rng, 1, rows)))
    return _unnamed(_shared("", dtype, cache, batch, positions, heads, prefix, rows, entries,
                            ragged=rng.random() < 0.5, partial=rng.random() < 0.4))


def _counts(text):
    return [int(x) for x in text.split(",")]


# ---- inputs --------------------------------------------------------------------------

def _pack8(rows):
    """Rows in 8 bits: 576 e4m3 values and their fp32 scale (the row's largest magnitude over 448)."""
    rows = rows.float()
    scale = rows.abs().amax(-1, keepdim=True) / E4M3_MAX
    q = (rows / scale).to(torch.float8_e4m3fn).view(torch.uint8)
    pad = torch.zeros(rows.shape[:-1] + (12,), dtype=torch.uint8, device=rows.device)
    return torch.cat([q, scale.view(torch.uint8), pad], -1)


def _frequencies(rope, dev):
    return (THETA ** (-torch.arange(rope // 2, dtype=torch.float64, device=dev) * 2 / rope)).float()


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dtype):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(to)

    def whole(low, high, *shape):  # low .. high
        return torch.randint(low, high + 1, shape, generator=gen, device=dev, dtype=torch.int32)

    def weights(n):
        return (1 + 0.1 * torch.randn(n, generator=gen, device=dev)).to(dtype)

    def form(rows):
        return rows if case["cache"] == "16" else _pack8(rows)

    def starts(counts):
        return torch.tensor([0] + counts, dtype=torch.int64, device=dev).cumsum(0).to(torch.int32)

    state = {"case": case}
    if case["op"] == "write":
        new = _counts(case["new"])
        n = sum(new)
        state["x"] = normal(n, ROW)
        if case["norm"]:
            state["weight"] = weights(LATENT)
        state["inv_freq"] = _frequencies(ROPE, dev)
        state["start"] = starts(new)
        counts = torch.tensor(new, device=dev)
        state["lengths"] = whole(0, case["before"], len(new)) + counts.to(torch.int32)
        request = torch.repeat_interleave(torch.arange(len(new), device=dev), counts)
        end = state["start"].long()[request + 1]
        state["positions"] = (state["lengths"].long()[request] - end
                              + torch.arange(n, device=dev)).to(torch.int32)
        shape = (n,) if case["staged"] else (len(new), max(new) + case["before"])
        if case["cache"] == "e4m3":
            state["rows"] = torch.zeros(shape + (ROW8_BYTES,), dtype=torch.uint8, device=dev)
        else:
            state["rows"] = torch.zeros(shape + (ROW,), dtype=dtype, device=dev)
    elif case["op"] == "read":
        B, N, K = case["batch"], case["rows"], case["entries"]
        state["rows"] = form(normal(B, N, ROW))
        if K:
            slots = torch.rand((B, N), generator=gen, device=dev).topk(K, dim=1).indices
            if case["holes"]:
                hole = torch.rand((B, K), generator=gen, device=dev) < case["holes"]
                hole[-1] = True
                slots = slots.masked_fill(hole, -1)
            state["slots"] = slots.to(torch.int32)
            state["out"] = torch.empty((B, K, ROW), dtype=TYPES[case["out"]], device=dev)
        else:
            lengths = _counts(case["lengths"])
            state["lengths"] = torch.tensor(lengths, dtype=torch.int32, device=dev)
            state["start"] = starts(lengths)
            state["out"] = torch.empty((sum(lengths), ROW), dtype=TYPES[case["out"]], device=dev)
    elif case["op"] == "rotate":
        n, dim = case["tokens"], case["dim"]
        state["positions"] = whole(0, 131071, n)
        state["inv_freq"] = _frequencies(case["rope"], dev)
        for name, heads in (("q", case["heads"]), ("k", case["keys"])):
            if heads:
                state[name] = normal(n, heads, dim)
                state[name + "_out"] = torch.empty_like(state[name])
                if case["norm"]:
                    state[name + "_weight"] = weights(dim)
    else:
        B, P, H, N, K = (case[k] for k in ("batch", "positions", "heads", "rows", "entries"))
        state["q"] = normal(B, P, H, ROW)
        state["prefix"] = form(normal(case["prefix"], ROW))
        state["rows"] = form(normal(B, N, ROW))
        if case["partial"]:
            state["prefix_lengths"] = whole(0, case["prefix"], B)
            state["prefix_lengths"][-1] = 0
        if K:
            slots = torch.rand((B * P, N), generator=gen, device=dev).topk(K, dim=1).indices
            if case["ragged"]:  # lists of different lengths, padded
                some = whole(0, K, B * P, 1)
                slots = slots.masked_fill(torch.arange(K, device=dev) >= some, -1)
            state["slots"] = slots.view(B, P, K).to(torch.int32)
        else:
            state["lengths"] = whole(P, N, B) if case["ragged"] else whole(N, N, B)
        state["out"] = torch.empty((B, P, H, LATENT), dtype=dtype, device=dev)
        state["lse"] = torch.empty((B, P, H), dtype=torch.float32, device=dev)
    return state


# ---- one pass ------------------------------------------------------------------------

def run(state):
    kind = state["case"]["op"]
    if own:
        return {"write": _own_write, "read": _own_read, "rotate": _own_rotate, "shared": _own_shared}[kind](state)
    return {"write": _plain_write, "read": _plain_read, "rotate": _plain_rotate, "shared": _plain_shared}[kind](state)


def _row_format(hs, case):
    return hs.HS_ROWS_E4M3 if case["cache"] == "e4m3" else hs.HS_ROWS_16BIT


def _rotation(hs, case):
    return hs.HS_ROTATE_PAIRS if case["pairs"] else hs.HS_ROTATE_HALVES


def _written(rows):
    """The cache as what it holds: 16-bit values, or e4m3 values and their scales."""
    if rows.dtype != torch.uint8:
        return [rows]
    return [rows[..., :ROW].view(torch.float8_e4m3fn), rows[..., ROW:ROW + 4].view(torch.float32)]


def _own_write(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    case = state["case"]
    place = {} if case["staged"] else {"start": state["start"], "lengths": state["lengths"]}
    hs.hs_latent_write(state["x"], state["rows"], weight=state.get("weight"), eps=EPS,
                       positions=state["positions"], inv_freq=state["inv_freq"],
                       rotation=_rotation(hs, case), row_format=_row_format(hs, case),
                       stream=torch.cuda.current_stream(), **place)
    return _written(state["rows"])


def _own_read(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    place = {k: state[k] for k in ("slots", "start", "lengths") if k in state}
    hs.hs_latent_read(state["rows"], state["out"], row_format=_row_format(hs, state["case"]),
                      stream=torch.cuda.current_stream(), **place)
    return state["out"]


def _own_rotate(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    hs.hs_norm_rotate(state["q"], state["q_out"], k=state.get("k"), k_out=state.get("k_out"),
                      q_weight=state.get("q_weight"), k_weight=state.get("k_weight"), eps=EPS,
                      positions=state["positions"], inv_freq=state["inv_freq"],
                      rotation=_rotation(hs, state["case"]), stream=torch.cuda.current_stream())
    return [state[k] for k in ("q_out", "k_out") if k in state]


def _own_shared(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    case = state["case"]
    if "workspace" not in state:  # kept for the program's life, as the handle is
        n = hs.hs_latent_attend_shared_workspace(case["batch"], case["positions"], case["heads"],
                                                 case["entries"] or case["rows"], case["prefix"],
                                                 row_format=_row_format(hs, case))
        state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    hs.hs_latent_attend_shared(state["q"], state["prefix"], state["rows"], state["out"], SCALE,
                               slots=state.get("slots"), lengths=state.get("lengths"),
                               prefix_lengths=state.get("prefix_lengths"),
                               row_format=_row_format(hs, case), lse=state["lse"],
                               workspace=state["workspace"], stream=torch.cuda.current_stream())
    return state["out"], state["lse"]


def _wide(rows):
    """Rows of either form as fp32 [..., 576]."""
    if rows.dtype != torch.uint8:
        return rows.float()
    scale = rows[..., ROW:ROW + 4].contiguous().view(torch.float32)
    return rows[..., :ROW].contiguous().view(torch.float8_e4m3fn).float() * scale


def _turned(x, positions, inv_freq, pairs):
    """x [n, ..., rope] turned by its positions; angles in 64 bits."""
    angle = positions.double()[:, None] * inv_freq.double()
    angle = angle.view((x.shape[0],) + (1,) * (x.dim() - 2) + (-1,))
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    if pairs:
        a, b = x[..., 0::2], x[..., 1::2]
        return torch.stack([a * cos - b * sin, a * sin + b * cos], -1).flatten(-2)
    a, b = x.chunk(2, -1)
    return torch.cat([a * cos - b * sin, a * sin + b * cos], -1)


def _places(start, lengths, n):
    """Request and row of each of n ragged tokens, which are their contexts' last."""
    t = torch.arange(n, device=start.device)
    start = start.long()
    request = torch.searchsorted(start, t, right=True) - 1
    return request, lengths.long()[request] - start[request + 1] + t


def _plain_write(state):
    case, x, rows = state["case"], state["x"].float(), state["rows"]
    latent = x[:, :LATENT]
    if case["norm"]:
        latent = latent * torch.rsqrt((latent * latent).mean(-1, keepdim=True) + EPS) * state["weight"].float()
    y = torch.cat([latent, _turned(x[:, LATENT:], state["positions"], state["inv_freq"], case["pairs"])], -1)
    if case["cache"] == "e4m3":
        scale = y.abs().amax(-1, keepdim=True) / E4M3_MAX
        q = (y / scale.masked_fill(scale == 0, 1.0)).to(torch.float8_e4m3fn).view(torch.uint8)
        y = torch.cat([q, scale.view(torch.uint8)], -1)
    else:
        y = y.to(rows.dtype)
    if case["staged"]:
        rows[:, :y.shape[1]] = y
    else:
        request, row = _places(state["start"], state["lengths"], y.shape[0])
        rows[..., :y.shape[1]][request, row] = y
    return _written(rows)


def _plain_read(state):
    case, rows, out = state["case"], state["rows"], state["out"]
    if case["entries"]:
        slots = state["slots"].long()
        request = torch.arange(case["batch"], device=slots.device)[:, None]
        found = _wide(rows[request, slots.clamp(min=0)]).masked_fill((slots < 0)[..., None], 0.0)
    else:
        request, row = _places(state["start"], state["lengths"], out.shape[0])
        found = _wide(rows[request, row])
    return found.to(out.dtype)


def _plain_rotate(state):
    case, found = state["case"], []
    for name in ("q", "k"):
        if name not in state:
            continue
        x = state[name].float()
        if case["norm"]:
            x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * state[name + "_weight"].float()
        at = case["dim"] - case["rope"]
        turned = _turned(x[..., at:], state["positions"], state["inv_freq"], case["pairs"])
        found.append(torch.cat([x[..., :at], turned], -1).to(state[name].dtype))
    return found


def _own_rows(state):
    """Scores' mask [B, P, 1, K] and own rows of a batch: listed, or the first of each context."""
    B, P, N = (state["case"][k] for k in ("batch", "positions", "rows"))
    dev = state["q"].device
    if "slots" in state:
        slots = state["slots"].long()
        request = torch.arange(B, device=dev)[:, None, None]
        return (slots >= 0)[:, :, None, :], state["rows"][request, slots.clamp(min=0)]
    last = state["lengths"].long()[:, None] - P + torch.arange(P, device=dev)
    return (torch.arange(N, device=dev) <= last[:, :, None])[:, :, None, :], state["rows"][:, None]


def _plain_shared(state):
    case, q = state["case"], state["q"].float()
    prefix = _wide(state["prefix"])
    mask, rows = _own_rows(state)
    rows = _wide(rows)
    first = torch.matmul(q, prefix.t()) * SCALE                      # [B, P, H, prefix]
    if case["partial"]:
        seen = torch.arange(case["prefix"], device=q.device) < state["prefix_lengths"].long()[:, None]
        first = first.masked_fill(~seen[:, None, None, :], -math.inf)
    second = (torch.matmul(q, rows.transpose(-1, -2)) * SCALE).masked_fill(~mask, -math.inf)
    top = torch.maximum(first.amax(-1, keepdim=True), second.amax(-1, keepdim=True))
    top = top.masked_fill(top == -math.inf, 0.0)
    first, second = torch.exp(first - top), torch.exp(second - top)
    total = first.sum(-1, keepdim=True) + second.sum(-1, keepdim=True)
    o = torch.matmul(first, prefix[:, :LATENT]) + torch.matmul(second, rows[..., :LATENT])
    o = o / total.masked_fill(total == 0, 1.0)
    return o.to(state["q"].dtype), (torch.log(total) + top).squeeze(-1)


# ---- the definitions in 64 bits ------------------------------------------------------

def _wide64(rows):
    if rows.dtype != torch.uint8:
        return rows.double()
    values = rows[..., :ROW].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
    return values * rows[..., ROW:ROW + 4].contiguous().view(torch.float32).double()


def exact(case, seed):
    state = prepare(case, seed)
    return {"write": _exact_write, "read": _exact_read, "rotate": _exact_rotate,
            "shared": _exact_shared}[case["op"]](state)


def _rotation64(x, positions, inv_freq, pairs):
    """Each pair of channels as a complex number, times exp(i angle)."""
    turn = torch.polar(torch.ones((), dtype=torch.float64, device=x.device),
                       positions.double()[:, None] * inv_freq.double())
    half = x.shape[-1] // 2
    re, im = (x[..., 0::2], x[..., 1::2]) if pairs else (x[..., :half], x[..., half:])
    z = torch.complex(re.contiguous(), im.contiguous()) * turn.view(turn.shape[:1] + (1,) * (x.dim() - 2) + (half,))
    if pairs:
        return torch.view_as_real(z).reshape(x.shape)
    return torch.cat([z.real, z.imag], -1)


def _exact_write(state):
    case, x = state["case"], state["x"].double()
    latent = x[:, :LATENT]
    if case["norm"]:
        latent = state["weight"].double() * latent / torch.sqrt(latent.square().mean(1, keepdim=True) + EPS)
    y = torch.cat([latent, _rotation64(x[:, LATENT:], state["positions"], state["inv_freq"], case["pairs"])], 1)
    parts = [y]
    if case["cache"] == "e4m3":
        scale = y.abs().amax(1, keepdim=True) / E4M3_MAX
        parts = [(y / scale.clamp(min=1e-300)).float().to(torch.float8_e4m3fn).double(), scale]
    if case["staged"]:
        return parts
    whole = [torch.zeros(state["rows"].shape[:2] + p.shape[1:], dtype=torch.float64, device=x.device) for p in parts]
    at = 0
    for b, n in enumerate(_counts(case["new"])):
        end = int(state["lengths"][b])
        for w, p in zip(whole, parts):
            w[b, end - n:end] = p[at:at + n]
        at += n
    return whole


def _exact_read(state):
    case, rows = state["case"], state["rows"]
    if case["entries"]:
        out = torch.zeros(state["out"].shape, dtype=torch.float64, device=rows.device)
        for b in range(case["batch"]):
            there = state["slots"][b] >= 0
            out[b][there] = _wide64(rows[b][state["slots"][b][there].long()])
        return out
    return torch.cat([_wide64(rows[b, :n]) for b, n in enumerate(_counts(case["lengths"]))])


def _exact_rotate(state):
    case, found = state["case"], []
    at = case["dim"] - case["rope"]
    for name in ("q", "k"):
        if name in state:
            y = state[name].double()
            if case["norm"]:
                y = state[name + "_weight"].double() * y / torch.sqrt(y.square().mean(-1, keepdim=True) + EPS)
            y[..., at:] = _rotation64(y[..., at:].clone(), state["positions"], state["inv_freq"], case["pairs"])
            found.append(y)
    return found


def _exact_shared(state):
    case, q = state["case"], state["q"]
    B, P, H, _ = q.shape
    out = torch.zeros((B, P, H, LATENT), dtype=torch.float64, device=q.device)
    lse = torch.full((B, P, H), -math.inf, dtype=torch.float64, device=q.device)
    for b in range(B):
        shared = int(state["prefix_lengths"][b]) if case["partial"] else case["prefix"]
        prefix = _wide64(state["prefix"][:shared])
        for p in range(P):
            if "slots" in state:
                picked = state["slots"][b, p]
                mine = state["rows"][b][picked[picked >= 0].long()]
            else:
                mine = state["rows"][b, :max(0, int(state["lengths"][b]) - P + 1 + p)]
            k = torch.cat([prefix, _wide64(mine)])
            if k.shape[0]:
                s = SCALE * (q[b, p].double() @ k.t())
                out[b, p] = torch.softmax(s, -1) @ k[:, :LATENT]
                lse[b, p] = torch.logsumexp(s, -1)
    return out, lse


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    wide = BYTES[case["dtype"]]
    row = (ROW8_BYTES - 12) if case.get("cache") == "e4m3" else ROW * wide
    if case["op"] == "write":
        n = sum(_counts(case["new"]))
        return {"bytes": n * (ROW * wide + row + 4), "flops": n * (4 * LATENT + 6 * ROPE)}
    if case["op"] == "read":
        n = case["batch"] * case["entries"] or sum(_counts(case["lengths"]))
        read = n * (1 - case["holes"]) * row + (4 * n if case["entries"] else 0)
        return {"bytes": int(read + n * ROW * BYTES[case["out"]]), "flops": n * ROW}
    if case["op"] == "rotate":
        n = case["tokens"] * (case["heads"] + case["keys"])
        return {"bytes": 2 * n * case["dim"] * wide + 4 * case["tokens"],
                "flops": n * (4 * case["dim"] * case["norm"] + 3 * case["rope"])}
    B, P, H, N, K = (case[k] for k in ("batch", "positions", "heads", "rows", "entries"))
    # lengths and lists that are drawn between 0 and all: one half on average
    prefix = case["prefix"] * (0.5 if case["partial"] else 1.0)
    mine = (K or N) * (0.5 if case["ragged"] else 1.0)
    read = case["prefix"] * row + B * min(N, mine * (P if K else 1)) * row + (4 * B * P * K if K else 4 * B)
    return {"bytes": int(read + B * P * H * ((ROW + LATENT) * wide + 4)),
            "flops": int(2 * B * P * H * (prefix + mine) * (ROW + LATENT))}
