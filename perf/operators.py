"""The operators beside the swap-in path, as cases to measure.

Three operators, over the rows that the swap-in path moves (a token's row: 512
latent channels and 64 rotary channels, which every attention head shares):

  attend   absorbed latent attention of single tokens or draft positions, over
           rows picked by a slot list (what a resolve step returns) or over the
           first rows of each request; rows in 16 bits or in 8 with a scale a row
  prefill  expanded latent attention of ragged prompts (keys and values of each
           head are products of the latent with two weights), causal
  norm     root-mean-square norm, with the residual's addition, into 16, 32 or
           8 bits with scales; it also writes the 8-bit rows of the cache

``run`` computes a case in plain torch operations, or with ``own`` through the
library's calls; both get the same state from ``prepare``.
"""
import math

import torch

own = False

LATENT, ROPE, ROW, HEAD = 512, 64, 576, 128
ROW8_BYTES = 592  # 576 e4m3 values, one fp32 scale, 12 bytes of padding
E4M3_MAX = 448.0
SCALE = (HEAD + ROPE) ** -0.5
EPS = 1e-6
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}


# ---- cases ---------------------------------------------------------------------------

def _attend(name, dtype, cache, batch, positions, heads, rows, entries=0, lengths="", holes=0.0):
    return {"name": name, "op": "attend", "dtype": dtype, "cache": cache, "batch": batch,
            "positions": positions, "heads": heads, "rows": rows, "entries": entries,
            "lengths": lengths, "holes": holes}


def _prefill(name, dtype, cache, heads, queries, keys):
    return {"name": name, "op": "prefill", "dtype": dtype, "cache": cache, "heads": heads,
            "queries": queries, "keys": keys}


def _norm(name, dtype, out, tokens, dim, carry=0, residual=False, group=0, cache_rows=False):
    return {"name": name, "op": "norm", "dtype": dtype, "out": out, "tokens": tokens, "dim": dim,
            "carry": carry, "residual": residual, "group": group, "cache_rows": cache_rows}


def listed():
    return [
        # one request's decode step: 256 indices in a buffer of 512 slots, the latency end
        _attend("attend_b1_k256", "bf16", "16", 1, 1, 16, 512, 256),
        # the decode step of the 64-request, 64K-context workload, all heads on one GPU
        _attend("attend_b64_k2048_h128", "bf16", "16", 64, 1, 128, 4096, 2048),
        # the 256-request workload (hot buffer and 512 tail slots), heads split over eight GPUs,
        # with the cache in 8 bits
        _attend("attend8_b256_k2048_h16", "bf16", "e4m3", 256, 1, 16, 4608, 2048),
        # draft positions with ragged, padded lists; one list is all padding
        _attend("attend_b7_p3_k333_h20", "bf16", "16", 7, 3, 20, 1500, 333, holes=0.1),
        # contexts still whole on the device: ragged lengths, one of a single token
        _attend("attend_dense_b4_h64", "fp16", "16", 4, 1, 64, 32768, lengths="32768,1,20001,777"),
        # one long context of 128K tokens in 8 bits
        _attend("attend8_dense_128k_h128", "bf16", "e4m3", 1, 1, 128, 131072, lengths="131072"),
        # short prompts taken together
        _prefill("prefill_short_h16", "bf16", "16", 16, "1,37,200,5", "1,37,200,5"),
        # one long prompt
        _prefill("prefill_8k_h32", "bf16", "16", 32, "8192", "8192"),
        # the next 512 tokens of a prompt whose first 15,872 rows are cached in 8 bits
        _prefill("prefill8_chunk_h16", "fp16", "e4m3", 16, "512", "16384"),
        # a single token's hidden state
        _norm("norm_1x4096", "bf16", "same", 1, 4096, residual=True),
        # a prompt's hidden states, into 8 bits with a scale for each 128 channels
        _norm("norm8_8192x4096", "bf16", "e4m3", 8192, 4096, residual=True, group=128),
        # a prompt's cache rows: the latent normed, the rotary channels as they are, one scale a row
        _norm("norm8_rows_5000", "bf16", "e4m3", 5000, LATENT, carry=ROPE, cache_rows=True),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "prefill", "norm"))
    if op == "attend":
        dtype, cache = rng.choice(("bf16", "bf16", "fp16")), rng.choice(("16", "e4m3"))
        heads = rng.choice((1, 8, 16, 20, 32, 64, 100, 128))
        positions = rng.choice((1, 1, 1, 2, 3))
        if rng.random() < 0.6:
            entries = _log(rng, 1, 2048)
            rows = entries + _log(rng, 1, 4096)
            batch = _log(rng, 1, max(1, min(256, (64 * 2048 * 128) // (positions * heads * entries),
                                            (256 * 4608) // rows)))
            holes = rng.choice((0.0, 0.05, 0.5)) if batch * positions > 1 and entries >= 32 else 0.0
            return {k: v for k, v in _attend("", dtype, cache, batch, positions, heads, rows, entries,
                                             holes=holes).items() if k != "name"}
        batch = _log(rng, 1, 16)
        most = max(1, min(131072, 4 * 131072 // batch, 131072 * 128 // (batch * positions * heads)))
        lengths = [_log(rng, 1, most) for _ in range(batch)]
        return {k: v for k, v in _attend("", dtype, cache, batch, positions, heads, max(lengths),
                                         lengths=",".join(map(str, lengths))).items() if k != "name"}
    if op == "prefill":
        heads = rng.choice((2, 8, 16, 32))
        batch = _log(rng, 1, 8)
        queries = [_log(rng, 1, 6144 // batch) for _ in range(batch)]
        keys = [q + rng.choice((0, 0, _log(rng, 1, 2048 // batch))) for q in queries]
        return {k: v for k, v in _prefill("", rng.choice(("bf16", "bf16", "fp16")),
                                          rng.choice(("16", "16", "e4m3")), heads,
                                          ",".join(map(str, queries)),
                                          ",".join(map(str, keys))).items() if k != "name"}
    if rng.random() < 0.3:
        return {k: v for k, v in _norm("", rng.choice(("bf16", "fp16")), "e4m3", _log(rng, 1, 16384),
                                       LATENT, carry=ROPE, cache_rows=True).items() if k != "name"}
    dim = _log(rng, 48, 16384)
    if rng.random() < 0.7:
        dim = -(-dim // 64) * 64
    tokens = _log(rng, 1, max(1, 8192 * 4096 // (2 * dim)))
    out = rng.choice(("same", "e4m3"))
    return {k: v for k, v in _norm("", rng.choice(("bf16", "fp16", "fp32")), out, tokens, dim,
                                   residual=rng.random() < 0.7,
                                   group=rng.choice((0, 128)) if out == "e4m3" else 0).items() if k != "name"}


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


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(seed)
    dtype = TYPES[case["dtype"]]

    def normal(*shape, std=1.0, to=dtype):
        return (torch.randn(shape, generator=gen, device=dev) * std).to(to)

    state = {"case": case}
    if case["op"] == "attend":
        B, P, H, N, K = (case[k] for k in ("batch", "positions", "heads", "rows", "entries"))
        state["q"] = normal(B, P, H, ROW)
        rows = normal(B, N, ROW)
        state["rows"] = rows if case["cache"] == "16" else _pack8(rows)
        if K:
            # K different slots of the N in random order, as a resolve step returns them
            slots = torch.rand((B * P, N), generator=gen, device=dev).topk(K, dim=1).indices
            if case["holes"]:
                hole = torch.rand((B * P, K), generator=gen, device=dev) < case["holes"]
                hole[-1] = True
                slots = slots.masked_fill(hole, -1)
            state["slots"] = slots.view(B, P, K).to(torch.int32)
        else:
            state["lengths"] = torch.tensor(_counts(case["lengths"]), dtype=torch.int32, device=dev)
        state["out"] = torch.empty((B, P, H, LATENT), dtype=dtype, device=dev)
        state["lse"] = torch.empty((B, P, H), dtype=torch.float32, device=dev)
    elif case["op"] == "prefill":
        H, nq, nk = case["heads"], _counts(case["queries"]), _counts(case["keys"])
        state["q"] = normal(sum(nq), H, HEAD + ROPE)
        rows = normal(sum(nk), ROW)
        state["rows"] = rows if case["cache"] == "16" else _pack8(rows)
        state["w_uk"] = normal(H, HEAD, LATENT, std=LATENT ** -0.5)
        state["w_uv"] = normal(H, HEAD, LATENT, std=LATENT ** -0.5)
        starts = [torch.tensor([0] + n, dtype=torch.int32, device=dev).cumsum(0).to(torch.int32)
                  for n in (nq, nk)]
        state["q_start"], state["k_start"] = starts
        state["out"] = torch.empty((sum(nq), H, HEAD), dtype=dtype, device=dev)
    else:
        n, d, carry = case["tokens"], case["dim"], case["carry"]
        state["x"] = normal(n, d + carry)
        state["weight"] = (1 + 0.1 * torch.randn(d, generator=gen, device=dev)).to(dtype)
        if case["residual"]:
            state["residual"] = normal(n, d, std=2.0)
            state["residual_out"] = torch.empty_like(state["residual"])
        if case["cache_rows"]:
            cache = torch.zeros((n, ROW8_BYTES), dtype=torch.uint8, device=dev)
            state["out"] = cache[:, :ROW].view(torch.float8_e4m3fn)
            state["scales"] = cache[:, ROW:ROW + 4].view(torch.float32)
        elif case["out"] == "e4m3":
            groups = -(-d // case["group"]) if case["group"] else 1
            state["out"] = torch.empty((n, d), dtype=torch.float8_e4m3fn, device=dev)
            state["scales"] = torch.empty((n, groups), dtype=torch.float32, device=dev)
        else:
            state["out"] = torch.empty((n, d), dtype=dtype, device=dev)
    return state


# ---- one pass ------------------------------------------------------------------------

def run(state):
    case = state["case"]
    if own:
        return {"attend": _own_attend, "prefill": _own_prefill, "norm": _own_norm}[case["op"]](state)
    return {"attend": _plain_attend, "prefill": _plain_prefill, "norm": _plain_norm}[case["op"]](state)


def _row_format(hs, case):
    return hs.HS_ROWS_E4M3 if case["cache"] == "e4m3" else hs.HS_ROWS_16BIT


def _own_attend(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    case = state["case"]
    if "workspace" not in state:  # kept for the program's life, as the handle is
        n = hs.hs_latent_attend_workspace(case["batch"], case["positions"], case["heads"],
                                          case["entries"] or case["rows"])
        state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    hs.hs_latent_attend(state["q"], state["rows"], state["out"], SCALE, slots=state.get("slots"),
                        lengths=state.get("lengths"), row_format=_row_format(hs, case),
                        lse=state["lse"], workspace=state["workspace"],
                        stream=torch.cuda.current_stream())
    return state["out"], state["lse"]


def _own_prefill(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    case = state["case"]
    if "workspace" not in state:
        n = hs.hs_latent_prefill_workspace(state["rows"].shape[0], case["heads"])
        state["workspace"] = torch.empty(n, dtype=torch.uint8, device="cuda")
    hs.hs_latent_prefill(state["q"], state["rows"], state["w_uk"], state["w_uv"], state["q_start"],
                         state["k_start"], state["out"], SCALE, row_format=_row_format(hs, case),
                         workspace=state["workspace"], stream=torch.cuda.current_stream())
    return state["out"]


def _own_norm(state):
    from hierarchical_kv_cache_hs_gb300 import hs
    case = state["case"]
    hs.hs_rms_norm(state["x"], state["weight"], state["out"], EPS, residual=state.get("residual"),
                   residual_out=state.get("residual_out"), carry=case["carry"],
                   scales=state.get("scales"), group=case["group"],
                   stream=torch.cuda.current_stream())
    return [state[k] for k in ("out", "scales", "residual_out") if k in state]


def _wide(rows):
    """Rows of either form as fp32 [..., 576]."""
    if rows.dtype != torch.uint8:
        return rows.float()
    scale = rows[..., ROW:ROW + 4].contiguous().view(torch.float32)
    return rows[..., :ROW].contiguous().view(torch.float8_e4m3fn).float() * scale


def _softmax_values(s, mask, v):
    """softmax(s) v over the allowed entries, and the log of the sum; nothing allowed gives 0 and -inf."""
    s = s.masked_fill(~mask, -math.inf)
    top = s.amax(-1, keepdim=True)
    top = top.masked_fill(top == -math.inf, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / total.masked_fill(total == 0, 1.0)
    return o, (torch.log(total) + top).squeeze(-1)


def _plain_attend(state):
    case, q = state["case"], state["q"].float()
    B, P, H, N, K = (case[k] for k in ("batch", "positions", "heads", "rows", "entries"))
    if K:
        slots = state["slots"].long()
        mask = (slots >= 0)[:, :, None, :]
        request = torch.arange(B, device=q.device)[:, None, None]
        k = _wide(state["rows"][request, slots.clamp(min=0)])            # [B, P, K, 576]
    else:
        at = torch.arange(N, device=q.device)
        last = state["lengths"].long()[:, None] - P + torch.arange(P, device=q.device)
        mask = (at <= last[:, :, None])[:, :, None, :]
        k = _wide(state["rows"])[:, None]
    s = torch.matmul(q, k.transpose(-1, -2)) * SCALE
    o, lse = _softmax_values(s, mask, k[..., :LATENT])
    return o.to(state["q"].dtype), lse


def _plain_prefill(state):
    q, rows = state["q"].float().transpose(0, 1), _wide(state["rows"])      # [H, Tq, 192]
    latent, rope = rows[:, :LATENT], rows[:, LATENT:]
    k = torch.matmul(latent, state["w_uk"].float().transpose(1, 2))         # [H, Tk, 128]
    v = torch.matmul(latent, state["w_uv"].float().transpose(1, 2))
    s = torch.matmul(q[..., :HEAD], k.transpose(1, 2)) + torch.matmul(q[..., HEAD:], rope.t())
    q0, k0 = state["q_start"].long(), state["k_start"].long()
    tq = torch.arange(q.shape[1], device=q.device)
    tk = torch.arange(rows.shape[0], device=q.device)
    rq = torch.searchsorted(q0, tq, right=True) - 1
    rk = torch.searchsorted(k0, tk, right=True) - 1
    # query i of a request sees its keys up to i + (keys - queries)
    last = k0[rq + 1] - (q0[rq + 1] - tq)
    mask = (rq[:, None] == rk[None]) & (tk[None] <= last[:, None])
    o, _ = _softmax_values(s * SCALE, mask[None], v)
    return o.transpose(0, 1).to(state["q"].dtype)


def _plain_norm(state):
    case = state["case"]
    x, d = state["x"].float(), case["dim"]
    out = []
    h, carried = x[:, :d], x[:, d:]
    if case["residual"]:
        h = h + state["residual"].float()
        out.append(h.to(state["x"].dtype))
    y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * state["weight"].float()
    if case["out"] == "same":
        return [y.to(state["x"].dtype)] + out
    y = torch.cat([y, carried], -1)
    n, width = y.shape
    group = case["group"] or width
    groups = -(-width // group)
    cells = torch.nn.functional.pad(y, (0, groups * group - width)).view(n, groups, group)
    scales = cells.abs().amax(-1) / E4M3_MAX
    q = cells / scales.masked_fill(scales == 0, 1.0)[..., None]
    q = q.view(n, groups * group)[:, :width].to(torch.float8_e4m3fn)
    return [q, scales] + out


# ---- the definitions in 64 bits ------------------------------------------------------

def _wide64(rows):
    if rows.dtype != torch.uint8:
        return rows.double()
    values = rows[..., :ROW].contiguous().view(torch.float8_e4m3fn).to(torch.float64)
    return values * rows[..., ROW:ROW + 4].contiguous().view(torch.float32).double()


def exact(case, seed):
    state = prepare(case, seed)
    return {"attend": _exact_attend, "prefill": _exact_prefill, "norm": _exact_norm}[case["op"]](state)


def _exact_attend(state):
    q, rows = state["q"], state["rows"]
    B, P, H, _ = q.shape
    out = torch.zeros((B, P, H, LATENT), dtype=torch.float64, device=q.device)
    lse = torch.full((B, P, H), -math.inf, dtype=torch.float64, device=q.device)
    counts = _counts(state["case"]["lengths"]) if state["case"]["lengths"] else None
    for b in range(B):
        for p in range(P):
            if counts is None:
                picked = state["slots"][b, p]
                k = rows[b, picked[picked >= 0].long()]
            else:
                k = rows[b, :max(0, counts[b] - P + 1 + p)]
            if k.shape[0]:
                k = _wide64(k)
                s = SCALE * (k @ q[b, p].double().t())                    # [n, H]
                lse[b, p] = torch.logsumexp(s, 0)
                out[b, p] = torch.exp(s - lse[b, p]).t() @ k[:, :LATENT]
    return out, lse


def _exact_prefill(state):
    nq, nk = _counts(state["case"]["queries"]), _counts(state["case"]["keys"])
    out = torch.zeros(state["out"].shape, dtype=torch.float64, device=state["q"].device)
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        rows = _wide64(state["rows"][k0:k0 + m])
        allowed = torch.ones((n, m), dtype=torch.bool, device=rows.device).tril(m - n)
        some = allowed.any(1)
        for h in range(state["case"]["heads"]):
            k = torch.cat([rows[:, :LATENT] @ state["w_uk"][h].double().t(), rows[:, LATENT:]], 1)
            s = SCALE * (state["q"][q0:q0 + n, h].double() @ k.t())
            p = torch.softmax(torch.where(allowed, s, -math.inf)[some], -1)
            out[q0:q0 + n, h][some] = p @ rows[:, :LATENT] @ state["w_uv"][h].double().t()
        q0, k0 = q0 + n, k0 + m
    return out


def _exact_norm(state):
    case, d = state["case"], state["case"]["dim"]
    h = state["x"][:, :d].double()
    if case["residual"]:
        h = h + state["residual"].double()
    y = state["weight"].double() * h / torch.sqrt(h.square().mean(1, keepdim=True) + EPS)
    y = torch.cat([y, state["x"][:, d:].double()], 1)
    found = [y]
    if case["out"] == "e4m3":
        pieces = torch.split(y, case["group"] or y.shape[1], dim=1)
        scales = [p.abs().amax(1, keepdim=True) / E4M3_MAX for p in pieces]
        found = [torch.cat([(p / s.clamp(min=1e-300)).float().to(torch.float8_e4m3fn).double()
                            for p, s in zip(pieces, scales)], 1), torch.cat(scales, 1)]
    return found + ([h] if case["residual"] else [])


# ---- what a pass cannot do without ---------------------------------------------------

def work(case):
    wide = BYTES[case["dtype"]]
    if case["op"] == "norm":
        n, d, width = case["tokens"], case["dim"], case["dim"] + case["carry"]
        moved = n * width * wide + d * wide
        if case["residual"]:
            moved += 2 * n * d * wide
        if case["out"] == "e4m3":
            moved += n * width + 4 * n * (-(-width // case["group"]) if case["group"] else 1)
        else:
            moved += n * width * wide
        return {"bytes": moved, "flops": 6 * n * d}
    row = ROW8_BYTES if case["cache"] == "e4m3" else ROW * wide
    if case["op"] == "attend":
        B, P, H, N, K = (case[k] for k in ("batch", "positions", "heads", "rows", "entries"))
        if K:
            pairs = B * P * K * (1 - case["holes"])
            read = B * min(N, P * K * (1 - case["holes"])) * row + 4 * B * P * K
        else:
            counts = _counts(case["lengths"])
            pairs = sum(max(0, n - P + 1 + p) for n in counts for p in range(P))
            read = sum(counts) * row + 4 * B
        return {"bytes": int(read + B * P * H * ((ROW + LATENT) * wide + 4)),
                "flops": int(2 * pairs * H * (ROW + LATENT))}
    H, nq, nk = case["heads"], _counts(case["queries"]), _counts(case["keys"])
    pairs = sum(max(0, m - n + 1 + i) for n, m in zip(nq, nk) for i in range(n))
    return {"bytes": sum(nk) * row + sum(nq) * H * (HEAD + ROPE + HEAD) * wide + 2 * H * HEAD * LATENT * wide,
            "flops": 2 * pairs * H * (HEAD + ROPE + HEAD) + 2 * sum(nk) * LATENT * 2 * HEAD * H}
