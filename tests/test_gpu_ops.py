"""The operators beside the swap-in path against plain 64-bit forms.

Tolerances count roundings to the 16-bit type (each at most half a step,
eps / 2 of the value) and the fp32 sums; the derivation stands at each check.
"""
import math

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

BF, HALF = torch.bfloat16, torch.float16
SCALE = 192 ** -0.5
NAN = float("nan")


@pytest.fixture(scope="module")
def hs():
    from hierarchical_kv_cache_hs_gb300 import hs as mod
    return mod


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape, dtype=BF, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)


def _pack8(rows):
    """Rows in 8 bits: [..., 592] bytes."""
    rows = rows.float()
    scale = rows.abs().amax(-1, keepdim=True) / 448.0
    q = (rows / scale.clamp(min=1e-30)).to(torch.float8_e4m3fn).view(torch.uint8)
    pad = torch.full(rows.shape[:-1] + (12,), 255, dtype=torch.uint8, device=rows.device)
    return torch.cat([q, scale.view(torch.uint8), pad], -1).contiguous()


def _wide(rows, e4m3):
    if not e4m3:
        return rows.double()
    scale = rows[..., 576:580].contiguous().view(torch.float32).double()
    return rows[..., :576].contiguous().view(torch.float8_e4m3fn).double() * scale


def _softmax_ref(s, v):
    """softmax(s) v, log-sum-exp and sum p |v| for s [m, n], v [n, d]; n may be 0."""
    if s.shape[1] == 0:
        zero = torch.zeros((s.shape[0], v.shape[1]), dtype=torch.float64, device=s.device)
        return zero, torch.full((s.shape[0],), -math.inf, dtype=torch.float64, device=s.device), zero
    p = torch.softmax(s, -1)
    return p @ v, torch.logsumexp(s, -1), p @ v.abs()


def _attend_ref(q, rows, picked, e4m3, scale):
    """picked[b][p]: row indices (long tensors)."""
    B, P, H, _ = q.shape
    o = torch.zeros((B, P, H, 512), dtype=torch.float64, device="cuda")
    mean_abs = torch.zeros_like(o)
    lse = torch.zeros((B, P, H), dtype=torch.float64, device="cuda")
    reach = torch.zeros((B, P, H, 1), dtype=torch.float64, device="cuda")
    for b in range(B):
        for p in range(P):
            k = _wide(rows[b][picked[b][p]], e4m3)
            s = scale * (q[b, p].double() @ k.t())
            o[b, p], lse[b, p], mean_abs[b, p] = _softmax_ref(s, k[:, :512])
            if k.shape[0]:
                reach[b, p] = abs(scale) * (q[b, p].double().abs() @ k.abs().t()).amax(-1, keepdim=True)
    return o, lse, mean_abs, reach


def _check_attend(out, lse, ref, dtype):
    o, want_lse, mean_abs, reach = ref
    half = torch.finfo(dtype).eps / 2
    # scores: 576 fp32 additions of terms that sum to at most `reach` in magnitude, each off by a
    # step of fp32 at most; exp, the log, and the sum over the rows add a few steps more
    score = 576 * 2.0 ** -23 * reach + 2.0 ** -18
    # out: its own rounding; each weight rounded once; a score off by e moves the mean by 2 e sum p|v|
    tol = half * o.abs() + (half + 2 * score) * mean_abs + 1e-30
    err = (out.double() - o).abs()
    assert torch.isfinite(out).all()
    assert bool((err <= tol).all()), (err / tol).max().item()
    # roundings are independent: two of at most half a step each, in the 2-norm
    assert err.norm() <= (1.5 * half + 1e-4) * o.norm() + 1e-30, (err.norm() / o.norm()).item()
    empty = want_lse == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    lse_err = (lse.double() - want_lse)[~empty].abs()
    assert (lse_err <= (score.squeeze(-1) + 2.0 ** -21 * want_lse.abs())[~empty]).all()


def _attend(hs, q, rows, scale=SCALE, e4m3=False, stream=None, **kw):
    B, P, H, _ = q.shape
    out = torch.full((B, P, H, 512), NAN, dtype=q.dtype, device="cuda")
    lse = torch.full((B, P, H), NAN, device="cuda")
    slots = kw.get("slots")
    n = slots.shape[-1] if slots is not None else rows.shape[1]
    ws = torch.full((hs.hs_latent_attend_workspace(B, P, H, n),), 255, dtype=torch.uint8, device="cuda")
    hs.hs_latent_attend(q, rows, out, scale, lse=lse, workspace=ws, stream=stream,
                        row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT, **kw)
    return out, lse


def _slot_case(B, P, H, N, K, dtype, e4m3, seed, holes=0.0, std=1.0):
    g = _gen(seed)
    q = _randn(g, B, P, H, 576, dtype=dtype, std=std)
    rows = _randn(g, B, N, 576, dtype=dtype)
    slots = torch.rand((B, P, N), generator=g, device="cuda").topk(K, -1).indices.int() if K else \
        torch.zeros((B, P, 0), dtype=torch.int32, device="cuda")
    if holes:
        slots = slots.masked_fill(torch.rand(slots.shape, generator=g, device="cuda") < holes, -1)
    # rows that no list names may hold anything
    if N > K:
        listed = torch.zeros((B, N), dtype=torch.bool, device="cuda")
        b = torch.arange(B, device="cuda")[:, None].expand(B, P * K)
        flat = slots.reshape(B, -1).long()
        listed[b[flat >= 0], flat[flat >= 0]] = True
        rows[~listed] = NAN
    if e4m3:
        rows = _pack8(rows)
    return q, rows, slots


def _picked(slots, N):
    return [[s[(s >= 0) & (s < N)].long() for s in req] for req in slots]


SIZES = [  # batch, positions, heads, rows, entries
    (1, 1, 1, 1, 1), (1, 1, 16, 512, 256), (2, 1, 128, 300, 64), (3, 2, 20, 130, 63), (1, 3, 7, 200, 65),
    (2, 1, 64, 129, 129), (5, 1, 100, 700, 513), (1, 1, 129, 150, 127), (2, 1, 200, 400, 333),
    (1, 1, 128, 4096, 2048), (40, 1, 16, 1100, 1000), (1, 1, 16, 9000, 8191), (160, 1, 8, 40, 31),
    (300, 1, 2, 20, 3), (2, 2, 256, 300, 128)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("size", SIZES)
def test_attend_slots(hs, size, dtype, e4m3):
    B, P, H, N, K = size
    q, rows, slots = _slot_case(B, P, H, N, K, dtype, e4m3, seed=sum(size))
    out, lse = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, N), e4m3, SCALE), dtype)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("case", ["holes", "far", "empty", "repeat", "none", "first", "last"])
def test_attend_masks(hs, case, e4m3):
    B, P, H, N, K = 3, 2, 24, 500, 200
    q, rows, slots = _slot_case(B, P, H, N, K, BF, e4m3, seed=7)
    slots = slots.clone()
    if case == "holes":
        slots[torch.rand(slots.shape, generator=_gen(1), device="cuda") < 0.6] = -1
    elif case == "far":  # out of range either way: absent, not read
        slots[:, :, ::3] = N
        slots[:, :, 1::3] = torch.tensor(2 ** 31 - 1, dtype=torch.int32)
        slots[0, 0, 2] = -2 ** 31
    elif case == "empty":
        slots[1, 0] = -1
        slots[2] = N + 5
    elif case == "repeat":
        slots[:] = slots[:, :, :1].clone()
    elif case == "none":
        slots = slots[:, :, :0]
    elif case == "first":
        slots[:, :, 1:] = -1
    else:
        slots[:, :, :-1] = -1
    out, lse = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, N), e4m3, SCALE), BF)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("P,H,lengths", [
    (1, 16, [1, 0, 5]), (1, 128, [700]), (4, 16, [3, 4, 130, 0, 1]), (2, 64, [64, 65, 127, 128, 129]),
    (1, 5, [5000, 1, 333]), (3, 128, [2050]), (130, 3, [200, 131])])
def test_attend_lengths(hs, P, H, lengths, dtype, e4m3):
    g = _gen(P + H)
    B, N = len(lengths), max(lengths) + 3
    q = _randn(g, B, P, H, 576, dtype=dtype)
    rows = _randn(g, B, N, 576, dtype=dtype)
    for b, n in enumerate(lengths):
        rows[b, n:] = NAN
    rows = _pack8(rows) if e4m3 else rows
    out, lse = _attend(hs, q, rows, e4m3=e4m3,
                       lengths=torch.tensor(lengths, dtype=torch.int32, device="cuda"))
    picked = [[torch.arange(max(0, n - P + 1 + p), device="cuda") for p in range(P)] for n in lengths]
    _check_attend(out, lse, _attend_ref(q, rows, picked, e4m3, SCALE), dtype)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,P,H,K", [
    (40, 1, 128, 2048), (17, 1, 129, 3000), (33, 1, 33, 2000), (5, 2, 100, 2000), (3, 1, 64, 2500), (90, 1, 40, 1999),
    (13, 1, 16, 3000), (7, 3, 20, 1501)])
def test_attend_slots_pieces(hs, B, P, H, K, e4m3):
    """Units cut in pieces and joined, many units and few; requests whose list is empty at its start, its end
    or throughout (pieces without a row); a second run gives the same bits."""
    q, rows, slots = _slot_case(B, P, H, K + 100, K, BF, e4m3, seed=B + H)
    slots[0, :, :K - 70] = -1
    slots[1, :, 70:] = -1
    slots[2] = -1
    out, lse = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, K + 100), e4m3, SCALE), BF)
    again, lse_again = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("P,H,lengths", [
    (1, 128, [9000, 1, 0, 63, 64, 65, 4000]), (1, 64, [6000, 1, 5001, 77]), (2, 130, [5000] * 3 + [1]),
    (1, 16, [12000, 3, 0, 700, 2500]), (1, 128, [1] * 40 + [5000]), (1, 40, [5000] + [1] * 40),
    (3, 24, [3000, 2, 1, 0] * 6), (1, 100, [0, 0, 0]), (1, 128, [4096] * 20)])
def test_attend_lengths_pieces(hs, P, H, lengths, e4m3):
    """Contexts of very unequal lengths, which the pieces' cut weighs with each unit's own time."""
    g = _gen(H + len(lengths))
    B, N = len(lengths), max(lengths + [4000])
    q = _randn(g, B, P, H, 576, dtype=BF)
    rows = _randn(g, B, N, 576, dtype=BF)
    for b, n in enumerate(lengths):
        rows[b, n:] = NAN
    rows = _pack8(rows) if e4m3 else rows
    device = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    out, lse = _attend(hs, q, rows, e4m3=e4m3, lengths=device)
    picked = [[torch.arange(max(0, n - P + 1 + p), device="cuda") for p in range(P)] for n in lengths]
    _check_attend(out, lse, _attend_ref(q, rows, picked, e4m3, SCALE), BF)
    again, lse_again = _attend(hs, q, rows, e4m3=e4m3, lengths=device)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


def test_attend_lengths_clamped(hs):
    g = _gen(3)
    q, rows = _randn(g, 3, 1, 8, 576), _randn(g, 3, 100, 576)
    out, lse = _attend(hs, q, rows, lengths=torch.tensor([1000, -5, 2 ** 31 - 1], dtype=torch.int32, device="cuda"))
    every = torch.arange(100, device="cuda")
    _check_attend(out, lse, _attend_ref(q, rows, [[every], [every[:0]], [every]], False, SCALE), BF)


@pytest.mark.parametrize("e4m3", [False, True])
def test_attend_strides(hs, e4m3):
    """q and out inside larger arrays in another axis order, padded rows, lists with strides."""
    B, P, H, N, K = 3, 2, 12, 90, 70
    q, rows, slots = _slot_case(B, P, H, N, K, BF, e4m3, seed=11)
    wide = torch.zeros((H, P, B, 600), dtype=BF, device="cuda")
    wide[..., 8:584] = q.permute(2, 1, 0, 3)
    qs = wide[..., 8:584].permute(2, 1, 0, 3)
    raw = rows.view(torch.uint8) if not e4m3 else rows
    padded = torch.full((B, N + 5, raw.shape[-1] + 48), 255, dtype=torch.uint8, device="cuda")
    padded[:, 2:N + 2, 16:16 + raw.shape[-1]] = raw
    rs = padded[:, 2:N + 2, 16:16 + raw.shape[-1]]
    ss = torch.zeros((P, B, K + 3), dtype=torch.int32, device="cuda")
    ss[:, :, 3:] = slots.transpose(0, 1)
    ss = ss[:, :, 3:].transpose(0, 1)
    hold = torch.full((P, B, H, 520), 3.0, dtype=BF, device="cuda")
    out = hold[..., :512].transpose(0, 1)
    ws = torch.empty(hs.hs_latent_attend_workspace(B, P, H, K), dtype=torch.uint8, device="cuda")
    hs.hs_latent_attend(qs, rs, out, SCALE, slots=ss, workspace=ws,
                        row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    want, _ = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    assert torch.equal(out, want) and (hold[..., 512:] == 3.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("std", [0.0, 30.0])
def test_attend_flat_and_peaked(hs, std, e4m3):
    """All scores equal, and scores of hundreds (one row takes nearly all the weight)."""
    q, rows, slots = _slot_case(2, 1, 16, 800, 700, BF, e4m3, seed=5, std=std)
    out, lse = _attend(hs, q, rows, e4m3=e4m3, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, 800), e4m3, SCALE), BF)


@pytest.mark.parametrize("scale", [-0.05, 0.0])
def test_attend_scale(hs, scale):
    q, rows, slots = _slot_case(2, 1, 16, 300, 200, BF, False, seed=6)
    out, lse = _attend(hs, q, rows, scale=scale, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, 300), False, scale), BF)


@pytest.mark.parametrize("dtype", [BF, HALF])
def test_attend_row_scales_of_many_sizes(hs, dtype):
    """8-bit rows whose scales span 2^-20 .. 2^6, some of them all zeros."""
    g = _gen(21)
    rows = torch.randn((2, 600, 576), generator=g, device="cuda")
    rows *= torch.exp2(torch.randint(-20, 7, (2, 600, 1), generator=g, device="cuda").float())
    rows[:, ::50] = 0
    rows = _pack8(rows)
    q = _randn(g, 2, 1, 16, 576, dtype=dtype, std=0.05)
    slots = torch.arange(600, dtype=torch.int32, device="cuda").expand(2, 1, 600)
    out, lse = _attend(hs, q, rows, e4m3=True, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, 600), True, SCALE), dtype)


@pytest.mark.parametrize("H", [16, 32])
@pytest.mark.parametrize("B,P,K", [(300, 3, 64), (1200, 1, 5), (400, 2, 100)])
def test_attend_short_units_of_unlike_queries(hs, B, P, K, H):
    """Many units of one tile (and of two) a worker, whose bf16 queries have unlike magnitudes: each is
    held in fp16 by a power of two of its own, which the next units' must not replace early."""
    q, rows, slots = _slot_case(B, P, H, K + 10, K, BF, True, seed=B + K + H)
    power = torch.randint(0, 6, (B, P, 1, 1), generator=_gen(B), device="cuda") * -4
    q = q * torch.exp2(power.float()).to(BF)
    out, lse = _attend(hs, q, rows, e4m3=True, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, K + 10), True, SCALE), BF)


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("H", [16, 64])
@pytest.mark.parametrize("beta", [1.0, 2.5, 6.0])
@pytest.mark.parametrize("least", [0.0, 2.0 ** -125])
@pytest.mark.parametrize("N,small", [(40, [3]), (40, [39]), (300, [0, 1]), (300, [299]), (300, [100, 130]),
                                     (6000, [5]), (6000, [3000]), (6000, [5999]), (64, list(range(64)))])
def test_attend_rows_of_no_scale_beside_low_scores(hs, N, small, least, beta, H, dtype):
    """8-bit rows of scale 0 (what the norm writes for zeros) or nearly 0 score 0.  The other rows score about
    -60 beta, in powers of two, so those take all the weight, in whichever tile or piece they come."""
    g = _gen(N + H)
    u = torch.randn((2, 1, 1, 576), generator=g, device="cuda")
    q = (u * (1 + 0.01 * torch.randn((2, 1, H, 1), generator=g, device="cuda"))).to(dtype)
    rows = _pack8(-beta * u[:, 0] + 0.1 * torch.randn((2, N, 576), generator=g, device="cuda"))
    rows[:, small, 576:580] = torch.full((1,), least, device="cuda").view(torch.uint8)
    if least == 0:
        rows[:, small, :576] = 0
    out, lse = _attend(hs, q, rows, e4m3=True, lengths=torch.tensor([N, N], dtype=torch.int32, device="cuda"))
    every = [torch.arange(N, device="cuda")]
    o, want_lse, mean_abs, reach = _attend_ref(q, rows, [every, every], True, SCALE)
    # as in _check_attend, and half of the least step that the type has
    half, step = torch.finfo(dtype).eps / 2, torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps
    score = 576 * 2.0 ** -23 * reach + 2.0 ** -18
    tol = half * o.abs() + (half + 2 * score) * mean_abs + step / 2 + 1e-30
    assert torch.isfinite(out).all() and ((out.double() - o).abs() <= tol).all()
    # a reference of 128 and more has steps of 2^-17, in the exponent and in the logarithm
    assert ((lse.double() - want_lse).abs() <= score.squeeze(-1) + 2.0 ** -16 + 2.0 ** -21 * want_lse.abs()).all()


@pytest.mark.parametrize("power", [-130, -124, -110, -88, -60, 60, 100, 115, 118])
@pytest.mark.parametrize("H", [16, 64])
def test_attend_bf16_queries_of_any_magnitude(hs, H, power):
    """8-bit rows with bf16 queries from the type's smallest values to its largest, under a scale that makes
    the scores ordinary ones."""
    q, rows, slots = _slot_case(2, 1, H, 300, 200, BF, True, seed=13)
    q = (q.double() * 2.0 ** power).to(BF)
    scale = SCALE * 2.0 ** min(-power, 126)
    out, lse = _attend(hs, q, rows, e4m3=True, slots=slots, scale=scale)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, 300), True, scale), BF)


def test_attend_nan_and_inf_propagate(hs):
    q, rows, slots = _slot_case(3, 1, 16, 300, 200, BF, False, seed=8)
    q[0, 0, 3] = NAN
    rows[1, slots[1, 0, 100].long(), 5] = NAN
    out, _ = _attend(hs, q, rows, slots=slots)
    assert out[0, 0, 3].isnan().all() and not out[0, 0, 2].isnan().any() and not out[0, 0, 4].isnan().any()
    assert out[1].isnan().all() and not out[2].isnan().any()


def test_attend_rows_past_4_gib(hs):
    """Row offsets beyond 32 bits, by slots and by the requests' stride."""
    N = 4_000_000  # 4.6 GB a request
    rows = torch.empty((2, N, 576), dtype=BF, device="cuda")
    g = _gen(9)
    slots = (N - 1 - torch.randperm(2000, generator=g, device="cuda")[:150]).int().expand(2, 1, 150).contiguous()
    rows[:, N - 2000:] = _randn(g, 2, 2000, 576)
    q = _randn(g, 2, 1, 16, 576)
    out, lse = _attend(hs, q, rows, slots=slots)
    _check_attend(out, lse, _attend_ref(q, rows, _picked(slots, N), False, SCALE), BF)


def test_attend_repeats_and_replays(hs):
    """The same bits again, on another stream, and from a CUDA graph with new inputs in place."""
    q, rows, slots = _slot_case(4, 1, 128, 900, 800, BF, True, seed=10)
    out, lse = _attend(hs, q, rows, e4m3=True, slots=slots)
    again, _ = _attend(hs, q, rows, e4m3=True, slots=slots)
    assert torch.equal(out, again)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(hs.hs_latent_attend_workspace(4, 1, 128, 800), dtype=torch.uint8, device="cuda")
    o2 = torch.empty_like(out)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        hs.hs_latent_attend(q, rows, o2, SCALE, slots=slots, row_format=hs.HS_ROWS_E4M3, workspace=ws,
                            stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(o2, out)
    q.copy_(_randn(_gen(12), 4, 1, 128, 576))
    graph.replay()
    torch.cuda.synchronize()
    want, _ = _attend(hs, q, rows, e4m3=True, slots=slots)
    assert torch.equal(o2, want) and not torch.equal(o2, out)


# ---- expanded form ---------------------------------------------------------------------

def _prefill(hs, q, rows, w_uk, w_uv, nq, nk, e4m3=False, **kw):
    start = [torch.tensor([0] + n, device="cuda").cumsum(0).int() for n in (nq, nk)]
    out = torch.full((q.shape[0], q.shape[1], 128), NAN, dtype=q.dtype, device="cuda")
    lse = torch.full(q.shape[:2], NAN, device="cuda")
    ws = torch.full((hs.hs_latent_prefill_workspace(rows.shape[0], q.shape[1]),), 255, dtype=torch.uint8,
                    device="cuda")
    hs.hs_latent_prefill(q, rows, w_uk, w_uv, start[0], start[1], out, SCALE, lse=lse, workspace=ws,
                         row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT, **kw)
    return out, lse


def _check_prefill(out, lse, q, rows, w_uk, w_uv, nq, nk, e4m3):
    dtype = q.dtype
    half = torch.finfo(dtype).eps / 2
    wide = _wide(rows, e4m3)
    off = total = 0.0
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        kv = wide[k0:k0 + m]
        allowed = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        some = allowed.any(1)
        for h in range(q.shape[1]):
            k = torch.cat([kv[:, :512] @ w_uk[h].double().t(), kv[:, 512:]], 1)
            v = kv[:, :512] @ w_uv[h].double().t()
            qh = q[q0:q0 + n, h].double()
            s = torch.where(allowed, SCALE * (qh @ k.t()), -math.inf)
            got, got_lse = out[q0:q0 + n, h], lse[q0:q0 + n, h]
            assert (got[~some] == 0).all() and (got_lse[~some] == -math.inf).all()
            if not some.any():
                continue
            p = torch.softmax(s[some], -1)
            o, mean_abs = p @ v, p @ v.abs()
            # a key's expanded channels are rounded once: a score moves by half a step of the sum of
            # magnitudes; the sums over 512 and 192 channels are fp32
            reach = SCALE * torch.where(allowed, qh.abs() @ k.abs().t(), 0.0).amax(-1, keepdim=True)[some]
            score = (half + 2.0 ** -12) * reach + 2.0 ** -18
            tol = half * o.abs() + (2 * half + 2.0 ** -12 + 2 * score) * mean_abs + 1e-30
            err = (got[some].double() - o).abs()
            assert torch.isfinite(got).all()
            assert bool((err <= tol).all()), (err / tol).max().item()
            lse_err = (got_lse[some].double() - torch.logsumexp(s[some], -1)).abs()
            assert (lse_err <= score.squeeze(-1) + 2.0 ** -20 * 20).all()
            off += err.square().sum().item()
            total += o.square().sum().item()
        q0, k0 = q0 + n, k0 + m
    # out, weight, value, and keys (0.8 of a step in the scores): independent, in the 2-norm
    assert off <= (2.5 * half + 1e-4) ** 2 * total


def _prompt_case(nq, nk, H, dtype, e4m3, seed):
    g = _gen(seed)
    q = _randn(g, sum(nq), H, 192, dtype=dtype)
    rows = _randn(g, sum(nk), 576, dtype=dtype)
    rows = _pack8(rows) if e4m3 else rows
    w_uk, w_uv = (_randn(g, H, 128, 512, dtype=dtype, std=512 ** -0.5) for _ in range(2))
    return q, rows, w_uk, w_uv


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("H,nq,nk", [
    (1, [1], [1]), (2, [128], [128]), (3, [129, 1, 0, 63], [129, 40, 0, 63]), (2, [257], [700]),
    (1, [5, 300], [2, 300]), (4, [64, 65, 127], [64, 65, 500]), (1, [1, 1, 1], [1, 513, 1000]),
    (2, [10, 0, 7], [0, 9, 7]), (1, [1300], [1300])])
def test_prefill(hs, H, nq, nk, dtype, e4m3):
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, H, dtype, e4m3, seed=H + sum(nk))
    out, lse = _prefill(hs, q, rows, w_uk, w_uv, nq, nk, e4m3)
    _check_prefill(out, lse, q, rows, w_uk, w_uv, nq, nk, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
def test_prefill_strides(hs, e4m3):
    nq, nk, H = [70, 33], [90, 33], 3
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, H, BF, e4m3, seed=2)
    wide = torch.zeros((H, 103, 208), dtype=BF, device="cuda")
    wide[..., 8:200] = q.transpose(0, 1)
    raw = rows if e4m3 else rows.view(torch.uint8)
    padded = torch.full((123, raw.shape[-1] + 32), 255, dtype=torch.uint8, device="cuda")
    padded[:, 16:16 + raw.shape[-1]] = raw
    got, lse = _prefill(hs, wide[..., 8:200].transpose(0, 1), padded[:, 16:16 + raw.shape[-1]], w_uk, w_uv,
                        nq, nk, e4m3)
    want, want_lse = _prefill(hs, q, rows, w_uk, w_uv, nq, nk, e4m3)
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


def test_prefill_leaves_other_tokens_and_ignores_unseen_rows(hs):
    """Tokens outside the requests stay; NaN in a row reaches only the queries that see it."""
    q, rows, w_uk, w_uv = _prompt_case([200], [200], 2, BF, False, seed=4)
    want, _ = _prefill(hs, q, rows, w_uk, w_uv, [150], [150])
    assert want[150:].isnan().all() and not want[:150].isnan().any()
    rows[100:] = NAN
    got, _ = _prefill(hs, q, rows, w_uk, w_uv, [150], [150])
    assert torch.equal(got[:100], want[:100]) and got[100:150].isnan().all()


def test_prefill_bad_starts_are_clamped(hs):
    q, rows, w_uk, w_uv = _prompt_case([60], [60], 2, BF, False, seed=5)
    want, _ = _prefill(hs, q, rows, w_uk, w_uv, [60], [60])
    got, _ = _prefill(hs, q, rows, w_uk, w_uv, [100], [100])
    assert torch.equal(got, want)


def test_prefill_replays(hs):
    nq, nk = [130, 7], [300, 7]
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, 4, BF, True, seed=6)
    want, _ = _prefill(hs, q, rows, w_uk, w_uv, nq, nk, True)
    start = [torch.tensor([0] + n, device="cuda").cumsum(0).int() for n in (nq, nk)]
    out = torch.empty_like(want)
    ws = torch.empty(hs.hs_latent_prefill_workspace(307, 4), dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_latent_prefill(q, rows, w_uk, w_uv, *start, out, SCALE, row_format=hs.HS_ROWS_E4M3,
                             workspace=ws, stream=torch.cuda.current_stream())
    for _ in range(2):
        graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("H,nq,nk", [
    (16, [520, 3], [2500, 700]), (20, [700], [5000]), (8, [512], [4000]), (3, [600], [2100]), (1, [515, 513, 1], [4000, 513, 900]),
    (16, [1100], [1100]), (24, [300, 0, 40, 513], [600, 5, 10, 2000])])
def test_prefill_pieces(hs, H, nq, nk, e4m3):
    """Sizes whose units are cut and joined, many units and few; a second run gives the same bits."""
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, H, BF, e4m3, seed=H + sum(nk))
    out, lse = _prefill(hs, q, rows, w_uk, w_uv, nq, nk, e4m3)
    _check_prefill(out, lse, q, rows, w_uk, w_uv, nq, nk, e4m3)
    again, lse_again = _prefill(hs, q, rows, w_uk, w_uv, nq, nk, e4m3)
    assert torch.equal(out, again) and torch.equal(lse, lse_again)


@pytest.mark.parametrize("scale", [-SCALE, 0.0, 1e-30])
@pytest.mark.parametrize("H,nq,nk", [(2, [257, 40], [257, 300]), (3, [600], [2100])])
def test_prefill_scale(hs, H, nq, nk, scale):
    """Negative scales and 0 (every seen row weighs the same)."""
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, H, BF, False, seed=17)
    start = [torch.tensor([0] + n, device="cuda").cumsum(0).int() for n in (nq, nk)]
    out = torch.full((sum(nq), H, 128), NAN, dtype=BF, device="cuda")
    lse = torch.full((sum(nq), H), NAN, device="cuda")
    ws = torch.empty(hs.hs_latent_prefill_workspace(sum(nk), H), dtype=torch.uint8, device="cuda")
    hs.hs_latent_prefill(q, rows, w_uk, w_uv, *start, out, scale, lse=lse, workspace=ws)
    half = 2.0 ** -8
    q0 = k0 = 0
    for n, m in zip(nq, nk):
        kv = rows[k0:k0 + m].double()
        allowed = torch.ones((n, m), dtype=torch.bool, device="cuda").tril(m - n)
        for h in range(H):
            k = torch.cat([kv[:, :512] @ w_uk[h].double().t(), kv[:, 512:]], 1)
            v = kv[:, :512] @ w_uv[h].double().t()
            qh = q[q0:q0 + n, h].double()
            s = torch.where(allowed, scale * (qh @ k.t()), -math.inf)
            o, want_lse, mean_abs = _softmax_ref(s, v)
            reach = abs(scale) * torch.where(allowed, qh.abs() @ k.abs().t(), 0.0).amax(-1, keepdim=True)
            score = (half + 2.0 ** -12) * reach + 2.0 ** -18
            tol = half * o.abs() + (2 * half + 2.0 ** -12 + 2 * score) * mean_abs + 1e-30
            err = (out[q0:q0 + n, h].double() - o).abs()
            assert bool((err <= tol).all()), (err / tol).max().item()
            assert ((lse[q0:q0 + n, h].double() - want_lse).abs() <= score.squeeze(-1) + 2.0 ** -20 * 20).all()
        q0, k0 = q0 + n, k0 + m


# ---- norm ------------------------------------------------------------------------------

def _norm_ref(x, w, eps, residual, carry):
    d = x.shape[1] - carry
    h = x[:, :d].double()
    if residual is not None:
        h = h + residual.double()
    y = h / torch.sqrt(h.square().mean(1, keepdim=True) + eps) * w.double()
    return torch.cat([y, x[:, d:].double()], 1)


NORM_SIZES = [(1, 1, 0), (1, 4096, 0), (3, 7, 0), (5, 64, 64), (2, 1000, 24), (4, 512, 64), (2, 333, 1),
              (300, 512, 64), (2, 16384, 0), (3, 5000, 3), (2, 8192, 8), (1000, 128, 0), (7, 2047, 0)]


@pytest.mark.parametrize("with_residual", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF, torch.float32])
@pytest.mark.parametrize("n,d,carry", NORM_SIZES)
def test_norm(hs, n, d, carry, dtype, with_residual):
    g = _gen(n + d)
    x, w = _randn(g, n, d + carry, dtype=dtype), _randn(g, d, dtype=dtype)
    residual = _randn(g, n, d, dtype=dtype, std=2.0) if with_residual else None
    ro = torch.full_like(residual, NAN) if with_residual else None
    out = torch.full_like(x, NAN)
    hs.hs_rms_norm(x, w, out, 1e-6, residual=residual, residual_out=ro, carry=carry)
    want = _norm_ref(x, w, 1e-6, residual, carry)
    half = torch.finfo(dtype).eps / 2
    # the sum over d, the root and two products in fp32: a few steps, the sum's about sqrt(d)
    wide = want[:, :d].abs()
    tol = (half * 1.01 + 2.0 ** -24 * (8 + math.sqrt(d))) * wide
    if with_residual:  # h may cancel: its rounding is relative to the terms, in h itself and in the root
        terms = x[:, :d].double().abs() + residual.double().abs()
        h = x[:, :d].double() + residual.double()
        root = 1 / torch.sqrt(h.square().mean(1, keepdim=True) + 1e-6)
        tol = tol + 2.0 ** -23 * (terms * root * w.double().abs() +
                                  wide * terms.norm(dim=1, keepdim=True) * root / math.sqrt(d))
    err = (out.double() - want).abs()
    assert torch.equal(out[:, d:], x[:, d:])
    assert (err[:, :d] <= tol + (2.0 ** -25 if dtype == HALF else 1e-37)).all()
    if with_residual:
        assert torch.equal(ro, (x[:, :d].float() + residual.float()).to(dtype))


@pytest.mark.parametrize("group", [0, 1, 16, 100, 128])
@pytest.mark.parametrize("dtype", [BF, HALF, torch.float32])
@pytest.mark.parametrize("n,d,carry", NORM_SIZES)
def test_norm_e4m3(hs, n, d, carry, dtype, group):
    g = _gen(n * d)
    x, w = _randn(g, n, d + carry, dtype=dtype), _randn(g, d, dtype=dtype)
    width = d + carry
    groups = -(-width // group) if group else 1
    out = torch.full((n, width), 255, dtype=torch.uint8, device="cuda")
    scales = torch.full((n, groups), NAN, device="cuda")
    hs.hs_rms_norm(x, w, out, 1e-6, carry=carry, scales=scales, group=group)
    want = _norm_ref(x, w, 1e-6, None, carry)
    pad = torch.nn.functional.pad(want, (0, groups * (group or width) - width)).view(n, groups, -1)
    s = pad.abs().amax(-1) / 448
    assert ((scales.double() - s).abs() <= 2.0 ** -22 * (8 + math.sqrt(d)) * s).all()
    each = scales.double().repeat_interleave(group or width, 1)[:, :width]
    got = out.view(torch.float8_e4m3fn).double() * each
    # half a step of e4m3 (2^-4 of the value; 2^-10 scales below its normal range), and fp32's
    assert ((got - want).abs() <= 2.0 ** -4 * 1.001 * want.abs() + 2.0 ** -10 * 1.001 * each).all()
    assert (got.abs().view(n, width) <= each * 448).all()


@pytest.mark.parametrize("more", [0, 1, 2 ** 31])
@pytest.mark.parametrize("width,carry", [(64, 0), (577, 65), (1000, 24), (1024, 0), (7000, 3), (8192, 64), (12739, 0)])
def test_norm_e4m3_group_of_the_whole_row(hs, width, carry, more):
    """A group as wide as the row, or wider by any amount, is one scale a row."""
    g = _gen(width)
    x, w = _randn(g, 40, width), _randn(g, width - carry)
    got = []
    for group in (0, min(width + more, 2 ** 31 - 1)):
        out = torch.full((40, width), 255, dtype=torch.uint8, device="cuda")
        scales = torch.full((40, 2), NAN, device="cuda")
        hs.hs_rms_norm(x, w, out, 1e-6, carry=carry, scales=scales[:, :1], group=group)
        assert scales[:, 1].isnan().all()
        got.append((out, scales[:, 0]))
    assert torch.equal(got[0][0], got[1][0]) and torch.equal(got[0][1], got[1][1])


@pytest.mark.parametrize("group", [0, 16, 100])
@pytest.mark.parametrize("dtype", [BF, HALF, torch.float32])
@pytest.mark.parametrize("n,d,carry", [(2000, 512, 512), (2000, 512, 511), (500, 1024, 1024), (300, 1000, 1001),
                                       (100, 4096, 4001), (50, 5000, 7001)])
def test_norm_e4m3_divides_by_the_scale(hs, n, d, carry, dtype, group):
    """Carried channels, whose values are exact: e4m3 of the fp32 quotient by the scale that is written, bit for bit."""
    g = _gen(n + d + carry)
    x, w = _randn(g, n, d + carry, dtype=dtype), _randn(g, d, dtype=dtype)
    width = d + carry
    out = torch.empty((n, width), dtype=torch.uint8, device="cuda")
    scales = torch.empty((n, -(-width // group) if group else 1), device="cuda")
    hs.hs_rms_norm(x, w, out, 1e-6, carry=carry, scales=scales, group=group)
    each = scales.repeat_interleave(group or width, 1)[:, :width]
    want = (x.float() / each).to(torch.float8_e4m3fn).view(torch.uint8)
    assert torch.equal(out[:, d:], want[:, d:])


@pytest.mark.parametrize("dtype", [BF, HALF, torch.float32])
@pytest.mark.parametrize("d,carry", [(6145, 0), (7001, 3), (12739, 64), (16384, 0)])
def test_norm_wide_rows_of_odd_alignment(hs, d, carry, dtype):
    """The widest rows, element by element: as the type, and as e4m3 with one scale."""
    g = _gen(d)
    x, w = _randn(g, 3, d + carry + 1, dtype=dtype)[:, 1:], _randn(g, d, dtype=dtype)
    out = torch.full((3, d + carry), NAN, dtype=dtype, device="cuda")
    hs.hs_rms_norm(x, w, out, 1e-6, carry=carry)
    want = _norm_ref(x, w, 1e-6, None, carry)
    half = torch.finfo(dtype).eps / 2
    tol = (half * 1.01 + 2.0 ** -24 * (8 + math.sqrt(d))) * want.abs()
    assert ((out.double() - want).abs() <= tol + (2.0 ** -25 if dtype == HALF else 1e-37)).all()
    q, s = torch.full((3, d + carry), 255, dtype=torch.uint8, device="cuda"), torch.full((3, 1), NAN, device="cuda")
    hs.hs_rms_norm(x, w, q, 1e-6, carry=carry, scales=s)
    top = want.abs().amax(1, keepdim=True) / 448
    assert ((s.double() - top).abs() <= 2.0 ** -22 * (8 + math.sqrt(d)) * top).all()
    got = q.view(torch.float8_e4m3fn).double() * s.double()
    assert ((got - want).abs() <= 2.0 ** -4 * 1.001 * want.abs() + 2.0 ** -10 * 1.001 * s.double()).all()


def test_norm_writes_cache_rows(hs):
    """The 8-bit row form, read back by the attention."""
    g = _gen(1)
    n = 257
    x, w = _randn(g, n, 576), _randn(g, 512)
    cache = torch.full((n, 592), 255, dtype=torch.uint8, device="cuda")
    hs.hs_rms_norm(x, w, cache[:, :576], 1e-6, carry=64, scales=cache[:, 576:580].view(torch.float32))
    assert (cache[:, 580:] == 255).all()
    want = _norm_ref(x, w, 1e-6, None, 64)
    got = _wide(cache, True)
    scale = cache[:, 576:580].view(torch.float32).double()
    assert ((got - want).abs() <= 2.0 ** -4 * 1.001 * want.abs() + 2.0 ** -10 * 1.001 * scale).all()
    q = _randn(g, 1, 1, 16, 576)
    out, lse = _attend(hs, q, cache[None], e4m3=True, lengths=torch.tensor([n], dtype=torch.int32, device="cuda"))
    _check_attend(out, lse, _attend_ref(q, cache[None], [[torch.arange(n, device="cuda")]], True, SCALE), BF)


def test_norm_in_place_strides_and_odd_alignment(hs):
    g = _gen(2)
    for d, off in ((768, 0), (768, 1), (333, 3), (1024, 4)):
        hold = _randn(g, 9, d + 40)
        x, w = hold[:, off:off + d], _randn(g, d + 8)[off:off + d] if off < 8 else _randn(g, d)
        rhold = _randn(g, 9, d + 24)
        residual = rhold[:, 5:5 + d]
        want = torch.empty((9, d), dtype=BF, device="cuda")
        want_r = torch.empty((9, d), dtype=BF, device="cuda")
        hs.hs_rms_norm(x.contiguous(), w.clone(), want, 1e-5, residual=residual.contiguous(), residual_out=want_r)
        keep, rkeep = hold.clone(), rhold.clone()
        hs.hs_rms_norm(x, w, x, 1e-5, residual=residual, residual_out=residual)
        assert torch.equal(x, want) and torch.equal(residual, want_r)
        keep[:, off:off + d], rkeep[:, 5:5 + d] = want, want_r
        assert torch.equal(hold, keep) and torch.equal(rhold, rkeep)


@pytest.mark.parametrize("d", [64, 333, 4096])
def test_norm_zeros_nan_inf_and_tiny(hs, d):
    x = torch.ones((5, d), device="cuda")
    x[0] = 0
    x[1, d // 2] = NAN
    x[2, 1] = math.inf
    x[3] = 1e-30
    x[4, 0] = -1e30  # its square overflows: the root is infinite and every value 0
    w = torch.ones(d, device="cuda")
    out = torch.empty_like(x)
    hs.hs_rms_norm(x, w, out, 1e-6)
    assert (out[0] == 0).all() and out[1].isnan().all() and out[2, 1].isnan() and (out[2, 2:] == 0).all()
    assert torch.allclose(out[3], torch.full_like(out[3], 1e-27), rtol=1e-5, atol=0)
    assert (out[4] == 0).all()
    q, s = torch.empty((5, d), dtype=torch.uint8, device="cuda"), torch.empty((5, 1), device="cuda")
    hs.hs_rms_norm(x, w, q, 1e-6, scales=s)
    v = q.view(torch.float8_e4m3fn).float()
    assert (v[0] == 0).all() and s[0] == 0 and s[1].isnan() and v[1].isnan().all() and s[2].isnan()
    assert torch.allclose((v * s)[3], torch.full((d,), 1e-27, device="cuda"), rtol=2 ** -4, atol=0)
    assert (v[4] == 0).all()


def test_norm_replays(hs):
    g = _gen(3)
    x, w, r = _randn(g, 64, 4096), _randn(g, 4096), _randn(g, 64, 4096)
    out, ro = torch.empty_like(x), torch.empty_like(r)
    hs.hs_rms_norm(x, w, out, 1e-6, residual=r, residual_out=ro)
    want, want_r = out.clone(), ro.clone()
    out.zero_(), ro.zero_()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_rms_norm(x, w, out, 1e-6, residual=r, residual_out=ro, stream=torch.cuda.current_stream())
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(ro, want_r)
