"""Rows written and read back, heads' norm and rotation, and attention over a shared
prefix, against plain 64-bit forms.

Tolerances count roundings to the output's type (each at most half a step, eps / 2 of
the value) and the fp32 steps before; the derivation stands at each check.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from test_gpu_ops import (BF, HALF, NAN, SCALE, _check_prefill, _gen, _pack8, _prefill, _prompt_case, _randn,  # noqa: E402
                          _softmax_ref, _wide)

F32 = torch.float32
EPS = 1e-6


@pytest.fixture(scope="module")
def hs():
    from hierarchical_kv_cache_hs_gb300 import hs as mod
    return mod


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _freq(rope):
    return (10000.0 ** (-torch.arange(rope // 2, dtype=torch.float64, device="cuda") * 2 / rope)).float()


def _half(dtype):
    return torch.finfo(dtype).eps / 2


def _least(dtype):
    """Half of the least step of a type."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def _turn64(x, positions, freq, pairs):
    """x [n, ..., rope] turned, and the sum of the magnitudes of each result's two terms."""
    angle = positions.double()[:, None] * freq.double()
    angle = angle.view((x.shape[0],) + (1,) * (x.dim() - 2) + (-1,))
    cos, sin = torch.cos(angle), torch.sin(angle)
    a, b = (x[..., 0::2], x[..., 1::2]) if pairs else x.chunk(2, -1)
    parts = [torch.stack([p, q], -1).flatten(-2) if pairs else torch.cat([p, q], -1) for p, q in (
        (a * cos - b * sin, a * sin + b * cos),
        ((a * cos).abs() + (b * sin).abs(), (a * sin).abs() + (b * cos).abs()))]
    # a position near 2^31 makes the reference's own angle off by 2^-22
    return parts[0], parts[1] + (a.abs() + b.abs()).repeat_interleave(2, -1) * 2.0 ** -2 if pairs else \
        parts[1] + (a.abs() + b.abs()).repeat((1,) * (a.dim() - 1) + (2,)) * 2.0 ** -2


def _norm64(x, weight):
    if weight is None:
        return x
    return weight.double() * x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS)


def _close(got, want, slack, dtype):
    """One rounding to the type, and fp32 steps: a mean of up to 1024 squares (its terms' sum off by at most
    their number of steps, halved by the root), the root's two steps, three products and, of a turn, a cosine
    and sine off by 2^-22 (two steps and the angle's own rounding, 2^-24 of up to pi) and its sum:
    2^-15 of a value with a norm's 1024 terms in any order, 2^-20 of a turn's terms."""
    tol = _half(dtype) * (1 + 2.0 ** -10) * want.abs() + slack + _least(dtype) + 1e-38
    err = (got.double() - want).abs()
    assert torch.isfinite(got).all() and bool((err <= tol).all()), (err / tol).max().item()


# ---- rotate ----------------------------------------------------------------------------

def _rotate_ref(x, weight, positions, freq, rope_at, pairs):
    y = _norm64(x.double(), weight)
    slack = 2.0 ** -15 * y.abs() if weight is not None else torch.zeros_like(y)
    if positions is not None:
        rope = 2 * freq.numel()
        part = slice(rope_at, rope_at + rope)
        turned, terms = _turn64(y[..., part].clone(), positions, freq, pairs)
        y[..., part] = turned
        slack[..., part] = (2.0 ** -20 + (2.0 ** -15 if weight is not None else 0)) * terms
    return y, slack


ROTATE = [  # tokens, heads, key heads, dim, rope, rope_at
    (1, 16, 0, 192, 64, 128), (64, 128, 0, 192, 64, 128), (3, 1, 0, 64, 64, 0), (5, 8, 2, 128, 128, 0),
    (7, 20, 1, 80, 80, 0), (2, 3, 3, 96, 32, 16), (33, 1, 1, 576, 64, 512), (300, 2, 0, 256, 128, 64),
    (1, 1, 0, 2, 2, 0), (4, 5, 2, 7, 4, 1), (9, 2, 1, 100, 50, 30), (3, 2, 0, 1024, 1024, 0), (2, 300, 5, 72, 24, 24),
    (1, 1, 1, 1000, 998, 1), (17, 64, 8, 128, 64, 64), (1025, 1, 0, 128, 64, 0), (70, 1, 1, 96, 64, 32),
    (33, 2, 1, 48, 16, 16), (50, 40, 4, 32, 32, 0), (5, 1, 0, 32, 16, 16), (130, 3, 0, 80, 80, 0), (300, 20, 0, 192, 64, 64)]


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("dtype", [BF, HALF, F32])
@pytest.mark.parametrize("size", ROTATE)
def test_rotate(hs, size, dtype, norm, pairs):
    n, heads, keys, dim, rope, at = size
    g = _gen(sum(size))
    q, k = _randn(g, n, heads, dim, dtype=dtype), _randn(g, n, keys, dim, dtype=dtype) if keys else None
    wq = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if norm else None
    wk = (1 + 0.1 * torch.randn(dim, generator=g, device="cuda")).to(dtype) if norm and keys else None
    positions = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq = _freq(rope)
    qo, ko = torch.full_like(q, NAN), torch.full_like(k, NAN) if keys else None
    hs.hs_norm_rotate(q, qo, k=k, k_out=ko, q_weight=wq, k_weight=wk, eps=EPS, positions=positions, inv_freq=freq,
                      rotation=hs.HS_ROTATE_PAIRS if pairs else hs.HS_ROTATE_HALVES, rope_at=at)
    for x, w, out in ((q, wq, qo), (k, wk, ko)):
        if x is not None:
            _close(out, *_rotate_ref(x, w, positions, freq, at, pairs), dtype)


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("dim", [128, 50])
def test_rotate_norm_only_and_neither(hs, dim, dtype):
    g = _gen(dim)
    q, k = _randn(g, 5, 3, dim, dtype=dtype), _randn(g, 5, 2, dim, dtype=dtype)
    w = _randn(g, dim, dtype=dtype)
    qo, ko = torch.empty_like(q), torch.empty_like(k)
    hs.hs_norm_rotate(q, qo, k=k, k_out=ko, q_weight=w, eps=EPS)
    y = _norm64(q.double(), w)
    _close(qo, y, 2.0 ** -15 * y.abs(), dtype)
    assert torch.equal(ko, k)


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("dim,rope,at", [(128, 128, 0), (192, 64, 128), (62, 30, 3)])
def test_rotate_strides_and_in_place(hs, dim, rope, at, pairs):
    """Queries inside wider arrays in another axis order; the output over the input; nothing beside is touched."""
    g = _gen(dim + rope)
    n, heads = 13, 6
    kind = hs.HS_ROTATE_PAIRS if pairs else hs.HS_ROTATE_HALVES
    positions = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq, w = _freq(rope), _randn(g, dim)
    hold = _randn(g, heads, n, dim + 16)
    before = hold.clone()
    x = hold[..., 8:8 + dim].transpose(0, 1)
    want = torch.empty((n, heads, dim), dtype=BF, device="cuda")
    hs.hs_norm_rotate(x.contiguous(), want, q_weight=w, eps=EPS, positions=positions, inv_freq=freq, rotation=kind, rope_at=at)
    out = torch.full((n, heads, dim + 3), 5.0, dtype=BF, device="cuda")  # rows of odd alignment
    hs.hs_norm_rotate(x, out[..., 1:1 + dim], q_weight=w, eps=EPS, positions=positions, inv_freq=freq, rotation=kind, rope_at=at)
    assert torch.equal(out[..., 1:1 + dim], want) or dim != 62 or torch.allclose(out[..., 1:1 + dim].float(), want.float())
    assert (out[..., 0] == 5).all() and (out[..., 1 + dim:] == 5).all()
    hs.hs_norm_rotate(x, x, q_weight=w, eps=EPS, positions=positions, inv_freq=freq, rotation=kind, rope_at=at)
    assert torch.equal(x, want)
    assert torch.equal(hold[..., :8], before[..., :8]) and torch.equal(hold[..., 8 + dim:], before[..., 8 + dim:])


@pytest.mark.parametrize("pairs", [True, False])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("where", ["x", "out", "both"])
@pytest.mark.parametrize("dtype", [BF, HALF, F32])
@pytest.mark.parametrize("dim,rope,at,heads", [(128, 128, 0, 6), (192, 64, 128, 6), (192, 64, 128, 1), (62, 30, 3, 6), (1024, 512, 256, 2)])
def test_rotate_odd_alignment(hs, dim, rope, at, heads, dtype, where, norm, pairs):
    """Inputs, outputs or both an element off every border: heads that would go in units go element by element."""
    g = _gen(dim + rope + heads)
    n = 13
    x = torch.full((n, heads, dim + 3), NAN, dtype=dtype, device="cuda")[..., 1:1 + dim] if where != "out" else \
        torch.empty((n, heads, dim), dtype=dtype, device="cuda")
    x.copy_(_randn(g, n, heads, dim, dtype=dtype))
    hold = torch.full((n, heads, dim + 3), 5.0, dtype=dtype, device="cuda")
    out = hold[..., 1:1 + dim] if where != "x" else torch.full((n, heads, dim), NAN, dtype=dtype, device="cuda")
    w = _randn(g, dim, dtype=dtype) if norm else None
    positions = torch.randint(0, 5000, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq = _freq(rope)
    hs.hs_norm_rotate(x, out, q_weight=w, eps=EPS, positions=positions, inv_freq=freq, rope_at=at,
                      rotation=hs.HS_ROTATE_PAIRS if pairs else hs.HS_ROTATE_HALVES)
    _close(out, *_rotate_ref(x, w, positions, freq, at, pairs), dtype)
    if where != "x":
        assert (hold[..., 0] == 5).all() and (hold[..., 1 + dim:] == 5).all()


@pytest.mark.parametrize("heads,keys", [(8, 2), (1, 1), (2, 1), (40, 4)])
def test_rotate_packed_in_place(hs, heads, keys):
    """Queries, keys and values side by side in one array, as a projection leaves them; rotated where they lie."""
    g = _gen(heads)
    n, dim = 70, 128
    hold = _randn(g, n, heads + 2 * keys, dim)
    before = hold.clone()
    positions = torch.randint(0, 9999, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq, wq, wk = _freq(dim), _randn(g, dim), _randn(g, dim)
    q, k = hold[:, :heads], hold[:, heads:heads + keys]
    hs.hs_norm_rotate(q, q, k=k, k_out=k, q_weight=wq, k_weight=wk, eps=EPS, positions=positions, inv_freq=freq)
    for got, x, w in ((q, before[:, :heads], wq), (k, before[:, heads:heads + keys], wk)):
        _close(got, *_rotate_ref(x, w, positions, freq, 0, True), BF)
    assert torch.equal(hold[:, heads + keys:], before[:, heads + keys:])


@pytest.mark.parametrize("heads", [2, 12])
def test_rotate_broadcast_input(hs, heads):
    """One head for all, one token for all: strides of 0."""
    g = _gen(heads + 50)
    x = _randn(g, 1, 1, 192).expand(33, heads, 192)
    out = torch.empty((33, heads, 192), dtype=BF, device="cuda")
    positions, freq, w = torch.arange(33, device="cuda", dtype=torch.int32), _freq(64), _randn(g, 192)
    hs.hs_norm_rotate(x, out, q_weight=w, eps=EPS, positions=positions, inv_freq=freq)
    _close(out, *_rotate_ref(x, w, positions, freq, 128, True), BF)


def test_rotate_into_the_absorbed_query(hs):
    """A query's last 64 channels, rotated into the last 64 of the absorbed query's 576."""
    g = _gen(1)
    n, heads = 20, 16
    q, positions, freq = _randn(g, n, heads, 192), _ints(list(range(100, 100 + n))), _freq(64)
    absorbed = torch.full((n, heads, 576), 3.0, dtype=BF, device="cuda")
    hs.hs_norm_rotate(q[..., 128:], absorbed[..., 512:], positions=positions, inv_freq=freq)
    want, slack = _rotate_ref(q[..., 128:], None, positions, freq, 0, True)
    _close(absorbed[..., 512:], want, slack, BF)
    assert (absorbed[..., :512] == 3).all()


@pytest.mark.parametrize("pairs", [True, False])
def test_rotate_far_positions(hs, pairs):
    """Angles of millions of turns, negative positions, frequencies of all sizes and signs."""
    freq = torch.tensor([1.0, 0.999, 0.5, 1e-3, 1e-6, 2.0 ** -40, 0.0, -0.7, 1e-38, 1e-42, 3.0, 100.0], device="cuda")
    values = [0, 1, -1, 131071, 1 << 20, (1 << 24) + 1, 2 ** 31 - 1, -2 ** 31, 1999999999]
    n = len(values)
    x = torch.zeros((n, 1, 24), device="cuda")
    x[..., 0::2 if pairs else 1] = 1.0
    if not pairs:
        x[..., 12:] = 0.0
    out = torch.empty_like(x)
    hs.hs_norm_rotate(x, out, positions=_ints(values), inv_freq=freq,
                      rotation=hs.HS_ROTATE_PAIRS if pairs else hs.HS_ROTATE_HALVES)
    got = out[:, 0].double().cpu().numpy()
    cos, sin = (got[:, 0::2], got[:, 1::2]) if pairs else (got[:, :12], got[:, 12:])
    angle = np.array(values, dtype=np.longdouble)[:, None] * freq.double().cpu().numpy().astype(np.longdouble)
    # the angle to 2^-31 of a turn (100 times that for the frequency 100), its rounding to fp32 (2^-25 of a turn,
    # 2^-22.3 rad), sine and cosine to two steps; the reference's pi is long enough
    tol = 2.0 ** -21 + 2 * math.pi * 2.0 ** -31 * np.maximum(1, freq.abs().cpu().numpy())
    assert (np.abs(cos - np.cos(angle).astype(float)) <= tol).all()
    assert (np.abs(sin - np.sin(angle).astype(float)) <= tol).all()


@pytest.mark.parametrize("freq", [1.0, 0.3, -1e-4])
def test_rotate_sine_and_cosine(hs, freq):
    """Angles in every part of a turn."""
    n = 65536
    x = torch.tensor([1.0, 0.0], device="cuda").repeat(n, 1, 1)
    out = torch.empty_like(x)
    f = torch.tensor([freq], device="cuda")
    positions = torch.arange(n, device="cuda", dtype=torch.int32)
    hs.hs_norm_rotate(x, out, positions=positions, inv_freq=f)
    angle = positions.cpu().numpy().astype(np.longdouble) * np.longdouble(f.item())
    # the angle: 2^-31 of a turn, and its distance from a quarter turn (pi / 4 at most) in 24 bits, 2^-25; the series
    # cut short 2^-24; its evaluation's roundings, steps of values up to 1: 3 half steps of 2^-24 with its last products
    tol = 2 * math.pi * 2.0 ** -31 + 2.0 ** -25 + 2.0 ** -24 + 3 * 2.0 ** -24
    got = out[:, 0].double().cpu().numpy()
    assert np.abs(got[:, 0] - np.cos(angle).astype(float)).max() <= tol
    assert np.abs(got[:, 1] - np.sin(angle).astype(float)).max() <= tol
    assert got[0, 0] == 1 and got[0, 1] == 0


def test_rotate_frequency_not_finite(hs):
    x = torch.ones((1, 1, 4), device="cuda")
    out = torch.empty_like(x)
    hs.hs_norm_rotate(x, out, positions=_ints([1]), inv_freq=torch.tensor([math.inf, 0.0], device="cuda"))
    assert out[0, 0, :2].isnan().all() and (out[0, 0, 2:] == 1).all()


# ---- write -----------------------------------------------------------------------------

def _write_ref(x, weight, positions, freq, pairs):
    """y [n][576] in 64 bits and how far fp32 may be from it."""
    y = torch.cat([_norm64(x[:, :512].double(), weight), x[:, 512:].double()], 1)
    slack = 2.0 ** -15 * y.abs() if weight is not None else torch.zeros_like(y)
    if positions is not None:
        y[:, 512:], terms = _turn64(y[:, 512:].clone(), positions, freq, pairs)
        slack[:, 512:] = 2.0 ** -20 * terms
    return y, slack


def _check_rows(rows, y, slack, e4m3, dtype):
    if not e4m3:
        _close(rows, y, slack, dtype)
        return
    scale = rows[:, 576:580].contiguous().view(F32).double()
    q = rows[:, :576].contiguous().view(torch.float8_e4m3fn).double()
    want = y.abs().amax(1, keepdim=True) / 448.0
    assert bool(((scale - want).abs() <= 2.0 ** -23 * want + slack.amax(1, keepdim=True) / 448 + 1e-44).all())
    some = scale[:, 0] > 0
    assert (q[~some] == 0).all()
    # the quotient in fp32, and a rounding to e4m3: half of 2^-3, or of its least step of 2^-9
    t, off = y[some] / scale[some], slack[some] / scale[some]
    err = (q[some] - t).abs()
    assert bool((err <= 2.0 ** -4 * (1 + 2.0 ** -20) * t.abs() + off + 2.0 ** -10).all()), err.max().item()


@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("turn", ["none", "pairs", "halves"])
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("n", [1, 7, 64, 1000])
def test_write_staged(hs, n, dtype, e4m3, turn, norm):
    g = _gen(n)
    x, w = _randn(g, n, 576, dtype=dtype), _randn(g, 512, dtype=dtype) if norm else None
    positions = torch.randint(0, 131072, (n,), generator=g, device="cuda", dtype=torch.int32) if turn != "none" else None
    freq = _freq(64) if turn != "none" else None
    width = 592 if e4m3 else 1152
    rows = torch.full((n + 2, width), 0xA5, dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, rows, weight=w, eps=EPS, positions=positions, inv_freq=freq,
                       rotation=hs.HS_ROTATE_HALVES if turn == "halves" else hs.HS_ROTATE_PAIRS,
                       row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    got = rows[:n] if e4m3 else rows[:n].view(dtype)
    _check_rows(got, *_write_ref(x, w, positions, freq, turn == "pairs"), e4m3, dtype)
    assert (rows[n:] == 0xA5).all()
    if e4m3:
        assert (rows[:n, 580:] == 0).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new,lengths", [
    ([1], [1]), ([1, 1, 1], [5, 1, 40]), ([3, 0, 40, 1, 0], [3, 7, 40, 33, 0]), ([0, 0, 5], [0, 0, 9]),
    ([10, 6, 4], [4, 50, 2]), ([2] * 100, list(range(2, 102))), ([1] * 1100, [i % 60 for i in range(1100)]),
    ([2] + [0] * 30 + [1] + [0] * 31 + [3] + [0] * 200 + [20, 1], [7] * 266), ([40] * 500, [44] * 500),
    ([0] * 40 + [1] + [0] * 40, [3] * 81)])
def test_write_contexts(hs, new, lengths, e4m3):
    """Ragged tokens at their contexts' ends.  Rows before 0 and behind the last are dropped, as are tokens
    of no request; nothing else changes."""
    g = _gen(len(new))
    n, B, N = sum(new), len(new), 48
    x, w = _randn(g, n + 3, 576), _randn(g, 512)
    positions = torch.randint(0, 999, (n + 3,), generator=g, device="cuda", dtype=torch.int32)
    start = _ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    width = 592 if e4m3 else 1152
    hold = torch.full((B, N + 1, width + 16), 0xA5, dtype=torch.uint8, device="cuda")
    rows = hold[:, :N, :width]
    hs.hs_latent_write(x, rows, weight=w, eps=EPS, positions=positions, inv_freq=_freq(64), start=start,
                       lengths=_ints(lengths), row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    y, slack = _write_ref(x, w, positions, _freq(64), True)
    touched = torch.zeros((B, N + 1), dtype=torch.bool, device="cuda")
    at, tokens, places = 0, [], []
    for b in range(B):
        for i in range(new[b]):
            row = lengths[b] - new[b] + i
            if 0 <= row < N:
                tokens.append(at + i)
                places.append((b, row))
        at += new[b]
    bs, rs = torch.tensor([p[0] for p in places]).cuda(), torch.tensor([p[1] for p in places]).cuda()
    touched[bs, rs] = True
    got = hold[bs, rs][:, :width].contiguous()
    _check_rows(got if e4m3 else got.view(BF), y[tokens], slack[tokens], e4m3, BF)
    assert (hold[~touched] == 0xA5).all() and (hold[..., width:] == 0xA5).all()
    if e4m3:
        assert (hold[touched][:, 580:592] == 0).all()


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("norm", [True, False])
def test_write_values_beside_borders(hs, dtype, norm):
    """8-bit values are those of the exact quotients, but for quotients that lie on a border of e4m3 within what the
    rotation, the norm's root and one rounding leave: 2^-20 of them (the rotary channels': of their pair)."""
    g = _gen(40)
    n = 3000
    x, w = _randn(g, n, 576, dtype=dtype), _randn(g, 512, dtype=dtype) if norm else None
    positions = torch.randint(0, 9999, (n,), generator=g, device="cuda", dtype=torch.int32)
    rows = torch.zeros((n, 592), dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, rows, weight=w, eps=EPS, positions=positions, inv_freq=_freq(64), row_format=hs.HS_ROWS_E4M3)
    y, _ = _write_ref(x, w, positions, _freq(64), True)
    q = 448 * y / y.abs().amax(-1, keepdim=True)
    got = rows[:, :576].contiguous().view(torch.float8_e4m3fn).double()
    want = q.float().to(torch.float8_e4m3fn).double()
    near = 2.0 ** -20 * q.abs()
    pair = q[:, 512:].abs().view(n, 32, 2).sum(-1, keepdim=True).expand(n, 32, 2).reshape(n, 64)
    near[:, 512:] = 2.0 ** -20 * pair
    off = (q - (got + want) / 2).abs()
    assert bool(((got == want) | (off <= near)).all())


def test_write_start_that_lies_outside(hs):
    """start and lengths of any value write nothing outside the rows."""
    x = _randn(_gen(2), 6, 576)
    hold = torch.full((3, 10, 576), 7.0, dtype=BF, device="cuda")
    for start, lengths in (([-5, 2, 2, 100], [2, 8, 4]), ([4, 2, 9, 1], [5, 6, 7]), ([0, 6, 6, 6], [2 ** 31 - 1, 0, 0]),
                           ([0, 6, 6, 6], [-2 ** 31, 0, 0])):
        hold[:] = 7.0
        hs.hs_latent_write(x, hold[:, 2:8], start=_ints(start), lengths=_ints(lengths))
        assert (hold[:, :2] == 7).all() and (hold[:, 8:] == 7).all()


@pytest.mark.parametrize("dtype", [BF, HALF])
def test_write_special_values(hs, dtype):
    """Zeros give scale 0; a NaN makes its own row's scale NaN; large and tiny values."""
    g = _gen(4)
    x = _randn(g, 6, 576, dtype=dtype)
    x[0] = 0
    x[1, 5] = NAN
    x[2, 570] = NAN
    x[3] *= 1e-3 if dtype == HALF else 1e-30
    x[4] *= 1e3 if dtype == HALF else 1e15
    rows = torch.zeros((6, 592), dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, rows, positions=_ints([3] * 6), inv_freq=_freq(64), row_format=hs.HS_ROWS_E4M3)
    scale = rows[:, 576:580].contiguous().view(F32)[:, 0]
    assert scale[0] == 0 and (rows[0, :576].view(torch.float8_e4m3fn).float() == 0).all()  # 0 or -0
    assert scale[1].isnan() and scale[2].isnan()
    keep = [0, 3, 4, 5]
    y, slack = _write_ref(x, None, _ints([3] * 6), _freq(64), True)
    _check_rows(rows[keep], y[keep], slack[keep], True, dtype)


@pytest.mark.parametrize("e4m3", [False, True])
def test_write_requests_in_turn(hs, e4m3):
    """Row i of every request side by side, then row i + 1 of every request: no two rows on one another."""
    B, N = 5, 12
    g = _gen(31)
    new, lengths = [3, 1, 0, 12, 2], [7, 1, 4, 12, 9]
    n, width = sum(new), 592 if e4m3 else 1152
    x, start = _randn(g, n, 576), _ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    kw = dict(start=start, lengths=_ints(lengths), row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    turns = torch.full((N, B, width), 0xA5, dtype=torch.uint8, device="cuda")
    apart = torch.full((B, N, width), 0xA5, dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, turns.transpose(0, 1), **kw)
    hs.hs_latent_write(x, apart, **kw)
    assert torch.equal(turns.transpose(0, 1), apart)
    one_row = torch.full((1, B, width), 0xA5, dtype=torch.uint8, device="cuda")  # a stride that no row uses
    hs.hs_latent_write(x, one_row.transpose(0, 1), **kw)
    assert torch.equal(one_row[0], apart[:, 0])
    with pytest.raises(hs.HsError):
        hs.hs_latent_write(x, turns.transpose(0, 1)[:, :1].expand(B, N, width), **kw)


def test_write_into_the_host_pool(hs):
    """A prompt's rows go to a handle's pinned pool as they are written, and come back from it."""
    B, S, R = 3, 64, 592
    new, lengths = [40, 1, 100], [40, 90, 128]
    g = _gen(8)
    n = sum(new)
    x, w = _randn(g, n, 576), _randn(g, 512)
    start = _ints(np.concatenate([[0], np.cumsum(new)]).tolist())
    positions = torch.arange(n, device="cuda", dtype=torch.int32)
    kw = dict(weight=w, eps=EPS, positions=positions, inv_freq=_freq(64), row_format=hs.HS_ROWS_E4M3)
    staged = torch.zeros((n, R), dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, staged, **kw)
    with hs.Handle(B, 128, R, S, 2) as h:
        pool = h.host_pool()
        pool[:] = 0
        hs.hs_latent_write(x, h, start=start, lengths=_ints(lengths), **kw)
        torch.cuda.synchronize()
        want = np.zeros_like(pool)
        for b, (at, m, end) in enumerate(zip(start.tolist(), new, lengths)):
            want[b, end - m:end] = staged[at:at + m].cpu().numpy()
        assert (pool == want).all()
        out = torch.full((n, 576), NAN, dtype=BF, device="cuda")
        hs.hs_latent_read(h, out, start=start, lengths=_ints(lengths), row_format=hs.HS_ROWS_E4M3)
        assert torch.equal(out, _wide(staged, True).float().to(BF))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("pages", ["base", "huge"])
def test_pool_in_either_placement(hs, pages, e4m3):
    """Contexts written into a pool of ordinary or of huge pages, read back from it, and resolved into the buffer."""
    if pages == "huge" and hs.hs_huge_page_bytes() == 0:
        pytest.skip("the host offers no transparent huge pages")
    B, S, C = 2, 128, 256
    new, lengths = [200, 31], [250, 31]
    g = _gen(32)
    n, R = sum(new), 592 if e4m3 else 1152
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    x, start, ends = _randn(g, n, 576), _ints([0, 200, 231]), _ints(lengths)
    staged, stream = torch.zeros((n, R), dtype=torch.uint8, device="cuda"), torch.cuda.current_stream()
    hs.hs_latent_write(x, staged, row_format=form)
    mode = hs.HS_POOL_PAGES_HUGE if pages == "huge" else hs.HS_POOL_PAGES_BASE
    hs.hs_set_host_pool_pages(mode)
    try:
        h = hs.Handle(B, C, R, S, 2)
    finally:
        hs.hs_set_host_pool_pages(hs.HS_POOL_PAGES_AUTO)
    with h:
        assert hs.hs_host_pool_pages(h.h) == mode
        pool = h.host_pool()
        pool[:] = 0xA5
        hs.hs_latent_write(x, h, start=start, lengths=ends, row_format=form, stream=stream)
        out = torch.full((n, 576), NAN, dtype=BF, device="cuda")
        hs.hs_latent_read(h, out, start=start, lengths=ends, row_format=form, stream=stream)
        torch.cuda.synchronize()
        want = np.full_like(pool, 0xA5)
        want[0, 50:250], want[1, :31] = staged[:200].cpu().numpy(), staged[200:].cpu().numpy()
        assert (pool == want).all()
        values = _wide(staged if e4m3 else staged.view(BF), e4m3).float().to(BF)
        assert torch.equal(out, values)
        topk = torch.stack([50 + torch.randperm(200, generator=g, device="cuda")[:20],
                            torch.randperm(31, generator=g, device="cuda")[:20]]).int()
        slots, picked = torch.empty((B, 20), dtype=torch.int32, device="cuda"), torch.empty((B, 20, 576), dtype=BF, device="cuda")
        h.resolve(topk, 20, slots, stream)
        hs.hs_latent_read(h, picked, slots=slots, row_format=form, dtype=BF, stream=stream)
        assert torch.equal(picked[0], values[topk[0].long() - 50]) and torch.equal(picked[1], values[200 + topk[1].long()])


# ---- read ------------------------------------------------------------------------------

def _check_read(out, want):
    """One product in fp32 of a 4-bit and a 24-bit significand, and one rounding (the product's own moves the
    rounding's place by 2^-24 of the value)."""
    tol = (_half(out.dtype) + 2.0 ** -24) * want.abs() + _least(out.dtype) + 1e-45
    assert bool(((out.double() - want).abs() <= tol).all())


@pytest.mark.parametrize("out_type", [BF, HALF, F32])
@pytest.mark.parametrize("kind", [BF, HALF, "e4m3"])
@pytest.mark.parametrize("B,N,K", [(1, 1, 1), (2, 50, 7), (5, 300, 129), (64, 20, 3), (3, 9, 0)])
def test_read_slots(hs, B, N, K, kind, out_type):
    g = _gen(B + N + K)
    e4m3 = kind == "e4m3"
    rows = _randn(g, B, N, 576, dtype=BF if e4m3 else kind)
    rows = _pack8(rows) if e4m3 else rows
    slots = torch.randint(-2, N + 2, (B, K + 3), generator=g, device="cuda", dtype=torch.int32)[:, 3:]
    if K > 4:
        slots[:, 1] = 2 ** 31 - 1
        slots[:, 2] = -2 ** 31
        slots[:, 4] = slots[:, 3]
    out = torch.full((B, K, 584), NAN, dtype=out_type, device="cuda")
    hs.hs_latent_read(rows, out[..., :576], slots=slots, row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    there = (slots >= 0) & (slots < N)
    want = _wide(rows, e4m3)[torch.arange(B, device="cuda")[:, None], slots.clamp(0, N - 1).long()]
    want = want.masked_fill(~there[..., None], 0.0)
    _check_read(out[..., :576], want)
    assert out[..., 576:].isnan().all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("counts,lengths", [
    ([5], None), ([3, 0, 20, 1], None), ([3, 0, 20, 1], [3, 9, 25, 30]), ([4, 4], [2, 33]), ([1] * 40, list(range(40))),
    ([2] + [0] * 30 + [1] + [0] * 31 + [3] + [0] * 200 + [20, 1], [9] * 266), ([0] * 40 + [1] + [0] * 40, None), ([1] * 70, None)])
def test_read_contexts(hs, counts, lengths, e4m3):
    g = _gen(len(counts))
    B, N, n = len(counts), 30, sum(counts)
    rows = _randn(g, B, N, 576)
    rows = _pack8(rows) if e4m3 else rows
    start = _ints(np.concatenate([[0], np.cumsum(counts)]).tolist())
    out = torch.full((n + 4, 576), 9.0, dtype=BF, device="cuda")
    hs.hs_latent_read(rows, out, start=start, lengths=None if lengths is None else _ints(lengths),
                      row_format=hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT)
    wide, at = _wide(rows, e4m3), 0
    for b, m in enumerate(counts):
        for i in range(m):
            row = i if lengths is None else lengths[b] - m + i
            _check_read(out[at + i], wide[b, row] if 0 <= row < N else torch.zeros_like(wide[b, 0]))
        at += m
    assert (out[n:] == 9).all()


@pytest.mark.parametrize("out_type", [BF, F32])
@pytest.mark.parametrize("e4m3", [False, True])
def test_read_rows_of_16_byte_alignment(hs, e4m3, out_type):
    """Rows inside wider ones, each 16 bytes past a border of 32; outputs likewise; the same row several times."""
    g = _gen(9)
    rows = _form(_randn(g, 3, 20, 576), e4m3)
    raw = rows if e4m3 else rows.view(torch.uint8)
    hold = torch.full((3, 21, raw.shape[-1] + 48), 255, dtype=torch.uint8, device="cuda")
    hold[:, :20, 16:16 + raw.shape[-1]] = raw
    inside = hold[:, :20, 16:16 + raw.shape[-1]]
    skip = 16 // torch.empty((), dtype=out_type).element_size()
    out = torch.full((3, 40, 576 + 2 * skip), NAN, dtype=out_type, device="cuda")
    slots = torch.randint(0, 20, (3, 40), generator=g, device="cuda", dtype=torch.int32)
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    hs.hs_latent_read(inside, out[..., skip:skip + 576], slots=slots, row_format=form, dtype=BF)
    _check_read(out[..., skip:skip + 576], _wide(rows, e4m3)[torch.arange(3, device="cuda")[:, None], slots.long()])
    assert out[..., :skip].isnan().all() and out[..., skip + 576:].isnan().all()


def test_read_special_values(hs):
    rows = _pack8(_randn(_gen(5), 1, 4, 576))
    rows[0, 1, 7] = 0x7F                                            # e4m3 NaN
    rows[0, 2, 576:580] = torch.tensor([math.inf], device="cuda").view(torch.uint8)
    out = torch.empty((1, 4, 576), device="cuda")
    hs.hs_latent_read(rows, out, slots=_ints([[0, 1, 2, 3]]), row_format=hs.HS_ROWS_E4M3, dtype=BF)
    assert torch.isfinite(out[0, [0, 3]]).all() and out[0, 1].isnan().sum() == 1
    assert (~torch.isfinite(out[0, 2])).all()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("nq,nk", [([30, 1, 200], [300, 500, 200]), ([5, 0, 129], [5, 0, 700])])
def test_read_contexts_for_a_prompt(hs, nq, nk, e4m3):
    """A prompt's next chunk: the cached rows of its contexts are read back, the chunk's own among them, and the
    prompt's attention takes them as its rows."""
    g = _gen(sum(nq))
    q, rows, w_uk, w_uv = _prompt_case(nq, nk, 2, BF, False, sum(nk))
    N, start = 720, _ints(np.concatenate([[0], np.cumsum(nk)]).tolist())
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    cache = torch.full((len(nk), N, 592 if e4m3 else 1152), 0xFF, dtype=torch.uint8, device="cuda")  # NaN
    positions, freq, w = torch.randint(0, 9999, (sum(nk),), generator=g, device="cuda", dtype=torch.int32), _freq(64), _randn(g, 512)
    hs.hs_latent_write(rows, cache, weight=w, eps=EPS, positions=positions, inv_freq=freq, start=start, lengths=_ints(nk), row_format=form)
    back = torch.full((sum(nk), 576), NAN, dtype=BF, device="cuda")
    hs.hs_latent_read(cache, back, start=start, lengths=_ints(nk), row_format=form)
    held = torch.cat([cache[b, :m] for b, m in enumerate(nk)])
    assert torch.equal(back, _wide(held if e4m3 else held.view(BF), e4m3).float().to(BF))
    _check_prefill(*_prefill(hs, q, back, w_uk, w_uv, nq, nk), q, back, w_uk, w_uv, nq, nk, False)


def test_read_handle_slots(hs):
    """What a resolve step returned, as values."""
    B, S, R, K = 2, 32, 1152, 16
    g = _gen(6)
    with hs.Handle(B, 64, R, S, 2) as h:
        rows = _randn(g, B, 64, 576)
        h.host_pool()[:] = rows.view(torch.uint8).cpu().numpy()
        topk = torch.stack([torch.randperm(64, generator=g, device="cuda")[:K] for _ in range(B)]).int()
        slots = torch.empty((B, K), dtype=torch.int32, device="cuda")
        h.resolve(topk, K, slots, torch.cuda.current_stream())
        out = torch.empty((B, K, 576), dtype=BF, device="cuda")
        hs.hs_latent_read(h, out, slots=slots, stream=torch.cuda.current_stream())
        assert torch.equal(out, torch.gather(rows, 1, topk.long()[..., None].expand(-1, -1, 576)))


# ---- shared ----------------------------------------------------------------------------

def _shared_ref(q, prefix, seen, rows, picked, e4m3, scale):
    """seen[b]: rows of the prefix; picked[b][p]: own rows."""
    B, P, H, _ = q.shape
    o = torch.zeros((B, P, H, 512), dtype=torch.float64, device="cuda")
    mean_abs, lse = torch.zeros_like(o), torch.zeros((B, P, H), dtype=torch.float64, device="cuda")
    reach = torch.zeros((B, P, H, 1), dtype=torch.float64, device="cuda")
    first = _wide(prefix, e4m3)
    for b in range(B):
        for p in range(P):
            k = torch.cat([first[:seen[b]], _wide(rows[b][picked[b][p]], e4m3)])
            s = scale * (q[b, p].double() @ k.t())
            o[b, p], lse[b, p], mean_abs[b, p] = _softmax_ref(s, k[:, :512])
            if k.shape[0]:
                reach[b, p] = abs(scale) * (q[b, p].double().abs() @ k.abs().t()).amax(-1, keepdim=True)
    return o, lse, mean_abs, reach


def _check_shared(out, lse, ref, dtype):
    o, want_lse, mean_abs, reach = ref
    half = _half(dtype)
    # scores: 576 fp32 additions of terms that sum to at most `reach` in magnitude, each off by a step of fp32 at
    # most; exp, the logs, the sums over the rows and the way of the own rows' part through its log add a few more
    score = 576 * 2.0 ** -23 * reach + 2.0 ** -17
    # out: its own rounding; that of the own rows' part; each weight rounded once; a score off by e moves the mean
    # by 2 e sum p|v|
    tol = half * o.abs() + (2 * half + 2 * score) * mean_abs + _least(dtype) + 1e-30
    err = (out.double() - o).abs()
    assert torch.isfinite(out).all()
    assert bool((err <= tol).all()), (err / tol).max().item()
    # roundings are independent: three of at most half a step each, in the 2-norm
    assert err.norm() <= (1.75 * half + 1e-4) * o.norm() + 1e-30, (err.norm() / o.norm()).item()
    empty = want_lse == -math.inf
    assert (lse[empty] == -math.inf).all() and (out[empty] == 0).all()
    lse_err = (lse.double() - want_lse)[~empty].abs()
    assert (lse_err <= (score.squeeze(-1) + 2.0 ** -20 * want_lse.abs())[~empty]).all()


def _shared(hs, q, prefix, rows, scale=SCALE, e4m3=False, stream=None, **kw):
    B, P, H, _ = q.shape
    out = torch.full((B, P, H, 512), NAN, dtype=q.dtype, device="cuda")
    lse = torch.full((B, P, H), NAN, device="cuda")
    slots = kw.get("slots")
    n = slots.shape[-1] if slots is not None else rows.shape[1]
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    ws = torch.full((hs.hs_latent_attend_shared_workspace(B, P, H, n, prefix.shape[0], form),), 255, dtype=torch.uint8, device="cuda")
    hs.hs_workspace_clear(ws)
    hs.hs_latent_attend_shared(q, prefix, rows, out, scale, lse=lse, workspace=ws, stream=stream, row_format=form, **kw)
    assert hs.hs_workspace_error(ws) == 0
    return out, lse


def _form(rows, e4m3):
    return _pack8(rows) if e4m3 else rows


SHARED = [  # batch, positions, heads, prefix, own rows
    (1, 1, 1, 1, 1), (2, 1, 16, 64, 5), (3, 1, 20, 129, 40), (1, 1, 128, 128, 10), (5, 3, 20, 1000, 70), (2, 1, 200, 333, 30),
    (64, 1, 16, 700, 100), (9, 1, 128, 2000, 64), (300, 1, 3, 65, 9), (1, 2, 7, 9000, 20), (40, 1, 128, 300, 33), (1, 1, 16, 1, 300),
    (200, 1, 128, 100, 3), (80, 1, 64, 5000, 2), (160, 1, 128, 2000, 5), (100, 1, 128, 600, 9)]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("size", SHARED)
def test_shared_lengths(hs, size, dtype, e4m3):
    """Ragged own contexts, some empty, behind a prefix that all see whole."""
    B, P, H, M, N = size
    g = _gen(sum(size))
    q, prefix, rows = (_randn(g, *s, dtype=dtype) for s in ((B, P, H, 576), (M, 576), (B, N, 576)))
    lengths = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    lengths[0] = N
    for b, n in enumerate(lengths.tolist()):
        rows[b, n:] = NAN
    prefix, rows = _form(prefix, e4m3), _form(rows, e4m3)
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, lengths=lengths)
    picked = [[torch.arange(max(0, n - P + 1 + p), device="cuda") for p in range(P)] for n in lengths.tolist()]
    _check_shared(out, lse, _shared_ref(q, prefix, [M] * B, rows, picked, e4m3, SCALE), dtype)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("size", [(3, 1, 16, 200, 90), (7, 2, 20, 600, 60), (70, 1, 16, 3000, 50), (20, 1, 128, 700, 40), (150, 1, 1, 400, 9),
                                  (90, 1, 128, 400, 10), (170, 1, 128, 300, 20)])
def test_shared_slots_and_lengths_of_the_prefix(hs, size, e4m3):
    """Own rows by lists with absent entries; prefixes of all lengths, 0 and values outside among them; what no one
    sees of either holds NaN."""
    B, P, H, M, N = size
    g = _gen(sum(size))
    q, prefix, rows = (_randn(g, *s) for s in ((B, P, H, 576), (M, 576), (B, N, 576)))
    K = N // 2
    slots = torch.rand((B, P, N), generator=g, device="cuda").topk(K, -1).indices.int()
    slots = slots.masked_fill(torch.rand(slots.shape, generator=g, device="cuda") < 0.4, -1)
    slots[1] = -1
    seen = torch.randint(0, M - 80, (B,), generator=g, device="cuda", dtype=torch.int32)
    seen[0], seen[1], seen[2] = 0, 0, M - 80
    prefix[M - 80:] = NAN
    prefix, rows = _form(prefix, e4m3), _form(rows, e4m3)
    given = seen.clone()
    given[0] = -7
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, slots=slots, prefix_lengths=given)
    picked = [[s[s >= 0].long() for s in req] for req in slots]
    ref = _shared_ref(q, prefix, seen.tolist(), rows, picked, e4m3, SCALE)
    _check_shared(out, lse, ref, BF)
    given[2] = 2 ** 31 - 1  # clamped; the shorter prefix is cut in other pieces, so the bits may differ
    _check_shared(*_shared(hs, q, prefix[:M - 80], rows, e4m3=e4m3, slots=slots, prefix_lengths=given), ref, BF)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
def test_shared_prefix_rows_that_are_not_finite(hs, value, e4m3):
    """They make the outputs of those that see them NaN, and no one else's."""
    if e4m3 and value != value:
        value = math.inf
    g = _gen(12)
    B, M = 6, 300
    q, prefix, rows = _randn(g, B, 1, 16, 576), _randn(g, M, 576), _randn(g, B, 20, 576)
    plain = _form(prefix.clone(), e4m3)
    prefix = _form(prefix, e4m3)
    if e4m3:
        prefix[200, 576:580] = torch.tensor([value], device="cuda").view(torch.uint8)
    else:
        prefix[200, 100] = value
    rows = _form(rows, e4m3)
    seen, lengths = _ints([300, 200, 0, 201, 150, 10]), _ints([20] * B)
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, lengths=lengths, prefix_lengths=seen)
    want, want_lse = _shared(hs, q, plain, rows, e4m3=e4m3, lengths=lengths, prefix_lengths=seen)
    assert out[[0, 3]].isnan().all()
    rest = [1, 2, 4, 5]
    assert torch.equal(out[rest], want[rest]) and torch.equal(lse[rest], want_lse[rest])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("size", [(1, 1, 16, 3001, 2048), (8, 1, 16, 2000, 2048), (5, 3, 20, 900, 1100), (1, 1, 128, 3001, 2048),
                                  (8, 1, 128, 5000, 1500), (40, 1, 16, 4000, 1030), (3, 1, 200, 300, 4096)])
def test_shared_long_lists(hs, size, e4m3):
    """Own rows by lists of more than 16 tiles: the own rows' part in pieces before the prefix's kernel, or in whole
    units beside it."""
    B, P, H, M, K = size
    g = _gen(sum(size))
    N = K + 37
    q, prefix, rows = _randn(g, B, P, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
    slots = torch.rand((B, P, N), generator=g, device="cuda").topk(K, -1).indices.int()
    slots = slots.masked_fill(torch.rand(slots.shape, generator=g, device="cuda") < 0.1, -1)
    picked = [[s[s >= 0].long() for s in req] for req in slots]
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, slots=slots)
    _check_shared(out, lse, _shared_ref(q, prefix, [M] * B, rows, picked, e4m3, SCALE), BF)
    seen = torch.randint(0, M + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, slots=slots, prefix_lengths=seen)
    _check_shared(out, lse, _shared_ref(q, prefix, seen.tolist(), rows, picked, e4m3, SCALE), BF)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("B,H,M", [(1, 16, 3001), (6, 16, 700), (2, 128, 1000)])
def test_shared_over_what_a_resolve_step_returned(hs, B, H, M, e4m3):
    """The own rows lie in a handle's device buffer, at the slots that its resolve steps return."""
    K, C, S = 1200, 3000, 1500
    g = _gen(B + H)
    q, prefix, rows = _randn(g, B, 1, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, C, 576), e4m3)
    form, raw = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT, rows.view(torch.uint8)
    stream = torch.cuda.current_stream()
    out, lse = torch.empty((B, 1, H, 512), dtype=BF, device="cuda"), torch.empty((B, 1, H), device="cuda")
    ws = torch.empty(hs.hs_latent_attend_shared_workspace(B, 1, H, K, M, form), dtype=torch.uint8, device="cuda")
    hs.hs_workspace_clear(ws)
    with hs.Handle(B, C, raw.shape[-1], S, 2) as h:
        h.host_pool()[:, :C] = raw.cpu().numpy()
        for step in range(2):  # the second evicts
            topk = torch.stack([torch.randperm(C, generator=g, device="cuda")[:K] for _ in range(B)]).int()
            slots = torch.full((B, 1, K), -5, dtype=torch.int32, device="cuda")
            h.resolve(topk, K, slots, stream)
            hs.hs_latent_attend_shared(q, prefix, h, out, SCALE, slots=slots, lse=lse, workspace=ws, row_format=form, stream=stream)
            picked = [[t.long()] for t in topk]
            _check_shared(out, lse, _shared_ref(q, prefix, [M] * B, rows, picked, e4m3, SCALE), BF)
        assert h.stats()["err_bits"] == 0 and hs.hs_workspace_error(ws) == 0


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("channel", [100, 540])
@pytest.mark.parametrize("size", [(6, 16), (3, 128)])
@pytest.mark.parametrize("value", [NAN, math.inf, -math.inf])
def test_shared_prefix_values_that_are_not_finite_without_lengths(hs, value, size, channel, dtype):
    """16-bit rows that all see, taken as they are: a NaN, or a score of +inf, makes a head's output NaN; a score of
    -inf is a weight of 0, and leaves all but an infinite latent channel (0 times it).  With lengths that cover the
    prefix such a row makes all of them NaN."""
    B, H = size
    g = _gen(B + channel)
    M = 300
    q, prefix, rows = _randn(g, B, 1, H, 576, dtype=dtype), _randn(g, M, 576, dtype=dtype), _randn(g, B, 20, 576, dtype=dtype)
    q[..., channel] = torch.where(q[..., channel] == 0, 1.0, q[..., channel])  # no 0 times infinity
    lengths, every = _ints([20] * B), [[torch.arange(20, device="cuda")] for _ in range(B)]
    prefix[200, channel] = value
    out, _ = _shared(hs, q, prefix, rows, lengths=lengths)
    score = q[:, 0, :, channel].double() * value
    below = score == -math.inf  # the others are +inf or NaN
    assert out[:, 0][~below].isnan().all() and (value != value or bool(below.any()) and bool((~below).any()))
    off = torch.zeros(512, dtype=torch.bool, device="cuda")
    off[channel:channel + 1] = True
    # without the row: a weight of 0 adds nothing, and the rows' order and tiles are those of zeros in its place
    without = torch.cat([prefix[:200], prefix[201:]])
    o, _, mean_abs, reach = _shared_ref(q, without, [M - 1] * B, rows, every, False, SCALE)
    half, score = _half(dtype), 576 * 2.0 ** -23 * reach + 2.0 ** -17
    tol = half * o.abs() + (2 * half + 2 * score) * mean_abs + _least(dtype) + 1e-30  # as in _check_shared
    err = (out.double() - o).abs()[:, 0][below][:, ~off]
    assert bool((err <= tol[:, 0][below][:, ~off]).all())
    out, _ = _shared(hs, q, prefix, rows, lengths=lengths, prefix_lengths=_ints([M] * B))
    assert out.isnan().all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_without_own_rows_or_prefix(hs, e4m3):
    g = _gen(13)
    B, P, H, M = 5, 1, 24, 500
    q, prefix, rows = _randn(g, B, P, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, 40, 576), e4m3)
    none = [[torch.arange(0, device="cuda")] for _ in range(B)]
    every = [[torch.arange(40, device="cuda")] for _ in range(B)]
    ref = _shared_ref(q, prefix, [M] * B, rows, none, e4m3, SCALE)
    for kw in (dict(lengths=_ints([0] * B)), dict(slots=_ints([[]] * B).view(B, 1, 0)), dict(slots=_ints([[-1, -1]] * B).view(B, 1, 2))):
        _check_shared(*_shared(hs, q, prefix, rows, e4m3=e4m3, **kw), ref, BF)
    _check_shared(*_shared(hs, q, prefix, rows[:, :0], e4m3=e4m3, lengths=_ints([7] * B)), ref, BF)
    ref = _shared_ref(q, prefix, [0] * B, rows, every, e4m3, SCALE)
    full = _ints([40] * B)
    _check_shared(*_shared(hs, q, prefix[:0], rows, e4m3=e4m3, lengths=full), ref, BF)
    _check_shared(*_shared(hs, q, prefix, rows, e4m3=e4m3, lengths=full, prefix_lengths=_ints([0] * B)), ref, BF)
    out, lse = _shared(hs, q, prefix, rows, e4m3=e4m3, lengths=_ints([0] * B), prefix_lengths=_ints([0] * B))
    assert (out == 0).all() and (lse == -math.inf).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_strides(hs, e4m3):
    """Queries and outputs inside larger arrays in another axis order, padded rows; no lse."""
    B, P, H, M, N = 3, 2, 12, 200, 30
    g = _gen(14)
    q, prefix, rows = _randn(g, B, P, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
    lengths = _ints([30, 2, 17])
    want, _ = _shared(hs, q, prefix, rows, e4m3=e4m3, lengths=lengths)
    wide = torch.zeros((H, P, B, 600), dtype=BF, device="cuda")
    wide[..., 8:584] = q.permute(2, 1, 0, 3)
    raw = prefix if e4m3 else prefix.view(torch.uint8)
    padded = torch.full((M + 5, raw.shape[-1] + 48), 255, dtype=torch.uint8, device="cuda")
    padded[2:M + 2, 16:16 + raw.shape[-1]] = raw
    hold = torch.full((P, B, H, 520), 3.0, dtype=BF, device="cuda")
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    ws = torch.empty(hs.hs_latent_attend_shared_workspace(B, P, H, N, M, form), dtype=torch.uint8, device="cuda")
    hs.hs_latent_attend_shared(wide[..., 8:584].permute(2, 1, 0, 3), padded[2:M + 2, 16:16 + raw.shape[-1]], rows,
                               hold[..., :512].transpose(0, 1), SCALE, lengths=lengths, workspace=ws, row_format=form)
    assert torch.equal(hold[..., :512].transpose(0, 1), want) and (hold[..., 512:] == 3).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_strides_with_lengths(hs, e4m3):
    """One query for all requests (a stride of 0), and prefix rows 16 bytes past borders of 32, with lengths."""
    B, H, M, N = 5, 16, 300, 20
    g = _gen(21)
    q, prefix, rows = _randn(g, 1, 1, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
    raw = prefix if e4m3 else prefix.view(torch.uint8)
    padded = torch.full((M, raw.shape[-1] + 48), 255, dtype=torch.uint8, device="cuda")
    padded[:, 16:16 + raw.shape[-1]] = raw
    seen, lengths = [300, 0, 129, 7, 256], [20, 1, 0, 9, 20]
    kw = dict(e4m3=e4m3, lengths=_ints(lengths), prefix_lengths=_ints(seen))
    picked = [[torch.arange(n, device="cuda")] for n in lengths]
    every = q.expand(B, 1, H, 576)
    got = _shared(hs, every, padded[:, 16:16 + raw.shape[-1]], rows, **kw)
    _check_shared(*got, _shared_ref(every, prefix, seen, rows, picked, e4m3, SCALE), BF)


@pytest.mark.parametrize("dtype", [BF, HALF])
@pytest.mark.parametrize("size", [(20, 2, 128, 54, 842), (16, 1, 16, 1, 700), (90, 1, 32, 30, 500), (5, 1, 16, 64, 2000)])
def test_shared_mostly_own_rows_are_rounded_once(hs, size, dtype):
    """The own rows' part comes unrounded into the join."""
    B, P, H, M, N = size
    g = _gen(sum(size))
    q, prefix, rows = (_randn(g, *s, dtype=dtype) for s in ((B, P, H, 576), (M, 576), (B, N, 576)))
    lengths = _ints([N] * B)
    out, _ = _shared(hs, q, prefix, rows, lengths=lengths)
    picked = [[torch.arange(N - P + 1 + p, device="cuda") for p in range(P)] for _ in range(B)]
    o = _shared_ref(q, prefix, [M] * B, rows, picked, False, SCALE)[0]
    # A rounding is off by at most half a step, u of the power of two below the value; evenly spread and over a
    # mantissa m whose logarithm is evenly spread, its 2-norm is u sqrt(E[1 / m^2] / 3) = u sqrt(3 / (8 ln 2) / 3) =
    # 0.425 u of the value's.  The weights (their errors independent, and values of no common sign) and the output:
    # 0.425 sqrt 2 = 0.601 u; the part rounded in between would make it 0.736.
    assert (out.double() - o).norm() <= 0.64 * _half(dtype) * o.norm()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("std,scale", [(0.0, SCALE), (30.0, SCALE), (1.0, -0.05), (1.0, 0.0)])
def test_shared_flat_and_peaked(hs, std, scale, e4m3):
    g = _gen(15)
    B, H, M, N = 4, 16, 900, 100
    q, prefix, rows = _randn(g, B, 1, H, 576, std=std), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
    out, lse = _shared(hs, q, prefix, rows, scale=scale, e4m3=e4m3, lengths=_ints([N] * B))
    every = [[torch.arange(N, device="cuda")] for _ in range(B)]
    _check_shared(out, lse, _shared_ref(q, prefix, [M] * B, rows, every, e4m3, scale), BF)


@pytest.mark.parametrize("rising", [True, False])
def test_shared_scores_that_rise_along_the_prefix(hs, rising):
    """Each tile's scores lie far above the last one's, so that the sums are rescaled at every tile; or far below."""
    g = _gen(16)
    B, H, M, N = 3, 16, 1500, 10
    u = torch.randn((1, 576), generator=g, device="cuda")
    ramp = torch.linspace(0, 2, M, device="cuda")[:, None]
    q = (u * (1 + 0.01 * torch.randn((B, 1, H, 1), generator=g, device="cuda"))).to(BF)
    prefix = (u * (ramp if rising else 2 - ramp) + 0.05 * torch.randn((M, 576), generator=g, device="cuda")).to(BF)
    rows = _randn(g, B, N, 576)
    out, lse = _shared(hs, q, prefix, rows, lengths=_ints([N] * B))
    every = [[torch.arange(N, device="cuda")] for _ in range(B)]
    _check_shared(out, lse, _shared_ref(q, prefix, [M] * B, rows, every, False, SCALE), BF)


@pytest.mark.parametrize("dtype", [BF, HALF])
def test_shared_row_scales_of_many_sizes(hs, dtype):
    g = _gen(17)
    prefix = torch.randn((700, 576), generator=g, device="cuda")
    prefix *= torch.exp2(torch.randint(-20, 7, (700, 1), generator=g, device="cuda").float())
    prefix[::50] = 0
    prefix, rows = _pack8(prefix), _pack8(_randn(g, 2, 50, 576))
    q = _randn(g, 2, 1, 16, 576, dtype=dtype, std=0.05)
    out, lse = _shared(hs, q, prefix, rows, e4m3=True, lengths=_ints([50, 50]))
    every = [[torch.arange(50, device="cuda")] for _ in range(2)]
    _check_shared(out, lse, _shared_ref(q, prefix, [700] * 2, rows, every, True, SCALE), dtype)


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_same_bits_again_on_another_stream_and_in_a_graph(hs, e4m3):
    g = _gen(18)
    B, H, M, N = 12, 16, 4000, 200
    q, prefix, rows = _randn(g, B, 1, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
    lengths, seen = _ints([N] * B), _ints([M - 10 * b for b in range(B)])
    kw = dict(e4m3=e4m3, lengths=lengths, prefix_lengths=seen)
    want, want_lse = _shared(hs, q, prefix, rows, **kw)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        out, lse = _shared(hs, q, prefix, rows, stream=side, **kw)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    ws = torch.empty(hs.hs_latent_attend_shared_workspace(B, 1, H, N, M, form), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        hs.hs_latent_attend_shared(q, prefix, rows, out, SCALE, lengths=lengths, prefix_lengths=seen, workspace=ws,
                                   row_format=form, stream=torch.cuda.current_stream())
    for _ in range(3):
        out.fill_(NAN)
        graph.replay()
        assert torch.equal(out, want)
    lengths.fill_(3)  # a replay reads what the arrays hold then
    seen.fill_(77)
    graph.replay()
    short, _ = _shared(hs, q, prefix, rows, **kw)
    assert torch.equal(out, short)


@pytest.mark.parametrize("partial", [False, True])
@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_calls_behind_one_another(hs, e4m3, partial):
    """Calls of several sizes on one stream, in one workspace, none waited for; each is followed at once by work that
    overwrites its inputs."""
    g = _gen(22)
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    sizes = [(20, 1, 16, 5000, 300), (3, 2, 20, 700, 500), (2, 1, 128, 20000, 40), (160, 1, 128, 300, 5), (1, 1, 1, 65, 3000)]
    ws = torch.empty(max(hs.hs_latent_attend_shared_workspace(B, P, H, N, M, form) for B, P, H, M, N in sizes), dtype=torch.uint8, device="cuda")
    made = []
    for B, P, H, M, N in sizes:
        q, prefix, rows = _randn(g, B, P, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
        lengths = torch.randint(0, N + 1, (B,), generator=g, device="cuda", dtype=torch.int32)
        seen = torch.randint(0, M + 1, (B,), generator=g, device="cuda", dtype=torch.int32) if partial else None
        kw = dict(lengths=lengths, prefix_lengths=seen)
        made.append((q, prefix, rows, kw, _shared(hs, q, prefix, rows, e4m3=e4m3, **kw)[0]))
    kept = [(q.clone(), prefix.clone(), rows.clone()) for q, prefix, rows, _, _ in made]
    outs = []
    for _ in range(4):
        for (q, prefix, rows, kw, _), copies in zip(made, kept):
            out = torch.empty(q.shape[:-1] + (512,), dtype=BF, device="cuda")
            hs.hs_latent_attend_shared(q, prefix, rows, out, SCALE, workspace=ws, row_format=form,
                                       stream=torch.cuda.current_stream(), **kw)
            for x in (q, prefix, rows):
                x.zero_()
            for x, copy in zip((q, prefix, rows), copies):
                x.copy_(copy)
            outs.append(out)
    for i, out in enumerate(outs):
        assert torch.equal(out, made[i % len(made)][4])


@pytest.mark.parametrize("e4m3", [False, True])
def test_shared_two_calls_at_once(hs, e4m3):
    """Calls on two streams that overlap, each with a workspace of its own."""
    g = _gen(19)
    form = hs.HS_ROWS_E4M3 if e4m3 else hs.HS_ROWS_16BIT
    calls = []
    for B, H, M, N in ((20, 16, 5000, 300), (3, 128, 9000, 40)):
        q, prefix, rows = _randn(g, B, 1, H, 576), _form(_randn(g, M, 576), e4m3), _form(_randn(g, B, N, 576), e4m3)
        lengths = _ints([N] * B)
        want, _ = _shared(hs, q, prefix, rows, e4m3=e4m3, lengths=lengths)
        ws = torch.empty(hs.hs_latent_attend_shared_workspace(B, 1, H, N, M, form), dtype=torch.uint8, device="cuda")
        calls.append((q, prefix, rows, lengths, torch.empty_like(want), ws, torch.cuda.Stream(), want))
    torch.cuda.synchronize()
    for _ in range(5):
        for q, prefix, rows, lengths, out, ws, stream, _ in calls:
            hs.hs_latent_attend_shared(q, prefix, rows, out, SCALE, lengths=lengths, workspace=ws, row_format=form, stream=stream)
    torch.cuda.synchronize()
    for call in calls:
        assert torch.equal(call[4], call[7])


_FIRST_IN_A_GRAPH = """
import torch
from hierarchical_kv_cache_hs_gb300 import hs
bf, i32 = torch.bfloat16, torch.int32
def randn(*s): return torch.randn(s, device="cuda").to(bf)
x, q, prefix, qa = randn(40, 576), randn(40, 16, 192), randn(300, 576), randn(2, 1, 16, 576)
rows, back = torch.zeros(2, 30, 576, dtype=bf, device="cuda"), torch.zeros(40, 576, dtype=bf, device="cuda")
start, lengths = (torch.tensor(v, dtype=i32, device="cuda") for v in ([0, 20, 40], [25, 30]))
positions, freq, turned = torch.arange(40, dtype=i32, device="cuda"), torch.rand(32, device="cuda"), torch.empty_like(q)
out = torch.zeros(2, 1, 16, 512, dtype=bf, device="cuda")
ws = torch.empty(hs.hs_latent_attend_shared_workspace(2, 1, 16, 30, 300), dtype=torch.uint8, device="cuda")
def calls(s):
    hs.hs_latent_write(x, rows, positions=positions, inv_freq=freq, start=start, lengths=lengths, stream=s)
    hs.hs_latent_read(rows, back, start=start, lengths=lengths, stream=s)
    hs.hs_norm_rotate(q, turned, positions=positions, inv_freq=freq, stream=s)
    hs.hs_latent_attend_shared(qa, prefix, rows, out, 0.07, lengths=lengths, prefix_lengths=lengths, workspace=ws, stream=s)
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    calls(torch.cuda.current_stream())
graph.replay()
torch.cuda.synchronize()
found = [t.clone() for t in (rows, back, turned, out)]
assert all(f.abs().sum() > 0 for f in found)
calls(torch.cuda.current_stream())
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(found, (rows, back, turned, out)))
"""


def test_no_tokens(hs):
    """Calls of no tokens change nothing, keys or not."""
    x, q, k = (torch.zeros(s, dtype=BF, device="cuda") for s in ((0, 576), (0, 16, 192), (0, 2, 192)))
    rows, out = torch.full((2, 3, 576), 7.0, dtype=BF, device="cuda"), torch.full((5, 576), 7.0, dtype=BF, device="cuda")
    start, lengths, none, freq, w = _ints([0, 0, 0]), _ints([1, 3]), _ints([]), _freq(64), torch.ones(192, dtype=BF, device="cuda")
    hs.hs_latent_write(x, rows, positions=none, inv_freq=freq, start=start, lengths=lengths)
    hs.hs_latent_write(x, rows[0], positions=none, inv_freq=freq)
    hs.hs_latent_read(rows, out[:0], start=start, lengths=lengths)
    hs.hs_latent_read(rows, out, start=start)
    hs.hs_norm_rotate(q, q, positions=none, inv_freq=freq)
    hs.hs_norm_rotate(q, q, k=k, k_out=k, q_weight=w, k_weight=w, eps=EPS, positions=none, inv_freq=freq)
    assert (rows == 7).all() and (out == 7).all()


def test_first_calls_in_a_graph():
    """A program whose first calls are captured."""
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_IN_A_GRAPH], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]


def test_rows_behind_32_bits(hs):
    """Rows whose byte offsets pass 2^32, written and read back."""
    n = 7_500_000  # 8-bit rows: 4.4 GB
    rows = torch.zeros((1, n, 592), dtype=torch.uint8, device="cuda")
    g = _gen(20)
    x = _randn(g, 33, 576)
    hs.hs_latent_write(x, rows, start=_ints([0, 33]), lengths=_ints([n]), row_format=hs.HS_ROWS_E4M3)
    staged = torch.zeros((33, 592), dtype=torch.uint8, device="cuda")
    hs.hs_latent_write(x, staged, row_format=hs.HS_ROWS_E4M3)
    assert torch.equal(rows[0, -33:], staged) and not rows[0, :-33].any()
    out = torch.empty((1, 33, 576), dtype=BF, device="cuda")
    hs.hs_latent_read(rows, out, slots=torch.arange(n - 33, n, dtype=torch.int32, device="cuda")[None], row_format=hs.HS_ROWS_E4M3)
    assert torch.equal(out[0], _wide(staged, True).float().to(BF))


@pytest.mark.parametrize("e4m3", [True, False])
def test_together_in_the_example(e4m3):
    """Rows written into the pool and as contexts, heads rotated, a shared prompt, rows read back, as a serving
    loop uses them."""
    from hierarchical_kv_cache_hs_gb300.examples import latent_decode as ex
    got = ex.run(e4m3=e4m3, seed=3)
    assert got["errors"] == 0 and got["waits_ran_out"] == 0
    assert got["read"] <= 2.0 ** -24  # fp32 values of rows: one product each
    # three roundings of at most half a step (weights, the own rows' part, output), in the 2-norm
    assert got["shared"] <= 1.75 * 2 ** -8 and got["decode"] <= 1.5 * 2 ** -8
