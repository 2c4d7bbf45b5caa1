"""The operators beside the swap-in path without a GPU: what the library and
the binding refuse, before any CUDA call."""
import ctypes

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def hs():
    from hierarchical_kv_cache_hs_gb300 import build
    build.build_libhs()
    from hierarchical_kv_cache_hs_gb300 import hs as mod
    return mod


def _attend(hs, **over):
    a = hs.hs_attend_t()
    a.dtype, a.row_format, a.batch, a.positions, a.heads, a.entries = 0, 0, 2, 1, 16, 64
    a.n_rows, a.q, a.rows, a.out, a.slots = 128, 1 << 20, 1 << 21, 1 << 22, 1 << 23
    a.row_stride, a.request_stride, a.scale = 1152, 128 * 1152, 0.1
    a.q_stride, a.out_stride = (16 * 576, 16 * 576, 576), (16 * 512, 16 * 512, 512)
    a.slots_stride = (64, 64)
    a.workspace, a.workspace_bytes = 1 << 24, 1 << 40
    for k, v in over.items():
        setattr(a, k, v)
    return hs.lib.hs_latent_attend(ctypes.byref(a), None)


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(dtype=-1), dict(row_format=2), dict(batch=0), dict(positions=0),
    dict(heads=0), dict(entries=-1), dict(n_rows=-1), dict(q=None), dict(out=None), dict(rows=None),
    dict(slots=None), dict(lengths=1 << 25), dict(scale=float("nan")), dict(scale=float("inf")),
    dict(q=(1 << 20) + 8), dict(out=(1 << 22) + 2), dict(rows=(1 << 21) + 8), dict(slots=(1 << 23) + 2),
    dict(lse=(1 << 26) + 2), dict(workspace=(1 << 24) + 8), dict(workspace_bytes=8), dict(workspace=None),
    dict(q_stride=(16 * 576, 16 * 576, 577)), dict(out_stride=(-512, 0, 512)), dict(row_stride=1136),
    dict(row_stride=1160), dict(request_stride=8), dict(slots_stride=(-1, 0)),
    dict(row_format=1, row_stride=576)])
def test_attend_refuses(hs, over):
    assert _attend(hs, **over) == hs.HS_ERR_ARG


@pytest.mark.parametrize("strides", [(0, 0, 512), (16 * 512, 0, 0), (504, 0, 512), (16 * 512, 16 * 512, 504)])
def test_attend_refuses_outputs_on_one_another(hs, strides):
    assert _attend(hs, out_stride=strides) == hs.HS_ERR_ARG


def test_attend_limits(hs):
    assert _attend(hs, batch=hs.HS_MAX_BATCH + 1) == hs.HS_ERR_LIMIT
    assert _attend(hs, heads=hs.HS_MAX_HEADS + 1) == hs.HS_ERR_LIMIT
    assert _attend(hs, positions=hs.HS_MAX_POSITIONS + 1) == hs.HS_ERR_LIMIT
    assert _attend(hs, n_rows=1 << 31) == hs.HS_ERR_LIMIT
    assert hs.lib.hs_latent_attend(None, None) == hs.HS_ERR_ARG


def _prefill(hs, **over):
    a = hs.hs_prefill_t()
    a.dtype, a.row_format, a.batch, a.heads, a.q_tokens, a.k_tokens = 0, 0, 2, 16, 100, 120
    a.q, a.rows, a.w_uk, a.w_uv, a.q_start, a.k_start, a.out = (1 << n for n in range(20, 27))
    a.row_stride, a.scale = 1152, 0.1
    a.q_stride, a.out_stride = (16 * 192, 192), (16 * 128, 128)
    a.workspace, a.workspace_bytes = 1 << 27, 1 << 40
    for k, v in over.items():
        setattr(a, k, v)
    return hs.lib.hs_latent_prefill(ctypes.byref(a), None)


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(row_format=-1), dict(batch=0), dict(heads=0), dict(q_tokens=-1), dict(k_tokens=-1),
    dict(q=None), dict(rows=None), dict(w_uk=None), dict(w_uv=None), dict(q_start=None),
    dict(k_start=None), dict(out=None), dict(scale=float("nan")), dict(q=(1 << 20) + 2),
    dict(rows=(1 << 21) + 8), dict(w_uk=(1 << 22) + 8), dict(w_uv=(1 << 23) + 4),
    dict(q_start=(1 << 24) + 1), dict(k_start=(1 << 25) + 2), dict(out=(1 << 26) + 8),
    dict(q_stride=(16 * 192, 191)), dict(out_stride=(-8, 128)), dict(row_stride=1024),
    dict(workspace=None), dict(workspace=(1 << 27) + 8), dict(workspace_bytes=100)])
def test_prefill_refuses(hs, over):
    assert _prefill(hs, **over) == hs.HS_ERR_ARG


@pytest.mark.parametrize("strides", [(0, 128), (16 * 128, 0), (120, 128), (16 * 128, 120)])
def test_prefill_refuses_outputs_on_one_another(hs, strides):
    assert _prefill(hs, out_stride=strides) == hs.HS_ERR_ARG


def test_prefill_limits_and_nothing_to_do(hs):
    assert _prefill(hs, heads=hs.HS_MAX_HEADS + 1) == hs.HS_ERR_LIMIT
    assert _prefill(hs, q_tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _prefill(hs, k_tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _prefill(hs, q_tokens=0, q=None, out=None) == hs.HS_OK
    assert hs.lib.hs_latent_prefill(None, None) == hs.HS_ERR_ARG


def _norm(hs, **over):
    a = hs.hs_norm_t()
    a.dtype, a.dim, a.carry, a.group, a.tokens = 0, 512, 64, 0, 4
    a.x, a.weight, a.out, a.scales = (1 << n for n in range(20, 24))
    a.x_stride, a.out_stride, a.scales_stride, a.eps = 576, 576, 1, 1e-6
    for k, v in over.items():
        setattr(a, k, v)
    return hs.lib.hs_rms_norm(ctypes.byref(a), None)


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(dim=0), dict(carry=-1), dict(group=-1), dict(tokens=-1), dict(x=None),
    dict(weight=None), dict(out=None), dict(residual=1 << 24), dict(residual_out=1 << 24),
    dict(scales=None, group=128), dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")),
    dict(x=(1 << 20) + 1), dict(weight=(1 << 21) + 1), dict(scales=(1 << 23) + 2),
    dict(scales=None, out=(1 << 22) + 1), dict(dtype=2, x=(1 << 20) + 2), dict(x_stride=-1),
    dict(out_stride=575), dict(group=64, scales_stride=8)])
def test_norm_refuses(hs, over):
    assert _norm(hs, **over) == hs.HS_ERR_ARG


def test_norm_limits_and_nothing_to_do(hs):
    assert _norm(hs, dim=hs.HS_MAX_NORM_DIM + 1) == hs.HS_ERR_LIMIT
    assert _norm(hs, carry=hs.HS_MAX_NORM_DIM) == hs.HS_ERR_LIMIT
    assert _norm(hs, tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _norm(hs, tokens=0, x=None, out=None) == hs.HS_OK
    assert hs.lib.hs_rms_norm(None, None) == hs.HS_ERR_ARG


def test_workspace_sizes(hs):
    assert hs.hs_latent_attend_workspace(1, 1, 1, 0) > 0
    assert hs.hs_latent_prefill_workspace(0, 1) > 0
    for call, args in ((hs.hs_latent_attend_workspace, (0, 1, 1, 1)),
                       (hs.hs_latent_attend_workspace, (1, 1, 1, -1)),
                       (hs.hs_latent_attend_workspace, (1, 1, 1, 1 << 31)),
                       (hs.hs_latent_prefill_workspace, (-1, 1)),
                       (hs.hs_latent_prefill_workspace, (1, 0))):
        with pytest.raises(hs.HsError):
            call(*args)


def test_binding_checks_tensors(hs):
    """Shapes, types, layouts and devices; CPU tensors never reach the library."""
    bf = torch.bfloat16
    good = dict(q=torch.zeros(2, 1, 4, 576, dtype=bf), rows=torch.zeros(2, 8, 576, dtype=bf),
                out=torch.zeros(2, 1, 4, 512, dtype=bf), scale=0.1,
                slots=torch.zeros(2, 1, 3, dtype=torch.int32))
    bad = [dict(), dict(q=good["q"].float()), dict(q=good["q"][0]), dict(q=good["q"][..., :512]),
           dict(out=good["out"].half()), dict(out=good["out"][:1]), dict(slots=None),
           dict(slots=good["slots"].long()), dict(slots=good["slots"][:1]),
           dict(lengths=torch.zeros(2, dtype=torch.int32)), dict(row_format=7),
           dict(rows=good["rows"].half()), dict(rows=good["rows"][:1]),
           dict(rows=torch.zeros(2, 8, 576, dtype=torch.uint8)), dict(row_format=hs.HS_ROWS_E4M3),
           dict(rows=good["rows"].transpose(1, 2).contiguous().transpose(1, 2)),
           dict(lse=torch.zeros(2, 1, 4)), dict(lse=torch.zeros(2, 1, 4, dtype=bf)),
           dict(workspace=torch.zeros(64, 2)[:, 0])]
    for over in bad:  # the first: everything fits but the device
        with pytest.raises(ValueError):
            hs.hs_latent_attend(**dict(good, **over))
    start = torch.zeros(3, dtype=torch.int32)
    good = dict(q=torch.zeros(5, 4, 192, dtype=bf), rows=torch.zeros(8, 576, dtype=bf),
                w_uk=torch.zeros(4, 128, 512, dtype=bf), w_uv=torch.zeros(4, 128, 512, dtype=bf),
                q_start=start, k_start=start, out=torch.zeros(5, 4, 128, dtype=bf), scale=0.1)
    for over in [dict(), dict(q=good["q"][0]), dict(w_uk=good["w_uk"][:2]), dict(w_uv=good["w_uv"].half()),
                 dict(k_start=start[:2]), dict(q_start=start.long()), dict(out=good["out"][:, :2]),
                 dict(rows=good["rows"][None]), dict(lse=torch.zeros(5))]:
        with pytest.raises(ValueError):
            hs.hs_latent_prefill(**dict(good, **over))
    good = dict(x=torch.zeros(3, 64), weight=torch.zeros(64), out=torch.zeros(3, 64), eps=1e-6)
    for over in [dict(), dict(x=good["x"][0]), dict(x=good["x"].double()), dict(weight=torch.zeros(63)),
                 dict(carry=64), dict(carry=-1), dict(out=good["out"].half()), dict(group=8),
                 dict(residual=good["x"]), dict(scales=torch.zeros(3, 1)),
                 dict(out=good["out"].to(torch.uint8), scales=torch.zeros(3, 2)),
                 dict(out=good["out"].to(torch.uint8), scales=torch.zeros(3, 1), group=-1)]:
        with pytest.raises(ValueError):
            hs.hs_rms_norm(**dict(good, **over))


@pytest.mark.parametrize("dtype", [torch.uint8, torch.int32, torch.float32])
def test_workspace_error_word(hs, dtype):
    space = torch.full((3, 64), 5, dtype=torch.uint8).view(dtype)
    assert hs.hs_workspace_error(space) == 0x05050505
    hs.hs_workspace_clear(space)
    assert hs.hs_workspace_error(space) == 0
    assert (space.view(-1).view(torch.uint8)[4:] == 5).all()
