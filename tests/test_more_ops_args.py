"""Rows written and read back, heads' norm and rotation, and attention over a shared
prefix without a GPU: what the library and the binding refuse, before any CUDA call."""
import ctypes
import shutil
import subprocess

import pytest

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def hs():
    from hierarchical_kv_cache_hs_gb300 import build
    build.build_libhs()
    from hierarchical_kv_cache_hs_gb300 import hs as mod
    return mod


def _call(fn, a, over):
    for k, v in over.items():
        setattr(a, k, type(getattr(a, k))(*v) if isinstance(v, tuple) else v)
    return fn(ctypes.byref(a), None)


def _write(hs, **over):
    a = hs.hs_write_t()
    a.dtype, a.row_format, a.rotation, a.batch, a.tokens, a.x_stride, a.eps = 0, 0, 1, 3, 10, 576, 1e-6
    a.x, a.weight, a.positions, a.inv_freq, a.start, a.lengths, a.rows = (1 << n for n in range(20, 27))
    a.n_rows, a.row_stride, a.request_stride = 100, 1152, 115200
    return _call(hs.lib.hs_latent_write, a, over)


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(dtype=-1), dict(row_format=2), dict(rotation=3), dict(rotation=-1), dict(batch=0), dict(tokens=-1),
    dict(x=None), dict(x=(1 << 20) + 8), dict(x_stride=580), dict(x_stride=-8), dict(weight=(1 << 21) + 2),
    dict(eps=-1.0), dict(eps=float("nan")), dict(eps=float("inf")), dict(positions=None), dict(inv_freq=None),
    dict(positions=(1 << 22) + 2), dict(inv_freq=(1 << 23) + 1), dict(lengths=None), dict(start=(1 << 24) + 2),
    dict(lengths=(1 << 25) + 2), dict(rows=None), dict(rows=(1 << 26) + 8), dict(n_rows=-1), dict(row_stride=1136),
    dict(row_stride=1160), dict(request_stride=115192), dict(request_stride=115184), dict(request_stride=-115200),
    dict(request_stride=0), dict(start=None, n_rows=9), dict(row_format=1, row_stride=576),
    dict(row_stride=1 << 62, request_stride=1 << 62), dict(n_rows=1, request_stride=1136)])
def test_write_refuses(hs, over):
    assert _write(hs, **over) == hs.HS_ERR_ARG


def test_write_limits_and_nothing_to_do(hs):
    assert _write(hs, tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _write(hs, batch=hs.HS_MAX_BATCH + 1) == hs.HS_ERR_LIMIT
    assert _write(hs, n_rows=1 << 31, row_stride=1152, request_stride=1152 << 31) == hs.HS_ERR_LIMIT
    assert _write(hs, tokens=0, x=None, rows=None) == hs.HS_OK
    assert hs.lib.hs_latent_write(None, None) == hs.HS_ERR_ARG


def _read(hs, **over):
    a = hs.hs_read_t()
    a.dtype, a.row_format, a.out_dtype, a.batch, a.entries, a.tokens = 0, 0, 0, 3, 4, 12
    a.rows, a.slots, a.out = (1 << n for n in range(20, 23))
    a.n_rows, a.row_stride, a.request_stride, a.slots_stride, a.out_stride = 100, 1152, 115200, 4, 576
    return _call(hs.lib.hs_latent_read, a, over)


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(row_format=-1), dict(out_dtype=3), dict(batch=0), dict(entries=-1), dict(tokens=11), dict(tokens=-1),
    dict(rows=None), dict(rows=(1 << 20) + 8), dict(slots=None), dict(slots=(1 << 21) + 1), dict(start=1 << 23),
    dict(out=None), dict(out=(1 << 22) + 8), dict(out_stride=572), dict(out_stride=580), dict(out_stride=-576),
    dict(out_dtype=2, out_stride=578), dict(n_rows=-1), dict(row_stride=1136), dict(row_stride=1160),
    dict(request_stride=8), dict(request_stride=-16), dict(slots_stride=-1), dict(slots=None, start=(1 << 23) + 2),
    dict(slots=None, start=1 << 23, lengths=(1 << 24) + 2)])
def test_read_refuses(hs, over):
    assert _read(hs, **over) == hs.HS_ERR_ARG


def test_read_limits_and_nothing_to_do(hs):
    assert _read(hs, slots=None, start=1 << 23, tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _read(hs, batch=hs.HS_MAX_BATCH + 1, entries=1, tokens=hs.HS_MAX_BATCH + 1) == hs.HS_ERR_LIMIT
    assert _read(hs, n_rows=1 << 31) == hs.HS_ERR_LIMIT
    assert _read(hs, entries=0, tokens=0, out=None, rows=None) == hs.HS_OK
    assert hs.lib.hs_latent_read(None, None) == hs.HS_ERR_ARG


def _rotate(hs, **over):
    a = hs.hs_rotate_t()
    a.dtype, a.rotation, a.dim, a.rope_at, a.rope, a.tokens, a.eps = 0, 1, 192, 128, 64, 5, 1e-6
    a.heads, a.x, a.out = (16, 2), (1 << 20, 1 << 21), (1 << 22, 1 << 23)
    a.weight, a.positions, a.inv_freq = (1 << 24, 1 << 25), 1 << 26, 1 << 27
    a.x_stride = a.out_stride = (16 * 192, 192, 2 * 192, 192)
    return _call(hs.lib.hs_norm_rotate, a, over)


@pytest.mark.parametrize("over", [
    dict(dtype=3), dict(rotation=3), dict(dim=0), dict(tokens=-1), dict(heads=(0, 2)), dict(heads=(16, 0)), dict(heads=(-1, 2)),
    dict(x=(1 << 20, 0)), dict(x=(0, 1 << 21)), dict(out=(0, 1 << 23)), dict(out=(1 << 22, 0)), dict(x=((1 << 20) + 1, 1 << 21)),
    dict(out=(1 << 22, (1 << 23) + 1)), dict(weight=(1 << 24, (1 << 25) + 1)), dict(dtype=2, x=((1 << 20) + 2, 1 << 21)),
    dict(rope=63), dict(rope=0), dict(rope=-2), dict(rope_at=130), dict(rope_at=-2), dict(rope=194, rope_at=0),
    dict(rotation=0), dict(positions=None), dict(inv_freq=None), dict(positions=(1 << 26) + 2), dict(inv_freq=(1 << 27) + 2),
    dict(eps=-1.0), dict(eps=float("nan")), dict(x_stride=(-1, 192, 384, 192)), dict(x_stride=(16 * 192, -1, 384, 192)),
    dict(out_stride=(16 * 192, 191, 384, 192)), dict(out_stride=(0, 192, 384, 192)), dict(out_stride=(15 * 192, 192, 384, 192)),
    dict(out_stride=(16 * 192, 192, 384, 0)), dict(out_stride=(192, 4 * 192, 384, 192))])
def test_rotate_refuses(hs, over):
    assert _rotate(hs, **over) == hs.HS_ERR_ARG


def test_rotate_limits_and_nothing_to_do(hs):
    assert _rotate(hs, dim=hs.HS_MAX_HEAD_CHANNELS + 1) == hs.HS_ERR_LIMIT
    assert _rotate(hs, heads=(hs.HS_MAX_HEADS + 1, 2)) == hs.HS_ERR_LIMIT
    assert _rotate(hs, heads=(1, hs.HS_MAX_HEADS + 1)) == hs.HS_ERR_LIMIT
    assert _rotate(hs, tokens=hs.HS_MAX_TOKENS + 1) == hs.HS_ERR_LIMIT
    assert _rotate(hs, tokens=0) == hs.HS_OK
    assert hs.lib.hs_norm_rotate(None, None) == hs.HS_ERR_ARG


def _shared(hs, prefix={}, **over):
    a, p = hs.hs_attend_t(), hs.hs_prefix_t()
    a.dtype, a.row_format, a.batch, a.positions, a.heads, a.entries = 0, 0, 2, 1, 16, 64
    a.n_rows, a.q, a.rows, a.out, a.slots = 128, 1 << 20, 1 << 21, 1 << 22, 1 << 23
    a.row_stride, a.request_stride, a.scale = 1152, 128 * 1152, 0.1
    a.q_stride, a.out_stride = (16 * 576, 16 * 576, 576), (16 * 512, 16 * 512, 512)
    a.slots_stride = (64, 64)
    a.workspace, a.workspace_bytes = 1 << 24, 1 << 40
    p.rows, p.n_rows, p.row_stride = 1 << 25, 1000, 1152
    for k, v in over.items():
        setattr(a, k, v)
    for k, v in prefix.items():
        setattr(p, k, v)
    return hs.lib.hs_latent_attend_shared(ctypes.byref(a), ctypes.byref(p), None)


@pytest.mark.parametrize("prefix", [
    dict(rows=None), dict(rows=(1 << 25) + 8), dict(n_rows=-1), dict(row_stride=1136), dict(row_stride=1160),
    dict(row_stride=-1152), dict(lengths=(1 << 26) + 2)])
def test_shared_refuses_prefixes(hs, prefix):
    assert _shared(hs, prefix) == hs.HS_ERR_ARG


@pytest.mark.parametrize("over", [
    dict(dtype=2), dict(row_format=2), dict(batch=0), dict(heads=0), dict(q=None), dict(out=None), dict(rows=None),
    dict(slots=None), dict(lengths=1 << 27), dict(scale=float("nan")), dict(out=(1 << 22) + 2), dict(lse=(1 << 26) + 2),
    dict(workspace=(1 << 24) + 8), dict(workspace=None), dict(workspace_bytes=1 << 20), dict(out_stride=(0, 0, 512)),
    dict(row_format=1, row_stride=576)])
def test_shared_refuses(hs, over):
    assert _shared(hs, **over) == hs.HS_ERR_ARG


def test_shared_limits(hs):
    assert _shared(hs, dict(n_rows=1 << 31)) == hs.HS_ERR_LIMIT
    assert _shared(hs, dict(row_stride=1 << 40)) == hs.HS_ERR_LIMIT
    assert _shared(hs, heads=hs.HS_MAX_HEADS + 1) == hs.HS_ERR_LIMIT
    assert _shared(hs, batch=4096, positions=1024, heads=1024) == hs.HS_ERR_LIMIT
    assert hs.lib.hs_latent_attend_shared(None, None, None) == hs.HS_ERR_ARG


def test_shared_workspace_sizes(hs):
    size = hs.hs_latent_attend_shared_workspace
    assert size(1, 1, 1, 0, 0) >= hs.hs_latent_attend_workspace(1, 1, 1, 0)
    assert size(4, 1, 16, 100, 5000) >= size(4, 1, 16, 100, 0) + 5000 * 1152
    for args in ((0, 1, 1, 1, 1), (1, 1, 1, -1, 1), (1, 1, 1, 1, -1), (1, 1, 1, 1, 1 << 31), (4096, 1024, 1024, 1, 1),
                 (1, 1, 1, 1, 1, 7)):
        with pytest.raises(hs.HsError):
            size(*args)


def _refused(call, good, bad):
    for over in [dict()] + bad:  # the first: everything fits but the device
        with pytest.raises(ValueError):
            call(**dict(good, **over))


def test_binding_checks_tensors(hs):
    """Shapes, types, layouts and devices; CPU tensors never reach the library."""
    bf, i32 = torch.bfloat16, torch.int32
    x, freq = torch.zeros(5, 576, dtype=bf), torch.zeros(32)
    start, lengths = torch.zeros(3, dtype=i32), torch.zeros(2, dtype=i32)
    good = dict(x=x, rows=torch.zeros(2, 9, 576, dtype=bf), weight=torch.zeros(512, dtype=bf), eps=1e-6,
                positions=torch.zeros(5, dtype=i32), inv_freq=freq, start=start, lengths=lengths)
    _refused(hs.hs_latent_write, good, [
        dict(x=x.float()), dict(x=x[0]), dict(x=x[:, :512]), dict(weight=good["weight"].float()), dict(weight=good["weight"][:64]),
        dict(positions=None), dict(inv_freq=None), dict(inv_freq=freq[:31]), dict(inv_freq=freq.double()), dict(rotation=0),
        dict(rotation=5), dict(positions=good["positions"][:4]), dict(positions=good["positions"].long()), dict(start=None),
        dict(lengths=None), dict(lengths=lengths[:1]), dict(start=start.long()), dict(rows=good["rows"][0]),
        dict(rows=good["rows"].half()), dict(row_format=hs.HS_ROWS_E4M3), dict(row_format=9),
        dict(rows=torch.zeros(2, 9, 576, dtype=torch.uint8))])
    good = dict(rows=torch.zeros(2, 9, 576, dtype=bf), out=torch.zeros(2, 4, 576, dtype=bf), slots=torch.zeros(2, 4, dtype=i32))
    _refused(hs.hs_latent_read, good, [
        dict(slots=None), dict(start=start), dict(lengths=lengths), dict(slots=good["slots"].long()), dict(slots=good["slots"][0]),
        dict(out=good["out"][:, :3]), dict(out=good["out"].double()), dict(out=torch.zeros(2, 8, 576, dtype=bf)[:, :4]),
        dict(rows=good["rows"][:1]), dict(dtype=torch.float32), dict(rows=torch.zeros(2, 9, 1152, dtype=torch.uint8), out=torch.zeros(2, 4, 576)),
        dict(slots=None, start=start), dict(slots=None, start=start, out=torch.zeros(8, 500, dtype=bf))])
    q = torch.zeros(5, 4, 192, dtype=bf)
    k = torch.zeros(5, 1, 192, dtype=bf)
    good = dict(q=q, q_out=q.clone(), k=k, k_out=k.clone(), q_weight=torch.zeros(192, dtype=bf), k_weight=torch.zeros(192, dtype=bf),
                eps=1e-6, positions=torch.zeros(5, dtype=i32), inv_freq=freq)
    _refused(hs.hs_norm_rotate, good, [
        dict(q=q[0]), dict(q=q.double()), dict(q_out=q[:, :3]), dict(q_out=q.half()), dict(k=None), dict(k_out=None),
        dict(k=None, k_out=None), dict(k=k[0]), dict(k=k[:4]), dict(q_weight=torch.zeros(64, dtype=bf)),
        dict(k_weight=torch.zeros(192)), dict(positions=None), dict(inv_freq=None), dict(inv_freq=torch.zeros(97)),
        dict(rope_at=129), dict(rope_at=-1), dict(rotation=0), dict(q=q.transpose(1, 2).contiguous().transpose(1, 2))])
    good = dict(q=torch.zeros(2, 1, 4, 576, dtype=bf), prefix=torch.zeros(7, 576, dtype=bf), rows=torch.zeros(2, 8, 576, dtype=bf),
                out=torch.zeros(2, 1, 4, 512, dtype=bf), scale=0.1, lengths=lengths, prefix_lengths=lengths)
    _refused(hs.hs_latent_attend_shared, good, [
        dict(prefix=good["prefix"].half()), dict(prefix=good["prefix"][None]), dict(prefix=good["prefix"][:, :512]),
        dict(row_format=hs.HS_ROWS_E4M3), dict(prefix_lengths=lengths.long()), dict(prefix_lengths=lengths[:1]),
        dict(lengths=None), dict(q=good["q"][0]), dict(lse=torch.zeros(2, 1, 4))])


def test_rotate_no_tokens_with_keys(hs):
    """Arrays of no tokens have no address; the heads are given all the same."""
    nowhere = dict(tokens=0, x=(0, 0), out=(0, 0), weight=(0, 0), positions=None, inv_freq=None)
    assert _rotate(hs, **nowhere) == hs.HS_OK
    assert _rotate(hs, heads=(16, 0), **nowhere) == hs.HS_OK
    assert _rotate(hs, heads=(16, -1), **nowhere) == hs.HS_ERR_ARG


@pytest.mark.parametrize("positions,heads", [(1, 128), (1, 16), (3, 20), (2, 200)])
@pytest.mark.parametrize("rows,prefix", [(0, 16384), (512, 16384), (5, 1), (2048, 3001)])
def test_shared_workspace_of_more_requests_is_no_smaller(hs, positions, heads, rows, prefix):
    """A workspace for the largest batch serves every smaller one; 152 and 304 units of 128 queries among them."""
    sizes = [hs.hs_latent_attend_shared_workspace(b, positions, heads, rows, prefix) for b in range(1, 2600)]
    assert sizes == sorted(sizes)


def test_shared_workspace_grows_with_each_size(hs):
    size = hs.hs_latent_attend_shared_workspace
    for axis, values in enumerate(([1, 7, 152, 153, 256, 4096], [1, 2, 3, 64], [1, 16, 32, 33, 48, 128, 129, 512],
                                   [0, 1, 64, 65, 512, 4096], [0, 1, 128, 129, 65536])):
        for base in ((1, 1, 16, 0, 1000), (5, 3, 20, 300, 3001), (150, 1, 128, 512, 16384), (20, 1, 32, 2048, 100)):
            got = [size(*base[:axis], v, *base[axis + 1:]) for v in values]
            assert got == sorted(got), (axis, base, got)


@pytest.mark.skipif(shutil.which("nm") is None, reason="needs nm")
def test_no_rotation_kernel_that_nothing_reaches(hs):
    """Heads of 16-bit types have at most 1024 / 8 units, 4 a lane of 32; the form of 8 is fp32's."""
    names = subprocess.run(["nm", "-C", hs.LIB_PATH], capture_output=True, text=True, check=True).stdout
    wide = [line for line in names.splitlines() if "hs_rotate_kernel<" in line and ", 8, 1>" in line]
    assert not [line for line in wide if "hs_rotate_kernel<float" not in line], wide


def test_handles_of_another_device_are_refused(hs, monkeypatch):
    """A handle's buffer and pool belong to the device it was created on; the tensors' may be another."""
    h = object.__new__(hs.Handle)  # of 2 requests, never created
    h.B, h.R, h.S, h.T, h.H, h.h = 2, 1152, 8, 0, 16, None
    here, there = torch.device("cuda", 0), torch.device("cuda", 1)
    monkeypatch.setattr(hs, "hs_device", lambda handle: 1)
    monkeypatch.setattr(hs, "hs_device_buffer", lambda handle: 1 << 20)
    monkeypatch.setattr(hs, "hs_host_pool", lambda handle: 1 << 21)
    for refused in (lambda: hs._rows_of(h, hs.HS_ROWS_16BIT, torch.bfloat16, here, (2,)), lambda: hs._pool_of(h, hs.HS_ROWS_16BIT, here)):
        with pytest.raises(ValueError, match="on device 1"):
            refused()
    assert hs._rows_of(h, hs.HS_ROWS_16BIT, torch.bfloat16, there, (2,)) == (1 << 20, 8, 1152, 8 * 1152)
    assert hs._pool_of(h, hs.HS_ROWS_16BIT, there) == (1 << 21, 16, 1152, 16 * 1152)
    assert hs.lib.hs_device(None) == hs.HS_ERR_ARG
