"""The gradient norm's C ABI on the CPU: argument errors come back before anything is enqueued."""
import ctypes

import pytest

pgq = pytest.importorskip("int6_weight_export_amd.pgq")

FAKE = 0x10000      # aligned, never dereferenced: every call here fails its checks
INF, NAN = float("inf"), float("nan")


def arrays(ptrs, numel, dtype):
    n = len(numel)
    return (ctypes.c_void_p * n)(*ptrs), (ctypes.c_int64 * n)(*numel), (ctypes.c_int32 * n)(*dtype), n


def norm(ptrs=(FAKE, FAKE + 0x1000), numel=(10, 20), dtype=(pgq.PGQ_F32, pgq.PGQ_BF16), n=None, grad_scale=1.0, scale_dev=None,
         max_norm=1.0, result=FAKE, ws=FAKE, ws_bytes=1 << 20):
    p, m, d, k = arrays(ptrs, numel, dtype)
    return pgq.pgq_grad_norm(p, m, d, k if n is None else n, grad_scale, scale_dev, max_norm, result, ws, ws_bytes, None, None)


def clip(ptrs=(FAKE, FAKE + 0x1000), numel=(10, 20), dtype=(pgq.PGQ_F32, pgq.PGQ_BF16), max_norm=1.0, result=FAKE, ws=FAKE,
         ws_bytes=1 << 20):
    p, m, d, k = arrays(ptrs, numel, dtype)
    return pgq.pgq_grad_clip(p, m, d, k, max_norm, result, ws, ws_bytes, None, None)


@pytest.mark.parametrize("args,want", [
    (dict(n=-1), pgq.PGQ_ERR_SHAPE), (dict(numel=(10, -1)), pgq.PGQ_ERR_SHAPE), (dict(numel=(10, (1 << 40) + 1)), pgq.PGQ_ERR_SHAPE),
    (dict(dtype=(pgq.PGQ_F32, 3)), pgq.PGQ_ERR_DTYPE), (dict(ptrs=(FAKE, 0)), pgq.PGQ_ERR_NULL), (dict(result=None), pgq.PGQ_ERR_NULL),
    (dict(ptrs=(FAKE + 2, FAKE)), pgq.PGQ_ERR_ALIGN), (dict(ptrs=(FAKE, FAKE + 1)), pgq.PGQ_ERR_ALIGN),
    (dict(result=FAKE + 2), pgq.PGQ_ERR_ALIGN), (dict(ws=FAKE + 32), pgq.PGQ_ERR_ALIGN), (dict(ws=None), pgq.PGQ_ERR_WORKSPACE),
    (dict(ws_bytes=127), pgq.PGQ_ERR_WORKSPACE), (dict(max_norm=-1.0), pgq.PGQ_ERR_PARAM), (dict(max_norm=NAN), pgq.PGQ_ERR_PARAM),
])
def test_argument_errors(args, want):
    assert norm(**args) == want
    if "n" not in args:
        assert clip(**args) == want


@pytest.mark.parametrize("args,want", [
    (dict(grad_scale=INF), pgq.PGQ_ERR_PARAM), (dict(grad_scale=NAN), pgq.PGQ_ERR_PARAM), (dict(scale_dev=FAKE + 2), pgq.PGQ_ERR_ALIGN),
])
def test_scale_errors(args, want):
    assert norm(**args) == want


def test_null_arrays():
    p, m, d, n = arrays((FAKE,), (4,), (pgq.PGQ_F32,))
    for a in ((None, m, d), (p, None, d), (p, m, None)):
        assert pgq.pgq_grad_norm(*a, n, 1.0, None, 1.0, FAKE, FAKE, 1 << 20, None, None) == pgq.PGQ_ERR_NULL
        assert pgq.pgq_grad_clip(*a, n, 1.0, FAKE, FAKE, 1 << 20, None, None) == pgq.PGQ_ERR_NULL
    need = ctypes.c_size_t(0)
    assert pgq.pgq_grad_norm_workspace(None, 1, ctypes.byref(need)) == pgq.PGQ_ERR_NULL
    assert pgq.pgq_grad_norm_workspace(m, 1, None) == pgq.PGQ_ERR_NULL


@pytest.mark.parametrize("ptrs,numel,dtype", [
    ((FAKE, FAKE), (10, 10), (pgq.PGQ_F32, pgq.PGQ_F32)), ((FAKE + 36, FAKE), (4, 10), (pgq.PGQ_F32, pgq.PGQ_F32)),
    ((FAKE, FAKE + 18), (10, 10), (pgq.PGQ_BF16, pgq.PGQ_BF16)),
])
def test_clipping_shared_memory_is_refused(ptrs, numel, dtype):
    assert clip(ptrs=ptrs, numel=numel, dtype=dtype) == pgq.PGQ_ERR_PARAM


def test_shared_memory_among_many():
    n = 400
    ptrs = [FAKE + 64 * i for i in range(n)]
    ptrs[333] = ptrs[2] + 4
    assert clip(ptrs=ptrs, numel=[8] * n, dtype=[pgq.PGQ_F32] * n) == pgq.PGQ_ERR_PARAM


@pytest.mark.parametrize("numel", [[], [0], [1], [16384], [16385], [5, 0, 7], [1 << 22] * 3, [1 << 35], [3] * 5000])
def test_workspace_grows_with_the_tiles_only_so_far(numel):
    a, need = (ctypes.c_int64 * len(numel))(*numel), ctypes.c_size_t(0)
    assert pgq.pgq_grad_norm_workspace(a, len(numel), ctypes.byref(need)) == pgq.PGQ_OK
    filled = sum(n > 0 for n in numel)
    assert need.value % 64 == 0 and 64 <= need.value <= 8192 + 8 * (2048 + filled)


def test_clipped_step_checks_its_factor():
    t = (pgq.pgq_adamw_tensor * 1)(pgq.pgq_adamw_tensor(FAKE, 0, FAKE, FAKE, 0, 0, 4, pgq.PGQ_F32, pgq.PGQ_F32, 1.0, 0.0))
    g, h = (ctypes.c_void_p * 1)(FAKE), pgq.pgq_adamw_hyper()
    assert pgq.pgq_adamw_hyper_at(1e-3, 0.9, 0.999, 1e-8, 1, 1.0, 0, ctypes.byref(h)) == pgq.PGQ_OK
    assert pgq.pgq_adamw_step_clipped(t, 1, 32, g, h, None, FAKE + 2, FAKE, 1 << 20, 0, None, None) == pgq.PGQ_ERR_ALIGN
    assert pgq.pgq_adamw_step_clipped(t, 1, 32, g, None, None, FAKE, FAKE, 1 << 20, 0, None, None) == pgq.PGQ_ERR_NULL


@pytest.mark.parametrize("numel", [[], [0], [1], [16384] * 1024, [16385] * 1023, [(1 << 22) + 13] * 3, [1 << 40], [1 << 40, 0, 5], [3] * 5000])
def test_workspace_is_the_counters_and_a_sum_a_tile(numel):
    """Seventeen counters of 256 bytes and eight bytes for every tile, of which there are at most 1024 and one more a tensor."""
    a, need = (ctypes.c_int64 * len(numel))(*numel), ctypes.c_size_t(0)
    assert pgq.pgq_grad_norm_workspace(a, len(numel), ctypes.byref(need)) == pgq.PGQ_OK
    filled = sum(n > 0 for n in numel)
    least = max(1, filled, min(1024, sum(numel) // 16384) // 2)
    assert 17 * 256 + 8 * least <= need.value <= 17 * 256 + 8 * (1024 + filled) + 56


def test_workspace_of_small_lists_is_counted_in_tiles_of_16384():
    for numel, tiles in (([1], 1), ([16384], 1), ([16385], 2), ([16384 * 3 + 1, 0, 7], 5), ([16384 * 1024], 1024)):
        a, need = (ctypes.c_int64 * len(numel))(*numel), ctypes.c_size_t(0)
        assert pgq.pgq_grad_norm_workspace(a, len(numel), ctypes.byref(need)) == pgq.PGQ_OK
        assert need.value == 17 * 256 + -(-8 * tiles // 64) * 64
