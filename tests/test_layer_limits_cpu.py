"""CPU tests of the largest sizes of the gated linear recurrence, the norm and the drafts: a launch holds fewer than 2^32
threads, and a call that would need more is refused before anything is enqueued.

Calls just below the limit are told from refused ones by what comes next, the check of a pointer: every call here has a
NULL in it and none can be launched."""
import pytest

import gated_delta_rule_104_amd as kda

OK, ERR_NULL, ERR_SHAPE = range(3)
F32, BF16 = 0, 1
A = 0x100000


@pytest.fixture(scope="module")
def lib():
    return kda.load()


@pytest.mark.parametrize("B,H,T,d,dt,rc", [
    ((1 << 18) - 8, 32, 1, 128, BF16, ERR_NULL), (1 << 18, 32, 1, 128, BF16, ERR_SHAPE),  # 2^24 tiles of 256 threads
    ((1 << 18) - 8, 32, 0, 128, F32, ERR_NULL), (1 << 18, 32, 0, 128, F32, ERR_SHAPE),
    (8, 32, 1 << 20, 128, BF16, ERR_NULL), (1, 1, (1 << 30), 8, BF16, ERR_NULL), (1 << 12, 32, 1 << 14, 128, BF16, ERR_SHAPE),
])
def test_recurrence(lib, B, H, T, d, dt, rc):
    # (a contiguous tensor of a billion tokens: rows of 8 values)
    assert lib.kda_glr_prefill(None, A, A + 64, None, None, A + 128, None, None, B, H, T, d, 1, dt, A, 1 << 50, None) == rc
    if T:
        assert lib.kda_glr_backward(None, A, A + 64, None, A + 128, A + 192, None, None, A + 256, A + 320, A + 384, None, None, None,
                                    B, H, T, d, 1, dt, A, 1 << 50, None) == rc


def test_recurrence_one_token(lib):
    f = lambda N, dt: lib.kda_glr_step(None, A, None, A + 64, A + 128, None, N, 32, 128, 1, dt, None)  # noqa: E731
    assert f((1 << 23) - 1, BF16) == ERR_NULL and f(1 << 23, BF16) == ERR_SHAPE  # 8 values a thread
    assert f((1 << 22) - 1, F32) == ERR_NULL and f(1 << 22, F32) == ERR_SHAPE


def test_norm(lib):
    def f(rows, d, dt, out=0):
        return lib.kda_rms_norm(None, None, None, None, A, A + 64 if out else None, None, None, 1, 1, rows, d, 0, 1e-6, 0, out, dt, None)
    for out in (0, 2):
        assert f((1 << 24) - 1, 4096, BF16, out) == ERR_NULL and f(1 << 24, 4096, BF16, out) == ERR_SHAPE  # 256 threads a row
        assert f((1 << 22) - 1, 32768, F32, out) == ERR_NULL and f(1 << 22, 32768, F32, out) == ERR_SHAPE  # 1024
        assert f((1 << 30) - 64, 64, F32, out) == ERR_NULL and f((1 << 30) - 63, 64, F32, out) == ERR_SHAPE  # 64 rows for 256


def test_norm_gradients(lib):
    def f(H, d, rows=1, per_head=1, dt=BF16):
        return lib.kda_rms_norm_backward(None, None, A, A + 64, None, A + 128, None, A + 192, None, 1, H, rows, d, per_head, 1e-6, 0, dt, A,
                                         1 << 50, None)
    assert f(1 << 23, 8) == ERR_NULL and f(1 << 24, 8) == ERR_SHAPE  # a workgroup a head
    assert f((1 << 23) - 2, 16) == ERR_NULL and f(1 << 23, 16) == ERR_SHAPE  # 32 threads a value of the weight
    assert f(1 << 24, 8, per_head=0) == ERR_NULL and f(1, 4096, rows=(1 << 31) - 65537) == ERR_NULL  # persistent workgroups


def test_drafts(lib):
    def f(N, V):
        return lib.kda_draft_verify(None, None, None, None, A, A + 64, None, A + 128, A + 192, N, 1, V, F32, A, 1 << 50, None)
    assert f((1 << 23) - 1, 100) == ERR_NULL and f(1 << 23, 100) == ERR_SHAPE  # 512 threads choose
    assert f((1 << 19) - 1, 131072) == ERR_NULL and f(1 << 19, 131072) == ERR_SHAPE  # 32 chunks of 256 threads
    c = lambda N: lib.kda_state_commit(None, A, A + 64, N, 2, 1, 2, 2, None)  # noqa: E731
    assert c((1 << 24) - 1) == ERR_NULL and c(1 << 24) == ERR_SHAPE
