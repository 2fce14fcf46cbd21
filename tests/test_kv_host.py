"""Order, errors and handles of the key/value cache's C entry points, on the host."""
import pytest

import kv_host


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    return kv_host.build(tmp_path_factory.mktemp("kv_host"))


@pytest.fixture
def cache(lib):
    for i in range(16):
        lib.fake_identity(i, 100 + i)
        lib.fake_capturing(i, 0)
    c = kv_host.Cache(lib)
    yield c
    lib.moe_kv_destroy(c.h)


def waits(log):
    return [x for x in log if x.startswith("wait")]


def test_another_stream_waits_and_the_same_one_does_not(cache):
    for s in (4, 4):
        assert cache.attention(s) == 0
    assert not waits(cache.log())
    assert cache.attention(5) == 0
    log = cache.log()
    assert log.index("wait 5") < log.index("attention 5")
    assert cache.select(4, pages=600) == 0  # scores in the workspace
    assert waits(cache.log()) == ["wait 4"]
    assert cache.select(5, pages=4) == 0  # none
    assert not waits(cache.log())


def test_default_stream_is_recorded_when_another_follows(cache):
    assert cache.attention(0) == 0 and cache.attention(0) == 0
    assert cache.log() == ["attention 0", "attention 0"]
    assert cache.attention(4) == 0
    assert cache.log()[:3] == ["record 0", "wait 4", "attention 4"]


def test_a_handle_value_that_names_a_new_stream_waits(cache, lib):
    """A stream that was destroyed (its work goes on) and whose handle value another one got; the
    per-thread default stream (handle 2), one stream in each thread."""
    for handle in (4, 2):
        lib.fake_identity(handle, 1000 + handle)
        assert cache.attention(handle) == 0
        cache.log()
        lib.fake_identity(handle, 2000 + handle)
        assert cache.attention(handle) == 0
        assert waits(cache.log()) == [f"wait {handle}"]


def test_a_capture_neither_waits_nor_records(cache, lib):
    assert cache.attention(4) == 0
    lib.fake_capturing(5, 1)
    cache.log()
    assert cache.attention(5) == 0
    assert cache.log() == ["attention 5"]


@pytest.mark.parametrize("call", ["append", "read", "attention", "select", "status"])
def test_a_wait_that_gave_up_is_reported_once_by_whichever_call_is_next(cache, lib, call):
    def run():
        return lib.moe_kv_status(cache.h) if call == "status" else getattr(cache, call)(4)

    assert run() == 0
    cache.log()
    lib.fake_raise(cache.h)
    assert run() == 4 and b"gave up" in lib.moe_kv_last_error(cache.h)
    assert cache.log() == []
    assert run() == 0
    assert lib.moe_kv_status(cache.h) == 0


def test_a_wait_that_gave_up_is_reported_to_a_capture_and_by_destroy(lib):
    c = kv_host.Cache(lib)
    assert c.attention(4) == 0
    lib.fake_capturing(5, 1)
    lib.fake_raise(c.h)
    c.log()
    assert c.attention(5) == 4 and c.log() == []
    lib.fake_capturing(5, 0)
    lib.fake_raise(c.h)
    assert lib.moe_kv_destroy(c.h) == 4 and b"gone" in lib.moe_kv_last_error(None)
    assert "free" in c.log()


class Error(RuntimeError):
    def __init__(self, status, text):
        super().__init__(text)
        self.status = status


def test_close_while_another_thread_is_in_a_call(lib, tmp_path_factory):
    """The cache stays open and usable, nothing is freed, and a later close frees it."""
    import threading

    c = kv_host.Cache(lib)
    m = kv_host.build_binding(kv_host.folder_of(lib))
    cache = m.Cache(Error, c.h.value, 0, True, 1, 64)
    cache.check()
    lib.fake_block(1)
    t = threading.Thread(target=cache.check)
    t.start()
    lib.fake_block(2)
    with pytest.raises(Error) as e:
        cache.close()
    assert e.value.status == 5
    with pytest.raises(Error) as e:  # one call at a time
        cache.check()
    assert e.value.status == 5
    assert "free" not in c.log()
    lib.fake_block(0)
    t.join()
    cache.check()
    cache.close()
    assert "free" in c.log()
    cache.close()
    with pytest.raises(Error, match="closed"):
        cache.check()


def test_budgets_that_rounds_cannot_number_are_refused(cache):
    """A chosen page is page_size / 16 blocks, which are counted in 32 bits."""
    import ctypes

    def attention(budget):
        return cache.L.moe_kv_attention(cache.h, 0, ctypes.byref(cache.batch()), ctypes.byref(cache.t), 1, ctypes.c_float(1.0), 1,
                                        ctypes.byref(cache.o), None, kv_host.P(4096), budget, kv_host.P(4))

    assert attention(1 << 20) == 0
    cache.log()
    for budget in (0x7fffffff, 0x7ffffff9):
        assert attention(budget) == 6 and b"budget" in cache.L.moe_kv_last_error(cache.h)
    assert cache.log() == []
