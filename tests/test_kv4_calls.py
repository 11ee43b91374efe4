"""How the calls of the 4-bit paged cache behave around their arithmetic, on the GPU."""
import numpy as np
import pytest
import torch

from test_kv4 import DEV, Setup, dev, host, pm, rows  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("clear", [True, False])
def test_the_error_word_waits_for_every_stream(pm, clear):  # noqa: F811
    """A call that is still queued on a side stream is reported by the read that follows it, and not
    once more by the next."""
    s = Setup(pm, [100, 100], [1, 1], 4, 2, 128, 32)
    s.fill()
    q = dev(rows(11, s.n, 4, 128))
    s.table[1, 2] = -5
    bad = s.make_batch(s.kv_len, s.start)
    assert s.cache.read_error() == 0
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)      # 50 ms and more
    s.cache.attend(bad, q, stream=side)
    assert s.cache.read_error(clear=clear) == pm.DEVERR_PAGE
    assert s.cache.read_error() == (0 if clear else pm.DEVERR_PAGE)
    assert s.cache.read_error() == 0


def test_a_cache_cannot_be_changed_from_outside(pm):  # noqa: F811
    """Its heads, pages and memory are what its calls check the tensors against."""
    s = Setup(pm, [40], [2], 8, 2, 128, 16)
    s.fill()
    q = dev(rows(21, 2, 8, 128))
    want, pages = s.cache.attend(s.batch, q), s.cache.pages().clone()
    for name, value in (("n_q_heads", 64), ("n_kv_heads", 8), ("head_dim", 64), ("page_tokens", 128)):
        setattr(s.cache.cfg, name, value)              # of a copy
        assert getattr(s.cache.cfg, name) != value
    for name, value in (("cfg", pm.KV4Config.make(16, 2)), ("buffer", s.cache.buffer[:256]), ("n_pages", 100),
                        ("device", torch.device("cpu"))):
        with pytest.raises(AttributeError):
            setattr(s.cache, name, value)
    s.cache.layer = 3                                  # a name of the caller's own
    assert torch.equal(s.cache.attend(s.batch, q), want) and torch.equal(s.cache.pages(), pages)


@pytest.mark.parametrize("T", [1, 4, 20, 70])
def test_lengths_that_change_under_a_call(pm, T):  # noqa: F811
    """The caller's mistake, a host that copies the next step's lengths while a call runs: what that
    call gives is not defined, but it ends, and the next one is right."""
    B = 24
    lens = [2000 + 40 * i for i in range(B)]
    s = Setup(pm, lens, [T] * B, 4, 2, 64, 32)
    s.fill()
    q = dev(rows(31, s.n, 4, 64))
    want = s.cache.attend(s.batch, q)
    first = s.batch.kv_len.clone()
    hosts = [torch.tensor(x, dtype=torch.int32).pin_memory() for x in ([0] * B, lens, [1] * B, lens[::-1])]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        for i in range(12):
            with torch.cuda.stream(side):
                s.batch.kv_len.copy_(hosts[i % 4], non_blocking=True)
            if i % 3 == 0:
                s.cache.attend(s.batch, q)
    torch.cuda.synchronize()
    s.batch.kv_len.copy_(first)
    assert not s.cache.read_error() & ~pm.DEVERR_BATCH
    assert torch.equal(s.cache.attend(s.batch, q), want) and s.cache.read_error() == 0
