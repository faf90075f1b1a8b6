"""CPU-only: cache descriptors and the device they were checked on."""
import threading

import pytest
import torch


@pytest.fixture(scope="module")
def kvc():
    from kv_cache_compression_split_gb300 import build
    build.build()
    import kv_cache_compression_split_gb300 as k
    k.lib()
    return k


class DeviceTensor:
    """What the binding asks of a CUDA tensor, without a GPU."""

    def __init__(self, address, shape, device=0):
        self.address, self.shape, self.index = address, torch.Size(shape), device
        self.is_cuda, self.device = True, torch.device("cuda", device)

    def data_ptr(self): return self.address
    def get_device(self): return self.index
    def is_contiguous(self): return True
    def stride(self): return torch.empty(self.shape, device="meta").stride()


def _slot_cache(kvc, device=0, base=1 << 20):
    t = lambda i, *s: DeviceTensor(base + 4096 * i, s, device)  # noqa: E731
    return kvc.SlotCache(K=t(0, 2, 2, 64, 64), V=t(1, 2, 2, 64, 64), pos=t(2, 2, 2, 64),
                         n=t(3, 2, 2), seqlen=t(4, 2))


def _quant_cache(kvc):
    t = lambda i, *s: DeviceTensor((1 << 20) + 4096 * i, s)  # noqa: E731
    return kvc.QuantCache(k_blocks=t(0, 1, 2, 4, 1280), v_blocks=t(1, 1, 2, 4, 1280),
                          k_res=t(2, 1, 2, 64, 64), v_res=t(3, 1, 2, 64, 64), len=t(4, 1), bits=4,
                          R=32)


@pytest.mark.parametrize("make", [_slot_cache, _quant_cache])
def test_a_kept_descriptor_belongs_to_the_device_it_was_checked_on(kvc, make, monkeypatch):
    """A cache of cuda:0 is taken while cuda:0 is the current device, refused on cuda:1 although
    its descriptor is kept, and taken again afterwards."""
    now = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    cache = make(kvc)
    d = cache.desc()
    assert cache.desc() is d
    now[0] = 1
    for _ in range(2):
        with pytest.raises(ValueError, match="expected the current device cuda:1"):
            cache.desc()
    now[0] = 0
    assert cache.desc() is d


def test_the_calls_refuse_a_cache_of_another_device(kvc, monkeypatch):
    now = [0]
    monkeypatch.setattr(torch.cuda, "current_device", lambda: now[0])
    monkeypatch.setattr(kvc, "_raw_stream", lambda dev: 0)
    cache = _slot_cache(kvc)
    cache.desc()
    now[0] = 1
    q, i32 = DeviceTensor(64, (4, 4, 64), 1), DeviceTensor(64, (3,), 1)
    other = _slot_cache(kvc, device=1, base=1 << 24)
    for call in (lambda: kvc.kvc_chunk_attend(cache, q, i32, q),
                 lambda: kvc.kvc_append_plan(cache, i32, DeviceTensor(64, (4, 2), 1)),
                 lambda: kvc.kvc_append_plan(other, i32, DeviceTensor(64, (4, 2), 1), out=cache),
                 lambda: kvc.kvc_append_packed(cache, q, q, DeviceTensor(64, (4, 2), 1))):
        with pytest.raises(ValueError, match="expected the current device cuda:1"):
            call()


def test_a_descriptor_is_kept_before_its_key(kvc, monkeypatch):
    """Whoever finds a new key finds the descriptor that goes with it."""
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    cache = _slot_cache(kvc)
    first = cache.desc()

    class Watch(dict):
        def __setitem__(self, key, value):
            seen.append(key)
            super().__setitem__(key, value)

    seen = []
    cache.n = DeviceTensor(1 << 22, (2, 2))
    state = Watch(cache.__dict__)
    object.__setattr__(cache, "__dict__", state)
    second = cache.desc()
    assert second is not first and seen[-1] == "_desc_key" and "_desc" in seen
    # and from other threads the two always go together
    wrong = []

    def reader():
        for _ in range(2000):
            d = cache.desc()
            if d.n != cache.n.data_ptr():
                wrong.append(d.n)

    threads = [threading.Thread(target=reader) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
