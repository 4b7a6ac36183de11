"""Two threads in the binding's first calls: neither sees the library half loaded (no GPU needed: calls without tokens)."""
import ctypes
import threading
import time

import pytest

import kda_gated_delta_rule_gb300 as kda
from kda_gated_delta_rule_gb300 import _build


class SlowLibrary(ctypes.CDLL):
    """Takes its time over the functions that calls with packed arguments look up by index."""
    lookups = 0

    def __getattr__(self, name):
        if name.startswith("__"):
            raise AttributeError(name)
        fn = super().__getitem__(name)
        setattr(self, name, fn)
        return fn

    def __getitem__(self, name):
        self.lookups += 1
        if self.lookups == 2:
            between.set()
        time.sleep(0.1)
        return super().__getitem__(name)


between = threading.Event()


@pytest.fixture
def unloaded(monkeypatch):
    _build.build()
    monkeypatch.setattr(kda, "_lib", None)
    monkeypatch.setattr(kda, "_packed", {})
    monkeypatch.setattr(kda.ctypes, "CDLL", SlowLibrary)
    between.clear()


@pytest.mark.parametrize("name", ["kda_qk_norm_rope", "kda_kv_read", "kda_paged_attention"])
def test_a_call_beside_the_loading_one(unloaded, name):
    cache = kda._pack_cache(0, 0, 0, 0, 0, 1, 16, 2, 64)
    args = {"kda_qk_norm_rope": (kda._pack_norm(0, 0, 256, 128, 1, 0, 0, 0, 0, 0, 0, 0, 0, 1e-6, 0, 4, 2, 64, 0, 0, 256, 128, 1, 0), 0),
            "kda_kv_read": (cache, 0, 0, 0, 0, 1, 0, 0),
            "kda_paged_attention": (kda._pack_attention(0, 1, 0, 1, 4, 0, 0, 0, 0, 0, 1, 16, 2, 64, 0, 0, 0, 0.1, 0.0, 0, 0, 1, 0,
                                                        0, 0, 0), 0)}[name]
    first = threading.Thread(target=kda.load)
    first.start()
    assert between.wait(60)
    kda._call(name, *args)  # while the other is between its look-ups
    first.join()
    for fn in kda._packed.values():
        assert fn.restype is ctypes.c_int and fn.argtypes
    kda._call(name, *args)
