"""The paged cache's binding on the CPU: what a call gets is what its caller gave."""

import pytest

import hierarchical_routed_sparse_hga_b200 as hga
from hierarchical_routed_sparse_hga_b200 import _lib

FAKE = 0x10000


def test_two_threads_with_their_own_configurations():
    """The cache keeps the C form of the last configuration.  Here another
    thread stores its own right behind each store of this one."""
    other = hga.Config(2, 32, 8, 128, 1, 1, scale=3.0)
    entry = (dict(other.__dict__), _lib.ctypes.byref(other.c()))

    class Shared(hga.PagedCache):
        @property
        def _kept(self):
            return self.__dict__.get("kept")

        @_kept.setter
        def _kept(self, value):
            self.__dict__["kept"] = None if value is None else entry

    cache = Shared.raw(FAKE, FAKE, FAKE, 100, 8 * 64 * 128, 64, 10)
    for scale in (0.5, 0.25):
        mine = hga.Config(2, 32, 8, 128, 1, 1, scale=scale)
        assert _lib._paged_cfg(cache, mine)._obj.scale == scale
    assert _lib._paged_cfg(cache, other)._obj.scale == 3.0


def test_a_kept_configuration_follows_its_changes():
    cache = hga.PagedCache.raw(FAKE, FAKE, FAKE, 100, 8 * 64 * 128, 64, 10)
    cfg = hga.Config(2, 32, 8, 128, 1, 1, scale=0.5)
    assert _lib._paged_cfg(cache, cfg)._obj.scale == 0.5
    assert _lib._paged_cfg(cache, cfg) is cache._kept[1]
    cfg.scale = 0.125
    assert _lib._paged_cfg(cache, cfg)._obj.scale == 0.125


def test_append_refuses_an_infinite_rope_base():
    """Its first pair would turn by the position itself, the others not at all."""
    cfg = hga.Config(2, 32, 8, 128, 1, 1)
    cache = hga.PagedCache.raw(FAKE, FAKE, FAKE, 100, 8 * 64 * 128, 64, 10)
    with pytest.raises(hga.HgaError) as e:
        hga.hga_paged_append(cfg, cache, FAKE, FAKE, FAKE, 32 * 128, 8 * 128, 1, None, FAKE, FAKE,
                             float("inf"), FAKE << 8, 0)
    assert e.value.status == hga.HGA_ERR_INVALID_ARG
