"""Argument checks of the shared-prefix attention and of the bounded cache that
need no GPU: workspace sizes and calls on host-only codecs."""
import ctypes

import pytest

import kv_cache_vector_09_b200 as tq


def _size(kc, vc, *shape):
    return tq.tq_attend_prefix_workspace_size(kc, vc, *shape)


def test_workspace_size_covers_queries_and_partials():
    kc, vc = tq.Codec(128, (3,), 128, 0, device=-1), tq.Codec(128, (4,), 0, 1, device=-1)
    # nothing to read: only the queries; more keys never need less
    sizes = [_size(kc, vc, 4, 32, 8, Tp, T) for Tp, T in ((0, 0), (1, 0), (64, 0), (4096, 0), (4096, 512), (131072, 512))]
    assert sizes == sorted(sizes) and sizes[1] > sizes[0]
    # a partial per query row and block at least
    assert sizes[-1] >= 4 * 32 * (128 + 2) * 4
    # codecs without the tensor-core kernel: prepared fp32 queries, value sketch in the partials
    kg, vg = tq.Codec(256, (3,), 64, 0, device=-1), tq.Codec(256, (2,), 64, 1, device=-1)
    assert _size(kg, vg, 2, 4, 2, 300, 70) >= 2 * 4 * (256 + 64) * 4 + 2 * 4 * (256 + 2 + 64) * 4
    assert _size(kc, vc, 0, 32, 8, 100, 10) >= 0


@pytest.mark.parametrize("shape,status", [((-1, 4, 2, 1, 1), 1), ((1, 3, 2, 1, 1), 1), ((1, 0, 1, 1, 1), 1),
                                          ((1, 4, 2, -1, 1), 1), ((1, 4, 2, 1, -1), 1), ((1, 66, 2, 1, 1), 2),
                                          ((2 ** 30, 4, 2, 1, 1), 2), ((1, 4, 2, 2 ** 31, 1), 2), ((1, 4, 2, 1, 2 ** 31), 2)])
def test_workspace_size_refuses_bad_shapes(shape, status):
    kc, vc = tq.Codec(128, (3,), 128, 0, device=-1), tq.Codec(128, (4,), 0, 1, device=-1)
    with pytest.raises(tq.TQError) as e:
        _size(kc, vc, *shape)
    assert e.value.status == status


def test_workspace_size_refuses_codec_pairs():
    k64, k128, k512 = (tq.Codec(d, (3,), 0, 0, device=-1) for d in (64, 128, 512))
    sketched = tq.Codec(128, (3,), 256, 0, device=-1)
    for kc, vc, status in ((k64, k128, 1), (k512, k512, 2), (k128, sketched, 2)):
        with pytest.raises(tq.TQError) as e:
            _size(kc, vc, 1, 4, 2, 10, 10)
        assert e.value.status == status
    lib, n = tq.c_api(), ctypes.c_size_t()
    assert lib.tq_attend_prefix_workspace_size(None, k128.handle, 1, 4, 2, 1, 1, ctypes.byref(n)) == 1
    assert lib.tq_attend_prefix_workspace_size(k128.handle, k128.handle, 1, 4, 2, 1, 1, None) == 1


def test_calls_on_a_host_only_codec_are_refused():
    lib, c = tq.c_api(), tq.Codec(128, (3,), 0, 0, device=-1)
    x = ctypes.byref(tq.tq_compressed())
    assert lib.tq_attend_prefix(c.handle, c.handle, None, 0, 1, 4, 2, 0.0, 1, x, x, 1, None, x, x, None, 0, None, 0, None, None) == 1
    assert "host-only" in tq.tq_last_error_string()
    assert lib.tq_mass_update(c.handle, None, 1, 4, 2, 10, None, None, 0.0, 1.0, None, None) == 1
    assert lib.tq_evict_select(c.handle, None, 1, 2, 10, None, 5, 0, 0, None, None, None, None) == 1
    assert lib.tq_copy_rows(c.handle, x, 1, x, 1, 1, 1, None, None, None) == 1
    for name in ("tq_attend_prefix", "tq_mass_update", "tq_evict_select", "tq_copy_rows"):
        assert getattr(lib, name)(None, *[0] * (len(getattr(lib, name).argtypes) - 1)) == 1
