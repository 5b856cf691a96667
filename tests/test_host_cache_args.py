"""The binding's own checks of the shared-prefix attention's tensors, and the
exact size of its workspace, without a GPU."""
import pytest
import torch

import kv_cache_vector_09_b200 as tq


class OnDevice(torch.Tensor):
    """A host tensor that says it is on the codec's device (which is a host-only
    codec here, so that the library refuses what the binding lets through)."""

    def get_device(self):
        return 3


def call(workspace):
    kc, vc = tq.Codec(128, (3,), 0, 0, device=-1), tq.Codec(128, (4,), 0, 1, device=-1)
    kc.device = vc.device = 3
    dev = lambda *s, dtype=torch.float32: torch.zeros(s, dtype=dtype).as_subclass(OnDevice)  # noqa: E731
    q = dev(1, 2, 128)
    cache = lambda c: tq.Compressed(dev(8, c.code_words, dtype=torch.int32), None, dev(8), None)  # noqa: E731
    tq.tq_attend_prefix(kc, vc, q, 1, 2, 1, 8, cache(kc), cache(vc), 0, None, None, dev(1, 2, 128), workspace, stream=0)


def test_a_workspace_elsewhere_is_refused_by_the_binding():
    good = torch.zeros(1 << 20, dtype=torch.uint8).as_subclass(OnDevice)
    with pytest.raises(tq.TQError, match="host-only"):      # all tensors in order: the library sees the call
        call(good)
    with pytest.raises(AssertionError, match="workspace"):  # on the host
        call(torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(AssertionError, match="workspace"):  # every second byte of a larger one
        call(torch.zeros(1 << 21, dtype=torch.uint8).as_subclass(OnDevice)[::2])


def up256(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("Tp,T,chunks", [
    (0, 0, 0), (1, 0, 1), (64, 0, 1), (65, 0, 2), (3000, 700, 47 + 11),   # 64 keys a chunk at least
    (40000, 0, 148), (0, 40000, 74),                                      # two blocks an SM over all units
    (200000, 0, 196), (0, 100000, 98),                                    # at most 1024 keys a chunk
])
def test_the_workspace_holds_every_partial(Tp, T, chunks):
    # d = 256: prepared fp32 queries, and per query row and chunk d values, the
    # maximum, the sum and m_v sketch entries; two units of prefix, four of own
    # keys, 148 SMs (taken where there is no GPU)
    kc, vc = tq.Codec(256, (3,), 64, 0, device=-1), tq.Codec(256, (2,), 64, 1, device=-1)
    rows = 2 * 4
    want = up256(4 * rows * (256 + 64)) + up256(4 * rows * chunks * (256 + 2 + 64))
    assert tq.tq_attend_prefix_workspace_size(kc, vc, 2, 4, 2, Tp, T) == want


@pytest.mark.parametrize("B,Tp,T,groups,blocks", [
    (1, 509, 63, 8, 9), (4, 32768, 512, 8, 18), (64, 16384, 64, 16, 9), (160, 4096, 0, 40, 3),
    (640, 4096, 0, 160, 4), (1, 0, 1, 8, 1), (3, 0, 0, 8, 0)])
def test_the_workspace_of_the_tensor_core_kernel(B, Tp, T, groups, blocks):
    # query images of two fp16 parts and a scale a row, 128 rows a group of
    # 128 / G sequences; a partial a row and block of its group.  160 groups on
    # 148 SMs: 4 blocks each are 5 waves of a quarter, 3 are 4 of a third
    kc, vc = tq.Codec(128, (3,), 128, 0, device=-1), tq.Codec(128, (4,), 0, 1, device=-1)
    Hq, Hkv = 32, 8
    want = up256(groups * 128 * (2 * 2 * (128 + 128) + 4)) + up256(4 * B * Hq * blocks * (128 + 2))
    assert tq.tq_attend_prefix_workspace_size(kc, vc, B, Hq, Hkv, Tp, T) == want


def test_no_sequence_needs_no_workspace():
    for d in (128, 256):
        kc, vc = tq.Codec(d, (3,), 64, 0, device=-1), tq.Codec(d, (2,), 0, 1, device=-1)
        assert tq.tq_attend_prefix_workspace_size(kc, vc, 0, 32, 8, 100, 10) == 0
