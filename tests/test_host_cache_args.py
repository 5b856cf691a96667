"""The binding's own checks of the shared-prefix attention's tensors, without a
GPU."""
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
