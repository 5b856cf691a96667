"""Sketches of more rows than the tensor-core quantiser's block can hold at
d = 128: the general encoder takes them, with the same records."""
import numpy as np
import pytest
import torch

import oracle as O
import synth
from parity_util import compare_compressed

pytestmark = pytest.mark.gpu

tq = pytest.importorskip("kv_cache_vector_09_b200")
DEV = torch.device("cuda", 0)


@pytest.mark.parametrize("m", [224, 256, 288])
@pytest.mark.parametrize("bits,dtype", [((1,), torch.bfloat16), ((3,), torch.float32), ((4,), torch.bfloat16)])
def test_quantize_wide_sketches(m, bits, dtype):
    x = synth.heavy_rows(m, 300, 128, n_out=2, dtype=dtype)
    codec, oc = tq.Codec(128, bits, m, 0), O.make_codec(128, bits, m, 0)
    got = tq.tq_quantize(codec, x.to(DEV), tq.Compressed.empty(codec, 300))
    compare_compressed(got, O.quantize(x.to(torch.float64).numpy(), oc), oc)


@pytest.mark.parametrize("m", [224, 256])
def test_rope_refuses_what_does_not_fit_and_leaves_the_next_call_alone(m):
    codec = tq.Codec(128, (4,), m, 0)
    x, cs = torch.randn((64, 128), device=DEV), tq.tq_rope_cache(1e4, 128, 64)
    out = tq.Compressed.empty(codec, 64)
    pos = torch.arange(64, dtype=torch.int32, device=DEV)
    if m == 224:
        tq.tq_quantize_rope(codec, x, cs, pos, out)
    else:
        with pytest.raises(tq.TQError) as e:
            tq.tq_quantize_rope(codec, x, cs, pos, out)
        assert e.value.status == 2
    small = tq.Codec(128, (4,), 64, 0)
    tq.tq_quantize(small, x, tq.Compressed.empty(small, 64))


def test_a_cache_with_256_sketch_rows_from_rows_to_attention():
    d, B, Hq, Hkv, Tp = 128, 2, 4, 2, 150
    rng = np.random.default_rng(0)
    kc, vc = tq.Codec(d, (4,), 256, 0), tq.Codec(d, (4,), 0, 1)
    x = [torch.from_numpy(rng.standard_normal((Hkv * Tp, d)).astype(np.float32)).to(DEV) for _ in range(2)]
    K, V = (tq.tq_quantize(c, t, tq.Compressed.empty(c, Hkv * Tp)) for c, t in zip((kc, vc), x))
    q = torch.from_numpy(rng.standard_normal((B, Hq, d)).astype(np.float32)).to(DEV)
    out = torch.empty((B, Hq, d), device=DEV)
    tq.tq_attend_prefix(kc, vc, q, B, Hq, Hkv, Tp, K, V, 0, None, None, out,
                        tq.workspace(tq.tq_attend_prefix_workspace_size(kc, vc, B, Hq, Hkv, Tp, 0), DEV))
    # the exact attention of the rows themselves: four bits and a wide sketch come near it
    k, v = (t.double().view(Hkv, Tp, d) for t in x)
    p = torch.softmax(torch.einsum("bkgd,ktd->bkgt", q.double().view(B, Hkv, 2, d), k) / d ** 0.5, -1)
    want = torch.einsum("bkgt,ktd->bkgd", p, v).reshape(B, Hq, d)
    # 4-bit Lloyd-Max leaves 0.0095 of a row's energy, 0.0975 of its norm: that much of the values, and, with logits
    # of one, as much of every weight; sqrt(2) 0.0975 = 0.14, times two for 4 x 2 rows of one draw
    assert (out.double() - want).norm() <= 0.3 * want.norm()
