"""One-token attention over a cache in 4 bits where a page is missing inside a run of whole strips, at its ends and behind it: that sequence's rows are
NaN, the others' the same bits as with all pages there."""
import numpy as np
import pytest

from serving_lib import problem
from test_gpu_serving import bits, ffa  # noqa: F401  (ffa is the fixture)

pytestmark = pytest.mark.gpu


# d, q heads, kv heads, page, warps of the kernel: a strip is 32 keys
@pytest.mark.parametrize("d,hq,hkv,page,warps", [(128, 16, 4, 64, 12), (128, 8, 1, 32, 12), (64, 16, 4, 64, 16), (64, 32, 2, 128, 8)])
def test_missing_pages_in_runs(ffa, d, hq, hkv, page, warps):
    import torch
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    block = 32 * warps
    keys = 5 * sms * block // (2 * hkv)   # two such sequences: 5 blocks a CTA and more, each the first or the last of few
    lens = [keys, keys + 3 * block + 5, 777]
    p, c = problem(lens, hq, hkv, d, page, "e2m1", d + page)
    good, gl = ffa.fwd_decode(**p, scale=0.1)
    assert not good.isnan().any()
    pages = -(-lens[1] // page)
    spots = {0, 1, pages - 1, pages - 2} | {int(x) for x in np.random.default_rng(d).integers(2, pages - 2, 24)}
    spots |= {(k * block + 32 * (warps - 1)) // page for k in (2, 3, 4)} | {(lens[1] // block * block - 1) // page}
    for i, spot in enumerate(sorted(spots)):
        kept = int(p["page_table"][1, spot])
        p["page_table"][1, spot] = (-1, c.shape[0], 2 ** 31 - 1)[i % 3]
        out, lse = ffa.fwd_decode(**p, scale=0.1)
        p["page_table"][1, spot] = kept
        assert out[1].isnan().all() and lse[:, 1].isnan().all(), spot
        for b in (0, 2):
            assert (bits(out[b]) == bits(good[b])).all() and (bits(lse[:, b]) == bits(gl[:, b])).all(), (spot, b)
    out, lse = ffa.fwd_decode(**p, scale=0.1)
    assert (bits(out) == bits(good)).all() and (bits(lse) == bits(gl)).all()
