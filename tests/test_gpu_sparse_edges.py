"""The sparse decode step's operators at their edges: the sizes, values and
streams where a result could be wrong although the ordinary cases are right."""
import numpy as np
import pytest
import torch

import paged_kv_cache_82_gb300 as pa
from tests import _sparse_ref as ref

pytestmark = pytest.mark.gpu


def _summarise_whole(kc, blocks, H, D, cache):
    """Records of `blocks` full blocks of one request."""
    got = torch.zeros(blocks, H, pa.bounds_bytes(D), dtype=torch.uint8, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    n = 16 * blocks
    pa.pa_summarise_blocks(kc, got, torch.arange(blocks, **i32)[None].contiguous(),
                           torch.tensor([n], **i32), torch.tensor([0, n], **i32), n, n, n,
                           cache_dtype=cache)
    assert pa.pa_get_device_error() == 0
    return ref.records(got, D)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("cache", ["f32", "int4"])
def test_codes_of_subnormal_keys(cache, D):
    """Keys of a few units of 2^-149: the scale is a subnormal of few bits, and
    quotients go past 127 on either side.  Codes stay in [-127, 127]."""
    rng = np.random.default_rng(D)
    unit = np.array([-130, 178, -178, 190, -190, -127, 1000, -1000, 65, 1, -1, -5000])
    B = len(unit)
    if cache == "f32":
        keys = np.broadcast_to(unit[:, None, None].astype(np.float64), (B, 16, D)) * 2.0 ** -149
        keys = keys.copy()
        keys[-1] *= rng.integers(1, 4, (16, D))
        kc = torch.from_numpy(keys.astype(np.float32)).view(B, 1, 16, D).cuda()
    else:  # codes of one sign, scales of a few units
        page = np.zeros((B, 1, pa.page_bytes_4bit("int4", D)), dtype=np.uint8)
        for b in range(B):
            code = int(np.sign(unit[b])) * (rng.integers(1, 8, (16, D)) if b % 3 == 2 else
                                            np.ones((16, D), dtype=np.int64))
            nib = (code & 15).astype(np.uint8)
            page[b, 0, :8 * D] = (nib[:, ::2] | nib[:, 1::2] << 4).reshape(-1)
            sc = np.full(16, abs(int(unit[b])), np.uint32)  # the bits of units of 2^-149
            page[b, 0, 8 * D:] = sc.view(np.uint8)
        kc = torch.from_numpy(page).cuda()
        keys = ref.decode_pages(kc, "int4", D)[:, 0]
    hi, lo, s = _summarise_whole(kc, B, 1, D, cache)
    for b in range(B):
        w = ref.bounds_of(keys[b])
        np.testing.assert_array_equal(hi[b, 0], w[0])
        np.testing.assert_array_equal(lo[b, 0], w[1])
        assert s[b, 0] == w[2]
