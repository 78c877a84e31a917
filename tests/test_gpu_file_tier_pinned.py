"""The file tier beside other users of pinned memory: the driver gives small pinned allocations out of one block, so
the RAM slots' own allocation need not start on a page."""
import pytest

import synth as S
from tests.helpers import LayerSpec, make_context

pytestmark = pytest.mark.gpu


def test_file_tier_context_beside_small_pinned_allocations(tmp_path):
    import torch
    spec = LayerSpec(512, 256, 16, 2, S.INT4, router=0, seed=3)
    probe = make_context(spec, 1, hbm_cache_bytes=1 << 40, register=False)
    rb = probe.stats()["record_bytes"]
    probe.close()
    stride = (rb + 4095) // 4096 * 4096
    held = []
    for i in range(6):
        held.append(torch.empty(300 + 512 * i, dtype=torch.uint8).pin_memory())
        ctx = make_context(spec, 1, hbm_cache_bytes=2 * spec.k * rb, pool_file=str(tmp_path / ("experts%d.bin" % i)),
                           host_cache_bytes=(2 * spec.k + 1) * stride)
        ctx.close()
