"""Weights of head norms on the way into the cache: bf16 ones give bit for bit what fp32 ones of the same
values give, in every layout and on both ways that a call's arguments are read."""

import pytest

from exact_attention_52_gb300 import api

from .test_gpu_cache import Pool, check_clean, i32
from .test_gpu_rope import table_of

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("compiled", [True, False])
@pytest.mark.parametrize("norms", ["q", "k", "qk"])
@pytest.mark.parametrize("page,T,lens,d,rot,interleaved", [(16, 1, [40, 1], 64, 64, False), (16, 5, [40, 5], 128, 64, True),
                                                           (64, 70, [300, 70], 128, 128, False),
                                                           (256, 300, [301, 700], 64, 32, False)])
def test_append_with_bf16_weights(page, T, lens, d, rot, interleaved, norms, compiled, monkeypatch):
    import torch
    if not compiled:
        monkeypatch.setattr(api, "_read", lambda *a: (None, None, None))
    pool = Pool(T, 2, 3, d, page, -(-max(lens) // page))
    q, k, v = (torch.randn(2, h, T, d, device="cuda").bfloat16() for h in (5, 3, 3))
    w = {x: (1.0 + 0.3 * torch.randn(d, device="cuda")).bfloat16() for x in norms}
    got = []
    for cast in (lambda x: x, lambda x: x.float()):
        dev = pool.dev()
        out = api.cache_append_rope(q, k, v, table_of(rot, interleaved), *dev, i32(lens),
                                    **{x + "_weight": cast(w[x]) for x in norms})
        got.append((out, *dev))
    check_clean()
    for x, y in zip(*got):
        assert torch.equal(x.view(torch.int16) if x.dtype == torch.bfloat16 else x, y.view(torch.int16) if
                           y.dtype == torch.bfloat16 else y)
