"""GPU test of the bounds of pages whose rows' scale bytes are any."""
import numpy as np
import pytest
import torch

import block_draft_proposal_amd as D
from gpu_helpers import DEV, require_gpu, say
from test_gpu_kv_sparse import check_bounds

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("low,high", [(0, 30), (0, 255), (100, 256), (225, 255)])
@pytest.mark.parametrize("kind,dim", [("e4m3", 64), ("e4m3", 128), ("e4m3", 256), ("i8", 64), ("i8", 128), ("i8", 256)])
def test_bounds_of_any_scale_byte(kind, dim, low, high):
    """Values down to fp32's smallest, which round outwards to a code of their
    sign, and beyond its largest; codes of all kinds."""
    require_gpu()
    say(f"scale bytes {kind} {dim} {low} {high}")
    n, heads, page = 40, 2, 5
    gen = torch.Generator(device=DEV).manual_seed(low + high + dim)
    shape = (n, heads, page, dim)
    codes = [torch.randint(0, 256, shape, generator=gen, device=DEV).to(torch.uint8) for _ in "kv"]
    if kind == "e4m3":
        for c in codes:
            c[(c & 0x7f) == 0x7f] = 0                    # NaN only in some pages
        codes[0][::9, 0, 1, 3] = 0x7f
        codes[0][1::3] &= 0x87                           # subnormal codes
    view = torch.float8_e4m3fn if kind == "e4m3" else torch.int8
    scales = [torch.randint(low, high, shape[:3], generator=gen, device=DEV).to(torch.uint8) for _ in "kv"]
    scales[0][::2] = scales[0][::2, :, :1]               # one scale to a page's rows, and several
    cache = D.KVCache(*(c.view(view) for c in codes), *scales)
    table = torch.randperm(n, generator=torch.Generator().manual_seed(3)).int()[None].to(DEV)
    check_bounds(cache, [cache.k, cache.v, cache.k_scale, cache.v_scale], table, table.cpu().numpy(), [0], [n * page])
