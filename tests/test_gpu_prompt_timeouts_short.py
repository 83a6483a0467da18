"""An expired wait of a block whose loads are all under way, or landed, when it gives
up: the warp that loads has found the end of the units and left its loop by then.  As
everywhere, the copies land before the block ends, the block's rows are NaN and the
calls after it are as before."""

import pytest
import torch

import speculative_decoding_verification_13_gb300 as sv
from test_gpu_prompt_timeouts import check, expire  # noqa: F401

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("D,n", [(128, [90] * 40), (64, [300, 20] * 20), (256, [60] * 50),
                                 (128, [200])])
@pytest.mark.parametrize("block", [0, 3])
def test_prompts_of_a_tile_or_two(expire, D, n, block):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(3)
    at = torch.tensor([0] + n, device=DEV).cumsum(0).int()
    q, k, v = (torch.randn(sum(n), h, D, device=DEV, generator=g).bfloat16() for h in (32, 8, 8))
    check(expire, block, lambda **kw: sv.prompt_attention(q, k, v, at, **kw),
          sv.prompt_attention_error)


@pytest.mark.parametrize("D,page", [(64, 16), (128, 7), (128, 64)])
@pytest.mark.parametrize("block", [0, 3])
def test_trees_of_a_tile_or_two(expire, D, page, block):  # noqa: F811
    g = torch.Generator(device=DEV).manual_seed(4)
    B, k, Hk, n = 24, 63, 8, 130
    pages = -(-n // page)
    i32 = dict(dtype=torch.int32, device=DEV)
    cache = torch.randn(B * pages, 1, 2, page, Hk * D, device=DEV, generator=g).bfloat16()
    spec = torch.randn(B, k + 1, 1, 2, Hk * D, device=DEV, generator=g).bfloat16()
    q = torch.randn(B * (k + 1), Hk * 4, D, device=DEV, generator=g).bfloat16()
    parent = torch.arange(k + 1, **i32).sub(1).clamp(min=0).div(2, rounding_mode="floor")
    args = (q, cache, 0, torch.full((B,), n, **i32), torch.arange(B * pages, **i32).view(B, pages),
            torch.full((B,), k, **i32), parent.int().repeat(B), spec)
    check(expire, block, lambda **kw: sv.tree_attention(*args, **kw), sv.tree_attention_error)
