"""Layouts that the forward's binding refuses before anything is launched."""
import pytest
import torch


@pytest.fixture(scope="module")
def sv():
    import os

    from speculative_decoding_verify_07_gb300 import build
    if not os.path.exists(build.LIB):
        build.build()
    from speculative_decoding_verify_07_gb300 import binding
    return binding


def cache(pages=4, heads=2, page=16, dim=64):
    k = torch.zeros((pages, heads, page, dim), dtype=torch.bfloat16)
    cu, kv = torch.tensor([0, 3], dtype=torch.int32), torch.tensor([3], dtype=torch.int32)
    return cu, kv, torch.zeros((1, 4), dtype=torch.int32), k, k.clone()


@pytest.mark.parametrize("make", [lambda t: t[:1].expand(3, -1, -1),                       # one token for all
                                  lambda t: t[:, :1].expand(-1, 2, -1),                    # one head for all
                                  lambda t: t.transpose(0, 1).contiguous().transpose(0, 1)])
def test_tokens_that_overlap_or_are_not_dense(sv, make):
    args = cache()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.spec_cache_write(make(x), x, *args)
    with pytest.raises(ValueError):
        sv.spec_cache_write(x, make(x), *args)
    with pytest.raises(ValueError):
        sv.spec_attend(make(x), *args, max_tokens=3, workspace=torch.zeros(1 << 20, dtype=torch.uint8))


def test_pages_that_overlap(sv):
    cu, kv, table, k, v = cache()
    x = torch.zeros((3, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        sv.spec_cache_write(x, x, cu, kv, table, k[:1].expand(4, -1, -1, -1), v[:1].expand(4, -1, -1, -1))
    with pytest.raises(ValueError):
        sv.spec_cache_write(x, x, cu, kv, table, k[:, :, ::2], v[:, :, ::2])
    with pytest.raises(ValueError):      # keys interleaved with values, values alone
        sv.spec_cache_write(x, x, cu, kv, table, torch.stack([k, v], 1)[:, 0], v)
