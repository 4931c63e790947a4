"""The 8-bit paged cache on the GPU at the ends of what its scale bytes hold."""
import pytest
import torch

import ops_oracle as oo
from test_gpu_kv_cache import check_write, sv  # noqa: F401  (sv: the fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("byte", [1, 9, 10, 247, 248, 252, 253, 254])
def test_groups_with_bytes_of_other_programs(sv, byte, dtype):  # noqa: F811
    """Writes behind a group's first token, into groups whose scale is not one
    that a write makes."""
    k, v, _, _ = oo.random_cache(3, 16, 2, 32, 16, byte)
    sc = torch.full((3, 2, 1), byte, dtype=torch.uint8)
    cache = sv.KVCache(k.cuda(), v.cuda(), sc.cuda(), sc.cuda())
    g = torch.Generator().manual_seed(byte)
    key, value = (torch.randn(6, 2, 32, generator=g) * s for s in (1e37, 1e-3))
    key[2], value[2] = 2.0 ** 127, -1.75 * 2.0 ** 127
    check_write(sv, cache, key.to(dtype), value.to(dtype), torch.tensor([3, 4, 5, 16 + 15, 32, 33]))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_the_largest_values_read_back(sv, dtype):  # noqa: F811
    """Up to 1.9296875 * 2^127 (the bf16 below 1.9375 * 2^127) the nearest
    code's value is finite; from there on it is 2^128."""
    cache = sv.make_kv_cache(2, 16, 1, 16, scale_tokens=1)
    x = torch.zeros(2, 1, 16)
    x[0, 0, 0], x[0, 0, 1] = 1.9296875 * 2.0 ** 127, -1.75 * 2.0 ** 127
    x[1, 0, 0], x[1, 0, 1], x[1, 0, 2] = 1.9375 * 2.0 ** 127, -torch.finfo(dtype).max, 2.0 ** 120
    slots = torch.tensor([3, 20]).cuda()
    sv.kv_write(cache, x.to(dtype).cuda(), x.to(dtype).cuda(), slots)
    for t in sv.kv_read(cache, slots, dtype=dtype):
        t = t.float().cpu()
        assert t[0, 0, 0] == 1.875 * 2.0 ** 127 and t[0, 0, 1] == -1.75 * 2.0 ** 127
        assert t[1, 0, 0] == float("inf") and t[1, 0, 1] == -float("inf") and t[1, 0, 2] == 2.0 ** 120
