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
