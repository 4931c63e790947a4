"""What the binding of the operators around a verification step refuses
before the library is called (CPU only)."""
import pytest
import torch


@pytest.fixture(scope="module")
def sv():
    import rejection_sampling_verify_03_amd as m
    return m


U8 = torch.uint8


@pytest.mark.parametrize("codes,scales", [
    (torch.float8_e5m2, U8), (torch.float8_e4m3fnuz, U8), (torch.float8_e5m2fnuz, U8), (torch.int8, U8),
    (torch.bool, U8), (torch.bfloat16, U8), (torch.float8_e8m0fnu, U8), (U8, torch.int8), (U8, torch.bool),
    (U8, torch.float8_e4m3fn), (U8, torch.float32)])
def test_caches_of_other_types(sv, codes, scales):
    """Codes are e4m3 (or bytes) and scales exponent bytes: another 8-bit type
    would be read as what it is not."""
    k = torch.zeros(2, 16, 1, 64, dtype=U8).to(codes) if codes != torch.float8_e8m0fnu else \
        torch.zeros(2, 16, 1, 64, dtype=U8).view(codes)
    sc = torch.zeros(2, 1, 1, dtype=U8).to(scales)
    with pytest.raises(TypeError):
        sv.KVCache(k, k.clone(), sc, sc.clone())
