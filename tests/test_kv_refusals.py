"""More refusals of the key/value cache entry points, on the host and before
any launch (CPU only)."""
import pytest

P, P2 = 0x10000, 0x20000                                    # never dereferenced


@pytest.fixture(scope="module")
def lib():
    import weight_only_quantized_quant_amd as W            # sets the argument types
    return W.lib


@pytest.mark.parametrize("cap", [0.0, 10.0])
def test_attention_scale_whose_exponent_overflows(lib, cap):
    """sm_scale * log2(e), by which scores go to base 2, has to be finite."""
    def call(sm):
        return lib.wq_kv_attention(P, 1024, P, P, 2, 4, 0, 8, 4, 128, P, P, P, P, 64, 10, P, 4, sm, cap, 0, P2, None,
                                   P, 1 << 40, None)
    for sm in (3.4e38, 3e38, 2.4e38, 1.8e38):
        assert call(sm) == 3, sm
    assert call(float("inf")) == 1
