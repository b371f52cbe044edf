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


def test_blocks_outputs_that_are_inputs(lib):
    """Every output of a step beside every input and every other output: equal pointers are refused."""
    names = ["ctx", "new", "free", "cur", "table", "slots", "pos", "cu", "kv", "state"]

    def call(**kw):
        a = {n: 0x100000 + 0x1000 * i for i, n in enumerate(names)}
        a.update(kw)
        return lib.wq_kv_blocks(a["ctx"], a["new"], 4, a["free"], 3, a["cur"], 64, a["table"], 8, 4, a["slots"],
                                a["pos"], a["cu"], a["kv"], a["state"], None)
    at = {n: 0x100000 + 0x1000 * i for i, n in enumerate(names)}
    for out in ["table", "slots", "pos", "cu", "kv", "state"]:
        for other in names:
            if other != out:
                assert call(**{out: at[other]}) == 1, (out, other)
