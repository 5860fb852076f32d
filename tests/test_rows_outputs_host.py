"""Outputs of one call that would be written over one another are refused by the C entry
points.  No GPU: the checks come before any launch."""
import pytest

FAKE, APART = 0x10000, 0x1000000   # never dereferenced
BF16, F32 = 0, 1


@pytest.fixture(scope="module")
def L():
    from fp8_gemms_b200 import _lib
    return _lib


@pytest.mark.parametrize("flags", [0, 1])
@pytest.mark.parametrize("dt", [BF16, F32])
def test_weight_gradients_in_one_buffer(L, dt, flags):
    """dweight and dbias: the same 64 elements, or some of them."""
    n = L.lm_layernorm_workspace_size(4, 64)
    size = 4 if flags or dt == F32 else 2

    def bwd(dw, db):
        return L.lib.lm_layernorm_bwd(FAKE, 64, FAKE, 64, None, FAKE, FAKE, 4, 64, dt, FAKE, 64, dw,
                                      db, FAKE, n, flags, None)

    def fused(dw, db):
        return L.lib.lm_dropout_add_layernorm_bwd(FAKE, 64, None, 0, FAKE, 64, None, FAKE, FAKE, 4,
                                                  64, dt, 0.1, FAKE, 0, FAKE, 64, APART, 64, dw, db,
                                                  FAKE, n, flags, None)
    for call in (bwd, fused):
        for apart in (0, size, 63 * size):
            assert call(2 * APART, 2 * APART + apart) == 1
            assert call(2 * APART + apart, 2 * APART) == 1


def test_statistics_in_one_buffer(L):
    def norm(mean, rstd):
        return L.lib.lm_layernorm_fwd(FAKE, 64, None, None, 4, 64, 1e-5, BF16, APART, 64, mean, rstd,
                                      None, None)

    def fused(mean, rstd):
        return L.lib.lm_dropout_add_layernorm_fwd(FAKE, 64, FAKE, 64, None, None, 4, 64, 1e-5, BF16,
                                                  0.1, FAKE, 0, APART, 64, 2 * APART, 64, mean, rstd,
                                                  None, None)
    for call in (norm, fused):
        for apart in (0, 4, 12):
            assert call(3 * APART, 3 * APART + apart) == 1
            assert call(3 * APART + apart, 3 * APART) == 1
