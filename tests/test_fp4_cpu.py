"""The cache in 4-bit floats without a GPU: byte accounting, refusals, and pins of the
tests' own reference."""
import numpy as np
import pytest

import fp4_ref
import paged_quantized_kv_kvq_gb300 as kvq
from paged_quantized_kv_kvq_gb300 import build as kbuild


@pytest.fixture(scope="module", autouse=True)
def _built():
    kbuild.build()


@pytest.mark.parametrize("nb,bs,hkv,d", [(9103, 16, 8, 128), (64, 16, 1, 64), (100, 32, 32, 128), (7, 64, 3, 64)])
def test_bytes(nb, bs, hkv, d):
    """4 bits a value and a byte for 16 of them; a page's parts stay 16-byte aligned."""
    lay = kvq.kvq_pool_layout_query(nb, bs, hkv, d, kvq.KVQ_FP4_E2M1)
    n = 2 * nb * bs * hkv * d
    assert lay["code_bytes"] == n // 2 and lay["scale_bytes"] == n // 16
    assert lay["page_bytes"] * nb * hkv == n // 2 + n // 16 and lay["page_bytes"] % 16 == 0
    assert lay["total_bytes"] == kvq.kvq_pool_bytes(nb, bs, hkv, d, kvq.KVQ_FP4_E2M1, 77)  # (the group is not looked at)


@pytest.mark.parametrize("nb,bs,hkv,d,status", [
    (8, 8, 8, 128, kvq.KVQ_ERR_UNSUPPORTED), (8, 48, 8, 128, kvq.KVQ_ERR_UNSUPPORTED), (8, 16, 8, 96, kvq.KVQ_ERR_UNSUPPORTED),
    (0, 16, 8, 128, kvq.KVQ_ERR_INVALID_ARG), (8, 16, 0, 128, kvq.KVQ_ERR_INVALID_ARG)])
def test_refusals(nb, bs, hkv, d, status):
    with pytest.raises(kvq.KVQError) as e:
        kvq.kvq_pool_layout_query(nb, bs, hkv, d, kvq.KVQ_FP4_E2M1)
    assert e.value.status == status
    assert kvq.kvq_pool_bytes(nb, bs, hkv, d, kvq.KVQ_FP4_E2M1) == 0


def test_nine_is_no_format():
    with pytest.raises(kvq.KVQError):
        kvq.kvq_pool_layout_query(8, 16, 8, 128, 9)


def test_reference_codes():
    """Ties go to the even code, 6 is the end, zeros keep their sign, NaN is the largest."""
    s = 4.0
    x = np.zeros((1, 16), np.float32)
    q = [6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -0.25, -0.26, -5, 5.01, 0, -0.0, 1.7, -6]
    x[0] = np.array(q) * s
    code, sb = fp4_ref.quantize(x)
    assert fp4_ref.SCALES[sb[0, 0]] == s
    assert code[0].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 8, 9, 14, 7, 0, 8, 3, 15]
    x[0, 3], x[0, 4] = np.nan, np.inf
    code, sb = fp4_ref.quantize(x)
    assert fp4_ref.SCALES[sb[0, 0]] == 10240 and code[0, 3] == 7 and code[0, 4] == 7
    assert (fp4_ref.quantize(np.full((1, 16), 6 * 2.0 ** -18))[0] == 0).all()


def test_reference_scales_are_fp16_bits():
    """Byte b stands for the fp16 whose bits are b << 7; quotients between two go to the nearer."""
    b = np.arange(len(fp4_ref.SCALES), dtype=np.uint16)
    assert np.array_equal((b << 7).view(np.float16).astype(np.float64), fp4_ref.SCALES)
    for i in (0, 1, 7, 8, 9, 100, 101, 0xE0, 0xE1):
        mid = (fp4_ref.SCALES[i] + fp4_ref.SCALES[i + 1]) / 2
        x = np.full((1, 16), mid * 6, np.float32)
        assert x[0, 0] == mid * 6
        assert fp4_ref.quantize(x)[1][0, 0] == (i if i % 2 == 0 else i + 1)
        x = np.nextafter(x, np.float32(np.inf))
        assert fp4_ref.quantize(x)[1][0, 0] in (i + 1, i if i % 2 == 0 else i + 1)


def test_quantization_error_is_bounded():
    """Codes are a sixth of the absmax apart at most at the top (2 of 6, half of that off)
    and the scale is within 1/16: every value is within (1/6)(17/16) of the group's absmax,
    or saturates within 1/16 of it."""
    x = (np.random.default_rng(0).standard_normal((500, 128)) * 2.0 ** np.random.default_rng(1).integers(-10, 10, (500, 1))).astype(np.float32)
    got = fp4_ref.values(*fp4_ref.quantize(x))
    amax = np.abs(x.reshape(500, 8, 16)).max(-1).repeat(16, -1)
    assert (np.abs(got - x) <= amax * (17 / 16 / 6) + 2.0 ** -17 * 3).all()
