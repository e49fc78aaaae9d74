"""CPU tests of host-side behaviour of the prompt calls beside their refusals.
Nothing here launches a kernel."""
import pytest


@pytest.fixture(scope="module")
def K():
    from quantized_kv_decode_gb300 import build
    build.build()
    import quantized_kv_decode_gb300 as K
    K.lib()
    return K


def test_a_release_library_lets_no_wait_run_out(K):
    lib = K._lib.load(K._lib.LIB_PATH)
    assert lib.kvq_debug_fail_wait(K._lib.KVQ_WAIT_K, 0) == K.KVQ_ERR_UNSUPPORTED


def test_the_package_has_every_flag_of_the_header(K):
    import os
    import re
    from tests.conftest import ROOT
    text = open(os.path.join(ROOT, "include", "kvq.h")).read()
    flags = {n: int(v, 16) for n, v in re.findall(r"#define (KVQ_FLAG_\w+)\s+(0x[0-9a-f]+)u", text)}
    assert len(flags) == 8
    for name, value in flags.items():
        assert getattr(K, name, None) == value, name


def test_two_fp16_numbers_hold_a_dequantized_value():
    """(q - z) s is the sum of its rounding to fp16 and the rest, exactly: the
    product is d m 2^e with |d| <= 255 + 2048 < 2^12, m < 2^11 and e >= -24 (an
    fp16 scale is a whole number of 2^-24), so it has 23 bits; the rounding
    takes 11 and leaves at most 2^11 units of 2^e, which fp16 holds.  All d and
    m, for the smallest scales, where fp16 has fewest bits, and for others."""
    import numpy as np
    d = np.arange(-2303, 2304, dtype=np.float64)
    for e in (-24, -20, -14, -10):
        for m0 in range(1, 2048, 64):
            s = (np.arange(m0, min(m0 + 64, 2048)) * 2.0 ** e)[:, None]
            assert np.array_equal(s, s.astype(np.float16))
            x = d * s
            hi = x.astype(np.float16).astype(np.float64)
            lo = (x - hi).astype(np.float16).astype(np.float64)
            here = np.abs(x) <= 65504
            assert np.array_equal((hi + lo)[here], x[here]), (e, m0)


def test_two_fp16_numbers_hold_an_nf4_value():
    """level s likewise: two 11-bit numbers, but a level is a whole number of
    2^-15 only (the innermost is 0.042), so that below s = 2 (a whole number of
    2^-9 from there on) the product may hold bits below fp16's smallest step,
    2^-24."""
    import numpy as np
    import oracle as O
    lv = O.nf4_levels().astype(np.float64)
    s = np.arange(1, 0x7C00, dtype=np.uint16).view(np.float16).astype(np.float64)[:, None]
    x = lv * s
    hi = x.astype(np.float16).astype(np.float64)
    lo = (x - hi).astype(np.float16).astype(np.float64)
    off = np.abs(hi + lo - x)
    assert off.max() <= 2.0 ** -25
    assert np.array_equal(lv * 2.0 ** 15, np.rint(lv * 2.0 ** 15))
    assert not off[s[:, 0] >= 2.0].any()


def test_no_attention_instance_that_nothing_reaches():
    """The mma.sync form of kvq_extend_attn is built for axis-aware caches (4
    and 8 bits) at every head_dim, and for the other formats at 256 only."""
    import os
    import re
    import shutil
    import subprocess
    from quantized_kv_decode_gb300 import build
    build.build()
    obj = os.path.join(build.BUILD, "kvq_extend.cu.o")
    if shutil.which("nm") is None or not os.path.exists(obj):
        pytest.skip("no nm, or no object files")
    out = subprocess.run(["nm", "-C", obj], capture_output=True, text=True, check=True).stdout
    got = {(int(b), int(d)) for b, d in re.findall(r"extend_kernel<(\d+), (\d+)>", out)}
    assert got == {(2, 256), (16, 256)} | {(b, d) for b in (4, 8) for d in (64, 128, 256)}
