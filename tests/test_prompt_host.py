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
