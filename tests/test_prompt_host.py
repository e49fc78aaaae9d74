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
