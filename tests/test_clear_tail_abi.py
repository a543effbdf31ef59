"""KDN_CLEAR_TAIL at the C ABI without a GPU: which calls take it and which refuse it."""
import os

import pytest
import torch

import kalman_delta_rule_amd as kda

P, G = 1 << 20, 1 << 32
TAIL = 0x400


@pytest.fixture(scope="module")
def L():
    from kalman_delta_rule_amd import _lib
    if not os.path.exists(_lib.LIB_PATH):
        from kalman_delta_rule_amd import build
        build.build_library()
    return _lib.lib()


def test_the_value():
    assert kda.api.KDN_CLEAR_TAIL == TAIL


@pytest.mark.skipif(torch.cuda.is_available(),
                    reason="stand-in pointers are only used where no GPU is visible")
@pytest.mark.parametrize("io", [0, 1])
def test_calls_that_take_it(L, io):
    msg = lambda: L.kdn_last_error_message().decode()
    f, t = io | TAIL, io | TAIL | 2
    # taken: the next refusal is of another argument
    assert L.kdn_conv_fwd(1, 8, 64, 7, f, 0, P, 64, P + G, None, None, None, 0, P + 2 * G, None, None) == -2
    assert "taps" in msg()
    assert L.kdn_conv_bwd(1, 8, 64, 7, f, 0, P, P, 64, P, None, None, None, 0, None, P, P, None, None, None, 0,
                          None) == -2
    assert "taps" in msg()
    assert L.kdn_rec_fwd(2, 8, 64, f, 5, 0, P, 64, P + G, 64, None, None, 0, P, None, None, None, 0, None) == -1
    assert "gate" in msg()
    assert L.kdn_rec_bwd(2, 8, 64, f, 5, 0, P, P, 64, P, 64, P, None, None, 0, None, P, P, None, None, 0, None) == -1
    assert "gate" in msg()
    # not beside other bits
    assert L.kdn_conv_fwd(1, 8, 64, 4, t, 0, P, 64, P + G, None, None, None, 0, P + 2 * G, None, None) == -1
    assert "io_dtype" in msg() and str(t) in msg()
    assert L.kdn_rec_fwd(2, 8, 64, t, 1, 0, P, 64, P + G, 64, None, None, 0, P, None, None, None, 0, None) == -1
    assert "io_dtype" in msg() and str(t) in msg()
    # no sequences, no tail
    assert L.kdn_layer_norm_fwd(4, 64, f, 1e-5, P, 64, None, None, P + G, None, None, None) == -1
    assert "io_dtype" in msg()
    assert L.kdn_conv_step(4, 64, 4, f, 0, P, 64, P + G, None, P + 3 * G, P + 2 * G, None) == -1
    assert "io_dtype" in msg()
    assert L.kdn_rec_step(4, 64, f, 1, 0, P, 64, P + G, 64, P + 2 * G, P + 3 * G, None) == -1
    assert "io_dtype" in msg()
