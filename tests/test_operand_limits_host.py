"""Row strides whose operand reaches 4 GiB are refused however large they are: the kernels
address an operand with 32-bit byte offsets. (Every call has too small a workspace, so a
stride that got past the check would show as -3.)"""
import pytest

from bit_nf4_quantized_05_amd import _lib

FAKE = 1 << 20
# (tokens, row stride): at the limit, far past it, and where 2 * tokens * stride leaves 64 bits
PAST = [(1 << 20, 2048), (100, 1 << 31), (1, 1 << 31), ((1 << 31) - 1, (1 << 32) - 8), ((1 << 31) - 1, 1 << 33), (4, 1 << 62),
        (1 << 30, 1 << 34), (8, 1 << 60)]
UNDER = [(1 << 20, 2040), (1, (1 << 31) - 8), (100, 64)]


def _multi_fwd(m, ld, which):
    return _lib.lib().qlora_multi_fwd(FAKE, FAKE, FAKE, FAKE, 64, 64, 0, FAKE, FAKE, FAKE, 2, 16, FAKE,
                                      ld if which == 0 else 64, m, FAKE, FAKE, ld if which == 1 else 64, FAKE, 0, None)


def _multi_bwd(m, ld, which):
    return _lib.lib().qlora_multi_bwd(FAKE, FAKE, FAKE, FAKE, 64, 64, 0, FAKE, FAKE, FAKE, 2, 16, FAKE,
                                      ld if which == 0 else 64, FAKE, ld if which == 1 else 64, m, FAKE, FAKE,
                                      ld if which == 2 else 64, FAKE, FAKE, FAKE, 0, None)


def _linear(name):
    def call(m, ld, which):
        return getattr(_lib.lib(), name)(FAKE, FAKE, FAKE, FAKE, 64, 64, 0, FAKE, FAKE, 16, 1.0, FAKE,
                                         ld if which == 0 else 64, m, FAKE, ld if which == 1 else 64, FAKE, 0, None)
    return call


def _lora_grads(m, ld, which):
    return _lib.lib().qlora_lora_grads(FAKE, FAKE, 16, 1.0, FAKE, ld if which == 0 else 64, FAKE, ld if which == 1 else 64,
                                       64, 64, m, FAKE, FAKE, FAKE, 0, None)


CALLS = {"qlora_multi_fwd": (_multi_fwd, 2), "qlora_multi_bwd": (_multi_bwd, 3),
         "qlora_linear_fwd_ex": (_linear("qlora_linear_fwd_ex"), 2),
         "qlora_linear_bwd_x_ex": (_linear("qlora_linear_bwd_x_ex"), 2), "qlora_lora_grads": (_lora_grads, 2)}


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m,ld", PAST)
def test_refused(name, m, ld):
    call, operands = CALLS[name]
    for which in range(operands):
        assert call(m, ld, which) == -2, which
        assert b"4 GiB" in _lib.lib().qn_last_error()


@pytest.mark.parametrize("name", CALLS)
@pytest.mark.parametrize("m,ld", UNDER)
def test_taken_up_to_the_limit(name, m, ld):
    call, operands = CALLS[name]
    for which in range(operands):
        assert call(m, ld, which) == -3, which
