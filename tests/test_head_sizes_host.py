"""The head's size query beside its call, without a GPU: the vocabulary's pieces are as small as the
head's rows need, and the query answers 0 exactly where the call refuses the sizes. The calls get a
workspace that is too small, so that none starts."""
import pytest

from bit_nf4_quantized_05_amd import _lib

FAKE = 1 << 20


def query(vocab, d, m, nf4, grad):
    return _lib.lib().qlora_head_loss_workspace_bytes(vocab, d, m, int(nf4), int(grad))


def call(vocab, d, m, nf4, grad, ldw=None):
    head = (None, 0, FAKE, FAKE, FAKE, FAKE, 0) if nf4 else (FAKE, ldw or d, None, None, None, None, 0)
    return _lib.lib().qlora_head_loss(*head, vocab, d, FAKE, d, m, FAKE, None, FAKE, FAKE if grad else None, d, FAKE, 0, None)


# rows of 32768 and more, whose pieces of 65536 (32768) rows would reach 4 GiB
LONG = [(65536, 32768, 17), (65536, 32704, 17), (128000, 32768, 17), (128000, 65536, 5), (65536, 1 << 20, 3), (256, (1 << 23) - 64, 2),
        (1024, (1 << 23) - 64, 2), (64, 1 << 24, 2)]


@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("vocab,d,m", LONG)
def test_long_rows_are_taken_in_smaller_pieces(vocab, d, m, nf4, grad):
    assert query(vocab, d, m, nf4, grad) > 0
    assert call(vocab, d, m, nf4, grad) == -3


@pytest.mark.parametrize("nf4", [False, True])
@pytest.mark.parametrize("grad", [False, True])
@pytest.mark.parametrize("vocab,d,m", LONG + [(256, 1 << 23, 2), (64, 1 << 25, 2), (1024, 1 << 29, 1), (1024, 64, 1 << 23),
                                              (1024, 64, 1 << 24), (1024, 64, 1 << 25), (1024, 63, 8), (0, 64, 8)])
def test_query_agrees_with_the_call(vocab, d, m, nf4, grad):
    rc = call(vocab, d, m, nf4, grad)
    assert rc == -3 if query(vocab, d, m, nf4, grad) else rc in (-1, -2)


@pytest.mark.parametrize("grad", [False, True])
def test_a_strided_head_needs_no_more_and_is_refused_at_4_gib_per_256_rows(grad):
    for ldw in (64, 32768, 40000, 1 << 20, (1 << 23) - 8):
        assert call(66000, 64, 17, False, grad, ldw) == -3
    assert call(66000, 64, 17, False, grad, 1 << 23) == -2
