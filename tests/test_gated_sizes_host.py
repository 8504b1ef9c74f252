"""The gated block's size queries beside its calls, without a GPU: on both sides of each limit the
query answers 0 exactly where the call refuses the sizes. The calls get a workspace that is too
small, so that none starts."""
import pytest

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib

FAKE = 1 << 20
WEIGHT = [FAKE, FAKE, FAKE, FAKE]
ADAPTERS = [FAKE, FAKE, 1.0, FAKE, FAKE, 1.0]


def fwd(d_ff, d_in, m, r, keep):
    return _lib.lib().qlora_gated_fwd(*WEIGHT, *WEIGHT, d_ff, d_in, 0, *ADAPTERS, r, 0, FAKE, d_in, m, FAKE, d_ff,
                                      FAKE if keep else None, 2 * d_ff if keep else 0, FAKE, 0, None)


def bwd(d_ff, d_in, m, r):
    return _lib.lib().qlora_gated_bwd(*WEIGHT, *WEIGHT, d_ff, d_in, 0, *ADAPTERS, r, 0, FAKE, 2 * d_ff, FAKE, d_ff, m, FAKE,
                                      2 * d_ff, FAKE, d_in, FAKE, 0, None)


LIMIT = 1 << 31         # bf16 elements of an operand
# d_ff, d_in, tokens, rank: the limits of GU (and dGU), H, X, the rank products, both weights
SIZES = [(28672, 8192, 40000, 64), (11008, 4096, 100000, 16), (28672, 8192, (LIMIT - 1) // 57344, 64),
         (28672, 8192, LIMIT // 57344 + 1, 64), (28672, 8192, (LIMIT - 1) // 28672, 64), (28672, 8192, LIMIT // 28672 + 1, 64),
         (64, 4096, LIMIT // 4096 - 1, 8), (64, 4096, LIMIT // 4096, 8), (64, 64, (LIMIT - 1) // 512, 256),
         (64, 64, LIMIT // 512, 256), (64, 64, LIMIT // 128 - 1, 0), (64, 64, LIMIT // 128, 0), (64, 64, LIMIT // 64 - 1, 0),
         (64, 64, LIMIT // 64, 0), (64, (LIMIT - 1) // 128 // 64 * 64, 5, 16), (64, LIMIT // 128, 5, 16),
         (64, 64, 1, 257), (96, 64, 1, 0), (64, 64, 0, 0), (11008, 4096, 1, 16), (11008, 4096, 2048, 64)]


@pytest.mark.parametrize("d_ff,d_in,m,r", SIZES)
def test_queries_agree_with_the_calls(d_ff, d_in, m, r):
    need = qn.gated_fwd_workspace_bytes(d_ff, d_in, m, r)
    rc = fwd(d_ff, d_in, m, r, keep=False)
    assert rc == -3 if need else rc in (-1, -2)
    # keeping G and U adds the limit of GU alone
    kept = fwd(d_ff, d_in, m, r, keep=True)
    assert kept == (-2 if rc == -3 and 2 * d_ff * m >= LIMIT else rc)
    rc = bwd(d_ff, d_in, m, r)
    assert rc == -3 if qn.gated_bwd_workspace_bytes(d_ff, d_in, m, r) else rc in (-1, -2)


def test_long_batches_that_keep_nothing_have_a_workspace():
    assert qn.gated_fwd_workspace_bytes(28672, 8192, 40000, 64) > 4 * 28672 * 8192
    assert qn.gated_fwd_workspace_bytes(11008, 4096, 100000, 16) > 4 * 11008 * 4096


def test_the_gradient_in_place_at_another_stride_is_refused():
    def call(GU, ldgu, dGU, lddgu, m):
        return _lib.lib().qlora_gated_bwd(*WEIGHT, *WEIGHT, 64, 128, 0, *ADAPTERS, 8, 0, GU, ldgu, FAKE, 64, m, dGU, lddgu, FAKE,
                                          128, FAKE, 0, None)

    # -3: the sizes and strides are taken, the workspace is too small
    assert call(2 * FAKE, 128, 2 * FAKE, 128, 3) == -3 and call(2 * FAKE, 160, 2 * FAKE, 160, 3) == -3
    assert call(2 * FAKE, 160, 2 * FAKE, 128, 3) == -1 and call(2 * FAKE, 128, 2 * FAKE, 160, 3) == -1
    assert call(2 * FAKE, 160, 2 * FAKE, 128, 1) == -3 and call(2 * FAKE, 160, 3 * FAKE, 128, 3) == -3
