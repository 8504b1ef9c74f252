"""Sizes of the multi-adapter calls that are not served: the size queries answer 0 for what
the calls refuse, and a pool that no call takes is refused when it is made."""
import pytest
import torch

import bit_nf4_quantized_05_amd as qn
from bit_nf4_quantized_05_amd import _lib

QUERIES = [qn.multi_linear_fwd_workspace_bytes, qn.multi_linear_bwd_workspace_bytes]


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("d_seq", [1, 2, 64, 65, 100, 5000])
@pytest.mark.parametrize("d_out,d_in,r", [(64, 64, 1), (64, 64, 8), (4096, 4096, 8), (64, 64, 24), (64, 64, 272),
                                          (64, 64, 0), (32, 64, 16), (64, 32, 16), (32, 32, 16), (96, 128, 16),
                                          (128, 96, 16), (64, 0, 16), (0, 64, 16), (-64, 64, 16)])
def test_queries_answer_0_on_bad_sizes(query, d_seq, d_out, d_in, r):
    assert query(d_out, d_in, d_seq, r, 8) == 0


@pytest.mark.parametrize("query", QUERIES)
@pytest.mark.parametrize("d_out,d_in,d_seq,r,n", [
    (64, 64, 0, 16, 1), (64, 64, -5, 16, 1), (64, 64, 100, 16, 0), (64, 64, 100, 16, 1025),
    (1 << 20, 1 << 12, 10, 16, 1),                       # a weight whose bf16 copy reaches 4 GiB
    (64, 4096, 1 << 19, 16, 1), (4096, 64, 1 << 19, 16, 1),      # activations that do
    (64, 64, 1 << 23, 256, 4),                           # rank products that do
    (1 << 33, 64, (1 << 31) - 1, 256, 1000)])            # partial sums past 2^63 bytes
def test_queries_answer_0_on_sizes_past_the_limits(query, d_out, d_in, d_seq, r, n):
    assert query(d_out, d_in, d_seq, r, n) == 0


@pytest.mark.parametrize("query", QUERIES)
def test_queries_answer_up_to_the_limits(query):
    assert query(64, 64, 1, 16, 1) > 0 and query(64, 64, 65, 256, 1024) > 0
    assert query((1 << 20) - 64, 2048, 1, 16, 1) > 0     # 2 * 2^31 - 2^18 bytes of weight
    assert query(64, 4096, (1 << 19) - 1, 16, 1) > 0


def _pool(n, r, d_out=64, d_in=128):
    return qn.AdapterPool(torch.zeros(n, r, d_in, dtype=torch.bfloat16), torch.zeros(n, d_out, r, dtype=torch.bfloat16),
                          torch.zeros(n))


@pytest.mark.parametrize("n,r", [(3, 1), (3, 8), (3, 24), (3, 272), (3, 0), (0, 16), (1025, 16)])
def test_pools_that_no_call_takes(n, r):
    with pytest.raises(ValueError):
        _pool(n, r)


def test_pools_at_the_limits():
    assert _pool(1, 16).r == 16 and _pool(2, 256).r == 256 and _pool(1024, 16, 1, 1).n == 1024
    with pytest.raises(ValueError):
        qn.alloc_pool(1025, 16, 64, 64, "cpu")
    with pytest.raises(ValueError):
        qn.alloc_pool(0, 16, 64, 64, "cpu")


def test_limit_is_the_headers():
    text = open(_lib.LIB_PATH.rsplit("/", 2)[0] + "/include/qlora_nf4.h").read()
    assert f"#define QN_MULTI_MAX_ADAPTERS {_lib.MULTI_MAX_ADAPTERS}\n" in text


FAKE = 1 << 20


@pytest.mark.parametrize("d_out,d_in,d_seq,r,n", [(64, 64, 8, 8, 2), (64, 96, 100, 16, 2), (64, 64, 100, 16, 1025),
                                                  (1 << 20, 1 << 12, 10, 16, 1), (64, 4096, 1 << 19, 16, 1),
                                                  (64, 64, 1 << 23, 256, 4)])
def test_calls_refuse_what_the_queries_answer_0_to(d_out, d_in, d_seq, r, n):
    lib = _lib.lib()
    ptrs = (FAKE, FAKE, FAKE, FAKE)
    pool = (FAKE, FAKE, FAKE, n, r)
    assert lib.qlora_multi_fwd(*ptrs, d_out, d_in, 0, *pool, FAKE, d_in, d_seq, FAKE, FAKE, d_out, FAKE, 1 << 60, None) == -2
    assert lib.qlora_multi_bwd(*ptrs, d_out, d_in, 0, *pool, FAKE, d_in, FAKE, d_out, d_seq, FAKE, FAKE, d_in, FAKE, FAKE,
                               FAKE, 1 << 60, None) == -2


@pytest.mark.parametrize("d_out,d_in,r", [(11008, 4096, 64), (4096, 4096, 16), (256, 256, 16), (4096, 11008, 256), (64, 64, 256)])
@pytest.mark.parametrize("d_seq", [513, 700, 2000, 4096, 20000])
def test_backward_workspace_does_not_grow_with_the_pool(d_out, d_in, r, d_seq):
    """Partial gradients are written by adapters of more than one slice (at least 128 tokens)
    only: of c > 128 tokens ceil(c / 128) <= 2 c / 128 slices, 2 d_seq / 128 over all adapters,
    and at most 4 MB are set aside past them."""
    sizes = [qn.multi_linear_bwd_workspace_bytes(d_out, d_in, d_seq, r, n) for n in (1, 8, 100, 1024)]
    slot = 4 * (d_out + d_in) * r
    without = qn.multi_linear_bwd_workspace_bytes(d_out, d_in, 512, r, 1) * d_seq // 512      # all else is linear in d_seq at most
    for size in sizes:
        assert size <= without + 2 * d_seq // 128 * slot + (4 << 20) + 4096
    assert sizes[-1] - sizes[0] <= max(2 * d_seq // 128 * slot, 4 << 20)


def test_backward_workspace_of_one_token_more():
    """512 tokens need no partial gradients; one more costs at most 8 slots of them."""
    few, more = (qn.multi_linear_bwd_workspace_bytes(11008, 4096, m, 64, 1024) for m in (512, 513))
    assert more - few <= 8 * 4 * (11008 + 4096) * 64 + (1 << 20)
