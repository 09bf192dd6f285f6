"""The bounded waits of the attention kernels over the 4-bit cache: in a build
whose CG_TEST_ATTN_TIMEOUT gives chosen waits up at once (cg_attention.h), with
copies and products in flight that are all valid, a call reports CG_ERR_TIMEOUT
and ends its blocks cleanly, and the product library then gives the same bits as
before."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

from kv_cache_compression_03_gb300 import build, cachegen as cg  # noqa: E402

from test_gpu_int4 import _dev, _ints, _rand  # noqa: E402


@pytest.fixture(scope="module")
def variant():
    return build.build_test_variant("test_cg_test_attn_timeout", ["CG_TEST_ATTN_TIMEOUT"])


# Single tokens: every warp gives up its second step, with more behind it than its ring holds.
# 64 and 16 rows of a KV head, 256: the softmax, an expanding warp, the copying warp or the
# issuing thread, by the block; one row tile in turns, and two, both cut into pieces.
@pytest.mark.parametrize("nq,ratio", [(1, 4), (1, 16), (16, 4), (64, 4)])
@pytest.mark.parametrize("dim,group", [(128, 32), (64, 64)])
def test_a_wait_that_runs_out_is_reported(variant, nq, ratio, dim, group):
    rng = np.random.default_rng(nq)
    heads, page, n, requests = 2, 64, 40000, 4
    pages = -(-n // page)
    cache = cg.Int4Cache(1, pages, page, heads, dim, group)
    x = _dev(_rand(rng, n, heads, dim))
    cache.store(x, x, _ints(np.arange(n)))
    args = (_dev(_rand(rng, requests * nq, heads * ratio, dim)), _ints(np.arange(requests + 1) * nq),
            _ints([n - 7 * r for r in range(requests)]), _ints([np.arange(pages)] * requests))
    before = cache.attention(*args, max_q_len=nq)
    cache.check()
    with cg.use_library(variant):
        for _ in range(3):
            cache.attention(*args, max_q_len=nq)
            with pytest.raises(cg.CacheGenError) as e:
                cache.check()
            assert e.value.status == cg.CG_ERR_TIMEOUT
    again = cache.attention(*args, max_q_len=nq)
    cache.check()
    assert torch.equal(before, again)
