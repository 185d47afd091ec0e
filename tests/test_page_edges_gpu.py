"""The paged 8-bit cache at the edges of what its calls take, against its definition in 64 bits
(tests/page_oracle.py)."""
import pytest
import torch

from tests.test_page_gpu import BF16, F32, Step

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("news", [None, [100, 3], [4, 3]])
@pytest.mark.parametrize("bad", [float("inf"), float("-inf")])
@pytest.mark.parametrize("code", [0x38, 0xB8])  # 1, -1
def test_attend_infinite_query_whose_scores_are_all_minus_infinity(dtype, news, bad, code):
    n0 = news[0] if news else 1
    s = Step([n0, 60], news, dtype=dtype, base=0.0, seed=37)
    s.pools[0].view(torch.uint8)[s.table[0, 0], 1, 0, 10] = code
    good = s.cache.attend(s.q, *s.pools)
    q = s.q.clone()
    q[0, 5, 10] = bad  # row 0 sees token 0 only; head 5 reads KV head 1
    out = s.cache.attend(q, *s.pools)
    torch.cuda.synchronize()
    assert out[0, 5].isnan().all()
    out[0, 5], good[0, 5] = 0, 0
    assert torch.equal(out, good)
