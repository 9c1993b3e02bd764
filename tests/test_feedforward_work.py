"""What the gated block's gradient asks for in working memory."""
import pytest

import exact_range_similarity_amd as ersj

FAKE = 0x10000  # only its alignment is looked at


def grad_work(x, kind, n, dim, hidden, ld=None):
    ld = ld or dim
    return ersj.lib().ersj_gated_grad_work(x, kind, n, dim, ld, FAKE, dim, FAKE, dim, hidden, 1, 0, 0)


@pytest.mark.parametrize("n,dim,hidden", [(256, 64, 128), (4096, 100, 72), (1 << 20, 384, 1024)])
def test_held_rows_take_one_plane(n, dim, hidden):
    # 32-bit rows are laid out as three bf16 planes; what codes stand for is one
    plane = n * -(-dim // 8) * 8 * 2
    assert grad_work(FAKE, 0, n, dim, hidden) - grad_work(None, 0, n, dim, hidden) == 2 * plane
    # 16-bit rows are read in place, and unpacked to one plane
    for kind in (1, 2):
        inplace = 0 if dim % 8 == 0 else plane
        assert grad_work(None, kind, n, dim, hidden) - grad_work(FAKE, kind, n, dim, hidden) == plane - inplace
