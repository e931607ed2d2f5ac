"""bdsa_cache_fork on many rows of few pages: the counts of rows that every CTA sums
take more shared memory than a kernel has without asking for it."""
import pytest

from test_gpu_cache import Fork

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bs,rows,width,free", [
    (11000, 3000, 1, None), (16000, 9000, 1, 2), (3000, 16000, 1, None), (16384, 16384, 1, None),
    (5000, 6300, 2, None), (5600, 5700, 1, None)])
def test_fork_many_narrow_rows(bs, rows, width, free):
    f = Fork(bs, rows, width, 16, bs, free=free, share=0.6)
    if free is None:
        f.check()
    else:  # the ring runs out
        f.check(bad=True)
