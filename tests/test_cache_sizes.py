"""Sizes that the calls on the paged cache take and refuse at the ends of their ranges, on the host
(no GPU: the checks touch no device state)."""
import os

import pytest

FAKE = 1 << 40  # an address that is never dereferenced


@pytest.fixture(scope="module")
def B():
    from draft_verification_amd import binding, build
    if not os.path.exists(binding.LIB_PATH):
        build.build()
    return binding


@pytest.fixture(scope="module")
def cfg(B):
    return B.Config(8, 8, 1000, B.SV_BF16, 0)


def copies(B, **more):
    d = dict(copies=FAKE, pools=FAKE, n_pools=3, pool_stride=100 * 512, page_stride=512, page_bytes=512, n_pages=100)
    d.update(more)
    return B.make_pages_copy_args(5, **d)


@pytest.mark.parametrize("pool_stride", [0, -1, 8, (1 << 46) + 16, 1 << 62, -(1 << 63)])
def test_the_stride_of_one_pool_is_not_looked_at(B, cfg, pool_stride):
    assert B.pages_copy_check(cfg, copies(B, n_pools=1, pool_stride=pool_stride)) == B.SV_OK
    assert B.pages_copy_check(cfg, copies(B, n_pools=2, pool_stride=pool_stride)) != B.SV_OK


@pytest.mark.parametrize("n_pages,page_stride", [(1 << 24, 1 << 40), ((1 << 24) - 1, 1 << 40), (1 << 23, 1 << 40),
                                                 (12345678, 1 << 40), (1 << 24, (1 << 39) + 16), (1 << 24, (1 << 22) + 16)])
def test_pools_that_overlap_are_refused_whatever_their_pages_take(B, cfg, n_pages, page_stride):
    """n_pages * page_stride may lie past 63 bits."""
    for pool_stride in (0, 512, page_stride, 1 << 46):
        args = copies(B, n_pages=n_pages, page_stride=page_stride, pool_stride=pool_stride)
        assert B.pages_copy_check(cfg, args) == B.SV_EINVAL
    args = copies(B, n_pages=1 << 24, page_stride=1 << 22, pool_stride=1 << 46)  # that just fit
    assert B.pages_copy_check(cfg, args) == B.SV_OK
