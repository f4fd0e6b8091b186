"""pkv_collect_errors' refusals, which come before any CUDA call, and the binding's name for what it collects."""
import pytest

import paged_kv_gqa_17_b200 as pkg
from paged_kv_gqa_17_b200 import binding as bd


@pytest.fixture(scope="module")
def L():
    from paged_kv_gqa_17_b200 import build

    build.build()
    return bd.lib()


def test_a_workspace_that_is_none_or_misaligned_is_refused(L):
    assert L.pkv_collect_errors(None, None) == -1
    assert L.pkv_collect_errors(257, None) == -2


def test_the_package_offers_the_status(L):
    assert pkg.unplanned_status is bd.unplanned_status
