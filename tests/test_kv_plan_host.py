"""The calls of the GPU tests reach every form of kv_attention."""

import os

import pytest

import bit_gemm_amd as nv
from kv_plan_cases import BOTH_WAYS, CALLS, JOINED, MANY, WINDOWS, check_plan


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not os.path.exists(nv.LIB_PATH):
        from bit_gemm_amd import build
        build.build()


@pytest.mark.parametrize("call", CALLS, ids=str)
def test_call_takes_the_form_it_names(call):
    check_plan(call)


def test_every_kernel_and_mask_is_there():
    """The seven kernels of head_dim and block size: windows on whole and on split contexts, split contexts that every
    token sees, both forms of the join, more than 64 sequences."""
    paths = {(64, 16), (64, 32), (128, 16), (128, 32), (128, 256), (256, 16), (256, 128)}

    def of(calls, **want):
        return {(c.d, c.rows) for c in calls if all(getattr(c, k) == v for k, v in want.items())}

    assert of(WINDOWS, split=False) == paths and of(WINDOWS, split=True) == paths
    assert of(BOTH_WAYS, split=True, causal=False) == paths
    assert of(JOINED, wide_join=True) == paths
    assert all(c.split and len(c.lens) > 64 for c in MANY) and {c.d for c in MANY} == {64, 128, 256}
    for c in WINDOWS:
        assert c.window % 32 and c.window < max(c.lens)
