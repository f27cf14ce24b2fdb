"""The paged-attention calls on the host, without a GPU: sizes and strides at
their limits, arguments that share a buffer."""

import ctypes

import pytest

from linear_attention_ssm_step_gb300 import _build, kda
from test_paged_host import UNSUPPORTED, fake_attention, fake_plan, fake_rope, no_gpu, put

pytestmark = no_gpu


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return kda.load_library()


def status(lib, p):
    """Of a call with these fake addresses. KDA_ELAUNCH: it passed the checks, and found no device."""
    if isinstance(p, kda.KdaPlanParams):
        return lib.kda_paged_plan(ctypes.byref(p), None)
    if isinstance(p, kda.KdaRopeParams):
        return lib.kda_rope_append(ctypes.byref(p), None)
    return lib.kda_paged_attention(ctypes.byref(p), 1 << 45, 1 << 30, None)


# ---------------------------------------------------------------- sizes

@pytest.mark.parametrize("tensor", ["q", "k", "v", "q_out"])
def test_rope_rows_whose_span_passes_64_bits(lib, tensor):
    """2^31 - 1 rows 2^39 elements apart: the span, 2^70, must not wrap in the check of what overlaps what."""
    p = fake_rope()
    p.num_tokens = 2 ** 31 - 1
    put("q_out_b_stride" if tensor == "q_out" else tensor + ".b_stride", 1 << 39)(p)
    assert status(lib, p) == UNSUPPORTED
    assert f"{tensor} has rows that span" in kda.kda_last_error()


@pytest.mark.parametrize("tensor", ["q", "out"])
def test_attention_rows_whose_span_passes_64_bits(lib, tensor):
    p = fake_attention()
    p.num_tokens = 2 ** 31 // 4 - 1
    put("out_b_stride" if tensor == "out" else "q.b_stride", 1 << 39)(p)
    assert status(lib, p) == UNSUPPORTED
    assert f"{tensor} has rows that span" in kda.kda_last_error()


def test_a_span_that_wraps_to_nothing_hides_no_overlap(lib):
    """2^31 - 1 rows of 2^33 elements (2^64 of them, less two rows): wrapped, an extent that ends before it begins, and
    in which q_out, although it stands there, does not lie."""
    p = fake_rope()
    p.num_tokens = 2 ** 31 - 1
    p.q.b_stride = 1 << 33
    assert status(lib, p) == UNSUPPORTED


@pytest.mark.parametrize("make", [fake_plan, fake_attention])
def test_table_stride_past_40_bits(lib, make):
    p = make()
    p.table_stride = 1 << 61
    assert status(lib, p) == UNSUPPORTED
    assert "table_stride" in kda.kda_last_error()
    p.num_requests, p.table_stride = 1, 1 << 61  # a stride that is not used
    if isinstance(p, kda.KdaPlanParams):
        assert status(lib, p) == kda.KDA_ELAUNCH
