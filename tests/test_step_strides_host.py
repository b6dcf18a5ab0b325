"""Strides that no address is made of are not looked at. CPU only: what is
refused is the argument after them."""

import ctypes

import pytest

import linear_attention_state_chunked_gb300 as L
from tests.test_step_host import append_args, attn_args, cache_desc, refused


@pytest.mark.parametrize("stride", [2, 8, 520, -256, 0])
def test_the_token_stride_of_one_token(stride):
    c = cache_desc()
    a = append_args(n=1, token_stride=stride, page_table_stride=4)
    refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(a), None), L.LIN_EINVAL, "page_table_stride")
    a = attn_args(n_q=1, token_stride=stride, page_table_stride=4)
    refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), None, 0, None), L.LIN_EINVAL,
            "page_table_stride")


@pytest.mark.parametrize("stride", [2, 8, 520, -256, 0])
def test_the_request_stride_of_one_request(stride):
    c, a = cache_desc(), attn_args(batch=1, req_stride=stride)
    refused(L.lib.lin_state_attn_decode(ctypes.byref(c), ctypes.byref(a), None, 0, None), L.LIN_EWORKSPACE, "workspace")


@pytest.mark.parametrize("axis,count", [("layer_stride", dict(layers=1)), ("page_stride", dict(pages=1)),
                                        ("token_stride", dict(ps=1)), ("head_stride", dict(H=1))])
@pytest.mark.parametrize("stride", [2, 520, -256, 0])
def test_a_cache_axis_of_one(axis, count, stride):
    c = cache_desc(**count)
    setattr(c, axis, stride)
    a = append_args(layer=5)
    refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(a), None), L.LIN_EINVAL, "layer 5")


def test_strides_that_are_used_still_have_to_fit():
    c = cache_desc()
    for kw in (dict(n=2, token_stride=520), dict(n=2, token_stride=-512), dict(n=1, req_stride=1544)):
        refused(L.lib.lin_state_kv_append(ctypes.byref(c), ctypes.byref(append_args(**kw)), None), L.LIN_EINVAL,
                "multiples of 16")
