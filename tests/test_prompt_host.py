"""Prompt operators, host side: refusals before any launch, the binding's checks, the
oracle's pins and the frequencies. CPU only."""

import ctypes
import math

import numpy as np
import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from linear_attention_state_chunked_gb300 import prompt
from oracle import lin_prompt_oracle as O
from oracle import lin_step_oracle as S
from tests.test_step_devices_host import Said, SaidOther
from tests.test_step_host import FAKE, cache_desc, refused

BF = torch.bfloat16


def filled(a, defaults, kw):
    for k, v in {**defaults, **kw}.items():
        setattr(a, k, v)
    return a


def plan_args(**kw):
    return filled(L.KVPlanArgsT(), dict(batch=3, n=2, tokens=6, page_size=4, num_pages=9, max_pages=5, page_table_stride=5,
                                        length=FAKE, page_table=FAKE, kv_len=FAKE + 64), kw)


def rope_args(**kw):
    return filled(L.RopeArgsT(), dict(tokens=4, num_q_heads=4, num_k_heads=2, head_dim=128, rot_dim=64, dtype=L.LIN_BF16,
                                      scale=1.0, q=FAKE, k=FAKE, v=FAKE, q_out=FAKE + 4096, q_stride=2048, k_stride=2048,
                                      v_stride=2048, q_out_stride=1024, position=FAKE, inv_freq=FAKE, slot=FAKE), kw)


def chunk_args(**kw):
    return filled(L.AttnChunkArgsT(), dict(batch=3, tokens=20, num_q_heads=8, out_dtype=L.LIN_BF16, max_pages=5, scale=0.1,
                                           q=FAKE, out=FAKE, token_stride=2048, page_table=FAKE, page_table_stride=5,
                                           cu_seqlens=FAKE, kv_len=FAKE), kw)


@pytest.mark.parametrize("change,code,text", [
    (dict(batch=-1), L.LIN_EINVAL, "negative"),
    (dict(tokens=-1), L.LIN_EINVAL, "negative"),
    (dict(num_free=-1), L.LIN_EINVAL, "negative"),
    (dict(page_size=0), L.LIN_EINVAL, "positive"),
    (dict(num_pages=0), L.LIN_EINVAL, "positive"),
    (dict(n=-1), L.LIN_EINVAL, "negative n"),
    (dict(parent=FAKE, n_new=FAKE), L.LIN_EINVAL, "exclude"),
    (dict(parent=FAKE, n=33), L.LIN_EUNSUPPORTED, "32 drafts"),
    (dict(length=None), L.LIN_EINVAL, "NULL"),
    (dict(page_table=None), L.LIN_EINVAL, "NULL"),
    (dict(page_table_stride=4), L.LIN_EINVAL, "page_table_stride"),
    (dict(kv_len=FAKE), L.LIN_EINVAL, "kv_len must not be"),
    (dict(n_new=FAKE + 64), L.LIN_EINVAL, "kv_len must not be"),
])
def test_plan_refusals(change, code, text):
    refused(L.lib.lin_state_kv_plan(ctypes.byref(plan_args(**change)), None), code, text)


def test_plan_batches_past_its_arithmetic_are_refused():
    refused(L.lib.lin_state_kv_plan(ctypes.byref(plan_args(batch=(1 << 30) + 1)), None), L.LIN_EUNSUPPORTED, "batch")


@pytest.mark.parametrize("change,code,text", [
    (dict(tokens=-1), L.LIN_EINVAL, "negative"),
    (dict(dtype=5), L.LIN_EINVAL, "dtype"),
    (dict(head_dim=100), L.LIN_EUNSUPPORTED, "multiple of 8"),
    (dict(head_dim=264), L.LIN_EUNSUPPORTED, "up to 256"),
    (dict(rot_dim=63), L.LIN_EINVAL, "rot_dim"),
    (dict(rot_dim=130), L.LIN_EINVAL, "rot_dim"),
    (dict(rot_dim=0), L.LIN_EINVAL, "rot_dim"),
    (dict(layer=2), L.LIN_EINVAL, "layer"),
    (dict(num_k_heads=3), L.LIN_EINVAL, "the cache has other"),
    (dict(dtype=L.LIN_F32), L.LIN_EINVAL, "the cache has other"),
    (dict(position=None), L.LIN_EINVAL, "NULL"),
    (dict(slot=None), L.LIN_EINVAL, "NULL"),
    (dict(v=None), L.LIN_EINVAL, "NULL"),
    (dict(q=FAKE + 8), L.LIN_EINVAL, "aligned"),
    (dict(k_stride=500), L.LIN_EINVAL, "rope: k"),
    (dict(q_stride=512), L.LIN_EINVAL, "rope: q"),
    (dict(q_out=FAKE), L.LIN_EINVAL, "in its input's place"),
])
def test_rope_refusals(change, code, text):
    c = cache_desc()
    refused(L.lib.lin_state_rope(ctypes.byref(c), ctypes.byref(rope_args(**change)), None), code, text)


def test_rope_with_nothing_to_write():
    refused(L.lib.lin_state_rope(None, ctypes.byref(rope_args(q_out=None)), None), L.LIN_EINVAL, "nothing to write")
    assert L.lib.lin_state_rope(None, ctypes.byref(rope_args(tokens=0)), None) == L.LIN_OK


@pytest.mark.parametrize("change,code,text", [
    (dict(layer=-1), L.LIN_EINVAL, "layer"),
    (dict(batch=65536), L.LIN_EINVAL, "batch"),
    (dict(tokens=-1), L.LIN_EINVAL, "tokens"),
    (dict(num_q_heads=7), L.LIN_EINVAL, "multiple"),
    (dict(num_q_heads=65538), L.LIN_EUNSUPPORTED, "65536"),
    (dict(out_dtype=9), L.LIN_EINVAL, "out_dtype"),
    (dict(max_pages=-1), L.LIN_EINVAL, "max_pages"),
    (dict(q=None), L.LIN_EINVAL, "NULL"),
    (dict(cu_seqlens=None), L.LIN_EINVAL, "NULL"),
    (dict(out=FAKE + 8), L.LIN_EINVAL, "aligned"),
    (dict(token_stride=1024), L.LIN_EINVAL, "token stride"),
    (dict(page_table_stride=4), L.LIN_EINVAL, "page_table_stride"),
    (dict(), L.LIN_EWORKSPACE, "workspace"),
])
def test_chunk_refusals(change, code, text):
    c = cache_desc()
    refused(L.lib.lin_state_attn_chunk(ctypes.byref(c), ctypes.byref(chunk_args(**change)), None, 0, None), code, text)


def test_chunk_empty_calls_and_workspaces():
    c = cache_desc()
    size = lambda **kw: L.lib.lin_state_attn_chunk_workspace(ctypes.byref(c), ctypes.byref(chunk_args(**kw)))  # noqa: E731
    for kw in (dict(batch=0), dict(tokens=0)):
        assert L.lib.lin_state_attn_chunk(ctypes.byref(c), ctypes.byref(chunk_args(**kw)), None, 0, None) == L.LIN_OK
        assert size(**kw) == 0
    assert size(num_q_heads=7) == 0
    # one sized for the largest call serves the smaller ones, and either output type
    most = size(batch=100, tokens=5000, num_q_heads=64, max_pages=500)
    for kw in (dict(), dict(batch=1, tokens=1), dict(tokens=400, out_dtype=L.LIN_F32), dict(num_q_heads=64)):
        assert 0 < size(**kw) <= most
    refused(L.lib.lin_state_attn_chunk(ctypes.byref(c), ctypes.byref(chunk_args()), FAKE + 8, most, None), L.LIN_EINVAL, "aligned")


# ---- the binding -----------------------------------------------------------------------------

class Reached(Exception):
    pass


@pytest.fixture
def no_launch(monkeypatch):
    def reached(*args):
        raise Reached

    for name in ("_call_plan", "_call_rope", "_call_chunk"):
        monkeypatch.setattr(prompt, name, reached)
    from linear_attention_state_chunked_gb300 import step
    monkeypatch.setattr(step, "_current_device", lambda: 0)
    monkeypatch.setattr(step, "_raw_stream", lambda device: 0)


def call(which):
    """(function, keyword tensors, the rest) of a call that would be launched."""
    i32 = dict(dtype=torch.int32)
    k = torch.zeros((1, 4, 8, 2, 64), dtype=BF)
    if which == "plan":
        t = dict(length=torch.zeros(3, **i32), n_new=torch.zeros(3, **i32), page_table=torch.zeros((3, 4), **i32),
                 free_pages=torch.zeros(5, **i32), cu_seqlens=torch.zeros(4, **i32), kv_len=torch.zeros(3, **i32),
                 position=torch.zeros(6, **i32), slot=torch.zeros(6, dtype=torch.int64), taken=torch.zeros(1, **i32),
                 status=torch.zeros(1, **i32))
        return L.lin_state_kv_plan, t, dict(page_size=8, num_pages=4)
    rows = torch.zeros((6, 2, 64), dtype=BF)
    if which == "rope":
        t = dict(cache_k=k, cache_v=k.clone(), q=torch.zeros((6, 4, 64), dtype=BF), q_out=torch.zeros((6, 4, 64), dtype=BF),
                 k=rows, k_out=rows.clone(), v=rows.clone(), position=torch.zeros(6, **i32), inv_freq=torch.zeros(32),
                 slot=torch.zeros(6, dtype=torch.int64), status=torch.zeros(1, **i32))
        return L.lin_state_rope, t, {}
    t = dict(cache_k=k, cache_v=k.clone(), q=torch.zeros((6, 4, 64), dtype=BF), out=torch.zeros((6, 4, 64), dtype=BF),
             page_table=torch.zeros((3, 4), **i32), cu_seqlens=torch.zeros(4, **i32), kv_len=torch.zeros(3, **i32),
             status=torch.zeros(1, **i32), workspace=torch.zeros(1 << 10, dtype=torch.uint8))
    return L.lin_state_attn_chunk, t, dict(layer=0)


def run(which, change=lambda name, t: t):
    fn, t, rest = call(which)
    t = {n: change(n, x.as_subclass(Said)) for n, x in t.items()}
    if "cache_k" in t:
        ck, cv = t.pop("cache_k"), t.pop("cache_v")
        return fn(L.KVCache(1, 4, 8, 2, 64, k=ck, v=cv), **t, **rest)
    return fn(**t, **rest)


@pytest.mark.parametrize("which", ["plan", "rope", "chunk"])
def test_a_call_on_its_gpu_is_made(which, no_launch):
    with pytest.raises(Reached):
        run(which)


@pytest.mark.parametrize("which,name", [(w, n) for w in ("plan", "rope", "chunk") for n in call(w)[1] if not n.startswith("cache")])
@pytest.mark.parametrize("kind", ["cpu", "cuda:1"])
def test_tensors_elsewhere_are_refused(which, name, kind, no_launch):
    def change(n, t):
        if n != name:
            return t
        return t.as_subclass(SaidOther) if kind == "cuda:1" else t.as_subclass(torch.Tensor)

    with pytest.raises(ValueError, match="cuda|CUDA"):
        run(which, change)


@pytest.mark.parametrize("which,name,bad", [
    ("plan", "n_new", lambda t: t[:2]), ("plan", "cu_seqlens", lambda t: t[:3]), ("plan", "slot", lambda t: t.int()),
    ("plan", "length", lambda t: t[None]), ("plan", "page_table", lambda t: t[:2]), ("plan", "kv_len", lambda t: t.long()),
    ("rope", "k", lambda t: t[:5]), ("rope", "q_out", lambda t: t[:, :2]), ("rope", "v", lambda t: t[:, :1]),
    ("rope", "inv_freq", lambda t: t.double()), ("rope", "position", lambda t: t[:5]), ("rope", "slot", lambda t: t.int()),
    ("rope", "k", lambda t: t.float()), ("rope", "q", lambda t: t.transpose(1, 2).contiguous().transpose(1, 2)),
    ("chunk", "q", lambda t: t[0]), ("chunk", "out", lambda t: t[:5]), ("chunk", "cu_seqlens", lambda t: t[:3]),
    ("chunk", "kv_len", lambda t: t.long()), ("chunk", "page_table", lambda t: t[:2]), ("chunk", "q", lambda t: t.float()),
    ("chunk", "workspace", lambda t: t[::2]),
])
def test_shapes_and_types_are_refused(which, name, bad, no_launch):
    with pytest.raises(ValueError):
        run(which, lambda n, t: bad(t) if n == name else t)


def test_rope_and_plan_arguments_that_go_together(no_launch):
    fn, t, _ = call("rope")
    t = {n: x.as_subclass(Said) for n, x in t.items()}
    cache = L.KVCache(1, 4, 8, 2, 64, k=t.pop("cache_k"), v=t.pop("cache_v"))
    with pytest.raises(ValueError, match="needs k, v and slot"):
        fn(cache, **{k: v for k, v in t.items() if k != "slot"})
    with pytest.raises(ValueError, match="one at least"):
        fn(position=t["position"], inv_freq=t["inv_freq"])
    fn, t, rest = call("plan")
    t = {n: x.as_subclass(Said) for n, x in t.items() if n not in ("position", "slot")}
    with pytest.raises(ValueError, match="tokens"):
        fn(**t, **rest)


# ---- frequencies and the oracle -------------------------------------------------------------

def test_frequencies():
    f, scale = L.rope_frequencies(64, 500.0, device="cpu")
    assert scale == 1.0 and f.dtype == torch.float32
    assert torch.allclose(f.double(), 500.0 ** (-torch.arange(0, 64, 2).double() / 64), rtol=1e-7)
    g, _ = L.rope_frequencies(64, 500.0, linear=4.0, device="cpu")
    assert torch.allclose(g * 4, f)
    g, _ = L.rope_frequencies(64, 500.0, ntk=4.0, device="cpu")
    assert g[0] == f[0] and math.isclose(float(f[-1] / g[-1]), 4.0, rel_tol=1e-6)
    g, scale = L.rope_frequencies(64, 10000.0, yarn=4.0, trained=2048, device="cpu")
    f, _ = L.rope_frequencies(64, 10000.0, device="cpu")
    turns = 2048 * f / (2 * math.pi)
    assert torch.equal(g[turns >= 32], f[turns >= 32]) and torch.allclose(g[turns <= 1] * 4, f[turns <= 1])
    assert ((g <= f) & (g >= f / 4 * 0.999999)).all() and math.isclose(scale, 0.1 * math.log(4.0) + 1.0)
    for bad in (dict(rot_dim=3), dict(rot_dim=64, linear=2.0, yarn=2.0), dict(rot_dim=64, ntk=0.5)):
        with pytest.raises(ValueError):
            L.rope_frequencies(device="cpu", **bad)


def test_oracle_rope_closed_forms():
    x = np.array([[[1.0, 0.0, 2.0, 5.0]]])
    y, _ = O.rope(x, [1], [math.pi / 2])
    assert np.allclose(y[0, 0], [0.0, 1.0, 2.0, 5.0], atol=1e-12)
    y, _ = O.rope(x, [3], [math.pi / 2, math.pi], interleaved=True, scale=2.0)
    assert np.allclose(y[0, 0], [0.0, -2.0, -4.0, -10.0], atol=1e-12)
    # a position as far as the type goes, against its remainder
    far, near = (1 << 31) - 1, ((1 << 31) - 1) % 8
    a, _ = O.rope(x, [far], [0.25 * math.pi])
    b, _ = O.rope(x, [near], [0.25 * math.pi])
    assert np.allclose(a, b, atol=1e-6)  # 2^31 of the frequency's own last place


def test_oracle_chunk_agrees_with_the_decode_oracle():
    """The newest tokens of a request are a chain of drafts."""
    rng = np.random.default_rng(0)
    ck, cv = rng.standard_normal((2, 9, 4, 2, 8))
    table = np.array([[3, 1, 8, 0], [2, -1, 5, 7]])
    lens, n = [14, 11], 5
    q = rng.standard_normal((2, n, 4, 8))
    want = S.attn_decode(ck, cv, q, table, lens, 0.3)
    got = O.attn_chunk(ck, cv, q.reshape(2 * n, 4, 8), table, [0, n, 2 * n], lens, 0.3)
    for a, b in zip(want, got):
        assert np.allclose(a.reshape(b.shape), b)


def test_oracle_plan_by_hand():
    table, taken, cu, kv, pos, slot, status = O.kv_plan([3, 0], [3, 1], [[5, -1], [-1, -1]], 4, 9, 6, [7, 2])
    assert table.tolist() == [[5, 7], [2, -1]] and taken == 2 and cu.tolist() == [0, 3, 4] and kv.tolist() == [6, 1]
    assert pos.tolist() == [3, 4, 5, 0, -1, -1] and slot.tolist() == [23, 28, 29, 8, -1, -1] and status == 0
