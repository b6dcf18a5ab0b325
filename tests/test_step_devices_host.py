"""The decode-step binding refuses every tensor that is not on the call's GPU
before anything is launched. CPU only: tensors that say they lie on a GPU, and
entry points that must not be reached."""

import pytest
import torch

import linear_attention_state_chunked_gb300 as L
from linear_attention_state_chunked_gb300 import step

BF = torch.bfloat16


class Said(torch.Tensor):
    """A CPU tensor that gives `gpu` as its device; slices and views do as well."""
    gpu = 0

    def get_device(self):
        return self.gpu

    @property
    def is_cuda(self):
        return True


class SaidOther(Said):
    gpu = 1


class Reached(Exception):
    pass


@pytest.fixture(autouse=True)
def no_launch(monkeypatch):
    def reached(*args):
        raise Reached

    for name in ("_call_append", "_call_attn", "_call_norm"):
        monkeypatch.setattr(step, name, reached)
    monkeypatch.setattr(step, "_current_device", lambda: 0)
    monkeypatch.setattr(step, "_raw_stream", lambda device: 0)


def on_gpu(t, kind=Said):
    return t.as_subclass(kind)


def elsewhere(t, kind):
    """The tensor on the CPU, or on another GPU."""
    return on_gpu(t, SaidOther) if kind == "cuda:1" else t.as_subclass(torch.Tensor)


def call(which):
    """A call that would be launched: (function, keyword tensors, the rest)."""
    i32 = dict(dtype=torch.int32)
    k = torch.zeros((1, 4, 8, 2, 64), dtype=BF)
    rows = torch.zeros((3, 2, 2, 64), dtype=BF)
    common = dict(page_table=torch.zeros((3, 4), **i32), status=torch.zeros(1, **i32))
    if which == "append":
        t = dict(cache_k=k, cache_v=k.clone(), k=rows, v=rows.clone(), pos=torch.zeros(3, **i32), **common)
        return L.lin_state_kv_append, t, dict(layer=0)
    if which == "append_tree":
        t = dict(cache_k=k, cache_v=k.clone(), k=rows, v=rows.clone(), pos=torch.zeros(3, **i32),
                 parent=torch.zeros((3, 2), **i32), accept_node=torch.zeros(3, **i32), **common)
        return L.lin_state_kv_append, t, dict(layer=0)
    if which == "attn":
        t = dict(cache_k=k, cache_v=k.clone(), q=torch.zeros((3, 2, 4, 64), dtype=BF),
                 out=torch.zeros((3, 2, 4, 64), dtype=BF), kv_len=torch.zeros(3, **i32),
                 parent=torch.zeros((3, 2), **i32), workspace=torch.zeros(1 << 22, dtype=torch.uint8), **common)
        return L.lin_state_attn_decode, t, dict(layer=0)
    x = torch.zeros((3, 64), dtype=BF)
    t = {n: x.clone() for n in ("x", "gate", "residual", "h_out", "y")}
    t.update({n: torch.zeros(64, dtype=BF) for n in ("w_post", "scale_w", "w_pre")})
    return L.lin_state_block_norm, t, dict(gate_act="silu")


def run(which, change):
    fn, t, rest = call(which)
    t = {n: change(n, on_gpu(x)) for n, x in t.items()}
    if "cache_k" in t:
        rest["cache"] = L.KVCache(1, 4, 8, 2, 64, k=t.pop("cache_k"), v=t.pop("cache_v"))
    fn(**t, **rest)


CASES = [(w, n) for w in ("append", "append_tree", "attn", "norm") for n in call(w)[1]]


@pytest.mark.parametrize("which", ["append", "append_tree", "attn", "norm"])
def test_a_call_on_one_gpu_is_made(which):
    with pytest.raises(Reached):
        run(which, lambda name, t: t)


@pytest.mark.parametrize("which,name", CASES)
@pytest.mark.parametrize("kind", ["cpu", "cuda:1"])
def test_one_tensor_elsewhere_is_refused(which, name, kind):
    pair = ("cache_k", "cache_v")  # one tensor's device is the cache's
    with pytest.raises(ValueError, match="cuda:|CUDA"):
        run(which, lambda n, t: elsewhere(t, kind) if n == name or (n in pair and name in pair) else t)


def test_a_cache_on_the_cpu_is_refused_by_both_calls():
    for which in ("append", "attn"):
        with pytest.raises(ValueError, match="cache: want a CUDA tensor"):
            run(which, lambda n, t: elsewhere(t, "cpu") if n.startswith("cache_") else t)


@pytest.mark.parametrize("which", ["append", "attn", "norm"])
def test_another_current_device_is_refused(which, monkeypatch):
    monkeypatch.setattr(step, "_current_device", lambda: 1)
    with pytest.raises(ValueError, match="not the current device"):
        run(which, lambda name, t: t)


def test_k_and_v_on_different_devices_are_refused():
    k = torch.zeros((1, 4, 8, 2, 64), dtype=BF)
    with pytest.raises(ValueError, match="one device"):
        L.KVCache(1, 4, 8, 2, 64, k=k, v=k.to("meta"))


@pytest.mark.parametrize("which", ["append", "attn"])
@pytest.mark.parametrize("bad", [torch.zeros(1), torch.zeros(1, dtype=torch.int64), torch.zeros(0, dtype=torch.int32)])
def test_status_is_one_int32_word(which, bad):
    with pytest.raises(ValueError, match="status"):
        run(which, lambda n, t: on_gpu(bad) if n == "status" else t)


def test_workspace_is_contiguous():
    with pytest.raises(ValueError, match="workspace"):
        run("attn", lambda n, t: on_gpu(torch.zeros((1 << 22, 2), dtype=torch.uint8))[:, 0] if n == "workspace" else t)
