"""csrc/attn_call.cpp without a GPU: it gives back what it does not take, and calls nothing then."""

import ctypes
import importlib.util
import os

import pytest

from exact_attention_52_gb300 import api

CALLS = []


@pytest.fixture(scope="module")
def module():
    pytest.importorskip("torch")
    if not os.path.exists(api.CALL_PATH):
        pytest.skip("not built")
    spec = importlib.util.spec_from_file_location("_attn_call", api.CALL_PATH)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    fake = ctypes.CFUNCTYPE(ctypes.c_size_t)(lambda: CALLS.append(1) or 0)  # stands for every function of the library
    m.bind(*[ctypes.cast(fake, ctypes.c_void_p).value] * len(api._CALL_FUNCTIONS))
    yield m
    lib = api.load_library()
    m.bind(*(ctypes.cast(getattr(lib, name), ctypes.c_void_p).value for name in api._CALL_FUNCTIONS))


def test_nothing_that_is_no_cuda_tensor_is_taken(module):
    import torch
    q = torch.zeros(1, 2, 4, 64).bfloat16()
    for t in (q, None, 3, "x", q.float(), q[0], torch.zeros(0)):
        assert module.cache_append(*[t] * 8, None, False, 0, 0) is None
        assert module.fwd_cache(*[t] * 7, None, False, None, -1, 0, None, None, t, 0, 0) is None
        assert module.fwd_sinks(t, t, t, 3, 1, 0, True, 0.5, None, None, 0, 0) is None
        assert module.bwd_sinks(*[t] * 6, 3, 1, 0, False, None, None, None, None, None, 0, 0) is None
    assert not CALLS


def test_a_wrong_number_of_arguments_is_given_back(module):
    for f in (module.cache_append, module.fwd_cache, module.fwd_sinks, module.bwd_sinks):
        for n in (0, 1, 11, 13, 16, 18):
            if n not in (12, 17):
                assert f(*[None] * n) is None
    assert not CALLS


def test_bind_wants_an_address_for_each_function(module):
    with pytest.raises(TypeError):
        module.bind(1, 2)


def test_calls_without_a_gpu_name_the_argument():
    torch = pytest.importorskip("torch")
    q = torch.zeros(1, 2, 4, 64).bfloat16()
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        api.fwd_sinks(q, q, q, 3, 1)
    with pytest.raises(ValueError, match="k must be a CUDA tensor"):
        api.cache_append(q, q, q, q, q, q, q, q)
    with pytest.raises(ValueError, match="unknown layout"):
        api.fwd_cache(q, q, q, q, q, q, q, layout="nbhd")


@pytest.mark.parametrize("what", ["no library", "another library", "another PyTorch"])
def test_a_module_that_does_not_fit_is_not_used(what, monkeypatch, tmp_path, module):
    """A file that cannot be loaded, or one built for another PyTorch or Python, leaves the calls
    to the half in Python, with a warning; what a call then answers is Python's."""
    torch = pytest.importorskip("torch")
    path = api.CALL_PATH
    if what == "no library":
        path = tmp_path / "_attn_call.so"
        path.write_bytes(b"not a library")
    elif what == "another library":
        path = api.LIB_PATH
    else:
        monkeypatch.setattr(torch, "__version__", "1.0")
    monkeypatch.setattr(api, "CALL_PATH", str(path))
    monkeypatch.setattr(api, "_calls", None)
    monkeypatch.setattr(torch.cuda, "is_available", lambda: True)  # as on a GPU machine, but for the device
    monkeypatch.setattr(torch.cuda, "init", lambda: None)
    with pytest.warns(RuntimeWarning, match="read their arguments in Python"):
        assert api._compiled_calls() is None
    assert api._compiled_calls() is None  # once
    q = torch.zeros(1, 2, 4, 64).bfloat16()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0, raising=False)
    with pytest.raises(ValueError, match="q must be a CUDA tensor"):
        api.fwd_sinks(q, q, q, 3, 1)


def test_the_module_says_what_it_was_built_for(module):
    import torch
    assert module.built_for == api._call_tag(torch)


def test_a_workspace_is_bytes_one_after_the_other():
    """Tensors whose bytes are fewer than their elements, or not in a row, are no workspace."""
    torch = pytest.importorskip("torch")
    one = torch.empty(1, dtype=torch.uint8)
    assert api._workspace_ok(torch, -1, torch.empty(512, dtype=torch.uint8), 512)
    assert api._workspace_ok(torch, -1, torch.empty(2, 64), 512)
    for t in (one.expand(512), torch.empty(1024, dtype=torch.uint8)[::2], torch.empty(511, dtype=torch.uint8),
              torch.empty(4, 64).t(), None, 512):
        assert not api._workspace_ok(torch, -1, t, 512)
        with pytest.raises(ValueError, match="workspace needs 512 contiguous bytes"):
            api._explain_workspace(torch.device("cpu"), t, 512)


def test_the_other_calls_take_no_smaller_workspace():
    """fwd_splitkv, bwd, bwd_window and bwd_strided look at the workspace that they are given."""
    torch = pytest.importorskip("torch")
    cpu = torch.device("cpu")
    ws = torch.empty(512, dtype=torch.uint8)
    assert api._checked_workspace(ws, 512, cpu) is ws
    assert api._checked_workspace(None, 512, cpu).numel() == 512
    for t in (ws[:511], ws[:1].expand(512), 3):
        with pytest.raises(ValueError, match="workspace needs 512"):
            api._checked_workspace(t, 512, cpu)
