"""CPU checks of the MoE operators' C ABI: the header's functions are the ones the
library exports and the binding declares, sizes and refusals are checked before
anything touches a GPU, and the 64-bit forms the GPU tests compare with hold what
they say."""
import ctypes
import os
import re

import pytest
import torch

import combine_topk_ids_dest_gb300 as ep
import moe_ref
from combine_topk_ids_dest_gb300 import _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
INVALID = ep.EP_ERR_INVALID_ARG


def test_header_and_exports_agree():
    text = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "ep_moe.h")).read(), flags=re.S)
    declared = sorted(set(re.findall(r"\b(ep_[a-z0-9_]+)\s*\(", text)))
    assert declared == sorted(_lib.MOE_EXPORTS)
    L = _lib.load()
    for name in declared:
        assert hasattr(L, name), name


def _message():
    return _lib.load().ep_last_error().decode()


def _experts(**kw):
    base = dict(num_experts=4, first_expert=0, top_k=2, hidden=128, intermediate=256, max_tokens=8, data=4096, group=0,
                down_group=None, scale_dtype=0)
    base.update(kw)
    b = base
    down = b["group"] if b["down_group"] is None else b["down_group"]
    w = [_lib.EpWeightC(b["data"], gr, 0, b["scale_dtype"]) for gr in (b["group"], down)]
    cfg = _lib.EpExpertsConfigC(b["num_experts"], b["first_expert"], b["top_k"], b["hidden"], b["intermediate"],
                                b["max_tokens"], *w)
    n = ctypes.c_size_t(0)
    return _lib.load().ep_experts_workspace_size(ctypes.byref(cfg), ctypes.byref(n)), n.value


@pytest.mark.parametrize("kw,frag", [
    (dict(num_experts=0), "num_experts"), (dict(num_experts=513), "num_experts"), (dict(first_expert=-1), "first_expert"),
    (dict(top_k=0), "top_k"), (dict(top_k=33), "top_k"), (dict(hidden=0), "hidden"), (dict(hidden=132), "hidden"),
    (dict(intermediate=12), "intermediate"), (dict(hidden=65544), "hidden"), (dict(max_tokens=0), "max_tokens"),
    (dict(max_tokens=65), "max_tokens"), (dict(data=0), "data"), (dict(data=4104), "16-byte"), (dict(group=48), "group"),
    (dict(group=32, down_group=0), "both"), (dict(group=64, hidden=96), "hidden"), (dict(group=32, data=4112), "128-byte"),
    (dict(group=32, scale_dtype=3), "scale_dtype"),
])
def test_experts_refusals(kw, frag):
    st, _ = _experts(**kw)
    assert st == INVALID
    assert frag in _message()


def test_experts_workspace_grows_with_tokens():
    assert _experts()[0] == ep.EP_OK
    assert 0 < _experts(max_tokens=1)[1] < _experts(max_tokens=64)[1]
    assert _experts(group=32)[0] == ep.EP_OK


@pytest.mark.parametrize("kw,frag", [
    (dict(group=16), "group"), (dict(cols=72), "cols"), (dict(rows=0), "rows"), (dict(mats=0), "mats"),
    (dict(scale_dtype=1), "scale_dtype"), (dict(cols=65600, group=32), "limited"), (dict(mats=3, gate_up=1), "odd"),
])
def test_packed_size_refusals(kw, frag):
    b = dict(scale_dtype=0, mats=1, rows=128, cols=128, group=32, gate_up=0)
    b.update(kw)
    w = _lib.EpIntWeightC(16, 16, 0, b["scale_dtype"], b["mats"], b["rows"], b["cols"], b["group"], b["gate_up"])
    n = ctypes.c_size_t(0)
    assert _lib.load().ep_weight_packed_size(ctypes.byref(w), ctypes.byref(n)) == INVALID
    assert frag in _message()


@pytest.mark.parametrize("rows,cols,group,zeros", [(128, 128, 128, 0), (129, 160, 32, 1), (1, 64, 64, 0)])
def test_packed_size_formula(rows, cols, group, zeros):
    w = _lib.EpIntWeightC(16, 16, 16 if zeros else 0, 0, 3, rows, cols, group, 0)
    n = ctypes.c_size_t(0)
    assert _lib.load().ep_weight_packed_size(ctypes.byref(w), ctypes.byref(n)) == ep.EP_OK
    tile = 128 * 128 // 2 + 128 * (128 // group) * (3 if zeros else 2)
    assert n.value == 3 * -(-rows // 128) * -(-cols // 128) * tile


def _linear(**kw):
    b = dict(inputs=256, outputs=100, max_tokens=4, data=4096, group=64)
    b.update(kw)
    cfg = _lib.EpLinearConfigC(b["inputs"], b["outputs"], b["max_tokens"], _lib.EpWeightC(b["data"], b["group"], 0, 0))
    n = ctypes.c_size_t(0)
    return _lib.load().ep_linear_workspace_size(ctypes.byref(cfg), ctypes.byref(n))


@pytest.mark.parametrize("kw,frag", [(dict(group=0), "group"), (dict(inputs=100), "inputs"), (dict(outputs=0), "outputs"),
                                     (dict(max_tokens=65), "max_tokens"), (dict(data=64), "128-byte")])
def test_linear_refusals(kw, frag):
    assert _linear() == ep.EP_OK
    assert _linear(**kw) == INVALID
    assert frag in _message()


def _router(**kw):
    b = dict(num_experts=16, top_k=2, hidden=64, dtype=0, scoring=0, num_groups=1, top_groups=1, renormalize=1, scale=1.0,
             weight=4096, bias=0)
    b.update(kw)
    cfg = _lib.EpRouterConfigC(*[b[f] for f, _ in _lib.EpRouterConfigC._fields_])
    h = ctypes.c_void_p()
    return _lib.load().ep_router_create(ctypes.byref(cfg), ctypes.byref(h))


@pytest.mark.parametrize("kw,frag", [
    (dict(num_experts=0), "num_experts"), (dict(num_experts=513), "num_experts"), (dict(hidden=60), "hidden"),
    (dict(dtype=3), "dtype"), (dict(scoring=2), "scoring"), (dict(num_groups=3), "num_groups"),
    (dict(num_groups=4, top_groups=5), "top_groups"), (dict(top_k=17), "top_k"),
    (dict(num_groups=4, top_groups=1, top_k=5), "top_k"), (dict(scale=float("nan")), "scale"),
    (dict(weight=0), "weight"), (dict(bias=2), "bias"),
])
def test_router_refusals(kw, frag):
    assert _router(**kw) == INVALID
    assert frag in _message()


def test_null_handles_fail_cleanly():
    L = _lib.load()
    assert L.ep_router_run(None, None, 0, 1, None, None, None, 0, None) == INVALID
    assert L.ep_experts_run(None, None, 0, None, None, 1, None, 0, None) == INVALID
    assert L.ep_linear_run(None, 0, None, 0, 1, None, 0, None) == INVALID
    assert L.ep_layer_run(None, None, None, 0, 1, None, None, None, 0, None) == INVALID
    assert L.ep_router_destroy(None) == L.ep_experts_destroy(None) == L.ep_linear_destroy(None) == ep.EP_OK


def test_creation_without_a_gpu_reports_an_error():
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    assert _router() in (ep.EP_ERR_CUDA, ep.EP_ERR_UNSUPPORTED)


def test_binding_wants_cuda_tensors():
    w = torch.zeros(8, 64, dtype=torch.bfloat16)
    for make in (lambda: ep.EpRouter(w, 2), lambda: ep.EpExperts(w, w, 2),
                 lambda: ep.Int4Weight(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.bfloat16))):
        with pytest.raises(ValueError, match="CUDA"):
            make()


def test_reference_forms():
    codes = torch.tensor([[0x80, 0x1F]], dtype=torch.uint8)  # codes 0, 8, 15, 1
    s = torch.tensor([[2.0, 0.5]], dtype=torch.bfloat16)
    assert moe_ref.dequant(codes, s).tolist() == [[-16.0, 0.0, 3.5, -3.5]]
    assert moe_ref.dequant(codes, s, torch.tensor([[1, 15]], dtype=torch.uint8)).tolist() == [[-2.0, 14.0, 0.0, -7.0]]
    sc = torch.tensor([[0.5, 0.25, 0.5, 0.125]], dtype=torch.float64)
    assert moe_ref.choice(sc, None, 3)[0].tolist() == [[0, 2, 1]]
    bias = torch.tensor([-torch.inf, 0.0, -torch.inf, 1.0])
    assert moe_ref.choice(sc, bias, 3)[0].tolist() == [[3, 1, -1]]
    assert moe_ref.choice(sc, None, 2, groups=2, top_groups=1)[0].tolist() == [[0, 1]]
    ids = torch.tensor([[3, 1, -1]])
    assert moe_ref.chosen_weights(sc, ids, True, 3.0).tolist() == [[1.0, 2.0, 0.0]]
