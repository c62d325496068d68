"""Refusals and sizes of the routed operators, without a GPU.

Every argument is checked before a device is touched, so the C calls answer
here with the status that the check gives; calls that pass all checks answer
FP8Q_ERR_CUDA or FP8Q_ERR_UNSUPPORTED_DEVICE on a machine without a B200.
"""
import ctypes

import pytest
import torch

from fp8_block_scaled_group_b200 import _lib, api

OK, NULL, SHAPE, ALIGN, WORKSPACE, CUDA, UNSUPPORTED, ARG = 0, 1, 2, 3, 4, 5, 7, 8
MAX_EXPERTS, MAX_TOPK, MAX_RANK = 384, 64, 256

BUF = ctypes.create_string_buffer(4096)
BASE = (ctypes.addressof(BUF) + 255) // 256 * 256  # aligned; never read, the checks come first
BIG = 1 << 40


def call(name, **change):
    """The call with valid arguments, but for the changed ones."""
    args = dict(DEFAULTS[name])
    for k, v in change.items():
        assert k in args
        args[k] = v
    return getattr(_lib.load(), name)(*args.values())


DEFAULTS = {
    "fp8q_moe_route": dict(ids=BASE, offsets=BASE, rows=BASE, pos=BASE, tokens=4, topk=2, experts=8, stream=None),
    "fp8q_grouped_linear": dict(x=BASE, offsets=BASE, rows=BASE, wq=BASE, ws=BASE, fmt=0, y=BASE, work=BASE, bytes=BIG, tokens=4,
                                total=8, experts=8, n=256, k=256, stream=None),
    "fp8q_moe_ffn": dict(x=BASE, ids=BASE, p=BASE, w1=BASE, s1=BASE, w2=BASE, s2=BASE, fmt=0, y=BASE, work=BASE, bytes=BIG, tokens=4,
                         topk=2, experts=8, d=256, i=128, stream=None),
    "fp8q_lora_linear": dict(x=BASE, wq=BASE, ws=BASE, fmt=0, ids=BASE, a=BASE, b=BASE, scaling=BASE, y=BASE, work=BASE, bytes=BIG, m=4,
                             n=256, k=256, adapters=3, rank=16, stream=None),
}


@pytest.mark.parametrize("name", DEFAULTS)
def test_valid_arguments_reach_the_device_check(name):
    if torch.cuda.is_available():
        pytest.skip("the pointers here are host memory")
    assert call(name) in (CUDA, UNSUPPORTED)


@pytest.mark.parametrize("name", DEFAULTS)
def test_null_pointers(name):
    for k, v in DEFAULTS[name].items():
        if v == BASE and not (name == "fp8q_grouped_linear" and k == "rows"):
            assert call(name, **{k: None}) == NULL, k


@pytest.mark.parametrize("name", DEFAULTS)
def test_misaligned_pointers(name):
    for k, v in DEFAULTS[name].items():
        if v == BASE and k != "work":
            assert call(name, **{k: BASE + 2}) == ALIGN, k
    for k in set(DEFAULTS[name]) & {"x", "wq", "y", "w1", "w2", "a", "b", "ws", "s1", "s2"}:
        assert call(name, **{k: BASE + 8}) == ALIGN, k


@pytest.mark.parametrize("name", ["fp8q_grouped_linear", "fp8q_moe_ffn", "fp8q_lora_linear"])
def test_workspace(name):
    need = {"fp8q_grouped_linear": lambda a: api.grouped_linear_workspace_bytes(a["tokens"], a["total"], a["experts"], a["n"], a["k"]),
            "fp8q_moe_ffn": lambda a: api.moe_ffn_workspace_bytes(a["tokens"], a["topk"], a["experts"], a["d"], a["i"]),
            "fp8q_lora_linear": lambda a: api.lora_linear_workspace_bytes(a["m"], a["n"], a["k"], a["adapters"], a["rank"])}[name](DEFAULTS[name])
    assert need > 0 and need % 256 == 0
    assert call(name, bytes=need - 1) == WORKSPACE
    assert call(name, work=BASE + 128) == WORKSPACE
    if not torch.cuda.is_available():
        assert call(name, bytes=need) in (CUDA, UNSUPPORTED)


@pytest.mark.parametrize("change", [dict(experts=0), dict(experts=MAX_EXPERTS + 1), dict(topk=0), dict(topk=MAX_TOPK + 1),
                                    dict(tokens=1 << 23, topk=2)])
def test_route_sizes(change):
    assert call("fp8q_moe_route", **change) == SHAPE


@pytest.mark.parametrize("change", [dict(n=0), dict(n=130), dict(k=64), dict(k=0), dict(experts=0), dict(experts=MAX_EXPERTS + 1),
                                    dict(tokens=1 << 23), dict(total=1 << 23), dict(n=1 << 20, k=1 << 11), dict(rows=None),
                                    dict(experts=256, n=1 << 23, k=128)])
def test_grouped_sizes(change):
    assert call("fp8q_grouped_linear", **change) == SHAPE
    change.pop("rows", None)
    if change:
        a = {**DEFAULTS["fp8q_grouped_linear"], **change}
        assert api.grouped_linear_workspace_bytes(a["tokens"], a["total"], a["experts"], a["n"], a["k"]) == 0


@pytest.mark.parametrize("change", [dict(d=100), dict(i=0), dict(i=192), dict(i=1 << 31), dict(experts=0), dict(experts=MAX_EXPERTS + 1), dict(topk=0),
                                    dict(topk=MAX_TOPK + 1), dict(tokens=1 << 22), dict(tokens=1 << 30), dict(tokens=1 << 20, d=1024)])
def test_moe_sizes(change):
    assert call("fp8q_moe_ffn", **change) == SHAPE


@pytest.mark.parametrize("change", [dict(d=100), dict(i=0), dict(i=192), dict(i=1 << 31), dict(i=1 << 30), dict(experts=0), dict(experts=MAX_EXPERTS + 1),
                                    dict(topk=0), dict(topk=MAX_TOPK + 1), dict(tokens=1 << 22), dict(tokens=1 << 30),
                                    dict(tokens=1 << 20, d=1024, i=128), dict(tokens=1 << 20, i=1024), dict(d=1 << 20, i=1 << 10),
                                    dict(experts=256, d=1 << 23), dict(experts=256, d=128, i=1 << 22)])
def test_moe_workspace_of_refused_sizes_is_zero(change):
    """The workspace query and the call refuse the same sizes: a program that asks first never allocates for a call that will not run."""
    assert call("fp8q_moe_ffn", **change) == SHAPE
    a = {**DEFAULTS["fp8q_moe_ffn"], **change}
    assert api.moe_ffn_workspace_bytes(a["tokens"], a["topk"], a["experts"], a["d"], a["i"]) == 0


def test_moe_workspace_of_the_largest_sizes():
    """Just inside the limits the query answers, and so does the call."""
    for change in (dict(tokens=(1 << 20) - 1, topk=2, d=1024, i=128), dict(experts=MAX_EXPERTS, tokens=1, topk=MAX_TOPK)):
        a = {**DEFAULTS["fp8q_moe_ffn"], **change}
        need = api.moe_ffn_workspace_bytes(a["tokens"], a["topk"], a["experts"], a["d"], a["i"])
        assert need > 0
        assert call("fp8q_moe_ffn", **change, bytes=need - 1) == WORKSPACE


@pytest.mark.parametrize("change", [dict(n=0), dict(n=100), dict(k=192), dict(rank=0), dict(rank=12), dict(rank=MAX_RANK + 8), dict(adapters=0),
                                    dict(adapters=1 << 23), dict(m=1 << 23), dict(n=1 << 20, k=1 << 11)])
def test_lora_sizes(change):
    assert call("fp8q_lora_linear", **change) == SHAPE
    a = {**DEFAULTS["fp8q_lora_linear"], **change}
    assert api.lora_linear_workspace_bytes(a["m"], a["n"], a["k"], a["adapters"], a["rank"]) == 0


@pytest.mark.parametrize("name", ["fp8q_grouped_linear", "fp8q_moe_ffn", "fp8q_lora_linear"])
def test_unknown_weight_format(name):
    assert call(name, fmt=2) == ARG and call(name, fmt=-1) == ARG


def test_nothing_to_do():
    assert call("fp8q_grouped_linear", tokens=0, x=None, y=None) == OK
    assert call("fp8q_grouped_linear", total=0, rows=BASE) == OK
    assert call("fp8q_moe_ffn", tokens=0, x=None) == OK
    assert call("fp8q_lora_linear", m=0, x=None, y=None) == OK


def test_python_refuses_what_is_not_on_a_device():
    ids = torch.zeros(3, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="topk_ids must be a CUDA tensor"):
        api.moe_route(ids, 8)
    with pytest.raises(ValueError, match="2-D"):
        api.moe_route(ids[0], 8)
    x = torch.zeros(3, 128, dtype=torch.bfloat16)
    w, s = torch.zeros(2, 128, 128, dtype=torch.uint8), torch.zeros(2, 1, 1)
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        api.grouped_linear(x, w, s, torch.zeros(3, dtype=torch.int32))
    with pytest.raises(ValueError, match="x must be a CUDA tensor"):
        api.lora_linear(x, w[0], s[0], torch.zeros(3, dtype=torch.int32), x[None, :, :128], torch.zeros(1, 128, 3, dtype=torch.bfloat16), torch.ones(1))
    with pytest.raises(ValueError, match="wq 3-D"):
        api.grouped_linear(x, w[0], s, torch.zeros(3, dtype=torch.int32))


def test_stalled_grouped_linear_refuses_what_the_call_refuses():
    lib, args = _lib.load(), dict(DEFAULTS["fp8q_grouped_linear"])

    def stalled(budget, **change):
        a = {**args, **change}
        stream = a.pop("stream")
        return lib.fp8q_diag_stalled_grouped_linear(*a.values(), budget, stream)

    assert stalled(0) == ARG and stalled(2_000_000_001) == ARG  # no budget, and past the second that a wait lasts at most
    assert stalled(1000, fmt=2) == ARG and stalled(1000, n=100) == SHAPE and stalled(1000, rows=None) == SHAPE
    assert stalled(1000, x=None) == NULL and stalled(1000, y=BASE + 8) == ALIGN and stalled(1000, bytes=1000) == WORKSPACE
    assert stalled(1000, tokens=0) == OK
    if not torch.cuda.is_available():
        assert stalled(1000) in (CUDA, UNSUPPORTED)
