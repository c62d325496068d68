"""The routing plan, the grouped projection and the mixture-of-experts FFN on the GPU.

The plan is compared exactly with its definition. The grouped projection is
compared row by row with the 64-bit form (tolerance derived in routed_ref),
over group sizes that end inside token blocks, empty groups, rows that no
group owns, both weight formats and both ways of naming rows. The FFN is
compared link by link: its gate|up, SiLU and down steps through the calls that
make them up, its last sum in 64 bits.
"""
import pytest
import torch

import routed_ref as ref
from fp8_block_scaled_group_b200 import api

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")


def random_ids(t, topk, experts, seed, drop=0.0):
    g = torch.Generator(device=DEV).manual_seed(seed)
    ids = torch.rand(t, experts, device=DEV, generator=g).topk(topk, dim=1).indices.int()
    return torch.where(torch.rand(t, topk, device=DEV, generator=g) < drop, -1, ids).contiguous()


# ------------------------------------------------------------------- plan --

def check_plan(ids, experts):
    got = api.moe_route(ids, experts)
    for a, b, name in zip(got, ref.route(ids.cpu(), experts), ("offsets", "rows", "pos")):
        assert torch.equal(a.cpu(), b), name


@pytest.mark.parametrize("t,topk,experts", [(1, 1, 1), (1, 8, 64), (25, 8, 64), (31, 3, 7), (256, 8, 384), (257, 8, 33),
                                            (1168, 8, 64), (4576, 6, 96), (16384, 8, 128)])
@pytest.mark.parametrize("drop", [0.0, 0.3])
def test_route(t, topk, experts, drop):
    check_plan(random_ids(t, topk, experts, 7 + t, drop), experts)


@pytest.mark.parametrize("t,topk,experts", [(16385, 8, 33), (20011, 9, 20), (50000, 16, 24)])
def test_route_past_what_shared_memory_holds(t, topk, experts):
    check_plan(random_ids(t, topk, experts, 8 + t, 0.1), experts)


@pytest.mark.parametrize("t,topk", [(40, 4), (900, 8)])
@pytest.mark.parametrize("fill", ["same", "none", "last", "wild"])
def test_route_uneven(t, topk, fill):
    ids = torch.zeros(t, topk, dtype=torch.int32, device=DEV)
    if fill == "same":
        ids += 5  # one expert gets every slot, the same token several times
    elif fill == "none":
        ids -= 1
    elif fill == "last":
        ids += 15
        ids[0, 0] = 0
    else:
        ids[:] = torch.randint(-(1 << 31), (1 << 31) - 1, (t, topk), device=DEV).int()
        ids[::3] = 2
    check_plan(ids, 16)


def test_route_of_no_tokens():
    offsets, rows, pos = api.moe_route(torch.empty(0, 4, dtype=torch.int32, device=DEV), 9)
    assert offsets.tolist() == [0] * 10 and rows.numel() == 0 and pos.shape == (0, 4)


# ------------------------------------------------- grouped projection --

def check_grouped(x, codes, scale, offsets, rows):
    total = x.shape[0] if rows is None else rows.numel()
    out = torch.full((total, codes.shape[1]), 7.5, dtype=torch.bfloat16, device=DEV)
    api.grouped_linear(x, codes, scale, offsets, rows=rows, out=out)
    y, err, written = ref.grouped(x, codes, scale, offsets, rows)
    assert api.device_error() == 0
    ref.assert_close(out[written], y[written], err[written])
    assert bool((out[~written] == 7.5).all()), "rows of no group were written"
    return out


def offsets_of(sizes, start=0):
    off = [start]
    for s in sizes:
        off.append(off[-1] + s)
    return torch.tensor(off, dtype=torch.int32, device=DEV)


SIZES = [[1], [0, 1, 0], [3, 0, 5, 1], [31, 32, 33, 1], [63, 64, 65], [255, 256, 257, 2], [0, 0, 700, 0, 1]]


@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: "-".join(map(str, s)))
@pytest.mark.parametrize("n,k", [(128, 128), (384, 512), (512, 1152)])
@pytest.mark.parametrize("fmt", ["block", "row"])
def test_grouped_in_order(sizes, n, k, fmt):
    x = ref.activations(sum(sizes) + 2, k, 11, DEV)  # two rows behind the last group
    codes, scale = ref.weights(len(sizes), n, k, fmt, 12, DEV)
    check_grouped(x, codes, scale, offsets_of(sizes), None)


@pytest.mark.parametrize("t,topk,experts,n,k", [(1, 8, 64, 512, 1024), (25, 8, 64, 256, 640), (300, 4, 8, 384, 512),
                                                (700, 5, 6, 256, 384), (130, 2, 40, 1280, 1152)])
@pytest.mark.parametrize("fmt", ["block", "row"])
def test_grouped_gathered(t, topk, experts, n, k, fmt):
    x = ref.activations(t, k, 21, DEV)
    codes, scale = ref.weights(experts, n, k, fmt, 22, DEV)
    offsets, rows, _ = api.moe_route(random_ids(t, topk, experts, 23, 0.1), experts)
    check_grouped(x, codes, scale, offsets, rows)


@pytest.mark.parametrize("most,n,k", [(60, 1408, 256), (200, 1408, 256), (90, 2048, 640), (400, 1280, 384)])
@pytest.mark.parametrize("fmt", ["block", "row"])
def test_grouped_many_tiles(most, n, k, fmt):
    """More tiles than are split: whole tiles in turn, experts of all sizes, some empty."""
    g = torch.Generator().manual_seed(most)
    sizes = [int(v) for v in torch.randint(0, most + 1, (80,), generator=g)]
    sizes[3] = sizes[40] = sizes[79] = 0
    x = ref.activations(sum(sizes), k, 15, DEV)
    codes, scale = ref.weights(len(sizes), n, k, fmt, 16, DEV)
    check_grouped(x, codes, scale, offsets_of(sizes), None)


@pytest.mark.parametrize("sizes", [[5, 40], [1], [3] * 10, [63, 0, 64, 1, 40] * 3, [150, 100], [160, 33, 96] * 2, [500, 130], [200] * 5, [1, 700, 0, 255]],
                         ids=lambda s: "-".join(map(str, s)))
def test_grouped_long_k(sizes):
    """Few tiles of a long K: their K range is split over the pairs and joined."""
    x = ref.activations(sum(sizes), 17408, 17, DEV)
    codes, scale = ref.weights(len(sizes), 256, 17408, "block", 18, DEV)
    check_grouped(x, codes, scale, offsets_of(sizes), None)


@pytest.mark.parametrize("rows_per", [3, 100])
def test_grouped_weights_past_2_31_bytes(rows_per):
    """The last experts' weights lie past 2^31 bytes of the weight tensor."""
    experts, n, k = 120, 4096, 5120
    codes = torch.zeros(experts, n, k, dtype=torch.uint8, device=DEV)
    scale = torch.ones(experts, n // 128, k // 128, device=DEV)
    codes[-2:], scale[-2:] = ref.weights(2, n, k, "block", 19, DEV)
    x = ref.activations(2 * rows_per, k, 20, DEV)
    offsets = offsets_of([0] * (experts - 2) + [rows_per, rows_per])
    y = api.grouped_linear(x, codes, scale, offsets)
    for e, at in ((-2, slice(0, rows_per)), (-1, slice(rows_per, None))):
        a, err = ref.product(ref.quantized(x[at]), ref.weight_value(codes[e], scale[e]))
        ref.assert_close(y[at], a, err)


def test_most_experts_and_choices():
    t, topk, experts, d, i = 40, 64, 384, 128, 128
    check_moe(t, topk, experts, d, i, "block", 0.1, 65)


def test_calls_at_once_on_two_streams():
    """Two projections in flight together, a workspace each, many times over."""
    parts = []
    for sizes, k, seed in (([3] * 60, 1024, 44), ([250] * 3, 17408, 45)):
        x = ref.activations(sum(sizes), k, seed, DEV)
        codes, scale = ref.weights(len(sizes), 1024, k, "block", seed + 5, DEV)
        off = offsets_of(sizes)
        want = api.grouped_linear(x, codes, scale, off)
        work = torch.empty(api.grouped_linear_workspace_bytes(x.shape[0], x.shape[0], len(sizes), 1024, k), dtype=torch.uint8, device=DEV)
        parts.append((x, codes, scale, off, work, want, torch.zeros_like(want), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for x, codes, scale, off, work, _, out, stream in parts:
            api.grouped_linear(x, codes, scale, off, workspace=work, out=out, stream=stream)
    torch.cuda.synchronize()
    for *_, want, out, _ in parts:
        assert torch.equal(want.view(torch.int16), out.view(torch.int16))
    assert api.device_error() == 0


def test_on_a_stream_with_tensors_of_the_calls_own():
    """Outputs and workspaces that the calls make while they run on another stream than the current one: neither the
    filling of one nor the next use of the other's memory on the current stream may overlap the call."""
    x = ref.activations(400, 1024, 48, DEV)
    w1, s1 = ref.weights(6, 512, 1024, "block", 49, DEV)
    w2, s2 = ref.weights(6, 1024, 256, "block", 50, DEV)
    ids = random_ids(400, 2, 6, 51)
    p = torch.rand(400, 2, device=DEV)
    want = api.moe_ffn(x, ids, p, w1, s1, w2, s2)
    offsets, rows, _ = api.moe_route(ids, 6)
    want_y = api.grouped_linear(x, w1, s1, offsets, rows=rows)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for _ in range(10):
        y = api.moe_ffn(x, ids, p, w1, s1, w2, s2, stream=stream)
        off, r, _ = api.moe_route(ids, 6, stream=stream)
        z = api.grouped_linear(x, w1, s1, off, rows=r, stream=stream)
        for size in (1 << 20, 1 << 22, 1 << 24):  # would be given the memory that the calls have let go
            torch.full((size,), 255, dtype=torch.uint8, device=DEV)
        torch.cuda.synchronize()
        assert torch.equal(y.view(torch.int16), want.view(torch.int16))
        assert torch.equal(z.view(torch.int16), want_y.view(torch.int16))


def test_refusals():
    x = ref.activations(8, 256, 46, DEV)
    codes, scale = ref.weights(4, 256, 256, "block", 47, DEV)
    off = offsets_of([2, 2, 2, 2])
    with pytest.raises(ValueError, match="contiguous"):
        api.grouped_linear(x.repeat(1, 2)[:, ::2], codes, scale, off)
    with pytest.raises(ValueError, match="offsets must be"):
        api.grouped_linear(x, codes, scale, off.long())
    with pytest.raises(ValueError, match="offsets must have shape"):
        api.grouped_linear(x, codes, scale, off[:-1].contiguous())
    with pytest.raises(ValueError, match="w_scale must have shape"):
        api.grouped_linear(x, codes, scale[:, :1].contiguous(), off)
    with pytest.raises(ValueError, match="workspace must be"):
        api.grouped_linear(x, codes, scale, off, workspace=torch.empty(1 << 20, device=DEV))
    with pytest.raises(RuntimeError, match="WORKSPACE"):
        api.grouped_linear(x, codes, scale, off, workspace=torch.empty(1 << 10, dtype=torch.uint8, device=DEV))
    with pytest.raises(ValueError, match="offsets must be a CUDA tensor"):
        api.grouped_linear(x, codes, scale, off.cpu())
    with pytest.raises(RuntimeError, match="SHAPE"):
        api.moe_route(torch.zeros(2, 65, dtype=torch.int32, device=DEV), 8)


@pytest.mark.parametrize("rows_per", [2, 300])
def test_grouped_with_plan_of_another_kind(rows_per):
    """Offsets that start past row 0, end early, overlap nothing but leave gaps, run backwards or past the end;
    rows that repeat and rows that name no token."""
    experts, n, k, t = 5, 256, 256, 40
    total = experts * rows_per
    x = ref.activations(t, k, 31, DEV)
    codes, scale = ref.weights(experts, n, k, "block", 32, DEV)
    rows = torch.randint(0, t, (total,), device=DEV).int()
    rows[1] = -1
    rows[-1] = t
    rows[total // 2] = rows[0]
    for off in ([1, rows_per, rows_per, 3 * rows_per, 4 * rows_per, 5 * rows_per - 1],
                [0, total, 2 * rows_per, total + 50, 0, 0],
                [-3, 2, 1, 1, 4 * rows_per, 4 * rows_per]):
        offsets = torch.tensor(off, dtype=torch.int32, device=DEV)
        if off[1] == total:
            # groups 0, 2 and 3 own the same rows: only that nothing else is touched is defined
            out = torch.full((total, n), 7.5, dtype=torch.bfloat16, device=DEV)
            api.grouped_linear(x, codes, scale, offsets, rows=rows, out=out)
            assert api.device_error() == 0 and bool(torch.isfinite(out.float()).all())
        else:
            check_grouped(x, codes, scale, offsets, rows)


def test_grouped_repeats_bit_for_bit_and_on_any_stream():
    x = ref.activations(25, 17408, 41, DEV)
    codes, scale = ref.weights(6, 512, 17408, "block", 42, DEV)  # split K ranges
    offsets, rows, _ = api.moe_route(random_ids(25, 4, 6, 43), 6)
    first = api.grouped_linear(x, codes, scale, offsets, rows=rows)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    outs = []
    for s in (None, stream) * 3:
        outs.append(torch.zeros_like(first))
        torch.cuda.synchronize()
        api.grouped_linear(x, codes, scale, offsets, rows=rows, out=outs[-1], stream=s)
        torch.cuda.synchronize()
    assert all(torch.equal(first.view(torch.int16), o.view(torch.int16)) for o in outs)


def test_grouped_rows_agree_with_the_plain_projection():
    """One expert that owns every row is the plain projection: the same sums in the same order."""
    x = ref.activations(300, 512, 51, DEV)
    codes, scale = ref.weights(1, 38 * 256, 512, "block", 52, DEV)  # enough tiles that K is not split
    got = api.grouped_linear(x, codes, scale, offsets_of([300]))
    want = api.linear(x, codes[0], scale[0])
    y, err = ref.product(ref.quantized(x), ref.weight_value(codes[0], scale[0]))
    ref.assert_close(got, y, err)
    ref.assert_close(want, y, err)


# --------------------------------------------------------------- the FFN --

def check_moe(t, topk, experts, d, i, fmt, drop, seed):
    x = ref.activations(t, d, seed, DEV)
    w1, s1 = ref.weights(experts, 2 * i, d, fmt, seed + 1, DEV)
    w2, s2 = ref.weights(experts, d, i, fmt, seed + 2, DEV)
    ids = random_ids(t, topk, experts, seed + 3, drop)
    p = torch.rand(t, topk, device=DEV, generator=torch.Generator(device=DEV).manual_seed(seed))
    p = torch.where(ids < 0, float("nan"), p)  # the weight of a dropped slot is never used
    y = api.moe_ffn(x, ids, p, w1, s1, w2, s2)
    offsets, rows, pos = api.moe_route(ids, experts)
    gu = api.grouped_linear(x, w1, s1, offsets, rows=rows)
    a, b, c = ref.grouped(x, w1, s1, offsets, rows)
    ref.assert_close(gu[c], a[c], b[c], "gate|up")
    gate, up = gu[:, :i].double(), gu[:, i:].double()
    h = ref.bf16_nearest(gate * torch.sigmoid(gate) * up)
    each = api.grouped_linear(h, w2, s2, offsets)
    a, b, c = ref.grouped(h, w2, s2, offsets, None)
    ref.assert_close(each[c], a[c], b[c], "down")
    at = pos.long()
    terms = torch.where(at[:, :, None] >= 0, each[at.clamp_min(0)].double() * p.double()[:, :, None], 0.0)
    # one fused multiply-add a slot, half a unit of 2^-23 of the magnitudes summed each
    ref.assert_close(y, terms.sum(1), topk * 2.0 ** -24 * terms.abs().sum(1), "combine")
    assert api.device_error() == 0


@pytest.mark.parametrize("t,topk,experts,d,i", [(1, 8, 64, 512, 256), (1, 1, 1, 128, 128), (25, 8, 64, 640, 256), (130, 3, 9, 384, 640),
                                                (700, 6, 8, 512, 384)])
@pytest.mark.parametrize("fmt,drop", [("block", 0.0), ("row", 0.2)])
def test_moe_ffn(t, topk, experts, d, i, fmt, drop):
    check_moe(t, topk, experts, d, i, fmt, drop, 60 + t)


@pytest.mark.parametrize("t", [2, 40, 150, 600])
def test_workspace_may_hold_anything(t):
    topk, experts, d, i = 4, 8, 384, 256
    x = ref.activations(t, d, 64, DEV)
    (w1, s1), (w2, s2) = ref.weights(experts, 2 * i, d, "block", 65, DEV), ref.weights(experts, d, i, "block", 66, DEV)
    ids, p = random_ids(t, topk, experts, 67, 0.2), torch.rand(t, topk, device=DEV)
    offsets, rows, _ = api.moe_route(ids, experts)
    moe, gu = [], []
    for fill in (0, 255):
        work = torch.full((api.moe_ffn_workspace_bytes(t, topk, experts, d, i),), fill, dtype=torch.uint8, device=DEV)
        moe.append(api.moe_ffn(x, ids, p, w1, s1, w2, s2, workspace=work))
        work = torch.full((api.grouped_linear_workspace_bytes(t, t * topk, experts, 2 * i, d),), fill, dtype=torch.uint8, device=DEV)
        gu.append(api.grouped_linear(x, w1, s1, offsets, rows=rows, workspace=work))
    assert torch.equal(moe[0].view(torch.int16), moe[1].view(torch.int16))
    assert torch.equal(gu[0].view(torch.int16), gu[1].view(torch.int16))


@pytest.mark.parametrize("t", [9, 150])
def test_same_expert_chosen_twice(t):
    """Choices that repeat an expert each count: two slots of half the weight are one of the whole."""
    experts, d, i = 6, 256, 128
    x = ref.activations(t, d, 55, DEV)
    (w1, s1), (w2, s2) = ref.weights(experts, 2 * i, d, "row", 56, DEV), ref.weights(experts, d, i, "row", 57, DEV)
    one = torch.randint(0, experts, (t, 1), device=DEV).int()
    y1 = api.moe_ffn(x, one, torch.ones(t, 1, device=DEV), w1, s1, w2, s2)
    y2 = api.moe_ffn(x, one.repeat(1, 2), torch.full((t, 2), 0.5, device=DEV), w1, s1, w2, s2)
    assert torch.equal(y1.view(torch.int16), y2.view(torch.int16))


def test_moe_ffn_of_dropped_slots_is_zero():
    t, topk, experts, d, i = 20, 4, 8, 256, 128
    w1, s1 = ref.weights(experts, 2 * i, d, "block", 71, DEV)
    w2, s2 = ref.weights(experts, d, i, "block", 72, DEV)
    ids = torch.full((t, topk), -1, dtype=torch.int32, device=DEV)
    out = torch.full((t, d), 3.0, dtype=torch.bfloat16, device=DEV)
    api.moe_ffn(ref.activations(t, d, 73, DEV), ids, torch.ones(t, topk, device=DEV), w1, s1, w2, s2, out=out)
    assert bool((out == 0).all())


def test_moe_layers_in_a_captured_graph():
    """Three layers in a row, as a decoder runs them, captured once with one workspace and replayed on new tokens."""
    t, topk, experts, d, i = 17, 4, 16, 512, 256
    layers = [(ref.weights(experts, 2 * i, d, "block", 80 + n, DEV), ref.weights(experts, d, i, "block", 90 + n, DEV)) for n in range(3)]
    x = ref.activations(t, d, 81, DEV)
    ids = random_ids(t, topk, experts, 82)
    p = torch.rand(t, topk, device=DEV)
    work = torch.empty(api.moe_ffn_workspace_bytes(t, topk, experts, d, i), dtype=torch.uint8, device=DEV)

    def step():
        h = x
        for (w1, s1), (w2, s2) in layers:
            h = (h + api.moe_ffn(h, ids, p, w1, s1, w2, s2, workspace=work) * 1e-2).contiguous()
        return h

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    for seed in (83, 84):
        x.copy_(ref.activations(t, d, seed, DEV))
        ids.copy_(random_ids(t, topk, experts, seed + 5, 0.2))
        graph.replay()
        replayed = got.clone()
        want = step()
        torch.cuda.synchronize()
        assert torch.equal(replayed.view(torch.int16), want.view(torch.int16))
    assert api.device_error() == 0


# ---------------------------------------------------- a row by itself --

@pytest.mark.parametrize("fmt", ["block", "row"])
@pytest.mark.parametrize("n,k", [(384, 512), (1280, 4096)])
def test_rows_have_the_same_bits_in_every_batch(n, k, fmt):
    """Up to K = 4096 the K blocks are never split (whole tiles idle 32 K blocks at most): a row's sum is then taken in
    one order, by whichever kernel its batch calls for, the plain projection's prefill kernel among them."""
    x = ref.activations(400, k, 53, DEV)
    codes, scale = ref.weights(1, n, k, fmt, 54, DEV)
    want = api.grouped_linear(x, codes, scale, offsets_of([400]))  # rows on M
    y, err = ref.product(ref.quantized(x), ref.weight_value(codes[0], scale[0]))
    ref.assert_close(want, y, err)
    assert torch.equal(want.view(torch.int16), api.linear(x, codes[0], scale[0]).view(torch.int16)), "plain"
    for m in (1, 31, 32, 56, 57, 100, 152, 153, 256):  # blocks of 64, of 160, rows on M
        got = api.grouped_linear(x[:m], codes, scale, offsets_of([m]))
        assert torch.equal(got.view(torch.int16), want[:m].view(torch.int16)), f"{m} rows"
    # the same rows as one expert's of three, unevenly, in a plan that calls for another kernel
    three, ts = codes.repeat(3, 1, 1), scale.repeat(3, *[1] * (scale.dim() - 1))
    for sizes in ([1, 399, 0], [130, 20, 250], [7, 60, 333]):
        got = api.grouped_linear(x, three, ts, offsets_of(sizes))
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), sizes


@pytest.mark.parametrize("rows_per", [3, 100, 300])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
def test_a_rows_nan_stays_in_its_row(rows_per, value):
    experts, n, k = 4, 384, 640
    x = ref.activations(experts * rows_per, k, 57, DEV)
    codes, scale = ref.weights(experts, n, k, "block", 58, DEV)
    off = offsets_of([rows_per] * experts)
    want = api.grouped_linear(x, codes, scale, off)
    bad = [1, rows_per, 2 * rows_per + 2, experts * rows_per - 1]
    hurt = x.clone()
    hurt[bad[0], 3] = hurt[bad[1], 600] = value
    hurt[bad[2:]] = value
    got = api.grouped_linear(hurt, codes, scale, off)
    keep = torch.ones(x.shape[0], dtype=torch.bool, device=DEV)
    keep[bad] = False
    assert torch.equal(want[keep].view(torch.int16), got[keep].view(torch.int16))
    # and through the whole layer: a token's NaN stays in the token
    w1, s1 = ref.weights(experts, 512, k, "block", 59, DEV)
    w2, s2 = ref.weights(experts, k, 256, "block", 60, DEV)
    ids, p = random_ids(x.shape[0], 2, experts, 61), torch.rand(x.shape[0], 2, device=DEV)
    a = api.moe_ffn(x, ids, p, w1, s1, w2, s2)
    b = api.moe_ffn(hurt, ids, p, w1, s1, w2, s2)
    assert torch.equal(a[keep].view(torch.int16), b[keep].view(torch.int16))
    assert api.device_error() == 0


def test_many_rows():
    """More rows than a grid's second axis could count, groups of half a million of them."""
    sizes = [1 << 19, 0, 1, (1 << 19) - 77]
    x = ref.activations(sum(sizes), 128, 62, DEV)
    codes, scale = ref.weights(len(sizes), 128, 128, "block", 63, DEV)
    check_grouped(x, codes, scale, offsets_of(sizes), None)
    check_moe(70001, 2, 5, 128, 128, "block", 0.1, 64)


def test_two_graphs_share_a_workspace():
    """Two captured layers of other sizes with one workspace, replayed in turn: neither finds anything of the other's."""
    parts = []
    need = 0
    for t, topk, experts, d, i, seed in ((9, 4, 16, 512, 256, 70), (300, 2, 3, 17408, 128, 71)):
        (w1, s1), (w2, s2) = ref.weights(experts, 2 * i, d, "block", seed, DEV), ref.weights(experts, d, i, "block", seed + 5, DEV)
        x, ids, p = ref.activations(t, d, seed, DEV), random_ids(t, topk, experts, seed, 0.2), torch.rand(t, topk, device=DEV)
        parts.append([x, ids, p, w1, s1, w2, s2])
        need = max(need, api.moe_ffn_workspace_bytes(t, topk, experts, d, i))
    work = torch.empty(need, dtype=torch.uint8, device=DEV)
    want = [api.moe_ffn(*a) for a in parts]
    graphs, outs = [], [torch.empty_like(w) for w in want]
    for a, out in zip(parts, outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            api.moe_ffn(*a, workspace=work, out=out)
    for turn in (0, 1, 1, 0, 1, 0, 0):
        outs[turn].zero_()
        graphs[turn].replay()
        assert torch.equal(outs[turn].view(torch.int16), want[turn].view(torch.int16))
    assert api.device_error() == 0


def test_layer_in_place():
    """The layer reads x before it writes y: the output may take the input's place."""
    t, topk, experts, d, i = 150, 3, 6, 384, 256
    (w1, s1), (w2, s2) = ref.weights(experts, 2 * i, d, "block", 76, DEV), ref.weights(experts, d, i, "block", 77, DEV)
    x, ids, p = ref.activations(t, d, 78, DEV), random_ids(t, topk, experts, 79, 0.1), torch.rand(t, topk, device=DEV)
    want = api.moe_ffn(x, ids, p, w1, s1, w2, s2)
    api.moe_ffn(x, ids, p, w1, s1, w2, s2, out=x)
    assert torch.equal(x.view(torch.int16), want.view(torch.int16))
