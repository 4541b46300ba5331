"""Edges of the paged-cache operators on the GPU: orders between units, weights near the types' ends, sizes near
32 bits.  Bounds and helpers are those of test_gpu_paged.
"""
import math

import pytest
import torch

import paged_refs
import test_gpu_paged as base
from test_gpu_paged import sdpa  # noqa: F401  (fixture)

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


# ------------------------------------------------------------------ one unit after the other
@pytest.mark.parametrize("fp8", [False, True], ids=["16_bits", "e4m3"])
def test_units_of_one_tile_behind_units_of_more(sdpa, fp8):  # noqa: F811
    """65 to 128 rows a key/value head: the chains take a unit's key tiles in turn and their sums meet in shared
    memory.  Behind a unit of two or three tiles comes one of a single tile, whose second chain has nothing to wait
    for: it must leave the sums before it alone until they are read.  About eight units a CTA, many times over."""
    b = 600
    lens = [(300, 100, 384, 60, 129, 128)[i % 6] for i in range(b)]
    news = [17 + i % 16 for i in range(b)]
    c = base._attend_case(41 + fp8, lens, news, 8, 2, 128, 16, BF, fp8)
    o, lse = base._call(sdpa, c)
    sdpa.sdpa_check_device_error()
    base._check(c, o, lse)
    for _ in range(60):
        x, y = base._call(sdpa, c)
        assert torch.equal(x, o) and torch.equal(y, lse)


# ------------------------------------------------------------------ weights near the types' ends
@pytest.mark.parametrize("n", [1, 9, 20, 40], ids=["rows_32", "rows_64", "rows_256", "both"])
def test_fp16_weights_far_below_a_sink_of_no_value(sdpa, n):  # noqa: F811
    """The first keys' one takes nearly all the weight and its value is zero, so O comes from 30,000 keys whose
    weights are near 2^-25 of the largest.  152 requests share the pages, so that a CTA sums a long run of keys under
    the sink's maximum.  P is raised by 2^7 at least before it is rounded to fp16: half a step is 2^-11 of a weight,
    and where P is below fp16's normal range 2^-25, which is 2^-32 of the row's largest weight (a weight never loses
    more than itself).  So |dO| <= 2^-11 A + sum_j min(w_ij, 2^-32 max_j w_ij) |v_j|, beside the other terms."""
    size, h, b = 30000, 4, 152
    c = base._attend_case(7, [size], [n], h, 1, 128, 64, HF, tree=False)
    scores = torch.tensor([23.0, 24.5, 25.2, 26.0], dtype=torch.float64) * math.log(2.0)
    q = torch.zeros(n, h, 128, device="cuda")
    q[:, :, 0] = scores.float().cuda()
    c["q"], c["scale"] = q.to(HF), 1.0
    c["kc"][..., 0] = 0.0
    c["vc"] = c["vc"].abs() + 0.5
    sink = c["table"][0][0], 5
    c["kc"][sink[0], 0, sink[1], 0] = 1.0
    c["vc"][sink[0], 0, sink[1]] = 0.0
    k = paged_refs.keys_of(c["kc"].cpu(), c["table"][0], size)[0]
    v = paged_refs.keys_of(c["vc"].cpu(), c["table"][0], size)[0]
    s = torch.einsum("nhd,jd->nhj", c["q"].cpu().double(), k)
    s = s.masked_fill(torch.arange(size)[None, None] > (size - n + torch.arange(n))[:, None, None], -math.inf)
    w = torch.softmax(s, -1)
    ref = w @ v
    least = torch.minimum(w, w.amax(-1, keepdim=True) * 2.0 ** -32) @ v
    big = s.amax().item()
    bound = (2.0 ** -11 + 2 * (big + 16) * 2.0 ** -21) * ref + least + 2.0 ** -11 * ref + 2.0 ** -25
    c["q"], c["table"], c["lens"], c["cu"] = c["q"].repeat(b, 1, 1), c["table"] * b, [size] * b, [n * i for i in range(b + 1)]
    o, lse = base._call(sdpa, c)
    sdpa.sdpa_check_device_error()
    off = ((o.cpu().double().view(b, n, h, 128) - ref).abs() / bound).max().item()
    assert off <= 1.0, f"O is {off:.2f} times its bound off"
    off = (lse.cpu().double().view(b, n, h) - torch.logsumexp(s, -1)).abs().max().item()
    assert off <= (2 * big + 16) * 2.0 ** -21


# ------------------------------------------------------------------ sizes near 32 bits
@pytest.mark.parametrize("bound", [2 ** 31 - 1, 2 ** 31 - 128, 2 ** 24])
def test_a_generous_bound_of_the_lengths(sdpa, bound):  # noqa: F811
    """max_seqlen_kv may be any upper bound."""
    c = base._attend_case(8, [700, 33], [9, 3], 8, 2, 128, 16, BF)
    o, lse = base._call(sdpa, c)
    mask = paged_refs.words_of(c["rows"], c["words"]).cuda()
    x, y = sdpa.attention_tree(c["q"], c["kc"], c["vc"], base._i32(c["table"]), base._i32(c["cu"]), base._i32(c["lens"]),
                               9, bound, tree_mask=mask, scale=c["scale"])
    sdpa.sdpa_check_device_error()
    assert torch.equal(x, o) and torch.equal(y, lse)


def test_plan_takes_back_no_more_pages_than_there_are(sdpa):  # noqa: F811
    """Requests that claim to hold 2^31 - 16 pages in all, sixteen times what exists: the returned pages that the
    ring has room for are taken, in order, and the count of the rest does not wrap."""
    b, blocks = 16, (1 << 27) - 1
    pages = blocks
    ring = torch.full((pages,), -3, dtype=torch.int32, device="cuda")
    table = torch.zeros(b, blocks, dtype=torch.int32, device="cuda")
    table[0, :5] = base._i32([7, 1, 4, 2, 9])
    got = sdpa.cache_plan(base._i32([0] * b), base._i32([-1] * b), base._i32([blocks] * b), base._i32([3, pages - 5, 0]), ring, table, 16, 0)
    torch.cuda.synchronize()
    assert got.ring_state.tolist() == [3, pages, 0] and got.held.tolist() == [0] * b
    assert ring[pages - 2:].tolist() == [7, 1] and ring[:3].tolist() == [4, 2, 9]
    assert (ring[3:pages - 2] == -3).all().item()
    assert table[0, :5].tolist() == [7, 1, 4, 2, 9] and not table[1:].any().item()


# ------------------------------------------------------------------ streams
def _behind_pending_writes(shapes, call):
    """call(other) while the current stream, asleep, still has to write to memory that was freed since."""
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    torch.cuda._sleep(400_000_000)
    pending = [torch.full(shape, 77, dtype=dtype, device="cuda") for shape, dtype in shapes for _ in range(4)]
    del pending
    got = call(other)
    other.synchronize()
    torch.cuda.synchronize()
    return got


def test_outputs_on_another_stream_are_not_what_the_current_one_still_writes(sdpa):  # noqa: F811
    """The outputs that a call allocates are written on `stream`: memory that was freed on the current stream, whose
    writes there are still to come, must not be handed to them."""
    c = base._attend_case(16, [3000, 700, 64], [16, 9, 3], 8, 2, 128, 32, BF)
    o, lse = base._call(sdpa, c)
    mask = paged_refs.words_of(c["rows"], c["words"]).cuda()
    table, cu, lens = base._i32(c["table"]), base._i32(c["cu"]), base._i32(c["lens"])
    size = sdpa.attention_tree_workspace(c["q"], c["kc"], 3, 16, 3000).numel()
    got = _behind_pending_writes([(o.shape, BF), (lse.shape, torch.float32), ((size,), torch.uint8)], lambda other: sdpa.attention_tree(
        c["q"], c["kc"], c["vc"], table, cu, lens, 16, 3000, tree_mask=mask, scale=c["scale"], stream=other))
    assert torch.equal(got[0], o) and torch.equal(got[1], lse)
    # the plan's outputs and the accepted lengths
    args = [base._i32(x) for x in ([5, 40], [20, 3], [1, 3], [0, 4, 0])]
    ring, table = base._i32(list(range(8))), base._i32([[4, -1, -1], [5, 6, 7]])
    want = sdpa.cache_plan(*args, ring.clone(), table.clone(), 16, 23)
    shapes = [(x.shape, torch.int32) for x in want if x is not None]
    got = _behind_pending_writes(shapes, lambda other: sdpa.cache_plan(*args, ring, table, 16, 23, stream=other))
    for x, y in zip(got, want):
        assert x is y is None or torch.equal(x, y)
    ctx, new, path, plen = (base._i32(x) for x in ([5, 40], [20, 3], [[0, 1], [2, -1]], [2, 1]))
    got = _behind_pending_writes([((2,), torch.int32)], lambda other: sdpa.cache_accept(
        c["kc"], c["vc"], table, ctx, new, path, plen, stream=other))
    assert got.tolist() == [7, 41]


def test_outputs_of_another_stream_wait_for_the_current_one(sdpa):  # noqa: F811
    """An output that was read on the current stream and dropped is not handed out on its own before that read."""
    c = base._attend_case(17, [900, 64], [16, 3], 8, 2, 128, 32, BF)
    o, _ = base._call(sdpa, c)
    mask = paged_refs.words_of(c["rows"], c["words"]).cuda()
    table, cu, lens = base._i32(c["table"]), base._i32(c["cu"]), base._i32(c["lens"])
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    got = sdpa.attention_tree(c["q"], c["kc"], c["vc"], table, cu, lens, 16, 900, tree_mask=mask, scale=c["scale"], stream=other)
    torch.cuda.current_stream().wait_stream(other)
    torch.cuda._sleep(400_000_000)
    read = got[0].clone()
    del got
    with torch.cuda.stream(other):
        taken = [torch.full(o.shape, 77, dtype=BF, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(read, o) and all((x == 77).all().item() for x in taken)
