"""The routing operators (MoERouter) against their definition in 64 bits."""
import numpy as np
import pytest

import _ops_ref as ref

pytestmark = pytest.mark.gpu


def settings(E, k, score="softmax", groups=1, kept=1, group_score="top2", renorm=True, scale=1.0):
    return dict(E=E, k=k, score=score, groups=groups, groups_kept=kept, group_score=group_score,
                renormalise=renorm, scale=scale)


def make(r):
    from persistent_megakernel_sm_gb300 import MoERouter
    return MoERouter(**r)


def dev(a, dtype=None):
    import torch
    t = torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).cuda()
    return t if dtype is None else t.to(dtype)


def forward(r, l, bias=None, dtype=None, counts=True):
    import torch
    T = len(l)
    logits = l if hasattr(l, "cuda") else dev(l, dtype)
    idx = torch.full((T, r["k"]), 77, dtype=torch.int32, device="cuda")
    w = torch.full((T, r["k"]), 77.0, device="cuda")
    c = torch.full((r["E"],), 77, dtype=torch.int32, device="cuda") if counts else None
    router = make(r)
    router.forward(logits, idx, w, bias=None if bias is None else dev(bias), counts=c)
    torch.cuda.synchronize()
    return idx.cpu().numpy(), w.cpu().numpy().astype(np.float64), None if c is None else c.cpu().numpy()


def weight_tolerance(l):
    """expf within 2 steps, its argument's rounding (|l - m| half steps, the
    spread at most), a sum of at most 8 + 5 additions twice over, a division and
    two products: under 24 half steps and the spread; the smallest numbers are
    flushed below 2^-126."""
    fin = np.where(np.isfinite(l), l, 0.0)
    spread = np.minimum(fin.max(1) - fin.min(1) + np.abs(fin).max(1), 200)
    return ((24 + 2 * spread) * ref.U32)[:, None]


def check(r, l, bias=None, dtype=None):
    idx, w, counts = forward(r, l, bias, dtype)
    want_idx, want_w = ref.route(l, r, bias)
    assert np.array_equal(idx, want_idx)
    assert np.all(np.abs(w - want_w) <= weight_tolerance(l) * np.abs(want_w) + 2.0 ** -126 * abs(r["scale"]))
    assert np.array_equal(counts, np.bincount(want_idx[want_idx >= 0], minlength=r["E"]))


CASES = [
    # T, settings, bias
    (1, settings(1, 1), False),
    (3, settings(5, 5, "sigmoid", renorm=False), False),
    (1, settings(256, 8, "sigmoid", 8, 4, scale=2.5), True),
    (33, settings(256, 8, "sigmoid", 8, 4, scale=2.5), True),
    (70, settings(160, 6, "softmax", 8, 3, "max", renorm=False, scale=16.0), False),
    (40, settings(64, 6, "softmax", renorm=False), True),
    (40, settings(64, 6, "softmax"), True),
    (17, settings(128, 16, "sigmoid"), False),
    (9, settings(60, 4, "sigmoid", 3, 2, "max", renorm=False), True),
    (9, settings(36, 3, "softmax", 12, 5), False),
    (20, settings(96, 1, "sigmoid", 32, 31), True),
    (12, settings(33, 7, "softmax", renorm=False), False),
    (300, settings(8, 2), False),
    (11, settings(32, 4, "sigmoid", 32, 9, "top2"), True),   # groups of one expert
    (11, settings(34, 4, "sigmoid", 2, 1, "top2"), False),
]


@pytest.mark.parametrize("case", range(len(CASES)))
def test_forward_fp32(case):
    T, r, biased = CASES[case]
    rng = np.random.default_rng(100 + case)
    bias = (0.1 * rng.standard_normal(r["E"])).astype(np.float32).astype(np.float64) if biased else None
    check(r, ref.clear_logits(rng, T, r, bias), bias)


@pytest.mark.parametrize("case", [0, 3, 4, 5, 6, 9, 11])
def test_forward_bf16_logits(case):
    import torch
    T, r, biased = CASES[case]
    rng = np.random.default_rng(200 + case)
    bias = (0.1 * rng.standard_normal(r["E"])).astype(np.float32).astype(np.float64) if biased else None
    check(r, ref.clear_logits(rng, T, r, bias, to=ref.bf16), bias, torch.bfloat16)


@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("biased", [False, True])
def test_masked_experts_and_rows(biased, group_score):
    rng = np.random.default_rng(7)
    r = settings(64, 8, "sigmoid", 8, 3, group_score)
    bias = (0.1 * rng.standard_normal(64)).astype(np.float32).astype(np.float64) if biased else None
    l = ref.clear_logits(rng, 24, r, bias, masked=0.6)
    l[3] = -np.inf                       # a row of nothing
    l[5] = -np.inf
    l[5, 17] = 0.25                      # a row of one expert
    l[6, :] = -np.inf
    l[6, [1, 9, 40]] = [1.0, 2.0, 3.0]   # fewer than k, in groups of one each
    check(r, l, bias)


def test_bias_of_minus_infinity_masks():
    rng = np.random.default_rng(8)
    r = settings(16, 4, "sigmoid")
    bias = (0.1 * rng.standard_normal(16)).astype(np.float32).astype(np.float64)
    l = ref.clear_logits(rng, 10, r, bias)
    bias[[0, 3, 5]] = -np.inf
    check(r, l, bias)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_ties_go_to_the_lower_expert_and_extremes_stay_finite(score, renorm):
    low = float(np.finfo(np.float32).min)
    l = np.zeros((7, 40))
    l[1] = low                                     # the type's lowest value everywhere: a tie, not a mask
    l[2] = -300.0
    l[2, 7] = -299.0
    l[3, ::2] = 80.0
    l[4] = np.repeat(np.arange(10.0), 4)           # ties of four
    l[5, 5] = -0.0                                 # both zeros are equal
    l[6, :20] = low
    r = settings(40, 6, score, renorm=renorm, scale=0.5)
    check(r, l)


@pytest.mark.parametrize("E,k", [(256, 8), (256, 16), (130, 5), (100, 16), (64, 6), (60, 16), (32, 3), (20, 16), (7, 7)])
def test_rows_of_many_equal_logits(E, k):
    """From no candidate beyond k to all experts alike, rows of both beside each
    other in a warp."""
    rng = np.random.default_rng(E + k)
    l = rng.integers(0, 4, (61, E)).astype(np.float64)
    l[::7] = rng.permuted(np.tile(np.arange(float(E)), (len(l[::7]), 1)), axis=1)   # none alike
    l[1::7] = 0.5                                                                  # all alike
    l[2::7, : E // 2] = -np.inf
    l[3::7, k // 2 :] = -np.inf                                                    # fewer than k
    l[4::7] = np.sort(l[4::7], axis=1)                                             # the best in a few lanes
    l[5::7] = np.arange(float(E))
    check(settings(E, k), l)


@pytest.mark.parametrize("E,groups", [(256, 32), (256, 16), (256, 8), (256, 2), (64, 4), (128, 16), (24, 3), (96, 4),
                                      (192, 8), (200, 5), (32, 2)])
@pytest.mark.parametrize("group_score", ["max", "top2"])
def test_groups_of_whole_lanes_and_others(E, groups, group_score):
    rng = np.random.default_rng(E + groups)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32).astype(np.float64)
    kept = max(1, groups // 2)
    k = min(6, E // groups * kept)
    for biased in (False, True):
        for score in ("softmax", "sigmoid"):
            r = settings(E, k, score, groups, kept, group_score)
            b = bias if biased else None
            check(r, ref.clear_logits(rng, 19, r, b, masked=0.3), b)
    # equal groups: the lower ones are kept
    r = settings(E, k, "sigmoid", groups, kept, group_score)
    check(r, np.zeros((3, E)))


def test_nan_and_infinite_logits_show():
    l = np.zeros((3, 40))
    l[0, 9] = np.nan
    l[1, 30] = np.inf
    l[2, 31] = np.inf
    idx, w, _ = forward(settings(40, 3, "softmax"), l)
    assert idx[0].tolist() == [9, 0, 1] and np.isnan(w[0]).all()
    assert idx[1].tolist() == [30, 0, 1] and np.isnan(w[1]).any()
    idx, w, _ = forward(settings(40, 3, "sigmoid", renorm=False), l)
    assert idx[2].tolist() == [31, 0, 1] and w[2].tolist() == [1.0, 0.5, 0.5]
    assert idx[0].tolist() == [9, 0, 1] and np.isnan(w[0, 0]) and w[0, 1:].tolist() == [0.5, 0.5]


def test_rows_of_a_wider_buffer_and_unaligned_rows():
    import torch
    rng = np.random.default_rng(9)
    for E, pad, first, dtype in ((64, 8, 0, torch.float32), (64, 3, 0, torch.float32), (64, 9, 1, torch.bfloat16),
                                 (61, 4, 2, torch.float32), (256, 16, 8, torch.bfloat16)):
        r = settings(E, 5, "softmax", renorm=False)
        wide = torch.full((50, E + pad), float("nan"), dtype=dtype, device="cuda")
        l = ref.bf16(rng.standard_normal((50, E)))
        wide[:, first:first + E] = dev(l, dtype)
        idx, w, counts = forward(r, wide[:, first:first + E])
        want_idx, want_w = ref.route(l, r)
        assert np.array_equal(idx, want_idx)
        assert np.all(np.abs(w - want_w) <= weight_tolerance(l) * want_w)
        assert counts.sum() == 250


def test_rows_over_four_gigabytes_apart():
    """Offsets that pass 32 bits, forward and back."""
    import torch
    r = settings(64, 6)
    wide = torch.empty(3, (1 << 31) + 64, dtype=torch.bfloat16, device="cuda")
    rng = np.random.default_rng(31)
    l = ref.clear_logits(rng, 3, r, None, to=ref.bf16)
    view = wide[:, :64]
    view.copy_(dev(l, torch.bfloat16))
    idx, w, counts = forward(r, view)
    want_idx, want_w = ref.route(l, r, None)
    assert np.array_equal(idx, want_idx)
    assert np.all(np.abs(w - want_w) <= weight_tolerance(l) * np.abs(want_w))
    grad = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    far = wide[:, 64:128]
    args = torch.from_numpy(idx).cuda(), dev(rng.standard_normal((3, 6)))
    make(r).backward(view, *args, grad)
    make(r).backward(view, *args, far)
    torch.cuda.synchronize()
    assert torch.equal(grad, far) and grad.abs().max() > 0


def test_no_rows_and_no_counts():
    import torch
    r = settings(64, 4)
    idx, w, counts = forward(r, np.zeros((0, 64)))
    assert idx.shape == (0, 4) and np.array_equal(counts, np.zeros(64))
    l = np.random.default_rng(1).standard_normal((5, 64)).astype(np.float32)
    idx, w, counts = forward(r, l, counts=False)
    assert counts is None and np.array_equal(idx, ref.route(l, r)[0])
    empty = torch.empty(0, 64, device="cuda")
    make(r).backward(empty, torch.empty(0, 4, dtype=torch.int32, device="cuda"), torch.empty(0, 4, device="cuda"), empty.clone())


def test_long_batch_counts_every_token():
    """More rows than the grid holds at once; counts by several blocks."""
    import torch
    rng = np.random.default_rng(11)
    T = 30011
    r = settings(64, 6, "softmax", renorm=False)
    l = rng.standard_normal((T, 64)).astype(np.float32)
    idx, w, counts = forward(r, l)
    assert np.array_equal(idx, np.argsort(-l, axis=1, kind="stable")[:, :6])
    assert np.array_equal(counts, np.bincount(idx.ravel(), minlength=64))
    p = torch.softmax(torch.from_numpy(l).double(), 1).numpy()
    want = np.take_along_axis(p, idx.astype(np.int64), 1)
    assert np.all(np.abs(w - want) <= weight_tolerance(l) * want)


# ------------------------------------------------------------------- gradient

GRADS = [
    (1, settings(1, 1)),
    (5, settings(64, 6, "softmax", renorm=False)),
    (33, settings(256, 8, "softmax", renorm=False, scale=2.5)),
    (33, settings(256, 8, "sigmoid", scale=2.5)),
    (19, settings(60, 4, "sigmoid", renorm=False)),
    (19, settings(128, 16, "softmax")),
    (7, settings(33, 3, "softmax", renorm=False)),
    (10000, settings(8, 2, "sigmoid")),
]


def backward(r, l, idx, gw, dtype=None, grad=None):
    import torch
    logits = dev(l, dtype)
    grad = torch.full_like(logits, 77.0) if grad is None else grad
    make(r).backward(logits, torch.from_numpy(np.ascontiguousarray(idx, dtype=np.int32)).cuda(), dev(gw), grad)
    torch.cuda.synchronize()
    return grad.float().cpu().numpy().astype(np.float64)


def grad_close(got, l, r, idx, gw, half_step):
    want, size = ref.route_grad(l, r, idx, gw)
    # the weights' error (twice: the share and 1 - s) and the sums over k slots
    tol = (2 * weight_tolerance(l) + 2 * (r["k"] + 4) * ref.U32) * size + half_step * np.abs(want) + 2.0 ** -126
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("case", range(len(GRADS)))
def test_backward(case, bf16):
    import torch
    T, r = GRADS[case]
    rng = np.random.default_rng(300 + case)
    T = min(T, 200) if case == 7 and bf16 else T
    l = ref.bf16(rng.standard_normal((T, r["E"])))
    idx = np.argsort(-l, axis=1, kind="stable")[:, :r["k"]]
    gw = rng.standard_normal((T, r["k"])).astype(np.float32).astype(np.float64)
    got = backward(r, l, idx, gw, torch.bfloat16 if bf16 else None)
    grad_close(got, l, r, idx, gw, ref.U16 if bf16 else ref.U32)


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [False, True])
def test_backward_of_masked_empty_and_repeated_slots(score, renorm):
    rng = np.random.default_rng(31)
    r = settings(48, 5, score, renorm=renorm)
    l = rng.standard_normal((8, 48)).astype(np.float32).astype(np.float64)
    l[:, 40:] = -np.inf
    l[2] = -np.inf
    idx = np.argsort(-l, axis=1, kind="stable")[:, :5].astype(np.int32)
    idx[1, 2:] = -1                       # slots without an expert
    idx[2] = -1                           # a row without any
    idx[3] = 7                            # one expert in every slot
    idx[4, :] = [3, 9, 3, 9, 3]
    idx[5, 1] = 48                        # outside
    idx[6, 0] = np.iinfo(np.int32).min
    idx[7, 2:] = [41, 45, 41]             # masked experts
    gw = rng.standard_normal((8, 5)).astype(np.float32).astype(np.float64)
    gw_in = gw.copy()
    gw_in[1, 2:] = np.nan                 # never read into anything
    got = backward(r, l, idx, gw_in)
    grad_close(got, l, r, np.where(idx >= 40, -1, idx), gw, ref.U32)
    assert np.all(got[2] == 0) and np.all(got[:, 40:] == 0)


def test_backward_is_the_differences_of_the_forward():
    """Along random directions, with the step and the fp32 noise of the weights
    in the bound: w's error (24 half steps each) over the step, and the third
    derivative's share of it (scores and shares have derivatives below 1)."""
    rng = np.random.default_rng(41)
    for r in (settings(64, 6, "softmax", renorm=False), settings(64, 6, "sigmoid"), settings(64, 6, "softmax")):
        l = rng.standard_normal((16, 64)).astype(np.float32).astype(np.float64)
        idx, _, _ = forward(r, l)
        gw = rng.standard_normal((16, 6)).astype(np.float32).astype(np.float64)
        grad = backward(r, l, idx, gw)
        h = 2.0 ** -8
        way = np.sign(rng.standard_normal(l.shape))
        # far from the edge of the choice: the kept logits are lifted by 8
        lift = l.copy()
        np.put_along_axis(lift, idx.astype(np.int64), np.take_along_axis(l, idx.astype(np.int64), 1) + 8.0, 1)
        idx, _, _ = forward(r, lift)
        grad = backward(r, lift, idx, gw)
        order = np.argsort(idx, axis=1)
        diffs = []
        for q in (h, -h):
            i2, w2, _ = forward(r, lift + q * way)
            o2 = np.argsort(i2, axis=1)
            assert np.array_equal(np.take_along_axis(i2, o2, 1), np.take_along_axis(idx, order, 1))
            diffs.append((np.take_along_axis(w2, o2, 1) * np.take_along_axis(gw, order, 1)).sum(1))
        diff = (diffs[0] - diffs[1]) / (2 * h)
        size = np.abs(gw).sum(1)
        assert np.all(np.abs(diff - (grad * way).sum(1)) <= size * (64 * ref.U32 / h + 8 * h * h))


def test_backward_into_rows_of_a_wider_buffer_leaves_the_rest():
    import torch
    rng = np.random.default_rng(51)
    r = settings(61, 4, "softmax", renorm=False)
    l = rng.standard_normal((30, 61)).astype(np.float32).astype(np.float64)
    idx = np.argsort(-l, axis=1, kind="stable")[:, :4]
    gw = rng.standard_normal((30, 4)).astype(np.float32).astype(np.float64)
    wide = torch.full((30, 70), 5.0, device="cuda")
    got = backward(r, l, idx, gw, grad=wide[:, 3:64])
    grad_close(got, l, r, idx, gw, ref.U32)
    rest = wide.cpu().numpy()
    assert np.all(rest[:, :3] == 5) and np.all(rest[:, 64:] == 5)


def test_graph_replay_and_side_stream_give_the_same_bits():
    import torch
    rng = np.random.default_rng(61)
    r = settings(256, 8, "sigmoid", 8, 4, scale=2.5)
    bias = dev(0.1 * rng.standard_normal(256))
    a, b = (dev(rng.standard_normal((500, 256))) for _ in range(2))
    gw = dev(rng.standard_normal((500, 8)))
    router = make(r)

    def buffers():
        return (torch.zeros(500, 8, dtype=torch.int32, device="cuda"), torch.zeros(500, 8, device="cuda"),
                torch.zeros(256, dtype=torch.int32, device="cuda"), torch.zeros(500, 256, device="cuda"))

    def both(l, o, stream=None):
        router.forward(l, o[0], o[1], bias=bias, counts=o[2], stream=stream)
        router.backward(l, o[0], gw, o[3], stream=stream)

    want = [buffers(), buffers()]
    both(a, want[0])
    both(b, want[1])
    torch.cuda.synchronize()
    x, got = a.clone(), buffers()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            both(x, got)
    for l, o in ((a, want[0]), (b, want[1]), (a, want[0])):
        x.copy_(l)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, o))
