"""moe_select where the order rests on what fp32 does not show, against the
64-bit definition (ops_ref.select)."""
import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no GPU visible", allow_module_level=True)

import routed_expert_ffn_moe_amd as moe  # noqa: E402
from test_ops_gpu import check_select, gen, run_select  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("logits,bias,k,score", [
    ([17.0, 17.0, 17.125], 0.0, 1, "sigmoid"),            # one fp32 key, 64-bit ones apart
    ([40.0, 50.0, 50.0], None, 1, "sigmoid"),             # equal 64-bit scores: the lowest index
    ([0.0, -20.0, -20.0, -19.875], 0.5, 2, "softmax"),    # scores far below the bias's rounding
    ([17.0, 3.0, 17.0, 17.125, 17.125], 0.0, 2, "sigmoid"),
    ([0.0, -690.0, -680.0, -680.0], None, 2, "softmax"),  # scores near the smallest 64-bit ones
    ([5.0, 5.0, 5.0, 5.0], None, 4, "sigmoid"),           # nothing behind the last place
])
def test_equal_scores_on_the_last_place(logits, bias, k, score):
    l = torch.tensor([logits], dtype=BF)
    check_select(l, None if bias is None else torch.full((len(logits),), bias), k, score=score)
    check_select(l.float(), None if bias is None else torch.full((len(logits),), bias), k, score=score)
    # the same among others that are far below
    wide = torch.full((1, 150), -3.0 if score == "sigmoid" else -700.0)
    wide[0, 20:20 + len(logits)] = l[0].float()
    check_select(wide, None if bias is None else torch.full((150,), bias), k, score=score)


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("bias", [None, "zero", "equal", "few"])
@pytest.mark.parametrize("ng,tg", [(1, 1), (8, 3)])
def test_few_distinct_scores(score, bias, ng, tg):
    """Rows of a few values whose fp32 keys are equal or next to equal."""
    g = gen(ng + len(bias or ""))
    v = torch.tensor([16.5, 17.0, 17.125, 17.25, 40.0, 50.0] if score == "sigmoid" else
                     [-20.0, -19.875, -19.75, -18.0, -17.5, 2.0])
    b = {None: None, "zero": torch.zeros(64), "equal": torch.full((64,), 0.25),
         "few": torch.tensor([0.0, 0.125, 0.25])[torch.randint(0, 3, (64,), generator=g)]}[bias]
    for n in (2, 3, 6):
        l = v[torch.randint(0, n, (40, 64), generator=g)]
        for k in (1, 3, 8):
            check_select(l.to(BF), b, k, "%d values, k=%d" % (n, k), score=score, n_group=ng, topk_group=tg,
                         group_score="top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("size", [1e2, 1e4, 1e6])
def test_group_keys_that_cancel(score, size):
    """Groups valued by the sum of two keys near +size and -size: the sum is of the
    scores' size, the rounding of the fp32 keys of theirs.  Biases are powers of two
    apart from the scores, so that 64-bit sums are exact to 1e-9."""
    g = gen(int(size))
    T, ng, per = 64, 8, 8
    l = torch.randn(T, ng * per, generator=g)
    b = torch.full((ng, per), -4 * size)
    b[:, 2], b[:, 5] = size, -size
    check_select(l, b.reshape(-1), 4, "size %g" % size, score=score, n_group=ng, topk_group=3, group_score="top2")
    # one group of such keys among ordinary ones
    c = torch.randn(ng, per, generator=g) * 0.1
    c[3] = b[3]
    check_select(l, c.reshape(-1), 4, "one of size %g" % size, score=score, n_group=ng, topk_group=3,
                 group_score="top2")


@pytest.mark.parametrize("score", ["sigmoid", "softmax"])
@pytest.mark.parametrize("renorm", [True, False])
def test_scores_below_the_smallest_fp32_value(score, renorm):
    """The selected scores are near e^-100 (softmax: all but one of them)."""
    g = gen(9)
    l = -100 + torch.randn(20, 48, generator=g)
    if score == "softmax":
        l[:, 5] = 0
    for b in (None, torch.randn(48, generator=g) * 0.1):
        check_select(l, b, 6, score=score, renorm=renorm)
        check_select(l, b, 6, score=score, renorm=renorm, n_group=6, topk_group=3, group_score="top2")
    # sums of scores from e^-80 to e^-700, and weights scaled up again
    for low in (-80.0, -87.0, -89.0, -104.0, -300.0, -690.0):
        check_select(low + torch.randn(8, 48, generator=g), None, 6, score=score, renorm=renorm)


def test_renormalised_weights_of_small_scores_sum_to_the_scale():
    idx, w = run_select((-95 - torch.arange(32.0)).view(1, 32).cuda(), None, 4, score="sigmoid", scale=2.5)
    assert idx.tolist() == [[0, 1, 2, 3]]
    assert abs(float(w.double().sum()) - 2.5) < 4 * 2.5 * 2.0 ** -24


def test_more_tokens_than_one_launch_takes():
    """70 million tokens: a wave each are more threads than a launch may have."""
    T = 70 * 10 ** 6
    l = torch.randint(-5, 6, (T, 2), dtype=torch.int8, device="cuda").to(BF)
    idx = torch.full((T + 1, 1), -7, dtype=torch.int32, device="cuda")
    w = torch.full((T + 1, 1), -7.0, device="cuda")
    moe.moe_select(moe.make_select(T, 2, 1, logits="bf16", renorm=False, score="sigmoid"), l, None, idx, w)
    torch.cuda.synchronize()
    assert int(idx[T]) == -7 and float(w[T]) == -7
    assert torch.equal(idx[:T, 0], (l[:, 1] > l[:, 0]).to(torch.int32))
    want = torch.sigmoid(l.amax(1).float())  # 11 different values
    assert float((w[:T, 0] - want).abs().max()) <= 2.0 ** -19
