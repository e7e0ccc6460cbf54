"""moe_gate on rows that leave fewer experts than places, among them chosen ones whose score is NaN: the places left hold
id -1 and weight 0, whatever the renormalisation's sum is."""
import numpy as np
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_gpu_gate import check, logits_of, run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def rows(bias):
    nan, ninf = float("nan"), -float("inf")
    logits = logits_of(4, 96, 19)
    logits[0, 3:] = ninf           # three left, one of them NaN
    logits[0, 1] = nan
    logits[1] = ninf               # the NaN one alone
    logits[1, 77] = nan
    logits[2] = ninf               # as many NaN as groups of 24: their values tie, and are compared in 64 bits
    logits[2, [5, 30, 50, 95]] = nan
    logits[2, [6, 31, 51, 94]] = 0.5
    logits[3, 5:] = ninf           # an infinity and a NaN
    logits[3, 0], logits[3, 4] = float("inf"), nan
    return logits, np.linspace(-0.1, 0.1, 96).astype(np.float32) if bias else None


@pytest.mark.parametrize("score", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
@pytest.mark.parametrize("groups", [1, 4])
@pytest.mark.parametrize("bias", [False, True])
@pytest.mark.parametrize("renorm", [0, 1])
def test_places_left_behind_a_nan(score, groups, bias, renorm):
    print(f"case: score={score} groups={groups} bias={bias} renorm={renorm}", flush=True)
    logits, b = rows(bias)
    kw = dict(score=score, n_groups=groups, top_groups=max(1, groups // 2), renorm=renorm, routed_scale=2.5)
    for group_score in (moe.GROUP_MAX, moe.GROUP_TOP2):
        for T in (4, 40):          # one launch, and two
            l = logits.repeat(T // 4, 1)
            ids, w, _ = run(l, 8, b, group_score=group_score, **kw)
            assert (ids == -1).any() and (w[ids == -1] == 0.0).all()
            check(l, 8, b, group_score=group_score, **kw)
