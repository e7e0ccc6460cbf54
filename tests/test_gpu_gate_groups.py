"""moe_gate among groups of experts that only 64 bits tell apart, against the plain 64-bit form: ids and counts equal,
weights within half a step of fp32."""
import numpy as np
import pytest

import quantized_expert_gemv_sigmoid_amd as moe
from test_gpu_gate import check

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


def close_groups(T, G, size, B, score, seed):
    """Logits and biases of G groups whose two experts of the largest c have biases +B and -B and sums of scores that lie
    0.1 to 2 times 2^-24 B apart: nearer than the roundings of two fp32 values of B, further than those of doubles."""
    rng = np.random.default_rng(seed)
    bias = np.full((G, size), -4.0 * B, np.float32)
    bias[:, 0], bias[:, 1] = B, -B
    logits = rng.standard_normal((T, G, size)).astype(np.float32)
    # (softmax: e^l in the place of the score, a group's sum 2 of about 2 G; both sums stay within a quarter of their mean)
    apart = min(2.0 ** -24 * B * (1 if score == 0 else 2 * G), 0.12)
    for t in range(T):
        for g in range(G):
            first, want = rng.uniform(0.3, 0.7), 1.0 + rng.uniform(0.1, 2.0) * rng.choice([-1, 1]) * apart
            if score == 0:
                pair = np.array([first, want - first])
                logits[t, g, :2] = np.log(pair / (1 - pair))
            else:
                logits[t, g, :2] = np.log(2.0 * np.array([first, want - first]))
    return logits.reshape(T, -1), bias.reshape(-1)


@pytest.mark.parametrize("B", [128.0, 1e3, 1e4, 1e6])
@pytest.mark.parametrize("G,size,top", [(2, 2, 1), (4, 2, 1), (8, 3, 3), (64, 2, 20)])
@pytest.mark.parametrize("score", [moe.SCORE_SIGMOID, moe.SCORE_SOFTMAX])
def test_groups_of_two_that_nearly_cancel(B, G, size, top, score):
    print(f"case: B={B} G={G} size={size} top={top} score={score}", flush=True)
    logits, bias = close_groups(200, G, size, B, score, int(B) + G)
    check(torch.as_tensor(logits).cuda(), 2 * top, bias, score=score, n_groups=G, top_groups=top, group_score=moe.GROUP_TOP2)


def test_groups_of_two_forced_on_and_off():
    bias = np.array([1e4, -1e4, 1e4, -1e4], np.float32)
    logits = torch.tensor([[-1.1433, 2.0082, -0.0998, 0.6138]], device="cuda")
    check(logits, 2, bias, n_groups=2, top_groups=1, group_score=moe.GROUP_TOP2)
    # the largest finite biases: sums past fp32's range, and of opposite signs
    for pairs in ((3e38, 3e38, 3e38, 3e38), (3e38, -3e38, 3e38, -3e38), (-3e38, -3e38, -3e38, -3e38), (3e38, 3.1e38, 3.2e38, 3.2e38),
                  (-3.1e38, -3e38, -3e38, -3e38), (-3e38, -3e38, -np.inf, -1e38), (-np.inf, -np.inf, -3e38, -3e38)):
        check(logits, 2, np.array(pairs, np.float32), n_groups=2, top_groups=1, group_score=moe.GROUP_TOP2)
