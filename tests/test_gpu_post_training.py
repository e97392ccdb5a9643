"""The post-training operators in one run, as a training step uses them: the
packed head's logits, the reference policy's from an 8-bit head, its token log
probabilities, the loss with its gradient by the logits, and the gradient by
the hidden states -- eagerly, on a side stream and as one captured graph.

Every stage is held to the fp64 oracle on what the GPU gave it; the step's
gradient as a whole to the oracle's own step.  There the logits may be off by
2e-3 rms (the forward's bound), so a probability by a factor exp(+-2 2e-3 rms)
and a coefficient by about as much; with rms below 4 (asserted) that is 3.3 %
of every entry, and the rest (bf16 gradient, fp16 codes) 0.6 %: 4 % in norm.
"""
import numpy as np
import pytest

from gpu_util import say
from oracle import forward, losses
from packed_quantized_lm_amd.synth import random_small_head, to_bf16_bits

pytestmark = pytest.mark.gpu
V, D, M = 3001, 512, 70


@pytest.fixture(scope="module")
def step():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    from packed_quantized_lm_amd import Fp8Head, PackedHead, policy_loss, preference_loss, token_logp, x_tensor_from_bits
    f = random_small_head(V, D, 40, 24, 64, M, seed=21)
    rng = np.random.default_rng(4)
    W = forward.dense_rows(f, np.arange(V))
    X = rng.normal(0, 1, (M, D))
    X *= 3.0 / np.sqrt(((X @ W.T) ** 2).mean())  # logits of rms 3
    f["X"] = to_bf16_bits(X)
    head = PackedHead(f)
    head.reserve(M)
    head.reserve_backward(M)
    ref = Fp8Head(torch.from_numpy(W.astype(np.float32)).cuda().bfloat16())
    s = dict(f=f, W=W, head=head, ref=ref, X=x_tensor_from_bits(f["X"]))
    dev = lambda a, t: torch.from_numpy(np.ascontiguousarray(a)).to("cuda", t)
    s["targets"] = dev(rng.integers(0, V, M), torch.int32)
    s["adv"] = dev(rng.normal(0, 1, M), torch.float32)
    w = (rng.random(M) < 0.9) / M
    s["weights"] = dev(w, torch.float32)
    s["mask"] = dev(w > 0, torch.float32)
    s["offsets"] = dev([0, 11, 30, 30, 47, 61, 66], torch.int32)
    y, _ = head.forward(s["X"])
    s["old"] = token_logp(y, s["targets"])[0] + dev(rng.normal(0, 0.05, M), torch.float32)

    def policy():
        logits, _ = head.forward(s["X"])
        ref_logp, _ = token_logp(ref.forward(s["X"]), s["targets"])
        loss, logp, dy = policy_loss(logits, s["targets"], s["old"], s["adv"], s["weights"], ref_logp, beta=0.05,
                                     grad_dtype=torch.bfloat16)
        return loss, logp, ref_logp, dy, head.backward(dy), logits

    def preference():
        logits, _ = head.forward(s["X"])
        ref_logp, _ = token_logp(ref.forward(s["X"], out_dtype=torch.bfloat16), s["targets"])
        loss, margins, logp, dy = preference_loss(logits, s["targets"], s["mask"], s["offsets"], ref_logp, beta=0.3,
                                                  grad_dtype=torch.float32)
        return loss, margins, logp, dy, head.backward(dy), logits
    s["policy"], s["preference"] = policy, preference
    yield s
    head.close()


def num(t):
    return t.double().cpu().numpy()


def close(got, want, rel):
    return np.linalg.norm(got - want) <= rel * np.linalg.norm(want)


def test_policy_step(step):
    say("post-training: policy step")
    loss, logp, ref_logp, dy, dX, logits = (num(t) for t in step["policy"]())
    t, f = step["targets"].cpu().numpy(), step["f"]
    assert np.sqrt((logits ** 2).mean()) < 4
    args = (num(step["old"]), num(step["adv"]), num(step["weights"]))
    # the stages, each on what the GPU gave it
    l64, lp64, g64, _ = losses.policy(logits, t, *args, ref_logp, 0.05)
    assert abs(loss - l64) < 1e-5 and np.abs(logp - lp64).max() < 1e-5
    assert close(dy, g64, 2.0 ** -8)
    assert close(dX, dy @ step["W"], 2.0 ** -8 + 2.0 ** -10)
    # the 8-bit reference: e4m3 codes of both operands are off by 2^-4 at most, which
    # 512 terms of either sign bring to well below 2^-4 of the logits' rms
    ref64 = losses.token_logp(forward.forward(f, f["X"]), t)
    assert np.abs(ref_logp - ref64).max() < 1.0 and np.abs(ref_logp - ref64).mean() < 0.25
    # the whole step
    _, _, g, _ = losses.policy(forward.forward(f, f["X"]), t, *args, ref_logp, 0.05)
    assert close(dX, g @ step["W"], 0.04)


def test_preference_step(step):
    say("post-training: preference step")
    loss, margins, logp, dy, dX, logits = (num(t) for t in step["preference"]())
    t, off = step["targets"].cpu().numpy(), step["offsets"].cpu().numpy()
    ref_logp = None
    from packed_quantized_lm_amd import token_logp
    import torch
    ref_logp = num(token_logp(step["ref"].forward(step["X"], out_dtype=torch.bfloat16), step["targets"])[0])
    l64, h64, _, g64, _ = losses.preference(logits, t, num(step["mask"]), off, ref_logp, 0.3)
    assert abs(loss - l64) < 1e-5 and np.abs(margins - h64).max() < 1e-4
    assert close(dy, g64, 1e-5)
    assert close(dX, dy @ step["W"], 2.0 ** -8 + 2.0 ** -10)
    assert not dX[66:].any()  # rows behind the last answer


def test_gradient_descends(step):
    """A small step against dX lowers the loss by its norm squared times the
    step, within the bf16 hidden states' rounding: the sign and size of the
    whole chain's gradient.  The loss is taken in fp64 at the moved states."""
    loss, _, ref_logp, _, dX, _ = (num(t) for t in step["policy"]())
    f, t = step["f"], step["targets"].cpu().numpy()
    X = num(step["X"])
    args = (num(step["old"]), num(step["adv"]), num(step["weights"]), ref_logp, 0.05)
    value = lambda x: losses.policy(x @ step["W"].T, t, *args)[0]
    n2 = (dX ** 2).sum()
    eta = 1e-4 * np.linalg.norm(X) / np.sqrt(n2)
    fall = (value(X + eta * dX) - value(X - eta * dX)) / (2 * eta)
    assert abs(fall - n2) <= 0.05 * n2


def test_whole_step_in_a_graph_and_on_a_side_stream(step):
    import torch
    for name in ("policy", "preference"):
        run = step[name]
        want = run()
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            got = run()
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = run()
        for i in range(3):
            step["adv"].normal_()
            step["X"].mul_(1.0 - 0.05 * i)
            graph.replay()
            torch.cuda.synchronize()
            kept = [x.clone() for x in out]
            assert all(torch.equal(a, b) for a, b in zip(kept, run())), (name, i)
            torch.cuda.synchronize()
