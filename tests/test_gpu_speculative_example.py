"""The speculative serving example end to end: every token it emits is the best one
of the plain model in 64 bits, given the tokens before it.

Tolerance: the example's logits pass through 4 layers in bf16 (unit roundoff 2^-8).
A layer adds o = 0.3 * attention to x of size about 1 and rounds q, k, v, the
attention, its product and the sum once each: an error of at most about 6 * 2^-8
of o plus 2^-8 of x per layer, 4 * (6 * 0.3 + 1) * 2^-8 < 0.05 of the hidden
state's rms at worst.  Logits have a standard deviation of 4, so that an emitted
token's logit lies within 2 * 4 * 0.05 = 0.4 (twice: its own and the best's) of the
best one's; FP8 caches (unit roundoff 2^-4 of k and v, averaged over no fewer than
one key) add 4 * 0.3 * 2 * 2^-4 = 0.15: 2 * 4 * 0.2 = 1.6."""
import os
import sys

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("no GPU", allow_module_level=True)

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
import speculative_serving as ex
from gpu_helpers import log


def plain_logits(s, seq, adapter):
    """Logits [len(seq)][VOCAB] of the model over one whole sequence, float64 on the CPU."""
    f = lambda t: t.double().cpu()
    H, K, D = s.HEADS, s.KV_HEADS, s.DIM
    nrm = lambda x: x * torch.rsqrt(x.square().mean(1, keepdim=True) + 1e-5)
    x = f(s.embed)[seq]
    n = len(seq)
    mask = torch.ones(n, n).tril().bool()
    for i, w in enumerate(s.layers):
        h = nrm(x)
        q, k, v = (h @ f(w["qkv"])).split([H * D, K * D, K * D], 1)
        if adapter >= 0:
            for t, sl in ((q, 2 * i), (v, 2 * i + 1)):
                A, B, scale = s.lora[adapter, sl]
                t += scale * (h @ f(A).T) @ f(B).T
        q, k, v = q.view(n, H, D), k.view(n, K, D), v.view(n, K, D)
        out = torch.empty(n, H, D, dtype=torch.float64)
        for hd in range(H):
            sc = (q[:, hd] @ k[:, hd * K // H].T * D ** -0.5).masked_fill(~mask, -float("inf"))
            out[:, hd] = torch.softmax(sc, 1) @ v[:, hd * K // H]
        x = x + out.view(n, H * D) @ f(w["o"])
    return nrm(x) @ f(s.head)


PROMPTS = [np.random.default_rng(3).integers(0, ex.Server.VOCAB, n).tolist() for n in (1, 33, 70)]


@pytest.mark.parametrize("n_drafts,fp8", [(0, False), (1, False), (4, False), (4, True)])
def test_every_token_is_the_plain_models_best(n_drafts, fp8):
    log("[case] example, %d drafts, fp8 %d" % (n_drafts, fp8))
    adapters = [2, -1, 0]
    s = ex.Server(PROMPTS, adapters, fp8=fp8, seed=5)
    free = ex.L.lora_pool_info(s.pool)[0]
    out = s.generate(24, n_drafts)
    assert s.proposed >= s.accepted and (n_drafts == 0 or s.proposed > 0)
    for seq, prompt, a in zip(out, PROMPTS, adapters):
        assert seq[:len(prompt)] == prompt and len(seq) == len(prompt) + 24
        logits = plain_logits(s, seq, a)
        at = torch.arange(len(prompt) - 1, len(seq) - 1)
        gap = logits[at].max(1).values - logits[at, torch.tensor(seq[len(prompt):])]
        assert gap.max() <= (1.6 if fp8 else 0.4), gap.max()
    assert s.close() == free


def test_sampling_steps_stay_within_the_vocabulary():
    log("[case] example, sampling")
    s = ex.Server(PROMPTS, [0, 1, -1], seed=6)
    out = s.generate(16, 3, temperature=1.0)
    assert all(0 <= t < s.VOCAB for seq in out for t in seq)
    s.close()
