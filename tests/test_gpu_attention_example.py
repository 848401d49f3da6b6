"""The tuning example with an attention block: what a batch's updates compare."""
import pytest

pytestmark = pytest.mark.gpu


def test_updates_of_a_batch_see_one_dropout_mask(monkeypatch):
    """With weights that do not move, the log probabilities of every update are those of
    the rollout bit for bit, ratios of one; the next batch has another mask."""
    import torch
    import hadamard_rank_linear_amd.tuning_study as ts
    print("\n[gpu-case] dropout masks of the tuning example", flush=True)
    seen, plain = [], ts.hlq.hlq_policy_loss_logits
    steps, models = [], []

    def loss(logits, actions, old, *args, **kw):
        now = ts.hlq.hlq_token_logprob_forward(logits, actions)[0]
        seen.append(torch.equal(now, old))
        steps.append(int(models[0].seed[1]))
        return plain(logits, actions, old, *args, **kw)

    class Model(ts.TokenModel):
        def __init__(self, *args, **kw):
            super().__init__(*args, **kw)
            models.append(self)
    monkeypatch.setattr(ts.hlq, "hlq_policy_loss_logits", loss)
    monkeypatch.setattr(ts, "TokenModel", Model)
    ts.tune_policy(steps=3, tokens=256, lr=0.0, updates=3, heads=4)
    assert seen == [True] * 9 and steps == [0] * 3 + [1] * 3 + [2] * 3
