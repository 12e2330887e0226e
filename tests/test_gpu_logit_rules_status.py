"""apply_logit_rules reports what its lists hold, whatever the penalties are."""
import numpy as np
import pytest
import torch

import gpu_util as U

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 300, 5000, 40000])
@pytest.mark.parametrize("neutral", ["absent", "values"])
@pytest.mark.parametrize("V", [64, 9001])
def test_token_ids_are_checked_without_penalties(cuda, T, neutral, V):
    """A token id past the vocabulary is reported where the penalties change nothing; one past
    the row's length is not looked at; the logits come out as they are."""
    pkv = U.lib()
    rng = np.random.default_rng(T)
    ids = rng.integers(-1, V, (3, T)).astype(np.int32)
    logits = torch.from_numpy(rng.normal(size=(3, V)).astype(np.float32)).to(cuda)
    kw = {}
    if neutral == "values":
        kw = {"repetition_penalties": torch.ones(3, device=cuda),
              "presence_penalties": torch.zeros(3, device=cuda),
              "frequency_penalties": torch.zeros(3, device=cuda)}
    lens = np.full(3, T, np.int32)
    lens[1] -= 1

    def call():
        st = pkv.new_status(cuda)
        out = pkv.apply_logit_rules(logits, token_ids=torch.from_numpy(ids).to(cuda),
                                    token_lens=torch.from_numpy(lens).to(cuda), status=st, **kw)
        assert torch.equal(out, logits)
        return U.status_word(st)
    assert call() == 0
    ids[1, T - 1] = V + 3                        # behind the row's tokens
    assert call() == 0
    ids[2, T - 1] = V
    assert call() == pkv.STATUS["BAD_TOKEN_ID"]
