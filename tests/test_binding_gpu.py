"""Image rows of the prefix pass from tokens."""
import pytest
import torch

from synth import inputs as I
from tests.test_language_gpu import BF16, ids_of, randn, rng

pytestmark = pytest.mark.gpu


def test_prefill_tokens_refuses_image_rows_of_another_type():
    from vla_dual_expert_b200 import Engine
    d = I.TINY
    e = Engine(d, 1, 16)
    try:
        e.load_from(I.Weights(d, seed=0))
        g = rng(71)
        table, ids, image = randn(g, 9, d.hidden_v, dtype=BF16), ids_of(g, (1, 5), 9), randn(g, 1, 8, d.hidden_v)
        for other in (image, image.half(), image.to(BF16).cpu()):
            with pytest.raises(TypeError, match="image_emb"):
                e.prefill_tokens(other, table, ids)
        wide = torch.cat([image, image], 2).to(BF16)[:, :, :d.hidden_v]   # rows that lie apart are taken
        assert torch.equal(e.prefill_tokens(wide, table, ids)[:, :8], image.to(BF16))
        e.sync()
    finally:
        e.close()
