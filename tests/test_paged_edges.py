"""Edges of the paged latent cache's operators: calls at the ends of what the
header allows, against plain 64-bit forms and exact integer arithmetic (B200).

The bounds of the attention's errors are those of test_paged_latent.py; others
stand beside their tests.
"""
import pytest
import torch

import gated_delta_rule_88_b200 as kda
from test_paged_latent import DEV

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ refused on the host
@pytest.mark.parametrize("how", ["attention", "append"])
def test_cache_of_one_page_repeated_is_refused(how):
    """expand() gives pages a stride of 0, which the library would take for its default."""
    cache = torch.ones(1, 32, 576, dtype=torch.bfloat16, device=DEV).expand(6, 32, 576)
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    lens = torch.tensor([3, 4], dtype=torch.int32, device=DEV)
    x = torch.ones(2, 4, 576, dtype=torch.bfloat16, device=DEV)
    with pytest.raises(ValueError, match="overlap"):
        if how == "attention":
            kda.kda_latent_attn(x, cache, table, lens)
        else:
            kda.kda_latent_append(x[:, 0], cache, table, lens)
    # one page of any stride is a pool of one page
    out, _ = kda.kda_latent_attn(x, cache[:1], torch.zeros_like(table), lens)
    assert kda.kda_get_device_error() == 0 and torch.equal(out, torch.ones_like(out))
