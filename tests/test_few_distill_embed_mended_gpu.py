"""Infinities, extreme values, second parts and streams of the few-token
layer, the distillation loss and the embedding."""

import numpy as np
import pytest
import torch

from _helpers import np64, require_gpu

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- embedding
@pytest.mark.parametrize("N", [40, 5000])
def test_embedding_the_lowest_id_is_an_error_where_there_is_no_padding(N):
    require_gpu()
    from mixture_experts_layer_side_gb300 import _lib
    from mixture_experts_layer_side_gb300.embedding import MoKEmbedding
    V, H = 50, 16
    ids = (torch.arange(N) % V).int()
    ids[7] = -2 ** 31
    table, dx = torch.randn(V, H), torch.randn(N, H)
    e = MoKEmbedding(V, H, N)
    for call in (lambda: e.forward(table.cuda(), ids.cuda()), lambda: e.backward(dx.cuda(), ids.cuda())):
        call()
        with pytest.raises(_lib.MokError) as err:
            e.check()
        assert err.value.status == 5
        e.check()
