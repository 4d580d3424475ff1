"""The Python examples of README.md, run in order, with fresh memory full of NaN: what they compute
rests on nothing that no call has written."""
import os
import re

import pytest
import torch

from fp4_kv_cache_kvq_gb300 import kvq
from tests import latent_reference as ref
from tests.helpers import ensure_built

pytestmark = pytest.mark.gpu
README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


@pytest.fixture(scope="module")
def names():
    ensure_built()
    empty = torch.empty

    def dirty(*args, **kw):
        x = empty(*args, **kw)
        return x.fill_(float("nan")) if x.is_floating_point() else x

    space = {}
    torch.manual_seed(0)
    torch.empty = dirty
    try:
        for block in re.findall(r"```python\n(.*?)```", open(README).read(), re.S):
            exec(block, space)
        torch.cuda.synchronize()
    finally:
        torch.empty = empty
    return space


def test_all_examples_ran(names):
    for name in ("k_hat", "out", "o", "o1"):
        assert names[name].is_cuda


def test_the_latent_decode_is_of_each_sequences_last_token(names):
    """out of decode_attn: the row of the chunk's last token, by its definition."""
    lat, qa, scale, o1 = names["lat"], names["qa"], names["scale"], names["o1"]
    L, R = lat.latent_dim, lat.rope_dim
    assert torch.isfinite(o1).all()
    for b, T in enumerate(names["new"].tolist()):
        codes, e = ref.read_pool(lat.pool, None, lat.max_pages_per_seq, b, T, lat.page_size, L, R)
        c, k = ref.decode(codes, e, L)
        x = qa[b, T - 1]
        p = ref.weights(x, torch.cat([c, k], -1), scale, torch.full((x.shape[0],), T - 1))
        want = p @ c
        tol = ref.attn_bound(x, c, k, ref.power(e - 127), p, scale, o1.dtype, want)
        assert ((o1[b].double() - want).abs() <= tol).all(), b


def test_the_expanded_prompt_is_finite(names):
    for b, n in enumerate(names["new"].tolist()):
        assert torch.isfinite(names["o"][b, :n]).all()
