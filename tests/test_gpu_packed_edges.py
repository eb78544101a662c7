"""Edges of packed and paged attention: scores and weights of any size, rows of no sequence,
non-finite queries, padded batches, callers with a context of their own, and the backward's
whole contract.  Bounds as in packed_util."""
import math

import pytest
import torch

import packed_util as U

pytestmark = pytest.mark.gpu

BF, HF = torch.bfloat16, torch.float16


@pytest.fixture(scope="module")
def P():
    from block_sparse_attention_stats_b200.build import build
    build()
    import block_sparse_attention_stats_b200 as P
    return P


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def rows(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * scale).to(dtype)


def pages_of(x, ps):
    """[H, n, d] rows as a cache [pages, H, ps, d], page i holding positions i ps .. (i + 1) ps - 1."""
    h, n, d = x.shape
    need = -(-n // ps)
    c = torch.full((h, need * ps, d), math.nan, dtype=x.dtype)
    c[:, :n] = x
    return c.view(h, need, ps, d).transpose(0, 1).contiguous()


# ---- scores of any size --------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", [HF, BF])
def test_scores_past_every_range(P, dtype):
    """Scores so large that their float32 spacing is whole powers of two: weights stay finite."""
    d, n = 64, 600
    q, k = torch.full((1, n, d), 6000.0).to(dtype), torch.full((1, n, d), 9000.0).to(dtype)
    k[0, ::7] = 8000.0
    v = rows(3, 1, n, d, dtype=dtype)
    for scale in (1e-3, 1.0):
        a = P.pisa_varlen_attention(q.cuda(), k.cuda(), v.cuda(), i32([0, n]), scale=scale)
        kc, vc = (pages_of(x, 16).cuda() for x in (k, v))
        b = P.pisa_paged_attention(q[:, :1].cuda(), kc, vc, i32([list(range(kc.shape[0]))]), i32([0, 1]), i32([n]),
                                   scale=scale)
        P.pisa_device_status()
        assert torch.isfinite(a.float()).all() and torch.isfinite(b.float()).all()
