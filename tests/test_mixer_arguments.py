"""Arguments of the token mixers that are refused on the host, and their neighbours that are not (no GPU)."""
import itertools

import pytest

import bit_dequant_expert_gemv_b200 as fmoe

P = 0x10000  # aligned, never read
V = fmoe.View


def overlap(tokens, heads, dim, ts, hs):
    at = sorted(t * ts + h * hs for t in range(tokens) for h in range(heads))
    return any(b - a < dim for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("tokens,heads", [(1, 1), (1, 3), (3, 1), (2, 2), (4, 3), (5, 7)])
def test_rows_that_overlap(tokens, heads):
    """Every pair of small strides, against all rows laid side by side. The read's cache has no pages, so that a view that
    is taken goes on to the check that refuses the call for its missing positions."""
    dim, seen = 64, set()
    cache = fmoe.KvCacheDesc(P, 1, heads, dim, 16, P, 4, 3, 4)
    fine = V(P, heads * dim, dim)
    for ts, hs in itertools.product(range(0, 9 * dim, 32), repeat=2):
        for views in ((V(P, ts, hs), fine), (fine, V(P, ts, hs))):
            code = fmoe.lib().fmoe_kv_read(cache, None, None, tokens, fmoe.FMOE_F32, *views, None)
            assert code == fmoe.FMOE_ERR_INVALID
            text = "positions is NULL" if not overlap(tokens, heads, dim, ts, hs) else "overlapping rows"
            assert text in fmoe.last_error(), (ts, hs)
            seen.add(text)
    assert len(seen) == 2 or tokens * heads == 1


def test_overlapping_results_of_every_call():
    """[2 tokens][2 heads] rows of 128 with both strides 128: the second head of a token is the first of the next."""
    both = V(P, 128, 128)
    delta = fmoe.DeltaDesc(2, 2, 128, 128, fmoe.FMOE_BF16, 1, 1e-6, 1.0, P, 512, 128, P, 512, 128, P, 512, 128, P, P, 2, P,
                           2 * 128 * 128, 8, None, both.ptr, both.token_stride, both.head_stride)
    L = fmoe.lib()
    assert L.fmoe_delta_step(delta, 2, None) == fmoe.FMOE_ERR_INVALID and "overlapping" in fmoe.last_error()
    cache = fmoe.KvCacheDesc(P, 10, 2, 128, 64, P, 4, 2, 4)
    attn = fmoe.AttnDesc(2, fmoe.FMOE_BF16, 2, 1, 256, 1.0, P, 512, 128, None, P, both.ptr, 128, 128)
    assert L.fmoe_attn_q4(cache, attn, None) == fmoe.FMOE_ERR_INVALID and "overlapping" in fmoe.last_error()
    tokens = fmoe.KvTokens(fmoe.FMOE_BF16, 2, P, 512, 128, P, 512, 128, P, None, P, 64, 0, 2, P, 512, 128, P, 128, 128)
    assert L.fmoe_kv_append(cache, tokens, None) == fmoe.FMOE_ERR_INVALID and "overlapping" in fmoe.last_error()


@pytest.mark.parametrize("scale", [float("nan"), float("inf"), -float("inf")])
def test_attention_scale_that_is_not_finite(scale):
    """Logits times no number are no weights: a NaN would come out as like weights for all positions."""
    cache = fmoe.KvCacheDesc(P, 10, 2, 128, 64, P, 4, 2, 4)
    attn = fmoe.AttnDesc(2, fmoe.FMOE_BF16, 2, 1, 256, scale, P, 512, 128, None, P, P, 512, 128)
    assert fmoe.lib().fmoe_attn_q4(cache, attn, None) == fmoe.FMOE_ERR_INVALID and "scale" in fmoe.last_error()


def test_version_has_the_token_mixers():
    assert fmoe.lib().fmoe_version() >= 10100
