"""What the cache operators' Python entry points refuse on CUDA tensors, before anything is launched."""
import pytest
import torch

pytestmark = pytest.mark.gpu
I32, U8, BF = torch.int32, torch.uint8, torch.bfloat16


@pytest.fixture(scope="module")
def gq():
    import causal_gqa_attention_fwd_gb300 as g
    g.lib()
    return g


def z(*shape, dtype=BF):
    return torch.zeros(*shape, dtype=dtype, device="cuda")


def q4_cache(n, H, P, D):
    return [z(n, H, P, w, dtype=U8) for w in (D // 2, D // 16) * 2]


def test_a_rotary_table_without_positions_is_not_no_rotation(gq):
    k, i, none = z(3, 2, 64), z(3, dtype=I32), z(0, 64, dtype=torch.float32)
    cache = z(1, 2, 16, 64)
    with pytest.raises(ValueError, match="no position"):
        gq.attn_cache_append(k, k, i, cache, cache.clone(), positions=i, rope_cos_sin=none)
    c = q4_cache(3, 2, 16, 64)
    with pytest.raises(ValueError, match="no position"):
        gq.attn_decode_q4_fwd(z(3, 2, 1, 64), *c, 1.0, 1.0, i, rope_cos_sin=none)
    with pytest.raises(ValueError, match="no position"):
        gq.attn_rope(k, None, i, none)


def test_rope_arguments(gq):
    q, i, tab = z(2, 4, 3, 64), z(2, 3, dtype=I32), z(8, 64, dtype=torch.float32)
    ok = gq.attn_rope(q, None, i, tab)
    assert ok[1] is None and ok[0].shape == q.shape
    with pytest.raises(ValueError, match="one entry a token"):
        gq.attn_rope(q, None, i[:, :2], tab)
    with pytest.raises(TypeError, match="int32"):
        gq.attn_rope(q, None, i.long(), tab)
    with pytest.raises(TypeError, match="bfloat16"):
        gq.attn_rope(q.half(), None, i, tab)
    with pytest.raises(ValueError, match="k must have"):
        gq.attn_rope(q, q[:1], i, tab)
    with pytest.raises(ValueError, match="repeat"):
        gq.attn_rope(q, None, i, tab, q_out=z(1, 4, 3, 64).expand(2, 4, 3, 64))
    with pytest.raises(ValueError, match="last dimension"):
        gq.attn_rope(q.transpose(2, 3).contiguous().transpose(2, 3), None, i, tab)
    with pytest.raises(gq.AttnError):                                     # rows not 16-byte aligned
        gq.attn_rope(z(2, 4, 3, 68)[..., 2:66], None, i, tab)
    with pytest.raises(ValueError, match="k_out without k"):
        gq.attn_rope(q, None, i, tab, k_out=q)


def test_plan_arguments(gq):
    i, t, f = z(2, dtype=I32), z(2, 4, dtype=I32), z(9, dtype=I32)
    with pytest.raises(ValueError, match="total_tokens"):
        gq.attn_cache_plan(i, i.clone(), t, 16, f)
    with pytest.raises(ValueError, match="entries"):
        gq.attn_cache_plan(i, i.clone(), t, 16, f, total_tokens=4, slots=z(3, dtype=I32))
    with pytest.raises(ValueError, match="block_table"):
        gq.attn_cache_plan(i, i.clone(), t[:1], 16, f, total_tokens=4)
    with pytest.raises(gq.AttnError):                                     # lengths replaced while they are read
        gq.attn_cache_plan(i, i.clone(), t, 16, f, total_tokens=4, lens_out=i)
    with pytest.raises(ValueError, match="contiguous"):
        gq.attn_cache_plan(i, i.clone(), z(2, 8, dtype=I32)[:, ::2], 16, f, total_tokens=4)
    c = z(1, dtype=I32)
    with pytest.raises(gq.AttnError):
        gq.attn_cache_plan(i, i.clone(), t, 16, f, cursor=c, cursor_out=c, total_tokens=4)


def test_append_gather_and_decode_arguments(gq):
    k, i, c = z(3, 2, 64), z(3, dtype=I32), q4_cache(2, 2, 16, 64)
    with pytest.raises(ValueError, match="slots"):
        gq.attn_cache_append_q4(k, k, i[:2], *c, 1.0, 1.0)
    with pytest.raises(ValueError, match="v must"):
        gq.attn_cache_append_q4(k, k[:2], i, *c, 1.0, 1.0)
    with pytest.raises(ValueError, match="k4_sf"):
        gq.attn_cache_append_q4(k, k, i, c[0], c[0], c[2], c[3], 1.0, 1.0)
    with pytest.raises(ValueError, match="positions without"):
        gq.attn_cache_append(k, k, i, z(1, 2, 16, 64), z(1, 2, 16, 64), positions=i)
    with pytest.raises(gq.AttnError):
        gq.attn_cache_append_q4(k, k, i, *c, 0.0, 1.0)
    with pytest.raises(ValueError, match="tokens"):
        gq.attn_cache_gather_q4(i, *c, 1.0, 1.0, k=z(2, 2, 64))
    q = z(2, 4, 1, 64)
    with pytest.raises(ValueError, match="cache_lens"):
        gq.attn_decode_q4_fwd(q, *c, 1.0, 1.0, i)
    with pytest.raises(gq.AttnError):                                     # a table shorter than the cache
        gq.attn_decode_q4_fwd(q, *c, 1.0, 1.0, i[:2], rope_cos_sin=z(15, 64, dtype=torch.float32))
    with pytest.raises(gq.AttnError):                                     # pages of 48
        gq.attn_decode_paged_q4_fwd(q, *q4_cache(2, 2, 48, 64), 1.0, 1.0, z(2, 1, dtype=I32), i[:2])
    with pytest.raises(gq.AttnError):
        gq.attn_decode_q4_fwd(q, *c, 1.0, 1.0, i[:2], workspace=z(256, dtype=U8))
    with pytest.raises(TypeError):
        gq.attn_decode_paged_q4_fwd(q, *c, 1.0, 1.0, None, i[:2])


def test_memory_that_runs_out_is_torchs_error(gq):
    """An output of 2^43 elements from a view that repeats one row."""
    q = z(1, 8, 512).expand(2 ** 31 - 1, 8, 512)
    with pytest.raises(torch.OutOfMemoryError):
        gq.attn_rope(q, None, z(4, dtype=I32), z(8, 64, dtype=torch.float32))


def test_rope_table_takes_a_device_index(gq):
    assert gq.attn_rope_table(3, 16, device=0).device == torch.device("cuda", 0)
