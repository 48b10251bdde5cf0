"""Groups that hold nothing but NaN: a NaN does not enter amax, so their scale is 0 (what a
group of zeros has), whichever kernel packs them: kv_pack, kv_append, kv_append_pages.
"""
import pytest


def with_nan_groups(d, dt):
    """k, v (256, 2, d): a channel of K and 32 features of V without a number, and the same
    values with zeros there."""
    import torch
    gen = torch.Generator(device="cuda").manual_seed(d)
    k, v = (torch.randn((256, 2, d), generator=gen, device="cuda").to(dt) for _ in range(2))
    out = []
    for x in (float("nan"), 0.0):
        a, b = k.clone(), v.clone()
        a[64:96, 1, 9] = x
        a[0:32, 0, 2:4] = x
        b[70, 0, :32] = x
        b[71:75, 1, -32:] = x
        out.append((a, b))
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("dt", ["bfloat16", "float32"])
@pytest.mark.parametrize("d", [64, 96, 128])
def test_their_scale_is_zero(d, dt):
    torch = pytest.importorskip("torch")
    from quantized_sparse_kv_gb300 import kvq
    dt = getattr(torch, dt)
    win = "f32" if dt == torch.float32 else "bf16"
    scales, records = [], []
    for k, v in with_nan_groups(d, dt):
        kb, vb = (x.transpose(0, 1)[None].contiguous() for x in (k, v))
        packed = kvq.pack(kb, vb, 64, win)
        grown = kvq.pack(kb[:, :, :40], vb[:, :, :40], 40, win, reserve=(8, 300))
        kvq.append(grown, kb[:, :, 40:], vb[:, :, 40:], 32)
        scales.append([c.used()[n] for c in (packed, grown) for n in ("k_scales", "v_scales")])
        for steps in ([256], [1] * 40 + [100, 1, 115]):
            state = kvq.PageState(1, 4, 64, 4, 32)
            cache = kvq.PagedCache(state, 2, d, win)
            cache.pool.zero_()
            first = 0
            for n in steps:
                plan = kvq.page_tables(state, torch.tensor([n], device="cuda"), n)
                kvq.append_pages(cache, plan, k[first:first + n], v[first:first + n])
                assert kvq.read_status(plan.status) == 0
                first += n
            # K scales, V scales of every record (include/kvq.h, kvq_paged_cache)
            rec = cache.pool.view(-1, 40 * d)
            records.append(torch.stack([rec[:, a * d:a * d + 4 * d] for a in (16, 36)])
                           .contiguous().view(torch.float32))
    for got, want in zip(*scales):
        assert int((want == 0).sum()) > 0 and torch.equal(got, want)
    assert int((records[2] == 0).sum()) > 0
    for got, want in zip(records[:2], records[2:]):
        assert torch.equal(got, want)
