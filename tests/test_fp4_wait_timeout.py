"""The warp-wide bounded wait of the 4-bit attention: it gives up at its limit
and on the abort flag, and costs next to nothing from then on.  No GPU is
faulted: the self-test's barriers are ones that nothing completes."""
import pytest
import torch

from _gpu_helpers import need_gpu

FAKE = 1 << 20  # an aligned non-null address; never dereferenced
LIMIT_NS = 1_000_000  # 1 ms


def test_host_validation():
    from conftest import build_lib
    build_lib()
    import long_context_decode_indexpool_b200 as spx
    for limit, res in ((0, FAKE), (999, FAKE), (1_000_000_001, FAKE), (LIMIT_NS, None),
                       (LIMIT_NS, FAKE + 4)):
        with pytest.raises(spx.SpxError) as e:
            spx.spx_selftest_warp_wait_timeout(limit, res, stream=0)
        assert e.value.status == 1, (limit, res)


@pytest.mark.gpu
def test_warp_wait_gives_up_and_later_waits_are_short():
    spx = need_gpu()
    assert spx.spx_device_error() == 0
    res = torch.full((7,), -1, dtype=torch.int64, device="cuda")
    spx.spx_selftest_warp_wait_timeout(LIMIT_NS, res)
    torch.cuda.synchronize()
    ok0, ok1, t0, t1, late, late_ok, skipped = res.cpu().tolist()
    assert ok0 == 0 and LIMIT_NS <= t0 < 200 * LIMIT_NS, (ok0, t0)
    # the second warp's own limit is a second
    assert ok1 == 0 and t1 < 200 * LIMIT_NS, (ok1, t1)
    # 16 waits of a warp that has not given up: two suspended attempts of about a
    # millisecond each, not their limits of two seconds
    assert late_ok == 0 and late < 200 * LIMIT_NS, (late_ok, late)
    # 16 of a warp that has: a look each
    assert 0 <= skipped < LIMIT_NS, skipped
    assert spx.spx_device_error() == 1
    assert spx.spx_device_error() == 0


@pytest.mark.gpu
def test_attention_right_after_a_timeout():
    spx = need_gpu()
    res = torch.zeros(7, dtype=torch.int64, device="cuda")
    spx.spx_selftest_warp_wait_timeout(LIMIT_NS, res)
    d = spx.dims(16, 1.0)
    codes = torch.full((1, 100, 256), 0x22, dtype=torch.uint8, device="cuda")  # ones
    scales = torch.full((1, 100, 16), 127, dtype=torch.uint8, device="cuda")
    q = torch.zeros(1, 16, 512, dtype=torch.bfloat16, device="cuda")
    out = torch.empty_like(q)
    n_vis = torch.tensor([100], dtype=torch.int64, device="cuda")
    ws = spx.workspace(spx.spx_latent_attn_fp4_workspace_size(d, 1, 1, 100), "cuda")
    spx.spx_latent_attn_fp4(d, 1, 1, q, codes, scales, 100, n_vis, 100, out, None, ws)
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 1  # the self-test's
    assert (out == 1.0).all()
    spx.spx_latent_attn_fp4(d, 1, 1, q, codes, scales, 100, n_vis, 100, out, None, ws)
    torch.cuda.synchronize()
    assert spx.spx_device_error() == 0
