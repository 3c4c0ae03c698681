"""GPU test that fp8 prefixes are read once however far the sequences may grow by the call's bound.  The form shows in what
is recorded of groups that are out of order: kvattn.h says that the calls that read prefixes once look at them."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


def _setup(kv, hq, hkv, groups, n, shared, own, seed=0):
    """groups of n sequences of `shared` + up to `own` tokens over random pages."""
    g = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    batch, whole, more = groups * n, shared // 16, own // 16 + 1
    blocks = groups * whole + batch * more
    pool = torch.randint(0, 0x58, (blocks, hkv, 1, 4224), generator=gen, dtype=torch.uint8, device="cuda")
    scales = pool.view(torch.float32)[..., 1024:]
    scales.copy_(torch.rand(scales.shape, generator=gen, device="cuda") * 0.05 + 0.01)
    table = np.empty((batch, whole + more), np.int32)
    for b in range(batch):
        table[b, :whole] = np.arange(whole) + b // n * whole
        table[b, whole:] = groups * whole + b * more + np.arange(more)
    lens = (shared + 1 + g.integers(0, own, batch)).astype(np.int32)
    q = torch.randn((batch, hq, 128), generator=gen, device="cuda").to(torch.bfloat16)
    i32 = lambda x: torch.from_numpy(np.asarray(x, np.int32)).cuda()  # noqa: E731
    return (kv.make_config(hq, hkv, 128, kv.BF16), kv.CacheFP8(pool), q, i32(table), i32(lens), int(lens.max()),
            i32(np.arange(0, batch + 1, n)), i32([shared] * groups))


@pytest.mark.parametrize("hq,hkv,groups,n,shared,own,once", [
    (64, 8, 1, 16, 8192, 300, True), (32, 8, 1, 64, 2048, 3000, True), (8, 2, 1, 64, 8192, 100, True),
    (64, 8, 4, 32, 8192, 200, True), (64, 8, 1, 4, 1024, 200, False), (8, 2, 8, 2, 512, 500, False)])
def test_form_by_bound(kvattn_lib, hq, hkv, groups, n, shared, own, once):
    kv = kvattn_lib
    cfg, cache, q, table, lens, most, cu, sh = _setup(kv, hq, hkv, groups, n, shared, own)
    wrong = cu.clone()
    wrong[0] = 1
    first = None
    for bound in (most, 2 * most, 131072, 1 << 20):
        kv.decode_shared_fp8(cfg, cache, q, table, lens, bound, wrong, sh, shared)
        assert (kv.get_device_status() == kv.STATUS_CODE["KVATTN_ERR_BAD_INDEX"]) == once, bound
        out = kv.decode_shared_fp8(cfg, cache, q, table, lens, bound, cu, sh, shared)
        assert kv.get_device_status() == 0 and bool(torch.isfinite(out).all())
        first = out if first is None else first
        if once:  # the same work whatever the bound
            assert torch.equal(out, first)
        else:  # two forms by sequence: each rounds the output (2^-8), and weights (2^-11 or less)
            assert float((out.float() - first.float()).abs().max()) <= 2.0 ** -6 * float(first.abs().max())
