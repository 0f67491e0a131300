"""Bounded waits where a kv head has few rows over an 8-bit cache: with a limit of one poll the waits for copies run out (many
requests ask memory for more than it brings in that time), the call ends at once and says so, and the handle works on."""
import time

import pytest

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

import hybrid_draft_tree_gb300 as g  # noqa: E402
from hybrid_draft_tree_gb300 import graft as gb  # noqa: E402


@pytest.mark.parametrize("batch,slots,page,dim,ctx,shape", [
    (300, 4, 128, 128, 2000, {}), (300, 4, 128, 128, 2000, dict(softcap=5.0, window=1500)), (152, 1, 8, 128, 3000, {}),
    (152, 4, 8, 64, 3000, {})])
def test_waits_for_the_copies_of_few_rows_run_out(cuda_ok, batch, slots, page, dim, ctx, shape):
    torch.cuda.set_device(0)
    gen = torch.Generator(device="cuda").manual_seed(slots)
    own = -(-(ctx + slots) // page)
    kv = g.GraftKV(g.graft_kv_default_config(8, 2, dim, page, batch * own, batch, slots, cache="e4m3"))
    cache = torch.randn((batch * own, 2, page, dim), generator=gen, device="cuda", dtype=torch.bfloat16).to(torch.float8_e4m3fn)
    q = torch.randn((batch * slots, 8 * dim), generator=gen, device="cuda", dtype=torch.bfloat16)
    table = torch.randperm(batch * own, generator=gen, device="cuda").int().view(batch, own)
    at = torch.full((batch,), ctx, dtype=torch.int32, device="cuda")
    want, out = torch.zeros_like(q), torch.zeros_like(q)
    call = lambda o: kv.attend(batch, slots, q, cache, cache, table, at, ctx, o, **shape)  # noqa: E731
    call(want)
    assert kv.sync() == 0
    expired = 0
    for _ in range(12):
        kv.set_wait_limit(1)
        start = time.perf_counter()
        call(out)
        flags = kv.sync(raise_on_error=False)
        assert time.perf_counter() - start < 0.5
        assert flags == gb.GRAFT_ERR_TIMEOUT or flags == 0 and torch.equal(out, want)
        expired += flags != 0
        kv.set_wait_limit(0)
        out.zero_()
        call(out)
        assert kv.sync() == 0 and torch.equal(out, want)
    assert expired > 0
