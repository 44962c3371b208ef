"""w4_draft_plan writes its outputs and the table's new entries and nothing else: every output
lies in the middle of a larger buffer whose rest is looked at afterwards."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")

from tests.test_gpu_draft import i32, plan_reference

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ops():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from w4a16_int4_quantized_gb300 import build
    build.build()
    from w4a16_int4_quantized_gb300 import ops as o
    return o


class Guarded:
    """n elements with 64 of `fill` on either side."""

    def __init__(self, n, dtype, fill):
        self.all = torch.full((n + 128,), fill, dtype=dtype, device="cuda")
        self.mid, self.n, self.fill = self.all[64:64 + n], n, fill

    def clean(self):
        return bool((self.all[:64] == self.fill).all()) and bool((self.all[64 + self.n:] == self.fill).all())


@pytest.mark.parametrize("ctx,new,page,width,n_free", [
    ([0, 0], [4, 4], 16, 4, 3), ([7] * 9, [128] * 9, 8, 20, 200), ([3, 1000, 17], [64, 64, 64], 16, 64, 2),
    ([30, 31, 40], [9, 9, 9], 16, 2, 9), ([12, 1, 0], [5, 0, 6], 7, 9, 9), ([5], [1], 16, 1, 0),
    (list(range(20)), [1] * 20, 64, 2, 40)])
@pytest.mark.parametrize("cap", ["none", "one", "short", "exact", "longer"])
@pytest.mark.parametrize("tree", [False, True])
def test_only_the_outputs_are_written(ops, ctx, new, page, width, n_free, cap, tree):
    g = np.random.default_rng(len(ctx) + page)
    B, total = len(ctx), sum(new)
    n = {"none": 0, "one": 1, "short": max(total - 3, 0), "exact": total, "longer": total + 37}[cap]
    host = np.full((B, width), -1, np.int32)
    ids = g.permutation(B * width + n_free).astype(np.int32)
    for b, c in enumerate(ctx):
        h = min(-(-c // page), width)
        host[b, :h] = ids[b * width: b * width + h]
    free = ids[B * width:]
    parents = g.integers(-1, 4, n).astype(np.int32) if tree else None
    table = Guarded(B * width, torch.int32, 55)
    table.mid.copy_(torch.from_numpy(host.reshape(-1)))
    cu, slots, pos, mask, taken = (Guarded(k, dt, 77) for k, dt in ((B + 1, torch.int32), (n, torch.int64), (n, torch.int32),
                                                                    (4 * n, torch.int32), (1, torch.int32)))
    d_ctx, d_new, d_free, d_par = i32(ctx), i32(new), i32(free), None if parents is None else i32(parents)
    st = ops.raw.w4_draft_plan(d_ctx.data_ptr(), d_new.data_ptr(), None if d_par is None else d_par.data_ptr() or None,
                               d_free.data_ptr() or None, n_free, table.mid.data_ptr(), B, width, page, n,
                               cu.mid.data_ptr(), slots.mid.data_ptr(), pos.mid.data_ptr(), mask.mid.data_ptr(),
                               taken.mid.data_ptr(), None)
    assert st == ops.W4_OK
    torch.cuda.synchronize()
    assert all(x.clean() for x in (table, cu, slots, pos, mask, taken))
    # without room for tokens every parent is one of those that are left out: roots
    want = plan_reference(ctx, new, parents, free, host, page, n)
    assert cu.mid.tolist() == want[0] and taken.mid.tolist() == [want[5]]
    assert np.array_equal(table.mid.cpu().numpy().reshape(B, width), want[1])
    assert slots.mid.tolist() == want[2] and pos.mid.tolist() == want[3]
    assert np.array_equal(mask.mid.cpu().numpy().reshape(n, 4), want[4])
