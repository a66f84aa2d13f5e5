"""coli_gemm_q8_lora with tables that are not those of its ids: a padded batch whose
last tokens the table does not hold, a request that has ended (its id is gone, the
table still lists it), a table made before a token changed its adapter.  Only the
tokens that the table has wrong may lose their rows, and a token without an adapter
keeps coli_gemm_q8's, whatever an earlier call has left in the workspace."""
import pytest
import torch

from quantized_moe_coli_amd import binding as B
from test_gpu_lora import Case, some_ids, tables
from test_gpu_q8 import gen

pytestmark = pytest.mark.gpu
# up to 64 tokens without an order, rings by it, tiles of 128 and 256, several workgroups of the
# order, and of several blocks each
SIZES = [(40, 1024), (65, 333), (64, 66000), (300, 4000), (600, 6145), (1500, 6144), (2500, 517), (9001, 130), (307277, 20)]


def changed(ids, L, what, seed):
    """The ids that the table is made from."""
    T = ids.numel()
    r = torch.rand(T, generator=gen(T, seed)).cuda()
    other = torch.randint(0, L, (T,), generator=gen(T, seed, 1), dtype=torch.int32).cuda()
    none = torch.full_like(ids, -1)
    bare = ids < 0
    if what == "missing":
        return torch.where(r < 0.1, none, ids)
    if what == "padded":
        return torch.where(torch.arange(T, device="cuda") >= T - T // 5, none, ids)
    if what == "listed":
        return torch.where(bare & (r < 0.5), other, ids)
    if what == "one listed":
        out = ids.clone()
        out[bare.nonzero()[0]] = 0
        return out
    if what == "all listed":
        return torch.where(bare, other, ids)
    if what == "moved":
        return torch.where(~bare & (r < 0.1), other, ids)
    if what == "empty":
        return none
    out = torch.where(bare & (r < 0.2), other, ids)
    out = torch.where(~bare & (r > 0.9), none, out)
    return torch.where(~bare & (r < 0.1), other, out)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("T,N", SIZES)
@pytest.mark.parametrize("what", ["missing", "padded", "listed", "one listed", "all listed", "moved", "empty", "any"])
def test_only_the_tokens_that_a_table_has_wrong_are_lost(dt, T, N, what):
    L = 6
    c = Case(dt, T, N, 64, 24, L, bare=0.25, bias=True)
    c.ids[T // 2] = -1
    first = c.run().clone()
    plain = torch.empty(T, N, dtype=c.dt, device="cuda")
    B.coli_gemm_q8(c.q, c.s, c.w.view(torch.uint8), c.ws, plain, bias=c.bias)
    bare = c.ids < 0
    assert torch.equal(first[bare], plain[bare])

    made = changed(c.ids, L, what, T)
    offs, perm = tables(made, L)
    keep = bare | (made == c.ids)
    assert keep.any() and (made != c.ids).any()
    ids = c.ids
    for earlier in range(3):  # what calls with other ids leave in the workspace
        c.ids = some_ids(T, L, L, "mixed", 0.1 * earlier, seed=50 + earlier)
        c.run()
        for _ in range(2):
            c.out.fill_(55.0)
            B.coli_gemm_q8_lora(c.q, c.s, c.w.view(torch.uint8), c.ws, c.lora, c.x, ids, offs, perm, c.y, c.work,
                                bias=c.bias)
            assert torch.equal(c.y[keep], first[keep])
            assert (c.out[:, N:] == 55.0).all()


@pytest.mark.parametrize("T,N", SIZES)
def test_a_workspace_that_another_call_has_used(T, N):
    """Batches of other sizes, ranks and ids, one after another in one workspace."""
    work = B.lora_workspace(T, 64)
    for seed, (rows, rank, bare) in enumerate([(T, 64, 0.0), (T, 16, 0.5), (max(1, T // 2), 64, 0.1), (T, 40, 1.0),
                                               (T, 40, 0.1)]):
        c = Case("bf16", rows, N, 64, rank, 7, bare=bare, seed=seed)
        c.check(c.run(work=work))
