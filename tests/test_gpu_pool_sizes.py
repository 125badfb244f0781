"""Page management of pools of millions of pages, smaller pools before larger ones:
the counting kernels' shared memory (one bit a page) grows from call to call."""
import pytest
import torch

from sparse_long_context_min_b200 import binding as B

pytestmark = pytest.mark.gpu

# the first needs just under 48 KB of bits in each of the 8 counting CTAs, which their other shared data
# carry past the default limit; the next ones raise the limit that the calls before set
SIZES = (3145700, 3200000, 4000000)


def _pool(num):
    """Pages of 16 tokens, one kv head of 64 dims (4.9 KB); contents are whatever the memory holds."""
    kv = dict(dtype=torch.bfloat16, device="cuda")
    f = dict(dtype=torch.float32, device="cuda")
    return B.Pool(torch.empty(num, 1, 16, 64, **kv), torch.empty(num, 1, 16, 64, **kv), torch.empty(num, 1, 64, **kv),
                  torch.empty(num, 1, 64, **kv), torch.empty(num, 1, 64, **f), torch.empty(num, 1, 64, **f),
                  torch.zeros(num, dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("max_pages", [8, 17000])      # counted in the cluster's launch, and in one of its own
def test_pools_of_growing_sizes(max_pages):
    i32 = dict(dtype=torch.int32, device="cuda")
    for num in SIZES:
        pool = _pool(num)
        ref = torch.zeros(num, **i32)
        table = torch.full((3, max_pages), -1, **i32)
        lens = torch.zeros(3, **i32)
        status = torch.zeros(1, **i32)
        live = torch.zeros(1, **i32)
        ws = torch.empty(B.workspace_size(B.OP_PAGES, 3, 0, 0, 0, num, 0, 0), dtype=torch.uint8, device="cuda")
        ref[1] = ref[num - 1] = 1                      # row 2 holds the pool's second and its last page
        table[2, 0], table[2, 1] = 1, num - 1
        lens[2] = 32
        B.reserve_pages(pool, ref, table, lens, torch.tensor([40, 0, 0], **i32), ws, status)
        lens[0] = 40
        B.fork_sequences(pool, ref, table, lens, torch.tensor([0], **i32), torch.tensor([1], **i32), ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0
        assert table[:, :4].tolist() == [[0, 2, 3, -1], [0, 2, 4, -1], [1, num - 1, -1, -1]]
        assert ref[:6].tolist() == [2, 1, 2, 1, 1, 0]
        B.free_pages(pool, ref, table, lens, torch.tensor([0], **i32), status)
        before = pool.k_pool[num - 1].clone()
        B.compact_pages(pool, ref, table, live, ws, status)
        torch.cuda.synchronize()
        assert int(status.item()) == 0 and int(live.item()) == 5
        assert table[:, :3].tolist() == [[-1, -1, -1], [0, 2, 4], [1, 3, -1]]
        assert ref[:6].tolist() == [1, 1, 1, 1, 1, 0] and int(ref[num - 1]) == 0
        assert torch.equal(pool.k_pool[3].view(torch.int16), before.view(torch.int16))
        del pool, ref, ws
        torch.cuda.empty_cache()
