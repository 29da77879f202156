"""The choice of the tokens to keep, and their move, against plain restatements (exact)."""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
if not torch.cuda.is_available():
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

from attn_util import randn  # noqa: E402
from budget_util import KV, Cache, keep_reference  # noqa: E402
from gpu_util import DEV  # noqa: E402
from ternary_bit_weight_gb300 import binding as tb  # noqa: E402

pytestmark = pytest.mark.gpu


def keep(c, budget, first, recent):
    out = torch.full((len(c.lens), c.Hkv, budget), 12345, dtype=torch.int32, device=DEV)
    new = torch.full((len(c.lens),), 12345, dtype=torch.int32, device=DEV)
    tb.tern_kv_keep(len(c.lens), c.Hkv, c.pages, c.page, c.weight, c.dev_table, c.per, c.dev_lens, budget, first, recent, out, new)
    return out, new


def expected(c, budget, first, recent):
    w = c.weight.cpu().numpy()
    out = np.full((len(c.lens), c.Hkv, budget), -1)
    for b, n in enumerate(c.lens):
        page, row = c.slots(b)
        hidden = (page < 0) | (page >= c.pages)
        for h in range(c.Hkv):
            x = np.where(hidden, np.nan, w[np.clip(page, 0, c.pages - 1), h, row])[:n]
            k = keep_reference(x, n, budget, first, recent)
            out[b, h, :len(k)] = k
    return out


def check_keep(c, budget, first, recent):
    got, new = keep(c, budget, first, recent)
    assert np.array_equal(got.cpu().numpy(), expected(c, budget, first, recent))
    assert new.tolist() == [min(n, budget) for n in c.lens]
    return got


LENS = [[577], [1], [0, 1, 2, 3, 5], [64, 65, 63, 0, 700], [31, 32, 33, 4096], [9000, 100]]


@pytest.mark.parametrize("lens", LENS)
@pytest.mark.parametrize("budget,first,recent", [(1, 0, 0), (1, 1, 0), (1, 0, 1), (64, 4, 16), (64, 32, 32), (512, 4, 64),
                                                 (64, 0, 63), (5000, 4, 64)])
def test_keep(lens, budget, first, recent):
    check_keep(Cache(sum(lens), lens, 3, 16, 16, "x16"), budget, first, recent)


@pytest.mark.parametrize("page", [1, 4, 32, 256])
def test_keep_pages(page):
    check_keep(Cache(page, [300, 77, 513], 2, 16, page, "x16"), 70, 4, 20)


def test_keep_ties_and_odd_weights():
    """Equal weights, zeros of both signs, negative ones, infinities, NaN, subnormal numbers, neighbours in the last bit."""
    c = Cache(4, [200, 333, 90], 4, 16, 16, "x16")
    values = torch.tensor([0.0, -0.0, 1.0, -1.0, float("inf"), float("-inf"), float("nan"), 1e-40, -1e-40, 2e-40, 3.4e38,
                           1.0 + 2.0 ** -23, 1.0 - 2.0 ** -24])
    g = torch.Generator().manual_seed(1)
    c.weight.copy_(values[torch.randint(0, len(values), tuple(c.weight.shape), generator=g)])
    for budget, first, recent in ((50, 0, 0), (100, 3, 7), (199, 0, 0), (30, 1, 29), (89, 0, 0), (330, 4, 4)):
        check_keep(c, budget, first, recent)
    c.weight.fill_(0.5)
    check_keep(c, 60, 2, 5)
    c.weight.fill_(float("nan"))
    check_keep(c, 60, 2, 5)


def test_keep_hidden_pages_and_lengths():
    c = Cache(5, [200, 100], 2, 16, 16, "x16")
    c.table[0, 3], c.table[0, 5], c.table[1, 0] = -1, c.pages, -5
    c.dev_table = c.table.to(DEV)
    for budget in (64, 150, 190):
        check_keep(c, budget, 0, 10)
    want, _ = keep(c, 64, 2, 3)
    c.dev_lens = torch.tensor([c.per * 16, 100], dtype=torch.int32, device=DEV)
    room, new = keep(c, 64, 2, 3)
    c.dev_lens = torch.tensor([1 << 30, 100], dtype=torch.int32, device=DEV)
    far, new2 = keep(c, 64, 2, 3)
    assert torch.equal(room, far) and torch.equal(new, new2) and torch.equal(room[1], want[1])
    c.dev_lens = torch.tensor([-3, 100], dtype=torch.int32, device=DEV)
    got, new = keep(c, 64, 2, 3)
    assert (got[0] == -1).all() and new.tolist() == [0, 64]


def test_keep_long():
    """More tokens than shared memory holds, and weights of one size: every digit decides."""
    c = Cache(6, [70000], 1, 16, 1024, "x16")
    check_keep(c, 30000, 4, 100)
    c.weight.copy_(1.0 + torch.randint(0, 4000, tuple(c.weight.shape), generator=torch.Generator().manual_seed(2)) * 2.0 ** -23)
    check_keep(c, 30000, 4, 100)
    check_keep(c, 69999, 0, 0)


@pytest.mark.parametrize("n", [1024, 1025, 2049, 4097, 8193, 16385, 32768, 32769])
def test_keep_capacities(n):
    """Either side of the sizes at which the keys move from one form to the next; some keys in every digit."""
    c = Cache(n, [n, n // 2], 1, 16, 128, "x16")
    c.weight.copy_((torch.randint(0, 1 << 31, tuple(c.weight.shape), generator=torch.Generator().manual_seed(n), dtype=torch.int64) *
                    2 - 1).to(torch.int32).view(torch.float32))      # any bits: NaN, negative, subnormal
    check_keep(c, n // 3, 4, 16)
    c.weight.uniform_(0.5, 0.50001)
    check_keep(c, n - 1, 0, 0)


def test_keep_empty_table():
    out, new = torch.full((2, 3, 5), 7, dtype=torch.int32, device=DEV), torch.full((2,), 7, dtype=torch.int32, device=DEV)
    w, lens = torch.zeros(1, device=DEV), torch.tensor([4, 0], dtype=torch.int32, device=DEV)
    tb.tern_kv_keep(2, 3, 0, 16, w, None, 0, lens, 5, 0, 0, out, new)
    assert (out == -1).all() and (new == 0).all()


# --------------------------------------------------------------------- moves

def compact(c, lists, to=None, to_per=0, err=None, weight=True, table=None):
    tb.tern_kv_compact(KV[c.kv], len(c.lens), c.Hkv, c.D, c.pages, c.page, c.k, c.v, c.ks, c.vs, c.weight if weight else None,
                       c.dev_table if table is None else table, c.per, lists, lists.shape[-1], to, to_per, err)


def moved(c, lists, to=None):
    """The planes afterwards, from copies taken before."""
    out = {n: p.clone().cpu() for n, p in c.planes().items()}
    old = {n: p.clone().cpu() for n, p in c.planes().items()}
    for b in range(len(c.lens)):
        page, row = c.slots(b)
        target = page if to is None else to[b].cpu().numpy()[np.arange(lists.shape[-1]) // c.page]
        for h in range(c.Hkv):
            for j, i in enumerate(lists[b, h].tolist()):
                if i < 0:
                    break
                if 0 <= page[i] < c.pages and 0 <= target[j] < c.pages:
                    for n in out:
                        out[n][target[j], h, j % c.page] = old[n][page[i], h, row[i]]
    return out


def same(c, want, skip=()):
    for n, p in c.planes().items():
        if n not in skip:
            assert torch.equal(p.cpu().view(torch.uint8), want[n].view(torch.uint8)), n


def random_lists(seed, c, budget):
    g = np.random.RandomState(seed)
    out = np.full((len(c.lens), c.Hkv, budget), -1, dtype=np.int32)
    for b, n in enumerate(c.lens):
        for h in range(c.Hkv):
            k = np.sort(g.choice(n, min(n, budget), replace=False))
            out[b, h, :len(k)] = k
    return torch.from_numpy(out).to(DEV)


@pytest.mark.parametrize("kv,D", [("x16", 128), ("x16", 16), ("x16", 80), ("e4m3", 128), ("i8", 64), ("i8", 16), ("e4m3", 48)])
@pytest.mark.parametrize("lens,budget", [([577], 512), ([40, 0, 7, 129], 64), ([1], 1), ([1500, 300], 700)])
def test_moves(kv, D, lens, budget):
    c = Cache(D + budget, lens, 3, D, 16, kv)
    lists = random_lists(1, c, budget)
    want = moved(c, lists.cpu())
    compact(c, lists)
    same(c, want)


@pytest.mark.parametrize("page", [1, 2, 8, 64, 512])
def test_move_pages(page):
    c = Cache(page, [300, 77, 513], 2, 64, page, "e4m3")
    lists = random_lists(2, c, 150)
    want = moved(c, lists.cpu())
    compact(c, lists, weight=False)
    want["weight"] = c.weight.cpu()
    same(c, want)


def test_moves_by_one():
    """The first token leaves: every place is written right after its neighbour has been read, over many blocks."""
    for kv in ("x16", "i8"):
        c = Cache(8, [20000, 4097], 2, 128, 32, kv)
        lists = torch.arange(1, 20000, dtype=torch.int32).repeat(2, 2, 1)
        lists[1, :, 4096:] = -1
        want = {n: p.clone() for n, p in c.planes().items()}
        for b, n in enumerate(c.lens):
            page, row = (torch.from_numpy(x).long().to(DEV) for x in c.slots(b))
            for p in c.planes():
                x = c.planes()[p][page[1:n], :, row[1:n]]
                want[p][page[:n - 1], :, row[:n - 1]] = x
        compact(c, lists.to(DEV))
        same(c, {n: p.cpu() for n, p in want.items()})


def test_moves_to_other_pages():
    """Lists in any order, entries more than once; the source stays."""
    c = Cache(9, [300, 50, 0], 2, 64, 16, "i8", spare=40)
    used = set(c.table.flatten().tolist())
    free = [p for p in range(c.pages) if p not in used]
    to = torch.tensor(free[:30], dtype=torch.int32).reshape(3, 10).to(DEV)
    g = np.random.RandomState(3)
    lists = torch.full((3, 2, 160), -1, dtype=torch.int32)
    for h in range(2):
        lists[0, h] = torch.from_numpy(g.randint(0, 300, 160))
        lists[1, h, :70] = torch.from_numpy(g.randint(0, 50, 70))
    want = moved(c, lists, to)
    compact(c, lists.to(DEV), to, 10)
    same(c, want)
    # the same table by its address: in place
    c = Cache(10, [100], 2, 64, 16, "i8")
    lists = random_lists(5, c, 60)
    want = moved(c, lists.cpu())
    compact(c, lists, c.dev_table, c.per)
    same(c, want)


def test_lists_that_do_not_ascend_are_refused():
    c = Cache(11, [100, 100], 2, 64, 16, "x16")
    lists = random_lists(6, c, 60)
    lists[0, 1, 30] = lists[0, 1, 29]            # twice the same
    lists[1, 0, 59] = c.per * 16                 # past the table
    want = moved(c, torch.where(torch.tensor([[[False], [True]], [[True], [False]]]), torch.full((), -1, dtype=torch.int32), lists.cpu()))
    err = torch.zeros(1, dtype=torch.int32, device=DEV)
    compact(c, lists, err=err)
    same(c, want)
    assert int(err) == 2


def test_move_hidden_pages():
    c = Cache(12, [200], 1, 64, 16, "e4m3")
    c.table[0, 2], c.table[0, 9] = -1, c.pages + 3
    c.dev_table = c.table.to(DEV)
    lists = random_lists(7, c, 120)
    want = moved(c, lists.cpu())
    compact(c, lists)
    same(c, want)


def test_nothing_moves_when_all_are_kept():
    c = Cache(13, [100, 33], 2, 64, 16, "x16")
    lists, new = keep(c, 128, 4, 16)
    want = {n: p.clone().cpu() for n, p in c.planes().items()}
    compact(c, lists)
    same(c, want)
    assert new.tolist() == [100, 33]


def test_far_cells():
    """Cells more than 2^32 bytes into the cache."""
    pages, page, D = 280000, 64, 128
    k = torch.zeros((pages, 1, page, D), dtype=torch.bfloat16, device=DEV)
    v = torch.zeros((pages, 1, page, D), dtype=torch.bfloat16, device=DEV)
    x = randn(1, 2 * page, D).to(torch.bfloat16).to(DEV)
    k[-2:] = x.reshape(2, 1, page, D)
    v[-2:] = -x.reshape(2, 1, page, D)
    table = torch.tensor([[pages - 2, pages - 1]], dtype=torch.int32, device=DEV)
    lists = torch.arange(1, 128, 2, dtype=torch.int32, device=DEV).reshape(1, 1, 64)
    tb.tern_kv_compact(0, 1, 1, D, pages, page, k, v, None, None, None, table, 2, lists, 64)
    assert torch.equal(k[-2, 0], x[1::2]) and torch.equal(v[-2, 0], -x[1::2])
    assert int(k[:-2].count_nonzero()) == 0


def test_captured():
    """Choice and move in one graph, replayed on new weights."""
    c = Cache(14, [500, 90], 2, 64, 16, "i8")
    lists = torch.empty((2, 2, 128), dtype=torch.int32, device=DEV)
    new = torch.empty(2, dtype=torch.int32, device=DEV)
    saved = {n: p.clone() for n, p in c.planes().items()}

    def step():
        tb.tern_kv_keep(2, 2, c.pages, 16, c.weight, c.dev_table, c.per, c.dev_lens, 128, 4, 32, lists, new)
        compact(c, lists)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for n, p in c.planes().items():
        p.copy_(saved[n])
    c.weight.copy_(torch.exp(randn(77, *c.weight.shape)))
    want_lists = expected(c, 128, 4, 32)
    want = moved(c, torch.from_numpy(want_lists).to(torch.int32))
    graph.replay()
    assert np.array_equal(lists.cpu().numpy(), want_lists) and new.tolist() == [128, 90]
    same(c, want)


@pytest.mark.parametrize("page", [1, 2, 4, 16])
@pytest.mark.parametrize("n", [130, 700, 3001, 40001])
def test_keep_of_a_plane_at_any_place(page, n):
    """Weights that begin at any fp32 number, and pages that hold fewer tokens than one access."""
    c = Cache(n + page, [n, n // 3, 0, 127], 2, 16, page, "x16")
    want = c.weight
    room = torch.empty(want.numel() + 4, device=DEV)
    for shift in range(4):
        c.weight = room[shift:shift + want.numel()].view(want.shape).copy_(want)
        check_keep(c, n // 2, 3, 20)


def test_keep_where_a_digit_settles_it():
    """As many tokens as are left to keep share the digits that are known: all of them, and no other."""
    n = 600
    for low in (0, 1, 7, 300):                       # of equal top digits, more than are kept or as many
        c = Cache(low, [n], 1, 16, 16, "x16")
        plane = torch.cat([torch.full((low,), 1.0) + torch.arange(low) * 2.0 ** -23, torch.linspace(50.0, 90.0, n - low)])
        flat = plane[torch.randperm(n, generator=torch.Generator().manual_seed(low))]
        page, row = c.slots(0)
        weight = c.weight.cpu()
        weight[page[:n], 0, row[:n]] = flat
        c.weight.copy_(weight)
        for budget in {max(1, n - low - 1), max(1, n - low), min(n - 1, n - low + 1), n - 1}:
            check_keep(c, budget, 0, 0)
