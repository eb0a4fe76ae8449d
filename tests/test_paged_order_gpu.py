"""GPU tests of what stands directly ahead of fa_paged_decode on its stream,
outside a graph, where the kernel may be launched early: a copy from the host,
a fill, a plan without a write, another stream's event.  Each call has to see
what that left, and gives the bits that it gives on an idle GPU."""

import numpy as np
import pytest
import torch

from varlen_flashattention_backward_gb300 import binding as fa
from varlen_flashattention_backward_gb300 import build as fb

from _paged import DTYPE

DEV = torch.device("cuda:0")
pytestmark = pytest.mark.gpu

PAGE, HEADS, HEADS_KV, DIM = 16, 8, 2, 64
A, B = [500, 37, 800], [90, 1000, 0]       # two sets of lengths over the same pages


@pytest.fixture(scope="module", autouse=True)
def built():
    fb.build()
    fa.lib()
    torch.cuda.set_device(DEV)


class Setting:
    """A cache, two tables over it and the outputs of every (table, lengths)."""

    def __init__(self, dtype, width):
        g = torch.Generator(device=DEV).manual_seed(7)
        draw = lambda *s: torch.randn(*s, generator=g, device=DEV).to(DTYPE[dtype])  # noqa: E731
        per = -(-max(A + B) // PAGE)
        n = 3 * per + 5
        self.k, self.v = draw(n, PAGE, HEADS_KV, DIM), draw(n, PAGE, HEADS_KV, DIM)
        self.q = draw(3, HEADS, DIM)
        rng = np.random.default_rng(1)
        self.tables = []
        for _ in range(2):
            t = np.full((3, max(per, width)), -1, np.int32)
            t[:, :per] = rng.permutation(n)[:3 * per].reshape(3, per)
            self.tables.append(torch.from_numpy(t))
        self.lens = [torch.tensor(x, dtype=torch.int32) for x in (A, B)]
        self.table, self.len = self.tables[0].to(DEV), self.lens[0].to(DEV)
        self.want = {}
        for i in (0, 1):
            for j in (0, 1):
                self.table.copy_(self.tables[i])
                self.len.copy_(self.lens[j])
                torch.cuda.synchronize()
                self.want[i, j] = self.decode()
                torch.cuda.synchronize()
        assert not torch.equal(self.want[0, 0][0], self.want[1, 0][0])

    def decode(self):
        return fa.paged_decode(self.q, self.k, self.v, self.table, self.len, 0.125, stats=True)


def same(got, want):
    return all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.fixture(scope="module", params=[("bf16", 0), ("bf16", 3000), ("fp32", 0), ("fp32", 3000)],
                ids=lambda p: f"{p[0]}-{'ranges' if p[1] else 'direct'}")
def setting(request):
    return Setting(*request.param)


def test_a_copy_from_the_host_ahead(setting):
    pinned = [x.pin_memory() for x in (*setting.tables, *setting.lens)]
    got = []
    for step in range(40):
        i, j = step & 1, (step >> 1) & 1
        setting.table.copy_(pinned[i], non_blocking=True)
        setting.len.copy_(pinned[2 + j], non_blocking=True)
        got.append(((i, j), setting.decode()))
    torch.cuda.synchronize()
    assert all(same(out, setting.want[at]) for at, out in got)


def test_a_copy_on_the_device_ahead(setting):
    tables, lens = [x.to(DEV) for x in setting.tables], [x.to(DEV) for x in setting.lens]
    got = []
    for step in range(40):
        i, j = step & 1, (step >> 1) & 1
        setting.len.copy_(lens[j])
        setting.table.copy_(tables[i])
        got.append(((i, j), setting.decode()))
    torch.cuda.synchronize()
    assert all(same(out, setting.want[at]) for at, out in got)


def test_a_fill_ahead(setting):
    setting.table.copy_(setting.tables[0])
    got = []
    for _ in range(20):
        setting.len.copy_(setting.lens[0])
        got.append(setting.decode())
        setting.len.zero_()
        got.append(setting.decode())
    torch.cuda.synchronize()
    for full, empty in zip(got[::2], got[1::2]):
        assert same(full, setting.want[0, 0])
        assert (empty[0] == 0).all() and (empty[1] == -np.inf).all() and (empty[2] == 0).all()


def test_rows_written_ahead(setting):
    # The query rows, as the kernel ahead leaves them.
    setting.table.copy_(setting.tables[0])
    setting.len.copy_(setting.lens[0])
    kept, other = setting.q.clone(), -2 * setting.q
    torch.cuda.synchronize()
    got = []
    for step in range(20):
        setting.q.copy_(other if step & 1 else kept)
        got.append(setting.decode())
    setting.q.copy_(kept)
    torch.cuda.synchronize()
    assert all(same(x, setting.want[0, 0]) for x in got[::2])
    assert all(same(x, got[1]) and not torch.equal(x[0], got[0][0]) for x in got[1::2])


def test_another_streams_event_ahead(setting):
    setting.table.copy_(setting.tables[0])
    side, main = torch.cuda.Stream(), torch.cuda.current_stream()
    lens = [x.to(DEV) for x in setting.lens]
    torch.cuda.synchronize()
    got = []
    for step in range(8):
        j = step & 1
        side.wait_stream(main)               # the decode before has read the lengths
        with torch.cuda.stream(side):
            torch.cuda._sleep(200000)
            setting.len.copy_(lens[j])
            event = torch.cuda.Event()
            event.record()
        main.wait_event(event)
        got.append(((0, j), setting.decode()))
    torch.cuda.synchronize()
    assert all(same(out, setting.want[at]) for at, out in got)


@pytest.mark.parametrize("max_tokens", [3, 40000])      # one CTA, and many with a second kernel
@pytest.mark.parametrize("width", [64, 3000])
def test_a_plan_without_a_write_ahead(width, max_tokens):
    """Lengths and tables grow in place, page by page, and the decode behind
    each plan sees both."""
    g = torch.Generator(device=DEV).manual_seed(3)
    n, steps = 200, 50
    k, v = (torch.randn(n, PAGE, HEADS_KV, DIM, generator=g, device=DEV).bfloat16() for _ in range(2))
    q = torch.randn(3, HEADS, DIM, generator=g, device=DEV).bfloat16()
    table = torch.full((3, width), -1, dtype=torch.int32, device=DEV)
    lens = torch.zeros(3, dtype=torch.int32, device=DEV)
    ring = torch.randperm(n, generator=g, device=DEV).int()
    state = torch.tensor([0, n], dtype=torch.int64, device=DEV)
    delta = torch.tensor([1, 17, 5], dtype=torch.int32, device=DEV)
    error = torch.zeros(1, dtype=torch.int32, device=DEV)
    torch.cuda.synchronize()
    got = []
    for _ in range(steps):
        fa.paged_plan(table, lens, delta, ring, state, PAGE, max(max_tokens, 23), seq_lens_out=lens,
                      free_state_out=state, error=error)
        got.append(fa.paged_decode(q, k, v, table, lens, 0.125, stats=True, error=error))
    torch.cuda.synchronize()
    assert int(error) == 0 and lens.tolist() == [steps, 17 * steps, 5 * steps]
    # Pages that a request holds stay where they are, so the last table serves all steps.
    for i, out in enumerate(got):
        lens.copy_(delta * (i + 1))
        torch.cuda.synchronize()
        assert same(out, fa.paged_decode(q, k, v, table, lens, 0.125, stats=True))
        torch.cuda.synchronize()
