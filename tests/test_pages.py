"""Pages of the exact tail: commit, fork and compact against a program of lists.

The operations move rows and hand out ids, so everything is compared exactly:
the state word for word, the pools bit for bit."""
import ctypes

import pytest
import torch

from kv_cache_compression_anchorkv_b200 import api, capi

gpu = pytest.mark.gpu


class Model:
    """The same pool as Python lists, one sequence after another."""

    def __init__(self, spec, K, V):
        self.spec, self.K, self.V = spec, K.clone(), V.clone()
        self.free = list(range(spec.n_pages - 1, -1, -1))
        self.refs = [0] * spec.n_pages
        self.len = [0] * spec.n_slots
        self.table = [[] for _ in range(spec.n_slots)]

    def state(self):
        s = self.spec
        head = [0, len(self.free)] + [0] * 14
        free = self.free + [-1] * (s.n_pages - len(self.free))
        rows = [x for r in self.table for x in r + [-1] * (s.max_pages - len(r))]
        return torch.tensor(head + free + self.refs + self.len + rows, dtype=torch.int32)

    def commit(self, K_new, V_new, n_accept, path):
        P = self.spec.page_size
        for b, n in enumerate(n_accept):
            for i in range(n):
                if self.len[b] % P == 0:
                    self.table[b].append(self.free.pop())
                    self.refs[self.table[b][-1]] = 1
                src = path[b][i] if path is not None else i
                self.K[:, self.table[b][-1], :, self.len[b] % P] = K_new[:, b, src]
                self.V[:, self.table[b][-1], :, self.len[b] % P] = V_new[:, b, src]
                self.len[b] += 1

    def fork(self, parents):
        P, n = self.spec.page_size, self.spec.n_pages
        old, old_len, old_refs = self.table, self.len, self.refs
        self.len = [old_len[p] if p >= 0 else 0 for p in parents]
        self.table, self.refs, copies, taken = [], [0] * n, [], set()
        for s, p in enumerate(parents):
            row = list(old[p]) if p >= 0 else []
            if self.len[s] % P and p in taken:
                copies.append((s, row.pop()))
            taken.add(p)
            for u in row:
                self.refs[u] += 1
            self.table.append(row)
        self.free += [u for u in range(n) if old_refs[u] and not self.refs[u]]
        for s, src in copies:
            dst = self.free.pop()
            self.table[s].append(dst)
            self.refs[dst] = 1
            m = self.len[s] % P
            for pool in (self.K, self.V):
                pool[:, dst, :, :m] = pool[:, src, :, :m].clone()

    def compact(self):
        n = self.spec.n_pages
        live = sum(1 for r in self.refs if r)
        holes = [u for u in range(live) if not self.refs[u]]
        to = dict(zip([u for u in range(live, n) if self.refs[u]], holes))
        for src, dst in to.items():
            self.refs[dst], self.refs[src] = self.refs[src], 0
            for pool in (self.K, self.V):
                pool[:, dst] = pool[:, src]
        self.table = [[to.get(u, u) for u in r] for r in self.table]
        self.free = list(range(n - 1, live - 1, -1))

    def same(self, state, K, V):
        assert torch.equal(state.cpu(), self.state())
        assert torch.equal(K.cpu().view(torch.uint8), self.K.view(torch.uint8))
        assert torch.equal(V.cpu().view(torch.uint8), self.V.view(torch.uint8))


def make(spec, seed=0):
    g = torch.Generator().manual_seed(seed)
    K, V = (torch.randn(spec.pool_shape, generator=g).to(spec.torch_dtype) for _ in range(2))
    return g, K, V


def drafts(spec, batch, n, g):
    shape = (spec.n_layers, batch, n, spec.n_kv_heads, spec.head_dim)
    return [torch.randn(shape, generator=g).to(spec.torch_dtype) for _ in range(2)]


def i32(x):
    return torch.tensor(x, dtype=torch.int32).cuda()


SPECS = [
    api.PageSpec(n_pages=40, page_size=16, n_slots=5, max_pages=9, n_layers=3, n_kv_heads=2, dtype="bf16"),
    api.PageSpec(n_pages=1100, page_size=32, n_slots=70, max_pages=12, n_layers=1, n_kv_heads=1, dtype="fp32"),
    api.PageSpec(n_pages=23, page_size=128, n_slots=3, max_pages=40, n_layers=2, n_kv_heads=3, dtype="bf16"),
]


def run_together(spec, in_place, steps=9, seed=3):
    """Commits, forks and compactions in turn, as beam decoding makes them."""
    g, K, V = make(spec, seed)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    m.same(state, Kg, Vg)
    ws = torch.empty(api.pages_workspace_bytes(spec), dtype=torch.uint8, device="cuda")

    def out():
        return None if in_place else torch.full_like(state, 12345)

    for step in range(steps):
        T = (1, 7, spec.page_size, 33)[step % 4]
        room = spec.max_pages * spec.page_size
        n = [min(int(torch.randint(0, T + 1, (1,), generator=g)), room - m.len[b]) for b in range(spec.n_slots)]
        need = sum(-(-(m.len[b] + n[b]) // spec.page_size) - -(-m.len[b] // spec.page_size) for b in range(spec.n_slots))
        if need > len(m.free):
            n = [0] * spec.n_slots
        path = None
        if step % 2:
            path = [torch.randperm(T, generator=g).tolist() for _ in range(spec.n_slots)]
        Kn, Vn = drafts(spec, spec.n_slots, T, g)
        m.commit(Kn, Vn, n, path)
        state = api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n),
                                 path=None if path is None else i32(path), state_out=out(), workspace=ws)
        m.same(state, Kg, Vg)
        if step % 2:
            parents = torch.randint(-1, spec.n_slots, (spec.n_slots,), generator=g).tolist()
            m.fork(parents)
            state = api.pages_fork(spec, state, Kg, Vg, i32(parents), state_out=out(), workspace=ws)
            m.same(state, Kg, Vg)
        if step % 3 == 2:
            m.compact()
            state = api.pages_compact(spec, state, Kg, Vg, state_out=out(), workspace=ws)
            m.same(state, Kg, Vg)
    assert api.read_status(state)[0] == 0


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("spec", SPECS, ids=lambda s: f"{s.n_pages}x{s.page_size}")
def test_commit_fork_compact_in_turn(spec, in_place):
    run_together(spec, in_place)


@gpu
def test_fewer_sequences_than_slots():
    spec = SPECS[0]
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    for n in ([5, 17], [16, 0], [0, 31]):
        Kn, Vn = drafts(spec, 2, 31, g)
        m.commit(Kn, Vn, n, None)
        api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n))
    m.same(state, Kg, Vg)


@gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_commit_of_no_sequences(in_place):
    """A step in which no sequence is left: the state is as it was."""
    spec = SPECS[0]
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    Kn, Vn = drafts(spec, 0, 5, g)
    got = api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32([]), path=i32([]).reshape(0, 5),
                           state_out=None if in_place else torch.full_like(state, -7))
    m.same(got, Kg, Vg)


@gpu
def test_many_slots_and_wide_tables():
    """More slots than threads of the state kernels, and a table far wider than what is used."""
    spec = api.PageSpec(n_pages=5000, page_size=16, n_slots=2100, max_pages=300, n_layers=1, n_kv_heads=1)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    n = torch.randint(0, 20, (spec.n_slots,), generator=g).tolist()
    Kn, Vn = drafts(spec, spec.n_slots, 20, g)
    m.commit(Kn, Vn, n, None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n))
    m.same(state, Kg, Vg)
    parents = torch.randint(-1, spec.n_slots, (spec.n_slots,), generator=g).tolist()
    m.fork(parents)
    api.pages_fork(spec, state, Kg, Vg, i32(parents))
    m.same(state, Kg, Vg)
    m.compact()
    api.pages_compact(spec, state, Kg, Vg)
    m.same(state, Kg, Vg)


@gpu
@pytest.mark.parametrize("slots", [2047, 2049, 3063, 3064, 3071, 3073, 4096])
def test_fork_of_as_many_slots_as_there_may_be(slots):
    """Shared memory goes with the slots: on both sides of the size that needs an attribute, and the most."""
    spec = api.PageSpec(n_pages=slots, page_size=16, n_slots=slots, max_pages=2, n_layers=1, n_kv_heads=1)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    n = torch.randint(0, 17, (slots,), generator=g).tolist()
    Kn, Vn = drafts(spec, slots, 16, g)
    m.commit(Kn, Vn, n, None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n))
    parents = torch.randint(-1, slots, (slots,), generator=g).tolist()
    m.fork(parents)
    api.pages_fork(spec, state, Kg, Vg, i32(parents))
    m.same(state, Kg, Vg)


REFUSED = [
    ("free", 1), ("table", 2), ("count", 3), ("count_below", 3), ("path", 3), ("parent", 3), ("parent_below", 3),
    ("len", 3), ("entry", 3), ("shared_tail", 3), ("no_page_to_fork", 1),
]


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("what,code", REFUSED)
def test_refused_operations_change_nothing(what, code, in_place):
    spec = api.PageSpec(n_pages=6, page_size=16, n_slots=3, max_pages=3, n_layers=2, n_kv_heads=2)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    Kn, Vn = drafts(spec, 3, 64, g)
    first = [20, 30, 5]
    m.commit(Kn, Vn, first, None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(first))      # five of six pages
    m.same(state, Kg, Vg)
    n, path, parents = [1, 1, 1], None, None
    if what == "free":
        n = [13, 3, 12]
    elif what == "table":
        n = [0, 0, 44]
    elif what == "count":
        n = [0, 65, 0]
    elif what == "count_below":
        n = [0, -1, 0]
    elif what == "path":
        path = torch.zeros(3, 64, dtype=torch.int32)
        path[2, 0] = 64
    elif what == "parent":
        parents = [0, 3, 1]
    elif what == "parent_below":
        parents = [0, -2, 1]
    elif what == "no_page_to_fork":
        n = [0, 0, 0]
    view = api.pages_view(spec, state)
    if what == "len":
        view["len"][1] = 49
    elif what == "entry":
        view["table"][1, 1] = 6
    elif what == "shared_tail":
        view["refs"][m.table[1][1]] = 2
    if what == "no_page_to_fork":
        # two tails of their own and one spare page: three forks of slot 0 need two new ones,
        # which the pages of slots 1 and 2 give; with those slots kept there is one
        spec2 = api.PageSpec(n_pages=4, page_size=16, n_slots=3, max_pages=3, n_layers=2, n_kv_heads=2)
        state = api.pages_init(spec2)
        Kg, Vg = (x[:, :4].contiguous() for x in (Kg, Vg))
        api.pages_commit(spec2, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32([50 - 16, 5, 0]))
        spec, parents = spec2, [0, 1, 1]
        view = api.pages_view(spec, state)
        assert int(view["n_free"]) == 0
    before, Kb, Vb = state.clone(), Kg.clone(), Vg.clone()
    out = None if in_place else torch.full_like(state, -7)
    if parents is not None or what in ("len", "entry"):
        got = api.pages_fork(spec, state, Kg, Vg, i32(parents or [0, 1, 2]), state_out=out)
    else:
        got = api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n),
                               path=None if path is None else path.cuda(), state_out=out)
    before[0] = code
    assert torch.equal(got, before)
    assert torch.equal(Kg, Kb) and torch.equal(Vg, Vb)
    with pytest.raises(capi.AnchorKVError):
        api.read_status(got)
    if what in ("len", "entry"):
        got2 = api.pages_compact(spec, state, Kg, Vg, state_out=None if in_place else out)
        assert torch.equal(got2, before)
        assert torch.equal(Kg, Kb) and torch.equal(Vg, Vb)


@gpu
@pytest.mark.parametrize("in_place", [True, False])
def test_bad_entries_seen_by_any_warp_are_refused_alike(in_place):
    """A table entry out of range that one warp of the state kernel meets early or late, many times over: the whole
    block refuses, and the scratch of a refused call serves the next one."""
    spec = api.PageSpec(n_pages=200, page_size=16, n_slots=100, max_pages=3, n_layers=1, n_kv_heads=1)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    Kn, Vn = drafts(spec, spec.n_slots, 30, g)
    n = torch.randint(0, 31, (spec.n_slots,), generator=g).tolist()
    n[0] = n[31] = n[32] = n[99] = 20
    m.commit(Kn, Vn, n, None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32(n))
    ws = torch.empty(api.pages_workspace_bytes(spec), dtype=torch.uint8, device="cuda")
    parents = i32(list(range(spec.n_slots)))
    for slots in ([0], [31], [32], [99], [0, 99], [31, 32]):
        broken = state.clone()
        for s in slots:
            api.pages_view(spec, broken)["table"][s, 0] = spec.n_pages
        want = broken.clone()
        want[0] = 3
        for op in (lambda st, out: api.pages_fork(spec, st, Kg, Vg, parents, state_out=out, workspace=ws),
                   lambda st, out: api.pages_compact(spec, st, Kg, Vg, state_out=out, workspace=ws)):
            for _ in range(25):
                st = broken.clone()
                assert torch.equal(op(st, None if in_place else torch.full_like(st, -7)), want)
    m.same(state, Kg, Vg)
    m.fork(list(range(spec.n_slots)))
    api.pages_fork(spec, state, Kg, Vg, parents, workspace=ws)
    m.same(state, Kg, Vg)


@gpu
@pytest.mark.parametrize("in_place", [True, False])
@pytest.mark.parametrize("what", ["held page without a holder", "last page without a holder", "free page with a holder"])
def test_counts_that_contradict_the_state_are_refused(what, in_place):
    """A page in use that counts as nobody's, or a free one that counts as somebody's: it could be handed out over
    rows that are still read, so nothing is done with such a state."""
    spec = api.PageSpec(n_pages=8, page_size=16, n_slots=3, max_pages=3, n_layers=2, n_kv_heads=2)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    Kn, Vn = drafts(spec, 3, 64, g)
    m.commit(Kn, Vn, [20, 33, 5], None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32([20, 33, 5]))
    view = api.pages_view(spec, state)
    if what == "free page with a holder":
        view["refs"][m.free[-1]] = 1
        ops = [lambda st, out: api.pages_commit(spec, st, Kg, Vg, Kn.cuda(), Vn.cuda(), i32([0, 0, 12]), state_out=out)]
    else:
        view["refs"][m.table[1][0 if what == "held page without a holder" else -1]] = 0
        ops = [lambda st, out: api.pages_compact(spec, st, Kg, Vg, state_out=out)]
    ops.append(lambda st, out: api.pages_fork(spec, st, Kg, Vg, i32([0, 1, 1]), state_out=out))
    want, Kb, Vb = state.clone(), Kg.clone(), Vg.clone()
    want[0] = 3
    for op in ops:
        st = state.clone()
        got = op(st, None if in_place else torch.full_like(st, -7))
        assert torch.equal(got, want)
        assert torch.equal(Kg, Kb) and torch.equal(Vg, Vb)


@gpu
def test_freed_pages_serve_the_forks_of_the_same_call():
    spec = api.PageSpec(n_pages=4, page_size=16, n_slots=3, max_pages=3, n_layers=2, n_kv_heads=2)
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    Kn, Vn = drafts(spec, 3, 40, g)
    m.commit(Kn, Vn, [10, 33, 0], None)
    api.pages_commit(spec, state, Kg, Vg, Kn.cuda(), Vn.cuda(), i32([10, 33, 0]))
    m.fork([0, 0, 0])
    api.pages_fork(spec, state, Kg, Vg, i32([0, 0, 0]))
    m.same(state, Kg, Vg)


@gpu
def test_captured_steps_replay():
    """A captured commit and fork on another stream replay as the eager calls."""
    spec = SPECS[0]
    g, K, V = make(spec)
    m, Kg, Vg = Model(spec, K, V), K.cuda(), V.cuda()
    state = api.pages_init(spec)
    ws = torch.empty(api.pages_workspace_bytes(spec), dtype=torch.uint8, device="cuda")
    Kn, Vn = drafts(spec, spec.n_slots, 5, g)
    n, parents = [3, 0, 5, 1, 2], [1, 0, 2, 2, 4]
    a = Kn.cuda(), Vn.cuda(), i32(n)
    par = i32(parents)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            api.pages_commit(spec, state, Kg, Vg, *a, workspace=ws)
            api.pages_fork(spec, state, Kg, Vg, par, workspace=ws)
        for _ in range(6):
            graph.replay()
            m.commit(Kn, Vn, n, None)
            m.fork(parents)
    side.synchronize()
    m.same(state, Kg, Vg)


# --- host side ---------------------------------------------------------------

FAKE = 0x10000


def call(name, *args):
    return getattr(capi.lib(), name)(*args)


@pytest.mark.parametrize("field,value,status", [
    ("n_pages", 0, capi.EINVAL), ("n_pages", (1 << 20) + 1, capi.EINVAL), ("page_size", 24, capi.EINVAL),
    ("page_size", 256, capi.EINVAL), ("n_slots", 0, capi.EINVAL), ("n_slots", 4097, capi.EINVAL),
    ("max_pages", 0, capi.EINVAL), ("max_pages", 65537, capi.EINVAL), ("n_layers", 0, capi.EINVAL),
    ("n_kv_heads", 0, capi.EINVAL), ("head_dim", 64, capi.EUNSUPPORTED)])
def test_bad_sizes_refused(field, value, status):
    spec = api.PageSpec(n_pages=8)
    setattr(spec, field, value)
    with pytest.raises(capi.AnchorKVError) as e:
        api.pages_state_bytes(spec)
    assert e.value.status == status
    with pytest.raises(capi.AnchorKVError):
        api.pages_workspace_bytes(spec)
    n = ctypes.c_size_t()
    assert call("anchorkv_pages_init", ctypes.byref(spec.c()), FAKE, None) == status
    assert call("anchorkv_pages_state_bytes", None, ctypes.byref(n)) == capi.EINVAL
    assert call("anchorkv_pages_state_bytes", ctypes.byref(spec.c()), None) == capi.EINVAL


def test_state_bytes():
    spec = api.PageSpec(n_pages=10, n_slots=3, max_pages=7)
    assert api.pages_state_bytes(spec) == 4 * (16 + 10 + 10 + 3 + 21) == 4 * spec.state_numel


@pytest.mark.parametrize("at,value,status", [
    (0, 0, capi.EINVAL), (1, 0, capi.EINVAL), (2, 0, capi.EINVAL), (3, 0, capi.EINVAL), (3, FAKE + 4096, capi.EINVAL),
    (4, 0, capi.EINVAL), (5, 8, capi.EINVAL), (6, -1, capi.EINVAL), (6, 5, capi.EINVAL), (7, 0, capi.EINVAL),
    (9, 0, capi.EINVAL), (10, 0, capi.EINVAL), (0, FAKE + 4, capi.EINVAL), (11, 64, capi.ENOSPC)])
def test_bad_commit_arguments_refused(at, value, status):
    spec = api.PageSpec(n_pages=8, n_slots=4)
    args = [FAKE, FAKE, FAKE + 4096, FAKE + 8192, FAKE, FAKE, 4, 2, None, FAKE, FAKE, 1 << 20]
    args[at] = value
    assert call("anchorkv_pages_commit", ctypes.byref(spec.c()), *args, None) == status


def test_commit_of_no_sequences_needs_no_rows():
    spec = api.PageSpec(n_pages=8, n_slots=4)
    args = [FAKE, FAKE, FAKE + 4096, FAKE + 8192, 0, 0, 0, 2, None, 0, FAKE, 64]
    assert call("anchorkv_pages_commit", ctypes.byref(spec.c()), *args, None) == capi.ENOSPC        # the next check


@pytest.mark.parametrize("at,value,status", [(0, 0, capi.EINVAL), (1, 0, capi.EINVAL), (2, 0, capi.EINVAL),
                                             (4, 0, capi.EINVAL), (5, 0, capi.EINVAL), (6, 64, capi.ENOSPC)])
def test_bad_fork_arguments_refused(at, value, status):
    spec = api.PageSpec(n_pages=8, n_slots=4)
    args = [FAKE, FAKE, FAKE + 4096, FAKE + 8192, FAKE, FAKE, 1 << 20]
    args[at] = value
    assert call("anchorkv_pages_fork", ctypes.byref(spec.c()), *args, None) == status
    if at != 4:
        del args[4]
        assert call("anchorkv_pages_compact", ctypes.byref(spec.c()), *args, None) == status


def test_unaligned_indices_refused():
    spec = api.PageSpec(n_pages=8, n_slots=4)
    for at in (8, 9):
        args = [FAKE, FAKE, FAKE + 4096, FAKE + 8192, FAKE, FAKE, 4, 2, FAKE, FAKE, FAKE, 1 << 20]
        args[at] = FAKE + 2
        assert call("anchorkv_pages_commit", ctypes.byref(spec.c()), *args, None) == capi.EINVAL
    args = [FAKE, FAKE, FAKE + 4096, FAKE + 8192, FAKE + 2, FAKE, 1 << 20]
    assert call("anchorkv_pages_fork", ctypes.byref(spec.c()), *args, None) == capi.EINVAL
