"""Cache and beam operators in the ways a program calls them: captured and replayed, two at once, on other streams, with
a workspace of its own, over offsets that are no offsets."""

import pytest
import torch

from gpu_common import DEV

pytestmark = pytest.mark.gpu
I32 = torch.int32


@pytest.fixture(scope="module")
def gdn():
    import gated_deltanet_03_amd as m
    m.load_library()
    return m


class Step:
    """One token for each of B * W sequences, and a prompt's chunk beside it: appended, attended over, selected, moved."""

    def __init__(self, seed, B=2, W=4, V=5003, Hq=8, Hkv=2, d=128, page=16, length=1500, chunk=300, dtype=torch.bfloat16):
        g = torch.Generator(device=DEV).manual_seed(seed)

        def r(*shape):
            return torch.randn(*shape, generator=g, device=DEV).to(dtype)
        N, cols = B * W, -(-length // page) + 2
        self.W, self.B, self.chunk = W, B, chunk
        self.kc, self.vc = r(N * cols, Hkv, page, d), r(N * cols, Hkv, page, d)
        self.table = torch.randperm(N * cols, generator=g, device=DEV).to(I32).view(N, cols)
        self.lens = torch.randint(1, length, (N,), generator=g, device=DEV).to(I32)
        self.q, self.k, self.v = r(N, 1, Hq, d), r(N, 1, Hkv, d), r(N, 1, Hkv, d)
        self.many = r(chunk, Hq, d)
        self.cu = torch.tensor([0] + [chunk] * N, dtype=I32, device=DEV)
        self.inv = 10000.0 ** (-torch.arange(d // 2, device=DEV, dtype=torch.float32) / (d // 2))
        self.logits = torch.randn(B, W, V, generator=g, device=DEV).to(dtype)
        self.scores = torch.randn(B, W, generator=g, device=DEV)
        self.state = r(3, N, 4, 32)

    def shuffle(self, seed):
        """Other contents in the same places."""
        other = Step(seed)
        for n, t in vars(other).items():
            if torch.is_tensor(t) and n != "inv":
                getattr(self, n).copy_(t)

    def run(self, gdn):
        q = gdn.gdn_cache_append(self.k, self.v, self.kc, self.vc, self.table, self.lens, q=self.q, inv_freq=self.inv)
        o = gdn.gdn_cache_attention(q, self.kc, self.vc, self.table, self.lens)
        many = gdn.gdn_cache_attention(self.many, self.kc, self.vc, self.table, self.lens + self.chunk, cu_seqlens=self.cu)
        tokens, parents, scores, done = gdn.gdn_beam_select(self.logits, self.scores, eos_token=3)
        moved = gdn.gdn_state_reorder(self.state, parents, axis=1)
        own = self.table[:, 0].reshape(self.B, self.W).contiguous()
        gdn.gdn_cache_copy_pages(self.kc, self.vc, own.gather(1, parents.long()).contiguous(), own)
        return [q, o, many, tokens, parents, scores, done, moved]


def eager(gdn, step, seed):
    step.shuffle(seed)
    out = [t.clone() for t in step.run(gdn)] + [step.kc.clone(), step.vc.clone()]
    step.shuffle(seed)
    return out


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b, strict=True))


def capture(gdn, step):
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step.run(gdn)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step.run(gdn)
    return graph, out


def test_captured_and_replayed(gdn):
    steps = [Step(1), Step(2)]
    graphs = [capture(gdn, s) for s in steps]
    for seed in range(10, 15):
        for step, (graph, out) in zip(steps, graphs):
            want = eager(gdn, step, seed)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            assert same(out + [step.kc, step.vc], want)


@pytest.mark.parametrize("d,dtype", [(256, torch.float16), (256, torch.float32), (32, torch.float32)])
def test_captured_in_every_size_of_shared_memory(gdn, d, dtype):
    """The first call of a kernel that asks for more LDS than 64 KB may be the captured one."""
    g = torch.Generator(device=DEV).manual_seed(d)

    def r(*shape):
        return torch.randn(*shape, generator=g, device=DEV).to(dtype)
    kc, vc = r(40, 2, 32, d), r(40, 2, 32, d)
    table = torch.arange(40, dtype=I32, device=DEV).view(1, 40)
    lens = torch.tensor([1200], dtype=I32, device=DEV)
    qs = [r(1, 1, 4, d), r(1, 600, 4, d)]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = [gdn.gdn_cache_attention(q, kc, vc, table, lens) for q in qs]
    for n in (1200, 700, 611):
        lens.fill_(n)
        want = [gdn.gdn_cache_attention(q, kc, vc, table, lens) for q in qs]
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert same(out, want)


def test_two_at_once(gdn):
    steps, streams = [Step(5), Step(6)], [torch.cuda.Stream(), torch.cuda.Stream()]
    want = [eager(gdn, s, 20 + i) for i, s in enumerate(steps)]
    torch.cuda.synchronize()
    got = []
    for step, stream in zip(steps, streams):
        with torch.cuda.stream(stream):
            got.append(step.run(gdn))
    torch.cuda.synchronize()
    for step, g, w in zip(steps, got, want):
        assert same(g + [step.kc, step.vc], w)


def test_own_workspaces_and_outputs(gdn):
    step = Step(7)
    N, B, W = step.B * step.W, step.B, step.W
    sh = gdn.gdn_cache_shape(N, 1, 8, 2, 128, gdn.GDN_BF16, 16, step.kc.shape[0], step.table.shape[1])
    need = gdn.gdn_cache_attention_workspace_bytes(sh, False)
    assert need > 0
    want = gdn.gdn_cache_attention(step.q, step.kc, step.vc, step.table, step.lens)
    ws, o = torch.full((need,), 255, dtype=torch.uint8, device=DEV), torch.empty_like(step.q)
    assert gdn.gdn_cache_attention(step.q, step.kc, step.vc, step.table, step.lens, workspace=ws, o=o) is o
    assert torch.equal(o, want)
    with pytest.raises(gdn.GdnError, match="workspace"):
        gdn.gdn_cache_attention(step.q, step.kc, step.vc, step.table, step.lens, workspace=ws[:need - 16])
    with pytest.raises(gdn.GdnError, match="o overlaps q"):
        gdn.gdn_cache_attention(step.q, step.kc, step.vc, step.table, step.lens, o=step.q)
    V = step.logits.shape[-1]
    need = gdn.gdn_beam_workspace_bytes(gdn.gdn_beam_shape(B, W, W, V, gdn.GDN_BF16, -1, 0, V))
    ws = torch.full((need,), 255, dtype=torch.uint8, device=DEV)
    outs = dict(tokens=torch.empty(B, W, dtype=I32, device=DEV), parents=torch.empty(B, W, dtype=I32, device=DEV),
                new_scores=torch.empty(B, W, device=DEV), new_finished=torch.empty(B, W, dtype=torch.bool, device=DEV))
    got = gdn.gdn_beam_select(step.logits, step.scores, workspace=ws, **outs)
    assert all(a is b for a, b in zip(got, outs.values()))
    assert same(got, gdn.gdn_beam_select(step.logits, step.scores))
    with pytest.raises(gdn.GdnError, match="workspace"):
        gdn.gdn_beam_select(step.logits, step.scores, workspace=ws[:need - 16])
    with pytest.raises(gdn.GdnError, match="new_scores overlaps scores"):
        gdn.gdn_beam_select(step.logits, step.scores, new_scores=step.scores)


@pytest.mark.parametrize("new", [3, 200])
def test_offsets_that_overlap(gdn, new):
    """Rows that several sequences claim: nothing is promised of them, but rows behind cu_seqlens[N] stay, and calls end."""
    g = torch.Generator(device=DEV).manual_seed(new)
    q = torch.randn(new + 2, 4, 64, generator=g, device=DEV)
    kc = torch.randn(50, 2, 16, 64, generator=g, device=DEV)
    table = torch.arange(50, dtype=I32, device=DEV).repeat(40, 1)
    lens = torch.full((40,), 800, dtype=I32, device=DEV)
    cu = torch.tensor([0] + [new, 0] * 20, dtype=I32, device=DEV)
    for offsets in (cu, cu.flip(0).contiguous(), cu * 1000, cu - 7):
        o = torch.full_like(q, 7.0)
        gdn.gdn_cache_attention(q, kc, kc.clone(), table, lens, cu_seqlens=offsets, o=o)
        if offsets is cu:
            assert bool((o[new:] == 7.0).all())
        k, v = q[:, :2].contiguous(), q[:, 2:].contiguous()
        gdn.gdn_cache_append(k, v, kc.clone(), kc.clone(), table, lens, cu_seqlens=offsets)
    torch.cuda.synchronize()


def test_profile_names(gdn):
    step = Step(9)
    gdn.gdn_profile_collect()
    gdn.gdn_profile_enable(True)
    try:
        step.run(gdn)
    finally:
        gdn.gdn_profile_enable(False)
    assert {k: n for k, (n, _) in gdn.gdn_profile_collect().items()} == {
        "cache_append_kernel": 1, "cache_attention_kernel": 2, "cache_attention_join_kernel": 2, "beam_part_kernel": 1,
        "beam_join_kernel": 1, "state_reorder_kernel": 2}


@pytest.mark.parametrize("new", [1, 60])
def test_nothing_there(gdn, new):
    """Tables without columns, caches without pages, no sequences, no tokens."""
    q, k = torch.randn(2, new, 4, 64, device=DEV), torch.randn(2, new, 2, 64, device=DEV)
    kc, none = torch.randn(3, 2, 16, 64, device=DEV), torch.empty(0, 2, 16, 64, device=DEV)
    lens, inv = torch.tensor([new, new + 5], dtype=I32, device=DEV), torch.ones(32, device=DEV)
    tables = torch.empty(2, 0, dtype=I32, device=DEV), torch.zeros(2, 30, dtype=I32, device=DEV)
    for cache, table in ((kc, tables[0]), (none, tables[0]), (none, tables[1])):
        other, was = cache.clone(), cache.clone()
        turned = gdn.gdn_cache_append(k, k, cache, other, table, lens, q=q, inv_freq=inv)
        assert not torch.equal(turned[1], q[1])                    # queries are turned all the same
        assert torch.equal(cache, was) and torch.equal(other, was)
        o = gdn.gdn_cache_attention(q, cache, other, table, lens)
        assert not o.any()
    for N, L in ((0, 3), (2, 0)):
        t, n = torch.zeros(N, 4, dtype=I32, device=DEV), torch.ones(N, dtype=I32, device=DEV)
        x, y = torch.empty(N, L, 4, 64, device=DEV), torch.empty(N, L, 2, 64, device=DEV)
        assert gdn.gdn_cache_attention(x, kc, kc.clone(), t, n).shape == x.shape
        assert gdn.gdn_cache_append(y, y, kc, kc.clone(), t, n, q=x, inv_freq=inv).shape == x.shape
    one, ones = torch.ones(0, 3, device=DEV), torch.ones(0, 3, 10, device=DEV)
    assert [t.shape for t in gdn.gdn_beam_select(ones, one, beams=5)] == [(0, 5)] * 4
    assert gdn.gdn_state_reorder(torch.ones(0, 8, device=DEV), torch.zeros(0, 4, dtype=I32, device=DEV)).shape == (0, 8)


def test_pages_of_caches_in_either_order(gdn):
    both = torch.randn(2, 9, 2, 16, 64, device=DEV)
    src = torch.tensor([[0, 0, 1], [4, -1, 3]], dtype=I32, device=DEV)
    dst = torch.tensor([[1, 2, 0], [5, 6, 4]], dtype=I32, device=DEV)
    want = both.clone()
    want[:, [1, 2, 0, 5, 4]] = both[:, [0, 0, 1, 4, 3]]
    for a, b in ((0, 1), (1, 0)):
        moved = both.clone()
        gdn.gdn_cache_copy_pages(moved[a], moved[b], src, dst)
        assert torch.equal(moved, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [32, 64, 128, 256])
@pytest.mark.parametrize("new", [1, 60, 300])
def test_keys_on_no_page_are_not_read(gdn, new, d, dtype):
    """Keys that the lengths promise, in a cache without pages and on numbers that are no page: no memory is behind them."""
    q = torch.randn(2, new, 4, d, device=DEV).to(dtype)
    lens = torch.tensor([new + 500, 900], dtype=I32, device=DEV)
    none, other = torch.empty(0, 2, 16, d, dtype=dtype, device=DEV), torch.empty(0, 2, 16, d, dtype=dtype, device=DEV)
    for number in (0, -1, 7):
        table = torch.full((2, 60), number, dtype=I32, device=DEV)
        assert not gdn.gdn_cache_attention(q, none, other, table, lens).any()
    bad = torch.full((1, 2, 16, d), float("nan"), dtype=dtype, device=DEV)
    table = torch.full((2, 60), -1, dtype=I32, device=DEV)
    assert not gdn.gdn_cache_attention(q, bad, bad.clone(), table, lens).any()
