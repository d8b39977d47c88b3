"""isoquant_dense_attend: attention of the newest tokens over the 16-bit
paged cache, against 64-bit attention of the same pages.  Weights keep 16 or
more bits (fp16 pages: 11), see tests/dense_ref.py for the bound."""
import pytest
import torch

from tests.dense_ref import attend64, check_attention

pytestmark = pytest.mark.gpu
D = 128
WEIGHT_BITS = {torch.bfloat16: 15, torch.float16: 11}


class Case:
    def __init__(self, csd, lens, H, G, nq=1, ps=64, dtype=torch.bfloat16, seed=0, poison=True, spread=1.0,
                 extra_pages=0):
        self.csd, self.lens, self.H, self.G, self.nq, self.ps, self.dtype = csd, lens, H, G, nq, ps, dtype
        signs, quats = csd.synthetic.rotation_params(seed, H)
        self.ctx = csd.isoquant_init(signs, quats)
        g = torch.Generator().manual_seed(seed + 17)
        B = len(lens)
        pages = [max(1, -(-L // ps)) for L in lens]
        total = sum(pages)
        order = torch.randperm(total, generator=g).to(torch.int32)
        # entries behind a sequence's pages are no page at all
        table = torch.full((B, max(pages) + extra_pages), -7, dtype=torch.int32)
        data = torch.randn((total, 2, H, ps, D), generator=g)
        data[:, 0] *= torch.exp(torch.rand((H, 1, D), generator=g) - 0.5) * spread
        data = data.to(dtype)
        at = 0
        for b, m in enumerate(pages):
            table[b, :m] = order[at:at + m]
            at += m
            tail = lens[b] - (m - 1) * ps
            if poison and tail < ps:  # slots behind the sequence hold what they like
                data[table[b, m - 1], :, :, max(0, tail):] = float("nan")
        self.table_cpu, self.data_cpu = table, data
        self.cache = csd.DenseCache(data.cuda(), ps)
        self.table = table.cuda()
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
        self.q = torch.randn((B, nq, H * G, D), generator=g).to(dtype)
        self.ws = csd.alloc_dense_workspace(self.ctx, B, nq, H * G)
        self.ws.fill_(-1)  # NaN patterns: nothing of the workspace may be taken over

    def run(self, causal=False, scale=0.0, **kw):
        out = torch.full(self.q.shape, float("nan"), dtype=self.dtype, device="cuda")
        self.csd.isoquant_dense_attend(self.ctx, self.cache, self.q.cuda(), self.table, self.seq_lens, self.ws, out,
                                       causal=causal, scale=scale, **kw)
        torch.cuda.synchronize()
        assert self.csd.isoquant_get_status(self.ctx) == 0
        return out

    def check(self, out, causal=False, scale=None):
        H, G, nq = self.H, self.G, self.nq
        data = self.cache.data
        for b, L in enumerate(self.lens):
            n = max(0, -(-L // self.ps))
            kv = data[self.table[b, :n].long()].transpose(0, 2).reshape(H, 2, n * self.ps, D)[:, :, :max(0, L)]
            rows = self.q[b].cuda().view(nq, H, G, D).transpose(0, 1).reshape(H, nq * G, D)
            at = torch.arange(nq).repeat_interleave(G)
            limits = L - nq + at + 1 if causal else torch.full_like(at, L)
            o, A, d = attend64(rows, kv[:, 0], kv[:, 1], limits, scale)
            got = out[b].view(nq, H, G, D).transpose(0, 1).reshape(H, nq * G, D)
            check_attention(got, o.cuda(), A.cuda(), d.cuda(), WEIGHT_BITS[self.dtype])
            blind = (limits <= 0).cuda()
            assert (got[:, blind] == 0).all()


DECODE = [  # lens, H, G, page size
    ([1], 1, 1, 32),
    ([1024], 1, 1, 64),
    ([63, 64, 65], 2, 8, 32),
    ([0, 1, 0, 31, 32, 33, 0], 3, 4, 32),
    ([255, 256, 257, 511], 4, 3, 256),
    ([5000, 1, 777], 8, 8, 128),
    ([20000], 2, 7, 64),
    ([300] * 40, 4, 8, 128),
    ([129, 4000], 1, 16, 64),
    ([100, 260], 2, 33, 64),
    ([130, 0, 90], 1, 71, 128),
    ([0, 0], 2, 4, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("lens,H,G,ps", DECODE)
def test_decode(cuda_lib, lens, H, G, ps, dtype):
    c = Case(cuda_lib, lens, H, G, 1, ps, dtype, seed=len(lens) + G)
    c.check(c.run())
    # causal is the same for a single newest token
    c.check(c.run(causal=True), causal=True)


CHUNKS = [  # lens, H, G, nq, page size
    ([10, 3, 1, 0], 2, 4, 5, 32),       # chunks longer than their sequence: rows that see nothing
    ([600, 130], 2, 4, 16, 128),
    ([300, 45], 2, 8, 2, 32),
    ([700, 300, 65], 4, 4, 9, 64),
    ([2000], 1, 8, 16, 256),
    ([333, 64], 1, 3, 50, 64),
    ([1500, 1499], 2, 1, 3, 64),
]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("lens,H,G,nq,ps", CHUNKS)
def test_chunk(cuda_lib, lens, H, G, nq, ps, causal, dtype):
    c = Case(cuda_lib, lens, H, G, nq, ps, dtype, seed=nq)
    c.check(c.run(causal=causal), causal=causal)


def test_many_sequences(cuda_lib):
    g = torch.Generator().manual_seed(3)
    lens = [int(x) for x in torch.randint(0, 200, (700,), generator=g)]
    c = Case(cuda_lib, lens, 1, 8, 1, 32, seed=5)
    c.check(c.run())


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("scale", [0.5, 1e-3])
def test_scales_and_peaked_softmax(cuda_lib, dtype, scale):
    """Scores of some hundred (one key takes nearly all) and nearly equal weights."""
    c = Case(cuda_lib, [900, 2500], 2, 8, 1, 64, dtype, seed=9, spread=3.0)
    c.check(c.run(scale=scale), scale=scale)


def test_infinite_and_nan_scores(cuda_lib):
    """A NaN key makes its rows NaN, like the formula; a key whose scores are
    -inf weighs nothing; other heads stay as they are."""
    csd = cuda_lib
    c = Case(csd, [200, 150], 2, 4, 1, 64, seed=12)
    clean = c.run()
    page, off = int(c.table_cpu[0, 100 // 64]), 100 % 64
    c.cache.data[page, 0, 0, off, 5] = float("nan")
    out = c.run()
    assert torch.isnan(out[0, 0, :4]).all()
    assert torch.equal(out[0, 0, 4:], clean[0, 0, 4:]) and torch.equal(out[1], clean[1])
    c.cache.data[page, 0, 0, off, 5] = 0.0
    # rows with positive q at dimension 7 give this key -inf
    c.cache.data[page, 0, 0, off, 7] = float("-inf")
    c.q[0, 0, :4, 7] = c.q[0, 0, :4, 7].abs() + 0.1
    out = c.run()
    kv = c.cache.data[c.table[0, :4].long()].transpose(0, 2).reshape(2, 2, 256, D)[:1, :, :200].double()
    kv = torch.cat([kv[:, :, :100], kv[:, :, 101:]], 2)
    o, A, d = attend64(c.q[0, 0, :4].cuda()[None], kv[:, 0], kv[:, 1], torch.full((4,), 199))
    check_attention(out[0, 0, :4][None], o, A, d, 15)


def test_bad_pages_are_flagged(cuda_lib):
    """Page-table entries outside the cache set their bit and read page 0;
    nothing else is touched and the next call is clean."""
    csd = cuda_lib
    c = Case(csd, [500, 300], 2, 4, 1, 64, seed=21)
    clean = c.run()
    bad = c.table.clone()
    bad[0, 3], bad[0, 5] = -1, c.cache.num_pages
    out = torch.full(c.q.shape, float("nan"), dtype=c.dtype, device="cuda")
    csd.isoquant_dense_attend(c.ctx, c.cache, c.q.cuda(), bad, c.seq_lens, c.ws, out)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(c.ctx) == csd.DEVERR_PAGE_RANGE
    assert torch.equal(out[1], clean[1])
    # lengths beyond the table count as missing pages too
    short = c.table[:, :2].contiguous()
    csd.isoquant_dense_attend(c.ctx, c.cache, c.q.cuda(), short, c.seq_lens, c.ws, out)
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(c.ctx) == csd.DEVERR_PAGE_RANGE
    assert torch.equal(c.run(), clean)


def test_streams_and_graphs(cuda_lib):
    """The call on another stream, captured and replayed with new inputs, and
    two captured calls with workspaces of their own replayed at once."""
    csd = cuda_lib
    a = Case(csd, [900, 20, 4000], 2, 8, 1, 64, seed=31)
    b = Case(csd, [100, 3000], 4, 4, 2, 128, seed=32)
    want_a, want_b = a.run(), b.run(causal=True)
    side = torch.cuda.Stream()
    qa, qb = a.q.cuda(), b.q.cuda()
    oa, ob = torch.zeros_like(qa), torch.zeros_like(qb)
    torch.cuda.synchronize()
    csd.isoquant_dense_attend(a.ctx, a.cache, qa, a.table, a.seq_lens, a.ws, oa, stream=side)
    side.synchronize()
    assert torch.equal(oa, want_a)
    graphs = []
    for c, q, o, causal in ((a, qa, oa, False), (b, qb, ob, True)):
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            csd.isoquant_dense_attend(c.ctx, c.cache, q, c.table, c.seq_lens, c.ws, o, causal=causal)
        graphs.append(gr)
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        oa.zero_(), ob.zero_()
        torch.cuda.synchronize()
        with torch.cuda.stream(s1):
            graphs[0].replay()
        with torch.cuda.stream(s2):
            graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(oa, want_a) and torch.equal(ob, want_b)
    # shorter sequences and other queries through the same graph
    a.lens = [30, 0, 1025]
    a.seq_lens.copy_(torch.tensor(a.lens, dtype=torch.int32))
    a.q = torch.randn(a.q.shape).to(a.dtype)
    qa.copy_(a.q)
    graphs[0].replay()
    torch.cuda.synchronize()
    a.check(oa)


def test_repeats_are_identical(cuda_lib):
    c = Case(cuda_lib, [7000, 300, 1], 4, 8, 1, 64, seed=41)
    first = c.run()
    for _ in range(5):
        assert torch.equal(c.run(), first)


def test_argument_errors(cuda_lib):
    import ctypes
    csd = cuda_lib
    L, p = csd.lib(), csd._ptr
    c = Case(csd, [100, 40], 2, 4, 1, 64, seed=51)
    q = c.q.cuda()
    out = torch.empty_like(q)
    s0 = csd._stream(None)

    def call(cache=c.cache._c, qp=None, B=2, nq=1, Hq=8, pt=None, maxp=None, sl=None, scale=0.0, ws=None, wb=None,
             o=None):
        return L.isoquant_dense_attend(c.ctx.handle, cache, qp or p(q), B, nq, Hq, pt or p(c.table),
                                       c.table.shape[1] if maxp is None else maxp, sl or p(c.seq_lens), 0, scale,
                                       ws or p(c.ws), c.ws.numel() * 4 if wb is None else wb, o or p(out), s0)

    def off(t, by=8):
        return ctypes.c_void_p(t.data_ptr() + by)

    data = c.cache.data.data_ptr()
    assert call(cache=None) == -1
    assert call(cache=csd._DenseCache(0, 1, 2, 64)) == -1
    assert call(cache=csd._DenseCache(data, 1, 0, 64)) == -1
    assert call(cache=csd._DenseCache(data, 0, 2, 64)) == -2
    assert call(cache=csd._DenseCache(data, 1, 2, 100)) == -2
    assert call(cache=csd._DenseCache(data + 2, 1, 2, 64)) == -6
    assert call(B=-1) == -1 and call(nq=0) == -1 and call(Hq=7) == -1 and call(maxp=0) == -1
    assert call(nq=1 << 30) == -1
    assert call(scale=-1.0) == -1 and call(scale=float("nan")) == -1 and call(scale=float("inf")) == -1
    assert call(qp=off(q)) == -6 and call(o=off(out)) == -6 and call(ws=off(c.ws)) == -6
    assert call(wb=csd.isoquant_dense_workspace_size(c.ctx, 2, 1, 8) - 1) == -4
    assert L.isoquant_last_launch_count(c.ctx.handle) == 0
    assert call(B=0) == 0 and L.isoquant_last_launch_count(c.ctx.handle) == 0
    torch.cuda.synchronize()
    assert csd.isoquant_get_status(c.ctx) == 0
    assert call() == 0
    torch.cuda.synchronize()
    c.check(out)
