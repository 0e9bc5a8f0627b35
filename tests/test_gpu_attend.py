"""moe_ffn_attend against its formula in 64 bits."""

import math
import random

import pytest

import fusion_backend_gb300 as fb

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAN, INF = float("nan"), float("inf")


def half_step(v, dtype):
    fi = torch.finfo(dtype)
    return v.abs() * (fi.eps / 2) + fi.smallest_normal * fi.eps / 2


class Case:
    """Sequences of (cached tokens, rows), their caches in pages of any order and what every row sees."""

    def __init__(self, seqs, Hq=8, Hkv=2, D=64, page=16, dtype=BF16, layout="token", mask=None, rest=0, seed=0, spread=1.0,
                 poison=False):
        self.seqs, self.Hq, self.Hkv, self.D, self.page = seqs, Hq, Hkv, D, page
        g = torch.Generator(device="cuda").manual_seed(seed)
        host = random.Random(seed)
        need = [-(-max(n, 0) // page) for n, _ in seqs]
        pages = sum(need) + 2
        shape = (pages, Hkv, page, D) if layout == "head" else (pages, page, Hkv, D)
        make = lambda: torch.randn(shape, generator=g, device="cuda").to(dtype)  # noqa: E731
        self.k, self.v = make(), make()
        if layout == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        self.table = torch.full((len(seqs), max(max(need), 1)), -5, dtype=torch.int32, device="cuda")
        at = 0
        for b, m in enumerate(need):
            self.table[b, :m] = order[at:at + m]
            at += m
        self.T = sum(n for _, n in seqs) + rest
        self.q = (torch.randn(self.T, Hq, D, generator=g, device="cuda") * spread).to(dtype)
        self.lens = torch.tensor([n for n, _ in seqs], dtype=torch.int32, device="cuda")
        starts = [0]
        for _, n in seqs:
            starts.append(starts[-1] + n)
        self.starts = starts
        self.q_start = torch.tensor(starts, dtype=torch.int32, device="cuda")
        self.mask = None
        if mask is not None:
            words = -(-max(n for _, n in seqs) // 32)
            bits = [[0] * words for _ in range(self.T)]
            for (_, n), t in zip(seqs, starts):
                for j in range(n):
                    if mask == "tree":
                        if j:
                            bits[t + j] = list(bits[t + host.randint(max(0, j - 4), j - 1)])
                        bits[t + j][j // 32] |= 1 << j % 32
                    elif mask == "random":
                        bits[t + j] = [host.getrandbits(32) for _ in range(words)]
                    elif mask == "none" and j % 2:
                        bits[t + j][j // 32] |= 1 << j % 32
            self.mask = torch.tensor([[w - 2**32 if w >= 2**31 else w for w in row] for row in bits], dtype=torch.int64,
                                     device="cuda").to(torch.int32)
        if poison:
            # whatever no token of a sequence lies in
            used = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
            for b, (length, _) in enumerate(seqs):
                i = torch.arange(length, device="cuda")
                used[self.table[b].long()[i // page], i % page] = True
            self.k[~used], self.v[~used] = NAN, INF
        self.pages = pages

    def seen(self, b):
        """bool [n, cached tokens]"""
        length, n = self.seqs[b]
        own = torch.arange(length, device="cuda") - (length - n)
        j = torch.arange(n, device="cuda")[:, None]
        if self.mask is None:
            ok = own[None] <= j
        else:
            rows = self.mask[self.starts[b]:self.starts[b] + n]
            at = own.clamp(min=0)
            inside = at // 32 < rows.shape[1]
            ok = (rows[:, (at // 32).clamp(max=rows.shape[1] - 1)] >> (at % 32) & 1).bool() & inside
        page = self.table[b].long()[torch.arange(length, device="cuda") // self.page]
        return ((own < 0)[None] | ok) & ((page >= 0) & (page < self.pages))[None]

    def reference(self, scale=None, softcap=0.0, terms=2.0**-16):
        """out, its error's bound, lse, its error's bound."""
        scale = self.D**-0.5 if scale is None else scale
        Hq, Hkv, D = self.Hq, self.Hkv, self.D
        out = torch.zeros(self.T, Hq, D, dtype=torch.float64, device="cuda")
        err, lse = torch.zeros_like(out), torch.full((self.T, Hq), -INF, dtype=torch.float64, device="cuda")
        lerr = torch.zeros_like(lse)
        for b, (length, n) in enumerate(self.seqs):
            if not length or not n:
                continue
            i = torch.arange(length, device="cuda")
            pg = self.table[b].long()[i // self.page].clamp(0, self.pages - 1)
            seen = self.seen(b)
            any_seen = seen.any(0)[:, None, None]
            zero = torch.zeros((), dtype=torch.float64, device="cuda")
            k = torch.where(any_seen, self.k[pg, i % self.page].double(), zero).repeat_interleave(Hq // Hkv, 1)
            v = torch.where(any_seen, self.v[pg, i % self.page].double(), zero).repeat_interleave(Hq // Hkv, 1)
            q = self.q[self.starts[b]:self.starts[b] + n].double()
            s = torch.einsum("jhd,ihd->hji", q, k) * scale
            size = torch.einsum("jhd,ihd->hji", q.abs(), k.abs()) * abs(scale)
            # a score: at most D / 8 + 10 additions and products in a row, each off by a step of fp32 at most
            ds = size * ((D / 8 + 10) * 2.0**-23)
            if softcap:
                s = softcap * torch.tanh(s / softcap)
                ds = ds + softcap * 2.0**-21
            s = s.masked_fill(~seen[None], -INF)
            top = s.amax(-1, keepdim=True)
            none = top == -INF
            p = torch.exp(s - top.masked_fill(none, 0.0))
            # an exponential: its argument's rounding (some products of size s) and its own 2 steps
            dp = ds + (s.abs().masked_fill(~seen[None], 0.0) + top.abs().masked_fill(none, 0.0) + 2) * 2.0**-22
            total = p.sum(-1, keepdim=True).masked_fill(none, 1.0)
            p = p / total
            e = (p * dp).sum(-1, keepdim=True)  # of the sum, relative
            # sums over the tokens: at most length / 8 + 64 roundings in a row
            adds = (length / 8 + 64) * 2.0**-23
            o = torch.einsum("hji,ihd->jhd", p, v)
            size = torch.einsum("hji,ihd->jhd", p, v.abs())
            d = torch.einsum("hji,ihd->jhd", p * dp, v.abs()) + size * (e.permute(1, 0, 2) + 2 * adds + terms)
            rows = slice(self.starts[b], self.starts[b] + n)
            out[rows], err[rows] = o, d
            lse[rows] = torch.where(none, top, top + torch.log(total))[..., 0].T
            lerr[rows] = (e[..., 0] + adds + (lse[rows].T.abs().masked_fill(none[..., 0], 0.0) + 8) * 2.0**-22).T
        return out, err, lse, lerr

    def call(self, **kw):
        return fb.moe_ffn_attend(self.q, self.k, self.v, self.table, self.lens, self.q_start, mask=self.mask, **kw)

    def check(self, out_dtype=None, scale=None, softcap=0.0, strided=False):
        dt = out_dtype or self.q.dtype
        full = torch.full((self.T, self.Hq, self.D + (3 if strided else 0)), 5.0, device="cuda", dtype=dt)
        out = full[..., :self.D]
        lse = torch.full((self.T, self.Hq), 5.0, device="cuda")
        assert self.call(scale=scale, softcap=softcap, out=out, lse=lse) is out
        end = self.starts[-1]
        assert bool((out[end:] == 5).all()) and bool((lse[end:] == 5).all()) and bool((full[..., self.D:] == 5).all())
        # weights as two numbers of the cache's type: 16 bits (bf16) or 22 of them; three of bf16 where out is fp32
        terms = 2.0**-16 if self.q.dtype == BF16 and dt != F32 else 2.0**-20
        want, err, wl, el = self.reference(scale, softcap, terms)
        d = (out.double() - want).abs() - err - half_step(want.abs() + err, dt)
        assert float(d[:end].max()) <= 0, float(d[:end].max())
        none = wl[:end] == -INF
        assert torch.equal(lse[:end] == -INF, none) and bool((out[:end][none] == 0).all())
        dl = ((lse.double() - wl).abs() - el)[:end][~none]
        assert dl.numel() == 0 or float(dl.max()) <= 0, float(dl.max())
        return out


SIZES = [
    dict(seqs=[(1, 1)]), dict(seqs=[(2, 1)]), dict(seqs=[(63, 1), (64, 1), (65, 1), (1, 1)]),
    dict(seqs=[(500, 1), (17, 1), (1300, 1)], page=24), dict(seqs=[(3000, 1)], D=128, Hq=32, Hkv=4),
    dict(seqs=[(129, 1)] * 20, D=128, Hq=16, Hkv=16), dict(seqs=[(400, 1), (90, 1)], D=256, Hq=8, Hkv=1, page=32),
    dict(seqs=[(700, 1), (33, 1)], D=80, Hq=14, Hkv=2, page=1), dict(seqs=[(333, 1)] * 3, D=96, Hq=6, Hkv=2, page=256),
    dict(seqs=[(260, 1)], D=192, Hq=16, Hkv=1, page=8), dict(seqs=[(77, 1)] * 2, D=8, Hq=3, Hkv=3, page=5),
    dict(seqs=[(1000, 1)], D=64, Hq=71, Hkv=1), dict(seqs=[(150, 1)], D=64, Hq=256, Hkv=2, page=64),
    dict(seqs=[(40, 3), (300, 8), (5, 5)], D=64), dict(seqs=[(1000, 16), (200, 9)], D=128, Hq=32, Hkv=4, page=64),
    dict(seqs=[(64, 64), (333, 61), (4000, 33)], D=64, Hq=4, Hkv=1), dict(seqs=[(300, 300)], D=64, Hq=4, Hkv=2),
    dict(seqs=[(900, 40), (50, 40)], D=80, Hq=12, Hkv=2, page=24), dict(seqs=[(500, 7)], D=256, Hq=16, Hkv=2),
    dict(seqs=[(130, 12)], D=192, Hq=8, Hkv=1, page=16), dict(seqs=[(2500, 5)] * 3, D=128, Hq=3, Hkv=1, page=128),
    dict(seqs=[(9000, 1), (20, 1), (3, 1), (7000, 1)], D=128, Hq=8, Hkv=1), dict(seqs=[(30000, 2)], D=64, Hq=2, Hkv=1),
]


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("i", range(len(SIZES)))
def test_values(i, dtype, layout):
    c = Case(**SIZES[i], dtype=dtype, layout=layout, seed=i, rest=i % 3, poison=True)
    c.check()


@pytest.mark.parametrize("mask", ["tree", "random", "none"])
@pytest.mark.parametrize("i", range(13, 21))
def test_masks(i, mask):
    Case(**SIZES[i], dtype=BF16 if i % 2 else F16, mask=mask, seed=i, poison=True).check(out_dtype=F32 if i % 3 else None)


@pytest.mark.parametrize("dtype,out", [(BF16, F32), (BF16, F16), (F16, F32), (F16, BF16)])
@pytest.mark.parametrize("i", [3, 4, 6, 7, 13, 14, 15, 17, 18])
def test_output_types_and_caps(i, dtype, out):
    c = Case(**SIZES[i], dtype=dtype, seed=i, spread=4.0)
    c.check(out_dtype=out)
    c.check(out_dtype=out, softcap=20.0, strided=True)
    c.check(out_dtype=out, scale=-0.3)
    c.check(out_dtype=out, scale=0.0)


def test_rows_that_see_nothing():
    """Sequences without tokens or rows, more rows than tokens, and rows whose mask is empty."""
    Case([(0, 1), (5, 1), (0, 3), (7, 0), (0, 0), (9, 2)], poison=True).check()
    # no cached token before the rows, and an empty mask for every other row
    Case([(6, 6), (40, 40), (1, 1)], mask="none").check()
    # lens below the number of rows: the first rows' own tokens are not there
    c = Case([(3, 5), (2, 33), (20, 4)], seed=4)
    c.check()
    Case([(3, 5), (2, 33)], mask="random", seed=5).check()


def test_no_pages():
    c = Case([(5, 1), (4, 2)])
    out, lse = torch.ones(3, 8, 64, device="cuda", dtype=BF16), torch.ones(3, 8, device="cuda")
    fb.moe_ffn_attend(c.q, c.k[:0], c.v[:0], c.table, c.lens, c.q_start, out=out, lse=lse)
    assert bool((out == 0).all()) and bool((lse == -INF).all())
    fb.moe_ffn_attend(c.q, c.k, c.v, c.table[:, :0], c.lens, c.q_start, out=out.fill_(1), lse=lse.fill_(1))
    assert bool((out == 0).all()) and bool((lse == -INF).all())


@pytest.mark.parametrize("i", [3, 4, 14, 17])
def test_bad_pages_and_lengths(i):
    """Page ids out of range hide their tokens; lengths past the table end at it, negative ones at 0."""
    c = Case(**SIZES[i], seed=i, mask="tree" if i > 12 else None)
    c.table[0, 1::3] = 2**31 - 1
    c.table[0, 2::5] = -1
    c.table[0, 0] = c.pages
    c.check()
    whole = c.table.shape[1] * c.page
    c = Case([(whole, n) for _, n in SIZES[i]["seqs"]], **{k: v for k, v in SIZES[i].items() if k != "seqs"}, seed=i)
    c.lens.fill_(2**31 - 1)
    c.check()
    c.lens.fill_(-3)
    out = torch.ones_like(c.q)
    c.call(out=out)
    assert float(out.float().abs().max()) == 0


def test_row_bounds_out_of_range():
    """q_start past T, negative or falling: rows inside T are computed or left, nothing else is touched."""
    c = Case([(50, 2), (60, 2), (70, 2)], rest=2)
    for bad in ([0, 2, 4, 100], [-7, 2, 4, 6], [0, 4, 2, 6], [0, 2, 2**31 - 1, 6]):
        full = torch.full((c.T + 4, c.Hq, c.D), 5.0, device="cuda", dtype=BF16)
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        fb.moe_ffn_attend(c.q, c.k, c.v, c.table, c.lens, starts, out=full[2:-2])
        assert bool((full[:2] == 5).all()) and bool((full[-2:] == 5).all())


@pytest.mark.parametrize("i", [13, 14, 15, 17, 18, 19])
@pytest.mark.parametrize("value", [NAN, INF, -INF])
def test_unseen_tokens_have_no_effect(i, value):
    """Infinities and NaN in drafted tokens reach the rows that see them, and no other."""
    c = Case(**SIZES[i], seed=i, mask="tree", dtype=BF16 if i % 2 else F16)
    clean = c.check().clone()
    length, n = c.seqs[0]
    at = length - n // 2 - 1  # one of the first sequence's own tokens
    page, slot = int(c.table[0, at // c.page]), at % c.page
    kept = c.k[page, slot].clone(), c.v[page, slot].clone()
    seen = c.seen(0)[:, at]
    c.v[page, slot, :, 3] = value
    got = c.call()
    assert torch.equal(got[:n][~seen], clean[:n][~seen]) and torch.equal(got[n:], clean[n:])
    hit = got[:n][seen][..., 3]
    assert bool(hit.isnan().all()) if math.isnan(value) else bool((hit == value).all())
    others = [d for d in range(c.D) if d != 3]
    assert torch.equal(got[:n][seen][..., others], clean[:n][seen][..., others])
    c.v[page, slot] = kept[1]
    c.k[page, slot, :, 0] = NAN
    got = c.call()
    assert torch.equal(got[:n][~seen], clean[:n][~seen]) and torch.equal(got[n:], clean[n:])
    assert bool(got[:n][seen].isnan().all())


def test_far_scores():
    """Scores that leave the exponential's range: the largest decides."""
    c = Case([(300, 1), (90, 4)], D=64, spread=60.0)
    c.check()
    c.check(scale=20.0)
    c.check(scale=20.0, out_dtype=F32, softcap=50.0)


def test_strides_and_alignment():
    """Queries and outputs of any stride and alignment, a table and a mask inside wider rows."""
    c = Case([(100, 3), (333, 20)], D=72, Hq=6, Hkv=3, mask="tree", seed=9)
    want = c.check(strided=True).clone()
    wide = torch.zeros(c.T, 7, 75, device="cuda", dtype=BF16)
    wide[:, 1:, 1:73] = c.q
    table = torch.full((2, c.table.shape[1] + 3), -9, dtype=torch.int32, device="cuda")
    table[:, 1:-2] = c.table
    mask = torch.full((c.T, 4), -1, dtype=torch.int32, device="cuda")
    mask[:, 2:3] = c.mask
    out = torch.zeros(c.Hq, c.T, 73, device="cuda", dtype=BF16).transpose(0, 1)[..., 1:]
    fb.moe_ffn_attend(wide[:, 1:, 1:73], c.k, c.v, table[:, 1:-2], c.lens, c.q_start, mask=mask[:, 2:3], out=out)
    assert torch.equal(out, want)


def test_large_offsets():
    """Pages past 2^31 elements of a cache."""
    if torch.cuda.mem_get_info()[0] < 20 * 2**30:
        pytest.skip("needs 10 GB")
    c = Case([(600, 1), (90, 5)], D=64, Hq=8, Hkv=2, page=16)
    pages = 2**31 // (16 * 2 * 64) + c.pages + 3
    k, v = (torch.empty(pages, 16, 2, 64, device="cuda", dtype=BF16) for _ in range(2))
    k[-c.pages:], v[-c.pages:] = c.k, c.v
    table = torch.where(c.table >= 0, c.table + (pages - c.pages), c.table)
    got = fb.moe_ffn_attend(c.q, k, v, table, c.lens, c.q_start)
    assert torch.equal(got, c.call())


@pytest.mark.parametrize("i", [2, 4, 14, 15, 21])
def test_repeats_graphs_streams_and_workspaces(i):
    """Equal bits in every call: on a stale workspace, on another stream, replayed with other lengths in between."""
    c = Case(**SIZES[i], seed=i, mask="tree" if i > 12 else None)
    want, wl = torch.zeros_like(c.q), torch.zeros(c.T, c.Hq, device="cuda")
    c.call(out=want, lse=wl)
    ws = torch.full((fb.moe_ffn_attend_workspace(c.T, len(c.seqs), c.Hq, c.Hkv, c.D),), 255, dtype=torch.uint8, device="cuda")
    out, lse = torch.zeros_like(want), torch.zeros_like(wl)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    c.call(out=out, lse=lse, workspace=ws, stream=stream)
    stream.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, wl)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.call(out=out, lse=lse, workspace=ws)
    lens = c.lens.clone()
    for step in (0, 1, 0):
        c.lens.copy_(torch.clamp(lens - step * 37, min=1))
        ws.random_(0, 256)
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        if step == 0:
            assert torch.equal(out, want) and torch.equal(lse, wl)
        else:
            assert torch.equal(out, c.call())


def test_a_sequence_by_itself_and_among_others():
    """What a sequence gets does not depend on the others but for the rounding of the sums."""
    big = Case([(2000, 4), (70, 1), (900, 16)], D=128, Hq=16, Hkv=4, mask="tree", seed=3)
    out = big.check()
    alone = torch.zeros_like(out)
    for b in range(3):
        rows = slice(big.starts[b], big.starts[b + 1])
        alone[rows] = fb.moe_ffn_attend(big.q[rows], big.k, big.v, big.table[b:b + 1], big.lens[b:b + 1],
                                        torch.tensor([0, big.seqs[b][1]], dtype=torch.int32, device="cuda"), mask=big.mask[rows])
    # (two results, each within its bound)
    _, err, _, _ = big.reference()
    d = (alone.double() - out.double()).abs() - 2 * (err + half_step(out.double().abs() + err, BF16))
    assert float(d.max()) <= 0


def test_many_sequences():
    host = random.Random(1)
    Case([(host.randint(0, 90), host.choice([1, 1, 2])) for _ in range(1500)], D=64, Hq=2, Hkv=1, page=16).check()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("page", [8, 64])
def test_many_units_of_many_rows(D, page):
    """Several units of a few steps for every block, one behind the other, the same bits every time."""
    host = random.Random(D)
    seqs = [(host.choice([16, 40, 64, 65, 128, 129, 300]), host.choice([16, 16, 3, 9])) for _ in range(1300)]
    c = Case(seqs, D=D, Hq=8, Hkv=1, page=page, mask="tree", seed=D, poison=True)
    want = c.check()
    for _ in range(5):
        assert torch.equal(c.call(), want)


@pytest.mark.parametrize("n,G", [(16, 8), (1, 64), (40, 3)])
def test_long_units_of_many_rows(n, G):
    """Many steps a block, parts of units in many blocks, the same bits every time."""
    c = Case([(8192, n), (5000, n), (7300, n)] + [(2048, n)] * 9, D=128, Hq=4 * G, Hkv=4, page=64, mask="tree" if n > 1 else None, seed=n)
    want = c.check()
    for _ in range(20):
        assert torch.equal(c.call(), want)


@pytest.mark.parametrize("i", [4, 9, 14, 15, 17, 19])
def test_a_row_that_is_not_finite_stays_alone(i):
    """NaN and infinities in one query touch no other row or head, whatever shares its tile."""
    c = Case(**SIZES[i], seed=i, mask="tree" if i > 12 else None)
    clean = c.check().clone()
    t, h = c.starts[-1] // 2, c.Hq // 2
    for value in (NAN, INF):
        c.q[t, h, 1] = value
        got = c.call()
        assert bool(got[t, h].isnan().all())
        got[t, h] = clean[t, h]
        assert torch.equal(got, clean)


def test_a_prompt():
    """Rows by the thousand, several tiles of a sequence, another one's next tokens beside them."""
    Case([(1500, 1000), (700, 1), (64, 64)], D=128, Hq=8, Hkv=2, page=32, seed=2).check()
    Case([(900, 900), (40, 2)], D=64, Hq=6, Hkv=2, page=16, dtype=F16, seed=3).check(out_dtype=F32)


def test_calls_on_two_streams_at_once():
    """Calls that overlap, each with a workspace of its own: narrow beside wide, the results of each alone."""
    cases = [Case([(3000, 16), (700, 16)], D=128, Hq=16, Hkv=2, page=64, mask="tree", seed=1),
             Case([(5000, 1)] * 6, D=128, Hq=16, Hkv=2, page=16, seed=2),
             Case([(900, 40)] * 3, D=64, Hq=8, Hkv=2, page=8, mask="tree", seed=3)]
    want = [c.call() for c in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    got = [[torch.zeros_like(w) for _ in range(10)] for w in want]
    ws = [torch.empty(fb.moe_ffn_attend_workspace(c.T, len(c.seqs), c.Hq, c.Hkv, c.D), dtype=torch.uint8, device="cuda")
          for c in cases]
    torch.cuda.synchronize()
    for k in range(10):
        for c, s, g, w in zip(cases, streams, got, ws):
            c.call(out=g[k], workspace=w, stream=s)
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert all(torch.equal(x, w) for x in g)


ODD = [
    dict(seqs=[(3000, 1), (700, 1)], D=128, Hq=16, Hkv=2), dict(seqs=[(300, 1)] * 400, D=64, Hq=8, Hkv=1),
    dict(seqs=[(700, 3), (130, 2)], D=80, Hq=12, Hkv=2, page=5), dict(seqs=[(400, 2), (90, 1)], D=256, Hq=8, Hkv=1, page=32),
    dict(seqs=[(260, 3)], D=192, Hq=16, Hkv=1, page=8), dict(seqs=[(3000, 16), (700, 9)], D=128, Hq=32, Hkv=4, page=64),
    dict(seqs=[(200, 16)] * 400, D=64, Hq=8, Hkv=1), dict(seqs=[(900, 40), (500, 40)], D=72, Hq=12, Hkv=2, page=24),
    dict(seqs=[(1500, 1000)], D=128, Hq=8, Hkv=2, page=32), dict(seqs=[(40000, 1)], D=64, Hq=2, Hkv=2)]


@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("i", range(len(ODD)))
def test_infinities_in_tokens_that_all_rows_see(i, dtype):
    """A value that is not finite makes its column so for its sequence and heads, wherever in the cache its token lies:
    weights are above 0, so an infinity stays one, NaN and infinities of both signs give NaN."""
    c = Case(**ODD[i], seed=i, dtype=dtype, mask="tree" if max(n for _, n in ODD[i]["seqs"]) > 1 else None, poison=True)
    clean = c.check().clone()
    G, b = c.Hq // c.Hkv, len(c.seqs) - 1
    rows, common = slice(c.starts[b], c.starts[b + 1]), c.seqs[b][0] - c.seqs[b][1]
    place = lambda at: (int(c.table[b, at // c.page]), at % c.page)  # noqa: E731
    for tokens, values, want in (([0], [INF], INF), ([common - 1], [-INF], -INF), ([common // 2], [NAN], NAN),
                                 ([1, common // 2], [INF, INF], INF), ([common // 3, common - 2], [-INF, INF], NAN)):
        kept = c.v.clone()
        for at, value in zip(tokens, values):
            c.v[place(at)][0, 3] = value
        got = c.call()
        hit = got[rows, :G, 3].clone()
        assert bool(hit.isnan().all()) if math.isnan(want) else bool((hit == want).all())
        got[rows, :G, 3] = clean[rows, :G, 3]
        assert torch.equal(got, clean)
        c.v.copy_(kept)


@pytest.mark.parametrize("i", range(len(ODD)))
def test_infinities_of_small_weights(i):
    """Tokens whose weights are far below what fp32 holds beside the largest one's: the formula's weights are above 0."""
    c = Case(**ODD[i], seed=i, dtype=F16 if i % 2 else BF16, spread=40.0)
    clean = c.call(out=torch.zeros_like(c.q))
    length, n = c.seqs[0]
    k = c.k[c.table[0].long()[torch.arange(length - n, device="cuda") // c.page], torch.arange(length - n, device="cuda") % c.page]
    score = k[:, 0].double() @ c.q[0, 0].double()
    least, most = int(score.argmin()), int(score.argmax())
    for at, value in ((least, INF), (most, -INF)):
        c.v[int(c.table[0, at // c.page]), at % c.page, 0, 5] = value
        got = c.call(out=torch.zeros_like(clean))
        G = c.Hq // c.Hkv
        want = INF if at == least else NAN
        hit = got[:n, :G, 5].clone()
        assert bool(hit.isnan().all()) if math.isnan(want) else bool((hit == want).all())
        got[:n, :G, 5] = clean[:n, :G, 5]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("D,n", [(64, 1), (128, 1), (64, 9), (128, 9), (256, 2)])
def test_an_infinity_gives_the_same_as_the_sequence_grows(D, n):
    """The same cached token while its tile is the last one, and once it is full."""
    c = Case([(800, n)], D=D, Hq=8, Hkv=1, seed=D + n)
    c.v[int(c.table[0, 2]), 5, 0, 1] = INF
    for length in (2 * 16 + 5 + n, 60, 64, 65, 128, 129, 300, 800):
        c.lens.fill_(max(length, 2 * 16 + 6 + n))
        got = c.call()
        assert bool((got[..., 1] == INF).all()) and bool(got[..., 0].isfinite().all())


@pytest.mark.parametrize("page,n", [(16, 1), (16, 40), (5, 1)])
def test_rows_of_sequences_without_tokens(page, n):
    """Thousands of them, beside sequences that have some: zeros, in strided rows too, and nothing beside them."""
    c = Case([(0, 4000), (300, n), (0, 1), (0, 77), (90, n)] + [(0, 1)] * 700 + [(40, n)], Hq=6, Hkv=2, D=72, page=page, rest=3)
    c.check()
    c.check(strided=True)
    c.check(out_dtype=F32)
    c.lens.zero_()
    out, lse = torch.ones_like(c.q), torch.ones(c.T, 6, device="cuda")
    c.call(out=out, lse=lse)
    end = c.starts[-1]
    assert bool((out[:end] == 0).all()) and bool((lse[:end] == -INF).all()) and bool((out[end:] == 1).all()) and bool((lse[end:] == 1).all())


def test_rows_of_sequences_without_tokens_hold_up_nobody():
    """512 rows of 32 heads of 128 are 4 MB of zeros: microseconds, and not a thread's work, element by element (30 ms)."""
    c = Case([(0, 512), (2000, 1)], D=128, Hq=32, Hkv=4)
    out, times = torch.ones_like(c.q), []
    for _ in range(5):
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        c.call(out=out)
        end.record()
        torch.cuda.synchronize()
        times.append(start.elapsed_time(end))
    assert min(times) < 3.0, times
    assert bool((out[:512] == 0).all())


@pytest.mark.parametrize("low", [-2**31, -2**31 + 1, -2**31 + 5, -1])
@pytest.mark.parametrize("page", [16, 5])
def test_row_starts_far_below_zero(low, page):
    """A sequence whose rows end below 0 has none, however far: the difference of its bounds passes 32 bits."""
    c = Case([(50, 2), (60, 20), (70, 2)], rest=3, page=page)
    for bad, has in (([0, 2, low, 24], [2, 0, 24]), ([4, low, low, 3], [0, 0, 3]), ([20, low, 10, low], [0, 10, 0])):
        full = torch.full((c.T + 4, c.Hq, c.D), 5.0, device="cuda", dtype=BF16)
        starts = torch.tensor(bad, dtype=torch.int32, device="cuda")
        got = fb.moe_ffn_attend(c.q, c.k, c.v, c.table, c.lens, starts, out=full[2:-2])
        rows = torch.zeros(c.T + 4, dtype=torch.bool, device="cuda")
        for b in range(3):
            first = max(bad[b], 0)
            rows[2 + first:2 + first + has[b]] = True
        assert bool((full[~rows] == 5).all()) and not bool((full[rows] == 5).all(-1).any())
        assert bool(got.isfinite().all())


@pytest.mark.parametrize("n", [1, 16])
@pytest.mark.parametrize("page", [8, 3])
def test_the_largest_batch(n, page):
    """65,536 sequences, a row or 16 of each, some without tokens or with fewer than rows, pages in any order."""
    B, D, most = 65536, 8, 24
    g = torch.Generator(device="cuda").manual_seed(n + page)
    lens = torch.randint(0, most + 1, (B,), generator=g, device="cuda").to(torch.int32)
    pages = 40000
    k, v = (torch.randn(pages, page, 1, D, generator=g, device="cuda").bfloat16() for _ in range(2))
    table = torch.randint(0, pages, (B, most // page), generator=g, device="cuda").to(torch.int32)
    q = torch.randn(B * n, 1, D, generator=g, device="cuda").bfloat16()
    starts = (torch.arange(B + 1, device="cuda") * n).to(torch.int32)
    out, lse = torch.full((B * n, 1, D), 5.0, device="cuda"), torch.full((B * n, 1), 5.0, device="cuda")
    fb.moe_ffn_attend(q, k, v, table, lens, starts, out=out, lse=lse)
    i = torch.arange(most, device="cuda")
    at = table.long()[:, i // page], (i % page)[None]
    keys, values = k[at][:, :, 0].double(), v[at][:, :, 0].double()  # [B, most, D]
    rows = q.view(B, n, D).double()
    s = torch.einsum("bjd,bid->bji", rows, keys) * D**-0.5
    # as in Case.reference, with sums of 24 tokens of 8 elements
    ds = torch.einsum("bjd,bid->bji", rows.abs(), keys.abs()) * (D**-0.5 * (D / 8 + 10) * 2.0**-23)
    own = i[None] - (lens[:, None] - n)
    seen = (own[:, None] <= torch.arange(n, device="cuda")[None, :, None]) & (i[None] < lens[:, None])[:, None]
    s = s.masked_fill(~seen, -INF)
    top = s.amax(-1, keepdim=True)
    none = top == -INF
    top = top.masked_fill(none, 0.0)
    p = torch.exp(s - top)
    total = p.sum(-1, keepdim=True).masked_fill(none, 1.0)
    p = p / total
    dp = ds + (s.abs().masked_fill(~seen, 0.0) + top.abs() + 2) * 2.0**-22
    e, adds = (p * dp).sum(-1, keepdim=True), (most / 8 + 64) * 2.0**-23
    want, size = torch.einsum("bji,bid->bjd", p, values), torch.einsum("bji,bid->bjd", p, values.abs())
    err = torch.einsum("bji,bid->bjd", p * dp, values.abs()) + size * (e + 2 * adds + 2.0**-20)
    d = (out.view(B, n, D).double() - want).abs() - err - half_step(want.abs() + err, F32)
    assert float(d.max()) <= 0, float(d.max())
    none = none.view(-1, 1)
    assert torch.equal(lse == -INF, none) and bool((out[none[:, 0]] == 0).all())
    wl, el = (top + torch.log(total)).view(-1, 1), e.view(-1, 1) + adds
    dl = ((lse.double() - wl).abs() - el - (wl.abs() + 8) * 2.0**-22)[~none]
    assert float(dl.max()) <= 0, float(dl.max())


def test_the_first_call_in_a_capture():
    """A process whose first calls of the library are captured, replayed then."""
    import os
    import subprocess
    import sys

    code = """
import torch
import fusion_backend_gb300 as fb
z = lambda *s, dtype=torch.bfloat16: torch.ones(s, device="cuda", dtype=dtype)
x, w = z(40, 256), z(64, 160, dtype=torch.uint8)
q, k, kc, vc = z(40, 8, 64), z(40, 1, 64), z(9, 16, 1, 64), z(9, 16, 1, 64)
i = torch.arange(40, device="cuda", dtype=torch.int32)
table, lens, starts = i[:3].view(1, 3).contiguous(), i[:1] + 40, i[:2] * 40
f = torch.zeros(32, device="cuda")
out, y, qo = torch.zeros_like(q), z(40, 64), torch.zeros_like(q)
ws = torch.empty(fb.moe_ffn_attend_workspace(40, 1, 8, 1, 64), dtype=torch.uint8, device="cuda")
graph = torch.cuda.CUDAGraph()
torch.cuda.synchronize()
with torch.cuda.graph(graph):
    fb.moe_ffn_project(x, w, out=y)
    fb.moe_ffn_append_kv(k, k, i, i, f, kc, vc, q=q, q_out=qo)
    fb.moe_ffn_attend(qo, kc, vc, table, lens, starts, out=out, workspace=ws)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (y, qo, kc, vc, out)]
fb.moe_ffn_project(x, w, out=y)
fb.moe_ffn_append_kv(k, k, i, i, f, kc, vc, q=q, q_out=qo)
fb.moe_ffn_attend(qo, kc, vc, table, lens, starts, out=out, workspace=ws)
assert all(torch.equal(a, b) for a, b in zip(got, (y, qo, kc, vc, out)))
assert bool((out == 1).all())
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]
