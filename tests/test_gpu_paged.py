"""The paged KV cache: page tables, the rotary write, and attention of new rows
over the pages, against plain implementations (in whole numbers, and in 64
bits).  Tolerances are error bounds of the arithmetic, element by element: a
rounding to bf16 counts 2^-8 of the value, a tensor-core sum one truncation of
2^-23 per 16-deep step, an exponential 2^-22.
"""
import math
import random

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

U, F32, TC = 2.0 ** -8, 2.0 ** -24, 2.0 ** -23


@pytest.fixture(scope="module")
def g():
    if not torch.cuda.is_available():
        pytest.fail("gpu tests need a CUDA device")
    from self_speculative_block_gb300 import build, gocr
    build.build()
    gocr.load()
    return gocr


def i32(a):
    return torch.tensor(a, dtype=torch.int32, device="cuda")


# ----------------------------------------------------------------------------
# page step
# ----------------------------------------------------------------------------

class Pool:
    """The page step in plain Python."""

    def __init__(self, R, width, ps, n_pages, order):
        self.ps, self.width, self.n_pages = ps, width, n_pages
        self.table = [[-1] * width for _ in range(R)]
        self.free, self.n_free = list(order), n_pages
        self.held = [0] * R

    def step(self, held, start, end, T):
        ps, cap = self.ps, self.width * self.ps
        pages = lambda n: -(-n // ps)
        sane = [0 <= s <= h and s <= e and h <= cap and e <= cap for h, s, e in zip(held, start, end)]
        cu = [0]
        for ok, s, e in zip(sane, start, end):
            cu.append(cu[-1] + (e - s if ok else 0))
        good = [ok and cu[r + 1] <= T for r, ok in enumerate(sane)]
        back = [self.table[r][i] for r in range(len(held)) if good[r] for i in range(pages(end[r]), pages(held[r]))]
        stack = self.free[:self.n_free] + back[::-1]
        self.free[:len(stack)] = stack
        pos, slots = [-1] * T, [-1] * T
        out_held, kv_len, asked, left = [], [], 0, len(stack)
        for r, (h, s, e) in enumerate(zip(held, start, end)):
            need = max(0, pages(e) - pages(h)) if good[r] else 0
            asked += need
            ok = good[r] and (need == 0 or asked <= len(stack))
            out_held.append(e if ok else h)
            kv_len.append(e if ok else 0)
            if not ok:
                continue
            for i in range(pages(h), pages(e)):
                left -= 1
                self.table[r][i] = stack[left]
            for x in range(s, e):
                pos[cu[r] + x - s] = x
                slots[cu[r] + x - s] = self.table[r][x // ps] * ps + x % ps
        self.n_free, self.held = left, out_held
        return dict(n_free=[left], held=out_held, kv_len=kv_len, cu_rows=[min(c, T) for c in cu], pos=pos, slots=slots)


def _pool(R, width, ps, n_pages, seed):
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    return Pool(R, width, ps, n_pages, order), torch.full((R, width), -1, dtype=torch.int32, device="cuda"), i32(order), i32([n_pages])


def _same_step(g, pool, table, free, n_free, held, start, end, T):
    want = pool.step(held, start, end, T)
    got = g.op_page_step(i32(held), i32(start), i32(end), table, free, n_free, pool.ps, T)
    for name, x in want.items():
        assert getattr(got, name).tolist() == x, name
    assert table.tolist() == pool.table
    assert free.tolist() == pool.free
    return got


@pytest.mark.parametrize("ps", [16, 64, 256])
@pytest.mark.parametrize("R", [1, 5, 32, 257, 700])
def test_page_step_follows_a_serving_run(g, R, ps):
    """Random steps of growth, windows over held positions, rollbacks and ends, with a pool that runs short."""
    rng = random.Random(R * 1000 + ps)
    width = 9
    pool, table, free, n_free = _pool(R, width, ps, max(4, R * 4), R)
    for _ in range(12):
        held, start, end = list(pool.held), [], []
        for h in held:
            kind = rng.random()
            cap = width * ps
            if kind < 0.5:
                s, e = h, min(cap, h + rng.randint(0, 3 * ps // 2))
            elif kind < 0.7:
                s = max(0, h - rng.randint(0, 40))
                e = min(cap, s + rng.randint(0, 60))
            elif kind < 0.85:
                s = e = rng.randint(0, h)
            elif kind < 0.95:
                s = e = 0
            else:
                s, e = rng.choice([(h + 1, h + 2), (h, h - 1), (-1, h), (h, cap + 1), (0, -5)])
            start.append(s)
            end.append(e)
        rows = sum(max(0, e - s) for s, e in zip(start, end))
        T = rng.choice([rows + 40, rows, max(0, rows - rng.randint(1, 50)), 0, 7])
        n_free = _same_step(g, pool, table, free, n_free, held, start, end, T).n_free


def test_page_step_growth_rolled_back_leaves_the_stack(g):
    R, ps = 40, 16
    pool, table, free, n_free = _pool(R, 30, ps, 900, 3)
    rng = random.Random(4)
    base = [rng.randint(0, 300) for _ in range(R)]
    n0 = _same_step(g, pool, table, free, n_free, [0] * R, [0] * R, base, sum(base)).n_free
    before = free[:int(n0)].tolist()
    n1 = _same_step(g, pool, table, free, n0, base, base, [b + 33 for b in base], 33 * R).n_free
    n2 = _same_step(g, pool, table, free, n1, [b + 33 for b in base], base, base, 0).n_free
    assert int(n2) == int(n0) and free[:int(n2)].tolist() == before


def test_page_step_takes_pages_that_the_same_call_gives_back(g):
    """An empty stack: the first request ends, the second takes its pages, the third finds none."""
    pool, table, free, n_free = _pool(3, 8, 16, 6, 5)
    n1 = _same_step(g, pool, table, free, n_free, [0, 0, 0], [0, 0, 0], [64, 32, 0], 96).n_free
    assert int(n1) == 0
    got = _same_step(g, pool, table, free, n1, [64, 32, 0], [0, 32, 0], [0, 96, 1], 65)
    assert got.held.tolist() == [0, 96, 0] and got.kv_len.tolist() == [0, 96, 0] and int(got.n_free) == 0


@pytest.mark.parametrize("R", [0, 4096])
def test_page_step_smallest_and_largest(g, R):
    ps, width = 16, 3
    pool, table, free, n_free = _pool(R, width, ps, 2 * 4096, 6)
    held = [0] * R
    end = [r % (width * ps + 1) for r in range(R)]
    n = _same_step(g, pool, table, free, n_free, held, held, end, sum(end) + 5).n_free
    _same_step(g, pool, table, free, n, pool.held, [0] * R, [0] * R, 0)


def test_page_step_bad_state_stays_in_bounds(g):
    """Stacks and tables that contradict the lengths: no page of such a step leads outside the cache."""
    n_pages, ps = 8, 16
    table = i32([[99, -7, 5, 2 ** 31 - 1], [3, 4, -2 ** 31, 8], [0, 1, 2, 3]])
    free = i32([2 ** 31 - 1, -5, 8, 1000, 7, 6, -1, 3])
    for n_free in (-3, 0, 8, 2 ** 31 - 1):
        s = g.op_page_step(i32([64, 0, 20]), i32([0, 0, 20]), i32([64, 0, 64]), table.clone(), free.clone(), i32([n_free]), ps, 128)
        torch.cuda.synchronize()
        assert int(s.slots.max()) < n_pages * ps and int(s.slots.min()) >= -1
        assert 0 <= int(s.n_free) <= n_pages


# ----------------------------------------------------------------------------
# a cache
# ----------------------------------------------------------------------------

LAYOUTS = ["head", "token", "interleaved", "pages-inside"]


def _empty_cache(layout, n_pages, Hkv, ps, d, fill=0.0):
    """K and V pages [n_pages, Hkv, ps, d] whose strides run in another order."""
    new = lambda *s: torch.full(s, fill, dtype=torch.bfloat16, device="cuda")
    if layout == "head":
        return new(n_pages, Hkv, ps, d), new(n_pages, Hkv, ps, d)
    if layout == "token":
        return tuple(new(n_pages, ps, Hkv, d).transpose(1, 2) for _ in range(2))
    if layout == "interleaved":  # one array of two layers' K and V pages; the second layer's
        both = new(n_pages, 2, 2, Hkv, ps, d)
        return both[:, 1, 0], both[:, 1, 1]
    return tuple(new(Hkv, ps, n_pages, d).permute(2, 0, 1, 3) for _ in range(2))


def _tables(kv_lens, ps, seed, width=None, spare=3):
    """A block table of shuffled pages and the number of pages; entries behind a request's pages lead nowhere."""
    pages = [-(-max(0, n) // ps) for n in kv_lens]
    n_pages = sum(pages) + spare
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    width = width or max(1, *pages)
    table, at = [], 0
    for i, n in enumerate(pages):
        n = min(n, width)
        table.append(order[at:at + n] + [(-1, n_pages, 2 ** 31 - 1, -2 ** 31)[i % 4]] * (width - n))
        at += n
    return table, n_pages


# ----------------------------------------------------------------------------
# rotary write
# ----------------------------------------------------------------------------

def _rotated(x, pos, theta):
    """The rotation in 64 bits, and the bound of the kernel's error."""
    d = x.shape[-1]
    inv = theta ** (-torch.arange(0, d, 2, dtype=torch.float64, device="cuda") / d)
    ang = pos.double()[:, None, None] * inv
    a, b = x[..., :d // 2].double(), x[..., d // 2:].double()
    y = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1)
    # an angle off by 2^-26 turns, sincospi by 2 ulp, two products and a sum, then the rounding
    f = (2 * math.pi * 2.0 ** -26 + 6 * F32) * torch.cat([a.abs() + b.abs()] * 2, -1)
    return y, f + U * (y.abs() + f) + 1e-38


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("Hq,Hkv,d,ps", [(12, 4, 128, 16), (4, 2, 64, 32), (1, 1, 128, 256), (7, 7, 64, 64), (64, 1, 64, 16)])
@pytest.mark.parametrize("T", [1, 2, 33, 500])
def test_kv_write(g, T, Hq, Hkv, d, ps, layout):
    r = torch.Generator(device="cuda").manual_seed(T + Hq + d)
    n_pages = -(-T // ps) + 3
    kc, vc = _empty_cache(layout, n_pages, Hkv, ps, d, fill=5.0)
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda").bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.randint(0, 1 << 20, (T,), generator=r, device="cuda", dtype=torch.int32)
    slots = torch.randperm(n_pages * ps, generator=r, device="cuda")[:T].to(torch.int32)
    out = g.op_kv_write_paged(q, k, v, pos, slots, kc, vc, theta=10000.0)
    for got, x in ((out, q), (kc[slots.long() // ps, :, slots.long() % ps], k)):
        val, tol = _rotated(x, pos, 10000.0)
        assert ((got.double() - val).abs() <= tol).all()
    assert torch.equal(vc[slots.long() // ps, :, slots.long() % ps], v)
    other = torch.ones((n_pages * ps,), dtype=torch.bool, device="cuda")
    other[slots.long()] = False
    for c in (kc, vc):
        assert (c.transpose(1, 2).reshape(n_pages * ps, Hkv, d)[other] == 5.0).all()


@pytest.mark.parametrize("theta", [1.0, 10000.0, 5e5])
def test_kv_write_far_positions(g, theta):
    """Angles of the farthest positions keep the precision of near ones; position 0 changes nothing."""
    pos = i32([0, 1, 2 ** 24 - 1, 2 ** 24 - 2, 12345678, 2 ** 31 - 1])
    T, Hq, Hkv, d, ps = 6, 2, 1, 128, 16
    q = torch.randn((T, Hq, d), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)).bfloat16()
    kc, vc = _empty_cache("head", 1, Hkv, ps, d)
    out = g.op_kv_write_paged(q, q[:, :1].contiguous(), q[:, 1:].contiguous(), pos, i32(list(range(T))), kc, vc, theta=theta)
    val, tol = _rotated(q, pos, theta)
    assert ((out.double() - val).abs() <= tol).all()
    assert torch.equal(out[0], q[0])


def test_kv_write_skips_rows_without_a_slot(g):
    """Slots outside the cache: nothing is written for them, whatever the rows hold."""
    T, Hq, Hkv, d, ps = 40, 4, 2, 64, 16
    kc, vc = _empty_cache("head", 3, Hkv, ps, d, fill=2.0)
    q, k = torch.ones((T, Hq, d), device="cuda").bfloat16(), torch.ones((T, Hkv, d), device="cuda").bfloat16()
    q[3:] = math.nan
    k[3:] = math.inf
    slots = i32([0, 47, 16] + [-1, 48, 2 ** 31 - 1, -2 ** 31] * 10)[:T]
    q_out = torch.full((T, Hq, d), 9.0, device="cuda").bfloat16()
    g.op_kv_write_paged(q, k, k, i32([0] * T), slots, kc, vc, q_out=q_out)
    assert (q_out[:3] == 1.0).all() and (q_out[3:] == 9.0).all()
    for c in (kc, vc):
        rows = c.transpose(1, 2).reshape(48, Hkv, d)
        assert (rows[[0, 16, 47]] == 1.0).all() and (rows == 1.0).sum() == 3 * Hkv * d and (rows == 2.0).sum() == 45 * Hkv * d


# ----------------------------------------------------------------------------
# attention
# ----------------------------------------------------------------------------

def _case(rows, kv_lens, Hq, Hkv, d, ps, layout, seed, pad=0, qscale=1.0, width=None, junk=math.nan):
    """Requests of rows[r] new rows and kv_lens[r] keys; every place of the cache that is no request's key holds junk."""
    r = torch.Generator(device="cuda").manual_seed(seed)
    table, n_pages = _tables(kv_lens, ps, seed, width)
    kc, vc = _empty_cache(layout, n_pages, Hkv, ps, d, fill=junk)
    K, V = [], []
    for i, n in enumerate(kv_lens):
        n = min(max(0, n), len(table[i]) * ps)
        k, v = (torch.randn((n, Hkv, d), generator=r, device="cuda").bfloat16() for _ in range(2))
        at = torch.arange(n, device="cuda")
        page = i32(table[i]).long()[at // ps]
        kc[page, :, at % ps], vc[page, :, at % ps] = k, v
        K.append(k)
        V.append(v)
    T = sum(rows) + pad
    q = (qscale * torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda")).bfloat16()[:, :Hq]
    cu = torch.tensor([0] + list(rows), device="cuda").cumsum(0).to(torch.int32)
    return dict(q=q, kc=kc, vc=vc, table=i32(table), cu=cu, kv_len=i32(kv_lens), K=K, V=V, rows=list(rows))


def _attend(g, c, kind, scale=None, **kw):
    return g.op_attention_paged(c["q"], c["kc"], c["vc"], c["table"], c["cu"], c["kv_len"], kind=kind, scale=scale, **kw)


def _check(g, c, kind, o, lse, scale=None):
    """o and lse of the requests' rows against 64 bits, within the bounds of the kernel's errors."""
    t0, (T, Hq, d) = 0, c["q"].shape
    scale = d ** -0.5 if scale is None else scale
    for r, n in enumerate(c["rows"]):
        kv = len(c["K"][r])
        G = Hq // c["K"][r].shape[1]
        rows = slice(t0, t0 + n)
        t0 += n
        if n == 0:
            continue
        last = torch.arange(kv - n, kv, device="cuda")
        if kind == g.FWD_DRAFT:
            last[1:] = kv - 1
        seen = torch.arange(kv, device="cuda")[None, :] <= last[:, None]
        none = last < 0
        assert (o[rows][none] == 0).all() and (lse[:, rows][:, none] == -math.inf).all()
        for h in range(Hq):
            Q, K, V = c["q"][rows, h].double(), c["K"][r][:, h // G].double(), c["V"][r][:, h // G].double()
            S = (Q @ K.T * scale).masked_fill(~seen, -math.inf)
            ref = torch.logsumexp(S, 1)
            P = torch.exp(S - ref[:, None]).masked_fill(none[:, None], 0.0)
            big = torch.where(seen, S, 0.0).abs().amax(1) if kv else torch.zeros(n, device="cuda")
            # relative error of an exponential: its argument's and its own; the parts of a split key axis are
            # joined with one more of each, and two roundings a part of 128 keys or more
            e = ((torch.where(seen, (Q.abs() @ K.abs().T) * scale, 0.0).amax(1) if kv else 0.0) * (d / 16 + 16) * TC
                 + 8 * big * F32 + 8 * F32)
            deep = (kv / 16 + 64) * TC
            O = P @ V
            tol = (U + 2 * e + deep)[:, None] * (P @ V.abs()) + U * O.abs() + 1e-38
            err = (o[rows, h].double() - O).abs()
            assert (err <= tol)[~none].all(), (r, h, float((err / tol)[~none].max()))
            err = (lse[h, rows].double() - ref).abs()
            assert (err <= e + kv * F32 + 4 * F32 * ref.abs())[~none].all(), (r, h, float(err[~none].max()))


HEADS = [(12, 4, 128), (4, 2, 64), (1, 1, 128), (5, 1, 64), (48, 3, 64), (64, 1, 128)]
CASES = {  # rows, kv_lens
    "one": ([1], [1]),
    "one-key-more": ([1], [2]),
    "tokens": ([1] * 9, [1, 15, 16, 17, 127, 128, 129, 500, 2000]),
    "windows": ([33] * 5, [33, 34, 160, 161, 1031]),
    "chunks": ([200, 129, 1], [200, 1000, 64]),
    "ragged": ([3, 0, 77, 1, 128, 0, 42], [3, 50, 300, 7, 128, 0, 1500]),
    "no-keys": ([5, 4, 40, 1], [0, 2, 13, -7]),
    "long-chunk": ([700], [1900]),
    "many": ([1, 2, 1, 33] * 40, [5, 2, 311, 70] * 40),
}


@pytest.mark.parametrize("kind", ["verify", "draft"])
@pytest.mark.parametrize("Hq,Hkv,d", HEADS)
@pytest.mark.parametrize("name", CASES)
def test_attention_paged(g, name, Hq, Hkv, d, kind):
    rows, kv = CASES[name]
    k = g.FWD_DRAFT if kind == "draft" else g.FWD_VERIFY
    i = list(CASES).index(name) + Hq
    c = _case(rows, kv, Hq, Hkv, d, [16, 32, 64, 128, 256][i % 5], LAYOUTS[i % 4], seed=i)
    o, lse = _attend(g, c, k)
    g.op_status()
    _check(g, c, k, o, lse)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("ps", [16, 32, 64, 128, 256])
def test_attention_paged_every_page_size_and_layout(g, ps, layout):
    c = _case([1, 33, 300], [ps + 1, 1000, 777], 6, 2, 128, ps, layout, seed=ps)
    o, lse = _attend(g, c, g.FWD_VERIFY)
    _check(g, c, g.FWD_VERIFY, o, lse)


@pytest.mark.parametrize("d", [64, 128])
def test_attention_paged_long_context(g, d):
    """One request whose key axis is split over the whole device, beside short ones."""
    c = _case([33, 1, 2], [40001, 1, 130], 3, 1, d, 16, "head", seed=d)
    for kind in (g.FWD_VERIFY, g.FWD_DRAFT):
        o, lse = _attend(g, c, kind)
        _check(g, c, kind, o, lse)


def test_attention_paged_growing_maxima(g):
    """Scores that grow along the keys by hundreds: the running maximum moves in every block and part."""
    c = _case([40, 1], [3000, 2500], 2, 1, 128, 16, "head", seed=4)
    for r, n in enumerate((3000, 2500)):
        ramp = torch.linspace(0.0, 12.0, n, device="cuda").bfloat16()
        c["K"][r][:, 0, 0] = ramp
        at = torch.arange(n, device="cuda")
        c["kc"][c["table"][r].long()[at // 16], 0, at % 16, 0] = ramp
    c["q"][:, :, 0] = 16.0
    o, lse = _attend(g, c, g.FWD_VERIFY, scale=1.0)
    _check(g, c, g.FWD_VERIFY, o, lse, scale=1.0)


def test_attention_paged_leaves_other_rows(g):
    """Rows behind the last request hold NaN: their outputs stay."""
    c = _case([33, 1, 7], [133, 50, 7], 4, 2, 128, 16, "head", seed=5, pad=20)
    T = 61
    c["q"][41:] = math.nan
    c["q"][50] = math.inf
    o, lse = torch.full((T, 4, 128), 7.0, device="cuda").bfloat16(), torch.full((4, T), 7.0, device="cuda")
    _attend(g, c, g.FWD_VERIFY, o=o, lse=lse)
    assert (o[41:] == 7.0).all() and (lse[:, 41:] == 7.0).all()
    _check(g, c, g.FWD_VERIFY, o, lse)


def test_attention_paged_keeps_nan_in_its_request(g):
    c = _case([33, 20, 1], [500, 260, 300], 4, 2, 64, 16, "head", seed=6)
    o, lse = _attend(g, c, g.FWD_VERIFY)
    at = torch.arange(260, device="cuda")
    for cache in (c["kc"], c["vc"]):
        cache[c["table"][1].long()[at // 16], :, at % 16] = math.nan
    c["q"][33:53] = math.inf
    o2, lse2 = _attend(g, c, g.FWD_VERIFY)
    keep = torch.ones(54, dtype=torch.bool, device="cuda")
    keep[33:53] = False
    assert torch.equal(o[keep], o2[keep]) and torch.equal(lse[:, keep], lse2[:, keep])
    assert torch.isnan(o2[33:53]).all()


def test_attention_paged_lengths_above_the_table(g):
    """kv_len above max_pages * page_size is taken for that; tables that lead nowhere read as zeros, within bounds."""
    c = _case([5], [64], 2, 1, 64, 16, "head", seed=7, width=4)
    want = _attend(g, c, g.FWD_VERIFY)
    for n in (65, 1000, 2 ** 31 - 1):
        c["kv_len"].fill_(n)
        got = _attend(g, c, g.FWD_VERIFY)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    c["kv_len"].fill_(64)
    c["table"][:] = i32([[-1, 2 ** 31 - 1, -2 ** 31, 10 ** 6]])
    o, lse = _attend(g, c, g.FWD_VERIFY)
    assert (o == 0).all()
    assert torch.allclose(lse.double(), torch.log(torch.arange(60.0, 65.0, dtype=torch.float64, device="cuda")).expand(2, 5), rtol=1e-6)


def test_attention_paged_row_ranges_out_of_order(g):
    """cu_rows beyond the rows or decreasing: clamped, in bounds."""
    c = _case([5, 6], [64, 70], 2, 1, 64, 16, "head", seed=8)
    for cu in ([0, 2 ** 31 - 1, 2 ** 31 - 1], [-2 ** 31, 5, 11], [11, 5, 0], [0, 11, 5]):
        c["cu"] = i32(cu)
        _attend(g, c, g.FWD_VERIFY)
    torch.cuda.synchronize()
    g.op_status()


def test_attention_paged_same_bits_again(g):
    c = _case([33] * 8 + [200], [1031, 2049, 33, 512, 700, 1500, 90, 4000, 900], 12, 4, 128, 16, "head", seed=9)
    o, lse = _attend(g, c, g.FWD_VERIFY)
    ws = torch.full((g.load().gocr_op_attention_paged_workspace(*c["q"].shape[:2], 4, 128),), 255, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        o2, lse2 = _attend(g, c, g.FWD_VERIFY, workspace=ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_attention_paged_nothing_to_do(g):
    c = _case([5], [9], 2, 1, 64, 16, "head", seed=10)
    e = g.op_attention_paged(c["q"][:0], c["kc"], c["vc"], c["table"], i32([0, 0]), c["kv_len"])
    assert e[0].shape == (0, 2, 64) and e[1].shape == (2, 0)
    o = torch.full((5, 2, 64), 3.0, device="cuda").bfloat16()
    g.op_attention_paged(c["q"], c["kc"], c["vc"], c["table"][:0], i32([0]), c["kv_len"][:0], o=o)
    g.op_attention_paged(c["q"], c["kc"], c["vc"], c["table"], i32([3, 3]), c["kv_len"], o=o)
    assert (o == 3.0).all()


def test_attention_paged_agrees_with_the_packed_one(g):
    """Prompts prefilled whole: the same attention as over packed sequences."""
    lens, Hq, Hkv, d = [200, 1, 333], 6, 2, 128
    c = _case(lens, lens, Hq, Hkv, d, 32, "token", seed=11)
    o, lse = _attend(g, c, g.FWD_VERIFY)
    po, plse = g.op_attention_packed(c["q"], torch.cat(c["K"]), torch.cat(c["V"]), c["cu"])
    assert (o.float() - po.float()).abs().max() <= 4 * U * po.abs().max()
    assert torch.allclose(lse, plse, rtol=1e-5, atol=1e-5)


# ----------------------------------------------------------------------------
# together: rounds of draft, verify and rollback over ragged requests
# ----------------------------------------------------------------------------

def _rounds(g, steps, graph=False):
    """Prefill in two chunks, then rounds of draft, verify and rollback of three requests; yields each forward's
    inputs and outputs.  Forwards are laid out for a few rows more than there are."""
    Hq, Hkv, d, ps, B, R = 4, 2, 64, 16, 7, 3
    r = torch.Generator(device="cuda").manual_seed(12)
    rng = random.Random(13)
    n_pages, width = 90, 40
    kc, vc = _empty_cache("head", n_pages, Hkv, ps, d, fill=math.nan)
    table, free, n_free = torch.full((R, width), -1, dtype=torch.int32, device="cuda"), i32(list(range(n_pages))), i32([n_pages])
    held = [0] * R
    plan = [([0] * R, [40, 17, 90], "verify"), ([40, 17, 90], [100, 18, 230], "verify")]
    p = [100, 18, 230]
    for _ in range(steps):
        plan.append((list(p), [x + B + 1 for x in p], "draft"))
        plan.append(([x + 1 for x in p], [x + B + 2 for x in p], "verify"))
        p = [x + rng.randint(2, B + 2) for x in p]
        plan.append((list(p), list(p), None))
    for start, end, kind in plan:
        n = [e - s for s, e in zip(start, end)]
        T = sum(n) + 3
        s = g.op_page_step(i32(held), i32(start), i32(end), table, free, n_free, ps, T)
        held, n_free = end, s.n_free
        assert s.held.tolist() == end
        if kind is None:
            continue
        qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda").bfloat16()
        q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
        rot = g.op_kv_write_paged(q, k, v, s.pos, s.slots, kc, vc, q_out=torch.zeros((T, Hq, d), device="cuda").bfloat16())
        o, lse = g.op_attention_paged(rot, kc, vc, table, s.cu_rows, s.kv_len,
                                      kind=g.FWD_DRAFT if kind == "draft" else g.FWD_VERIFY)
        yield start, end, kind, q, k, v, rot, o, lse


def test_paged_rounds_equal_a_dense_cache(g):
    dense = [[torch.zeros((0, 2, 64), device="cuda").bfloat16()] * 2 for _ in range(3)]
    for start, end, kind, q, k, v, rot, o, lse in _rounds(g, 6):
        t0, rows = 0, []
        pos = torch.cat([torch.arange(s, e, device="cuda") for s, e in zip(start, end)])
        turned, _ = _rotated(k[:len(pos)], pos, 10000.0)
        val, tol = _rotated(q[:len(pos)], pos, 10000.0)
        assert ((rot[:len(pos)].double() - val).abs() <= tol).all()
        c = dict(q=rot, K=[], V=[], rows=[])
        for r, (s, e) in enumerate(zip(start, end)):
            K, V = dense[r]
            K, V = (torch.cat([x[:s], y[t0:t0 + e - s].bfloat16()]) for x, y in ((K, turned), (V, v)))
            dense[r] = [K, V]
            t0 += e - s
            c["K"].append(K)
            c["V"].append(V)
            c["rows"].append(e - s)
        # the dense keys may round to the neighbouring bf16 where the kernel's fp32 value lies next to a border
        loose = dict(c, K=[x for x in c["K"]])
        _check_loose(g, loose, g.FWD_DRAFT if kind == "draft" else g.FWD_VERIFY, o, lse)


def _check_loose(g, c, kind, o, lse):
    """As _check; a key element that was rounded to the other neighbour is off by 2^-7 of its value at most, so a score
    by 2^-7 |q| |k| scale, if all of them were."""
    t0, (T, Hq, d) = 0, c["q"].shape
    for r, n in enumerate(c["rows"]):
        kv, rows = len(c["K"][r]), slice(t0, t0 + n)
        t0 += n
        last = torch.arange(kv - n, kv, device="cuda")
        if kind == g.FWD_DRAFT:
            last[1:] = kv - 1
        seen = torch.arange(kv, device="cuda")[None, :] <= last[:, None]
        for h in range(Hq):
            Q, K, V = (x.double() for x in (c["q"][rows, h], c["K"][r][:, h // 2], c["V"][r][:, h // 2]))
            S = (Q @ K.T * d ** -0.5).masked_fill(~seen, -math.inf)
            P = torch.softmax(S, 1)
            e = (Q.abs() @ K.abs().T * d ** -0.5).amax(1) * 2 ** -7
            tol = (U + torch.expm1(2 * e) + 1e-4)[:, None] * (P @ V.abs()) + U * (P @ V).abs()
            assert ((o[rows, h].double() - P @ V).abs() <= tol).all()
            assert ((lse[h, rows].double() - torch.logsumexp(S, 1)).abs() <= e + 1e-4).all()


def test_paged_forward_in_a_graph(g):
    """Page step, write and attention of a forward captured once and replayed for other lengths, on a side stream."""
    Hq, Hkv, d, ps, R, T = 4, 2, 128, 16, 5, 64
    r = torch.Generator(device="cuda").manual_seed(14)
    n_pages, width = 200, 40
    kc, vc = (torch.randn((n_pages, Hkv, ps, d), generator=r, device="cuda").bfloat16() for _ in range(2))
    table = torch.arange(R * width, device="cuda", dtype=torch.int32).view(R, width) % n_pages
    free, n_free = torch.arange(n_pages, device="cuda", dtype=torch.int32), i32([50])
    held, start, end = i32([0] * R), i32([0] * R), i32([0] * R)
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda").bfloat16()

    def forward(q_out, o, lse):
        s = g.op_page_step(held, start, end, table, free, n_free, ps, T)
        rot = g.op_kv_write_paged(qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], s.pos, s.slots, kc, vc, q_out=q_out)
        return s, g.op_attention_paged(rot, kc, vc, table, s.cu_rows, s.kv_len, o=o, lse=lse)
    new = lambda: (torch.zeros((T, Hq, d), device="cuda").bfloat16(), torch.zeros((T, Hq, d), device="cuda").bfloat16(),
                   torch.zeros((Hq, T), device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = new()
    with torch.cuda.stream(side):
        forward(*new())  # warm-up
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            s, _ = forward(*outs)
    for lens in ([(0, 10), (33, 40), (100, 101), (16, 16), (500, 533)], [(5, 6)] * R, [(600, 640), (0, 24), (1, 1), (0, 0), (0, 0)]):
        for t, x in ((held, [a for a, _ in lens]), (start, [a for a, _ in lens]), (end, [b for _, b in lens])):
            t.copy_(i32(x))
        saved = [x.clone() for x in (table, free, kc, vc)]
        for x in outs:
            x.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        got = [x.clone() for x in (*outs, table, free, kc, vc, s.pos, s.slots)]
        for x, y in zip((table, free, kc, vc), saved):
            x.copy_(y)
        eager = new()
        s2, _ = forward(*eager)
        for a, b in zip(got, (*eager, table, free, kc, vc, s2.pos, s2.slots)):
            assert torch.equal(a, b)


def test_paged_graph_with_copies_between(g):
    """Fills, copies and another stream's work before each call of a captured forward: the calls wait for them."""
    Hq, Hkv, d, ps, R, T = 4, 2, 64, 16, 3, 40
    r = torch.Generator(device="cuda").manual_seed(15)
    kc, vc = _empty_cache("head", 60, Hkv, ps, d)
    src = [torch.randn((T, h, d), generator=r, device="cuda").bfloat16() for h in (Hq, Hkv, Hkv)]
    q, k, v = (torch.zeros_like(x) for x in src)
    lens = [i32([0, 100, 7]), i32([0, 100, 7]), i32([9, 120, 8])]
    held, start, end = (torch.zeros_like(x) for x in lens)
    table, free = torch.arange(60, dtype=torch.int32, device="cuda").view(R, 20), torch.arange(60, dtype=torch.int32, device="cuda")
    n_free = i32([9])
    rot, o, lse = torch.zeros_like(q), torch.zeros_like(q), torch.zeros((Hq, T), device="cuda")
    side = torch.cuda.Stream()

    def forward():
        main = torch.cuda.current_stream()
        for a, b in zip((held, start, end), lens):
            a.copy_(b)
        s = g.op_page_step(held, start, end, table, free, n_free, ps, T)
        q.zero_()
        side.wait_stream(main)
        with torch.cuda.stream(side):
            k.copy_(src[1])
            v.copy_(src[2])
        main.wait_stream(side)
        q.copy_(src[0])
        g.op_kv_write_paged(q, k, v, s.pos, s.slots, kc, vc, q_out=rot)
        o.zero_()
        g.op_attention_paged(rot, kc, vc, table, s.cu_rows, s.kv_len, o=o, lse=lse)
        q.zero_()
        k.zero_()
    saved = table.clone(), free.clone()
    forward()
    torch.cuda.synchronize()
    want = [x.clone() for x in (rot, o, lse, kc, vc, table, free)]
    capture = torch.cuda.Stream()
    capture.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(capture):
        table.copy_(saved[0])
        free.copy_(saved[1])
        with torch.cuda.graph(graph, stream=capture):
            forward()
    for _ in range(3):
        torch.cuda.synchronize()
        for x in (rot, o, lse, kc, vc):
            x.zero_()
        table.copy_(saved[0])
        free.copy_(saved[1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((rot, o, lse, kc, vc, table, free), want):
            assert torch.equal(a, b)


def test_paged_offsets_past_32_bits(g):
    """A cache of more than 2^32 elements: pages at both of its ends, and slots of more than 2^22 positions."""
    Hq, Hkv, d, ps, n_pages = 8, 8, 128, 256, 16500
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB of device memory")
    kc, vc = (torch.empty((n_pages, ps, Hkv, d), dtype=torch.bfloat16, device="cuda").transpose(1, 2) for _ in range(2))
    assert kc.numel() > 1 << 32
    T = 600
    pages = [n_pages - 1, 0, n_pages - 2]
    table = i32([pages])
    r = torch.Generator(device="cuda").manual_seed(16)
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda").bfloat16()
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda")
    slots = (table[0].long()[pos.long() // ps] * ps + pos % ps).to(torch.int32)
    rot = g.op_kv_write_paged(q, k, v, pos, slots, kc, vc)
    K = torch.cat([kc[p].transpose(0, 1) for p in pages])[:T]
    assert torch.equal(torch.cat([vc[p].transpose(0, 1) for p in pages])[:T], v)
    val, tol = _rotated(k, pos, 10000.0)
    assert ((K.double() - val).abs() <= tol).all()
    c = dict(q=rot, kc=kc, vc=vc, table=table, cu=i32([0, T]), kv_len=i32([T]), K=[K], V=[v], rows=[T])
    _check(g, c, g.FWD_VERIFY, *_attend(g, c, g.FWD_VERIFY))


def test_attention_paged_most_requests(g):
    """4,096 requests, single tokens over one to five pages."""
    R = 4096
    rng = random.Random(17)
    kv = [rng.randint(1, 70) for _ in range(R)]
    c = _case([1] * R, kv, 2, 1, 64, 16, "head", seed=17)
    o, lse = _attend(g, c, g.FWD_VERIFY)
    K, V = (torch.zeros((R, 70, 64), dtype=torch.float64, device="cuda") for _ in range(2))
    for r in range(R):
        K[r, :kv[r]], V[r, :kv[r]] = c["K"][r][:, 0].double(), c["V"][r][:, 0].double()
    S = torch.einsum("rhd,rkd->rhk", c["q"].double(), K) * 64 ** -0.5
    S.masked_fill_(torch.arange(70, device="cuda")[None, None, :] >= i32(kv)[:, None, None], -math.inf)
    P = torch.softmax(S, -1)
    O = torch.einsum("rhk,rkd->rhd", P, V)
    # exponentials to 2^-16: scores of at most some tens, sums 70 long
    tol = (U + 2.0 ** -16) * torch.einsum("rhk,rkd->rhd", P, V.abs()) + U * O.abs()
    assert ((o.double() - O).abs() <= tol).all()
    assert ((lse.T.double() - torch.logsumexp(S, -1)).abs() <= 2.0 ** -16).all()


def test_page_step_most_rows(g):
    """2^24 rows of 4,096 requests, and the same with a row too few."""
    R, n, ps, width = 4096, 4096, 256, 17
    n_pages = R * (n // ps)
    order = torch.randperm(n_pages, generator=torch.Generator(device="cuda").manual_seed(18), device="cuda").to(torch.int32)
    for T in (1 << 24, (1 << 24) - 1):
        table = torch.full((R, width), -1, dtype=torch.int32, device="cuda")
        zero = torch.zeros((R,), dtype=torch.int32, device="cuda")
        s = g.op_page_step(zero, zero, zero + n, table, order.clone(), i32([n_pages]), ps, T)
        ok = R if T == 1 << 24 else R - 1  # requests whose rows fit
        want = order.flip(0)[:ok * (n // ps)].view(ok, n // ps)
        assert torch.equal(table[:ok, :n // ps], want) and (table[ok:] == -1).all() and int(s.n_free) == n_pages - want.numel()
        rows = ok * n
        pos = torch.arange(n, dtype=torch.int32, device="cuda")
        assert torch.equal(s.pos[:rows].view(ok, n), pos.expand(ok, n)) and (s.pos[rows:] == -1).all()
        assert torch.equal(s.slots[:rows].view(ok, n), want.repeat_interleave(ps, 1) * ps + pos % ps) and (s.slots[rows:] == -1).all()
        assert torch.equal(s.kv_len, torch.where(torch.arange(R, device="cuda") < ok, n, 0).to(torch.int32))


def test_attention_paged_most_keys(g):
    """One token over 2^24 keys: the longest table, a request on all of the device."""
    n, ps, d = 1 << 24, 256, 64
    r = torch.Generator(device="cuda").manual_seed(19)
    kc, vc = (torch.randn((n // ps, 1, ps, d), generator=r, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    table = torch.randperm(n // ps, generator=r, device="cuda").to(torch.int32)[None]
    q = torch.randn((1, 2, d), generator=r, device="cuda").bfloat16()
    o, lse = g.op_attention_paged(q, kc, vc, table, i32([0, 1]), i32([n]))
    S = torch.cat([torch.einsum("hd,nd->hn", q[0].double(), kc[p:p + 4096, 0].reshape(-1, d).double()) * d ** -0.5
                   for p in range(0, n // ps, 4096)], 1)  # (the order of the keys does not matter)
    ref = torch.logsumexp(S, 1)
    P = torch.exp(S - ref[:, None])
    V = [vc[p:p + 4096, 0].reshape(-1, d).double() for p in range(0, n // ps, 4096)]
    parts = P.split(4096 * ps, 1)
    O, bound = sum(p @ v for p, v in zip(parts, V)), sum(p @ v.abs() for p, v in zip(parts, V))
    # a piece's keys are summed 16 at a time in each of two chains, the pieces one after the other; exponentials to 2^-17
    deep = (n / 152 / 32 + 152 + 64) * TC + 2.0 ** -17
    assert ((o[0].double() - O).abs() <= (U + deep) * bound + U * O.abs()).all()
    assert ((lse[:, 0].double() - ref).abs() <= deep + 4 * F32 * ref.abs()).all()


def test_paged_most_rows(g):
    """2^20 rows of 4,096 whole prompts of 256: written and attended."""
    R, n, Hq, Hkv, d, ps = 4096, 256, 2, 1, 64, 64
    T = R * n
    r = torch.Generator(device="cuda").manual_seed(20)
    qkv = torch.randn((T, Hq + 2 * Hkv, d), generator=r, device="cuda", dtype=torch.bfloat16)
    q, k, v = qkv[:, :Hq], qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:]
    kc, vc = (torch.zeros((T // ps, Hkv, ps, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    slots = torch.arange(T, dtype=torch.int32, device="cuda").flip(0).view(R, n).flip(1).reshape(-1).contiguous()
    table = (slots.view(R, n // ps, ps)[:, :, 0] // ps).contiguous()
    rot = g.op_kv_write_paged(q, k, v, (torch.arange(T, device="cuda") % n).to(torch.int32), slots, kc, vc)
    cu = (torch.arange(R + 1, device="cuda") * n).to(torch.int32)
    o, lse = g.op_attention_paged(rot, kc, vc, table, cu, i32([n] * R))
    seen = torch.tril(torch.ones((n, n), dtype=torch.bool, device="cuda"))
    for a in range(0, R, 512):
        K, V = (c[table[a:a + 512].long()].reshape(512, n, d).double() for c in (kc, vc))
        Q = rot[a * n:(a + 512) * n].view(512, n, Hq, d).double()
        for h in range(Hq):
            S = (Q[:, :, h] @ K.transpose(1, 2) * d ** -0.5).masked_fill(~seen, -math.inf)
            P = torch.softmax(S, -1)
            O = P @ V
            tol = (U + 2.0 ** -16) * (P @ V.abs()) + U * O.abs()
            assert ((o[a * n:(a + 512) * n, h].view(512, n, d).double() - O).abs() <= tol).all()
            assert ((lse[h, a * n:(a + 512) * n].view(512, n).double() - torch.logsumexp(S, -1)).abs() <= 2.0 ** -16).all()


def test_attention_paged_graphs_that_share_a_workspace(g):
    """Two captured calls of different shapes with one workspace, replayed in turn."""
    cs = [_case([33] * 4, [700, 1500, 90, 4000], 12, 4, 128, 16, "head", seed=22), _case([1] * 9, [2000] * 9, 12, 4, 128, 16, "token", seed=23)]
    want = [_attend(g, c, g.FWD_VERIFY) for c in cs]
    ws = torch.empty((max(g.load().gocr_op_attention_paged_workspace(c["q"].shape[0], 12, 4, 128) for c in cs),),
                     dtype=torch.uint8, device="cuda")
    outs, graphs, stream = [], [], torch.cuda.Stream()
    torch.cuda.synchronize()
    for c in cs:
        outs.append((torch.zeros(c["q"].shape, dtype=torch.bfloat16, device="cuda"), torch.zeros((12, c["q"].shape[0]), device="cuda")))
        graphs.append(torch.cuda.CUDAGraph())
        torch.cuda.synchronize()
        with torch.cuda.graph(graphs[-1], stream=stream):
            _attend(g, c, g.FWD_VERIFY, workspace=ws, o=outs[-1][0], lse=outs[-1][1])
    for _ in range(4):
        for x in outs:
            x[0].zero_()
        for gr in graphs + graphs[::-1]:
            gr.replay()
        torch.cuda.synchronize()
        for w, x in zip(want, outs):
            assert torch.equal(w[0], x[0]) and torch.equal(w[1], x[1])


def test_paged_calls_on_two_streams(g):
    """Two programs at once, each with its own cache and workspace."""
    cs = [_case([33] * 6, [1031, 2049, 33, 512, 700, 1500], 12, 4, 128, 16, "head", seed=s) for s in (20, 21)]
    want = [_attend(g, c, g.FWD_VERIFY) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(5):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(_attend(g, cs[i], g.FWD_VERIFY))
    torch.cuda.synchronize()
    for w, all_ in zip(want, got):
        assert all(torch.equal(w[0], o) and torch.equal(w[1], l) for o, l in all_)
