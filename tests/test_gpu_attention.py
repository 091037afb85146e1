"""GPU parity of mxfp4_attention against a 64-bit softmax over the cache's values (bounds derived in cache_ref)."""
from __future__ import annotations

import ctypes

import numpy as np
import pytest
import torch

import cache_ref as ref
from gpu_util import DEV, say
from test_gpu_cache import angles, new_cache, rows

pytestmark = pytest.mark.gpu


class Case:
    """Packed queries of sequences with (queries, cached tokens), and a cache whose other bytes are garbage."""

    def __init__(self, lens, heads, kv, dim, page, seed, extra=0, wide=0, garbage=0xFF, qsize=2.0, first=0):
        r = np.random.default_rng(seed)
        self.lens, self.heads, self.kv, self.dim, self.page = lens, heads, kv, dim, page
        need = [-(-l // page) for _, l in lens]
        pages = sum(need) + 3
        width = max([1, *need]) + wide
        order = r.permutation(pages)
        # everything that no sequence holds: scale bytes `garbage` (255: NaN) and any code
        codes = [np.full((pages, kv, page, dim // 2), 0x77, np.uint8) for _ in range(2)]
        scales = [np.full((pages, kv, page, dim // 32), garbage, np.uint8) for _ in range(2)]
        self.table = np.full((len(lens), width), -7, np.int32)
        at = 0
        for s, (_, l) in enumerate(lens):
            mine = order[at:at + need[s]]
            self.table[s, :need[s]] = mine
            at += need[s]
            x = r.standard_normal((2, l, kv, dim)) * np.exp2(r.integers(-2, 2, (2, l, kv, 1)))
            x[:, :, :, 3] *= 5
            for i in range(2):
                c, e = ref.encode(x[i])
                j = np.arange(l)
                codes[i][mine[j // page], :, j % page] = c
                scales[i][mine[j // page], :, j % page] = e
        self.host = [codes[0], scales[0], codes[1], scales[1]]
        self.offsets = np.concatenate([[0], np.cumsum([n for n, _ in lens])]).astype(np.int32) + first
        self.tokens = int(self.offsets[-1]) + extra
        q = qsize * r.standard_normal((self.tokens, heads, dim))
        self.q = torch.from_numpy(q.astype(np.float32)).bfloat16()
        self.kv_lens = np.array([l for _, l in lens], np.int32)

    def rows_of(self, s):
        """Keys and values of sequence s in 64 bits, [l, kv, dim]."""
        l = self.lens[s][1]
        j = np.arange(l)
        pages = self.table[s, j // self.page]
        return [ref.decode(self.host[i][pages, :, j % self.page], self.host[i + 1][pages, :, j % self.page]) for i in (0, 2)]

    def device(self):
        on = lambda a: torch.from_numpy(a).to(DEV)   # noqa: E731
        return dict(q=self.q.to(DEV), cache=tuple(on(a) for a in self.host), page_table=on(self.table),
                    kv_lens=on(self.kv_lens), q_offsets=on(self.offsets))

    def check(self, out, scale, causal=True, window=0, sinks=None, only=None):
        got = out.float().cpu().numpy().astype(np.float64)
        for s, (n, _) in enumerate(self.lens):
            if n == 0 or (only is not None and s not in only):
                continue
            a = self.offsets[s]
            k, v = self.rows_of(s)
            want, bound = ref.attention(self.q[a:a + n].double().numpy(), k, v, scale, causal, window, sinks)
            g = got[a:a + n]
            assert np.array_equal(np.isnan(g), np.isnan(want)), s
            fine = ~np.isnan(want)
            off = np.abs(g - want)[fine] - bound[fine]
            assert off.size == 0 or off.max() <= 0, (s, off.max(), np.abs(want[fine]).max())


def run(gpu, case, causal=True, window=0, sinks=None, scale=None, **more):
    scale = case.dim ** -0.5 if scale is None else scale
    d = case.device()
    s = None if sinks is None else torch.from_numpy(sinks).to(DEV)
    out = gpu.mxfp4_attention(**d, scale=scale, causal=causal, window=window, sinks=s, **more)
    torch.cuda.synchronize()
    case.check(out, scale, causal, window, sinks)
    return out


LENS = {
    "one": [(1, 1)],
    "small": [(1, n) for n in (1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257)],
    "decode": [(1, n) for n in (777, 1, 300, 0, 1500, 64)],
    "long": [(1, 9001), (1, 4100)],
    "draft": [(4, 500), (1, 3), (0, 50), (7, 7), (3, 1000), (2, 129)],
    "empty": [(3, 0), (5, 2), (0, 0), (4, 4), (1, 0)],
    "chunk": [(70, 700), (33, 40), (129, 129)],
    "prompts": [(300, 300), (1, 1), (64, 64), (0, 0), (65, 65), (515, 515)],
}


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("heads,kv,dim,page", [(4, 4, 128, 16), (8, 2, 64, 16), (32, 8, 128, 64), (6, 2, 128, 32), (5, 1, 64, 128),
                                                (16, 1, 128, 16), (40, 2, 64, 64)])
def test_causal(gpu, lens, heads, kv, dim, page):
    say(f"attention: {lens}, {heads} / {kv} heads of {dim}, page {page}")
    run(gpu, Case(LENS[lens], heads, kv, dim, page, len(lens) + heads))


@pytest.mark.parametrize("lens", list(LENS))
@pytest.mark.parametrize("window", [1, 16, 100, 5000])
def test_windows_and_sinks(gpu, lens, window):
    say(f"attention: {lens}, window {window}, sinks")
    r = np.random.default_rng(window)
    sinks = (3 * r.standard_normal(16)).astype(np.float32)
    run(gpu, Case(LENS[lens], 16, 2, 64, 16, window), window=window, sinks=sinks)
    run(gpu, Case(LENS[lens], 8, 2, 128, 64, window), window=window)


@pytest.mark.parametrize("lens", list(LENS))
def test_without_a_mask(gpu, lens):
    say(f"attention: {lens}, no mask")
    r = np.random.default_rng(3)
    run(gpu, Case(LENS[lens], 8, 2, 128, 16, 1), causal=False)
    run(gpu, Case(LENS[lens], 16, 2, 64, 32, 2), causal=False, sinks=r.standard_normal(16).astype(np.float32))


def ragged(seed, seqs, most, queries):
    r = np.random.default_rng(seed)
    return [(int(r.integers(0, queries + 1)) if i else queries, int(r.integers(1, most + 1))) for i in range(seqs)]


# (form, heads, kv heads, head dim, page, sequences, table's extra pages)
FORMS = [
    (10, 32, 8, 128, 16, ragged(1, 40, 300, 1), 0), (10, 16, 8, 64, 64, ragged(2, 40, 300, 2), 0),
    (10, 8, 2, 128, 16, [(150, 150), (70, 70), (380, 380)], 0), (10, 16, 4, 64, 64, [(260, 260), (90, 200), (170, 170)], 0),
    (20, 32, 8, 128, 64, [(1500, 1500), (600, 700), (1, 900), (0, 8)], 0), (30, 64, 16, 64, 64, [(900, 900), (640, 700)], 0),
    (118, 8, 2, 128, 16, ragged(3, 30, 1900, 1), 0), (118, 8, 2, 64, 16, ragged(4, 60, 1500, 4), 0),
    (118, 16, 2, 128, 32, ragged(10, 16, 1800, 4), 0),
    (114, 8, 2, 128, 16, ragged(5, 20, 900, 1), 0), (114, 16, 4, 64, 64, ragged(6, 30, 700, 8), 0),
    (114, 32, 8, 64, 16, ragged(7, 50, 1200, 1), 0),
    (111, 32, 8, 128, 16, ragged(8, 200, 90, 1), 0), (111, 16, 8, 64, 16, ragged(9, 90, 600, 3), 0),
    (211, 16, 8, 128, 16, ragged(11, 160, 1300, 1), 0), (211, 16, 8, 64, 64, ragged(12, 80, 1100, 2), 0),
    (1211, 16, 8, 128, 16, ragged(13, 600, 150, 1), 60), (1211, 32, 8, 64, 16, ragged(14, 600, 100, 1), 60),
    (2214, 8, 2, 128, 64, ragged(15, 3, 5000, 2), 0), (2214, 8, 2, 64, 16, ragged(16, 4, 3000, 4), 0),
    (214, 8, 4, 128, 16, ragged(17, 40, 9000, 1), 0), (214, 8, 4, 64, 64, [(2, 9000)] * 20, 0),
    (224, 16, 4, 128, 16, ragged(18, 20, 9000, 8), 0), (224, 16, 4, 64, 64, ragged(19, 24, 9000, 8), 0),
    (2224, 16, 2, 128, 16, [(30, 32000), (5, 2000)], 0), (2224, 16, 2, 64, 16, [(14, 40000), (0, 9), (12, 2100)], 0),
    (1224, 32, 8, 128, 64, [(600, 900), (99, 4000)], 0), (1224, 64, 8, 64, 64, [(300, 2500)], 0),
]


@pytest.mark.parametrize("form,heads,kv,dim,page,lens,wide", FORMS, ids=lambda v: str(v) if isinstance(v, int) else None)
def test_every_form(gpu, form, heads, kv, dim, page, lens, wide):
    """Each form that a call can take, on ragged sequences, with a mask and without, a window, sinks and a missing page."""
    say(f"attention: form {form}, {heads} / {kv} heads of {dim}, {len(lens)} sequences")
    case = Case(lens, heads, kv, dim, page, form + dim, wide=wide)
    width = case.table.shape[1] * page
    choose = gpu.load_library().e2m1_mxfp4_attention_form
    choose.argtypes = [ctypes.c_int64] * 6
    assert choose(case.tokens, len(lens), heads, kv, dim, width) == form
    r = np.random.default_rng(form)
    sinks = (2 * r.standard_normal(heads)).astype(np.float32)
    run(gpu, case)
    run(gpu, case, causal=False, sinks=sinks)
    run(gpu, case, window=2**30, sinks=sinks)      # as wide as it likes: the same form
    run(gpu, case, window=77)
    d = case.device()
    s = max((i for i in range(len(lens)) if lens[i][0]), key=lambda i: lens[i][1])
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    size = gpu.mxfp4_attention_workspace_size(case.tokens, len(lens), heads, kv, dim)
    memory = torch.full((size + 4096,), 0xA5, dtype=torch.uint8, device=DEV)
    clean = gpu.mxfp4_attention(**d, workspace=memory[:size])
    assert (memory[size:] == 0xA5).all()
    assert torch.equal(clean, gpu.mxfp4_attention(**d))
    d["page_table"][s, 0] = 2**30
    out = gpu.mxfp4_attention(**d, err_flag=flag)
    assert flag.item() == 1
    a, b = case.offsets[s], case.offsets[s + 1]
    assert torch.equal(out[:a], clean[:a]) and torch.equal(out[b:], clean[b:])
    n, length = lens[s]
    k, v = case.rows_of(s)
    pos = length - n
    for i in sorted({0, n - 1}):     # without the first page's tokens
        if n and pos + i >= page:
            want, bound = ref.attention(case.q[a + i:a + i + 1].double().numpy(), k[page:pos + i + 1], v[page:pos + i + 1],
                                        dim ** -0.5, True, 0)
            assert (np.abs(out[a + i:a + i + 1].double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 7, 8, 12, 16, 17, 32, 33, 64])
def test_groups(gpu, group):
    say(f"attention: group {group}")
    run(gpu, Case([(1, 200), (2, 77), (3, 130)], 2 * group, 2, 128, 16, group))
    run(gpu, Case([(40, 200), (1, 77)], group, 1, 64, 32, group))


@pytest.mark.parametrize("scale,size", [(0.0, 2.0), (1.0, 3.0), (0.3, 30.0), (1e-3, 1000.0), (1e30, 1e-30)])
def test_scales(gpu, scale, size):
    """All keys alike, one key with nearly all of the weight, and sizes that cancel."""
    say(f"attention: scale {scale}, queries of {size}")
    run(gpu, Case([(1, 300), (20, 300), (90, 400)], 4, 2, 128, 16, 4, qsize=size), scale=scale)


@pytest.mark.parametrize("dim", [64, 128])
def test_scores_of_single_channels(gpu, dim):
    """Keys with one channel each against queries of many sizes: here the bound of a score has a single term, far below what
    a missing or misplaced part of a query would be off."""
    say(f"attention: single channels of {dim}")
    case = Case([(3, 2)] * dim, 2, 1, dim, 16, 26)
    r = np.random.default_rng(27)
    q = np.sign(r.standard_normal((case.tokens, 2, dim))) * np.exp2(r.uniform(-8, 0, (case.tokens, 2, dim)))
    case.q = torch.from_numpy(q.astype(np.float32)).bfloat16()
    for s in range(dim):
        page = case.table[s, 0]
        for i in (0, 2):
            x = np.zeros((2, 1, dim))
            x[0, 0, s] = 64.0 if i == 0 else 1.0
            x[1, 0, s] = 0.0 if i == 0 else -1.0
            case.host[i][page, :, :2], case.host[i + 1][page, :, :2] = (t.transpose(1, 0, 2) for t in ref.encode(x))
    run(gpu, case, causal=False, scale=0.5)


def test_sinks_at_the_ends(gpu):
    say("attention: sinks of all sizes")
    sinks = np.array([-np.inf, -1e4, 0, 80, 1e4, -3e38], np.float32)
    case = Case([(1, 100), (3, 0), (20, 50)], 6, 1, 64, 16, 5)
    out = run(gpu, case, sinks=sinks)
    assert not out[:, 4].any()      # nothing is left beside a sink that large


def test_infinite_sinks(gpu):
    """Nothing is left beside an infinite sink; a query that is not finite stays NaN."""
    say("attention: infinite sinks")
    for lens in ([(1, 100), (3, 0), (20, 50)], [(1, 5000)], [(300, 300)]):
        case = Case(lens, 4, 2, 64, 16, 6)
        d = case.device()
        d["q"][0, 1] = float("nan")
        d["q"][0, 3] = float("nan")
        sinks = torch.tensor([0, float("inf"), float("inf"), 0], device=DEV)
        out = gpu.mxfp4_attention(**d, sinks=sinks)
        assert not out[1:, 1:3].any() and not out[0, 2].any() and out[0, [1, 3]].isnan().all()
        assert not out[0, 0].isnan().any() and out[0, 0].any()


@pytest.mark.parametrize("garbage", [255, 254, 252, 0])
def test_what_is_not_seen_changes_nothing(gpu, garbage):
    """Whatever lies in unused places and in tokens that a query does not see."""
    say(f"attention: scale bytes {garbage} in unused places")
    lens = [(1, 17), (5, 70), (40, 130), (1, 333)]
    run(gpu, Case(lens, 8, 2, 128, 64, 6, wide=3, garbage=garbage))
    run(gpu, Case(lens, 8, 2, 64, 16, 6, wide=3, garbage=garbage), window=9)


@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("n", [1, 6, 90])
@pytest.mark.parametrize("zeros", [False, True])
def test_blocks_that_are_nan(gpu, dim, n, zeros):
    """Scale byte 255 in a key makes NaN of the rows and heads that see it, in a value of its block's channels there, and of
    nothing else."""
    say(f"attention: NaN blocks, {n} queries, heads of {dim}")
    case = Case([(n, 200), (n, 150)], 4, 2, dim, 16, 7)
    for j, what, head in ((197, 1, 0), (199, 3, 1), (150, 3, 0), (60, 1, 1)):
        at = case.table[0, j // 16], head, j % 16
        case.host[what][at][dim // 32 - 1] = 255
        if zeros:       # as the writer leaves them
            case.host[what - 1][at][dim // 2 - 16:] = 0
    run(gpu, case)
    run(gpu, case, window=3)
    run(gpu, case, causal=False)


def test_queries_that_are_not_finite(gpu):
    """Only their own rows show it."""
    say("attention: NaN and infinite queries")
    case = Case([(3, 40), (40, 90)], 4, 2, 64, 16, 8)
    d = case.device()
    clean = gpu.mxfp4_attention(**d)
    for t, h, x in ((1, 2, float("nan")), (7, 0, float("inf")), (30, 3, -float("inf"))):
        d["q"][t, h, 40] = x
    out = gpu.mxfp4_attention(**d)
    for t, h in ((1, 2), (7, 0), (30, 3)):
        assert torch.isnan(out[t, h]).all()
        out[t, h] = clean[t, h]
    assert torch.equal(out, clean)


def test_large_and_small_values(gpu):
    """Keys and values with scales at the ends of the range; denormal queries."""
    say("attention: values at the ends")
    for byte_k, byte_v, size, scale in ((20, 240, 1.0, 1.0), (220, 30, 1e-30, 1.0), (127, 5, 1e-39, 1e30)):
        case = Case([(1, 70), (35, 70)], 4, 2, 128, 16, 9, qsize=size)
        case.host[1][...] = np.where(case.host[1] == 255, 255, byte_k)
        case.host[3][...] = np.where(case.host[3] == 255, 255, byte_v)
        run(gpu, case, scale=scale)


def test_pages_that_are_not_there(gpu):
    """Tokens on pages outside the cache are not seen and set the flag; so do lengths past the table."""
    say("attention: pages outside")
    case = Case([(1, 70), (3, 70), (40, 100), (1, 40)], 8, 2, 128, 16, 10)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    run(gpu, case, err_flag=flag)
    assert flag.item() == 0
    d = case.device()
    clean = gpu.mxfp4_attention(**d)
    d["page_table"][0, 1] = 10**6
    d["page_table"][2, 0] = -1
    d["page_table"][3] = 2**31 - 1
    out = gpu.mxfp4_attention(**d, err_flag=flag)
    assert flag.item() == 1
    assert torch.equal(out[1:4], clean[1:4]) and not out[44].any()
    # without the missing page's tokens
    got = out.float().cpu().numpy()
    k, v = case.rows_of(0)
    keep = np.r_[0:16, 32:70]
    want, bound = ref.attention(case.q[:1].double().numpy(), k[keep], v[keep], 128 ** -0.5, True, 0)
    assert (np.abs(got[:1] - want) <= bound).all()
    k, v = case.rows_of(2)
    for i in (0, 10, 39):     # query i at 60 + i, the first 16 tokens gone
        want, bound = ref.attention(case.q[4 + i:5 + i].double().numpy(), k[16:61 + i], v[16:61 + i], 128 ** -0.5, True, 0)
        assert (np.abs(got[4 + i:5 + i] - want) <= bound).all()
    # a length past the table counts as the table's end; a negative one as none
    flag.zero_()
    d = case.device()
    d["kv_lens"][0] = 2**31 - 1
    d["kv_lens"][3] = -5
    table = d["page_table"]
    table[0] = torch.arange(7, device=DEV)      # all of its pages are there
    out = gpu.mxfp4_attention(**d, err_flag=flag)
    assert flag.item() == 1 and not out[44].any() and torch.equal(out[1:44], clean[1:44])
    flag.zero_()
    d["kv_lens"][0] = 70
    gpu.mxfp4_attention(**d, err_flag=flag)
    assert flag.item() == 0


def test_no_pages_at_all(gpu):
    say("attention: an empty cache and an empty table")
    case = Case([(2, 0), (1, 0)], 4, 2, 64, 16, 11)
    d = case.device()
    d["cache"] = tuple(t[:0] for t in d["cache"])
    assert not gpu.mxfp4_attention(**d).any()
    d["page_table"] = d["page_table"][:, :0].contiguous()
    assert not gpu.mxfp4_attention(**d).any()
    d["kv_lens"] += 5
    assert not gpu.mxfp4_attention(**d).any()
    none = gpu.mxfp4_attention(d["q"][:0], d["cache"], d["page_table"][:0], d["kv_lens"][:0], d["q_offsets"][:1])
    assert none.shape == (0, 4, 64)


@pytest.mark.parametrize("lens", [[(1, 50), (3, 70)], [(90, 90), (0, 3), (40, 100)]])
def test_rows_outside_the_sequences(gpu, lens):
    """Rows before the first offset and behind the last one stay as they were."""
    say(f"attention: rows outside, {lens}")
    case = Case(lens, 4, 2, 128, 16, 12, extra=37, first=5)
    d = case.device()
    out = torch.full_like(d["q"], 7.0)
    gpu.mxfp4_attention(**d, out=out)
    case.check(out, 128 ** -0.5)
    assert (out[:5] == 7).all() and (out[case.offsets[-1]:] == 7).all()
    bad = d["q_offsets"].clone()
    bad[-1] = 2**31 - 1        # past the rows: as far as they go
    bad[0] = -2**31
    gpu.mxfp4_attention(**{**d, "q_offsets": bad}, out=out)
    assert not (out == 7).all(-1).any()


@pytest.mark.parametrize("n", [1, 90])
@pytest.mark.parametrize("seqs", [3, 200])
def test_offsets_that_descend(gpu, n, seqs):
    """Nothing is written and the flag is set, also where rows would belong to many sequences."""
    say(f"attention: descending offsets, {seqs} sequences of {n}")
    case = Case([(n, 100)] * seqs, 4, 2, 64, 16, 25)
    d = case.device()
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    for change in ((1, 0, 10**6), (seqs - 1, seqs, -3), (0, seqs + 1, None)):
        off = d["q_offsets"].clone()
        if change[2] is None:
            off[0::2] = 0
            off[1::2] = case.tokens
        else:
            off[change[0]:change[1] + 1] = change[2]
            off[1] = case.tokens
        out = torch.full_like(d["q"], 7.0)
        flag.zero_()
        gpu.mxfp4_attention(**{**d, "q_offsets": off}, out=out, err_flag=flag)
        descends = bool((off[1:] < off[:-1]).any())
        assert descends and flag.item() == 1 and (out == 7).all()
    out = gpu.mxfp4_attention(**d)
    case.check(out, 64 ** -0.5)


def test_strided_queries(gpu):
    say("attention: queries inside a fused row")
    case = Case([(1, 90), (4, 44), (70, 100)], 4, 2, 128, 16, 13)
    d = case.device()
    want = gpu.mxfp4_attention(**d)
    wide = torch.randn(case.tokens, 8 * 128, device=DEV).bfloat16()
    wide[:, 128:640] = d["q"].view(case.tokens, -1)
    d["q"] = wide[:, 128:640].view(case.tokens, 4, 128)
    assert not d["q"].is_contiguous()
    assert torch.equal(gpu.mxfp4_attention(**d), want)
    d["q"] = d["q"].transpose(0, 1).contiguous().transpose(0, 1)
    with pytest.raises(ValueError):
        gpu.mxfp4_attention(**d)


@pytest.mark.parametrize("lens", ["decode", "draft", "chunk", "prompts", "long"])
def test_the_same_bits(gpu, lens):
    """Twice the same call, another stream, a workspace full of NaN, and a sequence in another batch."""
    say(f"attention: the same bits, {lens}")
    case = Case(LENS[lens], 8, 2, 128, 16, 14)
    d = case.device()
    want = gpu.mxfp4_attention(**d)
    size = gpu.mxfp4_attention_workspace_size(case.tokens, len(case.lens), 8, 2, 128)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    assert torch.equal(gpu.mxfp4_attention(**d, workspace=ws), want)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        out = gpu.mxfp4_attention(**d, stream=stream)
        torch.cuda.synchronize()
        assert torch.equal(out, want)


def test_two_calls_at_once(gpu):
    """Calls on two streams with workspaces of their own, and outputs and workspaces that the calls allocate."""
    say("attention: two streams at once")
    cases = [Case(LENS["long"], 8, 2, 128, 16, 28), Case(ragged(29, 40, 900, 2), 16, 8, 64, 16, 29)]
    devs = [c.device() for c in cases]
    want = [gpu.mxfp4_attention(**d) for d in devs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(4):
        got = [gpu.mxfp4_attention(**d, stream=s) for _ in range(3) for d, s in zip(devs, streams)]
        torch.cuda.synchronize()
        for i, g in enumerate(got):
            assert torch.equal(g, want[i % 2])


def test_graphs_that_share_a_workspace(gpu):
    """Two captured calls with one workspace, replayed in turn with eager calls between."""
    say("attention: graphs")
    cases = [Case(LENS["draft"], 8, 2, 128, 16, 15), Case(LENS["chunk"], 8, 2, 128, 16, 16), Case(LENS["long"], 8, 2, 128, 16, 17)]
    devs = [c.device() for c in cases]
    want = [gpu.mxfp4_attention(**d) for d in devs]
    size = max(gpu.mxfp4_attention_workspace_size(c.tokens, len(c.lens), 8, 2, 128) for c in cases)
    ws = torch.full((size,), 0xFF, dtype=torch.uint8, device=DEV)
    outs = [torch.empty_like(w) for w in want]
    torch.cuda.synchronize()
    graphs = []
    for d, o in zip(devs, outs):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            gpu.mxfp4_attention(**d, out=o, workspace=ws)
        graphs.append(g)
    for rep in range(4):
        for o in outs:
            o.fill_(float("nan"))
        torch.cuda.synchronize()
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert torch.equal(o, w), rep
        gpu.mxfp4_attention(**devs[rep % 3], out=torch.empty_like(want[rep % 3]), workspace=ws)
    # lengths are read at each replay, as a decoding loop needs them
    devs[0]["kv_lens"] -= 1
    graphs[0].replay()
    torch.cuda.synchronize()
    assert torch.equal(outs[0], gpu.mxfp4_attention(**devs[0])) and not torch.equal(outs[0], want[0])


def test_many_sequences(gpu):
    """More sequences than one step of the kernels' search takes, most of them empty."""
    say("attention: 1500 sequences")
    r = np.random.default_rng(18)
    lens = [(int(r.integers(0, 3)), int(r.integers(0, 40))) for _ in range(1500)]
    run(gpu, Case(lens, 4, 2, 64, 16, 18))
    lens = [(0, 5)] * 700 + [(1, 3)] + [(0, 9)] * 500 + [(2, 700)]
    run(gpu, Case(lens, 4, 2, 128, 16, 19))


@pytest.mark.slow
def test_long_context(gpu):
    """One sequence of 70000 tokens: four queries at its end, then a chunk of 300."""
    say("attention: 70000 tokens")
    run(gpu, Case([(4, 70001)], 8, 2, 128, 64, 20))
    run(gpu, Case([(300, 30011)], 4, 1, 128, 64, 21))
    run(gpu, Case([(1, 66000), (1, 5), (1, 20000)], 4, 1, 64, 16, 22), window=33333)


@pytest.mark.slow
def test_cache_past_32_bits(gpu):
    """A sequence on the last pages of a cache of more than 2^32 code bytes, and on pages across 2^31."""
    say("attention: cache past 32 bits")
    case = Case([(1, 300), (40, 200)], 8, 8, 128, 64, 23)
    per = 8 * 64 * 64
    pages = (1 << 32) // per + 16
    d = case.device()
    want = gpu.mxfp4_attention(**d)
    small = d["cache"][0].shape[0]
    for at in (pages - small, (1 << 31) // per - 2):
        big = tuple(torch.empty(pages, *t.shape[1:], dtype=torch.uint8, device=DEV) for t in d["cache"])
        for b, t in zip(big, d["cache"]):
            b[at:at + small] = t
        table = torch.where(d["page_table"] >= 0, d["page_table"] + at, d["page_table"])
        assert torch.equal(gpu.mxfp4_attention(**{**d, "cache": big, "page_table": table.contiguous()}), want)
        del big


def test_a_layer_of_a_decoder(gpu):
    """A prompt in two chunks, then single tokens, as a serving loop runs them: fused rows in, normed, rotated, cached,
    attended; each step's output against the softmax over what the cache holds, and against one whole prompt."""
    say("attention layer: prompt, chunk, decode")
    r = np.random.default_rng(24)
    heads, kv, dim, page, total = 8, 2, 128, 16, 120
    x = torch.from_numpy(r.standard_normal((total, (heads + 2 * kv) * dim)).astype(np.float32)).bfloat16().to(DEV)
    table = torch.from_numpy(angles(200, dim, 2)).to(DEV)
    w = torch.from_numpy(1 + 0.1 * r.standard_normal(dim)).bfloat16().to(DEV)
    pages = torch.from_numpy(r.permutation(10).astype(np.int32)).to(DEV)[None, :8].contiguous()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device=DEV)   # noqa: E731

    def slots_of(a, b):
        j = torch.arange(a, b, device=DEV)
        return pages[0, j // page].long() * page + j % page

    def step(cache, a, b):
        q = gpu.norm_rope_mxfp4_cache_write(x[a:b], table, torch.arange(a, b, device=DEV), slots_of(a, b), cache, q_weight=w, k_weight=w)
        return q, gpu.mxfp4_attention(q, cache, pages, i32(b), i32(0, b - a))

    cache = new_cache(10, kv, page, dim, 0xFF)
    qs, outs = zip(*[step(cache, a, b) for a, b in ((0, 50), (50, 110), *((i, i + 1) for i in range(110, 120)))])
    k, v = (t.double().cpu().numpy() for t in gpu.mxfp4_cache_read(cache, slots_of(0, total)))
    q, out = torch.cat(qs), torch.cat(outs)
    want, bound = ref.attention(q.double().cpu().numpy(), k, v, dim ** -0.5, True, 0)
    assert (np.abs(out.double().cpu().numpy() - want) <= bound).all()
    whole = new_cache(10, kv, page, dim, 0xFF)
    q2, out2 = step(whole, 0, total)
    assert torch.equal(q, q2) and all(torch.equal(a, b) for a, b in zip(cache, whole))
    assert (np.abs(out2.double().cpu().numpy() - want) <= bound).all()


def wide_head_case(dim, q, key, value):
    """One token's queries q [heads, dim] of one kv head against one cached token."""
    case = Case([(1, 1)], q.shape[0], 1, dim, 16, 30)
    case.q = torch.from_numpy(q.astype(np.float32)).bfloat16()[None]
    at = case.table[0, 0], 0, 0
    for i, x in ((0, key), (2, value)):
        case.host[i][at], case.host[i + 1][at] = ref.encode(x)
    return case


@pytest.mark.parametrize("dim", [64, 128])
def test_what_the_parts_of_a_query_leave(gpu, dim):
    """An element of scale q counts to within 2^-13 of its block's largest magnitude, also where a rounding on the way to a
    part would pass a border between two of its values: elements beside the middles of E2M3 neighbours.

    One token with the value 1 against a sink of the exact score: out = 1 / (1 + exp(sink - s)), so out shows the score's
    error, of scores near 2^13 times it. Counted beside it: the products' sum and the scale's roundings, (dim + 12) fp32 half
    steps of the score, 2 of the sink's way into powers of two, 2 half steps of bf16 for the weight, and out's own."""
    say(f"attention: parts of queries, heads of {dim}")
    r = np.random.default_rng(31)
    heads = 1024
    log2e = np.float64(np.float32(1.44269504088896340736))
    middles = np.arange(4.25, 7.5, 0.5)
    for middle in [*middles, 3.875, 3.9375]:
        for side in (-1, 1):
            first = 1 + r.integers(0, 128) / 128
            target = middle + side * 2.0**-6 * (1 - 2.0**-9)
            scale = np.float64(np.float32(target / 8 / (first * log2e)))
            q = np.zeros((heads, dim))
            c = 2 * r.integers(0, dim // 2, heads)            # even channels: the key's; odd ones: zeros in the key
            size = (1 + r.integers(0, 128, heads) / 128) * np.exp2(-r.integers(0, 3, heads))
            size[:heads // 2] = first
            q[np.arange(heads), c] = size * np.sign(r.standard_normal(heads))
            most = np.maximum(size, np.where(r.random(heads) < 0.5, 1.0, 1 + r.integers(0, 128, heads) / 128))
            most[:heads // 4] = first                         # the element is its block's largest
            beside = most > size
            q[np.arange(heads)[beside], c[beside] + 1] = most[beside]
            unit = 2.0 ** np.floor(np.log2(2.0**13 / (2 * scale)))
            key = np.where(np.arange(dim) % 2 == 0, unit, 0.0)
            s = scale * q[np.arange(heads), c] * unit
            case = wide_head_case(dim, q, key, np.ones(dim))
            sinks = s.astype(np.float32)
            out = gpu.mxfp4_attention(**case.device(), scale=float(scale), causal=False,
                                      sinks=torch.from_numpy(sinks).to(DEV))[0].double().cpu().numpy()
            delta = 2.0**-13 * scale * most * unit + (dim + 14) * ref.U_F32 * np.abs(s) + 2 * ref.U_BF16
            d = s - sinks.astype(np.float64)
            lo, hi = (1 / (1 + np.exp(-(d + x))) for x in (-delta, delta))
            assert (delta < 1.1).all() and (hi < 0.8).all()
            off = np.maximum(lo[:, None] * (1 - ref.U_BF16) - out, out - hi[:, None] * (1 + ref.U_BF16)).max(1)
            assert off.max() <= 0, (middle, side, scale, q[off.argmax(), c[off.argmax()]], off.max())


@pytest.mark.parametrize("lens", [[(1, 200)], [(1, 3000), (2, 40)], [(40, 300), (3, 70)], [(300, 300), (70, 90)]])
@pytest.mark.parametrize("byte", [0, 3, 120, 247, 250, 251, 252])
def test_rising_scores_of_values_at_the_ends(gpu, lens, byte):
    """Scores that rise from step to step, by less and by more than what moves the maximum, beside values with scale bytes at
    the ends of the range, as long as the magnitudes of a channel's values sum to less than 2^128: finite, and as exact."""
    say(f"attention: rising scores, values of byte {byte}, {lens}")
    dim = 64
    for rises in ((0, 3, 6, 8, 12), (1, 8, 0.5), (0, 6, 6, -6, 12), (0, 64, 96)):
        case = Case(lens, 4, 2, dim, 16, 32)
        case.q[:] = 0
        case.q[:, :, 5] = 1          # the score: channel 5 of the key, in powers of two
        for s, (_, l) in enumerate(lens):
            key, value = np.zeros((l, 2, dim)), np.zeros((l, 2, dim))
            for i, x in enumerate(rises):
                j = min(40 * i + 3, l - 1)
                key[j, :, 5] = x
                # magnitudes of a channel sum to less than 2^128: a 6, or a 1 and some 0.5, times 2^(byte - 127)
                if byte == 252:
                    value[j, :, i::len(rises)] = 6.0
                else:
                    value[j] = 1.0 if i == len(rises) - 1 else 0.5
                    value[j, :, ::2] *= -1
            page = case.table[s, np.arange(l) // 16]
            j = np.arange(l)
            case.host[0][page, :, j % 16], case.host[1][page, :, j % 16] = ref.encode(key)
            code = ref.nearest(np.abs(value)) | (np.signbit(value).astype(np.uint8) << 3)
            case.host[2][page, :, j % 16], case.host[3][page, :, j % 16] = code[..., ::2] | code[..., 1::2] << 4, byte
        out = run(gpu, case, scale=float(np.log(2)))
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("lens,room", [([(40, 200)], 112), ([(1, 200), (7, 30), (3, 118)], 112), ([(5, 5000), (2, 900)], 4000),
                                       ([(150, 400), (150, 150)], 320), ([(300, 700), (200, 300), (1, 640)], 640),
                                       ([(30, 33000)], 32000), ([(3, 2**31 - 1), (90, 2**31 - 1)], 640)])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 50), (False, 0)])
def test_lengths_past_the_table(gpu, lens, room, causal, window):
    """The last query is at the length less 1 wherever the table ends; tokens past the table are not seen, and flagged."""
    say(f"attention: lengths past a table of {room}, {lens}, causal {causal}, window {window}")
    heads, kv, dim = 8, 2, 128
    sinks = np.linspace(-1, 1, heads).astype(np.float32)
    case = Case([(n, min(l, room)) for n, l in lens], heads, kv, dim, 16, 33)
    case.table = case.table[:, :room // 16].copy()
    case.kv_lens = np.array([l for _, l in lens], np.int32)
    flag = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = gpu.mxfp4_attention(**case.device(), causal=causal, window=window, sinks=torch.from_numpy(sinks).to(DEV),
                              err_flag=flag).double().cpu().numpy()
    assert flag.item() == 1
    for s, (n, length) in enumerate(lens):
        k, v = case.rows_of(s)
        for i in sorted({0, 1, n // 3, n // 2, n - 2, n - 1} & set(range(n))):
            pos = length - n + i
            lo = max(0, pos - window + 1) if window else 0
            hi = min(pos + 1 if causal else length, room)
            lo = min(lo, hi)
            at = case.offsets[s] + i
            want, bound = ref.attention(case.q[at:at + 1].double().numpy(), k[lo:hi], v[lo:hi], dim ** -0.5, False, 0, sinks)
            assert (np.abs(got[at:at + 1] - want) <= bound).all(), (s, i)
            assert hi > lo or not got[at].any()


def test_pages_missing_from_an_empty_cache(gpu):
    """A token on a page that an empty cache does not have sets the flag, as on any other page that is not there; queries that
    see no token do not."""
    say("attention: an empty cache and its flag")
    for lens in ([(2, 40), (1, 5)], [(90, 100)], [(1, 5000)], [(300, 300), (300, 600)]):
        case = Case(lens, 4, 2, 64, 16, 34)
        d = case.device()
        d["cache"] = tuple(t[:0] for t in d["cache"])
        flag = torch.zeros(1, dtype=torch.int32, device=DEV)
        assert not gpu.mxfp4_attention(**d, err_flag=flag).any() and flag.item() == 1
        flag.zero_()
        d["kv_lens"].zero_()
        assert not gpu.mxfp4_attention(**d, err_flag=flag).any() and flag.item() == 0
        gpu.mxfp4_attention(**{**case.device(), "cache": d["cache"], "q_offsets": torch.zeros_like(d["q_offsets"])},
                            err_flag=flag)
        assert flag.item() == 0


@pytest.mark.parametrize("first", [True, False])
@pytest.mark.parametrize("form,heads,kv,dim,chunk", [(20, 32, 8, 128, (1900, 2600)), (30, 64, 16, 64, (1300, 1400)),
                                                     (1224, 32, 8, 128, (1300, 2000)), (224, 16, 4, 128, (100, 9000))])
def test_prompts_beside_long_contexts(gpu, form, heads, kv, dim, chunk, first):
    """A chunk of a prompt, drafts and single tokens after contexts of all lengths in one call, whatever its form."""
    say(f"attention: a chunk of {chunk} beside single tokens, form {form}, {first}")
    others = [(1, 12000), (1, 40), (4, 6001), (0, 700), (1, 1), (1, 2500)]
    case = Case([chunk, *others] if first else [*others, chunk], heads, kv, dim, 64, 35)
    choose = gpu.load_library().e2m1_mxfp4_attention_form
    choose.argtypes = [ctypes.c_int64] * 6
    assert choose(case.tokens, len(case.lens), heads, kv, dim, case.table.shape[1] * 64) == form
    run(gpu, case)
    run(gpu, case, window=1500, sinks=np.linspace(-2, 2, heads).astype(np.float32))
