"""The paged 8-bit caches: page plan, quantising append, indexer scores and
sparse MLA over 8-bit pages, against a plain 64-bit numpy statement of them
(oracle/fp8_ref.py). CPU: the oracle's own pins and every refusal of the entry
points. GPU: parity, masks that leave nothing, bad pages and rows, strides,
padding, graphs, streams, offsets beyond 32 bits, and the whole run from plan to layer."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import fp8_ref as F
from oracle import lsa_ref as R
from sparse_attention_03_b200 import lsa

gpu = pytest.mark.gpu


# ------------------------------------------------------------------ CPU: the oracle's pins


def test_e4m3_table_and_rounding_match_torchs_type():
    codes = np.array([c for c in range(256) if c & 0x7F != 0x7F], dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(F.e4m3_values(codes), want)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.uniform(-448, 448, 4000), rng.standard_normal(4000) * 2.0 ** rng.integers(-12, 4, 4000),
                        (F.E4M3[1:] + F.E4M3[:-1]) / 2]).astype(np.float32)  # the ties too
    got = F.e4m3_codes(x.astype(np.float64))
    want = torch.from_numpy(x).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(F.e4m3_values(got), F.e4m3_values(want))


def test_quant_scale_is_the_smallest_power_of_two():
    for a in (448.0, 448.0 * 2, np.nextafter(448.0, 1e9), 1.0, 1.75, 1.7500001, 2.0 ** -126, 3e38, 2.0 ** -133):
        codes, s = F.quant(np.array([a, -a / 3, 0.0]))
        assert a <= 448 * s and (s == 2.0 ** -126 or a > 224 * s)
        assert abs(F.dequant(codes, s)[0] - a) <= max(a / 16, s * 2.0 ** -10)
    codes, s = F.quant(np.zeros(5))
    assert s == 1.0 and not codes.any()
    codes, s = F.quant(np.array([1.0, np.inf]))
    assert np.isnan(s) and not codes.any()


def test_page_plan_oracle_on_a_worked_case():
    table = np.array([[7, -1, -1], [3, 4, -1], [-1, -1, -1]])
    t, seq, pos, slot, tot = F.page_plan([63, 128, 0], [3, 1, 0], [9, 5, 8], table, 6)
    assert t.tolist() == [[7, 9, -1], [3, 4, 5], [-1, -1, -1]]
    assert seq == [0, 0, 0, 1, -1, -1] and pos == [63, 64, 65, 128, -1, -1]
    assert slot == [7 * 64 + 63, 9 * 64, 9 * 64 + 1, 5 * 64, -1, -1] and tot == [4, 2]


# ------------------------------------------------------------------ CPU: refusals


def _fake(n=1):
    return ctypes.c_void_p(0x10000 * n)  # aligned, never dereferenced by the host checks


def _fakes(k, base=1):
    return (ctypes.c_void_p * k)(*[0x10000 * (base + i) for i in range(k)])


def _cfg(**kw):
    c = lsa.LsaConfig().c()
    for k, v in kw.items():
        setattr(c, k, v)
    return ctypes.byref(c)


def test_page_plan_refusals():
    lib = lsa.load()
    ok = [4, _fake(1), _fake(2), _fake(3), 10, _fake(4), 8, 16, _fake(5), _fake(6), _fake(7), _fake(8), None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.lsa_page_plan(*a)

    assert call(_0=0) == lsa.LSA_ERR_INVALID
    assert call(_0=lsa.PLAN_MAX_SEQ + 1) == lsa.LSA_ERR_UNSUPPORTED
    assert call(_4=-1) == lsa.LSA_ERR_INVALID
    assert call(_6=0) == lsa.LSA_ERR_INVALID
    assert call(_7=-1) == lsa.LSA_ERR_INVALID
    for i in (1, 2, 3, 5, 8, 9, 10, 11):
        assert call(**{f"_{i}": None}) == lsa.LSA_ERR_INVALID, i
    assert b"lsa_page_plan" in lib.lsa_last_error()


def test_append_refusals():
    lib = lsa.load()
    ok = [_cfg(), 4, _fake(1), 2, _fakes(2, 2), 576, _fakes(2, 4), _fake(6), 128, _fake(7), 100, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.lsa_fp8_append(*a)

    assert call(_0=None) == lsa.LSA_ERR_INVALID
    assert call(_0=_cfg(n_heads=16)) == lsa.LSA_ERR_UNSUPPORTED
    for i, bad in ((1, -1), (3, 3), (3, -1), (5, 575), (5, 580), (8, 127), (8, 132), (10, 0), (10, 2 ** 25)):
        assert call(**{f"_{i}": bad}) == lsa.LSA_ERR_INVALID, (i, bad)
    for i in (2, 4, 6, 7, 9):
        assert call(**{f"_{i}": None}) == lsa.LSA_ERR_INVALID, i
    assert call(_3=0, _7=None, _9=None) == lsa.LSA_ERR_INVALID          # nothing to append
    assert call(_4=(ctypes.c_void_p * 2)(0x10000, None)) == lsa.LSA_ERR_INVALID
    assert call(_6=(ctypes.c_void_p * 2)(0x10000, 0x10008)) == lsa.LSA_ERR_INVALID
    assert call(_7=ctypes.c_void_p(0x10008)) == lsa.LSA_ERR_INVALID
    assert call(_1=0, _2=None) == lsa.LSA_OK                             # no rows: nothing happens


def test_index_scores_refusals():
    lib = lsa.load()
    ok = [_cfg(), 4, 4, _fake(1), _fake(2), _fake(3), _fake(4), _fake(5), 100, _fake(6), 8, 500, _fake(7), 512,
          None, _fake(8), 1 << 30, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.lsa_fp8_index_scores(*a)

    assert call(_0=_cfg(index_head_dim=64)) == lsa.LSA_ERR_UNSUPPORTED
    for i, bad in ((1, -1), (2, 0), (8, 0), (8, 2 ** 25), (10, 0), (11, 0), (11, 2 ** 31 + 1), (13, 499)):
        assert call(**{f"_{i}": bad}) == lsa.LSA_ERR_INVALID, (i, bad)
    for i in (4, 5, 6, 7, 9, 12):
        assert call(**{f"_{i}": None}) == lsa.LSA_ERR_INVALID, i
    assert call(_1=5, _3=None) == lsa.LSA_ERR_INVALID                    # more rows than sequences, unmapped
    for i in (5, 6, 7, 14):
        assert call(**{f"_{i}": ctypes.c_void_p(0x10004)}) == lsa.LSA_ERR_INVALID, i
    assert call(_1=0, _4=None) == lsa.LSA_OK
    assert call(_1=4096, _2=1, _15=None, _16=0) == lsa.LSA_ERR_WORKSPACE
    assert call(_15=None, _16=0) == lsa.LSA_ERR_WORKSPACE


def test_sparse_mla_and_forward_refusals():
    lib = lsa.load()
    ok = [_cfg(), 2, 4, 4, _fake(1), _fake(2), _fakes(2, 3), _fakes(2, 5), 100, _fake(7), 8, _fake(8), _fake(9), 500,
          _fakes(2, 10), None, None, 0, None]

    def call(**at):
        a = list(ok)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.lsa_fp8_sparse_mla(*a)

    assert call(_0=_cfg(softmax_scale=0.0)) == lsa.LSA_ERR_INVALID
    assert call(_0=_cfg(cli_factor=3)) == lsa.LSA_ERR_UNSUPPORTED
    for i, bad in ((1, 0), (1, 3), (2, -1), (3, 0), (8, 0), (10, 0), (13, 0)):
        assert call(**{f"_{i}": bad}) == lsa.LSA_ERR_INVALID, (i, bad)
    assert call(_0=_cfg(cli_factor=1), _1=2) == lsa.LSA_ERR_INVALID
    for i in (5, 6, 7, 9, 12, 14):
        assert call(**{f"_{i}": None}) == lsa.LSA_ERR_INVALID, i
    assert call(_7=(ctypes.c_void_p * 2)(0x10000, 0x10008)) == lsa.LSA_ERR_INVALID
    assert call(_2=5, _4=None) == lsa.LSA_ERR_INVALID
    assert call(_2=0) == lsa.LSA_OK

    ok2 = [_cfg(), 4, 4, _fake(1), _fake(2), 5000, _fake(3), _fake(4), _fake(5), _fakes(2, 6), _fakes(2, 8), 100,
           _fake(10), 90, _fakes(2, 11), None, None, None, _fake(13), 1 << 30, None]

    def fwd(**at):
        a = list(ok2)
        for i, v in at.items():
            a[int(i[1:])] = v
        return lib.lsa_fp8_forward(*a)

    for i in (4, 6, 7, 8, 9, 10, 12, 14):
        assert fwd(**{f"_{i}": None}) == lsa.LSA_ERR_INVALID, i
    assert fwd(_16=_fake(14)) == lsa.LSA_ERR_INVALID                     # idx_out without count_out
    assert fwd(_18=None, _19=0) == lsa.LSA_ERR_WORKSPACE
    assert fwd(_19=1000) == lsa.LSA_ERR_WORKSPACE
    assert fwd(_1=0) == lsa.LSA_OK


def test_workspace_sizes():
    cfg = lsa.LsaConfig()
    assert lsa.workspace_size(cfg, lsa.OP_FP8_FORWARD, 16, 16, 131072) >= 16 * 131072 * 4
    # dense (no index pass): only the attention's own partials
    assert lsa.workspace_size(cfg, lsa.OP_FP8_FORWARD, 16, 16, 2000) == lsa.workspace_size(cfg, lsa.OP_FP8_MLA, 16, 16, 2000)
    for op in (lsa.OP_FP8_INDEX, lsa.OP_FP8_MLA, lsa.OP_FP8_FORWARD):
        assert lsa.workspace_size(cfg, op, 0, 1, 100) == 256
        assert lsa.workspace_size(cfg, op, -1, 1, 100) == 0


def test_binding_refuses_wrong_tensors_on_the_cpu():
    cfg = lsa.LsaConfig()
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(TypeError):
        lsa.page_plan(i.long(), i, i, i.view(4, 1), i, i, i, i[:2])
    with pytest.raises(ValueError):
        lsa.page_plan(i, i[:3], i, i.view(4, 1), i, i, i, i[:2])
    with pytest.raises(ValueError):                                      # not on a CUDA device
        lsa.page_plan(i, i, i, i.view(4, 1), i, i, i, i[:2])
    with pytest.raises(TypeError):
        lsa.fp8_index_scores(cfg, i, i, torch.zeros(4, 32, 128), torch.zeros(4, 32), None, i.view(4, 1), 10, None, None)


# ------------------------------------------------------------------ GPU helpers

CFG = lsa.LsaConfig  # short


def _bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).bfloat16()


def _vals(t):
    return t.double().cpu().numpy()


def _i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Caches:
    """Sequences of given lengths in shuffled pages: pools, block table, and the
    values the codes stand for (per sequence)."""

    def __init__(self, lens, seed=0, cli=1, extra_pages=3, first_page=0, key_scale=1.0, lat_scale=1.0):
        rng = np.random.default_rng(seed)
        per = [-(-n // F.PAGE) for n in lens]
        n_pages = sum(per) + extra_pages
        order = rng.permutation(n_pages) + first_page
        self.n_pages = n_pages + first_page
        self.table = np.full((len(lens), max(per)), -1, dtype=np.int64)
        self.lens, self.keys, self.lat, self.lat_s = lens, [], [[] for _ in range(cli)], [[] for _ in range(cli)]
        at = 0
        for s, n in enumerate(per):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.key_pages = lsa.key_pages(self.n_pages)
        self.latent_pages = [lsa.latent_pages(self.n_pages) for _ in range(cli)]
        for s, n in enumerate(lens):
            k = rng.standard_normal((n, F.KEY)) * key_scale * 2.0 ** rng.integers(-4, 4, (n, 1))
            c, sc = F.quant(_vals(_bf16(k)))
            self.keys.append(F.dequant(c, sc))
            self._put_keys(s, c, sc)
            for z in range(cli):
                x = rng.standard_normal((n, F.LAT)) * lat_scale * 2.0 ** rng.integers(-3, 2, (n, 1))
                c, sc = F.quant(_vals(_bf16(x)))
                self.lat[z].append(F.dequant(c, sc))
                self.lat_s[z].append(sc)
                self._put_lat(z, s, c, sc)
        self.block_table = _i32(self.table)

    def slots(self, s, n):
        t = np.arange(n)
        return torch.from_numpy(self.table[s][t // F.PAGE] * F.PAGE + t % F.PAGE).cuda()

    def _put_keys(self, s, c, sc):
        sl = self.slots(s, len(c))
        pg, row = sl // F.PAGE, sl % F.PAGE
        codes = self.key_pages[:, :8192].view(-1, F.PAGE, F.KEY)
        codes[pg, row] = torch.from_numpy(c).cuda()
        self.key_pages.view(torch.float32)[pg, 2048 + row] = torch.from_numpy(sc).float().cuda()

    def _put_lat(self, z, s, c, sc):
        flat = self.latent_pages[z].view(-1, F.LAT_ROW)
        sl = self.slots(s, len(c))
        flat[sl, :F.LAT] = torch.from_numpy(c).cuda()
        flat.view(torch.float32)[sl, F.LAT // 4] = torch.from_numpy(sc).float().cuda()


def _score_case(lens, rows, cfg, seed=0, n_seq_of=None, hist=False, max_len=None, ld_extra=0, caches=None, scale=1.0):
    """Runs the indexer for rows [(seq, pos)] and checks every written and unwritten entry."""
    rng = np.random.default_rng(seed + 1)
    c = caches or Caches(lens, seed)
    n, max_len = len(rows), max_len or max(lens)
    q = _bf16(rng.standard_normal((n, 32, 128)) * scale).cuda()
    w = torch.from_numpy((rng.standard_normal((n, 32)) / 32 ** 0.5).astype(np.float32)).cuda()
    seq, pos = _i32([r[0] for r in rows]), _i32([r[1] for r in rows])
    scores = torch.full((n, max_len + ld_extra), 7.0, device="cuda")
    ws = lsa.workspace(cfg, lsa.OP_FP8_INDEX, n, len(lens), max_len)
    h = lsa.topk_hist_buffer(n) if hist else None
    lsa.fp8_index_scores(cfg, None if n_seq_of == "identity" else seq, pos, q, w, c.key_pages, c.block_table, max_len,
                         scores, ws, topk_hist=h)
    err = lsa.device_error()
    got = scores.double().cpu().numpy()
    ocfg = R.LsaConfig(index_topk=cfg.index_topk, index_init_tokens=cfg.index_init_tokens,
                       index_local_tokens=cfg.index_local_tokens)
    qv, wv = _vals(q), w.double().cpu().numpy()
    for r, (s, p) in enumerate(rows):
        if s < 0:
            assert (got[r] == 7.0).all(), "a padding row was written"
            continue
        want = F.score_row(qv[r], wv[r], c.keys[s], p, ocfg)
        # fp32 sums of exact products: 128 truncated additions at most 2^-23 of the absolute sum each, then the
        # 32 heads' weighted sum (two roundings a head, 2^-24 each)
        qc, qs = F.quant(qv[r])
        mag = np.abs(F.dequant(qc, qs)) @ np.abs(c.keys[s][:p + 1]).T          # [32, n]
        tol = (np.abs(wv[r])[:, None] * mag).sum(0) * (128 * 2.0 ** -23 + 66 * 2.0 ** -24) + 1e-37
        fin = np.isfinite(want)
        np.testing.assert_array_equal(got[r, :p + 1][~fin], want[~fin])
        assert (np.abs(got[r, :p + 1][fin] - want[fin]) <= tol[fin]).all(), (r, s, p)
        assert (got[r, p + 1:] == 7.0).all(), "an entry past the row's position was written"
    return err, scores, pos, h, c


def _mla_tol(q, c_val, s, keys, weights, out, scale):
    """Bounds of the kernel's roundings: the output's bf16 (half a step, 2^-8 relative), the weights' two 4-bit
    pieces (2^-8), their smallest step (weight * scale is carried as u = hi + lo / 64 with lo an e4m3 of smallest
    step 2^-9, so u is off by at most 2^-16, and the largest u of a frame is at least 2: 2^-17 of the largest
    weight * scale, times the codes), and the logits' fp32 sums of 576 exact
    products (a truncated addition loses 2^-23 of the absolute sum) with the query's split (2^-22 of the row's
    largest element): delta, once in a weight and once in the sum."""
    c = c_val[np.asarray(keys)]
    delta = scale * (577 * 2.0 ** -23 * (np.abs(q) @ np.abs(c).T)
                     + 2.0 ** -22 * np.abs(q).max() * np.abs(c).sum(1)[None]).max(1) + 2.0 ** -18
    v = np.abs(c[:, :512])
    s = np.asarray(s)[np.asarray(keys)]
    s_loud = np.where(c.any(axis=1), s, 0.0)             # a row of zeros has an arbitrary scale, which does not count
    tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2 * delta[:, None] + 2.0 ** -16) * (weights @ v) \
        + 2.0 ** -17 * (weights * s_loud).max(1, keepdims=True) * (v / s[:, None]).sum(0)[None] + 1e-37
    return tol, delta + 2.0 ** -18


def _mla_case(c, rows, lists, cfg, seed=0, topk=None, q_scale=1.0, identity=False, ws="full", max_len=None, want_err=0,
              keep=None):
    """lists: per row its key list, or None for idx NULL (dense)."""
    rng = np.random.default_rng(seed + 2)
    n, n_sub, K = len(rows), len(c.lat), cfg.index_topk
    q = [_bf16(rng.standard_normal((n, 32, 576)) * q_scale).cuda() for _ in range(n_sub)]
    seq, pos = _i32([r[0] for r in rows]), _i32([r[1] for r in rows])
    idx = cnt = None
    if lists is not None:
        ih = np.full((n, K), -5, dtype=np.int64)
        for r, l in enumerate(lists):
            ih[r, :len(l)] = l
        idx, cnt = _i32(ih), _i32([len(l) for l in lists])
    out = [torch.full((n, 32, 512), 9.0, dtype=torch.bfloat16, device="cuda") for _ in range(n_sub)]
    lse = [torch.full((n, 32), 9.0, device="cuda") for _ in range(n_sub)]
    max_len = max_len or max(c.lens)
    w = lsa.workspace(cfg, lsa.OP_FP8_MLA, n, len(c.lens), max_len) if ws == "full" else ws
    lsa.fp8_sparse_mla(cfg, None if identity else seq, pos, q, c.latent_pages, c.block_table, idx, cnt, max_len, out,
                       lse, w)
    assert lsa.device_error() == want_err
    for z in range(n_sub):
        qv, o, l = _vals(q[z]), _vals(out[z]), lse[z].double().cpu().numpy()
        for r, (s, p) in enumerate(rows):
            if s == -1:
                assert (o[r] == 9.0).all() and (l[r] == 9.0).all(), "a padding row was written"
                continue
            keys = list(range(p + 1)) if lists is None else list(lists[r])
            keys = [k for k in keys if 0 <= k <= p and (keep is None or keep(s, k))]
            if s < 0 or not keys:
                assert (o[r] == 0).all() and np.isneginf(l[r]).all()
                continue
            want, wl, wt = F.attend(qv[r], c.lat[z][s], keys, cfg.softmax_scale)
            tol, ltol = _mla_tol(qv[r], c.lat[z][s], c.lat_s[z][s], keys, wt, want, cfg.softmax_scale)
            assert (np.abs(l[r] - wl) <= ltol).all(), (z, r, np.abs(l[r] - wl).max())
            assert (np.abs(o[r] - want) <= tol).all(), (z, r, (np.abs(o[r] - want) / tol).max())
    return out, lse


def _random_lists(rows, topk, rng, full=True):
    out = []
    for s, p in rows:
        m = min(p + 1, topk) if full else int(rng.integers(0, min(p + 1, topk) + 1))
        out.append([] if s < 0 else rng.permutation(p + 1)[:m].tolist())
    return out


# ------------------------------------------------------------------ GPU: plan


@gpu
@pytest.mark.parametrize("n_seq,hi,fresh_hi,cap_extra", [(1, 1, 1, 0), (1, 200, 130, 3), (5, 64, 1, 0), (33, 500, 70, 9),
                                                         (1000, 300, 5, 0), (1025, 130, 2, 1), (4100, 70, 3, 50),
                                                         (16384, 65, 2, 0)])
def test_page_plan(n_seq, hi, fresh_hi, cap_extra):
    rng = np.random.default_rng(n_seq + hi)
    cached = rng.integers(0, hi + 1, n_seq)
    fresh = rng.integers(0, fresh_hi + 1, n_seq)
    width = -(-(hi + fresh_hi) // 64) + 1
    pool = rng.permutation(n_seq * width + 7)
    table = np.full((n_seq, width), -1, dtype=np.int64)
    at = 0
    for s in range(n_seq):
        m = -(-int(cached[s]) // 64)
        table[s, :m] = pool[at:at + m]
        at += m
    free = pool[at:]
    cap = int(fresh.sum()) + cap_extra
    want = F.page_plan(cached, fresh, free, table, cap)
    bt, totals = _i32(table), _i32([5, 5])
    seq, pos, slot = (torch.full((cap,), 77, dtype=torch.int32, device="cuda") for _ in range(3))
    for _ in range(2):  # the same inputs give the same outputs
        lsa.page_plan(_i32(cached), _i32(fresh), _i32(free), bt, seq, pos, slot, totals)
        assert lsa.device_error() == 0
        np.testing.assert_array_equal(bt.cpu().numpy(), want[0])
        for got, exp in zip((seq, pos, slot, totals), want[1:]):
            np.testing.assert_array_equal(got.cpu().numpy(), exp)


@gpu
def test_page_plan_runs_out_of_room():
    cached, fresh = _i32([10, -1, 200, 60, 0]), _i32([60, 4, 1, 10, 65])
    table = np.full((5, 3), -1)
    table[0, 0], table[2, :] = 1, (2, 3, 4)
    table[3, 0] = -7                                     # a page the caller should own, but does not
    free = np.array([11, 2 ** 25])                       # one good page, one past any pool
    bt = _i32(table)
    seq, pos, slot, totals = _i32([0] * 100), _i32([0] * 100), _i32([0] * 100), _i32([0, 0])
    lsa.page_plan(cached, fresh, _i32(free), bt, seq, pos, slot, totals)
    assert lsa.device_error() == lsa.DEVERR_POS | lsa.DEVERR_COUNT | lsa.DEVERR_PAGE
    c2, f2 = [10, -1, 200, 60, 0], [60, 4, 1, 10, 65]
    want = F.page_plan(c2, f2, free, table, 100)
    np.testing.assert_array_equal(seq.cpu().numpy(), want[1])
    np.testing.assert_array_equal(pos.cpu().numpy(), want[2])
    np.testing.assert_array_equal(slot.cpu().numpy(), want[3])
    np.testing.assert_array_equal(totals.cpu().numpy(), want[4])
    got = bt.cpu().numpy()
    assert got[0].tolist() == [1, 11, -1] and got[2].tolist() == [2, 3, 4] and got[4].tolist()[:2] == [-1, -1]


# ------------------------------------------------------------------ GPU: append


def _append_rows(rng, n, d):
    x = rng.standard_normal((n, d)) * 2.0 ** rng.integers(-20, 20, (n, 1)).astype(np.float64)
    x[1 % n] = 0.0
    if n > 8:
        x[2] = 448.0 / 2 ** 30
        x[3, 0] = np.inf
        x[4, d - 1] = np.nan
        x[5] *= 1e38 / np.abs(x[5]).max()
        x[6] *= 1e-39 / np.abs(x[6]).max()               # bf16 subnormals: the scale stops at 2^-126
        x[7, ::2] *= 2.0 ** -30                           # elements far below the row's largest
    return _bf16(x)


@gpu
@pytest.mark.parametrize("n,n_sub,gap,keys", [(1, 1, 0, True), (1, 0, 0, True), (9, 2, 8, True), (64, 2, 0, False),
                                              (333, 1, 64, True), (1000, 2, 24, True)])
def test_append_codes_and_scales_bit_for_bit(n, n_sub, gap, keys):
    rng = np.random.default_rng(n)
    n_pages = -(-n // 64) + 2
    slot = rng.permutation(n_pages * 64)[:n]
    if n > 20:
        slot[::7] = -1
    def wide(d):  # rows `gap` elements apart, and the bits as fp64 values
        x = _append_rows(rng, n, d)
        y = torch.full((n, d + gap), 3.0, dtype=torch.bfloat16)
        y[:, :d] = x
        return y.cuda()[:, :d], x.double().numpy()
    lat = [wide(576) for _ in range(n_sub)]
    key = wide(128) if keys else None
    lp = [torch.full((n_pages, 64, 592), 0xAB, dtype=torch.uint8, device="cuda") for _ in range(n_sub)]
    kp = torch.full((n_pages, 8448), 0xAB, dtype=torch.uint8, device="cuda") if keys else None
    lsa.fp8_append(lsa.LsaConfig(), _i32(slot), [x[0] for x in lat], lp, key[0] if keys else None, kp)
    assert lsa.device_error() == 0

    def bits(s):
        return s.astype(np.float32).view(np.uint32)

    live = slot >= 0
    for z in range(n_sub):
        c, s = F.quant(lat[z][1])
        want = np.full((n_pages * 64, 592), 0xAB, dtype=np.uint8)
        want[slot[live], :576] = c[live]
        want[slot[live], 576:580] = s.astype(np.float32)[live, None].view(np.uint8)
        want[slot[live], 580:] = 0
        want[slot[live], 580] = (lat[z][1][live] == 0).all(axis=1)
        got = lp[z].view(-1, 592).cpu().numpy().copy()
        nan = np.isnan(s) & live
        assert np.isnan(got[slot[nan], 576:580].copy().view(np.float32)).all()
        got[slot[nan], 576:580] = want[slot[nan], 576:580]
        neg0 = ((got ^ want) == 0x80) & ((want & 0x7F) == 0)   # the sign of a zero is kept as torch keeps it
        np.testing.assert_array_equal(np.where(neg0, want, got), want)
    if keys:
        c, s = F.quant(key[1])
        got = kp.cpu().numpy()
        codes = got[:, :8192].reshape(-1, 128)
        sc = got[:, 8192:].copy().view(np.float32).reshape(-1)
        np.testing.assert_array_equal(F.e4m3_values(codes[slot[live]]), F.e4m3_values(c[live]))
        np.testing.assert_array_equal(sc[slot[live]], s[live].astype(np.float32))
        rest = np.setdiff1d(np.arange(n_pages * 64), slot[live])
        assert (codes[rest] == 0xAB).all() and (sc.view(np.uint32)[rest] == 0xABABABAB).all()


@gpu
def test_append_flags_slots_outside_the_pool():
    lp = [lsa.latent_pages(2)]
    x = torch.ones(4, 576, dtype=torch.bfloat16, device="cuda")
    lsa.fp8_append(lsa.LsaConfig(), _i32([128, -2, 127, 2 ** 31 - 1]), [x], lp)
    assert lsa.device_error() == lsa.DEVERR_PAGE
    rows = lp[0].view(-1, 592).cpu().numpy()
    assert rows[127, :576].all() and not rows[:127].any()


# ------------------------------------------------------------------ GPU: scores


TINY = dict(index_topk=8, index_init_tokens=2, index_local_tokens=4)


@gpu
@pytest.mark.parametrize("hist", [False, True])
@pytest.mark.parametrize("lens", [[1], [63], [64, 65], [1, 127, 128, 129], [300, 5, 2049, 700]])
def test_scores_decode(lens, hist):
    rows = [(s, n - 1) for s, n in enumerate(lens)]
    for cfg in (lsa.LsaConfig(), lsa.LsaConfig(**TINY)):
        err, scores, pos, h, _ = _score_case(lens, rows, cfg, hist=hist, ld_extra=3)
        assert err == 0
        if hist:  # the histogram is the top-k's own first pass over these scores
            _check_hist(rows, scores, h, cfg)


@gpu
def test_scores_rows_without_a_map_are_the_sequences():
    lens = [200, 64, 130]
    assert _score_case(lens, [(s, n - 1) for s, n in enumerate(lens)], lsa.LsaConfig(**TINY), n_seq_of="identity")[0] == 0


@gpu
@pytest.mark.parametrize("bound", [None, 120000])  # the bound on the lengths decides the kernel's form
@pytest.mark.parametrize("lens,new,pad", [([40], 40, 0), ([300], 37, 2), ([129, 700], 64, 5), ([17, 20, 260, 33], 17, 0),
                                          ([1500], 129, 1), ([300, 140, 64, 700] * 5, 4, 0), ([131, 260, 5, 400] * 5, 3, 0),
                                          ([131, 260, 65, 400] * 4, 6, 3)])
def test_scores_rows_of_prompts(lens, new, pad, bound):
    # many rows of few sequences (blocks of rows share key tiles; a block may span sequences and end in padding)
    rows = [(s, p) for s, n in enumerate(lens) for p in range(max(0, n - new), n)] + [(-1, -1)] * pad
    for cfg in (lsa.LsaConfig(**TINY), lsa.LsaConfig(index_topk=64, index_init_tokens=0, index_local_tokens=0)):
        err, *_ = _score_case(lens, rows, cfg, seed=len(lens), max_len=bound or max(lens) + 11)
        assert err == 0


def _check_hist(rows, scores, h, cfg):
    for r, (s, p) in enumerate(rows):
        lo, hi = cfg.index_init_tokens, p + 1 - cfg.index_local_tokens
        want = np.zeros(2048, dtype=np.int64)
        if s >= 0 and p + 1 > cfg.index_topk and hi > lo:
            f = scores[r, lo:hi].cpu().numpy().copy()
            f[f == 0] = 0.0
            u = f.view(np.uint32)
            np.add.at(want, np.where(u & 0x80000000, ~u, u | 0x80000000) >> 21, 1)
        np.testing.assert_array_equal(h[r, :2048].cpu().numpy(), want)
        assert not h[r, 2048:].cpu().numpy().any()


@gpu
@pytest.mark.parametrize("bound", [None, 60000, 60001])
def test_scores_of_prompt_rows_with_the_histogram(bound):
    lens = [300, 150]
    rows = [(s, p) for s, n in enumerate(lens) for p in range(n - 40, n)] + [(-1, -1)] * 3
    cfg = lsa.LsaConfig(**TINY)
    err, scores, pos, h, _ = _score_case(lens, rows, cfg, hist=True, max_len=bound)
    assert err == 0
    _check_hist(rows, scores, h, cfg)


@gpu
@pytest.mark.parametrize("hist", [False, True])
def test_scores_of_many_short_sequences(hist):
    # more rows than the GPU runs CTAs of the streaming form: each takes the tiles of several rows
    rng = np.random.default_rng(8)
    lens = rng.integers(1, 300, 500).tolist()
    rows = [(s, n - 1) for s, n in enumerate(lens)]
    for i in (0, 17, 18, 499):
        rows[i] = (-1, -1)
    cfg = lsa.LsaConfig(**TINY)
    err, scores, pos, h, _ = _score_case(lens, rows, cfg, hist=hist)
    assert err == 0
    if hist:
        _check_hist(rows, scores, h, cfg)


@gpu
@pytest.mark.parametrize("bound", [None, 60000])
def test_scores_padding_between_rows_and_unordered_positions(bound):
    rng = np.random.default_rng(5)
    lens = [200, 333]
    rows = [(int(s), int(rng.integers(0, lens[s]))) if i % 5 else (-1, -1) for i, s in enumerate(rng.integers(0, 2, 70))]
    assert _score_case(lens, rows, lsa.LsaConfig(**TINY), max_len=bound)[0] == 0


@gpu
@pytest.mark.parametrize("scale", [2.0 ** -60, 2.0 ** 40])
def test_scores_far_from_one(scale):
    lens = [150, 90]
    c = Caches(lens, 3, key_scale=scale)
    assert _score_case(lens, [(0, 149), (1, 89)], lsa.LsaConfig(**TINY), caches=c)[0] == 0
    rows = [(0, p) for p in range(100, 150)]
    assert _score_case(lens, rows, lsa.LsaConfig(**TINY), caches=c, scale=1 / scale)[0] == 0
    assert _score_case(lens, rows, lsa.LsaConfig(**TINY), caches=c, scale=1 / scale, max_len=60000)[0] == 0


@gpu
@pytest.mark.parametrize("many", [False, True])
def test_scores_bad_rows_and_pages(many):
    cfg = lsa.LsaConfig(**TINY)
    lens = [300, 128]
    c = Caches(lens, 1)
    bad = c.table.copy()
    bad[0, 2] = -1
    bad[0, 3] = c.n_pages
    c.block_table = _i32(bad)
    base = [(0, 299), (0, 130), (1, 127), (7, 5), (-2, 3), (1, 400)]
    rows = base + ([(0, 290)] * 60 if many else [])
    n, bound = len(rows), 60000 if many else 320
    rng = np.random.default_rng(0)
    q = _bf16(rng.standard_normal((n, 32, 128))).cuda()
    w = torch.from_numpy(rng.standard_normal((n, 32)).astype(np.float32)).cuda()
    scores = torch.full((n, bound), 7.0, device="cuda")
    ws = lsa.workspace(cfg, lsa.OP_FP8_INDEX, n, 2, bound)
    lsa.fp8_index_scores(cfg, _i32([r[0] for r in rows]), _i32([r[1] for r in rows]), q, w, c.key_pages, c.block_table,
                         bound, scores, ws)
    assert lsa.device_error() == lsa.DEVERR_PAGE | lsa.DEVERR_SEQ | lsa.DEVERR_POS
    got = scores.cpu().numpy()
    assert np.isneginf(got[0, 128:256]).all() and np.isfinite(got[0, 2:128]).all() and np.isinf(got[0, 296:300]).all()
    assert np.isfinite(got[1, 2:127]).all() and np.isposinf(got[1, 127:131]).all()
    assert np.isfinite(got[2, 2:124]).all()
    assert (got[3] == 7.0).all() and (got[4] == 7.0).all()
    ok = F.score_row(_vals(q)[2], w.double().cpu().numpy()[2], c.keys[1], 127, R.LsaConfig(8, 2, 4))
    assert np.allclose(got[2, 2:124], ok[2:124], rtol=1e-3, atol=1e-3)


@gpu
@pytest.mark.parametrize("many", [False, True])
def test_scores_of_non_finite_vectors_count_as_zero(many):
    # max(0, NaN) is 0, as in the bf16 indexer: a key or a query head that stands for NaN adds nothing
    cfg = lsa.LsaConfig(index_topk=8, index_init_tokens=0, index_local_tokens=1)
    c = Caches([200], 2)
    flat = c.key_pages.view(torch.float32)
    flat[int(c.table[0, 1]), 2048 + 5] = float("nan")    # key 69
    n, bound = (40, 60000) if many else (1, 200)
    q = _bf16(np.random.default_rng(1).standard_normal((n, 32, 128))).cuda()
    q[:, 3, 17] = float("inf")
    w = torch.ones(n, 32, device="cuda")
    scores = torch.zeros(n, bound, device="cuda")
    ws = lsa.workspace(cfg, lsa.OP_FP8_INDEX, n, 1, bound)
    lsa.fp8_index_scores(cfg, _i32([0] * n), _i32([199] * n), q, w, c.key_pages, c.block_table, bound, scores, ws)
    assert lsa.device_error() == 0
    got = scores[:, :199].double().cpu().numpy()
    assert np.isfinite(got).all() and (got[:, 69] == 0).all()
    qv = _vals(q)
    qv[:, 3] = 0
    for r in (0, n - 1):
        want = F.score_row(qv[r], np.ones(32), c.keys[0], 199, R.LsaConfig(8, 0, 1))[:199]
        want[69] = 0
        assert np.allclose(got[r], want, rtol=1e-4, atol=1e-4 * np.abs(want).max())


# ------------------------------------------------------------------ GPU: attention


@gpu
@pytest.mark.parametrize("lens", [[1], [2, 64], [65, 128, 127], [129, 700, 33, 2049]])
@pytest.mark.parametrize("dense", [False, True])
def test_mla_decode(lens, dense):
    rng = np.random.default_rng(len(lens))
    c = Caches(lens, 4, cli=2)
    rows = [(s, n - 1) for s, n in enumerate(lens)]
    cfg = lsa.LsaConfig()
    _mla_case(c, rows, None if dense else _random_lists(rows, 2048, rng), cfg)
    _mla_case(c, rows, None if dense else _random_lists(rows, 2048, rng), cfg, identity=True, ws=None)


@gpu
@pytest.mark.parametrize("topk,full", [(2048, True), (2048, False), (130, True), (9, True), (129, False)])
def test_mla_prompt_rows_padding_and_short_lists(topk, full):
    rng = np.random.default_rng(topk)
    lens = [2300, 40, 180]
    c = Caches(lens, 6, cli=1)
    rows = [(0, 2299), (0, 2200), (-1, -1), (1, 0), (1, 39), (2, 100), (2, 101), (-1, 5), (0, 64), (0, 2047), (0, 2048)]
    lists = _random_lists(rows, topk, rng, full)
    lists[4] = []                                         # a row with nothing selected
    cfg = lsa.LsaConfig(index_topk=topk, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    _mla_case(c, rows, lists, cfg)
    _mla_case(c, rows, lists, cfg, ws=None)


@gpu
def test_mla_dense_beyond_the_selection_size():
    # idx NULL over more keys than index_topk (several frames of the softmax), one and many rows
    c = Caches([5000], 8, cli=1)
    cfg = lsa.LsaConfig(index_topk=64, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    _mla_case(c, [(0, 4999)], None, cfg)
    _mla_case(c, [(0, 4999)], None, cfg, ws=None)
    _mla_case(c, [(0, 4999), (0, 3), (0, 2500)], None, cfg)


@gpu
@pytest.mark.parametrize("first", [6.0, 60.0])
def test_mla_dense_with_the_weight_in_front(first):
    # the first keys outweigh every later one: the weights' frame comes down again every 16 tiles
    rng = np.random.default_rng(19)
    n = 4500
    q = _bf16(rng.standard_normal((1, 32, 576))).cuda()
    x = rng.standard_normal((n, 576)) * 0.05
    mean = _vals(q)[0].mean(0)
    x[:3] = mean / (mean @ mean) * first * 192 ** 0.5
    lat = _bf16(x).cuda()
    c = Caches([n], 20, cli=1)
    t = torch.arange(n, device="cuda")
    cfg = lsa.LsaConfig(cli_factor=1)
    lsa.fp8_append(cfg, (torch.from_numpy(c.table[0]).cuda()[t // 64] * 64 + t % 64).int(), [lat], c.latent_pages)
    codes, s = F.quant(_vals(lat))
    c.lat[0][0], c.lat_s[0][0] = F.dequant(codes, s), s
    for ws in (None, lsa.workspace(cfg, lsa.OP_FP8_MLA, 1, 1, n)):
        out, lse = [torch.empty(1, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.empty(1, 32, device="cuda")]
        lsa.fp8_sparse_mla(cfg, None, _i32([n - 1]), [q], c.latent_pages, c.block_table, None, None, n, out, lse, ws)
        assert lsa.device_error() == 0
        want, wl, wt = F.attend(_vals(q)[0], c.lat[0][0], range(n), cfg.softmax_scale)
        tol, ltol = _mla_tol(_vals(q)[0], c.lat[0][0], s, range(n), wt, want, cfg.softmax_scale)
        assert (np.abs(lse[0][0].double().cpu().numpy() - wl) <= ltol).all()
        assert (np.abs(_vals(out[0])[0] - want) <= tol).all()


@gpu
def test_mla_rows_of_one_key_are_exact():
    # the output is the key's own value: 4 significant bits, exact in bf16 (and lse its logit)
    c = Caches([300], 24, cli=1)
    cfg = lsa.LsaConfig(index_topk=8, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    keys = [0, 5, 77, 128, 299, 131]
    n = len(keys)
    q = [_bf16(np.random.default_rng(0).standard_normal((n, 32, 576)) * 3).cuda()]
    idx = np.full((n, 8), -1)
    idx[:, 0] = keys
    out, lse = [torch.zeros(n, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.zeros(n, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, _i32([0] * n), _i32([299] * n), q, c.latent_pages, c.block_table, _i32(idx), _i32([1] * n), 300,
                       out, lse, None)
    assert lsa.device_error() == 0
    for r, k in enumerate(keys):
        want = np.broadcast_to(c.lat[0][0][k, :512], (32, 512))
        np.testing.assert_array_equal(_vals(out[0])[r], want)
        x = cfg.softmax_scale * (_vals(q[0])[r] @ c.lat[0][0][k])
        bound = cfg.softmax_scale * (577 * 2.0 ** -23 * (np.abs(_vals(q[0])[r]) @ np.abs(c.lat[0][0][k]))
                                     + 2.0 ** -22 * np.abs(_vals(q[0])[r]).max() * np.abs(c.lat[0][0][k]).sum()) + 2.0 ** -20
        assert (np.abs(lse[0][r].double().cpu().numpy() - x) <= bound).all()


@gpu
def test_mla_non_finite_queries_give_nan_for_their_row_alone():
    c = Caches([200], 23, cli=1)
    cfg = lsa.LsaConfig(cli_factor=1)
    q = [_bf16(np.random.default_rng(0).standard_normal((3, 32, 576))).cuda()]
    q[0][1, 5, 100] = float("inf")
    out, lse = [torch.zeros(3, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.zeros(3, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, _i32([0, 0, 0]), _i32([199, 150, 60]), q, c.latent_pages, c.block_table, None, None, 200,
                       out, lse, None)
    assert lsa.device_error() == 0
    assert torch.isnan(out[0][1]).all() and torch.isnan(lse[0][1]).all()
    for r, p in ((0, 199), (2, 60)):
        want, wl, wt = F.attend(_vals(q[0])[r], c.lat[0][0], range(p + 1), cfg.softmax_scale)
        tol, ltol = _mla_tol(_vals(q[0])[r], c.lat[0][0], c.lat_s[0][0], range(p + 1), wt, want, cfg.softmax_scale)
        assert (np.abs(_vals(out[0])[r] - want) <= tol).all()
        assert (np.abs(lse[0][r].double().cpu().numpy() - wl) <= ltol).all()


@gpu
def test_mla_many_rows_walk_every_cta():
    # more rows than the GPU has SMs, two sub-blocks: CTAs take several rows each
    rng = np.random.default_rng(3)
    c = Caches([260, 333], 9, cli=2)
    rows = [(i % 2, 259 - i // 2 if i % 2 == 0 else 332 - i // 2) for i in range(400)]
    rows[17] = rows[18] = (-1, -1)
    cfg = lsa.LsaConfig(index_topk=200, index_init_tokens=1, index_local_tokens=2)
    lists = _random_lists(rows, 200, rng)
    lists[33] = []
    _mla_case(c, rows, lists, cfg)


@gpu
@pytest.mark.parametrize("lat_scale,q_scale", [(2.0 ** -40, 2.0 ** 40), (2.0 ** 30, 2.0 ** -30), (8.0, 4.0), (2.0 ** -30, 1.0)])
def test_mla_scales_and_peaked_rows(lat_scale, q_scale):
    # peaked rows: logits of hundreds, the running maximum moves often; and flat ones
    rng = np.random.default_rng(11)
    c = Caches([900, 300], 12, cli=1, lat_scale=lat_scale)
    rows = [(0, 899), (1, 299), (0, 500)]
    cfg = lsa.LsaConfig(cli_factor=1)
    _mla_case(c, rows, _random_lists(rows, 2048, rng), cfg, q_scale=q_scale)


@gpu
def test_mla_keys_in_rising_order_of_their_logits():
    # each later tile beats the maximum so far: every tile rescales what came before
    c = Caches([1024], 13, cli=1)
    cfg = lsa.LsaConfig(cli_factor=1)
    q = _bf16(np.random.default_rng(15).standard_normal((1, 32, 576)) * 3).cuda()
    x = _vals(q)[0, 0] @ c.lat[0][0].T
    order = np.argsort(x)
    for keys in (order, order[::-1]):
        idx = _i32(np.concatenate([keys, np.full(1024, -1)])[None])
        out, lse = [torch.empty(1, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.empty(1, 32, device="cuda")]
        lsa.fp8_sparse_mla(cfg, None, _i32([1023]), [q], c.latent_pages, c.block_table, idx, _i32([1024]), 1024, out,
                           lse, None)
        assert lsa.device_error() == 0
        want, wl, wt = F.attend(_vals(q)[0], c.lat[0][0], keys, cfg.softmax_scale)
        tol, ltol = _mla_tol(_vals(q)[0], c.lat[0][0], c.lat_s[0][0], keys, wt, want, cfg.softmax_scale)
        assert (np.abs(lse[0][0].double().cpu().numpy() - wl) <= ltol).all()
        assert (np.abs(_vals(out[0])[0] - want) <= tol).all()


@gpu
def test_mla_a_row_of_zeros_takes_weight_but_no_precision():
    # a zero key holds most of the softmax; the others' small weights keep their 8 bits
    rng = np.random.default_rng(30)
    lat = _bf16(np.concatenate([np.zeros((1, 576)), rng.standard_normal((700, 576)) * 0.01])).cuda()
    c = Caches([701], 31, cli=1)
    t = torch.arange(701, device="cuda")
    slot = (torch.from_numpy(c.table[0]).cuda()[t // 64] * 64 + t % 64).int()
    cfg = lsa.LsaConfig(cli_factor=1)
    # every other key's logit is near -9 (in nats): q is opposed to the keys' common direction
    lat2 = _vals(lat)
    lat2[1:] += 0.3
    lat2 = _bf16(lat2).cuda()
    lat2[0] = 0
    lsa.fp8_append(cfg, slot, [lat2], c.latent_pages)
    codes, s = F.quant(_vals(lat2))
    c.lat[0][0], c.lat_s[0][0] = F.dequant(codes, s), s
    qq = _bf16(np.broadcast_to(-0.72 + 0.05 * rng.standard_normal((1, 32, 576)), (1, 32, 576))).cuda()
    out, lse = [torch.empty(1, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.empty(1, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, None, _i32([700]), [qq], c.latent_pages, c.block_table, None, None, 701, out, lse, None)
    assert lsa.device_error() == 0
    want, wl, wt = F.attend(_vals(qq)[0], c.lat[0][0], range(701), cfg.softmax_scale)
    assert wt[:, 0].min() > 0.5 and wt[:, 1:].max() < 2.0 ** -10
    tol, ltol = _mla_tol(_vals(qq)[0], c.lat[0][0], s, range(701), wt, want, cfg.softmax_scale)
    assert (np.abs(lse[0][0].double().cpu().numpy() - wl) <= ltol).all()
    assert (np.abs(_vals(out[0])[0] - want) <= tol).all()


@gpu
def test_mla_repeated_and_bad_indices_and_pages():
    c = Caches([300, 500], 14, cli=1)
    cfg = lsa.LsaConfig(index_topk=40, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    rows = [(0, 299), (1, 499), (1, 100)]
    lists = [[5, 5, 5, 64, 299, 0], list(range(100, 140)), [100, 99, 3]]
    _mla_case(c, rows, lists, cfg)
    bad = [[5, -1, 300, 64, 2 ** 31 - 1, 299], list(range(100, 140)), [101, 99, -7]]
    _mla_case(c, rows, bad, cfg, want_err=lsa.DEVERR_INDEX)
    t = c.table.copy()
    t[1, 2] = c.n_pages                                   # tokens 128..191 of sequence 1
    c.block_table = _i32(t)
    _mla_case(c, rows, lists, cfg, want_err=lsa.DEVERR_PAGE, keep=lambda s, k: not (s == 1 and 128 <= k < 192))


@gpu
def test_mla_bad_counts_sequences_and_positions():
    c = Caches([300], 14, cli=1)
    cfg = lsa.LsaConfig(index_topk=40, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    q = [_bf16(np.random.default_rng(0).standard_normal((4, 32, 576))).cuda()]
    idx = _i32(np.tile(np.arange(40), (4, 1)))
    out, lse = [torch.full((4, 32, 512), 9.0, dtype=torch.bfloat16, device="cuda")], [torch.zeros(4, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, _i32([0, 0, 3, 0]), _i32([299, 299, 5, 5000]), q, c.latent_pages, c.block_table, idx,
                       _i32([-3, 41, 2, 10]), 300, out, lse, None)
    assert lsa.device_error() == lsa.DEVERR_COUNT | lsa.DEVERR_SEQ | lsa.DEVERR_POS
    assert (out[0][0] == 0).all() and torch.isneginf(lse[0][0]).all()      # count -3: no keys
    assert (out[0][2] == 0).all() and torch.isneginf(lse[0][2]).all()      # unknown sequence
    want, wl, _ = F.attend(_vals(q[0])[1], c.lat[0][0], range(40), cfg.softmax_scale)
    assert np.allclose(lse[0][1].cpu().numpy(), wl, atol=1e-4)             # count 41: clamped to 40
    assert np.isfinite(_vals(out[0])).all()


@gpu
def test_mla_non_finite_keys_stay_where_they_are_selected():
    c = Caches([200], 15, cli=1)
    c.latent_pages[0].view(-1, 592).view(torch.float32)[c.slots(0, 200)[77], 144] = float("nan")
    cfg = lsa.LsaConfig(index_topk=64, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    rows = [(0, 199), (0, 199)]
    lists = [list(range(60)), list(range(70, 100))]
    ih = np.full((2, 64), -1)
    for r, l in enumerate(lists):
        ih[r, :len(l)] = l
    q = [_bf16(np.random.default_rng(0).standard_normal((2, 32, 576))).cuda()]
    out, lse = [torch.zeros(2, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.zeros(2, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, _i32([0, 0]), _i32([199, 199]), q, c.latent_pages, c.block_table, _i32(ih), _i32([60, 30]),
                       200, out, lse, None)
    assert lsa.device_error() == 0
    assert torch.isfinite(out[0][0]).all() and torch.isfinite(lse[0][0]).all()
    assert torch.isnan(out[0][1]).all() and torch.isnan(lse[0][1]).all()


# ------------------------------------------------------------------ GPU: large offsets, streams, graphs


@gpu
def test_offsets_beyond_32_bits():
    # pools of more than 2^32 bytes, the sequences in their last pages
    c = Caches([200, 70], 16, cli=1, first_page=115000)
    cfg = lsa.LsaConfig(index_topk=100, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    rows = [(0, 199), (1, 69)]
    assert c.latent_pages[0].numel() > 2 ** 32
    _mla_case(c, rows, _random_lists(rows, 100, np.random.default_rng(0)), cfg)
    x = torch.ones(1, 576, dtype=torch.bfloat16, device="cuda")
    last = c.n_pages * 64 - 1
    lsa.fp8_append(cfg, _i32([last]), [x], c.latent_pages)
    assert int(c.latent_pages[0].view(-1, 592)[last, 0]) == 0x78            # 1 = 2^-8 * 256
    del c
    k = Caches([200, 70], 16, cli=0, first_page=510000)
    assert k.key_pages.numel() > 2 ** 32
    assert _score_case([200, 70], rows, lsa.LsaConfig(**TINY), caches=k)[0] == 0
    assert _score_case([200, 70], [(0, p) for p in range(150, 200)], lsa.LsaConfig(**TINY), caches=k)[0] == 0


def _layer_inputs(rng, n, cli=2):
    q_idx = _bf16(rng.standard_normal((n, 32, 128))).cuda()
    w = torch.from_numpy((rng.standard_normal((n, 32)) / 32 ** 0.5).astype(np.float32)).cuda()
    q = [_bf16(rng.standard_normal((n, 32, 576))).cuda() for _ in range(cli)]
    out = [torch.zeros(n, 32, 512, dtype=torch.bfloat16, device="cuda") for _ in range(cli)]
    lse = [torch.zeros(n, 32, device="cuda") for _ in range(cli)]
    return q_idx, w, q, out, lse


@gpu
def test_serving_run_from_plan_to_layer():
    """Requests arrive, are planned, appended in two steps (a prompt chunk, then decode tokens) and attended;
    the last step runs as a captured graph too, twice, on a side stream."""
    rng = np.random.default_rng(21)
    cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    ocfg = R.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    n_seq, width, n_pages = 3, 8, 30
    bt = torch.full((n_seq, width), -1, dtype=torch.int32, device="cuda")
    lp, kp = [lsa.latent_pages(n_pages) for _ in range(2)], lsa.key_pages(n_pages)
    free = rng.permutation(n_pages)
    used = 0
    cached = np.zeros(n_seq, dtype=np.int64)
    vals = {"k": [np.zeros((0, 128))] * n_seq, "c0": [np.zeros((0, 576))] * n_seq, "c1": [np.zeros((0, 576))] * n_seq,
            "s0": [np.zeros(0)] * n_seq, "s1": [np.zeros(0)] * n_seq}
    for step, fresh in enumerate(([150, 64, 1], [1, 1, 1], [200, 1, 0], [1, 1, 1])):
        fresh = np.array(fresh)
        cap = int(fresh.sum()) + 2
        seq, pos, slot, totals = (torch.empty(k, dtype=torch.int32, device="cuda") for k in (cap, cap, cap, 2))
        lsa.page_plan(_i32(cached), _i32(fresh), _i32(free[used:]), bt, seq, pos, slot, totals)
        used += int(totals[1])
        k = _bf16(rng.standard_normal((cap, 128))).cuda()
        lat = [_bf16(rng.standard_normal((cap, 576))).cuda() for _ in range(2)]
        lsa.fp8_append(cfg, slot, lat, lp, k, kp)
        sh, ph = seq.cpu().numpy(), pos.cpu().numpy()
        for name, x in (("k", k), ("c0", lat[0]), ("c1", lat[1])):
            codes, sc = F.quant(_vals(x))
            d = F.dequant(codes, sc)
            vals[name] = [np.concatenate([v, d[sh == s]]) for s, v in enumerate(vals[name])]
            if name != "k":
                vals["s" + name[1]] = [np.concatenate([v, sc[sh == s]]) for s, v in enumerate(vals["s" + name[1]])]
        cached = cached + fresh
        max_len = int(cached.max())
        q_idx, w, q, out, lse = _layer_inputs(rng, cap)
        idx = torch.full((cap, 96), -1, dtype=torch.int32, device="cuda")
        cnt = torch.zeros(cap, dtype=torch.int32, device="cuda")
        ws = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, cap, n_seq, max_len)

        def layer():
            lsa.fp8_forward(cfg, seq, pos, max_len, q_idx, w, kp, q, lp, bt, out, lse, ws, idx_out=idx, count_out=cnt)

        layer()
        assert lsa.device_error() == 0
        if step == 3:  # captured and replayed, on another stream
            eager, eager_idx = [o.clone() for o in out], idx.clone()
            s2 = torch.cuda.Stream()
            s2.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s2):
                layer()
                g = torch.cuda.CUDAGraph()
                with torch.cuda.graph(g, stream=s2):
                    layer()
                for o in out:
                    o.zero_()
                g.replay()
                g.replay()
            torch.cuda.current_stream().wait_stream(s2)
            torch.cuda.synchronize()
            assert lsa.device_error() == 0
            # The selection is the same set in any order; the sums over it are the same bits for the same order.
            assert torch.equal(eager_idx.sort(dim=1).values, idx.sort(dim=1).values)
            for r in range(cap):
                if torch.equal(eager_idx[r], idx[r]):
                    assert all(torch.equal(a[r], b[r]) for a, b in zip(eager, out))
            del g
        ih, ch = idx.cpu().numpy(), cnt.cpu().numpy()
        for r in range(cap):
            if sh[r] < 0:
                assert not out[0][r].any()
                continue
            s, p = int(sh[r]), int(ph[r])
            sel = ih[r, :ch[r]]
            assert len(set(sel.tolist())) == ch[r] == min(p + 1, 96) and sel.min() >= 0 and sel.max() <= p
            sc = F.score_row(_vals(q_idx)[r], w.double().cpu().numpy()[r], vals["k"][s], p, ocfg)
            want_idx, gap = R.select_topk(sc, p, ocfg)
            if p + 1 > 96 and gap is not None and gap > 1e-4:
                np.testing.assert_array_equal(np.sort(sel), np.sort(want_idx))
            for z in range(2):
                c, cs = vals[f"c{z}"][s], vals[f"s{z}"][s]
                o, l, wt = F.attend(_vals(q[z])[r], c, sel, cfg.softmax_scale)
                tol, ltol = _mla_tol(_vals(q[z])[r], c, cs, sel, wt, o, cfg.softmax_scale)
                assert (np.abs(lse[z][r].double().cpu().numpy() - l) <= ltol).all()
                assert (np.abs(_vals(out[z])[r] - o) <= tol).all()


@gpu
@pytest.mark.parametrize("max_len", [300, 60000])     # the indexer's two forms
def test_captured_layer_follows_its_inputs(max_len):
    # lengths, sequences and pages change in place between replays; every replay is a call on what stands there
    cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    c = Caches([300, 260], 41, cli=2)
    n = 66
    rng = np.random.default_rng(42)
    q_idx, w, q, out, lse = _layer_inputs(rng, n)
    table = torch.full_like(c.block_table, -1)
    seq, pos = torch.full((n,), -1, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
    idx = torch.zeros(n, 96, dtype=torch.int32, device="cuda")
    cnt = torch.zeros(n, dtype=torch.int32, device="cuda")
    ws = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, n, 2, max_len)

    def layer():
        lsa.fp8_forward(cfg, seq, pos, max_len, q_idx, w, c.key_pages, q, c.latent_pages, table, out, lse, ws, idx_out=idx,
                        count_out=cnt)

    layer()                                              # all padding
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer()
    for step in range(3):
        s = np.sort(rng.integers(-1, 2, n))[::-1].copy()
        p = np.array([rng.integers(0, c.lens[k]) if k >= 0 else -1 for k in s])
        seq.copy_(_i32(s)); pos.copy_(_i32(p)); table.copy_(c.block_table)
        idx.fill_(-9)
        g.replay()
        assert lsa.device_error() == 0
        got, got_idx = [o.clone() for o in out], idx.clone()
        layer()
        assert lsa.device_error() == 0
        assert torch.equal(got_idx.sort(dim=1).values, idx.sort(dim=1).values)
        for r in range(n):
            assert int(cnt[r]) == (min(p[r] + 1, 96) if s[r] >= 0 else 0)
            if torch.equal(got_idx[r], idx[r]):          # sums in the same order: the same bits
                assert all(torch.equal(a[r], b[r]) for a, b in zip(got, out))
    del g


@gpu
def test_two_calls_at_once_on_two_streams():
    cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    calls = []
    for k, (n, max_len) in enumerate([(66, 60000), (3, 900)]):
        c = Caches([300, 900], 51 + k, cli=2)
        rng = np.random.default_rng(61 + k)
        q_idx, w, q, out, lse = _layer_inputs(rng, n)
        seq, pos = _i32(np.arange(n) % 2), _i32(rng.integers(100, 300, n))
        idx, cnt = torch.zeros(n, 96, dtype=torch.int32, device="cuda"), torch.zeros(n, dtype=torch.int32, device="cuda")
        ws = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, n, 2, max_len)
        calls.append((lambda st, a=(cfg, seq, pos, max_len, q_idx, w, c.key_pages, q, c.latent_pages, c.block_table, out,
                                    lse, ws), i=idx, t=cnt: lsa.fp8_forward(*a, idx_out=i, count_out=t, stream=st), out, idx))
    want = []
    for f, out, idx in calls:
        f(None)
        torch.cuda.synchronize()
        want.append(([o.clone() for o in out], idx.clone()))
    streams = [torch.cuda.Stream() for _ in calls]
    for _ in range(5):
        for (f, out, idx), st in zip(calls, streams):
            f(st)
    torch.cuda.synchronize()
    assert lsa.device_error() == 0
    for (f, out, idx), (o0, i0) in zip(calls, want):
        assert torch.equal(idx.sort(dim=1).values, i0.sort(dim=1).values)
        for r in range(idx.shape[0]):
            if torch.equal(idx[r], i0[r]):
                assert all(torch.equal(a[r], b[r]) for a, b in zip(out, o0))


@gpu
@pytest.mark.parametrize("max_len", [300, 60000])     # the indexer's two forms
def test_forward_padding_rows_with_any_position_select_nothing(max_len):
    rng = np.random.default_rng(31)
    cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    c = Caches([300], 32, cli=2)
    n = 70
    seq, pos = np.zeros(n, dtype=np.int64), 230 + np.arange(n)
    seq[[0, 20, 21, 69]], seq[40] = -1, 9            # padding rows with positions that look real; an unknown sequence
    q_idx, w, q, out, lse = _layer_inputs(rng, n)
    for o in out:
        o.fill_(9.0)
    idx = torch.full((n, 96), -7, dtype=torch.int32, device="cuda")
    cnt = torch.full((n,), -7, dtype=torch.int32, device="cuda")
    ws = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, n, 1, max_len)
    lsa.fp8_forward(cfg, _i32(seq), _i32(pos), max_len, q_idx, w, c.key_pages, q, c.latent_pages, c.block_table, out,
                    lse, ws, idx_out=idx, count_out=cnt)
    assert lsa.device_error() == lsa.DEVERR_SEQ
    for r in range(n):
        if seq[r] != 0:
            assert int(cnt[r]) == 0 and (idx[r] == -1).all()
            assert (out[0][r] == (9.0 if seq[r] == -1 else 0.0)).all()
        else:
            assert int(cnt[r]) == 96 and len(set(idx[r].tolist())) == 96 and 0 <= int(idx[r].min()) <= int(idx[r].max()) <= pos[r]
            assert torch.isfinite(out[0][r]).all() and not (out[0][r] == 9.0).all()


@gpu
def test_forward_dense_small_workspace_and_split_rows():
    rng = np.random.default_rng(22)
    lens = [90, 60]
    c = Caches(lens, 17, cli=2)
    cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
    q_idx, w, q, out, lse = _layer_inputs(rng, 2)
    # max_len <= topk: no index pass, no key pages needed
    lsa.fp8_forward(cfg, None, _i32([89, 59]), 90, None, None, None, q, c.latent_pages, c.block_table, out, lse, None)
    assert lsa.device_error() == 0
    for r, n in enumerate(lens):
        o, l, wt = F.attend(_vals(q[1])[r], c.lat[1][r], range(n), cfg.softmax_scale)
        tol, _ = _mla_tol(_vals(q[1])[r], c.lat[1][r], c.lat_s[1][r], range(n), wt, o, cfg.softmax_scale)
        assert (np.abs(_vals(out[1])[r] - o) <= tol).all()
    # a workspace of fewer rows than the call has: the same results, block by block, with and without a row map
    lens = [150, 300, 220, 97, 260]
    c = Caches(lens, 18, cli=2)
    q_idx, w, q, out, lse = _layer_inputs(rng, 5)
    pos, seq = _i32([n - 1 for n in lens]), _i32(range(5))
    full = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, 5, 5, 300)
    small = lsa.workspace(cfg, lsa.OP_FP8_FORWARD, 2, 5, 300)
    assert small.numel() < full.numel()
    got = []
    for sq, ws in ((seq, full), (None, full), (seq, small), (None, small)):
        o = [torch.zeros_like(x) for x in out]
        ix, cn = torch.zeros(5, 96, dtype=torch.int32, device="cuda"), torch.zeros(5, dtype=torch.int32, device="cuda")
        lsa.fp8_forward(cfg, sq, pos, 300, q_idx, w, c.key_pages, q, c.latent_pages, c.block_table, o, lse, ws, idx_out=ix,
                        count_out=cn)
        assert lsa.device_error() == 0
        got.append((o, ix.sort(1)[0]))
    for o, ix in got[1:]:
        assert torch.equal(ix, got[0][1])
        for a, b in zip(o, got[0][0]):
            assert (a.float() - b.float()).abs().max() <= 2.0 ** -6 * b.float().abs().max()


# ------------------------------------------------------------------ GPU: the attention's frames at their ends


def _sequence(lat, seed=0):
    """One sequence holding these latent rows (bf16 [n, 576]), put there by the append."""
    n = len(lat)
    c = Caches([n], seed, cli=1)
    t = torch.arange(n, device="cuda")
    slot = (torch.from_numpy(c.table[0]).cuda()[t // 64] * 64 + t % 64).int()
    lsa.fp8_append(lsa.LsaConfig(cli_factor=1), slot, [lat.cuda()], c.latent_pages)
    codes, s = F.quant(_vals(lat))
    c.lat[0][0], c.lat_s[0][0] = F.dequant(codes, s), s
    return c


def _attend_list(c, q, keys, ws):
    """The attention of one row (q bf16 [32, 576]) over its list, in this order; checked against the oracle."""
    cfg, n = lsa.LsaConfig(cli_factor=1), c.lens[0]
    idx = _i32(np.concatenate([keys, np.full(2048 - len(keys), -1)])[None])
    out = [torch.full((1, 32, 512), 9.0, dtype=torch.bfloat16, device="cuda")]
    lse = [torch.full((1, 32), 9.0, device="cuda")]
    w = lsa.workspace(cfg, lsa.OP_FP8_MLA, 1, 1, n) if ws else None
    lsa.fp8_sparse_mla(cfg, None, _i32([n - 1]), [q[None].cuda()], c.latent_pages, c.block_table, idx, _i32([len(keys)]),
                       n, out, lse, w)
    assert lsa.device_error() == 0
    want, wl, wt = F.attend(_vals(q), c.lat[0][0], keys, cfg.softmax_scale)
    tol, ltol = _mla_tol(_vals(q), c.lat[0][0], c.lat_s[0][0], keys, wt, want, cfg.softmax_scale)
    o, l = _vals(out[0])[0], lse[0][0].double().cpu().numpy()
    assert (np.abs(l - wl) <= ltol).all()
    assert (np.abs(o - want) <= tol).all()
    return o


@gpu
@pytest.mark.parametrize("ws", [False, True])      # one split, or several
@pytest.mark.parametrize("n,zero_at", [(2, 0), (2, 1), (90, 40), (700, 0), (700, 650)])
@pytest.mark.parametrize("amp,logit", [(1000.0, -41000.0), (2000.0, -139.0), (1e30, -400.0)])
def test_mla_a_row_of_zeros_above_rows_of_large_scale(ws, n, zero_at, amp, logit):
    # the row of zeros has the whole weight and every other row's is zero in fp32, beside a scale of up to 2^91
    rng = np.random.default_rng(n + zero_at)
    lat = _bf16(amp * rng.uniform(0.9, 1.0, (n, 576)))
    lat[zero_at] = 0
    q = _bf16(np.full((32, 576), logit * 192 ** 0.5 / (576 * 0.95 * amp)))
    c = _sequence(lat)
    o = _attend_list(c, q, np.arange(n), ws)
    assert (np.abs(o) <= 1e-20 * amp).all()


@gpu
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("top", [400.0 * 2.0 ** -126, 440.0 * 2.0 ** -125, 2.0 ** -60])
def test_mla_rows_of_the_smallest_scales(ws, top):
    # among many of their kind, and alone: one key's values come out exactly
    rng = np.random.default_rng(5)
    lat = _bf16(rng.uniform(-top, top, (300, 576)))
    lat[:, 0] = top
    c = _sequence(lat)
    assert (c.lat_s[0][0] == (2.0 ** -68 if top == 2.0 ** -60 else 2.0 ** -126 if top < 448 * 2.0 ** -126 else 2.0 ** -125)).all()
    q = _bf16(rng.standard_normal((32, 576)))
    _attend_list(c, q, np.arange(300), ws)
    for k in (0, 131, 299):
        o = _attend_list(c, q, np.array([k]), ws)
        normal = np.abs(c.lat[0][0][k, :512]) >= 2.0 ** -126
        assert normal.sum() > 500 and (o[:, normal] == c.lat[0][0][k, :512][normal]).all()


@gpu
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("loud,zeros,after,logit", [(128, 1, 0, -50.0), (128, 128, 128, -50.0), (256, 200, 300, -45.0),
                                                    (2048 - 128, 128, 0, -60.0), (128 * 15, 127, 1, -80.0)])
def test_mla_tiles_of_zero_rows_move_the_sums_and_the_output_alike(ws, loud, zeros, after, logit):
    # the maximum rises by far more than 2^60 in a tile whose rows are all zeros: what was summed so far falls with it
    rng = np.random.default_rng(loud)
    n = loud + zeros + after
    lat = _bf16(rng.uniform(0.5, 1.0, (n, 576)))
    lat[loud:loud + zeros] = 0
    q = _bf16(np.full((32, 576), logit * 192 ** 0.5 / (576 * 0.75)))
    c = _sequence(lat)
    o = _attend_list(c, q, np.arange(n), ws)
    assert (np.abs(o) <= 1e-14).all()


@gpu
def test_mla_a_new_frame_on_a_tile_of_zero_rows():
    # every 16 tiles the frame is set anew, here (the 17th) from rows of zeros alone, 2^23 above what came before
    rng = np.random.default_rng(7)
    n = 18 * 128
    lat = _bf16(rng.uniform(0.5, 1.0, (n, 576)))
    lat[16 * 128:17 * 128] = 0
    q = _bf16(np.full((32, 576), -16.0 * 192 ** 0.5 / (576 * 0.75)))
    c = _sequence(lat)
    cfg = lsa.LsaConfig(cli_factor=1)
    out, lse = [torch.empty(1, 32, 512, dtype=torch.bfloat16, device="cuda")], [torch.empty(1, 32, device="cuda")]
    lsa.fp8_sparse_mla(cfg, None, _i32([n - 1]), [q[None].cuda()], c.latent_pages, c.block_table, None, None, n, out, lse,
                       None)
    assert lsa.device_error() == 0
    want, wl, wt = F.attend(_vals(q), c.lat[0][0], range(n), cfg.softmax_scale)
    assert want.max() < 1e-4
    tol, ltol = _mla_tol(_vals(q), c.lat[0][0], c.lat_s[0][0], range(n), wt, want, cfg.softmax_scale)
    assert (np.abs(lse[0][0].double().cpu().numpy() - wl) <= ltol).all()
    assert (np.abs(_vals(out[0])[0] - want) <= tol).all()


@gpu
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("amp", [3e3, 1e5, 1e9, 1e15])
def test_mla_logits_whose_fp32_steps_are_whole_binades(ws, sign, amp):
    # logits from 2^24 to 2^100: an exponent added to one is lost in it. One key's values stay exact, and among many
    # the best one's stand alone (its lead is far above the logits' rounding)
    rng = np.random.default_rng(77)
    lat = _bf16(rng.standard_normal((300, 576)) * 3 + sign * 2.0) * amp
    lat = lat.bfloat16()
    q = (_bf16(rng.uniform(0.5, 1.5, (32, 576))) * amp).bfloat16()
    c = _sequence(lat)
    v = c.lat[0][0][:, :512]
    for k in (0, 131, 299):
        assert (_attend_list(c, q, np.array([k]), ws) == v[k]).all()
    x = lsa.LsaConfig().softmax_scale * (_vals(q) @ c.lat[0][0].T)
    for keys in (np.arange(300), np.argsort(x[5])):
        o = _attend_list(c, q, keys, ws)
        lead = np.sort(x, axis=1)
        clear = lead[:, -1] - lead[:, -2] > 2.0 ** -10 * np.abs(lead).max()
        assert clear.any() and (o[clear] == v[x.argmax(1)][clear]).all()


@gpu
@pytest.mark.parametrize("ws", [False, True])
def test_mla_partials_of_the_largest_values_stay_finite(ws):
    # values near bf16's largest: the sum over a split's keys is infinite in fp32 unless it is divided by its weights
    rng = np.random.default_rng(9)
    lat = _bf16(rng.uniform(2e38, 3e38, (700, 576)))
    q = _bf16(rng.standard_normal((32, 576)) * 1e-38)
    c = _sequence(lat)
    assert (c.lat_s[0][0] == 2.0 ** 120).mean() > 0.9 and c.lat[0][0].max() < 2.0 ** 128
    _attend_list(c, q, np.arange(700), ws)
    o = _attend_list(c, q, np.array([5]), ws)
    assert (o == c.lat[0][0][5, :512]).all()


@gpu
@pytest.mark.parametrize("bound", [400, 60000])     # the kernel's two forms
def test_scores_histogram_of_rows_without_a_sequence_or_past_their_table(bound):
    # positions that look real beside no sequence count nothing; one past the table counts what the row sees
    cfg = lsa.LsaConfig(**TINY)
    c = Caches([300, 150], 3)
    rows = [(s, p) for s, n in enumerate(c.lens) for p in range(n - 30, n)]
    rows[5:5] = [(-1, 250), (2, 250), (-9, 299), (0, 350), (-1, 2 ** 31 - 1), (0, -4)]
    rows += [(-1, 120), (-1, 299)]
    n = len(rows)
    rng = np.random.default_rng(4)
    q = _bf16(rng.standard_normal((n, 32, 128))).cuda()
    w = torch.from_numpy(rng.standard_normal((n, 32)).astype(np.float32)).cuda()
    scores = torch.full((n, bound), 7.0, device="cuda")
    h = lsa.topk_hist_buffer(n)
    ws = lsa.workspace(cfg, lsa.OP_FP8_INDEX, n, 2, bound)
    for _ in range(2):
        h.fill_(3)
        lsa.fp8_index_scores(cfg, _i32([r[0] for r in rows]), _i32([r[1] for r in rows]), q, w, c.key_pages, c.block_table,
                             bound, scores, ws, topk_hist=h)
        assert lsa.device_error() == lsa.DEVERR_SEQ | lsa.DEVERR_POS
    room = c.table.shape[1] * 64
    assert room == 320
    seen = [(-1 if s not in (0, 1) or p < 0 else s, min(p, room - 1)) for s, p in rows]
    for r, (s, p) in enumerate(seen):
        assert (scores[r, p + 1 if s >= 0 else 0:] == 7.0).all()
    _check_hist(seen, scores, h, cfg)


@gpu
def test_page_plan_at_the_largest_lengths():
    # a table wider than any pool: lengths go up to 2^31 - 64, and what is longer is refused like any other
    width, most = 2 ** 25 + 1, 2 ** 31 - 64
    bt = torch.full((3, width), -1, dtype=torch.int32, device="cuda")
    bt[0, 2 ** 25 - 2], bt[2, 0] = 7, 3
    cached, fresh = [most - 2, 2 ** 31 - 10, 3], [2, 5, 62]
    free = [11, 12]
    seq, pos, slot, totals = (_i32([55] * k) for k in (66, 66, 66, 2))
    lsa.page_plan(_i32(cached), _i32(fresh), _i32(free), bt, seq, pos, slot, totals)
    assert lsa.device_error() == lsa.DEVERR_POS
    assert totals.tolist() == [64, 1]
    assert seq.tolist() == [0] * 2 + [2] * 62 + [-1] * 2
    assert pos.tolist() == [most - 2, most - 1] + list(range(3, 65)) + [-1] * 2
    assert slot.tolist() == [7 * 64 + 62, 7 * 64 + 63] + [3 * 64 + i for i in range(3, 64)] + [11 * 64, -1, -1]
    assert int(bt[2, 1]) == 11 and int((bt != -1).sum()) == 3
    # the request that is one token too long for 32-bit columns
    lsa.page_plan(_i32([most]), _i32([1]), _i32(free), bt[:1], seq, pos, slot, totals)
    assert lsa.device_error() == lsa.DEVERR_POS and totals.tolist() == [0, 0] and int((bt != -1).sum()) == 3


def test_barrier_operations_order_plain_accesses():
    # published and consumed shared data are plain accesses: every arrival and wait is a barrier for the compiler too
    import re
    from pathlib import Path

    src = (Path(lsa.__file__).parent / "csrc" / "tc.cuh").read_text()
    for name in ("mbar_expect_tx", "mbar_arrive", "mbar_try_wait", "mbar_test"):
        body = re.search(rf"\b{name}\(uint64_t\* bar.*?\n}}\n", src, re.S).group(0)
        assert '"memory"' in body, name


# ------------------------------------------------------------------ GPU: layers at once and replayed, every row checked


class _Layer:
    """A layer call over sequences of its own, its outputs poisoned before each run."""

    def __init__(self, seed, n, max_len, lens):
        self.cfg = lsa.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
        self.c = Caches(lens, seed, cli=2)
        self.rng = np.random.default_rng(seed + 1)
        self.n, self.max_len = n, max_len
        self.q_idx, self.w, self.q, self.out, self.lse = _layer_inputs(self.rng, n)
        self.seq, self.pos = (torch.empty(n, dtype=torch.int32, device="cuda") for _ in range(2))
        self.idx = torch.empty(n, 96, dtype=torch.int32, device="cuda")
        self.cnt = torch.empty(n, dtype=torch.int32, device="cuda")
        self.ws = lsa.workspace(self.cfg, lsa.OP_FP8_FORWARD, n, len(lens), max_len)

    def new_rows(self):
        s = np.sort(self.rng.integers(-1, len(self.c.lens), self.n))[::-1].copy()
        self.seq.copy_(_i32(s))
        self.pos.copy_(_i32([self.rng.integers(0, self.c.lens[k]) if k >= 0 else -1 for k in s]))
        for x in (self.q_idx, *self.q):
            x.copy_(_bf16(self.rng.standard_normal(tuple(x.shape))))

    def poison(self):
        for t in (*self.out, *self.lse):
            t.fill_(9.0)
        self.idx.fill_(-9)
        self.cnt.fill_(-9)
        self.ws.fill_(0xFF)

    def run(self):
        lsa.fp8_forward(self.cfg, self.seq, self.pos, self.max_len, self.q_idx, self.w, self.c.key_pages, self.q,
                        self.c.latent_pages, self.c.block_table, self.out, self.lse, self.ws, idx_out=self.idx,
                        count_out=self.cnt)

    def check(self):
        ocfg = R.LsaConfig(index_topk=96, index_init_tokens=4, index_local_tokens=16)
        seq, pos, idx, cnt = (t.cpu().numpy() for t in (self.seq, self.pos, self.idx, self.cnt))
        qi, w = _vals(self.q_idx), self.w.double().cpu().numpy()
        q, out, lse = ([_vals(t) for t in ts] for ts in (self.q, self.out, self.lse))
        for r, (s, p) in enumerate(zip(seq, pos)):
            if s < 0:
                assert cnt[r] == 0 and (idx[r] == -1).all()
                assert all((o[r] == 9.0).all() for o in out) and all((l[r] == 9.0).all() for l in lse)
                continue
            sel = idx[r, :cnt[r]]
            assert len(set(sel.tolist())) == cnt[r] == min(p + 1, 96) and sel.min() >= 0 and sel.max() <= p
            want_idx, gap = R.select_topk(F.score_row(qi[r], w[r], self.c.keys[s], p, ocfg), p, ocfg)
            if p + 1 > 96 and gap is not None and gap > 1e-4:
                np.testing.assert_array_equal(np.sort(sel), np.sort(want_idx))
            for z in range(2):
                o, l, wt = F.attend(q[z][r], self.c.lat[z][s], sel, self.cfg.softmax_scale)
                tol, ltol = _mla_tol(q[z][r], self.c.lat[z][s], self.c.lat_s[z][s], sel, wt, o, self.cfg.softmax_scale)
                assert (np.abs(lse[z][r] - l) <= ltol).all()
                assert (np.abs(out[z][r] - o) <= tol).all()


@gpu
def test_layers_at_once_write_every_row():
    layers = [_Layer(71, 66, 60000, [300, 900]), _Layer(74, 3, 900, [900, 130]), _Layer(77, 40, 400, [400, 17, 250])]
    streams = [torch.cuda.Stream() for _ in layers]
    for _ in range(3):
        for a in layers:
            a.new_rows()
            a.poison()
        torch.cuda.synchronize()
        for _ in range(3):
            for a, st in zip(layers, streams):
                with torch.cuda.stream(st):
                    a.poison()
                    a.run()
        torch.cuda.synchronize()
        assert lsa.device_error() == 0
        for a in layers:
            a.check()


@gpu
@pytest.mark.parametrize("max_len", [300, 60000])     # the indexer's two forms
def test_replayed_layers_write_every_row(max_len):
    # two captured layers, replayed in turn with new rows and queries in place: nothing stands from an earlier run
    layers = [_Layer(81, 66, max_len, [300, 260]), _Layer(84, 5, max_len, [300, 90])]
    graphs = []
    for a in layers:
        a.new_rows()
        a.run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            a.run()
        graphs.append(g)
    for _ in range(3):
        for a, g in zip(layers, graphs):
            a.new_rows()
            a.poison()
            g.replay()
        torch.cuda.synchronize()
        assert lsa.device_error() == 0
        for a in layers:
            a.check()
    del graphs, g


# ------------------------------------------------------------------ GPU: rows that one key dominates, slots never filled


@gpu
@pytest.mark.parametrize("ws", [False, True])
@pytest.mark.parametrize("weight", [0.9, 0.99, 0.999])
@pytest.mark.parametrize("along", [20.0, 2.0])        # the sink's scale: half of the other rows', or eight times it
def test_mla_rows_that_a_sink_dominates(ws, weight, along):
    # the other keys' weights lie 2^-14 to 2^-21 below the sink's, where the steps of a weight's code (2^-16 of the
    # largest weight * scale and coarser) are of their own size: the error stays within those steps' sum
    rng = np.random.default_rng(int(weight * 1000))
    n = 2048
    u = rng.standard_normal(576)
    u /= np.linalg.norm(u)
    q = _bf16(along * u + 0.2 * rng.standard_normal((32, 576)))
    x = rng.standard_normal((n, 576))
    x[1:] -= np.outer(x[1:] @ u, u)                    # the others have no part in the heads' common direction
    x[0] = u * (np.log(weight / (1 - weight)) + np.log(n - 1)) * 192 ** 0.5 / along
    c = _sequence(_bf16(x))
    o = _attend_list(c, q, np.arange(n), ws)
    _, _, wt = F.attend(_vals(q), c.lat[0][0], range(n), lsa.LsaConfig().softmax_scale)
    # (the case is what it says: heads differ by their own parts' products with the sink)
    assert abs(np.median(np.log(wt[:, 0] / (1 - wt[:, 0]))) - np.log(weight / (1 - weight))) < 1
    assert np.isfinite(o).all()


@gpu
def test_slots_that_were_never_filled_hold_no_key():
    # a scale of 0 stands in no appended row: the attention skips it, the indexer's score of it is 0
    c = Caches([200], 91, cli=1)
    slots = c.slots(0, 200)
    for k in (3, 64, 130):
        c.latent_pages[0].view(-1, F.LAT_ROW)[slots[k]] = 0
        c.key_pages.view(torch.float32)[slots[k] // 64, 2048 + slots[k] % 64] = 0
    cfg = lsa.LsaConfig(index_topk=64, index_init_tokens=1, index_local_tokens=2, cli_factor=1)
    lists = [[3, 64, 130], [2, 3, 4, 64, 199], list(range(60, 120))]
    _mla_case(c, [(0, 199)] * 3, lists, cfg, keep=lambda s, k: k not in (3, 64, 130))
    q = _bf16(np.random.default_rng(1).standard_normal((1, 32, 128))).cuda()
    scores, w = torch.full((1, 200), 7.0, device="cuda"), torch.ones(1, 32, device="cuda")
    lsa.fp8_index_scores(cfg, None, _i32([199]), q, w, c.key_pages, c.block_table, 200, scores,
                         lsa.workspace(cfg, lsa.OP_FP8_INDEX, 1, 1, 200))
    assert lsa.device_error() == 0
    assert scores[0, [3, 64, 130]].tolist() == [0.0] * 3 and bool((scores[0] != 7.0).all())
