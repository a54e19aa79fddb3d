"""Attention over an 8-bit pool whose scales the library's own store does not write: zeros, subnormal
numbers and runs of entries outside the pool.  Bounds as in test_kv_q8_gpu; a key of V scale 0 has no
part in them but in the sum of the softmax."""
import numpy as np
import pytest
import torch

from oracle import attention as A, quantised as Q
from prefix_shared_kv_gb300 import rx
from prefix_shared_kv_gb300.session import bits_of
from test_kv_q8_gpu import (DEC_ERR, EXT_ERR, Pool, check_decode, check_extend, extend_case,
                            random_table, run_decode, run_extend)

pytestmark = pytest.mark.gpu

ZEROED = ["zero", "subnormal", "outside"]


def level(pool):
    """Scores within a few powers of two of one another: no later key stands out."""
    pool.ks *= np.float32(0.25)


def drop_v(pool, table_rows, first, last, how):
    """Keys first .. last - 1 of the requests in `table_rows` (which share them) without a V."""
    at = pool.table[table_rows[0], first:last]
    if how == "outside":
        for r in table_rows:
            pool.table[r, first:last] = -1
    else:
        pool.vs[at] = 0.0 if how == "zero" else np.float32(2.0 ** -130)


def crowded(cuda, rng, hq, hkv, lens, gone, how, shared=None):
    """A pool of 2,400 slots over which many requests' tables run, so that items are several steps
    long: each request (or, in `shared`, each group's prefix) begins with gone[b] slots without V."""
    without, n = 400, 2400
    pool = Pool(cuda, rng, hq, hkv, n, np.zeros((len(lens), max(lens)), np.int32))
    level(pool)
    pool.vs[:without] = 0.0 if how == "zero" else np.float32(2.0 ** -130)

    def row(length, first):
        first = min(first, length)
        head = np.full(first, -1) if how == "outside" else rng.permutation(without)[:first]
        return np.concatenate([head, without + rng.permutation(n - without)[:length - first]])

    for b, length in enumerate(lens):
        pool.table[b, :length] = row(length, 0 if shared else gone[b])
    for members, prefix, first in shared or ():
        pool.table[list(members), :prefix] = row(prefix, first)
    pool.upload()
    return pool


@pytest.mark.parametrize("how", ZEROED)
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 2), (8, 2), (8, 8), (32, 8), (6, 3), (8, 1)])
def test_decode_of_requests_that_begin_without_v(cuda, hq, hkv, how):
    """The first 32 (one warp's first step), 64, 256, 300 or all keys of a request have no V."""
    rng = np.random.default_rng(100 + hq + hkv)
    gone = ([32, 64, 300, 400, 0, 256] * 60)[:1200 // hkv + 100]
    lens = [400 if g == 400 else int(x)
            for g, x in zip(gone, rng.integers(1200, 2000, len(gone)))]
    pool = crowded(cuda, rng, hq, hkv, lens, gone, how)
    q, o, lse, ws, _ = run_decode(pool, rng, lens)
    assert rx.read_status(ws) == (rx.RX_ERR_RANGE if how == "outside" else rx.RX_OK)
    check_decode(pool, q, o, lse, lens, range(8))
    if how != "subnormal":
        assert (o[3] == 0).all()


@pytest.mark.parametrize("how", ["zero", "outside"])
@pytest.mark.parametrize("hq,hkv,members", [(8, 8, 12), (16, 2, 6), (8, 1, 5), (4, 4, 40),
                                            (32, 8, 16)])
def test_decode_of_shared_prefixes_that_begin_without_v(cuda, hq, hkv, members, how):
    """Groups of 10 to 64 rows a KV head: the narrow and the wide form, whole and split stages."""
    rng = np.random.default_rng(200 + hq + hkv + members)
    groups = 100 if hkv < 4 else 30
    first = [32, 300, 64, 0, 256] * (groups // 5)
    shared = [(range(g * members, (g + 1) * members), 1500, first[g]) for g in range(groups)]
    lens = [1500 + int(x) for x in rng.integers(0, 20, groups * members)]
    pool = crowded(cuda, rng, hq, hkv, lens, None, how, shared)
    q, o, lse, ws, _ = run_decode(pool, rng, lens, np.repeat(np.arange(groups), members),
                                  [1500] * groups)
    assert rx.read_status(ws) == (rx.RX_ERR_RANGE if how == "outside" else rx.RX_OK)
    check_decode(pool, q, o, lse, lens, [0, members - 1, members, 2 * members + 1, 4 * members])


@pytest.mark.parametrize("how", ZEROED)
def test_decode_without_v_in_the_middle_and_in_turns(cuda, how):
    rng = np.random.default_rng(300)
    lens = [900, 900]
    pool = Pool(cuda, rng, 8, 2, 2000, random_table(rng, 2000, lens))
    level(pool)
    drop_v(pool, [0], 200, 700, how)
    for k in range(0, 900, 64):
        drop_v(pool, [1], k, k + 32, how)
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens)
    check_decode(pool, q, o, lse, lens)


@pytest.mark.parametrize("how", ZEROED)
@pytest.mark.parametrize("hq,hkv,new", [(32, 8, [1, 1]), (48, 12, [2, 3]), (8, 1, [1, 2])])
def test_extend_of_few_new_tokens_that_begins_without_v(cuda, hq, hkv, new, how):
    """Plans that run as a decode."""
    prefix = [3000, 2500]
    rng, pool, _, _ = extend_case(cuda, 400 + hq, hq, hkv, prefix, new)
    level(pool)
    drop_v(pool, [0], 0, 32, how)
    drop_v(pool, [1], 0, 300, how)
    pool.upload()
    q, o, lse, ws = run_extend(pool, rng, prefix, new)
    assert ws.numel() < sum(prefix) * hkv * 522  # no expanded keys
    check_extend(pool, q, o, lse, prefix, new)


@pytest.mark.parametrize("how", ZEROED)
def test_extend_on_tiles_that_begins_without_v(cuda, how):
    prefix, new = [500, 40], [200, 90]
    rng, pool, _, _ = extend_case(cuda, 500, 8, 2, prefix, new)
    drop_v(pool, [0], 0, 300, how)
    drop_v(pool, [1], 0, 32, how)
    pool.upload()
    q, o, lse, ws = run_extend(pool, rng, prefix, new)
    check_extend(pool, q, o, lse, prefix, new)


class Signed(Pool):
    """A pool with V scales of either sign: the bounds go by their magnitude."""

    def rows(self, at):
        K, V, vs = super().rows(at)
        return K, V, np.abs(vs)


@pytest.mark.parametrize("signs", ["all negative", "mixed", "negative and large behind the first"])
@pytest.mark.parametrize("hq,hkv,members", [(8, 2, 1), (32, 8, 3), (32, 8, 16), (4, 4, 40), (8, 1, 20)])
def test_decode_of_negative_v_scales(cuda, hq, hkv, members, signs):
    rng = np.random.default_rng(600 + hq + members)
    prefix = 700
    lens = [prefix + 5 * b for b in range(members)] + [300]
    n = prefix + sum(lens) + 10
    pool = Signed(cuda, rng, hq, hkv, n, random_table(rng, n, lens, {0: (list(range(members)), prefix)}))
    level(pool)
    if signs == "all negative":
        pool.vs = -pool.vs
    elif signs == "mixed":
        pool.vs *= np.where(rng.random(pool.vs.shape) < 0.5, 1, -1).astype(np.float32)
    else:
        for b in (0, members):
            pool.vs[pool.table[b, 40:prefix if b < members else 300]] *= np.float32(-2.0 ** 30)
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens, [0] * members + [-1], [prefix])
    # 160 rows a KV head run on the extend's kernel, whose weights are bf16: 2^-8, not 2^-11, of a
    # weight (derived at the head of test_kv_q8_gpu)
    check_decode(pool, q, o, lse, lens, [0, members - 1, members],
                 EXT_ERR if members * hq // hkv > 128 else DEC_ERR)


def test_extend_of_negative_scales(cuda):
    """K scales too, on tiles and as a decode of few tokens."""
    for prefix, new in (([500, 40], [200, 90]), ([3000, 2500], [1, 2])):
        lens = [p + e for p, e in zip(prefix, new)]
        rng = np.random.default_rng(700 + sum(new))
        n = sum(lens) + 20
        pool = Signed(cuda, rng, 32, 8, n, random_table(rng, n, lens))
        pool.vs *= np.where(rng.random(pool.vs.shape) < 0.5, 1, -1).astype(np.float32)
        pool.ks *= np.where(rng.random(pool.ks.shape) < 0.5, 1, -1).astype(np.float32)
        pool.upload()
        q, o, lse, ws = run_extend(pool, rng, prefix, new)
        check_extend(pool, q, o, lse, prefix, new)


FORMS = [  # an extend on whole tiles (shared and own keys), with split keys, with cut items
    (8, 4, [100, 100, 30], [70, 20, 40], [(range(2), 100)]),
    (8, 2, [1000] * 4, [40] * 4, [(range(4), 1000)]),
    (24, 3, [2500], [830], [])]


@pytest.mark.parametrize("scale", [np.inf, -np.inf, np.nan])
@pytest.mark.parametrize("hq,hkv,prefix,new,groups", FORMS)
def test_extend_scales_of_keys_a_row_does_not_see_do_not_reach_it(cuda, hq, hkv, prefix, new, groups,
                                                                  scale):
    """The last new token of request 0 and a middle one of the last request have scales that are not
    finite: the rows before them, and the other requests' rows, are as before, bit for bit."""
    rng, pool, grp, gpl = extend_case(cuda, 800 + hq + sum(new), hq, hkv, prefix, new, groups)
    q, o, lse, ws = run_extend(pool, rng, prefix, new, grp, gpl)
    check_extend(pool, q, o, lse, prefix, new)
    last = len(new) - 1
    mid = new[last] // 2
    pool.vs[pool.table[0, prefix[0] + new[0] - 1]] = scale
    pool.vs[pool.table[last, prefix[last] + mid]] = scale
    pool.upload()
    _, o2, lse2, _ = run_extend(pool, rng, prefix, new, grp, gpl, q=q)
    sees = torch.zeros(len(o), dtype=torch.bool)
    sees[new[0] - 1] = True
    sees[len(o) - new[last] + mid:] = True
    assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2, lse)
    assert not torch.isfinite(o2[sees].float()).any()  # (code 0 of such a key: 0 * inf, NaN)
    pool.vs[pool.table[0, prefix[0] + new[0] - 1]] = 1
    pool.vs[pool.table[last, prefix[last] + mid]] = 1
    pool.ks[pool.table[0, prefix[0] + new[0] - 1]] = scale
    pool.ks[pool.table[last, prefix[last] + mid]] = scale
    pool.upload()
    _, o2, lse2, _ = run_extend(pool, rng, prefix, new, grp, gpl, q=q)
    assert torch.equal(o2[~sees], o[~sees]) and torch.equal(lse2[~sees], lse[~sees])


@pytest.mark.parametrize("bad", [-2 ** 31, -2 ** 31 + 1, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("hq,hkv,members", [(8, 2, 1), (32, 8, 16), (8, 1, 20)])
def test_decode_flags_every_entry_outside_the_pool(cuda, hq, hkv, members, bad):
    """The narrow, the wide and the tile form; no entry stands for "no key"."""
    rng = np.random.default_rng(900 + members)
    lens = [200 + b for b in range(members)]
    n = 200 + sum(lens) + 10
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens, {0: (list(range(members)), 200)}))
    pool.table[:, 133] = bad
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens, [0] * members, [200])
    assert rx.read_status(ws) == rx.RX_ERR_RANGE and rx.read_status(ws) == rx.RX_OK
    check_decode(pool, q, o, lse, lens, [0, members - 1],
                 EXT_ERR if members * hq // hkv > 128 else DEC_ERR)


@pytest.mark.parametrize("size", [90, 101, 120])
@pytest.mark.parametrize("hq,hkv,members", [(8, 2, 1), (32, 8, 16), (8, 1, 20)])
def test_decode_of_scores_far_below_zero(cuda, hq, hkv, members, size):
    """Scores of -2^size and keys at twice that, which weigh nothing, in either order: large K rows that
    point away from the query."""
    rng = np.random.default_rng(1000 + members)
    n_keys = 400
    lens = [n_keys] * members + [n_keys, 40]
    n = sum(lens) + 10
    pool = Pool(cuda, rng, hq, hkv, n,
                random_table(rng, n, lens, {0: (list(range(members)), n_keys)}))
    pool.scale = 0.125
    pool.kc[:], pool.ks[:] = 0, np.float32(2.0 ** (size + 3))
    pool.kc[:, :, 0] = 0xB8                                   # -1
    pool.kc[pool.table[0, 200:n_keys], :, 0] = 0xC0           # -2: of no weight
    pool.kc[pool.table[members, :200], :, 0] = 0xC0
    pool.upload()
    q = np.zeros((len(lens), hq, 128), np.uint16)
    q[:, :, 0] = 0x3F80                                       # 1
    q, o, lse, ws, _ = run_decode(pool, rng, lens, [0] * members + [-1, -1], [n_keys], q=q)
    assert rx.read_status(ws) == rx.RX_OK
    for b, seen in ((0, range(200)), (members - 1, range(200)), (members, range(200, n_keys)),
                    (members + 1, range(40))):
        at = pool.table[b, list(seen)]
        v = np.repeat(Q.values(pool.vc[at], pool.vs[at]), hq // hkv, axis=1)
        # A partial result's log-sum-exp is -2^size / ln 2 + log2(its keys) in float32, whose steps
        # there are 2^(size - 23): the count is lost, and partials of unlike counts are merged as
        # equals.  What is left of the definition is that o is a mean of the keys' rows with weights
        # of sum 1: it lies between their extremes, but for the roundings of weights and output.
        err = EXT_ERR if members * hq // hkv > 128 else DEC_ERR
        tol = (2.0 ** -8 + err + 2.0 ** -18) * 1.01 * np.abs(v).max(0)
        got = A.bf16_to_f64(bits_of(o[b]))
        assert ((got >= v.min(0) - tol) & (got <= v.max(0) + tol)).all() and (got != 0).any(), b
        # -2^size + log of the count, which float32 cannot tell from -2^size
        got = lse[b].double().cpu().numpy()
        assert (np.abs(got + 2.0 ** size) <= 2.0 ** (size - 22)).all(), b
