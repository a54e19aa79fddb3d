"""The 8-bit pool on the GPU against float64: store and read-back bit for bit, attention within
bounds derived from its roundings.

Bounds.  With u = 2^-8 (half a bf16 step) an output element may be off by u |o| for its own
rounding.  The weights of the decode's second product are fp16: off by 2^-11 of their value, or,
below 2^-14 of the largest term, by 2^-25 of it.  A score is a float32 sum of exact products over
128 values; 16 roundings of partial sums of at most S = scale * sum |q_d k_d|, each 2^-23 (the
tensor core's accumulator truncates), move it by 2^-19 S, and the exponentials and logarithms by
2^-19; a weight is the ratio of two such terms.  The extend's weights are bf16: 2^-8 of their value
(8 significant bits: a value in [1, 2) has steps of 2^-7 and is off by at most half of one, 2^-8;
1 + 2^-8 itself, a tie, is off by 2^-8 / (1 + 2^-8)), times the V scale's own rounding, 2^-24.
"""
import numpy as np
import pytest
import torch

from oracle import attention as A, quantised as Q
from prefix_shared_kv_gb300 import rx, workloads as W
from prefix_shared_kv_gb300.session import DeviceWorkload, bits_of, to_bf16, to_i32, workspace

pytestmark = pytest.mark.gpu


class Pool:
    """A random 8-bit pool on the host and on the device, and a descriptor over `table`."""

    def __init__(self, cuda, rng, hq, hkv, pool_size, table):
        self.hq, self.hkv, self.n = hq, hkv, pool_size
        self.table, self.scale = np.ascontiguousarray(table, np.int32), 128 ** -0.5
        k = rng.standard_normal((pool_size, hkv, 128)).astype(np.float32)
        v = rng.standard_normal((pool_size, hkv, 128)).astype(np.float32)
        k[:, :, ::37] *= 3
        v *= np.exp(rng.standard_normal((pool_size, hkv, 1))).astype(np.float32)
        self.kc, self.ks = Q.quantise(W.bf16_bits(k))
        self.vc, self.vs = Q.quantise(W.bf16_bits(v))
        self.cuda = cuda
        self.upload()

    def upload(self):
        dev = self.cuda
        self.dev = [torch.from_numpy(a).to(dev) for a in (self.kc, self.vc, self.ks, self.vs)]
        self.kv = rx.kv_q8(*self.dev)
        self.r2t = to_i32(self.table, dev)
        self.desc = rx.kv_desc(self.hq, self.hkv, self.n, self.r2t, self.scale)

    def rows(self, at):
        """K, V and V scales of slots `at`; slots outside the pool are zeros."""
        ok = (at >= 0) & (at < self.n)
        at = np.where(ok, at, 0)
        z = ok[:, None, None]
        return (np.where(z, Q.values(self.kc[at], self.ks[at]), 0.0),
                np.where(z, Q.values(self.vc[at], self.vs[at]), 0.0),
                np.where(ok[:, None], self.vs[at].astype(np.float64), 0.0))

    def check(self, o, lse, q, req_row, keys, visible, weight_err, what=""):
        """o, lse [n, hq(, 128)] of one request's query rows against the definition."""
        K, V, vs = self.rows(self.table[req_row, :keys].astype(np.int64))
        got, got_l = A.bf16_to_f64(bits_of(o)), lse.double().cpu().numpy()
        qf = A.bf16_to_f64(q)
        gq = self.hq // self.hkv
        for h in range(self.hq):
            kh = h // gq
            ro, rl, pv, sabs, big = Q.attend_rows(qf[:, h], K[:, kh], V[:, kh], vs[:, kh], visible,
                                                  self.scale)
            e_s = 2.0 ** -19 * sabs + 2.0 ** -19
            tol = (2.0 ** -8 * np.abs(ro) + (weight_err + 2 * e_s)[:, None] * pv * 1.01
                   + (keys * 2.0 ** -25 * 448 * big)[:, None])
            err = np.abs(got[:, h] - ro)
            assert (err <= tol + 1e-30).all(), (what, h, float((err / (tol + 1e-30)).max()))
            lerr = np.abs(got_l[:, h] - rl)
            fin = np.isfinite(rl)
            assert (got_l[~fin, h] == rl[~fin]).all()
            ltol = e_s + 2.0 ** -22 * np.abs(np.where(fin, rl, 0))
            assert (lerr[fin] <= ltol[fin]).all(), (what, h, float(lerr[fin].max()))


def random_table(rng, pool_size, lens, shared=None):
    """Rows of distinct random slots; requests of `shared` = {group: (members, prefix)} share."""
    perm = rng.permutation(pool_size).astype(np.int32)
    at, table = 0, np.zeros((len(lens), max(1, max(lens, default=1)) + 3), np.int32)
    for members, prefix in (shared or {}).values():
        for b in members:
            table[b, :prefix] = perm[at:at + prefix]
        at += prefix
    start = np.zeros(len(lens), int)
    for members, prefix in (shared or {}).values():
        start[members] = prefix
    for b, n in enumerate(lens):
        own = n - start[b]
        table[b, start[b]:n] = perm[at:at + own]
        at += own
    assert at <= pool_size
    return table


# ---- store and load ---------------------------------------------------------------------------

def _special_rows(bits, hkv):
    """Overwrites some rows with zeros, tiny, huge, infinite and NaN values."""
    flat = bits.reshape(-1, 128)
    n = len(flat)
    flat[0] = 0
    flat[1 % n, 5] = 0x8000                      # -0
    flat[2 % n] = 0x0001                         # the smallest subnormal
    flat[3 % n] = 0x7F7F                         # the largest finite value
    flat[4 % n, 127] = 0x7F80                    # +inf
    flat[5 % n, 0] = 0xFF80                      # -inf
    flat[6 % n, 64] = 0x7FC1                     # NaN
    flat[7 % n] = 0x0100                         # about 2^-125: around the scale's floor
    flat[8 % n] = np.where(np.arange(128) == 3, 0x0380, 0x0001)
    return bits


@pytest.mark.parametrize("hkv,T", [(2, 1), (8, 37), (32, 1000), (1, 0), (3, 517), (5, 64), (12, 41),
                                   (256, 9), (1, 20011)])
def test_store_is_the_definition_bit_for_bit(cuda, hkv, T):
    rng = np.random.default_rng(T + hkv)
    P = max(T, 64) + 100
    kn = W.normal_bf16(rng, (T, hkv, 128))
    vn = W.bf16_bits(rng.standard_normal((T, hkv, 128)) * np.exp(8 * rng.standard_normal((T, hkv, 1))))
    if T >= 9:
        _special_rows(kn, hkv)
        _special_rows(vn[::-1], hkv)
    slots = rng.permutation(P)[:T].astype(np.int32)
    if T > 20:
        slots[3], slots[11] = -1, P  # outside the pool: skipped
    code = np.full((P, hkv, 128), 0x55, np.uint8)
    scale = np.full((P, hkv), 7.0, np.float32)
    want = [code.copy(), code.copy(), scale.copy(), scale.copy()]
    ok = (slots >= 0) & (slots < P)
    for i, new in ((0, kn), (1, vn)):
        want[i][slots[ok]], want[2 + i][slots[ok]] = Q.quantise(new[ok])
    dev = [torch.from_numpy(a).to(cuda) for a in (code, code, scale, scale)]
    desc = rx.kv_desc(hkv, hkv, P, to_i32(np.zeros((1, 16), np.int32), cuda))
    rx.store_kv_q8(desc, rx.kv_q8(*dev), to_bf16(kn, cuda), to_bf16(vn, cuda), to_i32(slots, cuda))
    torch.cuda.synchronize()
    for got, w in zip(dev, want):
        np.testing.assert_array_equal(got.cpu().numpy(), w)


@pytest.mark.parametrize("hkv,T", [(2, 1), (8, 37), (32, 1000), (1, 0), (3, 517), (256, 9),
                                   (1, 20011)])
def test_load_is_the_definition_bit_for_bit(cuda, hkv, T):
    rng = np.random.default_rng(T + hkv)
    P = 300
    codes = [rng.integers(0, 254, (P, hkv, 128), dtype=np.uint8) for _ in range(2)]
    for c in codes:
        c[c >= 127] += 1  # every code but the NaNs (0x7f, 0xff)
    scales = [np.exp(20 * rng.standard_normal((P, hkv))).astype(np.float32) for _ in range(2)]
    scales[0][5], scales[1][6] = np.nan, Q.MIN_SCALE
    slots = rng.integers(0, P, T).astype(np.int32)  # slots repeat
    if T > 20:
        slots[:4] = (5, 6, -1, P)
    dev = [torch.from_numpy(a).to(cuda) for a in (*codes, *scales)]
    desc = rx.kv_desc(hkv, hkv, P, to_i32(np.zeros((1, 16), np.int32), cuda))
    out = [torch.full((T + 1, hkv, 128), 7.0, dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    rx.load_kv_q8(desc, rx.kv_q8(*dev), to_i32(slots, cuda), out[0][:T], out[1][:T])
    torch.cuda.synchronize()
    ok = (slots >= 0) & (slots < P)
    at = np.where(ok, slots, 0)
    for i in range(2):
        with np.errstate(all="ignore"):
            x = (Q.VALUES[codes[i][at]].astype(np.float32) * scales[i][at][..., None])
        x[~ok] = 0
        want = torch.from_numpy(x).to(torch.bfloat16)
        got = out[i][:T].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got.float()), torch.nan_to_num(want.float()))
        assert (out[i][T] == 7).all()  # the row behind the last is left alone


# ---- decode -----------------------------------------------------------------------------------

DEC_ERR = 2.0 ** -11  # fp16 weights
EXT_ERR = 2.0 ** -8 + 2.0 ** -24  # bf16 weights, the V scale's product


def run_decode(pool, rng, lens, group_of_req=None, group_prefix_len=None, group_parent=None,
               q=None, stream=None):
    B = len(lens)
    if q is None:
        q = W.normal_bf16(rng, (B, pool.hq, 128))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.decode_plan(plan, pool.desc, np.arange(B), lens, group_of_req, group_prefix_len,
                   group_parent)
    ws = workspace(plan.workspace_size(), pool.cuda)
    ws.fill_(0xFF)  # partials that the merge reads without a write would be NaN
    plan.upload(ws)
    o = torch.full((B, pool.hq, 128), 7.0, dtype=torch.bfloat16, device=pool.cuda)
    lse = torch.full((B, pool.hq), 7.0, device=pool.cuda)
    rx.decode_attn_q8(plan, pool.desc, pool.kv, to_bf16(q, pool.cuda), o, lse, ws)
    torch.cuda.synchronize()
    return q, o, lse, ws, plan


def check_decode(pool, q, o, lse, lens, pick=None, err=DEC_ERR):
    for b in (range(len(lens)) if pick is None else pick):
        pool.check(o[b:b + 1], lse[b:b + 1], q[b:b + 1], b, lens[b],
                   np.ones((1, lens[b]), bool), err, f"request {b} of {lens[b]} keys")


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (8, 1), (1, 1), (6, 3), (40, 5), (12, 12),
                                    (64, 8), (16, 16), (48, 24)])
def test_decode_own_keys(cuda, hq, hkv):
    rng = np.random.default_rng(hq * 100 + hkv)
    lens = [1, 2, 7, 8, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 255, 256, 257, 300,
            511, 513, 700]
    pool = Pool(cuda, rng, hq, hkv, sum(lens) + 50, random_table(rng, sum(lens) + 50, lens))
    q, o, lse, ws, _ = run_decode(pool, rng, lens)
    check_decode(pool, q, o, lse, lens)
    assert rx.read_status(ws) == rx.RX_OK


@pytest.mark.parametrize("hq,hkv,members", [(8, 2, 4), (8, 8, 3), (8, 8, 9), (8, 8, 16), (8, 1, 2),
                                            (16, 8, 11), (32, 8, 17), (8, 2, 40), (12, 3, 33),
                                            (4, 1, 64), (8, 8, 130), (8, 8, 192), (32, 8, 50),
                                            (8, 1, 33), (3, 3, 300), (16, 2, 24)])
def test_decode_shared_prefixes(cuda, hq, hkv, members):
    rng = np.random.default_rng(hq + 10 * hkv + members)
    prefixes = (300, 33)
    shared = {0: (list(range(members)), prefixes[0]),
              1: (list(range(members, 2 * members)), prefixes[1])}
    lens = [prefixes[b >= members] + int(rng.integers(0, 90)) for b in range(2 * members)] + [50, 1]
    lens[1] = prefixes[0]  # nothing of its own
    n = sum(prefixes) + sum(lens) + 10
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens, shared))
    grp = [0] * members + [1] * members + [-1, -1]
    q, o, lse, ws, _ = run_decode(pool, rng, lens, grp, prefixes)
    pick = None if members < 20 else [0, 1, members - 1, members, 2 * members - 1, 2 * members,
                                      2 * members + 1, 17, 18]
    # a group of more than 128 rows runs on the extend's kernel, with its weights' rounding
    check_decode(pool, q, o, lse, lens, pick, EXT_ERR if members * hq // hkv > 128 else DEC_ERR)
    assert rx.read_status(ws) == rx.RX_OK


def test_decode_long_requests_split_over_many_items(cuda):
    rng = np.random.default_rng(5)
    lens = [20000, 3, 9001]
    n = sum(lens) + 9
    pool = Pool(cuda, rng, 8, 2, n, random_table(rng, n, lens))
    q, o, lse, _, plan = run_decode(pool, rng, lens)
    check_decode(pool, q, o, lse, lens)


@pytest.mark.parametrize("hq,hkv,lens", [
    (1, 1, [20000, 1]),            # more than 32 partials for each of sixteen warps
    (2, 1, [70000, 1, 257]),
    (16, 16, [16001] + [40] * 24),  # many rows, one with many partials: eight warps each
    (1, 1, [9000] + [1] * 400),
    (4, 2, [300, 700, 1, 5])])
def test_decode_merges_any_number_of_partials(cuda, hq, hkv, lens):
    """The number of warps that merge a row follows its partials and the rows; half of the long
    request's keys have weights of 2^-200 and less, so that whole partials weigh nothing."""
    rng = np.random.default_rng(len(lens) + hq)
    n = sum(lens) + 9
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens))
    q = W.normal_bf16(rng, (len(lens), hq, 128))
    far = pool.table[0, :lens[0] // 2]
    # codes of the largest size, their sign against the first query head of each KV head
    pool.kc[far] = np.where(A.bf16_to_f64(q[0, ::hq // hkv]) < 0, 0x7E, 0xFE)
    pool.ks[far] *= 8
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens, q=q)
    check_decode(pool, q, o, lse, lens, range(min(len(lens), 5)))
    assert rx.read_status(ws) == rx.RX_OK


def test_decode_nan_and_out_of_pool_keys_in_the_prefix_of_a_very_large_group(cuda):
    rng = np.random.default_rng(60)
    members, prefix = 70, 200
    lens = [prefix + 5] * members + [30]
    pool = Pool(cuda, rng, 8, 2, 1500, random_table(rng, 1500, lens, {0: (list(range(members)),
                                                                          prefix)}))
    grp = [0] * members + [-1]
    clean = run_decode(pool, rng, lens, grp, [prefix])
    check_decode(pool, *clean[:3], lens, [0, 35, 69, 70], EXT_ERR)
    pool.vs[pool.table[0, 131], 0] = np.nan
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens, grp, [prefix], q=clean[0])
    assert torch.isnan(o[:members, :4].float()).all() and torch.isfinite(lse).all()
    assert torch.equal(o[:members, 4:], clean[1][:members, 4:]) and torch.equal(o[70], clean[1][70])
    pool.vs[pool.table[0, 131], 0] = 1
    pool.table[:members, 64] = 1500
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens, grp, [prefix], q=clean[0])
    assert rx.read_status(ws) == rx.RX_ERR_RANGE
    check_decode(pool, q, o, lse, lens, [0, 69, 70], EXT_ERR)


def test_decode_tree_and_grouping_give_the_same_result(cuda):
    rng = np.random.default_rng(6)
    lens = [500 + 7 * b for b in range(9)]
    n = 6000
    table = random_table(rng, n, lens)
    table[:, :200] = table[0, :200]
    table[:5, 200:400] = table[0, 200:400]
    pool = Pool(cuda, rng, 16, 4, n, table)
    args = ([1] * 5 + [0] * 4, [200, 400], [-1, 0])
    q, o, lse, _, _ = run_decode(pool, rng, lens, *args)
    check_decode(pool, q, o, lse, lens)
    _, o2, lse2, _, _ = run_decode(pool, rng, lens, q=q)
    check_decode(pool, q, o2, lse2, lens)


def test_decode_is_the_same_on_every_call(cuda):
    rng = np.random.default_rng(7)
    lens = [2000, 50, 999]
    pool = Pool(cuda, rng, 16, 2, 4000, random_table(rng, 4000, lens))
    q, o, lse, ws, plan = run_decode(pool, rng, lens)
    for _ in range(3):
        o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
        rx.decode_attn_q8(plan, pool.desc, pool.kv, to_bf16(q, cuda), o2, lse2, ws)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_decode_scales_of_very_different_size(cuda):
    """A key with a large score and a tiny V scale, one with a tiny score and a large V scale, zero
    rows, and scales that grow or fall along the keys by 2^80: no weight may be lost to the fp16
    range."""
    rng = np.random.default_rng(8)
    lens = [300, 300, 300, 40, 300]
    pool = Pool(cuda, rng, 8, 8, 2000, random_table(rng, 2000, lens))
    t = pool.table
    pool.vs[t[0, :300]] = np.float32(2.0) ** np.linspace(-40, 40, 300)[:, None].astype(np.float32)
    pool.vs[t[1, :300]] = np.float32(2.0) ** np.linspace(40, -40, 300)[:, None].astype(np.float32)
    pool.ks[t[2, 7]] *= 20
    pool.vs[t[2, 7]] = np.float32(2.0 ** -30)
    pool.vs[t[2, 9]] = np.float32(2.0 ** 20)
    pool.kc[t[3, :40]], pool.vc[t[3, :40]] = 0, 0
    pool.ks[t[3, :40]] = pool.vs[t[3, :40]] = Q.MIN_SCALE
    pool.vc[t[4, 11]], pool.vs[t[4, 11]] = 0, Q.MIN_SCALE
    pool.ks[t[4, 11]] *= 30
    pool.upload()
    q, o, lse, _, _ = run_decode(pool, rng, lens)
    check_decode(pool, q, o, lse, lens)


def test_decode_queries_of_every_size(cuda):
    rng = np.random.default_rng(9)
    lens = [200] * 6
    pool = Pool(cuda, rng, 8, 2, 1500, random_table(rng, 1500, lens))
    x = rng.standard_normal((6, 8, 128))
    x[0] = 0
    x[1] *= 1e-30
    x[2] *= 30.0
    x[3, :, 5] = 1000.0
    x[3, :, 6:] *= 1e-4
    x[4] *= 2.0 ** -120
    q, o, lse, _, _ = run_decode(pool, rng, lens, q=W.bf16_bits(x))
    check_decode(pool, q, o, lse, lens)


@pytest.mark.parametrize("members", [3, 14])
def test_decode_a_request_does_not_disturb_those_it_shares_a_prefix_with(cuda, members):
    """Garbage in one request's query (a padded row: huge, infinite, NaN) leaves the results of the
    others of its group as they were, bit for bit."""
    rng = np.random.default_rng(50 + members)
    lens = [150 + 3 * b for b in range(members)]
    pool = Pool(cuda, rng, 8, 2, sum(lens) + 300,
                random_table(rng, sum(lens) + 300, lens, {0: (list(range(members)), 140)}))
    q, o, lse, _, _ = run_decode(pool, rng, lens, [0] * members, [140])
    check_decode(pool, q, o, lse, lens)
    for bad in (W.bf16_bits(np.full(1, 1e30))[0], 0x7F80, 0x7FC1, 0x0001):
        q2 = q.copy()
        q2[1] = bad
        _, o2, lse2, _, _ = run_decode(pool, rng, lens, [0] * members, [140], q=q2)
        rest = [b for b in range(members) if b != 1]
        assert torch.equal(o2[rest], o[rest]) and torch.equal(lse2[rest], lse[rest])


@pytest.mark.parametrize("members,large", [(3, [1]), (3, [0, 1, 2]), (14, [2, 13]), (1, [0])])
def test_decode_queries_of_2_to_the_22_beside_ordinary_ones(cuda, members, large):
    """Keys so small that queries of 2^22 have ordinary scores: they are as exact as any."""
    rng = np.random.default_rng(70 + members + len(large))
    lens = [150 + 30 * b for b in range(members)]
    pool = Pool(cuda, rng, 8, 2, sum(lens) + 300,
                random_table(rng, sum(lens) + 300, lens, {0: (list(range(members)), 140)}))
    pool.ks *= np.float32(2.0 ** -22)
    pool.upload()
    x = rng.standard_normal((members, 8, 128))
    x[large] *= 2.0 ** 22
    x[large, 3] *= 8
    q, o, lse, _, _ = run_decode(pool, rng, lens, [0] * members, [140], q=W.bf16_bits(x))
    check_decode(pool, q, o, lse, lens)


def test_decode_nan_rows_reach_their_readers_only(cuda):
    rng = np.random.default_rng(10)
    lens = [100, 100, 100, 260]
    shared = {0: ([0, 1], 60)}
    pool = Pool(cuda, rng, 8, 4, 700, random_table(rng, 700, lens, shared))
    t = pool.table
    spare = [s for s in range(700) if s not in set(t[:, :260].ravel().tolist())]
    pool.ks[spare] = pool.vs[spare] = np.nan       # never read
    clean = run_decode(pool, rng, lens, [0, 0, -1, -1], [60])
    pool.ks[t[1, 80]] = np.nan                     # request 1's own key
    pool.vs[t[3, 255], 2] = np.nan                 # request 3, KV head 2: V only
    pool.upload()
    q, o, lse, _, _ = run_decode(pool, rng, lens, [0, 0, -1, -1], [60], q=clean[0])
    assert torch.isnan(o[1].float()).all() and torch.isnan(lse[1]).all()
    assert torch.isnan(o[3, 4:6].float()).all() and torch.isfinite(lse[3]).all()
    for b, rest in ((0, slice(None)), (2, slice(None)), (3, [0, 1, 2, 3, 6, 7])):
        assert torch.equal(o[b, rest], clean[1][b, rest]) and torch.equal(lse[b], clean[2][b])


def test_decode_entry_outside_the_pool_is_flagged_and_reads_as_zeros(cuda):
    rng = np.random.default_rng(11)
    lens = [90, 300]
    for bad in (-1, 1000, 2 ** 31 - 1):
        pool = Pool(cuda, rng, 8, 2, 1000, random_table(rng, 1000, lens))
        pool.table[1, 133] = bad
        pool.upload()
        q, o, lse, ws, _ = run_decode(pool, rng, lens)
        assert rx.read_status(ws) == rx.RX_ERR_RANGE and rx.read_status(ws) == rx.RX_OK
        check_decode(pool, q, o, lse, lens)
    pool.table[1, 133] = 5
    pool.table[1, 300:] = -7  # entries past the sequence are not read
    pool.upload()
    q, o, lse, ws, _ = run_decode(pool, rng, lens)
    assert rx.read_status(ws) == rx.RX_OK
    check_decode(pool, q, o, lse, lens)


def test_empty_batch_launches_nothing(cuda):
    rng = np.random.default_rng(12)
    pool = Pool(cuda, rng, 8, 2, 64, random_table(rng, 64, [8]))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    z = np.zeros(0, np.int32)
    rx.decode_plan(plan, pool.desc, z, z)
    ws = workspace(plan.workspace_size(), cuda)
    plan.upload(ws)
    e = torch.empty((0, 8, 128), dtype=torch.bfloat16, device=cuda)
    rx.decode_attn_q8(plan, pool.desc, pool.kv, e, e, torch.empty((0, 8), device=cuda), ws)
    torch.cuda.synchronize()


def test_slots_whose_offsets_pass_32_bits(cuda):
    """A pool of more than 2^32 codes: store to, read back from and attend over its last slots."""
    hkv, P = 32, (1 << 20) + 4096 + 7  # 4.3e9 codes in K and in V
    rng = np.random.default_rng(13)
    n = 200
    slots = np.concatenate([P - 1 - rng.permutation(4000)[:n - 3], [0, 5, 9]]).astype(np.int32)
    code = [torch.zeros((P, hkv, 128), dtype=torch.uint8, device=cuda) for _ in range(2)]
    scale = [torch.zeros((P, hkv), device=cuda) for _ in range(2)]
    kv = rx.kv_q8(*code, *scale)
    r2t = to_i32(np.array([slots]), cuda)
    desc = rx.kv_desc(hkv, hkv, P, r2t)
    kn, vn = (W.normal_bf16(rng, (n, hkv, 128)) for _ in range(2))
    rx.store_kv_q8(desc, kv, to_bf16(kn, cuda), to_bf16(vn, cuda), r2t[0])
    out = [torch.empty((n, hkv, 128), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    rx.load_kv_q8(desc, kv, r2t[0], *out)
    for new, got in ((kn, out[0]), (vn, out[1])):
        c, s = Q.quantise(new)
        want = torch.from_numpy(Q.VALUES[c].astype(np.float32) * s[..., None]).to(torch.bfloat16)
        assert torch.equal(got.cpu(), want)
    q = W.normal_bf16(rng, (1, hkv, 128))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.decode_plan(plan, desc, [0], [n])
    ws = workspace(plan.workspace_size(), cuda)
    plan.upload(ws)
    o = torch.empty((1, hkv, 128), dtype=torch.bfloat16, device=cuda)
    lse = torch.empty((1, hkv), device=cuda)
    rx.decode_attn_q8(plan, desc, kv, to_bf16(q, cuda), o, lse, ws)
    torch.cuda.synchronize()
    (kc, ks), (vc, vs) = Q.quantise(kn), Q.quantise(vn)
    for h in range(hkv):
        ro, rl, pv, sabs, big = Q.attend_rows(
            A.bf16_to_f64(q[:, h]), Q.values(kc, ks)[:, h], Q.values(vc, vs)[:, h],
            vs[:, h].astype(np.float64), np.ones((1, n), bool), 128 ** -0.5)
        e_s = 2.0 ** -19 * (sabs + 1)
        tol = (2.0 ** -8 * np.abs(ro) + (DEC_ERR + 2 * e_s)[:, None] * pv * 1.01
               + n * 2.0 ** -25 * 448 * big[:, None])
        assert (np.abs(A.bf16_to_f64(bits_of(o[:, h])) - ro) <= tol).all()
        assert np.abs(lse[0, h].item() - rl[0]) <= e_s[0] + 2.0 ** -22 * abs(rl[0])


def test_two_streams_and_a_captured_graph(cuda):
    """Plans of their own on two streams at once, and a store plus decode captured and replayed on
    inputs that change between the replays."""
    rng = np.random.default_rng(14)
    lens = [700, 64, 1]
    pool = Pool(cuda, rng, 16, 4, 2000, random_table(rng, 2000, lens))
    q = W.normal_bf16(rng, (2, 3, 16, 128))
    work = []
    for i in range(2):
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        rx.decode_plan(plan, pool.desc, np.arange(3), lens)
        ws = workspace(plan.workspace_size(), cuda)
        plan.upload(ws)
        work.append((plan, ws, to_bf16(q[i], cuda),
                     torch.empty((3, 16, 128), dtype=torch.bfloat16, device=cuda),
                     torch.empty((3, 16), device=cuda), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        for plan, ws, dq, o, lse, s in work:
            rx.decode_attn_q8(plan, pool.desc, pool.kv, dq, o, lse, ws, stream=s)
    torch.cuda.synchronize()
    for i, (plan, ws, dq, o, lse, s) in enumerate(work):
        check_decode(pool, q[i], o, lse, lens)

    plan, ws, dq, o, lse, _ = work[0]
    new = [W.normal_bf16(rng, (3, 4, 128)) for _ in range(4)]
    slots = np.array([pool.table[b, lens[b] - 1] for b in range(3)], np.int32)
    dk, dv, ds = to_bf16(new[0], cuda), to_bf16(new[1], cuda), to_i32(slots, cuda)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rx.store_kv_q8(pool.desc, pool.kv, dk, dv, ds)
        rx.decode_attn_q8(plan, pool.desc, pool.kv, dq, o, lse, ws)
    for k, v in (new[:2], new[2:]):
        dk.copy_(to_bf16(k, cuda))
        dv.copy_(to_bf16(v, cuda))
        o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        pool.kc[slots], pool.ks[slots] = Q.quantise(k)
        pool.vc[slots], pool.vs[slots] = Q.quantise(v)
        check_decode(pool, q[0], o, lse, lens)


# ---- extend -----------------------------------------------------------------------------------



def run_extend(pool, rng, prefix, new, group_of_req=None, group_prefix_len=None,
               group_parent=None, q=None):
    n = int(np.sum(new))
    if q is None:
        q = W.normal_bf16(rng, (n, pool.hq, 128))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.extend_plan(plan, pool.desc, np.arange(len(new)), prefix, new, group_of_req,
                   group_prefix_len, group_parent)
    ws = workspace(plan.workspace_size(), pool.cuda)
    plan.upload(ws)
    o = torch.full((n + 1, pool.hq, 128), 7.0, dtype=torch.bfloat16, device=pool.cuda)
    lse = torch.full((n + 1, pool.hq), 7.0, device=pool.cuda)
    rx.extend_attn_q8(plan, pool.desc, pool.kv, to_bf16(q, pool.cuda), o[:n], lse[:n], ws)
    torch.cuda.synchronize()
    assert (o[n] == 7).all() and (lse[n] == 7).all()  # the row behind the last is left alone
    return q, o[:n], lse[:n], ws


def check_extend(pool, q, o, lse, prefix, new, pick=None):
    cu = np.concatenate([[0], np.cumsum(new)])
    for r in (range(len(new)) if pick is None else pick):
        L = prefix[r] + new[r]
        if new[r] == 0:
            continue
        seen = np.arange(L)[None, :] <= (prefix[r] + np.arange(new[r]))[:, None]
        rows = slice(int(cu[r]), int(cu[r + 1]))
        pool.check(o[rows], lse[rows], q[rows], r, L, seen, EXT_ERR,
                   f"request {r}: {prefix[r]} cached, {new[r]} new")


def extend_case(cuda, seed, hq, hkv, prefix, new, groups=()):
    """groups: (members, shared prefix) each; other requests share nothing."""
    rng = np.random.default_rng(seed)
    lens = [p + e for p, e in zip(prefix, new)]
    shared = {g: (list(m), p) for g, (m, p) in enumerate(groups)}
    n = sum(lens) + 20
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens, shared))
    grp = np.full(len(new), -1)
    for g, (m, p) in enumerate(groups):
        grp[list(m)] = g
    return rng, pool, grp, [p for _, p in groups]


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (8, 1), (1, 1), (6, 3), (10, 5), (24, 12)])
def test_extend_lengths_and_heads(cuda, hq, hkv):
    prefix = [0, 0, 1, 63, 64, 65, 127, 200, 300, 5, 0]
    new = [1, 64, 63, 1, 65, 2, 128, 0, 17, 129, 150]
    rng, pool, grp, gpl = extend_case(cuda, hq * 10 + hkv, hq, hkv, prefix, new)
    q, o, lse, ws = run_extend(pool, rng, prefix, new)
    check_extend(pool, q, o, lse, prefix, new)
    assert rx.read_status(ws) == rx.RX_OK


@pytest.mark.parametrize("hq,hkv", [(8, 2), (4, 4), (8, 1)])
def test_extend_shared_prefixes(cuda, hq, hkv):
    prefix = [200] * 6 + [333] * 3 + [64, 0]
    new = [1, 40, 77, 3, 130, 20, 9, 64, 50, 30, 100]
    prefix[2], prefix[7] = 260, 400  # cached tokens of their own behind the shared prefix
    rng, pool, grp, gpl = extend_case(cuda, 3 + hq, hq, hkv, prefix, new,
                                      [(range(6), 200), (range(6, 9), 333)])
    q, o, lse, ws = run_extend(pool, rng, prefix, new, grp, gpl)
    check_extend(pool, q, o, lse, prefix, new)
    _, o2, lse2, _ = run_extend(pool, rng, prefix, new, q=q)  # the same without the groups
    check_extend(pool, q, o2, lse2, prefix, new)


def test_extend_many_items_per_sm_with_one_and_two_tiles(cuda):
    """More items than SMs, items of one tile among items of two, of few steps among many."""
    rng = np.random.default_rng(21)
    prefix = [int(x) for x in rng.integers(0, 500, 60)]
    new = [int(x) for x in rng.integers(1, 300, 60)]
    prefix[:20] = [150] * 20
    _, pool, grp, gpl = extend_case(cuda, 22, 16, 8, prefix, new, [(range(20), 150)])
    q, o, lse, ws = run_extend(pool, rng, prefix, new, grp, gpl)
    assert rx.read_status(ws) == rx.RX_OK
    check_extend(pool, q, o, lse, prefix, new, pick=[0, 7, 19, 20, 33, 41, 59])


def test_extend_long_prefix(cuda):
    prefix, new = [9000, 3001], [70, 5]
    rng, pool, _, _ = extend_case(cuda, 23, 4, 1, prefix, new)
    q, o, lse, _ = run_extend(pool, rng, prefix, new)
    check_extend(pool, q, o, lse, prefix, new)


@pytest.mark.parametrize("hq,hkv,prefix,new", [
    (8, 2, [1000] * 4, [40] * 4), (32, 8, [16000], [4]), (1, 1, [5000, 3], [1, 1]),
    (6, 3, [2111, 77, 600], [9, 33, 1]), (8, 1, [4096], [17]), (2, 2, [0], [900])])
def test_extend_small_batches_split_their_keys(cuda, hq, hkv, prefix, new):
    rng, pool, _, _ = extend_case(cuda, 31 + hq, hq, hkv, prefix, new)
    q, o, lse, ws = run_extend(pool, rng, prefix, new)
    check_extend(pool, q, o, lse, prefix, new)
    assert rx.read_status(ws) == rx.RX_OK


def test_extend_small_batches_with_a_shared_prefix_split_their_keys(cuda):
    prefix, new = [1500, 1500, 1530, 1500, 20], [3, 30, 1, 90, 2]
    rng, pool, grp, gpl = extend_case(cuda, 41, 8, 2, prefix, new, [(range(4), 1500)])
    q, o, lse, _ = run_extend(pool, rng, prefix, new, grp, gpl)
    check_extend(pool, q, o, lse, prefix, new)


@pytest.mark.parametrize("hq,hkv,prefix,new,groups,parents", [
    (64, 8, [4000], [340], [], None),          # fewer pairs of tiles than SMs, more tiles
    (24, 3, [2500], [830], [], None),
    (8, 1, [0], [4000], [], None),             # nothing cached: causal tiles of every length
    (16, 2, [4000, 100], [1250, 33], [], None),
    (20, 5, [2000] * 3, [300, 2, 700], [(0, 1, 2)], None),
    (40, 5, [3000] * 4, [130, 165, 200, 1], [(0, 1), (2,), (3,)], [-1, 0, 0])])
def test_extend_cuts_items_where_the_lists_end_apart(cuda, hq, hkv, prefix, new, groups, parents):
    """Batches of one to three items an SM: some items are cut, their rows merged, the others write
    theirs; the whole result twice, bit for bit."""
    rng = np.random.default_rng(hq + len(new))
    lens = [p + e for p, e in zip(prefix, new)]
    n = sum(lens) + 20
    shared = {0: (list(range(len(new))), prefix[0])} if groups else None
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens, shared))
    grp, gpl = None, None
    if groups:
        grp = [next(g for g, m in enumerate(groups) if b in m) for b in range(len(new))]
        gpl = [prefix[0]] if parents is None else [600, 2500, 2500]
    rows = int(np.sum(new))
    q = W.normal_bf16(rng, (rows, hq, 128))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.extend_plan(plan, pool.desc, np.arange(len(new)), prefix, new, grp, gpl, parents)
    assert plan.launches() == 3
    ws = workspace(plan.workspace_size(), cuda)
    results = []
    for fill in (0xFF, 0x00):  # partials that the merge reads without a write would be NaN
        ws.fill_(fill)
        plan.upload(ws)
        o = torch.full((rows + 1, hq, 128), 7.0, dtype=torch.bfloat16, device=cuda)
        lse = torch.full((rows + 1, hq), 7.0, device=cuda)
        rx.extend_attn_q8(plan, pool.desc, pool.kv, to_bf16(q, cuda), o[:rows], lse[:rows], ws)
        torch.cuda.synchronize()
        assert rx.read_status(ws) == rx.RX_OK
        assert (o[rows] == 7).all() and (lse[rows] == 7).all()
        results.append((o, lse))
    assert all(torch.equal(a, b) for a, b in zip(*results))
    check_extend(pool, q, o[:rows], lse[:rows], prefix, new)


@pytest.mark.parametrize("hq,hkv,prefix,new,groups", [
    (32, 8, [3000, 700, 0, 129, 64], [1, 1, 1, 1, 1], []),
    (48, 12, [2500] * 6, [2, 1, 3, 0, 17, 32], [((0, 1, 2, 3), 2400)]),
    (5, 5, [1900, 2000, 2100], [4, 3, 2], [((0, 2), 1900)]),
    (8, 1, [6000], [1], []),
    (40, 5, [1500] * 5 + [1501], [1, 2, 1, 1, 2, 1], [((0, 1, 2, 3, 4, 5), 1500)])])
def test_extend_of_few_new_tokens(cuda, hq, hkv, prefix, new, groups):
    rng, pool, grp, gpl = extend_case(cuda, hq + sum(new), hq, hkv, prefix, new, groups)
    q, o, lse, ws = run_extend(pool, rng, prefix, new, grp, gpl)
    check_extend(pool, q, o, lse, prefix, new)
    assert rx.read_status(ws) == rx.RX_OK
    # planned as a decode: no expanded keys in the workspace
    assert ws.numel() < sum(prefix[i] for i in range(len(new))) * hkv * 522 or sum(prefix) < 2000
    pool.vs[pool.table[0, 1], 0] = np.nan  # a key that request 0 reads, and who shares it
    pool.upload()
    q2, o2, lse2, ws = run_extend(pool, rng, prefix, new, grp, gpl, q=q)
    cu = np.concatenate([[0], np.cumsum(new)])
    for r in range(len(new)):
        shares = r == 0 or (groups and r in groups[0][0])
        got = o2[int(cu[r]):int(cu[r + 1])].float()
        assert torch.isnan(got[:, :hq // hkv]).all() if shares and new[r] else not torch.isnan(got).any()
    assert torch.isfinite(lse2).all()


@pytest.mark.parametrize("hq,hkv,prefix,groups", [(32, 16, 2000, 3), (64, 8, 1500, 2)])
def test_extend_splits_pairs_of_tiles(cuda, hq, hkv, prefix, groups):
    """Fewer pairs of tiles than SMs, too many tiles to split each: the pairs' keys are split."""
    members = 5
    new = [20, 21, 3, 30, 26] * groups
    if hq == 64:
        new = [33, 40, 2, 61, 9] * groups
    rng, pool, grp, gpl = extend_case(
        cuda, hq, hq, hkv, [prefix + 7] * len(new), new,
        [(range(g * members, (g + 1) * members), prefix) for g in range(groups)])
    q, o, lse, ws = run_extend(pool, rng, [prefix + 7] * len(new), new, grp, gpl)
    check_extend(pool, q, o, lse, [prefix + 7] * len(new), new)
    assert rx.read_status(ws) == rx.RX_OK


def test_every_form_of_extend_captured_and_on_two_streams(cuda):
    """Few new tokens, cut items and split pairs: three plans captured in one graph, replayed with new
    queries, and called on two streams at once, give what eager calls give, bit for bit."""
    rng = np.random.default_rng(31)
    forms = [(8, 2, [3000, 500], [1, 2]), (24, 3, [1500], [830]), (16, 16, [1200] * 2, [150, 149])]
    made = []
    for hq, hkv, prefix, new in forms:
        lens = [p + e for p, e in zip(prefix, new)]
        n = sum(lens) + 20
        pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, lens))
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        rx.extend_plan(plan, pool.desc, np.arange(len(new)), prefix, new)
        ws = workspace(plan.workspace_size(), cuda)
        plan.upload(ws)
        rows = sum(new)
        made.append((pool, plan, ws, torch.empty(rows, hq, 128, dtype=torch.bfloat16, device=cuda),
                     torch.empty(rows, hq, 128, dtype=torch.bfloat16, device=cuda),
                     torch.empty(rows, hq, device=cuda)))

    def call(m):
        pool, plan, ws, q, o, lse = m
        rx.extend_attn_q8(plan, pool.desc, pool.kv, q, o, lse, ws)

    def fresh(seed):
        g = torch.Generator(device=cuda).manual_seed(seed)
        for m in made:
            m[3].copy_(torch.randn(m[3].shape, generator=g, device=cuda))
            m[4].fill_(7)
            m[5].fill_(7)

    def results():
        torch.cuda.synchronize()
        return [t.clone() for m in made for t in m[4:]]

    want = []
    for seed in (1, 2):
        fresh(seed)
        for m in made:
            call(m)
        want.append(results())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        for m in made:
            call(m)
    for seed in (1, 2, 1):
        fresh(seed)
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(results(), want[seed - 1]))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    fresh(2)
    torch.cuda.synchronize()
    for _ in range(3):
        for i, m in enumerate(made):
            with torch.cuda.stream(streams[i % 2]):
                call(m)
    assert all(torch.equal(a, b) for a, b in zip(results(), want[1]))


def test_extend_every_code_and_scale(cuda):
    """Codes of every value (subnormal ones too) and scales over 2^60."""
    prefix, new = [254], [64]
    rng, pool, _, _ = extend_case(cuda, 24, 2, 2, prefix, new)
    at = pool.table[0, :254]
    every = np.array([c for c in range(256) if c not in (127, 255)], np.uint8)
    pool.vc[at] = every[(np.arange(254)[:, None, None] + np.arange(128)) % 254]
    pool.vs[at] = np.exp2(rng.integers(-30, 30, (254, 2))).astype(np.float32)
    pool.kc[at] = every[(np.arange(254)[:, None, None] + 3 * np.arange(128)) % 254]
    pool.ks[at] = np.float32(1 / 448)
    pool.upload()
    q, o, lse, _ = run_extend(pool, rng, prefix, new)
    check_extend(pool, q, o, lse, prefix, new)


def test_extend_nan_rows_reach_the_rows_that_see_them_only(cuda):
    prefix, new = [100, 100, 30], [70, 20, 40]
    rng, pool, grp, gpl = extend_case(cuda, 25, 8, 4, prefix, new, [(range(2), 100)])
    t = pool.table
    used = set(t[0, :170].tolist()) | set(t[1, :120].tolist()) | set(t[2, :70].tolist())
    spare = [s for s in range(pool.n) if s not in used]
    pool.ks[spare] = pool.vs[spare] = np.nan
    pool.upload()
    q, o, lse, _ = run_extend(pool, rng, prefix, new, grp, gpl)
    pool.ks[t[0, 130]] = np.nan         # new token 30 of request 0: rows 30 .. 69 see it
    pool.vs[t[1, 105], 1] = np.nan      # new token 5 of request 1, KV head 1
    pool.upload()
    _, o2, lse2, _ = run_extend(pool, rng, prefix, new, grp, gpl, q=q)
    assert torch.isnan(o2[30:70].float()).all() and torch.isnan(lse2[30:70]).all()
    assert torch.isnan(o2[75:90, 2:4].float()).all() and torch.isfinite(lse2[70:90]).all()
    same = torch.ones_like(o, dtype=torch.bool)
    same[30:70] = False
    same[75:90, 2:4] = False
    assert torch.equal(o2[same], o[same])
    assert torch.equal(lse2[:30], lse[:30]) and torch.equal(lse2[70:], lse[70:])


def test_extend_entry_outside_the_pool_is_flagged_and_reads_as_zeros(cuda):
    prefix, new = [150, 40], [10, 80]
    rng, pool, _, _ = extend_case(cuda, 26, 8, 2, prefix, new)
    for bad in (-1, -9, pool.n, 2 ** 31 - 1, -2 ** 31 + 1):
        pool.table[0, 99], pool.table[1, 41] = bad, 3
        pool.upload()
        q, o, lse, ws = run_extend(pool, rng, prefix, new)
        assert rx.read_status(ws) == rx.RX_ERR_RANGE
        check_extend(pool, q, o, lse, prefix, new)


def test_extend_empty_and_repeated(cuda):
    prefix, new = [20, 30], [0, 0]
    rng, pool, _, _ = extend_case(cuda, 27, 8, 2, prefix, new)
    run_extend(pool, rng, prefix, new)  # no new tokens: nothing is launched
    prefix, new = [200, 500], [90, 300]
    rng, pool, _, _ = extend_case(cuda, 28, 8, 2, prefix, new)
    q, o, lse, _ = run_extend(pool, rng, prefix, new)
    for _ in range(3):
        _, o2, lse2, _ = run_extend(pool, rng, prefix, new, q=q)
        assert torch.equal(o, o2) and torch.equal(lse, lse2)


def test_a_served_batch_through_the_8_bit_pool(cuda):
    """As a server uses the calls: a prompt is stored and extended in two chunks, then decoded token
    by token, in one captured step at the end; each output against attention over what the pool
    then holds, and the pool read back against its codes."""
    rng = np.random.default_rng(29)
    hq, hkv, n = 8, 2, 400
    pool = Pool(cuda, rng, hq, hkv, n, random_table(rng, n, [180, 150]))
    pool.kc[:], pool.vc[:], pool.ks[:], pool.vs[:] = 0, 0, 0, 0
    pool.upload()
    done = [0, 0]

    def store(count):
        at = np.concatenate([pool.table[r, done[r]:done[r] + count[r]] for r in range(2)])
        k, v = (W.normal_bf16(rng, (len(at), hkv, 128)) for _ in range(2))
        rx.store_kv_q8(pool.desc, pool.kv, to_bf16(k, cuda), to_bf16(v, cuda), to_i32(at, cuda))
        pool.kc[at], pool.ks[at] = Q.quantise(k)
        pool.vc[at], pool.vs[at] = Q.quantise(v)

    for count in ([100, 40], [70, 100]):
        store(count)
        q, o, lse, _ = run_extend(pool, rng, list(done), count)
        check_extend(pool, q, o, lse, list(done), count)
        done = [d + c for d, c in zip(done, count)]
    for _ in range(3):
        store([1, 1])
        done = [d + 1 for d in done]
        q, o, lse, _, _ = run_decode(pool, rng, list(done))
        check_decode(pool, q, o, lse, list(done))
    at = to_i32(pool.table[0, :done[0]], cuda)
    out = [torch.empty((done[0], hkv, 128), dtype=torch.bfloat16, device=cuda) for _ in range(2)]
    rx.load_kv_q8(pool.desc, pool.kv, at, *out)
    K, V, _ = pool.rows(pool.table[0, :done[0]].astype(np.int64))
    for got, want in zip(out, (K, V)):
        # one rounding to float32 and one to bf16
        assert (np.abs(A.bf16_to_f64(bits_of(got)) - want) <= 2.0 ** -8 * 1.001 * np.abs(want)).all()


@pytest.mark.parametrize("name", ["tiny", "tree"])
def test_a_workload_over_the_8_bit_pool(cuda, name):
    """The repository's own driver, every step: the tiny workload (extend, then decodes), and a radix
    tree's mixed batch."""
    wl = W.tiny() if name == "tiny" else W.tree_workload(
        41, 8, 8, depth=2, fanout=3, seg_lo=50, seg_hi=300, p_empty=0.0, n_decode=40, tail_hi=40,
        n_extend=6, own_hi=30, ext_lo=1, ext_hi=100)
    dw = DeviceWorkload(wl, cuda, kv_type=rx.RX_KV_E4M3)
    kp, vp = wl.k_pool, wl.v_pool
    for i, st in enumerate(wl.steps):
        dw.run_step(i)
        torch.cuda.synchronize()
        kp, vp = A.store_kv(kp, vp, st.k_new, st.v_new, st.store_slots)
        (kc, ks), (vc, vs) = Q.quantise(kp), Q.quantise(vp)
        ds = dw.steps[i]
        for got, want in zip(dw.kv.tensors, (kc, vc, ks, vs)):
            np.testing.assert_array_equal(got.view(torch.uint8).cpu().numpy().reshape(-1),
                                          want.view(np.uint8).reshape(-1))
        K, V = Q.values(kc, ks), Q.values(vc, vs)
        todo = []
        if st.extend is not None:
            e = st.extend
            todo.append((ds.ext_o, ds.ext_lse, e.q, EXT_ERR, Q.extend(
                e.q, K, V, wl.req_to_token, e.req_idx, e.prefix_len, e.extend_len, e.cu_q,
                wl.softmax_scale)))
        if st.decode is not None:
            d = st.decode
            todo.append((ds.dec_o, ds.dec_lse, d.q, DEC_ERR, Q.decode(
                d.q, K, V, wl.req_to_token, d.req_idx, d.seq_len, wl.softmax_scale)))
        for o, lse, q, err, (ro, rl) in todo:
            # |weights| sum to 1, |v| <= max |V|, S <= scale |q| |k| (Cauchy)
            big = np.abs(V).max()
            S = wl.softmax_scale * np.linalg.norm(A.bf16_to_f64(q), axis=-1) \
                * np.linalg.norm(K, axis=-1).max()
            e_s = 2.0 ** -19 * (S + 1)
            tol = 2.0 ** -8 * np.abs(ro) + ((err + 2 * e_s) * big)[..., None] + 2.0 ** -20 * big
            assert (np.abs(A.bf16_to_f64(bits_of(o)) - ro) <= tol).all()
            assert (np.abs(lse.double().cpu().numpy() - rl) <= e_s + 2.0 ** -22 * np.abs(rl)).all()


# ---- calls as the documentation allows them ----------------------------------------------------

def test_tensors_at_16_byte_but_not_32_byte_addresses(cuda):
    rng = np.random.default_rng(81)
    hkv, T, P = 4, 700, 900

    def odd(shape, dtype):  # a view that starts 16 bytes behind a 512-byte boundary
        n = int(np.prod(shape))
        size = torch.empty(0, dtype=dtype).element_size()
        base = torch.zeros(n + 64, dtype=dtype, device=cuda)
        view = base[16 // size:16 // size + n].view(shape)
        assert view.data_ptr() % 32 == 16
        return view

    code = [odd((P, hkv, 128), torch.uint8) for _ in range(2)]
    scale = [odd((P, hkv), torch.float32) for _ in range(2)]
    kv = rx.kv_q8(*code, *scale)
    new = [odd((T, hkv, 128), torch.bfloat16) for _ in range(2)]
    out = [odd((T, hkv, 128), torch.bfloat16) for _ in range(2)]
    bits = [W.normal_bf16(rng, (T, hkv, 128)) for _ in range(2)]
    for n, b in zip(new, bits):
        n.copy_(to_bf16(b, cuda))
    slots = rng.permutation(P)[:T].astype(np.int32)
    table = to_i32(np.array([slots]), cuda)
    desc = rx.kv_desc(8, hkv, P, table)
    rx.store_kv_q8(desc, kv, *new, to_i32(slots, cuda))
    rx.load_kv_q8(desc, kv, to_i32(slots, cuda), *out)
    want = [Q.quantise(b) for b in bits]
    for i in range(2):
        assert np.array_equal(code[i].cpu().numpy()[slots], want[i][0])
        assert np.array_equal(scale[i].cpu().numpy()[slots], want[i][1])
        x = torch.from_numpy(Q.VALUES[want[i][0]].astype(np.float32) * want[i][1][..., None])
        assert torch.equal(out[i].cpu(), x.to(torch.bfloat16))
    K, V = (Q.values(*w) for w in want)
    for kind in ("decode", "extend"):
        n = 1 if kind == "decode" else 50
        q, o, lse = odd((n, 8, 128), torch.bfloat16), odd((n, 8, 128), torch.bfloat16), odd(
            (n, 8), torch.float32)
        qb = W.normal_bf16(rng, (n, 8, 128))
        q.copy_(to_bf16(qb, cuda))
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        if kind == "decode":
            rx.decode_plan(plan, desc, [0], [T])
        else:
            rx.extend_plan(plan, desc, [0], [T - n], [n])
        ws = workspace(plan.workspace_size(), cuda)
        plan.upload(ws)
        (rx.decode_attn_q8 if kind == "decode" else rx.extend_attn_q8)(plan, desc, kv, q, o, lse, ws)
        torch.cuda.synchronize()
        at = np.arange(T)[None]
        ro, rl = Q.extend(qb, K, V, at, [0], [T - n], [n], [0, n], 128 ** -0.5)
        assert np.abs(A.bf16_to_f64(bits_of(o)) - ro).max() <= 2.0 ** -6 * np.abs(V).max()
        assert np.abs(lse.double().cpu().numpy() - rl).max() <= 1e-3


def test_nothing_is_written_outside_the_outputs(cuda):
    """Guard bands around the outputs, the pool and the workspace of every call."""
    rng = np.random.default_rng(82)
    band = 4096

    def guarded(shape, dtype):
        n = int(np.prod(shape))
        base = torch.full(((n + 2 * band) * torch.empty(0, dtype=dtype).element_size(),), 0xA5,
                          dtype=torch.uint8, device=cuda).view(dtype)
        return base, base[band:band + n].view(shape)

    def untouched(base, n):
        raw = base.view(torch.uint8).cpu().numpy()
        b = band * base.element_size()
        return (raw[:b] == 0xA5).all() and (raw[-b:] == 0xA5).all()

    P, hkv, hq = 700, 3, 12
    lens = [200, 333, 64]
    table = random_table(rng, P, lens)
    kept = [guarded((P, hkv, 128), torch.uint8) for _ in range(2)] + \
        [guarded((P, hkv), torch.float32) for _ in range(2)]
    kv = rx.kv_q8(*(t for _, t in kept))
    r2t = to_i32(table, cuda)
    desc = rx.kv_desc(hq, hkv, P, r2t)
    slots = to_i32(rng.permutation(P).astype(np.int32), cuda)
    new = [to_bf16(W.normal_bf16(rng, (P, hkv, 128)), cuda) for _ in range(2)]
    rx.store_kv_q8(desc, kv, *new, slots)
    out = [guarded((P, hkv, 128), torch.bfloat16) for _ in range(2)]
    rx.load_kv_q8(desc, kv, slots, out[0][1], out[1][1])
    kept += out
    for kind in ("decode", "extend"):
        n = 3 if kind == "decode" else 120
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        if kind == "decode":
            rx.decode_plan(plan, desc, np.arange(3), lens)
        else:
            rx.extend_plan(plan, desc, np.arange(3), [l - 40 for l in lens], [40] * 3)
        size = plan.workspace_size()
        ws = guarded((size,), torch.uint8)
        plan.upload(ws[1])
        o, lse = guarded((n, hq, 128), torch.bfloat16), guarded((n, hq), torch.float32)
        q = to_bf16(W.normal_bf16(rng, (n, hq, 128)), cuda)
        (rx.decode_attn_q8 if kind == "decode" else rx.extend_attn_q8)(
            plan, desc, kv, q, o[1], lse[1], ws[1])
        torch.cuda.synchronize()
        assert torch.isfinite(o[1].float()).all() and torch.isfinite(lse[1]).all()
        kept += [ws, o, lse]
    for base, t in kept:
        assert untouched(base, t.numel())


def test_extend_on_two_streams_and_in_a_captured_graph(cuda):
    prefix, new = [300, 40], [200, 90]
    rng, pool, _, _ = extend_case(cuda, 83, 16, 4, prefix, new)
    q = [W.normal_bf16(rng, (290, 16, 128)) for _ in range(2)]
    work = []
    for i in range(2):
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        rx.extend_plan(plan, pool.desc, [0, 1], prefix, new)
        ws = workspace(plan.workspace_size(), cuda)
        plan.upload(ws)
        work.append((plan, ws, to_bf16(q[i], cuda),
                     torch.empty((290, 16, 128), dtype=torch.bfloat16, device=cuda),
                     torch.empty((290, 16), device=cuda), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(10):
        for plan, ws, dq, o, lse, s in work:
            rx.extend_attn_q8(plan, pool.desc, pool.kv, dq, o, lse, ws, stream=s)
    torch.cuda.synchronize()
    for i in range(2):
        check_extend(pool, q[i], work[i][3], work[i][4], prefix, new)
    plan, ws, dq, o, lse, _ = work[0]
    slots = np.concatenate([pool.table[r, prefix[r]:prefix[r] + new[r]] for r in range(2)])
    rows = [W.normal_bf16(rng, (290, 4, 128)) for _ in range(4)]
    dk, dv, ds = to_bf16(rows[0], cuda), to_bf16(rows[1], cuda), to_i32(slots, cuda)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        rx.store_kv_q8(pool.desc, pool.kv, dk, dv, ds)
        rx.extend_attn_q8(plan, pool.desc, pool.kv, dq, o, lse, ws)
    for k, v in (rows[:2], rows[2:]):
        dk.copy_(to_bf16(k, cuda))
        dv.copy_(to_bf16(v, cuda))
        o.fill_(7)
        g.replay()
        torch.cuda.synchronize()
        pool.kc[slots], pool.ks[slots] = Q.quantise(k)
        pool.vc[slots], pool.vs[slots] = Q.quantise(v)
        check_extend(pool, q[0], o, lse, prefix, new)


def test_one_plan_serves_every_layer(cuda):
    """The same plan and workspace over several pools, one call right behind the other."""
    rng = np.random.default_rng(84)
    lens, prefix, new = [400, 70, 900], [300, 20, 850], [100, 50, 50]
    pools = [Pool(cuda, rng, 8, 4, 1500, random_table(rng, 1500, lens)) for _ in range(3)]
    for pl in pools[1:]:  # one table for all layers
        pl.table, pl.r2t, pl.desc = pools[0].table, pools[0].r2t, pools[0].desc
    for kind in ("decode", "extend"):
        n = 3 if kind == "decode" else 200
        plan = rx.Plan()
        plan.set_kv_type(rx.RX_KV_E4M3)
        if kind == "decode":
            rx.decode_plan(plan, pools[0].desc, np.arange(3), lens)
        else:
            rx.extend_plan(plan, pools[0].desc, np.arange(3), prefix, new)
        ws = workspace(plan.workspace_size(), cuda)
        plan.upload(ws)
        q = [W.normal_bf16(rng, (n, 8, 128)) for _ in pools]
        dq = [to_bf16(x, cuda) for x in q]
        res = [(torch.empty((n, 8, 128), dtype=torch.bfloat16, device=cuda),
                torch.empty((n, 8), device=cuda)) for _ in pools]
        torch.cuda.synchronize()
        for pl, x, (o, lse) in zip(pools, dq, res):
            (rx.decode_attn_q8 if kind == "decode" else rx.extend_attn_q8)(
                plan, pl.desc, pl.kv, x, o, lse, ws)
        torch.cuda.synchronize()
        for pl, x, (o, lse) in zip(pools, q, res):
            if kind == "decode":
                check_decode(pl, x, o, lse, lens)
            else:
                check_extend(pl, x, o, lse, prefix, new)


def test_other_softmax_scales_and_many_heads(cuda):
    rng = np.random.default_rng(85)
    lens = [130, 61, 4]
    for hq, hkv, scale in ((8, 8, 0.3), (256, 256, 0.02), (144, 72, 128 ** -0.5)):
        pool = Pool(cuda, rng, hq, hkv, 260, random_table(rng, 260, lens))
        pool.scale = float(np.float32(scale))
        pool.desc = rx.kv_desc(hq, hkv, 260, pool.r2t, scale)
        q, o, lse, _, _ = run_decode(pool, rng, lens)
        check_decode(pool, q, o, lse, lens)
        q, o, lse, _ = run_extend(pool, rng, [100, 1, 0], [30, 60, 4])
        check_extend(pool, q, o, lse, [100, 1, 0], [30, 60, 4])


def test_a_batch_of_thousands_of_short_requests(cuda):
    rng = np.random.default_rng(86)
    lens = [int(x) for x in rng.integers(1, 40, 3000)]
    n = sum(lens) + 10
    pool = Pool(cuda, rng, 4, 2, n, random_table(rng, n, lens))
    q, o, lse, ws, _ = run_decode(pool, rng, lens)
    pick = [0, 1, 2, 1499, 2998, 2999] + [int(x) for x in rng.integers(0, 3000, 60)]
    check_decode(pool, q, o, lse, lens, pick)
    assert torch.isfinite(o.float()).all() and rx.read_status(ws) == rx.RX_OK


def test_calls_without_a_workspace_refuse_an_8_bit_plan(cuda):
    rng = np.random.default_rng(87)
    pool = Pool(cuda, rng, 8, 2, 64, random_table(rng, 64, [8]))
    plan = rx.Plan()
    plan.set_kv_type(rx.RX_KV_E4M3)
    rx.decode_plan(plan, pool.desc, [0], [8])
    with pytest.raises(rx.RxError) as e:
        rx.decode_attn_noalloc(plan, pool.desc, 4096, 4096, 4096, 4096, 4096)
    assert e.value.status == rx.RX_ERR_INVALID and "8-bit pool" in str(e.value)
